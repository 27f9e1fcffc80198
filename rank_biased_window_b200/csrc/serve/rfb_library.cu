// rfb_library.cu -- the library's one translation unit: the attention entry
// points of rfb_attn.cu, and the host side of the serving operators (rotary
// positions, 8-bit cache append, attention over the cache, eviction), which
// share its error record, device queries and launch helpers.
#include "../rfb_attn.cu"

#include "cache_append.cuh"
#include "cache_attn.cuh"
#include "cache_evict.cuh"
#include "rotary.cuh"

namespace rfb {
namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// device_info() with the answer kept per thread: the short calls of a decode
// step come thousands of times a second from the same thread and device.
int current_device(DeviceInfo* out) {
  static thread_local DeviceInfo known;
  static thread_local int known_dev = -1;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, kSiteGetDevice);
  if (dev != known_dev) {
    if (int rc = device_info(&known)) return rc;
    known_dev = dev;
  }
  *out = known;
  return RFB_OK;
}

// ------------------------------------------------------------------ rotary
template <typename T, bool HALF, bool VEC>
int launch_rotary(RotArgs& a, int B, int sms, cudaStream_t st) {
  const int pairs = !VEC ? 1 : HALF ? Rot<T>::VEC : Rot<T>::VEC / 2;
  a.units = a.rot / (2 * pairs) + (a.d - a.rot) / (VEC ? Rot<T>::VEC : 1);
  // One thread per unit and group of heads.  More heads a thread share the
  // sine and cosine; fewer fill the chip: halve the group until there are 512
  // threads an SM (below that the call is latency, and one head is shortest).  One head a
  // thread: 103 us for 47 at 2 x 16384 tokens, 14.6 for 9.6 at 4097 of 16 fp32 heads; all
  // heads: 10.0 for 9.6 there, 6.2 for 5.9 at 512 tokens of 16 heads.
  const int heads = a.heads[0] + a.heads[1];
  const double units = static_cast<double>(B) * a.N * a.units;
  int per = heads;
  while (per > 1 && units * ((heads + per - 1) / per) < 512.0 * sms) per = (per + 1) / 2;
  a.heads_per_thread = per;
  const long long blocks =
      (static_cast<long long>(a.N) * a.units + kRotThreads - 1) / kRotThreads;
  const int groups = (heads + per - 1) / per;
  if (blocks * kRotThreads > 0xffffffffLL || B > 65535 || groups > 65535)
    return RFB_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), groups, B);
  launch_pdl(rotary_kernel<T, HALF, VEC>, grid, dim3(kRotThreads), 0, st, a);
  return launch_status();
}

template <typename T>
int dispatch_rotary(RotArgs& a, int B, bool half, int sms, cudaStream_t st) {
  constexpr int V = Rot<T>::VEC;
  bool vec = a.d % V == 0 && a.rot % (half ? 2 * V : V) == 0;
  for (int z = 0; z < 2; ++z)
    vec = vec && (a.heads[z] == 0 || (aligned16(a.x[z]) && aligned16(a.y[z]) &&
                                      a.sb[z] % V == 0 && a.sh[z] % V == 0 && a.sn[z] % V == 0));
  if (half)
    return vec ? launch_rotary<T, true, true>(a, B, sms, st)
               : launch_rotary<T, true, false>(a, B, sms, st);
  return vec ? launch_rotary<T, false, true>(a, B, sms, st)
             : launch_rotary<T, false, false>(a, B, sms, st);
}

// ------------------------------------------------------------------- cache
// Sizes shared by the cache entry points.  RFB_OK with *empty set when there
// is no head, row or token to work on.
int check_cache(int B, int heads_kv, int cap, int d, int r) {
  if (B < 0 || heads_kv < 0 || cap < 0 || d < 0 || r < 0) return RFB_ERR_INVALID_ARG;
  if (d != 32 && d != 64 && d != 128) return RFB_ERR_UNSUPPORTED;
  if (r > 64 || r % 8 != 0 || cap % kCacheBlock != 0) return RFB_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * heads_kv > 0x7fffffffLL / 4) return RFB_ERR_UNSUPPORTED;
  return RFB_OK;
}

// Row tiles and CTAs of the attention over the cache.
struct CaPlan {
  int tile, wr, row_segs, seg_rows, ctas, stages, smem, whole;
  size_t ml_bytes, o_bytes, score_bytes;
};

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

CaPlan plan_cache_attn(int B, int Hk, int R, int cap, int d, int r, bool mass, int sms) {
  CaPlan p;
  // Up to 8 rows in a tile of 16 would be half empty: 51.2 us for 35.2 (4 rows, d = 128).
  p.tile = R <= 8 ? 8 : 16;
  const int tiles = (R + p.tile - 1) / p.tile;
  p.wr = tiles >= 3 ? 4 : tiles;
  p.row_segs = (tiles + p.wr - 1) / p.wr;
  p.seg_rows = R < p.tile * p.wr ? R : p.tile * p.wr;
  // One wave of resident CTAs, fewer when that would leave warps without a block.
  const long long blocks = static_cast<long long>(B) * Hk * p.row_segs * (cap / kCacheBlock);
  const int wts = kCaWarps / p.wr;
  const long long most = (blocks + wts - 1) / wts;
  // Three CTAs share an SM's 227 KB (1 KB of each is the system's), or two where
  // three would leave a group of warps a single stage.
  const int stage = kCacheBlock * (2 * d + r);
  const auto fit = [&](int n) { return (227 * 1024 / n - 1024 - kCaRing) / (stage * wts); };
  const int resident = fit(3) >= 2 ? 3 : 2;
  const int wave = sms * resident;
  p.stages = fit(resident) < kCaMaxStages ? fit(resident) : kCaMaxStages;
  p.smem = kCaRing + p.stages * stage * wts;
  p.ctas = static_cast<int>(most < wave ? (most > 0 ? most : 1) : wave);
  // A CTA a segment, which needs no join of partials and lets the hardware even out the
  // CTAs: for short contexts and for segments that fill several waves.  Measured over
  // 0.02 to 8 waves of segments (1 to 450 sequences of 8 heads, d = 64): up to four blocks a
  // group of warps always (16 sequences to 128 tokens 6.2 us for 13.0, one of 500 tokens 7.5 for
  // 11.6, of 1000 11.0 for 9.3), else up to 16 for each wave of segments (450 sequences to 4096
  // tokens 207 us for 260, 225 to 1024 42 for 56, but 28 to 2048 21.9 for 17.3).  The same with
  // the mass, whose second kernel runs in any case (112 sequences to 512 tokens 20.3 us for
  // 25.8, one of 500 10.7 for 9.8), so that O and LSE do not depend on it.  By the capacity: the
  // lengths are on the device, so a short context in a large cache is cut all the same.
  const long long segs = static_cast<long long>(B) * Hk * p.row_segs;
  const long long group = (cap / kCacheBlock + wts - 1) / wts;
  p.whole = group <= 4 || group * wave <= 16 * segs;
  if (p.whole) p.ctas = static_cast<int>(segs);
  const size_t parts = p.whole ? 0 : static_cast<size_t>(p.ctas) * 2 * p.seg_rows;
  p.ml_bytes = round256(parts * sizeof(float2) + 1);
  p.o_bytes = round256(parts * d * sizeof(float));
  p.score_bytes = mass && p.tile == 8 ? static_cast<size_t>(B) * Hk * R * cap * sizeof(float) : 0;
  return p;
}

constexpr int kCaMaxSmem = 227 * 1024 / 2 - 1024;

template <int D, int RP, int QT, bool MASS>
int launch_cache_attn_main(const CacheAttnArgs& a, const CaPlan& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (int rc = ensure_smem(cache_attn_kernel<D, RP, QT, MASS>, kCaMaxSmem, done)) return rc;
  launch_pdl(cache_attn_kernel<D, RP, QT, MASS>, dim3(p.ctas), dim3(kCaThreads), p.smem, st, a);
  return launch_status();
}

template <int D, int RP>
int launch_cache_attn(const CacheAttnArgs& a, const CaPlan& p, cudaStream_t st) {
  const int rc = p.tile == 16 ? launch_cache_attn_main<D, RP, 2, false>(a, p, st)
                 : a.scores   ? launch_cache_attn_main<D, RP, 1, true>(a, p, st)
                              : launch_cache_attn_main<D, RP, 1, false>(a, p, st);
  if (rc != RFB_OK) return rc;
  const unsigned segs = static_cast<unsigned>(a.B * a.Hk * a.row_segs);
  const unsigned ctas = static_cast<unsigned>(p.ctas), partials = (ctas + segs - 1) / segs;
  const int per = join_rows(p.seg_rows, D, partials), row_sets = (p.seg_rows + per - 1) / per;
  const bool again = a.mass_out && !a.scores && a.cap > 0;  // recompute the weights
  const int again_chunks = (a.cap + kMassChunk - 1) / kMassChunk;
  if (again && per > 1 && !a.whole) {
    launch_pdl(cache_attn_combine_kernel<D, RP>, dim3(segs, row_sets + again_chunks), dim3(128), 0,
               st, a, ctas, per, row_sets);
    return launch_status();
  }
  const int chunks = a.scores ? (a.cap + mass_tokens(a.R) - 1) / mass_tokens(a.R) : 0;
  const int joins = a.whole ? 0 : row_sets;
  if (joins + chunks > 0)
    launch_pdl(cache_attn_combine_kernel<D, -1>, dim3(segs, joins + chunks), dim3(128), 0, st, a,
               ctas, per, joins);
  if (again)
    launch_pdl(cache_mass_kernel<D, RP>, dim3(static_cast<unsigned>(a.B * a.Hk), again_chunks),
               dim3(128), 0, st, a);
  return launch_status();
}

template <int D>
int dispatch_cache_attn(const CacheAttnArgs& a, const CaPlan& p, cudaStream_t st) {
  switch (pad_rank(a.r)) {
    case 0: return launch_cache_attn<D, 0>(a, p, st);
    case 16: return launch_cache_attn<D, 16>(a, p, st);
    case 32: return launch_cache_attn<D, 32>(a, p, st);
    default: return launch_cache_attn<D, 64>(a, p, st);
  }
}

// Launch with programmatic serialisation and, where cx * cy > 1, in clusters.
template <typename... KArgs, typename... Args>
void launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, unsigned cx,
                    unsigned cy, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cx;
  attr[1].val.clusterDim.y = cy;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cx * cy > 1 ? 2 : 1;
  (void)cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int KEYS>
int launch_select(const EvictArgs& a, int parts, cudaStream_t st) {
  launch_cluster(cache_select_kernel<KEYS>, dim3(a.heads * parts), dim3(kSelThreads), 0, parts, 1,
                 st, a, parts);
  return launch_status();
}

// The move after an eviction.
template <int D>
int launch_move(const EvictArgs& a, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done[2];
  constexpr int kMost = kMoveWarps * kMoveStages * move_stage_bytes(D, 64);
  const int stage = move_stage_bytes(D, a.r), smem = kMoveWarps * kMoveStages * stage;
  const dim3 block(kMoveWarps * 32);
  const int wave = sms * (227 * 1024 / (smem + 1024) < 8 ? 227 * 1024 / (smem + 1024) : 8);
  const int rows_cta = kCacheBlock * kMoveWarps;
  if (a.in_place) {
    if (int rc = ensure_smem(cache_move_kernel<D, true>, kMost, done[0])) return rc;
    // clusters as large as one wave of CTAs (the mass's are short) and the blocks allow
    int c = 1;
    while (c < 8 && 2 * c * a.heads * a.tensors <= wave && c * rows_cta < a.keep) c *= 2;
    launch_cluster(cache_move_kernel<D, true>, dim3(a.heads * (a.tensors + 1), c), block, smem, 1, c,
                   st, a);
  } else {
    if (int rc = ensure_smem(cache_move_kernel<D, false>, kMost, done[1])) return rc;
    const long long most = 2LL * a.heads * ((a.keep + rows_cta - 1) / rows_cta);
    launch_pdl(cache_move_kernel<D, false>,
               dim3(static_cast<unsigned>(most < wave ? most : wave), 3), block, smem, st, a);
  }
  return launch_status();
}

}  // namespace
}  // namespace rfb

using namespace rfb;

extern "C" {

int rfb_rotary(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
               const double* freqs, int B, int heads, int heads_kv, int N, int d, int rot,
               const long long* q_strides, const long long* k_strides, long long position_stride,
               int layout, int dtype, float amplitude, int inverse, void* stream) {
  if (B < 0 || heads < 0 || heads_kv < 0 || N < 0 || d < 0 || rot < 0) return RFB_ERR_INVALID_ARG;
  if ((layout != 0 && layout != 1) || dtype < 0 || dtype > 2 || !std::isfinite(amplitude) ||
      position_stride < 0)
    return RFB_ERR_INVALID_ARG;
  if (rot % 2 != 0 || rot > d || d > 1024 || heads > 65535 || heads_kv > 65535)
    return RFB_ERR_UNSUPPORTED;
  if (B == 0 || N == 0 || d == 0 || heads + heads_kv == 0) return RFB_OK;
  if ((heads > 0 && (!q || !q_out || !q_strides)) ||
      (heads_kv > 0 && (!k || !k_out || !k_strides)) || !positions || (rot > 0 && !freqs))
    return RFB_ERR_INVALID_ARG;
  const size_t elem = dtype == 2 ? 4 : 2;
  if (!aligned_to(q, elem) || !aligned_to(k, elem) || !aligned_to(q_out, elem) ||
      !aligned_to(k_out, elem) || !aligned_to(positions, 4) || !aligned_to(freqs, 8))
    return RFB_ERR_ALIGNMENT;
  DeviceInfo dev;
  if (int rc = current_device(&dev)) return rc;
  RotArgs a = {};
  a.x[0] = q, a.x[1] = k;
  a.y[0] = q_out, a.y[1] = k_out;
  a.heads[0] = heads, a.heads[1] = heads_kv;
  for (int z = 0; z < 2; ++z) {
    const long long* s = z ? k_strides : q_strides;
    if (a.heads[z] == 0) continue;
    a.sb[z] = s[0], a.sh[z] = s[1], a.sn[z] = s[2];
  }
  a.pos = positions;
  a.freq = freqs;
  a.pos_sb = position_stride;
  a.N = N, a.d = d, a.rot = rot;
  a.amp = amplitude;
  a.sign = inverse ? -1.f : 1.f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool half = layout == 0;
  if (dtype == 0) return dispatch_rotary<__nv_bfloat16>(a, B, half, dev.sms, st);
  if (dtype == 1) return dispatch_rotary<__half>(a, B, half, dev.sms, st);
  return dispatch_rotary<float>(a, B, half, dev.sms, st);
}

int rfb_cache_append(const void* k, const void* v, const void* w, const long long* strides,
                     void* k8, void* v8, void* w8, float* k_scale, float* v_scale, float* w_scale,
                     float* mass, const int* start, const int* counts, int B, int heads_kv, int n,
                     int cap, int d, int r, void* stream) {
  if (n < 0) return RFB_ERR_INVALID_ARG;
  if (int rc = check_cache(B, heads_kv, cap, d, r)) return rc;
  if (B > 65535 || heads_kv > 65535) return RFB_ERR_UNSUPPORTED;
  if (B == 0 || heads_kv == 0 || n == 0 || cap == 0) return RFB_OK;
  if (!k || !v || !k8 || !v8 || !k_scale || !v_scale || !start || !strides ||
      (r > 0 && (!w || !w8 || !w_scale)))
    return RFB_ERR_INVALID_ARG;
  AppendArgs a = {};
  const void* x[3] = {k, v, w};
  void* c[3] = {k8, v8, w8};
  float* s[3] = {k_scale, v_scale, w_scale};
  a.tensors = r > 0 ? 3 : 2;
  for (int z = 0; z < a.tensors; ++z) {
    if (!aligned16(x[z]) || !aligned16(c[z]) || !aligned_to(s[z], 4)) return RFB_ERR_ALIGNMENT;
    a.x[z] = static_cast<const __nv_bfloat16*>(x[z]);
    a.codes[z] = static_cast<uint8_t*>(c[z]);
    a.scales[z] = s[z];
    a.sb[z] = strides[3 * z], a.sh[z] = strides[3 * z + 1], a.sn[z] = strides[3 * z + 2];
    if (a.sb[z] % 8 || a.sh[z] % 8 || a.sn[z] % 8) return RFB_ERR_ALIGNMENT;
  }
  if (!aligned_to(mass, 4) || !aligned_to(start, 4) || !aligned_to(counts, 4)) return RFB_ERR_ALIGNMENT;
  a.mass = mass;
  a.start = start;
  a.counts = counts;
  a.Hk = heads_kv, a.n = n, a.cap = cap, a.d = d, a.r = r;
  a.blocks = static_cast<int>((static_cast<long long>(n) + kCacheBlock - 2) / kCacheBlock) + 1;
  if (a.blocks > cap / kCacheBlock) a.blocks = cap / kCacheBlock;
  DeviceInfo dev;
  if (int rc = current_device(&dev)) return rc;
  const long long units = static_cast<long long>(a.blocks) * a.tensors * (d > 64 ? 2 : 1);  // warps
  const dim3 grid(static_cast<unsigned>((units + kAppendWarps - 1) / kAppendWarps), heads_kv, B);
  const dim3 block(kAppendWarps * 32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 32) launch_pdl(cache_append_kernel<32>, grid, block, 0, st, a);
  else if (d == 64) launch_pdl(cache_append_kernel<64>, grid, block, 0, st, a);
  else launch_pdl(cache_append_kernel<128>, grid, block, 0, st, a);
  return launch_status();
}

size_t rfb_attn_fwd_cache_workspace_size(int B, int heads, int heads_kv, int Nq, int cap, int d,
                                         int with_mass) {
  if (check_cache(B, heads_kv, cap, d, 0) || heads_kv == 0 || heads < 0 || Nq < 0 ||
      heads % heads_kv != 0)
    return 0;
  const long long R = static_cast<long long>(heads / heads_kv) * Nq;
  if (B == 0 || R == 0 || R > 0x7fffffffLL) return 0;
  DeviceInfo dev;
  if (current_device(&dev)) return 0;
  // r = 0 needs the most: factors make stages larger, waves smaller, and a CTA a segment likelier
  const CaPlan p = plan_cache_attn(B, heads_kv, static_cast<int>(R), cap, d, 0, with_mass != 0, dev.sms);
  return p.ml_bytes + p.o_bytes + p.score_bytes;
}

int rfb_attn_fwd_cache(const void* q, const void* u, const void* k8, const void* v8, const void* w8,
                       const float* k_scale, const float* v_scale, const float* w_scale,
                       const int* lengths, const float* mass, float* mass_out, float decay, void* o,
                       float* lse, void* workspace, size_t workspace_bytes, int B, int heads,
                       int heads_kv, int Nq, int cap, int d, int r, float scale, int causal,
                       void* stream) {
  return rfb_attn_fwd_cache_counts(q, u, k8, v8, w8, k_scale, v_scale, w_scale, lengths, nullptr,
                                   mass, mass_out, decay, o, lse, workspace, workspace_bytes, B,
                                   heads, heads_kv, Nq, cap, d, r, scale, causal, stream);
}

int rfb_attn_fwd_cache_counts(const void* q, const void* u, const void* k8, const void* v8,
                              const void* w8, const float* k_scale, const float* v_scale,
                              const float* w_scale, const int* lengths, const int* counts,
                              const float* mass, float* mass_out, float decay, void* o, float* lse,
                              void* workspace, size_t workspace_bytes, int B, int heads,
                              int heads_kv, int Nq, int cap, int d, int r, float scale, int causal,
                              void* stream) {
  if (heads < 0 || Nq < 0 || !std::isfinite(scale) || !(scale > 0.f) || !std::isfinite(decay))
    return RFB_ERR_INVALID_ARG;
  if (int rc = check_cache(B, heads_kv, cap, d, r)) return rc;
  if (B == 0 || ((heads == 0 || Nq == 0) && (!mass_out || heads_kv == 0 || cap == 0))) return RFB_OK;
  if (heads_kv == 0 || heads % heads_kv != 0) return RFB_ERR_INVALID_ARG;
  const long long R = static_cast<long long>(heads / heads_kv) * Nq;
  if (R == 0) {
    if (cap > 65535 * 128) return RFB_ERR_UNSUPPORTED;
    if (!lengths) return RFB_ERR_INVALID_ARG;
    if (!aligned_to(mass, 4) || !aligned_to(mass_out, 4) || !aligned_to(lengths, 4))
      return RFB_ERR_ALIGNMENT;
    CacheAttnArgs a = {};
    a.lengths = lengths;
    a.mass = mass, a.mass_out = mass_out, a.decay = decay;
    a.Hk = heads_kv, a.cap = cap;
    launch_pdl(cache_decay_kernel, dim3(static_cast<unsigned>(B * heads_kv), (cap + 127) / 128),
               dim3(128), 0, static_cast<cudaStream_t>(stream), a);
    return launch_status();
  }
  if (R > (1LL << 24) || static_cast<long long>(B) * heads_kv * ((R + 7) / 8) > 0x7fffffffLL / (cap / kCacheBlock + 8) ||
      (mass_out && cap > 65000 * 128))
    return RFB_ERR_UNSUPPORTED;
  if (!q || !o || !lse || !lengths || (r > 0 && !u) ||
      (cap > 0 && (!k8 || !v8 || !k_scale || !v_scale || (r > 0 && (!w8 || !w_scale)))))
    return RFB_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(u) || !aligned16(k8) || !aligned16(v8) || !aligned16(w8) ||
      !aligned16(o) || !aligned_to(lse, 4) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) ||
      !aligned_to(w_scale, 4) || !aligned_to(mass, 4) || !aligned_to(mass_out, 4) ||
      !aligned_to(lengths, 4) || !aligned_to(counts, 4))
    return RFB_ERR_ALIGNMENT;
  DeviceInfo dev;
  if (int rc = current_device(&dev)) return rc;
  const CaPlan p = plan_cache_attn(B, heads_kv, static_cast<int>(R), cap, d, r,
                                   mass_out != nullptr, dev.sms);
  if (!workspace || workspace_bytes < p.ml_bytes + p.o_bytes + p.score_bytes)
    return RFB_ERR_WORKSPACE;
  if (!aligned16(workspace)) return RFB_ERR_ALIGNMENT;
  CacheAttnArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.u = static_cast<const __nv_bfloat16*>(u);
  a.k = static_cast<const uint8_t*>(k8);
  a.v = static_cast<const uint8_t*>(v8);
  a.w = static_cast<const uint8_t*>(w8);
  a.ks = k_scale, a.vs = v_scale, a.ws = w_scale;
  a.lengths = lengths;
  a.counts = counts;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + p.ml_bytes);
  a.scores = p.score_bytes ? reinterpret_cast<float*>(ws + p.ml_bytes + p.o_bytes) : nullptr;
  a.mass = mass, a.mass_out = mass_out, a.decay = decay;
  a.B = B, a.Hk = heads_kv, a.R = static_cast<int>(R), a.Nq = Nq, a.cap = cap, a.r = r;
  a.tile = p.tile, a.wr = p.wr, a.row_segs = p.row_segs;
  a.causal = causal;
  a.whole = p.whole;
  a.stages = p.stages;
  a.err_word = dev.err_word;
  a.wait_ns = g_wait_limit_ns.load();
  a.fail_site = g_fail_site.load();
  a.scale_log2 = scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 32   ? dispatch_cache_attn<32>(a, p, st)
         : d == 64 ? dispatch_cache_attn<64>(a, p, st)
                   : dispatch_cache_attn<128>(a, p, st);
}

int rfb_cache_evict(const void* k8, const void* v8, const void* w8, const float* k_scale,
                    const float* v_scale, const float* w_scale, const float* mass, void* k8_out,
                    void* v8_out, void* w8_out, float* k_scale_out, float* v_scale_out,
                    float* w_scale_out, float* mass_out, const int* lengths, int* new_lengths,
                    int* kept, int B, int heads_kv, int cap, int cap_out, int d, int r, int keep,
                    int recent, void* stream) {
  if (keep < 1 || recent < 0 || cap_out < 0) return RFB_ERR_INVALID_ARG;
  if (int rc = check_cache(B, heads_kv, cap, d, r)) return rc;
  if (cap_out % kCacheBlock != 0) return RFB_ERR_UNSUPPORTED;
  if (keep > cap_out) return RFB_ERR_INVALID_ARG;
  if (B == 0 || heads_kv == 0) return RFB_OK;
  const void* c[3] = {k8, v8, w8};
  void* co[3] = {k8_out, v8_out, w8_out};
  const float* s[3] = {k_scale, v_scale, w_scale};
  float* so[3] = {k_scale_out, v_scale_out, w_scale_out};
  EvictArgs a = {};
  a.tensors = r > 0 ? 3 : 2;
  int same = 0;
  for (int z = 0; z < a.tensors; ++z) {
    if (!c[z] || !co[z] || !s[z] || !so[z]) return RFB_ERR_INVALID_ARG;
    if (!aligned16(c[z]) || !aligned16(co[z]) || !aligned_to(s[z], 4) || !aligned_to(so[z], 4))
      return RFB_ERR_ALIGNMENT;
    same += (c[z] == co[z]) + (s[z] == so[z]);
    a.codes[z] = static_cast<const uint8_t*>(c[z]);
    a.to_codes[z] = static_cast<uint8_t*>(co[z]);
    a.scales[z] = s[z];
    a.to_scales[z] = so[z];
  }
  if (!mass || !mass_out || !lengths || !new_lengths || !kept || lengths == new_lengths)
    return RFB_ERR_INVALID_ARG;
  if (!aligned_to(mass, 4) || !aligned_to(mass_out, 4) || !aligned_to(lengths, 4) ||
      !aligned_to(new_lengths, 4) || !aligned_to(kept, 4))
    return RFB_ERR_ALIGNMENT;
  same += mass == mass_out;
  const int all = 2 * a.tensors + 1;
  if (same != 0 && (same != all || cap != cap_out)) return RFB_ERR_INVALID_ARG;  // all or none
  a.in_place = same == all;
  a.mass = mass;
  a.to_mass = mass_out;
  a.lengths = lengths;
  a.new_lengths = new_lengths;
  a.kept = kept;
  a.heads = B * heads_kv, a.Hk = heads_kv, a.cap = cap, a.to_cap = cap_out, a.d = d, a.r = r;
  a.keep = keep, a.recent = recent;
  DeviceInfo dev;
  if (int rc = current_device(&dev)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int bh = B * heads_kv;
  // A cluster of CTAs a (sequence, head) while that leaves SMs without one and
  // each CTA a few thousand tokens, or where the keys of one do not fit (8 heads of 65536
  // tokens: 60.6 us by one CTA each, 18.4 by eight; of 1024: 9.8 by one, 12.4 by eight).
  int parts = 1;
  while (parts < 8 && ((2 * parts * bh <= dev.sms && cap > 2048 * parts) ||
                       cap > parts * kSelMaxKeys * kSelThreads))
    parts *= 2;
  const int held = (cap + parts * kSelThreads - 1) / (parts * kSelThreads);
  int rc = held <= 2    ? launch_select<2>(a, parts, st)
           : held <= 8  ? launch_select<8>(a, parts, st)
           : held <= 16 ? launch_select<16>(a, parts, st)
           : held <= kSelMaxKeys ? launch_select<kSelMaxKeys>(a, parts, st)
                                 : RFB_ERR_UNSUPPORTED;
  if (held > kSelMaxKeys) {
    launch_pdl(cache_select_long_kernel, dim3(bh), dim3(kSelThreads), 0, st, a);
    rc = launch_status();
  }
  if (rc != RFB_OK) return rc;
  if (d == 32) return launch_move<32>(a, dev.sms, st);
  if (d == 64) return launch_move<64>(a, dev.sms, st);
  return launch_move<128>(a, dev.sms, st);
}

}  // extern "C"
