// cache_evict.cuh -- eviction by accumulated attention weight.
//
// Per sequence and head, of L tokens n = min(L, keep) stay: the last
// rec = min(recent, n), and of those before them the n - rec with the largest
// mass (ties: the lowest index; NaN ranks below everything), in their order.
//
// A selection finds them: the threshold among the masses as ordered integers,
// then one ordered compaction.  cache_select_kernel holds the keys in registers
// (up to kSelMaxKeys a thread) and finds the threshold digit by digit, four of 8 bits,
// from histograms, a cluster of CTAs a (sequence, head) where these are few;
// cache_select_long_kernel reads the masses again for each digit.  cache_move_kernel moves the kept
// rows to the front, 32 at a time: a token never moves back, so a block may be
// written once the blocks up to it have been read, and every later block's rows
// lie behind it.  A block whose tokens all stay is left as it is; others get the
// scale of their own values.
//
// The move is bound by HBM, the selection by latency (a few thousand keys a CTA, four
// digits, a meeting of the cluster for each): 64 heads of up to 16384 tokens, d = 128, cut
// to 8192 take 55.7 us, of which the selection 13 (under ncu), and in place, where clusters
// of up to 8 CTAs meet each round, 61.5; 8 heads of 1000 tokens 9 us, in place 12.
#pragma once
#include "../sm100.cuh"
#include "e4m3.cuh"

namespace rfb {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxKeys = 32;  // keys a thread of cache_select_kernel holds
constexpr int kMoveWarps = 8;
constexpr int kMoveStages = 2;

struct EvictArgs {
  const uint8_t* codes[3];
  const float* scales[3];
  const float* mass;
  uint8_t* to_codes[3];
  float* to_scales[3];
  float* to_mass;
  const int* lengths;
  int* new_lengths;
  int* kept;  // [B, Hk, keep], -1 behind the last
  int heads, Hk, cap, to_cap, d, r, keep, recent, tensors, in_place;  // heads: B Hk
};

// Order of the masses as integers: larger mass, larger key; NaN 0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t v = __float_as_uint(m + 0.0f);  // -0 to +0
  return (v & 0x80000000u) ? ~v : v | 0x80000000u;
}

struct Selection {
  int older, want;  // of the first `older` tokens, the `want` of largest mass stay
  int* kept;
  const float* mass;
};
// Part `part` of `parts` CTAs on one (sequence, head): what is known without the
// masses is written here, the new length, the recent tokens, the tail; done:
// nothing is left to select.
__device__ __forceinline__ Selection select_begin(const EvictArgs& a, int bh, int part, int parts,
                                                  bool& done) {
  const int b = bh / a.Hk, tid = part * kSelThreads + threadIdx.x, step = parts * kSelThreads;
  const int L = min(max(a.lengths[b], 0), a.cap);
  const int n = min(L, a.keep), rec = min(a.recent, n);
  Selection s;
  s.older = L - rec, s.want = n - rec;
  s.kept = a.kept + static_cast<long long>(bh) * a.keep;
  s.mass = a.mass + static_cast<long long>(bh) * a.cap;
  if (bh == b * a.Hk && tid == 0) a.new_lengths[b] = n;
  for (int i = n + tid; i < a.keep; i += step) s.kept[i] = -1;
  for (int i = tid; i < rec; i += step) s.kept[s.want + i] = s.older + i;
  if (s.want == s.older)  // nothing leaves
    for (int i = tid; i < s.older; i += step) s.kept[i] = i;
  done = s.want == s.older || s.want == 0;
  return s;
}

// Exclusive prefix over the warps of (tokens above the threshold, ties).
__device__ __forceinline__ void before_warp(uint32_t (*count)[2], uint32_t more, uint32_t ties,
                                            uint32_t& before_more, uint32_t& before_tie) {
  const int lane = lane_id(), warp = warp_id();
  if (lane == 0) count[warp][0] = more, count[warp][1] = ties;
  __syncthreads();
  before_more = __reduce_add_sync(0xffffffffu, lane < warp ? count[lane][0] : 0u);
  before_tie = __reduce_add_sync(0xffffffffu, lane < warp ? count[lane][1] : 0u);
}

// Writes 32 tokens (key k, valid ok) of the ordered compaction.
__device__ __forceinline__ void compact_32(int* kept, int i, bool ok, uint32_t k, uint32_t threshold,
                                           uint32_t left, uint32_t& tie, uint32_t& out) {
  const uint32_t below = (1u << lane_id()) - 1u;
  const bool is_tie = ok && k == threshold;
  const unsigned tm = __ballot_sync(0xffffffffu, is_tie);
  const bool stay = ok && (k > threshold || (is_tie && tie + __popc(tm & below) < left));
  const unsigned sm = __ballot_sync(0xffffffffu, stay);
  if (stay) kept[out + __popc(sm & below)] = i;
  out += __popc(sm);
  tie += __popc(tm);
}

// One 8-bit digit of the threshold from its histogram (one warp): the prefix of
// the `left`-th largest key grows by the digit, left becomes its rank among the keys
// with it. Lane l holds bins 255 - 8 l .. 248 - 8 l.
__device__ __forceinline__ void next_digit(const uint32_t* bins, int shift, uint32_t& prefix,
                                           uint32_t& left) {
  const int lane = lane_id();
  const uint4 hi = *reinterpret_cast<const uint4*>(bins + 252 - 8 * lane);
  const uint4 lo = *reinterpret_cast<const uint4*>(bins + 248 - 8 * lane);
  const uint32_t own[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += own[i];
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  uint32_t above = incl - sum, digit = 0, rank = 0;
  const bool here = above < left && left <= incl;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (here && above < left && left <= above + own[i]) digit = 255 - 8 * lane - i, rank = left - above;
    above += own[i];
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  prefix |= __shfl_sync(0xffffffffu, digit, from) << shift;
  left = __shfl_sync(0xffffffffu, rank, from);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, int rank) {
  uint32_t at, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// A cluster of `parts` CTAs a (sequence, head), each with a stretch of its tokens,
// parts * KEYS * kSelThreads >= cap: a thread holds its keys.  Each digit's
// histogram is summed over the cluster through distributed shared memory.
template <int KEYS>
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const EvictArgs a, int parts) {
  __shared__ __align__(16) uint32_t hist[4][256];
  __shared__ __align__(16) uint32_t sum[256];
  __shared__ uint32_t count[kSelWarps][2];
  __shared__ uint32_t all[2], found[2];
  (&hist[0][0])[threadIdx.x] = 0;
  grid_dep_wait();
  const int bh = blockIdx.x / parts, part = blockIdx.x - bh * parts;
  bool done;
  const Selection s = select_begin(a, bh, part, parts, done);
  if (done) return;
  const int lane = lane_id(), warp = warp_id();
  // the CTA's stretch, and in it the warp's, so that the compaction is in order
  const int per_cta = (s.older + parts - 1) / parts;
  const int end = min((part + 1) * per_cta, s.older);
  const int per = ((per_cta + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int lo = min(part * per_cta + warp * per, end), hi = min(lo + per, end);
  float m[KEYS];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const int i = lo + 32 * k + lane;
    m[k] = i < hi ? __ldg(s.mass + i) : 0.f;
  }
  uint32_t key[KEYS];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) key[k] = mass_key(m[k]);
  __syncthreads();
  uint32_t prefix = 0, left = s.want;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int shift = 24 - 8 * p;
    if (p == 0) {
      // keys of few exponents share bins: those that agree with the warp's first go in one step
#pragma unroll
      for (int k = 0; k < KEYS; ++k) {
        if (lo + 32 * k < hi) {
          const bool ok = lo + 32 * k + lane < hi;
          const uint32_t d = key[k] >> 24, d0 = __shfl_sync(0xffffffffu, d, 0);
          const unsigned same = __ballot_sync(0xffffffffu, ok && d == d0);
          if (lane == 0) atomicAdd(&hist[0][d0], __popc(same));
          if (ok && d != d0) atomicAdd(&hist[0][d], 1u);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < KEYS; ++k)
        if (lo + 32 * k + lane < hi && ((key[k] ^ prefix) >> (shift + 8)) == 0)
          atomicAdd(&hist[p][(key[k] >> shift) & 255u], 1u);
    }
    const uint32_t* bins = hist[p];
    if (parts > 1) {
      cluster_sync();
      if (threadIdx.x < 256) {
        uint32_t n = 0;
        for (int c = 0; c < parts; ++c) n += cluster_load(&hist[p][threadIdx.x], c);
        sum[threadIdx.x] = n;
      }
      bins = sum;
    }
    __syncthreads();
    if (warp == 0) {
      next_digit(bins, shift, prefix, left);
      if (lane == 0) found[0] = prefix, found[1] = left;
    }
    __syncthreads();
    prefix = found[0];
    left = found[1];
  }
  uint32_t more = 0, ties = 0;
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const bool ok = lo + 32 * k + lane < hi;
    more += ok && key[k] > prefix;
    ties += ok && key[k] == prefix;
  }
  more = __reduce_add_sync(0xffffffffu, more);
  ties = __reduce_add_sync(0xffffffffu, ties);
  uint32_t before_more, tie;
  before_warp(count, more, ties, before_more, tie);
  if (parts > 1) {
    if (warp == 0) {
      const uint32_t n = __reduce_add_sync(0xffffffffu, count[lane][0]);
      const uint32_t e = __reduce_add_sync(0xffffffffu, count[lane][1]);
      if (lane == 0) all[0] = n, all[1] = e;
    }
    cluster_sync();
    for (int c = 0; c < part; ++c) {
      before_more += cluster_load(&all[0], c);
      tie += cluster_load(&all[1], c);
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // no CTA leaves while it is read
  }
  uint32_t out = before_more + min(tie, left);
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const int i = lo + 32 * k + lane;
    if (lo + 32 * k < hi) compact_32(s.kept, i, i < hi, key[k], prefix, left, tie, out);
  }
  if (parts > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__global__ void __launch_bounds__(kSelThreads) cache_select_long_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[kSelWarps][256];
  __shared__ uint32_t total[256];
  __shared__ uint32_t s_prefix, s_want;
  __shared__ uint32_t count[kSelWarps][2];
  grid_dep_wait();
  bool done;
  const Selection sel = select_begin(a, blockIdx.x, 0, 1, done);
  if (done) return;
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
  const int older = sel.older, want = sel.want;
  const float* mass = sel.mass;

  // threshold: the want-th largest key, digit by digit
  uint32_t prefix = 0, left = want;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kSelWarps * 256; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = tid; i < older; i += kSelThreads) {
      const uint32_t k = mass_key(mass[i]);
      if ((k & mask) == prefix) atomicAdd(&hist[warp][(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 256) {
      uint32_t s = 0;
      for (int w = 0; w < kSelWarps; ++w) s += hist[w][tid];
      total[tid] = s;
    }
    __syncthreads();
    if (warp == 0) {  // bins from the top: lane l holds bins 255 - 8 l .. 248 - 8 l
      uint32_t own[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += own[i] = total[255 - 8 * lane - i];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      uint32_t above = incl - sum;
      if (above < left && left <= incl) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < left && left <= above + own[i]) {
            s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
            s_want = left - above;
          }
          above += own[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_want;
  }

  // ordered compaction: warp w holds a stretch of the tokens
  const int per = ((older + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int lo = min(warp * per, older), hi = min(lo + per, older);
  uint32_t more = 0, ties = 0;
  for (int i = lo + lane; i < hi; i += 32) {
    const uint32_t k = mass_key(mass[i]);
    more += k > prefix;
    ties += k == prefix;
  }
  more = __reduce_add_sync(0xffffffffu, more);
  ties = __reduce_add_sync(0xffffffffu, ties);
  uint32_t before_more, tie;
  before_warp(count, more, ties, before_more, tie);
  uint32_t out = before_more + min(tie, left);
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? mass_key(mass[i]) : 0u;
    compact_32(sel.kept, i, i < hi, k, prefix, left, tie, out);
  }
}

// A piece of P bytes of a row.
template <int P>
struct Piece;
template <>
struct Piece<16> {
  using T = uint4;
  static __device__ __forceinline__ uint32_t mag(const T& v) {  // two fp16
    return max_mag_e4m3x4(max_mag_e4m3x4(max_mag_e4m3x4(max_mag_e4m3x4(0u, v.x), v.y), v.z), v.w);
  }
  static __device__ __forceinline__ T shifted(const T& v, __half2 f) {
    return make_uint4(shift_codes4(v.x, f), shift_codes4(v.y, f), shift_codes4(v.z, f),
                      shift_codes4(v.w, f));
  }
  static __device__ __forceinline__ T scaled(const T& v, float f) {
    return make_uint4(requantise4(v.x, f), requantise4(v.y, f), requantise4(v.z, f),
                      requantise4(v.w, f));
  }
  static __device__ __forceinline__ void fetch(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
};
template <>
struct Piece<8> {
  using T = uint2;
  static __device__ __forceinline__ uint32_t mag(const T& v) {
    return max_mag_e4m3x4(max_mag_e4m3x4(0u, v.x), v.y);
  }
  static __device__ __forceinline__ T shifted(const T& v, __half2 f) {
    return make_uint2(shift_codes4(v.x, f), shift_codes4(v.y, f));
  }
  static __device__ __forceinline__ T scaled(const T& v, float f) {
    return make_uint2(requantise4(v.x, f), requantise4(v.y, f));
  }
  static __device__ __forceinline__ void fetch(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  }
};

__host__ __device__ constexpr int move_stage_bytes(int d, int r) {
  return kCacheBlock * (d > r ? d : r);
}

// A warp's share of a move: items first + round * step.  In place an item is a
// block of tensor z0 of (sequence, head) bh0.  Out of place items run over the blocks
// of all sequences and heads, of tensor z0 and then z0 + 1; a warp takes every
// step-th, so that sequences shorter than `keep` do not leave some warps idle.
template <bool IN_PLACE>
struct MoveWalk {
  const EvictArgs& a;
  int z0, bh0;
  long long first, step, items;
  int rounds, per_head;
  struct At {
    int z, bh, block;
  };
  // Rounds behind the last item, which are looked at a round ahead (but have no source),
  // are held at the last one, so that every place names a tensor and a head that exist.
  __host__ __device__ __forceinline__ At at(int round) const {
    const long long on = first + round * step, item = on < items ? on : items - 1;
    if (IN_PLACE) return At{z0, bh0, static_cast<int>(item)};
    const unsigned head = static_cast<unsigned>(item / per_head);
    const int block = static_cast<int>(item - static_cast<long long>(head) * per_head);
    const bool second = head >= static_cast<unsigned>(a.heads);
    return At{z0 + second, static_cast<int>(head - (second ? a.heads : 0)), block};
  }
  // this lane's row for that round's block, or -1
  __device__ __forceinline__ int source(int round) const {
    if (first + round * step >= items) return -1;
    const At p = at(round);
    const int n = min(min(max(a.lengths[p.bh / a.Hk], 0), a.cap), a.keep);
    const int i = p.block * kCacheBlock + static_cast<int>(lane_id());
    return i < n ? a.kept[static_cast<long long>(p.bh) * a.keep + i] : -1;
  }
};

// Tensors of rows of PPR pieces of P bytes (0: ppr of them, at most 8).  The
// rows of the next kMoveStages - 1 rounds are on their way into shared memory
// while a round is written.
template <int P, int PPR, bool IN_PLACE, typename Meet>
__device__ __forceinline__ void move_rows(const MoveWalk<IN_PLACE>& w, int ppr,
                                          unsigned char* ring, int stage_bytes, Meet meet) {
  using T = typename Piece<P>::T;
  constexpr int ITS = PPR ? PPR : 8;
  constexpr int S = kMoveStages;
  if (PPR) ppr = PPR;
  const EvictArgs& a = w.a;
  const int lane = lane_id();
  const uint32_t base = smem_u32(ring);
  int src[S + 1];
  float own[S];
#pragma unroll
  for (int k = 0; k < S; ++k) src[k] = w.source(k);
  const auto fetch = [&](int round, int rows_src, float& scale) {
    const auto p = w.at(round);
    const uint8_t* from = a.codes[p.z] + static_cast<long long>(p.bh) * a.cap * (ppr * P);
    scale = 0.f;
    if (rows_src >= 0)
      scale = a.scales[p.z][static_cast<long long>(p.bh) * (a.cap / kCacheBlock) +
                            rows_src / kCacheBlock];
    const uint32_t dst = base + (round % S) * stage_bytes;
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const int i = it * 32 + lane, row = min(i / ppr, 31);
      const int r = __shfl_sync(0xffffffffu, rows_src, row);
      if (it < ppr && r >= 0)
        Piece<P>::fetch(dst + i * P, from + (static_cast<long long>(r) * ppr + (i - row * ppr)) * P);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch(k, src[k], own[k]);
  for (int round = 0; round < w.rounds; ++round) {
    fetch(round + S - 1, src[S - 1], own[S - 1]);
    src[S] = w.source(round + S);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    __syncwarp();
    const auto at = w.at(round);
    const int j = at.block;
    const bool stays = __all_sync(0xffffffffu, src[0] == j * kCacheBlock + lane || src[0] < 0);
    const int rows = __popc(__ballot_sync(0xffffffffu, src[0] >= 0));
    const T* v = reinterpret_cast<const T*>(ring + (round % S) * stage_bytes);
    float top = 0.f;
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const int i = it * 32 + lane;
      const float f = __shfl_sync(0xffffffffu, own[0], min(i / ppr, 31));
      if (it < ppr && i < rows * ppr) {
        const float2 m = f16x2_to_f32x2(Piece<P>::mag(v[i]));
        top = fmaxf(top, fmaxf(m.x, m.y) * f);
      }
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    meet();
    // a block whose tokens all stay keeps its scale (lane 0's)
    const float s = stays ? __shfl_sync(0xffffffffu, own[0], 0) : scale_for(top), inv = 1.0f / s;
    T* out = reinterpret_cast<T*>(a.to_codes[at.z] + (static_cast<long long>(at.bh) * a.to_cap +
                                                   static_cast<long long>(j) * kCacheBlock) *
                                                      (ppr * P));
    const bool write = rows > 0 && !(IN_PLACE && stays);
    // rows that keep their scale are copied; a ratio that is no power of two in
    // fp16's range (or no power of two at all) takes the way over fp32
    const float ratio = src[0] >= 0 && !stays ? own[0] * inv : 1.0f;
    const int k = (__float_as_int(ratio) >> 23) - 127;
    const bool odd = (__float_as_int(ratio) & 0x7fffff) != 0 || k < -14 || k > 15;
    if (write) {
      if (__all_sync(0xffffffffu, ratio == 1.0f)) {
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int i = it * 32 + lane;
          if (it < ppr && i < rows * ppr) out[i] = v[i];
        }
      } else if (!__any_sync(0xffffffffu, odd)) {
        const uint32_t mine = static_cast<uint32_t>(k + 15) << 10;  // 2^k as fp16, k = 15: 0x7800
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int i = it * 32 + lane;
          const uint32_t f = __shfl_sync(0xffffffffu, mine | (mine << 16), min(i / ppr, 31));
          if (it < ppr && i < rows * ppr)
            out[i] = Piece<P>::shifted(v[i], *reinterpret_cast<const __half2*>(&f));
        }
      } else {
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int i = it * 32 + lane;
          const float f = __shfl_sync(0xffffffffu, ratio, min(i / ppr, 31));
          if (it < ppr && i < rows * ppr) out[i] = f == 1.0f ? v[i] : Piece<P>::scaled(v[i], f);
        }
      }
    }
    if (lane == 0 && write)
      a.to_scales[at.z][static_cast<long long>(at.bh) * (a.to_cap / kCacheBlock) + j] = s;
    __syncwarp();  // the stage has been read
#pragma unroll
    for (int k = 0; k < S; ++k) src[k] = src[k + 1];
#pragma unroll
    for (int k = 0; k < S - 1; ++k) own[k] = own[k + 1];
  }
}

template <bool IN_PLACE, typename Meet>
__device__ __forceinline__ void move_mass(const MoveWalk<IN_PLACE>& w, Meet meet) {
  const EvictArgs& a = w.a;
  const auto load = [&](int round, int src) {
    return src >= 0 ? a.mass[static_cast<long long>(w.at(round).bh) * a.cap + src] : 0.f;
  };
  int src = w.source(0);
  float m = load(0, src);
  for (int round = 0; round < w.rounds; ++round) {
    const int next = w.source(round + 1);
    const float m_next = load(round + 1, next);
    meet();
    const auto at = w.at(round);
    if (src >= 0)
      a.to_mass[static_cast<long long>(at.bh) * a.to_cap + at.block * kCacheBlock + lane_id()] = m;
    src = next;
    m = m_next;
  }
}

// In place: blockIdx.x is (tensor, sequence, head), gridDim.y CTAs on each, a
// cluster, kMoveWarps blocks a CTA and round; all reads of a round come before
// its writes (rows of later rounds lie behind what is written, so they may be
// read ahead).  Out of place: blockIdx.y is 0 for K and V, 1 for the factors, 2 for
// the mass, whose warps share the blocks of all sequences and heads evenly.
template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveWarps * 32) cache_move_kernel(const EvictArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  grid_dep_wait();
  const int warp = warp_id(), stage = move_stage_bytes(D, a.r);
  unsigned char* ring = smem + warp * kMoveStages * stage;
  if constexpr (IN_PLACE) {
    const int z = blockIdx.x / a.heads, bh = blockIdx.x - z * a.heads;
    const int n = min(min(max(a.lengths[bh / a.Hk], 0), a.cap), a.keep);
    const int step = kMoveWarps * gridDim.y, items = (n + kCacheBlock - 1) / kCacheBlock;
    const MoveWalk<true> w{a,    z,     bh,
                           static_cast<long long>(blockIdx.y) * kMoveWarps + warp,
                           step, items, (items + step - 1) / step, items};
    const auto meet = [&] {
      if (gridDim.y == 1)
        __syncthreads();
      else
        cluster_sync();
    };
    if (z == a.tensors)
      move_mass<true>(w, meet);
    else if (z == 2)
      move_rows<8, 0, true>(w, a.r / 8, ring, stage, meet);
    else
      move_rows<16, D / 16, true>(w, D / 16, ring, stage, meet);
  } else {
    const int kind = blockIdx.y;
    if (kind == 1 && a.tensors == 2) return;  // no factors
    const int per_head = (a.keep + kCacheBlock - 1) / kCacheBlock;
    const long long items = static_cast<long long>(a.heads) * per_head * (kind == 0 ? 2 : 1);
    const long long first = static_cast<long long>(blockIdx.x) * kMoveWarps + warp;
    const long long step = static_cast<long long>(gridDim.x) * kMoveWarps;
    const int rounds = first < items ? static_cast<int>((items - first + step - 1) / step) : 0;
    const MoveWalk<false> w{a, kind == 1 ? 2 : 0, 0, first, step, items, rounds, per_head};
    const auto meet = [] {};
    if (kind == 2)
      move_mass<false>(w, meet);
    else if (kind == 1)
      move_rows<8, 0, false>(w, a.r / 8, ring, stage, meet);
    else
      move_rows<16, D / 16, false>(w, D / 16, ring, stage, meet);
  }
}

}  // namespace rfb
