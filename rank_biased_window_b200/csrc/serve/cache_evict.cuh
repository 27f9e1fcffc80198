// cache_evict.cuh -- eviction by accumulated attention weight.
//
// Per sequence and head, of L tokens n = min(L, keep) stay: the last
// rec = min(recent, n), and of those before them the n - rec with the largest
// mass (ties: the lowest index; NaN ranks below everything), in their order.
//
// cache_select_kernel finds them: a radix selection over the masses as ordered
// integers (four 8-bit digits, one histogram per warp), then one ordered
// compaction.  cache_move_kernel moves the kept rows to the front, 32 at a
// time: a token never moves back, so a block may be written once the blocks up
// to it have been read, and every later block's rows lie behind it.  A block
// whose tokens all stay is left as it is; others get the scale of their own
// values.
#pragma once
#include "../sm100.cuh"
#include "e4m3.cuh"

namespace rfb {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveWarps = 8;

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
  int Hk, cap, to_cap, d, r, keep, recent, tensors, in_place;
};

// Order of the masses as integers: larger mass, larger key; NaN 0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t v = __float_as_uint(m + 0.0f);  // -0 to +0
  return (v & 0x80000000u) ? ~v : v | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[kSelWarps][256];
  __shared__ uint32_t total[256];
  __shared__ uint32_t s_prefix, s_want;
  __shared__ uint32_t w_keep[kSelWarps], w_tie[kSelWarps];
  grid_dep_wait();
  const int bh = blockIdx.x, b = bh / a.Hk;
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
  const int L = min(max(a.lengths[b], 0), a.cap);
  const int n = min(L, a.keep), rec = min(a.recent, n);
  const int older = L - rec, want = n - rec;
  int* kept = a.kept + static_cast<long long>(bh) * a.keep;
  if (bh == b * a.Hk && tid == 0) a.new_lengths[b] = n;
  for (int i = n + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  for (int i = tid; i < rec; i += kSelThreads) kept[want + i] = older + i;
  if (want == older) {  // nothing leaves
    for (int i = tid; i < older; i += kSelThreads) kept[i] = i;
    return;
  }
  if (want == 0) return;
  const float* mass = a.mass + static_cast<long long>(bh) * a.cap;

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
  if (lane == 0) w_keep[warp] = more, w_tie[warp] = ties;
  __syncthreads();
  uint32_t before_more = lane < warp ? w_keep[lane] : 0, before_tie = lane < warp ? w_tie[lane] : 0;
  before_more = __reduce_add_sync(0xffffffffu, before_more);
  before_tie = __reduce_add_sync(0xffffffffu, before_tie);
  uint32_t tie = before_tie, out = before_more + min(before_tie, left);
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? mass_key(mass[i]) : 0u;
    const bool is_tie = i < hi && k == prefix;
    const unsigned tm = __ballot_sync(0xffffffffu, is_tie);
    const bool stay = i < hi && (k > prefix || (is_tie && tie + __popc(tm & below) < left));
    const unsigned sm = __ballot_sync(0xffffffffu, stay);
    if (stay) kept[out + __popc(sm & below)] = i;
    out += __popc(sm);
    tie += __popc(tm);
  }
}

// One block's rows in registers: ITS pieces of P bytes a lane.
template <int P>
struct Piece;
template <>
struct Piece<16> {
  using T = uint4;
  static __device__ __forceinline__ uint32_t mag(const T& v) {
    const uint32_t m = __vmaxu4(__vmaxu4(finite_mag4(v.x), finite_mag4(v.y)),
                                __vmaxu4(finite_mag4(v.z), finite_mag4(v.w)));
    return max(max(m & 255u, (m >> 8) & 255u), max((m >> 16) & 255u, m >> 24));
  }
  static __device__ __forceinline__ T scaled(const T& v, float f) {
    return make_uint4(requantise4(v.x, f), requantise4(v.y, f), requantise4(v.z, f),
                      requantise4(v.w, f));
  }
};
template <>
struct Piece<8> {
  using T = uint2;
  static __device__ __forceinline__ uint32_t mag(const T& v) {
    const uint32_t m = __vmaxu4(finite_mag4(v.x), finite_mag4(v.y));
    return max(max(m & 255u, (m >> 8) & 255u), max((m >> 16) & 255u, m >> 24));
  }
  static __device__ __forceinline__ T scaled(const T& v, float f) {
    return make_uint2(requantise4(v.x, f), requantise4(v.y, f));
  }
};

// Moves 32 kept rows (src: this lane's, or -1) of one tensor into block j.
// `meet` separates the reads from the writes when the move is in place.
template <int P, int ITS, typename Meet>
__device__ __forceinline__ void move_rows(const uint8_t* from, const float* from_s, uint8_t* to,
                                          float* to_s, int cpr, int j, int src, bool active,
                                          Meet meet) {
  using T = typename Piece<P>::T;
  const int lane = lane_id();
  T v[ITS];
  float sc[ITS], own = 0.f, top = 0.f;
  if (active) {
    own = src >= 0 ? from_s[src / kCacheBlock] : 0.f;
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const int i = it * 32 + lane, row = min(i / cpr, 31);
      const int row_src = __shfl_sync(0xffffffffu, src, row);
      sc[it] = __shfl_sync(0xffffffffu, own, row);
      v[it] = T{};
      if (it < cpr && row_src >= 0)
        v[it] = *reinterpret_cast<const T*>(from + static_cast<long long>(row_src) * cpr * P +
                                            (i - row * cpr) * P);
    }
#pragma unroll
    for (int it = 0; it < ITS; ++it)
      top = fmaxf(top, f16x2_to_f32x2(e4m3_lo(Piece<P>::mag(v[it]))).x * sc[it]);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  }
  meet();
  if (active) {
    const float s = scale_for(top), inv = 1.0f / s;
    const int rows = __popc(__ballot_sync(0xffffffffu, src >= 0));
    uint8_t* out = to + static_cast<long long>(j) * kCacheBlock * cpr * P;
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const int i = it * 32 + lane;
      if (it < cpr && i < rows * cpr) {
        const float f = sc[it] * inv;
        reinterpret_cast<T*>(out)[i] = f == 1.0f ? v[it] : Piece<P>::scaled(v[it], f);
      }
    }
    if (lane == 0) to_s[j] = s;
  }
}

// Copies block j as it is (out of place).
template <int P>
__device__ __forceinline__ void copy_rows(const uint8_t* from, const float* from_s, uint8_t* to,
                                          float* to_s, int cpr, int j, int rows) {
  using T = typename Piece<P>::T;
  const long long at = static_cast<long long>(j) * kCacheBlock * cpr * P;
  for (int i = lane_id(); i < rows * cpr; i += 32)
    reinterpret_cast<T*>(to + at)[i] = reinterpret_cast<const T*>(from + at)[i];
  if (lane_id() == 0) to_s[j] = from_s[j];
}

// In place: one CTA a (sequence, head, tensor), kMoveWarps blocks a round, all
// reads of a round before its writes.  Out of place (gridDim.y parts): no order.
// Tensor index `tensors` is the mass.
template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) cache_move_kernel(const EvictArgs a) {
  grid_dep_wait();
  const int unit = blockIdx.x, bh = unit / (a.tensors + 1), z = unit - bh * (a.tensors + 1);
  const int b = bh / a.Hk, lane = lane_id(), warp = warp_id();
  const int n = min(min(max(a.lengths[b], 0), a.cap), a.keep);
  const int* kept = a.kept + static_cast<long long>(bh) * a.keep;
  const int blocks = (n + kCacheBlock - 1) / kCacheBlock;
  const int step = kMoveWarps * gridDim.y;
  const int rounds = (blocks + step - 1) / step;
  const int cpr = z == 2 ? a.r / 8 : D / 16, width = z == 2 ? a.r : D;
  const uint8_t* from = nullptr;
  const float* from_s = nullptr;
  uint8_t* to = nullptr;
  float* to_s = nullptr;
  if (z < a.tensors) {
    from = a.codes[z] + static_cast<long long>(bh) * a.cap * width;
    from_s = a.scales[z] + static_cast<long long>(bh) * (a.cap / kCacheBlock);
    to = a.to_codes[z] + static_cast<long long>(bh) * a.to_cap * width;
    to_s = a.to_scales[z] + static_cast<long long>(bh) * (a.to_cap / kCacheBlock);
  }
  const float* mass = a.mass + static_cast<long long>(bh) * a.cap;
  float* to_mass = a.to_mass + static_cast<long long>(bh) * a.to_cap;
  const auto meet = [&] {
    if (a.in_place) __syncthreads();
  };
  for (int round = 0; round < rounds; ++round) {
    const int j = round * step + blockIdx.y * kMoveWarps + warp;
    const int i = j * kCacheBlock + lane;
    const int src = i < n ? kept[i] : -1;
    const bool stays = __all_sync(0xffffffffu, src == i || src < 0);
    if (z == a.tensors) {
      const float m = src >= 0 ? mass[src] : 0.f;
      meet();
      if (src >= 0) to_mass[i] = m;
    } else {
      const bool active = j < blocks && !stays;
      if (j < blocks && stays && !a.in_place) {
        const int rows = __popc(__ballot_sync(0xffffffffu, src >= 0));
        if (z == 2)
          copy_rows<8>(from, from_s, to, to_s, cpr, j, rows);
        else
          copy_rows<16>(from, from_s, to, to_s, cpr, j, rows);
      }
      if (z == 2)
        move_rows<8, 8>(from, from_s, to, to_s, cpr, j, src, active, meet);
      else
        move_rows<16, D / 16>(from, from_s, to, to_s, D / 16, j, src, active, meet);
    }
  }
}

}  // namespace rfb
