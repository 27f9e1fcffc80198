// cache_append.cuh -- new rows of K, V (and the bias factor W) into the 8-bit
// cache.
//
// One warp (two at d = 128) owns one block of 32 tokens of one head and tensor, so
// a block's scale and codes have one writer and nothing is atomic: it takes the largest
// magnitude of the block's new rows, grows the scale if the rows before them
// have a smaller one (requantising those rows), and writes the new codes.
// Reads 2 bytes and writes 1 per element: bound by HBM for prompts (4 x 4001 tokens of 8
// heads, d = 128: 17.3 us, 5.6 TB/s), by the call for single tokens (3.8 us for 32 sequences).
#pragma once
#include "../sm100.cuh"
#include "e4m3.cuh"

namespace rfb {

constexpr int kAppendWarps = 8;

struct AppendArgs {
  const __nv_bfloat16* x[3];      // new k, v, w
  long long sb[3], sh[3], sn[3];  // strides in elements (rows of contiguous channels)
  uint8_t* codes[3];              // [B, Hk, cap, c]
  float* scales[3];               // [B, Hk, cap / 32]
  float* mass;                    // [B, Hk, cap] or null: zeroed for the new tokens
  const int* start;               // [B]
  const int* counts;              // [B] or null (all n)
  int Hk, n, cap, d, r, blocks, tensors;
};

// Larger magnitude of bf16 pairs, NaN ignored.
__device__ __forceinline__ uint32_t max_mag_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// CPR: 8-channel chunks of a row (0: r / 8, at most 8).  TEAM warps share the
// block, each with every TEAM-th run of 32 chunks: at d = 128 one warp would need
// 64 registers for its rows, which leaves too few warps to keep the loads going.
template <int CPR, int TEAM>
__device__ __forceinline__ void append_block(const AppendArgs& a, int z, int b, int h, int lo,
                                             int start, int end, uint32_t* exchange) {
  constexpr int ITS = (CPR ? CPR : 8) / TEAM;
  const int cpr = CPR ? CPR : a.r / 8;
  const int lane = lane_id(), warp = warp_id(), member = TEAM > 1 ? warp % TEAM : 0;
  const int c0 = member * 32 + lane;
  const __nv_bfloat16* x = a.x[z] + b * a.sb[z] + h * a.sh[z];
  uint4 v[ITS];
#pragma unroll
  for (int it = 0; it < ITS; ++it) {
    const int i = it * (32 * TEAM) + c0, row = i / cpr, t = lo + row;
    v[it] = make_uint4(0, 0, 0, 0);
    if (it < cpr && t >= start && t < end)
      v[it] = __ldg(reinterpret_cast<const uint4*>(x + (t - start) * a.sn[z] + (i - row * cpr) * 8));
  }
  uint32_t top = 0;
#pragma unroll
  for (int it = 0; it < ITS; ++it)
    top = max_mag_bf16x2(max_mag_bf16x2(max_mag_bf16x2(max_mag_bf16x2(top, v[it].x), v[it].y),
                                        v[it].z), v[it].w);
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  if (top >= 0x7f80u) {  // an infinity: it does not set the scale, so the rest once more
    top = 0;
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const uint32_t w[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = w[k] & 0x7fff7fffu;
        top = __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7f807f80u));
      }
    }
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  }
  if constexpr (TEAM > 1) {
    if (lane == 0) exchange[warp] = top;
    named_bar_sync(1 + warp / TEAM, 32 * TEAM);
    const uint32_t* team = exchange + warp / TEAM * TEAM;
#pragma unroll
    for (int k = 0; k < TEAM; ++k) top = max(top, team[k]);
  }
  const long long bh = static_cast<long long>(b) * a.Hk + h;
  float* sp = a.scales[z] + bh * (a.cap / kCacheBlock) + lo / kCacheBlock;
  uint8_t* codes = a.codes[z] + (bh * a.cap + lo) * (cpr * 8);
  float s = scale_for(__uint_as_float(top << 16));
  const int before = start - lo;  // rows of the block that are there already
  if (before > 0) {
    const float was = *sp;
    s = fmaxf(s, was);
    if (s != was) {
      const float ratio = was / s;
      for (int i = c0; i < before * cpr; i += 32 * TEAM) {
        uint2* p = reinterpret_cast<uint2*>(codes) + i;
        const uint2 c = *p;
        *p = make_uint2(requantise4(c.x, ratio), requantise4(c.y, ratio));
      }
    }
  }
  const float inv = 1.0f / s;
#pragma unroll
  for (int it = 0; it < ITS; ++it) {
    const int i = it * (32 * TEAM) + c0, row = i / cpr, t = lo + row;
    if (it < cpr && t >= start && t < end) {
      const uint32_t w[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = f32x2_to_e4m3x2(__uint_as_float(w[k] << 16) * inv,
                               __uint_as_float(w[k] & 0xffff0000u) * inv);
      reinterpret_cast<uint2*>(codes)[i] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
  }
  // every lane has read the old scale
  if constexpr (TEAM > 1)
    named_bar_sync(1 + warp / TEAM, 32 * TEAM);
  else
    __syncwarp();
  if (c0 == 0) *sp = s;
  if (z == 0 && a.mass != nullptr && member == 0) {
    const int t = lo + lane;
    if (t >= start && t < end) a.mass[bh * a.cap + t] = 0.0f;
  }
}

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_kernel(const AppendArgs a) {
  constexpr int TEAM = D / 64 > 1 ? D / 64 : 1;
  __shared__ uint32_t exchange[kAppendWarps];
  grid_dep_wait();
  const int warp = warp_id(), unit = (blockIdx.x * kAppendWarps + warp) / TEAM;
  const int j = unit / a.tensors, z = unit - j * a.tensors;
  if (j >= a.blocks) return;
  const int b = blockIdx.z, h = blockIdx.y;
  const int start = min(max(a.start[b], 0), a.cap);
  const int n = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  const int end = start + min(n, a.cap - start);  // rows beyond the capacity are dropped
  const long long lo = (static_cast<long long>(start / kCacheBlock) + j) * kCacheBlock;
  if (lo >= end || end == start) return;
  if (z == 2) {
    if (warp % TEAM == 0) append_block<0, 1>(a, z, b, h, static_cast<int>(lo), start, end, nullptr);
  } else {
    append_block<D / 8, TEAM>(a, z, b, h, static_cast<int>(lo), start, end, exchange);
  }
}

}  // namespace rfb
