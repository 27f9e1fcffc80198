// rotary.cuh -- rotary positions on queries and keys, forward and backward.
//
// Pair i of a head (rot / 2 pairs; channels beyond rot pass through) turns by
// the angle t = pos f_i:  y1 = a (x1 cos t - x2 sin t),
// y2 = a (x2 cos t + x1 sin t).  The rotation is orthogonal up to a, so the
// backward is the same kernel with -t on the gradients.
//
// The angle is formed in turns in fp64 and reduced there (fp32 would lose the
// angle of far positions); sine and cosine of the remainder's fp32 value are turned by
// what that leaves (up to 2^-26 of a turn, more than fp32's rounding of a sine near 0);
// that work is done once per token and pair and used for every head of q and k the
// thread goes over.  One read and one write of q and k: bound by HBM (2 x 16384 tokens,
// 8 + 8 heads, d = 64, forward and backward: 47.6 us, 5.6 TB/s; 4097 tokens of 16 fp32
// heads, d = 128: 10.6 us, 6.3 TB/s).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../sm100.cuh"

namespace rfb {

constexpr int kRotThreads = 128;

struct RotArgs {
  const void* x[2];        // q, k
  void* y[2];              // contiguous [B, heads, N, d]
  int heads[2];
  long long sb[2], sh[2], sn[2];  // input strides in elements
  const int* pos;          // [B, N], batch stride pos_sb (0: shared)
  const double* freq;      // rot / 2 angles per position
  long long pos_sb;
  int N, d, rot, units, heads_per_thread;
  float amp, sign;
};

template <typename T>
struct Rot;  // 16-byte vectors of T as floats
template <>
struct Rot<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ void load(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float to(float v) { return v; }
};
template <>
struct Rot<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ void load(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 to(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Rot<__half> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ void load(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half to(float v) { return __float2half_rn(v); }
};

// a cos t, +-a sin t of t = pos f.
__device__ __forceinline__ void rot_angle(const RotArgs& a, int pos, int pair, float& c, float& s) {
  const double turns = static_cast<double>(pos) * a.freq[pair] * 0.15915494309189535;  // 1 / 2 pi
  const double part = turns - rint(turns);
  const float r = static_cast<float>(part);
  const float rest = static_cast<float>(part - r) * 6.2831853f;  // |rest| < 2^-23
  float s0, c0;
  sincospif(2.0f * r, &s0, &c0);
  c = fmaf(-s0, rest, c0) * a.amp;
  s = fmaf(c0, rest, s0) * (a.amp * a.sign);
}

// VEC_OK: 16-byte vectors.  A unit is, in the half layout, VEC pairs (one
// vector of each half of the rotated part); interleaved, one vector of VEC / 2
// pairs; beyond rot one vector copied.  Otherwise a unit is one pair or one
// copied channel (any even rot, any strides).
template <typename T, bool HALF, bool VEC_OK>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotArgs a) {
  using R = Rot<T>;
  constexpr int V = R::VEC;
  constexpr int PAIRS = !VEC_OK ? 1 : HALF ? V : V / 2;
  grid_dep_wait();
  const unsigned idx = blockIdx.x * kRotThreads + threadIdx.x;  // N * units < 2^32
  const unsigned n = idx / static_cast<unsigned>(a.units);
  if (n >= static_cast<unsigned>(a.N)) return;
  const int unit = static_cast<int>(idx - n * a.units);
  const int b = blockIdx.z;
  const int turning = a.rot / (2 * PAIRS);  // units that rotate
  const bool copy = unit >= turning;
  // channel of the unit's first element (and of its second part)
  const int c0 = copy ? a.rot + (unit - turning) * (VEC_OK ? V : 1)
                      : HALF ? unit * PAIRS : unit * PAIRS * 2;
  const int c1 = HALF ? c0 + a.rot / 2 : c0 + 1;
  float cs[PAIRS], sn[PAIRS];
  if (!copy) {
    const int pos = a.pos[b * a.pos_sb + n];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) rot_angle(a, pos, unit * PAIRS + i, cs[i], sn[i]);
  }
  const int h0 = blockIdx.y * a.heads_per_thread, h1 = h0 + a.heads_per_thread;
#pragma unroll 1
  for (int z = 0; z < 2; ++z) {  // the group's heads of q, then of k
    const int skip = z ? a.heads[0] : 0;
    const int from = max(h0 - skip, 0), to = min(h1 - skip, a.heads[z]);
    if (from >= to) continue;
    const T* x = static_cast<const T*>(a.x[z]) + b * a.sb[z] + from * a.sh[z] + n * a.sn[z];
    T* y = static_cast<T*>(a.y[z]) +
           ((static_cast<long long>(b) * a.heads[z] + from) * a.N + n) * a.d;
    const long long in_step = a.sh[z], out_step = static_cast<long long>(a.N) * a.d;
    if constexpr (VEC_OK) {
      // the loads of BATCH heads go out before the first of their stores
      constexpr int BATCH = HALF ? 2 : 4;
      for (int h = from; h < to; h += BATCH, x += BATCH * in_step, y += BATCH * out_step) {
        uint4 v0[BATCH], v1[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          if (h + k >= to) break;
          v0[k] = __ldcs(reinterpret_cast<const uint4*>(x + k * in_step + c0));
          if (HALF && !copy) v1[k] = __ldcs(reinterpret_cast<const uint4*>(x + k * in_step + c1));
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          if (h + k >= to) break;
          T* yk = y + k * out_step;
          if (copy) {
            *reinterpret_cast<uint4*>(yk + c0) = v0[k];
          } else if constexpr (HALF) {
            float p[V], q[V], o0[V], o1[V];
            R::load(v0[k], p);
            R::load(v1[k], q);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              o0[i] = p[i] * cs[i] - q[i] * sn[i];
              o1[i] = q[i] * cs[i] + p[i] * sn[i];
            }
            *reinterpret_cast<uint4*>(yk + c0) = R::store(o0);
            *reinterpret_cast<uint4*>(yk + c1) = R::store(o1);
          } else {
            float p[V], o[V];
            R::load(v0[k], p);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              o[2 * i] = p[2 * i] * cs[i] - p[2 * i + 1] * sn[i];
              o[2 * i + 1] = p[2 * i + 1] * cs[i] + p[2 * i] * sn[i];
            }
            *reinterpret_cast<uint4*>(yk + c0) = R::store(o);
          }
        }
      }
    } else {
      for (int h = from; h < to; ++h, x += in_step, y += out_step) {
        if (copy) {
          y[c0] = x[c0];
        } else {
          const float p = R::one(x[c0]), q = R::one(x[c1]);
          y[c0] = R::to(p * cs[0] - q * sn[0]);
          y[c1] = R::to(q * cs[0] + p * sn[0]);
        }
      }
    }
  }
}

}  // namespace rfb
