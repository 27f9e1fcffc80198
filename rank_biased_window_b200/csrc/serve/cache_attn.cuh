// cache_attn.cuh -- attention of a few query tokens over the 8-bit cache, with
// the rank-factorised bias:
//
//     x_t = s ks (q . k8_t) + ws (u . w8_t),   O = sum_t exp(x_t - LSE) vs v8_t.
//
// The rows of one key head (its query heads times the new tokens) share every
// cached byte.  A warp takes 16 rows and walks over blocks of 32 tokens: the
// codes go from global memory straight into the registers that the MMA wants
// (the order of channels and of tokens inside a contraction is free, so each
// lane loads whole 8- or 16-byte pieces of rows and the queries are permuted to
// match), become fp16 there (exact) and enter m16n8k16 MMAs with fp32
// accumulators.  Softmax statistics and sums are fp32; the probabilities are
// rounded to fp16 for the product with V (2^-12 relative, below the bf16
// rounding of O).  Queries enter as fp16 scaled by a power of two per row,
// which holds every bf16 within 2^-29 of the row's largest exactly.
//
// Bound by HBM: 2 d + r bytes a token and head.  With at most 16 rows in a
// tile, 32 flop per byte, the register-level MMA runs at a fraction of its rate;
// tcgen05 would need the codes widened into shared memory first, which costs
// more than the product.
//
// Work split: the blocks of all (sequence, key head, row tile) segments form one
// line, cut into equal parts, one per CTA, so ragged lengths and few long
// sequences fill the chip alike.  A segment that one CTA holds whole is finished
// there; others leave (max, sum, O) partials, which cache_attn_combine_kernel
// joins in order (results do not depend on timing).
#pragma once
#include "../sm100.cuh"
#include "e4m3.cuh"

namespace rfb {

constexpr int kCaWarps = 4;
constexpr int kCaThreads = kCaWarps * 32;

struct CacheAttnArgs {
  const __nv_bfloat16* q;  // [B, Hk, R, d], R = group * Nq
  const __nv_bfloat16* u;  // [B, Hk, R, r]
  const uint8_t *k, *v, *w;
  const float *ks, *vs, *ws;
  const int* lengths;
  __nv_bfloat16* o;
  float* lse;
  float* scores;  // [B, Hk, R, cap] log2 scores for the mass, or null
  float* part_o;  // [ctas][2][rows of a segment][d]
  float2* part_ml;
  int B, Hk, R, Nq, cap, r;
  int wr;        // warps over row tiles: 1, 2 or 4
  int row_segs;  // segments of 16 wr rows
  int causal;
  float scale_log2;
};

__device__ __forceinline__ int cache_blocks(const CacheAttnArgs& a, int b) {
  return (min(max(a.lengths[b], 0), a.cap) + kCacheBlock - 1) / kCacheBlock;
}

// Blocks of sequences [0, b_end) (all lanes of the warp call it).
__device__ __forceinline__ long long blocks_before(const CacheAttnArgs& a, int b_end) {
  long long sum = 0;
  for (int b0 = 0; b0 < b_end; b0 += 32) {
    const int b = b0 + static_cast<int>(lane_id());
    const unsigned n = b < b_end ? cache_blocks(a, b) : 0;
    sum += __reduce_add_sync(0xffffffffu, n);
  }
  return sum;
}

// Sequence that holds block `at` of the per-sequence line, and the blocks before it.
__device__ __forceinline__ int sequence_of(const CacheAttnArgs& a, long long at, long long& before) {
  before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + static_cast<int>(lane_id());
    const int n = b < a.B ? cache_blocks(a, b) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (static_cast<int>(lane_id()) >= o) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + incl > at);
    if (past) {
      const int l = __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, incl - n, l);
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return a.B;
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w));
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
}

// O += P V for 16 rows and 32 tokens: p[kk] the A fragments of tokens 16 kk..,
// v[4 kk + i] the lane's piece of its i-th token there.  Channel tile n of the
// product holds channel g (D / 8) + n in column g.
template <int VW>
__device__ __forceinline__ void pv_product(const uint32_t (*p)[4], const uint32_t (*v)[VW],
                                           float (*o)[4]) {
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t a01 = __byte_perm(v[4 * kk][w], v[4 * kk + 1][w], 0x5140);
      const uint32_t a23 = __byte_perm(v[4 * kk][w], v[4 * kk + 1][w], 0x7362);
      const uint32_t b01 = __byte_perm(v[4 * kk + 2][w], v[4 * kk + 3][w], 0x5140);
      const uint32_t b23 = __byte_perm(v[4 * kk + 2][w], v[4 * kk + 3][w], 0x7362);
      mma_f16(o[4 * w], p[kk], e4m3_lo(a01), e4m3_lo(b01));
      mma_f16(o[4 * w + 1], p[kk], e4m3_hi(a01), e4m3_hi(b01));
      mma_f16(o[4 * w + 2], p[kk], e4m3_lo(a23), e4m3_lo(b23));
      mma_f16(o[4 * w + 3], p[kk], e4m3_hi(a23), e4m3_hi(b23));
    }
}

// Channel of the first of the four codes in word i of a lane's row piece, for
// rows of C channels (C / 16 words a lane; t = lane & 3).
template <int C>
__device__ __forceinline__ int piece_channel(int i, int t) {
  if constexpr (C >= 64) return (i / 4) * 64 + t * 16 + (i % 4) * 4;
  return t * (C / 4) + i * 4;
}
// The same for the factors, whose rows may end inside C (pieces of 8 bytes).
template <int C>
__device__ __forceinline__ int factor_channel(int i, int t) {
  if constexpr (C == 64) return (i / 2) * 32 + t * 8 + (i % 2) * 4;
  return t * (C / 4) + i * 4;
}

// A rows x C matrix of bf16 as fp16 A fragments, each row times 2^(14 - e) with
// e its exponent; back[] undoes it.
template <int C, bool FACTOR>
__device__ __forceinline__ void load_rows(const __nv_bfloat16* x, int stride, const bool* live,
                                          int t, uint32_t (*frag)[4], float* back) {
  float f[2][C / 4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < C / 16; ++i) {
      const int ch = FACTOR ? factor_channel<C>(i, t) : piece_channel<C>(i, t);
      uint2 v = make_uint2(0, 0);
      if (live[half] && ch < stride)
        v = __ldg(reinterpret_cast<const uint2*>(x + static_cast<long long>(half) * 8 * stride + ch));
      const float e[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                          __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[half][4 * i + k] = e[k];
        top = fmaxf(top, fabsf(e[k]));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // exponent held so that 2^(14 - e) and its inverse are normal
    const int e = min(max(__float_as_int(top) >> 23, 60), 194) - 127;
    const float to = pow2f(14 - e);
    back[half] = pow2f(e - 14);
#pragma unroll
    for (int i = 0; i < C / 4; ++i) f[half][i] *= to;
  }
#pragma unroll
  for (int i = 0; i < C / 16; ++i) {
    frag[i][0] = pack_f16x2(f[0][4 * i], f[0][4 * i + 1]);
    frag[i][1] = pack_f16x2(f[1][4 * i], f[1][4 * i + 1]);
    frag[i][2] = pack_f16x2(f[0][4 * i + 2], f[0][4 * i + 3]);
    frag[i][3] = pack_f16x2(f[1][4 * i + 2], f[1][4 * i + 3]);
  }
}

template <int D>
struct CaSmem {
  float o[kCaWarps][16][D + 4];
  float2 ml[kCaWarps][16];
};

template <int D, int RP, bool MASS>
__global__ void __launch_bounds__(kCaThreads, D == 128 ? 2 : 3)
    cache_attn_kernel(const CacheAttnArgs a) {
  constexpr int KW = D / 16;                  // K words of a lane and 8-token tile; QK steps
  constexpr int WW = RP / 16;                 // the same for the factors
  constexpr int VW = D / 32;                  // V words of a lane and token
  constexpr int NT = D / 8;                   // channel tiles of the PV product
  __shared__ CaSmem<D> sm;
  grid_dep_wait();
  const int lane = lane_id(), warp = warp_id();
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % a.wr, wt = warp / a.wr, wts = kCaWarps / a.wr;
  const int mult = a.Hk * a.row_segs;
  const long long W = blocks_before(a, a.B) * mult;
  long long at = W * blockIdx.x / gridDim.x;
  const long long stop = W * (blockIdx.x + 1) / gridDim.x;
  grid_dep_launch_next();
  if (at >= stop) return;
  long long before;
  int b = sequence_of(a, at / mult, before);
  int nb = cache_blocks(a, b);
  long long in_seq = at - before * mult;  // position inside sequence b's segments
  int seg = static_cast<int>(in_seq / nb);
  int blk0 = static_cast<int>(in_seq - static_cast<long long>(seg) * nb);
  const int seg_rows = min(a.R, 16 * a.wr);
  bool first = true;

  while (at < stop) {
    const int h = seg / a.row_segs, rs = seg - h * a.row_segs;
    const int blk1 = static_cast<int>(min(static_cast<long long>(nb), blk0 + (stop - at)));
    const int L = min(a.lengths[b], a.cap);
    const long long bh = static_cast<long long>(b) * a.Hk + h;
    const int row0 = (rs * a.wr + wr) * 16;

    // rows g and g + 8 of this warp's tile
    bool live[2];
    int lim[2];  // tokens the row sees
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + g + 8 * i;
      live[i] = row < a.R;
      lim[i] = L;
      if (a.causal && live[i]) lim[i] = max(min(L, L - a.Nq + 1 + row % a.Nq), 0);
    }
    const int lim_lo = __reduce_min_sync(0xffffffffu, min(lim[0], lim[1]));

    uint32_t qf[KW][4];
    float fq[2];
    load_rows<D, false>(a.q + (bh * a.R + row0 + g) * D, D, live, t, qf, fq);
    fq[0] *= a.scale_log2;
    fq[1] *= a.scale_log2;
    uint32_t uf[WW > 0 ? WW : 1][4];
    float fu[2] = {0.f, 0.f};
    if constexpr (RP > 0) {
      load_rows<RP, true>(a.u + (bh * a.R + row0 + g) * a.r, a.r, live, t, uf, fu);
      fu[0] *= kLog2e;
      fu[1] *= kLog2e;
    }

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float oacc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) oacc[i][k] = 0.f;
    float unit = 1.f;  // oacc is O / unit

    const uint8_t* kp = a.k + bh * a.cap * D;
    const uint8_t* vp = a.v + bh * a.cap * D;
    const uint8_t* wp = RP > 0 ? a.w + bh * a.cap * a.r : nullptr;
    const long long sbase = bh * (a.cap / kCacheBlock);
    uint32_t kr[4][KW], vr[8][VW], wreg[4][WW > 0 ? WW : 1];
    float ksc = 1.f, vsc = 1.f, wsc = 0.f;

    const auto load_k = [&](int blk) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = kp + (static_cast<long long>(blk) * kCacheBlock + 8 * j + g) * D;
        if constexpr (D >= 64) {
#pragma unroll
          for (int c = 0; c < KW / 4; ++c) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(p + 64 * c + 16 * t));
            kr[j][4 * c] = x.x, kr[j][4 * c + 1] = x.y, kr[j][4 * c + 2] = x.z, kr[j][4 * c + 3] = x.w;
          }
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(p + 8 * t));
          kr[j][0] = x.x, kr[j][1] = x.y;
        }
        if constexpr (RP > 0) {
          const uint8_t* pw = wp + (static_cast<long long>(blk) * kCacheBlock + 8 * j + g) * a.r;
#pragma unroll
          for (int i = 0; i < WW; ++i) wreg[j][i] = 0;
          if constexpr (RP == 16) {
            if (4 * t < a.r) wreg[j][0] = __ldg(reinterpret_cast<const uint32_t*>(pw + 4 * t));
          } else {
#pragma unroll
            for (int c = 0; c < WW / 2; ++c) {
              const int ch = factor_channel<RP>(2 * c, t);
              if (ch < a.r) {
                const uint2 x = __ldg(reinterpret_cast<const uint2*>(pw + ch));
                wreg[j][2 * c] = x.x, wreg[j][2 * c + 1] = x.y;
              }
            }
          }
        }
      }
      ksc = __ldg(a.ks + sbase + blk);
      if constexpr (RP > 0) wsc = __ldg(a.ws + sbase + blk);
    };
    // token 16 kk + 8 (i / 2) + 2 t + i % 2 of the block is vr[4 kk + i]
    const auto load_v = [&](int blk) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = 16 * (i / 4) + 8 * ((i / 2) & 1) + 2 * t + (i & 1);
        const uint8_t* p = vp + (static_cast<long long>(blk) * kCacheBlock + tok) * D + g * (D / 8);
        if constexpr (D == 128) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
          vr[i][0] = x.x, vr[i][1] = x.y, vr[i][2] = x.z, vr[i][3] = x.w;
        } else if constexpr (D == 64) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
          vr[i][0] = x.x, vr[i][1] = x.y;
        } else {
          vr[i][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        }
      }
      vsc = __ldg(a.vs + sbase + blk);
    };

    int blk = blk0 + wt;
    if (blk < blk1) {
      load_k(blk);
      load_v(blk);
    }
    for (; blk < blk1; blk += wts) {
      // scores of 16 rows x 32 tokens, in units of log2
      float x[4][4];
      const float f0 = fq[0] * ksc, f1 = fq[1] * ksc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KW; ++i) mma_f16(c, qf[i], e4m3_lo(kr[j][i]), e4m3_hi(kr[j][i]));
        x[j][0] = c[0] * f0, x[j][1] = c[1] * f0, x[j][2] = c[2] * f1, x[j][3] = c[3] * f1;
        if constexpr (RP > 0) {
          float cw[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < WW; ++i) mma_f16(cw, uf[i], e4m3_lo(wreg[j][i]), e4m3_hi(wreg[j][i]));
          x[j][0] = fmaf(cw[0], fu[0] * wsc, x[j][0]);
          x[j][1] = fmaf(cw[1], fu[0] * wsc, x[j][1]);
          x[j][2] = fmaf(cw[2], fu[1] * wsc, x[j][2]);
          x[j][3] = fmaf(cw[3], fu[1] * wsc, x[j][3]);
        }
      }
      const bool edge = (blk + 1) * kCacheBlock > lim_lo;  // a row does not see all of the block
      if (blk + wts < blk1) load_k(blk + wts);
      if (edge) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = blk * kCacheBlock + 8 * j + 2 * t + (k & 1);
            if (tok >= lim[k >> 1]) x[j][k] = -INFINITY;
          }
        // codes of no token (any bytes, the NaN code among them) do not enter the product
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = 16 * (i / 4) + 8 * ((i / 2) & 1) + 2 * t + (i & 1);
          if (blk * kCacheBlock + tok >= L)
#pragma unroll
            for (int k = 0; k < VW; ++k) vr[i][k] = 0;
        }
      }
      if constexpr (MASS) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (live[i]) {
            float* s = a.scores + (bh * a.R + row0 + g + 8 * i) * a.cap + blk * kCacheBlock + 2 * t;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float2*>(s + 8 * j) = make_float2(x[j][2 * i], x[j][2 * i + 1]);
          }
      }
      // running maximum and sum
      float mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v = fmax3(v, x[j][2 * i], x[j][2 * i + 1]);
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        mx[i] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
      }
      const bool moved = mx[0] != m[0] || mx[1] != m[1] || vsc != unit;
      if (__any_sync(0xffffffffu, moved)) {
        const float back = unit / vsc;
        unit = vsc;
        float al[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          al[i] = mx[i] == -INFINITY ? 1.f : fast_exp2(m[i] - mx[i]);
          m[i] = mx[i];
          l[i] *= al[i];
          al[i] *= back;
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          oacc[k][0] *= al[0], oacc[k][1] *= al[0];
          oacc[k][2] *= al[1], oacc[k][3] *= al[1];
        }
      }
      const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[j][k] = fast_exp2(x[j][k] - base[k >> 1]);
          l[k >> 1] += x[j][k];
        }
      // O += P V
      uint32_t p[2][4];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        p[kk][0] = pack_f16x2(x[2 * kk][0], x[2 * kk][1]);
        p[kk][1] = pack_f16x2(x[2 * kk][2], x[2 * kk][3]);
        p[kk][2] = pack_f16x2(x[2 * kk + 1][0], x[2 * kk + 1][1]);
        p[kk][3] = pack_f16x2(x[2 * kk + 1][2], x[2 * kk + 1][3]);
      }
      bool poison = false;  // a NaN in V that some rows may not see
      if (edge && a.causal) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < VW; ++k) any |= __vcmpeq4(vr[i][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        poison = __any_sync(0xffffffffu, any != 0);
      }
      if (!poison) {
        pv_product<VW>(p, vr, oacc);
      } else {
        // 0 x NaN is NaN, so a masked weight does not keep it out: row by row,
        // with the tokens that the row does not see as zeros
#pragma unroll 1
        for (int r = 0; r < 16; ++r) {
          const int lim_r = __shfl_sync(0xffffffffu, r < 8 ? lim[0] : lim[1], (r & 7) * 4);
          const bool mine = g == (r & 7);
          uint32_t pr[2][4], vm[8][VW];
          float c[NT][4];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int k = 0; k < 4; ++k) pr[kk][k] = mine && (k & 1) == (r >> 3) ? p[kk][k] : 0u;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int tok = 16 * (i / 4) + 8 * ((i / 2) & 1) + 2 * t + (i & 1);
#pragma unroll
            for (int k = 0; k < VW; ++k)
              vm[i][k] = blk * kCacheBlock + tok < lim_r ? vr[i][k] : 0u;
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) c[i][k] = 0.f;
          pv_product<VW>(pr, vm, c);
          if (mine) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              oacc[i][0] += r < 8 ? c[i][0] : 0.f, oacc[i][1] += r < 8 ? c[i][1] : 0.f;
              oacc[i][2] += r < 8 ? 0.f : c[i][2], oacc[i][3] += r < 8 ? 0.f : c[i][3];
            }
          }
        }
      }
      if (blk + wts < blk1) load_v(blk + wts);
    }

    // join the warps that share rows: channel 2 t (D / 8) + i of a row is oacc[i][0],
    // the next D / 8 oacc[i][1]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (t == 0) sm.ml[warp][g + 8 * i] = make_float2(m[i], l[i]);
#pragma unroll
      for (int k = 0; k < NT; k += 4)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(&sm.o[warp][g + 8 * i][(2 * t + e) * NT + k]) =
              make_float4(oacc[k][2 * i + e] * unit, oacc[k + 1][2 * i + e] * unit,
                          oacc[k + 2][2 * i + e] * unit, oacc[k + 3][2 * i + e] * unit);
    }
    __syncthreads();
    const bool whole = blk0 == 0 && blk1 == nb;
    const int slot = first ? 0 : 1;
    for (int i = threadIdx.x; i < 16 * a.wr * (D / 4); i += kCaThreads) {
      const int rr = i / (D / 4), c = (i - rr * (D / 4)) * 4;
      const int row = rs * a.wr * 16 + rr;
      if (row >= a.R) continue;
      const int w0 = rr / 16, r16 = rr % 16;
      float mm = -INFINITY;
      for (int w = 0; w < wts; ++w) mm = fmaxf(mm, sm.ml[w0 + w * a.wr][r16].x);
      const float base = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < wts; ++w) {
        const int ww = w0 + w * a.wr;
        const float f = fast_exp2(sm.ml[ww][r16].x - base);
        const float4 v = *reinterpret_cast<const float4*>(&sm.o[ww][r16][c]);
        ll = fmaf(sm.ml[ww][r16].y, f, ll);
        acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        const float inv = ll > 0.f ? 1.f / ll : ll;  // no token seen: O = 0; NaN stays
        const long long out = bh * a.R + row;
        *reinterpret_cast<uint2*>(a.o + out * D + c) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (c == 0) a.lse[out] = (mm + __log2f(ll)) * kLn2;
      } else {
        const long long p = (static_cast<long long>(blockIdx.x) * 2 + slot) * seg_rows + rr;
        *reinterpret_cast<float4*>(a.part_o + p * D + c) = acc;
        if (c == 0) a.part_ml[p] = make_float2(mm, ll);
      }
    }
    __syncthreads();
    first = false;
    at += blk1 - blk0;
    blk0 = 0;
    if (++seg == mult) {
      seg = 0;
      do {
        ++b;
      } while (b < a.B && cache_blocks(a, b) == 0);
      if (b < a.B) nb = cache_blocks(a, b);
    }
  }
}

// Joins the partials of the segments that several CTAs share and writes the
// rows of empty sequences.  D / 4 threads a row; blockIdx.x is (b, h, row
// segment).
template <int D>
__global__ void __launch_bounds__(128) cache_attn_combine_kernel(const CacheAttnArgs a, int ctas) {
  grid_dep_wait();
  constexpr int TPR = D / 4;
  const int seg_rows = min(a.R, 16 * a.wr);
  const int rr = blockIdx.y * (128 / TPR) + threadIdx.x / TPR;
  const int c = (threadIdx.x % TPR) * 4;
  const int mult = a.Hk * a.row_segs;
  const int b = blockIdx.x / mult, seg = blockIdx.x - b * mult;
  const int h = seg / a.row_segs, rs = seg - h * a.row_segs;
  const long long W = blocks_before(a, a.B) * mult;
  const int nb = cache_blocks(a, b);
  const long long s0 = blocks_before(a, b) * mult + static_cast<long long>(seg) * nb, s1 = s0 + nb;
  const int row = rs * a.wr * 16 + rr;
  if (rr >= seg_rows || row >= a.R) return;
  const long long out = (static_cast<long long>(b) * a.Hk + h) * a.R + row;
  if (nb == 0) {
    *reinterpret_cast<uint2*>(a.o + out * D + c) = make_uint2(0, 0);
    if (c == 0) a.lse[out] = -INFINITY;
    return;
  }
  // CTA i holds [W i / ctas, W (i + 1) / ctas)
  const auto start_of = [&](long long i) { return W * i / ctas; };
  long long i0 = s0 * ctas / W;
  while (start_of(i0 + 1) <= s0) ++i0;
  while (start_of(i0) > s0) --i0;
  if (start_of(i0 + 1) >= s1) return;  // one CTA had it whole
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (long long i = i0; i < ctas && start_of(i) < s1; ++i) {
    if (start_of(i + 1) == start_of(i)) continue;
    const int slot = start_of(i) >= s0 ? 0 : 1;  // the CTA's first segment, or a later one
    const long long p = (i * 2 + slot) * seg_rows + rr;
    const float2 ml = a.part_ml[p];
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + p * D + c);
    const float mn = fmaxf(m, ml.x);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = fast_exp2(m - base), e = fast_exp2(ml.x - base);
    m = mn;
    l = l * f + ml.y * e;
    acc.x = acc.x * f + v.x * e, acc.y = acc.y * f + v.y * e;
    acc.z = acc.z * f + v.z * e, acc.w = acc.w * f + v.w * e;
  }
  const float inv = l > 0.f ? 1.f / l : l;
  *reinterpret_cast<uint2*>(a.o + out * D + c) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0) a.lse[out] = (m + __log2f(l)) * kLn2;
}

// mass_out = decay mass + sum over the key head's rows of exp(x - LSE), for the
// tokens of each sequence; 4 tokens a thread.
__global__ void __launch_bounds__(128) cache_mass_kernel(const CacheAttnArgs a, const float* mass,
                                                         float* mass_out, float decay) {
  grid_dep_wait();
  const int bh = blockIdx.x, b = bh / a.Hk;
  const int t0 = (blockIdx.y * 128 + threadIdx.x) * 4;
  const int L = min(a.lengths[b], a.cap);
  if (t0 >= L) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* s = a.scores + static_cast<long long>(bh) * a.R * a.cap + t0;
  const float* lse = a.lse + static_cast<long long>(bh) * a.R;
#pragma unroll 4
  for (int i = 0; i < a.R; ++i) {
    const float z = lse[i];
    if (z == -INFINITY) continue;  // the row sees nothing
    const float4 x = *reinterpret_cast<const float4*>(s + static_cast<long long>(i) * a.cap);
    const float y = z * kLog2e;
    sum.x += fast_exp2(x.x - y), sum.y += fast_exp2(x.y - y);
    sum.z += fast_exp2(x.z - y), sum.w += fast_exp2(x.w - y);
  }
  const float add[4] = {sum.x, sum.y, sum.z, sum.w};
  const long long at = static_cast<long long>(bh) * a.cap + t0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t0 + k < L) mass_out[at + k] = mass ? fmaf(decay, mass[at + k], add[k]) : add[k];
}

}  // namespace rfb
