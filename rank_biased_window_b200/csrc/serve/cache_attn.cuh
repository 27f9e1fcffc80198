// cache_attn.cuh -- attention of a few query tokens over the 8-bit cache, with
// the rank-factorised bias:
//
//     x_t = s ks (q . k8_t) + ws (u . w8_t),   O = sum_t exp(x_t - LSE) vs v8_t.
//
// The rows of one key head (its query heads times the new tokens) share every cached
// byte.  A warp takes 8 or 16 rows and walks over blocks of 32 tokens, which one lane a
// tensor copies (bulk copies with mbarriers) into a ring in shared memory, as they lie
// in global memory; up to four warps of other rows share a ring.  From there each lane
// reads whole 8- or 16-byte pieces of rows (the order of channels and of tokens inside a
// contraction is free, so the queries are permuted to match), which become fp16 in
// registers (exact) and enter m16n8k16 MMAs with fp32 accumulators, keys and values as
// the row operand.  Softmax statistics and sums are fp32; the probabilities enter the
// product with V as two fp16 terms (2^-22 relative, so that O is what fp32 weights give:
// with one, 2^-11, one value of O in twelve came out a bf16 step away, with two one in a
// thousand; one takes 33.3 us for 34.9 at 64 rows, 196 for 207 at 450 sequences to 4096
// tokens, and is no faster where the bytes bind), lifted by 2^11 so that the first is
// normal down to 2^-25 of the largest: a token of small weight may have a large value.
// The largest is followed with a slack of 2^4, so that the sums are rescaled a few times
// a segment (2^15 is within fp16).  Queries enter as fp16 scaled by a power of two per
// row, which holds every bf16 within 2^-28 of the row's largest exactly.
//
// Bound by HBM for few rows: 2 d + r bytes a token and head (2 x 131000 tokens of
// 8 heads, d = 64, r = 32: 60.6 us, 5.6 TB/s; 16 sequences of up to 8190 tokens, 32
// heads on 8, d = 128: 35.6 us, 4.2 TB/s; some 7 to 10 us of each are the start and the
// end of the two kernels); by issue and latency for the 64 rows of 16 queries (8 sequences
// of up to 5003 tokens, 16 heads on 4: 34.9 us with the weights, 24.9 without).  With at
// most 16 rows in a tile, 32 flop per byte, the register-level MMA runs at a fraction
// of its rate and the bytes bind.  tcgen05 could multiply the codes as they are
// (kind::f8f6f4), but its other operand is 8 bits then too, with 4 of them significant:
// a bf16 query would take two terms and a weight of 22 bits six, and of a tile's 128 rows
// 64 at most are there.  Not measured.
//
// Work split: the blocks of all (sequence, key head, row tile) segments form one
// line, cut into equal parts, one per CTA, so ragged lengths and few long
// sequences fill the chip alike; a segment counts kCaSegmentCost blocks more than
// it has, since beginning one and joining its warps takes that long.  A segment that
// one CTA holds whole is finished there; others leave (max, sum, O) partials, which
// cache_attn_combine_kernel joins in order (results do not depend on timing).  Short
// contexts, and segments enough for several waves, take a CTA a segment instead
// (`whole`): no partials, no join.
#pragma once
#include "../sm100.cuh"
#include "e4m3.cuh"

namespace rfb {

constexpr int kCaWarps = 4;
constexpr int kCaThreads = kCaWarps * 32;
constexpr unsigned kCaSegmentCost = 4;
constexpr float kCaLift = 11.f;   // weights are held as 2^(x - max + 11) ...
constexpr float kCaSlack = 4.f;   // ... with a max that scores may pass by 2^4 before it moves
// From here on (2^22, where fp32 steps by 1/2) neither: max - 11 would round to a multiple
// of up to 16, and a weight past fp16's largest.
constexpr float kCaCoarse = 4194304.f;

struct CacheAttnArgs {
  const __nv_bfloat16* q;  // [B, Hk, R, d], R = group * Nq
  const __nv_bfloat16* u;  // [B, Hk, R, r]
  const uint8_t *k, *v, *w;
  const float *ks, *vs, *ws;
  const int* lengths;
  const int* counts;  // [B] or null: the sequence's queries are the first counts[b] of Nq
  __nv_bfloat16* o;
  float* lse;
  float* scores;  // [B, Hk, R, cap] log2 scores for the mass, or null
  const float* mass;
  float* mass_out;
  float decay;
  float* part_o;  // [ctas][2][rows of a segment][d]
  float2* part_ml;
  int B, Hk, R, Nq, cap, r;
  int tile;      // queries of a warp: 8 or 16
  int wr;        // warps over row tiles: 1, 2 or 4
  int row_segs;  // segments of tile * wr rows
  int causal;
  int whole;     // one CTA a segment, no partials
  int stages;
  float scale_log2;
  int* err_word;
  unsigned long long wait_ns;
  int fail_site;
};

__device__ __forceinline__ int cache_blocks(const CacheAttnArgs& a, int b) {
  return (min(max(a.lengths[b], 0), a.cap) + kCacheBlock - 1) / kCacheBlock;
}
// Whether queries of a sequence may see different tokens.
__device__ __forceinline__ bool masked(const CacheAttnArgs& a) { return a.causal || a.counts; }
// Tokens of the sequence's L that query row `row` sees; rows behind its own queries see none.
__device__ __forceinline__ int row_sees(const CacheAttnArgs& a, int b, int row, int L) {
  if (!masked(a) || row >= a.R) return L;
  const int n = a.counts ? min(max(a.counts[b], 0), a.Nq) : a.Nq, i = row % a.Nq;
  return i >= n ? 0 : a.causal ? max(min(L, L - n + 1 + i), 0) : L;
}
// Length on the line of a segment of n blocks: its cost, then its blocks; an
// empty one has none.
__device__ __forceinline__ unsigned line_length(int n) { return n > 0 ? n + kCaSegmentCost : 0u; }

// Line length of all sequences (one segment each), and of those before sequence b
// (all lanes call it).
__device__ __forceinline__ void count_line(const CacheAttnArgs& a, int b, unsigned& before,
                                             unsigned& total) {
  before = total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int x = b0 + static_cast<int>(lane_id());
    const unsigned n = x < a.B ? line_length(cache_blocks(a, x)) : 0;
    total += __reduce_add_sync(0xffffffffu, n);
    before += __reduce_add_sync(0xffffffffu, x < b ? n : 0u);
  }
}

// A line of length W cut over n CTAs: the first W % n hold W / n + 1, the rest W / n.
struct Cut {
  unsigned base, extra;
  __device__ __forceinline__ Cut(unsigned W, unsigned n) : base(W / n), extra(W - W / n * n) {}
  __device__ __forceinline__ unsigned start(unsigned i) const { return i * base + min(i, extra); }
  __device__ __forceinline__ unsigned holder(unsigned x) const {
    const unsigned fat = extra * (base + 1);
    return x < fat ? x / (base + 1) : extra + (x - fat) / max(base, 1u);
  }
};

// The CTA's part [at, stop) of the line and where it starts: sequence b, whose
// segments have nb blocks each; segment seg of it, `in` from that segment's start.
struct Place {
  unsigned at, stop;
  int b, nb, seg;
  unsigned in;
};
__device__ __forceinline__ Place place_of(const CacheAttnArgs& a, unsigned mult) {
  Place p = {};
  const int lane = lane_id();
  unsigned total = 0, n = 0, incl = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {  // at most 32 sequences: one round, kept below
    n = b0 + lane < a.B ? line_length(cache_blocks(a, b0 + lane)) : 0;
    incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    total += __shfl_sync(0xffffffffu, incl, 31);
  }
  const Cut cut(total * mult, gridDim.x);
  p.at = cut.start(blockIdx.x);
  p.stop = cut.start(blockIdx.x + 1);
  if (p.at >= p.stop) return p;
  const unsigned seq_at = p.at / mult;
  unsigned before = 0;
  for (int b0 = 0;; b0 += 32) {
    if (a.B > 32) {
      n = b0 + lane < a.B ? line_length(cache_blocks(a, b0 + lane)) : 0;
      incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + incl > seq_at);
    if (past) {
      const int l = __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, incl - n, l);
      p.b = b0 + l;
      p.nb = __shfl_sync(0xffffffffu, n, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  const unsigned in_seq = p.at - before * mult, len = p.nb;
  p.seg = in_seq / len;
  p.in = in_seq - p.seg * len;
  p.nb = len - kCaSegmentCost;
  return p;
}

// The same with a CTA a segment; an empty one has nb = 0.
__device__ __forceinline__ Place segment_of(const CacheAttnArgs& a, unsigned mult) {
  Place p = {};
  p.b = blockIdx.x / mult;
  p.seg = blockIdx.x - p.b * mult;
  p.nb = cache_blocks(a, p.b);
  p.stop = line_length(p.nb);
  return p;
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
// An 8 x 8 tile of 16-bit values, a row in the lanes of one g, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// O^T += V^T P^T for 16 tokens and 8 QT queries, P in two fp16 terms (p[q][0..1] and the
// rest of the fp32 weight, p[q][2..3]): v[i] the lane's piece of its i-th
// token (two of columns 2 t, 2 t + 1, two of the next 8), word w of it, i.e. channels
// g (D / 8) + 4 w + {0..3}, which are rows g and g + 8 of channel tiles 2 w, 2 w + 1.
template <int VW, int QT>
__device__ __forceinline__ void pv_words(const uint32_t (*p)[4], const uint32_t (*v)[VW], int w,
                                         float (*o)[QT][4]) {
  const uint32_t a01 = __byte_perm(v[0][w], v[1][w], 0x5140);
  const uint32_t a23 = __byte_perm(v[0][w], v[1][w], 0x7362);
  const uint32_t b01 = __byte_perm(v[2][w], v[3][w], 0x5140);
  const uint32_t b23 = __byte_perm(v[2][w], v[3][w], 0x7362);
  const uint32_t lo[4] = {e4m3_lo(a01), e4m3_hi(a01), e4m3_lo(b01), e4m3_hi(b01)};
  const uint32_t hi[4] = {e4m3_lo(a23), e4m3_hi(a23), e4m3_lo(b23), e4m3_hi(b23)};
#pragma unroll
  for (int q = 0; q < QT; ++q) {
    mma_f16(o[0][q], lo, p[q][0], p[q][1]);
    mma_f16(o[1][q], hi, p[q][0], p[q][1]);
    mma_f16(o[0][q], lo, p[q][2], p[q][3]);
    mma_f16(o[1][q], hi, p[q][2], p[q][3]);
  }
}
template <int VW, int QT>
__device__ __forceinline__ void pv_step(const uint32_t (*p)[4], const uint32_t (*v)[VW],
                                        float (*o)[QT][4]) {
#pragma unroll
  for (int w = 0; w < VW; ++w) pv_words<VW, QT>(p, v, w, o + 2 * w);
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

// One query row of C bf16 channels, the lane's t-th pieces.
template <int C, bool FACTOR>
__device__ __forceinline__ void fetch_row(const __nv_bfloat16* x, int channels, bool live, int t,
                                          uint2* raw) {
#pragma unroll
  for (int i = 0; i < C / 16; ++i) {
    const int ch = FACTOR ? factor_channel<C>(i, t) : piece_channel<C>(i, t);
    raw[i] = make_uint2(0, 0);
    if (live && ch < channels) raw[i] = __ldg(reinterpret_cast<const uint2*>(x + ch));
  }
}
// The row as fp16 B fragments, times 2^(14 - e) with e the exponent of its largest;
// returns 2^(e - 14).
template <int C>
__device__ __forceinline__ float row_fragments(const uint2* raw, uint32_t (*frag)[2]) {
  float f[C / 4], top = 0.f;
#pragma unroll
  for (int i = 0; i < C / 16; ++i) {
    const float e[4] = {__uint_as_float(raw[i].x << 16), __uint_as_float(raw[i].x & 0xffff0000u),
                        __uint_as_float(raw[i].y << 16), __uint_as_float(raw[i].y & 0xffff0000u)};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[4 * i + k] = e[k];
      top = fmaxf(top, fabsf(e[k]));
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // exponent held so that 2^(14 - e) and its inverse are normal: every one from 2^-112 up
  const int e = min(max(__float_as_int(top) >> 23, 15), 254) - 127;
  const float to = pow2f(14 - e);
#pragma unroll
  for (int i = 0; i < C / 16; ++i) {
    frag[i][0] = pack_f16x2(f[4 * i] * to, f[4 * i + 1] * to);
    frag[i][1] = pack_f16x2(f[4 * i + 2] * to, f[4 * i + 3] * to);
  }
  return pow2f(e - 14);
}

// ------------------------------------------------------------------ pipeline
// Shared memory of a CTA: barriers, the warps' (max, sum), then the ring: for
// each of the wts token groups `stages` stages of one block, K | V | W as they
// lie in global memory.
constexpr int kCaMaxStages = 8;
constexpr int kCaRing = 2048;  // offset of the ring

struct CaHead {
  uint64_t full[kCaWarps][kCaMaxStages];
  uint64_t empty[kCaWarps][kCaMaxStages];
  float2 ml[kCaWarps][16];
  uint32_t held[kCaWarps];
  int abort_flag, drain_flag;
};
static_assert(sizeof(CaHead) <= kCaRing, "");

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Column n of an 8-token tile is token (n & ~1) + ((n ^ n / 2) & 1): pairs of
// columns keep rows of both parities, so the 64-byte rows that lanes read
// together fall into different banks for K and for V.
__device__ __forceinline__ int tile_token(int n) { return (n & ~1) + ((n ^ (n >> 1)) & 1); }

// Token (of the block) of piece i of a lane in 16-token step kk.
__device__ __forceinline__ int piece_token(int kk, int i, int t) {
  return 16 * kk + 8 * (i / 2) + tile_token(2 * t + (i & 1));
}
// The lane's pieces of V in step kk; vrow is the block's first row at the lane's channels.
template <int D>
__device__ __forceinline__ void load_v(uint32_t (*v)[D / 32], uint32_t vrow, int kk, int t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = vrow + piece_token(kk, i, t) * D;
    if constexpr (D == 128) {
      const uint4 x = ld_shared_v4(p);
      v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
    } else if constexpr (D == 64) {
      const uint2 x = lds64(p);
      v[i][0] = x.x, v[i][1] = x.y;
    } else {
      v[i][0] = lds32(p);
    }
  }
}

// The product for a block that some query does not see whole.  Codes of no token
// (behind L: any bytes, the NaN code among them) enter as zeros.  A NaN in a
// token that only some queries see would reach the others through 0 x NaN: such a
// block goes query by query, with the tokens that it does not see as zeros.
template <int D, int QT>
__device__ __noinline__ void pv_edge_queries(const uint32_t (*p)[QT][4], uint32_t vrow, int tok0,
                                             const int (*lim)[2], float (*o)[QT][4]) {
  constexpr int VW = D / 32;
  const int lane = lane_id(), g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int q = 0; q < QT; ++q)
#pragma unroll 1
    for (int r = 0; r < 8; ++r) {
      const int lim_r = __shfl_sync(0xffffffffu, r & 1 ? lim[q][1] : lim[q][0], r >> 1);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t pr[1][4], v[4][VW];
        load_v<D>(v, vrow, kk, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[0][k] = g == r ? p[kk][q][k] : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (tok0 + piece_token(kk, k, t) >= lim_r)
#pragma unroll
            for (int w = 0; w < VW; ++w) v[k][w] = 0u;
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          float c[2][1][4] = {};
          pv_words<VW, 1>(pr, v, w, c);
          if (t == (r >> 1))
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              if (r & 1)
                o[2 * w + n][q][1] += c[n][0][1], o[2 * w + n][q][3] += c[n][0][3];
              else
                o[2 * w + n][q][0] += c[n][0][0], o[2 * w + n][q][2] += c[n][0][2];
            }
        }
      }
    }
}
template <int D, int QT>
__device__ __forceinline__ void pv_edge(const uint32_t (*p)[QT][4], uint32_t vrow, int tok0, int L,
                                        const int (*lim)[2], bool masked, float (*o)[QT][4]) {
  constexpr int VW = D / 32;
  const int t = lane_id() & 3;
  uint32_t nan = 0;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    uint32_t v[4][VW];
    load_v<D>(v, vrow, kk, t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 0; w < VW; ++w)
        if (tok0 + piece_token(kk, i, t) < L) nan |= __vcmpeq4(v[i][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  if (masked && __any_sync(0xffffffffu, nan != 0)) {
    float c[D / 16][QT][4] = {};
    uint32_t pc[2][QT][4];
    int lc[QT][2];
#pragma unroll
    for (int q = 0; q < QT; ++q) {
#pragma unroll
      for (int k = 0; k < 4; ++k) pc[0][q][k] = p[0][q][k], pc[1][q][k] = p[1][q][k];
      lc[q][0] = lim[q][0], lc[q][1] = lim[q][1];
    }
    pv_edge_queries<D, QT>(pc, vrow, tok0, lc, c);
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][q][k] += c[n][q][k];
    return;
  }
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    uint32_t v[4][VW];
    load_v<D>(v, vrow, kk, t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (tok0 + piece_token(kk, i, t) >= L)
#pragma unroll
        for (int w = 0; w < VW; ++w) v[i][w] = 0u;
    pv_step<VW, QT>(p[kk], v, o);
  }
}

// The rows of a segment without tokens.
template <int D>
__device__ __forceinline__ void empty_rows(const CacheAttnArgs& a, const Place& p, int tile) {
  const int h = p.seg / a.row_segs, rs = p.seg - h * a.row_segs, first = rs * a.wr * tile;
  const int rows = min(a.R - first, a.wr * tile);
  const long long row = (static_cast<long long>(p.b) * a.Hk + h) * a.R + first;
  uint4* o = reinterpret_cast<uint4*>(a.o + row * D);
  for (int i = threadIdx.x; i < rows * (D / 8); i += kCaThreads) o[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < rows; i += kCaThreads) a.lse[row + i] = -INFINITY;
}

// QT: tiles of 8 queries a warp holds.
template <int D, int RP, int QT, bool MASS>
__global__ void __launch_bounds__(kCaThreads, 3)
    cache_attn_kernel(const CacheAttnArgs a) {
  constexpr int KW = D / 16;                  // K words of a lane and token; QK steps
  constexpr int WW = RP / 16;                 // the same for the factors
  constexpr int VW = D / 32;                  // V words of a lane and token
  constexpr int NT = D / 16;                  // channel tiles of the PV product
  constexpr int QR = 8 * QT;                  // queries of a warp
  extern __shared__ __align__(1024) unsigned char smem[];
  CaHead& head = *reinterpret_cast<CaHead*>(smem);
  const int lane = lane_id(), warp = warp_id();
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % a.wr, wt = warp / a.wr, wts = kCaWarps / a.wr;
  const int stages = a.stages;
  const uint32_t v_off = kCacheBlock * D, w_off = 2 * kCacheBlock * D;
  const uint32_t w_bytes = RP > 0 ? kCacheBlock * a.r : 0, stage_bytes = w_off + w_bytes;
  const uint32_t ring = smem_u32(smem) + kCaRing + wt * stages * stage_bytes;
  const uint32_t full = smem_u32(&head.full[wt][0]), empty = smem_u32(&head.empty[wt][0]);
  if (warp == 0) {
    static_assert(kCaWarps * kCaMaxStages == 32, "one lane a pair of barriers");
    mbar_init(smem_u32(&head.full[0][0]) + 8 * lane, 1);
    mbar_init(smem_u32(&head.empty[0][0]) + 8 * lane, a.wr);
    if (lane == 0) head.abort_flag = head.drain_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitGuard guard{&head.abort_flag, a.err_word, a.wait_ns, a.fail_site};
  grid_dep_wait();
  const int mult = a.Hk * a.row_segs;
  const Place place = a.whole ? segment_of(a, mult) : place_of(a, mult);
  grid_dep_launch_next();
  unsigned at = place.at;
  const unsigned stop = place.stop;
  if (at >= stop) {
    if (a.whole) empty_rows<D>(a, place, QR);
    return;
  }
  int b = place.b, nb = place.nb, seg = place.seg;
  // this CTA's blocks [blk0, blk1) of the segment; none where its part ends within the cost
  const auto first_block = [](unsigned in) {
    return static_cast<int>(max(in, kCaSegmentCost) - kCaSegmentCost);
  };
  unsigned in = place.in;
  int blk0 = first_block(in), blk1 = min(nb, first_block(in + (stop - at)));
  const int seg_rows = min(a.R, QR * a.wr);
  bool first = true, dead = false;
  const bool leader = wr == 0;
  // ring position of the next block to load and to use, and its phase
  int in_stage = 0, in_phase = 0, out_stage = 0, out_phase = 0;
  int loads = 0;   // copies this warp started (the ring's s-th stage got loads s, s + stages, ...)
  int issued = 0;  // blocks of this segment (and the next) loaded by this group so far
  // lanes 0, 1, 2 copy K, V, W; each keeps where its next block starts
  const bool copies = lane < (RP > 0 ? 3 : 2);
  const uint8_t* const my_base = lane == 0 ? a.k : lane == 1 ? a.v : a.w;
  const float* const my_scales = lane == 0 ? a.ks : lane == 1 || RP == 0 ? a.vs : a.ws;
  const unsigned my_width = lane < 2 ? D : a.r, my_bytes = kCacheBlock * my_width;
  const unsigned my_step = wts * my_bytes;
  const uint8_t* src = nullptr;

  while (at < stop) {
    const int h = seg / a.row_segs, rs = seg - h * a.row_segs;
    const int L = min(a.lengths[b], a.cap);
    const long long bh = static_cast<long long>(b) * a.Hk + h;
    const int row0 = (rs * a.wr + wr) * QR;
    // the segment after this one
    const unsigned next_at = at + (nb + kCaSegmentCost - in);
    int nseg = seg + 1, nxb = b, nnb = nb;
    if (nseg == mult && next_at < stop) {
      nseg = 0;
      do {
        ++nxb;
      } while (nxb < a.B && cache_blocks(a, nxb) == 0);
      if (nxb < a.B) nnb = cache_blocks(a, nxb);
    }
    const int nblk1 = next_at < stop ? min(nnb, first_block(stop - next_at)) : 0;
    const int mine = max(blk1 - blk0 - wt + wts - 1, 0) / wts;      // this group's blocks here
    const int ahead = mine + max(nblk1 - wt + wts - 1, 0) / wts;    // and with the next segment's
    const long long nbh = static_cast<long long>(nxb) * a.Hk + nseg / a.row_segs;

    if (first) src = my_base + (bh * a.cap + (blk0 + wt) * kCacheBlock) * my_width;
    const uint8_t* const next_src = my_base + (nbh * a.cap + wt * kCacheBlock) * my_width;
    if (issued == mine) src = next_src;
    // Loads blocks until `upto` of them (counted from this segment's first) are under way.
    const auto pump = [&](int upto) {
      for (upto = min(upto, ahead); issued < upto;) {
        if (leader && !dead) {
          bool ok = true;
          if (a.wr > 1) ok = wait_warp(empty + 8 * in_stage, in_phase ^ 1, guard, 70);
          if (!ok) dead = true;
          if (ok) {
            const uint32_t bar = full + 8 * in_stage;
            if (lane == 0) mbar_expect_tx(bar, stage_bytes);
            if (copies) bulk_load(ring + in_stage * stage_bytes + lane * v_off, src, my_bytes, bar);
          }
          loads += ok;
        }
        if (++in_stage == stages) in_stage = 0, in_phase ^= 1;
        src = ++issued == mine ? next_src : src + my_step;
      }
    };
    // The queries are asked for before the blocks: behind a ring full of them they
    // would wait for all of it.
    uint2 raw_q[QT][KW], raw_u[QT][WW > 0 ? WW : 1];
    if (blk0 < blk1) {
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const int row = row0 + 8 * q + g;
        fetch_row<D, false>(a.q + (bh * a.R + row) * D, D, row < a.R, t, raw_q[q]);
        if constexpr (RP > 0)
          fetch_row<RP, true>(a.u + (bh * a.R + row) * a.r, a.r, row < a.R, t, raw_u[q]);
      }
    }
    // the block's scales, one in each of lanes 0, 1, 2
    const float* scales = my_scales + bh * (a.cap / kCacheBlock) + blk0 + wt;
    float scale = 0.f;
    if (copies && mine > 0) scale = __ldg(scales);
    // One block a group at first: a ring asked for whole at the start comes in the
    // order of the asking, and its last stages would hold up the others' first ones.
    pump(max(issued, 1));
    if (blk0 == blk1) break;  // only at the end of the part

    // Queries as B fragments (lane g: query g of each tile); scores, sums and O are
    // held for queries 2 t, 2 t + 1.
    uint32_t qf[QT][KW][2], uf[QT][WW > 0 ? WW : 1][2];
    float fq[QT][2], fu[QT][2];
    int lim[QT][2], lim_lo = L;  // tokens the query sees
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      const int row = row0 + 8 * q + g;
      const float f = row_fragments<D>(raw_q[q], qf[q]) * a.scale_log2;
      float e = 0.f;
      if constexpr (RP > 0) e = row_fragments<RP>(raw_u[q], uf[q]) * kLog2e;
      const int n = row_sees(a, b, row, L);
      lim_lo = min(lim_lo, n);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int from = 4 * (2 * t + k);
        fq[q][k] = __shfl_sync(0xffffffffu, f, from);
        fu[q][k] = __shfl_sync(0xffffffffu, e, from);
        lim[q][k] = __shfl_sync(0xffffffffu, n, from);
      }
    }
    lim_lo = __reduce_min_sync(0xffffffffu, lim_lo);

    // Weights are 2^(x - m), m the largest score up to a slack, less the lift: m moves (and
    // with it the sums) only when a score passes `over`.
    float m[QT][2], over[QT][2], l[QT][2], oacc[NT][QT][4];
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      m[q][0] = m[q][1] = 0.f;
      over[q][0] = over[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) oacc[i][q][k] = 0.f;
    }
    float unit = 1.f;  // oacc is O / unit

    pump(max(issued, 2));
    uint32_t held = 0;  // stage of the segment's last block: the warps join through it

    for (int i = 0; i < mine; ++i) {
      const int blk = blk0 + wt + i * wts;
      if (!wait_warp(full + 8 * out_stage, out_phase, guard, 71)) dead = true;
      const uint32_t st = ring + out_stage * stage_bytes;
      const float ks_now = __shfl_sync(0xffffffffu, scale, 0);
      const float vs_now = __shfl_sync(0xffffffffu, scale, 1);
      const float ws_now = RP > 0 ? __shfl_sync(0xffffffffu, scale, 2) : 0.f;
      scales += wts;
      if (copies && i + 1 < mine) scale = __ldg(scales);
      // scores in units of log2: x[j][q] of tokens g, g + 8 of half j (as tile_token
      // orders them) and queries 2 t, 2 t + 1
      float x[2][QT][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t kr[2][KW];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t p = st + (16 * j + 8 * e + tile_token(g)) * D;
          if constexpr (D >= 64) {
#pragma unroll
            for (int c = 0; c < KW / 4; ++c) {
              const uint4 v = ld_shared_v4(p + 64 * c + 16 * t);
              kr[e][4 * c] = v.x, kr[e][4 * c + 1] = v.y;
              kr[e][4 * c + 2] = v.z, kr[e][4 * c + 3] = v.w;
            }
          } else {
            const uint2 v = lds64(p + 8 * t);
            kr[e][0] = v.x, kr[e][1] = v.y;
          }
        }
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[j][q][k] = 0.f;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const uint32_t af[4] = {e4m3_lo(kr[0][k]), e4m3_lo(kr[1][k]), e4m3_hi(kr[0][k]),
                                  e4m3_hi(kr[1][k])};
#pragma unroll
          for (int q = 0; q < QT; ++q) mma_f16(x[j][q], af, qf[q][k][0], qf[q][k][1]);
        }
        if constexpr (RP > 0) {
          uint32_t wreg[2][WW];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t pw = st + w_off + (16 * j + 8 * e + tile_token(g)) * a.r;
#pragma unroll
            for (int k = 0; k < WW; ++k) wreg[e][k] = 0;
            if constexpr (RP == 16) {
              if (4 * t < a.r) wreg[e][0] = lds32(pw + 4 * t);
            } else {
#pragma unroll
              for (int k = 0; k < WW / 2; ++k) {
                const int ch = factor_channel<RP>(2 * k, t);
                if (ch < a.r) {
                  const uint2 v = lds64(pw + ch);
                  wreg[e][2 * k] = v.x, wreg[e][2 * k + 1] = v.y;
                }
              }
            }
          }
          float cw[QT][4] = {};
#pragma unroll
          for (int k = 0; k < WW; ++k) {
            const uint32_t af[4] = {e4m3_lo(wreg[0][k]), e4m3_lo(wreg[1][k]), e4m3_hi(wreg[0][k]),
                                    e4m3_hi(wreg[1][k])};
#pragma unroll
            for (int q = 0; q < QT; ++q) mma_f16(cw[q], af, uf[q][k][0], uf[q][k][1]);
          }
#pragma unroll
          for (int q = 0; q < QT; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[j][q][k] = fmaf(cw[q][k], fu[q][k & 1] * ws_now, x[j][q][k] * (fq[q][k & 1] * ks_now));
        } else {
#pragma unroll
          for (int q = 0; q < QT; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[j][q][k] *= fq[q][k & 1] * ks_now;
        }
      }
      const bool edge = (blk + 1) * kCacheBlock > lim_lo;  // a query does not see all of the block
      if (edge) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < QT; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (blk * kCacheBlock + 16 * j + 8 * (k >> 1) + tile_token(g) >= lim[q][k & 1])
                x[j][q][k] = -INFINITY;
      }
      if constexpr (MASS) {
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = row0 + 8 * q + 2 * t + e;
            if (row < a.R) {
              float* s = a.scores + (bh * a.R + row) * a.cap + blk * kCacheBlock + tile_token(g);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                s[16 * j] = x[j][q][e], s[16 * j + 8] = x[j][q][2 + e];
            }
          }
      }
      float mx[QT][2];
      bool moved = vs_now != unit;
#pragma unroll
      for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[q][e] = fmaxf(fmax3(x[0][q][e], x[0][q][2 + e], x[1][q][e]), x[1][q][2 + e]);
          moved |= mx[q][e] > over[q][e];
        }
      if (__any_sync(0xffffffffu, moved)) {
        const float back = unit / vs_now;
        unit = vs_now;
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = mx[q][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            al[e] = 1.f;
            if (v > over[q][e]) {
              const bool fine = fabsf(v) < kCaCoarse;
              v -= fine ? kCaLift : 0.f;
              al[e] = over[q][e] == -INFINITY ? 0.f : fast_exp2(m[q][e] - v);
              m[q][e] = v;
              over[q][e] = v + (fine ? kCaLift + kCaSlack : 0.f);
            }
            l[q][e] *= al[e];
            al[e] *= back;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) oacc[n][q][k] *= al[k & 1];
        }
      }
      uint32_t p[2][QT][4];
#pragma unroll
      for (int q = 0; q < QT; ++q) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[j][q][k] = fast_exp2(x[j][q][k] - m[q][k & 1]);
            l[q][k & 1] += x[j][q][k];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t high = pack_f16x2(x[j][q][2 * e], x[j][q][2 * e + 1]);
            const float2 h = f16x2_to_f32x2(high);
            p[j][q][e] = transpose8x8(high);
            p[j][q][2 + e] =
                transpose8x8(pack_f16x2(x[j][q][2 * e] - h.x, x[j][q][2 * e + 1] - h.y));
          }
        }
      }
      // O^T += V^T P^T
      const uint32_t vrow = st + v_off + g * (D / 8);
      if (!edge) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          uint32_t v[4][VW];
          load_v<D>(v, vrow, kk, t);
          pv_step<VW, QT>(p[kk], v, oacc);
        }
      } else {
        pv_edge<D, QT>(p, vrow, blk * kCacheBlock, L, lim, masked(a), oacc);
      }
      held = st;
      __syncwarp();  // the stage has been read
      if (a.wr > 1 && lane == 0 && i + 1 < mine) mbar_arrive(empty + 8 * out_stage);
      if (i + 1 < mine) {
        if (++out_stage == stages) out_stage = 0, out_phase ^= 1;
        pump(min(i + 1 + stages, 2 * i + 4));
      }
    }

    // Join the warps that share rows: the groups behind the first leave O in a
    // stage that is read out (tile wr in that of group wr, or their own), the
    // first adds them to its own.  Channel g (D / 8) + 2 n + i of query 2 t + e is
    // oacc[n][q][2 i + e].
#pragma unroll
    for (int q = 0; q < QT; ++q) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], o);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) oacc[n][q][k] *= unit;
    }
    // rows that saw nothing
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (over[q][e] == -INFINITY) m[q][e] = -INFINITY;
    const bool whole = blk0 == 0 && blk1 == nb;
    const int slot = first ? 0 : 1;
    if (wts > 1) {
      if (lane == 0 && wr == 0) head.held[wt] = mine > 0 ? held : 0u;
      if (g == 0) {
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            head.ml[warp][8 * q + 2 * t + e] = make_float2(m[q][e], l[q][e]);
      }
      __syncthreads();
      const uint32_t buf = head.held[a.wr == 1 ? wt : wr];
      static_assert(QT <= 2, "O of a warp has to fit into a stage's K and V");
      if (wt > 0 && mine > 0) {
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            st_shared_v4(buf + ((q * NT + n) * 32 + lane) * 16, __float_as_uint(oacc[n][q][0]),
                         __float_as_uint(oacc[n][q][1]), __float_as_uint(oacc[n][q][2]),
                         __float_as_uint(oacc[n][q][3]));
      }
      __syncthreads();
      if (wt == 0) {
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          float mm[2] = {m[q][0], m[q][1]}, base[2], f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            for (int w = 1; w < wts; ++w)
              mm[e] = fmaxf(mm[e], head.ml[w * a.wr + wr][8 * q + 2 * t + e].x);
            base[e] = mm[e] == -INFINITY ? 0.f : mm[e];
            f[e] = fast_exp2(m[q][e] - base[e]);
            l[q][e] *= f[e];
            m[q][e] = mm[e];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) oacc[n][q][k] *= f[k & 1];
          for (int w = 1; w < wts; ++w) {
            if (blk0 + w >= blk1) break;  // groups from here on had no block
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 ml = head.ml[w * a.wr + wr][8 * q + 2 * t + e];
              f[e] = fast_exp2(ml.x - base[e]);
              l[q][e] = fmaf(ml.y, f[e], l[q][e]);
            }
            const uint32_t from = head.held[a.wr == 1 ? w : wr];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 v = ld_shared_v4(from + ((q * NT + n) * 32 + lane) * 16);
              oacc[n][q][0] = fmaf(__uint_as_float(v.x), f[0], oacc[n][q][0]);
              oacc[n][q][1] = fmaf(__uint_as_float(v.y), f[1], oacc[n][q][1]);
              oacc[n][q][2] = fmaf(__uint_as_float(v.z), f[0], oacc[n][q][2]);
              oacc[n][q][3] = fmaf(__uint_as_float(v.w), f[1], oacc[n][q][3]);
            }
          }
        }
      }
    }
    if (wt == 0) {
#pragma unroll
      for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = row0 + 8 * q + 2 * t + e;
          if (row >= a.R) continue;
          if (whole) {
            // no token seen: O = 0; NaN stays
            const float inv = l[q][e] > 0.f ? 1.f / l[q][e] : l[q][e];
            const long long out = bh * a.R + row;
            uint32_t w[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
              w[n] = pack_bf16x2(oacc[n][q][e] * inv, oacc[n][q][2 + e] * inv);
            uint32_t* o = reinterpret_cast<uint32_t*>(a.o + out * D + g * (D / 8));
            if constexpr (NT >= 4) {
#pragma unroll
              for (int n = 0; n < NT; n += 4)
                *reinterpret_cast<uint4*>(o + n) = make_uint4(w[n], w[n + 1], w[n + 2], w[n + 3]);
            } else {
              *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
            }
            if (g == 0) a.lse[out] = (m[q][e] + __log2f(l[q][e])) * kLn2;
          } else {
            const long long r =
                (static_cast<long long>(blockIdx.x) * 2 + slot) * seg_rows + (row - rs * a.wr * QR);
            float4* o = reinterpret_cast<float4*>(a.part_o + r * D + g * (D / 8));
#pragma unroll
            for (int n = 0; n < NT; n += 2)
              o[n / 2] = make_float4(oacc[n][q][e], oacc[n][q][2 + e], oacc[n + 1][q][e],
                                     oacc[n + 1][q][2 + e]);
            if (g == 0) a.part_ml[r] = make_float2(m[q][e], l[q][e]);
          }
        }
    }
    // the held stages go back to the ring
    if (wts > 1) {
      fence_async_smem();
      __syncthreads();
    }
    if (mine > 0) {
      if (a.wr > 1 && lane == 0) mbar_arrive(empty + 8 * out_stage);
      if (++out_stage == stages) out_stage = 0, out_phase ^= 1;
    }
    issued -= mine;
    first = false;
    at = next_at;
    b = nxb, seg = nseg, nb = nnb;
    in = 0;
    blk0 = 0;
    blk1 = nblk1;
  }
  // every copy has been waited for above, unless a wait gave up
  if (dead && leader) {
    const WaitGuard drain{&head.drain_flag, a.err_word, kDrainTimeoutNs, -1};
    for (int s = 0; s < min(stages, loads); ++s)
      wait_bounded(full + 8 * s, ((loads - 1 - s) / stages) & 1, drain, 72);
  }
}

// Where the partials of segment (b, seg) lie: CTAs i0 .. i1 hold blocks of it, each
// as its first segment (slot 0), but for one that began in an earlier one.
struct Parts {
  unsigned i0, n;  // n == 0: no token; 1: the CTA finished the segment itself
  unsigned late;
  __device__ __forceinline__ long long index(unsigned k, int seg_rows, int rr) const {
    return (static_cast<long long>(i0 + k) * 2 + (k == 0 ? late : 0u)) * seg_rows + rr;
  }
};
__device__ __forceinline__ Parts parts_of(const CacheAttnArgs& a, int b, int seg, unsigned ctas) {
  if (a.whole) return Parts{0, cache_blocks(a, b) > 0 ? 1u : 0u, 0};
  const int mult = a.Hk * a.row_segs;
  unsigned before, total;
  count_line(a, b, before, total);
  const unsigned len = line_length(cache_blocks(a, b));
  if (len == 0) return Parts{0, 0, 0};
  const unsigned s0 = before * mult + seg * len;
  const Cut cut(total * mult, ctas);
  const unsigned i0 = cut.holder(s0 + kCaSegmentCost), i1 = cut.holder(s0 + len - 1);
  return Parts{i0, i1 - i0 + 1, cut.start(i0) < s0 ? 1u : 0u};
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// LSE in log2 units of the up to 8 rows of key head bh, joined from the partials
// again, so that the mass needs no kernel behind the join of O; +inf for rows that
// see nothing, whose weights are 0.  All 128 threads call it.
__device__ __forceinline__ void join_lse(const CacheAttnArgs& a, unsigned ctas, int bh, float* lse2) {
  const int b = bh / a.Hk, h = bh - b * a.Hk;
  const Parts parts = parts_of(a, b, h, ctas);
  const int row = threadIdx.x / 16, lane = threadIdx.x % 16;
  if (row >= a.R) return;  // whole half warps leave together
  const unsigned half = 0xffffu << (threadIdx.x & 16);
  float z;
  if (parts.n == 1) {
    z = __ldcg(a.lse + static_cast<long long>(bh) * a.R + row) * kLog2e;
  } else {
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (unsigned k = lane; k < parts.n; k += 16) {
      const float2 ml = __ldcg(a.part_ml + parts.index(k, a.R, row));
      const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
      l = l * fast_exp2(m - base) + ml.y * fast_exp2(ml.x - base);
      m = mn;
    }
    float top = m;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(half, top, o));
    l *= fast_exp2(m - (top == -INFINITY ? 0.f : top));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) l += __shfl_xor_sync(half, l, o);
    z = top + __log2f(l);
  }
  if (lane == 0) lse2[row] = z == -INFINITY ? INFINITY : z;
}

__device__ __forceinline__ void store_mass(const CacheAttnArgs& a, long long at, float add) {
  a.mass_out[at] = a.mass ? fmaf(a.decay, a.mass[at], add) : add;
}

// mass_out = decay mass + sum over the key head's rows of exp(x - LSE).  Up to 8
// rows leave their scores in the workspace (8 bytes of traffic a row and token, less
// than reading K again: a decode step 25.1 us against 39.5, 8 rows a key head 16.2
// against 19.3); with more rows the scores are computed again, beside the join
// where a segment has few partials, else behind it.

// From the scores: the warps of a CTA that share tokens take every
// mass_row_warps-th row each.
__host__ __device__ __forceinline__ int mass_row_warps(int R) { return R >= 4 ? 4 : R >= 2 ? 2 : 1; }
__host__ __device__ __forceinline__ int mass_tokens(int R) { return 512 / mass_row_warps(R); }

__device__ __forceinline__ void add_mass(const CacheAttnArgs& a, unsigned ctas, int bh, int chunk) {
  __shared__ float lse2[8];
  __shared__ float4 part[3][32];
  const int rw = mass_row_warps(a.R), warp = warp_id(), lane = lane_id();
  const int t0 = chunk * mass_tokens(a.R) + (warp / rw) * 128 + lane * 4;
  const int L = min(a.lengths[bh / a.Hk], a.cap);
  if (chunk * mass_tokens(a.R) >= L) return;
  join_lse(a, ctas, bh, lse2);
  __syncthreads();
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* s = a.scores + static_cast<long long>(bh) * a.R * a.cap + t0;
  if (t0 < L) {
#pragma unroll 8
    for (int i = warp % rw; i < a.R; i += rw) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(s + static_cast<long long>(i) * a.cap));
      const float z = lse2[i];
      sum.x += fast_exp2(x.x - z), sum.y += fast_exp2(x.y - z);
      sum.z += fast_exp2(x.z - z), sum.w += fast_exp2(x.w - z);
    }
  }
  if (rw > 1) {
    if (warp % rw) part[warp / rw * (rw - 1) + warp % rw - 1][lane] = sum;
    __syncthreads();
    if (warp % rw) return;
    for (int i = 0; i < rw - 1; ++i) {
      const float4 v = part[warp / rw * (rw - 1) + i][lane];
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
  }
  const float add[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t0 + k < L) store_mass(a, static_cast<long long>(bh) * a.cap + t0 + k, add[k]);
}

// Computed again: a warp holds a block of 32 tokens of K (and W) as MMA row operands
// and goes over all rows, 64 at a time from shared memory, as the main kernel does but
// with the final LSE; the weights of a token add up over the lanes of its row.
// Two blocks a warp (half the CTAs, 160 registers for 126) measured the same.
constexpr int kMassChunk = 4 * kCacheBlock;
constexpr int kMassRows = 64;

// LSE in log2 units of row r0 + threadIdx.x / 2, by two threads, for the 128 of a CTA;
// +inf for rows that see nothing and for those from r0 + rows on.
__device__ __forceinline__ float join_lse_row(const CacheAttnArgs& a, const Parts& parts, int bh,
                                              int r0, int rows) {
  const int rr = threadIdx.x / 2, seg_rows = min(a.R, a.tile * a.wr);
  float z = INFINITY;
  if (rr < rows && parts.n == 1) {
    z = __ldcg(a.lse + static_cast<long long>(bh) * a.R + r0 + rr) * kLog2e;
  } else if (rr < rows) {
    float m = -INFINITY, l = 0.f;
#pragma unroll 8
    for (unsigned k = threadIdx.x & 1; k < parts.n; k += 2) {
      const float2 ml = __ldcg(a.part_ml + parts.index(k, seg_rows, rr));
      const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
      l = l * fast_exp2(m - base) + ml.y * fast_exp2(ml.x - base);
      m = mn;
    }
    const unsigned both = 3u << (threadIdx.x & 30);
    const float top = fmaxf(m, __shfl_xor_sync(both, m, 1));
    l *= fast_exp2(m - (top == -INFINITY ? 0.f : top));
    z = top + __log2f(l + __shfl_xor_sync(both, l, 1));
  }
  return z == -INFINITY ? INFINITY : z;
}

// Pieces of `e4m3 rows` (two, tile_token(g) and 8 behind) of C channels as the MMA's row operand.
template <int W>
__device__ __forceinline__ void row_operand(const uint32_t (*r)[W], uint32_t (*f)[4]) {
#pragma unroll
  for (int k = 0; k < W; ++k) {
    f[k][0] = e4m3_lo(r[0][k]), f[k][1] = e4m3_lo(r[1][k]);
    f[k][2] = e4m3_hi(r[0][k]), f[k][3] = e4m3_hi(r[1][k]);
  }
}

// FROM_PARTS: the rows' LSE comes from the partials, so that the join of O is not waited
// for; else from a.lse.
template <int D, int RP, bool FROM_PARTS>
__device__ __forceinline__ void recompute_mass(const CacheAttnArgs& a, unsigned ctas, int bh,
                                               int chunk) {
  constexpr int KW = D / 16, WW = RP / 16;
  __shared__ uint2 sq[8][KW][32], su[WW > 0 ? 8 : 1][WW > 0 ? WW : 1][32];
  __shared__ float4 row_of[64];  // factors of K's and W's scores, -LSE, tokens seen
  __shared__ int fewest[4];      // of the warp's rows, tokens seen by the one that sees fewest
  const int b = bh / a.Hk, warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const int L = min(a.lengths[b], a.cap);
  if (chunk * kMassChunk >= L) return;
  const int blk = chunk * 4 + warp, tok0 = blk * kCacheBlock;
  const bool busy = tok0 < L;
  // the block, on its way while the rows are prepared
  uint32_t kr[2][2][KW], wr[2][2][WW > 0 ? WW : 1];
  float ks = 0.f, ws = 0.f;
  if (busy) {
    const long long line = static_cast<long long>(bh) * a.cap + tok0;
    const long long sat = static_cast<long long>(bh) * (a.cap / kCacheBlock) + blk;
    ks = __ldg(a.ks + sat);
    if constexpr (RP > 0) ws = __ldg(a.ws + sat);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const long long row = line + 16 * j + 8 * e + tile_token(g);
        const uint8_t* p = a.k + row * D;
        if constexpr (D >= 64) {
#pragma unroll
          for (int c = 0; c < KW / 4; ++c) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + 64 * c + 16 * t));
            kr[j][e][4 * c] = v.x, kr[j][e][4 * c + 1] = v.y;
            kr[j][e][4 * c + 2] = v.z, kr[j][e][4 * c + 3] = v.w;
          }
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + 8 * t));
          kr[j][e][0] = v.x, kr[j][e][1] = v.y;
        }
        if constexpr (RP > 0) {
          p = a.w + row * a.r;
#pragma unroll
          for (int k = 0; k < WW; ++k) wr[j][e][k] = 0;
          if constexpr (RP == 16) {
            if (4 * t < a.r) wr[j][e][0] = __ldg(reinterpret_cast<const uint32_t*>(p + 4 * t));
          } else {
#pragma unroll
            for (int k = 0; k < WW / 2; ++k) {
              const int ch = factor_channel<RP>(2 * k, t);
              if (ch < a.r) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + ch));
                wr[j][e][2 * k] = v.x, wr[j][e][2 * k + 1] = v.y;
              }
            }
          }
        }
      }
  }
  float sum[2][2] = {};
  static_assert(kMassRows == 64, "a segment's rows, where there are several");
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    Parts parts;
    if constexpr (FROM_PARTS)
      parts = parts_of(a, b, (bh - b * a.Hk) * a.row_segs + r0 / kMassRows, ctas);
    const int rows = min(64, a.R - r0);
    if (r0 > 0) __syncthreads();  // the rows before have been read
    uint2 raw[2][KW], raw_u[2][WW > 0 ? WW : 1];
    int few = L;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (8 * (warp + 4 * i) >= rows) break;
      const long long row = r0 + 8 * (warp + 4 * i) + g, line = static_cast<long long>(bh) * a.R + row;
      fetch_row<D, false>(a.q + line * D, D, row < a.R, t, raw[i]);
      if constexpr (RP > 0) fetch_row<RP, true>(a.u + line * a.r, a.r, row < a.R, t, raw_u[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = warp + 4 * i, row = r0 + 8 * q + g;
      if (8 * q >= rows) break;
      uint32_t frag[KW][2], uf[WW > 0 ? WW : 1][2];
      const float f = row_fragments<D>(raw[i], frag) * a.scale_log2;
#pragma unroll
      for (int k = 0; k < KW; ++k) sq[q][k][lane] = make_uint2(frag[k][0], frag[k][1]);
      float e = 0.f;
      if constexpr (RP > 0) {
        e = row_fragments<RP>(raw_u[i], uf) * kLog2e;
#pragma unroll
        for (int k = 0; k < WW; ++k) su[q][k][lane] = make_uint2(uf[k][0], uf[k][1]);
      }
      // a row that is none weighs nothing (its LSE is +inf)
      const int lim = row_sees(a, b, row, L);
      few = min(few, lim);
      if (t == 0) row_of[8 * q + g] = make_float4(f, e, 0.f, __int_as_float(lim));
    }
    few = __reduce_min_sync(0xffffffffu, few);
    if (lane == 0) fewest[warp] = few;
    __syncthreads();
    if constexpr (FROM_PARTS) {
      const float z = join_lse_row(a, parts, bh, r0, rows);
      if ((threadIdx.x & 1) == 0) row_of[threadIdx.x / 2].z = -z;
    } else if (threadIdx.x < 64) {
      const float z = threadIdx.x < rows
                          ? __ldcg(a.lse + static_cast<long long>(bh) * a.R + r0 + threadIdx.x) * kLog2e
                          : INFINITY;
      row_of[threadIdx.x].z = z == -INFINITY ? -INFINITY : -z;
    }
    __syncthreads();
    if (!busy) continue;
    const int tiles = (rows + 7) / 8;
    uint32_t af[2][KW][4], wf[2][WW > 0 ? WW : 1][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      row_operand<KW>(kr[j], af[j]);
      if constexpr (RP > 0) row_operand<WW>(wr[j], wf[j]);
    }
    const bool edge = tok0 + kCacheBlock > min(min(fewest[0], fewest[1]), min(fewest[2], fewest[3]));
#pragma unroll 2
    for (int q = 0; q < tiles; ++q) {
      const float4 of[2] = {row_of[8 * q + 2 * t], row_of[8 * q + 2 * t + 1]};
      const float f[2] = {of[0].x * ks, of[1].x * ks}, z[2] = {of[0].z, of[1].z};
      float x[2][4] = {};
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const uint2 v = sq[q][k][lane];
        mma_f16(x[0], af[0][k], v.x, v.y);
        mma_f16(x[1], af[1][k], v.x, v.y);
      }
      if constexpr (RP > 0) {
        float cw[2][4] = {};
#pragma unroll
        for (int k = 0; k < WW; ++k) {
          const uint2 v = su[q][k][lane];
          mma_f16(cw[0], wf[0][k], v.x, v.y);
          mma_f16(cw[1], wf[1][k], v.x, v.y);
        }
        const float e[2] = {of[0].y * ws, of[1].y * ws};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[j][k] = fmaf(cw[j][k], e[k & 1], fmaf(x[j][k], f[k & 1], z[k & 1]));
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[j][k] = fmaf(x[j][k], f[k & 1], z[k & 1]);
      }
      if (edge) {
        const int lim[2] = {__float_as_int(of[0].w), __float_as_int(of[1].w)};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (tok0 + 16 * j + 8 * (k >> 1) + tile_token(g) >= lim[k & 1]) x[j][k] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[j][k >> 1] += fast_exp2(x[j][k]);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = sum[j][e];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      const int tok = tok0 + 16 * j + 8 * e + tile_token(g);
      if (t == 0 && tok < L) store_mass(a, static_cast<long long>(bh) * a.cap + tok, v);
    }
}

// No query: what is there decays.
__global__ void __launch_bounds__(128) cache_decay_kernel(const CacheAttnArgs a) {
  grid_dep_wait();
  const int t = blockIdx.y * 128 + threadIdx.x;
  if (t < min(a.lengths[blockIdx.x / a.Hk], a.cap))
    store_mass(a, static_cast<long long>(blockIdx.x) * a.cap + t, 0.f);
}

// The weights alone, behind the join.
template <int D, int RP>
__global__ void __launch_bounds__(128) cache_mass_kernel(const CacheAttnArgs a) {
  grid_dep_wait();
  recompute_mass<D, RP, false>(a, 0, blockIdx.x, blockIdx.y);
}

// Rows of a CTA of the join: with up to 8 rows or many partials a segment one, whose
// partials go to D / 4 threads each, as many at once as fit; else as many rows as fit,
// each going over its partials in turn (64 rows of 14 partials, with the weights beside
// the join: 34.9 us against 36.7 one by one; 16 rows of 56: 41.4 against 32.8, 64 of 222:
// 92 against 70).
constexpr int kJoinFew = 16;
__host__ __device__ __forceinline__ int join_rows(int seg_rows, int d, unsigned partials) {
  return seg_rows <= 8 || partials > kJoinFew ? 1 : 128 / (d / 4);
}

template <int D>
__device__ __forceinline__ void store_row(const CacheAttnArgs& a, long long out, int c, float m,
                                          float l, float4 acc) {
  const float inv = l > 0.f ? 1.f / l : l;
  *reinterpret_cast<uint2*>(a.o + out * D + c) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0) a.lse[out] = (m + __log2f(l)) * kLn2;
}

// Joins the partials of a (b, h, row segment) that several CTAs share, in their
// order; writes the rows of an empty sequence.
template <int D>
__device__ __forceinline__ void join_many(const CacheAttnArgs& a, const Parts& parts, int bh, int rs,
                                          int first) {
  constexpr int TPR = D / 4;
  const int seg_rows = min(a.R, a.tile * a.wr), c = (threadIdx.x % TPR) * 4;
  const int rr = first + threadIdx.x / TPR, row = rs * a.wr * a.tile + rr;
  if (rr >= seg_rows || row >= a.R) return;
  const long long out = static_cast<long long>(bh) * a.R + row;
  if (parts.n == 0) {
    *reinterpret_cast<uint2*>(a.o + out * D + c) = make_uint2(0, 0);
    if (c == 0) a.lse[out] = -INFINITY;
    return;
  }
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr unsigned AT = 8;  // partials on their way at once
  for (unsigned k0 = 0; k0 < parts.n; k0 += AT) {
    float2 ml[AT];
    float4 v[AT];
#pragma unroll
    for (unsigned k = 0; k < AT; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < parts.n) {
        const long long p = parts.index(k0 + k, seg_rows, rr);
        ml[k] = __ldcg(a.part_ml + p);
        v[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + p * D + c));
      }
    }
    float mn = m;
#pragma unroll
    for (unsigned k = 0; k < AT; ++k) mn = fmaxf(mn, ml[k].x);
    const float base = mn == -INFINITY ? 0.f : mn, back = fast_exp2(m - base);
    m = mn;
    l *= back;
    acc.x *= back, acc.y *= back, acc.z *= back, acc.w *= back;
#pragma unroll
    for (unsigned k = 0; k < AT; ++k) {
      const float f = fast_exp2(ml[k].x - base);
      l = fmaf(ml[k].y, f, l);
      acc.x = fmaf(v[k].x, f, acc.x), acc.y = fmaf(v[k].y, f, acc.y);
      acc.z = fmaf(v[k].z, f, acc.z), acc.w = fmaf(v[k].w, f, acc.w);
    }
  }
  store_row<D>(a, out, c, m, l, acc);
}

template <int D>
__device__ __forceinline__ void join_one(const CacheAttnArgs& a, const Parts& parts, int bh, int rs,
                                         int rr) {
  constexpr int TPR = D / 4, PAR = 128 / TPR;
  __shared__ float weight[128];
  __shared__ float4 sum[128];
  __shared__ float s_max[4], s_l[4];
  const int seg_rows = min(a.R, a.tile * a.wr);
  const int c = (threadIdx.x % TPR) * 4, part = threadIdx.x / TPR, warp = warp_id();
  const int row = rs * a.wr * a.tile + rr;
  if (row >= a.R) return;
  const long long out = static_cast<long long>(bh) * a.R + row;
  const unsigned n = parts.n;
  if (n == 0) {
    if (part == 0) *reinterpret_cast<uint2*>(a.o + out * D + c) = make_uint2(0, 0);
    if (threadIdx.x == 0) a.lse[out] = -INFINITY;
    return;
  }
  // the values come with the statistics: up to 128 partials wait for one trip to memory
  float m = -INFINITY;
  for (unsigned k = threadIdx.x; k < n; k += 128)
    m = fmaxf(m, __ldcg(a.part_ml + parts.index(k, seg_rows, rr)).x);
  constexpr int AHEAD = 8;
  float4 v[AHEAD];
#pragma unroll
  for (unsigned j = 0; j < AHEAD; ++j)
    if (part + j * PAR < n)
      v[j] = __ldcg(reinterpret_cast<const float4*>(
          a.part_o + parts.index(part + j * PAR, seg_rows, rr) * D + c));
  m = warp_max(m);
  if (lane_id() == 0) s_max[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (unsigned k0 = 0; k0 < n; k0 += 128) {
    const unsigned k = k0 + threadIdx.x;
    if (k < n) {
      const float2 ml = __ldcg(a.part_ml + parts.index(k, seg_rows, rr));
      const float f = fast_exp2(ml.x - base);
      weight[threadIdx.x] = f;
      l = fmaf(ml.y, f, l);
    }
    __syncthreads();
    const unsigned top = min(128u, n - k0);
    if (k0 == 0) {
#pragma unroll
      for (unsigned j = 0; j < AHEAD; ++j)
        if (part + j * PAR < top) {
          const float f = weight[part + j * PAR];
          acc.x = fmaf(v[j].x, f, acc.x), acc.y = fmaf(v[j].y, f, acc.y);
          acc.z = fmaf(v[j].z, f, acc.z), acc.w = fmaf(v[j].w, f, acc.w);
        }
    }
#pragma unroll 4
    for (unsigned j = part + (k0 == 0 ? AHEAD * PAR : 0); j < top; j += PAR) {
      const float f = weight[j];
      const float4 x = __ldcg(reinterpret_cast<const float4*>(
          a.part_o + parts.index(k0 + j, seg_rows, rr) * D + c));
      acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
    }
    __syncthreads();
  }
  l = warp_sum(l);
  if (lane_id() == 0) s_l[warp] = l;
  sum[threadIdx.x] = acc;
  __syncthreads();
  if (part != 0) return;
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  for (int p = 1; p < PAR; ++p) {
    const float4 x = sum[threadIdx.x + p * TPR];
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
  }
  store_row<D>(a, out, c, m, l, acc);
}

// Joins the rows and, with mass, adds the weights up: blockIdx.y is a set of `per` rows of
// the segment blockIdx.x, a (b, h, row segment), or, from `row_sets` on, a chunk of
// tokens of the key head (taken by its first row segment).  Nothing is read before the
// wait for the main kernel, not even what a kernel before that one wrote (lengths, K, W,
// queries): it is the wait that makes earlier writes visible here.
// RP >= 0: the weights are recomputed from K and W, else they come from the scores.
template <int D, int RP>
__global__ void __launch_bounds__(128) cache_attn_combine_kernel(const CacheAttnArgs a,
                                                                 unsigned ctas, int per,
                                                                 int row_sets) {
  const int set = blockIdx.y, mult = a.Hk * a.row_segs;
  const int b = blockIdx.x / mult, seg = blockIdx.x - b * mult;
  const int h = seg / a.row_segs, rs = seg - h * a.row_segs, bh = b * a.Hk + h;
  grid_dep_wait();
  if (set < row_sets) {
    const Parts parts = parts_of(a, b, seg, ctas);
    if (parts.n == 1) return;  // one CTA had it whole
    if (RP < 0 && per == 1)
      join_one<D>(a, parts, bh, rs, set);
    else
      join_many<D>(a, parts, bh, rs, set * per);
    return;
  }
  if (rs != 0) return;
  if constexpr (RP >= 0)
    recompute_mass<D, RP, true>(a, ctas, bh, set - row_sets);
  else
    add_mass(a, ctas, bh, set - row_sets);
}

}  // namespace rfb
