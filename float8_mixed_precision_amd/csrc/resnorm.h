// Residual norm on gfx950: the norm behind a block, its gate, the residual, and
// the norm in front of the next block, forward and backward in one pass each.
//
//   t  = N(b; post)  (or b),   s = alpha x + gate t,   y = N(s; pre)
//   N(v; w, c) = (v - mean) rstd w + c                 (norm.h)
//   backward, with xh the normalized values:
//   dT = ds + rstd_pre (g - mean(g) - xh mean(g xh)),  g = dy w_pre
//   dx = alpha dT
//   db = rstd_post (h - mean(h) - xh mean(h xh)),      h = dT gate w_post
//   (without a post norm db = dT gate; RMS form: no mean(g), mean(h))
//
// s is rounded to the stream's type, and y and the backward pass are those of
// the rounded s.  Everything between is fp32.
//
// The columns' gradients come from four sums over rows, A = sum dT xh_post (sum
// dT b without a post norm), B = sum dT, C = sum dy xh_pre, D = sum dy:
//   dpost_w = gate A, dpost_b = gate B, dgate = w_post A + b_post B (A without a
//   post norm), dpre_w = C, dpre_b = D.
//
// Rows sit in registers between their reductions and are read once, as in
// norm.h, whose layouts, loads and sums these kernels use.
//
// Bound: HBM, few rows: latency.  8192 x 4096, bf16 stream, RMS, both norms and a gate:
// forward with maxima 35.3 us (201 MB, 5.7 TB/s) and its cast 23.2 (134 MB, 5.8),
// backward 79 us (420 MB with the partial sums, 5.3 TB/s) and its cast, which finishes
// them, 27.5 (a kernel of their own 6.3 beside a cast of 23.5); a large copy runs at 5.4 TB/s.
// An fp32 stream: forward 76.8 us with y (403 MB, 5.2 TB/s), backward 113.8 (604 MB, 5.3).
// Above 8192 columns a thread has 16 of them in 128 registers, and the kernels spill: 27 to
// 85 registers forward, 173 to 233 backward (four sums a column).  2048 x 16384, bf16 / fp32
// stream: forward 87 / 137 us (3.1 / 2.9 TB/s), with maxima 80 / 149, backward 385 / 464
// (1.0 / 1.3 TB/s), bound by that scratch memory; 2048 x 8192 26.5 / 35.0 and 38.4 / 63.6.
//
// Part of quantize.hip (included at its end).
#pragma once

#include "norm.h"

namespace fp8l {
namespace {

struct ResArgs {
  const void *b, *x;           // block output (bf16), stream
  const void *post_w, *post_b, *pre_w, *pre_b, *gate;   // NULL: 1 (biases: 0)
  int wf32;                    // type of the parameters
  int rms, post, pre;
  float alpha, eps;
  int64_t rows;
  int cols;
  void *s;
  uint16_t *y;                 // may be NULL
  float *mean_post, *rstd_post, *mean_pre, *rstd_pre;   // each may be NULL
  uint8_t *q;                  // NORM_ROWS
  float *scale, *amax;
  uint32_t *part;              // NORM_TW
  uint16_t *rowpart, *colpart; // NORM_RW: [rows], [gridDim.x][cols]
};

// Mean and 1 / sqrt(variance + eps) of a row held as f(k, j).
template <int LAY, int TPR, int CH, class F>
__device__ __forceinline__ void row_stats(F f, int rms, float eps, int t, int cols, float inv_n,
                                          float (*red)[16], int &slot, float &mean, float &rstd) {
  mean = 0.f;
  if (!rms) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
      s += chunk_sum<LAY, TPR>(k, t, cols, [&](int j) { return f(k, j); });
    mean = quotient(row_sum<TPR>(s, red, slot), (float)cols, inv_n);
  }
  float s2 = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k)
    s2 += chunk_sum<LAY, TPR>(k, t, cols, [&](int j) {
      const float d = f(k, j) - mean;
      return d * d;
    });
  rstd = inverse_root(row_sum<TPR>(s2, red, slot) * inv_n + eps);
}

// Eight fp32 values to a chunk of the stream (and the values as they are stored
// there).
template <int LAY, int TPR>
__device__ __forceinline__ void store_stream(float *row, float (&f)[8], bool ok, int k, int t,
                                             int cols) {
  if (ok) store_chunk<LAY, TPR>(row, f, k, t, cols);
}
template <int LAY, int TPR>
__device__ __forceinline__ void store_stream(uint16_t *row, float (&f)[8], bool ok, int k, int t,
                                             int cols) {
  uint32_t d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    d[j] = bf16x2_bits(f[2 * j], f[2 * j + 1]);
    f[2 * j] = __uint_as_float(d[j] << 16);
    f[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
  }
  if (ok) store_chunk<LAY, TPR>(row, d, k, t, cols);
}

// The maximum of a workgroup's u16 pairs, to part[blockIdx.x].
template <int BLK>
__device__ __forceinline__ void store_block_max(uint32_t pairs, uint32_t *part) {
  __shared__ uint32_t tw[16];
  const uint32_t m = wave_umax(hmax16(pairs));
  if ((threadIdx.x & 63) == 0) tw[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t a = tw[0];
#pragma unroll
    for (int i = 1; i < BLK / 64; ++i) a = max(a, tw[i]);
    part[blockIdx.x] = a;
  }
}

// The column maxima of a workgroup's row groups, joined in LDS (integer maxima:
// any order gives the same result), to dst[cols].  lds: TPR 8 CH words, read or
// written by no one else meanwhile.
template <int LAY, int TPR, int CH, int BLK>
__device__ __forceinline__ void store_column_max(const uint32_t (&cm)[CH][4], uint32_t *lds, int t,
                                                 int cols, uint16_t *dst) {
  if constexpr (BLK > TPR) {
    constexpr int SPAN = TPR * 8 * CH;
    __syncthreads();
    for (int c = threadIdx.x; c < SPAN; c += BLK) lds[c] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = chunk_start<TPR>(k, t) + 2 * j;
        atomicMax(&lds[c], cm[k][j] & 0xFFFFu);
        atomicMax(&lds[c + 1], cm[k][j] >> 16);
      }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += BLK) dst[c] = (uint16_t)lds[c];
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k) store_chunk<LAY, TPR>(dst, cm[k], k, t, cols);
  }
}

// --------------------------------------------------------------- forward --

// Rows are dealt to the workgroups as in k_norm.  gate w_post and gate b_post are
// one product each per column and call, kept in registers with the other norm's
// parameters; b and x of the next round load while this one is computed.
template <class TS, int LAY, int TPR, int CH, int MODE>
__global__ __launch_bounds__((block_threads<TPR, MODE>())) void k_resnorm(ResArgs p) {
  constexpr int BLK = block_threads<TPR, MODE>();
  constexpr int G = BLK / TPR;
  static_assert(MODE == NORM_Y || LAY == LAY_ALIGNED, "codes come from rows of whole chunks");
  __shared__ float red[2][16];
  __shared__ uint32_t redu[16];
  const int t = threadIdx.x % TPR;
  const int g = threadIdx.x / TPR;
  const int cols = p.cols;
  const float inv_n = 1.0f / (float)cols;
  uint32_t tw_max = 0;
  uint32_t cm[CH][4] = {};

  Pack<uint16_t> bn[CH];
  Pack<TS> xn[CH];
  auto load_row = [&](int64_t r0) {
    const int64_t at = min(r0 + g, p.rows - 1) * cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      load_chunk<LAY, TPR>(bn[k], static_cast<const uint16_t *>(p.b) + at, k, t, cols);
      load_chunk<LAY, TPR>(xn[k], static_cast<const TS *>(p.x) + at, k, t, cols);
    }
  };
  const int64_t step = (int64_t)gridDim.x * G;
  const int64_t first = (int64_t)blockIdx.x * G;
  load_row(first);
  float gw[CH][8], gb[CH][8], w[CH][8], c[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    float gate[8];
    load_param<LAY, TPR>(gate, p.gate, p.wf32, 1.f, k, t, cols);
    load_param<LAY, TPR>(gw[k], p.post_w, p.wf32, 1.f, k, t, cols);
    load_param<LAY, TPR>(gb[k], p.post_b, p.wf32, 0.f, k, t, cols);
    load_param<LAY, TPR>(w[k], p.pre_w, p.wf32, 1.f, k, t, cols);
    load_param<LAY, TPR>(c[k], p.pre_b, p.wf32, 0.f, k, t, cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      gw[k][j] *= gate[j];
      gb[k][j] *= gate[j];
    }
  }
  int slot = 0;
  for (int64_t r0 = first; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + g;
    const bool ok = r < p.rows;
    Pack<uint16_t> b[CH];
    Pack<TS> x[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      b[k] = bn[k];
      x[k] = xn[k];
    }
    if (r0 + step < p.rows) load_row(r0 + step);
    float mean = 0.f, rstd = 1.f;
    if (p.post) {
      row_stats<LAY, TPR, CH>([&](int k, int j) { return b[k].get(j); }, p.rms, p.eps, t, cols,
                              inv_n, red, slot, mean, rstd);
      if (t == 0 && ok) {
        if (p.mean_post) p.mean_post[r] = mean;
        if (p.rstd_post) p.rstd_post[r] = rstd;
      }
    }
    float s[CH][8];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s[k][j] = __builtin_fmaf(p.alpha, x[k].get(j),
                                 norm_value(b[k].get(j), mean, rstd, gw[k][j], gb[k][j]));
      store_stream<LAY, TPR>(static_cast<TS *>(p.s) + r * cols, s[k], ok, k, t, cols);
    }
    if (!p.pre) continue;                         // uniform
    row_stats<LAY, TPR, CH>([&](int k, int j) { return s[k][j]; }, p.rms, p.eps, t, cols, inv_n,
                            red, slot, mean, rstd);
    if (t == 0 && ok) {
      if (p.mean_pre) p.mean_pre[r] = mean;
      if (p.rstd_pre) p.rstd_pre[r] = rstd;
    }
    uint32_t rm = 0;
    uint32_t yb[CH][4];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        yb[k][j] =
            bf16x2_bits(norm_value(s[k][2 * j], mean, rstd, w[k][2 * j], c[k][2 * j]),
                        norm_value(s[k][2 * j + 1], mean, rstd, w[k][2 * j + 1], c[k][2 * j + 1]));
      if (p.y && ok) store_chunk<LAY, TPR>(p.y + r * cols, yb[k], k, t, cols);
      if (MODE != NORM_Y) {
        const uint32_t keep = ok && chunk_start<TPR>(k, t) < cols ? 0x7FFF7FFFu : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t m = yb[k][j] & keep;
          rm = pk_max(rm, m);
          if (MODE == NORM_RW) cm[k][j] = pk_max(cm[k][j], m);
        }
      }
    }
    if (MODE == NORM_TW) tw_max = pk_max(tw_max, rm);
    if (MODE == NORM_RW || MODE == NORM_ROWS) {
      // (the next round's sums put a barrier between these reads of redu and the
      // next writes)
      const uint32_t am = row_umax<TPR>(hmax16(rm), redu);
      if (MODE == NORM_RW && t == 0 && ok) p.rowpart[r] = (uint16_t)am;
      if (MODE == NORM_ROWS) {
        const float a = bf16_to_f32(am);
        const float sc = scale_from_amax<0>(a);
        if (t == 0 && ok) {
          p.scale[r] = sc;
          if (p.amax) p.amax[r] = a;
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int col = chunk_start<TPR>(k, t);
          const uint32_t *d = yb[k];
          const uint32_t q0 =
              fp8x4<0>(bf16_to_f32(d[0] & 0xFFFFu) * sc, bf16_to_f32(d[0] >> 16) * sc,
                       bf16_to_f32(d[1] & 0xFFFFu) * sc, bf16_to_f32(d[1] >> 16) * sc);
          const uint32_t q1 =
              fp8x4<0>(bf16_to_f32(d[2] & 0xFFFFu) * sc, bf16_to_f32(d[2] >> 16) * sc,
                       bf16_to_f32(d[3] & 0xFFFFu) * sc, bf16_to_f32(d[3] >> 16) * sc);
          if (col < cols && ok)
            *reinterpret_cast<uint2 *>(p.q + r * cols + col) = make_uint2(q0, q1);
        }
      }
    }
  }
  if (MODE == NORM_TW) store_block_max<BLK>(tw_max, p.part);
  if (MODE == NORM_RW) {
    __shared__ uint32_t cred[G > 1 ? TPR * 8 * CH : 1];
    store_column_max<LAY, TPR, CH, BLK>(cm, cred, t, cols, p.colpart + (size_t)blockIdx.x * cols);
  }
}

// -------------------------------------------------------------- backward --

struct ResBwdArgs {
  const void *dy, *ds;         // of y (bf16), of s (the stream's type); ds may be NULL
  const void *b, *s;
  const void *post_w, *pre_w, *gate;
  int wf32;
  int rms, post, pre;
  float alpha;
  const float *mean_post, *rstd_post, *mean_pre, *rstd_pre;
  int64_t rows;
  int cols;
  void *dx;                    // may be NULL
  uint16_t *db;
  float *sums;                 // [gridDim.x][4][cols] (A, B, C, D above), or NULL
  uint32_t *part;              // NORM_TW
  uint16_t *rowpart, *colpart; // NORM_RW
};

// Sums of two values over a row's TPR threads, in each of them (row_sum's
// scheme).
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 (*red2)[16], int &slot) {
  a = wave_sum(a);
  b = wave_sum(b);
  if (TPR == 64) return make_float2(a, b);
  float2 *red = red2[slot];
  slot ^= 1;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[wave] = make_float2(a, b);
  __syncthreads();
  constexpr int W = TPR / 64;
  const int first = wave / W * W;
  float2 s = red[first];
#pragma unroll
  for (int i = 1; i < W; ++i) {
    s.x += red[first + i].x;
    s.y += red[first + i].y;
  }
  return s;
}

// A workgroup walks its rows with a fixed set of columns per thread: the four
// sums of a column stay in registers, every tensor is read once.  w_pre and gate
// w_post are kept in LDS as fp32 (chunk k of thread t at [k][half][t]).  At the
// end the row groups add up in LDS in group order, the workgroup writes one
// partial row per sum and k_resnorm_bwd_finish adds those in a fixed order.
// Nothing is atomic but integer maxima: results do not vary between runs.
template <class TS, int LAY, int TPR, int CH, int MODE, int BLK>
__global__ __launch_bounds__(BLK) void k_resnorm_bwd(ResBwdArgs p) {
  constexpr int G = BLK / TPR;
  constexpr int SPAN = TPR * 8 * CH;
  static_assert(MODE == NORM_Y || LAY == LAY_ALIGNED, "codes come from rows of whole chunks");
  __shared__ float2 red[2][16];
  __shared__ uint32_t redu[16];
  __shared__ float4 lds_w[2][CH * 2 * TPR];       // w_pre, gate w_post
  const int t = threadIdx.x % TPR;
  const int g = threadIdx.x / TPR;
  const int cols = p.cols;
  const float inv_n = 1.0f / (float)cols;
  float sum[4][CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0][k][j] = sum[1][k][j] = sum[2][k][j] = sum[3][k][j] = 0.f;
    if (g == 0) {
      float w[8], gate[8];
      load_param<LAY, TPR>(w, p.pre_w, p.wf32, 1.f, k, t, cols);
      lds_w[0][(2 * k) * TPR + t] = make_float4(w[0], w[1], w[2], w[3]);
      lds_w[0][(2 * k + 1) * TPR + t] = make_float4(w[4], w[5], w[6], w[7]);
      load_param<LAY, TPR>(w, p.post_w, p.wf32, 1.f, k, t, cols);
      load_param<LAY, TPR>(gate, p.gate, p.wf32, 1.f, k, t, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= gate[j];
      lds_w[1][(2 * k) * TPR + t] = make_float4(w[0], w[1], w[2], w[3]);
      lds_w[1][(2 * k + 1) * TPR + t] = make_float4(w[4], w[5], w[6], w[7]);
    }
  }
  __syncthreads();
  auto weights = [&](int which, int k, float (&w)[8]) {
    const float4 a = lds_w[which][(2 * k) * TPR + t], b = lds_w[which][(2 * k + 1) * TPR + t];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  };
  // a round's rows load a round ahead, where registers allow it
  constexpr bool AHEAD = CH == 1;
  Pack<uint16_t> dyn[CH], bn[CH];
  Pack<TS> sn[CH], dsn[CH];
  float m1n = 0.f, r1n = 1.f, m2n = 0.f, r2n = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {                  // what is absent counts as zero
    dyn[k] = {};
    sn[k] = {};
    dsn[k] = {};
  }
  auto load_row = [&](int64_t r0) {
    const int64_t r = min(r0 + g, p.rows - 1), at = r * cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      load_chunk<LAY, TPR>(bn[k], static_cast<const uint16_t *>(p.b) + at, k, t, cols);
      if (p.ds) load_chunk<LAY, TPR>(dsn[k], static_cast<const TS *>(p.ds) + at, k, t, cols);
      if (p.pre) {
        load_chunk<LAY, TPR>(dyn[k], static_cast<const uint16_t *>(p.dy) + at, k, t, cols);
        load_chunk<LAY, TPR>(sn[k], static_cast<const TS *>(p.s) + at, k, t, cols);
      }
    }
    if (p.post) {
      r1n = p.rstd_post[r];
      m1n = p.rms ? 0.f : p.mean_post[r];
    }
    if (p.pre) {
      r2n = p.rstd_pre[r];
      m2n = p.rms ? 0.f : p.mean_pre[r];
    }
  };
  uint32_t tw_max = 0;
  uint32_t cm[CH][4] = {};
  int slot = 0;
  const int64_t step = (int64_t)gridDim.x * G;
  if (AHEAD) load_row((int64_t)blockIdx.x * G);
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < p.rows; r0 += step) {
    const bool ok = r0 + g < p.rows;
    const int64_t r = ok ? r0 + g : p.rows - 1;
    if (!AHEAD) load_row(r0);
    Pack<uint16_t> dy[CH], b[CH];
    Pack<TS> s[CH];
    float dt[CH][8];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      dy[k] = dyn[k];
      b[k] = bn[k];
      s[k] = sn[k];
#pragma unroll
      for (int j = 0; j < 8; ++j) dt[k][j] = dsn[k].get(j);
    }
    const float m1 = m1n, r1 = r1n, m2 = m2n, r2 = r2n;
    if (AHEAD && r0 + step < p.rows) load_row(r0 + step);
    if (p.pre) {
      float s1 = 0.f, s2 = 0.f;                   // sums of g xh and of g
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float w[8];
        weights(0, k, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = ok && owned<LAY, TPR>(k, j, t, cols);
          const float d = in ? dy[k].get(j) : 0.f;
          const float xh = (s[k].get(j) - m2) * r2;
          const float e = in ? d * xh : 0.f;
          s1 += e * w[j];
          s2 += d * w[j];
          sum[2][k][j] += e;
          sum[3][k][j] += d;
        }
      }
      const float2 a = row_sum2<TPR>(s1, s2, red, slot);
      const float c1 = a.x * inv_n, c2 = p.rms ? 0.f : a.y * inv_n;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float w[8];
        weights(0, k, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (s[k].get(j) - m2) * r2;
          dt[k][j] += (dy[k].get(j) * w[j] - c2 - xh * c1) * r2;
        }
      }
    }
    if (p.dx) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = p.alpha * dt[k][j];
        store_stream<LAY, TPR>(static_cast<TS *>(p.dx) + r * cols, f, ok, k, t, cols);
      }
    }
    float c1 = 0.f, c2 = 0.f;
    {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float w[8];
        weights(1, k, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = ok && owned<LAY, TPR>(k, j, t, cols);
          const float d = in ? dt[k][j] : 0.f;
          const float e = in ? d * ((b[k].get(j) - m1) * r1) : 0.f;
          s1 += e * w[j];
          s2 += d * w[j];
          sum[0][k][j] += e;
          sum[1][k][j] += d;
        }
      }
      if (p.post) {
        const float2 a = row_sum2<TPR>(s1, s2, red, slot);
        c1 = a.x * inv_n;
        c2 = p.rms ? 0.f : a.y * inv_n;
      }
    }
    uint32_t rm = 0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float w[8];
      weights(1, k, w);
      uint32_t d[4];
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = (dt[k][j] * w[j] - c2 - ((b[k].get(j) - m1) * r1) * c1) * r1;
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = bf16x2_bits(f[2 * j], f[2 * j + 1]);
      if (ok) store_chunk<LAY, TPR>(p.db + r * cols, d, k, t, cols);
      if (MODE != NORM_Y) {
        const uint32_t keep = ok && chunk_start<TPR>(k, t) < cols ? 0x7FFF7FFFu : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rm = pk_max(rm, d[j] & keep);
          if (MODE == NORM_RW) cm[k][j] = pk_max(cm[k][j], d[j] & keep);
        }
      }
    }
    if (MODE == NORM_TW) tw_max = pk_max(tw_max, rm);
    if (MODE == NORM_RW) {
      // (as in the forward pass: the next round's sums lie between)
      const uint32_t am = row_umax<TPR>(hmax16(rm), redu);
      if (t == 0 && ok) p.rowpart[r] = (uint16_t)am;
    }
  }
  if (MODE == NORM_TW) store_block_max<BLK>(tw_max, p.part);
  if (MODE == NORM_RW)
    store_column_max<LAY, TPR, CH, BLK>(cm, reinterpret_cast<uint32_t *>(lds_w[1]), t, cols,
                                        p.colpart + (size_t)blockIdx.x * cols);
  if (!p.sums) return;
  float *dst = p.sums + (size_t)blockIdx.x * 4 * cols;
  float *acc = reinterpret_cast<float *>(lds_w[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q < 2 ? !(p.post || p.gate) : !p.pre) continue;   // uniform: not asked for
    if (G > 1) {
      for (int i = 0; i < G; ++i) {
        __syncthreads();
        if (g == i) {
#pragma unroll
          for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float &a = acc[(k * 8 + j) * TPR + t];
              a = i == 0 ? sum[q][k][j] : a + sum[q][k][j];
            }
        }
      }
      __syncthreads();
    }
    if (g == 0) {
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (owned<LAY, TPR>(k, j, t, cols))
            dst[q * cols + column<LAY, TPR>(k, j, t, cols)] =
                G > 1 ? acc[(k * 8 + j) * TPR + t] : sum[q][k][j];
    }
  }
  static_assert(SPAN * sizeof(float) == sizeof(lds_w[0]), "one float per column");
}

// The parameters' gradients where no cast follows (res_finish, else beside the cast).
__global__ __launch_bounds__(64 * FIN_SLICES) void k_resnorm_bwd_finish(ResFinish p) {
  res_finish<FIN_SLICES>(p, (int)blockIdx.x);
}

// ---------------------------------------------------------------- launch --

template <class TS, int LAY, int MODE>
hipError_t launch_res(const ResArgs &a, int64_t max_blocks, int *blocks, hipStream_t stream) {
  auto launch = [&](auto tpr, auto ch) {
    constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
    constexpr int BLK = block_threads<TPR, MODE>();
    if (max_blocks > kComputeUnits * (2048 / BLK)) max_blocks = kComputeUnits * (2048 / BLK);
    int64_t nb = cdiv(a.rows, BLK / TPR);
    if (nb > max_blocks) nb = max_blocks;
    *blocks = (int)nb;
    hipLaunchKernelGGL((k_resnorm<TS, LAY, TPR, CH, MODE>), dim3((unsigned)nb), dim3(BLK), 0,
                       stream, a);
    return hipGetLastError();
  };
  if constexpr (LAY == LAY_SCALAR)
    return launch(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  else
    return with_shape<false>(a.cols, false, launch);
}

template <class TS, int LAY, int MODE>
hipError_t launch_res_bwd(const ResBwdArgs &a, int *blocks, hipStream_t stream) {
  auto launch = [&](auto tpr, auto ch) {
    constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
    constexpr int BLK = TPR > 512 ? TPR : 512 / TPR * TPR < 512 ? 2 * TPR : 512;
    int64_t nb = cdiv(a.rows, BLK / TPR);
    if (nb > kComputeUnits) nb = kComputeUnits;
    *blocks = (int)nb;
    hipLaunchKernelGGL((k_resnorm_bwd<TS, LAY, TPR, CH, MODE, BLK>), dim3((unsigned)nb), dim3(BLK),
                       0, stream, a);
    return hipGetLastError();
  };
  if constexpr (LAY == LAY_SCALAR)
    return launch(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  // (widths a little above a power of two, where twice the threads would be idle by
  // nearly half.  These / 512 and 1024 threads a row, us, bf16 stream: 1539 x 2050 19.5 /
  // 22.0, 2048 x 2560 19.0 / 21.7, 8192 x 2560 45.8 / 59.7, 512 x 5120 16.6 / 17.2, 2048 x
  // 4112 26.3 / 29.1, 8192 x 5120 99 / 103; fp32: 1539 x 2050 20.4 / 22.7, 2048 x 2560 21.2 /
  // 22.4, 8192 x 2560 75.0 / 70.9, 2048 x 5120 34.9 / 36.5, 8192 x 5120 146 / 143; with codes
  // these are ahead at each of them, by 0 to 23%.  Further widths have no shape of their own.)
  else if (a.cols > 256 * 8 && a.cols <= 320 * 8)
    return launch(std::integral_constant<int, 320>(), std::integral_constant<int, 1>());
  else if (a.cols > 512 * 8 && a.cols <= 640 * 8)
    return launch(std::integral_constant<int, 640>(), std::integral_constant<int, 1>());
  else
    return with_shape<false>(a.cols, false, launch);
}

ResArgs make_args(const ResIn &in) {
  ResArgs a = {};
  a.b = in.b;
  a.x = in.x;
  a.post_w = in.post_w;
  a.post_b = in.post_b;
  a.pre_w = in.pre_w;
  a.pre_b = in.pre_b;
  a.gate = in.gate;
  a.wf32 = in.wf32;
  a.rms = in.rms;
  a.post = in.post;
  a.pre = in.pre;
  a.alpha = in.alpha;
  a.eps = in.eps;
  a.rows = in.rows;
  a.cols = (int)in.cols;
  a.s = in.s;
  a.y = static_cast<uint16_t *>(in.y);
  a.mean_post = in.mean_post;
  a.rstd_post = in.rstd_post;
  a.mean_pre = in.mean_pre;
  a.rstd_pre = in.rstd_pre;
  return a;
}

// bytes of the backward's partial sums in front of the maxima
size_t res_sums_bytes(int64_t cols) {
  return (size_t)kComputeUnits * 4 * (size_t)cols * sizeof(float);   // a multiple of 256
}

// The maxima of a quantize in `ws`: where the kernel writes them and where the
// cast reads them.
template <class A>
void res_partials(A &a, CastSource &src, void *ws, bool rw) {
  if (rw) {
    a.rowpart = static_cast<uint16_t *>(ws);
    a.colpart = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + colpart_offset(a.rows));
    src.rowpart = a.rowpart;
    src.colpart = a.colpart;
    src.row_slices = 1;
  } else {
    a.part = static_cast<uint32_t *>(ws);
    src.part = a.part;
  }
}

}  // namespace

size_t resnorm_workspace_bytes(int64_t rows, int64_t cols, int scaling) {
  const size_t maxima = (scaling & FP8L_ROWWISE)
                            ? colpart_offset(rows) + (size_t)kMaxSlices * cols * sizeof(uint16_t)
                            : (size_t)TW_MAX_BLOCKS * sizeof(uint32_t);
  return (res_sums_bytes(cols) + maxima + 255) & ~(size_t)255;
}

hipError_t resnorm_fwd_launch(const ResIn &in, hipStream_t stream) {
  if (in.rows == 0) return hipSuccess;
  const ResArgs a = make_args(in);
  int nb;
  return with_layout(in.cols, [&](auto lay) {
    constexpr int LAY = decltype(lay)::value;
    return in.f32 ? launch_res<float, LAY, NORM_Y>(a, kMaxBlocks, &nb, stream)
                  : launch_res<uint16_t, LAY, NORM_Y>(a, kMaxBlocks, &nb, stream);
  });
}

hipError_t resnorm_rows_launch(const ResIn &in, void *q, float *scale, float *amax_out,
                               hipStream_t stream) {
  if (in.rows == 0) return hipSuccess;
  ResArgs a = make_args(in);
  a.q = static_cast<uint8_t *>(q);
  a.scale = scale;
  a.amax = amax_out;
  int nb;
  return in.f32 ? launch_res<float, LAY_ALIGNED, NORM_ROWS>(a, kMaxBlocks, &nb, stream)
                : launch_res<uint16_t, LAY_ALIGNED, NORM_ROWS>(a, kMaxBlocks, &nb, stream);
}

hipError_t resnorm_quantize_launch(const ResIn &in, int scaling, const Fp8Out &o, void *workspace,
                                   hipStream_t stream) {
  ResArgs a = make_args(in);
  CastSource src = {};
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  int nb = 0;
  res_partials(a, src, workspace, rw);
  if (in.rows > 0) {
    const hipError_t e =
        in.f32 ? (rw ? launch_res<float, LAY_ALIGNED, NORM_RW>(a, kMaxSlices, &nb, stream)
                     : launch_res<float, LAY_ALIGNED, NORM_TW>(a, TW_MAX_BLOCKS, &nb, stream))
               : (rw ? launch_res<uint16_t, LAY_ALIGNED, NORM_RW>(a, kMaxSlices, &nb, stream)
                     : launch_res<uint16_t, LAY_ALIGNED, NORM_TW>(a, TW_MAX_BLOCKS, &nb, stream));
    if (e != hipSuccess) return e;
  }
  if (rw) src.col_slices = nb;
  else src.nparts = nb;
  src.x = in.y;
  if (!in.y) {                                    // a bf16 stream: the cast normalizes s again
    src.x = in.s;
    src.w = in.pre_w;
    src.b = in.pre_b;
    src.wf32 = in.wf32;
    src.mean = in.rms ? nullptr : in.mean_pre;
    src.rstd = in.rstd_pre;
  }
  return quantize_cast_launch(&src, 1, in.rows, in.cols, scaling, &o, stream);
}

hipError_t resnorm_bwd_launch(const ResIn &in, const void *dy, const void *ds, const ResGrads &gr,
                              int scaling, const Fp8Out *o, void *workspace, hipStream_t stream) {
  ResBwdArgs a = {};
  a.dy = dy;
  a.ds = ds;
  a.b = in.b;
  a.s = in.s;
  a.post_w = in.post_w;
  a.pre_w = in.pre_w;
  a.gate = in.gate;
  a.wf32 = in.wf32;
  a.rms = in.rms;
  a.post = in.post;
  a.pre = in.pre;
  a.alpha = in.alpha;
  a.mean_post = in.mean_post;
  a.rstd_post = in.rstd_post;
  a.mean_pre = in.mean_pre;
  a.rstd_pre = in.rstd_pre;
  a.rows = in.rows;
  a.cols = (int)in.cols;
  a.dx = gr.dx;
  a.db = static_cast<uint16_t *>(gr.db);
  const bool wants = gr.dgate || gr.dpost_w || gr.dpost_b || gr.dpre_w || gr.dpre_b;
  a.sums = wants ? static_cast<float *>(workspace) : nullptr;
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  CastSource src = {};
  src.x = gr.db;
  if (o) res_partials(a, src, static_cast<uint8_t *>(workspace) + res_sums_bytes(in.cols), rw);
  int nb = 0;
  if (in.rows > 0) {
    hipError_t e;
    if (!o)
      e = with_layout(in.cols, [&](auto lay) {
        constexpr int LAY = decltype(lay)::value;
        return in.f32 ? launch_res_bwd<float, LAY, NORM_Y>(a, &nb, stream)
                      : launch_res_bwd<uint16_t, LAY, NORM_Y>(a, &nb, stream);
      });
    else if (in.f32)
      e = rw ? launch_res_bwd<float, LAY_ALIGNED, NORM_RW>(a, &nb, stream)
             : launch_res_bwd<float, LAY_ALIGNED, NORM_TW>(a, &nb, stream);
    else
      e = rw ? launch_res_bwd<uint16_t, LAY_ALIGNED, NORM_RW>(a, &nb, stream)
             : launch_res_bwd<uint16_t, LAY_ALIGNED, NORM_TW>(a, &nb, stream);
    if (e != hipSuccess) return e;
  }
  const ResFinish f = {a.sums, nb, a.cols, in.wf32, in.post, 0, in.post_w, in.post_b, in.gate,
                       gr.dgate, gr.dpost_w, gr.dpost_b, gr.dpre_w, gr.dpre_b};
  const bool beside = o && in.rows > 0;           // the cast's last workgroups finish them
  if (wants && beside) src.res = &f;
  if (wants && !beside) {
    hipLaunchKernelGGL(k_resnorm_bwd_finish, dim3((unsigned)(2 * cdiv(in.cols, 64))),
                       dim3(64 * FIN_SLICES), 0, stream, f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!o) return hipSuccess;
  if (rw) src.col_slices = nb;
  else src.nparts = nb;
  return quantize_cast_launch(&src, 1, in.rows, in.cols, scaling, o, stream);
}

}  // namespace fp8l
