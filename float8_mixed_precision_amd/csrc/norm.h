// Layer norm (and its RMS form) on gfx950, forward and backward: the producer
// of the feed-forward's fp8 input and the first step of its residual branch.
//
//   mean = sum_c x / C          (RMS form: mean = 0)
//   rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps)
//   xh   = (x - mean) rstd,   y = xh w + b
//   backward, g = dy w:
//   dx = rstd (g - mean_c(g) - xh mean_c(g xh))     (RMS form: no mean_c(g))
//   dw = sum_r dy xh,   db = sum_r dy
//
// All statistics and sums are fp32; the variance is taken about the mean
// from the values held in registers, so a large common offset costs no
// digits.  x is read once per pass.
//
// Bound: HBM where y or dx is written; the statistics pass of the quantize, which
// only reads, by vector instructions (k_norm).  A row (or the share of one) sits
// in registers between the reductions; TPR threads work on a row: one wave for up to 512 columns (no
// barrier, reductions by DPP), 128 to 1024 threads for more (with_shape).
//
// The quantize forms need y only as fp8 codes.  Per-token codes (no
// transposed copy) come out of the same pass, since a row's amax is known
// where the row is.  The training form takes one read pass here for the
// statistics and the amax partial maxima of y, and the cast pass
// (quantize.hip) reads x again, mostly from the Infinity Cache, and
// normalizes it once more: y itself is neither written nor read unless the
// caller asks for it.
//
// Part of quantize.hip (included at its end): the norm is the first half of
// a quantize.
#pragma once

#include "fp8l_internal.h"

#include <type_traits>

namespace fp8l {
namespace {

constexpr int NORM_Y = 0;      // y
constexpr int NORM_ROWS = 1;   // y (optional), codes and scale of each row
constexpr int NORM_TW = 2;     // y (optional), one |y| maximum per workgroup
constexpr int NORM_RW = 3;     // y (optional), row maxima, column maxima per workgroup

struct NormArgs {
  const void *x;
  const void *w, *b;           // NULL: 1 and 0
  int wf32;                    // w and b are fp32 (else bf16)
  int rms;
  float eps;
  int64_t rows;
  int cols;
  void *y;
  float *mean, *rstd;
  uint8_t *q;                  // NORM_ROWS
  float *scale, *amax;
  uint32_t *part;              // NORM_TW
  uint16_t *rowpart, *colpart; // NORM_RW: [rows], [gridDim.x][cols]
};

// Eight values of a row held by a thread, as loaded.
template <class T>
struct Pack;
template <>
struct Pack<uint16_t> {        // bf16
  uint32_t d[4];
  __device__ float get(int j) const {
    return (j & 1) ? __uint_as_float(d[j >> 1] & 0xFFFF0000u) : __uint_as_float(d[j >> 1] << 16);
  }
};
template <>
struct Pack<float> {
  float d[8];
  __device__ float get(int j) const { return d[j]; }
};

// How the columns of a row are dealt to its TPR threads, in CH chunks of 8:
//   LAY_ALIGNED  cols a multiple of 8: chunk k of thread t is the 8 columns
//                from (k TPR + t) 8, moved in 16-byte accesses
//   LAY_CHUNKS   any cols >= 8: the same, except that the chunk that would
//                pass the row's end is moved back to the row's last 8
//                columns; its columns that belong to the chunk before it are
//                left out of the sums, and stored twice with the same value.
//                Rows then start at any element: the accesses are unaligned
//   LAY_SCALAR   cols < 8: one column per thread and element
// Chunks wholly past the row read columns inside it and are left out.
constexpr int LAY_SCALAR = 0, LAY_CHUNKS = 1, LAY_ALIGNED = 2;

// first column of chunk k before it is moved back
template <int TPR>
__device__ __forceinline__ int chunk_start(int k, int t) {
  return (k * TPR + t) * 8;
}

// column of element j of chunk k as loaded and stored
template <int LAY, int TPR>
__device__ __forceinline__ int column(int k, int j, int t, int cols) {
  if (LAY == LAY_SCALAR) return min((k * 8 + j) * TPR + t, cols - 1);
  return min(chunk_start<TPR>(k, t), cols - 8) + j;
}

// whether element j of chunk k is this thread's to count
template <int LAY, int TPR>
__device__ __forceinline__ bool owned(int k, int j, int t, int cols) {
  if (LAY == LAY_SCALAR) return (k * 8 + j) * TPR + t < cols;
  const int c = chunk_start<TPR>(k, t);
  if (LAY == LAY_ALIGNED) return c < cols;
  return c < cols && min(c, cols - 8) + j >= c;
}

// Sum of f(j) over the elements of chunk k that are this thread's to count.
template <int LAY, int TPR, class F>
__device__ __forceinline__ float chunk_sum(int k, int t, int cols, F f) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (LAY == LAY_ALIGNED) s += f(j);            // all eight or none
    else s += owned<LAY, TPR>(k, j, t, cols) ? f(j) : 0.f;
  }
  return LAY != LAY_ALIGNED || chunk_start<TPR>(k, t) < cols ? s : 0.f;
}

// 16 bytes at any element's address
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Any16 {
  uint32_t d[4];
};

template <int LAY, class T>
__device__ __forceinline__ U4 load16_at(const T *p) {
  if (LAY == LAY_ALIGNED) return load16(p);
  const Any16<T> v = *reinterpret_cast<const Any16<T> *>(p);
  return {v.d[0], v.d[1], v.d[2], v.d[3]};
}

template <int LAY, class T>
__device__ __forceinline__ void store16_at(T *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  if (LAY == LAY_ALIGNED)
    *reinterpret_cast<uint4 *>(p) = make_uint4(a, b, c, d);
  else
    *reinterpret_cast<Any16<T> *>(p) = {{a, b, c, d}};
}

template <int LAY, int TPR>
__device__ __forceinline__ void load_chunk(Pack<uint16_t> &v, const uint16_t *row, int k, int t,
                                           int cols) {
  if (LAY == LAY_SCALAR) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = row[column<LAY, TPR>(k, 2 * j, t, cols)];
      const uint32_t hi = row[column<LAY, TPR>(k, 2 * j + 1, t, cols)];
      v.d[j] = lo | hi << 16;
    }
  } else {
    const U4 u = load16_at<LAY>(row + column<LAY, TPR>(k, 0, t, cols));
    v.d[0] = u.x; v.d[1] = u.y; v.d[2] = u.z; v.d[3] = u.w;
  }
}

template <int LAY, int TPR>
__device__ __forceinline__ void load_chunk(Pack<float> &v, const float *row, int k, int t,
                                           int cols) {
  if (LAY == LAY_SCALAR) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.d[j] = row[column<LAY, TPR>(k, j, t, cols)];
  } else {
    const float *p = row + column<LAY, TPR>(k, 0, t, cols);
    const U4 a = load16_at<LAY>(p), b = load16_at<LAY>(p + 4);
    v.d[0] = __uint_as_float(a.x); v.d[1] = __uint_as_float(a.y);
    v.d[2] = __uint_as_float(a.z); v.d[3] = __uint_as_float(a.w);
    v.d[4] = __uint_as_float(b.x); v.d[5] = __uint_as_float(b.y);
    v.d[6] = __uint_as_float(b.z); v.d[7] = __uint_as_float(b.w);
  }
}

// a chunk of w or b (either type; `none` where the pointer is NULL)
template <int LAY, int TPR>
__device__ __forceinline__ void load_param(float (&f)[8], const void *p, int wf32, float none,
                                           int k, int t, int cols) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = none;
  } else if (wf32) {
    Pack<float> v;
    load_chunk<LAY, TPR>(v, static_cast<const float *>(p), k, t, cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v.get(j);
  } else {
    Pack<uint16_t> v;
    load_chunk<LAY, TPR>(v, static_cast<const uint16_t *>(p), k, t, cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v.get(j);
  }
}

template <int LAY, int TPR>
__device__ __forceinline__ void store_chunk(float *row, const float (&f)[8], int k, int t,
                                            int cols) {
  if (LAY == LAY_SCALAR) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (owned<LAY, TPR>(k, j, t, cols)) row[column<LAY, TPR>(k, j, t, cols)] = f[j];
  } else if (chunk_start<TPR>(k, t) < cols) {
    float *p = row + column<LAY, TPR>(k, 0, t, cols);
    store16_at<LAY>(p, __float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
    store16_at<LAY>(p + 4, __float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                    __float_as_uint(f[7]));
  }
}

// d: the eight values as bf16 pairs
template <int LAY, int TPR>
__device__ __forceinline__ void store_chunk(uint16_t *row, const uint32_t (&d)[4], int k, int t,
                                            int cols) {
  if (LAY == LAY_SCALAR) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (owned<LAY, TPR>(k, j, t, cols))
        row[column<LAY, TPR>(k, j, t, cols)] =
            (uint16_t)((j & 1) ? d[j >> 1] >> 16 : d[j >> 1]);
  } else if (chunk_start<TPR>(k, t) < cols) {
    store16_at<LAY>(row + column<LAY, TPR>(k, 0, t, cols), d[0], d[1], d[2], d[3]);
  }
}

// ------------------------------------------------------------ reductions --

// Value of the lane that DPP control CTRL names: quad_perm [1,0,3,2] 0xB1,
// quad_perm [2,3,0,1] 0x4E, row_half_mirror 0x141, row_mirror 0x140.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}

// Sum over the 64 lanes, in every lane: within 16 lanes by DPP, then the
// four rows' sums through scalar registers.
__device__ __forceinline__ float wave_sum(float v) {
  v += dppf<0xB1>(v);
  v += dppf<0x4E>(v);
  v += dppf<0x141>(v);
  v += dppf<0x140>(v);
  const int i = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(i, 0)) +
          __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(i, 32)) +
          __int_as_float(__builtin_amdgcn_readlane(i, 48)));
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max(v, (uint32_t)dpp<0xB1>((int)v));
  v = max(v, (uint32_t)dpp<0x4E>((int)v));
  v = max(v, (uint32_t)dpp<0x141>((int)v));
  v = max(v, (uint32_t)dpp<0x140>((int)v));
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0),
                 (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32),
                 (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// Sum over a row's TPR threads, in each of them.  red2: one float per wave of
// the workgroup, in two copies that successive calls take in turn (slot):
// the barrier of the call between orders a write behind the reads of the
// call before that, so one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red2)[16], int &slot) {
  v = wave_sum(v);
  if (TPR == 64) return v;
  float *red = red2[slot];
  slot ^= 1;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  constexpr int W = TPR / 64;
  const int first = wave / W * W;
  float s = red[first];
#pragma unroll
  for (int i = 1; i < W; ++i) s += red[first + i];
  return s;
}

template <int TPR>
__device__ __forceinline__ uint32_t row_umax(uint32_t v, uint32_t *red) {
  v = wave_umax(v);
  if (TPR == 64) return v;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  constexpr int W = TPR / 64;
  const int first = wave / W * W;
  uint32_t s = red[first];
#pragma unroll
  for (int i = 1; i < W; ++i) s = max(s, red[first + i]);
  return s;
}

// s / n from inv = fl(1 / n): the residual of the first quotient corrects it,
// so that a row of equal values has that value as its mean (8192 x 4096: the
// division and the square root below took 3 of 16 vector instructions per
// element).
__device__ __forceinline__ float quotient(float s, float n, float inv) {
  const float q = s * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, n, s), inv, q);
}

// 1 / sqrt(v): the hardware estimate (1 ulp; it takes v below the normal range
// as 0, so such v are scaled first) and a Newton step with the residual 1 - v r^2
// in two terms, which leaves the rounding of the result alone.  v = 0 gives
// infinity, an infinite v 0, and NaN NaN: there the estimate stays.  (The step
// costs 8192 x 4096 with its quantize 38.50 -> 38.55 us, 8192 x 8192 rowwise 79.95 ->
// 80.25, y alone of 4096 x 4096 13.66 -> 13.86, of 65536 x 256 16.9 -> 17.3.)
__device__ __forceinline__ float inverse_root(float v) {
  const bool tiny = v < 0x1p-100f;
  const float u = tiny ? v * 0x1p64f : v;
  const float r = __builtin_amdgcn_rsqf(u);
  const float p = u * r;
  const float e = __builtin_fmaf(-__builtin_fmaf(u, r, -p), r, __builtin_fmaf(-p, r, 1.0f));
  return (__builtin_fabsf(e) < 1.0f ? __builtin_fmaf(0.5f * e, r, r) : r) * (tiny ? 0x1p32f : 1.0f);
}

// --------------------------------------------------------------- forward --

// Threads of a workgroup: NORM_RW leaves one partial row per workgroup, so it
// takes the largest; the others 256 where that holds a row.
template <int TPR, int MODE>
constexpr int block_threads() {
  return MODE == NORM_RW ? 1024 : TPR > 256 ? TPR : 256;
}

// Workgroup b takes rows b G + g, G row groups g of TPR threads each, then
// those gridDim.x G further on, and so on; every thread of a workgroup makes
// the same number of rounds (a row past the end is computed on row rows - 1
// and not stored).
//
// Measured, statistics and maxima of 8192 x 4096 bf16 (tensorwise): 17.1 us,
// 3.9 TB/s, with 256 threads a row and 2048 workgroups.  A plain read of the same
// 64 MiB takes 12.5 us from memory and 10.7 from the Infinity Cache; here a vector
// instruction issues in 0.89 of the cycles (7.8M of them, 15 an element and lane).
// With 512 threads 19.3 us; earlier forms of this kernel with a
// wave a row 30 us (its w and b take 128 registers, or twice the traffic of x
// when read per row: 29 us), two rows a round 17-21 against 16.6 side by side.
template <class T, int LAY, int TPR, int CH, int MODE>
__global__ __launch_bounds__((block_threads<TPR, MODE>())) void k_norm(NormArgs p) {
  constexpr int G = block_threads<TPR, MODE>() / TPR;
  constexpr bool BF = sizeof(T) == 2;
  static_assert(MODE == NORM_Y || (BF && LAY == LAY_ALIGNED),
                "codes come from bf16 rows of whole chunks");
  __shared__ float red[2][16];
  __shared__ uint32_t redu[16];
  const int t = threadIdx.x % TPR;
  const int g = threadIdx.x / TPR;
  const int cols = p.cols;
  const float inv_n = 1.0f / (float)cols;
  uint32_t tw_max = 0;
  uint32_t cm[CH][4];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[k][j] = 0;

  // a round's row is loaded a round ahead of its use
  Pack<T> vn[CH];
  auto load_row = [&](int64_t r0) {
    const T *xr = static_cast<const T *>(p.x) + min(r0 + g, p.rows - 1) * cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) load_chunk<LAY, TPR>(vn[k], xr, k, t, cols);
  };
  const int64_t step = (int64_t)gridDim.x * G;
  const int64_t first = (int64_t)blockIdx.x * G;
  load_row(first);
  // the columns of a thread are the same in every round: w and b stay in its
  // registers
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    load_param<LAY, TPR>(w[k], p.w, p.wf32, 1.f, k, t, cols);
    load_param<LAY, TPR>(b[k], p.b, p.wf32, 0.f, k, t, cols);
  }
  int slot = 0;
  for (int64_t r0 = first; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + g;
    const bool ok = r < p.rows;
    Pack<T> v[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = vn[k];
    if (r0 + step < p.rows) load_row(r0 + step);
    float mean = 0.f;
    if (!p.rms) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k)
        s += chunk_sum<LAY, TPR>(k, t, cols, [&](int j) { return v[k].get(j); });
      mean = quotient(row_sum<TPR>(s, red, slot), (float)cols, inv_n);
    }
    float s2 = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
      s2 += chunk_sum<LAY, TPR>(k, t, cols, [&](int j) {
        const float d = v[k].get(j) - mean;
        return d * d;
      });
    const float rstd = inverse_root(row_sum<TPR>(s2, red, slot) * inv_n + p.eps);
    if (t == 0 && ok) {
      if (p.mean && !p.rms) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
    uint32_t rm = 0;
    uint32_t yb[CH][4];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = norm_value(v[k].get(j), mean, rstd, w[k][j], b[k][j]);
      if constexpr (BF) {
#pragma unroll
        for (int j = 0; j < 4; ++j) yb[k][j] = bf16x2_bits(f[2 * j], f[2 * j + 1]);
        if (p.y && ok)
          store_chunk<LAY, TPR>(static_cast<uint16_t *>(p.y) + r * cols, yb[k], k, t, cols);
        if (MODE != NORM_Y) {
          const uint32_t keep = ok && chunk_start<TPR>(k, t) < cols ? 0x7FFF7FFFu : 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t m = yb[k][j] & keep;
            rm = pk_max(rm, m);
            if (MODE == NORM_RW) cm[k][j] = pk_max(cm[k][j], m);
          }
        }
      } else {
        if (ok) store_chunk<LAY, TPR>(static_cast<float *>(p.y) + r * cols, f, k, t, cols);
      }
    }
    if (MODE == NORM_TW) tw_max = pk_max(tw_max, rm);
    if (MODE == NORM_RW || MODE == NORM_ROWS) {
      // (the next round's row_sum puts a barrier between these reads of redu
      // and the next writes)
      const uint32_t am = row_umax<TPR>(hmax16(rm), redu);
      if (MODE == NORM_RW && t == 0 && ok) p.rowpart[r] = (uint16_t)am;
      if (MODE == NORM_ROWS) {
        const float a = bf16_to_f32(am);
        const float s = scale_from_amax<0>(a);
        if (t == 0 && ok) {
          p.scale[r] = s;
          if (p.amax) p.amax[r] = a;
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int c = chunk_start<TPR>(k, t);
          const uint32_t *d = yb[k];
          const uint32_t q0 =
              fp8x4<0>(bf16_to_f32(d[0] & 0xFFFFu) * s, bf16_to_f32(d[0] >> 16) * s,
                       bf16_to_f32(d[1] & 0xFFFFu) * s, bf16_to_f32(d[1] >> 16) * s);
          const uint32_t q1 =
              fp8x4<0>(bf16_to_f32(d[2] & 0xFFFFu) * s, bf16_to_f32(d[2] >> 16) * s,
                       bf16_to_f32(d[3] & 0xFFFFu) * s, bf16_to_f32(d[3] >> 16) * s);
          if (c < cols && ok) *reinterpret_cast<uint2 *>(p.q + r * cols + c) = make_uint2(q0, q1);
        }
      }
    }
  }
  if (MODE == NORM_TW) {
    __shared__ uint32_t tw[16];
    const uint32_t m = wave_umax(hmax16(tw_max));
    if ((threadIdx.x & 63) == 0) tw[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t a = tw[0];
#pragma unroll
      for (int i = 1; i < block_threads<TPR, MODE>() / 64; ++i) a = max(a, tw[i]);
      p.part[blockIdx.x] = a;
    }
  }
  if (MODE == NORM_RW) {
    // the column maxima of the workgroup's row groups meet in LDS (integer
    // maxima: any order gives the same result)
    constexpr int SPAN = TPR * 8 * CH;            // columns a group covers
    __shared__ uint32_t cred[G > 1 ? SPAN : 1];
    uint16_t *dst = p.colpart + (size_t)blockIdx.x * cols;
    if constexpr (G > 1) {
      for (int c = threadIdx.x; c < SPAN; c += block_threads<TPR, MODE>()) cred[c] = 0;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = chunk_start<TPR>(k, t) + 2 * j;
          atomicMax(&cred[c], cm[k][j] & 0xFFFFu);
          atomicMax(&cred[c + 1], cm[k][j] >> 16);
        }
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += block_threads<TPR, MODE>()) dst[c] = (uint16_t)cred[c];
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) store_chunk<LAY, TPR>(dst, cm[k], k, t, cols);
    }
  }
}

// -------------------------------------------------------------- backward --
//
// A workgroup walks its rows with a fixed set of columns per thread, so the
// weight's and bias's gradients accumulate in registers (fp32) and x and dy
// are read once; both row sums travel through one barrier.  At the end the
// row groups of a workgroup add up in LDS in group order and the workgroup
// writes one partial row per gradient; k_norm_bwd_finish adds the partials
// in a fixed order.  Nothing is atomic: results do not vary between runs.
struct NormBwdArgs {
  const void *dy, *x, *w;
  int wf32, rms;
  const float *mean, *rstd;
  int64_t rows;
  int cols;
  void *dx;                    // may be NULL
  float *part;                 // [gridDim.x][2][cols], or NULL: no dw, db
};

constexpr int BWD_THREADS = 1024;

// The weight is kept in LDS as fp32: 16 registers fewer per thread, which
// is what lets 16 waves of this kernel live on a compute unit.
template <class T, int LAY, int TPR, int CH>
__global__ __launch_bounds__(BWD_THREADS) void k_norm_bwd(NormBwdArgs p) {
  constexpr int G = BWD_THREADS / TPR;
  constexpr int SPAN = TPR * 8 * CH;
  constexpr bool BF = sizeof(T) == 2;
  __shared__ float2 red[2][16];
  // w as float4 pairs: chunk k of thread t at [k][half][t]
  __shared__ float4 lw[CH * 2 * TPR];
  const int t = threadIdx.x % TPR;
  const int g = threadIdx.x / TPR;
  const int wave = threadIdx.x >> 6;
  const int cols = p.cols;
  const float inv_n = 1.0f / (float)cols;
  float dw[CH][8], db[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.f;
    if (g == 0) {
      float w[8];
      load_param<LAY, TPR>(w, p.w, p.wf32, 1.f, k, t, cols);
      lw[(2 * k) * TPR + t] = make_float4(w[0], w[1], w[2], w[3]);
      lw[(2 * k + 1) * TPR + t] = make_float4(w[4], w[5], w[6], w[7]);
    }
  }
  __syncthreads();
  int slot = 0;
  // a round's rows are loaded a round ahead, while the sums of the one before
  // wait at their barrier (16 columns a thread leave no registers for it)
  constexpr bool AHEAD = CH == 1;
  Pack<T> xn[CH], dyn[CH];
  float rstd_n = 0.f, mean_n = 0.f;
  auto load_row = [&](int64_t r0) {
    const int64_t r = min(r0 + g, p.rows - 1);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      load_chunk<LAY, TPR>(xn[k], static_cast<const T *>(p.x) + r * cols, k, t, cols);
      load_chunk<LAY, TPR>(dyn[k], static_cast<const T *>(p.dy) + r * cols, k, t, cols);
    }
    rstd_n = p.rstd[r];
    mean_n = p.rms ? 0.f : p.mean[r];
  };
  const int64_t step = (int64_t)gridDim.x * G;
  if (AHEAD) load_row((int64_t)blockIdx.x * G);
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < p.rows; r0 += step) {
    const bool ok = r0 + g < p.rows;
    const int64_t r = ok ? r0 + g : p.rows - 1;
    if (!AHEAD) load_row(r0);
    Pack<T> x[CH], dy[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      x[k] = xn[k];
      dy[k] = dyn[k];
    }
    const float rstd = rstd_n, mean = mean_n;
    if (AHEAD && r0 + step < p.rows) load_row(r0 + step);
    float s1 = 0.f, s2 = 0.f;                     // sums of g xh and of g
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const float4 w0 = lw[(2 * k) * TPR + t], w1 = lw[(2 * k + 1) * TPR + t];
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = ok && owned<LAY, TPR>(k, j, t, cols);
        const float d = in ? dy[k].get(j) : 0.f;
        const float xh = (x[k].get(j) - mean) * rstd;
        const float e = in ? d * xh : 0.f;
        s1 += e * w[j];
        s2 += d * w[j];
        dw[k][j] += e;
        db[k][j] += d;
      }
    }
    if (p.dx) {
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[slot][wave] = make_float2(s1, s2);
        __syncthreads();
        constexpr int W = TPR / 64;
        const int first = wave / W * W;
        float2 a = red[slot][first];
#pragma unroll
        for (int i = 1; i < W; ++i) {
          a.x += red[slot][first + i].x;
          a.y += red[slot][first + i].y;
        }
        s1 = a.x;
        s2 = a.y;
        slot ^= 1;
      }
      const float c1 = s1 * inv_n;
      const float c2 = p.rms ? 0.f : s2 * inv_n;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float4 w0 = lw[(2 * k) * TPR + t], w1 = lw[(2 * k + 1) * TPR + t];
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (x[k].get(j) - mean) * rstd;
          f[j] = (dy[k].get(j) * w[j] - c2 - xh * c1) * rstd;
        }
        if constexpr (BF) {
          uint32_t d[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = bf16x2_bits(f[2 * j], f[2 * j + 1]);
          if (ok) store_chunk<LAY, TPR>(static_cast<uint16_t *>(p.dx) + r * cols, d, k, t, cols);
        } else {
          if (ok) store_chunk<LAY, TPR>(static_cast<float *>(p.dx) + r * cols, f, k, t, cols);
        }
      }
    }
  }
  if (!p.part) return;
  float *dst = p.part + (size_t)blockIdx.x * 2 * cols;
  // the row groups add up in LDS in group order, one gradient after the
  // other in the weight's place; slot i of the array is element j of chunk k
  // of thread t
  float *sum = reinterpret_cast<float *>(lw);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (G > 1) {
      for (int i = 0; i < G; ++i) {
        __syncthreads();
        if (g == i) {
#pragma unroll
          for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float &s = sum[(k * 8 + j) * TPR + t];
              const float v = half ? db[k][j] : dw[k][j];
              s = i == 0 ? v : s + v;
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
          if (owned<LAY, TPR>(k, j, t, cols)) {
            const int c = column<LAY, TPR>(k, j, t, cols);
            dst[half * cols + c] =
                G > 1 ? sum[(k * 8 + j) * TPR + t] : (half ? db[k][j] : dw[k][j]);
          }
    }
  }
  static_assert(SPAN * sizeof(float) == sizeof(lw), "one float per column");
}

// dw and db from `parts` partial rows.  Workgroup: 64 columns of one of the
// two, 16 slices of the partial rows (slice s takes rows s, s + 16, ...),
// joined in LDS in slice order.  parts = 0 (no rows) gives zeros.
constexpr int FIN_SLICES = 16;
__global__ __launch_bounds__(64 * FIN_SLICES) void k_norm_bwd_finish(
    const float *__restrict__ part, int parts, int cols, float *dw, float *db) {
  const int tiles = (cols + 63) / 64;
  const bool is_b = (int)blockIdx.x >= tiles;
  float *out = is_b ? db : dw;
  if (!out) return;
  const int c = ((int)blockIdx.x - (is_b ? tiles : 0)) * 64 + (threadIdx.x & 63);
  const int sl = threadIdx.x >> 6;
  const int cc = min(c, cols - 1);
  float s = 0.f;
  for (int i0 = sl; i0 < parts; i0 += FIN_SLICES * 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = min(i0 + FIN_SLICES * u, parts - 1);
      v[u] = part[(size_t)i * 2 * cols + (is_b ? cols : 0) + cc];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) s += i0 + FIN_SLICES * u < parts ? v[u] : 0.f;
  }
  __shared__ float red[FIN_SLICES][64];
  red[sl][threadIdx.x & 63] = s;
  __syncthreads();
  if (sl == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < FIN_SLICES; ++i) s += red[i][threadIdx.x];
    out[c] = s;
  }
}

// ---------------------------------------------------------------- launch --

constexpr int kComputeUnits = 256;
// most workgroups of a pass that leaves one partial row each
constexpr int kMaxSlices = kComputeUnits;

// Calls f with a pass's kernel shape (TPR, CH) for `cols` columns: 8 columns a
// thread, or 16 (`wide`, where WIDE allows it; and always for the widest rows).
template <bool WIDE, class F>
hipError_t with_shape(int cols, bool wide, F f) {
#define FP8L_SHAPE(TPR, CH)                                                  \
  if (cols <= (TPR) * 8 * (CH))                                              \
    return f(std::integral_constant<int, TPR>(), std::integral_constant<int, CH>());
  FP8L_SHAPE(64, 1)
  if constexpr (WIDE)
    if (wide) {
      FP8L_SHAPE(64, 2)
      FP8L_SHAPE(128, 2)
      FP8L_SHAPE(256, 2)
      FP8L_SHAPE(512, 2)
    }
  FP8L_SHAPE(128, 1)
  FP8L_SHAPE(256, 1)
  FP8L_SHAPE(512, 1)
  FP8L_SHAPE(1024, 1)
  FP8L_SHAPE(1024, 2)
#undef FP8L_SHAPE
  return hipErrorInvalidValue;
}

// The forward of bf16 rows takes 16 columns a thread where there are at least 4
// rows for every compute unit.  Measured, 16 columns against 8, us.  Per-token
// codes: 256 x 4096 4.1 / 3.7, 1024 x 4096 5.6 / 6.0, 4096 x 4096 14.9 / 16.5,
// 4096 x 8192 25.5 / 27.4; quantize rowwise 1024 x 4096 0.4 more, 4096 x 4096 1.2
// less, 16384 x 4096 11 less (83 in all); tensorwise 2048 x 4096 16.0 / 15.2, 16384 x
// 4096 66.7 / 72.1; y alone 4096 x 4096 13.3 / 12.5, 16384 x 4096 43.5 / 43.1.  (One
// rule for all of them, since their y is to be the same bits.)  fp32 rows take
// 8: 2048 x 4096 16.1 / 13.6, 4096 x 4096 24.0 / 22.1, more rows within 3%.
bool many_rows(int64_t rows) { return rows >= 4 * kComputeUnits; }

template <class T, int LAY, int MODE>
hipError_t launch_norm(const NormArgs &a, int64_t max_blocks, int *blocks, hipStream_t stream) {
  static_assert(TW_MAX_BLOCKS >= kComputeUnits * 8, "one maximum per workgroup");
  auto launch = [&](auto tpr, auto ch) {
    constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
    constexpr int BLK = block_threads<TPR, MODE>();
    // as many waves as a compute unit holds, each walking its rows
    if (max_blocks > kComputeUnits * (2048 / BLK)) max_blocks = kComputeUnits * (2048 / BLK);
    int64_t nb = cdiv(a.rows, BLK / TPR);
    if (nb > max_blocks) nb = max_blocks;
    *blocks = (int)nb;
    hipLaunchKernelGGL((k_norm<T, LAY, TPR, CH, MODE>), dim3((unsigned)nb), dim3(BLK), 0, stream,
                       a);
    return hipGetLastError();
  };
  if constexpr (LAY == LAY_SCALAR)
    return launch(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  else
    return with_shape<sizeof(T) == 2>(a.cols, many_rows(a.rows), launch);
}

template <class T, int LAY>
hipError_t launch_bwd(const NormBwdArgs &a, int *blocks, hipStream_t stream) {
  auto launch = [&](auto tpr, auto ch) {
    constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
    int64_t nb = cdiv(a.rows, BWD_THREADS / TPR);
    if (nb > kComputeUnits) nb = kComputeUnits;
    *blocks = (int)nb;
    hipLaunchKernelGGL((k_norm_bwd<T, LAY, TPR, CH>), dim3((unsigned)nb), dim3(BWD_THREADS), 0,
                       stream, a);
    return hipGetLastError();
  };
  if constexpr (LAY == LAY_SCALAR)
    return launch(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  else
    return with_shape<false>(a.cols, false, launch);
}

// f(LAY) for a width
template <class F>
hipError_t with_layout(int64_t cols, F f) {
  if (cols < 8) return f(std::integral_constant<int, LAY_SCALAR>());
  if (cols % 8) return f(std::integral_constant<int, LAY_CHUNKS>());
  return f(std::integral_constant<int, LAY_ALIGNED>());
}

// Where the rowwise partial maxima sit in a workspace: one row of [rows], then
// (on a 256-byte boundary) up to kMaxSlices rows of [cols].
size_t colpart_offset(int64_t rows) {
  return ((size_t)rows * sizeof(uint16_t) + 255) & ~(size_t)255;
}

NormArgs make_args(const NormIn &in, void *y, float *mean, float *rstd) {
  NormArgs a = {};
  a.x = in.x;
  a.w = in.w;
  a.b = in.b;
  a.wf32 = in.wf32;
  a.rms = in.rms;
  a.eps = in.eps;
  a.rows = in.rows;
  a.cols = (int)in.cols;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return a;
}

// Workgroups of a pass without partials (as many as the chip holds).
constexpr int64_t kMaxBlocks = 8 * kComputeUnits;

}  // namespace

size_t norm_workspace_bytes(int64_t rows, int64_t cols, int scaling) {
  // backward: two partial rows of fp32 per workgroup
  size_t bytes = (size_t)kComputeUnits * 2 * (size_t)cols * sizeof(float);
  const size_t fwd = (scaling & FP8L_ROWWISE)
                         ? colpart_offset(rows) + (size_t)kMaxSlices * cols * sizeof(uint16_t)
                         : (size_t)TW_MAX_BLOCKS * sizeof(uint32_t);
  if (bytes < fwd) bytes = fwd;
  return (bytes + 255) & ~(size_t)255;
}

hipError_t norm_fwd_launch(const NormIn &in, int f32, void *y, float *mean, float *rstd,
                           hipStream_t stream) {
  if (in.rows == 0) return hipSuccess;
  const NormArgs a = make_args(in, y, mean, rstd);
  int nb;
  return with_layout(in.cols, [&](auto lay) {
    constexpr int LAY = decltype(lay)::value;
    return f32 ? launch_norm<float, LAY, NORM_Y>(a, kMaxBlocks, &nb, stream)
               : launch_norm<uint16_t, LAY, NORM_Y>(a, kMaxBlocks, &nb, stream);
  });
}

hipError_t norm_rows_launch(const NormIn &in, void *y, float *mean, float *rstd, void *q,
                            float *scale, float *amax_out, hipStream_t stream) {
  if (in.rows == 0) return hipSuccess;
  NormArgs a = make_args(in, y, mean, rstd);
  a.q = static_cast<uint8_t *>(q);
  a.scale = scale;
  a.amax = amax_out;
  int nb;
  return launch_norm<uint16_t, LAY_ALIGNED, NORM_ROWS>(a, kMaxBlocks, &nb, stream);
}

hipError_t norm_quantize_launch(const NormIn &in, int scaling, void *y, float *mean, float *rstd,
                                const Fp8Out &o, void *workspace, hipStream_t stream) {
  NormArgs a = make_args(in, y, mean, rstd);
  CastSource src = {};
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  int nb = 0;
  if (rw) {
    a.rowpart = static_cast<uint16_t *>(workspace);
    a.colpart = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(workspace) +
                                             colpart_offset(in.rows));
    src.rowpart = a.rowpart;
    src.colpart = a.colpart;
    src.row_slices = 1;
  } else {
    a.part = static_cast<uint32_t *>(workspace);
    src.part = a.part;
  }
  if (in.rows > 0) {
    const hipError_t e =
        rw ? launch_norm<uint16_t, LAY_ALIGNED, NORM_RW>(a, kMaxSlices, &nb, stream)
           : launch_norm<uint16_t, LAY_ALIGNED, NORM_TW>(a, TW_MAX_BLOCKS, &nb, stream);
    if (e != hipSuccess) return e;
  }
  if (rw) src.col_slices = nb;
  else src.nparts = nb;
  src.x = y;
  if (!y) {
    src.x = in.x;
    src.w = in.w;
    src.b = in.b;
    src.wf32 = in.wf32;
    src.mean = in.rms ? nullptr : mean;
    src.rstd = rstd;
  }
  return quantize_cast_launch(&src, 1, in.rows, in.cols, scaling, &o, stream);
}

hipError_t norm_bwd_launch(const void *dy, const NormIn &in, int f32, const float *mean,
                           const float *rstd, void *dx, float *dw, float *db, void *workspace,
                           hipStream_t stream) {
  NormBwdArgs a = {};
  a.dy = dy;
  a.x = in.x;
  a.w = in.w;
  a.wf32 = in.wf32;
  a.rms = in.rms;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = in.rows;
  a.cols = (int)in.cols;
  a.dx = dx;
  a.part = dw || db ? static_cast<float *>(workspace) : nullptr;
  int nb = 0;
  if (in.rows > 0) {
    const hipError_t e = with_layout(in.cols, [&](auto lay) {
      constexpr int LAY = decltype(lay)::value;
      return f32 ? launch_bwd<float, LAY>(a, &nb, stream)
                 : launch_bwd<uint16_t, LAY>(a, &nb, stream);
    });
    if (e != hipSuccess) return e;
  }
  if (!a.part) return hipSuccess;
  const int tiles = (int)cdiv(in.cols, 64);
  hipLaunchKernelGGL(k_norm_bwd_finish, dim3((unsigned)(2 * tiles)), dim3(64 * FIN_SLICES), 0,
                     stream, a.part, nb, a.cols, dw, db);
  return hipGetLastError();
}

}  // namespace fp8l
