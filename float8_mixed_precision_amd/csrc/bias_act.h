// What surrounds a linear's epilogue as elementwise passes: the gradient through
// an activation and a bias of a given output gradient, the sums of columns behind a
// bias's gradient, and the quantize of act(z) where y itself was not stored.
//
//   dz = dy act'(z),  dbias = sum_m dz        (z absent: dz = dy)
//
// Bound: HBM.  The pass reads dy (and z) once, writes dz (unless it is dy) and takes
// the amax partial maxima and the column sums on the way; the cast reads dz again,
// mostly from the Infinity Cache.  8192 x 4096 without an activation: 14.5 us for the
// pass (67 MB read, 4.6 TB/s), 22.2 for the cast (134 MB, 6.0 TB/s).  8192 x 14336 with an
// activation: 138 (relu) to 140 us (gelu) for the pass (705 MB, 5.0 to 5.1 TB/s; the form
// chosen at run time costs no more than that), 82 for the cast.
//
// Part of quantize.hip (included at its end).
#pragma once

#include "act.h"

namespace fp8l {
namespace {

// ----------------------------------------------------------------- pass --

struct BiasActArgs {
  const uint16_t *x;           // dy, or z where act(z) is measured
  const uint16_t *z;           // backward: NULL without an activation
  uint16_t *out;               // dz, or NULL: not stored
  float *sums;                 // [tiles_r][cols], or NULL
  uint32_t *part;              // tensorwise: one maximum per workgroup
  uint16_t *rowpart, *colpart; // rowwise: [tiles_c][rows], [tiles_r][cols]
  ActConsts act;
  int form;
  int rows, cols, tiles_c;
};

// Tiles of AM_TR rows x AM_TC columns, one per workgroup: thread (cx, ry) takes the
// 8 columns cx of rows ry + 8 i, all 8 loads in flight together (rows and columns
// clamped into the matrix, results masked).  BWD false: maxima of act(x) alone.
template <bool BWD, bool RW>
__global__ __launch_bounds__(AM_THREADS) void k_bias_act(BiasActArgs p) {
  constexpr int NR = AM_TR / 8;
  const int tid = threadIdx.x;
  const int cx = tid & 31;
  const int ry = tid >> 5;
  const int tile_c = (int)blockIdx.x % p.tiles_c, tile_r = (int)blockIdx.x / p.tiles_c;
  const int r0 = tile_r * AM_TR;
  const int c = tile_c * AM_TC + cx * 8;
  const bool col_ok = c < p.cols;
  const int cl = col_ok ? c : 0;
  U4 x[NR], z[BWD ? NR : 1];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const size_t at = (size_t)min(r0 + ry + 8 * i, p.rows - 1) * p.cols + cl;
    x[i] = load16(p.x + at);
    if constexpr (BWD) z[i] = p.z ? load16(p.z + at) : U4{0, 0, 0, 0};
  }
  uint32_t tw = 0, cm[4] = {0, 0, 0, 0};
  float cs[8] = {};
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + ry + 8 * i;
    const bool ok = col_ok && r < p.rows;
    const uint32_t xd[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float f[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      f[2 * d] = __uint_as_float(xd[d] << 16);
      f[2 * d + 1] = __uint_as_float(xd[d] & 0xFFFF0000u);
    }
    uint32_t o[4];
    if constexpr (BWD) {
      if (p.z) {                                  // uniform
        const uint32_t zd[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          f[e] *= act_slope_any(p.act, p.form,
                                (e & 1) ? __uint_as_float(zd[e >> 1] & 0xFFFF0000u)
                                        : __uint_as_float(zd[e >> 1] << 16));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] += ok ? f[e] : 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = act_value_any(p.act, p.form, f[e]);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = bf16x2_bits(f[2 * d], f[2 * d + 1]);
    if (BWD && p.out && ok)
      *reinterpret_cast<uint4 *>(p.out + (size_t)r * p.cols + c) = make_uint4(o[0], o[1], o[2], o[3]);
    const uint32_t keep = ok ? 0x7FFF7FFFu : 0u;
    uint32_t rm = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t m = o[d] & keep;
      rm = pk_max(rm, m);
      if (RW) cm[d] = pk_max(cm[d], m);
    }
    if (RW) {
      // the 32 lanes of a half-wave share row r
      rm = half_wave_max(hmax16(rm));
      if (cx == 0 && r < p.rows) p.rowpart[(size_t)tile_c * p.rows + r] = (uint16_t)rm;
    } else {
      tw = pk_max(tw, rm);
    }
  }
  __shared__ float red[8][AM_TC];                 // by row phase
  if (RW) {
    uint32_t *cred = reinterpret_cast<uint32_t *>(red);
#pragma unroll
    for (int d = 0; d < 4; ++d) cred[ry * (AM_TC / 2) + cx * 4 + d] = cm[d];
    __syncthreads();
    if (tid < AM_TC / 2) {
      uint32_t m = cred[tid];
#pragma unroll
      for (int k = 1; k < 8; ++k) m = pk_max(m, cred[k * (AM_TC / 2) + tid]);
      const int cc = tile_c * AM_TC + tid * 2;
      if (cc < p.cols)
        *reinterpret_cast<uint32_t *>(p.colpart + (size_t)tile_r * p.cols + cc) = m;
    }
    __syncthreads();
  } else {
    uint32_t *tred = reinterpret_cast<uint32_t *>(red);
    tw = wave_max(hmax16(tw));
    if ((tid & 63) == 0) tred[tid >> 6] = tw;
    __syncthreads();
    if (tid == 0) p.part[blockIdx.x] = max(max(tred[0], tred[1]), max(tred[2], tred[3]));
    __syncthreads();
  }
  if (BWD && p.sums) {
    // the row phases add up in order
#pragma unroll
    for (int e = 0; e < 8; ++e) red[ry][cx * 8 + e] = cs[e];
    __syncthreads();
    const int cc = tile_c * AM_TC + tid;
    if (cc < p.cols) {
      float s = red[0][tid];
#pragma unroll
      for (int k = 1; k < 8; ++k) s += red[k][tid];
      p.sums[(size_t)tile_r * p.cols + cc] = s;
    }
  }
}

// Maxima of the tensorwise pass, reduced to at most TW_MAX_BLOCKS: workgroup b
// takes parts b, b + gridDim.x, ...
__global__ __launch_bounds__(AM_THREADS) void k_fold_maxima(const uint32_t *part, int n,
                                                            uint32_t *out) {
  uint32_t m = 0;
  for (int i = (int)(blockIdx.x + gridDim.x * threadIdx.x); i < n;
       i += (int)gridDim.x * AM_THREADS)
    m = max(m, part[i]);
  __shared__ uint32_t red[AM_THREADS / 64];
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = max(max(red[0], red[1]), max(red[2], red[3]));
}

__global__ __launch_bounds__(64 * FIN_SLICES) void k_column_sums(CastSums s) {
  column_sums<FIN_SLICES>(s, (int)blockIdx.x);
}

// ----------------------------------------------------------- rows alone --

// Codes, scale and amax of each row of act(x), for serving: a workgroup per row,
// which stays in the cache between the maximum and the cast.  Bound: latency, 3.9 us for
// one row of 14336; of 4096 rows the two reads, 39.9 us (59 M values, 3 bytes of each past
// the cache, 4.4 TB/s; 20.8 at 4096 columns, where half of the threads have no values).
__global__ __launch_bounds__(1024) void k_quantize_rows(const uint16_t *__restrict__ x,
                                                        ActConsts act, int form, int cols,
                                                        uint8_t *__restrict__ q,
                                                        float *__restrict__ scale,
                                                        float *__restrict__ amax_out) {
  const uint16_t *row = x + (size_t)blockIdx.x * cols;
  auto values = [&](int c, uint32_t (&o)[4]) {
    const U4 v = load16(row + c);
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    if (act.act != FP8L_ACT_NONE) {               // uniform
#pragma unroll
      for (int d = 0; d < 4; ++d)
        o[d] = bf16x2_bits(act_value_any(act, form, __uint_as_float(o[d] << 16)),
                           act_value_any(act, form, __uint_as_float(o[d] & 0xFFFF0000u)));
    }
  };
  uint32_t m = 0;
  for (int c = threadIdx.x * 8; c < cols; c += 1024 * 8) {
    uint32_t o[4];
    values(c, o);
#pragma unroll
    for (int d = 0; d < 4; ++d) m = pk_max(m, o[d] & 0x7FFF7FFFu);
  }
  __shared__ uint32_t red[16];
  m = wave_max(hmax16(m));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int w = 1; w < 16; ++w) m = max(m, red[w]);
  const float a = bf16_to_f32(m);
  const float s = scale_from_amax<0>(a);
  if (threadIdx.x == 0) {
    scale[blockIdx.x] = s;
    if (amax_out) amax_out[blockIdx.x] = a;
  }
  for (int c = threadIdx.x * 8; c < cols; c += 1024 * 8) {
    uint32_t o[4];
    values(c, o);
    uint2 r;
    r.x = fp8x4<0>(bf16_to_f32(o[0] & 0xFFFFu) * s, bf16_to_f32(o[0] >> 16) * s,
                   bf16_to_f32(o[1] & 0xFFFFu) * s, bf16_to_f32(o[1] >> 16) * s);
    r.y = fp8x4<0>(bf16_to_f32(o[2] & 0xFFFFu) * s, bf16_to_f32(o[2] >> 16) * s,
                   bf16_to_f32(o[3] & 0xFFFFu) * s, bf16_to_f32(o[3] >> 16) * s);
    *reinterpret_cast<uint2 *>(q + (size_t)blockIdx.x * cols + c) = r;
  }
}

// ------------------------------------------------------------- launches --

// The pass, its maxima where a quantize of [rows, cols] expects them in `ws`, and
// the cast of `cast` (an activation `act` applied there, or none) with the column sums
// that src names.
template <bool BWD>
hipError_t bias_act_pass(BiasActArgs a, const void *cast, int cast_act, int scaling,
                         const Fp8Out &o, void *ws, CastSource src, hipStream_t stream) {
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  src.x = cast;
  src.act = cast_act;
  if (rw) quantize_rowwise_partials(ws, a.rows, a.cols, &a.rowpart, &a.colpart);
  else a.part = static_cast<uint32_t *>(ws);
  const int64_t tiles_r = cdiv(a.rows, AM_TR), nb = tiles_r * cdiv(a.cols, AM_TC);
  a.tiles_c = (int)cdiv(a.cols, AM_TC);
  if (nb > 0) {
    if (rw)
      hipLaunchKernelGGL((k_bias_act<BWD, true>), dim3((unsigned)nb), dim3(AM_THREADS), 0, stream,
                         a);
    else
      hipLaunchKernelGGL((k_bias_act<BWD, false>), dim3((unsigned)nb), dim3(AM_THREADS), 0, stream,
                         a);
    if (!rw && nb > TW_MAX_BLOCKS)
      hipLaunchKernelGGL(k_fold_maxima, dim3(TW_MAX_BLOCKS / 2), dim3(AM_THREADS), 0, stream,
                         a.part, (int)nb, a.part + nb);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  src.rowpart = a.rowpart;
  src.colpart = a.colpart;
  src.row_slices = a.tiles_c;
  src.col_slices = (int)tiles_r;
  const bool fold = nb > TW_MAX_BLOCKS;
  src.part = fold ? a.part + nb : a.part;
  src.nparts = (int)(fold ? TW_MAX_BLOCKS / 2 : nb);
  return quantize_cast_launch(&src, 1, a.rows, a.cols, scaling, &o, stream);
}

}  // namespace

size_t bias_act_maxima_bytes(int64_t rows, int64_t cols, int scaling) {
  if (scaling & FP8L_ROWWISE) return quantize_workspace_bytes((rows + 15) / 16 * 16, cols, scaling);
  const size_t n = (size_t)(cdiv(rows, AM_TR) * cdiv(cols, AM_TC)) + TW_MAX_BLOCKS / 2;
  return (n * sizeof(uint32_t) + 255) & ~(size_t)255;
}

hipError_t column_sums_launch(const float *part, int slices, int64_t cols, void *out, int f32,
                              hipStream_t stream) {
  if (cols > 0)
    hipLaunchKernelGGL(k_column_sums, dim3((unsigned)cdiv(cols, 64)), dim3(64 * FIN_SLICES), 0,
                       stream, CastSums{part, slices, (int)cols, f32, 0, out});
  return hipGetLastError();
}

hipError_t quantize_rows_launch(const void *x, int act, int64_t rows, int64_t cols,
                                const Fp8Out &o, hipStream_t stream) {
  // (a launch takes fewer than 2^32 threads)
  constexpr int64_t PIECE = (int64_t)1 << 21;
  for (int64_t r = 0; r < rows; r += PIECE) {
    const int64_t n = rows - r < PIECE ? rows - r : PIECE;
    hipLaunchKernelGGL(k_quantize_rows, dim3((unsigned)n), dim3(1024), 0, stream,
                       static_cast<const uint16_t *>(x) + r * cols, act_consts(act), act_form(act),
                       (int)cols, static_cast<uint8_t *>(o.q) + r * cols, o.scale + r,
                       o.amax ? o.amax + r : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t quantize_act_launch(const void *x, int act, int64_t rows, int64_t cols, int scaling,
                               const Fp8Out &o, void *workspace, hipStream_t stream) {
  if (act == FP8L_ACT_NONE)
    return quantize_launch(x, rows, cols, scaling, o.q, o.qt, o.scale, o.scale_t, o.amax,
                           workspace, stream);
  BiasActArgs a = {};
  a.x = static_cast<const uint16_t *>(x);
  a.act = act_consts(act);
  a.form = act_form(act);
  a.rows = (int)rows;
  a.cols = (int)cols;
  return bias_act_pass<false>(a, x, act, scaling, o, workspace, CastSource{}, stream);
}

hipError_t bias_act_bwd_launch(const void *dy, const void *z, int act, int64_t rows, int64_t cols,
                               int scaling, void *dz, void *dbias, int dbias_f32, const Fp8Out &o,
                               void *maxima, float *sums, hipStream_t stream) {
  BiasActArgs a = {};
  a.x = static_cast<const uint16_t *>(dy);
  a.z = act == FP8L_ACT_NONE ? nullptr : static_cast<const uint16_t *>(z);
  a.out = static_cast<uint16_t *>(dz);
  a.sums = dbias ? sums : nullptr;
  a.act = act_consts(act);
  a.form = act_form(act);
  a.rows = (int)rows;
  a.cols = (int)cols;
  CastSource src = {};
  src.sums = a.sums;
  src.slices = (int)cdiv(rows, AM_TR);
  src.sums_f32 = dbias_f32;
  src.sums_out = dbias;
  const hipError_t e =
      bias_act_pass<true>(a, dz ? dz : dy, FP8L_ACT_NONE, scaling, o, maxima, src, stream);
  if (e != hipSuccess || !dbias || rows > 0) return e;
  return column_sums_launch(nullptr, 0, cols, dbias, dbias_f32, stream);
}

}  // namespace fp8l
