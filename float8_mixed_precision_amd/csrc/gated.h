// Gated feed-forward on gfx950: both projections with the gate in one kernel,
// and the gradient of w2's input with the gate's backward in one kernel.
//
//   a = x W1^T, b = x W3^T, h = silu(a) * b
//   dh = dy W2,  da = dh * b * silu'(a),  db = dh * silu(a)
//
// a, b and dh are rounded to bf16 before the gate, as the separate GEMM and
// elementwise passes round them: a and b are outputs themselves, and h, da and
// db are those of the stored a and b.  (The fp32 accumulators of the same
// operands come out of the same instructions in the same order as the plain
// GEMM's, so a, b and dh equal its outputs bit for bit.)
//
// Large M: the persistent GEMM with EPI_GATE / EPI_DGATE (gemm.hip).  Saved
// against the separate passes: a and b are not read back to form h, dh is
// neither written nor read, and the amax of h, da, db costs no pass.
//
// Few tokens (M <= SKINNY_M): the time is that of reading W1 and W3 once, and
// a tile of 256 rows would leave most compute units without a tile and most
// of each tile's work on padding.  k_gated_skinny: a workgroup owns 16 to 64
// columns of h, its 8 waves split the contraction and join through LDS.
// Weights go straight from memory to the MFMA operands (no byte of them is
// used twice); x comes from L2.
//
// Part of gemm.hip (included at its end).
#pragma once

#include "gemm_schedule.h"

namespace fp8l {
namespace {

// ---------------------------------------------------------- few tokens --

constexpr int SKINNY_M = 64;
constexpr int SK_WAVES = 8;

struct SkinnyArgs {
  const uint8_t *x, *w1, *w3;
  const float *sx, *s1, *s3;
  uint16_t *a, *b, *h;         // a, b: stored unless NULL
  int M, H, K, rowwise;
};

// 16 bytes of a row at its byte k, zeros from K on (K is a multiple of 16)
template <bool KFULL>
__device__ __forceinline__ v4u row_chunk(const uint8_t *row, int k, int K) {
  if (KFULL) return *reinterpret_cast<const v4u *>(row + k);
  const bool in = k < K;
  const v4u v = *reinterpret_cast<const v4u *>(row + (in ? k : 0));
  return in ? v : (v4u){0u, 0u, 0u, 0u};
}

__device__ __forceinline__ v8i frag(v4u lo, v4u hi) {
  return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// MB blocks of 16 tokens, CB blocks of 16 columns of h.  Lane l of a wave
// holds row l % 16 of an operand and the chunks of 16 bytes at l / 16 and l / 16
// + 4 of the 128-byte k-tile (the same for both operands), so that one load
// instruction reads 64 contiguous bytes of each of 16 weight rows.  Rows past
// M or H read the last row (not stored).  UN k-tiles of a wave load together.
// The waves join per block of tokens, so the LDS does not grow with M.
template <int MB, int CB, int UN, bool KFULL>
__global__ __launch_bounds__(64 * SK_WAVES) void k_gated_skinny(SkinnyArgs p) {
  static_assert(CB <= SK_WAVES, "one wave finishes each block of columns");
  __shared__ v4f red[SK_WAVES][2 * CB][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * (16 * CB);
  const int K = p.K;
  const int nk = (K + BK - 1) / BK;
  const int kl = (lane >> 4) * 16;
  const uint8_t *r1[CB], *r3[CB], *rx[MB];
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const size_t row = (size_t)min(n0 + c * 16 + (lane & 15), p.H - 1) * K;
    r1[c] = p.w1 + row;
    r3[c] = p.w3 + row;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
    rx[i] = p.x + (size_t)min(i * 16 + (lane & 15), p.M - 1) * K;
  v4f acc[2][CB][MB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[0][c][i] = acc[1][c][i] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int t0 = wave; t0 < nk; t0 += SK_WAVES * UN) {
    v4u f1[UN][CB][2], f3[UN][CB][2], fx[UN][MB][2];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int t = t0 + u * SK_WAVES;            // past the end: loaded again, not used
      const int k = (t < nk ? t : t0) * BK + kl;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          f1[u][c][e] = row_chunk<KFULL>(r1[c], k + e * 64, K);
          f3[u][c][e] = row_chunk<KFULL>(r3[c], k + e * 64, K);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) fx[u][i][e] = row_chunk<KFULL>(rx[i], k + e * 64, K);
      }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (t0 + u * SK_WAVES < nk) {               // wave-uniform
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const v8i b1 = frag(f1[u][c][0], f1[u][c][1]), b3 = frag(f3[u][c][0], f3[u][c][1]);
#pragma unroll
          for (int i = 0; i < MB; ++i) {
            const v8i ax = frag(fx[u][i][0], fx[u][i][1]);
            acc[0][c][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                b1, ax, acc[0][c][i], 0, 0, 0, 0, 0, 0);
            acc[1][c][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                b3, ax, acc[1][c][i], 0, 0, 0, 0, 0, 0);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    if (i) __syncthreads();                       // the round before has been read
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      red[wave][2 * c][lane] = acc[0][c][i];
      red[wave][2 * c + 1][lane] = acc[1][c][i];
    }
    __syncthreads();
    // wave c, lane l: token i 16 + l % 16, columns n0 + 16 c + 4 (l / 16) ...
    const int c = wave;
    const int m = i * 16 + (lane & 15);
    const int n = n0 + c * 16 + (lane >> 4) * 4;
    if (c < CB && m < p.M && n < p.H) {
      v4f a = red[0][2 * c][lane], b = red[0][2 * c + 1][lane];
#pragma unroll
      for (int w = 1; w < SK_WAVES; ++w) {
        a += red[w][2 * c][lane];
        b += red[w][2 * c + 1][lane];
      }
      const float ia = 1.0f / p.sx[p.rowwise ? m : 0];
      float i1[4], i3[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        i1[j] = 1.0f / p.s1[p.rowwise ? n + j : 0];
        i3[j] = 1.0f / p.s3[p.rowwise ? n + j : 0];
      }
      const uint2 pa = make_uint2(bf16x2_bits((a[0] * ia) * i1[0], (a[1] * ia) * i1[1]),
                                  bf16x2_bits((a[2] * ia) * i1[2], (a[3] * ia) * i1[3]));
      const uint2 pb = make_uint2(bf16x2_bits((b[0] * ia) * i3[0], (b[1] * ia) * i3[1]),
                                  bf16x2_bits((b[2] * ia) * i3[2], (b[3] * ia) * i3[3]));
      const size_t at = (size_t)m * p.H + n;
      if (p.a) {
        *reinterpret_cast<uint2 *>(p.a + at) = pa;
        *reinterpret_cast<uint2 *>(p.b + at) = pb;
      }
      *reinterpret_cast<uint2 *>(p.h + at) =
          make_uint2(gate_fwd2(pa.x, pb.x), gate_fwd2(pa.y, pb.y));
    }
  }
}

template <int MB, int CB, int UN>
hipError_t skinny_shape(const SkinnyArgs &p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.H + 16 * CB - 1) / (16 * CB))), block(64 * SK_WAVES);
  if (p.K % BK == 0)
    hipLaunchKernelGGL((k_gated_skinny<MB, CB, UN, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((k_gated_skinny<MB, CB, UN, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

// Columns per workgroup: x is read by every workgroup, so with more than 16
// tokens a workgroup takes as many columns as still leave nearly every compute
// unit one (14336 columns, K = 4096: 64 tokens 52 us with 16 columns, 40 with
// 32, 33 with 64; 32 tokens 37, 30, 28; one token 24, 25).
hipError_t skinny_launch(const SkinnyArgs &p, hipStream_t stream) {
  if (p.M <= 16) return skinny_shape<1, 1, 4>(p, stream);
  const bool c4 = p.H >= 64 * 192, c2 = p.H >= 32 * 192;
  if (p.M <= 32)
    return c4 ? skinny_shape<2, 4, 1>(p, stream)
              : c2 ? skinny_shape<2, 2, 2>(p, stream) : skinny_shape<2, 1, 2>(p, stream);
  return c4 ? skinny_shape<4, 4, 1>(p, stream)
            : c2 ? skinny_shape<4, 2, 2>(p, stream) : skinny_shape<4, 1, 2>(p, stream);
}

// ------------------------------------------------------------- launches --

// The persistent kernel over one problem.  args: A, sa, B, sb, C, M, N, K and
// the gate's own fields set; tile counts and the grid follow here.
template <int EPI, int FA>
hipError_t launch_gate(GateArgs &g, bool rowwise, int *blocks, hipStream_t stream) {
  constexpr int TN = is_gate(EPI) ? BN / 2 : BN;
  g.count = 1;
  g.tiles_m[0] = (g.M[0] + BM - 1) / BM;
  g.tiles_n[0] = (g.N[0] + TN - 1) / TN;
  g.total = g.tiles_m[0] * g.tiles_n[0];
  constexpr int kComputeUnits = 256;
  *blocks = g.total < kComputeUnits ? g.total : kComputeUnits;
  const bool kfull = g.K[0] % BK == 0;
  auto kern = rowwise ? (kfull ? k_gemm_fp8_pers<true, true, false, FA, false, EPI>
                               : k_gemm_fp8_pers<false, true, false, FA, false, EPI>)
                      : (kfull ? k_gemm_fp8_pers<true, false, false, FA, false, EPI>
                               : k_gemm_fp8_pers<false, false, false, FA, false, EPI>);
  hipLaunchKernelGGL(kern, dim3((unsigned)*blocks), dim3(THREADS), 0, stream, g);
  return hipGetLastError();
}

// Partial maxima of one output in its share of the workspace: rowwise the
// row maxima per wave of a tile (64 columns of h, 128 of da and db), then
// (256-byte aligned) the column maxima per 128 rows; tensorwise one u32 per wave
// of at most 256 workgroups.
int64_t row_slices(int64_t H, int tile) { return (H + tile - 1) / tile * 2; }
int64_t col_slices(int64_t M) { return (M + BM - 1) / BM * 2; }
size_t colpart_at(int64_t M, int64_t H) {
  return ((size_t)(row_slices(H, BN / 2) * M) * sizeof(uint16_t) + 255) & ~(size_t)255;
}
size_t gate_share_bytes(int64_t M, int64_t H, bool rowwise) {
  const size_t b = rowwise ? colpart_at(M, H) + (size_t)(col_slices(M) * H) * sizeof(uint16_t)
                           : (size_t)256 * 4 * sizeof(uint32_t);
  return (b + 255) & ~(size_t)255;
}

// The partial maxima of output o: where the kernel writes them (g) and where
// the cast reads them (src).
void set_partials(GateArgs &g, int o, CastSource &src, void *share, bool rowwise, int tile) {
  if (rowwise) {
    g.rowpart[o] = static_cast<uint16_t *>(share);
    g.colpart[o] = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(share) +
                                                colpart_at(g.M[0], g.N[0]));
    src.rowpart = g.rowpart[o];
    src.colpart = g.colpart[o];
    src.row_slices = (int)row_slices(g.N[0], tile);
    src.col_slices = (int)col_slices(g.M[0]);
  } else {
    g.part[o] = static_cast<uint32_t *>(share);
    src.part = g.part[o];
  }
}

hipError_t fill_zero(void *c, int64_t bytes, hipStream_t stream) {
  const int n16 = (int)(bytes / 16);
  const int nb = n16 < 256 * 1024 ? (n16 + 255) / 256 : 1024;
  hipLaunchKernelGGL((k_gemm_k0<false, false>), dim3((unsigned)nb), dim3(256), 0, stream, c, n16);
  return hipGetLastError();
}

}  // namespace

size_t gated_workspace_bytes(int64_t M, int64_t H, int scaling) {
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  size_t b = 2 * gate_share_bytes(M, H, rw);
  // the forms that leave the quantize or the gate to the separate passes
  const size_t q = quantize_workspace_bytes(M, H, scaling), s = swiglu_workspace_bytes(M, H, scaling);
  if (b < q) b = q;
  return b < s ? s : b;
}

hipError_t gated_fwd_launch(const uint8_t *xq, const float *sx, const uint8_t *w1q,
                            const float *s1, const uint8_t *w3q, const float *s3, int64_t M,
                            int64_t H, int64_t K, int scaling, uint16_t *a, uint16_t *b,
                            uint16_t *h, const Fp8Out *o, void *workspace, hipStream_t stream) {
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  if (M * H > 0 && K > 0 && M > SKINNY_M) {
    GateArgs g = {};
    g.A[0] = xq;
    g.sa[0] = sx;
    g.B[0] = w1q;
    g.sb[0] = s1;
    g.B2 = w3q;
    g.sb2 = s3;
    g.C[0] = h;
    g.M[0] = (int)M;
    g.N[0] = (int)H;
    g.K[0] = (int)K;
    g.a = a;
    g.b = b;
    g.maxima = o != nullptr;
    CastSource src = {};
    src.x = h;
    if (o) set_partials(g, 0, src, workspace, rw, BN / 2);
    int blocks = 0;
    const hipError_t e = a ? launch_gate<EPI_GATE_AB, 0>(g, rw, &blocks, stream)
                           : launch_gate<EPI_GATE, 0>(g, rw, &blocks, stream);
    if (e != hipSuccess || !o) return e;
    src.nparts = blocks * 4;
    return quantize_cast_launch(src, M, H, scaling, *o, stream);
  }
  if (M * H > 0) {
    hipError_t e;
    if (K > 0) {
      const SkinnyArgs p = {xq, w1q, w3q, sx, s1, s3, a, b, h, (int)M, (int)H, (int)K, rw};
      e = skinny_launch(p, stream);
    } else {                                     // an empty contraction: a = b = 0, h = 0
      e = fill_zero(h, 2 * M * H, stream);
      if (e == hipSuccess && a) e = fill_zero(a, 2 * M * H, stream);
      if (e == hipSuccess && a) e = fill_zero(b, 2 * M * H, stream);
    }
    if (e != hipSuccess) return e;
  }
  if (!o) return hipSuccess;
  return quantize_launch(h, M, H, scaling, o->q, o->qt, o->scale, o->scale_t, o->amax, workspace,
                         stream);
}

hipError_t gated_bwd_launch(const uint8_t *dyq, const float *sdy, const uint8_t *w2tq,
                            const float *sw2t, const uint16_t *a, const uint16_t *b, int64_t M,
                            int64_t H, int64_t D, int scaling, uint16_t *da, uint16_t *db,
                            const Fp8Out &qa, const Fp8Out &qb, void *workspace,
                            hipStream_t stream) {
  if (M * H == 0 || D == 0) {
    // dh is empty or zero: the elementwise pass on a zero dh (kept in da)
    if (M * H > 0) {
      const hipError_t e = fill_zero(da, 2 * M * H, stream);
      if (e != hipSuccess) return e;
    }
    return swiglu_bwd_launch(da, a, b, M, H, scaling, da, db, qa, qb, workspace, stream);
  }
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  GateArgs g = {};
  g.A[0] = dyq;
  g.sa[0] = sdy;
  g.B[0] = w2tq;
  g.sb[0] = sw2t;
  g.C[0] = da;
  g.M[0] = (int)M;
  g.N[0] = (int)H;
  g.K[0] = (int)D;
  g.a = const_cast<uint16_t *>(a);
  g.b = const_cast<uint16_t *>(b);
  g.C2 = db;
  g.maxima = 1;
  CastSource sa = {}, sb = {};
  sa.x = da;
  sb.x = db;
  set_partials(g, 0, sa, workspace, rw, BN);
  set_partials(g, 1, sb, static_cast<uint8_t *>(workspace) + gate_share_bytes(M, H, rw), rw, BN);
  int blocks = 0;
  hipError_t e = (scaling & FP8L_E5M2) ? launch_gate<EPI_DGATE, 1>(g, rw, &blocks, stream)
                                       : launch_gate<EPI_DGATE, 0>(g, rw, &blocks, stream);
  if (e != hipSuccess) return e;
  sa.nparts = sb.nparts = blocks * 4;
  e = quantize_cast_launch(sa, M, H, scaling, qa, stream);
  if (e != hipSuccess) return e;
  return quantize_cast_launch(sb, M, H, scaling, qb, stream);
}

}  // namespace fp8l
