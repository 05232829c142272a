// A Float8 linear with its epilogue on gfx950: bias, activation and residual where
// the output tile is finished, and the gradient through the activation where the
// next linear's product is.
//
//   z = x W^T + bias,  y = act(z) + residual        (act of the bf16 z)
//   dz = (dy W2) act'(z),  dbias = sum_m dz
//
// Large M: the persistent GEMM with EPI_ACT / EPI_DACT (gemm.hip).  Where its tiles
// are too few, the small tiles of gated.h (64 x 128) with the same forms.  Few tokens:
// below.
// The activations: act.h.
//
// Part of gemm.hip (included at its end).
#pragma once

namespace fp8l {
namespace {

// ---------------------------------------------------------- few tokens --
//
// As k_gated_skinny with one weight: a workgroup owns 16 columns of y, its 8
// waves split the contraction and join through LDS, weights go straight from
// memory to the matrix instruction's operands.  Bound: reading the weights; 1 x 14336 x
// 4096 takes 13.2 us, 4.4 TB/s (a plain read of as much 5.85).
struct ActSkinnyArgs {
  const uint8_t *x, *w;
  const float *sx, *sw;
  ActArgs e;                   // bias, res, act, a (z), C[0] (y), N[0]
  int M, N, K, rowwise;
};

// CB: blocks of 16 columns a workgroup owns.  Two of them keep twice the loads in
// flight and read x half as often: 1 x 14336 x 4096 13.2 us against 15.0 with one.  Below
// N = 8192 they would leave compute units without a workgroup.
template <bool KFULL, int FORM, int CB>
__global__ __launch_bounds__(64 * SK_WAVES) void k_act_skinny(ActSkinnyArgs p) {
  __shared__ v4f red[SK_WAVES][CB][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16 * CB;
  const int K = p.K;
  const int nk = (K + BK - 1) / BK;
  const int kl = (lane >> 4) * 16;
  const uint8_t *rw[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c)                    // (past N: the last row, not stored)
    rw[c] = p.w + (size_t)min(n0 + c * 16 + (lane & 15), p.N - 1) * K;
  const uint8_t *rx = p.x + (size_t)min(lane & 15, p.M - 1) * K;
  v4f acc[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c) acc[c] = (v4f){0.f, 0.f, 0.f, 0.f};
  // (loading a group of k-tiles while the one before it is multiplied gained nothing:
  // 13.2 us either way at 1 x 4096, K = 14336)
  for (int t0 = wave; t0 < nk; t0 += SK_WAVES * SK_UNROLL) {
    v4u fw[SK_UNROLL][CB][2], fx[SK_UNROLL][2];
#pragma unroll
    for (int u = 0; u < SK_UNROLL; ++u) {
      const int t = t0 + u * SK_WAVES;            // past the end: loaded again, not used
      const int k = (t < nk ? t : t0) * BK + kl;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int c = 0; c < CB; ++c) fw[u][c][e] = row_chunk<KFULL>(rw[c], k + e * 64, K);
        fx[u][e] = row_chunk<KFULL>(rx, k + e * 64, K);
      }
    }
#pragma unroll
    for (int u = 0; u < SK_UNROLL; ++u)
      if (t0 + u * SK_WAVES < nk) {               // wave-uniform
        const v8i ax = frag(fx[u][0], fx[u][1]);
#pragma unroll
        for (int c = 0; c < CB; ++c)
          acc[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              frag(fw[u][c][0], fw[u][c][1]), ax, acc[c], 0, 0, 0, 0, 0, 0);
      }
  }
#pragma unroll
  for (int c = 0; c < CB; ++c) red[wave][c][lane] = acc[c];
  __syncthreads();
  // wave c finishes column block c: lane l has token l % 16, columns 4 (l / 16) ...
  const int m = lane & 15;
  const int n = n0 + wave * 16 + (lane >> 4) * 4;
  if (wave >= CB || m >= p.M || n >= p.N) return;
  v4f a = red[0][wave][lane];
#pragma unroll
  for (int w = 1; w < SK_WAVES; ++w) a += red[w][wave][lane];
  const float ia = 1.0f / p.sx[p.rowwise ? m : 0];
  const size_t at = (size_t)m * p.N + n;
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const float2 b = bias_pair(p.e, n + j);
    f[j] = add32((a[j] * ia) * (1.0f / p.sw[p.rowwise ? n + j : 0]), b.x);
    f[j + 1] = add32((a[j + 1] * ia) * (1.0f / p.sw[p.rowwise ? n + j + 1 : 0]), b.y);
  }
  uint2 r = make_uint2(0u, 0u), z;
  if (p.e.res) r = *reinterpret_cast<const uint2 *>(p.e.res + at);
  const uint2 y = act_out4<FORM>(p.e.act, f, p.e.res != nullptr, r, z);
  if (p.e.a) *reinterpret_cast<uint2 *>(p.e.a + at) = z;
  if (p.e.C[0]) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.e.C[0]) + at) = y;
}

// Which calls it takes: up to 16 tokens, but where the contraction is long and a split
// one (below) has enough parts.  A workgroup's loads, half cache lines of 16 rows, take
// about 3 us for every 4096 of K at one token and 4.5 at 16, whatever N is.  Measured, six
// sets of weights in turn, this kernel / split, us, M x N x K: 1 x 14336 x 4096 14.9 /
// 17.0, 1 x 4096 x 14336 15.5 / 17.3, 4 x 4096 x 14336 16.2 / 17.8, 8 x 4096 x 14336 17.5 /
// 17.1, 16 x 4096 x 14336 20.4 / 17.9, 16 x 14336 x 4096 17.9 / 17.7, 16 x 4096 x 4096 6.8 /
// 9.8, 4 x 1024 x 14336 13.1 / 10.2, 8 x 512 x 14336 14.3 / 9.7.  Past N = 16384, where
// nothing is split, more than 4 tokens take the small tiles, which are then 128 or more:
// 8 x 32768 x 8192 42.0 (4 tokens, this kernel: 62.5; not measured against each other at
// one number of tokens).
bool act_few_tokens(int64_t M, int64_t N, int64_t K) {
  return M <= SKINNY_M && !(K >= 64 * BK && (M > 4 || N < 4096));
}

template <int FORM>
hipError_t act_skinny_launch(const ActSkinnyArgs &p, hipStream_t stream) {
  const dim3 block(64 * SK_WAVES);
  const bool wide = p.N >= 2 * 16 * 256;
  const dim3 grid((unsigned)((p.N + (wide ? 31 : 15)) / (wide ? 32 : 16)));
  const bool kfull = p.K % BK == 0;
  auto kern = wide ? (kfull ? k_act_skinny<true, FORM, 2> : k_act_skinny<false, FORM, 2>)
                   : (kfull ? k_act_skinny<true, FORM, 1> : k_act_skinny<false, FORM, 1>);
  hipLaunchKernelGGL(kern, grid, block, 0, stream, p);
  return hipGetLastError();
}

// ---------------------------------------------------- split contraction --
//
// Where one small tile per output leaves most of the compute units idle and the
// contraction is long, its k-tiles go to several workgroups (EPI_SPLIT), whose fp32
// sums this kernel adds in order and finishes.  A thread has 4 columns of a row and
// loads 8 parts together (a call of 50 x 4096 x 14336, us: not split 46.1, parts added one
// by one 22.1, eight at a time 16.9).
struct ActJoinArgs {
  ActArgs e;
  const float *sx, *sw;
  int parts, rowwise;
};
template <int FORM>
__global__ __launch_bounds__(256) void k_act_join(ActJoinArgs p, int64_t n4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const int N = p.e.N[0];
  const int m = (int)(i * 4 / N), n = (int)(i * 4 % N);
  const v4f *src = reinterpret_cast<const v4f *>(p.e.partial) + i;
  uint2 r = make_uint2(0u, 0u), z;
  if (p.e.res) r = *reinterpret_cast<const uint2 *>(p.e.res + (size_t)i * 4);
  v4f a = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < p.parts; s0 += 8) {
    v4f v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = src[(size_t)min(s0 + u, p.parts - 1) * n4];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (s0 + u < p.parts) a += v[u];
  }
  const float ia = 1.0f / p.sx[p.rowwise ? m : 0];
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const float2 b = bias_pair(p.e, n + j);
    f[j] = add32((a[j] * ia) * (1.0f / p.sw[p.rowwise ? n + j : 0]), b.x);
    f[j + 1] = add32((a[j + 1] * ia) * (1.0f / p.sw[p.rowwise ? n + j + 1 : 0]), b.y);
  }
  const uint2 y = act_out4<FORM>(p.e.act, f, p.e.res != nullptr, r, z);
  if (p.e.a) *reinterpret_cast<uint2 *>(p.e.a + (size_t)i * 4) = z;
  if (p.e.C[0]) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.e.C[0]) + (size_t)i * 4) = y;
}

// Parts of the contraction of an [M, N] output; 1: not split.  As many as fill the
// compute units with workgroups of 8 k-tiles or more (of 4 where there are fewer than 32
// k-tiles).  Measured, at most 256 workgroups of 8 / 512 of 8 / 256 of 4 k-tiles / not
// split, us: 50 x 4096 x 14336 17.0 / 18.8 / 16.9 / 45, 64 x 4096 x 4096 10.9 / 10.9 / 12.5 /
// 14.0, 128 x 4096 x 14336 21.0 / 22.3 / 20.9, 50 x 1024 x 14336 10.7 / 10.7 / 12.2, 64 x 2048
// x 2048 9.3 / 9.3 / 8.1, 20 x 512 x 1024 7.0 / 7.0 / 6.6.
constexpr int64_t SPLIT_TILES = 256;              // workgroups
int act_parts(int64_t M, int64_t N, int64_t K, int *part_kt) {
  const int64_t t = tiles(M, TM) * tiles(N, TB), nk = tiles(K, BK);
  const int64_t least = nk >= 32 ? 8 : 4;         // k-tiles of a part
  int64_t s = SPLIT_TILES / t;
  if (s > nk / least) s = nk / least;
  if (t > 128 || s < 2) return 1;
  *part_kt = (int)tiles(nk, s);
  return (int)tiles(nk, *part_kt);
}
size_t act_split_bytes(int64_t M, int64_t N) {
  // at most SPLIT_TILES tiles of partial sums
  const size_t tile = (size_t)TM * TB, mn = (size_t)M * (size_t)N;
  return (size_t)SPLIT_TILES * (mn < tile ? mn : tile) * sizeof(float);
}

template <int FORM>
hipError_t act_split_launch(ActArgs &g, const float *sx, const float *sw, bool rw, int parts,
                            hipStream_t stream) {
  g.tiles_m[0] = (int)tiles(g.M[0], TM);
  g.tiles_n[0] = (int)tiles(g.N[0], TB);
  g.total = g.tiles_m[0] * g.tiles_n[0];
  hipLaunchKernelGGL((k_gate_tile<EPI_SPLIT, 0, false>), dim3((unsigned)g.total, (unsigned)parts),
                     dim3(256), 0, stream, g);
  const ActJoinArgs p = {g, sx, sw, parts, rw};
  const int64_t n4 = (int64_t)g.M[0] * g.N[0] / 4;
  hipLaunchKernelGGL((k_act_join<FORM>), dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, stream,
                     p, n4);
  return hipGetLastError();
}

// An empty contraction: z = bias (EPI_ACT).  One thread per 8 values.
template <int FORM>
__global__ __launch_bounds__(256) void k_act_k0(ActArgs g, int64_t n8) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const int n = (int)(i * 8 % g.N[0]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 b0 = bias_pair(g, n + 4 * h), b1 = bias_pair(g, n + 4 * h + 2);
    const float f[4] = {b0.x, b0.y, b1.x, b1.y};
    const size_t at = (size_t)i * 8 + 4 * h;
    uint2 r = make_uint2(0u, 0u), z;
    if (g.res) r = *reinterpret_cast<const uint2 *>(g.res + at);
    const uint2 y = act_out4<FORM>(g.act, f, g.res != nullptr, r, z);
    if (g.a) *reinterpret_cast<uint2 *>(g.a + at) = z;
    if (g.C[0]) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.C[0]) + at) = y;
  }
}

// ------------------------------------------------------------- launches --

// f(form) for an activation
template <class F>
hipError_t with_form(int act, F f) {
  switch (act_form(act)) {
    case ACT_RELUS: return f(std::integral_constant<int, ACT_RELUS>());
    case ACT_SIG: return f(std::integral_constant<int, ACT_SIG>());
    case ACT_ERF: return f(std::integral_constant<int, ACT_ERF>());
    default: return f(std::integral_constant<int, ACT_ID>());
  }
}

// Slices of the column sums that a call's kernel writes.
int act_slices(int64_t M, int64_t N) { return (int)col_slices(small_tiles(M, N, BN), M); }

template <int EPI, int FA>
hipError_t launch_pers(const ActArgs &g, bool rowwise, int blocks, hipStream_t stream) {
  const bool kfull = g.K[0] % BK == 0;
  auto kern = rowwise ? (kfull ? k_gemm_fp8_pers<true, true, false, FA, false, EPI>
                               : k_gemm_fp8_pers<false, true, false, FA, false, EPI>)
                      : (kfull ? k_gemm_fp8_pers<true, false, false, FA, false, EPI>
                               : k_gemm_fp8_pers<false, false, false, FA, false, EPI>);
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(THREADS), 0, stream, g);
  return hipGetLastError();
}

// One problem, as launch_gate.  (8192 x 14336 x 4096, the GEMM alone: with gelu, z stored
// and y measured 345-420 us, 2.3-2.8 PFLOP/s; the gradient through gelu 430-450, where the
// plain GEMM takes 345.)  Small tiles up to 80 large ones, the limit of the gate's backward
// pass.  Here, small / large with the cast, us: forward with gelu, z, y and codes 40 large
// tiles (1040 x 1808 x 784) 16.4 / 36.9, rowwise 19.2 / 37.3, 64 (1024 x 4096 x 4096) 32.9 /
// 59.9, 35.4 / 61.9, 96 (1536 x 4096 x 4096) 48.4 / 61.6, 52.9 / 63.6, 112 (512 x 14336 x
// 4096) 55.1 / 62.9, 64.5 / 67.8, 128 (2048 x 4096 x 4096) 62.2 / 63.9, 68.6 / 64.4; gradient
// through gelu 40 tiles 16.1 / 35.0, 64 32.5 / 59.1, 96 48.8 / 60.4, 112 55.6 / 61.4, 128 59.2
// / 62.3, without an activation 52.9 / 50.5.  (So from 81 to 112 tiles the small ones would
// still be ahead, by up to a quarter.)
template <int EPI, int FA>
hipError_t launch_act(ActArgs &g, bool rowwise, int *nparts, hipStream_t stream) {
  g.count = 1;
  if (small_tiles(g.M[0], g.N[0], BN)) {
    g.tiles_m[0] = (int)tiles(g.M[0], TM);
    g.tiles_n[0] = (int)tiles(g.N[0], TB);
    g.total = *nparts = g.tiles_m[0] * g.tiles_n[0];
    if (rowwise)
      hipLaunchKernelGGL((k_gate_tile<EPI, FA, true>), dim3((unsigned)g.total), dim3(256), 0,
                         stream, g);
    else
      hipLaunchKernelGGL((k_gate_tile<EPI, FA, false>), dim3((unsigned)g.total), dim3(256), 0,
                         stream, g);
    return hipGetLastError();
  }
  g.tiles_m[0] = (int)tiles(g.M[0], BM);
  g.tiles_n[0] = (int)tiles(g.N[0], BN);
  g.total = g.tiles_m[0] * g.tiles_n[0];
  constexpr int kComputeUnits = 256;
  const int blocks = g.total < kComputeUnits ? g.total : kComputeUnits;
  *nparts = blocks * 4;                           // one per wave
  return is_act(EPI) && g.res ? launch_pers<is_act(EPI) ? EPI - EPI_ACT + EPI_ACT_RES : EPI, FA>(
                                    g, rowwise, blocks, stream)
                              : launch_pers<EPI, FA>(g, rowwise, blocks, stream);
}

}  // namespace

// The workspace: the maxima (this kernel's, or those of a pass of its own), then
// the column sums.
size_t linear_act_maxima_bytes(int64_t M, int64_t N, int scaling) {
  size_t b = gate_share_bytes(M, N, (scaling & FP8L_ROWWISE) != 0, BN);
  for (const size_t q : {quantize_workspace_bytes((M + 15) / 16 * 16, N, scaling),
                         bias_act_maxima_bytes(M, N, scaling)})
    if (b < q) b = q;
  return (b + 255) & ~(size_t)255;
}

size_t linear_act_workspace_bytes(int64_t M, int64_t N, int scaling) {
  // column sums: a slice per 32 rows at most (small tiles); or the partial sums of a
  // split contraction
  size_t sums = (size_t)(2 * tiles(M, TM)) * (size_t)N * sizeof(float);
  const size_t split = act_split_bytes(M, N);
  if (sums < split) sums = split;
  return linear_act_maxima_bytes(M, N, scaling) + ((sums + 255) & ~(size_t)255);
}

hipError_t linear_act_fwd_launch(const LinearActIn &in, int scaling, const Fp8Out *o,
                                 void *workspace, hipStream_t stream) {
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  const int64_t M = in.M, N = in.N, K = in.K;
  // (what is quantized: z stands for y where there is no activation)
  const void *y = in.y ? in.y : in.z;
  const int cast_act = in.y ? FP8L_ACT_NONE : in.act;
  ActArgs g = {};
  g.A[0] = in.xq;
  g.sa[0] = in.sx;
  g.B[0] = in.wq;
  g.sb[0] = in.sw;
  g.C[0] = in.y;
  g.M[0] = (int)M;
  g.N[0] = (int)N;
  g.K[0] = (int)K;
  g.a = in.z;
  g.bias = in.bias;
  g.bias_f32 = in.bias_f32;
  g.res = in.residual;
  g.act = act_consts(in.act);
  CastSource src = {};
  src.x = y;
  src.act = cast_act;
  bool measured = false;                          // the maxima are there
  if (M * N > 0) {
    const hipError_t e = with_form(in.act, [&](auto form) {
      constexpr int FORM = decltype(form)::value;
      if (K == 0) {
        const int64_t n8 = M * N / 8;
        hipLaunchKernelGGL((k_act_k0<FORM>), dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0,
                           stream, g, n8);
        return hipGetLastError();
      }
      if (act_few_tokens(M, N, K)) {
        const ActSkinnyArgs p = {in.xq, in.wq, in.sx, in.sw, g, (int)M, (int)N, (int)K, rw};
        return act_skinny_launch<FORM>(p, stream);
      }
      const int parts = act_parts(M, N, K, &g.part_kt);
      if (parts > 1) {
        g.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                              linear_act_maxima_bytes(M, N, scaling));
        return act_split_launch<FORM>(g, in.sx, in.sw, rw, parts, stream);
      }
      measured = o && o->qt;
      g.maxima = measured;
      g.keys = measured && !rw && !in.y && in.act != FP8L_ACT_NONE;
      if (measured) set_partials(g, 0, src, workspace, rw, BN);
      return launch_act<EPI_ACT + FORM, 0>(g, rw, &src.nparts, stream);
    });
    if (e != hipSuccess) return e;
  }
  if (!o) return hipSuccess;
  // (rows alone: neither qt nor its scales; also of no rows)
  if (!o->qt && !o->scale_t && rw) return quantize_rows_launch(y, cast_act, M, N, *o, stream);
  if (measured) return quantize_cast_launch(&src, 1, M, N, scaling, o, stream);
  return quantize_act_launch(y, cast_act, M, N, scaling, *o, workspace, stream);
}

hipError_t linear_act_bwd_launch(const uint8_t *dyq, const float *sdy, const uint8_t *wtq,
                                 const float *swt, const uint16_t *z, int act, int64_t M,
                                 int64_t H, int64_t D, int scaling, uint16_t *dz, void *dbias,
                                 int dbias_f32, const Fp8Out &o, void *workspace,
                                 hipStream_t stream) {
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  float *sums = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                          linear_act_maxima_bytes(M, H, scaling));
  if (M * H == 0 || D == 0) {                     // dz is empty or zero
    if (M * H > 0) {
      const hipError_t e = fill_zero(dz, 2 * M * H, stream);
      if (e != hipSuccess) return e;
    }
    if (dbias) {
      const hipError_t e = column_sums_launch(nullptr, 0, H, dbias, dbias_f32, stream);
      if (e != hipSuccess) return e;
    }
    return quantize_launch(dz, M, H, scaling, o.q, o.qt, o.scale, o.scale_t, o.amax, workspace,
                           stream);
  }
  ActArgs g = {};
  g.A[0] = dyq;
  g.sa[0] = sdy;
  g.B[0] = wtq;
  g.sb[0] = swt;
  g.C[0] = dz;
  g.M[0] = (int)M;
  g.N[0] = (int)H;
  g.K[0] = (int)D;
  g.a = const_cast<uint16_t *>(z);
  g.act = act_consts(act);
  g.maxima = 1;
  g.colsum = dbias ? sums : nullptr;
  CastSource src = {};
  src.x = dz;
  set_partials(g, 0, src, workspace, rw, BN);
  src.sums = g.colsum;
  src.slices = act_slices(M, H);
  src.sums_f32 = dbias_f32;
  src.sums_out = dbias;
  const hipError_t e = with_form(act, [&](auto form) {
    constexpr int EPI = EPI_DACT + decltype(form)::value;
    return (scaling & FP8L_E5M2) ? launch_act<EPI, 1>(g, rw, &src.nparts, stream)
                                 : launch_act<EPI, 0>(g, rw, &src.nparts, stream);
  });
  if (e != hipSuccess) return e;
  return quantize_cast_launch(&src, 1, M, H, scaling, &o, stream);
}

}  // namespace fp8l
