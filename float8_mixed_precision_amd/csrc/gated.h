// Gated feed-forward on gfx950: both projections with the gate in one kernel,
// and the gradient of w2's input with the gate's backward in one kernel.
//
//   a = x W1^T, b = x W3^T, h = silu(a) * b
//   dh = dy W2,  da = dh * b * silu'(a),  db = dh * silu(a)
//
// a, b and dh are rounded to bf16 before the gate, as the separate GEMM and
// elementwise passes round them: a and b are outputs themselves, and h, da and
// db are those of the stored a and b.  (In the large and small tiles the fp32
// accumulators of the same operands come out of the same instructions in the
// same order as the plain GEMM's, so a, b and dh equal its outputs bit for bit;
// the few-token kernel splits the contraction and adds in another order.)
//
// Large M: the persistent GEMM with EPI_GATE / EPI_DGATE (gemm.hip).  Saved
// against the separate passes: a and b are not read back to form h, dh is
// neither written nor read, and the amax of h, da, db costs no pass.
//
// In between, where those tiles are too few for the compute units:
// k_gate_tile, one tile of 64 rows x 64 columns of h (128 of da and db) per
// workgroup.
//
// Few tokens (at most one MFMA block, few_tokens): k_gated_skinny, bound by
// reading W1 and W3 once.  A workgroup owns 16 columns of h, its 8
// waves split the contraction and join through LDS; weights go straight from
// memory to the MFMA operands (no byte of them is used twice), x comes from L2.
//
// Part of gemm.hip (included at its end).
#pragma once

#include "gemm_schedule.h"

namespace fp8l {
namespace {

// ---------------------------------------------------------- few tokens --

constexpr int SKINNY_M = 16;
constexpr int SK_WAVES = 8;
constexpr int SK_UNROLL = 4;   // k-tiles of a wave that load together

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

// Lane l of a wave holds row l % 16 of an operand and the chunks of 16 bytes at
// l / 16 and l / 16 + 4 of the 128-byte k-tile (the same for both operands), so
// that one load instruction reads 64 contiguous bytes of each of 16 weight
// rows.  Rows past M read row M - 1 (not stored).
//
// One token, 14336 columns, K = 4096, rowwise: 25.5 us with six sets of weights in
// turn, 4.6 TB/s from memory (a plain read of 112 MiB: 20.1 us, 5.85 TB/s); 21.8 us
// with one set again and again, which the Infinity Cache then holds in part.
// Called from Python, one set: 23.8 us; with 4 waves and the same loads in flight
// 26, with 2 k-tiles together 28, with non-temporal loads 27.
template <bool KFULL>
__global__ __launch_bounds__(64 * SK_WAVES) void k_gated_skinny(SkinnyArgs p) {
  __shared__ v4f red[SK_WAVES][2][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16;
  const int K = p.K;
  const int nk = (K + BK - 1) / BK;
  const int kl = (lane >> 4) * 16;
  const uint8_t *r1 = p.w1 + (size_t)(n0 + (lane & 15)) * K;
  const uint8_t *r3 = p.w3 + (size_t)(n0 + (lane & 15)) * K;
  const uint8_t *rx = p.x + (size_t)min(lane & 15, p.M - 1) * K;
  v4f acc1 = {0.f, 0.f, 0.f, 0.f}, acc3 = acc1;
  for (int t0 = wave; t0 < nk; t0 += SK_WAVES * SK_UNROLL) {
    v4u f1[SK_UNROLL][2], f3[SK_UNROLL][2], fx[SK_UNROLL][2];
#pragma unroll
    for (int u = 0; u < SK_UNROLL; ++u) {
      const int t = t0 + u * SK_WAVES;            // past the end: loaded again, not used
      const int k = (t < nk ? t : t0) * BK + kl;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f1[u][e] = row_chunk<KFULL>(r1, k + e * 64, K);
        f3[u][e] = row_chunk<KFULL>(r3, k + e * 64, K);
        fx[u][e] = row_chunk<KFULL>(rx, k + e * 64, K);
      }
    }
#pragma unroll
    for (int u = 0; u < SK_UNROLL; ++u) {
      if (t0 + u * SK_WAVES < nk) {               // wave-uniform
        const v8i ax = frag(fx[u][0], fx[u][1]);
        acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(f1[u][0], f1[u][1]), ax, acc1,
                                                                0, 0, 0, 0, 0, 0);
        acc3 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(f3[u][0], f3[u][1]), ax, acc3,
                                                                0, 0, 0, 0, 0, 0);
      }
    }
  }
  red[wave][0][lane] = acc1;
  red[wave][1][lane] = acc3;
  __syncthreads();
  // lane l of the first wave: token l % 16, columns n0 + 4 (l / 16) ...
  const int m = lane & 15;
  const int n = n0 + (lane >> 4) * 4;
  if (wave > 0 || m >= p.M) return;
  v4f a = red[0][0][lane], b = red[0][1][lane];
#pragma unroll
  for (int w = 1; w < SK_WAVES; ++w) {
    a += red[w][0][lane];
    b += red[w][1][lane];
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
  *reinterpret_cast<uint2 *>(p.h + at) = make_uint2(gate_fwd2(pa.x, pb.x), gate_fwd2(pa.y, pb.y));
}

// Which calls it takes: up to 4 tokens, and up to 16 where the small tiles
// below, one per 64 columns, are fewer than three for every four compute
// units.  Measured, this kernel against the tiles, K = 4096, us for one token
// and for 16: H = 4096 7.5 / 15.1 and 8.3 / 15.3, 8192 13.5 / 15.4 and 15.0 / 16.3,
// 10240 19.3 / 21.3 and 21.6 / 21.0, 14336 24.1 / 23.0 (rowwise 24.3 / 27.4) and
// 29.5 / 24.3; 4 tokens 25.2 / 26.5, 8 tokens 26.7 / 23.4.  Those are of one set of
// weights, partly in the Infinity Cache.  From memory (H = 14336, six sets in
// turn, rowwise and tensorwise) this kernel is ahead for longer: one token 25.5 /
// 29.4 and 25.8 / 28.8, 4 tokens 26.2 / 29.4 and 26.5 / 28.9, 8 tokens 27.3 / 29.4 and
// 27.2 / 28.9, 16 tokens 29.7 / 29.4 and 30.0 / 28.9.  (With more tokens every
// workgroup reads all of x: a form with 4 token blocks took 33 us at 64 tokens
// and H = 14336, the tiles 28.)
bool few_tokens(int64_t M, int64_t H) { return M <= 4 || (M <= SKINNY_M && H < 64 * 192); }

hipError_t skinny_launch(const SkinnyArgs &p, hipStream_t stream) {
  const dim3 grid((unsigned)(p.H / 16)), block(64 * SK_WAVES);
  if (p.K % BK == 0)
    hipLaunchKernelGGL((k_gated_skinny<true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((k_gated_skinny<false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

// ---------------------------------------------------------- small tiles --
//
// Tile: 64 rows x 128 rows of the B slab (EPI_GATE: 64 of B and the same 64 of
// B2, 32 + 32 per wave column).  4 waves in a 2 x 2 grid own 32 x 64 each, 2 x 4
// blocks of the same MFMA.  Three 24 KB stages of one 128-byte k-tile, filled
// by DMA two k-tiles ahead, in the layout of the large kernel (16-byte chunk c
// of row r at c ^ h(r)); one barrier per k-tile.  Two workgroups live on a
// compute unit and cover each other's waits.  The epilogue works in the
// accumulators' own layout: 8-byte accesses of 4 columns, 32 contiguous bytes a
// row, no staging.
//
// Training forward of 1040 x 1808 (K = 784, rowwise, with the quantize of h) 20 us
// against 28 with the 75 tiles of the large kernel, backward of 528 x 4112 (K =
// 400, with both quantizes) 26 against 42 with its 51 tiles: too little work
// to fill the chip either way.  Of the forward's 15.7 us in this kernel the 56
// matrix instructions of a wave are less than 1; the rest (loads of 7 k-tiles two
// ahead, the epilogue of a launch that is one round of workgroups) is not
// broken down.
constexpr int TM = 64;
constexpr int TB = 128;                            // rows of the B slab
constexpr int T_STAGE = (TM + TB) * BK;            // 24 KB
constexpr int T_STAGES = 3;

// k-tiles of a part of a split contraction
__device__ __forceinline__ int part_kt(const ActArgs &g) { return g.part_kt; }
__device__ __forceinline__ int part_kt(const GateArgs &) { return 0; }

template <int EPI, int FA, bool RW>
__global__ __launch_bounds__(256) void k_gate_tile(typename ArgsOf<EPI>::type g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T_STAGES * T_STAGE];
  constexpr bool GATE = is_gate(EPI);
  constexpr bool ACT = is_act(EPI), DACT = is_dact(EPI), SPLIT = EPI == EPI_SPLIT;
  constexpr int NOUT = EPI == EPI_DGATE ? 2 : 1;   // tensors that are quantized
  constexpr int TN = GATE ? TB / 2 : TB;           // output columns of the tile
  constexpr int WC = TN / 2;                       // of a wave
  constexpr int NJ = WC / FR;                      // output blocks of a wave along n
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int M = g.M[0], N = g.N[0], K = g.K[0];
  // (EPI_SPLIT: the k-tiles of this part)
  const int first_kt = SPLIT ? (int)blockIdx.y * part_kt(g) : 0;
  const int nk = SPLIT ? min(part_kt(g), (K + BK - 1) / BK - first_kt) : (K + BK - 1) / BK;
  // workgroups are dealt to the XCDs round-robin; each XCD takes a contiguous
  // share of the tiles, rows fastest, so that it reads its own rows of B
  const int x = blockIdx.x % NUM_XCD, total = g.total;
  int q = blockIdx.x / NUM_XCD;
  for (int xx = 0; xx < x; ++xx) q += (total - xx + NUM_XCD - 1) / NUM_XCD;
  const int m0 = q % g.tiles_m[0] * TM, n0 = q / g.tiles_m[0] * TN;

  // DMA: wave w fills A rows w 16 + (0..15) and slab rows w 32 + (0..31) of B,
  // 8 rows an instruction.  Rows past the matrix fail the bounds check of the
  // vector offset and read as zero; so do chunks past K.
  const uint8_t *B = g.B[0];
  int nb0 = n0 + wave * 32;                        // first B row of this wave's part
  if (GATE) {
    B = (wave & 1) ? g.B2 : B;
    nb0 = n0 + (wave >> 1) * 32;
  }
  const int ma0 = m0 + wave * 16;
  const __amdgpu_buffer_rsrc_t rsA = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(g.A[0] + (size_t)min(ma0, M) * K), (short)0, max(M - ma0, 0) * K, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsB = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(B + (size_t)min(nb0, N) * K), (short)0, max(N - nb0, 0) * K, 0x00020000);
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)lds;
  const int lr = lane >> 3;
  auto fill = [&](int t) {
    const int k0 = (first_kt + t) * BK;
    const uint32_t st = base + (uint32_t)(t % T_STAGES * T_STAGE);
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int r = (i < 2 ? i : i - 2) * 8 + lr;  // row of this wave's part
      // h(r) of the slab row: parts start at multiples of 16 rows
      const int c = (lane & 7) ^ (r & 7) ^ ((r >> 3) & 1);
      const uint32_t off = k0 + c * 16 < K ? (uint32_t)r * (uint32_t)K + (uint32_t)(c * 16) : OOB;
      if (i < 2) dma16(rsA, st + (uint32_t)((wave * 16 + i * 8) * BK), off, (uint32_t)k0);
      else dma16(rsB, st + (uint32_t)((TM + wave * 32 + (i - 2) * 8) * BK), off, (uint32_t)k0);
    }
  };
  v4f acc[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[j][i] = (v4f){0.f, 0.f, 0.f, 0.f};
  // fragment reads: lane l, row l % 16, chunks 2 (l / 16) and 2 (l / 16) + 1
  const int l16 = lane & 15, g4 = lane >> 4;
  const int hr = (lane & 7) ^ ((lane >> 3) & 1);
  const int c0 = ((2 * g4) ^ hr) << 4, c1 = ((2 * g4 + 1) ^ hr) << 4;
  const int ra = (wm * 32 + l16) * BK, rb = (TM + wn * 64 + l16) * BK;
  // the places of the lane's outputs; their scales, and EPI_DGATE's a and b, are
  // read first of all
  const int mrow = m0 + wm * 32 + l16;
  const int ncol = n0 + wn * WC + g4 * 4;
  uint2 ga[GATE ? 1 : NJ][2], gb[GATE ? 1 : NJ][2];
  float bias[ACT ? NJ : 1][4];
  if constexpr (ACT || DACT) {
    // the residual or z, and the bias
    const uint16_t *in = ACT ? g.res : EPI != EPI_DACT + ACT_ID ? g.a : nullptr;
    if (in) {                                      // uniform
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          ga[j][i] = *reinterpret_cast<const uint2 *>(
              in + (size_t)min(mrow + i * FR, M - 1) * N + min(ncol + j * FR, N - 4));
    }
    if constexpr (ACT) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 b = bias_pair(g, ncol + j * FR + e);
          bias[j][e] = b.x;
          bias[j][e + 1] = b.y;
        }
    }
  }
  if constexpr (EPI == EPI_DGATE) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t at = (size_t)min(mrow + i * FR, M - 1) * N + min(ncol + j * FR, N - 4);
        ga[j][i] = *reinterpret_cast<const uint2 *>(g.a + at);
        gb[j][i] = *reinterpret_cast<const uint2 *>(g.b + at);
      }
  }
  float ia[2], ib[NJ][4], ib2[NJ][4];
#pragma unroll
  for (int i = 0; i < 2 && !SPLIT; ++i) ia[i] = g.sa[0][RW ? min(mrow + i * FR, M - 1) : 0];
#pragma unroll
  for (int j = 0; j < NJ && !SPLIT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = RW ? min(ncol + j * FR + e, N - 1) : 0;
      ib[j][e] = g.sb[0][at];
      if constexpr (GATE) ib2[j][e] = g.sb2[at];
    }
  fill(0);
  if (nk > 1) fill(1);
  for (int t = 0; t < nk; ++t) {
    // this wave's part of k-tile t has arrived (k-tile t + 1 may be on its way)
    if (t + 1 < nk) wait_vmcnt<6>();
    else wait_vmcnt0();
    wait_lgkm0();
    barrier_lds();                                 // all parts; k-tile t - 1 has been read
    if (t + 2 < nk) fill(t + 2);
    const uint8_t *st = lds + t % T_STAGES * T_STAGE;
    v8i fa[2], fb[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      fa[i] = frag(*reinterpret_cast<const v4u *>(st + ra + i * FR * BK + c0),
                   *reinterpret_cast<const v4u *>(st + ra + i * FR * BK + c1));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      fb[j] = frag(*reinterpret_cast<const v4u *>(st + rb + j * FR * BK + c0),
                   *reinterpret_cast<const v4u *>(st + rb + j * FR * BK + c1));
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i], acc[j][i], 0,
                                                                     FA, 0, 0, 0, 0);
  }

  // ---- epilogue: lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of its
  // blocks
  if constexpr (SPLIT) {
    float *dst = g.partial + (size_t)blockIdx.y * M * N;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = mrow + i * FR, n = ncol + j * FR;
        if (m < M && n < N) *reinterpret_cast<v4f *>(dst + (size_t)m * N + n) = acc[j][i];
      }
    return;
  }
  uint16_t *C = static_cast<uint16_t *>(g.C[0]);
  uint32_t rm[2][2] = {};                          // [output][i]: row maxima (u16 pairs)
  uint2 cm[2][NJ] = {};                            // [output][j]: column maxima
  float cs[DACT ? NJ : 1][4] = {};                 // column sums
#pragma unroll
  for (int i = 0; i < 2; ++i) ia[i] = 1.0f / ia[i];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int n = ncol + j * FR;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ib[j][e] = 1.0f / ib[j][e];
      if (GATE) ib2[j][e] = 1.0f / ib2[j][e];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = mrow + i * FR;
      const bool ok = m < M && n < N;
      const size_t at = (size_t)m * N + n;
      const v4f p = acc[j][i];
      const uint2 pa =
          make_uint2(bf16x2_bits((p[0] * ia[i]) * ib[j][0], (p[1] * ia[i]) * ib[j][1]),
                     bf16x2_bits((p[2] * ia[i]) * ib[j][2], (p[3] * ia[i]) * ib[j][3]));
      uint2 o[2] = {};
      if constexpr (GATE) {
        const v4f r = acc[j + NJ][i];
        const uint2 pb =
            make_uint2(bf16x2_bits((r[0] * ia[i]) * ib2[j][0], (r[1] * ia[i]) * ib2[j][1]),
                       bf16x2_bits((r[2] * ia[i]) * ib2[j][2], (r[3] * ia[i]) * ib2[j][3]));
        if (EPI == EPI_GATE_AB && ok) {
          *reinterpret_cast<uint2 *>(g.a + at) = pa;
          *reinterpret_cast<uint2 *>(g.b + at) = pb;
        }
        o[0] = make_uint2(gate_fwd2(pa.x, pb.x), gate_fwd2(pa.y, pb.y));
        if (ok) *reinterpret_cast<uint2 *>(C + at) = o[0];
      } else if constexpr (ACT) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = add32((p[e] * ia[i]) * ib[j][e], bias[j][e]);
        const uint2 r = g.res ? ga[j][i] : make_uint2(0u, 0u);
        uint2 z;
        o[0] = act_out4<form_of(EPI)>(g.act, f, g.res != nullptr, r, z);
        if (ok && g.a) *reinterpret_cast<uint2 *>(g.a + at) = z;
        if (ok && C) *reinterpret_cast<uint2 *>(C + at) = o[0];
      } else if constexpr (DACT) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = (p[e] * ia[i]) * ib[j][e];
        if constexpr (EPI != EPI_DACT + ACT_ID) {
          const float z[4] = {bf16_lo(ga[j][i].x), bf16_hi(ga[j][i].x), bf16_lo(ga[j][i].y),
                              bf16_hi(ga[j][i].y)};
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] *= act_slope<form_of(EPI)>(g.act, z[e]);
        }
        o[0] = make_uint2(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]));
        if (ok) *reinterpret_cast<uint2 *>(C + at) = o[0];
        // (a row past M repeats the last one)
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[j][e] += ok ? f[e] : 0.f;
      } else {
        gate_bwd2(pa.x, ga[j][i].x, gb[j][i].x, o[0].x, o[1].x);
        gate_bwd2(pa.y, ga[j][i].y, gb[j][i].y, o[0].y, o[1].y);
        if (ok) {
          *reinterpret_cast<uint2 *>(C + at) = o[0];
          *reinterpret_cast<uint2 *>(g.C2 + at) = o[1];
        }
      }
      const uint32_t keep = ok ? 0x7FFF7FFFu : 0u;
#pragma unroll
      for (int k = 0; k < NOUT; ++k) {
        const uint32_t v0 = o[k].x & keep, v1 = o[k].y & keep;
        rm[k][i] = pk_max(rm[k][i], pk_max(v0, v1));
        if (RW) cm[k][j] = make_uint2(pk_max(cm[k][j].x, v0), pk_max(cm[k][j].y, v1));
      }
    }
  }
  if constexpr (DACT) {
    if (g.colsum) {                                // uniform
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        // the 16 rows of a block add up in a fixed order
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int w = 1; w < 16; w <<= 1) cs[j][e] += __shfl_xor(cs[j][e], w);
        }
        const int n = ncol + j * FR;
        if (l16 == 0 && n < N)
          *reinterpret_cast<v4f *>(g.colsum + (size_t)(m0 / TM * 2 + wm) * N + n) =
              (v4f){cs[j][0], cs[j][1], cs[j][2], cs[j][3]};
      }
    }
  }
  if (!g.maxima) return;                           // uniform
#pragma unroll
  for (int k = 0; k < NOUT; ++k) {
    if (RW) {
      const int tile_n = n0 / TN, tile_m = m0 / TM;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t v = hmax16(rm[k][i]);
        v = max(v, (uint32_t)__shfl_xor((int)v, 16));
        v = max(v, (uint32_t)__shfl_xor((int)v, 32));
        if (lane < 16 && mrow + i * FR < M)
          g.rowpart[k][(size_t)(tile_n * 2 + wn) * M + mrow + i * FR] = (uint16_t)v;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint2 v = cm[k][j];
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          v.x = pk_max(v.x, (uint32_t)__shfl_xor((int)v.x, o));
          v.y = pk_max(v.y, (uint32_t)__shfl_xor((int)v.y, o));
        }
        const int n = ncol + j * FR;
        if (l16 == 0 && n < N)
          *reinterpret_cast<uint2 *>(g.colpart[k] + (size_t)(tile_m * 2 + wm) * N + n) = v;
      }
    } else {
      // one maximum per workgroup, through LDS that the main loop is done with
      uint32_t *red = reinterpret_cast<uint32_t *>(lds) + k * 4;
      const uint32_t v = wave_max(hmax16(pk_max(rm[k][0], rm[k][1])));
      if (k == 0) __syncthreads();
      if (lane == 0) red[wave] = v;
      __syncthreads();
      if (threadIdx.x == 0)
        g.part[k][blockIdx.x] = max(max(red[0], red[1]), max(red[2], red[3]));
    }
  }
}

// ------------------------------------------------------------- launches --

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// Whether an [M, H] output takes the small tiles (a large tile is 256 rows x
// bn columns): while the large ones leave about half the compute units
// without any.  Measured, small against large, in us.  Forward with a, b and
// the quantize of h: 112 large tiles 29 / 47 (80 x 14336), 48 / 49 (256 x 14336),
// 120 tiles 26 / 28, 128 tiles 35 / 35 and 49 / 49, 224 tiles 60 / 52, 256 tiles 45 /
// 34.  Backward: 51 tiles 23 / 33, 64 tiles 32 / 45 and 38 / 60, 85 tiles 44 / 40, 112
// tiles 55 / 60, 128 tiles 47 / 43.  One row of small tiles is better than one of
// large ones at any number: 64 x 28672, K = 8192, 224 tiles, 103 / 132; backward 112
// tiles 51 / 90; at 128 rows 137 / 154 but rowwise 154 / 129.  (No limit suits every
// shape: the backward's 80 has 112 tiles, 5 us better small, on the wrong side,
// with 85 and 128, 4 us better large, on the right one.  The tensorwise
// maxima, one per small tile, bound that number.)
constexpr int64_t SMALL_TILES = 128, SMALL_TILES_BWD = 80;
bool small_tiles(int64_t M, int64_t H, int bn) {
  return tiles(M, BM) * tiles(H, bn) <= (bn == BN ? SMALL_TILES_BWD : SMALL_TILES) ||
         (M <= TM && tiles(H, bn / 2) <= 8 * SMALL_TILES);
}

// One problem.  args: A, sa, B, sb, C, M, N, K and the gate's own fields set;
// tile counts and the grid follow here.  nparts: tensorwise maxima written.
template <int EPI, int FA>
hipError_t launch_gate(GateArgs &g, bool rowwise, int *nparts, hipStream_t stream) {
  constexpr int TN = is_gate(EPI) ? BN / 2 : BN;
  g.count = 1;
  if (small_tiles(g.M[0], g.N[0], TN)) {
    g.tiles_m[0] = (int)tiles(g.M[0], TM);
    g.tiles_n[0] = (int)tiles(g.N[0], TN / 2);
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
  g.tiles_n[0] = (int)tiles(g.N[0], TN);
  g.total = g.tiles_m[0] * g.tiles_n[0];
  constexpr int kComputeUnits = 256;
  const int blocks = g.total < kComputeUnits ? g.total : kComputeUnits;
  *nparts = blocks * 4;                           // one per wave
  const bool kfull = g.K[0] % BK == 0;
  auto kern = rowwise ? (kfull ? k_gemm_fp8_pers<true, true, false, FA, false, EPI>
                               : k_gemm_fp8_pers<false, true, false, FA, false, EPI>)
                      : (kfull ? k_gemm_fp8_pers<true, false, false, FA, false, EPI>
                               : k_gemm_fp8_pers<false, false, false, FA, false, EPI>);
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(THREADS), 0, stream, g);
  return hipGetLastError();
}

// Partial maxima of one output in its share of the workspace: rowwise the
// row maxima per wave column of the tiles, then (256-byte aligned) the column
// maxima per wave row; tensorwise one u32 per wave of at most 256 workgroups, or
// per workgroup of at most 8 SMALL_TILES.  A large tile holds 8 small ones.
// (Columns per large tile: bn; a small tile has half as many.)
int64_t row_slices(bool small, int64_t H, int bn) { return 2 * tiles(H, small ? bn / 2 : bn); }
int64_t col_slices(bool small, int64_t M) { return 2 * tiles(M, small ? TM : BM); }
size_t colpart_at(bool small, int64_t M, int64_t H, int bn) {
  return ((size_t)(row_slices(small, H, bn) * M) * sizeof(uint16_t) + 255) & ~(size_t)255;
}
size_t rowwise_share(bool small, int64_t M, int64_t H, int bn) {
  return colpart_at(small, M, H, bn) + (size_t)(col_slices(small, M) * H) * sizeof(uint16_t);
}
constexpr size_t TW_PARTS = 8 * SMALL_TILES > 4 * 256 ? 8 * SMALL_TILES : 4 * 256;
static_assert(TW_PARTS <= TW_MAX_BLOCKS, "the cast reduces at most that many");
// The size of a share does not fall as M or H grows, so that a workspace for
// the largest batch serves the smaller ones, although the small tiles leave up
// to four times the partials of the large ones: it is what the large tiles
// need, and at least what small tiles need for any M' <= M and H' <= H.  (They
// are at most 8 SMALL_TILES, each with 2 TM row and bn column maxima.)
size_t gate_share_bytes(int64_t M, int64_t H, bool rowwise, int bn) {
  size_t b = TW_PARTS * sizeof(uint32_t);
  if (rowwise) {
    const size_t most = 8 * SMALL_TILES * (2 * TM + bn) * sizeof(uint16_t) + 256;
    const size_t s = rowwise_share(true, M, H, bn);
    b = rowwise_share(false, M, H, bn);
    if (b < (s < most ? s : most)) b = s < most ? s : most;
  }
  return (b + 255) & ~(size_t)255;
}

// The partial maxima of output o: where the kernel writes them (g) and where
// the cast reads them (src).
void set_partials(GateArgs &g, int o, CastSource &src, void *share, bool rowwise, int bn) {
  if (rowwise) {
    const bool small = small_tiles(g.M[0], g.N[0], bn);
    g.rowpart[o] = static_cast<uint16_t *>(share);
    g.colpart[o] = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(share) +
                                                colpart_at(small, g.M[0], g.N[0], bn));
    src.rowpart = g.rowpart[o];
    src.colpart = g.colpart[o];
    src.row_slices = (int)row_slices(small, g.N[0], bn);
    src.col_slices = (int)col_slices(small, g.M[0]);
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
  size_t b = gate_share_bytes(M, H, rw, BN / 2);            // h
  const size_t d = 2 * gate_share_bytes(M, H, rw, BN);      // da and db
  if (b < d) b = d;
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
  if (M * H > 0 && K > 0 && !few_tokens(M, H)) {
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
    const hipError_t e = a ? launch_gate<EPI_GATE_AB, 0>(g, rw, &src.nparts, stream)
                           : launch_gate<EPI_GATE, 0>(g, rw, &src.nparts, stream);
    if (e != hipSuccess || !o) return e;
    return quantize_cast_launch(&src, 1, M, H, scaling, o, stream);
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
  set_partials(g, 1, sb, static_cast<uint8_t *>(workspace) + gate_share_bytes(M, H, rw, BN), rw,
               BN);
  const hipError_t e = (scaling & FP8L_E5M2)
                           ? launch_gate<EPI_DGATE, 1>(g, rw, &sa.nparts, stream)
                           : launch_gate<EPI_DGATE, 0>(g, rw, &sa.nparts, stream);
  if (e != hipSuccess) return e;
  sb.nparts = sa.nparts;
  const CastSource src[2] = {sa, sb};
  const Fp8Out out[2] = {qa, qb};
  return quantize_cast_launch(src, 2, M, H, scaling, out, stream);
}

}  // namespace fp8l
