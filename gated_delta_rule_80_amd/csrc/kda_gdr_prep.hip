// Chunk preparation of the gated delta rule with one decay per head: one
// workgroup of 4 waves per (chunk, value head) computes the chunk's
// Tm = (I + a)^-1 and P and its per-token scalars (kda_gdr.h) into a record.
//
// a and P are one matrix-core pass over the raw q and k rows (bf16 products are
// exact in the float32 accumulators; norms and gates are row and column factors).
// The cumulative log-decay is summed in float64 and kept as two floats, so the
// difference of two far cumulative sums keeps float32 precision for neighbours.
// Tm comes from the 16 x 16 diagonal blocks by substitution, one wave each, and
// from the blocks below them by T_ij = -T_ii sum_k A_ik T_kj, diagonal by
// diagonal, in float32 throughout.
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

template <int DK, typename IO, int PT>
__global__ __launch_bounds__(256) void kda_gdr_prep_kernel(GdrPrepParams p) {
  constexpr bool F32 = sizeof(IO) == 4;
  constexpr int C = gdr_chunk(F32);
  constexpr int NTL = C / 16;                // tiles per side
  constexpr GdrRecord RF = gdr_record(F32, PT == 2);
  using I = GImg<IO, DK>;
  constexpr int RC = I::RC, EPC = I::EPC, NU = DK / GOp<IO>::KU;
  constexpr int LA = C + 4;                  // row stride of the float32 matrices
  constexpr int IMG = C * DK * (int)sizeof(IO);
  constexpr int MAT = C * LA * 4;
  // Tm overwrites the k and q images once the products are done
  constexpr int BYTES = (2 * IMG > MAT ? 2 * IMG : MAT);
  __shared__ __attribute__((aligned(16))) char lds[BYTES];
  __shared__ __attribute__((aligned(16))) float As[C * LA];
  __shared__ float sc[kGdrScalars][C];
  IO* ik = reinterpret_cast<IO*>(lds);
  IO* iq = reinterpret_cast<IO*>(lds + IMG);
  float* Ts = reinterpret_cast<float*>(lds);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g4 = lane >> 4;
  const int pos = xcd_major(blockIdx.x, gridDim.x);
  const int h = pos % p.s.Hv, row = pos / p.s.Hv;
  const int b = row % p.s.B, slot = row / p.s.B;
  const int hk = h / (p.s.Hv / p.s.Hk);
  const GdrChunk ch = gdr_chunk_at(p.s, slot, b, h, C);
  if (ch.n == 0) return;  // uniform: a slot no sequence owns

  // ---- rows of q and k into LDS, their squared norms on the way
  for (int idx = tid; idx < 2 * C * RC; idx += 256) {
    const bool isq = idx >= C * RC;
    const int i = isq ? idx - C * RC : idx;
    const int t = i / RC, c = i % RC;
    const IO* src = isq ? static_cast<const IO*>(p.q) + (ch.tok + t) * p.s.qs
                        : static_cast<const IO*>(p.k) + (ch.tok + t) * p.s.ks;
    f32x4 raw = {0.f, 0.f, 0.f, 0.f};
    if (t < ch.n) raw = *reinterpret_cast<const f32x4*>(src + (size_t)hk * DK + c * EPC);
    *reinterpret_cast<f32x4*>((isq ? iq : ik) + (t * RC + GOp<IO>::template swz<RC>(t, c)) * EPC) = raw;
    const IO* x = reinterpret_cast<const IO*>(&raw);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < EPC; ++e) ss = fmaf(to_f32(x[e]), to_f32(x[e]), ss);
    ss = group_sum<RC>(ss);
    if (c == 0) sc[isq ? 4 : 3][t] = t < ch.n ? (p.l2 ? 1.0f / sqrtf(ss + p.eps) : 1.0f) : 0.f;
  }
  // ---- gates: wave 0, a lane per token
  if (wave == 0) {
    float gt = 0.f, bt = 0.f;
    if (lane < ch.n && lane < C) {
      const size_t at = (size_t)(ch.tok + lane) * p.s.Hv + h;
      gt = gdr_decay<IO>(p.g, at, p.A_log, p.dt_bias, h);
      bt = gdr_beta<IO>(p.beta, at, p.beta_logits);
    }
    double G = gt;
#pragma unroll
    for (int m = 1; m < C; m <<= 1) {
      const double y = __shfl_up(G, m, 64);
      if (lane >= m) G += y;
    }
    if (lane < C) {
      sc[5][lane] = (float)G;
      sc[6][lane] = (float)(G - (double)(float)G);
      sc[7][lane] = bt;
    }
  }
  __syncthreads();
  if (tid < C) {
    const float rk = sc[3][tid], sq = sc[4][tid] * p.scale;
    const float gam = expf(sc[5][tid] + sc[6][tid]);
    const float lam = expf((sc[5][C - 1] - sc[5][tid]) + (sc[6][C - 1] - sc[6][tid]));
    sc[0][tid] = gam * rk;
    sc[1][tid] = sc[7][tid] * lam * rk;
    sc[2][tid] = gam * sq;
  }
  __syncthreads();

  char* rec = p.rec + ch.rec * RF.bytes;
  IO* recP = reinterpret_cast<IO*>(rec + RF.p);
  // ---- a and P, tile by tile of the lower triangle
#pragma unroll 1
  for (int it = wave; it < NTL * NTL; it += 4) {
    const int ti = it / NTL, tj = it % NTL;
    if (tj > ti) {
      // the upper half of a diagonal 32 x 32 block is read as part of its rows
      if ((ti >> 1) == (tj >> 1))
#pragma unroll
        for (int n = 0; n < PT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            recP[(size_t)n * C * C + (16 * ti + 4 * g4 + e) * C + 16 * tj + r] = from_f32<IO>(0.f);
      continue;
    }
    f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const auto fb = g_row<IO, DK>(ik, 16 * tj + r, u, g4);
      gmma(kk, g_row<IO, DK>(ik, 16 * ti + r, u, g4), fb);
      gmma(qk, g_row<IO, DK>(iq, 16 * ti + r, u, g4), fb);
    }
    const int j = 16 * tj + r;
    const float ghj = sc[5][j], glj = sc[6][j], bj = sc[7][j] * sc[3][j];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * ti + 4 * g4 + e;
      float d = (sc[5][i] - ghj) + (sc[6][i] - glj);
      d = i >= j ? expf(d) * bj : 0.f;
      As[i * LA + j] = i > j ? d * sc[3][i] * kk[e] : 0.f;
      float pv = i >= j ? d * (sc[4][i] * p.scale) * qk[e] : 0.f;
#pragma unroll
      for (int n = 0; n < PT; ++n) {
        const IO hi = from_f32<IO>(pv);
        recP[(size_t)n * C * C + i * C + j] = hi;
        pv -= to_f32(hi);
      }
    }
  }
  __syncthreads();

  // ---- Tm: diagonal blocks, lane = column (the 4 lane groups do the same)
  if (wave < NTL) {
    const float* A = As + (16 * wave) * LA + 16 * wave;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == r ? 1.f : 0.f;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
#pragma unroll
      for (int j4 = 0; j4 < i; j4 += 4) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(A + i * LA + j4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j4 + e < i) x[i] = fmaf(-a[e], x[j4 + e], x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i >> 2) == g4) Ts[(16 * wave + i) * LA + 16 * wave + r] = x[i];
  }
  __syncthreads();
  // ---- and the blocks below them
#pragma unroll 1
  for (int d = 1; d < NTL; ++d) {
    const int i = d + wave, j = wave;
    if (i < NTL) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int k = j; k < i; ++k) {
        const f32x4 fa = *reinterpret_cast<const f32x4*>(As + (16 * i + r) * LA + 16 * k + 4 * g4);
        f32x4 fb;
#pragma unroll
        for (int e = 0; e < 4; ++e) fb[e] = Ts[(16 * k + 4 * g4 + e) * LA + 16 * j + r];
        gmma(acc, fa, fb);
      }
      const f32x4 fi = *reinterpret_cast<const f32x4*>(Ts + (16 * i + r) * LA + 16 * i + 4 * g4);
      f32x4 t = {0.f, 0.f, 0.f, 0.f};
      gmma(t, fi, acc);
#pragma unroll
      for (int e = 0; e < 4; ++e) Ts[(16 * i + 4 * g4 + e) * LA + 16 * j + r] = -t[e];
    }
    __syncthreads();
  }
  // ---- Tm and the scalars to the record
  IO* recT = reinterpret_cast<IO*>(rec + RF.t);
  for (int idx = tid; idx < C * C / EPC; idx += 256) {
    const int i = idx / (C / EPC), j = idx % (C / EPC) * EPC;
    float x[EPC];
#pragma unroll
    for (int e = 0; e < EPC; ++e) x[e] = (j >> 4) <= (i >> 4) ? Ts[i * LA + j + e] : 0.f;
    if constexpr (F32) {
      *reinterpret_cast<f32x4*>(recT + i * C + j) = f32x4{x[0], x[1], x[2], x[3]};
    } else {
      bf16x8 hi, lo;
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        hi[e] = (__bf16)x[e];
        lo[e] = (__bf16)(x[e] - (float)hi[e]);
      }
      *reinterpret_cast<bf16x8*>(recT + i * C + j) = hi;
      *reinterpret_cast<bf16x8*>(recT + C * C + i * C + j) = lo;
    }
  }
  float* recS = reinterpret_cast<float*>(rec + RF.sc);
  for (int idx = tid; idx < kGdrScalars * C; idx += 256) recS[idx] = sc[idx / C][idx % C];
}

template <typename IO>
static hipError_t launch_prep_t(const GdrPrepParams& p, int Dk, bool bwd, hipStream_t st) {
  const unsigned grid = (unsigned)((size_t)p.s.B * p.s.Hv * p.s.NT);
  if (grid == 0) return hipSuccess;
  constexpr int PB = sizeof(IO) == 4 ? 1 : 2;
#define KDA_GDR_PREP(D)                                                                          \
  if (bwd)                                                                                       \
    hipLaunchKernelGGL((kda_gdr_prep_kernel<D, IO, PB>), dim3(grid), dim3(256), 0, st, p);       \
  else                                                                                           \
    hipLaunchKernelGGL((kda_gdr_prep_kernel<D, IO, 1>), dim3(grid), dim3(256), 0, st, p);        \
  break
  switch (Dk) {
    case 32: KDA_GDR_PREP(32);
    case 64: KDA_GDR_PREP(64);
    case 128: KDA_GDR_PREP(128);
    default: return hipErrorInvalidValue;
  }
#undef KDA_GDR_PREP
  return hipGetLastError();
}

hipError_t launch_gdr_prep(const GdrPrepParams& p, int Dk, bool fp32, bool bwd, hipStream_t st) {
  return fp32 ? launch_prep_t<float>(p, Dk, bwd, st) : launch_prep_t<__bf16>(p, Dk, bwd, st);
}

}  // namespace kda
