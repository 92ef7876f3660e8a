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
//
// What bounds it: the rows read (32 KB a chunk) and the record written (20 KB), 3.8 TB/s
// at 64k tokens of 12 heads of 128 (150-170 us), while four workgroups a CU hide the
// chain of barriers of one (three, at 140 registers a lane, took 180-200 us).  One
// workgroup for all value heads of a key head, which forms the products once, measured
// 10% slower at 2 heads a key head.
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

// sum of squares of 16 bytes of a row (pairs taken from the whole vector: each 32-bit
// element cast to a pair was compiled to use element 0 four times)
__device__ __forceinline__ float squares(const u32x4& x, __bf16) {
  const bf16x8 v = __builtin_bit_cast(bf16x8, x);
  const bf16x2 a = __builtin_shufflevector(v, v, 0, 1), b = __builtin_shufflevector(v, v, 2, 3);
  const bf16x2 c = __builtin_shufflevector(v, v, 4, 5), d = __builtin_shufflevector(v, v, 6, 7);
  float s = __builtin_amdgcn_fdot2_f32_bf16(a, a, 0.f, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(b, b, s, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(c, c, s, false);
  return __builtin_amdgcn_fdot2_f32_bf16(d, d, s, false);
}
__device__ __forceinline__ float squares(const u32x4& x, float) {
  const f32x4 y = __builtin_bit_cast(f32x4, x);
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s = fmaf(y[e], y[e], s);
  return s;
}

template <int DK, typename IO, bool BWD>
__global__ __launch_bounds__(256, 4) void kda_gdr_prep_kernel(GdrPrepParams p) {
  constexpr bool F32 = sizeof(IO) == 4;
  constexpr int C = gdr_chunk(F32);
  constexpr int NTL = C / 16;                // tiles per side
  constexpr int TPU = GOp<IO>::TPU, NUC = NTL / TPU, TT = F32 ? 1 : 2;
  constexpr GdrRecord R = gdr_record(F32, BWD);
  using I = GImg<IO, DK>;
  using Frag = typename GOp<IO>::Frag;
  constexpr int RC = I::RC, EPC = I::EPC, NU = DK / GOp<IO>::KU;
  constexpr int LA = C + 4;                  // row stride of the float32 matrices
  constexpr int IMG = C * DK * (int)sizeof(IO);
  constexpr int MAT = C * LA * 4;
  // a and Tm overwrite the k and q images once the products are in registers
  constexpr int BYTES = (IMG > MAT ? 2 * IMG : 2 * MAT);
  __shared__ __attribute__((aligned(16))) char lds[BYTES];
  __shared__ __attribute__((aligned(16))) float sc[kGdrScalars][C];
  IO* ik = reinterpret_cast<IO*>(lds);
  IO* iq = reinterpret_cast<IO*>(lds + IMG);
  float* Ts = reinterpret_cast<float*>(lds);
  float* As = Ts + C * LA;

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g4 = lane >> 4;
  const int pos = xcd_major(blockIdx.x, gridDim.x);
  const int h = pos % p.s.Hv, row = pos / p.s.Hv;
  const int b = row % p.s.B, slot = row / p.s.B;
  const int hk = h / (p.s.Hv / p.s.Hk);
  const GdrChunk ch = gdr_chunk_at(p.s, slot, b, h, C);
  if (ch.n == 0) return;  // uniform: a slot no sequence owns

  // ---- every global load first: the rows of k and q (rows behind the sequence's end
  // lie behind the buffer: zeros), the gates
  constexpr int PIECES = C * RC;             // 16-byte pieces of one image
  constexpr int NL = (PIECES + 255) / 256;
  u32x4 raw[2][NL];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int stride = (int)(x ? p.s.qs : p.s.ks) * (int)sizeof(IO);
    const IO* base = (x ? static_cast<const IO*>(p.q) : static_cast<const IO*>(p.k)) +
                     ch.tok * (x ? p.s.qs : p.s.ks) + (size_t)hk * DK;
    const BufRes buf = make_buf(base, (unsigned)((ch.n - 1) * stride + DK * (int)sizeof(IO)));
#pragma unroll
    for (int it = 0; it < NL; ++it) {
      const int i = it * 256 + tid;
      raw[x][it] = __builtin_amdgcn_raw_buffer_load_b128(buf, i / RC * stride + i % RC * 16, 0, 0);
    }
  }
  // one wave, a lane per token: the gates; the decay summed in float64, in log2 units
  if (wave == 3) {
    float gt = 0.f, bt = 0.f;
    if (lane < ch.n && lane < C) {
      const size_t at = (size_t)(ch.tok + lane) * p.s.Hv + h;
      gt = gdr_decay<IO>(p.g, at, p.A_log, p.dt_bias, h);
      bt = gdr_beta<IO>(p.beta, at, p.beta_logits);
    }
    double G = (double)gt * 1.4426950408889634;
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
  // ---- rows into LDS, their norms on the way
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int it = 0; it < NL; ++it) {
      const int i = it * 256 + tid, t = i / RC, c = i % RC;
      if (PIECES % 256 != 0 && i >= PIECES) continue;
      *reinterpret_cast<u32x4*>((x ? iq : ik) + (t * RC + GOp<IO>::template swz<RC>(t, c)) * EPC) = raw[x][it];
      const float ss = group_sum<RC>(squares(raw[x][it], IO{}));
      if (c == 0) sc[x ? 4 : 3][t] = t < ch.n ? (p.l2 ? 1.0f / sqrtf(ss + p.eps) : 1.0f) : 0.f;
    }
  __syncthreads();

  // ---- the raw products: wave w has row tile w.  Both are formed so that a lane holds
  // 4 consecutive elements of a row of what is stored: k k^T by rows, q k^T by rows
  // (forward) or by columns (backward, which reads P^T).
  f32x4 kk[NTL], qk[NTL];
  if (wave < NTL) {
    Frag fw[NU], fx[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      fw[u] = g_row<IO, DK>(ik, 16 * wave + r, u, g4);
      if constexpr (!BWD) fx[u] = g_row<IO, DK>(iq, 16 * wave + r, u, g4);
    }
#pragma unroll
    for (int t = 0; t < NTL; ++t) {
      kk[t] = qk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (t <= wave) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const Frag f = t == wave ? fw[u] : g_row<IO, DK>(ik, 16 * t + r, u, g4);
          gmma(kk[t], f, fw[u]);
          if constexpr (!BWD) gmma(qk[t], f, fx[u]);
        }
      }
      if (BWD && t >= wave) {
#pragma unroll
        for (int u = 0; u < NU; ++u) gmma(qk[t], g_row<IO, DK>(iq, 16 * t + r, u, g4), fw[u]);
      }
    }
  }

  __syncthreads();  // every read of the images is done

  char* rec = p.rec + ch.rec * R.bytes;
  IO* recP = reinterpret_cast<IO*>(rec + R.p);
  if (tid < C) {
    const float rk = sc[3][tid], sq = sc[4][tid] * p.scale;
    const float gam = exp2_fast(sc[5][tid] + sc[6][tid]);
    const float lam = exp2_fast((sc[5][C - 1] - sc[5][tid]) + (sc[6][C - 1] - sc[6][tid]));
    sc[0][tid] = gam * rk;
    sc[1][tid] = sc[7][tid] * lam * rk;
    sc[2][tid] = gam * sq;
  }
  // ---- a and P
  if (wave < NTL) {
    const int i = 16 * wave + r;
    const float gi = sc[5][i], li = sc[6][i], ri = sc[3][i], si = sc[4][i] * p.scale, bi = sc[7][i] * ri;
#pragma unroll
    for (int tj = 0; tj < NTL; ++tj) {
      if (tj > wave) {
        // the upper half of a diagonal unit is part of its rows' fragments
        if (!BWD && tj / TPU == wave / TPU)
          store4(recP + tri_slot<IO, NUC, false>(i, 16 * tj + 4 * g4, 0, 1), 0.f, 0.f, 0.f, 0.f);
        continue;
      }
      const int j = 16 * tj + 4 * g4;
      const f32x4 gj = *reinterpret_cast<const f32x4*>(&sc[5][j]), lj = *reinterpret_cast<const f32x4*>(&sc[6][j]),
                  rj = *reinterpret_cast<const f32x4*>(&sc[3][j]), bj = *reinterpret_cast<const f32x4*>(&sc[7][j]);
      f32x4 av, pv;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float d = exp2_fast((gi - gj[e]) + (li - lj[e])) * (bj[e] * rj[e]);
        av[e] = d * ri * kk[tj][e];
        pv[e] = d * si * qk[tj][e];
        if (tj == wave) {
          av[e] = i > j + e ? av[e] : 0.f;
          pv[e] = i >= j + e ? pv[e] : 0.f;
        }
      }
      *reinterpret_cast<f32x4*>(&As[i * LA + j]) = av;
      if constexpr (!BWD) store4(recP + tri_slot<IO, NUC, false>(i, j, 0, 1), pv[0], pv[1], pv[2], pv[3]);
    }
    if constexpr (BWD) {
      // P^T, rows j = 16 wave + r: lanes hold i = 16 ti + 4 g4 ..
      const int j = i;
#pragma unroll
      for (int ti = 0; ti < NTL; ++ti) {
        const int i4 = 16 * ti + 4 * g4;
        if (ti < wave) {
          if (ti / TPU == wave / TPU)
#pragma unroll
            for (int k = 0; k < TT; ++k)
              store4(recP + tri_slot<IO, NUC, true>(j, i4, k, TT), 0.f, 0.f, 0.f, 0.f);
          continue;
        }
        const f32x4 g_i = *reinterpret_cast<const f32x4*>(&sc[5][i4]), l_i = *reinterpret_cast<const f32x4*>(&sc[6][i4]),
                    s_i = *reinterpret_cast<const f32x4*>(&sc[4][i4]);
        float pv[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = exp2_fast((g_i[e] - gi) + (l_i[e] - li)) * bi;
          pv[e] = d * (s_i[e] * p.scale) * qk[ti][e];
          if (ti == wave) pv[e] = i4 + e >= j ? pv[e] : 0.f;
          lo[e] = pv[e] - to_f32(from_f32<IO>(pv[e]));
        }
        store4(recP + tri_slot<IO, NUC, true>(j, i4, 0, TT), pv[0], pv[1], pv[2], pv[3]);
        if constexpr (!F32) store4(recP + tri_slot<IO, NUC, true>(j, i4, 1, TT), lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  __syncthreads();

  // ---- Tm: diagonal blocks, lane = column (the 4 lane groups do the same)
  if (wave < NTL) {
    int at = (16 * wave) * LA + 16 * wave;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == r ? 1.f : 0.f;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      // the next rows of a are addressed after these: all 15 at once would take 120
      // registers and a workgroup's place on the CU
      if (i == 7 || i == 10 || i == 12 || i == 14) asm volatile("" : "+v"(at), "+v"(x[i - 1]));
#pragma unroll
      for (int j4 = 0; j4 < i; j4 += 4) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(As + at + i * LA + j4);
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
#pragma unroll
  for (int d = 1; d < NTL; ++d) {
    const int i = d + wave, j = wave;
    if (i < NTL) {
      const f32x4 fi = *reinterpret_cast<const f32x4*>(Ts + (16 * i + r) * LA + 16 * i + 4 * g4);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < d; ++k) {
        const f32x4 fa = *reinterpret_cast<const f32x4*>(As + (16 * i + r) * LA + 16 * (j + k) + 4 * g4);
        f32x4 fb;
#pragma unroll
        for (int e = 0; e < 4; ++e) fb[e] = Ts[(16 * (j + k) + 4 * g4 + e) * LA + 16 * j + r];
        gmma(acc, fa, fb);
      }
      f32x4 t = {0.f, 0.f, 0.f, 0.f};
      gmma(t, fi, acc);
#pragma unroll
      for (int e = 0; e < 4; ++e) Ts[(16 * i + 4 * g4 + e) * LA + 16 * j + r] = -t[e];
    }
    __syncthreads();
  }
  // ---- Tm (for the backward also Tm^T) and the scalars to the record, a fragment a
  // wave at a time
#pragma unroll
  for (int n = 0; n < (BWD ? 2 : 1); ++n) {
    IO* to = reinterpret_cast<IO*>(rec + (n ? R.tt : R.t));
    int f = 0;
#pragma unroll
    for (int t = 0; t < NTL; ++t)
#pragma unroll
      for (int u = n ? t / TPU : 0; u < (n ? NUC : t / TPU + 1); ++u, ++f) {
        if (((f + n) & 3) != wave) continue;
        const int i = GOp<IO>::perm(t, r), j = GOp<IO>::KU * u + (GOp<IO>::KU / 4) * g4;
        const bool in = n ? (j >> 4) >= (i >> 4) : (j >> 4) <= (i >> 4);
        float x[EPC];
#pragma unroll
        for (int e = 0; e < EPC; ++e) x[e] = in ? (n ? Ts[(j + e) * LA + i] : Ts[i * LA + j + e]) : 0.f;
        if constexpr (F32) {
          *reinterpret_cast<f32x4*>(to + (f * 64 + lane) * 4) = f32x4{x[0], x[1], x[2], x[3]};
        } else {
          float lo[8];
#pragma unroll
          for (int e = 0; e < EPC; ++e) lo[e] = x[e] - (float)(__bf16)x[e];
          store8(to + (2 * f * 64 + lane) * 8, x);
          store8(to + ((2 * f + 1) * 64 + lane) * 8, lo);
        }
      }
  }
  float* recS = reinterpret_cast<float*>(rec + R.sc);
  for (int idx = tid; idx < kGdrScalars * C; idx += 256) recS[idx] = sc[idx / C][idx % C];
}

template <typename IO>
static hipError_t launch_prep_t(const GdrPrepParams& p, int Dk, bool bwd, hipStream_t st) {
  const unsigned grid = (unsigned)((size_t)p.s.B * p.s.Hv * p.s.NT);
  if (grid == 0) return hipSuccess;
#define KDA_GDR_PREP(D)                                                                          \
  if (bwd)                                                                                       \
    hipLaunchKernelGGL((kda_gdr_prep_kernel<D, IO, true>), dim3(grid), dim3(256), 0, st, p);     \
  else                                                                                           \
    hipLaunchKernelGGL((kda_gdr_prep_kernel<D, IO, false>), dim3(grid), dim3(256), 0, st, p);    \
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
