// Gradients of a chunk's q, k, g, beta in the gated delta rule with one decay per
// head, from the state S at the chunk's start, the gradient dS of its end state and
// the walks' Y and dX = dv: one workgroup per (chunk, query/key head), over the value
// heads of that head in turn (their sum is the gradient of shared rows, in one order,
// without atomics).
//
// With q' = scale q^, D_ij = e^{G_i - G_j}, w_j = b_j k^_j:
//   dq'_i  = gamma_i S dO_i  + sum_{j<=i} E1_ij w_j     E1_ij =  D_ij dO_i . Y_j
//   dke_i  = -gamma_i S dX_i + sum_{j<i}  E2_ij w_j     E2_ij = -D_ij dX_i . Y_j
//   dw_j   = lambda_j dS Y_j + sum_{i>=j} E1_ij q'_i + sum_{i>j} E2_ij k^_i
//   dk^ = dke + b dw;  db_j = k^_j . dw_j
//   dG_i = q'_i . dq'_i + k^_i . dke_i - b_i k^_i . dw_i, the chunk's last G also
//          gamma_C <S, dS> + sum_j b_j k^_j . (lambda_j dS Y_j);  dg = sums from the end
// Everything is formed transposed (channel x token): a lane holds 4 consecutive
// channels of one token, so the row dots are register sums.  A wave owns 16 channels
// (and, of narrow heads, a part of the tokens): S and dS are read once, as operands,
// and the rows of Y, dO, dX through LDS.  E1, E2 are formed once a workgroup, scaled
// for their use by rows and for that by columns, and take the place of Y, dO, dX;
// dq and dk take the place of q and k and leave in whole rows.
//
// It is bound by reading: 64 tokens, 64 KB of S and dS, 80 KB of rows.  A workgroup's
// phases are chained by barriers, so its 80 KB of LDS and 128 registers are held to
// where two share a CU and one reads while the other computes.  96 heads of 128, 4096
// tokens: 310-330 us, 3.4 TB/s (with every operand read into registers by each wave that
// uses it, one workgroup a CU: 750 us).
//
// E1, E2 are kept in two bf16 terms: they enter dG once by rows and once by columns
// and mostly cancel there, so one rounding each would leave dg with a relative error
// of 7e-3 instead of 2.4e-3.  S, dS, Y, dX are read as the walks stored them (one
// bf16 each with bf16 inputs).
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

// 4 consecutive elements of a row of an image, as floats
template <typename E, int K>
__device__ __forceinline__ f32x4 g_four(const E* img, int row, int k) {
  float x[4];
  load4(img + GImg<E, K>::at(row, k), x);
  return f32x4{x[0], x[1], x[2], x[3]};
}

__device__ __forceinline__ float frag_dot(const bf16x8& a, const bf16x8& b, float s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf((float)a[e], (float)b[e], s);
  return s;
}
__device__ __forceinline__ float frag_dot(const f32x4& a, const f32x4& b, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) s = fmaf(a[e], b[e], s);
  return s;
}

// acc += A B, B in all its terms
template <typename F, typename TB>
__device__ __forceinline__ void gmma_all(f32x4& acc, const F& a, const TB& b) {
#pragma unroll
  for (int k = 0; k < TB::N; ++k) gmma(acc, a, b.t[k]);
}

// sum over the 4 lane groups (lanes of one r)
__device__ __forceinline__ float sum_groups(float x) {
  x += __shfl_xor(x, 16, 64);
  x += __shfl_xor(x, 32, 64);
  return x;
}

// Computed here, not where it is used next: moved there, its operands would be live
// instead of it.
__device__ __forceinline__ void settle(f32x4& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void settle(float& x) { asm volatile("" : "+v"(x)); }

template <int DK, int DV, typename IO> struct GradShape {
  static constexpr bool F32 = sizeof(IO) == 4;
  static constexpr int C = gdr_chunk(F32), TL = C / 16;
  static constexpr int WC = DK / 16;                     // channel tiles, one per wave
  static constexpr int WT = 8 / WC < TL ? 8 / WC : TL;   // parts of the tokens
  static constexpr int TW = TL / WT, NW = WC * WT, NT = 64 * NW;
  static constexpr int NL = gdr_frags(F32), TERMS = F32 ? 1 : 2;
  static constexpr int ROWK = C * DK * (int)sizeof(IO), ROWV = C * DV * (int)sizeof(IO);
  static constexpr int LIST = NL * TERMS * 1024;         // one of E1, E2 by rows, by columns
  static constexpr int RED = WC * 4 * C * 4 + NW * 4;
  static constexpr int mx(int a, int b) { return a > b ? a : b; }
  // q, k | dO, dX, Y, then the four lists, then the sums over the waves
  static constexpr int BODY = 2 * ROWK + mx(mx(3 * ROWV, 4 * LIST), RED);
  // the scalars' copy, where two workgroups a CU leave room for it (all shapes but
  // 128 x 128, where they are read from the record); a phase of a small call would
  // otherwise begin with a wait for memory
  static constexpr int SCB = kGdrScalars * C * 4;
  static constexpr bool SCL = BODY + 2 * SCB <= 81920;
  static constexpr int LDS = BODY + (SCL ? 2 * SCB : 0);
};

template <int DK, int DV, typename IO, bool MULTI>
__global__ __launch_bounds__((GradShape<DK, DV, IO>::NT), 4) void kda_gdr_grad_kernel(GdrGradParams p) {
  using Op = GOp<IO>;
  using Frag = typename Op::Frag;
  using GS = GradShape<DK, DV, IO>;
  constexpr int C = GS::C, TL = GS::TL, TPU = Op::TPU, WC = GS::WC, TW = GS::TW, NT = GS::NT, NL = GS::NL;
  constexpr int NUV = DV / Op::KU, NUC = C / Op::KU;
  constexpr int JW = (4 * NL + GS::NW - 1) / GS::NW;  // blocks of pairs a wave forms
  constexpr GdrRecord R = gdr_record(GS::F32, true);
  using ET = Terms<IO, 2>;
  __shared__ __attribute__((aligned(16))) char lds[GS::LDS];
  IO* const iQ = reinterpret_cast<IO*>(lds);
  IO* const iK = reinterpret_cast<IO*>(lds + GS::ROWK);
  char* const area = lds + 2 * GS::ROWK;
  const IO* const iO = reinterpret_cast<const IO*>(area);
  const IO* const iX = reinterpret_cast<const IO*>(area + GS::ROWV);
  const IO* const iY = reinterpret_cast<const IO*>(area + 2 * GS::ROWV);
  float* const red = reinterpret_cast<float*>(area);   // [WC][4][C]
  float* const redS = red + WC * 4 * C;                // [waves]

  const int tid = threadIdx.x, wave = uniform(tid >> 6);
  int lane = tid & 63, r = lane & 15, g4 = lane >> 4;
  // what a phase reads is addressed in that phase: kept from one to the next (or over
  // the heads), the addresses and scalars would fill the registers
  const float* sc = nullptr;  // [scalar][token]: in the record, or
  const float* scl = nullptr; // the copy in LDS
  int fresh = 0;
  auto sc1 = [&](int i) { return GS::SCL ? scl[i] : sc[i]; };
  auto sc4 = [&](int i) { return *reinterpret_cast<const f32x4*>(GS::SCL ? scl + i : sc + i); };
  auto afresh = [&](const float* base) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" : "+v"(lane), "+s"(fresh));
    r = lane & 15;
    g4 = lane >> 4;
    sc = base + fresh;
  };
  const int wc = wave % WC, t0 = GS::WT == 1 ? 0 : wave / WC * TW, c0 = 16 * wc;
  const int pos = xcd_major(blockIdx.x, gridDim.x);
  const int hk = pos % p.s.Hk, row = pos / p.s.Hk;
  const int b = row % p.s.B, slot = row / p.s.B;
  const int G = MULTI ? p.s.Hv / p.s.Hk : 1;
  const GdrChunk ch0 = gdr_chunk_at(p.s, slot, b, hk * G, C);
  if (ch0.n == 0) return;  // uniform
  const int n = ch0.n;
  const long HD = (long)p.s.Hv * DV;

  // ---- rows behind the end read the last one; their scalars are zero
  GdrCopy<NT, C, DK, IO>::part(lds, static_cast<const IO*>(p.q) + ch0.tok * p.s.qs + (size_t)hk * DK, p.s.qs, n - 1,
                               wave);
  GdrCopy<NT, C, DK, IO>::part(lds + GS::ROWK, static_cast<const IO*>(p.k) + ch0.tok * p.s.ks + (size_t)hk * DK,
                               p.s.ks, n - 1, wave);

  f32x4 sumq[TW], sumk[TW];
#pragma unroll
  for (int t = 0; t < TW; ++t) sumq[t] = sumk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  float totq = 0.f, totk = 0.f;  // wave 0, token `lane`: q . sumq and k . sumk

#pragma unroll 1
  for (int gi = 0; gi < G; ++gi) {
    const int h = hk * G + gi;
    const size_t rec = ch0.rec + (size_t)gi;  // records of neighbouring heads are neighbours
    const float* const scalars = reinterpret_cast<const float*>(p.rec + rec * R.bytes + R.sc);  // [scalar][token]
    afresh(scalars);
    if constexpr (GS::SCL) {  // two copies in turn: wave 0 may still read the last head's
      char* to = lds + GS::BODY + (gi & 1) * GS::SCB;
      gdr_copy_flat<NT, GS::SCB>(to, reinterpret_cast<const char*>(scalars), wave);
      scl = reinterpret_cast<const float*>(to);
    }
    const size_t vo = ch0.tok * HD + (size_t)h * DV;
    GdrCopy<NT, C, DV, IO>::part(area, static_cast<const IO*>(p.dO) + vo, HD, n - 1, wave);
    GdrCopy<NT, C, DV, IO>::part(area + GS::ROWV, static_cast<const IO*>(p.dv) + vo, HD, n - 1, wave);
    GdrCopy<NT, C, DV, IO>::part(area + 2 * GS::ROWV, static_cast<const IO*>(p.y) + vo, HD, n - 1, wave);
    const size_t ckb = rec * (size_t)DK * DV;
    auto ckrow = [&](const void* base, int u) {  // unit u of channel c0 + r
      const int v = Op::KU * u + (Op::KU / 4) * g4;
      return *reinterpret_cast<const Frag*>(static_cast<const IO*>(base) + ckb + (v >> 4) * (DK * 16) + (c0 + r) * 16 +
                                            (v & 15));
    };
    f32x4 aw[TW];
    float qd[TW], ke[TW], kw1[TW], dot = 0.f;
    {
      Frag fS[NUV], fD[NUV];
#pragma unroll
      for (int u = 0; u < NUV; ++u) fS[u] = ckrow(p.ckS, u);
      wait_vmcnt<0>();
      __syncthreads();
      // ---- S dO, S dX
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        afresh(scalars);
        if (t == TW / 2)
#pragma unroll
          for (int u = 0; u < NUV; ++u) fD[u] = ckrow(p.ckdS, u);
        const int tk = Op::perm(t0 + t, r);
        f32x4 aq = {0.f, 0.f, 0.f, 0.f}, ae = aq;
#pragma unroll
        for (int u = 0; u < NUV; ++u) {
          gmma(aq, fS[u], g_row<IO, DV>(iO, tk, u, g4));
          gmma(ae, fS[u], g_row<IO, DV>(iX, tk, u, g4));
        }
        const float gam = exp2_fast(sc1(5 * C + tk) + sc1(6 * C + tk));
        qd[t] = ke[t] = 0.f;
        if (MULTI) {  // this head's dots: those of the sums, less what the heads before left
          const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 4 * g4), q4 = g_four<IO, DK>(iQ, tk, c0 + 4 * g4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            qd[t] = fmaf(-q4[e], sumq[t][e], qd[t]);
            ke[t] = fmaf(-k4[e], sumk[t][e], ke[t]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sumq[t][e] = fmaf(gam, aq[e], sumq[t][e]);
          sumk[t][e] = fmaf(-gam, ae[e], sumk[t][e]);
        }
        settle(sumq[t]);
        settle(sumk[t]);
        if (MULTI) {
          settle(qd[t]);
          settle(ke[t]);
        }
      }
      // ---- dS Y and <S, dS>
      afresh(scalars);
      if (t0 == 0)
#pragma unroll
        for (int u = 0; u < NUV; ++u) dot = frag_dot(fS[u], fD[u], dot);
      settle(dot);
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        afresh(scalars);
        const int tk = Op::perm(t0 + t, r);
        aw[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < NUV; ++u) gmma(aw[t], fD[u], g_row<IO, DV>(iY, tk, u, g4));
        const float lam =
            exp2_fast((sc1(5 * C + C - 1) - sc1(5 * C + tk)) + (sc1(6 * C + C - 1) - sc1(6 * C + tk)));
        const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 4 * g4);
        kw1[t] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          aw[t][e] *= lam;
          kw1[t] = fmaf(k4[e], aw[t][e], kw1[t]);
        }
        settle(aw[t]);
        settle(kw1[t]);
      }
    }
    // ---- pairs: block `job` is E1 or E2 (in turn), token tile t by rows i over the unit
    // u of j <= i (the first 2 NL blocks) or by columns j over the unit of i >= j; waves
    // past the last block form it again
    ET ev[JW];
#pragma unroll
    for (int jw = 0; jw < JW; ++jw) {
      const int job = wave * JW + jw < 4 * NL ? wave * JW + jw : 4 * NL - 1;
      const bool by_row = job < 2 * NL, second = job & 1;
      afresh(scalars);
      int t = 0, u = 0;
#pragma unroll
      for (int x = 0; x < TL; ++x)
#pragma unroll
        for (int y = 0; y < NUC; ++y) {
          if (y <= x / TPU && job >> 1 == tri_at<TPU, NUC, false>(x, y)) t = x, u = y;
          if (y >= x / TPU && job >> 1 == NL + tri_at<TPU, NUC, true>(x, y)) t = x, u = y;
        }
      const int tk = Op::perm(t, r);
      const IO* od = second ? iX : iO;
      const IO *ra = by_row ? iY : od, *rb = by_row ? od : iY;
      f32x4 m[TPU];
#pragma unroll
      for (int s = 0; s < TPU; ++s) m[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NUV; ++v) {
        const Frag fb = g_row<IO, DV>(rb, tk, v, g4);
#pragma unroll
        for (int s = 0; s < TPU; ++s) gmma(m[s], g_row<IO, DV>(ra, Op::perm(TPU * u + s, r), v, g4), fb);
        if (v % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
      const float Gh = sc1(5 * C + tk), Gl = sc1(6 * C + tk);
      const float sign = by_row ? 1.f : -1.f, sg = second ? -1.f : by_row ? 1.f : p.scale;
      const int dir = by_row ? 1 : -1, least = second ? 1 : 0;
      const int f0 = (by_row || second ? 3 : 4) * C;
#pragma unroll
      for (int s = 0; s < TPU; ++s) {
        const int x4 = Op::row4(TPU * u + s, g4);
        const f32x4 hx = sc4(5 * C + x4),
                    lx = sc4(6 * C + x4);
        f32x4 fx = sc4(f0 + x4);
        if (by_row) fx *= sc4(7 * C + x4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = exp2_fast(sign * ((Gh - hx[e]) + (Gl - lx[e]))) * (fx[e] * sg);
          m[s][e] *= d;
        }
        settle(m[s]);
#pragma unroll
        for (int e = 0; e < 4; ++e) m[s][e] = dir * (tk - (x4 + e)) >= least ? m[s][e] : 0.f;
      }
      ev[jw].set(m);
    }
    __syncthreads();  // Y, dO, dX have been read
    afresh(scalars);
#pragma unroll
    for (int jw = 0; jw < JW; ++jw) {
      const int job = wave * JW + jw < 4 * NL ? wave * JW + jw : 4 * NL - 1;
      const int l = (job < 2 * NL ? 0 : 2) + (job & 1), f = (job < 2 * NL ? job : job - 2 * NL) >> 1;
#pragma unroll
      for (int k = 0; k < ET::N; ++k)
        *reinterpret_cast<Frag*>(area + l * GS::LIST + ((f * ET::N + k) * 64 + lane) * 16) = ev[jw].t[k];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NUC; ++u) {
      const Frag fk = g_col<DK>(iK, u, c0, r, g4), fq = g_col<DK>(iQ, u, c0, r, g4);
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        afresh(scalars);
        const int tt = t0 + t;
        auto list = [&](int l, int f, int k) {
          return *reinterpret_cast<const Frag*>(area + l * GS::LIST + ((f * ET::N + k) * 64 + lane) * 16);
        };
        if (u <= tt / TPU) {  // uniform
          const int f = tri_at<TPU, NUC, false>(tt, u);
#pragma unroll
          for (int k = 0; k < ET::N; ++k) {
            gmma(sumq[t], fk, list(0, f, k));
            gmma(sumk[t], fk, list(1, f, k));
          }
        }
        if (u >= tt / TPU) {
          const int f = tri_at<TPU, NUC, true>(tt, u);
#pragma unroll
          for (int k = 0; k < ET::N; ++k) {
            gmma(aw[t], fq, list(2, f, k));
            gmma(aw[t], fk, list(3, f, k));
          }
        }
      }
    }
    // ---- row dots and the sums over the heads
    afresh(scalars);
    float kw[TW];
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const int tk = Op::perm(t0 + t, r);
      const float bt = sc1(7 * C + tk);
      const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 4 * g4), q4 = g_four<IO, DK>(iQ, tk, c0 + 4 * g4);
      kw[t] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qd[t] = fmaf(q4[e], sumq[t][e], qd[t]);
        ke[t] = fmaf(k4[e], sumk[t][e], ke[t]);
        kw[t] = fmaf(k4[e], aw[t][e], kw[t]);
        sumk[t][e] = fmaf(bt, aw[t][e], sumk[t][e]);
      }
      qd[t] = sum_groups(qd[t]);
      ke[t] = sum_groups(ke[t]);
      kw[t] = sum_groups(kw[t]);
      kw1[t] = sum_groups(kw1[t]);
    }
    dot = group_sum<64>(dot);
    __syncthreads();  // the lists have been read
#pragma unroll
    for (int t = 0; t < TW; ++t)  // lane group g stores sum g
      red[(wc * 4 + g4) * C + Op::perm(t0 + t, r)] = g4 == 0 ? qd[t] : g4 == 1 ? ke[t] : g4 == 2 ? kw[t] : kw1[t];
    if (lane == 0) redS[wave] = dot;
    __syncthreads();
    float q = 0.f, e = 0.f, w = 0.f, k1 = 0.f, all = 0.f;
    if (wave == 0) {
      if (lane < n) {
#pragma unroll
        for (int x = 0; x < WC; ++x) {
          q += red[(x * 4 + 0) * C + lane];
          e += red[(x * 4 + 1) * C + lane];
          w += red[(x * 4 + 2) * C + lane];
          k1 += red[(x * 4 + 3) * C + lane];
        }
      }
#pragma unroll
      for (int x = 0; x < GS::NW; ++x) all += redS[x];
    }
    if (MULTI) __syncthreads();  // the sums have been read
    if (wave == 0) {
      const int at_sc = lane < C ? lane : C - 1;
      const float bt = sc1(7 * C + at_sc), rk = sc1(3 * C + at_sc), rq = sc1(4 * C + at_sc);
      totq += q;
      totk += fmaf(bt, w, e);
      w *= rk;
      float dG = fmaf(q, rq * p.scale, e * rk) - bt * w;
      k1 = group_sum<64>(k1 * rk * bt);
      if (lane == C - 1) dG += exp2_fast(sc1(5 * C + C - 1) + sc1(6 * C + C - 1)) * all + k1;
#pragma unroll
      for (int m = 1; m < C; m <<= 1) {
        const float y = __shfl_down(dG, m, 64);
        if (lane + m < C) dG += y;
      }
      if (lane < n) {
        const size_t at = (size_t)(ch0.tok + lane) * p.s.Hv + h;
        float dg = dG, db = w;
        if (p.A_log != nullptr) {
          p.dg32[at] = dg;
          const float z = to_f32(static_cast<const IO*>(p.g)[at]) + p.dt_bias[h];
          dg *= -expf(p.A_log[h]) / (1.0f + expf(-z));
        }
        if (p.beta_logits) db *= bt * (1.0f - bt);
        static_cast<IO*>(p.dg)[at] = from_f32<IO>(dg);
        static_cast<IO*>(p.dbeta)[at] = from_f32<IO>(db);
      }
    }
  }
  // ---- through the norms, to the raw rows: x / |x|, dx = (dy - x^ (x^ . dy)) / |x|
  // (the norms of q and k, the same in every head's record)
  if (!GS::SCL) sc = reinterpret_cast<const float*>(p.rec + ch0.rec * R.bytes + R.sc);
  __syncthreads();
  if (wave == 0 && lane < C) {
    const float rq = sc1(4 * C + lane), rk = sc1(3 * C + lane);
    red[lane] = p.l2 ? totq * rq * rq : 0.f;
    red[C + lane] = p.l2 ? totk * rk * rk : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TW; ++t) {  // over the lane's own elements of q and k
    const int tk = Op::perm(t0 + t, r);
    const float rq = p.scale * sc1(4 * C + tk), rk = sc1(3 * C + tk), qd = red[tk], kd = red[C + tk];
    const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 4 * g4), q4 = g_four<IO, DK>(iQ, tk, c0 + 4 * g4);
    float dq[4], dk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dq[e] = rq * (sumq[t][e] - q4[e] * qd);
      dk[e] = rk * (sumk[t][e] - k4[e] * kd);
    }
    store4(iQ + GImg<IO, DK>::at(tk, c0 + 4 * g4), dq[0], dq[1], dq[2], dq[3]);
    store4(iK + GImg<IO, DK>::at(tk, c0 + 4 * g4), dk[0], dk[1], dk[2], dk[3]);
  }
  __syncthreads();
  constexpr int RC = GImg<IO, DK>::RC, EPC = GImg<IO, DK>::EPC;
#pragma unroll
  for (int it = 0; it < (2 * C * RC + NT - 1) / NT; ++it) {
    const int idx = it * NT + tid, i = idx % (C * RC), t = i / RC, c = i % RC;
    if (idx < 2 * C * RC && t < n)
      *reinterpret_cast<f32x4*>(static_cast<IO*>(idx < C * RC ? p.dq : p.dk) +
                                ((size_t)(ch0.tok + t) * p.s.Hk + hk) * DK + c * EPC) =
          *reinterpret_cast<const f32x4*>((idx < C * RC ? iQ : iK) + (t * RC + Op::template swz<RC>(t, c)) * EPC);
  }
}

template <int DK, int DV, typename IO>
static hipError_t launch_grad_v(const GdrGradParams& p, hipStream_t st) {
  const dim3 grid((unsigned)((size_t)p.s.B * p.s.Hk * p.s.NT)), block(GradShape<DK, DV, IO>::NT);
  if (p.s.Hv == p.s.Hk)
    hipLaunchKernelGGL((kda_gdr_grad_kernel<DK, DV, IO, false>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((kda_gdr_grad_kernel<DK, DV, IO, true>), grid, block, 0, st, p);
  return hipGetLastError();
}

template <int DK, typename IO>
static hipError_t launch_grad_t(const GdrGradParams& p, int Dv, hipStream_t st) {
  switch (Dv) {
    case 32: return launch_grad_v<DK, 32, IO>(p, st);
    case 64: return launch_grad_v<DK, 64, IO>(p, st);
    case 128: return launch_grad_v<DK, 128, IO>(p, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_gdr_grad(const GdrGradParams& p, int Dk, int Dv, bool fp32, hipStream_t st) {
  switch (Dk) {
    case 32: return fp32 ? launch_grad_t<32, float>(p, Dv, st) : launch_grad_t<32, __bf16>(p, Dv, st);
    case 64: return fp32 ? launch_grad_t<64, float>(p, Dv, st) : launch_grad_t<64, __bf16>(p, Dv, st);
    case 128: return fp32 ? launch_grad_t<128, float>(p, Dv, st) : launch_grad_t<128, __bf16>(p, Dv, st);
  }
  return hipErrorInvalidValue;
}

// dA_log and ddt_bias of one head per workgroup, summed in float64: with the decay
// -e^A softplus(z), the derivative by A is the decay itself, by the bias
// -e^A sigmoid(z).
template <typename IO>
__global__ __launch_bounds__(256) void kda_gdr_gate_kernel(GdrGateParams p) {
  __shared__ double red[2][4];
  const int h = blockIdx.x, tid = threadIdx.x;
  long t0 = 0, t1 = p.tokens;
  if (p.seqs.bounds != nullptr) {
    t0 = p.seqs.bounds[0];
    t1 = p.seqs.bounds[p.seqs.n_seqs];
  }
  const float rate = expf(p.A_log[h]), bias = p.dt_bias[h];
  double sA = 0.0, sb = 0.0;
  for (long t = t0 + tid; t < t1; t += 256) {
    const size_t at = (size_t)t * p.Hv + h;
    const float z = to_f32(static_cast<const IO*>(p.g)[at]) + bias, d = p.dg32[at];
    sA += (double)d * (double)(-rate * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)))));
    sb += (double)d * (double)(-rate / (1.0f + expf(-z)));
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    sA += __shfl_xor(sA, m, 64);
    sb += __shfl_xor(sb, m, 64);
  }
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = sA;
    red[1][tid >> 6] = sb;
  }
  __syncthreads();
  if (tid == 0) {
    if (p.dA_log != nullptr) p.dA_log[h] = (float)(red[0][0] + red[0][1] + red[0][2] + red[0][3]);
    if (p.ddt_bias != nullptr) p.ddt_bias[h] = (float)(red[1][0] + red[1][1] + red[1][2] + red[1][3]);
  }
}

hipError_t launch_gdr_gate(const GdrGateParams& p, bool fp32, hipStream_t st) {
  if (fp32)
    hipLaunchKernelGGL((kda_gdr_gate_kernel<float>), dim3((unsigned)p.Hv), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((kda_gdr_gate_kernel<__bf16>), dim3((unsigned)p.Hv), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace kda
