// Reverse walk of the gated delta rule with one decay per head: the chunks of a
// sequence from the last to the first, carrying the gradient dS of the chunk's end
// state.  The mirror image of the forward walk (kda_gdr_walk.hip), with the same
// split of the work: a wave owns 16 value columns and keeps the chain in registers.
//   dY = cy (K dS) + P^T dO;   dX = Tm^T dY (the gradient of v, an output)
//   dS <- gamma_C dS + Q^T (co dO) - K^T (cx dX)
// dS0 leaves in float32, so the operands on its path carry 3 bf16 terms (dY, co dO,
// cx dX) or 2 (dS, Tm, P), as in the forward.  dS at each chunk's end is kept for
// the gradient kernel in the element type.
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

template <int DK, int WV, typename IO>
struct GdrReverseLds {
  static constexpr bool F32 = sizeof(IO) == 4;
  static constexpr int C = gdr_chunk(F32), ES = (int)sizeof(IO), VB = 16 * WV;
  static constexpr int TT = F32 ? 1 : 2;  // terms of Tm and of P
  static constexpr int K = 0;
  static constexpr int Q = K + C * DK * ES;
  static constexpr int TB = TT * gdr_frags(F32) * 1024;
  static constexpr int SC = Q + C * DK * ES;  // sc, P^T, Tm^T as in the record
  static constexpr int P = SC + kGdrScalars * C * 4;
  static constexpr int T = P + TB;
  static constexpr int DO = T + TB;
  static constexpr int BYTES = DO + C * VB * ES;
};

template <int DK, int WV, typename IO>
__global__ __launch_bounds__(64 * WV) void kda_gdr_reverse_kernel(GdrReverseParams p, int Dv) {
  using L = GdrReverseLds<DK, WV, IO>;
  using Op = GOp<IO>;
  using Frag = typename Op::Frag;
  constexpr bool F32 = L::F32;
  constexpr int C = L::C, NT = 64 * WV, VB = 16 * WV;
  constexpr int CT = DK / 16, TL = C / 16;
  constexpr int NUK = DK / Op::KU, NUC = C / Op::KU;
  constexpr int TPU = Op::TPU, TT = L::TT, ES = L::ES;
  constexpr GdrRecord R = gdr_record(F32, true);
  constexpr int NSTORE = (F32 ? 4 : 1) * (CT + TL);  // stores of a chunk
  __shared__ __attribute__((aligned(16))) char lds[2 * L::BYTES];

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g4 = lane >> 4;
  int bh, vblk;
  gdr_walk_id(Dv / VB, bh, vblk);
  const int h = bh % p.s.Hv, b = bh / p.s.Hv, hk = h / (p.s.Hv / p.s.Hk);
  const GdrSpan sp = gdr_span(p.s, b, h, C);
  const int v0 = vblk * VB + 16 * wave;
  const long HD = (long)p.s.Hv * Dv;

  const IO* kb = static_cast<const IO*>(p.k) + sp.tok0 * p.s.ks + (size_t)hk * DK;
  const IO* qb = static_cast<const IO*>(p.q) + sp.tok0 * p.s.qs + (size_t)hk * DK;
  const IO* ob = static_cast<const IO*>(p.dO) + sp.tok0 * HD + (size_t)h * Dv + vblk * VB;

  GdrCopy<NT, C, DK, IO> ck, cq;
  GdrCopy<NT, C, VB, IO> co;
  ck.init(p.s.ks);
  cq.init(p.s.qs);
  co.init(HD);
  auto copy = [&](int n, char* buf) {
    const int last = sp.Tq - n * C - 1;
    const long t0 = (long)n * C;
    const char* rec = p.rec + (sp.rec0 + n * sp.rstride) * R.bytes;
    const IO* pk = kb + t0 * p.s.ks;
    const IO* pq = qb + t0 * p.s.qs;
    const IO* po = ob + t0 * HD;
    if (last >= C - 1) {
      ck.whole(buf + L::K, pk, wave);
      cq.whole(buf + L::Q, pq, wave);
      co.whole(buf + L::DO, po, wave);
    } else {
      ck.part(buf + L::K, pk, p.s.ks, last, wave);
      cq.part(buf + L::Q, pq, p.s.qs, last, wave);
      co.part(buf + L::DO, po, HD, last, wave);
    }
    static_assert(R.p == R.sc + kGdrScalars * C * 4 && R.tt == R.p + L::TB, "one run of the record");
    gdr_copy_flat<NT, kGdrScalars * C * 4 + 2 * L::TB>(buf + L::SC, rec + R.sc, wave);
  };

  f32x4 dS[CT];
  const size_t sbase = (size_t)bh * DK * Dv + v0 + r;
#pragma unroll
  for (int t = 0; t < CT; ++t) dS[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (p.dS_T != nullptr) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) dS[t][e] = p.dS_T[sbase + (size_t)(Op::row4(t, g4) + e) * Dv];
  }

  if (sp.nch > 0) copy(sp.nch - 1, lds);
  __builtin_amdgcn_s_waitcnt(0);  // the first chunk's copies have no stores behind them
#pragma unroll 1
  for (int n = sp.nch - 1, ib = 0; n >= 0; --n, ib ^= 1) {
    char* buf = lds + ib * L::BYTES;
    // as in the forward walk: the copies of chunk n have landed, the stores of
    // chunk n + 1 may be in flight
    wait_vmcnt<NSTORE>();
    lds_barrier();

    const IO* iK = reinterpret_cast<const IO*>(buf + L::K);
    const IO* iQ = reinterpret_cast<const IO*>(buf + L::Q);
    const IO* iT = reinterpret_cast<const IO*>(buf + L::T);
    const IO* iP = reinterpret_cast<const IO*>(buf + L::P);
    const IO* iO = reinterpret_cast<const IO*>(buf + L::DO);
    const float* sc = reinterpret_cast<const float*>(buf + L::SC);

    // reads one group of products ahead, as in the forward walk
    constexpr int HT = TL / 2;
    auto rows = [&](Frag (&f)[HT][NUK], int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int u = 0; u < NUK; ++u) f[t][u] = g_row<IO, DK>(iK, Op::perm(t0 + t, r), u, g4);
    };
    f32x4 dO[TL];  // in the accumulators' layout (one term holds a bf16 dO exactly)
    Frag ka[HT][NUK], kc[HT][NUK];
    rows(ka, 0);
#pragma unroll
    for (int t = 0; t < TL; ++t) dO[t] = g_acc<VB>(iO, t, 16 * wave, r, g4);  // before the copies are issued
    __builtin_amdgcn_sched_barrier(0);
    if (n > 0) copy(n - 1, lds + (ib ^ 1) * L::BYTES);
    __builtin_amdgcn_sched_barrier(0);  // the stores counted above come after the copies
    {
      const BufRes to = make_buf(static_cast<IO*>(p.ckpt) + (sp.rec0 + n * sp.rstride) * (size_t)DK * Dv,
                                 (unsigned)(DK * Dv * ES));
#pragma unroll
      for (int t = 0; t < CT; ++t)
        store_tile(to, Op::row4(t, g4), 16 * ES, v0 * DK * ES, dS[t], r, IO{});
    }
    // ---- dY = cy (K dS) + P^T dO
    Terms<IO, 2> s2[NUK];
#pragma unroll
    for (int u = 0; u < NUK; ++u) s2[u].set(&dS[TPU * u]);
    Terms<IO, 1> o1[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) o1[u].set(&dO[TPU * u]);
    f32x4 dY[TL];
    auto k_s = [&](const Frag (&f)[HT][NUK], int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t) dY[t0 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NUK; ++u)
#pragma unroll
        for (int i = 0; i < s2[u].N; ++i)
#pragma unroll
          for (int t = 0; t < HT; ++t) gmma(dY[t0 + t], f[t][u], s2[u].t[i]);
#pragma unroll
      for (int t = t0; t < t0 + HT; ++t) {
        const f32x4 cy = *reinterpret_cast<const f32x4*>(sc + C + Op::row4(t, g4));
#pragma unroll
        for (int e = 0; e < 4; ++e) dY[t][e] *= cy[e];
      }
    };
    // the upper triangles of units of P^T and Tm^T
    constexpr int NF = gdr_frags(F32);
    Frag fT[NF][TT], fP[NF][TT];
    auto tri = [&](Frag (&f)[NF][TT], const IO* list) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int k = 0; k < TT; ++k) f[i][k] = g_frag(list, i * TT + k, lane);
    };
    rows(kc, HT);
    if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
    k_s(ka, 0);
    tri(fP, iP);
    if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
    k_s(kc, HT);
    tri(fT, iT);
    if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < NUC; ++u)
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int t = 0; t < TPU * (u + 1); ++t) gmma(dY[t], fP[tri_at<TPU, NUC, true>(t, u)][k], o1[u].t[0]);
    // ---- dX = Tm^T dY
    Terms<IO, 3> y3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) y3[u].set(&dY[TPU * u]);
    f32x4 dX[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) dX[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NUC; ++u)
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int j = 0; j < y3[u].N; ++j)
          if (k + j < y3[u].N)  // the products below the third term are left out
#pragma unroll
            for (int t = 0; t < TPU * (u + 1); ++t) gmma(dX[t], fT[tri_at<TPU, NUC, true>(t, u)][k], y3[u].t[j]);
    // ---- dS = gamma_C dS + Q^T (co dO) - K^T (cx dX); the first while dX forms
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const f32x4 co = *reinterpret_cast<const f32x4*>(sc + 2 * C + Op::row4(t, g4));
#pragma unroll
      for (int e = 0; e < 4; ++e) dO[t][e] *= co[e];
    }
    Terms<IO, 3> o3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) o3[u].set(&dO[TPU * u]);
    const float lamC = exp2_fast(sc[5 * C + C - 1] + sc[6 * C + C - 1]);
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) dS[t][e] *= lamC;
    auto add_t = [&](const IO* img, const Terms<IO, 3> (&x)[NUC]) {
#pragma unroll
      for (int jj = 0; jj < CT / 2; ++jj) {
        Frag f0[NUC], f1[NUC];
        g_colp_pair<DK>(img, jj, r, g4, f0, f1);
#pragma unroll
        for (int u = 0; u < NUC; ++u)
#pragma unroll
          for (int k = 0; k < x[u].N; ++k) {
            gmma(dS[2 * jj], f0[u], x[u].t[k]);
            gmma(dS[2 * jj + 1], f1[u], x[u].t[k]);
          }
      }
    };
    add_t(iQ, o3);
    {
      // rows behind the sequence's end lie behind the buffer
      const int left = sp.Tq - n * C < C ? sp.Tq - n * C : C;
      const BufRes to = make_buf(static_cast<IO*>(p.dv) + (size_t)(sp.tok0 + n * C) * HD,
                                 (unsigned)(left * (int)HD * ES));
#pragma unroll
      for (int t = 0; t < TL; ++t)
        store_tile(to, Op::row4(t, g4), (int)HD * ES, (h * Dv + v0) * ES, dX[t], r, IO{});
    }
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const f32x4 cx = *reinterpret_cast<const f32x4*>(sc + Op::row4(t, g4));
#pragma unroll
      for (int e = 0; e < 4; ++e) dX[t][e] *= -cx[e];
    }
    Terms<IO, 3> x3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) x3[u].set(&dX[TPU * u]);
    add_t(iK, x3);
  }
  if (p.dS0 != nullptr) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) p.dS0[sbase + (size_t)(Op::row4(t, g4) + e) * Dv] = dS[t][e];
  }
}

template <int DK, typename IO>
static hipError_t launch_reverse_w(const GdrReverseParams& p, int Dv, hipStream_t st) {
  const int wv = gdr_walk_waves(Dv, sizeof(IO) == 4);
  const unsigned grid = (unsigned)((size_t)p.s.NS * p.s.Hv * (Dv / (16 * wv)));
  if constexpr (sizeof(IO) == 2)
    if (wv == 8) {
      hipLaunchKernelGGL((kda_gdr_reverse_kernel<DK, 8, IO>), dim3(grid), dim3(512), 0, st, p, Dv);
      return hipGetLastError();
    }
  if (wv == 4)
    hipLaunchKernelGGL((kda_gdr_reverse_kernel<DK, 4, IO>), dim3(grid), dim3(256), 0, st, p, Dv);
  else
    hipLaunchKernelGGL((kda_gdr_reverse_kernel<DK, 2, IO>), dim3(grid), dim3(128), 0, st, p, Dv);
  return hipGetLastError();
}

hipError_t launch_gdr_reverse(const GdrReverseParams& p, int Dk, int Dv, bool fp32, hipStream_t st) {
  switch (Dk) {
    case 32: return fp32 ? launch_reverse_w<32, float>(p, Dv, st) : launch_reverse_w<32, __bf16>(p, Dv, st);
    case 64: return fp32 ? launch_reverse_w<64, float>(p, Dv, st) : launch_reverse_w<64, __bf16>(p, Dv, st);
    case 128: return fp32 ? launch_reverse_w<128, float>(p, Dv, st) : launch_reverse_w<128, __bf16>(p, Dv, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
