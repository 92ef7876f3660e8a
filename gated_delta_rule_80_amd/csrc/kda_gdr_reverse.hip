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
  static constexpr int T = Q + C * DK * ES;
  static constexpr int P = T + TT * C * C * ES;
  static constexpr int DO = P + TT * C * C * ES;
  static constexpr int SC = DO + C * VB * ES;
  static constexpr int BYTES = SC + kGdrScalars * C * 4;
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
  constexpr int TPU = Op::TPU, TT = L::TT;
  constexpr GdrRecord R = gdr_record(F32, true);
  __shared__ __attribute__((aligned(16))) char lds[2 * L::BYTES];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g4 = lane >> 4;
  int bh, vblk;
  gdr_walk_id(Dv / VB, bh, vblk);
  const int h = bh % p.s.Hv, b = bh / p.s.Hv, hk = h / (p.s.Hv / p.s.Hk);
  const GdrSpan sp = gdr_span(p.s, b, h, C);
  const int v0 = vblk * VB + 16 * wave;
  const long HD = (long)p.s.Hv * Dv;

  const IO* kb = static_cast<const IO*>(p.k) + sp.tok0 * p.s.ks + (size_t)hk * DK;
  const IO* qb = static_cast<const IO*>(p.q) + sp.tok0 * p.s.qs + (size_t)hk * DK;
  const IO* ob = static_cast<const IO*>(p.dO) + sp.tok0 * HD + (size_t)h * Dv + vblk * VB;

  auto copy = [&](int n, char* buf) {
    const int last = sp.Tq - n * C - 1;
    const long t0 = (long)n * C;
    const char* rec = p.rec + (sp.rec0 + n * sp.rstride) * R.bytes;
    gdr_copy_rows<NT, C, DK, IO>(buf + L::K, kb + t0 * p.s.ks, p.s.ks, last, tid);
    gdr_copy_rows<NT, C, DK, IO>(buf + L::Q, qb + t0 * p.s.qs, p.s.qs, last, tid);
    gdr_copy_rows<NT, TT * C, C, IO>(buf + L::T, reinterpret_cast<const IO*>(rec + R.t), C, TT * C, tid);
    gdr_copy_rows<NT, TT * C, C, IO>(buf + L::P, reinterpret_cast<const IO*>(rec + R.p), C, TT * C, tid);
    gdr_copy_rows<NT, C, VB, IO>(buf + L::DO, ob + t0 * HD, HD, last, tid);
    gdr_copy_flat<NT, kGdrScalars * C * 4>(buf + L::SC, rec + R.sc, tid);
  };

  f32x4 dS[CT];
  const size_t sbase = (size_t)bh * DK * Dv + v0 + r;
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      dS[t][e] = p.dS_T != nullptr ? p.dS_T[sbase + (size_t)(Op::row4(t, g4) + e) * Dv] : 0.f;

  if (sp.nch > 0) copy(sp.nch - 1, lds);
#pragma unroll 1
  for (int n = sp.nch - 1, ib = 0; n >= 0; --n, ib ^= 1) {
    char* buf = lds + ib * L::BYTES;
    __builtin_amdgcn_s_waitcnt(0);
    lds_barrier();
    if (n > 0) copy(n - 1, lds + (ib ^ 1) * L::BYTES);

    const IO* iK = reinterpret_cast<const IO*>(buf + L::K);
    const IO* iQ = reinterpret_cast<const IO*>(buf + L::Q);
    const IO* iT = reinterpret_cast<const IO*>(buf + L::T);
    const IO* iP = reinterpret_cast<const IO*>(buf + L::P);
    const IO* iO = reinterpret_cast<const IO*>(buf + L::DO);
    const float* sc = reinterpret_cast<const float*>(buf + L::SC);

    IO* ck = static_cast<IO*>(p.ckpt) + (sp.rec0 + n * sp.rstride) * (size_t)DK * Dv +
             (size_t)(v0 / 16) * DK * 16 + r;
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) ck[(Op::row4(t, g4) + e) * 16] = from_f32<IO>(dS[t][e]);

    // ---- dO in the accumulators' layout; one term holds a bf16 dO exactly
    f32x4 dO[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) dO[t] = g_acc<VB>(iO, t, 16 * wave, r, g4);
    Terms<IO, 1> o1[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) o1[u].set(&dO[TPU * u]);
    // ---- dY = cy (K dS) + P^T dO
    Terms<IO, 2> s2[NUK];
#pragma unroll
    for (int u = 0; u < NUK; ++u) s2[u].set(&dS[TPU * u]);
    f32x4 dY[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NUK; ++u) {
        const Frag fk[1] = {g_row<IO, DK>(iK, Op::perm(t, r), u, g4)};
        gmma_terms<1>(acc, fk, s2[u]);
      }
      const f32x4 cy = *reinterpret_cast<const f32x4*>(sc + C + Op::row4(t, g4));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= cy[e];
#pragma unroll
      for (int u = t / TPU; u < NUC; ++u)
#pragma unroll
        for (int i = 0; i < TT; ++i) gmma(acc, g_colp<C>(iP + i * C * C, u, t, r, g4), o1[u].t[0]);
      dY[t] = acc;
    }
    // ---- dX = Tm^T dY
    Terms<IO, 3> y3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) y3[u].set(&dY[TPU * u]);
    f32x4 dX[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      dX[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = t / TPU; u < NUC; ++u) {
        Frag ft[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) ft[i] = g_colp<C>(iT + i * C * C, u, t, r, g4);
        gmma_terms<TT>(dX[t], ft, y3[u]);
      }
    }
#pragma unroll
    for (int t = 0; t < TL; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tt = n * C + Op::row4(t, g4) + e;
        if (tt < sp.Tq)
          static_cast<IO*>(p.dv)[(size_t)(sp.tok0 + tt) * HD + (size_t)h * Dv + v0 + r] =
              from_f32<IO>(dX[t][e]);
      }
    // ---- dS = gamma_C dS + Q^T (co dO) - K^T (cx dX)
    const float lamC = expf(sc[5 * C + C - 1] + sc[6 * C + C - 1]);
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const f32x4 cx = *reinterpret_cast<const f32x4*>(sc + Op::row4(t, g4));
      const f32x4 co = *reinterpret_cast<const f32x4*>(sc + 2 * C + Op::row4(t, g4));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dX[t][e] *= -cx[e];
        dO[t][e] *= co[e];
      }
    }
    Terms<IO, 3> x3[NUC], o3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) {
      x3[u].set(&dX[TPU * u]);
      o3[u].set(&dO[TPU * u]);
    }
#pragma unroll
    for (int t = 0; t < CT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) dS[t][e] *= lamC;
#pragma unroll
      for (int u = 0; u < NUC; ++u) {
        const Frag fk[1] = {g_colp<DK>(iK, u, t, r, g4)};
        gmma_terms<1>(dS[t], fk, x3[u]);
        const Frag fq[1] = {g_colp<DK>(iQ, u, t, r, g4)};
        gmma_terms<1>(dS[t], fq, o3[u]);
      }
    }
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
  const int wv = Dv % 64 == 0 ? 4 : 2;
  const unsigned grid = (unsigned)((size_t)p.s.NS * p.s.Hv * (Dv / (16 * wv)));
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
