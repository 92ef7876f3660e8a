// State walk of the gated delta rule with one decay per head: one workgroup of WV
// waves per (sequence, value head, block of 16 WV value columns) walks the chunks
// of its sequence in order; each wave owns 16 value columns and carries the whole
// chain K S -> X -> Y -> S' of a chunk in registers (kda_gdr_device.h), so the
// only thing the waves share is the chunk's data in LDS: k, q, v rows as the
// caller holds them and the record of the preparation.  The next chunk is copied
// into the other half of LDS (global-to-LDS loads, no registers) while this one
// computes; one barrier a chunk.
//
// Precision (bf16 inputs): S, X, Y are float32 accumulators.  As operands they are
// split into bf16 terms: S 2, X 3 and b lambda rk Y 3 where they lead to the
// state, which leaves in float32 (relative error about 5e-7 against float64);
// S 2, Y 2 and P 1 where they lead to the output, which is rounded to bf16.
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

template <int DK, int WV, typename IO, bool OUT>
struct GdrWalkLds {
  static constexpr bool F32 = sizeof(IO) == 4;
  static constexpr int C = gdr_chunk(F32), ES = (int)sizeof(IO), VB = 16 * WV;
  static constexpr int TT = F32 ? 1 : 2;
  static constexpr int K = 0;
  static constexpr int V = K + C * DK * ES;
  static constexpr int T = V + C * VB * ES;
  static constexpr int SC = T + TT * C * C * ES;
  static constexpr int Q = SC + kGdrScalars * C * 4;
  static constexpr int P = Q + (OUT ? C * DK * ES : 0);
  static constexpr int BYTES = P + (OUT ? C * C * ES : 0);
};

template <int DK, int WV, typename IO, bool OUT, bool CK>
__global__ __launch_bounds__(64 * WV) void kda_gdr_walk_kernel(GdrWalkParams p, int Dv) {
  using L = GdrWalkLds<DK, WV, IO, OUT>;
  using Op = GOp<IO>;
  using Frag = typename Op::Frag;
  constexpr bool F32 = L::F32;
  constexpr int C = L::C, NT = 64 * WV, VB = 16 * WV;
  constexpr int CT = DK / 16, TL = C / 16;             // tiles of the state and of the tokens
  constexpr int NUK = DK / Op::KU, NUC = C / Op::KU;   // contraction units
  constexpr int TPU = Op::TPU, TT = L::TT;
  constexpr GdrRecord R = gdr_record(F32, CK);
  __shared__ __attribute__((aligned(16))) char lds[2 * L::BYTES];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g4 = lane >> 4;
  int bh, vblk;
  gdr_walk_id(Dv / VB, bh, vblk);
  const int h = bh % p.s.Hv, b = bh / p.s.Hv, hk = h / (p.s.Hv / p.s.Hk);
  const GdrSpan sp = gdr_span(p.s, b, h, C);
  const int v0 = vblk * VB + 16 * wave;  // this wave's value columns
  const long HD = (long)p.s.Hv * Dv;

  const IO* kb = static_cast<const IO*>(p.k) + sp.tok0 * p.s.ks + (size_t)hk * DK;
  const IO* qb = static_cast<const IO*>(p.q) + sp.tok0 * p.s.qs + (size_t)hk * DK;
  const IO* vb = static_cast<const IO*>(p.v) + sp.tok0 * p.s.vs + (size_t)h * Dv + vblk * VB;

  auto copy = [&](int n, char* buf) {
    const int last = sp.Tq - n * C - 1;  // >= 0: the chunk exists
    const long t0 = (long)n * C;
    const char* rec = p.rec + (sp.rec0 + n * sp.rstride) * R.bytes;
    gdr_copy_rows<NT, C, DK, IO>(buf + L::K, kb + t0 * p.s.ks, p.s.ks, last, tid);
    gdr_copy_rows<NT, C, VB, IO>(buf + L::V, vb + t0 * p.s.vs, p.s.vs, last, tid);
    gdr_copy_rows<NT, TT * C, C, IO>(buf + L::T, reinterpret_cast<const IO*>(rec + R.t), C, TT * C, tid);
    gdr_copy_flat<NT, kGdrScalars * C * 4>(buf + L::SC, rec + R.sc, tid);
    if constexpr (OUT) {
      gdr_copy_rows<NT, C, DK, IO>(buf + L::Q, qb + t0 * p.s.qs, p.s.qs, last, tid);
      gdr_copy_rows<NT, C, C, IO>(buf + L::P, reinterpret_cast<const IO*>(rec + R.p), C, C, tid);
    }
  };

  // ---- initial state
  f32x4 S[CT];
  const size_t sbase = (size_t)bh * DK * Dv + v0 + r;
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[t][e] = p.S0 != nullptr ? p.S0[sbase + (size_t)(Op::row4(t, g4) + e) * Dv] : 0.f;

  if (sp.nch > 0) copy(0, lds);
#pragma unroll 1
  for (int n = 0; n < sp.nch; ++n) {
    char* buf = lds + (n & 1) * L::BYTES;
    // this wave's copies of chunk n have landed; after the barrier everybody's
    // have, and everybody is done with the other buffer
    __builtin_amdgcn_s_waitcnt(0);
    lds_barrier();
    if (n + 1 < sp.nch) copy(n + 1, lds + ((n + 1) & 1) * L::BYTES);

    const IO* iK = reinterpret_cast<const IO*>(buf + L::K);
    const IO* iV = reinterpret_cast<const IO*>(buf + L::V);
    const IO* iT = reinterpret_cast<const IO*>(buf + L::T);
    const IO* iQ = reinterpret_cast<const IO*>(buf + L::Q);
    const IO* iP = reinterpret_cast<const IO*>(buf + L::P);
    const float* sc = reinterpret_cast<const float*>(buf + L::SC);

    if constexpr (CK) {
      // the state at the chunk's start, for the gradients
      IO* ck = static_cast<IO*>(p.ckpt) + (sp.rec0 + n * sp.rstride) * (size_t)DK * Dv +
               (size_t)(v0 / 16) * DK * 16 + r;
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) ck[(Op::row4(t, g4) + e) * 16] = from_f32<IO>(S[t][e]);
    }

    // ---- X = V - cx (K S)
    Terms<IO, 2> s2[NUK];
#pragma unroll
    for (int u = 0; u < NUK; ++u) s2[u].set(&S[TPU * u]);
    f32x4 X[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NUK; ++u) {
        const Frag fk[1] = {g_row<IO, DK>(iK, Op::perm(t, r), u, g4)};
        gmma_terms<1>(acc, fk, s2[u]);
      }
      const f32x4 cx = *reinterpret_cast<const f32x4*>(sc + Op::row4(t, g4));
      const f32x4 v = g_acc<VB>(iV, t, 16 * wave, r, g4);
#pragma unroll
      for (int e = 0; e < 4; ++e) X[t][e] = fmaf(-cx[e], acc[e], v[e]);
    }
    // ---- O^T = co (S^T Q^T)
    f32x4 O[TL];
    if constexpr (OUT) {
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        O[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < NUK; ++u) {
          const Frag fq = g_row<IO, DK>(iQ, Op::perm(t, r), u, g4);
#pragma unroll
          for (int i = 0; i < s2[u].N; ++i) gmma(O[t], s2[u].t[i], fq);
        }
        const float co = sc[2 * C + Op::perm(t, r)];
#pragma unroll
        for (int e = 0; e < 4; ++e) O[t][e] *= co;
      }
    }
    // ---- Y = Tm X (lower triangle of units)
    Terms<IO, 3> x3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) x3[u].set(&X[TPU * u]);
    f32x4 Y[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      Y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u <= t / TPU; ++u) {
        Frag ft[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) ft[i] = g_row<IO, C>(iT + i * C * C, Op::perm(t, r), u, g4);
        gmma_terms<TT>(Y[t], ft, x3[u]);
      }
    }
    if constexpr (CK) {
#pragma unroll
      for (int t = 0; t < TL; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tt = n * C + Op::row4(t, g4) + e;
          if (tt < sp.Tq)
            static_cast<IO*>(p.y)[(size_t)(sp.tok0 + tt) * HD + (size_t)h * Dv + v0 + r] =
                from_f32<IO>(Y[t][e]);
        }
    }
    // ---- O^T += Y^T P^T
    if constexpr (OUT) {
      Terms<IO, 2> y2[NUC];
#pragma unroll
      for (int u = 0; u < NUC; ++u) y2[u].set(&Y[TPU * u]);
#pragma unroll
      for (int t = 0; t < TL; ++t) {
#pragma unroll
        for (int u = 0; u <= t / TPU; ++u) {
          const Frag fp = g_row<IO, C>(iP, Op::perm(t, r), u, g4);
#pragma unroll
          for (int i = 0; i < y2[u].N; ++i) gmma(O[t], y2[u].t[i], fp);
        }
        const int tt = n * C + Op::perm(t, r);
        if (tt < sp.Tq)
          store4(static_cast<IO*>(p.o) + (size_t)(sp.tok0 + tt) * HD + (size_t)h * Dv + v0 + 4 * g4,
                 O[t][0], O[t][1], O[t][2], O[t][3]);
      }
    }
    // ---- S = gamma_C S + K^T (cy Y)
    const float lamC = expf(sc[5 * C + C - 1] + sc[6 * C + C - 1]);
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const f32x4 cy = *reinterpret_cast<const f32x4*>(sc + C + Op::row4(t, g4));
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[t][e] *= cy[e];
    }
    Terms<IO, 3> y3[NUC];
#pragma unroll
    for (int u = 0; u < NUC; ++u) y3[u].set(&Y[TPU * u]);
#pragma unroll
    for (int t = 0; t < CT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] *= lamC;
#pragma unroll
      for (int u = 0; u < NUC; ++u) {
        const Frag fk[1] = {g_colp<DK>(iK, u, t, r, g4)};
        gmma_terms<1>(S[t], fk, y3[u]);
      }
    }
  }
  if (p.S_T != nullptr) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) p.S_T[sbase + (size_t)(Op::row4(t, g4) + e) * Dv] = S[t][e];
  }
}

template <int DK, int WV, typename IO>
static hipError_t launch_walk_t(const GdrWalkParams& p, int Dv, hipStream_t st) {
  const unsigned grid = (unsigned)((size_t)p.s.NS * p.s.Hv * (Dv / (16 * WV)));
  if (p.ckpt != nullptr)
    hipLaunchKernelGGL((kda_gdr_walk_kernel<DK, WV, IO, false, true>), dim3(grid), dim3(64 * WV), 0, st,
                       p, Dv);
  else
    hipLaunchKernelGGL((kda_gdr_walk_kernel<DK, WV, IO, true, false>), dim3(grid), dim3(64 * WV), 0, st,
                       p, Dv);
  return hipGetLastError();
}

template <int DK, typename IO>
static hipError_t launch_walk_w(const GdrWalkParams& p, int Dv, int wv, hipStream_t st) {
  switch (wv) {
    case 2: return launch_walk_t<DK, 2, IO>(p, Dv, st);
    case 4: return launch_walk_t<DK, 4, IO>(p, Dv, st);
  }
  return hipErrorInvalidValue;
}

template <typename IO>
static hipError_t launch_walk_d(const GdrWalkParams& p, int Dk, int Dv, int wv, hipStream_t st) {
  switch (Dk) {
    case 32: return launch_walk_w<32, IO>(p, Dv, wv, st);
    case 64: return launch_walk_w<64, IO>(p, Dv, wv, st);
    case 128: return launch_walk_w<128, IO>(p, Dv, wv, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_gdr_walk(const GdrWalkParams& p, int Dk, int Dv, bool fp32, hipStream_t st) {
  const int wv = Dv % 64 == 0 ? 4 : 2;
  return fp32 ? launch_walk_d<float>(p, Dk, Dv, wv, st) : launch_walk_d<__bf16>(p, Dk, Dv, wv, st);
}

}  // namespace kda
