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
  static constexpr int TB = TT * gdr_frags(F32) * 1024, PB = gdr_frags(F32) * 1024;
  static constexpr int SC = T + TB;
  static constexpr int Q = SC + kGdrScalars * C * 4;
  static constexpr int P = Q + (OUT ? C * DK * ES : 0);
  static constexpr int BYTES = P + (OUT ? PB : 0);
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
  constexpr int TPU = Op::TPU, TT = L::TT, ES = L::ES;
  constexpr GdrRecord R = gdr_record(F32, CK);
  // stores of a chunk: o, 4 columns each; or the state and Y
  constexpr int NSTORE = OUT ? TL : (F32 ? 4 : 1) * (CT + TL);
  static_assert(OUT != CK, "the stores are counted for one or the other");
  __shared__ __attribute__((aligned(16))) char lds[2 * L::BYTES];

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g4 = lane >> 4;
  int bh, vblk;
  gdr_walk_id(Dv / VB, bh, vblk);
  const int h = bh % p.s.Hv, b = bh / p.s.Hv, hk = h / (p.s.Hv / p.s.Hk);
  const GdrSpan sp = gdr_span(p.s, b, h, C);
  const int v0 = vblk * VB + 16 * wave;  // this wave's value columns
  const long HD = (long)p.s.Hv * Dv;

  const IO* kb = static_cast<const IO*>(p.k) + sp.tok0 * p.s.ks + (size_t)hk * DK;
  const IO* qb = static_cast<const IO*>(p.q) + sp.tok0 * p.s.qs + (size_t)hk * DK;
  const IO* vb = static_cast<const IO*>(p.v) + sp.tok0 * p.s.vs + (size_t)h * Dv + vblk * VB;

  GdrCopy<NT, C, DK, IO> ck, cq;
  GdrCopy<NT, C, VB, IO> cv;
  ck.init(p.s.ks);
  cv.init(p.s.vs);
  if constexpr (OUT) cq.init(p.s.qs);
  auto copy = [&](int n, char* buf) {
    const int last = sp.Tq - n * C - 1;  // >= 0: the chunk exists
    const long t0 = (long)n * C;
    const char* rec = p.rec + (sp.rec0 + n * sp.rstride) * R.bytes;
    const IO* pk = kb + t0 * p.s.ks;
    const IO* pq = qb + t0 * p.s.qs;
    const IO* pv = vb + t0 * p.s.vs;
    if (last >= C - 1) {
      ck.whole(buf + L::K, pk, wave);
      cv.whole(buf + L::V, pv, wave);
      if constexpr (OUT) cq.whole(buf + L::Q, pq, wave);
    } else {
      ck.part(buf + L::K, pk, p.s.ks, last, wave);
      cv.part(buf + L::V, pv, p.s.vs, last, wave);
      if constexpr (OUT) cq.part(buf + L::Q, pq, p.s.qs, last, wave);
    }
    // Tm and the scalars follow one another in the record and in LDS
    gdr_copy_flat<NT, L::TB + kGdrScalars * C * 4>(buf + L::T, rec + R.t, wave);
    if constexpr (OUT) gdr_copy_flat<NT, L::PB>(buf + L::P, rec + R.p, wave);
  };

  // ---- initial state
  f32x4 S[CT];
  const size_t sbase = (size_t)bh * DK * Dv + v0 + r;
#pragma unroll
  for (int t = 0; t < CT; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (p.S0 != nullptr) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = p.S0[sbase + (size_t)(Op::row4(t, g4) + e) * Dv];
  }

  if (sp.nch > 0) copy(0, lds);
  __builtin_amdgcn_s_waitcnt(0);  // the first chunk's copies have no stores behind them
#pragma unroll 1
  for (int n = 0; n < sp.nch; ++n) {
    char* buf = lds + (n & 1) * L::BYTES;
    // this wave's copies of chunk n have landed (the only vector memory operations
    // it issued after them are the stores of chunk n - 1: they may stay in flight); after the barrier everybody's have, and everybody is done with
    // the other buffer
    wait_vmcnt<NSTORE>();
    lds_barrier();

    // bytes of the chunk's rows of o, Y: what lies behind belongs to others
    const unsigned chunk_bytes = (unsigned)((sp.Tq - n * C < C ? sp.Tq - n * C : C) * (int)HD * ES);
    const IO* iK = reinterpret_cast<const IO*>(buf + L::K);
    const IO* iV = reinterpret_cast<const IO*>(buf + L::V);
    const IO* iT = reinterpret_cast<const IO*>(buf + L::T);
    const IO* iQ = reinterpret_cast<const IO*>(buf + L::Q);
    const IO* iP = reinterpret_cast<const IO*>(buf + L::P);
    const float* sc = reinterpret_cast<const float*>(buf + L::SC);

    // The reads of each product are issued one group of products ahead; the fences
    // keep the compiler from pulling a read and its use together, where every use
    // would wait out the whole LDS latency.
    constexpr int HT = TL / 2;  // token tiles of a group
    auto rows = [&](Frag (&f)[HT][NUK], const IO* img, int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int u = 0; u < NUK; ++u) f[t][u] = g_row<IO, DK>(img, Op::perm(t0 + t, r), u, g4);
    };
    f32x4 V[TL];
    Frag ka[HT][NUK], kc[HT][NUK];
    rows(ka, iK, 0);
#pragma unroll
    for (int t = 0; t < TL; ++t) V[t] = g_acc<VB>(iV, t, 16 * wave, r, g4);  // before the copies are issued
    __builtin_amdgcn_sched_barrier(0);
    if (n + 1 < sp.nch) copy(n + 1, lds + ((n + 1) & 1) * L::BYTES);
    __builtin_amdgcn_sched_barrier(0);  // the stores counted above come after the copies

    if constexpr (CK) {
      // the state at the chunk's start, for the gradients
      const BufRes to = make_buf(static_cast<IO*>(p.ckpt) + (sp.rec0 + n * sp.rstride) * (size_t)DK * Dv,
                                 (unsigned)(DK * Dv * ES));
#pragma unroll
      for (int t = 0; t < CT; ++t)
        store_tile(to, Op::row4(t, g4), 16 * ES, v0 * DK * ES, S[t], r, IO{});
    }

    // ---- X = V - cx (K S);  O^T = co (S^T Q^T)
    Terms<IO, 2> s2[NUK];
#pragma unroll
    for (int u = 0; u < NUK; ++u) s2[u].set(&S[TPU * u]);
    f32x4 X[TL], O[TL];
    auto k_s = [&](const Frag (&f)[HT][NUK], int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t) X[t0 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NUK; ++u)
#pragma unroll
        for (int i = 0; i < s2[u].N; ++i)
#pragma unroll
          for (int t = 0; t < HT; ++t) gmma(X[t0 + t], f[t][u], s2[u].t[i]);
    };
    auto s_q = [&](const Frag (&f)[HT][NUK], int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t) O[t0 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NUK; ++u)
#pragma unroll
        for (int i = 0; i < s2[u].N; ++i)
#pragma unroll
          for (int t = 0; t < HT; ++t) gmma(O[t0 + t], s2[u].t[i], f[t][u]);
#pragma unroll
      for (int t = 0; t < HT; ++t) {
        const float co = sc[2 * C + Op::perm(t0 + t, r)];
#pragma unroll
        for (int e = 0; e < 4; ++e) O[t0 + t][e] *= co;
      }
    };
    auto x_of = [&](int t0) {
#pragma unroll
      for (int t = t0; t < t0 + HT; ++t) {
        const f32x4 cx = *reinterpret_cast<const f32x4*>(sc + Op::row4(t, g4));
#pragma unroll
        for (int e = 0; e < 4; ++e) X[t][e] = fmaf(-cx[e], X[t][e], V[t][e]);
      }
    };
    // the lower triangle of units of Tm (and P) by token tile
    constexpr int NF = gdr_frags(F32);  // (tile, unit) pairs
    Frag fT[NF][TT], fP[NF];
    auto tri = [&]() {
#pragma unroll
      for (int i = 0; i < NF; ++i) {
#pragma unroll
        for (int k = 0; k < TT; ++k) fT[i][k] = g_frag(iT, i * TT + k, lane);
        if constexpr (OUT) fP[i] = g_frag(iP, i, lane);
      }
    };
    Terms<IO, 3> x3[NUC];
    rows(kc, iK, HT);
    if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
    k_s(ka, 0);
    if constexpr (OUT) rows(ka, iQ, 0);
    if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
    k_s(kc, HT);
    if constexpr (OUT) {
      rows(kc, iQ, HT);
      if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
      x_of(0);
      s_q(ka, 0);
      tri();
      if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
      x_of(HT);
#pragma unroll
      for (int u = 0; u < NUC; ++u) x3[u].set(&X[TPU * u]);
      s_q(kc, HT);
    } else {
      tri();
      if constexpr (WV <= 4) __builtin_amdgcn_sched_barrier(0);
      x_of(0);
      x_of(HT);
#pragma unroll
      for (int u = 0; u < NUC; ++u) x3[u].set(&X[TPU * u]);
    }
    // ---- Y = Tm X, term by term over all the tiles, so that consecutive products
    // go to different accumulators
    f32x4 Y[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) Y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NUC; ++u)
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int j = 0; j < x3[u].N; ++j)
          if (k + j < x3[u].N)  // the products below the third term are left out
#pragma unroll
            for (int t = TPU * u; t < TL; ++t) gmma(Y[t], fT[tri_at<TPU, NUC, false>(t, u)][k], x3[u].t[j]);
    if constexpr (CK) {
      const BufRes to = make_buf(static_cast<IO*>(p.y) + (size_t)(sp.tok0 + n * C) * HD, chunk_bytes);
#pragma unroll
      for (int t = 0; t < TL; ++t)
        store_tile(to, Op::row4(t, g4), (int)HD * ES, (h * Dv + v0) * ES, Y[t], r, IO{});
    }
    // ---- O^T += Y^T P^T
    if constexpr (OUT) {
      const BufRes ob = make_buf(static_cast<IO*>(p.o) + (size_t)(sp.tok0 + n * C) * HD, chunk_bytes);
      Terms<IO, 2> y2[NUC];
#pragma unroll
      for (int u = 0; u < NUC; ++u) y2[u].set(&Y[TPU * u]);
#pragma unroll
      for (int u = 0; u < NUC; ++u)
#pragma unroll
        for (int k = 0; k < y2[u].N; ++k)
#pragma unroll
          for (int t = TPU * u; t < TL; ++t) gmma(O[t], y2[u].t[k], fP[tri_at<TPU, NUC, false>(t, u)]);
#pragma unroll
      for (int t = 0; t < TL; ++t)
        store_four(ob, Op::perm(t, r) * (int)HD * ES + (h * Dv + v0 + 4 * g4) * ES, O[t], IO{});
    }
    // ---- S = gamma_C S + K^T (cy Y)
    const float lamC = exp2_fast(sc[5 * C + C - 1] + sc[6 * C + C - 1]);
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
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] *= lamC;
#pragma unroll
    for (int jj = 0; jj < CT / 2; ++jj) {
      Frag f0[NUC], f1[NUC];
      g_colp_pair<DK>(iK, jj, r, g4, f0, f1);
#pragma unroll
      for (int u = 0; u < NUC; ++u)
#pragma unroll
        for (int k = 0; k < y3[u].N; ++k) {
          gmma(S[2 * jj], f0[u], y3[u].t[k]);
          gmma(S[2 * jj + 1], f1[u], y3[u].t[k]);
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
    case 8:
      if constexpr (sizeof(IO) == 2) return launch_walk_t<DK, 8, IO>(p, Dv, st);
      break;
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
  const int wv = gdr_walk_waves(Dv, fp32);
  return fp32 ? launch_walk_d<float>(p, Dk, Dv, wv, st) : launch_walk_d<__bf16>(p, Dk, Dv, wv, st);
}

}  // namespace kda
