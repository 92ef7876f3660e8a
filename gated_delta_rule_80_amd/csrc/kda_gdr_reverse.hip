// Reverse walk of the gated delta rule with one decay per head: the chunks of a
// sequence from the last to the first, carrying the gradient dS of the chunk's end
// state.  The mirror image of the forward walk (kda_gdr_walk.hip), with the same
// split of the work: a wave owns NV tiles of 16 value columns and keeps the chain in
// registers, the chunk cut into slots that pair products with operand splits.
//   dY = cy (K dS) + P^T dO;   dX = Tm^T dY (the gradient of v, an output)
//   dS <- gamma_C dS + Q^T (co dO) - K^T (cx dX)
// dS0 leaves in float32, so the operands on its path carry 3 bf16 terms (dY, co dO,
// cx dX) or 2 (dS, Tm, P), as in the forward.  dS at each chunk's end is kept for
// the gradient kernel in the element type.
//
// It reads nothing of the forward walk (S, Y come in with the gradient kernel only), so
// both run in one launch, the reverse ones first: where the sequences are few or unlike,
// neither fills the card.  Measured with bf16, D = 128: 160 us where one after the other
// took 254 us (packed, 1 to 1500 tokens, 32 heads), 440-480 us against 510 us (96 heads,
// 4096 tokens: each in halves of a head by itself, together in whole ones).  A reverse
// chunk of a whole head takes 7 us, 170 products a wave and the splits of four operands
// (dY, co dO, cx dX, dS); like the forward walk it is bound by issuing them.
#include "kda_gdr_walk.h"

namespace kda {

template <int DK, int WV, int NV, typename IO>
struct GdrReverseLds {
  static constexpr bool F32 = sizeof(IO) == 4;
  static constexpr int C = gdr_chunk(F32), ES = (int)sizeof(IO), VB = 16 * NV * WV;
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

// STORE: with the outputs (dv, the kept dS)
template <int DK, int WV, int NV, typename IO, bool STORE>
__device__ __forceinline__ void gdr_reverse(const GdrReverseParams& p, int Dv, int blk, char* lds) {
  using L = GdrReverseLds<DK, WV, NV, IO>;
  using Op = GOp<IO>;
  using Frag = typename Op::Frag;
  constexpr bool F32 = L::F32;
  constexpr int C = L::C, NT = 64 * WV, VB = L::VB;
  constexpr int CT = DK / 16, TL = C / 16;
  constexpr int NUK = DK / Op::KU, NUC = C / Op::KU;
  constexpr int TPU = Op::TPU, TT = L::TT, ES = L::ES;
  constexpr GdrRecord R = gdr_record(F32, true);
  constexpr int NSTORE = STORE ? NV * (F32 ? 4 : 1) * (CT + TL) : 0;  // stores of a chunk
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g4 = lane >> 4;
  int bh, vblk, seg = 0;
  if (!gdr_walk_id(blk, Dv / VB, p.s.Hv / p.s.Hk, p.walks, bh, vblk)) return;  // uniform
  if (p.nseg > 1) {
    const int walks = p.s.B * p.s.Hv;
    seg = bh / walks + p.pass;  // the first segment needs no N'
    bh %= walks;
  }
  const int h = bh % p.s.Hv, b = bh / p.s.Hv, hk = h / (p.s.Hv / p.s.Hk);
  GdrSpan sp = gdr_span(p.s, b, h, C);
  if (p.nseg > 1) {
    const int c0 = seg * p.seg_len;
    sp.tok0 += (long)c0 * C;
    sp.Tq -= c0 * C;
    sp.nch = sp.nch - c0 < p.seg_len ? sp.nch - c0 : p.seg_len;
    sp.rec0 += c0 * sp.rstride;
  }
  const int v0 = vblk * VB + 16 * NV * wave;  // this wave's value columns
  const long HD = (long)p.s.Hv * Dv;

  const IO* kb = static_cast<const IO*>(p.k) + sp.tok0 * p.s.ks + (size_t)hk * DK;
  const IO* qb = static_cast<const IO*>(p.q) + sp.tok0 * p.s.qs + (size_t)hk * DK;
  const IO* ob = static_cast<const IO*>(p.dO) + sp.tok0 * HD + (size_t)h * Dv + vblk * VB;

  GdrCopy<NT, C, DK, IO> ck, cq;
  GdrCopy<NT, C, VB, IO> co;
  ck.init(p.s.ks);
  cq.init(p.s.qs);
  co.init(HD);
  auto copy = [&](int n, char* buf, int part) {  // in parts, as in the forward walk
    const int last = sp.Tq - n * C - 1;
    const long t0 = (long)n * C;
    const char* rec = p.rec + (sp.rec0 + n * sp.rstride) * R.bytes;
    const IO* pk = kb + t0 * p.s.ks;
    const IO* pq = qb + t0 * p.s.qs;
    const IO* po = ob + t0 * HD;
    if (part == 0) {
      if (last >= C - 1) {
        ck.whole(buf + L::K, pk, wave);
        co.whole(buf + L::DO, po, wave);
      } else {
        ck.part(buf + L::K, pk, p.s.ks, last, wave);
        co.part(buf + L::DO, po, HD, last, wave);
      }
    } else if (part == 1) {
      static_assert(R.p == R.sc + kGdrScalars * C * 4 && R.tt == R.p + L::TB, "one run of the record");
      gdr_copy_flat<NT, kGdrScalars * C * 4 + 2 * L::TB>(buf + L::SC, rec + R.sc, wave);
    } else {
      if (last >= C - 1)
        cq.whole(buf + L::Q, pq, wave);
      else
        cq.part(buf + L::Q, pq, p.s.qs, last, wave);
    }
  };

  f32x4 dS[NV][CT];
  Terms<IO, 2> s2[NV][NUK];
  const size_t sbase = (size_t)bh * DK * Dv + v0 + r;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int t = 0; t < CT; ++t) dS[v][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // where this walk's gradient comes from (NULL: zeros) and goes to (NULL: nowhere)
  const float* d_in = p.dS_T != nullptr ? p.dS_T + sbase : nullptr;
  float* d_out = p.dS0 != nullptr ? p.dS0 + sbase : nullptr;
  if (p.nseg > 1) {
    float* ends = p.ends + ((size_t)bh * p.nseg + seg) * DK * Dv + v0 + r;
    if (seg < p.nseg - 1) d_in = STORE ? ends : nullptr;
    if (!STORE) d_out = ends - (size_t)DK * Dv;
    else if (seg > 0) d_out = nullptr;
  }
  if (d_in != nullptr) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) dS[v][t][e] = d_in[16 * v + (size_t)(Op::row4(t, g4) + e) * Dv];
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int u = 0; u < NUK; ++u) s2[v][u].set(&dS[v][TPU * u]);

  if (sp.nch > 0)
    for (int part = 0; part < 3; ++part) copy(sp.nch - 1, lds, part);
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

    constexpr int HT = TL / 2;
    constexpr int NF = gdr_frags(F32);
    static_assert(HT == TPU && NUC == 2, "a half is a unit");
    auto rows = [&](Frag (&f)[HT][NUK], int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int u = 0; u < NUK; ++u) f[t][u] = g_row<IO, DK>(iK, Op::perm(t0 + t, r), u, g4);
    };
    f32x4 dY[NV][TL], dX[NV][TL];
    AccRaw<IO> dO[NV][TL];  // in the accumulators' layout
    Terms<IO, 1> o1[NV][NUC];  // one term holds a bf16 dO exactly
    Terms<IO, 3> o3[NV][NUC], y3[NV][NUC], x3[NV][NUC];
    Frag fT[NF][TT], fP[NF][TT];  // the upper triangles of units of Tm^T and P^T
    auto k_s = [&](const Frag (&f)[HT][NUK], int t0) {  // dY = cy (K dS)
#pragma unroll
      for (int u = 0; u < NUK; ++u)
#pragma unroll
        for (int i = 0; i < s2[0][u].N; ++i)
#pragma unroll
          for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (u == 0 && i == 0) dY[v][t0 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
              gmma(dY[v][t0 + t], f[t][u], s2[v][u].t[i]);
            }
#pragma unroll
      for (int t = t0; t < t0 + HT; ++t) {
        const f32x4 cy = *reinterpret_cast<const f32x4*>(sc + C + Op::row4(t, g4));
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) dY[v][t][e] *= cy[e];
      }
    };
    auto p_o = [&](int t0, int u) {  // dY += P^T dO
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int t = t0; t < t0 + HT; ++t)
#pragma unroll
          for (int v = 0; v < NV; ++v) gmma(dY[v][t], fP[tri_at<TPU, NUC, true>(t, u)][k], o1[v][u].t[0]);
    };
    auto tm_y = [&](int t0, int u, bool first) {  // dX += Tm^T dY
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int j = 0; j < y3[0][u].N; ++j)
          if (k + j < y3[0][u].N)  // the products below the third term are left out
#pragma unroll
            for (int t = t0; t < t0 + HT; ++t)
#pragma unroll
              for (int v = 0; v < NV; ++v) {
                if (first && k == 0 && j == 0) dX[v][t] = f32x4{0.f, 0.f, 0.f, 0.f};
                gmma(dX[v][t], fT[tri_at<TPU, NUC, true>(t, u)][k], y3[v][u].t[j]);
              }
    };
    auto o_of = [&](int u) {  // co dO, split
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        f32x4 z[HT];
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const f32x4 co = *reinterpret_cast<const f32x4*>(sc + 2 * C + Op::row4(HT * u + t, g4));
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][e] = co[e] * dO[v][HT * u + t][e];
        }
        o3[v][u].set(z);
      }
    };
    auto y_of = [&](int u) {
#pragma unroll
      for (int v = 0; v < NV; ++v) y3[v][u].set(&dY[v][HT * u]);
    };
    auto x_of = [&](int u) {  // -cx dX, split
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        f32x4 z[HT];
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const f32x4 cx = *reinterpret_cast<const f32x4*>(sc + Op::row4(HT * u + t, g4));
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][e] = -cx[e] * dX[v][HT * u + t][e];
        }
        x3[v][u].set(z);
      }
    };
    constexpr int GT = CT < 4 ? CT : 4;  // state tiles of a group
    auto add_t = [&](const IO* img, const Terms<IO, 3> (&x)[NV][NUC], int u) {
#pragma unroll
      for (int j = 0; j < CT; j += GT) {
        Frag f[GT];
        g_colp_tiles<DK>(img, u, j, r, g4, f);
#pragma unroll
        for (int k = 0; k < x[0][u].N; ++k)
#pragma unroll
          for (int t = 0; t < GT; ++t)
#pragma unroll
            for (int v = 0; v < NV; ++v) gmma(dS[v][j + t], f[t], x[v][u].t[k]);
      }
    };

    // ---- slot 1: K dS, second half
    Frag fa[HT][NUK], fb[HT][NUK];
    rows(fa, HT);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < TL; ++t) dO[v][t].template load<VB>(iO, t, 16 * (NV * wave + v), r, g4);
    __builtin_amdgcn_sched_barrier(0);  // (transposing reads the compiler sees: before the copies)
    char* nbuf = lds + (ib ^ 1) * L::BYTES;
    if (n > 0) copy(n - 1, nbuf, 0);
    __builtin_amdgcn_sched_barrier(0);
    rows(fb, 0);
    k_s(fa, HT);
    __builtin_amdgcn_sched_barrier(0);
    if (n > 0) copy(n - 1, nbuf, 1);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 2: K dS, first half, beside the split of co dO
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int k = 0; k < TT; ++k) fP[i][k] = g_frag(iP, i * TT + k, lane);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int u = 0; u < NUC; ++u) {
        f32x4 z[HT];
#pragma unroll
        for (int t = 0; t < HT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][e] = dO[v][HT * u + t][e];
        o1[v][u].set(z);
      }
    k_s(fb, 0);
    p_o(HT, 1);
    o_of(0);
    __builtin_amdgcn_sched_barrier(0);
    if (n > 0) copy(n - 1, nbuf, 2);
    __builtin_amdgcn_sched_barrier(0);  // the stores counted above come after the copies
    if constexpr (STORE) {
      const BufRes to = make_buf(static_cast<IO*>(p.ckpt) + (sp.rec0 + n * sp.rstride) * (size_t)DK * Dv,
                                 (unsigned)(DK * Dv * ES));
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = 0; t < CT; ++t)
          store_tile(to, Op::row4(t, g4), 16 * ES, (v0 + 16 * v) * DK * ES, dS[v][t], r, IO{});
    }
    // ---- slot 3: dY whole, beside the splits of its second half and of co dO
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int k = 0; k < TT; ++k) fT[i][k] = g_frag(iT, i * TT + k, lane);
    p_o(0, 0);
    p_o(0, 1);
    const float lamC = exp2_fast(sc[5 * C + C - 1] + sc[6 * C + C - 1]);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) dS[v][t][e] *= lamC;
    y_of(1);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 4: dX, second half, and dS += Q^T (co dO), beside the splits of dY's
    // first half and of co dO's second
    tm_y(HT, 1, true);
    add_t(iQ, o3, 0);
    y_of(0);
    o_of(1);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 5: dX, first half, beside the split of cx dX's second
    tm_y(0, 1, true);
    tm_y(0, 0, false);
    add_t(iQ, o3, 1);
    x_of(1);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 6: dS -= K^T (cx dX), second half, beside the split of the first
    add_t(iK, x3, 1);
    x_of(0);
    if constexpr (STORE) {
      // rows behind the sequence's end lie behind the buffer
      const int left = sp.Tq - n * C < C ? sp.Tq - n * C : C;
      const BufRes to = make_buf(static_cast<IO*>(p.dv) + (size_t)(sp.tok0 + n * C) * HD,
                                 (unsigned)(left * (int)HD * ES));
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = 0; t < TL; ++t)
          store_tile(to, Op::row4(t, g4), (int)HD * ES, (h * Dv + v0 + 16 * v) * ES, dX[v][t], r, IO{});
    }
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 7: the first half, and the split of dS as its tiles are done
    add_t(iK, x3, 0);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int u = 0; u < NUK; ++u) s2[v][u].set(&dS[v][TPU * u]);
  }
  if (d_out != nullptr) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) d_out[16 * v + (size_t)(Op::row4(t, g4) + e) * Dv] = dS[v][t][e];
  }
}

template <int DK, int WV, int NV, typename IO>
__global__ __launch_bounds__(64 * WV) void kda_gdr_two_walks_kernel(GdrReverseParams r, GdrWalkParams w, int Dv,
                                                                    int half) {
  constexpr int A = GdrReverseLds<DK, WV, NV, IO>::BYTES, B = GdrWalkLds<DK, WV, NV, IO, false>::BYTES;
  __shared__ __attribute__((aligned(16))) char lds[2 * (A > B ? A : B)];
  if ((int)blockIdx.x < half)
    gdr_reverse<DK, WV, NV, IO, true>(r, Dv, blockIdx.x, lds);
  else
    gdr_walk<DK, WV, NV, IO, false, true>(w, Dv, blockIdx.x - half, lds);
}

template <int DK, int WV, int NV, typename IO>
__global__ __launch_bounds__(64 * WV) void kda_gdr_reverse_kernel(GdrReverseParams r, int Dv) {
  __shared__ __attribute__((aligned(16))) char lds[2 * GdrReverseLds<DK, WV, NV, IO>::BYTES];
  gdr_reverse<DK, WV, NV, IO, false>(r, Dv, blockIdx.x, lds);
}

template <int DK, int WV, int NV, typename IO>
static hipError_t launch_ends_t(const GdrReverseParams& r, int Dv, hipStream_t st) {
  const size_t grid = gdr_walk_grid(r.walks, r.s.Hv / r.s.Hk, Dv / (16 * NV * WV));
  hipLaunchKernelGGL((kda_gdr_reverse_kernel<DK, WV, NV, IO>), dim3((unsigned)grid), dim3(64 * WV), 0, st, r, Dv);
  return hipGetLastError();
}

template <int DK, int WV, int NV, typename IO>
static hipError_t launch_two_t(const GdrReverseParams& r, const GdrWalkParams& w, int Dv, hipStream_t st) {
  // half: a multiple of 8, so that both roles keep their groups on one XCD
  const size_t half = gdr_walk_grid(w.walks, r.s.Hv / r.s.Hk, Dv / (16 * NV * WV));
  hipLaunchKernelGGL((kda_gdr_two_walks_kernel<DK, WV, NV, IO>), dim3((unsigned)(2 * half)), dim3(64 * WV), 0, st, r,
                     w, Dv, (int)half);
  return hipGetLastError();
}

template <int DK, typename IO>
static hipError_t launch_two_w(const GdrReverseParams& all_r, const GdrWalkParams& all_w, int Dv, hipStream_t st) {
  GdrReverseParams r = all_r;
  GdrWalkParams w = all_w;
  const int rows = r.s.NS * r.s.Hv;
  if (w.nseg > 1) {
    if (hipError_t e = launch_gdr_maps(w, DK, Dv, sizeof(IO) == 4, st); e != hipSuccess) return e;
    r.pass = 1;
    r.walks = rows * (r.nseg - 1);
    hipError_t e;
    if (Dv == 32) e = launch_ends_t<DK, 2, 1, IO>(r, Dv, st);
    else if (sizeof(IO) == 2 && gdr_whole_head(r.walks, Dv)) e = launch_ends_t<DK, sizeof(IO) == 2 ? 8 : 4, 1, IO>(r, Dv, st);
    else e = launch_ends_t<DK, 4, 1, IO>(r, Dv, st);
    if (e != hipSuccess) return e;
    GdrWalkParams c = w;
    c.starts = r.ends;
    if (e = launch_gdr_compose(c, DK, Dv, true, st); e != hipSuccess) return e;
  }
  w.pass = w.walk0 = r.pass = 0;
  w.walks = r.walks = rows * (w.nseg > 1 ? w.nseg : 1);
  if (Dv == 32) return launch_two_t<DK, 2, 1, IO>(r, w, Dv, st);
  if constexpr (sizeof(IO) == 2)
    if (gdr_whole_head(2l * w.walks, Dv)) return launch_two_t<DK, 8, 1, IO>(r, w, Dv, st);
  return launch_two_t<DK, 4, 1, IO>(r, w, Dv, st);
}

hipError_t launch_gdr_two_walks(const GdrReverseParams& r, const GdrWalkParams& w, int Dk, int Dv, bool fp32,
                                hipStream_t st) {
  switch (Dk) {
    case 32: return fp32 ? launch_two_w<32, float>(r, w, Dv, st) : launch_two_w<32, __bf16>(r, w, Dv, st);
    case 64: return fp32 ? launch_two_w<64, float>(r, w, Dv, st) : launch_two_w<64, __bf16>(r, w, Dv, st);
    case 128: return fp32 ? launch_two_w<128, float>(r, w, Dv, st) : launch_two_w<128, __bf16>(r, w, Dv, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
