// State walk of the gated delta rule with one decay per head: one workgroup of WV
// waves per (sequence, value head, block of 16 NV WV value columns) walks the chunks
// of its sequence in order; each wave owns NV tiles of 16 value columns and carries
// the whole chain K S -> X -> Y -> S' of a chunk in registers (kda_gdr_device.h), so
// the only thing the waves share is the chunk's data in LDS: k, q, v rows as the
// caller holds them and the record of the preparation.  The next chunk is copied
// into the other half of LDS (global-to-LDS loads, no registers) while this one
// computes; one barrier a chunk.
//
// Precision (bf16 inputs): S, X, Y are float32 accumulators.  As operands they are
// split into bf16 terms: S 2, X 3 and b lambda rk Y 3 where they lead to the
// state, which leaves in float32 (relative error about 5e-7 against float64);
// S 2, Y 2 and P 1 where they lead to the output, which is rounded to bf16.
//
// What bounds it: LDS holds one workgroup, so one or two waves per SIMD issue, in order,
// the matrix products of a chunk (154 of 16 x 16 x 32 a wave at D = 128) and the vector
// work of splitting their operands (about 550 instructions).  The chunk is therefore cut
// into slots, each with products of one half of the tokens beside the splitting of the
// other half.  Measured with bf16, D = 128 and a workgroup on every CU: 5.2 us a chunk of a
// whole head (8 waves; 256 walks of 128 chunks in 670 us, 890 TFLOP/s of products, the
// matrix units 48% busy), 3.3 us a chunk of half a head (4 waves, one a SIMD).  With a
// workgroup on every CU the chunk's 84 KB also come near the memory's rate (4.0 TB/s at 64k
// tokens of 12 heads).
#pragma once
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

template <int DK, int WV, int NV, typename IO, bool OUT>
struct GdrWalkLds {
  static constexpr bool F32 = sizeof(IO) == 4;
  static constexpr int C = gdr_chunk(F32), ES = (int)sizeof(IO), VB = 16 * NV * WV;
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

// workgroup blk of the launch; lds: 2 GdrWalkLds::BYTES
template <int DK, int WV, int NV, typename IO, bool OUT, bool CK>
__device__ __forceinline__ void gdr_walk(const GdrWalkParams& p, int Dv, int blk, char* lds) {
  using L = GdrWalkLds<DK, WV, NV, IO, OUT>;
  using Op = GOp<IO>;
  using Frag = typename Op::Frag;
  constexpr bool F32 = L::F32;
  constexpr int C = L::C, NT = 64 * WV, VB = L::VB;
  constexpr int CT = DK / 16, TL = C / 16;             // tiles of the state and of the tokens
  constexpr int NUK = DK / Op::KU, NUC = C / Op::KU;   // contraction units
  constexpr int TPU = Op::TPU, TT = L::TT, ES = L::ES;
  constexpr int NF = gdr_frags(F32);
  static_assert(NUC == 2, "the slots below take the chunk in two halves");
  constexpr GdrRecord R = gdr_record(F32, CK);
  // stores of a chunk: o, 4 columns each; or the state and Y
  constexpr int NSTORE = NV * (OUT ? TL : (CK ? (F32 ? 4 : 1) * (CT + TL) : 0));
  static_assert(!(OUT && CK), "the stores are counted for one or the other");
  // the maps' passes read Tm and the scalars only, which stand alike in both records
  constexpr GdrRecord RB = gdr_record(F32, true);
  static_assert(RB.t == R.t && RB.sc == R.sc, "one place in both records");
  const size_t rec_bytes = !OUT && !CK && p.bwd ? RB.bytes : R.bytes;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g4 = lane >> 4;
  int bh, vblk, seg = 0, nseg = p.nseg;
  if (!gdr_walk_id(blk, Dv / VB, p.s.Hv / p.s.Hk, p.walks, bh, vblk)) return;  // uniform
  bh += p.walk0;
  size_t seg_idx = 0;  // of this segment in starts and maps
  if (p.nseg > 1) {
    if (p.segstart == nullptr) {
      const int walks = p.s.B * p.s.Hv;
      seg = bh / walks + (p.pass == 2 ? 1 : 0);  // the first segment needs no M
      bh %= walks;
      seg_idx = (size_t)bh * nseg + seg;
    } else {
      const int id = bh / p.s.Hv, hh = bh % p.s.Hv;
      if (id >= uniform(p.segstart[p.s.NS])) return;  // uniform
      const int q = uniform(seq_of_slot(p.segstart, p.s.NS, id)), s0 = uniform(p.segstart[q]);
      nseg = uniform(p.segstart[q + 1]) - s0;
      seg = id - s0;
      if (p.pass != 0 && (seg == nseg - 1 || (p.pass == 2 && seg == 0))) return;  // uniform: no map needed
      seg_idx = (size_t)hh * p.nseg + id;
      bh = q * p.s.Hv + hh;
    }
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
  // a map's M: columns of the state in place of values, and no values
  const bool linear = !OUT && !CK && p.pass == 2;
  const int v0 = vblk * VB + 16 * NV * wave;  // this wave's value columns
  const long HD = (long)p.s.Hv * Dv;

  const IO* kb = static_cast<const IO*>(p.k) + sp.tok0 * p.s.ks + (size_t)hk * DK;
  const IO* qb = static_cast<const IO*>(p.q) + sp.tok0 * p.s.qs + (size_t)hk * DK;
  const IO* vb = static_cast<const IO*>(p.v) + sp.tok0 * p.s.vs + (size_t)h * Dv + vblk * VB;

  GdrCopy<NT, C, DK, IO> ck, cq;
  GdrCopy<NT, C, VB, IO> cv;
  ck.init(p.s.ks);
  cv.init(p.s.vs);
  if constexpr (OUT) cq.init(p.s.qs);
  // In three parts, which the slots below issue apart from one another: a wave that
  // issues all its copies at once waits for the address unit.
  auto copy = [&](int n, char* buf, int part) {
    const int last = sp.Tq - n * C - 1;  // >= 0: the chunk exists
    const long t0 = (long)n * C;
    const char* rec = p.rec + (sp.rec0 + n * sp.rstride) * rec_bytes;
    if (part == 0) {
      const IO* pk = kb + t0 * p.s.ks;
      const IO* pv = vb + t0 * p.s.vs;
      if (last >= C - 1) {
        ck.whole(buf + L::K, pk, wave);
        if (!linear) cv.whole(buf + L::V, pv, wave);
      } else {
        ck.part(buf + L::K, pk, p.s.ks, last, wave);
        if (!linear) cv.part(buf + L::V, pv, p.s.vs, last, wave);
      }
    } else if (part == 1) {
      // Tm and the scalars follow one another in the record and in LDS
      gdr_copy_flat<NT, L::TB + kGdrScalars * C * 4>(buf + L::T, rec + R.t, wave);
      if constexpr (OUT) gdr_copy_flat<NT, L::PB>(buf + L::P, rec + R.p, wave);
    } else if constexpr (OUT) {
      const IO* pq = qb + t0 * p.s.qs;
      if (last >= C - 1)
        cq.whole(buf + L::Q, pq, wave);
      else
        cq.part(buf + L::Q, pq, p.s.qs, last, wave);
    }
  };

  // ---- initial state, and its two terms as the first chunk's operand
  f32x4 S[NV][CT];
  Terms<IO, 2> s2[NV][NUK];
  const size_t sbase = (size_t)bh * DK * Dv + v0 + r;
  // where this walk's state comes from (NULL: zeros) and goes to (NULL: nowhere)
  const size_t seg_at = seg_idx * DK * Dv + v0 + r;
  const float* s_in = p.S0 != nullptr && seg == 0 ? p.S0 + sbase : nullptr;
  float* s_out = p.S_T != nullptr ? p.S_T + sbase : nullptr;
  if (p.nseg > 1) {
    if (p.pass == 0 && nseg > 1) s_in = p.starts + seg_at;
    if (p.pass == 0 && seg < nseg - 1) s_out = nullptr;
    if (p.pass == 1) s_out = p.starts + seg_at + (size_t)DK * Dv;
    if (p.pass == 2) s_out = p.maps + seg_at;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[v][t][e] = linear && Op::row4(t, g4) + e == v0 + 16 * v + r ? 1.f : 0.f;
  if (s_in != nullptr) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[v][t][e] = s_in[16 * v + (size_t)(Op::row4(t, g4) + e) * Dv];
  }
  if (p.nseg > 1 && p.pass == 1 && seg == 0) {
    // kept for the pass with outputs, whose last segments may write S_T over S0
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          p.starts[seg_at + 16 * v + (size_t)(Op::row4(t, g4) + e) * Dv] = S[v][t][e];
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int u = 0; u < NUK; ++u) s2[v][u].set(&S[v][TPU * u]);

  if (sp.nch > 0)
    for (int part = 0; part < 3; ++part) copy(0, lds, part);
  __builtin_amdgcn_s_waitcnt(0);  // the first chunk's copies have no stores behind them
#pragma unroll 1
  for (int n = 0; n < sp.nch; ++n) {
    char* buf = lds + (n & 1) * L::BYTES;
    // this wave's copies of chunk n have landed (the only vector memory operations
    // it issued after them are the stores of chunk n - 1: they may stay in flight);
    // after the barrier everybody's have, and everybody is done with the other
    // buffer
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

    constexpr int HT = TL / 2;  // token tiles of a half: one unit of the token contraction
    static_assert(HT == TPU, "a half is a unit");
    auto rows = [&](Frag (&f)[HT][NUK], const IO* img, int t0) {
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int u = 0; u < NUK; ++u) f[t][u] = g_row<IO, DK>(img, Op::perm(t0 + t, r), u, g4);
    };
    f32x4 X[NV][TL], O[NV][TL], Y[NV][TL];
    auto k_s = [&](const Frag (&f)[HT][NUK], int t0) {  // X = K S (as far as this half)
#pragma unroll
      for (int u = 0; u < NUK; ++u)
#pragma unroll
        for (int i = 0; i < s2[0][u].N; ++i)
#pragma unroll
          for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (u == 0 && i == 0) X[v][t0 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
              gmma(X[v][t0 + t], f[t][u], s2[v][u].t[i]);
            }
    };
    auto s_q = [&](const Frag (&f)[HT][NUK], int t0) {  // O^T = S^T Q^T
#pragma unroll
      for (int u = 0; u < NUK; ++u)
#pragma unroll
        for (int i = 0; i < s2[0][u].N; ++i)
#pragma unroll
          for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (u == 0 && i == 0) O[v][t0 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
              gmma(O[v][t0 + t], s2[v][u].t[i], f[t][u]);
            }
    };
    AccRaw<IO> V[NV][TL];
    Terms<IO, 3> x3[NV][NUC], y3[NV][NUC];
    Terms<IO, 2> y2[NV][NUC];
    auto x_of = [&](int u) {  // X = V - cx (K S), split
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int t = HT * u; t < HT * u + HT; ++t) {
          const f32x4 cx = *reinterpret_cast<const f32x4*>(sc + Op::row4(t, g4));
#pragma unroll
          for (int e = 0; e < 4; ++e) X[v][t][e] = fmaf(-cx[e], X[v][t][e], linear ? 0.f : V[v][t][e]);
        }
        x3[v][u].set(&X[v][TPU * u]);
      }
    };
    // the lower triangles of units of Tm and P
    Frag fT[NF][TT], fP[NF];
    auto tm_x = [&](int t0, int u) {  // Y += Tm X over one unit, tiles t0 .. of a half
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int j = 0; j < x3[0][u].N; ++j)
          if (k + j < x3[0][u].N)  // the products below the third term are left out
#pragma unroll
            for (int t = t0; t < t0 + HT; ++t)
#pragma unroll
              for (int v = 0; v < NV; ++v) {
                if (u == 0 && k == 0 && j == 0) Y[v][t] = f32x4{0.f, 0.f, 0.f, 0.f};
                gmma(Y[v][t], fT[tri_at<TPU, NUC, false>(t, u)][k], x3[v][u].t[j]);
              }
    };
    auto y_of = [&](int u) {  // Y split for the output, b lambda rk Y for the state
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (OUT) y2[v][u].set(&Y[v][TPU * u]);
        f32x4 z[HT];
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const f32x4 cy = *reinterpret_cast<const f32x4*>(sc + C + Op::row4(HT * u + t, g4));
#pragma unroll
          for (int e = 0; e < 4; ++e) z[t][e] = cy[e] * Y[v][HT * u + t][e];
        }
        y3[v][u].set(z);
      }
    };
    auto y_p = [&](int t0, int u) {  // O^T += Y^T P^T
#pragma unroll
      for (int k = 0; k < y2[0][u].N; ++k)
#pragma unroll
        for (int t = t0; t < t0 + HT; ++t)
#pragma unroll
          for (int v = 0; v < NV; ++v) gmma(O[v][t], y2[v][u].t[k], fP[tri_at<TPU, NUC, false>(t, u)]);
    };
    constexpr int GT = CT < 4 ? CT : 4;  // state tiles of a group
    auto kt_y = [&](int u) {  // S += K^T (b lambda rk Y)
#pragma unroll
      for (int j = 0; j < CT; j += GT) {
        Frag f[GT];
        g_colp_tiles<DK>(iK, u, j, r, g4, f);
#pragma unroll
        for (int k = 0; k < y3[0][u].N; ++k)
#pragma unroll
          for (int t = 0; t < GT; ++t)
#pragma unroll
            for (int v = 0; v < NV; ++v) gmma(S[v][j + t], f[t], y3[v][u].t[k]);
      }
    };

    // ---- slot 1: K S, first half
    Frag fa[HT][NUK], fb[HT][NUK];
    rows(fa, iK, 0);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < TL; ++t) V[v][t].template load<VB>(iV, t, 16 * (NV * wave + v), r, g4);
    __builtin_amdgcn_sched_barrier(0);  // (transposing reads the compiler sees: before the copies)
    char* nbuf = lds + ((n + 1) & 1) * L::BYTES;
    if (n + 1 < sp.nch) copy(n + 1, nbuf, 0);
    __builtin_amdgcn_sched_barrier(0);
    rows(fb, iK, HT);
    k_s(fa, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (n + 1 < sp.nch) copy(n + 1, nbuf, 1);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 2: K S, second half, beside the split of the first half's X and the
    // state's decay
    if constexpr (OUT) rows(fa, iQ, 0);
    k_s(fb, HT);
    x_of(0);
    __builtin_amdgcn_sched_barrier(0);
    if (OUT && n + 1 < sp.nch) copy(n + 1, nbuf, 2);
    __builtin_amdgcn_sched_barrier(0);  // the stores counted above come after the copies
    if constexpr (CK) {
      // the state at the chunk's start, for the gradients
      const BufRes to = make_buf(static_cast<IO*>(p.ckpt) + (sp.rec0 + n * sp.rstride) * (size_t)DK * Dv,
                                 (unsigned)(DK * Dv * ES));
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = 0; t < CT; ++t)
          store_tile(to, Op::row4(t, g4), 16 * ES, (v0 + 16 * v) * DK * ES, S[v][t], r, IO{});
    }
    const float lamC = exp2_fast(sc[5 * C + C - 1] + sc[6 * C + C - 1]);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[v][t][e] *= lamC;
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 3: O = co Q S beside the split of the second half's X
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int k = 0; k < TT; ++k) fT[i][k] = g_frag(iT, i * TT + k, lane);
    if constexpr (OUT) {
      rows(fb, iQ, HT);
      s_q(fa, 0);
      s_q(fb, HT);
    }
    x_of(1);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 4: Y = Tm X, first half
    if constexpr (OUT)
#pragma unroll
      for (int i = 0; i < NF; ++i) fP[i] = g_frag(iP, i, lane);
    tm_x(0, 0);
    if constexpr (OUT)
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        const float co = sc[2 * C + Op::perm(t, r)];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[v][t][e] *= co;
      }
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 5: Y, second half, beside the split of the first
    tm_x(HT, 0);
    tm_x(HT, 1);
    y_of(0);
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 6: the first half's share of S and O beside the split of the second
    kt_y(0);
    if constexpr (OUT) {
      y_p(0, 0);
      y_p(HT, 0);
    }
    y_of(1);
    if constexpr (CK) {
      const BufRes to = make_buf(static_cast<IO*>(p.y) + (size_t)(sp.tok0 + n * C) * HD, chunk_bytes);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = 0; t < TL; ++t)
          store_tile(to, Op::row4(t, g4), (int)HD * ES, (h * Dv + v0 + 16 * v) * ES, Y[v][t], r, IO{});
    }
    __builtin_amdgcn_sched_barrier(0);
    // ---- slot 7: the second half's share, the output's stores, and the split of S
    // for the next chunk as its tiles are done
    if constexpr (OUT) {
      y_p(HT, 1);
      const BufRes ob = make_buf(static_cast<IO*>(p.o) + (size_t)(sp.tok0 + n * C) * HD, chunk_bytes);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = 0; t < TL; ++t)
          store_four(ob, Op::perm(t, r) * (int)HD * ES + (h * Dv + v0 + 16 * v + 4 * g4) * ES, O[v][t], IO{});
    }
    kt_y(1);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int u = 0; u < NUK; ++u) s2[v][u].set(&S[v][TPU * u]);
  }
  if (s_out != nullptr) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_out[16 * v + (size_t)(Op::row4(t, g4) + e) * Dv] = S[v][t][e];
  }
}

}  // namespace kda
