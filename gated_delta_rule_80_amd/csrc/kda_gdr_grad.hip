// Gradients of a chunk's q, k, g, beta in the gated delta rule with one decay per
// head, from the state S at the chunk's start, the gradient dS of its end state and
// the walks' Y and dX = dv: one workgroup of 4 waves per (chunk, query/key head),
// over the value heads of that head in turn (their sum is the gradient of shared
// rows, in one order, without atomics).
//
// With q' = scale q^, D_ij = e^{G_i - G_j}, w_j = b_j k^_j:
//   dq'_i  = gamma_i S dO_i  + sum_{j<=i} E1_ij w_j     E1_ij =  D_ij dO_i . Y_j
//   dke_i  = -gamma_i S dX_i + sum_{j<i}  E2_ij w_j     E2_ij = -D_ij dX_i . Y_j
//   dw_j   = lambda_j dS Y_j + sum_{i>=j} E1_ij q'_i + sum_{i>j} E2_ij k^_i
//   dk^ = dke + b dw;  db_j = k^_j . dw_j
//   dG_i = q'_i . dq'_i + k^_i . dke_i - b_i k^_i . dw_i, the chunk's last G also
//          gamma_C <S, dS> + sum_j b_j k^_j . (lambda_j dS Y_j);  dg = sums from the end
// Everything is formed transposed (channel x token): a lane holds 4 consecutive
// channels of one token, so the row dots and the stores are contiguous.  A wave owns
// half of the chunk's tokens and half of the channels.
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

template <int DK, int DV, typename IO>
__global__ __launch_bounds__(256) void kda_gdr_grad_kernel(GdrGradParams p) {
  using Op = GOp<IO>;
  using Frag = typename Op::Frag;
  constexpr bool F32 = sizeof(IO) == 4;
  constexpr int C = gdr_chunk(F32), TL = C / 16, TPU = Op::TPU;
  constexpr int TW = TL / 2;             // token tiles of a wave
  constexpr int CW = DK / 16 / 2;        // channel tiles of a wave
  constexpr int NUV = DV / Op::KU, NUC = C / Op::KU;
  constexpr GdrRecord R = gdr_record(F32, true);
  using I = GImg<IO, DK>;
  constexpr int RC = I::RC, EPC = I::EPC;
  __shared__ __attribute__((aligned(16))) IO iK[C * DK];
  __shared__ __attribute__((aligned(16))) IO iQ[C * DK];
  __shared__ __attribute__((aligned(16))) float sc[kGdrScalars][C];
  __shared__ float red[2][4][C];
  __shared__ float redS[4];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g4 = lane >> 4;
  const int wt = wave & 1, wc = wave >> 1;
  const int pos = xcd_major(blockIdx.x, gridDim.x);
  const int hk = pos % p.s.Hk, row = pos / p.s.Hk;
  const int b = row % p.s.B, slot = row / p.s.B;
  const int G = p.s.Hv / p.s.Hk;
  const GdrChunk ch0 = gdr_chunk_at(p.s, slot, b, hk * G, C);
  if (ch0.n == 0) return;  // uniform
  const int n = ch0.n, last = n - 1;
  const long HD = (long)p.s.Hv * DV;

  // ---- q, k rows (rows behind the end read the last one; their scalars are zero)
  for (int idx = tid; idx < 2 * C * RC; idx += 256) {
    const bool isq = idx >= C * RC;
    const int i = isq ? idx - C * RC : idx;
    const int t = i / RC, c = i % RC, ts = t < last ? t : last;
    const IO* src = isq ? static_cast<const IO*>(p.q) + (ch0.tok + ts) * p.s.qs
                        : static_cast<const IO*>(p.k) + (ch0.tok + ts) * p.s.ks;
    *reinterpret_cast<f32x4*>((isq ? iQ : iK) + (t * RC + Op::template swz<RC>(t, c)) * EPC) =
        *reinterpret_cast<const f32x4*>(src + (size_t)hk * DK + c * EPC);
  }

  f32x4 sumq[CW][TW], sumk[CW][TW];
#pragma unroll
  for (int c = 0; c < CW; ++c)
#pragma unroll
    for (int t = 0; t < TW; ++t) sumq[c][t] = sumk[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int tile0 = TW * wt;        // this wave's first token tile
  const int c0 = 16 * CW * wc;      // and first channel

#pragma unroll 1
  for (int gi = 0; gi < G; ++gi) {
    const int h = hk * G + gi;
    const GdrChunk ch = gdr_chunk_at(p.s, slot, b, h, C);
    const float* rs = reinterpret_cast<const float*>(p.rec + ch.rec * R.bytes + R.sc);
    __syncthreads();  // the previous head's scalars and sums have been read
    for (int i = tid; i < kGdrScalars * C; i += 256) sc[i / C][i % C] = rs[i];
    __syncthreads();

    const IO* pO = static_cast<const IO*>(p.dO) + ch.tok * HD + (size_t)h * DV;
    const IO* pX = static_cast<const IO*>(p.dv) + ch.tok * HD + (size_t)h * DV;
    const IO* pY = static_cast<const IO*>(p.y) + ch.tok * HD + (size_t)h * DV;
    auto vrow = [&](const IO* base, int t, int u) {  // unit u of row t along the values
      const int ts = t < last ? t : last;
      return *reinterpret_cast<const Frag*>(base + ts * HD + Op::KU * u + (Op::KU / 4) * g4);
    };
    const size_t ckb = ch.rec * (size_t)DK * DV;
    const IO* pS = static_cast<const IO*>(p.ckS) + ckb;
    const IO* pD = static_cast<const IO*>(p.ckdS) + ckb;
    auto ckrow = [&](const IO* base, int c, int u) {  // unit u of channel c's row
      const int v = Op::KU * u + (Op::KU / 4) * g4;
      return *reinterpret_cast<const Frag*>(base + (size_t)(v >> 4) * DK * 16 + c * 16 + (v & 15));
    };

    // ---- this wave's tokens
    Frag fO[TW][NUV], fX[TW][NUV], fY[TW][NUV];
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int u = 0; u < NUV; ++u) {
        fO[t][u] = vrow(pO, 16 * (tile0 + t) + r, u);
        fX[t][u] = vrow(pX, 16 * (tile0 + t) + r, u);
        fY[t][u] = vrow(pY, 16 * (tile0 + t) + r, u);
      }
    // ---- S dO, S dX, dS Y and <S, dS>
    f32x4 aq[CW][TW], ae[CW][TW], aw[CW][TW];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < CW; ++c) {
#pragma unroll
      for (int t = 0; t < TW; ++t) aq[c][t] = ae[c][t] = aw[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NUV; ++u) {
        const Frag fs = ckrow(pS, c0 + 16 * c + r, u), fd = ckrow(pD, c0 + 16 * c + r, u);
        if (wt == 0) dot = frag_dot(fs, fd, dot);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          gmma(aq[c][t], fs, fO[t][u]);
          gmma(ae[c][t], fs, fX[t][u]);
          gmma(aw[c][t], fd, fY[t][u]);
        }
      }
    }
    const float GhC = sc[5][C - 1], GlC = sc[6][C - 1];
    float kw1[TW];
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const int tk = 16 * (tile0 + t) + r;
      const float gam = exp2_fast(sc[5][tk] + sc[6][tk]);
      const float lam = exp2_fast((GhC - sc[5][tk]) + (GlC - sc[6][tk]));
      kw1[t] = 0.f;
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 16 * c + 4 * g4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          aq[c][t][e] *= gam;
          ae[c][t][e] *= -gam;
          aw[c][t][e] *= lam;
          kw1[t] = fmaf(k4[e], aw[c][t][e], kw1[t]);
        }
      }
      kw1[t] *= sc[3][tk];
    }
    // ---- pairs: this wave's tokens as rows i (E, over j <= i)
#pragma unroll
    for (int u = 0; u < NUC; ++u) {
      if (TPU * u > tile0 + TW - 1) continue;  // uniform: no j of the unit precedes a token
      Terms<IO, 2> e1[TW], e2[TW];
      f32x4 mo[TW][TPU], mx[TW][TPU];
#pragma unroll
      for (int s = 0; s < TPU; ++s) {
        const int jt = TPU * u + s;
#pragma unroll
        for (int t = 0; t < TW; ++t) mo[t][s] = mx[t][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NUV; ++v) {
          const Frag fy = vrow(pY, Op::perm(jt, r), v);
#pragma unroll
          for (int t = 0; t < TW; ++t) {
            gmma(mo[t][s], fy, fO[t][v]);
            gmma(mx[t][s], fy, fX[t][v]);
          }
        }
        const int j4 = Op::row4(jt, g4);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          const int i = 16 * (tile0 + t) + r;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j4 + e;
            const float d = j <= i ? exp2_fast((sc[5][i] - sc[5][j]) + (sc[6][i] - sc[6][j])) * (sc[7][j] * sc[3][j])
                                   : 0.f;
            mo[t][s][e] *= d;
            mx[t][s][e] *= j < i ? -d : 0.f;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        e1[t].set(mo[t]);
        e2[t].set(mx[t]);
      }
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        const Frag fk = g_col<DK>(iK, u, c0 + 16 * c, r, g4);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          gmma_all(aq[c][t], fk, e1[t]);
          gmma_all(ae[c][t], fk, e2[t]);
        }
      }
    }
    // ---- and as columns j (over i >= j)
#pragma unroll
    for (int u = 0; u < NUC; ++u) {
      if (TPU * u + TPU - 1 < tile0) continue;  // uniform: every i of the unit precedes
      Terms<IO, 2> e1[TW], e2[TW];
      f32x4 mo[TW][TPU], mx[TW][TPU];
#pragma unroll
      for (int s = 0; s < TPU; ++s) {
        const int it = TPU * u + s;
#pragma unroll
        for (int t = 0; t < TW; ++t) mo[t][s] = mx[t][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NUV; ++v) {
          const Frag fo = vrow(pO, Op::perm(it, r), v), fx = vrow(pX, Op::perm(it, r), v);
#pragma unroll
          for (int t = 0; t < TW; ++t) {
            gmma(mo[t][s], fo, fY[t][v]);
            gmma(mx[t][s], fx, fY[t][v]);
          }
        }
        const int i4 = Op::row4(it, g4);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          const int j = 16 * (tile0 + t) + r;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = i4 + e;
            const float d = j <= i ? exp2_fast((sc[5][i] - sc[5][j]) + (sc[6][i] - sc[6][j])) : 0.f;
            mo[t][s][e] *= d * (sc[4][i] * p.scale);
            mx[t][s][e] *= j < i ? -d * sc[3][i] : 0.f;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        e1[t].set(mo[t]);
        e2[t].set(mx[t]);
      }
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        const Frag fq = g_col<DK>(iQ, u, c0 + 16 * c, r, g4);
        const Frag fk = g_col<DK>(iK, u, c0 + 16 * c, r, g4);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          gmma_all(aw[c][t], fq, e1[t]);
          gmma_all(aw[c][t], fk, e2[t]);
        }
      }
    }
    // ---- row dots and the sums over the heads
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const int tk = 16 * (tile0 + t) + r;
      float qd = 0.f, ke = 0.f, kw = 0.f;
      const float bt = sc[7][tk];
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 16 * c + 4 * g4);
        const f32x4 q4 = g_four<IO, DK>(iQ, tk, c0 + 16 * c + 4 * g4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qd = fmaf(q4[e], aq[c][t][e], qd);
          ke = fmaf(k4[e], ae[c][t][e], ke);
          kw = fmaf(k4[e], aw[c][t][e], kw);
          sumq[c][t][e] += aq[c][t][e];
          sumk[c][t][e] += fmaf(bt, aw[c][t][e], ae[c][t][e]);
        }
      }
      qd = sum_groups(qd * sc[4][tk] * p.scale);
      ke = sum_groups(ke * sc[3][tk]);
      kw = sum_groups(kw * sc[3][tk]);
      const float k1 = sum_groups(kw1[t]);
      if (g4 == 0) {
        red[wc][0][tk] = qd;
        red[wc][1][tk] = ke;
        red[wc][2][tk] = kw;
        red[wc][3][tk] = k1;
      }
    }
    dot = group_sum<64>(dot);
    if (lane == 0) redS[wave] = dot;
    __syncthreads();
    if (wave == 0) {
      float dG = 0.f, kw = 0.f, k1 = 0.f;
      if (lane < C) {
        kw = red[0][2][lane] + red[1][2][lane];
        k1 = sc[7][lane] * (red[0][3][lane] + red[1][3][lane]);
        dG = (red[0][0][lane] + red[1][0][lane]) + (red[0][1][lane] + red[1][1][lane]) - sc[7][lane] * kw;
      }
      k1 = group_sum<64>(k1);
      // waves 0 and 2 hold the two channel halves of <S, dS>
      if (lane == C - 1) dG += exp2_fast(GhC + GlC) * (redS[0] + redS[2]) + k1;
#pragma unroll
      for (int m = 1; m < C; m <<= 1) {
        const float y = __shfl_down(dG, m, 64);
        if (lane + m < C) dG += y;
      }
      if (lane < n) {
        const size_t at = (size_t)(ch.tok + lane) * p.s.Hv + h;
        float dg = dG, db = kw;
        if (p.A_log != nullptr) {
          p.dg32[at] = dg;
          const float z = to_f32(static_cast<const IO*>(p.g)[at]) + p.dt_bias[h];
          dg *= -expf(p.A_log[h]) / (1.0f + expf(-z));
        }
        if (p.beta_logits) db *= sc[7][lane] * (1.0f - sc[7][lane]);
        static_cast<IO*>(p.dg)[at] = from_f32<IO>(dg);
        static_cast<IO*>(p.dbeta)[at] = from_f32<IO>(db);
      }
    }
  }
  // ---- through the norms, to the raw rows
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    const int tk = 16 * (tile0 + t) + r;
    float qd = 0.f, kd = 0.f;
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 16 * c + 4 * g4);
      const f32x4 q4 = g_four<IO, DK>(iQ, tk, c0 + 16 * c + 4 * g4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qd = fmaf(q4[e], sumq[c][t][e], qd);
        kd = fmaf(k4[e], sumk[c][t][e], kd);
      }
    }
    qd = sum_groups(qd);
    kd = sum_groups(kd);
    if (g4 == 0) {
      red[wc][0][tk] = qd;
      red[wc][1][tk] = kd;
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    const int tk = 16 * (tile0 + t) + r;
    if (tk >= n) continue;
    const float rq = sc[4][tk], rk = sc[3][tk];
    // x / |x|: dx = (dy - x^ (x^ . dy)) / |x|
    const float qd = p.l2 ? rq * rq * (red[0][0][tk] + red[1][0][tk]) : 0.f;
    const float kd = p.l2 ? rk * rk * (red[0][1][tk] + red[1][1][tk]) : 0.f;
    const size_t at = ((size_t)(ch0.tok + tk) * p.s.Hk + hk) * DK + c0 + 4 * g4;
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      const f32x4 k4 = g_four<IO, DK>(iK, tk, c0 + 16 * c + 4 * g4);
      const f32x4 q4 = g_four<IO, DK>(iQ, tk, c0 + 16 * c + 4 * g4);
      float dq[4], dk[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dq[e] = p.scale * rq * (sumq[c][t][e] - q4[e] * qd);
        dk[e] = rk * (sumk[c][t][e] - k4[e] * kd);
      }
      store4(static_cast<IO*>(p.dq) + at + 16 * c, dq[0], dq[1], dq[2], dq[3]);
      store4(static_cast<IO*>(p.dk) + at + 16 * c, dk[0], dk[1], dk[2], dk[3]);
    }
  }
}

template <int DK, typename IO>
static hipError_t launch_grad_t(const GdrGradParams& p, int Dv, hipStream_t st) {
  const unsigned grid = (unsigned)((size_t)p.s.B * p.s.Hk * p.s.NT);
  switch (Dv) {
    case 32: hipLaunchKernelGGL((kda_gdr_grad_kernel<DK, 32, IO>), dim3(grid), dim3(256), 0, st, p); break;
    case 64: hipLaunchKernelGGL((kda_gdr_grad_kernel<DK, 64, IO>), dim3(grid), dim3(256), 0, st, p); break;
    case 128: hipLaunchKernelGGL((kda_gdr_grad_kernel<DK, 128, IO>), dim3(grid), dim3(256), 0, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
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
