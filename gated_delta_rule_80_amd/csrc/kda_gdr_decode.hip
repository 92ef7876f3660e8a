// Single tokens of the gated delta rule with one decay per head, on states in a
// pool: one workgroup per (row, value head).  A row names its state's slot; the
// rows of one slot are consecutive tokens of its sequence, in row order, and the
// workgroup of the first of them does them all, with the state read once, kept in
// registers and written once.
//
//   S_bar = e^g S;  y = v - S_bar^T k;  u = beta y;  S = S_bar + k u^T;  o = scale S^T q
// Both reductions over the key channels run in one sweep (o = S_bar^T q + (k.q) u).
//
// Bound by reading and writing the states: 240 slots of 96 heads, 128 x 128, two tokens
// each, 500-545 us, 5.8 TB/s; one token of 32 heads 6.5 us, the chain of one workgroup.
#include "kda_gdr_device.h"
#include "kda_launch.h"

namespace kda {

template <int DK, int DV, typename IO>
__global__ __launch_bounds__(256) void kda_gdr_decode_kernel(GdrDecodeParams p) {
  constexpr int VG = DV / 4, CG = 256 / VG, R = DK / CG;
  static_assert(R >= 1 && CG * R == DK, "decode tiling");
  __shared__ float sq[DK], sk[DK], sv[DV];
  __shared__ __attribute__((aligned(16))) float su[DV];
  __shared__ float red[3][4];
  __shared__ f32x4 part[2][CG][VG];
  __shared__ int before, next;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x % p.Hv;
  int row = blockIdx.x / p.Hv;
  const int hk = h / (p.Hv / p.Hk);
  const int vg = tid % VG, cg = tid / VG;
  const int slot = p.slots != nullptr ? p.slots[row] : row;
  if (slot < 0 || slot >= p.n_slots) return;  // uniform: a padding row
  float* S = p.S + ((size_t)slot * p.Hv + h) * DK * DV;

  // The rows of this slot.  A row that is not its slot's first leaves before it reads
  // the state: with two rows a slot, reading first cost 630 us where this takes 500-545 (240
  // slots of 96 heads, 128 x 128).
  int nxt = 0x7fffffff;  // the slot's next row after this one
  if (p.slots != nullptr) {
    if (tid == 0) {
      before = 0;
      next = 0x7fffffff;
    }
    __syncthreads();
    for (int j = tid; j < p.N; j += 256)
      if (p.slots[j] == slot) {
        if (j < row) before = 1;
        if (j > row) atomicMin(&next, j);
      }
    __syncthreads();
    if (before) return;  // uniform: an earlier row's workgroup does this one
    nxt = next;
  }
  f32x4 st[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    st[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (size_t)(cg * R + i) * DV) + vg);

  while (true) {
    // ---- the token: q, k rows with their sums, v, gates
    float xq = 0.f, xk = 0.f;
    if (tid < DK) {
      xq = to_f32(static_cast<const IO*>(p.q)[row * p.qs + (size_t)hk * DK + tid]);
      xk = to_f32(static_cast<const IO*>(p.k)[row * p.ks + (size_t)hk * DK + tid]);
    }
    if (tid < DV) sv[tid] = to_f32(static_cast<const IO*>(p.v)[row * p.vs + (size_t)h * DV + tid]);
    const size_t gi = (size_t)row * p.Hv + h;
    const float a = expf(gdr_decay<IO>(p.g, gi, p.A_log, p.dt_bias, h));
    const float bt = gdr_beta<IO>(p.beta, gi, p.beta_logits);
    float s_qq = group_sum<64>(xq * xq), s_kk = group_sum<64>(xk * xk), s_qk = group_sum<64>(xq * xk);
    if (lane == 0) {
      red[0][wave] = s_qq;
      red[1][wave] = s_kk;
      red[2][wave] = s_qk;
    }
    __syncthreads();
    s_qq = red[0][0] + red[0][1];  // q, k lie in the first DK <= 128 threads
    s_kk = red[1][0] + red[1][1];
    s_qk = red[2][0] + red[2][1];
    const float rq = (p.l2 ? 1.0f / sqrtf(s_qq + p.eps) : 1.0f) * p.scale;
    const float rk = p.l2 ? 1.0f / sqrtf(s_kk + p.eps) : 1.0f;
    const float kq = s_qk * rq * rk;
    if (tid < DK) {
      sq[tid] = xq * rq;
      sk[tid] = xk * rk;
    }
    __syncthreads();

    // ---- one sweep over the state
    f32x4 pk = {0.f, 0.f, 0.f, 0.f}, pq = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kc = sk[cg * R + i], qc = sq[cg * R + i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st[i][e] *= a;
        pk[e] = fmaf(st[i][e], kc, pk[e]);
        pq[e] = fmaf(st[i][e], qc, pq[e]);
      }
    }
    part[0][cg][vg] = pk;
    part[1][cg][vg] = pq;
    __syncthreads();
    if (tid < DV) {
      float sum_k = 0.f, sum_q = 0.f;
#pragma unroll
      for (int j = 0; j < CG; ++j) {
        sum_k += part[0][j][tid / 4][tid % 4];
        sum_q += part[1][j][tid / 4][tid % 4];
      }
      const float u = bt * (sv[tid] - sum_k);
      su[tid] = u;
      static_cast<IO*>(p.o)[((size_t)row * p.Hv + h) * DV + tid] = from_f32<IO>(fmaf(kq, u, sum_q));
    }
    __syncthreads();
    const f32x4 u4 = *reinterpret_cast<const f32x4*>(&su[4 * vg]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kc = sk[cg * R + i];
#pragma unroll
      for (int e = 0; e < 4; ++e) st[i][e] = fmaf(kc, u4[e], st[i][e]);
    }
    if (nxt == 0x7fffffff) break;
    // ---- the slot's next token
    row = nxt;
    __syncthreads();  // everybody has read sk and next
    if (tid == 0) next = 0x7fffffff;
    __syncthreads();
    for (int j = row + 1 + tid; j < p.N; j += 256)
      if (p.slots[j] == slot) atomicMin(&next, j);
    __syncthreads();
    nxt = next;
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    __builtin_nontemporal_store(st[i], reinterpret_cast<f32x4*>(S + (size_t)(cg * R + i) * DV) + vg);
}

template <int DK, typename IO>
static hipError_t launch_decode_t(const GdrDecodeParams& p, int Dv, hipStream_t st) {
  const unsigned grid = (unsigned)((size_t)p.N * p.Hv);
  switch (Dv) {
    case 32: hipLaunchKernelGGL((kda_gdr_decode_kernel<DK, 32, IO>), dim3(grid), dim3(256), 0, st, p); break;
    case 64: hipLaunchKernelGGL((kda_gdr_decode_kernel<DK, 64, IO>), dim3(grid), dim3(256), 0, st, p); break;
    case 128: hipLaunchKernelGGL((kda_gdr_decode_kernel<DK, 128, IO>), dim3(grid), dim3(256), 0, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_gdr_decode(const GdrDecodeParams& p, int Dk, int Dv, bool fp32, hipStream_t st) {
  if (p.N == 0) return hipSuccess;
  switch (Dk) {
    case 32: return fp32 ? launch_decode_t<32, float>(p, Dv, st) : launch_decode_t<32, __bf16>(p, Dv, st);
    case 64: return fp32 ? launch_decode_t<64, float>(p, Dv, st) : launch_decode_t<64, __bf16>(p, Dv, st);
    case 128: return fp32 ? launch_decode_t<128, float>(p, Dv, st) : launch_decode_t<128, __bf16>(p, Dv, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
