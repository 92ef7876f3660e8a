// Launches of the state walk (kda_gdr_walk.h) and the composition of its segments.
#include "kda_gdr_walk.h"

namespace kda {

template <int DK, int WV, int NV, typename IO>
__global__ __launch_bounds__(64 * WV) void kda_gdr_walk_kernel(GdrWalkParams p, int Dv) {
  __shared__ __attribute__((aligned(16))) char lds[2 * GdrWalkLds<DK, WV, NV, IO, true>::BYTES];
  gdr_walk<DK, WV, NV, IO, true, false>(p, Dv, blockIdx.x, lds);
}

// The maps of a split walk in one launch: its first `half` workgroups walk for N, the
// others for M (1000 float32 tokens of 8 heads, where each is a few workgroups: 52 us a
// call with a launch each, 42 so).
template <int DK, int WV, int NV, typename IO>
__global__ __launch_bounds__(64 * WV) void kda_gdr_maps_kernel(GdrWalkParams p, int Dv, int half, int walks_m) {
  __shared__ __attribute__((aligned(16))) char lds[2 * GdrWalkLds<DK, WV, NV, IO, false>::BYTES];
  const bool second = (int)blockIdx.x >= half;
  p.pass = second ? 2 : 1;
  if (second) p.walks = walks_m;
  gdr_walk<DK, WV, NV, IO, false, false>(p, second ? DK : Dv, (int)blockIdx.x - (second ? half : 0), lds);
}

// Composes the segments' starts: start_{s+1} = M_s start_s + N_s, in place in
// p.starts from s = 1 on; REV: the gradients at their ends, end_{s-1} = M_s^T end_s +
// N'_s, from the last segment but one down.  One workgroup per (walk, 16 value columns): a wave owns 16
// rows, the start goes round through LDS.  M and the start are split into three bf16
// terms each (float32 accuracy, 6 products).  Bound by the chain of steps: reading M
// is kept a step ahead, splitting it spread over as many waves as there are row tiles
// (19 steps of 12 heads, D = 128: 48-55 us; with 4 waves and no reads ahead 70 us).
template <int DK, bool REV>
__global__ __launch_bounds__(4 * DK) void kda_gdr_compose_kernel(GdrWalkParams p, int Dv) {
  constexpr int NU = DK / 32, LS = DK + 4;
  __shared__ __attribute__((aligned(16))) float st[2][16 * LS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g4 = lane >> 4;
  const int bh = blockIdx.x / (Dv / 16), v0 = blockIdx.x % (Dv / 16) * 16;
  int nseg = p.nseg;
  size_t idx = (size_t)bh * nseg;
  if (p.segstart != nullptr) {
    const int b = bh / p.s.Hv, s0 = uniform(p.segstart[b]);
    nseg = uniform(p.segstart[b + 1]) - s0;
    idx = (size_t)(bh % p.s.Hv) * p.nseg + s0;
    if (nseg == 0)  // a sequence without tokens has no segment to hand its state on
      for (int i = tid; i < 16 * DK; i += 4 * DK) {
        const size_t at = ((size_t)bh * DK + (i >> 4)) * Dv + v0 + (i & 15);
        p.S_T[at] = p.S0 != nullptr ? p.S0[at] : 0.f;
      }
  }
  if (nseg < 3) return;  // uniform: the second segment's start is there
  float* starts = p.starts + idx * DK * Dv + v0;
  const float* maps = p.maps + idx * DK * DK;

  auto terms = [](const float* x, bf16x8 (&t)[3]) {
    Terms<__bf16, 3> y;
    const f32x4 z[2] = {f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}};
    y.set(z);
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] = y.t[k];
  };
  const int row0 = 16 * wave;
  struct Rows {  // this wave's rows of M_s and N_s
    float m[NU][8];
    f32x4 n;
  };
  constexpr int D = REV ? -1 : 1;
  const int first = REV ? nseg - 2 : 1;
  auto fetch = [&](int i, Rows& x) {  // of step i (past the last: of the last)
    const int s = first + D * (i < nseg - 2 ? i : nseg - 3);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if constexpr (REV) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x.m[u][e] = maps[((size_t)s * DK + 32 * u + 8 * g4 + e) * DK + row0 + r];
      } else {
        load8(maps + ((size_t)s * DK + row0 + r) * DK + 32 * u + 8 * g4, x.m[u]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x.n[e] = starts[((size_t)(s + D) * DK + row0 + 4 * g4 + e) * Dv + r];
  };
  auto step = [&](int i, const Rows& x) {
    const int s = first + D * i;
    const float* in = st[s & 1];
    f32x4 acc = x.n;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      float y[8];
      load8(in + r * LS + 32 * u + 8 * g4, y);
      bf16x8 a[3], b[3];
      terms(y, b);
      terms(x.m[u], a);
#pragma unroll
      for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int k = 0; k + j < 3; ++k) gmma(acc, a[j], b[k]);
    }
    *reinterpret_cast<f32x4*>(&st[(s + 1) & 1][r * LS + row0 + 4 * g4]) = acc;
#pragma unroll
    for (int e = 0; e < 4; ++e) starts[((size_t)(s + D) * DK + row0 + 4 * g4 + e) * Dv + r] = acc[e];
  };
  // the state the chain begins with, column by column
  for (int i = tid; i < 16 * DK; i += 4 * DK)
    st[first & 1][(i & 15) * LS + (i >> 4)] = starts[((size_t)first * DK + (i >> 4)) * Dv + (i & 15)];
  const int steps = nseg - 2;
  Rows x, y;  // of this step and the next, whose reads are under way meanwhile
  fetch(0, x);
  lds_barrier();
  for (int i = 0; i < steps; i += 2) {
    fetch(i + 1, y);
    step(i, x);
    lds_barrier();
    if (i + 1 == steps) break;  // uniform
    fetch(i + 2, x);
    step(i + 1, y);
    lds_barrier();
  }
}

template <int DK, int WV, int NV, typename IO>
static hipError_t launch_pass(const GdrWalkParams& p, int Dv, hipStream_t st) {
  const dim3 grid((unsigned)gdr_walk_grid(p.walks, p.s.Hv / p.s.Hk, Dv / (16 * NV * WV))), block(64 * WV);
  if (grid.x == 0) return hipSuccess;
  hipLaunchKernelGGL((kda_gdr_walk_kernel<DK, WV, NV, IO>), grid, block, 0, st, p, Dv);
  return hipGetLastError();
}

// the walks of a pass: all, or all segments that need the map
static int pass_walks(const GdrWalkParams& p, int pass) {
  if (p.nseg <= 1) return p.s.NS * p.s.Hv;
  if (p.s.seqs.bounds != nullptr) return p.nseg * p.s.Hv;
  return p.s.NS * p.s.Hv * (p.nseg - pass);
}

template <int DK, int WV, int NV, typename IO>
static hipError_t launch_maps_t(const GdrWalkParams& p, int Dv, bool n, bool m, hipStream_t st) {
  const int share = p.s.Hv / p.s.Hk, walks_m = pass_walks(p, 2);
  const size_t half = n ? gdr_walk_grid(p.walks, share, Dv / (16 * NV * WV)) : 0;
  const size_t rest = m ? gdr_walk_grid(walks_m, share, DK / (16 * NV * WV)) : 0;
  hipLaunchKernelGGL((kda_gdr_maps_kernel<DK, WV, NV, IO>), dim3((unsigned)(half + rest)), dim3(64 * WV), 0, st, p, Dv,
                     (int)half, walks_m);
  return hipGetLastError();
}

// waves of a workgroup for `cols` value columns
template <typename IO> static int map_waves(const GdrWalkParams& p, int cols) {
  if (cols == 32) return 2;
  return sizeof(IO) == 2 && gdr_whole_head(pass_walks(p, 0), cols) ? 8 : 4;
}

template <int DK, typename IO>
static hipError_t launch_maps_d(const GdrWalkParams& all, int Dv, hipStream_t st) {
  GdrWalkParams p = all;
  p.walk0 = 0;
  p.walks = pass_walks(p, 1);
  const int wn = map_waves<IO>(p, Dv), wm = map_waves<IO>(p, DK);
  // together, or each with its own shape
  for (int wv : {2, 4, 8}) {
    const bool n = wn == wv, m = wm == wv;
    if (!n && !m) continue;
    hipError_t e;
    if (wv == 2) e = launch_maps_t<DK, 2, 1, IO>(p, Dv, n, m, st);
    else if (wv == 4) e = launch_maps_t<DK, 4, 1, IO>(p, Dv, n, m, st);
    else e = launch_maps_t<DK, sizeof(IO) == 2 ? 8 : 4, 1, IO>(p, Dv, n, m, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DK, typename IO>
static hipError_t launch_walk_d(const GdrWalkParams& all, int Dv, hipStream_t st) {
  GdrWalkParams p = all;
  p.walk0 = 0;
  p.walks = pass_walks(p, 0);
  if (Dv == 32) return launch_pass<DK, 2, 1, IO>(p, Dv, st);
  if constexpr (sizeof(IO) == 2)
    if (gdr_whole_head(p.walks, Dv)) {
      GdrWalkParams whole = p;
      const int rest = p.nseg > 1 || p.s.seqs.bounds != nullptr ? 0 : gdr_last_walks(p.walks);
      whole.walks -= rest;
      if (hipError_t e = launch_pass<DK, 8, 1, IO>(whole, Dv, st); e != hipSuccess || rest == 0) return e;
      whole.walk0 = whole.walks;
      whole.walks = rest;
      return launch_pass<DK, 4, 1, IO>(whole, Dv, st);
    }
  return launch_pass<DK, 4, 1, IO>(p, Dv, st);
}

template <typename IO>
static hipError_t launch_walk(const GdrWalkParams& p, int Dk, int Dv, hipStream_t st) {
  switch (Dk) {
    case 32: return launch_walk_d<32, IO>(p, Dv, st);
    case 64: return launch_walk_d<64, IO>(p, Dv, st);
    case 128: return launch_walk_d<128, IO>(p, Dv, st);
  }
  return hipErrorInvalidValue;
}

static hipError_t walk(const GdrWalkParams& p, int Dk, int cols, bool fp32, hipStream_t st) {
  return fp32 ? launch_walk<float>(p, Dk, cols, st) : launch_walk<__bf16>(p, Dk, cols, st);
}

template <bool REV> static hipError_t launch_compose(const GdrWalkParams& p, int Dk, int Dv, hipStream_t st) {
  const dim3 grid((unsigned)((size_t)p.s.NS * p.s.Hv * (Dv / 16)));
  switch (Dk) {
    case 32: hipLaunchKernelGGL((kda_gdr_compose_kernel<32, REV>), grid, dim3(128), 0, st, p, Dv); break;
    case 64: hipLaunchKernelGGL((kda_gdr_compose_kernel<64, REV>), grid, dim3(256), 0, st, p, Dv); break;
    case 128: hipLaunchKernelGGL((kda_gdr_compose_kernel<128, REV>), grid, dim3(512), 0, st, p, Dv); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}
hipError_t launch_gdr_compose(const GdrWalkParams& p, int Dk, int Dv, bool reverse, hipStream_t st) {
  return reverse ? launch_compose<true>(p, Dk, Dv, st) : launch_compose<false>(p, Dk, Dv, st);
}

// the segments' maps, and their starts from them
hipError_t launch_gdr_maps(const GdrWalkParams& p, int Dk, int Dv, bool fp32, hipStream_t st) {
  hipError_t e = hipErrorInvalidValue;
  switch (Dk) {
    case 32: e = fp32 ? launch_maps_d<32, float>(p, Dv, st) : launch_maps_d<32, __bf16>(p, Dv, st); break;
    case 64: e = fp32 ? launch_maps_d<64, float>(p, Dv, st) : launch_maps_d<64, __bf16>(p, Dv, st); break;
    case 128: e = fp32 ? launch_maps_d<128, float>(p, Dv, st) : launch_maps_d<128, __bf16>(p, Dv, st); break;
  }
  if (e != hipSuccess) return e;
  return launch_gdr_compose(p, Dk, Dv, false, st);
}

hipError_t launch_gdr_walk(const GdrWalkParams& p, int Dk, int Dv, bool fp32, hipStream_t st) {
  if (p.nseg > 1)
    if (hipError_t e = launch_gdr_maps(p, Dk, Dv, fp32, st); e != hipSuccess) return e;
  return walk(p, Dk, Dv, fp32, st);
}

}  // namespace kda
