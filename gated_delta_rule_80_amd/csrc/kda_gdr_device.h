// Matrix-core operands of the gated delta rule with one decay per head.
//
// The products of a chunk form a chain (K S -> X -> Tm X -> Y -> K^T Y -> S) whose
// links all keep the same 16 value columns, so one wave carries them through the
// whole chunk without passing anything through LDS: a 16 x 16 accumulator tile
// holds column lane % 16 and 4 consecutive rows per lane, and a matrix operand
// wants row/column lane % 16 and 8 (bf16) or 4 x 1 (float32) values along the
// contraction per lane.  With the rows of the tiles numbered as `perm` says, the
// accumulators of a unit (two tiles for bf16, one for float32) are, lane by lane,
// the next product's operand: the contraction may run in any order as long as
// both operands use the same one.
//
// bf16 products of float32 values: a value is split into bf16 terms (hi, then the
// rest's hi, ...; 8 bits of mantissa each) and the products of the terms are
// summed in the float32 accumulators.  q, k, v, dO are exact in one term.
#pragma once
#include "kda_device.h"
#include "kda_gdr.h"

namespace kda {

template <typename E> struct GOp;

template <> struct GOp<__bf16> {
  using Frag = bf16x8;
  static constexpr int KU = 32;         // contraction values per unit
  static constexpr int TPU = 2;         // accumulator tiles per unit
  // index of row m of tile `tile`
  __device__ __forceinline__ static int perm(int tile, int m) {
    return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3);
  }
  // first index of the 4 consecutive rows lane group g holds of tile `tile`
  __device__ __forceinline__ static int row4(int tile, int g) {
    return 32 * (tile >> 1) + 8 * g + 4 * (tile & 1);
  }
  // position of 16-byte chunk c of row `row` in an LDS image of RC chunks a row:
  // the 16 rows of a permuted tile reach distinct chunks (or RC of them), and so
  // do the 4 rows x 4 chunks of a transposing read
  template <int RC> __device__ __forceinline__ static int swz(int row, int c) {
    if constexpr (RC == 16) return c ^ (((row >> 3) & 3) | ((row & 3) << 2));
    else if constexpr (RC == 8) return c ^ (((row >> 3) & 1) | ((row & 3) << 1));
    else return c ^ (row & (RC - 1));
  }
};

template <> struct GOp<float> {
  using Frag = f32x4;
  static constexpr int KU = 16;
  static constexpr int TPU = 1;
  __device__ __forceinline__ static int perm(int tile, int m) { return 16 * tile + m; }
  __device__ __forceinline__ static int row4(int tile, int g) { return 16 * tile + 4 * g; }
  template <int RC> __device__ __forceinline__ static int swz(int row, int c) {
    return c ^ (row & (RC - 1) & 15);
  }
};

// A row-major LDS image with K elements per row, chunks permuted as GOp::swz says.
template <typename E, int K>
struct GImg {
  static constexpr int EPC = 16 / (int)sizeof(E);
  static constexpr int RC = K / EPC;
  static_assert(RC >= 2 && (RC & (RC - 1)) == 0, "rows hold a power of two of 16-byte chunks");
  __device__ __forceinline__ static int at(int row, int k) {
    return (row * RC + GOp<E>::template swz<RC>(row, k / EPC)) * EPC + k % EPC;
  }
  // source chunk (row, chunk in the row) of the image's 16-byte piece idx
  __device__ __forceinline__ static void source(int idx, int& row, int& c) {
    row = idx / RC;
    c = GOp<E>::template swz<RC>(row, idx % RC);
  }
};

// acc += A B over one unit
__device__ __forceinline__ void gmma(f32x4& acc, const bf16x8& a, const bf16x8& b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void gmma(f32x4& acc, const f32x4& a, const f32x4& b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
}

// Operand of unit u along row `row` of an image (this lane's row).
template <typename E, int K>
__device__ __forceinline__ typename GOp<E>::Frag g_row(const E* img, int row, int u, int g) {
  using I = GImg<E, K>;
  return *reinterpret_cast<const typename GOp<E>::Frag*>(
      img + (row * I::RC + GOp<E>::template swz<I::RC>(row, 4 * u + g)) * I::EPC);
}

// Operand along the rows of an image: contraction unit u over its rows, column
// index `col`.  The transposing LDS read gives lane i of 16 element i % 4 of what
// lane 4 e + i / 4 addressed, so a lane addresses row (its index / 4) and the
// 4-column block of (its index % 4): blocks of a permuted tile or natural ones.
template <int K>
__device__ __forceinline__ bf16x8 g_col_blk(const __bf16* img, int u, int blk, int r, int g) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  using I = GImg<__bf16, K>;
  bf16x8 f;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int row = 32 * u + 8 * g + 4 * hh + (r >> 2);
    const bf16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(img + I::at(row, blk)));
#pragma unroll
    for (int e = 0; e < 4; ++e) f[4 * hh + e] = v[e];
  }
  return f;
}
// columns perm(tile, lane)
template <int K>
__device__ __forceinline__ bf16x8 g_colp(const __bf16* img, int u, int tile, int r, int g) {
  return g_col_blk<K>(img, u, 32 * (tile >> 1) + 8 * (r & 3) + 4 * (tile & 1), r, g);
}
template <int K>
__device__ __forceinline__ f32x4 g_colp(const float* img, int u, int tile, int r, int g) {
  f32x4 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = img[GImg<float, K>::at(16 * u + 4 * g + e, 16 * tile + r)];
  return f;
}
// columns m0 + lane
template <int K>
__device__ __forceinline__ bf16x8 g_col(const __bf16* img, int u, int m0, int r, int g) {
  return g_col_blk<K>(img, u, m0 + 4 * (r & 3), r, g);
}
template <int K>
__device__ __forceinline__ f32x4 g_col(const float* img, int u, int m0, int r, int g) {
  f32x4 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = img[GImg<float, K>::at(16 * u + 4 * g + e, m0 + r)];
  return f;
}

// The 4 rows row4(tile, g) .. + 3 of column m0 + lane of an image, as floats: the
// accumulator's own layout.
template <int K>
__device__ __forceinline__ f32x4 g_acc(const __bf16* img, int tile, int m0, int r, int g) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  const int row = GOp<__bf16>::row4(tile, g) + (r >> 2);
  const bf16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
      (lds_bf16x4*)(img + GImg<__bf16, K>::at(row, m0 + 4 * (r & 3))));
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
template <int K>
__device__ __forceinline__ f32x4 g_acc(const float* img, int tile, int m0, int r, int g) {
  f32x4 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = img[GImg<float, K>::at(16 * tile + 4 * g + e, m0 + r)];
  return f;
}

// NT terms of one unit of a float32 quantity held in accumulators.
template <typename E, int NT> struct Terms;
template <int NT> struct Terms<__bf16, NT> {
  static constexpr int N = NT;
  bf16x8 t[NT];
  __device__ __forceinline__ void set(const f32x4* tiles) {  // tiles of the unit
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[e] = tiles[0][e]; x[4 + e] = tiles[1][e]; }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __bf16 h = (__bf16)x[e];
        t[n][e] = h;
        if (n + 1 < NT) x[e] -= (float)h;
      }
  }
};
template <int NT> struct Terms<float, NT> {
  static constexpr int N = 1;
  f32x4 t[1];
  __device__ __forceinline__ void set(const f32x4* tiles) { t[0] = tiles[0]; }
};

// acc += A B for an operand given in AT terms and one in BT terms: products of
// terms i, j with i + j < max(AT, BT) (the others are below the last kept term).
template <int AT, typename F, typename TB>
__device__ __forceinline__ void gmma_terms(f32x4& acc, const F (&a)[AT], const TB& b) {
  constexpr int LIM = AT > TB::N ? AT : TB::N;
#pragma unroll
  for (int i = 0; i < AT; ++i)
#pragma unroll
    for (int j = 0; j < TB::N; ++j)
      if (i + j < LIM) gmma(acc, a[i], b.t[j]);
}

// One chunk of a walk: where its rows stand and its record.
struct GdrSpan {
  long tok0;    // first token of the sequence
  int Tq;       // its tokens
  int nch;      // its chunks
  size_t rec0, rstride;
};
// sequence b, value head h; every index is clamped to the buffers
__device__ __forceinline__ GdrSpan gdr_span(const GdrShape& s, int b, int h, int C) {
  GdrSpan x;
  if (s.seqs.bounds == nullptr) {
    x.tok0 = (long)b * s.T;
    x.Tq = s.T;
    x.nch = s.NT;
    x.rstride = (size_t)s.B * s.Hv;
    x.rec0 = rec_slot(0, (size_t)b * s.Hv + h, x.rstride);
  } else {
    x.tok0 = s.seqs.bounds[b];
    x.Tq = s.seqs.bounds[b + 1] - s.seqs.bounds[b];
    int c0 = s.seqs.cstart[b];
    c0 = c0 < 0 ? 0 : (c0 > s.NT ? s.NT : c0);
    const int n = (x.Tq + C - 1) / C;
    x.nch = n < s.NT - c0 ? n : s.NT - c0;
    x.rstride = (size_t)s.Hv;
    x.rec0 = rec_slot(c0, h, x.rstride);
  }
  return x;
}
// chunk slot `slot` of row b (packed: slot of the head): its first token, how many
// of its C tokens exist (0: no such chunk) and its record
struct GdrChunk {
  long tok;
  int n;
  size_t rec;
};
__device__ __forceinline__ GdrChunk gdr_chunk_at(const GdrShape& s, int slot, int b, int h, int C) {
  GdrChunk x;
  if (s.seqs.bounds == nullptr) {
    x.tok = (long)b * s.T + (long)slot * C;
    x.n = s.T - slot * C;
    x.rec = rec_slot(slot, (size_t)b * s.Hv + h, (size_t)s.B * s.Hv);
  } else {
    x.n = 0;
    x.tok = 0;
    x.rec = rec_slot(slot, h, s.Hv);
    if (slot < s.seqs.cstart[s.seqs.n_seqs]) {
      const int i = seq_of_slot(s.seqs.cstart, s.seqs.n_seqs, slot);
      const int off = (slot - s.seqs.cstart[i]) * C;
      x.tok = (long)s.seqs.bounds[i] + off;
      x.n = s.seqs.bounds[i + 1] - s.seqs.bounds[i] - off;
    }
  }
  x.n = x.n < 0 ? 0 : (x.n > C ? C : x.n);
  return x;
}

// Copies rows of K elements (16-byte pieces permuted as GImg says) from global
// memory into an LDS image; rows past the last one read the last one.
template <int NT, int ROWS, int K, typename IO>
__device__ __forceinline__ void gdr_copy_rows(char* img, const IO* base, long stride, int last,
                                              int tid) {
  using I = GImg<IO, K>;
  constexpr int N = ROWS * I::RC;
  const int wbase = tid & ~63;
#pragma unroll
  for (int it = 0; it < (N + NT - 1) / NT; ++it) {
    const int idx = it * NT + tid;
    int row, c;
    I::source(idx, row, c);
    row = row < last ? row : last;
    if (N % NT == 0 || idx < N)
      __builtin_amdgcn_global_load_lds((const glb_void_t*)(base + row * stride + c * I::EPC),
                                       (lds_void_t*)(img + (size_t)(it * NT + wbase) * 16), 16, 0, 0);
  }
}
template <int NT, int BYTES>
__device__ __forceinline__ void gdr_copy_flat(char* img, const char* base, int tid) {
  constexpr int N = BYTES / 16;
  const int wbase = tid & ~63;
#pragma unroll
  for (int it = 0; it < (N + NT - 1) / NT; ++it) {
    const int idx = it * NT + tid;
    if (N % NT == 0 || idx < N)
      __builtin_amdgcn_global_load_lds((const glb_void_t*)(base + (size_t)idx * 16),
                                       (lds_void_t*)(img + (size_t)(it * NT + wbase) * 16), 16, 0, 0);
  }
}

// this workgroup's walk: (sequence, value head) and value block, the blocks of a
// walk on one XCD so that they share its q, k rows and records in L2
__device__ __forceinline__ void gdr_walk_id(int nv, int& bh, int& vblk) {
  const int pos = xcd_major(blockIdx.x, gridDim.x);
  vblk = pos % nv;
  bh = pos / nv;
}

// The gates of one token and head: the log-decay (a decay below e^-1000 is 0 in
// any use, and -inf must not meet -inf in a difference; NaN passes) and beta.
template <typename IO>
__device__ __forceinline__ float gdr_decay(const void* g, size_t i, const float* A_log,
                                           const float* dt_bias, int h) {
  float x = to_f32(static_cast<const IO*>(g)[i]);
  if (A_log != nullptr) {
    // softplus with full-precision functions: one value per token and head
    const float z = x + dt_bias[h];
    x = -expf(A_log[h]) * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
  }
  return x < -1000.f ? -1000.f : x;
}
template <typename IO>
__device__ __forceinline__ float gdr_beta(const void* beta, size_t i, int logits) {
  const float b = to_f32(static_cast<const IO*>(beta)[i]);
  return logits ? 1.0f / (1.0f + expf(-b)) : b;
}

}  // namespace kda
