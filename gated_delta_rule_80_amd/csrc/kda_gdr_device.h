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
// Unit u of N tiles from tile t0 on (t0 even, N = 2 or 4) of the columns of a bf16
// image: the transposing reads with their wait in one block, because the compiler has
// a transposing read that it can see wait for every global-to-LDS copy in flight, the
// next chunk's included.
__device__ __forceinline__ bf16x8 join4(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int K>
__device__ __forceinline__ void g_colp_tiles(const __bf16* img, int u, int t0, int r, int g, bf16x8 (&f)[2]) {
  typedef __attribute__((address_space(3))) const __bf16 lds_bf16;
  const int row = 32 * u + 8 * g + (r >> 2), c = 16 * t0 + 8 * (r & 3);
  const uint32_t a0 = (uint32_t)(uintptr_t)(lds_bf16*)(img + GImg<__bf16, K>::at(row, c));
  bf16x4 x0, x1, x2, x3;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4\n\t"
      "ds_read_b64_tr_b16 %1, %4 offset:%5\n\t"
      "ds_read_b64_tr_b16 %2, %4 offset:8\n\t"
      "ds_read_b64_tr_b16 %3, %4 offset:%6\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x0), "=&v"(x1), "=&v"(x2), "=&v"(x3)
      : "v"(a0), "n"(4 * K * 2), "n"(4 * K * 2 + 8));
  f[0] = join4(x0, x1);
  f[1] = join4(x2, x3);
}
template <int K>
__device__ __forceinline__ void g_colp_tiles(const __bf16* img, int u, int t0, int r, int g, bf16x8 (&f)[4]) {
  typedef __attribute__((address_space(3))) const __bf16 lds_bf16;
  const int row = 32 * u + 8 * g + (r >> 2), c = 16 * t0 + 8 * (r & 3);
  const uint32_t a0 = (uint32_t)(uintptr_t)(lds_bf16*)(img + GImg<__bf16, K>::at(row, c));
  const uint32_t a1 = (uint32_t)(uintptr_t)(lds_bf16*)(img + GImg<__bf16, K>::at(row, c + 32));
  bf16x4 x0, x1, x2, x3, y0, y1, y2, y3;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%10\n\t"
      "ds_read_b64_tr_b16 %2, %8 offset:8\n\t"
      "ds_read_b64_tr_b16 %3, %8 offset:%11\n\t"
      "ds_read_b64_tr_b16 %4, %9\n\t"
      "ds_read_b64_tr_b16 %5, %9 offset:%10\n\t"
      "ds_read_b64_tr_b16 %6, %9 offset:8\n\t"
      "ds_read_b64_tr_b16 %7, %9 offset:%11\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x0), "=&v"(x1), "=&v"(x2), "=&v"(x3), "=&v"(y0), "=&v"(y1), "=&v"(y2), "=&v"(y3)
      : "v"(a0), "v"(a1), "n"(4 * K * 2), "n"(4 * K * 2 + 8));
  f[0] = join4(x0, x1);
  f[1] = join4(x2, x3);
  f[2] = join4(y0, y1);
  f[3] = join4(y2, y3);
}
template <int K, int N>
__device__ __forceinline__ void g_colp_tiles(const float* img, int u, int t0, int r, int g, f32x4 (&f)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t) f[t] = g_colp<K>(img, u, t0 + t, r, g);
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

// The same kept as read until it is used.
template <typename E> struct AccRaw;
template <> struct AccRaw<__bf16> {
  bf16x4 v;
  template <int K> __device__ __forceinline__ void load(const __bf16* img, int tile, int m0, int r, int g) {
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (lds_bf16x4*)(img + GImg<__bf16, K>::at(GOp<__bf16>::row4(tile, g) + (r >> 2), m0 + 4 * (r & 3))));
  }
  __device__ __forceinline__ float operator[](int e) const { return (float)v[e]; }
};
template <> struct AccRaw<float> {
  f32x4 v;
  template <int K> __device__ __forceinline__ void load(const float* img, int tile, int m0, int r, int g) {
    v = g_acc<K>(img, tile, m0, r, g);
  }
  __device__ __forceinline__ float operator[](int e) const { return v[e]; }
};

// NT terms of one unit of a float32 quantity held in accumulators.
template <typename E, int NT> struct Terms;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// x - h[0] and x - h[1] as one instruction each (a two-element dot product with -1
// and 0; exact, as the rest of a rounding is representable).  The factors are kept in
// a register: as an inline constant -1.0 the instruction takes the other half.
__device__ __forceinline__ uint32_t pair_factor(uint32_t bits) {
  asm("" : "+s"(bits));
  return bits;
}
__device__ __forceinline__ float minus_low(bf16x2 h, float x) {
  return __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, pair_factor(0x0000bf80u)), x, false);
}
__device__ __forceinline__ float minus_high(bf16x2 h, float x) {
  return __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, pair_factor(0xbf800000u)), x, false);
}
template <int NT> struct Terms<__bf16, NT> {
  static constexpr int N = NT;
  bf16x8 t[NT];
  __device__ __forceinline__ void set(const f32x4* tiles) {  // tiles of the unit
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // pairs: one conversion instruction each
      f32x2 x = {tiles[q >> 1][2 * (q & 1)], tiles[q >> 1][2 * (q & 1) + 1]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bf16x2 h = __builtin_convertvector(x, bf16x2);
        t[n][2 * q] = h[0];
        t[n][2 * q + 1] = h[1];
        if (n + 1 < NT) {
          x[0] = minus_low(h, x[0]);
          x[1] = minus_high(h, x[1]);
        }
      }
    }
  }
};
template <int NT> struct Terms<float, NT> {
  static constexpr int N = 1;
  f32x4 t[1];
  __device__ __forceinline__ void set(const f32x4* tiles) { t[0] = tiles[0]; }
};

// Position of (token tile t, unit u) in the list of a triangle's fragments, tile by
// tile: units u <= t / TPU of each tile (lower), or u >= t / TPU (the transpose).
template <int TPU, int NU, bool UPPER> __host__ __device__ constexpr int tri_at(int t, int u) {
  int i = 0;
  for (int s = 0; s < NU * TPU; ++s)
    if (s < t) i += UPPER ? NU - s / TPU : s / TPU + 1;
  return i + (UPPER ? u - t / TPU : u);
}
// Offset in elements of element (i, j) of the matrix (j's fragment slot may be
// written in parts), term k of `terms`.
template <typename E, int NU, bool UPPER>
__device__ __forceinline__ int tri_slot(int i, int j, int k, int terms) {
  constexpr int KU = GOp<E>::KU, TPU = GOp<E>::TPU;
  const int t = KU == 32 ? 2 * (i >> 5) + ((i >> 2) & 1) : i >> 4;
  const int r = KU == 32 ? 4 * ((i >> 3) & 3) + (i & 3) : i & 15;
  const int u = j / KU, g = j % KU / (KU / 4), e = j % (KU / 4);
  return ((tri_at<TPU, NU, UPPER>(t, u) * terms + k) * 64 + r + 16 * g) * (KU / 4) + e;
}
// This lane's fragment f of a list in LDS.
template <typename E>
__device__ __forceinline__ typename GOp<E>::Frag g_frag(const E* list, int f, int lane) {
  return *reinterpret_cast<const typename GOp<E>::Frag*>(list + (f * 64 + lane) * (16 / (int)sizeof(E)));
}

// 2^x by the hardware instruction (1 ulp; results below 2^-126 are 0, and so is the
// decay they stand for to any use)
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A 4 x 4 transpose inside every quad of lanes: x[e] of lane j goes to element j of
// lane e, rounded to bf16.  Lane q of a quad then holds row q of the tile's 4 rows
// over 4 consecutive columns: one 8-byte store instead of four of 2 bytes.
__device__ __forceinline__ uint2 quad_transpose(const f32x4& x, int r) {
  const bf16x2 a = __builtin_convertvector((f32x2){x[0], x[1]}, bf16x2);
  const bf16x2 b = __builtin_convertvector((f32x2){x[2], x[3]}, bf16x2);
  const uint32_t d0 = __builtin_bit_cast(uint32_t, a), d1 = __builtin_bit_cast(uint32_t, b);
  const uint32_t o0 = (uint32_t)__builtin_amdgcn_mov_dpp((int)d0, 0xB1, 0xF, 0xF, false);  // lane ^ 1
  const uint32_t o1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)d1, 0xB1, 0xF, 0xF, false);
  // bytes 0-3 are the second argument's, 4-7 the first's: an even lane takes both
  // low halves (own first), an odd lane both high halves (own second)
  const uint32_t sel = (r & 1) ? 0x03020706u : 0x05040100u;
  const uint32_t p0 = __builtin_amdgcn_perm(o0, d0, sel), p1 = __builtin_amdgcn_perm(o1, d1, sel);
  const bool up = (r & 2) != 0;
  const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)(up ? p0 : p1), 0x4E, 0xF, 0xF, false);  // lane ^ 2
  return make_uint2(up ? got : p0, up ? p1 : got);
}

// Stores through a range-checked buffer (rows behind a sequence's end lie behind the
// range and are dropped): no branch, and every chunk issues the same number of them.
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
// One accumulator tile of a [row][16 columns] block, rows `ld` bytes apart: rows
// row0 .. + 3 of column col0 + r (row0 of this lane group), col0 in bytes.
__device__ __forceinline__ void store_tile(const BufRes& b, int row0, int ld, int col0, const f32x4& x, int r,
                                           __bf16) {
  const uint2 y = quad_transpose(x, r);
  __builtin_amdgcn_raw_buffer_store_b64((u32x2){y.x, y.y}, b, (row0 + (r & 3)) * ld + col0 + 8 * (r >> 2), 0, 0);
}
__device__ __forceinline__ void store_tile(const BufRes& b, int row0, int ld, int col0, const f32x4& x, int r,
                                           float) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, (float)x[e]), b, (row0 + e) * ld + col0 + 4 * r,
                                          0, 0);
}
// 4 consecutive elements at byte offset `at`
__device__ __forceinline__ void store_four(const BufRes& b, int at, const f32x4& x, __bf16) {
  const bf16x2 lo = __builtin_convertvector((f32x2){x[0], x[1]}, bf16x2);
  const bf16x2 hi = __builtin_convertvector((f32x2){x[2], x[3]}, bf16x2);
  __builtin_amdgcn_raw_buffer_store_b64((u32x2){__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)},
                                        b, at, 0, 0);
}
__device__ __forceinline__ void store_four(const BufRes& b, int at, const f32x4& x, float) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, at, 0, 0);
}

// Values that are the same in every lane, moved to scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long uniform(long x) {
  const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)x);
  const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)((unsigned long)x >> 32));
  return (long)(((unsigned long)hi << 32) | lo);
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
    x.tok0 = uniform(s.seqs.bounds[b]);
    x.Tq = uniform(s.seqs.bounds[b + 1]) - (int)x.tok0;
    int c0 = uniform(s.seqs.cstart[b]);
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

// Copies ROWS rows of K elements (16-byte pieces permuted as GImg says) from global
// memory into an LDS image, NT threads.  A thread's offsets from the first row do
// not change from chunk to chunk (32 bits: the host bounds the stride), so a whole
// chunk costs one load instruction per piece; in a chunk with fewer rows those
// past the last one read the last one.
template <int NT, int ROWS, int K, typename IO>
struct GdrCopy {
  using I = GImg<IO, K>;
  static constexpr int N = ROWS * I::RC, ITERS = (N + NT - 1) / NT;
  uint32_t off[ITERS];
  __device__ __forceinline__ static uint32_t offset(int it, uint32_t stride, int last) {
    int row, c;
    I::source(it * NT + (int)threadIdx.x, row, c);
    return (uint32_t)(row < last ? row : last) * stride + (uint32_t)c * 16;
  }
  __device__ __forceinline__ void init(long stride) {
#pragma unroll
    for (int it = 0; it < ITERS; ++it) off[it] = offset(it, (uint32_t)(stride * (long)sizeof(IO)), ROWS - 1);
  }
  // img, base and wave are the same in every lane
  __device__ __forceinline__ static void load(char* img, int it, const char* base, uint32_t o, int wave) {
    if (N % NT == 0 || it * NT + (int)threadIdx.x < N)
      __builtin_amdgcn_global_load_lds((const glb_void_t*)(base + o),
                                       (lds_void_t*)(img + (size_t)(it * NT + 64 * wave) * 16), 16, 0, 0);
  }
  __device__ __forceinline__ void whole(char* img, const IO* base, int wave) const {
#pragma unroll
    for (int it = 0; it < ITERS; ++it) load(img, it, reinterpret_cast<const char*>(base), off[it], wave);
  }
  __device__ __forceinline__ static void part(char* img, const IO* base, long stride, int last, int wave) {
#pragma unroll
    for (int it = 0; it < ITERS; ++it)
      load(img, it, reinterpret_cast<const char*>(base), offset(it, (uint32_t)(stride * (long)sizeof(IO)), last),
           wave);
  }
};
// BYTES consecutive bytes
template <int NT, int BYTES>
__device__ __forceinline__ void gdr_copy_flat(char* img, const char* base, int wave) {
  constexpr int N = BYTES / 16;
#pragma unroll
  for (int it = 0; it < (N + NT - 1) / NT; ++it) {
    const uint32_t idx = it * NT + threadIdx.x;
    if (N % NT == 0 || idx < (uint32_t)N)
      __builtin_amdgcn_global_load_lds((const glb_void_t*)(base + idx * 16u),
                                       (lds_void_t*)(img + (size_t)(it * NT + 64 * wave) * 16), 16, 0, 0);
  }
}

// this workgroup's walk of `count` (sequence, value head) and its value block; false: none.
// The heads that share q, k rows (`share` of them) and their value blocks run on one
// XCD, whose L2 serves their common rows; the groups go round the XCDs, so that a
// long sequence's heads and a short one's are spread evenly (packed prompts of 0 to
// 1024 tokens, 32 heads: 122 us with the walks listed XCD by XCD, 81 us as here).
__device__ __forceinline__ bool gdr_walk_id(int blk, int nv, int share, int count, int& bh, int& vblk) {
  share = gdr_walk_group(count, share);
  const int x = blk & 7, i = blk >> 3, unit = share * nv;
  const int member = i % unit;
  bh = (i / unit * 8 + x) * share + member / nv;
  vblk = member % nv;
  return bh < count;
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
