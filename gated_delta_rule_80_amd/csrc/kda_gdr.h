// The gated delta rule with one decay per head: workspace layout and parameter
// blocks shared by the host runtime (plain C++) and the kernels.
//
// Per value head (query/key head = value head / (Hv / Hk)) and chunk of C tokens,
// with G_i the cumulative log-decay inside the chunk, gamma_i = e^{G_i},
// lambda_i = e^{G_C - G_i}, D_ij = e^{G_i - G_j} (j <= i; every exponent <= 0, so
// no factoring is needed as it is for a decay per channel), k^, q^ the
// normalised rows (or the rows as given) and b = beta:
//   a_ij = D_ij (k^_i . k^_j) b_j   (j < i)        Tm = (I + a)^-1
//   p_ij = scale D_ij (q^_i . k^_j) b_j  (j <= i)
//   Y = Tm (V - gamma K^ S)         the part of each v that S does not hold yet
//   O = scale gamma Q^ S + p Y      S' = gamma_C S + (b lambda K^)^T Y
// Every scale is one number per token, so it multiplies accumulator rows and the
// matrix operands stay the raw q, k, v of the caller.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "kda_layout.h"

namespace kda {

// Tokens per chunk: the deepest whose two images of q, k, v and of the chunk's
// matrices fit LDS together (bf16 64, float32 32).
constexpr int gdr_chunk(bool fp32) { return fp32 ? 32 : 64; }

// One record per (sequence, value head, chunk), element type E.  A matrix is kept as
// the matrix-core operands the walks read, in their order: one fragment of 64 lanes x
// 16 bytes per (token tile, contraction unit) of its triangle (kda_gdr_device.h), so
// that a workgroup copies it to LDS as it stands and a lane's reads are consecutive.
//   Tm   [6 | 3][TT]  fragments in TT terms: bf16 keeps Tm as hi + lo (16 bits of
//                    mantissa), float32 as it is
//   sc   [8][C]      float32, per token: cx = gamma rk, cy = b lambda rk,
//                    co = scale gamma rq, rk, rq, G in log2 units (high part, low
//                    part), b; rows behind the sequence's end hold zeros in cx,
//                    cy, co, rk, rq, b
//   P    [6 | 3]     forward: one term (its products end in the output)
// or, for the backward (whose dS0 leaves in float32),
//   P^T, Tm^T [6 | 3][TT]
// where rk, rq are 1 / norm (1 without the normalisation).
struct GdrRecord {
  size_t t, sc, p, tt;  // byte offsets
  size_t bytes;         // 256-byte multiple
};
constexpr int kGdrScalars = 8;
// fragments of a triangle: bf16 4 token tiles x 2 units of 2 tiles, float32 2 x 2
constexpr int gdr_frags(bool fp32) { return fp32 ? 3 : 6; }

constexpr GdrRecord gdr_record(bool fp32, bool bwd) {
  const size_t C = (size_t)gdr_chunk(fp32), terms = fp32 ? 1 : 2;
  const size_t mat = (size_t)gdr_frags(fp32) * 1024;
  GdrRecord r{};
  r.t = 0;
  r.sc = terms * mat;
  r.p = r.sc + kGdrScalars * C * 4;
  r.tt = r.p + (bwd ? terms : 1) * mat;
  r.bytes = round_up(r.tt + (bwd ? terms * mat : 0), 256);
  return r;
}

// Where the rows of a call stand: B equal-length sequences, or packed ones with
// their tables in the workspace.  Records are chunk-major (rec_slot).
struct GdrShape {
  int B, T, Hk, Hv;  // B: rows of tokens (packed: 1)
  int NS;            // sequences
  int NT;            // chunk slots per (sequence, head); packed: per head
  long qs, ks, vs;   // elements between tokens of q, k, v
  SeqTables seqs;    // bounds NULL: equal lengths
};

// The split of B equal-length rows of nch chunks: segments per walk and their length.
// It triples the work of a chunk (two maps, then the outputs) for nseg times the
// parallelism, so it pays from 6 segments on, while workgroups stay within the 256
// CUs; segments of at least 4 chunks keep the composition (about 1 us a segment)
// below the walks.  Measured at 64k tokens, 12 heads, D = 128, bf16 (the whole call):
// 0.79 ms in 21 segments, 2.88 ms unsplit.  The backward does more beside its walks (three
// maps and two compositions) and fills the card with both of them sooner: it splits where
// the CUs leave room for 8 segments (64k tokens, 12 heads: 2.22 against 4.65 ms; 32 heads,
// 8 segments: 0.72 against 0.79 ms at 8192 tokens, 0.45 against 0.43 at 4096; 40 heads in 6
// segments would take 0.39 against 0.33 ms at 3000).
struct GdrSplit {
  int nseg, seg_len;
};
constexpr GdrSplit gdr_split(long walks, int nch, int Dv, bool fp32, bool bwd) {
  const long vb = Dv >= 128 && !fp32 ? 128 : (Dv >= 64 ? 64 : 32);
  long P = 256 / (walks * (Dv / vb) > 0 ? walks * (Dv / vb) : 1);
  if (bwd && P < 8) return {1, nch};
  if (nch / 4 < P) P = nch / 4;
  if (P > 64) P = 64;
  if (P < 6) return {1, nch};
  const int len = (int)((nch + P - 1) / P);
  return {(nch + len - 1) / len, len};
}

// Packed rows, whose lengths the host does not know: segments of a length that fills the
// CUs once, where the mean sequence has at least 6 of them.  {most segments, length}.
// Whole calls, bf16, D = 128, split and unsplit: 8000 tokens, 8 heads 174 and 363 us; four
// prompts of 4096, 8 heads 183 and 213 us; 20000 tokens, 32 heads 650 and 990 us.
constexpr GdrSplit gdr_split_packed(long tokens, int C, long n_seqs, long Hv, int Dv, bool fp32) {
  const long vb = Dv >= 128 && !fp32 ? 128 : (Dv >= 64 ? 64 : 32);
  const long nch = (tokens + C - 1) / C;
  long len = (nch * Hv * (Dv / vb) + 255) / 256;
  if (len < 4) len = 4;
  if (nch < 6 * len * n_seqs) return {1, (int)nch};
  return {(int)(tokens / (C * len) + n_seqs), (int)len};
}

// Whether a walk's workgroup takes 128 value columns (8 waves) or 64 (4 waves) with
// bf16 inputs; LDS holds one workgroup of either.  A chunk takes 5.2 and 3.3 us
// (kda_gdr_walk.h): up to 128 walks the halves find a CU each and are the faster, more
// walks' halves take two turns, 6.6 us.
constexpr bool gdr_whole_head(long walks, int Dv) { return Dv % 128 == 0 && walks > 128; }
// Of walks of one length, those that would occupy at most half of the CUs at the end,
// each a whole head: they are taken in halves of a head, on up to twice the CUs (384
// walks of 128 chunks: 1280 us as two turns of whole heads, 1090 us so).
constexpr int gdr_last_walks(long walks) { return walks > 256 && walks % 256 <= 128 ? (int)(walks % 256) : 0; }

// Of `share` walks with common q, k rows, how many stay together: all while there are
// four groups an XCD, fewer where a group would leave other XCDs idle (64 heads on one key
// head are a single group).
constexpr int gdr_walk_group(long count, int share) {
  while (share > 1 && (count + share - 1) / share < 32) share = (share + 1) / 2;
  return share;
}
// Workgroups of `count` walks in nv value blocks: whole groups, eight at a time
// (gdr_walk_id).
constexpr size_t gdr_walk_grid(long count, int share, int nv) {
  share = gdr_walk_group(count, share);
  return (size_t)((count + share - 1) / share + 7) / 8 * 8 * share * nv;
}

struct GdrPrepParams {
  GdrShape s;
  const void* q;
  const void* k;
  const void* g;
  const void* beta;
  const float* A_log;
  const float* dt_bias;
  int beta_logits, l2;
  float eps, scale;
  char* rec;
};

struct GdrWalkParams {
  GdrShape s;
  const void* q;
  const void* k;
  const void* v;
  const char* rec;
  const float* S0;  // NULL: zeros; may equal S_T
  float* S_T;       // NULL: not written
  void* o;          // NULL: no output
  // for the backward: Y [B][T][Hv][Dv] and the state at each chunk's start,
  // [record][Dv / 16][Dk][16], both in the element type; NULL otherwise
  void* y;
  void* ckpt;
  // split walk (nseg > 1; equal lengths): segments of seg_len chunks walk in
  // parallel.  The state after a run of chunks is affine in the state before it,
  // S_end = M S_start + N, so first every segment but the last is walked from zero
  // (the first from S0) for its N and with V = 0 from I for its M, then the starts
  // are composed in order, then every segment is walked with its output.
  //   starts [B Hv][nseg][Dk][Dv] float32: at index s + 1 first the N of segment s,
  //          then the state at the start of segment s + 1; index 0: S0
  //   maps   [B Hv][nseg][Dk][Dk] float32: M of segments 1 .. nseg - 2
  // Packed: each sequence has its own number of segments, segstart[b + 1] - segstart[b]
  // (device; nseg bounds their total), and [B Hv][nseg] above is [Hv][nseg] with the
  // sequences' segments behind one another.
  int nseg, seg_len;
  const int* segstart;
  float* starts;
  float* maps;
  int pass;  // 0: outputs; 1: N; 2: M
  int bwd;   // the records are the backward's
  int walk0, walks;  // set by the launcher: a launch's share of the walks (or segments)
};

struct GdrReverseParams {
  GdrShape s;
  const void* q;
  const void* k;
  const char* rec;
  const void* dO;     // [B][T][Hv][Dv]
  const float* dS_T;  // NULL: zeros
  float* dS0;         // NULL: not written
  void* dv;           // [B][T][Hv][Dv]
  void* ckpt;         // the gradient of each chunk's end state, layout as above
  // split as the forward walk: dS is affine too, dS_start = M^T dS_end + N' with the M of
  // the state, so every segment but the first is walked for its N' (pass 1, dS_end = 0;
  // the last from dS_T), the ends are composed from the last to the first, and every
  // segment is walked with its outputs (pass 0).
  //   ends [B Hv][nseg][Dk][Dv] float32: at index s - 1 first the N' of segment s, then
  //        the gradient at the end of segment s - 1 (the last index: not used)
  int nseg, seg_len;
  float* ends;
  int pass, walks;    // set by the launcher
};

struct GdrGradParams {
  GdrShape s;
  const void* q;
  const void* k;
  const char* rec;
  const void* dO;
  const void* dv;
  const void* y;
  const void* ckS;
  const void* ckdS;
  void* dq;
  void* dk;
  void* dg;        // io type
  void* dbeta;     // io type
  float* dg32;     // [B][T][Hv] gradient of the decay in float32, with raw projections
  int l2;
  float scale;
  const void* g;      // raw projections, with A_log
  const float* A_log;
  const float* dt_bias;
  int beta_logits;
};

struct GdrGateParams {  // sums over the tokens of one head each
  const void* g;
  const float* A_log;
  const float* dt_bias;
  const float* dg32;   // gradient of the decay
  float* dA_log;       // or NULL
  float* ddt_bias;     // or NULL
  long tokens;
  int Hv;
  SeqTables seqs;      // packed: only tokens [bounds[0], bounds[n_seqs]) count
};

struct GdrDecodeParams {
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  const void* beta;
  const float* A_log;
  const float* dt_bias;
  int beta_logits, l2;
  float eps, scale;
  float* S;
  const int* slots;  // NULL: row i uses slot i
  void* o;
  int N, n_slots, Hk, Hv;
  long qs, ks, vs;   // elements between rows
};

// ------------------------------------------------------------------ pages
struct PagesMoveParams {
  const char* src;
  char* dst;
  size_t src_layer, dst_layer;  // bytes between layers
  size_t page_bytes;
  int layers;
  const int* moves;
  const int* count;
  int cap;                      // most moves there can be
  // table entries to rename after a compaction (NULL: none)
  const int* table;
  int* table_out;
  const int* new_id;
  long n_table;
  int n_pages;
};

}  // namespace kda
