// Sparse attention on the tensor cores (bf16 layers, 64 heads x 512 dims,
// 64-dim rotated tail): "【#3】ds4.c を読み解く" §7 mixed attention; vLLM
// DeepSeek V4 page: shared K = V, inverse RoPE on the output, 128-token window.
//
// A query's rows — the raw window followed by the compressed rows of the
// top-k list (ratio 4) or of the visible range (ratio 128) — are gathered 128
// at a time into shared memory, in eight 64-dim blocks laid out with the
// 128-byte swizzle. Each tile is used twice by the tensor cores, which is
// where K = V pays:
//   S^T = K Q^T    M = 128 rows, N = 64 heads, K = 512   (tile read K-major)
//   O^T += V^T P^T M = 4 x 128 dims, N = 64 heads, K = 128 rows (tile read MN-major)
// S^T (64 columns) and O^T (256 columns) live in TMEM. The softmax thread of a
// row reads its 64 head scores from its TMEM lane and writes its probabilities
// as one 128-byte row of P. The running maximum of each head starts at the
// exact per-head maximum of the query's first tile and is only raised
// (rescaling O and the sums) when a later score exceeds it by 2^8, so later
// tiles need no reduction across rows; the per-head sums come from the tensor
// core (ones x P^T).
//
// Decode: a query's 64 heads are split into two groups of 32, each its own
// set of CTAs over the same rows (S^T then has N = 32; P keeps the 64-column
// layout with the other group's columns zero, so PV and the sums are the
// 64-head MMAs). The tiles of a (query, head group) are spread over a
// thread-block cluster (rank c takes tiles c, c + C, ...). Each CTA writes its
// normalised O and per-head (max, sum) to the workspace straight from TMEM;
// after one cluster barrier, rank c pulls heads [32c/C, 32(c+1)/C) of the
// group from every rank into its freed tile buffer (bulk copies from L2),
// combines them in rank order, rotates the tail back and writes bf16 rows.
// (On this part the L2 round trip moves these bytes faster than distributed
// shared memory does.) Splitting the heads halves each CTA's softmax and
// exchange and doubles the CTAs a small batch puts to work. A (query, head
// group) that fits one CTA (C = 1) and prefill write the output directly from
// registers: lane pairs (dims d, d + 1) swap one value per pair of heads, so
// each thread rotates and stores one head's bf16 pair.
//
// In decode on ratios 0 and 128 the rows of a tile are contiguous (the
// window is the whole 128-slot ring once p >= 127, a compressed tile is 128
// consecutive rows): such a tile is eight TMA boxes issued by one thread
// instead of 8192 16-byte gathers.
//
// Warps 0-3: softmax and output epilogue (TMEM lanes = rows, then dims);
// warps 4-7: gather loaders (cp.async, zero fill for masked rows) and the query
// rotation; warp 8: MMA issue (one thread) and TMEM allocation. Every wait is
// bounded (tc.cuh); a timeout sets the error word and the CTA winds down.
//
// Compressed rows in 4 bits (FP4; fp4rows.cuh) take the same two MMAs per tile, on a
// tile that the loaders convert to bf16 on the way: E2M1 times 2^k is exact in bf16, so
// the scores are those of the values that the rows stand for. What differs:
// - Warps 0-7 softmax (two per 32 TMEM lanes, half the heads each), 8-15 loaders, 16 MMA
//   issue. 544 threads of 96 registers.
// - Loaders read the next tile's records (384 bytes a row) into registers while this
//   tile's MMAs run, and convert and hand over the tile's blocks in pairs as PV frees
//   them; S^T starts on the first pairs meanwhile. About 16 integer and 4 bf16 operations
//   per eight dims.
// - The issuing code is warp-uniform with the thread elected by the instructions: the
//   same loop from a branch on lane 0 took twice the time per MMA.
// - Waits sleep on their barrier (mbar_sleep), and code that all warps run again and
//   again is kept short: the kernel is sensitive to instruction fetch (unrolled loops
//   made the chunk 30% slower).
// - A ratio-4 list is read once, checked for its end and turned into pool rows in
//   shared memory, a query ahead in a chunk. A full window comes by TMA, from the ring or
//   from the chunk, a box per loader warp.
// - A query's reference is its first tile's first row (kRaiseFp4). In a chunk the output
//   is written by softmax and loader warps together between two queries.
// - Any number of heads: groups of 64 (32 in decode of small batches), the last one
//   part-filled with zero queries that are not stored.
// Measured (one GB300): a tile takes 5.7 thousand cycles, of which 2.9 PV and 1.5 the
// rest of S^T; reads and writes of shared memory alone are 4.35 (S^T 192 KiB, PV 192,
// the tile's conversion 128, P and L 32, at 128 bytes a cycle), which is what bounds it;
// a query of a chunk costs another 4 thousand for its change of Q and O. 4096 queries of
// 640 rows x 64 heads: 457 us (bf16 rows 650), 0.40 of the burst bf16 rate; c128a decode,
// 32 sequences of 4,224 rows: 37 us (88); c4a decode, 8 sequences: 12.5 us (13.8), with
// q_ready 12.2 (13.1).
#include <cuda_bf16.h>

#include <atomic>
#include <cstddef>
#include <type_traits>

#include "common.cuh"
#include "fp4rows.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr int kH = 64, kD = 512, kNope = 448, kRows = 128;
constexpr int kQBlk = kH * 128;        // one 64-dim block of Q: 64 heads x 128 B
// Heads per CTA: decode splits a query's 64 heads over two clusters (every
// rank reads the same rows for half the heads); prefill keeps all 64.
template <int NH_>
struct Heads {
  static constexpr int NH = NH_;             // heads of this CTA
  static constexpr int HG = kH / NH;         // head groups per query
  static constexpr int NHF = NH / 32;        // 32-column halves of the S accumulator
  static constexpr int QBLK = NH * 128;      // one 64-dim block of this CTA's Q
};
constexpr int kKBlk = kRows * 128;     // one 64-dim block of the row tile
// Warps: softmax and epilogue, then the loaders, then the MMA issuer. 4-bit rows
// take eight loader warps (they convert every element of a tile) and eight softmax
// warps (two per 32 TMEM lanes, each with half the heads).
template <bool FP4>
struct Warps {
  static constexpr uint32_t NS = FP4 ? 8 : 4;          // softmax warps
  static constexpr uint32_t ST = 32 * NS;              // softmax threads
  static constexpr uint32_t NL = FP4 ? 8 : 4;          // loader warps
  static constexpr uint32_t LT = 32 * NL;              // loader threads
  static constexpr uint32_t MMA = NS + NL;             // the MMA issuer's warp
  static constexpr uint32_t THREADS = 32 * (MMA + 1);  // 288 or 544
};
constexpr int kNhDec = 32;             // heads per CTA in decode
constexpr uint32_t kMaxCluster = 16;   // cluster size; beyond 8 (the portable limit) when the
                                       // device allows non-portable sizes
constexpr float kRaiseLog2 = 8.0f;     // raise the running max beyond 2^8
// 4-bit rows start from the score of one valid row instead of the first tile's maximum
// (any reference gives the same softmax while nothing over- or underflows) and raise it
// beyond 2^60: P, O and L are floating point, so that only the range matters.
constexpr float kRaiseFp4 = 60.0f;
// The maximum of a first tile without a valid row: any later score raises it (O and L
// are zeros until then).
constexpr float kNoMax = -1e30f;

struct TcAttnParams {
  uint32_t ratio, batch, T, pos0, cap_raw, comp_cap, n_comp, top_k;
  RowMap map;         // rows of comp
  const uint32_t *seq_pos;   // [B] per-sequence positions (ragged decode) or NULL
  uint32_t cluster;   // decode: CTAs per query (one cluster); 0: prefill, persistent CTAs
  // decode tiles of contiguous rows by TMA instead of row gathers (ratios 0
  // and 128; 4-bit rows: every ratio): bit 0 the window tile as the whole 128-slot
  // ring, bit 1 (ratio 128) the compressed tiles (the visible rows, the same count for
  // every sequence); bit 2 (4-bit rows, chunk): a window inside the chunk
  uint32_t tma_rows;
  uint32_t n_q;       // queries = batch * T
  float c2;           // softmax scale * log2(e)
  uint32_t q_rotated; // q is rotated already
  uint32_t q_ready;   // q, positions, tables and error word may be read before the wait for the
                      // previous launch (DS4A_Q_READY)
  uint32_t n_heads, hg;   // 4-bit rows: heads of a query (1 .. 128), head groups of a query
  const __nv_bfloat16 *q, *ring, *chunk, *comp;   // (comp: bytes of 4-bit rows where FP4)
  const int32_t *topk;
  const float *cos, *sin;
  __nv_bfloat16 *out;
  // decode, C > 1: each rank's O / L as [n_q][C][64][512] bf16 (4-bit rows: fp32), and
  // its (max, sum) per head as [n_q][C][64][2] fp32
  __nv_bfloat16 *part;
  float *ml;
  int *err;
};

struct Smem {
  uint8_t q[8 * kQBlk];     // 64 KiB
  uint8_t kv[8 * kKBlk];    // 128 KiB; decode merge: afterwards the pulled slices (with p)
  uint8_t p[kRows * 128];   // 16 KiB; direct output: afterwards staging, [64 heads][128] bf16
  uint64_t kv_full, kv_empty[4];   // kv_full: the whole tile landed; kv_empty[m]: blocks 2m, 2m+1 free
  uint64_t q_full, q_empty, s_full, p_full, p_empty, o_full, o_empty, sm_bar;
  uint64_t q_tma;   // the query's eight Q blocks landed (TMA transaction count)
  uint64_t kv_tma;  // a tile loaded by TMA landed
  uint64_t kv_pair[4];   // 4-bit rows: blocks 2m, 2m+1 of the tile are written
  uint64_t mg_bar;  // decode merge: the peers' partial O slices landed
  alignas(16) float mref[kH], alpha[kH], lsh[kH], linv[kH];
  float tmax[4][kH];
  float mw[kH][kMaxCluster];        // decode merge: weight of each rank, per owned head
  uint32_t flagcnt[3], tmem, has_tiles;
  uint32_t n_end;   // decode over bf16 rows, ratio 4: rows up to the entry that ends the list
};
// 4-bit rows, ratio 4: the top-k lists of the query in work and the next one as pool
// rows (kNoRow: masked), staged by the loaders for every role; lists above kList entries
// take both halves, one query at a time
constexpr uint32_t kList = 1024, kNoRow = 0xffffffffu;
struct SmemFp4 : Smem {
  uint32_t rows[2 * kList];
  // per loader warp: bits 16 .. 31 the first place that ends the list (0xffff: none), bits
  // 0 .. 15 the place behind the last row (lists have at most 2048 places)
  uint32_t wend[2][8];
  uint64_t geo_full[2], geo_empty[2], ld_bar;
};
// the merge pulls at most C * ceil(64 / C) rows of 1 KiB (75 at C = 15)
constexpr uint32_t max_pulled_rows(uint32_t C = 1) {
  return C > kMaxCluster ? 0u
                         : (C * ((kH + C - 1) / C) > max_pulled_rows(C + 1) ? C * ((kH + C - 1) / C)
                                                                             : max_pulled_rows(C + 1));
}
static_assert(sizeof(SmemFp4) + 1024 <= 227 * 1024, "one block's shared memory");
static_assert(8 * kKBlk >= max_pulled_rows() * kD * 2, "pulled slices fit the row buffer");
static_assert(sizeof(Smem::q) + sizeof(Smem::kv) >= max_pulled_rows() * kD * 4 &&
                  offsetof(Smem, kv) == sizeof(Smem::q),
              "fp32 slices fit Q's buffer and the row buffer behind it");
static_assert(2 * kH * 128 == kRows * 128, "output staging fills the P buffer");

// Places that a query's rows can take at most, without reading its top-k list (whose rows
// may stand anywhere in it).
__device__ __forceinline__ uint32_t rows_bound(const TcAttnParams &P, uint32_t qi) {
  const uint32_t p = seq_base(P.seq_pos, P.pos0, qi / P.T) + qi % P.T;
  uint32_t n = min(p + 1, P.cap_raw);
  if (P.ratio == 4) n += min((p + 1) / 4, P.n_comp) ? P.top_k : 0u;
  else if (P.ratio == 128) n += min((p + 1) / 128, P.n_comp);
  return n;
}

// Query-level geometry shared by every role: tiles t0, t0 + ts, ... < t1.
struct QueryGeo {
  // p0: the sequence's first chunk position; vis: visible rows (ratio 4; else any number)
  uint32_t qi, b, p0, p, n_w, n_list, N, t0, t1, ts, vis;
  const int32_t *tk;
};

// A ratio-4 list ends at its first entry that is not visible. One warp: bits 16 .. 31 the
// place of that entry (n: none), bits 0 .. 15 the place behind the last visible row (lists
// have at most 2048 places).
static __device__ __noinline__ uint32_t list_scan(const int32_t *tk, uint32_t n, uint32_t vis) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t end = n, top = 0;
#pragma unroll 1
  for (uint32_t base = lane; base - lane < n; base += 512) {
    int32_t v[16];   // 16 loads in flight
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i) v[i] = base + 32 * i < n ? tk[base + 32 * i] : -1;
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i) {
      if ((uint32_t)v[i] < vis) top = base + 32 * i + 1;
      else if (v[i] >= 0) end = min(end, base + 32 * i);
    }
  }
  return redux_min_u32(end) << 16 | redux_max_u32(top);
}
// The place of the entry that ends the list alone (n: none), in little code where there is
// no such entry.
static __device__ __noinline__ uint32_t list_stop(const int32_t *tk, uint32_t n, uint32_t vis) {
  int32_t most = -1;
#pragma unroll 1
  for (uint32_t base = threadIdx.x & 31; base < n; base += 512) {
    int32_t v[16];
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i) v[i] = tk[min(base + 32 * i, n - 1)];
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i) most = max(most, v[i]);
  }
  // (negative entries as unsigned would be the largest)
  if (redux_max_u32((uint32_t)most + 1u) <= vis) return n;
  return list_scan(tk, n, vis) >> 16;
}

// SCAN: read the list for its end (a chunk over bf16 rows). Decode over bf16 rows gives every
// place of a list a row of a tile where as many rows are visible (the list is then full, or has
// holes), without reading it before the first gather: entries that are no visible row are masked
// one by one, those behind the list's end once the loaders have looked for it, while the first
// rows are on their way (c4a, 8 sequences, side by side with early queries: 13.0 us; with the
// list read by every role before the first gather 13.8, without any look for its end 12.6).
// Where fewer rows are visible than the list has places, it is read for its length (at
// position 500: 14.4 us, at 3,000 13.8). n_list: the length of a ratio-4 list where it is
// known (4-bit rows).
template <bool SCAN>
__device__ __forceinline__ QueryGeo query_geo(const TcAttnParams &P, uint32_t qi, uint32_t t0,
                                              uint32_t ts, uint32_t lane,
                                              uint32_t n_list = kNoRow) {
  QueryGeo g;
  g.qi = qi;
  g.b = qi / P.T;
  g.p0 = seq_base(P.seq_pos, P.pos0, g.b);
  g.p = g.p0 + qi % P.T;
  g.n_w = min(g.p + 1, P.cap_raw);
  g.tk = P.topk ? P.topk + (size_t)qi * P.top_k : nullptr;
  g.n_list = 0;
  g.vis = P.ratio == 4 ? min((g.p + 1) / 4, P.n_comp) : 0x80000000u;
  if (n_list != kNoRow) {
    g.n_list = n_list;
  } else if (P.ratio == 4 && !SCAN) {
    g.n_list = P.top_k;
    if (g.vis < P.top_k) {
      const uint32_t ends = list_scan(g.tk, P.top_k, g.vis);
      g.n_list = min(ends >> 16, ends & 0xffffu);
    }
  } else if (P.ratio == 4) {
    const uint32_t vis = g.vis;
    // the list ends at its first entry >= vis; 16 independent loads per round
    g.n_list = P.top_k;
    for (uint32_t base = 0; base < P.top_k; base += 512) {
      int32_t v[16];
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) {
        const uint32_t j = base + 32 * i + lane;
        v[i] = j < P.top_k ? g.tk[j] : -1;
      }
      uint32_t found = 0xffffffffu;
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) {
        const uint32_t bal = __ballot_sync(0xffffffffu, v[i] >= 0 && (uint32_t)v[i] >= vis);
        if (bal && found == 0xffffffffu) found = base + 32 * i + __ffs(bal) - 1;
      }
      if (found != 0xffffffffu) {
        g.n_list = found;
        break;
      }
    }
  } else if (P.ratio == 128) {
    g.n_list = min((g.p + 1) / 128, P.n_comp);
  }
  g.N = g.n_w + g.n_list;
  g.t0 = t0;
  g.t1 = (g.N + kRows - 1) / kRows;
  g.ts = ts;
  return g;
}

// How tile `tile` of a decode query loads: 0 row gathers, 1 the whole ring
// by TMA (the window of 128 rows, in slot order: the softmax does not depend
// on the order of the rows), 2 compressed rows 128 (tile - 1) .. by TMA, 3 (4-bit
// rows, chunk) a window that lies in the chunk, by TMA.
template <bool DEC, bool PAGED, bool FP4 = false>
__device__ __forceinline__ uint32_t tile_kind(const TcAttnParams &P, const QueryGeo &g,
                                              uint32_t tile) {
  if (FP4 && !DEC)
    return tile == 0 && (P.tma_rows & 4u) && g.p - g.p0 >= (uint32_t)kRows - 1 ? 3u : 0u;
  if (!DEC || g.n_w != (uint32_t)kRows) return 0;
  if (tile == 0) return (P.tma_rows & 1u) ? 1u : 0u;
  return (!PAGED && (P.tma_rows & 2u) && P.ratio == 128) ? 2u : 0u;
}

// Source row of list entry r (nullptr: masked).
template <bool PAGED>
__device__ __forceinline__ const __nv_bfloat16 *row_src(const TcAttnParams &P, const QueryGeo &g,
                                                        uint32_t r) {
  if (r < g.n_w) {
    const uint32_t pos = g.p - g.n_w + 1 + r;
    if (P.chunk && pos >= g.p0)
      return P.chunk + ((size_t)g.b * P.T + (pos - g.p0)) * kD;
    return P.ring + ((size_t)g.b * P.cap_raw + pos % P.cap_raw) * kD;
  }
  if (r < g.N) {
    const uint32_t j = r - g.n_w;
    const int32_t idx = P.ratio == 4 ? g.tk[j] : (int32_t)j;
    if ((uint32_t)idx < g.vis) {
      if (PAGED) return P.comp + P.map.row_of(g.b, (uint32_t)idx) * kD;
      return P.comp + ((size_t)g.b * P.comp_cap + (uint32_t)idx) * kD;
    }
  }
  return nullptr;
}

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Decode merge of rank `rank` of a C-CTA cluster (C > 1; threads 0..255):
// heads [64 rank / C, 64 (rank + 1) / C) of every rank's partial O land in the
// row-tile buffer as [j][i][512] fp32 and are combined in rank order with
// weights 2^(m_j - M) / sum_j 2^(m_j - M) l_j. A rank without rows left
// m = -inf and zeros; one with only masked rows left m = -inf and O = 0.
// CM: compile-time bound on the cluster size C (the loops over ranks unroll). FP4: the
// partials are fp32 (in bf16 they added a rounding to that of P: a c4a call's relative
// error 0.0026 against 0.0021, at the same time), pulled into Q's buffer and the
// tile's, and twice the threads combine them.
template <uint32_t CM, int NH, bool FP4>
__device__ __forceinline__ bool merge_heads(const TcAttnParams &P, Smem &S, uint32_t vq,
                                            uint32_t rank, uint32_t C, ErrWord ew) {
  const uint32_t HG = FP4 ? P.hg : (uint32_t)(kH / NH), HQ = FP4 ? P.n_heads : (uint32_t)kH;
  const uint32_t t = threadIdx.x, qi = vq / HG, hq0 = (vq % HG) * NH;
  const uint32_t h0 = rank * NH / C, h1 = (rank + 1) * NH / C, nh = h1 - h0;
  using PT = typename std::conditional<FP4, float, __nv_bfloat16>::type;
  constexpr uint32_t kMT = FP4 ? 512 : 256;   // threads
  const PT *part = reinterpret_cast<const PT *>(P.part) + (size_t)vq * C * NH * kD;
  const float *ml = P.ml + (size_t)vq * C * NH * 2;
  PT *recv = reinterpret_cast<PT *>(FP4 ? S.q : S.kv);
  // rank j's rows h0 .. h1 - 1 are contiguous: one bulk copy per rank
  if (t == 0) {
    fence_proxy_async_global();
    mbar_arrive_expect_tx(&S.mg_bar, C * nh * kD * sizeof(PT));
    for (uint32_t j = 0; j < C; ++j)
      bulk_load(recv + (size_t)j * nh * kD, part + ((size_t)j * NH + h0) * kD,
                nh * kD * sizeof(PT), &S.mg_bar);
  }
  if (t < nh) {
    const uint32_t h = h0 + t;
    float m[CM], l[CM], M = -INFINITY;
#pragma unroll
    for (uint32_t j = 0; j < CM; ++j) {
      m[j] = j < C ? __ldcg(ml + ((size_t)j * NH + h) * 2) : -INFINITY;   // written by peers
      l[j] = j < C ? __ldcg(ml + ((size_t)j * NH + h) * 2 + 1) : 0.f;
    }
#pragma unroll
    for (uint32_t j = 0; j < CM; ++j) M = fmaxf(M, m[j]);
    // O = sum_j f_j (O_j / L_j) with f_j = 2^(m_j - M) L_j / sum_i 2^(m_i - M) L_i
    float f[CM], L = 0.f;
#pragma unroll
    for (uint32_t j = 0; j < CM; ++j) {
      f[j] = m[j] == -INFINITY ? 0.f : exp2f(m[j] - M) * l[j];
      L += f[j];
    }
    const float li = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (uint32_t j = 0; j < CM; ++j) S.mw[t][j] = f[j] * li;
  }
  // rotation coefficients load while the slices land
  const uint32_t p = seq_base(P.seq_pos, P.pos0, qi / P.T) + qi % P.T, c = t & 127, d = 4 * c;
  float co0 = 1.f, si0 = 0.f, co1 = 1.f, si1 = 0.f;
  if (d >= (uint32_t)kNope) {
    const uint32_t fi = (d - kNope) >> 1;
    co0 = P.cos[(size_t)p * 32 + fi];
    si0 = P.sin[(size_t)p * 32 + fi];
    co1 = P.cos[(size_t)p * 32 + fi + 1];
    si1 = P.sin[(size_t)p * 32 + fi + 1];
  }
  const bool ok = mbar_wait(&S.mg_bar, 0, ew);
  named_bar_sync(1, kMT);
  if (!ok) return false;
#pragma unroll 1
  for (uint32_t i = t >> 7; i < nh; i += kMT / 128) {
    float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (uint32_t j = 0; j < CM; ++j) {
      const float f = S.mw[i][j];
      if (j < C && f != 0.f) {
        if (FP4) {
          const float4 v = *reinterpret_cast<const float4 *>(recv + (j * nh + i) * kD + d);
          a0 = fmaf(f, v.x, a0);
          a1 = fmaf(f, v.y, a1);
          a2 = fmaf(f, v.z, a2);
          a3 = fmaf(f, v.w, a3);
          continue;
        }
        const uint2 v = *reinterpret_cast<const uint2 *>(recv + (j * nh + i) * kD + d);
        a0 = fmaf(f, bf16lo(v.x), a0);
        a1 = fmaf(f, bf16hi(v.x), a1);
        a2 = fmaf(f, bf16lo(v.y), a2);
        a3 = fmaf(f, bf16hi(v.y), a3);
      }
    }
    // rotate back by -p: (x0, x1) -> (x0 c + x1 s, -x0 s + x1 c)
    const float r0 = a0 * co0 + a1 * si0, r1 = -a0 * si0 + a1 * co0;
    const float r2 = a2 * co1 + a3 * si1, r3 = -a2 * si1 + a3 * co1;
    if (!FP4 || hq0 + h0 + i < HQ)   // (a last group of heads may be part-filled)
      *reinterpret_cast<uint2 *>(P.out + ((size_t)qi * HQ + hq0 + h0 + i) * kD + d) =
          make_uint2(pack_bf16(r0, r1), pack_bf16(r2, r3));
  }
  return true;
}

// The eight dims of code word w, a lane's word of 64-dim block KB, as the 16-byte chunk of
// the bf16 tile. sl, sh: the scale bytes of the lane's blocks 0 .. 3 and 4 .. 6. E2M1
// times 2^-126 (fp4_pair_raw) becomes the bf16 value by one exact product with
// 2^(k + 126), a bf16 number while k <= 1 (byte <= 128: largest magnitude up to 12);
// `wide`: the row has a larger scale and takes two products.
template <uint32_t KB>
__device__ __forceinline__ uint4 fp4_chunk(uint32_t w, uint32_t sl, uint32_t sh, bool wide) {
  const uint32_t byte = ((KB < 4 ? sl : sh) >> (8 * (KB % 4))) & 255u;
  uint32_t o[4] = {fp4_pair_raw<0>(w), fp4_pair_raw<1>(w), fp4_pair_raw<2>(w), fp4_pair_raw<3>(w)};
  uint32_t m = byte * 0x00800080u + 0x3F003F00u;   // 2^(k + 126), twice
  if (wide) {
    const uint32_t up = 0x7E807E80u;               // 2^126, twice
    m = byte ? byte * 0x00800080u : 0x00400040u;   // 2^k
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&o[i]),
                                       *reinterpret_cast<const __nv_bfloat162 *>(&up));
      o[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&o[i]),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&m));
    o[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// A scale byte above 128 among the four of a word.
__device__ __forceinline__ uint32_t fp4_wide(uint32_t s) {
  return ((s & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & s & 0x80808080u;
}
constexpr uint32_t kFp4RowBytes = 384;   // D 512, n_rot 64, bf16

// DEC: decode (clusters of P.cluster CTAs per query) or prefill (persistent
// CTAs); PAGED: rows through the block table (4-bit rows look at it at run time);
// FP4: compressed rows in 4 bits; NH: heads per CTA. Instantiations keep each path's
// code to itself.
template <bool DEC, bool PAGED, bool FP4, int NH>
__global__ void __launch_bounds__(Warps<FP4>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
                   const __grid_constant__ CUtensorMap tmap_ring,
                   const __grid_constant__ CUtensorMap tmap_comp, TcAttnParams P) {
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned. Prefill takes an offset from the shared array itself,
  // so its accesses to S compile to shared-memory instructions (chunk
  // attention 795 -> 750 us); decode keeps the integer round trip and generic
  // accesses, which measured faster for its c4a and c128a calls (14.5 / 16.7
  // against 14.8 / 17.0 us)
  uint8_t *sbase;
  if (DEC && !FP4)
    sbase = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                        ~(uintptr_t)1023);
  else
    sbase = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  using SmemT = typename std::conditional<FP4, SmemFp4, Smem>::type;
  SmemT &S = *reinterpret_cast<SmemT *>(sbase);
  SmemFp4 &S4 = *reinterpret_cast<SmemFp4 *>(sbase);   // (4-bit rows only)
  // (4-bit rows: the same for the compiler too, so that the MMA issuer's branch and
  // its descriptors are warp-uniform)
  const uint32_t warp = FP4 ? uniform(threadIdx.x >> 5) : threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  // decode: cluster of C CTAs per (query, head group), rank c takes tiles
  // c, c + C, ...; prefill: one whole query at a time per CTA
  constexpr bool dec = DEC;
  using HS = Heads<NH>;
  using WP = Warps<FP4>;
  constexpr int NHF = HS::NHF, QBLK = HS::QBLK;
  // head groups of a query and its heads; 4-bit rows take any number of heads
  const uint32_t HG = FP4 ? P.hg : (uint32_t)HS::HG, HQ = FP4 ? P.n_heads : (uint32_t)kH;
  constexpr bool kScan = !DEC && !FP4;   // read the list for its end (see query_geo)
  // 4-bit rows, ratio 4: half `gb` of the staged lists (gn: lists before this one), the
  // length of the list in it, and its release
  const bool staged = FP4 && P.ratio == 4;
  const uint32_t n_half = P.top_k <= kList ? 2u : 1u;
  auto list_half = [&](uint32_t gn) { return n_half == 2 ? gn & 1 : 0u; };
  auto list_phase = [&](uint32_t gn) { return (n_half == 2 ? gn >> 1 : gn) & 1; };
  auto list_end = [&](uint32_t gb) {
    uint32_t e = 0xffffu, top = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      e = min(e, S4.wend[gb][w] >> 16);
      top = max(top, S4.wend[gb][w] & 0xffffu);
    }
    return min(e, top);
  };
  const uint32_t C = dec ? P.cluster : 1u;
  const uint32_t rank = dec ? cluster_ctarank() : 0u;
  const uint32_t vq = dec ? blockIdx.x / C : 0u;          // decode: (query, head group)
  // items (query, head group) i0, i0 + i_step, ... < n_items: one in decode; prefill
  // of bf16 rows has one group, so that an item is a query
  const uint32_t n_items = FP4 ? P.n_q * P.hg : dec ? P.n_q * HS::HG : P.n_q;
  const uint32_t i0 = dec ? vq : blockIdx.x, i_step = dec ? n_items : gridDim.x;
  auto item_q = [&](uint32_t it) { return FP4 || dec ? it / HG : it; };
  auto item_h = [&](uint32_t it) { return FP4 || dec ? (it % HG) * NH : 0u; };   // first head
  // The wait for the previous launch: in a chunk here; in decode behind the block's own
  // preparations (c4a over bf16 rows, 8 sequences: 13.8 us; here for every call 14.3) or,
  // with q_ready, in the loaders behind the first query's Q load (13.1).
  const bool ready = DEC && P.q_ready != 0;
  if (!DEC) pdl_wait();
  // (this launch's view of the error word: see ErrWord)
  int err_base = 0;
  if (ready || !DEC) err_base = *(volatile int *)P.err;
  if (NH < kH) {
    // heads NH .. 63 of every P row stay zero: the PV and sum MMAs read all
    // 64 columns, and those of the other group contribute nothing
    uint4 *pz = reinterpret_cast<uint4 *>(S.p);
    for (uint32_t i = threadIdx.x; i < kRows * 128 / 16; i += blockDim.x)
      pz[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }

  if (threadIdx.x == 0) {
    mbar_init(&S.kv_full, WP::LT);
    for (int i = 0; i < 4; ++i) mbar_init(&S.kv_empty[i], 1);
    mbar_init(&S.q_full, WP::LT);
    mbar_init(&S.q_empty, 1);
    mbar_init(&S.s_full, 1);
    mbar_init(&S.p_full, WP::ST);
    mbar_init(&S.p_empty, 1);
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_empty, FP4 && !DEC ? WP::NS + WP::NL : WP::NS);
    mbar_init(&S.sm_bar, WP::ST);
    mbar_init(&S.q_tma, 1);
    mbar_init(&S.kv_tma, 1);
    mbar_init(&S.mg_bar, 1);
    if (FP4) {
      for (int i = 0; i < 4; ++i) mbar_init(&S.kv_pair[i], WP::LT);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&S4.geo_full[i], 1);
        mbar_init(&S4.geo_empty[i], WP::NS + 1);   // softmax warps and the MMA issuer
      }
      mbar_init(&S4.ld_bar, WP::LT);
    }
    S.flagcnt[0] = S.flagcnt[1] = S.flagcnt[2] = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
    if (P.tma_rows) {
      prefetch_tmap(&tmap_ring);
      prefetch_tmap(&tmap_comp);
    }
  }
  if (warp == WP::MMA) tmem_alloc(&S.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  // TMEM columns: S^T 0..63, row sums L 64..127, an all-ones bf16 A operand
  // 128..159 (L = ones x P^T), O^T 256..511
  const uint32_t tmS = tmem, tmL = tmem + 64, tmOnes = tmem + 128, tmO = tmem + 256;
  if (warp < 4) {
    uint32_t ones[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) ones[i] = 0x3F803F80u;   // two bf16 1.0
    tmem_st32(tmOnes + ((warp * 32) << 16), ones);
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool loader = warp >= WP::NS && warp < WP::MMA;
  if (!loader || (DEC && !ready)) {
    pdl_wait();
    pdl_trigger();
    if (DEC && !ready) err_base = *(volatile int *)P.err;
  }
  const ErrWord ew{P.err, err_base};
  auto wait_warp = [&](uint64_t *bar, uint32_t parity, ErrWord e) {
    return FP4 ? mbar_wait_sleep(bar, parity, e) : mbar_wait_warp(bar, parity, e);
  };
  auto sync_group = [&](uint64_t *bar, uint32_t &phase, ErrWord e) {
    return FP4 ? group_sync_sleep(bar, phase, e) : group_sync(bar, phase, e);
  };

  // Chunks over 4-bit rows: a query's output is written by the softmax warps (dim
  // blocks 0 and 1) and the loaders (2 and 3), both idle between its last tile and the
  // first tile of the next query, whose PV waits for o_empty. Warp w has TMEM quarter
  // w % 4 and 32 heads; lanes 2 i, 2 i + 1 hold dims d, d + 1 and swap so that each
  // stores bf16 pairs of its own heads.
  float out_co = 1.f, out_si = 0.f;   // the rotation of this thread's dim (tail dims)
  auto out_coef = [&](uint32_t p) {   // (TMEM quarters 2, 3: dims 64 .. 127 of a block)
    if ((warp & 2) != 0) {
      const uint32_t fi = (32 * (warp & 3) + lane - 64) >> 1;
      out_co = P.cos[(size_t)p * 32 + fi];
      out_si = P.sin[(size_t)p * 32 + fi];
    }
  };
  auto write_out = [&](uint32_t it, uint32_t qn_prev, uint32_t m0) -> bool {
    const uint32_t qi = item_q(it), sq = warp & 3, hf = (warp >> 2) & 1;
    const uint32_t h0 = item_h(it) + 32 * hf, r = 32 * sq + lane, lane_base = (32 * sq) << 16;
    const float co = out_co, si = out_si;
    if (!wait_warp(&S.o_full, qn_prev & 1, ew)) return false;
    tc_fence_after();
    const bool odd = lane & 1;
    // 1 / L of head 32 hf + lane from this lane's copy (every TMEM row of L holds the
    // sums), then all 32 by broadcast; warps with the same heads write the same values
    uint32_t a[2][16];   // sixteen heads at a time, the next load in flight
    float li[32];
#pragma unroll
    for (int hs = 0; hs < 2; ++hs) tmem_ld16(tmL + lane_base + 32 * hf + 16 * hs, a[hs]);
    tmem_ld_wait();
    float l = 0.f;
#pragma unroll
    for (uint32_t h = 0; h < 32; ++h)
      if (lane == h) l = __uint_as_float(a[h / 16][h % 16]);
    S.linv[32 * hf + lane] = l > 0.f ? __fdividef(1.f, l) : 0.f;
    __syncwarp();
#pragma unroll
    for (uint32_t h = 0; h < 32; h += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(&S.linv[32 * hf + h]);
      li[h] = v.x;
      li[h + 1] = v.y;
      li[h + 2] = v.z;
      li[h + 3] = v.w;
    }
    __nv_bfloat16 *o = P.out + ((size_t)qi * HQ + h0) * kD + 128 * m0 + (r & ~1u);
    const uint32_t live = HQ > h0 ? HQ - h0 : 0u;   // heads there are
    tmem_ld16(tmO + lane_base + m0 * kH + 32 * hf, a[0]);
#pragma unroll 1
    for (uint32_t m = m0; m < m0 + 2; ++m, o += 128) {
#pragma unroll
      for (uint32_t hs = 0; hs < 2; ++hs) {
        tmem_ld_wait();
        if (hs == 0)
          tmem_ld16(tmO + lane_base + m * kH + 32 * hf + 16, a[1]);
        else if (m == m0)
          tmem_ld16(tmO + lane_base + (m + 1) * kH + 32 * hf, a[0]);
        else {   // everything read: the next query's PV may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.o_empty);
        }
        const uint32_t(&x)[16] = a[hs];
        if (m == 3 && sq >= 2) {   // the rotated tail, back by -p, in fp32
#pragma unroll
          for (uint32_t h = 0; h < 16; h += 2) {
            const float v0 = __uint_as_float(x[h]) * li[16 * hs + h];
            const float v1 = __uint_as_float(x[h + 1]) * li[16 * hs + h + 1];
            const float recv = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            const float x0 = odd ? recv : v0, x1 = odd ? v1 : recv;
            const uint32_t row = 16 * hs + h + (odd ? 1u : 0u);
            if (row < live)
              *reinterpret_cast<uint32_t *>(o + (size_t)row * kD) =
                  pack_bf16(x0 * co + x1 * si, -x0 * si + x1 * co);
          }
        } else {
#pragma unroll
          for (uint32_t h = 0; h < 16; h += 4) {
            const uint32_t w0 = pack_bf16(__uint_as_float(x[h]) * li[16 * hs + h],
                                          __uint_as_float(x[h + 1]) * li[16 * hs + h + 1]);
            const uint32_t w1 = pack_bf16(__uint_as_float(x[h + 2]) * li[16 * hs + h + 2],
                                          __uint_as_float(x[h + 3]) * li[16 * hs + h + 3]);
            // even lanes keep heads h, h + 2, odd lanes h + 1, h + 3
            const uint32_t mine = __byte_perm(w0, w1, odd ? 0x7632 : 0x5410);
            const uint32_t give = __byte_perm(w0, w1, odd ? 0x5410 : 0x7632);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
            const uint32_t lo = odd ? got : mine, hi = odd ? mine : got;
            const uint32_t row = 16 * hs + h + (odd ? 1u : 0u);
            if (row < live)
              *reinterpret_cast<uint32_t *>(o + (size_t)row * kD) = __byte_perm(lo, hi, 0x5410);
            if (row + 2 < live)
              *reinterpret_cast<uint32_t *>(o + (size_t)(row + 2) * kD) =
                  __byte_perm(lo, hi, 0x7632);
          }
        }
      }
    }
    return true;
  };

  if (loader) {
    // ------------------------------------------------------------ loaders
    const uint32_t lt = threadIdx.x - WP::ST, lw = warp - WP::NS;
    uint32_t n = 0, qn = 0, qt = 0, nk = 0;   // qt: Q loads issued, nk: TMA tiles issued
    // issue all eight 64-dim blocks of a tile (one cp.async group each) as
    // their slots free up; rows of this lane: lw*32 + lane/8 + 4i, chunk lane%8.
    // A tile of contiguous rows is eight TMA boxes of 128 rows x 64 dims
    // (one thread), in the same swizzled layout.
    auto issue_tile = [&](const QueryGeo &g, uint32_t tile, uint32_t n) -> bool {
      if (const uint32_t kind = tile_kind<DEC, PAGED>(P, g, tile)) {
        for (uint32_t kb = 0; kb < 8; ++kb) {
          if ((kb & 1) == 0 && !wait_warp(&S.kv_empty[kb >> 1], (n & 1) ^ 1, ew)) return false;
          if (lt == 0) {
            if (kb == 0) mbar_arrive_expect_tx(&S.kv_tma, 8 * kKBlk);
            if (kind == 1)
              tma_load_3d(S.kv + kb * kKBlk, &tmap_ring, &S.kv_tma, (int)(64 * kb), 0, (int)g.b);
            else
              tma_load_3d(S.kv + kb * kKBlk, &tmap_comp, &S.kv_tma, (int)(64 * kb),
                          (int)(kRows * (tile - 1)), (int)g.b);
          }
        }
        return true;
      }
      const __nv_bfloat16 *src[8];
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i)
        src[i] = row_src<PAGED>(P, g, tile * kRows + lw * 32 + (lane >> 3) + 4 * i);
      const uint32_t cc = lane & 7;
      for (uint32_t kb = 0; kb < 8; ++kb) {
        if ((kb & 1) == 0 && !wait_warp(&S.kv_empty[kb >> 1], (n & 1) ^ 1, ew)) return false;
        uint8_t *slot = S.kv + kb * kKBlk;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
          const uint32_t r = lw * 32 + (lane >> 3) + 4 * i;
          uint8_t *dst = slot + (r >> 3) * 1024 + (r & 7) * 128 + ((cc ^ (r & 7)) << 4);
          const __nv_bfloat16 *sp = src[i] ? src[i] + kb * 64 + cc * 8 : P.ring;
          cp_async16(dst, sp, src[i] ? 16u : 0u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      return true;
    };
    // this thread's chunks of the rows from n_end on, once they have landed: zeros
    auto zero_rows = [&](uint32_t tile, uint32_t n_end) {
      cp_async_wait_all();
#pragma unroll 1
      for (uint32_t e = 0; e < 64; ++e) {
        const uint32_t r = lw * 32 + (lane >> 3) + 4 * (e & 7), kb = e >> 3;
        if (tile * kRows + r >= n_end)
          *reinterpret_cast<uint4 *>(S.kv + kb * kKBlk + (r >> 3) * 1024 + (r & 7) * 128 +
                                     (((lane & 7) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
      }
    };
    // ---- 4-bit rows: thread lt holds lane lt % 8 of rows lt / 8 + 32 i. fetch_tile
    // loads their records into registers (12 16-byte loads in flight, each warp
    // load 128 contiguous bytes of four rows); store_tile converts them block pair by
    // block pair as the tile's slots free up. The next tile's records load while
    // this one's MMAs run.
    constexpr uint32_t kFR = FP4 ? kRows * 8 / WP::LT : 1;   // rows per thread
    uint4 rec[kFR][3];
    uint32_t tbl[kFR] = {};   // ratio 128, paged: table entries of the next tile's rows
    uint32_t cur_raw = 0;     // bit i: row i is in bf16 (the window)
    uint32_t gn = 0, gb = 0, ld_phase = 0;   // lists staged, the current one's half
    const uint32_t rsh = P.ratio == 4 ? 6u : 1u;   // log2 of the rows per block
    auto list_row = [&](uint32_t g_b, uint32_t idx, uint32_t blk) {
      // (as RowMap::phys: table entries outside the pool read block 0)
      if (P.map.table) return ((blk < P.map.n_blocks ? blk : 0u) << rsh) + (idx & ((1u << rsh) - 1));
      return g_b * P.comp_cap + idx;     // (below 2^32: checked on the host)
    };
    auto table_at = [&](uint32_t g_b, uint32_t idx) -> const int32_t * {
      const uint32_t lb = min(idx >> rsh, P.map.max_blocks - 1);
      return P.map.table + (size_t)g_b * P.map.max_blocks + lb;
    };
    // The list of a ratio-4 query as pool rows in shared memory. stage_load starts the
    // loads of up to kList entries (a chunk does so a few tiles ahead of the query),
    // stage_list finishes them, or does it all for longer lists; it returns the list's
    // length (kNoRow: a wait gave up).
    auto stage_load = [&](uint32_t qi) {
      const int32_t *tk = P.topk + (size_t)qi * P.top_k;
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i) {
        const uint32_t e = lt + WP::LT * i;
        tbl[i] = e < P.top_k ? ld_nc_u32(tk + e) : kNoRow;
      }
    };
    auto stage_list = [&](uint32_t qi) -> uint32_t {
      gb = list_half(gn);
      const uint32_t b = qi / P.T, p = seq_base(P.seq_pos, P.pos0, b) + qi % P.T;
      const uint32_t vis = min((p + 1) / 4, P.n_comp);
      if (!wait_warp(&S4.geo_empty[gb], list_phase(gn) ^ 1, ew)) return kNoRow;
      uint32_t end = 0xffffu, top = 0;
      for (uint32_t base = 0; base < P.top_k; base += kList) {
        uint32_t blk[kFR];
        if (base) {
#pragma unroll
          for (uint32_t i = 0; i < kFR; ++i) {
            const uint32_t e = base + lt + WP::LT * i;
            tbl[i] = e < P.top_k ? ld_nc_u32(P.topk + (size_t)qi * P.top_k + e) : kNoRow;
          }
        }
#pragma unroll
        for (uint32_t i = 0; i < kFR; ++i) {
          blk[i] = 0;
          if ((int32_t)tbl[i] >= 0 && tbl[i] >= vis) {
            end = min(end, base + lt + WP::LT * i);
            tbl[i] = kNoRow;
          }
          if ((int32_t)tbl[i] >= 0) top = base + lt + WP::LT * i + 1;
          if (P.map.table && (int32_t)tbl[i] >= 0) blk[i] = ld_nc_u32(table_at(b, tbl[i]));
        }
#pragma unroll
        for (uint32_t i = 0; i < kFR; ++i) {
          const uint32_t e = base + lt + WP::LT * i;
          if (e < P.top_k)
            S4.rows[gb * kList + e] = (int32_t)tbl[i] >= 0 ? list_row(b, tbl[i], blk[i]) : kNoRow;
        }
      }
      end = redux_min_u32(end);
      top = redux_max_u32(top);
      if (lane == 0) S4.wend[gb][lw] = end << 16 | top;
      if (!sync_group(&S4.ld_bar, ld_phase, ew)) return kNoRow;
      if (lt == 0) mbar_arrive(&S4.geo_full[gb]);
      ++gn;
      return list_end(gb);
    };
    // the table entries that the fetch of a tile will need (a tile ahead of it)
    auto look_tile = [&](const QueryGeo &g, uint32_t tile) {
      if (staged || !P.map.table) return;
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i) {
        const uint32_t r = tile * kRows + (lt >> 3) + 32 * i;
        tbl[i] = r >= g.n_w && r < g.N ? ld_nc_u32(table_at(g.b, r - g.n_w)) : 0u;
      }
    };
    auto fetch_tile = [&](const QueryGeo &g, uint32_t tile) {
      cur_raw = 0;
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i) {
        const uint32_t r = tile * kRows + (lt >> 3) + 32 * i;
        uint32_t row = kNoRow;   // (a masked row: zeros)
        if (r < g.n_w) cur_raw |= 1u << i;
        else if (r < g.N)
          row = staged ? S4.rows[gb * kList + (r - g.n_w)] : list_row(g.b, r - g.n_w, tbl[i]);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(P.comp) + (size_t)row * kFp4RowBytes +
                             16 * (lt & 7);
#pragma unroll
        for (uint32_t v = 0; v < 3; ++v)
          rec[i][v] = row != kNoRow ? ld_nc_v4(src + 128 * v) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    // Decode, ratio 4: the records of this rank's first tile straight from the list, so that
    // they load while the list is staged.
    auto fetch_first = [&](uint32_t qi) {
      const uint32_t b = qi / P.T, p = seq_base(P.seq_pos, P.pos0, b) + qi % P.T;
      const uint32_t n_w = min(p + 1, P.cap_raw), vis = min((p + 1) / 4, P.n_comp);
      const int32_t *tk = P.topk + (size_t)qi * P.top_k;
      uint32_t idx[kFR], blk[kFR];
      cur_raw = 0;
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i) {
        const uint32_t r = rank * kRows + (lt >> 3) + 32 * i;
        if (r < n_w) cur_raw |= 1u << i;
        idx[i] = r >= n_w && r - n_w < P.top_k ? ld_nc_u32(tk + (r - n_w)) : kNoRow;
      }
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i)
        blk[i] = P.map.table && idx[i] < vis ? ld_nc_u32(table_at(b, idx[i])) : 0u;
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i) {
        const uint8_t *src = reinterpret_cast<const uint8_t *>(P.comp) +
                             (size_t)list_row(b, idx[i], blk[i]) * kFp4RowBytes + 16 * (lt & 7);
#pragma unroll
        for (uint32_t v = 0; v < 3; ++v)
          rec[i][v] = idx[i] < vis ? ld_nc_v4(src + 128 * v) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    // this thread's chunk of row i in 64-dim block KB of the tile
    auto chunk_dst = [&](uint32_t i, uint32_t KB) {
      const uint32_t r = (lt >> 3) + 32 * i;
      return S.kv + KB * kKBlk + (r >> 3) * 1024 + (r & 7) * 128 + (((lt & 7) ^ (r & 7)) << 4);
    };
    auto store_tile = [&](const QueryGeo &g, uint32_t tile, uint32_t n) -> bool {
      if (const uint32_t kind = tile_kind<DEC, true, FP4>(P, g, tile)) {
        // the window by TMA, a box per loader warp: the ring's slots 0 .. 127, or chunk
        // rows p - p0 - 127 .. p - p0
        if (lt == 0) mbar_arrive_expect_tx(&S.kv_tma, 8 * kKBlk);
        if (!wait_warp(&S.kv_empty[lw >> 1], (n & 1) ^ 1, ew)) return false;
        if (lane == 0)
          tma_load_3d(S.kv + lw * kKBlk, &tmap_ring, &S.kv_tma, (int)(64 * lw),
                      kind == 3 ? (int)(g.p - g.p0) - (kRows - 1) : 0, (int)g.b);
#pragma unroll
        for (uint32_t m = 0; m < 4; ++m) mbar_arrive(&S.kv_pair[m]);
        return true;
      }
      const uint32_t j = lt & 7;
      uint32_t sl[kFR], sh[kFR], wide = 0;
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i) {   // a pair of lanes shares its scale bytes
        const uint32_t mine = rec[i][1].w, other = __shfl_xor_sync(0xffffffffu, mine, 1);
        sl[i] = j & 1 ? other : mine;
        sh[i] = j & 1 ? mine : other;
        if (fp4_wide(sl[i]) | fp4_wide(sh[i])) wide |= 1u << i;
      }
      if (__all_sync(0xffffffffu, cur_raw == 0 && wide == 0)) {
        // every row of this warp in 4 bits with ordinary scales: the rows' conversions
        // interleaved, each pair of blocks handed over at once. Two rounds of the
        // same code over four blocks each (unrolled, the code crowds the others' out of
        // the instruction cache); the last block is the rotated tail as it is.
#pragma unroll 1
        for (uint32_t v = 0; v < 2; ++v) {
#pragma unroll
          for (uint32_t half = 0; half < 2; ++half) {
            const uint32_t m = 2 * v + half;
            if (!wait_warp(&S.kv_empty[m], (n & 1) ^ 1, ew)) return false;
#pragma unroll
            for (uint32_t i = 0; i < kFR; ++i)
              *reinterpret_cast<uint4 *>(chunk_dst(i, 2 * m)) =
                  half ? fp4_chunk<2>(rec[i][0].z, sl[i], 0u, false)
                       : fp4_chunk<0>(rec[i][0].x, sl[i], 0u, false);
#pragma unroll
            for (uint32_t i = 0; i < kFR; ++i) {
              uint4 o = half ? fp4_chunk<3>(rec[i][0].w, sl[i], 0u, false)
                             : fp4_chunk<1>(rec[i][0].y, sl[i], 0u, false);
              if (half && v) o = rec[i][2];
              *reinterpret_cast<uint4 *>(chunk_dst(i, 2 * m + 1)) = o;
            }
            fence_proxy_async();
            mbar_arrive(&S.kv_pair[m]);
          }
#pragma unroll
          for (uint32_t i = 0; i < kFR; ++i) {
            rec[i][0] = rec[i][1];
            sl[i] = sh[i];
          }
        }
        return true;
      }
      const __nv_bfloat16 *raw[kFR];
#pragma unroll
      for (uint32_t i = 0; i < kFR; ++i)
        raw[i] = (cur_raw >> i) & 1
                     ? row_src<false>(P, g, tile * kRows + (lt >> 3) + 32 * i) + 8 * j
                     : nullptr;
#pragma unroll 1
      for (uint32_t m = 0; m < 4; ++m) {
        if (!wait_warp(&S.kv_empty[m], (n & 1) ^ 1, ew)) return false;
#pragma unroll 1
        for (uint32_t kb = 2 * m; kb < 2 * m + 2; ++kb)
#pragma unroll
          for (uint32_t i = 0; i < kFR; ++i) {
            uint8_t *dst = chunk_dst(i, kb);
            if ((cur_raw >> i) & 1) {
              cp_async16(dst, raw[i] + 64 * kb, 16u);
            } else {
              const uint4 a = rec[i][0], c = rec[i][1];
              const uint32_t w = kb == 0 ? a.x : kb == 1 ? a.y : kb == 2 ? a.z : kb == 3 ? a.w
                                 : kb == 4 ? c.x : kb == 5 ? c.y : c.z;
              const uint32_t sb = ((kb < 4 ? sl[i] : sh[i]) >> (8 * (kb % 4))) << 24;
              *reinterpret_cast<uint4 *>(dst) = kb == 7 ? rec[i][2] : fp4_chunk<3>(w, sb, 0u, true);
            }
          }
      }
      cp_async_wait_all();
      fence_proxy_async();
#pragma unroll
      for (uint32_t m = 0; m < 4; ++m) mbar_arrive(&S.kv_pair[m]);
      return true;
    };
    // Q (it needs no list): eight TMA boxes of 64 heads x 64 dims, in the
    // 128-byte swizzled K-major layout the S MMAs read. With q_ready the first
    // query's is issued before the wait for the previous launch: the queries, the
    // positions and the rotation tables were then written before that launch
    // began, while the top-k lists and the new raw row were not.
    auto issue_q = [&](uint32_t it) {
      if (FP4) {   // a box per loader warp; heads past the last one read as zeros
        if (lt == 0) mbar_arrive_expect_tx(&S.q_tma, 8 * QBLK);
        if (lane == 0)
          tma_load_3d(S.q + lw * QBLK, &tmap_q, &S.q_tma, (int)(64 * lw), (int)item_h(it),
                      (int)item_q(it));
        return;
      }
      if (lt == 0) {
        const uint32_t qi = item_q(it), hq0 = item_h(it);
        mbar_arrive_expect_tx(&S.q_tma, 8 * QBLK);
#pragma unroll
        for (uint32_t kb = 0; kb < 8; ++kb)
          tma_load_2d(S.q + kb * QBLK, &tmap_q, &S.q_tma, (int)(64 * kb), (int)(qi * kH + hq0));
      }
    };
    // (without q_ready, behind the wait: before the loop all the same for bf16 rows, chunk 648
    // against 660 us; in the loop for 4-bit rows, c4a decode 12.5 against 13.0)
    const bool q_early = (ready || (!FP4 && i0 < n_items)) && rank * kRows < rows_bound(P, item_q(i0));
    if (q_early) issue_q(i0);
    // The loaders' own wait for the previous launch (q_ready). Decode then reads
    // nothing of it before its list or, without one, its first rows, so its first
    // query's coefficients and, but for a list that is read for its length, its
    // geometry are prepared before the wait; prefill scans its lists, so it waits
    // here.
    uint32_t out_it = kNoRow;   // chunks over 4-bit rows: item whose output is to be written
    bool waited = DEC && !ready;
    auto wait_prev = [&]() {
      if (!waited) {
        pdl_wait();
        pdl_trigger();
        waited = true;
      }
    };
    if (kScan || FP4) wait_prev();
    for (uint32_t it = i0; it < n_items; it += i_step) {
      const uint32_t qi = item_q(it);
      if (rank * kRows >= rows_bound(P, qi)) continue;   // no rows for this rank
      if (!wait_warp(&S.q_empty, (qn & 1) ^ 1, ew)) goto done_loader;
      if (!(q_early && it == i0)) issue_q(it);
      {
        // this thread's 16-byte chunks of the tail: chunk lt (+ LT i) of
        // block 7 hold pairs 4 lc .. 4 lc + 3 of head id / 8; their
        // coefficients load while the list is read
        const uint32_t pq = seq_base(P.seq_pos, P.pos0, qi / P.T) + qi % P.T;
        constexpr uint32_t kQC = NH * 8 / WP::LT;   // tail chunks per loader thread
        float co[4 * kQC], si[4 * kQC];
#pragma unroll
        for (uint32_t i = 0; i < kQC; ++i) {
          const uint32_t id = lt + WP::LT * i, h = id >> 3, lc = (id & 7) ^ (h & 7);
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            if (FP4 && P.q_rotated) {   // (not needed, not waited for)
              co[4 * i + e] = si[4 * i + e] = 0.f;
              continue;
            }
            co[4 * i + e] = P.cos[(size_t)pq * 32 + 4 * lc + e];
            si[4 * i + e] = P.sin[(size_t)pq * 32 + 4 * lc + e];
          }
        }
        uint32_t n_list = kNoRow;
        if (DEC && P.ratio == 4) wait_prev();
        if (staged) {
          if (DEC || it == i0) stage_load(qi);   // (else started a few tiles ago)
          if (DEC) fetch_first(qi);
          n_list = stage_list(qi);
          if (n_list == kNoRow) goto done_loader;
        }
        QueryGeo g = query_geo<kScan>(P, qi, rank, C, lane, n_list);
        if (g.t0 >= g.t1) {          // the list is shorter than the bound: nothing to do
          // (Q still lands: wait for it so the buffer is never written twice at once)
          if (!wait_warp(&S.q_tma, qt & 1, ew)) goto done_loader;
          ++qt;
          continue;
        }
        // the first tile's rows start loading before Q is rotated
        wait_prev();
        if (FP4) {
          if (DEC && staged) {   // (fetched already; rows behind the list's end: none)
#pragma unroll
            for (uint32_t i = 0; i < kFR; ++i)
              if (g.t0 * kRows + (lt >> 3) + 32 * i >= g.N)
#pragma unroll
                for (uint32_t v = 0; v < 3; ++v) rec[i][v] = make_uint4(0u, 0u, 0u, 0u);
          } else {
            look_tile(g, g.t0);
            fetch_tile(g, g.t0);
            look_tile(g, g.t0 + g.ts);
          }
          if (!store_tile(g, g.t0, n)) goto done_loader;
        } else if (!issue_tile(g, g.t0, n)) {
          goto done_loader;
        }
        if (!wait_warp(&S.q_tma, qt & 1, ew)) goto done_loader;   // Q landed
        ++qt;
        // rotate the tail (dims 448..511 = block 7) at position p, in place
#pragma unroll
        for (uint32_t i = 0; i < kQC; ++i) {
          if (P.q_rotated) break;
          const uint32_t id = lt + WP::LT * i, h = id >> 3, pc = id & 7;
          uint4 *ptr = reinterpret_cast<uint4 *>(S.q + 7 * QBLK + h * 128 + pc * 16);
          uint4 v = *ptr;
          uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const float c = co[4 * i + e], sn = si[4 * i + e];
            const float x0 = bf16lo(w4[e]), x1 = bf16hi(w4[e]);
            w4[e] = pack_bf16(x0 * c - x1 * sn, x0 * sn + x1 * c);
          }
          *ptr = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        fence_proxy_async();
        mbar_arrive(&S.q_full);
        for (uint32_t tile = g.t0; tile < g.t1; tile += g.ts, ++n) {
          if (tile != g.t0) {
            if (FP4 ? !store_tile(g, tile, n) : !issue_tile(g, tile, n)) goto done_loader;
          }
          if (FP4) {   // (store_tile has handed the tile over)
            if (!DEC && tile == g.t0) {   // the last query's output, then this one's to come
              if (out_it != kNoRow && !write_out(out_it, qn - 1, 2)) goto done_loader;
              out_it = it;
              out_coef(g.p);
            }
            // (past the last tile every row is masked: the registers are dead until then)
            fetch_tile(g, tile + g.ts);
            look_tile(g, tile + 2 * g.ts);
            // the next query's list starts loading after the second tile (or the only one)
            if (!DEC && staged && it + i_step < n_items &&
                (tile == g.t0 + g.ts || (tile == g.t0 && g.t0 + g.ts >= g.t1)))
              stage_load(item_q(it + i_step));
            continue;
          }
          // one arrival per thread once all its rows of the tile landed: the
          // MMA issuer takes the tile whole (waits between the MMAs of one
          // accumulation halve their rate; issuing S pair by pair as the
          // blocks land measured slower)
          if (DEC && P.ratio == 4 && tile == g.t0) {
            // while the rows are on their way: the entry that ends the list, for the softmax
            // warps and the tiles to come; rows behind it (rare) become zeros after all, lest
            // a NaN of theirs meet its weight of 0
            const uint32_t n_end = g.n_w + list_stop(g.tk, P.top_k, g.vis);
            if (n_end < g.N) {
              zero_rows(tile, n_end);
              g.N = n_end;
            }
            if (lt == 0) S.n_end = n_end;
          }
          cp_async_wait_all();
          fence_proxy_async();
          if (tile_kind<DEC, PAGED>(P, g, tile)) {   // (one thread watches the TMA tile)
            if (lt == 0 && !mbar_wait(&S.kv_tma, nk & 1, ew)) goto done_loader;
            ++nk;
          }
          mbar_arrive(&S.kv_full);
        }
      }
      ++qn;
    }
    if (FP4 && !DEC && out_it != kNoRow && !write_out(out_it, qn - 1, 2)) goto done_loader;
  done_loader:
    cp_async_wait_all();
  } else if (warp == WP::MMA) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t idS = idesc_bf16_f32(kRows, NH);
    constexpr uint32_t idPV = idesc_bf16_f32(kRows, kH) | kIdescMajorA_MN | kIdescMajorB_MN;
    const uint32_t q_base = smem_u32(S.q), kv_base = smem_u32(S.kv), p_base = smem_u32(S.p);
    uint32_t n = 0, qn = 0, nk = 0;
    bool ok = true;
    // 4-bit rows: the whole warp runs this code and the instructions themselves
    // elect a thread, every branch is uniform (votes and shuffles), so that the
    // descriptors stay in uniform registers. Issued from a branch on lane 0 each MMA
    // first moves its descriptors there, and the issue, not the tensor core, sets
    // the pace (S^T 2000 to 4000 cycles a tile).
    QueryGeo g_next = {};   // (as in the softmax warps)
    uint32_t gn = 0;
    for (uint32_t it = i0; FP4 && it < n_items && ok; it += i_step) {
      const uint32_t qi = item_q(it), rank_u = uniform(rank);
      const bool ahead = !DEC && !staged && it != i0;
      if (!ahead && uniform(rank_u * kRows >= rows_bound(P, qi))) continue;
      uint32_t n_list = kNoRow;
      if (staged) {
        const uint32_t gb = list_half(gn);
        ok = mbar_wait_issue(&S4.geo_full[gb], list_phase(gn), ew);
        if (!ok) break;
        n_list = list_end(gb);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S4.geo_empty[gb]);   // (this warp needs no more of it)
        ++gn;
      }
      const QueryGeo g = ahead ? g_next : query_geo<kScan>(P, qi, rank, C, lane, n_list);
      const uint32_t t0 = uniform(g.t0), t1 = uniform(g.t1), ts = uniform(g.ts);
      if (t0 >= t1) continue;
      const bool tma0 = uniform(tile_kind<DEC, true, FP4>(P, g, t0)) != 0;   // (only a first tile)
      const uint32_t qd = desc_lo(q_base), kd = desc_lo(kv_base), pd = desc_lo(p_base);
      ok = mbar_wait_issue(&S.q_full, qn & 1, ew);
      for (uint32_t tile = t0; ok && tile < t1; tile += ts, ++n) {
        const bool first = tile == t0, last = tile + ts >= t1;
        if (first && tma0) ok = mbar_wait_issue(&S.kv_tma, nk++ & 1, ew);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (uint32_t m = 0; m < 4; ++m) {   // S^T starts while the tile's last blocks convert
          ok = ok && mbar_wait_issue(&S.kv_pair[m], n & 1, ew);
          if (!ok) break;
#pragma unroll
          for (uint32_t kb = 2 * m; kb < 2 * m + 2; ++kb)
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
              mma_bf16_elect(tmS, desc_at(kd + (kb * kKBlk + kk * 32) / 16 + desc_lbo(16), kDescHiK),
                             desc_at(qd + (kb * QBLK + kk * 32) / 16 + desc_lbo(16), kDescHiK), idS,
                             (kb | kk) ? 1u : 0u);
        }
        if (!ok) break;
        mma_commit_elect(&S.s_full);
        if (last) mma_commit_elect(&S.q_empty);
        if (!DEC && !staged && last && it + i_step < n_items)
          g_next = query_geo<kScan>(P, item_q(it + i_step), rank, C, lane);
        ok = mbar_wait_issue(&S.p_full, n & 1, ew);
        if (ok && first) ok = mbar_wait_issue(&S.o_empty, (qn & 1) ^ 1, ew);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc0 = first ? 0u : 1u;
#pragma unroll 1
        for (uint32_t m = 0; m < 4; ++m) {
#pragma unroll
          for (uint32_t kk = 0; kk < 8; ++kk)
            mma_bf16_elect(tmO + m * kH,
                           desc_at(kd + (2 * m * kKBlk + kk * 2048) / 16 + desc_lbo(kKBlk), kDescHiK),
                           desc_at(pd + kk * 2048 / 16 + desc_lbo(8192), kDescHiK), idPV,
                           kk ? 1u : acc0);
          mma_commit_elect(&S.kv_empty[m]);
        }
        constexpr uint32_t idL = idesc_bf16_f32(kRows, kH) | kIdescMajorB_MN;
#pragma unroll
        for (uint32_t kk = 0; kk < 8; ++kk)
          mma_bf16_ta_elect(tmL, tmOnes, desc_at(pd + kk * 2048 / 16 + desc_lbo(8192), kDescHiK),
                            idL, kk ? 1u : acc0);
        mma_commit_elect(&S.p_empty);
        if (last) mma_commit_elect(&S.o_full);
      }
      ++qn;
    }
    for (uint32_t it = i0; !FP4 && it < n_items && ok; it += i_step) {
      const uint32_t qi = item_q(it);
      if (rank * kRows >= rows_bound(P, qi)) continue;
      const QueryGeo g = query_geo<kScan>(P, qi, rank, C, lane);
      if (g.t0 >= g.t1) continue;
      if (lane == 0) {
        ok = mbar_wait(&S.q_full, qn & 1, ew);
        for (uint32_t tile = g.t0; ok && tile < g.t1; tile += g.ts, ++n) {
          const bool first = tile == g.t0, last = tile + g.ts >= g.t1;
          ok = mbar_wait(&S.kv_full, n & 1, ew);
          if (ok && tile_kind<DEC, PAGED>(P, g, tile)) ok = mbar_wait(&S.kv_tma, nk++ & 1, ew);
          if (!ok) break;
          tc_fence_after();
          for (uint32_t kb = 0; kb < 8; ++kb)
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
              mma_bf16(tmS, sdesc_sw128(kv_base + kb * kKBlk + kk * 32),
                       sdesc_sw128(q_base + kb * QBLK + kk * 32), idS, (kb | kk) ? 1u : 0u);
          mma_commit(&S.s_full);
          if (last) mma_commit(&S.q_empty);
          ok = mbar_wait(&S.p_full, n & 1, ew);
          if (ok && first) ok = mbar_wait(&S.o_empty, (qn & 1) ^ 1, ew);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (uint32_t m = 0; m < 4; ++m) {
#pragma unroll
            for (uint32_t kk = 0; kk < 8; ++kk) {
              const uint64_t ad = sdesc_sw128_mn(kv_base + 2 * m * kKBlk + kk * 2048, kKBlk, 1024);
              const uint64_t bd = sdesc_sw128_mn(p_base + kk * 2048, 8192, 1024);
              mma_bf16(tmO + m * kH, ad, bd, idPV, (first && kk == 0) ? 0u : 1u);
            }
            mma_commit(&S.kv_empty[m]);
          }
          // per-head row sums of P on the tensor core: every row of L = 1^T P^T
          constexpr uint32_t idL = idesc_bf16_f32(kRows, kH) | kIdescMajorB_MN;
#pragma unroll
          for (uint32_t kk = 0; kk < 8; ++kk)
            mma_bf16_ta(tmL, tmOnes, sdesc_sw128_mn(p_base + kk * 2048, 8192, 1024), idL,
                        (first && kk == 0) ? 0u : 1u);
          mma_commit(&S.p_empty);
          if (last) mma_commit(&S.o_full);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      n = __shfl_sync(0xffffffffu, n, 0);
      ++qn;
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const uint32_t sq = warp & 3, hh = warp >> 2;   // TMEM quarter; half of the heads (4-bit rows)
    const uint32_t r = 32 * sq + lane;       // tile row / TMEM lane, then dim within a block
    const uint32_t lane_base = (sq * 32) << 16;
    // heads of this thread: NPT parts of HB, the first from head hb0
    constexpr uint32_t HB = FP4 ? NH / 2 : 32, NPT = FP4 ? 1 : NHF;
    const uint32_t hb0 = FP4 ? hh * HB : 0u;
    uint32_t n = 0, qn = 0, sm_phase = 0;
    // P of heads hb .. hb + HB - 1 of row r from their scores `a` with the current
    // running maxima; flags a score above its head's maximum by more than 2^8
    auto p_half = [&](bool valid, const uint32_t (&a)[HB], uint32_t hb, bool &flag) {
      uint8_t *prow = S.p + (r >> 3) * 1024 + (r & 7) * 128;
      float top = -INFINITY;
#pragma unroll
        for (uint32_t c4 = 0; c4 < HB / 8; ++c4) {
          uint32_t w4[4];
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const uint32_t hl = 8 * c4 + 2 * e, h = hb + hl;
            const float t0 = fmaf(__uint_as_float(a[hl]), P.c2, -S.mref[h]);
            const float t1 = fmaf(__uint_as_float(a[hl + 1]), P.c2, -S.mref[h + 1]);
            if (FP4) top = fmaxf(top, fmaxf(t0, t1));
            else flag |= valid && (t0 > kRaiseLog2 || t1 > kRaiseLog2);
            w4[e] = valid ? pack_bf16(ex2_approx(t0), ex2_approx(t1)) : 0u;
          }
          *reinterpret_cast<uint4 *>(prow + (((hb / 8 + c4) ^ (r & 7)) << 4)) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      if (FP4) flag |= valid && top > kRaiseFp4;
    };
    // P row r from the scores in TMEM; returns whether a score exceeds its
    // head's running maximum by more than 2^8
    auto write_p = [&](bool valid) {
      bool flag = false;
#pragma unroll
      for (uint32_t hf = 0; hf < NPT; ++hf) {
        uint32_t a[HB];
        tmem_ld(tmS + lane_base + hb0 + HB * hf, a);
        tmem_ld_wait();
        p_half(valid, a, hb0 + HB * hf, flag);
      }
      return flag;
    };
    // chunks over 4-bit rows without a list: the next query's geometry, found while
    // waiting for a last tile
    QueryGeo g_next = {};
    uint32_t gn = 0;
    for (uint32_t it = i0; it < n_items; it += i_step) {
      const uint32_t qi = item_q(it), hq0 = item_h(it);
      const bool ahead = FP4 && !DEC && !staged && it != i0;
      const bool maybe = ahead || rank * kRows < rows_bound(P, qi);
      uint32_t n_list = kNoRow, gb = 0;
      if (staged && maybe) {
        gb = list_half(gn);
        if (!wait_warp(&S4.geo_full[gb], list_phase(gn), ew)) goto done_softmax;
        n_list = list_end(gb);
        ++gn;
      }
      QueryGeo g = g_next;
      if (maybe && !ahead) g = query_geo<kScan>(P, qi, rank, C, lane, n_list);
      const bool has_tiles = maybe && g.t0 < g.t1;
      // the rotation coefficients of this thread's tail dim in the direct
      // output (dim 384 + r of the last chunk), loaded while the tiles run
      float ep_co = 1.f, ep_si = 0.f;
      if (!(dec && C > 1) && !(FP4 && !DEC) && has_tiles && 384 + r >= (uint32_t)kNope) {
        const uint32_t fi = (384 + r - kNope) >> 1;
        ep_co = P.cos[(size_t)g.p * 32 + fi];
        ep_si = P.sin[(size_t)g.p * 32 + fi];
      }
      for (uint32_t tile = g.t0; has_tiles && tile < g.t1; tile += g.ts, ++n) {
        const bool first = tile == g.t0;
        const uint32_t row = tile * kRows + r;
        bool valid = row < g.n_w;
        if (!valid && row < g.N)
          valid = P.ratio != 4 || (FP4 ? S4.rows[gb * kList + (row - g.n_w)] != kNoRow
                                       : (uint32_t)g.tk[row - g.n_w] < g.vis);
        if (FP4 && !DEC && !staged && tile + g.ts >= g.t1 && it + i_step < n_items)
          g_next = query_geo<kScan>(P, item_q(it + i_step), rank, C, lane);
        if (!wait_warp(&S.s_full, n & 1, ew)) goto done_softmax;
        tc_fence_after();
        if (DEC && !FP4 && P.ratio == 4) {
          // (kv_full's phase is complete: the test orders the loaders' store of n_end before this)
          if (first) (void)mbar_test_wait(&S.kv_full, n & 1);
          valid = valid && row < S.n_end;
        }
        if (first) {
          // running maxima start at the exact per-head maxima of the first
          // tile's scaled scores: warp maxima of order-keyed values, then the
          // largest of the four warps. P of this tile then has no score above
          // its maximum (no raise to check).
          uint32_t *tkey = reinterpret_cast<uint32_t *>(&S.tmax[0][0]);   // [4][kH]
          if constexpr (FP4) {
            // This thread's scores stay in registers for P; after one barrier each warp
            // takes its heads' maxima from the four quarters itself (the warps with
            // the same heads store the same values).
            uint32_t a0[HB];
            tmem_ld(tmS + lane_base + hb0, a0);
            tmem_ld_wait();
            const uint32_t row0 = tile * kRows;
            const bool valid0 = row0 < g.n_w ||
                (row0 < g.N && (P.ratio != 4 || S4.rows[gb * kList + (row0 - g.n_w)] != kNoRow));
            if (valid0) {   // (the same for every thread) the tile's first row is the reference
              if (r == 0)
#pragma unroll
                for (uint32_t h = 0; h < HB; h += 4)
                  *reinterpret_cast<float4 *>(&S.mref[hb0 + h]) =
                      make_float4(__uint_as_float(a0[h]) * P.c2, __uint_as_float(a0[h + 1]) * P.c2,
                                  __uint_as_float(a0[h + 2]) * P.c2, __uint_as_float(a0[h + 3]) * P.c2);
              if (threadIdx.x == 0) S.flagcnt[n % 3] = 0;
            } else {
            uint32_t mine = 0u;
#pragma unroll
            for (uint32_t h = 0; h < HB; ++h) {
              const uint32_t u = __float_as_uint(__uint_as_float(a0[h]) * P.c2);
              const uint32_t key = valid ? ((u & 0x80000000u) ? ~u : (u | 0x80000000u)) : 0u;
              const uint32_t mk = redux_max_u32(key);
              if (lane == h) mine = mk;
            }
            if (lane < HB) tkey[sq * kH + hb0 + lane] = mine;
            if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
            const uint32_t hm = hb0 + (lane & (HB - 1));
            const uint32_t mk = max(max(tkey[0 * kH + hm], tkey[1 * kH + hm]),
                                    max(tkey[2 * kH + hm], tkey[3 * kH + hm]));
            const bool any_valid = mk != 0u;   // a valid row has a key above 0 for every head
            const float mx = __uint_as_float((mk & 0x80000000u) ? (mk & 0x7fffffffu) : ~mk);
            if (lane < HB) S.mref[hm] = any_valid ? mx : kNoMax;
            if (threadIdx.x == 0) S.flagcnt[n % 3] = 0;
            }
            if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
            // (then as every tile: P, with a raise where a score is far above)
          } else {
          // eight heads per step of a short loop: this runs once per query,
          // its code is fetched cold, and an unrolled form measured ~2 us of
          // instruction fetch
#pragma unroll 1
          for (uint32_t c = 0; c < (uint32_t)NH; c += 8) {
            uint32_t a8[8];
            tmem_ld8(tmS + lane_base + c, a8);
            tmem_ld_wait();
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
              const uint32_t u = __float_as_uint(__uint_as_float(a8[j]) * P.c2);
              const uint32_t key = valid ? ((u & 0x80000000u) ? ~u : (u | 0x80000000u)) : 0u;
              const uint32_t mk = redux_max_u32(key);
              if (lane == ((c + j) & 31)) tkey[sq * kH + c + j] = mk;
            }
          }
          if (threadIdx.x == 0) S.flagcnt[(n + 1) % 3] = 0;   // the next tile's raise count
          if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
          const uint32_t k0 = max(max(tkey[0 * kH], tkey[1 * kH]), max(tkey[2 * kH], tkey[3 * kH]));
          const bool any_valid = k0 != 0u;   // a valid row has a key above 0 for every head
          if (threadIdx.x < (uint32_t)NH) {
            const uint32_t mk = max(max(tkey[0 * kH + r], tkey[1 * kH + r]),
                                    max(tkey[2 * kH + r], tkey[3 * kH + r]));
            const float mx = __uint_as_float((mk & 0x80000000u) ? (mk & 0x7fffffffu) : ~mk);
            S.mref[r] = any_valid ? mx : kNoMax;
          }
          if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
          if (!wait_warp(&S.p_empty, (n & 1) ^ 1, ew)) goto done_softmax;
          // the scores (S stays until this tile's P is done)
          bool unused = false;
          if (NHF == 2) {
            uint32_t a0[32], a1[32];
            tmem_ld32(tmS + lane_base, a0);
            tmem_ld32(tmS + lane_base + 32, a1);
            tmem_ld_wait();
            p_half(valid, *reinterpret_cast<uint32_t(*)[HB]>(a0), 0, unused);
            p_half(valid, *reinterpret_cast<uint32_t(*)[HB]>(a1), 32, unused);
          } else {
            uint32_t a0[32];
            tmem_ld32(tmS + lane_base, a0);
            tmem_ld_wait();
            p_half(valid, *reinterpret_cast<uint32_t(*)[HB]>(a0), 0, unused);
          }
          fence_proxy_async();
          tc_fence_before();
          mbar_arrive(&S.p_full);
          continue;
          }
        }
        // P of this tile (the previous PV must be done with the buffer)
        if (!wait_warp(&S.p_empty, (n & 1) ^ 1, ew)) goto done_softmax;
        const bool flag = write_p(valid);
        const uint32_t fc = n % 3;
        if (threadIdx.x == 0) S.flagcnt[(n + 1) % 3] = 0;
        if (flag) atomicAdd(&S.flagcnt[fc], 1u);
        if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
        if (S.flagcnt[fc] != 0) {
          // rare path: exact tile max per head, raise the running max, rescale
          // O and L, rewrite P
#pragma unroll 1
          for (uint32_t hf = 0; hf < (FP4 ? HB / 8 : NPT); ++hf) {
            constexpr uint32_t W = FP4 ? 8 : HB;   // (short code where it runs rarely)
            const uint32_t hb = hb0 + W * hf;
            uint32_t a[W];
            tmem_ld(tmS + lane_base + hb, a);
            tmem_ld_wait();
#pragma unroll
            for (uint32_t h = 0; h < W; ++h) {
              const float v = warp_max(valid ? __uint_as_float(a[h]) * P.c2 : -INFINITY);
              if (lane == h) S.tmax[sq][hb + h] = v;
            }
          }
          if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
          if (threadIdx.x < (uint32_t)NH) {
            const float M = fmaxf(fmaxf(S.tmax[0][r], S.tmax[1][r]), fmaxf(S.tmax[2][r], S.tmax[3][r]));
            const float mo = S.mref[r], mn = fmaxf(mo, M);
            S.alpha[r] = exp2f(mo - mn);
            S.mref[r] = mn;
          }
          if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
          if (!first) {
#pragma unroll 1
            for (uint32_t m = FP4 ? hh : 0u; m < 5 * (uint32_t)NHF; m += FP4 ? 2 : 1) {   // O^T (4 dim blocks) then L
              uint32_t a[32];
              const uint32_t blk = m / NHF, hf = m % NHF;
              const uint32_t ta = (blk < 4 ? tmO + blk * kH : tmL) + 32 * hf + lane_base;
              tmem_ld32(ta, a);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < 32; ++h)
                a[h] = __float_as_uint(__uint_as_float(a[h]) * S.alpha[32 * hf + h]);
              tmem_st32(ta, a);
            }
            tmem_st_wait();
          }
          write_p(valid);
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&S.p_full);
      }
      if (staged && maybe) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S4.geo_empty[gb]);
      }
      if (FP4 && !DEC) {
        out_coef(g.p);
        if (!write_out(it, qn, 0)) goto done_softmax;
        ++qn;
        continue;
      }
      // ---- query end: per-head sums (any lane of L), then the output
      if (has_tiles) {
        if (!wait_warp(&S.o_full, qn & 1, ew)) goto done_softmax;
        tc_fence_after();
        if (warp < (uint32_t)NHF) {   // every row of L holds the sums: warp w keeps heads 32w + lane
          uint32_t a[32];
          tmem_ld32(tmL + lane_base + 32 * warp, a);
          tmem_ld_wait();
          float l = 0.f;
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i)
            if (lane == i) l = __uint_as_float(a[i]);
          S.lsh[32 * warp + lane] = l;
          S.linv[32 * warp + lane] = l > 0.f ? 1.f / l : 0.f;
        }
      }
      if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
      if (dec && C > 1) {
        // (max, sum) of this rank for the cluster merge; O follows from TMEM
        if (threadIdx.x < (uint32_t)NH) {
          float *ml = P.ml + ((size_t)(vq * C + rank) * NH + r) * 2;
          ml[0] = has_tiles && !(S.mref[r] <= kNoMax) ? S.mref[r] : -INFINITY;
          ml[1] = has_tiles ? S.lsh[r] : 0.f;
        }
        if (threadIdx.x == 0) S.has_tiles = has_tiles ? 1u : 0u;
      } else {
        // normalise, rotate the tail back by -p and store bf16 pairs straight
        // from registers, four 128-dim chunks (no staging, no barrier)
        // 1 / L per head, for the four chunks (from shared memory with 4-bit rows,
        // whose larger block has fewer registers per thread)
        float li[FP4 ? 1 : NH];
        if (!FP4) {
#pragma unroll
          for (int h = 0; h < NH; ++h) li[FP4 ? 0 : h] = S.linv[h];
        }
        auto linv = [&](int h) { return FP4 ? S.linv[h] : li[FP4 ? 0 : h]; };
        const bool odd = lane & 1;
#pragma unroll 1
        for (uint32_t m = FP4 ? 2 * hh : 0u; m < (FP4 ? 2 * hh + 2 : 4u); ++m) {
          const bool rot = m == 3 && r >= 64;   // warp-uniform: the rotated tail dims
          const float co = ep_co, si = ep_si;   // (the pair's coefficients: both lanes)
          __nv_bfloat16 *o = P.out + ((size_t)qi * HQ + hq0) * kD + m * 128;
          // (4-bit rows: the two head halves one after the other, for the registers)
          constexpr uint32_t NB = FP4 ? 1 : NHF;
          uint32_t ab[NB][32];
          if (!FP4) {
#pragma unroll
            for (uint32_t hf = 0; hf < (uint32_t)NHF; ++hf)
              tmem_ld32(tmO + lane_base + m * kH + 32 * hf, ab[FP4 ? 0 : hf]);
            tmem_ld_wait();
          }
#pragma unroll
          for (uint32_t hf = 0; hf < (uint32_t)NHF; ++hf) {
            uint32_t(&a32)[32] = ab[FP4 ? 0 : hf];
            if (FP4) {
              tmem_ld32(tmO + lane_base + m * kH + 32 * hf, a32);
              tmem_ld_wait();
            }
#pragma unroll
            for (int h = 0; h < 32; h += 2) {
              const float v0 = __uint_as_float(a32[h]) * linv(32 * hf + h);
              const float v1 = __uint_as_float(a32[h + 1]) * linv(32 * hf + h + 1);
              // lanes 2i, 2i + 1 hold dims d, d + 1 of heads h, h + 1: one
              // swap gives the even lane head h's pair and the odd lane head
              // h + 1's, rotated in place and stored as one bf16 pair
              const float recv = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
              float x0 = odd ? recv : v0, x1 = odd ? v1 : recv;
              if (rot) {   // (x0, x1) -> (x0 c + x1 s, -x0 s + x1 c)
                const float y0 = x0 * co + x1 * si, y1 = -x0 * si + x1 * co;
                x0 = y0;
                x1 = y1;
              }
              const uint32_t row = 32 * hf + h + (odd ? 1u : 0u);
              if (!FP4 || hq0 + row < HQ)
                *reinterpret_cast<uint32_t *>(o + (size_t)row * kD + (r & ~1u)) = pack_bf16(x0, x1);
            }
          }
        }
      }
      if (has_tiles) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.o_empty);
        ++qn;
      }
      // keep the shared sums alive until every thread has read them
      if (!sync_group(&S.sm_bar, sm_phase, ew)) goto done_softmax;
    }
  done_softmax:;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (dec && C > 1) {
    if constexpr (FP4) {
      // this rank's O / L as [NH heads][512] fp32 straight to the workspace: warp w reads
      // TMEM lanes 32 (w % 4) .. + 31 (dims) for 32 heads of its dim blocks (64 heads:
      // two of the four blocks, 32 heads: one), a 128-byte line per head and store
      if (warp < 16) {
        float *dst = reinterpret_cast<float *>(P.part) + ((size_t)vq * C + rank) * NH * kD;
        const uint32_t qw = warp & 3, hf = NHF == 2 ? (warp >> 2) & 1 : 0u;
        const uint32_t m0 = NHF == 2 ? 2 * (warp >> 3) : warp >> 2, m1 = m0 + (NHF == 2 ? 2 : 1);
        const bool had = S.has_tiles != 0;
#pragma unroll 1
        for (uint32_t m = m0; m < m1; ++m) {
          uint32_t a[32];
          if (had) {
            tmem_ld32(tmO + ((32 * qw) << 16) + m * kH + 32 * hf, a);
            tmem_ld_wait();
          }
          float *to = dst + (size_t)(32 * hf) * kD + m * 128 + 32 * qw + lane;
#pragma unroll
          for (int h = 0; h < 32; ++h)
            to[(size_t)h * kD] = had ? __uint_as_float(a[h]) * S.linv[32 * hf + h] : 0.f;
        }
      }
    } else {
    // this rank's O / L as [NH heads][512] bf16 straight to the workspace.
    // Warp w reads TMEM lanes 32 (w % 4) .. + 31 (dims) for heads 32 hf ..
    // + 31 of dim blocks m0 .. m1 - 1 (64 heads: hf = w / 4, every block; 32
    // heads: hf = 0, two blocks per warp); lanes 2i, 2i + 1 hold dims d, d + 1:
    // the even lane stores the bf16 pair of head h, the odd lane that of head
    // h + 1 (one swap each)
    if (warp < 8) {
      __nv_bfloat16 *dst = P.part + ((size_t)vq * C + rank) * NH * kD;
      const uint32_t qw = warp & 3, hf = NHF == 2 ? warp >> 2 : 0u, dl = 32 * qw + lane;
      const uint32_t m0 = NHF == 2 ? 0u : 2 * (warp >> 2), m1 = NHF == 2 ? 4u : m0 + 2;
      const bool had = S.has_tiles != 0, odd = lane & 1;
      float li[32];
#pragma unroll
      for (int h = 0; h < 32; ++h) li[h] = had ? S.linv[32 * hf + h] : 0.f;
#pragma unroll 1
      for (uint32_t m = m0; m < m1; ++m) {
        uint32_t a[32];
        if (had) {
          tmem_ld32(tmO + ((32 * qw) << 16) + m * kH + 32 * hf, a);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int h = 0; h < 32; ++h) a[h] = 0u;
        }
#pragma unroll
        for (int h = 0; h < 32; h += 2) {
          const float v0 = __uint_as_float(a[h]) * li[h], v1 = __uint_as_float(a[h + 1]) * li[h + 1];
          const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
          const uint32_t row = 32 * hf + h + (odd ? 1 : 0);
          const uint32_t w = odd ? pack_bf16(other, v1) : pack_bf16(v0, other);
          *reinterpret_cast<uint32_t *>(dst + (size_t)row * kD + m * 128 + (dl & ~1u)) = w;
        }
      }
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == WP::MMA) tmem_dealloc(tmem, 512);
  if (dec && C > 1) {
    cluster_sync_all();   // every rank's O and (max, sum) are in the workspace
    if (warp < (FP4 ? 16 : 8)) {
      if (C <= 8)
        merge_heads<8, NH, FP4>(P, S, vq, rank, C, ew);
      else
        merge_heads<kMaxCluster, NH, FP4>(P, S, vq, rank, C, ew);
    }
  }
}

// Largest number of clusters of each size (1..16) that fit on the device at
// once, per device; 0 = not yet asked, -1 = the size cannot be launched.
std::atomic<int> g_max_clusters[64][kMaxCluster + 1];
// Per device: 1 = cluster sizes above 8 allowed for the kernel, -1 = refused.
std::atomic<int> g_nonportable[64];

int max_active_clusters(uint32_t C, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int v = g_max_clusters[dev][C].load(std::memory_order_relaxed);
  if (v != 0) return v;
  if (C > 8) {
    int np = g_nonportable[dev].load(std::memory_order_relaxed);
    if (np == 0) {
      auto allow = [](auto *k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
               cudaSuccess;
      };
      np = allow(attn_tc_kernel<true, false, false, kNhDec>) &&
                   allow(attn_tc_kernel<true, true, false, kNhDec>)
               ? 1
               : -1;
      (void)cudaGetLastError();
      g_nonportable[dev].store(np, std::memory_order_relaxed);
    }
    if (np < 0) {
      g_max_clusters[dev][C].store(-1, std::memory_order_relaxed);
      return -1;
    }
  }
  // (the size may be asked for before the first launch; the limit is every launch's)
  (void)cudaFuncSetAttribute(attn_tc_kernel<true, false, false, kNhDec>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(C * 64);
  cfg.blockDim = dim3(Warps<false>::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&v, attn_tc_kernel<true, false, false, kNhDec>, &cfg) != cudaSuccess || v <= 0) {
    (void)cudaGetLastError();
    // beyond the portable size an unanswered query means the size is not used
    v = C > 8 ? -1 : num_sms() / (int)C;
  }
  if (v == 0) v = 1;
  g_max_clusters[dev][C].store(v, std::memory_order_relaxed);
  return v;
}

// Cluster size for a decode batch: fewest rounds of tiles, counting a whole
// extra round for every wave of clusters beyond the first (a wave also pays
// the query load and the merge, modelled as two tiles). Ties: fewer CTAs.
uint32_t pick_cluster(uint32_t n_tiles, uint32_t n_q, size_t smem) {
  uint32_t best = 1, best_cost = 0xffffffffu;
  const uint32_t cmax = n_tiles < kMaxCluster ? (n_tiles ? n_tiles : 1u) : kMaxCluster;
  for (uint32_t C = 1; C <= cmax; ++C) {
    const int actv = max_active_clusters(C, smem);
    if (actv < 1) continue;
    const uint32_t act = (uint32_t)actv;
    const uint32_t waves = (n_q + act - 1) / act, tiles = (n_tiles + C - 1) / C;
    const uint32_t cost = waves * (tiles + 2);
    if (cost < best_cost) {
      best = C;
      best_cost = cost;
    }
  }
  return best;
}

// Process-wide cluster size forced by ds4a_set_decode_cluster (0: automatic).
std::atomic<uint32_t> g_force_cluster{0};

// The cluster size a decode launch uses: the forced size (clamped to the
// query's tile count and 16) when the device can launch it, else pick_cluster.
uint32_t decode_cluster(uint32_t rows_max, uint32_t n_q, size_t smem) {
  const uint32_t n_tiles = (rows_max + kRows - 1) / kRows;
  const uint32_t cmax = n_tiles < kMaxCluster ? (n_tiles ? n_tiles : 1u) : kMaxCluster;
  uint32_t f = g_force_cluster.load(std::memory_order_relaxed);
  if (f) {
    if (f > cmax) f = cmax;
    if (max_active_clusters(f, smem) >= 1) return f;
  }
  return pick_cluster(n_tiles, n_q, smem);
}

// The same for the 4-bit kernels (their block and shared memory are larger): clusters
// of C CTAs that run at once, 0 where the size cannot be launched.
int max_active_clusters_fp4(uint32_t C) {
  static std::atomic<int> seen[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int v = seen[dev][C].load(std::memory_order_relaxed);
  if (v != 0) return v - 1;
  auto *k = attn_tc_kernel<true, true, true, kH>;
  const int smem = (int)sizeof(SmemFp4) + 1024;
  bool ok = true;
  for (auto *f : {k, attn_tc_kernel<true, true, true, kNhDec>}) {
    ok = ok && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
    if (C > 8)
      ok = ok && cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(C * 64);
  cfg.blockDim = dim3(Warps<true>::THREADS);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  v = 0;
  if (!ok || cudaOccupancyMaxActiveClusters(&v, k, &cfg) != cudaSuccess || v < 0) {
    (void)cudaGetLastError();
    v = C > 8 ? 0 : num_sms() / (int)C;   // (an unanswered query)
  }
  if (C == 1 && v < 1) v = 1;
  seen[dev][C].store(v + 1, std::memory_order_relaxed);
  return v;
}

// Heads per CTA and cluster size of a decode launch over 4-bit rows: the pair with
// the least time by what was measured on this part (64 heads, 1 to 76 sequences, 5 to 33
// tiles): a tile takes 2.5 us for 32 heads as for 64, and beside its tiles a wave of
// clusters takes, in tenths of a tile, 33 (32 heads, no merge) .. 54 (64 heads merged by
// 2 or 3 CTAs). A second wave takes as long as the first. Half the heads per CTA
// save the output exchange (c4a, 8 sequences: 12.6 us against 14.1), until they no
// longer fit at once (c128a, 32 sequences at 524,288: 64 us against 37).
struct DecodePlan {
  uint32_t nh, cluster;
};
DecodePlan fp4_decode_plan(uint32_t n_heads, uint32_t rows_max, uint32_t n_q) {
  const uint32_t n_tiles = (rows_max + kRows - 1) / kRows;
  uint32_t cmax = n_tiles < kMaxCluster ? (n_tiles ? n_tiles : 1u) : kMaxCluster;
  const uint32_t force = g_force_cluster.load(std::memory_order_relaxed);
  DecodePlan best{(uint32_t)kNhDec, 1};
  uint64_t best_cost = ~0ull;
  for (uint32_t nh : {(uint32_t)kNhDec, (uint32_t)kH}) {
    if (nh == kH && n_heads <= (uint32_t)kNhDec) continue;
    const uint64_t n_vq = (uint64_t)n_q * ((n_heads + nh - 1) / nh);
    for (uint32_t C = 1; C <= cmax; ++C) {
      if (force && C != (force < cmax ? force : cmax) && max_active_clusters_fp4(force < cmax ? force : cmax) > 0)
        continue;
      const int act = max_active_clusters_fp4(C);
      if (act < 1) continue;
      const bool half = nh == (uint32_t)kNhDec;
      const uint32_t fixed = C == 1 ? (half ? 33 : 42) : C <= 3 ? (half ? 44 : 54) : (half ? 39 : 45);
      const uint64_t waves = (n_vq + act - 1) / act, tiles = (n_tiles + C - 1) / C;
      const uint64_t cost = waves * (10 * tiles + fixed);
      if (cost < best_cost) {
        best = DecodePlan{nh, C};
        best_cost = cost;
      }
    }
  }
  return best;
}

}  // namespace

void attn_tc_force_cluster(uint32_t C) {
  g_force_cluster.store(C > kMaxCluster ? kMaxCluster : C, std::memory_order_relaxed);
}

uint32_t attn_tc_decode_cluster(uint32_t rows_max, uint32_t n_q, uint32_t n_heads, bool fp4) {
  if (fp4) return fp4_decode_plan(n_heads, rows_max, n_q).cluster;
  return decode_cluster(rows_max, n_q * Heads<kNhDec>::HG, sizeof(Smem) + 1024);
}

// (4-bit rows: any number of heads)
bool attn_tc_supported(int dtype, uint32_t H, uint32_t D, uint32_t n_rot, bool fp4) {
  return dtype == DS4A_BF16 && (fp4 || H == (uint32_t)kH) && D == (uint32_t)kD && n_rot == 64;
}

// Error word, then (decode) room for the partials of the largest cluster.
size_t attn_tc_ws_bytes(uint32_t batch, uint32_t T, uint32_t rows_max, uint32_t n_heads, bool fp4) {
  if (T != 1) return 256;
  const uint32_t n_tiles = (rows_max + kRows - 1) / kRows;
  const uint32_t cmax = n_tiles < kMaxCluster ? (n_tiles ? n_tiles : 1u) : kMaxCluster;
  if (cmax < 2) return 256;
  const uint32_t heads = (n_heads + kH - 1) / kH * kH;   // whole groups
  const size_t elem = fp4 ? sizeof(float) : sizeof(__nv_bfloat16);
  return 256 + (size_t)batch * cmax * heads * (kD * elem + 2 * sizeof(float));
}

cudaError_t launch_attention_tc(const AttnArgs &a, uint32_t rows_max, int *err, cudaStream_t s) {
  TcAttnParams P;
  P.ratio = a.ratio;
  P.batch = a.batch;
  P.T = a.T;
  P.pos0 = a.pos0;
  P.cap_raw = a.cap_raw;
  P.comp_cap = a.comp_cap;
  P.map = a.map;
  P.seq_pos = a.seq_pos;
  P.n_comp = a.n_comp;
  P.top_k = a.top_k;
  P.n_q = a.batch * a.T;
  P.c2 = a.scale * 1.4426950408889634f;
  P.q_rotated = a.q_rotated ? 1u : 0u;
  P.q_ready = a.q_ready ? 1u : 0u;
  P.q = static_cast<const __nv_bfloat16 *>(a.q);
  P.ring = static_cast<const __nv_bfloat16 *>(a.ring);
  P.chunk = static_cast<const __nv_bfloat16 *>(a.chunk);
  P.comp = static_cast<const __nv_bfloat16 *>(a.comp);
  P.topk = a.topk;
  P.cos = a.cos;
  P.sin = a.sin;
  P.out = static_cast<__nv_bfloat16 *>(a.out);
  P.part = reinterpret_cast<__nv_bfloat16 *>(static_cast<uint8_t *>(a.ws) + 256);
  P.ml = nullptr;
  P.err = err;
  const size_t smem = (a.fp4 ? sizeof(SmemFp4) : sizeof(Smem)) + 1024;
  // paged rows: an instantiation of its own, so the contiguous gathers carry
  // no table code
  const bool paged = a.map.table != nullptr, fp4 = a.fp4;
  const DecodePlan plan = fp4 && a.T == 1 ? fp4_decode_plan(a.n_heads, rows_max, P.n_q)
                                          : DecodePlan{(uint32_t)kNhDec, 0u};
  const uint32_t nh = a.T > 1 ? (uint32_t)kH : plan.nh;
  auto *k_dec = fp4     ? (nh == kH ? attn_tc_kernel<true, true, true, kH>
                                    : attn_tc_kernel<true, true, true, kNhDec>)
                : paged ? attn_tc_kernel<true, true, false, kNhDec>
                        : attn_tc_kernel<true, false, false, kNhDec>;
  auto *k_pf = fp4     ? attn_tc_kernel<false, true, true, kH>
               : paged ? attn_tc_kernel<false, true, false, kH>
                       : attn_tc_kernel<false, false, false, kH>;
  P.n_heads = a.n_heads;
  P.hg = (a.n_heads + nh - 1) / nh;
  static RaisedLimit smem_set[2][4];
  cudaError_t e = ensure_smem(a.T == 1 ? k_dec : k_pf, smem,
                              smem_set[a.T == 1][fp4 ? 2 + (nh == kH) : paged]);
  if (e != cudaSuccess) return e;
  CUtensorMap tq;
  if (fp4) {   // Q as [n_q][H][512]: boxes of one CTA's heads, zeros past the last head
    const uint64_t qd[3] = {(uint64_t)kD, (uint64_t)a.n_heads, (uint64_t)P.n_q};
    const uint64_t qs[2] = {(uint64_t)kD * 2, (uint64_t)a.n_heads * kD * 2};
    const uint32_t qb[3] = {64, nh, 1};
    e = make_tmap_bf16(&tq, a.q, 3, qd, qs, qb);
  } else {     // Q as [n_q * 64 heads][512] bf16 rows; boxes of one CTA's heads x 64 dims
    const uint64_t qd[2] = {(uint64_t)kD, (uint64_t)P.n_q * kH};
    const uint64_t qs[1] = {(uint64_t)kD * 2};
    const uint32_t qb[2] = {64, nh};
    e = make_tmap_bf16(&tq, a.q, 2, qd, qs, qb);
  }
  if (e != cudaSuccess) return e;
  // decode tiles of contiguous rows: the ring [B][128][512] (one box of its
  // 128 slots per 64 dims) and, on ratio 128 with one position for every
  // sequence, the visible compressed rows [B][n_list][512] (rows past n_list
  // read as zeros); a map that cannot be built leaves the gathers
  CUtensorMap tr = tq, tcmp = tq;
  P.tma_rows = 0;
  // (ratio 4 keeps its window on the gathers: its first rank runs the window
  // tile beside the list tiles, and by TMA it measured slower)
  // (with 4-bit rows the window is the largest tile: always by TMA; in a chunk, the
  // windows that lie inside it)
  if (fp4 && a.T >= (uint32_t)kRows && a.cap_raw == (uint32_t)kRows) {
    const uint64_t rd[3] = {(uint64_t)kD, (uint64_t)a.T, (uint64_t)a.batch};
    const uint64_t rs[2] = {(uint64_t)kD * 2, (uint64_t)a.T * kD * 2};
    const uint32_t rb[3] = {64, (uint32_t)kRows, 1};
    if (make_tmap_bf16(&tr, a.chunk, 3, rd, rs, rb) == cudaSuccess) P.tma_rows |= 4u;
  }
  // (not for a chunk of one token: its row is in the chunk, not yet in the ring)
  if (a.T == 1 && !a.chunk && a.cap_raw == (uint32_t)kRows && (a.ratio != 4 || fp4)) {
    const uint64_t rd[3] = {(uint64_t)kD, (uint64_t)a.cap_raw, (uint64_t)a.batch};
    const uint64_t rs[2] = {(uint64_t)kD * 2, (uint64_t)a.cap_raw * kD * 2};
    const uint32_t rb[3] = {64, (uint32_t)kRows, 1};
    if (make_tmap_bf16(&tr, a.ring, 3, rd, rs, rb) == cudaSuccess) P.tma_rows |= 1u;
    const uint32_t n_list = a.ratio == 128 ? min((a.pos0 + 1) / 128, a.n_comp) : 0u;
    if (a.ratio == 128 && !paged && !fp4 && !a.seq_pos && n_list >= (uint32_t)kRows) {
      const uint64_t cd[3] = {(uint64_t)kD, (uint64_t)n_list, (uint64_t)a.batch};
      const uint64_t cs[2] = {(uint64_t)kD * 2, (uint64_t)a.comp_cap * kD * 2};
      if (make_tmap_bf16(&tcmp, a.comp, 3, cd, cs, rb) == cudaSuccess) P.tma_rows |= 2u;
    }
  }
  if (a.T == 1) {
    // one cluster of P.cluster CTAs per (query, head group)
    const uint32_t n_vq = P.n_q * P.hg;
    P.cluster = fp4 ? plan.cluster : decode_cluster(rows_max, n_vq, smem);
    P.ml = reinterpret_cast<float *>(P.part + (size_t)n_vq * P.cluster * nh * kD * (fp4 ? 2 : 1));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = P.cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(n_vq * P.cluster);
    cfg.blockDim = dim3(fp4 ? Warps<true>::THREADS : Warps<false>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_dec, tq, tr, tcmp, P);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  P.cluster = 0;
  const uint64_t items = (uint64_t)P.n_q * P.hg;
  const uint32_t grid = (uint32_t)min(items, (uint64_t)num_sms());
  e = launch_pdl(k_pf, dim3(grid), dim3(fp4 ? Warps<true>::THREADS : Warps<false>::THREADS), smem, s, tq, tr, tcmp, P);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ds4a
