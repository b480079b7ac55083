// Attention of a step's new tokens over a paged cache of keys and values, on the tensor cores
// (bf16 queries; keys and values in bf16 or 8-bit floats).
//
// A row is one query head of one new token; the R = tokens x (H / K) rows of a key head share its
// keys (groups of up to RP rows where there are more). With few rows the products are done the
// other way round, so that the 128 keys of a tile fill the tensor core's 128 lanes:
//
//   S^T [128 keys][rows] = K [keys][D] . Q^T      A = the key tile as TMA leaves it (K-major)
//   O^T [D][rows]       += V^T [D][keys] . P^T    A = the value tile as TMA leaves it (MN-major)
//
// and each of 128 threads has one key's scores: weights are 2^(s - m) against a reference m per
// row that moves only when a score passes it by a margin (then the sums so far are rescaled),
// so a tile needs no maximum over its keys. P goes to shared memory as it comes, one key's
// weights in a row.
//
// Types. Weights are held as the sum of two bf16 (the second operand has 2 RP columns), which
// keeps 16 bits of them. Over an 8-bit cache nothing is widened: queries and weights are each
// split into two 8-bit floats, x = hi + lo / 16, whose products with the codes are exact. A bf16
// query has 8 significant bits, hi and lo 4 each; the largest entry of a row is brought to 2^7 .. 2^8
// and lo's step is 2^-13, so only entries below 2^-13 of the largest lose bits. A weight keeps 8 bits
// too, and below 2^-5 steps of 2^-13: a weight of 2^-14 is lost. So the reference there follows the row's weights
// down as well as up, and the sums, which have fp32's range, are brought along. A row
// whose weights of a tile all fall below 2 is noticed one tile later, and its reference lowered, unless the row's sum
// is 2 for each tile up to the next power of two: what all these tiles' keys can lose is then 2^-8 of it. Only while some
// row's sum is not enough are single tiles watched. (A key with 0.95 of the weight before 131,070 others: 0.05 of the
// output lost with a reference that only rises, 0.001 now. 19 sequences of 8,192 tokens with 1 / 4 / 8 new ones: 58.2 / 76.4 /
// 111 us, 58.0 / 72.6 / 106 with one that only rises; where scores spread by 5 around their mean, 8 new
// ones 195 against 139.) Sums are fp32.
//
// Work. The tiles of all sequences, key heads and row groups are one list, of which each block
// takes an even share, whatever the lengths. A part of a (sequence, key head, group) that a block
// does not hold whole is left as sums with their reference, and a second launch joins
// the parts in order.
//
// Every visible key and value is read once. Bound by HBM for up to 16 rows in long sequences: 8 of
// 131,072 tokens of 8 heads of 128 dims, bf16, 8 rows each 605 us (7.1 TB/s); 64 ragged ones up to
// 32,768 over an 8-bit cache 97 (5.8 TB/s). With more rows by a tile's chain of scores, weights and output
// product, of which an SM then has one: 16 ragged ones up to 16,384 with 40 rows each 39 us (4.0
// TB/s). Short calls by some ten steps of 0.3 to 1 us with cold code: a sequence of 4,096 tokens 11 us.
//
// Warps: 0 TMA, 1 MMA, 2 the block's list of segments, 3 queries, 4 .. 7 (4 .. 11 from 32 rows on)
// softmax and output. Every wait is bounded (tc.cuh).
#include <cuda_fp8.h>

#include "paged.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kTile = 128, kBox = kTile * 128;   // keys; bytes of a 128-byte column
constexpr uint32_t kSegs = 4, kMaxSlots = 16;
constexpr uint32_t kSmemSm = 228 * 1024, kSmemBlock = 1024;   // shared memory of an SM; reserved per block
constexpr uint32_t kLeast = 2;    // places of a share at least: fewer parts to join
// The most tiles of a sequence that is not divided: no parts and no join (28 sequences of 193 tokens, 2 heads: 11.2 us
// divided, 8.4; 12 of 419, 8 heads 13.7, 10.8).
constexpr uint32_t kWholeTiles = 4;
constexpr float kNoRef = 3e38f;   // -reference of a row that has seen no key
// 8 bits: a row's reference is lowered where a tile's weights are below 2^kLow, unless its sum is kEnough a tile. The
// largest weight of the first tile, 2^5, is that for kSure tiles. (kEnough 4, kSure 4: 8 new tokens as above 114 us.)
constexpr float kLow = 1.f, kEnough = 2.f;
constexpr uint32_t kSure = 16;

struct Segment {
  uint32_t b, kh, r0, nr;          // sequence, key head, first row and rows
  uint32_t first, pos0;            // packed index and position of the sequence's first token
  uint32_t tile0, nt;              // tiles (of 128 positions); nt 0: no more segments
  uint32_t whole;                  // bit 0: its first tile is here, bit 1: its last
  uint32_t blocks;                 // blocks behind this one that hold some of it
};

// What a block left of a segment that goes on in the next `blocks` ones (0: no such segment).
struct Part {
  uint32_t blocks, kh, r0, nr, first, pad[3];
};

struct Params {
  PagedArgs a;
  uint32_t G;           // query heads per key head
  uint32_t nbox, nmb;   // 128-byte columns of a key's row; blocks of 128 dims of the output
  uint32_t ubox;        // columns of a unit, what is loaded at once: a tile's keys or values of 128 dims
  uint32_t n_slots, n_q, n_p;   // units, query tiles and weight tiles held
  uint32_t g_mul;       // 2^32 / G + 1 (rows are below 2^18), 0: G is 1
  uint32_t q_vec;       // queries start on 16 bytes
  uint32_t whole;       // segments are not divided: no parts, a place each
  float c2;             // scale * log2(e)
  Part *parts;          // [blocks]
  // [blocks][2][RP][D], then (reference, sum) [blocks][2][RP][2]: of what began before a block, and of
  // what goes on behind it
  float *sums;
  int *err;
};

template <int RP, bool F8>
struct Cfg {
  static constexpr uint32_t kQRows = F8 ? 2 * RP : (RP < 16 ? 16 : RP);   // rows of the Q operand
  static constexpr uint32_t kPBytes = kTile * 2 * RP * (F8 ? 1 : 2);
  // softmax warps: four, which take a quarter of the keys each, or two such sets with every other
  // eight rows each
  static constexpr uint32_t kSets = RP >= 32 ? 2 : 1, kWarps = 4 * kSets, kThreads = 128 + 32 * kWarps;
  // What a segment costs beside its tiles, in tiles, for even shares. 64 ragged sequences over 8 bits, 8 rows: 129 us
  // with 0, 102 with 1, 97 with 2, 96 with 3; 16 ragged ones with 40 rows: 48.4 with 2, 40.9 with 3, 39.3 with 4, 40.0 with
  // 5, 41.7 with 8, over 8 bits 55.1, 47.2, 47.1, 47.7 and 50.1.
  static constexpr uint32_t kStart = RP <= 16 ? 2 : 4;
  static constexpr int kRows = RP / kSets;
  // few rows: two blocks a SM, so that one computes while the other starts, ends or waits (152 sequences of
  // 128 tokens: 46 us with one, 23 with two); 32 rows and more take the shared memory of one
  static constexpr uint32_t kPerSm = RP <= 16 ? 2 : 1;
  static constexpr float kOff = F8 ? 5.f : 0.f;     // weights are 2^(s - m + kOff)
  static constexpr float kTop = F8 ? 8.75f : 8.f;   // ... and at most 2^kTop (448 for 8 bits)
  static constexpr uint32_t kAll = kRows < 32 ? (1u << kRows) - 1 : 0xffffffffu;   // a bit for each row of a set
};

template <int RP>
struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full[2], q_empty[2], s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2], o_free, drain;
  uint32_t tmem;
  uint32_t start_b;
  uint32_t shares;
  uint64_t start_off, start_n, total, end;   // of the list of tiles: see below
  uint64_t scan[12];
  uint32_t bad;
  Segment seg[kSegs];
  alignas(16) float qs[kSegs][RP];   // factor of each row's scores (8-bit queries)
  alignas(16) float negm[RP];        // -reference of each row
  alignas(16) float fac[RP];
  alignas(16) float wmax[4][RP];
  alignas(16) uint32_t fine[2][8];   // rows with a weight of 2^kLow or more: of each warp, in this tile and the one before
  uint32_t enough[2][2], settled[2];   // rows whose sum is enough, of each set (halves of 64 rows); whether all are for all tiles
  uint64_t row_out[RP];              // packed token * H + head of each row (passes 2^32 where steps hold 2^22 tokens)
};

// Products with 8-bit operands, both E4M3, fp32 sums; from code that the whole warp runs.
__device__ __forceinline__ void mma_e4m3_elect(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// High half of the descriptor of an operand without swizzle, MN-major: 16 bytes along N by 8 along
// K are 128 contiguous bytes; `mn_step` bytes to the next 16 bytes along N. (The low half's leading byte
// offset is the step to the next 8 along K.)
__host__ __device__ constexpr uint32_t desc_hi_plain(uint32_t mn_step) { return (mn_step >> 4) | (1u << 14); }

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
  return u;
}
__device__ __forceinline__ uint16_t pack_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack_e4m3(uint16_t u) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(u, __NV_E4M3)));
}

// Reductions of R values over the warp, all at once: lane 32 / R * r ends up with value r (each step
// halves the values that a lane holds).
template <int R, typename Op>
__device__ __forceinline__ float warp_reduce_rows(float (&v)[R], uint32_t lane, Op op) {
  uint32_t o = 16;
#pragma unroll
  for (int n = R; n > 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  for (; o; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}
// The larger of two, a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }

// The waits of the chain from scores to output: a test, which a thread that issues products needs (a
// blocking wait would hold it until those in flight have drained), then blocking tries; the time is looked
// at when those have failed for long.
__device__ __forceinline__ bool wait_chain(uint64_t *bar, uint32_t parity, ErrWord err) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  bool ok = false;
  for (uint32_t i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  return __all_sync(0xffffffffu, mbar_wait_long(smem_u32(bar), parity, err.p, err.base));
}

// Two fp32 operations at once, each rounded as the single one.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The share that place x - 1 of a list of `total` is in: the largest c with total c / shares < x.
__device__ __forceinline__ uint32_t last_share(uint64_t x, uint32_t shares, uint64_t total) {
  const uint64_t n = x * shares - 1;
  return (n | total) >> 32 ? (uint32_t)(n / total) : (uint32_t)n / (uint32_t)total;
}
// a b / c, mostly in 32 bits.
__device__ __forceinline__ uint64_t mul_div(uint64_t a, uint32_t b, uint64_t c) {
  const uint64_t n = a * b;
  return (n | c) >> 32 ? n / c : (uint32_t)n / (uint32_t)c;
}

// One arrival of a warp.
__device__ __forceinline__ void warps_arrive(uint64_t *bar, uint32_t lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Hardware barrier of the softmax's `count` threads; the second tells whether any of them says so. (An mbarrier
// costs some 300 clocks to the waiting side, this 50. It cannot run out, so these warps enter a segment
// together or not at all and go through it whatever their other waits say.)
__device__ __forceinline__ void group_bar(uint32_t count) { named_bar_sync(1, count); }
__device__ __forceinline__ bool group_any(bool mine, uint32_t count) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)mine), "r"(count)
      : "memory");
  return any != 0;
}

// The tile behind j at which sums are looked at again.
__device__ __forceinline__ uint32_t next_look(uint32_t j) { return max(kSure, 2u << (31 - __clz(j))); }

// n / G
__device__ __forceinline__ uint32_t by_group(const Params &P, uint32_t n) { return P.g_mul ? __umulhi(n, P.g_mul) : n; }

__device__ __forceinline__ uint32_t tiles_of(const PagedItem &it) {
  if (it.cnt == 0) return 0;
  return it.hi > it.lo ? (it.hi + kTile - 1) / kTile - it.lo / kTile : 1u;   // (one without keys writes zeros)
}

// Physical block of logical block j of sequence b; n_blocks or more: not there.
__device__ __forceinline__ uint32_t phys_of(const PagedArgs &a, uint32_t b, uint32_t j) {
  return j < a.max_blocks ? (uint32_t)__ldg(a.table + (size_t)b * a.max_blocks + j) : 0xffffffffu;
}

// Physical block of a tile, from 32 entries at a time in the warp's lanes. look() before at(), apart so
// that the load overlaps a wait.
struct BlockList {
  uint32_t base, mine;
  __device__ __forceinline__ void start() { base = 0xffffffffu; }
  __device__ __forceinline__ void look(const PagedArgs &a, uint32_t b, uint32_t j, uint32_t lane) {
    if (base == 0xffffffffu || j - base >= 32) {
      base = j;
      mine = phys_of(a, b, j + lane);
    }
  }
  __device__ __forceinline__ uint32_t at(uint32_t j) { return __shfl_sync(0xffffffffu, mine, j - base); }
};

// Place of V(j) in the order of a segment's loads, K0 K1 V0 K2 V1 .. V(nt - 1).
__device__ __forceinline__ uint32_t place_v(uint32_t j, uint32_t nt) { return j + 1 < nt ? 2 * j + 2 : 2 * nt - 1; }

struct Ring {   // slot and parity of the loads, counted from the block's first
  uint32_t slot, phase;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// A value row of an unseen key, or the NaNs and infinities of one that only some rows see, made zeros in
// shared memory: 0 times them would be a NaN. Returns whether there were any of the latter. (Lanes start a
// piece of 16 bytes apart, so that eight of them cover all banks.)
template <bool F8>
__device__ __noinline__ bool clean_row(uint32_t row, uint32_t ubox, bool all, uint32_t lane) {
  bool found = false;
  for (uint32_t x = 0; x < ubox; ++x, row += kBox) {
    if (all) {
#pragma unroll
      for (uint32_t c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(row + 16 * ((c + lane) & 7)), "r"(0u) : "memory");
      continue;
    }
#pragma unroll 1
    for (uint32_t c = 0; c < 8; c += 4) {
      uint32_t v[4][4];
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[u][0]), "=r"(v[u][1]), "=r"(v[u][2]), "=r"(v[u][3])
                     : "r"(row + 16 * ((c + u + lane) & 7)));
      bool here = false;
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t keep = 0;
          if (F8) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) keep |= (v[u][i] >> k & 0x7fu) == 0x7fu ? 0u : 0xffu << k;
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 16) keep |= (v[u][i] >> k & 0x7f80u) == 0x7f80u ? 0u : 0xffffu << k;
          }
          here |= keep != 0xffffffffu;
          v[u][i] &= keep;
        }
      if (!here) continue;
      found = true;
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + 16 * ((c + u + lane) & 7)), "r"(v[u][0]),
                     "r"(v[u][1]), "r"(v[u][2]), "r"(v[u][3])
                     : "memory");
    }
  }
  return found;
}

// What clean_row took out of dim d for a row whose token is at p: the sum of the NaNs and infinities
// among the keys that some of the group's tokens (p_first .. p_last) see and others do not.
template <bool F8>
__device__ __noinline__ float taken_out(const PagedArgs &a, const Segment &sg, uint32_t p, uint32_t p_first,
                                        uint32_t p_last, uint32_t d) {
  float sum = 0.f;
  const uint32_t k0 = sg.tile0 * kTile, k1 = k0 + sg.nt * kTile;
  for (int side = 0; side < 2; ++side) {
    if (side == 0 && !a.window) continue;
    // side 0: the oldest keys, which later tokens' windows leave out; side 1: the new tokens' own
    uint32_t from = side ? p_first + 1 : (p_first + 1 > a.window ? p_first + 1 - a.window : 0u);
    uint32_t to = side ? p_last + 1 : (p_last + 1 > a.window ? p_last + 1 - a.window : 0u);
    from = max(from, k0);
    to = min(to, k1);
    if (side == 0) to = min(to, p_first + 1);   // (counted once)
    for (uint32_t key = from; key < to; ++key) {
      if (key > p || (a.window && p - key >= a.window)) continue;
      const uint32_t phys = phys_of(a, sg.b, key / 256);
      if (phys >= a.n_blocks) continue;
      const size_t at = (((size_t)phys * a.n_kv + sg.kh) * 256u + key % 256) * a.head_dim + d;
      if (F8) {
        if ((static_cast<const uint8_t *>(a.v)[at] & 0x7f) == 0x7f) sum = NAN;
      } else {
        const float v = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v)[at]);
        if (!(fabsf(v) <= 3.4e38f)) sum += v;
      }
    }
  }
  return sum;
}

template <int RP, bool F8>
__global__ void __launch_bounds__(Cfg<RP, F8>::kThreads, Cfg<RP, F8>::kPerSm)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, Params P) {
  using C = Cfg<RP, F8>;
  constexpr uint32_t kThreads = C::kThreads;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const PagedArgs &a = P.a;
  const uint32_t slot_bytes = P.ubox * kBox, q_bytes = C::kQRows * P.nbox * 128u;
  uint8_t *s_slot = smem, *s_q = s_slot + P.n_slots * slot_bytes, *s_p = s_q + P.n_q * q_bytes;
  Shared<RP> &S = *reinterpret_cast<Shared<RP> *>(s_p + P.n_p * C::kPBytes);
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5, D = a.head_dim;
  const uint32_t o_cols = P.nmb * 2 * RP;   // output sums, then two score tiles
  const uint32_t cols = o_cols + 2 * C::kQRows;
  const uint32_t alloc = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;

  if (t == 0) {
    for (uint32_t i = 0; i < P.n_slots; ++i) mbar_init(&S.full[i], 1), mbar_init(&S.empty[i], 1);
    for (uint32_t i = 0; i < kSegs; ++i) mbar_init(&S.seg_full[i], 1), mbar_init(&S.seg_empty[i], 3 + C::kWarps);
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.s_empty[i], C::kWarps);
      mbar_init(&S.p_full[i], C::kWarps);
      mbar_init(&S.pv_done[i], 1);
    }
    mbar_init(&S.o_free, C::kWarps);
    mbar_init(&S.drain, 1);
    S.start_n = 0;
    S.bad = 0;
    fence_mbar_init();
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 1) tmem_alloc(&S.tmem, alloc);
  pdl_wait();
  pdl_trigger();
  const ErrWord err{P.err, *(volatile int *)P.err};
  // ---- the block's share of the list: kStart places for each segment, then its tiles; each thread
  // counts some sequences'
  {
    const uint32_t per = (a.batch + kThreads - 1) / kThreads, b0 = min(a.batch, t * per), b1 = min(a.batch, b0 + per);
    auto weight = [&](uint32_t b) {
      const PagedItem it = paged_item(a, b);
      const uint32_t tiles = tiles_of(it);
      return (uint64_t)(tiles ? P.whole ? 1u : tiles + C::kStart : 0u) * a.n_kv * ((it.cnt * P.G + RP - 1) / RP);
    };
    uint64_t own = 0;
    for (uint32_t b = b0; b < b1; ++b) own += weight(b);
    uint64_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= (uint32_t)o) inc += x;
    }
    if (lane == 31) S.scan[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint64_t before = inc - own, total = 0;
    for (uint32_t w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += S.scan[w];
      total += S.scan[w];
    }
    const uint32_t least = P.whole ? 1u : kLeast;
    const uint32_t shares = (uint32_t)min((uint64_t)gridDim.x, (total + least - 1) / least), c = blockIdx.x;
    const uint64_t from = c < shares ? mul_div(total, c, shares) : total;
    const uint64_t to = c < shares ? mul_div(total, c + 1, shares) : total;
    if (from < to && before <= from && from < before + own) {   // (one thread, or none)
      uint64_t off = from - before;
      uint32_t b = b0;
      for (; b + 1 < b1; ++b) {
        const uint64_t w = weight(b);
        if (off < w) break;
        off -= w;
      }
      S.start_b = b;
      S.start_off = off;
      S.start_n = to - from;
    }
    if (t == 0) {
      S.total = total;
      S.shares = shares;
      S.end = to;
    }
    __syncthreads();
  }
  const uint32_t tmem = S.tmem;

  if (warp == 0) {
    // ---------------- TMA: key and value tiles
    const uint64_t pol = l2_evict_first_policy(), pol_n = l2_evict_normal_policy();
    Ring ring{0, 0};
    uint32_t issued = 0;
    bool ok = true;
    for (uint32_t s = 0; ok; ++s) {
      if (!wait_chain(&S.seg_full[s % kSegs], (s / kSegs) & 1, err)) break;
      const Segment sg = S.seg[s % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.seg_empty[s % kSegs]);
      if (sg.nt == 0) break;
      // (rows of several groups read the same tiles again)
      const uint64_t policy = a.max_new * P.G <= RP ? pol : pol_n;
      BlockList kl, vl;
      kl.start();
      vl.start();
      for (uint32_t e = 0; e < 2 * sg.nt; ++e) {
        const bool is_v = e + 1 == 2 * sg.nt || (e && !(e & 1));
        const uint32_t j = e + 1 == 2 * sg.nt ? sg.nt - 1 : is_v ? e / 2 - 1 : (e + 1) / 2, tile = sg.tile0 + j;
        BlockList &bl = is_v ? vl : kl;
        bl.look(a, sg.b, tile / 2, lane);
        uint32_t phys = bl.at(tile / 2);
        if (phys >= a.n_blocks) phys = 0;   // (its keys are masked)
        const int y = (int)((phys * a.n_kv + sg.kh) * 256u + (tile & 1) * kTile);
        for (uint32_t m = 0; m < P.nmb; ++m) {
          ok = mbar_wait_sleep(&S.empty[ring.slot], ring.phase ^ 1, err);
          if (!ok) break;
          if (lane == 0) {
            uint64_t *bar = &S.full[ring.slot];
            uint8_t *dst = s_slot + ring.slot * slot_bytes;
            mbar_arrive_expect_tx(bar, slot_bytes);
            for (uint32_t x = 0; x < P.ubox; ++x)   // (columns behind the row are filled with zeros)
              tma_load_2d_hint(dst + x * kBox, is_v ? &map_v : &map_k, bar,
                               (int)((m * P.ubox + x) * (F8 ? 128 : 64)), y, policy);
          }
          ++issued;
          ring.next(P.n_slots);
        }
        if (!ok) break;
      }
    }
    // every load of this block lands before it can end (bounded)
    const uint32_t left = min(issued, P.n_slots);
    for (uint32_t i = 0; i < left; ++i) {
      const uint32_t k = issued - left + i;
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&S.full[k % P.n_slots], (k / P.n_slots) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA (the whole warp runs this; one thread issues)
    constexpr uint32_t kFmt = F8 ? (1u << 4) : (1u << 4) | (1u << 7) | (1u << 10);
    constexpr uint32_t id_s = kFmt | ((C::kQRows >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t id_o = kFmt | ((2u * RP >> 3) << 17) | ((128u >> 4) << 24) | kIdescMajorA_MN | kIdescMajorB_MN;
    const uint32_t slot0 = uniform(desc_lo(smem_u32(s_slot))), unit = uniform(slot_bytes >> 4);
    const uint32_t q0 = uniform(desc_lo(smem_u32(s_q)) | desc_lbo(16)), p0 = uniform(desc_lo(smem_u32(s_p)) | desc_lbo(128));
    const uint32_t t_o = uniform(tmem), t_s = uniform(tmem + o_cols);
    // (128 dims: one column of 8-bit codes, two of bf16; a lone one is read twice: half of the lanes
    // is then not used)
    const uint32_t v_lbo = uniform(P.ubox == 2 ? desc_lbo(kBox) : 0u);
    Ring ring{0, 0};
    uint32_t sc = 0, pv = 0, qb = 0;   // score tiles issued, output products issued
    bool ok = true;
    auto scores = [&]() {
      const uint32_t sb = sc & 1, d = t_s + sb * C::kQRows;
      if (!wait_chain(&S.s_empty[sb], ((sc >> 1) & 1) ^ 1, err)) return false;
      for (uint32_t m = 0; m < P.nmb; ++m) {
        if (!wait_chain(&S.full[ring.slot], ring.phase, err)) return false;
        tc_fence_after();
        for (uint32_t x = 0; x < P.ubox && m * P.ubox + x < P.nbox; ++x) {
          const uint32_t ka = (slot0 | desc_lbo(16)) + ring.slot * unit + x * (kBox >> 4);
          const uint32_t qa = q0 + (qb * q_bytes >> 4) + (m * P.ubox + x) * C::kQRows * 8u;
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            const uint64_t ad = desc_at(ka + 2 * k, kDescHiK), bd = desc_at(qa + 2 * k, kDescHiK);
            if (F8)
              mma_e4m3_elect(d, ad, bd, id_s, m | x | k);
            else
              mma_bf16_elect(d, ad, bd, id_s, m | x | k);
          }
        }
        mma_commit_elect(&S.empty[ring.slot]);
        ring.next(P.n_slots);
      }
      mma_commit_elect(&S.s_full[sb]);
      ++sc;
      return true;
    };
    for (uint32_t s = 0; ok; ++s) {
      if (!(ok = wait_chain(&S.seg_full[s % kSegs], (s / kSegs) & 1, err))) break;
      const uint32_t nt = uniform(S.seg[s % kSegs].nt);
      warps_arrive(&S.seg_empty[s % kSegs], lane);
      if (nt == 0) break;
      qb = P.n_q == 2 ? s & 1 : 0u;
      if (!(ok = wait_chain(&S.q_full[qb], (P.n_q == 2 ? s >> 1 : s) & 1, err))) break;
      if (!(ok = scores())) break;
      if (nt == 1) mma_commit_elect(&S.q_empty[qb]);
      for (uint32_t j = 0; ok && j < nt; ++j) {
        if (j + 1 < nt) {
          if (!(ok = scores())) break;
          if (j + 2 == nt) mma_commit_elect(&S.q_empty[qb]);
        }
        if (j == 0 && s && !(ok = wait_chain(&S.o_free, (s - 1) & 1, err))) break;
        const uint32_t pb = P.n_p == 2 ? pv & 1 : 0u, use = P.n_p == 2 ? pv >> 1 : pv;
        if (!(ok = wait_chain(&S.p_full[pb], use & 1, err))) break;
        for (uint32_t m = 0; m < P.nmb; ++m) {
          if (!(ok = wait_chain(&S.full[ring.slot], ring.phase, err))) break;
          tc_fence_after();
          const uint32_t va = (slot0 | v_lbo) + ring.slot * unit, pa = p0 + (pb * C::kPBytes >> 4);
#pragma unroll
          for (uint32_t k = 0; k < (F8 ? 4u : 8u); ++k) {
            const uint64_t ad = desc_at(va + k * ((F8 ? 4096u : 2048u) >> 4), kDescHiK);
            const uint64_t bd = desc_at(pa + k * ((F8 ? 512u : 256u) >> 4), desc_hi_plain(2048));
            if (F8)
              mma_e4m3_elect(t_o + m * 2 * RP, ad, bd, id_o, j | k);
            else
              mma_bf16_elect(t_o + m * 2 * RP, ad, bd, id_o, j | k);
          }
          mma_commit_elect(&S.empty[ring.slot]);
          ring.next(P.n_slots);
        }
        if (!ok) break;
        mma_commit_elect(&S.pv_done[pb]);
        ++pv;
      }
    }
    if (!ok) {   // let the products in flight end (bounded)
      mma_commit_elect(&S.drain);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&S.drain, 0) && global_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- the segments: sequences 32 at a time, a lane each
    uint32_t b = S.start_b, base = b, s = 0;
    uint64_t off = S.start_off, left = S.start_n;
    PagedItem mine = {};
    if (left && b + lane < a.batch) mine = paged_item(a, b + lane);
    bool ok = true;
    while (left && b < a.batch) {
      if (b - base >= 32) {
        base = b;
        mine = PagedItem{};
        if (b + lane < a.batch) mine = paged_item(a, b + lane);
      }
      const uint32_t src = b - base;
      PagedItem it;
      it.first = __shfl_sync(0xffffffffu, mine.first, src);
      it.cnt = __shfl_sync(0xffffffffu, mine.cnt, src);
      it.pos0 = __shfl_sync(0xffffffffu, mine.pos0, src);
      it.lo = __shfl_sync(0xffffffffu, mine.lo, src);
      it.hi = __shfl_sync(0xffffffffu, mine.hi, src);
      const uint32_t tiles = tiles_of(it), groups = (it.cnt * P.G + RP - 1) / RP;
      if (tiles) {
        const uint32_t places = P.whole ? 1u : tiles + C::kStart;
        uint32_t kh = 0, rg = 0, o = 0;   // o: the first place of the segment here
        if (off) {
          const uint32_t i = (uint32_t)mul_div(off, 1, places);
          o = (uint32_t)(off - (uint64_t)i * places);
          kh = i / groups;
          rg = i % groups;
        }
        for (; kh < a.n_kv && left; o = 0) {
          const uint32_t n = (uint32_t)min((uint64_t)(places - o), left), e = o + n;
          const uint32_t t0 = o > C::kStart ? o - C::kStart : 0u;
          const uint32_t nt = P.whole ? tiles : e > C::kStart ? e - C::kStart - t0 : 0u;
          left -= n;
          if (nt == 0) break;   // (the share ends before the segment's first tile)
          if (!(ok = mbar_wait_sleep(&S.seg_empty[s % kSegs], ((s / kSegs) & 1) ^ 1, err))) break;
          if (lane == 0) {
            Segment &sg = S.seg[s % kSegs];
            sg.b = b;
            sg.kh = kh;
            sg.r0 = rg * RP;
            sg.nr = min((uint32_t)RP, it.cnt * P.G - sg.r0);
            sg.first = it.first;
            sg.pos0 = it.pos0;
            sg.tile0 = it.lo / kTile + t0;
            sg.nt = nt;
            const uint32_t rest = tiles - t0 - nt;   // (its other tiles follow the block's share)
            sg.whole = (t0 == 0 ? 1u : 0u) | (rest == 0 ? 2u : 0u);
            sg.blocks = rest ? last_share(S.end + rest, S.shares, S.total) - blockIdx.x : 0u;
            mbar_arrive(&S.seg_full[s % kSegs]);
          }
          __syncwarp();
          ++s;
          if (++rg == groups) {
            rg = 0;
            ++kh;
          }
        }
        if (!ok) break;
      }
      off = 0;
      ++b;
    }
    if (ok && mbar_wait_sleep(&S.seg_empty[s % kSegs], ((s / kSegs) & 1) ^ 1, err) && lane == 0) {
      S.seg[s % kSegs].nt = 0;
      mbar_arrive(&S.seg_full[s % kSegs]);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------- queries of a segment, as the second operand of the scores
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
    for (uint32_t s = 0;; ++s) {
      if (!wait_chain(&S.seg_full[s % kSegs], (s / kSegs) & 1, err)) break;
      const Segment sg = S.seg[s % kSegs];
      const uint32_t qb = P.n_q == 2 ? s & 1 : 0u;
      if (sg.nt == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.seg_empty[s % kSegs]);
        break;
      }
      if (!mbar_wait_sleep(&S.q_empty[qb], ((P.n_q == 2 ? s >> 1 : s) & 1) ^ 1, err)) break;
      uint8_t *dst = s_q + qb * q_bytes;
      // (rows of eights that nothing reads are left as they are)
      const uint32_t most = max(16u, (sg.nr + 7) & ~7u), rows = F8 ? min(most, (uint32_t)RP) : min(most, C::kQRows);
      const uint32_t tok_r0 = by_group(P, sg.r0), g_r0 = sg.r0 - tok_r0 * P.G;
      // 16-byte piece c of row r of the operand. 8-bit rows (hi r, lo RP + r) hold the bf16 row first: a column's
      // sixteen pieces in the places of its hi and lo.
      auto place = [&](uint32_t r, uint32_t c) {
        return dst + (c / 8) * C::kQRows * 128u + r * 128u + (((c & 7) ^ (r & 7)) << 4);
      };
      auto raw_place = [&](uint32_t r, uint32_t c) {
        return F8 ? place(c & 8 ? RP + r : r, (c >> 4) * 8 + (c & 7)) : place(r, c);
      };
      {
        const uint32_t pieces = P.nbox * (F8 ? 16 : 8), rpp = 32 / pieces, sub = lane / pieces, c = lane % pieces;
        const size_t wrap = a.q_stride - (size_t)P.G * D;   // from behind a token's heads to the next token's
        uint32_t g = g_r0;
        const __nv_bfloat16 *p = q + (sg.first + tok_r0) * a.q_stride + (size_t)(sg.kh * P.G + g) * D + 8 * c;
        auto advance = [&](uint32_t step) {   // a lane's rows are `step` apart
          p += step * D;
          for (g += step; g >= P.G; g -= P.G) p += wrap;
        };
        advance(sub);
        for (uint32_t r = sub; sub < rpp && r < rows; r += rpp, advance(rpp)) {
          const bool in = r < sg.nr && 8 * c < D;   // (zeros outside)
          if (P.q_vec) {   // (all rows on their way at once)
            cp_async16(raw_place(r, c), in ? p : q, in ? 16u : 0u);
          } else {
            uint32_t w[4] = {0, 0, 0, 0};
            if (in)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)__bfloat16_as_ushort(p[2 * i]) | (uint32_t)__bfloat16_as_ushort(p[2 * i + 1]) << 16;
            *reinterpret_cast<uint4 *>(raw_place(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      if constexpr (F8) {
        // half a warp per row, 16 elements a lane: q 2^k = hi + lo / 16, k so that the largest
        // entry is in [128, 256)
        const uint32_t c = lane & 15;
        const bool in = c < P.nbox * 8;
        const float ks = __ldg(a.k_scale + sg.kh) * P.c2;
        __syncwarp();
        for (uint32_t r0 = lane >> 4; r0 < rows; r0 += 4) {   // (both halves go on together, two rows each)
          uint32_t w[2][8], top[2];
#pragma unroll
          for (uint32_t u = 0; u < 2; ++u) {
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            if (in) {
              x0 = *reinterpret_cast<const uint4 *>(raw_place(r0 + 2 * u, 2 * c));
              x1 = *reinterpret_cast<const uint4 *>(raw_place(r0 + 2 * u, 2 * c + 1));
            }
            w[u][0] = x0.x, w[u][1] = x0.y, w[u][2] = x0.z, w[u][3] = x0.w;
            w[u][4] = x1.x, w[u][5] = x1.y, w[u][6] = x1.z, w[u][7] = x1.w;
            top[u] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top[u] = max(top[u], max(w[u][i] & 0x7fffu, w[u][i] >> 16 & 0x7fffu));
          }
#pragma unroll
          for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (uint32_t u = 0; u < 2; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
          __syncwarp();   // (the rows are in registers)
#pragma unroll
          for (uint32_t u = 0; u < 2; ++u) {
            const uint32_t r = r0 + 2 * u;
            // (a row with a NaN or an infinity becomes NaN)
            const int e = max((int)(top[u] >> 7) - 127, -119);
            const float up = top[u] >= 0x7f80u ? NAN : __uint_as_float((uint32_t)(127 + 7 - e) << 23);
            const float down = __uint_as_float((uint32_t)(127 - 7 + min(e, 127)) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float2 x[2];
#pragma unroll
              for (int k = 0; k < 2; ++k)
                x[k] = mul2(make_float2(__uint_as_float(w[u][2 * i + k] << 16), __uint_as_float(w[u][2 * i + k] & 0xffff0000u)),
                            make_float2(up, up));
              const uint16_t h0 = pack_e4m3(x[0].x, x[0].y), h1 = pack_e4m3(x[1].x, x[1].y);
              const float2 f0 = unpack_e4m3(h0), f1 = unpack_e4m3(h1);
              const float2 y0 = mul2(add2(x[0], make_float2(-f0.x, -f0.y)), make_float2(16.f, 16.f));
              const float2 y1 = mul2(add2(x[1], make_float2(-f1.x, -f1.y)), make_float2(16.f, 16.f));
              hi[i] = h0 | (uint32_t)h1 << 16;
              lo[i] = pack_e4m3(y0.x, y0.y) | (uint32_t)pack_e4m3(y1.x, y1.y) << 16;
            }
            if (in) {
              *reinterpret_cast<uint4 *>(place(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4 *>(place(RP + r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (c == 0) S.qs[s % kSegs][r] = down * ks;
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.q_full[qb]);
        mbar_arrive(&S.seg_empty[s % kSegs]);
      }
    }
  } else {
    // ---------------- softmax and output: a thread per key (then per dim) and kRows rows
    constexpr int R = C::kRows;
    const uint32_t quarter = warp & 3, me = quarter * 32 + lane, half = (warp - 4) / 4;
    const uint32_t t_lane = (quarter * 32) << 16, t_o = tmem + t_lane, t_s = tmem + o_cols + t_lane;
    // the group's rows in eights: this set's i-th eight start at row8(i); element r of its arrays is
    // row row8(r / 8) + r % 8
    constexpr int E = R / 8;
    auto row8 = [&](uint32_t i) { return (C::kSets * i + half) * 8; };
    constexpr uint32_t kGroup = C::kWarps * 32;
    uint32_t sc = 0, pv = 0, base = 0;   // score tiles, weight tiles, loads of the segments before
    Part part = {};
    bool ok = true;   // (false: a wait has run out; no more are made, and the results are void)
    // a row's score in units of log2 is x c2; that of a key that it does not see is -infinity
    const float c2 = F8 ? 1.f : P.c2, unseen = c2 > 0.f ? -INFINITY : INFINITY;
    auto p_buf = [&](uint32_t n) { return P.n_p == 2 ? n & 1 : 0u; };
    auto p_use = [&](uint32_t n) { return P.n_p == 2 ? n >> 1 : n; };
    // the output product n is done
    auto pv_wait = [&](uint32_t n) { ok = ok && wait_chain(&S.pv_done[p_buf(n)], p_use(n) & 1, err); };
    for (uint32_t s = 0;; ++s) {
      ok = ok && wait_chain(&S.seg_full[s % kSegs], (s / kSegs) & 1, err);
      if (group_any(!ok, kGroup)) break;
      const Segment sg = S.seg[s % kSegs];
      if (sg.nt == 0) {
        warps_arrive(&S.seg_empty[s % kSegs], lane);
        break;
      }
      const uint32_t tok_a = by_group(P, sg.r0);
      const uint32_t p_first = sg.pos0 + tok_a, p_last = sg.pos0 + by_group(P, sg.r0 + sg.nr - 1);
      if (half == 0 && me < RP) {
        const uint32_t tok = by_group(P, sg.r0 + me);
        S.row_out[me] = (uint64_t)(sg.first + tok) * a.n_heads + (sg.kh * P.G + sg.r0 + me - tok * P.G);
      }
      float l[R], nm[R];   // sums of this thread's keys, -references
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;
      // 8 bits. Threads me < RP of the first set know a sum of their row, exact at the tiles `next` and a lower bound after
      // new references, and tell which rows' are enough for tile j on (those behind the last row's are).
      float known = 0.f;
      auto put_enough = [&](uint32_t j) {
        const uint32_t lanes = RP < 32 ? (1u << (RP & 31)) - 1 : ~0u, eight = me / 8;
        const bool none = me >= sg.nr, yes = none || known >= kEnough * (float)min(next_look(j), sg.nt);
        const uint32_t bit = yes ? 1u << (eight / C::kSets * 8 + me % 8) : 0u;
#pragma unroll
        for (uint32_t i = 0; i < C::kSets; ++i) {
          const uint32_t rows = __reduce_or_sync(lanes, eight % C::kSets == i ? bit : 0u);
          if (lane == 0) S.enough[i][me / 32] = rows;
        }
        const bool settled = __all_sync(lanes, none || known >= kEnough * (float)sg.nt);
        if (lane == 0) S.settled[me / 32] = settled;
      };
      auto enough = [&](uint32_t i) { return (S.enough[i][0] | (RP == 64 ? S.enough[i][1] : 0u)) & C::kAll; };
      // whether some row's is not enough, and whether the tile before was watched
      uint32_t next = kSure;
      bool watch = false, watched = false;
      auto take_enough = [&](uint32_t j) {
        watch = (enough(0) & (C::kSets == 2 ? enough(1) : ~0u) & C::kAll) != C::kAll;
        next = S.settled[0] && (RP < 64 || S.settled[1]) ? ~0u : next_look(j);
        watched = false;
      };
      BlockList bl;
      bl.start();
      for (uint32_t j = 0; j < sg.nt; ++j, ++pv, ++sc) {
        if (F8 && j == next) {
          float v[R];
#pragma unroll
          for (int r = 0; r < R; ++r) v[r] = l[r];
          const float sum = warp_reduce_rows(v, lane, [](float u, float v) { return u + v; });
          const uint32_t r = lane / (32 / R);
          if (lane % (32 / R) == 0) S.wmax[quarter][row8(r / 8) + r % 8] = sum;
          group_bar(kGroup);
          if (half == 0 && me < RP) {
            known = S.wmax[0][me] + S.wmax[1][me] + S.wmax[2][me] + S.wmax[3][me];
            put_enough(j);
          }
          group_bar(kGroup);
          take_enough(j);
        }
        const uint32_t tile = sg.tile0 + j, key0 = tile * kTile, key = key0 + me, sb = sc & 1;
        bl.look(a, sg.b, tile / 2, lane);
        ok = ok && wait_chain(&S.s_full[sb], (sc >> 1) & 1, err);
        tc_fence_after();
        const bool held = bl.at(tile / 2) < a.n_blocks;
        const bool plain = held && key0 + kTile - 1 <= p_first && (!a.window || p_last - key0 < a.window);
        // (eights behind the last row are left out: nothing reads their columns)
        float x[R];   // scores
#pragma unroll
        for (int e = 0; e < E; ++e) {
          uint32_t v[8], w[8];
          if (e && row8(e) >= sg.nr) break;
          tmem_ld8(t_s + sb * C::kQRows + row8(e), v);
          if (F8) tmem_ld8(t_s + sb * C::kQRows + RP + row8(e), w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float2 u = make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            if (F8) {   // (in units of log2)
              u = fma2(make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), make_float2(0.0625f, 0.0625f), u);
              u = mul2(u, *reinterpret_cast<const float2 *>(&S.qs[s % kSegs][row8(e) + i]));
            }
            x[8 * e + i] = u.x;
            x[8 * e + i + 1] = u.y;
          }
        }
        tc_fence_before();
        warps_arrive(&S.s_empty[sb], lane);
        if (!plain) {   // unseen keys
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (e && row8(e) >= sg.nr) break;
            const uint32_t tok = by_group(P, sg.r0 + row8(e));
            uint32_t p = sg.pos0 + tok, g = sg.r0 + row8(e) - tok * P.G;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (!held || key > p || (a.window && p - key >= a.window)) x[8 * e + i] = unseen;
              if (++g == P.G) {
                g = 0;
                ++p;
              }
            }
          }
        }
        bool over = j == 0;   // a weight passes the margin, or (8 bits) a row's had fallen in the tile before
        if (j) {
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (e && row8(e) >= sg.nr) break;
#pragma unroll
            for (int r = 8 * e; r < 8 * e + 8; r += 2) {
              const float2 y = fma2(make_float2(x[r], x[r + 1]), make_float2(c2, c2), make_float2(nm[r], nm[r + 1]));
              top = fmaxf(top, fmaxf(y.x, y.y));
            }
          }
          bool low = false;
          if (F8 && watch) {
            uint32_t fine = ~0u;
            if (plain) {   // (keys that are not there say nothing)
#pragma unroll
              for (int e = 0; e < E; ++e) {
                if (e && row8(e) >= sg.nr) break;
#pragma unroll
                for (int r = 8 * e; r < 8 * e + 8; ++r)
                  if (fmaf(x[r], c2, nm[r]) < kLow) fine &= ~(1u << r);
              }
            }
            fine = __reduce_or_sync(0xffffffffu, fine);
            if (lane == 0) S.fine[sc & 1][warp - 4] = fine;
            if (watched)
#pragma unroll
              for (uint32_t i = 0; i < C::kSets; ++i) {
                const uint4 f = *reinterpret_cast<const uint4 *>(&S.fine[sc & 1 ^ 1][4 * i]);
                low |= ((f.x | f.y | f.z | f.w | enough(i)) & C::kAll) != C::kAll;
              }
            watched = true;
          }
          over = group_any(top > C::kTop || low, kGroup);
        }
        if (over) {   // new references, sums so far brought to them
          {
            float m[R];
#pragma unroll
            for (int r = 0; r < R; ++r) m[r] = x[r] * c2;
            const float top = warp_reduce_rows(m, lane, [](float u, float v) { return max_nan(u, v); });
            const uint32_t r = lane / (32 / R);
            if (lane % (32 / R) == 0) S.wmax[quarter][row8(r / 8) + r % 8] = top;
          }
          group_bar(kGroup);
          if (half == 0 && me < RP) {
            float m = S.wmax[0][me];
#pragma unroll
            for (int i = 1; i < 4; ++i) m = max_nan(m, S.wmax[i][me]);
            const float was = j ? S.negm[me] : kNoRef;
            float now;
            if constexpr (F8) {
              const float to = C::kOff - m, all = kEnough * (float)sg.nt;
              now = m == -INFINITY ? was : fminf(was, to);
              if (j && m + was < kLow && m != -INFINITY && known < kEnough * (float)min(next_look(j), sg.nt))
                now = fminf(to, was + ceilf(log2f(all / known)));   // (no lower than is enough for all tiles)
              if (m != m) now = m;
              known = known * ex2_approx(now - was) + ex2_approx(m + now);   // (its largest weight among them)
              if (j) put_enough(j);
            } else {
              const float least = m == -INFINITY ? was : fminf(was, C::kOff - m);
              now = m != m ? m : least;   // (fminf drops a NaN)
            }
            S.fac[me] = ex2_approx(now - was);
            S.negm[me] = now;
          }
          group_bar(kGroup);
#pragma unroll
          for (int r = 0; r < R; ++r) nm[r] = S.negm[row8(r / 8) + r % 8];
          if (F8 && j) {
            take_enough(j);
            if (watch) next = j + 1;   // (perhaps they are: the sums are looked at)
            watch = false;
          }
          if (j) {
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] *= S.fac[row8(r / 8) + r % 8];
            pv_wait(pv - 1);
            tc_fence_after();
#pragma unroll 1
            for (uint32_t c = 0; c < o_cols; c += RP)   // (hi and lo of each 128 dims)
#pragma unroll 1
              for (uint32_t e = 0; e < (uint32_t)E; ++e) {
                uint32_t v[8];
                tmem_ld8(t_o + c + row8(e), v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * S.fac[row8(e) + i]);
                tmem_st8(t_o + c + row8(e), v);
              }
            tmem_st_wait();
          }
        }
        // ---- weights, in two parts each
        if (pv >= P.n_p) pv_wait(pv - P.n_p);   // (the product before has read this place)
        uint8_t *dst = s_p + p_buf(pv) * C::kPBytes + (me / 8) * 128 + (me % 8) * 16;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (e && row8(e) >= sg.nr) break;
          uint32_t hi[4], lo[4];   // (8 bits: 16 of them, in two words each)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * e + 2 * i;
            const float2 y = fma2(make_float2(x[r], x[r + 1]), make_float2(c2, c2), make_float2(nm[r], nm[r + 1]));
            const float2 w = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            const float2 sum = add2(make_float2(l[r], l[r + 1]), w);
            l[r] = sum.x;
            l[r + 1] = sum.y;
            float2 h;
            if (F8) {
              hi[i] = pack_e4m3(w.x, w.y);
              h = unpack_e4m3((uint16_t)hi[i]);
            } else {   // (cut off rather than rounded)
              const uint32_t b0 = __float_as_uint(w.x), b1 = __float_as_uint(w.y);
              hi[i] = __byte_perm(b0, b1, 0x7632);
              h = make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u));
            }
            float2 rest = add2(w, make_float2(-h.x, -h.y));
            if (F8) rest = mul2(rest, make_float2(16.f, 16.f));
            lo[i] = F8 ? pack_e4m3(rest.x, rest.y) : pack_bf16(rest.x, rest.y);
          }
          if constexpr (!F8) {
            *reinterpret_cast<uint4 *>(dst + row8(e) / 8 * 2048) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(dst + (RP + row8(e)) / 8 * 2048) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            const uint2 h2 = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            const uint2 l2 = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            if constexpr (RP == 8) {
              *reinterpret_cast<uint4 *>(dst) = make_uint4(h2.x, h2.y, l2.x, l2.y);
            } else {   // (16 rows to 16 bytes)
              *reinterpret_cast<uint2 *>(dst + row8(e) / 16 * 2048 + row8(e) % 16) = h2;
              *reinterpret_cast<uint2 *>(dst + (RP + row8(e)) / 16 * 2048 + row8(e) % 16) = l2;
            }
          }
        }
        if (!plain && half == 0) {
          const bool all = held && key <= p_first && (!a.window || p_last - key < a.window);
          const bool any = held && key <= p_last && !(a.window && key < p_first && p_first - key >= a.window);
          // (the values are there: a slot is refilled only behind the products that this arrival starts)
          for (uint32_t m = 0; m < P.nmb; ++m) {
            const uint32_t k = (base + place_v(j, sg.nt)) * P.nmb + m, slot = k % P.n_slots;
            ok = ok && wait_chain(&S.full[slot], (k / P.n_slots) & 1, err);
            if (!all && clean_row<F8>(smem_u32(s_slot + slot * slot_bytes) + me * 128, P.ubox, !any, lane)) S.bad = 1;
            __syncwarp();
          }
        }
        fence_proxy_async();
        tc_fence_before();
        warps_arrive(&S.p_full[p_buf(pv)], lane);
      }
      base += 2 * sg.nt;
      // ---- the segment's end: sums over the keys, then the output, a thread per dim
      {
        const float sum = warp_reduce_rows(l, lane, [](float u, float v) { return u + v; });
        const uint32_t r = lane / (32 / R);
        if (lane % (32 / R) == 0) S.wmax[quarter][row8(r / 8) + r % 8] = sum;
      }
      group_bar(kGroup);
      const bool whole = sg.whole == 3, bad = *(volatile uint32_t *)&S.bad != 0;
      const uint32_t side = sg.whole & 1;   // (a part: 0 began in an earlier block, 1 goes on in the next)
      float *sums = P.sums + ((size_t)blockIdx.x * 2 + side) * RP * D;
      if (half == 0 && me < sg.nr) {
        const float sum = S.wmax[0][me] + S.wmax[1][me] + S.wmax[2][me] + S.wmax[3][me];
        if (whole) {
          if (a.lse)
            a.lse[S.row_out[me]] = sum == 0.f ? -INFINITY : (log2f(sum) - S.negm[me]) * 0.6931471805599453f;
        } else {
          float *ml = P.sums + (size_t)gridDim.x * 2 * RP * D + (((size_t)blockIdx.x * 2 + side) * RP + me) * 2;
          ml[0] = -S.negm[me];
          ml[1] = sum;
        }
        S.fac[me] = sum == 0.f ? 0.f : (F8 ? __ldg(a.v_scale + sg.kh) : 1.f) / sum;
      }
      pv_wait(pv - 1);
      tc_fence_after();
      group_bar(kGroup);
#pragma unroll 1
      for (uint32_t m = 0; m < P.nmb; ++m) {
        const uint32_t d = m * 128 + me;
#pragma unroll 1
        for (uint32_t e = 0; e < (uint32_t)E && row8(e) < sg.nr; ++e) {
          const uint32_t r0 = row8(e), nr = sg.nr - r0;
          uint32_t hi[8], lo[8];
          tmem_ld8(t_o + m * 2 * RP + r0, hi);
          tmem_ld8(t_o + m * 2 * RP + RP + r0, lo);
          tmem_ld_wait();
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o[i] = F8 ? fmaf(__uint_as_float(lo[i]), 0.0625f, __uint_as_float(hi[i]))
                      : __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
          if (bad && d < D)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < nr) o[i] += taken_out<F8>(a, sg, sg.pos0 + by_group(P, sg.r0 + r0 + i), p_first, p_last, d);
          if (d < D) {
            if (whole) {
              __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + d;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < nr) out[S.row_out[r0 + i] * D] = __float2bfloat16_rn(o[i] * S.fac[r0 + i]);
            } else {
              float *out = sums + (size_t)r0 * D + d;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < nr) out[(size_t)i * D] = o[i];
            }
          }
          __syncwarp();
        }
      }
      if (!whole && side) part = Part{sg.blocks, sg.kh, sg.r0, sg.nr, sg.first, {0u, 0u, 0u}};
      tc_fence_before();
      group_bar(kGroup);   // (the shared sums are free)
      if (half == 0 && me == 0) S.bad = 0;
      if (lane == 0) {
        mbar_arrive(&S.o_free);
        mbar_arrive(&S.seg_empty[s % kSegs]);
      }
    }
    if (half == 0 && me == 0) P.parts[blockIdx.x] = part;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, alloc);
  }
}

// Joins the parts of what begins in block blockIdx.x and goes on behind it, each row as the sum of its
// parts brought to the largest reference, always in the same order. Two rows at once, four warps
// each: a warp takes every fourth part, 32 parts on their way at once, and works out the
// weights of all parts for itself, a lane each.
constexpr uint32_t kJoinRows = 2, kJoinWarps = 4, kJoinThreads = 32 * kJoinWarps * kJoinRows;
template <int RP, bool F8, int DV>   // (D <= 128 DV)
__global__ void __launch_bounds__(kJoinThreads) paged_join_tc_kernel(Params P, uint32_t blocks) {
  __shared__ float4 s_acc[kJoinRows][kJoinWarps][32 * DV];
  const PagedArgs &a = P.a;
  const uint32_t c0 = blockIdx.x, D = a.head_dim, D4 = D / 4;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32 % kJoinWarps, sub = threadIdx.x / (32 * kJoinWarps);
  const float2 *ml = reinterpret_cast<const float2 *>(P.sums + (size_t)blocks * 2 * RP * D);
  // piece i: block c0 + i, what goes on (i = 0) or what began before
  auto at = [&](uint32_t i, uint32_t r) { return ((size_t)(c0 + i) * 2 + (i ? 0u : 1u)) * RP + r; };
  pdl_wait();
  pdl_trigger();
  const Part part = P.parts[c0];
  const uint32_t n = part.blocks + 1;   // pieces
  if (n == 1 || c0 + n > blocks) return;
  for (uint32_t r0 = blockIdx.y * kJoinRows; r0 < part.nr; r0 += gridDim.y * kJoinRows) {
    const uint32_t r = min(r0 + sub, part.nr - 1);   // (the last one twice)
    float2 mine = lane < n ? ml[at(lane, r)] : make_float2(-kNoRef, 0.f);
    float4 v[8][DV];
    auto fetch = [&](uint32_t i0) {
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) {
        const uint32_t i = i0 + warp + kJoinWarps * u;
#pragma unroll
        for (uint32_t k = 0; k < DV; ++k)
          if (i < n && lane + 32 * k < D4) v[u][k] = reinterpret_cast<const float4 *>(P.sums + at(i, r) * D)[lane + 32 * k];
      }
    };
    fetch(0);
    // the largest reference (a NaN if there is one)
    float m = mine.x;
    for (uint32_t i = lane + 32; i < n; i += 32) m = max_nan(m, ml[at(i, r)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    float4 acc[DV];
#pragma unroll
    for (int k = 0; k < DV; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t i0 = 0; i0 < n; i0 += 32) {
      if (i0) {
        mine = i0 + lane < n ? ml[at(i0 + lane, r)] : make_float2(-kNoRef, 0.f);
        fetch(i0);
      }
      const float w = mine.x <= -kNoRef ? -0.f : ex2_approx(mine.x - m);   // (-0: no key of the part is seen)
      l = fmaf(mine.y, w, l);
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) {
        const uint32_t i = warp + kJoinWarps * u;
        const float f = __shfl_sync(0xffffffffu, w, i);
        if (i0 + i < n && __float_as_uint(f) != 0x80000000u)   // (a NaN times 0 is one)
#pragma unroll
          for (int k = 0; k < DV; ++k) {
            acc[k].x = fmaf(v[u][k].x, f, acc[k].x);
            acc[k].y = fmaf(v[u][k].y, f, acc[k].y);
            acc[k].z = fmaf(v[u][k].z, f, acc[k].z);
            acc[k].w = fmaf(v[u][k].w, f, acc[k].w);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < DV; ++k) s_acc[sub][warp][lane + 32 * k] = acc[k];
    __syncthreads();
    l = warp_sum(l);
    const uint32_t row = part.r0 + r, tok = by_group(P, row);
    const size_t out = (size_t)(part.first + tok) * a.n_heads + (part.kh * P.G + row - tok * P.G);
    const float scale = l == 0.f ? 0.f : (F8 ? __ldg(a.v_scale + part.kh) : 1.f) / l;
    if (r0 + sub < part.nr) {
      const float *sums = reinterpret_cast<const float *>(s_acc[sub]);
      for (uint32_t d = warp * 32 + lane; d < D; d += 32 * kJoinWarps) {
        float o = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < kJoinWarps; ++w) o += sums[w * 128 * DV + d];
        static_cast<__nv_bfloat16 *>(a.out)[out * D + d] = __float2bfloat16_rn(o * scale);
      }
      if (a.lse && warp == 0 && lane == 0) a.lse[out] = l == 0.f ? -INFINITY : (log2f(l) + m) * 0.6931471805599453f;
    }
    __syncthreads();   // (the sums are free)
  }
}

// Rows of a group: the fewest that hold a sequence's, up to 64 (19 sequences of 8,192 tokens, 8 heads of 128 dims: 64 rows
// in groups of 64 / 32 / 16 take 108 / 189 / 192 us in bf16 and 111 / 140 / 145 over 8 bits; 8 rows in groups of 8 / 16 / 32
// 59 / 60 / 65 over 8 bits, with 128 tokens each 8.7 / 10.2 / 10.0).
uint32_t rows_of(const PagedArgs &a) {
  const uint32_t r = a.max_new * (a.n_heads / a.n_kv);
  return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : 64;
}

// The most tiles that a sequence can have.
uint64_t most_tiles(const PagedArgs &a) {
  const uint64_t all = 2ull * a.max_blocks, w = ((uint64_t)a.window + a.max_new) / kTile + 2;
  return a.window && w < all ? w : all;
}

// Blocks: one or two a SM (Cfg::kPerSm), or one a tile where there can be no more tiles.
uint32_t blocks_of(const PagedArgs &a) {
  const uint32_t rp = rows_of(a), groups = (a.max_new * (a.n_heads / a.n_kv) + rp - 1) / rp;
  uint64_t tiles = most_tiles(a);
  if (tiles <= kWholeTiles) tiles = 1;
  const uint64_t most = tiles * a.batch * a.n_kv * groups, sms = (uint64_t)num_sms() * (rp <= 16 ? 2 : 1);
  return (uint32_t)(most < sms ? most : sms);
}

cudaError_t make_map(CUtensorMap *m, const PagedArgs &a, const void *pool) {
  const uint64_t rows = (uint64_t)a.n_blocks * a.n_kv * 256;
  const bool f8 = a.kv_dtype == DS4A_E4M3;
  const uint64_t dims[2] = {a.head_dim, rows}, strides[1] = {(uint64_t)a.head_dim * (f8 ? 1 : 2)};
  const uint32_t box[2] = {f8 ? 128u : 64u, kTile};
  return f8 ? make_tmap_u8(m, pool, 2, dims, strides, box) : make_tmap_bf16(m, pool, 2, dims, strides, box);
}

template <int RP, bool F8>
cudaError_t launch_rp(const PagedArgs &a, cudaStream_t s) {
  using C = Cfg<RP, F8>;
  CUtensorMap mk, mv;
  cudaError_t e = make_map(&mk, a, a.k);
  if (e == cudaSuccess) e = make_map(&mv, a, a.v);
  if (e != cudaSuccess) return e;
  Params P;
  P.a = a;
  P.G = a.n_heads / a.n_kv;
  P.nbox = (a.head_dim * (F8 ? 1 : 2) + 127) / 128;
  P.nmb = (a.head_dim + 127) / 128;
  P.q_vec = aligned(16, {a.q}) && a.q_stride % 8 == 0;
  P.c2 = a.scale * 1.4426950408889634f;
  if (fabsf(P.c2) < 0x1p-126f) P.c2 = 0x1p-126f;   // (0 times the -infinity of an unseen key is a NaN)
  P.whole = most_tiles(a) <= kWholeTiles;
  P.ubox = F8 || P.nbox == 1 ? 1 : 2;
  P.g_mul = P.G > 1 ? (uint32_t)((1ull << 32) / P.G) + 1u : 0u;
  const uint32_t blocks = blocks_of(a), slot = P.ubox * kBox, q = C::kQRows * P.nbox * 128u;
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  P.err = reinterpret_cast<int *>(ws);
  P.parts = reinterpret_cast<Part *>(ws + 256);
  P.sums = reinterpret_cast<float *>(ws + 256 + (size_t)blocks * sizeof(Part));
  // two query and two weight tiles where four units fit beside them
  const uint32_t room = kSmemSm / C::kPerSm - kSmemBlock - 1024 - (uint32_t)sizeof(Shared<RP>);
  P.n_q = P.n_p = room >= 2 * (q + C::kPBytes) + 4 * slot ? 2 : 1;
  P.n_slots = (room - P.n_q * (q + C::kPBytes)) / slot;
  if (P.n_slots > kMaxSlots) P.n_slots = kMaxSlots;
  const size_t smem = 1024 + (size_t)P.n_slots * slot + P.n_q * (q + C::kPBytes) + sizeof(Shared<RP>);
  static RaisedLimit smem_set;
  auto *k = paged_attn_tc_kernel<RP, F8>;
  e = ensure_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(blocks), dim3(C::kThreads), smem, s, mk, mv, P);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (blocks > 1 && !P.whole) {   // (a lone block holds every segment whole)
    auto *join = a.head_dim <= 128 ? paged_join_tc_kernel<RP, F8, 1> : paged_join_tc_kernel<RP, F8, 2>;
    e = launch_pdl(join, dim3(blocks - 1, (RP < 32 ? RP : 32) / kJoinRows), dim3(kJoinThreads), 0, s, P, blocks);
    if (e != cudaSuccess) return e;
    note_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace

bool paged_attn_tc_takes(const PagedArgs &a) {
  return a.dtype == DS4A_BF16 && a.head_dim % (a.kv_dtype == DS4A_E4M3 ? 16 : 8) == 0;
}

size_t paged_attn_tc_ws_bytes(const PagedArgs &a) {
  return (size_t)blocks_of(a) * (sizeof(Part) + 2 * (size_t)rows_of(a) * (a.head_dim + 2) * 4);
}

cudaError_t launch_paged_attn_tc(const PagedArgs &a, cudaStream_t s) {
  const bool f8 = a.kv_dtype == DS4A_E4M3;
  switch (rows_of(a)) {
    case 8: return f8 ? launch_rp<8, true>(a, s) : launch_rp<8, false>(a, s);
    case 16: return f8 ? launch_rp<16, true>(a, s) : launch_rp<16, false>(a, s);
    case 32: return f8 ? launch_rp<32, true>(a, s) : launch_rp<32, false>(a, s);
    default: return f8 ? launch_rp<64, true>(a, s) : launch_rp<64, false>(a, s);
  }
}

}  // namespace ds4a
