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
// split into two 8-bit floats, x = hi + lo / 16, whose products with the codes are exact; a bf16
// query has 8 significant bits, hi and lo 4 each, so only entries below 2^-9 of the row's
// largest lose any. Sums are fp32.
//
// Work. The tiles of all sequences, key heads and row groups are one list, of which each block
// takes an even share, whatever the lengths. A part of a (sequence, key head, group) that a block
// does not hold whole is left as sums with their reference, and a second launch joins
// the parts in order. Bound by HBM: every visible key and value is read once.
//
// Warps: 0 TMA, 1 MMA, 2 the block's list of segments, 3 queries, 4 .. 7 softmax and output.
// Every wait is bounded (tc.cuh).
#include <cuda_fp8.h>

#include "paged.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kTile = 128, kThreads = 256, kBox = kTile * 128;   // keys; bytes of a 128-byte column
constexpr uint32_t kSegs = 4, kMaxSlots = 16;
constexpr uint32_t kSmemMost = 227 * 1024, kFixed = 8192;
constexpr float kNoRef = 3e38f;   // -reference of a row that has seen no key

struct Segment {
  uint32_t b, kh, r0, nr;          // sequence, key head, first row and rows
  uint32_t first, pos0;            // packed index and position of the sequence's first token
  uint32_t tile0, nt;              // tiles (of 128 positions); nt 0: no more segments
  uint32_t whole;                  // bit 0: its first tile is here, bit 1: its last
};

// What a block left of the segments that it does not hold whole: [0] the one that began before,
// [1] the one that goes on.
struct Part {
  uint32_t valid, last, b, kh, r0, nr, first, pad;
};

struct Params {
  PagedArgs a;
  uint32_t G;           // query heads per key head
  uint32_t nbox, nmb;   // 128-byte columns of a key's row; blocks of 128 dims of the output
  uint32_t n_slots, n_q;
  uint32_t q_vec;       // queries start on 16 bytes
  float c2;             // scale * log2(e)
  Part *parts;          // [blocks][2]
  float *sums;          // [blocks][2][RP][D], then (reference, sum) [blocks][2][RP][2]
  int *err;
};

template <int RP, bool F8>
struct Cfg {
  static constexpr uint32_t kQRows = F8 ? 2 * RP : (RP < 16 ? 16 : RP);   // rows of the Q operand
  static constexpr uint32_t kPBytes = kTile * 2 * RP * (F8 ? 1 : 2);
  static constexpr float kOff = F8 ? 5.f : 0.f;     // weights are 2^(s - m + kOff)
  static constexpr float kTop = F8 ? 8.75f : 8.f;   // ... and at most 2^kTop (448 for 8 bits)
};

struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full[2], q_empty[2], s_full[2], s_empty[2];
  uint64_t p_full, pv_done, o_free, group, drain;
  uint32_t tmem;
  uint32_t start_b;
  uint64_t start_off, start_n;
  uint64_t scan[kThreads / 32];
  uint32_t over[3], bad;
  Segment seg[kSegs];
  alignas(16) float qs[kSegs][64];   // factor of each row's scores (8-bit queries)
  alignas(16) float negm[64];        // -reference of each row
  alignas(16) float fac[64];
  alignas(16) float wmax[4][64];
};
static_assert(sizeof(Shared) <= kFixed - 1024, "fixed shared memory");

// Products with 8-bit operands, both E4M3, fp32 sums.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// Descriptor of an operand without swizzle, MN-major: 16 bytes along N by 8 along K are 128
// contiguous bytes; k_step bytes to the next 8 along K, mn_step to the next 16 bytes along N.
__device__ __forceinline__ uint64_t sdesc_plain_mn(uint32_t addr, uint32_t k_step, uint32_t mn_step) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(k_step >> 4) << 16) | ((uint64_t)(mn_step >> 4) << 32) |
         ((uint64_t)1 << 46);
}

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

// Largest value of the warp, a NaN if there is one (as FMA makes them).
__device__ __forceinline__ float warp_max_nan(float v) {
  const uint32_t u = __float_as_uint(v);
  const uint32_t k = redux_max_u32((u & 0x80000000u) ? ~u : u | 0x80000000u);
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// One arrival and one bounded wait for each of the softmax's four warps.
__device__ __forceinline__ bool warps_sync(uint64_t *bar, uint32_t &phase, uint32_t lane, ErrWord err) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  const bool ok = mbar_wait_warp(bar, phase, err);
  phase ^= 1;
  return ok;
}

__device__ __forceinline__ uint32_t tiles_of(const PagedItem &it) {
  if (it.cnt == 0) return 0;
  return it.hi > it.lo ? (it.hi + kTile - 1) / kTile - it.lo / kTile : 1u;   // (one without keys writes zeros)
}

// Physical block of logical block j of sequence b; n_blocks or more: not there.
__device__ __forceinline__ uint32_t phys_of(const PagedArgs &a, uint32_t b, uint32_t j) {
  return j < a.max_blocks ? (uint32_t)__ldg(a.table + (size_t)b * a.max_blocks + j) : 0xffffffffu;
}

// Physical block of a tile, from 32 entries at a time in the warp's lanes.
struct BlockList {
  uint32_t base, mine;
  __device__ __forceinline__ void start() { base = 0xffffffffu; }
  __device__ __forceinline__ uint32_t at(const PagedArgs &a, uint32_t b, uint32_t j, uint32_t lane) {
    if (base == 0xffffffffu || j - base >= 32) {
      base = j;
      mine = phys_of(a, b, j + lane);
    }
    return __shfl_sync(0xffffffffu, mine, j - base);
  }
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
// shared memory: 0 times them would be a NaN. Returns whether there were any of the latter.
template <bool F8>
__device__ __noinline__ bool clean_row(uint32_t row, uint32_t nbox, bool all) {
  bool found = false;
  for (uint32_t x = 0; x < nbox; ++x)
    for (uint32_t c = 0; c < 8; ++c) {
      const uint32_t at = row + x * kBox + 16 * c;
      uint32_t v[4] = {0, 0, 0, 0};
      if (!all) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(at));
        bool here = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t keep = 0;
          if (F8) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) keep |= (v[i] >> k & 0x7fu) == 0x7fu ? 0u : 0xffu << k;
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 16) keep |= (v[i] >> k & 0x7f80u) == 0x7f80u ? 0u : 0xffffu << k;
          }
          here |= keep != 0xffffffffu;
          v[i] &= keep;
        }
        if (!here) continue;
        found = true;
      }
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                   : "memory");
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
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, Params P) {
  using C = Cfg<RP, F8>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const PagedArgs &a = P.a;
  const uint32_t slot_bytes = P.nbox * kBox, q_bytes = C::kQRows * P.nbox * 128u;
  uint8_t *s_slot = smem, *s_q = s_slot + P.n_slots * slot_bytes, *s_p = s_q + P.n_q * q_bytes;
  Shared &S = *reinterpret_cast<Shared *>(s_p + C::kPBytes);
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5, D = a.head_dim;
  const uint32_t o_cols = P.nmb * 2 * RP;   // output sums, then two score tiles
  const uint32_t cols = o_cols + 2 * C::kQRows;
  const uint32_t alloc = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;

  if (t == 0) {
    for (uint32_t i = 0; i < P.n_slots; ++i) mbar_init(&S.full[i], 1), mbar_init(&S.empty[i], 1);
    for (uint32_t i = 0; i < kSegs; ++i) mbar_init(&S.seg_full[i], 1), mbar_init(&S.seg_empty[i], 7);
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.s_empty[i], 4);
    }
    mbar_init(&S.p_full, 4);
    mbar_init(&S.pv_done, 1);
    mbar_init(&S.o_free, 4);
    mbar_init(&S.group, 4);
    mbar_init(&S.drain, 1);
    S.start_n = 0;
    S.over[0] = S.over[1] = S.over[2] = S.bad = 0;
    fence_mbar_init();
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 1) tmem_alloc(&S.tmem, alloc);
  pdl_wait();
  pdl_trigger();
  const ErrWord err{P.err, *(volatile int *)P.err};
  // ---- the block's share of the list of tiles: each thread counts some sequences'
  {
    const uint32_t per = (a.batch + kThreads - 1) / kThreads, b0 = min(a.batch, t * per), b1 = min(a.batch, b0 + per);
    auto weight = [&](uint32_t b) {
      const PagedItem it = paged_item(a, b);
      return (uint64_t)tiles_of(it) * a.n_kv * ((it.cnt * P.G + RP - 1) / RP);
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
    // (no more shares than tiles, so that the parts of a segment are in neighbouring blocks)
    const uint64_t shares = min((uint64_t)gridDim.x, total), c = blockIdx.x;
    const uint64_t from = c < shares ? total * c / shares : total, to = c < shares ? total * (c + 1) / shares : total;
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
      if (!mbar_wait_warp(&S.seg_full[s % kSegs], (s / kSegs) & 1, err)) break;
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
        uint32_t phys = is_v ? vl.at(a, sg.b, tile / 2, lane) : kl.at(a, sg.b, tile / 2, lane);
        if (phys >= a.n_blocks) phys = 0;   // (its keys are masked)
        ok = mbar_wait_warp(&S.empty[ring.slot], ring.phase ^ 1, err);
        if (!ok) break;
        if (lane == 0) {
          uint64_t *bar = &S.full[ring.slot];
          uint8_t *dst = s_slot + ring.slot * slot_bytes;
          mbar_arrive_expect_tx(bar, slot_bytes);
          const int y = (int)((phys * a.n_kv + sg.kh) * 256u + (tile & 1) * kTile);
          for (uint32_t x = 0; x < P.nbox; ++x)
            tma_load_2d_hint(dst + x * kBox, is_v ? &map_v : &map_k, bar, (int)(x * (F8 ? 128 : 64)), y, policy);
        }
        ++issued;
        ring.next(P.n_slots);
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
    // ---------------- MMA
    if (lane == 0) {
      constexpr uint32_t kFmt = F8 ? (1u << 4) : (1u << 4) | (1u << 7) | (1u << 10);
      constexpr uint32_t id_s = kFmt | ((C::kQRows >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t id_o = kFmt | ((2u * RP >> 3) << 17) | ((128u >> 4) << 24) | kIdescMajorA_MN | kIdescMajorB_MN;
      const uint32_t slot0 = smem_u32(s_slot), q0 = smem_u32(s_q), p0 = smem_u32(s_p);
      const uint32_t t_o = tmem, t_s = tmem + o_cols;
      Ring ring{0, 0};
      uint32_t sc = 0, pv = 0;   // score tiles issued, output products issued
      bool ok = true;
      uint32_t qb = 0;
      auto scores = [&]() {
        const uint32_t sb = sc & 1;
        if (!mbar_wait(&S.s_empty[sb], ((sc >> 1) & 1) ^ 1, err) || !mbar_wait(&S.full[ring.slot], ring.phase, err))
          return false;
        tc_fence_after();
        for (uint32_t x = 0; x < P.nbox; ++x) {
          const uint32_t ka = slot0 + ring.slot * slot_bytes + x * kBox, qa = q0 + qb * q_bytes + x * C::kQRows * 128u;
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            const uint64_t ad = sdesc_sw128(ka + 32 * k), bd = sdesc_sw128(qa + 32 * k);
            if (F8)
              mma_e4m3(t_s + sb * C::kQRows, ad, bd, id_s, x | k);
            else
              mma_bf16(t_s + sb * C::kQRows, ad, bd, id_s, x | k);
          }
        }
        mma_commit(&S.empty[ring.slot]);
        mma_commit(&S.s_full[sb]);
        ring.next(P.n_slots);
        ++sc;
        return true;
      };
      for (uint32_t s = 0; ok; ++s) {
        if (!(ok = mbar_wait(&S.seg_full[s % kSegs], (s / kSegs) & 1, err))) break;
        const uint32_t nt = S.seg[s % kSegs].nt;
        mbar_arrive(&S.seg_empty[s % kSegs]);
        if (nt == 0) break;
        qb = s % P.n_q;
        if (!(ok = mbar_wait(&S.q_full[qb], (s / P.n_q) & 1, err))) break;
        if (!(ok = scores())) break;
        if (nt == 1) mma_commit(&S.q_empty[qb]);
        for (uint32_t j = 0; j < nt; ++j) {
          if (j + 1 < nt) {
            if (!(ok = scores())) break;
            if (j + 2 == nt) mma_commit(&S.q_empty[qb]);
          }
          if (!(ok = mbar_wait(&S.full[ring.slot], ring.phase, err))) break;
          if (j == 0 && s && !(ok = mbar_wait(&S.o_free, (s - 1) & 1, err))) break;
          if (!(ok = mbar_wait(&S.p_full, pv & 1, err))) break;
          tc_fence_after();
          for (uint32_t m = 0; m < P.nmb; ++m) {
            // 128 dims: one column of 8-bit codes, two of bf16 (a lone one is read twice: the
            // second half of the lanes is not used)
            const uint32_t x0 = F8 ? m : 2 * m, va = slot0 + ring.slot * slot_bytes + x0 * kBox;
            const uint32_t lbo = !F8 && x0 + 1 < P.nbox ? kBox : 0u;
#pragma unroll
            for (uint32_t k = 0; k < (F8 ? 4u : 8u); ++k) {
              const uint64_t ad = sdesc_sw128_mn(va + k * (F8 ? 4096u : 2048u), lbo, 1024);
              const uint64_t bd = sdesc_plain_mn(p0 + k * (F8 ? 512u : 256u), 128, 2048);
              if (F8)
                mma_e4m3(t_o + m * 2 * RP, ad, bd, id_o, j | k);
              else
                mma_bf16(t_o + m * 2 * RP, ad, bd, id_o, j | k);
            }
          }
          mma_commit(&S.empty[ring.slot]);
          mma_commit(&S.pv_done);
          ring.next(P.n_slots);
          ++pv;
        }
      }
      if (!ok) {   // let the products in flight end (bounded)
        mma_commit(&S.drain);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(&S.drain, 0) && global_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- the segments: sequences 32 at a time, a lane each
    uint32_t b = S.start_b, base = 0xffffffffu, s = 0;
    uint64_t off = S.start_off, left = S.start_n;
    PagedItem mine = {};
    bool ok = true;
    while (left && b < a.batch) {
      if (base == 0xffffffffu || b - base >= 32) {
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
      const uint32_t tiles = tiles_of(it), groups = (it.cnt * P.G + RP - 1) / RP, items = a.n_kv * groups;
      if (tiles) {
        uint32_t i = (uint32_t)(off / tiles), t0 = (uint32_t)(off % tiles);
        for (; i < items && left; ++i, t0 = 0) {
          const uint32_t nt = (uint32_t)min((uint64_t)(tiles - t0), left);
          if (!(ok = mbar_wait_warp(&S.seg_empty[s % kSegs], ((s / kSegs) & 1) ^ 1, err))) break;
          if (lane == 0) {
            Segment &sg = S.seg[s % kSegs];
            sg.b = b;
            sg.kh = i / groups;
            sg.r0 = (i % groups) * RP;
            sg.nr = min((uint32_t)RP, it.cnt * P.G - sg.r0);
            sg.first = it.first;
            sg.pos0 = it.pos0;
            sg.tile0 = it.lo / kTile + t0;
            sg.nt = nt;
            sg.whole = (t0 == 0 ? 1u : 0u) | (t0 + nt == tiles ? 2u : 0u);
            mbar_arrive(&S.seg_full[s % kSegs]);
          }
          __syncwarp();
          left -= nt;
          ++s;
        }
        if (!ok) break;
      }
      off = 0;
      ++b;
    }
    if (ok && mbar_wait_warp(&S.seg_empty[s % kSegs], ((s / kSegs) & 1) ^ 1, err) && lane == 0) {
      S.seg[s % kSegs].nt = 0;
      mbar_arrive(&S.seg_full[s % kSegs]);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------- queries of a segment, as the second operand of the scores
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
    for (uint32_t s = 0;; ++s) {
      if (!mbar_wait_warp(&S.seg_full[s % kSegs], (s / kSegs) & 1, err)) break;
      const Segment sg = S.seg[s % kSegs];
      const uint32_t qb = s % P.n_q;
      if (sg.nt == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.seg_empty[s % kSegs]);
        break;
      }
      if (!mbar_wait_warp(&S.q_empty[qb], ((s / P.n_q) & 1) ^ 1, err)) break;
      uint8_t *dst = s_q + qb * q_bytes;
      // 8 elements of a row (zeros outside)
      auto load8 = [&](uint32_t r, uint32_t d) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < sg.nr && d < D) {
          const uint32_t row = sg.r0 + r;
          const __nv_bfloat16 *p = q + (sg.first + row / P.G) * a.q_stride + (size_t)(sg.kh * P.G + row % P.G) * D + d;
          if (P.q_vec) {
            v = __ldg(reinterpret_cast<const uint4 *>(p));
          } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = (uint32_t)__bfloat16_as_ushort(p[2 * i]) | (uint32_t)__bfloat16_as_ushort(p[2 * i + 1]) << 16;
            v = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        return v;
      };
      auto place = [&](uint32_t r, uint32_t c) {   // 16-byte piece c of row r
        return dst + (c / 8) * C::kQRows * 128u + r * 128u + (((c & 7) ^ (r & 7)) << 4);
      };
      if constexpr (!F8) {
        const uint32_t pieces = P.nbox * 8, n = C::kQRows * pieces;   // (a multiple of 128)
        for (uint32_t i0 = lane; i0 < n; i0 += 128) {
          uint4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = load8((i0 + 32 * u) / pieces, (i0 + 32 * u) % pieces * 8);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4 *>(place((i0 + 32 * u) / pieces, (i0 + 32 * u) % pieces)) = v[u];
        }
      } else {
        // half a warp per row, 16 elements a lane: q 2^k = hi + lo / 16, k so that the largest
        // entry is in [128, 256)
        const uint32_t c = lane & 15;
        const float ks = __ldg(a.k_scale + sg.kh) * P.c2;
#pragma unroll 4
        for (uint32_t r = lane >> 4; r < RP; r += 2) {
          uint32_t w[8];
          *reinterpret_cast<uint4 *>(w) = load8(r, 16 * c);
          *reinterpret_cast<uint4 *>(w + 4) = load8(r, 16 * c + 8);
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7fffu, w[i] >> 16 & 0x7fffu));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // (a row with a NaN or an infinity becomes NaN)
          const int e = max((int)(top >> 7) - 127, -119);
          const float up = top >= 0x7f80u ? NAN : __uint_as_float((uint32_t)(127 + 7 - e) << 23);
          const float down = __uint_as_float((uint32_t)(127 - 7 + min(e, 127)) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              x[2 * k] = __uint_as_float(w[2 * i + k] << 16) * up;
              x[2 * k + 1] = __uint_as_float(w[2 * i + k] & 0xffff0000u) * up;
            }
            const uint16_t h0 = pack_e4m3(x[0], x[1]), h1 = pack_e4m3(x[2], x[3]);
            const float2 f0 = unpack_e4m3(h0), f1 = unpack_e4m3(h1);
            const uint16_t l0 = pack_e4m3((x[0] - f0.x) * 16.f, (x[1] - f0.y) * 16.f);
            const uint16_t l1 = pack_e4m3((x[2] - f1.x) * 16.f, (x[3] - f1.y) * 16.f);
            hi[i] = h0 | (uint32_t)h1 << 16;
            lo[i] = l0 | (uint32_t)l1 << 16;
          }
          if (c < P.nbox * 8) {
            *reinterpret_cast<uint4 *>(place(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(place(RP + r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          if (c == 0) S.qs[s % kSegs][r] = down * ks;
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
    // ---------------- softmax and output: a thread per key, then per dim
    const uint32_t quarter = warp & 3, me = quarter * 32 + lane;
    const uint32_t t_lane = (quarter * 32) << 16, t_o = tmem + t_lane, t_s = tmem + o_cols + t_lane;
    uint32_t sc = 0, pv = 0, ph = 0, tick = 0, base = 0;   // base: loads of the segments before
    Part left[2] = {};
    bool ok = true;
    for (uint32_t s = 0; ok; ++s) {
      if (!mbar_wait_warp(&S.seg_full[s % kSegs], (s / kSegs) & 1, err)) break;
      const Segment sg = S.seg[s % kSegs];
      if (sg.nt == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.seg_empty[s % kSegs]);
        break;
      }
      const uint32_t p_first = sg.pos0 + sg.r0 / P.G, p_last = sg.pos0 + (sg.r0 + sg.nr - 1) / P.G;
      float l[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) l[r] = 0.f;
      BlockList bl;
      bl.start();
      for (uint32_t j = 0; j < sg.nt; ++j) {
        const uint32_t tile = sg.tile0 + j, key0 = tile * kTile, key = key0 + me, sb = sc & 1;
        const bool held = bl.at(a, sg.b, tile / 2, lane) < a.n_blocks;
        // ---- scores, in units of log2
        if (!(ok = mbar_wait_warp(&S.s_full[sb], (sc >> 1) & 1, err))) break;
        tc_fence_after();
        float x[RP];
        {
          uint32_t v[RP];
          if constexpr (RP == 64) {
            uint32_t(&v0)[32] = *reinterpret_cast<uint32_t(*)[32]>(v);
            uint32_t(&v1)[32] = *reinterpret_cast<uint32_t(*)[32]>(v + 32);
            tmem_ld(t_s + sb * C::kQRows, v0);
            tmem_ld(t_s + sb * C::kQRows + 32, v1);
          } else {
            tmem_ld(t_s + sb * C::kQRows, v);
          }
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < RP; ++r) x[r] = __uint_as_float(v[r]);
          if constexpr (F8) {
            if constexpr (RP == 64) {
              uint32_t(&v0)[32] = *reinterpret_cast<uint32_t(*)[32]>(v);
              uint32_t(&v1)[32] = *reinterpret_cast<uint32_t(*)[32]>(v + 32);
              tmem_ld(t_s + sb * C::kQRows + RP, v0);
              tmem_ld(t_s + sb * C::kQRows + RP + 32, v1);
            } else {
              tmem_ld(t_s + sb * C::kQRows + RP, v);
            }
            tmem_ld_wait();
            const float *qs = S.qs[s % kSegs];
#pragma unroll
            for (int r = 0; r < RP; ++r) x[r] = fmaf(__uint_as_float(v[r]), 0.0625f, x[r]) * qs[r];
          } else {
#pragma unroll
            for (int r = 0; r < RP; ++r) x[r] *= P.c2;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.s_empty[sb]);
        ++sc;
        // ---- unseen keys
        const bool plain = held && key0 + kTile - 1 <= p_first && (!a.window || p_last - key0 < a.window);
        bool all = true, any = true;
        if (!plain) {
          all = held && key <= p_first && (!a.window || p_last - key < a.window);
          any = held && key <= p_last && !(a.window && key < p_first && p_first - key >= a.window);
          uint32_t tok = sg.r0 / P.G, g = sg.r0 % P.G;
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const uint32_t p = sg.pos0 + tok;
            if (!held || key > p || (a.window && p - key >= a.window)) x[r] = -INFINITY;
            if (++g == P.G) {
              g = 0;
              ++tok;
            }
          }
        }
        // ---- the reference moves where a weight would be too large
        bool mine = j == 0;
        if (j) {
#pragma unroll
          for (int r = 0; r < RP; ++r) mine |= x[r] + S.negm[r] > C::kTop;
        }
        if (__any_sync(0xffffffffu, mine) && lane == 0) S.over[tick] = 1;
        if (!(ok = warps_sync(&S.group, ph, lane, err))) break;
        const bool over = *(volatile uint32_t *)&S.over[tick] != 0;
        // (the place of the tile after next: last read before this barrier, set behind the next one)
        tick = tick == 2 ? 0 : tick + 1;
        if (me == 0) S.over[tick == 2 ? 0 : tick + 1] = 0;
        if (j) {   // the products before read the sums' old scale and P
          if (!(ok = mbar_wait_warp(&S.pv_done, pv & 1, err))) break;
          ++pv;
        }
        if (over) {
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float m = warp_max_nan(x[r]);
            if (lane == (r & 31)) S.wmax[quarter][r] = m;
          }
          if (!(ok = warps_sync(&S.group, ph, lane, err))) break;
          if (me < RP) {
            float m = S.wmax[0][me];
#pragma unroll
            for (int w = 1; w < 4; ++w) {
              const float y = S.wmax[w][me];
              m = y > m || y != y ? y : m;
            }
            const float was = j ? S.negm[me] : kNoRef, now = m == -INFINITY ? was : fminf(was, C::kOff - m);
            const float now_ = m != m ? m : now;   // (fminf drops a NaN)
            S.fac[me] = ex2_approx(now_ - was);
            S.negm[me] = now_;
          }
          if (!(ok = warps_sync(&S.group, ph, lane, err))) break;
#pragma unroll
          for (int r = 0; r < RP; ++r) l[r] *= S.fac[r];
          if (j) {
            tc_fence_after();
            for (uint32_t c = 0; c < o_cols; c += 8) {
              uint32_t v[8];
              tmem_ld8(t_o + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * S.fac[(c + i) % RP]);
              tmem_st8(t_o + c, v);
            }
            tmem_st_wait();
          }
        }
        // ---- weights, in two parts each
        uint8_t *dst = s_p + (me / 8) * 128 + (me % 8) * 16;
        if constexpr (!F8) {
#pragma unroll
          for (int r0 = 0; r0 < RP; r0 += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = r0 + 2 * i;
              const float w0 = ex2_approx(x[r] + S.negm[r]), w1 = ex2_approx(x[r + 1] + S.negm[r + 1]);
              l[r] += w0;
              l[r + 1] += w1;
              hi[i] = pack_bf16(w0, w1);
              lo[i] = pack_bf16(w0 - __uint_as_float(hi[i] << 16), w1 - __uint_as_float(hi[i] & 0xffff0000u));
            }
            *reinterpret_cast<uint4 *>(dst + r0 / 8 * 2048) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(dst + (RP + r0) / 8 * 2048) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        } else {
          uint32_t hi[RP / 4], lo[RP / 4];
#pragma unroll
          for (int i = 0; i < RP / 4; ++i) {
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 4 * i + k;
              w[k] = ex2_approx(x[r] + S.negm[r]);
              l[r] += w[k];
            }
            const uint16_t h0 = pack_e4m3(w[0], w[1]), h1 = pack_e4m3(w[2], w[3]);
            const float2 f0 = unpack_e4m3(h0), f1 = unpack_e4m3(h1);
            hi[i] = h0 | (uint32_t)h1 << 16;
            lo[i] = pack_e4m3((w[0] - f0.x) * 16.f, (w[1] - f0.y) * 16.f) |
                    (uint32_t)pack_e4m3((w[2] - f1.x) * 16.f, (w[3] - f1.y) * 16.f) << 16;
          }
          if constexpr (RP == 8) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
          } else {
#pragma unroll
            for (int g = 0; g < RP / 16; ++g) {
              *reinterpret_cast<uint4 *>(dst + g * 2048) = make_uint4(hi[4 * g], hi[4 * g + 1], hi[4 * g + 2], hi[4 * g + 3]);
              *reinterpret_cast<uint4 *>(dst + (RP / 16 + g) * 2048) =
                  make_uint4(lo[4 * g], lo[4 * g + 1], lo[4 * g + 2], lo[4 * g + 3]);
            }
          }
        }
        if (!plain) {
          // (the values are there: a slot is refilled only behind the products that this arrival starts)
          const uint32_t k = base + place_v(j, sg.nt), slot = k % P.n_slots;
          if (!(ok = mbar_wait_warp(&S.full[slot], (k / P.n_slots) & 1, err))) break;
          if (!all && clean_row<F8>(smem_u32(s_slot + slot * slot_bytes) + me * 128, P.nbox, !any)) S.bad = 1;
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full);
      }
      if (!ok) break;
      base += 2 * sg.nt;
      // ---- the segment's end: sums over the keys, then the output, a thread per dim
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float sum = warp_sum(l[r]);
        if (lane == (r & 31)) S.wmax[quarter][r] = sum;
      }
      if (!(ok = mbar_wait_warp(&S.pv_done, pv & 1, err))) break;
      ++pv;
      tc_fence_after();
      if (!(ok = warps_sync(&S.group, ph, lane, err))) break;
      const bool whole = sg.whole == 3, bad = *(volatile uint32_t *)&S.bad != 0;
      const uint32_t side = sg.whole & 1;   // (a part: 0 began in an earlier block, 1 goes on in the next)
      float *sums = P.sums + ((size_t)blockIdx.x * 2 + side) * RP * D;
      if (me < sg.nr) {
        const float sum = S.wmax[0][me] + S.wmax[1][me] + S.wmax[2][me] + S.wmax[3][me];
        if (whole) {
          const uint32_t row = sg.r0 + me;
          if (a.lse)
            a.lse[(size_t)(sg.first + row / P.G) * a.n_heads + sg.kh * P.G + row % P.G] =
                sum == 0.f ? -INFINITY : (log2f(sum) - S.negm[me]) * 0.6931471805599453f;
        } else {
          float *ml = P.sums + (size_t)gridDim.x * 2 * RP * D + (((size_t)blockIdx.x * 2 + side) * RP + me) * 2;
          ml[0] = -S.negm[me];
          ml[1] = sum;
        }
        S.fac[me] = sum == 0.f ? 0.f : (F8 ? __ldg(a.v_scale + sg.kh) : 1.f) / sum;
      }
      if (!(ok = warps_sync(&S.group, ph, lane, err))) break;
      for (uint32_t m = 0; m < P.nmb; ++m) {
        const uint32_t d = m * 128 + me;
#pragma unroll
        for (int r0 = 0; r0 < RP; r0 += 8) {
          uint32_t h[8], w[8];
          tmem_ld8(t_o + m * 2 * RP + r0, h);
          tmem_ld8(t_o + m * 2 * RP + RP + r0, w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t r = r0 + i, row = sg.r0 + r;
            if (r >= sg.nr || d >= D) break;
            float o = F8 ? fmaf(__uint_as_float(w[i]), 0.0625f, __uint_as_float(h[i]))
                         : __uint_as_float(h[i]) + __uint_as_float(w[i]);
            if (bad) o += taken_out<F8>(a, sg, sg.pos0 + row / P.G, p_first, p_last, d);
            if (whole)
              static_cast<__nv_bfloat16 *>(a.out)[((size_t)(sg.first + row / P.G) * a.n_heads + sg.kh * P.G + row % P.G) * D + d] =
                  __float2bfloat16_rn(o * S.fac[r]);
            else
              sums[(size_t)r * D + d] = o;
          }
          __syncwarp();
        }
      }
      if (!whole) left[side] = Part{1u, sg.whole >> 1, sg.b, sg.kh, sg.r0, sg.nr, sg.first, 0u};
      tc_fence_before();
      if (!(ok = warps_sync(&S.group, ph, lane, err))) break;   // (the shared sums are free)
      if (me == 0) S.bad = 0;
      if (lane == 0) {
        mbar_arrive(&S.o_free);
        mbar_arrive(&S.seg_empty[s % kSegs]);
      }
    }
    if (me == 0) {
      P.parts[blockIdx.x * 2] = left[0];
      P.parts[blockIdx.x * 2 + 1] = left[1];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, alloc);
  }
}

// Joins the parts of what begins in block blockIdx.x and goes on: rows blockIdx.y, + gridDim.y, ..
// each as the sum of its parts brought to the largest reference, in the order of the blocks.
template <int RP, bool F8>
__global__ void __launch_bounds__(256) paged_join_tc_kernel(Params P, uint32_t blocks) {
  pdl_wait();
  pdl_trigger();
  const PagedArgs &a = P.a;
  const uint32_t c0 = blockIdx.x, D = a.head_dim;
  const Part part = P.parts[2 * c0 + 1];
  if (!part.valid) return;
  uint32_t n = 1;
  for (; c0 + n < blocks; ++n)
    if (P.parts[2 * (c0 + n)].last) break;
  if (c0 + n >= blocks) return;
  const float *ml = P.sums + (size_t)blocks * 2 * RP * D;
  // piece i: block c0 + i, its second half (i = 0) or its first
  auto at = [&](uint32_t i, uint32_t r) { return ((size_t)(c0 + i) * 2 + (i ? 0u : 1u)) * RP + r; };
  for (uint32_t r = blockIdx.y; r < part.nr; r += gridDim.y) {
    float m = -kNoRef;
    bool nan = false;
    for (uint32_t i = threadIdx.x & 31; i <= n; i += 32) {
      const float x = ml[at(i, r) * 2];
      nan |= x != x;
      m = fmaxf(m, x);
    }
    m = __any_sync(0xffffffffu, nan) ? NAN : warp_max(m);
    float l = 0.f, o = 0.f;
    const uint32_t d = threadIdx.x;
    for (uint32_t i = 0; i <= n; ++i) {
      const size_t k = at(i, r);
      const float w = ml[2 * k] <= -kNoRef ? 0.f : ex2_approx(ml[2 * k] - m);
      l = fmaf(ml[2 * k + 1], w, l);
      if (d < D && (w != 0.f)) o = fmaf(P.sums[k * D + d], w, o);
    }
    const uint32_t row = part.r0 + r;
    const size_t out = (size_t)(part.first + row / P.G) * a.n_heads + part.kh * P.G + row % P.G;
    const float scale = l == 0.f ? 0.f : (F8 ? __ldg(a.v_scale + part.kh) : 1.f) / l;
    if (d < D) static_cast<__nv_bfloat16 *>(a.out)[out * D + d] = __float2bfloat16_rn(o * scale);
    if (a.lse && d == 0) a.lse[out] = l == 0.f ? -INFINITY : (log2f(l) + m) * 0.6931471805599453f;
  }
}

// Rows of a group: the fewest that hold a sequence's, up to 64.
uint32_t rows_of(const PagedArgs &a) {
  const uint32_t r = a.max_new * (a.n_heads / a.n_kv);
  return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : 64;
}

// Blocks: one a SM, or one a tile where there can be no more tiles.
uint32_t blocks_of(const PagedArgs &a) {
  const uint32_t rp = rows_of(a), groups = (a.max_new * (a.n_heads / a.n_kv) + rp - 1) / rp;
  uint64_t tiles = 2ull * a.max_blocks;
  if (a.window) {
    const uint64_t w = ((uint64_t)a.window + a.max_new) / kTile + 2;
    tiles = w < tiles ? w : tiles;
  }
  const uint64_t most = tiles * a.batch * a.n_kv * groups, sms = (uint64_t)num_sms();
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
  const uint32_t blocks = blocks_of(a), slot = P.nbox * kBox, q = C::kQRows * P.nbox * 128u;
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  P.err = reinterpret_cast<int *>(ws);
  P.parts = reinterpret_cast<Part *>(ws + 256);
  P.sums = reinterpret_cast<float *>(ws + 256 + (size_t)num_sms() * 2 * sizeof(Part));
  const uint32_t room = kSmemMost - kFixed - C::kPBytes;
  P.n_q = (room - 2 * q) / slot >= 3 ? 2 : 1;
  P.n_slots = (room - P.n_q * q) / slot;
  if (P.n_slots > kMaxSlots) P.n_slots = kMaxSlots;
  const size_t smem = 1024 + (size_t)P.n_slots * slot + P.n_q * q + C::kPBytes + sizeof(Shared);
  static RaisedLimit smem_set;
  auto *k = paged_attn_tc_kernel<RP, F8>;
  e = ensure_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(blocks), dim3(kThreads), smem, s, mk, mv, P);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (blocks > 1) {   // (a lone block holds every segment whole)
    e = launch_pdl(paged_join_tc_kernel<RP, F8>, dim3(blocks, 8), dim3(256), 0, s, P, blocks);
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
  return (size_t)num_sms() * 2 * (sizeof(Part) + (size_t)rows_of(a) * (a.head_dim + 2) * 4);
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
