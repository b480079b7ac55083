// Block tables, ragged positions and slot maps of a step from the requests'
// lengths (ds4a_block_tables), in one launch and without the host: a captured
// step replays with the lengths it finds.
//
// Every row b needs need_b = ceil(ctx_b / 256) blocks and holds held_b. Exclusive
// sums over the rows of the blocks to take, the blocks to give back and the new
// tokens place every row's share of the free list and of the packed tokens, so the
// result does not depend on the order in which anything runs. Each thread block
// computes the sums of all rows for itself (the lengths of a few thousand rows
// are a few KiB from L2; a second launch, or a wait between blocks, costs more)
// and then writes its share of the rows and tokens. The state that all of them
// read (held, the free list's head and count) is advanced by the block that
// arrives last at a ticket, after every block has taken its copy; none waits.
// Bound by the launch and a chain of latencies (8 decoding rows: 3.3 us), then by what
// each block does for all rows (2,048 rows with 239,593 tokens: 7.3 us, 11.8 where 47,533
// blocks change hands); by the stores of five words per token beyond some 10^6 tokens.
#include "common.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kBlockTokens = 256;   // token positions of a logical block

// Per row, six arrays in shared memory. A thread's consecutive rows (2^shift of them)
// are followed by one unused place, which keeps the threads' accesses to their j-th
// rows on different banks.
struct RowState {
  uint32_t *first;  // packed index of its first new token
  uint32_t *ctx;    // tokens it is to hold
  uint32_t *held;   // blocks it held before the call
  uint32_t *goff;   // blocks taken by the rows before it
  uint32_t *roff;   // blocks given back by the rows before it
  uint32_t *nw;     // its new tokens
};
constexpr uint32_t kRowWords = 6;

__device__ __forceinline__ uint32_t blocks_of(uint32_t ctx) {
  return ctx / kBlockTokens + (ctx % kBlockTokens ? 1u : 0u);
}

// Exclusive sums over the block of four values per thread; totals in tot.
template <uint32_t NT>
__device__ __forceinline__ void block_scan4(uint32_t (&v)[4], uint32_t (&tot)[4],
                                            uint32_t (*part)[4]) {
  constexpr uint32_t NW = NT / 32;
  const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t inc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) inc[k] = v[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= (uint32_t)o) inc[k] += x;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[w][k] = inc[k];
  __syncthreads();
  if (w < 4) {   // warp k sums the warps' totals of value k
    uint32_t x = lane < NW ? part[lane][w] : 0u;
#pragma unroll
    for (int o = 1; o < (int)NW; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= (uint32_t)o) x += y;
    }
    if (lane < NW) part[lane][w] = x;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = (w ? part[w - 1][k] : 0u) + inc[k] - v[k];
    tot[k] = part[NW - 1][k];
  }
}

// Row of token tok, the last of the B rows whose first token is at or before it (rows
// without new tokens share their first index with the row after them). WIDE: the warp looks
// up its 32 tokens' first and last row together, 32 rows at a time (step: the
// largest power of 32 below B), and the lanes search between the two, which are
// mostly one row; else each lane by halves (step: the largest power of two below B).
// (Whatever first[] holds, the result is below B.)
template <bool WIDE, typename First>
__device__ __forceinline__ uint32_t row_of_token(uint32_t tok, uint32_t B, uint32_t step,
                                                 First first) {
  uint32_t r0 = 0;
  if (!WIDE) {
    for (uint32_t w = step; w; w >>= 1)
      if (r0 + w < B && first(r0 + w) <= tok) r0 += w;
    return r0;
  }
  const uint32_t lane = threadIdx.x & 31, tok0 = tok - lane;
  uint32_t r1 = 0;
  for (uint32_t st = step; st; st >>= 5) {
    const uint32_t i0 = r0 + st * lane, i1 = r1 + st * lane;
    const bool b0 = i0 < B && first(i0) <= tok0, b1 = i1 < B && first(i1) <= tok0 + 31;
    const int n0 = __popc(__ballot_sync(0xffffffffu, b0)), n1 = __popc(__ballot_sync(0xffffffffu, b1));
    r0 += st * (max(n0, 1) - 1);
    r1 += st * (max(n1, 1) - 1);
  }
  for (uint32_t w = r1 > r0 ? 1u << (31 - __clz(r1 - r0)) : 0u; w; w >>= 1)
    if (r0 + w <= r1 && first(r0 + w) <= tok) r0 += w;
  return r0;
}

template <uint32_t NT, uint32_t TPT>
__global__ void __launch_bounds__(NT) block_tables_kernel(TablesArgs a) {
  constexpr uint32_t kThreads = NT, kWarps = NT / 32, kTokPerThread = TPT;
  extern __shared__ uint32_t words[];
  __shared__ uint32_t part[kWarps][4], last;
  pdl_wait();
  const uint32_t B = a.rows, n = a.n_blocks, t = threadIdx.x;
  const uint32_t head0 = a.state[0], count0 = a.state[1];
  const uint32_t len = B + (B >> a.shift) + 1;
  const RowState R{words, words + len, words + 2 * len, words + 3 * len, words + 4 * len,
                   words + 5 * len};
  auto at = [&](uint32_t b) { return b + (b >> a.shift); };
  // ---- every row's lengths into shared memory, then the sums, each thread over
  // consecutive rows
#pragma unroll 4
  for (uint32_t b = t; b < B; b += kThreads) {
    const uint32_t ctx = a.ctx_len[b], nw = a.new_len[b], held = a.held[b];
    R.ctx[at(b)] = ctx;
    R.nw[at(b)] = min(nw, ctx);
    R.held[at(b)] = min(held, a.max_blocks);
  }
  __syncthreads();
  const uint32_t b0 = min(B, t << a.shift), b1 = min(B, (t + 1) << a.shift);
  uint32_t v[4] = {0, 0, 0, 0}, tot[4];
  for (uint32_t b = b0; b < b1; ++b) {
    const uint32_t want = blocks_of(R.ctx[at(b)]), need = min(want, a.max_blocks);
    const uint32_t held = R.held[at(b)];
    v[0] += R.nw[at(b)];
    v[1] += need > held ? need - held : 0u;
    v[2] += held > need ? held - need : 0u;
    v[3] += want - need;
  }
  block_scan4<NT>(v, tot, part);
  for (uint32_t b = b0; b < b1; ++b) {
    const uint32_t need = min(blocks_of(R.ctx[at(b)]), a.max_blocks), held = R.held[at(b)];
    R.first[at(b)] = v[0];
    R.goff[at(b)] = v[1];
    R.roff[at(b)] = v[2];
    v[0] += R.nw[at(b)];
    v[1] += need > held ? need - held : 0u;
    v[2] += held > need ? held - need : 0u;
  }
  const uint32_t head = head0 % n, count = min(count0, n);
  const uint32_t total = tot[0], grow = tot[1], back = tot[2];
  __syncthreads();   // the rows are complete
  // The state's advance: by the block that draws the last ticket, when every block has
  // its copy. The ticket is drawn here and looked at when everything else is done, so
  // that nothing waits for it; a block that is alone needs none.
  auto advance = [&]() {
    for (uint32_t b = t; b < B; b += kThreads) {
      const uint32_t need = min(blocks_of(R.ctx[at(b)]), a.max_blocks), held = R.held[at(b)];
      const uint32_t g = need > held ? need - held : 0u;
      const uint32_t left = count > R.goff[at(b)] ? count - R.goff[at(b)] : 0u;
      a.held[b] = held > need ? need : held + min(g, left);
    }
    if (t == 0) {
      const uint32_t taken = min(count, grow);
      a.state[0] = (head + taken) % n;
      a.state[1] = count - taken + min(back, n - count);
      a.state[2] = grow - taken + tot[3];
      a.state[3] = 0;
    }
  };
  uint32_t ticket = 0;
  if (t == 0 && gridDim.x > 1) {
    __threadfence();
    ticket = atomicAdd(a.state + 3, 1u);
  }
  if (gridDim.x == 1) advance();
  // place `k` (< n) of the ring from its head (n <= 2^25)
  auto ring = [&](uint32_t k) { return head + k < n ? head + k : head + k - n; };
  // ---- rows: a warp per row
  const uint32_t lane = t & 31;
  for (uint32_t b = blockIdx.x * kWarps + (t >> 5); b < B; b += gridDim.x * kWarps) {
    const uint32_t ctx = R.ctx[at(b)], nw = R.nw[at(b)], held = R.held[at(b)];
    const uint32_t goff = R.goff[at(b)], roff = R.roff[at(b)];
    const uint32_t need = min(blocks_of(ctx), a.max_blocks);
    int32_t *row = a.table + (size_t)b * a.max_blocks;
    const uint32_t left = count > goff ? count - goff : 0u;
    for (uint32_t j = held + lane; j < need; j += 32) {
      const uint32_t i = j - held;
      row[j] = i < left ? a.free_list[ring(goff + i)] : -1;
    }
    for (uint32_t j = need + lane; j < held; j += 32) {
      const uint64_t place = (uint64_t)count + roff + (j - need);
      if (place < n) a.free_list[ring((uint32_t)place)] = row[j];
      row[j] = -1;
    }
    if (lane == 0) {
      if (a.seq_pos) a.seq_pos[b] = ctx - nw;
      if (a.cu_len) a.cu_len[b] = R.first[at(b)];
    }
  }
  if (blockIdx.x == 0 && t == 0 && a.cu_len) a.cu_len[B] = total;
  // ---- tokens: kTokPerThread per thread and round, a block apart
  const bool maps = a.tok_seq || a.tok_pos || a.raw_slot || a.slot4 || a.slot128;
  const uint64_t step = (uint64_t)gridDim.x * kThreads * kTokPerThread;
  for (uint64_t base = (uint64_t)blockIdx.x * kThreads * kTokPerThread + t;
       maps && base - lane < a.max_tokens; base += step) {   // (whole warps)
    uint32_t lo[kTokPerThread];
#pragma unroll
    for (uint32_t e = 0; e < kTokPerThread; ++e)
      lo[e] = row_of_token<(NT > 256)>((uint32_t)base + kThreads * e, B, a.search,
                                       [&](uint32_t b) { return R.first[at(b)]; });
    int32_t blk[kTokPerThread];
    uint32_t pos[kTokPerThread];
#pragma unroll
    for (uint32_t e = 0; e < kTokPerThread; ++e) {
      const uint64_t i = base + kThreads * e;
      blk[e] = -1;
      pos[e] = 0;
      if (i < total && i < a.max_tokens) {
        const uint32_t k = at(lo[e]), held = R.held[k];
        const uint32_t p = R.ctx[k] - R.nw[k] + ((uint32_t)i - R.first[k]), j = p / kBlockTokens;
        pos[e] = p;
        if ((p & 3) == 3 && j < a.max_blocks) {
          if (j < held) {
            blk[e] = a.table[(size_t)lo[e] * a.max_blocks + j];
          } else {
            const uint32_t left = count > R.goff[k] ? count - R.goff[k] : 0u;
            if (j - held < left) blk[e] = a.free_list[ring(R.goff[k] + (j - held))];
          }
        }
      }
    }
#pragma unroll
    for (uint32_t e = 0; e < kTokPerThread; ++e) {
      const uint64_t i = base + kThreads * e;
      if (i >= a.max_tokens) break;
      const bool live = i < total;
      const uint32_t p = pos[e], b = lo[e];
      const bool ok = blk[e] >= 0 && (uint32_t)blk[e] < n;
      if (a.tok_seq) a.tok_seq[i] = live ? (int32_t)b : -1;
      if (a.tok_pos) a.tok_pos[i] = live ? (int32_t)p : -1;
      // (slot p % cap_raw ends up with the sequence's last token there)
      if (a.raw_slot)
        a.raw_slot[i] = live && R.ctx[at(b)] - p <= a.cap_raw
                            ? (int32_t)(b * a.cap_raw + p % a.cap_raw) : -1;
      if (a.slot4) a.slot4[i] = ok ? blk[e] * 64 + (int32_t)(p % kBlockTokens / 4) : -1;
      if (a.slot128)
        a.slot128[i] = ok && (p & 127) == 127 ? blk[e] * 2 + (int32_t)(p % kBlockTokens / 128) : -1;
    }
  }
  if (gridDim.x > 1) {
    if (t == 0) last = ticket == gridDim.x - 1;
    __syncthreads();
    if (last) {
      __threadfence();
      advance();
    }
  }
}

}  // namespace

namespace {

template <uint32_t NT, uint32_t TPT>
cudaError_t launch_nt(TablesArgs a, cudaStream_t s) {
  a.search = 1;   // (see row_of_token)
  if (NT > 256) {
    while (32ull * a.search < a.rows) a.search *= 32;
  } else {
    while (2 * a.search < a.rows) a.search *= 2;
  }
  // a warp per row and a thread per TPT tokens, whichever asks for more blocks, while
  // the GPU has room for them (2,048 decoding rows: 7.2 us, in blocks of a row per
  // thread 13.6)
  const uint64_t by_tok = ((uint64_t)a.max_tokens + NT * TPT - 1) / (NT * TPT);
  const uint64_t by_row = (a.rows + NT / 32 - 1) / (NT / 32);
  uint64_t g = by_tok > by_row ? by_tok : by_row;
  if (g > (uint64_t)num_sms()) g = num_sms();
  if (NT <= 256) g = 1;   // (the call is small)
  a.shift = 0;   // rows per thread: 2^shift
  while (((uint64_t)NT << a.shift) < a.rows) ++a.shift;
  const size_t smem = (size_t)(a.rows + (a.rows >> a.shift) + 1) * kRowWords * sizeof(uint32_t);
  static RaisedLimit smem_set;
  auto *k = block_tables_kernel<NT, TPT>;
  // (the limit without the attribute counts the static arrays too)
  cudaError_t e = ensure_smem(k, smem + 1024, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3((uint32_t)g), dim3(NT), smem, s, a);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_tables(TablesArgs a, cudaStream_t s) {
  // Few rows and tokens: one small block, which needs no ticket (side by side, some
  // 0.4 us above today's figures: 8 decoding rows 3.3 us against 3.7 in large ones, 24 rows
  // 4.5 in three small ones against 4.3). Otherwise up to one block of 1,024 threads per
  // SM, which shares the sums over all rows among more threads (200 rows with 27,145
  // tokens: 5.6 us, in blocks of 256 threads 6.2; 2,048 rows with 239,593: 7.7 against 9.9;
  // 8,192 decoding: 9.0 against 18.8).
  return a.rows <= 16 && a.max_tokens <= 512 ? launch_nt<256, 2>(a, s) : launch_nt<1024, 1>(a, s);
}

}  // namespace ds4a
