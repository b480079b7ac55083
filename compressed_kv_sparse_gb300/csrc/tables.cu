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
// Bound by the launch and the latency of the sums; by the stores of five words per
// token beyond some 10^5 tokens.
#include "common.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWarps = kThreads / 32;
constexpr uint32_t kBlockTokens = 256;   // token positions of a logical block
constexpr uint32_t kTokPerThread = 4;

struct RowState {   // per row, in shared memory
  uint32_t first;   // packed index of its first new token
  uint32_t goff;    // blocks taken by the rows before it
  uint32_t roff;    // blocks given back by the rows before it
  uint32_t held;    // blocks it held before the call
};

__device__ __forceinline__ uint32_t blocks_of(uint32_t ctx) {
  return ctx / kBlockTokens + (ctx % kBlockTokens ? 1u : 0u);
}

// Exclusive sum over the block of three values per thread; totals in tot[3].
__device__ __forceinline__ void block_scan3(uint32_t (&v)[3], uint32_t (&tot)[3],
                                            uint32_t (*part)[3]) {
  const uint32_t lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t inc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    inc[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= (uint32_t)o) inc[k] += x;
    }
    if (lane == 31) part[w][k] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t before = 0, all = 0;
#pragma unroll
    for (uint32_t i = 0; i < kWarps; ++i) {
      if (i < w) before += part[i][k];
      all += part[i][k];
    }
    v[k] = before + inc[k] - v[k];
    tot[k] = all;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(TablesArgs a) {
  extern __shared__ RowState rows[];   // [B], then one word
  __shared__ uint32_t part[kWarps][3], last;
  pdl_wait();
  const uint32_t B = a.rows, n = a.n_blocks, t = threadIdx.x;
  const uint32_t head = a.state[0] % n, count = min(a.state[1], n);
  // ---- the sums, each thread over consecutive rows
  const uint32_t per = (B + kThreads - 1) / kThreads, b0 = min(B, t * per), b1 = min(B, b0 + per);
  uint32_t v[3] = {0, 0, 0}, tot[3], over = 0;
  for (uint32_t b = b0; b < b1; ++b) {
    const uint32_t ctx = a.ctx_len[b], nw = min(a.new_len[b], ctx);
    const uint32_t want = blocks_of(ctx), need = min(want, a.max_blocks);
    const uint32_t held = min(a.held[b], a.max_blocks);
    rows[b].held = held;
    v[0] += nw;
    v[1] += need > held ? need - held : 0u;
    v[2] += held > need ? held - need : 0u;
    over += want - need;
  }
  block_scan3(v, tot, part);
  for (uint32_t b = b0; b < b1; ++b) {
    const uint32_t ctx = a.ctx_len[b], nw = min(a.new_len[b], ctx);
    const uint32_t need = min(blocks_of(ctx), a.max_blocks), held = rows[b].held;
    rows[b].first = v[0];
    rows[b].goff = v[1];
    rows[b].roff = v[2];
    v[0] += nw;
    v[1] += need > held ? need - held : 0u;
    v[2] += held > need ? held - need : 0u;
  }
  uint32_t ov[3] = {over, 0, 0}, otot[3];
  block_scan3(ov, otot, part);   // (its barriers also publish rows[])
  const uint32_t total = tot[0], grow = tot[1], back = tot[2];
  // ---- the last block to get here advances the state: every block has its copy
  if (t == 0) {
    __threadfence();
    last = gridDim.x == 1 || atomicAdd(a.state + 3, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last) {
    __threadfence();
    for (uint32_t b = t; b < B; b += kThreads) {
      const uint32_t need = min(blocks_of(a.ctx_len[b]), a.max_blocks), held = rows[b].held;
      const uint32_t g = need > held ? need - held : 0u;
      const uint32_t left = count > rows[b].goff ? count - rows[b].goff : 0u;
      a.held[b] = held > need ? need : held + min(g, left);
    }
    if (t == 0) {
      const uint32_t taken = min(count, grow);
      a.state[0] = (head + taken) % n;
      a.state[1] = count - taken + min(back, n - count);
      a.state[2] = grow - taken + otot[0];
      a.state[3] = 0;
    }
  }
  // ---- rows: a warp per row
  const uint32_t lane = t & 31;
  for (uint32_t b = blockIdx.x * kWarps + (t >> 5); b < B; b += gridDim.x * kWarps) {
    const uint32_t ctx = a.ctx_len[b], nw = min(a.new_len[b], ctx);
    const uint32_t need = min(blocks_of(ctx), a.max_blocks);
    const RowState r = rows[b];
    int32_t *row = a.table + (size_t)b * a.max_blocks;
    const uint32_t left = count > r.goff ? count - r.goff : 0u;
    for (uint32_t j = r.held + lane; j < need; j += 32) {
      const uint32_t i = j - r.held;
      row[j] = i < left ? a.free_list[(uint32_t)(((uint64_t)head + r.goff + i) % n)] : -1;
    }
    for (uint32_t j = need + lane; j < r.held; j += 32) {
      const uint64_t place = (uint64_t)count + r.roff + (j - need);
      if (place < n) a.free_list[(uint32_t)((head + place) % n)] = row[j];
      row[j] = -1;
    }
    if (lane == 0) {
      if (a.seq_pos) a.seq_pos[b] = ctx - nw;
      if (a.cu_len) a.cu_len[b] = r.first;
    }
  }
  if (blockIdx.x == 0 && t == 0 && a.cu_len) a.cu_len[B] = total;
  // ---- tokens: four consecutive ones per thread
  const bool maps = a.tok_seq || a.tok_pos || a.raw_slot || a.slot4 || a.slot128;
  const uint32_t step = gridDim.x * kThreads * kTokPerThread;
  for (uint64_t i0 = (uint64_t)(blockIdx.x * kThreads + t) * kTokPerThread;
       maps && i0 < a.max_tokens; i0 += step) {
    // the row of token i0: the last one whose first token is at or before it
    // (rows without new tokens share their first index with the row after them)
    uint32_t lo = 0, hi = B;
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (rows[mid].first <= i0) lo = mid;
      else hi = mid;
    }
    uint32_t b = lo;
#pragma unroll
    for (uint32_t e = 0; e < kTokPerThread; ++e) {
      const uint64_t i = i0 + e;
      if (i >= a.max_tokens) break;
      int32_t seq = -1, pos = -1, raw = -1, s4 = -1, s128 = -1;
      if (i < total) {
        while (b + 1 < B && rows[b + 1].first <= i) ++b;
        const RowState r = rows[b];
        const uint32_t ctx = a.ctx_len[b], nw = min(a.new_len[b], ctx);
        const uint32_t p = ctx - nw + ((uint32_t)i - r.first);
        seq = (int32_t)b;
        pos = (int32_t)p;
        // (slot p % cap_raw ends up with the sequence's last token there)
        if (ctx - p <= a.cap_raw) raw = (int32_t)(b * a.cap_raw + p % a.cap_raw);
        const uint32_t j = p / kBlockTokens;
        if ((p & 3) == 3 && j < a.max_blocks) {
          int32_t blk;
          if (j < r.held) {
            blk = a.table[(size_t)b * a.max_blocks + j];
          } else {
            const uint32_t left = count > r.goff ? count - r.goff : 0u;
            blk = j - r.held < left
                      ? a.free_list[(uint32_t)(((uint64_t)head + r.goff + (j - r.held)) % n)]
                      : -1;
          }
          if (blk >= 0 && (uint32_t)blk < n) {
            s4 = blk * 64 + (int32_t)(p % kBlockTokens / 4);
            if ((p & 127) == 127) s128 = blk * 2 + (int32_t)(p % kBlockTokens / 128);
          }
        }
      }
      if (a.tok_seq) a.tok_seq[i] = seq;
      if (a.tok_pos) a.tok_pos[i] = pos;
      if (a.raw_slot) a.raw_slot[i] = raw;
      if (a.slot4) a.slot4[i] = s4;
      if (a.slot128) a.slot128[i] = s128;
    }
  }
  // (as at the end of norm_rope_kernel: a following launch may read positions
  // before its own wait, so the stores are done before this thread ends)
  __threadfence();
}

}  // namespace

cudaError_t launch_block_tables(const TablesArgs &a, cudaStream_t s) {
  // one block per 1024 tokens or 256 rows, whichever asks for more
  const uint64_t by_tok = ((uint64_t)a.max_tokens + kThreads * kTokPerThread - 1) /
                          (kThreads * kTokPerThread);
  const uint64_t by_row = (a.rows + 255) / 256;
  uint64_t g = by_tok > by_row ? by_tok : by_row;
  const uint64_t most = (uint64_t)num_sms();
  if (g > most) g = most;
  if (g < 1) g = 1;
  const size_t smem = (size_t)a.rows * sizeof(RowState);
  static DeviceSmem smem_set;
  cudaError_t e = ensure_smem(block_tables_kernel, smem, smem_set.here());
  if (e != cudaSuccess) return e;
  e = launch_pdl(block_tables_kernel, dim3((uint32_t)g), dim3(kThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace ds4a
