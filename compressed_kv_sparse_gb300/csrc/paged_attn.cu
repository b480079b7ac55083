// Attention of a step's new tokens over a paged cache of keys and values, on the CUDA cores: the
// exact path of fp32 layers and the one for sizes that the tensor-core kernel does not take.
//
// Rows (a sequence's tokens x the query heads of one key head) in groups of 8 or 16, keys in tiles of
// 32 or 64, the next tile on its way while one is worked on. A block scores a tile (a thread per
// key and part of the dims, all rows), updates each row's running maximum and sum (a warp
// per row) and adds the weighted values (a warp per eighth of the keys, a lane per four dims, all
// rows), so that a key or value is read from shared memory once for all rows. A sequence's
// tiles are shared among several blocks where there are few rows; each leaves its sums
// with their maximum, and a second launch joins them in order.
// Up to 8 rows half bound by HBM (8 sequences of 8,000 fp32 tokens, 8 heads of 128 dims, one row each 147 us, 3.6
// TB/s; 8 rows 156), beyond by the fp32 units and shared memory (128 rows 1,501 us, 22 TFLOP/s); short calls by two
// launches and a tile's steps (3 of a 1,024-token window 11.9 us). Other types than fp32 come one element a load (8 x 8,000
// tokens, 64 heads over 8 of 100 dims: bf16 454 us, 8 bits 326).
#include <cuda_fp8.h>

#include "paged.cuh"
#include "tc.cuh"

namespace ds4a {

namespace {

constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;
// Keys of a tile: 32 for 8 rows (8 x 8,000 tokens of 8 heads of 128 dims: 156 us, 64 keys 159; of 256 dims, where an SM
// holds one block of 64, 287 and 358); 64 for 16 rows (3 x 1,024 tokens, 10 rows of 80 dims: 11.8 us, 32 keys 15.4).
__host__ __device__ constexpr uint32_t tile_of(uint32_t R) { return R == 8 ? 32 : 64; }
// Blocks that an SM's registers have to have room for (16 rows of 256 dims take 249 a thread). Left to itself the
// compiler takes 137 for 8 rows, and one block a SM needs 222 us for what two do in 156. With 8 rows of more than 128
// dims two blocks cost 70 to 100 bytes of spills a thread, and are faster all the same (8 x 8,000 tokens of 256 dims 287 us,
// one block without spills 327; bf16 of 250 dims 745 and 1,027).
__host__ __device__ constexpr uint32_t blocks_per_sm(int R, int DV) { return R == 16 && DV == 2 ? 1 : 2; }
constexpr uint32_t kWsHead = 256;   // the status word's line
constexpr uint32_t kSmemMost = 227 * 1024, kSmemSm = 228 * 1024, kSmemBlock = 1024;

struct Params {
  PagedArgs a;
  uint32_t G, groups, splits;   // query heads per key head, row groups, shares of the keys
  uint32_t stages;              // key and value tiles in shared memory
  float *part;                  // [batch * max_new * H][splits][D], then (max, sum) of each
};

// The weight of a key that a row does not see, or of a share without any that it sees: a zero, told apart from one of
// a seen key that is too small for fp32.
constexpr float kUnseen = -0.f;
__device__ __forceinline__ bool is_unseen(float w) { return __float_as_uint(w) == 0x80000000u; }

template <typename T>
__device__ __forceinline__ float ld_kv(const T *p, size_t i) {
  return ld_f32(p, i);
}
__device__ __forceinline__ float ld_kv(const __nv_fp8_storage_t *p, size_t i) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3)));
}

// Floats of shared memory: queries, key tiles, value tiles, partial scores, weights, max, sum, factor.
__host__ __device__ constexpr uint32_t smem_floats(uint32_t D4, uint32_t R, uint32_t stages) {
  const uint32_t kTile = tile_of(R), kParts = kThreads / kTile;
  return R * 4 * D4 + stages * kTile * (4 * D4 + 4) + stages * kTile * 4 * D4 + kParts * R * kTile + kTile * (R + 4) + 3 * R;
}

// R: rows of a group. DV: fours of dims per lane (D <= 128 DV).
template <typename T, typename KV, int R, int DV>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(R, DV)) paged_attn_kernel(Params P) {
  constexpr uint32_t kTile = tile_of(R), kParts = kThreads / kTile;
  extern __shared__ __align__(16) float sm[];
  const PagedArgs &a = P.a;
  const uint32_t D = a.head_dim, D4 = (D + 3) / 4, VS = 4 * D4, KS = VS + 4, PS = R + 4, H = a.n_heads, K = a.n_kv;
  float *s_q = sm;                                      // [R][VS]
  float *s_k = s_q + R * VS;                            // [stage][kTile][KS]
  float *s_v = s_k + P.stages * kTile * KS;             // [stage][kTile][VS]
  float *s_s = s_v + P.stages * kTile * VS;             // [part][R][kTile]
  float *s_p = s_s + kParts * R * kTile;                     // [kTile][PS]
  float *s_m = s_p + kTile * PS, *s_l = s_m + R, *s_c = s_l + R;
  pdl_wait();
  pdl_trigger();
  const uint32_t split = blockIdx.x, kh = blockIdx.y / P.groups, rg = blockIdx.y % P.groups, b = blockIdx.z;
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const PagedItem it = paged_item(a, b);
  const uint32_t r0 = rg * R, all = it.cnt * P.G;
  if (r0 >= all) return;
  const uint32_t nr = min((uint32_t)R, all - r0);
  auto token = [&](uint32_t r) { return (r0 + r) / P.G; };
  auto head = [&](uint32_t r) { return kh * P.G + (r0 + r) % P.G; };
  // the keys that some row of the group sees, and those that all of them do
  const uint32_t p_first = it.pos0 + token(0), p_last = it.pos0 + token(nr - 1);
  const uint32_t k_lo = a.window && p_first + 1 > a.window ? p_first + 1 - a.window : 0u, k_hi = min(p_last + 1, it.hi);
  const uint32_t t_lo = it.lo / kTile, t_hi = (it.hi + kTile - 1) / kTile, nt = t_hi > t_lo ? t_hi - t_lo : 0u;
  const uint32_t t0 = t_lo + (uint32_t)((uint64_t)nt * split / P.splits);
  const uint32_t t1 = t_lo + (uint32_t)((uint64_t)nt * (split + 1) / P.splits);
  const float ks = a.k_scale ? __ldg(a.k_scale + kh) : 1.f, vs = a.v_scale ? __ldg(a.v_scale + kh) : 1.f;
  const bool async = sizeof(KV) == 4 && D % 4 == 0;   // (rows start on 16 bytes)
  // a tile's keys and values; rows that the group does not see are zeros (they may hold NaNs)
  auto load = [&](uint32_t stage, uint32_t tile) {
    const uint32_t phys = (uint32_t)__ldg(a.table + (size_t)b * a.max_blocks + tile / (256 / kTile));
    const bool held = phys < a.n_blocks;
    const size_t base = (((size_t)(held ? phys : 0u) * K + kh) * 256u + tile % (256 / kTile) * kTile) * D;
    const KV *kp = static_cast<const KV *>(a.k) + base, *vp = static_cast<const KV *>(a.v) + base;
    float *dk = s_k + stage * kTile * KS, *dv = s_v + stage * kTile * VS;
#pragma unroll 4
    for (uint32_t r = warp; r < kTile; r += kWarps) {
      const uint32_t key = tile * kTile + r;
      const bool seen = held && key >= k_lo && key < k_hi;
      if (async) {
#pragma unroll
        for (int i = 0; i < DV; ++i) {
          const uint32_t c = lane + 32 * i;
          if (c < D4) {
            cp_async16(dk + r * KS + 4 * c, kp + (size_t)r * D + 4 * c, seen ? 16u : 0u);
            cp_async16(dv + r * VS + 4 * c, vp + (size_t)r * D + 4 * c, seen ? 16u : 0u);
          }
        }
      } else {
        for (uint32_t c = lane; c < VS; c += 32) {
          const bool in = seen && c < D;
          dk[r * KS + c] = in ? ld_kv(kp, (size_t)r * D + c) : 0.f;
          dv[r * VS + c] = in ? ld_kv(vp, (size_t)r * D + c) : 0.f;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (t0 < t1) load(0, t0);
  for (uint32_t i = t; i < R * VS; i += kThreads) {
    const uint32_t r = i / VS, d = i % VS;
    s_q[i] = r < nr && d < D
                 ? ld_f32(static_cast<const T *>(a.q) + (it.first + token(r)) * a.q_stride, (size_t)head(r) * D + d) * (a.scale * ks)
                 : 0.f;
  }
  if (t < R) {
    s_m[t] = -INFINITY;
    s_l[t] = 0.f;
  }
  float4 acc[R][DV];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < DV; ++i) acc[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const uint32_t key = t % kTile, part = t / kTile, dq = (D4 + kParts - 1) / kParts;
  for (uint32_t tile = t0; tile < t1; ++tile) {
    const uint32_t stage = P.stages == 2 ? (tile - t0) & 1 : 0u;
    if (P.stages == 2 && tile + 1 < t1) {
      load(stage ^ 1, tile + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    {   // scores of one key over a part of the dims
      const float *kr = s_k + (stage * kTile + key) * KS;
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
      const uint32_t d1 = min(D4, (part + 1) * dq);
      for (uint32_t d = part * dq; d < d1; ++d) {
        const float4 x = *reinterpret_cast<const float4 *>(kr + 4 * d);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 y = *reinterpret_cast<const float4 *>(s_q + r * VS + 4 * d);
          s[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) s_s[(part * R + r) * kTile + key] = s[r];
    }
    __syncthreads();
    const uint32_t blk_ok = (uint32_t)__ldg(a.table + (size_t)b * a.max_blocks + tile / (256 / kTile));
    const bool held = blk_ok < a.n_blocks;
    for (uint32_t r = warp; r < R; r += kWarps) {
      const uint32_t p = it.pos0 + token(min(r, nr - 1));
      float x[kTile / 32], top = -INFINITY;   // (lanes per key)
#pragma unroll
      for (uint32_t i = 0; i < kTile / 32; ++i) {
        const uint32_t k = lane + 32 * i, pos = tile * kTile + k;
        x[i] = 0.f;
#pragma unroll
        for (uint32_t q = 0; q < kParts; ++q) x[i] += s_s[(q * R + r) * kTile + k];
        if (!held || pos > p || pos >= it.hi || (a.window && p - pos >= a.window)) x[i] = -INFINITY;
        top = fmaxf(top, x[i]);
      }
      const float m0 = s_m[r], m1 = fmaxf(m0, warp_max(top));
      // (nothing seen yet: no weights; a NaN stays one)
      const float c = m0 == -INFINITY ? 0.f : expf(m0 - m1);
      float sum = 0.f;
#pragma unroll
      for (uint32_t i = 0; i < kTile / 32; ++i) {
        const float e = x[i] == -INFINITY ? kUnseen : expf(x[i] - m1);
        s_p[(lane + 32 * i) * PS + r] = e;
        sum += e;
      }
      sum = warp_sum(sum);
      if (lane == 0) {
        s_m[r] = m1;
        s_l[r] = s_l[r] * c + sum;
        s_c[r] = c;
      }
    }
    __syncthreads();
    // a warp's eighth of the keys, four dims a lane (twice beyond 128)
    const bool plain = tile * kTile + kTile - 1 <= p_first && (!a.window || p_last - tile * kTile < a.window);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float c = s_c[r];
#pragma unroll
      for (int i = 0; i < DV; ++i) {
        acc[r][i].x *= c;
        acc[r][i].y *= c;
        acc[r][i].z *= c;
        acc[r][i].w *= c;
      }
    }
    const float *vt = s_v + stage * kTile * VS;
    for (uint32_t k = warp; k < kTile; k += kWarps) {
      float pr[R];
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(s_p + k * PS + r);
        pr[r] = f.x, pr[r + 1] = f.y, pr[r + 2] = f.z, pr[r + 3] = f.w;
      }
#pragma unroll
      for (int i = 0; i < DV; ++i) {
        const uint32_t c = lane + 32 * i;
        const float4 v = c < D4 ? *reinterpret_cast<const float4 *>(vt + k * VS + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        // (a key that only some rows see may hold a NaN; a seen one's counts, however small its weight)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (plain || !is_unseen(pr[r])) {
            acc[r][i].x = fmaf(pr[r], v.x, acc[r][i].x);
            acc[r][i].y = fmaf(pr[r], v.y, acc[r][i].y);
            acc[r][i].z = fmaf(pr[r], v.z, acc[r][i].z);
            acc[r][i].w = fmaf(pr[r], v.w, acc[r][i].w);
          }
      }
    }
    __syncthreads();   // the tile and the weights are free
    if (P.stages == 1 && tile + 1 < t1) load(0, tile + 1);
  }
  __syncthreads();
  // ---- the warps' sums, added in order through shared memory: [warp][R][VS] in the tiles' place
  float *red = s_k;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < DV; ++i)
      if (lane + 32 * i < D4) *reinterpret_cast<float4 *>(red + (warp * R + r) * VS + 4 * (lane + 32 * i)) = acc[r][i];
  __syncthreads();
  for (uint32_t i = t; i < nr * VS; i += kThreads) {
    const uint32_t r = i / VS, d = i % VS;
    if (d >= D) continue;
    const float m = s_m[r], l = s_l[r];
    float o = 0.f;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) o += red[w * R * VS + i];
    if (P.splits == 1) {
      const size_t row = (size_t)(it.first + token(r)) * H + head(r);
      st_elem(static_cast<T *>(a.out), row * D + d, l == 0.f ? 0.f : o / l * vs);
      if (a.lse && d == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
    } else {
      const size_t row = ((size_t)b * a.max_new + token(r)) * H + head(r), at = row * P.splits + split;
      P.part[at * D + d] = o;
      if (d == 0) {
        float *ml = P.part + (size_t)a.batch * a.max_new * H * P.splits * D + 2 * at;
        ml[0] = m;
        ml[1] = l;
      }
    }
  }
}

// A block per row: the shares' sums brought to their common maximum and added in order. Every
// warp works out the shares' weights for itself, 32 at a time, a lane each.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(Params P) {
  pdl_wait();
  pdl_trigger();
  const PagedArgs &a = P.a;
  const uint32_t D = a.head_dim, H = a.n_heads, h = blockIdx.x, tk = blockIdx.y, b = blockIdx.z, S = P.splits;
  const uint32_t d = threadIdx.x, lane = d & 31;
  const PagedItem it = paged_item(a, b);
  if (tk >= it.cnt) return;
  const size_t row = ((size_t)b * a.max_new + tk) * H + h, rows = (size_t)a.batch * a.max_new * H;
  const float *ml = P.part + rows * S * D + 2 * row * S, *part = P.part + row * S * D;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  bool nan = false;   // (fmaxf drops one)
  for (uint32_t s = lane; s < S; s += 32) m = fmaxf(m, ml[2 * s]), nan |= isnan(ml[2 * s + 1]);
  m = __any_sync(0xffffffffu, nan) ? NAN : warp_max(m);
  for (uint32_t s0 = 0; s0 < S; s0 += 32) {
    const float ls = s0 + lane < S ? ml[2 * (s0 + lane) + 1] : 0.f;
    const float w = ls == 0.f ? kUnseen : expf(ml[2 * (s0 + lane)] - m);
    l = fmaf(ls, w, l);
    for (uint32_t s = s0; s < min(S, s0 + 32); s += 8) {
      float v[8];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) v[u] = d < D && s + u < S ? part[(size_t)(s + u) * D + d] : 0.f;
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) {
        const float f = __shfl_sync(0xffffffffu, w, (s - s0 + u) & 31);
        if (s + u < S && !is_unseen(f)) acc = fmaf(v[u], f, acc);   // (a NaN times 0 is one)
      }
    }
  }
  l = warp_sum(l);
  const float vs = a.v_scale ? __ldg(a.v_scale + h / P.G) : 1.f;
  const size_t out = (size_t)(it.first + tk) * H + h;
  if (d < D) st_elem(static_cast<T *>(a.out), out * D + d, l == 0.f ? 0.f : acc / l * vs);
  if (a.lse && d == 0) a.lse[out] = l == 0.f ? -INFINITY : m + logf(l);
}

uint32_t group_rows(const PagedArgs &a) { return a.max_new * (a.n_heads / a.n_kv) <= 8 ? 8u : 16u; }

uint64_t blocks_unsplit(const PagedArgs &a) {
  const uint32_t G = a.n_heads / a.n_kv, R = group_rows(a);
  return (uint64_t)a.batch * a.n_kv * ((a.max_new * G + R - 1) / R);
}

// Shares of a sequence of `tiles` tiles at most: as many as fill the SMs (three blocks each, two for 16 rows),
// and up to eight blocks a SM where eight tiles are left to each, so that short sequences' SMs go on with
// long ones' shares (8 ragged sequences of 5,104 with 8 new tokens: 134 us with the former alone, 68); beyond 32 the
// join takes more than it saves (a sequence of 8,000 tokens, 8 heads of 64 dims: 57 shares 31 us, 32 25).
uint32_t splits_for(const PagedArgs &a, uint64_t tiles) {
  const uint64_t blocks = blocks_unsplit(a), sms = (uint64_t)num_sms();
  const uint64_t fill = ((group_rows(a) == 8 ? 3 : 2) * sms + blocks - 1) / blocks;
  uint64_t more = 8 * sms / blocks;
  if (more > tiles / 8) more = tiles / 8;
  uint64_t s = fill > more ? fill : more;
  if (s > 32 && 32 * blocks >= sms) s = 32;
  if (s > tiles) s = tiles;
  // (two tiles each where that still makes a block a SM)
  return (uint32_t)(s * 2 > tiles && blocks * tiles > 2 * sms ? (tiles + 1) / 2 : s);
}

// The most tiles of a sequence.
uint64_t most_tiles(const PagedArgs &a) {
  const uint32_t tile = tile_of(group_rows(a));
  const uint64_t all = 256ull / tile * a.max_blocks, w = ((uint64_t)a.window + a.max_new) / tile + 2;
  return a.window && w < all ? w : all;
}

// What a workspace has room for, whatever the window: at most as many shares as the SMs take.
uint32_t splits_most(const PagedArgs &a) {
  const uint64_t blocks = blocks_unsplit(a), s = (8ull * num_sms() + blocks - 1) / blocks, tiles = 256ull / tile_of(group_rows(a)) * a.max_blocks;
  return (uint32_t)(s < tiles ? s : tiles);
}

template <typename T, typename KV, int R, int DV>
cudaError_t launch_r(const PagedArgs &a, cudaStream_t s) {
  Params P;
  P.a = a;
  P.G = a.n_heads / a.n_kv;
  P.groups = (a.max_new * P.G + R - 1) / R;
  P.splits = splits_for(a, most_tiles(a));
  P.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + kWsHead);
  const uint32_t D4 = (a.head_dim + 3) / 4;
  // the next tile on its way, unless that leaves one block a SM and without it there are two (4 sequences of
  // 7,000, 48 rows of 128 dims, 2 / 8 heads: 125 / 373 us with one, 120 / 279 with two)
  auto per_sm = [&](uint32_t stages) { return kSmemSm / (smem_floats(D4, R, stages) * 4 + kSmemBlock); };
  P.stages = per_sm(2) >= 2 || per_sm(1) < 2 || blocks_per_sm(R, DV) < 2 ? 2 : 1;
  if (P.stages == 2 && smem_floats(D4, R, 2) * 4 > kSmemMost) P.stages = 1;
  const size_t smem = smem_floats(D4, R, P.stages) * 4;
  static RaisedLimit smem_set;
  auto *k = paged_attn_kernel<T, KV, R, DV>;
  cudaError_t e = ensure_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(P.splits, a.n_kv * P.groups, a.batch), dim3(kThreads), smem, s, P);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (P.splits > 1) {
    e = launch_pdl(paged_join_kernel<T>, dim3(a.n_heads, a.max_new, a.batch), dim3((a.head_dim + 31) / 32 * 32), 0, s, P);
    if (e != cudaSuccess) return e;
    note_launches(1);
  }
  return cudaGetLastError();
}
template <typename T, typename KV>
cudaError_t launch_t(const PagedArgs &a, cudaStream_t s) {
  if (group_rows(a) == 8) return a.head_dim <= 128 ? launch_r<T, KV, 8, 1>(a, s) : launch_r<T, KV, 8, 2>(a, s);
  return a.head_dim <= 128 ? launch_r<T, KV, 16, 1>(a, s) : launch_r<T, KV, 16, 2>(a, s);
}

}  // namespace

size_t paged_attn_ws_bytes(const PagedArgs &a) {
  if (paged_attn_tc_takes(a)) return kWsHead + paged_attn_tc_ws_bytes(a);
  const uint32_t S = splits_most(a);
  return kWsHead + (S > 1 ? (size_t)a.batch * a.max_new * a.n_heads * S * (a.head_dim + 2) * 4 : 0);
}

cudaError_t launch_paged_attn(const PagedArgs &a, cudaStream_t s) {
  if (paged_attn_tc_takes(a)) return launch_paged_attn_tc(a, s);
  if (a.kv_dtype == DS4A_E4M3)
    return a.dtype == DS4A_BF16 ? launch_t<__nv_bfloat16, __nv_fp8_storage_t>(a, s)
                                : launch_t<float, __nv_fp8_storage_t>(a, s);
  return a.dtype == DS4A_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_t<float, float>(a, s);
}

}  // namespace ds4a
