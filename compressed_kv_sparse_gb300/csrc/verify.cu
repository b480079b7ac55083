// Verification of drafted tokens against the target's probabilities (Leviathan et al.,
// "Fast Inference from Transformers via Speculative Decoding", section 2.3).
//
// Draft i stands while u_i q_i(x_i) < p_i(x_i). The token behind the last that stands is drawn
// from w = max(p - q, 0) of the one that fell, or from p, by the first running sum above u
// times the total. p and q are taken as whole multiples of 2^-s (s = 45, less beyond 131,072 tokens),
// so the sums are whole numbers: any order gives the same ones, and blocks and warps may share a row.
//
// A cluster of blocks per sequence. Every block tests the drafts for itself (a warp, a draft
// per lane), sums its share of the row (each warp consecutive chunks of 512 tokens, whose sums it
// keeps), and reads the others' sums through distributed shared memory; the warp in whose part
// the sum passes the threshold finds the chunk, reads it again (it is in the caches) and finds the token.
// Bound by HBM for many sequences: a row of p, and one of q where a draft fell, read once (256 sequences of 131,072
// tokens in fp32 38.1 us, 5.4 TB/s); for a few by the chain of drafts, a row's chunks, the cluster's sums and the second read
// (8 sequences of 50,021 tokens 6.1 us; with the chunk read again in four steps instead of one 6.6).
#include <type_traits>

#include "common.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kChunk = 512;   // tokens that a warp adds at once

struct Params {
  VerifyArgs a;
  uint32_t shift;    // s
  uint32_t part;     // tokens per block (a multiple of a chunk per warp)
};

// A probability (above 1: 1, negative and NaN: 0) as the whole number of 2^-s nearest to it, in two parts, hi
// 2^(s - 23) + lo: hi its nearest multiple of 2^-23, lo what is left of it. Adding 1, or 1.5 * 2^23 to a
// number below 2^22, rounds to whole steps that stand in the low bits; the conversion instructions take
// 16 clocks a warp. bits() of hi and lo carry constants, which differences drop.
struct Parts {
  uint32_t hi, lo;
};
constexpr uint32_t kHi0 = 0x3f800000u, kLo0 = 0x4b400000u;   // the bits of 1 and of 1.5 * 2^23
__device__ __forceinline__ Parts parts_of(float p, float scale) {   // p in [0, 1]
  const float t = p + 1.f, rest = p - (t - 1.f);
  return Parts{__float_as_uint(t), __float_as_uint(fmaf(rest, scale, 12582912.f))};
}
// a - b in units of 2^-s.
__device__ __forceinline__ int64_t difference(Parts a, Parts b, uint32_t hi_unit) {
  return (int64_t)(int32_t)(a.hi - b.hi) * (int32_t)hi_unit + (int32_t)(a.lo - b.lo);
}

template <typename T, bool VEC>
__device__ __forceinline__ void load4(float (&v)[4], const T *row, uint32_t i, uint32_t end) {
  if (VEC) {
    if (i < end) {   // (end is a multiple of 4)
      if (sizeof(T) == 4) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(row + i));
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(row + i));
        v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
      }
    } else {
      v[0] = v[1] = v[2] = v[3] = 0.f;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k < end ? ld_f32(row, i + k) : 0.f;
  }
}

// Weights of tokens i .. i + 3: p - q where positive, p without q; drop: this token's is 0.
__device__ __forceinline__ void weights(uint64_t (&w)[4], const float (&p)[4], const float (&q)[4], bool has_q,
                                        uint32_t i, uint32_t drop, float scale, uint32_t hi_unit) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = __saturatef(p[k]);
    const Parts y = has_q ? parts_of(fminf(x, __saturatef(q[k])), scale) : Parts{kHi0, kLo0};
    w[k] = i + k == drop ? 0ull : (uint64_t)difference(parts_of(x, scale), y, hi_unit);
  }
}

// floor(u total), exactly, for total below 2^62 and u (held to [0, 1)) = m 2^-e with m below 2^24: a whole number is above
// u total where it is above this. (In fp64 u total may round up to the running sum next to it.)
__device__ __forceinline__ uint64_t threshold(float u, uint64_t total) {
  const uint32_t bits = __float_as_uint(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f));
  const uint64_t m = bits >> 23 ? (bits & 0x7fffffu) | 0x800000u : bits;
  const uint32_t e = 150 - max(bits >> 23, 1u);                    // 24 .. 149
  const uint64_t lo = m * total, hi = __umul64hi(m, total);   // below 2^86
  return e < 64 ? lo >> e | hi << (64 - e) : e < 128 ? hi >> (e - 64) : 0ull;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// (Four blocks a SM hide the loads: 256 sequences of 131,072 tokens, three quarters with a draft that fell,
// take 38 us, with registers for three or two blocks a SM 50. Next chunks on their way in registers or shared memory leave
// room for two or three blocks: 54 to 60 on an earlier version that took 43.)
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(Params P) {
  extern __shared__ uint64_t s_chunks[];   // [warp][chunks of a warp]
  __shared__ uint64_t s_sum[2];         // this block's sum, of each of two attempts
  __shared__ uint64_t s_warp[kWarps];
  __shared__ uint32_t s_acc;
  const VerifyArgs &a = P.a;
  const uint32_t b = blockIdx.y, rank = blockIdx.x, nc = gridDim.x;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, N = a.max_drafts, V = a.vocab;
  pdl_wait();
  pdl_trigger();
  const uint32_t c0 = a.cu_len ? __ldg(a.cu_len + b) : b * (N + 1);
  const uint32_t cnt = a.cu_len ? __ldg(a.cu_len + b + 1) - c0 : N + 1;
  const bool there = cnt != 0 && cnt < 0x80000000u;
  const uint32_t m = there ? min(cnt - 1, N) : 0u;
  // ---- the drafts
  if (warp == 0) {
    uint32_t acc = 0;
    for (uint32_t i0 = 0; i0 < m; i0 += 32) {
      const uint32_t i = i0 + lane;
      bool ok = false;
      if (i < m) {
        const uint32_t x = (uint32_t)__ldg(a.drafts + (size_t)b * N + i);
        if (x < V) {
          const double u = (double)__ldg(a.u_accept + (size_t)b * N + i);
          const double p = (double)ld_f32(static_cast<const T *>(a.target) + (c0 + i) * a.target_stride, x);
          const double q =
              a.draft_probs ? (double)ld_f32(static_cast<const T *>(a.draft_probs) + ((size_t)b * N + i) * V, x)
                            : 1.0;
          ok = u * q < p;   // (two 24-bit numbers: their product is exact in 53 bits)
        }
      }
      const uint32_t bad = ~__ballot_sync(0xffffffffu, ok);
      if (bad) {
        acc = i0 + (uint32_t)__ffs(bad) - 1;
        break;
      }
      acc = i0 + 32;
    }
    if (lane == 0) s_acc = min(acc, m);
  }
  __syncthreads();
  const uint32_t acc = s_acc;
  const bool fell = acc < m;
  if (rank == 0) {
    for (uint32_t i = threadIdx.x; i <= N; i += kThreads)
      if (!there || i != acc)
        a.tokens[(size_t)b * (N + 1) + i] = i < acc ? __ldg(a.drafts + (size_t)b * N + i) : -1;
    if (threadIdx.x == 0) {
      a.n_out[b] = there ? acc + 1 : 0u;
      if (a.ctx_out) a.ctx_out[b] = __ldg(a.seq_pos + b) + (there ? acc + 1 : 0u);
    }
  }
  if (!there) return;   // (the whole cluster)
  // ---- the token behind them
  const T *p_row = static_cast<const T *>(a.target) + (c0 + acc) * a.target_stride;
  const T *q_row = static_cast<const T *>(a.draft_probs) + ((size_t)b * N + acc) * V;
  const float scale = __uint_as_float((P.shift + 127u) << 23);
  const uint32_t hi_unit = 1u << (P.shift - 23);
  const uint32_t wpart = P.part / kWarps, w0 = rank * P.part + warp * wpart, w1 = min(V, w0 + wpart);
  for (uint32_t attempt = 0; attempt < 2; ++attempt) {
    // (attempt 1: no weight was above zero; p alone)
    const bool has_q = fell && a.draft_probs && !attempt;
    const uint32_t drop = fell && !a.draft_probs && !attempt ? (uint32_t)__ldg(a.drafts + (size_t)b * N + acc)
                                                             : 0xffffffffu;
    // (a chunk's 16 tokens of a lane: i0 + 128 u + 4 lane + k)
    uint64_t *mine = s_chunks + warp * (wpart / kChunk);
    uint64_t sum = 0;
    auto add = [&](auto hq, uint32_t i0, const float (&p)[4][4], const float (&q)[4][4]) {
      // (sums of 16 parts stay in 32 bits)
      uint32_t hi = 0;
      int32_t lo = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = __saturatef(p[u][k]);
          const Parts f = parts_of(x, scale);
          if constexpr (decltype(hq)::value) {
            const Parts g = parts_of(fminf(x, __saturatef(q[u][k])), scale);   // (where q is larger: p - p)
            hi += f.hi - g.hi;
            lo += (int32_t)(f.lo - g.lo);
          } else {
            hi += f.hi - kHi0;
            lo += (int32_t)(f.lo - kLo0);
          }
        }
      uint64_t c = (uint64_t)hi * hi_unit + (int64_t)lo;
      c = warp_sum64(c);
      if (drop - i0 < kChunk && drop < w1)
        c -= (uint64_t)difference(parts_of(__saturatef(ld_f32(p_row, drop)), scale), Parts{kHi0, kLo0}, hi_unit);
      if (lane == 0) mine[(i0 - w0) / kChunk] = c;
      sum += c;
    };
    auto pass = [&](auto hq) {
      for (uint32_t i0 = w0; i0 < w1; i0 += kChunk) {
        float p[4][4], q[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          load4<T, VEC>(p[u], p_row, i0 + 128 * u + 4 * lane, w1);
          if (hq.value) load4<T, VEC>(q[u], q_row, i0 + 128 * u + 4 * lane, w1);
        }
        add(hq, i0, p, q);
      }
    };
    if (has_q)
      pass(std::true_type{});
    else
      pass(std::false_type{});
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    uint64_t before = 0, own = 0;
    for (uint32_t w = 0; w < kWarps; ++w) {
      const uint64_t x = s_warp[w];
      if (w < warp) before += x;
      own += x;
    }
    if (threadIdx.x == 0) s_sum[attempt] = own;
    cluster_sync_all();
    uint64_t total = 0;
    for (uint32_t r = 0; r < nc; ++r) {
      const uint64_t x = ld_cluster_u64(mapa_shared(smem_u32(&s_sum[attempt]), r));
      if (r < rank) before += x;
      total += x;
    }
    if (total == 0) {
      if (attempt == 0) continue;   // (the whole cluster; each attempt has a place of its own)
      if (rank == 0 && threadIdx.x == 0) a.tokens[(size_t)b * (N + 1) + acc] = (int32_t)V - 1;
      break;
    }
    const uint64_t thr = threshold(__ldg(a.u_sample + b), total);
    if (before <= thr && thr < before + sum) {   // this warp's part (the whole warp)
      __syncwarp();
      uint64_t run = before;
      uint32_t i0 = w0;
      for (uint32_t n = 0; run + mine[n] <= thr; ++n, i0 += kChunk) run += mine[n];   // (it is there)
      float p[4][4], q[4][4];   // (the whole chunk on its way at once)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        load4<T, VEC>(p[u], p_row, i0 + 128 * u + 4 * lane, w1);
        if (has_q) load4<T, VEC>(q[u], q_row, i0 + 128 * u + 4 * lane, w1);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {   // (it is in one of the four)
        const uint32_t i = i0 + 128 * u + 4 * lane;
        uint64_t w[4];
        weights(w, p[u], q[u], has_q, i, drop, scale, hi_unit);
        const uint64_t four = (w[0] + w[1]) + (w[2] + w[3]);
        uint64_t inc = four;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= (uint32_t)o) inc += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + inc > thr);
        if (hit) {
          if (lane == (uint32_t)__ffs(hit) - 1) {
            const uint64_t a0 = run + inc - four + w[0], a1 = a0 + w[1], a2 = a1 + w[2];
            const uint32_t k = a0 > thr ? 0u : a1 > thr ? 1u : a2 > thr ? 2u : 3u;
            a.tokens[(size_t)b * (N + 1) + acc] = (int32_t)(i + k);
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    break;
  }
  cluster_sync_all();   // (nobody reads this block's sum any more)
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s) {
  Params P;
  P.a = a;
  P.shift = 45;   // (V times 2^s stays below 2^62, a rest below 2^-24 times 2^s below 2^22)
  while ((1ull << (62 - P.shift)) < a.vocab) --P.shift;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft_probs);
  const uint32_t es = a.dtype == DS4A_BF16 ? 2 : 4;
  const bool vec = all % (4 * es) == 0 && a.vocab % 4 == 0 && a.target_stride % 4 == 0;
  // up to eight blocks a sequence while no more than four a SM come of it, which run at once (256 sequences of 131,072
  // tokens with eight each 46.6 us, four 40.2, two, as here, 38.1, one 46.6)
  uint32_t cluster = 8;
  while (cluster > 1 && (uint64_t)a.batch * cluster > 4ull * num_sms()) cluster /= 2;
  constexpr uint32_t kStep = kChunk * kWarps;
  P.part = ((a.vocab + cluster - 1) / cluster + kStep - 1) / kStep * kStep;
  const size_t smem = P.part / kChunk * sizeof(uint64_t);   // (at most 16 KiB)
  auto *k = a.dtype == DS4A_BF16 ? (vec ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>)
                                 : (vec ? verify_kernel<float, true> : verify_kernel<float, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(cluster, a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, P);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace ds4a
