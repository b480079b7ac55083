// Verification of drafted tokens against the target's probabilities (Leviathan et al.,
// "Fast Inference from Transformers via Speculative Decoding", section 2.3).
//
// Draft i stands while u_i q_i(x_i) < p_i(x_i). The token behind the last that stands is drawn
// from w = max(p - q, 0) of the one that fell, or from p, by the first running sum above u
// times the total. p and q are taken as whole multiples of 2^-s (s = 62 - ceil(log2 V)), so
// the sums are whole numbers: any order gives the same ones, and blocks and warps may share a row.
//
// A cluster of blocks per sequence. Every block tests the drafts for itself (a warp, a draft
// per lane), sums its share of the row (each warp consecutive tokens), and reads
// the others' sums through distributed shared memory; the warp in whose part the sum passes
// the threshold reads its part again (it is in the caches) and finds the token.
// Bound by HBM for many sequences: a row of p, and one of q where a draft fell, read once.
#include "common.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;

struct Params {
  VerifyArgs a;
  uint32_t shift;    // s
  uint32_t part;     // tokens per block (a multiple of 128 * kWarps)
};

// Whole multiples of 2^-s of a probability; above 1: 1, negative and NaN: 0.
__device__ __forceinline__ uint64_t fixed(float p, float scale) {
  return __float2ull_rn(fminf(fmaxf(p, 0.f), 1.f) * scale);
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
template <typename T, bool VEC>
__device__ __forceinline__ void weights(uint64_t (&w)[4], const float (&p)[4], const float (&q)[4], bool has_q,
                                        uint32_t i, uint32_t drop, float scale) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint64_t x = fixed(p[k], scale);
    if (has_q) {
      const uint64_t y = fixed(q[k], scale);
      x = x > y ? x - y : 0ull;
    }
    w[k] = i + k == drop ? 0ull : x;
  }
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

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) verify_kernel(Params P) {
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
  const uint32_t wpart = P.part / kWarps, w0 = rank * P.part + warp * wpart, w1 = min(V, w0 + wpart);
  for (uint32_t attempt = 0; attempt < 2; ++attempt) {
    // (attempt 1: no weight was above zero; p alone)
    const bool has_q = fell && a.draft_probs && !attempt;
    const uint32_t drop = fell && !a.draft_probs && !attempt ? (uint32_t)__ldg(a.drafts + (size_t)b * N + acc)
                                                             : 0xffffffffu;
    uint64_t sum = 0;
    for (uint32_t i0 = w0; i0 < w1; i0 += 512) {
      float p[4][4], q[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        load4<T, VEC>(p[u], p_row, i0 + 128 * u + 4 * lane, w1);
        if (has_q) load4<T, VEC>(q[u], q_row, i0 + 128 * u + 4 * lane, w1);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint64_t w[4];
        weights<T, VEC>(w, p[u], q[u], has_q, i0 + 128 * u + 4 * lane, drop, scale);
        sum += w[0] + w[1] + w[2] + w[3];
      }
    }
    sum = warp_sum64(sum);
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
    const float u = fminf(fmaxf(__ldg(a.u_sample + b), 0.f), 0x1.fffffep-1f);
    const uint64_t thr = (uint64_t)((double)u * (double)total);   // below total
    if (before <= thr && thr < before + sum) {   // this warp's part (the whole warp)
      uint64_t run = before;
      for (uint32_t i0 = w0; i0 < w1; i0 += 128) {
        const uint32_t i = i0 + 4 * lane;
        float p[4], q[4];
        uint64_t w[4];
        load4<T, VEC>(p, p_row, i, w1);
        if (has_q) load4<T, VEC>(q, q_row, i, w1);
        weights<T, VEC>(w, p, q, has_q, i, drop, scale);
        const uint64_t mine = w[0] + w[1] + w[2] + w[3];
        uint64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= (uint32_t)o) inc += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + inc > thr);
        if (hit) {
          if (lane == (uint32_t)__ffs(hit) - 1) {
            uint64_t r = run + inc - mine;
            uint32_t k = 0;
            for (; k < 3; ++k) {
              r += w[k];
              if (r > thr) break;
            }
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
  P.shift = 62;
  while ((1ull << (62 - P.shift)) < a.vocab) --P.shift;
  constexpr uint32_t kCluster = 8, kStep = 128 * kWarps;
  P.part = ((a.vocab + kCluster - 1) / kCluster + kStep - 1) / kStep * kStep;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft_probs);
  const uint32_t es = a.dtype == DS4A_BF16 ? 2 : 4;
  const bool vec = all % (4 * es) == 0 && a.vocab % 4 == 0 && a.target_stride % 4 == 0;
  auto *k = a.dtype == DS4A_BF16 ? (vec ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>)
                                 : (vec ? verify_kernel<float, true> : verify_kernel<float, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kCluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(kCluster, a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, P);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace ds4a
