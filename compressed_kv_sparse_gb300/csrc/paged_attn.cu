// Attention of a step's new tokens over a paged cache of keys and values, on the CUDA cores: the
// exact path of fp32 layers and the one for sizes that the tensor-core kernel does not take.
//
// Rows (a sequence's tokens x the query heads of one key head) in groups of up to 16, keys in
// tiles of 64: a block scores a tile (a thread per key and quarter of the rows), updates each
// row's running maximum and sum (a warp per row), and adds the weighted values (a thread
// per dim). A sequence's tiles are shared among several blocks where there are few rows; each
// leaves its sums with their maximum, and a second launch joins them in order.
#include <cuda_fp8.h>

#include "paged.cuh"

namespace ds4a {

namespace {

constexpr uint32_t kThreads = 256, kTile = 64, kRows = 16;
constexpr uint32_t kWsHead = 256;   // the status word's line

struct Params {
  PagedArgs a;
  uint32_t G, groups, splits;   // query heads per key head, row groups, shares of the keys
  float *part;                  // [batch * max_new * H][splits][D], then (max, sum) of each
};

template <typename T>
__device__ __forceinline__ float ld_kv(const T *p, size_t i) {
  return ld_f32(p, i);
}
__device__ __forceinline__ float ld_kv(const __nv_fp8_storage_t *p, size_t i) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3)));
}

template <typename T, typename KV>
__global__ void __launch_bounds__(kThreads) paged_attn_kernel(Params P) {
  extern __shared__ float sm[];
  const PagedArgs &a = P.a;
  const uint32_t D = a.head_dim, DP = D + 1, H = a.n_heads, K = a.n_kv;
  float *s_k = sm;                        // [64][D + 1]
  float *s_q = s_k + kTile * DP;          // [16][D]
  float *s_p = s_q + kRows * D;           // [16][64]
  float *s_m = s_p + kRows * kTile, *s_l = s_m + kRows, *s_c = s_l + kRows;   // max, sum, factor
  pdl_wait();
  pdl_trigger();
  const uint32_t split = blockIdx.x, kh = blockIdx.y / P.groups, rg = blockIdx.y % P.groups, b = blockIdx.z;
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const PagedItem it = paged_item(a, b);
  const uint32_t r0 = rg * kRows, all = it.cnt * P.G;
  if (r0 >= all) return;
  const uint32_t nr = min(kRows, all - r0);
  const uint32_t t_lo = it.lo / kTile, t_hi = (it.hi + kTile - 1) / kTile, nt = t_hi > t_lo ? t_hi - t_lo : 0u;
  const uint32_t t0 = t_lo + (uint32_t)((uint64_t)nt * split / P.splits);
  const uint32_t t1 = t_lo + (uint32_t)((uint64_t)nt * (split + 1) / P.splits);
  const float ks = a.k_scale ? __ldg(a.k_scale + kh) : 1.f, vs = a.v_scale ? __ldg(a.v_scale + kh) : 1.f;
  auto token = [&](uint32_t r) { return (r0 + r) / P.G; };
  auto head = [&](uint32_t r) { return kh * P.G + (r0 + r) % P.G; };
  for (uint32_t i = t; i < nr * D; i += kThreads) {
    const uint32_t r = i / D, d = i % D;
    s_q[i] = ld_f32(static_cast<const T *>(a.q) + (it.first + token(r)) * a.q_stride, (size_t)head(r) * D + d) * (a.scale * ks);
  }
  if (t < kRows) {
    s_m[t] = -INFINITY;
    s_l[t] = 0.f;
  }
  float acc[kRows];
#pragma unroll
  for (uint32_t i = 0; i < kRows; ++i) acc[i] = 0.f;
  // values: thread -> dim d, rows sub, sub + subs, ..
  const uint32_t subs = kThreads / D, sub = t / D, d = t % D;   // (D <= 256)
  for (uint32_t tile = t0; tile < t1; ++tile) {
    const uint32_t blk = tile / (256 / kTile);
    const uint32_t phys = (uint32_t)__ldg(a.table + (size_t)b * a.max_blocks + blk);
    if (phys >= a.n_blocks) continue;   // (the whole block)
    const size_t base = (((size_t)phys * K + kh) * 256u + tile % (256 / kTile) * kTile) * D;
    const KV *kp = static_cast<const KV *>(a.k) + base, *vp = static_cast<const KV *>(a.v) + base;
    __syncthreads();
    for (uint32_t i = t; i < kTile * D; i += kThreads) s_k[i / D * DP + i % D] = ld_kv(kp, i);
    __syncthreads();
    {
      const uint32_t key = t % kTile, q4 = t / kTile, pos = tile * kTile + key;
      float s[kRows / 4] = {0.f, 0.f, 0.f, 0.f};
      for (uint32_t e = 0; e < D; ++e) {
        const float x = s_k[key * DP + e];
#pragma unroll
        for (uint32_t i = 0; i < kRows / 4; ++i)
          if (q4 + 4 * i < nr) s[i] = fmaf(x, s_q[(q4 + 4 * i) * D + e], s[i]);
      }
#pragma unroll
      for (uint32_t i = 0; i < kRows / 4; ++i) {
        const uint32_t r = q4 + 4 * i;
        if (r >= nr) break;
        const uint32_t p = it.pos0 + token(r);
        const bool seen = pos <= p && pos < it.hi && (!a.window || p - pos < a.window);
        s_p[r * kTile + key] = seen ? s[i] : -INFINITY;
      }
    }
    __syncthreads();
    for (uint32_t r = warp; r < nr; r += kThreads / 32) {
      const float x0 = s_p[r * kTile + lane], x1 = s_p[r * kTile + 32 + lane], m0 = s_m[r];
      const float m1 = fmaxf(m0, warp_max(fmaxf(x0, x1)));
      // (nothing seen yet: no weights; a NaN stays one)
      const float e0 = x0 == -INFINITY ? 0.f : expf(x0 - m1), e1 = x1 == -INFINITY ? 0.f : expf(x1 - m1);
      const float c = m0 == -INFINITY ? 0.f : expf(m0 - m1);
      const float sum = warp_sum(e0 + e1);
      s_p[r * kTile + lane] = e0;
      s_p[r * kTile + 32 + lane] = e1;
      if (lane == 0) {
        s_m[r] = m1;
        s_l[r] = s_l[r] * c + sum;
        s_c[r] = c;
      }
    }
    __syncthreads();
    if (sub < subs) {
#pragma unroll
      for (uint32_t i = 0; i < kRows; ++i)
        if (sub + i * subs < nr) acc[i] *= s_c[sub + i * subs];
      for (uint32_t key = 0; key < kTile; ++key) {
        const float v = ld_kv(vp, (size_t)key * D + d);
#pragma unroll
        for (uint32_t i = 0; i < kRows; ++i) {
          if (sub + i * subs >= nr) break;
          const float p = s_p[(sub + i * subs) * kTile + key];
          if (p != 0.f) acc[i] = fmaf(p, v, acc[i]);   // (an unseen row may hold a NaN)
        }
      }
    }
  }
  __syncthreads();
  if (sub >= subs) return;
#pragma unroll
  for (uint32_t i = 0; i < kRows; ++i) {
    const uint32_t r = sub + i * subs;
    if (r >= nr) break;
    const float m = s_m[r], l = s_l[r];
    if (P.splits == 1) {
      const size_t row = (size_t)(it.first + token(r)) * H + head(r);
      st_elem(static_cast<T *>(a.out), row * D + d, l == 0.f ? 0.f : acc[i] / l * vs);
      if (a.lse && d == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
    } else {
      const size_t row = ((size_t)b * a.max_new + token(r)) * H + head(r), at = row * P.splits + split;
      P.part[at * D + d] = acc[i];
      if (d == 0) {
        float *ml = P.part + (size_t)a.batch * a.max_new * H * P.splits * D + 2 * at;
        ml[0] = m;
        ml[1] = l;
      }
    }
  }
}

// A block per row: the shares' sums brought to their common maximum and added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(Params P) {
  pdl_wait();
  pdl_trigger();
  const PagedArgs &a = P.a;
  const uint32_t D = a.head_dim, H = a.n_heads, h = blockIdx.x, tk = blockIdx.y, b = blockIdx.z;
  const PagedItem it = paged_item(a, b);
  if (tk >= it.cnt) return;
  const size_t row = ((size_t)b * a.max_new + tk) * H + h, rows = (size_t)a.batch * a.max_new * H;
  const float *ml = P.part + rows * P.splits * D + 2 * row * P.splits;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  bool nan = false;   // (fmaxf drops one)
  for (uint32_t s = 0; s < P.splits; ++s) m = fmaxf(m, ml[2 * s]), nan |= isnan(ml[2 * s + 1]);
  if (nan) m = NAN;
  const uint32_t d = threadIdx.x;
  for (uint32_t s = 0; s < P.splits; ++s) {
    if (ml[2 * s + 1] == 0.f) continue;
    const float c = expf(ml[2 * s] - m);
    l = fmaf(ml[2 * s + 1], c, l);
    if (d < D) acc = fmaf(P.part[(row * P.splits + s) * D + d], c, acc);
  }
  const float vs = a.v_scale ? __ldg(a.v_scale + h / P.G) : 1.f;
  const size_t out = (size_t)(it.first + tk) * H + h;
  if (d < D) st_elem(static_cast<T *>(a.out), out * D + d, l == 0.f ? 0.f : acc / l * vs);
  if (a.lse && d == 0) a.lse[out] = l == 0.f ? -INFINITY : m + logf(l);
}

// Shares of a sequence's keys: enough blocks for two a SM, 256 keys each at least.
uint32_t splits_of(const PagedArgs &a) {
  const uint32_t G = a.n_heads / a.n_kv, groups = (a.max_new * G + kRows - 1) / kRows;
  const uint64_t blocks = (uint64_t)a.batch * a.n_kv * groups, want = (uint64_t)num_sms() * 2;
  uint64_t s = (want + blocks - 1) / blocks, most = a.max_blocks;
  if (a.window) {
    const uint64_t w = ((uint64_t)a.window + a.max_new) / 256 + 1;
    most = w < most ? w : most;
  }
  if (s > most) s = most;
  return s < 1 ? 1u : (uint32_t)s;
}

template <typename T, typename KV>
cudaError_t launch_t(const PagedArgs &a, cudaStream_t s) {
  Params P;
  P.a = a;
  P.G = a.n_heads / a.n_kv;
  P.groups = (a.max_new * P.G + kRows - 1) / kRows;
  P.splits = splits_of(a);
  P.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + kWsHead);
  const size_t smem = ((size_t)kTile * (a.head_dim + 1) + kRows * a.head_dim + kRows * kTile + 3 * kRows) * 4;
  static RaisedLimit smem_set;
  auto *k = paged_attn_kernel<T, KV>;
  cudaError_t e = ensure_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(P.splits, a.n_kv * P.groups, a.batch), dim3(kThreads), smem, s, P);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (P.splits > 1) {
    e = launch_pdl(paged_join_kernel<T>, dim3(a.n_heads, a.max_new, a.batch), dim3(kThreads), 0, s, P);
    if (e != cudaSuccess) return e;
    note_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace

size_t paged_attn_ws_bytes(const PagedArgs &a) {
  if (paged_attn_tc_takes(a)) return kWsHead + paged_attn_tc_ws_bytes(a);
  const uint32_t S = splits_of(a);
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
