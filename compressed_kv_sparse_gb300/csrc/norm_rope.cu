// RMSNorm of every query head and of the shared K = V row of each token, the
// tail rotation and the insert of the row into the raw window, in one pass
// (vLLM DeepSeek V4 page, section "GPU 計算飽和": fused Q norm + KV RoPE + K
// insert; "【#3】ds4.c を読み解く" §8 tail-only RoPE).
//
// One warp owns one row (a head of a token, or the token's K = V row): the row
// stays in registers between the sum of squares and the scaled, rotated store, so
// each element is read once and written once. Bound by HBM at a chunk's size, by
// the launch at a decode step's.
#include "common.cuh"
#include "tc.cuh"

namespace ds4a {
namespace {

constexpr int kThreads = 256;
constexpr float kRmsEps = 1e-6f;

struct NormArgs {
  const void *q, *kv, *gamma_q, *gamma_kv;
  void *q_out, *kv_dst;
  uint64_t q_stride, kv_stride;   // elements between tokens
  const int32_t *pos, *slots;
  const float *cos, *sin;
  uint32_t n, H, D, n_rot, max_pos, n_dst;
  uint32_t per;      // rows per token: H (+ 1 with the K = V row)
  uint32_t rot_q;
  uint64_t n_rows;
};

// E elements of one row from / to memory as fp32 (E * sizeof(T) = 16, or 2
// elements one by one where the rows are not 16-byte aligned).
template <typename T, int E>
__device__ __forceinline__ void load_e(const T *p, float *v) {
  if (E * sizeof(T) == 16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = ld_f32(e, i);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = ld_f32(p, i);
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_e(T *p, const float *v) {
  if (E * sizeof(T) == 16) {
    uint4 u;
    T *e = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int i = 0; i < E; ++i) st_elem(e, i, v[i]);
    *reinterpret_cast<uint4 *>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) st_elem(p, i, v[i]);
  }
}

// NV: chunks of E elements per lane (D <= 32 E NV).
template <typename T, int E, int NV>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormArgs a) {
  pdl_wait();
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t step = (uint64_t)gridDim.x * (kThreads / 32);
  for (uint64_t r = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < a.n_rows;
       r += step) {
    const uint32_t tok = (uint32_t)(r / a.per), h = (uint32_t)(r % a.per);
    const bool is_q = h < a.H;
    const int32_t p = __ldg(a.pos + tok);
    if (p < 0 || (uint32_t)p >= a.max_pos) continue;   // warp-uniform: the row is left alone
    const T *src;
    T *dst;
    const T *gamma = static_cast<const T *>(is_q ? a.gamma_q : a.gamma_kv);
    if (is_q) {
      src = static_cast<const T *>(a.q) + tok * a.q_stride + (size_t)h * a.D;
      dst = static_cast<T *>(a.q_out) + ((size_t)tok * a.H + h) * a.D;
    } else {
      const int64_t s = a.slots ? (int64_t)__ldg(a.slots + tok) : (int64_t)tok;
      if (s < 0 || s >= (int64_t)a.n_dst) continue;
      src = static_cast<const T *>(a.kv) + tok * a.kv_stride;
      dst = static_cast<T *>(a.kv_dst) + (size_t)s * a.D;
    }
    float v[NV][E];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = E * (lane + 32 * i);
      if (c < a.D) {
        load_e<T, E>(src + c, v[i]);
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(v[i][e], v[i][e], ss);
      }
    }
    ss = warp_sum(ss);
    const float inv = 1.0f / sqrtf(ss / (float)a.D + kRmsEps);
    const uint32_t nope = a.D - a.n_rot;
    const bool rot = !is_q || a.rot_q;
    const float *co = a.cos + (size_t)p * (a.n_rot / 2), *si = a.sin + (size_t)p * (a.n_rot / 2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = E * (lane + 32 * i);
      if (c >= a.D) continue;
      float g[E];
      if (gamma) load_e<T, E>(gamma + c, g);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float x0 = v[i][e] * inv, x1 = v[i][e + 1] * inv;
        if (gamma) {
          x0 *= g[e];
          x1 *= g[e + 1];
        }
        if (rot && c + e >= nope) {
          const uint32_t f = (c + e - nope) / 2;
          const float cs = __ldg(co + f), sn = __ldg(si + f);
          const float r0 = x0 * cs - x1 * sn, r1 = x0 * sn + x1 * cs;
          x0 = r0;
          x1 = r1;
        }
        v[i][e] = x0;
        v[i][e + 1] = x1;
      }
      store_e<T, E>(dst + c, v[i]);
    }
  }
  // The attention starts its first query load before it waits for the previous
  // launch (griddepcontrol.wait). When that launch is this one, it has begun only
  // once every block here has ended, so it is enough that this thread's stores
  // are done for the whole GPU, copies by TMA included, before it ends. For the
  // same reason there is no early launch trigger.
  fence_proxy_async_global();
  __threadfence();
}

template <typename T, int E>
cudaError_t launch_e(const NormArgs &a, cudaStream_t s) {
  constexpr uint32_t rows_per_block = kThreads / 32;
  const uint64_t blocks = (a.n_rows + rows_per_block - 1) / rows_per_block;
  const uint64_t most = (uint64_t)num_sms() * 8 * 4;
  const dim3 grid((uint32_t)(blocks < most ? blocks : most));
  const uint32_t nv = (a.D + 32 * E - 1) / (32 * E);
  cudaError_t e;
  switch (nv) {
    case 1: e = launch_pdl(norm_rope_kernel<T, E, 1>, grid, dim3(kThreads), 0, s, a); break;
    case 2: e = launch_pdl(norm_rope_kernel<T, E, 2>, grid, dim3(kThreads), 0, s, a); break;
    case 3: case 4: e = launch_pdl(norm_rope_kernel<T, E, 4>, grid, dim3(kThreads), 0, s, a); break;
    default:
      e = nv <= 8 ? launch_pdl(norm_rope_kernel<T, E, 8>, grid, dim3(kThreads), 0, s, a)
                  : launch_pdl(norm_rope_kernel<T, E, 16>, grid, dim3(kThreads), 0, s, a);
  }
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const NormArgs &a, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.kv) |
                        reinterpret_cast<uintptr_t>(a.gamma_q) |
                        reinterpret_cast<uintptr_t>(a.gamma_kv) |
                        reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.kv_dst);
  // 16-byte chunks where every row starts on 16 bytes
  const bool vec = all % 16 == 0 && a.D % E == 0 && a.q_stride % E == 0 && a.kv_stride % E == 0;
  return vec ? launch_e<T, E>(a, s) : launch_e<T, 2>(a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &n, cudaStream_t s) {
  NormArgs a;
  a.q = n.q;
  a.kv = n.kv;
  a.gamma_q = n.q ? n.gamma_q : nullptr;
  a.gamma_kv = n.kv ? n.gamma_kv : nullptr;
  a.q_out = n.q_out;
  a.kv_dst = n.kv_dst;
  a.q_stride = n.q ? n.q_stride : 0;
  a.kv_stride = n.kv ? n.kv_stride : 0;
  a.pos = n.pos;
  a.slots = n.slots;
  a.cos = n.cos;
  a.sin = n.sin;
  a.n = n.n;
  a.H = n.q ? n.n_heads : 0;
  a.D = n.head_dim;
  a.n_rot = n.n_rot;
  a.max_pos = n.rope_max_pos;
  a.n_dst = n.n_dst;
  a.per = a.H + (n.kv ? 1u : 0u);
  a.rot_q = n.rot_q ? 1u : 0u;
  a.n_rows = (uint64_t)n.n * a.per;
  if (a.n_rows == 0) return cudaSuccess;
  return n.dtype == DS4A_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace ds4a
