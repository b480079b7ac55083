// RMSNorm of every query head and of the shared K = V row of each token, the
// tail rotation and the insert of the row into the raw window, in one pass
// (vLLM DeepSeek V4 page, section "GPU 計算飽和": fused Q norm + KV RoPE + K
// insert; "【#3】ds4.c を読み解く" §8 tail-only RoPE).
//
// One warp owns one row (a head of a token, or the token's K = V row): the row
// stays in registers between the sum of squares and the scaled, rotated store, so
// each element is read once and written once. Bound by HBM at a chunk's size (4096
// tokens of 64 heads x 512 in bf16: 91 us, 0.89 of the measured copy rate), by the
// launch and two dependent look-ups at a decode step's (8 tokens: 2.7 us).
#include "common.cuh"

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
};

// E consecutive elements of a row (E * sizeof(T) = 16, or 2 elements one by one
// where the rows are not 16-byte aligned).
template <typename T, int E>
struct Chunk {
  alignas(E * sizeof(T) == 16 ? 16 : sizeof(T)) T x[E];
  __device__ __forceinline__ void load(const T *p) {
    if (E * sizeof(T) == 16) {
      *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = p[i];
    }
  }
  __device__ __forceinline__ float get(int i) const { return ld_f32(x, i); }
};
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

// Warp w of W takes rows total w / W .. total (w + 1) / W - 1 of the n tokens' rows
// (a token's heads, then its K = V row), so that its loads follow one another in
// memory, the token and its position change rarely, and PF rows are in flight
// per warp. (For that chunk one block per token measured 163 us and one warp per row in
// a grid-wide stride 139 us: the look-ups of a short-lived warp are not hidden.)
// NV: chunks of E elements per lane (D <= 32 E NV). LAST: the rotated tail is whole
// chunks of each lane's last one (512 dims with a 64-dim tail, for instance): a lane then
// keeps its coefficients in registers for all rows of a token (looked up pair by pair
// for every row: 160 us). Three blocks of 80 registers and three rows ahead measured,
// side by side, 92 us, four of 64 and two rows 94, five of 48 and two rows 146.
template <typename T, int E, int NV, bool LAST>
__global__ void __launch_bounds__(kThreads, NV <= 2 ? 3 : 1) norm_rope_kernel(NormArgs a) {
  constexpr int PF = NV <= 2 ? 3 : NV <= 4 ? 2 : 1;
  pdl_wait();
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t total = (uint64_t)a.n * a.per, W = (uint64_t)gridDim.x * (kThreads / 32);
  const uint64_t w = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const uint64_t r0 = total * w / W, r1 = total * (w + 1) / W;
  const uint32_t n_rows = (uint32_t)(r1 - r0), nope = a.D - a.n_rot;
  Chunk<T, E> nx[PF][NV];   // the rows to come as they are stored
  uint32_t ltok = (uint32_t)(r0 / a.per), lh = (uint32_t)(r0 % a.per);   // the row loaded next
  uint32_t tok = ltok, h = lh;                                           // the row worked on
  auto load = [&](Chunk<T, E> (&x)[NV]) {
    const T *src = lh < a.H ? static_cast<const T *>(a.q) + ltok * a.q_stride + (size_t)lh * a.D
                            : static_cast<const T *>(a.kv) + ltok * a.kv_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = E * (lane + 32 * i);
      if (c < a.D) x[i].load(src + c);
    }
    if (++lh == a.per) {
      lh = 0;
      ++ltok;
    }
  };
#pragma unroll
  for (int k = 0; k < PF; ++k)
    if ((uint32_t)k < n_rows) load(nx[k]);
  int32_t p = n_rows ? __ldg(a.pos + tok) : -1;
  float co_r[E / 2], si_r[E / 2];   // LAST: this lane's coefficients (1, 0 outside the tail)
  const uint32_t c_last = E * (lane + 32 * (NV - 1));
  auto coefs = [&]() {
    const bool in = LAST && c_last >= nope && c_last < a.D && p >= 0 && (uint32_t)p < a.max_pos;
    const size_t at = in ? (size_t)p * (a.n_rot / 2) + (c_last - nope) / 2 : 0;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      co_r[e] = in ? __ldg(a.cos + at + e) : 1.f;
      si_r[e] = in ? __ldg(a.sin + at + e) : 0.f;
    }
  };
  coefs();
  const float inv_d = 1.f / (float)a.D;
  for (uint32_t base = 0; base < n_rows; base += PF) {
#pragma unroll
    for (int k = 0; k < PF; ++k) {
      if (base + k >= n_rows) break;
      float v[NV][E];
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = E * (lane + 32 * i) < a.D;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[i][e] = in ? nx[k][i].get(e) : 0.f;
          ss = fmaf(v[i][e], v[i][e], ss);
        }
      }
      if (base + k + PF < n_rows) load(nx[k]);
      const bool is_q = h < a.H, rot = !is_q || a.rot_q;
      // (a token whose position is out of range is left alone, as is a dropped K = V row)
      bool live = p >= 0 && (uint32_t)p < a.max_pos;
      int64_t slot = tok;
      if (!is_q && a.slots) slot = __ldg(a.slots + tok);
      live = live && (is_q || (slot >= 0 && slot < (int64_t)a.n_dst));
      ss = warp_sum(ss);
      const float inv = rsqrtf(fmaf(ss, inv_d, kRmsEps));
      const T *gamma = static_cast<const T *>(is_q ? a.gamma_q : a.gamma_kv);
      T *dst = is_q ? static_cast<T *>(a.q_out) + ((size_t)tok * a.H + h) * a.D
                    : static_cast<T *>(a.kv_dst) + (size_t)(live ? slot : 0) * a.D;
      const float *co = a.cos + (size_t)(live ? p : 0) * (a.n_rot / 2);
      const float *si = a.sin + (size_t)(live ? p : 0) * (a.n_rot / 2);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = E * (lane + 32 * i);
        if (!live || c >= a.D) continue;
        if (LAST) {
          Chunk<T, E> g;   // (no gain: ones)
#pragma unroll
          for (int e = 0; e < E; ++e) st_elem(g.x, e, 1.f);
          if (gamma) g.load(gamma + c);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = v[i][e] * inv * g.get(e);
          if (i == NV - 1 && rot) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float x0 = v[i][e], x1 = v[i][e + 1], cs = co_r[e / 2], sn = si_r[e / 2];
              if (c >= nope) {
                v[i][e] = x0 * cs - x1 * sn;
                v[i][e + 1] = x0 * sn + x1 * cs;
              }
            }
          }
          store_e<T, E>(dst + c, v[i]);
          continue;
        }
        Chunk<T, E> g;
        if (gamma) g.load(gamma + c);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          float x0 = v[i][e] * inv, x1 = v[i][e + 1] * inv;
          if (gamma) {
            x0 *= g.get(e);
            x1 *= g.get(e + 1);
          }
          if (rot && c + e >= nope) {
            const uint32_t f = (c + e - nope) / 2;
            const float cs = __ldg(co + f), sn = __ldg(si + f);
            const float y0 = x0 * cs - x1 * sn, y1 = x0 * sn + x1 * cs;
            x0 = y0;
            x1 = y1;
          }
          v[i][e] = x0;
          v[i][e + 1] = x1;
        }
        store_e<T, E>(dst + c, v[i]);
      }
      if (++h == a.per) {
        h = 0;
        ++tok;
        if (base + k + 1 < n_rows) {
          p = __ldg(a.pos + tok);
          coefs();
        }
      }
    }
  }
}

template <typename T, int E>
cudaError_t launch_e(const NormArgs &a, cudaStream_t s) {
  // one row per warp while the GPU has room for that, else a full GPU of warps
  const uint64_t total = (uint64_t)a.n * a.per, rows_per_block = kThreads / 32;
  const uint64_t blocks = (total + rows_per_block - 1) / rows_per_block;
  const uint64_t most = (uint64_t)num_sms() * 3;
  const dim3 grid((uint32_t)(blocks < most ? blocks : most));
  const uint32_t nv = (a.D + 32 * E - 1) / (32 * E);
  constexpr int kNvMax = 1024 / (32 * E);   // D <= 1024
  const uint32_t nope = a.D - a.n_rot;
  if (E * sizeof(T) == 16 && nope % E == 0) {
    void (*last)(NormArgs) = nullptr;
    if (nv == 1) last = norm_rope_kernel<T, E, 1, true>;
    if (nv == 2 && nope >= 32 * E) last = norm_rope_kernel<T, E, 2, true>;
    if (nv == 4 && nope >= 96 * E) last = norm_rope_kernel<T, E, 4, true>;
    if (last) {
      const cudaError_t e = launch_pdl(last, grid, dim3(kThreads), 0, s, a);
      if (e != cudaSuccess) return e;
      note_launches(1);
      return cudaGetLastError();
    }
  }
  auto *k = nv <= 1   ? norm_rope_kernel<T, E, 1, false>
            : nv <= 2 ? norm_rope_kernel<T, E, 2, false>
            : nv <= 4 ? norm_rope_kernel<T, E, 4, false>
                      : norm_rope_kernel<T, E, kNvMax, false>;
  cudaError_t e = launch_pdl(k, grid, dim3(kThreads), 0, s, a);
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
  if (a.n == 0 || a.per == 0) return cudaSuccess;
  return n.dtype == DS4A_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace ds4a
