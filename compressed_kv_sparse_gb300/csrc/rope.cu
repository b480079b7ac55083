// Rotary positions of whole tokens' heads (ds4a_rope), and the append of keys and values to
// a paged cache with the rotation on the way (ds4a_kv_append), in one kernel: rows are
// the heads of the tokens' queries, keys and values, 1 .. H + 2 K a token.
//
//   (x0, x1) -> (x0 c - x1 s, x0 s + x1 c) for the pairs of the rotated dims; fp32, each
//   product and sum rounded once, then one rounding to the stored type.
//
// A thread owns the same 2 E dims of every row that it takes: for pairs of halves E
// dims and the E dims n_rot / 2 behind them, otherwise two neighbouring chunks, so that both
// members of a pair are in its registers and a chunk is one 16-byte access. It keeps the
// coefficients while the token stays the same. Each element is read once and written once.
#include <cuda_fp8.h>

#include "common.cuh"

namespace ds4a {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kNone = 0xffffffffu;

struct RopeKernelArgs {
  const void *src[3];      // queries (or x), keys, values
  uint64_t stride[3];      // elements from token to token
  void *q_dst;
  uint64_t q_dst_stride;
  void *k_pool, *v_pool;
  const float *k_scale, *v_scale;
  const int32_t *pos, *seq, *table;
  const float *cos, *sin;
  uint32_t H, K, D, rot_at, n_rot, max_pos, half, inverse;
  uint32_t batch, max_blocks, n_blocks;
  uint32_t rows;           // rows per token
  uint32_t items;          // threads per row
  uint32_t rpb;            // rows per pass of the block
  uint32_t d_tok, d_row;   // rpb / rows, rpb % rows
  uint64_t total;          // n * rows
  uint64_t passes;         // ceil(total / rpb)
};

template <typename T, int E>
struct Vec {
  alignas(E * sizeof(T) == 16 ? 16 : sizeof(T)) T x[E];
  __device__ __forceinline__ void load(const T *p) {
    if (E * sizeof(T) == 16) {
      *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = p[i];
    }
  }
};
template <typename T, int E>
__device__ __forceinline__ void put(T *p, const float (&v)[E]) {
  Vec<T, E> o;
#pragma unroll
  for (int i = 0; i < E; ++i) st_elem(o.x, i, v[i]);
  if (E * sizeof(T) == 16) {
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(o.x);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = o.x[i];
  }
}
// E codes of values already multiplied by the scale's reciprocal.
template <int E>
__device__ __forceinline__ void put_e4m3(uint8_t *p, const float (&v)[E]) {
  if (E == 1) {
    *p = (uint8_t)__nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint16_t h[E / 2 ? E / 2 : 1];
#pragma unroll
    for (int i = 0; i + 1 < E; i += 2)
      h[i / 2] = __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1 < E ? i + 1 : i]), __NV_SATFINITE, __NV_E4M3);
    if (E == 8)
      *reinterpret_cast<uint2 *>(p) = make_uint2(h[0] | (uint32_t)h[E > 2 ? 1 : 0] << 16,
                                                 h[E > 4 ? 2 : 0] | (uint32_t)h[E > 6 ? 3 : 0] << 16);
    else
      *reinterpret_cast<uint32_t *>(p) = h[0] | (uint32_t)h[E > 2 ? 1 : 0] << 16;
  }
}

// E: elements of a chunk (16 bytes; 1 where rows or the rotated part do not start on
// 16 bytes). F8: the cache holds 8-bit floats. U: rows in flight per thread.
template <typename T, bool F8, int E, int U>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeKernelArgs a) {
  pdl_wait();
  pdl_trigger();
  const uint32_t sub = threadIdx.x / a.items, j = threadIdx.x % a.items;
  if (sub >= a.rpb) return;
  // ---- the thread's dims: chunks at da and db (kNone: none), which of them are rotated and how:
  // cross: pairs (a[e], b[e]) with coefficients ca + e; else pairs inside each chunk
  uint32_t da, db, ca = 0, cb = 0;
  bool cross = false, rota = false, rotb = false;
  const uint32_t nr = a.half ? a.n_rot / (2 * E) : 0;
  if (j < nr) {
    da = a.rot_at + E * j;
    db = da + a.n_rot / 2;
    ca = E * j;
    cross = true;
  } else {
    const uint32_t u = 2 * (j - nr);
    da = E * u;
    db = da + E;
    if (a.half) {   // (the rotated dims are other threads')
      if (da >= a.rot_at) da += a.n_rot;
      if (db >= a.rot_at) db += a.n_rot;
    } else {
      const uint32_t end = a.rot_at + a.n_rot;
      rota = da >= a.rot_at && da < end;
      rotb = db >= a.rot_at && db < end;
      ca = rota ? (da - a.rot_at) / 2 : 0;
      cb = rotb ? (db - a.rot_at) / 2 : 0;
      if (E == 1) {   // (a pair is a and b)
        cross = rota;
        rota = rotb = false;
      }
    }
    if (da >= a.D) da = kNone;
    if (db >= a.D) db = kNone;
  }
  const bool turn = cross || rota || rotb;
  float co[E], si[E];
  const uint64_t p0 = a.passes * blockIdx.x / gridDim.x, p1 = a.passes * (blockIdx.x + 1) / gridDim.x;
  uint64_t row = p0 * a.rpb + sub;
  uint32_t tok = (uint32_t)(row / a.rows), rr = (uint32_t)(row % a.rows);
  uint32_t have = kNone;                 // the token of the coefficients
  bool live = false, held = false;       // ... its position is in range, its block there
  size_t at = 0;                         // ... its row of head 0 in the pools
  const bool copy_all = a.src[0] != a.q_dst;   // (in place only the rotated dims move)
  for (uint64_t p = p0; p < p1; p += U) {
    Vec<T, E> xa[U], xb[U];
    uint32_t tk[U], rw[U];
    int32_t ps[U], sq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = p + u < p1 && row < a.total;
      tk[u] = in ? tok : kNone;
      rw[u] = rr;
      if (in) {
        const uint32_t kind = rr < a.H ? 0u : rr < a.H + a.K ? 1u : 2u;
        const uint32_t head = kind == 0 ? rr : kind == 1 ? rr - a.H : rr - a.H - a.K;
        const T *src = static_cast<const T *>(a.src[kind]) + tok * a.stride[kind] + (size_t)head * a.D;
        if (da != kNone) xa[u].load(src + da);
        if (db != kNone) xb[u].load(src + db);
        ps[u] = __ldg(a.pos + tok);
        sq[u] = a.seq ? __ldg(a.seq + tok) : 0;
      }
      row += a.rpb;
      tok += a.d_tok;
      rr += a.d_row;
      if (rr >= a.rows) {
        rr -= a.rows;
        ++tok;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (tk[u] == kNone) continue;
      if (tk[u] != have) {
        have = tk[u];
        const int32_t ps_ = ps[u];
        live = ps_ >= 0 && (a.n_rot == 0 || (uint32_t)ps_ < a.max_pos);
        held = false;
        if (a.seq) {
          const uint32_t blk = (uint32_t)ps_ / 256u;
          live = live && (uint32_t)sq[u] < a.batch && blk < a.max_blocks;
          if (live) {
            const uint32_t phys = (uint32_t)__ldg(a.table + (size_t)sq[u] * a.max_blocks + blk);
            held = phys < a.n_blocks;
            at = ((size_t)(held ? phys : 0u) * a.K * 256u + ((uint32_t)ps_ & 255u)) * a.D;
          }
        }
        if (live && turn) {
          const float *c = a.cos + (size_t)ps_ * (a.n_rot / 2), *s = a.sin + (size_t)ps_ * (a.n_rot / 2);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            // (inside: E / 2 coefficients of each chunk)
            const uint32_t i = cross ? ca + e : e < E / 2 ? ca + e : cb + e - E / 2;
            const bool on = cross || (e < E / 2 ? rota : rotb);
            co[e] = on ? __ldg(c + i) : 1.f;
            si[e] = on ? __ldg(s + i) : 0.f;
            if (a.inverse) si[e] = -si[e];
          }
        }
      }
      if (!live) continue;
      const uint32_t r = rw[u], kind = r < a.H ? 0u : r < a.H + a.K ? 1u : 2u;
      if (kind && !held) continue;
      if (kind == 0 && !copy_all && !turn) continue;
      float va[E], vb[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        va[e] = da != kNone ? ld_f32(xa[u].x, e) : 0.f;
        vb[e] = db != kNone ? ld_f32(xb[u].x, e) : 0.f;
      }
      if (kind != 2) {
        if (cross) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float x0 = va[e], x1 = vb[e];
            va[e] = __fsub_rn(__fmul_rn(x0, co[e]), __fmul_rn(x1, si[e]));
            vb[e] = __fadd_rn(__fmul_rn(x0, si[e]), __fmul_rn(x1, co[e]));
          }
        } else if (E > 1) {
#pragma unroll
          for (int e = 0; e + 1 < E; e += 2) {
            const int h = e / 2;
            if (rota) {
              const float x0 = va[e], x1 = va[e + (E > 1)];
              va[e] = __fsub_rn(__fmul_rn(x0, co[h]), __fmul_rn(x1, si[h]));
              va[e + (E > 1)] = __fadd_rn(__fmul_rn(x0, si[h]), __fmul_rn(x1, co[h]));
            }
            if (rotb) {
              const float x0 = vb[e], x1 = vb[e + (E > 1)], c = co[E / 2 + h], s = si[E / 2 + h];
              vb[e] = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
              vb[e + (E > 1)] = __fadd_rn(__fmul_rn(x0, s), __fmul_rn(x1, c));
            }
          }
        }
      }
      if (kind == 0) {
        T *dst = static_cast<T *>(a.q_dst) + have * a.q_dst_stride + (size_t)r * a.D;
        if (da != kNone) put<T, E>(dst + da, va);
        if (db != kNone) put<T, E>(dst + db, vb);
      } else {
        const uint32_t head = kind == 1 ? r - a.H : r - a.H - a.K;
        const size_t to = at + (size_t)head * 256u * a.D;
        void *pool = kind == 1 ? a.k_pool : a.v_pool;
        if (F8) {
          const float inv = __frcp_rn(__ldg((kind == 1 ? a.k_scale : a.v_scale) + head));
#pragma unroll
          for (int e = 0; e < E; ++e) {
            va[e] = __fmul_rn(va[e], inv);
            vb[e] = __fmul_rn(vb[e], inv);
          }
          uint8_t *dst = static_cast<uint8_t *>(pool) + to;
          if (da != kNone) put_e4m3<E>(dst + da, va);
          if (db != kNone) put_e4m3<E>(dst + db, vb);
        } else {
          T *dst = static_cast<T *>(pool) + to;
          if (da != kNone) put<T, E>(dst + da, va);
          if (db != kNone) put<T, E>(dst + db, vb);
        }
      }
    }
  }
}

template <typename T, bool F8>
cudaError_t launch_rows(RopeKernelArgs a, cudaStream_t s) {
  constexpr int EV = 16 / sizeof(T);
  uintptr_t all = 0;
  uint64_t sizes = a.D | a.rot_at | (a.half ? a.n_rot / 2 : a.n_rot);
  if (a.H) {
    all |= reinterpret_cast<uintptr_t>(a.src[0]) | reinterpret_cast<uintptr_t>(a.q_dst);
    sizes |= a.stride[0] | a.q_dst_stride;
  }
  if (a.K) {
    all |= reinterpret_cast<uintptr_t>(a.src[1]) | reinterpret_cast<uintptr_t>(a.src[2]);
    sizes |= a.stride[1] | a.stride[2];
  }
  const bool vec = all % 16 == 0 && sizes % EV == 0;
  const uint32_t e = vec ? EV : 1;
  const uint32_t nr = a.half ? a.n_rot / (2 * e) : 0;
  // (D - n_rot chunks that no half pairs, two to a thread)
  const uint32_t rest = (a.half ? a.D - a.n_rot : a.D) / e;
  a.items = nr + (rest + 1) / 2;
  if (a.items > kThreads) return cudaErrorInvalidValue;   // (D <= 512 for single elements)
  a.rpb = kThreads / a.items;
  a.d_tok = a.rpb / a.rows;
  a.d_row = a.rpb % a.rows;
  a.passes = (a.total + a.rpb - 1) / a.rpb;
  const uint64_t most = (uint64_t)num_sms() * 4;
  const dim3 grid((uint32_t)(a.passes < most ? a.passes : most));
  auto *k = vec ? rope_kernel<T, F8, EV, 4> : rope_kernel<T, F8, 1, 4>;
  const cudaError_t err = launch_pdl(k, grid, dim3(kThreads), 0, s, a);
  if (err != cudaSuccess) return err;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &r, cudaStream_t s) {
  RopeKernelArgs a = {};
  a.src[0] = r.x;
  a.stride[0] = r.x_stride;
  a.q_dst = r.y;
  a.q_dst_stride = r.y_stride;
  a.src[1] = r.k;
  a.stride[1] = r.k_stride;
  a.src[2] = r.v;
  a.stride[2] = r.v_stride;
  a.H = r.x ? r.n_heads : 0;
  a.K = r.k ? r.n_kv : 0;
  a.k_pool = r.k_pool;
  a.v_pool = r.v_pool;
  a.k_scale = r.k_scale;
  a.v_scale = r.v_scale;
  a.pos = r.pos;
  a.seq = r.seq;
  a.table = r.table;
  a.cos = r.cos;
  a.sin = r.sin;
  a.D = r.head_dim;
  a.rot_at = r.n_rot ? r.rot_at : 0;
  a.n_rot = r.n_rot;
  a.max_pos = r.max_pos;
  a.half = r.half;
  a.inverse = r.inverse;
  a.batch = r.batch;
  a.max_blocks = r.max_blocks;
  a.n_blocks = r.n_blocks;
  a.rows = a.H + 2 * a.K;
  a.total = (uint64_t)r.n * a.rows;
  if (a.total == 0) return cudaSuccess;
  const bool f8 = r.k && r.kv_dtype == DS4A_E4M3;
  if (r.dtype == DS4A_BF16)
    return f8 ? launch_rows<__nv_bfloat16, true>(a, s) : launch_rows<__nv_bfloat16, false>(a, s);
  return f8 ? launch_rows<float, true>(a, s) : launch_rows<float, false>(a, s);
}

}  // namespace ds4a
