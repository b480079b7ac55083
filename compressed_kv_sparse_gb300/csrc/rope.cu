// Rotary positions of whole tokens' heads (ds4a_rope), and the append of keys and values to
// a paged cache with the rotation on the way (ds4a_kv_append), in one kernel: rows are
// the heads of the tokens' queries, keys and values, 1 .. H + 2 K a token.
//
//   (x0, x1) -> (x0 c - x1 s, x0 s + x1 c) for the pairs of the rotated dims; fp32, each
//   product and sum rounded once, then one rounding to the stored type.
//
// A thread owns the same 2 E dims of every row that it takes: for pairs of halves E
// dims and the E dims n_rot / 2 behind them, otherwise two neighbouring chunks, so that both
// members of a pair are in its registers and a chunk is one 16-byte access. A thread takes
// some rows of one token after another, so that a token's coefficients are loaded once for
// four to eight rows, beside the rows themselves. Each element is read once and written once.
//
// Bound by HBM for many rows: 4,096 tokens of 64 heads of 512 dims, bf16 90 us (6.0 TB/s, 0.90 of a
// copy); the append of 8,192 tokens of 64 + 2 x 8 heads of 128 into 8 bits 64 us (5.0 TB/s: the
// conversions' issue slots). A few rows take 2.1 us, the launch and two dependent loads.
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
  uint32_t vec_tab;        // coefficients in fours on 16 bytes
  uint32_t batch, max_blocks, n_blocks;
  uint32_t n, rows;        // tokens, rows per token
  uint32_t items;          // threads per row
  // threads: tok_par tokens x row_par rows x items; a block's slice of a token's rows
  uint32_t tok_par, row_par, slice;
};

// E elements of a row in one access of 2 to 16 bytes.
template <int BYTES>
struct Word {};
template <>
struct Word<16> {
  using type = uint4;
};
template <>
struct Word<8> {
  using type = uint2;
};
template <>
struct Word<4> {
  using type = uint32_t;
};
template <>
struct Word<2> {
  using type = uint16_t;
};
template <>
struct Word<1> {
  using type = uint8_t;
};
template <typename T, int E>
struct alignas(E * sizeof(T)) Vec {
  using W = typename Word<E * sizeof(T)>::type;
  T x[E];
  __device__ __forceinline__ void load(const T *p) { *reinterpret_cast<W *>(x) = *reinterpret_cast<const W *>(p); }
};
template <typename T, int E>
__device__ __forceinline__ void put(T *p, const float (&v)[E]) {
  using W = typename Word<E * sizeof(T)>::type;
  Vec<T, E> o;
#pragma unroll
  for (int i = 0; i < E; ++i) st_elem(o.x, i, v[i]);
  *reinterpret_cast<W *>(p) = *reinterpret_cast<const W *>(o.x);
}
// E codes of values already multiplied by the scale's reciprocal.
template <int E>
__device__ __forceinline__ void put_e4m3(uint8_t *p, const float (&v)[E]) {
  using W = typename Word<E>::type;
  alignas(E) uint8_t c[E];
  if (E == 1) {
    c[0] = (uint8_t)__nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int i = 0; i + 1 < E; i += 2)
      *reinterpret_cast<uint16_t *>(c + i) =
          __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1 < E ? i + 1 : i]), __NV_SATFINITE, __NV_E4M3);
  }
  *reinterpret_cast<W *>(p) = *reinterpret_cast<const W *>(c);
}

// E: elements of a chunk (16 bytes, fewer where rows or the rotated part do not start on
// 16 bytes). F8: the cache holds 8-bit floats. U: rows in flight per thread.
template <typename T, bool F8, int E, int U>
__global__ void __launch_bounds__(kThreads, 2) rope_kernel(RopeKernelArgs a) {
  pdl_wait();
  pdl_trigger();
  const uint32_t sub = threadIdx.x / a.items, j = threadIdx.x % a.items;
  const uint32_t t_sub = sub / a.row_par, r_sub = sub % a.row_par;
  if (t_sub >= a.tok_par) return;
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
  const bool copy_all = a.src[0] != a.q_dst;   // (in place only the rotated dims move)
  const uint32_t row0 = blockIdx.y * a.slice + r_sub, row1 = min(a.rows, (blockIdx.y + 1) * a.slice);
  const uint32_t step = gridDim.x * a.tok_par;
  uint32_t tok = blockIdx.x * a.tok_par + t_sub;
  int32_t ps = tok < a.n ? __ldg(a.pos + tok) : 0, sq = a.seq && tok < a.n ? __ldg(a.seq + tok) : 0;
  for (; tok < a.n; tok += step) {
    // ---- the token's coefficients and place; the next token's position meanwhile
    const uint32_t next = tok + step;   // (n < 2^31)
    const int32_t ps1 = next < a.n ? __ldg(a.pos + next) : 0, sq1 = a.seq && next < a.n ? __ldg(a.seq + next) : 0;
    bool live = ps >= 0 && (a.n_rot == 0 || (uint32_t)ps < a.max_pos), held = false;
    size_t at = 0;   // its row of head 0 in the pools
    if (a.seq) {
      const uint32_t blk = (uint32_t)ps / 256u;
      live = live && (uint32_t)sq < a.batch && blk < a.max_blocks;
      if (live) {
        const uint32_t phys = (uint32_t)__ldg(a.table + (size_t)sq * a.max_blocks + blk);
        held = phys < a.n_blocks;
        at = ((size_t)(held ? phys : 0u) * a.K * 256u + ((uint32_t)ps & 255u)) * a.D;
      }
    }
    float co[E], si[E];   // (inside: E / 2 coefficients of each chunk)
    if (live && turn) {
      const float *c = a.cos + (size_t)ps * (a.n_rot / 2), *s = a.sin + (size_t)ps * (a.n_rot / 2);
      if (a.vec_tab && (E == 8 || (E == 4 && cross))) {   // (four neighbours at once)
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const uint32_t i = cross ? ca + e : e < E / 2 ? ca + e : cb + e - E / 2;
          const bool on = cross || (e < E / 2 ? rota : rotb);
          const float4 f = on ? __ldg(reinterpret_cast<const float4 *>(c + i)) : make_float4(1.f, 1.f, 1.f, 1.f);
          const float4 g = on ? __ldg(reinterpret_cast<const float4 *>(s + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float fv[4] = {f.x, f.y, f.z, f.w}, gv[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (e + k < E) {
              co[e + k] = fv[k];
              si[e + k] = gv[k];
            }
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t i = cross ? ca + e : e < E / 2 ? ca + e : cb + e - E / 2;
          const bool on = cross || (e < E / 2 ? rota : rotb);
          co[e] = on ? __ldg(c + i) : 1.f;
          si[e] = on ? __ldg(s + i) : 0.f;
        }
      }
      if (a.inverse)
#pragma unroll
        for (int e = 0; e < E; ++e) si[e] = -si[e];
    }
    // ---- its rows, U at a time
    for (uint32_t r0 = row0; r0 < row1; r0 += U * a.row_par) {
      Vec<T, E> xa[U], xb[U];
      float sc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t r = r0 + u * a.row_par;
        if (r >= row1) break;
        const uint32_t kind = r < a.H ? 0u : r < a.H + a.K ? 1u : 2u;
        const uint32_t head = kind == 0 ? r : kind == 1 ? r - a.H : r - a.H - a.K;
        const T *src = static_cast<const T *>(a.src[kind]) + tok * a.stride[kind] + (size_t)head * a.D;
        if (da != kNone) xa[u].load(src + da);
        if (db != kNone) xb[u].load(src + db);
        if (F8 && kind) sc[u] = __ldg((kind == 1 ? a.k_scale : a.v_scale) + head);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t r = r0 + u * a.row_par;
        if (r >= row1 || !live) break;
        const uint32_t kind = r < a.H ? 0u : r < a.H + a.K ? 1u : 2u;
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
          T *dst = static_cast<T *>(a.q_dst) + tok * a.q_dst_stride + (size_t)r * a.D;
          if (da != kNone) put<T, E>(dst + da, va);
          if (db != kNone) put<T, E>(dst + db, vb);
        } else {
          const uint32_t head = kind == 1 ? r - a.H : r - a.H - a.K;
          const size_t to = at + (size_t)head * 256u * a.D;
          void *pool = kind == 1 ? a.k_pool : a.v_pool;
          if (F8) {
            const float inv = __frcp_rn(sc[u]);
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
    ps = ps1;
    sq = sq1;
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
  uint32_t e = EV;   // the widest chunk that divides all
  while (e > 1 && (all % (e * sizeof(T)) || sizes % e)) e /= 2;
  const uint32_t nr = a.half ? a.n_rot / (2 * e) : 0;
  // (D - n_rot chunks that no half pairs, two to a thread)
  const uint32_t rest = (a.half ? a.D - a.n_rot : a.D) / e;
  a.items = nr + (rest + 1) / 2;
  if (a.items > kThreads) return cudaErrorInvalidValue;   // (D <= 512 for single elements)
  a.vec_tab = (reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin)) % 16 == 0 && a.n_rot % 8 == 0;
  // Few rows: all at once, a token's over several blocks. Otherwise 4 to 8 rows a thread (in fours),
  // as many tokens at once as fill the block best.
  const uint32_t par = kThreads / a.items, sms = (uint32_t)num_sms();
  a.row_par = par < a.rows ? par : a.rows;
  a.tok_par = par / a.row_par;
  a.slice = a.row_par;
  if ((uint64_t)a.n * a.rows > (uint64_t)par * sms * 4) {
    float best = 0.f;
    for (uint32_t tp = 1; tp <= par; ++tp) {
      const uint32_t rp = par / tp < a.rows ? par / tp : a.rows, turns = (a.rows + rp - 1) / rp;
      if (turns > 8 && tp > 1) break;
      const float used = (float)(rp * tp) / par * a.rows / (rp * ((turns + 3) / 4 * 4));
      if (used > best * 1.01f) {
        best = used;
        a.row_par = rp;
        a.tok_par = tp;
      }
    }
    a.slice = a.rows;
  }
  const uint32_t toks = (a.n + a.tok_par - 1) / a.tok_par;
  const dim3 grid(toks < sms * 4 ? toks : sms * 4, (a.rows + a.slice - 1) / a.slice);
  auto *k = e == 8   ? rope_kernel<T, F8, EV, 4>
            : e == 4 ? rope_kernel<T, F8, 4, 4>
            : e == 2 ? rope_kernel<T, F8, 2, 4>
                     : rope_kernel<T, F8, 1, 4>;
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
  a.n = r.n;
  if (a.n == 0 || a.rows == 0) return cudaSuccess;
  const bool f8 = r.k && r.kv_dtype == DS4A_E4M3;
  if (r.dtype == DS4A_BF16)
    return f8 ? launch_rows<__nv_bfloat16, true>(a, s) : launch_rows<__nv_bfloat16, false>(a, s);
  return f8 ? launch_rows<float, true>(a, s) : launch_rows<float, false>(a, s);
}

}  // namespace ds4a
