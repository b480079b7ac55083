// Compressed attention rows to and from their 4-bit form (ds4a_pack_rows,
// ds4a_unpack_rows): rows the caller has in the cache's type, a restored
// prefix for instance, into a cache that holds 4-bit rows, and back.
//
// Eight lanes per row, as the layout has it (fp4rows.cuh): a lane reads 8 dims of
// every 64-dim block (a warp reads 128 contiguous bytes of each of four rows),
// takes the largest magnitude of 16 dims with its neighbour, and writes its
// record as 16-byte vectors. One pass, no shared memory; bound by HBM.
#include "common.cuh"
#include "fp4rows.cuh"

namespace ds4a {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxBlocks = 16;                 // 64-dim blocks of a row (D <= 1024)
constexpr uint32_t kMaxWords = kMaxBlocks + 4;      // record words (16 + 2, padded)

struct RowsArgs {
  uint8_t *packed;        // the pool
  uint64_t n_pool;        // rows in it
  void *rows;             // [n][D]
  const int32_t *slots;   // [n] or NULL
  uint32_t n, D, n_rot;
  Fp4Layout L;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  if (VEC) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int h = 0; h < 8 / E; ++h) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p + h * E);
      const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
      for (int i = 0; i < E; ++i) v[h * E + i] = ld_f32(e, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ld_f32(p, i);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
  if (VEC) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int h = 0; h < 8 / E; ++h) {
      uint4 u;
      T *e = reinterpret_cast<T *>(&u);
#pragma unroll
      for (int i = 0; i < E; ++i) st_elem(e, i, v[h * E + i]);
      *reinterpret_cast<uint4 *>(p + h * E) = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) st_elem(p, i, v[i]);
  }
}

// Row of the pool that entry i goes to; false: none (skipped).
__device__ __forceinline__ bool pool_row(const RowsArgs &a, uint32_t i, uint64_t &row) {
  if (i >= a.n) return false;
  const int64_t s = a.slots ? (int64_t)__ldg(a.slots + i) : (int64_t)i;
  row = (uint64_t)s;
  return s >= 0 && row < a.n_pool;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) rows_pack_kernel(RowsArgs a) {
  const uint32_t i = blockIdx.x * (kThreads / 8) + threadIdx.x / 8, j = threadIdx.x & 7;
  uint64_t row;
  const bool live = pool_row(a, i, row);   // (the same for a row's eight lanes)
  const T *src = static_cast<const T *>(a.rows) + (size_t)(live ? i : 0) * a.D;
  uint32_t rec[kMaxWords];
#pragma unroll
  for (uint32_t w = 0; w < kMaxWords; ++w) rec[w] = 0;
  uint32_t own[kMaxBlocks / 4] = {0, 0, 0, 0};   // scale bytes, four per word, of every block
#pragma unroll
  for (uint32_t kb = 0; kb < kMaxBlocks; ++kb) {
    if (kb >= a.L.nb) break;
    const uint32_t d = 64 * kb + 8 * j;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live && d < a.L.nope) load8<T, VEC>(src + d, v);
    float am = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) am = fp4_amax(am, v[e]);
    am = fp4_amax(am, __shfl_xor_sync(0xffffffffu, am, 1));
    const uint32_t sb = fp4_scale_byte(am);
    rec[kb] = fp4_encode(v, sb);
    own[kb / 4] |= sb << (8 * (kb % 4));
  }
  if (!live) return;
  // this lane's scale words: blocks 4 ns (j % 2) + 4 s ..
  const uint32_t first = (j & 1) * a.L.ns;
#pragma unroll
  for (uint32_t w = 0; w < kMaxWords; ++w) {
    const uint32_t s = w - a.L.nb;
    if (w >= a.L.nb && s < a.L.ns) {
      uint32_t x = 0;
#pragma unroll
      for (uint32_t q = 0; q < kMaxBlocks / 4; ++q)
        if (q == first + s) x = own[q];
      rec[w] = x;
    }
  }
  uint8_t *dst = a.packed + row * a.L.row_bytes;
#pragma unroll
  for (uint32_t g = 0; g < kMaxWords / 4; ++g)
    if (4 * g < a.L.R)
      *reinterpret_cast<uint4 *>(dst + 128 * g + 16 * j) =
          make_uint4(rec[4 * g], rec[4 * g + 1], rec[4 * g + 2], rec[4 * g + 3]);
  T *tail = reinterpret_cast<T *>(dst + a.L.tail);
  if (VEC) {
    constexpr uint32_t E = 16 / sizeof(T);
    for (uint32_t c = j; c < a.n_rot / E; c += 8)
      reinterpret_cast<uint4 *>(tail)[c] = reinterpret_cast<const uint4 *>(src + a.L.nope)[c];
  } else {
    for (uint32_t c = j; c < a.n_rot; c += 8) tail[c] = src[a.L.nope + c];
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) rows_unpack_kernel(RowsArgs a) {
  const uint32_t i = blockIdx.x * (kThreads / 8) + threadIdx.x / 8, j = threadIdx.x & 7;
  uint64_t row;
  if (!pool_row(a, i, row)) return;
  const uint8_t *src = a.packed + row * a.L.row_bytes;
  T *dst = static_cast<T *>(a.rows) + (size_t)i * a.D;
  for (uint32_t kb = 0; kb < a.L.nb; ++kb) {
    const uint32_t d = 64 * kb + 8 * j;
    if (d >= a.L.nope) break;
    float v[8];
    fp4_decode(*reinterpret_cast<const uint32_t *>(src + fp4_word_at(kb, j)),
               src[fp4_scale_at(a.L, kb, j / 2)], v);
    store8<T, VEC>(dst + d, v);
  }
  const T *tail = reinterpret_cast<const T *>(src + a.L.tail);
  if (VEC) {
    constexpr uint32_t E = 16 / sizeof(T);
    for (uint32_t c = j; c < a.n_rot / E; c += 8)
      reinterpret_cast<uint4 *>(dst + a.L.nope)[c] = reinterpret_cast<const uint4 *>(tail)[c];
  } else {
    for (uint32_t c = j; c < a.n_rot; c += 8) dst[a.L.nope + c] = tail[c];
  }
}

template <typename T>
cudaError_t launch_t(bool pack, const RowsArgs &a, cudaStream_t s) {
  // 16-byte vectors where every row and its tail start on 16 bytes
  const bool vec = reinterpret_cast<uintptr_t>(a.rows) % 16 == 0 &&
                   a.D * sizeof(T) % 16 == 0 && a.n_rot * sizeof(T) % 16 == 0;
  auto *k = pack ? (vec ? rows_pack_kernel<T, true> : rows_pack_kernel<T, false>)
                 : (vec ? rows_unpack_kernel<T, true> : rows_unpack_kernel<T, false>);
  const uint32_t per = kThreads / 8;
  k<<<(a.n + per - 1) / per, kThreads, 0, s>>>(a);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_fp4(bool pack, int dtype, void *packed, uint64_t n_pool, void *rows,
                            const int32_t *slots, uint32_t n, uint32_t D, uint32_t n_rot,
                            cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const uint32_t es = dtype == DS4A_BF16 ? 2 : 4;
  const RowsArgs a{static_cast<uint8_t *>(packed), n_pool, rows, slots, n, D, n_rot,
                   fp4_layout(D, n_rot, es)};
  return dtype == DS4A_BF16 ? launch_t<__nv_bfloat16>(pack, a, s) : launch_t<float>(pack, a, s);
}

}  // namespace ds4a
