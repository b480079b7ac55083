// Compressed attention rows to and from their 4-bit form (ds4a_pack_rows,
// ds4a_unpack_rows): rows the caller has in the cache's type, a restored
// prefix for instance, into a cache that holds 4-bit rows, and back.
//
// Eight lanes per row, as the layout has it (fp4rows.cuh): a lane reads 8 dims of
// every 64-dim block (a warp reads 128 contiguous bytes of each of four rows),
// takes the largest magnitude of 16 dims with its neighbour, and writes its
// record as 16-byte vectors. One pass, no shared memory; bound by HBM (262,144 rows of
// 512 bf16 dims into random places: 64 us, 0.86 of the measured copy rate; back: 57 us, 0.95).
// Programmatic launches (1,024 rows packed and read back: 8.8 us, plain ones 9.6).
#include "common.cuh"
#include "fp4rows.cuh"

namespace ds4a {
namespace {

constexpr int kThreads = 256;

struct RowsArgs {
  uint8_t *packed;        // the pool
  uint64_t n_pool;        // rows in it
  void *rows;             // [n][D]
  const int32_t *slots;   // [n] or NULL
  uint32_t n, D, n_rot;
  Fp4Layout L;
};

template <typename T, bool VEC>
__device__ __forceinline__ void copy8(const T *p, T (&v)[8]) {
  if (VEC) {
#pragma unroll
    for (uint32_t h = 0; h < 8 * sizeof(T) / 16; ++h)
      reinterpret_cast<uint4 *>(v)[h] = reinterpret_cast<const uint4 *>(p)[h];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
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

// NB: 64-dim blocks that the code has room for (8: 512-wide rows and narrower, all
// loads of a row in flight at once; 16: any). FLASH: 512 dims with a 64-dim tail, the
// layout known at compile time (262,144 bf16 rows: packed in 64 us against 72; reading
// back is as fast without).
template <typename T, bool VEC, int NB, bool FLASH>
__global__ void __launch_bounds__(kThreads) rows_pack_kernel(RowsArgs a) {
  const uint32_t D = FLASH ? 512u : a.D, n_rot = FLASH ? 64u : a.n_rot;
  const Fp4Layout L = FLASH ? fp4_layout(512, 64, sizeof(T)) : a.L;
  constexpr uint32_t NW = NB + 4;   // record words
  const uint32_t i = blockIdx.x * (kThreads / 8) + threadIdx.x / 8, j = threadIdx.x & 7;
  pdl_wait();
  uint64_t row;
  const bool live = pool_row(a, i, row);   // (the same for a row's eight lanes)
  const T *src = static_cast<const T *>(a.rows) + (size_t)(live ? i : 0) * D;
  alignas(16) T raw[NB][8];
#pragma unroll
  for (uint32_t kb = 0; kb < NB; ++kb) {
    const uint32_t d = 64 * kb + 8 * j;
    if (live && d < L.nope) copy8<T, VEC>(src + d, raw[kb]);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) st_elem(raw[kb], e, 0.f);
  }
  constexpr uint32_t E = 16 / sizeof(T);
  uint4 tail0 = make_uint4(0u, 0u, 0u, 0u);
  if (VEC && live && j < n_rot / E) tail0 = reinterpret_cast<const uint4 *>(src + L.nope)[j];
  uint32_t rec[NW];
#pragma unroll
  for (uint32_t w = 0; w < NW; ++w) rec[w] = 0;
  uint32_t own[NB / 4];   // scale bytes, four per word, of every block
#pragma unroll
  for (uint32_t q = 0; q < NB / 4; ++q) own[q] = 0;
#pragma unroll
  for (uint32_t kb = 0; kb < NB; ++kb) {
    float v[8], am = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = ld_f32(raw[kb], e);
      am = fp4_amax(am, v[e]);
    }
    am = fp4_amax(am, __shfl_xor_sync(0xffffffffu, am, 1));
    const uint32_t sb = fp4_scale_byte(am);
    if (kb < L.nb) {
      rec[kb] = fp4_encode(v, sb);
      own[kb / 4] |= sb << (8 * (kb % 4));
    }
  }
  if (!live) return;
  // this lane's scale words: blocks 4 ns (j % 2) + 4 s ..
  const uint32_t first = (j & 1) * L.ns;
#pragma unroll
  for (uint32_t w = 0; w < NW; ++w) {
    const uint32_t s = w - L.nb;
    if (w >= L.nb && s < L.ns) {
      uint32_t x = 0;
#pragma unroll
      for (uint32_t q = 0; q < NB / 4; ++q)
        if (q == first + s) x = own[q];
      rec[w] = x;
    }
  }
  uint8_t *dst = a.packed + row * L.row_bytes;
#pragma unroll
  for (uint32_t g = 0; g < NW / 4; ++g)
    if (4 * g < L.R)
      *reinterpret_cast<uint4 *>(dst + 128 * g + 16 * j) =
          make_uint4(rec[4 * g], rec[4 * g + 1], rec[4 * g + 2], rec[4 * g + 3]);
  T *tail = reinterpret_cast<T *>(dst + L.tail);
  if (VEC) {
    if (j < n_rot / E) reinterpret_cast<uint4 *>(tail)[j] = tail0;
    for (uint32_t c = j + 8; c < n_rot / E; c += 8)
      reinterpret_cast<uint4 *>(tail)[c] = reinterpret_cast<const uint4 *>(src + L.nope)[c];
  } else {
    for (uint32_t c = j; c < n_rot; c += 8) tail[c] = src[L.nope + c];
  }
}

template <typename T, bool VEC, int NB>
__global__ void __launch_bounds__(kThreads) rows_unpack_kernel(RowsArgs a) {
  const uint32_t D = a.D, n_rot = a.n_rot;
  const Fp4Layout &L = a.L;
  constexpr uint32_t NW = NB + 4;
  const uint32_t i = blockIdx.x * (kThreads / 8) + threadIdx.x / 8, j = threadIdx.x & 7;
  pdl_wait();
  uint64_t row;
  const bool live = pool_row(a, i, row);
  const uint8_t *src = a.packed + (live ? row : 0) * L.row_bytes;
  T *dst = static_cast<T *>(a.rows) + (size_t)(live ? i : 0) * D;
  constexpr uint32_t E = 16 / sizeof(T);
  // (vectors by 4 words per lane; the pool's row 0 stands in for a skipped one)
  uint32_t rec[NW];
#pragma unroll
  for (uint32_t g = 0; g < NW / 4; ++g) {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (4 * g < L.R) u = *reinterpret_cast<const uint4 *>(src + 128 * g + 16 * j);
    rec[4 * g] = u.x;
    rec[4 * g + 1] = u.y;
    rec[4 * g + 2] = u.z;
    rec[4 * g + 3] = u.w;
  }
  const T *tail = reinterpret_cast<const T *>(src + L.tail);
  uint4 tail0 = make_uint4(0u, 0u, 0u, 0u);
  if (VEC && live && j < n_rot / E) tail0 = reinterpret_cast<const uint4 *>(tail)[j];
  // the pair's scale words: the even lane's, then the odd lane's
  uint32_t sc[NB / 4];
#pragma unroll
  for (uint32_t q = 0; q < NB / 4; ++q) sc[q] = 0;
#pragma unroll
  for (uint32_t w = 0; w < NW; ++w) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, rec[w], 1), s = w - L.nb;
    if (w >= L.nb && s < L.ns) {
      const uint32_t even = j & 1 ? other : rec[w], odd = j & 1 ? rec[w] : other;
#pragma unroll
      for (uint32_t q = 0; q < NB / 4; ++q) {
        if (q == s) sc[q] = even;
        if (q == L.ns + s) sc[q] = odd;
      }
    }
  }
  if (!live) return;
#pragma unroll
  for (uint32_t kb = 0; kb < NB; ++kb) {
    const uint32_t d = 64 * kb + 8 * j;
    if (d < L.nope) {
      float v[8];
      fp4_decode(rec[kb], (sc[kb / 4] >> (8 * (kb % 4))) & 255u, v);
      store8<T, VEC>(dst + d, v);
    }
  }
  if (VEC) {
    if (j < n_rot / E) reinterpret_cast<uint4 *>(dst + L.nope)[j] = tail0;
    for (uint32_t c = j + 8; c < n_rot / E; c += 8)
      reinterpret_cast<uint4 *>(dst + L.nope)[c] = reinterpret_cast<const uint4 *>(tail)[c];
  } else {
    for (uint32_t c = j; c < n_rot; c += 8) dst[L.nope + c] = tail[c];
  }
}

template <typename T, int NB>
cudaError_t launch_nb(bool pack, const RowsArgs &a, cudaStream_t s) {
  // 16-byte vectors where every row and its tail start on 16 bytes
  const bool vec = reinterpret_cast<uintptr_t>(a.rows) % 16 == 0 &&
                   a.D * sizeof(T) % 16 == 0 && a.n_rot * sizeof(T) % 16 == 0;
  auto *k = pack ? (vec ? rows_pack_kernel<T, true, NB, false> : rows_pack_kernel<T, false, NB, false>)
                 : (vec ? rows_unpack_kernel<T, true, NB> : rows_unpack_kernel<T, false, NB>);
  if (pack && NB == 8 && vec && a.D == 512 && a.n_rot == 64) k = rows_pack_kernel<T, true, 8, true>;
  const uint32_t per = kThreads / 8;
  const cudaError_t e = launch_pdl(k, dim3((a.n + per - 1) / per), dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(bool pack, const RowsArgs &a, cudaStream_t s) {
  return a.L.nb <= 8 ? launch_nb<T, 8>(pack, a, s) : launch_nb<T, 16>(pack, a, s);
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
