// kv4.cu -- the paged key/value cache held in 4 bits: new tokens in
// (redlite_kv4_append), stored values out (redlite_kv4_load).  The attention
// that reads it is kv4_decode.cu.  ("Red Lite dev16 -- complete
// full-attention parity", section "Pinned full-attention graph": grouped
// heads over a K/V cache.)
//
// Both kernels move bytes: a thread owns eight consecutive values of one
// token's head (one 32-bit code word), four threads a group of 32, so a
// group's minimum and maximum are two shuffles, every load and store of
// values is 16 bytes or more per thread, and no two tokens share a stored
// byte (no read-modify-write between threads).  Bound by the bytes of the
// unpacked side.
#include "kv4.cuh"

namespace redlite {
namespace {

struct Kv4Args {
  const void *k, *v;  // append: in; load: null
  void *ko, *vo;      // load: out
  int64_t k_stride, v_stride;
  const int32_t *cu, *start, *table;
  int n_seqs, n_tokens, n_heads, page_size, max_pages;
  int64_t n_pages;
  uint8_t *cache;
  int32_t *status;
};

// Where a row's tile lies, or null (a row behind the last sequence, or a page
// the table does not name: reported).
template <int D>
__device__ __forceinline__ uint8_t *row_tile(const Kv4Args &a, int64_t row, int head, int &tok, bool &skip) {
  const int s = find_seq(a.cu, a.n_seqs, row);
  skip = s < 0;
  if (skip) return nullptr;
  const int64_t pos = (int64_t)__ldg(a.start + s) + (row - __ldg(a.cu + s));
  if (pos < 0 || pos / a.page_size >= a.max_pages) {
    set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
    return nullptr;
  }
  const int64_t page = __ldg(a.table + (int64_t)s * a.max_pages + pos / a.page_size);
  if (page < 0 || page >= a.n_pages) {
    set_status(a.status, REDLITE_STATUS_BAD_PAGE);
    return nullptr;
  }
  const int in_page = (int)(pos % a.page_size);
  tok = in_page & 15;
  return a.cache + kv4_tile_offset<D>(page, a.n_heads, head, a.page_size, in_page >> 4);
}

// Threads of one value row (key or value of one token and head).
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4Args a) {
  constexpr int kWords = D / 8;
  const int64_t id = (int64_t)blockIdx.x * (256 / kWords) + threadIdx.x / kWords;
  const int w = threadIdx.x % kWords;
  const int64_t n = (int64_t)a.n_tokens * a.n_heads * 2;
  // a row's threads share these conditions, and the shuffles below stay
  // inside groups of four threads of one row
  const bool live = id < n;
  const bool is_v = id & 1;
  const int64_t row = (id >> 1) / a.n_heads;
  const int head = (int)((id >> 1) % a.n_heads);
  int tok = 0;
  bool skip = true;
  uint8_t *tile = live ? row_tile<D>(a, row, head, tok, skip) : nullptr;
  float x[8];
  if (tile) {
    const T *src = (is_v ? (const T *)a.v + row * a.v_stride : (const T *)a.k + row * a.k_stride) + head * D + w * 8;
    load8<T>(src, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
  bool finite = true;
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    finite = finite && isfinite(x[i]);
    x[i] = fminf(fmaxf(x[i], -65504.f), 65504.f);
    lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    finite = __shfl_xor_sync(0xffffffffu, (int)finite, o) && finite;
  }
  // step and minimum are stored in 16 bits (11 significant ones, a quarter of
  // a bit per value); the codes are chosen for the stored pair, with the
  // quotient in 64 bits so that a value next to the border between two codes
  // gets the nearer one
  __half mh = __float2half_rn(lo);
  const float m = __half2float(mh);
  __half dh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, m), 15.f));
  const double d = (double)__half2float(dh);
  uint32_t word = 0;
  if (d > 0.0 && finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double c = rint(((double)x[i] - (double)m) / d);
      word |= (uint32_t)fmin(fmax(c, 0.0), 15.0) << (4 * i);
    }
  }
  if (!finite) {  // a group that holds a NaN or an infinity reads back as NaN
    mh = __ushort_as_half(0x7fff);
    dh = mh;
  }
  if (!tile) return;
  const int g = w >> 2, c = w & 3;
  if (!is_v) {
    *reinterpret_cast<uint32_t *>(tile + kv4_k_word<D>(tok, g, c)) = word;
    if (c == 0) *reinterpret_cast<__half2 *>(tile + kv4_k_step<D>(tok, g)) = __halves2half2(dh, mh);
  } else {
    *reinterpret_cast<uint16_t *>(tile + kv4_v_unit<D>(tok, g, 2 * c)) = (uint16_t)word;
    *reinterpret_cast<uint16_t *>(tile + kv4_v_unit<D>(tok, g, 2 * c + 1)) = (uint16_t)(word >> 16);
    if (c == 0) {
      *reinterpret_cast<__half *>(tile + kv4_v_step<D>(tok, g)) = dh;
      *reinterpret_cast<__half *>(tile + kv4_v_min<D>(tok, g)) = mh;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_load_kernel(Kv4Args a) {
  constexpr int kWords = D / 8;
  const int64_t id = (int64_t)blockIdx.x * (256 / kWords) + threadIdx.x / kWords;
  const int w = threadIdx.x % kWords;
  if (id >= (int64_t)a.n_tokens * a.n_heads * 2) return;
  const bool is_v = id & 1;
  const int64_t row = (id >> 1) / a.n_heads;
  const int head = (int)((id >> 1) % a.n_heads);
  int tok = 0;
  bool skip = false;
  const uint8_t *tile = row_tile<D>(a, row, head, tok, skip);
  if (skip) return;
  const int g = w >> 2, c = w & 3;
  uint32_t word = 0;
  float d = 0.f, m = 0.f;  // a position without a page reads as zeros (reported)
  if (tile && !is_v) {
    word = *reinterpret_cast<const uint32_t *>(tile + kv4_k_word<D>(tok, g, c));
    const __half2 dm = *reinterpret_cast<const __half2 *>(tile + kv4_k_step<D>(tok, g));
    d = __low2float(dm), m = __high2float(dm);
  } else if (tile) {
    word = *reinterpret_cast<const uint16_t *>(tile + kv4_v_unit<D>(tok, g, 2 * c)) |
           ((uint32_t)*reinterpret_cast<const uint16_t *>(tile + kv4_v_unit<D>(tok, g, 2 * c + 1)) << 16);
    d = __half2float(*reinterpret_cast<const __half *>(tile + kv4_v_step<D>(tok, g)));
    m = __half2float(*reinterpret_cast<const __half *>(tile + kv4_v_min<D>(tok, g)));
  }
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(d, (float)((word >> (4 * i)) & 15u), m);  // d * code is exact
  T *dst = (is_v ? (T *)a.vo + row * a.v_stride : (T *)a.ko + row * a.k_stride) + head * D + w * 8;
  store8<T>(dst, x);
}

template <bool APPEND, typename T>
cudaError_t launch_rows(const Kv4Args &a, int D, cudaStream_t s) {
  const int64_t rows = (int64_t)a.n_tokens * a.n_heads * 2, per = 256 / (D / 8);
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  if (D == 256) {
    if (APPEND) kv4_append_kernel<T, 256><<<grid, 256, 0, s>>>(a);
    else kv4_load_kernel<T, 256><<<grid, 256, 0, s>>>(a);
  } else {
    if (APPEND) kv4_append_kernel<T, 128><<<grid, 256, 0, s>>>(a);
    else kv4_load_kernel<T, 128><<<grid, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <bool APPEND>
int run_rows(int32_t dtype, const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int32_t *cu,
             const int32_t *start, int32_t n_seqs, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
             int32_t page_size, const int32_t *table, int32_t max_pages, int64_t n_pages, void *cache, int32_t *status,
             void *stream) {
  if (!dtype_ok(dtype) || n_seqs < 0 || n_tokens < 0 || n_kv_heads < 1 || n_kv_heads > 1024) return REDLITE_EINVAL;
  if (!kv4_shape_ok(head_dim, page_size)) return REDLITE_EUNSUPPORTED;
  if (n_tokens == 0 || n_seqs == 0) return REDLITE_OK;
  if (max_pages < 1 || n_pages < 1 || !k || !v || !cu || !start || !table || !cache) return REDLITE_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return REDLITE_EINVAL;
  const int64_t row = (int64_t)n_kv_heads * head_dim;
  if (!stride_ok(k_stride, row, dtype) || !stride_ok(v_stride, row, dtype)) return REDLITE_EINVAL;
  if ((int64_t)n_tokens * n_kv_heads * 2 * (head_dim / 8) / 256 >= ((int64_t)1 << 31) - 1) return REDLITE_EUNSUPPORTED;
  Kv4Args a;
  a.k = k, a.v = v, a.ko = const_cast<void *>(k), a.vo = const_cast<void *>(v);
  a.k_stride = k_stride, a.v_stride = v_stride;
  a.cu = cu, a.start = start, a.table = table;
  a.n_seqs = n_seqs, a.n_tokens = n_tokens, a.n_heads = n_kv_heads, a.page_size = page_size, a.max_pages = max_pages;
  a.n_pages = n_pages, a.cache = (uint8_t *)cache, a.status = status;
  cudaError_t e;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == REDLITE_T_F32) e = launch_rows<APPEND, float>(a, head_dim, s);
  else if (dtype == REDLITE_T_BF16) e = launch_rows<APPEND, __nv_bfloat16>(a, head_dim, s);
  else e = launch_rows<APPEND, __half>(a, head_dim, s);
  return e == cudaSuccess ? REDLITE_OK : REDLITE_ECUDA;
}

}  // namespace
}  // namespace redlite

using namespace redlite;

extern "C" size_t redlite_kv4_page_bytes(int32_t n_kv_heads, int32_t head_dim, int32_t page_size) {
  if (n_kv_heads < 1 || n_kv_heads > 1024 || !kv4_shape_ok(head_dim, page_size)) return 0;
  return (size_t)n_kv_heads * (page_size / 16) * 20 * head_dim;
}

extern "C" int redlite_kv4_append(int32_t dtype, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                                  const int32_t *cu_tokens, const int32_t *start, int32_t n_seqs, int32_t n_tokens,
                                  int32_t n_kv_heads, int32_t head_dim, int32_t page_size, const int32_t *block_table,
                                  int32_t max_pages, int64_t n_pages, void *cache, int32_t *status, void *stream) {
  return run_rows<true>(dtype, k, v, k_stride, v_stride, cu_tokens, start, n_seqs, n_tokens, n_kv_heads, head_dim,
                        page_size, block_table, max_pages, n_pages, cache, status, stream);
}

extern "C" int redlite_kv4_load(int32_t dtype, const void *cache, int32_t n_kv_heads, int32_t head_dim,
                                int32_t page_size, const int32_t *block_table, int32_t max_pages, int64_t n_pages,
                                const int32_t *cu_tokens, const int32_t *start, int32_t n_seqs, int32_t n_tokens,
                                void *k, void *v, int64_t k_stride, int64_t v_stride, int32_t *status, void *stream) {
  return run_rows<false>(dtype, k, v, k_stride, v_stride, cu_tokens, start, n_seqs, n_tokens, n_kv_heads, head_dim,
                         page_size, block_table, max_pages, n_pages, const_cast<void *>(cache), status, stream);
}
