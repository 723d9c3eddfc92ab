// kv4.cu -- the paged key/value cache held in 4 bits: new tokens in
// (redlite_kv4_append), stored values out (redlite_kv4_load).  The attention
// that reads it is kv4_decode.cu.  ("Red Lite dev16 -- complete
// full-attention parity", section "Pinned full-attention graph": grouped
// heads over a K/V cache.)
//
// Both kernels move bytes: a thread owns eight consecutive values (one 32-bit
// code word) of a token's head, of the key and of the value, four threads a
// group of 32, so a group's minimum and maximum are two shuffles, every load
// and store of values is 16 bytes or more per thread, and no two tokens share
// a stored byte (no read-modify-write between threads).  The floor is the
// bytes of both sides; what bounds the kernels are instructions, so the place
// in the cache is found once for key and value and in 32 bits, and the
// quantiser keeps off the conversion and 64-bit units.  Measured: 8096 tokens
// of two heads of 256, bf16 in and fp32 out, 16 us in and 12 us out alone, 23 us
// for both in a row (their bytes take 9 us; 25 us with 32-bit values stored as
// each thread holds them); 16 tokens 5.8 us for both.  With
// 64-bit places and quotients: 40 us and 15 us.
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

// A block's rows: row i of `kRows` is head i % n_heads of token blockIdx.x *
// tokens + i / n_heads; more heads than rows continue in blockIdx.y.
template <int D>
struct Rows {
  static constexpr int kWords = D / 8, kRows = 256 / kWords;
  int64_t token;
  int head;
  bool live;
  __device__ __forceinline__ explicit Rows(const Kv4Args &a) {
    const unsigned i = threadIdx.x / kWords, heads = a.n_heads, tokens = heads < kRows ? kRows / heads : 1u;
    const unsigned t = heads < kRows ? i / heads : 0u;
    head = (int)(heads < kRows ? i - t * heads : blockIdx.y * kRows + i);
    token = (int64_t)blockIdx.x * tokens + t;
    live = t < tokens && head < a.n_heads && token < a.n_tokens;
  }
};

// Where a row's tile lies, or null (a row behind the last sequence, or a page
// the table does not name: reported).
template <int D>
__device__ __forceinline__ uint8_t *row_tile(const Kv4Args &a, int64_t row, int head, int &tok, bool &skip) {
  const int s = find_seq(a.cu, a.n_seqs, row);
  skip = s < 0;
  if (skip) return nullptr;
  const int64_t at = (int64_t)__ldg(a.start + s) + (row - __ldg(a.cu + s));
  const uint32_t pos = (uint32_t)at, p = pos / (uint32_t)a.page_size;  // a sum of two numbers below 2^31
  if (at < 0 || p >= (uint32_t)a.max_pages) {
    set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
    return nullptr;
  }
  const int64_t page = __ldg(a.table + (int64_t)s * a.max_pages + p);
  if (page < 0 || page >= a.n_pages) {
    set_status(a.status, REDLITE_STATUS_BAD_PAGE);
    return nullptr;
  }
  const int in_page = (int)(pos - p * (uint32_t)a.page_size);
  tok = in_page & 15;
  return a.cache + kv4_tile_offset<D>(page, a.n_heads, head, a.page_size, in_page >> 4);
}

// The first block reports sequences whose offsets do not ascend within the
// rows (what rows they leave to others is found row by row).
__device__ __forceinline__ void check_offsets(const Kv4Args &a) {
  if (blockIdx.x | blockIdx.y) return;
  for (int s = threadIdx.x; s < a.n_seqs; s += blockDim.x) {
    const int b = __ldg(a.cu + s), e = __ldg(a.cu + s + 1);
    if (b < 0 || e < b || e > a.n_tokens) set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
  }
}

// Codes of eight values and the step and minimum of their group of 32 (four
// threads).  Step and minimum are stored in 16 bits (11 significant ones, a
// quarter of a bit per value); the codes are chosen for the stored pair.
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], __half &dh, __half &mh) {
  float odd = 0.f;  // a NaN once a value is not finite
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) odd = fmaf(x[i], 0.f, odd), lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    odd += __shfl_xor_sync(0xffffffffu, odd, o);
  }
  // a value outside +-65504 gets the code of the end it lies behind
  lo = fminf(fmaxf(lo, -65504.f), 65504.f), hi = fminf(fmaxf(hi, -65504.f), 65504.f);
  mh = __float2half_rn(lo);
  const float m = __half2float(mh);
  dh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, m), 15.f));
  const float d = __half2float(dh);
  uint32_t word = 0;
  if (odd != 0.f) {  // a group that holds a NaN or an infinity reads back as NaN
    mh = dh = __ushort_as_half(0x7fff);
  } else if (d > 0.f) {
    // The quotient in fp32 is off by 15 x 2^-21 at most; the sum with 1.5 x
    // 2^23 rounds it to a whole number (ties to even) in its low bits.  One
    // within 2^-16 of the border between two codes is decided in 64 bits, by
    // the side of the border that the value lies on (16-bit inputs meet the
    // border itself once in a thousand).
    const float inv = __fdividef(1.f, d);
    uint32_t near = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fminf(fmaxf(__fsub_rn(x[i], m) * inv, 0.f), 15.f), z = y + 12582912.f;
      if (fabsf(y - (z - 12582912.f)) > 0.5f - 0x1p-16f) near |= 1u << (4 * i);
      word += (__float_as_uint(z) & 15u) << (4 * i);
    }
    while (near) {
      const int at = __ffs(near) - 1;
      near &= near - 1;
      float v = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) v = at == 4 * j ? x[j] : v;
      const float below = floorf(__fsub_rn(v, m) * inv);
      const double side = fma(-((double)below + 0.5), (double)d, (double)v - (double)m);
      const uint32_t k = (uint32_t)below, code = side > 0.0 || (side == 0.0 && (k & 1u)) ? k + 1 : k;
      word = (word & ~(15u << at)) | (code << at);
    }
  }
  return word;
}

template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4Args a) {
  after_predecessor();
  check_offsets(a);
  const Rows<D> row(a);
  const int w = threadIdx.x % Rows<D>::kWords, g = w >> 2, c = w & 3;
  // a row's threads share these conditions, and the shuffles stay inside
  // groups of four threads of one row
  float x[8], y[8];
  if (row.live) {
    load8<T>((const T *)a.k + row.token * a.k_stride + row.head * D + w * 8, x);
    load8<T>((const T *)a.v + row.token * a.v_stride + row.head * D + w * 8, y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
  }
  int tok = 0;
  bool skip = true;
  uint8_t *tile = row.live ? row_tile<D>(a, row.token, row.head, tok, skip) : nullptr;
  __half dk, mk, dv, mv;
  const uint32_t kw = quantise(x, dk, mk), vw = quantise(y, dv, mv);
  if (!tile) return;
  *reinterpret_cast<uint32_t *>(tile + kv4_k_word<D>(tok, g, c)) = kw;
  uint16_t *vu = reinterpret_cast<uint16_t *>(tile + kv4_v_unit<D>(tok, g, 2 * c));
  vu[0] = (uint16_t)vw, vu[32] = (uint16_t)(vw >> 16);  // the next eighth of the group lies 32 units on
  if (c == 0) {
    *reinterpret_cast<__half2 *>(tile + kv4_k_step<D>(tok, g)) = __halves2half2(dk, mk);
    *reinterpret_cast<__half *>(tile + kv4_v_step<D>(tok, g)) = dv;
    *reinterpret_cast<__half *>(tile + kv4_v_min<D>(tok, g)) = mv;
  }
}

// Nibbles 0 .. N-1 of a word.  d * code is exact; the code as the low bits of
// 2^23 + code.
template <int N>
__device__ __forceinline__ void expand(uint32_t word, float d, float m, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = fmaf(d, __uint_as_float(((word >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.f, m);
}
// The values of word w of a row.  32-bit ones go out by pairs of threads, each
// half of either's word, so that a store of the warp fills whole sectors.
template <typename T, int D>
__device__ __forceinline__ void put_words(T *row, int w, uint32_t word, float d, float m) {
  if constexpr (sizeof(T) == 4) {
    const int odd = w & 1;
    const uint32_t other = __shfl_xor_sync(D == 256 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16), word, 1);
    float x[4], y[4];
    expand((odd ? other : word) >> (16 * odd), d, m, x);
    expand((odd ? word : other) >> (16 * odd), d, m, y);
    float4 *p = reinterpret_cast<float4 *>(row + (w - odd) * 8) + odd;
    p[0] = make_float4(x[0], x[1], x[2], x[3]), p[2] = make_float4(y[0], y[1], y[2], y[3]);
  } else {
    float x[8];
    expand(word, d, m, x);
    store8<T>(row + w * 8, x);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_load_kernel(const Kv4Args a) {
  after_predecessor();
  check_offsets(a);
  const Rows<D> row(a);
  if (!row.live) return;
  const int w = threadIdx.x % Rows<D>::kWords, g = w >> 2, c = w & 3;
  int tok = 0;
  bool skip = false;
  const uint8_t *tile = row_tile<D>(a, row.token, row.head, tok, skip);
  if (skip) return;
  uint32_t kw = 0, vw = 0;
  float dk = 0.f, mk = 0.f, dv = 0.f, mv = 0.f;  // a position without a page reads as zeros (reported)
  if (tile) {
    kw = *reinterpret_cast<const uint32_t *>(tile + kv4_k_word<D>(tok, g, c));
    const uint16_t *vu = reinterpret_cast<const uint16_t *>(tile + kv4_v_unit<D>(tok, g, 2 * c));
    vw = vu[0] | ((uint32_t)vu[32] << 16);
    const __half2 dm = *reinterpret_cast<const __half2 *>(tile + kv4_k_step<D>(tok, g));
    dk = __low2float(dm), mk = __high2float(dm);
    dv = __half2float(*reinterpret_cast<const __half *>(tile + kv4_v_step<D>(tok, g)));
    mv = __half2float(*reinterpret_cast<const __half *>(tile + kv4_v_min<D>(tok, g)));
  }
  put_words<T, D>((T *)a.ko + row.token * a.k_stride + row.head * D, w, kw, dk, mk);
  put_words<T, D>((T *)a.vo + row.token * a.v_stride + row.head * D, w, vw, dv, mv);
}

template <bool APPEND, typename T>
cudaError_t launch_rows(const Kv4Args &a, int D, cudaStream_t s) {
  const int64_t per = a.n_heads, rows = 256 / (D / 8), tokens = per < rows ? rows / per : 1;
  const dim3 grid((unsigned)((a.n_tokens + tokens - 1) / tokens), (unsigned)((per + rows - 1) / rows));
  if (D == 256) return launch_early(APPEND ? kv4_append_kernel<T, 256> : kv4_load_kernel<T, 256>, grid, 256, 0, s, a);
  return launch_early(APPEND ? kv4_append_kernel<T, 128> : kv4_load_kernel<T, 128>, grid, 256, 0, s, a);
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
