// mixer.cuh -- element types and small device helpers shared by the token
// mixers (attention over packed prompts, the 4-bit key/value cache, the
// gated delta rule).
#pragma once

#include <utility>

#include "internal.cuh"
#include "ptx.cuh"

namespace redlite {

inline bool dtype_ok(int32_t t) { return t == REDLITE_T_F32 || t == REDLITE_T_BF16 || t == REDLITE_T_F16; }
inline int dtype_bytes(int32_t t) { return t == REDLITE_T_F32 ? 4 : 2; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
// A row stride in elements that keeps rows on 16-byte boundaries.
inline bool stride_ok(int64_t stride, int64_t row, int32_t dtype) {
  return stride >= row && stride <= ((int64_t)1 << 40) && (stride * dtype_bytes(dtype)) % 16 == 0;
}

// Launch a kernel that may be set up while the one in front of it in the
// stream still runs: the kernel calls after_predecessor() first, on every way
// out too, and touches nothing before (so whatever that kernel is, its results
// are there, and a kernel behind this one never overtakes it).  Of a call of a
// few us this hides the launch, 1 to 2 us.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
__device__ __forceinline__ void after_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Eight consecutive elements at a 16-byte aligned address, as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  if (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const T *e = reinterpret_cast<const T *>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
  if (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 a;
    T *e = reinterpret_cast<T *>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4 *>(p) = a;
  }
}

// Two fp32 values as a bf16 pair (lo in the low half), nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// x = hi + lo with hi, lo in fp16, for values below 2^15: what is left out is
// at most 2^-23 of x, or 2^-25 where x is small (fp16's smallest step).
__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_f16(a, b);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  lo = pack_f16(a - f.x, b - f.y);
}
// The power of two that takes m >= 0 into [2^14, 2^15) (2^126 at most), and
// its inverse: a row so scaled and split in two fp16 parts is held to 2^-23 of
// each element and 2^-39 of the row's largest.
__device__ __forceinline__ float scale_f16(float m, float &inv) {
  const int e = max(__float_as_int(m) >> 23, 15);
  inv = __int_as_float((e - 14) << 23);
  return __int_as_float((268 - e) << 23);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Warp tensor-core step: D[16x8] += A[16x16] B[16x8], bf16 in, fp32 sums.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D[16x8] += A[16x8] B[8x8], tf32 in (the low 13 bits of an operand are not read).
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, hi the nearest tf32 number: lo has 12 significant bits, of
// which the product reads 11 (2^-22 of x is left out).
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}

// An 8 x 8 matrix of 16-bit values, one row per four lanes, transposed.
__device__ __forceinline__ uint32_t movm(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void set_status(int32_t *status, int bits) {
  if (status) atomicOr(status, bits);
}

// The sequence a packed row belongs to: cu[s] <= row < cu[s + 1], or -1 for a
// row behind the last sequence (or in front of the first).  cu is not
// trusted: the result is checked, so a table that does not ascend gives -1 or
// a sequence that really holds the row.
__device__ __forceinline__ int find_seq(const int32_t *__restrict__ cu, int n_seqs, int64_t row) {
  int lo = 0, hi = n_seqs;  // the last s with cu[s] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= row) lo = mid;
    else hi = mid;
  }
  return (__ldg(cu + lo) <= row && row < __ldg(cu + lo + 1)) ? lo : -1;
}

}  // namespace redlite
