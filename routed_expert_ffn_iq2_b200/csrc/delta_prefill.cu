// delta_prefill.cu -- the gated delta rule over packed sequences, in chunks
// of 64 tokens (redlite_delta_prefill).  ("Red Lite dev15 -- DeltaNet
// projection bring-up", section "Field-derived recurrent dimensions".)
//
// Within a chunk, with c_i the sum of the log decays up to token i, S0 the
// state in front of it, G = K K^T, and rows written per token:
//   A_ij = beta_i exp(c_i - c_j) G_ij (j < i),   T = (I + A)^-1,
//   D = T (beta V - beta exp(c) K S0)                  (the updates d_i)
//   O = scale (exp(c) Q S0 + P D),  P_ij = exp(c_i - c_j) (Q K^T)_ij (j <= i)
//   S = exp(c_last) S0 + sum_i exp(c_last - c_i) k_i d_i^T
// T and P need no state, so delta_prep_kernel forms them for all chunks at
// once; delta_chain_kernel then walks the chunks of a sequence.  Everything in
// the chain is linear in the value columns, so a warp takes eight of them (the
// N of m16n8k16) and keeps its S [dk x 8] in fp32 accumulators:
//   K S -> D -> S
// each result going through movmatrix into the next product's B operand;
// columns meet nowhere.  A chain is serial, so the latency of a chunk bounds a
// call of few sequences: a second warp beside each takes the operands over
// shared memory and forms Q S + P D, which nothing waits for.  K, Q, T, P and
// the per-token factors come through shared memory by bulk copies.
//
// Precision: every operand of a product is held to 2^-22 or better (relative
// error of eight packed fp32 prompts against 64 bits 7.7e-7; the plain form in
// fp32, with 2^-24, 2.7e-7).  A row is scaled by a power of two that
// takes its largest element to 2^14 and split in two fp16 parts (11 bits
// each); products are hi hi + hi lo + lo hi, hi hi + lo hi where the other
// side (16-bit keys and queries) is one exact part.  bf16 outputs alone are
// made from the hi parts (2^-12 of each operand, under their own rounding of
// 2^-8).  Scales, norms (q, k over their length) and decays multiply results
// per token in fp32.  Sums of log decays are fp64, held as two fp32 numbers
// whose differences are rounded once.
//
// Measured (one B200): 16384 tokens, 16 / 32 heads of 128, bf16: 0.83 ms, of
// which 0.19 ms preparation and 0.64 ms the chain, 2.5 us a chunk; eight packed
// prompts of 3605 tokens, fp32: 0.26 ms.  The chain is bound by the latency of a
// warp (clocks of a chunk: 780 to split S, 870 K S, 570 beta V - K S split, 440
// T times it, 340 D out, 1100 D split and S; the products alone 1300) and, in
// fp32, by reads of shared memory (76%).  So operands are read and barriers
// looked at one step ahead of their use (0.88 and 0.27 ms without).  Two warps
// to a chain, each with one half of the keys, took 1.07 and 0.30 ms: the sums'
// way through shared memory (900) and what both compute outweigh the halves.
// Other forms of the chain, for the same two calls:
// value columns as rows, 16 to a warp 0.88 ms (chain alone) and 0.22 ms, 16 to
// two warps that share the keys 0.79 ms, columns 16 to a warp 1.09 and 0.21 ms,
// and on tcgen05 (128 columns as lanes, operands through tensor memory, two
// threads a column) 1.1 ms and 0.16 ms: there the products take 1.5k of a
// chunk's 7.8k cycles and the splits of S, R and D the rest.  Eight to a warp is
// kept: 0.70 and 0.21 ms.
//
// A chunk that meets a NaN or an infinity is walked token by token, so that
// what lies behind a token never reaches it.
#include <type_traits>

#include "delta.cuh"

namespace redlite {
namespace {

constexpr int C = 64;  // tokens of a chunk

// Per (chunk, value head): T and P as two fp16 planes each (rows scaled), the
// ten 16 x 16 blocks on and under the diagonal (row by row of blocks), a
// block's rows 32 bytes, their two 16-byte pieces swapped in every other group
// of four rows (no bank conflicts); ten per-token factors.  The second plane
// of P comes last: bf16 outputs are made without it, so it is neither written
// nor copied for them.
constexpr int kPlane = 10 * 512;
// fLast: [0] = exp(c_last); fT, fP: inverse scales of the rows of T and P;
// fR, fQ, fK, fNk, fNq hold the inverse scales of the keys' and queries' rows
enum { fBeta, fR, fQ, fK, fAlpha, fNk, fNq, fLast, fT, fP, kFactors };
constexpr int kThi = 0, kTlo = kPlane, kPhi = 2 * kPlane, kFactorsAt = 3 * kPlane, kPlo = kFactorsAt + kFactors * C * 4;
constexpr int kHeadBlock = kPlo + kPlane;
template <typename T>
constexpr bool kOutLo = !std::is_same<T, __nv_bfloat16>::value;  // outputs from both parts

// Per (chunk, key head): K and Q tiles (NK planes each), rows of 2 DK bytes,
// pieces swizzled the same way.
template <int NK, int DK>
__host__ __device__ constexpr int kq_bytes() {
  return 2 * NK * C * DK * 2;
}
template <int DK>
__device__ __forceinline__ uint32_t kq_off(int row, int piece) {
  return row * (DK * 2) + ((piece ^ (row & 7)) << 4);
}
// 16-byte piece `piece` (columns 8 piece ..) of row `row`; piece / 2 <= row / 16.
__device__ __forceinline__ uint32_t tp_off(int row, int piece) {
  const int bi = row >> 4, bj = piece >> 1;
  return (bi * (bi + 1) / 2 + bj) * 512 + (row & 15) * 32 + (((piece ^ (row >> 2)) & 1) << 4);
}

// Chunk slots: chunk i of sequence s has slot cu[s] / 64 + s + i, which
// leaves room for every sequence's last partial chunk without a prefix sum.
inline __host__ __device__ int64_t chunk_slots(int64_t n_tokens, int64_t n_seqs) { return n_tokens / C + n_seqs; }

struct Span {
  int start, len;  // rows of a sequence; len < 0: not a valid range
};
__device__ __forceinline__ Span seq_span(const DeltaArgs &a, int s) {
  const int b = __ldg(a.cu + s), e = __ldg(a.cu + s + 1);
  return Span{b, (b < 0 || e < b || e > a.n_tokens) ? -1 : e - b};
}

struct WsPlan {
  size_t kq, head, order, total;
};
inline WsPlan ws_plan(int64_t slots, int n_seqs, int n_k, int n_v, int dk) {
  WsPlan w;
  w.kq = 0;
  w.head = align256((size_t)slots * n_k * (2 * 2 * C * (size_t)dk * 2));
  w.order = align256(w.head + (size_t)slots * n_v * kHeadBlock);
  w.total = align256(w.order + (size_t)n_seqs * 4);
  return w;
}

// ------------------------------------------------------------------- prep

// The sequences by falling length (in steps of half a power of two), so that
// the chains that take longest start first.  One block.
__device__ void order_sequences(const DeltaArgs &a, int32_t *order, int *bucket) {
  const auto key = [&](int s) {
    const Span sp = seq_span(a, s);
    const unsigned n = (unsigned)((max(sp.len, 0) + C - 1) / C);
    if (n < 2) return 63 - (int)n;
    const int b = 31 - __clz(n);
    return 63 - (2 * b + (int)((n >> (b - 1)) & 1));
  };
  for (int i = threadIdx.x; i < 64; i += blockDim.x) bucket[i] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < a.n_seqs; s += blockDim.x) atomicAdd(bucket + key(s), 1);
  __syncthreads();
  if (threadIdx.x == 0) {
    int sum = 0;
    for (int i = 0; i < 64; ++i) {
      const int n = bucket[i];
      bucket[i] = sum, sum += n;
    }
  }
  __syncthreads();
  for (int s = threadIdx.x; s < a.n_seqs; s += blockDim.x) order[atomicAdd(bucket + key(s), 1)] = s;
}

constexpr int kPitchA = 68;                  // fp32 rows of A: B operands are read without bank conflicts
constexpr int kHeadA = C * kPitchA + 16;     // A of one head
constexpr int kPitchT = 20;                  // rows of a diagonal block of T
template <int NK, int DK>
__host__ __device__ constexpr int prep_smem() {
  return kq_bytes<NK, DK>() > 2 * kHeadA * 4 ? kq_bytes<NK, DK>() : 2 * kHeadA * 4;
}

// Y[16x16] += X[16x16] B[16x16] in tf32 parts (hi hi + hi lo + lo hi).  X: two
// accumulator tiles of 8 columns; B: fp32 rows of `pitch` in shared memory.
// The sum runs over the columns in the order in which X holds them.
__device__ __forceinline__ void block_product(float (&Y)[2][4], const float (&X)[2][4], const float *B, int pitch,
                                              int lane) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    uint32_t h[4], l[4];
    split_tf32(X[kb][0], h[0], l[0]), split_tf32(X[kb][2], h[1], l[1]);
    split_tf32(X[kb][1], h[2], l[2]), split_tf32(X[kb][3], h[3], l[3]);
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const float *p = B + (8 * kb + 2 * c) * pitch + 8 * nb + r;
      uint32_t b0, d0, b1, d1;
      split_tf32(p[0], b0, d0), split_tf32(p[pitch], b1, d1);
      mma_tf32(Y[nb], h, b0, b1);
      mma_tf32(Y[nb], l, b0, b1);
      mma_tf32(Y[nb], h, d0, d1);
    }
  }
}

// Rows r and r + 8 of a 16-row block (NB tiles of 8 columns, zeros from the
// n-th on; the t-th is that of columns 8 tile(t) ..): the scaled fp16 parts to
// two planes, the inverse scales to f.
struct SameTile {
  __device__ __forceinline__ int operator()(int t) const { return t; }
};
template <int NB, bool LO, typename Get, typename Tile = SameTile>
__device__ __forceinline__ void store_rows(uint8_t *hi, uint8_t *lo, float *f, int block, int n, int lane, Get get,
                                           Tile tile = Tile()) {
  const int r = lane >> 2, c = lane & 3;
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    const float *v = get(t);
    m0 = fmaxf(m0, fmaxf(fabsf(v[0]), fabsf(v[1]))), m1 = fmaxf(m1, fmaxf(fabsf(v[2]), fabsf(v[3])));
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  float i0, i1;
  const float s0 = scale_f16(m0, i0), s1 = scale_f16(m1, i1);
  if (c == 0) f[16 * block + r] = i0, f[16 * block + r + 8] = i1;
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    if (t >= n) break;
    const float *v = get(t);
    uint32_t h0, l0, h1, l1;
    split_f16(v[0] * s0, v[1] * s0, h0, l0);
    split_f16(v[2] * s1, v[3] * s1, h1, l1);
    const uint32_t o0 = tp_off(16 * block + r, tile(t)) + 4 * c, o1 = tp_off(16 * block + r + 8, tile(t)) + 4 * c;
    *reinterpret_cast<uint32_t *>(hi + o0) = h0, *reinterpret_cast<uint32_t *>(hi + o1) = h1;
    if (LO) *reinterpret_cast<uint32_t *>(lo + o0) = l0, *reinterpret_cast<uint32_t *>(lo + o1) = l1;
  }
}

// One block per (chunk slot, key head), eight warps.  The first four make
// K K^T and from it A (rows 16 role ..) and the diagonal blocks of T, the
// others Q K^T and P; roles turn with the block, since role 3 has most of the
// work and a warp's scheduler goes by its number.  The value heads of the key
// head go in pairs.  T is found by blocks of 16: the diagonal ones by
// substitution, a row per lane, then, in each row of blocks from the diagonal
// outwards,
//   T_wj = -(sum_{j < k <= w} T_wk A_kj) T_jj
// on the tensor cores, a warp per head and row of blocks.
template <typename T, int NK, int DK>
__global__ void __launch_bounds__(256, 2) delta_prep_kernel(const DeltaArgs a, const WsPlan w) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ double tail[2];
  __shared__ float2 sc[2][C];  // sums of log2 decays: high and low part
  __shared__ float snk[C], snq[C], sss[2][C], sb[2][C];
  __shared__ __align__(16) float td[2][4][16 * kPitchT];
  after_predecessor();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  if (blockIdx.x == 0)
    order_sequences(a, reinterpret_cast<int32_t *>(a.ws + w.order), reinterpret_cast<int *>(smem));
  // key heads next to each other: blocks that run together read whole rows
  const int64_t slot = blockIdx.x / a.n_k;
  const int kh = blockIdx.x % a.n_k, role = (warp + blockIdx.x) & 3, group = warp >> 2;
  // the last sequence whose first slot is not behind this one
  int lo = 0, hi = a.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)(__ldg(a.cu + mid) / C) + mid <= slot) lo = mid;
    else hi = mid;
  }
  const Span sp = seq_span(a, lo);
  const int64_t idx = slot - ((int64_t)(sp.start / C) + lo);
  if (sp.len < 0 || idx < 0 || idx * C >= sp.len) return;
  const int n = min(C, sp.len - (int)idx * C);
  const int64_t row0 = (int64_t)sp.start + idx * C;
  __syncthreads();

  // ---- K and Q rows: scaled fp16 parts into shared memory and the workspace,
  // sums of squares; a thread has several pieces on their way at a time
  const int per = a.n_v / a.n_k, half = tid >> 6, tok = tid & 63;
  float next_g, next_b;  // of this thread's token and head of a pair, on their way
  auto fetch_gb = [&](int h0) {
    next_g = next_b = 0.f;
    if (half < 2 && h0 + half < per && tok < n) {
      next_g = __ldg(a.g + (row0 + tok) * a.n_v + kh * per + h0 + half);
      next_b = __ldg(a.beta + (row0 + tok) * a.n_v + kh * per + h0 + half);
    }
  };
  fetch_gb(0);
  constexpr int kPieces = DK / 8, kTile = C * DK * 2, kRounds = 2 * C * kPieces / 256, kAhead = NK == 1 ? kRounds : 4;
  uint8_t *kq = a.ws + w.kq + ((size_t)slot * a.n_k + kh) * kq_bytes<NK, DK>();
#pragma unroll 1
  for (int r0 = 0; r0 < kRounds; r0 += kAhead) {
    constexpr int kLoads = (int)sizeof(T) / 2;
    uint4 raw[kAhead][kLoads];
#pragma unroll
    for (int it = 0; it < kAhead; ++it) {
      const int id = (r0 + it) * 256 + tid, which = id / (C * kPieces), row = id / kPieces % C, piece = id % kPieces;
      const T *src = (which ? (const T *)a.q + (row0 + row) * a.q_stride : (const T *)a.k + (row0 + row) * a.k_stride) +
                     (int64_t)kh * DK + piece * 8;
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        raw[it][e] = make_uint4(0u, 0u, 0u, 0u);
        if (row < n) raw[it][e] = __ldg(reinterpret_cast<const uint4 *>(src) + e);
      }
    }
#pragma unroll
    for (int it = 0; it < kAhead; ++it) {
      const int id = (r0 + it) * 256 + tid, which = id / (C * kPieces), row = id / kPieces % C, piece = id % kPieces;
      float ss = 0.f, mx = 0.f, x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = to_f32(reinterpret_cast<const T *>(raw[it])[e]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss), mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
      for (int o = 1; o < kPieces; o <<= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      }
      float inv;
      const float s = scale_f16(mx, inv);
      if (piece == 0) (which ? snq : snk)[row] = inv, sss[which][row] = ss;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= s;
      uint4 v, u;
      split_f16(x[0], x[1], v.x, u.x), split_f16(x[2], x[3], v.y, u.y);
      split_f16(x[4], x[5], v.z, u.z), split_f16(x[6], x[7], v.w, u.w);
      const uint32_t off = which * NK * kTile + kq_off<DK>(row, piece);
      *reinterpret_cast<uint4 *>(smem + off) = v;
      *reinterpret_cast<uint4 *>(kq + off) = v;
      if (NK == 2) {
        *reinterpret_cast<uint4 *>(smem + off + kTile) = u;
        *reinterpret_cast<uint4 *>(kq + off + kTile) = u;
      }
    }
  }
  __syncthreads();
  if (tid < 2 * C && a.qk_eps >= 0.f && (tid & (C - 1)) < n) {  // read behind the barriers below
    (tid < C ? snk : snq)[tid & (C - 1)] *= 1.f / sqrtf(sss[tid / C][tid & (C - 1)] + a.qk_eps);
  }
  // ---- rows 16 role .. of K K^T (first group) or Q K^T
  float G[8][4];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) G[t][e] = 0.f;
  const uint32_t base = ptx::smem_u32(smem);
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t ar[NK][4];
    const int arow = 16 * role + (lane & 15), apiece = 2 * ks + (lane >> 4);
#pragma unroll
    for (int p = 0; p < NK; ++p)
      ldsm4(base + (group * NK + p) * kTile + kq_off<DK>(arow, apiece), ar[p][0], ar[p][1], ar[p][2], ar[p][3]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t > role) break;  // columns behind the rows are not needed
      const int brow = 16 * t + (lane & 7) + ((lane >> 4) << 3), bpiece = 2 * ks + ((lane >> 3) & 1);
#pragma unroll
      for (int p = 0; p < NK; ++p) {
        uint32_t b[4];
        ldsm4(base + p * kTile + kq_off<DK>(brow, bpiece), b[0], b[1], b[2], b[3]);
#pragma unroll
        for (int s = 0; s + p < NK; ++s)
#pragma unroll
          for (int u = 0; u < 2; ++u) mma_f16(G[2 * t + u], ar[s], b[2 * u], b[2 * u + 1]);
      }
    }
  }
  float *sa = reinterpret_cast<float *>(smem);  // A of two heads (the tiles are read)
  for (int h0 = 0; h0 < per; h0 += 2) {
    __syncthreads();
    // ---- factors per token: of the first four warps, two take a head
    const int head = kh * per + h0 + half;
    const bool have = half < 2 && h0 + half < per;
    const float g = delta_clamp_g(next_g), b = next_b;
    fetch_gb(h0 + 2);
    double sum = g;
    if (half < 2) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (tok == 31) tail[half] = sum;
    }
    __syncthreads();
    if (half < 2) {
      if (tok >= 32) sum += tail[half];
      const double z = sum * 1.4426950408889634074;
      const float zh = (float)z;
      sc[half][tok] = make_float2(zh, (float)(z - (double)zh)), sb[half][tok] = b;
    }
    __syncthreads();
    // 2 to the difference of two sums: what is rounded is the difference
    auto decay = [&](float2 x, float2 y) { return ex2((x.x - y.x) + (x.y - y.y)); };
    if (have) {
      float *f = reinterpret_cast<float *>(a.ws + w.head + ((size_t)slot * a.n_v + head) * kHeadBlock + kFactorsAt);
      const float2 none = make_float2(0.f, 0.f), mine = sc[half][tok], last = sc[half][C - 1];
      const float gamma = decay(mine, none);
      f[fBeta * C + tok] = b;
      f[fR * C + tok] = b * gamma * snk[tok];
      f[fQ * C + tok] = tok < n ? a.scale * snq[tok] * gamma : 0.f;
      f[fK * C + tok] = tok < n ? snk[tok] * decay(last, mine) : 0.f;
      f[fAlpha * C + tok] = expf(g);
      f[fNk * C + tok] = snk[tok];
      f[fNq * C + tok] = a.scale * snq[tok];
      f[fLast * C + tok] = decay(last, none);
    }
    // ---- A (shared) or P (workspace) of both heads.  In front of the diagonal
    // block a decay is the product of that from the column to the block's
    // first row and that from there to the row.
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      if (h0 + q >= per) break;
      uint8_t *blk = a.ws + w.head + ((size_t)slot * a.n_v + kh * per + h0 + q) * kHeadBlock;
      const int i0 = 16 * role + r, i1 = i0 + 8;
      const float2 c0 = sc[q][i0], c1 = sc[q][i1], cb = sc[q][16 * role];
      const float w0 = group ? a.scale * snq[i0] : sb[q][i0] * snk[i0];
      const float w1 = group ? a.scale * snq[i1] : sb[q][i1] * snk[i1];
      const float e0 = w0 * decay(c0, cb), e1 = w1 * decay(c1, cb);
      float v[8][4];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int j = 8 * t + 2 * c;
        if ((t >> 1) < role) {
          const float f0 = decay(cb, sc[q][j]) * snk[j], f1 = decay(cb, sc[q][j + 1]) * snk[j + 1];
          v[t][0] = e0 * f0 * G[t][0], v[t][1] = e0 * f1 * G[t][1];
          v[t][2] = e1 * f0 * G[t][2], v[t][3] = e1 * f1 * G[t][3];
        } else if ((t >> 1) == role) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = e < 2 ? i0 : i1, jj = j + (e & 1);
            v[t][e] = jj < i || (jj == i && group) ? (e < 2 ? w0 : w1) * decay(e < 2 ? c0 : c1, sc[q][jj]) * snk[jj] * G[t][e]
                                                   : 0.f;
          }
        } else {
          v[t][0] = v[t][1] = v[t][2] = v[t][3] = 0.f;
        }
      }
      if (group) {
        store_rows<8, kOutLo<T>>(blk + kPhi, blk + kPlo, reinterpret_cast<float *>(blk + kFactorsAt) + fP * C, role,
                                 2 * role + 2, lane, [&](int t) { return v[t]; });
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if ((t >> 1) > role) break;
          float *p = sa + q * kHeadA + i0 * kPitchA + 8 * t + 2 * c;
          *reinterpret_cast<float2 *>(p) = make_float2(v[t][0], v[t][1]);
          *reinterpret_cast<float2 *>(p + 8 * kPitchA) = make_float2(v[t][2], v[t][3]);
        }
      }
    }
    // ---- diagonal blocks of T: lane 16 q + i has row i of head q's block
    if (!group) {
      __syncwarp();
      const int q = lane >> 4, i = lane & 15;
      const float *ad = sa + q * kHeadA + 16 * role * kPitchA + 16 * role;
      float t[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) t[j] = i == j ? 1.f : 0.f;
      if (h0 + q < per) {
#pragma unroll
        for (int k = 15; k > 0; --k) {
#pragma unroll
          for (int j4 = 0; j4 < (k + 3) / 4; ++j4) {
            const float4 x = *reinterpret_cast<const float4 *>(ad + k * kPitchA + 4 * j4);
            const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (4 * j4 + e < k) t[4 * j4 + e] = fmaf(-t[k], y[e], t[4 * j4 + e]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4 *>(&td[q][role][i * kPitchT + j]) = make_float4(t[j], t[j + 1], t[j + 2], t[j + 3]);
    }
    __syncthreads();
    // ---- the rest of row block `role` of head q: tiles by their distance d from the diagonal
    const int q = group;
    if (h0 + q >= per) continue;
    uint8_t *blk = a.ws + w.head + ((size_t)slot * a.n_v + kh * per + h0 + q) * kHeadBlock;
    float X[4][2][4];
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) X[d][nb][e] = 0.f;
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const float *p = &td[q][role][r * kPitchT + 8 * nb + 2 * c];
      X[0][nb][0] = p[0], X[0][nb][1] = p[1], X[0][nb][2] = p[8 * kPitchT], X[0][nb][3] = p[8 * kPitchT + 1];
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {
      if (d > role) break;
      const int j = role - d;
      float Y[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int e = 0; e < d; ++e)
        block_product(Y, X[e], sa + q * kHeadA + 16 * (role - e) * kPitchA + 16 * j, kPitchA, lane);
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) Y[nb][e] = -Y[nb][e];
      block_product(X[d], Y, td[q][j], kPitchT, lane);
    }
    // columns 16 (role - d) + 8 nb of the row: tile 2 (role - d) + nb
    store_rows<8, true>(blk + kThi, blk + kTlo, reinterpret_cast<float *>(blk + kFactorsAt) + fT * C, role, 2 * role + 2,
                        lane, [&](int t) { return X[t >> 1][t & 1]; },
                        [&](int t) { return 2 * (role - (t >> 1)) + (t & 1); });
  }
}

// ------------------------------------------------------------------ chain

constexpr int kChains = 4;            // chain warps per block, and as many output warps
constexpr int kCols = 8 * kChains;    // value columns per block

// What a chain warp hands to the output warp beside it, per chunk.
template <bool LO>
struct Handoff {
  uint4 s[LO ? 2 : 1][4][32];  // S as B operands, 32 keys each: hi parts, lo parts
  float4 d[4][32];             // D, 16 tokens each
  float2 scale[4];             // of S's columns 2 c, 2 c + 1
  int walk;                    // the chain warp writes this chunk's outputs
};
template <int kStages>
struct ChainBars {
  uint64_t full[kStages], empty[kStages];
  uint64_t s_ready[kChains], s_taken[kChains], d_ready[kChains], d_taken[kChains];
};
// The plan of a chain block's shared memory.
template <typename T, int NK, int DK>
struct Chain {
  static constexpr bool kLo = kOutLo<T>;
  static constexpr int kHead = kLo ? kHeadBlock : kPlo;  // bytes of a head's block that are used
  static constexpr int kStage = kq_bytes<NK, DK>() + kHead;
  static constexpr int kV = C * 8 * (int)sizeof(T);  // a chain warp's values of a chunk
  static constexpr int kRest = 2 * kChains * kV + kChains * (int)sizeof(Handoff<kLo>) + (int)sizeof(ChainBars<3>);
  static constexpr int kStages = 3 * kStage + kRest <= 227 * 1024 ? 3 : 2;
  static constexpr int kSmem = kStages * kStage + kRest;
  static_assert(kSmem <= 227 * 1024, "shared memory of a chain block");
};

// Largest of columns 2 c and 2 c + 1 over the rows of a warp's tiles.
__device__ __forceinline__ void col_max(float &m0, float &m1) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
}
// The B operand of 16 rows from an accumulator tile, columns scaled, in two parts.
__device__ __forceinline__ void split_tile(const float (&x)[4], float s0, float s1, uint32_t (&h)[2], uint32_t (&l)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    split_f16(x[2 * e] * s0, x[2 * e + 1] * s1, h[e], l[e]);
    h[e] = movm(h[e]), l[e] = movm(l[e]);
  }
}
__device__ __forceinline__ void zero(float (&x)[4][4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
}
// acc (+)= tiles [64 x 16] (rows in shared memory) times a B operand of 16 rows.
template <int DK>
__device__ __forceinline__ void load_rows(uint32_t tile, int ks, int lane, uint32_t (&a)[4][4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
    ldsm4(tile + kq_off<DK>(16 * t + (lane & 15), 2 * ks + (lane >> 4)), a[t][0], a[t][1], a[t][2], a[t][3]);
}
// The lower triangle's blocks (of a plane, and of the one `to_lo` bytes on) of
// 16 columns.
template <bool LO>
__device__ __forceinline__ void load_triangle(uint32_t planes, uint32_t to_lo, int ks, int lane, uint32_t (&p)[4][4], uint32_t (&q)[4][4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (t >= ks) {
      const uint32_t off = planes + tp_off(16 * t + (lane & 15), 2 * ks + (lane >> 4));
      ldsm4(off, p[t][0], p[t][1], p[t][2], p[t][3]);
      if (LO) ldsm4(off + to_lo, q[t][0], q[t][1], q[t][2], q[t][3]);
    }
}
// acc = L B: the triangle times the B operands of 64 rows; p[0] and q[0] hold
// its first 16 columns, the next ones are read while products run.
template <bool LO>
__device__ __forceinline__ void triangle(float (&acc)[4][4], uint32_t planes, uint32_t to_lo,
                                         const uint32_t (&h)[4][2], const uint32_t (&l)[4][2], int lane, uint32_t (&p)[2][4][4],
                                         uint32_t (&q)[2][4][4]) {
  float more[4][4];
  zero(acc), zero(more);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    if (ks < 3) load_triangle<LO>(planes, to_lo, ks + 1, lane, p[(ks + 1) & 1], q[(ks + 1) & 1]);
#pragma unroll
    for (int t = ks; t < 4; ++t) mma_f16(acc[t], p[ks & 1][t], h[ks][0], h[ks][1]);
    if (LO) {
#pragma unroll
      for (int t = ks; t < 4; ++t) mma_f16(more[t], p[ks & 1][t], l[ks][0], l[ks][1]);
#pragma unroll
      for (int t = ks; t < 4; ++t) mma_f16(more[t], q[ks & 1][t], h[ks][0], h[ks][1]);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] += more[t][e];
}
template <typename T>
__device__ __forceinline__ void store2(T *p, float x, float y);
template <>
__device__ __forceinline__ void store2<float>(float *p, float x, float y) {
  *reinterpret_cast<float2 *>(p) = make_float2(x, y);
}
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(__nv_bfloat16 *p, float x, float y) {
  *reinterpret_cast<uint32_t *>(p) = pack_bf16(x, y);
}
template <>
__device__ __forceinline__ void store2<__half>(__half *p, float x, float y) {
  *reinterpret_cast<uint32_t *>(p) = pack_f16(x, y);
}
// Two neighbours as they lie in memory.
template <typename T>
struct Pair {
  typedef uint32_t type;
};
template <>
struct Pair<float> {
  typedef float2 type;
};
template <typename T>
__device__ __forceinline__ float2 pair_f32(typename Pair<T>::type v) {
  if constexpr (sizeof(T) == 4) return v;
  else return make_float2(to_f32(reinterpret_cast<const T *>(&v)[0]), to_f32(reinterpret_cast<const T *>(&v)[1]));
}

// Four chain warps, four output warps and one warp that issues the copies.
// Block: (slice of 32 value columns, value head, sequence by falling length).
template <typename T, int NK, int DK>
__global__ void __launch_bounds__(32 * (2 * kChains + 1), 1) delta_chain_kernel(const DeltaArgs a, const WsPlan w,
                                                                                  const bool ordered) {
  extern __shared__ __align__(128) uint8_t smem[];
  using Plan = Chain<T, NK, DK>;
  constexpr int kStages = Plan::kStages, kStage = Plan::kStage, kTile = C * DK * 2, NT = DK / 16;
  constexpr bool kLo = Plan::kLo;
  uint8_t *vbuf = smem + kStages * kStage;
  Handoff<kLo> *handoff = reinterpret_cast<Handoff<kLo> *>(vbuf + 2 * kChains * Plan::kV);
  ChainBars<kStages> *bars = reinterpret_cast<ChainBars<kStages> *>(handoff + kChains);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int slices = a.dv / kCols;
  const int slice = blockIdx.x % slices, head = blockIdx.x / slices % a.n_v;
  const int kh = head / (a.n_v / a.n_k);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(bars->full + i, 1), ptx::mbar_init(bars->empty + i, 2 * kChains);
    for (int i = 0; i < kChains; ++i) {
      ptx::mbar_init(bars->s_ready + i, 1), ptx::mbar_init(bars->s_taken + i, 1);
      ptx::mbar_init(bars->d_ready + i, 1), ptx::mbar_init(bars->d_taken + i, 1);
    }
  }
  ptx::mbar_fence_init();
  after_predecessor();
  int seq = blockIdx.x / (slices * a.n_v);
  if (ordered) seq = *reinterpret_cast<const int32_t *>(a.ws + w.order + 4 * (size_t)seq);
  const int64_t slot = delta_slot(a, seq);
  __syncthreads();
  const Span sp = seq_span(a, seq);
  if (sp.len < 0) {
    if (tid == 0) set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
    return;
  }
  const int n_chunks = (sp.len + C - 1) / C;
  if (slot < 0) {
    for (int64_t i = tid; i < (int64_t)sp.len * kCols; i += blockDim.x)
      ((T *)a.out)[(sp.start + i / kCols) * a.out_stride + (int64_t)head * a.dv + slice * kCols + i % kCols] =
          from_f32<T>(0.f);
    return;
  }
  const int64_t slot0 = (int64_t)(sp.start / C) + seq;
  if (warp == 2 * kChains) {
    // ============================================================== copies
    if (lane == 0)
      for (int i = 0; i < n_chunks; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !ptx::mbar_wait_suspend(bars->empty + st, ((i / kStages) & 1) ^ 1)) {
          set_status(a.status, REDLITE_STATUS_TIMEOUT);
          // what is on its way still lands in this block
          for (int j = i - kStages; j < i; ++j) ptx::mbar_wait_suspend(bars->full + j % kStages, (j / kStages) & 1);
          break;
        }
        uint8_t *dst = smem + st * kStage;
        ptx::mbar_expect_tx(bars->full + st, kStage);
        ptx::bulk_g2s(dst, a.ws + w.kq + ((size_t)(slot0 + i) * a.n_k + kh) * kq_bytes<NK, DK>(), kq_bytes<NK, DK>(),
                      bars->full + st);
        ptx::bulk_g2s(dst + kq_bytes<NK, DK>(), a.ws + w.head + ((size_t)(slot0 + i) * a.n_v + head) * kHeadBlock,
                      Plan::kHead, bars->full + st);
      }
    return;
  }
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait_suspend(bar, parity));
    if (!ok && lane == 0) set_status(a.status, REDLITE_STATUS_TIMEOUT);
    return ok;
  };
  // the same for a phase that was looked at before (what came between hid the look)
  auto test = [](uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(ptx::smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok;
  };
  auto finish = [&](uint32_t came, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, came) || wait(bar, parity);
  };
  auto arrive = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };
  const int me = warp % kChains, col = slice * kCols + 8 * me;
  Handoff<kLo> &ho = handoff[me];
  T *const out = (T *)a.out + (int64_t)sp.start * a.out_stride + (int64_t)head * a.dv + col + 2 * c;

  if (warp >= kChains) {
    // ============================================== outputs: Q S + P D
    for (int i = 0; i < n_chunks; ++i) {
      const int st = i % kStages, n = min(C, sp.len - i * C);
      const uint32_t sQ = ptx::smem_u32(smem + st * kStage) + NK * kTile;
      const uint32_t sP = sQ + NK * kTile + kPhi;
      const float *f = reinterpret_cast<const float *>(smem + st * kStage + kq_bytes<NK, DK>() + kFactorsAt);
      if (!wait(bars->full + st, (i / kStages) & 1) || !wait(bars->s_ready + me, i & 1)) break;
      float O[4][4];
      zero(O);
      const float2 u = ho.scale[c];
#pragma unroll
      for (int k2 = 0; k2 < NT / 2; ++k2) {
        const uint4 h = ho.s[0][k2][lane];
        uint4 l = h;
        if (kLo) l = ho.s[kLo][k2][lane];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t h0 = e ? h.z : h.x, h1 = e ? h.w : h.y, l0 = e ? l.z : l.x, l1 = e ? l.w : l.y;
          uint32_t q[4][4];
          load_rows<DK>(sQ, 2 * k2 + e, lane, q);
#pragma unroll
          for (int t = 0; t < 4; ++t) mma_f16(O[t], q[t], h0, h1);
          if (kLo)
#pragma unroll
            for (int t = 0; t < 4; ++t) mma_f16(O[t], q[t], l0, l1);
          if (NK == 2) {
            load_rows<DK>(sQ + kTile, 2 * k2 + e, lane, q);
#pragma unroll
            for (int t = 0; t < 4; ++t) mma_f16(O[t], q[t], h0, h1);
          }
        }
      }
      arrive(bars->s_taken + me);
      if (!wait(bars->d_ready + me, i & 1)) break;
      float D[4][4], m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float4 y = ho.d[t][lane];
        D[t][0] = y.x, D[t][1] = y.y, D[t][2] = y.z, D[t][3] = y.w;
        m0 = fmaxf(m0, fmaxf(fabsf(y.x), fabsf(y.z))), m1 = fmaxf(m1, fmaxf(fabsf(y.y), fabsf(y.w)));
      }
      const bool walk = ho.walk;
      arrive(bars->d_taken + me);
      if (!walk) {
        uint32_t p[2][4][4], q[2][4][4];
        load_triangle<kLo>(sP, kPlo - kPhi, 0, lane, p[0], q[0]);
        col_max(m0, m1);
        float i0, i1;
        const float s0 = scale_f16(m0, i0), s1 = scale_f16(m1, i1);
        uint32_t h[4][2], l[4][2];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) split_tile(D[ks], s0, s1, h[ks], l[ks]);
        triangle<kLo>(D, sP, kPlo - kPhi, h, l, lane, p, q);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 16 * t + 8 * e + r;
            const float fq = f[fQ * C + j], fp = f[fP * C + j];
            if (j < n)
              store2<T>(out + (int64_t)(i * C + j) * a.out_stride, fmaf(D[t][2 * e] * fp, i0, O[t][2 * e] * u.x * fq),
                        fmaf(D[t][2 * e + 1] * fp, i1, O[t][2 * e + 1] * u.y * fq));
          }
      }
      arrive(bars->empty + st);
    }
    return;
  }

  // ================================================================ chain
  // state: rows = keys 16 t + r, + 8; columns = value columns col + 2 c, + 1.
  // The state is S * sg (a power of two per column).
  float S[NT][4], sg0 = 1.f, sg1 = 1.f;
  const int64_t s_at = ((slot * a.n_v + head) * (int64_t)DK + r) * a.dv + col + 2 * c;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 x = make_float2(0.f, 0.f);
      if (a.state_in) x = __ldg(reinterpret_cast<const float2 *>(a.state_in + s_at + (int64_t)(16 * t + 8 * e) * a.dv));
      S[t][2 * e] = x.x, S[t][2 * e + 1] = x.y;
    }
  // value rows of a chunk, this warp's eight columns: asynchronous copies into
  // a buffer of its own, zeros behind the end
  constexpr int kPer = 8 * (int)sizeof(T) / 16;  // 16-byte pieces per row
  auto fetch_v = [&](int i) {
    const uint32_t dst = ptx::smem_u32(vbuf + (2 * me + (i & 1)) * Plan::kV);
    const int n = min(C, sp.len - i * C);
#pragma unroll
    for (int it = 0; it < C * kPer / 32; ++it) {
      const int id = it * 32 + lane, row = id / kPer, piece = id % kPer;
      const T *src = (const T *)a.v + (int64_t)(sp.start + i * C + (row < n ? row : 0)) * a.v_stride +
                     (int64_t)head * a.dv + col + piece * (16 / (int)sizeof(T));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (uint32_t)(id * 16)), "l"(src),
                   "r"(row < n ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (n_chunks > 0) fetch_v(0);

  for (int i = 0; i < n_chunks; ++i) {
    const int st = i % kStages, n = min(C, sp.len - i * C);
    const uint32_t sK = ptx::smem_u32(smem + st * kStage), sT = sK + kq_bytes<NK, DK>();
    const float *f = reinterpret_cast<const float *>(smem + st * kStage + kq_bytes<NK, DK>() + kFactorsAt);
    const T *vt = reinterpret_cast<const T *>(vbuf + (2 * me + (i & 1)) * Plan::kV);
    const uint32_t full = test(bars->full + st, (i / kStages) & 1);
    const uint32_t s_free = i == 0 || test(bars->s_taken + me, (i - 1) & 1);
    const uint32_t d_free = i == 0 || test(bars->d_taken + me, (i - 1) & 1);
    // ---- the state in two parts
    float sm0 = 0.f, sm1 = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      sm0 = fmaxf(sm0, fmaxf(fabsf(S[t][0]), fabsf(S[t][2])));
      sm1 = fmaxf(sm1, fmaxf(fabsf(S[t][1]), fabsf(S[t][3])));
    }
    col_max(sm0, sm1);
    float u0, u1;
    uint32_t sh[NT][2], sl[NT][2];
    {
      const float s0 = scale_f16(sm0, u0), s1 = scale_f16(sm1, u1);
      u0 *= sg0, u1 *= sg1;
#pragma unroll
      for (int ks = 0; ks < NT; ++ks) split_tile(S[ks], s0, s1, sh[ks], sl[ks]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    if (i + 1 < n_chunks) fetch_v(i + 1);
    if (!finish(full, bars->full + st, (i / kStages) & 1)) break;
    // ---- K S (operands of every product are read one step ahead of it)
    float R[4][4], D[4][4];
    zero(R);
    constexpr int kSteps = NK * NT;
    uint32_t kr[2][4][4];
    load_rows<DK>(sK, 0, lane, kr[0]);
    // the rows' values and factors
    typename Pair<T>::type vr[8];
    float fb[8], fr[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      vr[m] = *reinterpret_cast<const typename Pair<T>::type *>(vt + (8 * m + r) * 8 + 2 * c);
      fb[m] = f[fBeta * C + 8 * m + r], fr[m] = f[fR * C + 8 * m + r];
    }
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
      const int ks = step / NK;
      if (step + 1 < kSteps) load_rows<DK>(sK + ((step + 1) % NK) * kTile, (step + 1) / NK, lane, kr[(step + 1) & 1]);
      const auto &k = kr[step & 1];
#pragma unroll
      for (int t = 0; t < 4; ++t) mma_f16(R[t], k[t], sh[ks][0], sh[ks][1]);
      if (step % NK == 0)
#pragma unroll
        for (int t = 0; t < 4; ++t) mma_f16(R[t], k[t], sl[ks][0], sl[ks][1]);
    }
    // ---- the state's parts to the output warp, while the products run
    if (i > 0 && !finish(s_free, bars->s_taken + me, (i - 1) & 1)) break;
#pragma unroll
    for (int k2 = 0; k2 < NT / 2; ++k2) {
      ho.s[0][k2][lane] = make_uint4(sh[2 * k2][0], sh[2 * k2][1], sh[2 * k2 + 1][0], sh[2 * k2 + 1][1]);
      if (kLo) ho.s[kLo][k2][lane] = make_uint4(sl[2 * k2][0], sl[2 * k2][1], sl[2 * k2 + 1][0], sl[2 * k2 + 1][1]);
    }
    if (r == 0) ho.scale[c] = make_float2(u0, u1);
    arrive(bars->s_ready + me);
    uint32_t tp[2][4][4], tq[2][4][4];
    load_triangle<true>(sT, kTlo - kThi, 0, lane, tp[0], tq[0]);
    // ---- beta V - beta exp(c) K S
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = 2 * t + e;
        const float2 v = pair_f32<T>(vr[m]);
        R[t][2 * e] = fmaf(fb[m], v.x, -fr[m] * (R[t][2 * e] * u0));
        R[t][2 * e + 1] = fmaf(fb[m], v.y, -fr[m] * (R[t][2 * e + 1] * u1));
        m0 = fmaxf(m0, fabsf(R[t][2 * e])), m1 = fmaxf(m1, fabsf(R[t][2 * e + 1]));
      }
    col_max(m0, m1);
    uint32_t h[4][2], l[4][2];
    float i0, i1, odd = 0.f;  // odd: a NaN or an infinity anywhere (x - x is not 0)
    {
      const float s0 = scale_f16(m0, i0), s1 = scale_f16(m1, i1);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) split_tile(R[ks], s0, s1, h[ks], l[ks]);
    }
    // ---- D = T R
    const float last = f[fLast * C];
    float ft[8], fk[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) ft[m] = f[fT * C + 8 * m + r], fk[m] = f[fK * C + 8 * m + r];
    triangle<true>(D, sT, kTlo - kThi, h, l, lane, tp, tq);
    // K^T of 16 tokens
    uint32_t kt[2][NT][4];
    auto load_keys = [&](int step) {  // step: tokens 16 (step / NK) .., plane step % NK
#pragma unroll
      for (int t = 0; t < NT; ++t)
        ldsm4t(sK + (step % NK) * kTile +
                   kq_off<DK>(16 * (step / NK) + (lane & 7) + ((lane >> 4) << 3), 2 * t + ((lane >> 3) & 1)),
               kt[step & 1][t][0], kt[step & 1][t][1], kt[step & 1][t][2], kt[step & 1][t][3]);
    };
    load_keys(0);
    // (at least 2^-108 of the old scale, so that f0 below stays in fp32 also
    // where nothing is left of the state)
    m0 = last * sg0 * fmaxf(sm0 * 0x1p-60f, 0x1p-108f), m1 = last * sg1 * fmaxf(sm1 * 0x1p-60f, 0x1p-108f);
    if (i > 0 && !finish(d_free, bars->d_taken + me, (i - 1) & 1)) break;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        D[t][2 * e] *= ft[2 * t + e] * i0, D[t][2 * e + 1] *= ft[2 * t + e] * i1;
        odd += (D[t][2 * e] - D[t][2 * e]) + (D[t][2 * e + 1] - D[t][2 * e + 1]);
      }
      ho.d[t][lane] = make_float4(D[t][0], D[t][1], D[t][2], D[t][3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        D[t][2 * e] *= fk[2 * t + e], D[t][2 * e + 1] *= fk[2 * t + e];
        m0 = fmaxf(m0, fabsf(D[t][2 * e])), m1 = fmaxf(m1, fabsf(D[t][2 * e + 1]));
      }
    }
    const bool walk = __any_sync(0xffffffffu, !(odd == 0.f));
    if (lane == 0) ho.walk = walk;
    arrive(bars->d_ready + me);
    if (!walk) {
      // ---- S = exp(c_last) S + K^T (exp(c_last - c) D), on the scale of the
      // updates (or of what is left of the state, if that is 2^60 larger)
      col_max(m0, m1);
      const float s0 = scale_f16(m0, i0), s1 = scale_f16(m1, i1), f0 = last * sg0 * s0, f1 = last * sg1 * s1;
      sg0 = i0, sg1 = i1;
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t][0] *= f0, S[t][1] *= f1, S[t][2] *= f0, S[t][3] *= f1;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) split_tile(D[ks], s0, s1, h[ks], l[ks]);
#pragma unroll
      for (int step = 0; step < 4 * NK; ++step) {
        const int ks = step / NK;
        if (step + 1 < 4 * NK) load_keys(step + 1);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(S[t], kt[step & 1][t], h[ks][0], h[ks][1]);
        if (step % NK == 0)
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(S[t], kt[step & 1][t], l[ks][0], l[ks][1]);
      }
    } else {
      // token by token from the state in front of the chunk
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t][0] *= sg0, S[t][1] *= sg1, S[t][2] *= sg0, S[t][3] *= sg1;
      sg0 = sg1 = 1.f;
      auto total = [&](float &p0, float &p1) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          p0 += __shfl_xor_sync(0xffffffffu, p0, o);
          p1 += __shfl_xor_sync(0xffffffffu, p1, o);
        }
      };
      auto value = [&](uint32_t tile, int j, int key) {  // the parts of one key's element
        float v = 0.f;
#pragma unroll
        for (int p = 0; p < NK; ++p)
          v += __half2float(__ushort_as_half(
              (uint16_t)ptx::lds16(tile + p * kTile + kq_off<DK>(j, key >> 3) + 2 * (key & 7))));
        return v;
      };
      for (int j = 0; j < n; ++j) {
        const float al = f[fAlpha * C + j], be = f[fBeta * C + j], nk = f[fNk * C + j], nq = f[fNq * C + j];
        float p0 = 0.f, p1 = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float k = value(sK, j, 16 * t + 8 * e + r);
            p0 = fmaf(k, S[t][2 * e], p0), p1 = fmaf(k, S[t][2 * e + 1], p1);
          }
        total(p0, p1);
        const float2 v = pair_f32<T>(*reinterpret_cast<const typename Pair<T>::type *>(vt + j * 8 + 2 * c));
        const float d0 = be * (v.x - al * nk * p0) * nk, d1 = be * (v.y - al * nk * p1) * nk;
        p0 = p1 = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float k = value(sK, j, 16 * t + 8 * e + r), q = value(sK + NK * kTile, j, 16 * t + 8 * e + r);
            S[t][2 * e] = fmaf(al, S[t][2 * e], k * d0), S[t][2 * e + 1] = fmaf(al, S[t][2 * e + 1], k * d1);
            p0 = fmaf(q, S[t][2 * e], p0), p1 = fmaf(q, S[t][2 * e + 1], p1);
          }
        total(p0, p1);
        if (r == 0) store2<T>(out + (int64_t)(i * C + j) * a.out_stride, p0 * nq, p1 * nq);
      }
    }
    arrive(bars->empty + st);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that gave up)
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      *reinterpret_cast<float2 *>(a.state_out + s_at + (int64_t)(16 * t + 8 * e) * a.dv) =
          make_float2(S[t][2 * e] * sg0, S[t][2 * e + 1] * sg1);
}

template <typename T, int NK, int DK>
cudaError_t launch_prefill(const DeltaArgs &a, const WsPlan &w, cudaStream_t s) {
  cudaError_t e;
  if (a.n_tokens > 0) {
    constexpr int smem = prep_smem<NK, DK>();
    e = cudaFuncSetAttribute(delta_prep_kernel<T, NK, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_early(delta_prep_kernel<T, NK, DK>, (unsigned)(chunk_slots(a.n_tokens, a.n_seqs) * a.n_k), 256, smem, s, a, w);
    if (e != cudaSuccess) return e;
  }
  constexpr int smem = Chain<T, NK, DK>::kSmem;
  e = cudaFuncSetAttribute(delta_chain_kernel<T, NK, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_early(delta_chain_kernel<T, NK, DK>, (unsigned)((int64_t)a.n_seqs * a.n_v * (a.dv / kCols)),
                      32 * (2 * kChains + 1), smem, s, a, w, a.n_tokens > 0);
}

template <typename T, int NK>
cudaError_t launch_prefill_dk(const DeltaArgs &a, const WsPlan &w, cudaStream_t s) {
  return a.dk == 128 ? launch_prefill<T, NK, 128>(a, w, s) : launch_prefill<T, NK, 64>(a, w, s);
}

}  // namespace
}  // namespace redlite

using namespace redlite;

extern "C" size_t redlite_delta_workspace_bytes(int32_t n_tokens, int32_t n_seqs, int32_t n_k_heads, int32_t n_v_heads,
                                                int32_t dk, int32_t dv) {
  if (n_tokens < 0 || n_seqs < 0 || n_k_heads < 1 || n_v_heads < 1 || n_v_heads > 1024 || n_v_heads % n_k_heads)
    return 0;
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return 0;
  return ws_plan(chunk_slots(n_tokens, n_seqs), n_seqs, n_k_heads, n_v_heads, dk).total;
}

extern "C" int redlite_delta_prefill(int32_t dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                     const void *v, int64_t v_stride, const float *g, const float *beta,
                                     const int32_t *cu, int32_t n_seqs, int32_t n_tokens, int32_t n_k_heads,
                                     int32_t n_v_heads, int32_t dk, int32_t dv, float scale, float qk_eps,
                                     const float *state_in, float *state_out, const int32_t *slots, int64_t n_slots,
                                     void *out, int64_t out_stride, void *workspace, size_t workspace_bytes,
                                     int32_t *status, void *stream) {
  const int rc = delta_check(dtype, q, q_stride, k, k_stride, v, v_stride, g, beta, n_seqs, n_tokens, n_k_heads,
                             n_v_heads, dk, dv, scale, state_in, state_out, slots, n_slots, out, out_stride);
  if (rc <= 0) return rc;
  if (!cu || !workspace || ((uintptr_t)workspace & 255)) return REDLITE_EINVAL;
  const int64_t slots_n = chunk_slots(n_tokens, n_seqs);
  if ((int64_t)n_seqs * n_v_heads * (dv / kCols) >= ((int64_t)1 << 31) - 1 || slots_n * n_k_heads >= ((int64_t)1 << 31) - 1)
    return REDLITE_EUNSUPPORTED;
  const WsPlan w = ws_plan(slots_n, n_seqs, n_k_heads, n_v_heads, dk);
  if (workspace_bytes < w.total) return REDLITE_ENOMEM;
  DeltaArgs a = {};
  a.q = q, a.k = k, a.v = v, a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.out_stride = out_stride, a.g = g, a.beta = beta, a.cu = cu, a.slots = slots;
  a.n_seqs = n_seqs, a.n_tokens = n_tokens, a.n_k = n_k_heads, a.n_v = n_v_heads, a.dk = dk, a.dv = dv;
  a.scale = scale, a.qk_eps = qk_eps, a.state_in = state_in, a.state_out = state_out, a.n_slots = n_slots;
  a.out = out, a.ws = (uint8_t *)workspace, a.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  // 16-bit keys and queries are one fp16 part (exact once scaled), fp32 ones two
  if (dtype == REDLITE_T_F32) e = launch_prefill_dk<float, 2>(a, w, s);
  else if (dtype == REDLITE_T_BF16) e = launch_prefill_dk<__nv_bfloat16, 1>(a, w, s);
  else e = launch_prefill_dk<__half, 1>(a, w, s);
  return e == cudaSuccess ? REDLITE_OK : REDLITE_ECUDA;
}
