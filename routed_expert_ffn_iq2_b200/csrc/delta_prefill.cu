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
// once; delta_chain_kernel then walks the chunks of a sequence.  Everything
// in the chain is linear in the value columns, so a warp takes 16 of them:
// it keeps S^T [16 x dk] in fp32 accumulators and chains
//   S^T K^T -> D^T -> S^T, O^T
// where each product's result is, register for register, the next one's A
// operand (m16n8k16, M = value columns).  Warps exchange nothing; K, Q, T, P
// and the per-token factors come through shared memory by bulk copies.  The
// chain of one head is serial, so the warps per block follow the number of
// chains: few chains go out as two-warp blocks over all multiprocessors.
//
// Precision: bf16 keys and queries enter the products unrounded; everything
// fp32 that meets a product (the state, T, P, the updates; fp32 and fp16
// keys and queries) is split in two bf16 parts, hi hi + hi lo + lo hi, which
// leaves out 2^-17 of each term.  Norms (q, k over their length) and decays
// multiply results per token in fp32, never the bf16 operands.  Sums of log
// decays are fp64 and only their differences are rounded.
//
// A chunk that meets a NaN or an infinity is walked token by token, so that
// what lies behind a token never reaches it.
#include "delta.cuh"

namespace redlite {
namespace {

constexpr int C = 64;  // tokens of a chunk

// Per (chunk, value head): T and P as two bf16 planes each, the ten 16 x 16
// blocks on and under the diagonal (row by row of blocks), a block's rows 32
// bytes, their two 16-byte pieces swapped in every other group of four rows
// (no bank conflicts); then eight per-token factors.
constexpr int kPlane = 10 * 512;
enum { kThi, kTlo, kPhi, kPlo, kPlanes };
enum { fBeta, fR, fQ, fK, fAlpha, fNk, fNq, fLast, kFactors };  // fLast: [0] = exp(c_last)
constexpr int kHeadBlock = kPlanes * kPlane + kFactors * C * 4;

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
  size_t kq, head, total;
};
inline WsPlan ws_plan(int64_t slots, int n_k, int n_v, int dk) {
  WsPlan w;
  w.kq = 0;
  w.head = align256((size_t)slots * n_k * (2 * 2 * C * (size_t)dk * 2));
  w.total = align256(w.head + (size_t)slots * n_v * kHeadBlock);
  return w;
}

// ------------------------------------------------------------------- prep

// Row i of T = (I + A)^-1 in registers, from T (I + A) = I:
//   t_j = (i == j) - sum_{k > j} t_k A_kj,  j = N - 1 .. 0
// A^T is read as broadcasts; rows above N are zero for this warp.
template <int N>
__device__ __forceinline__ void solve_row(const float *at, int i, float (&t)[C]) {
#pragma unroll
  for (int j = N - 1; j >= 0; --j) {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int k4 = j / 4; k4 < N / 4; ++k4) {
      const float4 x = *reinterpret_cast<const float4 *>(at + j * 68 + 4 * k4);
      if (4 * k4 > j) s0 = fmaf(t[4 * k4], x.x, s0);
      if (4 * k4 + 1 > j) s1 = fmaf(t[4 * k4 + 1], x.y, s1);
      if (4 * k4 + 2 > j) s2 = fmaf(t[4 * k4 + 2], x.z, s2);
      if (4 * k4 + 3 > j) s3 = fmaf(t[4 * k4 + 3], x.w, s3);
    }
    t[j] = (i == j ? 1.f : 0.f) - ((s0 + s1) + (s2 + s3));
  }
}

// One block per (chunk slot, key head), four warps: warp w takes rows 16 w ..
// of the two Gram matrices; then the value heads of the key head go in pairs,
// two warps (64 rows of T) each.
template <typename T, int NK, int DK>
__global__ void __launch_bounds__(128) delta_prep_kernel(const DeltaArgs a, const WsPlan w) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ double sc[2][C];
  __shared__ float snk[C], snq[C], sb[2][C], sg[2][C];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int64_t slot = blockIdx.x;
  const int kh = blockIdx.y;
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

  // ---- K and Q rows: bf16 parts into shared memory and the workspace, sums of squares
  constexpr int kPieces = DK / 8, kTile = C * DK * 2;
  uint8_t *kq = a.ws + w.kq + ((size_t)slot * a.n_k + kh) * kq_bytes<NK, DK>();
#pragma unroll 4
  for (int it = 0; it < 2 * C * kPieces / 128; ++it) {
    const int id = it * 128 + tid, which = id / (C * kPieces), row = id / kPieces % C, piece = id % kPieces;
    float x[8];
    if (row < n) {
      load8<T>((which ? (const T *)a.q + (row0 + row) * a.q_stride : (const T *)a.k + (row0 + row) * a.k_stride) +
                   (int64_t)kh * DK + piece * 8,
               x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = 1; o < kPieces; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (piece == 0) {
      const float f = a.qk_eps >= 0.f ? 1.f / sqrtf(ss + a.qk_eps) : 1.f;
      (which ? snq : snk)[row] = f;
    }
#pragma unroll
    for (int p = 0; p < NK; ++p) {
      uint4 v;
      v.x = pack_bf16(x[0], x[1]), v.y = pack_bf16(x[2], x[3]);
      v.z = pack_bf16(x[4], x[5]), v.w = pack_bf16(x[6], x[7]);
      const uint32_t off = (which * NK + p) * kTile + kq_off<DK>(row, piece);
      *reinterpret_cast<uint4 *>(smem + off) = v;
      *reinterpret_cast<uint4 *>(kq + off) = v;
      x[0] -= bf16_lo(v.x), x[1] -= bf16_hi(v.x), x[2] -= bf16_lo(v.y), x[3] -= bf16_hi(v.y);
      x[4] -= bf16_lo(v.z), x[5] -= bf16_hi(v.z), x[6] -= bf16_lo(v.w), x[7] -= bf16_hi(v.w);
    }
  }
  __syncthreads();
  // ---- rows 16 warp .. of K K^T and Q K^T
  float G[8][4], H[8][4];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) G[t][e] = H[t][e] = 0.f;
  const uint32_t base = ptx::smem_u32(smem);
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t ak[NK][4], aq[NK][4];
    const int arow = 16 * warp + (lane & 15), apiece = 2 * ks + (lane >> 4);
#pragma unroll
    for (int p = 0; p < NK; ++p) {
      ldsm4(base + p * kTile + kq_off<DK>(arow, apiece), ak[p][0], ak[p][1], ak[p][2], ak[p][3]);
      ldsm4(base + (NK + p) * kTile + kq_off<DK>(arow, apiece), aq[p][0], aq[p][1], aq[p][2], aq[p][3]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t > warp) break;  // columns behind the rows are not needed
      const int brow = 16 * t + (lane & 7) + ((lane >> 4) << 3), bpiece = 2 * ks + ((lane >> 3) & 1);
#pragma unroll
      for (int p = 0; p < NK; ++p) {
        uint32_t b[4];
        ldsm4(base + p * kTile + kq_off<DK>(brow, bpiece), b[0], b[1], b[2], b[3]);
#pragma unroll
        for (int s = 0; s + p < NK; ++s)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_bf16(G[2 * t + u], ak[s][0], ak[s][1], ak[s][2], ak[s][3], b[2 * u], b[2 * u + 1]);
            mma_bf16(H[2 * t + u], aq[s][0], aq[s][1], aq[s][2], aq[s][3], b[2 * u], b[2 * u + 1]);
          }
      }
    }
  }
  float *at = reinterpret_cast<float *>(smem);  // A^T of two heads, [64][68] each (the tiles are read)
  const int per = a.n_v / a.n_k;
  for (int h0 = 0; h0 < per; h0 += 2) {
    __syncthreads();
    // ---- factors per token: thread t of a half takes token t of its head
    const int half = tid >> 6, tok = tid & 63, head = kh * per + h0 + half;
    const bool have = h0 + half < per;
    float g = 0.f, b = 0.f;
    if (have && tok < n) {
      g = delta_clamp_g(__ldg(a.g + (row0 + tok) * a.n_v + head));
      b = __ldg(a.beta + (row0 + tok) * a.n_v + head);
    }
    double sum = g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    sc[half][tok] = sum, sb[half][tok] = b, sg[half][tok] = g;
    __syncthreads();
    if (tok >= 32) sum += sc[half][31];
    __syncthreads();
    sc[half][tok] = sum;
    __syncthreads();
    if (have) {
      float *f = reinterpret_cast<float *>(a.ws + w.head + ((size_t)slot * a.n_v + head) * kHeadBlock +
                                           kPlanes * kPlane);
      const double last = sc[half][C - 1];
      const float gamma = expf((float)sum);
      f[fBeta * C + tok] = b;
      f[fR * C + tok] = b * gamma * snk[tok];
      f[fQ * C + tok] = tok < n ? a.scale * snq[tok] * gamma : 0.f;
      f[fK * C + tok] = tok < n ? snk[tok] * expf((float)(last - sum)) : 0.f;
      f[fAlpha * C + tok] = expf(g);
      f[fNk * C + tok] = snk[tok];
      f[fNq * C + tok] = a.scale * snq[tok];
      f[fLast * C + tok] = expf((float)last);
    }
    // ---- A^T (shared) and P (workspace) of both heads
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (h0 + q >= per) break;
      uint8_t *blk = a.ws + w.head + ((size_t)slot * a.n_v + kh * per + h0 + q) * kHeadBlock;
      float *ah = at + q * C * 68;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * warp + r + 8 * (e >> 1), j = 8 * t + 2 * c + (e & 1);
          float x = 0.f, y = 0.f;
          if (j <= i) {
            const float dec = expf((float)(sc[q][i] - sc[q][j])) * snk[j];
            y = a.scale * snq[i] * dec * H[t][e];
            if (j < i) x = sb[q][i] * snk[i] * dec * G[t][e];
          }
          ah[j * 68 + i] = x;
          pv[e] = y;
        }
        if ((t >> 1) <= warp) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t ph, pl;
            split_bf16(pv[2 * e], pv[2 * e + 1], ph, pl);
            const uint32_t off = tp_off(16 * warp + r + 8 * e, t) + 4 * c;
            *reinterpret_cast<uint32_t *>(blk + kPhi * kPlane + off) = ph;
            *reinterpret_cast<uint32_t *>(blk + kPlo * kPlane + off) = pl;
          }
        }
      }
    }
    __syncthreads();
    // ---- T, a row per thread
    if (have) {
      float t[C];
      const int i = tok;
      if (tok < 32) {
#pragma unroll
        for (int j = 32; j < C; ++j) t[j] = 0.f;
        solve_row<32>(at + half * C * 68, i, t);
      } else {
        solve_row<64>(at + half * C * 68, i, t);
      }
      uint8_t *blk = a.ws + w.head + ((size_t)slot * a.n_v + head) * kHeadBlock;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        if ((p >> 1) > (i >> 4)) break;
        uint4 vh, vl;
        split_bf16(t[8 * p], t[8 * p + 1], vh.x, vl.x);
        split_bf16(t[8 * p + 2], t[8 * p + 3], vh.y, vl.y);
        split_bf16(t[8 * p + 4], t[8 * p + 5], vh.z, vl.z);
        split_bf16(t[8 * p + 6], t[8 * p + 7], vh.w, vl.w);
        *reinterpret_cast<uint4 *>(blk + kThi * kPlane + tp_off(i, p)) = vh;
        *reinterpret_cast<uint4 *>(blk + kTlo * kPlane + tp_off(i, p)) = vl;
      }
    }
  }
}

// ------------------------------------------------------------------ chain

template <typename T>
struct VTile {
  static constexpr int kPitch = sizeof(T) == 4 ? 20 : 24;  // elements per token row of 16 (no bank conflicts)
  static constexpr int kBytes = C * kPitch * (int)sizeof(T);
};

template <int NK, int DK>
__host__ __device__ constexpr int stage_bytes() {
  return kq_bytes<NK, DK>() + kHeadBlock;
}
constexpr int kStages = 2;
template <typename T, int NK, int DK, int W>
__host__ __device__ constexpr int chain_smem() {
  return kStages * stage_bytes<NK, DK>() + 2 * W * VTile<T>::kBytes + 64;
}

// W chain warps and one that issues the copies.  Block: (slice of 16 W value
// columns, value head, sequence).
template <typename T, int NK, int DK, int W>
__global__ void __launch_bounds__(32 * (W + 1), 1) delta_chain_kernel(const DeltaArgs a, const WsPlan w) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStage = stage_bytes<NK, DK>(), kTile = C * DK * 2, NT = DK / 8;
  uint8_t *vbuf = smem + kStages * kStage;
  uint64_t *full = reinterpret_cast<uint64_t *>(vbuf + 2 * W * VTile<T>::kBytes), *empty = full + kStages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int slices = a.dv / (16 * W);
  const int slice = blockIdx.x % slices, head = blockIdx.x / slices % a.n_v, seq = blockIdx.x / (slices * a.n_v);
  const int kh = head / (a.n_v / a.n_k);
  if (tid == 0)
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(full + i, 1), ptx::mbar_init(empty + i, W);
  ptx::mbar_fence_init();
  // in front of every way out: this grid must not end before the one that
  // writes the workspace
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t slot = delta_slot(a, seq);
  __syncthreads();
  const Span sp = seq_span(a, seq);
  if (sp.len < 0) {
    if (tid == 0) set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
    return;
  }
  const int n_chunks = (sp.len + C - 1) / C;
  if (slot < 0) {
    for (int i = tid; i < sp.len * 16 * W; i += blockDim.x)
      ((T *)a.out)[(int64_t)(sp.start + i / (16 * W)) * a.out_stride + (int64_t)head * a.dv + slice * 16 * W +
                   i % (16 * W)] = from_f32<T>(0.f);
    return;
  }
  const int64_t slot0 = (int64_t)(sp.start / C) + seq;
  if (warp == W) {
    if (lane == 0)
      for (int i = 0; i < n_chunks; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !ptx::mbar_wait_suspend(empty + st, ((i / kStages) & 1) ^ 1)) {
          set_status(a.status, REDLITE_STATUS_TIMEOUT);
          break;
        }
        uint8_t *dst = smem + st * kStage;
        ptx::mbar_expect_tx(full + st, kStage);
        ptx::bulk_g2s(dst, a.ws + w.kq + ((size_t)(slot0 + i) * a.n_k + kh) * kq_bytes<NK, DK>(), kq_bytes<NK, DK>(),
                      full + st);
        ptx::bulk_g2s(dst + kq_bytes<NK, DK>(), a.ws + w.head + ((size_t)(slot0 + i) * a.n_v + head) * kHeadBlock,
                      kHeadBlock, full + st);
      }
    return;
  }

  // ---- state: rows = value columns col + r, col + r + 8; columns = key index
  const int col = slice * 16 * W + 16 * warp;
  float S[NT][4];
  const int64_t s_at = (slot * a.n_v + head) * (int64_t)DK * a.dv + col;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[t][e] = a.state_in
                    ? __ldg(a.state_in + s_at + (int64_t)(8 * t + 2 * c + (e & 1)) * a.dv + r + 8 * (e >> 1))
                    : 0.f;
  // value rows of a chunk, this warp's 16 columns: asynchronous copies into a
  // buffer of its own, zeros behind the end
  constexpr int kPer = 16 * (int)sizeof(T) / 16;  // 16-byte pieces per row
  constexpr int kPitch = VTile<T>::kPitch;
  auto fetch_v = [&](int i) {
    const uint32_t dst = ptx::smem_u32(vbuf + (2 * warp + (i & 1)) * VTile<T>::kBytes);
    const int n = min(C, sp.len - i * C);
#pragma unroll
    for (int it = 0; it < C * kPer / 32; ++it) {
      const int id = it * 32 + lane, row = id / kPer, piece = id % kPer;
      const T *src = (const T *)a.v + (int64_t)(sp.start + i * C + (row < n ? row : 0)) * a.v_stride +
                     (int64_t)head * a.dv + col + piece * (16 / (int)sizeof(T));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       dst + (uint32_t)(row * kPitch * (int)sizeof(T) + piece * 16)),
                   "l"(src), "r"(row < n ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (n_chunks > 0) fetch_v(0);

  for (int i = 0; i < n_chunks; ++i) {
    const int st = i % kStages, n = min(C, sp.len - i * C);
    const uint32_t sK = ptx::smem_u32(smem + st * kStage), sQ = sK + NK * kTile;
    const uint32_t sT = sK + kq_bytes<NK, DK>(), sP = sT + kPhi * kPlane;
    const float *f = reinterpret_cast<const float *>(smem + st * kStage + kq_bytes<NK, DK>() + kPlanes * kPlane);
    T *vt = reinterpret_cast<T *>(vbuf + (2 * warp + (i & 1)) * VTile<T>::kBytes);
    if (i + 1 < n_chunks) {
      fetch_v(i + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if (!__all_sync(0xffffffffu, ptx::mbar_wait_suspend(full + st, (i / kStages) & 1))) {
      if (lane == 0) set_status(a.status, REDLITE_STATUS_TIMEOUT);
      break;
    }
    __syncwarp();
    float R[8][4], O[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) R[t][e] = O[t][e] = 0.f;
    // ---- S^T K^T and S^T Q^T
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t h[4], l[4];
      split_bf16(S[2 * ks][0], S[2 * ks][1], h[0], l[0]);
      split_bf16(S[2 * ks][2], S[2 * ks][3], h[1], l[1]);
      split_bf16(S[2 * ks + 1][0], S[2 * ks + 1][1], h[2], l[2]);
      split_bf16(S[2 * ks + 1][2], S[2 * ks + 1][3], h[3], l[3]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t off = kq_off<DK>(16 * t + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1));
#pragma unroll
        for (int p = 0; p < NK; ++p) {
          uint32_t b[4], d[4];
          ldsm4(sK + p * kTile + off, b[0], b[1], b[2], b[3]);
          ldsm4(sQ + p * kTile + off, d[0], d[1], d[2], d[3]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_bf16(R[2 * t + u], h[0], h[1], h[2], h[3], b[2 * u], b[2 * u + 1]);
            mma_bf16(O[2 * t + u], h[0], h[1], h[2], h[3], d[2 * u], d[2 * u + 1]);
            if (p == 0) {
              mma_bf16(R[2 * t + u], l[0], l[1], l[2], l[3], b[2 * u], b[2 * u + 1]);
              mma_bf16(O[2 * t + u], l[0], l[1], l[2], l[3], d[2 * u], d[2 * u + 1]);
            }
          }
        }
      }
    }
    // ---- beta V - beta exp(c) K S0, and the state's part of the output
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int j = 8 * t + 2 * c;
      const float2 fb = *reinterpret_cast<const float2 *>(f + fBeta * C + j);
      const float2 fr = *reinterpret_cast<const float2 *>(f + fR * C + j);
      const float2 fq = *reinterpret_cast<const float2 *>(f + fQ * C + j);
      R[t][0] = fmaf(fb.x, to_f32(vt[j * kPitch + r]), -fr.x * R[t][0]);
      R[t][1] = fmaf(fb.y, to_f32(vt[(j + 1) * kPitch + r]), -fr.y * R[t][1]);
      R[t][2] = fmaf(fb.x, to_f32(vt[j * kPitch + r + 8]), -fr.x * R[t][2]);
      R[t][3] = fmaf(fb.y, to_f32(vt[(j + 1) * kPitch + r + 8]), -fr.y * R[t][3]);
      O[t][0] *= fq.x, O[t][1] *= fq.y, O[t][2] *= fq.x, O[t][3] *= fq.y;
    }
    // ---- D^T = R^T T^T (T is lower triangular: 10 of 16 blocks)
    float D[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) D[t][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t h[4], l[4];
      split_bf16(R[2 * ks][0], R[2 * ks][1], h[0], l[0]);
      split_bf16(R[2 * ks][2], R[2 * ks][3], h[1], l[1]);
      split_bf16(R[2 * ks + 1][0], R[2 * ks + 1][1], h[2], l[2]);
      split_bf16(R[2 * ks + 1][2], R[2 * ks + 1][3], h[3], l[3]);
#pragma unroll
      for (int t = ks; t < 4; ++t) {
        const uint32_t off = tp_off(16 * t + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1));
        uint32_t b[4], d[4];
        ldsm4(sT + kThi * kPlane + off, b[0], b[1], b[2], b[3]);
        ldsm4(sT + kTlo * kPlane + off, d[0], d[1], d[2], d[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mma_bf16(D[2 * t + u], h[0], h[1], h[2], h[3], b[2 * u], b[2 * u + 1]);
          mma_bf16(D[2 * t + u], l[0], l[1], l[2], l[3], b[2 * u], b[2 * u + 1]);
          mma_bf16(D[2 * t + u], h[0], h[1], h[2], h[3], d[2 * u], d[2 * u + 1]);
        }
      }
    }
    // a NaN or an infinity anywhere: x - x is not 0
    float odd = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) odd += D[t][e] - D[t][e];
    const bool walk = __any_sync(0xffffffffu, !(odd == 0.f));
    __syncwarp();  // V is read: its buffer takes the outputs
    if (!walk) {
      const float last = f[fLast * C];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t][e] *= last;
      // ---- O^T += D^T P^T,  S^T += (D exp(c_last - c))^T K
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t h[4], l[4];
        split_bf16(D[2 * ks][0], D[2 * ks][1], h[0], l[0]);
        split_bf16(D[2 * ks][2], D[2 * ks][3], h[1], l[1]);
        split_bf16(D[2 * ks + 1][0], D[2 * ks + 1][1], h[2], l[2]);
        split_bf16(D[2 * ks + 1][2], D[2 * ks + 1][3], h[3], l[3]);
#pragma unroll
        for (int t = ks; t < 4; ++t) {
          const uint32_t off = tp_off(16 * t + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1));
          uint32_t b[4], d[4];
          ldsm4(sP + off, b[0], b[1], b[2], b[3]);
          ldsm4(sP + kPlane + off, d[0], d[1], d[2], d[3]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_bf16(O[2 * t + u], h[0], h[1], h[2], h[3], b[2 * u], b[2 * u + 1]);
            mma_bf16(O[2 * t + u], l[0], l[1], l[2], l[3], b[2 * u], b[2 * u + 1]);
            mma_bf16(O[2 * t + u], h[0], h[1], h[2], h[3], d[2 * u], d[2 * u + 1]);
          }
        }
        const float2 f0 = *reinterpret_cast<const float2 *>(f + fK * C + 16 * ks + 2 * c);
        const float2 f1 = *reinterpret_cast<const float2 *>(f + fK * C + 16 * ks + 8 + 2 * c);
        split_bf16(D[2 * ks][0] * f0.x, D[2 * ks][1] * f0.y, h[0], l[0]);
        split_bf16(D[2 * ks][2] * f0.x, D[2 * ks][3] * f0.y, h[1], l[1]);
        split_bf16(D[2 * ks + 1][0] * f1.x, D[2 * ks + 1][1] * f1.y, h[2], l[2]);
        split_bf16(D[2 * ks + 1][2] * f1.x, D[2 * ks + 1][3] * f1.y, h[3], l[3]);
#pragma unroll
        for (int t = 0; t < NT / 2; ++t) {
          const uint32_t off = kq_off<DK>(16 * ks + (lane & 15), 2 * t + (lane >> 4));
#pragma unroll
          for (int p = 0; p < NK; ++p) {
            uint32_t b[4];
            ldsm4t(sK + p * kTile + off, b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              mma_bf16(S[2 * t + u], h[0], h[1], h[2], h[3], b[2 * u], b[2 * u + 1]);
              if (p == 0) mma_bf16(S[2 * t + u], l[0], l[1], l[2], l[3], b[2 * u], b[2 * u + 1]);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vt[(8 * t + 2 * c + (e & 1)) * kPitch + r + 8 * (e >> 1)] = from_f32<T>(O[t][e]);
    } else {
      // token by token from the state in front of the chunk
      for (int j = 0; j < n; ++j) {
        float ks0 = 0.f, ks1 = 0.f;
        const float al = f[fAlpha * C + j], be = f[fBeta * C + j], nk = f[fNk * C + j], nq = f[fNq * C + j];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float2 k = make_float2(0.f, 0.f);
#pragma unroll
          for (int p = 0; p < NK; ++p) {
            const uint32_t x = ptx::lds32(sK + p * kTile + kq_off<DK>(j, t) + 4 * c);
            k.x += bf16_lo(x), k.y += bf16_hi(x);
          }
          ks0 = fmaf(k.x, S[t][0], fmaf(k.y, S[t][1], ks0));
          ks1 = fmaf(k.x, S[t][2], fmaf(k.y, S[t][3], ks1));
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          ks0 += __shfl_xor_sync(0xffffffffu, ks0, o);
          ks1 += __shfl_xor_sync(0xffffffffu, ks1, o);
        }
        const float d0 = be * (to_f32(vt[j * kPitch + r]) - al * nk * ks0) * nk;
        const float d1 = be * (to_f32(vt[j * kPitch + r + 8]) - al * nk * ks1) * nk;
        float o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float2 k = make_float2(0.f, 0.f), q = k;
#pragma unroll
          for (int p = 0; p < NK; ++p) {
            const uint32_t x = ptx::lds32(sK + p * kTile + kq_off<DK>(j, t) + 4 * c);
            const uint32_t y = ptx::lds32(sQ + p * kTile + kq_off<DK>(j, t) + 4 * c);
            k.x += bf16_lo(x), k.y += bf16_hi(x), q.x += bf16_lo(y), q.y += bf16_hi(y);
          }
          S[t][0] = fmaf(al, S[t][0], k.x * d0), S[t][1] = fmaf(al, S[t][1], k.y * d0);
          S[t][2] = fmaf(al, S[t][2], k.x * d1), S[t][3] = fmaf(al, S[t][3], k.y * d1);
          o0 = fmaf(q.x, S[t][0], fmaf(q.y, S[t][1], o0));
          o1 = fmaf(q.x, S[t][2], fmaf(q.y, S[t][3], o1));
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          o0 += __shfl_xor_sync(0xffffffffu, o0, o);
          o1 += __shfl_xor_sync(0xffffffffu, o1, o);
        }
        __syncwarp();
        if (c == 0) vt[j * kPitch + r] = from_f32<T>(o0 * nq), vt[j * kPitch + r + 8] = from_f32<T>(o1 * nq);
        __syncwarp();
      }
    }
    // ---- the stage is free; outputs leave as 16-byte pieces of rows
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty + st);
#pragma unroll
    for (int it = 0; it < C * kPer / 32; ++it) {
      const int id = it * 32 + lane, row = id / kPer, piece = id % kPer;
      if (row < n) {
        const uint4 v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(vt) +
                                                         row * kPitch * (int)sizeof(T) + piece * 16);
        *reinterpret_cast<uint4 *>((T *)a.out + (int64_t)(sp.start + i * C + row) * a.out_stride +
                                   (int64_t)head * a.dv + col + piece * (16 / (int)sizeof(T))) = v;
      }
    }
    __syncwarp();  // the buffer is read before the copies of the chunk after next go into it
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      a.state_out[s_at + (int64_t)(8 * t + 2 * c + (e & 1)) * a.dv + r + 8 * (e >> 1)] = S[t][e];
}

template <typename T, int NK, int DK, int W>
cudaError_t launch_chain(const DeltaArgs &a, const WsPlan &w, cudaStream_t s) {
  constexpr int smem = chain_smem<T, NK, DK, W>();
  static_assert(smem <= 227 * 1024, "shared memory of a chain block");
  cudaError_t e = cudaFuncSetAttribute(delta_chain_kernel<T, NK, DK, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.n_seqs * a.n_v * (a.dv / (16 * W))));
  cfg.blockDim = dim3(32 * (W + 1));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = a.n_tokens > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, delta_chain_kernel<T, NK, DK, W>, a, w);
}

template <typename T, int NK, int DK>
cudaError_t launch_prefill(const DeltaArgs &a, const WsPlan &w, int sms, cudaStream_t s) {
  if (a.n_tokens > 0) {
    constexpr int tiles = kq_bytes<NK, DK>(), at = 2 * C * 68 * 4, smem = tiles > at ? tiles : at;
    cudaError_t e =
        cudaFuncSetAttribute(delta_prep_kernel<T, NK, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<T, NK, DK>
        <<<dim3((unsigned)chunk_slots(a.n_tokens, a.n_seqs), (unsigned)a.n_k), 128, smem, s>>>(a, w);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // two warps per block while that does not make more blocks than there are
  // multiprocessors (a chain is serial: spread the few there are), else four
  const int64_t chains = (int64_t)a.n_seqs * a.n_v * (a.dv / 32);
  if (chains <= sms) return launch_chain<T, NK, DK, 2>(a, w, s);
  return launch_chain<T, NK, DK, 4>(a, w, s);
}

template <typename T, int NK>
cudaError_t launch_prefill_dk(const DeltaArgs &a, const WsPlan &w, int sms, cudaStream_t s) {
  return a.dk == 128 ? launch_prefill<T, NK, 128>(a, w, sms, s) : launch_prefill<T, NK, 64>(a, w, sms, s);
}

}  // namespace
}  // namespace redlite

using namespace redlite;

extern "C" size_t redlite_delta_workspace_bytes(int32_t n_tokens, int32_t n_seqs, int32_t n_k_heads, int32_t n_v_heads,
                                                int32_t dk, int32_t dv) {
  if (n_tokens < 0 || n_seqs < 0 || n_k_heads < 1 || n_v_heads < 1 || n_v_heads > 1024 || n_v_heads % n_k_heads)
    return 0;
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return 0;
  return ws_plan(chunk_slots(n_tokens, n_seqs), n_k_heads, n_v_heads, dk).total;
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
  if ((int64_t)n_seqs * n_v_heads * (dv / 32) >= ((int64_t)1 << 31) - 1 || slots_n >= ((int64_t)1 << 31) - 1)
    return REDLITE_EUNSUPPORTED;
  const WsPlan w = ws_plan(slots_n, n_k_heads, n_v_heads, dk);
  if (workspace_bytes < w.total) return REDLITE_ENOMEM;
  const int sms = sm_count();
  if (sms <= 0) return REDLITE_ECUDA;
  DeltaArgs a = {};
  a.q = q, a.k = k, a.v = v, a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.out_stride = out_stride, a.g = g, a.beta = beta, a.cu = cu, a.slots = slots;
  a.n_seqs = n_seqs, a.n_tokens = n_tokens, a.n_k = n_k_heads, a.n_v = n_v_heads, a.dk = dk, a.dv = dv;
  a.scale = scale, a.qk_eps = qk_eps, a.state_in = state_in, a.state_out = state_out, a.n_slots = n_slots;
  a.out = out, a.ws = (uint8_t *)workspace, a.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  // fp16 keys and queries are held exactly by two bf16 parts, fp32 ones to 2^-17
  if (dtype == REDLITE_T_F32) e = launch_prefill_dk<float, 2>(a, w, sms, s);
  else if (dtype == REDLITE_T_BF16) e = launch_prefill_dk<__nv_bfloat16, 1>(a, w, sms, s);
  else e = launch_prefill_dk<__half, 2>(a, w, sms, s);
  return e == cudaSuccess ? REDLITE_OK : REDLITE_ECUDA;
}
