// kv4_decode.cu -- attention of one query token per sequence over the paged
// 4-bit key/value cache (redlite_kv4_decode).  ("Red Lite dev16 -- complete
// full-attention parity", section "Pinned full-attention graph": grouped
// heads over a K/V cache.)
//
//   s_t = scale * q . K_t,  p = softmax(s),  o = sum_t p_t V_t,
//   K_t, V_t = m + d * code per group of 32 values.
//
// The floor is the cache's bytes (1.25 D per token and key/value head, both
// sides), each read once; what stands beside it is the conversion of the
// codes, so the kernel never forms the values.  Codes go to the tensor cores
// as exact small numbers (a shift, an and-or for two of them or more):
//   q . K_t   = sum_g 16 d_tg (q_g . (1 + code / 16)) + (m_tg - 16 d_tg) sum(q_g)
//   o of g    = sum_t (p_t d_tg) (code - 8) + sum_t p_t (m_tg + 8 d_tg)
// with the sums over m and d as products of their own (their stored fp16
// numbers are operands as they lie).  Where a code stands as 1 + code / 256
// (that needs no shift of its own), the query's element is 16 times as large.
// Two forms of the rest:
//   16-bit activations  a head's query scaled by a power of two into one fp16
//               part (exact for elements down to 2^-19 of the head's largest,
//               2^-22 for bf16; below, off by 2^-30 of that at most); p and p d
//               are rounded to fp16 (2^-10 of each term's p d (code - 8) in all
//               at most, of either sign; the sum over p m and the softmax's own
//               sum keep p whole).  The reference of the softmax is kept so that
//               neither p nor p d leaves fp16:
//               p <= 2^15 / max(1, |d|) for the largest |d| met so far.  Small
//               steps count as 2^lift times themselves, so that p d stays above
//               fp16's subnormal numbers: what falls below them all the same is
//               off by 2^-22 of the largest p d at most (without: by 2^-10 of it
//               for steps of 2^-21, 1.8 times the bound of 30,000 such tokens)
//   fp32        the query in three bf16 parts (exact); 16 d p and p in three.
//               Codes are centred in the scores too: q . K_t = sum_g 16 d_tg (q_g
//               . (code - 8) / 16) + (m_tg + 8 d_tg) sum(q_g), so that no sum is
//               much larger than what it stands for.
// Sums, maxima and the running softmax statistics are fp32.
//
// Split: the units of all sequences (128 tokens of one key/value head and up
// to 8 of its query heads; a sequence starts with kEntry units without tokens,
// which stand for the time its first tiles and its result take) form one list,
// cut evenly over a fixed grid; a
// block joins its eight warps (16 tokens each, tiles streamed into a
// per-warp ring by bulk copies) at the end of each run of units and writes
// either the output or one of its two partial results, which kv4_join_kernel
// adds up in a fixed order: no atomics, nothing kept from call to call.
//
// Measured (one B200, floor at 6550 GB/s in brackets): 16 contexts of 49k to
// 66k tokens, 32 heads on 8 of 128, fp16: 331 us, 3.5 TB/s [178 us]; 64 ragged
// contexts up to 8k, 16 heads on 2 of 256, bf16: 59 us [24 us]; one of 700
// tokens, fp32: 12 us.  No unit is saturated: integer units 53% of their rate,
// DRAM 34%, tensor cores 17%, 2.1 to 2.3 instructions a cycle.  With four warps
// a scheduler (128 registers, what the accumulators leave) latency shows: of a
// warp's 6 cycles an instruction it waits 1.4 for the one before it, 0.8 for
// the integer units and 0.4 to 0.8 each for shared memory, tiles and the other
// warps.  Heads of 256 spill some of their registers (200 to 350 bytes).  More
// than 8 query heads per key/value head go in blocks of 8, each of which reads
// and converts the cache for itself: 9 to 16 heads have twice the floor.
#include "kv4.cuh"

namespace redlite {
namespace {

constexpr int kWarps = 8;
constexpr int kUnit = 16 * kWarps;  // tokens of a unit
// Units that a sequence counts for on top: with none, a block of many short
// sequences ran 30% longer than the rest (64 ragged contexts: 71 us; 4: 62 us;
// 8: 68 us).
constexpr int kEntry = 4;
constexpr float kLazy = 8.f;        // log2 by which scores may pass the reference before sums are rescaled
constexpr float kTop = 15.f;        // log2 that p, and p |d|, stay below in fp16
// Steps are lifted where the largest of a run's first tile is below
// 2^(kLiftBelow - 1) (values of 2^-6 and less); at 2^-9 a p d of the largest p
// (2^6 at least) is 2^11 above fp16's smallest normal number.
constexpr int kLiftBelow = -8;

struct DecArgs {
  const void *q;
  void *out;
  int64_t q_stride, out_stride;
  const uint8_t *cache;
  const int32_t *table, *lens;
  int n_seqs, n_heads, n_kv, ratio, hb_count;  // hb_count: blocks of 8 query heads per key/value head
  int page_size, max_pages;
  int64_t n_pages;
  float scale_log2;
  float *part;  // [2 grid][8 * D + 16]
  int grid;
  int32_t *status;
};

// Units of a sequence, the entry ones included (0: it has none).
__device__ __forceinline__ int seq_units(const DecArgs &a, int s) {
  const int n = __ldg(a.lens + s);
  if (n <= 0 || (int64_t)n > (int64_t)a.max_pages * a.page_size) return 0;
  return (n - 1) / kUnit + 1 + kEntry;  // (a sum with n may leave 32 bits)
}

// Sum of the units of all sequences (of one head block), and where unit u of
// the list over sequences falls: the sequence and the units in front of it.
// Every thread of the block calls it; `sm` holds 4 + blockDim / 32 words.
__device__ __forceinline__ int64_t scan_units(const DecArgs &a, int64_t *sm) {
  // thread t counts sequences t * per .. ; their exclusive prefix in registers
  const int per = (a.n_seqs + blockDim.x - 1) / blockDim.x;
  const int s0 = min(a.n_seqs, (int)threadIdx.x * per), s1 = min(a.n_seqs, s0 + per);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += seq_units(a, s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sm[4 + warp] = inc;
  __syncthreads();
  int64_t base = 0, total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) base += sm[4 + w];
    total += sm[4 + w];
  }
  if (threadIdx.x == 0) sm[0] = total;
  const int64_t first = base + inc - mine;  // units in front of sequence s0
  // published for the caller: sm[1] target in, sm[2] sequence, sm[3] prefix
  const int64_t target = sm[1];
  if (mine && target >= first && target < first + mine) {
    int64_t p = first;
    for (int s = s0; s < s1; ++s) {
      const int n = seq_units(a, s);
      if (target < p + n) {
        sm[2] = s, sm[3] = p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
  return sm[0];
}

template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 1 : 3;  // parts of a query

template <int D>
struct DecSmem {
  static constexpr int NG = D / 32;
  static constexpr int kTile = 20 * D;
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kRing = kWarps * kStages * kTile;
};

template <typename T, int D>
constexpr int dec_smem_bytes() {
  return DecSmem<D>::kRing + kParts<T> * (D / 32) * 512 + 2 * (D / 32) * 32 + 8 * 4 + kWarps * 8 * 8 +
         kWarps * DecSmem<D>::kStages * 8 + (4 + kWarps) * 8 + 32;
}

// (1 + code / 16) pairs from nibble i of both halves of w, bf16.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  const uint32_t x = i == 0 ? w << 3 : w >> (4 * i - 3);
  return (x & 0x00780078u) | 0x3f803f80u;
}
// fp16 pairs from two shifts: 1 + code / 256 for nibbles 0 and 2, 1 + code / 16
// for nibbles 1 and 3.
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t x = w << 2, y = w >> 6;
  v[0] = (x & 0x003c003cu) | 0x3c003c00u, v[1] = (x & 0x03c003c0u) | 0x3c003c00u;
  v[2] = (y & 0x003c003cu) | 0x3c003c00u, v[3] = (y & 0x03c003c0u) | 0x3c003c00u;
}
// minus 1.5: (code - 8) / 16, exact
__device__ __forceinline__ uint32_t centre(uint32_t v) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x3fc03fc0u));
  return r;
}
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }
// The four (code - 8) pairs of w in fp16, exact: 1024 + code (or 1024 + 16
// code, from the second nibble where it stands) less what is too much.
__device__ __forceinline__ void codes_centred(uint32_t w, uint32_t (&v)[4]) {
  const __half2 k = __half2half2(__float2half(-1032.f)), f = __half2half2(__float2half(0.0625f)),
                t = __half2half2(__float2half(-72.f));
  const uint32_t x = w >> 8;
  v[0] = as_u32(__hadd2(as_h2((w & 0x000f000fu) | 0x64006400u), k));
  v[1] = as_u32(__hfma2(as_h2((w & 0x00f000f0u) | 0x64006400u), f, t));
  v[2] = as_u32(__hadd2(as_h2((x & 0x000f000fu) | 0x64006400u), k));
  v[3] = as_u32(__hfma2(as_h2((x & 0x00f000f0u) | 0x64006400u), f, t));
}
// D = A B (no sum in front).
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b));
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t &a, uint32_t &b) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ float h_lo(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)v)); }
__device__ __forceinline__ float h_hi(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)(v >> 16))); }

// Whether a partial result {m, l} holds any token.  Comparisons pass over a
// NaN, so tokens whose scores are all NaN leave m at -infinity; their sum is
// NaN then, and has to reach the result.
__device__ __forceinline__ bool counts(float2 ml) { return ml.x > -INFINITY || ml.y != 0.f; }

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps, 2) kv4_decode_kernel(const DecArgs a) {
  using S = DecSmem<D>;
  constexpr int NG = S::NG, NS = kParts<T>, kStages = S::kStages;
  constexpr bool kHalf = sizeof(T) == 2;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring_all = smem;
  uint4 *qf = reinterpret_cast<uint4 *>(smem + S::kRing);             // [NS][NG][32]
  float *qs = reinterpret_cast<float *>(qf + NS * NG * 32);          // [NG][8]
  float *qd = qs + NG * 8;                                           // [NG][8] sums as the products take them
  float *qinv = qd + NG * 8;                                         // [8] inverse scale of a head's query
  float2 *ml = reinterpret_cast<float2 *>(qinv + 8);                 // [kWarps][8] {m, l}
  uint64_t *bars = reinterpret_cast<uint64_t *>(ml + kWarps * 8);    // [kWarps][kStages]
  int64_t *scan = reinterpret_cast<int64_t *>(bars + kWarps * kStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  after_predecessor();  // (the joining kernel reads lengths as soon as this has returned everywhere)
  uint64_t *bar = bars + warp * kStages;
  uint8_t *ring = ring_all + warp * kStages * S::kTile;
  if (lane == 0)
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(bar + i, 1);
  ptx::mbar_fence_init();
  // units of the whole call, then of this block
  if (tid == 0) scan[1] = -1;
  __syncthreads();
  const int hh = a.n_kv * a.hb_count;
  const int64_t total = scan_units(a, scan) * hh;
  const int64_t parts = min((int64_t)a.grid, total);  // blocks that get units: at least one each
  const bool idle = blockIdx.x >= parts;
  const int64_t u_begin = idle ? 0 : total * blockIdx.x / parts, u_end = idle ? 0 : total * (blockIdx.x + 1) / parts;
  if (blockIdx.x == 0)
    for (int s = tid; s < a.n_seqs; s += blockDim.x) {
      const int n = __ldg(a.lens + s);
      if (n < 0 || (int64_t)n > (int64_t)a.max_pages * a.page_size) set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
    }
  if (u_begin >= u_end) return;
  if (tid == 0) scan[1] = u_begin / hh;
  __syncthreads();
  scan_units(a, scan);
  int seq = (int)scan[2];
  int64_t seq_base = scan[3];  // units (of one head block) in front of it
  __syncthreads();

  uint32_t phase = 0;  // bit i: parity of stage i's next completion
  int64_t u = u_begin;
  while (u < u_end) {
    int n_units = seq_units(a, seq);
    while ((seq_base + n_units) * hh <= u) {
      seq_base += n_units;
      n_units = seq_units(a, ++seq);
    }
    const int64_t in_seq = u - seq_base * hh;
    const int block_of = (int)(in_seq / n_units), first = (int)(in_seq % n_units);
    const int last = (int)min((int64_t)n_units, first + (u_end - u));
    u += last - first;
    const int j0 = max(0, first - kEntry), j1 = last - kEntry;  // units of tokens
    if (j1 <= j0) continue;
    const int kvh = block_of / a.hb_count, hb = block_of % a.hb_count;
    const int len = __ldg(a.lens + seq);
    const int head0 = kvh * a.ratio + hb * 8, n_h = min(8, a.ratio - hb * 8);

    // ---- the tiles of this warp: tile0 + kWarps * i, i < n_it
    const int tile0 = j0 * kWarps + warp, n_tiles = ((len - 1) >> 4) + 1;
    const int tile_end = min(n_tiles, j1 * kWarps);
    int n_it = tile0 < tile_end ? (tile_end - tile0 + kWarps - 1) / kWarps : 0;
    const int tiles_per_page = a.page_size >> 4;
    const int32_t *table = a.table + (int64_t)seq * a.max_pages;
    // lane i holds the place of tile number `batch + i`, or -1
    int batch = -32;
    int64_t my_at = -1;
    auto issue = [&](int it) {
      if (it - batch >= 32) {
        batch = it;
        my_at = -1;
        if (it + lane < n_it) {
          const unsigned t = tile0 + kWarps * (it + lane), p = t / (unsigned)tiles_per_page;
          const int64_t page = __ldg(table + p);
          if (page < 0 || page >= a.n_pages)
            set_status(a.status, REDLITE_STATUS_BAD_PAGE);
          else
            my_at = kv4_tile_offset<D>(page, a.n_kv, kvh, a.page_size, (int)(t - p * tiles_per_page));
        }
      }
      const int64_t at = __shfl_sync(0xffffffffu, my_at, it - batch);
      if (lane == 0) {
        const int st = it % kStages;
        if (at >= 0) {
          ptx::mbar_expect_tx(bar + st, S::kTile);
          ptx::bulk_g2s(ring + st * S::kTile, a.cache + at, S::kTile, bar + st);
        } else {
          ptx::mbar_arrive(bar + st);  // nothing is read: the tile is masked below
        }
      }
      return at >= 0;
    };
    uint32_t good = 0;  // bit i: the tile in stage i is real
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      if (i < n_it) good |= (uint32_t)issue(i) << i;

    // ---- queries of the block's heads as parts, and their sums per group
    auto query = [&](int g, int rr, int cc, float (&x)[8]) {
      if (rr < n_h) {
        load8<T>((const T *)a.q + (int64_t)seq * a.q_stride + (int64_t)(head0 + rr) * D + 32 * g + 8 * cc, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      }
    };
    if (kHalf) {
      // a warp per head; its largest element goes to 2^5, those at nibbles 0 and
      // 2 sixteen times as high, so that a group's sums stay below 2^14
      const int rr = warp;
      float y[NG / 4][8], mx = 0.f;
#pragma unroll
      for (int i = 0; i < NG / 4; ++i) {
        query(4 * i + (lane >> 3), rr, (lane >> 1) & 3, y[i]);  // two lanes per piece
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(y[i][e]));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float inv;
      const float s = scale_f16(mx, inv) * 0x1p-9f;
      if (lane == 0) qinv[rr] = inv * 0x1p9f;
#pragma unroll
      for (int i = 0; i < NG / 4; ++i) {
        const int g = 4 * i + (lane >> 3), cc = (lane >> 1) & 3;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= s;
        // elements 0, 4, 2, 6 meet nibbles 0 and 2, elements 1, 5, 3, 7 nibbles 1 and 3
        float far = (y[i][0] + y[i][4]) + (y[i][2] + y[i][6]), sum = (y[i][1] + y[i][5]) + (y[i][3] + y[i][7]);
#pragma unroll
        for (int o = 2; o <= 4; o <<= 1) {
          far += __shfl_xor_sync(0xffffffffu, far, o);
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if ((lane & 7) == 0) qs[g * 8 + rr] = far + sum, qd[g * 8 + rr] = fmaf(16.f, far, sum);
#pragma unroll
        for (int e = 0; e < 8; e += 2) y[i][e] *= 16.f;
        if ((lane & 1) == 0)  // pairs (0,4) (1,5) (2,6) (3,7): nibble i of both halves of a code word
          qf[g * 32 + rr * 4 + cc] = make_uint4(pack_f16(y[i][0], y[i][4]), pack_f16(y[i][1], y[i][5]),
                                                pack_f16(y[i][2], y[i][6]), pack_f16(y[i][3], y[i][7]));
      }
    } else {
      for (int i = tid; i < NG * 32; i += 32 * kWarps) {
        const int g = i >> 5, rr = (i >> 2) & 7, cc = i & 3;
        float x[8];
        query(g, rr, cc, x);
        float sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (cc == 0) qs[g * 8 + rr] = sum;
#pragma unroll
        for (int p = 0; p < NS; ++p) {
          uint4 w;
          w.x = pack_bf16(x[0], x[4]), w.y = pack_bf16(x[1], x[5]);
          w.z = pack_bf16(x[2], x[6]), w.w = pack_bf16(x[3], x[7]);
          qf[(p * NG + g) * 32 + (i & 31)] = w;
          x[0] -= bf16_lo(w.x), x[4] -= bf16_hi(w.x), x[1] -= bf16_lo(w.y), x[5] -= bf16_hi(w.y);
          x[2] -= bf16_lo(w.z), x[6] -= bf16_hi(w.z), x[3] -= bf16_lo(w.w), x[7] -= bf16_hi(w.w);
        }
      }
    }
    __syncthreads();
    // coefficients of {d, m} of groups c and c + 4 in a score of head r (in
    // units of 16 d): fp16 parts
    uint32_t ch[2] = {0u, 0u}, cl[2] = {0u, 0u};
    float to_log2 = a.scale_log2;
    if (kHalf) {
      to_log2 *= 16.f * qinv[r];
#pragma unroll
      for (int i = 0; i < NG / 4; ++i) {
        const int at = (c + 4 * i) * 8 + r;
        split_f16(-qd[at], qs[at] * 0.0625f, ch[i], cl[i]);
      }
    }

    float acc[NG][2][4], accm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][e][i] = 0.f;
    float m_run = -INFINITY, l_run = 0.f;  // of query head r; l over this thread's tokens
    int lift = 0;             // steps count as 2^lift times themselves in `acc`
    float room = kTop - 1.f;  // log2 that p may reach: kTop less that of the largest |d| met, 2 if that is less (16-bit types)

    for (int it = 0; it < n_it; ++it) {
      const int st = it % kStages;
      const uint32_t tile = ptx::smem_u32(ring + st * S::kTile);
      const bool came = ptx::mbar_wait_suspend(bar + st, (phase >> st) & 1u);
      if (!__all_sync(0xffffffffu, came)) {  // no more tiles are asked for, those on their way are waited for
        set_status(a.status, REDLITE_STATUS_TIMEOUT);
        ptx::mbar_wait_suspend(bar + st, (phase >> st) & 1u);
        n_it = min(n_it, it + kStages);
      }
      phase ^= 1u << st;
      const int tok0 = 16 * (tile0 + kWarps * it);
      const int live = ((good >> st) & 1u) ? len - tok0 : 0;  // tokens of this tile that count
      // ---- scores: C[token][head] over the groups
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      if (kHalf) {  // the terms of d and m alone
        uint32_t k[4];
        if (NG == 8) {
          ldsm4(tile + 8 * D + (lane & 15) * 32 + (lane >> 4) * 16, k[0], k[1], k[2], k[3]);
          mma_f16(s, k, ch[0], ch[1]);
          mma_f16(s, k, cl[0], cl[1]);
        } else {
          ldsm2(tile + 8 * D + (lane & 15) * 16, k[0], k[1]);
          mma_f16_k8(s, k[0], k[1], ch[0]);
          mma_f16_k8(s, k[0], k[1], cl[0]);
        }
      }
#pragma unroll
      for (int gq = 0; gq < NG / 4; ++gq) {
        const uint4 w0 = ptx::lds128(tile + gq * 512 + lane * 16);               // token r
        const uint4 w1 = ptx::lds128(tile + (NG / 4 + gq) * 512 + lane * 16);    // token r + 8
        const uint4 k0 = ptx::lds128(tile + 8 * D + r * (NG * 4) + gq * 16);      // {d, m} of four groups
        const uint4 k1 = ptx::lds128(tile + 8 * D + (r + 8) * (NG * 4) + gq * 16);
        const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w}, wb[4] = {w1.x, w1.y, w1.z, w1.w};
        const uint32_t ka[4] = {k0.x, k0.y, k0.z, k0.w}, kb[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
          const int g = gq * 4 + gg;
          uint32_t A0[4], A1[4];
          float x[4] = {0.f, 0.f, 0.f, 0.f};
          if (kHalf) {
            code_pairs(wa[gg], A0);
            code_pairs(wb[gg], A1);
            const uint4 b = qf[g * 32 + lane];
            const uint32_t p[4] = {A0[0], A1[0], A0[1], A1[1]}, q[4] = {A0[2], A1[2], A0[3], A1[3]};
            mma_f16_first(x, p, b.x, b.y);
            mma_f16(x, q, b.z, b.w);
            const float da = h_lo(ka[gg]), db = h_lo(kb[gg]);
            s[0] = fmaf(da, x[0], s[0]), s[1] = fmaf(da, x[1], s[1]);
            s[2] = fmaf(db, x[2], s[2]), s[3] = fmaf(db, x[3], s[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) A0[i] = centre(code_pair(wa[gg], i)), A1[i] = centre(code_pair(wb[gg], i));
#pragma unroll
            for (int p = 0; p < NS; ++p) {
              const uint4 b = qf[(p * NG + g) * 32 + lane];
              mma_bf16(x, A0[0], A1[0], A0[1], A1[1], b.x, b.y);
              mma_bf16(x, A0[2], A1[2], A0[3], A1[3], b.z, b.w);
            }
            const float2 sum = *reinterpret_cast<const float2 *>(qs + g * 8 + 2 * c);
            const float da = 16.f * h_lo(ka[gg]), db = 16.f * h_lo(kb[gg]);
            const float ma = fmaf(0.5f, da, h_hi(ka[gg])), mb = fmaf(0.5f, db, h_hi(kb[gg]));
            s[0] = fmaf(da, x[0], fmaf(ma, sum.x, s[0]));
            s[1] = fmaf(da, x[1], fmaf(ma, sum.y, s[1]));
            s[2] = fmaf(db, x[2], fmaf(mb, sum.x, s[2]));
            s[3] = fmaf(db, x[3], fmaf(mb, sum.y, s[3]));
          }
        }
      }
      // ---- to the layout of the second product: head r, tokens 2c, 2c+1, 2c+8, 2c+9
      float p[4];
      {
        const int src = 8 * c + (r >> 1);
        const float a0 = __shfl_sync(0xffffffffu, s[0], src), a1 = __shfl_sync(0xffffffffu, s[1], src);
        const float b0 = __shfl_sync(0xffffffffu, s[0], src + 4), b1 = __shfl_sync(0xffffffffu, s[1], src + 4);
        const float c0 = __shfl_sync(0xffffffffu, s[2], src), c1 = __shfl_sync(0xffffffffu, s[3], src);
        const float d0 = __shfl_sync(0xffffffffu, s[2], src + 4), d1 = __shfl_sync(0xffffffffu, s[3], src + 4);
        p[0] = (r & 1) ? a1 : a0, p[1] = (r & 1) ? b1 : b0;
        p[2] = (r & 1) ? c1 : c0, p[3] = (r & 1) ? d1 : d0;
      }
      // ---- steps of the four tokens
      const uint32_t vs = tile + 18 * D, vm = tile + 19 * D;
      uint32_t dw[4][NG / 2];
      int tk[4];
      bool on[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tk[i] = 2 * c + (i & 1) + 8 * (i >> 1), on[i] = tk[i] < live;
        p[i] *= to_log2;
        if (NG == 8) {
          const uint4 d = ptx::lds128(vs + tk[i] * 16);
          dw[i][0] = d.x, dw[i][1] = d.y, dw[i][NG / 2 - 2] = d.z, dw[i][NG / 2 - 1] = d.w;
        } else {
          const uint2 d = ptx::lds64(vs + tk[i] * 8);
          dw[i][0] = d.x, dw[i][1] = d.y;
        }
      }
      if (live < 16) {  // what lies behind the sequence may be anything
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = on[i] ? p[i] : -INFINITY;
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) dw[i][g] = on[i] ? dw[i][g] : 0u;
        }
      }
      float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (kHalf) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) any |= dw[i][g];
        // a step of 2 or more (`room` starts one below for the rest); the first
        // tile, which says whether steps are lifted, and every one while they are
        if (it == 0 || lift || __any_sync(0xffffffffu, any & 0x40004000u)) {
          __half2 big = __habs2(as_h2(dw[0][0]));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < NG / 2; ++g) big = __hmax2(big, __habs2(as_h2(dw[i][g])));
          big = __hmax2(big, as_h2(__shfl_xor_sync(0xffffffffu, as_u32(big), 1)));
          big = __hmax2(big, as_h2(__shfl_xor_sync(0xffffffffu, as_u32(big), 2)));
          // 2^n > top >= 2^(n - 1); at most 16
          const float top = fmaxf(__low2float(big), __high2float(big));
          const int n = (int)(__float_as_uint(top) >> 23) - 126;
          room = fminf(room, kTop - (float)min(16, max(0, n)));
          const int to = it == 0 ? (n < kLiftBelow ? min(1 - n, 15) : 0) : min(lift, max(0, 1 - n));
          if (to != lift && it > 0) {
            const float f = __int_as_float((127 + to - lift) << 23);
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[g][e][i] *= f;
          }
          lift = to;
        }
        if (lift) {
          const __half2 f = as_h2((uint32_t)(15 + lift) * 0x04000400u);  // 2^lift
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < NG / 2; ++g) dw[i][g] = as_u32(__hmul2(as_h2(dw[i][g]), f));
        }
      }
      // rescale only when a score passes the reference by 2^8 (16-bit types: by
      // what keeps p and p d in fp16) or the first one comes: the sums stay far
      // inside fp32 either way
      const float limit = kHalf ? room : kLazy;
      if (__any_sync(0xffffffffu, mx > m_run + limit || (m_run == -INFINITY && mx > -INFINITY))) {
        const float m_new = kHalf ? (mx > m_run + limit ? mx - (limit - kLazy) : m_run) : fmaxf(m_run, mx);
        const float f = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
        l_run *= f;
        m_run = m_new;
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * c), f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            acc[g][e][0] *= f0, acc[g][e][1] *= f1, acc[g][e][2] *= f0, acc[g][e][3] *= f1;
        accm[0] *= f0, accm[1] *= f1, accm[2] *= f0, accm[3] *= f1;
      }
      const float ref = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(p[i] - ref), l_run += p[i];
      // ---- values (the code unit of slot i is token tk[i])
      uint32_t vw[4][NG / 2];
      if (NG == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = ptx::lds128(tile + 10 * D + i * 512 + lane * 16);
          vw[i][0] = v.x, vw[i][1] = v.y, vw[i][NG / 2 - 2] = v.z, vw[i][NG / 2 - 1] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const uint4 v = ptx::lds128(tile + 10 * D + (i >> 1) * 512 + lane * 16);
          vw[i][0] = v.x, vw[i][1] = v.y, vw[i + 1][0] = v.z, vw[i + 1][1] = v.w;
        }
      }
      if (kHalf) {
        uint32_t ph[2], pl[2], k[4];
        split_f16(p[0], p[1], ph[0], pl[0]);
        split_f16(p[2], p[3], ph[1], pl[1]);
        // sums over m and d: rows r and r + 8 are m and d of group r (NG = 8),
        // rows r and r + 4 (NG = 4)
        if (NG == 8) {
          ldsm4t(((lane & 8) ? vs : vm) + ((lane & 7) + ((lane >> 4) << 3)) * 16, k[0], k[1], k[2], k[3]);
        } else {
          const uint32_t at = (r < 4 ? vm : vs) + 2 * (r & 3);
          k[0] = ptx::lds16(at + tk[0] * 8) | (ptx::lds16(at + tk[1] * 8) << 16);
          k[2] = ptx::lds16(at + tk[2] * 8) | (ptx::lds16(at + tk[3] * 8) << 16);
          k[1] = k[3] = 0u;
        }
        if (live < 16) {
          const uint32_t m0 = (on[0] ? 0xffffu : 0u) | (on[1] ? 0xffff0000u : 0u);
          const uint32_t m1 = (on[2] ? 0xffffu : 0u) | (on[3] ? 0xffff0000u : 0u);
          k[0] &= m0, k[1] &= m0, k[2] &= m1, k[3] &= m1;
        }
        mma_f16(accm, k, ph[0], ph[1]);
        mma_f16(accm, k, pl[0], pl[1]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = as_u32(__hmul2(as_h2(ph[0]), as_h2(__byte_perm(dw[0][g >> 1], dw[1][g >> 1], sel))));
          const uint32_t b1 = as_u32(__hmul2(as_h2(ph[1]), as_h2(__byte_perm(dw[2][g >> 1], dw[3][g >> 1], sel))));
          uint32_t X[4], Y[4];
          codes_centred(__byte_perm(vw[0][g >> 1], vw[1][g >> 1], sel), X);
          codes_centred(__byte_perm(vw[2][g >> 1], vw[3][g >> 1], sel), Y);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t A[4] = {X[2 * e], X[2 * e + 1], Y[2 * e], Y[2 * e + 1]};
            mma_f16(acc[g][e], A, b0, b1);
          }
        }
      } else {
        // three parts of p, of 16 d p and of m + 8 d
        auto parts = [](float x, float y, uint32_t (&w)[3]) {
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            w[i] = pack_bf16(x, y);
            x -= bf16_lo(w[i]), y -= bf16_hi(w[i]);
          }
        };
        uint32_t pa[3], pb[3];
        parts(p[0], p[1], pa);
        parts(p[2], p[3], pb);
        {
          // group r's m + 8 d of the four tokens (rows r: first part, rows r + 8:
          // second; then the third alone)
          float mid[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int g = r & (NG - 1);
            const float d = h_lo(ptx::lds16(vs + (tk[i] * NG + g) * 2)), m = h_lo(ptx::lds16(vm + (tk[i] * NG + g) * 2));
            mid[i] = on[i] && r < NG ? fmaf(8.f, d, m) : 0.f;
          }
          uint32_t ma[3], mb[3];
          parts(mid[0], mid[1], ma);
          parts(mid[2], mid[3], mb);
#pragma unroll
          for (int i = 0; i < 3; ++i) mma_bf16(accm, ma[0], ma[1], mb[0], mb[1], pa[i], pb[i]);
          mma_bf16(accm, ma[2], 0u, mb[2], 0u, pa[0], pb[0]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] *= 16.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float pd[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pd[i] = p[i] * ((g & 1) ? h_hi(dw[i][g >> 1]) : h_lo(dw[i][g >> 1]));
          uint32_t ba[3], bb[3];
          parts(pd[0], pd[1], ba);
          parts(pd[2], pd[3], bb);
          const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
          const uint32_t X = __byte_perm(vw[0][g >> 1], vw[1][g >> 1], sel);
          const uint32_t Y = __byte_perm(vw[2][g >> 1], vw[3][g >> 1], sel);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t a0 = centre(code_pair(X, 2 * e)), a1 = centre(code_pair(X, 2 * e + 1));
            const uint32_t a2 = centre(code_pair(Y, 2 * e)), a3 = centre(code_pair(Y, 2 * e + 1));
#pragma unroll
            for (int i = 0; i < 3; ++i) mma_bf16(acc[g][e], a0, a1, a2, a3, ba[i], bb[i]);
          }
        }
      }
      // ---- the stage is free again
      if (it + kStages < n_it) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        const uint32_t ok = issue(it + kStages);
        good = (good & ~(1u << st)) | (ok << st);
      }
    }

    // ---- join the warps (the rings are drained: they hold the results now)
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
    if (c == 0) ml[warp * 8 + r] = make_float2(m_run, l_run);
    __syncwarp();
    float *mine = reinterpret_cast<float *>(ring);  // [8 heads][D]
    // fp32: parts of the same sum; 16-bit types: rows of m, rows of d
    const float of_d = kHalf ? 8.f : 1.f;
    if (!kHalf || NG == 8) accm[0] = fmaf(of_d, accm[2], accm[0]), accm[1] = fmaf(of_d, accm[3], accm[1]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // group g's sum over m + 8 d sits in the lanes of row g (and of row g + 4: d, where NG = 4)
      float g0 = __shfl_sync(0xffffffffu, accm[0], g * 4 + c), g1 = __shfl_sync(0xffffffffu, accm[1], g * 4 + c);
      if (kHalf && NG == 4) {
        g0 = fmaf(8.f, __shfl_sync(0xffffffffu, accm[0], (g + 4) * 4 + c), g0);
        g1 = fmaf(8.f, __shfl_sync(0xffffffffu, accm[1], (g + 4) * 4 + c), g1);
      }
      float *h0 = mine + (2 * c) * D + 32 * g + 4 * r, *h1 = h0 + D;
      const float un = kHalf ? __int_as_float((127 - lift) << 23) : 1.f;
      auto sum = [&](float x, float y) { return kHalf ? fmaf(x, un, y) : x + y; };
      *reinterpret_cast<float4 *>(h0) = make_float4(sum(acc[g][0][0], g0), sum(acc[g][0][2], g0), sum(acc[g][1][0], g0),
                                                    sum(acc[g][1][2], g0));
      *reinterpret_cast<float4 *>(h1) = make_float4(sum(acc[g][0][1], g1), sum(acc[g][0][3], g1), sum(acc[g][1][1], g1),
                                                    sum(acc[g][1][3], g1));
    }
    __syncthreads();
    const bool whole = j0 == 0 && j1 == n_units - kEntry;
    float *part = a.part + (int64_t)(2 * blockIdx.x + (j0 > 0 ? 0 : 1)) * (8 * D + 16);
    for (int i = tid; i < 8 * D / 4; i += 32 * kWarps) {
      const int h = i / (D / 4), d4 = i % (D / 4);
      if (h >= n_h) continue;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * 8 + h].x);
      const float base = m == -INFINITY ? 0.f : m;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml[w * 8 + h];
        const float f = ex2(v.x - base);
        const float4 x =
            *reinterpret_cast<const float4 *>(ring_all + w * kStages * S::kTile + (size_t)(h * D + 4 * d4) * 4);
        if (counts(v)) {
          l = fmaf(f, v.y, l);
          o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
        }
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        T *dst = (T *)a.out + (int64_t)seq * a.out_stride + (int64_t)(head0 + h) * D + 4 * d4;
        dst[0] = from_f32<T>(o.x * inv), dst[1] = from_f32<T>(o.y * inv);
        dst[2] = from_f32<T>(o.z * inv), dst[3] = from_f32<T>(o.w * inv);
      } else {
        reinterpret_cast<float4 *>(part)[i] = o;
        if (d4 == 0) *reinterpret_cast<float2 *>(part + 8 * D + 2 * h) = make_float2(m, l);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncthreads();
  }
}

// One block per sequence and query head: adds the partial results of a head
// block's units in the order of the blocks that made them (four runs of
// blocks, then the runs), and writes zeros for a sequence without tokens.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const DecArgs a) {
  constexpr int kRuns = 1024 / D, kPart = 8 * D + 16;
  __shared__ int64_t scan[4 + 8];
  __shared__ float red[8];
  __shared__ float4 sum[kRuns][D / 4];
  __shared__ float run_l[kRuns];
  const int tid = threadIdx.x;
  const int seq = blockIdx.x / a.n_heads, head = blockIdx.x % a.n_heads;
  const int n_units = seq_units(a, seq);
  T *dst = (T *)a.out + (int64_t)seq * a.out_stride + (int64_t)head * D;
  // the lengths are not the other kernel's to write: what they say is found
  // while it still runs (but no block ends before it)
  if (n_units == 0) {
    after_predecessor();
    if (tid < D) dst[tid] = from_f32<T>(0.f);
    return;
  }
  if (tid == 0) scan[1] = -1;
  __syncthreads();
  // units in front of this sequence
  int64_t before = 0;
  for (int s = tid; s < seq; s += blockDim.x) before += seq_units(a, s);
#pragma unroll
  for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  __shared__ int64_t front[8];
  if ((tid & 31) == 0) front[tid >> 5] = before;
  const int hh = a.n_kv * a.hb_count;
  const int64_t total = scan_units(a, scan) * hh;
  before = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) before += front[w];
  const int kvh = head / a.ratio, in_kv = head % a.ratio, hb = in_kv >> 3, h = in_kv & 7;
  const int64_t base_u = before * hh + (int64_t)(kvh * a.hb_count + hb) * n_units;
  const int64_t u0 = base_u + kEntry, u1 = base_u + n_units - 1;  // units of tokens
  // block of unit u: the i with total * i / parts <= u < total * (i + 1) / parts
  const int64_t parts = min((int64_t)a.grid, total);
  const int i0 = (int)(((u0 + 1) * parts - 1) / total), i1 = (int)(((u1 + 1) * parts - 1) / total);
  after_predecessor();
  if (i0 == i1) return;  // one block saw all of it and wrote the output
  auto part = [&](int i) { return a.part + (int64_t)(2 * i + (i == i0 ? 1 : 0)) * kPart; };
  float m = -INFINITY;
  for (int i = i0 + tid; i <= i1; i += blockDim.x) m = fmaxf(m, *(part(i) + 8 * D + 2 * h));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
  const float base = m == -INFINITY ? 0.f : m;
  const int run = tid / (D / 4), d4 = tid % (D / 4);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int i = i0 + run; i <= i1; i += kRuns) {
    const float *p = part(i);
    const float2 v = *reinterpret_cast<const float2 *>(p + 8 * D + 2 * h);
    const float4 x = *(reinterpret_cast<const float4 *>(p + h * D) + d4);
    if (counts(v)) {
      const float f = ex2(v.x - base);
      l = fmaf(f, v.y, l);
      o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
    }
  }
  sum[run][d4] = o;
  if (d4 == 0) run_l[run] = l;
  __syncthreads();
  if (run == 0) {
    for (int k = 1; k < kRuns; ++k) {
      const float4 x = sum[k][d4];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      l += run_l[k];
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    dst[4 * d4] = from_f32<T>(o.x * inv), dst[4 * d4 + 1] = from_f32<T>(o.y * inv);
    dst[4 * d4 + 2] = from_f32<T>(o.z * inv), dst[4 * d4 + 3] = from_f32<T>(o.w * inv);
  }
}

template <typename T, int D>
cudaError_t launch_decode(const DecArgs &a, cudaStream_t s) {
  constexpr int smem = dec_smem_bytes<T, D>();
  cudaError_t e =
      cudaFuncSetAttribute(kv4_decode_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_early(kv4_decode_kernel<T, D>, a.grid, 32 * kWarps, smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_early(kv4_join_kernel<T, D>, (unsigned)(a.n_seqs * a.n_heads), 256, 0, s, a);
}
template <typename T>
cudaError_t launch_decode_t(const DecArgs &a, int D, cudaStream_t s) {
  return D == 256 ? launch_decode<T, 256>(a, s) : launch_decode<T, 128>(a, s);
}

// Blocks of a call: two per multiprocessor (what the kernel's shared memory
// and registers allow), for any sizes.
constexpr int kMaxGrid = 2 * 256;

}  // namespace
}  // namespace redlite

using namespace redlite;

extern "C" size_t redlite_kv4_decode_workspace_bytes(int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads,
                                                     int32_t head_dim) {
  if (n_seqs < 0 || n_kv_heads < 1 || n_heads < 1 || n_heads > 4096 || n_heads % n_kv_heads || !kv4_shape_ok(head_dim, 16))
    return 0;
  return (size_t)2 * kMaxGrid * (8 * head_dim + 16) * sizeof(float);
}

extern "C" int redlite_kv4_decode(int32_t dtype, const void *q, int64_t q_stride, int32_t n_seqs, int32_t n_heads,
                                  int32_t n_kv_heads, int32_t head_dim, const void *cache, int32_t page_size,
                                  const int32_t *block_table, int32_t max_pages, int64_t n_pages,
                                  const int32_t *lens, float scale, void *out, int64_t out_stride, void *workspace,
                                  size_t workspace_bytes, int32_t *status, void *stream) {
  if (!dtype_ok(dtype) || n_seqs < 0 || n_heads < 1 || n_heads > 4096 || n_kv_heads < 1 || n_kv_heads > 1024 ||
      n_heads % n_kv_heads)
    return REDLITE_EINVAL;
  if (!kv4_shape_ok(head_dim, page_size)) return REDLITE_EUNSUPPORTED;
  if (!(scale > 0.f) || !(scale < INFINITY)) return REDLITE_EINVAL;
  if (n_seqs == 0) return REDLITE_OK;
  if (max_pages < 1 || n_pages < 1 || !q || !cache || !block_table || !lens || !out || !workspace) return REDLITE_EINVAL;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(workspace)) return REDLITE_EINVAL;
  const int64_t row = (int64_t)n_heads * head_dim;
  if (!stride_ok(q_stride, row, dtype) || !stride_ok(out_stride, row, dtype)) return REDLITE_EINVAL;
  if ((int64_t)n_seqs * n_heads >= ((int64_t)1 << 31) - 1) return REDLITE_EUNSUPPORTED;
  if (workspace_bytes < redlite_kv4_decode_workspace_bytes(n_seqs, n_heads, n_kv_heads, head_dim)) return REDLITE_ENOMEM;
  const int sms = device_sms();
  if (sms <= 0) return REDLITE_ECUDA;
  DecArgs a;
  a.q = q, a.out = out, a.q_stride = q_stride, a.out_stride = out_stride;
  a.cache = (const uint8_t *)cache, a.table = block_table, a.lens = lens;
  a.n_seqs = n_seqs, a.n_heads = n_heads, a.n_kv = n_kv_heads, a.ratio = n_heads / n_kv_heads;
  a.hb_count = (a.ratio + 7) / 8;
  a.page_size = page_size, a.max_pages = max_pages, a.n_pages = n_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.part = (float *)workspace;
  a.status = status;
  // no more blocks than units the longest lengths could give
  const int64_t cap =
      (int64_t)n_seqs * n_kv_heads * a.hb_count * (((int64_t)max_pages * page_size + kUnit - 1) / kUnit + kEntry);
  a.grid = (int)std::min<int64_t>(std::min(2 * sms, kMaxGrid), cap);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == REDLITE_T_F32) e = launch_decode_t<float>(a, head_dim, s);
  else if (dtype == REDLITE_T_BF16) e = launch_decode_t<__nv_bfloat16>(a, head_dim, s);
  else e = launch_decode_t<__half>(a, head_dim, s);
  return e == cudaSuccess ? REDLITE_OK : REDLITE_ECUDA;
}
