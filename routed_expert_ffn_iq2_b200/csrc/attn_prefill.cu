// attn_prefill.cu -- causal attention over packed prompts with grouped heads
// (redlite_attn_prefill).  ("Red Lite dev16 -- complete full-attention
// parity", section "Pinned full-attention graph": 16 query heads on 2
// key/value heads of 256.)
//
//   O = softmax(scale Q K^T) V, one pass over the keys with a running
//   reference m and sum l per row: p = 2^(s - m), l += p, O += p V; when a
//   score passes m by more than 2^8 (and at a row's first keys), l and O are
//   rescaled by 2^(m - m') -- rare, and exact otherwise.
//
// Both products run on the tensor cores (tcgen05, fp32 accumulators in tensor
// memory), 4 D flops per visible pair, which is the bound: a tile of 128 rows
// by 128 keys takes 2 x 128 x 128 x D multiply-adds against 128 x 128
// exponentials.  One block per 128 rows, and two of them on a multiprocessor
// where heads are 128 wide (then in steps of 64 keys); the rows of a tile are
// tokens x the query heads that share a key/value head (the largest power of
// two G of them), so keys are read once for G heads and a prompt of a few
// tokens still fills its tile.
//   warp 0      one thread: TMA loads of Q (once) and of K and V in a ring of
//               stages (128B-swizzled boxes)
//   warp 1      issues the products.  Two score buffers are used in turn: the
//               scores of step i + 1 are issued in front of the second product
//               of step i, so the tensor cores work while the softmax does
//   warps 2, 3  zeros over the last values that no row sees; warp 2 allocates the
//               tensor memory too
//   warps 4 ..  softmax: thread = row.  A step's scores come out of tensor memory
//               in one read (in halves, read twice: 4.5 us more of the ragged
//               batch below), probabilities go back over them in the inputs' type (that
//               rounding, 2^-8 or 2^-11 of each p at most, is what the product's type
//               asks for; l sums the unrounded p), half a row at a time: the
//               second product starts on the first half of the keys
// A block's start and end (loads, first scores, rows out: 7 us) go by beside
// the other block's steps where there are two (one block of two row tiles, a
// softmax group each: 82 us for the ragged batch below).
//
// Measured (one B200): 16384 tokens, 16 heads on 2 of 256, bf16: 1.70 to 1.73 ms,
// 1.27 to 1.29 PFLOP/s (a long library product: 1.39); five ragged fp16 prompts,
// 3957 tokens of 32 heads on 8 of 128: 72 us, 660 TFLOP/s; three of 43 tokens
// together 7.7 us.  Rounding p costs: error against 64 bits 2.2e-3 of the output
// for the long bf16 prompt (1.6e-3 is the output's own rounding), 2.6e-4 for the
// fp16 batch (2.1e-4).  Tried without gain: two threads a row in the softmax,
// polynomials for a part of the exponentials, probabilities handed over in one
// piece, tiles of all sequences by their keys instead of sequence by sequence.
//
// A zero probability times a NaN or an infinity in V is a NaN that a masked
// key must not cause.  Of the keys that no row of a block sees (behind a
// sequence, or later tokens) the last product leaves out all it can, and the
// values of the up to 15 others are set to zero in shared memory (with NaN
// behind 8189 keys, 512 queries of 16 heads took 142 ms without, as every row
// of the last tile was computed again).  Among a block's own tokens, and where
// a sum over values past 10^36 leaves fp32, the columns of a row that are not
// finite are computed again by its warp from the keys it sees alone (a NaN in
// the last of 8192 values: 35 ms, 1 ms for each of a warp's 32 rows; one among
// the first keys: nothing that shows).
#include <cuda.h>

#include <type_traits>

#include "mixer.cuh"

namespace redlite {
namespace {

struct AttnArgs {
  const void *q, *k, *v;
  void *out;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const int32_t *cu_q, *cu_k;
  int n_seqs, n_q, n_k, n_heads, n_kv, group, log_group;
  float scale_log2;
  int32_t *status;
};

constexpr int kRows = 128;          // rows of a tile
constexpr float kLazy = 8.f;

template <int D>
struct Shape {
  static constexpr int kBlocks = D == 128 ? 2 : 1;         // on a multiprocessor
  static constexpr int kKeys = D == 128 ? 64 : 128;        // keys per step
  static constexpr int kSub = kKeys / 64;                  // stages per K or V tile
  static constexpr int kStageBytes = 64 * D * 2;           // kKeys keys x 128 values (K) or 64 x D (V)
  static constexpr int kRing = D == 128 ? 4 : 5;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr uint32_t kO = 2 * kKeys;                // first accumulator column of O, behind the scores
  static constexpr uint32_t kColumns = kO + D;
  static_assert(kKeys * 128 * 2 == kStageBytes, "K and V stages are of one size");
};

template <int D>
struct Bars {
  uint64_t q_full, full[Shape<D>::kRing], empty[Shape<D>::kRing], s_full[2], p_half[2], p_full[2], o_full, done, tail;
  uint32_t tmem;
  int dead;
};
template <int D>
constexpr int attn_smem() {
  return Shape<D>::kQBytes + Shape<D>::kRing * Shape<D>::kStageBytes + (int)sizeof(Bars<D>) + 1024;
}
static_assert(attn_smem<256>() <= 227 * 1024 && 2 * (attn_smem<128>() + 1024) <= 228 * 1024, "shared memory of a block");

__device__ __forceinline__ void tma_load3(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(ptx::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}

// Two fp32 operations at a time.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  return (uint64_t)__float_as_uint(x) | ((uint64_t)__float_as_uint(y) << 32);
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Descriptor of a tile whose rows run along K and whose 64-element row pieces
// (128 bytes, swizzled) run along N: `lead` bytes between 64-column pieces,
// 1024 between groups of 8 rows.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// D[tmem] (+)= A B, issued by the one thread of a converged warp whose `go` is
// set; descriptors as low and high word.  The whole warp walks the loop, so
// that addresses stay in uniform registers: issued from a branch that one
// thread takes, each product cost 110 cycles of moves into them, against the
// 64 that it runs.
template <bool ACC>
__device__ __forceinline__ void umma_ss(uint32_t go, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                        uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %7, 0;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, %6;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0), "r"(go)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t go, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.b32 q, %6, 0;\n setp.ne.b32 p, %5, 0;\n mov.b64 db, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(go)
      : "memory");
}
__device__ __forceinline__ void umma_done(uint32_t go, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n"
      " @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(ptx::smem_u32(bar)),
      "r"(go)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}

// Bounded wait; after one that gave up every later one returns at once.
template <int D>
__device__ __forceinline__ bool wait(Bars<D> *b, uint64_t *bar, uint32_t parity, int32_t *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  if (*(volatile int *)&b->dead) return false;
  if (ptx::mbar_wait_suspend(bar, parity)) return true;
  *(volatile int *)&b->dead = 1;
  set_status(status, REDLITE_STATUS_TIMEOUT);
  return false;
}

// The columns of one row that are not finite, by one warp, from the keys the
// row sees alone, fp32; eight keys at a time.  o is the mean so far, so that
// values near the end of bf16's range do not leave fp32's in a sum.  The walk
// ends where a NaN has reached every such column (nothing takes it away).
template <typename T, int D>
__device__ __noinline__ void row_again(const AttnArgs &a, int64_t q_row, int head, int64_t k_row0, int lim) {
  constexpr int E = D / 32, kAhead = 8;  // a lane has E neighbouring columns
  struct alignas(2 * E) Piece {
    T x[E];
  };
  const int lane = threadIdx.x & 31, kh = head / (a.n_heads / a.n_kv);
  const Piece *k = reinterpret_cast<const Piece *>((const T *)a.k + k_row0 * a.k_stride + (int64_t)kh * D) + lane;
  const Piece *v = reinterpret_cast<const Piece *>((const T *)a.v + k_row0 * a.v_stride + (int64_t)kh * D) + lane;
  Piece *out = reinterpret_cast<Piece *>((T *)a.out + q_row * a.out_stride + (int64_t)head * D) + lane;
  Piece r = *out;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  {
    const Piece x = reinterpret_cast<const Piece *>((const T *)a.q + q_row * a.q_stride + (int64_t)head * D)[lane];
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = to_f32(x.x[e]), o[e] = 0.f;
  }
  uint32_t open = 0;  // bit e: column e is not finite
#pragma unroll
  for (int e = 0; e < E; ++e) open |= (uint32_t)!(to_f32(r.x[e]) * 0.f == 0.f) << e;
  const int64_t k_step = a.k_stride / E, v_step = a.v_stride / E;  // rows lie on 16-byte boundaries
  for (int j = 0; j < lim; j += kAhead) {
    float s[kAhead];
    Piece y[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t at = min(j + u, lim - 1);
      const Piece x = k[at * k_step];
      y[u] = v[at * v_step];
      s[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s[u] = fmaf(q[e], to_f32(x.x[e]), s[u]);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1)
#pragma unroll
      for (int u = 0; u < kAhead; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], x);
    float mn = m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      s[u] = j + u < lim ? s[u] * a.scale_log2 : -INFINITY;
      mn = s[u] > mn ? s[u] : mn;  // a NaN leaves m and makes p a NaN
    }
    const float old = l * (m == -INFINITY ? 0.f : ex2(m - mn));
    l = old;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) s[u] = s[u] == -INFINITY ? 0.f : ex2(s[u] - mn), l += s[u];
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    bool done = true;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] *= old * inv;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j + u < lim) o[e] = fmaf(s[u] * inv, to_f32(y[u].x[e]), o[e]);
      done = done && (!((open >> e) & 1u) || o[e] != o[e]);
    }
    if (__all_sync(0xffffffffu, done)) break;
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if ((open >> e) & 1u) r.x[e] = from_f32<T>(o[e]);
  if (open) *out = r;
}

template <typename T, int D>
__global__ void __launch_bounds__(256, Shape<D>::kBlocks)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv, const AttnArgs a) {
  using Sh = Shape<D>;
  constexpr int kKeys = Sh::kKeys, kSub = Sh::kSub, kRing = Sh::kRing, kStageBytes = Sh::kStageBytes;
  constexpr bool kBf = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *sq = smem, *ring = smem + Sh::kQBytes;
  Bars<D> *b = reinterpret_cast<Bars<D> *>(ring + kRing * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  after_predecessor();
  if (threadIdx.x == 0) {
    for (const CUtensorMap *m : {&mq, &mk, &mv}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    ptx::mbar_init(&b->q_full, 1);
    for (int i = 0; i < kRing; ++i) ptx::mbar_init(b->full + i, 1), ptx::mbar_init(b->empty + i, 1);
    for (int i = 0; i < 2; ++i)
      ptx::mbar_init(b->s_full + i, 1), ptx::mbar_init(b->p_half + i, 128), ptx::mbar_init(b->p_full + i, 128);
    ptx::mbar_init(&b->o_full, 1), ptx::mbar_init(&b->done, 1), ptx::mbar_init(&b->tail, 1);
    b->dead = 0;
    ptx::mbar_fence_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(&b->tmem, Sh::kColumns);
    ptx::tmem_relinquish();
  }
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.n_seqs; s += blockDim.x) {
      const int b0 = __ldg(a.cu_q + s), e0 = __ldg(a.cu_q + s + 1), b1 = __ldg(a.cu_k + s), e1 = __ldg(a.cu_k + s + 1);
      if (b0 < 0 || e0 < b0 || e0 > a.n_q || b1 < 0 || e1 < b1 || e1 > a.n_k) set_status(a.status, REDLITE_STATUS_BAD_LENGTH);
    }
  // ---- which rows: the last tiles of the last sequences first (most keys).
  // The sequence is the last whose first slot is not behind this one: 32
  // places are looked at together.
  const int tile_tok = kRows >> a.log_group;
  const int hb = blockIdx.x % (a.n_heads >> a.log_group);
  const int64_t slot = (gridDim.x - 1 - blockIdx.x) / (a.n_heads >> a.log_group);
  int lo = 0;
  for (int n = a.n_seqs; n > 1;) {  // it is one of lo .. lo + n - 1
    const int step = (n + 31) >> 5, at = lo + lane * step;
    const bool in = lane * step < n && (int64_t)(__ldg(a.cu_q + at) / tile_tok) + at <= slot;
    const uint32_t found = __ballot_sync(0xffffffffu, in) | 1u;
    const int skip = (31 - __clz(found)) * step;
    lo += skip, n = min(step, n - skip);
  }
  const int q0 = __ldg(a.cu_q + lo), q1 = __ldg(a.cu_q + lo + 1), k0 = __ldg(a.cu_k + lo), k1 = __ldg(a.cu_k + lo + 1);
  const bool valid = q0 >= 0 && q1 >= q0 && q1 <= a.n_q && k0 >= 0 && k1 >= k0 && k1 <= a.n_k;
  const int64_t t0l = (slot - ((int64_t)(q0 / tile_tok) + lo)) * tile_tok;
  const int q_len = q1 - q0, k_len = k1 - k0;
  const bool work = valid && t0l >= 0 && t0l < q_len;
  const int t0 = work ? (int)t0l : 0;
  const int shift = k_len - q_len;  // query t sees keys 0 .. t + shift
  const int lim_max = work ? max(0, min(q_len, t0 + tile_tok) + shift) : 0;
  const int n_tiles = (lim_max + kKeys - 1) / kKeys;
  // the second product of the last step goes over `end` keys in steps of 16; of
  // the values it reads, those from `end` on are seen by no row
  const int end = lim_max - (n_tiles - 1) * kKeys;
  const bool cut = lim_max % 16 != 0;
  const int head0 = hb << a.log_group, kh = head0 / (a.n_heads / a.n_kv);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = b->tmem;

  if (warp == 0 && lane == 0 && n_tiles > 0) {
    // ================================================================ loads
    int st = 0;
    uint32_t ph = 1;  // parity with which an empty stage is waited for (the first round passes)
    bool first_round = true;
    bool tail = false;
    auto next = [&](uint64_t *bar) -> uint8_t * {  // null once a wait gave up: no copy is started any more
      if (!wait(b, b->empty + st, ph, a.status)) return nullptr;
      ptx::mbar_expect_tx(bar, kStageBytes);
      return ring + st * kStageBytes;
    };
    auto step = [&]() {
      if (++st == kRing) st = 0, ph ^= 1, first_round = false;
    };
    auto load_k = [&](int i) {
      for (int h = 0; h < D / 128; ++h) {
        uint8_t *dst = next(b->full + st);
        if (!dst) return;
        for (int d = 0; d < 2; ++d)
          tma_load3(dst + d * kKeys * 128, &mk, 128 * h + 64 * d, kh, k0 + i * kKeys, b->full + st);
        step();
      }
    };
    auto load_v = [&](int i) {
      for (int h = 0; h < kSub; ++h) {
        const bool last = cut && i == n_tiles - 1 && h == end / 64;  // full when warps 2 and 3 say so
        uint64_t *bar = last ? &b->tail : b->full + st;
        uint8_t *dst = next(bar);
        if (!dst) return;
        tail = tail || last;
        for (int d = 0; d < D / 64; ++d) tma_load3(dst + d * 8192, &mv, 64 * d, kh, k0 + i * kKeys + h * 64, bar);
        step();
      }
    };
    ptx::mbar_expect_tx(&b->q_full, Sh::kQBytes);
    for (int d = 0; d < D / 64; ++d) tma_load3(sq + d * 16384, &mq, 64 * d, head0, q0 + t0, &b->q_full);
    load_k(0);
    for (int i = 0; i < n_tiles && !*(volatile int *)&b->dead; ++i) {
      if (i + 1 < n_tiles) load_k(i + 1);
      load_v(i);
    }
    // after a wait that gave up: what is on its way still lands in this block
    if (*(volatile int *)&b->dead) {
      ptx::mbar_wait_suspend(&b->q_full, 0);
      if (tail) ptx::mbar_wait_suspend(&b->tail, 0);
      for (int s = 0; s < kRing; ++s)
        if (s < st || !first_round) ptx::mbar_wait_suspend(b->full + s, s < st ? ph ^ 1 : ph);
    }
  } else if (warp == 1 && n_tiles > 0) {
    // ============================================================= products
    constexpr uint32_t fmt = kBf ? ((1u << 7) | (1u << 10)) : 0u;
    constexpr uint32_t id_s = (1u << 4) | fmt | ((uint32_t)(kKeys >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t id_o = (1u << 4) | fmt | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t dq = ptx::sdesc_k_sw128(ptx::smem_u32(sq)), dk = ptx::sdesc_k_sw128(ptx::smem_u32(ring)),
                   dv = sdesc_mn_sw128(ptx::smem_u32(ring), 8192);
    const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv, q_hi = (uint32_t)(dq >> 32),
                   k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
    // (reductions: the compiler knows their results to be uniform)
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem), steps = __reduce_max_sync(0xffffffffu, (uint32_t)n_tiles),
                   last = __reduce_max_sync(0xffffffffu, (uint32_t)end);
    const uint32_t go = elect_one();
    uint32_t st = 0;  // ring stage of the next K or V tile
    uint32_t ph = 0;
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
      wait(b, bar, parity, a.status);
      __syncwarp();
      ptx::tc_fence_after();
    };
    auto step = [&]() {
      if (++st == kRing) st = 0, ph ^= 1;
    };
    auto scores = [&](uint32_t buf) {
#pragma unroll
      for (int h = 0; h < D / 128; ++h) {
        warp_wait(b->full + st, ph);
        const uint32_t ql = q_lo + 2 * h * (16384 >> 4), kl = k_lo + st * (kStageBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t oq = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4, ok = ((kk / 4) * kKeys * 128 + (kk % 4) * 32) >> 4;
          if (kk > 0 || h > 0) umma_ss<true>(go, tm + kKeys * buf, ql + oq, q_hi, kl + ok, k_hi, id_s);
          else umma_ss<false>(go, tm + kKeys * buf, ql + oq, q_hi, kl + ok, k_hi, id_s);
        }
        umma_done(go, b->empty + st);
        step();
      }
      umma_done(go, b->s_full + buf);
    };
    auto outputs = [&](uint32_t buf, bool first, uint32_t turn, uint32_t keys) {
#pragma unroll
      for (int h = 0; h < kSub; ++h) {
        warp_wait(b->full + st, ph);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          // the first or second half of the keys' probabilities
          const uint32_t key = 64 * h + 16 * kk;
          if (key % (kKeys / 2) == 0) warp_wait(key == 0 ? b->p_half + buf : b->p_full + buf, turn);
          if (key < keys)
            umma_ts(go, tm + Sh::kO, tm + kKeys * buf + key / 2, v_lo + st * (kStageBytes >> 4) + kk * (2048 >> 4), v_hi,
                    id_o, !first || key > 0);
        }
        umma_done(go, b->empty + st);
        step();
      }
      umma_done(go, &b->o_full);
    };
    warp_wait(&b->q_full, 0);
    scores(0);
    for (uint32_t i = 0; i < steps && !__any_sync(0xffffffffu, *(volatile int *)&b->dead); ++i) {
      if (i + 1 < steps) {
        // their buffer holds the probabilities of step i - 1: the product that
        // reads those has to be through (products of different accumulators
        // keep no order of their own)
        if (i > 0) warp_wait(&b->o_full, (i - 1) & 1);
        scores((i + 1) & 1);
      }
      outputs(i & 1, i == 0, (i >> 1) & 1, i + 1 < steps ? kKeys : last);
    }
    // (a row may come to its end two products ahead: o_full's parity would not
    // tell the last product from the one before the last)
    umma_done(go, &b->done);
  } else if ((warp == 2 || warp == 3) && cut) {
    // ====================== zeros for the values of the last step that no row
    // of the block sees: a probability of zero times a NaN there would be a NaN
    // in every row
    constexpr int kPieces = D / 8, kPass = 64 / kPieces;  // 16-byte pieces of a row; rows at a time
    // in front of these values lie the keys of all steps and all other values
    const int st = (D / 128 * n_tiles + kSub * (n_tiles - 1) + end / 64) % kRing;
    const int piece = (threadIdx.x - 64) % kPieces, r0 = end % 64 + (threadIdx.x - 64) / kPieces, r1 = (end % 64 | 15) + 1;
    uint8_t *rows = ring + st * kStageBytes + (piece >> 3) * 8192 + ((piece & 7) << 4);
    wait(b, &b->tail, 0, a.status);
#pragma unroll
    for (int i = 0; i < 16; i += kPass)
      if (r0 + i < r1) *reinterpret_cast<uint4 *>(rows + (r0 + i) * 128) = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (threadIdx.x == 64) ptx::mbar_arrive(b->full + st);
  } else if (warp >= 4 && work) {
    // ============================================================== softmax
    const int row0 = 32 * (warp & 3), row = row0 + lane;
    const int tok = t0 + (row >> a.log_group), head = head0 + (row & (a.group - 1));
    const bool mine = tok < q_len;
    const int lim = mine ? max(0, tok + shift + 1) : 0;
    const uint32_t lanes = (uint32_t)row0 << 16;
    const uint32_t t_o = tmem + lanes + Sh::kO;
    const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n_tiles && !*(volatile int *)&b->dead; ++i) {
      const int buf = i & 1;
      const uint32_t t_s = tmem + lanes + kKeys * buf;
      wait(b, b->s_full + buf, (i >> 1) & 1, a.status);
      __syncwarp();
      ptx::tc_fence_after();
      constexpr int kHalf = kKeys / 2;
      uint32_t s[kKeys];
      const int left = lim - i * kKeys;  // keys of this tile that the row sees
#pragma unroll
      for (int j = 0; j < kKeys; j += 32) tmem_ld32(t_s + j, s + j);
      ptx::tmem_wait_ld();
      if (__any_sync(0xffffffffu, left < kKeys)) {
#pragma unroll
        for (int j = 0; j < kKeys; ++j) s[j] = j < left ? s[j] : 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kKeys; j += 2)
        mx[(j >> 1) & 3] = fmaxf(fmaxf(mx[(j >> 1) & 3], __uint_as_float(s[j])), __uint_as_float(s[j + 1]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
      if (__any_sync(0xffffffffu, top > m + kLazy || (m == -INFINITY && top > -INFINITY))) {
        const float mn = fmaxf(m, top);
        const float f = m == -INFINITY ? 0.f : ex2(m - mn);
        m = mn;
        l *= f;
        if (i > 0) {
          // the product of the step in front has to be in
          wait(b, &b->o_full, (i - 1) & 1, a.status);
          __syncwarp();
          ptx::tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + d, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            ptx::tmem_st32x32b_x32(t_o + d, o);
          }
        }
      }
      const float neg = m == -INFINITY ? 0.f : -m;
      const uint64_t neg2 = pair(neg, neg);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[kHalf / 2];
#pragma unroll
        for (int j = 0; j < kHalf / 2; ++j) {
          const float2 z = unpair(fma2(pair(__uint_as_float(s[kHalf * h + 2 * j]), __uint_as_float(s[kHalf * h + 2 * j + 1])), scale2, neg2));
          const float x = ex2(z.x), y = ex2(z.y);
          sum[j & 1] = add2(sum[j & 1], pair(x, y));
          p[j] = kBf ? pack_bf16(x, y) : pack_f16(x, y);
        }
        // over scores that are in registers
#pragma unroll
        for (int j = 0; j < kHalf / 2; j += 16) tmem_st16(t_s + kHalf / 2 * h + j, p + j);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive((h == 0 ? b->p_half : b->p_full) + buf);
      }
      const float2 both = unpair(add2(sum[0], sum[1]));
      l += both.x + both.y;
    }
    // ---- rows out, through the warp's part of Q's place (the products that
    // read it are done), so that a store covers whole rows
    bool odd = false;
    if (n_tiles > 0) {
      wait(b, &b->done, 0, a.status);
      __syncwarp();
      ptx::tc_fence_after();
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    constexpr int kPieces = D / 8;  // of 16 bytes in a row
    uint8_t *mine_out = sq + row0 * D * 2;
#pragma unroll 1
    for (int d = 0; d < D; d += 32) {
      uint32_t o[32];
      if (n_tiles > 0) {
        tmem_ld32(t_o + d, o);
        ptx::tmem_wait_ld();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0u;
      }
      float chk = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[8 * j + e]) * inv, chk = fmaf(x[e], 0.f, chk);
        store8<T>(reinterpret_cast<T *>(mine_out + lane * D * 2 + (((d / 8 + j) ^ (lane & 7)) << 4)), x);
      }
      odd = odd || !(chk == 0.f);
    }
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < kPieces; ++i) {
      const int id = i * 32 + lane, r = id / kPieces, piece = id % kPieces;
      const int t = t0 + ((row0 + r) >> a.log_group), hd = head0 + ((row0 + r) & (a.group - 1));
      const uint4 v = *reinterpret_cast<const uint4 *>(mine_out + r * D * 2 + ((piece ^ (r & 7)) << 4));
      if (t < q_len)
        *reinterpret_cast<uint4 *>((T *)a.out + (int64_t)(q0 + t) * a.out_stride + (int64_t)hd * D + piece * 8) = v;
    }
    ptx::tc_fence_before();
    // (a sum that is NaN comes from a score that counts: the row is NaN)
    uint32_t again = __ballot_sync(0xffffffffu, odd && mine && l == l);
    __syncwarp();  // the rows are written: an odd one is written again
    while (again) {
      const int src = __ffs(again) - 1;
      again &= again - 1;
      __syncwarp();
      row_again<T, D>(a, q0 + __shfl_sync(0xffffffffu, tok, src), __shfl_sync(0xffffffffu, head, src), k0,
                      __shfl_sync(0xffffffffu, lim, src));
    }
  }
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc(tmem, Sh::kColumns);
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = nullptr;
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = (EncodeTiled)p;
  }
  return fn;
}

// [tokens, heads, D] rows of 2-byte elements; boxes of 64 x heads x tokens.
bool make_map(CUtensorMap *m, int32_t dtype, const void *p, int64_t stride, int64_t tokens, int heads, int D,
              int box_heads, int box_tokens) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, unit[3] = {1, 1, 1};
  return enc(m, dtype == REDLITE_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void *>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <typename T, int D>
int launch_attn(const AttnArgs &a, int32_t dtype, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const int tile_tok = kRows >> a.log_group;
  // without keys no K or V box is loaded; the maps still need an address
  const void *k = a.n_k > 0 ? a.k : a.q, *v = a.n_k > 0 ? a.v : a.q;
  const int64_t ks = a.n_k > 0 ? a.k_stride : a.q_stride, vs = a.n_k > 0 ? a.v_stride : a.q_stride;
  const int hk = a.n_k > 0 ? a.n_kv : a.n_heads;
  const int64_t nk = a.n_k > 0 ? a.n_k : a.n_q;
  if (!make_map(&mq, dtype, a.q, a.q_stride, a.n_q, a.n_heads, D, a.group, tile_tok) ||
      !make_map(&mk, dtype, k, ks, nk, hk, D, 1, Shape<D>::kKeys) || !make_map(&mv, dtype, v, vs, nk, hk, D, 1, 64))
    return REDLITE_ECUDA;
  if (cudaFuncSetAttribute(attn_prefill_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, attn_smem<D>()) != cudaSuccess)
    return REDLITE_ECUDA;
  const int64_t grid = ((int64_t)a.n_q / tile_tok + a.n_seqs) * (a.n_heads >> a.log_group);
  if (grid >= ((int64_t)1 << 31) - 1) return REDLITE_EUNSUPPORTED;
  return launch_early(attn_prefill_kernel<T, D>, (unsigned)grid, 256, attn_smem<D>(), s, mq, mk, mv, a) == cudaSuccess
             ? REDLITE_OK
             : REDLITE_ECUDA;
}

}  // namespace
}  // namespace redlite

using namespace redlite;

extern "C" int redlite_attn_prefill(int32_t dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                    const void *v, int64_t v_stride, const int32_t *cu_q, const int32_t *cu_k,
                                    int32_t n_seqs, int32_t n_q, int32_t n_k, int32_t n_heads, int32_t n_kv_heads,
                                    int32_t head_dim, float scale, void *out, int64_t out_stride, int32_t *status,
                                    void *stream) {
  if (!dtype_ok(dtype) || n_seqs < 0 || n_q < 0 || n_k < 0 || n_heads < 1 || n_heads > 4096 || n_kv_heads < 1 ||
      n_heads % n_kv_heads)
    return REDLITE_EINVAL;
  if (dtype == REDLITE_T_F32 || (head_dim != 128 && head_dim != 256)) return REDLITE_EUNSUPPORTED;
  if (!(scale > 0.f) || !(scale < INFINITY)) return REDLITE_EINVAL;
  if (n_seqs == 0 || n_q == 0) return REDLITE_OK;
  if (!q || !out || !cu_q || !cu_k || (n_k > 0 && (!k || !v))) return REDLITE_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return REDLITE_EINVAL;
  const int64_t row_q = (int64_t)n_heads * head_dim, row_k = (int64_t)n_kv_heads * head_dim;
  if (!stride_ok(q_stride, row_q, dtype) || !stride_ok(out_stride, row_q, dtype)) return REDLITE_EINVAL;
  if (n_k > 0 && (!stride_ok(k_stride, row_k, dtype) || !stride_ok(v_stride, row_k, dtype))) return REDLITE_EINVAL;
  if (q_stride >= (int64_t)1 << 38 || k_stride >= (int64_t)1 << 38 || v_stride >= (int64_t)1 << 38)
    return REDLITE_EUNSUPPORTED;
  AttnArgs a;
  a.q = q, a.k = k, a.v = v, a.out = out;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.out_stride = out_stride;
  a.cu_q = cu_q, a.cu_k = cu_k, a.n_seqs = n_seqs, a.n_q = n_q, a.n_k = n_k, a.n_heads = n_heads, a.n_kv = n_kv_heads;
  const int ratio = n_heads / n_kv_heads;
  a.log_group = 0;
  while (a.log_group < 6 && ratio % (2 << a.log_group) == 0) ++a.log_group;
  a.group = 1 << a.log_group;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == REDLITE_T_BF16)
    return head_dim == 256 ? launch_attn<__nv_bfloat16, 256>(a, dtype, s) : launch_attn<__nv_bfloat16, 128>(a, dtype, s);
  return head_dim == 256 ? launch_attn<__half, 256>(a, dtype, s) : launch_attn<__half, 128>(a, dtype, s);
}
