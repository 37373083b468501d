// Attention over packed prompts of different lengths in the explicit form
// (mla_prefill_packed): for token i and the tokens j of its own sequence that it sees,
//   s_ij = scale (q_nope_i . k_nope_j + q_pe_i . k_pe_j),  o_i = sum_j softmax(s_i)_j v_j.
//
// 2 (192 + 128) operations per (query, key, head) against 512 bytes of keys and values
// per key and head: bound by the tensor pipe, and on a long prompt by the power limit
// (the clock falls from 1.97 to 1.6 GHz; every instruction added to the softmax loop
// showed in the time).
//
// Work is cut along the packed rows, not along the sequences: a block is 256 rows of
// one head, whatever sequences they belong to, over the keys from its first row's
// sequence start to its last row.  A batch of short prompts so fills its tiles, the
// number of blocks is known to the host without the offsets, and a row's keys are just
// a range [lo, hi).  A persistent CTA takes blocks from the launch control, one after
// the other (a grid of blocks paid 12000 cycles a block for its start and end):
//   warp 3       plans the next block: which rows and head, which keys;
//   warp 0       loads by TMA: the queries of both 128-row tiles A and B, then keys and
//                values in 16 KB chunks round a ring;
//   warps 1, 2   issue the products of tile A and of tile B (tcgen05, M = N = 128): the
//                scores S = Q K^T into tensor memory and O += P V with P from there;
//   warps 4..11  softmax, a thread per query row: weights over the scores in place, and
//                the output at the end.
// While one tile's softmax runs, the other tile's products do: per key tile and query
// tile 1280 cycles of products (d_r = 64; 1024 without) stand against some 1500 of
// softmax, 1024 of them exponentials at the special-function units' rate.
//
// Measured (us; in long runs back to back, and over a few tens of passes): one prompt of
// 4096 tokens, 128 heads 637 and 550 (1.08 and 1.25 PFLOP/s; cuBLAS 1.38 and 1.62); 7
// prompts of 5120 tokens, 128 heads 392 and 337 to 354; 5 prompts of 7001 tokens, 32 heads in
// groups of 4 without the RoPE part 141 and 127; 67 prompts of 8191 tokens, 16 heads 57
// and 56; one of 17 tokens 6.8 to 7.5.  The causal form of one prompt of 4096 tokens, 32
// heads 160, not causal 268 (twice the products).
#include <math_constants.h>

#include "packed.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace mla {
uint64_t device_wait_limit_ns();
// tma_map_3d without the cache of encoded maps, for tensors that a caller passes anew
// each time (tma_host.cu)
bool tma_map_3d_fresh(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2,
                      uint32_t b0, uint32_t b1, uint32_t b2);

namespace {

using namespace sm100;

constexpr uint64_t kDrainNs = 100000000ull;

struct PackedParams {
  const __nv_bfloat16* q_nope;
  const __nv_bfloat16* q_pe;
  const __nv_bfloat16* k_nope;
  const __nv_bfloat16* k_pe;
  const __nv_bfloat16* v;
  const int32_t* cu;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  int64_t qn_tok, qn_head, qp_tok, qp_head, kn_tok, kn_head, kp_tok, v_tok, v_head;
  int n_tok, B, H, share, causal, blocks, wide, group, sorted;
  float scale_log2;
  uint64_t wait_ns;
};

MLA_DEVI float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    acc = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), acc);
    acc = fmaf(__uint_as_float(x[k] & 0xffff0000u), __uint_as_float(y[k] & 0xffff0000u), acc);
  }
  return acc;
}

// Row t of head h over the keys [lo, hi), by one warp: a lane scores one key of
// every 32 and owns four values of the output.  6 us per 32 keys where all warps of
// the GPU are at it, so that 32 rows of some 300000 keys take longer than the block's
// other warps may wait: `done` counts the steps for them.
template <bool PE>
MLA_DEVI void attend_row(const PackedParams& p, int t, int h, int lo, int hi, int lane, int* done) {
  const int g = h / p.share;
  const uint4* qn = reinterpret_cast<const uint4*>(p.q_nope + (int64_t)t * p.qn_tok + (int64_t)h * p.qn_head);
  const uint4* qp = reinterpret_cast<const uint4*>(p.q_pe + (int64_t)t * p.qp_tok + (int64_t)h * p.qp_head);
  float m = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    if (lane == 0) atomicAdd(done, 1);
    const int j = j0 + lane;
    float s = -CUDART_INF_F;
    if (j < hi) {
      const uint4* kn = reinterpret_cast<const uint4*>(p.k_nope + (int64_t)j * p.kn_tok + (int64_t)g * p.kn_head);
      float acc = 0.f;
#pragma unroll 4
      for (int c = 0; c < kDn / 8; ++c) acc = dot8(qn[c], kn[c], acc);
      if constexpr (PE) {
        const uint4* kp = reinterpret_cast<const uint4*>(p.k_pe + (int64_t)j * p.kp_tok);
#pragma unroll 4
        for (int c = 0; c < kDr / 8; ++c) acc = dot8(qp[c], kp[c], acc);
      }
      s = acc * p.scale_log2;
    }
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float m_new = fmaxf(m, top);
    const float ref = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float alpha = exp2f(m - ref);
    const float w = j < hi ? exp2f(s - ref) : 0.f;
    m = m_new;
    l = l * alpha + w;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= alpha;
    const int n = min(32, hi - j0);
    const __nv_bfloat16* v = p.v + (int64_t)j0 * p.v_tok + (int64_t)g * p.v_head + 4 * lane;
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const uint2 x = *reinterpret_cast<const uint2*>(v + (int64_t)k * p.v_tok);
      o[0] = fmaf(wk, __uint_as_float(x.x << 16), o[0]);
      o[1] = fmaf(wk, __uint_as_float(x.x & 0xffff0000u), o[1]);
      o[2] = fmaf(wk, __uint_as_float(x.y << 16), o[2]);
      o[3] = fmaf(wk, __uint_as_float(x.y & 0xffff0000u), o[3]);
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  // every score -inf: nothing to weigh, zeros and lse = -inf
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = (int64_t)t * p.H + h;
  *reinterpret_cast<uint2*>(p.out + row * kDv + 4 * lane) =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- tiles
constexpr int kThreads = 384;               // warp 0 loads, 1 and 2 MMA, 3 plans, 4..7 tile A, 8..11 tile B
constexpr int kRows = 256;                  // packed rows of a block: tile A the first 128, B the others
constexpr uint32_t kChunk = 128 * 128;      // 16 KB: 128 rows x 64 values, or 64 keys x 128 values
constexpr int kHeadGroup = 16;              // key and value heads whose blocks run side by side
constexpr int kMaxSorted = 128;             // blocks of rows that are put in order of their work

template <bool PE>
struct Cfg {
  static constexpr int kQk = PE ? 3 : 2;              // 64-value chunks of a query or key
  static constexpr int kSlots = PE ? 8 : 10;          // ring of K and V chunks
  static constexpr int kPer = kQk + 2;                // chunks of one key tile: K, then V in halves of 64 keys
  // K(j) may go in once the item kWait before it has been read, V(j) likewise: with 8
  // slots of which a key tile takes 3 + 2, K(j) ends at 5 j + 3 and needs V(j - 2), which
  // ends at 5 j - 5, gone; V(j) ends at 5 j + 5 and needs K(j - 1), which ends at 5 j - 2,
  // gone.  With 10 slots of 2 + 2, K(j) needs 4 j - 8 (V(j - 3)) and V(j) 4 j - 6 (K(j - 2)).
  static constexpr int kWait = PE ? 3 : 5;
  static constexpr uint32_t kRing = 2 * kQk * kChunk;
  static constexpr uint32_t kBars = kRing + kSlots * kChunk;
  static constexpr uint32_t kSmem = kBars + 1024 + 1024;
};
static_assert(Cfg<true>::kSmem <= 232448 && Cfg<false>::kSmem <= 232448, "shared memory budget");

// TMEM: scores (and the weights over them) of tile t at columns 128 t, outputs at 256 + 128 t
constexpr uint32_t kTmemO = 256;
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);
constexpr float kRescale = 256.f;             // a tile's weights beyond this ask for a new reference
constexpr float kBeyond = 1.152921504606847e18f;  // 2^60: no range is left to wait for it
// Barriers.  [2] per query tile: its queries are in / have been read, its scores are
// there, its output is there / has been read; P [2 t + half] its weights; [8] per ring
// item in turn; [2] per plan in turn.
constexpr int B_Q = 0, B_READ_Q = 2, B_S = 4, B_P = 6, B_O = 10, B_READ_O = 12, B_TURN = 14, B_DRAIN = 16, B_FULL = 18,
              B_EMPTY = 26, B_PLAN = 34, B_READ_PLAN = 36, B_NEXT = 38, B_BEGUN = 39, B_COUNT = 40;
// behind the barriers: the answer of the launch control, words, two plans
constexpr uint32_t kNextOff = 320, kWordsOff = 336, kPlanOff = 384;

// What a block of rows and a head needs, as the planning warp leaves it.
struct Plan {
  int h, q0;           // head (-1: no more work) and first row
  int k0, n;           // first key of the block's first key tile, key tiles
  int from[2], to[2];  // those of them that query tile A and B see
  // per 32 rows: those of a sequence, the first one's first key and its sequence's end,
  // whether all are of that sequence
  int first[8], last[8], lo[8], hi[8], one[8];
};
constexpr uint32_t kOrderOff = kPlanOff + 2 * sizeof(Plan);
static_assert(kOrderOff + kMaxSorted <= 1024 && kWordsOff + 48 <= kPlanOff && 8 * B_COUNT <= kNextOff, "layout");

MLA_DEVI uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
MLA_DEVI void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
MLA_DEVI uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
MLA_DEVI uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Four single-CTA MMAs of one chunk (K = 64 in steps of 16) in one go: one election
// and one set of operands for the four, descriptors advanced by the given steps (in
// their 16-byte units; tensor-memory A by columns).  `accumulate` is the first one's;
// the others always accumulate.
template <int kAStep, int kBStep>
MLA_DEVI void mma_1_x4_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b32 rx;\n\t.reg .b64 a, b;\n\t"
      "elect.sync rx|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "n"(kAStep), "n"(kBStep)
      : "memory");
}
template <int kAStep, int kBStep>
MLA_DEVI void mma_1_ts_x4_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b32 rx, a;\n\t.reg .b64 b;\n\t"
      "elect.sync rx|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s32 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s32 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "n"(kAStep), "n"(kBStep)
      : "memory");
}
// Moves a warpgroup's share of the register file: the sum over the block's
// warpgroups must not exceed what the block was launched with.
template <int kRegs>
MLA_DEVI void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
MLA_DEVI void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// The next block that has not been started, asked of the launch control: written to
// `answer` (16 bytes, counted on `bar`), read by next_block (negative: there is none).
MLA_DEVI void ask_next(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}
MLA_DEVI int next_block(uint32_t answer) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "mov.s32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(x)
      : "r"(answer)
      : "memory");
  return x;
}
MLA_DEVI void prefetch_map(const void* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
// 32 bytes to global memory
MLA_DEVI void stg256(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// maximum of three that keeps a NaN
MLA_DEVI float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool PE>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qp,
                       const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_kp,
                       const __grid_constant__ CUtensorMap tm_v, const PackedParams p) {
  using C = Cfg<PE>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sa = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (sa - raw);
  // warp-uniform, and known to be: what the MMA warps compute stays in uniform registers
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sa + C::kBars + 8u * i; };
  auto slot = [&](int s) -> uint32_t { return sa + C::kRing + (s % C::kSlots) * kChunk; };
  int* words = reinterpret_cast<int*>(sm + C::kBars + kWordsOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort_flag = words + 1;
  int* issued = words + 2;  // ring items, queries of tile A, of B
  int* done_over = words + 5;  // steps of rows that are done over
  Plan* plans = reinterpret_cast<Plan*>(sm + C::kBars + kPlanOff);
  const uint64_t wait_ns = p.wait_ns;
  auto wait = [&](int b, int parity) {
    return mbar_wait_converged(bar(b), parity & 1, abort_flag, p.status, wait_ns, done_over);
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive_local(bar(b));
    __syncwarp();
  };

  if (warp == 2 && lane == 0) {
    prefetch_map(&tm_qn);
    prefetch_map(&tm_kn);
    prefetch_map(&tm_v);
    if constexpr (PE) {
      prefetch_map(&tm_qp);
      prefetch_map(&tm_kp);
    }
  }
  int cu0 = 0, cu1 = 0;  // of the planning warp
  if (warp == 3) {
    pdl_wait();
    cu0 = min(max(p.cu[0], 0), p.n_tok);
    cu1 = min(max(p.cu[p.B], 0), p.n_tok);
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    issued[0] = issued[1] = issued[2] = *done_over = 0;
    for (int i = 0; i < B_COUNT; ++i) {
      int count = 1;
      if ((i >= B_P && i < B_P + 4) || (i >= B_READ_O && i < B_READ_O + 2)) count = 4;  // a softmax warp each
      if (i >= B_EMPTY && i < B_EMPTY + 8) count = 2;                                    // both MMA warps
      if (i >= B_READ_PLAN && i < B_READ_PLAN + 2) count = 11;                           // all warps but the planning one
      mbar_init(bar(i), count);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_1(smem_u32(tmem_slot), 512);
    tmem_relinquish_1();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // Every warp goes through the same plans, its own counters running on from one to
  // the next; a barrier's phase is the count of its uses.  One warp loads, so the
  // next block's keys and queries come in under the last block's tail, and its first
  // scores are formed under the last one's output.
  if (warp < 4) {
    regs_dec<80>();  // 384 threads launched with 168 registers: 128 x 80 + 256 x 208 is within that
    if (warp == 3) {
      // =========================== plans ===========================
      const uint32_t answer = sa + C::kBars + kNextOff;
      // the sequence of row r, for rows [cu0, cu1): its bounds
      auto find = [&](int r, int& lo, int& hi) {
        int a = 0, z = p.B;  // the count of entries cu[1 .. B] that are <= r
        while (a < z) {
          const int mid = a + (z - a) / 2;
          if (p.cu[mid + 1] <= r)
            a = mid + 1;
          else
            z = mid;
        }
        a = min(a, p.B - 1);
        lo = min(max(p.cu[a], 0), r);
        hi = max(min(p.cu[a + 1], p.n_tok), r + 1);
      };
      uint8_t* order = sm + C::kBars + kOrderOff;
      if (p.sorted) {
        // the blocks by falling number of key tiles, so that the last ones to be taken are short
        int mine[kMaxSorted / 32], rank[kMaxSorted / 32];
#pragma unroll
        for (int k = 0; k < kMaxSorted / 32; ++k) {
          const int b = lane + 32 * k, first = max(b * kRows, cu0), last = min(b * kRows + kRows, cu1) - 1;
          mine[k] = b < p.blocks ? 0 : -1;
          rank[k] = 0;
          if (b < p.blocks && first <= last) {
            int lo, hi, lo2;
            find(first, lo, hi);
            hi = last + 1;
            if (!p.causal) find(last, lo2, hi);
            mine[k] = (hi - lo + 127) >> 7;
          }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kMaxSorted / 32; ++k)
          for (int l = 0; l < 32 && 32 * k + l < p.blocks; ++l) {
            const int other = __shfl_sync(0xffffffffu, mine[k], l), b = 32 * k + l;
#pragma unroll
            for (int m = 0; m < kMaxSorted / 32; ++m) rank[m] += other > mine[m] || (other == mine[m] && b < lane + 32 * m);
          }
#pragma unroll
        for (int k = 0; k < kMaxSorted / 32; ++k)
          if (lane + 32 * k < p.blocks) order[rank[k]] = (uint8_t)(lane + 32 * k);
        __syncwarp();
      }
      int block = blockIdx.x;
      for (int w = 0;; ++w) {
        if (w >= 2 && !wait(B_READ_PLAN + (w & 1), (w >> 1) - 1)) break;
        Plan* pl = plans + (w & 1);
        if (block < 0) {
          if (lane == 0) pl->h = -1;
          arrive(B_PLAN + (w & 1));
          break;
        }
        // groups of heads whose keys and values L2 holds; in a group all heads of the
        // longest block first (unsorted: of the last rows, the longest when causal)
        const int per_group = p.group * p.blocks;
        const int grp = block / per_group, in = block - grp * per_group;
        const int gh = min(p.group, p.H - grp * p.group);
        const int h = grp * p.group + in % gh, at = in / gh;
        const int q0 = (p.sorted ? order[at] : p.blocks - 1 - at) * kRows;
        // lanes 0 .. 7: the first row of 32 that is in a sequence; lanes 8 .. 15: the last
        const int base = q0 + 32 * (lane & 7);
        const int first = max(base, cu0), last = min(base + 31, cu1 - 1);
        const int r = lane & 8 ? last : first;
        int lo = 0, hi = 0;
        const bool any = first <= last;
        if (any && lane < 16) find(r, lo, hi);
        __syncwarp();
        const int lo_last = __shfl_sync(0xffffffffu, lo, (lane & 7) + 8);
        const int hi_last = __shfl_sync(0xffffffffu, hi, (lane & 7) + 8);
        int kl = any ? lo : 0x7fffffff, kh = any ? (p.causal ? last + 1 : hi_last) : 0;
        for (int o = 1; o < 4; o <<= 1) {
          kl = min(kl, __shfl_xor_sync(0xffffffffu, kl, o));
          kh = max(kh, __shfl_xor_sync(0xffffffffu, kh, o));
        }
        const int kl_a = __shfl_sync(0xffffffffu, kl, 0), kl_b = __shfl_sync(0xffffffffu, kl, 4);
        const int kh_a = __shfl_sync(0xffffffffu, kh, 0), kh_b = __shfl_sync(0xffffffffu, kh, 4);
        if (lane < 8) {
          pl->first[lane] = any ? first : 0;
          pl->last[lane] = any ? last : -1;
          pl->lo[lane] = lo;
          pl->hi[lane] = hi;
          pl->one[lane] = lo == lo_last && last < hi;
        }
        const int k0 = min(kl_a, kl_b);
        if (lane == 0) {
          pl->h = h;
          pl->q0 = q0;
          pl->k0 = k0;
          pl->from[0] = kh_a > kl_a ? (kl_a - k0) / 128 : 0;
          pl->to[0] = kh_a > kl_a ? (kh_a - k0 + 127) / 128 : 0;
          pl->from[1] = kh_b > kl_b ? (kl_b - k0) / 128 : 0;
          pl->to[1] = kh_b > kl_b ? (kh_b - k0 + 127) / 128 : 0;
          pl->n = max(pl->to[0], pl->to[1]);
        }
        arrive(B_PLAN + (w & 1));
        if (w == 0 && blockIdx.x == 0) packed_check(p.cu, p.B, p.n_tok, p.status, lane, 32);
        // The next block is claimed when the loads of this one begin, not before: a block
        // held in store is one that an idle SM cannot take.
        if (!wait(B_BEGUN, w)) break;
        if (lane == 0) {
          fence_proxy_async_smem();  // the last answer has been read
          mbar_arrive_expect_tx_local(bar(B_NEXT), 16);
          ask_next(answer, bar(B_NEXT));
        }
        __syncwarp();
        if (!wait(B_NEXT, w)) {
          int give_up = 0;  // the answer must not outlive the block
          mbar_wait_converged(bar(B_NEXT), w & 1, &give_up, nullptr, kDrainNs);
          break;
        }
        block = next_block(answer);
      }
    } else if (warp == 0) {
      // =========================== loads ===========================
      // Items in the ring, each with a full and an empty barrier of eight taken in turn:
      // a key tile's K is item 2 j (kQk slots), its V item 2 j + 1 (two slots), j counting
      // the key tiles of all blocks.
      bool ok = true;
      int jj = 0, nq[2] = {0, 0};
      for (int w = 0; ok; ++w) {
        if (!wait(B_PLAN + (w & 1), w >> 1)) break;
        const Plan* pl = plans + (w & 1);
        const int h = pl->h, q0 = pl->q0, k0 = pl->k0, n = pl->n;
        const bool on[2] = {pl->to[0] > pl->from[0], pl->to[1] > pl->from[1]};
        arrive(B_READ_PLAN + (w & 1));
        if (h < 0) break;
        arrive(B_BEGUN);
        const int g = h / p.share;
        auto item = [&](int j, int v) {
          const int it = 2 * (jj + j) + v, old = it - C::kWait, key = k0 + 128 * j;
          if (old >= 0 && !wait(B_EMPTY + (old & 7), old >> 3)) return false;
          if (lane == 0) {
            const uint32_t f = bar(B_FULL + (it & 7));
            const int s = C::kPer * (jj + j) + (v ? C::kQk : 0);
            mbar_arrive_expect_tx_local(f, (v ? 2 : C::kQk) * kChunk);
            if (v == 0) {
              tma_load_3d_cta(slot(s), &tm_kn, f, 0, g, key);
              tma_load_3d_cta(slot(s + 1), &tm_kn, f, 64, g, key);
              if constexpr (PE) tma_load_3d_cta(slot(s + 2), &tm_kp, f, 0, 0, key);
            } else {
              // halves of 64 keys, 128 values each
              for (int half = 0; half < 2; ++half) {
                tma_load_3d_cta(slot(s + half), &tm_v, f, 0, g, key + 64 * half);
                tma_load_3d_cta(slot(s + half) + kChunk / 2, &tm_v, f, 64, g, key + 64 * half);
              }
            }
            issued[0] = it + 1;
          }
          __syncwarp();
          return true;
        };
        // Tile A's queries first: their place is free as soon as the last block's scores of
        // tile A are there, long before the ring has room for K(0) (the other way round cost
        // 3000 cycles a block).
        for (int i = 0; ok && i < 2; ++i) {
          if (on[i]) {
            if (nq[i] > 0) ok = wait(B_READ_Q + i, nq[i] - 1);
            if (!ok) break;
            ++nq[i];
            if (lane == 0) {
              // (rows past the end read as zeros)
              const uint32_t dst = sa + i * C::kQk * kChunk;
              mbar_arrive_expect_tx_local(bar(B_Q + i), C::kQk * kChunk);
              tma_load_3d_cta(dst, &tm_qn, bar(B_Q + i), 0, h, q0 + 128 * i);
              tma_load_3d_cta(dst + kChunk, &tm_qn, bar(B_Q + i), 64, h, q0 + 128 * i);
              if constexpr (PE) tma_load_3d_cta(dst + 2 * kChunk, &tm_qp, bar(B_Q + i), 0, h, q0 + 128 * i);
              issued[1 + i] = nq[i];
            }
            __syncwarp();
          }
          if (i == 0 && n > 0) ok = item(0, 0);
        }
        for (int j = 0; ok && j < n; ++j) {
          if (j > 0) ok = item(j, 0);
          if (ok) ok = item(j, 1);
        }
        jj += n;
      }
    } else {
      // =========================== MMA issue ===========================
      // One warp per query tile: P.V, then the next scores, while the other tile's
      // softmax runs under them.  (One warp for both issued 40 MMAs, six waits and four
      // commits per key tile, 3500 cycles of it, more than the 2560 that the tensor pipe
      // needs.)  The pipe takes a warp's products in order, so scores may follow the P.V
      // that reads the weights they overwrite without a wait between the two.
      const int i = warp - 1;
      bool ok = true;
      int jj = 0, its = 0, nq = 0;  // key tiles of all blocks, those seen, blocks with rows
      for (int w = 0; ok; ++w) {
        if (!wait(B_PLAN + (w & 1), w >> 1)) break;
        const Plan* pl = plans + (w & 1);
        const int h = pl->h, n = pl->n, from = pl->from[i], to = pl->to[i];
        arrive(B_READ_PLAN + (w & 1));
        if (h < 0) break;
        if (n == 0) continue;
        auto arrived = [&](int j, int v) {
          const int it = 2 * (jj + j) + v;
          return wait(B_FULL + (it & 7), it >> 3);
        };
        auto release = [&](int j, int v) { commit_1_elect(bar(B_EMPTY + ((2 * (jj + j) + v) & 7))); };
        auto sees = [&](int j) { return j >= from && j < to; };
        // scores over the block's K(j)
        auto scores = [&](int j) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::kQk; ++c)
            mma_1_x4_elect<2, 2>(tmem + 128u * i, desc_sw128(sa + (i * C::kQk + c) * kChunk, 16, 1024),
                                 desc_sw128(slot(C::kPer * (jj + j) + c), 16, 1024), kIdescS, c != 0);
          commit_1_elect(bar(B_S + i));
          if (j + 1 == to) commit_1_elect(bar(B_READ_Q + i));
        };
        // the weights of half a key tile times V(j): 16 keys a step, weights in 8 columns, V
        // rows 2 KB further on
        auto values = [&](int j, int half) {
          tc_fence_after();
          mma_1_ts_x4_elect<8, 128>(tmem + kTmemO + 128u * i, tmem + 128u * i + 32u * half,
                                    desc_sw128(slot(C::kPer * (jj + j) + C::kQk + half), kChunk / 2, 1024), kIdescPV,
                                    (j > from || half) ? 1u : 0u);
        };
        if (to > from) ok = wait(B_Q + i, nq);
        ok = ok && arrived(0, 0);
        if (!ok) break;
        if (sees(0)) scores(0);
        release(0, 0);
        for (int j = 0; ok && j < n; ++j) {
          const bool mine = sees(j), more = j + 1 < n;
          ok = arrived(j, 1);
          // the last block's output has been read
          if (mine && j == from && nq > 0) ok = ok && wait(B_READ_O + i, nq - 1);
          if (mine) ok = ok && wait(B_P + 2 * i, its);
          // in turn: A's products of key tile j, then B's, then A's of the next
          if (i + jj + j > 0) ok = ok && wait(B_TURN + i, i ? jj + j : jj + j - 1);
          if (!ok) break;
          if (mine) values(j, 0);
          if (more) ok = arrived(j + 1, 0);
          if (mine) ok = ok && wait(B_P + 2 * i + 1, its);
          if (!ok) break;
          if (mine) {
            values(j, 1);
            ++its;
            if (j + 1 == to) commit_1_elect(bar(B_O + i));
          }
          release(j, 1);
          if (sees(j + 1)) scores(j + 1);
          arrive(B_TURN + 1 - i);
          if (more) release(j + 1, 0);
        }
        jj += n;
        if (to > from) ++nq;
      }
      commit_1_elect(bar(B_DRAIN + i));
      int keep = 0;
      mbar_wait_converged(bar(B_DRAIN + i), 0, &keep, p.status, kDrainNs);
    }
  } else {
    regs_inc<208>();
    // ================ softmax: a thread per query row ================
    const int t = (warp - 4) >> 2;                     // query tile
    const int row = 32 * (warp & 3) + lane;            // its TMEM lane
    const int grp = 4 * t + (warp & 3);
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t cs = 128u * t, co = kTmemO + 128u * t;
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    bool ok = true;
    int its = 0, nq = 0;
    for (int w = 0; ok; ++w) {
      if (!wait(B_PLAN + (w & 1), w >> 1)) break;
      const Plan* pl = plans + (w & 1);
      const int h = pl->h, k0 = pl->k0, from = pl->from[t], to = pl->to[t];
      const int qi = pl->q0 + 128 * t + row;
      // the keys of this row: of its own sequence, up to itself when causal
      int lo = 0, hi = 0;
      if (h >= 0 && qi >= pl->first[grp] && qi <= pl->last[grp]) {
        lo = pl->lo[grp];
        hi = pl->hi[grp];
        if (!pl->one[grp]) {
          const PackedRow r = packed_own(p.cu, p.B, p.n_tok, qi);
          lo = r.lo;
          hi = r.hi;
        }
        if (p.causal && hi > lo) hi = qi + 1;
      }
      arrive(B_READ_PLAN + (w & 1));
      if (h < 0) break;
      if (to <= from) continue;
      float m_used = -CUDART_INF_F, l = 0.f;
      bool stale = true;  // the reference m_used has to be found (again)
      for (int j = from; j < to; ++j, ++its) {
        ok = wait(B_S + t, its);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tl + cs + 32u * c, sr[c]);
        tmem_wait_ld();
        const int kb = k0 + 128 * j;
        if (__any_sync(0xffffffffu, lo > kb || hi < kb + 128)) {
          const uint32_t a = (uint32_t)max(lo - kb, 0), n = (uint32_t)max(min(hi - kb, 128) - (int)a, 0);
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if ((uint32_t)k - a >= n) sr[k >> 5][k & 31] = 0xff800000u;
        }
        auto score = [&](int k) { return __uint_as_float(sr[k >> 5][k & 31]); };
        // The weights are 2^(s scale - m) for a reference m near the row's maximum so far,
        // not the maximum itself: any m gives the same quotient, as long as the weights
        // and their sums stay within fp32 and bf16's common range.  So m is found where
        // there is none and raised one tile after a weight went beyond 2^8; the loop over
        // rows that all have a reference takes no maximum.  A warp in which some row has
        // none yet (its sequence begins later, or it is of no sequence) takes one every
        // tile: one prompt of 4097 tokens, 128 heads 660 us, of 4224 tokens, where no warp
        // has such rows, 640.
        if (__any_sync(0xffffffffu, stale)) {
          float m4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = score(k);
#pragma unroll
          for (int k = 4; k < 124; k += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = max3(m4[i], score(k + 2 * i), score(k + 2 * i + 1));
          m4[0] = max3(m4[0], score(124), score(125));
          m4[1] = max3(m4[1], score(126), score(127));
          float mx = max3(max3(m4[0], m4[1], m4[2]), m4[3], m4[3]) * p.scale_log2;
          // a NaN or an infinite maximum: the row is done over in fp32 at the end
          if (!(mx < CUDART_INF_F)) l = CUDART_NAN_F;
          // the earlier tiles' largest weight counts as well: l is a bound of it
          if (l > 1.f) mx = fmaxf(mx, m_used + log2f(l));
          float alpha = 1.f;
          bool resc = false;
          if (mx > m_used) {
            // (with no weight so far there is nothing to rescale: O holds zeros for this row)
            alpha = ex2_approx(m_used - mx);
            resc = l != 0.f;
            l *= alpha;
            m_used = mx;
          }
          if (__any_sync(0xffffffffu, resc && j > from)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(tl + co + 32u * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st32(tl + co + 32u * c, o);
            }
            tmem_wait_st();
          }
          stale = m_used == -CUDART_INF_F;
        }
        const float ref = m_used == -CUDART_INF_F ? 0.f : -m_used;
        const uint64_t ref2 = pack2(ref, ref);
        uint64_t sum[2] = {0, 0};
        // the weights of 64 keys, in bf16 pairs over the scores and to the MMA warp
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int u = 64 * half + 2 * k;
            float p0, p1;
            unpack2(fma2(pack2(score(u), score(u + 1)), scale2, ref2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum[k & 1] = add2(sum[k & 1], pack2(p0, p1));
            pk[k] = pack_bf16(p0, p1);
          }
          tmem_st32(tl + cs + 32u * half, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_local(bar(B_P + 2 * t + half));
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        const float tile = s0 + s1;
        l += tile;
        stale = stale || tile > kRescale;
        // beyond 2^60 (a NaN included) within one tile: the row is done over as well
        if (!(tile < kBeyond)) l = CUDART_NAN_F;
      }
      // ---- o = O / l, lse
      ok = ok && wait(B_O + t, nq);
      ++nq;
      if (!ok) break;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t o[4][32], pk[64];
      float bad4[4] = {0.f, 0.f, 0.f, 0.f};  // a NaN once any value is infinite or not a number
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tl + co + 32u * c, o[c]);
      tmem_wait_ld();
      tc_fence_before();
      arrive(B_READ_O + t);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float x0 = __uint_as_float(o[c][2 * k]), x1 = __uint_as_float(o[c][2 * k + 1]);
          bad4[k & 3] = fmaf(x0, 0.f, fmaf(x1, 0.f, bad4[k & 3]));
          pk[16 * c + k] = pack_bf16(x0 * inv, x1 * inv);
        }
      const float bad = (bad4[0] + bad4[1]) + (bad4[2] + bad4[3]);
      const bool mine = hi > lo;
      const int64_t orow = (int64_t)qi * p.H + h;
      // The thread writes its own row, 32 bytes (a sector) at a time.  (Exchanging pieces among
      // four lanes so that they write whole lines together: 58.6 us for the 67 prompts of
      // 8191 tokens against 55.2, the shuffles cost more than the store unit saves.)
      if (mine) {
        __nv_bfloat16* dst = p.out + orow * kDv;
        if (p.wide) {
#pragma unroll
          for (int k = 0; k < 8; ++k) stg256(dst + 16 * k, pk + 8 * k);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            reinterpret_cast<uint4*>(dst)[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
      }
      if (mine && p.lse) p.lse[orow] = inv == 0.f ? -CUDART_INF_F : (m_used + log2f(l)) * 0.6931471805599453f;
      // An infinite or NaN value that a row does not see has met its zero weight in the
      // product with V (0 x inf): such rows, and those that see one, are done over from
      // the definition.  So are those whose weights add up to far less than the one that
      // the reference stands for: beyond scores of some 2^28 the reference's own rounding
      // moves the exponents by that much, down to weights that are all flushed to zero.
      const bool lost = l < 1.f / kRescale && m_used != -CUDART_INF_F;
      const bool odd = mine && (bad != 0.f || !(fabsf(l) < CUDART_INF_F) || lost);
      __syncwarp();
      for (uint32_t again = __ballot_sync(0xffffffffu, odd); again; again &= again - 1) {
        const int r = __ffs(again) - 1;
        attend_row<PE>(p, __shfl_sync(0xffffffffu, qi, r), h, __shfl_sync(0xffffffffu, lo, r),
                       __shfl_sync(0xffffffffu, hi, r), lane, done_over);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait that ran out may leave loads in flight: wait (bounded) for the last ones
    int give_up = 0;
    for (int i = 0; i < 2; ++i)
      if (issued[1 + i] > 0) mbar_wait(bar(B_Q + i), (issued[1 + i] - 1) & 1, &give_up, nullptr, kDrainNs);
    for (int it = max(0, issued[0] - 8); it < issued[0]; ++it)
      mbar_wait(bar(B_FULL + (it & 7)), (it >> 3) & 1, &give_up, nullptr, kDrainNs);
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc_1(tmem, 512);
}

template <bool PE>
cudaError_t launch_tiles(const mla_prefill_packed_args_t* a, const PackedParams& p, cudaStream_t stream) {
  using C = Cfg<PE>;
  // a dimension of one may come with any stride: the map needs a valid one
  auto bytes = [](int64_t stride, int64_t extent) { return (uint64_t)(extent > 1 ? 2 * stride : 256); };
  const uint64_t n = a->n_tok;
  CUtensorMap qn, qp = {}, kn, kp = {}, v;
  if (!tma_map_3d_fresh(&qn, a->q_nope, kDn, a->H, n, bytes(a->q_nope_head, a->H), bytes(a->q_nope_tok, n), 64, 1, 128) ||
      !tma_map_3d_fresh(&kn, a->k_nope, kDn, a->H_kv, n, bytes(a->k_nope_head, a->H_kv), bytes(a->k_nope_tok, n), 64, 1, 128) ||
      !tma_map_3d_fresh(&v, a->v, kDv, a->H_kv, n, bytes(a->v_head, a->H_kv), bytes(a->v_tok, n), 64, 1, 64))
    return cudaErrorInvalidValue;
  if (PE && (!tma_map_3d_fresh(&qp, a->q_pe, kDr, a->H, n, bytes(a->q_pe_head, a->H), bytes(a->q_pe_tok, n), 64, 1, 128) ||
             !tma_map_3d_fresh(&kp, a->k_pe, kDr, 1, n, 256, bytes(a->k_pe_tok, n), 64, 1, 128)))
    return cudaErrorInvalidValue;
  static PerDeviceOnce attrs;
  const cudaError_t e = once_per_device(attrs, [&]() {
    return cudaFuncSetAttribute(packed_attn_kernel<PE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(packed_attn_kernel<PE>, dim3((unsigned)((int64_t)p.blocks * a->H)), dim3(kThreads), C::kSmem, stream, qn,
                    qp, kn, kp, v, p);
}

}  // namespace

cudaError_t launch_prefill_packed(const mla_prefill_packed_args_t* a, cudaStream_t stream) {
  PackedParams p;
  p.q_nope = static_cast<const __nv_bfloat16*>(a->q_nope);
  p.q_pe = static_cast<const __nv_bfloat16*>(a->q_pe);
  p.k_nope = static_cast<const __nv_bfloat16*>(a->k_nope);
  p.k_pe = static_cast<const __nv_bfloat16*>(a->k_pe);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  p.cu = a->cu_seqlens;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.status = static_cast<uint32_t*>(a->workspace);
  p.qn_tok = a->q_nope_tok;
  p.qn_head = a->q_nope_head;
  p.qp_tok = a->q_pe_tok;
  p.qp_head = a->q_pe_head;
  p.kn_tok = a->k_nope_tok;
  p.kn_head = a->k_nope_head;
  p.kp_tok = a->k_pe_tok;
  p.v_tok = a->v_tok;
  p.v_head = a->v_head;
  p.n_tok = a->n_tok;
  p.B = a->B;
  p.H = a->H;
  p.share = a->H / a->H_kv;
  p.causal = a->causal;
  p.scale_log2 = a->softmax_scale * kLog2e;
  p.blocks = (int)(((int64_t)a->n_tok + kRows - 1) / kRows);
  p.wait_ns = device_wait_limit_ns();
  p.wide = (reinterpret_cast<uintptr_t>(a->out) & 31u) == 0;  // the ABI asks for 16 bytes
  // 16 key heads at a time: their keys and values stay in L2 while several blocks read
  // them (8 / 16 / 32 heads, long runs: 404 / 393 / 400 us for the 7 prompts, 645 / 642 / 650
  // for the long one).
  const int heads = kHeadGroup * p.share;
  p.group = heads < a->H ? heads : a->H;
  // Sorting pays once an SM takes more than one block (it evens out the end: the 5 grouped
  // prompts 168 -> 137 us); with fewer it would only delay the first.
  p.sorted = p.blocks <= kMaxSorted && (int64_t)p.blocks * a->H > device_sm_count();
  return a->d_r ? launch_tiles<true>(a, p, stream) : launch_tiles<false>(a, p, stream);
}

}  // namespace mla
