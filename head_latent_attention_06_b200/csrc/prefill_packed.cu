// Attention over packed prompts of different lengths in the explicit form
// (mla_prefill_packed).
#include <math_constants.h>

#include "packed.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace mla {
uint64_t device_wait_limit_ns();

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
  int n_tok, B, H, share, causal, blocks;
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
// every 32 and owns four values of the output.
template <bool PE>
MLA_DEVI void attend_row(const PackedParams& p, int t, int h, int lo, int hi, int lane) {
  const int g = h / p.share;
  const uint4* qn = reinterpret_cast<const uint4*>(p.q_nope + (int64_t)t * p.qn_tok + (int64_t)h * p.qn_head);
  const uint4* qp = reinterpret_cast<const uint4*>(p.q_pe + (int64_t)t * p.qp_tok + (int64_t)h * p.qp_head);
  float m = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = lo; j0 < hi; j0 += 32) {
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
constexpr int kThreads = 384;               // warp 0 loads, warps 1 and 2 MMA, warps 4..7 tile A, 8..11 tile B
constexpr int kRows = 256;                  // packed rows of a CTA: tile A the first 128, B the others
constexpr uint32_t kChunk = 128 * 128;      // 16 KB: 128 rows x 64 values, or 64 keys x 128 values
constexpr int kHeadGroup = 8;               // heads whose blocks run side by side

template <bool PE>
struct Cfg {
  static constexpr int kQk = PE ? 3 : 2;              // 64-value chunks of a query or key
  static constexpr int kSlots = PE ? 8 : 10;          // ring of K and V chunks
  static constexpr int kPer = kQk + 2;                // chunks of one key tile: K, then V in halves of 64 keys
  // K(j) may go in once the item kWaitK before it has been read, V(j) once the item
  // kWaitV before it has: with 8 slots of which a key tile takes 3 + 2, K(j) ends at 5 j + 3
  // and needs V(j - 2), which ends at 5 j - 5, gone; V(j) ends at 5 j + 5 and needs
  // K(j - 1), which ends at 5 j - 2, gone.  With 10 slots of 2 + 2, K(j) needs 4 j - 8
  // (V(j - 3)) and V(j) 4 j - 6 (K(j - 2)).
  static constexpr int kWaitK = PE ? 3 : 5, kWaitV = PE ? 3 : 5;
  static constexpr uint32_t kRing = 2 * kQk * kChunk;
  static constexpr uint32_t kBars = kRing + kSlots * kChunk;
  static constexpr uint32_t kSmem = kBars + 512 + 1024;
};
static_assert(Cfg<true>::kSmem <= 232448 && Cfg<false>::kSmem <= 232448, "shared memory budget");

// TMEM: scores (and the weights over them) of tile t at columns 128 t, outputs at 256 + 128 t
constexpr uint32_t kTmemO = 256;
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);
constexpr float kRescale = 256.f;             // a tile's weights beyond this ask for a new reference
constexpr float kBeyond = 1.152921504606847e18f;  // 2^60: no range is left to wait for it
constexpr int kPolyPairs = 0x00;              // of eight pairs of exponentials, those on the FMA pipe
// barriers; [2] per tile, P[2 t + half]
constexpr int B_Q = 0, B_S = 1, B_P = 3, B_O = 7, B_DRAIN = 9, B_FULL = 11, B_EMPTY = 19, B_TURN = 27, B_COUNT = 29;

struct Tiles {
  int k0;         // first key of the block's first key tile
  int n;          // key tiles
  int from[2], to[2];  // those of them that query tile A and B see
};

// 2^x by a polynomial on the FMA pipe: x = n + f, |f| <= 1/2, 2^f by the degree-4
// minimax polynomial of relative error 2.6e-6 (its coefficients come out of a Remez
// exchange), the exponent n added to the bits.  For finite x >= -126.
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
MLA_DEVI void exp2_poly2(uint64_t x, float& p0, float& p1) {
  float x0, x1;
  unpack2(x, x0, x1);
  x = pack2(fmaxf(x0, -126.f), fmaxf(x1, -126.f));
  const float kMagic = 12582912.f;  // 1.5 * 2^23: adding it leaves round(x) in the low mantissa bits
  const uint64_t t = add2(x, pack2(kMagic, kMagic));
  const uint64_t f = fma2(add2(t, pack2(-kMagic, -kMagic)), pack2(-1.f, -1.f), x);
  uint64_t r = pack2(0.009570102207362652f, 0.009570102207362652f);
  r = fma2(r, f, pack2(0.05591785907745361f, 0.05591785907745361f));
  r = fma2(r, f, pack2(0.240247443318367f, 0.240247443318367f));
  r = fma2(r, f, pack2(0.6931217908859253f, 0.6931217908859253f));
  r = fma2(r, f, pack2(0.9999992847442627f, 0.9999992847442627f));
  unpack2(r, p0, p1);
  float t0, t1;
  unpack2(t, t0, t1);
  p0 = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
  p1 = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
}
template <bool kOn>
struct Poly {
  static constexpr bool value = kOn;
};
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
  // warp-uniform, and known to be: what the MMA warp computes stays in uniform registers
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sa + C::kBars + 8u * i; };
  auto full = [&](int item) -> uint32_t { return bar(B_FULL + (item & 7)); };
  auto empty = [&](int item) -> uint32_t { return bar(B_EMPTY + (item & 7)); };
  auto slot = [&](int s) -> uint32_t { return sa + C::kRing + (s % C::kSlots) * kChunk; };
  int* words = reinterpret_cast<int*>(sm + C::kBars + 8 * B_COUNT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort_flag = words + 1;
  int* issued = words + 2;
  int* low = words + 4;    // [8] per softmax warp: the first key its rows see
  int* high = words + 12;  // [8] one past the last

  // blocks of a group of heads in turn, the last rows (the longest, when causal) first
  const int per_group = kHeadGroup * p.blocks;
  const int grp = blockIdx.x / per_group, in = blockIdx.x - grp * per_group;
  const int gh = min(kHeadGroup, p.H - grp * kHeadGroup);
  const int blk = p.blocks - 1 - in / gh, h = grp * kHeadGroup + in % gh;
  const int g = h / p.share;
  const int q0 = blk * kRows;
  const uint64_t wait_ns = p.wait_ns;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    *issued = 0;
    mbar_init(bar(B_Q), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(B_S + t), 1);
      mbar_init(bar(B_P + 2 * t), 4);
      mbar_init(bar(B_P + 2 * t + 1), 4);
      mbar_init(bar(B_O + t), 1);
      mbar_init(bar(B_DRAIN + t), 1);
      mbar_init(bar(B_TURN + t), 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 2);  // both query tiles have read it
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_1(smem_u32(tmem_slot), 512);
    tmem_relinquish_1();
  }
  pdl_trigger();
  pdl_wait();
  // ---- the keys of every row: of its own prompt, up to itself when causal
  const int t = (warp - 4) >> 2;                          // query tile of a softmax warp
  const int row = 32 * (warp & 3) + lane;                 // its TMEM lane
  const int qi = q0 + 128 * t + row;
  int lo = 0, hi = 0;
  if (warp >= 4) {
    const int first = q0 + 128 * t + 32 * (warp & 3);
    if (first < p.n_tok) {
      const PackedRow r = packed_row(p.cu, p.B, p.n_tok, first, lane);
      lo = r.lo;
      hi = r.hi;
      if (p.causal && hi > lo) hi = qi + 1;
    }
    const int a = __reduce_min_sync(0xffffffffu, hi > lo ? lo : 0x7fffffff);
    const int z = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      low[warp - 4] = a;
      high[warp - 4] = z;
    }
  } else if (blockIdx.x == 0 && warp >= 2) {
    packed_check(p.cu, p.B, p.n_tok, p.status, threadIdx.x - 64, 64);
  } else if (warp == 0 && lane == 0) {
    // both tiles' queries (rows past the end read as zeros)
    mbar_arrive_expect_tx_local(bar(B_Q), 2 * C::kQk * kChunk);
    for (int i = 0; i < 2; ++i) {
      const uint32_t dst = sa + i * C::kQk * kChunk;
      tma_load_3d_cta(dst, &tm_qn, bar(B_Q), 0, h, q0 + 128 * i);
      tma_load_3d_cta(dst + kChunk, &tm_qn, bar(B_Q), 64, h, q0 + 128 * i);
      if constexpr (PE) tma_load_3d_cta(dst + 2 * kChunk, &tm_qp, bar(B_Q), 0, h, q0 + 128 * i);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Tiles T;
  {
    int a[2], z[2];
    for (int i = 0; i < 2; ++i) {
      a[i] = min(min(low[4 * i], low[4 * i + 1]), min(low[4 * i + 2], low[4 * i + 3]));
      z[i] = max(max(high[4 * i], high[4 * i + 1]), max(high[4 * i + 2], high[4 * i + 3]));
    }
    T.k0 = min(a[0], a[1]);
    T.n = 0;
    for (int i = 0; i < 2; ++i) {
      const bool any = z[i] > a[i];
      T.from[i] = any ? (a[i] - T.k0) / 128 : 0;
      T.to[i] = any ? (z[i] - T.k0 + 127) / 128 : 0;
      T.n = max(T.n, T.to[i]);
    }
  }

  // 384 threads launched with 168 registers: 128 x 80 + 256 x 208 is within that
  if (warp < 4) {
    regs_dec<80>();
    if (warp == 0) {
    // =========================== loads ===========================
    // Items in the ring, each with a full and an empty barrier of eight taken in turn:
    // K(j) is item 2 j (kQk slots from kPer j on), V(j) item 2 j + 1 (two slots after
    // it).  An item goes into slots whose last holders have been read: see Cfg::kWaitK.
    int count = 0;
    bool ok = true;
    for (int j = 0; ok && j < T.n; ++j) {
      const int key = T.k0 + 128 * j;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int item = 2 * j + v, last = item - (v ? C::kWaitV : C::kWaitK);
        if (last >= 0) ok = ok && mbar_wait_converged(empty(last), (last >> 3) & 1, abort_flag, p.status, wait_ns);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t f = full(item);
          const int s = C::kPer * j + (v ? C::kQk : 0);
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
        }
        __syncwarp();
        count = item + 1;
      }
    }
    if (lane == 0) *issued = count;
  } else if (warp < 3) {
    // =========================== MMA issue ===========================
    // One warp per query tile: P.V, then the next scores, while the other tile's
    // softmax runs under them.  (One warp for both issued 40 MMAs, six waits and four
    // commits per key tile, 3500 cycles of it, more than the 2560 that the tensor pipe
    // needs.)  The pipe takes a warp's products in order, so scores may follow the P.V
    // that reads the weights they overwrite without a wait between the two.
    const int i = warp - 1;
    if (T.n > 0) {
      bool ok = mbar_wait_converged(bar(B_Q), 0, abort_flag, p.status, wait_ns);
      auto wait = [&](int b, int parity) { return mbar_wait_converged(bar(b), parity & 1, abort_flag, p.status, wait_ns); };
      auto arrived = [&](int item) { return wait(B_FULL + (item & 7), item >> 3); };
      auto sees = [&](int j) { return j >= T.from[i] && j < T.to[i]; };
      // scores over K(j)
      auto scores = [&](int j) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::kQk; ++c)
          mma_1_x4_elect<2, 2>(tmem + 128u * i, desc_sw128(sa + (i * C::kQk + c) * kChunk, 16, 1024),
                               desc_sw128(slot(C::kPer * j + c), 16, 1024), kIdescS, c != 0);
        commit_1_elect(bar(B_S + i));
      };
      // the weights of half a key tile times V(j): 16 keys a step, weights in 8 columns, V
      // rows 2 KB further on
      auto values = [&](int j, int half) {
        tc_fence_after();
        mma_1_ts_x4_elect<8, 128>(tmem + kTmemO + 128u * i, tmem + 128u * i + 32u * half,
                                  desc_sw128(slot(C::kPer * j + C::kQk + half), kChunk / 2, 1024), kIdescPV,
                                  (j > T.from[i] || half) ? 1u : 0u);
      };
      ok = ok && arrived(0);
      if (ok) {
        if (sees(0)) scores(0);
        commit_1_elect(empty(0));
      }
      for (int j = 0; ok && j < T.n; ++j) {
        const bool mine = sees(j), more = j + 1 < T.n;
        ok = arrived(2 * j + 1);
        if (mine) ok = ok && wait(B_P + 2 * i, j - T.from[i]);
        // in turn: A's products of key tile j, then B's, then A's of the next
        if (i + j > 0) ok = ok && wait(B_TURN + i, i ? j : j - 1);
        if (!ok) break;
        if (mine) values(j, 0);
        if (more) ok = arrived(2 * j + 2);
        if (mine) ok = ok && wait(B_P + 2 * i + 1, j - T.from[i]);
        if (!ok) break;
        if (mine) values(j, 1);
        if (mine && j + 1 == T.to[i]) commit_1_elect(bar(B_O + i));
        commit_1_elect(empty(2 * j + 1));
        if (sees(j + 1)) scores(j + 1);
        __syncwarp();
        if (lane == 0) mbar_arrive_local(bar(B_TURN + 1 - i));
        __syncwarp();
        if (more) commit_1_elect(empty(2 * j + 2));
      }
      commit_1_elect(bar(B_DRAIN + i));
      int keep = 0;
      mbar_wait_converged(bar(B_DRAIN + i), 0, &keep, p.status, kDrainNs);
    }
  }
  } else {
    regs_inc<208>();
    // ================ softmax: a thread per query row ================
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t cs = 128u * t, co = kTmemO + 128u * t;
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    float m_used = -CUDART_INF_F, l = 0.f;
    bool stale = true;  // the reference m_used has to be found (again)
    for (int j = T.from[t]; j < T.to[t]; ++j) {
      if (!mbar_wait_converged(bar(B_S + t), (j - T.from[t]) & 1, abort_flag, p.status, wait_ns)) break;
      tc_fence_after();
      uint32_t sr[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tl + cs + 32u * c, sr[c]);
      tmem_wait_ld();
      const int kb = T.k0 + 128 * j;
      const bool masked = __any_sync(0xffffffffu, lo > kb || hi < kb + 128);
      if (masked) {
        const uint32_t a = (uint32_t)max(lo - kb, 0), n = (uint32_t)max(min(hi - kb, 128) - (int)a, 0);
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if ((uint32_t)k - a >= n) sr[k >> 5][k & 31] = 0xff800000u;
      }
      auto score = [&](int k) { return __uint_as_float(sr[k >> 5][k & 31]); };
      // The weights are 2^(s scale - m) for a reference m near the row's maximum so far,
      // not the maximum itself: any m gives the same quotient, as long as the weights
      // and their sums stay within fp32 and bf16's common range.  So m is found where
      // there is none and raised one tile after a weight went beyond 2^8; the hot loop
      // takes no maximum.
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
        // the old tiles' largest weight counts as well: l is a bound of it
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
        if (__any_sync(0xffffffffu, resc)) {
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
      float top = 0.f;  // the largest exponent that the polynomial was given
      // the weights of 64 keys, in bf16 pairs over the scores and to the MMA warp; with
      // `poly` a part of the exponentials goes to the FMA pipe
      auto weights = [&](int half, auto poly) {
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int u = 64 * half + 2 * k;
          const uint64_t x = fma2(pack2(score(u), score(u + 1)), scale2, ref2);
          float p0, p1;
          if (decltype(poly)::value && ((kPolyPairs >> (k & 7)) & 1)) {
            unpack2(x, p0, p1);
            top = max3(top, p0, p1);
            exp2_poly2(x, p0, p1);
          } else {
            unpack2(x, p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
          }
          sum[k & 1] = add2(sum[k & 1], pack2(p0, p1));
          pk[k] = pack_bf16(p0, p1);
        }
        tmem_st32(tl + cs + 32u * half, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(bar(B_P + 2 * t + half));
      };
      if (masked || __any_sync(0xffffffffu, stale)) {
        // exact zeros for what is not seen
        weights(0, Poly<false>());
        weights(1, Poly<false>());
      } else {
        weights(0, Poly<true>());
        weights(1, Poly<true>());
      }
      float s0, s1;
      unpack2(add2(sum[0], sum[1]), s0, s1);
      const float tile = s0 + s1;
      l += tile;
      stale = stale || tile > kRescale;
      // beyond 2^60 (a NaN included) within one tile: the row is done over as well
      if (!(tile < kBeyond && top < 60.f)) l = CUDART_NAN_F;
    }
    // ---- o = O / l, lse
    const bool any = T.to[t] > T.from[t];
    if (any) {
      mbar_wait_converged(bar(B_O + t), 0, abort_flag, p.status, wait_ns);
      tc_fence_after();
    }
    const bool live = any && __shfl_sync(0xffffffffu, *abort_flag, 0) == 0;
    const bool mine = hi > lo;
    const float inv = l == 0.f || !live ? 0.f : 1.f / l;
    const int64_t orow = (int64_t)qi * p.H + h;
    bool odd = live && mine && !(fabsf(l) < CUDART_INF_F);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t o[32];
      if (live) {
        tmem_ld32(tl + co + 32u * c, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
      }
      float bad = 0.f;  // a NaN once any value is infinite or not a number
#pragma unroll
      for (int k = 0; k < 32; ++k) bad = fmaf(__uint_as_float(o[k]), 0.f, bad);
      odd = odd || (live && mine && bad != 0.f);
      if (mine) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + orow * kDv + 32 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[k] = make_uint4(pack_bf16(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                              pack_bf16(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                              pack_bf16(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                              pack_bf16(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
      }
    }
    if (mine && p.lse) p.lse[orow] = inv == 0.f ? -CUDART_INF_F : (m_used + log2f(l)) * 0.6931471805599453f;
    // An infinite or NaN value that a row does not see has met its zero weight in the
    // product with V (0 x inf): such rows, and those that see one, are done over from
    // the definition.
    __syncwarp();
    for (uint32_t again = __ballot_sync(0xffffffffu, odd); again; again &= again - 1) {
      const int r = __ffs(again) - 1;
      attend_row<PE>(p, __shfl_sync(0xffffffffu, qi, r), h, __shfl_sync(0xffffffffu, lo, r), __shfl_sync(0xffffffffu, hi, r),
                     lane);
    }
    tc_fence_before();
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    // no load may outlive the block: the queries of a block without keys, and after a
    // wait that ran out the last round of the ring (all waits bounded)
    int give_up = 0;
    mbar_wait(bar(B_Q), 0, &give_up, nullptr, kDrainNs);
    for (int i = *abort_flag ? max(0, *issued - 8) : *issued; i < *issued; ++i)
      mbar_wait(full(i), (i >> 3) & 1, &give_up, nullptr, kDrainNs);
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
  return a->d_r ? launch_tiles<true>(a, p, stream) : launch_tiles<false>(a, p, stream);
}

}  // namespace mla
