// Verification of drafted tokens (mla_verify_draft): rejection sampling against
// the target's probabilities with random numbers given by the caller.
//
// Sequence b accepts drafts while u q(x) < p(x); the token after them is drawn
// from w = max(p - q, 0) at the first rejected place, or from p behind the last
// draft, by inverting the running sum of w: the smallest j whose sum exceeds
// u * total.  Only one row of p and at most one of q are read, V values each: the
// operator is bound by reading them, or by latency when few sequences are there.
//
// One thread-block cluster per sequence (up to 8 CTAs, so that one sequence draws
// on 8 SMs' load paths; fewer when the batch fills the GPU by itself).  The row is
// cut into segments of 1024 values, a warp each, whose sums all go to the first
// CTA's shared memory; it finds the segment by a scan over the sums and then reads
// that segment alone again (4 KB, in L2 by then).  A segment in which nothing is left is
// read again at once for the target's own sum, which counts where nothing is left at all:
// cut to their 40 likeliest tokens nearly all segments of a row are.  With V near 10^5 values an fp32
// sum would move a boundary by more than many a token's probability: a lane carries
// the rounding errors of its differences and sums along, the sums of segments are
// fp64.  With u = 2^-24 and 32 weights to a lane, those errors are at most 32 u of the
// lane's sum and joining them rounds 32 times: a sum is within 32 u 32 u = 2^-38 of
// itself, and a boundary against the goal within 2^-36 of the total.  Each sum has one
// fixed order, so results repeat.
//
// Measured: 256 sequences, 3 drafts, 128000 fp32 values 46 us = 4.8 TB/s (0.73 of the
// copy rate; sequences whose drafts were all accepted read one row, the others two, and
// the search at the end is not hidden), in bf16 40 to 43 us, cut to 40 tokens 62 to 70 us
// in either; 33 sequences, 100003 bf16 values 8.7 us in a CUDA graph; one
// sequence, 32000 values 5.8 us in a CUDA graph, of which 2 us are the dependent reads of
// draft, probabilities and row and 2.5 us the search.
#include <math.h>

#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSeg = 1024;      // values of a segment
constexpr int kMaxSegs = 1024;  // V <= 2^20

struct VerifyParams {
  const void* p;
  const void* q;
  const int32_t* draft;
  const int32_t* num;
  const float* u_accept;
  const float* u_sample;
  const int32_t* seq_lens;
  int32_t* tokens;
  int32_t* accepted;
  int32_t* new_lens;
  uint32_t* status;
  int64_t p_seq, p_row, q_seq, q_row;
  int s_q, V;
};

MLA_DEVI float ld(const float* x, int64_t i) { return __ldg(x + i); }
MLA_DEVI float ld(const __nv_bfloat16* x, int64_t i) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(x) + i) << 16);
}

template <bool kOn>
struct Is {
  static constexpr bool value = kOn;
};

// What a drafting probability takes from x >= 0, which is no NaN: at most all of it; a NaN
// takes all, a negative value nothing
MLA_DEVI float less_of(float q, float x) { return fmaxf(fminf(q, x), 0.f); }

// What a value adds: only what is positive (a NaN is not)
MLA_DEVI double weight(double w) { return w > 0.0 ? w : 0.0; }

// a + b in fp32 and what its rounding took away (Knuth): together exact
MLA_DEVI float two_sum(float a, float b, float& low) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  low = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}

MLA_DEVI double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
MLA_DEVI double warp_scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Of 32 parts in lane order, the first whose running sum (from `run` on) exceeds the
// goal, else the last that adds anything (rounding may leave the goal unreached);
// `run` becomes the sum before it.  -1: none adds anything.
// `upto`: the running sums, this part's included.
MLA_DEVI int pick_of(double own, double upto, double goal, double& run) {
  const uint32_t over = __ballot_sync(0xffffffffu, own > 0.0 && upto > goal);
  const uint32_t some = __ballot_sync(0xffffffffu, own > 0.0);
  if (!some) return -1;
  const int l = over ? __ffs(over) - 1 : 31 - __clz(some);
  run = __shfl_sync(0xffffffffu, upto - own, l);
  return l;
}
MLA_DEVI int pick(double own, double goal, double& run, int lane) {
  return pick_of(own, run + warp_scan(own, lane), goal, run);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyParams p, int cluster) {
  __shared__ double sums[2][kMaxSegs];  // of what is left of p, and of p where nothing is left
  __shared__ double parts[32];          // of one segment
  __shared__ int first_bad[2];          // first rejected draft; whether an argument is bad
  __shared__ int found[2];              // the segment of the next token (-1: none), the row of sums it came from
  // No early trigger: new_lens may be the lengths that a decode reads before it waits.
  // Before anything else, each block says that it runs (nothing to release by that).
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster > 1 ? sm100::cluster_ctarank() : 0;
  const int b = blockIdx.x / cluster;
  const T* P = static_cast<const T*>(p.p) + b * p.p_seq;
  const T* Q = p.q ? static_cast<const T*>(p.q) + b * p.q_seq : nullptr;
  const int most = p.s_q - 1;
  int n = p.num ? p.num[b] : most;
  const bool bad_n = n < 0 || n > most;
  if (bad_n) n = 0;
  if (threadIdx.x == 0) {
    first_bad[0] = n;
    first_bad[1] = bad_n;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int x = p.draft[(int64_t)b * most + i];
    if (x < 0 || x >= p.V) {
      atomicMax(&first_bad[1], 2);
      continue;
    }
    const double qx = Q ? (double)ld(Q, i * p.q_row + x) : 1.0;
    if (!((double)p.u_accept[(int64_t)b * most + i] * qx < (double)ld(P, i * p.p_row + x))) atomicMin(&first_bad[0], i);
  }
  __syncthreads();
  if (cluster > 1) sm100::cluster_wait();  // the first CTA runs: its shared memory may be written
  const int a = first_bad[0], bad = first_bad[1];
  int next = -1;
  if (!bad) {
    const T* pr = P + a * p.p_row;
    const T* qr = a < n && Q ? Q + a * p.q_row : nullptr;
    const int certain = a < n && !Q ? p.draft[(int64_t)b * most + a] : -1;  // draft of probability one
    const int segs = (p.V + kSeg - 1) / kSeg;
    constexpr int kN = 16;
    for (int g = warp * cluster + rank; g < segs; g += kWarps * cluster) {
      const int j0 = g * kSeg + lane;
      const bool inside = (g + 1) * kSeg <= p.V;
      float acc = 0.f, low = 0.f;
      // kN values of each row, the loads of all of them without a branch between them, so
      // that they are on their way together
      auto add = [&](int j, auto whole, auto two) {
        float pv[kN], qv[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k) pv[k] = ld(pr, decltype(whole)::value ? j + 32 * k : min(j + 32 * k, p.V - 1));
#pragma unroll
        for (int k = 0; k < kN; ++k)
          qv[k] = !decltype(two)::value ? (j + 32 * k == certain ? 1.f : 0.f)
                                        : ld(qr, decltype(whole)::value ? j + 32 * k : min(j + 32 * k, p.V - 1));
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          // p - min(q, p) is zero or positive, and what rounding took from it comes out
          // exactly since p >= q >= 0 (Dekker); then the running sum with its rounding error
          const float x = decltype(whole)::value || j + 32 * k < p.V ? fmaxf(pv[k], 0.f) : 0.f, y = less_of(qv[k], x);
          const float d = __fsub_rn(x, y), e = __fsub_rn(__fsub_rn(x, d), y);
          float f;
          acc = two_sum(acc, d, f);
          low += e + f;
        }
      };
#pragma unroll 1
      for (int j = j0; j < j0 + kSeg; j += 32 * kN) {
        if (inside && qr)
          add(j, Is<true>(), Is<true>());
        else if (inside)
          add(j, Is<true>(), Is<false>());
        else if (qr)
          add(j, Is<false>(), Is<true>());
        else
          add(j, Is<false>(), Is<false>());
      }
      const double sum = warp_sum((double)acc + (double)low);
      // where nothing is left of the target, its own sum, in case nothing is left anywhere
      double whole = 0.0;
      if (sum == 0.0) {
        for (int k = 0; k < kSeg / 32; ++k) whole += weight((double)ld(pr, min(j0 + 32 * k, p.V - 1)) * (j0 + 32 * k < p.V ? 1.0 : 0.0));
        whole = warp_sum(whole);
      }
      if (lane < 2) {
        const uint32_t here = smem_u32(&sums[lane][g]);
        const double v = lane ? whole : sum;
        if (cluster > 1)
          asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(sm100::mapa(here, 0)), "d"(v) : "memory");
        else
          sums[lane][g] = v;
      }
    }
    if (cluster > 1) {
      sm100::cluster_arrive();
      sm100::cluster_wait();
    } else {
      __syncthreads();
    }
    if (rank != 0) return;
    double goal = 0.0, run = 0.0;
    if (warp == 0) {
      // a lane has `per` neighbouring segments
      const int per = (segs + 31) / 32, s0 = min(lane * per, segs), s1 = min(s0 + per, segs);
      auto own_of = [&](int row) {
        double x = 0.0;
        for (int g = s0; g < s1; ++g) x += sums[row][g];
        return x;
      };
      int row = 0, seg = -1;
      double own = own_of(0), upto = warp_scan(own, lane);
      double total = __shfl_sync(0xffffffffu, upto, 31);
      if (total == 0.0 && a < n) {
        row = 1;
        own = own_of(1);
        upto = warp_scan(own, lane);
        total = __shfl_sync(0xffffffffu, upto, 31);
      }
      if (total > 0.0 && total < INFINITY) {
        goal = (double)p.u_sample[b] * total;
        const int l = pick_of(own, upto, goal, run);
        seg = __shfl_sync(0xffffffffu, s0, l);
        const int many = __shfl_sync(0xffffffffu, s1, l) - seg;
        if (per > 1) seg += max(pick(lane < many ? sums[row][seg + lane] : 0.0, goal, run, lane), 0);
      }
      if (lane == 0) {
        found[0] = seg;
        found[1] = row;
      }
    }
    __syncthreads();
    const int seg = found[0], row = found[1];
    // the segment's values again, 128 to a warp, in 32 parts of 32
    auto value = [&](int j) {
      const float x = fmaxf(ld(pr, min(j, p.V - 1)), 0.f);
      const float qv = qr ? ld(qr, min(j, p.V - 1)) : j == certain ? 1.f : 0.f;  // loaded whatever `row` says
      return j < p.V ? (double)x - (row ? 0.0 : (double)less_of(qv, x)) : 0.0;
    };
    if (seg >= 0) {
      double x[kSeg / 32 / kWarps];
#pragma unroll
      for (int k = 0; k < kSeg / 32 / kWarps; ++k) x[k] = value(seg * kSeg + 128 * warp + 32 * k + lane);
#pragma unroll
      for (int k = 0; k < kSeg / 32 / kWarps; ++k) {
        x[k] = warp_sum(x[k]);
        if (lane == 0) parts[warp * (kSeg / 32 / kWarps) + k] = x[k];
      }
    }
    __syncthreads();
    if (warp != 0) return;
    if (seg >= 0) {
      const int part = pick(parts[lane], goal, run, lane);
      const int j = seg * kSeg + 32 * max(part, 0);
      const int at = pick(value(j + lane), goal, run, lane);
      if (part >= 0 && at >= 0) next = j + at;  // a sum above zero has a value above zero: else the rows changed meanwhile
    }
  } else {
    // the first CTA stays until the others, whatever they read, have written their last sum
    if (cluster > 1) {
      sm100::cluster_arrive();
      sm100::cluster_wait();
    }
    if (rank != 0 || warp != 0) return;
  }
  // outputs, by one warp
  const int kept = bad ? 0 : a;
  for (int i = lane; i < p.s_q; i += 32)
    p.tokens[(int64_t)b * p.s_q + i] = i < kept ? p.draft[(int64_t)b * most + i] : i == kept ? next : -1;
  if (lane == 0) {
    if (bad) set_status(p.status, bad == 2 ? MLA_ERR_BAD_TOKEN : MLA_ERR_BAD_SEQ_LEN);
    p.accepted[b] = kept;
    if (p.new_lens) p.new_lens[b] = bad ? p.seq_lens[b] : p.seq_lens[b] - (n - a);
  }
}

}  // namespace

cudaError_t launch_verify(const mla_verify_args_t* a, cudaStream_t stream) {
  VerifyParams p;
  p.p = a->target_probs;
  p.q = a->draft_probs;
  p.draft = a->draft_tokens;
  p.num = a->num_draft;
  p.u_accept = a->u_accept;
  p.u_sample = a->u_sample;
  p.seq_lens = a->seq_lens;
  p.tokens = a->tokens;
  p.accepted = a->num_accepted;
  p.new_lens = a->new_lens;
  p.status = static_cast<uint32_t*>(a->workspace);
  p.p_seq = a->target_seq;
  p.p_row = a->target_row;
  p.q_seq = a->draft_seq;
  p.q_row = a->draft_row;
  p.s_q = a->s_q;
  p.V = a->V;
  // a segment per warp, up to 8 CTAs, but no more than about eight CTAs an SM in all (four
  // are resident; 256 sequences of 128000 values in clusters of 2 / 4 / 8: 49 / 48 / 60 us)
  const int segs = (a->V + kSeg - 1) / kSeg;
  int cluster = 1;
  while (cluster < 8 && cluster * kWarps < segs && 2ll * cluster * a->B <= 8ll * device_sm_count()) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a->B * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (a->dtype == MLA_PROB_BF16) return cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, p, cluster);
  return cudaLaunchKernelEx(&cfg, verify_kernel<float>, p, cluster);
}

}  // namespace mla
