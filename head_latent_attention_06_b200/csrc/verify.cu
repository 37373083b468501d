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
// on 8 SMs' load paths).  The row is cut into segments of 1024 values, one warp
// each, whose sums all go to the first CTA's shared memory; it finds the segment
// with a scan over the sums and rescans that segment alone (4 KB, in L2 by then).
// Sums are fp64: with V near 10^5 values an fp32 sum would move a boundary by
// more than many a token's probability.  The differences p - q are exact in fp64
// but for a last bit.  Each sum has one fixed order, so results repeat.
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

// What a value adds: only what is positive (a NaN is not)
MLA_DEVI double weight(double w) { return w > 0.0 ? w : 0.0; }

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

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p, int cluster) {
  __shared__ double sums[2][kMaxSegs];  // of the weights, and of p alone
  __shared__ int first_bad[2];          // first rejected draft; whether an argument is bad
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
  const int a = first_bad[0], bad = first_bad[1];
  int next = -1;
  if (!bad) {
    // every CTA of the cluster is here: they read the same arguments
    const T* pr = P + a * p.p_row;
    const T* qr = a < n && Q ? Q + a * p.q_row : nullptr;
    const int certain = a < n && !Q ? p.draft[(int64_t)b * most + a] : -1;  // draft of probability one
    const int segs = (p.V + kSeg - 1) / kSeg;
    // a value's two weights: what is left of p, and p
    auto at = [&](int j, double& left, double& whole) {
      const double pv = (double)ld(pr, j);
      whole = weight(pv);
      left = qr ? weight(pv - (double)ld(qr, j)) : j == certain ? weight(pv - 1.0) : whole;
    };
    for (int g = warp * cluster + rank; g < segs; g += kWarps * cluster) {
      double sl = 0.0, sw = 0.0;
#pragma unroll 8
      for (int k = 0; k < kSeg / 32; ++k) {
        const int j = g * kSeg + 32 * k + lane;
        if (j < p.V) {
          double left, whole;
          at(j, left, whole);
          sl += left;
          sw += whole;
        }
      }
      sl = warp_sum(sl);
      sw = warp_sum(sw);
      if (lane < 2) {
        const uint32_t here = smem_u32(&sums[lane][g]);
        const double v = lane ? sw : sl;
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
    if (rank != 0 || warp != 0) return;
    // the total is the last running sum, so that u * total stays below it
    int row = 0;
    double total = 0.0;
    auto total_of = [&](int r) {
      double run = 0.0;
      for (int g0 = 0; g0 < segs; g0 += 32) {
        const double x = warp_scan(g0 + lane < segs ? sums[r][g0 + lane] : 0.0, lane);
        run += __shfl_sync(0xffffffffu, x, 31);
      }
      return run;
    };
    total = total_of(0);
    if (!(total > 0.0) && a < n) total = total_of(row = 1);
    if (total > 0.0 && total < INFINITY) {
      const double goal = (double)p.u_sample[b] * total;
      // the first segment whose running sum exceeds the goal (else the last that adds anything)
      double run = 0.0, base = 0.0;
      int seg = -1, last = -1;
      double last_base = 0.0;
      for (int g0 = 0; g0 < segs && seg < 0; g0 += 32) {
        const double own = g0 + lane < segs ? sums[row][g0 + lane] : 0.0;
        const double x = run + warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, own > 0.0 && x > goal);
        const uint32_t some = __ballot_sync(0xffffffffu, own > 0.0);
        if (over) {
          const int l = __ffs(over) - 1;
          seg = g0 + l;
          base = __shfl_sync(0xffffffffu, x - own, l);
        } else if (some) {
          const int l = 31 - __clz(some);
          last = g0 + l;
          last_base = __shfl_sync(0xffffffffu, x - own, l);
        }
        run = __shfl_sync(0xffffffffu, x, 31);
      }
      if (seg < 0) {
        seg = last;
        base = last_base;
      }
      run = base;
      for (int k = 0; k < kSeg / 32; ++k) {
        const int j = seg * kSeg + 32 * k + lane;
        double left = 0.0, whole = 0.0;
        if (j < p.V) at(j, left, whole);
        const double own = row ? whole : left;
        const double x = run + warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, own > 0.0 && x > goal);
        const uint32_t some = __ballot_sync(0xffffffffu, own > 0.0);
        if (over) {
          next = seg * kSeg + 32 * k + __ffs(over) - 1;
          break;
        }
        if (some) next = seg * kSeg + 32 * k + 31 - __clz(some);  // stands if rounding leaves the goal unreached
        run = __shfl_sync(0xffffffffu, x, 31);
      }
    }
  } else if (rank != 0 || warp != 0) {
    return;
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
  // one segment per warp, up to 8 CTAs
  const int segs = (a->V + kSeg - 1) / kSeg;
  int cluster = 1;
  while (cluster < 8 && cluster * kWarps < segs) cluster *= 2;
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
