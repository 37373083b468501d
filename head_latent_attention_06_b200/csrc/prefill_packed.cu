// Attention over packed prompts of different lengths in the explicit form
// (mla_prefill_packed).
#include <math_constants.h>

#include "packed.cuh"

namespace mla {
namespace {

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
  int n_tok, B, H, share, causal;
  float scale_log2;
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

template <bool PE>
__global__ void __launch_bounds__(128) packed_rows_kernel(const PackedParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) packed_check(p.cu, p.B, p.n_tok, p.status, threadIdx.x, 128);
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(w / p.H), h = (int)(w % p.H);
  if (t >= p.n_tok) return;
  const PackedSeq s = packed_find(p.cu, p.B, p.n_tok, t, lane);
  if (s.b < 0) return;
  attend_row<PE>(p, t, h, s.lo, p.causal ? t + 1 : s.hi, lane);
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
  const dim3 grid((unsigned)(((int64_t)a->n_tok * a->H + 3) / 4));
  return a->d_r ? launch_pdl(packed_rows_kernel<true>, grid, dim3(128), 0, stream, p)
                : launch_pdl(packed_rows_kernel<false>, grid, dim3(128), 0, stream, p);
}

}  // namespace mla
