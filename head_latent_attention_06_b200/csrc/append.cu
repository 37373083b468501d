// Appending packed tokens to the paged latent cache with the position rotation
// on the way (mla_append_kv).
//
// A token's cache row is its latent (512 values) and its RoPE key (64 values)
// after the rotation; the same rotation goes over the RoPE part of its query, H
// heads of 64 values.  Pair i of a vector turns by pos * base^(-2i/64): the same
// 32 angles for the key and for every head.
//
// Nothing is computed twice per byte: a token reads 1152 + 128 H bytes, writes
// its row and 128 + 128 H bytes, and does 3 operations a rotated value, so it is
// bound by memory.  A warp's 32 lanes hold the token's 32 angles, one sincos
// each, and hand them round by shuffles: a lane works on 16-byte pieces (four
// pairs) whose place in the vector is the same for all of its pieces, so the
// eight shuffles are done once a warp.  The angle is a fraction of a turn in fp64
// (positions beyond 10^5 turn thousands of times), its sine and cosine fp32.
//
// A warp has up to 32 heads (8 pieces of 16 bytes a lane, four in flight at a time);
// more heads take two or four warps a token, each with its own sincos, which are free
// beside the loads.  Measured: 16351 tokens, 128 heads, e4m3 cache 101 us = 5.6 TB/s, 0.85
// of the copy rate (bf16 92 us, q8_0 109, q4_0 108: more divisions a value); one step of 64 tokens, 128 heads, bf16 cache 2.8 us in a CUDA graph
// (0.34 us of bytes: launch and three dependent reads - offsets, length, page).  Without
// queries a token's own instructions bound it (65536 tokens, e4m3: 51 us); products with
// a reciprocal and a check for ties in place of its 18 divisions a lane: 56 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "packed.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kPieces = kDr / 8;  // 16-byte pieces of a RoPE vector

struct AppendParams {
  const __nv_bfloat16* c;
  const __nv_bfloat16* k_pe;
  const __nv_bfloat16* q_pe;
  __nv_bfloat16* k_out;
  __nv_bfloat16* q_out;
  uint8_t* kv;
  void* kv_scale;
  const int32_t* block_table;
  const int32_t* cu;
  const int32_t* seq_lens;
  uint32_t* status;
  int64_t c_tok, k_tok, q_tok, q_head, ko_tok, qo_tok, qo_head;
  int n_tok, B, H, max_pages, num_pages, warps_per_token;
  double turn;     // turns of pair 0 per position: 1 / 2 pi
  double fall[5];  // base^(-2^k / 32): the frequency of pair i is the product over the bits of i
};

MLA_DEVI void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
MLA_DEVI uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
MLA_DEVI void rotate8(float (&x)[8], const float (&cs)[4], const float (&sn)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = x[2 * k], b = x[2 * k + 1];
    x[2 * k] = a * cs[k] - b * sn[k];
    x[2 * k + 1] = a * sn[k] + b * cs[k];
  }
}

// One 8-value piece of the row into the cache; KIND as in the cache write: 0 bf16,
// 1 e4m3 (row scale `rs`), 2 q8_0, 3 q4_0.  Blocks of 32 values are four
// neighbouring lanes' pieces; `mask` names the lanes that store a piece.
template <int KIND>
MLA_DEVI void store_piece(const AppendParams& p, size_t slot, int piece, const float (&x)[8], float rs, uint32_t mask,
                          int lane) {
  if constexpr (KIND == 0) {
    *reinterpret_cast<uint4*>(p.kv + (slot * kRow + 8 * piece) * 2) = pack8(x);
  } else if constexpr (KIND == 1) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 q = make_float2(__fdiv_rn(x[2 * k], rs), __fdiv_rn(x[2 * k + 1], rs));
      q.x = fminf(fmaxf(q.x, -448.f), 448.f);
      q.y = fminf(fmaxf(q.y, -448.f), 448.f);
      w[k >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (16 * (k & 1));
    }
    *reinterpret_cast<uint2*>(p.kv + slot * kRow + 8 * piece) = make_uint2(w[0], w[1]);
  } else {
    constexpr float levels = KIND == 2 ? 127.f : 7.f;
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]));
    amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 2));
    const __half d = __float2half_rn(__fdiv_rn(amax, levels));
    const float df = __half2float(d);
    int code[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      code[k] = df > 0.f ? (int)fminf(fmaxf(rintf(__fdiv_rn(x[k], df)), -levels), levels) : 0;
    if constexpr (KIND == 2) {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k >> 2] |= (uint32_t)(uint8_t)code[k] << (8 * (k & 3));
      *reinterpret_cast<uint2*>(p.kv + slot * kRow + 8 * piece) = make_uint2(w[0], w[1]);
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) w |= (uint32_t)(code[k] + 8) << (4 * k);
      *reinterpret_cast<uint32_t*>(p.kv + slot * (kRow / 2) + 4 * piece) = w;
    }
    if ((lane & 3) == 0) static_cast<__half*>(p.kv_scale)[slot * (kRow / 32) + (piece >> 2)] = d;
  }
}

template <int KIND>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendParams p) {
  // No early trigger: the decode reads cache rows before it waits for its
  // predecessor, so kernels after this one may start only once it has completed.
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0) packed_check(p.cu, p.B, p.n_tok, p.status, threadIdx.x, 32 * kWarps);
  const int t = blockIdx.x * (kWarps / p.warps_per_token) + warp / p.warps_per_token;
  const int sub = warp % p.warps_per_token;
  if (t >= p.n_tok) return;

  // the row's pieces are on their way while the position is found
  uint4 cv[2], kv = make_uint4(0, 0, 0, 0);
  if (sub == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(p.c + (size_t)t * p.c_tok);
    cv[0] = src[lane];
    cv[1] = src[lane + 32];
    if (lane < kPieces) kv = reinterpret_cast<const uint4*>(p.k_pe + (size_t)t * p.k_tok)[lane];
  }
  const PackedSeq s = packed_find(p.cu, p.B, p.n_tok, t, lane);
  if (s.b < 0) return;
  const int L = p.seq_lens[s.b], n = s.hi - s.lo;
  if (L < n || L > p.max_pages * kPage) {
    if (lane == 0) set_status(p.status, MLA_ERR_BAD_SEQ_LEN);
    return;
  }
  const int pos = L - n + t - s.lo;
  const int page = p.block_table[(size_t)s.b * p.max_pages + pos / kPage];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) set_status(p.status, MLA_ERR_BAD_BLOCK_TABLE);
    return;
  }
  const size_t slot = (size_t)page * kPage + pos % kPage;

  // pair `lane`: turns = pos * f / 2 pi, its whole part dropped
  double f = p.turn;
#pragma unroll
  for (int k = 0; k < 5; ++k)
    if ((lane >> k) & 1) f *= p.fall[k];
  const double turns = (double)pos * f;
  float sn1, cs1, cs[4], sn[4];
  sincospif(2.f * (float)(turns - rint(turns)), &sn1, &cs1);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    cs[k] = __shfl_sync(0xffffffffu, cs1, 4 * (lane & 7) + k);
    sn[k] = __shfl_sync(0xffffffffu, sn1, 4 * (lane & 7) + k);
  }

  if (sub == 0) {
    float x[2][8], k[8];
    unpack8(cv[0], x[0]);
    unpack8(cv[1], x[1]);
    unpack8(kv, k);
    rotate8(k, cs, sn);
    float rs = 0.f;
    if constexpr (KIND == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rs = fmaxf(rs, fmaxf(fabsf(k[i]), fmaxf(fabsf(x[0][i]), fabsf(x[1][i]))));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rs = fmaxf(rs, __shfl_xor_sync(0xffffffffu, rs, o));
      rs = rs > 0.f ? __fdiv_rn(rs, 448.f) : 1.f;
      if (lane == 0) static_cast<float*>(p.kv_scale)[slot] = rs;
    }
    store_piece<KIND>(p, slot, lane, x[0], rs, 0xffffffffu, lane);
    store_piece<KIND>(p, slot, lane + 32, x[1], rs, 0xffffffffu, lane);
    if (lane < kPieces) {
      store_piece<KIND>(p, slot, kDc / 8 + lane, k, rs, (1u << kPieces) - 1, lane);
      if (p.k_out) reinterpret_cast<uint4*>(p.k_out + (size_t)t * p.ko_tok)[lane] = pack8(k);
    }
  }

  // query heads: piece i is piece i % 8 of head i / 8
  const int total = p.H * kPieces, stride = 32 * p.warps_per_token;
  const __nv_bfloat16* qs = p.q_pe + (size_t)t * p.q_tok;
  __nv_bfloat16* qd = p.q_out + (size_t)t * p.qo_tok;
  constexpr int kIn = 4;
  for (int i0 = sub * 32 + lane; i0 < total; i0 += kIn * stride) {
    uint4 v[kIn];
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      const int i = i0 + u * stride;
      if (i < total) v[u] = *reinterpret_cast<const uint4*>(qs + (i >> 3) * p.q_head + 8 * (i & 7));
    }
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      const int i = i0 + u * stride;
      if (i < total) {
        float x[8];
        unpack8(v[u], x);
        rotate8(x, cs, sn);
        *reinterpret_cast<uint4*>(qd + (i >> 3) * p.qo_head + 8 * (i & 7)) = pack8(x);
      }
    }
  }
}

}  // namespace

cudaError_t launch_append(const mla_append_args_t* a, cudaStream_t stream) {
  AppendParams p;
  p.c = static_cast<const __nv_bfloat16*>(a->c);
  p.k_pe = static_cast<const __nv_bfloat16*>(a->k_pe);
  p.q_pe = static_cast<const __nv_bfloat16*>(a->q_pe);
  p.k_out = static_cast<__nv_bfloat16*>(a->k_pe_out);
  p.q_out = static_cast<__nv_bfloat16*>(a->q_pe_out);
  p.kv = static_cast<uint8_t*>(a->kv_cache);
  p.kv_scale = a->kv_scale;
  p.block_table = a->block_table;
  p.cu = a->cu_seqlens;
  p.seq_lens = a->seq_lens;
  p.status = static_cast<uint32_t*>(a->workspace);
  p.c_tok = a->c_tok;
  p.k_tok = a->k_pe_tok;
  p.q_tok = a->q_pe_tok;
  p.q_head = a->q_pe_head;
  p.ko_tok = a->k_pe_out_tok;
  p.qo_tok = a->q_pe_out_tok;
  p.qo_head = a->q_pe_out_head;
  p.n_tok = a->n_tok;
  p.B = a->B;
  p.H = a->H;
  p.max_pages = a->max_pages_per_seq;
  p.num_pages = a->num_pages;
  // A warp per 32 heads, so that a lane has about 8 pieces; twice as many while that leaves
  // the GPU with at most two CTAs an SM (64 tokens, 128 heads: 2.8 us against 3.5; 16351
  // tokens in an e4m3 cache 121 us against 98).
  p.warps_per_token = a->H > 64 ? 4 : a->H > 32 ? 2 : 1;
  while (p.warps_per_token < kWarps && 8 * p.warps_per_token <= a->H &&
         (int64_t)a->n_tok * 2 * p.warps_per_token <= (int64_t)kWarps * 2 * device_sm_count())
    p.warps_per_token *= 2;
  p.turn = 0.15915494309189533577;
  for (int k = 0; k < 5; ++k) p.fall[k] = exp2(-(double)(1 << k) / (kDr / 2) * log2((double)a->rope_base));
  const int tokens = kWarps / p.warps_per_token;
  const dim3 grid((a->n_tok + tokens - 1) / tokens);
  const auto kernel = a->kv_dtype == MLA_KV_FP8_E4M3 ? append_kernel<1>
                      : a->kv_dtype == MLA_KV_Q8_0   ? append_kernel<2>
                      : a->kv_dtype == MLA_KV_Q4_0   ? append_kernel<3>
                                                     : append_kernel<0>;
  return launch_pdl(kernel, grid, dim3(32 * kWarps), 0, stream, p);
}

}  // namespace mla
