"""One MLA attention step through the C ABI.

``DecodeStep``: absorb -> paged decode -> combine -> up-project (the absorbed
form); it owns the intermediate device buffers (q_lat, o_lat, lse, out and the
workspace) and replays the four calls on the current stream.  ``FusedStep``: the
same step through ``mla_decode_step`` (one call; one launch where the shape
allows).  ``PrefillStep``: the explicit form for long chunks of new tokens (one
call, two kernels).  ``PackedPrefill``: whole prompts of different lengths, into
the cache and through the explicit form.  ``SpeculativeStep``: a decode step over
drafted tokens with its append and their verification.  None does arithmetic of
its own.
"""

from __future__ import annotations

import torch

from . import (D_C, D_N, D_R, D_V, alloc_workspace, make_append_args, make_decode_args, make_prefill_args,
               make_prefill_packed_args, make_step_args, make_verify_args, mla_absorb_q, mla_append_kv,
               mla_combine_splits, mla_decode_num_splits, mla_decode_paged, mla_decode_step,
               mla_decode_step_launches, mla_prefill, mla_prefill_packed, mla_up_proj_v, mla_verify_draft)


class DecodeStep:
    def __init__(self, *, q_nope, q_pe, w_uk, w_uv, kv_cache, kv_scale, block_table, seq_lens,
                 causal, softmax_scale, num_splits=0, max_seq_len=0, out=None):
        B, s_q, H, _ = q_nope.shape
        dev = q_nope.device
        self.B, self.s_q, self.H = B, s_q, H
        self.q_nope, self.q_pe, self.w_uk, self.w_uv = q_nope, q_pe, w_uk, w_uv
        self.q_lat = torch.empty(B, s_q, H, D_C, dtype=torch.bfloat16, device=dev)
        self.o_lat = torch.empty(B, s_q, H, D_C, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(B, s_q, H, dtype=torch.float32, device=dev)
        self.out = out if out is not None else torch.empty(B, s_q, H, D_V, dtype=torch.bfloat16,
                                                           device=dev)
        self.args = make_decode_args(q_lat=self.q_lat, q_pe=q_pe, kv_cache=kv_cache,
                                     kv_scale=kv_scale, block_table=block_table,
                                     seq_lens=seq_lens, o_lat=self.o_lat, lse=self.lse,
                                     causal=causal, softmax_scale=softmax_scale,
                                     num_splits=num_splits, max_seq_len=max_seq_len)
        self.workspace = alloc_workspace(self.args, device=dev)
        self.num_splits = mla_decode_num_splits(self.args)
        self._keep = (kv_cache, kv_scale, block_table, seq_lens)

    def absorb(self, stream=None):
        n_tok = self.B * self.s_q
        mla_absorb_q(self.q_nope.view(n_tok, self.H, D_N), self.w_uk,
                     self.q_lat.view(n_tok, self.H, D_C), stream)

    def attend(self, stream=None):
        mla_decode_paged(self.args, stream)
        mla_combine_splits(self.args, stream)

    def up_project(self, stream=None):
        n_tok = self.B * self.s_q
        mla_up_proj_v(self.o_lat.view(n_tok, self.H, D_C), self.w_uv,
                      self.out.view(n_tok, self.H, D_V), stream)

    def run(self, stream=None):
        self.absorb(stream)
        self.attend(stream)
        self.up_project(stream)
        return self.out

    def capture(self, fn=None):
        """Records ``fn`` (default: the whole step) into a CUDA graph and returns
        it; ``graph.replay()`` then issues all of its launches with one host call.
        The step allocates nothing, so the graph stays valid while the buffers
        (and the arguments captured in it) are unchanged."""
        fn = fn or self.run
        fn()                       # first call outside capture: one-time host setup
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        return g


def step_from_workload(w, device="cuda", num_splits=0):
    """Copy a ``mla_inputs.Workload`` to the device and build its ``DecodeStep``."""
    d = lambda t: None if t is None else t.to(device, non_blocking=False).contiguous()
    return DecodeStep(q_nope=d(w.q_nope), q_pe=d(w.q_pe), w_uk=d(w.w_uk), w_uv=d(w.w_uv),
                      kv_cache=d(w.kv_cache), kv_scale=d(w.kv_scale),
                      block_table=d(w.block_table), seq_lens=d(w.seq_lens), causal=w.causal,
                      softmax_scale=w.softmax_scale, num_splits=num_splits,
                      max_seq_len=max(w.lens) if w.lens else 0)


class FusedStep:
    """The decode step through one ``mla_decode_step`` call: owns out, lse and the
    workspace (which holds q_lat, o_lat and the step's flags)."""

    def __init__(self, *, q_nope, q_pe, w_uk, w_uv, kv_cache, kv_scale, block_table, seq_lens,
                 causal, softmax_scale, num_splits=0, max_seq_len=0, out=None, fuse=0):
        B, s_q, H, _ = q_nope.shape
        dev = q_nope.device
        self.B, self.s_q, self.H = B, s_q, H
        self.lse = torch.empty(B, s_q, H, dtype=torch.float32, device=dev)
        self.out = out if out is not None else torch.empty(B, s_q, H, D_V, dtype=torch.bfloat16,
                                                           device=dev)
        self.args = make_step_args(q_nope=q_nope, q_pe=q_pe, w_uk=w_uk, w_uv=w_uv, kv_cache=kv_cache,
                                   kv_scale=kv_scale, block_table=block_table, seq_lens=seq_lens,
                                   out=self.out, lse=self.lse, causal=causal,
                                   softmax_scale=softmax_scale, num_splits=num_splits,
                                   max_seq_len=max_seq_len, fuse=fuse)
        self.workspace = alloc_workspace(self.args, device=dev)
        self.launches = mla_decode_step_launches(self.args)
        self._keep = (q_nope, q_pe, w_uk, w_uv, kv_cache, kv_scale, block_table, seq_lens)

    def run(self, stream=None):
        mla_decode_step(self.args, stream)
        return self.out

    def capture(self):
        """One CUDA graph of the step (see ``DecodeStep.capture``)."""
        self.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        return g


def fused_from_workload(w, device="cuda", num_splits=0, fuse=0):
    """Copy a ``mla_inputs.Workload`` to the device and build its ``FusedStep``."""
    d = lambda t: None if t is None else t.to(device, non_blocking=False).contiguous()
    return FusedStep(q_nope=d(w.q_nope), q_pe=d(w.q_pe), w_uk=d(w.w_uk), w_uv=d(w.w_uv),
                     kv_cache=d(w.kv_cache), kv_scale=d(w.kv_scale),
                     block_table=d(w.block_table), seq_lens=d(w.seq_lens), causal=w.causal,
                     softmax_scale=w.softmax_scale, num_splits=num_splits,
                     max_seq_len=max(w.lens) if w.lens else 0, fuse=fuse)


class PrefillStep:
    """Explicit-form attention of s_q new tokens per sequence over the paged bf16
    cache: owns out, lse and the workspace (the per-head keys and values)."""

    def __init__(self, *, q_nope, q_pe, w_uk, w_uv, kv_cache, block_table, seq_lens, causal,
                 softmax_scale, max_seq_len, out=None):
        B, s_q, H, _ = q_nope.shape
        dev = q_nope.device
        self.B, self.s_q, self.H = B, s_q, H
        self.lse = torch.empty(B, s_q, H, dtype=torch.float32, device=dev)
        self.out = out if out is not None else torch.empty(B, s_q, H, D_V, dtype=torch.bfloat16,
                                                           device=dev)
        self.args = make_prefill_args(q_nope=q_nope, q_pe=q_pe, w_uk=w_uk, w_uv=w_uv,
                                      kv_cache=kv_cache, block_table=block_table,
                                      seq_lens=seq_lens, out=self.out, lse=self.lse,
                                      max_seq_len=max_seq_len, causal=causal,
                                      softmax_scale=softmax_scale)
        self.workspace = alloc_workspace(self.args, device=dev)
        self._keep = (q_nope, q_pe, w_uk, w_uv, kv_cache, block_table, seq_lens)

    def run(self, stream=None):
        mla_prefill(self.args, stream)
        return self.out


def prefill_from_workload(w, device="cuda", max_seq_len=None):
    """Copy a bf16-cache ``mla_inputs.Workload`` to the device and build its
    ``PrefillStep``."""
    d = lambda t: t.to(device, non_blocking=False).contiguous()
    return PrefillStep(q_nope=d(w.q_nope), q_pe=d(w.q_pe), w_uk=d(w.w_uk), w_uv=d(w.w_uv),
                       kv_cache=d(w.kv_cache), block_table=d(w.block_table),
                       seq_lens=d(w.seq_lens), causal=w.causal, softmax_scale=w.softmax_scale,
                       max_seq_len=max_seq_len or max(max(w.lens), w.spec.s_q))


class PackedPrefill:
    """Whole prompts of different lengths, packed one after another: their latents
    and rotated RoPE keys go into the paged cache, and their tokens attend to their
    own prompt in the explicit form.  q [n_tok][H][192] and kv [n_tok][H][256] are
    the query's and the per-head key and value up-projections' outputs, latent
    [n_tok][576] the joint down-projection's (latent and RoPE key); nothing in them
    is rotated yet.  seq_lens holds the prompts' lengths.  Owns out, lse, the
    rotated parts and the workspaces."""

    def __init__(self, *, q, kv, latent, kv_cache, kv_scale, block_table, cu_seqlens, seq_lens, softmax_scale,
                 rope_base=10000.0, out=None):
        n, H, _ = q.shape
        dev = q.device
        bf16 = torch.bfloat16
        self.q_pe = torch.empty(n, H, D_R, dtype=bf16, device=dev)
        self.k_pe = torch.empty(n, D_R, dtype=bf16, device=dev)
        self.lse = torch.empty(n, H, dtype=torch.float32, device=dev)
        self.out = out if out is not None else torch.empty(n, H, D_V, dtype=bf16, device=dev)
        self.append_args = make_append_args(
            c=latent[:, :D_C], k_pe=latent[:, D_C:], q_pe=q[..., D_N:], k_pe_out=self.k_pe, q_pe_out=self.q_pe,
            kv_cache=kv_cache, kv_scale=kv_scale, block_table=block_table, cu_seqlens=cu_seqlens, seq_lens=seq_lens,
            rope_base=rope_base)
        self.attend_args = make_prefill_packed_args(
            q_nope=q[..., :D_N], q_pe=self.q_pe, k_nope=kv[..., :D_N], k_pe=self.k_pe, v=kv[..., D_N:],
            cu_seqlens=cu_seqlens, out=self.out, lse=self.lse, causal=True, softmax_scale=softmax_scale)
        self.append_workspace = alloc_workspace(self.append_args)
        self.workspace = alloc_workspace(self.attend_args)
        self._keep = (q, kv, latent, kv_cache, kv_scale, block_table, cu_seqlens, seq_lens)

    def run(self, stream=None):
        mla_append_kv(self.append_args, stream)
        mla_prefill_packed(self.attend_args, stream)
        return self.out


class SpeculativeStep(DecodeStep):
    """One decode step over the last token and its s_q - 1 drafts of every sequence:
    appends their latents and rotated RoPE keys (latent [B * s_q][576], q_pe
    [B][s_q][H][64], not yet rotated), attends causally, and, once the model has
    turned the output into probabilities, verifies the drafts; ``seq_lens`` (the
    drafts included) then loses the rejected ones in place.  q_pe is read where it
    stands on every run, so its first two dimensions have to merge without a copy."""

    def __init__(self, *, latent, q_nope, q_pe, w_uk, w_uv, kv_cache, kv_scale, block_table, seq_lens,
                 softmax_scale, rope_base=10000.0, num_splits=0, max_seq_len=0, out=None):
        B, s_q, H, _ = q_pe.shape
        if B > 1 and s_q > 1 and q_pe.stride(0) != s_q * q_pe.stride(1):
            raise ValueError("q_pe's sequences must follow one another at its token stride")
        dev = q_pe.device
        rotated = torch.empty_like(q_pe, memory_format=torch.contiguous_format)
        super().__init__(q_nope=q_nope, q_pe=rotated, w_uk=w_uk, w_uv=w_uv, kv_cache=kv_cache, kv_scale=kv_scale,
                         block_table=block_table, seq_lens=seq_lens, causal=True, softmax_scale=softmax_scale,
                         num_splits=num_splits, max_seq_len=max_seq_len, out=out)
        self.cu_seqlens = torch.arange(0, B * s_q + 1, s_q, dtype=torch.int32, device=dev)
        self.append_args = make_append_args(
            c=latent[:, :D_C], k_pe=latent[:, D_C:], q_pe=q_pe.flatten(0, 1), q_pe_out=rotated.flatten(0, 1),
            kv_cache=kv_cache, kv_scale=kv_scale, block_table=block_table, cu_seqlens=self.cu_seqlens,
            seq_lens=seq_lens, rope_base=rope_base)
        self.append_workspace = alloc_workspace(self.append_args)
        self.tokens = torch.empty(B, s_q, dtype=torch.int32, device=dev)
        self.num_accepted = torch.empty(B, dtype=torch.int32, device=dev)
        self.seq_lens = seq_lens
        self.verify_workspace = torch.zeros(256, dtype=torch.uint8, device=dev)
        self._keep += (latent, q_pe)

    def append(self, stream=None):
        mla_append_kv(self.append_args, stream)

    def run(self, stream=None):
        self.append(stream)
        return super().run(stream)

    def verify(self, *, target_probs, draft_probs, draft_tokens, u_accept, u_sample, stream=None):
        args = make_verify_args(target_probs=target_probs, draft_probs=draft_probs, draft_tokens=draft_tokens,
                                u_accept=u_accept, u_sample=u_sample, seq_lens=self.seq_lens,
                                tokens=self.tokens, num_accepted=self.num_accepted, new_lens=self.seq_lens,
                                workspace=self.verify_workspace)
        mla_verify_draft(args, stream)
        return self.tokens, self.num_accepted
