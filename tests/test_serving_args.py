"""Refusals of the packed append, the packed prompt attention and the draft
verification (CPU): the C ABI's host checks on made-up pointers, none of which
reaches a launch, and the tensor builders' checks."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import head_latent_attention_06_b200 as mla
from head_latent_attention_06_b200 import build as mla_build
from oracle import serving

OK, INVALID, UNSUPPORTED, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
P = 0x10000
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load()


def append_args(**kw):
    a = mla.AppendArgs()
    for f in ("c", "k_pe", "q_pe", "k_pe_out", "q_pe_out", "kv_cache", "block_table", "cu_seqlens", "seq_lens", "workspace"):
        setattr(a, f, P)
    a.workspace_bytes = 256
    a.c_tok, a.k_pe_tok, a.q_pe_tok, a.q_pe_head = 576, 576, 192 * 16, 192
    a.k_pe_out_tok, a.q_pe_out_tok, a.q_pe_out_head = 576, 192 * 16, 192
    a.n_tok, a.B, a.H, a.d_c, a.d_r, a.page_size = 8, 2, 16, 512, 64, 64
    a.num_pages, a.max_pages_per_seq, a.kv_dtype, a.rope_base = 4, 2, 0, 10000.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def packed_args(**kw):
    a = mla.PrefillPackedArgs()
    for f in ("q_nope", "q_pe", "k_nope", "k_pe", "v", "cu_seqlens", "out", "lse", "workspace"):
        setattr(a, f, P)
    a.workspace_bytes = 256
    a.q_nope_tok, a.q_nope_head, a.q_pe_tok, a.q_pe_head = 16 * 192, 192, 16 * 192, 192
    a.k_nope_tok, a.k_nope_head, a.k_pe_tok, a.v_tok, a.v_head = 8 * 256, 256, 64, 8 * 256, 256
    a.n_tok, a.B, a.H, a.H_kv, a.d_n, a.d_r, a.d_v, a.causal, a.softmax_scale = 8, 2, 16, 8, 128, 64, 128, 1, 0.07
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def verify_args(**kw):
    a = mla.VerifyArgs()
    for f in ("target_probs", "draft_probs", "draft_tokens", "num_draft", "u_accept", "u_sample", "seq_lens", "tokens",
              "num_accepted", "new_lens", "workspace"):
        setattr(a, f, P)
    a.workspace_bytes = 256
    a.target_seq, a.target_row, a.draft_seq, a.draft_row = 4000, 1000, 3000, 1000
    a.target_seq, a.draft_seq = 5 * 1000, 4 * 1000
    a.B, a.s_q, a.V, a.dtype = 2, 5, 1000, 0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


REFUSED = [
    (append_args, "mla_append_kv", [
        (dict(B=-1), INVALID), (dict(H=-1), INVALID), (dict(n_tok=-1), INVALID), (dict(num_pages=-1), INVALID),
        (dict(max_pages_per_seq=0), INVALID), (dict(H=129), UNSUPPORTED), (dict(d_c=256), UNSUPPORTED),
        (dict(d_r=32), UNSUPPORTED), (dict(page_size=16), UNSUPPORTED), (dict(kv_dtype=4), UNSUPPORTED),
        (dict(n_tok=(1 << 30) + 1), UNSUPPORTED), (dict(B=(1 << 30) + 1), UNSUPPORTED), (dict(max_pages_per_seq=1 << 26), UNSUPPORTED),
        (dict(rope_base=0.0), INVALID), (dict(rope_base=float("inf")), INVALID), (dict(rope_base=float("nan")), INVALID),
        (dict(workspace=None), INVALID), (dict(workspace=P + 8), MISALIGNED), (dict(workspace_bytes=255), WS_SMALL),
        (dict(c=None), INVALID), (dict(k_pe=None), INVALID), (dict(q_pe=None), INVALID), (dict(q_pe_out=None), INVALID),
        (dict(H=0), INVALID), (dict(kv_cache=None), INVALID), (dict(cu_seqlens=None), INVALID), (dict(seq_lens=None), INVALID),
        (dict(block_table=None), INVALID), (dict(kv_dtype=1), INVALID), (dict(num_pages=0), INVALID),
        (dict(c=P + 8), MISALIGNED), (dict(q_pe_out=P + 2), MISALIGNED), (dict(k_pe_out=P + 2), MISALIGNED),
        (dict(kv_cache=P + 4), MISALIGNED), (dict(cu_seqlens=P + 2), MISALIGNED),
        (dict(c_tok=577), MISALIGNED), (dict(c_tok=0), INVALID), (dict(q_pe_head=-192), INVALID),
        (dict(q_pe_tok=1 << 38), UNSUPPORTED), (dict(k_pe_out_tok=64), INVALID), (dict(q_pe_out_head=64), INVALID),
        (dict(q_pe_out_tok=64 * 16), INVALID),
        # rows or heads of an output over one another (written over themselves, so that no other rule refuses them)
        (dict(k_pe_out_tok=56, k_pe_tok=56), INVALID), (dict(q_pe_out_tok=8, q_pe_tok=8), INVALID),
        (dict(q_pe_out_head=32, q_pe_head=32), INVALID),
    ]),
    (packed_args, "mla_prefill_packed", [
        (dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(H_kv=0), INVALID), (dict(n_tok=-1), INVALID),
        (dict(H_kv=3), INVALID), (dict(H_kv=32), INVALID), (dict(H=256), UNSUPPORTED), (dict(d_n=64), UNSUPPORTED),
        (dict(d_r=32), UNSUPPORTED), (dict(d_v=64), UNSUPPORTED), (dict(n_tok=(1 << 30) + 1), UNSUPPORTED), (dict(B=(1 << 30) + 1), UNSUPPORTED),
        (dict(softmax_scale=0.0), INVALID), (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID),
        (dict(softmax_scale=float("inf")), INVALID),
        (dict(workspace=None), INVALID), (dict(workspace=P + 4), MISALIGNED), (dict(workspace_bytes=0), WS_SMALL),
        (dict(q_nope=None), INVALID), (dict(k_nope=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
        (dict(cu_seqlens=None), INVALID), (dict(q_pe=None), INVALID), (dict(k_pe=None), INVALID), (dict(d_r=0), INVALID),
        (dict(q_nope=P + 8), MISALIGNED), (dict(v=P + 2), MISALIGNED), (dict(out=P + 8), MISALIGNED),
        (dict(lse=P + 2), MISALIGNED), (dict(cu_seqlens=P + 1), MISALIGNED),
        (dict(q_nope_tok=0), INVALID), (dict(v_head=0), INVALID), (dict(k_pe_tok=-64), INVALID), (dict(k_nope_head=100), MISALIGNED),
        (dict(v_tok=1 << 38), UNSUPPORTED),
    ]),
    (verify_args, "mla_verify_draft", [
        (dict(B=-1), INVALID), (dict(s_q=0), INVALID), (dict(V=0), INVALID), (dict(s_q=1025), UNSUPPORTED),
        (dict(V=(1 << 20) + 1), UNSUPPORTED), (dict(B=(1 << 24) + 1), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
        (dict(workspace=None), INVALID), (dict(workspace=P + 8), MISALIGNED), (dict(workspace_bytes=100), WS_SMALL),
        (dict(target_probs=None), INVALID), (dict(u_sample=None), INVALID), (dict(tokens=None), INVALID),
        (dict(num_accepted=None), INVALID), (dict(draft_tokens=None), INVALID), (dict(u_accept=None), INVALID),
        (dict(seq_lens=None), INVALID), (dict(target_probs=P + 2), MISALIGNED), (dict(draft_probs=P + 1, dtype=1), MISALIGNED),
        (dict(tokens=P + 2), MISALIGNED), (dict(target_row=-1), INVALID), (dict(draft_seq=-1), INVALID),
    ]),
]


@pytest.mark.parametrize("make,fn,change,code", [(m, f, c, code) for m, f, cs in REFUSED for c, code in cs])
def test_abi_refuses(lib, make, fn, change, code):
    assert getattr(lib, fn)(ctypes.byref(make(**change)), None) == code


@pytest.mark.parametrize("fn,size", [("mla_append_kv", "mla_append_workspace_size"),
                                     ("mla_prefill_packed", "mla_prefill_packed_workspace_size"),
                                     ("mla_verify_draft", "mla_verify_workspace_size")])
def test_abi_null_struct(lib, fn, size):
    n = ctypes.c_size_t(0)
    assert getattr(lib, fn)(None, None) == INVALID
    assert getattr(lib, size)(None, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("make,fn,empty", [(append_args, "mla_append_kv", dict(n_tok=0)), (append_args, "mla_append_kv", dict(B=0)),
                                           (packed_args, "mla_prefill_packed", dict(n_tok=0)),
                                           (packed_args, "mla_prefill_packed", dict(B=0)), (verify_args, "mla_verify_draft", dict(B=0))])
def test_abi_empty_work_is_fine(lib, make, fn, empty):
    """Nothing to do: accepted, and nothing is enqueued (there is no device here)."""
    assert getattr(lib, fn)(ctypes.byref(make(**empty)), None) == OK


def test_workspace_sizes(lib):
    assert mla.mla_append_workspace_size(append_args()) == 256
    assert mla.mla_prefill_packed_workspace_size(packed_args()) == 256
    assert mla.mla_verify_workspace_size(verify_args()) == 256
    with pytest.raises(mla.MlaError, match="MLA_ERR_UNSUPPORTED"):
        mla.mla_append_workspace_size(append_args(d_r=63))


C_PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include "mla.h"

int main(void) {
  /* host-side checks only: nothing here reaches a CUDA launch */
  size_t bytes = 0;
  mla_append_args_t a;
  memset(&a, 0, sizeof a);
  a.n_tok = 8; a.B = 2; a.H = 16; a.d_c = MLA_D_C; a.d_r = MLA_D_R; a.page_size = MLA_PAGE_SIZE;
  a.num_pages = 4; a.max_pages_per_seq = 2; a.kv_dtype = MLA_KV_Q4_0; a.rope_base = 10000.f;
  if (mla_append_workspace_size(&a, &bytes) != MLA_OK || bytes != 256) return 1;
  if (mla_append_kv(&a, 0) != MLA_ERR_INVALID_VALUE) return 2;          /* no workspace */
  mla_prefill_packed_args_t p;
  memset(&p, 0, sizeof p);
  p.n_tok = 8; p.B = 2; p.H = 16; p.H_kv = 4; p.d_n = MLA_D_QK_NOPE; p.d_v = MLA_D_V; p.causal = 1;
  p.softmax_scale = 0.0884f;
  if (mla_prefill_packed_workspace_size(&p, &bytes) != MLA_OK || bytes != 256) return 3;
  p.d_r = 32;
  if (mla_prefill_packed(&p, 0) != MLA_ERR_UNSUPPORTED) return 4;
  mla_verify_args_t v;
  memset(&v, 0, sizeof v);
  v.B = 2; v.s_q = 4; v.V = 1000; v.dtype = MLA_PROB_BF16;
  if (mla_verify_workspace_size(&v, &bytes) != MLA_OK || bytes != 256) return 5;
  if (mla_verify_draft(&v, 0) != MLA_ERR_INVALID_VALUE) return 6;
  if (strcmp(mla_status_string(MLA_ERR_BAD_TOKEN), "MLA_ERR_BAD_TOKEN") != 0) return 7;
  printf("%d %d %d\n", (int)sizeof a, (int)sizeof p, (int)sizeof v);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_c_program_calls_the_entry_points(tmp_path, lib):
    """From plain C; the binding's structs are as large as the header's."""
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text(C_PROGRAM)
    d = os.path.dirname(mla.LIB_PATH)
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(os.path.dirname(d), "include"),
                        str(src), "-o", str(exe), mla.LIB_PATH, f"-Wl,-rpath,{d}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.returncode
    assert [int(n) for n in r.stdout.split()] == [ctypes.sizeof(t) for t in (mla.AppendArgs, mla.PrefillPackedArgs, mla.VerifyArgs)]


# ------------------------------------------------------------------ builders

def append_tensors():
    z = torch.zeros
    return dict(c=z(6, 512, dtype=bf16), k_pe=z(6, 64, dtype=bf16), q_pe=z(6, 16, 64, dtype=bf16), k_pe_out=z(6, 64, dtype=bf16),
                q_pe_out=z(6, 16, 64, dtype=bf16), kv_cache=z(4, 64, 576, dtype=bf16), kv_scale=None,
                block_table=z(2, 3, dtype=i32), cu_seqlens=z(3, dtype=i32), seq_lens=z(2, dtype=i32))


def packed_tensors():
    z = torch.zeros
    return dict(q_nope=z(6, 16, 128, dtype=bf16), q_pe=z(6, 16, 64, dtype=bf16), k_nope=z(6, 4, 128, dtype=bf16),
                k_pe=z(6, 64, dtype=bf16), v=z(6, 4, 128, dtype=bf16), cu_seqlens=z(3, dtype=i32),
                out=z(6, 16, 128, dtype=bf16), lse=z(6, 16))


def verify_tensors():
    z = torch.zeros
    return dict(target_probs=z(2, 4, 50), draft_probs=z(2, 3, 50), draft_tokens=z(2, 3, dtype=i32), num_draft=z(2, dtype=i32),
                u_accept=z(2, 3), u_sample=z(2), seq_lens=z(2, dtype=i32), tokens=z(2, 4, dtype=i32),
                num_accepted=z(2, dtype=i32), new_lens=z(2, dtype=i32))


BUILDERS = [(mla.make_append_args, append_tensors, {}), (mla.make_prefill_packed_args, packed_tensors, dict(softmax_scale=0.07)),
            (mla.make_verify_args, verify_tensors, {})]


@pytest.mark.parametrize("build,tensors,kw", BUILDERS)
def test_builders_need_device_tensors(build, tensors, kw):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        build(**tensors(), **kw)


@pytest.mark.parametrize("which,field,bad,msg", [
    (0, "c", torch.zeros(6, 512), "c: dtype"), (0, "k_pe", torch.zeros(5, 64, dtype=bf16), "k_pe: shape"),
    (0, "k_pe", torch.zeros(64, 6, dtype=bf16).T, "k_pe: its innermost"), (0, "q_pe_out", None, "q_pe_out is required"),
    (0, "q_pe", None, "q_pe_out without q_pe"), (0, "block_table", torch.zeros(2, 6, dtype=i32)[:, :3], "block_table must be contiguous"),
    (0, "cu_seqlens", torch.zeros(2, dtype=i32), "cu_seqlens: shape"), (0, "seq_lens", torch.zeros(2), "seq_lens: dtype"),
    (0, "kv_cache", torch.zeros(4, 64, 576, dtype=torch.int8), "kv_scale is required"),
    (1, "q_pe", None, "q_pe and k_pe come together"), (1, "v", torch.zeros(6, 8, 128, dtype=bf16), "v: shape"),
    (1, "q_nope", torch.zeros(6, 16, 128, dtype=torch.float16), "q_nope: dtype"),
    (1, "out", torch.zeros(6, 16, 192, dtype=bf16)[..., :128], "out must be contiguous"),
    (1, "k_nope", torch.zeros(6, 128, dtype=bf16), "q_nope must be"), (1, "lse", torch.zeros(6, 8), "lse: shape"),
    (2, "draft_probs", torch.zeros(2, 3, 50, dtype=bf16), "draft_probs: dtype"), (2, "tokens", torch.zeros(2, 3, dtype=i32), "tokens: shape"),
    (2, "target_probs", torch.zeros(2, 50), "target_probs must be"), (2, "seq_lens", None, "seq_lens is required"),
    (2, "target_probs", torch.zeros(2, 50, 4).transpose(1, 2), "target_probs: its innermost"),
    (2, "u_accept", torch.zeros(2, 3, dtype=torch.float64), "u_accept: dtype"),
])
def test_builders_reject_bad_tensors(which, field, bad, msg):
    build, tensors, kw = BUILDERS[which]
    t = tensors()
    t[field] = bad
    with pytest.raises(ValueError, match=msg):
        build(**t, **kw)


def test_entry_points_make_the_tensors_device_current(monkeypatch):
    """Arguments on another device than the current one: the call is made with theirs
    current and on that device's stream."""
    seen = []
    current = [0]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev.index

        def __exit__(self, *exc):
            current[0] = self.before

    class Lib:
        def mla_append_kv(self, args, stream):
            seen.append((current[0], stream))
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(mla, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(mla, "_lib", Lib())
    a = append_args()
    for index in (0, 1):
        a.device = torch.device("cuda", index)
        mla.mla_append_kv(a)
    a.device = torch.device("cuda", 1)
    mla.mla_append_kv(a, stream=7)
    assert seen == [(0, 100), (1, 101), (1, 7)] and current[0] == 0


# ------------------------------------------------------------------ the oracle's own pins

def test_oracle_packed_attention_is_softmax():
    """Each sequence alone, by torch's softmax over a masked score matrix."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(9, h, 5, generator=g, dtype=torch.float64) for h in (4, 2, 2))
    cu = [0, 4, 4, 9]
    o, lse, mass, size = serving.attend_packed(q.numpy(), k.numpy(), v.numpy(), cu, 0.3, True)
    for lo, hi in ((0, 4), (4, 9)):
        s = torch.einsum("ihd,jhd->hij", q[lo:hi], k[lo:hi].repeat_interleave(2, 1)) * 0.3
        s = s.masked_fill(torch.ones(hi - lo, hi - lo, dtype=torch.bool).triu(1), -float("inf"))
        want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v[lo:hi].repeat_interleave(2, 1))
        assert np.allclose(o[lo:hi], want.numpy(), atol=1e-13)
        assert np.allclose(lse[lo:hi], s.logsumexp(-1).T.numpy(), atol=1e-13)


def test_oracle_verification_draws_from_the_target():
    """Summed over a fine grid of both random numbers, the first token's distribution is the target's."""
    p = np.array([[[0.5, 0.2, 0.3, 0.0], [0.25] * 4]])
    q = np.array([[[0.1, 0.6, 0.1, 0.2]]])
    n = 200
    grid = (np.arange(n) + 0.5) / n
    share = np.zeros(4)
    for x in range(4):
        for u in grid:
            for r in grid[::8]:
                t, a, new = serving.verify_draft(p, q, [[x]], [1], [[u]], [r], [7])
                assert new[0] == 6 + a[0]
                share[t[0, 0]] += q[0, 0, x] / (n * len(grid[::8]))
    # a draft's accepted share is off by less than one of the 200 points (weighted by
    # q <= 0.6); of the rejected 0.6 = sum max(p - q, 0), a token's share lies between two
    # boundaries, each off by less than one of the 25 points
    assert np.abs(share - p[0, 0]).max() < 0.6 / 200 + 2 * 0.6 / 25


def test_oracle_append_positions():
    rows, seq, pos = serving.packed_positions([2, 4, 4, 7], [10, 5, 3])
    assert rows.tolist() == [2, 3, 4, 5, 6] and seq.tolist() == [0, 0, 2, 2, 2] and pos.tolist() == [8, 9, 0, 1, 2]


def test_speculative_step_takes_no_copy_of_its_queries():
    """Queries whose sequences do not follow one another would be copied once and then be stale."""
    from head_latent_attention_06_b200.step import SpeculativeStep
    q = torch.zeros(3, 2, 4, 192, dtype=torch.bfloat16)
    names = ("latent", "q_nope", "w_uk", "w_uv", "kv_cache", "kv_scale", "block_table", "seq_lens")
    for bad in (q.transpose(0, 1)[..., 128:], q[:, :1].expand(3, 2, 4, 192)[..., 128:]):
        with pytest.raises(ValueError, match="q_pe"):
            SpeculativeStep(q_pe=bad, softmax_scale=1.0, **dict.fromkeys(names))


def test_speculative_step_verifies_all_its_drafts():
    """The step appends s_q tokens of every sequence, so all of them have s_q - 1 drafts."""
    import inspect
    from head_latent_attention_06_b200.step import SpeculativeStep
    assert "num_draft" not in inspect.signature(SpeculativeStep.verify).parameters


@pytest.mark.parametrize("n_tok,H,tok,head", [
    (8, 16, 64, 64),                        # each token's heads are the next token's, one on
    (8, 16, 128, 64),
    (2, 16, 64 * 15, 64),                   # the last head alone
    (8, 16, 1024, 1000),                    # partly over one another
    (8, 4, 64, 256),                        # heads outermost, too near
    (8, 128, 4096, 72),                     # far apart in both indices
    (1 << 30, 128, 1 << 37, 1 << 37),       # no product of theirs fits 64 bits
])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_refuses_query_outputs_over_one_another(lib, n_tok, H, tok, head, in_place):
    """Another token's head on the same values: neither stride shows it alone."""
    a = append_args(n_tok=n_tok, H=H, q_pe_out_tok=tok, q_pe_out_head=head)
    if in_place:
        a.q_pe_tok, a.q_pe_head = tok, head
    else:
        a.q_pe_out = 0x10000000
    assert lib.mla_append_kv(ctypes.byref(a), None) == INVALID
