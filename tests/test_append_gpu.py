"""GPU parity of the packed append (mla_append_kv) against the fp64 oracle.

Tolerances.  The rotation of a pair (x0, x1) is done in fp32 from an angle that is
exact to fp32's last bit: the reduced turn is rounded to fp32 (|2 turn| <= 1, so
the angle is off by at most pi 2^-25 < 2^-23), sine and cosine are within 2 ulp
(2^-23 each), and two products and their sum round three times: together below
8 * 2^-24 * (|x0| + |x1|) = ROT.  A value rounded to bf16 adds 2^-8 of itself.
The latent's values are inputs: their cache rows are compared bit for bit.
A rotated value in a code: half a step d / 2, what the clamp takes when the fp16
scale was rounded down (amax 2^-11), and ROT; an e4m3 code 2^-4 of its value or
half its smallest step, scale 2^-10.  Scales: their own rounding (fp16 2^-11, fp32
2^-24 for the maximum's ROT and twice 2^-24 for the division and the product).
"""

import numpy as np
import pytest
import torch

from mla_inputs import bf16_bits, f16_bits, fp8_bits, int8_bits
from oracle import cache_write as cw
from oracle import mla_oracle as om
from oracle import serving

pytestmark = pytest.mark.gpu

bf16, i32 = torch.bfloat16, torch.int32


def make(news, lens, H, kv, seed=1, head=0, tail=0, padded=False, gain=1.0, extra_pages=3):
    """CPU tensors of one packed append: `news` tokens per sequence, `lens` after it,
    `head` and `tail` rows of no sequence; `padded`: inputs as views of wider arrays."""
    g = torch.Generator().manual_seed(seed)
    rows = head + sum(news) + tail
    wide = 8 if padded else 0
    joint = (torch.randn(rows, 576 + wide, generator=g) * gain).to(bf16)
    q = torch.randn(rows, H, 192 if padded else 64, generator=g).to(bf16)
    pages = [(n + 63) // 64 for n in lens]
    P = max(1, sum(pages)) + extra_pages
    perm = torch.randperm(P, generator=g).to(i32)
    table = torch.full((len(lens), max(1, max(pages))), 0, dtype=i32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    scale = None
    if kv == "bf16":
        cache = torch.randn(P, 64, 576, generator=g).to(bf16)
    elif kv == "fp8":
        cache = torch.randn(P, 64, 576, generator=g).to(torch.float8_e4m3fn)
        scale = torch.rand(P, 64, generator=g) + 0.5
    elif kv == "q8_0":
        cache = torch.randint(-127, 128, (P, 64, 576), generator=g, dtype=torch.int8)
        scale = (torch.rand(P, 64, 18, generator=g) + 0.5).half()
    else:
        cache = torch.randint(0, 256, (P, 64, 288), generator=g, dtype=torch.uint8)
        scale = (torch.rand(P, 64, 18, generator=g) + 0.5).half()
    cu = torch.tensor([head] + list(head + np.cumsum(news)), dtype=i32)
    return dict(joint=joint, q=q, cache=cache, scale=scale, table=table, cu=cu, lens=torch.tensor(lens, dtype=i32), kv=kv)


def bits(t):
    if t.dtype == bf16:
        return bf16_bits(t)
    if t.dtype == torch.float8_e4m3fn:
        return fp8_bits(t)
    return int8_bits(t) if t.dtype == torch.int8 else t.numpy()


def run(mla, x, in_place=False, keep_k=True, rope_base=10000.0, stream=None):
    d = {k: v.cuda() if torch.is_tensor(v) else v for k, v in x.items()}
    H = d["q"].shape[1]
    q_pe = d["q"][..., -64:]
    c, k_pe = d["joint"][:, :512], d["joint"][:, 512:576]
    k_out = k_pe if in_place else torch.full((c.shape[0], 64), 7.0, dtype=bf16, device="cuda")
    q_out = q_pe if in_place else torch.full((c.shape[0], H, 64), 7.0, dtype=bf16, device="cuda")
    a = mla.make_append_args(c=c, k_pe=k_pe, q_pe=q_pe if H else None, k_pe_out=k_out if keep_k else None,
                             q_pe_out=q_out if H else None, kv_cache=d["cache"], kv_scale=d["scale"],
                             block_table=d["table"], cu_seqlens=d["cu"], seq_lens=d["lens"], rope_base=rope_base)
    ws = mla.alloc_workspace(a)
    mla.mla_append_kv(a, stream)
    status = mla.mla_get_status(ws, stream)
    torch.cuda.synchronize()
    return dict(cache=d["cache"].cpu(), scale=None if d["scale"] is None else d["scale"].cpu(), k=k_out.cpu(), q=q_out.cpu(),
                status=status)


def check(x, got, rope_base=10000.0, skip=()):
    """`skip`: packed rows that must have been left out."""
    c = om.bf16_to_f64(bf16_bits(x["joint"][:, :512]))
    k = om.bf16_to_f64(bf16_bits(x["joint"][:, 512:576]))
    q = om.bf16_to_f64(bf16_bits(x["q"][..., -64:]))
    rows, seq, pos, exact = serving.append_rows(c, k, x["cu"].numpy(), x["lens"].numpy(), rope_base)
    real = np.array([i for i in range(rows.size) if int(rows[i]) not in set(skip)], int)
    rows, seq, pos, exact = rows[real], seq[real], pos[real], exact[real]
    rot = lambda v: np.repeat(8 * 2.0 ** -24 * (np.abs(v[..., 0::2]) + np.abs(v[..., 1::2])), 2, axis=-1)
    # the rotated outputs
    if got["k"] is not None:
        d = np.abs(om.bf16_to_f64(bf16_bits(got["k"]))[rows] - exact[:, 512:])
        assert (d <= 2.0 ** -8 * np.abs(exact[:, 512:]) + rot(k[rows])).all(), d.max()
    if q.shape[1]:
        eq = cw.rope(q[rows], np.repeat(pos[:, None], q.shape[1], 1), rope_base)
        d = np.abs(om.bf16_to_f64(bf16_bits(got["q"]))[rows] - eq)
        assert (d <= 2.0 ** -8 * np.abs(eq) + rot(q[rows])).all(), d.max()
    # the cache: rows of the new tokens, and every other bit as it was
    table = x["table"].numpy()
    before, after = bits(x["cache"]), bits(got["cache"])
    keep = np.ones(after.shape[:2], bool)
    rk = rot(k[rows])
    for i in range(rows.size):
        page, r = int(table[seq[i], pos[i] // 64]), int(pos[i] % 64)
        keep[page, r] = False
        row, full = after[page, r], exact[i]
        top = np.abs(full[512:]).max()
        if x["kv"] == "bf16":
            assert np.array_equal(row[:512], bf16_bits(x["joint"][rows[i]:rows[i] + 1, :512])[0])
            d = np.abs(om.bf16_to_f64(row[512:]) - full[512:])
            assert (d <= 2.0 ** -8 * np.abs(full[512:]) + rk[i]).all()
        elif x["kv"] == "fp8":
            sc = float(got["scale"][page, r])
            amax = np.abs(full).max()
            want = amax / 448 if amax > 0 else 1.0
            assert abs(sc - want) <= (rk[i].max() / 448 if amax > 0 else 0) + 2.0 ** -23 * want
            d = np.abs(om.e4m3fn_to_f64(row) * sc - full)
            err = np.concatenate([np.zeros(512), rk[i]])
            assert (d <= 2.0 ** -4 * np.abs(full) + 2.0 ** -10 * sc + err + 2.0 ** -22 * np.abs(full)).all()
        else:
            levels = 127 if x["kv"] == "q8_0" else 7
            fn = cw.quantise_row_q8_0 if x["kv"] == "q8_0" else cw.quantise_row_q4_0
            want, wd = fn(full)
            sc = f16_bits(got["scale"])[page, r]
            n_lat = 512 if x["kv"] == "q8_0" else 256
            assert np.array_equal(row[:n_lat].view(np.uint8), np.asarray(want)[:n_lat].view(np.uint8))
            assert np.array_equal(sc[:16], np.asarray(wd, np.float16)[:16].view(np.uint16))
            if x["kv"] == "q8_0":
                code = row.view(np.int8).astype(np.float64)
            else:
                code = np.stack([row & 15, row >> 4], -1).reshape(-1).astype(np.float64) - 8
            d_blk = om.f16_to_f64(sc)
            for blk in (16, 17):
                part = slice(32 * blk, 32 * blk + 32)
                e = rk[i][32 * blk - 512:32 * blk - 480]
                amax = np.abs(full[part]).max()
                assert abs(d_blk[blk] - amax / levels) <= 2.0 ** -11 * amax / levels + 2.0 ** -25 + e.max() / levels
                off = np.abs(code[part] * d_blk[blk] - full[part])
                assert (off <= d_blk[blk] / 2 * (1 + 2.0 ** -20) + 2.0 ** -11 * amax + e).all()
    assert np.array_equal(before[keep], after[keep])
    if x["scale"] is not None:
        assert np.array_equal(x["scale"].numpy()[keep], got["scale"].numpy()[keep])


KINDS = ["bf16", "fp8", "q8_0", "q4_0"]


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("news,lens,H,kw", [
    ([1], [1], 16, {}),                                       # the first token of one sequence
    ([1] * 5, [1, 64, 65, 128, 300], 128, {}),                # one token each, on both sides of a page
    ([3, 0, 130, 1, 64], [3, 40, 200, 129, 64], 16, dict(head=2, tail=5, padded=True)),  # empty, ragged, padded batch
    ([7, 2], [100, 66], 0, {}),                               # no queries
    ([2, 1], [70, 1], 33, dict(padded=True)),                 # an odd number of heads, two warps a token
    ([4, 9], [4, 9], 65, dict(padded=True)),                  # four warps a token
    ([1], [17], 1, dict(gain=0.0)),                           # all-zero rows
])
def test_append_matches_oracle(cuda_lib, kv, news, lens, H, kw):
    x = make(news, lens, H, kv, **kw)
    got = run(cuda_lib, x)
    assert got["status"] == 0
    check(x, got)
    head, end = int(x["cu"][0]), int(x["cu"][-1])
    for t in (got["k"], got["q"]):          # rows of no sequence stay as they were
        assert bool((t[:head] == 7).all()) and bool((t[end:] == 7).all())


@pytest.mark.parametrize("kv", ["bf16", "q4_0"])
def test_append_in_place(cuda_lib, kv):
    """The rotated key and queries over their inputs (views of wider arrays)."""
    x = make([5, 70], [69, 70], 16, kv, padded=True, tail=3, seed=2)
    a, b = run(cuda_lib, x), run(cuda_lib, x, in_place=True)
    assert a["status"] == b["status"] == 0
    n = int(x["cu"][-1])
    assert torch.equal(a["k"][:n], b["k"][:n]) and torch.equal(a["q"][:n], b["q"][:n])
    assert np.array_equal(bits(a["cache"]), bits(b["cache"]))
    assert torch.equal(b["k"][n:], x["joint"][n:, 512:576]) and torch.equal(b["q"][n:], x["q"][n:, :, -64:])


def test_append_without_key_output_many_sequences(cuda_lib):
    """More sequences than one round of the search over the offsets covers, some empty."""
    rng = np.random.default_rng(5)
    news = [int(v) for v in rng.integers(0, 4, 1100)]
    lens = [n + int(v) for n, v in zip(news, rng.integers(0, 70, 1100))]
    x = make(news, lens, 1, "fp8", seed=3)
    got = run(cuda_lib, x, keep_k=False)
    assert got["status"] == 0
    got["k"] = None
    check(x, got)


@pytest.mark.parametrize("base,L", [(10000.0, 131072), (500000.0, 1 << 20), (1.0, 5000)])
def test_append_far_positions(cuda_lib, base, L):
    """The angle of far positions (the last pages of a long sequence)."""
    pages = (L + 63) // 64
    x = make([3], [100], 16, "bf16", seed=4)
    table = torch.zeros(1, pages, dtype=i32)
    table[0, -2:] = torch.tensor([1, 2])
    x["table"], x["lens"] = table, torch.tensor([L], dtype=i32)
    got = run(cuda_lib, x, rope_base=base)
    assert got["status"] == 0
    check(x, got, rope_base=base)


def test_append_skips_what_it_cannot_place(cuda_lib):
    """A length below the new tokens or past the block table, and a page outside the
    cache: recorded, that token left out, the others written."""
    x = make([2, 2, 2, 2], [10, 20, 30, 100], 16, "bf16", seed=6)
    x["lens"][0] = 1
    got = run(cuda_lib, x)
    assert got["status"] == 8                                  # MLA_ERR_BAD_SEQ_LEN
    check(dict(x, lens=torch.tensor([2, 20, 30, 100], dtype=i32)), got, skip=(0, 1))
    assert bool((got["k"][:2] == 7).all())
    x = make([2, 2], [10, 66], 16, "q8_0", seed=7)
    x["table"][1, 1] = 99
    got = run(cuda_lib, x)
    assert got["status"] == 7                                  # MLA_ERR_BAD_BLOCK_TABLE
    check(x, got, skip=(2, 3))
    x = make([1], [64], 16, "bf16", seed=8)
    x["lens"][0] = 65
    got = run(cuda_lib, x)
    assert got["status"] == 8 and torch.equal(got["cache"], x["cache"])
    x = make([3, 3], [10, 10], 16, "bf16", seed=9)
    x["cu"][1] = 50                                            # beyond the rows
    got = run(cuda_lib, x)
    assert got["status"] == 8


def test_append_on_another_stream_and_in_a_graph(cuda_lib):
    x = make([3, 1], [70, 9], 16, "q8_0", seed=10)
    want = run(cuda_lib, x)
    s = torch.cuda.Stream()
    got = run(cuda_lib, x, stream=s)
    assert got["status"] == 0 and torch.equal(got["cache"], want["cache"]) and torch.equal(got["q"], want["q"])
    d = {k: v.cuda() for k, v in x.items() if torch.is_tensor(v)}
    k_out = torch.zeros(4, 64, dtype=bf16, device="cuda")
    q_out = torch.zeros(4, 16, 64, dtype=bf16, device="cuda")
    a = cuda_lib.make_append_args(c=d["joint"][:, :512], k_pe=d["joint"][:, 512:576], q_pe=d["q"], k_pe_out=k_out,
                                  q_pe_out=q_out, kv_cache=d["cache"], kv_scale=d["scale"], block_table=d["table"],
                                  cu_seqlens=d["cu"], seq_lens=d["lens"])
    ws = cuda_lib.alloc_workspace(a)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cuda_lib.mla_append_kv(a)
    d["lens"].sub_(1)                                          # read when it is replayed
    g.replay()
    assert cuda_lib.mla_get_status(ws) == 0
    check(dict(x, lens=x["lens"] - 1), dict(cache=d["cache"].cpu(), scale=d["scale"].cpu(), k=k_out.cpu(), q=q_out.cpu()))




@pytest.mark.parametrize("kv", ["bf16", "q4_0"])
def test_append_far_pages(cuda_lib, kv):
    """Rows more than 2^32 bytes into the cache."""
    P = 60000 if kv == "bf16" else 250000
    x = make([3, 2], [66, 64], 16, kv, seed=12)
    small = x["cache"].shape[0]
    cache = torch.zeros(P, *x["cache"].shape[1:], dtype=x["cache"].dtype, device="cuda")
    scale = None if x["scale"] is None else torch.zeros(P, 64, 18, dtype=torch.float16, device="cuda")
    shift = P - small
    d = {k: v.cuda() for k, v in x.items() if torch.is_tensor(v)}
    k_out, q_out = torch.zeros(5, 64, dtype=bf16, device="cuda"), torch.zeros(5, 16, 64, dtype=bf16, device="cuda")
    cache[shift:] = d["cache"]
    if scale is not None:
        scale[shift:] = d["scale"]
    table = d["table"] + shift
    a = cuda_lib.make_append_args(c=d["joint"][:, :512], k_pe=d["joint"][:, 512:576], q_pe=d["q"], k_pe_out=k_out,
                                  q_pe_out=q_out, kv_cache=cache, kv_scale=scale, block_table=table,
                                  cu_seqlens=d["cu"], seq_lens=d["lens"])
    ws = cuda_lib.alloc_workspace(a)
    cuda_lib.mla_append_kv(a)
    assert cuda_lib.mla_get_status(ws) == 0
    check(x, dict(cache=cache[shift:].cpu(), scale=None if scale is None else scale[shift:].cpu(), k=k_out.cpu(), q=q_out.cpu()))
    assert not bool(cache[:shift].view(torch.uint8).any())


@pytest.mark.parametrize("kv", ["fp8", "q8_0", "q4_0"])
def test_append_codes_at_ties(cuda_lib, kv):
    """Values whose quotients are exactly between two codes, a hair beside that, and
    subnormal; rows from tiny to huge; each bit of the latents' codes and scales."""
    x = make([64], [64], 1, kv, seed=13)
    g = torch.Generator().manual_seed(13)
    rows = torch.zeros(64, 576)
    for i in range(64):
        e = 2.0 ** (2 * i - 64)
        if kv == "fp8":
            v = (torch.randint(-120, 121, (576,), generator=g).float() + 0.0) / 16      # ties of three mantissa bits
            v[::7] = torch.randint(-15, 16, (83,), generator=g).float() * 2.0 ** -10    # of the smallest steps
            v[5] = 448.0
        else:
            levels = 127 if kv == "q8_0" else 7
            v = torch.randint(-levels, levels, (576,), generator=g).float() + 0.5
            v[::3] *= 1 + 2.0 ** -7 * torch.randint(-1, 2, (192,), generator=g).float()
            v[::32] = levels
        rows[i] = v * e
    if kv != "fp8":
        rows[:, :] = rows.clamp(-3e4, 3e4)
    x["joint"] = rows.to(bf16)
    x["joint"][:, 512:] = 0
    got = run(cuda_lib, x)
    assert got["status"] == 0
    check(x, got)
    page = int(x["table"][0, 0])
    c = om.bf16_to_f64(bf16_bits(x["joint"]))
    n = 256 if kv == "q4_0" else 512          # (the key's zeros may come out of the rotation as -0)
    for i in range(64):
        if kv == "fp8":
            code, sc = cw.quantise_row_e4m3(c[i])
            assert got["scale"][page, i].item() == sc
        else:
            code, sc = (cw.quantise_row_q8_0 if kv == "q8_0" else cw.quantise_row_q4_0)(c[i])
            assert np.array_equal(f16_bits(got["scale"])[page, i][:16], np.asarray(sc, np.float16).view(np.uint16)[:16])
        assert np.array_equal(bits(got["cache"])[page, i][:n].view(np.uint8), np.asarray(code)[:n].view(np.uint8))


def test_append_single_rows(cuda_lib):
    """One token and one head: strides along them say nothing."""
    x = make([1], [130], 1, "q8_0", seed=14)
    d = {k: v.cuda() for k, v in x.items() if torch.is_tensor(v)}
    one = lambda t, *shape: t.as_strided(shape, (0,) * (len(shape) - 1) + (1,), t.storage_offset())
    k_out, q_out = torch.zeros(1, 64, dtype=bf16, device="cuda"), torch.zeros(1, 1, 64, dtype=bf16, device="cuda")
    a = cuda_lib.make_append_args(c=one(d["joint"], 1, 512), k_pe=one(d["joint"][:, 512:], 1, 64), q_pe=one(d["q"], 1, 1, 64),
                                  k_pe_out=one(k_out, 1, 64), q_pe_out=one(q_out, 1, 1, 64), kv_cache=d["cache"],
                                  kv_scale=d["scale"], block_table=d["table"], cu_seqlens=d["cu"], seq_lens=d["lens"])
    ws = cuda_lib.alloc_workspace(a)
    cuda_lib.mla_append_kv(a)
    assert cuda_lib.mla_get_status(ws) == 0
    check(x, dict(cache=d["cache"].cpu(), scale=d["scale"].cpu(), k=k_out.cpu(), q=q_out.cpu()))


@pytest.mark.parametrize("tok,head,H", [
    (64, 64 * 12 + 8, 16),       # heads outermost, a gap between them
    (16 * 64 + 24, 64, 16),      # tokens outermost
    (128, 192, 2),               # each in the other's gaps
    (72, 72 * 12, 5),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_query_outputs_in_any_order(cuda_lib, tok, head, H, in_place):
    """Strides of the rotated queries that leave every head of every token to itself;
    what lies between is not written."""
    x = make([2, 1] if H == 2 else [5, 7], [70, 9], H, "bf16", seed=15)
    n = int(x["cu"][-1])
    want = run(cuda_lib, x)
    d = {k: v.cuda() for k, v in x.items() if torch.is_tensor(v)}
    room = torch.full(((n - 1) * tok + (H - 1) * head + 64,), 7.0, dtype=bf16, device="cuda")
    q_out = room.as_strided((n, H, 64), (tok, head, 1))
    free = torch.ones(room.shape, dtype=torch.bool, device="cuda")
    free.as_strided((n, H, 64), (tok, head, 1)).fill_(False)
    if in_place:
        q_out.copy_(d["q"])
    a = cuda_lib.make_append_args(c=d["joint"][:, :512], k_pe=d["joint"][:, 512:576], q_pe=q_out if in_place else d["q"],
                                  q_pe_out=q_out, kv_cache=d["cache"], kv_scale=None, block_table=d["table"],
                                  cu_seqlens=d["cu"], seq_lens=d["lens"])
    ws = cuda_lib.alloc_workspace(a)
    cuda_lib.mla_append_kv(a)
    assert cuda_lib.mla_get_status(ws) == 0
    assert torch.equal(q_out.cpu(), want["q"]) and bool((room[free] == 7).all())
