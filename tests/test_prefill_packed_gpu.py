"""GPU parity of the packed prompt attention (mla_prefill_packed) against the fp64
oracle.

Tolerances, per row and head, from the exact quantities A = sum_j p_j |v_j| and
S = max_j softmax_scale sum_d |q_d k_jd|: an fp32 score is off by at most
d = 192 2^-23 S (192 products summed in fp32, in any order, and the scale), which
moves every p_j by the factor exp(2 d) at most, some 2.1 d of it; the exponential itself is off
by at most 2^-16 of its value; p is rounded to bf16 for the product with v (2^-8 of
it) and the output to bf16 (2^-8 of it).  So |o| is off by at most
(2^-8 + 2.1 d + 2^-15) A + 2^-8 |o|, and lse by d + 2^-15 + 2^-21 |lse|.
"""

import numpy as np
import pytest
import torch

from mla_inputs import bf16_bits
from oracle import mla_oracle as om
from oracle import serving

from parity_util import to_np

pytestmark = pytest.mark.gpu

bf16, i32 = torch.bfloat16, torch.int32


def make(lens, H, H_kv, d_r, seed=1, head=0, tail=0, fused=True, gain=1.0):
    """Packed inputs on the GPU; `fused`: views of the projections' outputs."""
    g = torch.Generator().manual_seed(seed)
    n = head + sum(lens) + tail
    r = lambda *s: (torch.randn(*s, generator=g) * gain).to(bf16).cuda()
    if fused and d_r:
        q, kv, lat = r(n, H, 192), r(n, H_kv, 256), r(n, 576)
        x = dict(q_nope=q[..., :128], q_pe=q[..., 128:], k_nope=kv[..., :128], k_pe=lat[:, 512:], v=kv[..., 128:])
    elif fused:
        t = r(n, H + 2 * H_kv, 128)
        x = dict(q_nope=t[:, :H], q_pe=None, k_nope=t[:, H:H + H_kv], k_pe=None, v=t[:, H + H_kv:])
    else:
        # heads outermost
        x = dict(q_nope=r(H, n, 128).transpose(0, 1), q_pe=r(H, n, d_r).transpose(0, 1) if d_r else None,
                 k_nope=r(H_kv, n, 128).transpose(0, 1), k_pe=r(n, d_r) if d_r else None,
                 v=r(H_kv, n, 128).transpose(0, 1))
    x["cu_seqlens"] = torch.tensor([head] + list(head + np.cumsum(lens)), dtype=i32).cuda()
    x["out"] = torch.full((n, H, 128), 7.0, dtype=bf16, device="cuda")
    x["lse"] = torch.full((n, H), 7.0, device="cuda")
    return x


def run(mla, x, causal=True, scale=None, stream=None):
    scale = scale or 1.0 / (192 if x["q_pe"] is not None else 128) ** 0.5
    a = mla.make_prefill_packed_args(**x, causal=causal, softmax_scale=scale)
    ws = mla.alloc_workspace(a)
    mla.mla_prefill_packed(a, stream)
    status = mla.mla_get_status(ws, stream)
    torch.cuda.synchronize()
    return status


def f64(t):
    return om.bf16_to_f64(bf16_bits(t.cpu().contiguous()))


def oracle_of(x, causal, scale=None):
    q, k, v = f64(x["q_nope"]), f64(x["k_nope"]), f64(x["v"])
    scale = scale or 1.0 / (192 if x["q_pe"] is not None else 128) ** 0.5
    if x["q_pe"] is not None:
        q = np.concatenate([q, f64(x["q_pe"])], -1)
        k = np.concatenate([k, np.repeat(f64(x["k_pe"])[:, None], k.shape[1], 1)], -1)
    return serving.attend_packed(q, k, v, x["cu_seqlens"].cpu().numpy(), scale, causal)


def check(x, ref, rows=None):
    o, lse, mass, size = ref
    got, got_lse = to_np(x["out"]), to_np(x["lse"])
    real = ~np.isnan(lse[:, 0]) if rows is None else rows
    d = 192 * 2.0 ** -23 * size[real]
    off = np.abs(got[real] - o[real])
    tol = (2.0 ** -8 + 2.1 * d + 2.0 ** -15)[..., None] * mass[real] + 2.0 ** -8 * np.abs(o[real])
    assert (off <= tol).all(), (float((off / np.maximum(tol, 1e-30)).max()), np.argwhere(off > tol)[:3])
    off = np.abs(got_lse[real] - lse[real])
    assert (off <= d + 2.0 ** -15 + 2.0 ** -21 * np.abs(lse[real])).all(), float(off.max())


def untouched(x):
    cu = x["cu_seqlens"].tolist()
    for t in (x["out"], x["lse"]):
        assert bool((t[:cu[0]] == 7).all()) and bool((t[cu[-1]:] == 7).all())


CASES = [
    # lens, H, H_kv, d_r, extra
    ([1], 1, 1, 64, {}),
    ([1], 16, 2, 0, {}),
    ([17], 16, 16, 64, {}),
    ([1, 0, 2, 0, 0, 5], 4, 4, 64, dict(head=3, tail=4)),            # empty sequences, rows of none
    ([127, 128, 129], 2, 2, 64, {}),                                 # about a key tile
    ([255, 256, 257], 2, 1, 0, dict(tail=1)),                        # about a query block
    ([3, 130, 300, 64, 1, 200], 4, 4, 64, {}),                       # boundaries inside tiles
    ([3, 130, 300, 64, 1, 200], 8, 2, 0, dict(fused=False)),         # grouped, heads outermost
    ([600], 3, 3, 64, dict(fused=False)),                            # an odd number of heads
    ([512], 6, 2, 64, {}),                                           # grouped heads with the shared key
    ([40] * 30, 2, 2, 64, dict(tail=9)),                             # many sequences in a tile
    ([1] * 300, 1, 1, 0, {}),                                        # one token each
    ([200, 77], 2, 2, 64, dict(gain=6.0)),                           # peaked softmax, large scores
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,H_kv,d_r,kw", CASES)
def test_packed_matches_oracle(cuda_lib, lens, H, H_kv, d_r, kw, causal):
    x = make(lens, H, H_kv, d_r, **kw)
    assert run(cuda_lib, x, causal) == 0
    check(x, oracle_of(x, causal))
    untouched(x)


def test_packed_long_sampled(cuda_lib):
    """A long prompt between short ones: sampled rows against the definition."""
    x = make([5, 5000, 300], 4, 2, 64, seed=3)
    assert run(cuda_lib, x) == 0
    check_rows(x, [4, 5, 132, 133, 1000, 2600, 4999, 5004, 5005, 5304])


@pytest.mark.parametrize("causal", [True, False])
def test_packed_more_blocks_than_the_gpu_holds(cuda_lib, causal):
    """Blocks in order of their work, several to an SM, an odd number of heads."""
    x = make([500, 3, 0, 130, 256, 340], 41, 41, 64, seed=11, tail=2)
    assert run(cuda_lib, x, causal) == 0
    check(x, oracle_of(x, causal))
    untouched(x)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,H_kv,d_r,kw", [
    ([127, 128, 129], 80, 80, 64, {}),
    ([255, 256, 257], 52, 4, 0, dict(tail=1)),
    ([3, 130, 300, 64, 1, 200], 52, 13, 64, dict(fused=False)),
    ([40] * 14, 60, 60, 0, dict(head=2, tail=9)),
    ([200, 177], 76, 38, 64, dict(gain=6.0)),
])
def test_packed_grids_that_fill_the_gpu(cuda_lib, lens, H, H_kv, d_r, kw, causal):
    """More (block, head) pairs than multiprocessors, of few rows each."""
    x = make(lens, H, H_kv, d_r, **kw)
    assert run(cuda_lib, x, causal) == 0
    check(x, oracle_of(x, causal))
    untouched(x)


def test_packed_more_rows_than_are_sorted(cuda_lib):
    """More than 128 blocks of rows: taken from the end on."""
    x = make([20000, 13800, 1, 700], 4, 1, 0, seed=12)
    assert run(cuda_lib, x) == 0
    check_rows(x, [0, 127, 4097, 12345, 19999, 20000, 20128, 33799, 33800, 33801, 34500])


def test_packed_offsets_beyond_32_bits(cuda_lib):
    """More than 2^31 query and output values."""
    n, H = 132000, 128                       # 2.16e9 values each
    lens = [250] * (n // 250)
    q = torch.zeros(n, H, 128, dtype=bf16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(13)
    q[-250:] = torch.randn(250, H, 128, generator=g, device="cuda").to(bf16)
    k, v = (torch.randn(n, 1, 128, generator=g, device="cuda").to(bf16) for _ in range(2))
    x = dict(q_nope=q, q_pe=None, k_nope=k, k_pe=None, v=v, cu_seqlens=torch.tensor([0] + list(np.cumsum(lens)), dtype=i32).cuda(),
             out=torch.empty(n, H, 128, dtype=bf16, device="cuda"), lse=torch.empty(n, H, device="cuda"))
    assert run(cuda_lib, x) == 0
    check_rows(x, [250, 131071, n - 250, n - 1])


def test_packed_scores_that_keep_rising(cuda_lib):
    """Scores that rise along the prompt by less than, about and far more than the range
    that the running reference leaves open, and one that falls."""
    for steps, H in ((0.02, 2), (0.2, 2), (2.0, 2), (-0.2, 2), (0.2, 54), (2.0, 54)):
        x = make([700], H, 1, 0, seed=14)
        x["q_nope"].zero_()
        x["k_nope"].zero_()
        x["q_nope"][:, :, 0] = 128 ** 0.5                       # the score is k's first value
        x["k_nope"][:, 0, 0] = (torch.arange(700, device="cuda") * steps).to(bf16)
        assert run(cuda_lib, x) == 0
        check(x, oracle_of(x, True))
    # one key far above all before it, and a far higher one in the same tile
    x["k_nope"].zero_()
    x["k_nope"][300, 0, 0] = 90.0
    x["k_nope"][333, 0, 0] = 1000.0
    x["k_nope"][650, 0, 0] = 1100.0
    assert run(cuda_lib, x) == 0
    check(x, oracle_of(x, True))


def test_packed_nothing_to_do(cuda_lib):
    """Rows, but no sequence with any."""
    x = make([0, 0, 0], 4, 4, 64, seed=15, tail=300)
    assert run(cuda_lib, x) == 0
    untouched(x)


def test_packed_wait_that_runs_out(cuda_lib):
    """At a limit of 1 ns the kernel gives up, says so and leaves the context usable."""
    x = make([300, 100], 16, 16, 64, seed=16)
    cuda_lib.mla_set_device_wait_limit(1)
    try:
        assert run(cuda_lib, x) == 6
    finally:
        cuda_lib.mla_set_device_wait_limit(0)
    assert run(cuda_lib, x) == 0
    check(x, oracle_of(x, True))


def test_packed_two_streams_at_once(cuda_lib):
    """Calls that overlap share nothing."""
    xs = [make([400, 300], 32, 32, 64, seed=17 + i) for i in range(2)]
    args = [cuda_lib.make_prefill_packed_args(**x, causal=True, softmax_scale=1 / 192 ** 0.5) for x in xs]
    ws = cuda_lib.alloc_workspace(args[0])
    args[1].workspace, args[1].workspace_bytes = args[0].workspace, args[0].workspace_bytes
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in zip(args, streams):
            cuda_lib.mla_prefill_packed(a, s)
    torch.cuda.synchronize()
    assert cuda_lib.mla_get_status(ws) == 0
    for x in xs:
        first, lse = x["out"].clone(), x["lse"].clone()
        x["out"].fill_(7)
        assert run(cuda_lib, x) == 0
        assert torch.equal(first, x["out"]) and torch.equal(lse, x["lse"])


def one_row(q, k, v):
    """The last row of a causal prompt: q [H][d], k and v [keys][H_kv][..]."""
    q, k, v = f64(q), f64(k), f64(v)
    share, scale = q.shape[0] // k.shape[1], q.shape[1] ** -0.5
    out = []
    for h in range(q.shape[0]):
        kk, vv = k[:, h // share], v[:, h // share]
        s = kk @ q[h] * scale
        p = np.exp(s - s.max())
        out.append(((p / p.sum()) @ vv, s.max() + np.log(p.sum()), (p / p.sum()) @ np.abs(vv),
                    (np.abs(kk) @ np.abs(q[h])).max() * scale))
    return [np.stack([o[i] for o in out])[None] for i in range(4)]


def check_rows(x, rows):
    """These rows of a causal batch against the definition."""
    cu = x["cu_seqlens"].tolist()
    for t in rows:
        lo = max(c for c in cu if c <= t)
        q, k = x["q_nope"][t], x["k_nope"][lo:t + 1]
        if x["q_pe"] is not None:
            q = torch.cat([q, x["q_pe"][t]], -1)
            k = torch.cat([k, x["k_pe"][lo:t + 1, None].expand(-1, k.shape[1], -1)], -1)
        o, lse, mass, size = one_row(q, k, x["v"][lo:t + 1])
        part = dict(out=x["out"][t:t + 1], lse=x["lse"][t:t + 1])
        check(part, (o, lse, mass, size))


@pytest.mark.parametrize("H", [2, 80])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_packed_unseen_values_have_no_effect(cuda_lib, bad, H):
    """NaN and infinities in tokens that a row does not see: later tokens of its
    prompt, other prompts, rows of no prompt.  Rows that see them are not compared."""
    lens = [130, 90, 200]
    x = make(lens, H, H, 64, seed=4, head=1, tail=30)
    ref = oracle_of(x, True)
    spoilt = [0, 100, 131, 220, 400, 421, 425, 450]
    for t in spoilt:
        for name in ("k_nope", "k_pe", "v"):
            x[name][t] = bad
    x["q_nope"][425:] = bad
    assert run(cuda_lib, x) == 0
    cu = [1, 131, 221, 421]
    good = np.zeros(sum(lens) + 31, bool)
    for lo, hi in zip(cu, cu[1:]):
        stop = min([t for t in spoilt if lo <= t < hi] + [hi])
        good[lo:stop] = True
    check(x, ref, good)
    untouched(x)
    # rows that see one hold what the definition gives there: not a number for NaN
    if bad != bad:
        assert bool(torch.isnan(x["out"][100]).all()) and bool(torch.isnan(x["out"][130]).all())


def test_packed_one_bad_query_stays_alone(cuda_lib):
    x = make([300], 2, 2, 64, seed=5)
    ref = oracle_of(x, True)
    x["q_nope"][77] = float("nan")
    assert run(cuda_lib, x) == 0
    good = np.ones(300, bool)
    good[77] = False
    check(x, ref, good)
    assert bool(torch.isnan(x["out"][77]).all())


def test_packed_all_scores_minus_infinity(cuda_lib):
    """A row whose every score is -inf weighs nothing: zeros and lse = -inf."""
    x = make([3], 2, 2, 0, seed=6)
    x["q_nope"].fill_(1.0)
    x["k_nope"].fill_(1.0)
    x["k_nope"][0, :, 0] = -float("inf")
    assert run(cuda_lib, x) == 0
    assert bool((x["out"][0] == 0).all()) and bool(torch.isneginf(x["lse"][0]).all())
    assert bool(torch.isfinite(x["lse"][1:]).all())


def test_packed_without_lse_repeats_and_replays(cuda_lib):
    """Bit-identical again, on another stream, and replayed from a graph with other
    offsets in place."""
    x = make([100, 300, 57], 4, 4, 64, seed=7)
    assert run(cuda_lib, x) == 0
    first, lse = x["out"].clone(), x["lse"].clone()
    x["out"].fill_(7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert run(cuda_lib, x, stream=s) == 0
    assert torch.equal(first, x["out"]) and torch.equal(lse, x["lse"])
    x["lse"] = None
    x["out"].fill_(7)
    a = cuda_lib.make_prefill_packed_args(**x, causal=True, softmax_scale=1 / 192 ** 0.5)
    ws = cuda_lib.alloc_workspace(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.mla_prefill_packed(a)
    g.replay()
    assert cuda_lib.mla_get_status(ws) == 0 and torch.equal(first, x["out"])
    x["cu_seqlens"][1] = 40
    g.replay()
    assert cuda_lib.mla_get_status(ws) == 0
    got = x["out"].clone()
    x["lse"] = torch.empty(457, 4, device="cuda")
    assert run(cuda_lib, x) == 0
    assert torch.equal(got, x["out"])


def test_packed_bad_offsets_are_reported(cuda_lib):
    x = make([50, 50], 2, 2, 64, seed=8)
    x["cu_seqlens"][1] = 120
    assert run(cuda_lib, x) == 8


def test_packed_prefill_agrees_with_the_cached_form(cuda_lib):
    """Prompts appended to the cache and attended there in the explicit form give what
    the packed attention gives on the same up-projected keys and values."""
    from head_latent_attention_06_b200.step import PackedPrefill, PrefillStep
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g)
    L, B, H = 192, 2, 16
    n = B * L
    latent = r(n, 576).to(bf16).cuda()
    q = r(n, H, 192).to(bf16).cuda()
    w_uk, w_uv = ((r(H, 128, 512) / 512 ** 0.5).to(bf16).cuda() for _ in range(2))
    c = latent[:, :512].double()
    kv = torch.cat([torch.einsum("tc,hnc->thn", c, w.double()) for w in (w_uk, w_uv)], -1).to(bf16)
    cache = torch.zeros(8, 64, 576, dtype=bf16, device="cuda")
    table = torch.tensor([[5, 0, 3], [1, 7, 2]], dtype=i32, device="cuda")
    lens = torch.tensor([L, L], dtype=i32, device="cuda")
    cu = torch.tensor([0, L, 2 * L], dtype=i32, device="cuda")
    scale = 1 / 192 ** 0.5
    step = PackedPrefill(q=q, kv=kv, latent=latent, kv_cache=cache, kv_scale=None, block_table=table, cu_seqlens=cu,
                         seq_lens=lens, softmax_scale=scale)
    step.run()
    assert cuda_lib.mla_get_status(step.workspace) == 0 and cuda_lib.mla_get_status(step.append_workspace) == 0
    ref = PrefillStep(q_nope=q[..., :128].reshape(B, L, H, 128).contiguous(), q_pe=step.q_pe.view(B, L, H, 64), w_uk=w_uk,
                      w_uv=w_uv, kv_cache=cache, block_table=table, seq_lens=lens, causal=True, softmax_scale=scale,
                      max_seq_len=L)
    ref.run()
    assert cuda_lib.mla_get_status(ref.workspace) == 0
    x = dict(q_nope=q[..., :128], q_pe=step.q_pe, k_nope=kv[..., :128], k_pe=step.k_pe, v=kv[..., 128:], cu_seqlens=cu,
             out=step.out, lse=step.lse)
    want = oracle_of(x, True)
    check(x, want)
    # the cached form rounds the same keys and values from fp32 sums: a whole bf16 step
    # (2^-7) where the sum falls the other way, in a score and in v, besides each side's
    # own tolerance
    d = 192 * 2.0 ** -23 * want[3] + 2.0 ** -7 * want[3]
    tol = 2 * ((2.0 ** -8 + 2.1 * d + 2.0 ** -15)[..., None] * want[2] + 2.0 ** -8 * np.abs(want[0])) + 2.0 ** -7 * want[2]
    assert (np.abs(to_np(step.out) - to_np(ref.out).reshape(n, H, 128)) <= tol).all()


def test_packed_output_at_16_bytes_and_single_rows(cuda_lib):
    """An output that starts 16 bytes into a sector; inputs of one row and one head whose
    strides along those say nothing."""
    x = make([300, 20], 5, 5, 64, seed=18)
    want = oracle_of(x, True)
    room = torch.full((320 * 5 * 128 + 16,), 7.0, dtype=bf16, device="cuda")
    x["out"] = room[8:8 + 320 * 5 * 128].view(320, 5, 128)
    assert x["out"].data_ptr() % 32 == 16
    assert run(cuda_lib, x) == 0
    check(x, want)
    assert bool((room[:8] == 7).all()) and bool((room[-8:] == 7).all())
    x = make([1], 1, 1, 64, seed=19)
    want = oracle_of(x, True)
    for name in ("q_nope", "q_pe", "k_nope", "v"):
        x[name] = x[name].as_strided(x[name].shape, (0, 0, 1), x[name].storage_offset())
    x["k_pe"] = x["k_pe"].as_strided((1, 64), (0, 1), x["k_pe"].storage_offset())
    assert run(cuda_lib, x) == 0
    check(x, want)


def top_residues(x, causal):
    """Per row and head of a batch whose values are the same along a query and along a key
    (shared by all heads, d_r = 0): how far the top score, times the scale in base 2, lies
    above its own rounding to fp32."""
    a, b = x["q_nope"][..., 0].double().cpu().numpy(), x["k_nope"][:, 0, 0].double().cpu().numpy()
    scale2 = np.float32(np.float32(1 / 128 ** 0.5) * np.float32(1.4426950408889634))
    res = np.zeros(a.shape)
    cu = x["cu_seqlens"].tolist()
    for lo, hi in zip(cu, cu[1:]):
        for t in range(lo, hi):
            keys = b[lo:t + 1 if causal else hi]
            s = 128 * np.where(a[t] > 0, a[t] * keys.max(), a[t] * keys.min())
            exact = s * float(scale2)                  # 24 and 23 bits: exact in 64
            res[t] = exact - exact.astype(np.float32)
    return res


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("small", [1.0, 2.0 ** -90])
def test_packed_scores_beyond_the_exponent_range(cuda_lib, small, causal):
    """Finite scores so large (some 2^26 to 2^37) that their rounding to fp32 takes away or
    adds more than the range of an exponential: the top key alone has weight, or the keys
    that share the top score, for every row, of one key tile or several.

    A score is 128 equal products of 8-bit by 8-bit significands: exact in fp32 whatever the
    order.  Two that differ do so by at least 200 2^7 128 / sqrt(128) > 10^5, so all other
    weights are zero in 64 bits too and the top ones equal; their sum with v and its
    quotient by their number take some eight fp32 roundings (2^-20) of the mean |v|, the output half
    a bf16 step (2^-8).  Where the reference's rounding is small the top weight is 2^r for the
    residue r, no power of two, and is rounded to bf16 for the product with v while the sum that
    divides it is not: another 2^-8 of the mean |v|.  lse: the scale's, the logarithm base's and the score's roundings,
    seven of 2^-24, below 2^-21 of it."""
    g = torch.Generator().manual_seed(20)
    lens, H = [700, 90, 1], 3
    x = make(lens, H, 1, 0, seed=20)
    n = sum(lens)
    sign = torch.where(torch.rand(n, H, generator=g) < 0.3, -1.0, 1.0)
    x["q_nope"] = (200 * 500 ** torch.rand(n, H, generator=g) * sign).to(bf16).cuda()[..., None].repeat(1, 1, 128)
    x["k_nope"] = (2e4 + 8e4 * torch.rand(n, 1, generator=g)).to(bf16).cuda()[..., None].repeat(1, 1, 128)
    x["v"] = x["v"] * small
    res = top_residues(x, causal)
    assert (res < -126).sum() > 20 and (res > 60).sum() > 20 and ((res > -126) & (res < -8)).sum() > 20 and (np.abs(res) < 8).sum() > 20
    assert run(cuda_lib, x, causal) == 0
    o, lse, mass, _ = oracle_of(x, causal)
    assert (np.abs(to_np(x["out"]) - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -20) * mass).all()
    assert (np.abs(to_np(x["lse"]) - lse) <= 2.0 ** -21 * np.abs(lse)).all()


def test_packed_rows_done_over_outlast_the_wait_limit(cuda_lib):
    """A prompt whose every row sees a NaN is done over by single warps, 32 rows of up to
    16000 keys each, far longer than the limit set here, while the block's other warps
    wait: that is progress, not a wait that ran out.  The prompt beside it comes out
    right."""
    lens = [200, 16000]
    x = make(lens, 10, 10, 64, seed=21)
    ref_rows = [0, 57, 199]
    x["k_nope"][200] = float("nan")
    cuda_lib.mla_set_device_wait_limit(5_000_000)
    try:
        assert run(cuda_lib, x) == 0
    finally:
        cuda_lib.mla_set_device_wait_limit(0)
    check_rows(x, ref_rows)
    assert bool(torch.isnan(x["out"][200:]).all())
