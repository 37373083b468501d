"""GPU parity of the draft verification (mla_verify_draft) against the fp64 oracle:
all results are whole numbers and have to be equal.  The oracle sums in another
order than the kernel, which is within 2^-38 of the exact sum: 32 differences carry their
errors, each below 2^-24 of the sum, and joining the 32 errors costs at most 32 roundings of
2^-24 of 33 such errors.  A random u_sample falls between the two sums of some
token with a chance below V 2^-38: below 10^-3 over the some 10^7 values here."""

import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu

f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


def make(B, S, V, dtype=f32, seed=1, ragged=False, sharp=2.5, noise=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, S + 1, V, generator=g)
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :S] + noise * torch.randn(B, S, V, generator=g), -1).to(dtype)
    draft = torch.stack([torch.multinomial(q[b].float(), 1, generator=g)[:, 0] for b in range(B)]) if S else torch.zeros(B, 0)
    num = torch.randint(0, S + 1, (B,), generator=g) if ragged else torch.full((B,), S)
    return dict(target_probs=p, draft_probs=q, draft_tokens=draft.to(i32), num_draft=num.to(i32),
                u_accept=torch.rand(B, S, generator=g), u_sample=torch.rand(B, generator=g),
                seq_lens=torch.randint(S + 1, 5000, (B,), generator=g).to(i32))


def run(mla, x, in_place=False, stream=None, **kw):
    d = {k: None if v is None else v.cuda() for k, v in x.items()}
    d.update(kw)
    B, s_q, _ = d["target_probs"].shape
    tokens = torch.full((B, s_q), 55, dtype=i32, device="cuda")
    acc = torch.full((B,), 55, dtype=i32, device="cuda")
    new = d["seq_lens"] if in_place else torch.full((B,), 55, dtype=i32, device="cuda")
    a = mla.make_verify_args(**d, tokens=tokens, num_accepted=acc, new_lens=new)
    ws = mla.alloc_workspace(a)
    mla.mla_verify_draft(a, stream)
    status = mla.mla_get_status(ws, stream)
    torch.cuda.synchronize()
    return status, tokens.cpu().numpy(), acc.cpu().numpy(), new.cpu().numpy()


def oracle_of(x):
    n = lambda t: None if t is None else t.float().numpy() if t.is_floating_point() else t.numpy()
    S = x["target_probs"].shape[1] - 1
    num = x["num_draft"] if x["num_draft"] is not None else torch.full((x["target_probs"].shape[0],), S)
    return serving.verify_draft(n(x["target_probs"]), n(x["draft_probs"]), n(x["draft_tokens"]), n(num), n(x["u_accept"]),
                                n(x["u_sample"]), n(x["seq_lens"]))


def check(got, want):
    status, tokens, acc, new = got
    assert status == 0
    np.testing.assert_array_equal(acc, want[1])
    np.testing.assert_array_equal(tokens, want[0])
    np.testing.assert_array_equal(new, want[2])


@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("B,S,V,ragged", [
    (1, 0, 1, False), (1, 1, 2, False), (3, 2, 7, True), (5, 4, 31, True), (2, 3, 1000, False), (4, 3, 1024, True),
    (4, 3, 1025, True), (3, 5, 8191, True), (2, 2, 8193, False), (9, 4, 32000, True), (3, 7, 100003, True),
    (2, 1, 1 << 20, False), (130, 3, 2049, True), (2, 1023, 65, True), (40, 8, 16, True), (700, 2, 3000, True), (300, 1, 9000, False),
])
def test_verify_matches_oracle(cuda_lib, B, S, V, ragged, dtype):
    x = make(B, S, V, dtype, seed=B + S + V, ragged=ragged)
    check(run(cuda_lib, x), oracle_of(x))


def test_verify_follows_the_target_distribution(cuda_lib):
    """The first token of many verifications with one draft is distributed as the
    target: each token's share within 5 standard deviations."""
    V, N = 8, 40000
    g = torch.Generator().manual_seed(12)
    p = torch.softmax(torch.randn(V, generator=g), -1)
    q = torch.softmax(torch.randn(V, generator=g), -1)
    x = dict(target_probs=p.expand(N, 2, V), draft_probs=q.expand(N, 1, V),
             draft_tokens=torch.multinomial(q.expand(N, V), 1, generator=g).to(i32), num_draft=None,
             u_accept=torch.rand(N, 1, generator=g), u_sample=torch.rand(N, generator=g),
             seq_lens=torch.full((N,), 9, dtype=i32))
    status, tokens, acc, new = run(cuda_lib, x)
    assert status == 0
    share = np.bincount(tokens[:, 0], minlength=V) / N
    sd = np.sqrt(p.numpy() * (1 - p.numpy()) / N)
    assert (np.abs(share - p.numpy()) <= 5 * sd).all()
    np.testing.assert_array_equal(new, 9 - (1 - acc))


@pytest.mark.parametrize("in_place", [False, True])
def test_verify_certain_drafts_views_and_in_place(cuda_lib, in_place):
    """Drafts without probabilities, probabilities as views of a wider array at an
    odd offset, lengths written over themselves."""
    x = make(6, 3, 500, seed=3, sharp=6.0)
    x["draft_probs"] = None
    x["draft_tokens"] = x["target_probs"][:, :3].argmax(-1).to(i32)
    x["num_draft"] = None
    wide = torch.zeros(6, 5, 517)
    wide[:, :4, 3:503] = x["target_probs"]
    want = oracle_of(x)
    check(run(cuda_lib, x, in_place, target_probs=wide.cuda()[:, :4, 3:503]), want)
    assert 0 < want[1].sum() < 18          # some accepted, some not


def test_verify_edges(cuda_lib):
    """u at its ends, equal distributions, a draft above the target everywhere, zero
    probabilities, all accepted, none drafted."""
    V = 3000
    x = make(8, 2, V, seed=4)
    x["num_draft"] = torch.tensor([2, 2, 2, 2, 2, 0, 1, 2], dtype=i32)
    top = 1 - 2.0 ** -24
    x["u_sample"] = torch.tensor([0.0, top, 0.5, 0.0, top, 0.0, top, 0.3])
    x["draft_probs"][2] = x["target_probs"][2, :2]                # equal: always accepted for u < 1
    x["u_accept"][2] = top
    x["draft_probs"][3] = x["target_probs"][3, :2] + 0.5          # nothing left: the target itself
    x["u_accept"][3] = top
    x["target_probs"][4, 0, : V // 2] = 0.0                       # zeros in front and behind
    x["target_probs"][4, 0, V // 2 + 5:] = 0.0
    x["u_accept"][4] = top
    x["target_probs"][7, 0] = 0.0                                 # nothing at all: rejected, no token
    want = oracle_of(x)
    check(run(cuda_lib, x), want)
    assert want[1][2] == 2 and want[1][3] == 0 and want[0][7, 0] == -1
    assert V // 2 <= want[0][4, 0] < V // 2 + 5


def test_verify_truncated_distributions(cuda_lib):
    """Only a few tokens have any probability (a cut to the likeliest): whole segments
    of zeros, drafts outside the target's set, sets that are the same."""
    x = make(12, 3, 20000, seed=9, ragged=True)
    for name, cut in (("target_probs", 40), ("draft_probs", 60)):
        t = x[name]
        low = t.topk(cut, -1).values[..., -1:]
        t[t < low] = 0.0
        t /= t.sum(-1, keepdim=True)
    x["draft_probs"][:4] = x["target_probs"][:4, :3]
    x["u_accept"][:4] = 1 - 2.0 ** -24
    g = torch.Generator().manual_seed(10)
    x["draft_tokens"] = torch.stack([torch.multinomial(q, 1, generator=g)[:, 0] for q in x["draft_probs"]]).to(i32)
    check(run(cuda_lib, x), oracle_of(x))


def test_verify_close_boundaries(cuda_lib):
    """u_sample a hair on either side of a running sum: what 32-bit sums would miss."""
    V = 60000
    x = make(2, 0, V, seed=11, sharp=0.5)
    p = x["target_probs"][:, 0].double().numpy()
    sums = np.cumsum(p, -1)
    j = 41234
    for b, eps in ((0, 1e-6), (1, -1e-6)):
        edge = (sums[b, j] + eps * p[b, j]) / sums[b, -1]
        u = np.float32(edge)
        x["u_sample"][b] = float(u)
    check(run(cuda_lib, x), oracle_of(x))


def test_verify_not_a_number(cuda_lib):
    """NaN weighs nothing, an infinite sum gives no token; other sequences are as ever."""
    x = make(4, 1, 2000, seed=5)
    want = oracle_of(x)
    x["target_probs"][1] = float("nan")
    x["target_probs"][2, :, 7] = float("inf")
    x["draft_tokens"][2] = 3
    x["u_accept"][2] = 0.999
    x["draft_probs"][2, 0, 3] = 1.0
    x["target_probs"][2, 0, 3] = 0.0
    status, tokens, acc, new = run(cuda_lib, x)
    assert status == 0 and tokens[1, 0] == -1 and acc[1] == 0 and tokens[2, 0] == -1 and acc[2] == 0
    for b in (0, 3):
        np.testing.assert_array_equal(tokens[b], want[0][b])
        assert acc[b] == want[1][b] and new[b] == want[2][b]


@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("V", [1, 50, 1024, 1100, 40000])
def test_verify_outside_the_range_of_probabilities(cuda_lib, V, dtype):
    """Values below zero count as zero on both sides, infinities and NaN among them:
    rows that are all negative, a few of them, a draft row of infinities, of NaN."""
    x = make(8, 1, V, dtype, seed=14)
    x["u_accept"][:] = 1 - 2.0 ** -24
    x["target_probs"][0] = -0.1
    x["draft_probs"][0] = -0.2
    x["target_probs"][1] *= -1
    x["draft_probs"][1] *= -2
    x["target_probs"][2, :, ::2] *= -1
    x["draft_probs"][2, :, ::3] *= -1
    x["draft_probs"][3] *= -1
    x["draft_probs"][4] = float("inf")
    x["draft_probs"][5] = float("nan")
    x["draft_probs"][6, :, ::5] = -float("inf")
    x["target_probs"][6, :, ::7] = -float("inf")
    x["target_probs"][7, :, V // 2] = float("inf")
    x["draft_probs"][7] = float("inf")
    at = x["draft_tokens"][:4, 0].long()
    x["draft_probs"][torch.arange(4), 0, at] = 2.0                                 # rejected
    want = oracle_of(x)
    check(run(cuda_lib, x), want)
    assert (want[1][[0, 1, 2, 3, 4, 5, 7]] == 0).all() and (want[0][[0, 1, 7], 0] == -1).all()


@pytest.mark.parametrize("field,value,code", [("draft_tokens", 2000, 9), ("draft_tokens", -1, 9), ("num_draft", 3, 8),
                                              ("num_draft", -1, 8)])
def test_verify_reports_bad_arguments(cuda_lib, field, value, code):
    x = make(3, 2, 2000, seed=6)
    want = oracle_of(x)
    if field == "num_draft":
        x[field][1] = value
    else:
        x[field][1, 1] = value
    status, tokens, acc, new = run(cuda_lib, x)
    assert status == code
    assert (tokens[1] == -1).all() and acc[1] == 0 and new[1] == int(x["seq_lens"][1])
    for b in (0, 2):
        np.testing.assert_array_equal(tokens[b], want[0][b])
    # a draft behind num_draft is not looked at
    if field == "draft_tokens":
        x["num_draft"][1] = 1
        assert run(cuda_lib, x)[0] == 0


@pytest.mark.parametrize("V", [9000, 100003])
def test_verify_bad_sequences_among_clusters(cuda_lib, V):
    """Sequences that end early beside others whose blocks share their sums, many times over."""
    x = make(24, 2, V, seed=13, ragged=True)
    x["num_draft"][3::4] = 2
    want = oracle_of(x)
    x["num_draft"][1::4] = torch.tensor([3, -1, 3, -7, 9, 3], dtype=i32)
    x["draft_tokens"][3::4, 0] = torch.tensor([V, -1, V + 9, -5, 2 ** 30, V], dtype=i32)
    for _ in range(20):
        status, tokens, acc, new = run(cuda_lib, x)
        assert status in (8, 9)
        assert (tokens[1::2] == -1).all() and (acc[1::2] == 0).all()
        np.testing.assert_array_equal(new[1::2], x["seq_lens"][1::2].numpy())
        for got, ref in ((tokens, want[0]), (acc, want[1]), (new, want[2])):
            np.testing.assert_array_equal(got[::2], ref[::2])


def test_verify_on_another_stream_and_in_a_graph(cuda_lib):
    x = make(5, 3, 9000, seed=7, ragged=True)
    want = oracle_of(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(run(cuda_lib, x, stream=s), want)
    d = {k: v.cuda() for k, v in x.items()}
    out = dict(tokens=torch.zeros(5, 4, dtype=i32, device="cuda"), num_accepted=torch.zeros(5, dtype=i32, device="cuda"),
               new_lens=torch.zeros(5, dtype=i32, device="cuda"))
    a = cuda_lib.make_verify_args(**d, **out)
    ws = cuda_lib.alloc_workspace(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.mla_verify_draft(a)
    y = make(5, 3, 9000, seed=8, ragged=True)
    for k, v in y.items():
        d[k].copy_(v)
    g.replay()
    status = cuda_lib.mla_get_status(ws)
    check((status, *(t.cpu().numpy() for t in out.values())), oracle_of(y))
