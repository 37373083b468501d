"""Random numbers that fall just beside a running sum of the draft verification's
weights: u is fixed in fp32 first, and one probability is then moved until the sum up
to a chosen token is above or below u times the total by some 2^-36 of it, counted in
whole multiples of 2^-149.

The kernel's bound, with u = 2^-24: a lane adds 32 weights whose sum is A.  The rounding
errors of its differences add up to u A at most, those of its 31 additions to 31 u A,
and each is found exactly; joining them rounds some 32 times, each time by at most u of
32 u A: 2^-38 A in all.  So the sum up to a boundary and u_sample times the total are each
within 2^-38 of their value, and the fp64 sums add less than 2^-42 for 1024 segments:
together below 2^-36 of the total.
"""

import numpy as np
import pytest
import torch

from oracle import serving

f32, i32 = torch.float32, torch.int32
UNIT = 2.0 ** 149
DELTA = 1.25 * 2.0 ** -36


def whole(x):
    """fp32 values as whole multiples of 2^-149."""
    return [int(v) for v in np.asarray(x, np.float64) * UNIT]


def sums_of(p, q):
    """Exact running sums of max(p - q, 0)."""
    w = [max(a - b, 0) for a, b in zip(whole(p), whole(q))]
    out, at = [], 0
    for v in w:
        at += v
        out.append(at)
    return w, out


def one_case(rng, V, draft, where, edge, side):
    """(p, q, u, expected token): rows of one sequence, u some `where` of the way; the
    boundary is the last weight of a 1024-token segment (`edge`) or inside one."""
    logits = rng.normal(size=V)
    soft = lambda x: (np.exp(x) / np.exp(x).sum()).astype(np.float32)
    p, q = soft(logits), soft(logits + 0.7 * rng.normal(size=V))
    if not draft:
        q[:] = 0.0
    near = int(where * V)
    i = near // 2                                     # the probability that is moved
    p[i], q[i] = 4e-6, 0.0
    w, sums = sums_of(p, q)
    j = (near // 1024 + 1) * 1024 - 1 if edge else near // 1024 * 1024 + 517
    while w[j] == 0:
        j -= 1
    u = np.float32(sums[j] / sums[-1])
    uf = float(u)
    T = sums[-1] / UNIT
    # 2^26 u is whole: the difference that has to be made up, exactly
    gap = float(np.longdouble(sums[-1] * int(uf * 2 ** 26) - sums[j] * 2 ** 26) / np.longdouble(2) ** 175)
    p[i] = np.float32(float(p[i]) + (gap + side * DELTA * T) / (1 - uf))
    w, sums = sums_of(p, q)
    off = sums[j] * 2 ** 26 - sums[-1] * int(uf * 2 ** 26)
    assert off * side > 0 and 2 ** -36 < abs(off) / (sums[-1] * 2 ** 26) < 2 ** -35
    want = next(k for k, s in enumerate(sums) if s * 2 ** 26 > sums[-1] * int(uf * 2 ** 26))
    after = next(k for k in range(j + 1, V) if w[k] > 0)
    assert want == (j if side > 0 else after)
    assert min(w[j], w[after]) > sums[-1] * 2.0 ** -30 and 0 < uf < 1
    return p, q, u, want


def make(V, seed=1):
    rng = np.random.default_rng(seed)
    cases = [one_case(rng, V, draft, where, edge, side) for draft in (False, True) for where in (0.3, 0.7)
             for edge in (False, True) for side in (1, -1)]
    B = len(cases)
    x = dict(target_probs=torch.zeros(B, 2, V), draft_probs=torch.zeros(B, 1, V), draft_tokens=torch.zeros(B, 1, dtype=i32),
             num_draft=torch.zeros(B, dtype=i32), u_accept=torch.full((B, 1), 1 - 2.0 ** -24), u_sample=torch.zeros(B),
             seq_lens=torch.full((B,), 100, dtype=i32))
    for b, (p, q, u, _) in enumerate(cases):
        x["target_probs"][b, 0] = torch.from_numpy(p)
        x["draft_probs"][b, 0] = torch.from_numpy(q)
        x["u_sample"][b] = float(u)
        x["num_draft"][b] = int(q.any())
        x["draft_tokens"][b, 0] = int(np.argmax(q - p))           # rejected
    return x, np.array([c[3] for c in cases])


@pytest.mark.parametrize("V", [2500, 60000])
def test_boundaries_tell_sums_apart(V):
    """The 64-bit definition is on the right side of every one (its running sums are off by
    less than 2 V 2^-53 < 2^-36 of the total); 32-bit sums are not."""
    x, want = make(V)
    n = lambda k: x[k].numpy()
    tokens, acc, _ = serving.verify_draft(*(n(k) for k in ("target_probs", "draft_probs", "draft_tokens", "num_draft",
                                                           "u_accept", "u_sample", "seq_lens")))
    assert (acc == 0).all() and (tokens[:, 0] == want).all()
    w = np.maximum(n("target_probs")[:, 0] - n("draft_probs")[:, 0], 0)
    low = np.cumsum(w, -1, dtype=np.float32)
    got = [int(np.searchsorted(s, np.float32(u * s[-1]), side="right")) for s, u in zip(low, n("u_sample"))]
    assert (np.array(got) != want).sum() >= 4


@pytest.mark.gpu
@pytest.mark.parametrize("V,copies", [(2500, 1), (60000, 1), (2500, 40), (60000, 4)])
def test_verify_beside_a_boundary(cuda_lib, V, copies):
    """Clusters of eight blocks down to single ones."""
    x, want = make(V)
    d = {k: t.repeat(copies, *([1] * (t.dim() - 1))).cuda() for k, t in x.items()}
    B = want.size * copies
    out = dict(tokens=torch.zeros(B, 2, dtype=i32, device="cuda"), num_accepted=torch.full((B,), 9, dtype=i32, device="cuda"),
               new_lens=torch.zeros(B, dtype=i32, device="cuda"))
    a = cuda_lib.make_verify_args(**d, **out)
    ws = cuda_lib.alloc_workspace(a)
    cuda_lib.mla_verify_draft(a)
    assert cuda_lib.mla_get_status(ws) == 0
    assert (out["num_accepted"] == 0).all()
    np.testing.assert_array_equal(out["tokens"][:, 0].cpu().numpy(), np.tile(want, copies))
    np.testing.assert_array_equal(out["new_lens"].cpu().numpy(), np.tile(100 - x["num_draft"].numpy(), copies))
