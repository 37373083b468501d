"""Cases that time the serving operators around the attention: appending packed
tokens to the paged latent cache with the position rotation on the way
(``mla_append_kv``), causal attention over packed prompts in the explicit form
(``mla_prefill_packed``) and the verification of drafted tokens
(``mla_verify_draft``).

``run`` computes them from elementary torch operations where ``own`` is false and
through the framework's entry points where it is true; both read the same inputs.
"""

import math
import random

import numpy as np
import torch

own = False

D_C, D_R, D_N, D_V, PAGE, BLOCK = 512, 64, 128, 128, 64, 32
ROW = D_C + D_R
ROPE_BASE = 10000.0
ROW_BYTES = {"bf16": 2 * ROW, "e4m3": ROW + 4, "q8_0": ROW + 2 * (ROW // BLOCK), "q4_0": ROW // 2 + 2 * (ROW // BLOCK)}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence, one new token: the smallest append of a decode step (4-bit cache)
        dict(name="append-one-q4", op="append", B=1, new=1, ragged=False, ctx=256, H=16, kv="q4_0", tail=0),
        # a decode step's append for a full batch with all heads (bf16 cache, 4096-token contexts)
        dict(name="append-step-bf16", op="append", B=64, new=64, ragged=False, ctx=4096, H=128, kv="bf16", tail=0),
        # a speculative step: 1 to 9 tokens per sequence, odd batch, int8 cache
        dict(name="append-drafts-q8", op="append", B=47, new=211, ragged=True, ctx=1000, H=128, kv="q8_0", tail=3),
        # whole prompts of different lengths into an e4m3 cache, all heads, a padded batch
        dict(name="append-prompts-e4m3", op="append", B=12, new=16351, ragged=True, ctx=0, H=128, kv="e4m3", tail=33),
        # one short prompt on a 16-head shard: latency
        dict(name="packed-short", op="packed", B=1, n=17, ragged=False, H=16, H_kv=16, d_r=64, tail=0),
        # many short prompts (chat turns) on a 16-head shard
        dict(name="packed-many", op="packed", B=67, n=8191, ragged=True, H=16, H_kv=16, d_r=64, tail=1),
        # grouped heads without a separate rotated part: a drafting model's prompts
        dict(name="packed-grouped", op="packed", B=5, n=7001, ragged=True, H=32, H_kv=8, d_r=0, tail=0),
        # ragged prompts, all heads
        dict(name="packed-ragged", op="packed", B=7, n=5120, ragged=True, H=128, H_kv=128, d_r=64, tail=40),
        # one long prompt, all heads
        dict(name="packed-long", op="packed", B=1, n=4096, ragged=False, H=128, H_kv=128, d_r=64, tail=0),
        # one sequence with four drafts: latency
        dict(name="verify-one", op="verify", B=1, drafts=4, ragged=False, V=32000, dtype="fp32", accept=0.7),
        # a ragged batch, odd vocabulary, bf16 probabilities
        dict(name="verify-odd-bf16", op="verify", B=33, drafts=7, ragged=True, V=100003, dtype="bf16", accept=0.8),
        # a full batch over a large vocabulary
        dict(name="verify-batch", op="verify", B=256, drafts=3, ragged=False, V=128000, dtype="fp32", accept=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "packed", "verify"])
    if op == "append":
        B = _log(rng, 1, 128)
        new = max(B, min(_log(rng, B, 16384), 16384))
        return dict(op=op, B=B, new=new, ragged=new > B, ctx=rng.choice([0, 1, 63, 64, 517, 2048]),
                    H=rng.choice([0, 16, 32, 64, 128]), kv=rng.choice(list(ROW_BYTES)), tail=rng.choice([0, 0, 5]))
    if op == "packed":
        d_r = rng.choice([0, 64, 64])
        H = rng.choice([8, 16, 32, 64, 128])
        H_kv = H if d_r else rng.choice([1, H // 8, H // 4, H // 2])
        n = _log(rng, 1, 4096 if H > 32 else 8192)
        B = min(n, _log(rng, 1, 64))
        # the plain form pads: keep its scores below those of the longest listed prompt
        while B > 1 and B * H * max(_lens(B, n, True)) ** 2 > 128 * 4096 ** 2:
            B //= 2
        if B * H * max(_lens(B, n, B > 1)) ** 2 > 128 * 4096 ** 2:
            n = 4096
        return dict(op=op, B=B, n=n, ragged=B > 1, H=H, H_kv=H_kv, d_r=d_r, tail=rng.choice([0, 0, 7]))
    B, drafts = _log(rng, 1, 256), rng.randint(1, 8)
    V = _log(rng, 1000, 128000)
    drafts = max(1, min(drafts, 256 * 3 * 128000 // (B * V)))
    return dict(op=op, B=B, drafts=drafts, ragged=rng.random() < 0.5, V=V, dtype=rng.choice(["fp32", "bf16"]),
                accept=rng.choice([0.5, 0.7, 0.9]))


def _lens(B, total, ragged):
    """Lengths (at least one each) of B sequences that add up to `total`: equal, or spread unevenly."""
    if not ragged:
        return [total // B] * B
    rng = random.Random(1000003 * B + total)
    w = [rng.random() ** 2 + 0.02 for _ in range(B)]
    lens = [1 + int((total - B) * x / sum(w)) for x in w]
    lens[rng.randrange(B)] += total - sum(lens)
    return lens


def _verify_plan(case):
    """Drafts and planned acceptances of every sequence."""
    B, S = case["B"], case["drafts"]
    rng = random.Random(7919 * B + S)
    num = [rng.randint(0, S) if case["ragged"] else S for _ in range(B)]
    acc = []
    for n in num:
        a = 0
        while a < n and rng.random() < case["accept"]:
            a += 1
        acc.append(a)
    return num, acc


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _INPUTS[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _ints([0] + list(np.cumsum(lens)))


def _append_inputs(case, g):
    lens = _lens(case["B"], case["new"], case["ragged"])
    after = [case["ctx"] + n for n in lens]
    rows = sum(lens) + case["tail"]
    pages = [(n + PAGE - 1) // PAGE for n in after]
    P = sum(pages)
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + list(np.cumsum(pages)), device="cuda")
    col = torch.arange(max(pages), device="cuda")
    table = perm[(first[:-1, None] + col).clamp(max=P - 1)]
    # the joint down-projection's output, latent and key side by side: two strided views
    joint = _randn(g, rows, ROW).to(torch.bfloat16)
    # the query projection's output, 192 values a head, whose last 64 are rotated
    q = _randn(g, rows, case["H"], D_N + D_R).to(torch.bfloat16)
    x = dict(c=joint[:, :D_C], k_pe=joint[:, D_C:], q_pe=q[..., D_N:], table=table.contiguous(), cu=_cu(lens),
             lens=_ints(after), k_out=torch.zeros(rows, D_R, dtype=torch.bfloat16, device="cuda"),
             q_out=torch.zeros(rows, case["H"], D_R, dtype=torch.bfloat16, device="cuda"))
    kv = case["kv"]
    if kv == "bf16":
        x["cache"], x["scale"] = _randn(g, P, PAGE, ROW).to(torch.bfloat16), None
    elif kv == "e4m3":
        x["cache"] = _randn(g, P, PAGE, ROW).to(torch.float8_e4m3fn)
        x["scale"] = torch.rand(P, PAGE, generator=g, device="cuda") + 0.5
    elif kv == "q8_0":
        x["cache"] = torch.randint(-127, 128, (P, PAGE, ROW), generator=g, device="cuda", dtype=torch.int8)
        x["scale"] = (torch.rand(P, PAGE, ROW // BLOCK, generator=g, device="cuda") * 0.02 + 0.01).half()
    else:
        lo = torch.randint(1, 16, (P, PAGE, ROW // 2), generator=g, device="cuda", dtype=torch.uint8)
        hi = torch.randint(1, 16, (P, PAGE, ROW // 2), generator=g, device="cuda", dtype=torch.uint8)
        x["cache"] = lo | (hi << 4)
        x["scale"] = (torch.rand(P, PAGE, ROW // BLOCK, generator=g, device="cuda") * 0.3 + 0.2).half()
    return x


def _packed_inputs(case, g):
    lens = _lens(case["B"], case["n"], case["ragged"])
    rows, H, H_kv, d_r = sum(lens) + case["tail"], case["H"], case["H_kv"], case["d_r"]
    if d_r:
        # the up-projection's output holds every head's key and value side by side
        q = _randn(g, rows, H, D_N + d_r).to(torch.bfloat16)
        kv = _randn(g, rows, H_kv, D_N + D_V).to(torch.bfloat16)
        k_pe = _randn(g, rows, d_r).to(torch.bfloat16)
        x = dict(q_nope=q[..., :D_N], q_pe=q[..., D_N:], k_nope=kv[..., :D_N], k_pe=k_pe, v=kv[..., D_N:])
    else:
        # one fused projection's output: queries, keys, values
        qkv = _randn(g, rows, H + 2 * H_kv, D_N).to(torch.bfloat16)
        x = dict(q_nope=qkv[:, :H], q_pe=None, k_nope=qkv[:, H:H + H_kv], k_pe=None, v=qkv[:, H + H_kv:])
    x["cu"] = _cu(lens)
    x["longest"] = max(lens)
    x["scale"] = 1.0 / math.sqrt(D_N + d_r)
    x["out"] = torch.zeros(rows, H, D_V, dtype=torch.bfloat16, device="cuda")
    x["lse"] = torch.zeros(rows, H, device="cuda")
    return x


def _verify_inputs(case, g):
    B, S, V = case["B"], case["drafts"], case["V"]
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    logits = 2.5 * _randn(g, B, S + 1, V)
    p = torch.softmax(logits, -1).to(dtype)
    # the drafting model's distribution: near the target's
    q = torch.softmax(logits[:, :S].add_(_randn(g, B, S, V), alpha=0.7), -1).to(dtype)
    del logits
    num, acc = (torch.tensor(v, device="cuda") for v in _verify_plan(case))
    # drafts drawn from q; where a rejection is planned, a token that the draft rates above the target
    flat = q.view(-1, V).float()
    pick = torch.rand(B * S, 1, generator=g, device="cuda") * flat.sum(-1, keepdim=True)
    tok = torch.searchsorted(flat.cumsum(-1), pick).clamp(max=V - 1).view(B, S)
    del flat
    step = torch.arange(S, device="cuda")
    rejects = (step == acc[:, None]) & (acc < num)[:, None]
    tok = torch.where(rejects, (q.float() - p[:, :S].float()).argmax(-1), tok)
    ratio = (p[:, :S].gather(-1, tok[..., None]).double() / q.gather(-1, tok[..., None]).double().clamp(min=1e-30)).squeeze(-1).clamp(max=1.0)
    r = torch.rand(B, S, generator=g, device="cuda", dtype=torch.float64)
    u = torch.where(rejects, ratio + (1 - ratio) * (0.1 + 0.8 * r), ratio * (0.05 + 0.9 * r))
    u = torch.where((step > acc[:, None]) | (step >= num[:, None]), r, u).float().clamp(max=1 - 2.0 ** -24)
    lens = torch.randint(S + 1, 4097, (B,), generator=g, device="cuda", dtype=torch.int32)
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")
    return dict(p=p, q=q, tok=tok.to(torch.int32), num=num.to(torch.int32), u=u,
                u_last=torch.rand(B, generator=g, device="cuda"), lens=lens, tokens=ints(B, S + 1), accepted=ints(B),
                new_lens=ints(B))


_INPUTS = {"append": _append_inputs, "packed": _packed_inputs, "verify": _verify_inputs}


def prepare(case, seed):
    x = _inputs(case, seed)
    x["case"] = case
    if own:
        import head_latent_attention_06_b200 as mla
        if case["op"] == "append":
            x["args"] = mla.make_append_args(
                c=x["c"], k_pe=x["k_pe"], q_pe=x["q_pe"] if case["H"] else None, k_pe_out=x["k_out"],
                q_pe_out=x["q_out"] if case["H"] else None, kv_cache=x["cache"], kv_scale=x["scale"],
                block_table=x["table"], cu_seqlens=x["cu"], seq_lens=x["lens"], rope_base=ROPE_BASE)
        elif case["op"] == "packed":
            x["args"] = mla.make_prefill_packed_args(
                q_nope=x["q_nope"], q_pe=x["q_pe"], k_nope=x["k_nope"], k_pe=x["k_pe"], v=x["v"], cu_seqlens=x["cu"],
                out=x["out"], lse=x["lse"], causal=True, softmax_scale=x["scale"])
        else:
            x["args"] = mla.make_verify_args(
                target_probs=x["p"], draft_probs=x["q"], draft_tokens=x["tok"], num_draft=x["num"], u_accept=x["u"],
                u_sample=x["u_last"], seq_lens=x["lens"], tokens=x["tokens"], num_accepted=x["accepted"],
                new_lens=x["new_lens"])
        x["workspace"] = mla.alloc_workspace(x["args"])
        x["mla"] = mla
    return x


# ------------------------------------------------------------------ the operators

def run(state):
    return _RUN[state["case"]["op"]](state)


def _owner(cu, rows):
    """Sequence of every row (rows behind the last one get the last), and whether it has one."""
    t = torch.arange(rows, device=cu.device)
    b = torch.searchsorted(cu, t.to(cu.dtype), right=True) - 1
    return t, b.clamp(max=cu.numel() - 2), t < cu[-1]


def _rotate(x, cos, sin):
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * cos - x1 * sin, x0 * sin + x1 * cos), -1).flatten(-2)


def _held(cache, scale, kv):
    """What the cache stands for: bf16 and e4m3 as they are, integer codes times their block's scale."""
    if kv == "q4_0":
        cache = torch.stack((cache & 15, cache >> 4), -1).to(torch.int8) - 8
    if kv in ("q8_0", "q4_0"):
        cache = cache.view(*cache.shape[:2], ROW // BLOCK, BLOCK) * scale[..., None]
    return cache


def _append(s):
    kv = s["case"]["kv"]
    if own:
        s["mla"].mla_append_kv(s["args"])
    else:
        t, b, real = _owner(s["cu"], s["c"].shape[0])
        pos = s["lens"][b] - s["cu"][b + 1] + t
        theta = ROPE_BASE ** (-torch.arange(0, D_R, 2, device="cuda", dtype=torch.float64) / D_R)
        angle = pos[:, None].double() * theta
        cos, sin = angle.cos().float(), angle.sin().float()
        k = _rotate(s["k_pe"].float(), cos, sin)
        s["k_out"].copy_(torch.where(real[:, None], k.bfloat16(), s["k_out"]))
        q = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None])
        s["q_out"].copy_(torch.where(real[:, None, None], q.bfloat16(), s["q_out"]))
        row = torch.cat((s["c"].float(), k), -1)
        at = s["table"][b, (pos // PAGE).clamp(max=s["table"].shape[1] - 1)].long() * PAGE + pos % PAGE
        # rows behind the last sequence repeat the last real row
        last = s["cu"][-1].long() - 1
        src = torch.minimum(t, last)
        at, row = at[src], row[src]
        flat = s["cache"].view(-1, s["cache"].shape[-1])
        if kv == "bf16":
            flat[at] = row.bfloat16()
        elif kv == "e4m3":
            amax = row.abs().amax(-1, keepdim=True)
            sc = torch.where(amax > 0, amax / 448.0, 1.0)
            flat.view(torch.uint8)[at] = (row / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s["scale"].view(-1)[at] = sc[:, 0]
        else:
            levels = 127 if kv == "q8_0" else 7
            blocks = row.view(-1, ROW // BLOCK, BLOCK)
            d = (blocks.abs().amax(-1) / levels).half()
            df = d.float()[..., None]
            code = torch.where(df > 0, torch.round(blocks / df).clamp(-levels, levels), 0.0).view(-1, ROW)
            if kv == "q4_0":
                n = (code + 8).to(torch.uint8)
                flat[at] = n[:, 0::2] | (n[:, 1::2] << 4)
            else:
                flat[at] = code.to(torch.int8)
            s["scale"].view(-1, ROW // BLOCK)[at] = d
    out = dict(cache=_held(s["cache"], s["scale"], kv), k_pe=s["k_out"], q_pe=s["q_out"])
    if kv == "e4m3":
        out["scale"] = s["scale"]
    return out


def _packed(s):
    if own:
        s["mla"].mla_prefill_packed(s["args"])
        return dict(out=s["out"], lse=s["lse"])
    t, b, real = _owner(s["cu"], s["q_nope"].shape[0])
    i = torch.arange(s["longest"], device="cuda")
    # the packed sequences as a padded batch
    at = (s["cu"][:-1, None] + i).clamp(max=t.numel() - 1).long()
    q, k = s["q_nope"][at].float(), s["k_nope"][at].float()
    v = s["v"][at].float()
    share = q.shape[2] // k.shape[2]
    k, v = k.repeat_interleave(share, 2), v.repeat_interleave(share, 2)
    scores = q.permute(0, 2, 1, 3) @ k.permute(0, 2, 3, 1)
    if s["q_pe"] is not None:
        scores += s["q_pe"][at].float().permute(0, 2, 1, 3) @ s["k_pe"][at].float()[:, None].transpose(2, 3)
    scores *= s["scale"]
    lens = (s["cu"][1:] - s["cu"][:-1])[:, None, None, None]
    scores.masked_fill_((i[None, :] > i[:, None]) | (i >= lens), -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    o = ((scores @ v.permute(0, 2, 1, 3)) / total).bfloat16().transpose(1, 2)
    lse = (top + total.log()).squeeze(-1).transpose(1, 2)
    pos = (t - s["cu"][b]).clamp(max=s["longest"] - 1)
    return dict(out=torch.where(real[:, None, None], o[b, pos], s["out"]),
                lse=torch.where(real[:, None], lse[b, pos], s["lse"]))


def _verify(s):
    if own:
        s["mla"].mla_verify_draft(s["args"])
        return dict(tokens=s["tokens"], accepted=s["accepted"], new_lens=s["new_lens"])
    p, q, tok, num = s["p"], s["q"], s["tok"].long(), s["num"].long()
    B, S = tok.shape
    px = p[:, :S].gather(-1, tok[..., None]).squeeze(-1).double()
    qx = q.gather(-1, tok[..., None]).squeeze(-1).double()
    step = torch.arange(S + 1, device="cuda")
    good = (s["u"].double() * qx < px) & (step[:S] < num[:, None])
    a = good.long().cumprod(-1).sum(-1)
    b = torch.arange(B, device="cuda")
    target = p[b, a].double()
    draft = torch.where((a < num)[:, None], q[b, a.clamp(max=S - 1)].double(), 0.0)
    rest = (target - draft).clamp(min=0)
    # a draft that is nowhere below the target leaves nothing: the target itself then
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, target)
    acc = rest.cumsum(-1)
    new = (acc <= s["u_last"].double()[:, None] * acc[:, -1:]).sum(-1)
    padded = torch.cat((tok, tok[:, :1]), 1)
    tokens = torch.where(step < a[:, None], padded, torch.where(step == a[:, None], new[:, None], -1))
    return dict(tokens=tokens.int(), accepted=a.int(), new_lens=(s["lens"] - (num - a)).int())


_RUN = {"append": _append, "packed": _packed, "verify": _verify}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "append":
        n, H = case["new"], case["H"]
        moved = n * (2 * ROW + ROW_BYTES[case["kv"]] + 2 * D_R + 4 * H * D_R)
        return {"bytes": moved, "flops": 3 * n * (H + 1) * D_R}
    if case["op"] == "packed":
        H, H_kv, d_r = case["H"], case["H_kv"], case["d_r"]
        pairs = sum(L * (L + 1) // 2 for L in _lens(case["B"], case["n"], case["ragged"]))
        values = H * (D_N + d_r) + H_kv * (D_N + D_V) + d_r + H * D_V
        return {"bytes": case["n"] * (2 * values + 4 * H), "flops": 2 * pairs * H * (D_N + d_r + D_V)}
    num, acc = _verify_plan(case)
    size = 4 if case["dtype"] == "fp32" else 2
    rows = case["B"] + sum(a < n for a, n in zip(acc, num))
    return {"bytes": rows * case["V"] * size, "flops": 2 * rows * case["V"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](case, _inputs(case, seed))


def _exact_append(case, x):
    """Token by token positions on the host, complex rotation, codes from 64-bit quotients."""
    kv, cu, after = case["kv"], x["cu"].tolist(), x["lens"].tolist()
    n = cu[-1]
    pos = np.concatenate([np.arange(L - (hi - lo), L) for lo, hi, L in zip(cu, cu[1:], after)])
    seq = np.repeat(np.arange(len(after)), np.diff(cu))
    table = x["table"].cpu().numpy()
    at = torch.from_numpy(table[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE).cuda()
    turn = np.exp(1j * pos[:, None] * ROPE_BASE ** (-np.arange(D_R // 2) / (D_R / 2)))
    turn = torch.from_numpy(turn).cuda()

    def turned(v):
        z = torch.view_as_complex(v.double().reshape(*v.shape[:-1], D_R // 2, 2).contiguous())
        w = turn if v.dim() == 2 else turn[:, None]
        return torch.view_as_real(z * w).flatten(-2)

    k_out, q_out = x["k_out"].double(), x["q_out"].double()
    k_out[:n] = turned(x["k_pe"][:n])
    if case["H"]:
        q_out[:n] = turned(x["q_pe"][:n])
    row = torch.cat([x["c"][:n].double(), k_out[:n]], 1)
    cache = x["cache"]
    if kv == "bf16":
        held = cache.double().view(-1, ROW)
        held[at] = row
        return dict(cache=held.view(cache.shape), k_pe=k_out, q_pe=q_out)
    if kv == "e4m3":
        held, scale = cache.double().view(-1, ROW), x["scale"].double().view(-1)
        top = row.abs().amax(1)
        sc = torch.where(top > 0, top / 448, torch.ones_like(top))
        held[at], scale[at] = row / sc[:, None], sc
        return dict(cache=held.view(cache.shape), k_pe=k_out, q_pe=q_out, scale=scale.view(x["scale"].shape))
    code = cache
    if kv == "q4_0":
        code = torch.stack([cache % 16, cache // 16], -1).double() - 8
    held = code.double().reshape(-1, ROW // BLOCK, BLOCK) * x["scale"].double().reshape(-1, ROW // BLOCK, 1)
    levels = 127 if kv == "q8_0" else 7
    blocks = row.view(n, ROW // BLOCK, BLOCK)
    d = (blocks.abs().amax(2, keepdim=True) / levels).half().double()
    near = torch.round(blocks / d.clamp(min=1e-30)).clamp(-levels, levels)
    held[at] = near * d
    return dict(cache=held.view(*cache.shape[:2], ROW // BLOCK, BLOCK), k_pe=k_out, q_pe=q_out)


def _exact_packed(case, x):
    """Sequence by sequence, a few heads at a time."""
    H, share = case["H"], case["H"] // case["H_kv"]
    out, lse = x["out"].double(), x["lse"].double()
    cu = x["cu"].tolist()
    for lo, hi in zip(cu, cu[1:]):
        L = hi - lo
        future = torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1)
        for h0 in range(0, H, 16):
            hs = torch.arange(h0, min(H, h0 + 16), device="cuda")
            q = x["q_nope"][lo:hi, hs].double()
            k = x["k_nope"][lo:hi, hs // share].double()
            if case["d_r"]:
                q = torch.cat([q, x["q_pe"][lo:hi, hs].double()], -1)
                k = torch.cat([k, x["k_pe"][lo:hi, None].double().expand(-1, hs.numel(), -1)], -1)
            z = torch.einsum("ihd,jhd->hij", q, k) * x["scale"]
            z = z.masked_fill(future, -math.inf)
            norm = torch.logsumexp(z, -1)
            out[lo:hi, hs] = torch.einsum("hij,jhd->ihd", torch.exp(z - norm[..., None]), x["v"][lo:hi, hs // share].double())
            lse[lo:hi, hs] = norm.T
    return dict(out=out, lse=lse)


def _exact_verify(case, x):
    """One sequence after the other on the host."""
    num, tok = x["num"].tolist(), x["tok"].tolist()
    u, last, lens = x["u"].double().cpu().numpy(), x["u_last"].double().cpu().numpy(), x["lens"].tolist()
    B, S = case["B"], case["drafts"]
    tokens, accepted, new_lens = np.full((B, S + 1), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        a = 0
        while a < num[b]:
            j = tok[b][a]
            if not u[b, a] * float(x["q"][b, a, j]) < float(x["p"][b, a, j]):
                break
            tokens[b, a] = j
            a += 1
        w = x["p"][b, a].double().cpu().numpy()
        if a < num[b]:
            left = np.maximum(w - x["q"][b, a].double().cpu().numpy(), 0)
            w = left if left.sum() > 0 else w
        sums = np.cumsum(w)
        tokens[b, a] = np.searchsorted(sums, last[b] * sums[-1], side="right")
        accepted[b], new_lens[b] = a, lens[b] - (num[b] - a)
    return dict(tokens=tokens, accepted=accepted, new_lens=new_lens)


_EXACT = {"append": _exact_append, "packed": _exact_packed, "verify": _exact_verify}
