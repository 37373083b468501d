"""The serving operators together, as an engine runs them: packed prompts into the
cache and through the packed attention, a speculative step on top (append of the
drafted tokens, causal decode over them, verification), and the step after it,
whose sequences have lost the rejected drafts."""

import numpy as np
import pytest
import torch

from mla_inputs import bf16_bits
from oracle import cache_write as cw
from oracle import mla_oracle as om
from oracle import serving

from parity_util import TOL, check_lse, errors, to_np

pytestmark = pytest.mark.gpu

bf16, i32 = torch.bfloat16, torch.int32
H, SCALE, BASE = 16, 1 / 192 ** 0.5, 10000.0


def f64(t):
    return om.bf16_to_f64(bf16_bits(t.cpu().contiguous()))


@pytest.mark.parametrize("kv_dtype", ["bf16", "q8_0"])
def test_prompts_then_drafts(cuda_lib, kv_dtype):
    from head_latent_attention_06_b200.step import PackedPrefill, SpeculativeStep
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)
    prompts, s_q, V = [100, 1, 64, 190], 3, 500
    B, n = len(prompts), sum(prompts)
    w_uk, w_uv = ((r(H, 128, 512) / 512 ** 0.5).to(bf16) for _ in range(2))
    latent = [r(L + 2 * s_q, 576).to(bf16) for L in prompts]          # the prompt, then two steps' tokens
    q = [r(L + 2 * s_q, H, 192).to(bf16) for L in prompts]
    P = 4 * B
    table = torch.randperm(P, generator=g).to(i32).view(B, 4).cuda()
    if kv_dtype == "bf16":
        cache, scale = torch.zeros(P, 64, 576, dtype=bf16, device="cuda"), None
    else:
        cache = torch.zeros(P, 64, 576, dtype=torch.int8, device="cuda")
        scale = torch.zeros(P, 64, 18, dtype=torch.float16, device="cuda")
    lens = torch.tensor(prompts, dtype=i32, device="cuda")
    cu = torch.tensor([0] + list(np.cumsum(prompts)), dtype=i32, device="cuda")
    pick = lambda xs: torch.cat([x[:L] for x, L in zip(xs, prompts)]).cuda()
    lat_d, q_d = pick(latent), pick(q)
    c = lat_d[:, :512].double()
    kv = torch.cat([torch.einsum("tc,hnc->thn", c, w.cuda().double()) for w in (w_uk, w_uv)], -1).to(bf16)
    pre = PackedPrefill(q=q_d, kv=kv, latent=lat_d, kv_cache=cache, kv_scale=scale, block_table=table, cu_seqlens=cu,
                        seq_lens=lens, softmax_scale=SCALE, rope_base=BASE)
    pre.run()
    assert cuda_lib.mla_get_status(pre.append_workspace) == 0 and cuda_lib.mla_get_status(pre.workspace) == 0

    # exact: rotate, attend over the rotated prompt with the same bf16 keys and values
    at = 0
    for b, L in enumerate(prompts):
        pos = np.arange(L)
        k_pe = cw.rope(f64(latent[b][:L, 512:]), pos, BASE)
        q_pe = cw.rope(f64(q[b][:L, :, 128:]), np.repeat(pos[:, None], H, 1), BASE)
        kvb = f64(kv[at:at + L])
        qq = np.concatenate([f64(q[b][:L, :, :128]), q_pe], -1)
        kk = np.concatenate([kvb[..., :128], np.repeat(k_pe[:, None], H, 1)], -1)
        o, lse, _, _ = serving.attend_packed(qq, kk, kvb[..., 128:], [0, L], SCALE, True)
        ma, rl = errors(to_np(pre.out[at:at + L]), o)
        assert ma <= TOL["bf16"][0] + 2.0 ** -8 * np.abs(o).max() and rl <= TOL["bf16"][1], (b, ma, rl)
        check_lse(to_np(pre.lse[at:at + L]), lse, TOL["bf16"][0])
        at += L

    # two speculative steps; between them the lengths lose the rejected drafts
    lens = lens + s_q
    used = [list(range(L)) for L in prompts]                          # rows of `latent` in the cache, by position
    for step in range(2):
        rows = [list(range(L + step * s_q, L + (step + 1) * s_q)) for L in prompts]
        sp = SpeculativeStep(
            latent=torch.cat([x[i] for x, i in zip(latent, rows)]).cuda(),
            q_nope=torch.stack([x[i][..., :128] for x, i in zip(q, rows)]).contiguous().cuda(),
            q_pe=torch.stack([x[i][..., 128:] for x, i in zip(q, rows)]).cuda(), w_uk=w_uk.cuda(), w_uv=w_uv.cuda(),
            kv_cache=cache, kv_scale=scale, block_table=table, seq_lens=lens, softmax_scale=SCALE, rope_base=BASE)
        before = lens.tolist()
        sp.run()
        assert cuda_lib.mla_get_status(sp.append_workspace) == 0 and cuda_lib.mla_get_status(sp.workspace) == 0
        out, lse = to_np(sp.out), to_np(sp.lse)
        for b in range(B):
            have = used[b] + rows[b]
            assert len(have) == before[b]
            pos = np.arange(len(have))
            lat = f64(latent[b][have])
            k_pe = cw.rope(lat[:, 512:], pos, BASE)
            wk, wv = f64(w_uk), f64(w_uv)
            kk = np.concatenate([np.einsum("tc,hnc->thn", lat[:, :512], wk), np.repeat(k_pe[:, None], H, 1)], -1)
            vv = np.einsum("tc,hnc->thn", lat[:, :512], wv)
            qb = f64(q[b][rows[b]])
            qq = np.concatenate([qb[..., :128], cw.rope(qb[..., 128:], np.repeat(pos[-s_q:, None], H, 1), BASE)], -1)
            full = np.concatenate([np.zeros((len(have) - s_q, H, 192)), qq])
            o, ol, _, _ = serving.attend_packed(full, kk, vv, [0, len(have)], SCALE, True)
            ma, rl = errors(out[b], o[-s_q:])
            # an int8 code is off by up to 1/254 of its block's largest value (some 2.5 sigma):
            # 0.01 sigma, uniform over the step, so 0.6 % of sigma in keys and in values
            slack = 0.0 if kv_dtype == "bf16" else 3 * 0.006
            assert ma <= TOL["bf16"][0] + 2 * slack and rl <= TOL["bf16"][1] + slack, (step, b, ma, rl)
            check_lse(lse[b], ol[-s_q:], TOL["bf16"][0] + 2 * slack)
        # the model's tail stands in: probabilities from the outputs
        w_out = r(H * 128, V).cuda() / 20
        target = torch.softmax(sp.out.float().flatten(2) @ w_out, -1)
        draft = torch.softmax((sp.out.float().flatten(2) @ w_out)[:, :s_q - 1] + 0.5 * r(B, s_q - 1, V).cuda(), -1)
        tok = torch.stack([torch.multinomial(d, 1)[:, 0] for d in draft]).to(i32)
        u, last = torch.rand(B, s_q - 1, generator=g).cuda(), torch.rand(B, generator=g).cuda()
        tokens, accepted = sp.verify(target_probs=target, draft_probs=draft, draft_tokens=tok, u_accept=u, u_sample=last)
        assert cuda_lib.mla_get_status(sp.verify_workspace) == 0
        want = serving.verify_draft(target.cpu().numpy(), draft.cpu().numpy(), tok.cpu().numpy(), [s_q - 1] * B,
                                    u.cpu().numpy(), last.cpu().numpy(), before)
        np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
        np.testing.assert_array_equal(accepted.cpu().numpy(), want[1])
        assert lens.tolist() == want[2].tolist()
        for b in range(B):
            used[b] = used[b] + rows[b][:1 + int(want[1][b])]
        lens.add_(s_q)
