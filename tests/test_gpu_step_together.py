"""The operators around a verification step as a rollout uses them: prompts into
the cache, drafted tokens rotated, attention over the shared prompts, adjusted
logits, rejection sampling, commit -- two steps, each against plain 64-bit forms."""
import math

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from tests import step_ref, tree_ref

pytestmark = pytest.mark.gpu
i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


@pytest.mark.parametrize("dtype, D", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_rollout_steps(dtype, D):
    g = torch.Generator().manual_seed(D)
    P, B, T, Hq, Hkv, ps, V = 2, 5, 4, 4, 2, 16, 997
    starts, prompts = [0, 3, 5], [70, 33]
    freq, factor = mtp.rope_frequencies(D, scaling="parts", factor=4.0, original_length=64)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    pages = torch.randperm(P * 5 + B * 2, generator=g).int()
    prefix_table, table = pages[:P * 5].view(P, 5).contiguous(), pages[P * 5:].view(B, 2).contiguous()
    kc, vc = (torch.full((len(pages), ps, Hkv, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    cuda = lambda *ts: [t.cuda() for t in ts]  # noqa: E731
    d_prefix, d_table, d_freq, d_starts = cuda(prefix_table, table, freq, torch.tensor(starts, dtype=i32))
    plen = torch.tensor(prompts, dtype=i32)

    # the prompts' keys and values, rotated on the way
    k, v = rand(P, 70, Hkv, D).to(dtype), rand(P, 70, Hkv, D).to(dtype)
    r = mtp.mtp_cache_append(*cuda(k, v), kc, vc, d_prefix, torch.zeros(P, dtype=i32, device="cuda"), plen.cuda(), inv_freq=d_freq, factor=factor)
    assert r.cache_len.tolist() == prompts and r.row_flags.tolist() == [0, 0]
    text_k, text_v = [[] for _ in range(B)], [[] for _ in range(B)]  # of each sequence, as the cache holds them
    want, tol = step_ref.rope(k, torch.arange(70, dtype=i32).expand(P, 70), freq, factor=factor)
    for p in range(P):
        at = torch.arange(prompts[p])
        page = prefix_table[p].long()[at // ps]
        got = kc.cpu()[page, at % ps]
        assert ((got.double() - want[p, :prompts[p]]).abs() <= tol[p, :prompts[p]]).all()
        for b in range(starts[p], starts[p + 1]):
            text_k[b], text_v[b] = list(got), list(v[p, :prompts[p]])

    group = torch.tensor([0, 0, 0, 1, 1])
    lens = torch.zeros(B, dtype=i32)
    history, hist_len = torch.full((B, 40), -1, dtype=i32), torch.zeros(B, dtype=i32)
    proj = rand(Hq * D, V) * 0.3
    last = torch.randint(V, (B,), generator=g, dtype=i32)
    for step in range(2):
        drafts = torch.randint(V, (B, T - 1), generator=g, dtype=i32)
        tokens = torch.cat([last[:, None], drafts], 1)
        q, k, v = (rand(B, T, h, D).to(dtype) for h in (Hq, Hkv, Hkv))
        pos = plen[group][:, None] + lens[:, None] + torch.arange(T, dtype=i32)
        d_q, d_k, d_v, d_pos, d_len = cuda(q, k, v, pos, lens)
        rot = mtp.mtp_rope(d_q, d_k, d_pos, d_freq, factor=factor, out=mtp.RopeResult(d_q, d_k))  # in place
        for x, y in ((q, rot.q), (k, rot.k)):
            want, tol = step_ref.rope(x, pos, freq, factor=factor)
            assert ((y.cpu().double() - want).abs() <= tol).all()
        a = mtp.mtp_prefix_attention(rot.q, rot.k, d_v, kc, vc, d_prefix, plen.cuda(), d_starts, d_table, d_len)
        assert a.row_flags.tolist() == [0] * B
        n = torch.tensor([len(t) for t in text_k])
        one = lambda ts: torch.cat([torch.stack(t) for t in ts])[:, None]  # noqa: E731
        flat = torch.zeros(B, int(n.max()), dtype=i32)
        for b in range(B):
            flat[b, :n[b]] = torch.arange(n[b]) + n[:b].sum()
        want, _, tol, _, _ = tree_ref.attention(rot.q.cpu(), rot.k.cpu(), v, one(text_k), one(text_v), flat, n)
        assert ((a.out.cpu().double() - want).abs() <= tol).all()

        # target logits from the attention, the drafter's beside them; a grammar that forbids some words
        target = (a.out.flatten(2).float() @ proj.cuda()).contiguous()
        draft = (target[:, :T - 1] + 0.5 * rand(B, T - 1, V).cuda()).contiguous()
        words = torch.rand(B, T, (V + 31) // 32 * 32, generator=g) < 0.6
        words[..., :64] = True
        bits = (words.view(B, T, -1, 32).long() << torch.arange(32)).sum(-1)
        mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int()
        rho, f, p = torch.full((B,), 1.2), torch.full((B,), 0.3), torch.full((B,), 0.1)
        d_tok, d_hist, d_hl, d_mask = cuda(tokens, history, hist_len, mask)
        pen = dict(repetition=rho.cuda(), frequency=f.cuda(), presence=p.cuda())
        before = target.cpu()
        z = mtp.mtp_adjust_logits(target, d_hist, d_hl, tokens=d_tok, mask=d_mask, out=mtp.AdjustResult(target, None), **pen)  # in place
        want, tol, _ = step_ref.adjust(before, history, hist_len, tokens=tokens, repetition=rho, frequency=f, presence=p, mask=mask)
        got = z.logits.cpu().double()
        assert torch.equal(got.isinf(), want.isinf()) and ((got - want).abs()[want.isfinite()] <= tol[want.isfinite()]).all()
        zd = mtp.mtp_adjust_logits(draft, d_hist, d_hl, tokens=d_tok[:, :T - 1].contiguous(), mask=d_mask[:, :T - 1], **pen)

        # rejection sampling: every token is one that the grammar allows where it stands
        u = torch.rand(B, T, generator=g)
        s = mtp.mtp_rs_verify(z.logits, zd.logits, d_tok[:, 1:].contiguous(), torch.ones(B, device="cuda"), u.cuda())
        assert s.row_flags.tolist() == [0] * B
        out, acc = s.tokens.cpu(), s.accept_len.cpu()
        for b in range(B):
            for j in range(int(acc[b]) + 1):
                assert words[b, j, int(out[b, j])], (b, j)
        c = mtp.mtp_tree_commit(d_tok, s.tokens, None, rot.k, d_v, kc, vc, d_table, d_len, s.accept_len + 1)
        torch.cuda.synchronize()
        assert torch.equal(c.accept_len.cpu(), acc) and torch.equal(c.cache_len.cpu(), lens + acc + 1)
        for b in range(B):
            m = int(acc[b]) + 1
            at = torch.arange(int(lens[b]), int(lens[b]) + m)
            page = table[b].long()[at // ps]
            assert torch.equal(kc.cpu()[page, at % ps], rot.k[b, :m].cpu()) and torch.equal(vc.cpu()[page, at % ps], v[b, :m])
            text_k[b] += list(rot.k[b, :m].cpu())
            text_v[b] += list(v[b, :m])
            history[b, int(hist_len[b]):int(hist_len[b]) + m] = tokens[b, :m]
            hist_len[b] += m
            last[b] = out[b, m - 1]
        lens = c.cache_len.cpu()
