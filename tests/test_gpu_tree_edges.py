"""Tree attention, reorder and commit on the GPU at the edges of their use:
waits that run out, streams, graphs, page tables wider than the text."""
import math
import random

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from tests import tree_ref
from tests.test_gpu_tree_ops import attn_case, check_attention, check_commit, commit_case, on_gpu

pytestmark = pytest.mark.gpu
i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


# ------------------------------------------------------ waits that run out --

def attend(g, B, T, Hq, D, fill=7.0):
    """Outputs that were something else before, flags among them."""
    out = mtp.TreeAttentionResult(torch.full((B, T, Hq, D), fill, dtype=torch.bfloat16, device="cuda"),
                                  torch.full((B, T, Hq), fill, device="cuda"), torch.full((B,), 12345, dtype=i32, device="cuda"))
    r = mtp.mtp_tree_attention(**g, out=out)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("T, Hq, Hkv, D, ps, lens, ctas", [
    (2, 8, 2, 64, 16, [40, 0, 300], (0, 1, 2, 3, 4, 5)),             # whole units, up to 32 rows
    (8, 16, 2, 128, 32, [129, 500, 64], (0, 1, 3, 5)),               # 64 rows
    (64, 16, 2, 128, 32, [129, 500], (0, 1, 2, 3, 4, 5, 6, 7)),      # 512 rows, two row tiles
    (3, 8, 2, 256, 32, [100, 33], (0, 1, 2, 3)),                     # heads of 256
    (2, 8, 2, 64, 16, [6000, 10, 2500], (0, 1, 60, 100, 140)),       # split units
    (8, 16, 2, 128, 32, [5000, 4000], (0, 1, 50, 151)),
    (64, 16, 2, 128, 32, [3000, 64], (0, 1, 40, 75, 101)),
    (3, 8, 2, 256, 32, [4000, 33], (0, 70, 140)),
])
def test_a_wait_that_runs_out_is_reported(T, Hq, Hkv, D, ps, lens, ctas):
    """The loader of one CTA leaves out a signal (test-only tuning fields), so
    the waits of that CTA give up after 20 ms.  Whichever head, tile or row
    tile it has: the call ends, every row is NaN or what it is without the
    fault, a sequence with a row of the CTA is flagged MTP_ROW_TIMEOUT and no
    other, and the next call is right again."""
    B = len(lens)
    x = attn_case(len(lens) + T, "bf16", B, T, Hq, Hkv, D, ps, lens, nodes=[T] + [max(1, T - 1)] * (B - 1))
    g = on_gpu(x)
    good = attend(g, B, T, Hq, D)
    assert good.row_flags.tolist() == [0] * B
    check_attention(x, good.out, None, good.lse, 7.0)
    seen = 0
    for cta in ctas:
        with mtp.tuning(fault_wait_us=20000, fault_skip_position=1 + cta):
            r = attend(g, B, T, Hq, D)
        lost = r.out.isnan().all(3)                      # [B, T, Hq]
        same = (r.out == good.out).all(3)
        assert (lost | same).all(), cta
        assert torch.equal(r.lse.isnan(), lost) and torch.equal(r.lse[~lost], good.lse[~lost])
        hit = lost.flatten(1).any(1)
        assert r.row_flags.tolist() == [mtp.ROW_TIMEOUT if h else 0 for h in hit.tolist()], cta
        seen += int(hit.any())
        if hit.any():
            with pytest.raises(mtp.MTPError) as e:
                mtp.check_row_flags(r.row_flags)
            assert e.value.status == mtp.MTP_ERR_TIMEOUT
    assert seen >= 2
    again = attend(g, B, T, Hq, D)
    assert torch.equal(again.out, good.out) and torch.equal(again.lse, good.lse) and again.row_flags.tolist() == [0] * B


# ------------------------------------------------------------------ commit --

@pytest.mark.parametrize("T, nodes, tree", [(1, None, "chain"), (9, [9, 0, 4], "random"), (64, None, "chain"), (64, [64, 33, 1], "random")])
@pytest.mark.parametrize("lens", [None, [0, 70, 5]])
def test_verification_alone(T, nodes, tree, lens):
    """Without keys, values, caches and table: the outputs of the whole call."""
    x = commit_case(T, "bf16", 1, 3, T, 1, 16, 16, lens or [0, 0, 0], 0.9, nodes, tree)
    g = on_gpu(x)
    want = mtp.mtp_tree_commit(**g)
    r = mtp.mtp_tree_commit(g["tokens"], g["target_tokens"], g["parents"], n_nodes=g["n_nodes"],
                            cache_len=None if lens is None else g["cache_len"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    check_commit(x, mtp.CommitResult(*(t.cpu() for t in r)), g["k_cache"], g["v_cache"])
    assert r.row_flags.tolist() == [0, 0, 0]


def test_verification_alone_flags():
    t = torch.tensor([[3, 5, 6]] * 4, dtype=i32)
    target = torch.tensor([[5, 6, 7], [5, -1, 7], [9, 0, 0], [5, 6, 7]], dtype=i32)
    up = torch.tensor([[-1, 0, 1], [-1, 0, 1], [-1, 0, 1], [-1, 1, 0]], dtype=i32)
    lens = torch.tensor([4, 4, -1, 4], dtype=i32)
    r = mtp.mtp_tree_commit(t.cuda(), target.cuda(), up.cuda(), cache_len=lens.cuda())
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] + [mtp.ROW_BAD_ID] * 3
    assert r.accept_len.tolist() == [2, -1, -1, -1] and r.cache_len.tolist() == [7, 4, -1, 4]
    assert r.tokens.tolist() == [[5, 6, 7]] + [[-1] * 3] * 3


# ------------------------------------------------------- another stream --

def calls():
    """name -> (function of the keyword arguments, its inputs on the GPU)."""
    torch.manual_seed(1)
    attn = on_gpu(attn_case(5, "bf16", 2, 4, 8, 2, 64, 16, [3000, 40]))
    whole = on_gpu(attn_case(6, "f32", 2, 4, 8, 2, 64, 16, [300, 40]))
    z, scores, T = torch.randn(2, 3, 30011, device="cuda"), torch.zeros(2, 3, device="cuda"), torch.ones(2, device="cuda")
    states, up = torch.randn(2, 2, 3, 64, device="cuda"), torch.tensor([[0, 2], [1, 1]], dtype=i32, device="cuda")
    c = on_gpu(commit_case(7, "bf16", 2, 3, 9, 2, 16, 16, [3, 16, 40]))
    return {
        "attention": lambda **k: mtp.mtp_tree_attention(**attn, with_lse=True, **k),
        "attention f32": lambda **k: mtp.mtp_tree_attention(**whole, with_lse=True, **k),
        "select": lambda **k: mtp.mtp_beam_select(z, scores, T, 9, **k),
        "reorder": lambda **k: mtp.mtp_beam_reorder(states, up, **k),
        "commit": lambda **k: mtp.mtp_tree_commit(**c, **k),
    }


@pytest.mark.parametrize("name", ["attention", "attention f32", "select", "reorder", "commit"])
def test_outputs_on_another_stream_are_nobody_elses(name):
    """Memory freed on the current stream, whose work that writes it is still
    queued, is not what a call on another stream gets for its outputs and
    workspace."""
    f = calls()[name]
    want = [None if t is None else t.clone() for t in f()]
    side = torch.cuda.Stream()
    f(stream=side)
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want if t is not None] + [1 << k for k in range(4, 24)]
    torch.cuda._sleep(100_000_000)
    for n in sizes * 3:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xff)
    r = f(stream=side)
    side.synchronize()
    kept = [None if t is None else t.cpu() for t in r]
    torch.cuda.synchronize()
    for t, k, w in zip(r, kept, want):
        if t is not None:
            assert torch.equal(t, w) and torch.equal(k, w.cpu())


def test_outputs_freed_while_they_are_read():
    """Outputs of a call on another stream, read on the current one and let go:
    the next call on that stream does not write over them."""
    f = calls()["reorder"]
    want = f().states.clone()
    side = torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(side):
            r = f(stream=side)
        r = f(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(20_000_000)
        got.append(r.states.clone())
        del r
        with torch.cuda.stream(side):
            junk = [torch.full_like(want, 9.0) for _ in range(8)]
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


# ------------------------------------------------------- pages and tables --

def test_bad_page_of_a_very_large_page_size():
    """Length and page size whose sum passes 2^31: the page is looked at."""
    ps, n = 1_200_000_000, 1_100_000_000
    cache = torch.zeros(1, ps, 1, 1, dtype=torch.bfloat16, device="cuda")
    new = torch.ones(2, 1, 1, 1, dtype=torch.bfloat16, device="cuda")
    r = mtp.mtp_tree_attention(new, new, new, cache, cache, torch.tensor([[0], [-1]], dtype=i32, device="cuda"),
                               torch.tensor([n, n], dtype=i32, device="cuda"), with_lse=True)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0, mtp.ROW_BAD_ID]
    assert r.out[1].isnan().all() and r.lse[1].isnan().all()
    # n keys of score 0 and one of score 1; sums of float32 in a few thousand parts
    want = math.log(n + math.e)
    assert abs(r.lse[0].item() - want) < 1e-4 and 0 <= r.out[0].item() < 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, D, ps", [(1, 128, 16), (9, 64, 64), (40, 128, 24), (3, 256, 256)])
def test_table_wider_than_the_text(dtype, T, D, ps):
    """A table for the longest text a server allows, what lies behind a
    sequence's pages no page numbers at all."""
    x = attn_case(T + D, dtype, 3, T, 8, 2, D, ps, [0, 70, 333])
    good = on_gpu(x)
    plain = mtp.mtp_tree_attention(**good, with_lse=True)
    check_attention(x, plain.out, None, plain.lse)
    wide = torch.full((3, 8192 // ps), -7, dtype=i32)
    wide[1::2] = 1 << 30
    for b in range(3):
        n = -(-int(x["cache_len"][b]) // ps)
        wide[b, :n] = x["page_table"][b, :n]
    r = mtp.mtp_tree_attention(**dict(good, page_table=wide.cuda()), with_lse=True)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0, 0, 0]
    check_attention(x, r.out, None, r.lse)


# ------------------------------------------------- graphs and the chain's way --

def test_commit_and_reorder_graphs_and_streams():
    """Captured once and replayed with other tokens, parents and lengths, and
    the same on a given stream."""
    x = commit_case(21, "bf16", 2, 3, 12, 2, 64, 16, [3, 16, 40], 0.7)
    g = on_gpu(x)
    first = {k: g[k].clone() for k in ("k_cache", "v_cache")}
    states, up = torch.randn(2, 3, 4, 33, device="cuda"), torch.zeros(3, 4, dtype=i32, device="cuda")
    mtp.mtp_tree_commit(**g)
    mtp.mtp_beam_reorder(states, up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mtp.mtp_tree_commit(**g)
        s = mtp.mtp_beam_reorder(states, up)
    side = torch.cuda.Stream()
    for seed in range(3):
        y = commit_case(100 + seed, "bf16", 2, 3, 12, 2, 64, 16, [3, 16, 40], 0.7)
        for k in ("tokens", "target_tokens", "parents"):
            g[k].copy_(y[k])
            x[k] = y[k]
        x["cache_len"] = torch.tensor([seed, 40 - seed, 20], dtype=i32)
        g["cache_len"].copy_(x["cache_len"])
        up.copy_(torch.randint(0, 4, (3, 4)))
        for run in (graph.replay, None):
            for k in first:
                g[k].copy_(first[k])
            torch.cuda.synchronize()
            if run:
                run()
                got, moved = r, s
            else:
                got, moved = mtp.mtp_tree_commit(**g, stream=side), mtp.mtp_beam_reorder(states, up, stream=side)
            torch.cuda.synchronize()
            check_commit(dict(x, k_cache=first["k_cache"].cpu(), v_cache=first["v_cache"].cpu()),
                         mtp.CommitResult(*(t.cpu() for t in got)), g["k_cache"], g["v_cache"])
            want = torch.stack([states[:, b, up[b].long()] for b in range(3)], 1)
            assert torch.equal(moved.states, want) and got.row_flags.tolist() == moved.row_flags.tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chain_verified_by_rejection_sampling_and_committed(dtype):
    """mtp_rs_verify decides how many drafts of a chain stand; its tokens are
    the commit's target tokens, and accept_len + 1 its nodes."""
    B, gamma, V, Hkv, D, ps = 24, 5, 4099, 2, 64, 16
    g = torch.Generator().manual_seed(11)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    target = torch.randn(B, gamma + 1, V, generator=g) * 2
    draft = target[:, :gamma] + 0.4 * torch.randn(B, gamma, V, generator=g)
    target, draft = target.to(dt), draft.to(dt)
    ids = torch.distributions.Categorical(logits=draft.float()).sample().to(i32)
    u = torch.rand(B, gamma + 1, generator=g)
    bad = target.clone()
    bad[5, 0, 7] = math.nan                       # a flagged sequence commits nothing
    v = mtp.mtp_rs_verify(bad.cuda(), draft.cuda(), ids.cuda(), torch.ones(B).cuda(), u.cuda())
    x = commit_case(31, dtype, 2, B, gamma + 1, Hkv, D, ps, [(7 * b) % 50 for b in range(B)], tree="chain")
    x["tokens"] = torch.cat([torch.full((B, 1), 9, dtype=i32), ids], 1)
    x["target_tokens"] = v.tokens.cpu()
    x["n_nodes"] = v.accept_len.cpu() + 1
    c = on_gpu(x)
    r = mtp.mtp_tree_commit(c["tokens"], v.tokens, None, c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], c["page_table"],
                            c["cache_len"], v.accept_len + 1)
    torch.cuda.synchronize()
    check_commit(x, mtp.CommitResult(*(t.cpu() for t in r)), c["k_cache"], c["v_cache"])
    assert torch.equal(r.accept_len, v.accept_len) and torch.equal(r.tokens, v.tokens)
    assert r.row_flags.tolist() == [0] * B and v.accept_len.tolist()[5] == -1
    assert len(set(v.accept_len.tolist())) > 3    # rejections at several places, and none


# ------------------------------------------------------------- precision --

@pytest.mark.parametrize("B, T, Hq, Hkv, D, L", [(1, 1, 8, 8, 64, 60013), (24, 1, 8, 8, 64, 1900), (2, 4, 8, 2, 128, 5001)])
def test_float32_keeps_its_bits(B, T, Hq, Hkv, D, L):
    """The error of all outputs together, relative to their size.  With random
    values it is that of a weight, and u = 2^-24: a score of size 2, in two sums
    of D / 2 roundings of at most u of it (uniform, so u / sqrt 3 each, on
    partial sums of half its square on average), 2 u sqrt(D / 12) = 2.8e-7 or
    3.9e-7; the exponent, up to 17, rounded once, 17 u ln 2 / sqrt 3 = 4.1e-7;
    the power's two units, 1.2e-7; the output's sums of 64 and then of a few
    hundred tiles, less than 2e-7: together below 6.5e-7.  The bound is half as
    much again."""
    x = attn_case(B + L, "f32", B, T, Hq, Hkv, D, 16, [L] * B, "chain")
    g = on_gpu(x)
    r = mtp.mtp_tree_attention(**g)
    torch.cuda.synchronize()
    far = size = 0.0
    for b in range(B):
        at = torch.arange(L, device="cuda")
        page, row = g["page_table"][b].long()[at // 16], at % 16
        K = torch.cat([g["k_cache"][page, row], g["k_new"][b]]).double()
        V = torch.cat([g["v_cache"][page, row], g["v_new"][b]]).double()
        q = g["q"][b].double().view(T, Hkv, Hq // Hkv, D)
        s = torch.einsum("thgd,shd->thgs", q, K) * D ** -0.5
        s[..., L:] += torch.full((T, T), -math.inf, device="cuda", dtype=torch.float64).triu(1)[:, None, None]
        o = torch.einsum("thgs,shd->thgd", torch.softmax(s, -1), V).reshape(T, Hq, D)
        far += (r.out[b].double() - o).square().sum().item()
        size += o.square().sum().item()
    assert math.sqrt(far / size) < 1e-6


@pytest.mark.parametrize("dtype, T, D", [("bf16", 1, 64), ("bf16", 9, 128), ("bf16", 40, 64), ("bf16", 3, 256), ("f32", 1, 64), ("f32", 9, 96)])
def test_scores_up_to_2_to_the_29(dtype, T, D):
    """Queries and keys of whole numbers, a scale of 2^21 and scores of up to
    2^21 D: every row is the mean of the values whose keys have its largest score.
    The products with log2(e) round by up to 16 there, in all weights of a row
    alike; what is left is the sum of the weights' and the output's rounding."""
    x = attn_case(D + T, dtype, 2, T, 8, 2, D, 16, [700, 33], "random")
    g = torch.Generator().manual_seed(D)
    for k in ("q", "k_new", "k_cache"):
        x[k] = torch.randint(-1, 2, x[k].shape, generator=g).to(x[k].dtype)
    r = mtp.mtp_tree_attention(**on_gpu(x), scale=2.0 ** 21, with_lse=True)
    torch.cuda.synchronize()
    half = torch.finfo(x["q"].dtype).eps / 2
    for b in range(2):
        n = int(x["cache_len"][b])
        at = torch.arange(n)
        page, row = x["page_table"][b].long()[at // 16], at % 16
        see = torch.cat([torch.ones(T, n, dtype=torch.bool), tree_ref.ancestors(x["parents"][b].tolist(), T)], 1)
        for hq in range(8):
            K = torch.cat([x["k_cache"][page, row, hq // 4], x["k_new"][b, :, hq // 4]]).double()
            V = torch.cat([x["v_cache"][page, row, hq // 4], x["v_new"][b, :, hq // 4]]).double()
            s = (x["q"][b, :, hq].double() @ K.T).masked_fill(~see, -math.inf)
            top = s.amax(1, keepdim=True)
            w = (s == top).double()
            w = w / w.sum(1, keepdim=True)
            want, mass = w @ V, w @ V.abs()
            assert ((r.out[b, :, hq].double().cpu() - want).abs() <= 2.1 * half * mass + 2.0 ** -20 * mass).all()
            assert ((r.lse[b, :, hq].double().cpu() - top[:, 0] * 2.0 ** 21).abs() <= 2.0 ** -22 * (top[:, 0] * 2.0 ** 21).abs() + 10).all()
