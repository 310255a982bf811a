"""Beam selection on the GPU at the edges of its ranges: logits that are no
numbers, masks that leave a few tokens, low temperatures, neighbouring
scores."""
import math

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp

pytestmark = pytest.mark.gpu
i32 = torch.int32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_bad_logit_in_every_vector_of_the_first_rounds(dtype, bad):
    """Whichever warp meets it, and however early: the sequence is flagged."""
    vec = 8 if dtype == "bf16" else 4
    B, V = 1100, 1100 * vec + 3
    z = torch.zeros(B, 1, V, dtype=DTYPES[dtype])
    at = torch.arange(B) * vec + torch.arange(B) % vec
    z[torch.arange(B), 0, at] = bad
    z = torch.cat([z, torch.zeros_like(z[:1])]).cuda()
    scores, T = torch.zeros(B + 1, 1, device="cuda"), torch.ones(B + 1, device="cuda")
    for _ in range(20):
        r = mtp.mtp_beam_select(z, scores, T, 3)
        torch.cuda.synchronize()
        assert r.row_flags.tolist() == [mtp.ROW_NONFINITE] * B + [0]
        assert (r.tokens[:B] == -1).all() and r.tokens[B].tolist() == [0, 1, 2]


def exact_scores(z, scores, T):
    """[B, W, V] float64: scores[w] + ln softmax(z_w / T)(v), from the
    difference to the row's largest logit, so that it holds at any T."""
    x = z.double()
    x = (x - x.amax(2, keepdim=True)) / T.double()[:, None, None]
    x = x - x.exp().sum(2, keepdim=True).log() + scores.double()[:, :, None]
    return x.masked_fill((scores == -math.inf)[:, :, None] | z.isneginf(), -math.inf)


def check_exact(z, scores, T, K, r):
    """Every returned candidate is looked up in the 64-bit scores.

    Within a beam the order is that of the logits, equal ones by index, and
    must be met exactly.  A score is off by at most tol: exponents x = (z -
    max) log2(e) / T by three roundings, 3 |x| 2^-24, which changes a sum that
    holds 2^0 by at most 3 max(x 2^-x) 2^-24 ln 2 < 2^-23 per term's share, x
    itself of terms that weigh (x < 24) by 2^-18; powers 2^-21; sums of fewer
    than 256 terms in a row 2^-16 at the very worst and far less here (100,000
    elements over 256 threads and four sums each: 2^-18); with the output's own
    rounding 2^-16 + 2^-23 |score|.  Between beams candidates closer than two
    such errors may come in either order."""
    exact = exact_scores(z, scores, T)
    B, W, V = z.shape
    for b in range(B):
        tok, par, val = r.tokens[b].tolist(), r.parents[b].tolist(), r.scores[b].tolist()
        n = min(K, int((exact[b] > -math.inf).sum()))
        assert all(p == (-1, -1, -math.inf) for p in zip(tok[n:], par[n:], val[n:])), (b, n, tok, par)
        assert all(0 <= t < V for t in tok[:n]) and all(0 <= p < W for p in par[:n]), (b, tok, par)
        got = [exact[b, p, t].item() for p, t in zip(par[:n], tok[:n])]
        tol = [2.0 ** -16 + 2.0 ** -23 * abs(s) for s in got]
        for s, v, e in zip(got, val, tol):
            v32 = torch.tensor(s).float().item()
            assert v == v32 or abs(v - s) <= e, (b, s, v)
        for i in range(n - 1):
            assert got[i] >= got[i + 1] - tol[i] - tol[i + 1], (b, i, got[i], got[i + 1])
        for w in range(W):
            mine = [t for t, p in zip(tok[:n], par[:n]) if p == w]
            if scores[b, w] == -math.inf:
                assert not mine
                continue
            order = torch.sort(z[b, w].double() + 0.0, descending=True, stable=True).indices[:len(mine) + 1].tolist()
            assert mine == order[:len(mine)], (b, w, mine, order)
            if n == K and n > 0 and len(order) > len(mine):
                left = exact[b, w, order[-1]].item()
                assert left <= got[-1] + tol[-1] + 2.0 ** -16 + 2.0 ** -23 * abs(left), (b, w, left, got[-1])


def select(z, scores, T, K):
    r = mtp.mtp_beam_select(z.cuda(), scores.cuda(), T.cuda(), K)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * z.shape[0]
    r = mtp.BeamResult(*(t.cpu() for t in r))
    check_exact(z, scores, T, K, r)
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [10007, 24576])
def test_three_tokens_left_at_every_border(dtype, V):
    """All but three neighbouring tokens masked, the three at every place
    where a vector, and so a part of a row, may begin."""
    vec, B, K = (8 if dtype == "bf16" else 4), 64, 6
    lse = math.log(math.e + math.e ** 2 + math.e ** 3)
    starts = list(range(vec, V - 1, vec))
    for s0 in range(0, len(starts), B):
        at = torch.tensor((starts[s0:s0 + B] * B)[:B], device="cuda")
        z = torch.full((B, 1, V), -math.inf, dtype=DTYPES[dtype], device="cuda")
        for d in (-1, 0, 1):
            z[torch.arange(B), 0, at + d] = 2.0 + d
        r = mtp.mtp_beam_select(z, torch.zeros(B, 1, device="cuda"), torch.ones(B, device="cuda"), K)
        want = torch.stack([at + 1, at, at - 1] + [torch.full_like(at, -1)] * 3, 1)
        assert torch.equal(r.tokens.long(), want), (s0, r.tokens, want)
        assert (r.scores[:, :3] - torch.tensor([3 - lse, 2 - lse, 1 - lse], device="cuda")).abs().max() < 1e-5
        assert (r.scores[:, 3:] == -math.inf).all() and (r.row_flags == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B, W, V, left", [(1, 1, 5003, 3), (1, 4, 151936, 50), (1, 1, 151936, 8), (16, 5, 50257, 50), (3, 2, 20011, 200),
                                           (1, 64, 9001, 2), (40, 16, 4099, 40)])
def test_few_tokens_left(dtype, B, W, V, left):
    """Grammar masks and top-k filters: -inf but for a few tokens at random."""
    for seed in range(6):
        g = torch.Generator().manual_seed(1000 * V + seed)
        z = torch.full((B, W, V), -math.inf)
        at = torch.randint(V, (B, W, left), generator=g)
        z.scatter_(2, at, torch.randn(B, W, left, generator=g) * 3)
        z = z.to(DTYPES[dtype])
        select(z, -torch.rand(B, W, generator=g).cumsum(1), 0.5 + torch.rand(B, generator=g), min(64, W * V, 1 + 13 * seed))


def test_three_tokens_of_one_row():
    z = torch.full((1, 1, 5003), -math.inf)
    z[0, 0, 2510:2513] = torch.tensor([3.0, 2.0, 1.0])
    assert select(z, torch.zeros(1, 1), torch.ones(1), 6).tokens.tolist() == [[2510, 2511, 2512, -1, -1, -1]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1e30, 100.0, 1e-2, 1e-3, 1e-4, 1e-5, 3e-6, 1e-6, 1e-7, 1e-9, 1e-20, 1e-37, 4e-39, 1e-44])
def test_any_temperature(dtype, T):
    """Down to what stands for greedy: rows with one dominating logit of either
    sign, rows of small numbers, and rows of two equal best ones."""
    g = torch.Generator().manual_seed(7)
    W, V = 6, 20011
    z = torch.randn(4, W, V, generator=g) * 3
    top = torch.randint(V, (W,), generator=g)
    z[0] -= 200                                    # negative rows
    for w in range(W):
        z[0, w, top[w]] = -10.0 - 6.3 * w
        z[1, w, top[w]] = 10.0 + 6.3 * w
    z[2] *= 1e-6
    z[3, :, 17] = z[3, :, 19000] = 39.7
    z = z.to(DTYPES[dtype])
    scores = -torch.rand(4, W, generator=g).cumsum(1)
    r = select(z, scores, torch.full((4,), T), 12)
    if T < 1e-3:  # each beam's best first, in the order of the beams
        first = torch.sort(z[1].double(), descending=True, stable=True, dim=1).indices[:, 0]
        assert r.tokens[1, :W].tolist() == first.tolist() and r.parents[1, :W].tolist() == list(range(W))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_masks_of_the_lowest_value(dtype, T):
    """A mask of the type's lowest number: a row of nothing else is uniform."""
    low = torch.finfo(DTYPES[dtype]).min
    V = 9001
    z = torch.full((3, 2, V), low, dtype=DTYPES[dtype])
    z[1, 0, 5000], z[1, 0, 77] = 1.5, 1.0
    z[1, 1, 8000] = -2.0
    z[2] = torch.randn(2, V).to(z.dtype)
    z[2, :, ::3] = low
    r = select(z, torch.tensor([[0.0, -1.0]] * 3), torch.full((3,), T), 3)
    assert r.tokens[0].tolist() == [0, 1, 2] and r.parents[0].tolist() == [0, 0, 0]
    assert abs(r.scores[0, 0].item() + math.log(V)) < 1e-5


@pytest.mark.parametrize("V", [20011, 151936])
def test_neighbouring_logits_beside_a_large_one(V):
    """Logits of one row that differ by less than a float32 difference to the
    row's largest can tell, the larger one in a later part."""
    z = torch.full((2, 1, V), -100.0)
    z[:, 0, 3] = 12.0
    for b in range(2):
        for i, at in enumerate(range(100, V, V // 7)):
            z[b, 0, at] = 1.0 + i * 2.0 ** -23
    z[1, 0, 3] = 3e4
    r = select(z, torch.zeros(2, 1), torch.ones(2), 8)
    assert r.tokens[0].tolist() == r.tokens[1].tolist() == [3] + sorted(range(100, V, V // 7), reverse=True)[:7]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_whose_scores_float64_does_not_tell_apart(dtype):
    """The larger logit comes first wherever in the row, and the smaller beam
    before it."""
    V, W = 30011, 3
    z = torch.full((2, W, V), -50.0)
    z[0] = 2.0 ** -126 * torch.randint(1, 100, (W, V), generator=torch.Generator().manual_seed(3))
    for i, at in enumerate(range(50, V, 2000)):
        z[1, :, at] = (1 + i) * 2.0 ** -100
    z[1, :, 5] = 1.0
    r = select(z.to(DTYPES[dtype]), torch.zeros(2, W), torch.tensor([1.0, 1.0]), 40)
    assert r.parents[0].tolist() == [0] * 40


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B, W, V, K", [(1, 1, 1, 1), (3, 4, 3, 12), (2, 5, 50257, 64), (1, 4, 151936, 8), (1, 64, 257, 64), (20, 8, 2048, 16),
                                        (70, 3, 8191, 33), (1, 2, 32000, 64), (9, 16, 20011, 32)])
@pytest.mark.parametrize("spread", [0.02, 3.0])
def test_returned_candidates_have_the_scores_they_claim(dtype, B, W, V, K, spread):
    """The ordinary sizes, every returned token looked up; a spread of 0.02
    leaves bfloat16 few different values and float32 close ones."""
    g = torch.Generator().manual_seed(V * K)
    z = (torch.randn(B, W, V, generator=g) * spread).to(DTYPES[dtype])
    select(z, -torch.rand(B, W, generator=g).cumsum(1), 0.2 + 2 * torch.rand(B, generator=g), K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_rows_and_rising_rows(dtype):
    g = torch.Generator().manual_seed(5)
    z = torch.empty(3, 4, 40003)
    z[0] = torch.randint(0, 4, (40003,), generator=g).float()
    z[1] = torch.linspace(-20, 20, 40003)
    z[2] = torch.linspace(20, -20, 40003)
    select(z.to(DTYPES[dtype]), torch.zeros(3, 4), torch.ones(3), 64)
