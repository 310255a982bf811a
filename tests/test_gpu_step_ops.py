"""Rotary positions, cache append and logit adjustment on the GPU against plain
64-bit forms (tests/step_ref.py, which derives the tolerances)."""
import math
import random

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from tests import step_ref

pytestmark = pytest.mark.gpu
i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
DTYPES = {"f32": f32, "bf16": bf16}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


def near(got, want, tol):
    """Every element within its bound; NaN and infinities equal."""
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, torch.zeros_like(got), (got - want).abs())
    bad = ~(off <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), float((off / tol.clamp(min=1e-300))[bad].max()))


# ------------------------------------------------------------------ rope --

ROPE = [
    # dtype, B, T, Hq, Hkv, D, pairs, interleaved
    ("bf16", 1, 1, 1, 1, 64, 32, False),
    ("bf16", 2, 3, 8, 2, 128, 64, False),
    ("bf16", 2, 3, 8, 2, 128, 64, True),
    ("bf16", 3, 17, 5, 1, 96, 32, False),
    ("bf16", 3, 17, 5, 1, 96, 32, True),
    ("bf16", 1, 9, 32, 8, 256, 128, False),
    ("bf16", 2, 5, 3, 3, 80, 13, False),
    ("bf16", 2, 5, 3, 3, 80, 13, True),
    ("bf16", 1, 4, 4, 1, 33, 16, False),
    ("bf16", 1, 3, 2, 1, 255, 1, True),
    ("bf16", 4, 700, 2, 1, 64, 32, False),
    ("f32", 1, 1, 1, 1, 2, 1, False),
    ("f32", 2, 6, 8, 2, 96, 32, True),
    ("f32", 2, 6, 8, 2, 96, 48, False),
    ("f32", 1, 7, 3, 2, 100, 25, False),
    ("f32", 1, 7, 3, 2, 1, 0, False),
    ("f32", 3, 900, 2, 1, 36, 4, True),
]


def rope_case(seed, dtype, B, T, Hq, Hkv, D, n, far=100000):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    q, k = torch.randn(B, T, Hq, D, generator=g).to(dt), torch.randn(B, T, Hkv, D, generator=g).to(dt)
    pos = torch.randint(0, far, (B, T), generator=g, dtype=i32)
    return q, k, pos, torch.tensor([10000.0 ** (-i / max(n, 1)) for i in range(n)], dtype=f32)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c)))
def test_rope(case, inverse):
    dtype, B, T, Hq, Hkv, D, n, pairs = case
    q, k, pos, freq = rope_case(D + T, dtype, B, T, Hq, Hkv, D, n)
    r = mtp.mtp_rope(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), interleaved=pairs, factor=1.25, inverse=inverse)
    alone = mtp.mtp_rope(k.cuda(), None, pos.cuda(), freq.cuda(), interleaved=pairs, factor=1.25, inverse=inverse)
    torch.cuda.synchronize()
    near(r.q, *step_ref.rope(q, pos, freq, pairs, 1.25, inverse))
    near(r.k, *step_ref.rope(k, pos, freq, pairs, 1.25, inverse))
    assert alone.k is None and torch.equal(alone.q, r.k)


@pytest.mark.parametrize("positions", [[0, 1, 2 ** 24 + 1, 2 ** 31 - 1], [-1, -12345, -2 ** 31, 123456789]])
def test_rope_far_positions(positions):
    """Positions whose product with a frequency no float32 holds, and negative ones."""
    q, k, _, _ = rope_case(1, "f32", 1, 4, 2, 1, 64, 32)
    pos = torch.tensor([positions], dtype=i32)
    freq = torch.tensor([1.0, 0.99999994, 0.5, 1e-4, 1e-8, 1e-38, 1e-42, 0.0, -0.3] + [0.7 ** i for i in range(23)], dtype=f32)
    r = mtp.mtp_rope(q.cuda(), k.cuda(), pos.cuda(), freq.cuda())
    near(r.q, *step_ref.rope(q, pos, freq))
    near(r.k, *step_ref.rope(k, pos, freq))


def test_rope_frequency_that_is_no_number():
    q, k, pos, freq = rope_case(2, "f32", 1, 3, 2, 1, 16, 4)
    freq[1], freq[2] = math.inf, math.nan
    r = mtp.mtp_rope(q.cuda(), k.cuda(), pos.cuda(), freq.cuda()).q.cpu()
    lost = torch.tensor([i % 8 in (1, 2, 5, 6) and i < 8 for i in range(16)])
    assert r[..., lost].isnan().all() and not r[..., ~lost].isnan().any()
    assert torch.equal(r[..., 8:], q[..., 8:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_rope_is_its_inverse_and_gradient(dtype, pairs):
    """The inverse takes a rotation back, and it is the gradient: <g, rope(x + d)
    - rope(x - d)> = 2 <inverse(g), d>, rope being linear."""
    q, _, pos, freq = rope_case(3, dtype, 2, 40, 4, 1, 64, 24)
    a = [t.cuda() for t in (pos, freq)]
    there = mtp.mtp_rope(q.cuda(), None, *a, interleaved=pairs).q
    back = mtp.mtp_rope(there, None, *a, interleaved=pairs, inverse=True).q
    # each way is off by at most the bound of step_ref.rope
    size = q.double().abs().amax()
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    assert (back.double().cpu() - q.double()).abs().max() <= 2.01 * size * 2 * (16 * step_ref.U + eps)
    if dtype == "f32":
        g = torch.Generator().manual_seed(4)
        d, w = torch.randn(q.shape, generator=g), torch.randn(q.shape, generator=g)
        up, down = (mtp.mtp_rope((q + s * d).cuda(), None, *a, interleaved=pairs).q.double().cpu() for s in (1, -1))
        grad = mtp.mtp_rope(w.cuda(), None, *a, interleaved=pairs, inverse=True).q.double().cpu()
        left, right = (w.double() * (up - down)).sum(), 2 * (grad * d.double()).sum()
        scale = (w.abs().double() * (up.abs() + down.abs())).sum() + 2 * (grad.abs() * d.abs().double()).sum()
        assert abs(left - right) <= 32 * step_ref.U * scale


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_strides_and_places(dtype):
    """Parts of a projection, other orders, addresses off 16 bytes, positions of
    one row for all, outputs in place and into a new projection."""
    q, k, pos, freq = rope_case(5, dtype, 3, 6, 4, 2, 64, 24)
    want = mtp.mtp_rope(q.cuda(), k.cuda(), pos.cuda(), freq.cuda())
    qkv = torch.cat([q, k, k], 2).cuda()
    out = torch.full_like(qkv, 7.0)
    mtp.mtp_rope(qkv[:, :, :4], qkv[:, :, 4:6], pos.cuda(), freq.cuda(), out=mtp.RopeResult(out[:, :, :4], out[:, :, 4:6]))
    assert torch.equal(out[:, :, :4], want.q) and torch.equal(out[:, :, 4:6], want.k) and (out[:, :, 6:] == 7).all()
    here = qkv.clone()
    mtp.mtp_rope(here[:, :, :4], here[:, :, 4:6], pos.cuda(), freq.cuda(), out=mtp.RopeResult(here[:, :, :4], here[:, :, 4:6]))
    assert torch.equal(here[:, :, :6], out[:, :, :6]) and torch.equal(here[:, :, 6:], qkv[:, :, 6:])
    swapped = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    odd = torch.zeros(3, 6, 2, 67, dtype=q.dtype, device="cuda")[..., 1:65]
    odd.copy_(k)
    r = mtp.mtp_rope(swapped, odd, pos.cuda(), freq.cuda())
    assert torch.equal(r.q, want.q) and torch.equal(r.k, want.k)
    row = pos[:1].cuda()
    r = mtp.mtp_rope(q.cuda(), None, row.expand(3, 6), freq.cuda())
    assert torch.equal(r.q, mtp.mtp_rope(q.cuda(), None, row.repeat(3, 1), freq.cuda()).q)


def test_rope_empty():
    e = torch.zeros(0, 3, 2, 64, device="cuda")
    assert mtp.mtp_rope(e, e, torch.zeros(0, 3, dtype=i32, device="cuda"), torch.ones(8, device="cuda")).q.shape == e.shape
    e = torch.zeros(2, 0, 2, 64, device="cuda")
    assert mtp.mtp_rope(e, None, torch.zeros(2, 0, dtype=i32, device="cuda"), torch.ones(8, device="cuda")).q.shape == e.shape


def test_rope_memory_that_meets_is_refused():
    x = torch.zeros(2, 4, 4, 64, device="cuda")
    p, f = torch.zeros(2, 4, dtype=i32, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(mtp.MTPError):
        mtp.mtp_rope(x[:, :3], None, p[:, :3], f, out=mtp.RopeResult(x[:, 1:], None))
    with pytest.raises(mtp.MTPError):  # every token into one place
        mtp.mtp_rope(x, None, p, f, out=mtp.RopeResult(torch.zeros(2, 1, 4, 64, device="cuda").expand(2, 4, 4, 64), None))


# ---------------------------------------------------------------- append --

def append_case(seed, dtype, B, T, Hq, Hkv, D, n, page, lens, news):
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    q, k, _, freq = rope_case(seed, dtype, B, T, Hq, Hkv, D, n)
    v = torch.randn(k.shape, generator=g).to(k.dtype)
    P = max(1, -(-max(a + b for a, b in zip(lens, news)) // page))
    ids = list(range(B * P + 2))
    rng.shuffle(ids)
    cache = [torch.randn(B * P + 2, page, Hkv, D, generator=g).to(k.dtype) for _ in range(2)]
    return dict(q=q, k=k, v=v, inv_freq=freq, k_cache=cache[0], v_cache=cache[1], page_table=torch.tensor(ids[:B * P], dtype=i32).view(B, P),
                cache_len=torch.tensor(lens, dtype=i32), n_new=torch.tensor(news, dtype=i32))


def check_append(x, r, kc, vc, positions=None, interleaved=False, factor=1.0, fill=7.0):
    B, T = x["k"].shape[:2]
    ps = kc.shape[1]
    pos = x["cache_len"][:, None] + torch.arange(T, dtype=i32) if positions is None else positions
    q, q_tol = step_ref.rope(x["q"], pos, x["inv_freq"], interleaved, factor)
    k, k_tol = step_ref.rope(x["k"], pos, x["inv_freq"], interleaved, factor)
    K, V, K_tol = x["k_cache"].double().clone(), x["v_cache"].clone(), torch.zeros(x["k_cache"].shape, dtype=torch.float64)
    for b in range(B):
        n, m = int(x["cache_len"][b]), int(x["n_new"][b])
        at = torch.arange(n, n + m)
        page = x["page_table"][b].long()[at // ps]
        K[page, at % ps], K_tol[page, at % ps], V[page, at % ps] = k[b, :m], k_tol[b, :m], x["v"][b, :m]
        for got, want, tol in ((r.q, q, q_tol), (r.k, k, k_tol)):
            if got is not None:
                near(got[b, :m], want[b, :m], tol[b, :m])
                assert (got[b, m:] == fill).all()
    near(kc, K, K_tol)
    assert torch.equal(vc.cpu(), V)
    assert r.cache_len.tolist() == (x["cache_len"] + x["n_new"]).tolist()


def run_append(x, **kw):
    g = {k: v.cuda() for k, v in x.items()}
    out = mtp.AppendResult(torch.full_like(g["cache_len"], 99), torch.full_like(g["q"], 7.0), torch.full_like(g["k"], 7.0),
                           torch.full_like(g["cache_len"], 99))
    r = mtp.mtp_cache_append(**g, out=out, **{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * len(x["cache_len"])
    check_append(x, r, g["k_cache"], g["v_cache"], **kw)
    return r, g


@pytest.mark.parametrize("case", [
    ("bf16", 1, 1, 4, 1, 128, 64, 16, [0], [1]),
    ("bf16", 3, 4, 8, 2, 128, 64, 16, [15, 16, 100], [4, 1, 0]),
    ("bf16", 2, 100, 2, 2, 96, 24, 24, [5, 47], [100, 33]),
    ("bf16", 2, 5, 3, 1, 50, 9, 7, [6, 20], [5, 2]),
    ("bf16", 5, 900, 1, 1, 64, 32, 64, [0, 1, 63, 64, 1000], [900, 0, 1, 899, 64]),
    ("f32", 2, 3, 4, 2, 64, 16, 1, [3, 0], [3, 2]),
    ("f32", 2, 300, 2, 1, 256, 128, 128, [127, 400], [300, 129]),
], ids=lambda c: "-".join(map(str, c[:8])))
@pytest.mark.parametrize("interleaved", [False, True])
def test_cache_append(case, interleaved):
    run_append(append_case(len(case[8]) + case[2], *case), interleaved=interleaved, factor=0.75)


def test_cache_append_given_positions():
    """Positions of their own (behind a shared prefix, say), and no rotation."""
    x = append_case(9, "bf16", 3, 4, 4, 2, 64, 32, 16, [15, 16, 100], [4, 1, 0])
    run_append(x, positions=x["cache_len"][:, None] + torch.arange(4, dtype=i32) + 5000)
    g = {k: v.cuda() for k, v in x.items() if k not in ("q", "inv_freq")}
    r = mtp.mtp_cache_append(**g, with_keys=True)
    plain = dict(x, inv_freq=x["inv_freq"][:0])
    assert r.q is None and r.row_flags.tolist() == [0, 0, 0]
    for b, m in enumerate(x["n_new"].tolist()):
        assert torch.equal(r.k[b, :m].cpu(), x["k"][b, :m])
    check_append(plain, mtp.AppendResult(r.cache_len, None, None, None), g["k_cache"], g["v_cache"])


def test_cache_append_strides():
    """Parts of one projection in place, caches with heads outside the tokens or
    keys and values in one tensor, addresses off 16 bytes."""
    x = append_case(10, "bf16", 3, 4, 4, 2, 64, 32, 16, [15, 16, 100], [4, 1, 3])
    a, g = run_append(x)
    for make in (lambda c: c.transpose(1, 2).contiguous().transpose(1, 2), lambda c: torch.stack([c, c], 1)[:, 0],
                 lambda c: torch.cat([c, c], 3)[..., 1:65].copy_(c)):
        kc, vc = (make(x[n].cuda()) for n in ("k_cache", "v_cache"))
        qkv = torch.cat([x["q"], x["k"], x["v"]], 2).cuda()
        q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
        r = mtp.mtp_cache_append(k, v, kc, vc, g["page_table"], g["cache_len"], g["n_new"], q=q, inv_freq=g["inv_freq"],
                                 out=mtp.AppendResult(torch.zeros_like(a.cache_len), q, k, None))
        assert torch.equal(kc, g["k_cache"]) and torch.equal(vc, g["v_cache"])
        for b, m in enumerate(x["n_new"].tolist()):
            assert torch.equal(r.q[b, :m], a.q[b, :m]) and torch.equal(r.k[b, :m], a.k[b, :m])
            assert torch.equal(r.q[b, m:].cpu(), x["q"][b, m:])


def test_cache_append_flags():
    """Bad lengths, counts and room: nothing is written.  A bad page: the
    sequence keeps its length, nothing of the other sequences changes."""
    x = append_case(11, "bf16", 6, 5, 2, 1, 64, 32, 16, [3, 40, 30, 3, 14, 60], [5] * 6)
    cap = x["page_table"].shape[1] * 16
    good, _ = run_append(x)
    x["cache_len"][1], x["n_new"][2], x["cache_len"][3], x["page_table"][4, 1] = -1, 6, cap - 4, x["k_cache"].shape[0]
    x["page_table"][5, 0] = -7  # not among the pages of its new tokens
    g = {k: v.cuda() for k, v in x.items()}
    q = torch.full_like(g["q"], 7.0)
    r = mtp.mtp_cache_append(**g, out=mtp.AppendResult(torch.zeros_like(g["cache_len"]), q, None, torch.zeros_like(g["cache_len"])))
    torch.cuda.synchronize()
    bad = mtp.ROW_BAD_ID
    assert r.row_flags.tolist() == [0, bad, bad, bad, bad, 0]
    assert r.cache_len.tolist() == [8, -1, 30, cap - 4, 14, 65]
    assert (q[1:4] == 7).all() and torch.equal(q[0], good.q[0]) and torch.equal(q[4], good.q[4])
    touched = torch.zeros(x["k_cache"].shape[:2], dtype=torch.bool)
    for b, at in ((0, range(3, 8)), (4, range(14, 16)), (5, range(60, 65))):
        for t in at:
            touched[int(x["page_table"][b, t // 16]), t % 16] = True
    same = (g["k_cache"].cpu() == x["k_cache"]).all(-1).all(-1) & (g["v_cache"].cpu() == x["v_cache"]).all(-1).all(-1)
    assert torch.equal(same, ~touched)


def test_cache_append_far_pages():
    """Pages beyond 2^32 elements of the caches."""
    pages = (1 << 32) // (16 * 2 * 128) + 4
    kc = torch.zeros(pages, 16, 2, 128, dtype=bf16, device="cuda")
    x = append_case(12, "bf16", 1, 3, 2, 2, 128, 64, 16, [15], [3])
    table = torch.tensor([[pages - 1, pages - 2]], dtype=i32, device="cuda")
    g = {k: v.cuda() for k, v in x.items()}
    want, near_by = run_append(x)
    g.update(k_cache=kc, v_cache=kc.clone(), page_table=table)
    mtp.mtp_cache_append(**g)
    for n in ("k_cache", "v_cache"):
        for t in range(15, 18):
            assert torch.equal(g[n][table[0, t // 16].long(), t % 16], near_by[n][x["page_table"][0, t // 16].long(), t % 16])
    assert g["k_cache"].count_nonzero() <= 3 * 2 * 128


# ---------------------------------------------------------------- adjust --

def adjust_case(seed, dtype, B, S, V, L, tree=False, bias=0, mask=False, nodes=None):
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    words = lambda *s: (V ** torch.rand(*s, generator=g) - 1).int().clamp(0, V - 1)  # noqa: E731
    x = dict(logits=(torch.randn(B, S, V, generator=g) * 4).to(DTYPES[dtype]), history=words(B, L),
             history_len=torch.tensor([rng.randint(0, L) for _ in range(B)], dtype=i32), tokens=words(B, S),
             repetition=1 + torch.rand(B, generator=g), frequency=torch.rand(B, generator=g) - 0.3, presence=torch.rand(B, generator=g) - 0.3)
    x["prompt_len"] = torch.tensor([rng.randint(0, int(n)) for n in x["history_len"]], dtype=i32)
    x["parents"] = torch.tensor([[-1] + [rng.randint(-1, i - 1) for i in range(1, S)] for _ in range(B)], dtype=i32) if tree else None
    x["n_nodes"] = None if nodes is None else torch.tensor(nodes, dtype=i32)
    x["bias_ids"], x["bias"] = (words(B, bias), torch.randn(B, bias, generator=g)) if bias else (None, None)
    if bias > 3:
        x["bias_ids"][:, 1] = -1
        x["bias_ids"][:, 2:4] = x["bias_ids"][:, :1]
    x["mask"] = None
    if mask:
        x["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, S, (V + 31) // 32), generator=g).int()
        x["mask"][0, 0] = 0
        x["mask"][-1, -1] = -1
    return x


def run_adjust(x, in_place=False):
    g = {k: None if v is None else v.cuda() for k, v in x.items()}
    z = g["logits"]
    out = mtp.AdjustResult(z if in_place else torch.full_like(z, 7.0), torch.full((z.shape[0],), 99, dtype=i32, device="cuda"))
    r = mtp.mtp_adjust_logits(**g, out=out)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * z.shape[0]
    want, tol, live = step_ref.adjust(x["logits"], x["history"], x["history_len"], x["prompt_len"], x["tokens"], x["parents"], x["n_nodes"],
                                      x["repetition"], x["frequency"], x["presence"], x["bias_ids"], x["bias"], x["mask"])
    near(r.logits[live.cuda()], want[live], tol[live])
    left = r.logits.cpu()[~live]
    assert torch.equal(left, x["logits"][~live]) if in_place else (left == 7).all()
    return r


ADJUST = [
    # dtype, B, S, V, L, tree, bias, mask, nodes
    ("bf16", 1, 1, 1, 1, False, 0, False, None),
    ("bf16", 2, 3, 5, 9, False, 2, True, None),
    ("bf16", 2, 4, 151936, 3000, False, 0, False, None),
    ("bf16", 1, 2, 50257, 100, True, 12, True, None),
    ("bf16", 3, 7, 1031, 40, True, 5, True, [7, 0, 3]),
    ("bf16", 40, 2, 9000, 500, False, 20, True, None),
    ("bf16", 2, 64, 4099, 77, True, 0, True, None),
    ("bf16", 2, 33, 2048, 64, False, 8, False, [33, 12]),
    ("f32", 1, 1, 31, 0, False, 3, True, None),
    ("f32", 2, 5, 33, 70, True, 0, True, None),
    ("f32", 2, 4, 32000, 2001, False, 1024, True, None),
    ("f32", 3, 6, 50257, 999, True, 300, False, [6, 1, 0]),
    ("f32", 70, 1, 8193, 64, False, 0, True, None),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", ADJUST, ids=lambda c: "-".join(map(str, c[:8])))
def test_adjust_logits(case, in_place):
    run_adjust(adjust_case(case[3] + case[2], *case), in_place)


@pytest.mark.parametrize("seed", range(20))
def test_adjust_logits_random(seed):
    rng = random.Random(seed)
    B, S, V, L = rng.randint(1, 9), rng.choice([1, 2, 5, 16, 64]), rng.randint(1, 20000), rng.randint(0, 600)
    x = adjust_case(seed, rng.choice(["bf16", "f32"]), B, S, V, L, rng.random() < 0.5, rng.choice([0, 1, 50]), rng.random() < 0.5,
                    [rng.randint(0, S) for _ in range(B)] if rng.random() < 0.5 else None)
    for name in ("prompt_len", "tokens", "repetition", "frequency", "presence"):
        if rng.random() < 0.2:
            x[name] = None
    if x["tokens"] is None:
        x["parents"] = None
    run_adjust(x, rng.random() < 0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adjust_logits_alone(dtype):
    """Each part on its own, and none: the logits unchanged, bit for bit."""
    x = adjust_case(50, dtype, 2, 3, 3001, 50, bias=4, mask=True)
    none = mtp.mtp_adjust_logits(x["logits"].cuda())
    assert torch.equal(none.logits.cpu(), x["logits"])
    keys = dict.fromkeys(x)
    for names in (("mask",), ("bias_ids", "bias"), ("history", "history_len", "repetition"), ("tokens", "presence"),
                  ("history", "history_len", "prompt_len", "frequency")):
        y = dict(keys, logits=x["logits"], **{n: x[n] for n in names})
        run_adjust(y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adjust_logits_of_no_number(dtype):
    """Infinities and NaN pass through where they are allowed; a masked NaN is
    -inf; a text of one word; empty places; nothing allowed."""
    x = adjust_case(51, dtype, 2, 4, 1000, 5000, bias=6, mask=True)
    x["history"][0], x["history_len"][0], x["prompt_len"][0] = 17, 5000, 3
    x["history"][1, ::3], x["tokens"][1, 0], x["tokens"][1, 2] = -1, -1, -5
    z = x["logits"]
    z[:, :, 10::7], z[:, :, 11::7], z[:, :, 12::7] = math.nan, -math.inf, math.inf
    z[:, :, 17] = 3.0
    lowest = torch.finfo(z.dtype).min
    z[1, :, 13::7] = lowest
    x["repetition"][1], x["frequency"][1], x["presence"][1] = 1.0, 0.0, 0.0  # (the lowest value stays one)
    x["bias_ids"][1] = 13
    x["mask"][0, 1], x["mask"][1] = 0, -1
    r = run_adjust(x)
    assert (r.logits[0, 1] == -math.inf).all()


def test_adjust_logits_shared_mask():
    """One mask for all sequences or all rows by strides of 0, words of a wider row."""
    x = adjust_case(52, "bf16", 3, 4, 777, 60, mask=True)
    g = {k: None if v is None else v.cuda() for k, v in x.items()}
    m, W = g["mask"], x["mask"].shape[2]
    for part in (m[:1].expand(3, 4, W), m[:, :1].expand(3, 4, W), torch.cat([m, m], 2)[:, :, 3:3 + W], m.transpose(0, 1)[:3, :3].expand(3, 3, W)):
        rows = dict(g, mask=part)
        if part.shape[1] == 3:
            rows.update(logits=g["logits"][:, :3].contiguous(), tokens=g["tokens"][:, :3].contiguous())
        assert not part.is_contiguous()
        assert torch.equal(mtp.mtp_adjust_logits(**rows).logits, mtp.mtp_adjust_logits(**dict(rows, mask=part.contiguous())).logits)


@pytest.mark.parametrize("in_place", [False, True])
def test_adjust_logits_flags(in_place):
    """Bad sequences are NaN throughout and flagged, the others as without them."""
    x = adjust_case(53, "bf16", 10, 3, 20000, 90, tree=True, bias=4, nodes=[2] * 10)
    x["history_len"][:], x["prompt_len"][:] = 90, 20
    good = run_adjust(x).logits
    g = {k: None if v is None else v.cuda() for k, v in x.items()}
    g["history"][1, 89] = 20000
    g["history_len"][2] = 91
    g["prompt_len"][3] = 91
    g["n_nodes"][4] = 4
    g["parents"][5, 1] = 1
    g["tokens"][6, 1] = 20000
    g["bias_ids"][7, 3] = 2 ** 31 - 1
    g["repetition"][8] = 0.0
    g["presence"][9] = math.nan
    g["tokens"][0, 2] = 20000  # behind the last node: not looked at
    z = g["logits"].clone()
    out = mtp.AdjustResult(z if in_place else torch.full_like(z, 7.0), torch.zeros(10, dtype=i32, device="cuda"))
    r = mtp.mtp_adjust_logits(**dict(g, logits=z), out=out)
    assert r.row_flags.tolist() == [0] + [mtp.ROW_BAD_ID] * 7 + [mtp.ROW_NONFINITE] * 2
    assert r.logits[1:, :2].isnan().all() and r.logits[4].isnan().all() and not r.logits[5, 2].isnan().any()
    assert torch.equal(r.logits[0, :2], good[0, :2])


def test_adjust_logits_is_repeatable():
    x = {k: None if v is None else v.cuda() for k, v in adjust_case(54, "f32", 4, 4, 30000, 2000, bias=900).items()}
    x["bias_ids"] %= 5  # sums of many
    a = mtp.mtp_adjust_logits(**x).logits
    for _ in range(5):
        assert torch.equal(a, mtp.mtp_adjust_logits(**x).logits)


# ------------------------------------------------------- graphs, streams --

def test_step_operators_in_graphs_and_on_streams():
    """Captured calls replayed with other inputs, on two streams at a time, and
    calls on a given stream."""
    x, y = append_case(60, "bf16", 3, 4, 4, 2, 64, 32, 16, [15, 16, 90], [4, 1, 3]), adjust_case(61, "bf16", 3, 4, 9001, 300, bias=3, mask=True)
    g = {k: v.cuda() for k, v in x.items()}
    h = {k: None if v is None else v.cuda() for k, v in y.items()}
    pos = torch.arange(4, dtype=i32, device="cuda") + g["cache_len"][:, None]

    def calls(**kw):
        a = mtp.mtp_cache_append(**g, with_keys=True, **kw)
        return a, mtp.mtp_rope(g["q"], g["k"], pos, g["inv_freq"], **kw), mtp.mtp_adjust_logits(**h, **kw)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, r, z = calls()
    side = torch.cuda.Stream()
    for turn in range(3):
        g["q"].mul_(0.5)
        g["cache_len"].add_(1)
        h["history_len"].sub_(1).clamp_(min=0)
        h["prompt_len"].clamp_(max=0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        a2, r2, z2 = calls(stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert a.row_flags.tolist() == [0, 0, 0] and z.row_flags.tolist() == [0, 0, 0]
        assert torch.equal(a.cache_len, a2.cache_len) and torch.equal(r.q, r2.q) and torch.equal(r.k, r2.k)
        assert torch.equal(z.logits, z2.logits)
        for b, m in enumerate(x["n_new"].tolist()):
            assert torch.equal(a.q[b, :m], a2.q[b, :m]) and torch.equal(a.k[b, :m], a2.k[b, :m])


def test_rope_of_the_longest_sequence():
    """The blocks of a sequence whose tokens end at the last 32-bit number."""
    T = (1 << 31) - 1
    q = torch.empty(1, T, 1, 1, dtype=bf16, device="cuda").uniform_()
    r = mtp.mtp_rope(q, None, torch.zeros(1, 1, dtype=i32, device="cuda").expand(1, T), torch.empty(0, device="cuda"))
    assert torch.equal(r.q.view(torch.int16), q.view(torch.int16))
