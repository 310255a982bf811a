"""Refusals of the operators around a verification step, without a GPU: the
binding's checks of its arguments and the C ABI's answers; the frequencies of
rotary positions."""
import ctypes
import math

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from mtp_speculative_decoding_row_gb300 import build as mtp_build
from tests import step_ref

i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    mtp_build.build()


@pytest.fixture(autouse=True)
def no_launch(monkeypatch, request):
    if "lib" in request.fixturenames:
        return

    def no_library(*a, **k):
        raise AssertionError("the library must not be called")

    monkeypatch.setattr(mtp, "load_library", no_library)


@pytest.fixture
def lib():
    mtp_build.build()
    return mtp.load_library()


# --------------------------------------------------------------- binding --

def rope_args(**new):
    a = dict(q=torch.zeros(2, 3, 4, 64), k=torch.zeros(2, 3, 2, 64), positions=torch.zeros(2, 3, dtype=i32), inv_freq=torch.ones(32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    (dict(q=torch.zeros(2, 3, 4, 64, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (dict(q=torch.zeros(6, 4, 64)), ValueError, "dimensions"),
    (dict(q=torch.zeros(2, 3, 4, 257), k=None), ValueError, "elements"),
    (dict(k=torch.zeros(2, 3, 2, 32)), ValueError, "k must|out.k"),
    (dict(k=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)), TypeError, "k must|out.k"),
    (dict(q=torch.zeros(2, 3, 64, 4).transpose(2, 3)), ValueError, "contiguous in its last"),
    (dict(positions=torch.zeros(2, 4, dtype=i32)), ValueError, "positions"),
    (dict(positions=torch.zeros(2, 3, dtype=torch.int64)), TypeError, "positions"),
    (dict(positions=None), ValueError, "positions"),
    (dict(inv_freq=torch.ones(33)), ValueError, "more than pairs"),
    (dict(inv_freq=torch.ones(32, dtype=torch.float64)), TypeError, "inv_freq"),
    (dict(inv_freq=torch.ones(64)[::2]), ValueError, "inv_freq must be contiguous"),
    (dict(factor=math.inf), ValueError, "factor"),
    (dict(factor=1e39), ValueError, "factor"),
    (dict(factor="2"), TypeError, "real number"),
    (dict(out=mtp.RopeResult(torch.zeros(2, 3, 4, 64), None)), ValueError, "out.k is required"),
    (dict(k=None, out=mtp.RopeResult(torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64))), ValueError, "out.k is of no use"),
    (dict(out=mtp.RopeResult(torch.zeros(2, 3, 4, 32), torch.zeros(2, 3, 2, 64))), ValueError, "out.q"),
    ({}, ValueError, "CUDA"),
])
def test_rope_refusals(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_rope(**rope_args(**new))


def append_args(**new):
    a = dict(k=torch.zeros(2, 3, 2, 64), v=torch.zeros(2, 3, 2, 64), k_cache=torch.zeros(5, 16, 2, 64), v_cache=torch.zeros(5, 16, 2, 64),
             page_table=torch.zeros(2, 2, dtype=i32), cache_len=torch.zeros(2, dtype=i32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    (dict(k=torch.zeros(2, 3, 2, 64, dtype=torch.float64)), TypeError, "float32 or bfloat16"),
    (dict(v=torch.zeros(2, 3, 1, 64)), ValueError, "v must"),
    (dict(k_cache=torch.zeros(5, 16, 2, 32)), ValueError, "k_cache"),
    (dict(v_cache=torch.zeros(4, 16, 2, 64)), ValueError, "v_cache"),
    (dict(page_table=torch.zeros(3, 2, dtype=i32)), ValueError, "page_table"),
    (dict(cache_len=torch.zeros(2)), TypeError, "cache_len"),
    (dict(n_new=torch.zeros(3, dtype=i32)), ValueError, "n_new"),
    (dict(q=torch.zeros(2, 3, 4, 64)), ValueError, "q is of no use without inv_freq"),
    (dict(positions=torch.zeros(2, 3, dtype=i32)), ValueError, "positions are of no use"),
    (dict(inv_freq=torch.ones(33)), ValueError, "more than pairs"),
    (dict(inv_freq=torch.ones(8), positions=torch.zeros(2, 2, dtype=i32)), ValueError, "positions"),
    (dict(with_keys=True, out=mtp.AppendResult(torch.zeros(2, dtype=i32), None, None, None)), ValueError, "with_keys needs"),
    (dict(out=mtp.AppendResult(None, None, None, None)), ValueError, "out.cache_len is required"),
    (dict(out=mtp.AppendResult(torch.zeros(2, dtype=i32), torch.zeros(2, 3, 4, 64), None, None)), ValueError, "out.q is of no use"),
    ({}, ValueError, "CUDA"),
])
def test_cache_append_refusals(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_cache_append(**append_args(**new))


def prefix_args(**new):
    a = dict(q=torch.zeros(2, 3, 4, 64), k_new=torch.zeros(2, 3, 2, 64), v_new=torch.zeros(2, 3, 2, 64), k_cache=torch.zeros(5, 16, 2, 64),
             v_cache=torch.zeros(5, 16, 2, 64), prefix_table=torch.zeros(1, 3, dtype=i32), prefix_len=torch.zeros(1, dtype=i32),
             group_start=torch.zeros(2, dtype=i32), page_table=torch.zeros(2, 2, dtype=i32), cache_len=torch.zeros(2, dtype=i32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    (dict(q=torch.zeros(2, 3, 4, 64, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (dict(k_new=torch.zeros(2, 3, 3, 64)), ValueError, "heads"),
    (dict(prefix_table=torch.zeros(0, 3, dtype=i32), prefix_len=torch.zeros(0, dtype=i32), group_start=torch.zeros(1, dtype=i32)), ValueError, "at least one prefix"),
    (dict(prefix_table=torch.zeros(1, 0, dtype=i32)), ValueError, "at least one prefix"),
    (dict(prefix_table=torch.zeros(3, dtype=i32)), ValueError, "prefix_table"),
    (dict(prefix_len=torch.zeros(2, dtype=i32)), ValueError, "prefix_len"),
    (dict(group_start=torch.zeros(1, dtype=i32)), ValueError, "group_start"),
    (dict(group_start=torch.zeros(2, dtype=torch.int64)), TypeError, "group_start"),
    (dict(page_table=torch.zeros(3, 2, dtype=i32)), ValueError, "page_table"),
    (dict(scale=-1.0), ValueError, "scale"),
    (dict(q=torch.zeros(2, 65, 4, 64)), ValueError, "nodes"),
    (dict(with_lse=True, out=mtp.TreeAttentionResult(torch.zeros(2, 3, 4, 64), None, None)), ValueError, "with_lse needs"),
    ({}, ValueError, "CUDA"),
])
def test_prefix_attention_refusals(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_prefix_attention(**prefix_args(**new))


def adjust_args(**new):
    a = dict(logits=torch.zeros(2, 3, 100), history=torch.zeros(2, 7, dtype=i32), history_len=torch.zeros(2, dtype=i32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    (dict(logits=torch.zeros(2, 3, 100, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (dict(logits=torch.zeros(2, 100)), ValueError, "dimensions"),
    (dict(logits=torch.zeros(2, 65, 10)), ValueError, "rows of a sequence"),
    (dict(logits=torch.zeros(2, 100, 3).transpose(1, 2)), ValueError, "logits must be contiguous"),
    (dict(history_len=None), ValueError, "history_len is required"),
    (dict(history=None), ValueError, "of no use without history"),
    (dict(history=None, history_len=None, prompt_len=torch.zeros(2, dtype=i32)), ValueError, "of no use without history"),
    (dict(history=torch.zeros(2, 7)), TypeError, "history"),
    (dict(parents=torch.zeros(2, 3, dtype=i32)), ValueError, "parents are of no use"),
    (dict(tokens=torch.zeros(2, 4, dtype=i32)), ValueError, "tokens"),
    (dict(n_nodes=torch.zeros(1, dtype=i32)), ValueError, "n_nodes"),
    (dict(repetition=torch.ones(2, dtype=torch.float64)), TypeError, "repetition"),
    (dict(presence=torch.ones(3)), ValueError, "presence"),
    (dict(bias=torch.ones(2, 1)), ValueError, "of no use without each other"),
    (dict(bias_ids=torch.zeros(2, 1, dtype=i32), bias=torch.ones(2, 2)), ValueError, "bias"),
    (dict(bias_ids=torch.zeros(2, 1025, dtype=i32), bias=torch.ones(2, 1025)), ValueError, "at most 1024"),
    (dict(mask=torch.zeros(2, 3, 3, dtype=i32)), ValueError, "mask"),
    (dict(mask=torch.zeros(2, 3, 4)), TypeError, "mask"),
    (dict(out=mtp.AdjustResult(torch.zeros(2, 3, 99), None)), ValueError, "out.logits"),
    ({}, ValueError, "CUDA"),
])
def test_adjust_logits_refusals(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_adjust_logits(**adjust_args(**new))


# ----------------------------------------------------------------- C ABI --

P, L, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float


class Rope(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k", "q_out", "k_out", "positions", "inv_freq")] + \
        [(n, L * 3) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")] + [("pos_stride", L * 2)] + \
        [(n, I) for n in ("dtype", "B", "T", "Hq", "Hkv", "D", "pairs", "interleaved", "inverse")] + [("factor", F)]


class Append(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k", "v", "q_out", "k_out", "k_cache", "v_cache", "positions", "page_table", "cache_len", "n_new", "inv_freq",
                                 "new_len", "row_flags")] + \
        [(n, L * 3) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride", "k_out_stride", "k_cache_stride", "v_cache_stride")] + \
        [("pos_stride", L * 2)] + \
        [(n, I) for n in ("dtype", "B", "T", "Hq", "Hkv", "D", "pairs", "interleaved", "num_pages", "page_size", "max_pages")] + [("factor", F)]


class Tree(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k_new", "v_new", "k_cache", "v_cache", "page_table", "cache_len", "parents", "n_nodes", "out", "lse", "row_flags",
                                 "workspace")] + [("workspace_bytes", L)] + \
        [(n, L * 3) for n in ("q_stride", "k_new_stride", "v_new_stride", "k_cache_stride", "v_cache_stride")] + \
        [(n, I) for n in ("dtype", "B", "T", "Hq", "Hkv", "D", "num_pages", "page_size", "max_pages")] + [("scale", F)]


class Prefix(ctypes.Structure):
    _fields_ = [("own", Tree), ("prefix_table", P), ("prefix_len", P), ("group_start", P), ("prefixes", I), ("max_prefix_pages", I)]


class Adjust(ctypes.Structure):
    _fields_ = [(n, P) for n in ("logits", "out", "history", "history_len", "prompt_len", "tokens", "parents", "n_nodes", "repetition", "frequency",
                                 "presence", "bias_ids", "bias", "mask", "row_flags")] + [("mask_stride", L * 2)] + \
        [(n, I) for n in ("dtype", "B", "S", "V", "L", "n_bias")]


def fill(cls, **values):
    """Every pointer 1 GB from the next, never dereferenced: the checks answer first."""
    s = cls()
    k = 0
    for name, kind in cls._fields_:
        if kind is P:
            k += 1
            setattr(s, name, k << 30)
    for name, v in values.items():
        if isinstance(v, tuple):
            getattr(s, name)[:] = v
        else:
            setattr(s, name, v)
    return s


def answer(f, s):
    return f(bytes(s), None)


def rope_abi(**new):
    a = dict(q_stride=(768, 256, 64), k_stride=(384, 128, 64), q_out_stride=(768, 256, 64), k_out_stride=(384, 128, 64), pos_stride=(3, 1), dtype=0,
             B=2, T=3, Hq=4, Hkv=2, D=64, pairs=32, factor=1.0)
    a.update(new)
    return fill(Rope, **a)


@pytest.mark.parametrize("new, status", [
    (dict(dtype=7), 2), (dict(B=-1), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(D=257), 1), (dict(pairs=33), 1), (dict(pairs=-1), 1),
    (dict(factor=math.nan), 1), (dict(Hq=65537), 1), (dict(q=None), 1), (dict(k_out=None), 1), (dict(positions=None), 1), (dict(inv_freq=None), 1),
    (dict(q=(1 << 30) + 2), 3), (dict(q_out_stride=(0, 256, 64)), 1), (dict(q_stride=(-768, 256, 64)), 1), (dict(q_stride=(1 << 40, 256, 64)), 1),
    (dict(q_out=(1 << 30) + 64), 1), (dict(q_out=2 << 30), 1), (dict(k_out=(2 << 30) - 4), 1),
    (dict(B=0), 0), (dict(T=0), 0), (dict(Hq=0, Hkv=0), 0),
])
def test_rope_host_validation(lib, new, status):
    assert answer(lib.mtp_rope, rope_abi(**new)) == status


def append_abi(**new):
    s = (384, 128, 64)
    a = dict(q_stride=(768, 256, 64), k_stride=s, v_stride=s, q_out_stride=(768, 256, 64), k_out_stride=s, k_cache_stride=(2048, 128, 64),
             v_cache_stride=(2048, 128, 64), pos_stride=(3, 1), dtype=0, B=2, T=3, Hq=4, Hkv=2, D=64, pairs=32, num_pages=5, page_size=16, max_pages=2,
             factor=1.0)
    a.update(new)
    return fill(Append, **a)


@pytest.mark.parametrize("new, status", [
    (dict(dtype=7), 2), (dict(B=-1), 1), (dict(T=0), 1), (dict(Hkv=0), 1), (dict(D=257), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(max_pages=0), 1), (dict(max_pages=1 << 28, page_size=16), 1), (dict(k=None), 1), (dict(v_cache=None), 1), (dict(new_len=None), 1),
    (dict(q_out=None), 1), (dict(inv_freq=None), 1), (dict(k_cache_stride=(0, 128, 64)), 1), (dict(k=(6 << 30) + 1024), 1), (dict(v=7 << 30), 1),
    (dict(q_out=(6 << 30) + 64), 1), (dict(q_out=3 << 30), 1), (dict(k_out=1 << 30), 1), (dict(new_len=10 << 30), 1), (dict(row_flags=(9 << 30) + 12), 1),
    (dict(new_len=(11 << 30) + 4), 1), (dict(v=(3 << 30) + 2), 3), (dict(B=0), 0),
])
def test_cache_append_host_validation(lib, new, status):
    assert answer(lib.mtp_cache_append, append_abi(**new)) == status


def prefix_abi(own=(), **new):
    a = dict(q_stride=(768, 256, 64), k_new_stride=(384, 128, 64), v_new_stride=(384, 128, 64), k_cache_stride=(2048, 128, 64),
             v_cache_stride=(2048, 128, 64), dtype=1, B=2, T=3, Hq=4, Hkv=2, D=64, num_pages=5, page_size=16, max_pages=2, scale=0.125)
    a.update(own)
    b = dict(prefixes=1, max_prefix_pages=3)
    b.update(new)
    s = fill(Prefix, **b)
    s.own = fill(Tree, **a)
    return s


@pytest.mark.parametrize("own, new, status", [
    (dict(dtype=7), {}, 2), (dict(T=65), {}, 1), (dict(Hq=5), {}, 1), (dict(scale=0.0), {}, 1), ({}, dict(prefixes=0), 1), ({}, dict(prefixes=1 << 21), 1),
    ({}, dict(max_prefix_pages=0), 1), ({}, dict(max_prefix_pages=1 << 28), 1), (dict(B=1 << 20, T=64, Hq=64, Hkv=64), {}, 1),
    ({}, dict(prefix_table=None), 1), ({}, dict(prefix_len=None), 1), ({}, dict(group_start=None), 1), (dict(q=None), {}, 1), (dict(workspace=None), {}, 1),
    (dict(workspace=(13 << 30) + 8), {}, 3), (dict(out=(10 << 30) + 1), {}, 3), (dict(B=0), {}, 0),
])
def test_prefix_attention_host_validation(lib, own, new, status):
    assert answer(lib.mtp_prefix_attention, prefix_abi(own, **new)) == status
    if status == 1 and "scale" not in own and None not in {**own, **new}.values():
        assert lib.mtp_prefix_attention_workspace(bytes(prefix_abi(own, **new))) == -1


def adjust_abi(**new):
    a = dict(mask_stride=(12, 4), dtype=1, B=2, S=3, V=100, L=8, n_bias=5)
    a.update(new)
    return fill(Adjust, **a)


@pytest.mark.parametrize("new, status", [
    (dict(dtype=7), 2), (dict(B=-1), 1), (dict(B=(1 << 20) + 1), 1), (dict(S=0), 1), (dict(S=65), 1), (dict(V=0), 1), (dict(V=(1 << 24) + 1), 1),
    (dict(L=-1), 1), (dict(L=(1 << 28) + 1), 1), (dict(n_bias=1025), 1), (dict(n_bias=-1), 1), (dict(logits=None), 1), (dict(out=None), 1),
    (dict(history=None), 1), (dict(history_len=None), 1), (dict(tokens=None), 1), (dict(bias=None), 1), (dict(bias_ids=None), 1),
    (dict(mask_stride=(-1, 4)), 1), (dict(out=(1 << 30) + 16), 1), (dict(logits=(1 << 30) + 8), 3), (dict(out=(2 << 30) + 2), 3), (dict(B=0), 0),
])
def test_adjust_logits_host_validation(lib, new, status):
    assert answer(lib.mtp_adjust_logits, adjust_abi(**new)) == status


def test_null_arguments(lib):
    for f in (lib.mtp_rope, lib.mtp_cache_append, lib.mtp_prefix_attention, lib.mtp_adjust_logits):
        assert f(None, None) == 1
    assert lib.mtp_prefix_attention_workspace(None) == -1


# ----------------------------------------------------------- frequencies --

def test_rope_frequencies():
    f, factor = mtp.rope_frequencies(8, 10000.0)
    assert factor == 1.0 and f.dtype == torch.float32 and f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-6)
    g, factor = mtp.rope_frequencies(8, 10000.0, scaling="linear", factor=4.0)
    assert factor == 1.0 and torch.equal(g, f / 4)
    g, _ = mtp.rope_frequencies(8, 10000.0, scaling="base", factor=4.0)
    assert g[0] == 1.0 and g[3].item() == pytest.approx(0.001 / 4, rel=1e-6)
    assert mtp.rope_frequencies(2, scaling="base", factor=2.0)[0].tolist() == [1.0]
    g, factor = mtp.rope_frequencies(128, 10000.0, scaling="parts", factor=8.0, original_length=4096)
    f, _ = mtp.rope_frequencies(128, 10000.0)
    turns = 4096 * f.double() / (2 * math.pi)
    fast, slow = turns > 32, turns < 1
    assert fast.any() and slow.any() and torch.equal(g[fast], f[fast]) and torch.allclose(g[slow], f[slow] / 8, rtol=1e-6)
    between = ~(fast | slow)
    assert (g[between] < f[between]).all() and (g[between] > f[between] / 8).all()
    assert factor == pytest.approx(0.1 * math.log(8) + 1)


@pytest.mark.parametrize("kw, text", [
    (dict(rotary_dim=7), "even"), (dict(rotary_dim=0), "even"), (dict(base=0.0), "base"), (dict(factor=2.0), "of no use"), (dict(scaling="other"), "scaling"),
    (dict(scaling="linear", factor=0.5), "factor"), (dict(scaling="parts", factor=2.0), "original_length"),
    (dict(scaling="parts", factor=2.0, original_length=100, slow=4.0, fast=4.0), "original_length"),
])
def test_rope_frequencies_refusals(kw, text):
    with pytest.raises(ValueError, match=text):
        mtp.rope_frequencies(**{"rotary_dim": 8, **kw})


def test_reference_angles_are_exact():
    """The tests' own angles against products of a few bits, which float64 holds."""
    pos = torch.tensor([[0, 1, 3, 1 << 20, -5]])
    f = torch.tensor([1.0, 0.5, 2.0 ** -10])
    want = pos.double()[..., None] * f.double()
    got = step_ref.angles(pos, f)
    assert torch.allclose(got.cos(), want.cos(), atol=1e-9) and torch.allclose(got.sin(), want.sin(), atol=1e-9)


# ------------------------------------------- outputs that are another tensor --

FUSED = dict(q_stride=(1536, 512, 64), k_stride=(1536, 512, 64), q_out_stride=(1536, 512, 64), k_out_stride=(1536, 512, 64))  # 4 + 2 + 2 heads
Q0, K0, KO = 1 << 30, (1 << 30) + 4 * 64 * 4, 4 << 30


@pytest.mark.parametrize("new", [
    dict(FUSED, k=Q0, q_out=Q0),                            # q in place, and the same memory is k
    dict(FUSED, k=K0 - 256, q_out=Q0),                      # k begins in q's last head
    dict(FUSED, q_out=3 << 30, k=Q0, k_out=Q0),             # k in place, and the same memory is q
    dict(FUSED, q_out=KO, k_out=KO),                        # both outputs in one place
    dict(FUSED, q_out=KO, k_out=KO + 512 * 4),              # one token on
    dict(FUSED, q_out=Q0, k=K0, k_stride=(1536, 500, 64)),  # ranges that meet, strides that differ
])
def test_rope_refuses_outputs_on_other_tensors(lib, new):
    assert answer(lib.mtp_rope, rope_abi(**new)) == 1


@pytest.mark.parametrize("new", [
    dict(FUSED, k=K0, q_out=Q0, k_out=K0),                  # both in place, of one tensor
    dict(FUSED, q_out=KO, k_out=KO + 4 * 64 * 4),           # outputs of one tensor
    dict(FUSED, k=K0, q_out=Q0, k_out=K0, Hkv=1, k_stride=(1536, 512, 7), k_out_stride=(1536, 512, 7)),
    dict(FUSED, k=Q0 + 256, q_out=Q0, k_out=Q0 + 256, Hq=2, Hkv=2, q_stride=(1536, 512, 192), k_stride=(1536, 512, 192),
         q_out_stride=(1536, 512, 192), k_out_stride=(1536, 512, 192)),  # heads of (q, k, v)
])
def test_rope_takes_parts_of_one_tensor(lib, new):
    assert answer(lib.mtp_rope, rope_abi(**new)) != 1


S3 = (384, 128, 64)


@pytest.mark.parametrize("new", [
    dict(v=2 << 30, k_out=2 << 30),                                   # v is k, which is rotated in place
    dict(k=1 << 30, k_stride=(768, 256, 64), q_out=1 << 30, k_out=None),  # q in place, k its first heads
    dict(v=1 << 30, v_stride=(768, 256, 64), q_out=1 << 30),          # q in place, v its first heads
    dict(v_cache=6 << 30),                                            # one cache for both
    dict(v_cache=(6 << 30) + 64 * 4),                                 # a head on
    dict(q_out=4 << 30, k_out=(4 << 30) + 256, k_out_stride=(768, 256, 64)),
])
def test_cache_append_refuses_outputs_on_other_tensors(lib, new):
    assert answer(lib.mtp_cache_append, append_abi(**new)) == 1


@pytest.mark.parametrize("new", [
    dict(k_cache_stride=(4096, 128, 64), v_cache_stride=(4096, 128, 64), v_cache=(6 << 30) + 2048 * 4),  # pages of keys, then values
    dict(k_cache_stride=(4096, 256, 64), v_cache_stride=(4096, 256, 64), v_cache=(6 << 30) + 128 * 4),   # of tokens
    dict(k=K0, v=K0 + 512, q_out=Q0, k_out=K0, q_stride=(1536, 512, 64), q_out_stride=(1536, 512, 64), k_stride=(1536, 512, 64),
         k_out_stride=(1536, 512, 64), v_stride=(1536, 512, 64)),
])
def test_cache_append_takes_parts_of_one_tensor(lib, new):
    assert answer(lib.mtp_cache_append, append_abi(**new)) != 1
