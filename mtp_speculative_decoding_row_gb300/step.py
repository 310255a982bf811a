"""Binding of the operators around a verification step (see "Around a
verification step" in ``include/mtp_rs.h``): rotary positions, appending to the
paged cache, and the adjustment of logits.

Argument marshalling only, as for the tree-draft operators: the checks of the
tensors and the call of the library are native (``csrc/binding.cpp``).
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import mtp_speculative_decoding_row_gb300 as _m

from .tree import _call, _on

MAX_BIAS = 1024


class RopeResult(NamedTuple):
    q: "object"  # [B, T, Hq, D], the inputs' dtype
    k: "object"  # [B, T, Hkv, D] or None


class AppendResult(NamedTuple):
    cache_len: "object"  # [B] int32: cached tokens after the call
    q: "object"          # [B, T, Hq, D] rotated queries, or None
    k: "object"          # [B, T, Hkv, D] rotated keys, or None
    row_flags: "object"  # [B] int32


class AdjustResult(NamedTuple):
    logits: "object"     # [B, S, V], the logits' dtype
    row_flags: "object"  # [B] int32


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                     original_length: Optional[int] = None, slow: float = 1.0, fast: float = 32.0):
    """The angles per token of a rotary embedding, as mtp_rope takes them:
    (inv_freq [rotary_dim / 2] float32 on the CPU, the factor of the rotated
    elements).

    inv_freq[i] = base ** (-2 i / rotary_dim); for texts `factor` times as long
    as the model was trained on, by `scaling`:
      "linear"  inv_freq / factor
      "base"    the base times factor ** (d / (d - 2)), so that the slowest angle
                is that of "linear" and the fastest is left
      "parts"   angles that turn more than `fast` times in `original_length` tokens
                are left, those that turn less than `slow` times divided by
                factor, the others in between in proportion; the rotated
                elements are multiplied by 0.1 ln(factor) + 1."""
    torch = _m._torch()
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not (base > 0 and factor >= 1 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError(f"base must be positive and factor at least 1, got {base} and {factor}")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f'scaling must be None, "linear", "base" or "parts", got {scaling!r}')
    if scaling is None and factor != 1:
        raise ValueError("factor is of no use without scaling")
    if scaling == "base":
        base *= factor ** (rotary_dim / (rotary_dim - 2)) if rotary_dim > 2 else 1.0
    f = torch.tensor([base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_length is None or not 0 < slow < fast:
            raise ValueError("parts needs original_length and 0 < slow < fast")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.float(), 0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0


def mtp_rope(q, k, positions, inv_freq, *, interleaved: bool = False, factor: float = 1.0, inverse: bool = False,
             out: Optional[RopeResult] = None, stream=None) -> RopeResult:
    """Rotary positions of queries and keys (see mtp_rope in include/mtp_rs.h);
    with `inverse` those of their gradients.

    q [B, T, Hq, D] and k [B, T, Hkv, D] or None (float32 or bfloat16; any
    strides but a contiguous last dimension), positions [B, T] int32 (any
    strides), inv_freq [n] float32: the first 2 n elements of each head are
    rotated, pairs (i, n + i) or with `interleaved` (2 i, 2 i + 1), and
    multiplied by `factor`.  `out` may hold q and k themselves (in place)."""
    torch = _m._torch()
    index = q.get_device()
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            out = mine = RopeResult(torch.empty(q.shape, dtype=q.dtype, device=q.device),
                                    None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device))
        _call("rope", (q, k, positions, inv_freq, bool(interleaved), factor, bool(inverse), out.q, out.k, on.raw(torch, index, mine)))
    return out


def mtp_cache_append(k, v, k_cache, v_cache, page_table, cache_len, n_new=None, *, q=None, inv_freq=None, positions=None,
                     interleaved: bool = False, factor: float = 1.0, with_keys: bool = False, out: Optional[AppendResult] = None,
                     stream=None) -> AppendResult:
    """Keys and values of new tokens written behind the cached ones, keys and
    queries rotated on the way (see mtp_cache_append in include/mtp_rs.h).

    k and v [B, T, Hkv, D], k_cache and v_cache [num_pages, page_size, Hkv, D]
    (written in place), page_table [B, max_pages], cache_len [B], n_new [B]
    (None: T) int32; with inv_freq [n] float32 keys and q [B, T, Hq, D] are
    rotated as by mtp_rope, at positions [B, T] int32 or (None) cache_len + t.
    Returns cache_len [B] after the call, the rotated queries, the rotated keys
    (with with_keys, or where `out` has them) and row_flags [B]; rows of tokens
    >= n_new are left as they were (undefined in outputs allocated here)."""
    torch = _m._torch()
    index = k.get_device()
    if out is not None and with_keys and out.k is None:
        raise ValueError("mtp_cache_append: with_keys needs out.k")
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            e = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
            n = lambda: torch.empty(k.shape[:1], dtype=torch.int32, device=k.device)  # noqa: E731
            out = mine = AppendResult(n(), None if q is None else e(q), e(k) if with_keys else None, n())
        _call("cache_append", (k, v, k_cache, v_cache, page_table, cache_len, n_new, q, inv_freq, positions, bool(interleaved), factor,
                               out.cache_len, out.q, out.k, out.row_flags, on.raw(torch, index, mine)))
    return out


def mtp_adjust_logits(logits, history=None, history_len=None, *, prompt_len=None, tokens=None, parents=None, n_nodes=None,
                      repetition=None, frequency=None, presence=None, bias_ids=None, bias=None, mask=None,
                      out: Optional[AdjustResult] = None, stream=None) -> AdjustResult:
    """Penalties for repeated tokens, biases and masks on the logits of a drafted
    chain or tree (see mtp_adjust_logits in include/mtp_rs.h).

    logits [B, S, V] (float32 or bfloat16, contiguous, starting on 16 bytes);
    history [B, L], history_len [B], prompt_len [B], tokens and parents [B, S],
    n_nodes [B] int32; repetition, frequency, presence [B] float32; bias_ids
    int32 and bias float32 [B, n]; mask [B, S, ceil(V / 32)] int32, bit v % 32 of
    word v / 32 set where v is allowed (any strides but contiguous words).  Every
    one but the logits may be None.  `out` may hold the logits themselves (in
    place: only what changes is written)."""
    torch = _m._torch()
    index = logits.get_device()
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            out = mine = AdjustResult(torch.empty(logits.shape, dtype=logits.dtype, device=logits.device),
                                      torch.empty(logits.shape[:1], dtype=torch.int32, device=logits.device))
        _call("adjust_logits", (logits, history, history_len, prompt_len, tokens, parents, n_nodes, repetition, frequency, presence,
                                bias_ids, bias, mask, out.logits, out.row_flags, on.raw(torch, index, mine)))
    return out
