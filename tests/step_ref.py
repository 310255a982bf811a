"""Plain 64-bit forms of the operators around a verification step, on the CPU,
for the tests, each with the error bound of a kernel that computes in float32."""
import math
from fractions import Fraction

import torch

U = 2.0 ** -24  # the rounding of float32


def _turn():
    """1 / 2 pi to 300 bits (pi by Machin's formula)."""
    def arctan(x):
        t = s = (1 << 320) // x
        k, sign = 1, -1
        while t:
            t //= x * x
            k += 2
            s += sign * (t // k)
            sign = -sign
        return s

    return Fraction(1 << 320, 2 * 4 * (4 * arctan(5) - arctan(239)))


TURN = _turn()


def angles(positions, inv_freq):
    """position * frequency modulo 2 pi, float64 [.., n]: the product and its
    remainder are exact."""
    fs = [Fraction(float(f)) * TURN for f in inv_freq]
    ps = [int(p) for p in positions.flatten()]
    a = torch.tensor([[float((p * f) % 1) * 2 * math.pi for f in fs] for p in ps], dtype=torch.float64)
    return a.view(*positions.shape, len(fs))


def rope(x, positions, inv_freq, interleaved=False, factor=1.0, inverse=False):
    """(rotated x [B, T, H, D], its error bound).  A cosine or sine is off by at
    most 2 ulp = 4 u (the device function) + pi/4 u (its argument's rounding) + u
    (the factor), a product and a sum by u each: together 8 u of factor (|a| +
    |b|); then the output's own rounding."""
    n = len(inv_freq)
    f = float(torch.tensor(factor, dtype=torch.float32))
    t = angles(positions, inv_freq)[:, :, None]
    cos, sin = t.cos() * f, t.sin() * (-f if inverse else f)
    y = x.double().clone()
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x.double()[..., lo], x.double()[..., hi]
    y[..., lo], y[..., hi] = a * cos - b * sin, b * cos + a * sin
    tol = torch.zeros_like(y)
    size = (a.abs() + b.abs()) * abs(f) * 8 * U * 1.01
    half = torch.finfo(x.dtype).eps / 2 * 1.01
    tol[..., lo] = size + half * y[..., lo].abs()
    tol[..., hi] = size + half * y[..., hi].abs()
    return y, tol


def adjust(z, history=None, lens=None, prompts=None, tokens=None, parents=None, nodes=None, repetition=None, frequency=None,
           presence=None, bias_ids=None, bias=None, mask=None):
    """(adjusted logits [B, S, V], error bound, rows that are written [B, S]).
    Each of the four steps rounds once by u of what it has, n biases n - 1 times
    more of their absolute sum; then the output's own rounding."""
    B, S, V = z.shape
    out, tol, live = z.double().clone(), torch.zeros(B, S, V, dtype=torch.float64), torch.zeros(B, S, dtype=torch.bool)
    half = torch.finfo(z.dtype).eps / 2 * 1.01
    for b in range(B):
        text = [] if history is None else history[b, :int(lens[b])].tolist()
        m = 0 if prompts is None else int(prompts[b])
        n = S if nodes is None else int(nodes[b])
        rho, f, p = (d if t is None else float(t[b]) for t, d in ((repetition, 1.0), (frequency, 0.0), (presence, 0.0)))
        up = list(range(-1, S - 1)) if parents is None else parents[b].tolist()
        for s in range(n):
            live[b, s] = True
            count, seen = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.bool)
            late = list(text[m:])
            i = s if tokens is not None else -1
            while i >= 0:
                late.append(int(tokens[b, i]))
                i = up[i]
            late = torch.tensor([t for t in late if t >= 0], dtype=torch.long)
            count.index_add_(0, late, torch.ones(len(late), dtype=torch.float64))
            seen[torch.tensor([t for t in text[:m] if t >= 0], dtype=torch.long)] = True
            seen |= count > 0
            x = z[b, s].double()
            x = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
            size = torch.where(seen, x.abs(), torch.zeros_like(x))
            x = x - f * count - p * (count > 0)
            size = size + 2 * (abs(f) * count + x.abs() * (count > 0) + abs(p) * (count > 0))
            if bias_ids is not None:
                ids = bias_ids[b].long()
                at, some = ids[ids >= 0], bias[b].double()[ids >= 0]
                total, large, many = (torch.zeros(V, dtype=torch.float64) for _ in range(3))
                total.index_add_(0, at, some)
                large.index_add_(0, at, some.abs())
                many.index_add_(0, at, torch.ones_like(some))
                x = x + total
                size = size + large * many + torch.where(many > 0, x.abs(), torch.zeros_like(x))
            if mask is not None:
                v = torch.arange(V)
                x = torch.where((mask[b, s].long()[v // 32] >> (v % 32)) & 1 == 0, -math.inf, x)
            out[b, s] = x
            tol[b, s] = torch.nan_to_num(size, nan=0.0, posinf=0.0) * U * 1.01
            changed = seen | (tol[b, s] > 0)
            tol[b, s] += torch.where(changed & x.isfinite(), x.abs() * half, torch.zeros_like(x))
    return out, tol, live
