"""Attention over the 4-bit cache for rows with sets of seen keys of their own
(trees of drafted tokens, windows with sinks), in 64 bits from the calls'
definitions, with the bounds of kv4_bounds.py for any set of seen keys."""
import math

import torch

import kv4_bounds as B
import kv4_reference as R


def seen_rows(length, news, rows, window=0, sinks=0, masks=None):
    """[rows, length]: what the first `rows` new tokens of a sequence see.
    masks: sets of drafted tokens, one a row (None: causal)."""
    first = length - news
    out = torch.zeros(rows, max(0, length), dtype=torch.bool)
    for i in range(rows):
        if masks is None:
            x = first + i
            lo = max(0, x - window + 1) if window else 0
            for j in range(max(0, x + 1)):
                out[i, j] = j >= lo or j < sinks
        else:
            drafted = [j for j in masks[i] if 0 <= j < news]
            for j in drafted:
                if first + j >= 0:
                    out[i, first + j] = True
            for j in range(max(0, first)):
                out[i, j] = not window or j >= first + len(drafted) - window or j < sinks
    return out


def pack(masks, words):
    """int32 [rows, words] of sets of drafted tokens."""
    out = torch.zeros(len(masks), words, dtype=torch.int64)
    for i, m in enumerate(masks):
        for j in m:
            out[i, j // 32] |= 1 << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def tree(g, news, reach=4):
    """Ancestors and itself of each drafted token of a random tree."""
    masks = []
    for j in range(news):
        parent = j - 1 - int(torch.randint(0, reach, (1,), generator=g))
        masks.append({j} | (masks[parent] if parent >= 0 else set()))
    return masks


def exact(K, V, q, seen, scale, dtype, kernel):
    """One head.  K, V: (step, lo, code) [m, D]; q [rows, D] float64; seen [rows, m].
    Returns (out, lse, bound of out, bound of lse, mean square of the scores' errors),
    as kv4_bounds.exact for causal rows."""
    k, v = (t[1] + t[0] * t[2] for t in (K, V))
    m, D = k.shape
    u = R.U[dtype]
    if m == 0:
        z = torch.zeros(len(q), D, dtype=torch.float64, device=q.device)
        return z, torch.full((len(q),), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0], z[:, 0]
    some = seen.any(0)
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    # a key that no row sees may hold anything
    k, v = torch.where(some[:, None], k, zero), torch.where(some[:, None], v, zero)
    K, V = (tuple(torch.where(some[:, None], x, zero) for x in t) for t in (K, V))
    s = (scale * (q @ k.T)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[:, None]), zero)
    out = p @ v
    sc = abs(scale)

    def most(x):  # over the keys that each row sees
        return torch.where(seen, x, zero).amax(-1)
    n = seen.sum(-1).double()[:, None]
    if kernel == "streaming":
        ds = most((D / 8 + 8) * B.E * sc * (q.abs() @ (K[1].abs() + 143 * K[0]).T))
        rough = torch.zeros_like(ds)
        top = torch.stack([V[0][row].amax() if row.any() else zero for row in seen])
        operand = B.H * (p @ (V[0] * (V[2] - 8).abs())) + (2.0 ** -36 * n[:, 0] * top)[:, None]
        small = 2 * n * B.E * (p @ (V[1].abs() + 151 * V[0]))
    else:
        norm = sc * torch.sqrt((q * q) @ (k * k).T)
        wide = B.wide_v(V, dtype)
        mk = torch.maximum(K[1].abs(), (K[1] + 15 * K[0]).abs()).amax(-1)
        mk = torch.where((mk >= 2.0 ** -8) & (mk <= 2.0 ** 15), torch.ones_like(mk), mk)
        low = 2.0 ** -21 * sc * q.abs().sum(-1, keepdim=True) * mk if dtype == "bf16" else 0.0
        ds = most(6 * B.H * norm + (D + 8) * B.E * sc * (q.abs() @ k.abs().T) + low)
        rough = (p * (norm * B.H) ** 2).sum(-1)
        operand = 2 * (u if wide else B.H) * (p @ v.abs()) + 2.0 ** -31 * (seen.double() @ v.abs()) \
            + (0.0 if wide or dtype != "bf16" else 2.0 ** -21)
        small = 2 * n * B.E * (p @ v.abs())
    tol = 1.01 * (torch.expm1(2 * ds)[:, None] * (p @ v.abs()) + operand + small) + u * out.abs() + B.TINY[dtype]
    tol_lse = ds + (n[:, 0] + 8) * B.E + 4 * B.E * (torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse)) + 80)
    return out, lse, tol, tol_lse, rough
