"""How far the attention over the 4-bit cache may be from 64 bits, from what its
two kernels round.  With e = 2^-23 (an fp32 rounding, or truncation, per
operation), h = 2^-11 (fp16's unit roundoff), u the cache's type's, and n keys:

Both.  A score that is off by ds changes a probability by a factor within
exp(+-2 ds) (once itself, once through the sum).  The result is rounded once:
u |exact|, or half the type's smallest subnormal.

Streaming kernel.  Codes and Q are exact.  Scores are fp32 sums of terms up to
|q| (|lo| + 143 step) (a code enters as 64 + n, and 64 comes off), rounded once
for 8 products or more and a few times at the end:
  ds = (D / 8 + 8) e scale sum_d |q_d| (|lo_d| + 143 step_d).
p * step is rounded to fp16, and multiplies n - 8: h p step |n - 8| a key, or
2^-36 of the largest step where it is subnormal.  The sums carry terms up to
p (|lo| + 151 step) in fp32: 2 n e of them.

Prompt kernel.  K and V are rounded to fp16: h of each, and 2^-21 for the bf16
cache's small parameters (of a key's largest |K|, where that is not in 2^-8 ..
2^15 and so has a power of two of its own).  Where
a bf16 group of V is out of fp16's range, V and P are rounded to bf16.  The D
errors of a score are of either sign:
  ds = 6 h scale sqrt(sum_d (q_d K_d)^2) + (D + 8) e scale sum |q_d K_d|
(six times the norm of the largest errors: more than ten standard deviations).
P is rounded to fp16 as well: h p, or 2^-31 where it is subnormal.

The 2-norm of all errors relative to the results' own.  Rounding to a unit
roundoff w leaves 0.42 w of a value (root mean square over its binade); rounding
errors of the operands are of either sign and add up in squares like the results
themselves, those of the scores in proportion to their norm above:
  0.5 sqrt(u^2 + 2 h^2 + (h scale norm of the products)^2),
with 3 u^2 where V and P are bf16."""
import math

import torch

import kv4_reference as R

E, H = 2.0 ** -23, 2.0 ** -11
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


def parts(pool, dim, group, dtype):
    """((step, lo, code) of K, of V), each [..., 64, dim] in float64, of a pool's blocks."""
    ng, half, par = dim // group, R.PAGE * dim // 2, R.PAGE * (dim // group) * 4
    out = []
    for w in range(2):
        codes = pool[..., w * half:(w + 1) * half].unflatten(-1, (R.PAGE, dim // 2))
        nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        if w == 0:
            at = torch.tensor([[R.k_nibble(dim, d) for d in range(dim)]] * R.PAGE)
        else:
            at = torch.tensor([[R.v_nibble(dim, d, t) for d in range(dim)] for t in range(R.PAGE)])
        p = pool[..., 2 * half + w * par:2 * half + (w + 1) * par].contiguous().view(R.TD[dtype]).double()
        p = p.unflatten(-1, (R.PAGE, ng, 2)).repeat_interleave(group, -2)
        out.append((p[..., 0], p[..., 1], nib.gather(-1, at.to(pool.device).expand(nib.shape)).double()))
    return out


def rows_of(x, pages, head, m):
    """The m rows of one sequence and head of parts [pages, heads, 64, dim]."""
    return tuple(t[pages, head].reshape(-1, t.shape[-1])[:m] for t in x)


def wide_v(V, dtype):
    """Whether some value's group may stand outside fp16's range: not 2^-8 .. 2^11."""
    top = torch.maximum(V[1].abs(), (V[1] + 15 * V[0]).abs())
    return dtype == "bf16" and bool(((top != 0) & ((top < 2.0 ** -8) | (top > 2.0 ** 11))).any())


def exact(K, V, q, positions, window, scale, dtype, kernel):
    """One head.  K, V: (step, lo, code) [m, D]; q [rows, D], positions of the rows.
    Returns (out, lse, bound of out, bound of lse, mean square of ds's statistical part)."""
    k, v = (t[1] + t[0] * t[2] for t in (K, V))
    m, D = k.shape
    u = R.U[dtype]
    if m == 0:
        z = torch.zeros(len(q), D, dtype=torch.float64, device=q.device)
        return z, torch.full((len(q),), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0], z[:, 0]
    j = torch.arange(m, device=q.device)[None, :]
    seen = j <= positions[:, None]
    if window:
        seen &= j > positions[:, None] - window
    s = (scale * (q @ k.T)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[:, None]),
                    torch.zeros_like(s))
    out = p @ v
    sc = abs(scale)

    def most(x):  # over the keys that each row sees
        return torch.where(seen, x, torch.zeros_like(x)).amax(-1)
    n = seen.sum(-1).double()[:, None]
    if kernel == "streaming":
        ds = most((D / 8 + 8) * E * sc * (q.abs() @ (K[1].abs() + 143 * K[0]).T))
        rough = torch.zeros_like(ds)
        top = torch.where(seen[:, :, None], V[0][None], torch.zeros(1, dtype=torch.float64, device=q.device)).amax((1, 2)) \
            if m * len(q) * D < 1 << 24 else V[0].max().expand(len(q))
        operand = H * (p @ (V[0] * (V[2] - 8).abs())) + (2.0 ** -36 * n[:, 0] * top)[:, None]
        small = 2 * n * E * (p @ (V[1].abs() + 151 * V[0]))
    else:
        norm = sc * torch.sqrt((q * q) @ (k * k).T)
        wide = wide_v(V, dtype)
        m = torch.maximum(K[1].abs(), (K[1] + 15 * K[0]).abs()).amax(-1)
        m = torch.where((m >= 2.0 ** -8) & (m <= 2.0 ** 15), torch.ones_like(m), m)  # others have their own power of two
        low = 2.0 ** -21 * sc * q.abs().sum(-1, keepdim=True) * m if dtype == "bf16" else 0.0
        ds = most(6 * H * norm + (D + 8) * E * sc * (q.abs() @ k.abs().T) + low)
        rough = (p * (norm * H) ** 2).sum(-1)
        operand = 2 * (u if wide else H) * (p @ v.abs()) + 2.0 ** -31 * (seen.double() @ v.abs()) + (0.0 if wide or dtype != "bf16" else 2.0 ** -21)
        small = 2 * n * E * (p @ v.abs())
    tol = 1.01 * (torch.expm1(2 * ds)[:, None] * (p @ v.abs()) + operand + small) + u * out.abs() + TINY[dtype]
    tol_lse = ds + (n[:, 0] + 8) * E + 4 * E * (torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse)) + 80)
    return out, lse, tol, tol_lse, rough


class Totals:
    """Sums over a case's heads for the 2-norm, and whether zeros would have passed."""

    def __init__(self, dtype, wide=False):
        self.wide, self.u, self.err, self.ref, self.rough, self.zeros_fail = wide, R.U[dtype], 0.0, 0.0, 0.0, 0

    def add(self, got, out, tol, rough):
        self.err += (got - out).square().sum().item()
        self.ref += out.square().sum().item()
        self.rough += (rough[:, None] * out.square()).sum().item()
        self.zeros_fail += int((out.abs() > tol).sum())

    def check(self):
        rel = math.sqrt(self.err / self.ref)
        limit = 0.5 * math.sqrt((3 if self.wide else 1) * self.u ** 2 + 2 * H ** 2 + self.rough / self.ref)
        assert rel <= limit, (rel, limit)
        assert self.zeros_fail > 0  # a result of all zeros would have been found
        return rel
