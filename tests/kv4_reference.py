"""Plain 64-bit forms of the 4-bit cache, its attention and its pages, from the
layout's and the calls' definitions in dcc.h / kv4.cuh, for the tests."""
import math

import numpy as np
import torch

TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # unit roundoffs
PAGE = 64


def block_bytes(dim, group):
    return PAGE * dim + 2 * PAGE * (dim // group) * 4


def k_nibble(dim, d):
    """Place of channel d in a K row."""
    word = ((d % 32) // 8) * (dim // 32) + d // 32
    return word * 8 + d % 8


def v_nibble(dim, d, tok):
    """Place of channel d in the V row of token tok of the page."""
    c = d % 8
    if dim == 128 and (tok // 4) % 2 == 1:
        c ^= 4
    return c * (dim // 8) + 2 * (d // 16) + (d % 16) // 8


def decode(block, dim, group, dtype):
    """(K, V) values [64, dim] in float64 of one block (uint8 array)."""
    ng, half, par = dim // group, PAGE * dim // 2, PAGE * (dim // group) * 4
    out = []
    for w in range(2):
        codes = block[w * half:(w + 1) * half].reshape(PAGE, dim // 2)
        nib = np.stack([codes & 15, codes >> 4], -1).reshape(PAGE, dim)
        raw = np.ascontiguousarray(block[2 * half + w * par:2 * half + (w + 1) * par])
        p = torch.from_numpy(raw).view(TD[dtype]).double().numpy().reshape(PAGE, ng, 2)
        x = np.empty((PAGE, dim))
        for d in range(dim):
            for t in range(PAGE):
                n = k_nibble(dim, d) if w == 0 else v_nibble(dim, d, t)
                x[t, d] = p[t, d // group, 1] + p[t, d // group, 0] * nib[t, n]
        out.append(x)
    return out


_places = {}


def values(pool, dim, group, dtype):
    """K and V values [..., 64, dim] (float64 tensors) of a pool's blocks."""
    key = (dim,)
    if key not in _places:
        k = [[k_nibble(dim, d) for d in range(dim)] for _ in range(PAGE)]
        v = [[v_nibble(dim, d, t) for d in range(dim)] for t in range(PAGE)]
        _places[key] = (torch.tensor(k), torch.tensor(v))
    ng, half, par = dim // group, PAGE * dim // 2, PAGE * (dim // group) * 4
    out = []
    for w in range(2):
        codes = pool[..., w * half:(w + 1) * half].unflatten(-1, (PAGE, dim // 2))
        nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        at = _places[key][w].to(pool.device).expand(nib.shape)
        p = pool[..., 2 * half + w * par:2 * half + (w + 1) * par].contiguous().view(TD[dtype]).double()
        p = p.unflatten(-1, (PAGE, ng, 2)).repeat_interleave(group, -2)
        out.append(p[..., 1] + p[..., 0] * nib.gather(-1, at).double())
    return out


def quantise(x, group, dtype):
    """Values (float64) that x reads back as."""
    y = x.double().unflatten(-1, (-1, group))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    span = (hi - lo).to(torch.float32)  # a range past fp32 has no step
    step = (span.double() / 15).to(torch.float32).to(TD[dtype]).double()
    code = torch.where(step > 0, ((y - lo) / torch.where(step > 0, step, torch.ones_like(step))).round(),
                       torch.zeros_like(y)).clamp(0, 15)
    out = lo + step * code
    bad = ~torch.isfinite(y).all(-1, keepdim=True) | ~torch.isfinite(step)
    return torch.where(bad, torch.full_like(out, math.nan), out).flatten(-2)


def random_pool(g, layers, pages, heads, dim, group, dtype, garbage=True):
    """A pool whose blocks hold random codes, sensible params; where garbage,
    a second return marks nothing -- callers overwrite unused rows."""
    half, par = PAGE * dim // 2, PAGE * (dim // group) * 4
    pool = torch.empty(layers, pages, heads, block_bytes(dim, group), dtype=torch.uint8)
    pool[..., :2 * half] = torch.randint(0, 256, (layers, pages, heads, 2 * half), generator=g, dtype=torch.uint8)
    shape = (layers, pages, heads, par // 2)
    step = (0.25 * torch.exp(0.5 * torch.randn(shape, generator=g))).to(TD[dtype])
    lo = (-7.0 * step.float() + 0.5 * torch.randn(shape, generator=g)).to(TD[dtype])
    pool[..., 2 * half:] = torch.stack([step, lo], -1).view(torch.uint8).reshape(layers, pages, heads, 2 * par)
    return pool


def poison(pool, table, lens, dim, group):
    """NaN params and all-ones codes in every row that no sequence holds."""
    half, par = PAGE * dim // 2, PAGE * (dim // group) * 4
    used = torch.zeros(pool.shape[1], PAGE, dtype=torch.bool)
    for row, m in zip(table.tolist(), lens):
        for j in range(m):
            used[row[j // PAGE], j % PAGE] = True
    dead = ~used
    for w in range(2):
        codes = pool[..., w * half:(w + 1) * half].unflatten(-1, (PAGE, dim // 2))
        codes.transpose(2, 3)[:, dead] = 255
        p = pool[..., 2 * half + w * par:2 * half + (w + 1) * par].unflatten(-1, (PAGE, par // PAGE))
        p.transpose(2, 3)[:, dead] = 255  # 0xffff: a NaN in both types


def attention(K, V, q, positions, window, scale):
    """One head: K, V [len, D], q [rows, D] (float64), positions per row.
    Returns out, lse, sum p|V| and max over the seen keys of scale * sum |q K|."""
    n, m = q.shape[0], K.shape[0]
    D = q.shape[1]
    if m == 0:
        z = torch.zeros(n, D, dtype=torch.float64)
        return z, torch.full((n,), -math.inf, dtype=torch.float64), z, torch.zeros(n, dtype=torch.float64)
    j = torch.arange(m, device=K.device)[None, :]
    pos = positions[:, None]
    seen = (j <= pos) & (j >= 0)
    if window:
        seen &= j > pos - window
    s = (scale * (q @ K.T)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[:, None]),
                    torch.zeros_like(s))
    mag = (abs(scale) * (q.abs() @ K.abs().T)).masked_fill(~seen, 0.0).amax(-1)
    return p @ V, lse, p @ V.abs(), mag


class PageBook:
    """The page calls, one request after the other."""

    def __init__(self, table, lens, refs):
        self.table, self.lens, self.refs = [list(r) for r in table], list(lens), list(refs)
        self.copies = []

    def _lowest(self):
        for p, r in enumerate(self.refs):
            if r == 0:
                return p
        return None

    def _drop(self, s):
        for j, p in enumerate(self.table[s]):
            if p >= 0:
                self.refs[p] -= 1
                self.table[s][j] = -1
        self.lens[s] = 0

    def free(self, seqs):
        skipped, seen = 0, set()
        for s in seqs:
            if s < 0 or s >= len(self.lens) or s in seen:
                skipped += 1
                continue
            seen.add(s)
            self._drop(s)
        return [self.refs.count(0), skipped, 0]

    def fork(self, src, dst):
        named = {}
        for i, d in enumerate(dst):
            if 0 <= d < len(self.lens):
                named.setdefault(d, i)
        for d in named:
            self._drop(d)
        left = [p for p, r in enumerate(self.refs) if r == 0]
        fails = given = 0
        for i, (s, d) in enumerate(zip(src, dst)):
            if named.get(d) != i or s < 0 or s >= len(self.lens) or s in named:
                fails += 1
                continue
            m = self.lens[s]
            full, part = m // PAGE, m % PAGE > 0
            if part and not left:
                fails += 1
                continue
            for j in range(full):
                self.refs[self.table[s][j]] += 1
                self.table[d][j] = self.table[s][j]
            if part:
                p = left.pop(0)
                self.refs[p] = 1
                self.table[d][full] = p
                self.copies.append((self.table[s][full], p))
                given += 1
            self.lens[d] = m
        return [self.refs.count(0), fails, given]

    def reserve(self, add):
        left = [p for p, r in enumerate(self.refs) if r == 0]
        wanted = fails = given = 0
        room = len(left)
        for s, a in enumerate(add):
            if a <= 0:
                continue
            held, new = -(-self.lens[s] // PAGE), -(-(self.lens[s] + a) // PAGE)
            if new > len(self.table[s]):
                fails += 1
                continue
            wanted += new - held
            if new > held and wanted > room:
                fails += 1
                continue
            for j in range(held, new):
                p = left.pop(0)
                self.refs[p] = 1
                self.table[s][j] = p
                given += 1
            self.lens[s] += a
        return [self.refs.count(0), fails, given]

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        m = len(live)
        movers = [p for p in live if p >= m]
        slots = [p for p, r in enumerate(self.refs) if r == 0 and p < m]
        remap = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        for p, q in zip(movers, slots):
            remap[p] = q
        refs = [0] * len(self.refs)
        for p, r in enumerate(self.refs):
            if r > 0:
                refs[remap[p]] = r
        table = [[remap[p] if p >= 0 else -1 for p in row] for row in self.table]
        return table, refs, remap, list(zip(movers, slots)), [len(self.refs) - m, len(movers)]
