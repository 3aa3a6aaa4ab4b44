"""Cases, plain forms and exact values of the operators around the row-parallel
layer of a tensor-parallel decoder: the 4-bit key/value cache (append, read,
attention), its pages (fork, compact) and the column-parallel linear layer.

Every operator works on n virtual ranks at once; rank r holds its own heads or
rows.  With ``own`` false, ``run`` is the plain form in elementary torch
operations in 32 bits; with ``own`` true it makes the framework's calls.

Cache layout (64 tokens per page, one block per page and key/value head):
  K codes 64 x D/2 bytes | V codes 64 x D/2 | K params 64 x D/group x (step, lo)
  | V params, each param of the cache's 16-bit type; value = lo + step * code.
"""
import math

import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    attend = dict(op="attend", n=8, heads=1, dim=128, group=64, dtype="bf16", window=0)
    linear = dict(op="linear", n=8, dtype="bf16", residual=False)
    return [
        # one decode step's new token of 64 running requests, quantised into the cache of 8 ranks
        dict(name="append-token", op="append", n=8, seqs=64, new=1, length=4096, heads=1, dim=128, group=64, dtype="bf16"),
        # four prompts of uneven length written at once, fp16 with small groups and two heads a rank
        dict(name="append-prompt", op="append", n=8, seqs=4, new=4099, length=4099, heads=2, dim=128, group=32, dtype="fp16"),
        # a single request early in its answer: the latency of one decode step
        dict(attend, name="decode-short", seqs=1, new=1, length=777, share=8),
        # a serving batch of uneven requests with idle slots, the usual decode step
        dict(attend, name="decode-batch", seqs=64, new=1, length=8192, share=8),
        # one very long document, few query heads per cache head, finer groups
        dict(attend, name="decode-long", seqs=1, new=1, length=131109, share=4, heads=2, group=32, dtype="fp16"),
        # verification of five drafted tokens under a sliding window, 64-wide heads
        dict(attend, name="verify", seqs=16, new=5, length=3001, share=4, heads=2, dim=64, group=32, dtype="fp16", window=1024),
        # a chunk of a prompt against what is cached already
        dict(attend, name="prompt-chunk", seqs=1, new=2048, length=8192, share=8),
        # a beam step: half of the beams are dropped and refilled from the others, partial pages copied
        dict(name="fork-beams", op="fork", n=8, seqs=128, length=2085, layers=4, heads=1, dim=128, group=64, dtype="bf16"),
        # a half-empty pool squeezed so that its tail can be given back
        dict(name="compact-pool", op="compact", n=8, seqs=256, length=2085, layers=4, heads=1, dim=128, group=64, dtype="bf16"),
        # one token through the column-parallel layer (bandwidth of the weights)
        dict(linear, name="linear-token", tokens=1, rows=1024, k=8192, act="silu"),
        # a decode batch, fp16, into the residual stream
        dict(linear, name="linear-batch", tokens=64, rows=3584, k=8192, act="gelu", dtype="fp16", residual=True),
        # a prompt chunk (tensor-core rate)
        dict(linear, name="linear-prompt", tokens=2048, rows=3584, k=8192, act="gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "attend", "fork", "compact", "linear", "linear"])
    n = rng.choice([1, 2, 4, 8])
    cache = dict(op=op, n=n, heads=rng.choice([1, 2, 3, 4]), dim=rng.choice([64, 128]), group=rng.choice([32, 64]),
                 dtype=rng.choice(["bf16", "fp16"]))
    if op == "linear":
        c = dict(op=op, n=n, dtype=cache["dtype"], tokens=_log(rng, 1, 2048), rows=8 * _log(rng, 2, 448),
                 k=8 * _log(rng, 8, 1024), act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 residual=rng.random() < 0.5)
        return c
    if op == "append":
        c = dict(cache, seqs=_log(rng, 1, 64), new=_log(rng, 1, 2048))
        c["new"] = max(1, min(c["new"], 32768 // (c["seqs"] * c["heads"])))
        return dict(c, length=c["new"] + _log(rng, 1, 2048))
    if op in ("fork", "compact"):
        c = dict(cache, layers=rng.choice([1, 2, 4]), seqs=_log(rng, 2, 128 if op == "fork" else 256),
                 length=_log(rng, 1, 2085))
        while c["seqs"] > 2 and c["seqs"] * c["length"] * c["layers"] * c["heads"] * c["n"] > 256 * 2085 * 32:
            c["seqs"] = c["seqs"] // 2
        return c
    c = dict(cache, share=rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), seqs=_log(rng, 1, 64), length=_log(rng, 1, 131072))
    form = rng.random()
    c["new"] = 1 if form < 0.5 else rng.randint(2, 8) if form < 0.7 else _log(rng, 9, 2048)
    c["length"] = max(c["length"], c["new"])
    c["window"] = _log(rng, 16, 4096) if rng.random() < 0.25 else 0
    while c["seqs"] > 1 and (c["seqs"] * c["length"] * c["heads"] * n > 1 << 21
                             or c["seqs"] * c["length"] * c["heads"] * c["share"] * n * c["new"] > 1 << 29):
        c["seqs"] //= 2
    while c["length"] * c["heads"] * n > 1 << 21 or c["length"] * c["heads"] * c["share"] * n * c["new"] > 1 << 29:
        if c["new"] > 16 and c["length"] < 4 * c["new"]:
            c["new"] = c["new"] // 2 + 1
        c["length"] = max(c["new"], c["length"] // 2 + 1)
        if c["length"] == c["new"] and c["new"] <= 16:
            break
    return c


def _lengths(case):
    """Tokens each sequence holds after this step's new ones, and how many of
    them are new (an idle slot holds none and still has one row of queries)."""
    B, L, new = case["seqs"], case["length"], case["new"]
    lens, news = [], []
    for s in range(B):
        m = L if s == 0 else max(1, L - (s * 7919 * 13) % max(1, (15 * L) // 16))
        t = new if new == 1 or s == 0 else max(1, min(new, m))
        if case["op"] == "append" and new > 1:
            t = max(1, new - (s * 613) % max(1, new // 2))
            m = t + (L - new)
        if case["op"] == "attend" and new == 1 and s % 32 == 31:
            m = 0  # an idle slot
        lens.append(max(m, t) if m else 0)
        news.append(t)
    return lens, news


def _block(dim, group):
    return PAGE * dim + 2 * PAGE * (dim // group) * 4


# ------------------------------------------------------------------ inputs
def _pool(g, n, layers, pages, case):
    """Pages of a cache in use: bell-shaped codes, steps and minima as such K/V have."""
    dim, group, t = case["dim"], case["group"], TYPES[case["dtype"]]
    H, blk, codes, ng = case["heads"], _block(dim, group), PAGE * dim, dim // group
    pool = torch.empty(n, layers, pages, H, blk, dtype=torch.uint8, device="cuda")
    for r in range(n):
        shape = (layers, pages, H, codes)
        a = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
        b = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
        low = ((a & 15) + (b & 15)) >> 1
        pool[r, ..., :codes] = low | ((((a >> 4) + (b >> 4)) >> 1) << 4)
        par = (layers, pages, H, 2 * PAGE * ng)
        step = (0.3 * torch.exp(0.25 * torch.randn(par, device="cuda", generator=g))).to(t)
        lo = (-7.5 * step.float() + 0.2 * torch.randn(par, device="cuda", generator=g)).to(t)
        pool[r, ..., codes:] = torch.stack([step, lo], -1).view(torch.uint8).reshape(layers, pages, H, -1)
    return pool


def _pages(lens, maxp, g, spare):
    """A page table of pages in random order, as after some time of serving."""
    need = [-(-m // PAGE) for m in lens]
    total = sum(need) + spare
    order = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    row = torch.arange(maxp, device="cuda")[None, :]
    cnt = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(cnt, 0) - cnt
    table = torch.where(row < cnt, order[(first + row).clamp(max=total - 1)], -1)
    return table.to(torch.int32).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t = TYPES[case["dtype"]]
    n = case["n"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] == "linear":
        T, R, K = case["tokens"], case["rows"], case["k"]
        s = {"case": case, "x": normal(T, K).to(t), "w": torch.empty(n, R, K, dtype=t, device="cuda"),
             "bias": (0.1 * normal(n, R)).to(t), "y": torch.empty(n, T, R, dtype=t, device="cuda")}
        for r in range(n):
            s["w"][r] = (normal(R, K) / math.sqrt(K)).to(t)
        s["res"] = normal(n, T, R).to(t) if case["residual"] else None
        return s
    H, D = case["heads"], case["dim"]
    s = {"case": case}
    if case["op"] in ("append", "attend"):
        lens, news = _lengths(case)
        maxp = max(-(-m // PAGE) for m in lens)
        s["table"], pages = _pages(lens, maxp, g, 3)
        s["pool"] = _pool(g, n, 1, pages, case)
        s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for x in news:
            starts.append(starts[-1] + x)
        s["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        T = starts[-1]
        s["tokens"], s["new"] = T, max(news)
        seq = torch.repeat_interleave(torch.arange(len(news), device="cuda"), torch.tensor(news, device="cuda"))
        s["seq"] = seq  # the sequence of each new token, and its position
        s["pos"] = s["len"][seq] - s["start"][seq + 1] + torch.arange(T, device="cuda")
        if case["op"] == "append":
            for name in ("k", "v"):  # a per-channel scale and offset, as projections give
                scale = torch.exp(0.4 * normal(n, 1, H, D))
                s[name] = (normal(n, T, H, D) * scale + 0.3 * normal(n, 1, H, D)).to(t)
                s[name + "_out"] = torch.empty_like(s[name])
        else:
            Hq = H * case["share"]
            s["q"] = normal(n, T, Hq, D).to(t)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(n, T, Hq, dtype=torch.float32, device="cuda") if case["new"] == 1 else None
        return s
    B, L = case["seqs"], case["length"]
    lens = [max(1, L - (i * 389) % max(1, L // 2)) for i in range(B)]
    maxp = -(-L // PAGE) + 1
    s["table"], pages = _pages(lens, maxp, g, B + 5)
    s["pool"] = _pool(g, n, case["layers"], pages, case)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["info"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    order = torch.randperm(B, device="cuda", generator=g).to(torch.int32)
    if case["op"] == "fork":
        s["dst"] = order[:B // 2].contiguous()
        pick = torch.randint(0, B - B // 2, (B // 2,), device="cuda", generator=g)
        s["src"] = order[B // 2:][pick].contiguous()  # some are taken more than once
    else:  # half of the sequences have ended
        ended = order[:B // 2].long()
        s["table"][ended] = -1
        s["len"][ended] = 0
        s["new_table"] = torch.empty_like(s["table"])
        s["remap"] = torch.empty(pages, dtype=torch.int32, device="cuda")
    live = s["table"][s["table"] >= 0].long()
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda").index_add_(
        0, live, torch.ones_like(live, dtype=torch.int32))
    s["new_refs"] = torch.empty_like(s["refs"])
    return s


# ------------------------------------------------------------------ the plain forms
def _order(dim):
    """Channel held by each stored nibble: of a K row, and of a V row by its token."""
    p = torch.arange(dim, device="cuda")
    word, nib, j = p // 8, p % 8, dim // 32
    k = 32 * (word % j) + 8 * (word // j) + nib
    size = dim // 8
    tok = torch.arange(PAGE, device="cuda")[:, None]
    swap = 4 * ((tok >> 2) & 1) if dim == 128 else 0 * tok
    chunk, m = (p // size)[None, :] ^ swap, (p % size)[None, :]
    return k, 16 * (m >> 1) + chunk + 8 * (m & 1)


def _parts(pool, case):
    """Views of a pool's K and V codes and (step, lo) params."""
    D, t, ng = case["dim"], TYPES[case["dtype"]], case["dim"] // case["group"]
    c, q = PAGE * D // 2, PAGE * ng * 4
    lead = pool.shape[:-1]

    def codes(a):
        return pool[..., a:a + c].unflatten(-1, (PAGE, D // 2))

    def params(a):
        return pool.view(t)[..., a // 2:(a + q) // 2].unflatten(-1, (PAGE, ng, 2))
    assert len(lead) == 4
    return codes(0), params(2 * c), codes(c), params(2 * c + q)


def _values(codes, params, order, group):
    """lo + step * code of unpacked rows [..., PAGE, D/2] in channel order."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    out = torch.empty_like(c)
    out.scatter_(-1, order.expand(c.shape), c)
    par = params.float().repeat_interleave(group, -2)
    return par[..., 1] + par[..., 0] * out.float()


def _append(s):
    case = s["case"]
    D, G, t = case["dim"], case["group"], TYPES[case["dtype"]]
    kc, kp, vc, vp = _parts(s["pool"], case)
    ko, vo = _order(D)
    slot = (s["pos"] % PAGE).long()
    page = s["table"].long()[s["seq"], (s["pos"] // PAGE).long()]
    outs = []
    for x, codes, params, order in ((s["k"], kc, kp, ko.expand(PAGE, D)), (s["v"], vc, vp, vo)):
        y = x.float().unflatten(-1, (D // G, G))
        lo = y.amin(-1)
        step = ((y.amax(-1) - lo) / 15.0).to(t)
        unit = torch.where(step > 0, step.float(), torch.full_like(lo, math.inf))  # a constant group: codes 0
        c = torch.round((y - lo[..., None]) / unit[..., None]).clamp(0, 15).to(torch.uint8).flatten(-2)
        stored = c.gather(-1, order[slot][None, :, None, :].expand(c.shape))
        packed = stored[..., 0::2] | (stored[..., 1::2] << 4)
        codes[:, 0, page, :, slot] = packed.transpose(0, 1)
        params[:, 0, page, :, slot] = torch.stack([step, lo.to(t)], -1).transpose(0, 1)
        back = _values(codes[:, 0, page, :, slot], params[:, 0, page, :, slot],
                       order[slot][:, None, None, :], G)  # as the cache holds it now
        outs.append(back.transpose(0, 1).to(t).contiguous())
    return {"k": outs[0], "v": outs[1]}


def _attend(s):
    case = s["case"]
    D, G, t, n, H, share = case["dim"], case["group"], TYPES[case["dtype"]], case["n"], case["heads"], case["share"]
    B, T, new = case["seqs"], s["tokens"], s["new"]
    ko, vo = _order(D)
    pages = s["table"].long().clamp(min=0)
    parts = [p[:, 0, pages] for p in _parts(s["pool"], case)]  # [n, B, maxp, H, PAGE, ...]
    keys = _values(parts[0], parts[1], ko, G).transpose(2, 3).flatten(3, 4)  # [n, B, H, L, D]
    values = _values(parts[2], parts[3], vo, G).transpose(2, 3).flatten(3, 4)
    L = keys.shape[3]
    row = torch.arange(new, device="cuda")[None, :] + s["start"][:-1, None]  # [B, new]
    there = row < s["start"][1:, None]
    at = row.clamp(max=T - 1).long()
    q = s["q"].float()[:, at].unflatten(3, (H, share)).permute(0, 1, 3, 4, 2, 5).flatten(3, 4)  # [n,B,H,share*new,D]
    score = torch.matmul(q, keys.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    score = score.unflatten(3, (share, new))  # [n, B, H, share, new, L]
    pos = torch.where(there, s["pos"][at], -1)[:, :, None]
    j = torch.arange(L, device="cuda")
    seen = (j <= pos) & (j < s["len"][:, None, None])
    if case["window"]:
        seen &= j > pos - case["window"]
    score = score.masked_fill(~seen[None, :, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p.flatten(3, 4), values * (j < s["len"][:, None])[None, :, None, :, None])
    o = o.unflatten(3, (share, new)).permute(0, 1, 4, 2, 3, 5).flatten(3, 4)[:, there]  # [n, T, Hq, D]
    if s["lse"] is None:
        return {"out": o.to(t)}
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 1, 4, 2, 3).flatten(3, 4)[:, there]
    return {"out": o.to(t), "lse": lse}


def _lowest(free, k):
    """The k-th (from 1) lowest page of those that are free; the count where there is none."""
    return torch.searchsorted(torch.cumsum(free.int(), 0), k)


def _fork(s):
    table, refs, lens, src, dst = s["table"], s["refs"], s["len"], s["src"].long(), s["dst"].long()
    old = table[dst]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    L, row = lens[src], table[src]
    full, part = L // PAGE, L % PAGE > 0
    want = torch.cumsum(part.int(), 0)
    free = refs == 0
    fails = part & (want > free.sum())
    new = _lowest(free, want.to(torch.int64))
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    shared = (j < full[:, None]) & ~fails[:, None]
    refs.index_add_(0, row.clamp(min=0).flatten().long(), shared.flatten().int())
    made = part & ~fails
    fresh, last = new[made], row.gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0][made].long()
    refs[fresh] = 1
    s["pool"][:, :, fresh] = s["pool"][:, :, last]
    own_page = (j == full[:, None]) & made[:, None]
    table[dst] = torch.where(shared, row, torch.where(own_page, new[:, None].int(), -1)).int()
    lens[dst] = torch.where(fails, 0, L)
    s["info"][:3] = torch.stack([(refs == 0).sum(), fails.sum(), made.sum()]).int()
    return {"table": table, "refs": refs, "len": lens, "info": s["info"][:3], "pool": s["pool"].view(torch.int64)}


def _compact(s):
    table, refs = s["table"], s["refs"]
    live = refs > 0
    count = live.sum()
    index = torch.arange(refs.numel(), device="cuda")
    moves = live & (index >= count)
    slot = _lowest(~live, torch.cumsum(moves.int(), 0))
    remap = torch.where(moves, slot, torch.where(live, index, -1)).int()
    src = index[moves]
    s["pool"][:, :, slot[moves]] = s["pool"][:, :, src]
    s["remap"].copy_(remap)
    s["new_refs"].zero_()
    s["new_refs"][remap[live].long()] = refs[live]
    s["new_table"].copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], -1))
    s["info"][:2] = torch.stack([(~live).sum(), moves.sum()]).int()
    return {"table": s["new_table"], "refs": s["new_refs"], "remap": s["remap"], "info": s["info"][:2],
            "pool": s["pool"].view(torch.int64)}


def _act(y, act, erf=torch.erf, tanh=torch.tanh, exp=torch.exp):
    if act == "relu":
        return torch.where(y > 0, y, torch.zeros_like(y))
    if act == "gelu":
        return 0.5 * y * (1 + erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "silu":
        return y / (1 + exp(-y))
    return y


def _linear(s):
    case = s["case"]
    y = torch.matmul(s["x"].float(), s["w"].float().transpose(-1, -2)) + s["bias"].float()[:, None]
    y = _act(y, case["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(TYPES[case["dtype"]])}


# ------------------------------------------------------------------ the framework's calls
def _cache(s):
    """The handle of a cache that a serving program makes once."""
    from driven_collective_communication_gb300 import dcc
    case = s["case"]
    return dcc.Kv4Cache(list(s["pool"]), s["table"], s["len"], s.get("refs"), kv_heads=case["heads"],
                        head_dim=case["dim"], group=case["group"], dtype=case["dtype"])


def _run_own(s):
    from driven_collective_communication_gb300 import dcc
    op, case = s["case"]["op"], s["case"]
    if "h" not in s:  # what a program sets up once: the handle, the ranks' buffers as lists, a workspace
        s["h"] = h = {} if op == "linear" else {"cache": _cache(s)}
        for name in ("k", "v", "k_out", "v_out", "q", "out", "lse", "w", "bias", "res", "y"):
            if s.get(name) is not None:
                h[name] = dcc.Ranks(list(s[name]))
        if op == "linear":
            h["x"] = dcc.Ranks([s["x"]] * case["n"])
        elif op == "attend":
            h["ws"] = h["cache"].attention_workspace(s["q"].shape[2])
        elif op in ("fork", "compact"):
            h["ws"] = h["cache"].pages_workspace()
    h = s["h"]
    if op == "linear":
        dcc.dcc_linear(h["w"], h["x"], h["y"], bias=h["bias"], residual=h.get("res"), act=case["act"])
        return {"y": s["y"]}
    cache = h["cache"]
    if op == "append":
        cache.append(h["k"], h["v"], s["start"])
        cache.read(h["k_out"], h["v_out"], s["start"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attend":
        cache.attention(h["q"], h["out"], s["start"], max_new=s["new"], workspace=h["ws"], lse=h.get("lse"),
                        window=case["window"])
        return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}
    if op == "fork":
        cache.fork(s["src"], s["dst"], workspace=h["ws"], info=s["info"])
        return {"table": s["table"], "refs": s["refs"], "len": s["len"], "info": s["info"][:3],
                "pool": s["pool"].view(torch.int64)}
    cache.compact(s["new_table"], s["new_refs"], s["remap"], workspace=h["ws"], info=s["info"])
    return {"table": s["new_table"], "refs": s["new_refs"], "remap": s["remap"], "info": s["info"][:2],
            "pool": s["pool"].view(torch.int64)}


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "attend": _attend, "fork": _fork, "compact": _compact,
            "linear": _linear}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n = case["n"]
    if case["op"] == "linear":
        T, R, K = case["tokens"], case["rows"], case["k"]
        io = n * R * K + T * K + n * R + n * T * R * (2 if case["residual"] else 1)
        return {"bytes": 2 * io, "flops": 2 * n * T * R * K}
    D, H = case["dim"], case["heads"]
    held = D // 2 + 4 * (D // case["group"])  # bytes of one token's K (or V) of one head
    if case["op"] == "append":
        T = sum(_lengths(case)[1])
        return {"bytes": 2 * n * T * H * (2 * D + held + held + 2 * D), "flops": 0}
    if case["op"] == "attend":
        lens, news = _lengths(case)
        w, pairs, keys = case["window"], 0, 0
        for m, t in zip(lens, news):
            if m:
                pairs += sum(min(x + 1, w) if w else x + 1 for x in range(m - t, m))
                keys += min(m, w + t - 1) if w else m
        T, Hq = sum(news), H * case["share"]
        b = 2 * n * H * keys * held + n * T * Hq * D * 4 + (n * T * Hq * 4 if case["new"] == 1 else 0)
        return {"bytes": b, "flops": 4 * n * Hq * D * pairs}
    B, L = case["seqs"], case["length"]
    lens = [max(1, L - (i * 389) % max(1, L // 2)) for i in range(B)]
    page = case["layers"] * H * _block(D, case["group"]) * n
    maxp = -(-L // PAGE) + 1
    if case["op"] == "fork":  # one partial page for each dropped beam, and the rows of the table
        return {"bytes": (B // 2) * (2 * page + 16 * maxp), "flops": 0}
    pages = sum(-(-m // PAGE) for m in lens) + B + 5
    live = sum(-(-m // PAGE) for m in lens) // 2
    moved = live * (pages - live) // pages  # pages in random order
    return {"bytes": moved * 2 * page + 8 * B * maxp + 12 * pages, "flops": 0}


# ------------------------------------------------------------------ 64 bits
def _exact_rows(s, r, h, b, which):
    """K or V of one sequence and head, from the layout's definition, in 64 bits."""
    case = s["case"]
    D, group, t = case["dim"], case["group"], TYPES[case["dtype"]]
    m = int(s["len"][b])
    pages = s["table"][b, :-(-m // PAGE)].long()
    blk = s["pool"][r, 0, pages, h]  # [pages, block]
    base, half = (0 if which == "k" else PAGE * D // 2), PAGE * D // 2
    ng = D // group
    raw = blk[:, base:base + half].reshape(-1, D // 2)[:m].to(torch.int64)
    pbase = PAGE * D + (0 if which == "k" else PAGE * ng * 4)
    par = blk[:, pbase:pbase + PAGE * ng * 4].contiguous().view(t).reshape(-1, ng, 2)[:m].double()
    d = torch.arange(D, device="cuda")
    if which == "k":  # where channel d sits in the row
        place = ((d % 32) // 8 * (D // 32) + d // 32) * 8 + d % 8
        place = place.expand(m, D)
    else:
        tok = torch.arange(m, device="cuda")[:, None] % PAGE
        chunk = (d % 8)[None, :].expand(m, D)
        if D == 128:
            chunk = torch.where(tok % 8 >= 4, (chunk + 4) % 8, chunk)
        place = chunk * (D // 8) + 2 * (d // 16) + (d % 16) // 8
    code = (torch.gather(raw, 1, place // 2) >> (4 * (place % 2))) & 15
    return par[:, :, 1].repeat_interleave(group, 1) + par[:, :, 0].repeat_interleave(group, 1) * code.double()


def exact(case, seed):
    s = prepare(case, seed)
    t, op = TYPES[case["dtype"]], case["op"]
    if op == "linear":
        out = []
        for r in range(case["n"]):
            y = s["x"].double() @ s["w"][r].double().T + s["bias"][r].double()
            y = _act(y, case["act"])
            out.append(y if s["res"] is None else y + s["res"][r].double())
        return {"y": torch.stack(out)}
    if op == "append":
        outs = {}
        for name in ("k", "v"):
            x = s[name].double().unflatten(-1, (-1, case["group"]))
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            step = ((hi - lo) / 15).to(t).double()
            code = torch.where(step > 0, ((x - lo) / torch.where(step > 0, step, 1.0)).round().clamp(0, 15), 0.0)
            outs[name] = (lo + step * code).flatten(-2)
        return outs
    if op != "attend":
        return None
    n, T, H, share, D = case["n"], s["tokens"], case["heads"], case["share"], case["dim"]
    if 4 * work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(n, T, H * share, D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, T, H * share), -math.inf, dtype=torch.float64, device="cuda")
    starts, lens = s["start"].tolist(), s["len"].tolist()
    for b in range(case["seqs"]):
        m, a, z = lens[b], starts[b], starts[b + 1]
        if m == 0:
            continue
        pos = torch.arange(m - (z - a), m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None, :]
        hidden = j > pos
        if case["window"]:
            hidden |= j <= pos - case["window"]
        for r in range(n):
            for h in range(H):
                K, V = _exact_rows(s, r, h, b, "k"), _exact_rows(s, r, h, b, "v")
                q = s["q"][r, a:z, h * share:(h + 1) * share].double().transpose(0, 1)  # [share, new, D]
                x = (q @ K.T) / math.sqrt(D)
                x = x.masked_fill(hidden, -math.inf)
                L = torch.logsumexp(x, -1)
                out[r, a:z, h * share:(h + 1) * share] = (torch.exp(x - L[..., None]) @ V).transpose(0, 1)
                lse[r, a:z, h * share:(h + 1) * share] = L.T
    return {"out": out, "lse": lse} if s["lse"] is not None else {"out": out}
