"""Cases, plain forms and exact values of the operators that a serving program
with drafted tokens and long streams adds to the decoder's: attention of a tree
of drafted tokens and attention with a sliding window and first tokens that stay
visible, both over the 4-bit key/value cache; the accepted drafted tokens kept in
that cache; and log probabilities, entropy and top alternatives of
vocabulary-parallel logits.

Every operator works on n virtual ranks at once; rank r holds its own heads or
columns.  With ``own`` false, ``run`` is the plain form in elementary torch
operations in 32 bits; with ``own`` true it makes the framework's calls.

Cache layout (64 tokens per page, one block per page and key/value head):
  K codes 64 x D/2 bytes | V codes 64 x D/2 | K params 64 x D/group x (step, lo)
  | V params, each param of the cache's 16-bit type; value = lo + step * code.
"""
import math

import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    cache = dict(n=8, heads=1, dim=128, group=64, dtype="bf16")
    tree = dict(cache, op="tree", share=8, window=0, sinks=0)
    sinks = dict(cache, op="sinks", share=8, sinks=4)
    keep = dict(cache, op="keep")
    tops = dict(op="logprobs", n=8, scale=1.0)
    return [
        # a single request's small tree early in its answer: the latency of one verification step
        dict(tree, name="tree-one", seqs=1, new=8, length=777, share=4),
        # a serving batch of uneven requests, each with a tree of up to 32 drafted tokens
        dict(tree, name="tree-batch", seqs=32, new=32, length=4096),
        # one very long document and a wide tree, few query heads per cache head, finer groups
        dict(tree, name="tree-long", seqs=1, new=63, length=131109, share=4, heads=2, group=32, dtype="fp16"),
        # small trees of streaming requests with a window and kept first tokens, 64-wide heads
        dict(tree, name="tree-window", seqs=16, new=13, length=3001, share=4, heads=2, dim=64, group=32, dtype="fp16",
             window=1024, sinks=4),
        # one streaming request: the latency of one decode step
        dict(sinks, name="sinks-one", seqs=1, new=1, length=5001, window=1024, share=4, heads=2, dim=64, group=32,
             dtype="fp16"),
        # long-running streams with idle slots, the usual decode step
        dict(sinks, name="sinks-decode", seqs=64, new=1, length=16384, window=4000),
        # chunks of two prompts of a streaming model
        dict(sinks, name="sinks-prompt", seqs=2, new=2048, length=8192, window=1024, sinks=64),
        # drafted chains of five, some of each accepted, and room for the next ones: nothing moves
        dict(keep, name="keep-chain", seqs=64, new=5, length=1030, layers=4, tree=False),
        # drafted trees: the accepted branch moves to the front in all layers
        dict(keep, name="keep-tree", seqs=64, new=32, length=601, layers=16, tree=True),
        # one sampled token of a small vocabulary, logits in 32 bits
        dict(tops, name="logprobs-token", tokens=1, columns=4000, vocab=32000, dtype="fp32", top=5),
        # the rows of eight drafted trees: the best token of each and the drafted tokens' probabilities
        dict(tops, name="logprobs-batch", tokens=256, columns=16384, vocab=131000, dtype="bf16", top=1),
        # a prompt scored with alternatives, odd shards, at a temperature
        dict(tops, name="logprobs-prompt", tokens=2048, columns=19001, vocab=152003, dtype="fp16", top=20, scale=1.25),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "sinks", "sinks", "sinks", "keep", "logprobs", "logprobs"])
    n = rng.choice([1, 2, 4, 8])
    if op == "logprobs":
        c = dict(op=op, n=n, dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=_log(rng, 1, 2048),
                 columns=_log(rng, 1000, 152064) // n + 1, top=rng.choice([0, 1, 2, 5, 20, 50]),
                 scale=rng.choice([1.0, 1.25, 0.7]))
        while c["tokens"] * c["columns"] * n > 2048 * 8 * 19001 // 2:
            c["tokens"] = c["tokens"] // 2 + 1
        return dict(c, vocab=n * c["columns"] - rng.randint(0, min(n * c["columns"] - 900, c["columns"] - 1)))
    c = dict(op=op, n=n, heads=rng.choice([1, 2, 3, 4]), dim=rng.choice([64, 128]), group=rng.choice([32, 64]),
             dtype=rng.choice(["bf16", "fp16"]))
    if op == "keep":
        c = dict(c, seqs=_log(rng, 1, 64), new=_log(rng, 1, 128), layers=rng.choice([1, 2, 5, 16]),
                 tree=rng.random() < 0.7)
        c["length"] = c["new"] + _log(rng, 1, 1000)
        while c["seqs"] > 1 and c["seqs"] * (c["length"] + 64) * c["layers"] * c["heads"] * n > 64 * 640 * 128:
            c["seqs"] = c["seqs"] // 2
        return c
    c = dict(c, share=rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), seqs=_log(rng, 1, 64), length=_log(rng, 1, 131072))
    if op == "tree":
        c["new"] = _log(rng, 1, 256)
        c["window"] = _log(rng, 16, 4096) if rng.random() < 0.3 else 0
    else:
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        c["window"] = _log(rng, 16, 8192)
    c["sinks"] = rng.choice([1, 4, 16, 64, 100]) if c["window"] else 0
    c["length"] = max(c["length"], c["new"])

    def large(x):
        keys = x["length"] * x["heads"] * n
        return x["seqs"] * keys > 1 << 21 or x["seqs"] * keys * x["share"] * x["new"] > 1 << 29
    while c["seqs"] > 1 and large(c):
        c["seqs"] //= 2
    while large(c) and c["length"] > 16:
        if c["new"] > 16 and c["length"] < 4 * c["new"]:
            c["new"] = c["new"] // 2 + 1
        c["length"] = max(c["new"], c["length"] // 2 + 1)
    return c


def _lengths(case):
    """Tokens each sequence holds with this step's new ones, and how many of them are new."""
    B, L, new = case["seqs"], case["length"], case["new"]
    lens, news = [], []
    for s in range(B):
        m = L if s == 0 else max(1, L - (s * 7919 * 13) % max(1, (15 * L) // 16))
        if case["op"] == "keep":
            m = L - (s * 389) % max(1, L // 2)
        t = new if new == 1 or s == 0 else max(1, min(m, new - (s * 613) % max(1, new // 2)))
        if case["op"] != "keep" and s % 32 == 31:  # an idle slot, of a decode step with a row of its own
            m, t = 0, 1 if new == 1 else 0
        lens.append(max(m, t) if m else 0)
        news.append(t)
    return lens, news


def _kept(case, news):
    """How many of its drafted tokens each sequence accepts."""
    return [min(t, 1 + (s * 5) % 7) for s, t in enumerate(news)]


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


def _trees(case, news, g):
    """Ancestors (and itself) of each drafted token, [sequences, new, new]: token j
    continues the cached text or one of the few tokens before it."""
    B, new = case["seqs"], max(1, case["new"])
    j = torch.arange(new, device="cuda")
    back = (torch.rand(B, new, device="cuda", generator=g) ** 2 * 6).long()
    parent = j[None, :] - 1 - back
    sees = torch.eye(new, device="cuda").repeat(B, 1, 1)
    step = (j[None, None, :] == parent[:, :, None]).float()  # [B, token, parent]
    for _ in range(new.bit_length()):
        sees = ((sees + torch.matmul(step, sees)) > 0).float()
        step = (torch.matmul(step, step) > 0).float()
    return sees > 0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t, n = TYPES[case["dtype"]], case["n"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] == "logprobs":
        T, C, V, k = case["tokens"], case["columns"], case["vocab"], case["top"]
        x = torch.empty(n, T, C, dtype=t, device="cuda")
        loud = 1.0 + 2.0 * torch.rand(T, 1, device="cuda", generator=g)  # rows from flat to peaked
        rows = torch.arange(T, device="cuda")[:, None]
        for r in range(n):
            ids = r * C + torch.arange(C, device="cuda")[None, :]
            y = normal(T, C) * loud
            # every 16th row is restricted by a grammar
            x[r] = y.masked_fill_((rows % 16 == 15) & (ids % 97 != 0), -math.inf).to(t)
        target = torch.randint(0, V, (T,), device="cuda", generator=g)
        rows = rows[:, 0]
        target = torch.where(rows % 16 == 15, target - target % 97, target)
        target = torch.where(rows % 23 == 22, -1, target).to(torch.int32)  # rows without a token to score
        out = dict(dtype=torch.float32, device="cuda")
        return {"case": case, "logits": x, "target": target, "logprob": torch.empty(T, **out),
                "entropy": torch.empty(T, **out), "ids": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                "top": torch.empty(T, k, **out)}

    H, D = case["heads"], case["dim"]
    s = {"case": case}
    lens, news = _lengths(case)
    starts = [0]
    for x in news:
        starts.append(starts[-1] + x)
    T = starts[-1]
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["news"] = torch.tensor(news, device="cuda")
    s["tokens"], s["new"] = T, max(news)
    # the sequence of each new token, and its number there
    s["seq"] = torch.repeat_interleave(torch.arange(len(news), device="cuda"), s["news"])
    s["num"] = torch.arange(T, device="cuda") - s["start"][s["seq"]]
    maxp = max(-(-m // PAGE) for m in lens) + (1 if case["op"] == "keep" else 0)
    spare = 3 if case["op"] != "keep" else 2 * case["seqs"]
    s["table"], pages = _pages(lens, maxp, g, spare)
    s["pool"] = _pool(g, n, case.get("layers", 1), pages, case)
    if case["op"] == "keep":
        kept = _kept(case, news)
        s["kept"] = torch.tensor(kept, dtype=torch.int32, device="cuda")
        s["add"] = torch.tensor([a - b for a, b in zip(news, kept)], dtype=torch.int32, device="cuda")
        # an ascending choice of so many drafted tokens; a chain keeps its first ones
        order = torch.rand(case["seqs"], case["new"], device="cuda", generator=g)
        j = torch.arange(case["new"], device="cuda")[None, :]
        if not case["tree"]:
            order = j.float().expand(order.shape)
        place = torch.where(j < s["news"][:, None], order, 2.0 + j).argsort(-1).argsort(-1)
        chosen = place < s["kept"][:, None]
        path = torch.where(chosen, j, case["new"] + j).sort(-1).values
        s["path"] = torch.where(path < case["new"], path, -1).to(torch.int32)[s["seq"], s["num"]].contiguous()
        live = s["table"][s["table"] >= 0].long()
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda").index_add_(
            0, live, torch.ones_like(live, dtype=torch.int32))
        s["info"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        s["room"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "tree":
        words = -(-s["new"] // 32)
        sees = _trees(case, news, g)[s["seq"], s["num"]]  # [tokens, new]
        sees &= torch.arange(case["new"], device="cuda")[None, :] < s["news"][s["seq"]][:, None]
        bits = torch.zeros(T, 32 * words, dtype=torch.int64, device="cuda")
        bits[:, :sees.shape[1]] = sees
        w = (bits.view(T, words, 32) << torch.arange(32, device="cuda")).sum(-1)
        s["mask"] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    Hq = H * case["share"]
    s["q"] = normal(n, T, Hq, D).to(t)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n, T, Hq, dtype=torch.float32, device="cuda") if case["new"] == 1 else None
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

    def codes(a):
        return pool[..., a:a + c].unflatten(-1, (PAGE, D // 2))

    def params(a):
        return pool.view(t)[..., a // 2:(a + q) // 2].unflatten(-1, (PAGE, ng, 2))
    return codes(0), params(2 * c), codes(c), params(2 * c + q)


def _values(codes, params, order, group):
    """lo + step * code of unpacked rows [..., PAGE, D/2] in channel order."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    out = torch.empty_like(c)
    out.scatter_(-1, order.expand(c.shape), c)
    par = params.float().repeat_interleave(group, -2)
    return par[..., 1] + par[..., 0] * out.float()


def _seen(s, L):
    """Which of L cached positions each new token sees: [tokens, L]."""
    case = s["case"]
    W, S = case["window"], case["sinks"]
    num, first = s["num"][:, None], (s["len"] - s["news"])[s["seq"]][:, None]
    j = torch.arange(L, device="cuda")[None, :]
    if case["op"] == "sinks":
        x = first + num
        return (j <= x) & ((j > x - W) | (j < S)) & (j < s["len"][s["seq"]][:, None])
    d = j - first  # a drafted token's number
    word = s["mask"].gather(1, (d // 32).clamp(0, s["mask"].shape[1] - 1))
    drafted = (d >= 0) & (d < s["news"][s["seq"]][:, None]) & (((word >> (d % 32)) & 1) == 1)
    context = d < 0
    if W:
        count = drafted.sum(-1, keepdim=True)
        context &= (j >= first + count - W) | (j < S)
    return drafted | context


def _attend(s):
    case = s["case"]
    D, G, t, H, share = case["dim"], case["group"], TYPES[case["dtype"]], case["heads"], case["share"]
    T, new = s["tokens"], s["new"]
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
    seen = _seen(s, L)[at] & there[:, :, None]  # [B, new, L]
    score = score.masked_fill(~seen[None, :, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    j = torch.arange(L, device="cuda")
    o = torch.matmul(p.flatten(3, 4), values * (j < s["len"][:, None])[None, :, None, :, None])
    o = o.unflatten(3, (share, new)).permute(0, 1, 4, 2, 3, 5).flatten(3, 4)[:, there]  # [n, T, Hq, D]
    if s["lse"] is None:
        return {"out": o.to(t)}
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 1, 4, 2, 3).flatten(3, 4)[:, there]
    return {"out": o.to(t), "lse": lse}


def _keep(s):
    """Keep the accepted tokens, then let each sequence hold as many as before."""
    case = s["case"]
    table, refs, lens, kept = s["table"], s["refs"], s["len"], s["kept"].long()
    maxp = table.shape[1]
    moved = s["num"] < kept[s["seq"]]  # new tokens that some accepted one goes to
    seq, dst = s["seq"][moved], s["num"][moved]
    first = (lens - s["news"])[seq].long()
    src = s["path"][moved].long()
    places = []
    for x in (first + src, first + dst):
        places.append((table[seq, x // PAGE].long(), x % PAGE))
    (sp, ss), (dp, ds) = places
    D = case["dim"]
    kc, kp, vc, vp = _parts(s["pool"], case)
    new = []
    for part in (kc, kp, vc, vp):
        rows = part.permute(2, 4, 0, 1, 3, *range(5, part.dim()))[sp, ss]  # [rows, n, layers, H, ...]
        if part is vc and D == 128:  # the chunks' halves change places with bit 2 of the token
            swap = ((ss ^ ds) >> 2) & 1 == 1
            rows = torch.where(swap.view(-1, 1, 1, 1, 1), rows.roll(D // 4, -1), rows)
        new.append(rows)
    for part, rows in zip((kc, kp, vc, vp), new):
        part.permute(2, 4, 0, 1, 3, *range(5, part.dim()))[dp, ds] = rows
    held = -(-lens // PAGE)
    lens -= (s["news"] - kept).int()
    now = -(-lens // PAGE)
    j = torch.arange(maxp, device="cuda")[None, :]
    gone = (j >= now[:, None]) & (j < held[:, None])
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().int())
    table.masked_fill_(gone, -1)
    s["info"][:3] = torch.stack([(refs == 0).sum(), 0 * kept.sum(), (src != dst).sum()]).int()
    lens += s["add"]
    then = -(-lens // PAGE)
    want = then - now
    index = torch.cumsum(want, 0)[:, None] - want[:, None] + j - now[:, None] + 1
    free = torch.cumsum((refs == 0).int(), 0)
    grows = (j >= now[:, None]) & (j < then[:, None])
    given = torch.searchsorted(free, index.int().contiguous())
    table.copy_(torch.where(grows, given.int(), table))
    refs[given[grows]] = 1
    s["room"][:3] = torch.stack([(refs == 0).sum(), 0 * want.sum(), want.sum()]).int()
    return _books(s)


def _books(s):
    return {"table": s["table"], "refs": s["refs"], "len": s["len"], "info": s["info"][:3], "room": s["room"][:3],
            "pool": s["pool"].view(torch.int64)}


def _logprobs(s):
    case = s["case"]
    T, V, k, outs = case["tokens"], case["vocab"], case["top"], []
    for a in range(0, T, 256):
        x = s["logits"][:, a:a + 256].float().transpose(0, 1).flatten(1)[:, :V]
        target = s["target"][a:a + 256].long()[:, None]
        y = x * case["scale"]
        m = y.amax(-1, keepdim=True)
        e = torch.exp(y - m)
        z = e.sum(-1, keepdim=True)
        log = y - m - torch.log(z)
        p = e / z
        entropy = -torch.where(p > 0, p * log, torch.zeros_like(p)).sum(-1)
        lp = torch.where(target >= 0, log.gather(1, target.clamp(min=0)), torch.zeros_like(z))[:, 0]
        if k == 1:
            ids = (x == x.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
        else:
            ids = x.sort(dim=-1, descending=True, stable=True).indices[:, :k]
        outs.append((lp, entropy, ids.int()[:, :k], log.gather(1, ids)[:, :k]))
    lp, entropy, ids, top = (torch.cat(t) for t in zip(*outs))
    return {"logprob": lp, "entropy": entropy, "ids": ids, "top": top}


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    from driven_collective_communication_gb300 import dcc
    op, case = s["case"]["op"], s["case"]
    if "h" not in s:  # what a program sets up once: the handle, the ranks' buffers as lists, a workspace
        s["h"] = h = {}
        if op == "logprobs":
            h["logits"] = dcc.Ranks(list(s["logits"]))
            h["ws"] = dcc.token_logprobs_workspace(case["n"], case["tokens"], case["columns"], case["top"])
        else:
            h["cache"] = dcc.Kv4Cache(list(s["pool"]), s["table"], s["len"], s.get("refs"), kv_heads=case["heads"],
                                      head_dim=case["dim"], group=case["group"], dtype=case["dtype"])
            if op == "keep":
                h["ws"] = h["cache"].pages_workspace()
            else:
                for name in ("q", "out", "lse"):
                    h[name] = None if s[name] is None else dcc.Ranks(list(s[name]))
                h["ws"] = h["cache"].attention_workspace(s["q"].shape[2])
    h = s["h"]
    if op == "logprobs":
        dcc.dcc_token_logprobs(h["logits"], s["target"], s["logprob"], h["ws"], entropy=s["entropy"], top_ids=s["ids"],
                               top_logprobs=s["top"], vocab=case["vocab"], scale=case["scale"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}
    cache = h["cache"]
    if op == "keep":
        cache.keep(s["start"], s["path"], s["kept"], workspace=h["ws"], info=s["info"])
        cache.reserve(s["add"], workspace=h["ws"], info=s["room"])
        return _books(s)
    if op == "tree":
        cache.attention_tree(h["q"], h["out"], s["start"], s["mask"], max_new=s["new"], workspace=h["ws"],
                             lse=h["lse"], window=case["window"], sinks=case["sinks"])
    else:
        cache.attention_sinks(h["q"], h["out"], s["start"], max_new=s["new"], workspace=h["ws"], lse=h["lse"],
                              window=case["window"], sinks=case["sinks"])
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _attend, "sinks": _attend, "keep": _keep, "logprobs": _logprobs}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n = case["n"]
    if case["op"] == "logprobs":
        T, size = case["tokens"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * (case["vocab"] * size + 12 + 8 * case["top"]), "flops": 5 * T * case["vocab"]}
    D, H = case["dim"], case["heads"]
    held = D // 2 + 4 * (D // case["group"])  # bytes of one token's K (or V) of one head
    lens, news = _lengths(case)
    if case["op"] == "keep":  # each accepted token but a few moves; the table's rows and the counts are looked at
        moved = sum(_kept(case, news)) if case["tree"] else 0
        return {"bytes": moved * 4 * held * H * n * case["layers"] + 4 * case["seqs"] * (6 + news[0]), "flops": 0}
    W, S, pairs, keys = case["window"], case["sinks"], 0, 0
    for m, t in zip(lens, news):
        if m == 0:
            continue
        first = m - t
        if case["op"] == "tree":  # each drafted token sees the context and about six drafted tokens
            context = min(first, W + min(S, max(0, first - W))) if W else first
            pairs += t * (context + min(t, 6))
            keys += context + t
        else:
            pairs += sum(min(x + 1, W + min(S, max(0, x + 1 - W))) for x in range(first, m))
            keys += min(m, W + t - 1 + min(S, max(0, first - W + 1)))
    T, Hq = sum(news), H * case["share"]
    b = 2 * n * H * keys * held + n * T * Hq * D * 4 + (n * T * Hq * 4 if case["new"] == 1 else 0)
    return {"bytes": b, "flops": 4 * n * Hq * D * pairs}


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


def _exact_logprobs(s):
    case = s["case"]
    V, k, out = case["vocab"], case["top"], {"logprob": [], "entropy": [], "ids": [], "top": []}
    for t in range(case["tokens"]):
        x = s["logits"][:, t].reshape(-1)[:V]
        y = x.double() * case["scale"]
        log = y - torch.logsumexp(y, -1)
        aim = int(s["target"][t])
        out["logprob"].append(log[aim] if aim >= 0 else torch.zeros_like(log[0]))
        out["entropy"].append(torch.special.entr(torch.exp(log)).sum())
        # one whole number a token: the value's place in order, then the lowest id first
        b = x.float().view(torch.int32).long()
        b = torch.where(x == 0, 0, torch.where(b < 0, -(b & 0x7fffffff), b))
        ids = torch.topk((b << 32) + (V - torch.arange(V, device="cuda")), k).indices
        out["ids"].append(ids.int())
        out["top"].append(log[ids])
    return {name: torch.stack(v) for name, v in out.items()}


def exact(case, seed):
    op = case["op"]
    if op == "keep":
        return None
    if op != "logprobs" and 4 * case["seqs"] * case["length"] * case["new"] * case["n"] * case["heads"] \
            * case["share"] * case["dim"] > 4e12:
        return None
    s = prepare(case, seed)
    if op == "logprobs":
        return _exact_logprobs(s)
    n, T, H, share, D = case["n"], s["tokens"], case["heads"], case["share"], case["dim"]
    W, S = case["window"], case["sinks"]
    out = torch.zeros(n, T, H * share, D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, T, H * share), -math.inf, dtype=torch.float64, device="cuda")
    starts, lens = s["start"].tolist(), s["len"].tolist()
    for b in range(case["seqs"]):
        m, a, z = lens[b], starts[b], starts[b + 1]
        if m == 0 or a == z:
            continue
        first = m - (z - a)
        hidden = torch.ones(z - a, m, dtype=torch.bool, device="cuda")
        if op == "tree":
            word = s["mask"][a:z].long() & 0xffffffff
            bit = [(word[:, d // 32] >> (d % 32)) & 1 for d in range(z - a)]
            draft = torch.stack(bit, 1) == 1
            hidden[:, first:] = ~draft
            if W:
                for i, c in enumerate(draft.sum(-1).tolist()):
                    hidden[i, max(0, min(first, first + c - W)):first] = False
                    hidden[i, :min(S, first)] = False
            else:
                hidden[:, :first] = False
        else:
            x = torch.arange(first, m, device="cuda")[:, None]
            j = torch.arange(m, device="cuda")[None, :]
            hidden = (j > x) | ((j <= x - W) & (j >= S))
        for r in range(n):
            for h in range(H):
                K, V = _exact_rows(s, r, h, b, "k"), _exact_rows(s, r, h, b, "v")
                q = s["q"][r, a:z, h * share:(h + 1) * share].double().transpose(0, 1)  # [share, new, D]
                x = ((q @ K.T) / math.sqrt(D)).masked_fill(hidden, -math.inf)
                L = torch.logsumexp(x, -1)
                out[r, a:z, h * share:(h + 1) * share] = (torch.exp(x - L[..., None]) @ V).transpose(0, 1)
                lse[r, a:z, h * share:(h + 1) * share] = L.T
    return {"out": out, "lse": lse} if s["lse"] is not None else {"out": out}
