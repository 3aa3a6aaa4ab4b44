"""Decoding with drafted trees over N virtual ranks: every step verifies a small
tree of tokens for each sequence at once and keeps the branch that the model
agrees with.

Per step and sequence: room for the tree's rows (dcc_kv4_reserve), the decoder
block with its rows in the cache and the tree's attention over it
(dcc_kv4_attention_tree), the vocabulary-parallel output layer (dcc_linear), the
best tokens of every row with their log probabilities (dcc_token_logprobs), and
the accepted branch moved to the front of the cache (dcc_kv4_keep).  The next
tree is drafted from the last accepted row's top alternatives.  With a window the
prompts see its tokens and the first ones only (dcc_kv4_attention_sinks).

  python -m driven_collective_communication_gb300.examples.speculate
"""
import torch

from driven_collective_communication_gb300 import dcc
from driven_collective_communication_gb300.examples.decode_block import Block, norm

TREE = [-1, 0, 0, 0, 1, 1, 2, 4]  # the parent of each drafted token; 0 is the last sampled one


def ancestors(parents):
    """For each drafted token, those that its row sees: itself and its ancestors."""
    out = []
    for j, p in enumerate(parents):
        out.append([*(out[p] if p >= 0 else []), j])
    return out


class Speculator(Block):
    """A decoder block between an embedding and a vocabulary-parallel output layer."""

    def __init__(self, vocab=1000, top=4, window=0, sinks=0, parents=TREE, **shape):
        super().__init__(**shape)
        g = torch.Generator(device="cuda").manual_seed(7)
        self.vocab, self.top, self.window, self.sinks, self.parents = vocab, top, window, sinks, parents
        self.columns = -(-vocab // self.n // 8) * 8  # of a rank; the last ones are padding
        self.embed = torch.randn(vocab, self.hidden, device="cuda", generator=g).bfloat16()
        self.w_head = [(2 * torch.randn(self.columns, self.hidden, device="cuda", generator=g)
                        * self.hidden ** -0.5).bfloat16() for _ in range(self.n)]
        sees = ancestors(parents)
        self.words = -(-len(parents) // 32)
        rows = torch.zeros(len(parents), self.words, dtype=torch.int64)
        for j, s in enumerate(sees):
            for a in s:
                rows[j, a // 32] |= 1 << (a % 32)
        self.tree = torch.where(rows >= 1 << 31, rows - (1 << 32), rows).to(torch.int32).cuda()
        self.sees = torch.zeros(len(parents), len(parents), dtype=torch.bool, device="cuda")
        for j, s in enumerate(sees):
            self.sees[j, s] = True
        self.mask = None  # of the batch: drafted rows, or None for a prompt
        self.ws_logprobs = dcc.token_logprobs_workspace(self.n, 1, self.columns, top)

    def attend(self, q, out, start, max_new):
        if self.mask is None:
            self.cache.attention_sinks(q, out, start, max_new, self.ws_attention, self.window, self.sinks)
        else:
            self.cache.attention_tree(q, out, start, self.mask, max_new, self.ws_attention, window=self.window,
                                      sinks=self.sinks)

    def unseen(self, s, length, t):
        j = torch.arange(length, device="cuda")[None, :]
        first = length - t
        if self.mask is None:
            x = torch.arange(first, length, device="cuda")[:, None]
            return (j > x) | ((j <= x - self.window) & (j >= self.sinks) if self.window else j < 0)
        hide = torch.zeros(t, length, dtype=torch.bool, device="cuda")
        hide[:, first:] = ~self.sees
        if self.window:
            count = self.sees.sum(-1, keepdim=True)
            hide[:, :first] = (j[:, :first] < first + count - self.window) & (j[:, :first] >= self.sinks)
        return hide

    def score(self, h, target):
        """Log probabilities of the target tokens (-1: none), entropy, and the best tokens of every row of h."""
        T = h.shape[0]
        logits = [torch.empty(T, self.columns, dtype=torch.bfloat16, device="cuda") for _ in range(self.n)]
        dcc.dcc_linear(self.w_head, [norm(h)] * self.n, logits)
        lp, entropy = (torch.empty(T, dtype=torch.float32, device="cuda") for _ in range(2))
        ids = torch.empty(T, self.top, dtype=torch.int32, device="cuda")
        tops = torch.empty(T, self.top, dtype=torch.float32, device="cuda")
        dcc.dcc_token_logprobs(logits, target, lp, self.ws_logprobs, entropy=entropy, top_ids=ids, top_logprobs=tops,
                               vocab=self.vocab)
        return lp, entropy, ids, tops, logits


def draft(model, best, g):
    """A tree's tokens: the last sampled one, its best alternatives below it, and below those any."""
    tokens = torch.randint(0, model.vocab, (len(model.parents),), device="cuda", generator=g, dtype=torch.int32)
    tokens[0] = best[0]
    children = [j for j, p in enumerate(model.parents) if p == 0]
    for j, t in zip(children, best[1:].tolist()):
        tokens[j] = t
    return tokens


def accept(model, tokens, best):
    """The branch from the root on whose tokens the model itself would have taken."""
    path = [0]
    while True:
        hits = [j for j, p in enumerate(model.parents) if p == path[-1] and tokens[j] == best[path[-1]]]
        if not hits:
            return path
        path.append(hits[0])


def run(model=None, prompts=(200, 65, 300), steps=4, verbose=True):
    """Prompts, then `steps` verified trees.  Returns, per pass, the largest
    difference from the plain form relative to its root mean square, that of the
    log probabilities, and the tokens kept."""
    model = model or Speculator()
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    B, N = len(prompts), len(model.parents)
    seen = []

    def one(news, tokens, mask):
        start = model.grow(news)
        model.mask = mask
        h = model.embed[tokens.long()]
        got, want = model.forward(h, start, max(news)), model.plain(h, start, news)
        off = ((got.float() - want.float()).abs().max() / want.float().square().mean().sqrt()).item()
        lp, _, ids, _, logits = model.score(got, tokens)
        x = torch.cat([t.float() for t in logits], 1)[:, :model.vocab]
        plain = torch.log_softmax(x, -1).gather(1, tokens.long()[:, None])[:, 0]
        assert torch.equal(ids[:, 0], (x == x.amax(-1, keepdim=True)).int().argmax(-1).int())  # (the lowest of equals)
        return start, ids, off, (lp - plain).abs().max().item()

    def keep(start, paths):
        flat = [x for p in paths for x in p + [-1] * (N - len(p))]
        kept, before = [len(p) for p in paths], model.cache.lengths.tolist()
        info = torch.zeros(4, **i32)
        model.cache.keep(start, torch.tensor(flat, **i32), torch.tensor(kept, **i32), model.ws_pages, info)
        assert dcc.dcc_local_check() == dcc.DCC_OK and int(info[1]) == 0
        assert model.cache.lengths.tolist() == [m - N + k for m, k in zip(before, kept)]
        return kept

    tokens = torch.randint(0, model.vocab, (sum(prompts),), generator=g, **i32)
    start, ids, off, lp = one(list(prompts), tokens, None)
    seen.append((off, lp, list(prompts)))
    last = [ids[e - 1] for e in start[1:].tolist()]  # the best tokens after each prompt
    for step in range(steps):
        trees = [draft(model, b, g) for b in last]
        start, ids, off, lp = one([N] * B, torch.cat(trees), model.tree.repeat(B, 1))
        best = ids.view(B, N, -1)
        if step % 2:
            # (an untrained model agrees with few drafts: all are given up, and come
            # again with a child of the root that it will agree with)
            seen.append((off, lp, keep(start, [[]] * B)))
            for s in range(B):
                trees[s][1] = best[s, 0, 0]
            start, ids, off, lp = one([N] * B, torch.cat(trees), model.tree.repeat(B, 1))
            best = ids.view(B, N, -1)
        paths = [accept(model, trees[s].tolist(), best[s, :, 0].tolist()) for s in range(B)]
        last = [best[s, p[-1]] for s, p in enumerate(paths)]
        seen.append((off, lp, keep(start, paths)))
        if verbose:
            print("step %d: %s kept, %s cached; off by %.4f of the rms, log probabilities by %.1e"
                  % (step, seen[-1][2], model.cache.lengths.tolist(), off, lp))
    return seen


if __name__ == "__main__":
    run()
