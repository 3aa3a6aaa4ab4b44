"""A tensor-parallel decoder block over N virtual ranks: prompts, then token by
token, then a beam step, on one GPU.

Per rank: a column-parallel projection to Q, K, V (dcc_linear), K and V into
the 4-bit cache, attention over it, the row-parallel output projection fused
with the AllReduce and the residual (dcc_linear_allreduce_tokens_residual), and
the same pair around the activation for the feed-forward half.  Pages come from
dcc_kv4_reserve; the beam step drops one sequence and refills it from another
(dcc_kv4_fork).

  python -m driven_collective_communication_gb300.examples.decode_block
"""
import torch

from driven_collective_communication_gb300 import dcc


class Block:
    """One decoder block; rank r holds Q heads r * q_heads .. and kv heads likewise."""

    def __init__(self, n=4, q_heads=8, kv_heads=1, dim=128, hidden=1024, ff=4096, seqs=3, max_tokens=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.q_heads, self.kv_heads, self.dim, self.hidden = n, q_heads, kv_heads, dim, hidden
        width = (q_heads + 2 * kv_heads) * dim

        def weight(rows, k):
            return [(torch.randn(rows, k, device="cuda", generator=g) * k ** -0.5).bfloat16() for _ in range(n)]
        self.w_qkv, self.w_out = weight(width, hidden), weight(hidden, q_heads * dim)
        self.w_up, self.w_down = weight(ff // n, hidden), weight(hidden, ff // n)
        self.b_qkv = [(0.1 * torch.randn(width, device="cuda", generator=g)).bfloat16() for _ in range(n)]
        self.b_up = [(0.1 * torch.randn(ff // n, device="cuda", generator=g)).bfloat16() for _ in range(n)]
        pages = max_tokens // dcc.DCC_KV4_PAGE
        self.cache = dcc.Kv4Cache.create(n, 1, seqs * pages, seqs, pages, kv_heads, dim, 64, "bf16")
        self.ws_attention = self.cache.attention_workspace(q_heads)
        self.ws_pages = self.cache.pages_workspace()
        self.buffers = {}

    def _buffers(self, tokens):
        """The activations of a batch size, registered once."""
        if tokens not in self.buffers:
            def make(width):
                return [torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda") for _ in range(self.n)]
            qkv = make((self.q_heads + 2 * self.kv_heads) * self.dim)
            b = {"qkv": qkv, "attn": make(self.q_heads * self.dim), "up": make(self.w_up[0].shape[0]),
                 "h": make(self.hidden)}
            self.buffers[tokens] = b
        return self.buffers[tokens]

    def forward(self, h, start, max_new):
        """h [tokens, hidden]; start: int32 (seqs + 1,), the rows of each
        sequence, whose lengths already count them.  Returns the new h."""
        n, D, Hq, Hkv, T = self.n, self.dim, self.q_heads, self.kv_heads, h.shape[0]
        b = self._buffers(T)
        for x in b["h"]:
            x.copy_(h)  # every rank holds the residual stream
        comm = dcc.Comm(n)  # (windows are per communicator; a server registers its arenas once)
        with comm:
            for r in range(n):
                for t in (self.w_out[r], self.w_down[r], b["attn"][r], b["up"][r]):
                    comm.register(r, "input", t)
                comm.register(r, "output", b["h"][r])
            x = norm(h)
            dcc.dcc_linear(self.w_qkv, [x] * n, b["qkv"], bias=self.b_qkv)
            heads = [t.view(T, Hq + 2 * Hkv, D) for t in b["qkv"]]
            self.cache.append([t[:, Hq:Hq + Hkv] for t in heads], [t[:, Hq + Hkv:] for t in heads], start)
            self.attend([t[:, :Hq] for t in heads], [t.view(T, Hq, D) for t in b["attn"]], start, max_new)
            self._row_parallel(comm, self.w_out, b["attn"], b["h"], T)
            x = norm(b["h"][0])
            dcc.dcc_linear(self.w_up, [x] * n, b["up"], bias=self.b_up, act="silu")
            self._row_parallel(comm, self.w_down, b["up"], b["h"], T)
            assert comm.check() == dcc.DCC_OK and dcc.dcc_local_check() == dcc.DCC_OK
        return b["h"][0].clone()

    def attend(self, q, out, start, max_new):
        self.cache.attention(q, out, start, max_new, self.ws_attention)

    def unseen(self, s, length, t):
        """[t, length]: the positions that sequence s's t newest rows do not see."""
        return torch.arange(length, device="cuda")[None, :] > torch.arange(length - t, length, device="cuda")[:, None]

    def _row_parallel(self, comm, weight, x, h, tokens):
        """h <- h + sum over ranks of x W^T, at most 256 tokens at a time."""
        rows, kp = weight[0].shape
        for t0 in range(0, tokens, 256):
            m = min(256, tokens - t0)
            part = [t[t0:t0 + m] for t in h]
            dcc.dcc_linear_allreduce_tokens_residual(comm.handle, weight, [t[t0:t0 + m] for t in x], part, part, m, rows,
                                                     kp, "bf16")

    def grow(self, new):
        """Lengths and pages for `new` more tokens per sequence."""
        info = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.cache.reserve(torch.tensor(new, dtype=torch.int32, device="cuda"), self.ws_pages, info)
        if int(info[1]):
            raise RuntimeError("the cache is full")
        starts = [0]
        for t in new:
            starts.append(starts[-1] + t)
        return torch.tensor(starts, dtype=torch.int32, device="cuda")

    def plain(self, h, start, news):
        """The same block in plain torch operations, with the cache's own keys
        and values (read back): what forward() returns up to rounding."""
        n, D, Hq, Hkv, T = self.n, self.dim, self.q_heads, self.kv_heads, h.shape[0]
        x, out = norm(h).float(), h.float()
        lens = self.cache.lengths.tolist()
        whole = [0]
        for m in lens:
            whole.append(whole[-1] + m)
        k, v = ([torch.empty(whole[-1], Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(n)] for _ in range(2))
        self.cache.read(k, v, torch.tensor(whole, dtype=torch.int32, device="cuda"))
        for r in range(n):
            qkv = (x @ self.w_qkv[r].float().T + self.b_qkv[r].float()).bfloat16().float().view(T, Hq + 2 * Hkv, D)
            attn = torch.zeros(T, Hq, D, device="cuda")
            row = 0
            for s, t in enumerate(news):
                keys, vals = k[r][whole[s]:whole[s + 1]].float(), v[r][whole[s]:whole[s + 1]].float()
                hide = self.unseen(s, lens[s], t)
                for q in range(Hq):
                    g = q // (Hq // Hkv)
                    score = (qkv[row:row + t, q] @ keys[:, g].T * D ** -0.5).masked_fill(hide, float("-inf"))
                    attn[row:row + t, q] = torch.softmax(score, -1) @ vals[:, g]
                row += t
            out += attn.view(T, -1).bfloat16().float() @ self.w_out[r].float().T
        out = out.bfloat16()
        x, y = norm(out).float(), out.float()
        for r in range(n):
            up = x @ self.w_up[r].float().T + self.b_up[r].float()
            y += (up / (1 + torch.exp(-up))).bfloat16().float() @ self.w_down[r].float().T
        return y.bfloat16()


def norm(h):
    f = h.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)).bfloat16()


def run(block=None, prompts=(200, 65, 300), steps=3, verbose=True):
    """Prompts, a beam step, then `steps` tokens; returns the largest difference
    from the plain form relative to its root mean square, per pass."""
    block = block or Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    seen = []

    def one(name, news):
        start = block.grow(news)
        h = torch.randn(sum(news), block.hidden, device="cuda", generator=g).bfloat16()
        got, want = block.forward(h, start, max(news)).float(), block.plain(h, start, news).float()
        seen.append(((got - want).abs().max() / want.square().mean().sqrt()).item())
        if verbose:
            print("%-18s %4d tokens, %s cached: off by %.4f of the rms" % (name, sum(news), block.cache.lengths.tolist(),
                                                                          seen[-1]))
    one("prompts", list(prompts))
    i32 = dict(dtype=torch.int32, device="cuda")
    block.cache.fork(torch.tensor([2], **i32), torch.tensor([1], **i32), block.ws_pages)  # 1 continues 2's text
    for i in range(steps):
        one("token %d" % i, [1] * len(prompts))
    return seen


if __name__ == "__main__":
    run()
