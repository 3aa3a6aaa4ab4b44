"""The decoder's calls launched after one another with no host wait between
them: each kernel may start while the one before it ends, so results must be
those of the same calls with a wait after each."""
import pytest
import torch

import kv4_reference as R
from test_gpu_kv4 import batch, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64)])
@pytest.mark.parametrize("tokens", [16, 64, 300])
def test_prompt_attention_and_linear_layers_in_turn(dcc, dtype, dim, group, tokens):
    """Kernels that share the tensor memory of an SM, small ones beside large
    ones: attention of a prompt, a layer of few tokens, one of many."""
    g = torch.Generator().manual_seed(7)
    n, lens, news = 8, [700, 300], [130, 100]
    cache, _, _ = make_cache(dcc, g, n, lens, 1, dim, group, dtype)
    t = R.TD[dtype]
    q = [torch.randn(230, 4, dim, generator=g).to(t).cuda() for _ in range(n)]
    attn = [torch.empty_like(x) for x in q]
    w = [(torch.randn(256, 4 * dim, generator=g) * 0.05).to(t).cuda() for _ in range(n)]
    ws = cache.attention_workspace(4)
    few = [x.view(230, -1)[:tokens] if tokens <= 230 else torch.randn(tokens, 4 * dim, generator=g).to(t).cuda() for x in attn]
    y = [torch.empty(tokens, 256, dtype=t, device="cuda") for _ in range(n)]
    z = [torch.empty(230, 256, dtype=t, device="cuda") for _ in range(n)]
    rows = [x.view(230, -1) for x in attn]
    start = batch(news)

    def step(wait):
        cache.attention(q, attn, start, max_new=130, workspace=ws)
        wait()
        dcc.dcc_linear(w, few, y, act="gelu")
        wait()
        dcc.dcc_linear(w, rows, z, act="silu")
        wait()

    step(torch.cuda.synchronize)
    want = [x.clone() for x in attn + y + z]
    for x in attn + y + z:
        x.zero_()
    for _ in range(50):
        step(lambda: None)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    assert all(torch.equal(a, b) for a, b in zip(attn + y + z, want))


class Decoder:
    """A small decoder step on n ranks that only enqueues: what every token runs."""

    def __init__(self, dcc, comm, dtype, n=4, seqs=3, share=4, dim=64, hidden=256):
        g = torch.Generator().manual_seed(11)
        t = R.TD[dtype]
        self.dcc, self.comm, self.n, self.share, self.dim, self.hidden, self.dtype = dcc, comm, n, share, dim, hidden, dtype
        self.cache = dcc.Kv4Cache.create(n, 2, 40, seqs, 12, 1, dim, 32, dtype)

        def weights(rows, k):
            return [(torch.randn(rows, k, generator=g) * 0.3 * k ** -0.5).to(t).cuda() for _ in range(n)]
        width = (share + 2) * dim
        self.w_qkv, self.w_out, self.w_up, self.w_down = weights(width, hidden), weights(hidden, share * dim), \
            weights(128, hidden), weights(hidden, 128)

        def buffers(tokens, rows):
            return [torch.zeros(tokens, rows, dtype=t, device="cuda") for _ in range(n)]
        self.h, self.qkv, self.attn, self.up = buffers(seqs, hidden), buffers(seqs, width), buffers(seqs, share * dim), \
            buffers(seqs, 128)
        self.total = buffers(seqs, hidden)
        self.ws, self.wp = self.cache.attention_workspace(share), self.cache.pages_workspace()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.add, self.start = torch.ones(seqs, **i32), torch.arange(seqs + 1, **i32)
        self.info = torch.zeros(4, **i32)
        self.src, self.dst = torch.tensor([0], **i32), torch.tensor([2], **i32)
        self.gone, self.remap = torch.tensor([1], **i32), torch.zeros(40, **i32)
        for r in range(n):
            for x in (self.w_out[r], self.w_down[r], self.attn[r], self.up[r], self.h[r]):
                comm.register(r, "input", x)
            comm.register(r, "output", self.h[r])
            comm.register(r, "output", self.total[r])

    def step(self, stream=None, pages=False):
        d, T, s = self.dcc, len(self.h[0]), stream
        self.cache.reserve(self.add, self.wp, self.info, stream=s)
        for layer in range(2):
            d.dcc_linear(self.w_qkv, self.h, self.qkv, stream=s)
            heads = [x.view(T, self.share + 2, self.dim) for x in self.qkv]
            self.cache.append([x[:, self.share:-1] for x in heads], [x[:, self.share + 1:] for x in heads], self.start,
                              layer=layer, stream=s)
            self.cache.attention([x[:, :self.share] for x in heads], [x.view(T, self.share, self.dim) for x in self.attn],
                                 self.start, 1, self.ws, layer=layer, stream=s)
            d.dcc_linear_allreduce_tokens_residual(self.comm.handle, self.w_out, self.attn, self.h, self.h, T, self.hidden,
                                                   self.share * self.dim, self.dtype, stream=s)
            d.dcc_linear(self.w_up, self.h, self.up, act="silu", stream=s)
            d.dcc_linear_allreduce_tokens_residual(self.comm.handle, self.w_down, self.up, self.h, self.h, T, self.hidden,
                                                   128, self.dtype, stream=s)
        d.dcc_allreduce(self.comm.handle, self.h, self.total, T * self.hidden, self.dtype, stream=s)
        if pages:
            self.cache.fork(self.src, self.dst, self.wp, self.info, stream=s)
            self.cache.free(self.gone, self.wp, self.info, stream=s)
            self.cache.compact(self.cache.table, self.cache.refs, self.remap, self.wp, self.info, stream=s)

    def state(self):
        c = self.cache
        return [x.clone() for x in (*self.h, *self.total, *self.attn, c.table, c.lengths, c.refs, self.info, self.remap)]

    def reset(self, tokens):
        g = torch.Generator().manual_seed(12)
        for p in self.cache.pools:
            p.zero_()
        self.cache.table.fill_(-1)
        self.cache.lengths.zero_()
        self.cache.refs.zero_()
        self.remap.zero_()
        for r in range(self.n):
            self.h[r].copy_(torch.randn(self.h[r].shape, generator=g))
        self.add.fill_(tokens)  # (rows of the cache that no step writes stay zero)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("pdl", [True, False])
@pytest.mark.parametrize("pages", [False, True])
def test_decode_steps_launched_ahead_and_captured(dcc, dtype, pdl, pages):
    """Decode steps with a wait after each, all launched at once, and replayed
    from a CUDA graph: the same states."""
    steps = 8
    with dcc.Comm(4) as comm:
        dcc.dcc_set_pdl(comm.handle, pdl)
        d = Decoder(dcc, comm, dtype)
        stream = torch.cuda.Stream()

        def go(wait, step):
            d.reset(30)
            torch.cuda.synchronize()
            states = []
            for _ in range(steps):
                step()
                if wait:
                    torch.cuda.synchronize()
                    states.append(d.state())
            torch.cuda.synchronize()
            assert comm.check() == dcc.DCC_OK and dcc.dcc_local_check() == dcc.DCC_OK
            return states or [d.state()]

        def same(a, b):
            return all(torch.equal(x, y) for x, y in zip(a, b))
        want = go(True, lambda: d.step(pages=pages))
        assert all(torch.isfinite(x.float()).all() for x in want[-1][:8]) and want[-1][0].any()
        assert not torch.equal(want[0][0], want[-1][0])
        assert same(go(False, lambda: d.step(pages=pages))[-1], want[-1])
        assert same(go(False, lambda: d.step(stream, pages))[-1], want[-1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            d.step(pages=pages)
        for got, exp in zip(go(True, graph.replay), want):
            assert same(got, exp)
        assert same(go(False, graph.replay)[-1], want[-1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prompt_and_layers_captured(dcc, dtype):
    """The prompt kernel and both layer kernels in a graph, replayed on other inputs."""
    g = torch.Generator().manual_seed(13)
    n, lens, news, t = 8, [700, 300], [130, 100], R.TD[dtype]
    cache, _, _ = make_cache(dcc, g, n, lens, 1, 128, 64, dtype)
    q = [torch.zeros(230, 8, 128, dtype=t, device="cuda") for _ in range(n)]
    k, v = ([torch.zeros(230, 1, 128, dtype=t, device="cuda") for _ in range(n)] for _ in range(2))
    out = [torch.empty_like(x) for x in q]
    back = [[torch.empty_like(x) for x in k] for _ in range(2)]
    w = [(torch.randn(264, 1024, generator=g) * 0.05).to(t).cuda() for _ in range(n)]
    y = [torch.empty(230, 264, dtype=t, device="cuda") for _ in range(n)]
    z = [torch.empty(460, 264, dtype=t, device="cuda") for _ in range(n)]
    many = [torch.zeros(460, 1024, dtype=t, device="cuda") for _ in range(n)]
    ws, start = cache.attention_workspace(8), batch(news)

    def run():
        cache.append(k, v, start)
        cache.read(back[0], back[1], start)
        cache.attention(q, out, start, max_new=130, workspace=ws)
        dcc.dcc_linear(w, [x.view(230, -1) for x in out], y, act="gelu")
        dcc.dcc_linear(w, many, z, act="relu")

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for turn in range(3):
        for x in (*q, *k, *v, *many):
            x.copy_(torch.randn(x.shape, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*out, *back[0], *back[1], *y, *z)]
        run()
        assert dcc.dcc_local_check() == dcc.DCC_OK
        assert got[0].any() and all(torch.equal(a, b) for a, b in zip(got, (*out, *back[0], *back[1], *y, *z)))
