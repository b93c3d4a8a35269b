"""The serving-step operators in a run, as a server uses them (runner.ServingBatch): ragged chunks,
decode steps, a captured decode graph, over a window with sinks, a shared prefix, and all keys.

Each step's outputs are checked stage by stage in 64 bits: the cache rows against the norm and
rotation of every row fed so far (at the slots that a plain count of pages gives), and the attention
against a direct softmax over the cached keys. Bounds are those of the stages' own tests.
"""
import numpy as np
import pytest

from tests.conftest import cuda_available
from tests.test_qk_rope import oracle_rows
from tests.test_window import visible

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(),
                                                  reason="needs a CUDA device")]

HQ, HKV, D, PS, ROT = 8, 2, 128, 16, 64


class Server:
    """A ServingBatch with the rows that were fed to it."""

    def __init__(self, seed, batch, max_len, dtype="f16", prefix=0, **kw):
        import torch
        from paged_kv_long_b200 import binding
        from paged_kv_long_b200.runner import ServingBatch
        self.g = torch.Generator().manual_seed(seed)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        self.rope = binding.rope_table(max_len, ROT)
        self.w = [(1 + 0.3 * torch.randn(D, generator=self.g)).to(self.dt).cuda()
                  for _ in range(2)]
        pages = prefix // PS + batch * (-(-max_len // PS))
        self.s = ServingBatch(HQ, HKV, D, PS, dtype, batch, max_len, self.rope, pages,
                              prefix_len=prefix, q_weight=self.w[0], k_weight=self.w[1], **kw)
        self.prefix = prefix
        self.kept = [[] for _ in range(batch)]  # (k, v) rows of each request, in order
        self.head = []                          # the prefix's

    def rows(self, n):
        import torch
        return [torch.randn(n, h, D, generator=self.g).to(self.dt) for h in (HQ, HKV, HKV)]

    def rotated(self, x, w, pos):
        table = self.rope.double().cpu().numpy()[pos]
        cos, sin = np.split(table, 2, axis=1)
        return oracle_rows(x.double().numpy(), w.double().cpu().numpy(), cos, sin, False, 1e-6)

    def check_rows(self, got, x, w, pos):
        import torch
        want, bound = self.rotated(x, w, pos)
        u = torch.finfo(self.dt).eps / 2
        lim = u * np.abs(want) + 32 * 2.0**-24 * bound * (1 + u) + u * 2.0**-14
        assert (np.abs(got.double().cpu().numpy() - want) <= lim).all()

    def cached(self, b, n):
        """Keys and values of request b's first n positions, read through its table row, checked
        against what was fed."""
        import torch
        table = self.s.block_table[b].cpu().numpy()
        slot = torch.from_numpy(table[np.arange(n) // PS].astype(np.int64) * PS
                                + np.arange(n) % PS).cuda()
        k, v = (p.flatten(0, 1)[slot] for p in (self.s.k_pool, self.s.v_pool))
        fed = self.head + self.kept[b]
        assert torch.equal(v.cpu(), torch.cat([r[1] for r in fed])[:n])
        self.check_rows(k, torch.cat([r[0] for r in fed])[:n], self.w[1], np.arange(n))
        return k.double().cpu().numpy(), v.double().cpu().numpy()

    def check_attention(self, b, pos, q, out, window=0, sinks=0):
        """One row of request b at position pos: rotated queries q, attention out."""
        import torch
        k, v = self.cached(b, pos + 1)
        if window:
            key = visible(pos, window, sinks)
            k, v = k[key], v[key]
        u = torch.finfo(self.dt).eps / 2
        q = q.double().cpu().numpy().reshape(HKV, HQ // HKV, D)
        x = np.einsum("hgd,nhd->hgn", q, k) * D ** -0.5
        a = np.einsum("hgd,nhd->hgn", np.abs(q), np.abs(k)).max() * D ** -0.5
        w = np.exp(x - x.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        want = np.einsum("hgn,nhd->hgd", w, v)
        wide = np.einsum("hgn,nhd->hgd", w, np.abs(v))
        rel = 2 * (2 * D * 2.0**-24 * a + 2.0**-20) + (len(k) + 64) * 2.0**-23
        lim = u * np.abs(want) + (u + rel) * (1 + u) * wide + u * 2.0**-14
        lim += len(k) * 2.0**-25 * np.abs(v).max()
        got = out.double().cpu().numpy().reshape(want.shape)
        assert (np.abs(got - want) <= lim).all(), (b, pos)

    def feed(self, q_lens):
        """Rows of the step's chunks, remembered per request."""
        q, k, v = self.rows(int(np.sum(q_lens)))
        at = 0
        for b, n in enumerate(q_lens):
            self.kept[b].append((k[at:at + n], v[at:at + n]))
            at += n
        return q, k, v


def run(srv, chunks, decodes, replays, **attn):
    """Chunk steps, decode steps and graph replays; every request's last row of each is checked."""
    import torch
    from paged_kv_long_b200 import binding
    binding.device_error(reset=True)
    batch = srv.s.batch
    pos = np.full(batch, srv.prefix)
    for q_lens in chunks:
        q, k, v = srv.feed(q_lens)
        out = srv.s.step(q.cuda(), k.cuda(), v.cuda(), q_lens)
        torch.cuda.synchronize()
        ends = np.cumsum(q_lens)
        for b in range(batch):
            if q_lens[b]:
                at, last = ends[b] - 1, pos[b] + q_lens[b] - 1
                srv.check_rows(srv.s.q_rot[at:at + 1], q[at:at + 1], srv.w[0], [last])
                srv.check_attention(b, last, srv.s.q_rot[at], out[at], **attn)
        pos += q_lens
    static = None
    for i in range(decodes + replays):
        q, k, v = (x.cuda() for x in srv.feed([1] * batch))
        if i < decodes:
            out, q_rot = srv.s.decode(q, k, v), srv.s.q_rot
        else:
            if static is None:
                static = [x.clone() for x in (q, k, v)]
                graph, graph_out = srv.s.capture_decode(*static)
                q_rot = srv.s.q_rot
            for t, x in zip(static, (q, k, v)):
                t.copy_(x)
            graph.replay()
            srv.s.replayed()
            out = graph_out
        torch.cuda.synchronize()
        for b in range(batch):
            srv.check_attention(b, pos[b], q_rot[b], out[b], **attn)
        pos += 1
        assert (srv.s.hist == pos).all() and (srv.s.hist_lens.cpu().numpy() == pos).all()
    assert binding.device_error(reset=True)[0] == 0
    if static is not None:
        del graph


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gpu_windowed_serving(dtype):
    srv = Server(1, 3, 400, dtype, window=50, n_sinks=4)
    run(srv, [[100, 0, 33], [7, 200, 0], [1, 1, 1]], 2, 3, window=50, sinks=4)


def test_gpu_serving_over_a_shared_prefix():
    import torch
    srv = Server(2, 4, 300, prefix=96)
    q, k, v = srv.rows(96)
    srv.head = [(k, v)]
    out = srv.s.write_prefix(q.cuda(), k.cuda(), v.cuda())
    torch.cuda.synchronize()
    assert out.shape == (96, HQ, D) and torch.isfinite(out).all()
    run(srv, [[5, 0, 40, 17]], 2, 3)
    used = int(srv.s.pages_used)  # the prefix's six pages once, then each request's own
    assert used == 6 + sum(-(-int(n) // PS) - 6 for n in srv.s.hist)


def test_gpu_serving_over_all_keys():
    run(Server(3, 2, 300), [[20, 31]], 2, 2)


def test_gpu_two_servers_share_the_device():
    """Steps of two servers in turn on two streams: nothing is shared between them."""
    import torch
    a, b = Server(4, 2, 200, window=30, n_sinks=2), Server(5, 2, 200, window=64)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for srv, s in ((a, streams[0]), (b, streams[1])):
        fed = srv.feed([40, 50])
        with torch.cuda.stream(s):
            outs.append(srv.s.step(*(x.cuda() for x in fed), [40, 50]))
    for _ in range(3):
        for i, (srv, s) in enumerate(((a, streams[0]), (b, streams[1]))):
            fed = srv.feed([1, 1])
            with torch.cuda.stream(s):
                outs[i] = srv.s.decode(*(x.cuda() for x in fed))
    torch.cuda.synchronize()
    for r in range(2):
        a.check_attention(r, (40, 50)[r] + 2, a.s.q_rot[r], outs[0][r], window=30, sinks=2)
        b.check_attention(r, (40, 50)[r] + 2, b.s.q_rot[r], outs[1][r], window=64)


@pytest.mark.parametrize("window", [0, 40])
def test_gpu_step_of_more_requests_than_a_launch_holds(window):
    attn = dict(window=window, sinks=2) if window else {}
    kw = dict(window=window, n_sinks=2) if window else {}
    run(Server(6, 300, 64, **kw), [[1] * 300, [0, 3] * 150], 1, 0, **attn)


@pytest.mark.parametrize("window", [0, 1000])
def test_gpu_chunk_of_more_rows_than_a_launch_holds(window):
    """16,600 rows of one request: more than 512 row blocks. Rows on both sides of each cut, and a
    step without any row."""
    import torch
    from paged_kv_long_b200 import binding
    attn = dict(window=window, sinks=2) if window else {}
    srv = Server(7, 2, 16700, "bf16", **(dict(window=window, n_sinks=2) if window else {}))
    binding.device_error(reset=True)
    q, k, v = srv.feed([20, 9])
    srv.s.step(q.cuda(), k.cuda(), v.cuda(), [20, 9])
    lens = [16600, 77]
    edges = [r[1] for r in srv.s._runs(np.array(lens, np.int32))]
    assert len(edges) > 1
    q, k, v = srv.feed(lens)
    out = srv.s.step(q.cuda(), k.cuda(), v.cuda(), lens)
    none = [x[:0].cuda() for x in (q, k, v)]
    q_rot = srv.s.q_rot
    assert srv.s.step(*none, [0, 0]).shape == (0, HQ, D)
    torch.cuda.synchronize()
    assert binding.device_error(reset=True)[0] == 0
    for row in {0, 16599, 16600, 16676}.union(*({e - 1, e} for e in edges[:-1])):
        b, pos = (0, 20 + row) if row < 16600 else (1, 9 + row - 16600)
        srv.check_attention(b, pos, q_rot[row], out[row], **attn)


def test_gpu_refused_steps_then_accepted_ones():
    """Steps without room change nothing: what follows is as if they had not been asked for."""
    import torch
    srv = Server(8, 3, 96, window=50, n_sinks=4)
    state = lambda: [t.clone() for t in (srv.s.k_pool, srv.s.v_pool,  # noqa: E731
                                         srv.s.block_table, srv.s.pages_used, srv.s.hist_lens)]
    before = state()
    q, k, v = (x.cuda() for x in srv.rows(3 + 97))
    with pytest.raises(ValueError, match="request 1 would hold 97"):
        srv.s.step(q, k, v, [3, 97, 0])
    assert all(torch.equal(a, b) for a, b in zip(state(), before))
    run(srv, [[3, 90, 0], [5, 4, 96]], 0, 0, window=50, sinks=4)
    with pytest.raises(ValueError, match="request 2"):
        srv.s.decode(q[:3], k[:3], v[:3])
    run_on = [[2, 2, 0]]  # up to the last rows of request 1
    pos = srv.s.hist.copy()
    q, k, v = srv.feed(run_on[0])
    out = srv.s.step(q.cuda(), k.cuda(), v.cuda(), run_on[0])
    torch.cuda.synchronize()
    for b, row in ((0, 1), (1, 3)):
        srv.check_attention(b, pos[b] + 1, srv.s.q_rot[row], out[row], window=50, sinks=4)


def test_gpu_constructor_leaves_nothing_pending():
    """Steps on a fresh stream right after the constructor need no wait: its fills are done, and so
    is the work that its tensors may come from."""
    import torch
    torch.cuda._sleep(20_000_000)  # about 10 ms of the constructor's stream
    srv = Server(9, 2, 200, window=64)
    assert torch.cuda.current_stream().query()
    s = torch.cuda.Stream()
    fed = srv.feed([40, 50])
    with torch.cuda.stream(s):
        out = srv.s.step(*(x.cuda() for x in fed), [40, 50])
    s.synchronize()
    for b, row in ((0, 39), (1, 89)):
        srv.check_attention(b, (39, 49)[b], srv.s.q_rot[row], out[row], window=64)


def test_gpu_device_is_the_one_of_the_constructor():
    """Given without a number: the device that is current then, whatever is current at a step."""
    import torch
    srv = Server(10, 2, 64)
    assert srv.s.device == srv.s.k_pool.device == torch.device("cuda", torch.cuda.current_device())
