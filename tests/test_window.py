"""Sliding-window attention with sinks on paged pools (pa_window_*): the row at position p sees
key j <= p with j > p - window or j < n_sinks.

The oracle is a direct softmax in 64 bits over each row's own key list. In every case the pool
slots that no row sees hold NaN and the table entries of pages that no row sees are -1 (given back).

Tolerance, element by element, with u = eps(type) / 2 and W = sum_j w_j |v_j| (w the softmax
weights): the output is rounded once (u |out|), each probability once before the product (u W;
fp16 probabilities below its normal range by at most 2^-25 each, against a sum of at least 1:
n 2^-25 max|v|). The fp32 parts: a score is off by at most 2 D 2^-24 sum|q k| scale (products of
16-bit values are exact, D additions, truncated or rounded), which moves each weight by that
relative amount, in the numerator and the sum, as the exponential's own 2^-20 does; the sums over
n keys and up to 32 partials add (n + 64) 2^-23 W.
"""
import ctypes
import math

import numpy as np
import pytest

from tests.conftest import cuda_available

gpu = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def _gpu(f):
    for m in gpu:
        f = m(f)
    return f


def _binding():
    from paged_kv_long_b200 import binding
    return binding


def visible(p, window, sinks):
    """The keys that the row at position p sees."""
    lo = max(0, p + 1 - window)
    return np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, p + 1)])


class Case:
    """A batch of chunks (rows[b] query rows after hist[b] keys), on the host as torch tensors."""

    def __init__(self, seed, rows, hist, window, sinks, Hq, Hkv, D, PS, dtype, ramp=False):
        import torch
        self.rows, self.hist = [int(r) for r in rows], [int(h) for h in hist]
        self.window, self.sinks, self.dtype = window, sinks, dtype
        self.Hq, self.Hkv, self.D, self.PS = Hq, Hkv, D, PS
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        g = torch.Generator().manual_seed(seed)
        B = len(self.rows)
        total = [h + r if r else 0 for r, h in zip(self.rows, self.hist)]
        stride = max(1, max(math.ceil(t / PS) for t in total))
        self.table = np.full((B, stride), -1, np.int32)
        seen = []
        for r, h, t in zip(self.rows, self.hist, total):
            s = np.zeros(stride * PS, bool)
            if r:
                s[:min(sinks, t)] = True
                s[max(0, h + 1 - window):t] = True
            seen.append(s)
        held = np.array([s.reshape(stride, PS).any(1) for s in seen])
        num_pages = int(held.sum()) + 2
        ids = torch.randperm(num_pages, generator=g).numpy().astype(np.int32)
        self.table[held] = ids[:num_pages - 2]
        self.k = torch.full((num_pages, PS, Hkv, D), float("nan"), dtype=self.dt)
        self.v = self.k.clone()
        for b, s in enumerate(seen):
            key = np.flatnonzero(s)
            if len(key):
                slot = torch.from_numpy(self.table[b, key // PS].astype(np.int64) * PS + key % PS)
                for pool in (self.k, self.v):
                    x = torch.randn(len(key), Hkv, D, generator=g)
                    if ramp and pool is self.k:  # scores grow along the keys
                        x[..., 0] += torch.from_numpy(key * (64.0 / max(total))).float()[:, None]
                    pool.flatten(0, 1)[slot] = x.to(self.dt)
        n = sum(self.rows)
        self.q = torch.randn(n, Hq, D, generator=g)
        if ramp:
            self.q[..., 0] = 4.0
        self.q = self.q.to(self.dt)

    def oracle(self, pick=None):
        """(row indices, fp64 outputs, bounds) of the picked packed rows (all by default)."""
        import torch
        G, D, scale = self.Hq // self.Hkv, self.D, self.D ** -0.5
        kf, vf = self.k.flatten(0, 1), self.v.flatten(0, 1)
        u, at, idx, outs, lims = torch.finfo(self.dt).eps / 2, 0, [], [], []
        for b, (r, h) in enumerate(zip(self.rows, self.hist)):
            for i in range(r):
                if pick is None or at + i in pick:
                    key = visible(h + i, self.window, self.sinks)
                    slot = self.table[b, key // self.PS].astype(np.int64) * self.PS + key % self.PS
                    assert (slot >= 0).all()
                    k = kf[torch.from_numpy(slot)].double().numpy()
                    v = vf[torch.from_numpy(slot)].double().numpy()
                    q = self.q[at + i].double().numpy().reshape(self.Hkv, G, D)
                    x = np.einsum("hgd,nhd->hgn", q, k) * scale
                    a = np.einsum("hgd,nhd->hgn", np.abs(q), np.abs(k)).max() * scale
                    w = np.exp(x - x.max(-1, keepdims=True))
                    w /= w.sum(-1, keepdims=True)
                    out = np.einsum("hgn,nhd->hgd", w, v)
                    wide = np.einsum("hgn,nhd->hgd", w, np.abs(v))
                    n = len(key)
                    rel = 2 * (2 * D * 2.0**-24 * a + 2.0**-20) + (n + 64) * 2.0**-23
                    lim = u * np.abs(out) + (u + rel) * (1 + u) * wide + u * 2.0**-14
                    if self.dtype == "f16":
                        lim += n * 2.0**-25 * np.abs(v).max()
                    idx.append(at + i)
                    outs.append(out.reshape(self.Hq, D))
                    lims.append(lim.reshape(self.Hq, D))
            at += r
        return np.array(idx), np.array(outs), np.array(lims)

    def check(self, got, pick=None, what=""):
        idx, want, lim = self.oracle(pick)
        got = got.double().cpu().numpy()[idx]
        assert np.isfinite(got).all(), f"{what}: non-finite output"
        err = np.abs(got - want)
        assert (err <= lim).all(), f"{what}: {(err / lim).max():.3f} of the bound"

    def device(self):
        import torch
        return (self.q.cuda(), self.k.cuda(), self.v.cuda(),
                torch.from_numpy(self.table).cuda())


def run_prefill(c, num_sms=None):
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    wp = bd.window_plan(c.Hq, c.Hkv, c.D, c.PS, c.rows, c.hist, c.window, c.sinks, c.dtype,
                        num_sms=num_sms)
    q, k, v, t = c.device()
    out, ws = torch.full_like(q, float("nan")), bd.workspace(wp.plan)
    if ws is not None:
        ws.fill_(float("nan"))
    got = bd.window_prefill(wp, q, k, v, t, out, ws)
    torch.cuda.synchronize()
    assert bd.device_error(reset=True)[0] == 0
    return wp, got


def run_decode(c, num_sms=148):
    """Rows with no key are in the batch as length 0 (c.rows[b] == 0)."""
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    B = len(c.rows)
    lens = np.array([h + r if r else 0 for r, h in zip(c.rows, c.hist)], np.int32)
    wp = bd.window_decode_plan(c.Hq, c.Hkv, c.D, c.PS, B, max(1, int(lens.max())), c.window,
                               c.sinks, c.dtype, num_sms=num_sms)
    _, k, v, t = c.device()
    full = torch.zeros(B, c.Hq, c.D, dtype=c.dt)
    live = torch.from_numpy(lens > 0)
    full[live] = c.q
    out, ws = torch.full_like(full, float("nan")).cuda(), bd.workspace(wp.plan)
    if ws is not None:
        ws.fill_(float("nan"))
    got = bd.window_decode(wp, full.cuda(), k, v, t, torch.from_numpy(lens).cuda(), out, ws)
    torch.cuda.synchronize()
    assert bd.device_error(reset=True)[0] == 0
    got = got.cpu()
    assert (got[~live] == 0).all()
    return wp, got[live]


# ------------------------------------------------------------------------------------ CPU


def test_oracle_full_window_is_causal_attention():
    from oracle import oracle
    c = Case(1, [5], [19], 1000, 0, 4, 2, 64, 16, "f16")
    p = oracle.Problem(q=c.q.view(dtype=__import__("torch").int16).numpy().view(np.uint16),
                       k=c.k.view(dtype=__import__("torch").int16).numpy().view(np.uint16),
                       v=c.v.view(dtype=__import__("torch").int16).numpy().view(np.uint16),
                       hist_len=19, dtype="f16", page_table=c.table[0])
    ref, _ = oracle.attend(p)
    np.testing.assert_allclose(c.oracle()[1], ref.reshape(5, 4, 64), atol=1e-12)


def test_oracle_window_one_returns_the_rows_own_value():
    c = Case(2, [3, 1], [0, 40], 1, 0, 2, 1, 64, 16, "bf16")
    _, out, _ = c.oracle()
    for row, (b, p) in enumerate([(0, 0), (0, 1), (0, 2), (1, 40)]):
        v = c.v[int(c.table[b, p // 16]), p % 16, 0].double().numpy()
        np.testing.assert_array_equal(out[row], np.stack([v, v]))


def tiles_of(items, wp, window, sinks, rows, hist, G, Hkv, per):
    """{global row block: its list of KV tiles} expected from the definition."""
    want, rb = {}, 0
    for r, h in zip(rows, hist):
        units = math.ceil(math.ceil(r * G / 128) / per)
        for local in range(units * Hkv):
            u = units - 1 - local // Hkv
            first = u * per * 128 // G
            last = min(r - 1, ((u + 1) * per * 128 - 1) // G)
            keys = np.unique(np.concatenate([visible(h + t, window, sinks)
                                             for t in range(first, last + 1)]))
            want[rb + local] = len(np.unique(keys // 128))
        rb += units * Hkv
    return want


@pytest.mark.parametrize("seed", range(40))
def test_plan_items_cover_the_visible_tiles_once(seed):
    """Every row block's items cover exactly its visible KV tiles, in whole runs; a row block with
    several items has a workspace slot for each."""
    bd = _binding()
    rng = np.random.default_rng(seed)
    Hkv = int(rng.choice([1, 2, 4]))
    G = int(rng.choice([1, 3, 6, 8, 16]))
    D = int(rng.choice([64, 128, 256]))
    B = int(rng.choice([1, 1, 2, 7]))
    rows = rng.integers(0 if B > 1 else 1, 260, B)
    rows[0] = max(1, rows[0])
    hist = rng.integers(0, 3000, B)
    window, sinks = int(rng.choice([1, 2, 127, 128, 129, 500, 10**6])), int(
        rng.choice([0, 1, 127, 128, 129, 400]))
    if rng.random() < 0.2:
        rows[:] = np.minimum(rows, 1)
        rows[0] = 1
    try:
        wp = bd.window_plan(Hkv * G, Hkv, D, 16, rows, hist, window, sinks, "f16", num_sms=148)
    except bd.PaError as e:
        assert e.status == -2  # more than 512 row blocks
        return
    p = wp.plan
    items = bd.window_schedule_items(wp)
    assert len(items) == p.units
    want = tiles_of(items, wp, window, sinks, rows, hist, G, Hkv, p.ctas_per_unit)
    runs = {}
    for rb, k0, k1, slot in items.tolist():
        assert k0 < k1
        runs.setdefault(rb, []).append((k0, k1, slot))
    assert set(runs) == set(want)
    slots = []
    for rb, parts in runs.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == want[rb]
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
        if len(parts) == 1:
            assert parts[0][2] == -1
        else:
            slots += [x[2] for x in parts]
    assert sorted(slots) == list(range(len(slots)))
    assert p.ws_bytes == len(slots) * p.ctas_per_unit * 128 * (D + 1) * 4


def test_decode_plan_shares_the_visible_tiles():
    bd = _binding()
    mk = lambda **a: bd.window_decode_plan(**{**dict(  # noqa: E731
        n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=16, batch=1, max_seq_len=32768,
        window=1000, n_sinks=4, dtype="f16", num_sms=148), **a}).plan
    # G 8 at D 256: CTAs that share the tiles (1 sink tile + 8 + 1, two heads) and the units'
    # starts, two each at least
    p = mk()
    assert p.units == 11 and p.splits == 1 and p.hist_len == 32768 and p.policy == 5
    assert p.ws_bytes == 11 * 2 * 8 * 257 * 4
    assert mk(n_sinks=0, window=1).units == 2 and mk(n_sinks=0, window=129).units == 3
    assert mk(max_seq_len=100).units == 2 and mk(batch=64).units == 296
    assert mk(batch=64, num_sms=5).units == 10
    assert mk(window=2**40).units == 257     # a window past 2^31 sees every key anyway
    # G 16: uniform splits of the single-CTA kernel
    p = mk(n_q_heads=32)
    assert p.splits == 10 and p.units == 20 and p.ws_bytes == 10 * 32 * 257 * 4
    assert mk(n_q_heads=32, batch=200).splits == 1 and mk(n_q_heads=32, batch=200).ws_bytes == 0
    p = mk(head_dim=64, batch=3, window=10**6)
    assert p.splits == 32 and p.units == 3 * 2 * 32


def test_refusals():
    """Checked before any device work: these run without a GPU."""
    bd = _binding()
    lib = bd.load_library()
    name = lambda st: bd.STATUS[st]  # noqa: E731
    for bad in (dict(window=0), dict(n_sinks=-1), dict(window=-5)):
        with pytest.raises(ValueError):
            bd.window_plan(**{**dict(n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16,
                                     q_lens=[1], hist_lens=[3], window=4, num_sms=148), **bad})
        with pytest.raises(ValueError):
            bd.window_decode_plan(**{**dict(n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16,
                                            batch=1, max_seq_len=9, window=4, num_sms=148), **bad})
    p = bd.Plan()
    ql, hl = np.array([1], np.int32), np.array([3], np.int64)
    raw = lambda w, s: name(lib.pa_window_plan(  # noqa: E731
        148, 4, 2, 64, 16, 1, ql.ctypes.data, hl.ctypes.data, w, s, 0, 0.0, ctypes.byref(p)))
    assert raw(0, 0) == raw(1, -1) == "PA_ERR_INVALID_ARG" and raw(1, 0) == "PA_OK"
    raw = lambda w, s: name(lib.pa_window_decode_plan(  # noqa: E731
        148, 4, 2, 64, 16, 1, 9, w, s, 0, 0.0, ctypes.byref(p)))
    assert raw(0, 0) == raw(1, -1) == "PA_ERR_INVALID_ARG" and raw(1, 0) == "PA_OK"
    for bad in (dict(head_dim=96), dict(page_size=24), dict(n_q_heads=5), dict(batch=0),
                dict(max_seq_len=0), dict(max_seq_len=2**31)):
        with pytest.raises(bd.PaError):
            bd.window_decode_plan(**{**dict(n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16,
                                            batch=1, max_seq_len=9, window=4, num_sms=148), **bad})

    wd = bd.window_decode_plan(16, 2, 256, 16, 4, 1000, 200, 4, "f16", num_sms=148)
    wp = bd.window_plan(16, 2, 256, 16, [1, 2], [50, 60], 200, 4, "f16", num_sms=148)
    dp = bd.decode_plan(16, 2, 256, 16, 4, 1000, "f16", num_sms=148)
    bp = bd.batch_plan(16, 2, 256, 16, [1, 2], [50, 60], "f16", num_sms=148)
    f = ctypes.c_void_p(1 << 20)
    big = 1 << 40
    ref = ctypes.byref

    def decode(plan, w=200, s=4, q=f, table=f, stride=64, lens=f, pages=100, out=f, ws=f, n=big):
        return name(lib.pa_window_decode(ref(plan), w, s, q, f, f, table, stride, lens, pages, out,
                                         ws, n, None))

    def prefill(b, w=200, s=4, q=f, stride=64, pages=100, out=f):
        ql, hl = b.q_lens.ctypes.data, b.hist_lens.ctypes.data
        return name(lib.pa_window_prefill(ref(b.plan), ql, hl, w, s, q, f, f, f, stride, pages,
                                          out, f, big, None))

    bad = "PA_ERR_INVALID_ARG"
    # each entry point takes its own plans only
    assert decode(dp) == decode(wp.plan) == decode(bp.plan) == bad
    assert prefill(bp) == bad
    assert name(lib.pa_decode(ref(wd.plan), f, f, f, f, 64, f, 100, f, f, big, None)) == bad
    assert name(lib.pa_combine(ref(wd.plan), f, big, f, None)) == bad
    assert name(lib.pa_combine(ref(wp.plan), f, big, f, None)) == bad
    ql, hl = wp.q_lens.ctypes.data, wp.hist_lens.ctypes.data
    assert name(lib.pa_batch_prefill(ref(wp.plan), ql, hl, f, f, f, f, 64, 100, f, f, big,
                                     None)) == bad
    assert name(lib.pa_batch_combine(ref(wp.plan), ql, hl, f, big, f, None)) == bad
    assert name(lib.pa_prefill(ref(wp.plan), f, f, f, f, 100, wp.plan.hist_len, 3, f, f, big,
                               None)) == bad
    # arguments
    assert decode(wd.plan, w=0) == decode(wd.plan, s=-1) == decode(wd.plan, q=None) == bad
    assert decode(wd.plan, w=900) == bad      # another window: its tiles, CTAs and workspace
    assert decode(wd.plan, lens=None) == decode(wd.plan, out=None) == decode(wd.plan, table=None)
    assert decode(wd.plan, stride=0) == decode(wd.plan, pages=0) == bad
    assert decode(wd.plan, ws=None) == decode(wd.plan, n=16) == "PA_ERR_WORKSPACE"
    assert decode(wd.plan, pages=1 << 27) == "PA_ERR_UNSUPPORTED"
    assert prefill(wp, w=0) == prefill(wp, q=None) == prefill(wp, out=None) == bad
    assert prefill(wp, stride=3) == bad       # 62 keys need four pages
    wp.q_lens[1] = 300                        # not the lengths that the plan was made from
    assert prefill(wp) == bad


def test_an_output_over_the_queries_is_refused():
    """Whole or in part, by the window and the prefix calls; an output right behind the queries
    gets past that check (to the tensor maps, which need a GPU's driver here)."""
    bd = _binding()
    lib, ref = bd.load_library(), ctypes.byref
    q, f, big = 1 << 30, ctypes.c_void_p(1 << 20), 1 << 40
    wd = bd.window_decode_plan(16, 2, 256, 16, 4, 1000, 200, 4, "f16", num_sms=148)
    wp = bd.window_plan(16, 2, 256, 16, [1, 3], [50, 60], 200, 4, "f16", num_sms=148)
    pp = bd.prefix_decode_plan(16, 2, 256, 16, 4, 320, 1000, "f16", num_sms=148)
    n = 4 * 16 * 256 * 2  # bytes of q, and of the output
    runs = (lambda out: lib.pa_window_decode(ref(wd.plan), 200, 4, q, f, f, f, 64, f, 100, out, f,
                                             big, None),
            lambda out: lib.pa_window_prefill(ref(wp.plan), *wp.lens_ptrs, 200, 4, q, f, f, f, 64,
                                              100, out, f, big, None),
            lambda out: lib.pa_prefix_decode(ref(pp.plan), 320, q, f, f, f, f, 64, f, 100, out, f,
                                             big, None))
    for run in runs:
        for out in (q, q + 16, q - 16, q + n - 16, q - n + 16):
            assert bd.STATUS[run(out)] == "PA_ERR_INVALID_ARG"
        if not cuda_available():
            assert bd.STATUS[run(q + n)] == bd.STATUS[run(q - n)] == "PA_ERR_CUDA"


def test_plan_keeps_its_own_lengths():
    bd = _binding()
    rows, hist = np.array([3, 5], np.int32), np.array([9, 0], np.int64)
    wp = bd.window_plan(4, 2, 64, 16, rows, hist, 4, num_sms=148)
    rows += 100
    hist += 100
    assert wp.q_lens.tolist() == [3, 5] and wp.hist_lens.tolist() == [9, 0]


def test_binding_refuses_the_other_plan():
    bd = _binding()
    wd = bd.window_decode_plan(16, 2, 256, 16, 4, 1000, 200, 4, "f16", num_sms=148)
    wp = bd.window_plan(16, 2, 256, 16, [1], [50], 200, 4, "f16", num_sms=148)
    with pytest.raises(ValueError):
        bd.window_decode(wp, None, None, None, None, None)
    with pytest.raises(ValueError):
        bd.window_prefill(wd, None, None, None, None)
    with pytest.raises(ValueError):
        bd.window_schedule_items(wd)


# ------------------------------------------------------------------------------------ GPU

DECODE = [
    # lens, window, sinks, Hq, Hkv, D, PS, dtype, num_sms
    ([1], 1, 0, 8, 1, 256, 16, "f16", 148),
    ([1, 2, 16, 17], 1, 1, 16, 2, 128, 16, "bf16", 148),
    ([700, 0, 129, 128, 127], 128, 0, 16, 2, 256, 16, "f16", 1),
    ([700, 0, 129, 256, 385, 1], 129, 4, 16, 2, 256, 64, "bf16", 148),
    ([2000, 1999, 1, 300], 500, 130, 24, 4, 256, 128, "bf16", 3),   # sinks over two tiles
    ([5000, 40, 1024, 1025], 1000, 4, 32, 8, 128, 32, "f16", 148),
    ([900, 901, 902], 10**6, 0, 8, 8, 128, 16, "f16", 148),           # the whole sequence
    ([900, 901, 902], 300, 10**6, 8, 8, 128, 16, "f16", 148),
    ([3000, 5, 129], 257, 20, 32, 2, 64, 16, "bf16", 148),            # G 16: single-CTA kernel
    ([3000, 0, 5], 64, 300, 4, 4, 64, 128, "f16", 2),
    ([4000, 3], 130, 1, 32, 2, 256, 16, "f16", 148),                  # G 16 at D 256
    ([9000, 8999], 8000, 4, 8, 1, 256, 16, "f16", 100),
    ([1500], 1000, 300, 8, 1, 128, 64, "bf16", 2),                  # four CTAs
    ([1500, 77], 1100, 300, 8, 1, 64, 64, "bf16", 1),               # one unit over both runs
]


@_gpu
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_gpu_window_decode(i):
    lens, w, s, Hq, Hkv, D, PS, dtype, sms = DECODE[i]
    c = Case(100 + i, [min(1, n) for n in lens], [max(0, n - 1) for n in lens], w, s, Hq, Hkv, D,
             PS, dtype)
    wp, got = run_decode(c, sms)
    c.check(got, what=f"{wp.plan.units} units")


@_gpu
@pytest.mark.parametrize("D,Hq,Hkv,B", [(128, 16, 2, 300), (256, 8, 1, 257), (128, 3, 3, 700),
                                        (64, 4, 2, 300)])
@pytest.mark.parametrize("sms", [148, 7])
def test_gpu_window_decode_large_batches(D, Hq, Hkv, B, sms):
    """More sequences than the scan has runs, many of them empty: CTAs' shares begin and end
    anywhere (several sequences inside one share, shares inside one sequence)."""
    rng = np.random.default_rng(B + sms)
    lens = rng.integers(0, 700, B)
    lens[rng.random(B) < 0.3] = 0
    lens[:3], lens[-2:] = 0, 0
    lens[5] = 20000
    c = Case(B, np.minimum(lens, 1), np.maximum(lens - 1, 0), 10000, 5, Hq, Hkv, D, 16, "f16")
    _, got = run_decode(c, sms)
    c.check(got)


@_gpu
@pytest.mark.parametrize("i", [2, 3, 4, 5, 8, 10])
def test_gpu_one_row_batches_with_host_lengths(i):
    """The same steps as batches of one-row chunks."""
    lens, w, s, Hq, Hkv, D, PS, dtype, _ = DECODE[i]
    c = Case(100 + i, [min(1, n) for n in lens], [max(0, n - 1) for n in lens], w, s, Hq, Hkv, D,
             PS, dtype)
    _, got = run_prefill(c)
    c.check(got)


PREFILL = [
    # rows, hist, window, sinks, Hq, Hkv, D, PS, dtype
    ([1], [0], 1, 0, 4, 1, 64, 16, "f16"),
    ([40], [0], 7, 0, 4, 2, 128, 16, "bf16"),
    ([40], [1000], 7, 3, 8, 1, 256, 16, "f16"),
    ([300], [700], 128, 4, 8, 1, 256, 16, "f16"),               # CTA pairs, pages of 16
    ([300], [700], 129, 130, 8, 1, 256, 64, "bf16"),            # CTA pairs, sinks over two tiles
    ([257], [333], 300, 20, 6, 1, 256, 128, "bf16"),            # G 6: Q loaded by threads
    ([500], [0], 200, 1, 12, 2, 256, 32, "f16"),
    ([2, 0, 77, 1, 130], [9, 50, 1111, 300, 0], 100, 20, 32, 8, 128, 32, "bf16"),
    ([2, 0, 200, 1, 130], [900, 50, 1111, 300, 0], 257, 4, 16, 2, 256, 16, "f16"),
    ([130, 33], [2000, 140], 500, 4, 32, 2, 64, 64, "bf16"),
    ([8, 3], [2000, 140], 500, 200, 4, 4, 64, 16, "f16"),       # 8 packed rows: small Q
    ([150], [20], 10**6, 0, 4, 2, 128, 16, "f16"),              # the whole sequence
    ([150], [600], 50, 10**6, 4, 2, 256, 16, "f16"),
    ([64, 64], [128, 64], 64, 0, 8, 8, 128, 64, "bf16"),        # window ends on tile borders
]


@_gpu
@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_gpu_window_prefill(i):
    rows, hist, w, s, Hq, Hkv, D, PS, dtype = PREFILL[i]
    c = Case(200 + i, rows, hist, w, s, Hq, Hkv, D, PS, dtype)
    _, got = run_prefill(c)
    c.check(got)


@_gpu
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 1, 256, "f16"), (4, 1, 128, "bf16"),
                                            (4, 1, 64, "f16")])
@pytest.mark.parametrize("sms", [148, 37, 2])
def test_gpu_window_prefill_cut_row_blocks(Hq, Hkv, D, dtype, sms):
    """Few row blocks of many tiles: the schedule cuts them, parts start and end anywhere in the
    tile list (between the sinks' run and the window's too)."""
    c = Case(300 + sms, [70], [3000], 2500, 300, Hq, Hkv, D, 16, dtype)
    wp, got = run_prefill(c, num_sms=sms)
    if sms == 148:
        assert wp.plan.ws_bytes > 0
    c.check(got, pick=set(range(0, 70, 3)) | {69})


@_gpu
def test_gpu_scores_that_grow_along_the_window():
    for i, (D, Hq) in enumerate([(256, 8), (128, 8), (64, 8)]):
        c = Case(400 + i, [130, 1], [1500, 900], 700, 10, Hq, 1, D, 16, "f16", ramp=True)
        _, got = run_prefill(c)
        c.check(got, pick={0, 1, 64, 129, 130}, what=f"D={D}")
        c = Case(410 + i, [1, 1], [1500, 900], 700, 10, Hq, 1, D, 16, "f16", ramp=True)
        c.check(run_decode(c)[1], what=f"decode D={D}")


@_gpu
@pytest.mark.parametrize("seed", range(24))
def test_gpu_window_fuzz(seed):
    rng = np.random.default_rng(9000 + seed)
    Hkv = int(rng.choice([1, 2, 3]))
    G = int(rng.choice([1, 2, 3, 4, 8, 12]))
    D = int(rng.choice([64, 128, 256]))
    PS = int(rng.choice([16, 32, 64, 128]))
    dtype = str(rng.choice(["f16", "bf16"]))
    window = int(2 ** rng.uniform(0, 12))
    sinks = int(rng.choice([0, 1, 4, 16, 100, 128, 129, 260]))
    B = int(rng.choice([1, 2, 5]))
    hist = (2 ** rng.uniform(0, 12.5, B)).astype(int) - 1
    if seed % 2:
        rows = np.ones(B, int)
        rows[1:] = rng.integers(0, 2, B - 1)
        c = Case(seed, rows, hist, window, sinks, Hkv * G, Hkv, D, PS, dtype)
        c.check(run_decode(c, int(rng.choice([148, 1, 2, 5])))[1])
    else:
        rows = rng.integers(0, 200, B)
        rows[0] = max(1, rows[0])
        c = Case(seed, rows, hist, window, sinks, Hkv * G, Hkv, D, PS, dtype)
        n = int(rows.sum())
        _, got = run_prefill(c, int(rng.choice([148, 148, 11])))
        c.check(got, pick=set(rng.integers(0, n, 12).tolist()) | {0, n - 1})


@_gpu
def test_gpu_repeated_runs_and_full_windows_agree_with_the_framework():
    """Bit for bit the same on a second run. A window of the whole sequence is pa_batch_prefill and
    pa_decode rounded to the type: both sides are within the bound of the 64-bit values (theirs
    without the output's rounding), so they are within twice that of one another."""
    import torch
    bd = _binding()
    for seed, D, Hq in ((7, 128, 8), (8, 256, 8), (9, 64, 4)):
        c = Case(seed, [33, 1], [100, 300], 10**6, 0, Hq, 2, D, 16, "f16")
        _, a = run_prefill(c)
        _, b = run_prefill(c)
        assert torch.equal(a, b)
        q, k, v, t = c.device()
        bp = bd.batch_plan(Hq, 2, D, 16, c.rows, c.hist, "f16")
        want = bd.batch_prefill(bp, q, k, v, t)
        _, _, lim = c.oracle()
        assert (np.abs((a.double() - want.double()).cpu().numpy()) <= 2 * lim).all()
        c = Case(seed + 10, [1, 1], [100, 300], 10**6, 0, Hq, 2, D, 16, "f16")
        _, a = run_decode(c)
        assert torch.equal(a, run_decode(c)[1])
        q, k, v, t = c.device()
        dp = bd.decode_plan(Hq, 2, D, 16, 2, 301, "f16")
        lens = torch.tensor([101, 301], dtype=torch.int32, device="cuda")
        want = bd.decode(dp, q, k, v, t, lens).cpu()
        _, _, lim = c.oracle()
        assert (np.abs((a.double() - want.double()).numpy()) <= 2 * lim).all()


@_gpu
def test_gpu_bad_lengths_and_pages_are_reported():
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    c = Case(9, [1, 1], [500, 300], 100, 4, 8, 1, 128, 16, "f16")
    q, k, v, t = c.device()
    wp = bd.window_decode_plan(8, 1, 128, 16, 2, 501, 100, 4, "f16")
    lens = torch.tensor([501, 100000], dtype=torch.int32, device="cuda")
    bd.window_decode(wp, q, k.nan_to_num(), v.nan_to_num(), t, lens)
    assert bd.device_error(reset=True)[0] == -6
    bad = c.table.copy()
    bad[0, 500 // 16] = k.shape[0]  # the page of the newest key
    lens[1] = 301
    bd.window_decode(wp, q, k, v, torch.from_numpy(bad).cuda(), lens)
    assert bd.device_error(reset=True)[0] == -6


@_gpu
def test_gpu_window_decode_graph_replay_and_streams():
    """One captured graph on a side stream, replayed while the lengths change on the device."""
    import torch
    bd = _binding()
    B, n = 3, 900
    c = Case(10, [1] * B, [n - 1] * B, 10**6, 0, 8, 2, 256, 16, "bf16")  # every key is in the pool
    q, k, v, t = c.device()
    k, v = k.nan_to_num(), v.nan_to_num()
    wp = bd.window_decode_plan(8, 2, 256, 16, B, n, 200, 4, "bf16")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(q), bd.workspace(wp.plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bd.window_decode(wp, q, k, v, t, lens, out, ws, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bd.window_decode(wp, q, k, v, t, lens, out, ws, stream=s)
    for new in ([n, n, n], [1, 300, n], [0, 205, 128]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        step = Case.__new__(Case)
        step.__dict__.update(c.__dict__)
        live = [i for i in range(B) if new[i]]
        step.window, step.sinks = 200, 4
        step.rows, step.hist = [min(1, x) for x in new], [max(0, x - 1) for x in new]
        step.q = c.q[live]
        step.check(out[live], what=str(new))
        assert all((out[i] == 0).all() for i in range(B) if not new[i])
    del g


@_gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (8, 8, 64), (24, 2, 128)])
@pytest.mark.parametrize("L", [100, 5000])
def test_gpu_nan_reaches_the_output(Hq, Hkv, D, L):
    """A query or the keys of a sequence with a NaN, or an infinite query: that head's row is NaN
    whether its keys are split or not, and no other row changes."""
    import torch
    bd = _binding()
    gen = torch.Generator(device="cuda").manual_seed(L + D)
    B, PS = 3, 16
    n = -(-L // PS)
    k, v = (torch.randn(B * n, PS, Hkv, D, generator=gen, device="cuda").half() for _ in range(2))
    table = torch.arange(B * n, device="cuda", dtype=torch.int32).view(B, n)
    lens = torch.full((B,), L, device="cuda", dtype=torch.int32)
    q = torch.randn(B, Hq, D, generator=gen, device="cuda").half()
    wd = bd.window_decode_plan(Hq, Hkv, D, PS, B, L, 10**6, 0, "f16")
    wp = bd.window_plan(Hq, Hkv, D, PS, [1] * B, [L - 1] * B, 10**6, 0, "f16")
    dp = bd.decode_plan(Hq, Hkv, D, PS, B, L, "f16")
    common = (L // 2) // PS
    pd = bd.prefix_decode_plan(Hq, Hkv, D, PS, B, common * PS, L, "f16")
    shared = table.clone()
    shared[:, :common] = table[0, :common]
    runs = {"window decode": lambda q, k: bd.window_decode(wd, q, k, v, table, lens),
            "window prefill": lambda q, k: bd.window_prefill(wp, q, k, v, table),
            "decode": lambda q, k: bd.decode(dp, q, k, v, table, lens),
            "prefix decode": lambda q, k: bd.prefix_decode(pd, q, k, v, table[0, :common].clone(),
                                                           shared, lens)}
    bad_q = q.clone()
    bad_q[1, 0, 3], bad_q[2, 1, 5] = float("nan"), float("inf")
    bad_k = k.clone()
    bad_k[n + common:2 * n, :, :, 0] = float("nan")  # sequence 1's keys past the shared pages
    for name, run in runs.items():
        want, got, keys = run(q, k), run(bad_q, k), run(q, bad_k)
        rows = torch.zeros(B, Hq, dtype=torch.bool, device="cuda")
        rows[1, 0] = rows[2, 1] = True
        assert bool(got[rows].isnan().all()), name
        assert torch.equal(got[~rows], want[~rows]), name
        assert bool(keys[1].isnan().all()), name
        assert torch.equal(keys[[0, 2]], want[[0, 2]]), name


@_gpu
@pytest.mark.parametrize("Hq,Hkv,D,PS", [(16, 2, 256, 64), (8, 4, 64, 16)])
def test_gpu_pages_past_2_to_31_elements(Hq, Hkv, D, PS):
    """Pages whose elements lie past 2^31 (their bytes past 2^32) of a pool: attention and the cache
    write give the bits that the same pages give in a small one, and write nowhere else."""
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    gen = torch.Generator(device="cuda").manual_seed(D)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()  # noqa: E731
    B, L, prefix = 4, 1500, 1024
    n, common = -(-L // PS), prefix // PS
    pages = common + B * (n - common)
    far = 2**31 // (PS * Hkv * D) + 1  # the first of the far pages
    small = [rand(pages, PS, Hkv, D) for _ in range(2)]
    large = [torch.zeros(far + pages, PS, Hkv, D, dtype=torch.half, device="cuda")
             for _ in range(2)]
    for x, y in zip(large, small):
        x[far:] = y
    table = torch.arange(n, device="cuda", dtype=torch.int32).repeat(B, 1)
    table[:, common:] += (n - common) * torch.arange(B, device="cuda", dtype=torch.int32)[:, None]
    lens = torch.tensor([L, 1300, prefix, 77], dtype=torch.int32, device="cuda")
    q, rows = rand(B, Hq, D), rand(231, Hq, D)
    wd = bd.window_decode_plan(Hq, Hkv, D, PS, B, L, 700, 20, "f16")
    wp = bd.window_plan(Hq, Hkv, D, PS, [1, 200, 30, 0], [L - 1, 1000, 900, 5], 700, 20, "f16")
    pd = bd.prefix_decode_plan(Hq, Hkv, D, PS, B, prefix, L, "f16")
    for run in (lambda k, v, t: bd.window_decode(wd, q, k, v, t, lens),
                lambda k, v, t: bd.window_prefill(wp, rows, k, v, t),
                lambda k, v, t: bd.prefix_decode(pd, q, k, v, t[0, :common].clone(), t, lens)):
        assert torch.equal(run(*small, table), run(*large, table + far))
    T = 100
    x = [rand(T, h, D) for h in (Hq, Hkv, Hkv)]
    slots = torch.randperm(pages * PS, generator=gen, device="cuda")[:T].int()
    pos, rope = torch.arange(T, dtype=torch.int32, device="cuda"), bd.rope_table(T, D)
    a = bd.qk_rope_append(*x, pos, slots, rope, *small)
    b = bd.qk_rope_append(*x, pos, slots + far * PS, rope, *large)
    assert torch.equal(a, b) and bd.device_error(reset=True)[0] == 0
    for x, y in zip(large, small):
        assert torch.equal(x[far:], y) and not x[:far].any()
