"""Decode over a shared prefix (pa_prefix_decode): the first prefix_len keys of every sequence are
the same pages, read and multiplied once for the batch; each sequence's own keys follow.

The result is decode attention of each whole sequence: the oracle is a direct softmax in 64 bits
over each sequence's keys, with the tolerance of the window tests (the same roundings: one of each
probability, one of the output, fp32 between).
"""
import ctypes
import math

import numpy as np
import pytest

from tests.conftest import cuda_available
from tests.test_window import Case

gpu = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def _gpu(f):
    for m in gpu:
        f = m(f)
    return f


def _binding():
    from paged_kv_long_b200 import binding
    return binding


class PrefixCase(Case):
    """Sequences of lens[b] keys whose first `prefix` are shared pages. Slots that hold no key are
    NaN; the block table's entries over the prefix, and past a sequence, are -1."""

    def __init__(self, seed, lens, prefix, Hq, Hkv, D, PS, dtype, ramp=False):
        import torch
        self.Hq, self.Hkv, self.D, self.PS, self.dtype = Hq, Hkv, D, PS, dtype
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        self.lens, self.prefix, self.window, self.sinks = [int(n) for n in lens], prefix, 10**9, 0
        g = torch.Generator().manual_seed(seed)
        B, common = len(lens), prefix // PS
        stride = max(common, max(math.ceil(n / PS) for n in self.lens))
        own = [max(0, math.ceil(n / PS) - common) for n in self.lens]
        num_pages = common + sum(own) + 2
        ids = torch.randperm(num_pages, generator=g).numpy().astype(np.int32)
        self.prefix_table, at = ids[:common].copy(), common
        self.table = np.full((B, stride), -1, np.int32)  # with the prefix: what the oracle reads
        self.block_table = self.table.copy()
        for b, n in enumerate(own):
            self.table[b, :common] = self.prefix_table
            self.block_table[b, common:common + n] = ids[at:at + n]
            self.table[b, common:common + n] = ids[at:at + n]
            at += n
        self.k = torch.full((num_pages, PS, Hkv, D), float("nan"), dtype=self.dt)
        self.v = self.k.clone()
        for b in [None] + list(range(B)):
            key = np.arange(prefix) if b is None else np.arange(prefix, max(prefix, self.lens[b]))
            page = self.prefix_table[key // PS] if b is None else self.table[b, key // PS]
            slot = torch.from_numpy(page.astype(np.int64) * PS + key % PS)
            for pool in (self.k, self.v):
                x = torch.randn(len(key), Hkv, D, generator=g)
                if ramp and pool is self.k:
                    x[..., 0] += torch.from_numpy(key * (64.0 / max(self.lens))).float()[:, None]
                pool.flatten(0, 1)[slot] = x.to(self.dt)
        self.rows = [min(1, n) for n in self.lens]
        self.hist = [max(0, n - 1) for n in self.lens]
        self.full_q = torch.randn(B, Hq, D, generator=g)
        if ramp:
            self.full_q[..., 0] = 4.0
        self.full_q = self.full_q.to(self.dt)
        self.live = torch.tensor([n > 0 for n in self.lens])
        self.q = self.full_q[self.live]

    def run(self, num_sms=148, max_len=None, stream=None):
        import torch
        bd = _binding()
        bd.device_error(reset=True)
        pp = bd.prefix_decode_plan(self.Hq, self.Hkv, self.D, self.PS, len(self.lens), self.prefix,
                                   max_len or max(1, max(self.lens)), self.dtype, num_sms=num_sms)
        q = self.full_q.cuda()
        out = torch.full_like(q, float("nan"))
        ws = bd.workspace(pp.plan)
        ws.fill_(float("nan"))
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        got = bd.prefix_decode(pp, q, self.k.cuda(), self.v.cuda(), dev(self.prefix_table),
                               dev(self.block_table), dev(np.array(self.lens, np.int32)), out, ws,
                               stream=stream)
        torch.cuda.synchronize()
        assert bd.device_error(reset=True)[0] == 0
        got = got.cpu()
        assert (got[~self.live] == 0).all()
        return pp, got[self.live]


# ------------------------------------------------------------------------------------ CPU


def test_oracle_is_attention_over_prefix_and_own_keys():
    """Sequences that are equal past the prefix and have equal queries get equal outputs, and a
    prefix of equal keys and values counts by its length."""
    import torch
    c = PrefixCase(1, [40, 33, 0], 32, 2, 1, 64, 16, "f16")
    _, out, _ = c.oracle()
    assert len(out) == 2
    key = np.arange(40)
    slot = c.table[0, key // 16].astype(np.int64) * 16 + key % 16
    k = c.k.flatten(0, 1)[torch.from_numpy(slot)].double().numpy()[:, 0]
    v = c.v.flatten(0, 1)[torch.from_numpy(slot)].double().numpy()[:, 0]
    for h in range(2):
        x = k @ c.q[0, h].double().numpy() / 8
        w = np.exp(x - x.max())
        np.testing.assert_allclose(out[0, h], w @ v / w.sum(), atol=1e-13)


def test_plan_fields_and_workspace():
    bd = _binding()
    mk = lambda **a: bd.prefix_decode_plan(**{**dict(  # noqa: E731
        n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=16, batch=32, prefix_len=32768,
        max_seq_len=33792, dtype="f16", num_sms=148), **a}).plan
    p = mk()  # 256 packed rows a head: one CTA pair per head and split, a wave of 74 pairs at most
    assert p.q_tiles == 2 and p.ctas_per_unit == 2 and 1 < 2 * p.splits <= 74
    assert p.policy == 6 and p.hist_len == 33792
    # the own part: two CTAs on each SM that the prefix's pairs leave, 8 tiles and a start a unit
    aside = 148 - 2 * 2 * p.splits
    assert 2 * 4 <= p.units <= min(2 * aside, 32 * 2 * 9 // 2)
    q = mk(max_seq_len=33000)                         # fewer own keys: fewer SMs aside
    assert q.splits >= p.splits and q.units <= p.units
    # the prefix's units do not fit one wave: one part after the other, each on every SM
    q = mk(batch=1024, n_q_heads=32, n_kv_heads=8, head_dim=128)
    assert q.units == 296
    assert p.ws_bytes == (p.splits * 512 + 512 + 2 * p.units * 8) * 257 * 4
    p = mk(batch=4)
    assert p.q_tiles == 1 and p.ctas_per_unit == 1
    p = mk(head_dim=64)                               # uniform splits: 32 partials at most
    assert p.splits <= 30 and p.units >= 64
    assert p.ws_bytes == (p.splits + p.units // 64) * 512 * 65 * 4
    assert mk(prefix_len=16).splits == 1
    for bad in (dict(prefix_len=0), dict(prefix_len=24), dict(batch=0), dict(max_seq_len=0),
                dict(head_dim=96), dict(page_size=8), dict(n_q_heads=15),
                dict(prefix_len=2**31), dict(max_seq_len=2**31)):
        with pytest.raises(bd.PaError):
            mk(**bad)


def test_refusals():
    """Checked before any device work: these run without a GPU."""
    bd = _binding()
    lib = bd.load_library()
    pp = bd.prefix_decode_plan(16, 2, 256, 16, 4, 320, 1000, "f16", num_sms=148)
    dp = bd.decode_plan(16, 2, 256, 16, 4, 1000, "f16", num_sms=148)
    f, big, ref = ctypes.c_void_p(1 << 20), 1 << 40, ctypes.byref
    bad = "PA_ERR_INVALID_ARG"

    def call(plan=pp.plan, prefix=320, q=f, k=f, pre=f, table=f, stride=64, lens=f, pages=100,
             out=f, ws=f, n=big):
        return bd.STATUS[lib.pa_prefix_decode(ref(plan), prefix, q, k, f, pre, table, stride,
                                              lens, pages, out, ws, n, None)]

    assert call(plan=dp) == call(prefix=0) == call(prefix=8) == bad
    assert call(prefix=640) == bad            # another prefix: its splits, units and workspace
    assert call(q=None) == call(k=None) == call(pre=None) == call(table=None) == bad
    assert call(lens=None) == call(out=None) == call(stride=0) == call(pages=0) == bad
    assert call(q=ctypes.c_void_p((1 << 20) + 4)) == bad
    assert call(ws=None) == call(n=64) == "PA_ERR_WORKSPACE"
    assert call(pages=1 << 27) == "PA_ERR_UNSUPPORTED"
    name = lambda st: bd.STATUS[st]  # noqa: E731
    assert name(lib.pa_decode(ref(pp.plan), f, f, f, f, 64, f, 100, f, f, big, None)) == bad
    assert name(lib.pa_combine(ref(pp.plan), f, big, f, None)) == bad
    assert name(lib.pa_window_decode(ref(pp.plan), 10, 0, f, f, f, f, 64, f, 100, f, f, big,
                                     None)) == bad


def test_a_step_past_the_32_bit_slots_is_refused_before_anything_runs():
    """128 sequences x 2 heads x 2^24 KV tiles of a table row: refused before the tensor maps (which
    need a GPU's driver), and so before the prefix's kernel; 32 sequences get past it."""
    bd = _binding()
    lib, f = bd.load_library(), ctypes.c_void_p(1 << 20)
    for B, want in ((128, "PA_ERR_UNSUPPORTED"), (32, "PA_ERR_CUDA")):
        if want == "PA_ERR_CUDA" and cuda_available():
            continue
        pp = bd.prefix_decode_plan(16, 2, 256, 16, B, 320, 1000, "f16", num_sms=148)
        assert bd.STATUS[lib.pa_prefix_decode(ctypes.byref(pp.plan), 320, f, f, f, f, f, 1 << 27,
                                              f, 100, ctypes.c_void_p(1 << 30), f, 1 << 40,
                                              None)] == want
        wd = bd.window_decode_plan(16, 2, 256, 16, B, 1000, 2**31 - 1, 4, "f16", num_sms=148)
        assert bd.STATUS[lib.pa_window_decode(ctypes.byref(wd.plan), 2**31 - 1, 4, f, f, f, f,
                                              1 << 27, f, 100, ctypes.c_void_p(1 << 30), f,
                                              1 << 40, None)] == want


# ------------------------------------------------------------------------------------ GPU

CASES = [
    # lens, prefix, Hq, Hkv, D, PS, dtype, num_sms
    ([17], 16, 8, 1, 256, 16, "f16", 148),
    ([16, 16], 16, 16, 2, 128, 16, "bf16", 148),               # no own keys
    ([300, 0, 129, 1, 144, 145], 144, 16, 2, 256, 16, "f16", 148),  # padded, inside the prefix
    ([700, 640, 641, 100, 0], 640, 16, 2, 128, 64, "bf16", 148),
    ([3000] * 5 + [2100] * 4, 2080, 32, 8, 128, 32, "f16", 148),
    ([1300 + 37 * i for i in range(17)], 1296, 8, 1, 256, 16, "bf16", 148),  # 136 rows: a pair
    ([1200 + 7 * i for i in range(40)], 1152, 24, 4, 256, 128, "f16", 148),  # G 6, two units
    ([1200 + 7 * i for i in range(40)], 1152, 8, 8, 128, 128, "f16", 5),     # G 1, few CTAs
    ([900, 530, 0, 514, 2000], 512, 32, 2, 64, 16, "bf16", 148),  # G 16 at D 64: uniform splits
    ([900, 530, 0, 100, 2000], 528, 4, 4, 64, 16, "f16", 148),    # the boundary inside a tile
    ([900, 530, 0, 100, 2000], 528, 32, 2, 256, 16, "f16", 148),  # G 16 at D 256
    ([5000, 4097], 4096, 8, 2, 256, 64, "bf16", 9),
]


@_gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_gpu_prefix_decode(i):
    *shape, sms = CASES[i]
    c = PrefixCase(500 + i, *shape)
    pp, got = c.run(sms)
    c.check(got, what=f"{pp.plan.splits} prefix splits, {pp.plan.units} units")


@_gpu
def test_gpu_growing_scores_and_other_stream():
    import torch
    for i, (Hq, D) in enumerate([(8, 256), (8, 128), (8, 64)]):
        c = PrefixCase(600 + i, [1500, 1290, 1281], 1280, Hq, 1, D, 16, "f16", ramp=True)
        c.check(c.run()[1], what=f"D={D}")
    s = torch.cuda.Stream()
    c.check(c.run(stream=s)[1])


@_gpu
def test_gpu_lengths_past_the_plans_estimate():
    """max_seq_len only sizes the launch."""
    c = PrefixCase(700, [3000, 300, 290], 256, 16, 2, 256, 16, "f16")
    c.check(c.run(max_len=257)[1])


@_gpu
@pytest.mark.parametrize("seed", range(16))
def test_gpu_prefix_fuzz(seed):
    rng = np.random.default_rng(7000 + seed)
    Hkv, G = int(rng.choice([1, 2, 3])), int(rng.choice([1, 3, 4, 8, 12]))
    D, PS = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128]))
    B = int(2 ** rng.uniform(0, 6))
    prefix = PS * int(2 ** rng.uniform(0, math.log2(3000 / PS)))
    lens = prefix + (2 ** rng.uniform(0, 10, B)).astype(int) - 1
    lens[rng.random(B) < 0.15] = 0
    lens[rng.random(B) < 0.1] = max(1, prefix // 2)
    c = PrefixCase(seed, lens, prefix, Hkv * G, Hkv, D, PS, str(rng.choice(["f16", "bf16"])))
    if not any(lens):
        return
    c.check(c.run(int(rng.choice([148, 148, 3])))[1])


@_gpu
def test_gpu_prefix_decode_equals_decode_and_repeats():
    """Bit for bit the same on a second run, and near pa_decode on the whole table."""
    import torch
    bd = _binding()
    c = PrefixCase(800, [2100, 2055, 2048, 3000], 2048, 16, 2, 256, 16, "f16")
    _, a = c.run()
    assert torch.equal(a, c.run()[1])
    dp = bd.decode_plan(16, 2, 256, 16, 4, 3000, "f16")
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    want = bd.decode(dp, c.full_q.cuda(), c.k.cuda(), c.v.cuda(), dev(c.table),
                     dev(np.array(c.lens, np.int32))).cpu()
    # both round their probabilities: twice the bound of one
    _, _, lim = c.oracle()
    assert (np.abs(a.double().numpy() - want.double().numpy()) <= 2 * lim).all()


@_gpu
def test_gpu_graph_replay_follows_lengths_and_reports_bad_pages():
    import torch
    bd = _binding()
    n = [900, 900, 900]
    c = PrefixCase(900, n, 512, 8, 2, 128, 16, "bf16")
    q, k, v = c.full_q.cuda(), c.k.cuda(), c.v.cuda()
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    pre, table = dev(c.prefix_table), dev(c.block_table)
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    pp = bd.prefix_decode_plan(8, 2, 128, 16, 3, 512, 900, "bf16")
    out, ws = torch.empty_like(q), bd.workspace(pp.plan)
    bd.prefix_decode(pp, q, k, v, pre, table, lens, out, ws)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bd.prefix_decode(pp, q, k, v, pre, table, lens, out, ws, stream=s)
    bd.device_error(reset=True)
    for new in (n, [513, 700, 0], [1, 512, 900]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        step = PrefixCase.__new__(PrefixCase)
        step.__dict__.update(c.__dict__)
        live = [i for i in range(3) if new[i]]
        step.rows, step.hist = [min(1, x) for x in new], [max(0, x - 1) for x in new]
        step.q = c.full_q[live]
        step.check(out[live], what=str(new))
        assert all((out[i] == 0).all() for i in range(3) if not new[i])
    del g
    assert bd.device_error(reset=True)[0] == 0
    bad = c.prefix_table.copy()
    bad[3] = -1
    bd.prefix_decode(pp, q, k.nan_to_num(), v.nan_to_num(), dev(bad), table, lens, out, ws)
    assert bd.device_error(reset=True)[0] == -6


@_gpu
@pytest.mark.parametrize("op", ["prefix", "window"])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (8, 8, 64)])
def test_gpu_calls_in_a_row_share_a_workspace(op, Hq, Hkv, D):
    """The kernels of a call overlap (the own keys run beside the prefix, the merge starts early):
    calls one after another on one workspace, with the queries and lengths copied in between them
    in stream order, on two streams at once, give the bits of calls that ran alone."""
    import torch
    bd = _binding()
    PS, B, prefix, most = 16, 12, 4096, 4096 + 900
    rng = np.random.default_rng(D + Hkv)
    gen = torch.Generator(device="cuda").manual_seed(D)
    n = -(-most // PS)
    table = torch.from_numpy(rng.permutation(B * n).astype(np.int32).reshape(B, n)).cuda()
    table[:, :prefix // PS] = table[0, :prefix // PS].clone()
    pre = table[0, :prefix // PS].clone()
    k, v = (torch.randn(B * n, PS, Hkv, D, generator=gen, device="cuda").half() for _ in range(2))
    steps = 24
    qs = torch.randn(steps, B, Hq, D, generator=gen, device="cuda").half()
    lens = torch.from_numpy(rng.integers(prefix - 3, most, (steps, B)).astype(np.int32)).cuda()
    if op == "prefix":
        plan = bd.prefix_decode_plan(Hq, Hkv, D, PS, B, prefix, most, "f16")
    else:
        plan = bd.window_decode_plan(Hq, Hkv, D, PS, B, most, 2000, 5, "f16")

    def call(q, length, out, ws, stream=None):
        if op == "prefix":
            return bd.prefix_decode(plan, q, k, v, pre, table, length, out, ws, stream)
        return bd.window_decode(plan, q, k, v, table, length, out, ws, stream)

    alone = []
    for i in range(steps):
        alone.append(call(qs[i].clone(), lens[i].clone(), None, bd.workspace(plan.plan)))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    state = [(torch.empty_like(qs[0]), torch.empty_like(lens[0]), torch.empty_like(qs[0]),
              bd.workspace(plan.plan)) for _ in streams]
    keep = [torch.empty(steps, B, Hq, D, dtype=torch.half, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for i in range(steps):
        for j, s in enumerate(streams):
            q, length, out, ws = state[j]
            at = i if j == 0 else steps - 1 - i
            with torch.cuda.stream(s):
                q.copy_(qs[at])
                length.copy_(lens[at])
                call(q, length, out, ws)
                keep[j][at].copy_(out)
    torch.cuda.synchronize()
    for i in range(steps):
        assert torch.equal(keep[0][i], alone[i]) and torch.equal(keep[1][i], alone[i]), i
    assert bd.device_error(reset=True)[0] == 0
