"""Calls given a stream that is not the current one, or tensors of a device that is not: a call runs
on its tensors' device, and the tensors that it makes itself come from the memory of the stream
that its kernels run on.

A block that the current stream has freed may be handed out again to work of that stream at once,
because it runs behind the block's last use. Kernels on another stream do not: written there, the
block is still in use by whatever the current stream has pending.
"""
import ctypes

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


# ------------------------------------------------------------------------------------ CPU


class FakeStream:
    """A stream that knows when it is the current one."""

    def __init__(self, handle):
        self.cuda_stream, self.inside = handle, False


@pytest.fixture
def fake_device(monkeypatch):
    """torch tensors that say they are on device 0, a library that notes the streams it is given,
    and torch's allocations noted with the stream that was current: (library's calls, allocations,
    the stream that torch has made current)."""
    import torch
    bd = _binding()
    calls, made, current = [], [], [None]

    class On(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

        def record_stream(self, stream):
            made.append(("recorded", stream))

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                calls.append((name, args[-1]))
                return 0
            return fn

    class Switch:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, current[0] = current[0], self.stream

        def __exit__(self, *exc):
            current[0] = self.before

    def noting(make):
        def fn(*args, **kw):
            made.append((make.__name__, current[0]))
            kw.pop("device", None)
            return make(*args, **kw).as_subclass(On)
        return fn

    def on(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype).as_subclass(On)

    empty_like, empty, new_empty = torch.empty_like, torch.empty, torch.Tensor.new_empty
    monkeypatch.setattr(bd, "load_library", lambda path=None: Lib())
    monkeypatch.setattr(torch, "empty_like", noting(empty_like))
    monkeypatch.setattr(torch, "empty", noting(empty))
    monkeypatch.setattr(On, "new_empty", noting(new_empty))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 7)
    monkeypatch.setattr(torch.cuda, "stream", Switch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "the current one")
    return calls, made, on


def _window_call(bd, on, stream):
    import torch
    wp = bd.WindowPlan(_plan_on_host(bd, 5), 100, 4)
    wp.ws_numel = 64
    pool = on(9, 16, 2, 128, dtype=torch.float16)
    return bd.window_decode(wp, on(3, 8, 128, dtype=torch.float16), pool, pool,
                            on(3, 4, dtype=torch.int32), on(3, dtype=torch.int32), stream=stream)


def _plan_on_host(bd, policy):
    p = bd.Plan()
    p.n_q_heads, p.n_kv_heads, p.head_dim, p.page_size, p.group = 8, 2, 128, 16, 4
    p.batch = p.chunk_rows = 3
    p.policy, p.ws_bytes = policy, 256
    return p


def _prefix_call(bd, on, stream):
    import torch
    pp = bd.PrefixPlan(_plan_on_host(bd, 6), 32)
    pool = on(9, 16, 2, 128, dtype=torch.float16)
    return bd.prefix_decode(pp, on(3, 8, 128, dtype=torch.float16), pool, pool,
                            on(2, dtype=torch.int32), on(3, 4, dtype=torch.int32),
                            on(3, dtype=torch.int32), stream=stream)


def _tables_call(bd, on, stream):
    import torch
    i32 = torch.int32
    return bd.block_tables(on(3, dtype=i32), on(3, dtype=i32), on(9, dtype=i32), on(1, dtype=i32),
                           on(3, 4, dtype=i32), 5, 16, 9, stream=stream)


def _rope_call(bd, on, stream):
    import torch
    f16, i32 = torch.float16, torch.int32
    pool = on(9, 16, 2, 64, dtype=f16)
    return bd.qk_rope_append(on(5, 8, 64, dtype=f16), on(5, 2, 64, dtype=f16),
                             on(5, 2, 64, dtype=f16), on(5, dtype=i32), on(5, dtype=i32),
                             on(20, 64, dtype=torch.float32), pool, pool, stream=stream)


CALLS = {"window": (_window_call, 2), "prefix": (_prefix_call, 2), "tables": (_tables_call, 1),
         "rope": (_rope_call, 1)}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_made_by_a_call_are_the_calls_streams(fake_device, name):
    calls, made, on = fake_device
    call, n = CALLS[name]
    call(_binding(), on, None)  # without a stream: all on the current one
    assert [s for _, s in made] == [None] * n and [s for _, s in calls] == [7]
    del calls[:], made[:]
    s = FakeStream(ctypes.c_void_p(11))
    call(_binding(), on, s)
    assert [x for _, x in calls] == [s.cuda_stream]
    allocated = [x for what, x in made if what != "recorded"]
    assert allocated == [s] * n
    # what the caller gets back is kept for the current stream's work as well; the workspace is not
    assert [x for what, x in made if what == "recorded"] == ["the current one"]


def _older_calls(bd, on):
    """name -> (a call of the entry points without a window or prefix, tensors that it makes)."""
    import torch
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    pool, table = on(9, 16, 2, 128, dtype=f16), on(9, dtype=i32)
    q, rows = on(3, 8, 128, dtype=f16), on(3, 2, 128, dtype=f16)
    tables, lens = on(3, 4, dtype=i32), on(3, dtype=i32)
    out, ws = on(3, 8, 128, dtype=f32), on(64, dtype=f32)
    p = _plan_on_host(bd, 0)
    p.paged, p.splits, p.hist_len = 1, 2, 60
    bp = bd.BatchPlan(p, [1, 1, 1], [9, 9, 9])
    return {
        "append": (lambda s: bd.kv_append(rows, rows, pool, pool, table, 60, s), 0),
        "publish": (lambda s: bd.kv_publish(rows, rows, pool, pool, table, 0, 3, s), 0),
        "prefill": (lambda s: bd.prefill(p, q, pool, pool, table, out, ws, s), 0),
        "combine": (lambda s: bd.combine(p, ws, out, s), 0),
        "both": (lambda s: bd.prefill_combine(p, q, pool, pool, table, stream=s), 2),
        "noalloc": (lambda s: bd.prefill_noalloc(p, q, pool, pool, table, out, s), 0),
        "decode": (lambda s: bd.decode(p, q, pool, pool, tables, lens, stream=s), 2),
        "batch": (lambda s: bd.batch_prefill(bp, q, pool, pool, tables, stream=s), 2),
    }


OLDER = ("append", "publish", "prefill", "combine", "both", "noalloc", "decode", "batch")


@pytest.mark.parametrize("name", OLDER)
def test_older_calls_too(fake_device, name):
    calls, made, on = fake_device
    call, n = _older_calls(_binding(), on)[name]
    del made[:]
    s = FakeStream(ctypes.c_void_p(11))
    call(s)
    assert calls and [x for _, x in calls] == [s.cuda_stream] * len(calls)
    assert [x for what, x in made if what != "recorded"] == [s] * n
    assert [x for what, x in made if what == "recorded"] == ["the current one"] * (n > 0)


@pytest.mark.parametrize("name", OLDER + tuple(CALLS))
def test_calls_run_on_the_device_of_their_tensors(fake_device, monkeypatch, name):
    """Device 1 is current, the tensors are on device 0."""
    import torch
    calls, _, on = fake_device
    bd = _binding()
    entered = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append((self.index, len(calls)))

        def __exit__(self, *exc):
            entered.append((None, len(calls)))

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + d)
    monkeypatch.setattr(torch.cuda, "device", Device)
    if name in CALLS:
        CALLS[name][0](bd, on, None)
    else:
        _older_calls(bd, on)[name][0](None)
    assert calls and [x for _, x in calls] == [70] * len(calls)
    # each launch stands between entering device 0 and leaving it
    assert entered == [e for i in range(len(calls)) for e in ((0, i), (None, i + 1))]


@pytest.mark.parametrize("name", ["prefill", "decode", "batch"])
def test_tensors_of_two_devices_are_refused(fake_device, name):
    import torch
    _, _, on = fake_device
    bd = _binding()
    far = on(9, 16, 2, 128, dtype=torch.float16)
    far.get_device = lambda: 1
    near, p = on(9, 16, 2, 128, dtype=torch.float16), _plan_on_host(bd, 0)
    p.paged, p.splits = 1, 2
    q, i32 = on(3, 8, 128, dtype=torch.float16), torch.int32
    with pytest.raises(ValueError, match="one device"):
        if name == "prefill":
            bd.prefill(p, q, far, near, on(9, dtype=i32), None)
        elif name == "decode":
            bd.decode(p, q, near, far, on(3, 4, dtype=i32), on(3, dtype=i32))
        else:
            bd.batch_prefill(bd.BatchPlan(p, [1] * 3, [9] * 3), q, near, far, on(3, 4, dtype=i32))


# ------------------------------------------------------------------------------------ GPU


def _inputs(Hq=16, Hkv=2, D=256, PS=16, B=6, L=900):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    n = -(-L // PS)
    pool = [torch.randn(B * n, PS, Hkv, D, generator=g, device="cuda").half() for _ in range(2)]
    table = torch.arange(B * n, device="cuda", dtype=torch.int32).view(B, n)
    q = torch.randn(B, Hq, D, generator=g, device="cuda").half()
    return q, pool[0], pool[1], table, torch.full((B,), L, device="cuda", dtype=torch.int32)


@_gpu
@pytest.mark.parametrize("op", ["window decode", "window prefill", "prefix decode", "tables",
                                "rope"])
def test_gpu_call_on_another_stream_leaves_memory_of_pending_work(op):
    """The current stream frees tensors of the sizes that the call makes, with work on them still
    pending. The call on another stream gets other memory, and the right results."""
    import torch
    bd = _binding()
    q, k, v, table, lens = _inputs()
    B, Hq, D = q.shape
    PS, Hkv, L = 16, 2, 900
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "window decode":
        plan = bd.window_decode_plan(Hq, Hkv, D, PS, B, L, 500, 4, "f16")
        call = lambda s: [bd.window_decode(plan, q, k, v, table, lens, stream=s)]  # noqa: E731
    elif op == "window prefill":
        plan = bd.window_plan(Hq, Hkv, D, PS, [1] * B, [L - 1] * B, 500, 4, "f16")
        call = lambda s: [bd.window_prefill(plan, q, k, v, table, stream=s)]  # noqa: E731
    elif op == "prefix decode":
        shared = table.clone()
        shared[:, :40] = table[0, :40]
        pre = table[0, :40].clone()
        plan = bd.prefix_decode_plan(Hq, Hkv, D, PS, B, 640, L, "f16")
        call = lambda s: [bd.prefix_decode(plan, q, k, v, pre, shared, lens,  # noqa: E731
                                           stream=s)]
    elif op == "tables":
        free, used = torch.arange(500, **i32), torch.zeros(1, **i32)
        rows, hist = torch.full((B,), 300, **i32), torch.zeros(B, **i32)
        call = lambda s: bd.block_tables(rows, hist, free, used, table, 1800,  # noqa: E731
                                         PS, 500, stream=s)
    else:
        T = 900
        g = torch.Generator(device="cuda").manual_seed(6)
        x = [torch.randn(T, h, D, generator=g, device="cuda").half() for h in (Hq, Hkv, Hkv)]
        at, rope = torch.arange(T, **i32), bd.rope_table(T, D)
        call = lambda s: [bd.qk_rope_append(*x, at, at, rope, k, v, stream=s)]  # noqa: E731
    want = [t.clone() for t in call(None)]
    ws = 0 if op in ("tables", "rope") else plan.ws_numel
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    nbytes = want[0].untyped_storage().nbytes() if op != "tables" else 4 * (2 * 1800 + 2 * B + 2)
    held = [torch.empty(nbytes, dtype=torch.uint8, device="cuda"),
            torch.empty(max(1, ws), dtype=torch.float32, device="cuda")]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # about 10 ms of the current stream's time
    for t in held:
        t.fill_(255)               # the pending work on the freed memory
    pointers = {t.untyped_storage().data_ptr() for t in held}
    del held, t
    got = call(s)
    assert not pointers & {t.untyped_storage().data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
