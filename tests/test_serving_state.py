"""What a ServingBatch knows and refuses on the host. On a GPU the refused steps are followed by
accepted ones; without one the state sits on the CPU (plans are host code) and nothing is launched.
"""
import numpy as np
import pytest

from tests.conftest import cuda_available


def serving(batch=2, max_len=128, num_pages=None, rope_rows=None, heads=(8, 2, 64), **kw):
    """A ServingBatch on the CPU, and the tensors that its steps change, with their copies."""
    import torch
    from paged_kv_long_b200.runner import ServingBatch
    rope = torch.zeros(rope_rows or max_len, 32)
    pages = batch * -(-max_len // 16) if num_pages is None else num_pages
    s = ServingBatch(*heads, 16, "f16", batch, max_len, rope, pages, device="cpu", num_sms=148,
                     **kw)
    state = (s.k_pool, s.v_pool, s.block_table, s.pages_used, s.hist_lens)
    return s, state, [t.clone() for t in state]


def rows(s, n):
    import torch
    Hq, Hkv, D, _ = s.shape
    return [torch.ones(n, h, D, dtype=torch.float16) for h in (Hq, Hkv, Hkv)]


def unchanged(s, state, before, hist):
    import torch
    assert all(torch.equal(a, b) for a, b in zip(state, before))
    assert (s.hist == hist).all() and s.q_rot is None


@pytest.fixture
def no_launches(monkeypatch):
    """Fails the test at the first launch of a step."""
    from paged_kv_long_b200 import binding

    def launched(*args, **kw):
        pytest.fail("the step was under way")

    for name in ("block_tables", "qk_rope_append"):
        monkeypatch.setattr(binding, name, launched)


@pytest.mark.parametrize("q_lens", [[3], [3, 4, 5], [-1, 4], [[3, 4]]])
def test_chunks_that_are_not_the_batchs_change_nothing(no_launches, q_lens):
    s, state, before = serving(window=50)
    with pytest.raises(ValueError, match="q_lens"):
        s.step(*rows(s, 3), q_lens)
    unchanged(s, state, before, 0)


def test_rows_of_another_shape_type_or_device_change_nothing(no_launches):
    s, state, before = serving()
    q, k, v = rows(s, 7)
    for bad in ((q[:6], k, v), (q, k[:, :1], v), (q, k, v.float()), (q, k.to("meta"), v)):
        with pytest.raises(ValueError):
            s.step(*bad, [3, 4])
    with pytest.raises(ValueError):
        s.decode(q, k, v)  # two requests, seven rows
    unchanged(s, state, before, 0)


@pytest.mark.parametrize("window", [0, 50])
def test_a_step_that_cannot_be_planned_changes_nothing(no_launches, window):
    """600 KV heads: more row blocks than a launch's schedule holds, however few the rows."""
    from paged_kv_long_b200 import binding
    s, state, before = serving(heads=(600, 600, 64), window=window, max_len=16)
    with pytest.raises(binding.PaError, match="UNSUPPORTED"):
        s.step(*rows(s, 2), [1, 1])
    unchanged(s, state, before, 0)


def test_a_request_past_its_last_row_changes_nothing(no_launches):
    """Past its table row (three pages), or past the rotation table where that is shorter; by a
    chunk or a token."""
    for kw, most in ((dict(max_len=40, rope_rows=99), 48), (dict(max_len=64, rope_rows=41), 41)):
        s, state, before = serving(num_pages=50, **kw)
        more = f"request 1 would hold {most + 1} rows; the most is {most}"
        with pytest.raises(ValueError, match=more):
            s.step(*rows(s, most + 4), [3, most + 1])
        unchanged(s, state, before, 0)
        s.hist += [7, most]  # as if replayed
        with pytest.raises(ValueError, match=more):
            s.decode(*rows(s, 2))
        s.check_room([most - 7, 0])
        with pytest.raises(ValueError, match="request 0"):
            s.check_room([most - 6, 0])
        unchanged(s, state, before, [7, most])


@pytest.mark.parametrize("prefix", [0, 48])
def test_a_step_past_the_free_pages_changes_nothing(no_launches, prefix):
    """Seven pages past the prefix's three: whole pages of each request's own rows count."""
    shared = prefix // 16
    s, state, before = serving(max_len=200, num_pages=7 + shared, prefix_len=prefix)
    unchanged(s, state, before, prefix)
    s.check_room([16 * 6, 16])
    for lens in ([16 * 6 + 1, 16], [16 * 7, 1], [16 * 6, 17]):
        with pytest.raises(ValueError, match=f"{8 + shared} pages of {7 + shared}"):
            s.step(*rows(s, sum(lens)), lens)
    s.hist += [16 * 6, 16]
    with pytest.raises(ValueError, match=f"{9 + shared} pages"):  # both begin a page
        s.decode(*rows(s, 2))
    s.hist[:] = prefix
    s.check_room(48)
    with pytest.raises(ValueError, match=f"{8 + shared} pages"):  # 49 replays: 4 pages each
        s.check_room(49)
    unchanged(s, state, before, prefix)


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("seed", range(6))
def test_launches_of_a_step_cover_its_rows(window, seed):
    """Too many requests, or rows, for one launch: the launches' chunks laid end to end are the
    step's, each behind the keys that come before it; a step that fits is one launch."""
    rng = np.random.default_rng(seed)
    batch = int(rng.choice([1, 3, 257, 600]))
    s, _, _ = serving(batch=batch, max_len=40000, num_pages=4, window=window, heads=(8, 4, 64))
    s.hist += rng.integers(0, 300, batch)
    lens = rng.integers(0, 2, batch) * rng.integers(0, 60, batch)
    if seed % 2 or batch < 4:
        lens[rng.integers(0, batch)] = 30000
    runs = s._runs(lens.astype(np.int32))
    if max(lens) == 30000 or np.ptp(np.flatnonzero(lens)) >= 256:
        assert len(runs) > 1
    at, done, end = 0, np.zeros(batch, int), 0
    for r0, r1, b0, b1, plan in runs:
        assert r0 == end and r1 > r0
        q, h = plan.q_lens, plan.hist_lens
        assert len(q) == len(h) == b1 - b0 and q.sum() == r1 - r0
        some = q > 0  # (no row, no history that counts)
        assert (h[some] == (s.hist + done)[b0:b1][some]).all()
        # packed order: every request before the run's first is done, the last may go on
        assert (done[:b0] == lens[:b0]).all() and (done[b0 + 1:] == 0).all()
        done[b0:b1] += q
        end = r1
    assert (done == lens).all() and end == lens.sum()
    small = np.zeros(batch, np.int32)
    small[:100:7] = 3
    fits = s._runs(small)
    assert sum(r[1] - r[0] for r in fits) == small.sum()
    if batch < 257:
        assert [r[:4] for r in fits] == [(0, small.sum(), 0, batch)]
    assert s._runs(np.zeros(batch, np.int32)) == []


def test_plans_and_captures_are_the_own_devices(monkeypatch):
    """A batch on device 1 while device 0 is current: plans for device 1's SMs, and a capture that
    device 1's stream is in (the calls themselves go by their tensors)."""
    import contextlib
    import types
    import torch
    from paged_kv_long_b200 import binding
    sms = {0: 100, 1: 37}
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "get_device_properties", lambda d: types.SimpleNamespace(
        multi_processor_count=sms[d if isinstance(d, int) else d.index]))
    assert binding._num_sms() == 100 and binding._num_sms(torch.device("cuda", 1)) == 37
    s, _, _ = serving()
    s.device, inside = torch.device("cuda", 1), []

    @contextlib.contextmanager
    def switched(device):
        inside.append(device)
        yield
        inside.pop()

    seen = []
    monkeypatch.setattr(torch.cuda, "device", switched)
    monkeypatch.setattr(torch.cuda, "CUDAGraph", lambda: seen.append(("graph", *inside)))
    monkeypatch.setattr(torch.cuda, "graph", lambda g: switched("capture"))
    monkeypatch.setattr(s, "decode", lambda q, k, v: seen.append(("decode", *inside)))
    s.capture_decode(None, None, None)
    assert seen == [("graph", s.device), ("decode", s.device, "capture")] and not inside


def test_a_prefix_without_room_is_refused():
    """Past the table row, the pages, or the rotation table (whose rows the device would skip)."""
    for kw in (dict(max_len=40, rope_rows=99, prefix_len=64), dict(prefix_len=64, num_pages=3),
               dict(prefix_len=64, rope_rows=63), dict(prefix_len=-16)):
        with pytest.raises(ValueError, match="a prefix of"):
            serving(**kw)
    assert serving(prefix_len=64, rope_rows=64, num_pages=4)[0].most_rows == 64


def test_lengths_past_32_bits_are_not_folded(no_launches):
    """2^32 + 3 rows are not 3."""
    s, state, before = serving()
    with pytest.raises(ValueError):
        s.step(*rows(s, 7), np.array([2**32 + 3, 4]))
    unchanged(s, state, before, 0)
