"""Step tables (pa_block_tables): pages for a step's new rows, the block table's new entries, every
new row's position and pool slot, on the device from the requests' lengths.

The oracle is a plain loop over the requests. Its outputs are whole numbers: GPU tests compare
every entry for equality, on ordinary steps, on steps whose lists run out, and on bad lengths.
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


def oracle_tables(q_lens, hist, free, used, table, max_rows, PS, num_pages):
    """The definition, one request and one row at a time. (slots, positions, cu, seq, used, table,
    error)"""
    table = table.copy()
    stride = table.shape[1]
    slots = np.full(max_rows, -1, np.int32)
    pos = np.full(max_rows, -1, np.int32)
    cu, seq, error = [0], [], False
    error |= used < 0 or used > len(free)
    used = min(max(used, 0), len(free))

    def take():
        nonlocal used, error
        if used >= len(free):
            error = True
            return -1
        e = int(free[used])
        used += 1
        if not 0 <= e < num_pages:
            error = True
            return -1
        return e

    for b, (r, h) in enumerate(zip(q_lens.tolist(), hist.tolist())):
        error |= r < 0 or h < 0
        r, h = max(r, 0), max(h, 0)
        seq.append(h + r)
        old, need = math.ceil(h / PS), math.ceil((h + r) / PS)
        error |= r > 0 and need > stride
        for i in range(old, min(need, stride)):
            table[b, i] = take()
        for i in range(r):
            row, p = cu[-1] + i, h + i
            if row >= max_rows:
                error = True
                break
            pos[row] = p
            e = int(table[b, p // PS]) if p // PS < stride else -1
            if 0 <= e < num_pages:
                slots[row] = e * PS + p % PS
            else:
                error = True
        cu.append(cu[-1] + r)
    return slots, pos, np.array(cu, np.int32), np.array(seq, np.int32), used, table, error


def make(seed, B, max_r, max_h, PS, extra=3, min_r=0):
    """A step over a shuffled pool: requests own the pages of their cached keys."""
    rng = np.random.default_rng(seed)
    r = rng.integers(min_r, max_r + 1, B).astype(np.int32)
    h = rng.integers(0, max_h + 1, B).astype(np.int32)
    old = -(-h // PS)
    need = -(-(h + r) // PS)
    stride = max(1, int(need.max()))
    used = 5
    num_pages = int(need.sum()) + used + extra
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, stride), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :old[b]] = ids[at:at + old[b]]
        at += old[b]
    return r, h, ids[at:].copy(), used, table, int(r.sum()), num_pages


def run(r, h, free, used, table, max_rows, PS, num_pages):
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    t = dev(table)
    out = bd.block_tables(dev(r), dev(h), dev(free), dev(np.array([used], np.int32)), t, max_rows,
                          PS, num_pages)
    st, _ = bd.device_error(reset=True)
    return [x.cpu().numpy() for x in out], t.cpu().numpy(), st


def check(case, max_rows=None, PS=16):
    r, h, free, used, table, rows, num_pages = case
    max_rows = rows if max_rows is None else max_rows
    want = oracle_tables(r, h, free, used, table, max_rows, PS, num_pages)
    got, t, st = run(r, h, free, used, table, max_rows, PS, num_pages)
    for g, w, name in zip(got, want, ("slots", "positions", "cu_q_lens", "seq_lens")):
        np.testing.assert_array_equal(g, w, err_msg=name)
    assert got[4][0] == want[4]
    np.testing.assert_array_equal(t, want[5])
    assert (st == -6) == want[6]
    return want


# ------------------------------------------------------------------------------------ CPU


def test_oracle_on_a_step_worked_by_hand():
    r, h = np.array([3, 0, 2, 17], np.int32), np.array([15, 40, 32, 0], np.int32)
    table = np.array([[9, -1, -1], [4, 5, 6], [7, 8, -1], [-1, -1, -1]], np.int32)
    free = np.array([99, 1, 2, 3, 0, 10], np.int32)
    slots, pos, cu, seq, used, t, err = oracle_tables(r, h, free, 1, table, 24, 16, 11)
    assert pos[:6].tolist() == [15, 16, 17, 32, 33, 0] and seq.tolist() == [18, 40, 34, 17]
    assert slots[:5].tolist() == [9 * 16 + 15, 16, 17, 2 * 16, 2 * 16 + 1]
    assert slots[5:22].tolist() == list(range(48, 64)) + [0]
    assert slots[22:].tolist() == [-1, -1] and cu.tolist() == [0, 3, 3, 5, 22]
    assert t.tolist() == [[9, 1, -1], [4, 5, 6], [7, 8, 2], [3, 0, -1]] and used == 5 and not err


def test_refusals():
    lib, bd = _binding().load_library(), _binding()
    p, q = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)

    def call(batch=2, q_lens=p, ps=16, pages=10, free=p, n_free=4, used=p, used_out=q, table=q,
             stride=4, rows=8, slots=q, pos=q, cu=q, seq=q):
        return bd.STATUS[lib.pa_block_tables(batch, q_lens, p, ps, pages, free, n_free, used,
                                             used_out, table, stride, rows, slots, pos, cu, seq,
                                             None)]

    bad = "PA_ERR_INVALID_ARG"
    assert call(batch=0) == bad and call(q_lens=None) == bad and call(pages=0) == bad
    assert call(free=None) == bad and call(n_free=-1) == bad and call(table=None) == bad
    assert call(stride=0) == bad and call(rows=-1) == bad and call(slots=None) == bad
    # every block reads the inputs while others write: nothing in place
    assert call(used_out=p) == call(seq=p) == call(slots=p) == call(table=p) == bad
    assert call(ps=24) == call(ps=8) == call(ps=256) == "PA_ERR_UNSUPPORTED"
    assert call(batch=4097) == "PA_ERR_UNSUPPORTED"
    assert call(pages=1 << 27) == "PA_ERR_UNSUPPORTED"  # 2^31 slots


def test_outputs_that_meet_inputs_or_one_another_are_refused():
    """Not only at equal pointers: an output that begins inside an input, or ends in one."""
    lib, bd = _binding().load_library(), _binding()
    B, F, stride, rows = 3, 9, 4, 8
    words = dict(q_lens=B, hist_lens=B, free=F, used=1, used_out=1, table=B * stride, slots=rows,
                 pos=rows, cu=B + 1, seq=B)
    apart = {name: (1 + i) << 20 for i, name in enumerate(words)}

    def call(**move):
        a = {**apart, **move}
        return bd.STATUS[lib.pa_block_tables(B, a["q_lens"], a["hist_lens"], 16, 10, a["free"], F,
                                             a["used"], a["used_out"], a["table"], stride, rows,
                                             a["slots"], a["pos"], a["cu"], a["seq"], None)]

    outs = ("used_out", "table", "slots", "pos", "cu", "seq")
    for out in outs:
        for other in words:
            if other != out:
                last = apart[other] + 4 * (words[other] - 1)  # its last word
                assert call(**{out: apart[other]}) == "PA_ERR_INVALID_ARG", (out, other)
                assert call(**{out: last}) == "PA_ERR_INVALID_ARG", (out, other)
                before = apart[other] - 4 * (words[out] - 1)  # the output's last word on its first
                assert call(**{out: before}) == "PA_ERR_INVALID_ARG", (out, other)
                if not cuda_available():  # side by side: past the checks (no device here)
                    assert call(**{out: last + 4}) == "PA_ERR_CUDA", (out, other)


def test_binding_refuses_cpu_tensors():
    import torch
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        _binding().block_tables(z, z, z, z[:1], z[None], 4, 16, 8)


# ------------------------------------------------------------------------------------ GPU


@_gpu
@pytest.mark.parametrize("B,max_r,max_h,PS", [
    (1, 1, 0, 16), (1, 1, 100, 16), (1, 5000, 77, 128), (32, 1, 3000, 16), (33, 40, 500, 64),
    (255, 3, 200, 32), (256, 70, 300, 16), (257, 5, 64, 16), (1000, 30, 100, 32),
    (4096, 2, 40, 16),
])
def test_gpu_step_tables(B, max_r, max_h, PS):
    case = make(B + PS, B, max_r, max_h, PS, min_r=1 if B == 1 else 0)
    check(case, PS=PS)
    # a captured step's room for more rows than came: -1 behind the last request
    check(case, max_rows=case[5] + 37, PS=PS)


@_gpu
def test_gpu_no_rows_at_all():
    r, h, free, used, table, _, num_pages = make(3, 6, 0, 90, 16)
    want = check((r, h, free, used, table, 0, num_pages), max_rows=9)
    assert (want[0] == -1).all() and want[4] == used
    check((r, h, free, used, table, 0, num_pages), max_rows=0)


@_gpu
@pytest.mark.parametrize("seed", range(4))
def test_gpu_free_list_runs_out(seed):
    r, h, free, used, table, rows, num_pages = make(40 + seed, 20, 60, 100, 16, min_r=1)
    need = int((-(-(h + r) // 16) - -(-h // 16)).sum())
    want = check((r, h, free[:used + need // 2], used, table, rows, num_pages))
    assert want[6] and (want[0] == -1).any() and want[4] == used + need // 2
    check((r, h, free[:0], 0, table, rows, num_pages))


@_gpu
def test_gpu_bad_lengths_pages_and_counters_are_reported():
    r, h, free, used, table, rows, num_pages = make(50, 12, 40, 100, 16, min_r=1)
    bad = table.copy()
    b = int(np.argmax(h % 16))
    bad[b, h[b] // 16] = num_pages  # a partly filled page that is no page
    want = check((r, h, free, used, bad, rows, num_pages))
    assert want[6]
    f = free.copy()
    f[used] = -3
    assert check((r, h, f, used, table, rows, num_pages))[6]
    neg = r.copy()
    neg[4] = -7
    assert check((neg, h, free, used, table, rows, num_pages))[6]
    neg = h.copy()
    neg[5] = -1
    assert check((r, neg, free, used, table, rows, num_pages))[6]
    assert check((r, h, free, -2, table, rows, num_pages))[6]
    assert check((r, h, free, len(free) + 9, table, rows, num_pages))[6]
    # fewer row entries than rows; rows past the end of a table row
    assert check((r, h, free, used, table, rows, num_pages), max_rows=rows - 5)[6]
    assert check((r, h, free, used, np.ascontiguousarray(table[:, :-2]), rows, num_pages))[6]


@_gpu
def test_gpu_lengths_near_2_to_31_stay_in_bounds():
    """Sums that no pool could hold stop at 2^31 - 1 instead of wrapping; nothing is written past
    the outputs or the table."""
    big = 2**31 - 1
    r = np.array([3, big, 5, big], np.int32)
    h = np.array([0, 10, 7, 2], np.int32)
    table = np.array([[-1, -1], [1, -1], [2, -1], [3, -1]], np.int32)
    free = np.array([4, 5, 6], np.int32)
    got, t, st = run(r, h, free, 0, table, 40, 16, 8)
    assert st == -6
    assert got[0][:3].tolist() == [64, 65, 66] and got[1][:3].tolist() == [0, 1, 2]
    assert got[1][3:40].tolist() == list(range(10, 47))
    # request 1 holds page 1 and takes one more (its row ends there): page 5
    assert got[0][3:25].tolist() == list(range(16 + 10, 32)) + list(range(80, 96))
    assert (got[0][25:] == -1).all()
    assert t.tolist() == [[4, -1], [1, 5], [2, -1], [3, 6]]
    assert got[2].tolist() == [0, 3, big - 7, big - 2, big] and got[3].tolist() == [3, big, 12, big]


@_gpu
def test_gpu_captured_step_follows_lengths_on_the_device():
    """One captured graph, replayed while lengths, table and page counter change in place: the
    counter is handed on from step to step."""
    import torch
    bd = _binding()
    PS, B, steps = 16, 5, 6
    rng = np.random.default_rng(8)
    num_pages = 200
    free = rng.permutation(num_pages).astype(np.int32)
    table, hist, used = np.full((B, 20), -1, np.int32), np.zeros(B, np.int32), 0
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    t, h_d, r_d, f_d = dev(table), dev(hist), dev(np.ones(B, np.int32)), dev(free)
    used_d = dev(np.zeros(1, np.int32))
    out = bd.block_tables(r_d, h_d, f_d, used_d, dev(table), 64, PS, num_pages)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bd.block_tables(r_d, h_d, f_d, used_d, t, 64, PS, num_pages, out=out, stream=s)
        used_d.copy_(out.pages_used)
        h_d.copy_(out.seq_lens)
    bd.device_error(reset=True)
    for i in range(steps):
        r = (rng.integers(0, 13, B) if i % 2 else np.ones(B)).astype(np.int32)
        r_d.copy_(dev(r))
        g.replay()
        torch.cuda.synchronize()
        want = oracle_tables(r, hist, free, used, table, 64, PS, num_pages)
        for got, w in zip(out, want[:4]):
            np.testing.assert_array_equal(got.cpu().numpy(), w)
        table, used, hist = want[5], want[4], want[3]
        np.testing.assert_array_equal(t.cpu().numpy(), table)
    assert bd.device_error(reset=True)[0] == 0
    del g
