"""Head norm, rotation and cache write in one pass (pa_qk_rope_append).

The oracle is the definition in 64 bits (numpy, one head at a time over all rows). An output of
the kernel is the oracle's value with fp32 arithmetic and one rounding, so it may be off by

  u |y|  +  c (|x| f + |x'| f') / rms,   u = eps(type) / 2, c = 32 * 2^-24,

f, f' the two factors (weight times cosine or sine) and x, x' the pair: the rounding, then the
fp32 part. In that part the sum of squares of D <= 256 values takes at most 8 + 5 roundings in
sequence per lane and shuffle (13 half-weighted by the root), 1/sqrt two, the factors one each,
the products and the sum three: under 32 roundings of 2^-24 each. Values below the type's normal
range round by half of the smallest step instead of u |y|.
"""
import ctypes

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


def oracle_rows(x, w, cos, sin, inter, eps):
    """fp64 (rows [T, H, D], bound of the fp32 part [T, H, D])."""
    T, H, D = x.shape
    half = cos.shape[1]
    inv = np.ones((T, H, 1))
    if w is None:
        w = np.ones(D)
    else:
        inv = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps)
    y = x * inv * w
    out, bound = y.copy(), np.abs(y)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        c, s = cos[:, None, i], sin[:, None, i]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        bound[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
        bound[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return out, bound


def make(seed, T, Hq, Hkv, D, rot, PS, dtype, norm="16", fused=False, pad=0, max_pos=4096,
         scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if fused:
        row = torch.zeros(T, (Hq + 2 * Hkv) * D + 8, dtype=dt)  # a wider row than the three need
        row[:] = (scale * rnd(T, row.shape[1])).to(dt)
        q = row[:, :Hq * D].unflatten(1, (Hq, D))
        k = row[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = row[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    else:
        row = None
        q, k, v = ((scale * rnd(T, h, D)).to(dt) for h in (Hq, Hkv, Hkv))
    pages = -(-T // PS) + 2
    slots = torch.randperm(pages * PS, generator=g)[:T].int()
    if pad:
        slots[T - pad:] = -1
    pos = torch.randint(0, max_pos, (T,), generator=g).int()
    pos[0] = max_pos - 1
    weights = [None, None]
    if norm:
        wt = torch.float32 if norm == "32" else dt
        weights = [(1 + 0.3 * rnd(D)).to(wt) for _ in range(2)]
        if norm == "q":
            weights[1] = None
    return dict(row=row, q=q, k=k, v=v, slots=slots, pos=pos, qw=weights[0], kw=weights[1],
                dt=dt, pages=pages, PS=PS, rot=rot, max_pos=max_pos)


def run_and_check(c, inter=False, eps=1e-6, in_place=False, stream=None):
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    T, Hq, D = c["q"].shape
    Hkv = c["k"].shape[1]
    if c["row"] is not None:
        row = c["row"].cuda()
        q = row[:, :Hq * D].unflatten(1, (Hq, D))
        k = row[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = row[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    else:
        q, k, v = dev(c["q"]), dev(c["k"]), dev(c["v"])
    rope = bd.rope_table(c["max_pos"], c["rot"])
    g = torch.Generator().manual_seed(5)
    before = [torch.randn(c["pages"], c["PS"], Hkv, D, generator=g).to(c["dt"]) for _ in range(2)]
    kp, vp = before[0].cuda(), before[1].cuda()
    q_out = q if in_place else torch.full((T, Hq, D), 7.0, dtype=c["dt"], device="cuda")
    got = bd.qk_rope_append(q, k, v, dev(c["pos"]), dev(c["slots"]), rope, kp, vp, dev(c["qw"]),
                            dev(c["kw"]), eps=eps, interleaved=inter, q_out=q_out, stream=stream)
    torch.cuda.synchronize()
    assert bd.device_error(reset=True)[0] == 0
    assert got is q_out
    f64 = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    table = rope.double().cpu().numpy()[c["pos"].numpy()]
    cos, sin = np.split(table, 2, axis=1)
    live = c["slots"].numpy() >= 0
    u = torch.finfo(c["dt"]).eps / 2
    tiny = float(torch.finfo(c["dt"]).smallest_normal) * u

    def close(got, want, bound):
        lim = u * np.abs(want) + 32 * 2.0**-24 * bound * (1 + u) + tiny
        err = np.abs(f64(got) - want)
        assert np.isfinite(f64(got)).all() and (err <= lim).all(), float((err - lim).max())

    want, bound = oracle_rows(f64(c["q"]), f64(c["qw"]), cos, sin, inter, eps)
    close(got.cpu()[live], want[live], bound[live])
    kept = c["q"][~live] if in_place else torch.full((int((~live).sum()), Hq, D), 7.0,
                                                     dtype=c["dt"])
    assert torch.equal(got.cpu()[~live], kept)
    want, bound = oracle_rows(f64(c["k"]), f64(c["kw"]), cos, sin, inter, eps)
    at = c["slots"].long()[live]
    flat_k, flat_v = kp.cpu().flatten(0, 1), vp.cpu().flatten(0, 1)
    close(flat_k[at], want[live], bound[live])
    assert torch.equal(flat_v[at], c["v"][live])
    rest = torch.ones(len(flat_k), dtype=torch.bool)
    rest[at] = False  # every other slot keeps its bits
    assert torch.equal(flat_k[rest], before[0].flatten(0, 1)[rest])
    assert torch.equal(flat_v[rest], before[1].flatten(0, 1)[rest])


# ------------------------------------------------------------------------------------ CPU


def test_oracle_against_complex_rotation_and_unit_rms():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 64))
    ang = rng.uniform(0, 6, (5, 16))
    for inter in (False, True):
        y, _ = oracle_rows(x, np.ones(64), np.cos(ang), np.sin(ang), inter, 0.0)
        np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)  # a rotation keeps the norm
        n = x / np.sqrt((x * x).mean(-1, keepdims=True))
        z = n[..., 0:32:2] + 1j * n[..., 1:32:2] if inter else n[..., :16] + 1j * n[..., 16:32]
        z = z * np.exp(1j * ang)[:, None, :]
        a, b = (y[..., 0:32:2], y[..., 1:32:2]) if inter else (y[..., :16], y[..., 16:32])
        np.testing.assert_allclose(a, z.real, atol=1e-12)
        np.testing.assert_allclose(b, z.imag, atol=1e-12)
        np.testing.assert_allclose(y[..., 32:], n[..., 32:], atol=1e-12)


def test_rope_table_is_cosines_then_sines_of_64_bit_angles():
    t = _binding().rope_table(1000, 32, 500.0, device="cpu").numpy()
    p, i = np.arange(1000)[:, None], np.arange(16)[None, :]
    ang = p * 500.0 ** (-2 * i / 32)
    np.testing.assert_allclose(t[:, :16], np.cos(ang), atol=2.0**-24)
    np.testing.assert_allclose(t[:, 16:], np.sin(ang), atol=2.0**-24)


def test_refusals():
    lib, bd = _binding().load_library(), _binding()
    p = ctypes.c_void_p(1 << 20)
    odd = ctypes.c_void_p((1 << 20) + 8)

    def call(Hq=4, Hkv=2, D=128, PS=16, dtype=0, rows=3, q=p, qs=512, k=p, ks=256, v=p, vs=256,
             pos=p, slots=p, rope=p, rot=128, max_pos=100, qw=p, eps=1e-6, out=p, kp=p, pages=8):
        return bd.STATUS[lib.pa_qk_rope_append(Hq, Hkv, D, PS, dtype, rows, q, qs, k, ks, v, vs,
                                               pos, slots, rope, rot, max_pos, 0, qw, p, 0, eps,
                                               out, kp, p, pages, None)]

    bad, uns = "PA_ERR_INVALID_ARG", "PA_ERR_UNSUPPORTED"
    assert call(Hq=0) == call(Hkv=0) == call(dtype=2) == call(rows=-1) == call(max_pos=0) == bad
    assert call(pages=0) == call(q=None) == call(slots=None) == call(rope=None) == bad
    assert call(q=odd) == call(qw=odd) == call(kp=odd) == call(out=odd) == bad
    assert call(qs=520) == bad                # q_out is q: its rows must be q_out's
    assert call(out=ctypes.c_void_p(1 << 21), qs=520, rows=0) == "PA_OK"
    assert call(qs=504) == call(ks=260) == call(vs=248) == bad  # short or not a multiple of 8
    assert call(eps=-1.0) == call(eps=float("nan")) == call(eps=float("inf")) == bad
    assert call(D=96) == call(PS=24) == call(rot=8) == call(rot=144) == call(rot=24) == uns
    assert call(pages=1 << 27) == uns
    assert call(Hq=1 << 30, qs=1 << 38) == call(Hkv=1 << 30, ks=1 << 38, vs=1 << 38) == uns
    assert call(rows=0) == "PA_OK"  # nothing to do


MOST_Q, MOST_KV = 65535, 32767


def test_most_heads():
    """One past the heads whose sets a warp's 32-bit shares hold is refused, and the shares of the
    accepted most cover every set once (the kernel's own arithmetic, in 32 bits)."""
    lib, bd = _binding().load_library(), _binding()
    p = ctypes.c_void_p(1 << 20)

    def call(Hq, Hkv, D):
        return bd.STATUS[lib.pa_qk_rope_append(Hq, Hkv, D, 16, 0, 0, p, Hq * D, p, Hkv * D, p,
                                               Hkv * D, p, p, p, 64, 100, 0, None, None, 0, 1e-6,
                                               p, p, p, 8, None)]

    for D in (64, 128, 256):
        assert call(MOST_Q, 1, D) == call(1, MOST_KV, D) == "PA_OK"
        assert call(MOST_Q + 1, 1, D) == call(1, MOST_KV + 1, D) == "PA_ERR_UNSUPPORTED"
        hpw = 256 // D
        for heads in (MOST_Q, 2 * MOST_KV):
            sets = -(-heads // hpw)
            for n in (1, 13, 221, sets):
                parts = -(-sets // n)
                part = np.arange(parts + 1, dtype=np.uint32)
                edge = part * np.uint32(sets) // np.uint32(parts)  # wraps as the kernel's would
                assert edge[0] == 0 and edge[-1] == sets and (np.diff(edge.astype(int)) > 0).all()


def test_rotated_queries_over_an_input_are_refused():
    """q_out may be q; inside q, or in k or v, it may not be (one fused row holds all three)."""
    lib, bd = _binding().load_library(), _binding()
    Hq, Hkv, D, T = 8, 2, 64, 5
    row = (Hq + 2 * Hkv) * D  # elements of a fused row
    f, base = ctypes.c_void_p(1 << 20), 1 << 30

    def call(out, q=base, k=base + 2 * Hq * D, v=base + 2 * (Hq + Hkv) * D, stride=row):
        return bd.STATUS[lib.pa_qk_rope_append(Hq, Hkv, D, 16, 0, T, q, stride, k, stride, v,
                                               stride, f, f, f, 64, 100, 0, None, None, 0, 1e-6,
                                               out, f, f, 8, None)]

    bad, nbytes = "PA_ERR_INVALID_ARG", 2 * T * Hq * D
    end = base + 2 * T * row
    for out in (base, base + 16, base + 2 * Hq * D, end - 16, base - nbytes + 16):
        assert call(out) == bad, out - base
    apart = dict(q=base, k=base + (1 << 24), v=base + (2 << 24), stride=Hq * D)
    last = 2 * ((T - 1) * Hq * D + Hkv * D)  # bytes that k's (and v's) rows span
    for out in (base + 16, base - 16, apart["k"], apart["k"] + last - 16, apart["v"] - nbytes + 16):
        assert call(out, **apart) == bad
    if not cuda_available():  # past the checks (no device here)
        ok = "PA_ERR_CUDA"
        assert call(end) == call(base - nbytes) == ok
        assert call(base, **apart) == call(base + nbytes, **apart) == ok
        assert call(apart["k"] + last, **apart) == call(apart["v"] - nbytes, **apart) == ok


def test_binding_refuses_cpu_tensors_and_types():
    import torch
    z = torch.zeros(2, 2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        _binding().qk_rope_append(z, z, z, None, None, None, z[None], z[None])
    with pytest.raises(TypeError):
        _binding().qk_rope_append(z.float(), z, z, None, None, None, z[None], z[None])


# ------------------------------------------------------------------------------------ GPU

CASES = [
    # T, Hq, Hkv, D, rot, PS, dtype, norm, fused, pad, interleaved
    (1, 16, 2, 256, 256, 16, "f16", "16", False, 0, False),
    (1, 1, 1, 64, 16, 16, "bf16", "32", False, 0, True),
    (32, 16, 2, 256, 256, 16, "f16", "16", True, 0, False),
    (33, 24, 4, 256, 128, 64, "bf16", "16", True, 2, True),
    (65, 32, 8, 128, 48, 32, "bf16", "32", True, 5, False),   # pairs three lanes apart
    (7, 8, 8, 128, 128, 128, "f16", "", False, 1, True),      # no norm
    (130, 5, 1, 128, 112, 16, "f16", "q", False, 0, False),   # queries normed, keys not
    (50, 32, 2, 64, 64, 128, "f16", "16", False, 0, True),
    (301, 3, 3, 64, 32, 16, "bf16", "16", True, 300, False),  # one row that is no padding
    (1000, 17, 1, 256, 80, 16, "bf16", "32", True, 0, False),
    (2048, 24, 4, 256, 64, 64, "bf16", "16", False, 0, False),
]


@_gpu
@pytest.mark.parametrize("case", CASES, ids=[f"T{c[0]}_{c[1]}q{c[2]}kv_D{c[3]}_rot{c[4]}"
                                             for c in CASES])
def test_gpu_qk_rope(case):
    *shape, inter = case
    run_and_check(make(sum(case[:5]), *shape), inter)


@_gpu
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, MOST_Q, 1, 256), (1, 1, MOST_KV, 64),
                                        (2, MOST_Q, 3, 64)])
def test_gpu_most_heads(T, Hq, Hkv, D):
    run_and_check(make(7, T, Hq, Hkv, D, 32, 16, "f16", max_pos=64))


@_gpu
def test_gpu_in_place_and_on_another_stream():
    import torch
    run_and_check(make(1, 40, 16, 2, 256, 256, 16, "f16"), in_place=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = make(2, 40, 16, 2, 256, 256, 16, "f16")
    torch.cuda.synchronize()
    run_and_check(c, stream=s)


@_gpu
@pytest.mark.parametrize("scale,eps", [(1e-4, 1e-6), (2e3, 0.0), (1.0, 10.0)])
def test_gpu_small_and_large_rows(scale, eps):
    run_and_check(make(3, 21, 8, 2, 128, 128, 16, "f16", scale=scale), eps=eps)


@_gpu
def test_gpu_infinite_value_stays_in_its_pair():
    """Without a norm, an infinity reaches its own pair only, and none past rot_dim."""
    import torch
    bd = _binding()
    D, rot = 64, 32
    for inter in (False, True):
        x = torch.ones(1, 1, D, dtype=torch.bfloat16, device="cuda")
        x[0, 0, 2] = float("inf")
        x[0, 0, 40] = float("inf")
        kp = torch.zeros(1, 16, 1, D, dtype=torch.bfloat16, device="cuda")
        vp = torch.zeros_like(kp)
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        q = bd.qk_rope_append(x, x, x, i32(1), i32(0), bd.rope_table(4, rot), kp, vp,
                              interleaved=inter)
        pair = {2, 3} if inter else {2, 18}
        for y in (q[0, 0], kp[0, 0, 0]):
            gone = {i for i in range(D) if not torch.isfinite(y[i])}
            assert gone == pair | {40} and y[40] == float("inf")
        assert torch.equal(vp[0, 0], x[0])


@_gpu
@pytest.mark.parametrize("what", ["slot", "position", "negative position"])
def test_gpu_bad_rows_are_skipped_and_reported(what):
    import torch
    bd = _binding()
    bd.device_error(reset=True)
    c = make(4, 9, 4, 2, 64, 64, 16, "f16")
    slots, pos = c["slots"].clone(), c["pos"].clone()
    if what == "slot":
        slots[3] = c["pages"] * 16
    else:
        pos[3] = c["max_pos"] if what == "position" else -1
    kp = torch.zeros(c["pages"], 16, 2, 64, dtype=c["dt"], device="cuda")
    vp, q_out = torch.zeros_like(kp), torch.zeros_like(c["q"]).cuda()
    bd.qk_rope_append(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), pos.cuda(), slots.cuda(),
                      bd.rope_table(c["max_pos"], 64), kp, vp, q_out=q_out)
    assert bd.device_error(reset=True)[0] == -6
    rows = q_out.abs().sum((1, 2)).cpu() > 0
    assert rows.tolist() == [i != 3 for i in range(9)]
    written = (vp.abs().sum((2, 3)) > 0).flatten().cpu().nonzero().flatten()
    assert set(written.tolist()) == {int(s) for i, s in enumerate(c["slots"]) if i != 3}


@_gpu
def test_gpu_binding_refusals():
    import torch
    bd = _binding()
    c = make(6, 4, 4, 2, 64, 64, 16, "f16")
    q, k, v = c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
    kp = torch.zeros(c["pages"], 16, 2, 64, dtype=c["dt"], device="cuda")
    vp, rope = torch.zeros_like(kp), bd.rope_table(c["max_pos"], 64)
    args = dict(q=q, k=k, v=v, positions=c["pos"].cuda(), slots=c["slots"].cuda(), rope=rope,
                k_pool=kp, v_pool=vp)
    for name, value in [("k", k[:3]), ("k", k.bfloat16()), ("v", v.transpose(1, 2)),
                        ("positions", c["pos"].long().cuda()), ("slots", c["slots"][:3].cuda()),
                        ("rope", rope.half()), ("v_pool", vp[:1]), ("q", q.flatten(1)),
                        ("q_weight", torch.ones(32, device="cuda")),
                        ("q_weight", torch.ones(64, device="cuda").bfloat16())]:
        with pytest.raises((TypeError, ValueError)):
            bd.qk_rope_append(**{**args, name: value})
