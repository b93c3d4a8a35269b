"""Cases and plain forms of the serving-step operators: tables and slot maps of a step, the
queries' and keys' norm and rotation with the cache write, attention over a sliding window with a
few first keys that stay visible, and a decode step whose requests share a long prefix.

``run`` computes an operator in elementary torch operations (32-bit arithmetic, rounded once),
or, where ``own`` is true, by the calls a user of the package makes. ``exact`` computes the same
outputs in 64 bits, one sequence or one head type at a time.
"""
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------- cases


def listed():
    return [
        # One decode step of a serving batch: 32 requests, one new token each (latency).
        dict(name="tables decode 32", op="tables", batch=32, min_rows=1, max_rows=1, min_hist=1024,
             max_hist=32768, page_size=16, lens=1),
        # The largest step: over 100K new rows of 1,000 requests.
        dict(name="tables prefill 1000", op="tables", batch=1000, min_rows=1, max_rows=300,
             min_hist=0, max_hist=32768, page_size=64, lens=3),
        # A decode step's queries, keys and values of 32 requests (16 query heads, 2 KV heads).
        dict(name="rope decode 32", op="rope", rows=32, pad=0, n_q_heads=16, n_kv_heads=2,
             head_dim=256, rot_dim=256, page_size=16, dtype="f16", norm=True, interleaved=False,
             fused=True, max_pos=32768),
        # An odd step of single tokens and chunks with padded rows, half of each head rotated.
        dict(name="rope odd 1003", op="rope", rows=1003, pad=21, n_q_heads=32, n_kv_heads=8,
             head_dim=128, rot_dim=64, page_size=32, dtype="bf16", norm=True, interleaved=True,
             fused=True, max_pos=131072),
        # A whole 32,768-token prompt in one call.
        dict(name="rope prompt 32768", op="rope", rows=32768, pad=0, n_q_heads=16, n_kv_heads=2,
             head_dim=256, rot_dim=256, page_size=16, dtype="f16", norm=True, interleaved=False,
             fused=True, max_pos=32768),
        # One request's next token at 32K keys (latency).
        dict(name="window decode 1", op="decode", batch=1, min_len=32768, max_len=32768,
             window=4096, sinks=4, n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=16,
             dtype="f16", lens=4),
        # The serving batch: 32 requests of 1K to 32K keys.
        dict(name="window decode 32", op="decode", batch=32, min_len=1024, max_len=32768,
             window=4096, sinks=4, n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=16,
             dtype="f16", lens=5),
        # A padded batch (some rows hold no request) with an odd window and short sequences.
        dict(name="window decode 100", op="decode", batch=100, min_len=0, max_len=5000,
             window=1001, sinks=20, n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=32,
             dtype="bf16", lens=6),
        # The last 2,048-row chunk of a 32K prompt.
        dict(name="window chunk 2048", op="prefill", batch=1, min_rows=2048, max_rows=2048,
             min_hist=30720, max_hist=30720, window=4096, sinks=4, n_q_heads=16, n_kv_heads=2,
             head_dim=256, page_size=16, dtype="f16", lens=7),
        # Ragged chunks of several requests in one step.
        dict(name="window batch 6", op="prefill", batch=6, min_rows=1, max_rows=300, min_hist=0,
             max_hist=9000, window=1001, sinks=20, n_q_heads=32, n_kv_heads=8, head_dim=128,
             page_size=32, dtype="bf16", lens=8),
        # 32 requests with one 32K-token prompt in common, each some hundred tokens past it.
        dict(name="prefix decode 32", op="prefix", batch=32, pad=0, prefix=32768, max_own=1024,
             n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=16, dtype="f16", lens=9),
        # A small padded batch on a short common prompt.
        dict(name="prefix decode 7", op="prefix", batch=7, pad=2, prefix=2080, max_own=300,
             n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=32, dtype="bf16", lens=10),
    ]


def _log_int(rng, lo, hi):
    """A whole number of lo..hi, spread evenly over its logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random() + rng.random())))


HEADS = ((16, 2, 256), (24, 4, 256), (8, 1, 256), (32, 8, 128), (16, 2, 128), (8, 8, 128),
         (32, 2, 64), (4, 4, 64))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(("tables", "rope", "decode", "prefill", "prefix"))
    seed = rng.randrange(1 << 30)
    ps = rng.choice((16, 32, 64, 128))
    if op == "tables":
        batch = _log_int(rng, 1, 1000)
        lo = rng.choice((0, 1))
        return dict(op=op, batch=batch, min_rows=lo, max_rows=_log_int(rng, 1, 290),
                    min_hist=0, max_hist=_log_int(rng, 100, 32768), page_size=ps, lens=seed)
    hq, hkv, d = rng.choice(HEADS)
    dtype = rng.choice(("f16", "bf16"))
    if op == "rope":
        most = 32768 if hq * d <= 4096 else 8192
        rows = _log_int(rng, 1, most)
        return dict(op=op, rows=rows, pad=min(rng.choice((0, 0, 1, 17)), rows - 1), n_q_heads=hq,
                    n_kv_heads=hkv, head_dim=d, rot_dim=16 * rng.randint(1, d // 16),
                    page_size=ps, dtype=dtype, norm=rng.random() < 0.75,
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5, max_pos=131072)
    if op == "prefix":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, pad=rng.randint(0, batch // 4),
                    prefix=ps * _log_int(rng, 1, 32768 // ps), max_own=_log_int(rng, 1, 1024),
                    n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=ps, dtype=dtype, lens=seed)
    window, sinks = _log_int(rng, 1, 4096), rng.choice((0, 1, 4, 20, 128, 200))
    shape = dict(window=window, sinks=sinks, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                 page_size=ps, dtype=dtype, lens=seed)
    if op == "decode":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 16, 32768)
        return dict(op=op, batch=batch, min_len=rng.choice((0, 1, hi // 2)), max_len=hi, **shape)
    batch = rng.choice((1, 1, 2, 5, 9))
    rows = _log_int(rng, 2, 1400 if batch == 1 else 150)
    return dict(op=op, batch=batch, min_rows=rng.choice((0, 1)) if batch > 1 else rows,
                max_rows=rows, min_hist=0, max_hist=_log_int(rng, 1, 32768), **shape)


def _lens(case):
    """(new rows, cached keys) of each sequence, by the case alone."""
    rng = random.Random(case["lens"])
    if case["op"] == "prefix":  # the keys past the prefix count as new rows here
        own_keys = [rng.randint(0, case["max_own"]) for _ in range(case["batch"])]
        return own_keys, [case["prefix"]] * case["batch"]
    if case["op"] == "decode":
        lens = [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"])]
        lens[0] = max(lens[0], 1)
        return [min(1, n) for n in lens], [max(0, n - 1) for n in lens]
    rows = [rng.randint(case["min_rows"], case["max_rows"]) for _ in range(case["batch"])]
    rows[0] = max(rows[0], 1)
    hist = [rng.randint(case["min_hist"], case["max_hist"]) for _ in range(case["batch"])]
    return rows, hist


def _visible(case):
    """Per sequence: first and last row's key ranges as (sink keys, first key of the earliest
    row's window, keys), and the visible (query, key) pairs of all rows."""
    out, pairs = [], 0
    w, s = case["window"], case["sinks"]
    for r, h in zip(*_lens(case)):
        total = h + r if r else 0
        lo = max(0, h + 1 - w)
        out.append((min(s, total), lo, total))
        for p in range(h, h + r):
            first = max(0, p + 1 - w)
            pairs += p + 1 - first + min(s, first)
    return out, pairs


def work(case):
    if case["op"] == "tables":
        rows, hist = _lens(case)
        ps = case["page_size"]
        new = sum(-(-(r + h) // ps) - -(-h // ps) for r, h in zip(rows, hist))
        old = sum(1 for r, h in zip(rows, hist) if r and h % ps)  # a page that is partly filled
        # lengths and outputs per request, slot and position per row, new pages read and written
        return {"bytes": 4 * (4 * len(rows) + 2 * sum(rows) + 2 * new + old + 3), "flops": 0}
    hq, hkv, d = case["n_q_heads"], case["n_kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        n = case["rows"] - case["pad"]
        heads = 2 * (hq + 2 * hkv) * d * 2  # each head's 16-bit row in and out
        angles = 4 * case["rot_dim"] * min(n, case["max_pos"])
        return {"bytes": n * (heads + 8) + angles, "flops": n * (hq + hkv) * d * 6}
    if case["op"] == "prefix":  # the prefix is read once for all
        lens = _lens(case)[0][case["pad"]:]
        keys = case["prefix"] + sum(lens)
        pairs = case["prefix"] * len(lens) + sum(lens)
        return {"bytes": 2 * keys * hkv * d * 2 + 2 * case["batch"] * hq * d * 2,
                "flops": 4 * d * hq * pairs}
    seen, pairs = _visible(case)
    keys = 0
    for sinks, lo, total in seen:
        keys += total - lo + min(sinks, lo)
    rows = sum(_lens(case)[0])
    return {"bytes": 2 * keys * hkv * d * 2 + 2 * rows * hq * d * 2,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, gen)
    if case["op"] == "rope":
        return _prepare_rope(case, gen)
    if case["op"] == "prefix":
        return _prepare_prefix(case, gen)
    return _prepare_window(case, gen)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_tables(case, gen):
    rows, hist = _lens(case)
    ps = case["page_size"]
    old = [-(-h // ps) for h in hist]
    new = [-(-(h + r) // ps) - o for r, h, o in zip(rows, hist, old)]
    stride = max(o + n for o, n in zip(old, new))
    used = 7  # pages of the free list that earlier steps took
    pages = sum(old) + sum(new) + used + 5
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(rows), stride), -1, dtype=torch.int32, device="cuda")
    owned = torch.arange(stride, device="cuda")[None, :] < _ints(old)[:, None]
    table[owned] = ids[:sum(old)]
    return dict(case=case, q_lens=_ints(rows), hist_lens=_ints(hist),
                free_pages=ids[sum(old):].contiguous(), pages_used=_ints([used]), table=table,
                rows=sum(rows), num_pages=pages)


def _prepare_rope(case, gen):
    n, hq, hkv, d = case["rows"], case["n_q_heads"], case["n_kv_heads"], case["head_dim"]
    dt, ps = DTYPES[case["dtype"]], case["page_size"]
    dev = "cuda"
    if case["fused"]:  # the rows of one projection: queries, keys and values side by side
        qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=gen, device=dev).to(dt)
        q, k, v = (x.view(n, -1, d) for x in qkv.split((hq * d, hkv * d, hkv * d), dim=1))
    else:
        q, k, v = (torch.randn(n, h, d, generator=gen, device=dev).to(dt) for h in (hq, hkv, hkv))
    # positions of runs of up to 512 rows that begin anywhere below max_pos
    first = torch.randint(0, case["max_pos"] - min(512, case["max_pos"] - 1), (n // 512 + 1,),
                          generator=gen, device=dev)
    at = torch.arange(n, device=dev)
    positions = (first[at // 512] + at % 512).to(torch.int32)
    num_pages = -(-n // ps) + 3
    pages = torch.randperm(num_pages, generator=gen, device=dev)
    slots = (pages[at // ps] * ps + at % ps).to(torch.int32)
    if case["pad"]:
        slots[n - case["pad"]:] = -1
    freq = 10000.0 ** (-torch.arange(0, case["rot_dim"], 2, device=dev, dtype=torch.float64)
                       / case["rot_dim"])
    angle = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * freq
    rope = torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)
    weights = [None, None]
    if case["norm"]:
        weights = [(1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(dt) for _ in range(2)]
    pools = [torch.zeros(num_pages, ps, hkv, d, dtype=dt, device=dev) for _ in range(2)]
    return dict(case=case, q=q, k=k, v=v, positions=positions, slots=slots, rope=rope,
                q_weight=weights[0], k_weight=weights[1], k_pool=pools[0], v_pool=pools[1],
                q_out=torch.zeros(n, hq, d, dtype=dt, device=dev))


def _prepare_window(case, gen):
    rows, hist = _lens(case)
    hq, hkv, d, ps = (case[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "page_size"))
    dt, dev = DTYPES[case["dtype"]], "cuda"
    seen, _ = _visible(case)
    stride = max(1, max(-(-t // ps) for _, _, t in seen))
    sinks, lo, total = (torch.tensor(x, device=dev)[:, None] for x in zip(*seen))
    page = torch.arange(stride, device=dev)[None, :] * ps
    # pages behind every window and past the sinks were given back to the pool
    held = (page < total) & ((page < sinks) | (page + ps > lo))
    num_pages = int(held.sum()) + 2
    table = torch.full((len(rows), stride), -1, dtype=torch.int32, device=dev)
    table[held] = torch.randperm(num_pages, generator=gen,
                                 device=dev)[:num_pages - 2].to(torch.int32)
    pools = [torch.randn(num_pages, ps, hkv, d, generator=gen, device=dev).to(dt)
             for _ in range(2)]
    n = len(rows) if case["op"] == "decode" else sum(rows)
    q = torch.randn(n, hq, d, generator=gen, device=dev).to(dt)
    state = dict(case=case, q=q, k_pool=pools[0], v_pool=pools[1], table=table,
                 q_lens=_ints(rows), hist_lens=_ints(hist), seq_lens=_ints([x[2] for x in seen]),
                 max_rows=max(rows), max_keys=max(t - l for _, l, t in seen))
    if own:  # the plan of the step, which every layer of a model shares
        from paged_kv_long_b200 import binding as pa
        if case["op"] == "decode":
            state["plan"] = pa.window_decode_plan(
                hq, hkv, d, ps, len(rows), max(1, max(x[2] for x in seen)), case["window"],
                case["sinks"], dtype=case["dtype"])
        else:
            state["plan"] = pa.window_plan(hq, hkv, d, ps, rows, hist, case["window"],
                                           case["sinks"], dtype=case["dtype"])
    return state


def _prepare_prefix(case, gen):
    own_keys, _ = _lens(case)
    hq, hkv, d, ps = (case[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "page_size"))
    dt, dev, batch, common = DTYPES[case["dtype"]], "cuda", case["batch"], case["prefix"] // ps
    lens = [case["prefix"] + n if b >= case["pad"] else 0 for b, n in enumerate(own_keys)]
    stride = max(1, -(-max(lens) // ps))
    # every request's table row begins with the same pages; rows without a request hold none
    page = torch.arange(stride, device=dev)[None, :]
    seq = torch.tensor(lens, device=dev)[:, None]
    table = torch.where((page < common) & (seq > 0), page, -1).to(torch.int32)
    mine = (page >= common) & (page * ps < seq)
    num_pages = common + int(mine.sum()) + 2
    table[mine] = torch.arange(common, num_pages - 2, device=dev, dtype=torch.int32)
    ids = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.where(table >= 0, ids[table.long().clamp(min=0)], table)
    pools = [torch.randn(num_pages, ps, hkv, d, generator=gen, device=dev).to(dt)
             for _ in range(2)]
    state = dict(case=case, q=torch.randn(batch, hq, d, generator=gen, device=dev).to(dt),
                 k_pool=pools[0], v_pool=pools[1], table=table, prefix_table=ids[:common].clone(),
                 seq_lens=_ints(lens), own_keys=max(lens) - case["prefix"] if any(lens) else 0)
    if own:  # the plan of the step, which every layer of a model shares
        from paged_kv_long_b200 import binding as pa
        state["plan"] = pa.prefix_decode_plan(hq, hkv, d, ps, batch, case["prefix"],
                                              max(1, max(lens)), dtype=case["dtype"])
    return state


# --------------------------------------------------------------------------------------- run


def run(s):
    op = s["case"]["op"]
    if op == "tables":
        return _own_tables(s) if own else _plain_tables(s)
    if op == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    if op == "prefix":
        return _own_prefix(s) if own else _plain_prefix(s)
    return _own_window(s) if own else _plain_window(s)


def _own_tables(s):
    from paged_kv_long_b200 import binding as pa
    t = pa.block_tables(s["q_lens"], s["hist_lens"], s["free_pages"], s["pages_used"], s["table"],
                        s["rows"], s["case"]["page_size"], s["num_pages"])
    return dict(slots=t.slots, positions=t.positions, cu_q_lens=t.cu_q_lens, seq_lens=t.seq_lens,
                pages_used=t.pages_used, table=s["table"])


def _own_rope(s):
    from paged_kv_long_b200 import binding as pa
    q = pa.qk_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"],
                          s["k_pool"], s["v_pool"], q_weight=s["q_weight"],
                          k_weight=s["k_weight"], eps=1e-6, interleaved=s["case"]["interleaved"],
                          q_out=s["q_out"])
    return dict(q=q, k_pool=s["k_pool"], v_pool=s["v_pool"])


def _own_window(s):
    from paged_kv_long_b200 import binding as pa
    if s["case"]["op"] == "decode":
        return pa.window_decode(s["plan"], s["q"], s["k_pool"], s["v_pool"], s["table"],
                                s["seq_lens"])
    return pa.window_prefill(s["plan"], s["q"], s["k_pool"], s["v_pool"], s["table"])


def _own_prefix(s):
    from paged_kv_long_b200 import binding as pa
    return pa.prefix_decode(s["plan"], s["q"], s["k_pool"], s["v_pool"], s["prefix_table"],
                            s["table"], s["seq_lens"])


def _plain_tables(s):
    ps = s["case"]["page_size"]
    rows, hist, table = s["q_lens"].long(), s["hist_lens"].long(), s["table"]
    cu = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    old = (hist + ps - 1) // ps
    new = (hist + rows + ps - 1) // ps - old
    taken = torch.cat([new.new_zeros(1), new.cumsum(0)])
    # the pages of the step: request b takes the next new[b] of the free list
    page = torch.arange(table.shape[1], device=table.device)[None, :]
    nth = page - old[:, None]
    fresh = (nth >= 0) & (nth < new[:, None])
    at = (s["pages_used"].long() + taken[:-1, None] + nth).clamp(0, s["free_pages"].numel() - 1)
    table.copy_(torch.where(fresh, s["free_pages"][at], table))
    b = torch.repeat_interleave(torch.arange(rows.numel(), device=rows.device), rows,
                                output_size=s["rows"])
    pos = hist[b] + torch.arange(s["rows"], device=rows.device) - cu[b]
    slots = table[b, pos // ps].long() * ps + pos % ps
    return dict(slots=slots.int(), positions=pos.int(), cu_q_lens=cu.int(),
                seq_lens=(hist + rows).int(), pages_used=(s["pages_used"] + taken[-1:]).int(),
                table=table)


def _plain_rotate(x, weight, cos, sin, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    half = cos.shape[-1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([rot, rest], dim=-1)


def _plain_rope(s):
    case = s["case"]
    n = case["rows"] - case["pad"]  # rows behind the last request are left as they were
    dt = s["q"].dtype
    cos, sin = s["rope"][s["positions"][:n].long()].chunk(2, dim=-1)
    inter = case["interleaved"]
    s["q_out"][:n] = _plain_rotate(s["q"][:n], s["q_weight"], cos, sin, inter).to(dt)
    slots = s["slots"][:n].long()
    s["k_pool"].flatten(0, 1)[slots] = _plain_rotate(s["k"][:n], s["k_weight"], cos, sin,
                                                     inter).to(dt)
    s["v_pool"].flatten(0, 1)[slots] = s["v"][:n]
    return dict(q=s["q_out"], k_pool=s["k_pool"], v_pool=s["v_pool"])


def _plain_window(s):
    case = s["case"]
    hq, hkv, d, ps = (case[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "page_size"))
    w, g, dev = case["window"], hq // hkv, s["q"].device
    rows, hist = s["q_lens"].long(), s["hist_lens"].long()
    total = s["seq_lens"].long()
    # every sequence's keys: the sinks, then the union of its rows' windows
    lo = (hist + 1 - w).clamp(min=0)[:, None]
    sink = torch.arange(case["sinks"], device=dev)[None, :].expand(len(rows), -1)
    near = lo + torch.arange(s["max_keys"], device=dev)[None, :]
    key = torch.cat([sink, near], dim=1)
    there = (key < total[:, None]) & torch.cat([sink < lo, near >= 0], dim=1)
    page = s["table"].gather(1, (key // ps).clamp(max=s["table"].shape[1] - 1)).long()
    slot = page.clamp(min=0) * ps + key % ps
    k, v = (torch.where(there[:, :, None, None], p.flatten(0, 1)[slot], 0).float()
            .permute(0, 2, 1, 3) for p in (s["k_pool"], s["v_pool"]))  # [B, Hkv, keys, D]
    # the rows, padded to the longest chunk; in a decode step row b belongs to sequence b
    r = torch.arange(s["max_rows"], device=dev)[None, :]
    first = (torch.arange(len(rows), device=dev) if case["op"] == "decode"
             else rows.cumsum(0) - rows)[:, None]
    live = r < rows[:, None]
    q = s["q"][(first + r).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(len(rows), -1, hkv, g, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (q @ k.transpose(-1, -2)) * d ** -0.5  # [B, Hkv, rows * G, keys]
    pos = hist[:, None] + r
    sees = (key[:, None, :] <= pos[:, :, None]) & there[:, None, :] & (
        (key[:, None, :] > pos[:, :, None] - w) | (key[:, None, :] < case["sinks"]))
    sees = sees.repeat_interleave(g, dim=1)[:, None]
    score = torch.where(sees, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    out = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.view(len(rows), hkv, -1, g, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    if case["op"] == "decode":
        return torch.where(live[:, :, None, None], out, 0)[:, 0].to(s["q"].dtype)
    return out[live].to(s["q"].dtype)


def _plain_prefix(s):
    case = s["case"]
    hq, hkv, d, ps = (case[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "page_size"))
    b, g, common, dev = case["batch"], hq // hkv, case["prefix"], s["q"].device
    seq = s["seq_lens"].long()[:, None]
    q = s["q"].float().view(b, hkv, g, d)
    # the common keys, once for all requests: [Hkv, prefix, D]
    kc, vc = (p[s["prefix_table"].long()].flatten(0, 1).float().transpose(0, 1)
              for p in (s["k_pool"], s["v_pool"]))
    qc = q.transpose(0, 1).flatten(1, 2)  # [Hkv, B * G, D]
    shared = (qc @ kc.transpose(1, 2)).view(hkv, b, g, common).transpose(0, 1)
    # each request's own keys: [B, Hkv, keys, D]
    key = common + torch.arange(s["own_keys"], device=dev)[None, :].expand(b, -1)
    there = key < seq
    page = s["table"].gather(1, (key // ps).clamp(max=s["table"].shape[1] - 1)).long()
    slot = page.clamp(min=0) * ps + key % ps
    ko, vo = (torch.where(there[:, :, None, None], p.flatten(0, 1)[slot], 0).float()
              .transpose(1, 2) for p in (s["k_pool"], s["v_pool"]))
    score = torch.cat([shared, q @ ko.transpose(2, 3)], dim=-1) * d ** -0.5
    sees = torch.cat([(seq > 0).expand(b, common), there], dim=1)[:, None, None, :]
    score = torch.where(sees, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    out = (p[..., :common].transpose(0, 1).flatten(1, 2) @ vc).view(hkv, b, g, d).transpose(0, 1)
    out = (out + p[..., common:] @ vo) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.flatten(1, 2).to(s["q"].dtype)


# ------------------------------------------------------------------------------------- exact


def exact(case, seed):
    if case["op"] == "tables":  # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(s)
    return _exact_rope(s) if case["op"] == "rope" else _exact_window(s)


def _exact_rope(s):
    case, n = s["case"], s["case"]["rows"] - s["case"]["pad"]
    half, inter = case["rot_dim"] // 2, case["interleaved"]
    table = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None, :]

    def turned(x, weight):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + 1e-6)
            y = y * weight.double()
        y = y.clone()
        if inter:
            z = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * turn
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    q = turned(s["q"], s["q_weight"])
    q[n:] = 0
    pools = []
    for rows, pool in ((turned(s["k"], s["k_weight"]), s["k_pool"]), (s["v"].double(),
                                                                     s["v_pool"])):
        out = torch.zeros(pool.shape, dtype=torch.float64, device=pool.device)
        out.view(-1, *pool.shape[2:]).index_copy_(0, s["slots"][:n].long(), rows[:n])
        pools.append(out)
    return dict(q=q, k_pool=pools[0], v_pool=pools[1])


def _exact_window(s):
    case = s["case"]
    hq, hkv, d, ps = (case[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "page_size"))
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    at = 0
    for b, (rows, hist) in enumerate(zip(*_lens(case))):
        row0, at = (b, at) if case["op"] == "decode" else (at, at + rows)
        if not rows:
            continue
        key = torch.arange(hist + rows, device=dev)
        key = key[(key < case["sinks"]) | (key > hist - case["window"])]
        slot = s["table"][b].long()[key // ps] * ps + key % ps
        k, v = (p.view(-1, hkv, d)[slot].double() for p in (s["k_pool"], s["v_pool"]))
        pos = torch.arange(hist, hist + rows, device=dev)[:, None]
        hide = (key > pos) | ((key <= pos - case["window"]) & (key >= case["sinks"]))
        for h in range(hq):
            x = s["q"][row0:row0 + rows, h].double() @ k[:, h // (hq // hkv)].T / d ** 0.5
            weight = torch.softmax(x.masked_fill(hide, -torch.inf), dim=-1)
            out[row0:row0 + rows, h] = weight @ v[:, h // (hq // hkv)]
    return out


def _exact_prefix(s):
    case = s["case"]
    hkv, d, ps = (case[x] for x in ("n_kv_heads", "head_dim", "page_size"))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["seq_lens"].tolist()):
        if not n:
            continue
        key = torch.arange(n, device=out.device)
        slot = s["table"][b].long()[key // ps] * ps + key % ps
        k, v = (p.view(-1, hkv, d)[slot].double() for p in (s["k_pool"], s["v_pool"]))
        for h in range(hkv):
            mine = slice(h * case["n_q_heads"] // hkv, (h + 1) * case["n_q_heads"] // hkv)
            x = s["q"][b, mine].double() @ k[:, h].T / d ** 0.5
            out[b, mine] = torch.softmax(x, dim=-1) @ v[:, h]
    return out
