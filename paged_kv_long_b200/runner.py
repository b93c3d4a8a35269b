"""Run a whole workload (a sequence of pieces over one KV cache) through libpa on one GPU.

One step is what a prefill engine does for the chunk's attention: for every piece, plan it
(host), then pa_prefill and, when the piece is split, pa_combine on the same stream. Plans,
outputs and the workspace are made once; ``run()`` only enqueues kernels.
"""
from __future__ import annotations

import numpy as np

from . import binding
from .inputs import Inputs


def _dev_tensor(bits: np.ndarray, dtype: str, device):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    t = t.view(torch.bfloat16 if dtype == "bf16" else torch.float16)
    return t.to(device)


class DeviceWorkload:
    def __init__(self, inp: Inputs, device="cuda", paged: bool = True, splits: int | None = None,
                 policy: str = "makespan", num_sms: int | None = None):
        import torch
        wl = inp.wl
        self.wl, self.paged, self.device = wl, paged, torch.device(device)
        self.q = _dev_tensor(inp.q, wl.dtype, self.device)
        if paged:
            self.k = _dev_tensor(inp.k_pool, wl.dtype, self.device)
            self.v = _dev_tensor(inp.v_pool, wl.dtype, self.device)
            self.table = torch.from_numpy(inp.page_table).to(self.device)
        else:
            self.k = _dev_tensor(inp.k_logical, wl.dtype, self.device)
            self.v = _dev_tensor(inp.v_logical, wl.dtype, self.device)
            self.table = None
        if splits is None:
            splits = wl.splits
        self.plans = []
        for h, r in wl.pieces:
            self.plans.append(binding.plan(wl.n_q_heads, wl.n_kv_heads, wl.head_dim, wl.page_size,
                                           r, h, wl.dtype, wl.scale, splits, policy, paged,
                                           num_sms))
        self.outs = [torch.empty((r, wl.n_q_heads, wl.head_dim), dtype=torch.float32,
                                 device=self.device) for _, r in wl.pieces]
        ws_elems = max(p.ws_bytes for p in self.plans) // 4
        self.ws = torch.empty(max(ws_elems, 4), dtype=torch.float32, device=self.device)

    def piece_inputs(self, i: int):
        h, r = self.wl.pieces[i]
        off = h - self.wl.first_pos
        q = self.q[off:off + r]
        if self.paged:
            return q, self.k, self.v, self.table
        # contiguous K/V of exactly H+R rows for this piece
        return q, self.k[:h + r], self.v[:h + r], None

    def run_piece(self, i: int, stream=None):
        q, k, v, tab = self.piece_inputs(i)
        p = self.plans[i]
        binding.prefill(p, q, k, v, tab, self.outs[i], self.ws, stream)
        binding.combine(p, self.ws, self.outs[i], stream)

    def run(self, stream=None):
        for i in range(len(self.wl.pieces)):
            self.run_piece(i, stream)

    def capture(self, stream=None):
        """The whole step (every chunk's prefill and combine) captured as one CUDA graph: the
        plans, tensor maps and work-item tables are taken at capture (kernel parameters hold
        them by value), so a replay launches the same work with no host-side planning."""
        import torch
        stream = stream or torch.cuda.Stream(self.device)
        stream.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(stream):
            self.run(stream)  # once outside the capture: lazy library and kernel set-up
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self.run(torch.cuda.current_stream(self.device))
        return graph

    def outputs_host(self) -> list[np.ndarray]:
        return [o.cpu().numpy() for o in self.outs]

    def run_streamed(self, host_q, host_k, host_v, host_table, host_outs, copy_in, compute,
                     copy_out):
        """One step from pinned host memory to pinned host memory with the copies overlapped:
        the K/V pools and the page table go first (every chunk reads pages all over the pool);
        then chunk i's query rows are copied on `copy_in` while earlier chunks compute on
        `compute`, and chunk i's output goes back on `copy_out` while later chunks compute.
        host_q [rows, Hq, D], host_k / host_v like the device pools, host_table int32,
        host_outs: one pinned fp32 tensor per chunk. Enqueues only; returns the event that
        completes with the last output copy."""
        import torch
        wl = self.wl
        compute.wait_stream(copy_out)  # the previous step's outputs have left
        with torch.cuda.stream(copy_in):
            self.k.copy_(host_k, non_blocking=True)
            self.v.copy_(host_v, non_blocking=True)
            if self.table is not None:
                self.table.copy_(host_table, non_blocking=True)
        done = None
        for i, (h, r) in enumerate(wl.pieces):
            off = h - wl.first_pos
            with torch.cuda.stream(copy_in):
                self.q[off:off + r].copy_(host_q[off:off + r], non_blocking=True)
                ready = torch.cuda.Event()
                ready.record(copy_in)
            compute.wait_event(ready)
            self.run_piece(i, compute)
            out_ready = torch.cuda.Event()
            out_ready.record(compute)
            copy_out.wait_event(out_ready)
            with torch.cuda.stream(copy_out):
                host_outs[i].copy_(self.outs[i], non_blocking=True)
                done = torch.cuda.Event(enable_timing=True)
                done.record(copy_out)
        # the next step's copies into q / the pools must not overtake this step's reads
        compute_done = torch.cuda.Event()
        compute_done.record(compute)
        copy_in.wait_event(compute_done)
        return done


class PrefillRoutes:
    """The two bulk-prefill routes of a cold prompt (history 0, chunks in order), with the same
    plans' schedules and the same outputs:

    * paged (the hot path): each chunk's K/V, as the projection leaves them in a contiguous
      [R, Hkv, D] buffer, are appended to their pages (pa_kv_append), then prefill reads every
      key through the page table;
    * staged: the projection writes each chunk's K/V straight into a contiguous staging buffer
      [T, Hkv, D] at the chunk's positions, prefill reads the staged keys contiguously, and the
      chunk's rows are then published to their pages (pa_kv_publish).

    Both leave the same page pools behind. ``k_new``/``v_new`` stand for the projection's output
    (the staged route's staging buffer holds the same rows)."""

    def __init__(self, inp: Inputs, device="cuda", policy: str = "makespan",
                 num_sms: int | None = None):
        import torch
        wl = inp.wl
        assert wl.first_pos == 0, "the routes start from an empty cache"
        self.wl, self.device = wl, torch.device(device)
        self.q = _dev_tensor(inp.q, wl.dtype, self.device)
        self.kv_new = (_dev_tensor(inp.k_logical, wl.dtype, self.device),
                       _dev_tensor(inp.v_logical, wl.dtype, self.device))
        self.staged = (self.kv_new[0].clone(), self.kv_new[1].clone())
        shape = inp.k_pool.shape
        dt = self.q.dtype
        self.pools = {r: (torch.zeros(shape, dtype=dt, device=self.device),
                          torch.zeros(shape, dtype=dt, device=self.device))
                      for r in ("paged", "staged")}
        self.table = torch.from_numpy(inp.page_table).to(self.device)
        self.plans = {}
        for route, paged in (("paged", True), ("staged", False)):
            self.plans[route] = [binding.plan(wl.n_q_heads, wl.n_kv_heads, wl.head_dim,
                                              wl.page_size, r, h, wl.dtype, wl.scale, 0, policy,
                                              paged, num_sms) for h, r in wl.pieces]
        self.outs = {r: [torch.empty((n, wl.n_q_heads, wl.head_dim), dtype=torch.float32,
                                     device=self.device) for _, n in wl.pieces]
                     for r in ("paged", "staged")}
        ws = max(p.ws_bytes for ps in self.plans.values() for p in ps) // 4
        self.ws = torch.empty(max(ws, 4), dtype=torch.float32, device=self.device)

    def run_paged(self, stream=None):
        kp, vp = self.pools["paged"]
        for i, (h, r) in enumerate(self.wl.pieces):
            binding.kv_append(self.kv_new[0][h:h + r], self.kv_new[1][h:h + r], kp, vp,
                              self.table, h, stream)
            p = self.plans["paged"][i]
            binding.prefill(p, self.q[h:h + r], kp, vp, self.table, self.outs["paged"][i],
                            self.ws, stream)
            binding.combine(p, self.ws, self.outs["paged"][i], stream)

    def run_staged(self, stream=None):
        kp, vp = self.pools["staged"]
        ks, vs = self.staged
        for i, (h, r) in enumerate(self.wl.pieces):
            p = self.plans["staged"][i]
            binding.prefill(p, self.q[h:h + r], ks[:h + r], vs[:h + r], None,
                            self.outs["staged"][i], self.ws, stream)
            binding.combine(p, self.ws, self.outs["staged"][i], stream)
            binding.kv_publish(ks, vs, kp, vp, self.table, h, r, stream)


class ServingBatch:
    """One attention layer's cache for a batch of requests, advanced step by step on the current
    stream: pages, positions and slots of the step's rows (block_tables), head norms, rotation and
    the cache write (qk_rope_append), then attention — over a sliding window with sinks, over a
    prefix that all requests share (decode steps), or over every key.

    ``step`` takes ragged chunks with host lengths, ``decode`` one token per request with every
    length on the device, so that ``capture_decode`` can record it once as a CUDA graph and each
    replay is the next token's step. A shared prefix is written first (``write_prefix``); every
    request then begins after it. Pages are taken from the free list in order and not given back.

    The constructor waits for its own work (and what its stream held before), so the first step may
    run on any stream; steps on different streams are the caller's to order.
    """

    def __init__(self, n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, dtype: str,
                 batch: int, max_len: int, rope, num_pages: int, window: int = 0, n_sinks: int = 0,
                 prefix_len: int = 0, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, device="cuda", num_sms: int | None = None):
        import torch
        if window and prefix_len:
            raise ValueError("a shared prefix is not windowed: give one of window, prefix_len")
        if prefix_len % page_size:
            raise ValueError("prefix_len must be a multiple of the page size")
        self.shape = (n_q_heads, n_kv_heads, head_dim, page_size)
        self.dtype, self.batch = dtype, batch
        self.device = torch.empty(0, device=device).device  # "cuda": the one that is current now
        if self.device.type == "cuda" and num_sms is None:
            num_sms = binding._num_sms(self.device)
        self.num_sms = num_sms
        self.window, self.n_sinks, self.prefix_len = window, n_sinks, prefix_len
        self.rope, self.q_weight, self.k_weight = rope, q_weight, k_weight
        self.eps, self.interleaved = eps, interleaved
        dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        i32 = dict(dtype=torch.int32, device=self.device)
        pool = (num_pages, page_size, n_kv_heads, head_dim)
        self.k_pool = torch.zeros(pool, dtype=dt, device=self.device)
        self.v_pool = torch.zeros(pool, dtype=dt, device=self.device)
        self.free_pages = torch.arange(num_pages, **i32)
        shared = prefix_len // page_size
        self.block_table = torch.full((batch, -(-max_len // page_size)), -1, **i32)
        # a request's most rows: each needs a place in its table row and a rotation
        self.most_rows = min(self.block_table.shape[1] * page_size, rope.shape[0])
        if not 0 <= prefix_len <= self.most_rows or shared > num_pages:
            raise ValueError(f"a prefix of {prefix_len} rows: a request holds {self.most_rows} at "
                             f"most, and there are {num_pages} pages of {page_size}")
        self.prefix_table = self.free_pages[:shared]
        self.block_table[:, :shared] = self.prefix_table
        self.pages_used = torch.full((1,), shared, **i32)
        self.hist_lens = torch.full((batch,), prefix_len, **i32)
        self.ones = torch.ones(batch, **i32)
        self.hist = np.full(batch, prefix_len, dtype=np.int64)  # the host's copy
        self.q_rot = None                                       # the last step's rotated queries
        args = (*self.shape, batch)
        if window:
            self.plan = binding.window_decode_plan(*args, max_len, window, n_sinks, dtype,
                                                   num_sms=num_sms)
        elif prefix_len:
            self.plan = binding.prefix_decode_plan(*args, prefix_len, max_len, dtype,
                                                   num_sms=num_sms)
        else:
            self.plan = binding.decode_plan(*args, max_len, dtype, num_sms=num_sms)
        if self.device.type == "cuda":
            torch.cuda.current_stream(self.device).synchronize()

    def check_room(self, rows):
        """Raise ValueError unless each request b can take rows[b] more rows (one number: all of
        them that many): none may pass its table row (max_len in whole pages) or the rotation
        table, and the free list has to hold the pages. Past any of these the device skips a row and
        goes on (binding.device_error tells), so ``step`` and ``decode`` ask first; the replays of a
        captured step cannot, so ask for as many rows as there will be replays before them."""
        shared, PS = self.prefix_table.shape[0], self.shape[3]
        lens = self.hist + np.asarray(rows)
        if (lens > self.most_rows).any():
            b = int(np.argmax(lens > self.most_rows))
            raise ValueError(f"request {b} would hold {lens[b]} rows; the most is {self.most_rows}")
        need = int((-(-lens // PS)).sum()) - (self.batch - 1) * shared
        if need > self.k_pool.shape[0]:
            raise ValueError(f"the requests would hold {need} pages of {self.k_pool.shape[0]}")

    def _check_rows(self, q, k, v, rows: int):
        """The step's tensors hold its rows (checked before anything is cached)."""
        Hq, Hkv, D, _ = self.shape
        for name, t, heads in (("q", q, Hq), ("k", k, Hkv), ("v", v, Hkv)):
            want = ((rows, heads, D), self.k_pool.dtype, self.device)
            if (tuple(t.shape), t.dtype, t.device) != want:
                raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}, {t.dtype}, "
                                 f"{t.device}")

    def _cache(self, q, k, v, q_lens, rows: int):
        """Tables of the step, then the rotated queries; keys and values go into the pools."""
        t = binding.block_tables(q_lens, self.hist_lens, self.free_pages, self.pages_used,
                                 self.block_table, rows, self.shape[3], self.k_pool.shape[0])
        self.q_rot = binding.qk_rope_append(q, k, v, t.positions, t.slots, self.rope, self.k_pool,
                                            self.v_pool, self.q_weight, self.k_weight, self.eps,
                                            self.interleaved)
        self.pages_used.copy_(t.pages_used)
        self.hist_lens.copy_(t.seq_lens)
        return t

    def write_prefix(self, q, k, v):
        """The shared prefix's rows (prefix_len of them) into its pages; returns their causal
        attention [prefix_len, Hq, D] fp32."""
        import torch
        Hq, Hkv, D, PS = self.shape
        n = self.prefix_len
        at = torch.arange(n, dtype=torch.int32, device=self.device)
        slots = self.prefix_table[(at // PS).long()] * PS + at % PS
        q = binding.qk_rope_append(q, k, v, at, slots, self.rope, self.k_pool, self.v_pool,
                                   self.q_weight, self.k_weight, self.eps, self.interleaved)
        p = binding.plan(Hq, Hkv, D, PS, n, 0, self.dtype, num_sms=self.num_sms)
        return binding.prefill_combine(p, q, self.k_pool, self.v_pool, self.prefix_table)

    def step(self, q, k, v, q_lens):
        """Chunks of q_lens[b] rows (host lengths), packed in order; returns their attention
        [sum q_lens, Hq, D] (fp32 without a window). A step whose chunks or attention are refused
        has changed nothing: both are checked, and the attention planned, before its rows are
        cached."""
        import torch
        q_lens = np.asarray(q_lens, dtype=np.int64)
        if q_lens.shape != (self.batch,) or (q_lens < 0).any():
            raise ValueError("q_lens must hold a number of rows, 0 or more, for each request")
        rows = int(q_lens.sum())
        self._check_rows(q, k, v, rows)
        self.check_room(q_lens)
        q_lens = q_lens.astype(np.int32)  # below 2^31: there is room for them
        runs = self._runs(q_lens)
        lens = torch.from_numpy(q_lens).to(self.device)
        self._cache(q, k, v, lens, rows)
        self.hist += q_lens
        attend = binding.window_prefill if self.window else binding.batch_prefill
        out = torch.empty(q.shape, dtype=q.dtype if self.window else torch.float32,
                          device=self.device)
        for r0, r1, b0, b1, plan in runs:
            attend(plan, self.q_rot[r0:r1], self.k_pool, self.v_pool, self.block_table[b0:b1],
                   out[r0:r1])
        return out

    def _runs(self, q_lens):
        """The attention launches of a step: (packed rows r0 .. r1, requests b0 .. b1, their plan).
        One, unless the planner has no room for so many row blocks or requests: then the rows are
        halved until it has (every key is cached before any row attends, so a chunk may be cut)."""
        def planned(lens, hist):
            if self.window:
                return binding.window_plan(*self.shape, lens, hist, self.window, self.n_sinks,
                                           self.dtype, num_sms=self.num_sms)
            return binding.batch_plan(*self.shape, lens, hist, self.dtype, num_sms=self.num_sms)

        edge = np.concatenate([[0], np.cumsum(q_lens, dtype=np.int64)])

        def cut(r0, r1):
            b0 = int(np.searchsorted(edge, r0, "right")) - 1  # the requests with rows in between
            b1 = int(np.searchsorted(edge, r1, "left"))
            at = np.clip(edge[b0:b1 + 1], r0, r1)
            try:
                return [(r0, r1, b0, b1,
                         planned(np.diff(at), self.hist[b0:b1] + at[:-1] - edge[b0:b1]))]
            except binding.PaError as e:
                if binding.STATUS[e.status] != "PA_ERR_UNSUPPORTED" or r1 - r0 < 2:
                    raise
            mid = (r0 + r1) // 2
            return cut(r0, mid) + cut(mid, r1)

        rows = int(edge[-1])
        if rows == 0:
            return []
        try:
            return [(0, rows, 0, self.batch, planned(q_lens, self.hist))]
        except binding.PaError as e:
            if binding.STATUS[e.status] != "PA_ERR_UNSUPPORTED":
                raise
        return cut(0, rows)

    def decode(self, q, k, v):
        """One token per request; returns its attention [batch, Hq, D] (fp32 without a window or
        a shared prefix). The host's lengths advance when this runs, not when a graph replays."""
        self._check_rows(q, k, v, self.batch)
        self.check_room(1)
        t = self._cache(q, k, v, self.ones, self.batch)
        self.hist += 1
        pools = (self.k_pool, self.v_pool)
        if self.window:
            return binding.window_decode(self.plan, self.q_rot, *pools, self.block_table,
                                         t.seq_lens)
        if self.prefix_len:
            return binding.prefix_decode(self.plan, self.q_rot, *pools, self.prefix_table,
                                         self.block_table, t.seq_lens)
        return binding.decode(self.plan, self.q_rot, *pools, self.block_table, t.seq_lens)

    def capture_decode(self, q, k, v):
        """The decode step on these (static) tensors as a CUDA graph: (graph, its output). Run
        ``decode`` once before. Each replay is the next token's step: rewrite q, k and v in place,
        replay, and count it with ``replayed`` before host lengths are needed again. Replays do not
        ask for room (``check_room``)."""
        import torch
        with torch.cuda.device(self.device):  # a capture is of the current device's stream
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = self.decode(q, k, v)
        self.hist -= 1  # captured, not run
        return graph, out

    def replayed(self, steps: int = 1):
        self.hist += steps
