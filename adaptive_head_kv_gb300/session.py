"""A small driver over the C ABI that owns the device buffers (through torch)
for one batch of heads: profile -> plan -> compact -> decode steps.

It only allocates and passes pointers; every step runs in the library's
kernels.
"""
from __future__ import annotations

import json

import torch

from . import fastgen as fg


def make_params(B, L, H, n, d, dtype, T, r_l, r_f, scale=0.0, Hkv=0) -> fg.Params:
    code = {"bf16": fg.FG_BF16, "fp32": fg.FG_FP32, torch.bfloat16: fg.FG_BF16,
            torch.float32: fg.FG_FP32}[dtype]
    return fg.Params(B, L, H, n, d, code, T, r_l, r_f, scale, Hkv)


GUARD_BYTES = 4096
GUARD_FILL = 0x5A


class FastGenSession:
    """Owns the buffers of one batch of heads.  With guard=True every buffer
    the library writes gets GUARD_BYTES of canary bytes on both sides, and
    check_guards() reports any that changed (a bounds check for tests).
    refresh_period > 0 selects the opt-in refresh of the frequent sets every
    that many generation steps (fastgen_decode_attn_refresh)."""

    def __init__(self, params: fg.Params, special_ids, punct_ids, max_new_tokens: int,
                 device="cuda", stream=None, guard=False, refresh_period=0):
        self.p = params
        self.refresh_period = int(refresh_period)
        self.state = None
        self._ids = None
        self.device = torch.device(device)
        self.stream = stream
        self.max_new = int(max_new_tokens)
        self.guard = guard
        self._guards = []
        G, n = params.B * params.L * params.H, params.n
        self.G = G
        self.Gkv = params.B * params.L * (params.Hkv or params.H)  # caches (key/value heads)
        self.tdtype = torch.bfloat16 if params.dtype == fg.FG_BF16 else torch.float32
        dev = self.device
        self.special = torch.as_tensor(special_ids, dtype=torch.int32, device=dev)
        self.punct = torch.as_tensor(punct_ids, dtype=torch.int32, device=dev)
        E = self._empty
        self.policy = E((G,), torch.int8)
        self.mass = E((G, 5), torch.float32)
        self.cost = E((G, 5), torch.int32)
        self.colsum = E((G, n), torch.float32)
        self.keep = E((G, n), torch.uint8)
        self.kept = E((G,), torch.int32)
        self.ws = E((fg.fastgen_profile_workspace_bytes(params),), torch.uint8)
        self.plan = E((fg.fastgen_plan_bytes(params, self.max_new),), torch.uint8)
        self.dev_err = E((1,), torch.int32)
        self.dev_err.zero_()
        self.out = E((G, params.d), self.tdtype)
        self.info = None
        self.K_pool = self.V_pool = self.pos_pool = None
        self.dws = None

    def profile(self, Q, K, token_ids):
        self._ids = token_ids
        fg.fastgen_profile(self.p, Q, K, token_ids, self.special, self.punct, self.policy,
                           self.mass, self.cost, self.colsum, self.keep, self.kept, self.ws,
                           self.dev_err, self.stream)

    def profile_attn(self, Q, K, V, token_ids, out):
        """profile() plus the prompt attention output out [G, n, d] = A V."""
        fg.fastgen_profile_attn(self.p, Q, K, V, token_ids, self.special, self.punct,
                                self.policy, self.mass, self.cost, self.colsum, self.keep,
                                self.kept, out, self.ws, self.dev_err, self.stream)
        return out

    def profile_with_policy(self, Q, K, token_ids, policy_map):
        """Phase 1 under a saved head-policy map (one FG_POLICY_* per query
        head, host or device): keep codes of each head's saved entry on this
        prompt; only heads whose entry contains C_frequent are scored."""
        self.policy.copy_(torch.as_tensor(policy_map, dtype=torch.int8).reshape(-1),
                          non_blocking=True)
        fg.fastgen_profile_with_policy(self.p, Q, K, token_ids, self.special, self.punct,
                                       self.policy, self.colsum, self.keep, self.kept, self.ws,
                                       self.dev_err, self.stream)

    def prefill_with_policy(self, Q, K, V, token_ids, policy_map):
        Q, K = self._ready(Q, K)
        self.profile_with_policy(Q, K, token_ids, policy_map)
        self.compact(K, V)

    def _ready(self, Q, K):
        """A prompt's queries and keys as they are profiled and cached."""
        return Q, K

    def compact(self, K, V):
        if self.pos_pool is not None:  # pools from an earlier prompt: plan and gather in one call
            done, self.info = fg.fastgen_plan_compact(self.p, self.policy, self.keep, self.max_new,
                                                      self.plan, K, V, self.K_pool, self.V_pool,
                                                      self.pos_pool, self.stream)
            self._size_decode_workspace()
            if done:
                self._init_refresh()
                return
        else:
            self.info = fg.fastgen_compact_plan(self.p, self.policy, self.keep, self.max_new,
                                                self.plan, self.stream)
        rows = int(self.info.pool_rows)
        if self.pos_pool is None or self.pos_pool.numel() < rows:
            d = self.p.d
            self.K_pool = self._empty((rows, d), self.tdtype)
            self.V_pool = self._empty((rows, d), self.tdtype)
            self.pos_pool = self._empty((rows,), torch.int32)
        self._size_decode_workspace()
        fg.fastgen_compact(self.p, K, V, self.keep, self.plan, self.info, self.K_pool,
                           self.V_pool, self.pos_pool, self.stream)
        self._init_refresh()

    def _init_refresh(self):
        """Accumulated scores and frequent slots of the new caches (refresh mode)."""
        if self.refresh_period <= 0:
            return
        need = fg.fastgen_refresh_state_bytes(self.p, self.info)
        if self.state is None or self.state.numel() < need:
            self.state = self._empty((max(need, 256),), torch.uint8)
        fg.fastgen_refresh_init(self.p, self.plan, self.info, self.pos_pool, self.colsum,
                                self._ids, self.special, self.punct, self.state, self.stream)

    def _size_decode_workspace(self):
        need = fg.fastgen_decode_workspace_bytes(self.p, self.info)
        if self.dws is None or self.dws.numel() < need:
            self.dws = self._empty((max(need, 256),), torch.uint8)

    def prefill(self, Q, K, V, token_ids):
        Q, K = self._ready(Q, K)
        self.profile(Q, K, token_ids)
        self.compact(K, V)

    def prefill_host(self, hQ, hK, hV, htoken_ids, Q, K, V, token_ids):
        """prefill() from pinned host tensors: Q (with the ids), K and V are
        copied in that order on one copy stream, and profiling starts as soon
        as Q and K are on the device, so the V copy overlaps it.  One copy at
        a time keeps the host link at its full rate: on the GB300 machines used,
        three concurrent 21 GB copies shared about half of it (103 GB/s in
        all against 211 GB/s for one)."""
        main = torch.cuda.current_stream(self.device)
        if not hasattr(self, "_copy_stream"):
            self._copy_stream = torch.cuda.Stream(self.device)
        cs = self._copy_stream
        cs.wait_stream(main)  # the buffers are free once earlier work is done
        qk_ready, v_ready = torch.cuda.Event(), torch.cuda.Event()
        with torch.cuda.stream(cs):
            token_ids.copy_(htoken_ids, non_blocking=True)
            Q.copy_(hQ, non_blocking=True)
            K.copy_(hK, non_blocking=True)
            qk_ready.record(cs)
            V.copy_(hV, non_blocking=True)
            v_ready.record(cs)
        main.wait_event(qk_ready)
        Q, K = self._ready(Q, K)
        self.profile(Q, K, token_ids)
        main.wait_event(v_ready)
        self.compact(K, V)

    def decode(self, q, k_new, v_new, new_ids, pos, out=None):
        """One generation step: q [G, d] per query head, k_new/v_new [Gkv, d]
        per key/value head, new_ids [B]; returns out [G, d]."""
        out = self.out if out is None else out
        if self.refresh_period > 0:
            fg.fastgen_decode_attn_refresh(self.p, self.plan, self.info, self.K_pool, self.V_pool,
                                           self.pos_pool, q, k_new, v_new, new_ids, self.special,
                                           self.punct, pos, self.refresh_period, out, self.state,
                                           self.dws, self.dev_err, self.stream)
            return out
        fg.fastgen_decode_attn(self.p, self.plan, self.info, self.K_pool, self.V_pool,
                               self.pos_pool, q, k_new, v_new, new_ids, self.special, self.punct,
                               pos, out, self.dws, self.dev_err, self.stream)
        return out

    def row_scores(self):
        """Accumulated score of every pool row (refresh mode; host copy)."""
        rows = int(self.info.pool_rows)
        return self.state[: rows * 4].view(torch.float32).cpu()

    def capture_decode(self, q, k, v, new_ids, pos0):
        """Captures len(q) consecutive decode calls (inputs q [steps, G, d],
        k, v [steps, Gkv, d] and new_ids [steps, B] on the device, positions pos0,
        pos0 + 1, ...) as one CUDA graph; returns (graph, outs [steps, G, d]).
        Replaying it runs those steps on the session's current caches.  The
        plan and pools must not be reallocated between replays."""
        steps = q.shape[0]
        outs = self._empty((steps, self.G, self.p.d), self.tdtype)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for st in range(steps):
                self.decode(q[st], k[st], v[st], new_ids[st], pos0 + st, out=outs[st])
        return graph, outs

    def _empty(self, shape, dtype):
        if not self.guard:
            return torch.empty(shape, dtype=dtype, device=self.device)
        nbytes = int(torch.Size(shape).numel()) * torch.empty((), dtype=dtype).element_size()
        body = (nbytes + 255) // 256 * 256
        raw = torch.full((GUARD_BYTES + body + GUARD_BYTES,), GUARD_FILL, dtype=torch.uint8,
                         device=self.device)
        view = raw[GUARD_BYTES:GUARD_BYTES + nbytes].view(dtype).view(shape)
        self._guards.append((raw, body))
        return view

    def check_guards(self):
        """Number of guard buffers whose canaries changed (0 when none did)."""
        bad = 0
        for raw, body in self._guards:
            lo = raw[:GUARD_BYTES]
            hi = raw[GUARD_BYTES + body:]
            if bool((lo != GUARD_FILL).any()) or bool((hi != GUARD_FILL).any()):
                bad += 1
        return bad

    def descriptors(self):
        """Host copy of the per-cache descriptors (for inspection and tests)."""
        import ctypes

        raw = self.plan[: self.Gkv * ctypes.sizeof(fg.HeadDesc)].cpu().numpy().tobytes()
        return (fg.HeadDesc * self.Gkv).from_buffer_copy(raw)


class PagedSession(FastGenSession):
    """A session whose caches are paged 8-bit ones: the same calls, with rows
    of e4m3 codes in pages that a cache takes when it grows, several tokens
    at a time (append), and a position per sequence.

    rope (fastgen.Rope): the prefill calls, append and decode then take queries
    and keys as projected and rotate them at their positions (profile, compact
    and profile_attn take them rotated); None: they are taken as they are.
    in_place: the prefill calls rotate the caller's Q and K themselves; without
    it the session keeps a second pair of their size.
    pages: size of the page pool; None gives the worst case (every cache
    growing by max_new_tokens rows).  A smaller pool that runs out is reported
    as FG_ECAPACITY by fastgen_read_error(dev_err).

    Captured append and decode calls keep the workspace they were captured
    with.  A later prompt that wants more pages than there are gets a new cache
    (self.cache); replaying calls captured on the one before then does nothing
    and is reported as FG_EINVAL."""

    def __init__(self, params: fg.Params, special_ids, punct_ids, max_new_tokens: int,
                 device="cuda", stream=None, guard=False, rope=None, pages=None, in_place=False):
        super().__init__(params, special_ids, punct_ids, max_new_tokens, device, stream, guard)
        self.rope, self.pages, self.in_place = rope, pages, in_place
        self.cache = self._new_cache()
        self.aws = None
        self._held = []  # what captured calls may still use
        self._rotated = None

    def _new_cache(self):
        Gkv, E, i32 = self.Gkv, self._empty, torch.int32
        return fg.PagedCache(
            self.p, None, None, None, None,
            E((fg.fastgen_paged_table_len(self.p, self.max_new),), i32), E((Gkv, 6), i32),
            E((Gkv,), i32), E((1,), i32))

    def _on_stream(self):
        """Context in which torch works on the session's device and stream."""
        s = self.stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, self.device)
        return torch.cuda.stream(torch.cuda.current_stream(self.device) if s is None else s)

    def _hold(self, ws):
        """Keeps the workspace and the cache of a call that is being captured."""
        if self.stream is None and self.device.index in (None, torch.cuda.current_device()):
            captured = torch.cuda.is_current_stream_capturing()
        else:
            with self._on_stream():
                captured = torch.cuda.is_current_stream_capturing()
        if captured:
            self._held += [x for x in (ws, self.cache) if all(x is not y for y in self._held)]

    def _grown(self, ws, need):
        """A workspace of `need` bytes: ws, or a larger one."""
        if ws is not None and ws.numel() >= need:
            return ws
        with self._on_stream():
            self._release(ws)
            return self._empty((max(need, 256 if ws is None else ws.numel() * 3 // 2),),
                               torch.uint8)

    def _release(self, *buffers):
        """Buffers about to be dropped: their memory is free once the session's calls so far are
        through (call on the session's stream)."""
        for x in buffers:
            if x is not None:
                x.record_stream(torch.cuda.current_stream(x.device))

    def rotate(self, Q, K, pos=None, out=None):
        """Q and K rotated at pos [B, n] (None: 0 .. n-1) into `out` (a pair;
        None: buffers of the session, reused by the next call)."""
        if out is None:
            if self._rotated is None:
                with self._on_stream():
                    self._rotated = (torch.empty_like(Q), torch.empty_like(K))
            out = self._rotated
        fg.fastgen_rope(self.p, Q, K, pos, self.rope, out[0], out[1], self.stream)
        return out

    def _ready(self, Q, K):
        if self.rope is None:
            return Q, K
        return self.rotate(Q, K, out=(Q, K) if self.in_place else None)

    def compact(self, K, V):
        """Plans the paged caches of the profiled prompt and codes its kept
        rows; K as it was profiled (rotated)."""
        self.info = fg.fastgen_paged_plan(self.p, self.policy, self.keep, self.max_new, self.cache,
                                          self.stream)
        want = self.info.max_pages if self.pages is None else max(self.pages, self.info.pages)
        if self.cache.exps is None or self.cache.c.n_pages < want:
            if any(x is self.cache for x in self._held):
                self._retire()
            rows, d, c = want * fg.FG_PAGE_ROWS, self.p.d, self.cache
            with self._on_stream():
                self._release(c.k_pages, c.v_pages, c.exps, c.pos)
                c.set_pages(self._empty((rows, d), torch.uint8),
                            self._empty((rows, d), torch.uint8), self._empty((want, 8), torch.int8),
                            self._empty((rows,), torch.int32))
        self._size_decode_workspace()
        fg.fastgen_compact_q8(self.p, K, V, self.keep, self.cache, self.dev_err, self.stream)

    def _retire(self):
        """A cache of new buffers for the planned prompt: captured calls hold the addresses of the
        page pool that is about to be replaced.  The old cache's descriptors and work list then
        allow nothing, so that a replay touches no page and reports FG_EINVAL."""
        old = self.cache
        with self._on_stream():
            self.cache = self._new_cache()
        self.info = fg.fastgen_paged_plan(self.p, self.policy, self.keep, self.max_new, self.cache,
                                          self.stream)
        with self._on_stream():
            self._release(old.k_pages, old.v_pages, old.exps, old.pos)
            old.sched.zero_()
            old.rows.zero_()
            old.caches.copy_(torch.tensor([fg.FG_POLICY_FULL, -1, 0, 0, 0, 0], dtype=torch.int32,
                                          device=old.caches.device).expand(self.Gkv, 6))
        old.k_pages = old.v_pages = old.exps = old.pos = None

    def reschedule(self):
        """Splits the decode work by the caches' present sizes (worth a call every
        few hundred tokens of a long generation: a full cache's later rows all
        go to one thread block.  32 caches with 8192 rows since the prompt: 77 us
        a step, after this call 14.  It waits for the GPU, 30 us; steps captured
        before it are void: they are reported as FG_EINVAL and do nothing)."""
        self.cache.schedule(self.p, self.stream)
        self._size_decode_workspace()

    def _size_decode_workspace(self):
        self.dws = self._grown(self.dws, fg.fastgen_decode_q8_workspace_bytes(self.p, self.cache))

    def _positions(self, pos):
        """pos, or that position for every sequence, made on the session's stream."""
        if not isinstance(pos, int):
            return pos
        with self._on_stream():
            return torch.full((self.p.B,), pos, dtype=torch.int32, device=self.device)

    def descriptors(self):
        """Host copy of the paged descriptors."""
        import ctypes

        raw = self.cache.caches.cpu().numpy().tobytes()
        assert len(raw) == self.Gkv * ctypes.sizeof(fg.PagedDesc)
        return (fg.PagedDesc * self.Gkv).from_buffer_copy(raw)

    def append(self, k_new, v_new, new_ids, pos, n_new=None):
        """Appends m tokens to every cache: k_new, v_new [Gkv, m, d], new_ids
        [B, m], pos [B] (or an int) the first new position of each sequence (< 0:
        left out), n_new [B] the tokens of each (None: m)."""
        m = new_ids.numel() // self.p.B
        self.aws = self._grown(self.aws, fg.fastgen_append_q8_workspace_bytes(self.p, m))
        self._hold(self.aws)
        fg.fastgen_append_q8(self.p, self.cache, k_new, v_new, new_ids, n_new, self.special,
                             self.punct, self._positions(pos), self.rope, self.aws, self.dev_err,
                             self.stream)

    def decode(self, q, k_new, v_new, new_ids, pos, out=None):
        """One generation step at pos [B] (or an int): the tokens appended, then
        q [G, d] attending; k_new = v_new = None attends only."""
        out = self.out if out is None else out
        self._hold(self.dws)
        fg.fastgen_decode_attn_q8(self.p, self.cache, q, k_new, v_new, new_ids, self.special,
                                  self.punct, self._positions(pos), self.rope, out, self.dws,
                                  self.dev_err, self.stream)
        return out


POLICY_MAP_FORMAT = "fastgen-head-policy-map"


def save_policy_map(path, params: fg.Params, policy) -> None:
    """Writes a profiled policy (one FG_POLICY_* per query head, flat index
    g = (b*L + l)*H + h) to a JSON file with the shape it was profiled on."""
    pol = [int(x) for x in torch.as_tensor(policy).reshape(-1).cpu().tolist()]
    G = params.B * params.L * params.H
    if len(pol) != G:
        raise ValueError(f"policy has {len(pol)} entries, the shape has {G} heads")
    doc = dict(format=POLICY_MAP_FORMAT, version=1, B=params.B, L=params.L, H=params.H,
               Hkv=params.Hkv or params.H, n=params.n, T=float(params.T),
               r_l=float(params.r_l), r_f=float(params.r_f),
               policies=list(fg.POLICY_NAMES), policy=pol)
    with open(path, "w") as f:
        json.dump(doc, f)


def load_policy_map(path, params: fg.Params) -> torch.Tensor:
    """Reads a map written by save_policy_map for the same B, L, H and Hkv
    (the prompt length may differ); returns int8 [G] on the CPU."""
    with open(path) as f:
        doc = json.load(f)
    if doc.get("format") != POLICY_MAP_FORMAT or doc.get("version") != 1:
        raise ValueError("not a head-policy map")
    want = dict(B=params.B, L=params.L, H=params.H, Hkv=params.Hkv or params.H)
    got = {k: doc.get(k) for k in want}
    if got != want:
        raise ValueError(f"map was saved for {got}, the shape is {want}")
    pol = doc["policy"]
    if len(pol) != params.B * params.L * params.H or any(not 0 <= p <= 4 for p in pol):
        raise ValueError("malformed policy list")
    return torch.tensor(pol, dtype=torch.int8)

