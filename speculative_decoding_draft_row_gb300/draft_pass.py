"""The chained draft pass: per step, for all streams at once (streams are the GEMV rows), window
attention, wo and w2 residual GEMVs (FP8 row-scaled, added to bf16), the vocabulary head with its
fused top-1; after the last step, the accept-prefix count of the drafts against the round's draws.

Follows the TFE draft head page (#42): commit "pass kernels and FP8 linears" (a 5-step pass over 4
streams: attention, wo, w2 and the top-1 per step) and the update "main3x heads, pass kernels, FP8
linears" (wo and w2 in e4m3 with a row scale; a pass's steps captured once as a CUDA graph and
replayed). The steps' inputs (q, k, v, the w2 input, positions) are staged in fixed buffers so the
whole pass can be captured. Every computation is a libtfd call; this module only marshals buffers.

Three options, all off by default, serve requests of their own kind (the pages' pass is greedy, with
one set of weights and contexts of a ring):

* ``adapters`` gives wo, w2 and/or the head low-rank adapters; each stream names its own
  (``adapter_ids``, -1 for none), and its term is added to the projection's result.
* ``sampled`` draws each step's draft from the filtered distribution of its logits (temperature,
  top-k, top-p, min-p and the random numbers are fixed buffers per stream) and keeps the
  distributions; the accept is then the rejection accept against the target's distributions ``p``,
  which also draws the round's next token.
* ``paged`` keeps keys and values in pages that all streams share instead of rings, so that contexts
  can be of any length: each step plans its row's page from the positions (a pass that starts before the
  last one's end gives the pages of drafts that were turned down back), appends it and attends.
"""
import torch

from . import tfd


def unit_f32(v):
    """Random numbers in [0, 1) as float32, still below 1: a double from 1 - 2^-25 on would round to
    1, which the draws refuse. Numbers of 1 and more stay there."""
    t = v if hasattr(v, "dtype") else torch.as_tensor(v, dtype=torch.float64)
    t = torch.as_tensor(t)
    f = t.to(torch.float32)
    return f if t.dtype != torch.float64 else torch.where((t < 1) & (f >= 1), 1 - 2.0 ** -24, f)


class DraftPass:
    def __init__(self, wo_codes, wo_scales, w2_codes, w2_scales, head, head_fmt, head_scales,
                 k_ring, v_ring, window, steps, eps=1e-6, rope_base=10000.0, adapters=None,
                 adapter_scales=None, sampled=False, paged=None):
        """``adapters``: {"wo" | "w2" | "head": (a [adapters][rank][in], b [adapters][out][rank])},
        all with the same number of adapters; ``adapter_scales`` float32 [adapters] or None.
        ``paged``: dict(cache=KvPages, table [streams][max pages], held [streams], free_ids [pages],
        n_free [1]), all updated in place; k_ring and v_ring are then None, window -1 (all tokens) or
        any, and the cache may have fewer heads than the queries."""
        dev = head.device
        self.steps = steps
        self.paged = dict(paged) if paged is not None else None
        if paged is None:
            self.S, self.ring, self.H, self.D = k_ring.shape
            kv_heads = self.H
        else:
            if k_ring is not None or v_ring is not None:
                raise ValueError("paged: the rings are not used (None)")
            cache = paged["cache"]
            self.S, self.ring, self.D, kv_heads = paged["table"].shape[0], None, cache.dim, cache.heads
            self.H = wo_codes.shape[1] // self.D
        self.hidden = wo_codes.shape[0]
        self.inner = w2_codes.shape[1]
        self.window, self.eps, self.rope_base = window, eps, rope_base
        self.wo, self.wo_s, self.w2, self.w2_s = wo_codes, wo_scales, w2_codes, w2_scales
        self.head, self.head_fmt, self.head_s = head, head_fmt, head_scales
        self.k_ring, self.v_ring = k_ring, v_ring
        S, H, D = self.S, self.H, self.D
        bf = torch.bfloat16
        self.q = torch.zeros((steps, S, H, D), dtype=bf, device=dev)
        self.k = torch.zeros((steps, S, kv_heads, D), dtype=bf, device=dev)
        self.v = torch.zeros_like(self.k)
        self.u = torch.zeros((steps, S, self.inner), dtype=bf, device=dev)
        self.pos = torch.zeros((steps, S), dtype=torch.int32, device=dev)
        self.resid = torch.zeros((S, self.hidden), dtype=bf, device=dev)
        self.attn = torch.zeros((S, H * D), dtype=bf, device=dev)
        self.drafts = torch.zeros((S, steps), dtype=torch.int32, device=dev)
        self.draft_vals = torch.zeros((S, steps), dtype=torch.float32, device=dev)
        self.n_asked = torch.zeros(S, dtype=torch.int32, device=dev)
        self.draws = torch.zeros((S, steps), dtype=torch.int32, device=dev)
        self.n_kept = torch.zeros(S, dtype=torch.int32, device=dev)
        self.asked_hist = torch.zeros(steps, dtype=torch.int64, device=dev)
        self.kept_hist = torch.zeros(steps, dtype=torch.int64, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ws = tfd.zeroed_workspace(tfd.tfd_head_gemv_workspace(S, head.shape[0], 1), dev)
        if self.paged is not None:
            i32 = dict(dtype=torch.int32, device=dev)
            self.one_row = torch.ones(S, **i32)
            self.row_start = torch.zeros(S + 1, **i32)
            self.slots, self.slot_pos = torch.zeros(S, **i32), torch.zeros(S, **i32)
            self.attn_ws = tfd.zeroed_workspace(
                tfd.tfd_paged_attn_workspace(1, H, kv_heads, D), dev)
        self.graph = None
        self.adapters = dict(adapters or {})
        if set(self.adapters) - {"wo", "w2", "head"}:
            raise ValueError("adapters: wo, w2 and head can have them")
        self.adapter_scales = adapter_scales
        self.adapter_ids = torch.full((S,), -1, dtype=torch.int32, device=dev)
        self.sampled = sampled
        vocab = head.shape[0]
        f32 = dict(dtype=torch.float32, device=dev)
        self.logits = None
        if sampled or "head" in self.adapters:
            self.logits = torch.zeros((S, vocab), **f32)
            self.topk_ws = tfd.zeroed_workspace(tfd.tfd_topk_workspace(S, vocab, 1), dev)
            self.top_val = torch.zeros((S, 1), **f32)
            self.top_id = torch.zeros((S, 1), dtype=torch.int32, device=dev)
        if sampled:
            self.temperature, self.top_p = torch.ones(S, **f32), torch.ones(S, **f32)
            self.min_p = torch.zeros(S, **f32)
            self.top_k = torch.zeros(S, dtype=torch.int32, device=dev)
            self.u_draft = torch.zeros((steps, S), **f32)
            self.u_accept, self.u_next = torch.zeros((S, steps), **f32), torch.zeros(S, **f32)
            self.q_dist = torch.zeros((S, steps, vocab), **f32)
            self.p_dist = torch.zeros((S, steps + 1, vocab), **f32)
            self.next_ids = torch.zeros(S, dtype=torch.int32, device=dev)
            self.next_prob = torch.zeros(S, **f32)

    def load(self, qs, ks, vs, us, pos0, resid, n_asked=None, draws=None):
        """Copy one pass's inputs into the fixed buffers (host or device tensors)."""
        for t in range(self.steps):
            self.q[t].copy_(qs[t], non_blocking=True)
            self.k[t].copy_(ks[t], non_blocking=True)
            self.v[t].copy_(vs[t], non_blocking=True)
            self.u[t].copy_(us[t], non_blocking=True)
        p0 = torch.as_tensor(pos0, dtype=torch.int32)
        self.pos.copy_(torch.stack([p0 + t for t in range(self.steps)]), non_blocking=True)
        self.resid.copy_(resid, non_blocking=True)
        if n_asked is not None:
            self.n_asked.copy_(torch.as_tensor(n_asked, dtype=torch.int32), non_blocking=True)
        if draws is not None:
            self.draws.copy_(torch.as_tensor(draws, dtype=torch.int32), non_blocking=True)

    def load_sampling(self, u_draft, u_accept, u_next, temperature=None, top_k=None, top_p=None,
                      min_p=None, p_dist=None):
        """Copy a sampled pass's random numbers (u_draft [steps][S], u_accept [S][steps], u_next
        [S]), settings [S] and the target's distributions p_dist [S][steps + 1][vocab]."""
        given = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, p_dist=p_dist)
        for name, v in given.items():
            if v is not None:
                buf = getattr(self, name)
                buf.copy_(torch.as_tensor(v).to(buf.dtype), non_blocking=True)
        for name, v in dict(u_draft=u_draft, u_accept=u_accept, u_next=u_next).items():
            if v is not None:
                getattr(self, name).copy_(unit_f32(v), non_blocking=True)

    def load_adapter_ids(self, ids):
        """Copy each stream's adapter (-1: none)."""
        self.adapter_ids.copy_(torch.as_tensor(ids, dtype=torch.int32), non_blocking=True)

    def add_adapter(self, name, x, y):
        if name in self.adapters:
            a, b = self.adapters[name]
            tfd.tfd_lora(x, a, b, self.adapter_ids, base=y, y=y, scales=self.adapter_scales,
                         dev_status=self.status)

    def step_attn(self, t):
        if self.paged is not None:
            p, cache = self.paged, self.paged["cache"]
            tfd.tfd_page_plan(self.pos[t], self.one_row, cache.page_size, p["table"], p["held"],
                              p["free_ids"], p["n_free"], row_start=self.row_start,
                              slots=self.slots, pos=self.slot_pos, dev_status=self.status)
            tfd.tfd_paged_append(self.k[t], self.v[t], self.slots, self.slot_pos, cache,
                                 eps=self.eps, rope_base=self.rope_base, dev_status=self.status)
            tfd.tfd_paged_attn(self.q[t], cache, p["table"], self.pos[t], self.row_start, 1,
                               window=self.window, eps=self.eps, rope_base=self.rope_base,
                               out=self.attn, ws=self.attn_ws, dev_status=self.status)
            return
        tfd.tfd_window_attn(self.q[t], self.k[t], self.v[t], self.pos[t], self.k_ring, self.v_ring,
                            self.window, eps=self.eps, rope_base=self.rope_base, out=self.attn,
                            dev_status=self.status)

    def step_wo(self):
        tfd.tfd_head_gemv(self.wo, tfd.W_FP8_ROW, self.wo_s, self.attn, tfd.OUT_ADD_BF16,
                          y=self.resid)
        self.add_adapter("wo", self.attn, self.resid)

    def step_w2(self, t):
        tfd.tfd_head_gemv(self.w2, tfd.W_FP8_ROW, self.w2_s, self.u[t], tfd.OUT_ADD_BF16,
                          y=self.resid)
        self.add_adapter("w2", self.u[t], self.resid)

    def step_head(self, t):
        if self.logits is not None:
            tfd.tfd_head_gemv(self.head, self.head_fmt, self.head_s, self.resid, tfd.OUT_F32,
                              y=self.logits)
            self.add_adapter("head", self.resid, self.logits)
            if self.sampled:
                # the draft and its probability under the distribution it was drawn from
                tfd.tfd_sample(self.logits, self.u_draft[t], self.temperature, self.top_k,
                               self.top_p, self.min_p, ids=self.drafts[:, t],
                               prob=self.draft_vals[:, t], probs=self.q_dist[:, t],
                               dev_status=self.status)
            else:
                tfd.tfd_topk(self.logits, 1, vals=self.top_val, ids=self.top_id, ws=self.topk_ws)
                self.drafts[:, t:t + 1].copy_(self.top_id)
                self.draft_vals[:, t:t + 1].copy_(self.top_val)
            return
        tfd.tfd_head_gemv(self.head, self.head_fmt, self.head_s, self.resid, tfd.OUT_NONE, topk=1,
                          top_vals=self.draft_vals[:, t:t + 1], top_ids=self.drafts[:, t:t + 1],
                          ws=self.ws)

    def enqueue_step(self, t):
        self.step_attn(t)
        self.step_wo()
        self.step_w2(t)
        self.step_head(t)

    def enqueue_accept(self):
        if self.sampled:
            tfd.tfd_accept_sampled(self.p_dist, self.q_dist, self.drafts, self.n_asked,
                                   self.u_accept, self.u_next, n_kept=self.n_kept,
                                   next_ids=self.next_ids, next_prob=self.next_prob,
                                   asked_hist=self.asked_hist, kept_hist=self.kept_hist,
                                   dev_status=self.status)
            return
        tfd.tfd_accept(self.drafts, self.n_asked, self.draws, n_kept=self.n_kept,
                       asked_hist=self.asked_hist, kept_hist=self.kept_hist,
                       dev_status=self.status)

    def enqueue(self):
        for t in range(self.steps):
            self.enqueue_step(t)
        self.enqueue_accept()

    def launches(self):
        """Kernels of this library one pass launches: per step attention, wo, w2 and head, one more
        for each adapted projection, one for a draft taken from written logits, two for pages; the
        accept."""
        per = 4 + (2 if self.paged is not None else 0) + len(self.adapters) + \
            (1 if self.logits is not None else 0)
        return per * self.steps + 1

    def capture(self):
        """Capture one whole pass as a CUDA graph (replayed by run())."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.enqueue()                          # warm: builds and loads the library
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.enqueue()
        return self.graph

    def run(self):
        if self.graph is not None:
            self.graph.replay()
        else:
            self.enqueue()
