"""The draft pass with per-stream adapters and sampled drafts: each step against the oracle applied to
the GPU's own inputs of that step, then the rejection accept, captured and replayed; and the options
that change nothing (no adapter, temperature 0) against the greedy pass."""
import numpy as np
import pytest
import torch

from helpers import assert_bf16_rounding, assert_fp32_close, gemv_bf16_err, need_gpu, np32
from oracle import gemv as og
from oracle.lora import lora as oracle_lora
from oracle.quant import quant_fp8_row
from oracle.sample import accept_sampled as oracle_accept_sampled
from oracle.sample import sample as oracle_sample
from speculative_decoding_draft_row_gb300 import tfd
from speculative_decoding_draft_row_gb300.draft_pass import DraftPass
from synth import inputs

pytestmark = pytest.mark.gpu

S, H, D, HIDDEN, INNER, VOCAB, RING, WINDOW, STEPS = 5, 2, 128, 256, 96, 2500, 40, 31, 4


def build(adapters=(), sampled=False, rank=16, na=3):
    wo = quant_fp8_row(inputs.linear(HIDDEN, H * D, 700).float().numpy())
    w2 = quant_fp8_row(inputs.linear(HIDDEN, INNER, 701).float().numpy())
    head = inputs.normal_bf16((VOCAB, HIDDEN), 0.2, 702)
    kr = inputs.normal_bf16((S * RING, H, D), 1.0, 703).reshape(S, RING, H, D)
    vr = inputs.normal_bf16((S * RING, H, D), 1.0, 704).reshape(S, RING, H, D)
    shapes = dict(wo=(HIDDEN, H * D), w2=(HIDDEN, INNER), head=(VOCAB, HIDDEN))
    ad = {}
    for i, name in enumerate(adapters):
        out, inp = shapes.get(name, (HIDDEN, HIDDEN))
        ad[name] = (inputs.normal_bf16((na, rank, inp), inp ** -0.5, 710 + i).cuda(),
                    inputs.normal_bf16((na, out, rank), 0.3, 720 + i).cuda())
    scales = torch.tensor([0.5, 1.0, 2.0], device="cuda") if adapters else None
    dp = DraftPass(torch.from_numpy(wo[0]).cuda(), torch.from_numpy(wo[1]).cuda(),
                   torch.from_numpy(w2[0]).cuda(), torch.from_numpy(w2[1]).cuda(), head.cuda(),
                   tfd.W_BF16, None, kr.clone().cuda(), vr.clone().cuda(), WINDOW, STEPS,
                   adapters=ad, adapter_scales=scales, sampled=sampled)
    qs, ks, vs = ([inputs.normal_bf16((S, H, D), 1.0, 730 + 3 * t + i) for t in range(STEPS)]
                  for i in range(3))
    us = [inputs.normal_bf16((S, INNER), 1.0, 760 + t) for t in range(STEPS)]
    resid = inputs.normal_bf16((S, HIDDEN), 1.0, 770)
    asked = np.array([4, 4, 3, 2, 4], np.int32)
    dp.load(qs, ks, vs, us, [33, 34, 35, 100, 60], resid.cuda(), asked)
    return dp, dict(wo=wo, w2=w2, head=head.float().numpy(), resid=resid)


def settings(dp):
    rng = np.random.default_rng([0, 97, 0])
    f = np.float32
    p = rng.random((S, STEPS + 1, VOCAB)).astype(f) ** 8
    p /= p.sum(-1, keepdims=True)
    dp.load_sampling(rng.random((STEPS, S), dtype=f), rng.random((S, STEPS), dtype=f) * f(0.5),
                     rng.random(S, dtype=f), temperature=np.array([0.7, 1, 0, 1.3, 1], f),
                     top_k=np.array([0, 50, 0, 20, 0]), top_p=np.array([0.9, 1, 1, 0.8, 0.95], f),
                     min_p=np.array([0, 0.02, 0, 0, 0.01], f), p_dist=p)


def test_each_step_against_the_oracle():
    need_gpu()
    dp, o = build(("wo", "w2", "head"), True)
    ids = np.array([2, -1, 0, 1, 2], np.int32)
    dp.load_adapter_ids(ids)
    settings(dp)
    sc = np32(dp.adapter_scales)

    def linear(name, codes, scales, x, before, after, what):
        # the projection rounds to bf16 and the adapter's sum again: each within half a step
        acc, mag = og.gemv_acc(codes, x, og.W_FP8_ROW, scales), \
            og.gemv_abs_scale(codes, x, og.W_FP8_ROW, scales)
        a, b = (np32(v) for v in dp.adapters[name])
        mid = before + acc
        err = gemv_bf16_err(mag, mid) + 2.0 ** -8 * (np.abs(mid) + gemv_bf16_err(mag, mid))
        ex, m2, _ = oracle_lora(x, a, b, ids, mid, sc)
        none = ids == -1
        assert_bf16_rounding(after[~none], ex[~none], (err + gemv_bf16_err(m2, ex))[~none], what)
        assert_bf16_rounding(after[none], mid[none], gemv_bf16_err(mag, mid)[none], what)

    for t in range(STEPS):
        dp.step_attn(t)
        torch.cuda.synchronize()
        before = np32(dp.resid)
        dp.step_wo()
        torch.cuda.synchronize()
        mid = np32(dp.resid)
        linear("wo", *o["wo"], np32(dp.attn), before, mid, f"step {t} wo")
        dp.step_w2(t)
        torch.cuda.synchronize()
        after = np32(dp.resid)
        linear("w2", *o["w2"], np32(dp.u[t]), mid, after, f"step {t} w2")
        dp.step_head(t)
        torch.cuda.synchronize()
        a, b = (np32(v) for v in dp.adapters["head"])
        ex, mag, _ = oracle_lora(after, a, b, ids, after @ o["head"].T.astype(np.float64), sc)
        mag += np.abs(after) @ np.abs(o["head"]).T
        assert_fp32_close(np32(dp.logits), ex, mag, f"step {t} logits")
        oi, op, margin = oracle_sample(np32(dp.logits), dp.u_draft[t].cpu().numpy(),
                                       *(v.cpu().numpy() for v in (dp.temperature, dp.top_k,
                                                                   dp.top_p, dp.min_p)))
        assert (margin > 1e-8).all()
        assert np.array_equal(dp.drafts[:, t].cpu().numpy(), oi)
        q = dp.q_dist[:, t].double().cpu().numpy()
        assert (np.abs(q - op) <= 2.5 * 2.0 ** -22 * op + 2.0 ** -44).all()
        assert np.array_equal(dp.draft_vals[:, t].cpu().numpy(),
                              dp.q_dist[:, t].cpu().numpy()[np.arange(S), oi])
    dp.enqueue_accept()
    torch.cuda.synchronize()
    k, nx, _, margin, bad = oracle_accept_sampled(*(v.cpu().numpy() for v in (
        dp.p_dist, dp.q_dist, dp.drafts, dp.n_asked, dp.u_accept, dp.u_next)))
    assert not bad.any() and (margin > 1e-8).all()
    assert np.array_equal(dp.n_kept.cpu().numpy(), k)
    assert np.array_equal(dp.next_ids.cpu().numpy(), nx)
    assert dp.status.item() == 0


@pytest.mark.parametrize("adapters,sampled", [((), True), (("wo", "w2", "head"), True),
                                              (("head",), False), (("wo",), False)])
def test_replayed_equals_eager(adapters, sampled):
    need_gpu()
    pair = [build(adapters, sampled)[0] for _ in range(2)]
    for dp in pair:
        dp.load_adapter_ids([0, 1, -1, 2, 0])
        if sampled:
            settings(dp)
    dp1, dp2 = pair
    dp1.enqueue()
    dp2.capture()
    dp1.enqueue()
    dp2.run()
    torch.cuda.synchronize()
    for name in ("drafts", "resid", "n_kept", "k_ring", "draft_vals") + \
            (("q_dist", "next_ids") if sampled else ()):
        assert torch.equal(getattr(dp1, name), getattr(dp2, name)), name
    assert dp1.status.item() == 0 and dp2.status.item() == 0


def test_no_adapter_and_temperature_zero_are_the_greedy_pass():
    need_gpu()
    ref, _ = build()
    ref.enqueue()
    for adapters, sampled in ((("wo", "w2", "head"), False), (("wo", "w2", "head"), True),
                              ((), True)):
        dp, _ = build(adapters, sampled)
        if sampled:
            z = np.zeros
            dp.load_sampling(z((STEPS, S)) + 0.99, z((S, STEPS)), z(S), temperature=z(S))
        dp.enqueue()
        torch.cuda.synchronize()
        assert torch.equal(dp.drafts, ref.drafts) and torch.equal(dp.resid, ref.resid)
        if not sampled:
            assert torch.equal(dp.draft_vals, ref.draft_vals)


def test_unknown_projection_is_refused():
    need_gpu()
    with pytest.raises(ValueError):
        build(("wq",))


def test_draw_then_accept_in_a_row():
    """Drafts drawn into the columns of an array, their distributions written beside, and the accept
    that reads both, without a wait between the calls: the same as with one."""
    need_gpu()
    S, W, n = 3, 4, 9001
    g = torch.Generator().manual_seed(3)
    lq = 3 * torch.randn((W, S, n), generator=g).cuda()
    lp = (2.5 * torch.randn((S * (W + 1), n), generator=g)).cuda()
    u = torch.rand((2 * W + 3, S), generator=g).cuda()
    up = torch.rand(S * (W + 1), generator=g).cuda()
    asked = torch.full((S,), W, dtype=torch.int32, device="cuda")

    def step(sync):
        drafts = torch.empty((S, W), dtype=torch.int32, device="cuda")
        q = torch.empty((S, W, n), device="cuda")
        for t in range(W):
            tfd.tfd_sample(lq[t], u[t], ids=drafts[:, t], probs=q[:, t])
            sync()
        p = tfd.tfd_sample(lp, up, want_probs=True)[2]
        sync()
        out = tfd.tfd_accept_sampled(p.view(S, W + 1, n), q, drafts, asked,
                                     u[W:2 * W].t().contiguous(), u[2 * W])
        sync()
        return [drafts, q, p, *out]

    want = step(torch.cuda.synchronize)
    for _ in range(5):
        got = step(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
