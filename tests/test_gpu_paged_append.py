"""GPU parity of tfd_paged_append: bf16 keys held to their rounding, E4M3 codes to theirs and their scales
to fp32, values exact, everything else in the cache untouched."""
import numpy as np
import pytest
import torch

from helpers import KEY_REL, assert_bf16_rounding, need_gpu, np32
from oracle.numerics import e4m3_decode, e4m3_encode
from oracle.paged import turned
from oracle.quant import quant_fp8_row
from speculative_decoding_draft_row_gb300 import tfd
from synth import inputs

pytestmark = pytest.mark.gpu


def make_cache(pages, page, heads, dim, fmt, layout, tid=900):
    """A filled cache: tokens first ("nhd"), heads first ("hnd"), or keys and values interleaved."""
    n = pages * page * heads * dim
    if fmt == "bf16":
        flat = inputs.normal_bf16((2, n), 1.0, tid).cuda()
    else:
        flat = torch.from_numpy(np.random.default_rng(tid).integers(0, 120, (2, n), np.uint8)).cuda()
    if layout == "nhd":
        k, v = (t.view(pages, page, heads, dim) for t in flat)
    elif layout == "hnd":
        k, v = (t.view(pages, heads, page, dim).transpose(1, 2) for t in flat)
    else:
        both = flat.view(pages, page, 2, heads, dim)
        k, v = both[:, :, 0], both[:, :, 1]
    sc = [None, None] if fmt == "bf16" else [
        torch.rand((pages, heads, page), device="cuda") for _ in range(2)]
    return tfd.KvPages(k, v, *sc)


def values(t):
    """bf16 values, or codes."""
    return t.cpu().numpy() if t.dtype == torch.uint8 else np32(t)


def e4m3(x):
    return e4m3_decode(e4m3_encode(np.asarray(x, np.float64).astype(np.float32)))


def check(cache, before, k_rows, v_rows, slots, pos, **kw):
    """kw: gamma, norm, rotate, eps, base as the oracle takes them."""
    k_ex, pair = turned(k_rows, pos, **kw)
    exact = not kw.get("norm", True) and not kw.get("rotate", True)
    err = 0.0 * pair if exact else KEY_REL * pair
    page, at = slots // cache.page_size, slots % cache.page_size
    mine = slots >= 0
    page, at = page[mine], at[mine]
    rest = np.ones((cache.pages, cache.page_size), bool)
    rest[page, at] = False
    k, v = values(cache.k), values(cache.v)
    assert np.array_equal(k[rest], before[0][rest]) and np.array_equal(v[rest], before[1][rest])
    k_ex, err, v_rows = k_ex[mine], err[mine], v_rows[mine]
    if cache.k.dtype == torch.bfloat16:
        assert_bf16_rounding(k[page, at], k_ex, err, "keys")
        assert np.array_equal(v[page, at], v_rows)
        return
    ks, vs = (np32(t).transpose(0, 2, 1) for t in (cache.k_scales, cache.v_scales))
    for got, b in ((ks, before[2]), (vs, before[3])):
        assert np.array_equal(got[rest], b.transpose(0, 2, 1)[rest])
    n, heads, dim = v_rows.shape
    codes, scale = quant_fp8_row(v_rows.reshape(-1, dim).astype(np.float32))
    assert np.array_equal(v[page, at].reshape(-1, dim), codes)
    assert np.array_equal(vs[page, at].reshape(-1), scale)
    s = ks[page, at].astype(np.float64)
    amax = np.abs(k_ex).max(-1)
    # the largest magnitude within its element's error, the division within half a step
    assert (np.abs(s - amax / 448) <= err.max(-1) / 448 + 2.0 ** -24 * amax / 448 + 2.0 ** -149).all()
    x = np.divide(k_ex, s[..., None], out=np.array(k_ex), where=s[..., None] > 0)
    e = np.divide(err, s[..., None], out=np.zeros_like(err), where=s[..., None] > 0)
    assert_bf16_rounding(e4m3_decode(k[page, at]), x, e + 2.0 ** -23 * np.abs(x), "codes", rnd=e4m3)


def run(rows, heads, dim, page, fmt="bf16", layout="nhd", norm=True, rope=True, gamma=True, eps=1e-6,
        base=10000.0, skip=False, tid=910, k=None, v=None, pos=None):
    pages = -(-(rows + 5) // page) + 1
    cache = make_cache(pages, page, heads, dim, fmt, layout)
    before = [values(cache.k).copy(), values(cache.v).copy()]
    if fmt != "bf16":
        before += [np32(cache.k_scales).copy(), np32(cache.v_scales).copy()]
    g = np.random.default_rng(tid)
    kv = inputs.normal_bf16((rows, 2 * heads * dim + 8), 1.0, tid)  # rows of a wider array
    k = kv[:, :heads * dim].reshape(rows, heads, dim) if k is None else k
    v = kv[:, heads * dim:2 * heads * dim].reshape(rows, heads, dim) if v is None else v
    wide = torch.zeros((rows, 2 * heads * dim + 8), dtype=torch.bfloat16, device="cuda")
    kd, vd = (wide[:, i * heads * dim:(i + 1) * heads * dim].view(rows, heads, dim) for i in (0, 1))
    kd.copy_(k)
    vd.copy_(v)
    gm = inputs.normal_bf16((dim,), 0.5, tid + 1) if gamma else None
    slots = g.permutation(pages * page)[:rows]
    if skip:
        slots[::3] = -1
    pos = g.integers(0, 300000, rows) if pos is None else np.asarray(pos)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tfd.tfd_paged_append(kd, vd, i32(slots), i32(pos) if rope else None, cache,
                         k_gamma=None if gm is None else gm.cuda(), norm=norm, rope=rope, eps=eps,
                         rope_base=base, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(cache, before, np32(k), np32(v), slots, pos, gamma=None if gm is None else np32(gm),
          norm=norm, rotate=rope, eps=eps, base=base)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,heads,page,layout", [(1, 1, 1, "nhd"), (7, 3, 16, "hnd"),
                                                    (65, 8, 24, "both"), (130, 32, 64, "nhd"),
                                                    (33, 17, 5, "hnd"), (9, 9, 1024, "both")])
def test_layouts_heads_and_pages(rows, heads, page, layout, dim, fmt):
    need_gpu()
    run(rows, heads, dim, page, fmt, layout, skip=rows > 2)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("norm,rope,gamma", [(False, False, False), (True, False, True),
                                             (False, True, False), (True, True, False)])
def test_each_step_alone(norm, rope, gamma, fmt):
    need_gpu()
    run(20, 5, 128, 16, fmt, norm=norm, rope=rope, gamma=gamma, eps=1e-5, base=500000.0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_zero_rows_tiny_rows_and_far_positions(fmt):
    need_gpu()
    k = inputs.normal_bf16((6, 2, 128), 1.0, 930)
    v = inputs.normal_bf16((6, 2, 128), 1.0, 931)
    k[0] = 0
    v[1] = 0
    k[2] *= 2.0 ** -60
    v[3] *= 2.0 ** -120
    v[4] *= 2.0 ** 100
    run(6, 2, 128, 16, fmt, k=k, v=v, pos=[0, 1, 2 ** 31 - 1, 2 ** 30, 99999, 5], eps=1e-30)


def test_rows_like_the_absorbed_ones():
    """The same keys as tfd_absorb writes, up to a rounding: both within KEY_REL of the exact key."""
    need_gpu()
    S, n, H, D, ring = 2, 9, 4, 128, 16
    k = inputs.normal_bf16((S, n, H, D), 1.0, 940).cuda()
    v = inputs.normal_bf16((S, n, H, D), 1.0, 941).cuda()
    rings = [torch.zeros((S, ring, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p0 = torch.tensor([3, 100], dtype=torch.int32, device="cuda")
    tfd.tfd_absorb(k, v, p0, *rings)
    cache = tfd.KvPages(*(torch.zeros_like(t) for t in rings))   # a ring as a page
    pos = (p0[:, None] + torch.arange(n, device="cuda")).to(torch.int32)
    slots = (pos % ring + ring * torch.arange(S, device="cuda")[:, None]).to(torch.int32)
    tfd.tfd_paged_append(k.view(-1, H, D), v.view(-1, H, D), slots.view(-1), pos.reshape(-1), cache)
    torch.cuda.synchronize()
    assert torch.equal(cache.v, rings[1])
    ex, pair = turned(np32(k).reshape(-1, H, D), pos.view(-1).cpu().numpy())
    at = slots.view(-1).long()
    for t in (cache.k, rings[0]):
        assert_bf16_rounding(np32(t.view(-1, H, D)[at]), ex, KEY_REL * pair, "keys")


@pytest.mark.parametrize("slots,pos", [([0, 64, 1], [0, 0, 0]), ([0, -2, 1], [0, 0, 0]),
                                       ([0, 2, 1], [0, -1, 0])])
def test_bad_slots_and_positions_are_left_out(slots, pos):
    need_gpu()
    cache = make_cache(4, 16, 2, 64, "bf16", "nhd")
    before = values(cache.k).copy()
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
    tfd.tfd_paged_append(x, x, i32(slots), i32(pos), cache, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == tfd.ERR_DEVICE_DATA
    k, v = values(cache.k).reshape(64, 2, 64), values(cache.v).reshape(64, 2, 64)
    assert np.array_equal(k[2:], before.reshape(64, 2, 64)[2:])
    assert (v[0] == 1).all() and (v[1] == 1).all()


def test_a_slot_behind_2_to_the_32_elements():
    need_gpu()
    pages, page, heads, dim = 16500, 256, 16, 64          # 4.3e9 elements each
    k, v = (torch.empty((pages, page, heads, dim), dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    k[0], v[0] = 0, 0
    cache = tfd.KvPages(k, v)
    x = inputs.normal_bf16((2, heads, dim), 1.0, 950).cuda()
    last = pages * page - 1
    slots = torch.tensor([last, last - page], dtype=torch.int32, device="cuda")
    tfd.tfd_paged_append(x, x, slots, None, cache, norm=False, rope=False)
    torch.cuda.synchronize()
    assert torch.equal(k[-1, -1], x[0]) and torch.equal(v[-2, -1], x[1])
    assert not k[0].any() and not v[0].any()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,heads,page,layout", [(4000, 3, 16, "nhd"), (1300, 17, 64, "hnd"), (2500, 8, 24, "both")])
def test_prompts(rows, heads, page, layout, dim, fmt):
    """More warps' work than the GPU holds at once: items of four steps, a warp's second one loaded ahead."""
    need_gpu()
    run(rows, heads, dim, page, fmt, layout, skip=True, tid=960)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_prompts_as_they_are(fmt):
    """Without normalisation or rotation, in items of four steps: bf16 keys copied."""
    need_gpu()
    run(2500, 8, 128, 16, fmt, norm=False, rope=False, gamma=False, tid=970)
