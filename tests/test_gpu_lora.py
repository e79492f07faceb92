"""GPU parity of tfd_lora against the oracle. Tolerance: fp32 sums within 1e-5 of the magnitude
|base| + |s| |B| (|A| |x|), as for the other products here (h as two bf16 parts adds 2^-17 = 7.7e-6
of |B| |h| at most where y is bf16); bf16 outputs to their rounding of that, plus the fp32 add."""
import numpy as np
import pytest
import torch

from helpers import (assert_bf16_rounding, assert_fp32_close, gemv_bf16_err, need_gpu, np32)
from oracle.lora import lora as oracle_lora
from speculative_decoding_draft_row_gb300 import tfd

pytestmark = pytest.mark.gpu


def make(R, k, n, rank, na, dtype=torch.bfloat16, seed=0, none=True, sort=False):
    g = torch.Generator().manual_seed(seed + R * 31 + n)
    x = torch.randn((R, k), generator=g).bfloat16().cuda()
    a = (torch.randn((na, rank, k), generator=g) / k ** 0.5).bfloat16().cuda()
    b = (0.3 * torch.randn((na, n, rank), generator=g)).bfloat16().cuda()
    ids = torch.randint(-1 if none else 0, na, (R,), generator=g).int()
    if sort:
        ids = ids.sort()[0]
    s = (0.5 + torch.rand(na, generator=g)).cuda()
    base = (2 * torch.randn((R, n), generator=g)).to(dtype).cuda()
    return x, a, b, ids.cuda(), base, s


def check(y, x, a, b, ids, base, s, what=""):
    ex, mag, _ = oracle_lora(np32(x), np32(a), np32(b), ids.cpu().numpy(),
                             None if base is None else np32(base),
                             None if s is None else np32(s))
    if y.dtype == torch.float32:
        assert_fp32_close(np32(y), ex, mag, what)
    else:
        assert_bf16_rounding(np32(y), ex, gemv_bf16_err(mag, ex), what)


@pytest.mark.parametrize("R,k,n,rank,na", [
    (1, 8, 1, 8, 1), (1, 4096, 4096, 16, 1), (1, 256, 163840, 16, 2), (2, 40, 33, 24, 3),
    (5, 264, 95, 40, 2), (16, 4096, 4096, 16, 16), (16, 11008, 512, 32, 8), (17, 512, 1000, 64, 1),
    (31, 1000, 4100, 128, 4), (33, 512, 777, 16, 1), (64, 256, 640, 32, 2), (129, 264, 257, 8, 5),
    (256, 128, 136, 48, 3), (257, 128, 136, 48, 3), (300, 256, 520, 128, 2), (700, 136, 65, 16, 90),
    (1031, 512, 384, 64, 4), (2050, 256, 512, 32, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_the_oracle(R, k, n, rank, na, dtype):
    need_gpu()
    x, a, b, ids, base, s = make(R, k, n, rank, na, dtype, sort=R % 2 == 0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = tfd.tfd_lora(x, a, b, ids, base=base, scales=s, dev_status=st)
    torch.cuda.synchronize()
    check(y, x, a, b, ids, base, s)
    assert st.item() == 0


@pytest.mark.parametrize("R", [3, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_base_in_place_and_no_scales(R, dtype):
    need_gpu()
    x, a, b, ids, base, s = make(R, 512, 520, 16, 4, dtype)
    mode = tfd.OUT_F32 if dtype == torch.float32 else tfd.OUT_BF16
    y = tfd.tfd_lora(x, a, b, ids, out_mode=mode)
    check(y, x, a, b, ids, None, None, "no base")
    assert not y[ids == -1].any()
    out = tfd.tfd_lora(x, a, b, ids, base=base, scales=s)
    z = base.clone()
    assert tfd.tfd_lora(x, a, b, ids, base=z, y=z, scales=s) is z
    assert torch.equal(z, out) and torch.equal(z[ids == -1], base[ids == -1])


@pytest.mark.parametrize("R", [6, 270])
@pytest.mark.parametrize("dtype,pad", [(torch.float32, 1), (torch.bfloat16, 3),
                                       (torch.bfloat16, 8)])
def test_strides_and_what_lies_beyond(R, dtype, pad):
    need_gpu()
    k, n = 264, 203
    x, a, b, ids, base, s = make(R, k, n, 24, 3, dtype)
    ref = tfd.tfd_lora(x, a, b, ids, base=base, scales=s)
    xw = torch.full((R, k + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    bw = torch.full((R, n + pad), 5.0, dtype=dtype, device="cuda")
    yw = torch.full((R + 1, n + 2 * pad), -7.0, dtype=dtype, device="cuda")
    xw[:, :k], bw[:, :n] = x, base
    tfd.tfd_lora(xw[:, :k], a, b, ids, base=bw[:, :n], y=yw[:R, pad:pad + n], scales=s)
    torch.cuda.synchronize()
    assert torch.equal(yw[:R, pad:pad + n], ref)
    assert (yw[R] == -7).all() and (yw[:, :pad] == -7).all() and (yw[:, pad + n:] == -7).all()


@pytest.mark.parametrize("R", [9, 400])
def test_bad_ids_and_one_rows_infinities_stay_its_own(R):
    need_gpu()
    x, a, b, ids, base, s = make(R, 256, 300, 16, 3, none=False)
    ref = tfd.tfd_lora(x, a, b, ids, base=base, scales=s)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = ids.clone()
    bad[2], bad[5] = 3, -2
    x2 = x.clone()
    x2[7, 11], x2[8, 3] = float("inf"), float("nan")
    y = tfd.tfd_lora(x2, a, b, bad, base=base, scales=s, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == tfd.ERR_DEVICE_DATA
    assert torch.equal(y[2], base[2]) and torch.equal(y[5], base[5])
    rest = [r for r in range(R) if r not in (2, 5, 7, 8)]
    assert torch.equal(y[rest], ref[rest])
    assert not torch.isfinite(y[7]).any() and torch.isnan(y[8]).all()


def test_a_row_does_not_depend_on_its_company():
    """The same rows in another order, with other adapters beside them: the same bits when the
    launch shape is the same."""
    need_gpu()
    x, a, b, ids, base, s = make(200, 512, 513, 32, 7)
    ref = tfd.tfd_lora(x, a, b, ids, base=base, scales=s)
    p = torch.randperm(200, generator=torch.Generator().manual_seed(1)).cuda()
    y = tfd.tfd_lora(x[p].contiguous(), a, b, ids[p].contiguous(), base=base[p].contiguous(),
                     scales=s)
    assert torch.equal(y, ref[p])
    all_none = torch.full_like(ids, -1)
    assert torch.equal(tfd.tfd_lora(x, a, b, all_none, base=base, scales=s), base)


def test_beside_a_projection_captured_and_replayed():
    """y = W x by tfd_head_gemv, the adapters added in place, then the top-1 of the sums."""
    need_gpu()
    R, k, n = 16, 512, 5000
    x, a, b, ids, _, s = make(R, k, n, 16, 4, torch.float32, seed=3)
    w = (torch.randn((n, k), generator=torch.Generator().manual_seed(4)) * 0.02).bfloat16().cuda()
    y = torch.zeros((R, n), device="cuda")
    ws = tfd.zeroed_workspace(tfd.tfd_topk_workspace(R, n, 1))
    vals = torch.zeros((R, 1), device="cuda")
    top = torch.zeros((R, 1), dtype=torch.int32, device="cuda")

    def step():
        tfd.tfd_head_gemv(w, tfd.W_BF16, None, x, tfd.OUT_F32, y=y)
        tfd.tfd_lora(x, a, b, ids, base=y, y=y, scales=s)
        tfd.tfd_topk(y, 1, vals=vals, ids=top, ws=ws)

    step()
    torch.cuda.synchronize()
    base = np32(x) @ np32(w).T
    ex, mag, _ = oracle_lora(np32(x), np32(a), np32(b), ids.cpu().numpy(), base, np32(s))
    mag += np.abs(np32(x)) @ np.abs(np32(w)).T
    assert_fp32_close(np32(y), ex, mag)
    first = (y.clone(), top.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    y.zero_()
    top.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first[0]) and torch.equal(top, first[1])


def test_binding_refuses_wrong_tensors():
    need_gpu()
    x, a, b, ids, base, s = make(4, 64, 64, 8, 2)
    for bad in (dict(x=x.float()), dict(a=a.float()), dict(a=a[:, :, :32]), dict(b=b[:1]),
                dict(adapter_ids=ids.long()), dict(scales=s[:1]), dict(base=base[:3]),
                dict(base=base.float(), y=base.clone()), dict(x=x.t())):
        args = dict(x=x, a=a, b=b, adapter_ids=ids, base=base, scales=s)
        args.update(bad)
        with pytest.raises(ValueError):
            tfd.tfd_lora(**args)
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tfd.TfdError):                 # y overlaps base, shifted
        tfd.tfd_lora(x, a, b, ids, base=flat[:256].view(4, 64), y=flat[8:264].view(4, 64))


@pytest.mark.parametrize("R,k,n,rank,na", [
    (300, 64, 64, 8, 1), (513, 72, 77, 16, 1), (640, 264, 200, 24, 2), (1000, 1032, 130, 40, 3),
    (777, 4096, 520, 64, 2), (1500, 512, 1000, 128, 5), (400, 128, 33, 96, 1),
    (17000, 64, 1500, 64, 1), (24600, 72, 520, 16, 2), (20500, 64, 200, 128, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sort", [True, False])
def test_prompts(R, k, n, rank, na, dtype, sort):
    """Tiles of many rows of one adapter, whole rows of y 16-byte aligned and n at any size; rows
    without an adapter; nothing beyond n is written; in place gives the same bits."""
    need_gpu()
    x, a, b, ids, base, s = make(R, k, n, rank, na, dtype, seed=5, sort=sort)
    wide = (n + 8 + 7) // 8 * 8
    bw = torch.full((R, wide), 5.0, dtype=dtype, device="cuda")
    yw = torch.full((R, wide), -7.0, dtype=dtype, device="cuda")
    bw[:, :n] = base
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = tfd.tfd_lora(x, a, b, ids, base=bw[:, :n], y=yw[:, :n], scales=s, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(y, x, a, b, ids, base, s)
    assert (yw[:, n:] == -7).all() and torch.equal(y[ids == -1], base[ids == -1])
    tfd.tfd_lora(x, a, b, ids, base=bw[:, :n], y=bw[:, :n], scales=s)
    torch.cuda.synchronize()
    assert torch.equal(bw[:, :n], y) and (bw[:, n:] == 5).all()
    z = torch.empty_like(yw)
    tfd.tfd_lora(x, a, b, ids, y=z[:, :n])
    torch.cuda.synchronize()
    check(z[:, :n], x, a, b, ids, None, None, "no base")
    assert not z[:, :n][ids == -1].any()


@pytest.mark.parametrize("R,k,n,rank,na", [(3, 128, 256, 16, 2), (16, 512, 8000, 16, 4),
                                           (1000, 256, 512, 64, 2)])
def test_calls_in_a_row(R, k, n, rank, na):
    """Each call of a run in one stream reads what the one before it wrote, eager and captured: the
    launches are placed early and must still wait for each other's results."""
    need_gpu()
    x, a, b, ids, base, s = make(R, k, n, rank, na, torch.float32, seed=11)
    s = 0.1 * s
    want = base.clone()
    for _ in range(12):
        tfd.tfd_lora(x, a, b, ids, base=want, y=want, scales=s)
        torch.cuda.synchronize()
    y = base.clone()
    torch.cuda.synchronize()
    for _ in range(12):
        tfd.tfd_lora(x, a, b, ids, base=y, y=y, scales=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    y.copy_(base)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y.copy_(base)
        for _ in range(12):
            tfd.tfd_lora(x, a, b, ids, base=y, y=y, scales=s)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
