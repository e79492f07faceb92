"""tfd_lora where a low-rank sum is infinite or out of bf16's range, or the base cancels it: in the form
for few rows and in the one for prompts (more than 256 rows, 16-byte aligned), at ranks that fill a
tile and that do not."""
import numpy as np
import pytest
import torch

from helpers import assert_fp32_close, need_gpu, np32
from oracle.lora import lora as oracle_lora
from speculative_decoding_draft_row_gb300 import tfd

pytestmark = pytest.mark.gpu

RANKS = [8, 16, 24, 40, 64, 72, 128]


def positive(R, k, n, rank, seed):
    """Positive activations and adapters, so that an infinite activation makes every low-rank sum +inf;
    the outputs of odd number have negative rows of B."""
    g = torch.Generator().manual_seed(seed)
    x = (0.5 + torch.rand((R, k), generator=g)).bfloat16().cuda()
    a = ((0.5 + torch.rand((1, rank, k), generator=g)) / k).bfloat16().cuda()
    b = (0.5 + torch.rand((1, n, rank), generator=g)).bfloat16()
    b[:, 1::2] *= -1
    return x, a, b.cuda(), torch.zeros(R, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("R", [3, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_infinite_activation_gives_the_formulas_infinities(R, rank, dtype):
    need_gpu()
    k, n = 264, 136
    x, a, b, ids = positive(R, k, n, rank, 7)
    base = torch.ones((R, n), dtype=dtype, device="cuda")
    ref = tfd.tfd_lora(x, a, b, ids, base=base)
    x2 = x.clone()
    x2[1, 5], x2[2, k - 1] = float("inf"), -float("inf")
    y = tfd.tfd_lora(x2, a, b, ids, base=base)
    torch.cuda.synchronize()
    ex, _, _ = oracle_lora(np32(x2), np32(a), np32(b), ids.cpu().numpy(), np32(base))
    assert np.isinf(ex[1:3]).all()
    assert np.array_equal(np32(y)[1:3], ex[1:3].astype(np.float32))
    rest = [r for r in range(R) if r not in (1, 2)]
    assert torch.equal(y[rest], ref[rest]) and torch.isfinite(y[rest]).all()


@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("R", [3, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_low_rank_sum_beyond_bf16s_range(R, rank, dtype):
    """h = 2^127 (1.9921875 + 0.0078) is finite in fp32 and rounds to infinity in bf16; B brings it back.
    h and its products are exact; the fp32 sum of a row adds 3 rank rounded products of one sign: at
    most 3 rank 2^-24 relative, h's two parts 2^-16 where y is bf16, then y's own rounding."""
    need_gpu()
    k, n = 64, 72
    x = torch.zeros((R, k), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** 127 * 1.9921875, 2.0 ** 120 * 0.99609375
    a = torch.zeros((1, rank, k), dtype=torch.bfloat16, device="cuda")
    a[:, :, :2] = 1
    b = torch.full((1, n, rank), 2.0 ** -120, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(R, dtype=torch.int32, device="cuda")
    mode = tfd.OUT_F32 if dtype == torch.float32 else tfd.OUT_BF16
    y = tfd.tfd_lora(x, a, b, ids, out_mode=mode)
    torch.cuda.synchronize()
    want = rank * (2.0 ** 7 * 1.9921875 + 0.99609375)
    rel = 3 * rank * 2.0 ** -24 + (0 if dtype == torch.float32 else 2.0 ** -16 + 2.0 ** -8)
    got = np32(y).astype(np.float64)
    assert (np.abs(got - want) <= rel * want).all(), (got.min(), got.max(), want)


@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("R", [3, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_base_that_cancels_the_adapters_term(R, rank, dtype):
    """What is left shows how exactly h enters its product. One activation a rank, so h = s (a x) has
    two roundings at most and only the scale's counts (a x is exact in fp32): 2^-24 relative. The
    products with B add 3 rank + 1 fp32 sums of |B||h| at most, 2^-24 each; h's parts 2^-17 where y is
    bf16; then y's own rounding."""
    need_gpu()
    k, n = 256, 72
    g = torch.Generator().manual_seed(rank + R)
    x = (1 + torch.rand((R, k), generator=g)).bfloat16().cuda()
    a = torch.zeros((1, rank, k))
    a[0, torch.arange(rank), torch.arange(rank)] = 1 + torch.rand(rank, generator=g)
    a = a.bfloat16().cuda()
    b = torch.randn((1, n, rank), generator=g).bfloat16().cuda()
    s = torch.tensor([1.2345678], device="cuda")
    ids = torch.zeros(R, dtype=torch.int32, device="cuda")
    h = np32(s).astype(np.float64) * (np32(x).astype(np.float64) @ np32(a)[0].T.astype(np.float64))
    b64 = np32(b)[0].astype(np.float64)
    term, mag = h @ b64.T, np.abs(h) @ np.abs(b64).T
    base = torch.from_numpy(-term).to(dtype).cuda()
    y = tfd.tfd_lora(x, a, b, ids, base=base, scales=s)
    torch.cuda.synchronize()
    left = term + base.double().cpu().numpy()
    tol = mag * ((3 * rank + 3) * 2.0 ** -24 + (2.0 ** -17 if dtype == torch.bfloat16 else 0))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    err = np.abs(np32(y).astype(np.float64) - left)
    assert (err <= tol + half * (np.abs(left) + tol)).all(), (err / mag).max()


@pytest.mark.parametrize("na,named", [(64, 1), (300, 6), (4096, 3)])
@pytest.mark.parametrize("R", [40, 1100])
def test_a_large_table_of_which_few_are_named(na, named, R):
    need_gpu()
    k, n, rank = 72, 136, 16
    g = torch.Generator().manual_seed(na + R)
    x = torch.randn((R, k), generator=g).bfloat16().cuda()
    a = (torch.randn((na, rank, k), generator=g) / k ** 0.5).bfloat16().cuda()
    b = (0.3 * torch.randn((na, n, rank), generator=g)).bfloat16().cuda()
    s = (0.5 + torch.rand(na, generator=g)).cuda()
    base = torch.randn((R, n), generator=g).cuda()
    which = torch.randperm(na, generator=g)[:named]
    which[0] = na - 1
    ids = which[torch.randint(0, named, (R,), generator=g)].int()
    ids[::7] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = tfd.tfd_lora(x, a, b, ids.cuda(), base=base, scales=s, dev_status=st)
    torch.cuda.synchronize()
    ex, mag, _ = oracle_lora(np32(x), np32(a), np32(b), ids.numpy(), np32(base), np32(s))
    assert_fp32_close(np32(y), ex, mag)
    assert st.item() == 0 and torch.equal(y[::7], base[::7])
