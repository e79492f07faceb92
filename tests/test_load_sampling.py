"""A sampled pass's random numbers on their way into its float32 buffers (on the CPU)."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from speculative_decoding_draft_row_gb300.draft_pass import DraftPass

S, STEPS = 3, 2
BELOW = np.nextafter(1.0, 0.0)  # numpy's largest random number


def load(**kw):
    shapes = dict(u_draft=(STEPS, S), u_accept=(S, STEPS), u_next=(S,), temperature=(S,))
    bufs = SimpleNamespace(**{k: torch.full(v, -7.0) for k, v in shapes.items()},
                           top_k=torch.zeros(S, dtype=torch.int32))
    given = dict(u_draft=None, u_accept=None, u_next=None)
    given.update(kw)
    DraftPass.load_sampling(bufs, **given)
    return bufs


@pytest.mark.parametrize("make", [np.asarray, torch.tensor, lambda v: v],
                         ids=["numpy", "tensor", "list"])
@pytest.mark.parametrize("name,shape", [("u_draft", (STEPS, S)), ("u_accept", (S, STEPS)),
                                        ("u_next", (S,))])
def test_doubles_below_one_stay_below_one(make, name, shape):
    v = np.full(shape, 0.3)
    v.flat[0], v.flat[1], v.flat[2] = BELOW, 1 - 2.0 ** -25, 0.0
    if make is torch.tensor:
        given = torch.tensor(v, dtype=torch.float64)
    else:
        given = make(v.tolist() if make is not np.asarray else v)
    got = getattr(load(**{name: given}), name)
    assert got.dtype == torch.float32 and (got < 1).all()
    want = np.minimum(v.astype(np.float32), np.float32(1 - 2.0 ** -24))
    assert np.array_equal(got.numpy(), want)


def test_numbers_outside_stay_outside_and_floats_as_they_are():
    u = np.array([1.0, -1e-3, np.nan])
    got = load(u_next=u).u_next.numpy()
    assert got[0] == 1 and got[1] < 0 and np.isnan(got[2])
    f = np.array([1 - 2.0 ** -24, 0.0, 0.5], np.float32)
    assert np.array_equal(load(u_next=f).u_next.numpy(), f)


def test_settings_are_converted_as_before():
    got = load(temperature=np.array([0.7, 1.0, 0.0]), top_k=np.array([5, 0, 7]))
    assert np.array_equal(got.temperature.numpy(), np.array([0.7, 1.0, 0.0], np.float32))
    assert got.top_k.tolist() == [5, 0, 7] and (got.u_next == -7).all()
