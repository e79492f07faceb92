"""The strides that the Python binding passes on for the rejection accept (a fake library, CPU tensors)."""
import pytest
import torch

from speculative_decoding_draft_row_gb300 import tfd


class FakeLibrary:
    def tfd_accept_sampled(self, *args):
        self.args = args
        return 0


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLibrary()
    monkeypatch.setattr(tfd, "_lib", lib)
    monkeypatch.setattr(tfd, "_current_device", lambda: -1)  # what a CPU tensor's get_device() says
    monkeypatch.setattr(tfd, "_stream", lambda stream, dev=None: 0)
    return lib


def accept(p, q):
    S, W = q.shape[:2]
    return tfd.tfd_accept_sampled(p, q, torch.zeros((S, W), dtype=torch.int32),
                                  torch.full((S,), W, dtype=torch.int32), torch.zeros((S, W)),
                                  torch.zeros(S))


@pytest.mark.parametrize("S,W,of", [(3, 1, 4), (1, 1, 4), (1, 3, 4), (3, 1, 1)])
def test_the_first_drafts_of_a_larger_array(S, W, of, fake):
    """One draft a stream of an array that keeps more: its rows are evenly spaced, `of` rows apart."""
    n = 10
    q = torch.zeros((S, of, n))[:, :W]
    accept(torch.zeros((S, W + 1, n)), q)
    assert fake.args[1] == n                             # ldp
    assert fake.args[3] == (of * n if W == 1 and S > 1 else n)


def test_uneven_rows_are_refused(fake):
    n = 10
    with pytest.raises(ValueError):
        accept(torch.zeros((2, 3, n)), torch.zeros((2, 4, n))[:, :2])
    with pytest.raises(ValueError):
        accept(torch.zeros((2, 4, n))[:, :3], torch.zeros((2, 2, n)))
