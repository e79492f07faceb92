"""Host-side argument checks of the sampled-drafting calls: refused before the GPU is touched."""
import pytest

from speculative_decoding_draft_row_gb300 import tfd

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced by refused calls


def sample_call(**kw):
    a = dict(x=FAKE, fmt=1, rows=2, n=100, ld=100, t=None, k=None, p=None, mp=None, u=FAKE, m=None,
             ids=FAKE, prob=None, ldt=0, probs=None, ldp=0, st=None, stream=None)
    a.update(kw)
    return tfd.library().tfd_sample(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), 1), (dict(u=None), 1), (dict(ids=None), 1), (dict(fmt=2), 1), (dict(fmt=-1), 1),
    (dict(rows=0), 1), (dict(n=0), 1), (dict(ld=99), 1), (dict(ldt=-1), 1), (dict(x=FAKE + 2), 1),
    (dict(t=FAKE + 2), 1), (dict(ids=FAKE + 1), 1), (dict(probs=FAKE * 2, ldp=99), 1),
    (dict(probs=FAKE * 2 + 2, ldp=100), 1), (dict(probs=FAKE + 16, ldp=100), 1),
    (dict(n=(1 << 20) + 1, ld=1 << 21), 2), (dict(rows=(1 << 24) + 1), 2),
])
def test_sample_refusals(bad, code):
    assert sample_call(**bad) == code


@pytest.mark.parametrize("out", ["ids", "prob", "probs"])
@pytest.mark.parametrize("inp", ["x", "t", "k", "p", "mp", "u", "m"])
def test_sample_overlaps(out, inp):
    """An output that shares its last bytes with an input."""
    a = {name: FAKE * (i + 1) for i, name in
         enumerate(["x", "t", "k", "p", "mp", "u", "m", "ids", "prob", "probs"])}
    size = dict(ids=8 * 4, prob=8 * 4, probs=(7 * 120 + 100) * 4)[out]
    a[inp] = a[out] + size - 4 if inp != "x" else a[out] + size - 16
    assert sample_call(rows=8, ldp=120, **a) == 1


def accept_sampled_call(**kw):
    a = dict(p=FAKE, ldp=100, q=FAKE, ldq=100, n=100, nq=100, m=None, d=FAKE, na=FAKE, u=FAKE,
             un=FAKE, streams=4, win=5, nk=FAKE, nx=FAKE, pr=None, ah=None, kh=None, st=None,
             stream=None)
    a.update(kw)
    return tfd.library().tfd_accept_sampled(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(p=None), 1), (dict(q=None), 1), (dict(d=None), 1), (dict(na=None), 1), (dict(u=None), 1),
    (dict(un=None), 1), (dict(nk=None), 1), (dict(nx=None), 1), (dict(streams=0), 1),
    (dict(win=0), 1), (dict(win=513), 1), (dict(n=0), 1), (dict(ldp=99), 1), (dict(ldq=99), 1),
    (dict(nq=50), 1), (dict(nq=0, m=FAKE), 1), (dict(p=FAKE + 2), 1), (dict(q=FAKE + 1), 1),
    (dict(u=FAKE + 2), 1), (dict(ah=FAKE), 1), (dict(ah=FAKE + 4, kh=FAKE), 1),
    (dict(n=1 << 21, ldp=1 << 21, nq=1 << 21, ldq=1 << 21), 2),
])
def test_accept_sampled_refusals(bad, code):
    assert accept_sampled_call(**bad) == code


@pytest.mark.parametrize("out", ["nk", "nx", "pr", "ah", "kh"])
@pytest.mark.parametrize("inp", ["p", "q", "m", "d", "na", "u", "un"])
def test_accept_sampled_overlaps(out, inp):
    """An output that is, or ends in, an input."""
    a = {name: FAKE * (i + 1) for i, name in
         enumerate(["p", "q", "m", "d", "na", "u", "un", "nk", "nx", "pr", "ah", "kh"])}
    for at in (a[out], a[out] + (40 if out in ("ah", "kh") else 16) - 4):
        assert accept_sampled_call(**dict(a, **{inp: at})) == 1


def lora_call(**kw):
    a = dict(x=FAKE, rows=2, k=64, ldx=64, a=FAKE, b=FAKE, na=3, rank=8, n=100, ids=FAKE, s=None,
             out=2, base=None, ldb=0, y=FAKE * 2, ldy=100, st=None, stream=None)
    a.update(kw)
    return tfd.library().tfd_lora(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(ids=None), 1), (dict(y=None), 1),
    (dict(out=0), 1), (dict(out=3), 1), (dict(rows=0), 1), (dict(k=60), 1), (dict(k=0), 1),
    (dict(ldx=56), 1), (dict(ldx=68), 1), (dict(n=0), 1), (dict(na=0), 1), (dict(rank=0), 1),
    (dict(rank=12), 1), (dict(ldy=99), 1), (dict(base=FAKE * 3, ldb=99), 1), (dict(x=FAKE + 8), 1),
    (dict(a=FAKE + 8), 1), (dict(y=FAKE * 2 + 1), 1), (dict(ids=FAKE + 2), 1),
    (dict(y=FAKE), 1),                                          # y overlaps x
    (dict(base=FAKE * 2 + 200, ldb=100), 1),                    # y overlaps base, shifted
    (dict(base=FAKE * 2, ldb=104), 1),                          # the same base, another stride
    (dict(rank=136), 2), (dict(na=4097), 2), (dict(rows=(1 << 18) + 1, y=FAKE << 20), 2),
    (dict(a=FAKE * 2 + 16), 1), (dict(b=FAKE * 2 - 16), 1),     # y overlaps an adapter
    (dict(ids=FAKE * 2 + 396), 1), (dict(s=FAKE * 2 - 8), 1),   # y overlaps ids, scales
])
def test_lora_refusals(bad, code):
    assert lora_call(**bad) == code
