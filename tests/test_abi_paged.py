"""Host-side argument checks of the paged cache's calls: refused before the GPU is touched; and what the
Python binding refuses."""
import ctypes

import pytest
import torch

from speculative_decoding_draft_row_gb300 import tfd

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced by refused calls


def plan_call(**kw):
    a = dict(lens=FAKE, n_new=FAKE * 2, requests=4, page=16, table=FAKE * 3, ldt=8, max_pages=8,
             held=FAKE * 4, free=FAKE * 5, pages=100, n_free=FAKE * 6, row_start=FAKE * 7,
             slots=FAKE * 8, pos=FAKE * 9, rows=24, st=None, stream=None)
    a.update(kw)
    return tfd.library().tfd_page_plan(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(lens=None), 1), (dict(n_new=None), 1), (dict(table=None), 1), (dict(held=None), 1),
    (dict(free=None), 1), (dict(n_free=None), 1), (dict(row_start=None), 1), (dict(slots=None), 1),
    (dict(pos=None), 1), (dict(slots=None, pos=None), 1), (dict(rows=-1), 1), (dict(requests=0), 1),
    (dict(page=0), 1), (dict(page=1025), 1), (dict(max_pages=0), 1), (dict(ldt=7), 1),
    (dict(pages=0), 1), (dict(pages=1 << 28), 1), (dict(lens=FAKE + 2), 1), (dict(st=FAKE * 20 + 1), 1),
    (dict(requests=8193), 2), (dict(requests=8192, max_pages=1 << 18, ldt=1 << 18), 2),
    (dict(rows=1 << 31), 2),
])
def test_plan_refusals(bad, code):
    assert plan_call(**bad) == code


SIZES = dict(lens=16, n_new=16, table=(3 * 8 + 8) * 4, held=16, free=400, n_free=4, row_start=20,
             slots=96, pos=96)


@pytest.mark.parametrize("out", ["table", "held", "free", "n_free", "row_start", "slots", "pos"])
@pytest.mark.parametrize("other", list(SIZES))
def test_plan_overlaps(out, other):
    if out != other:
        base = {n: FAKE * (i + 1) for i, n in enumerate(SIZES)}
        assert plan_call(**dict(base, **{other: base[out] + SIZES[out] - 4})) == 1


def cache(**kw):
    a = dict(k=FAKE * 16, v=FAKE * 32, ks=None, vs=None, sp=16 * 8 * 128, st=8 * 128, sh=128, pages=10,
             page=16, heads=8, dim=128, fmt=0)
    a.update(kw)
    return ctypes.byref(tfd._KvPages(*a.values()))


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(fmt=2), 1), (dict(pages=0), 1), (dict(page=0), 1),
    (dict(page=1025, sp=1025 * 1024), 1), (dict(heads=0), 1), (dict(heads=1025), 1),
    (dict(pages=1 << 27), 1), (dict(dim=96), 2), (dict(dim=256), 2), (dict(sh=132), 1),
    (dict(sp=0), 1), (dict(st=-1024), 1), (dict(k=FAKE + 8), 1), (dict(fmt=1), 1),
    (dict(fmt=1, ks=FAKE, vs=FAKE + 2), 1), (dict(fmt=1, ks=FAKE, vs=FAKE, sh=136), 1),
    (dict(sh=64), 1), (dict(st=512), 1), (dict(sp=8 * 128), 1),          # vectors that share elements
    (dict(sp=1 << 46), 1),
]


def append_call(c=None, **kw):
    a = dict(k=FAKE, ldk=1024, v=FAKE * 2, ldv=1024, slots=FAKE * 3, pos=FAKE * 4, rows=6, qk=3, g=None,
             eps=1e-6, base=1e4, c=c or cache(), st=None, stream=None)
    a.update(kw)
    return tfd.library().tfd_paged_append(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(rows=0), 1),
    (dict(c=None), 1), (dict(qk=4), 1), (dict(qk=-1), 1), (dict(eps=-1.0), 1), (dict(base=0.0), 1),
    (dict(eps=float("nan")), 1), (dict(ldk=1016), 1), (dict(ldv=1028), 1), (dict(k=FAKE + 8), 1),
    (dict(slots=FAKE + 2), 1), (dict(g=FAKE + 1), 1), (dict(rows=1 << 29), 2), (dict(ldk=1 << 31), 2),
])
def test_append_refusals(bad, code):
    if "c" in bad:
        assert tfd.library().tfd_paged_append(FAKE, 1024, FAKE * 2, 1024, FAKE * 3, FAKE * 4, 6, 3, None,
                                              1e-6, 1e4, None, None, None) == code
    else:
        assert append_call(**bad) == code


CACHE_END = 9 * 16 * 1024 + 16 * 1024  # elements


@pytest.mark.parametrize("what", ["k", "v", "slots", "pos", "g", "st"])
@pytest.mark.parametrize("of", [FAKE * 16, FAKE * 32])
def test_append_overlaps_the_cache(what, of):
    assert append_call(**{what: of + 2 * CACHE_END - 16}) == 1


def attn_call(c=None, **kw):
    a = dict(q=FAKE, ldq=4096, rows=6, q_heads=32, c=c or cache(), table=FAKE * 3, ldt=8, max_pages=8,
             lens=FAKE * 4, row_start=FAKE * 5, requests=4, max_new=6, pos=FAKE * 6, tree=None, window=-1,
             qk=3, g=None, eps=1e-6, base=1e4, scale=0.0, out=FAKE * 7, ldo=4096, lse=None, ws=FAKE * 64,
             wsb=1 << 30, st=None, stream=None)
    a.update(kw)
    return tfd.library().tfd_paged_attn(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(row_start=None), 1),
    (dict(out=None), 1), (dict(rows=0), 1), (dict(requests=0), 1), (dict(max_new=0), 1),
    (dict(max_new=33), 1), (dict(max_pages=0), 1), (dict(ldt=7), 1), (dict(window=-2), 1),
    (dict(q_heads=4), 1), (dict(q_heads=36), 1), (dict(q_heads=65 * 8, ldq=1 << 17, ldo=1 << 17), 1),
    (dict(qk=8), 1), (dict(eps=-1.0), 1), (dict(base=-1.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ldq=4088), 1),
    (dict(ldq=4100), 1), (dict(ldo=4095), 1), (dict(q=FAKE + 8), 1), (dict(out=FAKE * 7 + 8), 1),
    (dict(pos=FAKE + 2), 1), (dict(tree=FAKE + 2), 1), (dict(ws=FAKE * 64 + 8), 1),
    (dict(ws=None), 3), (dict(wsb=1000), 3), (dict(requests=8193), 2), (dict(rows=1 << 27), 2),
])
def test_attn_refusals(bad, code):
    assert attn_call(**bad) == code


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches(bad, code):
    assert append_call(cache(**bad)) == code
    assert attn_call(cache(**bad)) == code


def test_layouts_that_are_fine():
    """What a refused pointer shows: the cache was looked at first and found in order."""
    for c in (cache(sh=16 * 128, st=128), cache(sp=2 * 16384), cache(pages=1, sp=8),
              cache(heads=1, sh=8, st=128, sp=2048), cache(fmt=1, ks=FAKE, vs=FAKE),
              cache(v=FAKE * 16 + 256, sh=256, st=2048, sp=16 * 2048), cache(page=1, st=8, sp=1024)):
        assert attn_call(c, rows=1 << 27) == 2


def test_strides_that_the_attention_refuses():
    """A cache of pages 2^31 elements apart takes rows, and is refused by the attention alone."""
    c = cache(sp=1 << 31)
    assert attn_call(c) == 2
    assert append_call(c, k=None) == 1                    # looked at behind the cache


@pytest.mark.parametrize("out,size", [("out", 5 * 8192 + 8192), ("lse", 6 * 32 * 4), ("ws", 4096),
                                      ("st", 4)])
@pytest.mark.parametrize("inp", ["q", "table", "lens", "row_start", "pos", "tree", "g", "k", "v", "out"])
def test_attn_overlaps(out, size, inp):
    if out == inp:
        return
    at = dict(out=FAKE * 7, lse=FAKE * 8, ws=FAKE * 64, st=FAKE * 9)
    if inp in ("k", "v"):
        assert attn_call(cache(**{inp: at[out] + max(0, size - 16)}), **at) == 1
    else:
        assert attn_call(**dict(at, **{inp: at[out] + max(0, size - 16)})) == 1


def test_attn_workspace():
    w = tfd.library().tfd_paged_attn_workspace
    assert 0 < w(1, 32, 8, 128) < w(6, 32, 8, 128)
    assert w(0, 32, 8, 128) == w(33, 32, 8, 128) == w(1, 30, 8, 128) == w(1, 32, 8, 96) == 0
    assert w(1, 4, 8, 128) == w(1, 65, 1, 128) == w(1, 8, 0, 64) == 0


# ---- the binding ---------------------------------------------------------------------------------

class FakeLibrary:
    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLibrary()
    monkeypatch.setattr(tfd, "_lib", lib)
    monkeypatch.setattr(tfd, "_current_device", lambda: -1)  # what a CPU tensor's get_device() says
    monkeypatch.setattr(tfd, "_stream", lambda stream, dev=None: 0)
    return lib


BF = torch.bfloat16


def pages(shape=(5, 4, 2, 64), dtype=BF):
    return torch.zeros(shape, dtype=dtype), torch.zeros(shape, dtype=dtype)


def test_cache_strides():
    k, v = pages()
    c = tfd.KvPages(k, v).c
    assert (c.page_stride, c.token_stride, c.head_stride) == (512, 128, 64)
    assert (c.pages, c.page_size, c.heads, c.dim, c.fmt) == (5, 4, 2, 64, 0)
    k, v = (t.transpose(1, 2) for t in pages((5, 2, 4, 64)))
    c = tfd.KvPages(k, v).c
    assert (c.page_stride, c.token_stride, c.head_stride) == (512, 64, 256)
    both = torch.zeros((5, 2, 4, 2, 64), dtype=BF)           # keys and values of a page side by side
    c = tfd.KvPages(both[:, 0], both[:, 1]).c
    assert (c.page_stride, c.token_stride, c.v - c.k) == (1024, 128, 1024)
    sc = torch.zeros((5, 2, 4))
    for dt in (torch.uint8, torch.float8_e4m3fn):
        assert tfd.KvPages(*pages(dtype=dt), sc, sc).c.fmt == 1


def test_caches_that_are_refused():
    k, v = pages()
    sc = torch.zeros((5, 2, 4))
    k8, v8 = pages(dtype=torch.uint8)
    for args in ((k, v[:4]), (k, v8), (k.float(), v.float()), (k[0], v[0]), (k, v, sc, sc), (k8, v8),
                 (k8, v8, sc, None), (k8, v8, sc, sc.transpose(1, 2)), (k8, v8, sc.double(), sc),
                 (k, v.transpose(1, 2).contiguous().transpose(1, 2)),
                 (k.transpose(2, 3), v.transpose(2, 3))):
        with pytest.raises(ValueError):
            tfd.KvPages(*args)


def test_rows_of_one_projections_output(fake):
    cache = tfd.KvPages(*pages())
    kv = torch.zeros((3, 2, 2, 64), dtype=BF)
    i = torch.zeros(3, dtype=torch.int32)
    tfd.tfd_paged_append(kv[:, 0], kv[:, 1], i, i, cache)
    assert fake.args[1] == fake.args[3] == 256
    with pytest.raises(ValueError):
        tfd.tfd_paged_append(kv[:, 0].transpose(1, 2), kv[:, 1], i, i, cache)
    with pytest.raises(ValueError):
        tfd.tfd_paged_append(kv[:, 0], kv[:, 1], i.long(), i, cache)


def test_attn_arguments(fake):
    cache = tfd.KvPages(*pages())
    i = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros((2, 9), dtype=torch.int32)[:, :6]
    ws = torch.zeros(16)
    ok = dict(q=torch.zeros((3, 4, 64), dtype=BF), cache=cache, table=table, lens=i[:2], row_start=i,
              max_new=2, ws=ws)
    out, lse = tfd.tfd_paged_attn(**ok)
    assert fake.args[6:8] == (9, 6) and out.shape == (3, 256) and lse is None
    for bad in (dict(q=torch.zeros((3, 4, 128), dtype=BF)), dict(q=torch.zeros((3, 4, 64))),
                dict(row_start=i[:2]), dict(pos=i[:2]), dict(tree=i.long()), dict(table=table.long()),
                dict(lse=torch.zeros((3, 2))), dict(out=torch.zeros((3, 256)))):
        with pytest.raises(ValueError):
            tfd.tfd_paged_attn(**dict(ok, **bad))
    assert tfd.tfd_paged_attn(**ok, want_lse=True)[1].shape == (3, 4)


def test_plan_arguments(fake):
    i = torch.zeros(2, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    free = torch.zeros(7, dtype=torch.int32)
    table = torch.zeros((2, 5), dtype=torch.int32)
    start, slots, pos = tfd.tfd_page_plan(i, i, 16, table, i.clone(), free, one, rows=11)
    assert start.numel() == 3 and slots.numel() == pos.numel() == 11
    assert tfd.tfd_page_plan(i, i, 16, table, i.clone(), free, one)[1:] == (None, None)
    assert fake.args[14] == 0
    with pytest.raises(ValueError):
        tfd.tfd_page_plan(i, i.long(), 16, table, i.clone(), free, one)
    with pytest.raises(ValueError):
        tfd.tfd_page_plan(i, i, 16, table.T, i.clone(), free, one)
