"""What the tests of the paged attention share: caches whose unused places hold NaN, and the check of every
row against the oracle.

Tolerances of an output, before its bf16 rounding: with each seen token's log-weight known to within
eta_j the output is within sum_j p_j eta_j |v_j - out| (first order, times 1.01). eta_j has
* (2^-16 + 2^-18) (A_j + max A): q' in two 16-bit parts (2^-8 each), and q', its products and the
  subtraction of the maximum in fp32, as in ``helpers``; A_j = scale sum_e m_e |k_je|;
* for E4M3 keys 2^-23 A_most: q' over a power of two, its largest magnitude in [128, 256), enters as four
  E4M3 parts, each within 2^-4 of what is left (2^-16 in all) or, where that is less than half a step of the
  smallest numbers, within 2^-10; the last two stand for 2^-8 of what they are, so within 2^-18 / 2^7;
* 2^-20: exponentials and their arguments.
The weights in two bf16 parts add 2^-16 sum_j p_j |v_j| (for E4M3, as f16, 2^-11: half a step is at most 2^-11
of the value; what is below f16's smallest step counts for less than 2^-30 of the largest weight), and their sums, whose fp32 adds may each cut off
2^-23, 2^-17 and 2^-23 a 8 tokens. A log-sum is within max_j eta_j, 2^-20, 2^-23 of itself and the
sum's 2^-24 a token.
"""
import numpy as np
import torch

from helpers import assert_bf16_rounding, np32
from oracle.numerics import e4m3_decode
from oracle.paged import attend, turned
from speculative_decoding_draft_row_gb300 import tfd
from synth import inputs


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    """Requests over a cache of random pages; places that no token has hold NaN (codes and scales too)."""

    def __init__(self, lens, new, q_heads, heads, dim, page, fmt="bf16", layout="nhd", tid=800,
                 spare_rows=2, kv_std=1.0, q_std=1.0):
        self.lens, self.new = np.array(lens), np.array(new)
        self.q_heads, self.heads, self.dim, self.page, self.fmt = q_heads, heads, dim, page, fmt
        R, tokens = len(lens), self.lens + self.new
        need = -(-tokens // page)
        pages = int(need.sum()) + 2
        g = np.random.default_rng(tid)
        ids = g.permutation(pages)
        self.table = np.full((R, int(need.max()) + 1), -1)
        at = 0
        for r in range(R):
            self.table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
        used = np.zeros((pages, page), bool)
        for r in range(R):
            for t in range(tokens[r]):
                used[self.table[r, t // page], t % page] = True
        shape = (pages, page, heads, dim)
        if fmt == "bf16":
            k, v = (inputs.normal_bf16(shape, kv_std, tid + i) for i in (1, 2))
            k[torch.from_numpy(~used)] = float("nan")
            v[torch.from_numpy(~used)] = float("nan")
            self.kv = [np32(k), np32(v)]
            sc = [None, None]
        else:
            k, v = (torch.from_numpy(g.integers(0, 256, shape, np.uint8)) for _ in range(2))
            k[(k & 127) == 127] = 0x7E
            v[(v & 127) == 127] = 0x7E
            sc = [torch.from_numpy((g.random((pages, heads, page), np.float32) + 0.5) * kv_std / 250)
                  for _ in range(2)]
            self.kv = [e4m3_decode(t.numpy()) * s.numpy().transpose(0, 2, 1)[..., None].astype(float)
                       for t, s in zip((k, v), sc)]
            off = torch.from_numpy(~used)
            k[off], v[off] = 0x7F, 0xFF
            for s in sc:
                s[off[:, None, :].expand_as(s)] = float("nan")
            sc = [s.cuda() for s in sc]
        k, v = k.cuda(), v.cuda()
        if layout == "hnd":
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        elif layout == "both":
            both = torch.stack([k, v], 2)
            k, v = both[:, :, 0], both[:, :, 1]
        self.cache = tfd.KvPages(k, v, *sc)
        self.row_start = np.concatenate([[0], np.cumsum(self.new)])
        self.rows = int(self.row_start[-1]) + spare_rows
        wide = inputs.normal_bf16((self.rows, q_heads * dim + 8), q_std, tid + 3).cuda()
        self.q = wide[:, :q_heads * dim].view(self.rows, q_heads, dim)  # rows of a wider array
        self.gamma = inputs.normal_bf16((dim,), 0.5, tid + 4).cuda()
        self.ws = None

    def tokens(self, r):
        """Keys and values of request r, [tokens][heads][dim]."""
        n = int(self.lens[r] + self.new[r])
        t = np.arange(n)
        return [x[self.table[r, t // self.page], t % self.page] for x in self.kv]

    def run(self, tree=None, pos=None, window=-1, norm=True, rope=True, gamma=True, scale=0.0, st=None,
            max_new=None, lse=True, **kw):
        max_new = max_new or max(1, int(self.new.max()))
        if self.ws is None or self.ws_new != max_new:
            self.ws = tfd.zeroed_workspace(tfd.tfd_paged_attn_workspace(
                max_new, self.q_heads, self.heads, self.dim))
            self.ws_new = max_new
        out = torch.full((self.rows, self.q_heads * self.dim + 16), 7.0, dtype=torch.bfloat16,
                         device="cuda")
        ls = torch.full((self.rows, self.q_heads), 7.0, device="cuda") if lse else None
        tfd.tfd_paged_attn(self.q, self.cache, i32(self.table), i32(self.lens), i32(self.row_start),
                           max_new, pos=None if pos is None else i32(pos),
                           tree=None if tree is None else i32(np.asarray(tree, np.uint32).view(np.int32)),
                           window=window, q_gamma=self.gamma if gamma and norm else None, norm=norm,
                           rope=rope, scale=scale, out=out[:, :self.q_heads * self.dim], lse=ls,
                           ws=self.ws, dev_status=st, **kw)
        return out, ls

    def check(self, tree=None, pos=None, window=-1, norm=True, rope=True, gamma=True, scale=0.0,
              requests=None, got=None, what=""):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        if got is None:
            got = self.run(tree, pos, window, norm, rope, gamma, scale, st)
        torch.cuda.synchronize()
        assert st.item() == 0
        out, lse = (np32(t) for t in got)
        used = int(self.row_start[-1])
        width = self.q_heads * self.dim
        assert (out[:, width:] == 7).all() and (out[used:] == 7).all() and (lse[used:] == 7).all()
        sc = 1.0 / np.sqrt(self.dim) if scale == 0 else scale
        for r in range(len(self.lens)) if requests is None else requests:
            a, b = self.row_start[r], self.row_start[r + 1]
            n, length = b - a, int(self.lens[r])
            if n == 0:
                continue
            words = None if tree is None else [int(w) & ((1 << n) - 1) for w in tree[a:b]]
            at = [length + (j if tree is None else bin(words[j]).count("1") - 1) for j in range(n)] \
                if pos is None else pos[a:b]
            qx, mag = turned(np32(self.q)[a:b], np.maximum(at, 0), np32(self.gamma) if gamma else None,
                             norm, rope)
            k, v = self.tokens(r)
            y, ls, t = attend(qx, k, v, length, words, window, sc, mag)
            part, f8 = 2.0 ** -16 + 2.0 ** -18, 2.0 ** -23 if self.fmt != "bf16" else 0.0
            tok = length + n
            err = 1.01 * (part * t["dev_a"] + (2.0 ** -20 + f8 * t["a_most"][..., None]) * t["dev"]) + \
                ((2.0 ** -16 if self.fmt == "bf16" else 2.0 ** -11) + 2.0 ** -17 + 2.0 ** -23 * tok / 8) * \
                t["abs_out"]
            assert_bf16_rounding(out[a:b, :width].reshape(y.shape), y, err, f"{what} request {r}")
            fin = np.isfinite(ls)
            assert np.array_equal(lse[a:b][~fin], ls[~fin])
            lim = 2 * part * t["a"] + f8 * t["a_most"] + 2.0 ** -20 + 2.0 ** -24 * tok
            lim = lim + 2.0 ** -23 * np.abs(np.where(fin, ls, 0))
            d = np.abs(np.where(fin, lse[a:b] - np.where(fin, ls, 0), 0))
            assert (d <= lim).all(), (what, r, (d / lim).max())
        return got


def random_tree(n, g):
    """Words of a tree whose row j hangs on an earlier row."""
    words = [1]
    for j in range(1, n):
        words.append(words[int(g.integers(0, j))] | 1 << j)
    return words
