"""The 8-bit paged cache, its attention and the block-sparse attention against
the float64 oracle.

Tolerances.  Codes: half a step of the code, plus 2^-20 of the value for the two
fp32 roundings of x * (Q / amax) and the one of the scale.  Attention: P is
rounded to bf16 twice (hi + lo), 2^-8 * 2^-8 of itself; a logit is off by at most
(D / 16 + 2) * 2^-23 * sum |q k| / sqrt(D) (one fp32 rounding, truncation
allowed for, per matrix step) plus 2^-22 of itself for the scaling, which moves
P by twice that; the sums over tokens and warps add at most (tiles + 64) * 2^-23.
All of it relative to sum p |v|.  On the 8-bit cache P is fp16 (rounded twice, less
than the bf16 term above), where besides a value below fp16's smallest step is lost:
that step is 2^-24, P's largest value at least 2^8 and the sum of P at least that, so a
weight p = P / max P is off by at most half a step over 2^8, 2^-33, or by itself where it
is smaller, and an output by at most sum min(2^-33, p) |v| more.
"""
import math

import numpy as np
import pytest
import torch

from oracle import pages_oracle as P
from slow_sparse_kv_sfi_b200 import sfi as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = ["e4m3", "int8"]
PAGE = 16


def _fmt(f):
    return {"e4m3": S.FMT_E4M3, "int8": S.FMT_INT8}[f]


class Case:
    """A bf16 cache, its 8-bit cache (filled with garbage), a block index, queries."""

    def __init__(self, B, Hq, Hkv, D, lens, fmt="e4m3", seed=0, spare=3, slack=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.D, self.G, self.fmt = B, Hq, Hkv, D, Hq // Hkv, fmt
        self.lens = list(lens)
        self.L = max(max(self.lens), 1)
        self.max_pages = -(-self.L // PAGE) + slack
        self.n = B * self.max_pages + spare
        self.pt = torch.randperm(self.n, generator=g)[:B * self.max_pages].to(torch.int32).view(B, -1).contiguous()
        k = torch.randn(self.n, Hkv, PAGE, D, generator=g)
        k *= torch.exp(0.5 * torch.randn(self.n, Hkv, PAGE, 1, generator=g))
        self.k = k.to(torch.bfloat16)
        self.v = torch.randn(self.n, Hkv, PAGE, D, generator=g).to(torch.bfloat16)
        self.q = (torch.randn(B, Hq, D, generator=g) * 2).to(torch.bfloat16)
        self.g = g
        self.shape = S.make_shape(B, Hq, Hkv, D, self.max_pages, self.n)

    def up(self):
        n, Hkv, D, B = self.n, self.Hkv, self.D, self.B
        d = lambda t: t.to(DEV).contiguous()  # noqa: E731
        self.kd, self.vd, self.ptd, self.qd = d(self.k), d(self.v), d(self.pt), d(self.q)
        self.lend = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.kc = torch.full((n, Hkv, PAGE, D), 0x5B, dtype=torch.uint8, device=DEV)
        self.vc = torch.full((n, Hkv, PAGE, D), 0x5B, dtype=torch.uint8, device=DEV)
        self.ks = torch.full((n, Hkv), float("nan"), device=DEV)
        self.vs = torch.full((n, Hkv), float("nan"), device=DEV)
        self.ktail = torch.full((B, Hkv, PAGE, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.vtail = torch.full((B, Hkv, PAGE, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.bounds = torch.full((n, Hkv, 2, D), 77, dtype=torch.int8, device=DEV)
        self.bscale = torch.full((n, Hkv), float("nan"), device=DEV)
        self.kv = S.make_kv(self.kd, self.vd, self.ptd, None, self.err)
        self.q8 = S.make_quant_kv(self.kc, self.vc, self.ks, self.vs, self.ktail, self.vtail, self.ptd,
                                  _fmt(self.fmt), self.err)
        self.ix = S.make_block_index(self.bounds, self.bscale, self.ptd, self.err)
        self.ws = torch.zeros(S.sfi_block_workspace_size(self.shape), dtype=torch.uint8, device=DEV)
        self.out = torch.full((B, self.Hq, D), float("nan"), device=DEV)
        self.lse = torch.full((B, self.Hq), float("nan"), device=DEV)
        return self

    def error(self):
        torch.cuda.synchronize()
        return S.sfi_poll_error(self.kv)

    def rows(self, pool, b, h, n):
        """bf16 rows [0, n) of a sequence's head in float64."""
        x = pool[self.pt[b].long(), h].reshape(-1, self.D)[:n]
        return x.double().numpy()

    def quant_rows(self, which, b, h, n, blocks=None):
        """What the 8-bit cache on the device holds, in float64 (all blocks, or the listed ones)."""
        codes = (self.kc if which == "k" else self.vc).cpu().numpy()
        scale = (self.ks if which == "k" else self.vs).cpu().double().numpy()
        tail = (self.ktail if which == "k" else self.vtail).cpu().double().numpy()
        out = []
        for j in (range(-(-n // PAGE)) if blocks is None else blocks):
            if (j + 1) * PAGE <= n:
                p = int(self.pt[b, j])
                out.append(P.code_values(codes[p, h], self.fmt) * scale[p, h])
            else:
                out.append(tail[b, h, :n - j * PAGE])
        return np.concatenate(out) if out else np.zeros((0, self.D))


def check_attn(got, lse, q, K, V, what):
    """got [G, D], lse [G] (device results) against the oracle's attention over rows K, V."""
    o, ref_lse, pv, s = P.attention(q, K, V)
    D = q.shape[1]
    if len(K) == 0:
        assert np.all(got == 0) and np.all(lse == -np.inf), what
        return
    dz = (D / 16 + 2) * 2.0 ** -23 * s + 2.0 ** -22 * np.abs(s)
    rel = 2.0 ** -16 + 2 * dz + (len(K) / 16 + 64) * 2.0 ** -23
    z = q @ K.T / math.sqrt(D)
    tol = rel[:, None] * pv + np.minimum(2.0 ** -33, np.exp(z - z.max(1, keepdims=True))) @ np.abs(V) + 1e-30
    assert np.all(np.abs(got - o) <= tol), (what, (np.abs(got - o) / tol).max())
    assert np.all(np.abs(lse - ref_lse) <= 2 * dz + (len(K) / 16 + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(ref_lse)), what


def check_all(c, K_of, V_of, lens=None):
    out, lse, q = c.out.cpu().double().numpy(), c.lse.cpu().double().numpy(), c.q.double().numpy()
    for b, n in enumerate(lens or c.lens):
        for h in range(c.Hkv):
            r = slice(h * c.G, (h + 1) * c.G)
            check_attn(out[b, r], lse[b, r], q[b, r], K_of(b, h, n), V_of(b, h, n), (b, h, n))


# ------------------------------------------------------------------ store, append, load
def check_pages(c, lens, b, h):
    n = lens[b]
    kc, vc = c.kc.cpu().numpy(), c.vc.cpu().numpy()
    for codes, scale, pool in ((kc, c.ks, c.k), (vc, c.vs, c.v)):
        scale = scale.cpu().double().numpy()
        x = c.rows(pool, b, h, n)
        for j in range(n // PAGE):
            p = int(c.pt[b, j])
            page = x[j * PAGE:(j + 1) * PAGE]
            want = P.page_scale(page, c.fmt)
            assert abs(scale[p, h] - want) <= 2.0 ** -24 * want
            y = P.code_values(codes[p, h], c.fmt) * scale[p, h]
            assert np.all(np.abs(y - page) <= P.half_step(page, want, c.fmt) * (1 + 2.0 ** -20) + 2.0 ** -20 * np.abs(page))
    for j in range(n // PAGE):
        p = int(c.pt[b, j])
        codes, u = P.page_bounds(c.rows(c.k, b, h, n)[j * PAGE:(j + 1) * PAGE])
        assert np.array_equal(c.bounds[p, h].cpu().numpy().astype(np.int64), codes)
        assert float(c.bscale[p, h]) == u


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq,Hkv,lens", [
    (64, 4, 2, [1]), (128, 3, 3, [15, 16, 0, 17]), (64, 2, 2, [33, 1, 48]), (128, 8, 2, [250, 3, 129])])
def test_store_and_load(fmt, D, Hq, Hkv, lens):
    c = Case(len(lens), Hq, Hkv, D, lens, fmt, seed=1, slack=1).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend, index=c.ix)
    assert c.error() == 0
    written = torch.zeros(c.n, dtype=torch.bool)
    for b, n in enumerate(lens):
        written[c.pt[b, :n // PAGE].long()] = True
        r = n % PAGE
        last = c.pt[b, n // PAGE] if r else 0
        assert torch.equal(c.ktail[b, :, :r].cpu(), c.k[last, :, :r]) and torch.equal(c.vtail[b, :, :r].cpu(), c.v[last, :, :r])
        assert torch.isnan(c.ktail[b, :, r:]).all() and torch.isnan(c.vtail[b, :, r:]).all()
        for h in range(Hkv):
            check_pages(c, lens, b, h)
    # pages of no sequence, and pages that are not full, are left as they were
    rest = ~written.to(DEV)
    assert (c.kc[rest] == 0x5B).all() and (c.vc[rest] == 0x5B).all() and (c.bounds[rest] == 77).all()
    assert torch.isnan(c.ks[rest]).all() and torch.isnan(c.vs[rest]).all() and torch.isnan(c.bscale[rest]).all()

    k2, v2 = torch.full_like(c.kd, 9.0), torch.full_like(c.vd, 9.0)
    S.sfi_quant_load(c.shape, c.q8, S.make_kv(k2, v2, c.ptd, None, c.err), 0, c.L, lens=c.lend)
    assert c.error() == 0
    want_k, want_v = torch.full_like(c.k, 9.0), torch.full_like(c.v, 9.0)
    for b, n in enumerate(lens):
        for want, codes, scale, tail in ((want_k, c.kc, c.ks, c.ktail), (want_v, c.vc, c.vs, c.vtail)):
            for j in range(-(-n // PAGE)):
                p = int(c.pt[b, j])
                if (j + 1) * PAGE <= n:
                    vals = torch.from_numpy(P.code_values(codes[p].cpu().numpy(), fmt)).float()
                    want[p] = (vals * scale[p].cpu()[:, None, None]).to(torch.bfloat16)
                else:
                    want[p][:, :n - j * PAGE] = tail[b, :, :n - j * PAGE].cpu()
    assert torch.equal(k2.cpu(), want_k) and torch.equal(v2.cpu(), want_v)


@pytest.mark.parametrize("fmt", FMTS)
def test_store_in_chunks_and_uniform_length(fmt):
    """Chunk by chunk equals at once; lens = None equals lens of L."""
    c = Case(2, 4, 2, 128, [77, 77], fmt, seed=2).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 77, index=c.ix)
    one = [t.clone() for t in (c.kc, c.vc, c.ks, c.vs, c.bounds, c.bscale, c.ktail)]
    for t in (c.kc, c.vc, c.bounds):
        t.fill_(0x5B if t.dtype == torch.uint8 else 77)
    for t in (c.ks, c.vs, c.bscale, c.ktail, c.vtail):
        t.fill_(float("nan"))
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 32, index=c.ix)
    S.sfi_quant_store(c.shape, c.kv, c.q8, 32, 64, lens=torch.full((2,), 64, dtype=torch.int32, device=DEV), index=c.ix)
    S.sfi_quant_store(c.shape, c.kv, c.q8, 64, 77, lens=c.lend, index=c.ix)
    assert c.error() == 0
    for a, b in zip(one, (c.kc, c.vc, c.ks, c.vs, c.bounds, c.bscale, c.ktail)):
        assert torch.equal(torch.nan_to_num(a.float(), nan=-1e9), torch.nan_to_num(b.float(), nan=-1e9))
    # the index alone, from the bf16 cache
    b0, s0 = c.bounds.clone(), c.bscale.clone()
    c.bounds.fill_(77)
    c.bscale.fill_(float("nan"))
    S.sfi_block_build(c.shape, c.kv, c.ix, 0, 40)
    S.sfi_block_build(c.shape, c.kv, c.ix, 32, 77, lens=c.lend)
    assert c.error() == 0
    assert torch.equal(b0, c.bounds) and torch.equal(torch.nan_to_num(s0), torch.nan_to_num(c.bscale))


@pytest.mark.parametrize("fmt", FMTS)
def test_store_extreme_values(fmt):
    """A page of zeros, of denormals, of the largest values, with an infinity, with a NaN."""
    c = Case(1, 1, 1, 64, [96], fmt, seed=3)
    big = P.BF16_MAX
    k = c.k
    pg = c.pt[0].long()
    k[pg[0]] = 0.0
    k[pg[1]] = 1e-39
    k[pg[2], 0, 3, 5] = big
    k[pg[2], 0, 4, 6] = -big
    k[pg[3], 0, 1, 1] = float("inf")
    k[pg[4], 0, 15, 63] = float("nan")
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 96, index=c.ix)
    assert c.error() == 0
    codes, ks = c.kc.cpu(), c.ks.cpu()
    for j in (0, 1):
        assert (codes[pg[j]] == 0).all()
        assert abs(float(ks[pg[j], 0]) / (2.0 ** -100 / P.QMAX[fmt]) - 1) <= 2.0 ** -24
    y = P.code_values(codes[pg[2], 0].numpy(), fmt) * float(ks[pg[2], 0])
    assert abs(y[3, 5] / big - 1) <= 2.0 ** -22 and abs(y[4, 6] / -big - 1) <= 2.0 ** -22
    for j in (3, 4):
        assert (codes[pg[j]] == 0).all() and torch.isnan(ks[pg[j], 0])
    for j in range(6):
        codes_, u = P.page_bounds(k[pg[j], 0].double().numpy())
        assert np.array_equal(c.bounds[pg[j], 0].cpu().numpy(), codes_), j
        assert float(c.bscale[pg[j], 0]) == u


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_append_token_by_token_equals_store(fmt, D):
    """Ragged sequences, one of which stays empty, grown from nothing: the codes, scales and
    bounds of a store of the whole."""
    lens = [37, 0, 48, 16]
    c = Case(4, 2, 2, D, lens, fmt, seed=4).up()
    for t in range(1, 49):
        now = [min(t, n) for n in lens]
        ln = torch.tensor([n if t <= n else 0 for n in now], dtype=torch.int32, device=DEV)
        at = torch.tensor([max(n - 1, 0) for n in now])
        pages = c.pt.long()[torch.arange(4), at // PAGE]
        S.sfi_quant_append(c.shape, c.q8, c.L, c.k[pages, :, at % PAGE].to(DEV).contiguous(),
                           c.v[pages, :, at % PAGE].to(DEV).contiguous(), lens=ln, index=c.ix)
    assert c.error() == 0
    d = Case(4, 2, 2, D, lens, fmt, seed=4).up()
    S.sfi_quant_store(d.shape, d.kv, d.q8, 0, d.L, lens=d.lend, index=d.ix)
    for a, b in ((c.kc, d.kc), (c.vc, d.vc), (c.bounds, d.bounds)):
        assert torch.equal(a, b)
    for a, b in ((c.ks, d.ks), (c.vs, d.vs), (c.bscale, d.bscale)):
        assert torch.equal(torch.nan_to_num(a, nan=-1.0), torch.nan_to_num(b, nan=-1.0))
    for b, n in enumerate(lens):
        assert torch.equal(c.ktail[b, :, :n % PAGE], d.ktail[b, :, :n % PAGE])
        assert torch.equal(c.vtail[b, :, :n % PAGE], d.vtail[b, :, :n % PAGE])


# ------------------------------------------------------------------ attention over the 8-bit cache
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,Hq,Hkv,D,lens", [
    (1, 1, 1, 64, [1]), (1, 4, 2, 64, [1025]), (3, 7, 1, 128, [16, 0, 31]), (2, 32, 8, 128, [2000, 333]),
    (2, 16, 1, 64, [90, 515]), (1, 18, 2, 128, [3001]), (5, 5, 5, 64, [15, 17, 32, 0, 4096]),
    (1, 8, 8, 128, [40000])])
def test_quant_attention(fmt, B, Hq, Hkv, D, lens):
    c = Case(B, Hq, Hkv, D, lens, fmt, seed=5, slack=2).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend, lse=c.lse)
    assert c.error() == 0
    check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n), lambda b, h, n: c.quant_rows("v", b, h, n))
    first = c.out.clone()
    c.out.fill_(float("nan"))
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend)      # no lse
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)                                          # and the same bits again


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_is_read_exactly(fmt):
    """V rows hold every code; one token holds all the weight, so the output is the code's value,
    but for P's two fp16 roundings (2^-11 * 2^-11 of it) and four fp32 ones: less than 2^-21, and
    neighbouring codes are 2^-7 or more apart."""
    c = Case(1, 1, 1, 128, [64], fmt, seed=6).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 64)
    vals = [x for x in range(256) if not (fmt == "e4m3" and (x & 127) == 127)]
    codes = torch.tensor((vals + vals)[:128 * 2], dtype=torch.uint8).view(2, 128)
    unit = torch.zeros(128)
    unit[0] = 1.0
    for row in range(2):
        c.k[:] = 0
        page = int(c.pt[0, 2])
        c.k[page, 0, 5] = (unit * 4000.0).to(torch.bfloat16)
        c.kd.copy_(c.k)
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 64)
        c.vc[page, 0, 5] = codes[row].to(DEV)
        c.vs[page, 0] = 0.5
        c.qd.copy_((unit * 16).to(torch.bfloat16).view(1, 1, 128))
        S.sfi_quant_attn(c.shape, c.q8, 64, c.qd, c.out, c.ws)
        assert c.error() == 0
        want = P.code_values(codes[row].numpy(), fmt) * 0.5
        assert np.all(np.abs(c.out.cpu().double().numpy()[0, 0] - want) <= 2.0 ** -21 * np.abs(want))


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_attention_ignores_what_is_not_there(fmt):
    """NaN in the tail past the length, in pages past it and in pages of nobody; a page of NaN scale
    reaches its own head alone."""
    lens = [70, 16]
    c = Case(2, 4, 2, 128, lens, fmt, seed=7, slack=2).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    # (codes 0x5B, NaN scales and NaN tails are what every other place holds)
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend, lse=c.lse)
    assert c.error() == 0
    check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n), lambda b, h, n: c.quant_rows("v", b, h, n))
    good = c.out.clone()
    c.ks[int(c.pt[0, 1]), 1] = float("nan")
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend, lse=c.lse)
    torch.cuda.synchronize()
    assert torch.isnan(c.out[0, 2:]).all() and torch.isnan(c.lse[0, 2:]).all()
    assert torch.equal(c.out[0, :2], good[0, :2]) and torch.equal(c.out[1], good[1])


def test_quant_attention_large_and_lowest_values():
    """Logits of thousands, growing along the sequence, and rows of the lowest bf16 value."""
    c = Case(1, 2, 1, 64, [300], "int8", seed=8)
    ramp = torch.arange(300).float()
    for j in range(300):
        c.k[int(c.pt[0, j // PAGE]), 0, j % PAGE] = (c.k[int(c.pt[0, j // PAGE]), 0, j % PAGE].float()
                                                      * (1 + ramp[j])).to(torch.bfloat16)
    c.v[int(c.pt[0, 3]), 0, 2] = -3.0e30
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 300)
    S.sfi_quant_attn(c.shape, c.q8, 300, c.qd, c.out, c.ws, lse=c.lse)
    assert c.error() == 0
    check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n), lambda b, h, n: c.quant_rows("v", b, h, n))


def test_bad_pages_and_lengths_are_latched():
    c = Case(3, 2, 2, 64, [80, 64, 48], "e4m3", seed=9).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend, index=c.ix)
    assert c.error() == 0
    K, V = (lambda b, h, n: c.quant_rows("k", b, h, n)), (lambda b, h, n: c.quant_rows("v", b, h, n))
    # a page number outside the pool: its tokens are passed over, the rest stands
    keep = c.pt.clone()
    for bad in (-1, c.n, 2 ** 31 - 1):
        c.ptd[1, 2] = bad
        S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend, lse=c.lse)
        assert c.error() == 5 | (15 << 8)
        check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n, [0, 1, 3] if b == 1 else None),
                  lambda b, h, n: c.quant_rows("v", b, h, n, [0, 1, 3] if b == 1 else None))
        sel = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV).expand(3, 2, 4).contiguous()
        S.sfi_block_attn(c.shape, c.kv, c.L, c.qd, sel, 4, c.out, c.ws, lens=c.lend)
        assert c.error() == 5 | (15 << 8)
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
        assert c.error() == 5 | (13 << 8)
        S.sfi_block_select(c.shape, c.ix, c.L, c.qd, 0, 1, 3, torch.empty(3, 2, 3, dtype=torch.int32, device=DEV),
                           c.ws, lens=c.lend)
        assert c.error() == 5 | (14 << 8)
        c.ptd.copy_(keep)
    # a length outside [0, L]: the sequence counts as empty
    for bad in (-1, 81, 2 ** 31 - 1):
        ln = torch.tensor([80, bad, 48], dtype=torch.int32, device=DEV)
        S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=ln, lse=c.lse)
        assert c.error() == 5 | (12 << 8)
        check_all(c, K, V, [80, 0, 48])
        before = c.kc.clone()
        S.sfi_quant_append(c.shape, c.q8, c.L, c.kd[:3, :, 0].contiguous(), c.vd[:3, :, 0].contiguous(),
                           lens=torch.tensor([0, bad, 0], dtype=torch.int32, device=DEV))
        assert S.sfi_quant_poll_error(c.q8) == 5 | (12 << 8)
        assert torch.equal(before, c.kc)


# ------------------------------------------------------------------ block selection
def select_ref(c, K, n_sink, n_recent):
    nb = -(-c.L // PAGE)
    out = np.zeros((c.B, c.Hkv, K), np.int32)
    for b, n in enumerate(c.lens):
        for h in range(c.Hkv):
            bounds, scale = np.zeros((nb, 2, c.D), np.int64), np.zeros(nb)
            rows = c.rows(c.k, b, h, n)
            for j in range(n // PAGE):
                bounds[j], scale[j] = P.page_bounds(rows[j * PAGE:(j + 1) * PAGE])
            u = P.block_scores(c.q[b, h * c.G:(h + 1) * c.G].double().numpy(), bounds, scale)
            out[b, h] = P.select(u, n, n_sink, n_recent, K)
    return out


@pytest.mark.parametrize("B,Hq,Hkv,D,lens,n_sink,n_recent,K", [
    (1, 1, 1, 64, [1], 0, 1, 1), (1, 4, 2, 64, [1025], 4, 64, 13), (3, 7, 1, 128, [160, 0, 31], 0, 1, 4),
    (2, 32, 8, 128, [2000, 333], 4, 16, 20), (2, 16, 1, 64, [900, 515], 17, 33, 57), (1, 18, 2, 128, [3001], 4, 100, 40),
    (1, 2, 2, 64, [70000], 4, 64, 300)])
def test_select(B, Hq, Hkv, D, lens, n_sink, n_recent, K):
    c = Case(B, Hq, Hkv, D, lens, seed=10, slack=1).up()
    S.sfi_block_build(c.shape, c.kv, c.ix, 0, c.L, lens=c.lend)
    sel = torch.full((B, Hkv, K + 3), -7, dtype=torch.int32, device=DEV)
    S.sfi_block_select(c.shape, c.ix, c.L, c.qd, n_sink, n_recent, K, sel, c.ws, lens=c.lend)
    assert c.error() == 0
    assert np.array_equal(sel[..., :K].cpu().numpy(), select_ref(c, K, n_sink, n_recent))
    assert (sel[..., K:] == -7).all()


@pytest.mark.parametrize("rows", [3, 15, 16, 23, 27, 34, 46, 75, 149])
def test_select_rows_at_once(rows):
    """Row counts around those at which a row gets fewer of the GPU's multiprocessors."""
    n = 16 * 16 * 8 * 2 + 5   # blocks for every warp of the largest cluster, and some for a second one
    c = Case(1, rows, rows, 64, [n * PAGE - 3] if rows < 20 else [700 * PAGE + 1], seed=23, slack=1).up()
    S.sfi_block_build(c.shape, c.kv, c.ix, 0, c.L)
    sel = torch.full((1, rows, 40), -7, dtype=torch.int32, device=DEV)
    S.sfi_block_select(c.shape, c.ix, c.L, c.qd, 4, 64, 40, sel, c.ws)
    assert c.error() == 0
    b, s, pt = c.bounds.cpu().numpy(), c.bscale.cpu().double().numpy(), c.pt[0].numpy()
    nb = -(-c.L // PAGE)
    q = c.q[0].double().numpy()
    for h in range(rows):
        u = P.block_scores(q[h:h + 1], b[pt[:nb], h].astype(np.int64), s[pt[:nb], h])
        assert np.array_equal(sel[0, h].cpu().numpy(), P.select(u, c.L, 4, 64, 40)), h


def test_select_ties_zeros_and_extreme_queries():
    """Equal pages (ties to the lower block), a zero query, and queries of 1e38, 1e-38, NaN and infinity."""
    c = Case(1, 6, 1, 64, [800], seed=11)
    page = c.k[int(c.pt[0, 7])].clone()
    for j in range(3, 40):
        c.k[int(c.pt[0, j])] = page
    for q in (torch.zeros(6, 64), torch.full((6, 64), 1e38), torch.randn(6, 64) * 1e-38,
              torch.cat([torch.full((1, 64), float("nan")), torch.randn(4, 64), torch.full((1, 64), -float("inf"))])):
        c.q = q.to(torch.bfloat16).view(1, 6, 64)
        c.up()
        S.sfi_block_build(c.shape, c.kv, c.ix, 0, 800)
        sel = torch.empty(1, 1, 12, dtype=torch.int32, device=DEV)
        S.sfi_block_select(c.shape, c.ix, 800, c.qd, 4, 20, 12, sel, c.ws)
        assert c.error() == 0
        big = float(np.finfo(np.float32).max)
        nb = 50
        bounds, scale = zip(*(P.page_bounds(c.rows(c.k, 0, 0, 800)[j * 16:j * 16 + 16]) for j in range(nb)))
        u = np.clip(P.block_scores(c.q[0].double().numpy(), np.stack(bounds), np.array(scale)), -big, big)
        assert np.array_equal(sel[0, 0].cpu().numpy(), P.select(u, 800, 4, 20, 12))


# ------------------------------------------------------------------ block-sparse attention
def listed(c, pool, b, h, n, blocks):
    rows = c.rows(pool, b, h, n)
    parts = [rows[j * PAGE:min((j + 1) * PAGE, n)] for j in blocks if 0 <= j * PAGE < n]
    return np.concatenate(parts) if parts else np.zeros((0, c.D))


@pytest.mark.parametrize("B,Hq,Hkv,D,lens,K", [
    (1, 1, 1, 64, [1], 1), (1, 4, 2, 64, [1025], 13), (3, 7, 1, 128, [160, 0, 31], 4), (2, 32, 8, 128, [2000, 333], 60),
    (2, 16, 1, 64, [900, 515], 57), (1, 18, 2, 128, [3001], 188), (1, 8, 8, 128, [20000], 700)])
def test_block_attention_over_listed_blocks(B, Hq, Hkv, D, lens, K):
    c = Case(B, Hq, Hkv, D, lens, "int8", seed=12, slack=1)
    # lists of any order, with entries past the end, negative and repeated ones, and the last block among them
    nb = -(-c.L // PAGE)
    sel = torch.randint(0, nb, (B, Hkv, K), generator=c.g, dtype=torch.int32)
    sel[0, 0, 0] = (lens[0] - 1) // PAGE
    if K > 3:
        sel[:, :, 1] = -1
        sel[:, :, 2] = 2 ** 31 - 1
        sel[:, 0, 3] = sel[:, 0, 0]
    for b, n in enumerate(lens):     # rows past the end of the last page hold NaN
        if n % PAGE:
            c.k[int(c.pt[b, n // PAGE]), :, n % PAGE:] = float("nan")
            c.v[int(c.pt[b, n // PAGE]), :, n % PAGE:] = float("nan")
    c.up()
    wide = torch.full((B, Hkv, K + 5), 0, dtype=torch.int32)
    wide[..., :K] = sel
    wided = wide.to(DEV)
    S.sfi_block_attn(c.shape, c.kv, c.L, c.qd, wided, K, c.out, c.ws, lens=c.lend, lse=c.lse)
    assert c.error() == 0
    check_all(c, lambda b, h, n: listed(c, c.k, b, h, n, sel[b, h].tolist()),
              lambda b, h, n: listed(c, c.v, b, h, n, sel[b, h].tolist()))
    for fmt in FMTS:
        c.fmt = fmt
        c.up()
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
        S.sfi_quant_block_attn(c.shape, c.q8, c.L, c.qd, wided, K, c.out, c.ws, lens=c.lend, lse=c.lse)
        assert c.error() == 0
        kc = {}

        def rows(which, b, h, n):
            if (which, b, h) not in kc:
                kc[which, b, h] = c.quant_rows(which, b, h, n)
            r = kc[which, b, h]
            parts = [r[j * PAGE:min((j + 1) * PAGE, n)] for j in sel[b, h].tolist() if 0 <= j * PAGE < n]
            return np.concatenate(parts) if parts else np.zeros((0, c.D))

        check_all(c, lambda b, h, n: rows("k", b, h, n), lambda b, h, n: rows("v", b, h, n))


def test_all_blocks_listed_equal_dense_attention():
    c = Case(2, 8, 2, 128, [515, 515], seed=13).up()
    nb = 33
    sel = torch.arange(nb, dtype=torch.int32, device=DEV).expand(2, 2, nb).contiguous()
    S.sfi_block_attn(c.shape, c.kv, 515, c.qd, sel, nb, c.out, c.ws, lse=c.lse)
    p = S.make_params(4, 64, 16, 0.2, 0.2, 0.5, 0.5, 0.5, 32, 8)
    ws = torch.zeros(S.sfi_workspace_size(c.shape, p), dtype=torch.uint8, device=DEV)
    ref, ref_lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    S.sfi_dense_attn(c.shape, c.kv, 515, c.qd, ref, ws, S.DenseExtras(ref_lse.data_ptr(), None, None, 0, None, 0, 0))
    assert c.error() == 0
    check_all(c, lambda b, h, n: c.rows(c.k, b, h, n), lambda b, h, n: c.rows(c.v, b, h, n))
    # both are within their bound of the oracle: 2^-15 of sum p |v| <= max |v| between them
    assert float((c.out - ref).abs().max()) <= 2.0 ** -13 * float(c.v.float().abs().max())
    assert float((c.lse - ref_lse).abs().max()) <= 1e-4


def test_offsets_past_32_bits():
    """Pools whose pages lie past 2^32 bytes (8-bit) and past 2^32 elements' bytes (bf16)."""
    B, Hq, Hkv, D, n = 1, 4, 2, 128, 1100000
    lens = [40]
    c = Case(B, Hq, Hkv, D, lens, "int8", seed=14)
    far = [n - 1, n - 70000, n // 2 + 11]
    c.shape = S.make_shape(B, Hq, Hkv, D, 3, n)
    pt = torch.tensor([far], dtype=torch.int32, device=DEV)
    kq = torch.empty(n, Hkv, PAGE, D, dtype=torch.uint8, device=DEV)
    vq = torch.empty(n, Hkv, PAGE, D, dtype=torch.uint8, device=DEV)
    ks, vs = torch.empty(n, Hkv, device=DEV), torch.empty(n, Hkv, device=DEV)
    kb = torch.empty(n, Hkv, PAGE, D, dtype=torch.bfloat16, device=DEV)
    for j in range(3):
        kb[far[j]] = c.k[int(c.pt[0, j])].to(DEV)
    kv = S.make_kv(kb, kb, pt)
    small = c.pt.clone()
    shape = c.shape
    c.up()
    c.shape = shape
    bounds = torch.empty(n, Hkv, 2, D, dtype=torch.int8, device=DEV)
    bscale = torch.empty(n, Hkv, device=DEV)
    q8 = S.make_quant_kv(kq, vq, ks, vs, c.ktail, c.vtail, pt, S.FMT_INT8)
    ix = S.make_block_index(bounds, bscale, pt)
    S.sfi_quant_store(c.shape, kv, q8, 0, 40, index=ix)
    S.sfi_quant_attn(c.shape, q8, 40, c.qd, c.out, c.ws, lse=c.lse)
    torch.cuda.synchronize()
    for j in range(2):     # bring the far pages to where the checks look
        p = int(small[0, j])
        c.kc[p], c.vc[p], c.ks[p], c.vs[p] = kq[far[j]], vq[far[j]], ks[far[j]], vs[far[j]]
    check_all(c, lambda b, h, m: c.quant_rows("k", b, h, m), lambda b, h, m: c.quant_rows("v", b, h, m))
    sel = torch.tensor([[[0, 1, 2]] * 2], dtype=torch.int32, device=DEV)
    S.sfi_block_attn(c.shape, kv, 40, c.qd, sel, 3, c.out, c.ws, lse=c.lse)
    torch.cuda.synchronize()
    check_all(c, lambda b, h, m: c.rows(c.k, b, h, m), lambda b, h, m: c.rows(c.k, b, h, m))


# ------------------------------------------------------------------ as they are used
def _decode_step(c, sel, K, k_new, v_new, lens):
    S.sfi_quant_append(c.shape, c.q8, c.L, k_new, v_new, lens=lens, index=c.ix)
    S.sfi_block_select(c.shape, c.ix, c.L, c.qd, 4, 20, K, sel, c.ws, lens=lens)
    S.sfi_quant_block_attn(c.shape, c.q8, c.L, c.qd, sel, K, c.out, c.ws, lens=lens, lse=c.lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_loop_in_a_replayed_graph(fmt):
    """store, then append -> select -> attend for 40 tokens: the captured step replayed with growing
    lengths gives what eager calls give, and those agree with the oracle."""
    B, Hq, Hkv, D, K, steps = 2, 8, 2, 64, 9, 40
    start = [150, 0]
    final = [n + steps for n in start]
    mk = lambda: Case(B, Hq, Hkv, D, final, fmt, seed=15).up()  # noqa: E731
    eager, graph = mk(), mk()
    res = {}
    for name, c in (("eager", eager), ("graph", graph)):
        ln = torch.tensor(start, dtype=torch.int32, device=DEV)
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=ln, index=c.ix)
        sel = torch.zeros(B, Hkv, K, dtype=torch.int32, device=DEV)
        k_new = torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device=DEV)
        v_new = torch.zeros_like(k_new)
        g = None
        if name == "graph":
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                _decode_step(c, sel, K, k_new, v_new, ln)
        res[name] = []
        for t in range(steps):
            at = torch.tensor([n + t for n in start])
            pages = c.pt.long()[torch.arange(B), at // PAGE]
            k_new.copy_(c.k[pages, :, at % PAGE])
            v_new.copy_(c.v[pages, :, at % PAGE])
            ln += 1
            if g is not None:
                g.replay()
            else:
                _decode_step(c, sel, K, k_new, v_new, ln)
            res[name].append((sel.clone(), c.out.clone(), c.lse.clone()))
        assert c.error() == 0
        if name == "eager":
            c.lens = final
            assert np.array_equal(sel.cpu().numpy(), select_ref(c, K, 4, 20))
            blocks = sel.cpu()
            check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n, [j for j in blocks[b, h].tolist() if j * PAGE < n]),
                      lambda b, h, n: c.quant_rows("v", b, h, n, [j for j in blocks[b, h].tolist() if j * PAGE < n]))
    for a, b in zip(res["eager"], res["graph"]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_graphs_share_a_workspace_and_another_stream():
    """Two captured attention calls on one workspace, replayed in turn; and a call on a stream of its own."""
    a = Case(1, 8, 2, 128, [5000], "e4m3", seed=16).up()
    b = Case(1, 8, 2, 128, [5000], "int8", seed=17).up()
    want = []
    for c in (a, b):
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L)
        S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lse=c.lse)
        want.append(c.out.clone())
    torch.cuda.synchronize()
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, a.ws, lse=c.lse)
        graphs.append(g)
    for _ in range(3):
        for c, g in zip((a, b), graphs):
            c.out.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    st = torch.cuda.Stream()
    a.out.fill_(float("nan"))
    st.wait_stream(torch.cuda.current_stream())
    S.sfi_quant_attn(a.shape, a.q8, a.L, a.qd, a.out, a.ws, stream=st)
    st.synchronize()
    assert torch.equal(a.out, want[0])


def test_restored_pages_feed_the_packed_path():
    """An 8-bit cache loaded back into bf16 pages serves sfi_dense_attn like any other cache."""
    c = Case(2, 8, 2, 128, [400, 400], "int8", seed=18).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 400)
    k2, v2 = torch.zeros_like(c.kd), torch.zeros_like(c.vd)
    kv2 = S.make_kv(k2, v2, c.ptd, None, c.err)
    S.sfi_quant_load(c.shape, c.q8, kv2, 0, 400)
    p = S.make_params(4, 64, 16, 0.2, 0.2, 0.5, 0.5, 0.5, 32, 8)
    ws = torch.zeros(S.sfi_workspace_size(c.shape, p), dtype=torch.uint8, device=DEV)
    S.sfi_dense_attn(c.shape, kv2, 400, c.qd, c.out, ws,
                     S.DenseExtras(c.lse.data_ptr(), None, None, 0, None, 0, 0))
    assert c.error() == 0
    kc, vc = k2.cpu(), v2.cpu()
    check_all(c, lambda b, h, n: c.rows(kc, b, h, n), lambda b, h, n: c.rows(vc, b, h, n))


@pytest.mark.parametrize("what", ["equal", "two values", "one far outlier", "zeros", "bad page"])
@pytest.mark.parametrize("nb,K", [(700, 300), (5000, 700), (5000, 4999), (16384, 40)])
def test_select_uneven_scores(what, nb, K):
    """Score distributions that crowd one bin of the selection's histogram: all equal (ties to the
    lower block), two values, an outlier far above the rest, zeros; and a page that cannot be read."""
    D, n = 64, nb * PAGE
    g = torch.Generator().manual_seed(3)
    bounds = torch.zeros(nb, 1, 2, D, dtype=torch.int8)
    scale = torch.ones(nb, 1)
    q = torch.zeros(1, 1, D)
    q[..., 0] = 127.0
    if what == "equal":
        bounds[:, :, 0, 0] = 5
    elif what == "two values":
        bounds[:, :, 0, 0] = torch.randint(0, 2, (nb, 1), generator=g).to(torch.int8) * 9
    elif what == "one far outlier":
        bounds[:, :, 0, 0] = torch.randint(-127, 128, (nb, 1), generator=g).to(torch.int8)
        scale[nb // 2] = 2.0 ** 100
    elif what == "bad page":
        bounds[:, :, 0, 0] = torch.randint(-127, 128, (nb, 1), generator=g).to(torch.int8)
    bounds[:, :, 1] = bounds[:, :, 0]
    pt = torch.arange(nb, dtype=torch.int32).view(1, nb)
    u = P.block_scores(q[0].double().numpy(), bounds[:, 0].numpy().astype(np.int64), scale[:, 0].double().numpy())
    if what == "bad page":
        pt[0, nb // 3] = -5
        u[nb // 3] = -np.inf
    shape = S.make_shape(1, 1, 1, D, nb, nb)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = [t.to(DEV).contiguous() for t in (bounds, scale, pt)]
    ix = S.make_block_index(*d, err=err)
    sel = torch.empty(1, 1, K, dtype=torch.int32, device=DEV)
    ws = torch.empty(S.sfi_block_workspace_size(shape), dtype=torch.uint8, device=DEV)
    S.sfi_block_select(shape, ix, n, q.to(torch.bfloat16).to(DEV), 4, 20, K, sel, ws)
    torch.cuda.synchronize()
    assert int(err.item()) == (5 | (14 << 8) if what == "bad page" else 0)
    assert np.array_equal(sel[0, 0].cpu().numpy(), P.select(u, n, 4, 20, K))


@pytest.mark.parametrize("B,Hq,Hkv,L", [(25, 16, 4, 272), (100, 3, 3, 33), (297, 1, 1, 300), (1, 16, 1, 9000), (7, 64, 4, 700),
                                        (2, 8, 8, 17)])
def test_calls_stay_inside_their_workspace(B, Hq, Hkv, L):
    """Rows of every count, cut into pieces or not, of one length and ragged: nothing behind the
    reported size is written, and the results stand."""
    c = Case(B, Hq, Hkv, 64, [L] * B, "int8", seed=19).up()
    need = c.ws.numel()
    big = torch.zeros(need + (1 << 20), dtype=torch.uint8, device=DEV)
    big[need:] = 0x3C
    c.ws = big[:need]
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, L, index=c.ix)
    nb = -(-L // PAGE)
    sel = torch.arange(nb, dtype=torch.int32, device=DEV).expand(B, Hkv, nb).contiguous()
    outs = []
    for lens in (None, c.lend):
        S.sfi_quant_attn(c.shape, c.q8, L, c.qd, c.out, c.ws, lens=lens, lse=c.lse)
        outs.append(c.out.clone())
        S.sfi_quant_block_attn(c.shape, c.q8, L, c.qd, sel, nb, c.out, c.ws, lens=lens, lse=c.lse)
        outs.append(c.out.clone())
        few = torch.empty(B, Hkv, min(nb, 3), dtype=torch.int32, device=DEV)
        S.sfi_block_select(c.shape, c.ix, L, c.qd, 0, 1, min(nb, 3), few, c.ws, lens=lens)
    assert c.error() == 0
    assert (big[need:] == 0x3C).all()
    check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n), lambda b, h, n: c.quant_rows("v", b, h, n))
    for o in outs[:-1]:   # all of them attend to everything; the cuts differ
        assert float((o - outs[-1]).abs().max()) <= 1e-5 * float(c.v.float().abs().max())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq", [(64, 3), (128, 6), (128, 13)])
def test_value_scales_far_apart(fmt, D, Hq):
    """Pages of values from 1e-25 to 1e30, the weight on small ones: pages 2^6 and more below the
    largest scale so far, and scales that rise along the sequence."""
    n = 20 * PAGE + 5
    c = Case(1, Hq, 1, D, [n], fmt, seed=20)
    unit = torch.zeros(D)
    unit[0] = 1.0
    amp = [1.0, 1e30, 1e-3, 1e25, 1e-25, 1.0, 1e28, 1e3] * 3
    for j in range(21):
        p = int(c.pt[0, j])
        c.v[p] = (c.v[p].float() * amp[j]).to(torch.bfloat16)
        # logits: high where the values are small, hundreds lower elsewhere
        big = amp[j] >= 1e25
        c.k[p, 0] = (c.k[p, 0].float() * 0.3 + unit * (-300.0 if big else 0.0)).to(torch.bfloat16)
    c.q[0, :, 0] = 12.0
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, n)
    S.sfi_quant_attn(c.shape, c.q8, n, c.qd, c.out, c.ws, lse=c.lse)
    assert c.error() == 0
    assert float(c.out.abs().max()) < 1e4
    check_all(c, lambda b, h, m: c.quant_rows("k", b, h, m), lambda b, h, m: c.quant_rows("v", b, h, m))


@pytest.mark.parametrize("B,Hq,Hkv,D,lens", [
    (1, 16, 1, 64, [9001]), (1, 64, 4, 128, [6000]), (3, 32, 2, 128, [4097, 0, 65]), (2, 24, 2, 64, [9000, 1]),
    (2, 32, 2, 64, [5000, 5000]), (40, 16, 1, 64, [7000] + [1] * 38 + [300])])
def test_rows_in_many_pieces(B, Hq, Hkv, D, lens):
    """Few rows of many heads: of one length, of very uneven ones, and as lists of blocks; a NaN in
    one head's query stays there; a second call gives the same bits."""
    c = Case(B, Hq, Hkv, D, lens, "int8", seed=22)
    c.q[0, Hq // Hkv - 2, 3] = float("nan")
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    nb = -(-c.L // PAGE)
    sel = torch.arange(nb, dtype=torch.int32).flip(0).expand(B, Hkv, nb).contiguous().to(DEV)
    calls = [lambda n: S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=n, lse=c.lse),
             lambda n: S.sfi_quant_block_attn(c.shape, c.q8, c.L, c.qd, sel, nb, c.out, c.ws, lens=n, lse=c.lse)]
    K, V = {}, {}
    for b, n in enumerate(lens):
        for h in range(Hkv):
            K[b, h], V[b, h] = c.quant_rows("k", b, h, n), c.quant_rows("v", b, h, n)
    for call in calls:
        for n in (c.lend, None) if min(lens) == c.L else (c.lend,):
            got = []
            for _ in range(2):
                c.out.fill_(float("nan"))
                c.lse.fill_(float("nan"))
                call(n)
                assert c.error() == 0
                got.append((c.out.clone(), c.lse.clone()))
            bits = [[x.view(torch.int32) for x in g] for g in got]
            assert all(torch.equal(x, y) for x, y in zip(*bits))
            bad = Hq // Hkv - 2
            assert torch.isnan(c.out[0, bad]).all() and torch.isnan(c.lse[0, bad])
            out, lse, q = c.out.cpu().double().numpy(), c.lse.cpu().double().numpy(), c.q.double().numpy()
            for b in range(B):
                for h in range(Hkv):
                    G = Hq // Hkv
                    hs = [x for x in range(h * G, h * G + G) if (b, x) != (0, bad)]
                    check_attn(out[b, hs], lse[b, hs], q[b, hs], K[b, h], V[b, h], (b, h))


def test_replay_with_other_lengths_in_many_pieces():
    """A captured call whose lengths change between replays: rows in many pieces, in one, and empty."""
    c = Case(3, 32, 2, 64, [4000, 4000, 4000], "e4m3", seed=24).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L)
    V = c.v.float().abs().max().item()
    lens = torch.full((3,), 4000, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=lens, lse=c.lse)
    for now in ([4000, 16, 0], [0, 0, 0], [1600, 4000, 4000], [32, 0, 3984], [4000, 4000, 4000]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        c.out.fill_(float("nan"))
        c.lse.fill_(float("nan"))
        g.replay()
        assert c.error() == 0
        out, lse = c.out.cpu().double().numpy(), c.lse.cpu().double().numpy()
        for b, n in enumerate(now):
            q = c.q[b].double().numpy()
            for h in range(2):
                K, W = c.quant_rows("k", b, h, n), c.quant_rows("v", b, h, n)
                check_attn(out[b, h * 16:h * 16 + 16], lse[b, h * 16:h * 16 + 16], q[h * 16:h * 16 + 16], K, W, (now, b, h))
        assert np.abs(out).max() <= 2 * V


@pytest.mark.parametrize("Hq", [4, 8, 16])
def test_nan_stays_where_it_is(Hq):
    """A NaN in one head's query, and a page of values that is not finite."""
    c = Case(2, Hq, 1, 64, [100, 70], "e4m3", seed=21)
    c.q[0, 1, 3] = float("nan")
    c.v[int(c.pt[1, 2]), 0, 4, 5] = float("inf")
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend, lse=c.lse)
    assert c.error() == 0
    assert torch.isnan(c.out[0, 1]).all() and torch.isnan(c.lse[0, 1])
    assert torch.isnan(c.out[1]).all() and torch.isfinite(c.lse[1]).all()
    K, V = c.quant_rows("k", 0, 0, 100), c.quant_rows("v", 0, 0, 100)
    out, lse, q = c.out.cpu().double().numpy(), c.lse.cpu().double().numpy(), c.q.double().numpy()
    rest = [h for h in range(Hq) if h != 1]
    check_attn(out[0, rest], lse[0, rest], q[0, rest], K, V, "the other heads")


def test_one_workspace_serves_several_shapes():
    cases = [Case(1, 8, 2, 128, [3000], "e4m3", seed=22).up(), Case(5, 16, 8, 64, [700, 0, 33, 650, 16], "int8", seed=23).up(),
             Case(1, 16, 1, 128, [5000], "int8", seed=24).up()]
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for c in cases:
            c.out.fill_(float("nan"))
            S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
            S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, ws, lens=c.lend, lse=c.lse)
            assert c.error() == 0
            check_all(c, lambda b, h, n: c.quant_rows("k", b, h, n), lambda b, h, n: c.quant_rows("v", b, h, n))


def test_length_goes_back_within_the_page():
    """Tokens appended, dropped and appended again inside the page, over its end included."""
    c = Case(1, 2, 2, 64, [32], "int8", seed=25).up()
    tok = lambda t, d: (c.k[c.pt[0, t // PAGE].long(), :, t % PAGE] * d)[None].to(DEV).contiguous()  # noqa: E731
    for t in range(16):
        S.sfi_quant_append(c.shape, c.q8, t + 1, tok(t, 2.0), tok(t, 2.0))
    for t in range(11, 16):                       # back to 11 tokens, on with others
        S.sfi_quant_append(c.shape, c.q8, t + 1, tok(t, 1.0), tok(t, 1.0))
    assert c.error() == 0
    p = int(c.pt[0, 0])
    want = c.k[p].float().clone()
    want[:, :11] *= 2
    for h in range(2):
        x = want[h].double().numpy()
        y = P.code_values(c.kc[p, h].cpu().numpy(), "int8") * float(c.ks[p, h])
        assert np.all(np.abs(y - x) <= P.half_step(x, P.page_scale(x, "int8"), "int8") * (1 + 2.0 ** -20) + 2.0 ** -20 * np.abs(x))
    S.sfi_quant_attn(c.shape, c.q8, 13, c.qd, c.out, c.ws, lse=c.lse)     # 13 tokens: the tail's rows
    torch.cuda.synchronize()
    rows = lambda b, h, n: want[h, :13].to(torch.bfloat16).double().numpy()  # noqa: E731
    check_all(c, rows, rows, [13])
