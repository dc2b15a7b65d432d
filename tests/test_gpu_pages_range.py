"""The 8-bit cache, its attention and the block-sparse attention at the ends of
the number range, against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import pages_oracle as P
from slow_sparse_kv_sfi_b200 import sfi as S

from test_gpu_pages import DEV, FMTS, PAGE, Case, check_all, listed

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection
def _signs(n):
    return torch.tensor([1.0, -1.0, -1.0, 1.0, -1.0]).repeat(-(-n // 5))[:n]


SCORES = {   # queries of a group (from rows of N(0, 1)), size of the keys
    "infinity": (lambda q: q.index_fill(1, torch.tensor([3]), math.inf), 0.1),
    "minus infinity in one head": (lambda q: torch.cat([q[:1].index_fill(1, torch.tensor([5]), -math.inf), q[1:]]), 0.01),
    "1e36": (lambda q: q * 1e36, 0.01),
    "1e38, small keys": (lambda q: (q * 1e38).clamp(-3e38, 3e38), 1e-6),
    "1e38, large keys": (lambda q: (q * 1e38).clamp(-3e38, 3e38), 1e38),
    "heads far apart": (lambda q: q * 10.0 ** (40.0 * torch.arange(len(q)) / (len(q) - 1) - 3.0)[:, None].clamp(max=1e37), 1e-3),
    "subnormal": (lambda q: q * 1e-25, 1e-18),
    "small queries, large keys": (lambda q: q * 1e-38, 1e30),
    "nothing left": (lambda q: q.abs() * 1e-30, 1e-30),
}


@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 12)])
@pytest.mark.parametrize("what", list(SCORES))
def test_select_scores_at_the_ends_of_the_range(what, D, Hq):
    """Scores are the definition's, rounded once to fp32 and held to its finite range, whatever the
    sizes of queries and keys; a zero of either sign is a zero."""
    make, size = SCORES[what]
    nb = 65
    n = nb * PAGE - 3
    c = Case(1, Hq, 1, D, [n], seed=31)
    k = c.k.float()
    if what == "nothing left":   # some pages' scores are below zero by less than fp32 holds
        for j in range(nb):
            k[int(c.pt[0, j])] = k[int(c.pt[0, j])].abs() * _signs(nb)[j]
    c.k = (k * size).clamp(-3e38, 3e38).to(torch.bfloat16)
    c.q = make(torch.randn(Hq, D, generator=c.g)).to(torch.bfloat16).view(1, Hq, D)
    c.up()
    S.sfi_block_build(c.shape, c.kv, c.ix, 0, n)
    K = 12
    sel = torch.empty(1, 1, K, dtype=torch.int32, device=DEV)
    S.sfi_block_select(c.shape, c.ix, n, c.qd, 0, 1, K, sel, c.ws)
    assert c.error() == 0
    bounds, scale = zip(*(P.page_bounds(c.rows(c.k, 0, 0, n)[j * PAGE:(j + 1) * PAGE]) for j in range(nb - 1)))
    u = P.block_scores(c.q[0].double().numpy(), np.stack(bounds), np.array(scale))
    big = float(np.finfo(np.float32).max)
    u = np.append(np.clip(u, -big, big).astype(np.float32).astype(np.float64), 0.0)
    if what in ("nothing left", "1e38, large keys"):
        assert len(set(u)) < 5
    else:
        assert np.abs(u).max() < big and len(set(u)) > 30
    assert np.array_equal(sel[0, 0].cpu().numpy(), P.select(u, n, 0, 1, K))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top", [math.inf, P.BF16_MAX, 1.0])
def test_bounds_of_dimensions_far_apart(D, top):
    """A dimension whose values are far below the page's unit still gets outward bounds: 1 above
    zero, -1 below it."""
    c = Case(1, 2, 2, D, [32], seed=32)
    tiny = (1e-12, -1e-12, 1e-39, -1e-39, 0.0)
    for j in range(2):
        page = c.k[int(c.pt[0, j])]
        page[:, :, :5] = torch.tensor(tiny)
        page[:, 3, 7] = top * (1 - 2 * j)
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 32, index=c.ix)
    got = [(c.bounds.clone(), c.bscale.clone())]
    c.bounds.fill_(77)
    S.sfi_block_build(c.shape, c.kv, c.ix, 0, 32)
    got.append((c.bounds.clone(), c.bscale.clone()))
    assert c.error() == 0
    for bounds, scale in got:
        for j in range(2):
            p = int(c.pt[0, j])
            for h in range(2):
                codes, u = P.page_bounds(c.k[p, h].double().numpy())
                assert codes[0, 0] == 1 and codes[1, 1] == -1 and codes[0, 2] == 1 and codes[1, 3] == -1
                assert np.array_equal(bounds[p, h].cpu().numpy().astype(np.int64), codes), (j, h)
                assert float(scale[p, h]) == u


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("B,Hq,Hkv,D,lens", [
    (1, 3, 1, 64, [1]), (4, 6, 1, 128, [5, 16, 0, 17]), (1, 13, 1, 128, [300]), (2, 8, 2, 128, [5000, 31]),
    (1, 16, 1, 64, [9001])])
@pytest.mark.parametrize("equal", [False, True])
def test_values_near_the_largest(B, Hq, Hkv, D, lens, equal):
    """Values up to the largest bf16 one, in full pages and in the page that is not full, logits that rise
    along the sequence: the weighted mean is finite, and the output is it."""
    c = Case(B, Hq, Hkv, D, lens, seed=33, slack=1)
    size = torch.ones_like(c.v, dtype=torch.float64) if equal else torch.rand(c.v.shape, generator=c.g, dtype=torch.float64) * 0.5 + 0.5
    sign = 1.0 if equal else torch.where(torch.rand(c.v.shape, generator=c.g) < 0.3, -1.0, 1.0)
    c.v = (size * P.BF16_MAX * sign).to(torch.bfloat16)
    assert torch.isfinite(c.v).all()
    nb = -(-c.L // PAGE)
    for j in range(nb):
        for b in range(B):
            p = int(c.pt[b, j])
            c.k[p] = (c.k[p].float() * (0.3 + j / nb)).to(torch.bfloat16)
    sel = torch.arange(nb, dtype=torch.int32).flip(0).expand(B, Hkv, nb).contiguous().to(DEV)
    for fmt in FMTS:
        c.fmt = fmt
        c.up()
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
        K, V = {}, {}
        for b, n in enumerate(lens):
            for h in range(Hkv):
                K[b, h], V[b, h] = c.quant_rows("k", b, h, n), c.quant_rows("v", b, h, n)
        for call in (lambda: S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend, lse=c.lse),
                     lambda: S.sfi_quant_block_attn(c.shape, c.q8, c.L, c.qd, sel, nb, c.out, c.ws, lens=c.lend, lse=c.lse)):
            c.out.fill_(float("nan"))
            call()
            assert c.error() == 0
            assert torch.isfinite(c.out).all()
            check_all(c, lambda b, h, n: K[b, h], lambda b, h, n: V[b, h])
    c.out.fill_(float("nan"))
    S.sfi_block_attn(c.shape, c.kv, c.L, c.qd, sel, nb, c.out, c.ws, lens=c.lend, lse=c.lse)
    assert c.error() == 0
    assert torch.isfinite(c.out).all()
    check_all(c, lambda b, h, n: c.rows(c.k, b, h, n), lambda b, h, n: c.rows(c.v, b, h, n))


@pytest.mark.parametrize("Hq", [4, 16])
def test_one_block_of_the_largest_values_many_times(Hq):
    """The page that is not full, with values of the largest size, listed 500 times; and a full one."""
    K, n = 500, 40
    for block in (1, 2):
        c = Case(1, Hq, 1, 64, [n], "e4m3", seed=34, slack=K)
        c.v[:] = P.BF16_MAX
        c.up()
        sel = torch.full((1, 1, K), block, dtype=torch.int32, device=DEV)
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, n)
        kq, vq = c.quant_rows("k", 0, 0, n, [block]), c.quant_rows("v", 0, 0, n, [block])
        S.sfi_quant_block_attn(c.shape, c.q8, n, c.qd, sel, K, c.out, c.ws, lse=c.lse)
        assert c.error() == 0
        check_all(c, lambda b, h, m: np.concatenate([kq] * K), lambda b, h, m: np.concatenate([vq] * K))
        S.sfi_block_attn(c.shape, c.kv, n, c.qd, sel, K, c.out, c.ws, lse=c.lse)
        assert c.error() == 0
        check_all(c, lambda b, h, m: listed(c, c.k, b, h, m, [block] * K), lambda b, h, m: listed(c, c.v, b, h, m, [block] * K))


@pytest.mark.parametrize("Hq", [4, 8, 16])
def test_largest_values_without_weight(Hq):
    """Values of the largest size where the logits are hundreds lower: the others keep their precision,
    in 8-bit pages, in the page that is not full and in bf16 pages."""
    n, D = 12 * PAGE + 9, 64
    c = Case(1, Hq, 1, D, [n], "int8", seed=35)
    unit = torch.zeros(D)
    unit[0] = 1.0
    for j in range(13):
        p = int(c.pt[0, j])
        far = j in (1, 6)
        if far:
            c.v[p] = P.BF16_MAX
        c.k[p] = (c.k[p].float() * 0.3 + unit * (-300.0 if far else 0.0)).to(torch.bfloat16)
    c.q[0, :, 0] = 12.0
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, n)
    S.sfi_quant_attn(c.shape, c.q8, n, c.qd, c.out, c.ws, lse=c.lse)
    assert c.error() == 0
    assert float(c.out.abs().max()) < 10
    check_all(c, lambda b, h, m: c.quant_rows("k", b, h, m), lambda b, h, m: c.quant_rows("v", b, h, m))
    sel = torch.arange(13, dtype=torch.int32, device=DEV).view(1, 1, 13)
    S.sfi_block_attn(c.shape, c.kv, n, c.qd, sel, 13, c.out, c.ws, lse=c.lse)
    assert c.error() == 0
    check_all(c, lambda b, h, m: c.rows(c.k, b, h, m), lambda b, h, m: c.rows(c.v, b, h, m))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 7), (128, 16)])
@pytest.mark.parametrize("low,below", [((22.0, 30.0), [3, 7, 12, 20, 33, 50, 60, 63]), ((27.5, 28.0), [50, 52, 54, 56, 58, 60, 62, 63])])
def test_weights_of_pages_below_the_largest(fmt, D, Hq, low, below):
    """Pages whose value scales are 2 to 60 times below the largest, small weights on them, and nearly all the
    weight on a token whose values are zero.

    P times (scale / largest scale so far) is held as two fp16 parts, the second with steps of at least
    2^-24: off by at most 2^-25.  The largest P is at least 2^8 and the factor at least 2^-6 (pages below that
    take their factor behind the product), so a weight p = P / sum P is off by at most 2^-27 on top of what
    check_attn's other terms allow, or by itself where it is smaller."""
    below = [1] * 8 + below   # a page of the largest values first in each of up to 8 warps
    n = len(below) * PAGE
    c = Case(1, Hq, 1, D, [n], fmt, seed=36)
    unit = torch.zeros(D)
    unit[0] = 1.0
    for j, f in enumerate(below):
        p = int(c.pt[0, j])
        x = torch.randn(PAGE, D, generator=c.g)
        c.v[p, 0] = (x.abs() / x.abs().max() * (64.0 / f)).to(torch.bfloat16)
        # logits so far (in powers of two) below the largest one's
        less = low[0] + (low[1] - low[0]) * torch.rand(PAGE, 1, generator=c.g)
        c.k[p, 0] = (unit * (-less * math.log(2.0) * math.sqrt(D) / 8.0)).to(torch.bfloat16)
        if j < 8:
            c.k[p, 0] = (unit * -300.0).to(torch.bfloat16)    # the largest values: no weight at all
            c.k[p, 0, 0] = 0.0
            c.v[p, 0, 0] = 0.0
    c.q[:] = 0.0
    c.q[0, :, 0] = 8.0
    c.up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, n)
    K, V = c.quant_rows("k", 0, 0, n), c.quant_rows("v", 0, 0, n)
    nb = len(below)
    sel = torch.arange(nb, dtype=torch.int32, device=DEV).view(1, 1, nb)
    for call in (lambda: S.sfi_quant_attn(c.shape, c.q8, n, c.qd, c.out, c.ws),
                 lambda: S.sfi_quant_block_attn(c.shape, c.q8, n, c.qd, sel, nb, c.out, c.ws)):
        c.out.fill_(float("nan"))
        call()
        assert c.error() == 0
        q = c.q[0].double().numpy()
        o, _, pv, s = P.attention(q, K, V)
        dz = (D / 16 + 2) * 2.0 ** -23 * s + 2.0 ** -22 * s
        rel = 2.0 ** -16 + 2 * dz + (nb + 64) * 2.0 ** -23
        z = q @ K.T / math.sqrt(D)
        p = np.exp(z - z.max(1, keepdims=True))
        got = c.out[0].cpu().double().numpy()
        assert np.all(np.abs(got - o) <= rel[:, None] * pv + np.minimum(2.0 ** -27, p) @ np.abs(V) + 1e-30)
