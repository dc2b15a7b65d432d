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
