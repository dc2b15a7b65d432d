"""Block selection over rows longer than one CTA's shared memory."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as P
from slow_sparse_kv_sfi_b200 import sfi as S

from test_gpu_pages import DEV, PAGE

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection, more than 16384 blocks
@pytest.mark.parametrize("D,Hq,Hkv,blocks,K", [
    (64, 2, 1, [16385], 40), (128, 12, 1, [16390, 0, 900], 1000), (64, 16, 1, [20001, 700, 16384, 3], 9000),
    (128, 8, 2, [40000, 1, 39999], 5000), (64, 3, 3, [70003], 700)])
@pytest.mark.parametrize("what", ["mixed", "ties", "bad pages"])
def test_select_long_rows(D, Hq, Hkv, blocks, K, what):
    """Rows scored by one kernel and selected by another: ragged lengths, sequences that are empty or shorter
    than K blocks, equal scores, pages that cannot be read; nothing behind the workspace is written."""
    B, G = len(blocks), Hq // Hkv
    lens = [max(n * PAGE - 5 * (b % 2), 0) for b, n in enumerate(blocks)]
    L, nb, pool = max(lens), max(blocks), 512
    g = torch.Generator().manual_seed(41)
    bounds = torch.randint(-127, 128, (pool, Hkv, 2, D), generator=g).to(torch.int8)
    bounds = torch.stack([bounds.amax(2), bounds.amin(2)], dim=2)
    scale = torch.exp2(torch.randint(-6, 3, (pool, Hkv), generator=g).float())
    if what == "ties":
        bounds, scale = bounds[:2].repeat(pool // 2, 1, 1, 1), torch.ones(pool, Hkv)
    pt = torch.randint(0, pool, (B, nb + 3), generator=g, dtype=torch.int32)
    bad = torch.zeros(B, nb + 3, dtype=torch.bool)
    if what == "bad pages":
        bad[:, ::97] = True
        pt[bad] = torch.tensor([-1, pool, 2 ** 31 - 1], dtype=torch.int32).repeat(int(bad.sum()) // 3 + 1)[:int(bad.sum())]
    q = (torch.randn(B, Hq, D, generator=g) * 3).to(torch.bfloat16)
    shape = S.make_shape(B, Hq, Hkv, D, nb + 3, pool)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = [t.to(DEV).contiguous() for t in (bounds, scale, pt)]
    ix = S.make_block_index(*d, err=err)
    need = S.sfi_block_workspace_size(shape)
    big = torch.zeros(need + (1 << 20), dtype=torch.uint8, device=DEV)
    big[need:] = 0x3C
    sel = torch.full((B, Hkv, K + 2), -7, dtype=torch.int32, device=DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    n_sink, n_recent = 20, 70
    S.sfi_block_select(shape, ix, L, q.to(DEV), n_sink, n_recent, K, sel, big[:need], lens=ln)
    torch.cuda.synchronize()
    assert (big[need:] == 0x3C).all()
    first = sel.clone()
    S.sfi_block_select(shape, ix, L, q.to(DEV), n_sink, n_recent, K, sel, big[:need], lens=ln)
    torch.cuda.synchronize()
    assert torch.equal(first, sel)
    got = sel.cpu().numpy()
    assert (got[..., K:] == -7).all()
    reached = False
    j = np.arange(nb)
    for b in range(B):
        read = (j * PAGE < lens[b]) & (j * PAGE >= n_sink) & ((j + 1) * PAGE <= lens[b] - n_recent)
        reached |= bool((read & bad[b, :nb].numpy()).any())
        for h in range(Hkv):
            pages = pt[b, :nb].clamp(0, pool - 1).long()
            # (a page's score once, then by page number)
            u = P.block_scores(q[b, h * G:(h + 1) * G].double().numpy(), bounds[:, h].numpy().astype(np.int64),
                               scale[:, h].double().numpy())[pages.numpy()]
            u = np.where(bad[b, :nb].numpy(), -np.inf, u)
            assert np.array_equal(got[b, h, :K], P.select(u, lens[b], n_sink, n_recent, K)), (b, h)
    assert int(err.item()) == ((5 | (14 << 8)) if reached else 0)
    assert reached == (what == "bad pages")
