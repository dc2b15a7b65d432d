"""Block selection over rows longer than one CTA's shared memory; ranges, bad pages and bad
lengths of the cache calls; a workspace that was not zero."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as P
from slow_sparse_kv_sfi_b200 import sfi as S

from test_gpu_pages import DEV, FMTS, PAGE, Case

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


# ------------------------------------------------------------------ ranges of sfi_quant_load, bad pages
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 2)])
@pytest.mark.parametrize("lo", [16, 32, 64])
def test_load_from_a_later_page(fmt, D, Hkv, lo):
    """[pos_lo, len) of every sequence, whether it ends before pos_lo, there, inside its page or later;
    every other row is left alone."""
    lens = [100, lo - 5, lo, lo + 7, 0, 96, lo + 16]
    c = Case(len(lens), Hkv, Hkv, D, lens, fmt, seed=42, slack=1).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    k2, v2 = torch.full_like(c.kd, 9.0), torch.full_like(c.vd, 9.0)
    S.sfi_quant_load(c.shape, c.q8, S.make_kv(k2, v2, c.ptd, None, c.err), lo, c.L, lens=c.lend)
    assert c.error() == 0
    want_k, want_v = torch.full_like(c.k, 9.0), torch.full_like(c.v, 9.0)
    for b, n in enumerate(lens):
        for want, which in ((want_k, "k"), (want_v, "v")):
            for h in range(Hkv):
                rows = torch.from_numpy(c.quant_rows(which, b, h, n)).float().to(torch.bfloat16)
                for t in range(lo, n):
                    want[int(c.pt[b, t // PAGE]), h, t % PAGE] = rows[t]
    assert torch.equal(k2.cpu(), want_k) and torch.equal(v2.cpu(), want_v)


@pytest.mark.parametrize("fmt", FMTS)
def test_load_with_bad_pages_and_lengths(fmt):
    """A page number outside the pool, in either table, and a length outside [0, L]: latched, and what
    they name is passed over."""
    lens = [60, 48]
    c = Case(2, 2, 2, 64, lens, fmt, seed=43, slack=1).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    good_k, good_v = torch.full_like(c.kd, 9.0), torch.full_like(c.vd, 9.0)
    S.sfi_quant_load(c.shape, c.q8, S.make_kv(good_k, good_v, c.ptd, None, c.err), 0, c.L, lens=c.lend)
    assert c.error() == 0
    err2 = torch.zeros(1, dtype=torch.int32, device=DEV)
    for bad in (-1, c.n, 2 ** 31 - 1):
        other = c.ptd.clone()
        other[0, 1] = bad
        want_k, want_v = good_k.clone(), good_v.clone()
        want_k[int(c.pt[0, 1])] = 9.0
        want_v[int(c.pt[0, 1])] = 9.0
        for where in ("target", "source"):
            k2, v2 = torch.full_like(c.kd, 9.0), torch.full_like(c.vd, 9.0)
            kv2 = S.make_kv(k2, v2, other if where == "target" else c.ptd, None, err2)
            q2 = S.make_quant_kv(c.kc, c.vc, c.ks, c.vs, c.ktail, c.vtail, other if where == "source" else c.ptd,
                                 c.q8.format, c.err)
            S.sfi_quant_load(c.shape, q2, kv2, 0, c.L, lens=c.lend)
            assert S.sfi_quant_poll_error(q2) == (5 | (13 << 8) if where == "source" else 0)
            assert S.sfi_poll_error(kv2) == (5 | (13 << 8) if where == "target" else 0)
            assert torch.equal(k2, want_k) and torch.equal(v2, want_v)
    for bad in (-3, c.L + 1, 2 ** 31 - 1):
        k2, v2 = torch.full_like(c.kd, 9.0), torch.full_like(c.vd, 9.0)
        ln = torch.tensor([bad, 48], dtype=torch.int32, device=DEV)
        S.sfi_quant_load(c.shape, c.q8, S.make_kv(k2, v2, c.ptd, None, err2), 0, c.L, lens=ln)
        assert S.sfi_quant_poll_error(c.q8) == 5 | (12 << 8)
        want_k = torch.full_like(c.kd, 9.0)
        for j in range(3):
            want_k[int(c.pt[1, j])] = good_k[int(c.pt[1, j])]
        assert torch.equal(k2, want_k)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_that_fills_a_page_nobody_has(fmt):
    """The page number is looked up when the page fills: a bad one is latched, the token still reaches
    the tail, and no page is written; the other sequence's page and a sound index are."""
    c = Case(2, 4, 2, 128, [32, 32], fmt, seed=44).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, 31, index=c.ix)
    tok_k = torch.stack([c.kd[int(c.pt[b, 1]), :, 15] for b in range(2)]).contiguous()
    tok_v = torch.stack([c.vd[int(c.pt[b, 1]), :, 15] for b in range(2)]).contiguous()
    before = c.kc.clone(), c.vc.clone(), c.ks.clone(), c.bounds.clone()
    for bad in (-1, c.n, 2 ** 31 - 1):
        other = c.ptd.clone()
        other[0, 1] = bad
        for table, index_table in ((other, c.ptd), (c.ptd, other)):
            c.kc.copy_(before[0]), c.vc.copy_(before[1]), c.ks.copy_(before[2]), c.bounds.copy_(before[3])
            ix_err = torch.zeros(1, dtype=torch.int32, device=DEV)
            q2 = S.make_quant_kv(c.kc, c.vc, c.ks, c.vs, c.ktail, c.vtail, table, c.q8.format, c.err)
            ix = S.make_block_index(c.bounds, c.bscale, index_table, ix_err)
            S.sfi_quant_append(c.shape, q2, 32, tok_k, tok_v, index=ix)
            code = 5 | (13 << 8)
            assert S.sfi_quant_poll_error(q2) == (code if table is other else 0)
            assert int(ix_err.item()) == (code if index_table is other else 0)
            p0, p1 = int(c.pt[0, 1]), int(c.pt[1, 1])
            assert torch.equal(c.ktail[:, :, 15], tok_k) and torch.equal(c.vtail[:, :, 15], tok_v)
            changed = (c.kc != before[0]).flatten(1).any(1)
            assert bool(changed[p1]) and bool(changed[p0]) == (table is not other) and int(changed.sum()) == 1 + (table is not other)
            seen = (c.bounds != before[3]).flatten(1).any(1)
            assert bool(seen[p1]) and bool(seen[p0]) == (index_table is not other) and int(seen.sum()) == 1 + (index_table is not other)


@pytest.mark.parametrize("fill", [0x7F, 0xFF, 0x01])
def test_workspace_that_was_not_zero_is_latched(fill):
    """Counts that no call can have left: latched, whatever the number of a row's pieces; after a zero fill
    the call gives its result again."""
    c = Case(2, 8, 2, 64, [4000, 1500], "int8", seed=45).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend)
    assert c.error() == 0
    want = c.out.clone()
    c.ws.fill_(fill)
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend)
    assert c.error() == 5 | (16 << 8)
    c.ws.zero_()
    c.out.fill_(float("nan"))
    S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.out, c.ws, lens=c.lend)
    assert c.error() == 0
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("D,Hq,Hkv,nb,K", [(64, 2, 1, 262144, 1000), (64, 80, 80, 33000, 30), (128, 40, 40, 131073, 50)])
def test_select_longest_and_many_long_rows(D, Hq, Hkv, nb, K):
    """The most blocks there may be, and so many long rows that they do not all run at once."""
    g = torch.Generator().manual_seed(46)
    pool = 300
    bounds = torch.randint(-127, 128, (pool, Hkv, 2, D), generator=g).to(torch.int8)
    bounds = torch.stack([bounds.amax(2), bounds.amin(2)], dim=2)
    scale = torch.exp2(torch.randint(-3, 3, (pool, Hkv), generator=g).float())
    pt = torch.randint(0, pool, (1, nb), generator=g, dtype=torch.int32)
    q = (torch.randn(1, Hq, D, generator=g) * 3).to(torch.bfloat16)
    shape = S.make_shape(1, Hq, Hkv, D, nb, pool)
    d = [t.to(DEV).contiguous() for t in (bounds, scale, pt)]
    ix = S.make_block_index(*d)
    ws = torch.zeros(S.sfi_block_workspace_size(shape), dtype=torch.uint8, device=DEV)
    sel = torch.empty(1, Hkv, K, dtype=torch.int32, device=DEV)
    n = nb * PAGE - 1
    S.sfi_block_select(shape, ix, n, q.to(DEV), 4, 64, K, sel, ws)
    torch.cuda.synchronize()
    G = Hq // Hkv
    for h in range(Hkv):
        u = P.block_scores(q[0, h * G:(h + 1) * G].double().numpy(), bounds[:, h].numpy().astype(np.int64),
                           scale[:, h].double().numpy())[pt[0].numpy()]
        assert np.array_equal(sel[0, h].cpu().numpy(), P.select(u, n, 4, 64, K)), h
    if nb == 262144:
        one = S.make_shape(1, Hq, Hkv, D, nb + 1, pool)
        ws = torch.zeros(S.sfi_block_workspace_size(one), dtype=torch.uint8, device=DEV)
        more = S.make_block_index(d[0], d[1], torch.zeros(1, nb + 1, dtype=torch.int32, device=DEV))
        with pytest.raises(S.SFIError):
            S.sfi_block_select(one, more, nb * PAGE + 1, q.to(DEV), 4, 64, K, sel, ws)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 16)])
@pytest.mark.parametrize("ragged", [False, True])
def test_attention_over_four_million_tokens(fmt, D, Hq, ragged):
    """A row of 262145 pages (a few different ones, many times each) beside a short one: the definition with
    every page counted as often as it occurs.  Sums of n tokens lose at most (tiles of a warp + pieces + 64)
    steps of 2^-23: 262145 tiles over 148 or more CTAs of 4 or more warps, 443 a warp at most, and as many
    pieces."""
    nb, pool = 262145, 40
    n = nb * PAGE - 11                       # the last page is not full
    lens = [n, 20] if ragged else [n]
    B = len(lens)
    c = Case(B, Hq, 1, D, [pool * PAGE] + [20] * (B - 1), fmt, seed=47, spare=0).up()
    S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend)
    own = c.pt[0].long()
    pick = torch.randint(0, pool, (nb,), generator=c.g)
    pt = torch.zeros(B, nb, dtype=torch.int32)
    pt[0] = own[pick].to(torch.int32)
    if ragged:
        pt[1, :2] = c.pt[1, :2]
    ptd = pt.to(DEV)
    shape = S.make_shape(B, Hq, 1, D, nb, c.n)
    kt, vt = (torch.randn(B, 1, PAGE, D, generator=c.g).to(torch.bfloat16) for _ in range(2))
    ktd, vtd = kt.to(DEV), vt.to(DEV)
    if ragged:
        ktd[1], vtd[1] = c.ktail[1], c.vtail[1]
    q8 = S.make_quant_kv(c.kc, c.vc, c.ks, c.vs, ktd, vtd, ptd, c.q8.format, c.err)
    ws = torch.zeros(S.sfi_block_workspace_size(shape), dtype=torch.uint8, device=DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV) if ragged else None
    S.sfi_quant_attn(shape, q8, n, c.qd, c.out, ws, lens=ln, lse=c.lse)
    assert c.error() == 0
    K, V = c.quant_rows("k", 0, 0, pool * PAGE), c.quant_rows("v", 0, 0, pool * PAGE)
    times = np.bincount(pick[:nb - 1].numpy(), minlength=pool).astype(np.float64).repeat(PAGE)
    K = np.concatenate([K, kt[0, 0, :5].double().numpy()])
    V = np.concatenate([V, vt[0, 0, :5].double().numpy()])
    times = np.concatenate([times, np.ones(5)])
    q = c.q[0].double().numpy()
    z = q @ K.T / np.sqrt(D)
    m = z.max(1, keepdims=True)
    w = np.exp(z - m) * times
    total = w.sum(1, keepdims=True)
    o, pv = w @ V / total, w @ np.abs(V) / total
    s = (np.abs(q) @ np.abs(K).T).max(1) / np.sqrt(D)
    dz = (D / 16 + 2) * 2.0 ** -23 * s + 2.0 ** -22 * s
    steps = (2 * 443 + 64) * 2.0 ** -23
    tol = (2.0 ** -16 + 2 * dz + steps)[:, None] * pv + np.minimum(2.0 ** -27, w / times / total) @ (times[:, None] * np.abs(V))
    assert np.all(np.abs(c.out[0].cpu().double().numpy() - o) <= tol)
    lse = (m + np.log(total))[:, 0]
    assert np.all(np.abs(c.lse[0].cpu().double().numpy() - lse) <= 2 * dz + steps + 2.0 ** -22 * np.abs(lse))
    if ragged:
        o, _, pv, s = P.attention(c.q[1].double().numpy(), c.quant_rows("k", 1, 0, 20), c.quant_rows("v", 1, 0, 20))
        assert np.all(np.abs(c.out[1].cpu().double().numpy() - o) <= 1e-4 * pv)


def test_two_streams_with_workspaces_of_their_own():
    """append -> select -> attend on two streams at once, each with its own workspace: the results of each
    alone."""
    cs = [Case(2, 16, 4, 128, [3000, 900], "e4m3", seed=48).up(), Case(3, 8, 2, 64, [2000, 64, 5000], "int8", seed=49).up()]
    K = 12
    sels = [torch.zeros(c.B, c.Hkv, K, dtype=torch.int32, device=DEV) for c in cs]

    def step(c, sel, stream=None):
        S.sfi_quant_append(c.shape, c.q8, c.L, c.kd[:c.B, :, 0].contiguous(), c.vd[:c.B, :, 0].contiguous(), lens=c.lend,
                           index=c.ix, stream=stream)
        S.sfi_block_select(c.shape, c.ix, c.L, c.qd, 4, 20, K, sel, c.ws, lens=c.lend, stream=stream)
        S.sfi_quant_block_attn(c.shape, c.q8, c.L, c.qd, sel, K, c.out, c.ws, lens=c.lend, lse=c.lse, stream=stream)
        S.sfi_quant_attn(c.shape, c.q8, c.L, c.qd, c.full, c.ws, lens=c.lend, stream=stream)

    want = []
    for c, sel in zip(cs, sels):
        c.full = torch.empty_like(c.out)
        S.sfi_quant_store(c.shape, c.kv, c.q8, 0, c.L, lens=c.lend - 1, index=c.ix)
        step(c, sel)
        torch.cuda.synchronize()
        want.append([x.clone() for x in (sel, c.out, c.lse, c.full)])
        for x in (sel, c.out, c.lse, c.full):
            x.fill_(-7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(25):
        for c, sel, st in zip(cs, sels, streams):
            with torch.cuda.stream(st):
                step(c, sel, st)
    torch.cuda.synchronize()
    for c, sel, w in zip(cs, sels, want):
        assert c.error() == 0
        for x, y in zip((sel, c.out, c.lse, c.full), w):
            assert torch.equal(x, y)
