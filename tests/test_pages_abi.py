"""Host-side refusals of the 8-bit cache and block-sparse calls, and the pins
of their oracle; nothing here touches a GPU."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import pages_oracle as P


@pytest.fixture(scope="module")
def S():
    from slow_sparse_kv_sfi_b200 import build, sfi
    build.build()
    sfi.lib()
    return sfi


def _quant(S, **kw):
    f = dict(k_pool=32, v_pool=32, k_scale=16, v_scale=16, k_tail=16, v_tail=16, page_table=16, err=None, format=0)
    f.update(kw)
    return S.QuantKV(**f)


def _calls(S, sh, q8, kv, ix, L, q=16, out=16, sel=16, K=4, ld=4, n_sink=4, n_recent=16, ws=16, wsb=1 << 30, tok=16,
           lo=0):
    r = C.byref
    lib = S.lib()
    n = lambda x: None if x is None else r(x)  # noqa: E731
    return {
        "store": lambda: lib.sfi_quant_store(n(sh), n(kv), n(q8), n(ix), lo, L, None, None),
        "append": lambda: lib.sfi_quant_append(n(sh), n(q8), n(ix), L, None, tok, tok, None),
        "load": lambda: lib.sfi_quant_load(n(sh), n(q8), n(kv), lo, L, None, None),
        "attn": lambda: lib.sfi_quant_attn(n(sh), n(q8), L, None, q, out, None, ws, wsb, None),
        "build": lambda: lib.sfi_block_build(n(sh), n(kv), n(ix), lo, L, None, None),
        "select": lambda: lib.sfi_block_select(n(sh), n(ix), L, None, q, n_sink, n_recent, K, sel, ld, ws, wsb, None),
        "block": lambda: lib.sfi_block_attn(n(sh), n(kv), L, None, q, sel, ld, K, out, None, ws, wsb, None),
        "qblock": lambda: lib.sfi_quant_block_attn(n(sh), n(q8), L, None, q, sel, ld, K, out, None, ws, wsb, None),
    }


ALL = ["store", "append", "load", "attn", "build", "select", "block", "qblock"]


def _ok(S):
    return dict(sh=S.make_shape(1, 4, 2, 64, 10, 10), q8=_quant(S), kv=S.PagedKV(32, 32, 16, None, None),
                ix=S.BlockIndex(16, 16, 16, None), L=100)


@pytest.mark.parametrize("name", ALL)
def test_shapes_are_refused(S, name):
    for sh, code in ((None, 1), (S.make_shape(1, 4, 3, 64, 10, 10), 2), (S.make_shape(1, 4, 2, 96, 10, 10), 3),
                     (S.make_shape(1, 32, 1, 64, 10, 10), 3), (S.make_shape(0, 4, 2, 64, 10, 10), 2)):
        a = _ok(S)
        a["sh"] = sh
        assert _calls(S, **a)[name]() == code
    a = _ok(S)
    a["L"] = 161                                         # longer than the page table
    assert _calls(S, **a)[name]() == 2
    a["L"] = -1
    assert _calls(S, **a)[name]() == 2


@pytest.mark.parametrize("field", ["k_pool", "v_pool", "k_scale", "v_scale", "k_tail", "v_tail", "page_table"])
def test_quant_cache_pointers_are_refused(S, field):
    for name in ("store", "append", "load", "attn", "qblock"):
        a = _ok(S)
        a["q8"] = _quant(S, **{field: None})
        assert _calls(S, **a)[name]() == 1
        if field not in ("k_scale", "v_scale", "page_table"):
            # pools 32-byte aligned, tails 16
            a["q8"] = _quant(S, **{field: 16 if field.endswith("pool") else 24})
            assert _calls(S, **a)[name]() == 1
        a["q8"] = None
        assert _calls(S, **a)[name]() == 1


def test_formats_ranges_and_pointers_are_refused(S):
    a = _ok(S)
    for name in ("store", "append", "load", "attn", "qblock"):
        assert _calls(S, **{**a, "q8": _quant(S, format=2)})[name]() == 3
    for name in ("store", "load", "build"):
        assert _calls(S, lo=8, **a)[name]() == 2         # pos_lo not a multiple of 16
        assert _calls(S, lo=-16, **a)[name]() == 2
        assert _calls(S, lo=112, **a)[name]() == 0       # an empty range: nothing to do
        assert _calls(S, **{**a, "L": 0})[name]() == 0
        assert _calls(S, **{**a, "kv": S.PagedKV(16, 24, 16, None, None)})[name]() == 1
    for name in ("append", "attn", "select", "block", "qblock"):
        assert _calls(S, **{**a, "L": 0})[name]() == 2
    assert _calls(S, tok=None, **a)["append"]() == 1
    assert _calls(S, tok=24, **a)["append"]() == 1
    for name in ("store", "append", "build", "select"):
        assert _calls(S, **{**a, "ix": S.BlockIndex(24, 16, 16, None)})[name]() == 1
        assert _calls(S, **{**a, "ix": S.BlockIndex(16, None, 16, None)})[name]() == 1
        assert _calls(S, **{**a, "ix": S.BlockIndex(16, 16, None, None)})[name]() == 1
    for name in ("build", "select"):
        assert _calls(S, **{**a, "ix": None})[name]() == 1
    for name in ("attn", "select", "block", "qblock"):
        assert _calls(S, q=None, **a)[name]() == 1
        assert _calls(S, q=24, **a)[name]() == 1
        assert _calls(S, ws=None, **a)[name]() == 7
        assert _calls(S, ws=24, **a)[name]() == 7
        assert _calls(S, wsb=64, **a)[name]() == 7
    for name in ("attn", "block", "qblock"):
        assert _calls(S, out=None, **a)[name]() == 1
    for name in ("select", "block", "qblock"):
        assert _calls(S, sel=None, **a)[name]() == 1
        assert _calls(S, K=0, **a)[name]() == 2
        assert _calls(S, K=5, ld=4, **a)[name]() == 2
    assert _calls(S, K=8, ld=8, **a)["select"]() == 2    # more than ceil(100 / 16) = 7 blocks
    assert _calls(S, K=2, ld=8, **a)["select"]() == 2    # fewer than the 3 always taken
    assert _calls(S, n_recent=0, **a)["select"]() == 2
    assert _calls(S, n_sink=-1, **a)["select"]() == 2
    assert _calls(S, **{**a, "kv": S.PagedKV(32, 16, 16, None, None)})["block"]() == 1
    assert _calls(S, K=11, ld=11, **a)["block"]() == 2   # more entries than pages of a sequence
    assert S.lib().sfi_quant_poll_error(None, C.byref(C.c_int32())) == 1
    assert S.lib().sfi_block_workspace_size(C.byref(a["sh"]), None) == 1
    big = S.make_shape(40000, 4, 2, 64, 10, 10)
    for name in ("attn", "select", "block", "qblock"):   # more (sequence, head) pairs than a grid holds
        assert _calls(S, **{**a, "sh": big})[name]() == 3


def test_workspace_grows_with_the_cache(S):
    small = S.sfi_block_workspace_size(S.make_shape(1, 4, 2, 64, 10, 10))
    assert 0 < small < S.sfi_block_workspace_size(S.make_shape(1, 4, 2, 64, 1000, 1000))


def test_python_tensor_checks(S):
    z = torch.zeros
    with pytest.raises(ValueError, match="dtype"):
        S._arg(z(4), "x", (torch.int32,))
    with pytest.raises(ValueError, match="shape"):
        S._arg(z(4), "x", (torch.float32,), (5,))
    with pytest.raises(ValueError, match="contiguous"):
        S._arg(z(4, 4).t(), "x", (torch.float32,))
    with pytest.raises(ValueError, match="device"):
        S._arg(z(4), "x", (torch.float32,))
    ix = S.BlockIndex(16, 16, 16, None)
    ix.dims = (1, 2, 64, 10, 11)
    with pytest.raises(ValueError, match="num_pages"):
        S._dims(S.make_shape(1, 4, 2, 64, 10, 10), ix)


# ------------------------------------------------------------------ oracle pins
def test_oracle_e4m3_table():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(P.e4m3_values(), want)


def test_oracle_unit_and_bounds():
    assert P.unit(127.0) == 1.0 and P.unit(127.5) == 2.0 and P.unit(63.5) == 0.5 and P.unit(0.0) == 2.0 ** -126
    k = np.array([[254.0, -3.0], [2.0, 5.0]])
    codes, u = P.page_bounds(k)
    assert u == 2.0 and codes.tolist() == [[127, 3], [1, -2]]


def test_oracle_score_by_hand():
    # q = [1, -2]: 2 > 127 * 2^-6, so the unit is 2^-5 and the codes are 32, -64
    q = np.array([[1.0, -2.0]])
    e = P.unit(2.0)
    assert e == 2.0 ** -5
    b = np.array([[[10, 4], [-10, -3]]])
    # max(32 * 10, 32 * -10) + max(-64 * 4, -64 * -3) = 320 + 192
    assert P.block_scores(q, b, np.array([0.5]))[0] == 512 * e * 0.5


def test_oracle_select_forced_and_ties():
    u = np.array([0.0, 5.0, 1.0, 5.0, 5.0, 0.0, 9.0])
    # 100 tokens: blocks 5 (tokens 80..95) and 6 hold the last 16; block 0 the first 4
    assert P.select(u, 100, 4, 16, 5).tolist() == [0, 1, 3, 5, 6]
    assert P.select(u, 20, 4, 16, 3).tolist() == [0, 1, 2]
    assert P.select(u, 0, 4, 16, 2).tolist() == [0, 1]


def test_oracle_attention_matches_torch():
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(3, 64)), g.normal(size=(21, 64)), g.normal(size=(21, 64))
    o, lse, _, _ = P.attention(q, k, v)
    z = torch.tensor(q @ k.T) / math.sqrt(64)
    np.testing.assert_allclose(o, (torch.softmax(z, -1) @ torch.tensor(v)).numpy(), rtol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(z, -1).numpy(), rtol=1e-12)
    assert np.all(P.attention(q, k[:0], v[:0])[0] == 0)
