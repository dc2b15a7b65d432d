"""What the Python calls of the 8-bit cache and the block index refuse before anything is launched."""
import pytest
import torch

from slow_sparse_kv_sfi_b200 import sfi as S

B, HKV, D, PAGES, N = 2, 3, 64, 5, 11


def _kv(n=N, hkv=HKV, d=D, b=B, pages=PAGES, **kw):
    z = torch.zeros
    f = dict(k=z(n, hkv, 16, d, dtype=torch.bfloat16), v=z(n, hkv, 16, d, dtype=torch.bfloat16),
             pt=z(b, pages, dtype=torch.int32))
    f.update(kw)
    return S.make_kv(f["k"], f["v"], f["pt"])


def test_bf16_cache_of_other_sizes_is_refused():
    shape = S.make_shape(B, 2 * HKV, HKV, D, PAGES, N)
    S._dims(shape, _kv())
    S._dims(shape, S.PagedKV(16, 16, 16, None, None))     # made of addresses: the caller's word
    S._dims(shape, _kv(n=N + 1, b=B + 1))                  # more pages and sequences than the layer uses
    for kw in (dict(n=N - 1), dict(hkv=1), dict(d=128), dict(b=1), dict(pages=PAGES - 1), dict(pages=PAGES + 1)):
        with pytest.raises(ValueError, match="PagedKV"):
            S._dims(shape, _kv(**kw))


def test_bf16_cache_of_other_tensors_is_refused():
    shape = S.make_shape(B, 2 * HKV, HKV, D, PAGES, N)
    z = torch.zeros
    for kw in (dict(k=z(N, HKV, 16, D)), dict(v=z(N, HKV, 16, D, dtype=torch.float16)),
               dict(v=z(N - 1, HKV, 16, D, dtype=torch.bfloat16)),
               dict(k=z(N, HKV, D, 16, dtype=torch.bfloat16).transpose(2, 3)),
               dict(k=z(N, HKV, 8, D, dtype=torch.bfloat16), v=z(N, HKV, 8, D, dtype=torch.bfloat16)),
               dict(pt=z(B, PAGES, dtype=torch.int64)), dict(pt=z(PAGES, B, dtype=torch.int32).t()),
               dict(pt=z(B * PAGES, dtype=torch.int32))):
        with pytest.raises(ValueError, match="PagedKV"):
            S._dims(shape, _kv(**kw))


def test_a_part_of_another_device_is_refused():
    shape = S.make_shape(B, 2 * HKV, HKV, D, PAGES, N)
    with pytest.raises(ValueError, match="device"):
        S._dims(shape, _kv(), dev=0)
    ix = S.BlockIndex(16, 16, 16, None)
    ix.dims, ix.device = (B, HKV, D, PAGES, N), 1
    with pytest.raises(ValueError, match="device"):
        S._dims(shape, ix, dev=0)
    S._dims(shape, ix, dev=1)


@pytest.mark.parametrize("fmt,dtype", [("FMT_E4M3", torch.int8), ("FMT_INT8", torch.float8_e4m3fn),
                                       ("FMT_INT8", torch.float32)])
def test_pools_of_the_other_format_are_refused(fmt, dtype):
    z = torch.zeros
    pool = z(N, HKV, 16, D).to(dtype)
    s, t = z(N, HKV), z(B, HKV, 16, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dtype"):
        S.make_quant_kv(pool, pool, s, s, t, t, z(B, PAGES, dtype=torch.int32), getattr(S, fmt))
    u8 = z(N, HKV, 16, D, dtype=torch.uint8)
    with pytest.raises(ValueError, match="fmt"):
        S.make_quant_kv(u8, u8, s, s, t, t, z(B, PAGES, dtype=torch.int32), 2)


@pytest.mark.gpu
def test_calls_refuse_a_cache_that_is_not_the_shapes():
    """Every call that takes the bf16 cache; nothing is launched."""
    dev, z = "cuda", torch.zeros
    shape = S.make_shape(B, 2 * HKV, HKV, D, PAGES, N)
    pt = z(B, PAGES, dtype=torch.int32, device=dev)
    q8 = S.make_quant_kv(z(N, HKV, 16, D, dtype=torch.uint8, device=dev), z(N, HKV, 16, D, dtype=torch.uint8, device=dev),
                         z(N, HKV, device=dev), z(N, HKV, device=dev), z(B, HKV, 16, D, dtype=torch.bfloat16, device=dev),
                         z(B, HKV, 16, D, dtype=torch.bfloat16, device=dev), pt, S.FMT_INT8)
    ix = S.make_block_index(z(N, HKV, 2, D, dtype=torch.int8, device=dev), z(N, HKV, device=dev), pt)
    pool = z(N - 4, HKV, 16, D, dtype=torch.bfloat16, device=dev)
    kv = S.make_kv(pool, pool.clone(), pt)
    q, out = z(B, 2 * HKV, D, dtype=torch.bfloat16, device=dev), z(B, 2 * HKV, D, device=dev)
    sel, ws = z(B, HKV, 2, dtype=torch.int32, device=dev), z(S.sfi_block_workspace_size(shape), dtype=torch.uint8, device=dev)
    for call in (lambda: S.sfi_quant_store(shape, kv, q8, 0, 40), lambda: S.sfi_quant_load(shape, q8, kv, 0, 40),
                 lambda: S.sfi_block_build(shape, kv, ix, 0, 40),
                 lambda: S.sfi_block_attn(shape, kv, 40, q, sel, 2, out, ws)):
        with pytest.raises(ValueError, match="num_pages"):
            call()
    torch.cuda.synchronize()
