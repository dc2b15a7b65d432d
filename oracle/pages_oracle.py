"""CPU oracle for the 8-bit paged cache and the block-sparse attention.

TEST INFRASTRUCTURE ONLY, like sfi_oracle: plain numpy float64, no code shared
with the CUDA path.  bf16 inputs are converted to float64 exactly.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}
AMAX_FLOOR = 2.0 ** -100
BF16_MAX = float(np.uint32(0x7F7F0000).view(np.float32))


def e4m3_values() -> np.ndarray:
    """Value of every e4m3 code (0x7f and 0xff: NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else (-v if s else v)
    return out


def code_values(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Values of uint8 codes, before the scale."""
    if fmt == "e4m3":
        return e4m3_values()[codes]
    return codes.view(np.int8).astype(np.float64)


def page_scale(x: np.ndarray, fmt: str) -> float:
    """Scale of one page x [16, D]: NaN when a value is not finite."""
    if not np.isfinite(x).all():
        return math.nan
    return max(np.abs(x).max(), AMAX_FLOOR) / QMAX[fmt]


def half_step(x: np.ndarray, scale: float, fmt: str) -> np.ndarray:
    """Half the spacing of the codes' values around each x of a page."""
    if fmt == "int8":
        return np.full(x.shape, 0.5 * scale)
    e = np.floor(np.log2(np.maximum(np.abs(x) / scale, 2.0 ** -6)))
    return 0.5 * 2.0 ** (e - 3) * scale


def unit(amax: float) -> float:
    """Smallest power of two u >= 2^-126 with amax <= 127 u."""
    e = -126
    while amax > 127.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def tame(x: np.ndarray) -> np.ndarray:
    """NaN -> 0, infinities -> the largest finite bf16."""
    return np.clip(np.where(np.isnan(x), 0.0, x), -BF16_MAX, BF16_MAX)


def page_bounds(k: np.ndarray):
    """(hi, lo) codes [2, D] and the scale of one page's keys k [16, D]."""
    k = tame(k)
    hi, lo = k.max(0), k.min(0)
    u = unit(max(np.abs(hi).max(), np.abs(lo).max()))
    return np.stack([np.ceil(hi / u), np.floor(lo / u)]).astype(np.int64), u


def block_scores(q: np.ndarray, bounds: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """u_j of one KV group: q [G, D], bounds [nb, 2, D] integers, scale [nb]."""
    out = np.full(len(bounds), -np.inf)
    for row in tame(q):
        e = unit(np.abs(row).max())
        c = np.rint(row / e).astype(np.int64)
        whole = np.maximum(c * bounds[:, 0], c * bounds[:, 1]).sum(-1)
        out = np.maximum(out, whole * e * scale)
    return out


def select(u: np.ndarray, n: int, n_sink: int, n_recent: int, K: int) -> np.ndarray:
    """K ascending blocks of a sequence of n tokens; u covers the launch's blocks."""
    j = np.arange(len(u))
    u = np.where((j * PAGE < n_sink) | ((j + 1) * PAGE > n - n_recent), np.inf, u)
    u = np.where(j * PAGE >= n, -np.inf, u)
    return np.sort(np.argsort(-u, kind="stable")[:K])


def attention(q: np.ndarray, K: np.ndarray, V: np.ndarray):
    """q [G, D] over rows K, V [n, D]: out, lse, and per head what its error
    bound is made of: sum_j p_j |v_j| and the largest sum_d |q_d k_jd| / sqrt(D)."""
    G, D = q.shape
    if len(K) == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G)
    z = q @ K.T / math.sqrt(D)
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    s = (np.abs(q) @ np.abs(K).T).max(1) / math.sqrt(D)
    return p @ V / l, (m + np.log(l))[:, 0], p @ np.abs(V) / l, s
