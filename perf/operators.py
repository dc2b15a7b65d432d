"""What the operators of the 8-bit cache and of the block-sparse attention are measured on.

Three groups of operators next to the bf16 paged cache and its attention:

* the 8-bit paged cache: pages of 16 tokens stored as e4m3 or int8 codes with one
  scale per (page, KV head) for the keys and one for the values; the tokens of a
  page that is not full yet stay bf16 in a tail.  Stored from bf16 pages, appended
  to token by token, and loaded back into bf16 pages;
* single-token attention that reads that cache;
* single-token attention over the K pages that an integer score picks for each
  (sequence, KV head), on the bf16 cache and on the 8-bit one.

``run`` makes one pass: the plain forms below in torch, or, where ``own`` is set,
the calls a user makes of the library.
"""
import math

import torch

own = False

PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}
AMAX_FLOOR = 2.0 ** -100      # the scale of a page of zeros (or of smaller values) is this / QMAX


def _case(name, kind, B, Hq, Hkv, D, L, ragged=False, fmt="", K=0, n_sink=4, n_recent=64):
    return dict(name=name, kind=kind, B=B, Hq=Hq, Hkv=Hkv, D=D, L=L, ragged=ragged, fmt=fmt, K=K,
                n_sink=n_sink, n_recent=n_recent)


def listed():
    return [
        # a prompt's cache taken into 8 bits, one token appended (it completes the page), and restored
        _case("cache-8k-e4m3", "cache", 4, 16, 8, 128, 8208, fmt="e4m3"),
        # the same for a batch of prompts of different lengths, one of them empty
        _case("cache-32k-int8-ragged", "cache", 8, 32, 8, 128, 32767, ragged=True, fmt="int8"),
        # decoding one short conversation: a call whose time is its latency
        _case("attn8-1k-int8", "attn8", 1, 4, 2, 64, 1025, fmt="int8"),
        # an ordinary decode batch
        _case("attn8-8k-e4m3", "attn8", 4, 16, 8, 128, 8201, fmt="e4m3"),
        # a batch of ragged lengths
        _case("attn8-32k-int8-ragged", "attn8", 8, 32, 8, 128, 32769, ragged=True, fmt="int8"),
        # long contexts
        _case("attn8-128k-e4m3", "attn8", 2, 32, 8, 128, 131073, fmt="e4m3"),
        # sixteen query heads per KV head, a large batch
        _case("attn8-64k-e4m3-g16", "attn8", 16, 64, 4, 128, 65537, fmt="e4m3"),
        # block-sparse decoding over the bf16 cache: short, ordinary and ragged, long
        _case("blocks-1k", "blocks", 1, 4, 2, 64, 1025, K=13),
        _case("blocks-32k-ragged", "blocks", 8, 32, 8, 128, 32769, ragged=True, K=308, n_recent=256),
        _case("blocks-128k", "blocks", 2, 32, 8, 128, 131073, K=1229, n_recent=256),
        # block-sparse decoding over the 8-bit cache
        _case("blocks8-8k-int8", "blocks8", 4, 16, 8, 128, 8195, fmt="int8", K=103, n_recent=128),
        _case("blocks8-64k-e4m3-g16", "blocks8", 16, 64, 4, 128, 65537, fmt="e4m3", K=820, n_recent=256),
    ]


def draw(rng):
    kind = rng.choice(["cache", "attn8", "attn8", "blocks", "blocks8"])
    Hq, Hkv = rng.choice([(4, 2), (16, 8), (32, 8), (64, 4), (8, 8), (7, 1), (12, 4)])
    D = rng.choice([64, 128])
    B = int(round(2 ** rng.uniform(0, 4)))
    L = int(round(2 ** rng.uniform(0, 17)))
    room = 8 * 8 * 32768 * 128 if kind in ("cache", "blocks") else 16 * 4 * 65536 * 128
    L = max(1, min(L, room // (B * Hkv * D)))
    n_recent = rng.choice([1, 64, 128, 256])
    n_sink = rng.choice([0, 4, 17])
    nb = -(-L // PAGE)
    forced = -(-n_sink // PAGE) + -(-n_recent // PAGE) + 1
    K = min(nb, max(forced, int(nb * rng.uniform(0.02, 0.3))))
    return _case("", kind, B, Hq, Hkv, D, L, ragged=rng.random() < 0.5,
                 fmt="" if kind == "blocks" else rng.choice(["e4m3", "int8"]),
                 K=K if kind in ("blocks", "blocks8") else 0, n_sink=n_sink, n_recent=n_recent)


def _lens(c):
    """Length of every sequence: L, or (ragged) L for the first, nothing for the third and less for the others."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [0 if b == 2 else c["L"] - c["L"] * ((b * 37) % 64) // 64 for b in range(c["B"])]


# ------------------------------------------------------------------ inputs
def _keys(g, n, Hkv, D, dev):
    """Rows of N(0, 1), each times a LogNormal(0, 0.5), one in 200 of them ten times larger."""
    x = torch.randn(n, Hkv, PAGE, D, generator=g, device=dev)
    s = torch.exp(0.5 * torch.randn(n, Hkv, PAGE, 1, generator=g, device=dev))
    s = torch.where(torch.rand(n, Hkv, PAGE, 1, generator=g, device=dev) < 0.005, s * 10, s)
    return x.mul_(s).to(torch.bfloat16)


def _encode(x, fmt):
    """Codes and scales of pages x [..., 16, D] in 32 bits: scale = amax / QMAX, code = round(x * (QMAX / amax))."""
    x = x.float()
    amax = x.abs().amax(dim=(-2, -1)).clamp_min(AMAX_FLOOR)
    top = torch.full_like(amax, QMAX[fmt])
    scale, inv = amax / top, top / amax
    y = (x * inv[..., None, None]).clamp(-QMAX[fmt], QMAX[fmt])
    if fmt == "e4m3":
        return y.to(torch.float8_e4m3fn).view(torch.uint8), scale
    return torch.round(y).to(torch.int8).view(torch.uint8), scale


def _decode(codes, scale, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float() * scale[..., None, None]


def _exponent(amax):
    """The smallest e >= -126 with amax <= 127 * 2^e."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 7 + (m > 127.0 / 128.0).to(e.dtype), -126).clamp_min(-126)


def _pow2(e):
    return torch.exp2(e.double()).float()


def _bounds(k):
    """Codes of the largest and smallest value of each dimension over a page's keys (k [..., 16, D]), rounded outwards, and their scale."""
    k = k.float()
    hi, lo = k.amax(-2), k.amin(-2)
    scale = _pow2(_exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1)))
    codes = torch.stack([torch.ceil(hi / scale[..., None]), torch.floor(lo / scale[..., None])], dim=-2)
    return codes.to(torch.int8), scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, D, L = c["B"], c["Hq"], c["Hkv"], c["D"], c["L"]
    lens = _lens(c)
    max_pages = -(-L // PAGE) + 1
    n = B * max_pages + 3
    pt = torch.randperm(n, generator=g, device=dev)[:B * max_pages].to(torch.int32).view(B, max_pages).contiguous()
    k_pool = _keys(g, n, Hkv, D, dev)
    v_pool = torch.randn(n, Hkv, PAGE, D, generator=g, device=dev).to(torch.bfloat16)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    s = dict(case=c, pt=pt, lens=ln if c["ragged"] else None, ln=ln, n=n, max_pages=max_pages)
    if c["kind"] == "cache":
        s["before"] = (ln - 1).clamp_min(0)
        s.update(k_pool=k_pool, v_pool=v_pool, k_back=torch.zeros_like(k_pool), v_back=torch.zeros_like(v_pool))
        s["k_new"] = _keys(g, B, Hkv, D, dev)[:, :, 0].contiguous()
        s["v_new"] = torch.randn(B, Hkv, D, generator=g, device=dev).to(torch.bfloat16)
    else:
        # a query is the sum of three unit keys of its sequence, eight times, and noise
        pos = (torch.rand(B, Hq, 3, generator=g, device=dev) * ln.clamp_min(1)[:, None, None]).long()
        head = (torch.arange(Hq, device=dev) // (Hq // Hkv))[None, :, None].expand(B, Hq, 3)
        rows = k_pool[pt.long()[torch.arange(B, device=dev)[:, None, None], pos // PAGE], head, pos % PAGE].float()
        rows = rows / rows.norm(dim=-1, keepdim=True).clamp_min(1e-30)
        s["q"] = (8 * rows.sum(2) + 0.3 * torch.randn(B, Hq, D, generator=g, device=dev)).to(torch.bfloat16)
        s["out"] = torch.empty(B, Hq, D, device=dev)
        s["lse"] = torch.empty(B, Hq, device=dev)
        if c["kind"] in ("blocks", "blocks8"):
            s["bounds"], s["bscale"] = _bounds(k_pool)
            s["sel"] = torch.empty(B, Hkv, c["K"], dtype=torch.int32, device=dev)
        if c["kind"] == "blocks":
            s.update(k_pool=k_pool, v_pool=v_pool)
        else:
            last = pt.long().gather(1, (ln.long() // PAGE)[:, None])[:, 0]
            s["k_tail"], s["v_tail"] = k_pool[last].contiguous(), v_pool[last].contiguous()
            s["k_codes"], s["k_scale"] = _encode(k_pool, c["fmt"])
            s["v_codes"], s["v_scale"] = _encode(v_pool, c["fmt"])
    if own:
        s["plan"] = _plan(s)
    return s


# ------------------------------------------------------------------ plain forms
def _rows(pool, pt):
    """[B, Hkv, pages * 16, D] of pages [n, Hkv, 16, D]."""
    x = pool[pt]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, x.shape[4])


def _attend(q, k, v, ok):
    """softmax(q k / sqrt(D)) v over the positions where ok; nothing to attend to: 0 and -inf."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    z = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), k.transpose(-1, -2)) / math.sqrt(D)
    z = torch.where(ok[:, :, None, :], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(m), 0.0, m))
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, torch.where(ok[..., None], v, 0.0))
    lse = torch.log(l) + torch.where(torch.isinf(m), 0.0, m)
    return torch.where(l > 0, o / l, 0.0).view(B, Hq, D), lse.view(B, Hq)


def _plain_cache(s):
    c = s["case"]
    P = -(-c["L"] // PAGE)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    pt, ln = s["pt"][:, :P].long(), s["ln"].long()
    pos = torch.arange(P * PAGE, device=pt.device).view(1, P, PAGE)
    at = (pos == (ln - 1)[:, None, None])[:, :, None, :, None]           # where the appended token lies
    full = (torch.arange(P, device=pt.device)[None, :] + 1) * PAGE <= ln[:, None]
    there = (pos < ln[:, None, None])[:, :, None, :, None]
    back, scales = [], []
    # keys and values alike
    for pool, new in ((s["k_pool"], s["k_new"]), (s["v_pool"], s["v_new"])):
        x = torch.where(at, new.view(B, 1, Hkv, 1, D), pool[pt])         # [B, P, Hkv, 16, D]
        codes, scale = _encode(x, c["fmt"])
        y = torch.where(full[:, :, None, None, None], _decode(codes, scale, c["fmt"]).to(torch.bfloat16), x)
        out = torch.zeros_like(pool)
        out[pt] = torch.where(there, y, torch.zeros_like(y))
        back.append(out)
        kept = torch.zeros(s["n"], Hkv, device=pt.device)
        kept[pt] = torch.where(full[:, :, None], scale, torch.zeros_like(scale))
        scales.append(kept)
        if pool is s["k_pool"]:
            codes, bs = _bounds(x)
            bound = torch.zeros(s["n"], Hkv, 2, D, device=pt.device)
            bound[pt] = torch.where(full[:, :, None, None, None], codes.float() * bs[..., None, None], 0.0)
    return back + scales + [bound]


def _plain_select(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    nb = -(-c["L"] // PAGE)
    pt, ln = s["pt"][:, :nb].long(), s["ln"].long()[:, None, None]
    q = s["q"].float()
    qs = _pow2(_exponent(q.abs().amax(-1)))
    qc = torch.round(q / qs[..., None]).view(B, Hkv, Hq // Hkv, D)
    b = s["bounds"][pt].permute(0, 2, 3, 4, 1).float()                   # [B, Hkv, 2, D, nb]
    whole = torch.matmul(qc.clamp_min(0), b[:, :, 0]) + torch.matmul(qc.clamp_max(0), b[:, :, 1])
    u = whole * qs.view(B, Hkv, -1, 1) * s["bscale"][pt].permute(0, 2, 1)[:, :, None]
    big = torch.finfo(torch.float32).max
    u = u.amax(2).clamp(-big, big)
    j = torch.arange(nb, device=pt.device)[None, None]
    always = (j * PAGE < c["n_sink"]) | ((j + 1) * PAGE > ln - c["n_recent"])
    u = torch.where(j * PAGE >= ln, -math.inf, torch.where(always, math.inf, u))
    top = torch.sort(u, dim=-1, descending=True, stable=True).indices[..., :c["K"]]
    return torch.sort(top, dim=-1).values.to(torch.int32)


def _chosen(s, pool, scale, tail, sel):
    """The rows [B, Hkv, K * 16, D] of the chosen pages, in 32 bits."""
    c = s["case"]
    page = s["pt"].long().gather(1, sel.long().view(c["B"], -1)).view(sel.shape)
    head = torch.arange(c["Hkv"], device=sel.device)[None, :, None]
    x = pool[page, head]
    if scale is not None:
        x = _decode(x, scale[page, head], c["fmt"])
        partly = sel == (s["ln"] // PAGE)[:, None, None]
        x = torch.where(partly[..., None, None], tail[:, :, None].float(), x)
    return x.float().view(c["B"], c["Hkv"], -1, c["D"])


def _plain(s):
    c = s["case"]
    if c["kind"] == "cache":
        return _plain_cache(s)
    ln = s["ln"][:, None, None]
    if c["kind"] == "attn8":
        P = -(-c["L"] // PAGE)
        pt = s["pt"][:, :P].long()
        pos = torch.arange(P * PAGE, device=pt.device)[None, None]
        cut = pos // PAGE == ln // PAGE                                  # the page that is not full: the tail's rows
        slot = pos.view(-1) % PAGE
        k = torch.where(cut[..., None], s["k_tail"][:, :, slot].float(), _rows(_decode(s["k_codes"], s["k_scale"], c["fmt"]), pt))
        v = torch.where(cut[..., None], s["v_tail"][:, :, slot].float(), _rows(_decode(s["v_codes"], s["v_scale"], c["fmt"]), pt))
        return list(_attend(s["q"], k, v, (pos < ln).expand(-1, c["Hkv"], -1)))
    sel = _plain_select(s)
    if c["kind"] == "blocks":
        k, v = _chosen(s, s["k_pool"], None, None, sel), _chosen(s, s["v_pool"], None, None, sel)
    else:
        k = _chosen(s, s["k_codes"], s["k_scale"], s["k_tail"], sel)
        v = _chosen(s, s["v_codes"], s["v_scale"], s["v_tail"], sel)
    pos = (sel[..., None] * PAGE + torch.arange(PAGE, device=sel.device)).view(c["B"], c["Hkv"], -1)
    return [sel] + list(_attend(s["q"], k, v, pos < ln))


# ------------------------------------------------------------------ the library's calls
def _plan(s):
    from slow_sparse_kv_sfi_b200 import sfi as S
    c, dev = s["case"], "cuda"
    n, Hkv, D = s["n"], c["Hkv"], c["D"]
    p = dict(S=S, shape=S.make_shape(c["B"], c["Hq"], Hkv, D, s["max_pages"], n))
    p["ws"] = torch.zeros(S.sfi_block_workspace_size(p["shape"]), dtype=torch.uint8, device=dev)
    fmt = {"e4m3": S.FMT_E4M3, "int8": S.FMT_INT8}.get(c["fmt"])
    if c["kind"] == "cache":
        z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
        s["k_codes"], s["v_codes"] = z(n, Hkv, PAGE, D, dtype=torch.uint8), z(n, Hkv, PAGE, D, dtype=torch.uint8)
        s["k_scale"], s["v_scale"] = z(n, Hkv), z(n, Hkv)
        s["k_tail"], s["v_tail"] = z(c["B"], Hkv, PAGE, D, dtype=torch.bfloat16), z(c["B"], Hkv, PAGE, D, dtype=torch.bfloat16)
        s["bounds"], s["bscale"] = z(n, Hkv, 2, D, dtype=torch.int8), z(n, Hkv)
        p["back"] = S.make_kv(s["k_back"], s["v_back"], s["pt"])
    if "k_pool" in s:
        p["kv"] = S.make_kv(s["k_pool"], s["v_pool"], s["pt"])
    if "k_codes" in s:
        p["qkv"] = S.make_quant_kv(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"], s["pt"], fmt)
    if "bounds" in s:
        p["index"] = S.make_block_index(s["bounds"], s["bscale"], s["pt"])
    return p


def _own(s):
    c, p = s["case"], s["plan"]
    S, shape, L, lens = p["S"], p["shape"], c["L"], s["lens"]
    if c["kind"] == "cache":
        S.sfi_quant_store(shape, p["kv"], p["qkv"], 0, L - 1, lens=s["before"] if c["ragged"] else None, index=p["index"])
        S.sfi_quant_append(shape, p["qkv"], L, s["k_new"], s["v_new"], lens=lens, index=p["index"])
        S.sfi_quant_load(shape, p["qkv"], p["back"], 0, L, lens=lens)
        return [s["k_back"], s["v_back"], s["k_scale"], s["v_scale"], torch.mul(s["bounds"], s["bscale"][..., None, None])]
    if c["kind"] == "attn8":
        S.sfi_quant_attn(shape, p["qkv"], L, s["q"], s["out"], p["ws"], lens=lens, lse=s["lse"])
        return [s["out"], s["lse"]]
    S.sfi_block_select(shape, p["index"], L, s["q"], c["n_sink"], c["n_recent"], c["K"], s["sel"], p["ws"], lens=lens)
    if c["kind"] == "blocks":
        S.sfi_block_attn(shape, p["kv"], L, s["q"], s["sel"], c["K"], s["out"], p["ws"], lens=lens, lse=s["lse"])
    else:
        S.sfi_quant_block_attn(shape, p["qkv"], L, s["q"], s["sel"], c["K"], s["out"], p["ws"], lens=lens, lse=s["lse"])
    return [s["sel"], s["out"], s["lse"]]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c = case
    lens = _lens(c)
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    el = 1 if c["fmt"] else 2
    if c["kind"] == "cache":
        # bf16 rows in, codes out, codes in, bf16 rows out; scales and bounds of the full pages
        full = sum(n // PAGE for n in lens)
        by = sum(lens) * Hkv * D * 2 * (2 + 1 + 1 + 2) + full * Hkv * (2 * D + 12)
        return {"bytes": by, "flops": sum(lens) * Hkv * D * 2 * 4}
    by = B * Hq * D * (2 + 4) + B * Hq * 4
    if c["kind"] == "attn8":
        rows = sum(lens)
        by += rows * Hkv * D * 2 + sum(-(-n // PAGE) for n in lens) * (Hkv * 8 + 4)
        return {"bytes": by, "flops": 4 * rows * Hq * D}
    # the bounds of every page, then the chosen pages
    nb = [-(-n // PAGE) for n in lens]
    rows = sum(min(n, c["K"] * PAGE) for n in lens)
    by += sum(nb) * (Hkv * (2 * D + 4) + 4) + rows * Hkv * D * 2 * el + B * Hkv * c["K"] * 8
    return {"bytes": by, "flops": 4 * rows * Hq * D + 4 * sum(nb) * Hq * D}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _e4m3_nearest(y):
    """Nearest value of 4 significant bits (ties to even), spacing 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _page_values(x, fmt):
    """What pages x [..., 16, D] in float64 stand for after storing, and their scales."""
    amax = x.abs().amax((-2, -1), keepdim=True).clamp_min(AMAX_FLOOR)
    y = x * (QMAX[fmt] / amax)
    y = _e4m3_nearest(y) if fmt == "e4m3" else torch.round(y)
    return y * (amax / QMAX[fmt]), (amax / QMAX[fmt])[..., 0, 0]


def _unit(amax):
    """Smallest power of two u >= 2^-126 with amax <= 127 u."""
    u = torch.exp2(torch.ceil(torch.log2((amax / 127).clamp_min(2.0 ** -126))))
    u = torch.where(amax <= 127 * u / 2, u / 2, u)
    return torch.where(amax > 127 * u, 2 * u, u).clamp_min(2.0 ** -126)


def _exact_cache(s):
    c, d = s["case"], torch.float64
    shape = s["k_pool"].shape
    n, Hkv, _, D = shape
    out = [torch.zeros(shape, dtype=d, device="cuda") for _ in range(2)]
    scl = [torch.zeros(n, Hkv, dtype=d, device="cuda") for _ in range(2)]
    bound = torch.zeros(n, Hkv, 2, D, dtype=d, device="cuda")
    for b, ln in enumerate(_lens(c)):
        if ln == 0:
            continue
        P = -(-ln // PAGE)
        pages = s["pt"][b, :P].long()
        for i, (pool, new) in enumerate(((s["k_pool"], s["k_new"]), (s["v_pool"], s["v_new"]))):
            x = pool[pages].to(d)
            x[(ln - 1) // PAGE, :, (ln - 1) % PAGE] = new[b].to(d)
            whole = ln // PAGE
            if ln % PAGE:
                out[i][pages[-1], :, :ln % PAGE] = x[-1, :, :ln % PAGE]
            y, sc = _page_values(x[:whole], c["fmt"])
            out[i][pages[:whole]] = y
            scl[i][pages[:whole]] = sc
            if i == 0 and whole:
                hi, lo = x[:whole].amax(2), x[:whole].amin(2)
                u = _unit(torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True))
                bound[pages[:whole], :, 0] = torch.ceil(hi / u) * u
                bound[pages[:whole], :, 1] = torch.floor(lo / u) * u
    return out + scl + [bound]


def _exact_select(s, b, g, ln):
    """Block numbers of KV head g of sequence b, ascending."""
    c = s["case"]
    nb, G = -(-c["L"] // PAGE), c["Hq"] // c["Hkv"]
    pages = s["pt"][b, :nb].long()
    bound = s["bounds"][pages, g].double() * s["bscale"][pages, g].double()[:, None, None]
    q = s["q"][b, g * G:(g + 1) * G].double()
    u = _unit(q.abs().amax(-1, keepdim=True))
    q = torch.round(q / u) * u
    score = torch.maximum(q[:, None] * bound[None, :, 0], q[:, None] * bound[None, :, 1]).sum(-1).amax(0)
    j = torch.arange(nb, device="cuda")
    score[j * PAGE < c["n_sink"]] = math.inf
    score[(j + 1) * PAGE > ln - c["n_recent"]] = math.inf
    score[j * PAGE >= ln] = -math.inf
    order = torch.argsort(score, descending=True, stable=True)[:c["K"]]
    return torch.sort(order).values


def exact(case, seed):
    s = prepare(case, seed)
    c, d = case, torch.float64
    if c["kind"] == "cache":
        return _exact_cache(s)
    B, Hq, Hkv, D, fmt = c["B"], c["Hq"], c["Hkv"], c["D"], c["fmt"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=d, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=d, device="cuda")
    sel = torch.zeros(B, Hkv, c["K"], dtype=torch.int32, device="cuda") if c["K"] else None
    kind = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}.get(fmt)
    for b, ln in enumerate(_lens(c)):
        for g in range(Hkv):
            if sel is not None:
                chosen = _exact_select(s, b, g, ln)
                sel[b, g] = chosen.to(torch.int32)
                chosen = chosen[chosen * PAGE < ln]
            else:
                chosen = torch.arange(-(-ln // PAGE), device="cuda")
            if ln == 0:
                continue
            pages = s["pt"][b].long()[chosen]
            kv = []
            for x in "kv":
                if fmt:
                    r = s[x + "_codes"].view(kind)[pages, g].to(d) * s[x + "_scale"][pages, g].to(d)[:, None, None]
                    r[chosen == ln // PAGE] = s[x + "_tail"][b, g].to(d)
                else:
                    r = s[x + "_pool"][pages, g].to(d)
                kv.append(r.reshape(-1, D))
            pos = (chosen[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)
            k, v = (r[pos < ln] for r in kv)
            z = s["q"][b, g * G:(g + 1) * G].to(d) @ k.T / math.sqrt(D)
            out[b, g * G:(g + 1) * G] = torch.softmax(z, -1) @ v
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(z, -1)
    return ([sel] if sel is not None else []) + [out, lse]
