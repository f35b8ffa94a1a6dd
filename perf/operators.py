"""What the paged-cache operators are measured on: the cases, their inputs, the operators in plain torch form and
in 64 bits, and the calls of the framework (where ``own`` is true).

Three operators:
  * "attn":  attention of one new token per sequence over a paged key-value cache;
  * "qk":    norm of query and key heads, position rotation, and the append of keys and values to the cache;
  * "pages": freeing, forking, copying and compacting the cache's pages.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short sequence: a prompt's first decode steps, where a call's latency is all there is
        _attn("attn one short", "bf16", 1, 8, 2, 64, 16, 37, 0, 1),
        # a serving batch of ragged grouped-query sequences, bf16 pages
        _attn("attn ragged batch", "bf16", 64, 32, 8, 128, 16, 16384, 0, 2),
        # few long contexts over an e4m3 cache
        _attn("attn long e4m3", "e4m3", 4, 64, 8, 128, 64, 131072, 0, 3),
        # the 500K-token context of the decode workload: 4 x 131072 compressed entries, one latent head of 512
        # that serves as key and value, 128 query heads
        _attn("attn latent 500K", "bf16", 4, 128, 1, 512, 64, 131072, 0, 0, latent=True),
        # 32-bit cache, odd head dim and page size, a recent window only
        _attn("attn f32 window", "f32", 7, 12, 4, 96, 48, 9001, 4097, 4),
        # one token's heads: normalised, rotated and appended to bf16 pages
        _qk("qk one token", "bf16", 1, 32, 8, 128, 128, False, True, "bf16", 16, 5),
        # a decode batch into an e4m3 cache
        _qk("qk batch e4m3", "bf16", 203, 64, 8, 128, 128, False, True, "e4m3", 64, 6),
        # a prompt's chunk into bf16 pages
        _qk("qk prompt", "bf16", 16384, 32, 8, 128, 128, False, True, "bf16", 64, 7),
        # the indexer's query heads: interleaved rotation of the head's first half, no norm, no cache
        _qk("rotate indexer heads", "f32", 4099, 64, 1, 128, 64, True, False, "", 0, 8),
        # a beam step of a small model: prune the children, fork their parents again, copy the last pages
        _pages("pages fork beams", "fork", "bf16", 4, 32, 2, 64, 16, 5, 40, 700),
        # parallel samples of many long prompts, 64-token pages of 8 heads
        _pages("pages fork samples", "fork", "bf16", 64, 600, 8, 128, 64, 8, 32, 8000),
        # packing a fragmented latent cache of 1 GB to its front
        _pages("pages compact", "compact", "bf16", 64, 512, 1, 512, 64, 0, 128, 16384),
    ]


def _attn(name, dtype, B, Hq, Hkv, D, page, most, window, ragged, latent=False):
    return {"name": name, "op": "attn", "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "most": most, "window": window, "ragged": ragged, "latent": latent}


def _qk(name, dtype, T, Hq, Hkv, D, rot, interleaved, norm, cache, page, fill):
    return {"name": name, "op": "qk", "dtype": dtype, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "interleaved": interleaved, "norm": norm, "cache": cache, "page": page, "fill": fill}


def _pages(name, do, dtype, parents, rows, Hkv, D, page, children, max_pages, n_pages):
    """parents own pages; with "fork" each has `children` forks among the other rows."""
    return {"name": name, "op": "pages", "do": do, "dtype": dtype, "parents": parents, "rows": rows, "Hkv": Hkv,
            "D": D, "page": page, "children": children, "max_pages": max_pages, "n_pages": n_pages}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    fill = rng.randrange(1, 1 << 30)
    kind = rng.choice(["attn", "attn", "attn", "qk", "qk", "pages"])
    if kind == "attn":
        dtype = rng.choice(["bf16", "bf16", "e4m3", "f32"])
        page = rng.choice([1, 8, 16, 17, 32, 48, 64, 100, 128, 256])
        latent = rng.random() < 0.25
        if latent:
            Hkv, D, Hq = 1, 512, rng.choice([8, 16, 32, 64, 128, 128, 128])
        else:
            Hkv, D = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
            Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16])
        B, most = _log(rng, 1, 256), _log(rng, 1, 131072)
        # no more than the largest listed case: 268 MB of rows, or that case's products in 32 bits
        while B > 1 and B * most * Hkv * D * SIZE[dtype] > 1 << 28:
            B //= 2
        while most * Hkv * D * SIZE[dtype] > 1 << 28 or B * Hq * most * D > 1 << 34:
            most = most * 2 // 3
        window = _log(rng, 1, most) if rng.random() < 0.3 else 0
        c = _attn("", dtype, B, Hq, Hkv, D, page, most, window, fill if rng.random() < 0.8 else 0, latent)
    elif kind == "qk":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = rng.choice([32, 64, 80, 96, 128, 128, 192, 256, 512])
        rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randrange(0, D // 2)])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        cache = rng.choice(["", dtype, "e4m3" if dtype == "bf16" else dtype])
        T = _log(rng, 1, 16384)
        while T * (Hq + 2 * Hkv) * D * SIZE[dtype] > 1 << 27:
            T //= 2
        c = _qk("", dtype, T, Hq, Hkv, D, rot, rng.random() < 0.4, rng.random() < 0.7, cache,
                rng.choice([1, 8, 16, 17, 48, 64, 128]) if cache else 0, fill)
    else:
        do = rng.choice(["fork", "compact"])
        dtype, page = rng.choice(["bf16", "e4m3", "f32"]), rng.choice([1, 8, 16, 17, 48, 64, 128])
        Hkv, D = rng.choice([(1, 512), (1, 128), (2, 64), (4, 96), (8, 128), (3, 80)])
        parents = _log(rng, 1, 64)
        children = rng.choice([1, 2, 3, 4, 8]) if do == "fork" else 0
        max_pages = _log(rng, 1, 256)
        n_pages = parents * (max_pages + children) + _log(rng, 2, 1000)
        while n_pages * page * Hkv * D * SIZE[dtype] > 1 << 27:
            page, max_pages = max(1, page // 2), max(1, max_pages // 2)
            n_pages = parents * (max_pages + children) + 2 + n_pages // 8
        c = _pages("", do, dtype, parents, parents * (1 + children) + rng.randrange(0, 9), Hkv, D, page, children,
                   max_pages, n_pages)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs

def _lengths(c):
    """Sequence lengths of an attention case: all `most`, or spread over [0, most] (over their logarithm) with one
    of `most` among them."""
    if not c["ragged"]:
        return [c["most"]] * c["B"]
    r = random.Random(c["ragged"])
    n = [_log(r, 1, c["most"]) if r.random() < 0.95 else 0 for _ in range(c["B"])]
    n[r.randrange(c["B"])] = c["most"]
    return n


def _rows(gen, dtype, shape):
    """Cache rows and, for e4m3, their scales (one of each row, its largest magnitude / 448)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16 if dtype != "f32" else torch.float32)
    if dtype != "e4m3":
        return x, None
    scale = x.abs().amax(-1).float().clamp(min=1e-6) / E4M3_MAX
    return (x.float() / scale[..., None]).to(torch.float8_e4m3fn), scale


def _table(gen, counts, max_pages, n_pages):
    """A page table whose rows hold `counts` pages each, scattered over the pool."""
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    cnt = torch.tensor(counts, device="cuda")
    first = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(max_pages, device="cuda")
    held = col[None, :] < cnt[:, None]
    return torch.where(held, order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).int().contiguous()


def _freq(c):
    """Radians per position of each rotated pair (base 10000), in 64 bits."""
    half = c["rot"] // 2
    return torch.tensor([10000.0 ** (-2.0 * i / c["rot"]) for i in range(half)], dtype=torch.float64, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"c": c}
    if c["op"] == "attn":
        _prepare_attn(c, gen, s)
    elif c["op"] == "qk":
        _prepare_qk(c, gen, s)
    else:
        _prepare_pages(c, gen, s, seed)
    if own:
        _handles(c, s)
    return s


def _prepare_attn(c, gen, s):
    lens, page = _lengths(c), c["page"]
    counts = [-(-n // page) for n in lens]
    max_pages = max(1, max(counts))
    n_pages = sum(counts) + 3
    s["max_len"] = max(lens)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"] = _table(gen, counts, max_pages, n_pages)
    shape = (n_pages, page, c["Hkv"], c["D"])
    s["k"], s["k_scale"] = _rows(gen, c["dtype"], shape)
    s["v"], s["v_scale"] = (s["k"], s["k_scale"]) if c["latent"] else _rows(gen, c["dtype"], shape)
    qt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    # scores of a spread of 2: a few entries carry much of the weight, as in a trained model
    s["q"] = (2 * torch.randn((c["B"], c["Hq"], c["D"]), generator=gen, device="cuda")).to(qt)
    s["scale"] = c["D"] ** -0.5
    s["out"] = torch.zeros((c["B"], c["Hq"], c["D"]), dtype=qt, device="cuda")
    s["lse"] = torch.zeros((c["B"], c["Hq"]), dtype=torch.float32, device="cuda")


def _prepare_qk(c, gen, s):
    T, Hq, Hkv, D, dt = c["T"], c["Hq"], c["Hkv"], c["D"], DT[c["dtype"]]
    # one projection's output holds a token's query, key and value heads side by side
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, device="cuda").to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["wq"], s["wk"] = [(1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt) if c["norm"] else None
                        for _ in range(2)]
    s["eps"] = 1e-6
    s["freq"] = _freq(c)
    s["q_out"] = torch.zeros((T, Hq, D), dtype=dt, device="cuda")
    s["k_out"] = None if c["cache"] else torch.zeros((T, Hkv, D), dtype=dt, device="cuda")
    if not c["cache"]:
        # positions of packed sequences, up to a million
        s["pos"] = torch.randint(0, 1 << 20, (T,), generator=gen, device="cuda").int()
        return
    page = c["page"]
    if T <= 256:      # a decode step: token t is the newest of sequence t
        r = random.Random(c["fill"])
        before = [r.randrange(0, 8 * page) for _ in range(T)]
        s["pos"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["seq"] = torch.arange(T, dtype=torch.int32, device="cuda")
        counts = [n // page + 1 for n in before]
    else:             # a chunk of one prompt, from a position of its own on
        first = c["fill"] % 1000
        s["pos"] = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
        s["seq"] = torch.zeros(T, dtype=torch.int32, device="cuda")
        counts = [-(-(first + T) // page)]
    n_pages = sum(counts) + 2
    s["table"] = _table(gen, counts, max(counts), n_pages)
    shape = (n_pages, page, Hkv, D)
    for x in ("k", "v"):
        s[x + "_cache"] = torch.zeros(shape, device="cuda").to(DT[c["cache"]])
        s[x + "_scale"] = torch.ones(shape[:-1], device="cuda") if c["cache"] == "e4m3" else None


def _prepare_pages(c, gen, s, seed):
    r = random.Random(seed)
    page, P, W, N = c["page"], c["parents"], c["max_pages"], c["n_pages"]
    lens = [r.randrange(1, W * page + 1) for _ in range(P)]
    lens[0] = W * page if c["do"] == "compact" else max(1, W * page - 1)
    counts = [-(-n // page) for n in lens]
    table = torch.full((c["rows"], W), -1, dtype=torch.int32, device="cuda")
    table[:P] = _table(gen, counts, W, N)
    s["k"], s["k_scale"] = _rows(gen, c["dtype"], (N, page, c["Hkv"], c["D"]))
    s["v"], s["v_scale"] = _rows(gen, c["dtype"], (N, page, c["Hkv"], c["D"])) if c["Hkv"] > 1 else (s["k"], s["k_scale"])
    s["table"] = table
    s["len"] = torch.zeros(c["rows"], dtype=torch.int32, device="cuda")
    s["len"][:P] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["refs"] = torch.zeros(N, dtype=torch.int32, device="cuda")
    s["refs"][table[table >= 0].long()] = 1
    if c["do"] == "fork":
        n = P * c["children"]
        s["src"] = torch.arange(P, dtype=torch.int32, device="cuda").repeat_interleave(c["children"])
        s["dst"] = torch.arange(P, P + n, dtype=torch.int32, device="cuda")
        s["copy_src"], s["copy_dst"] = (torch.full((n,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        _fork(c, s)      # the children of the step before
    else:
        s["table_out"], s["refs_out"] = torch.zeros_like(table), torch.zeros_like(s["refs"])
        s["move_src"], s["move_dst"] = (torch.full((N,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        s["moves"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        live = s["refs"] > 0
        s["n_moves"] = int(live[int(live.sum()):].sum())   # a program knows its pool's fill


def _handles(c, s):
    """What a user's program keeps beside its tensors."""
    from lookahead_sparse_kv_index_b200 import lsa

    if c["op"] == "attn":
        s["cache"] = lsa.PageCache(s["k"], None if c["latent"] else s["v"], s["k_scale"],
                                   None if c["latent"] else s["v_scale"])
        size = lsa.paged_attn_workspace_size(s["cache"], c["B"], c["Hq"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    elif c["op"] == "qk":
        s["rope"] = lsa.Rope(s["freq"], interleaved=c["interleaved"])
        s["cache"] = lsa.PageCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]) if c["cache"] else None
    else:
        s["cache"] = lsa.PageCache(s["k"], None if s["v"] is s["k"] else s["v"], s["k_scale"],
                                   None if s["v"] is s["k"] else s["v_scale"])
        s["pages"] = lsa.PageTable(s["table"], s["len"], s["refs"], c["page"])
        if c["do"] == "compact":
            s["ws"] = torch.empty(lsa.page_compact_workspace_size(c["n_pages"]), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------- runs

def run(state):
    s, c = state, state["c"]
    if own:
        return _own(c, s)
    if c["op"] == "attn":
        return _attention(c, s)
    if c["op"] == "qk":
        return _norm_rotate(c, s)
    if c["do"] == "fork":
        _free(s)
        _fork(c, s)
        own_page = s["table"][s["src"].long(), 0]      # held by the parent: copied onto itself where nothing is
        _copy(s, torch.where(s["copy_src"] < 0, own_page, s["copy_src"]).long(),
              torch.where(s["copy_dst"] < 0, own_page, s["copy_dst"]).long())
        return _page_outputs(c, s)
    return _compact(c, s)


def _own(c, s):
    from lookahead_sparse_kv_index_b200 import lsa

    if c["op"] == "attn":
        lsa.paged_attn(s["q"], s["cache"], s["table"], s["len"], s["out"], s["ws"], lse=s["lse"],
                       window=c["window"], scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "qk":
        if c["cache"]:
            lsa.qk_norm_rope(s["q"], s["k"], s["v"], q_out=s["q_out"], q_weight=s["wq"], k_weight=s["wk"],
                             eps=s["eps"], pos=s["pos"], rope=s["rope"], cache=s["cache"], table=s["table"],
                             seq=s["seq"], at=s["pos"])
        else:
            lsa.qk_norm_rope(s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"], q_weight=s["wq"],
                             k_weight=s["wk"], eps=s["eps"], pos=s["pos"], rope=s["rope"])
        return _qk_outputs(c, s)
    if c["do"] == "fork":
        lsa.page_free(s["pages"], s["dst"])
        lsa.page_fork(s["pages"], s["src"], s["dst"], s["copy_src"], s["copy_dst"])
        lsa.page_copy(s["cache"], s["copy_src"], s["copy_dst"])
    else:
        lsa.page_compact(s["pages"], s["table_out"], s["refs_out"], s["move_src"], s["move_dst"], s["moves"], s["ws"])
        lsa.page_copy(s["cache"], s["move_src"], s["move_dst"], count=s["moves"])
    return _page_outputs(c, s)


def _gather(x, scale, slot):
    """Cache rows in 32 bits at flat (page, slot) indices [B, n] -> [B, n, Hkv, D]."""
    flat = x.reshape(-1, *x.shape[2:])
    if x.dtype == torch.float8_e4m3fn:
        return flat.view(torch.uint8)[slot].view(x.dtype).float() * scale.reshape(-1, x.shape[2])[slot][..., None]
    return flat[slot].float()


def _attention(c, s):
    B, Hkv, D, page, n = c["B"], c["Hkv"], c["D"], c["page"], max(1, s["max_len"])
    pos = torch.arange(n, device="cuda")
    slot = s["table"].clamp(min=0).long()[:, pos // page] * page + pos % page
    length = s["len"].long()[:, None]
    seen = pos < length
    if c["window"]:
        seen &= pos >= length - c["window"]
    k = _gather(s["k"], s["k_scale"], slot)
    v = k if c["latent"] else _gather(s["v"], s["v_scale"], slot)
    q = s["q"].float().reshape(B, Hkv, -1, D)
    a = torch.einsum("bhgd,bnhd->bhgn", q, k) * s["scale"]
    a.masked_fill_(~seen[:, None, None, :], -math.inf)
    m = a.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(a - m)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgn,bnhd->bhgd", p, v) / total.clamp(min=torch.finfo(torch.float32).tiny)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return {"out": o.reshape(B, -1, D).to(s["q"].dtype), "lse": lse.reshape(B, -1)}


def _rotate(x, cos, sin, interleaved):
    """x [T, H, rot] with cos, sin [T, 1, rot / 2]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _norm_rotate(c, s):
    # far positions lose their angle in 32 bits: the angle is taken in 64
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    rot = c["rot"]

    def heads(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        if rot:
            x = torch.cat((_rotate(x[..., :rot], cos, sin, c["interleaved"]), x[..., rot:]), -1)
        return x

    s["q_out"].copy_(heads(s["q"], s["wq"]))
    k = heads(s["k"], s["wk"])
    if not c["cache"]:
        s["k_out"].copy_(k)
        return _qk_outputs(c, s)
    at = s["pos"].long()
    page = s["table"][s["seq"].long(), at // c["page"]].long()
    _append(c, s, "k", k, page, at % c["page"])
    _append(c, s, "v", s["v"].float(), page, at % c["page"])
    return _qk_outputs(c, s)


def _append(c, s, name, x, page, slot):
    cache, scales = s[name + "_cache"], s[name + "_scale"]
    if c["cache"] == "e4m3":
        amax = x.abs().amax(-1)
        scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
        scales[page, slot] = scale
        cache.view(torch.uint8)[page, slot] = (x / scale[..., None]).to(cache.dtype).view(torch.uint8)
    else:
        cache[page, slot] = x.to(cache.dtype)


def _qk_outputs(c, s):
    out = {"q": s["q_out"]}
    if c["cache"]:
        out |= {"k": s["k_cache"], "v": s["v_cache"]}
        if c["cache"] == "e4m3":
            out |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    else:
        out["k"] = s["k_out"]
    return out


def _free(s):
    """The rows dst give their pages back."""
    rows = s["dst"].long()
    held = s["table"][rows]
    s["refs"].scatter_add_(0, held.clamp(min=0).long().flatten(), -(held >= 0).int().flatten())
    s["table"][rows] = -1
    s["len"][rows] = 0


def _fork(c, s):
    """Each dst row shares the full pages of its src row and gets a page of its own for a last page in part filled:
    the lowest free pages, in the order of dst."""
    src, dst, page, N = s["src"].long(), s["dst"].long(), c["page"], c["n_pages"]
    length = s["len"][src]
    full, part = length // page, length % page > 0
    col = torch.arange(c["max_pages"], device="cuda")
    shared = col[None, :] < full[:, None]
    held = s["table"][src]
    s["refs"].scatter_add_(0, torch.where(shared, held, 0).long().flatten(), shared.int().flatten())
    free = s["refs"] == 0
    rank = torch.cumsum(free, 0) - 1
    order = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    order.scatter_(0, torch.where(free, rank, N), torch.arange(N, dtype=torch.int32, device="cuda"))
    new = order[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    last = held.gather(1, full.clamp(max=c["max_pages"] - 1).long()[:, None])[:, 0]
    child = torch.where(shared, held, -1)
    child = torch.where(part[:, None] & (col[None, :] == full[:, None]), new[:, None], child)
    s["table"][dst] = child
    s["len"][dst] = length
    s["refs"].scatter_add_(0, torch.where(part, new, 0).long(), part.int())
    s["copy_src"].copy_(torch.where(part, last, -1))
    s["copy_dst"].copy_(torch.where(part, new, -1))


def _copy(s, src, dst):
    """Pages src onto pages dst (a pair of the same page changes nothing)."""
    s["k"].view(torch.uint8)[dst] = s["k"].view(torch.uint8)[src]
    if s["k_scale"] is not None:
        s["k_scale"][dst] = s["k_scale"][src]
    if s["v"] is s["k"]:
        return
    s["v"].view(torch.uint8)[dst] = s["v"].view(torch.uint8)[src]
    if s["v_scale"] is not None:
        s["v_scale"][dst] = s["v_scale"][src]


def _compact(c, s):
    """Held pages behind the first n_held move, in order, into the free ones among them, in order."""
    refs, N = s["refs"], c["n_pages"]
    page = torch.arange(N, dtype=torch.int32, device="cuda")
    live = refs > 0
    front = page < live.sum()
    leave, enter = live & ~front, ~live & front
    for_list = torch.full((2, N + 1), -1, dtype=torch.int32, device="cuda")
    for_list[0].scatter_(0, torch.where(leave, torch.cumsum(leave, 0) - 1, N), torch.where(leave, page, -1))
    for_list[1].scatter_(0, torch.where(enter, torch.cumsum(enter, 0) - 1, N), torch.where(enter, page, -1))
    s["move_src"].copy_(for_list[0, :N])
    s["move_dst"].copy_(for_list[1, :N])
    s["moves"].copy_(leave.sum())
    src, dst = for_list[0, : s["n_moves"]].long(), for_list[1, : s["n_moves"]].long()
    to = page.clone()
    to[src] = dst.int()
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], -1))
    s["refs_out"].copy_(torch.where(front, refs, 0))
    s["refs_out"][dst] = refs[src]
    _copy(s, src, dst)
    return _page_outputs(c, s)


def _page_outputs(c, s):
    out = {"k": s["k"]}
    if s["v"] is not s["k"]:
        out["v"] = s["v"]
    if c["do"] == "fork":
        return out | {n: s[n] for n in ("table", "len", "refs", "copy_src", "copy_dst")}
    return out | {n: s[n] for n in ("table_out", "refs_out", "move_src", "move_dst", "moves")}


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "attn":
        seen = [min(n, c["window"] or n) for n in _lengths(c)]
        row = c["Hkv"] * (c["D"] * SIZE[c["dtype"]] + (4 if c["dtype"] == "e4m3" else 0))
        io = SIZE["f32" if c["dtype"] == "f32" else "bf16"]
        return {"bytes": sum(seen) * row * (1 if c["latent"] else 2) + 4 * sum(-(-n // c["page"]) for n in seen)
                + c["B"] * c["Hq"] * (2 * c["D"] * io + 4), "flops": 4 * c["Hq"] * c["D"] * sum(seen)}
    if c["op"] == "qk":
        x, D = SIZE[c["dtype"]], c["D"]
        rows = c["Hq"] + c["Hkv"] * (2 if c["cache"] else 1)
        out = c["Hq"] * D * x + (2 * c["Hkv"] * (D * SIZE[c["cache"]] + (4 if c["cache"] == "e4m3" else 0))
                                 if c["cache"] else c["Hkv"] * D * x)
        flops = c["T"] * rows * D * 7
        return {"bytes": c["T"] * (rows * D * x + out + (12 if c["cache"] else 4)), "flops": flops}
    one = c["page"] * c["Hkv"] * (c["D"] * SIZE[c["dtype"]] + (4 if c["dtype"] == "e4m3" else 0))
    one *= 2 if c["Hkv"] > 1 else 1
    half = c["max_pages"] / 2        # rows are filled to half their width on average
    if c["do"] == "fork":
        n = c["parents"] * c["children"]
        tails = n * (1 - 1 / c["page"])
        return {"bytes": int(2 * tails * one + n * half * 4 * 2 + c["n_pages"] * 4 + 1), "flops": 0}
    held = min(c["n_pages"], c["parents"] * half)
    moves = held * (1 - held / c["n_pages"])
    return {"bytes": int(2 * moves * one + c["rows"] * c["max_pages"] * 8 + c["n_pages"] * 8 + 1), "flops": 0}


# ------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    """What run returns, from the definitions in 64 bits; the pages' outputs are whole numbers and copies."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["op"] == "attn" else _exact_qk(case, s)


def _values(x, scale):
    return x.double() if scale is None else x.double() * scale.double()[..., None]


def _exact_attn(c, s):
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    outs = torch.zeros((c["B"], Hq, D), dtype=torch.float64, device="cuda")
    lses = torch.full((c["B"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        pages = s["table"][b, lo // page: -(-n // page)].long()
        cut = slice(lo - lo // page * page, n - lo // page * page)
        for h in range(Hkv):
            pick = lambda x, z: _values(x[pages, :, h], None if z is None else z[pages, :, h]).reshape(-1, D)[cut]  # noqa: E731
            K, V = pick(s["k"], s["k_scale"]), pick(s["v"], s["v_scale"])
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            score = s["q"][b, mine].double() @ K.T * s["scale"]
            outs[b, mine] = torch.softmax(score, -1) @ V
            lses[b, mine] = torch.logsumexp(score, -1)
    return {"out": outs, "lse": lses}


def _exact_qk(c, s):
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None, None] * s["freq"])
    half = c["rot"] // 2

    def heads(x, w):
        y = x.double()
        if w is not None:
            y = y / (y.square().sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * w.double()
        if half:
            first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
            second = first + (1 if c["interleaved"] else half)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": heads(s["q"], s["wq"]), "k": heads(s["k"], s["wk"])}
    if not c["cache"]:
        return out
    at = s["pos"].long()
    where = (s["table"][s["seq"].long(), at // c["page"]].long(), at % c["page"])
    rows = {"k": out["k"], "v": s["v"].double()}
    for x, y in rows.items():
        if c["cache"] == "e4m3":
            amax = y.abs().amax(-1)
            size = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
            y = y / size[..., None]
            out[x + "_scale"] = s[x + "_scale"].double()
            out[x + "_scale"][where] = size
        out[x] = s[x + "_cache"].double()
        out[x][where] = y
    return out
