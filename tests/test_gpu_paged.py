"""Parity of the paged-cache operators (lsa_paged_attn, lsa_qk_norm_rope, lsa_page_*) with 64-bit plain forms.

Tolerances.  Attention, per query head, with A = scale * max_t sum_d |q_d k_td|, n entries and V = max |v|:
a score is an fp32 sum of D products (each sum and product off by at most 2^-23 of the terms' magnitude, tensor-core
sums may round down), scaled by constants of two roundings: |da| <= (D + 8) 2^-23 A.  A weight 2^x is off by its
argument's rounding (|x| <= 2 A / ln 2 in units of 2^-24, within the bound above) and by 2^-21 of ex2: within w = 2 (D +
16) 2^-23 A + 2^-15 of itself, relative.  For its product with V it is held in 32 bits (f32), in two bf16 pieces (half a
step of what half a step left: 2^-16, within w) or, for e4m3 rows, in one f16 number times the row's scale (half a step of
f16, r = 2^-11 of it; r = 0 otherwise).  Sums over the entries add at most n 2^-23.  So |dout| <= (2 w + r + n 2^-22) V +
half a step of the output's type, and |dlse| <= w + n 2^-23 + 2^-21 |lse| + 2^-22 (log2 and its product with ln 2).
Norm and rotation: the mean of squares is off by (D / 2 + 8) 2^-24 relative, half of that in its root; weights, root and
products add 4 roundings; an angle is off by 2^-24 pi, its sin and cos by 2 units: each output is within
((D / 4 + 12) 2^-24 + 2^-20) (|a| + |b|) plus half a step of its type.
e4m3 rows: half a step, 2^-4 of the value (2^-10 of the scale among the subnormals), with the scale within the
largest element's own error.
"""
import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_cases import lsa_mod
from paged_ref import i32

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    return lsa_mod()


def _rows(g, dtype, shape):
    x = torch.randn(shape, generator=g)
    if dtype != "e4m3":
        return x.to(DT[dtype]), None
    s = x.abs().amax(-1) / 448 * (0.25 + torch.rand(shape[:-1], generator=g))   # scales of their own
    return (x / s[..., None]).clamp(-448, 448).to(DT[dtype]), s


def _poison(x, keep):
    """NaN in every slot [n_pages, page_size] that no sequence holds."""
    bad = torch.full(x.shape[2:], float("nan")).to(x.dtype)
    y = x.clone()
    y.view(torch.uint8).reshape(*x.shape[:2], -1)[~keep] = bad.reshape(-1).view(torch.uint8)
    return y


class Case:
    def __init__(self, dtype, Hq, Hkv, D, page, lens, latent=False, window=0, seed=0, layout="nshd", q_scale=2.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.window, self.page, self.lens = dtype, window, page, list(lens)
        B, counts = len(lens), [-(-max(0, n) // page) for n in lens]
        n_pages, width = sum(counts) + 3, max(counts + [1]) + 1
        order = torch.randperm(n_pages, generator=g).tolist()
        self.table = np.full((B, width), 1 << 30, np.int32)          # never followed past a sequence's end
        keep = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(counts[b]):
                p = order.pop()
                self.table[b, i] = p
                keep[p, :min(page, n - i * page)] = True
        shape = (n_pages, page, Hkv, D)
        k, ks = _rows(g, dtype, shape)
        v, vs = (k, ks) if latent else _rows(g, dtype, shape)
        self.k64, self.v64 = ref.values(k, ks), ref.values(v, vs)
        qt = DT["f32" if dtype == "f32" else "bf16"]
        self.q = (q_scale * torch.randn((B, Hq, D), generator=g)).to(qt)
        self.scale = D ** -0.5
        self.ks = None if ks is None else torch.where(keep[..., None], ks, float("nan")).cuda()
        self.vs = self.ks if latent else None if vs is None else torch.where(keep[..., None], vs, float("nan")).cuda()
        k, v = _poison(k, keep), _poison(v, keep)
        if layout == "nhsd":          # slots inside heads
            k, v = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (k, v))
        elif layout == "pair":        # one tensor holds a page's keys, then its values
            both = torch.stack((k.view(torch.uint8), v.view(torch.uint8)), 1).cuda().view(k.dtype)
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = k.cuda(), v.cuda()
        self.k, self.v, self.latent = k, k if latent else v, latent

    def cache(self, lsa):
        if self.latent:
            return lsa.PageCache(self.k, None, self.ks)
        return lsa.PageCache(self.k, self.v, self.ks, self.vs)

    def run(self, lsa, lens=None, table=None, err=None, with_lse=True, stream=None, q=None):
        cache = self.cache(lsa)
        B, Hq, D = self.q.shape
        ws = torch.full((lsa.paged_attn_workspace_size(cache, B, Hq),), 255, dtype=torch.uint8, device="cuda")   # NaN
        q = self.q.cuda() if q is None else q
        # a row behind the last sequence, which has to stay as it is
        out = torch.full((B + 1, Hq, D), 7.0, dtype=q.dtype, device="cuda")
        lse = torch.full((B + 1, Hq), 7.0, device="cuda")
        lsa.paged_attn(q, cache, i32(self.table if table is None else table), i32(self.lens if lens is None else lens),
                       out[:B], ws, lse=lse[:B] if with_lse else None, window=self.window, scale=self.scale, err=err,
                       stream=stream)
        torch.cuda.synchronize()
        assert (out[B] == 7).all() and (lse[B] == 7).all()
        return out[:B], lse[:B]

    def check(self, lsa, **kw):
        out, lse = self.run(lsa, **kw)
        lens, table = kw.get("lens") or self.lens, self.table if kw.get("table") is None else kw["table"]
        q = self.q.double().numpy()
        o, z, A, V = ref.attention(q, self.k64, self.v64, table, lens, self.page, self.window, self.scale)
        D, n = q.shape[2], np.array([[max(1, m)] for m in lens])
        w = 2 * (D + 16) * 2.0 ** -23 * A + 2.0 ** -15
        r = 2.0 ** -11 if self.dtype == "e4m3" else 0.0
        tol = ((2 * w + r + n * 2.0 ** -22) * V)[..., None] + HALF_STEP["f32" if self.dtype == "f32" else "bf16"] * np.abs(o)
        d = np.abs(out.double().cpu().numpy() - o)
        assert (d <= tol + 1e-30).all(), f"out: {np.nanmax(d - tol)} over its bound, at {np.argwhere(~(d <= tol + 1e-30))[:3]}"
        z_gpu = lse.double().cpu().numpy()
        assert ((z == -np.inf) == (z_gpu == -np.inf)).all()
        fin = z > -np.inf
        dz = np.abs(np.where(fin, z_gpu, 0) - np.where(fin, z, 0))
        tz = w + n * 2.0 ** -23 + 2.0 ** -21 * np.abs(np.where(fin, z, 0)) + 2.0 ** -22
        assert (dz <= tz).all(), f"lse: {np.max(dz - tz)} over its bound"
        return out, lse


TYPES = ["f32", "bf16", "e4m3"]
# query heads, kv heads, head dim
HEADS = [(1, 1, 64), (8, 8, 32), (6, 2, 64), (8, 1, 128), (10, 2, 128), (24, 2, 96), (16, 1, 80), (33, 1, 64),
         (32, 2, 256), (20, 4, 192), (9, 1, 512), (4, 2, 16), (64, 1, 128), (5, 1, 48), (12, 1, 320)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_attention_heads(lsa, dtype, Hq, Hkv, D):
    Case(dtype, Hq, Hkv, D, 16, [0, 1, 15, 16, 17, 33, 130, 700], seed=D + Hq).check(lsa)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256, 1000])
def test_attention_page_sizes(lsa, dtype, page):
    Case(dtype, 8, 2, 64, page, [1, page - 1, page, page + 1, 3 * page + 2, 999], seed=page).check(lsa)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq", [1, 7, 16, 128])
def test_attention_latent(lsa, dtype, Hq):
    Case(dtype, Hq, 1, 512, 64, [0, 1, 63, 64, 65, 200, 1500], latent=True, seed=Hq).check(lsa)


@pytest.mark.parametrize("dtype,Hq,lens", [("bf16", 128, [4000, 1, 0, 9001]), ("bf16", 100, [300, 129]),
                                           ("e4m3", 64, [5000]), ("bf16", 256, [64, 128, 700])])
def test_attention_latent_long(lsa, dtype, Hq, lens):
    Case(dtype, Hq, 1, 512, 48, lens, latent=True, seed=Hq + 1).check(lsa)


@pytest.mark.parametrize("page", [1, 8, 16, 24, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("window,layout", [(0, "nshd"), (0, "nhsd"), (203, "nshd"), (256, "nhsd")])
def test_attention_latent_pages_and_windows(lsa, page, window, layout):
    """Rows that lie side by side in a page or do not, windows that begin inside a tile, bad pages, two latent heads."""
    c = Case("bf16", 40, 2, 512, page, [1, 64, 200, 0, 1000, 3001, 128], latent=True, seed=page, window=window, layout=layout)
    c.check(lsa)
    table = c.table.copy()
    table[4, 300 // page], table[5, 2900 // page], table[2, 0] = -1, 1 << 29, -7
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(lsa, table=table, err=err)
    assert err.item() == (1 if window == 0 or 2900 >= 3001 - window else 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_split_over_the_length(lsa, dtype):
    Case(dtype, 8, 1, 128, 64, [20001], seed=1).check(lsa)
    Case(dtype, 8, 2, 64, 16, [9000, 0, 0, 1, 33000, 0], seed=2).check(lsa)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_many_sequences(lsa, dtype):
    r = np.random.default_rng(3)
    lens = np.where(r.random(700) < 0.2, 0, r.integers(0, 300, 700)).tolist() + [4000]
    Case(dtype, 4, 2, 32, 8, lens, seed=3).check(lsa)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_attention_window(lsa, dtype, window):
    Case(dtype, 6, 2, 64, 16, [0, 1, 16, 99, 100, 101, 1000, 6000], window=window, seed=window).check(lsa)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["nhsd", "pair"])
def test_attention_layouts_and_strided_queries(lsa, dtype, layout):
    c = Case(dtype, 6, 3, 64, 16, [40, 1, 500], layout=layout, seed=5)
    qkv = torch.full((3, 6 + 6, 64), float("nan"), dtype=c.q.dtype, device="cuda")
    qkv[:, :6] = c.q.cuda()
    a, _ = c.check(lsa, q=qkv[:, :6])
    b, _ = c.run(lsa)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_sharp_scores(lsa, dtype):
    """Scores in the hundreds: one entry takes all the weight; the bound grows with the scores."""
    Case(dtype, 8, 2, 64, 16, [5, 300, 2000], seed=6, q_scale=60.0).check(lsa)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_bad_pages_are_left_out_and_reported(lsa, dtype):
    c = Case(dtype, 4, 2, 64, 16, [100, 40, 3000], seed=7)
    table = c.table.copy()
    table[0, 1], table[0, 3], table[2, 100] = -1, 1 << 20, -(1 << 31)
    table[1, :3] = -5                                  # nothing of sequence 1 is left
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.check(lsa, table=table, err=err)
    assert err.item() == 1 and (out[1] == 0).all() and (lse[1] == -np.inf).all()
    c.check(lsa, table=table)                          # no error word


def test_attention_lengths_outside_the_table(lsa):
    c = Case("bf16", 4, 2, 64, 16, [100, 40], seed=8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(lsa, lens=[-3, 40], err=err)
    assert err.item() == 0
    # row 1 holds 3 pages; rows reach 8: a length past them is cut, and the entries without a page are left out
    out, _ = c.run(lsa, lens=[100, 1 << 30], err=err)
    assert err.item() in (1, 3)
    a, _ = c.run(lsa)
    assert torch.equal(out[0], a[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_infinite_and_nan_scores(lsa, dtype):
    c = Case(dtype, 2, 1, 64, 16, [50, 50, 50, 300], seed=9)
    c.q = c.q.abs() + 0.01                             # positive: an entry of -inf keys scores -inf
    page = c.table[:, 0]
    for x in (c.k64,):
        x[page[0], 3] = -np.inf                        # one entry without weight
        for i in range(4):
            x[c.table[1, i]] = -np.inf                 # a sequence without any
        x[page[2], 5] = np.nan
        x[page[3], 0] = -np.inf
    k = torch.from_numpy(c.k64).to(c.k.dtype).cuda()
    c.k.copy_(torch.where(torch.isnan(c.k), c.k, k))
    c.k[int(page[2]), 5] = float("nan")
    out, lse = c.run(lsa)
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()
    o, z, _, _ = ref.attention(c.q.double().numpy(), c.k64, c.v64, c.table, c.lens, 16, 0, c.scale)
    for b in (0, 3):
        np.testing.assert_allclose(out[b].double().cpu().numpy(), o[b], rtol=2e-2, atol=2e-2)
        np.testing.assert_allclose(lse[b].double().cpu().numpy(), z[b], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_same_bits_on_another_stream_in_a_graph_and_without_lse(lsa, dtype):
    c = Case(dtype, 8, 2, 128, 16, [3000, 1, 0, 700], seed=10)
    a, za = c.check(lsa)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, zb = c.run(lsa, stream=s)
    d, _ = c.run(lsa, with_lse=False)
    assert torch.equal(a, b) and torch.equal(za, zb) and torch.equal(a, d)
    cache, q, table, lens = c.cache(lsa), c.q.cuda(), i32(c.table), i32(c.lens)
    ws = torch.empty(lsa.paged_attn_workspace_size(cache, 4, 8), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(a), torch.zeros_like(za)
    call = lambda: lsa.paged_attn(q, cache, table, lens, out, ws, lse=lse, scale=c.scale)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    # a replay follows the lengths that are there then
    lens.copy_(i32([10, 5, 0, 699]))
    g.replay()
    b, zb = c.run(lsa, lens=[10, 5, 0, 699])
    # (bit for bit: sequence 1 now reads slots that no one has written, which hold NaN)
    assert torch.equal(out.view(torch.uint8), b.view(torch.uint8)) and torch.equal(lse.view(torch.uint8),
                                                                                   zb.view(torch.uint8))
    lens.copy_(i32(c.lens))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a) and torch.equal(lse, za)


@pytest.mark.parametrize("Hq", [20, 128])
def test_attention_latent_sharp_scores(lsa, Hq):
    """Scores in the hundreds: the references move from tile to tile, and what was summed up is rescaled."""
    Case("bf16", Hq, 1, 512, 64, [5, 300, 2000, 9000], latent=True, seed=Hq, q_scale=60.0).check(lsa)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,tile,latent", [("bf16", 4, 1, 128, 64, False), ("e4m3", 4, 1, 128, 128, False),
                                                       ("f32", 4, 1, 128, 32, False), ("bf16", 16, 1, 512, 64, True)])
@pytest.mark.parametrize("B", [2, 30, 70])
def test_attention_where_segments_are_whole_or_split(lsa, dtype, Hq, Hkv, D, tile, latent, B):
    """Reaches of 5 and 8 tiles, where few and many segments change from one way to the other, and one entry more."""
    for tiles in (5, 8):
        for more in (0, 1):
            n = tiles * tile + more
            lens = [n, 0, n - 1, 1, tile] + [(37 * i) % (n + 1) for i in range(B)]
            Case(dtype, Hq, Hkv, D, 1, lens[:B], latent=latent, seed=B + n).check(lsa)


def test_attention_two_calls_at_once(lsa):
    """Calls on two streams with workspaces of their own, over one cache."""
    for dtype, Hq, D, latent in (("bf16", 8, 128, False), ("bf16", 40, 512, True), ("f32", 8, 64, False)):
        c = Case(dtype, Hq, 1, D, 16, [3000, 1, 0, 9000, 700], latent=latent, seed=11)
        want, lse = c.check(lsa)
        cache, q, table, lens = c.cache(lsa), c.q.cuda(), i32(c.table), i32(c.lens)
        streams = [torch.cuda.Stream() for _ in range(2)]
        ws = [torch.empty(lsa.paged_attn_workspace_size(cache, 5, Hq), dtype=torch.uint8, device="cuda") for _ in streams]
        outs = [torch.zeros((6,) + want.shape, dtype=want.dtype, device="cuda") for _ in streams]
        torch.cuda.synchronize()
        for i in range(6):
            for s, w, o in zip(streams, ws, outs):
                lsa.paged_attn(q, cache, table, lens, o[i], w, scale=c.scale, stream=s)
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(x, want) for x in o)


def test_attention_offsets_past_32_bits(lsa):
    """A cache of more than 2^32 bytes, with a sequence on its last pages."""
    n_pages, page, D = 70000, 64, 512                  # 4.6 GB of bf16 rows
    k = torch.zeros((n_pages, page, 1, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    use = [n_pages - 1, 3, n_pages - 2, 66000]
    for p in use:
        k[p] = torch.randn((page, 1, D), generator=g, device="cuda").bfloat16()
    q = torch.randn((1, 16, D), generator=g, device="cuda").bfloat16()
    cache, n = lsa.PageCache(k), 4 * page - 5
    ws = torch.empty(lsa.paged_attn_workspace_size(cache, 1, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    lsa.paged_attn(q, cache, i32([use]), i32([n]), out, ws)
    small = k[use].double().cpu().numpy()
    o, _, _, _ = ref.attention(q.double().cpu().numpy(), small, small, np.arange(4, dtype=np.int32)[None], [n], page, 0,
                               D ** -0.5)
    np.testing.assert_allclose(out.double().cpu().numpy(), o, rtol=2.0 ** -7, atol=1e-3)


# ------------------------------------------------------------------- norm, rotation, append

QK = [(1, 8, 2, 128, 128, False), (3, 4, 1, 64, 32, True), (5, 6, 3, 80, 20, False), (7, 2, 2, 96, 62, False),
      (2, 3, 1, 512, 512, False), (2, 3, 1, 512, 2, True), (9, 5, 5, 256, 128, True), (4, 4, 2, 16, 6, False),
      (6, 1, 1, 48, 0, False), (700, 8, 2, 128, 64, False), (33, 16, 4, 32, 32, True), (5000, 4, 1, 64, 64, False),
      (3, 3, 1, 512, 254, False)]


def _tol(size, y, D, dtype):
    return ((D / 4 + 12) * 2.0 ** -24 + 2.0 ** -20) * size + HALF_STEP[dtype] * np.abs(y) + 1e-37


@pytest.mark.parametrize("dtype,kind", [("f32", ""), ("bf16", ""), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "e4m3"),
                                        ("f32", "e4m3")])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved", QK)
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope_append(lsa, dtype, kind, T, Hq, Hkv, D, rot, interleaved, norm):
    g = torch.Generator().manual_seed(T * 7 + D + rot)
    dt, page, eps = DT[dtype], 5, 1e-5
    qkv = (3 * torch.randn((T, Hq + 2 * Hkv, D), generator=g)).to(dt)
    if Hkv > 1:
        qkv[0, Hq + Hkv] = 0                          # a value row of zeros
    wq, wk = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norm else None for _ in range(2)]
    pos = torch.randint(-50, 1 << 21, (T,), generator=g).int()
    freq, _ = lsa.rope_frequencies(rot, 10000.0) if rot else (torch.zeros(0, dtype=torch.float64), 1.0)
    mscale, inverse = 1.25, T % 2 == 0
    dev = qkv.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    rope = lsa.Rope(freq.cuda(), interleaved, inverse, mscale)
    q_out = torch.zeros((T, Hq, D), dtype=dt, device="cuda")
    k_out = torch.zeros((T, Hkv, D), dtype=dt, device="cuda") if kind in ("", "bf16") else None
    kw = {}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if kind:
        rows = min(T, 6)
        seq = torch.arange(T) % rows
        at = torch.arange(T) // rows + 2
        at[::7] = -1                                  # not appended
        if T > 1:
            seq[1] = -1
        width = int(at.max().clamp(min=0)) // page + 1
        n_pages = rows * width + 2
        table = torch.randperm(n_pages, generator=g)[:rows * width].reshape(rows, width)
        kc, vc = (torch.full((n_pages, page, Hkv, D), 3.0, device="cuda").to(DT[kind]) for _ in range(2))
        ks, vs = (torch.full((n_pages, page, Hkv), 9.0, device="cuda") if kind == "e4m3" else None for _ in range(2))
        kw = dict(cache=lsa.PageCache(kc, vc, ks, vs), table=i32(table), seq=i32(seq), at=i32(at), v=v, err=err)
    lsa.qk_norm_rope(q, k, q_out=q_out, k_out=k_out, q_weight=None if wq is None else wq.cuda(),
                     k_weight=None if wk is None else wk.cuda(), eps=eps, pos=i32(pos), rope=rope, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    x = qkv.double().numpy()
    n64 = lambda w: None if w is None else w.double().numpy()  # noqa: E731
    args = (eps, pos.numpy(), freq.numpy(), rot, interleaved, inverse, mscale)
    yq, sq = ref.norm_rope(x[:, :Hq], n64(wq), *args)
    yk, sk = ref.norm_rope(x[:, Hq:Hq + Hkv], n64(wk), *args)
    yv = x[:, Hq + Hkv:]
    d = np.abs(q_out.double().cpu().numpy() - yq)
    assert (d <= _tol(sq, yq, D, dtype)).all(), np.max(d - _tol(sq, yq, D, dtype))
    if k_out is not None:
        assert (np.abs(k_out.double().cpu().numpy() - yk) <= _tol(sk, yk, D, dtype)).all()
    if not kind:
        return
    written = np.zeros((n_pages, page), bool)
    for name, c, s, y, size in (("k", kc, ks, yk, sk), ("v", vc, vs, yv, np.abs(yv))):
        got = ref.values(c, s)
        for t in range(T):
            if at[t] < 0 or seq[t] < 0:
                continue
            p, o = int(table[seq[t], int(at[t]) // page]), int(at[t]) % page
            written[p, o] = True
            if kind != "e4m3":
                assert (np.abs(got[p, o] - y[t]) <= _tol(size[t], y[t], D, kind)).all(), (name, t)
                continue
            own = ((D / 4 + 12) * 2.0 ** -24 + 2.0 ** -20) * size[t]
            want = np.abs(y[t]).max(-1) / 448
            want[want == 0] = 1
            sc = s[p, o].double().cpu().numpy()
            assert (np.abs(sc - want) <= own.max(-1) / 448 + want * 2.0 ** -23).all(), (name, t)
            assert (np.abs(got[p, o] - y[t]) <= 2.0 ** -4 * np.abs(y[t]) + 2.0 ** -10 * sc[:, None] + 2 * own).all(), (name, t)
        left = torch.from_numpy(~written).cuda()
        assert (c[left].float() == 3).all() and (s is None or (s[left] == 9).all()), name


@pytest.mark.parametrize("dtype,kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("shape", [(11, 3, 2, 256, 38), (300, 5, 1, 64, 20), (4, 2, 1, 512, 98), (2, 3, 3, 16, 10),
                                   (3, 2, 1, 80, 78)])
def test_norm_rope_interleaved_parts_that_turn_in_part(lsa, dtype, kind, shape):
    """Interleaved pairs of which a lane's 16 bytes hold some that turn and some that do not."""
    test_norm_rope_append(lsa, dtype, kind, *shape, True, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 20, True), (256, 38, True), (64, 20, False), (128, 64, True)])
def test_elements_that_do_not_turn_never_meet_their_neighbours(lsa, dtype, D, rot, interleaved):
    g = torch.Generator(device="cuda").manual_seed(D + rot)
    x = torch.randn((5, 3, D), generator=g, device="cuda").to(DT[dtype])
    bad = x.clone()
    bad[:, :, rot], bad[:, :, rot + 1], bad[:, :, D - 1] = float("inf"), float("nan"), -float("inf")
    freq, _ = lsa.rope_frequencies(rot)
    rope, pos, out, want = lsa.Rope(freq.cuda(), interleaved), i32(range(5)), torch.empty_like(x), torch.empty_like(x)
    lsa.qk_norm_rope(x, q_out=want, pos=pos, rope=rope)
    lsa.qk_norm_rope(bad, q_out=out, pos=pos, rope=rope)
    want[:, :, rot], want[:, :, rot + 1], want[:, :, D - 1] = float("inf"), float("nan"), -float("inf")
    bits = {"f32": torch.int32, "bf16": torch.int16}[dtype]
    keep = torch.arange(D, device="cuda") != rot + 1
    assert torch.equal(out[:, :, keep].view(bits), want[:, :, keep].view(bits)) and out[:, :, rot + 1].isnan().all()


def test_norm_rope_in_place_queries_only_and_latent_append(lsa):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((9, 6, 64), generator=g, device="cuda")
    freq, _ = lsa.rope_frequencies(64)
    rope, pos = lsa.Rope(freq.cuda()), i32(range(9))
    out = torch.empty((9, 6, 64), device="cuda")
    lsa.qk_norm_rope(x, q_out=out, pos=pos, rope=rope)
    y = x.clone()
    lsa.qk_norm_rope(y, q_out=y, pos=pos, rope=rope)
    assert torch.equal(out, y)
    back = torch.empty_like(y)
    lsa.qk_norm_rope(y, q_out=back, pos=pos, rope=lsa.Rope(freq.cuda(), inverse=True))
    assert (back - x).abs().max() <= 2.0 ** -18 * x.abs().max()
    # one kv head whose rows are keys and values
    k = torch.randn((9, 1, 64), generator=g, device="cuda")
    rows = torch.zeros((4, 4, 1, 64), device="cuda")
    lsa.qk_norm_rope(x, k, q_out=out, pos=pos, rope=rope, cache=lsa.PageCache(rows), table=i32([[2, 0, 3]]),
                     seq=i32([0] * 9), at=pos)
    kk = torch.empty_like(k)
    lsa.qk_norm_rope(x, k, q_out=out, k_out=kk, pos=pos, rope=rope)
    assert torch.equal(torch.cat((rows[2], rows[0], rows[3]))[:9], kk) and (rows[1] == 0).all()
    # no token: nothing is launched
    lsa.qk_norm_rope(x[:0], q_out=out[:0], pos=pos[:0], rope=rope)


def test_rotation_gradient_is_the_inverse_rotation(lsa):
    """d/dx of <c, R x> is R^-1 c, against differences in 64 bits of the formula and against the kernel's own."""
    g = torch.Generator(device="cuda").manual_seed(3)
    freq, _ = lsa.rope_frequencies(32)
    c = torch.randn((5, 2, 48), generator=g, device="cuda")
    pos = i32([0, 1, 77, 1000, 500000])
    grad = torch.empty_like(c)
    lsa.qk_norm_rope(c, q_out=grad, pos=pos, rope=lsa.Rope(freq.cuda(), inverse=True))
    c64, p = c.double().cpu().numpy(), pos.cpu().numpy()
    x = np.random.default_rng(0).standard_normal(c64.shape)
    for i in (0, 5, 15, 16, 31, 32, 47):
        e = np.zeros(48)
        e[i] = 1.0
        step = lambda s: (c64 * ref.norm_rope(x + s * e, None, 0, p, freq.numpy(), 32, False, False, 1.0)[0]).sum(-1)  # noqa: E731
        diff = (step(1.0) - step(-1.0)) / 2               # the rotation is linear: the difference is its gradient
        size = np.abs(c64).max(-1) * 2
        assert (np.abs(grad[..., i].double().cpu().numpy() - diff) <= 2.0 ** -19 * size).all(), i


def test_append_refuses_entries_outside_the_table(lsa):
    x = torch.randn((5, 2, 32), device="cuda")
    k = torch.randn((5, 1, 32), device="cuda")
    rows = torch.zeros((3, 4, 1, 32), device="cuda")
    vals = torch.zeros_like(rows)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = i32([[0, 1], [2, 9], [-1, -1]])
    # row 5 of 3, entry 8 of 8, page 9 of 3, page -1; and one good token
    lsa.qk_norm_rope(x, k, k, q_out=x, cache=lsa.PageCache(rows, vals), table=table, seq=i32([5, 0, 1, 2, 1]),
                     at=i32([0, 8, 4, 0, 3]), err=err)
    torch.cuda.synchronize()
    assert err.item() == 1
    assert torch.equal(rows[2, 3], k[4]) and torch.equal(vals[2, 3], k[4])
    rows[2, 3] = 0
    assert (rows == 0).all()


# ------------------------------------------------------------------------------------- pages

class Pool:
    """The library's books beside the model's."""

    def __init__(self, lsa, n_rows, max_pages, n_pages, page_size):
        self.lsa, self.m = lsa, ref.Books(n_rows, max_pages, n_pages, page_size)
        self.pt = lsa.PageTable.empty(n_rows, max_pages, n_pages, page_size)

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.pt.table.cpu().numpy(), self.m.table())
        assert self.pt.len.tolist() == self.m.len
        assert self.pt.refs.tolist() == self.m.refs

    def _err(self, want, err):
        torch.cuda.synchronize()
        assert err.item() == {None: 0, "invalid": 1, "capacity": 3}[want], (want, err.item())

    def grow(self, add):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lsa.page_grow(self.pt, i32(add), err)
        self._err(self.m.grow(add), err)
        self.same()

    def fork(self, src, dst):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cs, cd = i32([5] * len(src)), i32([5] * len(src))
        self.lsa.page_fork(self.pt, i32(src), i32(dst), cs, cd, err)
        want, ms, md = self.m.fork(src, dst)
        self._err(want, err)
        assert cs.tolist() == ms and cd.tolist() == md
        self.same()
        return cs, cd

    def free(self, rows):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lsa.page_free(self.pt, i32(rows), err)
        self._err(self.m.free(rows), err)
        self.same()

    def compact(self, in_place):
        n, pt = self.m.n_pages, self.pt
        t, r = (pt.table, pt.refs) if in_place else (torch.full_like(pt.table, 5), torch.full_like(pt.refs, 5))
        src, dst, moves = i32([5] * n), i32([5] * n), i32([5])
        ws = torch.full((self.lsa.page_compact_workspace_size(n),), 255, dtype=torch.uint8, device="cuda")
        before = pt.table.clone(), pt.refs.clone()
        self.lsa.page_compact(pt, t, r, src, dst, moves, ws)
        torch.cuda.synchronize()
        if not in_place:
            assert torch.equal(pt.table, before[0]) and torch.equal(pt.refs, before[1])
            self.pt = self.lsa.PageTable(t, pt.len, r, pt.page_size)
        ms, md, m = self.m.compact()
        assert moves.item() == m and src.tolist() == ms and dst.tolist() == md
        self.same()
        return src, dst, moves


@pytest.mark.parametrize("n_rows,max_pages,n_pages,page,seed", [(1, 1, 1, 1, 0), (5, 4, 13, 3, 1), (40, 30, 300, 16, 2),
                                                               (1500, 9, 6001, 7, 3), (64, 700, 40000, 64, 4),
                                                               (3000, 30, 70001, 3, 5)])
def test_page_books_against_the_model(lsa, n_rows, max_pages, n_pages, page, seed):
    r = np.random.default_rng(seed)
    pool = Pool(lsa, n_rows, max_pages, n_pages, page)
    pool.same()
    for step in range(14):
        some = r.random(n_rows) < 0.5
        pool.grow(np.where(some, r.integers(-3, max(2, page * max_pages // 6), n_rows), 0).tolist())
        empty = [i for i, n in enumerate(pool.m.len) if n == 0]
        if empty:
            dst = r.permutation(empty)[: int(r.integers(1, len(empty) + 1))].tolist()
            pool.fork(r.integers(0, n_rows, len(dst)).tolist(), dst)
        if step % 3 == 2:
            pool.compact(in_place=step % 2 == 0)
        pool.free(r.integers(0, n_rows, int(r.integers(1, n_rows + 1))).tolist())     # some rows named twice
    pool.compact(in_place=True)


def test_page_calls_that_do_not_fit_change_nothing(lsa):
    pool = Pool(lsa, 4, 3, 5, 4)
    pool.grow([5, 0, 9, 0])            # 2 + 3 pages: the pool is full
    pool.grow([4, 0, 0, 0])            # no page left
    pool.grow([3, 0, 0, 0])            # fits in the last page
    pool.grow([5, 0, 0, 0])            # past max_pages
    pool.grow([0, (1 << 31) - 1, 0, 0])
    pool.fork([2], [1])                # the last page is in part filled, and no page is left
    pool.fork([0], [1])                # full pages alone: shared
    pool.fork([0], [2])                # not empty
    pool.fork([0, 2], [3, 3])          # named twice
    pool.fork([4], [3])
    pool.fork([0], [-1])
    pool.free([0, 0, 7, -1])
    pool.free([1, 2, 3])
    assert pool.m.refs == [0] * 5


def test_page_books_with_bad_entries_stay_in_bounds(lsa):
    """Entries that name no page, or a free one, are not followed."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pt = lsa.PageTable(i32([[7, -9, 1], [0, 0, 0]]), i32([12, 0]), i32([0, 1, 0, 0]), 4)
    cs, cd = i32([5]), i32([5])
    lsa.page_fork(pt, i32([0]), i32([1]), cs, cd, err)
    torch.cuda.synchronize()
    assert err.item() == 0 and pt.table[1].tolist() == [7, -9, 1] and pt.refs.tolist() == [0, 2, 0, 0]
    pt.table[1, 2] = 3
    lsa.page_free(pt, i32([1]), err)
    torch.cuda.synchronize()
    assert err.item() == 1 and pt.refs.tolist() == [0, 2, 0, 0] and pt.table[1].tolist() == [-1, -1, -1]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,layout", [((9, 16, 2, 64), "nshd"), ((9, 5, 3, 48), "nhsd"), ((7, 1, 1, 512), "nshd"),
                                          ((6, 100, 1, 32), "pair"), ((5, 33, 4, 80), "gaps"), ((5, 64, 8, 256), "nshd")])
def test_page_copy(lsa, dtype, shape, layout):
    g = torch.Generator().manual_seed(1)
    k, ks = _rows(g, dtype, shape)
    v, vs = _rows(g, dtype, shape)
    if ks is not None:
        ks, vs = ks.cuda(), vs.cuda()
    if layout == "nhsd":
        k, v = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (k, v))
    elif layout == "pair":
        both = torch.stack((k.view(torch.uint8), v.view(torch.uint8)), 1).cuda().view(k.dtype)
        k, v = both[:, 0], both[:, 1]
    elif layout == "gaps":                       # rows 32 elements apart from their neighbours
        big = torch.zeros((*shape[:3], 2 * (shape[3] + 32))).to(k.dtype).cuda()
        big[..., :shape[3]], big[..., shape[3] + 32:2 * shape[3] + 32] = k.cuda(), v.cuda()
        k, v = big[..., :shape[3]], big[..., shape[3] + 32:2 * shape[3] + 32]
    else:
        k, v = k.cuda(), v.cuda()
    bits = lambda x: x.clone().view(torch.uint8) if x is not None else None  # noqa: E731
    src, dst = [0, 3, -1, 2, 0], [4, 1, 2, -1, 0]
    want = [bits(x) for x in (k, v, ks, vs)]
    for w in want:
        if w is not None:
            w[4], w[1] = w[0].clone(), w[3].clone()
    lsa.page_copy(lsa.PageCache(k, v, ks, vs), i32(src), i32(dst))
    torch.cuda.synchronize()
    for x, w in zip((k, v, ks, vs), want):
        assert w is None or torch.equal(bits(x), w)
    if layout == "gaps":
        big.view(torch.uint8)
        e = k.element_size()
        raw = big.view(torch.uint8).reshape(*shape[:3], -1)
        assert (raw[..., shape[3] * e:(shape[3] + 32) * e] == 0).all() and (raw[..., (2 * shape[3] + 32) * e:] == 0).all()


def test_page_copy_counts_and_bad_pages(lsa):
    k = torch.arange(6, device="cuda", dtype=torch.float32)[:, None, None, None].expand(6, 4, 1, 16).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = lsa.PageCache(k)
    for count, want in ((0, [0, 1, 2, 3, 4, 5]), (-4, [0, 1, 2, 3, 4, 5]), (1, [0, 0, 2, 3, 4, 5]), (9, [0, 0, 2, 5, 4, 5])):
        lsa.page_copy(cache, i32([0, 5]), i32([1, 3]), count=i32([count]), err=err)
        assert k[:, 3, 0, 15].tolist() == want and err.item() == 0
    lsa.page_copy(cache, i32([6, 0]), i32([1, 1 << 30]), err=err)
    assert k[:, 0, 0, 0].tolist() == [0, 0, 2, 5, 4, 5] and err.item() == 1


# ---------------------------------------------------------------- together, as a program uses them

@pytest.mark.parametrize("kind", TYPES)
def test_decode_steps_over_forked_and_packed_pages(lsa, kind):
    """Prompts are appended, decode steps grow, append and attend, a sequence is forked twice, its parent freed, and the
    pool packed; every step's attention against 64 bits over the heads that were appended."""
    Hq, Hkv, D, page, n_rows, eps = 6, 2, 64, 8, 6, 1e-6
    dtype = "f32" if kind == "f32" else "bf16"
    g = torch.Generator(device="cuda").manual_seed(4)
    pool = Pool(lsa, n_rows, 12, 40, page)
    kc, vc = (torch.zeros((40, page, Hkv, D), device="cuda").to(DT[kind]) for _ in range(2))
    ks, vs = (torch.zeros((40, page, Hkv), device="cuda") if kind == "e4m3" else None for _ in range(2))
    cache = lsa.PageCache(kc, vc, ks, vs)
    freq, m = lsa.rope_frequencies(D, 10000.0, "yarn", 4.0, 32)
    rope = lsa.Rope(freq.cuda(), mscale=m)
    wq, wk = (1 + 0.1 * torch.randn((2, D), generator=g, device="cuda")).to(DT[dtype])
    hist = {r: [] for r in range(n_rows)}         # (key, value) rows in 64 bits, as they lie in the cache
    ws = torch.empty(lsa.paged_attn_workspace_size(cache, n_rows, Hq), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(new):
        """new: tokens of each row; attends with each row's last token."""
        pool.grow([new.get(r, 0) for r in range(n_rows)])
        seq = [r for r in new for _ in range(new[r])]
        at = [pool.m.len[r] - new[r] + i for r in new for i in range(new[r])]
        x = torch.randn((len(seq), Hq + 2 * Hkv, D), generator=g, device="cuda").to(DT[dtype])
        q_out = torch.empty((len(seq), Hq, D), dtype=DT[dtype], device="cuda")
        lsa.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q_out=q_out, q_weight=wq, k_weight=wk, eps=eps,
                         pos=i32(at), rope=rope, cache=cache, table=pool.pt.table, seq=i32(seq), at=i32(at), err=err)
        x64, pos = x.double().cpu().numpy(), np.array(at)
        args = (eps, pos, freq.numpy(), D, False, False, m)
        yq, sq = ref.norm_rope(x64[:, :Hq], wq.double().cpu().numpy(), *args)
        yk, sk = ref.norm_rope(x64[:, Hq:Hq + Hkv], wk.double().cpu().numpy(), *args)
        assert (np.abs(q_out.double().cpu().numpy() - yq) <= _tol(sq, yq, D, dtype)).all()
        K, V = ref.values(kc, ks), ref.values(vc, vs)
        for t, (r, a) in enumerate(zip(seq, at)):
            p = pool.m.rows[r][a // page]
            lim = 2.0 ** -4 * np.abs(yk[t]) + 2.0 ** -9 * np.abs(yk[t]).max() / 448 + 2.0 ** -16 * sk[t] \
                if kind == "e4m3" else _tol(sk[t], yk[t], D, dtype)
            assert (np.abs(K[p, a % page] - yk[t]) <= lim).all()
            hist[r].append((K[p, a % page].copy(), V[p, a % page].copy()))
        last = {r: max(i for i, s in enumerate(seq) if s == r) for r in new}
        return torch.stack([q_out[last[r]] if r in last else torch.zeros_like(q_out[0]) for r in range(n_rows)])

    def attend(q):
        out, lse = torch.empty_like(q), torch.empty((n_rows, Hq), device="cuda")
        lsa.paged_attn(q, cache, pool.pt.table, pool.pt.len, out, ws, lse=lse, err=err)
        torch.cuda.synchronize()
        for r in range(n_rows):
            if not hist[r]:
                assert (out[r] == 0).all() and (lse[r] == -np.inf).all()
                continue
            K, V = (np.stack([h[i] for h in hist[r]]) for i in (0, 1))     # [n, Hkv, D]
            o, z, A, vm = ref.attention(q[r:r + 1].double().cpu().numpy(), K[:, None], V[:, None],
                                        np.arange(len(K), dtype=np.int32)[None], [len(K)], 1, 0, D ** -0.5)
            w = 2 * (D + 16) * 2.0 ** -23 * A + 2.0 ** -15
            f16 = 2.0 ** -11 if kind == "e4m3" else 0.0
            tol = ((2 * w + f16 + len(K) * 2.0 ** -22) * vm)[..., None] + HALF_STEP[dtype] * np.abs(o)
            assert (np.abs(out[r:r + 1].double().cpu().numpy() - o) <= tol).all(), r
            assert np.abs(lse[r:r + 1].double().cpu().numpy() - z).max() <= w.max() + 1e-4
        return out

    def fork(src, dst):
        cs, cd = pool.fork(src, dst)
        lsa.page_copy(cache, cs, cd, err=err)
        for s, d in zip(src, dst):
            hist[d] = list(hist[s])

    attend(append({0: 19, 1: 8, 2: 1}))                      # prompts
    for _ in range(3):
        attend(append({0: 1, 1: 1, 2: 1}))
    fork([0, 0, 1], [3, 4, 5])
    q = append({r: 1 for r in range(n_rows)})                # the forks go their own ways
    attend(q)
    pool.free([0, 2])
    hist[0], hist[2] = [], []
    out = attend(q)
    src, dst, moves = pool.compact(in_place=True)
    lsa.page_copy(cache, src, dst, count=moves, err=err)
    assert torch.equal(out, attend(q)) and moves.item() > 0
    for _ in range(9):
        attend(append({1: 1, 3: 1, 4: 1, 5: 1}))
    assert err.item() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_captured_decode_step_follows_the_books(lsa, kind):
    """grow, norm/rotate/append and attention captured once: each replay is the next step, as without a graph."""
    B, Hq, Hkv, D, page, steps = 5, 8, 2, 64, 4, 11
    g = torch.Generator(device="cuda").manual_seed(12)
    xs = torch.randn((steps, B, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
    freq, _ = lsa.rope_frequencies(D)
    rope = lsa.Rope(freq.cuda())
    add = i32([1, 1, 0, 1, 2])                      # row 2 waits; row 4 leaves a hole that later steps do not write

    def run(captured):
        pages = lsa.PageTable.empty(B, 8, B * 8, page)
        k, v = (torch.zeros((B * 8, page, Hkv, D), device="cuda").to(DT[kind]) for _ in range(2))
        ks, vs = (torch.ones((B * 8, page, Hkv), device="cuda") if kind == "e4m3" else None for _ in range(2))
        cache = lsa.PageCache(k, v, ks, vs)
        ws = torch.empty(lsa.paged_attn_workspace_size(cache, B, Hq), dtype=torch.uint8, device="cuda")
        x, at = torch.empty_like(xs[0]), torch.empty_like(pages.len)
        q, out = torch.empty((B, Hq, D), dtype=x.dtype, device="cuda"), torch.empty((B, Hq, D), dtype=x.dtype, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")

        def step():
            at.copy_(pages.len)
            lsa.page_grow(pages, add, err)
            at.masked_fill_(add == 0, -1)
            lsa.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q_out=q, pos=at, rope=rope, cache=cache,
                             table=pages.table, at=at, err=err)
            lsa.paged_attn(q, cache, pages.table, pages.len, out, ws, err=err)

        got = []
        if captured:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):              # loads the kernels
                x.copy_(xs[0])
                step()
            torch.cuda.synchronize()
            pages.table.fill_(-1)
            pages.len.zero_()
            pages.refs.zero_()
            k.zero_(), v.zero_()
            if ks is not None:
                ks.fill_(1), vs.fill_(1)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for i in range(steps):
            x.copy_(xs[i])
            graph.replay() if captured else step()
            got.append(out.clone())
        torch.cuda.synchronize()
        assert err.item() == 0 and pages.len.tolist() == (steps * add).tolist()
        return torch.stack(got), pages.table.clone(), k.view(torch.uint8).clone()

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
