"""Calls of the paged-cache operators at the edges of what their descriptions allow."""
import numpy as np
import pytest
import torch

from gpu_cases import lsa_mod
from paged_ref import i32
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu

# type, query heads, kv heads, head dim, latent: one of each kernel
KERNELS = [("f32", 4, 2, 64, False), ("bf16", 4, 2, 64, False), ("e4m3", 4, 2, 64, False), ("bf16", 16, 1, 512, True)]


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    return lsa_mod()


@pytest.mark.parametrize("dtype,Hq,Hkv,D,latent", KERNELS)
@pytest.mark.parametrize("lens", [[37, 1, 0], [3000, 20, 0, 9000]])
def test_the_output_may_take_the_queries_place(lsa, dtype, Hq, Hkv, D, latent, lens):
    """Whole and split segments; a longer stride between queries, where rows would meet, is refused."""
    c = Case(dtype, Hq, Hkv, D, 16, lens, latent=latent, seed=20)
    want, _ = c.check(lsa)
    cache, table, n, B = c.cache(lsa), i32(c.table), i32(c.lens), len(lens)
    ws = torch.empty(lsa.paged_attn_workspace_size(cache, B, Hq), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        q = c.q.cuda()
        lsa.paged_attn(q, cache, table, n, q, ws, scale=c.scale)
        assert torch.equal(q, want)
    wide = torch.zeros((B, Hq + 1, D), dtype=q.dtype, device="cuda")
    with pytest.raises(lsa.LsaError, match="overlaps"):
        lsa.paged_attn(wide[:, :Hq], cache, table, n, wide.view(-1)[:B * Hq * D].view(B, Hq, D), ws, scale=c.scale)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,latent", KERNELS)
@pytest.mark.parametrize("page,width", [(16, 20), (64, 150)])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("over", [1, 1 << 20, (1 << 31) - 1])
def test_lengths_past_the_table_are_cut_and_reported(lsa, dtype, Hq, Hkv, D, latent, page, width, window, over):
    """Every page of the long row is good, so nothing but its length is reported: it is the row of a full table."""
    reach = page * width
    c = Case(dtype, Hq, Hkv, D, page, [40, reach, 7], latent=latent, seed=21, window=window)
    table = np.ascontiguousarray(c.table[:, :width])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, lse = c.check(lsa, table=table, err=err)
    assert err.item() == 0
    out, z = c.run(lsa, table=table, lens=[40, min(reach + over, (1 << 31) - 1), 7], err=err)
    assert err.item() == 3
    assert torch.equal(out, want) and torch.equal(z, lse)
    out, z = c.run(lsa, table=table, lens=[40, min(reach + over, (1 << 31) - 1), 7])      # no error word
    assert torch.equal(out, want) and torch.equal(z, lse)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,latent", KERNELS)
def test_the_length_of_any_sequence_of_a_long_batch_is_reported(lsa, dtype, Hq, Hkv, D, latent):
    B, page, width = 1100, 8, 2
    c = Case(dtype, Hq, Hkv, D, page, [(7 * b) % 17 for b in range(B)], latent=latent, seed=22)
    table = np.ascontiguousarray(np.where(c.table < 1 << 30, c.table, 0)[:, :width])      # every entry names a page
    want, _ = c.run(lsa, table=table, lens=[min(n, 16) for n in c.lens])
    for b in (0, 640, B - 1):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lens = list(c.lens)
        lens[b] = 17
        out, _ = c.run(lsa, table=table, lens=lens, err=err)
        assert err.item() == 3
        keep = torch.arange(B, device="cuda") != b
        assert torch.equal(out[keep].view(torch.uint8), want[keep].view(torch.uint8))


@pytest.mark.parametrize("kind,Hq,Hkv,D,latent", [("f32", 4, 1, 256, False), ("bf16", 8, 2, 256, False),
                                                 ("e4m3", 8, 2, 512, False), ("bf16", 16, 1, 512, True)])
def test_append_copy_and_attention_past_32_bits(lsa, kind, Hq, Hkv, D, latent):
    """The same calls over the last pages of a cache of 4.6 GB a tensor and over a small one: the same bits."""
    page, n = 64, 3 * 64 + 17
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kind]
    qt = torch.float32 if kind == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(23)
    x = torch.randn((n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(qt)
    freq, _ = lsa.rope_frequencies(64)
    rope = lsa.Rope(freq.cuda())
    at = i32(range(n))
    many = 4_600_000_000 // (page * Hkv * D * dt.itemsize)

    def run(n_pages, use, to):
        k = torch.zeros((n_pages, page, Hkv, D), dtype=dt, device="cuda")
        v = None if latent else torch.zeros_like(k)
        ks, vs = (torch.zeros((n_pages, page, Hkv), device="cuda") if kind == "e4m3" else None for _ in range(2))
        cache = lsa.PageCache(k, v, ks, vs)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = torch.empty((n, Hq, D), dtype=qt, device="cuda")
        lsa.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], None if latent else x[:, Hq + Hkv:], q_out=q, pos=at, rope=rope,
                         cache=cache, table=i32([use]), seq=i32([0] * n), at=at, err=err)
        lsa.page_copy(cache, i32(use), i32(to), err=err)
        ws = torch.empty(lsa.paged_attn_workspace_size(cache, 2, Hq), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty((2, Hq, D), dtype=qt, device="cuda"), torch.empty((2, Hq), device="cuda")
        lsa.paged_attn(q[-2:].contiguous(), cache, i32([use, to]), i32([n, n]), out, ws, lse=lse, err=err)
        assert err.item() == 0
        return out.clone(), lse.clone(), q

    a = run(many, [many - 1, 3, many - 2, many - 9], [many - 4, many - 5, 0, many - 7])
    b = run(9, [8, 3, 7, 1], [6, 5, 0, 2])
    assert a[0].isfinite().all() and a[0].abs().amax(-1).min() > 0
    for s, t in zip(a, b):
        assert torch.equal(s, t)
