"""Calls of lsa_paged_attn at the edges of what its description allows."""
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
