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
