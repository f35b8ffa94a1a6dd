"""Roundings of norm, rotation and append (lsa_qk_norm_rope) that the bounds of test_gpu_paged.py are too wide to see."""
import numpy as np
import pytest
import torch

from gpu_cases import lsa_mod
from paged_ref import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    return lsa_mod()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Hkv,D,rot,interleaved", [(300, 4, 128, 128, False), (77, 1, 512, 64, True), (9, 2, 16, 6, False),
                                                     (50, 3, 80, 20, False), (40, 2, 96, 62, False)])
def test_e4m3_codes_are_the_rounded_quotients(lsa, dtype, T, Hkv, D, rot, interleaved):
    """Values are appended as they are: scale = max|v| / 448 and code = v / scale, each rounded once, to the bit (fp32
    division, then the conversion, on the CPU).  Keys without norm and rotation too."""
    g = torch.Generator().manual_seed(D)
    q = torch.zeros((T, 1, D), dtype=dtype, device="cuda")
    k, v = ((torch.randn((T, Hkv, D), generator=g) * 10.0 ** torch.randint(-6, 6, (T, Hkv, 1), generator=g)).to(dtype)
            for _ in range(2))
    v[0] = 0
    if dtype == torch.float32:
        v[1] = 1e-38 * torch.rand((Hkv, D), generator=g)       # max|v| / 448 is below the normal numbers
    kc, vc = (torch.zeros((T, 1, Hkv, D), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros((T, 1, Hkv), device="cuda") for _ in range(2))
    order = torch.randperm(T, generator=g)
    freq, _ = lsa.rope_frequencies(rot)
    for rope, pos in ((None, None), (lsa.Rope(freq.cuda(), interleaved), i32([0] * T))):     # angle 0: the same
        for x in (kc, vc, ks, vs):
            x.zero_()
        lsa.qk_norm_rope(q, k.cuda(), v.cuda(), q_out=torch.empty_like(q), pos=pos, rope=rope,
                         cache=lsa.PageCache(kc, vc, ks, vs), table=i32(order[:, None]), at=i32([0] * T))
        for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
            x = x.float()
            top = x.abs().amax(-1)
            s = torch.where(top > 0, torch.clamp(top / 448.0, min=float(np.finfo(np.float32).tiny)), 1.0)
            want = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(scales[order, 0].cpu(), s)
            a, b = codes[order, 0].cpu().view(torch.uint8), want.view(torch.uint8)
            zero = ((a | b) & 0x7F) == 0                      # (a rotation by 0 may turn -0 into 0)
            assert ((a == b) | zero).all(), f"{int(((a != b) & ~zero).sum())} of {a.numel()} codes differ"
