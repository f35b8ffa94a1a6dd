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


@pytest.mark.parametrize("inverse", [False, True])
def test_the_angle_is_not_rounded_to_fp32(lsa, inverse):
    """Angles next to half a turn, where the sine is small and shows the angle's own error.  An odd position times
    freq = pi (1 - u) is a turn's half less pos u pi, |sin| < 2^-5: off by a unit of sincospi and half a step of its
    correction by what the angle's rounding left, 1.5 * 2^-29 (and 2^-45 of the fp64 angle): 2^-28 bounds it.  Half turns
    rounded to fp32 alone are off by up to 2^-25, the sine by up to pi 2^-25, eleven times the bound."""
    T, half = 257, 64
    r = np.random.default_rng(0)
    pos = 2 * r.integers(0, 40, T) + 1
    u = r.uniform(0, 2.0 ** -5 / 4 / 81, half)
    freq = np.pi * (1 - u)
    x = torch.zeros((T, 1, 2 * half), device="cuda")
    x[:, :, :half] = 1                                    # (1, 0) turns to (cos, sin)
    out = torch.empty_like(x)
    lsa.qk_norm_rope(x, q_out=out, pos=i32(pos), rope=lsa.Rope(torch.from_numpy(freq).cuda(), inverse=inverse))
    got = out[:, 0, half:].double().cpu().numpy()
    phi = pos[:, None] * freq * (-1.0 if inverse else 1.0)
    want = np.sin(phi)
    assert np.abs(want).max() < 2.0 ** -5
    assert np.abs(got - want).max() <= 2.0 ** -28
    assert np.abs(out[:, 0, :half].double().cpu().numpy() - np.cos(phi)).max() <= 1.5 * 2.0 ** -23
    # what the test is for: the same with the half turns rounded to fp32 fails by far
    h = 2 * (phi / (2 * np.pi) - np.rint(phi / (2 * np.pi)))
    assert np.abs(np.sin(np.pi * h.astype(np.float32).astype(np.float64)) - want).max() > 5 * 2.0 ** -28
