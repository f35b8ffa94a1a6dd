"""Attention over e4m3 rows whose scales differ much (lsa_paged_attn), against the 64-bit plain form.

Bound.  A row's weight p (2^x of its score below the running max) times its V scale s enters the product with V as one
f16 number.  Held relative to a head's largest product so far (of rows that are not all zeros) so that this comes to lie
at 2^9 or above, an f16 is off by half its step: 2^-11 of p s, or 2^-25 where it is no normal number, i.e. 2^-34 of the
largest product.  A code is at most 448.  So beside the bounds of test_gpu_paged.py (w of a weight, n 2^-22 of the sums,
half a step of bf16),
    |dout_d| <= (2 w + 2^-11 + n 2^-22) sum_t p_t |v_td| + n 448 2^-34 max_t p_t s_t + 2^-8 |o_d|
with p the softmax's weights.
"""
import numpy as np
import pytest
import torch

from gpu_cases import lsa_mod
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    return lsa_mod()


def _at(c, b, t):
    """Page and slot of entries t of sequence b."""
    t = np.atleast_1d(np.asarray(t))
    return c.table[b, t // c.page].astype(np.int64), (t % c.page).astype(np.int64)


def _dev(i):
    return torch.from_numpy(i).cuda()


def _set_values(c, b, t, scale=None, codes=None):
    """Gives entries t of sequence b other value scales (a factor) or codes ([D] for all heads), the 64-bit form too."""
    p, s = _at(c, b, t)
    pc, sc = _dev(p), _dev(s)
    if codes is not None:
        x = torch.as_tensor(codes, dtype=torch.float32).to(torch.float8_e4m3fn)
        rows = x.expand(len(p), *c.v.shape[2:]).contiguous()
        c.v.view(torch.uint8)[pc, sc] = rows.view(torch.uint8).cuda()
    if scale is not None:
        c.vs[pc, sc] = torch.as_tensor(scale, dtype=torch.float32, device="cuda").reshape(-1, 1).expand(len(p), c.vs.shape[2])
    c.v64[p, s] = c.v[pc, sc].cpu().float().numpy().astype(np.float64) * c.vs[pc, sc].cpu().numpy().astype(np.float64)[..., None]
    if c.latent:
        c.k64[p, s] = c.v64[p, s]


def _scale_of(c, b, t):
    p, s = _at(c, b, t)
    return c.vs[_dev(p), _dev(s)].cpu().numpy().astype(np.float64)


def _set_key(c, b, t, score):
    """The key of entry t becomes one whose score under every head of its group is about `score` (the group's queries are
    the same)."""
    p, s = _at(c, b, t)
    Hkv, D = c.k.shape[2:]
    q = c.q.float().reshape(c.q.shape[0], Hkv, -1, D)[b, :, 0]
    k = q * (score / c.scale / (q * q).sum(-1, keepdim=True))
    ks = k.abs().amax(-1) / 448
    ks[ks == 0] = 1.0                              # a score of 0: a key of zeros
    codes = (k / ks[..., None]).to(torch.float8_e4m3fn)
    c.k.view(torch.uint8)[_dev(p), _dev(s)] = codes.view(torch.uint8).cuda()[None]
    c.ks[_dev(p), _dev(s)] = ks.cuda()[None]
    c.k64[p, s] = codes.float().numpy().astype(np.float64) * ks.numpy().astype(np.float64)[..., None]


def _same_queries(c):
    """Every head of a group asks the same."""
    B, Hq, D = c.q.shape
    Hkv = c.k.shape[2]
    c.q = c.q.reshape(B, Hkv, -1, D)[:, :, :1].expand(B, Hkv, Hq // Hkv, D).reshape(B, Hq, D).contiguous()


def _check(lsa, c):
    out, _ = c.run(lsa)
    got = out.double().cpu().numpy()
    B, Hq, D = c.q.shape
    G = Hq // c.k.shape[2]
    assert np.isfinite(got).all()
    for b in range(B):
        n = c.lens[b]
        p, s = _at(c, b, np.arange(n))
        sc = _scale_of(c, b, np.arange(n))
        for j in range(Hq):
            K, V, q = c.k64[p, s, j // G], c.v64[p, s, j // G], c.q[b, j].double().numpy()
            a = c.scale * (K @ q)
            A = c.scale * np.max(np.abs(K) @ np.abs(q))
            e = np.exp(a - a.max())
            e /= e.sum()
            o = e @ V
            w = 2 * (D + 16) * 2.0 ** -23 * A + 2.0 ** -15
            some = (V != 0).any(-1)
            top = (e * np.abs(sc[:, j // G]) * some).max()
            tol = (2 * w + 2.0 ** -11 + n * 2.0 ** -22) * (e @ np.abs(V)) + n * 448 * 2.0 ** -34 * top + 2.0 ** -8 * np.abs(o)
            d = np.abs(got[b, j] - o)
            assert (d <= tol + 1e-37).all(), (b, j, np.max(d / (tol + 1e-37)), np.max(np.abs(o)))


HEADS = [(4, 4, 64, False), (12, 2, 128, False), (16, 1, 80, False), (8, 1, 256, False), (33, 1, 64, False),
         (40, 2, 128, False), (9, 1, 512, True)]


@pytest.mark.parametrize("Hq,Hkv,D,latent", HEADS)
@pytest.mark.parametrize("size", [1e-2, 1e-4, 1e-6, 1e-8])
def test_rows_of_zeros_at_scale_one_among_small_values(lsa, Hq, Hkv, D, latent, size):
    """What lsa_qk_norm_rope writes for a value of zeros: scale 1, beside rows of amax / 448."""
    c = Case("e4m3", Hq, Hkv, D, 16, [300, 1, 37, 5000], latent=latent, seed=D)
    r = np.random.default_rng(D)
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        zero = r.random(n) < 0.05
        zero[0] = n > 1
        _set_values(c, b, t, scale=size * _scale_of(c, b, t)[:, 0])
        _set_values(c, b, t[zero], scale=np.ones(int(zero.sum())), codes=np.zeros(D))
    _check(lsa, c)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 64), (12, 2, 128), (8, 1, 256)])
@pytest.mark.parametrize("octaves,score", [(20, -13.0), (40, -27.0), (40, -60.0), (90, -62.0), (30, 5.0)])
def test_an_entry_of_a_large_scale_and_little_weight(lsa, Hq, Hkv, D, octaves, score):
    """One row's scale is far above the others', and its weight as far below, at the sequence's front, middle and end."""
    c = Case("e4m3", Hq, Hkv, D, 16, [300, 300, 3000, 300], seed=D + octaves, q_scale=1.0)
    _same_queries(c)
    for b, t in enumerate((0, 150, 2999, 17)):
        _set_key(c, b, t, score)
        _set_values(c, b, t, scale=_scale_of(c, b, t)[:, 0] * 2.0 ** octaves)
    _check(lsa, c)


@pytest.mark.parametrize("Hq,Hkv,D,latent", HEADS[:-1])
@pytest.mark.parametrize("q_scale", [0.1, 2.0, 20.0])
def test_scales_of_any_size(lsa, Hq, Hkv, D, latent, q_scale):
    """Scales from 2^-60 to 2^40, in rising, falling and random order, rows of zeros among them."""
    c = Case("e4m3", Hq, Hkv, D, 16, [200, 200, 3000, 64], seed=D + 1, q_scale=q_scale)
    r = np.random.default_rng(D + 1)
    for b, n in enumerate(c.lens):
        e = r.uniform(-60, 40, n)
        e = np.sort(e) if b == 0 else -np.sort(-e) if b == 1 else e
        _set_values(c, b, np.arange(n), scale=2.0 ** e)
        t = np.flatnonzero(r.random(n) < 0.1)
        _set_values(c, b, t, codes=np.zeros(D))
    _check(lsa, c)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 64), (12, 2, 128)])
def test_one_scale_for_all_and_an_entry_of_small_codes_with_most_weight(lsa, Hq, Hkv, D):
    """Rows of another writer: one scale for all, and the entry that takes nearly all weight holds the smallest codes."""
    c = Case("e4m3", Hq, Hkv, D, 16, [300, 2000], seed=3, q_scale=1.0)
    _same_queries(c)
    for b, n in enumerate(c.lens):
        _set_values(c, b, np.arange(n), scale=np.full(n, 0.125))
        _set_key(c, b, n // 2, 16.0)
        _set_values(c, b, n // 2, codes=2.0 ** -9 * (1 - 2 * (np.arange(D) % 2)))
    _check(lsa, c)


def test_scores_that_rise_over_the_sequence_with_falling_scales(lsa):
    """The running max moves from step to step, and the products' reference with it."""
    c = Case("e4m3", 4, 4, 64, 16, [640, 333], seed=5, q_scale=1.0)
    for b, n in enumerate(c.lens):
        for t in range(0, n, 32):
            _set_key(c, b, t, 0.15 * t)
        _set_values(c, b, np.arange(n), scale=2.0 ** (20 - 0.2 * np.arange(n)))
    _check(lsa, c)


def test_nan_rows_and_infinite_scales_show(lsa):
    c = Case("e4m3", 4, 2, 64, 16, [100, 100, 100], seed=6)
    _set_values(c, 0, 50, codes=np.full(64, np.nan))
    _set_values(c, 1, 50, scale=np.array([np.inf]), codes=np.ones(64))
    out, lse = c.run(lsa)
    assert torch.isnan(out[0]).all() and torch.isfinite(lse).all() and torch.isfinite(out[2]).all()
    assert (out[1] == float("inf")).all()
