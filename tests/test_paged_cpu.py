"""The paged-cache operators without a GPU: refused arguments (no CUDA call is reached), the bindings' checks, the
struct mirrors, the host-side frequencies, and the model of the pages' books that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_ref as ref

BIG = 1 << 20


@pytest.fixture(scope="module")
def lsa():
    from lookahead_sparse_kv_index_b200 import build

    build.build()
    from lookahead_sparse_kv_index_b200 import lsa as mod

    return mod


def _cache(lsa, **kw):
    a = dict(k=BIG, v=2 * BIG, k_scale=None, v_scale=None, dtype=lsa.BF16, page_size=16, Hkv=2, D=64, n_pages=10,
             page_stride=16 * 2 * 64, slot_stride=2 * 64, head_stride=64)
    a.update(kw)
    return lsa.PageCacheDesc(*[a[n] for n, _ in lsa.PageCacheDesc._fields_])


CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(dtype=7), 1), (dict(page_size=0), 1), (dict(Hkv=0), 1),
          (dict(n_pages=0), 1), (dict(D=40), 5), (dict(D=528), 5), (dict(dtype=2), 1), (dict(k_scale=BIG), 1),
          (dict(k=BIG + 8), 1), (dict(page_stride=16 * 2 * 64 + 4), 1), (dict(slot_stride=32), 1),
          (dict(head_stride=-64), 1), (dict(n_pages=1 << 27), 1), (dict(page_stride=1 << 60), 1),
          (dict(v=BIG, dtype=2, k_scale=BIG, v_scale=2 * BIG), 1)]


def _attn(lsa, cache=None, no_cache=False, **kw):
    a = dict(Q=BIG, qt=lsa.BF16, qs=4 * 64, table=BIG, ts=8, mp=8, sl=BIG, B=3, Hq=4, window=0, scale=1.0, out=BIG,
             lse=None, ws=BIG, wsb=1 << 30)
    a.update(kw)
    c = _cache(lsa) if cache is None else cache
    return lsa.lib.lsa_paged_attn(a["Q"], a["qt"], a["qs"], None if no_cache else ctypes.byref(c), a["table"], a["ts"],
                                  a["mp"], a["sl"], a["B"], a["Hq"], a["window"], a["scale"], a["out"], a["lse"],
                                  a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,status", CACHES)
def test_bad_caches_are_refused_everywhere(lsa, kw, status):
    c = _cache(lsa, **kw)
    assert _attn(lsa, c) == status
    assert lsa.lib.lsa_last_error() != b""
    assert lsa.lib.lsa_page_copy(ctypes.byref(c), BIG, BIG, 3, None, None, None) == status
    assert lsa.lib.lsa_paged_attn_workspace_size(ctypes.byref(c), 3, 4) == 0
    assert _qk(lsa, cache=c) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), 1), (dict(table=None), 1), (dict(sl=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(no_cache=True), 1), (dict(B=0), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(qt=0), 5), (dict(qt=9), 1),
    (dict(qs=4 * 64 - 8), 1), (dict(qs=4 * 64 + 4), 1), (dict(Q=BIG + 8), 1), (dict(out=BIG + 2), 1), (dict(mp=0), 1),
    (dict(ts=7), 1), (dict(mp=1 << 27, ts=1 << 27), 1), (dict(window=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(wsb=16), 1), (dict(ws=BIG + 4), 1),
])
def test_attention_rejects_bad_arguments(lsa, kw, status):
    assert _attn(lsa, **kw) == status
    assert lsa.lib.lsa_last_error() != b""


def test_attention_rejects_reaches_past_int32_steps(lsa):
    """Places of entries are int32 and step past the end: 2^30 entries a row are the limit."""
    size = _cache(lsa).page_size
    most = (1 << 30) // size
    assert _attn(lsa, mp=most + 1, ts=most + 1) == 1 and b"2^30" in lsa.lib.lsa_last_error()
    assert _attn(lsa, mp=most, ts=most, scale=0.0) == 1 and b"scale" in lsa.lib.lsa_last_error()


def test_attention_workspace_does_not_depend_on_lengths(lsa):
    c = _cache(lsa)
    size = lsa.lib.lsa_paged_attn_workspace_size(ctypes.byref(c), 1, 4)
    assert size > 0 and size == lsa.lib.lsa_paged_attn_workspace_size(ctypes.byref(c), 200, 4)
    assert lsa.lib.lsa_paged_attn_workspace_size(ctypes.byref(c), 0, 4) == 0
    assert lsa.lib.lsa_paged_attn_workspace_size(None, 1, 4) == 0


def _qk(lsa, cache=None, rope=None, **kw):
    a = dict(q=BIG, qs=4 * 64, qo=2 * BIG, qos=4 * 64, k=3 * BIG, ks=2 * 64, ko=4 * BIG, kos=2 * 64, v=None, vs=2 * 64,
             dt=lsa.BF16, T=5, Hq=4, Hkv=2, D=64, wq=None, wk=None, eps=1e-6, pos=BIG, table=None, ts=8, rows=3, mp=8,
             seq=None, at=None)
    if cache is not None:
        a.update(v=5 * BIG, table=BIG, at=BIG)
        if cache.v == cache.k:
            a["v"] = None
    a.update(kw)
    return lsa.lib.lsa_qk_norm_rope(a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"], a["v"],
                                    a["vs"], a["dt"], a["T"], a["Hq"], a["Hkv"], a["D"], a["wq"], a["wk"], a["eps"],
                                    a["pos"], None if rope is None else ctypes.byref(rope),
                                    None if cache is None else ctypes.byref(cache), a["table"], a["ts"], a["rows"],
                                    a["mp"], a["seq"], a["at"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(dt=2), 5), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1),
    (dict(D=72), 5), (dict(D=528, qs=9999 * 8, qos=9999 * 8, ks=9999 * 8, kos=9999 * 8), 5), (dict(qs=8), 1),
    (dict(ks=2 * 64 + 4), 1), (dict(q=BIG + 4), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(v=BIG), 1),
    (dict(wq=BIG + 4), 1), (dict(wk=BIG + 2), 1), (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1),
    (dict(q=2 * BIG, qs=8 * 64), 1), (dict(k=4 * BIG, ks=8 * 64), 1),
])
def test_norm_rope_rejects_bad_arguments(lsa, kw, status):
    assert _qk(lsa, **kw) == status
    assert lsa.lib.lsa_last_error() != b""


def test_norm_rope_rejects_outputs_over_other_inputs(lsa):
    """An output may be its own input; over any other operand, rows would be written before they are read."""
    c, row = _cache(lsa), 2 * 64 * 2                                       # bytes of a token's keys
    for kw in (dict(qo=3 * BIG), dict(ko=BIG), dict(qo=4 * BIG), dict(ko=5 * BIG),      # k, q, k_out, v
               dict(qo=BIG + 16), dict(ko=3 * BIG + row), dict(ko=3 * BIG - row + 16),  # a shifted input of its own
               dict(k=4 * BIG, v=4 * BIG), dict(q=2 * BIG + 4 * 64 * 2)):
        assert _qk(lsa, cache=c, **kw) == 1, kw
        assert b"overlaps" in lsa.lib.lsa_last_error(), kw
    # parts of one projection's rows [q | k | v], in place, pass this check (and fail the next)
    one = dict(q=BIG, qo=BIG, k=BIG + 4 * 64 * 2, ko=BIG + 4 * 64 * 2, v=BIG + 6 * 64 * 2, qs=512, qos=512, ks=512,
               kos=512, vs=512)
    assert _qk(lsa, cache=c, **one, eps=-1.0) == 1 and b"eps" in lsa.lib.lsa_last_error()
    assert _qk(lsa, cache=c, **{**one, "ko": BIG + 5 * 64 * 2}) == 1 and b"overlaps" in lsa.lib.lsa_last_error()


def test_norm_rope_rejects_bad_rotations_and_caches(lsa):
    R = lsa.RopeDesc
    assert _qk(lsa, rope=R(BIG, 63, 0, 0, 1.0)) == 1                       # odd
    assert _qk(lsa, rope=R(BIG, 66, 0, 0, 1.0)) == 1                       # more than D
    assert _qk(lsa, rope=R(BIG, -2, 0, 0, 1.0)) == 1
    assert _qk(lsa, rope=R(None, 64, 0, 0, 1.0)) == 1                      # no frequencies
    assert _qk(lsa, rope=R(BIG, 64, 0, 0, -1.0)) == 1
    assert _qk(lsa, rope=R(BIG, 64, 0, 0, 1.0), pos=None) == 1
    c = _cache(lsa)
    for kw in (dict(v=None), dict(table=None), dict(at=None), dict(rows=0), dict(mp=0), dict(ts=7),
               dict(Hkv=1, ks=64, vs=64), dict(mp=1 << 28, ts=1 << 28), dict(vs=64)):
        assert _qk(lsa, cache=c, **kw) == 1, kw
    assert _qk(lsa, cache=c, dt=lsa.F32) == 5                              # bf16 rows of fp32 heads
    latent = _cache(lsa, v=BIG)
    assert _qk(lsa, cache=latent, v=BIG) == 1                              # values of a latent cache
    assert _qk(lsa, T=0) == 0                                              # nothing to do


def _books(lsa, **kw):
    a = dict(table=BIG, len=BIG, refs=BIG, n_rows=4, max_pages=8, page_size=16, n_pages=100)
    a.update(kw)
    return ctypes.byref(lsa.PageTableDesc(*[a[n] for n, _ in lsa.PageTableDesc._fields_]))


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), 1), (dict(len=None), 1), (dict(refs=None), 1), (dict(n_rows=0), 1), (dict(max_pages=0), 1),
    (dict(page_size=0), 1), (dict(n_pages=0), 1), (dict(n_rows=65537), 5), (dict(n_pages=(1 << 24) + 1), 5),
    (dict(max_pages=1 << 20, page_size=1 << 11), 1),
])
def test_bad_books_are_refused_everywhere(lsa, kw, status):
    L, b = lsa.lib, _books(lsa, **kw)
    assert L.lsa_page_grow(b, BIG, None, None) == status
    assert L.lsa_page_fork(b, BIG, BIG, 2, BIG, BIG, None, None) == status
    assert L.lsa_page_free(b, BIG, 2, None, None) == status
    assert L.lsa_page_compact(b, BIG, BIG, BIG, BIG, BIG, BIG, 1 << 30, None) == status


def test_page_calls_reject_bad_arguments(lsa):
    L, b, c = lsa.lib, _books(lsa), ctypes.byref(_cache(lsa))
    assert L.lsa_page_grow(None, BIG, None, None) == 1
    assert L.lsa_page_grow(b, None, None, None) == 1
    assert L.lsa_page_fork(b, BIG, BIG, -1, BIG, BIG, None, None) == 1
    assert L.lsa_page_fork(b, BIG, BIG, 5, BIG, BIG, None, None) == 1      # more forks than rows
    assert L.lsa_page_fork(b, None, BIG, 2, BIG, BIG, None, None) == 1
    assert L.lsa_page_fork(b, BIG, BIG, 2, None, BIG, None, None) == 1
    assert L.lsa_page_fork(b, None, None, 0, None, None, None, None) == 0
    assert L.lsa_page_free(b, BIG, -1, None, None) == 1
    assert L.lsa_page_free(b, None, 1, None, None) == 1
    assert L.lsa_page_free(b, None, 0, None, None) == 0
    for i in range(6):
        args = [BIG] * 6
        args[i] = None
        assert L.lsa_page_compact(b, *args, 1 << 30, None) == 1, i
    assert L.lsa_page_compact(b, *[BIG] * 6, 16, None) == 1                # workspace
    assert L.lsa_page_compact(b, *[BIG] * 5, BIG + 8, 1 << 30, None) == 1
    assert lsa.page_compact_workspace_size(0) == 0 and lsa.page_compact_workspace_size((1 << 24) + 1) == 0
    assert lsa.page_compact_workspace_size(1) >= 8
    assert L.lsa_page_copy(None, BIG, BIG, 3, None, None, None) == 1
    assert L.lsa_page_copy(c, BIG, BIG, -1, None, None, None) == 1
    assert L.lsa_page_copy(c, None, BIG, 1, None, None, None) == 1
    assert L.lsa_page_copy(c, None, None, 0, None, None, None) == 0


def test_struct_mirrors(lsa):
    for which, s in ((10, lsa.PageCacheDesc), (11, lsa.RopeDesc), (12, lsa.PageTableDesc)):
        assert lsa.lib.lsa_struct_size(which) == ctypes.sizeof(s)


def test_bindings_check_their_tensors(lsa):
    k = torch.zeros((4, 8, 2, 32))
    for bad in (k[0], k.half(), k.transpose(2, 3)):
        with pytest.raises(ValueError):
            lsa.PageCache(bad)
    with pytest.raises(ValueError):
        lsa.PageCache(k, torch.zeros((4, 8, 2, 16)))
    with pytest.raises(ValueError):
        lsa.PageCache(k, k.transpose(1, 2).contiguous().transpose(1, 2))   # other strides
    with pytest.raises(ValueError):
        lsa.PageCache(k, k.clone(), torch.zeros((4, 8, 3)))
    cache = lsa.PageCache(k, k.clone())
    q, i = torch.zeros((3, 4, 32)), torch.zeros(3, dtype=torch.int32)
    table, ws = torch.zeros((3, 5), dtype=torch.int32), torch.zeros(1 << 20)
    calls = [dict(Q=q[:, :, :16]), dict(Q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(out=q.double()),
             dict(out=torch.zeros((2, 4, 32))), dict(seq_len=i[:2]), dict(seq_len=i.long()), dict(table=table[:2]),
             dict(table=table.long()), dict(table=table.t()[:3]), dict(lse=torch.zeros((3, 3))),
             dict(err=torch.zeros(2, dtype=torch.int32)), {}]              # the last: tensors on the CPU
    for kw in calls:
        a = dict(Q=q, out=q.clone(), seq_len=i, table=table, lse=None, err=None)
        a.update(kw)
        with pytest.raises(ValueError):
            lsa.paged_attn(a["Q"], cache, a["table"], a["seq_len"], a["out"], ws, lse=a["lse"], err=a["err"])
    with pytest.raises(ValueError):
        lsa.qk_norm_rope(q, q_out=q, pos=i[:1], rope=lsa.Rope(torch.zeros(16, dtype=torch.float64)))
    with pytest.raises(ValueError):
        lsa.qk_norm_rope(q, q, q, q_out=q, cache=lsa.PageCache(torch.zeros((4, 8, 4, 32))))     # no table
    with pytest.raises(ValueError):
        lsa.Rope(torch.zeros(16))
    with pytest.raises(ValueError):
        lsa.PageTable(table, i[:2], i, 8)


def test_rope_frequencies(lsa):
    f, m = lsa.rope_frequencies(64, 10000.0)
    want = 10000.0 ** (-np.arange(32) / 32.0)
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-14)
    assert m == 1.0
    f, m = lsa.rope_frequencies(64, 10000.0, "linear", 8.0)
    np.testing.assert_allclose(f.numpy(), want / 8, rtol=1e-14)
    f, m = lsa.rope_frequencies(64, 10000.0, "ntk", 8.0)
    assert f[0] == 1.0 and m == 1.0
    np.testing.assert_allclose(f[-1], want[-1] / 8, rtol=1e-12)            # the lowest is squeezed by the factor
    f, m = lsa.rope_frequencies(64, 10000.0, "yarn", 8.0, 4096, 32.0, 1.0)
    assert abs(m - (0.1 * math.log(8.0) + 1)) < 1e-6
    turns = 4096 * want / (2 * math.pi)
    g = (want - f.numpy()) / (want - want / 8)                             # 0 keeps, 1 squeezes
    assert (np.diff(g) >= -1e-12).all()
    assert np.abs(g[turns > 40]).max() < 1e-12 and np.abs(g[turns < 0.7] - 1).max() < 1e-12
    f1, m1 = lsa.rope_frequencies(64, 10000.0, "yarn", 1.0, 4096)
    np.testing.assert_allclose(f1.numpy(), want, rtol=1e-14)
    assert m1 == 1.0
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(base=1.0), dict(kind="linear", factor=0.5),
                dict(kind="ntk", rot_dim=2, factor=2.0), dict(kind="yarn", factor=2.0),
                dict(kind="yarn", factor=2.0, orig_len=10, beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(lsa.LsaError):
            lsa.rope_frequencies(**{"rot_dim": 64, **bad})
    with pytest.raises(ValueError):
        lsa.rope_frequencies(64, kind="other")


def test_the_books_model_itself():
    """A hand-worked run: 2 entries a page, 6 pages, 3 rows of up to 4."""
    b = ref.Books(3, 4, 6, 2)
    assert b.grow([3, 0, 2]) is None and b.rows == [[0, 1], [], [2]] and b.refs == [1, 1, 1, 0, 0, 0]
    assert b.fork([0], [1]) == (None, [1], [3]) and b.rows[1] == [0, 3] and b.refs == [2, 1, 1, 1, 0, 0]
    assert b.free([0, 0]) is None and b.refs == [1, 0, 1, 1, 0, 0] and b.len == [0, 3, 2]
    assert b.compact() == ([3] + [-1] * 5, [1] + [-1] * 5, 1) and b.rows == [[], [0, 1], [2]]
    assert b.refs == [1, 1, 1, 0, 0, 0]
    assert b.grow([9, 0, 0]) == "capacity" and b.grow([0, 0, 7]) == "capacity"
    assert b.fork([1], [2])[0] == "invalid"


def test_the_attention_form_itself():
    """One entry returns its value; equal keys the mean; the window and the table's holes leave entries out."""
    k = np.zeros((3, 2, 1, 16))
    v = np.arange(6, dtype=np.float64).reshape(3, 2, 1, 1) * np.ones(16)
    q = np.ones((1, 2, 16))
    table = np.array([[2, 0, 1]], np.int32)
    run = lambda n, w=0, t=table: ref.attention(q, k, v, t, [n], 2, w, 0.5)  # noqa: E731
    assert (run(1)[0] == 4).all() and (run(2)[0] == 4.5).all() and (run(3)[0] == 3.0).all()
    assert np.allclose(run(3)[1], math.log(3))
    assert (run(3, 1)[0] == 0).all() and (run(3, 2)[0] == 2.5).all()
    assert (run(3, 0, np.array([[-1, 0, 1]], np.int32))[0] == 0).all()
    assert (run(0)[1] == -np.inf).all()
