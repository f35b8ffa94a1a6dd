"""Calls of the paged-cache operators that are refused on the host (no CUDA call is reached): operands that share memory,
numbers that a C type would cut."""
import ctypes

import pytest
import torch

from test_paged_cpu import BIG, _books, _cache, _qk


@pytest.fixture(scope="module")
def lsa():
    from lookahead_sparse_kv_index_b200 import build

    build.build()
    from lookahead_sparse_kv_index_b200 import lsa as mod

    return mod


def test_norm_rope_rejects_outputs_over_what_else_it_reads_or_writes(lsa):
    """Weights, positions, frequencies, the table, the error word, the cache's rows and scales: bytes that meet an output."""
    c = _cache(lsa, dtype=lsa.E4M3, k=10 * BIG, v=11 * BIG, k_scale=12 * BIG, v_scale=13 * BIG)
    span = 9 * c.page_stride + 15 * c.slot_stride + c.head_stride + 64           # bytes of the cache's keys
    rope = lsa.RopeDesc(14 * BIG, 64, 0, 0, 1.0)
    last = 4 * 4 * 64 * 2                                                         # q_out's last token
    apart = dict(pos=15 * BIG, table=16 * BIG, seq=17 * BIG, at=18 * BIG, wq=19 * BIG, wk=20 * BIG)
    for kw in (dict(qo=10 * BIG), dict(qo=10 * BIG + span - 16), dict(qo=11 * BIG - last), dict(ko=12 * BIG),
               dict(ko=13 * BIG + 16), dict(qo=14 * BIG), dict(qo=15 * BIG), dict(ko=16 * BIG), dict(ko=17 * BIG),
               dict(ko=18 * BIG), dict(qo=19 * BIG), dict(qo=20 * BIG + 112), dict(wq=2 * BIG + last + 256),
               dict(at=4 * BIG)):
        assert _qk(lsa, cache=c, rope=rope, **{**apart, **kw}) == 1, kw
        assert b"overlaps" in lsa.lib.lsa_last_error(), kw
    a = dict(q=BIG, qo=2 * BIG, T=5)
    assert lsa.lib.lsa_qk_norm_rope(a["q"], 256, a["qo"], 256, None, 0, None, 0, None, 0, lsa.BF16, 5, 4, 0, 64, None, None,
                                    1e-6, None, None, None, None, 0, 0, 0, None, None, 2 * BIG + 4 * 256, None) == 1
    assert b"overlaps err" in lsa.lib.lsa_last_error()


def test_attention_rejects_outputs_over_its_operands(lsa):
    """out may be Q itself; any other shared byte of out, lse, the workspace and the error word is refused."""
    c = _cache(lsa, dtype=lsa.E4M3, k=30 * BIG, v=31 * BIG, k_scale=32 * BIG, v_scale=33 * BIG)
    span = 9 * c.page_stride + 15 * c.slot_stride + c.head_stride + 64           # bytes of the cache's keys
    need = lsa.lib.lsa_paged_attn_workspace_size(ctypes.byref(c), 3, 4)
    row, out_bytes = 4 * 64 * 2, 3 * 4 * 64 * 2
    assert 0 < need < 16 * BIG
    a = dict(Q=BIG, table=2 * BIG, sl=3 * BIG, out=4 * BIG, lse=5 * BIG, ws=8 * BIG, wsb=need, err=7 * BIG)

    def call(**kw):
        x = {**a, "qs": 4 * 64, **kw}
        return lsa.lib.lsa_paged_attn(x["Q"], lsa.BF16, x["qs"], ctypes.byref(c), x["table"], 8, 8, x["sl"], 3, 4, 0, 1.0,
                                      x["out"], x["lse"], x["ws"], x["wsb"], x["err"], None)

    for kw in (dict(out=BIG + 16), dict(out=BIG - out_bytes + 16), dict(out=BIG, qs=5 * 64), dict(out=2 * BIG),
               dict(out=2 * BIG + 3 * 8 * 4 - 16), dict(out=3 * BIG), dict(out=30 * BIG), dict(out=31 * BIG + span - 16),
               dict(out=32 * BIG), dict(out=33 * BIG), dict(lse=4 * BIG + out_bytes - 4), dict(lse=BIG + row), dict(lse=3 * BIG),
               dict(ws=BIG), dict(ws=4 * BIG), dict(ws=BIG - need + 16), dict(ws=5 * BIG), dict(out=8 * BIG + need // 32 * 16),
               dict(ws=2 * BIG), dict(ws=33 * BIG), dict(err=4 * BIG), dict(err=8 * BIG + need - 4), dict(err=3 * BIG + 8)):
        assert call(**kw) == 1, kw
        assert b"overlaps" in lsa.lib.lsa_last_error(), kw


def test_page_calls_reject_lists_over_each_other_and_the_books(lsa):
    """What a call writes may not be what it reads elsewhere; packing in place means the whole table, the whole counts."""
    L = lsa.lib
    b = _books(lsa, table=BIG, len=2 * BIG, refs=3 * BIG)                        # 4 rows of 8 pages, 100 pages
    refused = lambda status: status == 1 and b"overlaps" in L.lsa_last_error()   # noqa: E731
    fork = dict(src=4 * BIG, dst=5 * BIG, cs=6 * BIG, cd=7 * BIG)
    for kw in (dict(cs=4 * BIG), dict(cs=5 * BIG + 4), dict(cd=4 * BIG + 4), dict(cd=6 * BIG), dict(cs=BIG + 124),
               dict(cd=2 * BIG), dict(cs=3 * BIG + 396), dict(src=BIG), dict(dst=2 * BIG + 8), dict(src=3 * BIG)):
        x = {**fork, **kw}
        assert refused(L.lsa_page_fork(b, x["src"], x["dst"], 2, x["cs"], x["cd"], None, None)), kw
    for rows in (BIG, 2 * BIG + 12, 3 * BIG + 200):
        assert refused(L.lsa_page_free(b, rows, 3, None, None)), rows
    size = lsa.page_compact_workspace_size(100)
    pack = dict(t=4 * BIG, r=5 * BIG, ms=6 * BIG, md=7 * BIG, n=8 * BIG, ws=9 * BIG)
    for kw in (dict(t=BIG + 4), dict(r=3 * BIG + 4), dict(r=BIG), dict(t=3 * BIG), dict(t=2 * BIG), dict(ms=BIG), dict(md=3 * BIG),
               dict(ms=2 * BIG), dict(md=6 * BIG + 396), dict(n=6 * BIG), dict(n=2 * BIG), dict(ws=3 * BIG), dict(ws=BIG),
               dict(ws=4 * BIG), dict(ms=9 * BIG + size - 4), dict(r=4 * BIG + 64)):
        x = {**pack, **kw}
        assert refused(L.lsa_page_compact(b, x["t"], x["r"], x["ms"], x["md"], x["n"], x["ws"], size, None)), kw


def test_bindings_refuse_numbers_that_their_types_would_cut(lsa):
    """ctypes takes an int32 modulo 2^32: a window of 2^32 + 5 would be one of 5."""
    cache = lsa.PageCache(torch.zeros((4, 8, 2, 32)))
    q, i = torch.zeros((3, 4, 32)), torch.zeros(3, dtype=torch.int32)
    table, ws = torch.zeros((3, 5), dtype=torch.int32), torch.zeros(1 << 10)
    for window in (1 << 31, (1 << 32) + 5, -(1 << 32)):
        with pytest.raises(ValueError, match="window"):
            lsa.paged_attn(q, cache, table, i, q.clone(), ws, window=window)
    for size in (1 << 31, (1 << 32) + 16):
        with pytest.raises(ValueError, match="page_size"):
            lsa.PageTable(table, i, i, size)
    with pytest.raises(ValueError, match="rot_dim"):
        lsa.rope_frequencies((1 << 32) + 64)
    with pytest.raises(ValueError, match="B="):
        lsa.paged_attn_workspace_size(cache, (1 << 32) + 1, 4)
    with pytest.raises(ValueError, match="Hq="):
        lsa.paged_attn_workspace_size(cache, 1, (1 << 32) + 4)
