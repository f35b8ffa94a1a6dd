"""Calls of the paged-cache operators whose operands share memory are refused on the host (no CUDA call is reached)."""
import pytest

from test_paged_cpu import BIG, _cache, _qk


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
