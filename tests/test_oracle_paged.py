"""Pins of the paged cache's oracle (CPU): hand-worked steps, closed forms and the dense
attention of the other oracle."""
import numpy as np
import pytest

import oracle


def test_map_hand_worked():
    # pages of 4; row 0 holds 3 and gets 2, row 1 is free and gets 5, row 2 (6 tokens) ends, row 3 stays free
    table = np.array([[9, -1, -1], [-1, -1, -1], [4, 7, -1], [-1, -1, -1]], np.int32)
    ring = np.array([1, 2, 3, 5, 6, 8, 0, 0, 0, 0], np.int32)
    r = oracle.page_map([3, -1, 6, -1], [2, 5, -1, 0], table, ring, [0, 6], 4, 9)
    assert r["kv_len"].tolist() == [5, 5, -1, -1]
    assert r["table"].tolist() == [[9, 1, -1], [2, 3, -1], [4, 7, -1], [-1, -1, -1]]
    assert r["ring_pos"].tolist() == [3, 8] and r["ring"].tolist() == [1, 2, 3, 5, 6, 8, 4, 7, 0, 0]
    assert r["slot"].tolist() == [39, 4, 8, 9, 10, 11, 12, -1, -1]
    assert r["row"].tolist() == [0, 0, 1, 1, 1, 1, 1, -1, -1]
    assert r["pos"].tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert r["cu"].tolist() == [0, 2, 7, 7, 7]


@pytest.mark.parametrize("kv, new, pos, cap, code", [
    ([3], [2], [0, 0], 4, 4),    # a page is needed, none is free
    ([3], [6], [0, 6], 4, 4),    # more tokens than slots
    ([3], [10], [0, 6], 99, 4),  # more tokens than the table row holds
    ([13], [0], [0, 6], 4, 3),   # a length above the table row
    ([-2], [0], [0, 6], 4, 3),
    ([0], [-2], [0, 6], 4, 3),
    ([0], [1], [5, 4], 4, 3),    # ring positions the wrong way round
    ([0], [1], [0, 9], 4, 3),    # more free pages than the ring holds
    ([4], [-1], [0, 8], 4, 3),   # a page comes back to a full ring
])
def test_map_refusals(kv, new, pos, cap, code):
    with pytest.raises(oracle.paged.Refused) as e:
        oracle.page_map(kv, new, np.zeros((1, 3), np.int32), np.arange(8, dtype=np.int32), pos, 4, cap)
    assert e.value.code == code


def test_attn_equals_dense_attention_over_the_gathered_rows():
    g = np.random.default_rng(1)
    N, P, Hkv, H, d = 9, 4, 2, 6, 8
    k, v, q = g.normal(size=(N, P, Hkv, d)), g.normal(size=(N, P, Hkv, d)), g.normal(size=(2, H, d))
    table = np.array([[3, 0, 8], [5, 1, 2]], np.int32)
    o, lse, _ = oracle.page_attn(q, k, v, table, [10, 5], 0.3)
    for r, n in enumerate((10, 5)):
        kk = np.concatenate([k[p] for p in table[r]])[:n]
        vv = np.concatenate([v[p] for p in table[r]])[:n]
        for h in range(H):
            ro, rl = oracle.attend(q[r, h][None], kk[:, h // 3], vv[:, h // 3], 0.3)
            np.testing.assert_allclose(o[r, h], ro[0], rtol=1e-12)
            np.testing.assert_allclose(lse[r, h], rl[0], rtol=1e-12)


def test_attn_windows_selection_and_empty_rows():
    g = np.random.default_rng(2)
    k, v, q = g.normal(size=(5, 4, 1, 8)), g.normal(size=(5, 4, 1, 8)), g.normal(size=(1, 1, 8))
    table = np.array([[0, 1, 2, 3, 4]], np.int32)
    full = oracle.page_attn(q, k, v, table, [18], 0.5)
    for kw in ({"sink": 18, "window": 1}, {"sink": 0, "window": 18}, {"sink": 9, "window": 9},
               {"sel": np.array([[[0, 1, 2, 3, 4, -1]]])}):
        np.testing.assert_allclose(oracle.page_attn(q, k, v, table, [18], 0.5, **kw)[0], full[0], rtol=1e-12)
    # sink 4 + window 6 of 18 tokens = pages 0, 3 and 4
    a = oracle.page_attn(q, k, v, table, [18], 0.5, sink=4, window=6)
    b = oracle.page_attn(q, k, v, table, [18], 0.5, sel=np.array([[[0, 3, 4]]]))
    np.testing.assert_allclose(a[0], b[0], rtol=1e-12)
    o, lse, _ = oracle.page_attn(q, k, v, table, [0], 0.5)
    assert (o == 0).all() and lse[0, 0] == -np.inf
    assert np.isnan(oracle.page_attn(q, k, v, table, [-1], 0.5)[0]).all()


def test_select_by_hand():
    # scores: page j of row 0 has mean (s_j, 0); the group's queries add up to (1, 0)
    s = [3.0, 5.0, 5.0, -1.0, np.nan, 5.0, 2.0]
    kbar = np.zeros((8, 1, 2))
    kbar[:7, 0, 0] = s
    q = np.array([[[0.25, 1.0], [0.75, -1.0]]])
    table = np.array([[0, 1, 2, 3, 4, 5, 6]], np.int32)
    pick = lambda topk, first=0, last=0, n=28: oracle.page_select(q, kbar, table, [n], 4, topk, first, last)[0, 0].tolist()  # noqa: E731
    assert pick(2) == [1, 2]  # a tie keeps the lower page
    assert pick(4) == [0, 1, 2, 5]
    assert pick(3, 1, 1) == [0, 1, 6]
    assert pick(6) == [0, 1, 2, 3, 5, 6]  # the NaN is last
    assert pick(9) == [0, 1, 2, 3, 4, 5, 6, -1, -1]
    assert pick(2, n=5) == [0, 1] and pick(2, n=0) == [-1, -1] and pick(2, n=-1) == [-1, -1]


def test_means():
    x = np.arange(24, dtype=np.float64).reshape(4, 2, 3)
    np.testing.assert_allclose(oracle.page_means(x, 2), [[3, 4, 5], [6, 7, 8]])
