"""Pins of the paged cache's oracle (oracle/paged.py): against the dense cache's definitions where the
two describe the same thing, and by hand."""
import numpy as np

import oracle
import oracle.paged as paged

H, D, P, bits = 2, 32, 16, 3


def _cal(seed):
    rng = np.random.default_rng(seed)
    mx = rng.uniform(0.5, 2, H * D).astype(np.float32)
    mn = rng.uniform(-2, -0.5, H * D).astype(np.float32)
    c = oracle.calibrate(mx, mn, 4, 5, bits)
    return c["labels"], c["scale"], c["zero"]


def _pools(rng, n_pages):
    shape = (n_pages, H, P, D * bits // 8)
    return rng.integers(0, 256, shape, dtype=np.uint8), rng.integers(0, 256, shape, dtype=np.uint8)


def test_append_and_read_back_equal_the_dense_cache():
    rng = np.random.default_rng(0)
    k, _ = _pools(rng, 5)
    table = np.array([[3, 1], [0, 4]], np.int32)
    cal = _cal(1)
    x = rng.standard_normal((20, H, D)).astype(np.float32)
    start, lens = np.array([0, 19, 20]), np.array([20, 1])
    out = paged.append(k, x, start, lens, table, *cal, bits)
    whole = oracle.kv_quant(np.ascontiguousarray(x.transpose(1, 0, 2)[None]), *cal, bits)[0]
    assert np.array_equal(out[3, :, 1:], whole[:, :15]) and np.array_equal(out[1, :, :4], whole[:, 15:19])
    assert np.array_equal(out[0, :, 0], whole[:, 19])
    assert np.array_equal(out[3, :, 0], k[3, :, 0]) and np.array_equal(out[2], k[2])
    assert np.array_equal(out[0, :, 1:], k[0, :, 1:]) and np.array_equal(out[4], k[4])
    got = paged.values(out, table, 0, 20, D, *cal, bits)[1:]
    dense = oracle.kv_dequant(whole[None], D, *cal, bits)[0].transpose(1, 0, 2)[:19]
    assert np.array_equal(got, dense)


def test_attention_of_one_token_equals_the_dense_decode_step():
    rng = np.random.default_rng(2)
    k, v = _pools(rng, 4)
    table, lens = np.array([[2, 0, 3]], np.int32), np.array([37])
    kc, vc = _cal(3), _cal(4)
    q = rng.standard_normal((1, H, D)).astype(np.float32)
    w0 = rng.random((4, H, P)).astype(np.float32)
    out, w, _ = paged.attention(q, np.array([0, 1]), lens, table, k, v, kc, vc, bits, weights=w0)
    dk = np.ascontiguousarray(paged.gather(k, table, 0, 37).transpose(1, 0, 2)[None])
    dv = np.ascontiguousarray(paged.gather(v, table, 0, 37).transpose(1, 0, 2)[None])
    ref, _ = oracle.kv_decode_attention(q, dk, dv, 37, D, *kc, *vc, bits)
    np.testing.assert_allclose(out[0], ref[0], rtol=1e-12, atol=1e-12)
    grown = w - w0
    np.testing.assert_allclose(grown.sum(axis=(0, 2)), 1.0, rtol=1e-6)
    assert (grown[1] == 0).all() and (grown[3, :, 5:] == 0).all()


def test_attention_is_causal_and_grouped_heads_share_keys():
    """A chunk's rows equal each token's own decode step at its own length; a row without positions is 0."""
    rng = np.random.default_rng(5)
    k, v = _pools(rng, 3)
    table = np.array([[1, 2], [0, 0]], np.int32)
    kc, vc = _cal(6), _cal(7)
    q = rng.standard_normal((6, 2 * H, D)).astype(np.float32)
    start, lens = np.array([0, 4, 6]), np.array([21, 1])
    out, _, _ = paged.attention(q, start, lens, table, k, v, kc, vc, bits)
    for i in range(4):
        one, _, _ = paged.attention(q[i:i + 1], np.array([0, 1]), np.array([18 + i]), table[:1], k, v, kc, vc, bits)
        np.testing.assert_allclose(out[i], one[0], rtol=1e-12)
    assert (out[4] == 0).all() and (out[5] != 0).any()  # positions -1 and 0
    V0 = paged.values(v, table, 1, 1, D, *vc, bits)[0]
    np.testing.assert_allclose(out[5], V0.repeat(2, axis=0), rtol=1e-12)


def test_eviction_keeps_the_largest_and_the_recent_in_order():
    rng = np.random.default_rng(8)
    k, v = _pools(rng, 3)
    w = rng.random((3, H, P)).astype(np.float32)
    table, lens = np.array([[2, 0]], np.int32), np.array([20])
    row = np.array([5, 1, 9, 5, 0, 5, 2, 9, 5, 1, 1, 1, 1, 1, 1, 1, 7, 7, 0, 0], np.float32)
    w[2, 0], w[0, 0, :4] = row[:16], row[16:]
    k2, v2, w2, new, kept = paged.evict(k, v, w, lens, table, 6, 2)
    assert new.tolist() == [6]
    assert kept[0, 0].tolist() == [2, 7, 16, 17, 18, 19]  # 9, 9, 7, 7 and the last two
    assert w2[2, 0, :6].tolist() == [9, 9, 7, 7, 0, 0] and np.array_equal(w2[2, 0, 6:], w[2, 0, 6:])
    assert np.array_equal(k2[2, 0, 1], k[2, 0, 7]) and np.array_equal(v2[2, 0, 3], v[0, 0, 1])
    assert np.array_equal(k2[0], k[0]) and np.array_equal(k2[1], k[1])
    _, _, _, _, kept = paged.evict(k, v, w, lens, table, 7, 2)  # the tie of the four fives: position 0
    assert kept[0, 0].tolist() == [0, 2, 7, 16, 17, 18, 19]
    _, _, _, new, kept = paged.evict(k, v, w, np.array([3]), table, 5, 2)
    assert new.tolist() == [3] and kept[0, 1].tolist() == [0, 1, 2, -1, -1]
