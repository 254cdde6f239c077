"""The bar on the norm of a paged attention output's error (tests/paged_bars.py) passes the rounded definition and rejects
mistakes planted in it, on the CPU."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
from tests import paged_bars, test_gpu_paged


def _softmax(x):
    e = np.exp(x - np.where(np.isfinite(x), x, -np.inf).max(axis=-1, keepdims=True, initial=-1e300))
    e = np.where(np.isfinite(x), e, 0.0)
    return e / np.maximum(e.sum(axis=-1, keepdims=True), 1e-300)


def _mutants(parts, c, q64):
    """Outputs of a softmax whose scores, or whose mask, are wrong."""
    def outputs(change):
        return np.concatenate([np.einsum("anp,pad->nad", _softmax(change(x, K, b)), V) for b, (K, V, x, _) in enumerate(parts)])

    def last_dropped(x, K, b):
        x = x.copy()
        n, L = x.shape[1:]
        for i in range(n):
            if L - n + i > 0:
                x[:, i, L - n + i] = -np.inf
        return x

    def first_dropped(x, K, b):
        x = x.copy()
        x[:, :, :1] = np.where(np.arange(x.shape[1])[:, None] + x.shape[2] - x.shape[1] > 0, -np.inf, x[:, :, :1])
        return x

    def next_seen(x, K, b):
        x = x.copy()
        n, L = x.shape[1:]
        for i in range(n - 1):
            x[:, i, L - n + i + 1] = np.einsum("ad,ad->a", q64[c.start[b] + i], K[L - n + i + 1]) / K.shape[2] ** 0.5
        return x

    yield "unchanged", outputs(lambda x, K, b: x)
    yield "scores times 0.9", outputs(lambda x, K, b: 0.9 * x)
    yield "scores times 1.1", outputs(lambda x, K, b: 1.1 * x)
    yield "last position dropped", outputs(last_dropped)
    yield "first position dropped", outputs(first_dropped)
    if max(x.shape[1] for _, _, x, _ in parts) > 8:
        yield "next position seen", outputs(next_seen)


@pytest.mark.parametrize("case", paged_bars.CASES, ids=str)
def test_the_bar_rejects_planted_mistakes(case, monkeypatch):
    H, G, D, bits, page, ns, lens, dtype, sums = case
    monkeypatch.setattr(test_gpu_paged, "DEV", "cpu")
    c = test_gpu_paged.Case(H, D, bits, page, ns, lens, seed=61, sums=sums)
    q64 = paged_bars.queries(c, G, dtype).double().numpy()
    ref = paged.attention(q64, c.start, c.lens, c.table, c.k0, c.v0, c.k_cal, c.v_cal, bits)
    for name, out in _mutants(ref[2], c, q64):
        got = torch.from_numpy(out).to(paged_bars.TD[dtype]).double().numpy()
        if name == "unchanged":
            err, limit = paged_bars.check_norm(c, q64, got, dtype, ref)
            assert err < limit
            continue
        with pytest.raises(AssertionError, match="bar"):
            paged_bars.check_norm(c, q64, got, dtype, ref)
            pytest.fail(f"{name}: passed")
