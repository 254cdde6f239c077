"""Paged attention at its edges: rows that see nothing, and what surrounds them (against oracle/paged.py, with the bars of
tests/test_gpu_paged.py)."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
from post_activation_quantization_b200 import rptq
from tests import paged_bars
from tests.gpu_common import DEV, to_np
from tests.test_gpu_paged import TD, Case, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_activation_quantization_b200 import build
    build.build()
    rptq.lib()
    yield
    assert rptq.rptq_device_error() == 0


def _attend_into_sevens(c, Hq, dtype):
    q = c.queries(Hq, dtype)
    out = torch.full((c.T, Hq, c.D), 7.0, dtype=TD[dtype], device=DEV)
    c.attend(q.to(DEV), out=out)
    return q, out


@pytest.mark.parametrize("sums", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 3)])
@pytest.mark.parametrize("ns,lens", [
    ([140, 40], [100, 25]),              # one block holds rows before position 0 and rows that see something
    ([140, 40, 150], [100, 25, 1500]),   # the same with the positions in two parts
    ([300, 1, 33], [40, 0, 33])])        # a block of 128 rows that all lie before position 0; an empty cache
def test_rows_before_position_0_are_0_in_a_chunk(ns, lens, D, bits, dtype, sums):
    c = Case(1, D, bits, 16, ns, lens, seed=51, sums=sums)
    z = c.v_cal[2][c.v_cal[0]]
    assert ((z < 0) | (z > 2 ** bits - 1)).any()  # channels whose values do not reach 0
    q, out = _attend_into_sevens(c, 2, dtype)
    for b, (n, L) in enumerate(zip(ns, lens)):
        assert (out[c.start[b]:c.start[b] + max(0, n - L)] == 0).all()
    check_attention(c, q, out, dtype, weights=c.d["w"])


@pytest.mark.parametrize("D,bits,page,dtype,sums", [(64, 4, 16, "f32", False), (128, 3, 64, "f16", False), (128, 4, 128, "bf16", False),
                                                    (64, 3, 16, "bf16", True), (128, 3, 32, "f32", True)])
def test_decode_rings_that_turn_many_times(D, bits, page, dtype, sums):
    """One row to a K/V head: its query fragments lie in the last stage of every warp's ring until the first turn fills it.
    Three to thirty turns a warp, the same result every time and the definition's."""
    B = 80
    c = Case(8, D, bits, page, [1] * B, [4000 - 47 * b for b in range(B)], seed=52, sums=sums)
    q = c.queries(8, dtype)
    qd = q.to(DEV)
    first = c.attend(qd)
    w1 = c.d["w"].clone() if sums else None
    for _ in range(20):
        if sums:
            c.d["w"].copy_(torch.from_numpy(c.w0))
        assert torch.equal(c.attend(qd), first)
        assert not sums or torch.equal(c.d["w"], w1)
    check_attention(c, q, first, dtype, weights=c.d["w"])


@pytest.mark.parametrize("ns", [[1, 1], [150, 3]])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("dtype,sums", [("bf16", False), ("f16", True), ("f32", False), ("f32", True)])
def test_no_position_anywhere(ns, D, dtype, sums):
    """max_len = 0: every row is 0, no sum changes, no workspace is needed; a sequence that has positions all the same is out
    of range."""
    c = Case(2, D, 3, 16, ns, [0, 0], seed=53, rows_behind=2, sums=sums)
    c.max_len = 0
    assert rptq.rptq_kv_paged_attention_workspace_size(c.T, 4, 2, D, TD[dtype], 2, c.max_q, 0, sums) == 0
    _, out = _attend_into_sevens(c, 4, dtype)
    assert (out[:-2] == 0).all() and (out[-2:] == 7).all()
    c.d["lens"][1] = 1
    _, out = _attend_into_sevens(c, 4, dtype)
    assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_RANGE
    assert (out[:ns[0]] == 0).all() and (out[ns[0]:] == 7).all()
    assert not sums or torch.equal(c.d["w"].cpu(), torch.from_numpy(c.w0))


def test_eviction_with_the_largest_budget():
    """A budget that no length reaches: the index of the list of kept positions goes up to 2^31 - 2."""
    c = Case(1, 32, 4, 16, [0], [70], seed=54, sums=True)
    d = c.d
    new, kept = rptq.rptq_kv_paged_evict(d["k"], d["v"], d["w"], d["lens"], d["table"], 4, 2 ** 31 - 1, 5)
    assert new.tolist() == [70] and kept.shape == (1, 1, 2 ** 31 - 1)
    assert kept[0, 0, :70].tolist() == list(range(70))
    assert all(bool((part == -1).all()) for part in kept[0, 0, 70:].split(1 << 28))
    assert torch.equal(d["k"].cpu(), torch.from_numpy(c.k0)) and torch.equal(d["w"].cpu(), torch.from_numpy(c.w0))


def _above_a_tail(D, bits, n, dtype, sums, drop=25.5):
    """(output, its 64-bit value, tail's value times its positions): position 0 (value 0) scores `drop` binary orders above all
    others, whose value is the largest there is, so that the output is the tail's alone."""
    H, L, qmax = 80, 2048, 2 ** bits - 1  # (heads enough that the positions of a chunk are not split: one maximum for all)
    c = Case(H, D, bits, 16, [n], [L], seed=55, sums=sums)
    one = lambda s: (np.zeros(H * D, np.int32), np.array([s], np.float32), np.zeros(1, np.int32))  # noqa: E731
    c.k_cal, c.v_cal = one(1.0), one(0.5)
    c.k0[:], c.v0[:] = 0, 255  # all codes 0; all codes qmax
    c.k0[c.table[0, 0], :, 0], c.v0[c.table[0, 0], :, 0] = 255, 0
    for name, x in (("k", c.k0), ("v", c.v0)):
        c.d[name].copy_(torch.from_numpy(x))
    c.d["kc"], c.d["vc"] = ([torch.from_numpy(x).to(DEV) for x in cal] for cal in (c.k_cal, c.v_cal))
    q = torch.full((n, H, D), drop * np.log(2.0) / (qmax * D ** 0.5), dtype=torch.float64).to(TD[dtype])
    got = to_np(c.attend(q.to(DEV))).astype(np.float64)
    ref = paged.attention(to_np(q).astype(np.float64), c.start, c.lens, c.table, c.k0, c.v0, c.k_cal, c.v_cal, bits)[0]
    unit = 0.5 * qmax * (L - 1)
    assert (ref > unit * 2.0 ** -(drop + 0.2)).all() and (ref < unit * 2.0 ** -(drop - 0.2)).all()
    return got, ref, unit


@pytest.mark.parametrize("D,bits,n,dtype,sums", [
    (64, 4, 40, "f16", True), (128, 3, 40, "bf16", True), (64, 3, 40, "f16", False), (128, 4, 40, "bf16", False),
    (64, 4, 1, "f16", True), (128, 3, 1, "f16", False), (64, 3, 1, "bf16", False)])
def test_one_position_above_a_long_tail(D, bits, n, dtype, sums):
    """A weight is held as fp16 times at least 2^4 where the largest is 1, so it is off by at most half of fp16's smallest
    step: 2^-25 / 2^4 = 2^-29 of the largest, for each of the L - 1 positions of the tail (weights of 2^-25.5).  Beside that, of the
    result: the output's rounding, eps / 2; 2^-11 for scores (q' is exact here; sums of D products of fp32's precision: 25.5 ln 2
    (D/4 + 32) 2^-24 < 7e-5), exponentials (7.5e-5), codes as subnormals in the values' products (6e-5) and sums cut off
    at 2^-23 in L / 16 steps (2e-5), together below 2^-11 = 4.9e-4; 2^-9 where the scores' codes are subnormals too (decode, bf16
    without sums: 6e-5 of a score of 25.5 ln 2 = 17.7)."""
    got, ref, unit = _above_a_tail(D, bits, n, dtype, sums)
    rel = 2.0 ** -11 + torch.finfo(TD[dtype]).eps / 2 + (2.0 ** -9 if dtype == "bf16" and n == 1 and not sums else 0.0)
    err, tol = np.abs(got - ref), unit * 2.0 ** -29 + rel * ref
    assert (err <= tol).all(), f"worst error {err.max():.3e} of {ref.max():.3e}, over its bar {(err / tol).max():.3g}"


@pytest.mark.parametrize("D,bits,n,sums", [(64, 3, 40, False), (128, 4, 40, True), (64, 4, 1, False), (128, 3, 1, True), (64, 4, 3, False)])
def test_one_position_above_a_long_tail_in_fp32(D, bits, n, sums):
    """Two fp16 parts times at least 2^13 (many rows) or 2^11 (few): half of the smallest step is 2^-25 / 2^13 = 2^-38 or 2^-36 of the
    largest weight.  Of the result: scores 25.5 ln 2 (D/4 + 32) 2^-24 < 7e-5 and 17.7 2^-22 for q' in 22 bits, exponents below 64 rounded to 2^-19, the rest less: 1e-4."""
    got, ref, unit = _above_a_tail(D, bits, n, "f32", sums)
    err, tol = np.abs(got - ref), unit * 2.0 ** (-38 if n > 8 else -36) + 1e-4 * ref
    assert (err <= tol).all(), f"worst error {err.max():.3e} of {ref.max():.3e}, over its bar {(err / tol).max():.3g}"


def test_read_back_refuses_rows_that_are_not_outs():
    c = Case(2, 64, 3, 16, [3], [20], seed=56)
    args = lambda **k: rptq.rptq_kv_paged_dequant(c.d["k"], c.d["table"], c.d["start"], c.d["lens"] * 0, *c.d["kc"], 3, **k)  # noqa: E731
    want = args(T=3)
    out = torch.empty_like(want)
    assert args(out=out) is out and torch.equal(out, want)
    assert args(T=3, out=out) is out and torch.equal(out, want)
    for T in (0, 2, 4):
        with pytest.raises(rptq.RptqError):
            args(T=T, out=out)


def test_rows_of_one_head_may_have_any_head_stride():
    """[T, 1, D] as a transposed [1, T, D]: dense rows, whatever the stride of the one head."""
    c = Case(1, 64, 3, 16, [3], [20], seed=57)
    d, x = c.d, c.tokens(c.mk, "f16").to(DEV)
    odd = x.reshape(1, 3, 64).transpose(0, 1)
    assert odd.shape == (3, 1, 64) and odd.stride(1) != 64
    pools = []
    for k in (x, odd):
        pool = d["k"].clone()
        rptq.rptq_kv_paged_append(k, None, d["start"], d["lens"], d["table"], pool, None, *d["kc"], None, None, None, 3)
        pools.append(pool)
    assert torch.equal(*pools)
    assert torch.equal(c.attend(odd), c.attend(x))


@pytest.mark.parametrize("seed", [71, 72])
@pytest.mark.parametrize("case", paged_bars.CASES, ids=str)
def test_attention_of_16_bits_in_norm(case, seed):
    """Every 16-bit kernel within a bar that a mask off by one position does not pass."""
    H, G, D, bits, page, ns, lens, dtype, sums = case
    c = Case(H, D, bits, page, ns, lens, seed=seed, sums=sums)
    q = paged_bars.queries(c, G, dtype)
    got = to_np(c.attend(q.to(DEV))).astype(np.float64)
    err, bar = paged_bars.check_norm(c, to_np(q).astype(np.float64), got, dtype)
    print(f"error {err:.2e} bar {bar:.2e}")
