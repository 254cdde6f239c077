"""Paged attention at its edges: rows that see nothing, and what surrounds them (against oracle/paged.py, with the bars of
tests/test_gpu_paged.py)."""
import pytest
import torch

from post_activation_quantization_b200 import rptq
from tests.gpu_common import DEV
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
