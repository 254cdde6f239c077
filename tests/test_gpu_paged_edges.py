"""Paged attention at its edges: rows that see nothing, and what surrounds them (against oracle/paged.py, with the bars of
tests/test_gpu_paged.py)."""
import numpy as np
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
