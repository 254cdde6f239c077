"""The paged cache's host-side checks, without a GPU: what is refused, with which status, and what an
empty problem does (the pointers are never read)."""
import ctypes

import pytest

from post_activation_quantization_b200 import rptq

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
A = P(16 * 1024)  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from post_activation_quantization_b200 import build
    build.build()
    return rptq.lib()


def _append(lib, **c):
    a = dict(k=A, v=A, dtype=2, T=4, H=2, D=64, stride=128, start=A, lens=A, B=2, table=A, max_pages=3, n_pages=9, page=16,
             ck=A, sk=A, zk=A, cv=A, sv=A, zv=A, g=4, bits=3, kp=A, vp=A, w=None) | c
    return lib.rptq_kv_paged_append(*a.values(), None)


def _dequant(lib, **c):
    a = dict(pages=A, H=2, D=64, bits=3, start=A, begin=A, B=2, table=A, max_pages=3, n_pages=9, page=16, T=4, cl=A, s=A,
             z=A, g=4, out=A, dtype=2) | c
    return lib.rptq_kv_paged_dequant(*a.values(), None)


def _attend(lib, **c):
    a = dict(q=A, dtype=2, T=4, Hq=4, H=2, D=64, stride=256, start=A, lens=A, B=2, max_q=3, max_len=40, table=A, max_pages=3,
             n_pages=9, page=16, kp=A, vp=A, ck=A, sk=A, zk=A, cv=A, sv=A, zv=A, g=4, bits=3, scale=0.0, out=A, w=None,
             ws=A, ws_bytes=1 << 40) | c
    return lib.rptq_kv_paged_attention(*a.values(), None)


def _evict(lib, **c):
    a = dict(kp=A, vp=A, w=A, B=2, H=2, D=64, bits=3, lens=A, table=A, max_pages=3, n_pages=9, page=16, max_len=40, budget=8,
             recent=2, new=P(32 * 1024), kept=A) | c
    return lib.rptq_kv_paged_evict(*a.values(), None)


CALLS = [_append, _dequant, _attend, _evict]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad,status", [
    (dict(bits=5), UNSUPPORTED), (dict(D=40), UNSUPPORTED), (dict(D=288), UNSUPPORTED), (dict(H=0), UNSUPPORTED),
    (dict(H=600), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(B=-1), INVALID), (dict(max_pages=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(max_pages=1 << 27), UNSUPPORTED), (dict(n_pages=1 << 31), UNSUPPORTED), (dict(table=None), INVALID)])
def test_shapes_every_call_refuses(lib, call, bad, status):
    if call is _attend and "H" in bad:
        bad = bad | dict(Hq=max(bad["H"], 1))
    assert call(lib, **bad) == status


@pytest.mark.parametrize("call,bad,status", [
    (_append, dict(dtype=3), UNSUPPORTED), (_append, dict(T=-1), INVALID), (_append, dict(g=0), INVALID),
    (_append, dict(stride=127), INVALID), (_append, dict(stride=132), INVALID),  # below a row; not 16 bytes
    (_append, dict(k=None, v=None), INVALID), (_append, dict(k=P(16 * 1024 + 8)), INVALID),
    (_append, dict(vp=P(16 * 1024 + 4)), INVALID), (_append, dict(sv=None), INVALID), (_append, dict(start=None), INVALID),
    (_append, dict(k=None, w=A), INVALID), (_append, dict(T=1 << 31), UNSUPPORTED),
    (_dequant, dict(dtype=7), UNSUPPORTED), (_dequant, dict(T=-1), INVALID), (_dequant, dict(out=None), INVALID),
    (_dequant, dict(out=P(16 * 1024 + 2)), INVALID), (_dequant, dict(begin=None), INVALID),
    (_attend, dict(dtype=-1), UNSUPPORTED), (_attend, dict(Hq=3), INVALID), (_attend, dict(Hq=1), INVALID),
    (_attend, dict(T=-1), INVALID), (_attend, dict(max_len=49), INVALID), (_attend, dict(max_len=-1), INVALID),
    (_attend, dict(max_q=-1), INVALID), (_attend, dict(scale=-1.0), INVALID), (_attend, dict(scale=float("nan")), INVALID),
    (_attend, dict(scale=float("inf")), INVALID), (_attend, dict(stride=255), INVALID), (_attend, dict(stride=260), INVALID),
    (_attend, dict(q=None), INVALID), (_attend, dict(out=P(16 * 1024 + 4)), INVALID), (_attend, dict(zk=None), INVALID),
    (_attend, dict(T=1 << 31), UNSUPPORTED), (_attend, dict(T=1 << 30), UNSUPPORTED),  # T Hq
    (_attend, dict(w=A, ws=None), WORKSPACE), (_attend, dict(w=A, ws_bytes=8), WORKSPACE),
    (_attend, dict(w=A, ws=P(16 * 1024 + 8)), WORKSPACE),
    (_evict, dict(budget=0), INVALID), (_evict, dict(recent=-1), INVALID), (_evict, dict(recent=9), INVALID),
    (_evict, dict(max_len=49), INVALID), (_evict, dict(w=None), INVALID), (_evict, dict(kept=None), INVALID),
    (_evict, dict(new=A), INVALID), (_evict, dict(new=P(16 * 1024 + 4)), INVALID)])  # new_lens over lens
def test_arguments_each_call_refuses(lib, call, bad, status):
    assert call(lib, **bad) == status


def test_empty_problems_read_no_pointer(lib):
    none = dict.fromkeys(("start", "lens", "table"))
    for T, B in ((0, 2), (4, 0)):
        e = none | dict(T=T, B=B)
        assert _append(lib, k=None, v=None, kp=None, vp=None, ck=None, sk=None, zk=None, cv=None, sv=None, zv=None, **e) == OK
        assert _attend(lib, q=None, kp=None, vp=None, out=None, ws=None, ws_bytes=0, w=A, **e) == OK
        assert _dequant(lib, pages=None, out=None, start=None, begin=None, table=None, T=T, B=B) == OK
    assert _attend(lib, max_q=0, q=None, **none) == OK
    assert _evict(lib, B=0, kp=None, vp=None, w=None, lens=None, table=None, new=None, kept=None) == OK


def test_workspace_size_rules(lib):
    f = lib.rptq_kv_paged_attention_workspace_size
    assert f(4, 4, 2, 64, 2, 2, 3, 40, 1) > 0
    for bad in ((0, 4, 2, 64, 2, 2, 3, 40, 1), (4, 3, 2, 64, 2, 2, 3, 40, 1), (4, 4, 2, 64, 9, 2, 3, 40, 1),
                (4, 4, 2, 64, 2, 0, 3, 40, 1), (4, 4, 2, 64, 2, 2, 0, 40, 1), (4, 4, 2, 64, 2, 2, 3, 0, 1)):
        assert f(*bad) == 0
