"""GPU parity of the paged packed K/V cache against its 64-bit definition (oracle/paged.py).

Append, read-back and eviction move or round exactly: bytes, fp32 values, sums and positions are equal.
(16-bit read-backs are the fp32 value rounded once more, as on the host.)

Attention's bars follow from the arithmetic.  With q'_d = q_d s_d and the code k_pd (the part
-q'_d z_d of a score is the same for every position and drops out of the softmax):
  * a score is scale * sum_d q'_d k_pd.  q' is rounded to 22 bits (two fp16 parts; fp32 inputs, and
    every type when the running sums are kept) or to 11 (one fp16; half a step is 2^-11), and summed in
    fp32 in D/16 or D steps of one rounding each on values no larger than sum|q' k|; each tensor-core
    step is counted as 4 roundings:  e_x = scale (r + (D/4 + 32) u) sum_d |q'_d| k_pd, u = 2^-24, r =
    2^-21 or 2^-11, with the constant part's own rounding, (|z| <= 2^21) at most the same sum with |z|;
  * a weight is off by a factor e^(2 max e_x), by its exponential (2^-21), by its rounding to fp16 parts
    (2^-21, or 2^-10 for a numerator and a denominator of 11 bits) and, below the smallest part, by
    2^-24 of the row's largest weight;
  * sums over L positions take at most L/4 + 64 fp32 roundings, each counted 4 times;
  * out_d = s_d (sum_p w_p k_pd - z_d), where a kernel may take the codes about one of them, c <= 2 h - 1, h = 2^(bits-1), as
    s_d (sum_p w_p (k_pd - c) - (z_d - c)): the rounded sum is then up to sum_p w_p |k_pd - c| < 2 h whatever sum_p w_p k_pd
    is (all codes 0: -c), so errors are relative to s_d (sum_p w_p k_pd + |z_d| + 2 h) = `mag`;
  * the output is rounded to its type: half a step, eps/2, relative."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.paged as paged
from post_activation_quantization_b200 import rptq, synthetic
from tests.gpu_common import DEV, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_activation_quantization_b200 import build
    build.build()
    rptq.lib()
    yield
    assert rptq.rptq_device_error() == 0


class Case:
    """Pools of random codes, a page table in random order, calibrations, and their device copies."""

    def __init__(self, H, D, bits, page, ns, lens, seed=0, rows_behind=0, sums=False, outliers=0.01):
        rng = self.rng = np.random.default_rng(seed + 1000 * H + D)
        self.H, self.D, self.bits, self.P = H, D, bits, page
        self.start = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
        self.lens = np.array(lens, np.int32)
        self.T = int(self.start[-1]) + rows_behind
        self.max_q, self.max_len = max(max(ns), 1), max(max(lens), 1)
        B, mp = len(lens), -(-self.max_len // page) + 1
        n_pages = B * mp + 2
        self.table = rng.permutation(n_pages)[:B * mp].reshape(B, mp).astype(np.int32)
        shape = (n_pages, H, page, D * bits // 8)
        self.k0 = rng.integers(0, 256, shape, dtype=np.uint8)
        self.v0 = rng.integers(0, 256, shape, dtype=np.uint8)
        self.mk = synthetic.channel_model(H * D, seed, outliers, tag=1)
        self.mv = synthetic.channel_model(H * D, seed, outliers, tag=2)
        self.k_cal, self.v_cal = self._cal(self.mk), self._cal(self.mv)
        self.w0 = (rng.random((n_pages, H, page)) * 3).astype(np.float32) if sums else None
        d = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        self.d = dict(k=d(self.k0), v=d(self.v0), w=d(self.w0), start=d(self.start), lens=d(self.lens), table=d(self.table),
                      kc=[d(x) for x in self.k_cal], vc=[d(x) for x in self.v_cal])

    def _cal(self, m):
        c, hw = m.center.numpy(), m.half_width.numpy()
        cal = oracle.calibrate((c + hw).astype(np.float32), (c - hw).astype(np.float32), min(16, c.size), 5, self.bits)
        return cal["labels"], cal["scale"], cal["zero"]

    def tokens(self, m, dtype):
        u = torch.from_numpy(self.rng.uniform(-1.1, 1.1, (self.T, self.H * self.D)).astype(np.float32))
        return (m.center + m.half_width * u).to(TD[dtype]).reshape(self.T, self.H, self.D)

    def queries(self, Hq, dtype):
        hw = self.mk.half_width.numpy().reshape(self.H, self.D).repeat(Hq // self.H, axis=0)
        return torch.from_numpy((self.rng.standard_normal((self.T, Hq, self.D)) * 2 / hw).astype(np.float32)).to(TD[dtype])

    def attend(self, q, out=None, **kw):
        d = self.d
        return rptq.rptq_kv_paged_attention(q, d["start"], d["lens"], d["table"], d["k"], d["v"], *d["kc"], *d["vc"], self.bits,
                                            max_q=self.max_q, max_len=self.max_len, out=out, weights=d["w"], **kw)


def _per_channel(cal, H, D):
    return [a.astype(np.float64).reshape(H, D) for a in (cal[1][cal[0]], cal[2][cal[0]])]


def check_attention(c, q, out, dtype, scale=0.0, weights=None, k=None, v=None):
    """out (and the grown sums) against the definition, within the module's bars."""
    H, D, G = c.H, c.D, q.shape[1] // c.H
    sc = scale or 1 / math.sqrt(D)
    k, v = c.k0 if k is None else k, c.v0 if v is None else v
    q64 = to_np(q).astype(np.float64)
    ref, w_ref, parts = paged.attention(q64, c.start, c.lens, c.table, k, v, c.k_cal, c.v_cal, c.bits, sc, c.w0)
    sk, zk = (a.repeat(G, axis=0) for a in _per_channel(c.k_cal, H, D))
    sv, zv = (a.repeat(G, axis=0) for a in _per_channel(c.v_cal, H, D))
    wide = dtype == "f32"
    rx = 2.0 ** -21 if wide or c.w0 is not None else 2.0 ** -11
    rw = 2.0 ** -20 if wide else 2.0 ** -10
    got = to_np(out).astype(np.float64)
    w_tol = None if c.w0 is None else np.abs(w_ref) * U + 1e-30
    for b, (K, V, x, w) in enumerate(parts):
        n, L = c.start[b + 1] - c.start[b], c.lens[b]
        if n == 0 or L == 0:
            continue
        rows = slice(c.start[b], c.start[b] + n)
        code = np.abs(K / sk + zk)  # [L, Hq, D]
        qs = np.abs(q64[rows]) * sk
        top = np.where(np.isfinite(x), np.einsum("nad,pad->anp", qs, code + np.abs(zk) * 0), 0.0).max(axis=2)
        e_x = sc * (rx + (D / 4 + 32) * U) * top + sc * 4 * U * np.einsum("nad,ad->an", qs, np.abs(zk))
        sums = 4 * (L / 4 + 64) * U
        rel = np.expm1(2 * e_x) + 2.0 ** -21 + rw + sums  # [Hq, n]
        qmax = 2 ** c.bits - 1
        mag = sv * np.abs(np.einsum("anp,pad->nad", w, V / sv + zv)) + sv * (np.abs(zv) + 2 ** c.bits)
        tol = rel.T[..., None] * mag + sv * qmax * L * U * (w.max(axis=2).T[..., None] * 2) + 8 * U * mag
        tol = tol + np.abs(ref[rows]) * torch.finfo(TD[dtype]).eps / 2 * (1 + 1e-6) + 1e-30
        if dtype == "f16":
            tol = tol + 2.0 ** -25
        err = np.abs(got[rows] - ref[rows])
        assert (err <= tol).all(), f"sequence {b}: worst error {err.max():.3e}, worst over its bar {(err / tol).max():.3g}"
        empty = ~np.isfinite(x).any(axis=2)  # rows that see nothing are exactly 0
        assert (got[rows].transpose(1, 0, 2)[empty] == 0).all()
        if w_tol is not None:
            e_w = np.expm1(2 * e_x) + 2.0 ** -20 + sums
            t = ((w * e_w[..., None]).reshape(H, G * n, L).sum(axis=1) + (G * n + 4) * U * w.reshape(H, G * n, L).sum(axis=1)).T
            pos = np.arange(L)
            w_tol[c.table[b, pos // c.P], :, pos % c.P] += t
    if weights is not None:
        err = np.abs(to_np(weights).astype(np.float64) - w_ref)
        assert (err <= w_tol).all(), f"sums: worst error {err.max():.3e}, over its bar {(err / w_tol).max():.3g}"


# ---- append and read-back ------------------------------------------------------------------------
RAGGED = [
    # H, D, bits, page, new rows, lengths, dtype
    (1, 32, 3, 16, [1], [1], "f32"),
    (3, 64, 4, 16, [1, 0, 1, 1], [17, 5, 16, 300], "f16"),
    (5, 128, 3, 64, [3, 70, 1], [3, 131, 64], "bf16"),
    (2, 96, 3, 32, [40, 2], [33, 2], "f32"),  # seven rows fall before position 0
    (96, 128, 3, 64, [1, 1, 1], [64, 65, 2048], "bf16"),
    (2, 256, 4, 256, [300, 1, 17], [301, 256, 18], "f16"),
    (17, 64, 3, 128, [200], [200], "bf16"),
]


@pytest.mark.parametrize("H,D,bits,page,ns,lens,dtype", RAGGED)
def test_append_equals_the_definition(H, D, bits, page, ns, lens, dtype):
    c = Case(H, D, bits, page, ns, lens, seed=3, rows_behind=2, sums=True)
    k, v = c.tokens(c.mk, dtype), c.tokens(c.mv, dtype)
    wide = torch.zeros((c.T, 3 * H, D), dtype=TD[dtype])  # K and V as slices of a wider row
    wide[:, H:2 * H], wide[:, 2 * H:] = k, v
    wide = wide.to(DEV)
    d = c.d
    rptq.rptq_kv_paged_append(wide[:, H:2 * H], wide[:, 2 * H:], d["start"], d["lens"], d["table"], d["k"], d["v"], *d["kc"],
                              *d["vc"], bits, weights=d["w"])
    k_ref, w_ref = paged.append(c.k0, oracle._f32(k), c.start, c.lens, c.table, *c.k_cal, bits, c.w0)
    v_ref = paged.append(c.v0, oracle._f32(v), c.start, c.lens, c.table, *c.v_cal, bits)
    assert np.array_equal(to_np(d["k"]), k_ref) and np.array_equal(to_np(d["v"]), v_ref)
    assert np.array_equal(to_np(d["w"]), w_ref)


def test_append_of_one_tensor_leaves_the_other():
    c = Case(4, 64, 3, 16, [2, 1], [20, 9], seed=4)
    v = c.tokens(c.mv, "bf16")
    d = c.d
    rptq.rptq_kv_paged_append(None, v.to(DEV), d["start"], d["lens"], d["table"], None, d["v"], None, None, None, *d["vc"], 3)
    assert np.array_equal(to_np(d["v"]), paged.append(c.v0, oracle._f32(v), c.start, c.lens, c.table, *c.v_cal, 3))
    rptq.rptq_kv_paged_append(v.to(DEV), None, d["start"], d["lens"], d["table"], d["k"], None, *d["kc"], None, None, None, 3)
    assert np.array_equal(to_np(d["k"]), paged.append(c.k0, oracle._f32(v), c.start, c.lens, c.table, *c.k_cal, 3))


@pytest.mark.parametrize("H,D,bits,page,ns,lens,dtype", RAGGED)
def test_read_back_equals_the_definition(H, D, bits, page, ns, lens, dtype):
    n = [min(a, b) for a, b in zip(ns, lens)]
    c = Case(H, D, bits, page, n, lens, seed=5, rows_behind=3)
    begin = c.lens - np.array(n, np.int32)
    out = torch.full((c.T, H, D), 7.0, dtype=TD[dtype], device=DEV)
    got = rptq.rptq_kv_paged_dequant(c.d["k"], c.d["table"], c.d["start"], torch.from_numpy(begin).to(DEV), *c.d["kc"], bits,
                                     out=out)
    assert got is out
    ref = [paged.values(c.k0, c.table, b, lens[b], D, *c.k_cal, bits)[begin[b]:] for b in range(len(lens))]
    ref = torch.from_numpy(np.concatenate(ref)).to(TD[dtype])
    assert torch.equal(out[:-3].cpu(), ref) and (out[-3:] == 7).all()


# ---- attention -----------------------------------------------------------------------------------
ATTEND = [
    # H, group, D, bits, page, new rows, lengths, dtype, sums
    (3, 1, 64, 4, 16, [1], [1], "f32", False),
    (3, 1, 64, 4, 16, [1], [509], "f32", True),
    (2, 1, 128, 3, 64, [1, 1, 1, 1], [1, 63, 64, 65], "f16", False),
    (4, 1, 128, 3, 64, [1, 0, 1, 1], [2048, 900, 0, 1999], "bf16", True),  # no new row; an empty cache
    (2, 1, 128, 4, 128, [1, 1], [5000, 37], "bf16", False),
    (1, 4, 128, 4, 32, [1, 1], [777, 31], "bf16", True),
    (2, 8, 64, 3, 16, [1, 2, 1], [130, 258, 15], "f16", False),
    (2, 1, 128, 3, 64, [5, 3, 1], [200, 2, 64], "f32", True),  # rows before position 0 see nothing
    (2, 2, 64, 4, 16, [7, 16, 9], [100, 16, 33], "bf16", False),
    (1, 3, 128, 3, 64, [11, 2], [65, 300], "f32", False),
    (1, 8, 128, 4, 64, [33, 6], [333, 6], "f16", False),
    (1, 1, 128, 3, 64, [129, 64, 1], [700, 64, 500], "f16", False),
    (1, 2, 64, 3, 16, [150, 257], [151, 257], "bf16", True),
    (2, 1, 128, 4, 128, [300], [1111], "bf16", True),
    (1, 1, 128, 3, 256, [140, 20], [400, 10], "f32", True),
    (1, 4, 64, 4, 32, [90, 1, 0, 5], [600, 601, 3, 5], "f16", True),
    (2, 1, 96, 3, 16, [3, 40], [50, 41], "bf16", True),
    (1, 2, 32, 4, 32, [1, 70], [3, 100], "f32", False),
    (1, 1, 256, 3, 64, [2, 1], [90, 1], "f16", False),
    (1, 2, 64, 4, 32, [20, 3], [700, 3], "f32", False),
    (1, 1, 64, 3, 16, [300], [2100], "f32", True),
    (1, 1, 128, 4, 64, [260, 9, 2], [1500, 9, 2], "f32", False),
    (2, 4, 128, 4, 64, [2, 1], [900, 40], "f32", True),
    (1, 8, 64, 3, 16, [1, 1], [640, 15], "f32", False),
    (1, 1, 64, 4, 16, [9, 12], [9, 12], "f32", True),  # shorter than the 16 positions whose mean is taken off
    (1, 2, 128, 3, 64, [8, 1], [2000, 3], "f16", False),
]


@pytest.mark.parametrize("H,G,D,bits,page,ns,lens,dtype,sums", ATTEND)
def test_attention_equals_the_definition(H, G, D, bits, page, ns, lens, dtype, sums):
    c = Case(H, D, bits, page, ns, lens, seed=11, rows_behind=2, sums=sums)
    q = c.queries(H * G, dtype)
    qd = torch.zeros((c.T, H * G + 3, D), dtype=TD[dtype], device=DEV)  # rows of a wider tensor
    qd[:, :H * G] = q.to(DEV)
    out = torch.full((c.T, H * G, D), 7.0, dtype=TD[dtype], device=DEV)
    got = c.attend(qd[:, :H * G], out=out)
    assert got is out and (out[c.start[-1]:] == 7).all()  # rows of no sequence stay
    check_attention(c, q, out, dtype, weights=c.d["w"])
    assert np.array_equal(to_np(c.d["k"]), c.k0) and np.array_equal(to_np(c.d["v"]), c.v0)


@pytest.mark.parametrize("ns,lens", [([1, 1], [900, 70]), ([200, 30], [900, 70])])
def test_attention_with_its_own_scale_and_bounds_above_the_need(ns, lens):
    c = Case(2, 128, 3, 64, ns, lens, seed=12, sums=True)
    c.max_q, c.max_len = 4 * c.max_q, (c.table.shape[1]) * 64  # bounds, not exact
    q = c.queries(4, "bf16")
    out = c.attend(q.to(DEV), scale=0.31)
    check_attention(c, q, out, "bf16", scale=0.31, weights=c.d["w"])


@pytest.mark.parametrize("n", [1, 150])
def test_one_position_far_above_the_rest(n):
    """A score far above all others: the softmax is that position's V row, exactly once."""
    c = Case(1, 128, 4, 16, [n], [400], seed=13, outliers=0.0, sums=True)
    q = c.queries(1, "f32") * 60
    out = c.attend(q.to(DEV))
    check_attention(c, q, out, "f32", weights=c.d["w"])


@pytest.mark.parametrize("n,dtype,sums", [(1, "bf16", True), (6, "f16", True), (200, "bf16", True), (200, "f16", False),
                                          (130, "f32", False)])
def test_attention_is_the_same_every_time(n, dtype, sums):
    c = Case(2, 128, 3, 64, [n, n, 1], [2000, 1300, 777], seed=14, sums=sums)
    q = c.queries(4, dtype).to(DEV)
    first = c.attend(q)
    w1 = c.d["w"].clone() if sums else None
    for _ in range(10):
        if sums:
            c.d["w"].copy_(torch.from_numpy(c.w0))
        assert torch.equal(c.attend(q), first)
        assert not sums or torch.equal(c.d["w"], w1)


def test_shared_pages_may_be_read_by_two_sequences():
    c = Case(2, 64, 4, 16, [1, 1], [64, 50], seed=15)
    c.table[1] = c.table[0]
    c.d["table"].copy_(torch.from_numpy(c.table))
    q = c.queries(2, "f16")
    check_attention(c, q, c.attend(q.to(DEV)), "f16")


# ---- eviction ------------------------------------------------------------------------------------
@pytest.mark.parametrize("H,D,bits,page,lens,budget,recent", [
    (3, 128, 3, 64, [2000, 1024, 1025, 5], 1024, 100), (2, 64, 3, 16, [40, 33, 32], 32, 32), (1, 32, 4, 16, [17], 16, 0),
    (2, 96, 3, 32, [500, 1], 1, 1), (4, 128, 4, 128, [5000, 4000], 999, 7), (8, 64, 4, 256, [700], 699, 5),
    (2, 256, 4, 16, [300, 0, 299], 150, 149), (1, 128, 3, 64, [33000], 4096, 511),
    (100, 32, 4, 16, [70, 64, 33], 33, 5), (2, 128, 4, 128, [9000, 3], 1000, 0)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_eviction_equals_the_definition(H, D, bits, page, lens, budget, recent, kind):
    c = Case(H, D, bits, page, [0] * len(lens), lens, seed=21, sums=True)
    w = c.w0
    if kind == "ties":
        w[:] = np.floor(w * 3) / 8
        w[::2] = 0
    elif kind == "odd":
        at = c.rng.random(w.shape)
        w[at < 0.1] = np.nan
        w[(at > 0.1) & (at < 0.2)] = -0.0
        w[(at > 0.2) & (at < 0.3)] = 0.0
        w[(at > 0.3) & (at < 0.31)] = np.inf
        w[(at > 0.4) & (at < 0.5)] *= -1e-42
        w[(at > 0.9) & (at < 0.95)] = -np.inf
    d = c.d
    d["w"].copy_(torch.from_numpy(w))
    new, kept = rptq.rptq_kv_paged_evict(d["k"], d["v"], d["w"], d["lens"], d["table"], bits, budget, recent,
                                         max_len=c.max_len)
    k, v, ws, n_ref, kept_ref = paged.evict(c.k0, c.v0, w, c.lens, c.table, budget, recent)
    assert np.array_equal(to_np(new), n_ref)
    assert np.array_equal(to_np(kept), kept_ref)
    assert np.array_equal(to_np(d["k"]), k) and np.array_equal(to_np(d["v"]), v)
    assert np.array_equal(to_np(d["w"]).view(np.uint32), ws.view(np.uint32))


# ---- together ------------------------------------------------------------------------------------
@pytest.mark.parametrize("D,bits,page,dtype", [(128, 3, 64, "bf16"), (64, 4, 16, "f16")])
def test_prompt_steps_eviction_and_more_steps(D, bits, page, dtype):
    """Chunks, decode steps, an eviction, more steps: every call against the definition on the caches as
    they then are."""
    H, G, B = 2, 2, 2
    c = Case(H, D, bits, page, [1] * B, [900] * B, seed=31, sums=True)
    d = c.d
    k, v = c.k0, c.v0
    lens = np.zeros(B, np.int32)
    for step, ns in enumerate([[200, 37], [130, 0], [1, 1], [1, 1], "evict", [1, 1], [5, 1]]):
        if ns == "evict":
            new, _ = rptq.rptq_kv_paged_evict(d["k"], d["v"], d["w"], d["lens"], d["table"], bits, 64, 20)
            k, v, w, new_ref, _ = paged.evict(k, v, c.w0, lens, c.table, 64, 20)
            assert np.array_equal(to_np(new), new_ref) and np.array_equal(to_np(d["k"]), k)
            assert np.array_equal(to_np(d["v"]), v) and np.array_equal(to_np(d["w"]), w)
            lens, c.w0 = new_ref, w
            continue
        lens = (lens + np.array(ns)).astype(np.int32)
        c.lens, c.start = lens, np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
        c.T, c.max_q, c.max_len = sum(ns), max(ns), int(lens.max())
        d["lens"], d["start"] = torch.from_numpy(lens).to(DEV), torch.from_numpy(c.start).to(DEV)
        kn, vn, q = c.tokens(c.mk, dtype), c.tokens(c.mv, dtype), c.queries(H * G, dtype)
        rptq.rptq_kv_paged_append(kn.to(DEV), vn.to(DEV), d["start"], d["lens"], d["table"], d["k"], d["v"], *d["kc"], *d["vc"],
                                  bits, weights=d["w"])
        k, c.w0 = paged.append(k, oracle._f32(kn), c.start, lens, c.table, *c.k_cal, bits, c.w0)
        v = paged.append(v, oracle._f32(vn), c.start, lens, c.table, *c.v_cal, bits)
        assert np.array_equal(to_np(d["k"]), k) and np.array_equal(to_np(d["v"]), v)
        out = c.attend(q.to(DEV))
        check_attention(c, q, out, dtype, weights=d["w"], k=k, v=v)
        c.w0 = to_np(d["w"]).copy()  # later steps are checked on the sums as they are


def test_captured_step_follows_the_tables():
    """One decode step captured as a graph and replayed with grown lengths; a chunk on another stream."""
    c = Case(4, 128, 3, 64, [1, 1, 1], [300, 64, 129], seed=32, sums=True)
    d = c.d
    kn, vn, q = (x.to(DEV) for x in (c.tokens(c.mk, "bf16"), c.tokens(c.mv, "bf16"), c.queries(8, "bf16")))
    out = torch.empty_like(q)
    c.max_len = c.table.shape[1] * 64  # a bound for every replay
    ws = torch.empty(max(16, rptq.rptq_kv_paged_attention_workspace_size(3, 8, 4, 128, torch.bfloat16, 3, 1, c.max_len, True)),
                     dtype=torch.uint8, device=DEV)

    def step():
        rptq.rptq_kv_paged_append(kn, vn, d["start"], d["lens"], d["table"], d["k"], d["v"], *d["kc"], *d["vc"], 3, weights=d["w"])
        c.attend(q, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    k, v = to_np(d["k"]), to_np(d["v"])
    for _ in range(3):
        c.lens = c.lens + 1
        d["lens"].add_(1)
        w0 = to_np(d["w"]).copy()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        k, c.w0 = paged.append(k, oracle._f32(kn.cpu()), c.start, c.lens, c.table, *c.k_cal, 3, w0)
        v = paged.append(v, oracle._f32(vn.cpu()), c.start, c.lens, c.table, *c.v_cal, 3)
        assert np.array_equal(to_np(d["k"]), k)
        check_attention(c, q.cpu(), out, "bf16", weights=d["w"], k=k, v=v)


@pytest.mark.parametrize("n", [1, 150])
def test_calls_on_other_streams(n):
    """Two problems on two streams at once, each with its own workspace and outputs from the binding, while the current stream
    reuses what the allocator hands it; results equal the ones alone."""
    cs = [Case(4, 128, 3, 64, [n, n], [900, 700], seed=33 + i, sums=True) for i in range(2)]
    qs = [c.queries(8, "bf16").to(DEV) for c in cs]
    alone, sums = [], []
    for c, q in zip(cs, qs):
        alone.append(c.attend(q).clone())
        sums.append(c.d["w"].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for turn in range(5):
        for c in cs:
            c.d["w"].copy_(torch.from_numpy(c.w0))
        torch.cuda.synchronize()
        outs = []
        for c, q, s in zip(cs, qs, streams):
            outs.append(c.attend(q, stream=s))  # the current stream stays what it is
            for _ in range(3):
                torch.full((1 << 20,), float(turn), device=DEV)
        torch.cuda.synchronize()
        for i, c in enumerate(cs):
            assert torch.equal(outs[i], alone[i]) and torch.equal(c.d["w"], sums[i])


def test_two_graphs_share_a_workspace_in_turn():
    """A decode step and a chunk captured apart with one workspace between them, replayed in turn on one stream."""
    c = Case(2, 128, 4, 16, [1, 1], [500, 333], seed=35, sums=True)
    k = Case(2, 128, 4, 16, [140, 3], [500, 333], seed=35, sums=True)
    ws = torch.empty(max(rptq.rptq_kv_paged_attention_workspace_size(x.T, 4, 2, 128, torch.float16, 2, x.max_q, x.max_len, True)
                         for x in (c, k)), dtype=torch.uint8, device=DEV)
    graphs = []
    for x in (c, k):
        q = x.queries(4, "f16").to(DEV)
        want = x.attend(q).clone()
        sums = x.d["w"].clone()
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.attend(q, out=out, workspace=ws)
        graphs.append((x, g, out, want, sums, q))  # q stays alive: the graph reads it
    for _ in range(3):
        for x, g, out, want, sums, _ in graphs:
            x.d["w"].copy_(torch.from_numpy(x.w0))
            out.zero_()
            ws.fill_(0xA5)  # garbage: nothing of the last call may be counted on
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(x.d["w"], sums)


# ---- what only the device can see ------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 140])
def test_bad_tables_are_reported_and_left_out(n):
    """Sequence 1 is too long, sequence 2's rows run backwards, sequence 3 has a page id outside the pool."""
    c = Case(2, 64, 3, 16, [n, 1, 1, 1, 1], [200, 40, 40, 40, 30], seed=41, sums=True)
    d = c.d
    lens, start, table = c.lens.copy(), c.start.copy(), c.table.copy()
    bad = lens.copy()
    bad[1] = 10 ** 6
    d["lens"].copy_(torch.from_numpy(bad))
    q = c.queries(2, "bf16").to(DEV)
    ref = c.attend(q, out=torch.full_like(q, 7))
    assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_RANGE
    assert (ref[n] == 7).all() and not (ref[n + 1:] == 7).all(dim=(1, 2)).any()
    d["lens"].copy_(torch.from_numpy(lens))
    for broken in ([0, n + 5, n + 1, n + 3, n + 4, n + 4], [0, n, -4, n + 2, n + 3, n + 4], [0, n, n + 1, n + 9, n + 3, n + 4]):
        d["start"].copy_(torch.tensor(broken, dtype=torch.int32))
        c.attend(q)
        assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_RANGE
        k = d["k"].clone()
        rptq.rptq_kv_paged_append(q, q, d["start"], d["lens"], d["table"], d["k"], d["v"], *d["kc"], *d["vc"], 3)
        rptq.rptq_kv_paged_dequant(d["k"], d["table"], d["start"], d["lens"] * 0, *d["kc"], 3, T=c.T)
        rptq.rptq_device_error()
        d["k"].copy_(k)
    d["start"].copy_(torch.from_numpy(start))
    for value in (-1, 10 ** 8):
        t = table.copy()
        t[3, 1] = value
        d["table"].copy_(torch.from_numpy(t))
        k0, v0, w0 = (d[x].clone() for x in "kvw")
        c.attend(q)
        assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_PAGE
        d["w"].copy_(w0)
        rptq.rptq_kv_paged_dequant(d["k"], d["table"], d["start"], d["lens"] * 0 + 20, *d["kc"], 3, T=c.T)
        assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_PAGE
        new, kept = rptq.rptq_kv_paged_evict(d["k"], d["v"], d["w"], d["lens"], d["table"], 3, 20, 3)
        assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_PAGE
        assert new.tolist() == [20, 20, 20, 40, 20] and (kept[3] == -1).all() and (kept[0] >= 0).all()
        pg = torch.from_numpy(table[3]).long().to(DEV)
        assert all(torch.equal(d[x][pg], y[pg]) for x, y in zip("kvw", (k0, v0, w0)))
        for x, y in zip("kvw", (k0, v0, w0)):
            d[x].copy_(y)
    d["table"].copy_(torch.from_numpy(table))
    d["lens"][0] = -3
    new, kept = rptq.rptq_kv_paged_evict(d["k"], d["v"], d["w"], d["lens"], d["table"], 3, 20, 3)
    assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_RANGE
    assert new.tolist() == [-3, 20, 20, 20, 20] and (kept[0] == -1).all()


def test_a_cluster_id_out_of_range_is_reported():
    c = Case(2, 128, 3, 16, [1, 130], [20, 130], seed=42)
    c.d["kc"][0][5] = 99
    c.attend(c.queries(2, "f16").to(DEV))
    assert rptq.rptq_device_error() == rptq.RPTQ_DEVERR_CLUSTER_ID


def test_binding_refuses_wrong_tensors():
    c = Case(2, 64, 3, 16, [1], [20], seed=43, sums=True)
    d = c.d
    q = c.queries(2, "bf16").to(DEV)
    args = lambda **k: ([k.get("q", q)] + [k.get(x, d[x]) for x in ("start", "lens", "table", "k", "v")] + d["kc"] + d["vc"] + [3])  # noqa: E731
    kw = dict(max_q=1, max_len=20)
    rptq.rptq_kv_paged_attention(*args(), **kw)
    for bad in (dict(q=q.cpu()), dict(q=q.to(torch.float64)), dict(q=q[:, :, :32]), dict(start=d["start"].long()),
                dict(lens=d["lens"][:0]), dict(table=d["table"].cpu()), dict(k=d["k"][:, :1]), dict(v=d["v"].to(torch.int8)),
                dict(q=q.transpose(0, 1)[:1]), dict(k=d["k"].transpose(0, 1))):
        with pytest.raises(rptq.RptqError):
            rptq.rptq_kv_paged_attention(*args(**bad), **kw)
    for bad in (dict(out=torch.empty_like(q, dtype=torch.float32)), dict(weights=d["w"][:1]), dict(weights=d["w"].half()),
                dict(weights=d["w"], workspace=torch.empty(1, dtype=torch.uint8, device=DEV))):
        with pytest.raises(rptq.RptqError):
            rptq.rptq_kv_paged_attention(*args(), **kw, **bad)
    with pytest.raises(rptq.RptqError):
        rptq.rptq_kv_paged_evict(d["k"], d["v"], d["w"], d["lens"], d["table"], 3, 8, new_lens=d["lens"])
