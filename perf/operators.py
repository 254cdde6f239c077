"""The paged packed K/V cache as it is measured: cases, inputs, plain forms and what each pass has to move.

Four operators over one cache whose positions live in pages of packed 3- or 4-bit codes, each channel
quantized with the scale and zero point of its cluster:

  append   new tokens' K and V quantized into the pages at the end of their sequences;
  attend   causal softmax attention of each sequence's newest tokens (one, or a chunk) over all its
           positions, with or without adding every position's attention weight to its running sum;
  evict    every head keeps its most recent positions and those of the largest running sums, moved
           together to the front of the sequence's pages;
  dequant  positions read back as dense values.

What a pass holds in 3 or 4 bits is returned as the values it stands for (the read-back is a part of the
pass on both sides).  With `own` false `run` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's append of a full serving batch (the 32-head 3-bit cache)
        dict(name="append step 64x32", op="append", B=64, n=1, n_spread=0, L=2048, spread=1900, H=32, Hq=32, D=128,
             bits=3, page=64, dtype="f16"),
        # prompts of unequal length admitted together into the 96-head cache
        dict(name="append prompts 96h", op="append", B=9, n=1100, n_spread=371, L=1300, spread=200, H=96, Hq=96, D=128,
             bits=3, page=64, dtype="bf16"),
        # the smallest call: one token of one short sequence, the 12-head model in fp32
        dict(name="decode 1x12", op="attend", B=1, n=1, n_spread=0, L=509, spread=0, H=12, Hq=12, D=64, bits=4,
             page=16, dtype="f32", weights=False),
        # a decode step over the 32-head 3-bit cache at 2048 positions
        dict(name="decode 16x32", op="attend", B=16, n=1, n_spread=0, L=2048, spread=0, H=32, Hq=32, D=128, bits=3,
             page=64, dtype="f16", weights=False),
        # a decode step of unequal sequences over the 96-head cache, keeping the running weights for eviction
        dict(name="decode 8x96 weights", op="attend", B=8, n=1, n_spread=0, L=2047, spread=900, H=96, Hq=96, D=128,
             bits=3, page=64, dtype="bf16", weights=True),
        # long contexts, four query heads to a K/V head, two sequences
        dict(name="decode long grouped", op="attend", B=2, n=1, n_spread=0, L=131001, spread=40000, H=8, Hq=32, D=128,
             bits=4, page=128, dtype="bf16", weights=False),
        # a chunk of prompt tokens behind what the cache holds already, unequal sequences
        dict(name="chunk 2048 32h", op="attend", B=3, n=2048, n_spread=700, L=5999, spread=2500, H=32, Hq=32, D=128,
             bits=3, page=64, dtype="f16", weights=False),
        # a chunk over grouped heads that also keeps the running weights
        dict(name="chunk 1024 weights", op="attend", B=2, n=1024, n_spread=90, L=8100, spread=1111, H=8, Hq=32, D=128,
             bits=4, page=32, dtype="bf16", weights=True),
        # a full batch cut back to half its positions
        dict(name="evict 16x32", op="evict", B=16, L=2048, spread=500, H=32, D=128, bits=3, page=64, dtype="f16",
             budget=1024, recent=256),
        # one long context cut to an eighth
        dict(name="evict long 8h", op="evict", B=1, L=32700, spread=0, H=8, D=128, bits=4, page=128, dtype="bf16",
             budget=4096, recent=511),
        # a short window of a small model read back in fp32
        dict(name="dequant window", op="dequant", B=5, n=77, n_spread=20, L=509, spread=200, H=12, D=64, bits=4,
             page=16, dtype="f32"),
        # whole sequences of the 96-head cache read back
        dict(name="dequant whole 96h", op="dequant", B=8, n=2048, n_spread=300, L=2048, spread=0, H=96, D=128, bits=3,
             page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict", "dequant"])
    c = dict(op=op, D=rng.choice([64, 128, 128]), bits=rng.choice([3, 4]), page=rng.choice([16, 32, 64, 128]),
             dtype=rng.choice(["f16", "bf16", "bf16", "f32"]))
    H = rng.choice([4, 8, 12, 16, 32, 40])
    if op == "append":
        T = _log(rng, 1, 8000)
        B = min(T, _log(rng, 1, 64))
        n = -(-T // B)
        c.update(B=B, n=n, n_spread=rng.randrange(n), L=n + _log(rng, 1, 2000), spread=0, H=H, Hq=H)
        c["spread"] = rng.randrange(c["L"] - n + 1)
        return c
    if op == "attend":
        group = rng.choice([1, 1, 2, 4, 8]) if H <= 16 else 1
        if rng.random() < 0.6:  # a decode step, or a few tokens of each sequence
            B, n = _log(rng, 1, 24), rng.choice([1, 1, 1, 2, 3, 5])
            L = _log(rng, 40, max(80, min(100000, 2_500_000 // (B * H))))
        else:
            B, n = rng.randrange(1, 4), _log(rng, 17, 1500)
            L = n + _log(rng, 1, 5000)
        L = max(L, n)
        c.update(B=B, n=n, n_spread=rng.randrange(n), L=L, spread=rng.randrange(L - n + 1), H=H, Hq=H * group,
                 weights=rng.random() < 0.4)
        return c
    L = _log(rng, 60, 4000) if op == "dequant" else _log(rng, 60, 20000)
    B = max(1, min(16, _log(rng, 1, 16), 400_000 // (L * H)))
    c.update(B=B, L=L, spread=rng.randrange(L // 2), H=H)
    if op == "evict":
        c["budget"] = max(2, int(L * rng.uniform(0.1, 0.9)))
        c["recent"] = rng.randrange(c["budget"])
    else:
        c["n"] = rng.randrange(1, L + 1)
        c["n_spread"] = rng.randrange(c["n"])
    return c


def _lengths(case):
    """(positions, new or read positions) of each sequence: the case's own raggedness, no seed in it."""
    lens = [case["L"] - (7919 * b) % (case["spread"] + 1) for b in range(case["B"])]
    n = [case.get("n", 0) - (104729 * b) % (case.get("n_spread", 0) + 1) for b in range(case["B"])]
    return lens, [min(x, y) for x, y in zip(n, lens)]


# ---- inputs --------------------------------------------------------------------------------------

def _model(C, qmax, gen):
    """Channel ranges as OPT-like activations have them (centre ~ N(0, 2), half width ~ LogNormal(0, 1), one channel in a
    hundred a hundred times larger) and the clusters' parameters: channels of like range together."""
    dev = "cuda"
    centre = 2.0 * torch.randn(C, generator=gen, device=dev)
    hw = torch.randn(C, generator=gen, device=dev).exp()
    big = torch.rand(C, generator=gen, device=dev) < 0.01
    factor = torch.where(big, 100.0, 1.0)
    centre, hw = centre * factor, hw * factor
    g = min(32, C)
    order = torch.argsort(centre + hw)
    labels = torch.empty(C, dtype=torch.int64, device=dev)
    labels[order] = torch.arange(C, device=dev) * g // C
    hi = torch.full((g,), -torch.inf, device=dev).scatter_reduce(0, labels, centre + hw, "amax")
    lo = torch.full((g,), torch.inf, device=dev).scatter_reduce(0, labels, centre - hw, "amin")
    scale = (hi - lo) / qmax
    zero = torch.round(-lo / scale).to(torch.int32)
    return dict(centre=centre, hw=hw, labels=labels.to(torch.int32), scale=scale, zero=zero)


def _draw_values(shape, m, gen):
    """[..., H, D] values of the model's channels."""
    u = torch.rand(shape, generator=gen, device="cuda") * 2.0 - 1.0
    C = shape[-2] * shape[-1]
    return (m["centre"] + m["hw"] * u.reshape(-1, C)).reshape(shape)


def _pool(n_pages, page, H, D, bits, m, gen):
    """Pages [n_pages, H, page, D * bits / 8] of the model's quantized values."""
    out = torch.empty((n_pages, H, page, D * bits // 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (page * H * D))
    for p in range(0, n_pages, step):
        k = min(step, n_pages - p)
        x = _draw_values((k, page, H, D), m, gen)
        out[p:p + k] = _pack(_codes(x, m, bits), bits).permute(0, 2, 1, 3)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, B, H, D, bits, page = (case[k] for k in ("op", "B", "H", "D", "bits", "page"))
    dt = _DT[case["dtype"]]
    lens, n = _lengths(case)
    max_pages = -(-max(lens) // page) + 1
    n_pages = B * max_pages + 3
    mk, mv = _model(H * D, 2 ** bits - 1, gen), _model(H * D, 2 ** bits - 1, gen)
    st = dict(case=case, mk=mk, mv=mv, dtype=dt, bits=bits, page=page, D=D, max_len=max(lens), max_q=max(n),
              table=torch.randperm(n_pages, generator=gen, device="cuda")[:B * max_pages].reshape(B, max_pages).to(torch.int32),
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              start=torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda"),
              k_pages=_pool(n_pages, page, H, D, bits, mk, gen), v_pages=_pool(n_pages, page, H, D, bits, mv, gen))
    T = sum(n)
    st["T"] = T
    if op == "append":
        # the K and V parts of a fused projection's output: rows of (Hq + 2 H) heads
        qkv = torch.empty((T, case["Hq"] + 2 * H, D), dtype=dt, device="cuda")
        qkv[:, -2 * H:-H] = _draw_values((T, H, D), mk, gen).to(dt)
        qkv[:, -H:] = _draw_values((T, H, D), mv, gen).to(dt)
        st["k"], st["v"] = qkv[:, -2 * H:-H], qkv[:, -H:]
        st["begin"] = st["lens"] - torch.tensor(n, dtype=torch.int32, device="cuda")
    if op == "attend":
        Hq = case["Hq"]
        # each channel carries a like share of a score, whatever its range, as in a trained model
        hw = mk["hw"].reshape(H, 1, D).expand(H, Hq // H, D).reshape(Hq, D)
        st["q"] = (torch.randn((T, Hq, D), generator=gen, device="cuda") * 3.0 / hw).to(dt)
    if op == "dequant":
        st["begin"] = st["lens"] - torch.tensor(n, dtype=torch.int32, device="cuda")
    if case.get("weights") or op == "evict":
        # running sums of attention weights: few large ones, many near zero, some exactly equal
        w = torch.rand((n_pages, H, page), generator=gen, device="cuda")
        w = w ** 8 * 20.0
        st["weights"] = torch.where(w < 0.01, torch.zeros_like(w), torch.round(w * 4096.0) / 4096.0)
    if op == "evict":
        kept = [min(x, case["budget"]) for x in lens]
        st["budget"], st["recent"] = case["budget"], case["recent"]
        st["kept_T"] = sum(kept)
        st["kept_start"] = torch.tensor([0] + list(np.cumsum(kept)), dtype=torch.int32, device="cuda")
        st["kept_begin"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


def work(case):
    lens, n = _lengths(case)
    H, D, bits = case["H"], case["D"], case["bits"]
    es = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    T, row = sum(n), H * D * bits / 8  # row: one position's codes of K or of V
    val = H * D * es
    if case["op"] == "append":
        return {"bytes": 2 * T * (val + row) + 2 * T * (row + val), "flops": 0}  # quantize; read back
    if case["op"] == "dequant":
        return {"bytes": 2 * T * (row + val), "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(x, case["budget"]) for x in lens)
        moved = sum(min(x, case["budget"]) for x in lens if x > case["budget"])
        # the sums read, the kept rows and sums read and written, what stayed read back
        return {"bytes": 4 * H * sum(lens) + moved * (4 * row + 4 * H) + 2 * kept * (row + val), "flops": 0}
    Hq = case["Hq"]
    pairs = sum(k * x - k * (k - 1) // 2 for k, x in zip(n, lens))
    by = 2 * T * Hq * D * es + sum(2 * x * row for x, k in zip(lens, n) if k)
    if case["weights"]:
        by += 8 * H * sum(x for x, k in zip(lens, n) if k)
    return {"bytes": by, "flops": 4 * pairs * Hq * D}


# ---- plain forms -----------------------------------------------------------------------------------

def _per_channel(m):
    k = m["labels"].long()
    return m["scale"][k], m["zero"][k]


def _codes(x, m, bits):
    """clamp(rint(x / s) + z, 0, qmax) of [..., H, D], in 32 bits."""
    s, z = _per_channel(m)
    H, D = x.shape[-2:]
    q = torch.round(x.float() / s.reshape(H, D)) + z.reshape(H, D)
    return q.clamp(0, 2 ** bits - 1).to(torch.int32)


def _pack(q, bits):
    """Codes [..., D] -> bytes [..., D * bits / 8]: 4-bit low nibble first, 3-bit eight to a 24-bit little-endian word."""
    if bits == 4:
        return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8)
    e = q.reshape(*q.shape[:-1], -1, 8)
    w = (e << (3 * torch.arange(8, device=q.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    return torch.stack((w & 255, (w >> 8) & 255, w >> 16), -1).reshape(*q.shape[:-1], -1).to(torch.uint8)


def _unpack(b, bits):
    b = b.to(torch.int32)
    if bits == 4:
        return torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)
    e = b.reshape(*b.shape[:-1], -1, 3)
    w = e[..., 0] | (e[..., 1] << 8) | (e[..., 2] << 16)
    return ((w.unsqueeze(-1) >> (3 * torch.arange(8, device=b.device, dtype=torch.int32))) & 7).reshape(*b.shape[:-1], -1)


def _tokens(st, start, T):
    """(sequence, index in it) of every row of a ragged batch."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start.long(), t, right=True) - 1
    return b, t - start.long()[b]


def _slots(st, b, pos):
    """(page, slot) of position pos of sequence b."""
    return st["table"].long()[b, pos // st["page"]], pos % st["page"]


def _read(st, pages, m, start, begin, T):
    b, i = _tokens(st, start, T)
    p, s = _slots(st, b, begin.long()[b] + i)
    q = _unpack(pages[p, :, s], st["bits"])
    sc, z = _per_channel(m)
    H, D = q.shape[-2:]
    return ((q - z.reshape(H, D)).float() * sc.reshape(H, D)).to(st["dtype"])


def _dense(st, pages):
    """[B, H, max_len, bytes or nothing more] of every sequence's positions in order."""
    B, mp = st["table"].shape
    x = pages[st["table"].long()]  # [B, mp, H, page, ...]
    x = x.transpose(1, 2)
    return x.reshape(B, x.shape[1], mp * st["page"], *x.shape[4:])[:, :, :st["max_len"]]


def _plain_append(st):
    b, i = _tokens(st, st["start"], st["T"])
    p, s = _slots(st, b, st["begin"].long()[b] + i)
    st["k_pages"][p, :, s] = _pack(_codes(st["k"], st["mk"], st["bits"]), st["bits"])
    st["v_pages"][p, :, s] = _pack(_codes(st["v"], st["mv"], st["bits"]), st["bits"])
    return [_read(st, st["k_pages"], st["mk"], st["start"], st["begin"], st["T"]),
            _read(st, st["v_pages"], st["mv"], st["start"], st["begin"], st["T"])]


def _values(st, pages, m):
    q = _unpack(_dense(st, pages), st["bits"])
    s, z = _per_channel(m)
    B, H, L, D = q.shape
    return (q - z.reshape(H, 1, D)).float() * s.reshape(H, 1, D)


def _plain_attend(st):
    c = st["case"]
    H, Hq, D, N = c["H"], c["Hq"], c["D"], st["max_q"]
    G, L, B = Hq // H, st["max_len"], c["B"]
    b, i = _tokens(st, st["start"], st["T"])
    q = torch.zeros((B, N, Hq, D), device="cuda")
    q[b, i] = st["q"].float()
    q = q.reshape(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    x = torch.matmul(q, _values(st, st["k_pages"], st["mk"]).transpose(2, 3)).reshape(B, H, G, N, L)
    x *= 1.0 / math.sqrt(D)
    n = (st["start"][1:] - st["start"][:-1]).long()
    row = torch.arange(N, device="cuda")
    limit = st["lens"].long()[:, None] - n[:, None] + row  # the last position that row sees
    seen = (torch.arange(L, device="cuda") <= limit[..., None]) & (row < n[:, None])[..., None]
    x.masked_fill_(~seen[:, None, None], -torch.inf)
    x -= x.amax(-1, keepdim=True).clamp_min(-3e38)
    x.exp_()
    x /= x.sum(-1, keepdim=True).clamp_min(1e-30)
    out = torch.matmul(x.reshape(B, H, G * N, L), _values(st, st["v_pages"], st["mv"]))
    out = out.reshape(B, H, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[b, i].to(st["dtype"])
    if not c["weights"]:
        return [out]
    w = x.sum((2, 3))  # [B, H, L]
    pos = torch.arange(L, device="cuda")
    held = (pos < st["lens"][:, None]).nonzero()
    p, s = _slots(st, held[:, 0], held[:, 1])
    st["weights"][p, :, s] += w[held[:, 0], :, held[:, 1]]
    return [out, st["weights"]]


def _plain_evict(st):
    budget, recent, L = st["budget"], st["recent"], st["max_len"]
    lens = st["lens"].long()
    w = _dense(st, st["weights"])  # [B, H, L]
    B, H = w.shape[:2]
    pos = torch.arange(L, device="cuda")
    new = lens.clamp_max(budget)
    if L <= budget:
        w = torch.nn.functional.pad(w, (0, budget - L + 1))
        pos = torch.arange(budget + 1, device="cuda")
    key = torch.where(pos >= (lens[:, None] - recent), torch.inf, w.transpose(0, 1)).transpose(0, 1)
    key = torch.where((pos < lens[:, None])[:, None], key, -torch.inf)
    kept = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.sort(kept, dim=-1).values
    j = torch.arange(budget, device="cuda")
    whole = (lens <= budget)[:, None, None]
    kept = torch.where(whole, j, kept)
    live = (j < new[:, None])[:, None]
    kept = torch.where(live, kept, -1)
    move = (live & ~whole).expand(B, H, budget).nonzero()
    b, h, to = move[:, 0], move[:, 1], move[:, 2]
    p, s = _slots(st, b, kept[b, h, to])
    p2, s2 = _slots(st, b, to)
    for x in (st["k_pages"], st["v_pages"], st["weights"]):
        x[p2, h, s2] = x[p, h, s]
    a = (st["kept_start"], st["kept_begin"], st["kept_T"])
    return [new.to(torch.int32), kept.to(torch.int32), st["weights"], _read(st, st["k_pages"], st["mk"], *a),
            _read(st, st["v_pages"], st["mv"], *a)]


# ---- the framework's calls -------------------------------------------------------------------------

def _cal(m):
    return m["labels"], m["scale"], m["zero"]


def _own(st):
    from post_activation_quantization_b200 import rptq
    op, mk, mv, bits = st["case"]["op"], _cal(st["mk"]), _cal(st["mv"]), st["bits"]

    def read(pages, m, start, begin, T):
        return rptq.rptq_kv_paged_dequant(pages, st["table"], start, begin, *m, bits, T=T, out_dtype=st["dtype"])

    if op == "append":
        rptq.rptq_kv_paged_append(st["k"], st["v"], st["start"], st["lens"], st["table"], st["k_pages"], st["v_pages"],
                                  *mk, *mv, bits)
        return [read(st["k_pages"], mk, st["start"], st["begin"], st["T"]),
                read(st["v_pages"], mv, st["start"], st["begin"], st["T"])]
    if op == "attend":
        out = rptq.rptq_kv_paged_attention(st["q"], st["start"], st["lens"], st["table"], st["k_pages"], st["v_pages"],
                                           *mk, *mv, bits, max_q=st["max_q"], max_len=st["max_len"],
                                           weights=st.get("weights"))
        return [out] + ([st["weights"]] if "weights" in st else [])
    if op == "evict":
        new, kept = rptq.rptq_kv_paged_evict(st["k_pages"], st["v_pages"], st["weights"], st["lens"], st["table"], bits,
                                             budget=st["budget"], recent=st["recent"], max_len=st["max_len"])
        a = (st["kept_start"], st["kept_begin"], st["kept_T"])
        return [new, kept, st["weights"], read(st["k_pages"], mk, *a), read(st["v_pages"], mv, *a)]
    return [read(st["k_pages"], mk, st["start"], st["begin"], st["T"]),
            read(st["v_pages"], mv, st["start"], st["begin"], st["T"])]


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "append":
        return _plain_append(st)
    if op == "attend":
        return _plain_attend(st)
    if op == "evict":
        return _plain_evict(st)
    a = (st["start"], st["begin"], st["T"])
    return [_read(st, st["k_pages"], st["mk"], *a), _read(st, st["v_pages"], st["mv"], *a)]


# ---- the definition in 64 bits -----------------------------------------------------------------------

def _bits_of(rows, bits):
    """Codes of packed rows [..., bytes] as doubles: the bytes' bits in order, `bits` of them to a code."""
    x = (rows.unsqueeze(-1) >> torch.arange(8, device=rows.device, dtype=torch.uint8)) & 1
    x = x.reshape(*rows.shape[:-1], -1, bits)
    v = x[..., 0].double()
    for k in range(1, bits):
        v += x[..., k].double() * 2.0 ** k
    return v


def _sequence(st, pages, b, n, h=None):
    """Rows [n, H, bytes] (or [n, bytes] of one head) of the first n positions of sequence b."""
    ids = st["table"][b, :-(-n // st["page"])].long()
    if h is None:
        return pages[ids].transpose(1, 2).reshape(-1, pages.shape[1], pages.shape[3])[:n]
    return pages[ids, h].reshape(-1, pages.shape[3])[:n]


def _value64(rows, m, bits, h=None):
    s, z = m["scale"].double()[m["labels"].long()], m["zero"].double()[m["labels"].long()]
    v = _bits_of(rows, bits)
    D = v.shape[-1]
    s, z = s.reshape(-1, D), z.reshape(-1, D)
    return (v - (z if h is None else z[h])) * (s if h is None else s[h])


def _rows64(st, pages, m, first, count):
    out = [_value64(_sequence(st, pages, b, f + k)[f:], m, st["bits"]) for b, (f, k) in enumerate(zip(first, count))]
    return torch.cat(out)


def exact(case, seed):
    st = prepare(case, seed)
    lens, n = _lengths(case)
    H, D, bits, op = case["H"], case["D"], case["bits"], case["op"]
    if op == "dequant":
        first = [x - k for x, k in zip(lens, n)]
        return [_rows64(st, st["k_pages"], st["mk"], first, n), _rows64(st, st["v_pages"], st["mv"], first, n)]
    if op == "append":
        got = []
        for x, m in ((st["k"], st["mk"]), (st["v"], st["mv"])):
            s, z = m["scale"][m["labels"].long()].reshape(H, D), m["zero"].double()[m["labels"].long()].reshape(H, D)
            # the quotient is the 32-bit one by definition: round(x / s) of exact halves hangs on it
            q = torch.clamp(torch.round((x.float() / s).double()) + z, 0.0, 2.0 ** bits - 1.0)
            got.append((q - z) * s.double())
        return got
    if op == "evict":
        w = st["weights"].double().cpu().numpy()
        table = st["table"].cpu().numpy()
        P, budget, recent = st["page"], case["budget"], case["recent"]
        new_w, ks, vs = w.copy(), [], []
        for b, L in enumerate(lens):
            keep = np.tile(np.arange(min(L, budget)), (H, 1))
            at = table[b][np.arange(L) // P], np.arange(L) % P
            if L > budget:
                for h in range(H):
                    old = w[at[0][:L - recent], h, at[1][:L - recent]]
                    best = np.lexsort((np.arange(old.size), -old))[:budget - recent]
                    keep[h] = np.concatenate((np.sort(best), np.arange(L - recent, L)))
                    j = np.arange(budget)
                    new_w[table[b][j // P], h, j % P] = w[at[0][keep[h]], h, at[1][keep[h]]]
            k = torch.from_numpy(keep.T.copy()).cuda()  # [kept, H]
            hh = torch.arange(H, device="cuda")
            ks.append(_value64(_sequence(st, st["k_pages"], b, L)[k, hh], st["mk"], bits))
            vs.append(_value64(_sequence(st, st["v_pages"], b, L)[k, hh], st["mv"], bits))
        return [None, None, torch.from_numpy(new_w), torch.cat(ks), torch.cat(vs)]
    Hq = case["Hq"]
    G = Hq // H
    out = torch.empty((st["T"], Hq, D), dtype=torch.float64, device="cuda")
    w = st["weights"].double() if case["weights"] else None
    t0 = 0
    for b, (L, k) in enumerate(zip(lens, n)):
        if k:
            pos = torch.arange(L, device="cuda")
            hidden = pos[None, :] > (L - k + torch.arange(k, device="cuda"))[:, None]
            ids, slot = st["table"][b].long()[pos // st["page"]], pos % st["page"]
            for h in range(H):
                kk = _value64(_sequence(st, st["k_pages"], b, L, h), st["mk"], bits, h)
                vv = _value64(_sequence(st, st["v_pages"], b, L, h), st["mv"], bits, h)
                for a in range(h * G, (h + 1) * G):
                    x = st["q"][t0:t0 + k, a].double() @ kk.T / math.sqrt(D)
                    p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                    out[t0:t0 + k, a] = p @ vv
                    if w is not None:
                        w[ids, h, slot] += p.sum(0)
        t0 += k
    return [out] if w is None else [out, w]
