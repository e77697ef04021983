"""What is measured of the serving operators on the packed KV cache.

Six operators: decode attention and chunked prefill attention under a sliding
window with sink tokens, decode attention of a batch that shares a prefix,
block tables and slot maps from request lengths, the append of new tokens into
cache pages, and decode attention over those pages.

Packed rows: d codes of `bits` bits of the rotated unit vector, in the
library's layout, and a float16 norm.  The plain forms below work in the
rotated domain with elementary torch operations in float32 (the compressor's
threshold decisions in float64); `exact` reconstructs K and V in the original
domain in float64 and attends there.
"""

import math
import random

import numpy as np
import torch

own = False

F16, F32 = "float16", "float32"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(op, **kw):
    c = {"op": op, "dtype": F16, "bits": 3, "variant": 0, "lens": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one request of a local-attention layer late in a long context: latency
        _case("window_decode", name="window_decode_one", B=1, Hq=32, Hkv=4, d=128, T=32768, W=1024, S=4),
        # a full serving batch of ragged requests, wide heads
        _case("window_decode", name="window_decode_batch", B=32, Hq=16, Hkv=8, d=256, T=16384, W=4096, S=16, lens=1),
        # one prompt chunk of an interactive request
        _case("window_prefill", name="window_prefill_chunk", B=1, Tq=256, Hq=32, Hkv=4, d=128, T=4096, W=1024, S=4),
        # two long prompts, chunked by 2048
        _case("window_prefill", name="window_prefill_long", B=2, Tq=2048, Hq=32, Hkv=4, d=128, T=8192, W=2048, S=16,
              lens=2),
        # four samples drawn from one prompt
        _case("prefix_decode", name="prefix_decode_few", B=4, Hq=32, Hkv=4, d=128, Tp=4096, T=128, lens=3),
        # many requests behind one long document
        _case("prefix_decode", name="prefix_decode_many", B=64, Hq=32, Hkv=4, d=128, Tp=65536, T=512, lens=4),
        # a decode step: one new token a request
        _case("block_tables", name="block_tables_step", B=64, P=64, T=8192, new=1, lens=5),
        # a mixed step: prompt chunks and single tokens of many requests
        _case("block_tables", name="block_tables_mixed", B=512, P=16, T=4096, new=256, lens=6),
        # the new tokens of a decode step, the widest codes, float32 activations
        _case("paged_append", name="paged_append_step", N=32, Hkv=8, d=256, P=64, bits=4, dtype=F32, lens=7),
        # a prompt's tokens, scattered over pages
        _case("paged_append", name="paged_append_prompt", N=8191, Hkv=4, d=128, P=64, lens=8),
        # small pages, float32 queries, 4-bit codes
        _case("paged_decode", name="paged_decode_ragged", B=16, Hq=32, Hkv=4, d=128, P=16, T=8192, W=0, S=0, bits=4,
              dtype=F32, lens=9),
        # a long-context serving batch
        _case("paged_decode", name="paged_decode_long", B=16, Hq=16, Hkv=8, d=256, P=64, T=16384, W=0, S=0, lens=10),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm, as often odd as it falls."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_decode", "window_prefill", "prefix_decode", "block_tables", "paged_append",
                     "paged_decode"])
    half = rng.random() < 0.7
    c = _case(op, lens=rng.randrange(1 << 20), variant=rng.choice([0, 0, 1]), dtype=F16 if half else F32,
              bits=rng.choice([3, 3, 3, 2, 4]) if half else rng.choice([2, 3, 4]), d=rng.choice([128, 128, 256]))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 3])
    if op in ("window_decode", "paged_decode"):
        T = _log_int(rng, 1, 16384)
        c.update(B=_log_int(rng, 1, 32), Hkv=Hkv, Hq=Hkv * min(G, 4), T=T, W=_log_int(rng, 1, 4096),
                 S=rng.choice([0, 1, 4, 64, 130]))
        if op == "paged_decode":
            c.update(P=rng.choice([16, 32, 64, 128]), B=_log_int(rng, 1, 16))
            if rng.random() < 0.5:
                c.update(W=0, S=0)     # no window
    elif op == "window_prefill":
        c.update(B=rng.choice([1, 2]), Hkv=rng.choice([1, 2, 4]), Tq=_log_int(rng, 1, 1024), bits=3, dtype=F16,
                 W=_log_int(rng, 1, 2048), S=rng.choice([0, 1, 4, 64, 130]))
        c.update(Hq=c["Hkv"] * rng.choice([1, 2, 4, 8]), T=max(c["Tq"], _log_int(rng, 1, 8192)))
    elif op == "prefix_decode":
        c.update(B=_log_int(rng, 1, 64), Hkv=min(Hkv, 4), Tp=_log_int(rng, 1, 32768), T=_log_int(rng, 1, 512))
        c.update(Hq=c["Hkv"] * G)
    elif op == "block_tables":
        c.update(B=_log_int(rng, 1, 512), P=rng.choice([16, 32, 64, 128]), T=_log_int(rng, 1, 8192),
                 new=_log_int(rng, 1, 256))
    else:
        c.update(N=_log_int(rng, 1, 4096), Hkv=Hkv, P=rng.choice([16, 32, 64, 128]))
    return c


def _up(n, m):
    return (n + m - 1) // m * m


def _lens(c):
    """Tokens a row holds: a listed case's or a drawn one's own, the same for every seed."""
    r = random.Random(c["lens"])
    B, T = c["B"], c["T"]
    if c["op"] == "window_prefill":
        return [r.randint(c["Tq"], T) if c["lens"] else T for _ in range(B)]
    if c["op"] == "block_tables":
        return [r.randint(0, T) for _ in range(B)]
    return [r.randint(max(1, T // 2), T) if c["lens"] else T for _ in range(B)]


def _new_lens(c):
    r = random.Random(c["lens"] + 1)
    if c["new"] == 1:
        return [1] * c["B"]
    return [r.choice([0, 1, r.randint(1, c["new"]), c["new"]]) for _ in range(c["B"])]


def _spans(c):
    """(tokens a decode query of each row sees) of a window_decode or paged_decode case."""
    W, S = c["W"], c["S"]
    if c["op"] == "paged_decode" and W == 0:
        return _lens(c)
    return [t - max(0, max(S, t - W) - min(S, t)) if t > S else t for t in _lens(c)]


def work(case):
    c = case
    e = 2 if c["dtype"] == F16 else 4
    if c["op"] == "block_tables":
        L, n, P = _lens(c), _new_lens(c), c["P"]
        pages = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(L, n))
        return {"bytes": 8 * c["B"] + 4 * sum(1 for a, b in zip(L, n) if a % P and b) + 8 * pages + 8 * _slots(c)
                + 4 * (c["B"] + 1) + 4 * c["B"] + 4, "flops": 0}
    d = c["d"]
    row = d * c["bits"] // 8 + 2
    rot = 2 * (d * int(math.log2(d)) + 16 * d // 4 * 2)
    par = c["Hkv"] * 4 * d * 4
    if c["op"] == "paged_append":
        return {"bytes": c["N"] * c["Hkv"] * 2 * (d * e + row) + 8 * c["N"] + par,
                "flops": c["N"] * c["Hkv"] * 2 * (rot + 2 * d)}
    if c["op"] in ("window_decode", "paged_decode"):
        v = sum(_spans(c))
        nb = v * c["Hkv"] * 2 * row + c["B"] * c["Hq"] * d * 2 * e + par + 4 * c["B"]
        if c["op"] == "paged_decode":
            nb += 4 * sum(-(-x // c["P"]) for x in _spans(c))
        return {"bytes": nb, "flops": 4 * c["Hq"] * d * v + 2 * c["B"] * c["Hq"] * rot}
    if c["op"] == "prefix_decode":
        L = sum(_lens(c))
        return {"bytes": (c["Tp"] + L) * c["Hkv"] * 2 * row + c["B"] * c["Hq"] * d * 2 * e + par + 4 * c["B"] + 4,
                "flops": 4 * c["Hq"] * d * (c["B"] * c["Tp"] + L) + 2 * c["B"] * c["Hq"] * rot}
    # window_prefill: keys that any query of the chunk sees, and each query's own count
    Tq, W, S, keys, dots = c["Tq"], c["W"], c["S"], 0, 0
    for t in _lens(c):
        lo0 = max(0, t - Tq - W + 1)
        keys += t - max(0, lo0 - min(S, t))
        for p in range(t - Tq, t):
            lo = max(0, p - W + 1)
            dots += p + 1 - max(0, lo - min(S, p + 1))
    return {"bytes": keys * c["Hkv"] * 2 * row + 2 * c["B"] * Tq * c["Hq"] * d * e + par + 4 * c["B"],
            "flops": 4 * c["Hq"] * d * dots + 2 * c["B"] * Tq * c["Hq"] * rot}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_books = {}


def _codebook(bits):
    """Lloyd-Max levels and thresholds of N(0, 1), float64."""
    if bits not in _books:
        n = 1 << bits
        pdf = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
        cdf = np.vectorize(lambda x: 0.5 * (1 + math.erf(x / math.sqrt(2))))
        c = np.linspace(-2, 2, n)
        for _ in range(5000):
            t = (c[1:] + c[:-1]) / 2
            lo, hi = np.r_[-40.0, t], np.r_[t, 40.0]
            new = (pdf(lo) - pdf(hi)) / (cdf(hi) - cdf(lo))
            new = (new - new[::-1]) / 2
            done = np.abs(new - c).max() < 2e-15
            c = new
            if done:
                break
        _books[bits] = (c, (c[1:] + c[:-1]) / 2)
    return _books[bits]


def _pack(codes, bits):
    """uint8 rows of codes [..., d] (integers) in the library's layout."""
    x = codes.to(torch.int32)
    d = x.shape[-1]
    if bits == 3:
        x = x.reshape(*x.shape[:-1], d // 32, 32)
        sh = torch.arange(8, device=x.device, dtype=torch.int32) * 4
        body = x[..., :24].reshape(*x.shape[:-1], 3, 8)
        tail = x[..., None, 24:] >> torch.arange(3, device=x.device, dtype=torch.int32)[:, None] & 1
        w = ((body | tail << 3) << sh).sum(-1).to(torch.int32)
        return w.reshape(*w.shape[:-2], d // 32 * 3).contiguous().view(torch.uint8)
    per = 8 // bits
    sh = torch.arange(per, device=x.device, dtype=torch.int32) * bits
    return (x.reshape(*x.shape[:-1], d // per, per) << sh).sum(-1).to(torch.uint8)


def _unpack(rows, bits):
    """int32 codes [..., d] of uint8 rows."""
    if bits == 3:
        w = rows.contiguous().view(torch.int32)
        w = w.reshape(*w.shape[:-1], -1, 3, 1) >> torch.arange(8, device=w.device, dtype=torch.int32) * 4 & 15
        tail = w[..., 0, :] >> 3 | w[..., 1, :] >> 3 << 1 | w[..., 2, :] >> 3 << 2
        x = torch.cat([(w & 7).flatten(-2), tail], dim=-1)
        return x.flatten(-2)
    per = 8 // bits
    sh = torch.arange(per, device=rows.device, dtype=torch.int32) * bits
    return (rows.to(torch.int32)[..., None] >> sh & (1 << bits) - 1).flatten(-2)


def _params(g, heads, d, variant):
    q = torch.randn(heads, d // 4, 2, 4, generator=g, device="cuda")
    q = q / q.square().sum(-1, keepdim=True).sqrt()
    if variant == 1:
        q[:, :, 1] = torch.tensor([1.0, 0, 0, 0], device="cuda")
    return q.reshape(heads, d // 4, 8).contiguous()


def _cache(g, shape, d, bits):
    """Packed rows and norms of `shape` vectors: the codes that rotated vectors get, and norms of a heavy-tailed
    cache.  The rows are drawn from 16,384 different ones."""
    t = torch.tensor(_codebook(bits)[1], dtype=torch.float32, device="cuda")
    y = torch.randn(16384, d, generator=g, device="cuda")
    pool = _pack(torch.bucketize(y, t), bits)
    n = math.prod(shape)
    pick = torch.randint(0, 16384, (n,), generator=g, device="cuda")
    rows = pool.index_select(0, pick).reshape(*shape, -1)
    norms = (math.sqrt(d) * torch.exp(0.5 * torch.randn(*shape, generator=g, device="cuda"))).to(torch.float16)
    return rows, norms


def _had(d):
    """The Sylvester matrix, float64."""
    m = torch.ones(1, 1, dtype=torch.float64)
    while m.shape[0] < d:
        m = torch.cat([torch.cat([m, m], 1), torch.cat([m, -m], 1)], 0)
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _slots(c):
    """Room of the slot map: the step's new tokens, up to a fixed shape as a captured step has."""
    return _up(max(1, sum(_new_lens(c))), 64)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    s = {"case": c}
    if c["op"] == "block_tables":
        L, new, P, B = _lens(c), _new_lens(c), c["P"], c["B"]
        have = [-(-x // P) for x in L]
        cols = -(-(c["T"] + c["new"]) // P)
        n_pages = sum(have) + sum(-(-(a + b) // P) for a, b in zip(L, new)) + 8
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(cols, device="cuda")[None, :] < _i32(have)[:, None]
        table[held] = perm[:sum(have)]
        s.update(seq_lens=_i32(L), new_lens=_i32(new), free_pages=perm[sum(have):].contiguous(), table=table,
                 table0=table.clone(), n_slots=_slots(c))
        return s
    d, bits, Hkv = c["d"], c["bits"], c["Hkv"]
    dt = getattr(torch, c["dtype"])
    s.update(params_k=_params(g, Hkv, d, c["variant"]), params_v=_params(g, Hkv, d, c["variant"]))
    # constants that a program in plain operations keeps on the device: H_d / sqrt(d), levels, thresholds
    book = _codebook(bits)
    exactly = c["op"] == "paged_append"
    s["had"] = (_had(d) / math.sqrt(d)).to("cuda", torch.float64 if exactly else torch.float32)
    s["cent"] = torch.tensor(book[0] / math.sqrt(d), dtype=torch.float32, device="cuda")
    s["thr"] = torch.tensor(book[1] / math.sqrt(d), dtype=torch.float64, device="cuda")
    if c["op"] == "paged_append":
        N, P = c["N"], c["P"]
        n_pages = -(-N // P) + 7
        # requests' tokens fill pages in runs; a few padded places of the step carry no token
        pages = torch.randperm(n_pages, generator=g, device="cuda")[: -(-N // P)]
        slot = (pages[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)[:N].contiguous()
        if N > 16:
            slot[N - 2:] = -1
        x = torch.randn(2, N, Hkv, d, generator=g, device="cuda")
        x = x / torch.sqrt((torch.randn(2, N, Hkv, d, 4, generator=g, device="cuda").square()).mean(-1) + 0.05)
        s.update(k=x[0].to(dt).contiguous(), v=x[1].to(dt).contiguous(), slot=slot)
        s["pages_k"], s["norms_k"] = _cache(g, (n_pages, Hkv, P), d, bits)
        s["pages_v"], s["norms_v"] = _cache(g, (n_pages, Hkv, P), d, bits)
        return s
    B, Hq = c["B"], c["Hq"]
    s["seq_lens"] = _i32(_lens(c))
    if c["op"] == "window_prefill":
        s["q"] = torch.randn(B, c["Tq"], Hq, d, generator=g, device="cuda").to(dt)
    else:
        s["q"] = torch.randn(B, Hq, d, generator=g, device="cuda").to(dt)
    if c["op"] == "paged_decode":
        P, T = c["P"], c["T"]
        cols = -(-T // P)
        n_pages = B * cols + 3
        s["table"] = torch.randperm(n_pages, generator=g, device="cuda")[: B * cols].to(torch.int32).reshape(B, cols)
        s["pages_k"], s["norms_k"] = _cache(g, (n_pages, Hkv, P), d, bits)
        s["pages_v"], s["norms_v"] = _cache(g, (n_pages, Hkv, P), d, bits)
        return s
    room = _up(c["T"], 8)
    s["k"], s["norms_k"] = _cache(g, (B, Hkv, room), d, bits)
    s["v"], s["norms_v"] = _cache(g, (B, Hkv, room), d, bits)
    if c["op"] == "prefix_decode":
        room = _up(c["Tp"], 8)
        s["prefix_k"], s["prefix_norms_k"] = _cache(g, (Hkv, room), d, bits)
        s["prefix_v"], s["prefix_norms_v"] = _cache(g, (Hkv, room), d, bits)
        s["prefix_len"] = _i32([c["Tp"]])
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _rotation(params, had):
    """[heads][d][d] matrices R: 4 x 4 quaternion blocks after the orthonormal Walsh-Hadamard matrix `had`."""
    heads, nb = params.shape[:2]
    d = 4 * nb
    p = params.to(had.dtype)
    w, x, y, z = p[..., 0], p[..., 1], p[..., 2], p[..., 3]
    left = torch.stack([w, -x, -y, -z, x, w, -z, y, y, z, w, -x, z, -y, x, w], -1).reshape(heads, nb, 4, 4)
    w, x, y, z = p[..., 4], -p[..., 5], -p[..., 6], -p[..., 7]
    right = torch.stack([w, -x, -y, -z, x, w, z, -y, y, -z, w, x, z, y, -x, w], -1).reshape(heads, nb, 4, 4)
    return ((right @ left) @ had.reshape(1, nb, 4, d)).reshape(heads, d, d)


def _values(s, rows, norms):
    """float32 rotated-domain vectors that packed rows stand for."""
    codes = _unpack(rows, s["case"]["bits"])
    return s["cent"].index_select(0, codes.reshape(-1)).reshape(codes.shape) * norms.float()[..., None]


def _soft(z):
    """Weights of scores z (-inf: not seen); a row that sees nothing has weight nowhere."""
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-38)


def _attend(s, q, k, v, seen):
    """q [B][Hq][d] over k, v [B][Hkv][n][d] (rotated domain), seen [B][n]."""
    c = s["case"]
    B, Hq, d = q.shape
    Hkv = c["Hkv"]
    qr = q.float().reshape(B, Hkv, Hq // Hkv, d) @ _rotation(s["params_k"], s["had"]).transpose(1, 2)
    z = qr @ k.transpose(2, 3) * (1 / math.sqrt(d))
    p = _soft(z.masked_fill(~seen[:, None, None, :], -math.inf))
    return ((p @ v) @ _rotation(s["params_v"], s["had"])).reshape(B, Hq, d).to(q.dtype)


def _seen_tokens(c, lens, W):
    """Token indices [B][n] that cover each row's sinks and window, and which of them it sees."""
    S, T = c["S"], c["T"]
    ns, nw = min(S, T), min(W, T)
    sink = torch.arange(ns, device=lens.device).expand(c["B"], ns)
    near = lens.long()[:, None] - 1 - torch.arange(nw, device=lens.device)
    tok = torch.cat([sink, near], 1)
    seen = torch.cat([sink < lens[:, None], near >= ns], 1)
    return tok.clamp(0, T - 1), seen


def _plain_window_decode(s):
    c = s["case"]
    tok, seen = _seen_tokens(c, s["seq_lens"], c["W"])
    at = tok[:, None, :].expand(-1, c["Hkv"], -1)
    kv = []
    for rows, norms in ((s["k"], s["norms_k"]), (s["v"], s["norms_v"])):
        r = torch.gather(rows, 2, at[..., None].expand(-1, -1, -1, rows.shape[-1]))
        kv.append(_values(s, r, torch.gather(norms, 2, at)))
    return _attend(s, s["q"], kv[0], kv[1], seen)


def _plain_paged_decode(s):
    c = s["case"]
    P = c["P"]
    tok, seen = _seen_tokens(c, s["seq_lens"], c["W"] or c["T"])
    page = torch.gather(s["table"].long(), 1, tok // P)[:, None, :]
    head = torch.arange(c["Hkv"], device=tok.device)[None, :, None]
    at = (page * c["Hkv"] + head) * P + (tok % P)[:, None, :]
    kv = []
    for rows, norms in ((s["pages_k"], s["norms_k"]), (s["pages_v"], s["norms_v"])):
        r = rows.reshape(-1, rows.shape[-1]).index_select(0, at.reshape(-1)).reshape(*at.shape, -1)
        kv.append(_values(s, r, norms.reshape(-1)[at]))
    return _attend(s, s["q"], kv[0], kv[1], seen)


def _plain_window_prefill(s):
    c = s["case"]
    B, Tq, Hq, d = s["q"].shape
    Hkv, W, S = c["Hkv"], c["W"], c["S"]
    k = _values(s, s["k"], s["norms_k"])
    v = _values(s, s["v"], s["norms_v"])
    q = s["q"].float().reshape(B, Tq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    z = q @ _rotation(s["params_k"], s["had"]).transpose(1, 2) @ k.transpose(2, 3) * (1 / math.sqrt(d))
    pos = s["seq_lens"].long()[:, None, None] - Tq + torch.arange(Tq, device=q.device)[None, :, None]
    j = torch.arange(k.shape[2], device=q.device)
    seen = (j <= pos) & ((j > pos - W) | (j < S))
    z = z.reshape(B, Hkv, Hq // Hkv, Tq, -1).masked_fill(~seen[:, None, None], -math.inf)
    o = _soft(z).reshape(B, Hkv, -1, k.shape[2]) @ v @ _rotation(s["params_v"], s["had"])
    return o.reshape(B, Hkv, Hq // Hkv, Tq, d).permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, d).to(s["q"].dtype)


def _plain_prefix_decode(s):
    c = s["case"]
    B, Hq, d = s["q"].shape
    Hkv = c["Hkv"]
    G = Hq // Hkv
    pk = _values(s, s["prefix_k"], s["prefix_norms_k"])
    pv = _values(s, s["prefix_v"], s["prefix_norms_v"])
    k, v = _values(s, s["k"], s["norms_k"]), _values(s, s["v"], s["norms_v"])
    qr = s["q"].float().reshape(B, Hkv, G, d) @ _rotation(s["params_k"], s["had"]).transpose(1, 2)
    every = qr.transpose(0, 1).reshape(Hkv, B * G, d)
    zp = (every @ pk.transpose(1, 2)).reshape(Hkv, B, G, -1).transpose(0, 1)
    seen_p = torch.arange(pk.shape[1], device=qr.device) < s["prefix_len"]
    zp = zp.masked_fill(~seen_p, -math.inf)
    seen = torch.arange(k.shape[2], device=qr.device) < s["seq_lens"][:, None]
    zo = (qr @ k.transpose(2, 3)).masked_fill(~seen[:, None, None, :], -math.inf)
    p = _soft(torch.cat([zp, zo], -1) * (1 / math.sqrt(d)))
    n = zp.shape[-1]
    o = (p[..., :n].transpose(0, 1).reshape(Hkv, B * G, n) @ pv).reshape(Hkv, B, G, d).transpose(0, 1)
    o = o + p[..., n:] @ v
    return (o @ _rotation(s["params_v"], s["had"])).reshape(B, Hq, d).to(s["q"].dtype)


def _plain_block_tables(s):
    P, N, table = s["case"]["P"], s["n_slots"], s["table"]
    table.copy_(s["table0"])
    L, new, free = s["seq_lens"].long(), s["new_lens"].long(), s["free_pages"]
    cols = table.shape[1]
    fits = L + new <= cols * P
    have, need = (L + P - 1) // P, (L + new + P - 1) // P
    take = torch.where(fits, need - have, 0)
    cum = take.cumsum(0)
    ok = fits & ((take == 0) | (cum <= free.numel()))
    first = cum - take
    col = torch.arange(cols, device=L.device)
    fresh = ok[:, None] & (col >= have[:, None]) & (col < need[:, None])
    src = (first[:, None] + col - have[:, None]).clamp(0, max(0, free.numel() - 1))
    table.copy_(torch.where(fresh, free[src], table))
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    i = torch.arange(N, device=L.device)
    b = (torch.searchsorted(start, i, right=True) - 1).clamp(0, L.numel() - 1)
    pos = L[b] + i - start[b]
    page = table[b, (pos // P).clamp(0, cols - 1)].long()
    slot = torch.where((i < start[-1]) & ok[b], page * P + pos % P, -1)
    used = torch.where(ok, cum, 0).amax().reshape(1)
    total = torch.where(ok, L + new, L)
    return {"table": table, "slot_map": slot, "row_start": start.to(torch.int32), "total_lens": total.to(torch.int32),
            "pages_used": used.to(torch.int32)}


def _plain_paged_append(s):
    c = s["case"]
    P, Hkv, bits = c["P"], c["Hkv"], c["bits"]
    slot = s["slot"]
    ok = slot >= 0
    head = torch.arange(Hkv, device=slot.device)
    at = ((slot // P)[:, None] * Hkv + head) * P + (slot % P)[:, None]
    at = at[ok].reshape(-1)
    for x, rows, norms, par in ((s["k"], s["pages_k"], s["norms_k"], s["params_k"]),
                                (s["v"], s["pages_v"], s["norms_v"], s["params_v"])):
        x = x[ok].double()
        n = x.square().sum(-1, keepdim=True).sqrt()
        y = (x / n.clamp_min(1e-300)).transpose(0, 1) @ _rotation(par, s["had"]).transpose(1, 2)
        codes = (y.transpose(0, 1)[..., None] > s["thr"]).sum(-1)
        rows.reshape(-1, rows.shape[-1])[at] = _pack(codes, bits).reshape(at.numel(), -1)
        norms.reshape(-1)[at] = n.to(torch.float16).reshape(-1)
    # the rows bit for bit: every code is the float64 decision
    return [s["pages_k"], s["pages_v"], s["norms_k"], s["norms_v"]]


_plain = {"window_decode": _plain_window_decode, "window_prefill": _plain_window_prefill,
          "prefix_decode": _plain_prefix_decode, "block_tables": _plain_block_tables,
          "paged_append": _plain_paged_append, "paged_decode": _plain_paged_decode}


# ---------------------------------------------------------------------------
# The calls that a user makes
# ---------------------------------------------------------------------------

def _own(s):
    import compressed_space_attention_b200 as isoq

    c = s["case"]
    op = c["op"]
    if op == "block_tables":
        s["table"].copy_(s["table0"])
        slot, start, total, used = isoq.isoq_build_block_tables(s["seq_lens"], s["new_lens"], s["free_pages"],
                                                                s["table"], c["P"], s["n_slots"])
        return {"table": s["table"], "slot_map": slot, "row_start": start, "total_lens": total, "pages_used": used}
    bits, variant = c["bits"], c["variant"]
    if op == "paged_append":
        isoq.isoq_paged_append(s["k"], s["v"], s["pages_k"], s["pages_v"], s["norms_k"], s["norms_v"], s["slot"],
                               s["params_k"], s["params_v"], bits, variant)
        return [s["pages_k"], s["pages_v"], s["norms_k"], s["norms_v"]]
    par = (s["params_k"], s["params_v"], bits, variant)
    if op == "paged_decode":
        return isoq.isoq_paged_decode_attention(s["q"], s["pages_k"], s["pages_v"], s["norms_k"], s["norms_v"],
                                                s["table"], s["seq_lens"], *par, max_len=c["T"],
                                                window=c["W"] or None, n_sink=c["S"])
    cache = (s["k"], s["v"], s["norms_k"], s["norms_v"], s["seq_lens"])
    if op == "window_decode":
        return isoq.isoq_decode_attention_window(s["q"], *cache, *par, window=c["W"], n_sink=c["S"])
    if op == "window_prefill":
        return isoq.isoq_prefill_attention_window(s["q"], *cache, *par, window=c["W"], n_sink=c["S"])
    return isoq.isoq_decode_attention_prefix(s["q"], s["prefix_k"], s["prefix_v"], s["prefix_norms_k"],
                                             s["prefix_norms_v"], s["prefix_len"], *cache, *par)


def run(state):
    return _own(state) if own else _plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definition in 64 bits, in the original domain
# ---------------------------------------------------------------------------

def _hamilton(p, q):
    a, b, c, d = p.unbind(-1)
    e, f, g, h = q.unbind(-1)
    return torch.stack([a * e - b * f - c * g - d * h, a * f + b * e + c * h - d * g,
                        a * g - b * h + c * e + d * f, a * h + b * g - c * f + d * e], -1)


def _wht(x):
    d = x.shape[-1]
    h = 1
    while h < d:
        y = x.reshape(*x.shape[:-1], d // (2 * h), 2, h)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
        h *= 2
    return x / math.sqrt(d)


_flip = (1.0, -1.0, -1.0, -1.0)


def _exact_vectors(rows, norms, bits, d, par):
    """float64 vectors of packed rows [n][...] of one head, rotated back."""
    raw = rows.reshape(-1, rows.shape[-1]).to(torch.int64)
    bit = (raw[..., None] >> torch.arange(8, device=raw.device) & 1).reshape(raw.shape[0], -1)
    if bits == 3:
        g = bit.reshape(raw.shape[0], d // 32, 3, 8, 4)
        body = (g[..., 0] + 2 * g[..., 1] + 4 * g[..., 2]).reshape(raw.shape[0], d // 32, 24)
        last = g[:, :, 0, :, 3] + 2 * g[:, :, 1, :, 3] + 4 * g[:, :, 2, :, 3]
        code = torch.cat([body, last], -1).reshape(raw.shape[0], d)
    else:
        b = bit.reshape(raw.shape[0], d, bits)
        code = sum(b[..., i] << i for i in range(bits))
    c = torch.tensor(_codebook(bits)[0], dtype=torch.float64, device=raw.device)[code] / math.sqrt(d)
    flip = torch.tensor(_flip, dtype=torch.float64, device=raw.device)
    p = par.double()
    u = _hamilton(_hamilton(p[:, :4] * flip, c.reshape(-1, d // 4, 4)), p[:, 4:])
    return _wht(u.reshape(-1, d)) * norms.reshape(-1).double()[:, None]


def exact(case, seed):
    c = dict(case)
    if c["op"] == "block_tables":
        return None
    s = prepare(case, seed)
    bits, d, Hkv = c["bits"], c["d"], c["Hkv"]
    if c["op"] == "paged_append":
        out = []
        for x, norms in ((s["k"], s["norms_k"]), (s["v"], s["norms_v"])):
            n = norms.double()
            live = (s["slot"] >= 0).nonzero().reshape(-1)
            for h in range(Hkv):
                n[s["slot"][live] // c["P"], h, s["slot"][live] % c["P"]] = torch.sqrt((x[live, h].double() ** 2).sum(-1))
            out.append(n)
        return [None, None] + out
    q = s["q"].double()
    B, Hq = q.shape[0], c["Hq"]
    G = Hq // Hkv
    o = torch.zeros_like(q)
    lens = _lens(c)

    def own_rows(which, b, h, idx):
        par = s["params_" + which][h]
        if c["op"] == "paged_decode":
            page, off = s["table"][b].long()[idx // c["P"]], idx % c["P"]
            return _exact_vectors(s["pages_" + which][page, h, off], s["norms_" + which][page, h, off], bits, d, par)
        return _exact_vectors(s[which][b, h, idx], s["norms_" + which][b, h, idx], bits, d, par)

    shared = []
    if c["op"] == "prefix_decode":
        shared = [[_exact_vectors(s["prefix_" + w][h, :c["Tp"]], s["prefix_norms_" + w][h, :c["Tp"]], bits, d,
                                  s["params_" + w][h]) for w in ("k", "v")] for h in range(Hkv)]
    for b in range(B):
        t = lens[b]
        if c["op"] in ("window_decode", "paged_decode"):
            W = c["W"] if c["op"] == "window_decode" or c["W"] else t
            idx = torch.tensor([j for j in range(t) if j >= t - W or j < c["S"]], device="cuda")
        else:
            idx = torch.arange(t, device="cuda")
        for h in range(Hkv):
            k, v = own_rows("k", b, h, idx), own_rows("v", b, h, idx)
            if shared:
                k, v = torch.cat([shared[h][0], k]), torch.cat([shared[h][1], v])
            for i in range(h * G, h * G + G):
                if c["op"] == "window_prefill":
                    p = torch.arange(t - c["Tq"], t, device="cuda")[:, None]
                    hid = (idx > p) | ((idx <= p - c["W"]) & (idx >= c["S"]))
                    z = (q[b, :, i] @ k.T / math.sqrt(d)).masked_fill(hid, -math.inf)
                    o[b, :, i] = torch.softmax(z, -1) @ v
                else:
                    o[b, i] = torch.softmax(k @ q[b, i] / math.sqrt(d), 0) @ v
    return o
