"""The serving operators at the edges of what their documentation allows:
streams given by argument, pages dropped behind the window, magnitudes next to
float16's limits, alignments and cluster sizes that ordinary calls do not
reach.  Tolerances as in test_parity_serving, unless a test derives its own."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import compressed_space_attention_b200 as isoq  # noqa: E402
import oracle as O  # noqa: E402
from isoq_testlib import f16_half_ulp  # noqa: E402
from oracle import serving as S  # noqa: E402
from test_parity_serving import DEV, F16, F32, _cache, _check, _pages, _params, _t  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument_without_workspace(raw):
    """Calls on two streams given by argument, none with a workspace or an
    output of its own, while the current stream allocates and writes blocks of
    the workspaces' sizes: the bits of the same calls one after the other."""
    g = np.random.default_rng(20)
    d, hq, hkv, b, tmax, p = 128, 32, 4, 6, 6144, 64
    lens = np.full(b, 6000, np.int32)
    cache, prefix = [_t(c) for c in _cache(g, (b, hkv, tmax), d, 3)], [_t(c) for c in _cache(g, (hkv, 4096), d, 3)]
    pages, table = _pages(g, lens, hkv, d, 3, p, tmax // p)
    pages, table = [_t(x) for x in pages], _t(table)
    par, dl = [_t(x) for x in _params(hkv, d, 0)], _t(lens)
    plen = torch.tensor([4000], dtype=torch.int32, device=DEV)
    q = _t(g.standard_normal((b, hq, d)).astype(F16))
    qc = _t(g.standard_normal((b, 40, hq, d)).astype(F16))
    calls = [lambda **k: isoq.isoq_decode_attention_window(q, *cache, dl, *par, 3, 0, 5000, 64, **k),
             lambda **k: isoq.isoq_decode_attention_prefix(q, *prefix, plen, *cache, dl, *par, 3, 0, **k),
             lambda **k: isoq.isoq_paged_decode_attention(q, *pages, table, dl, *par, 3, 0, **k),
             lambda **k: isoq.isoq_prefill_attention_window(qc, *cache, dl, *par, 3, 0, 600, 5, **k),
             lambda **k: isoq.isoq_decode_attention(q, *cache, dl, *par, 3, 0, **k)]
    sizes = [isoq.isoq_decode_window_workspace_size(b, hq, hkv, tmax, d, 5000, 64),
             isoq.isoq_decode_prefix_workspace_size(b, hq, hkv, 4096, tmax, d),
             isoq.isoq_decode_workspace_size(b, hq, hkv, tmax, d)]
    assert min(sizes) > 0
    alone = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(6):
        outs = []
        for i, f in enumerate(calls):
            s = streams[(i + turn) % 2]
            outs.append(f(stream=s.cuda_stream if raw else s))
            for n in sizes:
                torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for a, o in zip(alone, outs):
            assert torch.equal(a, o)
    assert isoq.isoq_check_device_error() == 0


def _drop_unseen_pages(table, lens, p, max_len, window, n_sink, fill):
    """The table with `fill` at every page that holds no token its row's query sees."""
    out = table.copy()
    for b, t in enumerate(lens):
        t = min(max(int(t), 0), max_len)
        pages = {j // p for j in S.seen_tokens(t - 1, t, window, n_sink)}
        out[b, [c for c in range(table.shape[1]) if c not in pages]] = fill
    return out


@pytest.mark.parametrize("p", [16, 32])
@pytest.mark.parametrize("dtype,d,bits,hq,hkv", [(F16, 128, 3, 8, 2), (F16, 256, 3, 2, 2), (F32, 128, 4, 6, 2),
                                                 (F16, 512, 2, 4, 1)])
def test_pages_that_no_query_sees_are_not_followed(dtype, d, bits, hq, hkv, p):
    """Pages behind the window and between it and the sinks are gone from the
    table (-1, or an index beyond the pool): no error, the same outputs, in
    one launch and in many splits."""
    g = np.random.default_rng(p + d)
    tmax = 6400
    lens = np.array([333, 48, 17, 1, 0, 640, 5000, 6399], np.int32)
    cols = tmax // p
    pages, table = _pages(g, lens, hkv, d, bits, p, cols)
    par = _params(hkv, d, 0)
    q = g.standard_normal((len(lens), hq, d)).astype(dtype)
    dev, dpar, scale = [_t(x) for x in pages], [_t(x) for x in par], 1 / np.sqrt(d)
    for window, n_sink, fill in [(1, 0, -1), (17, 0, 1 << 30), (40, 5, -1), (100, 16, -1), (15, 33, 1 << 30), (4200, 17, -1)]:
        rows = np.arange(len(lens)) if window > 1000 else np.arange(6)
        max_len = tmax if window > 1000 else 640
        gone = _drop_unseen_pages(table, lens, p, max_len, window, n_sink, fill)
        got = isoq.isoq_paged_decode_attention(_t(q[rows]), *dev, _t(gone[rows]), _t(lens[rows]), *dpar, bits, 0,
                                               max_len=max_len, window=window, n_sink=n_sink)
        ref = S.paged_decode(q[rows], pages, table[rows], lens[rows], *par, bits, 0, scale, max_len, window, n_sink)
        _check(got, ref, dtype, q, pages[2], pages[3], scale)


def _queries(g, shape, kind):
    """float16 queries and the scale that keeps their scores moderate.
    "large": rows of +-60,000 in a Walsh-Hadamard pattern, whose transform
    gathers in one coordinate (far above 65,504 once rotated), and random
    signs of it; "tiny": float16's subnormal numbers; "mixed": large, ordinary
    and tiny rows in turn (a large row's scores are far apart)."""
    d = shape[-1]
    rows = int(np.prod(shape[:-1]))
    q = g.standard_normal((rows, d))
    if kind == "tiny":
        return (q * 4e-7).astype(F16).reshape(shape), 1 / (4e-7 * np.sqrt(d))
    had = np.array([[1.0]])
    while had.shape[0] < d:
        had = np.block([[had, had], [had, -had]])
    big = 60000 * had[g.integers(0, d, rows)] * np.where(g.random((rows, 1)) < 0.5, 1, g.choice([-1, 1], (rows, d)))
    if kind == "large":
        return big.astype(F16).reshape(shape), 1 / (60000 * np.sqrt(d))
    turn = np.arange(rows)[:, None] % 3
    return np.where(turn == 0, big, np.where(turn == 1, q, 4e-7 * q)).astype(F16).reshape(shape), 1 / np.sqrt(d)


@pytest.mark.parametrize("kind", ["large", "tiny", "mixed"])
@pytest.mark.parametrize("d,rows", [(128, 8), (128, 9), (128, 130), (256, 23), (256, 24), (256, 130)])
def test_prefix_of_any_query_magnitude(d, rows, kind):
    """Rows just below and above the ones that take the tcgen05 split."""
    g = np.random.default_rng(rows)
    tp, tmax = 700, 40
    prefix, cache = _cache(g, (1, tp), d, 3), _cache(g, (rows, 1, tmax), d, 3)
    par = _params(1, d, 0)
    q, scale = _queries(g, (rows, 1, d), kind)
    lens, plen = g.integers(0, tmax + 1, rows).astype(np.int32), np.array([tp - 3], np.int32)
    got = isoq.isoq_decode_attention_prefix(_t(q), *map(_t, prefix), _t(plen), *map(_t, cache), _t(lens), *map(_t, par), 3,
                                            0, scale=scale)
    some = sorted(set(range(min(rows, 24))) | {rows - 1})
    ref = S.prefix_decode(q[some], prefix, tp - 3, *[c[some] for c in cache], lens[some], *par, 3, 0, scale)
    _check(got[some], ref, F16, q, cache[2], cache[3], scale)


@pytest.mark.parametrize("kind", ["large", "tiny", "mixed"])
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (128, 8, 1), (256, 2, 2), (256, 8, 1)])
def test_prefill_of_any_query_magnitude(d, hq, hkv, kind):
    """The windowed and the plain chunk; both at d = 128 and 256."""
    g = np.random.default_rng(d + hq)
    tmax, tq = 320, 24
    lens = np.array([300, 24], np.int32)
    cache, par = _cache(g, (2, hkv, tmax), d, 3), _params(hkv, d, 0)
    q, scale = _queries(g, (2, tq, hq, d), kind)
    args = (*map(_t, cache), _t(lens), *map(_t, par), 3, 0)
    for window, n_sink, call in [(150, 20, lambda: isoq.isoq_prefill_attention_window(_t(q), *args, 150, 20, scale=scale)),
                                 (1 << 30, 0, lambda: isoq.isoq_prefill_attention(_t(q), *args, scale=scale))]:
        ref = S.window_prefill(q, *cache, lens, *par, 3, 0, scale, window, n_sink)
        _check(call(), ref, F16, q, cache[2], cache[3], scale)


@pytest.mark.parametrize("v_norm,hidden", [(1e-4, 1e-4), (1e-4, 65504.0), (0.01, 65504.0), (3.0, 3.0), (30000.0, 1e-7)])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", ["prefix", "window", "plain"])
def test_many_small_weights_count_whatever_the_v_norms(form, d, v_norm, hidden):
    """One token's score is 12 (log2) above those of 8,191 others, and all have
    one V vector, which therefore is the output: it misses what a form loses of
    the 8,191 weights of 2^-12 (2/3 of the sum).  Norms that unscaled float16
    weights cannot hold; behind the window, norms that no query sees, other
    than the seen ones.  Tolerance: half a float16 step of the value, and
    2^-15 of the V vector (its length is v_norm) for the float16 centroids
    (1.9e-5 relative) and the float32 sums."""
    g = np.random.default_rng(d)
    n, t = 8192, 8192 + (200 if form == "window" else 0)
    par = _params(1, d, 0)
    one = _cache(g, (1, 1), d, 3)
    k, v = (np.repeat(x, t, axis=1) for x in one[:2])
    nk, nv = np.full((1, t), 8.0, F16), np.full((1, t), v_norm, F16)
    nv[:, :t - n] = hidden
    top = t - n + 40
    nk[:, top] = 16.0
    q1 = g.standard_normal(d).astype(F16)
    unit_k, unit_v = (O.dequantize(x[:, :1], np.ones((1, 1), F16), p, 3, 0, d)[0, 0] for x, p in zip((k, v), par))
    unit = float(q1.astype(np.float64) @ unit_k)
    scale = 12 * np.log(2) / (8 * unit)
    args = (*map(_t, par), 3, 0)
    if form == "prefix":
        rows = 9 if d == 128 else 24
        q = np.tile(q1, (rows, 1, 1))
        own = _cache(g, (rows, 1, 8), d, 3)
        got = isoq.isoq_decode_attention_prefix(_t(q), _t(k), _t(v), _t(nk), _t(nv), _t(np.array([t], np.int32)),
                                                *map(_t, own), _t(np.zeros(rows, np.int32)), *args, scale=scale)
    else:
        q = q1.reshape(1, 1, 1, d)
        cache = [_t(x[None]) for x in (k, v, nk, nv)]
        lens = _t(np.array([t], np.int32))
        got = isoq.isoq_prefill_attention(_t(q), *cache, lens, *args, scale=scale) if form == "plain" else \
            isoq.isoq_prefill_attention_window(_t(q), *cache, lens, *args, n, 0, scale=scale)
    assert isoq.isoq_check_device_error() == 0
    ref = float(F16(v_norm)) * unit_v
    err = np.abs(got.cpu().numpy().astype(np.float64).reshape(-1, d) - ref)
    assert (err <= f16_half_ulp(ref) + 2.0 ** -15 * float(F16(v_norm))).all(), (err.max(), np.abs(ref).max())


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("tmax,window,n_sink", [(504, 400, 5), (504, 300, 200), (3000, 900, 700), (3000, 2200, 640), (504, 600, 3)])
def test_v_norms_whose_largest_lies_anywhere(d, tmax, window, n_sink):
    """The seen tokens' V norms are 2^-13 but for 32 tokens of 3: among the
    sinks, where the window begins, in its last tokens; and 65,504 where no
    query sees them.  A scale that left the 32 out would overflow."""
    g = np.random.default_rng(d + tmax)
    cache, par = _cache(g, (1, 1, tmax), d, 3), _params(1, d, 0)
    t, tq = tmax - 3, 2
    q = g.standard_normal((1, tq, 1, d)).astype(F16)
    lo = max(t - tq - window + 1, 0)
    for at in (0, lo, max(lo, 128 * (lo // 128 + 1) - 32), t - 34):
        nv = np.full((1, 1, tmax), 2.0 ** -13, F16)
        nv[..., at:at + 32] = 3
        seen = set(S.seen_tokens(t - 2, t, window, n_sink)) | set(S.seen_tokens(t - 1, t, window, n_sink))
        nv[..., [j for j in range(tmax) if j not in seen]] = 65504
        got = isoq.isoq_prefill_attention_window(_t(q), *map(_t, (*cache[:3], nv)), _t(np.array([t], np.int32)), *map(_t, par),
                                                 3, 0, window, n_sink)
        ref = S.window_prefill(q, *cache[:3], nv, [t], *par, 3, 0, 1 / np.sqrt(d), window, n_sink)
        _check(got, ref, F16, q, cache[2], nv, 1 / np.sqrt(d))


@pytest.mark.parametrize("dtype,d,bits,hq,hkv,b,t", [(F16, 256, 3, 32, 4, 32, 1024), (F16, 128, 3, 32, 4, 24, 1024),
                                                     (F16, 256, 3, 16, 4, 32, 1000), (F32, 512, 4, 4, 4, 32, 1024),
                                                     (F32, 512, 2, 8, 8, 16, 520), (F32, 256, 3, 16, 4, 16, 2048)])
def test_decode_of_batches_that_fill_the_gpu(dtype, d, bits, hq, hkv, b, t):
    """Batches next to what one resident wave of clusters takes, on both sides."""
    g = np.random.default_rng(d + b)
    cache, par = _cache(g, (b, hkv, t), d, bits), _params(hkv, d, 0)
    lens = g.integers(1, t + 1, b).astype(np.int32)
    lens[:3] = t, 1, 0
    q = g.standard_normal((b, hq, d)).astype(dtype)
    got = isoq.isoq_decode_attention_window(_t(q), *map(_t, cache), _t(lens), *map(_t, par), bits, 0, t)
    rows = [0, 1, 2, 3, b // 2, b - 1]
    ref = S.window_decode(q[rows], *[c[rows] for c in cache], lens[rows], *par, bits, 0, 1 / np.sqrt(d), t, 0)
    _check(got[rows], ref, dtype, q, cache[2], cache[3], 1 / np.sqrt(d))


def test_every_error_since_the_last_check_is_named():
    """A slot beyond the pages, a request without room and an append to a full
    row before one check: one status, all three named, then nothing."""
    g = np.random.default_rng(30)
    par = [_t(x) for x in _params(1, 128, 0)]
    pages, cache = [_t(x) for x in _cache(g, (2, 1, 16), 128, 3)], [_t(x) for x in _cache(g, (1, 1, 8), 128, 3)]
    kv = _t(g.standard_normal((2, 1, 1, 128)).astype(F16))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    bad_slot = lambda: isoq.isoq_paged_append(kv[0], kv[1], *pages, torch.tensor([32], device=DEV), *par, 3, 0)  # noqa: E731
    no_room = lambda: isoq.isoq_build_block_tables(i32(0), i32(5), i32(), torch.zeros((1, 1), dtype=torch.int32, device=DEV), 16, 5)  # noqa: E731
    full_row = lambda: isoq.isoq_decode_append(kv[0], kv[1], *cache, i32(8), *par, 3, 0)  # noqa: E731
    said = {"slot outside the pages": bad_slot, "no room for a request": no_room, "held Tmax tokens": full_row}
    assert isoq.isoq_check_device_error() == 0
    for what, call in said.items():
        call()
        assert isoq.isoq_check_device_error() == isoq.ISOQ_ERR_INVALID_ARG
        assert [w for w in said if w in isoq.last_error()] == [what]
        assert isoq.isoq_check_device_error() == 0
    for call in said.values():
        call()
    assert isoq.isoq_check_device_error() == isoq.ISOQ_ERR_INVALID_ARG
    assert all(w in isoq.last_error() for w in said), isoq.last_error()
    assert isoq.isoq_check_device_error() == 0


def _row_tile_ranks(b, tq, hq, hkv, tmax, window, n_sink):
    """CTAs that share a row tile's tokens in the d = 128 windowed prefill."""
    per = 128 // (hq // hkv)
    ctas = -(-tq // per) * hkv * b
    w, s = min(window + per, tmax), min(n_sink, tmax)
    blocks, near, sink = -(-tmax // 32), -(-w // 32) + 1, -(-s // 32)
    if near < blocks and sink < blocks and near + sink < blocks:
        blocks = near + sink
    return max(1, min(148 // ctas, 8, (blocks // 4 + 1) // 2))


@pytest.mark.parametrize("b,tq,hq,hkv,lens,window,n_sink,ranks", [
    (1, 8, 8, 1, [3971], 4000, 0, 8), (1, 16, 8, 1, [2500], 1500, 300, 7), (1, 100, 8, 4, [3000], 2000, 5, 8),
    (3, 30, 4, 4, [3999, 700, 29], 4000, 0, 8), (2, 60, 8, 8, [1300, 1111], 900, 40, 5), (1, 1, 1, 1, [1700], 1500, 130, 7),
    (1, 1, 2, 2, [700], 400, 100, 3), (2, 40, 8, 8, [4000, 260], 2600, 700, 8), (1, 130, 1, 1, [2047], 1, 2047, 8),
    (1, 4, 8, 1, [5], 4000, 9, 8)])
def test_prefill_clusters_of_every_size(b, tq, hq, hkv, lens, window, n_sink, ranks):
    """Clusters of 3 to 8 CTAs, odd ones among them, whose shares of a row
    tile's tokens are uneven or empty, sinks in other CTAs than the window."""
    tmax = 4000
    assert _row_tile_ranks(b, tq, hq, hkv, tmax, window, n_sink) == ranks
    g = np.random.default_rng(ranks + tq)
    cache, par = _cache(g, (b, hkv, tmax), 128, 3), _params(hkv, 128, 0)
    q, lens = g.standard_normal((b, tq, hq, 128)).astype(F16), np.array(lens, np.int32)
    got = isoq.isoq_prefill_attention_window(_t(q), *map(_t, cache), _t(lens), *map(_t, par), 3, 0, window, n_sink)
    rows = sorted({0, tq // 3, tq // 2, tq - 1})
    ref = S.window_prefill(q, *cache, lens, *par, 3, 0, 1 / np.sqrt(128), window, n_sink, rows=rows)
    _check(got[:, rows], ref[:, rows], F16, q, cache[2], cache[3], 1 / np.sqrt(128))


def _four_bytes_on(x):
    """The same float16 tensor, its data 4 bytes past an 8-byte boundary."""
    flat = torch.zeros(x.numel() + 8, dtype=x.dtype, device=x.device)
    at = 2 if flat.data_ptr() % 8 == 0 else 0
    flat = flat[at:at + x.numel()].view(x.shape)
    assert flat.data_ptr() % 8 == 4
    return flat.copy_(x)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("variant", [isoq.ISOQ_FULL, isoq.ISOQ_FAST])
@pytest.mark.parametrize("which", ["q", "out"])
def test_window_prefill_of_queries_off_an_8_byte_boundary(hq, hkv, variant, which):
    """d = 128 with q or out aligned to 4 bytes only: the other kernel."""
    g = np.random.default_rng(hq)
    tmax, tq = 328, 70
    lens = np.array([328, 90], np.int32)
    cache, par = _cache(g, (2, hkv, tmax), 128, 3), _params(hkv, 128, variant)
    q = g.standard_normal((2, tq, hq, 128)).astype(F16)
    dq = _t(q)
    out = torch.empty_like(dq)
    if which == "q":
        dq = _four_bytes_on(dq)
    else:
        out = _four_bytes_on(out)
    for window, n_sink in [(100, 70), (9999, 0)]:
        got = isoq.isoq_prefill_attention_window(dq, *map(_t, cache), _t(lens), *map(_t, par), 3, variant, window, n_sink, out=out)
        assert got is out
        ref = S.window_prefill(q, *cache, lens, *par, 3, variant, 1 / np.sqrt(128), window, n_sink)
        _check(got, ref, F16, q, cache[2], cache[3], 1 / np.sqrt(128))


@pytest.mark.parametrize("d,b,hq,hkv", [(128, 10, 4, 2), (128, 60, 3, 1), (256, 26, 2, 2), (256, 40, 8, 2)])
@pytest.mark.parametrize("tmax", [41, 4097])
def test_prefix_on_tcgen05_with_own_caches_of_odd_rooms(d, b, hq, hkv, tmax):
    """The prefix on tcgen05, the rows' own caches (a room that is no multiple
    of 8) on the CUDA cores."""
    g = np.random.default_rng(b + tmax)
    tp = 333
    cache, prefix, par = _cache(g, (b, hkv, tmax), d, 3), _cache(g, (hkv, tp), d, 3), _params(hkv, d, 0)
    q = g.standard_normal((b, hq, d)).astype(F16)
    lens = g.integers(0, tmax + 1, b).astype(np.int32)
    lens[:2] = 0, tmax
    got = isoq.isoq_decode_attention_prefix(_t(q), *map(_t, prefix), _t(np.array([tp], np.int32)), *map(_t, cache), _t(lens),
                                            *map(_t, par), 3, 0)
    rows = [0, 1, 2, b // 2, b - 1]
    ref = S.prefix_decode(q[rows], prefix, tp, *[c[rows] for c in cache], lens[rows], *par, 3, 0, 1 / np.sqrt(d))
    _check(got[rows], ref, F16, q, cache[2], cache[3], 1 / np.sqrt(d))


@pytest.mark.parametrize("d,hq,hkv", [(128, 2, 2), (128, 8, 1), (256, 2, 2), (256, 8, 1)])
def test_prefill_at_positions_next_to_the_largest(d, hq, hkv):
    """Lengths at both ends of int32 (the cache holds the first Tmax tokens of
    so long a row): the positions of a tile's rows do not wrap around."""
    g = np.random.default_rng(d + hq)
    tmax, tq, top = 320, 24, 2 ** 31 - 1
    lens = np.array([top, top - 60, -2 ** 31, 300], np.int32)
    cache, par = _cache(g, (4, hkv, tmax), d, 3), _params(hkv, d, 0)
    q = g.standard_normal((4, tq, hq, d)).astype(F16)
    for window, n_sink in [(top - 150, 0), (top - 100, 33), (top, 0), (64, 10)]:
        got = isoq.isoq_prefill_attention_window(_t(q), *map(_t, cache), _t(lens), *map(_t, par), 3, 0, window, n_sink)
        rows = [0, 11, 23]
        ref = S.window_prefill(q, *cache, lens, *par, 3, 0, 1 / np.sqrt(d), window, n_sink, rows=rows)
        _check(got[:, rows], ref[:, rows], F16, q, cache[2], cache[3], 1 / np.sqrt(d))
        assert not got[2].any()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window", [0, 1])
def test_small_v_norms_of_sinks_behind_an_empty_window(d, window):
    """One sink of norm 0.002 (and, with a window of 1, the query's own token,
    whose score is far lower): the output is the sink's V vector, whatever the
    norms of the chunk's other tokens.  Tolerance as above."""
    g = np.random.default_rng(d)
    tmax, t, tq = 848, 468, 4
    cache, par = _cache(g, (1, 1, tmax), d, 3), _params(1, d, 0)
    cache[2][:], cache[3][:] = 1e-3, 65504
    cache[2][..., 0], cache[3][..., 0] = 16, 0.002
    own = list(range(t - tq, t))
    cache[3][..., own if window else []] = 0.002
    unit_k, unit_v = (O.dequantize(x[0, :, :1], np.ones((1, 1), F16), p, 3, 0, d)[0, 0] for x, p in zip(cache[:2], par))
    q1 = g.standard_normal(d).astype(F16)
    scale = 60 * np.log(2) / (16 * float(q1.astype(np.float64) @ unit_k))
    q = np.tile(q1, (1, tq, 1, 1))
    got = isoq.isoq_prefill_attention_window(_t(q), *map(_t, cache), _t(np.array([t], np.int32)), *map(_t, par), 3, 0, window, 1,
                                             scale=scale)
    assert isoq.isoq_check_device_error() == 0
    ref = float(F16(0.002)) * unit_v
    err = np.abs(got.cpu().numpy().astype(np.float64).reshape(-1, d) - ref)
    assert (err <= f16_half_ulp(ref) + 2.0 ** -15 * float(F16(0.002))).all(), (err.max(), np.abs(ref).max())
