"""GPU parity of the serving operators with their float64 restatement.

Tolerances.  Codes, norms, tables and slots: equal.  Attention, float16
output: the library's bar, 2e-3 plus half a float16 ulp of the value.
Attention, float32 output: a query row's scores are sums of d terms in
float32, |z| <= max s^K ||q|| scale = Z here, so they are off by at most about
(sqrt(d) + 8) 2^-24 Z (independent roundings), a weight by twice that
relative, and the output by 2 (sqrt(d) + 8) 2^-24 Z max s^V plus
2^-21 max s^V for its own sums and the inverse rotation.
"""

import numpy as np
import pytest

import oracle as O
import synth
from isoq_testlib import check_attention
from oracle import serving as S

torch = pytest.importorskip("torch")
import compressed_space_attention_b200 as isoq  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, F32 = np.float16, np.float32


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _cache(g, shape, d, bits):
    """Random codes and heavy-tailed norms of `shape` vectors."""
    rows = [g.integers(0, 256, size=(*shape, d * bits // 8), dtype=np.uint8) for _ in range(2)]
    return [*rows, (np.sqrt(d) * g.lognormal(0, 0.5, shape)).astype(F16), g.lognormal(1.0, 0.5, shape).astype(F16)]


def _params(hkv, d, variant):
    return [O.make_params(d, variant, seed=s, n_heads=hkv) for s in (1, 2)]


def _check(got, ref, dtype, q, nk, nv, scale):
    got = got.cpu().numpy()
    assert isoq.isoq_check_device_error() == 0
    assert got.dtype == dtype and np.isfinite(got).all()
    if dtype == F16:
        check_attention(got, ref, F16)
        return
    d = q.shape[-1]
    z = float(np.max(nk[np.isfinite(nk)], initial=0)) * float(np.linalg.norm(q.astype(np.float64), axis=-1).max()) * scale
    tol = (2 * (np.sqrt(d) + 8) * 2.0 ** -24 * z + 2.0 ** -21) * float(np.max(nv[np.isfinite(nv)], initial=0))
    assert np.abs(got - ref).max() <= tol, (np.abs(got - ref).max(), tol)


def _poison(cache, lens, window, n_sink):
    """NaN and infinite norms, and all-ones codes, at every token no query sees."""
    out = [c.copy() for c in cache]
    for b, t in enumerate(lens):
        t = min(max(int(t), 0), cache[0].shape[2])
        seen = set(S.seen_tokens(t - 1, t, window, n_sink))
        hidden = [j for j in range(cache[0].shape[2]) if j not in seen]
        out[0][b][:, hidden] = out[1][b][:, hidden] = 255
        out[2][b][:, hidden] = np.nan
        out[3][b][:, hidden] = np.inf
    return out


# (dtype, d, bits, Hq, Hkv): both splits, every group rounding, shared heads of 1 to 16
HEADS = [(F16, 128, 3, 8, 8), (F16, 128, 3, 8, 4), (F16, 128, 3, 6, 2), (F16, 128, 3, 16, 2), (F16, 128, 3, 24, 2),
         (F16, 256, 3, 2, 2), (F16, 256, 3, 16, 8), (F16, 256, 3, 5, 1), (F16, 256, 3, 16, 1), (F16, 128, 4, 8, 2),
         (F16, 128, 2, 4, 4), (F16, 512, 3, 4, 2), (F16, 512, 4, 16, 1), (F32, 128, 3, 8, 2), (F32, 256, 4, 6, 2),
         (F32, 512, 2, 3, 1), (F32, 128, 4, 12, 1)]


@pytest.mark.parametrize("dtype,d,bits,hq,hkv", HEADS)
def test_window_decode(dtype, d, bits, hq, hkv):
    """Ragged rows (empty, one token, shorter and longer than window and
    sinks, past the room), sinks inside, beside and apart from the window;
    whatever no query sees is poisoned."""
    g = np.random.default_rng(d + bits + hq)
    tmax = 704
    lens = np.array([0, 1, 5, 64, 300, 511, 704, 9999, -3], np.int32)
    b = len(lens)
    variant = isoq.ISOQ_FAST if hq == 6 else (isoq.ISOQ_PLANAR if hq == 5 else isoq.ISOQ_FULL)
    cache = _cache(g, (b, hkv, tmax), d, bits)
    par = _params(hkv, d, variant)
    q = g.standard_normal((b, hq, d)).astype(dtype)
    scale = 1 / np.sqrt(d)
    for window, n_sink in [(1, 0), (97, 4), (200, 33), (32, 130), (704, 0), (300, 250)]:
        c = _poison(cache, lens, window, n_sink)
        got = isoq.isoq_decode_attention_window(_t(q), *map(_t, c), _t(lens), *map(_t, par), bits, variant, window, n_sink)
        ref = S.window_decode(q, *cache, lens, *par, bits, variant, scale, window, n_sink)
        _check(got, ref, dtype, q, cache[2], cache[3], scale)


@pytest.mark.parametrize("tmax", [1, 7, 33, 263])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_window_decode_odd_rooms_and_norm_offsets(tmax, dtype):
    """Rooms that are no multiple of 8, norms 2 bytes off a 16-byte boundary,
    and a window and sinks that leave rows empty."""
    g = np.random.default_rng(tmax)
    d, bits, hq, hkv, b = 128, 3, 4, 2, 3
    lens = np.array([tmax, max(1, tmax // 2), 1], np.int32)
    cache = _cache(g, (b, hkv, tmax), d, bits)
    par = _params(hkv, d, 0)
    q = g.standard_normal((b, hq, d)).astype(dtype)
    dev = [_t(c) for c in cache]
    for i in (2, 3):   # the same norms, one element into a larger buffer
        flat = torch.empty(dev[i].numel() + 1, dtype=torch.float16, device=DEV)
        flat[1:] = dev[i].reshape(-1)
        dev[i] = flat[1:].view(b, hkv, tmax)
    for window, n_sink in [(0, 0), (0, 3), (5, 0), (tmax, 1), (2 ** 63 - 1, 2 ** 63 - 1)]:
        got = isoq.isoq_decode_attention_window(_t(q), *dev, _t(lens), *map(_t, par), bits, 0, window, n_sink, scale=0.05)
        ref = S.window_decode(q, *cache, lens, *par, bits, 0, 0.05, window, n_sink)
        _check(got, ref, dtype, q, cache[2], cache[3], 0.05)
        if window == 0 and n_sink == 0:
            assert not got.any()


def test_window_of_everything_is_the_plain_decode():
    """window >= Tmax sees what isoq_decode_attention sees."""
    g = np.random.default_rng(3)
    d, bits, hq, hkv, b, tmax = 128, 3, 8, 2, 3, 1000
    lens = np.array([1000, 517, 64], np.int32)
    cache = [_t(c) for c in _cache(g, (b, hkv, tmax), d, bits)]
    par = [_t(p) for p in _params(hkv, d, 0)]
    q = _t(g.standard_normal((b, hq, d)).astype(F16))
    a = isoq.isoq_decode_attention(q, *cache, _t(lens), *par, bits, 0)
    w = isoq.isoq_decode_attention_window(q, *cache, _t(lens), *par, bits, 0, window=1 << 40)
    assert (a.float() - w.float()).abs().max() <= 2e-3


@pytest.mark.parametrize("window,n_sink", [(1024, 4), (4096, 0), (7000, 640)])
def test_window_decode_on_outlier_kv(window, n_sink, prefill_kv):
    """Heavy-tailed K/V with outlier channels, 32,768 tokens, several splits."""
    kv = prefill_kv
    q = synth.queries(1, 32, 128, seed=9)
    lens = np.array([32768 - 37], np.int32)
    cache = [kv["oracle_k"][0][None], kv["oracle_v"][0][None], kv["oracle_k"][1][None], kv["oracle_v"][1][None]]
    par = [kv["params_k"], kv["params_v"]]
    got = isoq.isoq_decode_attention_window(_t(q), *map(_t, cache), _t(lens), *map(_t, par), 3, 0, window, n_sink)
    ref = S.window_decode(q, *cache, lens, *par, 3, 0, 1 / np.sqrt(128), window, n_sink)
    _check(got, ref, F16, q, cache[2], cache[3], 1 / np.sqrt(128))


@pytest.mark.parametrize("dtype,d,bits,hq,hkv", [HEADS[i] for i in (0, 2, 4, 6, 8, 9, 11, 13, 16)])
def test_window_and_paged_decode_in_many_splits(dtype, d, bits, hq, hkv):
    """Lists of seen tokens too long for one cluster: the three launches, sinks
    and window in different splits, rows much shorter than the longest."""
    g = np.random.default_rng(d + bits + hq)
    tmax, p = 6400, 64
    lens = np.array([6400, 5011, 4097, 90, 0], np.int32)
    b = len(lens)
    cache = _cache(g, (b, hkv, tmax), d, bits)
    par = _params(hkv, d, 0)
    q = g.standard_normal((b, hq, d)).astype(dtype)
    scale = 1 / np.sqrt(d)
    n = b * (tmax // p)
    table = g.permutation(n).astype(np.int32).reshape(b, -1)
    pages = [np.empty((n, hkv, p, *c.shape[3:]), c.dtype) for c in cache]
    for i, c in enumerate(cache):
        for r in range(b):
            pages[i][table[r]] = c[r].reshape(hkv, tmax // p, p, *c.shape[3:]).swapaxes(0, 1)
    dev, dpages, dpar, dl = [_t(c) for c in cache], [_t(x) for x in pages], [_t(x) for x in par], _t(lens)
    for window, n_sink in [(4300, 300), (6400, 0)]:
        assert isoq.isoq_decode_window_workspace_size(b, hq, hkv, tmax, d, window, n_sink) > 0
        ref = S.window_decode(q, *cache, lens, *par, bits, 0, scale, window, n_sink)
        got = isoq.isoq_decode_attention_window(_t(q), *dev, dl, *dpar, bits, 0, window, n_sink)
        _check(got, ref, dtype, q, cache[2], cache[3], scale)
        paged = isoq.isoq_paged_decode_attention(_t(q), *dpages, _t(table), dl, *dpar, bits, 0, window=window, n_sink=n_sink)
        _check(paged, ref, dtype, q, cache[2], cache[3], scale)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 4), (128, 8, 4), (128, 8, 2), (128, 16, 2), (256, 4, 4), (256, 16, 2)])
def test_window_prefill(d, hq, hkv):
    """Chunks at the end of ragged rows (one longer than its row), windows that
    end inside a tile, sinks that fill one tile and more; tokens that no
    query sees are poisoned."""
    g = np.random.default_rng(d + hq)
    bits, tmax, tq = 3, 520, 37
    lens = np.array([500, 130, 20, 37], np.int32)
    b = len(lens)
    cache = _cache(g, (b, hkv, tmax), d, bits)
    variant = isoq.ISOQ_FAST if hq == 16 else isoq.ISOQ_FULL
    par = _params(hkv, d, variant)
    q = g.standard_normal((b, tq, hq, d)).astype(F16)
    scale = 1 / np.sqrt(d)
    for window, n_sink in [(1, 0), (50, 4), (200, 70), (64, 64), (9999, 0), (0, 0), (0, 3)]:
        c = [x.copy() for x in cache]
        for i, t in enumerate(lens):
            seen = set()
            for p in range(max(0, t - tq), t):
                seen |= set(S.seen_tokens(p, tmax, window, n_sink))
            hidden = [j for j in range(tmax) if j not in seen]
            c[2][i][:, hidden] = np.nan
            c[3][i][:, hidden] = np.inf
        got = isoq.isoq_prefill_attention_window(_t(q), *map(_t, c), _t(lens), *map(_t, par), bits, variant, window, n_sink)
        ref = S.window_prefill(q, *cache, lens, *par, bits, variant, scale, window, n_sink)
        _check(got, ref, F16, q, cache[2], cache[3], scale)


def test_window_prefill_long_chunk_sampled():
    """1,024 queries over 3,000 tokens: the rows of several tiles, sampled."""
    g = np.random.default_rng(5)
    d, hq, hkv, tq, tmax = 128, 8, 2, 1024, 3000
    lens = np.array([2999], np.int32)
    cache = _cache(g, (1, hkv, tmax), d, 3)
    par = _params(hkv, d, 0)
    q = g.standard_normal((1, tq, hq, d)).astype(F16)
    got = isoq.isoq_prefill_attention_window(_t(q), *map(_t, cache), _t(lens), *map(_t, par), 3, 0, 700, 5)
    rows = [0, 1, 31, 32, 500, 703, 1000, 1023]
    ref = S.window_prefill(q, *cache, lens, *par, 3, 0, 1 / np.sqrt(d), 700, 5, rows=rows)
    _check(got[:, rows], ref[:, rows], F16, q, cache[2], cache[3], 1 / np.sqrt(d))


@pytest.mark.parametrize("dtype,d,bits,hq,hkv", HEADS)
@pytest.mark.parametrize("b", [1, 5])
def test_prefix_decode(dtype, d, bits, hq, hkv, b):
    """A prefix as a view of a larger cache, shorter than its room; own parts
    that are empty, one token and longer."""
    g = np.random.default_rng(d + bits + hq + b)
    tmax, room, tp = 264, 640, 600
    lens = np.array([0, 1, 77, 264, 31][:b] if b > 1 else [130], np.int32)
    variant = isoq.ISOQ_FAST if hq == 6 else isoq.ISOQ_FULL
    cache = _cache(g, (b, hkv, tmax), d, bits)
    prefix = _cache(g, (hkv, room), d, bits)
    par = _params(hkv, d, variant)
    q = g.standard_normal((b, hq, d)).astype(dtype)
    scale = 1 / np.sqrt(d)
    for plen in (0, 1, 333, 600, 5000):
        view = [_t(x)[:, :tp] for x in prefix]
        got = isoq.isoq_decode_attention_prefix(_t(q), *view, _t(np.array([plen], np.int32)), *map(_t, cache), _t(lens),
                                                *map(_t, par), bits, variant)
        ref = S.prefix_decode(q, [x[:, :tp] for x in prefix], plen, *cache, lens, *par, bits, variant, scale)
        _check(got, ref, dtype, q, np.concatenate([prefix[2].ravel(), cache[2].ravel()]),
               np.concatenate([prefix[3].ravel(), cache[3].ravel()]), scale)


@pytest.mark.parametrize("d,hq,hkv,b", [(128, 32, 4, 20), (128, 8, 1, 33), (128, 24, 8, 50), (256, 16, 8, 70),
                                        (256, 8, 2, 100)])
@pytest.mark.parametrize("variant", [isoq.ISOQ_FULL, isoq.ISOQ_FAST])
def test_prefix_decode_of_large_batches(d, hq, hkv, b, variant):
    """Batches whose query rows fill one and several 128-row tiles, on
    heavy-tailed K/V."""
    g = np.random.default_rng(b)
    tp, tmax = 1352, 72
    par = _params(hkv, d, variant)
    kv = synth.student_t_kv(hkv, tp, d, seed=b)
    k, nk = O.quantize(kv[0][0].astype(np.float64), par[0], 3, variant)
    v, nv = O.quantize(kv[1][0].astype(np.float64), par[1], 3, variant)
    prefix = [k, v, nk, nv]
    cache = _cache(g, (b, hkv, tmax), d, 3)
    lens = g.integers(0, tmax + 1, b).astype(np.int32)
    q = synth.queries(b, hq, d, seed=b + 1)
    plen = np.array([tp - 5], np.int32)
    got = isoq.isoq_decode_attention_prefix(_t(q), *map(_t, prefix), _t(plen), *map(_t, cache), _t(lens), *map(_t, par), 3,
                                            variant)
    rows = sorted(set([0, 1, b // 2, b - 2, b - 1]))
    ref = S.prefix_decode(q[rows], prefix, plen[0], *[c[rows] for c in cache], lens[rows], *par, 3, variant,
                          1 / np.sqrt(d))
    _check(got[rows], ref, F16, q, cache[2], cache[3], 1 / np.sqrt(d))


def test_prefix_of_nothing_and_empty_rows():
    g = np.random.default_rng(8)
    d, hq, hkv, b, tmax = 128, 4, 2, 2, 64
    cache = [_t(c) for c in _cache(g, (b, hkv, tmax), d, 3)]
    par = [_t(p) for p in _params(hkv, d, 0)]
    q = _t(g.standard_normal((b, hq, d)).astype(F16))
    none = [torch.empty(s, dtype=t, device=DEV) for s, t in (((hkv, 0, 48), torch.uint8), ((hkv, 0, 48), torch.uint8),
                                                             ((hkv, 0), torch.float16), ((hkv, 0), torch.float16))]
    zero, lens = torch.zeros(1, dtype=torch.int32, device=DEV), torch.tensor([64, 0], dtype=torch.int32, device=DEV)
    got = isoq.isoq_decode_attention_prefix(q, *none, zero, *cache, lens, *par, 3, 0)
    ref = isoq.isoq_decode_attention(q, *cache, lens, *par, 3, 0)
    assert isoq.isoq_check_device_error() == 0
    assert (got.float() - ref.float()).abs().max() <= 2e-3 and not got[1].any()


def _pages(g, lens, hkv, d, bits, p, max_pages, spare=3):
    """Shuffled pages behind a table whose unused entries are out of range."""
    need = [-(-max(int(t), 0) // p) for t in lens]
    n = sum(need) + spare
    ids = g.permutation(n).astype(np.int32)
    table = np.full((len(lens), max_pages), 1 << 30, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :min(k, max_pages)] = ids[at:at + min(k, max_pages)]
        at += k
    return _cache(g, (n, hkv, p), d, bits), table


@pytest.mark.parametrize("p", [16, 32, 64, 256])
@pytest.mark.parametrize("dtype,d,bits,hq,hkv", [HEADS[i] for i in (0, 2, 4, 6, 8, 9, 11, 13, 16)])
def test_paged_decode(dtype, d, bits, hq, hkv, p):
    """Rows that end inside a page and a tile; the table's unused entries are
    never followed; windows and sinks over pages."""
    g = np.random.default_rng(p + d + hq)
    lens = np.array([0, 1, 16, 33, 400, 517, 640], np.int32)
    max_pages = -(-640 // p)
    pages, table = _pages(g, lens, hkv, d, bits, p, max_pages)
    par = _params(hkv, d, 0)
    q = g.standard_normal((len(lens), hq, d)).astype(dtype)
    scale = 1 / np.sqrt(d)
    dev = [_t(x) for x in pages]
    for max_len, window, n_sink in [(None, None, 0), (520, None, 0), (None, 90, 5), (640, 250, 70)]:
        got = isoq.isoq_paged_decode_attention(_t(q), *dev, _t(table), _t(lens), *map(_t, par), bits, 0, max_len=max_len,
                                               window=window, n_sink=n_sink)
        ref = S.paged_decode(q, pages, table, lens, *par, bits, 0, scale, max_len or max_pages * p,
                             window if window is not None else 1 << 30, n_sink)
        _check(got, ref, dtype, q, pages[2], pages[3], scale)


@pytest.mark.parametrize("dtype,bits", [(F16, 3), (F32, 4)])
def test_bad_pages_are_reported(dtype, bits):
    """A page index out of range in one row: the error word says so, the other
    rows are right."""
    g = np.random.default_rng(1)
    lens = np.array([100, 200], np.int32)
    pages, table = _pages(g, lens, 2, 128, bits, 32, 8)
    bad = table.copy()
    bad[0, 2] = -7
    par = _params(2, 128, 0)
    q = g.standard_normal((2, 4, 128)).astype(dtype)
    got = isoq.isoq_paged_decode_attention(_t(q), *map(_t, pages), _t(bad), _t(lens), *map(_t, par), bits, 0)
    assert isoq.isoq_check_device_error() == isoq.ISOQ_ERR_INVALID_ARG
    assert isoq.isoq_check_device_error() == 0
    ref = S.paged_decode(q, pages, table, lens, *par, bits, 0, 1 / np.sqrt(128), 256, 1 << 30, 0)
    _check(got[1:], ref[1:], dtype, q, pages[2], pages[3], 1 / np.sqrt(128))


@pytest.mark.parametrize("seed", range(6))
def test_block_tables(seed):
    """Random steps, decode steps, rows that do not fit, a slot map with room
    to spare and one that is too short; more requests than one pass holds."""
    g = np.random.default_rng(seed)
    b = [1, 7, 64, 300, 1025, 2500][seed]
    p = [16, 64, 32, 16, 128, 256][seed]
    cols = int(g.integers(3, 40))
    lens = g.integers(-2, cols * p, b).astype(np.int32)
    new = np.where(g.random(b) < 0.5, 1, g.integers(0, 3 * p, b)).astype(np.int32)
    if seed >= 3:
        new[g.integers(0, b, 3)] = -1
        lens[g.integers(0, b, 3)] = cols * p
    total = int(np.maximum(new, 0).sum())
    need = int((-(-(np.maximum(lens, 0) + np.maximum(new, 0)) // p) - -(-np.maximum(lens, 0) // p)).sum())
    for n_slots, n_free, head in [(total + 100, need + 5, 0), (max(total - 7, 0), need + 9, 3), (total, need // 2, 0)]:
        free = g.permutation(n_free + 10000)[:n_free].astype(np.int32)
        table = g.integers(0, 10000, (b, cols)).astype(np.int32)
        dt = _t(table)
        hd = torch.tensor([head], dtype=torch.int32, device=DEV)
        slot, start, tot, used = isoq.isoq_build_block_tables(_t(lens), _t(new), _t(free), dt, p, n_slots, free_head=hd)
        r = S.block_tables(lens, new, free, p, table, n_slots, head)
        np.testing.assert_array_equal(dt.cpu().numpy(), r[0])
        np.testing.assert_array_equal(slot.cpu().numpy(), r[1])
        np.testing.assert_array_equal(start.cpu().numpy(), r[2])
        np.testing.assert_array_equal(tot.cpu().numpy(), r[3])
        assert int(used) == r[4]
        assert isoq.isoq_check_device_error() == (isoq.ISOQ_ERR_INVALID_ARG if r[5] else 0)


@pytest.mark.parametrize("variant", [isoq.ISOQ_FULL, isoq.ISOQ_FAST, isoq.ISOQ_PLANAR])
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d,bits", [(128, 2), (128, 3), (128, 4), (256, 2), (256, 3), (256, 4), (512, 2), (512, 3), (512, 4)])
def test_paged_append_is_exact(variant, dtype, d, bits):
    """Heavy-tailed tokens, a zero vector, skipped and out-of-range slots: the
    pages are the restatement's bit for bit, and nothing else is written."""
    g = np.random.default_rng(d + bits)
    n, hkv, p, n_pages = 150, 2, 16, 13
    kv = [x[0].transpose(1, 0, 2).copy() for x in synth.student_t_kv(hkv, n, d, seed=d + bits, dtype=dtype)]
    kv[0][7] = 0
    slot = g.permutation(n_pages * p)[:n].astype(np.int64)
    slot[[3, 50]] = -1
    slot[[60, 61]] = [n_pages * p, 1 << 40]
    pages = _cache(g, (n_pages, hkv, p), d, bits)
    par = _params(hkv, d, variant)
    dev = [_t(x) for x in pages]
    isoq.isoq_paged_append(_t(kv[0]), _t(kv[1]), *dev, _t(slot), *map(_t, par), bits, variant)
    assert isoq.isoq_check_device_error() == isoq.ISOQ_ERR_INVALID_ARG   # the two slots beyond the pages
    ref = S.paged_append(kv[0], kv[1], pages, slot, *par, bits, variant)
    for got, want in zip(dev, ref):
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))


@pytest.mark.parametrize("d,bits", [(128, 3), (256, 4), (512, 3)])
def test_paged_append_decides_next_to_thresholds(d, bits):
    """Vectors most of whose rotated coordinates lie within a few float32
    roundings of a threshold, and norms next to float16 rounding boundaries:
    the codes and norms are still the float64 ones."""
    g = np.random.default_rng(d)
    n, hkv, p = 64, 2, 64
    par = _params(hkv, d, 0)
    _, thr = O.make_codebook(d, bits)
    kv = []
    for which in (0, 1):
        x = np.empty((n, hkv, d), F32)
        for h in range(hkv):
            for i in range(n):
                # coordinates at thresholds, the rest scaled so that the norm is 1
                y = thr[g.integers(0, len(thr), d)]
                free = slice(0, d // 4)
                y[free] = 0
                rest = 1 - (y ** 2).sum()
                if rest <= 0:
                    y *= 0.9 / np.linalg.norm(y)
                    rest = 1 - (y ** 2).sum()
                u = g.standard_normal(d // 4)
                y[free] = u * np.sqrt(rest) / np.linalg.norm(u)
                s = 10 * (1 + 2.0 ** -11 * (2 * g.integers(0, 500) + 1))
                x[i, h] = (s * O.rotate_inverse(y, par[which][h], 0)).astype(F32)
        kv.append(x)
    slot = g.permutation(n).astype(np.int64)
    pages = _cache(g, (1, hkv, p), d, bits)
    dev = [_t(a) for a in pages]
    isoq.isoq_paged_append(_t(kv[0]), _t(kv[1]), *dev, _t(slot), *map(_t, par), bits, 0)
    assert isoq.isoq_check_device_error() == 0
    for got, want in zip(dev, S.paged_append(kv[0], kv[1], pages, slot, *par, bits, 0)):
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))


def test_paged_append_of_extreme_magnitudes():
    """float32 vectors whose squares under- or overflow float32."""
    g = np.random.default_rng(2)
    d, hkv, p = 128, 1, 16
    x = g.standard_normal((4, hkv, d))
    x = (x * np.array([1e-25, 1e-18, 1e20, 1e17])[:, None, None]).astype(F32)
    par = _params(hkv, d, 0)
    pages = _cache(g, (1, hkv, p), d, 3)
    dev = [_t(a) for a in pages]
    slot = np.arange(4, dtype=np.int64)
    isoq.isoq_paged_append(_t(x), _t(x), *dev, _t(slot), *map(_t, par), 3, 0)
    with np.errstate(over="ignore"):
        ref = S.paged_append(x, x, pages, slot, *par, 3, 0)
    for got, want in zip(dev, ref):
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))


def _serve(g, d, hq, hkv, b, p, bits, dtype):
    """A paged server: prompts, then decode steps, all through one set of pages."""
    max_len = 200
    cols = -(-max_len // p)
    n_pages = b * cols
    par = _params(hkv, d, 0)
    pages = _cache(g, (n_pages, hkv, p), d, bits)
    free = g.permutation(n_pages).astype(np.int32)
    return dict(par=par, pages=pages, free=free, cols=cols, max_len=max_len)


@pytest.mark.parametrize("dtype,d,bits,hq,hkv,p", [(F16, 128, 3, 8, 2, 16), (F32, 128, 4, 6, 2, 32), (F16, 256, 3, 4, 4, 64)])
def test_a_paged_server_runs(dtype, d, bits, hq, hkv, p):
    """Tables, append and attention together, as a server runs them: prompts of
    different lengths, then decode steps, each checked with the restatement."""
    g = np.random.default_rng(p)
    b = 5
    sv = _serve(g, d, hq, hkv, b, p, bits, dtype)
    pages, par, free = [x.copy() for x in sv["pages"]], sv["par"], sv["free"]
    table = np.full((b, sv["cols"]), -1, np.int32)
    dev, dtab, dpar, dfree = [_t(x) for x in pages], _t(table), [_t(x) for x in par], _t(free)
    lens_d = torch.zeros(b, dtype=torch.int32, device=DEV)
    head_d = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens, head = np.zeros(b, np.int32), 0
    for step in range(5):
        new = g.integers(0, 150, b).astype(np.int32) if step == 0 else np.ones(b, np.int32)
        n = int(new.sum()) + 3     # padded, as a captured step is
        kv = g.standard_normal((2, n, hkv, d)).astype(dtype)
        q = g.standard_normal((b, hq, d)).astype(dtype)
        slot, _, lens_d, used = isoq.isoq_build_block_tables(lens_d, _t(new), dfree, dtab, p, n, free_head=head_d)
        head_d = head_d + used
        isoq.isoq_paged_append(_t(kv[0]), _t(kv[1]), *dev, slot, *dpar, bits, 0)
        got = isoq.isoq_paged_decode_attention(_t(q), *dev, dtab, lens_d, *dpar, bits, 0, max_len=sv["max_len"])
        table, rslot, _, lens, rused, failed = S.block_tables(lens, new, free, p, table, n, head)
        head += rused
        pages = list(S.paged_append(kv[0], kv[1], pages, rslot, *par, bits, 0))
        assert not failed and int(head_d) == head
        np.testing.assert_array_equal(dtab.cpu().numpy(), table)
        for x, y in zip(dev, pages):
            np.testing.assert_array_equal(x.cpu().numpy().view(np.uint8), y.view(np.uint8))
        ref = S.paged_decode(q, pages, table, lens, *par, bits, 0, 1 / np.sqrt(d), sv["max_len"], 1 << 30, 0)
        _check(got, ref, dtype, q, pages[2], pages[3], 1 / np.sqrt(d))


def test_captured_and_replayed_on_other_streams():
    """Window, prefix and paged decode captured into graphs that share one
    workspace, replayed in turn on another stream with new inputs: the same
    bits as eager calls, every time."""
    g = np.random.default_rng(4)
    d, hq, hkv, b, tmax, p = 128, 8, 2, 3, 512, 32
    lens = np.array([512, 100, 333], np.int32)
    cache = [_t(c) for c in _cache(g, (b, hkv, tmax), d, 3)]
    prefix = [_t(c) for c in _cache(g, (hkv, 256), d, 3)]
    pages, table = _pages(g, lens, hkv, d, 3, p, 16)
    pages, table = [_t(x) for x in pages], _t(table)
    par = [_t(x) for x in _params(hkv, d, 0)]
    q, dl = torch.empty(b, hq, d, dtype=torch.float16, device=DEV), _t(lens)
    plen = torch.tensor([200], dtype=torch.int32, device=DEV)
    n = max(isoq.isoq_decode_window_workspace_size(b, hq, hkv, tmax, d, tmax, 0),
            isoq.isoq_decode_prefix_workspace_size(b, hq, hkv, 256, tmax, d))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    calls = [lambda o: isoq.isoq_decode_attention_window(q, *cache, dl, *par, 3, 0, 100, 4, out=o, workspace=ws),
             lambda o: isoq.isoq_decode_attention_prefix(q, *prefix, plen, *cache, dl, *par, 3, 0, out=o, workspace=ws),
             lambda o: isoq.isoq_paged_decode_attention(q, *pages, table, dl, *par, 3, 0, out=o, workspace=ws)]
    q.normal_()
    outs = [torch.empty_like(q) for _ in calls]
    for f, o in zip(calls, outs):
        f(o)
    torch.cuda.synchronize()
    graphs = []
    for f, o in zip(calls, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f(o)
        graphs.append(gr)
    other = torch.cuda.Stream()
    for seed in range(3):
        torch.manual_seed(seed)
        q.normal_()
        eager = [f(torch.empty_like(q)).clone() for f in calls]
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            for gr in graphs:
                gr.replay()
            again = [f(torch.empty_like(q)) for f in calls]
        other.synchronize()
        for a, o, e in zip(again, outs, eager):
            assert torch.equal(o, e) and torch.equal(a, e)
    assert isoq.isoq_check_device_error() == 0


def test_outputs_and_workspaces_end_where_they_say():
    """Sentinels behind the output and the workspace stay."""
    g = np.random.default_rng(6)
    d, hq, hkv, b, tmax = 128, 6, 2, 3, 9000
    cache = [_t(c) for c in _cache(g, (b, hkv, tmax), d, 4)]
    par = [_t(x) for x in _params(hkv, d, 0)]
    q = _t(g.standard_normal((b, hq, d)).astype(F32))
    lens = _t(np.array([9000, 2, 250], np.int32))
    n = isoq.isoq_decode_window_workspace_size(b, hq, hkv, tmax, d, 8000, 7)
    ws = torch.full((n + 256,), 77, dtype=torch.uint8, device=DEV)
    out = torch.full((b + 1, hq, d), 5.0, device=DEV)
    isoq.isoq_decode_attention_window(q, *cache, lens, *par, 4, 0, 8000, 7, out=out[:b], workspace=ws[:n])
    assert (ws[n:] == 77).all() and (out[b] == 5).all() and (out[:b] != 5).all()
    with pytest.raises(isoq.IsoqError, match="workspace too small"):
        isoq.isoq_decode_attention_window(q, *cache, lens, *par, 4, 0, 8000, 7, workspace=ws[:n - 256])


@pytest.mark.parametrize("dtype,d,bits,hq,hkv", [(F16, 128, 3, 8, 2), (F16, 256, 3, 4, 2), (F32, 128, 4, 6, 2)])
@pytest.mark.parametrize("p", [16, 64])
def test_what_lies_behind_a_row_is_ignored(dtype, d, bits, hq, hkv, p):
    """NaN and infinite norms behind each row's end, in its last page and in the
    pages of no row, and behind the prefix's length."""
    g = np.random.default_rng(p + d)
    lens = np.array([1, 37, 130, 0], np.int32)
    b, tmax, room = len(lens), 160, 96
    pages, table = _pages(g, lens, hkv, d, bits, p, -(-tmax // p))
    cache, prefix = _cache(g, (b, hkv, tmax), d, bits), _cache(g, (hkv, room), d, bits)
    par = _params(hkv, d, 0)
    q = g.standard_normal((b, hq, d)).astype(dtype)
    scale = 1 / np.sqrt(d)
    bad_pages, bad_cache, bad_prefix = ([x.copy() for x in c] for c in (pages, cache, prefix))
    used = np.zeros(pages[0].shape[0] * p, bool)
    for i, t in enumerate(lens):
        for j in range(t):
            used[table[i, j // p] * p + j % p] = True
        bad_cache[2][i][:, t:], bad_cache[3][i][:, t:] = np.nan, np.inf
    off = ~used.reshape(-1, p)
    for h in range(hkv):
        bad_pages[2][:, h][off], bad_pages[3][:, h][off] = np.inf, np.nan
    bad_prefix[2][:, 61:], bad_prefix[3][:, 61:] = np.nan, np.inf
    dl, dp = _t(lens), [_t(x) for x in par]
    got = isoq.isoq_paged_decode_attention(_t(q), *map(_t, bad_pages), _t(table), dl, *dp, bits, 0)
    _check(got, S.paged_decode(q, pages, table, lens, *par, bits, 0, scale, tmax, 1 << 30, 0), dtype, q, pages[2], pages[3], scale)
    got = isoq.isoq_decode_attention_prefix(_t(q), *map(_t, bad_prefix), _t(np.array([61], np.int32)), *map(_t, bad_cache), dl,
                                            *dp, bits, 0)
    _check(got, S.prefix_decode(q, prefix, 61, *cache, lens, *par, bits, 0, scale), dtype, q,
           np.concatenate([prefix[2].ravel(), cache[2].ravel()]), np.concatenate([prefix[3].ravel(), cache[3].ravel()]), scale)


def test_two_calls_at_once_and_the_same_bits_every_time():
    """Calls on two streams at once, each with its own output: the bits of the
    same calls one after the other, and of a second round."""
    g = np.random.default_rng(12)
    d, hq, hkv, b, tmax = 128, 32, 4, 6, 6144
    lens = np.full(b, 6000, np.int32)
    cache, prefix = [_t(c) for c in _cache(g, (b, hkv, tmax), d, 3)], [_t(c) for c in _cache(g, (hkv, 4096), d, 3)]
    par, dl = [_t(x) for x in _params(hkv, d, 0)], _t(lens)
    plen = torch.tensor([4000], dtype=torch.int32, device=DEV)
    q = _t(g.standard_normal((b, hq, d)).astype(F16))
    qc = _t(g.standard_normal((b, 40, hq, d)).astype(F16))
    calls = [lambda: isoq.isoq_decode_attention_window(q, *cache, dl, *par, 3, 0, 5000, 64),
             lambda: isoq.isoq_decode_attention_window(q, *cache, dl, *par, 3, 0, 700, 3),
             lambda: isoq.isoq_decode_attention_prefix(q, *prefix, plen, *cache, dl, *par, 3, 0),
             lambda: isoq.isoq_prefill_attention_window(qc, *cache, dl, *par, 3, 0, 600, 5)]
    alone = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        outs = []
        for s, f in zip(streams, calls):
            with torch.cuda.stream(s):
                outs.append(f())
        torch.cuda.synchronize()
        for a, o in zip(alone, outs):
            assert torch.equal(a, o)
    assert isoq.isoq_check_device_error() == 0


def test_offsets_beyond_32_bits():
    """Pages and rows more than 4 GiB into their pool: the bits of the same
    tokens in a small one."""
    g = np.random.default_rng(13)
    d, bits, hq, hkv, p, b = 256, 3, 16, 8, 256, 2
    lens = np.array([700, 300], np.int32)
    small = [_t(x) for x in _cache(g, (6, hkv, p), d, bits)]
    table = _t(np.array([[0, 1, 2], [3, 4, 5]], np.int32))
    n = 24000                                    # 4.7 GB of packed K
    large = [torch.empty((n, *x.shape[1:]), dtype=x.dtype, device=DEV) for x in small]
    for x, y in zip(large, small):
        x[-6:] = y
    par, dl = [_t(x) for x in _params(hkv, d, 0)], _t(lens)
    for dtype in (F16, F32):
        q = _t(g.standard_normal((b, hq, d)).astype(dtype))
        a = isoq.isoq_paged_decode_attention(q, *small, table, dl, *par, bits, 0)
        c = isoq.isoq_paged_decode_attention(q, *large, table + (n - 6), dl, *par, bits, 0)
        assert torch.equal(a, c)
    kv = _t(g.standard_normal((2, 3, hkv, d)).astype(F16))
    slot = torch.tensor([5, 700, 1100], dtype=torch.int64, device=DEV)
    isoq.isoq_paged_append(kv[0], kv[1], *small, slot, *par, bits, 0)
    isoq.isoq_paged_append(kv[0], kv[1], *large, slot + (n - 6) * p, *par, bits, 0)
    for x, y in zip(large, small):
        assert torch.equal(x[-6:].contiguous().view(torch.uint8), y.view(torch.uint8))
    del large
    # one row of 6.3 million tokens x 8 heads, of which the last are seen
    t, near = 6291456, 640
    row = [torch.empty((1, hkv, t, *x.shape[3:]), dtype=x.dtype, device=DEV) for x in small]
    tail = [x.reshape(6, hkv, p, *x.shape[3:])[:3].transpose(0, 1).reshape(1, hkv, 3 * p, *x.shape[3:]).contiguous() for x in small]
    for x, y in zip(row, tail):
        x[:, :, -3 * p:] = y
    q = _t(g.standard_normal((1, hq, d)).astype(F16))
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    a = isoq.isoq_decode_attention_window(q, *tail, one * (3 * p), *par, bits, 0, near)
    c = isoq.isoq_decode_attention_window(q, *row, one * t, *par, bits, 0, near)
    assert torch.equal(a, c)
    qc = _t(g.standard_normal((1, 20, hq, d)).astype(F16))
    a = isoq.isoq_prefill_attention_window(qc, *tail, one * (3 * p), *par, bits, 0, near)
    c = isoq.isoq_prefill_attention_window(qc, *row, one * t, *par, bits, 0, near)
    assert (a.float() - c.float()).abs().max() <= 2e-3
    assert isoq.isoq_check_device_error() == 0


def test_append_of_a_slot_map_longer_than_the_tokens():
    g = np.random.default_rng(14)
    pages = _cache(g, (2, 1, 16), 128, 3)
    dev, par = [_t(x) for x in pages], _params(1, 128, 0)
    kv = g.standard_normal((2, 3, 1, 128)).astype(F16)
    slot = np.array([4, -1, 31, 9, 9], np.int64)
    isoq.isoq_paged_append(_t(kv[0]), _t(kv[1]), *dev, _t(slot), *map(_t, par), 3, 0)
    isoq.isoq_paged_append(_t(kv[0][:0]), _t(kv[1][:0]), *dev, _t(slot), *map(_t, par), 3, 0)
    assert isoq.isoq_check_device_error() == 0
    for got, want in zip(dev, S.paged_append(kv[0], kv[1], pages, slot[:3], *par, 3, 0)):
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))


def test_block_tables_of_lengths_near_the_largest():
    """Lengths and sums of new tokens next to and beyond 2^31: those requests
    do not fit, and nothing overflows."""
    free = np.arange(8, dtype=np.int32)
    lens = np.array([2 ** 31 - 1, 2 ** 31 - 200, 10, 0], np.int32)
    new = np.array([1, 150, 2 ** 31 - 1, 3], np.int32)
    table = np.full((4, 2), 5, np.int32)
    dt = _t(table)
    out = isoq.isoq_build_block_tables(_t(lens), _t(new), _t(free), dt, 256, 2000)
    ref = S.block_tables(lens, new, free, 256, table, 2000)
    assert isoq.isoq_check_device_error() == isoq.ISOQ_ERR_INVALID_ARG
    np.testing.assert_array_equal(dt.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(out[0].cpu().numpy(), ref[1])
    np.testing.assert_array_equal(out[1].cpu().numpy(), ref[2])
    np.testing.assert_array_equal(out[2].cpu().numpy(), ref[3])
    assert int(out[3]) == ref[4]
