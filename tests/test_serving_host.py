"""The serving entry points on the host: their refusals come before any
device work, their workspace sizes follow the shapes, and the float64
restatement agrees with ordinary attention over the reconstructed cache."""

import math

import numpy as np
import pytest

import oracle as O
from oracle import serving as S

import compressed_space_attention_b200 as isoq

P = 1 << 20      # a well-aligned address that is never dereferenced on the host
BAD, UNSUP = isoq.ISOQ_ERR_INVALID_ARG, isoq.ISOQ_ERR_UNSUPPORTED
D128 = dict(q=P, dtype=0, pk=P, pv=P, nk=P, nv=P, lens=P, B=2, Hq=8, Hkv=2, Tmax=256, d=128, bits=3, variant=0, prk=P,
            prv=P, scale=0.1, window=64, n_sink=4, out=P, ws=P, ws_bytes=1 << 40)


def _window(**kw):
    a = {**D128, "window": 16384, "Tmax": 1 << 15, **kw}
    return isoq.lib().isoq_decode_attention_window(
        a["q"], a["dtype"], a["pk"], a["pv"], a["nk"], a["nv"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["Tmax"], a["d"],
        a["bits"], a["variant"], a["prk"], a["prv"], a["scale"], a["window"], a["n_sink"], a["out"], a["ws"],
        a["ws_bytes"], None)


def _prefill(**kw):
    a = {**D128, "Tq": 4, **kw}
    return isoq.lib().isoq_prefill_attention_window(
        a["q"], a["dtype"], a["pk"], a["pv"], a["nk"], a["nv"], a["lens"], a["B"], a["Tq"], a["Hq"], a["Hkv"], a["Tmax"],
        a["d"], a["bits"], a["variant"], a["prk"], a["prv"], a["scale"], a["window"], a["n_sink"], a["out"], None)


def _prefix(**kw):
    a = {**D128, "xk": P, "xv": P, "xnk": P, "xnv": P, "xlen": P, "Tp": 512, "stride": 512, **kw}
    return isoq.lib().isoq_decode_attention_prefix(
        a["q"], a["dtype"], a["xk"], a["xv"], a["xnk"], a["xnv"], a["xlen"], a["Tp"], a["stride"], a["pk"], a["pv"],
        a["nk"], a["nv"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["Tmax"], a["d"], a["bits"], a["variant"], a["prk"],
        a["prv"], a["scale"], a["out"], a["ws"], a["ws_bytes"], None)


def _paged(**kw):
    a = {**D128, "window": 1 << 15, "Tmax": 1 << 15, "table": P, "n_pages": 64, "page": 16, "max_pages": 2048, **kw}
    return isoq.lib().isoq_paged_decode_attention(
        a["q"], a["dtype"], a["pk"], a["pv"], a["nk"], a["nv"], a["table"], a["lens"], a["B"], a["Hq"], a["Hkv"],
        a["n_pages"], a["page"], a["max_pages"], a["Tmax"], a["d"], a["bits"], a["variant"], a["prk"], a["prv"],
        a["scale"], a["window"], a["n_sink"], a["out"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [_window, _prefill, _prefix, _paged])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(pk=None), BAD), (dict(nv=None), BAD), (dict(lens=None), BAD), (dict(prv=None), BAD),
    (dict(out=None), BAD), (dict(B=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=9), BAD), (dict(Tmax=0), BAD),
    (dict(Tmax=1 << 31), BAD), (dict(d=64), UNSUP), (dict(bits=5), UNSUP), (dict(variant=3), UNSUP),
    (dict(dtype=2), UNSUP), (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(pk=P + 8), UNSUP),
    (dict(prk=P + 4), UNSUP), (dict(lens=P + 2), UNSUP), (dict(B=65536), BAD)])
def test_attention_refusals(call, kw, status):
    assert call(**kw) == status
    assert isoq.last_error()


@pytest.mark.parametrize("call", [_window, _prefill, _paged])
@pytest.mark.parametrize("kw", [dict(window=-1), dict(n_sink=-1)])
def test_window_refusals(call, kw):
    assert call(**kw) == BAD


@pytest.mark.parametrize("call", [_window, _prefix, _paged])
@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=P + 128), dict(ws_bytes=1024), dict(Hq=34)])
def test_workspace_refusals(call, kw):
    assert call(**kw) == (UNSUP if "Hq" in kw else BAD)


@pytest.mark.parametrize("kw,status", [
    (dict(Tp=-1), BAD), (dict(Tp=1 << 31, stride=1 << 31), BAD), (dict(stride=511), BAD), (dict(xk=None), BAD),
    (dict(xnv=None), BAD), (dict(xlen=None), BAD), (dict(xk=P + 8), UNSUP), (dict(xnk=P + 1), UNSUP)])
def test_prefix_refusals(kw, status):
    assert _prefix(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(page=8), UNSUP), (dict(page=48), UNSUP), (dict(page=512), UNSUP), (dict(n_pages=0), BAD),
    (dict(max_pages=0), BAD), (dict(max_pages=2047), BAD), (dict(table=None), BAD), (dict(table=P + 2), UNSUP)])
def test_paged_refusals(kw, status):
    assert _paged(**kw) == status


def _append(**kw):
    a = dict(k=P, v=P, dtype=0, pk=P, pv=P, nk=P, nv=P, slot=P, N=4, Hkv=2, n_pages=8, page=16, d=128, bits=3, variant=0,
             prk=P, prv=P)
    a.update(kw)
    return isoq.lib().isoq_paged_append(a["k"], a["v"], a["dtype"], a["pk"], a["pv"], a["nk"], a["nv"], a["slot"], a["N"],
                                        a["Hkv"], a["n_pages"], a["page"], a["d"], a["bits"], a["variant"], a["prk"],
                                        a["prv"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), BAD), (dict(slot=None), BAD), (dict(N=-1), BAD), (dict(Hkv=0), BAD), (dict(n_pages=0), BAD),
    (dict(N=1 << 31), BAD), (dict(page=24), UNSUP), (dict(d=96), UNSUP), (dict(bits=1), UNSUP), (dict(variant=4), UNSUP),
    (dict(dtype=7), UNSUP), (dict(k=P + 8), UNSUP), (dict(pv=P + 8), UNSUP), (dict(slot=P + 4), UNSUP)])
def test_append_refusals(kw, status):
    assert _append(**kw) == status


def test_append_of_nothing_is_a_no_op():
    assert _append(N=0) == isoq.ISOQ_OK


def _tables(**kw):
    a = dict(lens=P, new=2 * P, free=3 * P, head=None, n_free=10, B=4, page=16, max_pages=8, table=4 * P, n_slots=32,
             slots=5 * P, start=6 * P, total=7 * P, used=8 * P)
    a.update(kw)
    return isoq.lib().isoq_build_block_tables(a["lens"], a["new"], a["free"], a["head"], a["n_free"], a["B"], a["page"],
                                              a["max_pages"], a["table"], a["n_slots"], a["slots"], a["start"],
                                              a["total"], a["used"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(lens=None), BAD), (dict(free=None), BAD), (dict(table=None), BAD), (dict(slots=None), BAD),
    (dict(used=None), BAD), (dict(B=0), BAD), (dict(max_pages=0), BAD), (dict(n_free=-1), BAD), (dict(n_slots=-1), BAD),
    (dict(page=20), UNSUP), (dict(slots=P + 4), UNSUP), (dict(total=P), BAD), (dict(total=P + 12), BAD),
    (dict(start=6 * P, used=6 * P + 16), BAD), (dict(free=4 * P + 64), BAD), (dict(head=5 * P + 8), BAD)])
def test_block_table_refusals(kw, status):
    assert _tables(**kw) == status


def test_workspace_sizes():
    w = isoq.isoq_decode_window_workspace_size
    assert w(0, 8, 2, 256, 128, 64, 4) == 0 and w(2, 9, 2, 256, 128, 64, 4) == 0 and w(2, 8, 2, 256, 96, 64, 4) == 0
    assert w(2, 8, 2, 256, 128, -1, 0) == 0
    small, large = w(1, 8, 2, 1 << 20, 128, 8192, 4), w(1, 8, 2, 1 << 20, 128, 1 << 20, 0)
    assert 0 < small < large and small % 256 == 0
    # the work of a window does not follow the room of the cache
    assert small == w(1, 8, 2, 1 << 24, 128, 8192, 4)
    # windows and sinks beyond the room are the room, up to the largest integer
    assert w(3, 8, 2, 9000, 128, 2 ** 63 - 1, 2 ** 63 - 1) == w(3, 8, 2, 9000, 128, 9000, 0)
    # a list of seen tokens that one cluster holds needs none
    assert w(1, 8, 2, 1 << 24, 128, 256, 4) == 0 and w(300, 8, 2, 1 << 24, 128, 256, 4) > 0
    x = isoq.isoq_decode_prefix_workspace_size
    assert x(2, 8, 2, 0, 256, 128) > 0 and x(2, 8, 2, -1, 256, 128) == 0 and x(2, 8, 2, 64, 0, 128) == 0


def _cache(g, shape, d, bits):
    return (g.integers(0, 256, size=(*shape, d * bits // 8), dtype=np.uint8),
            g.integers(0, 256, size=(*shape, d * bits // 8), dtype=np.uint8),
            g.lognormal(1.5, 0.4, shape).astype(np.float16), g.lognormal(1.0, 0.4, shape).astype(np.float16))


def test_restated_window_agrees_with_reconstructed_attention():
    g = np.random.default_rng(0)
    c = _cache(g, (2, 2, 40), 128, 3)
    pr = [O.make_params(128, O.FULL, seed=s, n_heads=2) for s in (1, 2)]
    q = g.standard_normal((2, 4, 128))
    a = (*c, [40, 23], *pr, 3, O.FULL, 0.1, 9, 2)
    np.testing.assert_allclose(S.window_decode(q, *a), S.window_decode(q, *a, reconstructed=True), atol=1e-5)


def test_restated_seen_tokens():
    assert S.seen_tokens(9, 10, 3, 2) == [0, 1, 7, 8, 9]
    assert S.seen_tokens(9, 10, 0, 0) == [] and S.seen_tokens(9, 10, 0, 1) == [0]
    assert S.seen_tokens(3, 10, 100, 0) == [0, 1, 2, 3] and S.seen_tokens(1, 10, 1, 5) == [0, 1]
    assert S.seen_tokens(12, 10, 4, 0) == [9]


def test_restated_block_tables():
    table = np.full((3, 3), -1, np.int32)
    table[0, 0] = 7
    t, slots, start, total, used, failed = S.block_tables([5, 0, 3], [12, 33, 99], [1, 2, 3, 4, 5], 16, table, 60)
    assert t.tolist() == [[7, 1, -1], [2, 3, 4], [-1, -1, -1]] and failed == [2] and used == 4
    assert total.tolist() == [17, 33, 3] and start.tolist() == [0, 12, 45, 144]
    assert slots[:13].tolist() == [117, 118, 119, 120, 121, 122, 123, 124, 125, 126, 127, 16, 32]
    assert slots[44] == 64 and (slots[45:] == -1).all()


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pr = torch.zeros(2, 32, 8)
    args = [f16(2, 8, 128), u8(2, 2, 64, 48), u8(2, 2, 64, 48), f16(2, 2, 64), f16(2, 2, 64), i32(2), pr, pr]
    call = lambda *a, **k: isoq.isoq_decode_attention_window(*a, bits=3, variant=0, window=8, **k)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(*args)
    for i, bad, exc in ((1, u8(2, 2, 64, 64), ValueError), (3, f16(2, 2, 63), ValueError), (4, i32(2, 2, 64), TypeError),
                        (5, i32(3), ValueError), (5, i32(2).long(), TypeError), (0, f16(3, 8, 128), ValueError),
                        (0, f16(2, 128, 8).transpose(1, 2), ValueError), (6, pr[:1], ValueError), (6, pr.half(), TypeError)):
        a = list(args)
        a[i] = bad
        with pytest.raises(exc):
            call(*a)
    with pytest.raises(ValueError):
        isoq.isoq_build_block_tables(i32(2), i32(2), i32(4), i32(2, 4), 16)
    with pytest.raises(ValueError, match="fewer entries"):
        isoq.isoq_paged_append(f16(3, 2, 128), f16(3, 2, 128), u8(4, 2, 16, 48), u8(4, 2, 16, 48), f16(4, 2, 16),
                               f16(4, 2, 16), torch.zeros(2, dtype=torch.int64), pr, pr, 3, 0)
