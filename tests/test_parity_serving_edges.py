"""The serving operators at the edges of what their documentation allows:
streams given by argument, pages dropped behind the window, magnitudes next to
float16's limits, alignments and cluster sizes that ordinary calls do not
reach.  Tolerances as in test_parity_serving, unless a test derives its own."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import compressed_space_attention_b200 as isoq  # noqa: E402
from test_parity_serving import DEV, F16, _cache, _pages, _params, _t  # noqa: E402

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
