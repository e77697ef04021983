"""Float64 restatement of the serving operators around the packed cache:
attention under a sliding window with sink tokens, attention of a batch that
shares a prefix, and the paged cache (block tables, append, attention).

Each is the decode of ``isoquant.decode_attention`` over an explicit list of
tokens; nothing here is shared with the CUDA library.
"""

from __future__ import annotations

import numpy as np

from .isoquant import decode_attention, decode_attention_reconstructed, quantize


def seen_tokens(pos: int, length: int, window: int, n_sink: int):
    """Tokens j < length that the query at position pos sees: j <= pos with
    j > pos - window or j < n_sink."""
    return [j for j in range(min(pos + 1, length)) if j > pos - window or j < n_sink]


def _attend(q, pk, pv, nk, nv, params_k, params_v, bits, variant, scale, reconstructed=False):
    """One batch row: q [Hq][d] over pk, pv [Hkv][n][...]."""
    n = pk.shape[1]
    if n == 0:
        return np.zeros(q.shape, dtype=np.float64)
    f = decode_attention_reconstructed if reconstructed else decode_attention
    return f(q[None], pk[None], pv[None], nk[None], nv[None], [n], params_k, params_v, bits, variant, scale)[0]


def window_decode(q, pk, pv, nk, nv, seq_lens, params_k, params_v, bits, variant, scale, window, n_sink,
                  reconstructed=False):
    """q [B][Hq][d] over [B][Hkv][Tmax][...]; the query of row b sits at T - 1."""
    out = []
    for b in range(q.shape[0]):
        t = min(max(int(seq_lens[b]), 0), pk.shape[2])
        j = seen_tokens(t - 1, t, window, n_sink)
        out.append(_attend(q[b], pk[b][:, j], pv[b][:, j], nk[b][:, j], nv[b][:, j], params_k, params_v, bits, variant,
                           scale, reconstructed))
    return np.stack(out)


def window_prefill(q, pk, pv, nk, nv, seq_lens, params_k, params_v, bits, variant, scale, window, n_sink, rows=None):
    """q [B][Tq][Hq][d]; rows: the query indices to compute (the others stay
    zero), all of them if None."""
    bsz, tq = q.shape[:2]
    out = np.zeros(q.shape, dtype=np.float64)
    for b in range(bsz):
        for t in range(tq) if rows is None else rows:
            p = int(seq_lens[b]) - tq + t
            j = seen_tokens(p, pk.shape[2], window, n_sink) if p >= 0 else []
            out[b, t] = _attend(q[b, t], pk[b][:, j], pv[b][:, j], nk[b][:, j], nv[b][:, j], params_k, params_v, bits,
                                variant, scale)
    return out


def prefix_decode(q, prefix, prefix_len, pk, pv, nk, nv, seq_lens, params_k, params_v, bits, variant, scale):
    """prefix: (pk, pv, nk, nv) of [Hkv][Tp][...]; rows attend to both parts."""
    n = min(max(int(prefix_len), 0), prefix[0].shape[1])
    out = []
    for b in range(q.shape[0]):
        t = min(max(int(seq_lens[b]), 0), pk.shape[2])
        both = [np.concatenate([p[:, :n], c[b][:, :t]], axis=1) for p, c in zip(prefix, (pk, pv, nk, nv))]
        out.append(_attend(q[b], *both, params_k, params_v, bits, variant, scale))
    return np.stack(out)


def paged_rows(pages, block_table_row, tokens):
    """[Hkv][n][...] of pages [n_pages][Hkv][P][...] at a row's tokens."""
    p = pages.shape[2]
    page = np.asarray(block_table_row)[[j // p for j in tokens]].astype(int) if len(tokens) else np.zeros(0, int)
    return np.stack([pages[i, :, j % p] for i, j in zip(page, tokens)], axis=1) if len(tokens) else \
        pages[:0].reshape(pages.shape[1], 0, *pages.shape[3:])


def paged_decode(q, pages, block_table, seq_lens, params_k, params_v, bits, variant, scale, max_len, window, n_sink):
    """pages: (pk, pv, nk, nv) of [n_pages][Hkv][P][...]."""
    out = []
    for b in range(q.shape[0]):
        t = min(max(int(seq_lens[b]), 0), max_len)
        j = seen_tokens(t - 1, t, window, n_sink)
        out.append(_attend(q[b], *[paged_rows(x, block_table[b], j) for x in pages], params_k, params_v, bits, variant,
                           scale))
    return np.stack(out)


def block_tables(seq_lens, new_lens, free_pages, page_tokens, block_table, n_slots, free_head=0):
    """Returns (block_table, slot_map, row_start, total_lens, pages_used, rows
    that did not fit); one row after the other."""
    p = page_tokens
    table = np.array(block_table)
    slot_map = np.full(n_slots, -1, dtype=np.int64)
    row_start, total, failed = [0], [], []
    taken = used = 0          # pages asked for so far; pages taken
    for b, (length, new) in enumerate(zip(seq_lens, new_lens)):
        length, new = max(int(length), 0), int(new)
        n = max(new, 0)
        first = row_start[-1]
        row_start.append(first + n)
        fits = new >= 0 and length + new <= min(table.shape[1] * p, 2 ** 31 - 1) and (n == 0 or first + n <= n_slots)
        have, need = -(-length // p), -(-(length + n) // p)
        take = need - have if fits else 0
        if fits and (take == 0 or free_head + taken + take <= len(free_pages)):
            table[b, have:have + take] = free_pages[free_head + taken:free_head + taken + take]
            if take:
                used = taken + take
            for i in range(n):
                t = length + i
                slot_map[first + i] = int(table[b, t // p]) * p + t % p
            total.append(length + n)
        else:
            failed.append(b)
            total.append(length)
        taken += take
    return table, slot_map, np.array([min(x, 2 ** 31 - 1) for x in row_start], np.int32), np.array(total, np.int32), used, failed


def paged_append(k_new, v_new, pages, slot_map, params_k, params_v, bits, variant):
    """New page arrays (pk, pv, nk, nv) with tokens [N][Hkv][d] at their slots."""
    pk, pv, nk, nv = [np.array(x) for x in pages]
    p = pk.shape[2]
    live = [i for i in range(k_new.shape[0]) if 0 <= slot_map[i] < pk.shape[0] * p]
    if live:
        for x, params, codes, norms in ((k_new, params_k, pk, nk), (v_new, params_v, pv, nv)):
            c, n = quantize(np.asarray(x, np.float64)[live].transpose(1, 0, 2), params, bits, variant)
            for i, token in enumerate(live):
                page, off = divmod(int(slot_map[token]), p)
                codes[page, :, off], norms[page, :, off] = c[:, i], n[:, i]
    return pk, pv, nk, nv
