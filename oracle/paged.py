"""Paged cache, one query per row: the definitions, in fp64 / whole numbers (NumPy).

Shares no code with the GPU path.  Rows are plain Python lists of tokens; pages are
looked up one at a time.
"""
from __future__ import annotations

import numpy as np


class Refused(Exception):
    """A step that does not fit: nothing changes.  `code` is the device error word."""

    def __init__(self, code):
        super().__init__(code)
        self.code = code


def page_map(kv_len, new_len, table, ring, ring_pos, page, max_tokens):
    """One step.  Returns dict(kv_len, ring_pos, slot, row, pos, cu, table, ring); raises Refused."""
    R, W = table.shape
    n = len(ring)
    taken, returned = int(ring_pos[0]), int(ring_pos[1])
    table, ring = table.copy(), ring.copy()
    pages = lambda t: -(-t // page)  # noqa: E731
    for a, b in zip(kv_len, new_len):
        if a < -1 or a > W * page or b < -1:
            raise Refused(3)
    if not 0 <= taken <= returned <= taken + n:
        raise Refused(3)
    back = sum(pages(max(a, 0)) for a, b in zip(kv_len, new_len) if b < 0)
    if back > n - (returned - taken):
        raise Refused(3)
    need = 0
    for a, b in zip(kv_len, new_len):
        a, b = max(int(a), 0), int(b)
        if a + max(b, 0) > W * page:
            raise Refused(4)
        if b >= 0:
            need += pages(a + b) - pages(a)
    if need > returned - taken or sum(max(int(b), 0) for b in new_len) > max_tokens:
        raise Refused(4)
    slot, row, pos, cu, out = [], [], [], [0], []
    for r in range(R):
        a, b = int(kv_len[r]), int(new_len[r])
        held = max(a, 0)
        if b < 0:
            for j in range(pages(held)):
                ring[returned % n] = table[r, j]
                returned += 1
            out.append(-1)
        else:
            for j in range(pages(held), pages(held + b)):
                table[r, j] = ring[taken % n]
                taken += 1
            for t in range(held, held + b):
                slot.append(int(table[r, t // page]) * page + t % page)
                row.append(r)
                pos.append(t)
            out.append(-1 if a < 0 and b == 0 else held + b)
        cu.append(len(slot))
    pad = [-1] * (max_tokens - len(slot))
    return {"kv_len": np.array(out, np.int32), "ring_pos": np.array([taken, returned], np.int64),
            "slot": np.array(slot + pad, np.int64), "row": np.array(row + pad, np.int32),
            "pos": np.array(pos + pad, np.int32), "cu": np.array(cu, np.int32), "table": table, "ring": ring}


def visible_tokens(n, sink=0, window=0):
    """Token numbers a query sees of a row of n tokens."""
    return [t for t in range(max(n, 0)) if window == 0 or t < sink or t >= n - window]


def page_means(stored, upto):
    """Mean of rows [0, upto) of one page [P, Hkv, d] -> [Hkv, d]."""
    return np.asarray(stored[:upto], np.float64).sum(0) / upto


def page_select(q, kbar, table, kv_len, page, topk, sink_pages=0, local_pages=0):
    """q [R, H, d], kbar [N, Hkv, d] fp64 -> int32 [R, Hkv, topk]."""
    R, H, _ = q.shape
    N, Hkv, _ = kbar.shape
    out = np.full((R, Hkv, topk), -1, np.int32)
    for r in range(R):
        n = -(-max(int(kv_len[r]), 0) // page)
        for g in range(Hkv):
            qs = q[r, g * (H // Hkv):(g + 1) * (H // Hkv)].sum(0)
            rank = []
            for j in range(n):
                pg = int(table[r, j])
                ok = 0 <= pg < N
                with np.errstate(invalid="ignore", over="ignore"):
                    v = float(np.dot(qs, kbar[pg, g])) if ok else -np.inf
                forced = j < sink_pages or j >= n - local_pages
                # forced first, then valid scores, NaN and bad pages last; ties to the lower page
                rank.append((0 if forced else 2 if (not ok or np.isnan(v)) else 1,
                             0.0 if forced or not ok or np.isnan(v) else -v, j))
            kept = sorted(j for _, _, j in sorted(rank)[:topk])
            out[r, g, :len(kept)] = kept
    return out


def page_attn(q, k, v, table, kv_len, scale, sink=0, window=0, sel=None):
    """q [R, H, d]; k, v [N, P, Hkv, d] (fp64, scales applied) -> (o, lse, terms).

    Rows of length -1 give NaN (no value).  terms [R, H, 3]: the largest |scale * q.k| sum of
    magnitudes, the largest |v| and the number of visible tokens, for error bounds.
    """
    R, H, d = q.shape
    N, P, Hkv, _ = k.shape
    o = np.full((R, H, d), np.nan)
    lse = np.full((R, H), np.nan)
    terms = np.zeros((R, H, 3))
    for r in range(R):
        n = int(kv_len[r])
        if n < 0:
            continue
        for g in range(Hkv):
            toks = visible_tokens(n, sink, window)
            if sel is not None:
                pages = [int(j) for j in sel[r, g] if j >= 0]
                toks = [t for j in pages for t in range(j * P, min(n, (j + 1) * P))]
            at = [(int(table[r, t // P]), t % P) for t in toks]
            at = [(a, b) for a, b in at if 0 <= a < N]
            kk = np.array([k[a, b, g] for a, b in at]).reshape(len(at), d)
            vv = np.array([v[a, b, g] for a, b in at]).reshape(len(at), d)
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                if not at:
                    o[r, h], lse[r, h] = 0.0, -np.inf
                    continue
                s = scale * (kk @ q[r, h])
                m = s.max()
                p = np.exp(s - m)
                o[r, h] = p @ vv / p.sum()
                lse[r, h] = m + np.log(p.sum())
                terms[r, h] = [scale * (np.abs(kk) @ np.abs(q[r, h])).max(), np.abs(vv).max(), len(at)]
    return o, lse, terms
