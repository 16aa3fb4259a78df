"""Oracle of the step plan and the 8-bit key / value cache (test infrastructure only).

Plain numpy: whole numbers for the plan; the insert with its rounding decisions in
fp32, as the definition states them; the attention in fp64 over the decoded cache.
Shares no code with the library.
"""

from __future__ import annotations

import numpy as np

from .csa_oracle import e4m3_decode, e4m3_encode

MIN_SCALE = np.float32(2.0 ** -100)


def step_plan(cached, n_new, free_blocks, table, P: int, n_rows: int):
    """(table, row_start, seq_id, pos, slot, used) for lengths that fit everywhere."""
    table = np.array(table, dtype=np.int64)
    row_start, seq, pos, slot, used = [0], [], [], [], 0
    for b, (c, n) in enumerate(zip(cached, n_new)):
        held, need = -(-c // P), -(-(c + n) // P)
        table[b, held:need] = free_blocks[used:used + need - held]
        table[b, need:] = -1
        used += need - held
        for p in range(c, c + n):
            seq.append(b)
            pos.append(p)
            slot.append(table[b, p // P] * P + p % P)
        row_start.append(row_start[-1] + n)
    pad = [-1] * (n_rows - len(seq))
    return table, np.array(row_start), np.array(seq + pad), np.array(pos + pad), np.array(slot + pad), used


def store(x, row_start, cached, table, codes, scale):
    """Insert rows x [T, heads, dim] into copies of codes [blocks, heads, P, dim] (bytes) and scale
    [blocks, heads] (fp32); returns them."""
    x, codes, scale = np.asarray(x, np.float32), np.array(codes), np.array(scale, np.float32)
    P = codes.shape[2]
    for b in range(len(cached)):
        r0, r1, c = row_start[b], row_start[b + 1], cached[b]
        end = c + r1 - r0
        for j in range(c // P, -(-end // P) if r1 > r0 else 0):
            blk, p0, p1 = table[b][j], max(c, j * P), min(end, (j + 1) * P)
            old = p0 - j * P
            for h in range(codes.shape[1]):
                new = x[r0 + p0 - c:r0 + p1 - c, h]
                fin = np.isfinite(new)
                amax = np.max(np.abs(np.where(fin, new, 0)))
                was = scale[blk, h] if old else np.float32(0)
                to = max(was, np.float32(amax * np.float32(1.0 / 448.0)), MIN_SCALE)
                inv = np.float32(1) / to
                if old and to > was:
                    v = e4m3_decode(codes[blk, h, :old]).astype(np.float32) * np.float32(was * inv)
                    codes[blk, h, :old] = e4m3_encode(v)
                with np.errstate(invalid="ignore", over="ignore"):
                    y = np.where(np.isnan(new), np.float32(0), new) * inv
                codes[blk, h, old:old + p1 - p0] = e4m3_encode(np.clip(y, -448, 448))
                scale[blk, h] = to
    return codes, scale


def gather(codes, scale, table_row, n: int, head: int):
    """Decoded rows [n, dim] of one sequence and head."""
    P = codes.shape[2]
    ids = np.asarray(table_row[: -(-n // P)], np.int64)
    v = e4m3_decode(codes[ids, head]) * scale[ids, head].astype(np.float64)[:, None, None]
    return v.reshape(-1, codes.shape[3])[:n]


def sees(p, n: int, first, prefix: int, window: int):
    """[rows, n] truth values: which keys the rows at positions p see, of n tokens stored."""
    p, first, t = np.asarray(p)[:, None], np.asarray(first)[:, None], np.arange(n)[None]
    near = t <= p
    if window:
        near = near & (p - t < window)
    return (t >= first) & (near | (t < prefix))


def attend(q, k, v, p, see, scale: float, softcap: float = 0.0, slopes=None):
    """q [rows, group, dim] of one key head over k, v [n, dim]: out, lse, the weighted mean of |v| (what an
    error of the weights is measured against) and a bound of the scores' magnitude before masking."""
    q = np.asarray(q, np.float64)
    a = np.einsum("rgd,nd->rgn", q, k) * scale
    mag = np.einsum("rgd,nd->rgn", np.abs(q), np.abs(k)) * scale
    if softcap:
        a = softcap * np.tanh(a / softcap)
    if slopes is not None:
        dist = np.abs(np.asarray(p)[:, None] - np.arange(len(k))[None])
        a = a - np.asarray(slopes, np.float64)[None, :, None] * dist[:, None]
        mag = mag + np.abs(np.asarray(slopes, np.float64))[None, :, None] * dist[:, None]
    a = np.where(see[:, None], a, -np.inf)
    m = np.max(a, axis=-1, keepdims=True, initial=-np.inf)
    e = np.exp(a - np.where(np.isinf(m), 0.0, m))
    s = e.sum(-1, keepdims=True)
    w = e / np.where(s > 0, s, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(s))[..., 0]
    # errors of scores that carry no weight do not count
    mag = np.max(np.where(w > 1e-12, mag, 0.0), axis=-1, initial=0.0)
    return w @ v, lse, w @ np.abs(v), mag
