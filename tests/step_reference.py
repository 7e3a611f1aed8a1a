"""Plain 64-bit implementations, from the formulas, of the operators around a
serving step: the batch's tables, the normed and turned heads, attention to an
encoder's states. They share no code with the library."""
import numpy as np
import torch

import oracle

BLOCK = 16
# Half a step of a type, relative to the value (torch.finfo(t).eps / 2), and half its smallest subnormal
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}

ERR_SEQ_LEN, ERR_BLOCK_ID, ERR_CAPACITY, ERR_POSITION = 4, 2, 64, 128


def batch(start, new, ids, tables, num_blocks, capacity):
    """(tables, slots, positions, cu, lens, error bits) of pqkv_build_batch."""
    tables = np.array(tables, np.int64)
    most = tables.shape[1]
    cu, lens, slots, positions, err, taken, full = [0], [], [], [], 0, 0, False
    for b, (s, n) in enumerate(zip([int(x) for x in start], [int(x) for x in new])):
        if s < 0 or n < 0 or s + n > BLOCK * most:
            err |= ERR_SEQ_LEN
            s = n = 0
        have, need = -(-s // BLOCK), -(-(s + n) // BLOCK)
        full = full or cu[-1] + n > capacity or taken + need - have > len(ids)
        if full:
            err |= ERR_CAPACITY
            cu.append(cu[-1])
            lens.append(0)
            continue
        for j in range(have, need):
            good = 0 <= ids[taken] < num_blocks
            tables[b, j] = ids[taken] if good else -1
            err |= 0 if good else ERR_BLOCK_ID
            taken += 1
        for p in range(s, s + n):
            id = tables[b, p // BLOCK]
            good = 0 <= id < num_blocks
            slots.append(id * BLOCK + p % BLOCK if good else -1)
            positions.append(p)
            err |= 0 if good else ERR_BLOCK_ID
        cu.append(cu[-1] + n)
        lens.append(s + n)
    rest = capacity - cu[-1]
    return tables, np.array(slots + [-1] * rest), np.array(positions + [0] * rest), np.array(cu), np.array(lens), err


def norm_rope(x, weight, eps, positions, axis_of_pair, table, interleaved):
    """(rows, magnitude) in 64 bits: x [T][H][D] normed (weight None: not) and turned (table None: not); the
    magnitude |a c| + |b s| bounds what 32-bit arithmetic rounds."""
    y = x.double().numpy().copy()
    T, H, D = y.shape
    if weight is not None:
        y = y / np.sqrt((y ** 2).sum(-1, keepdims=True) / D + eps) * weight.double().numpy()
    z, size = y.copy(), np.abs(y)
    if table is None:
        return z, size
    rot = table.shape[1]
    pos = np.asarray(positions).reshape(-1, T)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        p = pos[axis_of_pair[i] if axis_of_pair else 0]
        ok = (p >= 0) & (p < table.shape[0])
        at = np.where(ok, p, 0)
        c = table[at, i].double().numpy()[:, None]
        s = table[at, rot // 2 + i].double().numpy()[:, None]
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
        size[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    if rot:
        for p in pos:
            bad = (p < 0) | (p >= table.shape[0])
            z[bad], size[bad] = 0, 0
    return z, size


def rope_tolerance(z, size, dtype):
    """Half a step of the output, and of 32-bit arithmetic: the mean square of at most 128 values by sums of
    depth 11 (eleven roundings of 2^-24, halved by the root), the quotient's root (two steps of 2^-23), three
    products and a sum: below 16 * 2^-24 of |a c| + |b s|."""
    return HALF[dtype] * np.abs(z) + (1 + HALF[dtype]) * 2.0 ** -20 * size + TINY[dtype]


def cross(cache, q, cu, tables, lens, scale, ranges=None, max_q_len=None):
    """(out, tolerance) in 64 bits over the oracle's dequantized states. The tolerance adds up the kernel's
    roundings, with A = sum p |v| of a row and one output channel:
      output             HALF |out|
      P                  half a step of its type relative to p: f16 2^-11 A (plus, for p below 2^-14, 2^-25 |v| a
                         key, over a row sum of at least 1, and twice that where FP8's V scales differ by up
                         to 2); bf16 2^-8 A, and where a KV head has at most 16
                         query rows P_hi + P_lo, (2^-8)^2 A
      scores             fp32 sums of D exact products, D 2^-24 sum |q k| scale, and the exponent's argument and
                         2^x, 4 * 2^-24 (|score| log2 e + 8): each shifts p and the row sum, so twice
      sums over L keys   L 2^-24 A, in O and in the row sum, so twice
      FP8 V scales       the ratio to the largest, 2 * 2^-23 A"""
    T, Hq, D = q.shape
    qn = q.double().numpy()
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    H = cache.H
    f16_p = cache.dt != oracle.DT_BF16
    most = max_q_len or max(int(x) for x in np.diff(cu))
    half_p = 2.0 ** -11 if f16_p else 2.0 ** -16 if most * (Hq // H) <= 16 else 2.0 ** -8
    for b, L in enumerate(int(x) for x in lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        if rows.start == rows.stop or L <= 0 or L > BLOCK * tables.shape[1]:
            continue
        for h in range(H):
            k, v, ok = oracle.gather(cache, tables[b], L, h)
            k, v = np.where(ok[:, None], k, 0), np.where(ok[:, None], v, 0)
            for n in range(h * (Hq // H), (h + 1) * (Hq // H)):
                s = qn[rows, n] @ k.T * scale
                size = np.abs(qn[rows, n]) @ np.abs(k).T * abs(scale)
                seen = np.broadcast_to(ok, s.shape).copy()
                if ranges is not None:
                    t = np.arange(L)
                    seen &= (t >= ranges[rows, :1]) & (t < ranges[rows, 1:])
                s = np.where(seen, s, -np.inf)
                top = s.max(-1, keepdims=True)
                p = np.exp(s - np.where(np.isinf(top), 0, top))
                total = p.sum(-1, keepdims=True)
                p = p / np.where(total > 0, total, 1)
                o, mag = p @ v, p @ np.abs(v)
                shift = np.where(seen, D * 2.0 ** -24 * size + 4 * 2.0 ** -24 * (np.abs(np.where(seen, s, 0)) * 1.4427 + 8),
                                 0).max(-1, keepdims=True)
                rel = half_p + 2 * shift + 2 * L * 2.0 ** -24 + 2.0 ** -22
                out[rows, n] = o
                tol[rows, n] = HALF[q.dtype] * np.abs(o) + (1 + HALF[q.dtype]) * (
                    rel * mag + (2.0 ** -24 * np.abs(v).sum(0) if f16_p else 0)) + TINY[q.dtype]
    return out, tol
