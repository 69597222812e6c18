"""The rotation by several position axes, step by step in numpy: binary32 products, cosine and
sine in binary64 rounded once, every later product and sum rounded to binary32, one rounding to
bf16.  And a serving step's page tables in Python integers."""
from __future__ import annotations

import numpy as np


def axis_frequencies(theta, sections, interleaved=False, own=False, scale=1.0):
    """(w_j in binary32, axis of frequency j)."""
    half = sum(sections)
    if interleaved:
        left, axis = list(sections), []
        while len(axis) < half:
            for a in range(len(sections)):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    axis = np.array(axis)
    part = np.zeros(half)
    for j in range(half):
        part[j] = (axis[:j] == axis[j]).sum() / sections[axis[j]] if own else 2.0 * j / (2.0 * half)
    return (np.power(float(theta), -part) / scale).astype(np.float32), axis


def round_bf16(x):
    """binary32 values to bf16 bits, to nearest even."""
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rotate(bits, pos, theta, sections, interleaved=False, own=False, scale=1.0, bwd=False):
    """bits: bf16 bits [T, H, d]; pos: [axes, T].  Rows with a position outside [0, 2^24) stay."""
    w, axis = axis_frequencies(theta, sections, interleaved, own, scale)
    ok = ((pos >= 0) & (pos < 1 << 24)).all(axis=0)
    phi = np.where(ok, pos, 0)[axis].T.astype(np.float32) * w[None, :]
    c, s = (f(phi.astype(np.float64)).astype(np.float32)[:, None, :] for f in (np.cos, np.sin))
    s = -s if bwd else s
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    half = x.shape[2] // 2
    a, b = x[..., :half], x[..., half:]
    y = np.concatenate([a * c - b * s, b * c + a * s], axis=2)
    return np.where(ok[:, None, None], round_bf16(y), bits)


NO_PAGES, TABLE_FULL, STACK_FULL, TOKENS_PAST_END, NEGATIVE = 1, 2, 4, 8, 16


def step(free, count, table, past, new, page, max_tokens, finished=None):
    """One serving step, sequence by sequence; a dict of what it leaves behind."""
    free, table = list(free), [list(r) for r in table]
    width, status, kv, cu, slots = (len(table[0]) if table else 0), 0, [], [0], []
    past, new = list(past), list(new)
    for i in range(len(past)):
        if past[i] < 0 or new[i] < 0:
            status |= NEGATIVE
        past[i], new[i] = max(past[i], 0), max(new[i], 0)
        if finished is not None and finished[i]:
            for x in table[i][:min(-(-past[i] // page), width)]:
                if x >= 0:
                    if count < len(free):
                        free[count] = x
                        count += 1
                    else:
                        status |= STACK_FULL
            past[i] = 0
    for i, (p, n) in enumerate(zip(past, new)):
        kv.append(p + n)
        if p + n > width * page:
            status |= TABLE_FULL
        for j in range(min(-(-p // page), width), min(-(-(p + n) // page), width)):
            if count > 0:
                count -= 1
                table[i][j] = free[count]
            else:
                table[i][j] = -1
                status |= NO_PAGES
        for q in range(p, p + n):
            at = table[i][q // page] if q // page < width else -1
            slots.append(at * page + q % page if at >= 0 else -1)
        cu.append(cu[-1] + n)
    if max_tokens and cu[-1] > max_tokens:               # (without slots there is no end to pass)
        status |= TOKENS_PAST_END
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return dict(free=free, count=count, table=table, cu=cu, kv=kv, slots=slots, status=status)
