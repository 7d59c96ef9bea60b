"""Plain statements of the paged-cache operators for the tests: the page plan
one request and one page at a time, the 8-bit rounding in 64 bits, and the
attention of a token in 64 bits from its key list.  Host only (numpy)."""
from __future__ import annotations

import numpy as np
import torch


def plan(length, n_new, table, stack, count, page, capacity):
    """One step, request by request and token by token.  Returns a dict of the
    new state and the step's tokens; the arguments stay as they are."""
    B, M = table.shape
    length, table, stack = [int(x) for x in length], table.copy(), stack.copy()
    n_new = [int(x) for x in n_new]
    room = M * page
    sane = [0 <= L <= room for L in length]
    status = [2] * B
    stack_ok = 0 <= count <= len(stack)
    top, wanted = count, count
    for b in range(B):                      # finished requests, in order
        if n_new[b] != -1 or not sane[b] or not stack_ok:
            continue
        pages = table[b, :-(-length[b] // page)]
        wanted += len(pages)
        if wanted > len(stack) and len(pages):
            continue
        stack[top:top + len(pages)] = pages
        top += len(pages)
        status[b] = 0
    out_len = [0 if n == -1 and st == 0 else L for n, L, st in zip(n_new, length, status)]
    cu = np.concatenate([[0], np.cumsum([max(n, 0) for n in n_new])]).astype(np.int64)
    slot, pos = np.full(capacity, -1, np.int64), np.full(capacity, -1, np.int64)
    row = np.full(capacity, -1, np.int32)
    left, dry = (top if stack_ok else 0), False
    for b in range(B):                      # the others, in order
        n, L = n_new[b], length[b]
        if n < 0 or not sane[b] or L + n > room or cu[b + 1] > capacity:
            continue
        used, total = -(-L // page), -(-(L + n) // page)
        if total > used and (dry or total - used > left):
            dry, status[b] = True, 1
            continue
        for p in range(used, total):
            left -= 1
            table[b, p] = stack[left]
        status[b], out_len[b] = 0, L + n
        for x in range(n):
            t, at = int(cu[b]) + x, L + x
            pos[t], row[t] = at, b
            pg = int(table[b, at // page])
            slot[t] = pg * page + at % page if pg >= 0 else -1
    return dict(length=np.array(out_len), count=left if stack_ok else count, table=table,
                stack=stack, cu_new=cu, slot=slot, pos=pos, row=row, status=np.array(status))


# every non-negative e4m3 value, in the order of its code
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def e4m3_round(y):
    """The code value nearest to y (|y| <= 448), halves to the even code."""
    a = np.abs(y)
    hi = np.searchsorted(E4M3, a).clip(1, 126)
    lo = hi - 1
    down, up = a - E4M3[lo], E4M3[hi] - a
    pick = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.copysign(E4M3[pick], y)


def quantise(x):
    """(codes' values, scales) of rows x (float32 array [..., D]): the scale
    and the quotient in fp32 (one correctly rounded division each), the code by
    search among all 8-bit values."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        scale = np.where(np.isfinite(amax), amax / np.float32(448), np.float32(np.nan))
        scale = scale.astype(np.float32)
        y = (x / scale[..., None]).astype(np.float32)
    live = (scale > 0)[..., None]
    y = np.where(live, np.clip(y, -448, 448), 0).astype(np.float64)
    return e4m3_round(y), scale


def attend(q, keys, values, scale):
    """out [G, D], lse [G] in 64 bits of queries q [G, D] over rows keys,
    values [n, D], and the bounds that tolerances need: the largest sum of
    |q_d k_d| * scale of a score, and the largest |v|."""
    G, D = q.shape
    if len(keys) == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), 0.0, 0.0
    s = scale * (q @ keys.T)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    size = abs(scale) * (np.abs(q) @ np.abs(keys).T).max()
    return p @ values / total, (m + np.log(total))[:, 0], float(size), float(np.abs(values).max())


def tolerances(n, D, size, vmax, out_dtype):
    """Bounds on |lse| and |out| errors of n keys.
    A score is a sum of D products in 32 bits: off by at most (D + 4) 2^-23
    `size` (twice the half step 2^-24 per addition, as matrix instructions
    round by cutting).  exp and log are approximations good to 2^-21 of the
    base-2 argument's unit; sums of n positive terms run in at least 8 chains:
    (n / 8 + 64) 2^-23 relative.  A probability is then off by twice the
    score's error and the value sum by as much of vmax; weights kept as two
    16-bit parts add 2^-16.  The output is rounded once, by eps / 2."""
    score = (D + 4) * 2.0 ** -23 * size + 2.0 ** -21
    sums = (n / 8 + 64) * 2.0 ** -23
    lse = score + sums
    out = (2 * score + 2 * sums + 2.0 ** -16 * (out_dtype == torch.bfloat16)) * vmax
    return lse, out, torch.finfo(out_dtype).eps / 2
