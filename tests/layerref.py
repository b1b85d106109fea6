"""Plain references of the page plan, the norm and rotation and the shared-prefix attention for the tests (test
infrastructure; shares no code with the library)."""
import math

import torch

import pagedref

NO_PAGE, BAD_PAGE, OVERFLOW = 256, 64, 8


def plan(table, page, n_pages, lens, m, held, stack, n_free, n_rows, packed, n_new=None, trim=False):
    """Lists in, a dict of lists out: one request after the other, the free pages a Python list."""
    B, cap = len(lens), len(table[0]) * page
    count = [m if n_new is None else max(0, min(m, n_new[r])) for r in range(B)]
    table, stack, status = [list(t) for t in table], list(stack), [0] * B
    at = 0
    for r in range(B):
        if lens[r] < 0 or lens[r] + count[r] > cap:
            status[r] = OVERFLOW
        elif held[r] < 0 or held[r] > len(table[0]) or held[r] * page < lens[r]:
            status[r] = BAD_PAGE
        else:
            at += count[r]
            if packed and count[r] and at > n_rows:
                status[r] = OVERFLOW
    need = [held[r] if status[r] else -(-(lens[r] + count[r]) // page) for r in range(B)]
    if not trim:
        need = [max(need[r], held[r]) for r in range(B)]
    free = stack[:n_free]
    for r in range(B):
        free += table[r][need[r]:held[r]]
    dry = False
    for r in range(B):
        if need[r] <= held[r]:
            continue
        if dry or need[r] - held[r] > len(free):
            dry, status[r], need[r] = True, NO_PAGE, held[r]
            continue
        for i in range(held[r], need[r]):
            table[r][i] = free.pop()
    if len(free) > n_free:
        stack[n_free:len(free)] = free[n_free:]
    slots, pos, start = [], [], [0]
    for r in range(B):
        c = 0 if status[r] else count[r]
        js = list(range(lens[r], lens[r] + c))
        slots += [table[r][j // page] * page + j % page for j in js]
        pos += js
        start.append(start[-1] + c)
        if not packed:
            slots += [-1] * (m - c)
            pos += [-1] * (m - c)
    slots += [-1] * (n_rows - len(slots))
    pos += [-1] * (n_rows - len(pos))
    return dict(table=table, held=need, stack=stack, n_free=len(free), slots=slots, pos=pos, start=start,
                lens=[lens[r] + start[r + 1] - start[r] for r in range(B)], status=status)


def norm_rope(x, weight, eps, pos, inv_freq, rot, interleaved, factor):
    """float64 (y, sum of the sizes of each element's two terms) of [T, H, D]."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * weight.double()
    out, size = y.clone(), y.abs()
    if rot:
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = pos.double()[:, None, None] * inv_freq
        c, s = factor * torch.cos(t), factor * torch.sin(t)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = abs(factor) * (y[..., a].abs() + y[..., b].abs())
    return out, size


def check_norm_rope(got, ref, size):
    """Half a step of the output's type, and what 32 bits add: the angle, held to 2^-24 of half a turn, is off by at most
    pi 2^-24, sine and cosine by 2 units of 2^-24 more; their products with factor and weight, the element, the sum and
    the norm's factor each round once (5 units); the factor itself is off by half of what a sum of 128 squares in 12
    steps is (6 units) and 2 of the root's.  19 units of 2^-24 of the terms' sizes, taken as 2^-19."""
    step, tiny = torch.finfo(got.dtype).eps / 2, torch.finfo(got.dtype).smallest_normal
    tol = step * (ref.abs() + 2.0 ** -19 * size) + 2.0 ** -19 * size + tiny * torch.finfo(got.dtype).eps
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def joined(k_pool, v_pool, table, lens, prefix_table, prefix_len, start):
    """Each request's prefix and own slots one after the other, in pools of one page a request: (k, v, table, lens)."""
    B = len(lens)
    group = [-1] * B
    for g in reversed(range(len(prefix_len))):
        if 0 <= start[g] <= start[g + 1] <= B:
            for r in range(start[g], start[g + 1]):
                group[r] = g
    most = max([1] + [lens[r] + (prefix_len[group[r]] if group[r] >= 0 else 0) for r in range(B)])
    k = torch.zeros(B, most, *k_pool.shape[2:], dtype=k_pool.dtype, device=k_pool.device)
    v, total = torch.zeros_like(k), []
    for r in range(B):
        at = 0
        parts = [(table[r], lens[r])]
        if group[r] >= 0:
            parts.insert(0, (prefix_table[group[r]], prefix_len[group[r]]))
        for row, n in parts:
            if n:
                k[r, at:at + n], v[r, at:at + n] = pagedref.slots(k_pool, row, n), pagedref.slots(v_pool, row, n)
            at += n
        total.append(at)
    return k, v, torch.arange(B, dtype=torch.int32)[:, None], torch.tensor(total, dtype=torch.int32)


def scale_of(D):
    return 1 / math.sqrt(D)
