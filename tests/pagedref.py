"""Plain references of the paged cache's operators for the tests: float64
attention over gathered slots, append and eviction by loops (test
infrastructure; shares no code with the library)."""
import math

import torch


def make_pool(n_pages, page, Hkv, D, dtype, layout, gen, device):
    """[n_pages, page, Hkv, D] normal values; layout "head" keeps each head's slots together in memory."""
    shape = (n_pages, page, Hkv, D) if layout == "slot" else (n_pages, Hkv, page, D)
    x = torch.randn(shape, generator=gen, dtype=torch.float32).to(dtype).to(device)
    return x if layout == "slot" else x.transpose(1, 2)


def slots(pool, table_row, n):
    """The first n slots of a request: [n, Hkv, D]."""
    page = pool.shape[1]
    ids = table_row[: (n + page - 1) // page].long().to(pool.device)
    return pool[ids].flatten(0, 1)[:n]


def attention(q, k_pool, v_pool, table, lens, scale):
    """float64 (out, lse, weights per KV head and slot, error scale of out, error of the scores).

    The error of a score: products of 16-bit values are exact in 32 bits and their sum over D <= 128 terms is
    taken in 32 bits, every partial sum at most sum |q_i k_i|; with at most 2 D roundings of 2^-24 each (or of
    2^-23 where the adder truncates) it is off by at most 2^-16 sum |q_i k_i|, and the base change and the
    subtraction of the maximum add 2^-22 of the largest score."""
    B, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    cap = table.shape[1] * k_pool.shape[1]
    q64 = q.double().view(B, Hkv, G, D)
    out = torch.zeros(B, Hkv, G, D, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    lse = torch.full((B, Hkv, G), -math.inf, dtype=torch.float64, device=q.device)
    ds = torch.zeros_like(lse)
    w_all = torch.zeros(B, Hkv, cap, dtype=torch.float64, device=q.device)
    for r in range(B):
        n = int(lens[r])
        if n == 0:
            continue
        k, v = slots(k_pool, table[r], n).double(), slots(v_pool, table[r], n).double()
        s = torch.einsum("hgd,lhd->hgl", q64[r], k) * scale
        lse[r] = torch.logsumexp(s, -1)
        w = torch.exp(s - lse[r][..., None])
        out[r] = torch.einsum("hgl,lhd->hgd", w, v)
        size[r] = torch.einsum("hgl,lhd->hgd", w, v.abs())
        # scores that carry no weight (below 2^-40 of the largest) carry no error either
        mag = torch.einsum("hgd,lhd->hgl", q64[r].abs(), k.abs()) * scale
        mag = torch.where(w > 2.0 ** -40 * w.amax(-1, keepdim=True), mag, 0.0)
        ds[r] = mag.amax(-1) * 2.0 ** -16 + s.abs().amax(-1) * 2.0 ** -22
        w_all[r, :, :n] = w.sum(1)
    return out.view(B, Hq, D), lse.view(B, Hq), w_all, size.view(B, Hq, D), ds.view(B, Hq)


def check_attention(got_out, got_lse, q, k_pool, v_pool, table, lens, scale, acc=None, acc_out=None, fill=None):
    """out: half a step of its type, and the weights' error (2 ds from numerator and denominator, 2^-16 from
    weights held as two 16-bit terms, 2^-14 from sums of at most 2^17 terms in 32 bits, which in a tree of
    tiles are far fewer) times sum w |v|.  lse, acc likewise."""
    out, lse, w, size, ds = attention(q, k_pool, v_pool, table, lens, scale)
    step = torch.finfo(got_out.dtype).eps / 2
    tiny = torch.finfo(got_out.dtype).smallest_normal
    tol = step * out.abs() * (1 + 2.0 ** -8) + size * (2 * ds[..., None] + 2.0 ** -14) + tiny
    err = (got_out.double() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if got_lse is not None:
        empty = torch.isneginf(lse)
        assert torch.equal(torch.isneginf(got_lse), empty)
        tol = ds + 2.0 ** -20 * (1 + lse.abs())
        err = torch.where(empty, 0.0, (got_lse.double() - lse).abs())
        assert bool((err <= torch.where(empty, 1.0, tol)).all()), float((err / tol).max())
    if acc is not None:
        B, Hkv, cap = acc.shape
        live = torch.arange(cap, device=acc.device)[None, None] < lens.to(acc.device).view(B, 1, 1)
        ref = acc.double() + w
        G = q.shape[1] // Hkv
        tol = w * (2 * ds.view(B, Hkv, G).amax(-1)[..., None] + 2.0 ** -16) + 2.0 ** -23 * ref.abs() + 1e-30
        err = (acc_out.double() - ref).abs()
        assert bool((err <= tol)[live.expand_as(err)].all()), float((err / tol)[live.expand_as(err)].max())
        assert bool((acc_out == fill)[~live.expand_as(err)].all()), "slots past the sequence were written"


def append(k_new, v_new, k_pool, v_pool, table, lens, seen, acc, pos, rows=None, n_new=None):
    """In place on CPU tensors; returns the new lengths and counts."""
    B, n_rows, page = k_new.shape[0], k_new.shape[1], k_pool.shape[1]
    cap = table.shape[1] * page
    new_len, new_seen = lens.clone(), seen.clone()
    for r in range(B):
        take = list(range(n_rows)) if rows is None else []
        if rows is not None:
            for x in rows[r].tolist():
                if x < 0:
                    break
                take.append(x)
        if n_new is not None:
            take = take[: max(0, int(n_new[r]))]
        n = int(lens[r])
        if n + len(take) > cap:
            continue
        for i, x in enumerate(take):
            p, at = int(table[r, (n + i) // page]), (n + i) % page
            k_pool[p, at], v_pool[p, at] = k_new[r, x], v_new[r, x]
            if acc is not None:
                acc[r, :, n + i] = 0.0
                pos[r, :, n + i] = int(seen[r]) + i
        new_len[r] += len(take)
        new_seen[r] += len(take)
    return new_len, new_seen


def evict(k_pool, v_pool, table, lens, seen, acc, pos, budget, sink, recent, acc_out, pos_out):
    """In place on CPU tensors (acc_out, pos_out may be acc, pos); returns the new lengths."""
    B, Hkv, _ = acc.shape
    page = k_pool.shape[1]
    a_in, p_in = acc.clone(), pos.clone()
    for r in range(B):
        n = int(lens[r])
        for h in range(Hkv):
            a, p = a_in[r, h, :n].tolist(), p_in[r, h, :n].tolist()
            safe = [x < sink or x >= int(seen[r]) - recent for x in p]
            val = [math.inf if x != x else x for x in a]
            order = sorted(range(n), key=lambda s: (not safe[s], 0.0 if safe[s] else -val[s], s))
            keep = set(order[:budget])
            src = [s for s in range(min(n, budget))]
            if n > budget:
                late = [s for s in range(budget, n) if s in keep]
                holes = [s for s in range(budget) if s not in keep]
                assert len(late) == len(holes)
                for x, y in zip(holes, late):
                    src[x] = y
                    pt, at, ps, fr = int(table[r, x // page]), x % page, int(table[r, y // page]), y % page
                    k_pool[pt, at, h], v_pool[pt, at, h] = k_pool[ps, fr, h], v_pool[ps, fr, h]
            for s in range(len(src)):
                acc_out[r, h, s], pos_out[r, h, s] = a_in[r, h, src[s]], p_in[r, h, src[s]]
    return lens.clamp(max=budget)
