"""Cases of the operators around the paged cache's attention: the page plan (page tables and slot maps from request
lengths), the norm and rotation of queries and keys on their way into the cache, and one-token attention of a batch
whose requests share long prefixes.

Each case runs in two forms: the plain one, elementary torch operations in 32 bits (64 for angles), and (``own``) the
calls of ``draft_tree_build_gb300.bastion``.

The cache: key and value pools [pages, page, Hkv, D], a page table [B, max_pages] per request and the number of used
slots ``seq_len`` [B].  Slot s of the pools is slot s % page of page s // page.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of the serving batch: a token each, one request in 32 needs a page
        {"name": "plan_step_b64", "op": "plan", "B": 64, "page": 32, "L": 16384, "m": 1, "packed": False, "ended": 0,
         "short": False},
        # the drafted trees of 32 requests get their slots
        {"name": "plan_tree_b32_n128", "op": "plan", "B": 32, "page": 16, "L": 4096, "m": 128, "packed": False,
         "ended": 0, "short": False},
        # prompts of mixed lengths come in, packed, while other requests end and give their pages back
        {"name": "plan_prompts_b64_m8192", "op": "plan", "B": 64, "page": 16, "L": 16384, "m": 8192, "packed": True,
         "ended": 8, "short": False},
        # one token of one request, its key and value stored in their page: latency alone
        {"name": "rope_step_t1", "op": "rope", "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "rot": 128,
         "interleaved": False, "norm": True, "far": 4096, "page": 16, "layout": "slot", "store": True},
        # the drafted trees of 32 requests, rows kept for the commit: no cache
        {"name": "rope_tree_t4096", "op": "rope", "T": 4096, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "rot": 128,
         "interleaved": False, "norm": True, "far": 16384, "page": 16, "layout": "slot", "store": False},
        # a small model's odd head group, part of the head turned in pairs, far positions, no norm, half precision
        {"name": "rope_part_t5003", "op": "rope", "T": 5003, "Hq": 14, "Hkv": 2, "D": 64, "dtype": "f16", "rot": 32,
         "interleaved": True, "norm": False, "far": 1000000, "page": 8, "layout": "head", "store": True},
        # prompts on their way into the cache
        {"name": "rope_prompt_t32768", "op": "rope", "T": 32768, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "rot": 128, "interleaved": False, "norm": True, "far": 131072, "page": 64, "layout": "head", "store": True},
        # four samples of one short prompt: latency
        {"name": "prefix_b4_l300", "op": "prefix", "groups": 1, "B": 4, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 16, "layout": "slot", "P": 300, "plens": "equal", "L": 33},
        # a batch behind one long system prompt
        {"name": "prefix_b64_l16384", "op": "prefix", "groups": 1, "B": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 32, "layout": "head", "P": 16384, "plens": "equal", "L": 512},
        # eight samples for each of eight prompts of mixed lengths, an odd head group, half precision
        {"name": "prefix_g8_b61_d64_f16", "op": "prefix", "groups": 8, "B": 61, "Hq": 14, "Hkv": 2, "D": 64,
         "dtype": "f16", "page": 8, "layout": "head", "P": 8190, "plens": "mixed", "L": 257},
        # many requests over one document: more rows than one pass of the tensor cores takes
        {"name": "prefix_b256_l32768", "op": "prefix", "groups": 1, "B": 256, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 64, "layout": "slot", "P": 32768, "plens": "equal", "L": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "prefix", "prefix"])
    page, layout = rng.choice([8, 16, 32, 64, 128]), rng.choice(["slot", "head"])
    D, dtype = rng.choice([64, 128]), rng.choice(["bf16", "f16"])
    Hkv, G = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    if op == "plan":
        B, packed = _log(rng, 1, 300), rng.random() < 0.5
        m = _log(rng, 1, 64 * 8192 // B if 64 * 8192 // B < 8192 else 8192)
        return {"op": op, "B": B, "page": page, "L": m + rng.randint(0, 8192), "m": m, "packed": packed,
                "ended": rng.randint(0, B // 4), "short": rng.random() < 0.2}
    if op == "rope":
        case = {"op": op, "Hkv": Hkv, "Hq": Hkv * G, "D": D, "dtype": dtype, "page": page, "layout": layout}
        # no more elements than the largest listed case's
        T = _log(rng, 1, max(1, min(32768, 32768 * 48 * 128 // ((G + 2) * Hkv * D))))
        rot = rng.choice([D, D, D // 2, D // 4])
        return case | {"T": T, "rot": rot, "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.5,
                       "far": _log(rng, max(64, T), 1 << 20), "store": rng.random() < 0.6}
    B = _log(rng, 1, 256)
    groups = rng.choice([1, 1, min(B, 3), _log(rng, 1, B)])
    # no more work, and no more cached tokens, than half of the largest listed case's
    top = 256 * 32768 * 32 * 128 // (2 * B * Hkv * G * D)
    top = max(64, min(32768, top, 4 * 32768 * 8 // (groups * Hkv)))
    return {"op": op, "groups": groups, "B": B, "Hkv": Hkv, "Hq": Hkv * G, "D": D, "dtype": dtype, "page": page,
            "layout": layout, "P": _log(rng, 1, top), "plens": rng.choice(["equal", "mixed"]),
            "L": _log(rng, 1, max(2, min(1024, top)))}


# --------------------------------------------------------------------------- inputs

def _generator(seed, salt):
    return torch.Generator("cuda").manual_seed((int(seed) * 1000003 + salt) % (1 << 62))


def _pool(case, n_pages, g):
    """A pool [pages, page, Hkv, D]; kept head by head in memory where the layout says so."""
    p, H, D = case["page"], case["Hkv"], case["D"]
    shape = (n_pages, p, H, D) if case["layout"] == "slot" else (n_pages, H, p, D)
    x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
    return x if case["layout"] == "slot" else x.transpose(1, 2)


def _ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


def _prepare_plan(case, g):
    B, page, m = case["B"], case["page"], case["m"]
    max_pages = -(-case["L"] // page)
    rand = lambda: torch.rand(B, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    count = 1 + (rand() * m).long().clamp(max=m - 1)  # a token at least
    count[0] = m
    n = (rand() * (case["L"] - count + 1)).long().clamp(min=0)
    held = (n + page - 1) // page
    order = torch.randperm(B, generator=g, device="cuda")
    over = order[:case["ended"]]  # these ended: their pages go back
    n[over], count[over] = 0, 0
    rows = B * m if not case["packed"] else max(m, B * m * 3 // 4)  # a step's budget of tokens, as a scheduler has it
    if case["packed"]:
        count = torch.where(count.cumsum(0) <= rows, count, 0)
    held[over] = held[over].clamp(min=1)
    used = int(held.sum())
    need = int(((n + count + page - 1) // page - held).clamp(min=0).sum())
    given_back = int(held[over].sum())
    free = max(1, need // 2 - given_back) if case["short"] else need + 64
    n_pages = B * max_pages + 64
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    on = torch.arange(max_pages, device="cuda")[None] < held[:, None]
    table[on] = ids[:used]
    stack = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    stack[:free] = ids[used:used + free]
    return {"table": table, "seq_len": n.to(torch.int32), "n_new": count.to(torch.int32), "held": held.to(torch.int32),
            "stack": stack, "n_free": torch.full((1,), free, dtype=torch.int32, device="cuda"), "max_pages": max_pages,
            "rows": rows, "held_out": _ints(B), "n_free_out": _ints(1), "seq_len_out": _ints(B),
            "row_start": _ints(B + 1) if case["packed"] else None,
            "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"), "pos": _ints(rows),
            "status": _ints(B)}


def _prepare_rope(case, g):
    T, Hq, H, D, rot, dt = case["T"], case["Hq"], case["Hkv"], case["D"], case["rot"], DTYPES[case["dtype"]]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # one projection gives queries, keys and values of a token side by side
    qkv = randn(T, Hq + 2 * H, D).to(dt)
    st = {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "v": qkv[:, Hq + H:], "status": _ints(1), "eps": 1e-6}
    start = int(torch.randint(0, case["far"] - T + 1, (1,), generator=g, device="cuda"))
    st["pos"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
    # a long context's frequencies: a base of a million, the angles' size kept by a factor near one
    st["inv_freq"] = 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    st["factor"] = 1.0 if case["norm"] else 1.1386
    st["q_weight"] = (1 + 0.2 * randn(D)).to(dt) if case["norm"] else None
    st["k_weight"] = (1 + 0.2 * randn(D)).to(dt) if case["norm"] else None
    st["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    if case["store"]:
        n_pages = -(-T // case["page"]) + 3
        st["k_pool"], st["v_pool"] = _pool(case, n_pages, g), _pool(case, n_pages, g)
        page = torch.randperm(n_pages, generator=g, device="cuda")
        i = torch.arange(T, device="cuda")
        st["slots"] = page[i // case["page"]] * case["page"] + i % case["page"]
    else:
        st["k_out"] = torch.zeros(T, H, D, dtype=dt, device="cuda")
    return st


def _prepare_prefix(case, g):
    B, H, D, page, groups = case["B"], case["Hkv"], case["D"], case["page"], case["groups"]
    own_pages, pre_pages = -(-case["L"] // page), -(-case["P"] // page)
    n_pages = B * own_pages + groups * pre_pages
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    u = torch.rand(B, generator=g, device="cuda", dtype=torch.float64)
    lens = (u * (case["L"] + 1)).floor().clamp(max=case["L"])
    lens[0] = case["L"]
    plens = torch.full((groups,), case["P"], dtype=torch.float64, device="cuda")
    if case["plens"] == "mixed":
        v = torch.rand(groups, generator=g, device="cuda", dtype=torch.float64)
        plens = torch.where(torch.arange(groups, device="cuda") > 0, (plens * (0.125 + 0.875 * v)).floor().clamp(min=1),
                            plens)
    start = (torch.arange(groups + 1, device="cuda") * B) // groups
    q = (2 * torch.randn(B, case["Hq"], D, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    return {"table": ids[:B * own_pages].view(B, own_pages).contiguous(),
            "prefix_table": ids[B * own_pages:].view(groups, pre_pages).contiguous(),
            "seq_len": lens.to(torch.int32), "prefix_len": plens.to(torch.int32), "group_start": start.to(torch.int32),
            "k": _pool(case, n_pages, g), "v": _pool(case, n_pages, g), "scale": 1 / math.sqrt(D), "status": _ints(B),
            # queries of spread 2: scores of spread 2, a few tokens in a hundred carry the weight
            "q": q, "out": torch.zeros_like(q), "lse": torch.zeros(B, case["Hq"], device="cuda")}


def prepare(case, seed):
    make = {"plan": _prepare_plan, "rope": _prepare_rope, "prefix": _prepare_prefix}[case["op"]]
    return {"case": case, **make(case, _generator(seed, 11))}


# --------------------------------------------------------------------------- plain forms

def _plain_plan(st):
    case = st["case"]
    B, page, m, cap = case["B"], case["page"], case["m"], st["max_pages"] * case["page"]
    table, held, n = st["table"], st["held"].long(), st["seq_len"].long()
    count = st["n_new"].long().clamp(0, m)
    need = (n + count + page - 1) // page
    ok = n + count <= cap
    if case["packed"]:  # first come, first served
        ok &= (count == 0) | (torch.where(ok, count, 0).cumsum(0) <= st["rows"])
    back = torch.where(ok, (held - need).clamp(min=0), 0)
    more = torch.where(ok, (need - held).clamp(min=0), 0)
    n_free, n_back = int(st["n_free"]), int(back.sum())
    ok &= (more == 0) | (more.cumsum(0) <= n_free + n_back)
    more = torch.where(ok, more, 0)
    n_more = int(more.sum())
    i = torch.arange(st["max_pages"], device="cuda")[None]
    given = table[(i >= need[:, None]) & (i < held[:, None]) & (back > 0)[:, None]]
    stack = torch.cat([st["stack"][:n_free], given])
    table[(i >= held[:, None]) & (i < need[:, None]) & (more > 0)[:, None]] = stack[len(stack) - n_more:].flip(0)
    left = n_free + n_back - n_more
    if left > n_free:
        st["stack"][n_free:left] = given[:left - n_free]
    count = torch.where(ok, count, 0)
    start = torch.cat([count.new_zeros(1), count.cumsum(0)])
    if case["packed"]:
        x = torch.arange(st["rows"], device="cuda")
        r = (torch.searchsorted(start, x, right=True) - 1).clamp(max=B - 1)
        j, on = n[r] + x - start[r], x < start[-1]
    else:
        r = torch.arange(B, device="cuda")[:, None].expand(B, m).reshape(-1)
        x = torch.arange(m, device="cuda")[None].expand(B, m).reshape(-1)
        j, on = n[r] + x, x < count[r]
    at = table[r, (j // page).clamp(max=st["max_pages"] - 1)].long() * page + j % page
    got = {"slots": torch.where(on, at, -1), "pos": torch.where(on, j, -1).to(torch.int32), "table": table,
           "held": torch.where(ok, need, held).to(torch.int32), "stack": st["stack"],
           "n_free": torch.full_like(st["n_free"], left), "seq_len": (n + count).to(torch.int32)}
    return {**got, "row_start": start.to(torch.int32)} if case["packed"] else got


def _turn(x, cos, sin, rot, interleaved):
    """The first rot elements of x [T, H, D] turned by the angles [T, rot / 2], in pairs (2i, 2i + 1) or
    (i, i + rot / 2)."""
    y, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    angle = st["pos"].double()[:, None] * st["inv_freq"]
    cos, sin = (torch.cos(angle) * st["factor"]).float(), (torch.sin(angle) * st["factor"]).float()

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        return _turn(x, cos, sin, case["rot"], case["interleaved"]).to(dt)

    q, k = one(st["q"], st["q_weight"]), one(st["k"], st["k_weight"])
    if not case["store"]:
        return {"q": q, "k": k}
    at, slot = st["slots"] // case["page"], st["slots"] % case["page"]
    st["k_pool"][at, slot], st["v_pool"][at, slot] = k, st["v"]
    return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _part(q, k, v, live, scale):
    """Softmax parts in 32 bits: q [N, H, R, D], k and v [N, S, H, D], live [N, S]."""
    s = torch.matmul(q, k.permute(0, 2, 3, 1).float()) * scale
    s = torch.where(live[:, None, None], s, -math.inf)
    top = s.amax(-1).clamp(min=-3e38)
    p = torch.exp(s - top[..., None])
    v = torch.where(live[:, None, :, None], v.permute(0, 2, 1, 3).float(), 0.0)
    return top, p.sum(-1), torch.matmul(p, v)


def _plain_prefix(st):
    case = st["case"]
    B, H, D, G = case["B"], case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    start = st["group_start"].long()
    groups, widest = case["groups"], -(-B // case["groups"])
    member = start[:-1, None] + torch.arange(widest, device="cuda")  # [groups, widest] requests
    on = member < start[1:, None]
    member = member.clamp(max=B - 1)
    q = st["q"].float().view(B, H, G, D)
    k = st["k"][st["prefix_table"].long()].flatten(1, 2)
    v = st["v"][st["prefix_table"].long()].flatten(1, 2)
    live = torch.arange(k.shape[1], device="cuda")[None] < st["prefix_len"][:, None]
    rows = q[member].permute(0, 2, 1, 3, 4).reshape(groups, H, widest * G, D)
    top, total, o = _part(rows, k, v, live, st["scale"])
    # back to [B, H, G]
    back = lambda x: x.view(groups, H, widest, G, -1).permute(0, 2, 1, 3, 4)[on]  # noqa: E731
    top, total, o = back(top).squeeze(-1), back(total).squeeze(-1), back(o)
    k, v = st["k"][st["table"].long()].flatten(1, 2), st["v"][st["table"].long()].flatten(1, 2)
    live = torch.arange(k.shape[1], device="cuda")[None] < st["seq_len"][:, None]
    top2, total2, o2 = _part(q, k, v, live, st["scale"])
    most = torch.maximum(top, top2)
    a, b = torch.exp(top - most) * (total > 0), torch.exp(top2 - most) * (st["seq_len"] > 0)[:, None, None]
    total = a * total + b * total2
    out = (a[..., None] * o + b[..., None] * o2) / total[..., None]
    return {"out": out.view(B, H * G, D).to(st["q"].dtype), "lse": (most + torch.log(total)).view(B, H * G)}


# --------------------------------------------------------------------------- the framework's calls

def _own_plan(st):
    from draft_tree_build_gb300 import bastion
    case = st["case"]
    if "ws" not in st:
        st["ws"] = bastion.workspace(bastion.bastion_paged_plan_workspace_bytes(case["B"]), "cuda")
    bastion.bastion_paged_plan(st["table"], case["page"], st["seq_len"], case["m"], st["held"], st["held_out"],
                               st["stack"], st["n_free"], st["n_free_out"], st["slots"], st["pos"], st["ws"],
                               st["status"], n_new=st["n_new"], row_start=st["row_start"],
                               seq_len_out=st["seq_len_out"], trim=True)
    got = {"slots": st["slots"], "pos": st["pos"], "table": st["table"], "held": st["held_out"], "stack": st["stack"],
           "n_free": st["n_free_out"], "seq_len": st["seq_len_out"]}
    return {**got, "row_start": st["row_start"]} if case["packed"] else got


def _own_rope(st):
    from draft_tree_build_gb300 import bastion
    case = st["case"]
    more = dict(v=st["v"], k_pool=st["k_pool"], v_pool=st["v_pool"], slots=st["slots"]) if case["store"] else \
        dict(k_out=st["k_out"])
    bastion.bastion_qk_norm_rope(st["q"], st["k"], st["pos"], st["inv_freq"], st["q_out"], st["status"],
                                 q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
                                 interleaved=case["interleaved"], factor=st["factor"], **more)
    if not case["store"]:
        return {"q": st["q_out"], "k": st["k_out"]}
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _own_prefix(st):
    from draft_tree_build_gb300 import bastion
    case = st["case"]
    if "ws" not in st:
        st["ws"] = bastion.workspace(bastion.bastion_paged_prefix_attention_workspace_bytes(
            case["B"], case["Hq"], case["Hkv"], case["D"], case["groups"]), "cuda")
    bastion.bastion_paged_prefix_attention(st["q"], st["k"], st["v"], st["table"], st["seq_len"], st["prefix_table"],
                                           st["prefix_len"], st["group_start"], st["scale"], st["out"], st["ws"],
                                           st["status"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "rope": _own_rope, "prefix": _own_prefix}[op](state)
    return {"plan": _plain_plan, "rope": _plain_rope, "prefix": _plain_prefix}[op](state)


# --------------------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "plan":
        B, page, m = case["B"], case["page"], case["m"]
        tokens = (B - case["ended"]) * (m + 1) / 2
        rows = B * m if not case["packed"] else max(m, B * m * 3 // 4)
        # lengths, counts and held pages both ways; 12 bytes for every row; the new rows' table entries, of which the
        # new pages come from the free list
        return {"bytes": 24.0 * B + 12 * rows + 4 * max(B, tokens / page) + 4 * tokens / page, "flops": 0}
    D, Hq, H, es = case["D"], case["Hq"], case["Hkv"], 2
    if op == "rope":
        heads = Hq + (2 if case["store"] else 1) * H
        per = 2.0 * heads * D * es + 4 + (8 if case["store"] else 0)
        flops = (Hq + H) * ((4.0 * D if case["norm"] else 0) + 3 * case["rot"])
        return {"bytes": case["T"] * per, "flops": case["T"] * flops}
    B, groups, P, L = case["B"], case["groups"], case["P"], case["L"]
    mean = P if case["plens"] == "equal" else (P + (groups - 1) * P * 9 / 16) / groups
    mine = (L + (B - 1) * L / 2)
    row = 2 * D * es
    moved = (groups * mean + mine) * H * row + (groups * mean + mine) / case["page"] * 4 + B * Hq * (2 * D * es + 4) + 4 * B
    return {"bytes": moved, "flops": 4.0 * Hq * D * (B * mean + mine)}


def _exact_plan(case, st):
    """One request after the other, with a Python list for the free pages."""
    B, page, m = case["B"], case["page"], case["m"]
    if B * m > 600_000:
        return None
    n, new, held = st["seq_len"].tolist(), st["n_new"].tolist(), st["held"].tolist()
    table, stack, free = st["table"].tolist(), st["stack"].tolist(), int(st["n_free"])
    new = [max(0, min(m, x)) for x in new]
    ok, at = [], 0
    for r in range(B):
        fits = n[r] + new[r] <= st["max_pages"] * page
        at += new[r] if fits and case["packed"] else 0
        ok.append(fits and (new[r] == 0 or at <= st["rows"]))
    need = [-(-(n[r] + new[r]) // page) for r in range(B)]
    top = stack[:free]
    for r in range(B):  # pages come back first
        if ok[r]:
            top += table[r][need[r]:held[r]]
    dry = False
    for r in range(B):
        k = need[r] - held[r]
        if not ok[r] or k <= 0:
            continue
        dry = dry or k > len(top)
        if dry:
            ok[r] = False
            continue
        for i in range(held[r], need[r]):
            table[r][i] = top.pop()
    if len(top) > free:
        stack[free:len(top)] = top[free:]
    slots, pos, start = [], [], [0]
    for r in range(B):
        k = new[r] if ok[r] else 0
        js = range(n[r], n[r] + k)
        pad = [-1] * (0 if case["packed"] else m - k)
        slots += [table[r][j // page] * page + j % page for j in js] + pad
        pos += list(js) + pad
        start.append(start[-1] + k)
    pad = [-1] * (st["rows"] - len(slots))
    ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    got = {"slots": torch.tensor(slots + pad, dtype=torch.int64), "pos": ints(pos + pad), "table": ints(table),
           "held": ints([need[r] if ok[r] else held[r] for r in range(B)]), "stack": ints(stack),
           "n_free": ints([len(top)]), "seq_len": ints([n[r] + start[r + 1] - start[r] for r in range(B)])}
    return {**got, "row_start": ints(start)} if case["packed"] else got


def _exact_rope(case, st):
    rot, half = case["rot"], case["rot"] // 2
    i = torch.arange(half, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    # complex numbers: a pair times factor * exp(1j * angle)
    angle = st["pos"].double()[:, None] * st["inv_freq"]
    phase = torch.polar(torch.full_like(angle, st["factor"]), angle)[:, None]

    def one(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + st["eps"]) * w.double()
        z = torch.complex(y[..., lo], y[..., hi]) * phase
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    q, k = one(st["q"].clone(), st["q_weight"]), one(st["k"].clone(), st["k_weight"])
    if not case["store"]:
        return {"q": q, "k": k}
    page = case["page"]
    kp, vp = st["k_pool"].double(), st["v_pool"].double()
    kp[st["slots"] // page, st["slots"] % page] = k
    vp[st["slots"] // page, st["slots"] % page] = st["v"].double()
    return {"q": q, "k_pool": kp, "v_pool": vp}


def _exact_prefix(case, st):
    B, H, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    G = case["Hq"] // H
    lens, plens, start = st["seq_len"].tolist(), st["prefix_len"].tolist(), st["group_start"].tolist()
    q = st["q"].double().view(B, H, G, D)
    out = torch.zeros(B, H, G, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, G, dtype=torch.float64, device="cuda")

    def cached(table, n):
        ids = table[:-(-n // page)].long()
        return st["k"][ids].flatten(0, 1)[:n].double(), st["v"][ids].flatten(0, 1)[:n].double()

    for x in range(case["groups"]):
        kp, vp = cached(st["prefix_table"][x], plens[x])
        for r in range(start[x], start[x + 1]):
            k, v = cached(st["table"][r], lens[r])
            k, v = torch.cat([kp, k]), torch.cat([vp, v])
            s = torch.einsum("hgd,lhd->hgl", q[r], k) * st["scale"]
            lse[r] = torch.logsumexp(s, -1)
            out[r] = torch.einsum("hgl,lhd->hgd", torch.exp(s - lse[r][..., None]), v)
    return {"out": out.view(B, H * G, D), "lse": lse.view(B, H * G)}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    return {"plan": _exact_plan, "rope": _exact_rope, "prefix": _exact_prefix}[case["op"]](case, prepare(case, seed))
