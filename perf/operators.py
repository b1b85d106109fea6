"""Cases of the paged key-value cache operators: append, one-token attention
(with the accumulated attention weight of every cached token) and eviction by
that weight.

Each case runs in two forms: the plain one, elementary torch operations in 32
bits, and (``own``) the calls of ``draft_tree_build_gb300.bastion``.

The cache: key and value pools [pages, page, Hkv, D], a page table [B, max_pages]
per request, the number of used slots ``seq_len`` [B], and per request, KV head
and slot the accumulated weight ``acc`` and the token position ``pos``
[B, Hkv, max_pages * page].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one short chat turn on an idle server: latency alone
        {"name": "attend_b1_l300", "op": "attend", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 16, "layout": "slot", "L": 300, "lens": "equal", "weights": False},
        # one request over a long document: few rows, a long axis to split
        {"name": "attend_b1_l131072", "op": "attend", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 64, "layout": "slot", "L": 131072, "lens": "equal", "weights": False},
        # the tree attention workload's cache (8 requests, context 4096) read by plain decoding
        {"name": "attend_b8_l4096", "op": "attend", "B": 8, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 16, "layout": "slot", "L": 4096, "lens": "equal", "weights": False},
        # the serving step's cache: 64 requests of up to 16384 tokens, all lengths mixed
        {"name": "attend_b64_l16384_mixed", "op": "attend", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 32, "layout": "head", "L": 16384, "lens": "mixed", "weights": False},
        # a small model's odd head group, half precision, short pages, very uneven lengths, empty requests
        {"name": "attend_b33_g7_d64_f16", "op": "attend", "B": 33, "Hq": 14, "Hkv": 2, "D": 64, "dtype": "f16",
         "page": 8, "layout": "head", "L": 8190, "lens": "ragged", "weights": False},
        # a decode step of a cache that is kept within a budget: the weights are accumulated
        {"name": "attend_weights_b32_l2065", "op": "attend", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 16, "layout": "slot", "L": 2065, "lens": "equal", "weights": True},
        # the weights' bookkeeping on long prompts, before their first eviction
        {"name": "attend_weights_b8_l32768", "op": "attend", "B": 8, "Hq": 32, "Hkv": 4, "D": 128, "dtype": "bf16",
         "page": 64, "layout": "slot", "L": 32768, "lens": "mixed", "weights": True},
        # the accepted path of a verified tree enters the cache
        {"name": "append_path_b32", "op": "append", "B": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16,
         "layout": "slot", "L": 4096, "rows": 128, "m": 17, "path": True},
        # prompts of mixed lengths enter the cache
        {"name": "append_prompt_b8_m8192", "op": "append", "B": 8, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64,
         "layout": "head", "L": 8192, "rows": 8192, "m": 8192, "path": False},
        # steady decoding: a step's tokens came in, as many leave
        {"name": "evict_step_b32", "op": "evict", "B": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16,
         "layout": "slot", "L": 2065, "lens": "equal", "budget": 2048, "sink": 4, "recent": 256},
        # long prompts are cut to the budget
        {"name": "evict_prompt_b8_l32768", "op": "evict", "B": 8, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64,
         "layout": "head", "L": 32768, "lens": "mixed", "budget": 4096, "sink": 4, "recent": 512},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    case = {"op": op, "B": _log(rng, 1, 64), "Hkv": Hkv, "D": D, "dtype": rng.choice(["bf16", "f16"]),
            "page": rng.choice([8, 16, 32, 64, 128]), "layout": rng.choice(["slot", "head"])}
    # no more cached tokens than half of the largest listed case's
    top = max(64, min(131072, 64 * 16384 // (2 * case["B"]) * 8 // Hkv))
    if op == "attend":
        case |= {"Hq": Hkv * G, "L": _log(rng, 1, top), "lens": rng.choice(["equal", "mixed", "ragged"]),
                 "weights": rng.random() < 0.4}
    elif op == "append":
        path = rng.random() < 0.5
        m = rng.randint(1, 33) if path else _log(rng, 1, min(top, 32768))
        case |= {"rows": rng.randint(m, 256) if path else m, "m": m, "path": path, "L": m + rng.randint(0, 4096)}
    else:
        L = _log(rng, 16, min(top, 65536))
        budget = rng.randint(max(1, L // 16), L)
        sink = min(rng.randint(0, 8), budget)
        case |= {"L": L, "lens": rng.choice(["equal", "mixed"]), "budget": budget, "sink": sink,
                 "recent": rng.randint(0, max(0, (budget - sink) // 2))}
    return case


# --------------------------------------------------------------------------- inputs

def _generator(seed, salt):
    return torch.Generator("cuda").manual_seed((int(seed) * 1000003 + salt) % (1 << 62))


def _lengths(case, g):
    """Used slots per request: all alike, uniform over the range, or spread over its logarithm with empty ones."""
    B, L = case["B"], case["L"]
    if case.get("lens", "equal") == "equal":
        return torch.full((B,), L, dtype=torch.int32, device="cuda")
    u = torch.rand(B, generator=g, device="cuda", dtype=torch.float64)
    if case["lens"] == "mixed":
        n = (L / 8 + u * (L - L / 8)).floor().clamp(min=1)
    else:
        n = torch.exp(u * math.log(L + 1)).floor() - 1
    n[0] = L  # one request fills the range
    return n.clamp(0, L).to(torch.int32)


def _pool(case, n_pages, g):
    """A pool [pages, page, Hkv, D]; kept head by head in memory where the layout says so."""
    p, H, D = case["page"], case["Hkv"], case["D"]
    shape = (n_pages, p, H, D) if case["layout"] == "slot" else (n_pages, H, p, D)
    x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
    return x if case["layout"] == "slot" else x.transpose(1, 2)


def _table(B, max_pages, g):
    """Every request's pages, anywhere in the pool, as a serving allocator leaves them."""
    order = torch.randperm(B * max_pages, generator=g, device="cuda").to(torch.int32)
    return order.view(B, max_pages)


def prepare(case, seed):
    g = _generator(seed, 7)
    B, H, D, page, op = case["B"], case["Hkv"], case["D"], case["page"], case["op"]
    dt = DTYPES[case["dtype"]]
    max_pages = -(-case["L"] // page)
    cap = max_pages * page
    st = {"case": case, "cap": cap, "status": torch.zeros(B, dtype=torch.int32, device="cuda"),
          "table": _table(B, max_pages, g), "k": _pool(case, B * max_pages, g), "v": _pool(case, B * max_pages, g)}
    zeros = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "attend":
        st["seq_len"] = _lengths(case, g)
        st["scale"] = 1 / math.sqrt(D)
        # queries of spread 2: scores of spread 2, a few tokens in a hundred carry the weight
        st["q"] = (2 * torch.randn(B, case["Hq"], D, generator=g, device="cuda")).to(dt)
        st["out"], st["lse"] = torch.empty_like(st["q"]), zeros(B, case["Hq"])
        if case["weights"]:
            # what some ten earlier steps left
            st["acc"] = torch.rand(B, H, cap, generator=g, device="cuda") * (20 * case["Hq"] / H / case["L"])
            st["acc_out"] = zeros(B, H, cap)
    elif op == "append":
        m, n = case["m"], case["rows"]
        st["k_new"] = torch.randn(B, n, H, D, generator=g, device="cuda").to(dt)
        st["v_new"] = torch.randn(B, n, H, D, generator=g, device="cuda").to(dt)
        u = torch.rand(B, generator=g, device="cuda")
        count = 1 + (u * m).long().clamp(max=m - 1)  # at least the root, or one prompt token
        count[0] = m
        if case["path"]:  # a root path of rising node numbers, then -1
            nodes = torch.rand(B, n, generator=g, device="cuda").argsort(1)[:, :m].sort(1).values
            nodes[:, 0] = 0
            end = torch.arange(m, device="cuda")[None] >= count[:, None]
            st["rows"], st["n_new"] = nodes.masked_fill(end, -1).to(torch.int32).contiguous(), None
        else:
            st["rows"], st["n_new"] = None, count.to(torch.int32)
        room = torch.rand(B, generator=g, device="cuda") * (case["L"] - count + 1)
        st["seq_len"] = room.long().clamp(min=0).to(torch.int32)
        st["n_seen"] = st["seq_len"] + 11
        st["acc"], st["pos"] = torch.rand(B, H, cap, generator=g, device="cuda"), ints(B, H, cap)
        st["seq_len_out"], st["n_seen_out"] = ints(B), ints(B)
    else:
        st["seq_len"] = _lengths(case, g)
        # heavy-tailed weights; positions out of order, as earlier evictions leave them, the newest last
        st["acc"] = torch.randn(B, H, cap, generator=g, device="cuda").mul_(2).exp_()
        st["n_seen"] = st["seq_len"] + 1000
        R = case["recent"]
        slot = torch.arange(cap, device="cuda")
        old = torch.rand(B, H, cap, generator=g, device="cuda").argsort(-1)  # a permutation of the slots
        last = st["seq_len"].view(B, 1, 1) - R
        tail = slot >= last
        old_rank = torch.where(tail, cap, old).argsort(-1).argsort(-1)  # the old slots' positions, out of order
        new = (st["n_seen"].view(B, 1, 1) - R + (slot - last)).expand(B, H, cap)
        st["pos"] = torch.where(tail, new, old_rank).to(torch.int32)
        st["acc_out"], st["pos_out"], st["seq_len_out"] = zeros(B, H, cap), ints(B, H, cap), ints(B)
    return st


# --------------------------------------------------------------------------- plain forms

def _cached(pool, table, case):
    """The requests' slots in order: [B, cap, Hkv, D]."""
    x = pool[table.long().clamp(min=0)]
    return x.reshape(x.shape[0], -1, x.shape[3], x.shape[4])


def _plain_attend(st):
    case = st["case"]
    B, H, D = case["B"], case["Hkv"], case["D"]
    G = case["Hq"] // H
    live = torch.arange(st["cap"], device="cuda")[None] < st["seq_len"][:, None]
    k = _cached(st["k"], st["table"], case).permute(0, 2, 3, 1).float()
    s = torch.matmul(st["q"].float().view(B, H, G, D), k) * st["scale"]
    del k
    s = torch.where(live[:, None, None], s, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).view(B, H * G)
    p = p / total.clamp(min=1e-30)
    v = _cached(st["v"], st["table"], case).permute(0, 2, 1, 3).float()
    v = torch.where(live[:, None, :, None], v, 0.0)
    out = torch.matmul(p, v).view(B, H * G, D).to(st["q"].dtype)
    lse = torch.where(st["seq_len"][:, None] > 0, lse, -math.inf)
    if not case["weights"]:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "acc": torch.where(live[:, None], st["acc"] + p.sum(2), 0.0)}


def _plain_append(st):
    case = st["case"]
    m, page = case["m"], case["page"]
    i = torch.arange(m, device="cuda")[None]
    if st["rows"] is not None:
        take = st["rows"].long()
        on = (take >= 0).long().cumprod(1) > 0
    else:
        take = i.expand(case["B"], m)
        on = i < st["n_new"][:, None]
    count = on.sum(1).to(torch.int32)
    b, j = on.nonzero(as_tuple=True)
    slot = st["seq_len"].long()[b] + j
    page_id, at = st["table"].long()[b, slot // page], slot % page
    st["k"][page_id, at] = st["k_new"][b, take[b, j]]
    st["v"][page_id, at] = st["v_new"][b, take[b, j]]
    st["acc"][b, :, slot] = 0.0
    st["pos"][b, :, slot] = (st["n_seen"].long()[b] + j).to(torch.int32)[:, None]
    return {"k": st["k"], "v": st["v"], "acc": st["acc"], "pos": st["pos"],
            "seq_len": st["seq_len"] + count, "n_seen": st["n_seen"] + count}


def _plain_evict(st):
    case = st["case"]
    B, H, page, cap, budget = case["B"], case["Hkv"], case["page"], st["cap"], case["budget"]
    slot = torch.arange(cap, device="cuda")
    n, seen = st["seq_len"].view(B, 1, 1), st["n_seen"].view(B, 1, 1)
    live = slot < n
    safe = (st["pos"] < case["sink"]) | (st["pos"] >= seen - case["recent"])
    key = torch.where(live, torch.where(safe, math.inf, st["acc"]), -math.inf)
    rank = torch.argsort(key, dim=-1, descending=True, stable=True).argsort(-1)
    keep = live & (rank < budget)
    hole = (slot < budget) & live & ~keep
    late = (slot >= budget) & keep
    b, h, to = hole.nonzero(as_tuple=True)
    at = late.nonzero(as_tuple=True)[2]  # as many for each request and head, in the same order
    table = st["table"].long()
    to_page, at_page = table[b, to // page], table[b, at // page]
    st["k"][to_page, to % page, h] = st["k"][at_page, at % page, h]
    st["v"][to_page, to % page, h] = st["v"][at_page, at % page, h]
    head = live & (slot < budget)
    acc, pos = torch.where(head, st["acc"], 0.0), torch.where(head, st["pos"], 0)
    acc[b, h, to], pos[b, h, to] = st["acc"][b, h, at], st["pos"][b, h, at]
    return {"k": st["k"], "v": st["v"], "acc": acc, "pos": pos, "seq_len": st["seq_len"].clamp(max=budget)}


# --------------------------------------------------------------------------- the framework's calls

def _own_attend(st):
    from draft_tree_build_gb300 import bastion
    case = st["case"]
    if "ws" not in st:
        st["ws"] = bastion.workspace(bastion.bastion_paged_attention_workspace_bytes(
            case["B"], case["Hq"], case["Hkv"], case["D"], st["cap"], case["weights"]), "cuda")
    bastion.bastion_paged_attention(st["q"], st["k"], st["v"], st["table"], st["seq_len"], st["scale"], st["out"],
                                    st["ws"], st["status"], lse=st["lse"], acc=st.get("acc"),
                                    acc_out=st.get("acc_out"))
    got = {"out": st["out"], "lse": st["lse"]}
    return {**got, "acc": st["acc_out"]} if case["weights"] else got


def _own_append(st):
    from draft_tree_build_gb300 import bastion
    case = st["case"]
    if "ws" not in st:
        st["ws"] = bastion.workspace(bastion.bastion_paged_append_workspace_bytes(case["B"]), "cuda")
    bastion.bastion_paged_append(st["k_new"], st["v_new"], st["k"], st["v"], st["table"], st["seq_len"],
                                 st["seq_len_out"], st["ws"], st["status"], rows=st["rows"], n_new=st["n_new"],
                                 acc=st["acc"], pos=st["pos"], n_seen=st["n_seen"], n_seen_out=st["n_seen_out"])
    return {"k": st["k"], "v": st["v"], "acc": st["acc"], "pos": st["pos"], "seq_len": st["seq_len_out"],
            "n_seen": st["n_seen_out"]}


def _own_evict(st):
    from draft_tree_build_gb300 import bastion
    case = st["case"]
    if "ws" not in st:
        st["ws"] = bastion.workspace(bastion.bastion_paged_evict_workspace_bytes(
            case["B"], case["Hkv"], st["cap"]), "cuda")
    bastion.bastion_paged_evict(st["k"], st["v"], st["table"], st["seq_len"], st["n_seen"], st["acc"], st["pos"],
                                case["budget"], case["sink"], case["recent"], st["seq_len_out"], st["acc_out"],
                                st["pos_out"], st["ws"], st["status"])
    return {"k": st["k"], "v": st["v"], "acc": st["acc_out"], "pos": st["pos_out"], "seq_len": st["seq_len_out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "evict": _own_evict}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}[op](state)


# --------------------------------------------------------------------------- work and exact values

def _mean_length(case):
    """Used slots of a request, on average over the seeds; request 0 has them all."""
    B, L, lens = case["B"], case["L"], case.get("lens", "equal")
    mean = L if lens == "equal" else L * 9 / 16 if lens == "mixed" else max(0.0, L / math.log(L + 1) - 1.5)
    return (L + (B - 1) * mean) / B


def work(case):
    B, H, D, es = case["B"], case["Hkv"], case["D"], 2
    row = 2 * D * es  # a token's key and value of one head
    if case["op"] == "attend":
        tokens, Hq = B * _mean_length(case), case["Hq"]
        moved = tokens * H * row + tokens / case["page"] * 4 + B * Hq * (2 * D * es + 4) + 4 * B
        moved += tokens * H * 8 if case["weights"] else 0
        return {"bytes": moved, "flops": 4.0 * tokens * Hq * D}
    if case["op"] == "append":
        tokens = (case["m"] + (B - 1) * (case["m"] + 1) / 2)
        return {"bytes": tokens * H * (2 * row + 8) + 20 * B + (4 * B * case["m"] if case["path"] else 0), "flops": 0}
    n, budget = _mean_length(case), case["budget"]
    kept = min(n, budget)
    over = max(0.0, n - budget)
    new = min(over, case["recent"])  # the newest stay: those past the budget fill holes
    moves = new + (over - new) * max(0, kept - case["recent"] - case["sink"]) / max(1.0, n - case["recent"])
    return {"bytes": B * H * (8 * n + 8 * kept + moves * 2 * row) + 16 * B, "flops": 0}


def exact(case, seed):
    """The same outputs from the definitions, request by request, in 64 bits."""
    st = prepare(case, seed)
    B, H, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    lens, table = st["seq_len"].tolist(), st["table"].tolist()

    def places(r, slots):
        return [table[r][s // page] for s in slots], [s % page for s in slots]

    if case["op"] == "attend":
        G = case["Hq"] // H
        out = torch.zeros(B, H, G, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, G), -math.inf, dtype=torch.float64, device="cuda")
        acc = torch.zeros(B, H, st["cap"], dtype=torch.float64, device="cuda")
        q = st["q"].double().view(B, H, G, D)
        for r in range(B):
            n = lens[r]
            if n == 0:
                continue
            ids = st["table"][r, : -(-n // page)].long()
            k = st["k"][ids].flatten(0, 1)[:n].double()
            v = st["v"][ids].flatten(0, 1)[:n].double()
            s = torch.einsum("hgd,lhd->hgl", q[r], k) * st["scale"]
            lse[r] = torch.logsumexp(s, -1)
            w = torch.exp(s - lse[r][..., None])
            out[r] = torch.einsum("hgl,lhd->hgd", w, v)
            if case["weights"]:
                acc[r, :, :n] = st["acc"][r, :, :n].double() + w.sum(1)
        got = {"out": out.view(B, H * G, D), "lse": lse.view(B, H * G)}
        return {**got, "acc": acc} if case["weights"] else got
    if case["op"] == "append":
        if B * case["m"] > 20000:
            return None
        seen = st["n_seen"].tolist()
        rows = st["rows"].tolist() if st["rows"] is not None else None
        count = [case["m"]] * B if rows is not None else st["n_new"].tolist()
        for r in range(B):
            take = list(range(count[r])) if rows is None else rows[r]
            take = take[: take.index(-1)] if -1 in take else take
            count[r] = len(take)
            slots = list(range(lens[r], lens[r] + len(take)))
            pages, at = places(r, slots)
            st["k"][pages, at] = st["k_new"][r, take]
            st["v"][pages, at] = st["v_new"][r, take]
            st["acc"][r, :, slots] = 0.0
            st["pos"][r, :, slots] = torch.arange(seen[r], seen[r] + len(take), dtype=torch.int32, device="cuda")
        add = torch.tensor(count, dtype=torch.int32, device="cuda")
        return {"k": st["k"].double(), "v": st["v"].double(), "acc": st["acc"].double(), "pos": st["pos"],
                "seq_len": st["seq_len"] + add, "n_seen": st["n_seen"] + add}
    if B * H * case["L"] > 1_000_000:
        return None
    acc, pos, seen = st["acc"].double().cpu(), st["pos"].cpu(), st["n_seen"].tolist()
    new_acc, new_pos = torch.zeros_like(acc), torch.zeros_like(pos)
    for r in range(B):
        n = lens[r]
        for h in range(H):
            a, p = acc[r, h, :n].tolist(), pos[r, h, :n].tolist()
            safe = [x < case["sink"] or x >= seen[r] - case["recent"] for x in p]
            best = sorted(range(n), key=lambda s: (not safe[s], 0.0 if safe[s] else -a[s], s))
            keep = set(best[: case["budget"]])
            late = iter(s for s in range(case["budget"], n) if s in keep)
            pairs = [(s, s if s in keep else next(late)) for s in range(min(n, case["budget"]))]
            to, at = [x for x, y in pairs if x != y], [y for x, y in pairs if x != y]
            src = torch.tensor([y for _, y in pairs], dtype=torch.long)
            new_acc[r, h, : len(pairs)], new_pos[r, h, : len(pairs)] = acc[r, h, src], pos[r, h, src]
            if to:
                (tp, ta), (sp, sa) = places(r, to), places(r, at)
                st["k"][tp, ta, h], st["v"][tp, ta, h] = st["k"][sp, sa, h], st["v"][sp, sa, h]
    return {"k": st["k"].double(), "v": st["v"].double(), "acc": new_acc, "pos": new_pos,
            "seq_len": st["seq_len"].clamp(max=case["budget"])}
