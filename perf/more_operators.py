"""What is measured of the operators around a paged cache: the positions of a drafted tree's nodes, rotary positions
of queries and keys, prompts appended to the cache with their keys rotated, and the attention of a batch of drafted
trees whose sequences share a long prefix.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64), or with ``own`` set
through the library's entry points; ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BASE = 10000.0  # of the rotation's frequencies
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one drafted block's path behind a context: once a pass, in front of every layer
        {"name": "positions one block", "op": "positions", "B": 1, "T": 17, "ctx": 4001, "prefix": 0, "tree": "chain"},
        # a large batch of drafted trees over a prefix, unused nodes among them
        {"name": "positions many trees", "op": "positions", "B": 4096, "T": 63, "ctx": 100001, "prefix": 5000, "tree": "random"},
        # one token's heads out of the projection's row: the smallest call
        {"name": "rope one token", "op": "rope", "rows": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "layout": "half",
         "dt": "bf16", "split": True, "far": 4002, "factor": 1.0, "amplitude": 1.0},
        # a quarter of odd-sized heads, adjacent pairs, stretched and scaled for positions up to a million, fp32
        {"name": "rope partial far fp32", "op": "rope", "rows": 4003, "Hq": 20, "Hkv": 5, "D": 80, "rot": 20,
         "layout": "interleaved", "dt": "fp32", "split": False, "far": 1000000, "factor": 8.0, "amplitude": 1.2079},
        # the rows of 960 sequences' blocks of 17 positions, out of the projection's rows
        {"name": "rope many blocks", "op": "rope", "rows": 16320, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "layout": "half",
         "dt": "bf16", "split": True, "far": 32768, "factor": 1.0, "amplitude": 1.0},
        # a block's tokens behind a sequence's cache
        {"name": "append one block", "op": "append", "B": 1, "rows": 17, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "layout": "half", "dt": "bf16", "q": True, "ctx": 4001, "prefix": 0, "page": 16},
        # keys and values alone (of context that is projected for a drafter), ragged, fp32, half of each head, behind a prefix
        {"name": "append ragged fp32", "op": "append", "B": 37, "rows": 3001, "Hq": 0, "Hkv": 3, "D": 96, "rot": 48,
         "layout": "interleaved", "dt": "fp32", "q": False, "ctx": 1500, "prefix": 777, "page": 1},
        # prompts of 16 sequences at once, their queries too
        {"name": "append prompts", "op": "append", "B": 16, "rows": 65536, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "layout": "half", "dt": "bf16", "q": True, "ctx": 0, "prefix": 0, "page": 64},
        # a few answers to one prompt, one token each
        {"name": "shared few tokens", "op": "shared", "B": 4, "T": 1, "Hkv": 8, "group": 4, "D": 128, "prefix": 4001, "ctx": 77,
         "page": 16, "tree": "chain"},
        # many answers to one prompt, one token each, of lengths from 0 to 1024
        {"name": "shared many tokens", "op": "shared", "B": 256, "T": 1, "Hkv": 8, "group": 4, "D": 128, "prefix": 16384,
         "ctx": 1024, "page": 64, "tree": "chain"},
        # trees of 63 drafted nodes, some unused, over a long document
        {"name": "shared trees", "op": "shared", "B": 12, "T": 63, "Hkv": 4, "group": 6, "D": 64, "prefix": 60001, "ctx": 3000,
         "page": 256, "tree": "random"},
        # a batch of drafted blocks of 16 tokens behind the last verified one, one system prompt
        {"name": "shared blocks", "op": "shared", "B": 64, "T": 17, "Hkv": 8, "group": 4, "D": 128, "prefix": 16384, "ctx": 2048,
         "page": 64, "tree": "chain"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["positions", "rope", "rope", "append", "append", "shared", "shared", "shared"])
    tree = rng.choice(["chain", "random"])
    if op == "positions":
        return {"op": op, "B": _log(rng, 1, 4096), "T": rng.randint(1, 64), "ctx": _log(rng, 1000, 1000000),
                "prefix": rng.choice([0, _log(rng, 1, 100000)]), "tree": tree}
    if op == "shared":
        D, T, Hkv, group = rng.choice([64, 128]), _log(rng, 1, 64), rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8])
        prefix, ctx = _log(rng, 1, 65536), rng.choice([0, _log(rng, 1, 2000)])
        most = 0.9 * 64 * 17 * 32 * 128 * 16384 / (T * Hkv * group * D * (prefix + ctx))
        B = _log(rng, 1, max(1, min(256, int(most))))
        return {"op": op, "B": B, "T": T, "Hkv": Hkv, "group": group, "D": D, "prefix": prefix, "ctx": ctx,
                "page": rng.choice([1, 16, 32, 64, 256]), "tree": tree}
    D = rng.choice([64, 80, 96, 128, 256])
    case = {"op": op, "rows": _log(rng, 1, 8192), "Hq": rng.randint(1, 32), "Hkv": rng.randint(1, 8), "D": D,
            "rot": rng.choice([D, D, D // 2, D // 4]), "layout": rng.choice(["half", "half", "interleaved"]),
            "dt": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "rope":
        return case | {"split": rng.random() < 0.6, "far": _log(rng, 100, 1000000), "factor": rng.choice([1.0, 4.0]),
                       "amplitude": rng.choice([1.0, 1.1386])}
    case["q"] = rng.random() < 0.6
    if not case["q"]:
        case["Hq"] = 0
    return case | {"B": _log(rng, 1, 256), "ctx": rng.choice([0, _log(rng, 1, 2000)]), "prefix": rng.choice([0, _log(rng, 1, 50000)]),
                   "page": rng.choice([1, 16, 32, 64, 128])}


# ---------------------------------------------------------------- inputs


def _lens(case):
    """Lengths of the sequences' own caches: from 0 to `ctx` in even steps (prepare shuffles them)."""
    B, ctx = case["B"], case["ctx"]
    return [ctx] if B == 1 else [ctx * b // (B - 1) for b in range(B)]


def _pool(case, gen, tokens, dtype):
    """A page pool with room for tokens[i] tokens of each table's row, and the rows' pages in the order of a long-lived
    pool (shuffled), entries past a row's pages set to -1."""
    page = case["page"]
    need = [-(-t // page) for t in tokens]
    width, total = max(1, max(need)), sum(tokens) // page + len(tokens) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    col = torch.arange(width, device="cuda")
    there = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(there, order[(first[:, None] + col).clamp_max(total - 1)], -1).to(torch.int32).contiguous()
    shape = (total, case["Hkv"], page, case["D"])
    pools = [torch.randn(shape, generator=gen, device="cuda", dtype=dtype) for _ in range(2)]
    return pools[0], pools[1], table


def _parents(case, gen):
    B, T = case["B"], case["T"]
    node = torch.arange(T, device="cuda")
    if case["tree"] == "chain":
        parents = (node - 1).expand(B, T)
    else:  # each node below an earlier one or the context's last token; one in sixteen is unused
        parents = (torch.rand(B, T, generator=gen, device="cuda") * (node + 1)).floor().long() - 1
        unused = torch.rand(B, T, generator=gen, device="cuda") < 1 / 16
        parents = torch.where(unused & (node > 0), -2, parents)
    return parents.to(torch.int32).contiguous()


def _frequencies(rot, factor):
    return (BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / factor).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda dt, *s: torch.randn(s, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    shuffled = lambda v: torch.tensor(v, device="cuda")[torch.randperm(len(v), generator=gen, device="cuda")]  # noqa: E731
    st, op = {"case": case}, case["op"]
    if op == "positions":
        st["parents"] = _parents(case, gen)
        st["lens"] = torch.randint(0, case["ctx"] + 1, (case["B"],), generator=gen, device="cuda", dtype=torch.int32)
        st["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
        return st
    if op == "shared":
        B, T, D = case["B"], case["T"], case["D"]
        lens = shuffled(_lens(case))
        # the prefix's pages are of the same pool as the sequences'
        st["k_pages"], st["v_pages"], table = _pool(case, gen, lens.tolist() + [case["prefix"]], torch.bfloat16)
        page = case["page"]
        st["table"] = table[:B, :max(1, -(-case["ctx"] // page))].contiguous()
        st["prefix_table"] = table[B, :max(1, -(-case["prefix"] // page))].contiguous()
        st["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
        st["lens"] = lens.to(torch.int32)
        st["q"] = (1.5 * randn(torch.float32, B, T, case["Hkv"] * case["group"], D)).bfloat16()
        st["k_new"], st["v_new"] = (randn(torch.bfloat16, B, T, case["Hkv"], D) for _ in range(2))
        st["parents"] = _parents(case, gen)
        return st
    dt, rows, Hq, Hkv, D = DTYPES[case["dt"]], case["rows"], case["Hq"], case["Hkv"], case["D"]
    if op == "append" or case["split"]:  # heads of q, k and v side by side in the rows of one projection
        qkv = randn(dt, rows, Hq + 2 * Hkv, D)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        st["q"], st["k"], st["v"] = randn(dt, rows, Hq, D), randn(dt, rows, Hkv, D), None
    if op == "rope":
        st["freqs"] = _frequencies(case["rot"], case["factor"])
        st["positions"] = torch.randint(0, case["far"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
        return st
    if not case["q"]:
        st["q"] = None
    B = case["B"]
    st["freqs"] = _frequencies(case["rot"], 1.0)
    cuts = torch.randint(0, rows + 1, (B - 1,), generator=gen, device="cuda").sort().values  # tokens of each: none to many
    ends = torch.tensor([0, rows], device="cuda")
    starts = torch.cat([ends[:1], cuts, ends[1:]])
    lens = shuffled(_lens(case))
    st["k_pages"], st["v_pages"], st["table"] = _pool(case, gen, (lens + starts[1:] - starts[:-1]).tolist(), dt)
    st["starts"], st["lens"] = starts.to(torch.int32), lens.to(torch.int32)
    st["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms


def _positions(st):
    parents, lens = st["parents"].long(), st["lens"].long()
    B, T = parents.shape
    used = parents >= -1
    above = (parents[:, :, None] == torch.arange(T, device=parents.device)) & used[:, None, :]
    # itself and its ancestors, by powers of the parent relation
    reach = torch.matrix_power(torch.eye(T, device=parents.device) + above.float(), T) > 0
    depth = reach.sum(dim=2) - 1
    return (st["prefix_len"].long() + lens[:, None] + torch.where(used, depth, 0)).to(torch.int32)


def _rotated(x, positions, freqs, layout, amplitude):
    rot = 2 * freqs.numel()
    angle = positions.double()[:, None, None] * freqs.double()
    c, s = (amplitude * angle.cos()).float(), (amplitude * angle.sin()).float()
    f = x.float()
    head, tail = f[..., :rot], f[..., rot:]
    if layout == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([head, tail], dim=-1).to(x.dtype)


def _rope(st):
    case = st["case"]
    turn = lambda x: _rotated(x, st["positions"], st["freqs"], case["layout"], case["amplitude"])  # noqa: E731
    out = [turn(st["q"]), turn(st["k"])]
    return out if st["v"] is None else out + [st["v"].contiguous()]


def _append(st):
    case, starts, lens = st["case"], st["starts"].long(), st["lens"].long()
    page = case["page"]
    row = torch.arange(case["rows"], device=starts.device)
    b = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    at = lens[b] + row - starts[b]
    pages = st["table"].long()[b, at // page]
    turn = lambda x: _rotated(x, at + st["prefix_len"], st["freqs"], case["layout"], 1.0)  # noqa: E731
    st["k_pages"][pages, :, at % page] = turn(st["k"])
    st["v_pages"][pages, :, at % page] = st["v"]
    out = [st["k_pages"], st["v_pages"], (lens + starts[1:] - starts[:-1]).to(torch.int32)]
    return out + [turn(st["q"])] if case["q"] else out


def _shared(st):
    q, parents, lens = st["q"].float(), st["parents"].long(), st["lens"].long()
    B, T, Hq, D = q.shape
    Hkv, page = st["k_pages"].shape[1:3]
    S, P, g = st["table"].shape[1] * page, st["prefix_table"].shape[0] * page, Hq // Hkv
    rows = q.view(B, T, Hkv, g, D)

    def cached(pool, table, n):  # [..., n, Hkv, D]
        pos = torch.arange(n, device=q.device)
        return pool[table.long().clamp_min(0)[..., pos // page], :, pos % page]

    # all rows of the batch against the prefix
    far = torch.arange(P, device=q.device) < st["prefix_len"]
    kp = cached(st["k_pages"], st["prefix_table"], P).float().permute(1, 2, 0).contiguous()
    vp = torch.where(far[:, None, None], cached(st["v_pages"], st["prefix_table"], P).float(), 0.0).transpose(0, 1).contiguous()
    sp = (rows.permute(2, 0, 1, 3, 4).reshape(Hkv, B * T * g, D) @ kp / math.sqrt(D)).masked_fill_(~far, -math.inf)
    # each sequence's against its own cache and the nodes that a node sees: itself and its ancestors
    used = parents >= -1
    above = torch.eye(T, device=q.device) + (parents[:, :, None] == torch.arange(T, device=q.device)).float()
    tree = (torch.matrix_power(above, T) > 0) & used[:, None, :]
    near = torch.arange(S, device=q.device) < lens[:, None]
    sees = torch.cat([near[:, None, :].expand(B, T, S), tree], dim=2) & used[:, :, None]
    ko = torch.cat([cached(st["k_pages"], st["table"], S), st["k_new"]], dim=1).float().permute(0, 2, 3, 1).contiguous()
    vo = torch.cat([cached(st["v_pages"], st["table"], S), st["v_new"]], dim=1).float()
    vo = torch.where(torch.cat([near, used], dim=1)[:, :, None, None], vo, 0.0).transpose(1, 2).contiguous()
    so = rows.permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, D) @ ko / math.sqrt(D)
    so = so.masked_fill_(~sees.repeat_interleave(g, dim=1)[:, None], -math.inf)
    # one softmax over both
    by_seq = lambda x: x.view(Hkv, B, T * g, -1).transpose(0, 1)  # noqa: E731
    by_head = lambda x: x.transpose(0, 1).reshape(Hkv, B * T * g, -1)  # noqa: E731
    top = torch.maximum(by_seq(sp.amax(dim=2)), so.amax(dim=3, keepdim=True))
    top = torch.where(top == -math.inf, 0.0, top)
    wp, wo = sp.sub_(by_head(top)).exp_(), so.sub_(top).exp_()
    total = by_seq(wp.sum(dim=2)) + wo.sum(dim=3, keepdim=True)
    out = (by_seq(wp @ vp) + wo @ vo) / torch.where(total == 0, 1.0, total)
    out = out.view(B, Hkv, T, g, D).permute(0, 2, 1, 3, 4)
    return torch.where(used[:, :, None, None, None], out, 0.0).reshape(B, T, Hq, D).bfloat16()


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import draft_selection_position_amd as dfs

        if op == "positions":
            return dfs.tree_positions(st["parents"], st["lens"], st["prefix_len"])
        if op == "rope":
            got = dfs.rope(st["q"], st["k"], st["v"], st["positions"], st["freqs"], layout=case["layout"],
                           amplitude=case["amplitude"])
            return [t for t in got if t is not None]
        if op == "append":
            q, lens = dfs.cache_append(st["q"], st["k"], st["v"], st["starts"], st["freqs"], st["k_pages"], st["v_pages"],
                                       st["table"], st["lens"], layout=case["layout"], prefix_len=st["prefix_len"])
            return [st["k_pages"], st["v_pages"], lens] + ([q] if case["q"] else [])
        return dfs.tree_attention_shared(st["q"], st["k_new"], st["v_new"], st["parents"], st["k_pages"], st["v_pages"],
                                         st["prefix_table"], st["prefix_len"], st["table"], st["lens"])
    return {"positions": _positions, "rope": _rope, "append": _append, "shared": _shared}[op](st)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "positions":
        return {"bytes": 8 * case["B"] * case["T"] + 4 * case["B"] + 4, "flops": case["B"] * case["T"]}
    if op == "shared":
        lens, B, T, D, Hkv = _lens(case), case["B"], case["T"], case["D"], case["Hkv"]
        Hq = Hkv * case["group"]
        new = 2 * 2 * B * T * D * (Hq + Hkv) + 4 * B * (T + 1)  # q and the output, the nodes' K and V, parents, lengths
        cache = sum(4 * Hkv * D * n + 4 * -(-n // case["page"]) for n in lens + [case["prefix"]])
        return {"bytes": new + cache, "flops": 4 * Hq * D * T * (sum(lens) + B * case["prefix"] + B)}
    rows, D, es = case["rows"], case["D"], 2 if case["dt"] == "bf16" else 4
    v = op == "append" or case["split"]
    return {"bytes": 2 * rows * D * es * (case["Hq"] + (2 if v else 1) * case["Hkv"]) + 4 * rows,
            "flops": 3 * rows * case["rot"] * (case["Hq"] + case["Hkv"])}


# ---------------------------------------------------------------- the definitions in 64 bits


def _turned(x, positions, freqs, layout, amplitude):
    """Pair i of each head, as a complex number, times amplitude exp(i position freqs[i])."""
    n = freqs.numel()
    y = x.double().clone()
    one = slice(0, n) if layout == "half" else slice(0, 2 * n, 2)
    two = slice(n, 2 * n) if layout == "half" else slice(1, 2 * n, 2)
    turn = torch.polar(torch.full_like(freqs.double(), amplitude), freqs.double()[None] * positions.double()[:, None])
    z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * turn[:, None, :]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "positions":
        out = []
        for row, n in zip(st["parents"].tolist(), st["lens"].tolist()):
            depth = []
            for p in row:  # a node's parent comes before it
                depth.append(depth[p] + 1 if p >= 0 and row[p] >= -1 else 0)
            out.append([case["prefix"] + n + d for d in depth])
        return torch.tensor(out, dtype=torch.int32)
    if op == "rope":
        out = [_turned(st[x], st["positions"], st["freqs"], case["layout"], case["amplitude"]) for x in ("q", "k")]
        return out if st["v"] is None else out + [st["v"].double()]
    if op == "append":
        starts, lens, page = st["starts"].tolist(), st["lens"].tolist(), case["page"]
        at = torch.cat([torch.arange(starts[b + 1] - starts[b]) + lens[b] for b in range(case["B"])]).cuda()
        turned = [None if st[x] is None else _turned(st[x], at + case["prefix"], st["freqs"], case["layout"], 1.0) for x in "qk"]
        k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
        for b in range(case["B"]):
            rows = slice(starts[b], starts[b + 1])
            pages = st["table"][b].long()[at[rows] // page]
            k_pages[pages, :, at[rows] % page] = turned[1][rows]
            v_pages[pages, :, at[rows] % page] = st["v"][rows].double()
        new = torch.tensor([lens[b] + starts[b + 1] - starts[b] for b in range(case["B"])], dtype=torch.int32)
        return [k_pages, v_pages, new] + ([turned[0]] if case["q"] else [])
    q, parents = st["q"].double(), st["parents"].tolist()
    B, T, Hq, D = q.shape
    page, g, P = case["page"], case["group"], case["prefix"]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lists = lambda pool, table, n: pool[table[:-(-n // page)].long()].transpose(1, 2).reshape(-1, case["Hkv"], D)[:n].double()  # noqa: E731
    shared = [lists(p, st["prefix_table"], P) for p in (st["k_pages"], st["v_pages"])]
    for b, n in enumerate(st["lens"].tolist()):
        k, v = (torch.cat([pre, lists(p, st["table"][b], n), new[b].double()]).transpose(0, 1).contiguous()
                for pre, p, new in zip(shared, (st["k_pages"], st["v_pages"]), (st["k_new"], st["v_new"])))
        hidden = torch.ones(T, P + n + T, dtype=torch.bool)
        for t in range(T):
            if parents[b][t] < -1:
                continue
            hidden[t, :P + n] = False
            a = t
            while a >= 0 and parents[b][a] >= -1:
                hidden[t, P + n + a] = False
                a = parents[b][a]
        seen = (~hidden).any(dim=1).cuda()[None, None, :, None]
        hidden = hidden.cuda()[None]
        rows = q[b].view(T, case["Hkv"], g, D).permute(1, 2, 0, 3)  # [Hkv, g, T, D]
        for h in range(case["Hkv"]):
            s = (rows[h].reshape(g * T, D) @ k[h].t().contiguous()).view(g, T, -1) / math.sqrt(D)
            p = torch.nan_to_num(torch.softmax(s.masked_fill(hidden, -math.inf), dim=2))
            o = (p.view(g * T, -1) @ v[h]).view(g, T, D)
            out[b, :, h * g:(h + 1) * g] = torch.where(seen[0], o, 0.0).transpose(0, 1)
    return out
