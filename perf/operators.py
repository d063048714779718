"""The serving operators on a paged KV cache: what is measured, and on what.

A decoded context sits in a paged pool ``[L][n_pool][2][bt][C]`` (C = KV heads
x head_dim).  Requests that continue it are sequences of their own: a row of
block numbers, a length, and a reference count per block.  The operators are
the page calls (copy, fork, free, compact) and the attention of a batch whose
sequences share their leading blocks.

Every input comes from the seed.  Ragged lengths are the same numbers for
every seed, dealt to the requests in a seeded order, so a case has one amount
of work.
"""
import math
import random

import torch

own = False

NO_BLOCK = -1


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _attend(name, **kw):
    c = dict(op="attend", name=name, R=1, nq=1, Hq=64, Hkv=8, D=128, bt=16, shared=0, lo=1, hi=512, empty=0,
             dtype="fp16", L=2)
    c.update(kw)
    return c


def listed():
    return [
        # One request decoding over its own short context: the smallest call, all latency.
        _attend("attend-1req-700", R=1, lo=700, hi=700),
        # Multi-head attention (32 x 128, 4096 channels): a short system prompt shared, long ragged contexts of the
        # requests' own, two padded batch slots; 256-token blocks, bf16.
        _attend("attend-mha-24req-ragged", R=24, Hq=32, Hkv=32, bt=256, shared=2, lo=1, hi=4096, empty=2, dtype="bf16"),
        # A 16384-token context decoded once and continued by 64 requests, each a few hundred tokens in.
        _attend("attend-64req-16k-shared", R=64, shared=1024, lo=1, hi=512),
        # The largest: 128 requests with four drafted tokens each over a 32768-token context.
        _attend("attend-128req-4draft-32k", R=128, nq=4, bt=64, shared=512, lo=4, hi=384),
        # A second answer from one short context: one partial block copied, latency.
        dict(name="fork-1of-700", op="fork", n=1, L=32, C=1024, bt=16, parent=700, reserve=40, spare=16),
        # 32 requests admitted on one 4000-token context in 256-token blocks: the copies of the last partial block count.
        dict(name="fork-32of-4000", op="fork", n=32, L=32, C=1024, bt=256, parent=4000, reserve=300, spare=9),
        # A few blocks moved between two places of a pool.
        dict(name="copy-8-blocks", op="copy", n=8, L=32, C=1024, bt=16, pool=64),
        # A long context's blocks (80 layers) copied out of a pool's shared region.
        dict(name="copy-500-blocks-80L", op="copy", n=500, L=80, C=1024, bt=16, pool=1003),
        # One finished request among four gives its blocks back: latency.
        dict(name="free-1of-4", op="free", n=1, slots=4, blocks=45, width=64),
        # A whole batch of long requests sharing a prefix ends at once.
        dict(name="free-256of-300", op="free", n=256, slots=300, blocks=700, width=1024),
        # A small pool after a few requests ended.
        dict(name="compact-90", op="compact", L=32, C=1024, bt=16, pool=90, slots=5, blocks=9, width=16),
        # A serving pool, four tenths of it holes.
        dict(name="compact-1500-80L", op="compact", L=80, C=1024, bt=16, pool=1500, slots=30, blocks=30, width=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "fork", "copy", "free", "compact"])
    if op == "attend":
        while True:
            Hkv, g = rng.choice([1, 4, 8, 8, 32]), rng.choice([1, 4, 5, 7, 8, 8])
            if Hkv * g > 64:
                continue
            D, bt, nq = rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32, 64, 256]), rng.choice([1, 1, 1, 2, 4, 5])
            R = _log(rng, 1, 128)
            shared = rng.choice([0, _log(rng, 16, 32768) // bt, _log(rng, 1024, 32768) // bt])
            hi = _log(rng, nq, 4096)
            c = dict(op=op, R=R, nq=nq, Hq=Hkv * g, Hkv=Hkv, D=D, bt=bt, shared=shared, lo=nq if rng.random() < 0.5 else hi,
                     hi=hi, empty=rng.choice([0, 0, R // 4]), dtype=rng.choice(["fp16", "bf16"]), L=2)
            w, top = work(c), work(listed()[3])
            if w["flops"] <= top["flops"] and R * hi * Hkv * D <= 1 << 27:
                return c
    if op == "fork":
        return dict(op=op, n=_log(rng, 1, 32), L=rng.choice([2, 32, 32]), C=rng.choice([512, 1024, 1024]),
                    bt=rng.choice([16, 32, 64, 256]), parent=_log(rng, 1, 4000), reserve=rng.randint(0, 300), spare=rng.randint(3, 20))
    if op == "copy":
        n = _log(rng, 1, 500)
        return dict(op=op, n=n, L=rng.choice([2, 32, 80]), C=rng.choice([64, 1024, 1024]), bt=rng.choice([8, 16]), pool=2 * n + rng.randint(1, 30))
    if op == "free":
        slots = _log(rng, 1, 300)
        return dict(op=op, n=rng.randint(1, slots), slots=slots, blocks=_log(rng, 2, 700), width=rng.randint(701, 1024))
    slots, blocks = rng.randint(2, 30), rng.randint(1, 30)
    return dict(op=op, L=rng.choice([2, 32, 80]), C=rng.choice([64, 1024, 1024]), bt=rng.choice([8, 16]),
                pool=slots * blocks + rng.randint(0, 600), slots=slots, blocks=blocks, width=blocks + rng.randint(0, 9))


def _own_lens(c):
    """Tokens of each request after the shared blocks: an even spread over [lo, hi], empty slots last."""
    n = c["R"] - c["empty"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(n - 1, 1) for i in range(n)] + [0] * c["empty"]


def _held(c):
    """compact: how many of a slot's blocks are left, by slot (every third slot ended)."""
    return [0 if s % 3 == 1 else c["blocks"] - s % 2 * (c["blocks"] // 3) for s in range(c["slots"])]


def _compact_moves(c, ids):
    live = sorted(ids)
    return sum(b >= len(live) for b in live)


def work(c):
    if c["op"] == "attend":
        P, lens, row = c["shared"] * c["bt"], _own_lens(c), c["Hkv"] * c["D"]
        tokens = P + sum(lens)
        seen = sum(max(0, P + n - c["nq"] + 1 + i) for n in lens if n for i in range(c["nq"]))
        qo = c["R"] * c["nq"] * c["Hq"]
        return {"bytes": tokens * row * 2 * 2 + qo * c["D"] * 2 * 2 + qo * 4, "flops": 4.0 * seen * c["Hq"] * c["D"]}
    if c["op"] == "fork":
        tail = c["parent"] % c["bt"]
        blocks = -(-(c["parent"] + c["reserve"]) // c["bt"])
        return {"bytes": c["n"] * (2 * tail * 2 * c["L"] * c["C"] * 2 + 12 * blocks), "flops": 0}
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * 2 * c["L"] * c["bt"] * c["C"] * 2, "flops": 0}
    if c["op"] == "free":
        return {"bytes": c["n"] * (8 * c["width"] + 8 * c["blocks"]), "flops": 0}
    # The live blocks are spread evenly at random: the moves are the live ones past n_live, pool-wide.
    live = sum(_held(c))
    moves = live * (c["pool"] - live) / c["pool"]
    return {"bytes": 2 * moves * 2 * c["L"] * c["bt"] * c["C"] * 2 + 8 * c["slots"] * c["width"] + 8 * c["pool"], "flops": 0}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(L, n, bt, C, dtype, g):
    x = torch.empty((L, n, 2, bt, C), dtype=dtype, device="cuda")
    sigma = torch.exp(0.5 * torch.randn(C, generator=g, device="cuda"))
    for l in range(L):
        x[l] = torch.randn((n, 2, bt, C), generator=g, device="cuda", dtype=torch.float32 if n * bt * C < 1 << 24 else dtype) * sigma.to(dtype)
    return x


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case=c)
    if c["op"] == "attend":
        dtype = torch.float16 if c["dtype"] == "fp16" else torch.bfloat16
        R, bt, P, C = c["R"], c["bt"], c["shared"] * c["bt"], c["Hkv"] * c["D"]
        lens = _own_lens(c)
        rng.shuffle(lens)
        need = [-(-n // bt) for n in lens]
        n_pool = c["shared"] + sum(need) + 7
        ids = list(range(n_pool))
        rng.shuffle(ids)
        width = c["shared"] + max(need) + 1
        table = torch.full((R + 1, width), NO_BLOCK, dtype=torch.int32)
        table[:, : c["shared"]] = torch.tensor(ids[: c["shared"]], dtype=torch.int32)
        at = c["shared"]
        for r, n in enumerate(need):
            table[r + 1, c["shared"]: c["shared"] + n] = torch.tensor(ids[at: at + n], dtype=torch.int32)
            at += n
        s["pool"] = _pool(c["L"], n_pool, bt, C, dtype, g)
        s["tables"] = table.cuda()
        s["lens"] = _ints([P] + [P + n if n else 0 for n in lens])  # slot 0 is the context itself
        s["slots"] = _ints(range(1, R + 1))
        s["q"] = (1.5 * torch.randn((R, c["nq"], c["Hq"], c["D"]), generator=g, device="cuda")).to(dtype)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((R, c["nq"], c["Hq"]), dtype=torch.float32, device="cuda")
        s["refs"] = torch.ones(n_pool, dtype=torch.int32, device="cuda")
        s["width"] = max(need) * bt  # what a program knows of its longest request
    elif c["op"] == "fork":
        bt, n = c["bt"], c["n"]
        held, width = -(-c["parent"] // bt), -(-(c["parent"] + c["reserve"]) // bt) + 2
        n_pool = held + n * (width - 2 - c["parent"] // bt) + c["spare"]
        ids = list(range(n_pool))
        rng.shuffle(ids)
        table = torch.full((n + 1, width), NO_BLOCK, dtype=torch.int32)
        table[0, :held] = torch.tensor(ids[:held], dtype=torch.int32)
        refs = torch.zeros(n_pool, dtype=torch.int32)
        refs[torch.tensor(ids[: held + c["spare"] // 2])] = 1
        s["pool"] = _pool(c["L"], n_pool, bt, c["C"], torch.float16, g)
        _meta(s, table, [c["parent"]] + [0] * n, refs)
        s["parent"], s["child"], s["reserve"] = _ints([0] * n), _ints(range(1, n + 1)), _ints([c["reserve"]] * n)
    elif c["op"] == "copy":
        ids = list(range(c["pool"]))
        rng.shuffle(ids)
        s["pool"] = _pool(c["L"], c["pool"], c["bt"], c["C"], torch.float16, g)
        s["src"], s["dst"] = _ints(ids[: c["n"]]), _ints(ids[c["n"]: 2 * c["n"]])
        _meta(s, torch.full((1, 1), NO_BLOCK, dtype=torch.int32), [0], torch.ones(c["pool"], dtype=torch.int32))
    elif c["op"] == "free":
        # half of every row is shared by all slots, half is the slot's own
        both, mine = c["blocks"] // 2, c["blocks"] - c["blocks"] // 2
        n_pool = both + mine * c["slots"] + 5
        ids = torch.randperm(n_pool, generator=g, device="cuda").to(torch.int32).cpu()
        table = torch.full((c["slots"], c["width"]), NO_BLOCK, dtype=torch.int32)
        table[:, :both] = ids[:both]
        table[:, both: both + mine] = ids[both: both + mine * c["slots"]].view(c["slots"], mine)
        refs = torch.zeros(n_pool, dtype=torch.int32)
        refs[ids[:both].long()] = c["slots"]
        refs[ids[both: both + mine * c["slots"]].long()] = 1
        s["pool"] = torch.zeros((1, n_pool, 2, 16, 8), dtype=torch.float16, device="cuda")
        _meta(s, table, [16 * c["blocks"] - 3] * c["slots"], refs)
        s["ended"] = _ints(rng.sample(range(c["slots"]), c["n"]))
    else:
        ids = list(range(c["pool"]))
        rng.shuffle(ids)
        table = torch.full((c["slots"], c["width"]), NO_BLOCK, dtype=torch.int32)
        refs = torch.zeros(c["pool"], dtype=torch.int32)
        at = 0
        for k, n in enumerate(_held(c)):
            row = torch.tensor(ids[at: at + n], dtype=torch.int32)
            table[k, :n] = row
            refs[row.long()] = 1
            at += n
        if c["slots"] > 2 and c["blocks"] > 1:  # the first block is shared by two sequences
            first = int(table[0, 0])
            refs[int(table[2, 0])] -= 1
            table[2, 0] = first
            refs[first] += 1
        s["pool"] = _pool(c["L"], c["pool"], c["bt"], c["C"], torch.float16, g)
        _meta(s, table, [n * c["bt"] for n in _held(c)], refs)
        s["remap"] = torch.empty(c["pool"], dtype=torch.int32, device="cuda")
    if own:
        from kv_cache_compression_decode_gb300 import paged
        s["cache"] = paged.PagedCache(s["pool"], s["tables"], s["lens"], s["refs"])
    return s


def _meta(s, table, lens, refs):
    """Tables, lengths and references in one buffer, with a copy of it: a pass starts from the same state each time."""
    flat = torch.cat([table.reshape(-1), torch.tensor(lens, dtype=torch.int32), refs]).cuda()
    n, m = table.numel(), len(lens)
    s["start"], s["state"] = flat, flat.clone()
    s["tables"], s["lens"], s["refs"] = s["state"][:n].view(table.shape), s["state"][n: n + m], s["state"][n + m:]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op not in ("attend", "copy"):
        s["state"].copy_(s["start"])
    (_own if own else _plain)[op](s)
    if op == "attend":
        return {"out": s["out"], "lse": s["lse"]}
    r = {"tables": s["tables"], "lens": s["lens"], "refs": s["refs"]}
    if op != "free":
        r["pool_bits"] = s["pool"].view(torch.int16)
    if op == "compact":
        r["remap"] = s["remap"]
    return r


def _own_attend(s):
    c = s["case"]
    s["cache"].attend(1, s["q"], slots=s["slots"], shared_slot=0, shared_blocks=c["shared"], out=s["out"], lse=s["lse"])


_own = {
    "attend": _own_attend,
    "fork": lambda s: s["cache"].fork(s["parent"], s["child"], s["reserve"]),
    "copy": lambda s: s["cache"].copy(s["src"], s["dst"]),
    "free": lambda s: s["cache"].free(s["ended"]),
    "compact": lambda s: s["cache"].compact(s["remap"]),
}


def _plain_attend(s):
    c = s["case"]
    P, bt, g, R, nq = c["shared"] * c["bt"], c["bt"], c["Hq"] // c["Hkv"], c["R"], c["nq"]
    kv = s["pool"][1]
    slots = s["slots"].long()
    q = s["q"].float().view(R, nq, c["Hkv"], g, c["D"]).permute(2, 0, 1, 3, 4) * (1.0 / math.sqrt(c["D"]))  # [k, R, nq, g, D]
    lens = s["lens"][slots]
    lim = (lens[:, None] - nq + 1 + torch.arange(nq, device="cuda")).clamp(min=0)  # [R, nq]
    both = kv[s["tables"][0, : c["shared"]].long()].view(-1, 2, bt, c["Hkv"], c["D"]).float()
    k0, v0 = both.permute(1, 3, 0, 2, 4).reshape(2, c["Hkv"], P, c["D"]).unbind(0)
    n_own = s["width"]
    mine = s["tables"][slots, c["shared"]: c["shared"] + n_own // bt].long().clamp(min=0)
    k1, v1 = kv[mine].view(R, -1, 2, bt, c["Hkv"], c["D"]).permute(2, 4, 0, 1, 3, 5).reshape(2, c["Hkv"], R, n_own, c["D"]).unbind(0)
    at = torch.arange(n_own, device="cuda")
    seen = (P + at < lim[:, :, None])[None, :, :, None, :]  # [1, R, nq, 1, n_own]
    used = (P + at < lens[:, None])[None, :, :, None]
    s0 = q.reshape(c["Hkv"], -1, c["D"]) @ k0.transpose(1, 2)
    s0 = s0.view(c["Hkv"], R, nq, g, P).masked_fill_((lim == 0)[None, :, :, None, None], -math.inf)
    s1 = (q.reshape(c["Hkv"], R, nq * g, c["D"]) @ k1.float().transpose(2, 3)).view(c["Hkv"], R, nq, g, n_own)
    s1 = s1.masked_fill(~seen, -math.inf)
    m = s1.amax(-1) if P == 0 else torch.maximum(s0.amax(-1), s1.amax(-1))
    m = m.masked_fill(m == -math.inf, 0.0)
    s0 = s0.sub_(m[..., None]).exp_()
    s1 = (s1 - m[..., None]).exp()
    z = s0.sum(-1) + s1.sum(-1)
    o = (s0.view(c["Hkv"], R * nq * g, P) @ v0).view(c["Hkv"], R, nq, g, c["D"])
    o = o + (s1.view(c["Hkv"], R, nq * g, n_own) @ v1.float().masked_fill(~used, 0.0)).view(o.shape)
    o = torch.where(z[..., None] > 0, o / z[..., None], 0.0)
    s["out"].copy_(o.permute(1, 2, 0, 3, 4).reshape(s["out"].shape))
    s["lse"].copy_((m + torch.log(z)).permute(1, 2, 0, 3).reshape(s["lse"].shape))


def _plain_fork(s):
    bt, pool, tables, refs = s["case"]["bt"], s["pool"], s["tables"], s["refs"]
    parent, child = s["parent"].long(), s["child"].long()
    n = s["lens"][parent].long()
    full, total = n // bt, (n + s["reserve"] + bt - 1) // bt
    first = (total - full).cumsum(0) - (total - full)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    col = torch.arange(tables.shape[1], device="cuda")
    old = tables[parent]
    fresh = free[(first[:, None] + col - full[:, None]).clamp(0, refs.numel() - 1)].to(torch.int32)
    row = torch.where(col < full[:, None], old, torch.where(col < total[:, None], fresh, NO_BLOCK))
    # the parents' last partial blocks, rows below the length
    last = full.clamp(max=tables.shape[1] - 1)[:, None]
    src = old.gather(1, last)[:, 0].long().clamp(min=0)
    dst = torch.where(n % bt > 0, row.gather(1, last)[:, 0].long(), src)
    keep = torch.arange(bt, device="cuda") < (n % bt)[:, None]
    pool[:, dst] = torch.where(keep[None, :, None, :, None], pool[:, src], pool[:, dst])
    tables[child] = row
    s["lens"][child] = n.to(torch.int32)
    refs.index_add_(0, row.clamp(min=0).reshape(-1).long(), (row >= 0).to(torch.int32).reshape(-1))


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]


def _plain_free(s):
    at = s["ended"].long()
    row = s["tables"][at].reshape(-1)
    s["refs"].index_add_(0, row.clamp(min=0).long(), -(row >= 0).to(torch.int32))
    s["tables"][at] = NO_BLOCK
    s["lens"][at] = 0


def _plain_compact(s):
    refs, tables = s["refs"], s["tables"]
    live = refs > 0
    ids = torch.arange(refs.numel(), device="cuda")
    n = live.sum()
    src, dst = torch.nonzero(live & (ids >= n))[:, 0], torch.nonzero(~live & (ids < n))[:, 0]
    s["pool"][:, dst] = s["pool"][:, src]
    remap = torch.where(live, ids, NO_BLOCK).to(torch.int32)
    remap[src] = dst.to(torch.int32)
    s["remap"].copy_(remap)
    tables.copy_(torch.where(tables >= 0, remap[tables.clamp(min=0).long()], tables))
    refs[dst] = refs[src]
    refs[src] = 0


_plain = {"attend": _plain_attend, "fork": _plain_fork, "copy": _plain_copy, "free": _plain_free, "compact": _plain_compact}


# ---------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """Attention request by request and head by head in 64 bits; the page calls compute no numbers."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    c, kv = s["case"], s["pool"][1].double()
    tables, lens = s["tables"].tolist(), s["lens"].tolist()
    g = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for r, slot in enumerate(s["slots"].tolist()):
        n = lens[slot]
        blocks = torch.tensor(tables[slot][: -(-n // c["bt"])], dtype=torch.int64, device="cuda")
        rows = kv[blocks].permute(1, 0, 2, 3).reshape(2, -1, c["Hkv"], c["D"])[:, :n]
        for i in range(c["nq"]):
            seen = n - c["nq"] + 1 + i
            if seen <= 0:
                continue
            q = s["q"][r, i].double().view(c["Hkv"], g, c["D"])
            x = torch.einsum("kgd,tkd->kgt", q, rows[0, :seen]) / math.sqrt(c["D"])
            lse[r, i] = torch.logsumexp(x, -1).view(-1)
            out[r, i] = torch.einsum("kgt,tkd->kgd", torch.softmax(x, -1), rows[1, :seen]).reshape(c["Hq"], c["D"])
    return {"out": out, "lse": lse}
