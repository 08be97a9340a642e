"""Cases of the row operators that follow a sort: token rows grouped by expert and back, with the router's
weights and their gradient, and embedding rows looked up by id, with the table's gradient by sorted ids.

Every operator is written twice: in plain torch operations in 32 bits, and as the library's entry points (used
where `own` is true).  `exact` gives the same outputs in 64 bits from the operators' definitions:

  dispatch      the stable order of the slots (t, k) by expert; expert e's rows start at offsets[e], a multiple of
                `align`; rows[r] = x[t] for the slot (t, k) at row r, zeros in the rows that hold no slot
  combine       out[t] = sum over k of w[t, k] * rows[row_of_slot[t, k]], without the slots that have no row
  combine_grad  d_rows[r] = w[t, k] * d_out[t], zeros in the rows without a slot;
                d_w[t, k] = d_out[t] . rows[row_of_slot[t, k]], 0 for a slot without a row
  lookup        out[i] = scale * table[ids[i] - first], zeros where that is outside the table
  grad          grad[v] = (grad[v] +) scale * sum of d_out[i] over the i with ids[i] - first == v
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}


def listed():
    return [
        # one token of a request being answered, routed over many experts: latency alone
        dict(name="dispatch 1x8", op="dispatch", tokens=1, top_k=8, experts=256, first=0, routed=256, hidden=7168,
             align=1, dtype="bf16", ids="i64"),
        # a training micro-batch over few experts, rows padded to the 128-row tiles of a matrix product
        dict(name="dispatch 4095x2 pad", op="dispatch", tokens=4095, top_k=2, experts=8, first=0, routed=8,
             hidden=4096, align=128, dtype="bf16", ids="i64"),
        # a long batch over many experts: the largest row movement
        dict(name="dispatch 65536x8", op="dispatch", tokens=65536, top_k=8, experts=128, first=0, routed=128,
             hidden=2048, align=1, dtype="bf16", ids="i32"),
        # a decoding batch coming back from its experts
        dict(name="combine 64x8", op="combine", tokens=64, top_k=8, experts=256, first=0, routed=256, hidden=7168,
             align=1, dtype="bf16", weights="f32"),
        # a prompt batch on a shard of the experts: the slots of the other shards have no row here
        dict(name="combine 16384x8 shard", op="combine", tokens=16384, top_k=8, experts=48, first=8, routed=64,
             hidden=4096, align=16, dtype="bf16", weights="f32"),
        # a small training step held in 32 bits
        dict(name="combine_grad 2047x2 f32", op="combine_grad", tokens=2047, top_k=2, experts=8, first=0, routed=8,
             hidden=1032, align=1, dtype="f32", weights="f32"),
        # a training batch's way back through the weighted sum
        dict(name="combine_grad 16384x8", op="combine_grad", tokens=16384, top_k=8, experts=64, first=0, routed=64,
             hidden=4096, align=1, dtype="bf16", weights="bf16"),
        # the newest token of each of 32 requests
        dict(name="lookup 32", op="lookup", tokens=32, vocab=131072, first=0, all_ids=131072, hidden=8192,
             dtype="bf16", ids="i64", scale=1.0),
        # a training batch on a quarter of a sharded vocabulary, scaled by sqrt(hidden)
        dict(name="lookup 131072 shard", op="lookup", tokens=131072, vocab=65536, first=65536, all_ids=262144,
             hidden=2048, dtype="bf16", ids="i64", scale=45.254833995939045),
        # a short step into a 32-bit gradient that is kept over micro-batches
        dict(name="grad 999 add", op="grad", tokens=999, vocab=32000, first=0, all_ids=32000, hidden=1024,
             dtype="bf16", ids="i64", grad="f32", add=True, scale=1.0),
        # a training batch's whole table gradient
        dict(name="grad 8192 whole", op="grad", tokens=8192, vocab=50257, first=0, all_ids=50257, hidden=2048,
             dtype="bf16", ids="i64", grad="bf16", add=False, scale=1.0),
        # a long batch into a kept 32-bit gradient: runs of thousands of equal ids beside single ones
        dict(name="grad 131072 add", op="grad", tokens=131072, vocab=131072, first=0, all_ids=131072, hidden=4096,
             dtype="bf16", ids="i32", grad="f32", add=True, scale=64.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _hidden(rng):
    h = _log(rng, 64, 8192)
    step = rng.choice([128, 128, 8, 1])  # mostly whole cache lines, some rows that end inside one
    h = max(64, h // step * step)
    return h + 8 if h == 3 * 1024 else h


def draw(rng):
    c = _drawn(rng)
    while work(c)["bytes"] > 2 << 30:  # the largest listed cases' size
        for size in ("tokens", "vocab", "all_ids", "first"):
            if size in c and (size != "tokens" or c["tokens"] > 1):
                c[size] //= 2
    return c


def _drawn(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "lookup", "grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    hidden = _hidden(rng)
    ids = rng.choice(["i32", "i64"])
    if op in ("lookup", "grad"):
        vocab = _log(rng, 1000, 131072)
        tokens = _log(rng, 1, 131072)
        shards = rng.choice([1, 1, 1, 2, 4]) if tokens >= 64 else 1  # so that some ids fall into the shard
        first = vocab * rng.randrange(shards)
        scale = rng.choice([1.0, math.sqrt(hidden)])
        c = dict(op=op, tokens=tokens, vocab=vocab, first=first, all_ids=vocab * shards, hidden=hidden, dtype=dtype,
                 ids=ids, scale=scale)
        if op == "grad":
            c["grad"] = rng.choice(["f32", "f32", dtype])
            c["add"] = rng.choice([True, False])
        return c
    experts = _log(rng, 4, 384)
    top_k = min(rng.randint(1, 8), experts)
    tokens = _log(rng, 1, 65536)
    routed, first = experts, 0
    if tokens >= 64 and rng.random() < 0.3:
        routed = 2 * experts
        first = rng.choice([0, experts])
    align = rng.choice([1, 1, 1, 16, 128])
    c = dict(op=op, tokens=tokens, top_k=top_k, experts=experts, first=first, routed=routed, hidden=hidden,
             align=align if tokens * top_k >= 64 else 1, dtype=dtype)
    if op == "dispatch":
        c["ids"] = ids
    else:
        c["weights"] = rng.choice(["f32", dtype])
    return c


def _row_count(case):
    """Rows that hold every slot whatever the router says: each expert in use may leave align - 1 rows empty."""
    slots, align = case["tokens"] * case["top_k"], case["align"]
    return (slots + min(case["experts"], slots) * (align - 1)) // align * align


def _route(case, gen):
    """A router's choice: top_k different experts for each token, some experts much more popular than others."""
    like = torch.randn(case["routed"], generator=gen, device="cuda")
    score = torch.randn(case["tokens"], case["routed"], generator=gen, device="cuda") + 0.7 * like
    value, ids = torch.topk(score, case["top_k"], dim=1)
    return ids, torch.softmax(value, dim=1)


def _plan(ids, case):
    """The stable order of the slots by expert: (slot_of_row, row_of_slot, offsets, counts)."""
    experts, align, count = case["experts"], case["align"], _row_count(case)
    flat = ids.reshape(-1).long() - case["first"]
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    by, order = torch.sort(key, stable=True)
    start = torch.searchsorted(by, torch.arange(experts + 1, device=by.device))
    counts = start[1:] - start[:-1]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=by.device)
    offsets[1:] = torch.cumsum((counts + align - 1) // align * align, 0)
    row = offsets[by] + torch.arange(by.numel(), device=by.device) - start[by]
    row_of_slot = torch.empty_like(row)
    row_of_slot[order] = torch.where(by < experts, row, torch.full_like(row, -1))
    slot_of_row = torch.full((count + 1,), -1, dtype=torch.int64, device=by.device)
    slot_of_row[torch.where(by < experts, row, torch.full_like(row, count))] = order
    return slot_of_row[:count].int(), row_of_slot.view(ids.shape).int(), offsets.int(), counts.int()


def _tokens(case, gen):
    """Token ids as text has them: the r-th most frequent id about 1/r as often as the first, in any order of ids."""
    u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(case["all_ids"] + 1.0)) - 1.0).long().clamp(0, case["all_ids"] - 1)
    place = torch.randperm(case["all_ids"], generator=gen, device="cuda")
    return place[rank].to(DTYPES[case["ids"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, hidden = DTYPES[case["dtype"]], case["hidden"]

    def normal(*shape, dtype=dtype, std=1.0):
        got = torch.empty(*shape, dtype=dtype, device="cuda")
        return got.normal_(0.0, std, generator=gen)

    def room(*shape, dtype=dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = {"case": case, "temp": None}
    if case["op"] == "lookup":
        s["ids"] = _tokens(case, gen)
        s["table"] = normal(case["vocab"], hidden, std=0.02)
        s["out"] = room(case["tokens"], hidden)
    elif case["op"] == "grad":
        s["ids"] = _tokens(case, gen)
        s["d_out"] = normal(case["tokens"], hidden, std=0.02)
        s["grad"] = normal(case["vocab"], hidden, dtype=DTYPES[case["grad"]], std=0.02)  # what earlier micro-batches left
    else:
        tokens, top_k, count = case["tokens"], case["top_k"], _row_count(case)
        ids, weights = _route(case, gen)
        if case["op"] == "dispatch":
            s["x"] = normal(tokens, hidden)
            s["ids"] = ids.to(DTYPES[case["ids"]]).contiguous()
            s["rows"] = room(count, hidden)
            s["plan"] = (room(count, dtype=torch.int32), room(tokens, top_k, dtype=torch.int32),
                         room(case["experts"] + 1, dtype=torch.int32), room(case["experts"], dtype=torch.int32))
        else:
            s["slot_of_row"], s["row_of_slot"], _, _ = _plan(ids, case)
            s["rows"] = normal(count, hidden)
            s["weights"] = weights.to(DTYPES[case["weights"]]).contiguous()
            if case["op"] == "combine":
                s["out"] = room(tokens, hidden)
            else:
                s["d_out"] = normal(tokens, hidden)
                s["d_rows"] = room(count, hidden)
                s["d_weights"] = torch.empty_like(s["weights"])
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from sorting_lsd_radix_gb300 import gbsort

    c = s["case"]
    if c["op"] == "dispatch":
        rows, plan, s["temp"] = gbsort.gbs_expert_dispatch(
            s["x"], s["ids"], c["experts"], first_expert=c["first"], row_align=c["align"], rows_out=s["rows"],
            plan_out=s["plan"], temp=s["temp"], return_temp=True)
        return rows, *plan
    if c["op"] == "combine":
        return gbsort.gbs_expert_combine(s["rows"], s["row_of_slot"], s["weights"], out=s["out"])
    if c["op"] == "combine_grad":
        return gbsort.gbs_expert_combine_grad(s["d_out"], s["rows"], s["slot_of_row"], s["row_of_slot"], s["weights"],
                                              d_rows_out=s["d_rows"], d_weights_out=s["d_weights"])
    if c["op"] == "lookup":
        return gbsort.gbs_embedding_lookup(s["table"], s["ids"], scale=c["scale"], first_id=c["first"], out=s["out"])
    grad, s["temp"] = gbsort.gbs_embedding_grad(s["d_out"], s["ids"], s["grad"], scale=c["scale"],
                                                first_id=c["first"], accumulate=c["add"], temp=s["temp"],
                                                return_temp=True)
    return grad


def _picked(s):
    """The slots' rows in 32 bits, zeros for the slots without one."""
    row = s["row_of_slot"].long()
    return torch.where((row >= 0)[..., None], s["rows"][row.clamp(min=0)].float(), torch.zeros((), device="cuda"))


def _run_plain(s):
    c = s["case"]
    dtype, zero = DTYPES[c["dtype"]], torch.zeros((), device="cuda")
    if c["op"] == "dispatch":
        plan = _plan(s["ids"], c)
        slot = plan[0].long()
        rows = torch.where((slot >= 0)[:, None], s["x"][slot.clamp(min=0) // c["top_k"]], zero.to(dtype))
        return rows, *plan
    if c["op"] == "combine":
        return (_picked(s) * s["weights"].float()[..., None]).sum(1).to(dtype)
    if c["op"] == "combine_grad":
        slot, d_out = s["slot_of_row"].long(), s["d_out"].float()
        at = slot.clamp(min=0)
        d_rows = s["weights"].float().reshape(-1)[at][:, None] * d_out[at // c["top_k"]]
        d_rows = torch.where((slot >= 0)[:, None], d_rows, zero).to(dtype)
        return d_rows, (_picked(s) * d_out[:, None, :]).sum(2).to(s["weights"].dtype)
    at = s["ids"].long() - c["first"]
    inside = (at >= 0) & (at < c["vocab"])
    if c["op"] == "lookup":
        got = s["table"][torch.where(inside, at, torch.zeros_like(at))].float() * c["scale"]
        return torch.where(inside[:, None], got, zero).to(dtype)
    total = torch.zeros(c["vocab"] + 1, c["hidden"], device="cuda")  # one row more for the ids outside
    total.index_add_(0, torch.where(inside, at, torch.full_like(at, c["vocab"])), s["d_out"].float())
    total = total[:c["vocab"]] * c["scale"]
    s["grad"].copy_(s["grad"].float() + total if c["add"] else total)
    return s["grad"]


def exact(case, seed):
    """The outputs in 64 bits, slot by slot and id by id from the definitions."""
    s = prepare(case, seed)
    tokens, hidden = case["tokens"], case["hidden"]
    if case["op"] in ("lookup", "grad"):
        ids = s["ids"].cpu().numpy().astype(np.int64) - case["first"]
        here = np.flatnonzero((ids >= 0) & (ids < case["vocab"]))
        place = torch.from_numpy(here).cuda()
        if case["op"] == "lookup":
            out = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
            out[place] = s["table"][torch.from_numpy(ids[here]).cuda()].double().mul_(case["scale"])
            return out
        out = s["grad"].double() if case["add"] else torch.zeros(case["vocab"], hidden, dtype=torch.float64,
                                                                 device="cuda")
        to = torch.from_numpy(ids[here]).cuda()
        for c in range(0, hidden, 512):  # a block of columns at a time
            part = s["d_out"][place, c:c + 512].double() * case["scale"]
            block = out[:, c:c + 512].contiguous()
            out[:, c:c + 512] = block.index_put_((to,), part, accumulate=True)
        return out
    count, top_k, align, experts = _row_count(case), case["top_k"], case["align"], case["experts"]
    if case["op"] == "dispatch":
        expert = s["ids"].cpu().numpy().astype(np.int64).reshape(-1) - case["first"]
        expert[(expert < 0) | (expert >= experts)] = -1
        slot_of_row, offsets = np.full(count, -1, np.int64), [0]
        for e in range(experts):
            mine = np.flatnonzero(expert == e)
            slot_of_row[offsets[-1]:offsets[-1] + mine.size] = mine
            offsets.append(offsets[-1] + -(-mine.size // align) * align)
        used = np.flatnonzero(slot_of_row >= 0)
        rows = torch.zeros(count, hidden, dtype=torch.float64, device="cuda")
        rows[torch.from_numpy(used).cuda()] = s["x"].double()[torch.from_numpy(slot_of_row[used] // top_k).cuda()]
        row_of_slot = np.full(tokens * top_k, -1, np.int64)
        row_of_slot[slot_of_row[used]] = used
        counts = np.bincount(expert[expert >= 0], minlength=experts)
        return rows, slot_of_row, row_of_slot.reshape(tokens, top_k), np.array(offsets), counts
    row = s["row_of_slot"].long()
    weights = s["weights"].double()
    if case["op"] == "combine":
        out = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
        for k in range(top_k):
            at = torch.nonzero(row[:, k] >= 0)[:, 0]
            out[at] += weights[at, k][:, None] * s["rows"][row[at, k]].double()
        return out
    d_rows = torch.zeros(count, hidden, dtype=torch.float64, device="cuda")
    d_weights = torch.zeros(tokens, top_k, dtype=torch.float64, device="cuda")
    for k in range(top_k):
        at = torch.nonzero(row[:, k] >= 0)[:, 0]
        d_out = s["d_out"][at].double()
        d_rows[row[at, k]] = weights[at, k][:, None] * d_out
        d_weights[at, k] = torch.einsum("th,th->t", d_out, s["rows"][row[at, k]].double())
    return d_rows, d_weights


def _touched(case):
    """(tokens whose id is in the table, different ones among them), expected for _tokens' distribution.

    The ids in any order put a table of a share of all ids on that share of the ranks."""
    rank = np.arange(case["all_ids"], dtype=np.float64)
    p = np.log((rank + 2.0) / (rank + 1.0)) / math.log(case["all_ids"] + 1.0)
    share = case["vocab"] / case["all_ids"]
    return case["tokens"] * share, float(np.sum(-np.expm1(case["tokens"] * np.log1p(-p)))) * share


def work(case):
    width = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4, "i64": 8}
    h, e = case["hidden"], width[case["dtype"]]
    if case["op"] in ("lookup", "grad"):
        n = case["tokens"]
        inside, different = _touched(case)
        if case["op"] == "lookup":
            return {"bytes": n * width[case["ids"]] + (different + n) * h * e, "flops": inside * h}
        g = width[case["grad"]]
        table = 2 * different * h * g if case["add"] else case["vocab"] * h * g
        return {"bytes": n * width[case["ids"]] + inside * h * e + table, "flops": inside * h}
    tokens, slots, count = case["tokens"], case["tokens"] * case["top_k"], _row_count(case)
    inside = slots * case["experts"] / case["routed"]
    if case["op"] == "dispatch":
        plan = slots * (width[case["ids"]] + 4) + count * 4 + case["experts"] * 8
        return {"bytes": plan + tokens * h * e + count * h * e, "flops": 0}
    w = width[case["weights"]]
    if case["op"] == "combine":
        return {"bytes": slots * (4 + w) + inside * h * e + tokens * h * e, "flops": 2 * inside * h}
    return {"bytes": slots * (4 + 2 * w) + count * 4 + tokens * h * e + inside * h * e + count * h * e,
            "flops": 3 * inside * h}
