"""Cases of the operators that select: a router's choice of experts with its gradient, and a beam search's choice of
its next beams with the reordering of their states.

Every operator is written twice: in plain torch operations, in 32 bits where an order does not hang on the last bits
and in 64 where it does, and as the library's entry points (used where `own` is true).  `exact` gives the same outputs
in 64 bits from the operators' definitions:

  route       s = softmax or sigmoid of the logits; an expert's choice value is s + bias (without a bias the logit's
              own order).  The experts lie in `groups` of equal size; a group is worth the sum of its `group_top` best
              choice values, the `top_groups` best groups are kept, and ids[t] are their top_k best experts, best
              first, ties to the lowest index.  w = scale * s[ids], with `renorm` divided by the sum over k of s[ids]
  route_grad  the logits' gradient of w for given ids
  select      v[i, w] = score[i] + log_softmax(logits[i])[w] over a batch's beams i and tokens w; the num_out best, best
              first, ties to the lowest (beam, token).  A finished beam has one candidate: the end token at its score
  reorder     state[b, j] = state[b, parent[b, j]], in place or into another buffer
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}
WIDTH = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4, "i64": 8}
END = 2  # the end token's id


def listed():
    return [
        # one token of a request being answered, by groups with a balancing bias: latency alone
        dict(name="route 1 of 256 groups", op="route", tokens=1, experts=256, top_k=8, kind="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", ids="i64", weights="f32"),
        # a training micro-batch over few experts
        dict(name="route 4095 of 8", op="route", tokens=4095, experts=8, top_k=2, kind="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="bf16", ids="i32", weights="f32"),
        # a long batch by groups with a balancing bias: the largest choice
        dict(name="route 65536 of 256 groups", op="route", tokens=65536, experts=256, top_k=8, kind="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", ids="i32", weights="f32"),
        # a small step held in 16 bits, an odd count of experts
        dict(name="route_grad 2047 of 60", op="route_grad", tokens=2047, experts=60, top_k=4, kind="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0, dtype="bf16", ids="i32", weights="f32"),
        # a training batch's weights without renormalisation: every logit has a gradient
        dict(name="route_grad 65536 of 128", op="route_grad", tokens=65536, experts=128, top_k=8, kind="softmax",
             bias=False, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0, dtype="f32", ids="i32",
             weights="f32"),
        # the way back of the choice by groups
        dict(name="route_grad 16384 of 256", op="route_grad", tokens=16384, experts=256, top_k=8, kind="sigmoid",
             bias=True, groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", ids="i64",
             weights="f32"),
        # one request with four beams, a vocabulary whose rows start anywhere
        dict(name="select 1x4 of 50257", op="select", batch=1, beams=4, vocab=50257, num_out=8, finished=0.0,
             dtype="bf16"),
        # a batch of translations in 32 bits, some beams finished
        dict(name="select 16x5 of 32000", op="select", batch=16, beams=5, vocab=32000, num_out=5, finished=0.2,
             dtype="f32"),
        # a large serving batch over a large vocabulary
        dict(name="select 64x8 of 131072", op="select", batch=64, beams=8, vocab=131072, num_out=16, finished=0.0,
             dtype="bf16"),
        # one layer's keys of one request with four beams, 129 positions of a buffer for 512
        dict(name="reorder 1x4 layer", op="reorder", outer=1, batch=1, beams=4, into=4, heads=8, most=512, length=129,
             dim=128, place=True, dtype="bf16"),
        # a prompt's cache, all layers, handed to the beams that start from it
        dict(name="reorder 4x1 to 5", op="reorder", outer=24, batch=4, beams=1, into=5, heads=8, most=400, length=333,
             dim=64, place=False, dtype="bf16"),
        # the caches of eight layers of a serving batch, in place
        dict(name="reorder 16x8 layers", op="reorder", outer=16, batch=16, beams=8, into=8, heads=4, most=512,
             length=501, dim=128, place=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "select", "select", "reorder"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        experts = groups * max(2, _log(rng, 4, 512) // groups)
        top_groups = rng.randint(1, groups)
        top_k = min(rng.randint(1, 8), top_groups * (experts // groups))
        return dict(op=op, tokens=_log(rng, 1, 65536 if experts <= 256 else 32768), experts=experts, top_k=top_k,
                    kind=rng.choice(["softmax", "sigmoid"]), bias=rng.choice([True, False]), groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]), renorm=rng.choice([True, False]),
                    scale=rng.choice([1.0, 2.5]), dtype=dtype, ids=rng.choice(["i32", "i64"]),
                    weights=rng.choice(["f32", dtype]))
    if op == "select":
        c = dict(op=op, batch=_log(rng, 1, 64), beams=rng.randint(1, 16), vocab=_log(rng, 1000, 262144), num_out=0,
                 finished=rng.choice([0.0, 0.0, 0.2]), dtype=dtype)
        c["num_out"] = c["beams"] * rng.choice([1, 2])
        while work(c)["bytes"] > 134 << 20:
            c["batch" if c["batch"] > 1 else "vocab"] //= 2
        return c
    beams, place = rng.randint(2, 16), rng.choice([True, True, False])
    most = _log(rng, 16, 1024)
    c = dict(op=op, outer=_log(rng, 1, 64), batch=_log(rng, 1, 32), beams=beams, into=beams, heads=rng.randint(1, 16),
             most=most, length=rng.randint(1, most), dim=rng.choice([64, 128, 128, rng.randint(1, 200)]), place=place,
             dtype=rng.choice(["bf16", "bf16", "f16", "f32", "i32"]))
    if not place:
        c["beams"] = rng.choice([1, beams])
    while c["outer"] * c["batch"] * c["into"] * c["heads"] * c["most"] * c["dim"] * WIDTH[c["dtype"]] > 1 << 30:
        for size in ("most", "length", "batch", "outer"):
            c[size] = max(1, c[size] // 2)
    return c


def _normal(gen, *shape, dtype=torch.float32, std=1.0):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _taken(case):
    """How often a beam is another's parent, by its place: a good beam has more children than a bad one."""
    edge = np.sqrt(np.arange(case["beams"] + 1) / case["beams"])
    return edge[1:] - edge[:-1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "temp": None}
    dtype = DTYPES[case["dtype"]]
    if case["op"] in ("route", "route_grad"):
        tokens, experts = case["tokens"], case["experts"]
        like = torch.randn(experts, generator=gen, device="cuda")  # some experts are more popular than others
        s["logits"] = (torch.randn(tokens, experts, generator=gen, device="cuda") + 0.7 * like).to(dtype)
        # what balancing made of the popular experts' scores
        s["bias"] = _normal(gen, experts, std=0.02) - 0.03 * like if case["bias"] else None
        s["ids"] = torch.empty(tokens, case["top_k"], dtype=DTYPES[case["ids"]], device="cuda")
        s["weights"] = torch.empty(tokens, case["top_k"], dtype=DTYPES[case["weights"]], device="cuda")
        if case["op"] == "route_grad":
            s["ids"].copy_(_plain_ids(s)[0])
            s["d_weights"] = _normal(gen, tokens, case["top_k"], dtype=DTYPES[case["weights"]])
            s["d_logits"] = torch.empty_like(s["logits"])
        return s
    if case["op"] == "select":
        batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
        s["logits"] = _normal(gen, batch * beams, vocab, dtype=dtype, std=2.5)
        s["scores"] = -4.0 * torch.rand(batch, beams, generator=gen, device="cuda").cumsum(1)  # best first
        s["finished"] = torch.rand(batch, beams, generator=gen, device="cuda") < case["finished"]
        shape = (batch, case["num_out"])
        s["out"] = (torch.empty(shape, device="cuda"), torch.empty(shape, dtype=torch.int32, device="cuda"),
                    torch.empty(shape, dtype=torch.int32, device="cuda"))
        return s
    shape = (case["outer"], case["batch"], case["beams"], case["heads"], case["most"], case["dim"])
    length = case["length"]
    if dtype.is_floating_point:
        whole = _normal(gen, *shape, dtype=dtype)
    else:
        whole = torch.randint(-(1 << 31), 1 << 31, shape, generator=gen, device="cuda", dtype=torch.int64).to(dtype)
    s["state"] = whole[..., :length, :]  # the positions in use of a buffer for more
    u = torch.rand(case["batch"], case["into"], generator=gen, device="cuda", dtype=torch.float64)
    s["parents"] = (u * u * case["beams"]).int().clamp(0, case["beams"] - 1)
    s["out"] = None
    if not case["place"]:
        s["out"] = torch.empty(*shape[:2], case["into"], *shape[3:], dtype=dtype, device="cuda")[..., :length, :]
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from sorting_lsd_radix_gb300 import gbsort

    c = s["case"]
    if c["op"] == "route":
        return gbsort.gbs_expert_route(
            s["logits"], c["top_k"], score_type=_kind(gbsort, c), bias=s["bias"], num_groups=c["groups"],
            top_groups=c["top_groups"], group_top=c["group_top"], renormalise=c["renorm"], scale=c["scale"],
            ids_out=s["ids"], weights_out=s["weights"])
    if c["op"] == "route_grad":
        return gbsort.gbs_expert_route_grad(s["d_weights"], s["logits"], s["ids"], score_type=_kind(gbsort, c),
                                            renormalise=c["renorm"], scale=c["scale"], d_logits_out=s["d_logits"])
    if c["op"] == "select":
        finished = s["finished"] if c["finished"] else None
        out, s["temp"] = gbsort.gbs_beam_select(s["logits"], s["scores"], c["num_out"], finished=finished, end_id=END,
                                                out=s["out"], temp=s["temp"], return_temp=True)
        return out
    return gbsort.gbs_beam_reorder(s["state"], s["parents"], dim=1, out=s["out"])


def _kind(gbsort, c):
    return gbsort.GBS_SCORE_SOFTMAX if c["kind"] == "softmax" else gbsort.GBS_SCORE_SIGMOID


def _scores(logits, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _best(values, count):
    """The `count` largest of each row, largest first, ties to the lowest index."""
    got, at = torch.sort(values, dim=1, descending=True, stable=True)
    return got[:, :count], at[:, :count]


def _plain_ids(s):
    """(ids, the logits in 32 bits).  Choice values are compared in 64 bits: with a bias, thousands of tokens have some
    that are closer to each other than 32 bits tell apart."""
    c, logits = s["case"], s["logits"].float()
    sums = c["groups"] > 1 and c["group_top"] > 1
    choice = _scores(logits.double(), c["kind"]) if c["bias"] or sums else logits
    if c["bias"]:
        choice = choice + s["bias"].double()
    order = choice if c["bias"] else logits
    if c["groups"] > 1:
        tokens, each = logits.size(0), c["experts"] // c["groups"]
        best, _ = _best(choice.view(tokens * c["groups"], each), c["group_top"])
        _, kept = _best(best.sum(1).view(tokens, c["groups"]), c["top_groups"])
        inside = torch.zeros(tokens, c["groups"], dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        order = torch.where(inside.repeat_interleave(each, 1), order, torch.full_like(order, -math.inf))
    return _best(order, c["top_k"])[1], logits


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        ids, logits = _plain_ids(s)
        w = torch.gather(_scores(logits, c["kind"]), 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return ids.to(s["ids"].dtype), (w * c["scale"]).to(s["weights"].dtype)
    if c["op"] == "route_grad":
        ids, g = s["ids"].long(), s["d_weights"].float() * c["scale"]
        score = _scores(s["logits"].float(), c["kind"])
        w = torch.gather(score, 1, ids)
        if c["renorm"]:  # by the sum first
            total = w.sum(1, keepdim=True)
            g = (g - (g * w).sum(1, keepdim=True) / total) / total
        d = torch.zeros_like(score).scatter_add_(1, ids, g)
        if c["kind"] == "sigmoid":
            d = d * score * (1.0 - score)
        else:
            d = score * (d - (d * score).sum(1, keepdim=True))
        return d.to(s["logits"].dtype)
    if c["op"] == "select":
        batch, beams, vocab = c["batch"], c["beams"], c["vocab"]
        logits = s["logits"].double()  # a long sum, and candidates of different beams that come close
        top = logits.amax(1, keepdim=True)
        lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
        score = s["scores"].double().reshape(-1, 1)
        value, at = _best(logits, min(c["num_out"], vocab))
        value = score + (value - lse)
        over = s["finished"].reshape(-1, 1)
        first = torch.arange(value.size(1), device="cuda") == 0
        value = torch.where(over, torch.where(first, score, -math.inf), value)
        at = torch.where(over, END, at)
        beam = torch.arange(beams, device="cuda").repeat(batch)[:, None].expand_as(at)
        got, order = _best(value.reshape(batch, -1), c["num_out"])
        gone = got == -math.inf
        beam = torch.gather(beam.reshape(batch, -1), 1, order).masked_fill(gone, -1)
        token = torch.gather(at.reshape(batch, -1), 1, order).masked_fill(gone, -1)
        return got.float(), beam.int(), token.int()
    row = torch.arange(c["batch"], device="cuda")[:, None]
    picked = s["state"][:, row, s["parents"].long()]
    to = s["state"] if c["place"] else s["out"]
    return to.copy_(picked)


def exact(case, seed):
    """The outputs from the definitions, token by token and beam by beam."""
    s = prepare(case, seed)
    if case["op"] == "reorder":
        state, parents = s["state"], s["parents"].cpu().tolist()
        out = torch.empty(*state.shape[:2], case["into"], *state.shape[3:], dtype=state.dtype, device=state.device)
        for b, of in enumerate(parents):
            for j, i in enumerate(of):
                out[:, b, j] = state[:, b, i]
        return out
    if case["op"] == "select":
        return _exact_select(case, s)
    logits = s["logits"].double().cpu().numpy()
    tokens, experts = logits.shape
    if case["kind"] == "sigmoid":
        score = 0.5 * (1.0 + np.tanh(0.5 * logits))
    else:
        score = np.exp(logits - np.logaddexp.reduce(logits, axis=1, keepdims=True))
    if case["op"] == "route":
        ids = _exact_ids(case, s, logits, score)
        w = np.take_along_axis(score, ids, 1)
        return ids, case["scale"] * (w / w.sum(1, keepdims=True) if case["renorm"] else w)
    ids, g = s["ids"].long().cpu().numpy(), s["d_weights"].double().cpu().numpy() * case["scale"]
    p = np.take_along_axis(score, ids, 1)
    out = np.zeros_like(score)
    if case["kind"] == "sigmoid":
        if case["renorm"]:
            q = p / p.sum(1, keepdims=True)
            part = q * (1.0 - p) * (g - (g * q).sum(1, keepdims=True))
        else:
            part = g * p * (1.0 - p)
    elif case["renorm"]:
        q = p / p.sum(1, keepdims=True)
        part = q * (g - (g * q).sum(1, keepdims=True))
    else:
        out -= score * (g * p).sum(1, keepdims=True)
        part = g * p
    for k in range(case["top_k"]):
        out[np.arange(tokens), ids[:, k]] += part[:, k]
    return out


def _exact_ids(case, s, logits, score):
    choice = score + s["bias"].double().cpu().numpy() if case["bias"] else logits
    tokens, experts = logits.shape
    groups, each = case["groups"], experts // case["groups"]
    if groups > 1:
        worth = choice if case["bias"] or case["group_top"] == 1 else score
        worth = np.sort(worth.reshape(tokens, groups, each), 2)[:, :, ::-1][:, :, :case["group_top"]].sum(2)
        kept = np.argsort(-worth, 1, kind="stable")[:, :case["top_groups"]]
        inside = np.zeros((tokens, groups), bool)
        np.put_along_axis(inside, kept, True, 1)
        choice = np.where(np.repeat(inside, each, 1), choice, -np.inf)
    return np.argsort(-choice, 1, kind="stable")[:, :case["top_k"]]


def _exact_select(case, s):
    beams, count = case["beams"], case["num_out"]
    score, finished = s["scores"].double().cpu().numpy(), s["finished"].cpu().numpy()
    values = np.full((case["batch"], count), -np.inf)
    which, tokens = np.full((case["batch"], count), -1), np.full((case["batch"], count), -1)
    for b in range(case["batch"]):
        found = []
        rows = s["logits"][b * beams:(b + 1) * beams].double().cpu().numpy()
        for i in range(beams):
            if finished[b, i]:
                found.append((-score[b, i], i, END))
                continue
            row = rows[i]
            lse = row.max() + math.log(math.fsum(np.exp(row - row.max())))
            least = np.partition(row, -min(count, row.size))[-min(count, row.size)]
            found += [(-(score[b, i] + (row[w] - lse)), i, int(w)) for w in np.flatnonzero(row >= least)]
        for k, (v, i, w) in enumerate(sorted(found)[:count]):
            values[b, k], which[b, k], tokens[b, k] = -v, i, w
    return values, which, tokens


def work(case):
    if case["op"] in ("route", "route_grad"):
        logits = case["tokens"] * case["experts"] * WIDTH[case["dtype"]]
        slots = case["tokens"] * case["top_k"]
        plan = slots * (WIDTH[case["ids"]] + WIDTH[case["weights"]])
        if case["op"] == "route":
            return {"bytes": logits + plan + 4 * case["experts"] * case["bias"],
                    "flops": 2 * case["tokens"] * case["experts"]}
        if case["kind"] == "softmax" and not case["renorm"]:  # every score is part of the gradient
            return {"bytes": 2 * logits + plan, "flops": 5 * case["tokens"] * case["experts"]}
        return {"bytes": logits + plan + slots * WIDTH[case["dtype"]], "flops": 8 * slots}
    if case["op"] == "select":
        rows = case["batch"] * case["beams"]
        logits = rows * case["vocab"] * (1.0 - case["finished"])
        return {"bytes": logits * WIDTH[case["dtype"]] + rows * 5 + case["batch"] * case["num_out"] * 12,
                "flops": 4 * logits}
    share = _taken(case)
    each = case["outer"] * case["batch"] * case["heads"] * case["length"] * case["dim"] * WIDTH[case["dtype"]]
    others = case["into"] - 1 if case["place"] else case["into"]
    read = float(np.sum(1.0 - (1.0 - share) ** others))
    written = float(np.sum(1.0 - share)) if case["place"] else case["into"]
    return {"bytes": each * (read + written) + 4 * case["batch"] * case["into"], "flops": 0}
