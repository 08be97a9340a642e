"""Row operators on the GPU against plain implementations in 64 bits.

Rows that are only moved, and every index, are compared exactly.  Sums are compared within the bound of
their own arithmetic: m products added in 32 bits in any order are off by at most (m + 2) * 2^-24 of the
sum of their magnitudes, and the result's rounding adds half a unit of its type's last place."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
# half a unit in the last place, relative, and the smallest value's absolute step
UNIT = {torch.float32: (2.0 ** -24, 2.0 ** -149), torch.float16: (2.0 ** -11, 2.0 ** -25),
        torch.bfloat16: (2.0 ** -8, 2.0 ** -133)}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sorting_lsd_radix_gb300 import build as gbuild
    gbuild.build()
    from sorting_lsd_radix_gb300 import gbsort
    gbsort.load()
    return gbsort


def _gen(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) % (1 << 31))


def _normal(gen, *shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, magnitude, terms):
    """|got - want| within the bound for `terms` products whose magnitudes add up to `magnitude`."""
    rel, least = UNIT[got.dtype]
    bound = (terms + 2) * EPS32 * magnitude * (1 + rel) + rel * np.abs(want) + least
    off = np.abs(_f64(got) - want)
    assert np.all(off <= bound), f"off by {np.max(off - bound)} more than the bound"


def plan_by_hand(ids, experts, first=0, align=1, num_rows=None):
    """The order of the slots, expert by expert."""
    flat = ids.cpu().numpy().astype(np.int64).reshape(-1)
    e = flat - first
    e[(flat < first) | (e >= experts)] = -1
    if num_rows is None:
        used = min(experts, flat.size)
        num_rows = (flat.size + used * (align - 1)) // align * align
    slot_of_row, row_of_slot, offsets, counts = np.full(num_rows, -1), np.full(flat.size, -1), [0], []
    order = np.argsort(np.where(e < 0, experts, e), kind="stable")
    at = 0
    for c in np.bincount(e[e >= 0], minlength=experts):
        mine = order[at:at + c]
        slot_of_row[offsets[-1]:offsets[-1] + c] = mine
        row_of_slot[mine] = offsets[-1] + np.arange(c)
        at += c
        counts.append(c)
        offsets.append(offsets[-1] + -(-c // align) * align)
    return slot_of_row, row_of_slot.reshape(ids.shape), np.array(offsets), np.array(counts)


def check_plan(plan, want):
    for got, w, name in zip(plan, want, ("slot_of_row", "row_of_slot", "offsets", "counts")):
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), w), name


def routed(gen, tokens, top_k, experts, low=0, dtype=torch.int64):
    """Expert ids in [low, low + experts), squared so that some experts are popular."""
    u = torch.rand(tokens, top_k, generator=gen, device="cuda")
    return (low + (u * u * experts).long().clamp(max=experts - 1)).to(dtype)


# tokens, top_k, experts, align: single tokens, sizes around a warp, a tile and the change from
# one launch to counted tiles (16384 slots), one expert, the most experts, every tile partly full
PLANS = [(0, 2, 4, 1), (0, 1, 3, 16), (1, 1, 1, 1), (1, 8, 256, 1), (1, 8, 256, 128), (3, 5, 7, 4), (31, 1, 2, 1),
         (33, 2, 1024, 1), (64, 256, 300, 2), (257, 3, 1000, 16), (2048, 8, 64, 1), (2049, 8, 64, 1), (16384, 1, 1, 128),
         (16385, 1, 9, 1), (4099, 7, 1024, 128), (40000, 3, 33, 5), (300, 256, 1024, 1)]


@pytest.mark.parametrize("tokens,top_k,experts,align", PLANS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_is_the_stable_order(g, tokens, top_k, experts, align, dtype):
    ids = routed(_gen(1, tokens, experts), tokens, top_k, experts, dtype=dtype)
    plan, temp = g.gbs_expert_sort(ids, experts, row_align=align, return_temp=True)
    check_plan(plan, plan_by_hand(ids, experts, 0, align))
    assert g.gbs_get_status(temp) == g.GBS_OK


@pytest.mark.parametrize("tokens,top_k", [(5, 3), (700, 4), (9000, 2)])
@pytest.mark.parametrize("first", [0, 5, -7, 2 ** 31 - 20])
def test_sort_of_a_shard(g, tokens, top_k, first):
    """Ids below and above the shard's, and the types' extremes, have no row."""
    ids = routed(_gen(2, tokens, first), tokens, top_k, 40, low=first - 8)
    ids[0, 0], ids[-1, -1] = -1, 2 ** 63 - 1
    ids[tokens // 2, 0] = -2 ** 63
    check_plan(g.gbs_expert_sort(ids, 24, first_expert=first, row_align=4),
               plan_by_hand(ids, 24, first, 4))
    narrow = ids.clamp(-2 ** 31, 2 ** 31 - 1).int()
    check_plan(g.gbs_expert_sort(narrow, 24, first_expert=first), plan_by_hand(narrow, 24, first, 1))


def test_sort_with_no_slot_kept_and_with_spare_rows(g):
    ids = torch.full((50, 2), -1, device="cuda")
    check_plan(g.gbs_expert_sort(ids, 6), plan_by_hand(ids, 6))
    ids = routed(_gen(3), 50, 2, 6)
    check_plan(g.gbs_expert_sort(ids, 6, row_align=8, num_rows=1000), plan_by_hand(ids, 6, 0, 8, 1000))


def test_sort_above_the_long_tiles(g):
    """More than 2^22 slots: tiles of 4096 slots."""
    ids = routed(_gen(4), (1 << 22) // 8 + 77, 8, 129, dtype=torch.int32)
    check_plan(g.gbs_expert_sort(ids, 128, row_align=2), plan_by_hand(ids, 128, 0, 2))


# row lengths that take every word width, end inside a warp's segment, and cross several
LENGTHS = [1, 2, 8, 33, 130, 256, 517, 1000, 1029, 2056]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("row_len", LENGTHS)
@pytest.mark.parametrize("tokens,top_k,experts,align", [(0, 2, 4, 1), (1, 8, 256, 16), (37, 3, 5, 4), (9001, 2, 3, 1)])
def test_dispatch_and_gather_move_rows(g, dtype, row_len, tokens, top_k, experts, align):
    gen = _gen(5, row_len, tokens)
    ids, x = routed(gen, tokens, top_k, experts + 1), _normal(gen, tokens, row_len, dtype=dtype)
    want = plan_by_hand(ids, experts, 0, align)
    rows, plan = g.gbs_expert_dispatch(x, ids, experts, row_align=align)
    check_plan(plan, want)
    slot = torch.from_numpy(want[0]).cuda()
    if tokens:
        expect = torch.where((slot >= 0)[:, None], x[slot.clamp(min=0) // top_k], torch.zeros((), dtype=dtype, device="cuda"))
    else:
        expect = torch.zeros(slot.numel(), row_len, dtype=dtype, device="cuda")
    assert torch.equal(rows, expect)
    again = torch.full_like(rows, float("nan"))
    assert g.gbs_expert_gather(x, plan[0], plan[1], rows_out=again) is again
    assert torch.equal(again, expect)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_with_strides(g, dtype):
    """Rows inside wider ones, at odd places, and one row for all tokens; what lies between is left alone."""
    gen = _gen(6)
    for row_len, start, width in ((64, 8, 80), (64, 1, 67), (65, 3, 96)):
        wide = _normal(gen, 200, width, dtype=dtype)
        x, ids = wide[:, start:start + row_len], routed(gen, 200, 2, 9)
        room = torch.full((400, width), 7.0, dtype=dtype, device="cuda")
        rows, plan = g.gbs_expert_dispatch(x, ids, 9, rows_out=room[:, start:start + row_len])
        slot = plan[0].long()
        assert torch.equal(rows, x[slot // 2])
        room[:, start:start + row_len] = 7.0
        assert torch.all(room == 7.0)
        rows.copy_(x[slot // 2])
        back = torch.full((200, width), 7.0, dtype=dtype, device="cuda")
        out = g.gbs_expert_combine(rows, plan[1], out=back[:, start:start + row_len])
        assert torch.equal(out, (x.float() * 2).to(dtype))
        back[:, start:start + row_len] = 7.0
        assert torch.all(back == 7.0)
    one = _normal(gen, 1, 64, dtype=dtype).expand(200, 64)
    rows, plan = g.gbs_expert_dispatch(one, ids, 9)
    assert torch.equal(rows, one[:1].expand(400, 64))
    weights = _normal(gen, 200, 2)
    d_rows, d_weights = g.gbs_expert_combine_grad(one, rows, plan[0], plan[1], weights)
    flat = g.gbs_expert_combine_grad(one.contiguous(), rows, plan[0], plan[1], weights)
    assert torch.equal(d_rows, flat[0]) and torch.equal(d_weights, flat[1])


def combine_by_hand(rows, row_of_slot, weights):
    r, y = row_of_slot.cpu().numpy(), _f64(rows)
    w = np.ones(r.shape) if weights is None else _f64(weights)
    terms = np.where((r >= 0)[..., None], np.where(r >= 0, w, 0)[..., None] * y[np.maximum(r, 0)], 0)
    return terms.sum(1), np.abs(terms).sum(1)


MOVES = [(1, 1, 1, 1), (1, 8, 64, 16), (5, 3, 4, 8), (64, 2, 3, 1), (130, 8, 16, 1), (33, 17, 40, 4), (20, 70, 90, 1),
         (2500, 4, 6, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight_type", ["f32", "row", None])
@pytest.mark.parametrize("row_len", [1, 6, 40, 513, 2048])
@pytest.mark.parametrize("tokens,top_k,experts,align", MOVES)
def test_combine_and_its_gradient(g, dtype, weight_type, row_len, tokens, top_k, experts, align):
    gen = _gen(7, row_len, tokens, top_k)
    plan = g.gbs_expert_sort(routed(gen, tokens, top_k, experts + 1), experts, row_align=align)
    slot_of_row, row_of_slot = plan[:2]
    rows = _normal(gen, slot_of_row.numel(), row_len, dtype=dtype)
    rows[slot_of_row < 0] = float("nan")  # never read
    weights = None
    if weight_type:
        weights = _normal(gen, tokens, top_k, dtype=torch.float32 if weight_type == "f32" else dtype)
        weights[row_of_slot < 0] = float("inf")  # never used
    out = g.gbs_expert_combine(rows, row_of_slot, weights)
    rows_known = torch.where((slot_of_row >= 0)[:, None], rows, torch.zeros_like(rows))
    want, magnitude = combine_by_hand(rows_known, row_of_slot, weights)
    _close(out, want, magnitude, top_k)
    if weights is None:
        return
    d_out = _normal(gen, tokens, row_len, dtype=dtype)
    d_rows, d_weights = g.gbs_expert_combine_grad(d_out, rows, slot_of_row, row_of_slot, weights)
    slot, r = slot_of_row.cpu().numpy(), row_of_slot.cpu().numpy()
    at, d, w = np.maximum(slot, 0), _f64(d_out), _f64(torch.where(row_of_slot >= 0, weights, torch.zeros_like(weights)))
    want = np.where((slot >= 0)[:, None], w.reshape(-1)[at][:, None] * d[at // top_k], 0)
    _close(d_rows, want, np.abs(want), 1)
    terms = np.where((r >= 0)[..., None], d[:, None, :] * _f64(rows_known)[np.maximum(r, 0)], 0)
    _close(d_weights, terms.sum(2), np.abs(terms).sum(2), row_len)


def test_gradients_agree_with_differences(g):
    """combine is linear in the rows and in the weights: a central difference is exact up to rounding."""
    gen = _gen(8)
    tokens, top_k, row_len, h = 6, 3, 24, 0.25
    ids = routed(gen, tokens, top_k, 5)
    x = _normal(gen, tokens, row_len)
    rows, (slot_of_row, row_of_slot, _, _) = g.gbs_expert_dispatch(x, ids, 4)
    weights, d_out = _normal(gen, tokens, top_k), _normal(gen, tokens, row_len)

    def loss(rows, weights):
        return float((g.gbs_expert_combine(rows, row_of_slot, weights).double() * d_out.double()).sum())

    d_rows, d_weights = g.gbs_expert_combine_grad(d_out, rows, slot_of_row, row_of_slot, weights)
    # each loss is off by at most the sum of its outputs' bounds, each difference by that over h
    _, magnitude = combine_by_hand(rows.abs() + h, row_of_slot, weights.abs() + h)
    slack = (top_k + 3) * EPS32 * float((np.abs(_f64(d_out)) * magnitude).sum()) / h
    for t in range(tokens):
        for k in range(top_k):
            if row_of_slot[t, k] < 0:
                assert float(d_weights[t, k]) == 0.0
                continue
            e = torch.zeros_like(weights)
            e[t, k] = h
            diff = (loss(rows, weights + e) - loss(rows, weights - e)) / (2 * h)
            assert abs(diff - float(d_weights[t, k])) <= 2 * slack
    for r in range(0, rows.shape[0], 3):
        e = torch.zeros_like(rows)
        e[r, r % row_len] = h
        diff = (loss(rows + e, weights) - loss(rows - e, weights)) / (2 * h)
        assert abs(diff - float(d_rows[r, r % row_len])) <= 2 * slack
    # dispatch's gradient is combine without weights
    d_x = g.gbs_expert_combine(d_rows, row_of_slot)
    for t in range(tokens):
        e = torch.zeros_like(x)
        e[t, t] = h
        up, down = (g.gbs_expert_gather(x + s * e, slot_of_row, row_of_slot).double() for s in (1, -1))
        diff = float(((up - down) * d_rows.double()).sum()) / (2 * h)
        assert abs(diff - float(d_x[t, t])) <= 2 * slack


def test_infinities_and_nans_go_where_the_formulas_send_them(g):
    ids = torch.tensor([[0, 1], [1, 0], [0, 1]], device="cuda")
    slot_of_row, row_of_slot, _, _ = g.gbs_expert_sort(ids, 2)
    rows = torch.ones(6, 8, device="cuda")
    rows[row_of_slot[0, 0], 0], rows[row_of_slot[1, 1], 1] = float("inf"), float("nan")
    weights = torch.tensor([[0.5, 0.5], [0.25, 0.75], [1.0, 2.0]], device="cuda")
    out = g.gbs_expert_combine(rows, row_of_slot, weights)
    assert out[0, 0] == float("inf") and torch.isnan(out[1, 1])
    assert torch.isfinite(out).sum() == out.numel() - 2
    _, d_weights = g.gbs_expert_combine_grad(torch.ones(3, 8, device="cuda"), rows, slot_of_row, row_of_slot, weights)
    assert d_weights[0, 0] == float("inf") and torch.isnan(d_weights[1, 1])
    assert torch.isfinite(d_weights).sum() == 4


IDS = [(0, 10), (1, 1), (1, 1000), (7, 3), (33, 33), (64, 2), (257, 100), (1000, 9000), (5000, 17), (16385, 20000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("row_len", [1, 6, 40, 513, 2048])
@pytest.mark.parametrize("n,vocab", IDS)
def test_lookup(g, dtype, row_len, n, vocab):
    gen = _gen(9, n, row_len)
    table = _normal(gen, vocab, row_len, dtype=dtype)
    ids = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    assert torch.equal(g.gbs_embedding_lookup(table, ids), table[ids])
    narrow = ids.int()
    narrow[::3] -= vocab  # below the shard
    got = g.gbs_embedding_lookup(table, narrow + 11, scale=0.3, first_id=11)
    want = _f64(table)[ids.cpu().numpy()] * float(np.float32(0.3))
    want[::3] = 0
    _close(got, want, np.abs(want), 1)
    assert not torch.any(got[::3])


def test_lookup_shapes_strides_and_shards(g):
    gen = _gen(10)
    wide = _normal(gen, 90, 200, dtype=torch.bfloat16)
    ids = torch.randint(0, 90, (3, 5, 2), generator=gen, device="cuda")
    table = wide[:, 3:131]
    assert torch.equal(g.gbs_embedding_lookup(table, ids), table[ids])
    parts = [g.gbs_embedding_lookup(table[a:a + 30], ids, first_id=a) for a in (0, 30, 60)]
    assert torch.equal(parts[0] + parts[1] + parts[2], table[ids])
    ids[0, 0, 0], ids[1, 1, 1], ids[2, 4, 0] = -1, 2 ** 63 - 1, -2 ** 63
    got = g.gbs_embedding_lookup(table, ids, scale=-1.0)
    assert not torch.any(got[0, 0, 0]) and not torch.any(got[1, 1, 1]) and not torch.any(got[2, 4, 0])
    assert not torch.any(torch.signbit(got[0, 0, 0]))
    assert not torch.any(g.gbs_embedding_lookup(table[:0], ids))


def grad_by_hand(d_out, ids, grad, scale, first, accumulate, skip=None):
    """(sums, magnitudes, most terms of a row), a row of ids at a time."""
    i = ids.cpu().numpy().astype(np.int64).reshape(-1)
    inside = (i >= first) & (i - first < grad.shape[0]) & (i != (skip if skip is not None else first - 1))
    d = _f64(d_out).reshape(i.size, grad.shape[1])[inside] * float(np.float32(scale))
    at = i[inside] - first
    total = _f64(grad) if accumulate else np.zeros(grad.shape)
    size = np.abs(total)
    order = np.argsort(at, kind="stable")
    if order.size:
        start = np.flatnonzero(np.diff(at[order], prepend=-1))
        total[at[order][start]] += np.add.reduceat(d[order], start, axis=0)
        size[at[order][start]] += np.add.reduceat(np.abs(d[order]), start, axis=0)
    return total, size, int(np.bincount(at).max()) if at.size else 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("grad_type", ["f32", "row"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("row_len", [1, 6, 136, 513, 2056])
@pytest.mark.parametrize("n,vocab", IDS)
def test_embedding_grad(g, dtype, grad_type, accumulate, row_len, n, vocab):
    if n * row_len > 1 << 24 or vocab * row_len > 1 << 23:
        row_len //= 4
    gen = _gen(11, n, row_len)
    d_out = _normal(gen, n, row_len, dtype=dtype)
    # squared: the first ids have long runs of equal keys
    u = torch.rand(n, generator=gen, device="cuda")
    ids = (u ** 3 * vocab).to(torch.int64 if row_len % 2 else torch.int32)
    grad = _normal(gen, vocab, row_len, dtype=torch.float32 if grad_type == "f32" else dtype)
    want, magnitude, terms = grad_by_hand(d_out, ids, grad, 0.7, 0, accumulate)
    before = grad.clone()
    got, temp = g.gbs_embedding_grad(d_out, ids, grad, scale=0.7, accumulate=accumulate, return_temp=True)
    assert got is grad
    _close(grad, want, magnitude, terms + 1)
    assert g.gbs_get_status(temp) == g.GBS_OK
    again = g.gbs_embedding_grad(d_out, ids, before, scale=0.7, accumulate=accumulate, temp=temp)
    assert torch.equal(again, grad)  # equal bits


# lengths of one id's run around the chunks of sorted positions, and places of the run in them
@pytest.mark.parametrize("before", [0, 1, 31, 32, 63])
@pytest.mark.parametrize("run", [1, 2, 31, 32, 33, 64, 65, 127, 300, 5000])
def test_embedding_grad_runs(g, before, run):
    gen = _gen(12, before, run)
    ids = torch.cat([torch.arange(before), torch.full((run,), 100), torch.arange(101, 140), torch.tensor([140] * 70)])
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(run))].cuda()
    d_out = _normal(gen, ids.numel(), 72)
    for accumulate in (False, True):
        grad = _normal(gen, 150, 72)
        want, magnitude, terms = grad_by_hand(d_out, ids, grad, 1.0, 0, accumulate)
        g.gbs_embedding_grad(d_out, ids, grad, accumulate=accumulate)
        _close(grad, want, magnitude, terms + 1)


# list lengths on both sides of each form of the ids' order, and keys of one, two and three digits
@pytest.mark.parametrize("n,vocab", [(8192, 3), (8193, 900), (8193, 3_000_000), (20_000, 1 << 20), (1 << 20, 70_000),
                                     ((1 << 20) + 1, 70_000), (1_500_000, 1), (1 << 17, 900_000), ((1 << 17) + 1, 20_000),
                                     ((1 << 17) + 1, 3_000_000), (1 << 19, 1000), ((1 << 19) + 1, 1000),
                                     (9216, 900), (9217, 900), (9216, 3_000_000)])
def test_embedding_grad_orders(g, n, vocab):
    gen = _gen(22, n)
    ids = (torch.rand(n, generator=gen, device="cuda") ** 2 * (vocab + 2)).long() - 1  # some on either side
    d_out = _normal(gen, n, 2)
    for accumulate in (False, True):
        grad = _normal(gen, vocab, 2)
        want, magnitude, terms = grad_by_hand(d_out, ids, grad, 1.0, 0, accumulate)
        g.gbs_embedding_grad(d_out, ids, grad, accumulate=accumulate)
        _close(grad, want, magnitude, terms + 1)


@pytest.mark.parametrize("vocab", [(1 << 24) - 2, (1 << 24) - 1, 1 << 24, (1 << 24) + 9])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_embedding_grad_at_the_end_of_a_long_table(g, vocab, id_type):
    """Neighbouring keys around 2^24, where f32 stops telling whole numbers apart, and ids past the table."""
    gen = _gen(23, vocab)
    ids = (vocab - 40 + torch.randint(0, 45, (5000,), generator=gen, device="cuda")).to(id_type)
    d_out = _normal(gen, 5000, 2)
    grad = _normal(gen, vocab, 2)
    want, magnitude, terms = grad_by_hand(d_out, ids.long(), grad, 1.0, 0, True)
    g.gbs_embedding_grad(d_out, ids, grad, accumulate=True)
    _close(grad[-64:], want[-64:], magnitude[-64:], terms + 1)
    assert np.array_equal(_f64(grad[:-64]), want[:-64])


@pytest.mark.parametrize("dtype,row_len", [(torch.float32, 24), (torch.bfloat16, 40), (torch.float16, 21)])
@pytest.mark.parametrize("n", [70_001, 200_003])
def test_embedding_grad_of_long_lists(g, dtype, row_len, n):
    """Chunks of every length; runs from one position to a third of the list."""
    gen = _gen(21, n, row_len)
    u = torch.rand(n, generator=gen, device="cuda")
    ids = torch.where(u < 0.3, torch.full_like(u, 777), torch.exp((u - 0.3) / 0.7 * np.log(5001.0)) - 1).long()
    d_out = _normal(gen, n, row_len, dtype=dtype)
    for accumulate in (False, True):
        grad = _normal(gen, 5000, row_len)
        want, magnitude, terms = grad_by_hand(d_out, ids, grad, 1.0, 0, accumulate)
        g.gbs_embedding_grad(d_out, ids, grad, accumulate=accumulate)
        _close(grad, want, magnitude, terms + 1)


def test_embedding_grad_of_a_shard_with_padding(g):
    gen = _gen(13)
    ids = torch.randint(0, 300, (40, 25), generator=gen, device="cuda")
    ids[3, 4], ids[5, 6], ids[7, 8] = -1, 2 ** 63 - 1, -2 ** 63
    d_out = _normal(gen, 40, 25, 64, dtype=torch.bfloat16)
    d_out[ids == 130] = float("nan")  # the padding's gradient is never read into a sum
    grad = _normal(gen, 100, 96)
    view, rest = grad[:, 16:80], grad[:, 80:].clone()
    zeroed = torch.where((ids == 130)[..., None], torch.zeros_like(d_out), d_out)
    want, magnitude, terms = grad_by_hand(zeroed, ids, view, 2.0, 100, True, skip=130)
    g.gbs_embedding_grad(d_out, ids, view, scale=2.0, first_id=100, padding_id=130, accumulate=True)
    _close(view, want, magnitude, terms + 1)
    assert torch.equal(grad[:, 80:], rest)
    g.gbs_embedding_grad(d_out, ids, view, first_id=10 ** 9)  # no id inside: every row is zeroed
    assert not torch.any(view) and torch.equal(grad[:, 80:], rest)


def test_embedding_grad_of_a_broadcast_row(g):
    ids = torch.randint(0, 50, (999,), generator=_gen(14), device="cuda")
    row = _normal(_gen(15), 1, 128, dtype=torch.bfloat16)
    grad = torch.empty(50, 128, device="cuda")
    g.gbs_embedding_grad(row.expand(999, 128), ids, grad)
    counts = torch.bincount(ids, minlength=50)
    want = _f64(row) * counts.cpu().numpy()[:, None]
    _close(grad, want, np.abs(want), int(counts.max()))


def test_embedding_grad_agrees_with_differences(g):
    """lookup is linear in the table."""
    gen = _gen(16)
    table, ids = _normal(gen, 12, 16), torch.randint(-2, 14, (40,), generator=gen, device="cuda")
    d_out, h = _normal(gen, 40, 16), 0.5
    grad = g.gbs_embedding_grad(d_out, ids, torch.empty_like(table), scale=1.5)
    slack = 4 * EPS32 * 1.5 * float((d_out.abs().double() * (float(table.abs().max()) + h)).sum()) / h \
        + 42 * EPS32 * 1.5 * float(d_out.abs().double().sum())
    for v in range(12):
        e = torch.zeros_like(table)
        e[v, v] = h
        up, down = (g.gbs_embedding_lookup(table + s * e, ids, scale=1.5).double() for s in (1, -1))
        assert abs(float(((up - down) * d_out.double()).sum()) / (2 * h) - float(grad[v, v])) <= slack


def test_offsets_past_32_bits(g):
    """Tables and rows of more than 2^32 bytes."""
    gen = _gen(17)
    vocab, row_len = 700_001, 4096
    table = torch.empty(vocab, row_len, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(vocab - 1000, vocab, (500,), generator=gen, device="cuda")
    table[vocab - 1000:] = _normal(gen, 1000, row_len, dtype=torch.bfloat16)
    assert torch.equal(g.gbs_embedding_lookup(table, ids), table[ids])
    d_out = _normal(gen, 500, row_len, dtype=torch.bfloat16)
    want, magnitude, terms = grad_by_hand(d_out, ids - (vocab - 1000), table[vocab - 1000:], 1.0, 0, True)
    g.gbs_embedding_grad(d_out, ids, table, accumulate=True)
    _close(table[vocab - 1000:], want, magnitude, terms + 1)
    del table
    tokens, top_k = 300_000, 8
    ids = routed(gen, tokens, top_k, 16)
    x = _normal(gen, tokens, 1024, dtype=torch.bfloat16)
    rows, plan = g.gbs_expert_dispatch(x, ids, 16)
    assert torch.equal(rows[-5000:], x[plan[0][-5000:].long() // top_k])
    assert torch.equal(rows[:5000], x[plan[0][:5000].long() // top_k])
    out = g.gbs_expert_combine(rows, plan[1])
    assert torch.equal(out, (x.float() * top_k).to(torch.bfloat16))
    d_rows, d_weights = g.gbs_expert_combine_grad(x, rows, plan[0], plan[1], torch.ones(tokens, top_k, device="cuda"))
    assert torch.equal(d_rows, rows)
    want = (x[-1000:].double() ** 2).sum(1).cpu().numpy()[:, None].repeat(top_k, 1)
    _close(d_weights[-1000:], want, want, 1024)


def test_calls_with_every_output_given(g):
    """A caller's outputs and work buffer: the same results as when the calls make them, the caller's own tensors
    back, and the same refusals."""
    assert g._fast is not None  # the compiled calls are built and loaded
    gen = _gen(23)
    tokens, top_k, experts, row_len = 300, 3, 10, 72
    for dtype, ids_type, weight_type in ((torch.bfloat16, torch.int64, torch.float32),
                                         (torch.float32, torch.int32, torch.float32),
                                         (torch.float16, torch.int32, torch.float16)):
        ids, x = routed(gen, tokens, top_k, experts + 2, dtype=ids_type), _normal(gen, tokens, row_len, dtype=dtype)
        rows, plan, temp = g.gbs_expert_dispatch(x, ids, experts, first_expert=1, row_align=4, return_temp=True)
        rows2, plan2 = torch.empty_like(rows), tuple(torch.empty_like(t) for t in plan)
        got = g.gbs_expert_dispatch(x, ids, experts, first_expert=1, row_align=4, rows_out=rows2, plan_out=plan2, temp=temp)
        assert got[0] is rows2 and got[1] is plan2
        assert torch.equal(rows, rows2) and all(torch.equal(a, b) for a, b in zip(plan, plan2))
        for t in plan2:
            t.fill_(7)
        assert g.gbs_expert_sort(ids, experts, 1, 4, plan_out=plan2, temp=temp) is plan2
        assert all(torch.equal(a, b) for a, b in zip(plan, plan2))
        rows2.fill_(7)
        assert g.gbs_expert_gather(x, plan[0], plan[1], rows_out=rows2) is rows2 and torch.equal(rows, rows2)
        weights = _normal(gen, tokens, top_k, dtype=weight_type)
        for w in (weights, None):
            out = g.gbs_expert_combine(rows, plan[1], w)
            out2 = torch.empty_like(out)
            assert g.gbs_expert_combine(rows, plan[1], w, out=out2) is out2 and torch.equal(out, out2)
        d = g.gbs_expert_combine_grad(x, rows, plan[0], plan[1], weights)
        d2 = tuple(torch.empty_like(t) for t in d)
        got = g.gbs_expert_combine_grad(x, rows, plan[0], plan[1], weights, *d2)
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(got, d2, d))
        words = torch.randint(-3, 60, (tokens,), generator=gen, device="cuda").to(ids_type)
        out = g.gbs_embedding_lookup(x[:50], words, scale=0.5, first_id=2)
        assert g.gbs_embedding_lookup(x[:50], words, scale=0.5, first_id=2, out=out2) is out2 and torch.equal(out, out2)
        grad, temp = g.gbs_embedding_grad(x, words, torch.ones(50, row_len, device="cuda"), 0.5, 2, 7, True, return_temp=True)
        grad2 = torch.ones(50, row_len, device="cuda")
        assert g.gbs_embedding_grad(x, words, grad2, 0.5, 2, 7, True, temp=temp) is grad2 and torch.equal(grad, grad2)
        # a work buffer that is too small is replaced, and the call done
        small, bigger = temp[:256], g.gbs_embedding_grad(x, words, torch.ones_like(grad), 0.5, 2, 7, True, temp=temp[:256],
                                                         return_temp=True)
        assert torch.equal(bigger[0], grad) and bigger[1].numel() > small.numel()
        for bad in (dict(out=out2[:, :8]), dict(out=out2[:7]), dict(out=out2[:, ::2]), dict(out=out2.cpu())):
            with pytest.raises(ValueError):
                g.gbs_embedding_lookup(x[:50], words, **bad)
            with pytest.raises(ValueError):
                g.gbs_expert_combine(rows, plan[1], weights, **bad)
        with pytest.raises(TypeError):
            g.gbs_embedding_lookup(x[:50], words, out=out2.double())
        with pytest.raises(TypeError):
            g.gbs_expert_combine(rows, plan[1].long(), weights, out=out2)
        with pytest.raises(ValueError):
            g.gbs_expert_combine(rows, plan[1], weights[1:], out=out2)
        with pytest.raises(ValueError):
            g.gbs_expert_dispatch(x, ids, experts, rows_out=rows2, plan_out=(*plan2[:3], plan2[3][1:]), temp=temp)
        with pytest.raises(g.GbsError):  # fewer rows than the slots may need
            g.gbs_expert_dispatch(x, ids, experts, row_align=4, rows_out=rows2[:-4], plan_out=(plan2[0][:-4], *plan2[1:]), temp=temp)


def test_calls_on_another_stream(g):
    """Everything a call makes belongs to its stream; the same results as on the current one."""
    gen = _gen(18)
    ids, x = routed(gen, 3000, 4, 20), _normal(gen, 3000, 264, dtype=torch.float16)
    words = torch.randint(0, 500, (3000,), generator=gen, device="cuda")
    rows, plan = g.gbs_expert_dispatch(x, ids, 20)
    grad = g.gbs_embedding_grad(x, words, torch.empty(500, 264, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        rows2, plan2 = g.gbs_expert_dispatch(x, ids, 20, stream=handle)
        out2 = g.gbs_expert_combine(rows2, plan2[1], stream=handle)
        grad2 = g.gbs_embedding_grad(x, words, torch.empty(500, 264, device="cuda"), stream=handle)
        side.synchronize()
        assert torch.equal(rows, rows2) and all(torch.equal(a, b) for a, b in zip(plan, plan2))
        assert torch.equal(out2, g.gbs_expert_combine(rows, plan[1]))
        assert torch.equal(grad, grad2)


def test_calls_in_a_cuda_graph(g):
    gen = _gen(19)
    ids, x = routed(gen, 40, 4, 20), _normal(gen, 40, 512, dtype=torch.bfloat16)
    words = torch.randint(0, 90, (700,), generator=gen, device="cuda")
    d_out = _normal(gen, 700, 512, dtype=torch.bfloat16)
    grad = torch.empty(90, 512, device="cuda")
    rows, plan, temp = g.gbs_expert_dispatch(x, ids, 20, return_temp=True)
    out = g.gbs_expert_combine(rows, plan[1])
    _, temp2 = g.gbs_embedding_grad(d_out, words, grad, return_temp=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gbs_expert_dispatch(x, ids, 20, rows_out=rows, plan_out=plan, temp=temp)
        g.gbs_expert_combine(rows, plan[1], out=out)
        g.gbs_embedding_grad(d_out, words, grad, temp=temp2)
    ids.copy_(routed(gen, 40, 4, 20))
    words.copy_(torch.randint(0, 90, (700,), generator=gen, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    check_plan(plan, plan_by_hand(ids, 20))
    assert torch.equal(rows, x[plan[0].long() // 4])
    want, magnitude, terms = grad_by_hand(d_out, words, grad, 1.0, 0, False)
    _close(grad, want, magnitude, terms + 1)


def test_embedding_grad_reports_a_sort_that_timed_out(g):
    """A tile of the ids' sort that never publishes its counts: the bounded wait ends, the status says so, and
    the next call is right."""
    gen = _gen(20)
    n = (1 << 20) + 4 * g.gbs_debug_radix_tile_keys(4, value_bytes=4) + 3  # a length that the radix sort takes
    ids = torch.randint(0, 5000, (n,), generator=gen, device="cuda")
    d_out, grad = _normal(gen, n, 8), torch.zeros(5000, 8, device="cuda")
    temp = g.gbs_embedding_grad(d_out, ids, grad, return_temp=True)[1]
    torch.cuda.synchronize()
    g.gbs_debug_set_lookback_fault(0, 1, 1 << 12)
    try:
        g.gbs_embedding_grad(d_out, ids, torch.zeros_like(grad), temp=temp)
        assert g.gbs_get_status(temp) == g.GBS_ERR_TIMEOUT
    finally:
        g.gbs_debug_set_lookback_fault(-1, 0, 0)
    again = g.gbs_embedding_grad(d_out, ids, torch.zeros_like(grad), temp=temp)
    assert g.gbs_get_status(temp) == g.GBS_OK
    assert torch.equal(again, grad)


class _PlainModel(torch.nn.Module):
    """RoutedModel's formulas by torch's own indexing, in 64 bits."""

    def __init__(self, model):
        super().__init__()
        self.top_k, self.scale = model.top_k, float(np.float32(model.scale))
        for name, value in model.named_parameters():
            setattr(self, name, torch.nn.Parameter(value.detach().double()))

    def loss(self, ids):
        x = self.table[ids[:-1]] * self.scale
        score, experts = torch.topk(x @ self.router.t(), self.top_k, dim=-1)
        up, down = self.up[experts], self.down[experts]
        y = torch.einsum("tkho,tko->tkh", down, torch.nn.functional.silu(torch.einsum("tkoh,th->tko", up, x)))
        x = x + (torch.softmax(score, -1)[..., None] * y).sum(1)
        return torch.nn.functional.cross_entropy(x @ self.table.t(), ids[1:])


def test_a_model_trains_through_the_operators(g):
    """One step's gradients in 32 bits against 64 bits, and a loss that falls in 16 bits."""
    from sorting_lsd_radix_gb300 import routed
    torch.manual_seed(5)
    model = routed.RoutedModel(vocab=300, hidden=72, inner=40, num_experts=6, top_k=2, dtype=torch.float32)
    ids = torch.randint(0, 300, (257,), generator=_gen(24), device="cuda")
    plain = _PlainModel(model)
    allowed = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        loss, want = model.loss(ids), plain.loss(ids)
        loss.backward()
        want.backward()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allowed
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    for name, value in model.named_parameters():
        exact = getattr(plain, name).grad
        # some ten products of 40 to 300 terms lie behind each value: well under 1e-4 of the gradient's norm in 32 bits
        assert float((value.grad.double() - exact).norm()) <= 1e-4 * float(exact.norm()), name
    model = routed.RoutedModel(vocab=512, hidden=64, inner=64, num_experts=4, top_k=2)
    optimizer = torch.optim.AdamW(model.parameters(), lr=3e-3)
    text = (torch.arange(513, device="cuda") * 7919) % 509
    losses = []
    for _ in range(20):
        optimizer.zero_grad()
        losses.append(model.loss(text))
        losses[-1].backward()
        optimizer.step()
    assert float(losses[-1].detach()) < 0.7 * float(losses[0].detach())


def test_gradients_of_broadcast_and_padded_inputs(g):
    """What autograd sends back: a sum's gradient has stride 0 everywhere, and padding gets none."""
    from sorting_lsd_radix_gb300 import routed
    gen = _gen(25)
    table = _normal(gen, 40, 24).requires_grad_()
    ids = torch.randint(0, 40, (3, 50), generator=gen, device="cuda")
    routed.embedding(table, ids, 2.0, padding_id=7).sum().backward()
    want = 2.0 * torch.bincount(ids.view(-1), minlength=40).double()
    want[7] = 0
    assert torch.equal(table.grad.double(), want[:, None].expand(40, 24))
    x, weights = _normal(gen, 30, 24).requires_grad_(), torch.rand(30, 2, generator=gen, device="cuda").requires_grad_()
    rows, slot_of_row, row_of_slot, _, _ = routed.expert_dispatch(x, routed_ids := routed_pairs(gen, 30), 5, row_align=4)
    routed.expert_combine(rows, weights, slot_of_row, row_of_slot).sum().backward()
    kept = ((routed_ids >= 0) & (routed_ids < 5)).double()
    want = (kept * weights.detach().double()).sum(1)
    _close(x.grad, want[:, None].expand(30, 24).cpu().numpy(), want[:, None].expand(30, 24).cpu().numpy(), 2)
    sums = x.detach().double().sum(1)[:, None] * kept
    _close(weights.grad, sums.cpu().numpy(), (x.detach().double().abs().sum(1)[:, None] * kept).cpu().numpy(), 24)


def routed_pairs(gen, tokens):
    """Two different experts of six for each token; five of them are here."""
    return torch.topk(torch.rand(tokens, 6, generator=gen, device="cuda"), 2, dim=1)[1]


@pytest.mark.parametrize("n,row_len", [(64, 64), (900, 1024), (5000, 96), (9000, 40), (20_000, 33)])
def test_calls_in_a_row_see_each_other(g, n, row_len):
    """Every call reads what the one before it wrote and writes over what an earlier one read, with nothing between
    them; each pair of calls is exact and undoes itself, so that the rows come back bit by bit."""
    gen = _gen(31, n)
    x = _normal(gen, n, row_len)
    a, b, rows, back = x.clone(), torch.empty_like(x), torch.empty(2 * n, row_len, device="cuda"), torch.empty_like(x)
    ones = torch.ones(n, 1, device="cuda")
    parts = torch.tensor([0.5, 0.5], device="cuda").repeat(n, 1)
    turns, plans = [], []
    for k in range(6):
        perm = torch.randperm(n, generator=gen, device="cuda")
        pairs = torch.stack([torch.randint(0, 4, (n,), generator=gen, device="cuda"),
                             torch.randint(4, 8, (n,), generator=gen, device="cuda")], 1)
        turns.append((perm, pairs, pairs[:, :1].contiguous()))
        plans.append((g.gbs_expert_sort(pairs, 8), g.gbs_expert_sort(turns[-1][2], 8)))
    torch.cuda.synchronize()
    for (perm, pairs, single), (two, one) in zip(turns, plans):
        g.gbs_embedding_lookup(a, perm, out=b)                                    # b[i] = a[perm[i]]
        g.gbs_embedding_grad(b, perm, a)                                          # a[perm[i]] = b[i]
        g.gbs_expert_dispatch(a, pairs, 8, rows_out=rows)
        g.gbs_expert_combine(rows, two[1], parts, out=b)                          # x / 2 + x / 2
        g.gbs_expert_gather(b, one[0], one[1], rows_out=rows[:n])
        g.gbs_expert_combine(rows[:n], one[1], ones, out=back)
        g.gbs_expert_combine_grad(back, rows[:n], one[0], one[1], ones, d_rows_out=rows[n:])
        g.gbs_expert_combine(rows[n:], one[1], None, out=a)
    assert torch.equal(a, x)
    assert torch.equal(b, x)
