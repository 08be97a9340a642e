"""Row operators on the GPU at the ends of their ranges."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_rows import (EPS32, UNIT, _close, _gen, _normal, check_plan, g, grad_by_hand,  # noqa: E402,F401
                                 plan_by_hand)

pytestmark = pytest.mark.gpu

LAST = 2 ** 63 - 1


def _ids_at_the_end(gen, shape, first):
    """Ids first .. 2^63 - 1, and as many from -2^63 on, which come after them in arithmetic modulo 2^64."""
    near = torch.randint(0, LAST - first + 1, shape, generator=gen, device="cuda") + first
    low = torch.randint(0, 6, shape, generator=gen, device="cuda") - 2 ** 63
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.5, near, low)


@pytest.mark.parametrize("tokens,top_k", [(7, 3), (700, 4), (9000, 2)])
def test_experts_at_the_last_ids(g, tokens, top_k):
    """A shard that would end past 2^63 - 1: the lowest ids are not in it."""
    first = LAST - 2
    ids = _ids_at_the_end(_gen(1, tokens), (tokens, top_k), first)
    # first + 8 experts is above 2^63: in whole numbers only 2^63 - 3 .. 2^63 - 1 are there
    shifted = torch.where(ids >= first, ids - first, torch.full_like(ids, -1))
    check_plan(g.gbs_expert_sort(ids, 8, first_expert=first), plan_by_hand(shifted, 8))


# lists that are compared, placed directly, sorted by digits and by the radix sort
@pytest.mark.parametrize("n", [60, 3000, 20_000, 700_000])
def test_embedding_at_the_last_ids(g, n):
    gen, first, vocab = _gen(2, n), LAST - 4, 9
    ids = _ids_at_the_end(gen, (n,), first)
    shifted = torch.where(ids >= first, ids - first, torch.full_like(ids, -1))
    table, d_out = _normal(gen, vocab, 8), _normal(gen, n, 8)
    want = torch.where((shifted >= 0)[:, None], table[shifted.clamp(min=0)], torch.zeros((), device="cuda"))
    assert torch.equal(g.gbs_embedding_lookup(table, ids, first_id=first), want)
    want, magnitude, terms = grad_by_hand(d_out, shifted, table, 1.0, 0, True)
    g.gbs_embedding_grad(d_out, ids, table, first_id=first, accumulate=True)
    _close(table, want, magnitude, terms + 1)


def _address(t):
    return t.data_ptr() if t is not None else None


# rows of one pack, a short kernel's and a long kernel's, odd ones
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("row_len", [8, 500, 513, 2048])
def test_combine_grad_without_weights_or_their_gradient(g, dtype, row_len):
    """Weights that are ones, and a weights' gradient that nobody wants: the same rows, and nothing else is read."""
    gen = _gen(3, row_len)
    tokens, top_k = 300, 3
    ids = torch.randint(-1, 6, (tokens, top_k), generator=gen, device="cuda")
    slot_of_row, row_of_slot = g.gbs_expert_sort(ids, 5, row_align=4)[:2]
    rows, d_out = _normal(gen, slot_of_row.numel(), row_len, dtype=dtype), _normal(gen, tokens, row_len, dtype=dtype)
    weights = _normal(gen, tokens, top_k)
    rows[slot_of_row < 0] = float("nan")
    ones = torch.ones_like(weights)
    with_ones = g.gbs_expert_combine_grad(d_out, rows, slot_of_row, row_of_slot, ones)
    unread = torch.full_like(rows, float("nan"))
    d_rows, none = g.gbs_expert_combine_grad(d_out, unread, slot_of_row, row_of_slot, None)
    assert none is None and torch.equal(d_rows, with_ones[0])
    assert torch.equal(d_rows, g.gbs_expert_gather(d_out, slot_of_row, row_of_slot))
    given = torch.empty_like(d_rows)
    assert g.gbs_expert_combine_grad(d_out, unread, slot_of_row, row_of_slot, None, given)[0] is given
    assert torch.equal(given, d_rows)
    want = g.gbs_expert_combine_grad(d_out, rows, slot_of_row, row_of_slot, weights)
    for w, d_w in ((weights, None), (None, torch.empty_like(weights)), (None, None)):
        given.fill_(7)
        st = g.load().gbs_expert_combine_grad(
            g._ROW_TYPE[dtype], d_out.data_ptr(), row_len, rows.data_ptr() if d_w is not None else None, row_len,
            slot_of_row.numel(), slot_of_row.data_ptr(), row_of_slot.data_ptr(), g.GBS_ROW_F32, _address(w), tokens, top_k,
            row_len, given.data_ptr(), row_len, _address(d_w), torch.cuda.current_stream().cuda_stream)
        assert st == g.GBS_OK
        assert torch.equal(given, want[0] if w is not None else with_ones[0])
        assert d_w is None or torch.equal(d_w, with_ones[1])


def test_routed_combine_without_weights(g):
    from sorting_lsd_radix_gb300 import routed
    gen = _gen(4)
    x = _normal(gen, 40, 24).requires_grad_()
    ids = torch.randint(-1, 5, (40, 2), generator=gen, device="cuda")
    rows, slot_of_row, row_of_slot, _, _ = routed.expert_dispatch(x, ids, 5)
    routed.expert_combine(rows, None, slot_of_row, row_of_slot).sum().backward()
    kept = (ids >= 0).sum(1).float()
    assert torch.equal(x.grad, kept[:, None].expand(40, 24))


# rows whose blocks of columns, 32 packs each, are more than a grid has places for in its second direction
@pytest.mark.parametrize("dtype,row_len", [(torch.float32, 1 << 23), (torch.bfloat16, (1 << 21) + 1), (torch.bfloat16, 40)])
@pytest.mark.parametrize("vocab", [2, 131])
def test_whole_gradient_of_no_ids(g, dtype, row_len, vocab):
    """Every row is zeroed, however long the rows, and nothing beside them."""
    room = torch.ones(vocab + 1, row_len, dtype=dtype, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    d_out = torch.empty(0, row_len, dtype=dtype, device="cuda")
    _, temp = g.gbs_embedding_grad(d_out, ids, room[:vocab], return_temp=True)
    assert not torch.any(room[:vocab]) and torch.all(room[vocab] == 1)
    assert g.gbs_get_status(temp) == g.GBS_OK
    room.fill_(1)
    g.gbs_embedding_grad(d_out, ids, room[:vocab], accumulate=True, temp=temp)
    assert torch.all(room == 1)


def test_the_longest_rows(g):
    """Rows of 2^23 values through every operator."""
    gen, row_len = _gen(5), 1 << 23
    x = _normal(gen, 3, row_len)
    ids = torch.tensor([2, 0, 5], device="cuda")
    assert torch.equal(g.gbs_embedding_lookup(x, ids[:2]), x[ids[:2]])
    grad = torch.ones(3, row_len, device="cuda")
    g.gbs_embedding_grad(x, ids, grad)
    assert torch.equal(grad, torch.stack([x[1], torch.zeros_like(x[0]), x[0]]))
    rows, plan = g.gbs_expert_dispatch(x, ids.view(3, 1), 4, row_align=2)
    assert torch.equal(rows[plan[1][:2, 0].long()], x[:2]) and int((plan[0] < 0).sum()) == rows.size(0) - 2
    assert torch.equal(g.gbs_expert_combine(rows, plan[1])[:2], x[:2])
    assert torch.equal(g.gbs_expert_combine_grad(x, rows, plan[0], plan[1], None)[0], rows)


@pytest.mark.parametrize("dtype,row_len", [(torch.float32, 512), (torch.bfloat16, 2560)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_grad_reports_a_row_that_does_not_come(g, dtype, row_len, accumulate):
    """A row of one chunk that is never copied: the bounded waits end, the status says so, nothing of a row that has not
    come is stored, the other chunks are right, and so is the next call."""
    gen, n, vocab, chunk, held = _gen(6, row_len), 5000, 6000, 8, 3  # chunk: what lists of this length are cut into
    ids = torch.randperm(n, generator=gen, device="cuda")  # each id once: chunk c holds the ids chunk * c ..
    d_out, grad = _normal(gen, n, row_len, dtype=dtype), _normal(gen, vocab, row_len)
    kept = grad.clone()
    want, temp = g.gbs_embedding_grad(d_out, ids, grad.clone(), accumulate=accumulate, return_temp=True)
    assert g.gbs_get_status(temp) == g.GBS_OK
    g.gbs_debug_set_ring_fault(held, 1 << 12)
    try:
        g.gbs_embedding_grad(d_out, ids, grad, accumulate=accumulate, temp=temp)
        assert g.gbs_get_status(temp) == g.GBS_ERR_TIMEOUT
    finally:
        g.gbs_debug_set_ring_fault(-1, 0)
    first = chunk * held  # its first row came and was stored; the second did not
    assert torch.equal(grad[:first + 1], want[:first + 1]) and torch.equal(grad[first + chunk:], want[first + chunk:])
    assert torch.equal(grad[first + 1:first + chunk], kept[first + 1:first + chunk])
    again = g.gbs_embedding_grad(d_out, ids, kept, accumulate=accumulate, temp=temp)
    assert g.gbs_get_status(temp) == g.GBS_OK
    assert torch.equal(again, want)


def test_work_buffers_that_are_not_whole(g):
    """Strided, expanded and host tensors are refused, by the sorts as by the row operators; an empty one is replaced."""
    ids = torch.randint(0, 4, (600, 2), generator=_gen(7), device="cuda")
    plan, temp = g.gbs_expert_sort(ids, 4, return_temp=True)
    n = 4 * temp.numel() + 4096
    room = torch.empty(2 * n, dtype=torch.uint8, device="cuda")
    keys = ids.view(-1).int()
    for bad in (room[::2], room[:1].expand(n), torch.empty(n, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="temp"):
            g.gbs_expert_sort(ids, 4, plan_out=plan, temp=bad)
        with pytest.raises(ValueError, match="temp"):
            g.gbs_expert_sort(ids, 4, temp=bad)
        with pytest.raises(ValueError, match="temp"):
            g.gbs_sort_keys(keys, temp=bad)
    nothing = room[:0]
    out, made = g.gbs_sort_keys(keys, torch.full_like(keys, -1), temp=nothing, return_temp=True)
    assert torch.equal(out, keys.sort()[0]) and made.numel() > 0
    assert torch.equal(g.gbs_expert_sort(ids, 4, plan_out=tuple(torch.empty_like(t) for t in plan), temp=nothing)[1], plan[1])


def chunk_of(n, row_len):
    """Sorted positions of a chunk, as the gradient cuts lists above the short ones."""
    chunk = 32 if row_len < 256 else 64
    while chunk > 8 and n // chunk * -(-row_len // 1024) < 152 * 16:
        chunk //= 2
    return chunk


def ids_with_runs(runs, n, seed):
    """(ids, keys): n ids in any order whose sorted order has the runs [(length, key)], then single ones; keys skip
    every third number, so that some rows have no id."""
    length = [c for c in runs]
    length += [1] * (n - sum(length))
    key = torch.arange(len(length)) * 3 // 2
    ids = torch.repeat_interleave(key, torch.tensor(length))
    assert ids.numel() == n
    return ids[torch.randperm(n, generator=torch.Generator().manual_seed(seed))].cuda(), int(key[-1]) + 2


def border_runs(chunk):
    """Runs that begin `before` positions before a border of two chunks and end `after` positions behind it."""
    runs, at = [], 0
    for before in (0, 1, 2, chunk // 2, chunk - 1, chunk, chunk + 1):
        for after in (0, 1, 2, chunk - 1, chunk, chunk + 1, 2 * chunk - 1, 2 * chunk, 2 * chunk + 1, 40 * chunk):
            if before + after == 0:
                continue
            single = (-at - before) % chunk
            runs += [1] * single + [before + after]
            at += single + before + after
    return runs


def check_grad(g, d_out, ids, vocab, grad_type, accumulate, seed):
    """The gradient against sums in 64 bits, made on the GPU."""
    grad = _normal(_gen(seed), vocab, d_out.size(1), dtype=grad_type)
    want = grad.double() if accumulate else torch.zeros(vocab, d_out.size(1), dtype=torch.float64, device="cuda")
    size = want.abs()
    want.index_add_(0, ids, d_out.double())
    size.index_add_(0, ids, d_out.double().abs())
    terms = torch.bincount(ids, minlength=vocab)[:, None] + 1
    _, temp = g.gbs_embedding_grad(d_out, ids, grad, accumulate=accumulate, return_temp=True)
    assert g.gbs_get_status(temp) == g.GBS_OK
    rel, least = UNIT[grad_type]
    # 64-bit sums in any order are exact beside this
    bound = (terms + 2) * EPS32 * size * (1 + rel) + rel * want.abs() + least
    off = (grad.double() - want).abs()
    assert bool((off <= bound).all()), f"off by {float((off - bound).max())} more than the bound"
    if not accumulate:
        unnamed = torch.bincount(ids, minlength=vocab) == 0
        assert bool(unnamed.any()) and not torch.any(grad[unnamed])
    return grad


# the ring (one and two slices of columns), short rows, odd ones by twos and by single values
ROWS = [(torch.float32, 256), (torch.bfloat16, 2304), (torch.float32, 24), (torch.bfloat16, 40), (torch.bfloat16, 258),
        (torch.float32, 33)]


@pytest.mark.parametrize("dtype,row_len,chunk", [(*r, c) for r in ROWS for c in (8, 16, 32, 64) if c <= 32 or r[1] >= 256])
def test_embedding_grad_runs_around_borders(g, dtype, row_len, chunk):
    """Runs that begin and end on both sides of the borders between chunks, for every length of chunk: those that end
    within a chunk's length behind a border belong to the chunk before it, longer ones are cut and joined."""
    runs = border_runs(chunk)
    n = max(sum(runs) + 1025, 152 * 16 * chunk // -(-row_len // 1024) + chunk if chunk > 8 else 0)
    assert chunk_of(n, row_len) == chunk and n > 1024
    ids, vocab = ids_with_runs(runs, n, row_len)
    d_out = _normal(_gen(8, n, row_len), n, row_len, dtype=dtype)
    for accumulate in (False, True):
        check_grad(g, d_out, ids, vocab, torch.float32, accumulate, 9)
    # runs of any length one behind another
    gen = torch.Generator().manual_seed(chunk)
    runs, left = [], n - 1
    while left > 0:
        runs.append(min(left, int(torch.randint(1, 4 * chunk, (1,), generator=gen))))
        left -= runs[-1]
    ids, vocab = ids_with_runs(runs, n, row_len)
    for accumulate in (False, True):
        check_grad(g, d_out, ids, vocab, dtype, accumulate, 10)


@pytest.mark.parametrize("row_len", [1024, 1029])
def test_long_dispatch_of_a_shard_with_empty_rows(g, row_len):
    """Rows that move in a launch of their own (512 MB and more), some of them without a slot."""
    gen = _gen(11, row_len)
    tokens, top_k, experts, first = 150_000, 2, 60, 7
    ids = torch.randint(0, first + experts + 5, (tokens, top_k), generator=gen, device="cuda", dtype=torch.int32)
    x = _normal(gen, tokens, row_len, dtype=torch.bfloat16)
    rows, plan = g.gbs_expert_dispatch(x, ids, experts, first_expert=first, row_align=128)
    assert rows.numel() * 2 >= 512 << 20
    check_plan(plan, plan_by_hand(ids, experts, first, 128))
    slot = plan[0].long()
    assert int((slot < 0).sum()) > 30_000
    want = torch.where((slot >= 0)[:, None], x[slot.clamp(min=0) // top_k], torch.zeros((), dtype=x.dtype, device="cuda"))
    assert torch.equal(rows, want)


@pytest.mark.parametrize("padding", [None, -1, -100])
def test_no_padding(g, padding):
    """A negative padding_id is none: it does not count from the table's end."""
    gen = _gen(12)
    ids, d_out = torch.randint(-3, 9, (500,), generator=gen, device="cuda"), _normal(gen, 500, 8)
    want, magnitude, terms = grad_by_hand(d_out, ids, torch.empty(9, 8), 1.0, 0, False)
    _close(g.gbs_embedding_grad(d_out, ids, torch.empty(9, 8, device="cuda"), padding_id=padding), want, magnitude, terms + 1)
