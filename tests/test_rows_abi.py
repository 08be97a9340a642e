"""Host-side checks of the row operators' C ABI and binding that need no GPU: refusals and work-buffer sizes
come back before anything is launched, so the addresses here are never followed."""
import ctypes

import pytest

from sorting_lsd_radix_gb300 import build as gbuild
from sorting_lsd_radix_gb300 import gbsort

torch = pytest.importorskip("torch")
A = 1 << 40  # an address
ROOM = 1 << 30


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gbsort.load()


def _temp(call, args, room=None, temp=A):
    size = ctypes.c_size_t(room if room is not None else 0)
    st = call(None if room is None else temp, ctypes.byref(size), *args)
    return st, size.value


def _sort(**kw):
    a = dict(kind=gbsort.GBS_I64, ids=A, tokens=100, top_k=4, experts=16, first=0, align=1, rows=400, slot=A, row=A,
             offsets=A, counts=A, stream=None)
    a.update(kw)
    return tuple(a.values())


def _dispatch(**kw):
    a = dict(type=gbsort.GBS_ROW_BF16, x=A, x_stride=64, row_len=64, kind=gbsort.GBS_I32, ids=A, tokens=100, top_k=4,
             experts=16, first=0, align=1, rows=400, out=A, out_stride=64, slot=A, row=A, offsets=A, counts=A,
             stream=None)
    a.update(kw)
    return tuple(a.values())


def _gather(**kw):
    a = dict(type=gbsort.GBS_ROW_F16, x=A, x_stride=64, tokens=100, top_k=4, row_len=64, slot=A, row=A, rows=400, out=A,
             out_stride=64, stream=None)
    a.update(kw)
    return tuple(a.values())


def _combine(**kw):
    a = dict(type=gbsort.GBS_ROW_F16, rows=A, stride=64, count=400, row=A, weight_type=gbsort.GBS_ROW_F32, weights=A,
             tokens=100, top_k=4, row_len=64, out=A, out_stride=64, stream=None)
    a.update(kw)
    return tuple(a.values())


def _combine_grad(**kw):
    a = dict(type=gbsort.GBS_ROW_F16, d_out=A, d_stride=64, rows=A, stride=64, count=400, slot=A, row=A,
             weight_type=gbsort.GBS_ROW_F32, weights=A, tokens=100, top_k=4, row_len=64, out=A, out_stride=64, d_w=A,
             stream=None)
    a.update(kw)
    return tuple(a.values())


def _lookup(**kw):
    a = dict(type=gbsort.GBS_ROW_F32, table=A, stride=64, vocab=1000, kind=gbsort.GBS_I32, ids=A, n=50, first=0,
             scale=1.0, row_len=64, out=A, out_stride=64, stream=None)
    a.update(kw)
    return tuple(a.values())


def _grad(**kw):
    a = dict(type=gbsort.GBS_ROW_BF16, d_out=A, d_stride=64, kind=gbsort.GBS_I32, ids=A, n=50, first=0, padding=-1,
             scale=1.0, vocab=1000, row_len=64, grad_type=gbsort.GBS_ROW_F32, grad=A, grad_stride=64, add=0, stream=None)
    a.update(kw)
    return tuple(a.values())


INVALID, UNSUPPORTED = gbsort.GBS_ERR_INVALID_ARG, gbsort.GBS_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad,want", [
    (dict(kind=gbsort.GBS_U32), INVALID), (dict(kind=9), INVALID), (dict(top_k=0), INVALID),
    (dict(experts=0), INVALID), (dict(align=0), INVALID), (dict(rows=399), INVALID),
    (dict(align=8, rows=511), INVALID),  # 400 slots of 16 experts in eights: up to 512 rows
    (dict(ids=None), INVALID), (dict(slot=None), INVALID), (dict(row=None), INVALID), (dict(offsets=None), INVALID),
    (dict(counts=None), INVALID), (dict(ids=A + 4), INVALID), (dict(slot=A + 2), INVALID), (dict(row=A + 1), INVALID),
    (dict(offsets=A + 3), INVALID), (dict(counts=A + 2), INVALID),
    (dict(top_k=257, rows=25700), UNSUPPORTED), (dict(experts=1025), UNSUPPORTED),
    (dict(tokens=1 << 29, rows=(1 << 31) - 1), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(tokens=(1 << 64) // 4 + 1), UNSUPPORTED), (dict(align=(1 << 24) + 1), UNSUPPORTED),
    (dict(experts=1024, align=1 << 24, rows=(1 << 31) - 1), UNSUPPORTED)])  # more rows than 2^31 - 1
def test_sort_refuses(lib, bad, want):
    assert _temp(lib.gbs_expert_sort, _sort(**bad), ROOM)[0] == want


@pytest.mark.parametrize("bad,want", [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(x=A + 1), INVALID), (dict(out=A + 1), INVALID), (dict(out_stride=63), INVALID), (dict(out_stride=0), INVALID),
    (dict(row_len=(1 << 24) + 1, out_stride=1 << 25), UNSUPPORTED), (dict(x_stride=1 << 60), UNSUPPORTED),
    (dict(out_stride=1 << 60), UNSUPPORTED), (dict(rows=399), INVALID), (dict(kind=gbsort.GBS_F32), INVALID)])
def test_dispatch_refuses(lib, bad, want):
    assert _temp(lib.gbs_expert_dispatch, _dispatch(**bad), ROOM)[0] == want


@pytest.mark.parametrize("bad,want", [
    (dict(type=5), INVALID), (dict(top_k=0), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(slot=None), INVALID), (dict(row=None), INVALID), (dict(slot=A + 2), INVALID), (dict(out_stride=10), INVALID),
    (dict(top_k=300), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(tokens=1 << 30), UNSUPPORTED)])
def test_gather_refuses(lib, bad, want):
    assert lib.gbs_expert_gather(*_gather(**bad)) == want


@pytest.mark.parametrize("bad,want", [
    (dict(type=5), INVALID), (dict(weight_type=gbsort.GBS_ROW_BF16), INVALID), (dict(weight_type=7), INVALID),
    (dict(rows=None), INVALID), (dict(out=None), INVALID), (dict(row=None), INVALID), (dict(weights=A + 2), INVALID),
    (dict(rows=A + 1), INVALID), (dict(out_stride=1), INVALID), (dict(top_k=0), INVALID),
    (dict(row_len=1 << 25, out_stride=1 << 25), UNSUPPORTED)])
def test_combine_refuses(lib, bad, want):
    assert lib.gbs_expert_combine(*_combine(**bad)) == want


@pytest.mark.parametrize("bad,want", [
    (dict(type=5), INVALID), (dict(weight_type=gbsort.GBS_ROW_BF16), INVALID), (dict(d_out=None), INVALID),
    (dict(rows=None), INVALID), (dict(out=None), INVALID), (dict(slot=None), INVALID), (dict(row=None), INVALID),
    (dict(d_w=A + 2), INVALID), (dict(out_stride=3), INVALID), (dict(count=1 << 31), UNSUPPORTED)])
def test_combine_grad_refuses(lib, bad, want):
    assert lib.gbs_expert_combine_grad(*_combine_grad(**bad)) == want


@pytest.mark.parametrize("bad,want", [
    (dict(type=5), INVALID), (dict(kind=gbsort.GBS_U64), INVALID), (dict(table=None), INVALID), (dict(ids=None), INVALID),
    (dict(out=None), INVALID), (dict(table=A + 2), INVALID), (dict(ids=A + 2), INVALID), (dict(out_stride=63), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(vocab=(1 << 31) - 1), UNSUPPORTED), (dict(stride=1 << 60), UNSUPPORTED)])
def test_lookup_refuses(lib, bad, want):
    assert lib.gbs_embedding_lookup(*_lookup(**bad)) == want


@pytest.mark.parametrize("bad,want", [
    (dict(type=5), INVALID), (dict(kind=gbsort.GBS_U64), INVALID), (dict(grad_type=gbsort.GBS_ROW_F16), INVALID),
    (dict(grad_type=4), INVALID), (dict(d_out=None), INVALID), (dict(ids=None), INVALID), (dict(grad=None), INVALID),
    (dict(d_out=A + 1), INVALID), (dict(grad=A + 2), INVALID), (dict(ids=A + 1), INVALID), (dict(grad_stride=8), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(vocab=(1 << 31) - 1), UNSUPPORTED),
    (dict(row_len=1 << 25, grad_stride=1 << 25), UNSUPPORTED)])
def test_embedding_grad_refuses(lib, bad, want):
    assert _temp(lib.gbs_embedding_grad, _grad(**bad), 1 << 40)[0] == want


def test_work_buffers(lib):
    for call, args in ((lib.gbs_expert_sort, _sort), (lib.gbs_expert_dispatch, _dispatch), (lib.gbs_embedding_grad, _grad)):
        st, need = _temp(call, args())
        assert st == gbsort.GBS_OK and need >= 256
        assert _temp(call, args(), need - 1)[0] == gbsort.GBS_ERR_TEMP_TOO_SMALL
        assert _temp(call, args(), ROOM, temp=A + 16)[0] == INVALID
        assert call(A, None, *args()) == INVALID
    # the size of a query does not need the arrays
    nothing = dict(ids=None, slot=None, row=None, offsets=None, counts=None)
    assert _temp(lib.gbs_expert_sort, _sort(**nothing)) == _temp(lib.gbs_expert_sort, _sort())
    assert _temp(lib.gbs_expert_dispatch, _dispatch(x=None, out=None, **nothing)) == \
        _temp(lib.gbs_expert_dispatch, _dispatch())
    # counts of long calls grow with their tiles, not with slots times experts
    st, need = _temp(lib.gbs_expert_sort, _sort(tokens=1 << 28, experts=1024, rows=1 << 30))
    assert st == gbsort.GBS_OK and need < (1 << 30) * 2
    # a long id list: the sort's buffers and a fraction of the rows
    st, need = _temp(lib.gbs_embedding_grad, _grad(n=1 << 20, row_len=4096, grad_stride=4096))
    assert st == gbsort.GBS_OK and need < (1 << 20) * 4096 * 2 // 3


def test_num_rows():
    rows = gbsort.gbs_expert_num_rows
    assert rows(0, 8, 128) == 0 and rows(100, 8) == 100 and rows(100, 8, 1) == 100
    assert rows(3, 8, 16) == 48                      # three experts in use
    assert rows(100, 8, 16) == (100 + 8 * 15) // 16 * 16
    for slots in range(1, 40):                       # no split of the slots needs more
        for experts in (1, 2, 5):
            for align in (2, 3, 8):
                worst = max(sum(-(-c // align) * align for c in split) for split in _splits(slots, experts))
                assert worst <= rows(slots, experts, align)


def _splits(slots, experts):
    """Ways to deal slots that leave the most rows without one: all but one expert get 1 more than a multiple."""
    for small in range(min(experts, slots)):
        rest = slots - small
        yield [1] * small + [rest] + [0] * (experts - small - 1)


def test_binding_checks_its_arguments(lib):
    x, ids = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int64)
    plan = (torch.zeros(12, dtype=torch.int32), torch.zeros(6, 2, dtype=torch.int32))
    w, words = torch.zeros(6, 2), torch.zeros(6, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_expert_dispatch(x, ids, 4)
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_expert_combine(torch.zeros(12, 8), plan[1], w)
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_embedding_lookup(x, words)
    with pytest.raises(TypeError):  # ids are integers of 32 or 64 bits
        gbsort.gbs_expert_sort(ids.short(), 4)
    with pytest.raises(ValueError):
        gbsort.gbs_expert_sort(ids.view(-1), 4)
    with pytest.raises(ValueError):
        gbsort.gbs_expert_sort(ids, 0)
    with pytest.raises(ValueError):
        gbsort.gbs_expert_sort(ids, 4, row_align=0)
    with pytest.raises(ValueError):  # ids as they lie in memory
        gbsort.gbs_expert_sort(torch.zeros(6, 4, dtype=torch.int64)[:, ::2], 4)
    with pytest.raises(TypeError):
        gbsort.gbs_expert_dispatch(x.double(), ids, 4)
    with pytest.raises(ValueError):  # a row's values are neighbours
        gbsort.gbs_expert_dispatch(torch.zeros(6, 16)[:, ::2], ids, 4)
    with pytest.raises(ValueError):
        gbsort.gbs_expert_dispatch(x[:5], ids, 4)
    with pytest.raises(TypeError):
        gbsort.gbs_expert_dispatch(x, ids, 4, rows_out=torch.zeros(12, 8, dtype=torch.float16))
    with pytest.raises(TypeError):  # weights in 32 bits or the rows' type
        gbsort.gbs_expert_combine(torch.zeros(12, 8), plan[1], w.half())
    with pytest.raises(TypeError):
        gbsort.gbs_expert_combine(torch.zeros(12, 8), plan[1].long(), w)
    with pytest.raises(ValueError):
        gbsort.gbs_expert_combine_grad(x[:, :7], torch.zeros(12, 8), *plan, w)
    with pytest.raises(TypeError):
        gbsort.gbs_embedding_grad(x.half(), words, torch.zeros(9, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gbsort.gbs_embedding_grad(x, words, torch.zeros(9, 7))
    with pytest.raises(ValueError):
        gbsort.gbs_embedding_grad(x, words.view(2, 3), torch.zeros(9, 8))
    with pytest.raises(ValueError):
        gbsort.gbs_embedding_lookup(x, words, out=torch.zeros(5, 8))


def test_binding_without_weights_checks_its_arguments(lib):
    """No weights: no gradient of them either, and the other arguments' checks as with weights."""
    rows, d_out = torch.zeros(12, 8), torch.zeros(6, 8)
    plan = (torch.zeros(12, dtype=torch.int32), torch.zeros(6, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_expert_combine_grad(d_out, rows, *plan, None)
    with pytest.raises(ValueError, match="without weights"):
        gbsort.gbs_expert_combine_grad(d_out, rows, *plan, None, d_weights_out=torch.zeros(6, 2))
    with pytest.raises(ValueError):
        gbsort.gbs_expert_combine_grad(d_out[:, :7], rows, *plan, None)
    with pytest.raises(ValueError):
        gbsort.gbs_expert_combine_grad(d_out, rows, *plan, None, d_rows_out=rows[:11])


MAX_LEN = gbsort.GBS_MAX_ROW_LEN


def test_limits_one_past(lib):
    """The longest rows and alignments are taken, one more is not, and no order has more than 2^31 - 1 rows."""
    most = (1 << 31) - 1
    assert lib.gbs_expert_num_rows(400, 1024, MAX_LEN) > most
    assert _temp(lib.gbs_expert_sort, _sort(experts=1024, align=MAX_LEN, rows=most), ROOM)[0] == UNSUPPORTED
    assert _temp(lib.gbs_expert_sort, _sort(experts=1, align=MAX_LEN, rows=most))[0] == gbsort.GBS_OK
    assert _temp(lib.gbs_expert_sort, _sort(experts=1, align=MAX_LEN + 1, rows=most))[0] == UNSUPPORTED
    # the longest alignment whose worst case has 2^31 - 1 rows or fewer, and the next
    assert _temp(lib.gbs_expert_sort, _sort(experts=400, align=5368709, rows=most))[0] == gbsort.GBS_OK
    assert _temp(lib.gbs_expert_sort, _sort(experts=400, align=5368710, rows=most))[0] == UNSUPPORTED
    long = MAX_LEN + 1
    assert _temp(lib.gbs_expert_dispatch, _dispatch(row_len=MAX_LEN))[0] == gbsort.GBS_OK
    assert _temp(lib.gbs_embedding_grad, _grad(row_len=MAX_LEN))[0] == gbsort.GBS_OK
    assert _temp(lib.gbs_expert_dispatch, _dispatch(row_len=long, out_stride=long), ROOM)[0] == UNSUPPORTED
    assert lib.gbs_expert_gather(*_gather(row_len=long, out_stride=long)) == UNSUPPORTED
    assert lib.gbs_expert_combine(*_combine(row_len=long, out_stride=long)) == UNSUPPORTED
    assert lib.gbs_expert_combine_grad(*_combine_grad(row_len=long, out_stride=long)) == UNSUPPORTED
    assert lib.gbs_embedding_lookup(*_lookup(row_len=long, out_stride=long)) == UNSUPPORTED
    assert _temp(lib.gbs_embedding_grad, _grad(row_len=long, grad_stride=long), 1 << 40)[0] == UNSUPPORTED


def test_refusals_without_weights(lib):
    """Null weights and a null gradient of them take no checks away from the other arguments."""
    nothing = dict(weights=None, d_w=None, rows=None)
    for bad in (dict(d_out=None), dict(out=None), dict(slot=None), dict(row=None), dict(out_stride=3), dict(d_out=A + 1)):
        assert lib.gbs_expert_combine_grad(*_combine_grad(**{**nothing, **bad})) == INVALID
    # rows are read for the weights' gradient, with weights or without
    assert lib.gbs_expert_combine_grad(*_combine_grad(weights=None, rows=None)) == INVALID
    assert lib.gbs_expert_combine_grad(*_combine_grad(d_w=None, weight_type=gbsort.GBS_ROW_BF16)) == INVALID
    assert lib.gbs_expert_combine(*_combine(weights=None, rows=None)) == INVALID
