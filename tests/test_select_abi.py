"""Host-side checks of the operators that select, that need no GPU: refusals come back before anything is launched, so
the addresses here are never followed."""
import ctypes
import os
import re

import pytest

from sorting_lsd_radix_gb300 import build as gbuild
from sorting_lsd_radix_gb300 import gbsort

torch = pytest.importorskip("torch")
A = 1 << 40  # an address
INVALID, UNSUPPORTED = gbsort.GBS_ERR_INVALID_ARG, gbsort.GBS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gbsort.load()


def _route(**kw):
    a = dict(type=gbsort.GBS_ROW_BF16, logits=A, stride=64, tokens=100, experts=64, top_k=4, score=0, bias=A, groups=8,
             top_groups=4, group_top=2, renorm=1, scale=1.0, id_type=gbsort.GBS_I32, ids=A,
             weight_type=gbsort.GBS_ROW_F32, weights=A, stream=None)
    a.update(kw)
    return tuple(a.values())


def _route_grad(**kw):
    a = dict(type=gbsort.GBS_ROW_BF16, weight_type=gbsort.GBS_ROW_F32, d_weights=A, logits=A, stride=64, tokens=100,
             experts=64, top_k=4, id_type=gbsort.GBS_I64, ids=A, score=1, renorm=0, scale=1.0, out=A, out_stride=64,
             stream=None)
    a.update(kw)
    return tuple(a.values())


SHARED = [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(weight_type=gbsort.GBS_ROW_F16), INVALID),
    (dict(weight_type=7), INVALID), (dict(id_type=gbsort.GBS_U32), INVALID), (dict(score=2), INVALID),
    (dict(score=-1), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID), (dict(top_k=65), INVALID),
    (dict(logits=None), INVALID), (dict(logits=A + 1), INVALID), (dict(ids=None), INVALID), (dict(ids=A + 2), INVALID),
    (dict(experts=1025), UNSUPPORTED), (dict(top_k=257, experts=512), UNSUPPORTED), (dict(tokens=1 << 29), UNSUPPORTED),
    (dict(tokens=(1 << 64) - 1), UNSUPPORTED), (dict(stride=1 << 60), UNSUPPORTED)]


@pytest.mark.parametrize("bad,want", SHARED + [
    (dict(groups=0), INVALID), (dict(groups=3), INVALID), (dict(top_groups=0), INVALID), (dict(top_groups=9), INVALID),
    (dict(group_top=0), INVALID), (dict(group_top=3), INVALID), (dict(groups=64, top_groups=4), UNSUPPORTED),
    (dict(top_k=9, top_groups=1), INVALID), (dict(bias=A + 2), INVALID), (dict(weights=None), INVALID),
    (dict(weights=A + 2), INVALID)])
def test_route_refuses(lib, bad, want):
    assert lib.gbs_expert_route(*_route(**bad)) == want


@pytest.mark.parametrize("bad,want", SHARED + [
    (dict(d_weights=None), INVALID), (dict(d_weights=A + 1), INVALID), (dict(out=None), INVALID),
    (dict(out=A + 1), INVALID), (dict(out_stride=63), INVALID), (dict(out_stride=1 << 60), UNSUPPORTED)])
def test_route_grad_refuses(lib, bad, want):
    assert lib.gbs_expert_route_grad(*_route_grad(**bad)) == want


def test_no_tokens(lib):
    nothing = dict(tokens=0, logits=None, ids=None)
    assert lib.gbs_expert_route(*_route(weights=None, bias=None, **nothing)) == gbsort.GBS_OK
    assert lib.gbs_expert_route_grad(*_route_grad(d_weights=None, out=None, **nothing)) == gbsort.GBS_OK


def test_route_binding_checks_its_arguments(lib):
    logits, ids, w = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 2)
    route, grad = gbsort.gbs_expert_route, gbsort.gbs_expert_route_grad
    for call in (lambda: route(logits, 2), lambda: route(logits, 2, bias=torch.zeros(8), ids_out=ids, weights_out=w),
                 lambda: grad(w, logits, ids)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for bad in (dict(logits=logits.double(), top_k=2), dict(logits=logits, top_k=2, bias=torch.zeros(8).half()),
                dict(logits=logits, top_k=2, ids_out=ids.short()), dict(logits=logits, top_k=2, weights_out=w.half())):
        with pytest.raises(TypeError):
            route(**bad)
    for bad in (dict(logits=logits[0], top_k=2), dict(logits=torch.zeros(6, 16)[:, ::2], top_k=2),
                dict(logits=logits, top_k=0), dict(logits=logits, top_k=2 ** 64 + 2),
                dict(logits=logits, top_k=2, num_groups=-1), dict(logits=logits, top_k=2, bias=torch.zeros(9)),
                dict(logits=logits, top_k=2, bias=torch.zeros(16)[::2]), dict(logits=logits, top_k=3, ids_out=ids),
                dict(logits=logits, top_k=2, weights_out=torch.zeros(2, 6).t())):
        with pytest.raises(ValueError):
            route(**bad)
    for bad in ((w[:5], logits, ids), (w, logits, ids[:, :1]), (w, logits, ids.view(-1)), (w, logits, ids[:5]),
                (w, logits, ids, 0, False, 1.0, torch.zeros(6, 7)), (torch.zeros(6, 0), logits, ids[:, :0])):
        with pytest.raises(ValueError):
            grad(*bad)
    with pytest.raises(TypeError):
        grad(w.half(), logits, ids)
    with pytest.raises(TypeError):
        grad(w, logits, ids.short())


@pytest.mark.parametrize("bad", [dict(group_top=2 ** 64 + 1), dict(group_top=-2 ** 64 + 2), dict(score_type=2 ** 32),
                                 dict(score_type=2 ** 32 + 1), dict(score_type=-2 ** 32), dict(score_type=2 ** 64)])
def test_integers_that_would_wrap_are_refused(lib, bad):
    """Each would be a valid value's low bits, by ctypes or by the compiled calls' narrowing."""
    logits, ids, w = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 2)
    with pytest.raises(ValueError, match="signed integer"):
        gbsort.gbs_expert_route(logits, 2, **bad)
    with pytest.raises(ValueError, match="signed integer"):
        gbsort.gbs_expert_route(logits, 2, ids_out=ids, weights_out=w, **bad)
    if "score_type" in bad:
        with pytest.raises(ValueError, match="signed integer"):
            gbsort.gbs_expert_route_grad(w, logits, ids, d_logits_out=torch.zeros(6, 8), **bad)


def _select(**kw):
    a = dict(type=gbsort.GBS_ROW_BF16, logits=A, stride=1000, batch=3, beams=4, vocab=1000, scores=A, finished=None,
             end=2, count=8, scores_out=A, beams_out=A, tokens_out=A, stream=None)
    a.update(kw)
    return tuple(a.values())


def _sized(lib, args, room=1 << 30, temp=A):
    size = ctypes.c_size_t(room)
    return lib.gbs_beam_select(temp, ctypes.byref(size), *args), size.value


@pytest.mark.parametrize("bad,want", [
    (dict(type=3), INVALID), (dict(beams=0), INVALID), (dict(vocab=0), INVALID), (dict(count=0), INVALID),
    (dict(beams=33), UNSUPPORTED), (dict(count=65), UNSUPPORTED), (dict(vocab=1 << 31), UNSUPPORTED),
    (dict(batch=1 << 30), UNSUPPORTED), (dict(batch=1 << 62), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(logits=A + 1), INVALID), (dict(stride=1 << 62), UNSUPPORTED),
    (dict(scores=None), INVALID), (dict(scores=A + 2), INVALID), (dict(scores_out=None), INVALID),
    (dict(beams_out=None), INVALID), (dict(tokens_out=None), INVALID), (dict(scores_out=A + 1), INVALID),
    (dict(beams_out=A + 2), INVALID), (dict(tokens_out=A + 3), INVALID)])
def test_select_refuses(lib, bad, want):
    assert _sized(lib, _select(**bad))[0] == want


def test_select_work_buffer(lib):
    st, need = _sized(lib, _select(logits=None, scores=None, scores_out=None, beams_out=None, tokens_out=None), 0, None)
    assert st == gbsort.GBS_OK and need >= 256
    assert _sized(lib, _select(), need - 1)[0] == gbsort.GBS_ERR_TEMP_TOO_SMALL
    assert _sized(lib, _select(), temp=A + 16)[0] == INVALID
    assert lib.gbs_beam_select(A, None, *_select()) == INVALID
    # a list for each of a row's slices, not for each logit
    st, need = _sized(lib, _select(batch=64, beams=8, vocab=131072, stride=131072, count=16), 0, None)
    assert st == gbsort.GBS_OK and need < 64 * 8 * 131072 * 2 // 100
    # no beam at all needs a header
    assert _sized(lib, _select(batch=0, logits=None, scores=None, scores_out=None, beams_out=None, tokens_out=None), 0, None) == (gbsort.GBS_OK, 256)


def _reorder(**kw):
    a = dict(state=A, s=(1 << 20, 1 << 16, 1 << 12, 256), out=2 * A, t=(1 << 20, 1 << 16, 1 << 12, 256), outer=2, batch=3,
             beams=4, into=4, segments=5, bytes=256, parents=A, stream=None)
    a.update(kw)
    a["s"], a["t"] = (None if x is None else (ctypes.c_size_t * 4)(*x) for x in (a["s"], a["t"]))
    return tuple(a.values())


@pytest.mark.parametrize("bad,want", [
    (dict(s=None), INVALID), (dict(t=None), INVALID), (dict(beams=33), UNSUPPORTED), (dict(into=33), UNSUPPORTED),
    (dict(beams=0), INVALID), (dict(state=None), INVALID), (dict(out=None), INVALID), (dict(parents=None), INVALID),
    (dict(parents=A + 2), INVALID), (dict(bytes=1 << 31), UNSUPPORTED), (dict(segments=1 << 40), UNSUPPORTED),
    (dict(batch=1 << 31), UNSUPPORTED),
    # places that would be written twice
    (dict(bytes=257), INVALID), (dict(t=(1 << 20, 1 << 16, 0, 256)), INVALID), (dict(t=(1 << 20, 1 << 16, 1279, 256)), INVALID),
    (dict(t=(1 << 16, 1 << 16, 1 << 12, 256)), INVALID), (dict(t=(1 << 62, 1 << 16, 1 << 12, 256)), UNSUPPORTED),
    (dict(s=(1 << 62, 1 << 16, 1 << 12, 256)), UNSUPPORTED),
    # in place: the same strides, and no beam that is not there
    (dict(out=A, t=(1 << 20, 1 << 16, 1 << 13, 256)), INVALID), (dict(out=A, into=5), INVALID)])
def test_reorder_refuses(lib, bad, want):
    assert lib.gbs_beam_reorder(*_reorder(**bad)) == want


@pytest.mark.parametrize("beams,into,s", [
    (4, 2, (1 << 20, 1 << 13, 1 << 12, 256)),  # a batch's beams 2 and 3 are the next one's 0 and 1
    (4, 1, (1 << 20, 1 << 12, 1 << 12, 256)), (4, 1, (1 << 20, 1 << 16, 1280 - 1, 256)),
    (4, 1, (1 << 20, 1 << 16, 0, 256)), (2, 1, (1 << 20, 1 << 16, 1 << 20, 256))])
def test_reorder_in_place_refuses_beams_that_overlap(lib, beams, into, s):
    """Read as one batch's, written as another's in the same launch."""
    assert lib.gbs_beam_reorder(*_reorder(out=A, beams=beams, into=into, s=s, t=s)) == INVALID


def test_nothing_to_reorder(lib):
    for none in (dict(outer=0), dict(batch=0), dict(into=0), dict(segments=0), dict(bytes=0)):
        assert lib.gbs_beam_reorder(*_reorder(state=None, out=None, parents=None, **none)) == gbsort.GBS_OK


def test_beam_binding_checks_its_arguments(lib):
    logits, scores = torch.zeros(6, 100), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_beam_select(logits, scores)
    for bad in (dict(scores=scores.double()), dict(finished=scores), dict(logits=logits.double())):
        with pytest.raises(TypeError):
            gbsort.gbs_beam_select(**{**dict(logits=logits, scores=scores), **bad})
    for bad in (dict(scores=scores[0]), dict(logits=logits[:4]), dict(num_out=0), dict(end_id=1 << 31),
                dict(finished=torch.zeros(3, 3, dtype=torch.bool)), dict(scores=torch.zeros(3, 2).t()),
                dict(logits=torch.zeros(6, 200)[:, ::2]), dict(num_out=2, out=(torch.zeros(2, 3),) * 3)):
        with pytest.raises(ValueError):
            gbsort.gbs_beam_select(**{**dict(logits=logits, scores=scores), **bad})
    state, parents = torch.zeros(4, 2, 3, 5, 8), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_beam_reorder(state, parents, 1)
    with pytest.raises(TypeError):
        gbsort.gbs_beam_reorder(state, parents.long(), 1)
    with pytest.raises(TypeError):
        gbsort.gbs_beam_reorder(state, parents, 1, out=state.half())
    for bad in ((state, parents), (state, parents, 4), (state, parents, -1), (state, parents[:, :2], 1),
                (state, parents, 1, torch.zeros(4, 2, 2, 5, 8)), (state, parents[0], 1),
                (torch.zeros(3, 4, 2, 3, 5)[:, :2], parents, 2), (torch.zeros(4, 2, 3, 5, 8, 9)[..., :4, :6, :3], parents, 1)):
        with pytest.raises(ValueError):
            gbsort.gbs_beam_reorder(*bad)


def test_no_logit_of_a_finished_beam_is_loaded():
    """The rows of finished beams may have nothing behind them: by the source, since a load of them is seen in no
    result."""
    with open(os.path.join(gbuild.CSRC, "beam.cu")) as f:
        source = f.read()
    kernel = source[source.index("beam_slice_kernel(const SelectParams p) {"):]
    kernel = kernel[:kernel.index("\n}\n")]
    look = kernel.index("if (p.finished && p.finished[row]) return;")
    helpers = re.findall(r"auto (\w+) = \[&\][^\n]*\n.*?\n    \};\n", kernel, flags=re.S)
    before = re.sub(r"auto (\w+) = \[&\][^\n]*\n.*?\n    \};\n", "", kernel[:look], flags=re.S)
    assert {"load", "value_at"} <= set(helpers)
    assert not re.search(r"\b(load\w*|value_at|prefetch\w*)\(|logits\[", before)


@pytest.mark.parametrize("shape,dim", [((2, 0, 3, 4, 5), 2), ((0, 2, 3, 4, 5), 2), ((3, 4, 2, 0, 5), 0), ((3, 4, 0), 0), ((3, 4, 6, 0), 0),
                                       ((2, 3, 4, 0, 5, 7), 1)])
def test_an_empty_state_is_no_layout(lib, shape, dim):
    """It gets as far as the check of its device, also where its dimensions do not merge."""
    state = torch.zeros(*(n + 1 for n in shape))[tuple(slice(0, n) for n in shape)]
    with pytest.raises(ValueError, match="CUDA"):
        gbsort.gbs_beam_reorder(state, torch.zeros(shape[dim], shape[dim + 1], dtype=torch.int32), dim)
