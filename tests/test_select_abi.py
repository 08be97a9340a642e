"""Host-side checks of the operators that select, that need no GPU: refusals come back before anything is launched, so
the addresses here are never followed."""
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
