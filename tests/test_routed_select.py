"""The router's autograd function and the model's beam search on the CPU, with the library's calls replaced by plain
torch operations; and on the GPU, the operators as a model runs them together."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")
from sorting_lsd_radix_gb300 import gbsort, routed  # noqa: E402


class Plain:
    """The entry points that the functions here call, in plain torch operations on detached tensors."""
    GBS_SCORE_SOFTMAX, GBS_SCORE_SIGMOID = 0, 1

    @staticmethod
    def _weights(logits, ids, score_type, renormalise, scale):
        score = torch.sigmoid(logits) if score_type else torch.softmax(logits, 1)
        w = torch.gather(score, 1, ids.long())
        return scale * (w / w.sum(1, keepdim=True) if renormalise else w)

    @staticmethod
    @torch.no_grad()
    def gbs_expert_route(logits, top_k, score_type=0, bias=None, num_groups=1, top_groups=1, group_top=1, renormalise=False,
                         scale=1.0):
        assert num_groups == top_groups == 1
        score = torch.sigmoid(logits) if score_type else torch.softmax(logits, 1)
        ids = torch.sort(score if bias is None else score + bias, dim=1, descending=True, stable=True)[1][:, :top_k].int()
        return ids, Plain._weights(logits, ids, score_type, renormalise, scale)

    @staticmethod
    def gbs_expert_route_grad(d_weights, logits, ids, score_type=0, renormalise=False, scale=1.0):
        with torch.enable_grad():
            l = logits.detach().clone().requires_grad_()
            w = Plain._weights(l, ids, score_type, renormalise, scale)
            return torch.autograd.grad(w, l, d_weights.detach())[0]

    @staticmethod
    @torch.no_grad()
    def gbs_beam_select(logits, scores, num_out=None, finished=None, end_id=0, temp=None, return_temp=False):
        batch, beams = scores.shape
        value = scores.view(-1, 1) + torch.log_softmax(logits.double(), 1)
        if finished is not None:
            once = torch.full_like(value, -math.inf)
            once[:, end_id] = scores.view(-1)
            value = torch.where(finished.view(-1, 1), once, value)
        got, at = torch.sort(value.view(batch, -1), dim=1, descending=True, stable=True)
        got, at = got[:, :num_out or beams], at[:, :num_out or beams]
        gone = torch.isneginf(got)
        return (got.float(), (at // logits.size(1)).int().masked_fill(gone, -1),
                (at % logits.size(1)).int().masked_fill(gone, -1)), temp

    @staticmethod
    @torch.no_grad()
    def gbs_beam_reorder(state, parents):
        old = state.clone()
        for b, of in enumerate(parents.tolist()):
            for j, i in enumerate(of):
                if i >= 0:
                    state[b, j] = old[b, i]
        return state


@pytest.fixture
def plain(monkeypatch):
    monkeypatch.setattr(routed, "gbsort", Plain)


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score_type", [0, 1])
def test_first_derivative(plain, score_type, renormalise):
    gen = torch.Generator().manual_seed(5)
    logits = torch.randn(7, 9, generator=gen, dtype=torch.float64).requires_grad_()
    bias = torch.randn(9, generator=gen, dtype=torch.float64)

    def weights(l):
        ids, w = routed.expert_route(l, 3, score_type, bias, renormalise=renormalise, scale=2.5)
        assert not ids.requires_grad
        return w

    assert torch.autograd.gradcheck(weights, (logits,))
    # a gradient that is expanded, as a sum sends it back
    got, = torch.autograd.grad(weights(logits).sum(), logits)
    want, = torch.autograd.grad((weights(logits) * 1.0).sum(), logits)
    assert torch.equal(got, want)


def test_second_derivative_is_refused(plain):
    logits = torch.randn(4, 6, dtype=torch.float64).requires_grad_()
    first, = torch.autograd.grad((routed.expert_route(logits, 2)[1] ** 2).sum(), logits, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((first ** 2).sum() + (logits ** 2).sum()).backward()


class PlainRows(Plain):
    """Plain, with the binding's own check of a matrix."""

    @staticmethod
    def gbs_expert_route(logits, top_k, *args):
        gbsort._matrix(logits, "logits", *logits.shape, logits.dtype)
        return Plain.gbs_expert_route(logits, top_k, *args)

    @staticmethod
    def gbs_expert_route_grad(d_weights, logits, ids, *args):
        gbsort._matrix(logits, "logits", *logits.shape, logits.dtype)
        assert d_weights.is_contiguous()
        return Plain.gbs_expert_route_grad(d_weights, logits, ids, *args)


def _layouts(logits):
    """The same values transposed, in every other column, and expanded."""
    wide = torch.zeros(logits.size(0), 2 * logits.size(1), dtype=logits.dtype, device=logits.device)
    wide[:, ::2] = logits
    return logits.t().contiguous().t(), wide[:, ::2], logits[:1].expand_as(logits), logits[:, :1].expand_as(logits)


def check_layouts(device):
    d_w = torch.arange(21.0, device=device).view(7, 3)
    for logits in _layouts(torch.randn(7, 9, generator=torch.Generator().manual_seed(8)).to(device)):
        got = []
        for x in (logits, logits.contiguous()):
            leaf = x.detach().requires_grad_()
            ids, w = routed.expert_route(leaf, 3, renormalise=True)
            got.append((ids, w.detach(), torch.autograd.grad(w, leaf, d_w)[0]))
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_logits_of_any_layout(monkeypatch):
    monkeypatch.setattr(routed, "gbsort", PlainRows)
    check_layouts("cpu")


class Table(torch.nn.Module):
    """A model whose next token depends on the last one: a table of logits, zeros behind no token."""
    search = routed.RoutedModel.search

    def __init__(self, logits):
        super().__init__()
        self.logits = logits

    def forward(self, ids):
        ids = ids.long()
        return torch.where((ids >= 0)[:, None], self.logits[ids.clamp(min=0)], 0.0)


def every_sequence(logits, first, steps, end_id):
    """All sequences with their scores, best first: a sequence that has ended goes on with end_id at no cost."""
    p = torch.log_softmax(logits.double().cpu(), 1)
    found = {}
    for tokens in itertools.product(range(p.size(0)), repeat=steps):
        score, last, ended = 0.0, first, False
        for t in tokens:
            if ended and t != end_id:
                break
            if not ended:
                score += float(p[last, t])
            last, ended = t, ended or t == end_id
        else:
            found[tokens] = score
    return sorted(found.items(), key=lambda f: -f[1])


def check_search(model, first, steps, beams, end_id=None):
    """With beams enough for every sequence of all but the last token the search is exhaustive."""
    tokens, scores = model.search(first, steps, beams, end_id)
    for b, start in enumerate(first.tolist()):
        want = every_sequence(model.logits, start, steps, end_id)
        score = dict(want)
        got = [tuple(t) for t in tokens[b].tolist()]
        assert len(set(got[:len(want)])) == min(beams, len(want))
        for k in range(beams):
            if k >= len(want):
                assert scores[b, k] == -math.inf and set(got[k]) == {-1}
                continue
            # each step's value is rounded once; sequences of the same steps in another order tie
            near = steps * 2.0 ** -24 * (abs(want[k][1]) + 120)
            assert abs(float(scores[b, k]) - want[k][1]) <= near and abs(score[got[k]] - want[k][1]) <= 2 * near


CASES = [(5, 3, 25, None), (5, 3, 25, 2), (3, 3, 27, None), (3, 3, 27, 0), (2, 5, 16, 1), (4, 1, 9, None), (3, 4, 32, 1)]


@pytest.mark.parametrize("vocab,steps,beams,end_id", CASES)
def test_search_finds_the_best(plain, vocab, steps, beams, end_id):
    gen = torch.Generator().manual_seed(vocab * steps)
    check_search(Table(3 * torch.randn(vocab, vocab, generator=gen)), torch.arange(min(3, vocab)), steps, beams, end_id)


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sorting_lsd_radix_gb300 import build as gbuild
    gbuild.build()
    gbsort.load()
    return gbsort


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,steps,beams,end_id", CASES)
def test_search_finds_the_best_on_the_gpu(g, vocab, steps, beams, end_id):
    gen = torch.Generator().manual_seed(vocab * steps)
    logits = (3 * torch.randn(vocab, vocab, generator=gen)).cuda()
    check_search(Table(logits), torch.arange(min(3, vocab), device="cuda"), steps, beams, end_id)


@pytest.mark.gpu
def test_a_routed_layer_and_its_gradients(g):
    """Route, dispatch, the experts, combine, and the way back, by groups with a bias and masked experts, against
    autograd through the same formulas in 64 bits.  Tokens without an expert get nothing."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    tokens, experts, hidden, top_k = 300, 32, 48, 3

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x, router, scales = normal(tokens, hidden).requires_grad_(), normal(experts, hidden).requires_grad_(), normal(experts, hidden)
    bias, mask = 0.1 * normal(experts), torch.zeros(tokens, experts, device="cuda")
    mask[torch.rand(tokens, experts, generator=gen, device="cuda") < 0.3] = -math.inf
    mask[5], mask[6, 1:], mask[6, 0] = -math.inf, -math.inf, 0.0
    args = dict(score_type=g.GBS_SCORE_SIGMOID, bias=bias, num_groups=4, top_groups=2, group_top=2, renormalise=True, scale=2.5)
    ids, weights = routed.expert_route(x @ router.t() / 7 + mask, top_k, **args)
    rows, slot_of_row, row_of_slot, offsets, counts = routed.expert_dispatch(x, ids, experts, row_align=8)
    owner = torch.repeat_interleave(torch.arange(experts, device="cuda"), torch.diff(offsets))
    padded = torch.zeros(rows.size(0), hidden, device="cuda")
    padded[:owner.numel()] = scales[owner]
    y = routed.expert_combine(rows * padded, weights, slot_of_row, row_of_slot)
    assert int(counts.sum()) == int((ids >= 0).sum()) and (ids[5] == -1).all() and (y[5] == 0).all()
    assert (ids[6] >= 0).sum() == 1
    d_y = normal(tokens, hidden)
    y.backward(d_y)

    x64, router64 = x.detach().double().requires_grad_(), router.detach().double().requires_grad_()
    here = ids >= 0
    s = torch.sigmoid(torch.gather(x64 @ router64.t() / 7, 1, ids.long().clamp(min=0))) * here
    w64 = 2.5 * s / s.sum(1, keepdim=True).clamp(min=1e-300)
    y64 = (w64[..., None] * (x64[:, None, :] * scales.double()[ids.long().clamp(min=0)])).sum(1)
    y64.backward(d_y.double())
    # products of 32 bits summed over 48 and 300 terms, behind scores of the order of one
    for got, want in ((y, y64), (x.grad, x64.grad), (router.grad, router64.grad)):
        size = want.abs().max()
        assert ((got.double() - want).abs() <= 2.0 ** -24 * 400 * size + 2.0 ** -20 * want.abs()).all()


@pytest.mark.gpu
def test_the_model_searches_as_it_predicts(g):
    """The best of the beams is as good as the greedy answer, and its score is the sum of the model's own predictions.
    Each of them is a logarithm of 32-bit logits: off by 2^-24 of the logits' size and of log(vocab)."""
    torch.manual_seed(3)
    model = routed.RoutedModel(vocab=400, hidden=64, inner=32, num_experts=8, top_k=2, dtype=torch.float32)
    first = torch.tensor([1, 7, 399], device="cuda")
    tokens, scores = model.search(first, steps=5, beams=6)
    one, greedy = model.search(first, steps=5, beams=1)
    assert (scores[:, :-1] >= scores[:, 1:]).all() and (scores[:, 0] >= greedy[:, 0] - 1e-4).all()
    with torch.no_grad():
        for t, s in ((tokens, scores), (one, greedy)):
            before = torch.cat([first[:, None, None].expand(3, t.size(1), 1).int(), t[:, :, :-1]], 2)
            logits = model(before.reshape(-1)).double()
            want = torch.gather(torch.log_softmax(logits, 1), 1, t.reshape(-1, 1).long()).view(t.shape).sum(2)
            size = logits.abs().max() + 10
            assert ((s.double() - want).abs() <= 2.0 ** -24 * 5 * (100 + 80 * size)).all()
    assert (one[:, 0, 0] == model(first.int()).argmax(1)).all()


@pytest.mark.gpu
def test_logits_of_any_layout_on_the_gpu(g):
    check_layouts("cuda")
