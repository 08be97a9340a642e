"""The autograd functions of routed.py on the CPU, with the library's calls replaced by plain torch operations."""
import pytest

torch = pytest.importorskip("torch")
from sorting_lsd_radix_gb300 import routed  # noqa: E402


class Plain:
    """The entry points that routed.py calls, in plain torch operations.  They work on detached tensors, as calls of a
    compiled library do: autograd sees nothing of what happens in them."""

    @staticmethod
    @torch.no_grad()
    def gbs_expert_dispatch(x, expert_ids, num_experts, first_expert=0, row_align=1):
        key = expert_ids.reshape(-1) - first_expert
        inside = (key >= 0) & (key < num_experts)
        by, order = torch.sort(torch.where(inside, key, num_experts), stable=True)
        counts = torch.bincount(by, minlength=num_experts + 1)[:num_experts]
        offsets = torch.zeros(num_experts + 1, dtype=torch.int64)
        offsets[1:] = torch.cumsum((counts + row_align - 1) // row_align * row_align, 0)
        slot_of_row = torch.full((key.numel() + num_experts * (row_align - 1),), -1)
        row_of_slot = torch.full((key.numel(),), -1)
        at = 0
        for e, c in enumerate(counts.tolist()):
            mine = order[at:at + c]
            row_of_slot[mine] = torch.arange(c) + offsets[e]
            slot_of_row[offsets[e]:offsets[e] + c] = mine
            at += c
        rows = x[slot_of_row.clamp(min=0) // expert_ids.size(1)] * (slot_of_row >= 0)[:, None]
        return rows, (slot_of_row.int(), row_of_slot.view(expert_ids.shape).int(), offsets.int(), counts.int())

    @staticmethod
    def _picked(rows, row_of_slot):
        return rows[row_of_slot.clamp(min=0).long()] * (row_of_slot >= 0)[..., None]

    @staticmethod
    @torch.no_grad()
    def gbs_expert_combine(rows, row_of_slot, weights=None):
        picked = Plain._picked(rows, row_of_slot)
        return (picked if weights is None else picked * weights[..., None]).sum(1)

    @staticmethod
    @torch.no_grad()
    def gbs_expert_combine_grad(d_out, rows, slot_of_row, row_of_slot, weights):
        slot = slot_of_row.clamp(min=0).long()
        d_rows = d_out[slot // row_of_slot.size(1)] * (slot_of_row >= 0)[:, None]
        if weights is None:
            return d_rows, None
        d_weights = (Plain._picked(rows, row_of_slot) * d_out[:, None, :]).sum(2)
        return d_rows * weights.reshape(-1)[slot][:, None], d_weights

    @staticmethod
    @torch.no_grad()
    def gbs_embedding_lookup(table, ids, scale=1.0, first_id=0):
        return table[ids - first_id] * scale

    @staticmethod
    @torch.no_grad()
    def gbs_embedding_grad(d_out, ids, grad, scale=1.0, first_id=0, padding_id=None, accumulate=False):
        return grad.zero_().index_add_(0, ids - first_id, d_out * scale)


@pytest.fixture
def plain(monkeypatch):
    monkeypatch.setattr(routed, "gbsort", Plain)


def _problem():
    gen = torch.Generator().manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64).requires_grad_()

    experts = torch.topk(torch.rand(12, 6, generator=gen), 2, dim=1)[1]
    return normal(12, 5), experts, torch.rand(12, 2, generator=gen, dtype=torch.float64).requires_grad_(), normal(9, 5), \
        torch.randint(0, 9, (12,), generator=gen)


def test_first_derivatives(plain):
    x, experts, weights, table, ids = _problem()

    def out(x, weights):
        rows, slot_of_row, row_of_slot, _, _ = routed.expert_dispatch(x, experts, 5, row_align=4)
        return routed.expert_combine(rows, weights, slot_of_row, row_of_slot)

    assert torch.autograd.gradcheck(out, (x, weights))
    assert torch.autograd.gradcheck(lambda t: routed.embedding(t, ids, 2.0), (table,))


@pytest.mark.parametrize("which", ["dispatch", "combine", "embedding"])
def test_second_derivatives_are_refused(plain, which):
    """A gradient made of the library's calls has no derivative of its own: asking for it is an error, where a part
    of the answer would else be left out without a word."""
    x, experts, weights, table, ids = _problem()
    rows, slot_of_row, row_of_slot, _, _ = routed.expert_dispatch(x, experts, 5)
    if which == "dispatch":
        of, loss = x, (rows ** 2).sum()
    elif which == "combine":
        of, loss = weights, (routed.expert_combine(rows.detach(), weights, slot_of_row, row_of_slot) ** 2).sum()
    else:
        of, loss = table, (routed.embedding(table, ids) ** 2).sum()
    first, = torch.autograd.grad(loss, of, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((first ** 2).sum() + (of ** 2).sum()).backward()


def test_a_plan_edited_before_the_backward_pass_is_noticed(plain):
    """The dispatch keeps its order as autograd keeps tensors: an edit in place is an error, not another gradient."""
    x, experts, _, _, _ = _problem()
    rows, _, row_of_slot, _, _ = routed.expert_dispatch(x, experts, 5)
    row_of_slot[0] = -1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        rows.sum().backward()


def test_saved_tensor_hooks_see_the_plan(plain):
    x, experts, _, _, _ = _problem()
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        _, _, row_of_slot, _, _ = routed.expert_dispatch(x, experts, 5)
    assert any(t.shape == row_of_slot.shape and torch.equal(t, row_of_slot) for t in kept)


def test_combine_without_weights(plain):
    x, experts, _, _, _ = _problem()

    def out(x):
        rows, slot_of_row, row_of_slot, _, _ = routed.expert_dispatch(x, experts, 5, row_align=4)
        return routed.expert_combine(rows, None, slot_of_row, row_of_slot)

    assert torch.autograd.gradcheck(out, (x,))
