"""Row operators on the GPU at the ends of their ranges."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_rows import _close, _gen, _normal, check_plan, g, grad_by_hand, plan_by_hand  # noqa: E402,F401

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
