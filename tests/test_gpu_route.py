"""Routing to experts on the GPU against a plain implementation in 64 bits.

The choice is compared exactly.  A weight is a score, or a quotient of scores, of at most 32 experts a lane: its
error in units of 2^-24 is at most the sums' 37, the exponentials' and quotients' 4 each, the products' 2, and what an
exponent's rounding makes of it, its distance from the largest: 64 + top_k + 2 * distance covers them all, twice the
distance since numerator and sum have it.  The result's rounding adds half a unit of its type's last place.  The
gradient is a score times a difference of two terms: the same units of the terms' magnitudes, for two scores."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

EPS32 = 2.0 ** -24
UNIT = {torch.float32: (2.0 ** -24, 2.0 ** -126), torch.float16: (2.0 ** -11, 2.0 ** -25),
        torch.bfloat16: (2.0 ** -8, 2.0 ** -126)}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# the plain forms take infinities apart with where, after the fact
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:.*encountered in.*:RuntimeWarning")]


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


def _normal(gen, *shape, dtype=torch.float32, std=1.0):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _by(values, closed):
    """Indices along the last axis: open before closed ones, then by value, NaN above all, ties to the lowest."""
    nan = np.isnan(values)
    at = np.broadcast_to(np.arange(values.shape[-1]), values.shape)
    with np.errstate(invalid="ignore"):
        return np.lexsort((at, -np.where(nan, np.inf, values), ~nan, np.broadcast_to(closed, values.shape)), axis=-1)


def scores(l, kind, g):
    if kind == g.GBS_SCORE_SIGMOID:
        t = np.exp(-np.abs(l))
        return np.where(l >= 0, 1.0, t) / (1.0 + t)
    with np.errstate(invalid="ignore"):
        top = np.max(l, axis=1, keepdims=True, initial=-np.inf)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def ids_by_hand(g, l, top_k, kind, bias=None, groups=1, top_groups=1, group_top=1):
    tokens, experts = l.shape
    s, each = scores(l, kind, g), experts // groups
    dead = np.isneginf(l) | (np.isneginf(bias) if bias is not None else False)
    value = s + bias if bias is not None else l
    closed = dead
    if groups > 1:
        by = (value if bias is not None or group_top == 1 else s).reshape(tokens, groups, each)
        gone = dead.reshape(tokens, groups, each)
        order = _by(by, gone)[..., :group_top]
        best = np.where(np.take_along_axis(gone, order, 2), 0.0, np.take_along_axis(by, order, 2))
        worth = np.where(np.isnan(np.where(gone, 0.0, by)).any(2), np.nan, best.sum(2))
        none = gone.all(2)
        kept = np.zeros((tokens, groups), bool)
        np.put_along_axis(kept, _by(worth, none)[:, :top_groups], True, 1)
        closed = dead | ~np.repeat(kept & ~none, each, 1)
    order = _by(value, closed)[:, :top_k]
    return np.where(np.take_along_axis(closed, order, 1), -1, order)


def weights_by_hand(g, l, ids, kind, renorm, scale):
    """(weights, units of error) of the ids, those without an expert zero."""
    s = scores(l, kind, g)
    here = ids >= 0
    p = np.where(here, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    x = np.where(here, np.take_along_axis(l, np.maximum(ids, 0), 1), 0.0)
    if renorm:  # of scores divided by the largest chosen one's exponential, so that the sum does not vanish
        top = np.where(here, x, -np.inf).max(1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        if kind == g.GBS_SCORE_SIGMOID:
            top = np.minimum(top, 0.0)
            p = np.exp(np.minimum(x, 0.0) - top) / (1.0 + np.exp(-np.abs(x)))
        else:
            p = np.exp(x - top)
        p = np.where(here, p, 0.0)
        total = p.sum(1, keepdims=True)
        p = p / np.where(total == 0, 1.0, total)
    far = np.abs(x) if kind == g.GBS_SCORE_SIGMOID else np.where(here, np.max(l, 1, keepdims=True) - x, 0.0)
    return scale * p, 64 + ids.shape[1] + 2 * np.where(np.isfinite(far), far, 0.0)


def check(g, logits, top_k, kind, bias=None, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0, **out):
    ids, w = g.gbs_expert_route(logits, top_k, score_type=kind, bias=bias, num_groups=groups, top_groups=top_groups,
                                group_top=group_top, renormalise=renorm, scale=scale, **out)
    l, b = _f64(logits), None if bias is None else _f64(bias)
    want = ids_by_hand(g, l, top_k, kind, b, groups, top_groups, group_top)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want), f"token {np.flatnonzero((got != want).any(1))[:5]}"
    expect, units = weights_by_hand(g, l, want, kind, renorm, scale)
    rel, least = UNIT[w.dtype]
    bound = units * EPS32 * np.abs(expect) * (1 + rel) + rel * np.abs(expect) + least
    off = np.abs(_f64(w) - expect)
    assert np.all(off <= bound), f"off by {np.max(off - bound)} more than the bound"
    return ids, w


# experts around every change of the lanes and experts of a lane
EXPERTS = [1, 2, 7, 8, 9, 31, 32, 33, 60, 64, 65, 100, 128, 129, 160, 255, 256, 257, 384, 512, 513, 1000, 1024]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", EXPERTS)
def test_route(g, experts, dtype, kind):
    gen = _gen(1, experts, kind)
    for turn, tokens in enumerate((1, 37, 300)):
        logits, bias = _normal(gen, tokens, experts, dtype=dtype, std=2.0), _normal(gen, experts, std=0.1)
        for top_k in sorted({1, min(2, experts), min(8, experts), min(experts, 40)}):
            for with_bias in (False, True):
                check(g, logits, top_k, kind, bias if with_bias else None, renorm=(turn + top_k + with_bias) % 2 == 0,
                      scale=2.5 if turn else 1.0)


@pytest.mark.parametrize("top_k", [256, 129])
def test_route_of_many(g, top_k):
    gen = _gen(2, top_k)
    for experts in (256, 700, 1024):
        logits = _normal(gen, 9, experts)
        check(g, logits, top_k, 0, renorm=True)
        check(g, logits, top_k, 1, _normal(gen, experts))


# experts, groups, kept: groups inside a lane, of a lane's experts, of several lanes, across their borders
GROUPS = [(8, 8, 3), (8, 2, 1), (16, 4, 2), (60, 5, 2), (64, 8, 4), (96, 32, 7), (128, 8, 8), (160, 8, 3), (256, 8, 4),
          (256, 32, 5), (256, 2, 1), (320, 10, 4), (512, 16, 4), (1024, 32, 9), (1000, 8, 1)]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,groups,kept", GROUPS)
def test_route_by_groups(g, experts, groups, kept, dtype, kind):
    gen = _gen(3, experts, groups, kind)
    logits, bias = _normal(gen, 150, experts, dtype=dtype), _normal(gen, experts, std=0.1)
    top_k = min(8, kept * experts // groups)
    for group_top in (1, 2):
        for b in (None, bias):
            check(g, logits, top_k, kind, b, groups, kept, group_top, renorm=group_top == 2, scale=2.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", [8, 60, 256, 512, 1024])
def test_ties_go_to_the_lowest(g, experts, dtype):
    gen = _gen(4, experts)
    flat = torch.zeros(40, experts, dtype=dtype, device="cuda")
    few = torch.randint(-2, 3, (200, experts), generator=gen, device="cuda").to(dtype)
    few[::3] *= -0.0  # zeros of both signs are equal
    none, half = torch.zeros(experts, device="cuda"), torch.full((experts,), 0.5, device="cuda")
    steps = torch.randint(0, 2, (experts,), generator=gen, device="cuda") * 0.25
    for kind in (0, 1):
        for bias in (None, none, half, steps):
            for logits in (flat, few):
                check(g, logits, 3, kind, bias)
                check(g, logits, 4, kind, bias, groups=4, top_groups=2, group_top=2)
                check(g, logits, 4, kind, bias, groups=4, top_groups=3, group_top=1)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("experts", [8, 64, 256, 1024])
def test_choices_that_32_bits_cannot_tell_apart(g, experts, kind):
    """Biases that bring every score to the same value but for their own rounding: the order is that of 64 bits."""
    gen = _gen(5, experts, kind)
    for dtype in DTYPES:
        logits = _normal(gen, 1, experts, dtype=dtype).expand(20, experts)
        s = torch.from_numpy(scores(_f64(logits[:1]), kind, g)[0])
        bias = (1.0 - s).float().cuda()
        value = s.numpy() + _f64(bias)
        assert np.ptp(value) < 1e-6 and np.unique(value).size > 1
        check(g, logits, min(8, experts), kind, bias)
        check(g, logits, 2, kind, bias, groups=4, top_groups=2, group_top=2)
        check(g, logits, 2, kind, bias, groups=4, top_groups=2, group_top=1)
        # neighbours in 32 bits
        base = torch.full((30, experts), 1.0, device="cuda")
        base += torch.randint(0, 40, base.shape, generator=gen, device="cuda") * 2.0 ** -23
        check(g, base, min(8, experts), kind)
        check(g, base, 2, kind, groups=4, top_groups=3, group_top=2)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("experts", [20, 60, 128, 256, 505, 942])
def test_neighbours_among_many(g, experts, kind):
    """Many logits a few units in the last place apart, more of them than are chosen: none of those left is above any
    of those taken."""
    gen = _gen(22, experts)
    for tokens in (300, 4100):
        steps = torch.randint(0, 5, (tokens, experts), generator=gen, device="cuda") * 2.0 ** -21
        logits = torch.round(_normal(gen, tokens, experts) * 2) / 2 + steps
        for top_k in (3, 8):
            check(g, logits, top_k, kind, renorm=True)
            check(g, logits, top_k, kind, torch.zeros(experts, device="cuda"), renorm=True)
            check(g, logits, top_k, kind, torch.randint(0, 3, (experts,), generator=gen, device="cuda") * 2.0 ** -22)
            check(g, logits[:, :experts // 4 * 4], top_k, kind, None, 4, 3, 2)


@pytest.mark.parametrize("kind", [0, 1])
def test_weights_of_small_scores(g, kind):
    """A bias chooses experts whose scores nearly vanish: their weights are as exact as any."""
    gen = _gen(23, kind)
    for experts in (7, 60, 256):
        logits = _normal(gen, 500, experts, std=30.0)
        logits[:, 0] = 90.0
        bias = torch.rand(experts, generator=gen, device="cuda") * 40
        bias[0] = -100.0
        check(g, logits, 5, kind, bias, renorm=True)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("experts,groups,kept", [(8, 4, 2), (8, 4, 4), (60, 5, 2), (64, 8, 3), (160, 8, 8), (256, 8, 4), (256, 8, 8),
                                                 (1024, 32, 9)])
def test_groups_of_the_lowest_biases(g, experts, groups, kept, kind):
    """A bias of the type's lowest value masks nothing for good: groups whose two best add up to less than 32 bits hold
    come after all others, and before those without an expert."""
    gen = _gen(24, experts, kept)
    least, each = torch.finfo(torch.float32).min, experts // groups
    for tokens in (5, 4100):
        logits = _normal(gen, tokens, experts)
        logits[1, :each], logits[2, each:] = -float("inf"), -float("inf")
        for bias in (torch.full((experts,), least), torch.full((experts,), least / 2), torch.full((experts,), -least),
                     torch.where(torch.arange(experts) // each == groups - 1, 0.5, least),
                     torch.where(torch.arange(experts) // each < 2, -float("inf"), least),
                     torch.where(torch.arange(experts) % each == 1, 0.25, least),
                     torch.where(torch.arange(experts) % 2 == 0, -least, least)):
            for dtype in DTYPES:
                check(g, logits.to(dtype), min(8, kept * each), kind, bias.cuda(), groups, kept, 2, renorm=True)
                check(g, logits.to(dtype), min(8, kept * each), kind, bias.cuda(), groups, kept, 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_experts(g, dtype):
    gen = _gen(6)
    inf = float("inf")
    for experts in (8, 40, 256, 600):
        logits = _normal(gen, 60, experts, dtype=dtype)
        logits[torch.rand(60, experts, generator=gen, device="cuda") < 0.6] = -inf
        logits[3], logits[17], logits[40, 1:] = -inf, torch.finfo(dtype).min, -inf
        logits[5, ::2] = torch.finfo(dtype).min
        bias = _normal(gen, experts)
        bias[::3] = -inf
        for kind in (0, 1):
            for b in (None, bias):
                for renorm in (False, True):
                    check(g, logits, 5, kind, b, renorm=renorm)
                    check(g, logits, 4, kind, b, 4, 2, 2, renorm=renorm)
                    check(g, logits, 4, kind, b, 2, 1, 1, renorm=renorm)
        ids, w = g.gbs_expert_route(logits[3:4], 5, renormalise=True)
        assert (ids == -1).all() and (w == 0).all()


def test_far_logits(g):
    """Sums that would vanish or overflow in 32 bits."""
    for kind in (0, 1):
        for low in (-3e38, -300.0, -80.0, 80.0, 3e38):
            logits = torch.full((3, 20), low, device="cuda")
            logits[1, 4], logits[2, 5] = low * 0.999, low * 1.001 if abs(low) < 1e38 else low
            check(g, logits, 3, kind, renorm=True)
            check(g, logits, 3, 0)


def test_nan_and_infinity_show(g):
    nan, inf = float("nan"), float("inf")
    logits = torch.arange(64, device="cuda", dtype=torch.float32).repeat(4, 1) / 16
    logits[1, 9], logits[2, 30] = nan, inf
    for kind in (0, 1):
        for bias in (None, torch.zeros(64, device="cuda")):
            for groups in (1, 4):
                ids, w = g.gbs_expert_route(logits, 2, score_type=kind, bias=bias, num_groups=groups,
                                            top_groups=max(1, groups // 2), group_top=2, renormalise=True)
                assert ids[0].tolist() == [63, 62] and ids[3].tolist() == [63, 62]
                assert torch.isfinite(w[0]).all() and torch.isfinite(w[3]).all()
                if kind == 1 or bias is None and groups == 1:
                    assert ids[1, 0] == 9
                # an infinite logit's sigmoid is 1, and its group's two best add up to less than others' do
                if groups == 1 and (kind == 1 or bias is None):
                    assert ids[2, 0] == 30
                assert torch.isnan(w[1]).any()
    # a masked expert's row is not poisoned, nor are others
    logits[1, 9] = -inf
    ids, w = g.gbs_expert_route(logits[1:2], 2)
    assert ids[0].tolist() == [63, 62] and torch.isfinite(w).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_places(g, dtype):
    gen = _gen(7)
    wide = _normal(gen, 50, 700, dtype=dtype)
    for start in (0, 1, 2, 3, 8):
        for experts in (8, 60, 256):
            check(g, wide[:, start:start + experts], 4, 0)
            check(g, wide[::2, start:start + experts], 4, 1, _normal(gen, experts + 1)[1:])
    row = _normal(gen, 1, 128, dtype=dtype).expand(33, 128)
    check(g, row, 4, 0)
    ids, weights = torch.empty(50, 4, dtype=torch.int64, device="cuda"), torch.empty(50, 4, dtype=dtype, device="cuda")
    got = check(g, wide[:, :60], 4, 0, renorm=True, ids_out=ids, weights_out=weights)
    assert got[0] is ids and got[1] is weights
    ids, w = g.gbs_expert_route(wide[:0], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_rows_past_32_bits(g):
    """Rows more than 2^32 bytes and 2^31 values from the first."""
    gen = _gen(8)
    rows, stride = 40, 1 << 27
    wide = torch.empty((rows - 1) * stride + 64, dtype=torch.bfloat16, device="cuda").as_strided((rows, 64), (stride, 1))
    wide.copy_(_normal(gen, rows, 64))
    ids, _ = check(g, wide, 4, 0)
    d = g.gbs_expert_route_grad(torch.ones(rows, 4, device="cuda"), wide, ids, d_logits_out=wide.clone())
    assert torch.equal(d, g.gbs_expert_route_grad(torch.ones(rows, 4, device="cuda"), wide.contiguous(), ids))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,groups,kept", [(129, 3, 1), (160, 8, 3), (200, 1, 1), (256, 8, 4), (256, 32, 5), (256, 2, 1)])
def test_many_tokens_of_many_experts(g, experts, groups, kept, dtype, kind):
    """From 4096 tokens on two share a warp: plain rows, equal values, masks, and values that 32 bits cannot tell
    apart, beside one another."""
    gen = _gen(21, experts, groups)
    tokens = 4097
    logits, bias = _normal(gen, tokens, experts), _normal(gen, experts, std=0.1)
    logits[1::7] = torch.randint(-3, 4, logits[1::7].shape, generator=gen, device="cuda").float()
    logits[2::7][torch.rand(logits[2::7].shape, generator=gen, device="cuda") < 0.7] = -float("inf")
    logits[3::70] = -float("inf")
    logits[4::70] = torch.finfo(dtype).min
    logits = logits.to(dtype)
    top_k = min(8, kept * experts // groups)
    for b in (None, bias, torch.zeros(experts, device="cuda")):
        for group_top in (1, 2):
            check(g, logits, top_k, kind, b, groups, kept, group_top, renorm=group_top == 1, scale=2.5)
    one = _normal(gen, 1, experts, dtype=dtype).expand(tokens, experts)
    s = torch.from_numpy(scores(_f64(one[:1]), kind, g)[0])
    check(g, one, top_k, kind, (1.0 - s).float().cuda(), groups, kept, 2)
    # two rows by turns, one of them close: the warp's other token is unharmed
    pair = torch.where(torch.arange(tokens, device="cuda")[:, None] % 2 == 0, one.float(), _normal(gen, tokens, experts)).to(dtype)
    check(g, pair, top_k, kind, (1.0 - s).float().cuda(), groups, kept, 2, renorm=True)


def test_many_tokens(g):
    logits = _normal(_gen(9), 300_001, 8, dtype=torch.bfloat16)
    ids, w = g.gbs_expert_route(logits, 2, renormalise=True)
    value, order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), order[:, :2])
    want = torch.softmax(value[:, :2].double(), 1)
    assert ((w.double() - want).abs() <= (66 + 2 * 12) * EPS32 * want + EPS32).all()


# ---------------------------------------------------------------------------
# the gradient
# ---------------------------------------------------------------------------


def grad_by_hand(g, l, ids, d_w, kind, renorm, scale):
    """(gradient, magnitude of its terms)."""
    s, out, size = scores(l, kind, g), np.zeros_like(l), np.zeros_like(l)
    here = (ids >= 0) & (ids < l.shape[1])
    at = np.where(here, ids, 0)
    d_w = np.where(here, d_w, 0.0)
    p = np.where(here, np.take_along_axis(s, at, 1), 0.0)
    q = weights_by_hand(g, l, np.where(here, ids, -1), kind, True, 1.0)[0]
    x = np.take_along_axis(l, at, 1)
    rest = 1.0 / (1.0 + np.exp(x)) if kind == g.GBS_SCORE_SIGMOID else np.ones_like(x)
    gw = d_w * scale
    if renorm:
        part = q * rest * (gw - (gw * q).sum(1, keepdims=True))
        much = q * rest * (np.abs(gw) + (np.abs(gw) * q).sum(1, keepdims=True))
    elif kind == g.GBS_SCORE_SIGMOID:
        part = gw * p * rest
        much = np.abs(part)
    else:
        part, much = gw * p, np.abs(gw * p)
        out -= s * part.sum(1, keepdims=True)
        size += s * much.sum(1, keepdims=True)
    for k in range(ids.shape[1]):
        rows = np.flatnonzero(here[:, k])
        out[rows, ids[rows, k]] += part[rows, k]
        size[rows, ids[rows, k]] += much[rows, k]
    return out, size


def check_grad(g, logits, ids, d_w, kind, renorm, scale=1.0, **out):
    d = g.gbs_expert_route_grad(d_w, logits, ids, score_type=kind, renormalise=renorm, scale=scale, **out)
    l = _f64(logits)
    want, size = grad_by_hand(g, l, ids.cpu().numpy(), _f64(d_w), kind, renorm, scale)
    rel, least = UNIT[d.dtype]
    far = np.abs(l) if kind == g.GBS_SCORE_SIGMOID else np.max(l, 1, keepdims=True) - l
    units = 2 * (64 + ids.shape[1] + 2 * np.max(np.where(np.isfinite(far) & (far < 100), far, 0.0), 1, keepdims=True))
    bound = units * EPS32 * size * (1 + rel) + rel * np.abs(want) + least
    off = np.abs(_f64(d) - want)
    assert d.dtype == logits.dtype and np.all(off <= bound), f"off by {np.max(off - bound)} more than the bound"
    return d


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", EXPERTS)
def test_gradient(g, experts, dtype, kind, renorm):
    gen = _gen(11, experts)
    for tokens in (1, 37, 200):
        logits = _normal(gen, tokens, experts, dtype=dtype, std=2.0)
        for top_k in sorted({1, min(2, experts), min(8, experts), min(experts, 40)}):
            ids, w = g.gbs_expert_route(logits, top_k, score_type=kind)
            weight_type = dtype if top_k == 2 else torch.float32
            d_w = _normal(gen, tokens, top_k, dtype=weight_type)
            check_grad(g, logits, ids.long() if top_k == 1 else ids, d_w, kind, renorm, 2.5)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", [0, 1])
def test_gradient_by_differences(g, kind, renorm):
    """Central differences of the weights in 64 bits, the choice held: off by h^2 / 6 of the third derivative, which is
    at most 4 * |g| * scale here, and 2^-52 / h of the weights."""
    gen = _gen(12, kind)
    logits, h = _normal(gen, 5, 12), 2.0 ** -12
    ids, _ = g.gbs_expert_route(logits, 3, score_type=kind)
    d_w = _normal(gen, 5, 3)
    got = _f64(g.gbs_expert_route_grad(d_w, logits, ids, score_type=kind, renormalise=renorm, scale=1.5))
    l, at, by = _f64(logits), ids.cpu().numpy(), _f64(d_w)
    for e in range(12):
        step = np.zeros((1, 12))
        step[0, e] = h
        up = (by * weights_by_hand(g, l + step, at, kind, renorm, 1.5)[0]).sum(1)
        down = (by * weights_by_hand(g, l - step, at, kind, renorm, 1.5)[0]).sum(1)
        size = 1.5 * np.abs(by).sum(1)
        assert np.all(np.abs(got[:, e] - (up - down) / (2 * h)) <= size * (4 * h * h / 6 + 2.0 ** -52 / h * 4 + 160 * EPS32))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_masked_rows_and_odd_ids(g, dtype, kind, renorm):
    gen = _gen(13)
    for experts in (8, 40, 256):
        logits = _normal(gen, 30, experts, dtype=dtype)
        logits[torch.rand(30, experts, generator=gen, device="cuda") < 0.5] = -float("inf")
        logits[4], logits[9] = -float("inf"), torch.finfo(dtype).min
        ids, _ = g.gbs_expert_route(logits, 6, score_type=kind)
        assert (ids[4] == -1).all()
        d_w = _normal(gen, 30, 6)
        d = check_grad(g, logits, ids, d_w, kind, renorm)
        assert (d[4] == 0).all() and (d[logits == -float("inf")] == 0).all()
        # ids beyond the experts add nothing, the same one twice counts twice
        plain = _normal(gen, 30, experts, dtype=dtype)
        ids = torch.randint(0, 4, (30, 6), generator=gen, device="cuda")
        ids[3, 2], ids[5, 0], ids[7, :] = experts, -2 ** 40, 2 ** 40
        d = check_grad(g, plain, ids, d_w, kind, renorm)
        assert (d[7] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_strides(g, dtype):
    gen = _gen(14)
    wide, out = _normal(gen, 40, 300, dtype=dtype), torch.full((40, 300), 7.0, dtype=dtype, device="cuda")
    for start, experts in ((0, 256), (1, 256), (3, 61), (8, 8)):
        logits = wide[:, start:start + experts]
        ids, _ = g.gbs_expert_route(logits, 3)
        for renorm in (False, True):
            check_grad(g, logits, ids, _normal(gen, 40, 3), 0, renorm, d_logits_out=out[:, start:start + experts])
            assert (out[:, :start] == 7).all() and (out[:, start + experts:] == 7).all()
            out.fill_(7.0)


def test_equal_calls_give_equal_bits(g):
    gen = _gen(15)
    logits = _normal(gen, 3000, 256)
    ids = torch.randint(0, 3, (3000, 40), generator=gen, device="cuda")  # every expert many times
    d_w = _normal(gen, 3000, 40)
    first = [g.gbs_expert_route_grad(d_w, logits, ids, score_type=k, renormalise=r) for k in (0, 1) for r in (False, True)]
    for _ in range(5):
        again = [g.gbs_expert_route_grad(d_w, logits, ids, score_type=k, renormalise=r) for k in (0, 1) for r in (False, True)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ---------------------------------------------------------------------------
# in use
# ---------------------------------------------------------------------------


def test_streams_and_graphs(g):
    gen = _gen(16)
    a, b = _normal(gen, 500, 64), _normal(gen, 500, 64)
    want = [g.gbs_expert_route(t, 4, renormalise=True) for t in (a, b)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids, w = g.gbs_expert_route(a, 4, renormalise=True, stream=side)
    d = g.gbs_expert_route_grad(w, a, ids, renormalise=True, stream=side)
    side.synchronize()
    assert torch.equal(ids, want[0][0]) and torch.equal(w, want[0][1])
    at, d_w = a.clone(), want[0][1].clone()
    out = [torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), torch.empty_like(a)]
    g.gbs_expert_route(at, 4, renormalise=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gbs_expert_route(at, 4, renormalise=True, ids_out=out[0], weights_out=out[1])
        g.gbs_expert_route_grad(d_w, at, out[0], renormalise=True, d_logits_out=out[2])
    for source, (ids, w) in zip((a, b, a), (want[0], want[1], want[0])):
        at.copy_(source)
        graph.replay()
        assert torch.equal(out[0], ids) and torch.equal(out[1], w)
        assert torch.equal(out[2], g.gbs_expert_route_grad(d_w, source, ids, renormalise=True))
    del d


def test_refusals_on_the_gpu(g):
    logits = torch.zeros(6, 16, device="cuda")
    for bad in (dict(top_k=0), dict(top_k=17), dict(top_k=5, num_groups=4), dict(top_k=2, num_groups=3),
                dict(top_k=2, num_groups=4, top_groups=5), dict(top_k=2, num_groups=4, top_groups=0),
                dict(top_k=2, group_top=3), dict(top_k=2, score_type=2), dict(top_k=2, bias=torch.zeros(15, device="cuda")),
                dict(top_k=2, ids_out=torch.zeros(6, 3, dtype=torch.int32, device="cuda")),
                dict(top_k=2, bias=torch.zeros(16)), dict(top_k=2, ids_out=torch.zeros(6, 2, dtype=torch.int32))):
        with pytest.raises((ValueError, g.GbsError)):
            g.gbs_expert_route(logits, **bad)
    with pytest.raises(TypeError):
        g.gbs_expert_route(logits, 2, weights_out=torch.zeros(6, 2, dtype=torch.float16, device="cuda"))
    ids = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        g.gbs_expert_route_grad(torch.zeros(6, 3, device="cuda"), logits, ids)
    with pytest.raises(ValueError):
        g.gbs_expert_route_grad(torch.zeros(6, 2, device="cuda"), logits, ids, d_logits_out=torch.zeros(6, 15, device="cuda"))


def test_compiled_calls_and_the_binding_agree(g, monkeypatch):
    """Calls with every output given go through the compiled calls, others through the binding."""
    gen = _gen(17)
    got = []
    logits = [_normal(gen, 40, 96, dtype=d)[:, :64] for d in DTYPES]
    bias, d_w = _normal(gen, 64), _normal(gen, 40, 4)
    for fast in (True, False):
        if fast and g._fast is None:
            pytest.skip("the compiled calls are not built")
        if not fast:
            monkeypatch.setattr(g, "_fast", None)
        results = []
        for x in logits:
            for kw in (dict(), dict(bias=bias, score_type=1, num_groups=4, top_groups=2, group_top=2, renormalise=True, scale=2.5)):
                for ids_type, w_type in ((torch.int32, torch.float32), (torch.int64, x.dtype)):
                    ids, w = torch.empty(40, 4, dtype=ids_type, device="cuda"), torch.empty(40, 4, dtype=w_type, device="cuda")
                    results += [t.clone() for t in g.gbs_expert_route(x, 4, ids_out=ids, weights_out=w, **kw)]
                    grad = {k: kw[k] for k in ("score_type", "renormalise", "scale") if k in kw}
                    results.append(g.gbs_expert_route_grad(d_w.to(w_type), x, ids, d_logits_out=torch.empty_like(x), **grad))
        got.append(results)
    assert len(got[0]) == 36 and all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(g.GbsError):
        g.gbs_expert_route(logits[0], 4, num_groups=5, ids_out=ids, weights_out=w)


@pytest.mark.parametrize("bad", [dict(group_top=2 ** 64 + 1), dict(score_type=2 ** 32), dict(score_type=2 ** 32 + 1),
                                 dict(score_type=-2 ** 32)])
def test_integers_that_would_wrap_are_refused(g, bad):
    """By the compiled calls as by the binding, with every output given."""
    logits, ids, w = torch.zeros(6, 8, device="cuda"), torch.zeros(6, 2, dtype=torch.int32, device="cuda"), torch.zeros(6, 2, device="cuda")
    with pytest.raises((ValueError, g.GbsError)):
        g.gbs_expert_route(logits, 2, ids_out=ids, weights_out=w, **bad)
    if "score_type" in bad:
        with pytest.raises((ValueError, g.GbsError)):
            g.gbs_expert_route_grad(w, logits, ids, d_logits_out=torch.zeros(6, 8, device="cuda"), **bad)
