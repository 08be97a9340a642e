"""Beam search's selection and reordering on the GPU against plain implementations in 64 bits.

A value is score + logit - log of a sum.  Off, in units of 2^-24 of the sum: the exponentials 4, their exponents'
rounding the distance from the largest logit, on average at most ln(vocab), in two places and at a second base; 31 + 5 +
8 additions and three rescalings of 4.  60 + 4 * ln(vocab) covers them; the value's rounding to 32 bits adds 2^-24 of it.
Candidates further apart than that come in their order; those of one beam always do."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:.*encountered in.*:RuntimeWarning")]

EPS32 = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
INF = float("inf")


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


def best_by_hand(l, scores, finished, end_id, count):
    """(values, beams, tokens) of one batch, and all candidates by (beam, token): l [beams, vocab] in 64 bits."""
    found, value = [], {}
    for i in range(l.shape[0]):
        if scores[i] == -np.inf:
            continue
        if finished[i]:
            found.append((i, end_id))
            value[i, end_id] = scores[i]
            continue
        top = l[i].max()
        if top == -np.inf:
            continue
        lse = np.log(np.exp(l[i] - top).sum())
        order = np.argsort(-l[i], kind="stable")[:count]
        for w in order:
            if l[i, w] != -np.inf:
                found.append((i, int(w)))
                value[i, int(w)] = scores[i] + ((l[i, w] - top) - lse)
    found.sort(key=lambda c: (-value[c], c))
    return found[:count], value


def check(g, logits, scores, count, finished=None, end_id=0, exactly=False, **kw):
    got = g.gbs_beam_select(logits, scores, count, finished=finished, end_id=end_id, **kw)
    if kw.get("return_temp"):
        got, temp = got
        assert g.gbs_get_status(temp) == g.GBS_OK
    values, beams, tokens = (t.cpu().numpy() for t in got)
    batch, width = scores.shape
    count = width if count is None else count
    l, s = logits.double().cpu().numpy().reshape(batch, width, -1), scores.double().cpu().numpy()
    done = np.zeros((batch, width), bool) if finished is None else finished.cpu().numpy().astype(bool)
    near = EPS32 * (60 + 4 * np.log(l.shape[2] + 1))
    for b in range(batch):
        want, value = best_by_hand(l[b], s[b], done[b], end_id, count)
        n = len(want)
        assert (beams[b, n:] == -1).all() and (tokens[b, n:] == -1).all() and (values[b, n:] == -np.inf).all()
        mine = list(zip(beams[b, :n].tolist(), tokens[b, :n].tolist()))
        assert len(set(mine)) == n
        for k in range(n):
            v = value[want[k]]
            off = 0 if done[b, mine[k][0]] else near
            assert mine[k] in value, f"batch {b} place {k}: {mine[k]}"
            assert abs(values[b, k] - value[mine[k]]) <= off + EPS32 * abs(v) + 1e-37
            if mine[k] != want[k]:  # another one, as close as the sums are off
                assert not exactly and abs(value[mine[k]] - v) <= 2 * near, f"batch {b} place {k}: {mine[k]}, not {want[k]}"
        for i in range(width):  # a beam's own candidates keep the logits' order
            own = [w for beam, w in mine if beam == i and not done[b, i]]
            assert own == sorted(own, key=lambda w: (-l[b, i, w], w))
    return got


# vocabularies around slices, packs of 16 bytes and warps, of both lengths of slices
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 257, 1000, 2047, 2048, 2049, 8192, 8193, 32000, 50257, 70000])
@pytest.mark.parametrize("batch,beams,count", [(1, 1, 1), (1, 4, 8), (3, 5, 5), (2, 16, 32), (1, 32, 64)])
def test_select(g, vocab, batch, beams, count, dtype):
    gen = _gen(1, vocab, batch)
    logits = _normal(gen, batch * beams, vocab, dtype=dtype, std=2.5)
    scores = -3.0 * torch.rand(batch, beams, generator=gen, device="cuda")
    check(g, logits, scores, count, return_temp=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,batch,beams", [(300, 40, 8), (8200, 40, 4), (33000, 64, 3)])
def test_select_of_many_batches(g, vocab, batch, beams, dtype):
    gen = _gen(2, vocab)
    logits = _normal(gen, batch * beams, vocab, dtype=dtype, std=2.5)
    scores = -3.0 * torch.rand(batch, beams, generator=gen, device="cuda")
    finished = torch.rand(batch, beams, generator=gen, device="cuda") < 0.3
    scores[torch.rand(batch, beams, generator=gen, device="cuda") < 0.2] = -INF
    scores[0], finished[1], scores[2, 1:] = -INF, True, -INF
    check(g, logits, scores, 2 * beams, finished, end_id=vocab - 1)
    check(g, logits, scores, None, finished.to(torch.uint8) * 7, end_id=2)


@pytest.mark.parametrize("vocab", [300_000, 1_200_001])
def test_select_of_many_slices(g, vocab):
    """More slices of a row than are merged at once."""
    gen = _gen(3)
    for batch, beams in ((1, 2), (8, 4)):
        check(g, _normal(gen, batch * beams, vocab, dtype=torch.bfloat16, std=2.0), -torch.rand(batch, beams, device="cuda"), 40)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,vocab", [(1, 5000), (60, 20000)])
def test_ties_go_to_the_lowest(g, dtype, batch, vocab):
    """Rows of one value (every logit reaches the bound), of two, and steps; beams at the same score."""
    gen = _gen(4)
    beams = 3
    flat = torch.zeros(batch * beams, vocab, dtype=dtype, device="cuda")
    scores = torch.zeros(batch, beams, device="cuda")
    got = check(g, flat, scores, 6)
    assert got[1].tolist() == [[0] * 6] * batch and got[2].tolist() == [list(range(6))] * batch
    two = torch.randint(0, 2, flat.shape, generator=gen, device="cuda").to(dtype)
    two[:, 1::3] *= -0.0
    check(g, two, scores, 16)
    few = torch.randint(-9, 10, flat.shape, generator=gen, device="cuda").to(dtype)
    check(g, few, scores, 16)


def test_logarithm_of_a_whole_number(g):
    """n logits of 0 have the sum n in whatever order it is formed, so a value shows the logarithm alone.  Its series is
    off by at most 2^-24 of u^2 / 2 a few times over, u below 1 / 59: 5e-11; the beam's score is log n to 32 bits, so
    that what is left is of that size.  The value's own rounding adds 2^-24 of it."""
    most, count = 4096, 1024
    n = torch.cat([torch.arange(1, count, device="cuda"), torch.tensor([most], device="cuda")])
    logits = torch.zeros(count, most, device="cuda").masked_fill_(torch.arange(most, device="cuda") >= n[:, None], -INF)
    exact = torch.log(n.double())
    for dtype in DTYPES:
        for scores in (torch.log(n.double()).float(), torch.zeros(count, device="cuda")):
            values, _, tokens = g.gbs_beam_select(logits.to(dtype), scores[:, None].contiguous(), 1)
            want = scores.double() - exact
            assert (tokens == 0).all() and ((values[:, 0].double() - want).abs() <= 5e-11 + EPS32 * want.abs()).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_mislead_the_bound(g, dtype):
    """Sorted rows, and rows whose best logits belong to one thread, one group, one slice or one end."""
    vocab, gen = 20000, _gen(5)
    base = torch.sort(_normal(gen, 1, vocab), dim=1)[0].to(dtype)
    rows = [base, base.flip(1)]
    for place in (slice(0, 8), slice(0, 128), slice(8192, 16384), slice(19990, 20000), slice(0, 20000, 2048)):
        row = _normal(gen, 1, vocab, std=0.01).to(dtype) - 20
        row[:, place] += 30
        rows.append(row)
    rows.append(torch.where(torch.arange(vocab, device="cuda") // 8 % 64 == 0, -50.0, rows[2].float())[None, 0].to(dtype))
    for group in (0, 1, 7):  # one warp's logits far below all others
        row = _normal(gen, 1, vocab, dtype=dtype)
        row[0, (torch.arange(vocab, device="cuda") // 8 % 256) // 32 == group] = -100
        rows.append(row)
    logits = torch.cat(rows)
    for count in (1, 5, 16, 64):
        check(g, logits, torch.zeros(logits.size(0), 1, device="cuda"), count)
        check(g, logits.repeat(30, 1), torch.zeros(30 * logits.size(0), 1, device="cuda"), count)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_logits(g, dtype):
    gen = _gen(6)
    for vocab in (50, 9000, 30001):
        logits = _normal(gen, 40, vocab, dtype=dtype)
        logits[torch.rand(40, vocab, generator=gen, device="cuda") < 0.7] = -INF
        logits[3], logits[4, 1:], logits[5, :-2], logits[9] = -INF, -INF, -INF, -INF
        logits[6], logits[7, ::2] = torch.finfo(dtype).min, torch.finfo(dtype).min
        logits[8], logits[10] = torch.finfo(dtype).max / 2, 5e4
        check(g, logits, -torch.rand(10, 4, generator=gen, device="cuda"), 12)
        check(g, logits, -torch.rand(40, 1, generator=gen, device="cuda"), 64)


def test_far_logits(g):
    """Sums by a base that would overflow, next to ones that do not."""
    logits = torch.full((6, 9000), -3e38, device="cuda")
    logits[1, 70], logits[2, 8500], logits[3] = 0.0, -1e38, 3e38
    logits[4], logits[4, 5] = -90.0, 90.0
    logits[5, ::2] = 2e37
    check(g, logits, torch.zeros(6, 1, device="cuda"), 8)
    check(g, logits.repeat(40, 1), torch.zeros(240, 1, device="cuda"), 8)


# values that stand for "masked", or where logits can lie far out: on both sides of 2^20, from where on sums are formed
# about the largest logit itself, and up to where the product with log2(e) overflows
FAR = [9e5, 2.0 ** 20, 1.2e6, 1e9, 5e9, 1e10, 1e12, 1e20, 1e30, 1e36, 3e38]


class Repeated:
    """A call of many times the same batches, whose rows are cut into slices of several chunks."""

    def __init__(self, g, times):
        self.g, self.times = g, times

    def gbs_beam_select(self, logits, scores, count, finished=None, end_id=0):
        assert finished is None
        got = self.g.gbs_beam_select(logits.repeat(self.times, 1), scores.repeat(self.times, 1), count)
        first = tuple(t[:scores.size(0)] for t in got)
        assert all(torch.equal(t.view(self.times, *f.shape), f.expand(self.times, *f.shape)) for t, f in zip(got, first))
        return first


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("far", FAR)
def test_logits_of_any_size_beside_ordinary_ones(g, far, dtype, sign):
    """Whole packs, threads, chunks, slices, ends and rows of one far value."""
    vocab, gen = 20000, _gen(18)
    at = torch.arange(vocab, device="cuda")
    pack = at // 8
    places = [at >= 16000, at < 8192, at < 4096, pack % 3 == 0, pack % 256 < 128, at != 12345, at >= 0, at == 7, at < 0,
              (at >= 8192) & (at < 16384), at % 2 == 0, pack % 256 // 32 == 3]
    logits = _normal(gen, len(places), vocab, dtype=dtype, std=3.0)
    logits[torch.stack(places)] = sign * far
    scores = torch.zeros(len(places), 1, device="cuda")
    for count in (1, 8):
        check(g, logits, scores, count)
        check(Repeated(g, 20), logits, scores, count)
        check(Repeated(g, 80), logits, scores, count)
    check(g, logits, -torch.rand(3, 4, generator=gen, device="cuda"), 16)


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("middle", [2.0 ** 20, 1e6, 2.0 ** 21, 5e4])
def test_rows_around_a_far_value(g, middle, sign):
    """Logits on both sides of the border between the two ways of forming a sum, within one row."""
    gen = _gen(19)
    for std in (0.5, 4.0, 300.0):
        logits = sign * middle + _normal(gen, 6, 20000, std=std)
        logits[1] = torch.sort(logits[1])[0]
        logits[2] = torch.sort(logits[2], descending=True)[0]
        logits[3, :8192] = -1e10
        logits[4, 8192:] = -1e30
        for times in (1, 40, 160):
            check(Repeated(g, times), logits, torch.zeros(6, 1, device="cuda"), 8)


def test_nan_shows(g):
    nan = float("nan")
    for batch in (1, 40):
        logits, scores = _normal(_gen(7), batch * 3, 9000), torch.zeros(batch, 3, device="cuda")
        logits[1, 8], logits[2, 8700] = nan, INF
        values, beams, _ = g.gbs_beam_select(logits, scores, 4)
        assert torch.isnan(values[0]).all() and (beams[0] > 0).all()
        if batch > 1:
            check(g, logits[3:], scores[1:], 4)
        for part in (slice(0, 9000), slice(100, 9000), slice(0, 8192)):  # whole threads, chunks and rows of NaN
            logits[2] = -INF
            logits[2, part] = nan
            values, beams, _ = g.gbs_beam_select(logits[2:3], scores[:1, :1].contiguous(), 4)
            assert torch.isnan(values).all() and (beams == 0).all()
        scores[0, 0] = nan
        values, beams, _ = g.gbs_beam_select(logits[:3], scores[:1], 4)
        assert torch.isnan(values).all() and (beams == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_places(g, dtype):
    gen = _gen(8)
    wide = _normal(gen, 12, 9100, dtype=dtype)
    scores = -torch.rand(3, 4, generator=gen, device="cuda")
    for start, vocab in ((0, 9000), (1, 9000), (3, 9001), (8, 517), (5, 9095)):
        check(g, wide[:, start:start + vocab], scores, 8)
    check(g, wide[::2], scores[:, :2].contiguous(), 3)
    check(g, wide[:1].expand(12, 9100), scores, 8)
    out = tuple(torch.empty(3, 8, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
    got = check(g, wide, scores, 8, out=out)
    assert all(a is b for a, b in zip(got, out))
    dirty = torch.full((4096,), 0xff, dtype=torch.uint8, device="cuda")
    empty = g.gbs_beam_select(wide[:0], scores[:0], 8, temp=dirty)
    assert empty[0].shape == (0, 8) and g.gbs_get_status(dirty) == g.GBS_OK


def test_rows_past_32_bits(g):
    gen = _gen(9)
    rows, stride, vocab = 40, 1 << 27, 20000
    wide = torch.empty((rows - 1) * stride + vocab, dtype=torch.bfloat16, device="cuda").as_strided((rows, vocab), (stride, 1))
    wide.copy_(_normal(gen, rows, vocab))
    check(g, wide, -torch.rand(10, 4, generator=gen, device="cuda"), 8)


def test_values_close_across_beams(g):
    """Equal rows at equal scores tie exactly: the lowest beam first, then the lowest token."""
    row = _normal(_gen(10), 1, 30000)
    logits, scores = row.expand(4, 30000), torch.full((1, 4), -1.5, device="cuda")
    got = check(g, logits, scores, 8)
    best = torch.sort(row[0], descending=True, stable=True)[1][:2].tolist()
    assert got[1][0].tolist() == [0, 1, 2, 3] * 2 and got[2][0].tolist() == [best[0]] * 4 + [best[1]] * 4


def test_work_buffer_and_streams(g):
    gen = _gen(11)
    logits = [_normal(gen, 20, 30000, dtype=torch.bfloat16) for _ in range(2)]
    scores = -torch.rand(5, 4, generator=gen, device="cuda")
    want = [g.gbs_beam_select(x, scores, 8) for x in logits]
    temp = torch.full((1 << 22,), 0xff, dtype=torch.uint8, device="cuda")  # whatever it held before
    got, same = g.gbs_beam_select(logits[0], scores, 8, temp=temp, return_temp=True)
    assert same is temp and g.gbs_get_status(temp) == g.GBS_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = g.gbs_beam_select(logits[1], scores, 8, temp=temp, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    # two graphs, each with its own buffer, replayed by turns with other inputs
    x, graphs, outs = logits[0].clone(), [], []
    for count in (8, 4):
        out = tuple(torch.empty(5, count, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
        _, own = g.gbs_beam_select(x, scores, count, out=out, return_temp=True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gbs_beam_select(x, scores, count, out=out, temp=own)
        graphs.append((graph, own))
        outs.append(out)
    for which in (1, 0, 1):
        x.copy_(logits[which])
        for (graph, _), out in zip(graphs, outs):
            graph.replay()
        for out in outs:
            assert all(torch.equal(a, b[:, :a.size(1)]) for a, b in zip(out, want[which]))


def test_equal_calls_give_equal_bits(g):
    gen = _gen(12)
    logits, scores = _normal(gen, 64, 50257, dtype=torch.float16), -torch.rand(16, 4, device="cuda")
    first = g.gbs_beam_select(logits, scores, 16)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(first, g.gbs_beam_select(logits, scores, 16)))


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------


def reorder_by_hand(state, parents, dim, out=None):
    src, to = state.clone(), (state if out is None else out).clone()
    s, t = src.movedim((dim, dim + 1), (0, 1)), to.movedim((dim, dim + 1), (0, 1))
    for b, of in enumerate(parents.tolist()):
        for j, i in enumerate(of):
            if 0 <= i < s.size(1):
                t[b, j] = s[b, i]
    return to


def _state(gen, shape, dtype):
    if dtype.is_floating_point:
        return _normal(gen, *shape).to(dtype)
    return torch.randint(0, 100, shape, generator=gen, device="cuda").to(dtype)


SHAPES = [((3, 4, 50), 0), ((2, 5, 1), 0), ((1, 1, 7), 0), ((2, 8, 3, 16, 40), 0), ((6, 2, 16, 4, 9, 8), 1), ((2, 3, 1, 31, 2, 5), 2),
          ((3, 32, 1, 100, 3), 0), ((2, 17), 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int64, torch.uint8, torch.bool])
@pytest.mark.parametrize("shape,dim", SHAPES)
def test_reorder(g, shape, dim, dtype):
    gen = _gen(13, shape)
    batch, beams = shape[dim], shape[dim + 1]
    for low, high in ((0, beams), (-1, beams + 1), (0, 1)):
        state = _state(gen, shape, dtype)
        parents = torch.randint(low, high, (batch, beams), generator=gen, device="cuda", dtype=torch.int32)
        want = reorder_by_hand(state, parents, dim)
        assert g.gbs_beam_reorder(state, parents, dim) is state
        assert torch.equal(state, want)
        for into in (1, beams, min(32, beams + 3)):
            parents = torch.randint(low, high, (batch, into), generator=gen, device="cuda", dtype=torch.int32)
            out = _state(gen, (*shape[:dim + 1], into, *shape[dim + 2:]), dtype)
            want, before = reorder_by_hand(state, parents, dim, out), state.clone()
            assert g.gbs_beam_reorder(state, parents, dim, out=out) is out
            assert torch.equal(out, want) and torch.equal(state, before)


def test_every_permutation_and_function(g):
    """All maps of four beams to four, in place: permutations, cycles, chains, stars."""
    maps = torch.tensor(list(itertools.product(range(4), repeat=4)), dtype=torch.int32, device="cuda")
    for dtype, length in ((torch.int32, 33), (torch.bfloat16, 3), (torch.float32, 1024)):
        state = torch.arange(256 * 4 * length, device="cuda").view(256, 4, length).to(dtype)
        want = torch.gather(state, 1, maps.long()[:, :, None].expand(256, 4, length))
        assert torch.equal(g.gbs_beam_reorder(state, maps), want)


@pytest.mark.parametrize("beams", [2, 3, 4, 7, 8, 13, 16, 32])
def test_cycles_in_place_by_every_unit(g, beams):
    """Each beam goes where another one comes from: cycles both ways and reversals, in units of 1 to 16 bytes, with and
    without a shorter end."""
    gen = _gen(20, beams)
    at = torch.arange(beams, dtype=torch.int32, device="cuda")
    parents = torch.stack([(at + 1) % beams, (at - 1) % beams, beams - 1 - at, at ^ 1 if beams % 2 == 0 else at])
    for length, pad in ((1, 0), (3, 0), (2, 0), (4, 0), (8, 0), (16, 0), (64, 0), (5, 3), (6, 2), (12, 4), (24, 8), (40, 8), (333, 3),
                        (4096, 0), (5001, 7)):
        whole = torch.randint(0, 256, (4, beams, length + pad), generator=gen, device="cuda", dtype=torch.uint8)
        want = whole.clone()
        want[:, :, :length] = torch.gather(whole[:, :, :length], 1, parents.long()[:, :, None].expand(4, beams, length))
        g.gbs_beam_reorder(whole[:, :, :length], parents)
        assert torch.equal(whole, want)


@pytest.mark.parametrize("into", [1, 2, 5])
def test_in_place_into_fewer_beams(g, into):
    """The state's first beams as the target: the others are read and left as they are.  Batches whose beams overlap are
    refused in place, and read all the same into another buffer."""
    gen = _gen(21, into)
    state = _normal(gen, 2, 3, 5, 77)
    parents = torch.randint(-1, 6, (3, into), generator=gen, device="cuda", dtype=torch.int32)
    want = state.clone()
    want[:, :, :into] = reorder_by_hand(state, parents, 1, state[:, :, :into])
    out = state[:, :, :into]
    assert g.gbs_beam_reorder(state, parents, 1, out=out) is out and torch.equal(state, want)
    flat = _normal(gen, 3 * 2 + 5, 77)
    windows = flat.as_strided((3, 5, 77), (2 * 77, 77, 1))
    target, before = torch.zeros(3, into, 77, device="cuda"), flat.clone()
    want = reorder_by_hand(windows, parents, 0, target)
    assert torch.equal(g.gbs_beam_reorder(windows, parents, out=target), want)
    with pytest.raises(g.GbsError):
        g.gbs_beam_reorder(windows, parents, out=windows[:, :into])
    assert torch.equal(flat, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
def test_reorder_cut_and_strided(g, dtype):
    """Caches in use up to a length, views at any place; what lies beyond is left as it is."""
    gen = _gen(14)
    whole = _state(gen, (4, 3, 6, 5, 40, 24), dtype)
    parents = torch.randint(0, 6, (3, 6), generator=gen, device="cuda", dtype=torch.int32)
    for length in (1, 7, 39, 40):
        mine, want = whole.clone(), whole.clone()
        want[..., :length, :] = reorder_by_hand(whole[..., :length, :], parents, 1)
        g.gbs_beam_reorder(mine[..., :length, :], parents, 1)
        assert torch.equal(mine, want)
    # heads before beams
    mine = whole.clone().permute(0, 1, 3, 2, 4, 5)[:, 0]  # [4, heads 5, beams 6, 40, 24]
    heads = parents[:1].expand(5, 6).contiguous()
    want = reorder_by_hand(mine, heads, 1)
    assert torch.equal(g.gbs_beam_reorder(mine, heads, 1), want)
    # rows that start anywhere
    flat = _state(gen, (3, 6, 1001), dtype)
    for start, end in ((1, 1001), (3, 990), (16, 17)):
        mine, want = flat.clone(), flat.clone()
        want[:, :, start:end] = reorder_by_hand(flat[:, :, start:end], parents, 0)
        g.gbs_beam_reorder(mine[:, :, start:end], parents)
        assert torch.equal(mine, want)
    # an expanded source, and one in other places than its target
    one = _state(gen, (3, 1, 500), dtype).expand(3, 6, 500)
    assert torch.equal(g.gbs_beam_reorder(one, parents, out=torch.empty(3, 6, 500, dtype=dtype, device="cuda")), one)
    source, target = flat[:, :, 5:500], torch.zeros(3, 6, 600, dtype=dtype, device="cuda")[:, :, 2:497]
    assert torch.equal(g.gbs_beam_reorder(source, parents, out=target), reorder_by_hand(source, parents, 0, target))


def test_reorder_past_32_bits(g):
    """States of more than 2^32 bytes, and strides beyond."""
    gen = _gen(15)
    state = torch.empty(2, 2, 4, 1 << 28, dtype=torch.bfloat16, device="cuda")
    for o, b, j in itertools.product(range(2), range(2), range(4)):
        state[o, b, j] = o * 8 + b * 4 + j
    parents = torch.tensor([[3, 3, 1, 2], [1, 0, -1, 3]], dtype=torch.int32, device="cuda")
    g.gbs_beam_reorder(state, parents, 1)
    for o, b, j in itertools.product(range(2), range(2), range(4)):
        parent = int(parents[b, j])
        assert (state[o, b, j] == o * 8 + b * 4 + (parent if parent >= 0 else j)).all()
    del state
    wide = torch.empty(7 * (1 << 30) + 1000, dtype=torch.bfloat16, device="cuda").as_strided((2, 4, 1000), (1 << 32, 1 << 30, 1))
    wide.copy_(_normal(gen, 2, 4, 1000))
    want = reorder_by_hand(wide, parents, 0)
    assert torch.equal(g.gbs_beam_reorder(wide, parents), want)


def test_reorder_streams_and_graphs(g):
    gen = _gen(16)
    state = _normal(gen, 3, 4, 1000)
    parents = torch.randint(0, 4, (3, 4), generator=gen, device="cuda", dtype=torch.int32)
    side = torch.cuda.Stream()
    want = reorder_by_hand(state, parents, 0)
    torch.cuda.synchronize()
    g.gbs_beam_reorder(state, parents, stream=side)
    side.synchronize()
    assert torch.equal(state, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gbs_beam_reorder(state, parents)
    for _ in range(3):
        parents.copy_(torch.randint(0, 4, (3, 4), generator=gen, device="cuda", dtype=torch.int32))
        want = reorder_by_hand(state, parents, 0)
        graph.replay()
        assert torch.equal(state, want)


def test_refusals_on_the_gpu(g):
    logits, scores = torch.zeros(6, 100, device="cuda"), torch.zeros(2, 3, device="cuda")
    for bad in (dict(num_out=0), dict(num_out=65), dict(num_out=2 ** 64 + 1), dict(end_id=2 ** 31),
                dict(finished=torch.zeros(2, 2, dtype=torch.bool, device="cuda")), dict(finished=torch.zeros(2, 3, dtype=torch.bool)),
                dict(out=(torch.zeros(2, 2, device="cuda"),) * 3)):
        with pytest.raises((ValueError, TypeError, g.GbsError)):
            g.gbs_beam_select(logits, scores, **bad)
    with pytest.raises(ValueError):
        g.gbs_beam_select(logits[:5], scores)
    with pytest.raises(g.GbsError):
        g.gbs_beam_select(torch.zeros(33, 10, device="cuda"), torch.zeros(1, 33, device="cuda"))
    state, parents = torch.zeros(2, 3, 8, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for call in (lambda: g.gbs_beam_reorder(state, parents[:, :2]), lambda: g.gbs_beam_reorder(state, parents.long()),
                 lambda: g.gbs_beam_reorder(state, parents, dim=2), lambda: g.gbs_beam_reorder(state, parents, dim=-1),
                 lambda: g.gbs_beam_reorder(state, parents.cpu()), lambda: g.gbs_beam_reorder(state[:, :1].expand(2, 3, 8), parents),
                 lambda: g.gbs_beam_reorder(state, parents, out=state[:, :, :7]),
                 lambda: g.gbs_beam_reorder(torch.zeros(2, 3, 4, 4, 8, device="cuda")[:, :, :3, :3, :5], parents)):
        with pytest.raises((ValueError, TypeError, g.GbsError)):
            call()


def test_compiled_calls_and_the_binding_agree(g, monkeypatch):
    """Calls with every output given go through the compiled calls, others through the binding."""
    gen = _gen(17)
    logits, scores = _normal(gen, 12, 5000, dtype=torch.bfloat16), -torch.rand(3, 4, generator=gen, device="cuda")
    finished = torch.rand(3, 4, generator=gen, device="cuda") < 0.5
    states = [_normal(gen, 2, 3, 4, 5, 40, 8)[..., :33, :], _normal(gen, 2, 3, 4, 77), _normal(gen, 3, 4),
              _normal(gen, 2, 5, 3, 4, 10).permute(0, 2, 3, 1, 4)]
    parents = torch.randint(-1, 4, (3, 4), generator=gen, device="cuda", dtype=torch.int32)
    got = []
    for fast in (True, False):
        if fast and g._fast is None:
            pytest.skip("the compiled calls are not built")
        if not fast:
            monkeypatch.setattr(g, "_fast", None)
        out = tuple(torch.empty(3, 8, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
        temp = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        results = []
        for f in (None, finished, finished.to(torch.uint8)):
            results += [t.clone() for t in g.gbs_beam_select(logits, scores, 8, finished=f, end_id=7, out=out, temp=temp)]
        for state in states:
            dim = 0 if state.dim() == 2 else 1
            results.append(g.gbs_beam_reorder(state.clone(memory_format=torch.preserve_format), parents, dim).clone())
            target = torch.zeros_like(state)
            results.append(g.gbs_beam_reorder(state, parents, dim, out=target))
        got.append(results)
    assert len(got[0]) == 17 and all(torch.equal(a, b) for a, b in zip(*got))
    for bad in (dict(num_out=65), dict(num_out=0), dict(end_id=2 ** 31)):
        with pytest.raises((ValueError, g.GbsError)):
            g.gbs_beam_select(logits, scores, **{**dict(num_out=8, out=out, temp=temp), **bad})


@pytest.mark.parametrize("shape,dim", [((2, 0, 3, 4, 5), 2), ((3, 4, 2, 0, 5), 0), ((3, 4, 0), 0), ((2, 3, 4, 0, 5, 7), 1), ((0, 4, 5), 0)])
def test_an_empty_state(g, shape, dim):
    state = torch.zeros(*(n + 1 for n in shape), device="cuda")[tuple(slice(0, n) for n in shape)]
    parents = torch.zeros(shape[dim], shape[dim + 1], dtype=torch.int32, device="cuda")
    assert g.gbs_beam_reorder(state, parents, dim) is state
