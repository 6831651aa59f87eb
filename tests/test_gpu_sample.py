"""Sampling against the float64 oracle (GPU only).

A token equals the oracle's unless u or top-p lies within 2^-38 of a border (the
weights are rounded to 2^-44 of the largest, the oracle's sums are in long
doubles): none of these inputs does, which the test asserts.  The log probability
is rounded once to fp32: half a step, 2^-24 of it, plus 2^-40 for the mass.
"""

import numpy as np
import pytest
import torch

import bit_ptq_vla_amd as q
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dt=torch.float32):
    return None if a is None else torch.tensor(np.asarray(a), dtype=dt, device=DEV)


def run(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, workspace=True):
    """On the given device logits; NumPy settings."""
    rows = logits.shape[0]
    args = (dev(u), dev(temperature), dev(top_k, torch.int32), dev(top_p), dev(min_p))
    if workspace:
        token, logprob = q.qlin_sample(logits, *args)
    else:
        token = torch.empty(rows, dtype=torch.int32, device=DEV)
        logprob = torch.empty(rows, dtype=torch.float32, device=DEV)
        ptr = [None if a is None else a.data_ptr() for a in args]
        ld = logits.stride(0) if rows > 1 else -(-logits.shape[1] // 8) * 8
        q._check(q.load().qlin_sample(logits.data_ptr(), q._TORCH_TO_QLIN[logits.dtype], rows, logits.shape[1], ld, *ptr,
                                      token.data_ptr(), logprob.data_ptr(), None, 0, q._stream(logits.device)), "sample")
    torch.cuda.synchronize()
    return token.cpu().numpy(), logprob.cpu().numpy()


def check(logits, u, workspace=True, **settings):
    x = logits.detach().cpu().double().numpy()
    token, logprob = run(logits, u, workspace=workspace, **settings)
    for r in range(len(x)):
        one = {n: (np.float32(v[r]).item() if n != "top_k" else int(v[r])) for n, v in settings.items() if v is not None}
        want, lp, near = oracle.sample(x[r], float(np.float32(u[r])), **one)
        assert near > 2.0 ** -38, "the input lies on a border"
        assert token[r] == want, (r, one, token[r], want)
        if np.isnan(lp):
            assert np.isnan(logprob[r])
        else:
            assert abs(float(logprob[r]) - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -38


def draw(rows, vocab, dtype, seed, std=2.5, shift=0.0):
    g = np.random.default_rng(seed)
    pitch = -(-vocab // 8) * 8
    x = torch.from_numpy((shift + std * g.standard_normal((rows, pitch))).astype(np.float32)).to(DT[dtype]).to(DEV)
    return x[:, :vocab], g


def copy(x):
    """A copy whose rows are 16-byte aligned, as x's are."""
    y = torch.empty((x.shape[0], -(-x.shape[1] // 8) * 8), dtype=x.dtype, device=DEV)[:, :x.shape[1]]
    return y.copy_(x)


SIZES = [(1, 1), (3, 2), (2, 7), (4, 8), (5, 9), (3, 63), (2, 1000), (2, 8191), (2, 8193), (3, 32003), (1, 65537), (2, 257152)]


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_sizes_and_filters(rows, vocab, dtype, workspace):
    x, g = draw(rows, vocab, dtype, vocab + rows)
    u = lambda: g.random(rows).astype(np.float32)  # noqa: E731
    f = lambda lo, hi: g.uniform(lo, hi, rows).astype(np.float32)  # noqa: E731
    check(x, u(), workspace)
    check(x, u(), workspace, temperature=f(0.3, 1.5))
    check(x, u(), workspace, top_k=g.integers(1, 100, rows))
    check(x, u(), workspace, temperature=f(0.3, 1.5), top_p=f(0.5, 0.99))
    check(x, u(), workspace, temperature=f(0.3, 1.5), min_p=f(0.01, 0.2))
    check(x, u(), workspace, temperature=f(0.7, 2.0), top_k=g.integers(1, vocab + 2, rows), top_p=f(0.3, 0.99), min_p=f(1e-4, 0.01))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_many_rows_with_their_own_settings(dtype):
    rows, vocab = 300, 2051
    x, g = draw(rows, vocab, dtype, 9)
    s = dict(temperature=g.uniform(0.5, 1.3, rows).astype(np.float32), top_k=g.integers(5, 200, rows),
             top_p=g.uniform(0.7, 0.99, rows).astype(np.float32), min_p=g.uniform(0.0, 0.1, rows).astype(np.float32))
    s["temperature"][::7] = 0.0
    s["top_k"][::5] = 0
    s["top_p"][::4] = 1.0
    s["min_p"][::3] = 0.0
    check(x, g.random(rows).astype(np.float32), **s)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_flat_rows_and_equal_logits(dtype, workspace):
    """More elements in a bin of the first histogram than are sorted at once."""
    rows, vocab = 4, 50001
    x, g = draw(rows, vocab, dtype, 21, std=1e-3, shift=1.0)
    y = copy(x)
    y[0] = 1.5                                        # one key
    y[1, ::3] = 1.25                                  # few
    y[2] = torch.linspace(-1e-6, 1e-6, vocab).to(y)
    for z in (x, y):
        check(z, g.random(rows).astype(np.float32), workspace)
        check(z, g.random(rows).astype(np.float32), workspace, top_k=[30000, 7, 49999, 2500], temperature=np.full(rows, 0.9, np.float32))
        check(z, g.random(rows).astype(np.float32), workspace, top_p=g.uniform(0.1, 0.9, rows).astype(np.float32))


def test_equal_logits_take_the_lowest_indices():
    x = torch.zeros((3, 4096), dtype=torch.float16, device=DEV)
    x[:, 1::2] = -0.0                                 # the zeros are equal
    u = np.array([0.0, 0.5, 0.999], np.float32)
    assert run(x, u)[0].tolist() == [0, 2048, 4091]
    assert run(x, u, top_k=[10, 10, 10])[0].tolist() == [0, 5, 9]
    assert run(x, u, temperature=[0.0, 0.0, -1.0])[0].tolist() == [0, 0, 0]
    x[:, 7] = 1.0
    assert run(x, u, temperature=[0.0, float("nan"), 1e-30])[0].tolist() == [7, 7, 7]


def test_borders_of_the_settings():
    x, g = draw(8, 777, "f32", 4)
    u = g.random(8).astype(np.float32)
    inf, nan = float("inf"), float("nan")
    plain = run(x, u)
    for s in (dict(top_k=[0] * 8), dict(top_k=[-5] * 8), dict(top_k=[777] * 8), dict(top_k=[2 ** 31 - 1] * 8),
              dict(top_p=[1.0] * 8), dict(top_p=[nan] * 8), dict(top_p=[inf] * 8), dict(min_p=[0.0] * 8),
              dict(min_p=[-1.0] * 8), dict(min_p=[nan] * 8), dict(temperature=[1.0] * 8)):
        got = run(x, u, **s)
        assert np.array_equal(got[0], plain[0]) and np.array_equal(got[1], plain[1]), s
    top = x.argmax(1).cpu().numpy()
    for s in (dict(top_k=[1] * 8), dict(top_p=[0.0] * 8), dict(top_p=[-1.0] * 8), dict(top_p=[1e-30] * 8),
              dict(min_p=[1.0] * 8), dict(min_p=[2.0] * 8), dict(min_p=[inf] * 8)):
        got = run(x, u, **s)
        assert np.array_equal(got[0], top) and np.all(got[1] == 0), s
    assert np.array_equal(run(x, [0.0, -1.0, nan, 0.0, 0.0, 0.0, 0.0, 0.0])[0], top)
    last = x.argmin(1).cpu().numpy()
    assert np.array_equal(run(x, [1.0, 2.0, inf, 1.0, 1.0, 1.0, 1.0, 1.0])[0], last)
    flat = run(x, u, temperature=[inf] * 8)           # equal weights, the order of the logits
    order = np.argsort(-x.cpu().numpy(), axis=1, kind="stable")
    assert np.array_equal(flat[0], [order[r, int(np.floor(float(u[r]) * 777))] for r in range(8)])


def test_masked_infinite_and_nan_logits():
    inf, nan = float("inf"), float("nan")
    x, g = draw(6, 999, "bf16", 5)
    x = copy(x)
    x[0, ::2] = -inf
    x[1, 5:] = torch.finfo(torch.bfloat16).min
    x[2, 100:] = nan
    x[3] = -inf
    x[4] = -inf
    x[4, 998] = -3e38
    x[5, 7] = x[5, 200] = inf
    u = np.array([0.7, 0.6, 0.9, 0.5, 0.999, 0.6], np.float32)
    check(x, u)
    check(x, u, top_p=np.full(6, 0.8, np.float32), top_k=[50] * 6)
    token, logprob = run(x, u)
    assert token[3] == -1 and np.isnan(logprob[3]) and token[4] == 998 and token[5] == 200
    assert run(x, u, temperature=[0.0] * 6)[0].tolist()[3:] == [-1, 998, 7]
    assert run(copy(torch.full((1, 5), nan, device=DEV)), [0.2])[0].tolist() == [-1]


def test_one_row_in_any_company_and_captured():
    x, g = draw(64, 32000, "f16", 6)
    u = g.random(64).astype(np.float32)
    p = np.full(64, 0.95, np.float32)
    token, logprob = run(x, u, top_p=p)
    for r in (0, 17, 63):
        got = run(x[r:r + 1], u[r:r + 1], top_p=p[:1])
        assert got[0][0] == token[r] and got[1][0] == logprob[r]
    for rows in (1, 64):
        du, dp = dev(u[:rows]), dev(p[:rows])
        work = q.sample_workspace(rows, 32000, DEV)
        out = (torch.empty(rows, dtype=torch.int32, device=DEV), None)
        y = copy(x[:rows])
        graph = torch.cuda.CUDAGraph()
        q.qlin_sample(y, du, top_p=dp, out=out, workspace=work)
        with torch.cuda.graph(graph):
            q.qlin_sample(y, du, top_p=dp, out=out, workspace=work)
        for k in range(3):
            y.copy_(x[:rows].roll(k, 1))
            want = run(y, u[:rows], top_p=p[:rows])[0]
            out[0].fill_(-7)
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(out[0].cpu().numpy(), want)


def test_frequencies_follow_the_weights():
    """20000 evenly spread u over one row: each token's share is its weight to one part in 20000, either side."""
    n = 20000
    x = torch.tensor([0.0, 1.0, -1.0, 0.5, 1.0], device=DEV).repeat(n, 1).contiguous()
    pitch = torch.zeros((n, 8), device=DEV)
    pitch[:, :5] = x
    token, logprob = run(pitch[:, :5], (np.arange(n) / n).astype(np.float32))
    w = np.exp(np.array([0.0, 1.0, -1.0, 0.5, 1.0]))
    w /= w.sum()
    share = np.bincount(token, minlength=5) / n
    assert np.all(np.abs(share - w) <= 2.0 / n)
    assert np.allclose(np.exp(logprob.astype(np.float64)), w[token], rtol=1e-6)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_a_small_top_k_behind_a_min_p_that_keeps_many(dtype):
    """Rows of which min-p keeps thousands and top-k a few, ties among them."""
    x, g = draw(9, 6000, dtype, 77, std=0.6)
    x[3] = (x[3] * 4).round() / 4
    x[4] = 0.25
    top_k = np.array([1, 2, 37, 100, 250, 256, 200, 255, 16])
    min_p = np.array([0.01, 0.02, 0.005, 0.01, 0.5, 0.01, 0.002, 0.03, 0.01])
    top_p = np.array([1.0, 0.9, 0.8, 0.7, 0.6, 0.95, 1.0, 0.5, 0.99])
    for shift in range(3):
        check(x, g.random(9), top_k=top_k, min_p=min_p, top_p=np.roll(top_p, shift), temperature=np.full(9, 0.9 + 0.2 * shift))


@pytest.mark.parametrize("vocab", [40, 1500, 5000])
@pytest.mark.parametrize("top", [255, 256, 511, 2 ** 19 + 255])
def test_zeros_among_denormals(vocab, top):
    """Elements at and around zero, whose weights are equal and whose order is that of
    their bits: the parts that the row is narrowed to end at, above and right below zero."""
    g = np.random.default_rng(vocab + top)
    rows = 9
    steps = g.integers(-300, 256, (rows, vocab))
    steps[:, ::3] = 0
    steps[3] = g.integers(-300, 1, vocab)
    steps[4] = g.integers(-2 ** 22, 256, vocab)
    steps[5] = np.where(g.random(vocab) < 0.5, 0, -1)
    steps[:, vocab // 2] = top
    x = np.ldexp(steps.astype(np.float64), -149).astype(np.float32)
    x[:, 1::4] = np.where(x[:, 1::4] == 0, np.float32(-0.0), x[:, 1::4])
    x[6, 5:9] = -1.0
    y = torch.zeros((rows, -(-vocab // 8) * 8))
    y[:, :vocab] = torch.from_numpy(x)
    y = y.to(DEV)[:, :vocab]
    assert np.array_equal(y.cpu().numpy().view(np.int32), x.view(np.int32))
    for workspace in (True, False):
        check(y, (np.arange(rows) + g.random(rows)) / rows, workspace)
        check(y, (np.arange(rows) + g.random(rows))[::-1] / rows, workspace, top_p=g.uniform(0.3, 0.99, rows))
        check(y, g.random(rows), workspace, top_k=g.integers(vocab // 3, vocab, rows))


def row_at_a_border(n, share):
    """A leader and n elements, one to each 32nd part of an octave from ten octaves below it:
    float32 logits, and a u (or top-p) that asks for 1 + share of the leader's weight."""
    x = -(np.arange(n) + 320.3) * np.log(2) / 32
    x = np.concatenate([[0.0], x]).astype(np.float32)
    w = lambda v: np.exp(np.asarray(v, np.longdouble))  # noqa: E731
    u = np.float32(1 / float(w(x).sum()))
    for at in (70, 330):                              # two elements' last bits bring the sum there
        ulps = np.arange(-4000, 4001)
        v = (x[at].view(np.int32) + ulps.astype(np.int32)).view(np.float32)
        total = w(np.delete(x, at)).sum() + w(v)
        x[at] = v[np.argmin(np.abs(total * np.longdouble(u) - (1 + share)))]
    return x, u


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("n,share", [(480, 2.0 ** -37), (480, -2.0 ** -37), (1400, 2.0 ** -36.5), (1400, -2.0 ** -37), (1700, 2.0 ** -37)])
def test_many_light_elements_at_a_border(n, share, workspace):
    """What a leader's weight and many far lighter ones sum to, one to a bin: listed at once,
    and in bins."""
    x, u = row_at_a_border(n, share)
    for vocab in (len(x), 50001):                     # (a row that is split, too)
        y = torch.full((1, -(-vocab // 8) * 8), -np.inf)
        y[0, vocab - len(x):vocab] = torch.from_numpy(x)
        y = y.to(DEV)[:, :vocab]
        check(y, [u], workspace)
        check(y, [0.9999], workspace, top_p=[u])
        check(y, [u], workspace, min_p=[1e-30])
        check(y, [u], workspace, top_k=[vocab - 1])


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("low", [-31.0, -32.3, -33.0, -40.0])
def test_a_wide_tail(low, workspace):
    """2^18 elements that weigh 2^-45 to 2^-58 of the largest each."""
    vocab = 2 ** 18
    x = torch.full((2, vocab), low, device=DEV)
    x[:, 0] = 0.0
    x[1, 1] = -1e-9
    if low > -40:
        check(x, [0.5, 0.5], workspace)
        check(x, [0.25, 0.75], workspace, top_p=[0.9, 0.5])
    check(x, [0.25, 0.25], workspace, top_k=[vocab - 5, 2])
    token, _ = run(x[:1], [1.0], workspace=workspace)
    # u = 1 - 2^-48: 2^-40 of the mass from the last one, at most
    assert vocab - 1 - token[0] <= 2.0 ** -40 / np.exp(low) + 1


@pytest.mark.parametrize("rows,vocab", [(1, 49153), (2, 50001), (64, 49999), (65, 49999), (85, 81927), (3, 65544), (128, 131072), (17, 131079), (1, 2 ** 18)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_split_rows(rows, vocab, dtype):
    """Rows that are split over blocks, and those next to them that are not: the same tokens,
    and the oracle's."""
    x, g = draw(rows, vocab, dtype, rows + vocab)
    u = g.random(rows).astype(np.float32)
    s = dict(temperature=g.uniform(0.5, 1.3, rows), top_k=g.integers(1, 400, rows), top_p=g.uniform(0.6, 1.1, rows),
             min_p=np.where(g.random(rows) < 0.5, 0.0, g.uniform(0.0, 0.05, rows)))
    s["temperature"][::5] = 0.0
    s["top_k"][::3] = 0
    few = slice(0, 4)
    for names in ((), ("temperature",), ("temperature", "top_p"), ("top_k",), tuple(s)):
        now = {n: s[n] for n in names}
        split, whole = run(x, u, **now), run(x, u, workspace=False, **now)
        assert np.array_equal(split[0], whole[0]) and np.array_equal(split[1], whole[1], equal_nan=True)
        check(x[few], u[few], **{n: v[few] for n, v in now.items()})


def test_split_rows_with_masks_flat_parts_and_captured():
    inf, nan = float("inf"), float("nan")
    rows, vocab = 6, 70000
    x, g = draw(rows, vocab, "f32", 31)
    x = copy(x)
    x[0, :40000] = -inf                                # parts without an element
    x[1, 30000:] = 0.5                                 # equal logits over parts
    x[2, 5:] = nan
    x[3] = -inf
    x[4, ::2] = -1e30                                  # parts whose largest lies far below
    x[4, 20000:] = -1e30
    x[5, 100] = x[5, 69999] = inf
    u = np.array([0.7, 0.6, 0.9, 0.5, 0.999, 0.6], np.float32)
    assert q.sample_workspace(rows, vocab, DEV) is not None
    for s in ({}, dict(top_p=np.full(rows, 0.8)), dict(top_k=[60000] * rows, temperature=np.full(rows, 0.7)), dict(temperature=np.zeros(rows))):
        check(x, u, **s)
        check(x, u, workspace=False, **s)
    du, work = dev(u), q.sample_workspace(rows, vocab, DEV)
    out = (torch.empty(rows, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV))
    y = copy(x)
    graph = torch.cuda.CUDAGraph()
    q.qlin_sample(y, du, out=out, workspace=work)
    with torch.cuda.graph(graph):
        q.qlin_sample(y, du, out=out, workspace=work)
    for k in range(3):
        y.copy_(x.roll(k, 0))
        want = run(y, u)
        work.fill_(255)
        out[0].fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out[0].cpu().numpy(), want[0]) and np.array_equal(out[1].cpu().numpy(), want[1], equal_nan=True)
