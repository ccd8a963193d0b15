"""Sampling from logits against the float64 oracle: kept sets and tokens exactly, probabilities to float's rounding."""
import numpy as np
import pytest
import torch

from oracle import zf_serve_oracle as R
from tests import helpers as H

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def check(zf, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """One call against the oracle, row by row."""
    n, V = logits.shape
    f = lambda x, t=np.float32: None if x is None else torch.as_tensor(np.asarray(x, t)).cuda()  # noqa: E731
    probs = torch.full((n, V), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(temperature=f(temperature), top_k=f(top_k, np.int32), top_p=f(top_p), min_p=f(min_p))
    tokens = zf.sample_tokens(logits.cuda(), f(u), probs=probs, status=status, **kw)
    alone = zf.sample_tokens(logits.cuda(), f(u), **kw)
    assert torch.equal(tokens, alone)
    tokens, probs = tokens.cpu().numpy(), probs.double().cpu().numpy()
    x = logits.double().numpy()
    bad = 0
    for r in range(n):
        one = {k: float(v[r]) for k, v in (("temperature", kw["temperature"]), ("top_p", kw["top_p"]), ("min_p", kw["min_p"])) if v is not None}
        if top_k is not None:
            one["top_k"] = int(top_k[r])
        kept = R.sample(x[r], **one)
        if kept is None or not 0 <= u[r] < 1:
            assert tokens[r] == -1 and not probs[r].any()
            bad = 1
            continue
        want = kept / kept.sum()
        # weights to 2^-30, their float value, the factor and the product rounded (2^-24 each); below 2^-100 of the
        # largest they may be 0
        assert (np.abs(probs[r] - want) <= 2.0 ** -22 * want + 2.0 ** -100).all(), (r, np.abs(probs[r] - want).max())
        assert not probs[r][kept == 0].any()
        token, near = R.draw(kept, float(np.float32(u[r])))
        assert tokens[r] in near, (r, tokens[r], token)
    assert int(status.item()) == (zf.DEV_BAD_PROBS if bad else 0)
    return tokens


def logits_of(n, V, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(n, V, generator=g)
    x[:, ::max(1, V // 7)] += 6 * torch.rand(n, x[:, ::max(1, V // 7)].shape[1], generator=g)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 8192, 50001])
def test_filters(zf, V, dtype):
    n = 12
    rng = np.random.default_rng(V)
    u = rng.random(n).astype(np.float32)
    u[0], u[1] = 0.0, np.float32(1 - 2.0 ** -24)
    x = logits_of(n, V, V, dtype)
    t = (0.3 + 1.5 * rng.random(n)).astype(np.float32)
    k = rng.integers(0, min(V, 300) + 2, n)
    p = (0.05 + rng.random(n)).astype(np.float32)
    m = (0.3 * rng.random(n) * (rng.random(n) < 0.7)).astype(np.float32)
    check(zf, x, u)
    check(zf, x, u, temperature=t)
    check(zf, x, u, top_k=k)
    check(zf, x, u, top_p=p, temperature=t)
    check(zf, x, u, min_p=m)
    check(zf, x, u, t, k, p, m)


def test_greedy_takes_the_first_of_equal_largest(zf):
    x = torch.tensor([[1.0, 5, 5, 2], [-3, -3, -3, -3], [0.0, -0.0, -1, 0], [-0.0, 0.0, -1, 0]])
    assert check(zf, x, [0.9] * 4, temperature=[0.0, 1e-7, 0.0, 0.0]).tolist() == [1, 0, 0, 0]


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lowest_index(zf, dtype):
    """All logits equal, thousands of equal ones beside others, and logits of few values: more ties than are listed."""
    V = 6000
    same = torch.zeros(4, V)
    steps = torch.randint(0, 3, (4, V), generator=torch.Generator().manual_seed(1)).float()
    near = torch.zeros(4, V)
    near[:, ::2] = 1e-3
    for x in (same, steps, near):
        x = x.to(dtype)
        u = [0.0, 0.3, 0.6, 0.99]
        check(zf, x, u, top_k=[1, 1500, 4097, 5999])
        check(zf, x, u, top_p=[0.25, 0.5, 0.75, 1 / 3])
        check(zf, x, u, top_k=[3000] * 4, top_p=[0.25, 0.5, 0.9, 0.999])
        check(zf, x, u, min_p=[1.0, 0.5, 0.2, 0.0], top_p=[0.5] * 4)


def test_close_logits(zf):
    """A whole vocabulary within a thousandth: all in the histogram's first bin."""
    x = 1e-3 * torch.randn(3, 40000, generator=torch.Generator().manual_seed(5))
    check(zf, x, [0.1, 0.5, 0.9], top_p=[0.1, 0.5, 0.999])
    check(zf, x, [0.1, 0.5, 0.9], top_k=[1, 20000, 39999], top_p=[0.4, 0.5, 0.9])
    check(zf, x + 4096, [0.1, 0.5, 0.9], top_k=[5, 20000, 39999], temperature=[1e-5, 1.0, 1e3])


def test_far_logits(zf):
    """Steep and flat temperatures, logits far apart, weights that vanish."""
    x = logits_of(6, 5000, 9, spread=40.0)
    check(zf, x, np.linspace(0, 0.99, 6), temperature=[1e-3, 0.1, 1, 30, 1e4, 1e30], top_p=[0.9] * 6, top_k=[4000, 0, 10, 0, 7, 0])
    x[:, 1::3] = -float("inf")
    x[:, 2::50] = float("nan")
    check(zf, x, np.linspace(0, 0.99, 6), top_k=[4999, 100, 3000, 0, 5000, 1], top_p=[1.0, 0.99, 0.5, 0.9, 1.0, 0.1])
    big = torch.tensor([[3e38, -3e38, 2.9e38, 0.0], [1e-40, 0.0, -1e-40, 1e-45]])
    check(zf, big, [0.5, 0.5], top_p=[0.9, 0.6])


def test_rows_that_cannot_be_sampled(zf):
    x = torch.zeros(12, 50)
    x[0], x[1, 3], x[2] = -float("inf"), float("inf"), float("nan")
    t, k, p, m, u = np.ones(12), np.zeros(12), np.ones(12), np.zeros(12), np.full(12, 0.5)
    t[3], t[4], t[5], k[6], p[7], p[8], m[9], u[10], u[11] = np.nan, -1, np.inf, -1, np.nan, -0.5, 1.01, 1.0, -0.1
    tokens = check(zf, x, u, t, k, p, m)
    assert (tokens == -1).all()
    x[:] = 0
    assert check(zf, x[:2], [0.5, 0.5], min_p=[-1.0, 1.0]).tolist() == [25, 25]


@pytest.mark.parametrize("V,dtype", [(128000, torch.bfloat16), (256000, torch.float32), (1300001, torch.float32),
                                     (2097152, torch.float16)])
def test_large_vocabularies(zf, V, dtype):
    """Over many CTAs; rows too large for shared memory."""
    x = logits_of(3, V, 3, dtype)
    check(zf, x, [0.1, 0.5, 0.999])
    check(zf, x, [0.1, 0.5, 0.999], top_k=[50, 20000, 0], top_p=[0.9, 0.99, 0.7], min_p=[0, 0, 1e-4])


def test_many_rows(zf):
    x = logits_of(700, 300, 4)
    check(zf, x, np.random.default_rng(1).random(700).astype(np.float32), top_p=np.full(700, 0.8), top_k=np.full(700, 40))


def test_strides_and_offsets(zf):
    """Rows of a padded or sliced matrix, at any alignment."""
    for dtype in TYPES:
        wide = logits_of(5, 1111, 6, dtype).cuda()
        u = torch.rand(5, generator=torch.Generator().manual_seed(2)).cuda()
        for cut in (slice(0, 1000), slice(1, 1001), slice(8, 1008), slice(3, 90)):
            a = zf.sample_tokens(wide[:, cut], u, top_p=u * 0 + 0.9)
            b = zf.sample_tokens(wide[:, cut].contiguous(), u, top_p=u * 0 + 0.9)
            assert torch.equal(a, b)
        t = wide[:, :64].t()                                          # a transposed one is copied
        assert torch.equal(zf.sample_tokens(t, torch.rand(64, device="cuda") * 0 + 0.5), zf.sample_tokens(t.contiguous(), torch.full((64,), 0.5, device="cuda")))


def test_probabilities_alone_and_captured(zf):
    x, u = logits_of(9, 3000, 8).cuda(), torch.rand(9).cuda()
    p = torch.full((9,), 0.9, device="cuda")
    both, only = torch.empty(9, 3000, device="cuda"), torch.empty(9, 3000, device="cuda")
    tokens = zf.sample_tokens(x, u, top_p=p, probs=both)
    assert zf.sample_tokens(x, top_p=p, probs=only) is None and torch.equal(both, only)
    out = torch.empty(9, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zf.sample_tokens(x, u, top_p=p, probs=only, tokens=out)
    for _ in range(2):
        x.add_(torch.randn(9, 3000, device="cuda"))
        want = zf.sample_tokens(x, u, top_p=p, probs=both)
        g.replay()
        assert torch.equal(out, want) and torch.equal(both, only)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = zf.sample_tokens(x, u, top_p=p, stream=s)
    s.synchronize()
    assert torch.equal(again, want)


def test_behind_a_late_writer(zf):
    """The kernel ahead lets the next one start and then writes the logits and the top-k."""
    late = H.late_writer()
    x, k = logits_of(20, 50000, 11, torch.bfloat16).cuda(), torch.arange(20, dtype=torch.int32, device="cuda") * 30
    u, p = torch.rand(20, device="cuda"), torch.full((20,), 0.8, device="cuda")
    want = zf.sample_tokens(x, u, top_k=k, top_p=p)
    d_x, d_k = torch.zeros_like(x), torch.zeros_like(k)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    s = torch.cuda.current_stream().cuda_stream
    assert late(k.data_ptr(), d_k.data_ptr(), 20, x.data_ptr(), d_x.data_ptr(), x.numel() // 2, 300000, s) == 0
    zf.sample_tokens(d_x, u, top_k=d_k, top_p=p, tokens=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_few_and_many_candidates(zf, dtype):
    """Around the number of candidates that are listed at once, by top-k and by min-p, with ties across the border."""
    V = 20000
    g = torch.Generator().manual_seed(12)
    x = (torch.randn(8, V, generator=g) * 3).to(dtype)
    tied = (torch.randn(8, V, generator=g) * 3).round().to(dtype)
    u = torch.rand(8, generator=g).numpy()
    for y in (x, tied):
        check(zf, y, u, top_k=[1, 2, 500, 511, 512, 513, 600, 1024])
        check(zf, y, u, top_k=[1, 2, 500, 511, 512, 513, 600, 1024], top_p=[0.0, 0.3, 0.9, 0.999, 0.5, 0.99, 0.7, 0.2])
        check(zf, y, u, min_p=[1.0, 0.9, 0.5, 0.2, 0.1, 0.05, 0.01, 1e-30], top_p=[0.9, 0.0, 0.5, 0.7, 0.9, 0.95, 0.99, 0.3])
        check(zf, y, u, top_k=[3, 9, 40, 100, 300, 505, 30, 20], min_p=[1.0, 0.9, 0.5, 0.2, 0.1, 0.05, 0.01, 1e-30],
              top_p=[0.9, 0.0, 0.5, 0.7, 0.9, 0.95, 0.99, 0.3], temperature=[0.1, 0.5, 1.0, 2.0, 5.0, 1.5, 0.01, 1.0])


@pytest.mark.parametrize("rows", [1, 12, 64])
def test_top_k_border_is_the_same_for_all_warps(zf, rows):
    """Top-k past the listed candidates, its border among many equal logits, and top-p behind it: every warp has to work
    with the same border, so tokens and distributions are the same bits in every call."""
    V = 128000
    g = torch.Generator().manual_seed(21)
    x = (3 * torch.randn(rows, V, generator=g)).to(torch.bfloat16)   # (some 140 equal ones at the thousandth place)
    u = torch.rand(rows, generator=g).numpy()
    k = np.array([600, 700, 999, 1000, 1001, 1500, 2000, 2500, 3001, 4000, 4500, 5000])[np.arange(rows) % 12]
    p = np.array([0.9, 0.99, 0.5, 0.7, 0.999])[np.arange(rows) % 5].astype(np.float32)
    if rows <= 12:
        check(zf, x, u, top_k=k, top_p=p)
    kw = dict(top_k=torch.as_tensor(k, dtype=torch.int32).cuda(), top_p=torch.from_numpy(p).cuda())
    x, u = x.cuda(), torch.from_numpy(u).cuda()
    first = torch.empty(rows, V, device="cuda")
    want = zf.sample_tokens(x, u, probs=first, **kw)
    again = torch.empty_like(first)
    for _ in range(30):
        tokens = zf.sample_tokens(x, u, probs=again, **kw)
        assert torch.equal(tokens, want) and torch.equal(again, first)


def test_a_negative_min_p_is_none(zf):
    """No weight is below it, so it keeps all, like 0; NaN and what is above 1 are refused."""
    x, u = logits_of(6, 3000, 14), np.linspace(0, 0.99, 6)
    m = np.array([-1.0, -1e-30, -0.0, -np.inf, -3e38, -0.5], np.float32)
    tokens = check(zf, x, u, min_p=m, top_p=[0.9] * 6)
    assert tokens.tolist() == check(zf, x, u, top_p=[0.9] * 6).tolist()
    assert check(zf, x[:2], u[:2], min_p=[np.nan, 1.5]).tolist() == [-1, -1]


def test_the_flattest_temperatures_and_the_farthest_logits(zf):
    """Temperatures up to the largest float, where the histogram's one bin has every logit; differences beyond it."""
    x, u = logits_of(4, 5000, 15), [0.1, 0.4, 0.7, 0.99]
    t = np.array([1e36, 1.5e37, 1e38, 3.4e38], np.float32)
    check(zf, x, u, temperature=t, top_p=[0.3, 0.5, 0.9, 1.0])
    k, p, m = np.array([1, 600, 3000, 0]), np.array([0.9, 0.9, 0.5, 0.999]), np.array([0.5, 1.0, 0.0, 1e-30])
    some = [0, 2, 3]
    check(zf, x[some], np.array(u)[some], temperature=t[some], top_k=k[some], top_p=p[some], min_p=m[some])
    # min_p 1: exp(-d / t) is 1 - d / t, d / t some 10^-36, for all but the largest: only that one is kept (the oracle's
    # float64 rounds them all to 1)
    largest = int(x[1].argmax())
    assert int((x[1] == x[1].max()).sum()) == 1
    f = lambda v, d=torch.float32: torch.tensor([v], dtype=d, device="cuda")  # noqa: E731
    probs = torch.empty(1, 5000, device="cuda")
    token = zf.sample_tokens(x[1:2].cuda(), f(0.4), temperature=f(1.5e37), top_k=f(600, torch.int32), top_p=f(0.9),
                             min_p=f(1.0), probs=probs)
    assert token.item() == largest and probs[0, largest] == 1 and probs.sum() == 1
    far = torch.tensor([[3e38, -3e38, 2e38, 1e38, -3.4e38]])
    same = torch.tensor([[3e38, -float("inf"), 2e38, 1e38, -float("inf")]])
    a, b = (torch.empty(1, 5, device="cuda") for _ in range(2))
    one = torch.full((1,), 1e38, device="cuda")
    zf.sample_tokens(far.cuda(), probs=a, temperature=one)
    zf.sample_tokens(same.cuda(), probs=b, temperature=one)
    assert torch.equal(a, b)
    check(zf, same, [0.5], temperature=[1e38])
