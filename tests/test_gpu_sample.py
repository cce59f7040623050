"""GPU tests of sample_logits against its definition in 64 bits (numpy), and
of the INT8 head with the sampler behind it.

Tokens have to be equal.  A probability is one weight over a sum, each a
whole number of 2^-44 of the largest weight, rounded once to fp32: within
2^-24 relative, plus 2^-43 absolute for the units and n 2^-45 relative for
the sum of n of them."""
import numpy as np
import pytest
import torch

import synth
from helpers import bf16_tensor

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
INF = float("inf")


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_gemm_speculative_b200 as m
    return m


def pick(row, u, temp, k, p, q):
    """(token, probability) of one row by the definition."""
    row = np.where(np.isnan(row), -np.inf, row.astype(np.float64))
    best = int(np.argmax(row))
    if row[best] == -np.inf:
        return -1, 0.0
    if not temp > 0:
        return best, 1.0
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        away = row - row[best]
        w = np.where(row == row[best], 1.0, np.exp(away / temp))
        if row[best] == np.inf:
            w = (row == np.inf).astype(np.float64)
    rank = np.argsort(-row, kind="stable")
    keep = np.ones(len(row), bool)
    if p < 1:
        sums = np.cumsum(w[rank])
        before = np.concatenate([[0.0], sums[:-1]])
        keep[rank] &= before < p * sums[-1]
    if k > 0:
        keep[rank[k:]] = False
    if q > 0 and row[best] != np.inf:
        keep &= away >= temp * np.log(min(q, 1.0))
    keep[best] = True
    ids = np.flatnonzero(keep & (w >= 2.0 ** -45))
    sums = np.cumsum(w[ids])
    over = np.flatnonzero(sums > u * sums[-1])
    at = over[0] if len(over) else len(ids) - 1
    return int(ids[at]), float(w[ids[at]] / sums[-1])


def check(mxg, logits, u, temp=None, k=None, p=None, q=None):
    M, V = logits.shape

    def dev(v, dtype):
        return None if v is None else torch.tensor(np.broadcast_to(v, (M,)).copy(), dtype=dtype,
                                                   device=DEV)
    args = (dev(temp, torch.float32), dev(k, torch.int32), dev(p, torch.float32),
            dev(q, torch.float32))
    ud = dev(u, torch.float32)
    tokens, probs = mxg.sample_logits(logits, ud, *args)
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    host = logits.float().cpu().numpy()

    def at(t, m, off):
        return off if t is None else t[m].item()
    for m in range(M):
        want, prob = pick(host[m], ud[m].item(), at(args[0], m, 1.0), at(args[1], m, 0),
                          at(args[2], m, 1.0), at(args[3], m, 0.0))
        what = f"row {m} of {M} x {V}: {[at(a, m, None) for a in args]}, u {ud[m].item()}"
        assert tokens[m] == want, what
        assert abs(probs[m] - prob) <= prob * (2.0 ** -24 + V * 2.0 ** -45) + 2.0 ** -43, what
    return tokens


def rows(M, V, dtype, seed, sigma=2.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(M, V, generator=g, device=DEV) * sigma).to(dtype)


def uniform(M, seed):
    return np.random.default_rng(seed).random(M).astype(np.float32)


SIZES = [1, 2, 7, 31, 32, 33, 100, 511, 512, 513, 1000, 4096, 4097, 5003, 8200, 16389, 32003,
         70001]
BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@BOTH
@pytest.mark.parametrize("V", SIZES)
def test_sample_sizes(mxg, V, dtype):
    M = 12
    t = np.resize(np.float32([1.0, 0.7, 1.3, 0.0]), M)
    k = np.resize(np.int32([0, 40, 3]), M)
    p = np.resize(np.float32([1.0, 0.9, 0.95, 0.5, 0.99]), M)
    q = np.resize(np.float32([0.0, 0.02]), M)
    check(mxg, rows(M, V, dtype, V), uniform(M, V), t, k, p, q)


@BOTH
@pytest.mark.parametrize("which", ["none", "t", "k", "p", "q", "kp", "kq", "pq", "kpq"])
@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_sample_filters(mxg, which, M, dtype):
    rng = np.random.default_rng(M)
    t = rng.choice(np.float32([0.3, 0.8, 1.0, 2.0]), M) if which != "none" else None
    k = rng.integers(1, 300, M).astype(np.int32) if "k" in which else None
    p = rng.uniform(0.05, 0.999, M).astype(np.float32) if "p" in which else None
    q = rng.uniform(0.0001, 0.5, M).astype(np.float32) if "q" in which else None
    check(mxg, rows(M, 9001, dtype, M), uniform(M, M), t, k, p, q)


@pytest.mark.parametrize("V,dtype", [(248320, torch.bfloat16), (248320, torch.float32),
                                     (393216, torch.bfloat16), (393215, torch.float32)])
@pytest.mark.parametrize("M", [1, 20])
def test_sample_vocabularies(mxg, V, dtype, M):
    rng = np.random.default_rng(V)
    check(mxg, rows(M, V, dtype, M), uniform(M, V), rng.choice(np.float32([0.7, 1.0]), M),
          rng.choice(np.int32([0, 50, 1000, 100000]), M),
          rng.choice(np.float32([0.8, 0.95, 1.0]), M), rng.choice(np.float32([0.0, 0.05]), M))


@BOTH
@pytest.mark.parametrize("V", [1, 40, 3000, 33000])
def test_sample_flat_rows(mxg, V, dtype):
    """Equal logits: every border falls among ties, lowest indices first."""
    M = 16
    u = np.float32([0, 0.25, 0.5, 0.75, 0.999, 0.125, 0.3, 0.6] * 2)
    logits = torch.full((M, V), -3.5, device=DEV, dtype=dtype)
    check(mxg, logits, u)
    check(mxg, logits, u, p=np.float32([0.5] * 8 + [0.9] * 8))
    check(mxg, logits, u, k=np.int32([1, 2, 3, 7, 20, 39, 40, 4000] * 2))
    check(mxg, logits, u, k=7, p=np.float32([0.001] * 8 + [0.7] * 8), q=1.0)


@BOTH
@pytest.mark.parametrize("levels", [2, 3, 17])
def test_sample_few_distinct_values(mxg, levels, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(levels)
    M = 24
    logits = (torch.randint(0, levels, (M, 6007), generator=g, device=DEV) * 0.5 - 1.0).to(dtype)
    rng = np.random.default_rng(levels)
    check(mxg, logits, uniform(M, 5), 0.9, rng.integers(1, 5000, M).astype(np.int32),
          rng.uniform(0.01, 1.0, M).astype(np.float32), rng.choice(np.float32([0, 0.3]), M))


@BOTH
def test_sample_masked_and_special_entries(mxg, dtype):
    V = 2050
    logits = rows(12, V, dtype, 9)
    logits[0] = -INF                                   # nothing to take
    logits[1] = float("nan")
    logits[2, 1:] = -INF                               # one entry
    logits[3, :-1] = -INF
    logits[4, ::2] = -INF
    logits[5, 100:] = float("nan")
    logits[6, [7, 1999]] = INF                         # +inf takes it all
    logits[7] = torch.finfo(dtype).min                 # the lowest value is no mask
    logits[8, 5:] = torch.finfo(dtype).min
    logits[9] = 0.0
    logits[9, ::3] = -0.0                              # one value, lowest index first
    logits[10] = torch.finfo(dtype).max
    logits[10, 3] = torch.finfo(dtype).min
    logits[11, 17] = float("nan")
    u = np.float32([0.5, 0.2, 0.9, 0.1, 0.7, 0.4, 0.6, 0.99, 0.3, 0.34, 0.5, 0.8])
    got = check(mxg, logits, u)
    assert list(got[:4]) == [-1, -1, 0, V - 1] and got[6] == 1999
    check(mxg, logits, u, 0.7, 50, 0.9, 0.01)
    check(mxg, logits, u, 0.0, 50, 0.9, 0.01)
    check(mxg, logits, u, 1.5, 10 ** 6, 0.5, 1e-30)
    check(mxg, logits, u, 1.0, 700, None, None)


@BOTH
def test_sample_parameters_at_their_ends(mxg, dtype):
    M = 10
    logits = rows(M, 1500, dtype, 2)
    u = uniform(M, 2)
    nan = float("nan")
    check(mxg, logits, u, np.float32([1e-45, 1e-6, 1e6, 3e38, INF, -1, nan, 0.0, 1e-3, 30]))
    check(mxg, logits, u, 1.0, np.int32([0, -1, 1, 2, 1499, 1500, 1501, 2 ** 31 - 1, -2 ** 31, 5]))
    check(mxg, logits, u, 1.0, None,
          np.float32([0.0, -1.0, 1e-30, 1e-7, 0.99999994, 1.0, 2.0, 0.5, -INF, INF]))
    check(mxg, logits, u, 1.0, None, None,
          np.float32([0.0, -1.0, 1.0, 2.0, INF, 1e-38, 0.999999, nan, 0.5, 1e-45]))
    edge = np.float32([0.0, 1.0, 2.0, -1.0, INF, -INF, 0.99999994, 1e-45, 0.5, 0.0])
    check(mxg, logits, edge)
    check(mxg, logits, edge, 0.8, 30, 0.9, 0.001)
    got = mxg.sample_logits(logits, torch.full((M,), nan, device=DEV))[0]
    last = mxg.sample_logits(logits, torch.full((M,), 2.0, device=DEV))[0]
    assert torch.equal(got, last)
    # NaN filters are off
    off = torch.full((M,), nan, device=DEV)
    ud = torch.tensor(u, device=DEV)
    assert torch.equal(mxg.sample_logits(logits, ud, top_p=off, min_p=off)[0],
                       mxg.sample_logits(logits, ud)[0])


@BOTH
def test_sample_strided_and_unaligned_rows(mxg, dtype):
    wide = rows(9, 4003, dtype, 5)
    for lo, hi in [(0, 4003), (1, 4002), (3, 3000), (5, 6), (7, 4003)]:
        check(mxg, wide[:, lo:hi], uniform(9, lo), 0.9, 60, 0.95)
    one = wide[:1, 5:3999]
    check(mxg, one, uniform(1, 1), 0.9, 60, 0.95)
    check(mxg, wide[::2], uniform(5, 1), 0.9, None, 0.9)


def test_sample_wide_spread_of_values(mxg):
    """Most of the mass in one entry, the rest far below it; huge logits."""
    for scale in (1e-3, 30.0, 1e4, 1e30):
        logits = rows(8, 3001, torch.float32, 4) * scale
        check(mxg, logits, uniform(8, 4), 1.0, 2000, 0.9)
        check(mxg, logits, uniform(8, 5), 1.0, None, 0.9999)


def test_sample_follows_the_distribution(mxg):
    """Evenly spaced random numbers: every token as often as its share, to
    within one (the number of steps in an interval)."""
    M, V = 4000, 57
    logits = rows(1, V, torch.float32, 1, 1.5).expand(M, V).contiguous()
    u = torch.arange(M, device=DEV, dtype=torch.float64).add(0.5).div(M).float()
    tokens, probs = mxg.sample_logits(logits, u)
    share = torch.softmax(logits[0].double(), 0) * M
    count = torch.bincount(tokens.long(), minlength=V).double()
    assert ((count - share).abs() <= 1.001).all()
    assert torch.equal(tokens, torch.sort(tokens).values)


def test_sample_outputs_streams_and_graphs(mxg):
    logits, u = rows(6, 12345, torch.bfloat16, 1), torch.rand(6, device=DEV)
    p = torch.full((6,), 0.9, device=DEV)
    want = mxg.sample_logits(logits, u, top_p=p)
    tokens = torch.full((8,), 77, dtype=torch.int32, device=DEV)
    probs = torch.full((8,), 7.0, device=DEV)
    got = mxg.sample_logits(logits, u, top_p=p, tokens=tokens[:6], probs=probs[:6])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert tokens[6:].tolist() == [77, 77] and probs[6:].tolist() == [7.0, 7.0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxg.sample_logits(logits, u, top_p=p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = mxg.sample_logits(logits, u, top_p=p)
        second = mxg.sample_logits(logits, u)
    logits.copy_(rows(6, 12345, torch.bfloat16, 2))
    for _ in range(3):
        u.copy_(torch.rand(6, device=DEV))
        graph.replay()
        assert torch.equal(first[0], mxg.sample_logits(logits, u, top_p=p)[0])
        assert torch.equal(second[0], mxg.sample_logits(logits, u)[0])
    call, (t, _) = mxg.prepare_sample_logits(logits, u, top_p=p)
    call()
    assert torch.equal(t, first[0])


def test_sample_reproducible_whatever_the_batch(mxg):
    """A row's token does not depend on the rows beside it (which change how
    many CTAs it gets)."""
    M, V = 300, 40000
    logits, u = rows(M, V, torch.float32, 6), torch.rand(M, device=DEV)
    p = torch.full((M,), 0.97, device=DEV)
    k = torch.full((M,), 5000, dtype=torch.int32, device=DEV)
    want = mxg.sample_logits(logits, u, top_k=k, top_p=p)
    for n in (1, 3, 20, 100):
        got = mxg.sample_logits(logits[:n], u[:n], top_k=k[:n], top_p=p[:n])
        assert torch.equal(got[0], want[0][:n]) and torch.equal(got[1], want[1][:n])
    for _ in range(5):
        assert torch.equal(mxg.sample_logits(logits, u, top_k=k, top_p=p)[0], want[0])


def alone(mxg, logits, u, t=None, k=None, p=None, q=None):
    """Every row in a call of its own: clusters, which the tests above hold to
    the definition."""
    out = [mxg.sample_logits(logits[m:m + 1], u[m:m + 1],
                             *[None if v is None else v[m:m + 1] for v in (t, k, p, q)])
           for m in range(len(u))]
    return torch.cat([a for a, _ in out]), torch.cat([b for _, b in out])


def both(mxg, logits, u, *filters):
    got, want = mxg.sample_logits(logits, u, *filters), alone(mxg, logits, u, *filters)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    return got[0]


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 255, 257, 2000, 16384, 32003, 40001, 131072, 248320])
def test_sample_batches_of_bf16_rows(mxg, V):
    """A batch that gives every row an SM counts values; the tokens and
    probabilities are those of the rows by themselves, bit by bit."""
    M = 40 if V > 40000 else 64
    rng = np.random.default_rng(V)
    logits = rows(M, V, torch.bfloat16, V)
    u = torch.tensor(uniform(M, V), device=DEV)
    u[0], u[1], u[2] = 0.0, 0.99999994, float("nan")
    t = torch.tensor(rng.choice(np.float32([0.0, 0.5, 1.0, 1.5, 1e-6, 1e6]), M), device=DEV)
    k = torch.tensor(rng.choice(np.int32([0, 1, 50, 1000, V, 2 ** 31 - 1]), M), device=DEV)
    p = torch.tensor(rng.choice(np.float32([1.0, 0.0, 0.3, 0.9, 0.999, 0.99999994]), M), device=DEV)
    q = torch.tensor(rng.choice(np.float32([0.0, 1e-30, 0.02, 0.9, 1.0]), M), device=DEV)
    both(mxg, logits, u, t, k, p, q)
    both(mxg, logits, u, None, k)
    both(mxg, logits, u, t, None, p)
    off = torch.ones(M, device=DEV)
    both(mxg, logits, u, t, None, off, q)          # the filters given but off
    both(mxg, logits, u, None, torch.zeros(M, dtype=torch.int32, device=DEV))


def test_sample_batches_of_masked_and_special_rows(mxg):
    M, V = 48, 2051
    logits = rows(M, V, torch.bfloat16, 9)
    low, nan = torch.finfo(torch.bfloat16).min, float("nan")
    logits[0] = -INF
    logits[1] = nan
    logits[2, 1:] = -INF
    logits[3, :-1] = -INF
    logits[4, ::2] = -INF
    logits[5, 100:] = nan
    logits[6, [7, 1999]] = INF
    logits[7] = low
    logits[8, 5:] = low
    logits[9] = 0.0
    logits[9, ::3] = -0.0
    logits[10] = torch.finfo(torch.bfloat16).max
    logits[10, 3] = low
    logits[11, 17] = nan
    logits[12] = 0.0
    logits[13] = -0.0
    logits[14, ::2], logits[14, 1::2] = 1e-40, -1e-40       # below the normal numbers
    logits[15].view(torch.int16)[5:900] = -1                # NaN with its sign set
    logits[16].view(torch.int16)[5:900] = 0x7FFF
    logits[17] = INF
    logits[18, ::2], logits[18, 1::2] = INF, -INF
    logits[19] = -1e-40
    logits[19, 5] = 0.0
    logits[20, :] = -1.0
    logits[20, 2050] = -0.99609375
    u = torch.tensor(uniform(M, 4), device=DEV)

    def of(v, dtype=torch.float32):
        return torch.full((M,), v, dtype=dtype, device=DEV)
    got = both(mxg, logits, u, None, of(0, torch.int32))
    assert got[:4].tolist() == [-1, -1, 0, V - 1] and int(got[6]) in (7, 1999)
    check(mxg, logits, u.cpu().numpy(), 0.7, 50, 0.9, 0.01)
    for q in (0.0, 1e-38, 0.3, 0.9962, 1.0):
        both(mxg, logits, u, of(1.0), of(700, torch.int32), None, of(q))
        both(mxg, logits, u, of(0.6), None, of(0.9), of(q))
    both(mxg, logits, u, of(0.0), of(5, torch.int32))
    both(mxg, logits, u, of(1e30), None, of(0.5))


@pytest.mark.parametrize("V", [66000, 140000, 300000])
def test_sample_batches_of_values_that_occur_often(mxg, V):
    """More than 65535 entries of one value, of either sign, with borders at,
    above and below them."""
    M = 42
    g = torch.Generator(device=DEV)
    g.manual_seed(V)
    logits = rows(M, V, torch.bfloat16, V)
    logits[:6] = -2.0                                       # all of a row
    logits[6:12] = 0.5
    few = torch.rand(V, generator=g, device=DEV) < 0.002
    logits[12:18] = torch.where(few, logits[12:18], -2.0)   # nearly all of it
    logits[18:24] = torch.where(few, logits[18:24], 0.5)
    logits[24:30, 65537:] = -1.0
    logits[24:30, :65537] = 1.0                             # the same magnitude
    logits[30:36, :65536] = -INF
    logits[36:39, :65536] = 0.0
    logits[36:39, :65536:2] = -0.0
    u = torch.tensor(uniform(M, V), device=DEV)
    t = torch.ones(M, device=DEV)
    k = torch.tensor(np.resize(np.int32([0, 100, 65535, 65536, 65600, V - 1]), M), device=DEV)
    p = torch.tensor(np.resize(np.float32([0.5, 0.9, 0.999, 0.1]), M), device=DEV)
    both(mxg, logits, u, t, k)
    both(mxg, logits, u, t, None, p)
    both(mxg, logits, u, t, k, p, torch.tensor(np.resize(np.float32([0, 0.05, 0.5]), M), device=DEV))
    check(mxg, logits[::3], u[::3].cpu().numpy(), 0.9, 65600, 0.95)


def test_sample_batches_at_any_address(mxg):
    wide = rows(40, 5003, torch.bfloat16, 5)
    u = torch.tensor(uniform(40, 5), device=DEV)
    p = torch.full((40,), 0.95, device=DEV)
    for lo, hi in [(0, 5003), (1, 5002), (3, 3000), (5, 6), (7, 5003), (6, 14)]:
        both(mxg, wide[:, lo:hi], u, None, None, p)
    # the mass at one end of long rows: the second pass starts from either
    logits = rows(40, 150000, torch.bfloat16, 6)
    logits[:, :20] += torch.linspace(-30, 30, 40, device=DEV)[:, None].bfloat16()
    logits[:, -20:] += torch.linspace(30, -30, 40, device=DEV)[:, None].bfloat16()
    logits[::7, 70000:70020] += 25.0
    for v in (0.0, 0.3, 0.5, 0.7, 0.9999):
        both(mxg, logits, torch.full_like(u, v), None, None, p)


@pytest.mark.parametrize("M", [128, 148, 149, 300])
def test_sample_batches_beside_the_number_of_sms(mxg, M):
    logits, u = rows(M, 17001, torch.bfloat16, M), torch.rand(M, device=DEV)
    p = torch.full((M,), 0.9, device=DEV)
    both(mxg, logits, u, None, None, p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = mxg.sample_logits(logits, u, top_p=p)
        second = mxg.sample_logits(logits, u, top_p=p)
    logits.copy_(rows(M, 17001, torch.bfloat16, M + 1))
    graph.replay()
    want = alone(mxg, logits, u, None, None, p)
    for got in (first, second):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_sample_batches_without_filters(mxg):
    logits, u = rows(110, 65543, torch.bfloat16, 3), torch.rand(110, device=DEV)
    both(mxg, logits, u, torch.rand(110, device=DEV) + 0.5)


@pytest.mark.parametrize("M", [1, 5, 32])
def test_step_with_adapters_head_and_sampler(mxg, M):
    """A decode step of requests with their own adapters and sampling
    parameters: INT4 projection, its adapters, INT8 head, tokens."""
    K, N, V, R, L = 512, 512, 1000, 16, 4
    lay, head = synth.int4_layer(M, K, N, 128, seed=M), synth.int8_layer(M, N, 1024, 128, seed=1)

    def repack(fn, layer):
        return fn(torch.from_numpy(layer.qweight).to(DEV),
                  torch.from_numpy(layer.scales.view(np.int16)).to(DEV), 128)
    w, hw = repack(mxg.w4a16_repack, lay), repack(mxg.w8a16_repack, head)
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    x = bf16_tensor(lay.X, DEV)
    a = (torch.randn(L, R, K, generator=g, device=DEV) * K ** -0.5).bfloat16()
    b = (torch.randn(L, N, R, generator=g, device=DEV) * R ** -0.5).bfloat16()
    index = torch.randint(-1, L, (M,), generator=g, device=DEV).int()
    u = torch.rand(M, generator=g, device=DEV)
    temp = torch.rand(M, generator=g, device=DEV) * 20
    k = torch.full((M,), 40, dtype=torch.int32, device=DEV)
    p = torch.full((M,), 0.95, device=DEV)

    def step():
        y = mxg.w4a16_gemm(x, w, N, K)
        h = mxg.lora_add(x, a, b, index, y, out=y)
        return h, mxg.w8a16_gemm_sample(h, hw, 1024, N, u, temp, k, p, vocab=V)
    h, (tokens, probs, logits) = step()
    # the parts, one by one
    y = mxg.w4a16_gemm(x, w, N, K)
    for i in range(L):
        r = index == i
        y[r] = (y[r].double() + (x[r].double() @ a[i].double().T) @ b[i].double().T).bfloat16()
    assert (h.double() - y.double()).abs().max() <= 2.0 ** -7 * y.double().abs().max()
    assert torch.equal(logits, mxg.w8a16_gemm(h, hw, 1024, N))
    check_tokens = [pick(logits[m, :V].float().cpu().numpy(), u[m].item(), temp[m].item(), 40,
                         p[m].item(), 0.0)[0] for m in range(M)]
    assert tokens.tolist() == check_tokens
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gs = step()
    graph.replay()
    assert torch.equal(gh, h) and torch.equal(gs[0], tokens) and torch.equal(gs[1], probs)
