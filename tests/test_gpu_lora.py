"""GPU parity of the low-rank adapters of many requests (lora_add) against
the formula in 64 bits, through the binding.

Tolerance, from the arithmetic: with mag = s (|x| |A|^T) |B|^T and
dmag = s |x A^T| |B|^T,
  - the result is rounded once to bf16: 2^-8 |out|;
  - a tensor-core step adds 16 products to an fp32 sum, within 2^-22 of the
    largest magnitude in it; a sum of K products takes at most K / 128 + 16
    such steps and additions, one of R products R / 8 + 2:
    (K / 128 + R / 8 + 18) 2^-22 mag;
  - an inner product is kept as two bf16 halves: 2^-16 dmag.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_gemm_speculative_b200 as m
    return m


def case(M, K, N, R, L, seed=0, index=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)
    x = randn(M, K).bfloat16()
    a = (randn(L, R, K) * K ** -0.5).bfloat16()
    b = (randn(L, N, R) * R ** -0.5).bfloat16()
    y = randn(M, N).bfloat16()
    s = torch.rand(L, generator=g, device=DEV) + 0.5
    if index is None:
        index = torch.randint(-1, L, (M,), generator=g, device=DEV)
    return x, a, b, index.to(torch.int32).to(DEV), y, s


def reference(x, a, b, index, y, s):
    """(out, bound) in 64 bits."""
    K, R = a.shape[2], a.shape[1]
    out, bound = y.double(), torch.zeros_like(y, dtype=torch.float64)
    for i in range(a.shape[0]):
        rows = (index == i).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        xd, ad, bd = x[rows].double(), a[i].double(), b[i].double()
        si = 1.0 if s is None else float(s[i].double())
        inner = xd @ ad.T
        out[rows] += si * (inner @ bd.T)
        mag = abs(si) * ((xd.abs() @ ad.abs().T) @ bd.abs().T)
        dmag = abs(si) * (inner.abs() @ bd.abs().T)
        bound[rows] = (K / 128 + R / 8 + 18) * 2.0 ** -22 * mag + 2.0 ** -16 * dmag
    return out, bound + 2.0 ** -8 * out.abs()


def check(got, x, a, b, index, y, s):
    ref, bound = reference(x, a, b, index, y, s)
    worst = ((got.double() - ref).abs() / bound.clamp(min=1e-300)).max()
    assert got.isfinite().all()
    assert worst <= 1.0, f"an element exceeds its bound by x{float(worst):.2f}"
    bare = (index < 0) | (index >= a.shape[0])
    assert torch.equal(got[bare], y[bare])     # no adapter: y itself


@pytest.mark.parametrize("M", [1, 2, 5, 7, 8, 9, 16, 33, 63, 64, 65, 130, 257])
@pytest.mark.parametrize("K,N,R,L", [(512, 512, 16, 4), (1032, 200, 8, 3), (72, 1288, 40, 6),
                                     (5120, 96, 64, 2), (256, 320, 128, 5)])
def test_lora_parity(mxg, M, K, N, R, L):
    x, a, b, index, y, s = case(M, K, N, R, L, seed=M + K + N + R)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 48, 56, 64, 72, 88, 96, 104, 112, 120, 128])
def test_lora_every_rank(mxg, R):
    x, a, b, index, y, s = case(37, 776, 264, R, 3, seed=R)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)


@pytest.mark.parametrize("K,N", [(8, 8), (8, 17408), (17408, 8), (24, 40), (40, 24), (520, 136),
                                 (5120, 17408), (17408, 5120)])
@pytest.mark.parametrize("M", [1, 70])
def test_lora_sizes(mxg, M, K, N):
    x, a, b, index, y, s = case(M, K, N, 16, 5, seed=K + N)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)


@pytest.mark.parametrize("pattern", ["one", "none", "all_apart", "halves", "out_of_range", "runs",
                                     "last_token"])
@pytest.mark.parametrize("M", [1, 64, 200])
@pytest.mark.parametrize("R", [8, 32, 64])
def test_lora_index_patterns(mxg, pattern, M, R):
    L = max(M, 4)
    i = torch.arange(M)
    index = {"one": torch.full((M,), 2), "none": torch.full((M,), -1), "all_apart": L - 1 - i,
             "halves": i % 2, "out_of_range": torch.tensor([-2 ** 31, 2 ** 31 - 1, L, 0])[i % 4],
             "runs": (i // 7) % 3 - 1, "last_token": torch.where(i == M - 1, 1, -1)}[pattern]
    x, a, b, index, y, s = case(M, 264, 328, R, L, seed=M + R, index=index)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)


def test_lora_prefill_chunk(mxg):
    M, L = 8192, 8
    index = torch.arange(M) // 700 % (L + 1) - 1
    x, a, b, index, y, s = case(M, 640, 1032, 16, L, seed=1, index=index)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)


def test_lora_without_scales_equals_ones(mxg):
    x, a, b, index, y, s = case(9, 512, 512, 16, 3)
    one = torch.ones_like(s)
    assert torch.equal(mxg.lora_add(x, a, b, index, y),
                       mxg.lora_add(x, a, b, index, y, scales=one))
    check(mxg.lora_add(x, a, b, index, y), x, a, b, index, y, None)


@pytest.mark.parametrize("M", [1, 5, 100])
def test_lora_exact_integers(mxg, M):
    """Small integers: every product and sum is exact, so the result is the
    bf16 nearest the exact one, bit for bit."""
    g = torch.Generator().manual_seed(M)
    L, R, K, N = 3, 24, 264, 136

    def ints(n, *shape):
        return torch.randint(-n, n + 1, shape, generator=g).to(DEV)
    x, a, b = ints(2, M, K), ints(1, L, R, K), ints(2, L, N, R)
    y, index = ints(100, M, N), torch.randint(-1, L, (M,), generator=g).to(DEV, torch.int32)
    s = torch.tensor([0.5, 2.0, 4.0], device=DEV)
    want = y.double()
    for i in range(L):
        r = index == i
        want[r] += float(s[i]) * ((x[r].double() @ a[i].double().T) @ b[i].double().T)
    got = mxg.lora_add(x.bfloat16(), a.bfloat16(), b.bfloat16(), index, y.bfloat16(), scales=s)
    assert torch.equal(got, want.float().bfloat16())


@pytest.mark.parametrize("M", [1, 6, 90])
def test_lora_in_place_and_column_ranges(mxg, M):
    """In place on a column range of a fused projection's output, x a column
    range too: the columns beside it and the rows behind stay as they were."""
    x, a, b, index, y, s = case(M, 512, 256, 16, 4, seed=M)
    want = mxg.lora_add(x, a, b, index, y, scales=s)
    fused = torch.randn(M + 2, 800, device=DEV).bfloat16()
    fused[:M, 264:520] = y
    before = fused.clone()
    wide = torch.zeros(M, 1024, device=DEV, dtype=torch.bfloat16)
    wide[:, 128:640] = x
    part = fused[:M, 264:520]
    assert mxg.lora_add(wide[:, 128:640], a, b, index, part, scales=s, out=part) is part
    assert torch.equal(part, want)
    before[:M, 264:520] = want
    assert torch.equal(fused, before)
    # from one column range to another of the same buffer
    fused[:M, 264:520] = y
    mxg.lora_add(x, a, b, index, fused[:M, 264:520], scales=s, out=fused[:M, 520:776])
    assert torch.equal(fused[:M, 520:776], want) and torch.equal(fused[:M, 264:520], y)


def test_lora_reproducible_and_order_of_tokens(mxg):
    """The same bits every time, and a token's result does not depend on its
    place in the batch."""
    x, a, b, index, y, s = case(150, 1024, 512, 32, 7, seed=3)
    one = mxg.lora_add(x, a, b, index, y, scales=s)
    for _ in range(20):
        assert torch.equal(mxg.lora_add(x, a, b, index, y, scales=s), one)
    p = torch.randperm(150, device=DEV)
    again = mxg.lora_add(x[p].contiguous(), a, b, index[p].contiguous(), y[p].contiguous(),
                         scales=s)
    assert torch.equal(again, one[p])


def test_lora_non_finite_activations_stay_in_their_rows(mxg):
    x, a, b, index, y, s = case(70, 256, 256, 16, 2, seed=4, index=torch.arange(70) % 3 - 1)
    clean = mxg.lora_add(x, a, b, index, y, scales=s)
    x = x.clone()
    x[4, 7], x[35, 0], x[3, 1] = float("inf"), float("nan"), float("nan")   # row 3: no adapter
    got = mxg.lora_add(x, a, b, index, y, scales=s)
    others = torch.ones(70, dtype=torch.bool, device=DEV)
    others[[4, 35]] = False
    assert torch.equal(got[others], clean[others])
    assert not got[35].isfinite().any() and not got[4].isfinite().any()


def test_lora_streams_and_graphs(mxg):
    """Another stream than the current one; two captured graphs replayed in
    turn and at once, on inputs that changed since the capture."""
    cases = [case(5, 2048, 1024, 16, 4, seed=i) for i in (10, 11)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxg.lora_add(*cases[0][:5], scales=cases[0][5], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(got, *cases[0])
    graphs, outs = [], []
    for x, a, b, index, y, s in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t = mxg.lora_add(x, a, b, index, y, scales=s)
            outs.append(mxg.lora_add(x, a, b, index, t, scales=s))   # a second one behind it
        graphs.append(graph)
    for x, a, b, index, y, s in cases:
        x.copy_(torch.randn_like(x.float()).bfloat16())
        index.copy_(torch.randint(-1, 4, (5,), device=DEV).int())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        x, a, b, index, y, s = c
        mid = mxg.lora_add(x, a, b, index, y, scales=s)
        assert torch.equal(out, mxg.lora_add(x, a, b, index, mid, scales=s))


def test_lora_behind_a_kernel_that_writes_its_inputs(mxg):
    """Adapters, index and y written by the kernel right before the call."""
    x, a, b, index, y, s = case(33, 1024, 640, 16, 6, seed=8)
    want = mxg.lora_add(x, a, b, index, y, scales=s)
    a2, b2, i2, y2 = (torch.zeros_like(t) for t in (a, b, index, y))
    for last in range(4):
        for t in (a2, b2, i2, y2):
            t.zero_()
        order = [(a2, a), (b2, b), (i2, index), (y2, y)]
        for dst, src in order[:last] + order[last + 1:] + [order[last]]:
            dst.copy_(src)
        assert torch.equal(mxg.lora_add(x, a2, b2, i2, y2, scales=s), want)
        i2.fill_(-1)      # and changed right behind it


def test_lora_prepared_call(mxg):
    x, a, b, index, y, s = case(12, 512, 512, 16, 3)
    call, out = mxg.prepare_lora_add(x, a, b, index, y, scales=s)
    call()
    check(out, x, a, b, index, y, s)
    x.copy_(torch.flip(x, [0]))
    call()
    check(out, x, a, b, index, y, s)


@pytest.mark.parametrize("R", [16, 32, 64, 128])
@pytest.mark.parametrize("M,K,N,L", [(700, 520, 8712, 150),     # many parts per CTA, few CTAs a tile
                                     (64, 4104, 264, 80),       # several groups per cluster of eight
                                     (200, 4096, 512, 3)])      # groups above 16 tokens, scattered
def test_lora_scattered_batches(mxg, M, K, N, L, R):
    x, a, b, index, y, s = case(M, K, N, R, L, seed=M + R)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)
    y2 = y.clone()
    assert torch.equal(mxg.lora_add(x, a, b, index, y2, scales=s, out=y2),
                       mxg.lora_add(x, a, b, index, y, scales=s))


@pytest.mark.parametrize("R", [16, 64])
def test_lora_runs_at_every_offset(mxg, R):
    """Runs of one adapter that start and end anywhere in the blocks, some as
    long as a box of 16 tokens, between tokens without an adapter."""
    lengths = [16, 1, 17, 15, 64, 3, 33, 48, 16, 32, 31, 70, 16, 5, 128]
    index = torch.cat([torch.full((n,), i % 4 - 1) for i, n in enumerate(lengths)])
    x, a, b, index, y, s = case(len(index), 328, 520, R, 3, seed=R, index=index)
    check(mxg.lora_add(x, a, b, index, y, scales=s), x, a, b, index, y, s)


def test_lora_workspace_and_status_word(mxg):
    """A workspace of the caller's, full of anything; its status word is
    cleared; a workspace that is too small is refused before a launch."""
    x, a, b, index, y, s = case(40, 512, 256, 24, 4, seed=6)
    need = mxg.lora_workspace_bytes(40, 256, 512, 24)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    got = mxg.lora_add(x, a, b, index, y, scales=s, workspace_buf=ws)
    check(got, x, a, b, index, y, s)
    assert mxg.mxg_workspace_status(ws) == 0
    assert (ws[need:] == 0x5A).all()
    with pytest.raises(mxg.MxgError):
        mxg.lora_add(x, a, b, index, y, workspace_buf=ws[: need - 16])


def test_lora_calls_at_once_on_two_streams(mxg):
    cases = [case(33, 2048, 2048, 16, 8, seed=i) for i in (20, 21)]
    want = [mxg.lora_add(*c[:5], scales=c[5]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [mxg.lora_add(*c[:5], scales=c[5], stream=st) for c, st in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("share", [1, 3, 4, 5, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("R", [8, 32, 64, 128])
def test_lora_scattered_groups_of_every_size(mxg, share, R):
    """`share` tokens of every 64 have the first adapter, the others the second
    or none, in any order: rows in fours, with some left over, of column ranges
    whose neighbours hold NaN."""
    M, K, N = 147, 200, 312
    g = torch.Generator(device=DEV)
    g.manual_seed(share)
    index = torch.cat([torch.where(torch.randperm(64, generator=g, device=DEV) < share, 0, i % 2 * 2 - 1)
                       for i in range(3)])[:M]
    x, a, b, index, y, s = case(M, K, N, R, 2, seed=R, index=index)
    wide_x = torch.full((M, K + 24), float("nan"), device=DEV).bfloat16()
    wide_y = torch.full((M, N + 40), float("nan"), device=DEV).bfloat16()
    wide_x[:, 16:16 + K] = x
    wide_y[:, 8:8 + N] = y
    got = mxg.lora_add(wide_x[:, 16:16 + K], a, b, index, wide_y[:, 8:8 + N], scales=s)
    check(got, x, a, b, index, y, s)
    # by themselves, in a run of rows: the same bits
    mine = (index == 0).nonzero()[:, 0]
    alone = mxg.lora_add(x[mine].contiguous(), a, b, index[mine].contiguous(),
                         y[mine].contiguous(), scales=s)
    assert torch.equal(alone, got[mine])
