"""lora_add where its parts meet: formula, tolerance and helpers are those of
test_gpu_lora.py."""
import pytest
import torch

from test_gpu_lora import DEV, case, check, mxg  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [16, 32, 64, 128])
@pytest.mark.parametrize("sizes", [(5, 20, 3, 17, 1, 18), (20, 5, 39), (1, 63), (40, 1, 23),
                                   (16, 17, 16, 15)])
def test_lora_groups_of_few_and_of_many_tokens_in_turn(mxg, sizes, R):
    """So many blocks that a cluster takes several of a block's groups: their
    activations come by 16-byte copies (up to 16 tokens) and by boxes or
    gathers (more), one behind the other through the same slots."""
    M, K, N, L = 1024, 4104, 136, 7
    g = torch.Generator().manual_seed(len(sizes) + R)
    one = torch.cat([torch.full((n,), i) for i, n in enumerate(sizes)])
    for order in ("runs", "scattered"):
        index = torch.cat([(one if order == "runs" else one[torch.randperm(64, generator=g)])
                           for _ in range(M // 64)])
        x, a, b, index, y, s = case(M, K, N, R, L, seed=R, index=index)
        want = mxg.lora_add(x, a, b, index, y, scales=s)
        check(want, x, a, b, index, y, s)
        for _ in range(5):
            assert torch.equal(mxg.lora_add(x, a, b, index, y, scales=s), want)


def one_adapter(a, b, x, y, N=40):
    """lora_add of one adapter with the given ranks' weights: x [M][8], a
    [R][8], b [R] and y [M] the same in every column."""
    M = len(x)

    def dev(v):
        return torch.tensor(v, dtype=torch.float64, device=DEV).bfloat16()
    bb = dev(b)[None, None, :].expand(1, N, len(b)).contiguous()
    return (dev(x), dev(a)[None], bb, torch.zeros(M, dtype=torch.int32, device=DEV),
            dev(y)[:, None].expand(M, N).contiguous())


@pytest.mark.parametrize("M", [1, 9, 20])
def test_lora_inner_products_keep_24_bits(mxg, M):
    """Two ranks that cancel but for the last bits of an inner product: every
    product and sum of the formula is exact, and so is the result."""
    R = 8
    for e in range(10, 24):
        # out = 2 (1 + 2^-9 + 2^-e) - 2 (1 + 2^-9)
        x = [[1.0, 2.0 ** -9, 2.0 ** -e, 0, 0, 0, 0, 0]] * M
        a = [[0.0] * 8 for _ in range(R)]
        a[0] = [1.0, 1.0, 1.0, 0, 0, 0, 0, 0]
        a[5] = [1.0, 1.0, 0.0, 0, 0, 0, 0, 0]
        b = [2.0, 0, 0, 0, 0, -2.0, 0, 0]
        got = mxg.lora_add(*one_adapter(a, b, x, [0.0] * M))
        assert (got.double() == 2.0 ** (1 - e)).all(), e


@pytest.mark.parametrize("M", [1, 20, 70])
def test_lora_infinite_inner_products(mxg, M):
    """An infinity in x: the row's products are infinities of the factors'
    signs, NaN where a zero meets it; the other rows keep their bits."""
    inf = float("inf")
    x, a, b, index, y, s = case(M, 72, 96, 24, 1, seed=M, index=torch.zeros(M))
    clean = mxg.lora_add(x, a, b, index, y, scales=s)
    row = M // 2
    for value in (inf, -inf, float("nan")):
        x2 = x.clone()
        x2[row] = 0.0
        x2[row, 5] = value
        a2 = a.clone()
        a2[0, :, 5] = 0.0                    # T = NaN in every rank ...
        got = mxg.lora_add(x2, a2, b, index, y, scales=s)
        assert got[row].isnan().all()
        a2[0, :, 5] = 1.0                    # ... and +-inf in every rank
        b2 = b.abs() + 1.0
        got = mxg.lora_add(x2, a2, b2, index, y, scales=s)
        want = torch.full_like(y[row], value)
        assert torch.equal(got[row].isnan(), want.isnan())
        assert value != value or torch.equal(got[row], want)
        b2[0, 3, 7] = -1.0                   # one of the other sign: inf - inf
        got = mxg.lora_add(x2, a2, b2, index, y, scales=s)
        assert got[row, 3].isnan() and (value != value or torch.equal(got[row, 4:], want[4:]))
        others = torch.arange(M, device=DEV) != row
        got = mxg.lora_add(x2, a, b, index, y, scales=s)
        assert torch.equal(got[others], clean[others])


@pytest.mark.parametrize("R", [8, 16, 40, 64, 128])
@pytest.mark.parametrize("M", [1, 20, 70])
def test_lora_infinite_weights(mxg, M, R):
    """Infinities and NaN in one adapter's B: what 64 bits make of them, in its
    column and its adapter's tokens; every other output keeps its bits.  The
    last column tile has fewer columns than a full one."""
    inf, nan = float("inf"), float("nan")
    x, a, b, index, y, s = case(M, 72, 296, R, 2, seed=M + R, index=torch.arange(M) % 2)
    clean = mxg.lora_add(x, a, b, index, y, scales=s)
    b2 = b.clone()
    b2[0, 5, 3], b2[0, 6, R - 1], b2[0, 7, 0] = inf, -inf, nan
    b2[0, 260, 1], b2[0, 260, 4] = inf, -inf          # either inf, -inf or, of unlike signs, NaN
    got = mxg.lora_add(x, a, b2, index, y, scales=s)
    cols = [5, 6, 7, 260]
    mine = index == 0
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[mine.nonzero(), torch.tensor(cols, device=DEV)] = False
    assert torch.equal(got[keep], clean[keep])
    inner = x[mine].double() @ a[0].double().T
    want = torch.stack([y[mine, c].double() + float(s[0]) * (inner * b2[0, c].double()).sum(1)
                        for c in cols], 1)
    have = got[mine][:, cols].double()
    assert not want.isfinite().any() and torch.equal(have.isnan(), want.isnan())
    assert torch.equal(have[~have.isnan()], want[~want.isnan()])


def test_lora_infinite_weights_and_zeros(mxg):
    """Infinity times an inner product of 0 is NaN, times one of 2^-140 it is
    an infinity; an infinite product stays one whatever the last bits of the
    inner product (1 - 2^-9 + 2^-20: parts of either sign)."""
    inf = float("inf")
    a = [[0.0] * 8 for _ in range(8)]
    a[2] = [1.0, -1.0, 1.0, 2.0 ** -70, 0, 0, 0, 0]
    for row, sign in (([0.0] * 8, 0), ([0, 0, 0, 2.0 ** -70, 0, 0, 0, 0], 1),
                      ([0, 0, 0, -2.0 ** -70, 0, 0, 0, 0], -1),
                      ([1.0, 2.0 ** -9, 2.0 ** -20, 0, 0, 0, 0, 0], 1),
                      ([-1.0, -2.0 ** -9, 2.0 ** -20, 0, 0, 0, 0, 0], -1),
                      ([2.0 ** 127, 0, 0, 0, 0, 0, 0, 0], 1), ([-1.0, 0, 0, 0, 0, 0, 0, 0], -1)):
        b = [0.0, 0, inf, 0, 0, 0, 0, 0]
        got = mxg.lora_add(*one_adapter(a, b, [row], [3.0]))
        if sign == 0:
            assert got.isnan().all(), row
        else:
            assert (got == sign * inf).all(), row


def test_lora_largest_inner_products(mxg):
    """An inner product above the largest bf16 (and in fp32) times a small
    weight is finite."""
    a = [[0.0] * 8 for _ in range(8)]
    a[1] = [1.0, 1.0, 0, 0, 0, 0, 0, 0]
    x = [[255 * 2.0 ** 120, 2.0 ** 119, 0, 0, 0, 0, 0, 0]]     # above 255 2^120, the largest bf16
    got = mxg.lora_add(*one_adapter(a, [0, 2.0 ** -127, 0, 0, 0, 0, 0, 0], x, [0.0]))
    assert (got.double() == 2.0).all()       # 255.5 / 128 rounds to 2
