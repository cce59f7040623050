"""Long runs through the weight-streaming kernel's ring, right behind a re-pack
into a buffer in use: the weights lie partly in L2 and the copies of a ring's
stages land out of order.  Every output of every call, against 64 bits and,
bit for bit, against the first call on the same weights."""
import pytest
import torch

from helpers import ELEM_TOL, FROB_TOL
from test_gpu_sample import pick

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
G = 128


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_gemm_speculative_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def words(rows, cols, seed):
    return torch.randint(-2 ** 31, 2 ** 31, (rows, cols), generator=gen(seed), device=DEV,
                         dtype=torch.int64).int()


def scales(K, N, seed, unit):
    z = torch.randn(K // G, N, generator=gen(seed), device=DEV).abs_()
    return (unit * (0.1 + z)).half()


def codes_times_scales(qweight, sc, bits):
    """GPTQ words [K * bits / 32][N] and scales [K / G][N] -> fp64 [K][N]."""
    per = 32 // bits
    shift = torch.arange(0, 32, bits, device=DEV, dtype=torch.int32)[None, :, None]
    q = (qweight[:, None, :] >> shift) & (2 ** bits - 1)
    q = q.reshape(qweight.shape[0] * per, -1).double() - 2 ** (bits - 1)
    return q * sc.double().repeat_interleave(G, 0)


def near(y, ref, what):
    """The parity criteria of the layer, on the device."""
    err, rms = (y.double() - ref).abs(), ref.square().mean().sqrt()
    assert (err.square().sum() / ref.square().sum()).sqrt() <= FROB_TOL, what
    bad = err > ELEM_TOL * (ref.abs() + rms)
    cols = bad.any(0).nonzero()[:, 0]
    assert not len(cols), f"{what}: {len(cols)} wrong columns, from {int(cols[0])} on"


def repeat(mxg, layers, repack, gemm, M, N, rounds, what):
    """layers: (words, scales, fp64 reference of every output)."""
    first = [None] * len(layers)
    packed = None
    for i in range(rounds * len(layers)):
        qw, sc, ref = layers[i % len(layers)]
        packed = None            # the next one takes the same memory
        packed = repack(qw, sc)
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        gemm(packed, y)
        if first[i % len(layers)] is None:
            near(y, ref, f"{what}, call {i}")
            first[i % len(layers)] = y
        diff = (y != first[i % len(layers)]).any(0).nonzero()[:, 0]
        assert not len(diff), f"{what}, call {i}: {len(diff)} columns differ, from {int(diff[0])} on"
    return packed, first[(rounds * len(layers) - 1) % len(layers)]


def activations(M, K, seed):
    return torch.randn(M, K, generator=gen(seed), device=DEV).bfloat16()


@pytest.mark.parametrize("M", [1, 5, 16])
def test_int8_head_behind_repacks(mxg, M):
    K, N = 5120, 248320
    x = activations(M, K, M)
    layers = []
    for seed in (1, 2):
        qw, sc = words(K // 4, N, seed), scales(K, N, seed, 1e-3)
        ref = torch.cat([x.double() @ codes_times_scales(qw[:, n:n + 16384], sc[:, n:n + 16384], 8)
                         for n in range(0, N, 16384)], 1)
        layers.append((qw, sc, ref))
    packed, y = repeat(mxg, layers, lambda qw, sc: mxg.w8a16_repack(qw, sc, G),
                       lambda p, out: mxg.w8a16_gemm(x, p, N, K, G, out=out), M, N, 30,
                       f"int8 head, M = {M}")
    # and the tokens of the logits that have been looked at
    u = torch.rand(M, generator=gen(3), device=DEV)
    p = torch.full((M,), 0.9, device=DEV)
    tokens, _, logits = mxg.w8a16_gemm_sample(x, packed, N, K, u, top_p=p)
    assert torch.equal(logits, y)
    rows = y.float().cpu().numpy()
    for m in range(M):
        assert tokens[m].item() == pick(rows[m], u[m].item(), 1.0, 0, p[m].item(), 0.0)[0]


@pytest.mark.parametrize("M,K,N", [(5, 5120, 10240), (16, 5120, 17408), (16, 17408, 5120),
                                   (9, 5120, 5120), (5, 5120, 34816)])
def test_int4_layers_behind_repacks(mxg, M, K, N):
    x = activations(M, K, M)
    layers = []
    for seed in (1, 2):
        qw, sc = words(K // 8, N, seed), scales(K, N, seed, 1e-2)
        layers.append((qw, sc, x.double() @ codes_times_scales(qw, sc, 4)))
    repeat(mxg, layers, lambda qw, sc: mxg.w4a16_repack(qw, sc, G),
           lambda p, out: mxg.w4a16_gemm(x, p, N, K, G, out=out), M, N, 30,
           f"int4, M = {M}, {K} -> {N}")


@pytest.mark.parametrize("M,K,N", [(1, 5120, 17408), (5, 5120, 17408), (16, 5120, 5120)])
def test_mxfp8_layers_behind_repacks(mxg, M, K, N):
    x = activations(M, K, M)
    layers = []
    for seed in (1, 2):
        wq = torch.randint(0, 256, (N, K), generator=gen(seed), device=DEV, dtype=torch.uint8)
        wq[(wq & 0x7F) == 0x7F] = 0          # the two NaN codes
        ws = torch.randint(118, 124, (N, K // 32), generator=gen(seed), device=DEV,
                           dtype=torch.uint8)
        w = wq.view(torch.float8_e4m3fn).double() * torch.exp2(
            ws.double() - 127).repeat_interleave(32, 1)
        layers.append((wq, ws, x.double() @ w.T))
    repeat(mxg, layers, mxg.mxfp8_repack,
           lambda p, out: mxg.mxfp8_gemm_packed(x, p, N, K, out=out), M, N, 30,
           f"mxfp8, M = {M}, {K} -> {N}")
