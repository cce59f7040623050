"""The ring of the weight-streaming kernel, from the host's plan (no GPU).

Two warps take a tile's stages in turn.  A warp's wait for a filling of a slot
names the filling's parity only, and ends at once while the filling before it
is still on its way, unless the warp has waited for that one itself: every
filling of a slot has to go to the same warp, so whole turns have to go round
the ring."""
import ctypes

import pytest

SIZES = [64, 192, 512, 1024, 2048, 4096, 5120, 6144, 8192, 10240, 14336, 17408, 34816]


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_gemm_speculative_b200 as m
    return m


def rings(mxg, bits, Ns, Ks, sms):
    for G in (128, 64, 32) if bits else (64,):
        for M in (1, 5, 8, 9, 16, 17, 24, 25, 32):
            for K in Ks:
                for N in Ns:
                    if K % G or (bits == 0 and (M > 16 or N < 128)):
                        continue
                    try:
                        yield (G, M, K, N), mxg.mxg_selftest_stream_ring(bits, M, N, K, G, sms=sms)
                    except mxg.MxgError as e:
                        # re-packed MXFP8 takes resident activations only
                        assert bits == 0 and e.status == mxg.MXG_ERR_UNSUPPORTED_SHAPE, (G, M, K, N)


@pytest.mark.parametrize("sms", [148, 132, 1])
@pytest.mark.parametrize("bits", [4, 8, 0])
def test_whole_turns_go_round_the_ring(mxg, bits, sms):
    seen = set()
    for what, (stages, turns) in rings(mxg, bits, SIZES + [128256, 151936, 248320], SIZES, sms):
        assert turns == (2 if what[1] <= 16 else 1), what
        assert stages % turns == 0 and stages >= 2 * turns, (what, stages, turns)
        seen.add(stages)
    assert seen


def test_the_measured_layers(mxg):
    """(bits, M, K, N): stages.  As many as fit would be five for the head,
    seven and eleven for the first two INT4 layers, five for MXFP8."""
    for (bits, M, K, N), stages in {(8, 5, 5120, 248320): 4, (4, 16, 5120, 17408): 6,
                                    (4, 5, 5120, 10240): 10, (4, 5, 5120, 17408): 10,
                                    (0, 5, 5120, 17408): 4}.items():
        assert mxg.mxg_selftest_stream_ring(bits, M, N, K)[0] == stages, (bits, M, K, N)


def test_refusals(mxg):
    lib = mxg.raw_lib()
    a, b = ctypes.c_int(0), ctypes.c_int(0)

    def call(bits=4, M=5, N=512, K=512, G=128, sms=148, smem=227 * 1024, stages=a, turns=b):
        return lib.mxg_selftest_stream_ring(bits, M, N, K, G, sms, smem,
                                            None if stages is None else ctypes.byref(stages),
                                            None if turns is None else ctypes.byref(turns))
    assert call() == 0 and a.value % b.value == 0
    for bad in (dict(bits=5), dict(bits=-1), dict(sms=0), dict(smem=0), dict(stages=None),
                dict(turns=None)):
        assert call(**bad) == mxg.MXG_ERR_INVALID_ARG, bad
    for bad in (dict(M=0), dict(M=33), dict(N=96), dict(N=0), dict(K=0), dict(K=100), dict(G=96),
                dict(bits=0, M=17), dict(bits=0, K=0), dict(bits=0, N=0), dict(smem=1024)):
        assert call(**bad) == mxg.MXG_ERR_UNSUPPORTED_SHAPE, bad
