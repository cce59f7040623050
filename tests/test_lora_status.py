"""lora_status: what it refuses before it touches a device, what the binding
passes on, and (on the GPU) a recorded wait that ran out."""
import ctypes

import pytest
import torch

from test_binding_marshal import fake as fake_lib  # noqa: F401  (fixture)


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_gemm_speculative_b200 as m
    return m


def test_refusals(mxg):
    lib = mxg.raw_lib()
    v = ctypes.c_int(7)
    for args in ((None, 0, None), (ctypes.byref(v), 2, None), (ctypes.byref(v), -1, None)):
        assert lib.lora_status(*args) == mxg.MXG_ERR_INVALID_ARG
    for limit in (0, -1, 10000001):
        assert lib.mxg_selftest_lora_wait_timeout(limit, None) == mxg.MXG_ERR_INVALID_ARG
    assert v.value == 7


def test_binding(fake_lib, monkeypatch):  # noqa: F811
    m, lib = fake_lib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_raw_device", None)      # no driver here
    assert m.lora_status() == 0 and m.lora_status(reset=True, device="cuda:0") == 0
    assert [(c[0], c[1][1]) for c in lib.calls[-2:]] == [("lora_status", 0), ("lora_status", 1)]


@pytest.mark.gpu
def test_a_wait_that_ran_out_is_reported(mxg):
    dev = torch.device("cuda", 0)
    assert mxg.lora_status(reset=True) == 0
    mxg.mxg_selftest_lora_wait_timeout(2000)        # 2 ms limit on a wait nothing ends
    assert mxg.lora_status() == mxg.MXG_ERR_TIMEOUT
    # a call clears its own workspace's word, not this one
    x, a, b = (torch.ones(s, device=dev).bfloat16() for s in ((3, 64), (1, 8, 64), (1, 40, 8)))
    index, y = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(3, 40, device=dev).bfloat16()
    out = mxg.lora_add(x, a, b, index, y)
    assert (out == 512).all()
    side = torch.cuda.Stream()
    assert mxg.lora_status(stream=side) == mxg.MXG_ERR_TIMEOUT
    assert mxg.lora_status(reset=True) == mxg.MXG_ERR_TIMEOUT
    assert mxg.lora_status() == 0
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = mxg.lora_add(x, a, b, index, y)
            with pytest.raises(mxg.MxgError) as e:
                mxg.lora_status()
        assert e.value.status == mxg.MXG_ERR_CAPTURE
        out.zero_()
        graph.replay()
    side.synchronize()
    assert (out == 512).all() and mxg.lora_status() == 0
