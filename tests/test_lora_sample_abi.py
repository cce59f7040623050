"""lora_add and sample_logits without a GPU: what the C ABI refuses before
any launch, what the binding refuses before the C call, and the arguments it
passes on."""
import ctypes

import pytest
import torch

from test_binding_marshal import _val, bf16, fake as fake_lib  # noqa: F401  (fixture)



@pytest.fixture()
def fake(fake_lib, monkeypatch):  # noqa: F811
    """The recording library, with CPU tensors let through."""
    monkeypatch.setattr(fake_lib[0], "_need_cuda", lambda t, name: None)
    return fake_lib


P = ctypes.c_void_p
OK, INVALID, SHAPE, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp8_gemm_speculative_b200 as m
    return m.raw_lib()


def lora(lib, **kw):
    # aligned, never dereferenced on these paths
    a = dict(X=4096, ldx=512, A=8192, B=8192, scales=None, index=4096, Y=65536, ldy=256,
             Out=1 << 20, ldo=256, M=4, N=256, K=512, R=16, L=2, ws=4096, bytes=0)
    a.update(kw)
    return lib.lora_add(P(a["X"]), a["ldx"], P(a["A"]), P(a["B"]), P(a["scales"]), P(a["index"]),
                        P(a["Y"]), a["ldy"], P(a["Out"]), a["ldo"], a["M"], a["N"], a["K"], a["R"],
                        a["L"], P(a["ws"]), a["bytes"], None)


def test_lora_refusals(lib):
    assert lora(lib) == WORKSPACE                  # everything else is in order
    for name in ("X", "A", "B", "index", "Y", "Out", "ws"):
        assert lora(lib, **{name: None}) == INVALID, name
        assert lora(lib, **{name: 4098}) == INVALID, name
    assert lora(lib, index=4100) == WORKSPACE      # 4-byte aligned is enough
    assert lora(lib, scales=4100) == WORKSPACE
    assert lora(lib, scales=4098) == INVALID
    for bad in (dict(M=0), dict(M=-1), dict(L=0), dict(ldx=504), dict(ldy=248), dict(ldo=248),
                dict(ldx=516), dict(ldy=260), dict(ldo=260), dict(ldy=0), dict(ldy=-256),
                dict(Out=65536, ldo=512)):
        assert lora(lib, **bad) == INVALID, bad
    assert lora(lib, Out=65536) == WORKSPACE       # in place
    for bad in (dict(R=0), dict(R=4), dict(R=12), dict(R=136), dict(N=0, ldy=256), dict(N=252),
                dict(K=508), dict(K=0), dict(M=2097089), dict(K=-8), dict(N=-8)):
        assert lora(lib, **bad) == SHAPE, bad
    assert lora(lib, bytes=256 + 4 * 16 * 4 - 1) == WORKSPACE
    assert lib.lora_workspace_bytes(4, 256, 512, 16) == 256 + 4 * 16 * 4
    assert lib.lora_workspace_bytes(2097088, 8, 8, 128) == 256 + 2097088 * 512
    for bad in ((0, 256, 512, 16), (4, 250, 512, 16), (4, 256, 511, 16), (4, 256, 512, 15),
                (4, 256, 512, 256)):
        assert lib.lora_workspace_bytes(*bad) == 0


def sample(lib, **kw):
    a = dict(logits=4098, dtype=0, ld=100, M=2, V=100, u=4100, t=None, k=None, p=None, q=None,
             tokens=4100, probs=None)
    a.update(kw)
    return lib.sample_logits(P(a["logits"]), a["dtype"], a["ld"], a["M"], a["V"], P(a["u"]),
                             P(a["t"]), P(a["k"]), P(a["p"]), P(a["q"]), P(a["tokens"]),
                             P(a["probs"]), None)


def test_sample_refusals(lib):
    for bad in (dict(logits=None), dict(logits=4097), dict(dtype=1), dict(dtype=2), dict(dtype=-1),
                dict(ld=99), dict(ld=-100), dict(M=0), dict(u=None), dict(u=4098),
                dict(tokens=None), dict(tokens=4097), dict(t=4098), dict(k=4098), dict(p=4098),
                dict(q=4098), dict(probs=4098)):
        assert sample(lib, **bad) == INVALID, bad
    for bad in (dict(V=0), dict(V=-5), dict(V=393217, ld=393217), dict(M=(1 << 27) + 1)):
        assert sample(lib, **bad) == SHAPE, bad


def test_lora_binding(fake):
    m, lib = fake
    x, a, b, y = bf16(3, 64), bf16(2, 16, 64), bf16(2, 40, 16), bf16(3, 40)
    index, s = torch.zeros(3, dtype=torch.int32), torch.ones(2)
    out = m.lora_add(x, a, b, index, y, scales=s)
    name, args = lib.calls[-1]
    assert name == "lora_add" and out.shape == (3, 40) and out.dtype == torch.bfloat16
    got = [_val(v) for v in args[:-1]]
    assert got[:15] == [x.data_ptr(), 64, a.data_ptr(), b.data_ptr(), s.data_ptr(),
                        index.data_ptr(), y.data_ptr(), 40, out.data_ptr(), 40, 3, 40, 64, 16, 2]
    assert got[16] == 256 + 3 * 16 * 4 and args[-1] == ("stream", None, x.device)
    # in place, on a column range
    wide = bf16(3, 128)
    part = wide[:, 40:80]
    assert m.lora_add(x, a, b, index, part, out=part) is part
    got = [_val(v) for v in lib.calls[-1][1]]
    assert got[4] is None and got[6] == got[8] == part.data_ptr() and got[7] == got[9] == 128
    # side by side in one buffer
    m.lora_add(x, a, b, index, part, out=wide[:, 80:120])
    call, res = m.prepare_lora_add(x, a, b, index, y, scales=s)
    n = len(lib.calls)
    call()
    assert len(lib.calls) == n + 1 and _val(lib.calls[-1][1][8]) == res.data_ptr()

    good = dict(x=x, a=a, b=b, index=index, y=y, scales=s)
    for bad in (dict(x=bf16(3, 72)), dict(x=bf16(64)), dict(x=x.float()), dict(a=bf16(16, 64)),
                dict(a=a.float()), dict(b=bf16(3, 40, 16)), dict(b=bf16(2, 40, 8)),
                dict(b=b.transpose(0, 1)), dict(a=bf16(2, 64, 16).transpose(1, 2)),
                dict(index=index.long()), dict(index=torch.zeros(4, dtype=torch.int32)),
                dict(index=torch.zeros(6, dtype=torch.int32)[::2]), dict(y=bf16(3, 48)),
                dict(y=bf16(2, 40)), dict(y=bf16(40, 3).T), dict(scales=torch.ones(3)),
                dict(scales=torch.ones(2).double()), dict(out=bf16(3, 48)), dict(out=y.float()),
                dict(out=wide[:, 40:80], y=wide[:, 48:88]), dict(out=wide[1:, 40:80], y=wide[:2, 0:40]),
                dict(workspace_buf=torch.zeros(4096))):
        with pytest.raises(ValueError):
            m.lora_add(**{**good, **bad})
    for K, N, R in ((64, 40, 12), (60, 40, 16), (64, 44, 16)):
        with pytest.raises(m.MxgError):
            m.lora_add(bf16(3, K), bf16(2, R, K), bf16(2, N, R), index, bf16(3, N))


def test_sample_binding(fake):
    m, lib = fake
    logits, u = bf16(3, 50), torch.zeros(3)
    k, p = torch.zeros(3, dtype=torch.int32), torch.ones(3)
    tokens, probs = m.sample_logits(logits, u, p, k, None, p)
    name, args = lib.calls[-1]
    got = [_val(v) for v in args[:-1]]
    assert name == "sample_logits"
    assert got == [logits.data_ptr(), 0, 50, 3, 50, u.data_ptr(), p.data_ptr(), k.data_ptr(), None,
                   p.data_ptr(), tokens.data_ptr(), probs.data_ptr()]
    assert tokens.dtype == torch.int32 and probs.dtype == torch.float32
    wide = torch.zeros(3, 64)
    m.sample_logits(wide[:, 3:50], u)
    got = [_val(v) for v in lib.calls[-1][1][:-1]]
    assert got[:5] == [wide.data_ptr() + 12, 1, 64, 3, 47]
    call, (t, _) = m.prepare_sample_logits(logits, u, top_k=k)
    call()
    assert _val(lib.calls[-1][1][10]) == t.data_ptr()
    good = dict(logits=logits, u=u)
    for bad in (dict(logits=logits.half()), dict(logits=bf16(50)), dict(logits=bf16(50, 3).T),
                dict(u=None), dict(u=u.double()), dict(u=torch.zeros(2)),
                dict(temperature=torch.ones(3, 1)), dict(top_k=k.long()), dict(top_p=torch.ones(4)),
                dict(min_p=p.double()), dict(tokens=torch.zeros(3)),
                dict(probs=torch.zeros(6)[::2])):
        with pytest.raises(ValueError):
            m.sample_logits(**{**good, **bad})


def test_head_and_sampler_binding(fake):
    m, lib = fake
    packed = torch.zeros(int(m._lib._real.w8a16_packed_bytes(128, 192, 128)), dtype=torch.uint8)
    u = torch.zeros(2)
    tokens, probs, logits = m.w8a16_gemm_sample(bf16(2, 128), packed, 192, 128, u, vocab=150)
    assert [c[0] for c in lib.calls[-2:]] == ["w8a16_gemm_ex", "sample_logits"]
    got = [_val(v) for v in lib.calls[-1][1][:-1]]
    assert got[:5] == [logits.data_ptr(), 0, 192, 2, 150] and logits.shape == (2, 192)
    for vocab in (0, 193, -1):
        with pytest.raises(ValueError):
            m.w8a16_gemm_sample(bf16(2, 128), packed, 192, 128, u, vocab=vocab)
