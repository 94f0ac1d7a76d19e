"""The mixing operators' C ABI and binding without a GPU: declarations, sizes and
refusals.  Fake device addresses; every call returns before any launch."""
import ctypes
import os
import re
import types

import pytest
import torch

import depthwise_convolution_amd as dw

from .test_sequence_devices import OnGpu

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "dwconv_mix.h")
A = 1 << 40          # fake addresses, 1 GiB apart
X, W, B, Y, Z, P, Q, R, V, U = (A + (k << 30) for k in range(10))


@pytest.fixture(scope="module")
def L():
    return dw.lib()


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def _refuses(L, name, defaults, bad):
    for changes, code in bad:
        a = dict(defaults, **changes)
        assert list(a) == list(defaults)
        assert dw.STATUS[getattr(L, name)(*a.values())] == code, (name, changes)


def test_header_and_binding_agree(L):
    assert set(re.findall(r"\b(dwconv_\w+)\s*\(", _text())) == set(dw.MIX_EXPORTS)
    for name in dw.MIX_EXPORTS:
        assert hasattr(L, name) and callable(getattr(dw, name))
    d = dict(re.findall(r"#define\s+(DWCONV_\w+)\s+(\d+)", _text()))
    assert int(d["DWCONV_ATTENTION_MAX_DIM"]) == dw.ATTENTION_MAX_DIM
    assert int(d["DWCONV_T_I8"]) == dw.T_I8 and int(d["DWCONV_I8_MAX_K"]) == dw.I8_MAX_K
    # the largest sum of products of 8-bit numbers fits into 32 bits, one more does not
    assert dw.I8_MAX_K * 128 * 128 < 1 << 31 <= (dw.I8_MAX_K + 1) * 128 * 128


HEADS = dict(H=4, KV=2, Dk=16, Dv=32)
HEADS_BAD = [
    (dict(H=0), "BAD_DIM"), (dict(KV=0), "BAD_DIM"), (dict(KV=3), "BAD_DIM"),
    (dict(KV=8), "BAD_DIM"), (dict(H=1 << 17), "BAD_DIM"), (dict(Dk=0), "BAD_DIM"),
    (dict(Dk=257), "BAD_DIM"), (dict(Dv=-1), "BAD_DIM"), (dict(Dv=257), "BAD_DIM"),
    (dict(type=3), "BAD_WTYPE"), (dict(type=-1), "BAD_WTYPE"),
    (dict(scale=float("nan")), "BAD_EPILOGUE"), (dict(scale=float("inf")), "BAD_EPILOGUE"),
    (dict(q=None), "NULL_PTR"), (dict(k=None), "NULL_PTR"), (dict(v=None), "NULL_PTR"),
    (dict(g=None), "NULL_PTR"), (dict(seqs=0), "BAD_DIM"),
    (dict(ldq=63), "ROW_STRIDE"), (dict(ldk=31), "ROW_STRIDE"), (dict(ldv=63), "ROW_STRIDE"),
    (dict(ldq=1 << 21), "ROW_STRIDE"), (dict(ldv=-64), "ROW_STRIDE"),
    (dict(q=X + 1), "MISALIGNED"), (dict(g=B + 2), "MISALIGNED"),
]


def test_attention_fwd_refuses(L):
    n = dw.dwconv_attention_workspace_size(False, torch.bfloat16, 2, 1000, False, *HEADS.values())
    assert n > 0
    d = dict(q=X, ldq=64, k=P, ldk=32, v=Q, ldv=64, type=2, g=B, scale=0.25, h0=R, y=Y, ldy=128,
             hT=Z, ws=U, wsb=n, seqs=2, tokens=1000, offsets=None, **HEADS, stream=None)
    _refuses(L, "dwconv_attention_fwd", d, HEADS_BAD + [
        (dict(y=None), "NULL_PTR"), (dict(ldy=127), "ROW_STRIDE"), (dict(tokens=-1), "BAD_DIM"),
        (dict(seqs=1 << 20, tokens=1 << 11), "BAD_DIM"), (dict(tokens=1 << 40), "BAD_DIM"),
        (dict(y=X), "ALIAS"), (dict(y=P + 2), "ALIAS"), (dict(hT=R), "ALIAS"),
        (dict(hT=Y), "ALIAS"), (dict(y=B), "ALIAS"), (dict(ws=Z), "ALIAS"), (dict(y=V, offsets=V),
                                                                            "ALIAS"),
        (dict(ws=None), "WORKSPACE"), (dict(wsb=n - 1), "WORKSPACE"), (dict(ws=U + 8), "WORKSPACE"),
        (dict(hT=Z + 2), "MISALIGNED"), (dict(h0=R + 1), "MISALIGNED"),
        (dict(offsets=V + 2), "MISALIGNED")])


def test_attention_step_refuses(L):
    d = dict(q=X, ldq=64, k=P, ldk=32, v=Q, ldv=64, type=1, g=B, scale=0.25, h=R, y=Y, ldy=128,
             seqs=3, **HEADS, stream=None)
    _refuses(L, "dwconv_attention_step", d, HEADS_BAD + [
        (dict(h=None), "NULL_PTR"), (dict(y=None), "NULL_PTR"), (dict(h=X), "ALIAS"),
        (dict(y=R), "ALIAS"), (dict(y=Q), "ALIAS"), (dict(ldy=1), "ROW_STRIDE"),
        (dict(h=R + 1), "MISALIGNED")])


def test_attention_grad_refuses(L):
    n = dw.dwconv_attention_workspace_size(True, torch.float32, 2, 500, False, *HEADS.values())
    d = dict(dy=Y, lddy=128, q=X, ldq=64, k=P, ldk=32, v=Q, ldv=64, type=0, g=B, scale=0.25, h0=R,
             dhT=R + (1 << 25), dq=Z, lddq=64, dk=Z + (1 << 25), lddk=32, dv=Z + (2 << 25),
             lddv=64, dh0=V, ws=U, wsb=n, seqs=2, tokens=500, offsets=None, **HEADS, stream=None)
    _refuses(L, "dwconv_attention_grad", d, HEADS_BAD[:-2] + [
        (dict(q=X + 2), "MISALIGNED"), (dict(g=B + 2), "MISALIGNED"),
        (dict(dy=None), "NULL_PTR"), (dict(lddy=64), "ROW_STRIDE"), (dict(lddq=63), "ROW_STRIDE"),
        (dict(lddk=0), "ROW_STRIDE"), (dict(lddv=1 << 21), "ROW_STRIDE"), (dict(dq=Y), "ALIAS"),
        (dict(dk=Z), "ALIAS"), (dict(dv=Q), "ALIAS"), (dict(dh0=R), "ALIAS"),
        (dict(dh0=R + (1 << 25)), "ALIAS"), (dict(ws=X), "ALIAS"), (dict(ws=None), "WORKSPACE"),
        (dict(wsb=n - 1), "WORKSPACE"), (dict(tokens=-1), "BAD_DIM")])


NORM_BAD = [
    (dict(x=None), "NULL_PTR"), (dict(type=3), "BAD_WTYPE"), (dict(act=4), "BAD_EPILOGUE"),
    (dict(N=-1), "BAD_DIM"), (dict(P=0), "BAD_DIM"), (dict(C=0), "BAD_DIM"),
    (dict(groups=0), "BAD_DIM"), (dict(groups=5), "BAD_DIM"), (dict(groups=96), "BAD_DIM"),
    (dict(N=1 << 20, P=1 << 11), "BAD_DIM"), (dict(N=1 << 62), "BAD_DIM"),
    (dict(P=1 << 62), "BAD_DIM"), (dict(ldx=47), "ROW_STRIDE"), (dict(ldx=1 << 40), "ROW_STRIDE"),
    (dict(x=X + 1), "MISALIGNED"), (dict(w=W + 2), "MISALIGNED"), (dict(ws=None), "WORKSPACE"),
    (dict(ws=U + 8), "WORKSPACE"), (dict(wsb=7), "WORKSPACE"), (dict(ws=X), "ALIAS"),
]


def test_norm_refuses(L):
    n = dw.dwconv_norm_workspace_size(False, torch.float16, 3, 500, 48, 6)
    assert n > 0
    d = dict(x=X, ldx=48, type=1, w=W, b=B, eps=1e-5, act=3, y=Y, ldy=48, stats=R, ws=U, wsb=n,
             N=3, P=500, C=48, groups=6, stream=None)
    _refuses(L, "dwconv_norm_fwd", d, NORM_BAD + [
        (dict(y=None), "NULL_PTR"), (dict(eps=-1e-9), "BAD_EPILOGUE"),
        (dict(eps=float("nan")), "BAD_EPILOGUE"), (dict(eps=float("inf")), "BAD_EPILOGUE"),
        (dict(ldy=1), "ROW_STRIDE"), (dict(y=X, ldy=64), "ALIAS"), (dict(y=X + 2), "ALIAS"),
        (dict(y=W), "ALIAS"), (dict(stats=Y), "ALIAS"), (dict(stats=X, y=X), "ALIAS"),
        (dict(wsb=n - 1), "WORKSPACE")])
    n = dw.dwconv_norm_workspace_size(True, torch.float16, 3, 500, 48, 6)
    d = dict(dy=Y, lddy=48, x=X, ldx=48, type=1, w=W, b=B, act=3, stats=R, dx=Z, lddx=48, dw=P,
             db=P + 4096, ws=U, wsb=n, N=3, P=500, C=48, groups=6, stream=None)
    _refuses(L, "dwconv_norm_grad", d, NORM_BAD + [
        (dict(dy=None), "NULL_PTR"), (dict(stats=None), "NULL_PTR"), (dict(dx=X), "ALIAS"),
        (dict(dx=Y, lddx=64), "ALIAS"), (dict(db=P + 4), "ALIAS"), (dict(dw=W), "ALIAS"),
        (dict(lddx=2), "ROW_STRIDE"), (dict(lddy=2), "ROW_STRIDE"), (dict(wsb=n - 1), "WORKSPACE")])


def test_quantize_rows_refuses(L):
    d = dict(x=X, ldx=32, type=2, q=Q, ldq=32, scale=R, M=20, K=32, stream=None)
    _refuses(L, "dwconv_quantize_rows", d, [
        (dict(x=None), "NULL_PTR"), (dict(q=None), "NULL_PTR"), (dict(scale=None), "NULL_PTR"),
        (dict(type=3), "BAD_WTYPE"), (dict(M=-1), "BAD_DIM"), (dict(M=1 << 31), "BAD_DIM"),
        (dict(K=0), "BAD_DIM"), (dict(ldx=31), "ROW_STRIDE"), (dict(ldq=31), "ROW_STRIDE"),
        (dict(q=X), "ALIAS"), (dict(scale=Q), "ALIAS"), (dict(scale=R + 2), "MISALIGNED"),
        (dict(x=X + 1), "MISALIGNED")])


def test_linear_i8_refuses(L):
    d = dict(x=X, ldx=32, xtype=3, xs=R, w=W, ldw=32, ws=R + 4096, type=2, b=B, act=3, res=P,
             ldres=48, y=Y, ldy=48, space=U, spaceb=1 << 28, M=20, N=48, K=32, stream=None)
    _refuses(L, "dwconv_linear_i8", d, [
        (dict(x=None), "NULL_PTR"), (dict(xs=None), "NULL_PTR"), (dict(w=None), "NULL_PTR"),
        (dict(ws=None), "NULL_PTR"), (dict(y=None), "NULL_PTR"), (dict(type=3), "BAD_WTYPE"),
        (dict(xtype=1), "BAD_WTYPE"), (dict(xtype=4), "BAD_WTYPE"),
        (dict(xtype=2), "BAD_WTYPE"),       # scales of an x that is to be quantised
        (dict(act=4), "BAD_EPILOGUE"), (dict(M=-1), "BAD_DIM"), (dict(M=1 << 31), "BAD_DIM"),
        (dict(N=0), "BAD_DIM"), (dict(K=0), "BAD_DIM"), (dict(K=131072, ldx=1 << 18), "BAD_DIM"),
        (dict(ldx=31), "ROW_STRIDE"), (dict(ldw=31), "ROW_STRIDE"), (dict(ldw=1 << 21), "ROW_STRIDE"),
        (dict(ldy=47), "ROW_STRIDE"), (dict(ldres=47), "ROW_STRIDE"), (dict(y=X), "ALIAS"),
        (dict(y=W), "ALIAS"), (dict(y=R), "ALIAS"), (dict(y=P), "ALIAS"), (dict(y=B), "ALIAS"),
        (dict(b=B + 1), "MISALIGNED"), (dict(xs=R + 2), "MISALIGNED"), (dict(y=Y + 1), "MISALIGNED")])
    n = dw.dwconv_linear_i8_workspace_size(torch.bfloat16, torch.bfloat16, 400, 48, 32)
    assert n >= 400 * 36
    own = dict(d, xtype=2, xs=None, M=400, spaceb=n)
    _refuses(L, "dwconv_linear_i8", own, [
        (dict(space=None), "WORKSPACE"), (dict(spaceb=n - 1), "WORKSPACE"),
        (dict(space=U + 8), "WORKSPACE"), (dict(space=Y), "ALIAS"), (dict(x=X + 1), "MISALIGNED")])


def test_sizes(L):
    out = ctypes.c_longlong(0)
    bf16 = torch.bfloat16
    # a batch of two chunks has nothing to link, whoever's heads are shared
    assert dw.dwconv_attention_workspace_size(False, bf16, 2, 128, False, 4, 2, 64, 64) == 0
    assert dw.dwconv_attention_workspace_size(True, bf16, 2, 70, True, 2, 2, 24, 24) == 0
    assert dw.dwconv_attention_workspace_size(True, bf16, 1, 70, True, 4, 2, 24, 40) == \
        4 * 70 * 4 * (24 + 40)
    # enough sequences and heads fill the chip by themselves
    assert dw.dwconv_attention_workspace_size(False, bf16, 64, 1000, False, 16, 2, 64, 64) == 0
    assert dw.dwconv_attention_workspace_size(False, bf16, 1, 1000, False, 16, 2, 64, 64) > 0
    assert dw.dwconv_norm_workspace_size(False, bf16, 100, 1, 96, 6) == 0
    assert dw.dwconv_norm_workspace_size(True, bf16, 0, 50, 96, 6) == 0
    assert dw.dwconv_linear_i8_workspace_size(torch.int8, bf16, 40, 100, 512) == 0
    assert dw.dwconv_linear_i8_workspace_size(bf16, bf16, 8, 100, 512) == 0     # in one launch
    assert dw.dwconv_linear_i8_workspace_size(bf16, bf16, 0, 100, 512) == 0
    for name, args in (("dwconv_attention_workspace_size", (0, 2, 2, 9, 0, 4, 3, 8, 8)),
                       ("dwconv_norm_workspace_size", (0, 2, 2, 9, 10, 4)),
                       ("dwconv_linear_i8_workspace_size", (3, 2, 2, 9, 1 << 20))):
        assert dw.STATUS[getattr(L, name)(*args, ctypes.byref(out))] == "BAD_DIM"
        assert dw.STATUS[getattr(L, name)(*args, None)] == "NULL_PTR"


def test_the_product_s_kernels():
    bf16 = torch.bfloat16
    assert dw.dwconv_linear_i8_describe(False, bf16, 8, 256, 512) == ("few_rows_quantized", 1)
    assert dw.dwconv_linear_i8_describe(True, bf16, 8, 256, 512)[0] == "few_rows"
    # up to 16 rows, and up to 32768 elements of them
    assert dw.dwconv_linear_i8_describe(False, bf16, 16, 256, 2048)[0] == "few_rows_quantized"
    assert dw.dwconv_linear_i8_describe(False, bf16, 16, 256, 2049)[0] == "few_rows"
    assert dw.dwconv_linear_i8_describe(False, bf16, 17, 256, 64)[0] == "few_rows"
    assert dw.dwconv_linear_i8_describe(False, bf16, 4096, 4096, 4096) == ("tile_256", 1)
    assert dw.dwconv_linear_i8_describe(True, bf16, 4096, 4096, 4096, aligned=False)[0] == \
        "tile_128_registers"
    assert dw.dwconv_linear_i8_describe(True, bf16, 128, 256, 65536)[1] > 1


def test_binding_refuses_cpu_tensors_and_wrong_types():
    q, k, x = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 2, 8), torch.zeros(2, 3, 8)
    g, s, w = torch.zeros(4), torch.zeros(2, 4, 2), torch.zeros(4, 8, dtype=torch.int8)
    for call in (lambda: dw.linear_attention(q, k, k, g),
                 lambda: dw.linear_attention_step(q[0], k[0], k[0], g, torch.zeros(3, 4, 8, 8)),
                 lambda: dw.linear_attention_grad(q, q, k, k, g),
                 lambda: dw.group_norm(x, 4), lambda: dw.group_norm_grad(x, x, s, 4),
                 lambda: dw.quantize_rows(x), lambda: dw.linear_i8(x, w, g)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: dw.linear_attention([1.0], k, k, g), lambda: dw.group_norm([1.0], 1),
                 lambda: dw.quantize_rows("x"), lambda: dw.linear_i8([1.0], w, g)):
        with pytest.raises(TypeError):
            call()


def _on(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def test_stream_of_another_device():
    q, x = _on(2, 3, 4, 8), _on(2, 3, 8)
    w = _on(4, 8, dtype=torch.int8)
    other = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1))
    for call in (lambda: dw.linear_attention(q, q, q, x, stream=other),
                 lambda: dw.linear_attention_step(q[0], q[0], q[0], x, x, stream=other),
                 lambda: dw.linear_attention_grad(q, q, q, q, x, stream=other),
                 lambda: dw.group_norm(x, 4, stream=other),
                 lambda: dw.group_norm_grad(x, x, x, 4, stream=other),
                 lambda: dw.quantize_rows(x, stream=other),
                 lambda: dw.linear_i8(x, w, x, stream=other)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_attention_refuses_more_workgroups_than_a_grid_holds(L):
    """Before anything is enqueued: 2^29 sequences of one token, 4 heads."""
    d = dict(q=1 << 44, ldq=4, k=2 << 44, ldk=2, v=3 << 44, ldv=2, type=0, g=B, scale=1.0,
             h0=None, y=4 << 44, ldy=4, hT=None, ws=None, wsb=0, seqs=1 << 29, tokens=1,
             offsets=None, H=4, KV=2, Dk=1, Dv=1, stream=None)
    _refuses(L, "dwconv_attention_fwd", d, [({}, "BAD_DIM")])
