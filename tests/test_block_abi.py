"""Operators around the FFN: refusals of the C entry points and of the binding
before anything is enqueued. No GPU is needed: every call fails on the host or
has nothing to do."""

import ctypes

import pytest

import activation_sparse_ffn_gate_amd as tw
from activation_sparse_ffn_gate_amd._lib import _Q4

torch = pytest.importorskip("torch")

OK, E_ARG, E_UNSUP, E_WS = 0, -1, -2, -3
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: validation fails first
BF16, F32, E4M3 = 0, 1, 2


def _with(args, **at):
    args = list(args)
    for k, v in at.items():
        args[int(k[1:])] = v
    return args


def test_dropout_refusals():
    f = tw.lib().twell_dropout
    ok = [FAKE, F32, None, 4, 16, 0.1, 1, 2, FAKE, BF16, None]
    nan = float("nan")
    for at, want in (({"_0": None}, E_ARG), ({"_8": None}, E_ARG), ({"_3": -1}, E_ARG), ({"_4": 0}, E_ARG),
                     ({"_5": -0.1}, E_ARG), ({"_5": 1.0}, E_ARG), ({"_5": nan}, E_ARG), ({"_5": 1 - 2.0**-18}, E_ARG),
                     ({"_1": E4M3}, E_UNSUP), ({"_9": E4M3}, E_UNSUP), ({"_1": 7}, E_UNSUP), ({"_9": -1}, E_UNSUP),
                     ({"_3": (1 << 24) + 1}, E_UNSUP), ({"_4": (1 << 24) + 1}, E_UNSUP),
                     ({"_3": 1 << 24, "_4": 1 << 24}, E_UNSUP)):
        assert f(*_with(ok, **at)) == want, at
    assert f(*_with(ok, _0=None, _3=0, _8=None)) == OK  # no rows: nothing to do
    assert f(*_with(ok, _3=0, _5=2.0)) == E_ARG


def test_add_rmsnorm_refusals():
    f = tw.lib().twell_add_rmsnorm
    #      0     1    2     3     4    5  6   7     8    9  10 11    12    13    14    15    16    17
    ok = [FAKE, F32, None, FAKE, BF16, 4, 16, 1e-6, 0.1, 1, 2, FAKE, BF16, FAKE, E4M3, FAKE, None, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_13": None}, E_ARG), ({"_5": -1}, E_ARG),
                     ({"_6": 0}, E_ARG), ({"_6": 16385}, E_UNSUP), ({"_5": (1 << 24) + 1}, E_UNSUP),
                     ({"_7": -1e-6}, E_ARG), ({"_7": float("nan")}, E_ARG), ({"_7": float("inf")}, E_ARG),
                     ({"_8": 1.5}, E_ARG), ({"_1": E4M3}, E_UNSUP), ({"_4": E4M3}, E_UNSUP), ({"_12": E4M3}, E_UNSUP),
                     ({"_14": F32}, E_UNSUP), ({"_15": None}, E_ARG), ({"_14": BF16}, E_ARG)):
        assert f(*_with(ok, **at)) == want, at
    assert f(*_with(ok, _0=None, _3=None, _5=0, _13=None)) == OK


def test_add_rmsnorm_backward_refusals():
    f = tw.lib().twell_add_rmsnorm_backward
    ws = tw.rmsnorm_workspace_bytes(4, 16)
    assert ws >= 16 * 4 and ws % 256 == 0
    #      0     1    2     3     4     5     6    7     8  9   10   11 12 13    14    15    16    17   18  19
    ok = [FAKE, F32, None, FAKE, BF16, FAKE, F32, FAKE, 4, 16, 0.1, 1, 2, FAKE, FAKE, BF16, FAKE, FAKE, ws, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_5": None}, E_ARG), ({"_7": None}, E_ARG),
                     ({"_13": None, "_14": None}, E_ARG), ({"_16": None}, E_ARG), ({"_8": -1}, E_ARG),
                     ({"_9": 16385}, E_UNSUP), ({"_1": E4M3}, E_UNSUP), ({"_4": 9}, E_UNSUP), ({"_6": E4M3}, E_UNSUP),
                     ({"_15": E4M3}, E_UNSUP), ({"_10": 1.0}, E_ARG), ({"_17": None}, E_WS), ({"_18": ws - 1}, E_WS),
                     ({"_17": ctypes.c_void_p(FAKE.value + 8)}, E_WS)):
        assert f(*_with(ok, **at)) == want, at
    assert tw.rmsnorm_workspace_bytes(0, 16) == 0 and tw.rmsnorm_workspace_bytes(4, 16385) == 0
    assert tw.rmsnorm_workspace_bytes(-1, 16) == 0


def _q4(codes=FAKE.value, scales=FAKE.value, zeros=0):
    return ctypes.byref(_Q4(codes, scales, zeros))


def test_q4_refusals():
    L = tw.lib()
    #      0     1     2     3      4  5   6   7   8     9    10  11  12
    ok = [FAKE, BF16, None, _q4(), 4, 32, 64, 32, FAKE, F32, None, 0, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_3": _q4(codes=0)}, E_ARG),
                     ({"_3": _q4(scales=0)}, E_ARG), ({"_8": None}, E_ARG), ({"_4": -1}, E_ARG), ({"_5": 0}, E_ARG),
                     ({"_6": 0}, E_ARG), ({"_7": 0}, E_UNSUP), ({"_7": 16}, E_UNSUP), ({"_7": 256}, E_UNSUP),
                     ({"_1": 5}, E_UNSUP), ({"_9": E4M3}, E_UNSUP), ({"_1": E4M3}, E_ARG), ({"_2": FAKE}, E_ARG),
                     ({"_4": (1 << 20) + 1}, E_UNSUP), ({"_5": (1 << 24) + 1}, E_UNSUP),
                     ({"_6": (1 << 24) + 1}, E_UNSUP)):
        assert L.twell_q4_matmul(*_with(ok, **at)) == want, at
    assert L.twell_q4_matmul(*_with(ok, _0=None, _4=0, _8=None)) == OK
    assert L.twell_q4_matmul(*_with(ok, _4=1 << 18, _5=1 << 16)) == E_UNSUP  # 2^34 elements of y
    # more than 16 rows: x as matrix operands needs room
    assert tw.q4_workspace_bytes(torch.bfloat16, 16, 32, 64) == 0
    ws = tw.q4_workspace_bytes(torch.bfloat16, 17, 32, 64)
    assert ws >= 32 * 64 * 2 and ws % 256 == 0
    assert L.twell_q4_matmul(*_with(ok, _4=17)) == E_WS
    assert L.twell_q4_matmul(*_with(ok, _4=17, _10=FAKE, _11=ws - 1)) == E_WS
    assert L.twell_q4_matmul(*_with(ok, _4=17, _10=ctypes.c_void_p(FAKE.value + 128), _11=ws)) == E_WS
    # a long K over few units is split: partial sums need room
    assert tw.q4_workspace_bytes(torch.bfloat16, 4, 32, 1 << 16) >= 2 * 4 * 32 * 4
    for bad in ((-1, 32, 64), (4, 0, 64), (4, 32, 0), (0, 32, 64), (1 << 19, 32, 64)):
        assert tw.q4_workspace_bytes(torch.bfloat16, *bad) == 0

    #      0     1     2     3      4      5  6   7   8   9     10   11   12 13
    ok = [FAKE, BF16, None, _q4(), _q4(), 4, 32, 64, 32, FAKE, F32, None, 0, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_4": _q4(codes=0)}, E_ARG), ({"_9": None}, E_ARG),
                     ({"_8": 48}, E_UNSUP), ({"_10": E4M3}, E_UNSUP), ({"_1": E4M3}, E_ARG), ({"_5": -1}, E_ARG)):
        assert L.twell_q4_gateup(*_with(ok, **at)) == want, at
    assert L.twell_q4_gateup(*_with(ok, _5=0)) == OK
    ws = tw.q4_workspace_bytes(torch.bfloat16, 17, 32, 64, gated=True)
    assert L.twell_q4_gateup(*_with(ok, _5=17)) == E_WS
    assert L.twell_q4_gateup(*_with(ok, _5=17, _11=FAKE, _12=ws - 256)) == E_WS

    size = lambda M, d, F: tw.ffn_q4_workspace_bytes(torch.bfloat16, M, d, F)  # noqa: E731
    ws = size(4, 64, 32)
    assert ws >= 4 * 32 * 4 and ws % 256 == 0
    assert size(0, 64, 32) == 0 and size(4, 64, 0) == 0 and size(4, 0, 32) == 0
    #      0     1     2     3      4      5      6  7   8   9   10    11    12  13
    ok = [FAKE, BF16, None, _q4(), _q4(), _q4(), 4, 64, 32, 32, FAKE, FAKE, ws, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_4": None}, E_ARG), ({"_5": None}, E_ARG),
                     ({"_10": None}, E_ARG), ({"_11": None}, E_WS), ({"_12": ws - 1}, E_WS),
                     ({"_11": ctypes.c_void_p(FAKE.value + 16)}, E_WS), ({"_9": 100}, E_UNSUP), ({"_1": E4M3}, E_ARG)):
        assert L.twell_ffn_forward_q4(*_with(ok, **at)) == want, at
    assert L.twell_ffn_forward_q4(*_with(ok, _6=0)) == OK

    f = L.twell_q4_quantize
    assert f(None, 4, 64, 32, FAKE, FAKE, None) == E_ARG
    assert f(FAKE, 4, 64, 32, None, FAKE, None) == E_ARG
    assert f(FAKE, 4, 64, 32, FAKE, None, None) == E_ARG
    assert f(FAKE, 4, 64, 33, FAKE, FAKE, None) == E_UNSUP
    assert f(FAKE, 1 << 24, 1 << 24, 32, FAKE, FAKE, None) == E_UNSUP


def test_binding_refuses_host_tensors_and_odd_seeds():
    x = torch.zeros(4, 16)
    w = torch.ones(16)
    q = tw.Q4(torch.zeros(8, 8, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.bfloat16), None, 16, 32)
    for call in (lambda: tw.dropout(x, 0.1, 1), lambda: tw.add_rmsnorm(x, w), lambda: tw.q4_matmul(x, q),
                 lambda: tw.add_rmsnorm_backward(x, x, w, w[:4]), lambda: tw.q4_gateup(x, q, q),
                 lambda: tw.ffn_forward_q4(x, q, q, q), lambda: tw.q4_quantize(x.bfloat16())):
        with pytest.raises(ValueError, match="device tensor"):
            call()
