"""Layer norm, low-rank adapters, the gradients' norm and the optimizer's step: refusals of the C entry
points and of the binding before anything is enqueued, and what the binding hands over.
No GPU is needed: every call fails on the host, has nothing to do, or is recorded."""

import ctypes

import pytest

import activation_sparse_ffn_gate_amd as tw
from activation_sparse_ffn_gate_amd import _block, _optim
from activation_sparse_ffn_gate_amd._lib import _AdamwTensor, _Grad

torch = pytest.importorskip("torch")

OK, E_ARG, E_UNSUP, E_WS = 0, -1, -2, -3
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: validation fails first
BF16, F32, E4M3 = 0, 1, 2
NAN, INF = float("nan"), float("inf")


def _with(args, **at):
    args = list(args)
    for k, v in at.items():
        args[int(k[1:])] = v
    return args


def test_layernorm_refusals():
    f = tw.lib().twell_add_layernorm
    #      0     1    2     3     4    5     6  7   8     9    10 11 12    13    14    15    16    17    18    19
    ok = [FAKE, F32, None, FAKE, None, BF16, 4, 16, 1e-5, 0.1, 1, 2, FAKE, BF16, FAKE, E4M3, FAKE, None, None, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_14": None}, E_ARG), ({"_6": -1}, E_ARG),
                     ({"_7": 0}, E_ARG), ({"_7": 16385}, E_UNSUP), ({"_6": (1 << 24) + 1}, E_UNSUP),
                     ({"_8": -1e-5}, E_ARG), ({"_8": NAN}, E_ARG), ({"_8": INF}, E_ARG), ({"_9": 1.0}, E_ARG),
                     ({"_1": E4M3}, E_UNSUP), ({"_5": 3}, E_UNSUP), ({"_13": E4M3}, E_UNSUP), ({"_15": F32}, E_UNSUP),
                     ({"_16": None}, E_ARG), ({"_15": BF16}, E_ARG)):
        assert f(*_with(ok, **at)) == want, at
    assert f(*_with(ok, _0=None, _6=0, _14=None)) == OK

    f = tw.lib().twell_add_layernorm_backward
    ws = tw.layernorm_workspace_bytes(4, 16)
    assert ws >= 16 * 8 and ws % 256 == 0 and tw.layernorm_workspace_bytes(400, 600) >= 100 * 600 * 8
    #      0     1    2     3     4     5     6     7     8     9 10  11  12 13 14    15    16    17    18    19    20 21
    ok = [FAKE, F32, None, FAKE, BF16, FAKE, BF16, FAKE, FAKE, 4, 16, 0.1, 1, 2, FAKE, FAKE, BF16, FAKE, FAKE, FAKE, ws,
          None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_5": None}, E_ARG), ({"_7": None}, E_ARG),
                     ({"_8": None}, E_ARG), ({"_14": None, "_15": None}, E_ARG), ({"_17": None}, E_ARG),
                     ({"_9": -1}, E_ARG), ({"_10": 16385}, E_UNSUP), ({"_1": E4M3}, E_UNSUP), ({"_4": 9}, E_UNSUP),
                     ({"_6": E4M3}, E_UNSUP), ({"_16": E4M3}, E_UNSUP), ({"_11": 1.0}, E_ARG), ({"_19": None}, E_WS),
                     ({"_20": ws - 1}, E_WS), ({"_19": ctypes.c_void_p(FAKE.value + 8)}, E_WS)):
        assert f(*_with(ok, **at)) == want, at
    assert tw.layernorm_workspace_bytes(0, 16) == 0 and tw.layernorm_workspace_bytes(4, 16385) == 0


def test_lora_refusals():
    f = tw.lib().twell_lora
    #      0     1     2     3     4     5     6    7  8  9   10  11 12    13    14   15
    y = type(FAKE)(FAKE.value + 4096)
    ok = [FAKE, BF16, None, FAKE, FAKE, FAKE, None, 2, 4, 32, 64, 5, FAKE, y, F32, None]
    for at, want in (({"_0": None}, E_ARG), ({"_3": None}, E_ARG), ({"_4": None}, E_ARG), ({"_5": None}, E_ARG),
                     ({"_12": None}, E_ARG), ({"_13": None}, E_ARG), ({"_7": -1}, E_ARG), ({"_8": -1}, E_ARG),
                     ({"_9": 0}, E_ARG), ({"_10": 0}, E_ARG), ({"_11": 0}, E_ARG), ({"_11": 257}, E_UNSUP),
                     ({"_8": (1 << 18) + 1}, E_UNSUP), ({"_9": (1 << 22) + 1}, E_UNSUP),
                     ({"_10": (1 << 24) + 1}, E_UNSUP), ({"_8": 1 << 18, "_9": 1 << 16}, E_UNSUP),
                     ({"_7": 1 << 31}, E_UNSUP), ({"_14": E4M3}, E_UNSUP), ({"_1": 4}, E_UNSUP), ({"_1": E4M3}, E_ARG),
                     ({"_2": FAKE}, E_ARG), ({"_13": FAKE}, E_ARG)):  # y at x
        assert f(*_with(ok, **at)) == want, at
    assert f(*_with(ok, _0=None, _8=0, _13=None)) == OK


def _grads(*items):
    return (_Grad * len(items))(*items), len(items)


def test_grad_norm_refusals():
    L = tw.lib()
    f, size = L.twell_grad_norm, L.twell_grad_norm_workspace_bytes
    one = _grads((FAKE.value, 100, F32))
    ws = size(*one)
    assert ws % 256 == 0 and ws >= 8
    assert size(*_grads((FAKE.value, 1 << 34, BF16), (FAKE.value, 1, F32))) >= 8 * ((1 << 34) // 8192 + 1)
    for bad, want in ((_grads((None, 5, F32)), E_ARG), (_grads((FAKE.value, -1, F32)), E_ARG),
                      (_grads((FAKE.value, 5, E4M3)), E_UNSUP), (_grads((FAKE.value, (1 << 34) + 1, F32)), E_UNSUP),
                      ((None, 1), E_ARG), ((None, -1), E_ARG)):
        assert f(*bad, 1.0, FAKE, FAKE, 1 << 30, None) == want
        assert size(*bad) == 0
    for norm in (0.0, -1.0, NAN):
        assert f(*one, norm, FAKE, FAKE, ws, None) == E_ARG
    assert f(*one, 1.0, None, FAKE, ws, None) == E_ARG
    assert f(*one, 1.0, FAKE, None, ws, None) == E_WS and f(*one, 1.0, FAKE, FAKE, ws - 1, None) == E_WS
    assert f(*one, 1.0, FAKE, ctypes.c_void_p(FAKE.value + 8), ws, None) == E_WS


def _tensor(scales=False, **kw):
    p = FAKE.value
    s = p if scales else None
    t = _AdamwTensor(p, p, p, p, s, s, p, p, p, s, s, None, 100, 0.1, F32)
    for k, v in kw.items():
        setattr(t, k, v)
    return (_AdamwTensor * 1)(t)


def test_adamw_refusals():
    f = tw.lib().twell_adamw
    #      0          1  2    3  4     5    6     7     8     9 10 11
    ok = [_tensor(), 1, F32, 1, 1e-3, 0.9, 0.99, 1e-8, None, 1, 2, None]
    for at, want in (({"_0": None}, E_ARG), ({"_1": -1}, E_ARG), ({"_3": 0}, E_ARG), ({"_4": -1.0}, E_ARG),
                     ({"_4": NAN}, E_ARG), ({"_4": INF}, E_ARG), ({"_5": 1.0}, E_ARG), ({"_5": -0.1}, E_ARG),
                     ({"_6": 1.0}, E_ARG), ({"_6": NAN}, E_ARG), ({"_7": -1e-8}, E_ARG), ({"_2": BF16}, E_UNSUP),
                     ({"_0": _tensor(n=-1)}, E_ARG), ({"_0": _tensor(n=(1 << 34) + 1)}, E_UNSUP),
                     ({"_0": _tensor(g_type=E4M3)}, E_UNSUP), ({"_0": _tensor(weight_decay=-1.0)}, E_ARG),
                     ({"_0": _tensor(weight_decay=NAN)}, E_ARG), ({"_0": _tensor(True)}, E_ARG), ({"_2": E4M3}, E_ARG)):
        assert f(*_with(ok, **at)) == want, at
    for name in ("p", "g", "m", "v", "p_out", "m_out", "v_out"):
        assert f(*_with(ok, _0=_tensor(**{name: None}))) == E_ARG, name
    for name in ("m_scale", "v_scale", "m_scale_out", "v_scale_out"):
        assert f(*_with(ok, _0=_tensor(True, **{name: None}), _2=E4M3)) == E_ARG, name
    # nothing to do
    assert f(*_with(ok, _0=None, _1=0)) == OK
    assert f(*_with(ok, _0=_tensor(n=0, p=None, g=None))) == OK


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 16), torch.ones(16)
    a = tw.Adapters(torch.zeros(2, 3, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 3, dtype=torch.bfloat16))
    t = tw.AdamTensors.zero(x)
    for call in (lambda: tw.add_layernorm(x, w), lambda: tw.add_layernorm_backward(x, x, w, w[:4], w[:4]),
                 lambda: tw.lora_add(x, a, torch.zeros(4, dtype=torch.int32), x[:, :8]), lambda: tw.grad_norm([x]),
                 lambda: tw.adamw_step([t], [x], 1, 1e-3)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    for call in (lambda: tw.grad_norm([]), lambda: tw.adamw_step([], [], 1, 1e-3)):
        with pytest.raises(ValueError, match="empty"):
            call()


@pytest.fixture
def calls(monkeypatch):
    """Entry points that record their arguments in a list, on host tensors."""
    seen = []
    for module in (_block, _optim):
        monkeypatch.setattr(module, "_call", lambda fn, name, device, *args: seen.append((name, args)))
    monkeypatch.setattr(_block, "_rows", lambda x, name, dtypes: (x.device, x.shape, x.data_ptr()))
    monkeypatch.setattr(_optim, "_device", lambda tensors, name: torch.device("cpu", 0))

    def ptr(t, name, shape, dtypes, device):
        if t.dtype not in dtypes:
            raise TypeError(name)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(name)
        return t.data_ptr()

    for module in (_block, _optim):
        monkeypatch.setattr(module, "_ptr", ptr)

    def refuse(t, name, *a):
        raise ValueError(name)

    monkeypatch.setattr(_optim, "_refuse", refuse)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    return seen


def test_scratch_is_a_calls_own(calls):
    x, w = torch.zeros(4, 64), torch.ones(64)
    for make in (lambda **kw: tw.add_layernorm_backward(x, x, w, w[:4], w[:4], **kw),
                 lambda **kw: tw.grad_norm([x, w], **kw)):
        ws = tw.Workspace(torch.device("cpu"))
        make(workspace=ws)
        address, size = calls[-1][1][-2:]
        address = getattr(address, "value", address)
        assert address % 256 == 0 and ws.buf.data_ptr() <= address and address + size <= ws.buf.data_ptr() + ws.buf.numel()
        with pytest.raises(ValueError, match="control block"):
            make(workspace=tw.Workspace(torch.device("cpu"), zeroed=True))


def test_adamw_step_hands_over_each_tensor(calls):
    p = [torch.zeros(3, 5), torch.zeros(700), torch.zeros(0)]
    t = [tw.AdamTensors.zero(q, torch.float8_e4m3fn, copy=torch.zeros_like(q, dtype=torch.bfloat16)) for q in p]
    assert [tuple(s.m_scale.shape) for s in t] == [(1,), (3,), (0,)]
    g = [torch.zeros(3, 5), torch.zeros(700, dtype=torch.bfloat16), torch.zeros(0)]
    tw.adamw_step(t, g, 3, 0.1, weight_decay=[0.5, 0.0, 0.0], seed=7, offset=8)
    name, (listed, count, state, step, lr, b1, b2, eps, scale, seed, offset) = calls[0]
    assert (name, count, state, step, lr, b1, b2, eps, scale, seed, offset) == ("twell_adamw", 3, E4M3, 3, 0.1, 0.9, 0.999,
                                                                               1e-8, None, 7, 8)
    elements = lambda data: (_AdamwTensor * 3).from_buffer_copy(data)  # noqa: E731
    for i, (s, q, d) in enumerate(zip(t, g, (0.5, 0.0, 0.0))):
        e = elements(listed)[i]
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            assert (getattr(e, k) or 0) == (getattr(e, k + "_out") or 0) == getattr(s, k).data_ptr(), k
        assert (e.g or 0) == q.data_ptr() and (e.copy or 0) == s.copy.data_ptr() and e.n == q.numel()
        assert e.weight_decay == d and e.g_type == (BF16 if q.dtype == torch.bfloat16 else F32)
    new = [tw.AdamTensors.zero(torch.ones_like(q), torch.float8_e4m3fn) for q in p]
    tw.adamw_step(t, g, 3, 0.1, out=new)
    e = elements(calls[1][1][0])[1]
    assert e.p == p[1].data_ptr() and e.p_out == new[1].p.data_ptr() and e.v_scale_out == new[1].v_scale.data_ptr()
    assert e.copy is None

    f32 = [tw.AdamTensors.zero(q) for q in p]
    for bad in (dict(grads=g[:2]), dict(out=new[:2]), dict(weight_decay=[0.1]), dict(tensors=[t[0], t[0], t[2]], grads=[g[0], g[0], g[2]]),
                dict(tensors=[t[0], f32[1], t[2]]), dict(out=f32), dict(grads=[g[0].t(), g[1], g[2]]), dict(seed=-1),
                dict(tensors=[tw.AdamTensors(t[0].p, t[0].m, t[0].v), t[1], t[2]]),
                dict(tensors=[tw.AdamTensors(f32[0].p, f32[0].m, f32[0].v, t[0].m_scale, t[0].v_scale), f32[1], f32[2]])):
        with pytest.raises((ValueError, TypeError)):
            tw.adamw_step(**{**dict(tensors=t, grads=g, step=1, lr=0.1), **bad})
    assert ctypes.sizeof(_AdamwTensor) == len(listed) // 3 and ctypes.sizeof(_Grad) == len(_optim._GRAD(1, 2, 3))
    grad = _Grad.from_buffer_copy(_optim._GRAD(1, 2, 3))
    assert (grad.g, grad.n, grad.g_type) == (1, 2, 3)
    with pytest.raises(TypeError):
        tw.adamw_step(t, [g[0].half(), *g[1:]], 1, 0.1)
    with pytest.raises(TypeError):
        tw.adamw_step([tw.AdamTensors(q, q.bfloat16(), q.bfloat16()) for q in p], g, 1, 0.1)
    assert len(calls) == 2


def test_adamw_step_refuses_a_place_of_two(calls):
    """Of two workgroups that write one place, or one that reads what another one writes, any may come first."""
    for state in (torch.float32, torch.float8_e4m3fn):
        make = lambda: tw.AdamTensors.zero(torch.zeros(300), state, copy=torch.zeros(300, dtype=torch.bfloat16))  # noqa: E731
        a, b, c, d = (make() for _ in range(4))
        g = [torch.zeros(300) for _ in range(2)]
        fields = ["p", "m", "v", "copy"] + (["m_scale", "v_scale"] if state is not torch.float32 else [])
        for k in fields:
            twice = tw.AdamTensors(b.p, b.m, b.v, b.m_scale, b.v_scale, b.copy)
            setattr(twice, k, getattr(a, k))
            with pytest.raises(ValueError, match="twice"):
                tw.adamw_step([a, twice], g, 1, 0.1)
            with pytest.raises(ValueError, match="twice"):
                tw.adamw_step([c, d], g, 1, 0.1, out=[a, twice])
            if k != "copy":
                other = tw.AdamTensors(d.p, d.m, d.v, d.m_scale, d.v_scale)
                setattr(other, k, getattr(a, k))  # the old value of the first tensor
                with pytest.raises(ValueError, match="old value"):
                    tw.adamw_step([a, b], g, 1, 0.1, out=[c, other])
        with pytest.raises(ValueError, match="gradient"):
            tw.adamw_step([a, b], [b.p, g[1]], 1, 0.1)
        assert not calls
        # one gradient for two tensors, and new values in part of their own places
        tw.adamw_step([a, b], [g[0], g[0]], 1, 0.1)
        tw.adamw_step([a, b], g, 1, 0.1, out=[tw.AdamTensors(a.p, c.m, a.v, a.m_scale, c.v_scale), d])
        calls.clear()
