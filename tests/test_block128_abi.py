"""Host checks of weights in blocks of 128 (products and the layer on them) and of the router's groups:
configs and arguments that are refused before anything reaches a device, plans, streams of another device."""
import ctypes
import types

import pytest

from mixture_experts_routed_dispatch_amd import moe

P = 0x1000          # an aligned address that no refused call may touch
OK, BAD, NO, ROOM, STATE = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_ERR_STATE


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from mixture_experts_routed_dispatch_amd import build
        build.build()
    return moe.lib()


def product(R=8, N=256, K=128, E=2, training=1, wgrad_accumulate=0):
    return moe.ProductConfig(R, N, K, E, training, wgrad_accumulate)


# ------------------------------------------------------------------ products

@pytest.mark.parametrize("change,expect", [
    (dict(R=-1), BAD), (dict(N=0), BAD), (dict(K=-128), BAD), (dict(E=0), BAD), (dict(training=2), BAD),
    (dict(wgrad_accumulate=-1), BAD), (dict(N=64), NO), (dict(N=200), NO), (dict(K=192), NO), (dict(E=257), NO),
    (dict(training=0, wgrad_accumulate=1), NO), (dict(R=(1 << 24) + 1, training=0), NO),
    (dict(N=1 << 16, K=1 << 15), NO), (dict(R=1 << 18, N=1 << 14, E=1), NO)])
def test_product_configs(L, change, expect):
    c = ctypes.byref(product(**change))
    assert L.moe_product_workspace_bytes(c) == 0
    assert L.moe_product_forward(c, P, P, P, P, P, P, P, 1 << 40, None) == expect
    assert L.moe_product_backward(c, P, P, P, P, P, P, P, P, P, 1 << 40, None) == expect
    assert L.moe_product_prepare_weights(c, P, P, P, None) == expect
    assert L.moe_product_expand_weights(c, P, P, P, None) == expect


def test_product_limits(L):
    need = lambda **c: L.moe_product_workspace_bytes(ctypes.byref(product(**c)))
    assert need(R=1 << 24, training=0) > 0 and need(R=0) > 0
    assert need(N=1 << 15, K=(1 << 16) - 128, E=1) > 0
    assert need(R=(1 << 18) - 256, N=1 << 14, E=1) > 0
    # the forward's workspace is x in 8 bits, its scales and the few rows' order
    assert need(R=1 << 20, N=256, K=512, training=0) <= (1 << 20) * (512 + 16) + (1 << 17)
    assert L.moe_product_workspace_bytes(None) == 0


def test_product_arguments(L):
    c = product()
    need = L.moe_product_workspace_bytes(ctypes.byref(c))
    names = ("x", "m", "w_q", "w_s", "y", "status", "ws")

    def forward(c=c, nbytes=need, **change):
        a = dict.fromkeys(names, P)
        a.update(change)
        return L.moe_product_forward(ctypes.byref(c), *[a[n] for n in names], nbytes, None)

    for n in ("x", "m", "w_q", "w_s", "y"):
        assert forward(**{n: None}) == BAD, n
    for n in ("x", "w_q", "y", "ws"):
        assert forward(**{n: P + 8}) == BAD, n
    assert forward(w_s=P + 2) == BAD
    assert forward(ws=None) == ROOM and forward(nbytes=need - 1) == ROOM
    assert L.moe_product_forward(None, P, P, P, P, P, P, P, need, None) == BAD
    # no rows: nothing is read, written or launched
    assert forward(product(R=0), x=None, m=None, w_q=None, w_s=None, y=None, ws=None) == OK

    names2 = ("dy", "x", "m", "w_q", "w_s", "dx", "dw", "status", "ws")

    def backward(c=c, nbytes=need, **change):
        a = dict.fromkeys(names2, P)
        a.update(change)
        return L.moe_product_backward(ctypes.byref(c), *[a[n] for n in names2], nbytes, None)

    for n in ("dy", "x", "m", "w_q", "w_s"):
        assert backward(**{n: None}) == BAD, n
    for n in ("dy", "x", "w_q", "dx", "dw", "ws"):
        assert backward(**{n: P + 8}) == BAD, n
    assert backward(w_s=P + 2) == BAD and backward(dx=None, dw=None) == BAD
    assert backward(ws=None) == ROOM and backward(nbytes=need - 1) == ROOM
    assert backward(product(training=0)) == STATE
    assert L.moe_product_backward(None, P, P, P, P, P, P, P, P, P, need, None) == BAD


def test_conversion_arguments(L):
    q = lambda *a: L.moe_quantize_block128(*a, None)
    assert q(P, -1, 128, P, P) == BAD and q(P, 4, 0, P, P) == BAD and q(P, 4, 192, P, P) == BAD
    assert q(None, 4, 128, P, P) == BAD and q(P, 4, 128, None, P) == BAD and q(P, 4, 128, P, None) == BAD
    assert q(P + 8, 4, 128, P, P) == BAD and q(P, 4, 128, P + 8, P) == BAD and q(P, 4, 128, P, P + 2) == BAD
    c = ctypes.byref(product(training=0))
    for f, a in ((L.moe_product_prepare_weights, (16, 16, 4)), (L.moe_product_expand_weights, (16, 4, 16))):
        for i in range(3):
            args = [P] * 3
            for bad in (None, P + a[i] // 2):
                args[i] = bad
                assert f(c, *args, None) == BAD
        assert f(None, P, P, P, None) == BAD


def test_python_checks_of_products(monkeypatch):
    import torch
    for bad, status in ((dict(R=4, N=100, K=128), NO), (dict(R=-4, N=128, K=128), BAD),
                        (dict(R=4, N=128, K=128, wgrad_accumulate=True), NO)):
        with pytest.raises(moe.MoeError) as e:
            moe.Product(**bad)
        assert e.value.status == status
    cpu = torch.device("cpu")
    p = moe.Product.__new__(moe.Product)
    p.R, p.N, p.K, p.E, p.device, p._index = 4, 256, 128, 2, cpu, 0
    p._in, p._out, p._weights, p._scales = moe._dense(4, 128), moe._dense(4, 256), moe._dense(2, 256, 128), moe._dense(2, 2, 1)
    p._cfg = product(R=4, wgrad_accumulate=1)
    p._call = lambda f, stream, *a: "called"
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    x, dy, w = bf(4, 128), bf(4, 256), bf(2, 256, 128)
    q, s, m = torch.zeros(2, 256, 128, dtype=torch.uint8), torch.zeros(2, 2, 1), torch.zeros(3, dtype=torch.int32)
    good = dict(x=x, w_q=q, w_s=s, m_indptr=m)
    assert p.forward(**good) == "called" and p.forward(**dict(good, w_q=q.view(torch.float8_e4m3fn))) == "called"
    for name, t in (("x", x.float()), ("x", x[:, :64]), ("x", bf(5, 128)), ("x", bf(128, 4).t()), ("w_q", q.view(torch.int8)),
                    ("w_q", q[:1]), ("w_q", q.view(torch.float8_e5m2)), ("w_s", s.double()), ("w_s", s[0]), ("m_indptr", m.long()),
                    ("m_indptr", m[:2]), ("y", bf(4, 255))):
        with pytest.raises(ValueError, match=name + ": "):
            p.forward(**dict(good, **{name: t}))
    back = dict(good, dy=dy, dw=w)
    assert p.backward(**back) == "called" and p.backward(**dict(back, dw=None), need_dw=False) == "called"
    for name, t in (("dy", x), ("dx", dy), ("dw", w.float()), ("x", x.half()), ("w_s", s.half())):
        with pytest.raises(ValueError, match=name + ": "):
            p.backward(**dict(back, **{name: t}))
    with pytest.raises(ValueError, match="dw: "):
        p.backward(**dict(back, dw=None))
    with pytest.raises(ValueError, match="w: "):
        p.prepare_weights(w.float())


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("cfg,expect", [
    (dict(T=8, d=256, I=128, E=8, k=2), OK), (dict(T=300, d=384, I=640, E=8, k=2), OK),
    (dict(T=0, d=256, I=128, E=8, k=2), OK), (dict(T=8, d=256, I=128, E=8, k=2, path=1), OK),
    (dict(T=8, d=192, I=128, E=8, k=2), NO), (dict(T=8, d=256, I=64, E=8, k=2), NO),
    (dict(T=8, d=256, I=128, E=8, k=2, training=1), NO), (dict(T=8, d=256, I=128, E=8, k=2, mega=1), NO),
    (dict(T=64, d=256, I=128, E=8, k=8, path=2), NO), (dict(T=8, d=256, I=128, E=257, k=2), NO)])
def test_layer_plans(L, cfg, expect):
    T, d, I, E, k = (cfg[n] for n in ("T", "d", "I", "E", "k"))
    c = moe.MoeConfig(T, d, I, E, k, moe.MOE_FP8_BLOCK128, cfg.get("training", 0), cfg.get("path", 0), 0, 0, 0, cfg.get("mega", 0))
    h = ctypes.c_void_p()
    assert L.moe_plan(ctypes.byref(c), ctypes.byref(h)) == expect
    if expect != OK:
        return
    text = moe.moe_plan_explain(h.value)
    assert "E4M3 with a scale per 128" in text
    decode = 0 < T * k <= 256 and cfg.get("path", 0) != 1
    if T:
        assert ("expert outputs [R, d] FP32" in text) == decode and ("16-bit integers" in text) == (not decode)
        w = moe.weights(P, P)
        assert L.moe_forward(h, P, P, P, ctypes.byref(w), P, None) == BAD              # no scales
        assert L.moe_forward_routed(h, P, P, ctypes.byref(w), P, None) == (NO if decode else BAD)
        for i in range(4):                               # 16-byte alignment of codes, scales, x and y
            w = moe.weights(*[P + 8 * (i == j) for j in range(4)])
            assert L.moe_forward(h, P, P, P, ctypes.byref(w), P, None) == BAD
            assert L.moe_expand_weights(h, ctypes.byref(w), P, P, None) == BAD
        w = moe.weights(P, P, P, P)
        assert L.moe_forward(h, P + 8, P, P, ctypes.byref(w), P, None) == BAD
        assert L.moe_forward(h, P, P, P, ctypes.byref(w), P + 8, None) == BAD
        assert L.moe_forward(h, P, P, P, ctypes.byref(w), P, None) == ROOM
        assert L.moe_backward(h, P, P, ctypes.byref(w), P, P, P, P, None) != OK
    assert L.moe_prepare_weights(h, P, P, P + 8, P, P, P, None) == BAD
    assert L.moe_prepare_weights(h, P, P, P, None, P, P, None) == BAD
    assert L.moe_prepare_weights_backward(h, P, P, P, P, P, P, None) != OK
    L.moe_plan_destroy(h)


class Stop(Exception):
    """Raised in place of a launch."""


def test_streams_and_tensors_of_another_device(monkeypatch):
    import torch

    def stop(*a, **k):
        raise Stop

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stop)
    stream = lambda i: types.SimpleNamespace(device=torch.device("cuda", i), cuda_stream=0x1000)
    p = moe.Product.__new__(moe.Product)
    p.device, p._index = torch.device("cuda", 0), 0
    with pytest.raises(ValueError, match="cuda:1"):
        p._call(stop, stream(1))
    with pytest.raises(Stop):
        p._call(stop, stream(0))
    layer = moe.Layer.__new__(moe.Layer)
    layer.plan, layer.precision = 0, moe.MOE_FP8_BLOCK128
    layer.T, layer.E, layer.I, layer.d, layer.k = 2, 4, 128, 256, 2
    layer._rows, layer._mxfp4 = moe._dense(2, 256), None
    layer._weights = moe._dense(4, 256, 256), moe._dense(4, 256, 128)
    layer._block128 = (4, 2, 2), (4, 2, 1)
    for name in ("moe_forward", "moe_forward_routed", "moe_prepare_weights", "moe_expand_weights"):
        monkeypatch.setattr(moe, name, stop)

    def t(shape=(2, 256), dtype=torch.bfloat16, index=0, contiguous=True):
        return types.SimpleNamespace(shape=shape, dtype=dtype, is_contiguous=lambda: contiguous, get_device=lambda: index,
                                     device=torch.device("cuda", index), data_ptr=lambda: 0x1000)

    monkeypatch.setattr(moe, "_new", lambda *a: t())
    u8 = torch.uint8
    w = [t((4, 256, 256), u8), t((4, 256, 128), torch.float8_e4m3fn), t((4, 2, 2), torch.float32), t((4, 2, 1), torch.float32)]
    calls = [lambda s, w=w, x=t(): layer.forward(x, t(), t(), *w, y=t(), stream=s),
             lambda s, w=w, x=t(): layer.forward(x, t(), t(), *w, stream=s),
             lambda s, w=w, x=t(): layer.forward_routed(x, t(), *w, stream=s),
             lambda s, w=w, x=t(): layer.expand_weights(w[0], w[2], w[1], w[3], stream=s)]
    for f in calls:
        with pytest.raises(ValueError, match="cuda:1"):
            f(stream(1))
        with pytest.raises(Stop):
            f(stream(0))
        for i, other in ((0, dict(dtype=torch.int8)), (0, dict(index=1)), (1, dict(shape=(4, 128, 256))), (1, dict(contiguous=False)),
                         (2, dict(dtype=torch.float16)), (3, dict(shape=(4, 1, 2))), (3, dict(index=1))):
            bad = list(w)
            bad[i] = t(**dict(dict(shape=w[i].shape, dtype=w[i].dtype), **other))
            with pytest.raises(ValueError, match=("w13_q", "w2_q", "w13_s", "w2_s")[i]):
                f(stream(0), w=bad)
    for f in calls[:3]:
        with pytest.raises(ValueError, match="elsewhere"):
            f(stream(0), x=t(index=1))
    monkeypatch.setattr(moe, "_check", lambda *a: None)
    with pytest.raises(ValueError, match="cuda:1"):
        layer.prepare_weights(t(), t(), stream=stream(1))
    with pytest.raises(Stop):
        layer.prepare_weights(t(), t(), stream=stream(0))


# ------------------------------------------------------------------ the router's groups

def router(groups, top_groups, group_top, E=64, k=4):
    return moe.RouterConfig(8, E, k, 0, 1, 1, 1.0, 0.0, groups, top_groups, group_top)


@pytest.mark.parametrize("cfg,expect", [
    ((-1, 1, 1), BAD), ((0, 1, 0), BAD), ((0, 0, 1), BAD), ((8, 0, 1), BAD), ((8, 9, 1), BAD), ((8, 4, 0), BAD), ((8, 4, 3), BAD),
    ((8, -4, 1), BAD), ((7, 4, 1), NO), ((64, 8, 1), NO), ((32, 2, 2, 32, 2), NO), ((8, 1, 1, 64, 9), NO), ((16, 1, 2, 64, 5), NO)])
def test_router_groups(L, cfg, expect):
    c = ctypes.byref(router(*cfg))
    assert L.moe_router_workspace_bytes(c) == 0
    assert L.moe_router_forward(c, P, None, None, P, P, P, P, P, P, 1 << 20, None) == expect
    assert L.moe_router_backward(c, P, P, None, P, P, P, P, None) == expect
    with pytest.raises(moe.MoeError) as e:
        g, t, n = cfg[:3]
        moe.Router(8, *(cfg[3:] or (64, 4)), groups=g, top_groups=t, group_top=n)
    assert e.value.status == expect


def test_router_groups_limits(L):
    for cfg in ((8, 8, 2), (1, 1, 1), (32, 2, 2), (8, 1, 1, 64, 8), (32, 32, 1, 32, 32), (2, 1, 2, 4, 2)):
        assert L.moe_router_workspace_bytes(ctypes.byref(router(*cfg))) > 0, cfg
