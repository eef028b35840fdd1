"""Host checks of the products and of the layer on weights in blocks of 128 at the edges of their use."""
import pytest

from mixture_experts_routed_dispatch_amd import moe
from tests.test_block128_abi import BAD, L, OK, P, ROOM, STATE, product  # noqa: F401


def test_gradients_of_no_rows(L):
    """With no rows the input gradient is empty: its pointer, like those of dy, x and the weights, may be null.  Nothing is
    launched for it."""
    import ctypes
    call = lambda c, dx=None, dw=None, ws=None, nbytes=0: L.moe_product_backward(
        ctypes.byref(c), None, None, None, None, None, dx, dw, None, ws, nbytes, None)
    for E in (1, 2):
        for add in (0, 1):
            c = product(R=0, E=E, wgrad_accumulate=add)
            assert call(c) == OK and call(c, dx=P) == OK
            assert call(c, dw=P) == ROOM and call(c, dw=P + 8) == BAD
    assert call(product(R=0, training=0)) == STATE
    assert call(product(R=8)) == BAD and call(product(R=0, N=100)) != OK


def test_tensors_of_the_layer(monkeypatch):
    """x, ids, scores and y (x_rows, m_indptr and out) of another type, size or order are refused before the call;
    batches of several axes, and flat ones, are not."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)           # the "device" of CPU tensors
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    called = []
    monkeypatch.setattr(moe, "moe_forward", lambda *a: called.append("forward"))
    monkeypatch.setattr(moe, "moe_forward_routed", lambda *a: called.append("routed"))
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    T, d, I, E, k = 6, 256, 128, 4, 2
    layer = moe.Layer.__new__(moe.Layer)
    layer.plan, layer.precision, layer._mxfp4, layer._rows = 0, moe.MOE_FP8_BLOCK128, None, moe._dense(T, d)
    layer.T, layer.d, layer.I, layer.E, layer.k = T, d, I, E, k
    layer._weights = moe._dense(E, 2 * I, d), moe._dense(E, d, I)
    layer._set_block128()
    w = [torch.zeros(E, 2 * I, d, dtype=torch.uint8), torch.zeros(E, d, I, dtype=torch.uint8),
         torch.zeros(E, 2 * I // 128, d // 128), torch.zeros(E, d // 128, I // 128)]
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = dict(x=bf(T, d), ids=i32(T, k), scores=torch.zeros(T, k), y=bf(T, d))
    forward = lambda **c: layer.forward(*[dict(good, **c)[n] for n in ("x", "ids", "scores")], *w, y=dict(good, **c)["y"])
    routed = dict(x_rows=bf(T * k, d), m_indptr=i32(E + 1), out=bf(T * k, d))
    forward_routed = lambda **c: layer.forward_routed(*[dict(routed, **c)[n] for n in ("x_rows", "m_indptr")], *w,
                                                      out=dict(routed, **c)["out"])
    forward()
    forward_routed()
    forward(x=bf(2, 3, d), ids=i32(2, 3, k), scores=torch.zeros(2, 3, k), y=bf(3, 2, d))
    forward(x=bf(T * d), ids=i32(T * k), scores=torch.zeros(T * k), y=None)
    forward_routed(x_rows=bf(T, k, d), out=None)
    forward_routed(x_rows=bf(T, d), out=bf(T, d))        # rows of segments that end there
    assert called == ["forward", "routed", "forward", "forward", "routed", "routed"]
    del called[:]
    for f, name, tensors in (
            (forward, "x", [torch.zeros(T, d), bf(T, d).half(), bf(d, T).t(), bf(T, 2 * d)[:, ::2], bf(T + 1, d), bf(T - 1, d),
                            bf(T, d // 2), bf(d, T)]),
            (forward, "ids", [torch.zeros(T, k, dtype=torch.int64), i32(k, T).t(), i32(T, k + 1), i32(T, 1), i32(k, T), torch.zeros(T, k)]),
            (forward, "scores", [bf(T, k), torch.zeros(T, k).double(), torch.zeros(k, T).t(), torch.zeros(T, k + 1)[:, :k], torch.zeros(T)]),
            (forward, "y", [torch.zeros(T, d), bf(T + 1, d), bf(T, 2 * d)[:, :d], bf(T - 1, d)]),
            (forward_routed, "x_rows", [torch.zeros(T * k, d), bf(d, T * k).t(), bf(T * k, 2 * d), bf(T * k, 2 * d)[:, :d]]),
            (forward_routed, "m_indptr", [i32(E), torch.zeros(E + 1, dtype=torch.int64), i32(2 * E + 2)[::2]]),
            (forward_routed, "out", [torch.zeros(T * k, d), bf(d, T * k).t(), bf(2 * T * k, d // 2)])):
        for t in tensors:
            with pytest.raises(ValueError, match="^" + name + ": "):
                f(**{name: t})
    assert not called


def test_structs_of_the_binding_are_those_of_the_header(tmp_path):
    """The library reads structs of the header's size: the binding's have that size, field by field."""
    import ctypes
    import os
    import subprocess
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    pairs = [("moe_config_t", moe.MoeConfig), ("moe_weights_t", moe.MoeWeights), ("moe_router_config_t", moe.RouterConfig),
             ("moe_norm_config_t", moe.NormConfig), ("moe_product_config_t", moe.ProductConfig)]
    lines = []
    for c, py in pairs:
        lines.append('printf("%%d\\n", (int)sizeof(%s));' % c)
        lines += ['printf("%%d\\n", (int)offsetof(%s, %s));' % (c, f[0]) for f in py._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "moe.h"\nint main(void) { %s return 0; }\n' % " ".join(lines))
    subprocess.run(["gcc", "-I", include, str(src), "-o", str(tmp_path / "sizes")], check=True)
    out = list(map(int, subprocess.run([str(tmp_path / "sizes")], check=True, capture_output=True, text=True).stdout.split()))
    want = []
    for _, py in pairs:
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f[0]).offset for f in py._fields_]
    assert out == want and ctypes.sizeof(moe.RouterConfig) == 44
