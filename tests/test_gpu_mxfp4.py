"""MXFP4 expert weights: the conversion against its definition in numpy, and the layer on them
against the float64 oracle on the same (expanded, hence exact) weights, with the BF16 bars of
tests/gpu_util.py: the products take exact BF16 weights, and round a and o no further than the BF16
layer does (a's remainder: tests/test_gpu_mxfp4_activation.py).
"""
import numpy as np
import pytest

import oracle
from mixture_experts_routed_dispatch_amd import inputs
from tests.gpu_util import BF16, bf16_dev, check, dev, device_inputs, np_of, say

pytestmark = pytest.mark.gpu
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    oracle.build(force=False)
    return moe


def quantized(bits):
    """What BF16 bit patterns [..., K] become in MXFP4, as float64: the definition, value by value."""
    v = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(-1, 32)
    top = np.abs(v).max(1, keepdims=True)
    with np.errstate(divide="ignore"):
        s = np.where(top > 0, np.ceil(np.log2(top / 6)), -126.0)
    s = np.where(top > 6 * 2.0 ** s, s + 1, np.where((top > 0) & (top <= 3 * 2.0 ** s), s - 1, s))
    s = np.clip(s, -126, 127)
    a = np.abs(v) / 2.0 ** s
    hi = np.searchsorted(GRID, a, side="left").clip(1, 7)
    lo = hi - 1
    dl, dh = a - GRID[lo], GRID[hi] - a
    pick = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return (np.sign(v) * GRID[pick] * 2.0 ** s).reshape(bits.shape)


def test_conversion_of_every_magnitude(moe):
    """Every finite BF16 pattern with an exponent of at least -100 as an element, below block
    maxima whose scale puts it everywhere on the grid, ties included."""
    import torch
    rng = np.random.default_rng(0)
    d, I, E = 512, 128, 4
    n13, n2 = E * 2 * I * d, E * d * I
    # a block: a maximum of random mantissa, the others from 2^-6 of it up to it
    e = rng.integers(40, 240, (n13 + n2) // 32)
    m = rng.integers(0, 128, e.shape)
    top = (e << 7 | m)
    el = top[:, None] - rng.integers(0, 7 * 128, (e.size, 32))
    at = rng.integers(0, 32, e.size)
    el[np.arange(e.size), at] = top
    el[rng.random(el.shape) < 0.02] = 0
    el[::97] = 0                                       # blocks of zeros
    bits = (el | (rng.integers(0, 2, el.shape) << 15)).astype(np.uint16).reshape(-1)
    w13, w2 = bits[:n13].reshape(E, 2 * I, d), bits[n13:].reshape(E, d, I)
    layer = moe.Layer(1, d, I, E, 1, precision=moe.MOE_MXFP4)
    packed = layer.prepare_weights(bf16_dev(w13), bf16_dev(w2))
    g13, g2 = layer.expand_weights(*packed)
    assert np.array_equal(np_of(g13), quantized(w13))
    assert np.array_equal(np_of(g2), quantized(w2))
    # values that are on the grid already keep themselves and their bytes
    again = layer.prepare_weights(g13, g2)
    h13, h2 = layer.expand_weights(*again)
    assert torch.equal(h13, g13) and torch.equal(h2, g2)
    # and the layout is the documented one: tile, piece, block, element
    codes, scales = packed[0].cpu().numpy(), packed[1].cpu().numpy()
    S = d // 128
    for e_, tile, s, q, n, i in rng.integers(0, [E, 2 * I // 16, S, 4, 16, 32], (300, 6)):
        row = 8 * tile + n if n < 8 else I + 8 * tile + n - 8
        byte = codes[e_, ((tile * S + s) * 64 + 16 * q + n) * 16 + i // 2]
        c = (byte >> (4 * (i & 1))) & 15
        x = 2.0 ** (float(scales[e_, tile, s // 4, 16 * q + n, s % 4]) - 127)
        assert float(g13[e_, row, 128 * s + 32 * q + i]) == (-1) ** (c >> 3) * GRID[c & 7] * x


@pytest.mark.parametrize("d,I,E", [(128, 128, 1), (384, 128, 3), (640, 384, 2), (2048, 768, 2)])
def test_conversion_shapes(moe, d, I, E):
    inp = inputs.generate(1, d, I, E, 1, "uniform", seed=d)
    layer = moe.Layer(1, d, I, E, 1, precision=moe.MOE_MXFP4)
    g13, g2 = layer.expand_weights(*layer.prepare_weights(bf16_dev(inp.w13), bf16_dev(inp.w2)))
    assert np.array_equal(np_of(g13), quantized(inp.w13))
    assert np.array_equal(np_of(g2), quantized(inp.w2))


def run4(moe, inp, path=0, act=0):
    import torch
    t = device_inputs(inp)
    layer = moe.Layer(inp.T, inp.d, inp.I, inp.E, inp.k, precision=moe.MOE_MXFP4, path=path, activation=act)
    packed = layer.prepare_weights(t["w13"], t["w2"])
    e13, e2 = layer.expand_weights(*packed)
    y = layer.forward(t["x"], t["ids"], t["scores"], packed[0], packed[2], packed[1], packed[3])
    torch.cuda.synchronize()
    assert layer.status() == (moe.MOE_OK, 0)
    return t, layer, packed, e13, e2, y


def bits_of(t):
    import torch
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


SHAPES = [(1, 256, 128, 8, 2), (1, 2048, 768, 128, 8), (1, 384, 640, 16, 5), (1, 128, 128, 40, 32), (1, 256, 128, 1, 1),
          (2, 256, 128, 8, 2), (7, 640, 384, 12, 3), (32, 2048, 768, 128, 8), (16, 4096, 256, 16, 4),
          (5, 1024, 2048, 16, 8), (256, 256, 128, 4, 1), (64, 256, 256, 6, 4), (32, 512, 128, 64, 8)]


@pytest.mark.parametrize("T,d,I,E,k", SHAPES)
def test_decode_against_the_oracle(moe, T, d, I, E, k):
    say("mxfp4 decode", T, d, I, E, k)
    inp = inputs.generate(T, d, I, E, k, "uniform", seed=T + d)
    t, layer, packed, e13, e2, y = run4(moe, inp)
    ref = oracle.forward_tokens(inp.x, inp.ids, inp.scores, bits_of(e13), bits_of(e2))
    check("y", np_of(y), ref, **BF16)


@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("T", [1, 20])
def test_decode_activations(moe, act, T):
    inp = inputs.generate(T, 256, 256, 8, 4, "uniform", seed=40 + act)
    t, layer, packed, e13, e2, y = run4(moe, inp, act=act)
    import torch
    full = moe.Layer(T, 256, 256, 8, 4, activation=act)
    ref = full.forward(t["x"], t["ids"], t["scores"], e13, e2)
    # the same roundings, another order of the FP32 sums: BF16 bars
    check("y", np_of(y), np_of(ref), **BF16)


def test_decode_with_all_tokens_on_one_expert(moe):
    """48 rows of one expert: three groups of 16 rows an item."""
    inp = inputs.generate(48, 256, 128, 8, 1, "uniform", seed=9)
    inp.ids[:] = 5
    t, layer, packed, e13, e2, y = run4(moe, inp)
    ref = oracle.forward_tokens(inp.x, inp.ids, inp.scores, bits_of(e13), bits_of(e2))
    check("y", np_of(y), ref, **BF16)


@pytest.mark.parametrize("T,d,I,E,k,path", [(300, 256, 128, 8, 2, 0), (64, 512, 256, 16, 8, 0), (9, 256, 128, 8, 2, 1),
                                            (1000, 2048, 768, 16, 8, 0)])
def test_prefill_is_the_bf16_layer_on_the_expanded_weights(moe, T, d, I, E, k, path):
    import torch
    inp = inputs.generate(T, d, I, E, k, "uniform", seed=T)
    t, layer, packed, e13, e2, y = run4(moe, inp, path=path)
    full = moe.Layer(T, d, I, E, k, path=moe.MOE_PATH_PREFILL)
    ref = full.forward(t["x"], t["ids"], t["scores"], e13, e2)
    assert torch.equal(y, ref)
    # rows in expert order
    m_indptr, gather, slots, probs = full.dispatch(t["ids"], t["scores"])
    rows = t["x"][gather.long()].contiguous()
    a = layer.forward_routed(rows, m_indptr, packed[0], packed[2], packed[1], packed[3])
    assert torch.equal(a, full.forward_routed(rows, m_indptr, e13, e2))


def test_invalid_routing_is_flagged_and_left_out(moe):
    import torch
    for T in (1, 6):
        inp = inputs.generate(T, 256, 128, 8, 4, "uniform", seed=3)
        t, layer, packed, e13, e2, y = run4(moe, inp)
        bad = t["ids"].clone()
        bad[0, 1] = 8
        a, s13, c, s2 = packed
        layer.forward(t["x"], bad, t["scores"], a, c, s13, s2)
        st, flags = layer.status()
        assert st == moe.MOE_ERR_ROUTING and flags & moe.MOE_DEV_ID_OUT_OF_RANGE
        y2 = layer.forward(t["x"], t["ids"], t["scores"], a, c, s13, s2)
        assert torch.equal(y, y2) and layer.status() == (moe.MOE_OK, 0)


def test_static_scratch_and_graph_replay(moe):
    import torch
    for T in (1, 3, 32):
        shapes = (T, 512, 256, 16, 4)
        inps = [inputs.generate(*shapes, "uniform", seed=s) for s in (1, 2, 3)]
        t, layer, packed, e13, e2, y0 = run4(moe, inps[0])
        a, s13, c, s2 = packed
        ins = [device_inputs(i) for i in inps]
        fwd = lambda i: layer.forward(i["x"], i["ids"], i["scores"], a, c, s13, s2)
        want = [fwd(i) for i in ins]
        assert torch.equal(want[0], y0)
        w = moe.weights(a.data_ptr(), c.data_ptr(), s13.data_ptr(), s2.data_ptr())
        ys = torch.empty_like(y0)
        i = ins[1]
        moe.moe_forward_static(layer.plan, i["x"].data_ptr(), i["ids"].data_ptr(), i["scores"].data_ptr(), w,
                               ys.data_ptr(), int(torch.cuda.current_stream().cuda_stream))
        assert torch.equal(ys, want[1])
        buf = {k: v.clone() for k, v in ins[0].items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fwd(buf)
        for j in (0, 1, 2, 0):
            for k in ("x", "ids", "scores"):
                buf[k].copy_(ins[j][k])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[j])
            assert torch.equal(fwd(ins[(j + 1) % 3]), want[(j + 1) % 3])


def test_weight_refusals(moe):
    import torch
    layer = moe.Layer(1, 256, 128, 2, 1, precision=moe.MOE_MXFP4)
    w13 = torch.zeros(2, 256, 256, dtype=torch.bfloat16, device=dev())
    w2 = torch.zeros(2, 256, 128, dtype=torch.bfloat16, device=dev())
    packed = layer.prepare_weights(w13, w2)
    for bad in (w13.float(), w13[:1], w13.transpose(1, 2)):
        with pytest.raises(ValueError):
            layer.prepare_weights(bad, w2)
    with pytest.raises(ValueError):
        layer.expand_weights(packed[0], packed[1][:, :1], packed[2], packed[3])
    with pytest.raises(moe.MoeError):
        layer.forward(torch.zeros(1, 256, dtype=torch.bfloat16, device=dev()),
                      torch.zeros(1, 1, dtype=torch.int32, device=dev()), torch.ones(1, 1, device=dev()), packed[0],
                      packed[2])                       # the scales are missing


def test_weights_of_other_shapes_are_refused(moe):
    """The kernels address the weights by the plan's sizes: codes and scales in the wrong places,
    another layer's, or tensors on the host never reach them."""
    import torch
    for T, path in ((1, 0), (4, 0), (4, moe.MOE_PATH_PREFILL)):
        layer = moe.Layer(T, 256, 128, 4, 2, precision=moe.MOE_MXFP4, path=path)
        w = [torch.zeros(4, 256, 256, dtype=torch.bfloat16, device=dev()), torch.zeros(4, 256, 128, dtype=torch.bfloat16, device=dev())]
        w13, s13, w2, s2 = layer.prepare_weights(*w)
        x = torch.zeros(T, 256, dtype=torch.bfloat16, device=dev())
        ids = torch.tensor([[0, 3]] * T, dtype=torch.int32, device=dev())
        scores = torch.ones(T, 2, device=dev())
        good = (x, ids, scores, w13, w2, s13, s2)
        assert not layer.forward(*good).any()
        for at, bad in ((3, s13), (4, w13), (5, w2), (6, s2[:1]), (3, w13[:3]), (4, w2.cpu()), (0, x.cpu()), (2, scores.cpu()),
                        (3, w13[:1].expand(4, -1))):
            args = list(good)
            args[at] = bad
            with pytest.raises(ValueError):
                layer.forward(*args)
        if path:
            rows = torch.zeros(2 * T, 256, dtype=torch.bfloat16, device=dev())
            m_indptr = torch.zeros(5, dtype=torch.int32, device=dev())
            with pytest.raises(ValueError):
                layer.forward_routed(rows, m_indptr, w13, s13, w2, s2)


@pytest.mark.parametrize("T", [1, 2, 6, 32])
def test_entries_of_invalid_ids_add_nothing(moe, T):
    """y of a batch with ids out of range is that of the same batch with their scores 0, whatever an
    earlier call left in the workspace (here NaN in every word)."""
    import torch
    inp = inputs.generate(T, 256, 128, 16, 4, "uniform", seed=3)
    t, layer, packed, e13, e2, y = run4(moe, inp)
    a, s13, c, s2 = packed
    bad, scores = t["ids"].clone(), t["scores"].clone()
    bad[0, 1], bad[-1, 3], bad[T // 2, 0] = 16, -1, 1 << 30
    scores[0, 1] = scores[-1, 3] = scores[T // 2, 0] = 0
    want = layer.forward(t["x"], t["ids"], scores, a, c, s13, s2)
    layer.workspace.fill_(255)
    torch.cuda.synchronize()
    moe.moe_bind_workspace(layer.plan, layer.workspace.data_ptr(), layer.workspace.numel())
    got = layer.forward(t["x"], bad, t["scores"], a, c, s13, s2)
    assert torch.equal(got, want)
    assert layer.status() == (moe.MOE_ERR_ROUTING, moe.MOE_DEV_ID_OUT_OF_RANGE)
