"""What the W2 products of the MXFP4 decode make of a, the gated activation, whatever the number of
tokens: its BF16 rounding and the rounded remainder, two operand rows.

x is made of -1, 0 and 1 and W13 of E2M1 values times 2^-3, so that g and u are sums of multiples of
2^-4 below 2^7: exact in FP32, and so is a = max(g, 0) u (ReGLU), of up to 22 bits.  With u = 2^-24:
  a as two operands is off by at most 2^-8 2^-8 |a| (a half step of the remainder, itself a half
  step of a at most), a sum of 2 I products of them by 2 I u in whatever order, the k terms of y by
  2 k u, all relative to the sum of magnitudes M = sum_j s_j sum_i |a_ji w2_i|; y by a half step, 2^-8.
A single BF16 operand is off by up to 2^-8 |a|, which where y is small next to M is beyond that bar."""
import pytest

from tests.gpu_util import dev, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    return moe


def make(T, d, I, E, k, seed):
    import torch
    g = torch.Generator(device=dev()).manual_seed(seed)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=dev())
    ri = lambda hi, *s: torch.randint(0, hi, s, generator=g, device=dev())
    sign = lambda *s: 1.0 - 2.0 * ri(2, *s)
    w13 = (grid[ri(8, E, 2 * I, d)] * sign(E, 2 * I, d) / 8).bfloat16()
    w2 = (grid[ri(8, E, d, I)] * sign(E, d, I) / 16).bfloat16()
    x = (ri(3, T, d) - 1).bfloat16()
    ids = torch.rand(T, E, generator=g, device=dev()).argsort(1)[:, :k].int().contiguous()
    scores = torch.rand(T, k, generator=g, device=dev()) + 0.1
    return x, ids, scores, w13, w2


def exact(x, ids, scores, w13, w2):
    """(y, M) in 64 bits."""
    import torch
    I = w2.shape[2]
    y = torch.zeros(x.shape, dtype=torch.float64, device=dev())
    m = torch.zeros_like(y)
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = x[t].double() @ w13[e].double().T
        a = gu[:, :I].clamp(min=0) * gu[:, I:]
        s = scores[t, j].double()[:, None]
        y.index_add_(0, t, s * (a @ w2[e].double().T))
        m.index_add_(0, t, s * (a.abs() @ w2[e].double().abs().T))
    return y, m


# one group and several of an expert's rows, counts on both sides of 8 and of 16
SHAPES = [(1, 256, 128, 8, 4), (2, 256, 128, 8, 2), (7, 384, 640, 12, 3), (8, 256, 128, 1, 1), (9, 256, 128, 1, 1),
          (16, 128, 256, 1, 1), (17, 256, 128, 2, 1), (32, 512, 128, 64, 8), (32, 256, 128, 8, 8), (256, 256, 128, 4, 1)]


@pytest.mark.parametrize("T,d,I,E,k", SHAPES)
def test_activation_keeps_its_remainder(moe, T, d, I, E, k):
    import torch
    say("mxfp4 activation", T, d, I, E, k)
    x, ids, scores, w13, w2 = make(T, d, I, E, k, 7 * T + I)
    layer = moe.Layer(T, d, I, E, k, precision=moe.MOE_MXFP4, path=moe.MOE_PATH_DECODE, activation=moe.MOE_ACT_REGLU)
    packed = layer.prepare_weights(w13, w2)
    e13, e2 = layer.expand_weights(*packed)
    assert torch.equal(e13, w13) and torch.equal(e2, w2)
    y = layer.forward(x, ids, scores, packed[0], packed[2], packed[1], packed[3])
    assert layer.status() == (moe.MOE_OK, 0)
    ref, m = exact(x, ids, scores, w13, w2)
    bar = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + (2 * I + 2 * k) * 2.0 ** -24) * m
    over = (y.double() - ref).abs() / bar
    print("  largest share of the bar: %.2f" % float(over.max()), flush=True)
    assert (over <= 1).all(), float(over.max())
