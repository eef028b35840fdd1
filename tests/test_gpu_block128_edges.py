"""Weights in blocks of 128 at the edges of their use: empty batches, numbers that are not finite, outputs of
unlike size, arguments of wrong form, the status word, operands that end with their memory.  Layers are held to the
bounds that tests/test_gpu_block128.py derives."""
import pytest

from tests.gpu_util import dev, say
from tests.test_gpu_block128 import INF, NAN, layer_case, moe, randn, routing, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("need", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("E", [1, 3])
def test_gradients_of_no_rows(moe, need, E):
    """A batch of no tokens: an empty dx, and dW of zeros (or as it was, where gradients are added up)."""
    import torch
    for add in (False, True):
        p = moe.Product(0, 256, 128, E=E, training=True, wgrad_accumulate=add)
        w_q, w_s = p.prepare_weights(randn(0, E, 256, 128))
        x = torch.empty(0, 128, dtype=torch.bfloat16, device=dev())
        dy = torch.empty(0, 256, dtype=torch.bfloat16, device=dev())
        m = torch.zeros(E + 1, dtype=torch.int32, device=dev()) if E > 1 else None
        before = randn(1, E, 256, 128)
        dx, dw = p.backward(dy, x, w_q, w_s, m_indptr=m, dw=before.clone(), need_dx=need[0], need_dw=need[1])
        assert dx.shape == (0, 128) if need[0] else dx is None
        if need[1]:
            assert torch.equal(dw, before) if add else (dw == 0).all()
        else:
            assert dw is None


@pytest.mark.parametrize("R,N,K,E", [(70, 128, 256, 1), (300, 256, 384, 3), (4099, 256, 128, 1)])
def test_not_finite_rows_reach_the_weight_gradient(moe, R, N, K, E):
    """An infinity or NaN of dy makes its matrix' row of dW NaN, one of x its column, and nothing else; rows behind
    the last segment are not read."""
    import torch
    say("not finite", R, N, K, E)
    p = moe.Product(R, N, K, E=E, training=True)
    x, dy, w = randn(R, R, K), randn(R + 1, R, N, std=0.1), randn(N, E, N, K)
    w_q, w_s = p.prepare_weights(w)
    m = torch.tensor([0, R - 5, R - 5, R - 2][:E] + [R - 2], dtype=torch.int32, device=dev())
    good = [p.backward(dy, x, w_q, w_s, m_indptr=m), (None, p.backward(dy, x, None, None, m_indptr=m, need_dx=False)[1])]
    assert torch.equal(good[0][1], good[1][1])
    last = R - 6                                         # in matrix 0, in its last block of 32 rows
    dy[1, 3], dy[40, 77], dy[last, N - 1], dy[33, N - 2] = NAN, INF, -INF, -NAN
    x[0, K - 1], x[35, 64], x[last, 5] = -INF, NAN, INF
    dy[R - 1, 9], x[R - 2, 9] = NAN, INF
    bad = torch.zeros(E, N, K, dtype=torch.bool, device=dev())
    for n in (3, 77, N - 1, N - 2):
        bad[0, n] = True
    for k in (K - 1, 64, 5):
        bad[0, :, k] = True
    bad_dx = torch.zeros(R, K, dtype=torch.bool, device=dev())
    for r in (1, 40, 33, last):
        bad_dx[r] = True
    dx, dw = p.backward(dy, x, w_q, w_s, m_indptr=m)
    _, only = p.backward(dy, x, None, None, m_indptr=m, need_dx=False)
    for got in (dw, only):
        assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], good[0][1][~bad])
    live = slice(0, R - 2)
    assert torch.equal(dx[live].isnan(), bad_dx[live]) and torch.equal(dx[live][~bad_dx[live]], good[0][0][live][~bad_dx[live]])


@pytest.mark.parametrize("T,k", [(20, 2), (400, 2)])
@pytest.mark.parametrize("power", [8, 12])
def test_columns_beside_a_large_one(moe, T, k, power):
    """One output in every 128 is 2^power the others' size: the others are as exact as without it, on either path.  (FP16
    in units of a power of two is off by at most 2^-11 of each value: 2^-12 of the norm, where the bound leaves 1.5e-3.)"""
    import torch
    from tests import block128_ref as ref
    d, I, E = 384, 256, 8
    layer, x, ids, scores, p = layer_case(moe, T, d, I, E, k)
    w2 = randn(77, E, d, I, std=I ** -0.5)
    w2[:, 37::128] *= 2.0 ** power
    _, _, q2, s2 = layer.prepare_weights(randn(78, E, 2 * I, d, std=d ** -0.5), w2)
    y = layer.forward(x, ids, scores, p[0], q2, p[1], s2)
    want = ref.layer(x, ids, scores, ref.matrix(p[0], p[1]), ref.matrix(q2, s2))
    small = torch.ones(d, dtype=torch.bool, device=dev())
    small[37::128] = False
    for cols in (small, ~small):
        a, b = y[:, cols].double(), want[:, cols]
        rel = float((a - b).norm() / b.norm())
        say("  T %d, 2^%d: rel %.2e" % (T, power, rel))
        assert rel <= 2.5e-3


def test_the_status_word_is_clear_before_the_first_call(moe):
    """A flag that a call on another stream sets right after the object was made stays set, however late the stream
    is that the object was made on."""
    import torch
    x, m = randn(0, 300, 128), torch.tensor([0, 200, 100, 300], dtype=torch.int32, device=dev())
    first = moe.Product(300, 128, 128, E=3)
    w_q, w_s = first.prepare_weights(randn(1, 3, 128, 128))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                        # some 10 ms of the current stream
    p = moe.Product(300, 128, 128, E=3)
    y = torch.empty(300, 128, dtype=torch.bfloat16, device=dev())
    p.forward(x, w_q, w_s, m_indptr=m, y=y, stream=side)
    assert p.status() == (moe.MOE_ERR_ROUTING, moe.MOE_DEV_BAD_INDPTR)
    assert p.status() == (moe.MOE_OK, 0)
    # and one right after the word was read and cleared
    p.forward(x, w_q, w_s, m_indptr=m, y=y, stream=side)
    p.status()
    p.forward(x, w_q, w_s, m_indptr=m, y=y, stream=side)
    assert p.status() == (moe.MOE_ERR_ROUTING, moe.MOE_DEV_BAD_INDPTR)


def test_products_are_made_before_a_capture(moe):
    """Made while its stream is captured, a product's clear of the status word would be replayed with every graph."""
    import torch
    p = moe.Product(4, 128, 128)
    x, (w_q, w_s) = randn(0, 4, 128), p.prepare_weights(randn(1, 1, 128, 128))
    want = p.forward(x, w_q, w_s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captur"):
            moe.Product(4, 128, 128)
        y = p.forward(x, w_q, w_s)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def last_of(t):
    """t at the end of a buffer, NaN (all bits set) right before and behind it."""
    import torch
    n = t.numel()
    room = torch.full((n + 8192,), -1, dtype=torch.int16, device=dev()).view(torch.bfloat16)
    out = room[4096:4096 + n].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("K", [128, 256, 384, 640, 1152])
@pytest.mark.parametrize("R,E", [(1, 1), (1, 3), (2, 1), (2, 2), (3, 1), (19, 3)])
def test_few_rows_of_few_steps(moe, R, E, K):
    """Rows whose loads ahead, and whose last whole load, would pass their end: waves of no steps, of one, of a part of a
    load; a segment of all rows, empty ones around it."""
    import torch
    from tests import block128_ref as ref
    N = 256
    p = moe.Product(R, N, K, E=E)
    x = last_of(randn(R, R, K))
    w_q, w_s = p.prepare_weights(randn(K, E, N, K, std=K ** -0.5))
    for first in range(E):
        m = None if E == 1 else torch.tensor([0] * (first + 1) + [R] * (E - first), dtype=torch.int32, device=dev())
        y = p.forward(x, w_q, w_s, m_indptr=m)
        assert within(y, ref.rows_value(x), ref.matrix(w_q, w_s)[first])


@pytest.mark.parametrize("T,d,I,k", [(1, 128, 128, 1), (1, 384, 640, 1), (1, 640, 1152, 3), (2, 128, 128, 1), (2, 384, 128, 1)])
def test_decode_of_few_steps(moe, T, d, I, k):
    from tests import block128_ref as ref
    layer, x, ids, scores, p = layer_case(moe, T, d, I, 5, k)
    x = last_of(x)
    y = layer.forward(x, ids, scores, p[0], p[2], p[1], p[3])
    want = ref.layer(x, ids, scores, ref.matrix(p[0], p[1]), ref.matrix(p[2], p[3]))
    rel = float((y.double() - want).norm() / want.norm())
    say("  rel %.2e" % rel)
    assert rel <= 2.5e-3


def test_the_most_rows(moe):
    """2^24 rows, the last of them in a segment of their own: outputs and gradients equal those of a short call."""
    import torch
    R, N, K, n = 1 << 24, 128, 128, 700
    p, few = moe.Product(R, N, K, E=2, training=True), moe.Product(n, N, K, training=True)
    q, s = p.prepare_weights(randn(0, 2, N, K, std=K ** -0.5))
    x = torch.zeros(R, K, dtype=torch.bfloat16, device=dev())
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device=dev())
    x[-n:], dy[-n:] = randn(1, n, K), randn(2, n, N)
    m = torch.tensor([0, R - n, R], dtype=torch.int32, device=dev())
    y = p.forward(x, q, s, m_indptr=m)
    xs, dys, qs, ss = x[-n:].clone(), dy[-n:].clone(), q[1:].clone(), s[1:].clone()
    assert torch.equal(y[-n:], few.forward(xs, qs, ss)) and not y[:-n].any()
    del y
    dx, dw = p.backward(dy, x, q, s, m_indptr=m)
    a, b = few.backward(dys, xs, qs, ss)
    assert torch.equal(dx[-n:], a) and not dx[:-n].any()
    # The long product adds its rows up in five pieces.  700 rows are 11 steps of 64 and those pieces: up to 16 additions on
    # either side, each off by at most 2^-23 of the terms' magnitudes; so both may round to BF16 a step apart
    terms = dys.double().abs().T @ xs.double().abs() * 1.13          # (values in 8 bits are up to a sixteenth larger)
    err = (dw[1].double() - b[0].double()).abs()
    assert (dw[0] == 0).all() and bool((err <= 2.0 ** -7 * b[0].double().abs() + 32 * 2.0 ** -23 * terms).all())
    assert p.status() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("T,calls", [(256, 1), (24, 8), (1, 64)])
@pytest.mark.parametrize("act", [0, 2])
def test_decode_sums_hold_their_digits(moe, T, calls, act):
    """The activation's output in 8 bits, seen through W2 = 1: its codes are those of the sums in 64 bits.  FP32 sums of 2048
    terms are off by about 2^-23 of their rms; the borders between codes lie 2^-4 to 2^-3 of a value apart, so that 2^-19 of
    the elements of that size fall on the other side, and of those down to a sixteenth of it 2^-15.  (Sums off by 2^-16 move
    2^-9.3: 861 of 524288.)"""
    import torch
    from tests import block128_ref as ref
    d, E = 2048, 4
    layer = moe.Layer(T, d, d, E, 1, precision=moe.MOE_FP8_BLOCK128, activation=act)
    w13_q, w13_s, _, _ = layer.prepare_weights(randn(1, E, 2 * d, d, std=d ** -0.5), randn(2, E, d, d))
    one = torch.eye(d, device=dev()).expand(E, d, d).contiguous()
    w2_q = one.to(torch.float8_e4m3fn).view(torch.uint8)
    w2_s = torch.ones(E, d // 128, d // 128, device=dev())
    w13 = ref.matrix(w13_q, w13_s)
    moved = total = 0
    for seed in range(calls):
        x = randn(100 + seed, T, d)
        ids, scores = routing(seed, T, E, 1)
        y = layer.forward(x, ids, scores, w13_q, w2_q, w13_s, w2_s).double()
        xv = ref.rows_value(x)
        for e in range(E):
            t = (ids[:, 0] == e).nonzero()[:, 0]
            gu = xv[t] @ w13[e].T
            want = ref.rows_value(ref.act(act, gu[:, :d]) * gu[:, d:])
            # y rounds to BF16; a neighbouring code is a sixteenth of the value away at least
            moved += int(((y[t] - want).abs() > 2.0 ** -6 * want.abs()).sum())
            total += want.numel()
    say("  %d of %d elements moved" % (moved, total))
    assert moved <= total * 2.0 ** -15
