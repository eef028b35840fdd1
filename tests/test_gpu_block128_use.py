"""Weights in blocks of 128 and the router's groups as they are used: on streams, captured and replayed, several
calls at once, on static scratch, past 32-bit offsets, at the largest matrix, and together in one block.
Equal calls give equal bits; the block as a whole is held to 2e-2 of its norm in float64 (its 8-bit
operands are quantized alike in both, so that only borders crossed by BF16 roundings of h differ)."""
import pytest

from tests.gpu_util import dev, say
from tests.test_gpu_block128 import layer_case, moe, randn, routing, starts, within  # noqa: F401
from tests.test_gpu_streams import both, flat

pytestmark = pytest.mark.gpu


def products(moe, R, N, K, E, seed=0):
    p = moe.Product(R, N, K, E=E, training=True)
    q, s = p.prepare_weights(randn(seed, E, N, K, std=K ** -0.5))
    m = starts(seed + 1, R, E, total=R - 3) if E > 1 else None
    x, dy = randn(seed + 2, R, K), randn(seed + 3, R, N)
    return p, q, s, m, x, dy


def calls(moe):
    """(object, call on a stream) for each entry point, in each of its forms by size; of outputs the rows that are
    written (those behind the last segment are not)."""
    out = []
    for R, N, K, E in ((1, 512, 256, 1), (5, 256, 640, 3), (300, 256, 384, 1), (4096, 256, 128, 1), (1500, 384, 256, 4)):
        p, q, s, m, x, dy = products(moe, R, N, K, E, seed=R)
        live = R if m is None else int(m[-1])
        out.append((p, lambda st=None, p=p, x=x, q=q, s=s, m=m, n=live: p.forward(x, q, s, m_indptr=m, stream=st)[:n]))

        def backward(st=None, p=p, dy=dy, x=x, q=q, s=s, m=m, n=live):
            dx, dw = p.backward(dy, x, q, s, m_indptr=m, stream=st)
            return dx[:n], dw
        out.append((p, backward))
        out.append((p, lambda st=None, p=p, q=q, s=s: p.expand_weights(q, s, stream=st)))
    for T, E, k, G in ((1, 64, 4, 8), (300, 256, 8, 8), (3000, 60, 4, 6)):
        r = moe.Router(T, E, k, groups=G, top_groups=G // 2, group_top=2, balance_coef=0.01, score=moe.MOE_SCORE_SIGMOID)
        z, b = randn(T, T, E), randn(E, E).float() * 0.1
        out.append((r, lambda st=None, r=r, z=z, b=b: r.forward(z, bias=b, stream=st)))
    return out


def test_streams(moe):
    for o, f in calls(moe):
        say(type(o).__name__, getattr(o, "R", getattr(o, "T", None)))
        both(f)


def test_layer_on_a_stream(moe):
    for T in (1, 20, 400):
        layer, x, ids, scores, p = layer_case(moe, T, 256, 384, 8, 2)
        both(lambda s: layer.forward(x, ids, scores, p[0], p[2], p[1], p[3], stream=s))
        w13, w2 = both(lambda s: layer.expand_weights(*p, stream=s))
        both(lambda s: layer.prepare_weights(w13, w2, stream=s))


def test_streams_and_graphs_at_once(moe):
    import torch
    for o, f in calls(moe):
        say(type(o).__name__, getattr(o, "R", getattr(o, "T", None)))
        want = flat(f())
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                graphs.append((g, flat(f())))
        for _ in range(3):
            for _, out in graphs:
                for t in out:
                    t.zero_()
            torch.cuda.synchronize()
            for s, (g, out) in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
            got = [flat(f(streams[2])), flat(f())]
            torch.cuda.synchronize()
            for out in got + [out for _, out in graphs]:
                assert len(out) == len(want) and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T", [1, 24, 700])
def test_layer_captured_and_on_static_scratch(moe, T):
    import torch
    layer, x, ids, scores, p = layer_case(moe, T, 384, 256, 12, 3)
    cases = [(randn(50 + i, T, 384),) + routing(60 + i, T, 12, 3) for i in range(3)]
    run = lambda x, i, s: layer.forward(x, i, s, p[0], p[2], p[1], p[3])
    want = [run(*c) for c in cases]
    buf = [t.clone() for t in cases[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*buf)
    y = torch.zeros(T, 384, dtype=torch.bfloat16, device=dev())
    w = moe.weights(p[0].data_ptr(), p[2].data_ptr(), p[1].data_ptr(), p[3].data_ptr())
    for n in (0, 1, 2, 1):
        for a, b in zip(buf, cases[n]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[n])
        assert torch.equal(run(*cases[(n + 1) % 3]), want[(n + 1) % 3])
        a = cases[n]
        moe.moe_forward_static(layer.plan, a[0].data_ptr(), a[1].data_ptr(), a[2].data_ptr(), w, y.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
        assert torch.equal(y, want[n])


@pytest.mark.parametrize("R,N,K,E", [(4096, 256, 128, 1), (5000, 128, 384, 2), (2500, 256, 256, 1)])
def test_split_gradients(moe, R, N, K, E):
    """Rows cut into pieces: the gradient of each matrix equals that of the operands' values in float64, and adds
    to what is there; a matrix without rows keeps it.  (The pieces' sums are FP32, added in order.)"""
    import torch
    from tests import block128_ref as ref
    p, q, s, m, x, dy = products(moe, R, N, K, E, seed=R)
    if E > 1:
        m = torch.tensor([0, 0, R - 3], dtype=torch.int32, device=dev())
    at = [0, R] if m is None else m.tolist()
    dx, dw = p.backward(dy, x, q, s, m_indptr=m)
    again = p.backward(dy, x, q, s, m_indptr=m)[1]
    assert torch.equal(dw, again)
    more = moe.Product(R, N, K, E=E, training=True, wgrad_accumulate=True)
    before = randn(9, E, N, K)
    total = before.clone()
    more.backward(dy, x, q, s, m_indptr=m, dw=total)
    for e in range(E):
        a, b = at[e], at[e + 1]
        if a == b:
            assert (dw[e] == 0).all() and torch.equal(total[e], before[e])
            continue
        assert within(dw[e], ref.mx_columns(dy[a:b]).T.contiguous(), ref.mx_columns(x[a:b]).T.contiguous())
        assert torch.equal(total[e], (before[e].float() + dw[e].float()).bfloat16())


def test_rows_past_32_bits(moe):
    """Rows that start more than 2^32 elements into their tensors: the last ones equal those of a short call."""
    import torch
    from tests import block128_ref as ref
    R, K, N, n = 260000, 16384, 128, 700
    p, few = moe.Product(R, N, K, training=True), moe.Product(n, N, K, training=True)
    q, s = p.prepare_weights(randn(0, 1, N, K, std=K ** -0.5))
    x = torch.zeros(R, K, dtype=torch.bfloat16, device=dev())
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device=dev())
    x[-n:], dy[-n:] = randn(1, n, K), randn(2, n, N)
    y = p.forward(x, q, s)
    assert torch.equal(y[-n:], few.forward(x[-n:].clone(), q, s)) and (y[:-n] == 0).all()
    dx, _ = p.backward(dy, None, q, s, need_dw=False)
    assert torch.equal(dx[-n:], few.backward(dy[-n:].clone(), None, q, s, need_dw=False)[0])
    assert (dx[:R - n:1000] == 0).all()
    del dx, y
    # of the weights: blocks of 32 rows are counted from the segment's first
    two = moe.Product(R, N, K, E=2, training=True)
    m = torch.tensor([0, R - n, R], dtype=torch.int32, device=dev())
    q2, s2 = torch.cat([q, q]), torch.cat([s, s])
    _, dw = two.backward(dy, x, q2, s2, m_indptr=m, need_dx=False)
    assert (dw[0] == 0).all()
    assert within(dw[1], ref.mx_columns(dy[-n:]).T.contiguous(), ref.mx_columns(x[-n:]).T.contiguous())


def test_the_longest_matrix(moe):
    """N K just below 2^31: the last outputs, and the input gradient of them, equal those of a short matrix."""
    import torch
    N, K, R, n = (1 << 24) - 256, 128, 100, 512
    p, few = moe.Product(R, N, K, training=True), moe.Product(R, n, K, training=True)
    w = torch.zeros(1, N, K, dtype=torch.bfloat16, device=dev())
    w[0, -n:] = randn(0, n, K)
    q, s = p.prepare_weights(w)
    sq, ss = few.prepare_weights(w[:, -n:].clone())
    assert torch.equal(q[:, -n:], sq) and torch.equal(s[:, -n // 128:], ss)
    assert torch.equal(p.expand_weights(q, s)[:, -n:], few.expand_weights(sq, ss))
    del w
    x = randn(1, R, K)
    y = p.forward(x, q, s)
    assert torch.equal(y[:, -n:], few.forward(x, sq, ss)) and (y[:, :100000] == 0).all()
    y.zero_()
    y[:, -n:] = randn(2, R, n)
    dx, dw = p.backward(y, x, q, s)
    a, b = few.backward(y[:, -n:].contiguous(), x, sq, ss)
    assert torch.equal(dx, a) and torch.equal(dw[:, -n:], b)
    assert (dw[:, :100000] == 0).all()


@pytest.mark.parametrize("T,d,I,E,k", [(1, 256, 128, 16, 4), (30, 512, 256, 32, 4), (500, 384, 256, 16, 3)])
def test_together(moe, T, d, I, E, k):
    """norm, gate product, router with groups, layer, output product, norm: against float64 on the same ids."""
    import torch
    from tests import block128_ref as ref
    g = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=g).to(dev())
    w1, w2, bias, wg = 1 + 0.1 * rn(d), 1 + 0.1 * rn(d), 0.1 * rn(E), rn(E, d) * d ** -0.5
    norm = moe.BlockNorm(T, d, eps=1e-6)
    router = moe.Router(T, E, k, score=moe.MOE_SCORE_SIGMOID, groups=4, top_groups=2, group_top=2, scale=1.5)
    layer = moe.Layer(T, d, I, E, k, precision=moe.MOE_FP8_BLOCK128)
    packed = layer.prepare_weights(randn(1, E, 2 * I, d, std=d ** -0.5), randn(2, E, d, I, std=I ** -0.5))
    inner, outer = moe.Product(T, d, d), moe.Product(T, d, d)
    qi, qo = inner.prepare_weights(randn(3, 1, d, d, std=d ** -0.5)), outer.prepare_weights(randn(4, 1, d, d, std=d ** -0.5))

    def step(x):
        _, h = norm.forward(x, w_pre=w1)
        u = inner.forward(h, *qi)
        ids, scores, _, _, _ = router.forward(u.float() @ wg.T, bias=bias, stats=False)
        y = outer.forward(layer.forward(u, ids, scores, packed[0], packed[2], packed[1], packed[3]), *qo)
        z, out = norm.forward(x, y, w_pre=w2)
        return z, out, h, u, ids, scores, y

    xs = [rn(T, d).bfloat16() for _ in range(3)]
    eager = [step(x) for x in xs]
    assert layer.status() == (moe.MOE_OK, 0)
    mat = lambda a, b: ref.matrix(a, b)
    for x, (z, out, h, u, ids, scores, y) in zip(xs, eager):
        x64 = x.double()
        hn = x64 / (x64.square().mean(1, keepdim=True) + 1e-6).sqrt() * w1.double()
        un = ref.rows_value(hn.bfloat16()) @ mat(*qi)[0].T
        logits = un @ wg.double().T
        sig = logits.sigmoid().gather(1, ids.long())
        sc = 1.5 * sig / sig.sum(1, keepdim=True)
        yn = ref.layer(un.bfloat16(), ids, sc.float(), mat(packed[0], packed[1]), mat(packed[2], packed[3]))
        yn = ref.rows_value(yn.bfloat16()) @ mat(*qo)[0].T
        zn = x64 + yn
        on = zn / (zn.square().mean(1, keepdim=True) + 1e-6).sqrt() * w2.double()
        for name, a, b in (("u", u, un), ("scores", scores, sc), ("y", y, yn), ("out", out, on)):
            e = float((a.double() - b).norm() / b.norm())
            say("  %s %.2e" % (name, e))
            assert e <= 2e-2
        # the choice: of the groups whose two largest keys have the largest sums (keys of u as computed)
        keys = (u.float() @ wg.T).double().sigmoid() + bias.double()
        sums = keys.view(T, 4, -1).topk(2, 2).values.sum(2)
        chosen = ids.long() // (E // 4)
        least = sums.gather(1, chosen).amin(1)
        assert (least >= sums.topk(2, 1).values[:, 1] - 1e-5).all()
    buf = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    for i in (0, 1, 2, 1):
        buf.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager[i]))
        assert all(torch.equal(a, b) for a, b in zip(step(xs[(i + 1) % 3]), eager[(i + 1) % 3]))


def test_products_in_training(moe):
    """A step of autograd through two products: the gradients equal the entry points' own, captured too."""
    import torch

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, p, q, s):
            ctx.p = p
            ctx.save_for_backward(x, q, s)
            return p.forward(x, q, s)

        @staticmethod
        def backward(ctx, dy):
            x, q, s = ctx.saved_tensors
            dx, ctx.p.dw = ctx.p.backward(dy.contiguous(), x, q, s)
            return dx, None, None, None

    R, d, N = 400, 256, 512
    a, b = moe.Product(R, N, d, training=True), moe.Product(R, d, N, training=True)
    qa, qb = a.prepare_weights(randn(1, 1, N, d, std=d ** -0.5)), b.prepare_weights(randn(2, 1, d, N, std=N ** -0.5))
    x, dy = randn(3, R, d), randn(4, R, d)
    leaf = x.clone().requires_grad_()
    h = Linear.apply(leaf, a, *qa)
    y = Linear.apply(torch.relu(h), b, *qb)
    y.backward(dy)
    dh, dwb = b.backward(dy, torch.relu(h.detach()), *qb)
    dh = torch.where(h.detach() > 0, dh, torch.zeros_like(dh))
    dx, dwa = a.backward(dh, x, *qa)
    assert torch.equal(leaf.grad, dx) and torch.equal(a.dw, dwa) and torch.equal(b.dw, dwb)
