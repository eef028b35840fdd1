"""The operators around the layer as a Mixture-of-Experts block runs them: norm -> router -> experts ->
norm of the output, gate, residual and the next block's norm, forward and backward against float64
autograd on the CPU (the choice of experts taken from the router), and a decode step with 4-bit
weights, eager and captured.  Every tensor between the calls is BF16 or FP32 as the calls take it, so
the whole is held to the layer's norm-wise BF16 budget of 2e-2 (tests/gpu_util.py)."""
import pytest

from tests.gpu_util import dev, rel, say

pytestmark = pytest.mark.gpu
BUDGET = 2e-2
EPS = 1e-5


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    return moe


def params(d, I, E, seed):
    import torch
    g = torch.Generator(device=dev()).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev())
    return dict(w1=1 + 0.1 * rn(d), wg=rn(E, d) * d ** -0.5, w13=(rn(E, 2 * I, d) * d ** -0.5).bfloat16(),
                w2=(rn(E, d, I) * I ** -0.5).bfloat16(), w_post=1 + 0.1 * rn(d), gate=0.5 * rn(d),
                w_next=1 + 0.1 * rn(d)), g


def reference(p, x, ids, mask, score, scale, coef, alpha):
    """(z, h2, loss) in float64 with the given experts; p and x: float64 leaves on the CPU."""
    import torch
    rms = lambda v, w: v * (v.square().mean(1, keepdim=True) + EPS).rsqrt() * w
    h = rms(x, p["w1"])
    logits = h @ p["wg"].T
    s = torch.softmax(logits, 1) if score == 0 else torch.sigmoid(logits)
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * scale
    live = torch.ones(x.shape[0], 1, dtype=torch.float64) if mask is None else mask.double()[:, None]
    w = w * live
    I = p["w2"].shape[2]
    gu = torch.einsum("tkid,td->tki", p["w13"][ids], h)
    a = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    y = (torch.einsum("tkdi,tki->tkd", p["w2"][ids], a) * w[..., None]).sum(1)
    z = x + alpha * p["gate"] * rms(y, p["w_post"])
    E, k = s.shape[1], ids.shape[1]
    counts = torch.zeros(E, dtype=torch.float64)
    counts.index_add_(0, ids[live[:, 0] > 0].flatten(), torch.ones(int(live.sum()) * k, dtype=torch.float64))
    n = live.sum()
    loss = coef * E / (k * n * n) * (counts * (s / s.sum(1, keepdim=True) * live).sum(0)).sum()
    return z, rms(z, p["w_next"]), loss


@pytest.mark.parametrize("T,d,I,E,k,score,masked", [(96, 256, 128, 8, 2, 0, False), (131, 512, 256, 16, 4, 1, True)])
def test_training_block(moe, T, d, I, E, k, score, masked):
    import torch
    say("block", T, d, I, E, k, score, masked)
    p, g = params(d, I, E, 3)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev())
    x, dz, dh2 = rn(T, d).bfloat16(), rn(T, d).bfloat16(), rn(T, d).bfloat16()
    mask = torch.rand(T, generator=g, device=dev()) > 0.2 if masked else None
    alpha, scale, coef = 0.8, 1.5, 5.0                 # a balance loss whose gradient shows
    n1 = moe.BlockNorm(T, d, eps=EPS)
    n2 = moe.BlockNorm(T, d, eps=EPS, residual_scale=alpha, gate=moe.MOE_GATE_CHANNEL)
    router = moe.Router(T, E, k, score=score, scale=scale, balance_coef=coef)
    layer = moe.Layer(T, d, I, E, k, training=True)
    out = dict(w_post=p["w_post"], gate=p["gate"], w_pre=p["w_next"])

    _, h = n1.forward(x, w_pre=p["w1"])
    logits = h.float() @ p["wg"].T
    ids, scores, counts, _, loss = router.forward(logits, mask=mask)
    y = layer.forward(h, ids, scores, p["w13"], p["w2"])
    z, h2 = n2.forward(x, y, **out)

    dres, dy, dw_post, dgate, dw_next = n2.backward(dz, dh2, z, y, **out)
    dhe, dw13, dw2, dscores = layer.backward(dy, h, p["w13"], p["w2"])
    dlogits = router.backward(dscores, logits, ids, counts, dloss=torch.ones((), device=dev()), mask=mask)
    dwg = dlogits.T @ h.float()
    dh = (dhe.float() + dlogits @ p["wg"]).bfloat16()
    dx, _, _, _, dw1 = n1.backward(dres, dh, x, w_pre=p["w1"])
    assert layer.status() == (moe.MOE_OK, 0)

    leaves = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    xr = x.double().cpu().requires_grad_()
    zr, hr, lr = reference(leaves, xr, ids.long().cpu(), None if mask is None else mask.cpu(), score, scale, coef, alpha)
    ((zr * dz.double().cpu()).sum() + (hr * dh2.double().cpu()).sum() + lr).backward()
    got = dict(z=(z, zr), h2=(h2, hr), loss=(loss, lr), dx=(dx, xr.grad), w1=(dw1, leaves["w1"].grad),
               wg=(dwg, leaves["wg"].grad), w13=(dw13, leaves["w13"].grad), w2=(dw2, leaves["w2"].grad),
               w_post=(dw_post, leaves["w_post"].grad), gate=(dgate, leaves["gate"].grad),
               w_next=(dw_next, leaves["w_next"].grad))
    for name, (a, b) in got.items():
        e = rel(a.double().cpu().numpy(), b.detach().numpy())
        print("  %s: %.2e" % (name, e), flush=True)
        assert e <= BUDGET, (name, e)


@pytest.mark.parametrize("T", [1, 5, 32])
def test_decode_block_with_4bit_weights(moe, T):
    import torch
    d, I, E, k = 512, 256, 16, 4
    p, g = params(d, I, E, 7)
    alpha = 0.8
    n1 = moe.BlockNorm(T, d, eps=EPS)
    n2 = moe.BlockNorm(T, d, eps=EPS, residual_scale=alpha, gate=moe.MOE_GATE_CHANNEL)
    router = moe.Router(T, E, k)
    layer = moe.Layer(T, d, I, E, k, precision=moe.MOE_MXFP4)
    packed = layer.prepare_weights(p["w13"], p["w2"])
    w13, w2 = layer.expand_weights(*packed)
    out = dict(w_post=p["w_post"], gate=p["gate"], w_pre=p["w_next"])

    def step(x):
        _, h = n1.forward(x, w_pre=p["w1"])
        ids, scores, _, _, _ = router.forward((h.float() @ p["wg"].T), stats=False)
        y = layer.forward(h, ids, scores, packed[0], packed[2], packed[1], packed[3])
        return n2.forward(x, y, **out) + (ids,)

    xs = [torch.randn(T, d, generator=g, device=dev()).bfloat16() for _ in range(3)]
    eager = [step(x) for x in xs]
    assert layer.status() == (moe.MOE_OK, 0)
    ref = {n: t.double().cpu() for n, t in p.items()}
    ref["w13"], ref["w2"] = w13.double().cpu(), w2.double().cpu()
    for x, (z, h2, ids) in zip(xs, eager):
        zr, hr, _ = reference(ref, x.double().cpu(), ids.long().cpu(), None, 0, 1.0, 0.0, alpha)
        assert rel(z.double().cpu().numpy(), zr.numpy()) <= BUDGET
        assert rel(h2.double().cpu().numpy(), hr.numpy()) <= BUDGET
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


def test_offsets_past_32_bits(moe):
    """Rows that start more than 2^31 elements (2^32 bytes) into their tensors: the last rows equal
    those of a short call on the same values."""
    import torch
    torch.manual_seed(17)
    T, E, k, n = (1 << 23) + 37, 256, 4, 70
    z = torch.zeros(T, E, dtype=torch.bfloat16, device=dev())
    z[-n:] = torch.randn(n, E, device=dev()).bfloat16()
    mask = torch.zeros(T, dtype=torch.bool, device=dev())
    mask[-n:] = True
    r, small = moe.Router(T, E, k, balance_coef=0.1), moe.Router(n, E, k, balance_coef=0.1)
    a, b = r.forward(z, mask=mask), small.forward(z[-n:].clone())
    assert torch.equal(a[0][-n:], b[0]) and torch.equal(a[1][-n:], b[1]) and torch.equal(a[2], b[2])
    ds = torch.randn(T, k, device=dev())
    one = torch.ones((), device=dev())
    ga = r.backward(ds, z, a[0], a[2], dloss=one, mask=mask)
    gb = small.backward(ds[-n:].clone(), z[-n:].clone(), b[0], b[2], dloss=one)
    assert torch.equal(ga[-n:], gb) and (ga[:1000] == 0).all()
    del z, a, ga, ds
    T, d, n = (1 << 17) + 9, 16384, 11
    mk = lambda: torch.zeros(T, d, dtype=torch.bfloat16, device=dev())
    x, y, dz, dh = mk(), mk(), mk(), mk()
    for t in (x, y, dz, dh):
        t[-n:] = torch.randn(n, d, device=dev()).bfloat16()
    w = torch.rand(d, device=dev()) + 0.5
    big, few = moe.BlockNorm(T, d, gate=moe.MOE_GATE_CHANNEL), moe.BlockNorm(n, d, gate=moe.MOE_GATE_CHANNEL)
    args = dict(w_post=w, gate=w, w_pre=w)
    za, ha = big.forward(x, y, **args)
    zb, hb = few.forward(x[-n:].clone(), y[-n:].clone(), **args)
    assert torch.equal(za[-n:], zb) and torch.equal(ha[-n:], hb)
    ga = big.backward(dz, dh, za, y, **args)
    gb = few.backward(dz[-n:].clone(), dh[-n:].clone(), zb, y[-n:].clone(), **args)
    assert torch.equal(ga[0][-n:], gb[0]) and torch.equal(ga[1][-n:], gb[1])
    for p, q in zip(ga[2:], gb[2:]):                    # the same terms in another order: 2e-5 of their magnitudes
        assert (p - q).abs().max() <= 2e-5 * q.abs().max() * n


def test_4bit_weights_past_32_bits(moe):
    """Codes of more than 2^31 bytes: the last expert's output against float64 on its expanded weights."""
    import torch
    torch.manual_seed(18)
    d, I, E, k = 4096, 2048, 256, 2
    w13 = torch.zeros(E, 2 * I, d, dtype=torch.bfloat16, device=dev())
    w2 = torch.zeros(E, d, I, dtype=torch.bfloat16, device=dev())
    for e in (0, E - 1):
        w13[e] = (torch.randn(2 * I, d, device=dev()) * d ** -0.5).bfloat16()
        w2[e] = (torch.randn(d, I, device=dev()) * I ** -0.5).bfloat16()
    for T in (1, 3):
        layer = moe.Layer(T, d, I, E, k, precision=moe.MOE_MXFP4)
        packed = layer.prepare_weights(w13, w2)
        assert packed[0].numel() >= 1 << 31
        x = torch.randn(T, d, device=dev()).bfloat16()
        ids = torch.tensor([[E - 1, 0]] * T, dtype=torch.int32, device=dev())
        sc = torch.rand(T, k, device=dev())
        y = layer.forward(x, ids, sc, packed[0], packed[2], packed[1], packed[3])
        e13, e2 = layer.expand_weights(*packed)
        ref = torch.zeros(T, d, dtype=torch.float64, device=dev())
        for j, e in enumerate((E - 1, 0)):
            gu = x.double() @ e13[e].double().T
            ref += (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ e2[e].double().T * sc[:, j:j + 1].double()
        assert rel(y.double().cpu().numpy(), ref.cpu().numpy()) <= 5e-3
        del e13, e2, packed, layer
