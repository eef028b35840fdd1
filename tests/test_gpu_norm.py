"""Block norm kernels (include/moe.h, norm section) against float64.

Bars, with u = 2^-24: a mean of d <= 16384 squares is summed in chains of 16 per lane, 6 levels and
at most 16 waves, so its relative error is below 40 u; with the square root's half of it and a few
roundings a normed value is within 60 u = 3.6e-6 of itself: REL = 1e-5.  z adds two terms, so its bar
is REL (|x| + |alpha gate n|) and half a step of its type (BF16: 2^-8 |z|).  h is compared with the
norm of the kernel's own stored z.  In the backward each value is a sum of terms whose magnitudes
are added up in the reference; the bar is 2e-5 of that sum, and half a step.  Sums over tokens run
in chains of at most T / 256 + 80 <= 200 steps: 2e-5 of the sum of magnitudes covers them.
"""
import pytest

from tests.gpu_util import dev, say

pytestmark = pytest.mark.gpu
REL = 1e-5
HALF = 2.0 ** -8
EPS = 1e-5


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    return moe


def close(name, got, ref, mag, bf16, rel=REL):
    import torch
    got = got.double()
    assert torch.isfinite(got).all(), name
    bar = rel * mag + (HALF * ref.abs() if bf16 else 0)
    bad = (got - ref).abs() - bar
    assert (bad <= 1e-30).all(), (name, float(bad.max()), float(ref.abs().max()))


def make(T, d, f32, gate, post, pre, seed):
    import torch
    g = torch.Generator(device=dev()).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev())
    res = torch.float32 if f32 else torch.bfloat16
    return dict(x=(2 * rn(T, d)).to(res), y=rn(T, d).bfloat16(), dz=rn(T, d).to(res), dh=rn(T, d).bfloat16(),
                w_post=1 + 0.1 * rn(d) if post else None, w_pre=1 + 0.1 * rn(d) if pre else None,
                gate={0: None, 1: rn(d), 2: rn(T)}[gate])


def rms(v):
    return (v.square().mean(1, keepdim=True) + EPS).rsqrt()


SHAPES = [(1, 8), (3, 64), (17, 104), (5, 512), (33, 520), (1031, 1024), (2, 1032), (777, 2048), (300, 2056),
          (65, 4096), (9, 5000), (31, 8192), (6, 8200), (11, 16384), (4099, 256)]
FORMS = [(0, True, True), (1, True, True), (2, True, True), (1, False, True), (2, False, False), (0, False, True),
         (1, True, False)]                             # gate, w_post, w_pre


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
def test_forward_and_backward(moe, T, d, f32):
    import torch
    alpha = 0.7
    for gate, post, pre in FORMS:
        say("norm", T, d, f32, gate, post, pre)
        v = make(T, d, f32, gate, post, pre, T * 7 + d)
        n = moe.BlockNorm(T, d, eps=EPS, residual_scale=alpha, gate=gate, residual_f32=f32)
        args = dict(w_post=v["w_post"], gate=v["gate"], w_pre=v["w_pre"])
        z, h = n.forward(v["x"], v["y"], **args)
        x, y = v["x"].double(), v["y"].double()
        q = rms(y) if post else 1.0
        wq = v["w_post"].double() if post else 1.0
        g = 1.0 if gate == 0 else v["gate"].double() if gate == 1 else v["gate"].double()[:, None]
        ny = y * q * wq
        close("z", z, x + alpha * g * ny, x.abs() + (alpha * g * ny).abs(), not f32)
        zs = z.double()
        r = rms(zs)
        if pre:
            ref = zs * r * v["w_pre"].double()
            close("h", h, ref, ref.abs(), True)
        else:
            assert h is None
        dh = v["dh"] if pre else None
        dx, dy, dwq, dg, dwp = n.backward(v["dz"], dh, z, v["y"], **args)
        G = v["dz"].double()
        mG = G.abs()
        if pre:
            dh, wp = v["dh"].double(), v["w_pre"].double()
            a, b = r * wp * dh, zs * r ** 3 * (wp * dh * zs).mean(1, keepdim=True)
            mb = zs.abs() * r ** 3 * (wp * dh * zs).abs().mean(1, keepdim=True)
            G = G + a - b
            mG = mG + a.abs() + mb
            t = dh * zs * r
            close("dw_pre", dwp, t.sum(0), t.abs().sum(0), False, 2e-5)
        close("dx", dx, G, mG, not f32, 2e-5)
        dn, mn = alpha * g * G, abs(alpha) * (g.abs() if gate else 1.0) * mG
        if gate:
            t, mt = alpha * G * ny, alpha * mG * ny.abs()
            close("dgate", dg, t.sum(0 if gate == 1 else 1), mt.sum(0 if gate == 1 else 1), False, 2e-5)
        if post:
            t, mt = dn * y * q, mn * (y * q).abs()
            close("dw_post", dwq, t.sum(0), mt.sum(0), False, 2e-5)
            u, mu = dn * wq, mn * wq.abs()
            ref = q * u - y * q ** 3 * (u * y).mean(1, keepdim=True)
            mag = q * mu + y.abs() * q ** 3 * (mu * y.abs()).mean(1, keepdim=True)
            close("dy", dy, ref, mag, True, 2e-5)
        else:
            assert dwq is None
            close("dy", dy, dn, mn, True, 2e-5)
        if not gate:
            assert dg is None
        if not pre:
            assert dwp is None


@pytest.mark.parametrize("f32", [False, True])
def test_first_norm_alone_and_missing_stream_gradient(moe, f32):
    """y None: h = norm(x) with the stream untouched; dz None: only h's gradient."""
    import torch
    T, d = 19, 320
    v = make(T, d, f32, 0, False, True, 8)
    n = moe.BlockNorm(T, d, eps=EPS, residual_f32=f32)
    z, h = n.forward(v["x"], w_pre=v["w_pre"])
    assert z is v["x"]
    x, wp, dh = v["x"].double(), v["w_pre"].double(), v["dh"].double()
    r = rms(x)
    ref = x * r * wp
    close("h", h, ref, ref.abs(), True)
    mag = (r * wp * dh).abs() + x.abs() * r ** 3 * (wp * dh * x).abs().mean(1, keepdim=True)
    own = r * wp * dh - x * r ** 3 * (wp * dh * x).mean(1, keepdim=True)
    for dz in (None, v["dz"]):
        dx, dy, dwq, dg, dwp = n.backward(dz, v["dh"], v["x"], w_pre=v["w_pre"])
        assert dy is None and dwq is None and dg is None
        add = 0 if dz is None else dz.double()
        close("dx", dx, add + own, mag + abs(add), not f32, 2e-5)
        t = dh * x * r
        close("dw_pre", dwp, t.sum(0), t.abs().sum(0), False, 2e-5)


def test_gradient_against_differences(moe):
    """dx, dy and the parameters' gradients against central differences of the float64 formula."""
    import torch
    T, d, alpha = 3, 16, 0.6
    v = make(T, d, True, 1, True, True, 21)
    n = moe.BlockNorm(T, d, eps=EPS, residual_scale=alpha, gate=1, residual_f32=True)
    args = dict(w_post=v["w_post"], gate=v["gate"], w_pre=v["w_pre"])
    z, _ = n.forward(v["x"], v["y"], **args)
    got = n.backward(v["dz"], v["dh"], z, v["y"], **args)
    names = ["x", "y", "w_post", "gate", "w_pre"]
    p = {k: v[k].double().cpu() for k in names + ["dz", "dh"]}

    def f(q):
        nn = q["y"] * rms(q["y"]) * q["w_post"]
        zz = q["x"] + alpha * q["gate"] * nn
        return float((zz * p["dz"]).sum() + (zz * rms(zz) * q["w_pre"] * p["dh"]).sum())

    h = 1e-5
    for name, g in zip(names, got):
        g = g.double().cpu()
        for i in range(p[name].numel()):
            hi, lo = dict(p), dict(p)
            hi[name], lo[name] = p[name].clone(), p[name].clone()
            hi[name].view(-1)[i] += h
            lo[name].view(-1)[i] -= h
            ref = (f(hi) - f(lo)) / (2 * h)
            # truncation and cancellation of the difference: 1e-8; dy is BF16: half a step
            assert abs(float(g.view(-1)[i]) - ref) <= 1e-4 + HALF * abs(ref), (name, i)


def test_zero_rows_and_rows_with_nan(moe):
    import torch
    T, d = 40, 256
    v = make(T, d, False, 1, True, True, 5)
    args = dict(w_post=v["w_post"], gate=v["gate"], w_pre=v["w_pre"])
    n = moe.BlockNorm(T, d, eps=1e-30, gate=1)
    v["x"][3], v["y"][3] = 0, 0
    z, h = n.forward(v["x"], v["y"], **args)
    assert (z[3] == 0).all() and (h[3] == 0).all() and torch.isfinite(h).all()
    v["dz"][3], v["dh"][3] = 0, 0
    grads = n.backward(v["dz"], v["dh"], z, v["y"], **args)
    assert all(torch.isfinite(g).all() for g in grads) and (grads[0][3] == 0).all() and (grads[1][3] == 0).all()
    # a row of NaN stays in its row
    x2 = v["x"].clone()
    x2[7] = float("nan")
    z2, h2 = n.forward(x2, v["y"], **args)
    keep = [t for t in range(T) if t != 7]
    assert torch.equal(z2[keep], z[keep]) and torch.equal(h2[keep], h[keep])
    assert torch.isnan(z2[7]).all() and torch.isnan(h2[7]).all()


def test_in_place_and_empty(moe):
    import torch
    T, d = 50, 1000
    for f32 in (False, True):
        v = make(T, d, f32, 2, True, True, 6)
        n = moe.BlockNorm(T, d, gate=2, residual_f32=f32)
        args = dict(w_post=v["w_post"], gate=v["gate"], w_pre=v["w_pre"])
        z, h = n.forward(v["x"], v["y"], **args)
        x = v["x"].clone()
        z2, h2 = n.forward(x, v["y"], z=x, **args)
        assert z2 is x and torch.equal(x, z) and torch.equal(h, h2)
        a = n.backward(v["dz"], v["dh"], z, v["y"], **args)
        dz = v["dz"].clone()
        b = n.backward(dz, v["dh"], z, v["y"], dx=dz, **args)
        assert b[0] is dz and all(torch.equal(p, q) for p, q in zip(a, b))
    n = moe.BlockNorm(0, 64, gate=1)
    e = torch.empty(0, 64, device=dev(), dtype=torch.bfloat16)
    w = torch.ones(64, device=dev())
    z, h = n.forward(e, e, w_post=w, gate=w, w_pre=w)
    assert z.shape == h.shape == (0, 64)
    dx, dy, dwq, dg, dwp = n.backward(e, e, z, e, w_post=w, gate=w, w_pre=w)
    assert dx.shape == dy.shape == (0, 64) and all((g == 0).all() for g in (dwq, dg, dwp))


def test_refusals(moe):
    import torch
    v = make(8, 64, False, 1, True, True, 6)
    n = moe.BlockNorm(8, 64, gate=1)
    args = dict(w_post=v["w_post"], gate=v["gate"], w_pre=v["w_pre"])
    z, _ = n.forward(v["x"], v["y"], **args)
    for k, bad in (("x", v["x"].float()), ("x", v["x"][:7]), ("y", v["y"].t().contiguous().t()), ("y", v["y"].cpu())):
        with pytest.raises(ValueError):
            n.forward(**{**dict(x=v["x"], y=v["y"]), k: bad}, **args)
    with pytest.raises(ValueError):
        n.forward(v["x"], v["y"], **{**args, "w_pre": v["w_pre"].bfloat16()})
    with pytest.raises(ValueError):
        n.forward(v["x"], v["y"], **{**args, "gate": torch.ones(8, device=dev())})
    with pytest.raises(moe.MoeError):
        n.forward(v["x"], v["y"], w_post=v["w_post"], w_pre=v["w_pre"])              # the gate is missing
    with pytest.raises(moe.MoeError):
        n.forward(v["x"])                                                              # nothing to do
    with pytest.raises(moe.MoeError):
        n.backward(v["dz"], None, z, v["y"], **args)                                   # dh is missing
    off = torch.empty(8 * 64 + 1, device=dev(), dtype=torch.bfloat16)[1:].view(8, 64)
    with pytest.raises(moe.MoeError):
        n.forward(off, v["y"], **args)                                                 # not 16-byte aligned


def test_run_to_run_streams_and_graphs(moe):
    import torch
    T, d = 3001, 2048
    vs = [make(T, d, False, 1, True, True, s) for s in (1, 2, 3)]

    def step(n, v, stream=None):
        args = dict(w_post=v["w_post"], gate=v["gate"], w_pre=v["w_pre"])
        z, h = n.forward(v["x"], v["y"], stream=stream, **args)
        return (z, h) + n.backward(v["dz"], v["dh"], z, v["y"], stream=stream, **args)

    n = moe.BlockNorm(T, d, gate=1)
    want = [step(n, v) for v in vs]
    torch.cuda.synchronize()
    two = [moe.BlockNorm(T, d, gate=1) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for m, s, v in zip(two, streams, vs):
            got.append(step(m, v, s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    buf = {k: t.clone() for k, t in vs[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(n, buf)
    for i in (0, 1, 2, 0):
        for k in buf:
            buf[k].copy_(vs[i][k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(step(n, vs[(i + 1) % 3]), want[(i + 1) % 3]))
