"""Router kernels (include/moe.h, router section) against float64 numpy.

ids are compared exactly: the reference orders float64 keys, ties to the lowest index.  Bars on
values, with u = 2^-24 (FP32's half step): a score is e^x of |x| <= 32 (argument rounding
32 u * 2, exp2 and reciprocal 2 u each, a sum of 256 terms in 16-term chains and 4 levels: 20 u,
two roundings more), below 100 u = 6e-6 relative: REL = 1e-5.  A sum over T rows adds its terms in
chains of at most T / 1024 + 30 <= 100 steps: 100 u more, still within 1e-5 + 1e-5.  A gradient is
a difference of terms of at most S = |s ds| + p |D| sums; its bar is 2e-5 of the row's largest
term.  BF16 outputs add half a step, 2^-8 of the value.
"""
import math

import numpy as np
import pytest

from tests.gpu_util import dev, say

pytestmark = pytest.mark.gpu
REL = 1e-5


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    return moe


def make(T, E, dtype, seed, bias=False, mask=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E, generator=g) * 1.5).to(dtype)
    b = torch.randn(E, generator=g) * 0.05 if bias else None
    m = torch.rand(T, generator=g) > 0.2 if mask else None
    return z, b, m


def scores64(z, score):
    with np.errstate(all="ignore"):
        if score == 1:
            s = 1 / (1 + np.exp(-z))
            return s, s / s.sum(1, keepdims=True)
        e = np.exp(z - z.max(1, keepdims=True))
        s = e / e.sum(1, keepdims=True)
        return s, s


def ref_forward(z, b, m, k, score, normalize, scale, coef):
    z = z.double().numpy()
    T, E = z.shape
    s, p = scores64(z, score)
    key = z if b is None else s + b.double().numpy()
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, 1)
    if normalize:
        w = w / w.sum(1, keepdims=True)
    w = w * scale
    live = np.ones(T, bool) if m is None else m.numpy()
    ids[~live] = np.arange(k)
    w[~live] = 0
    counts = np.bincount(ids[live].ravel(), minlength=E)
    psum = p[live].sum(0)
    n = int(live.sum())
    loss = coef * E / (k * n * n) * (counts * psum).sum() if n else 0.0
    return ids, w, counts, psum, loss


def ref_backward(z, m, ids, counts, ds, dloss, k, score, normalize, scale, coef):
    import torch
    z = z.double().requires_grad_()
    E = z.shape[1]
    s = torch.softmax(z, 1) if score == 0 else torch.sigmoid(z)
    live = torch.ones(z.shape[0], 1, dtype=torch.float64) if m is None else m.double()[:, None]
    w = s.gather(1, torch.from_numpy(ids))
    if normalize:
        w = w / w.sum(1, keepdim=True)
    total = (w * scale * live * ds.double()).sum()
    if dloss is not None and counts.sum() > 0:         # no rows: the loss is the constant 0
        n = counts.sum() / k
        p = s / s.sum(1, keepdim=True)
        f = torch.from_numpy(counts.astype(np.float64))
        total = total + dloss * coef * E / (k * n * n) * (f * (p * live).sum(0)).sum()
    total.backward()
    return z.grad.numpy()


CASES = [  # T, E, k, score, normalize, dtype, bias, mask
    (1, 128, 8, 0, 1, "f32", False, False),
    (1, 5, 1, 1, 1, "bf16", True, True),
    (16, 64, 8, 0, 1, "f32", False, False),
    (17, 64, 32, 0, 0, "f32", False, True),
    (33, 7, 7, 1, 0, "f32", True, False),              # every expert, rows of 28 bytes
    (100, 1, 1, 0, 1, "bf16", False, False),
    (257, 60, 6, 0, 1, "bf16", True, True),
    (1031, 128, 17, 1, 1, "bf16", True, False),
    (4096, 256, 32, 0, 0, "f32", True, False),
    (4097, 130, 8, 1, 1, "f32", False, True),          # the larger workgroups' first size
    (8192, 128, 8, 0, 1, "f32", False, True),
    (16401, 256, 8, 1, 1, "bf16", True, True),
    (70001, 16, 2, 0, 1, "f32", False, False),
]


@pytest.mark.parametrize("T,E,k,score,normalize,dtype,bias,mask", CASES)
def test_forward_and_backward(moe, T, E, k, score, normalize, dtype, bias, mask):
    import torch
    say("router", T, E, k, score, normalize, dtype, bias, mask)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    z, b, m = make(T, E, dt, T + E, bias, mask)
    d = dev()
    on = lambda t: None if t is None else t.to(d)
    scale, coef = 2.5, 0.1
    r = moe.Router(T, E, k, score=score, normalize=normalize, scale=scale, balance_coef=coef)
    zd, bd, md = on(z), on(b), on(m)
    ids, w, counts, psum, loss = r.forward(zd, bias=bd, mask=md)
    ri, rw, rc, rp, rl = ref_forward(z, b, m, k, score, normalize, scale, coef)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert (np.abs(w.cpu().numpy() - rw) <= REL * np.abs(rw)).all()
    assert (np.abs(psum.cpu().numpy() - rp) <= 2 * REL * np.abs(rp)).all()
    assert abs(float(loss) - rl) <= 2 * REL * abs(rl)
    # without counts and loss: the same ids and scores
    i2, w2, c2, p2, l2 = r.forward(zd, bias=bd, mask=md, stats=False)
    assert torch.equal(i2, ids) and torch.equal(w2, w) and c2 is None and p2 is None and l2 is None
    # gradient, with and without the balance loss
    g = torch.Generator().manual_seed(5)
    ds = torch.randn(T, k, generator=g)
    for dloss in (None, 3.0):
        dl = None if dloss is None else torch.tensor([dloss], device=d)
        got = r.backward(on(ds), zd, ids, counts, dloss=dl, mask=md)
        assert got.dtype == dt
        ref = ref_backward(z, m, ri.copy(), rc, ds, dloss, k, score, normalize, scale, coef)
        # the row's largest term: scale |ds| and the weighted mean of them, at most twice the largest
        top = 2 * scale * np.abs(ds.numpy()).max(1, keepdims=True)
        got = got.float().cpu().numpy().astype(np.float64)
        if m is not None:
            assert (got[~m.numpy()] == 0).all()
        half = 2.0 ** -8 if dtype == "bf16" else 0.0
        bar = 2e-5 * top + half * np.abs(ref) + 2e-5 * coef
        assert (np.abs(got - ref) <= bar).all(), float((np.abs(got - ref) - bar).max())


def test_gradient_against_differences(moe):
    """d/dz of sum ds scores + 2 loss by central differences of the float64 formula, on a row set
    whose choice does not change within the step."""
    import torch
    T, E, k = 6, 12, 3
    for score in (0, 1):
        z, _, _ = make(T, E, torch.float32, 77 + score)
        ds = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
        r = moe.Router(T, E, k, score=score, normalize=True, scale=1.5, balance_coef=0.3)
        ids, _, counts, _, _ = r.forward(z.to(dev()))
        got = r.backward(ds.to(dev()), z.to(dev()), ids, counts, dloss=torch.tensor(2.0, device=dev())).cpu().numpy()
        ri = ids.cpu().numpy()
        rc = counts.cpu().numpy()

        def f(zz):
            s, p = scores64(zz, score)
            w = np.take_along_axis(s, ri, 1)
            w = 1.5 * w / w.sum(1, keepdims=True)
            return (w * ds.double().numpy()).sum() + 2 * 0.3 * E / (k * T * T) * (rc * p.sum(0)).sum()

        z0, h = z.double().numpy(), 1e-5
        for t in range(T):
            for e in range(E):
                a, b = z0.copy(), z0.copy()
                a[t, e] += h
                b[t, e] -= h
                assert abs((f(a) - f(b)) / (2 * h) - got[t, e]) < 2e-5


def test_ties_go_to_the_lowest_index(moe):
    import torch
    T, E, k = 40, 100, 9
    g = torch.Generator().manual_seed(3)
    z = torch.randint(-2, 3, (T, E), generator=g).float()
    z[0] = 0.0
    z[1, ::2] = -0.0                                  # -0 and +0 tie
    z[1, 1::2] = 0.0
    for b in (None, torch.zeros(E), torch.randint(0, 2, (E,), generator=g) * 0.25):
        for score in (0, 1):
            r = moe.Router(T, E, k, score=score)
            ids = r.forward(z.to(dev()), bias=None if b is None else b.to(dev()))[0].cpu().numpy()
            assert np.array_equal(ids, ref_forward(z, b, None, k, score, True, 1.0, 0.0)[0])


def test_near_ties_with_a_bias_are_ordered_exactly(moe):
    """Keys s + b that FP32 cannot tell apart or rounds into the wrong order: the bias is set so
    that every expert's key lies within a few 2^-24 of one half."""
    import torch
    T, E, k = 64, 128, 8
    g = torch.Generator().manual_seed(4)
    for score in (0, 1):
        row = torch.randn(1, E, generator=g)
        s = torch.from_numpy(scores64(row.double().numpy(), score)[0])
        b = (0.5 - s[0]).float()
        z = row.repeat(T, 1) + 1e-7 * torch.randn(T, E, generator=g)
        ri = ref_forward(z, b, None, k, score, True, 1.0, 0.0)[0]
        r = moe.Router(T, E, k, score=score)
        got = r.forward(z.to(dev()), bias=b.to(dev()))[0].cpu().numpy()
        assert np.array_equal(got, ri)
        # a true tie at the border next to a key between them that only 64 bits see
        z2 = z.clone()
        z2[:, 1] = z2[:, 0]
        b2 = b.clone()
        b2[1] = b2[0]
        ri = ref_forward(z2, b2, None, k, score, True, 1.0, 0.0)[0]
        assert np.array_equal(r.forward(z2.to(dev()), bias=b2.to(dev()))[0].cpu().numpy(), ri)


@pytest.mark.parametrize("k", [3, 8, 12, 20])
def test_few_near_pairs_with_a_bias(moe, k):
    """Keys that are spread but for pairs a few 2^-24 apart, at every place of the order."""
    import torch
    T, E = 300, 96
    g = torch.Generator().manual_seed(40 + k)
    for score in (0, 1):
        z = torch.randn(T, E, generator=g)
        s = torch.from_numpy(scores64(z.double().numpy(), score)[0])
        # one bias for all rows: pairs are made in the logits of sigmoid scores, or of softmax rows by
        # equal logits with biases that differ by a rounding
        b = torch.randn(E, generator=g) * 0.1
        if score == 1:
            target = s[:, 0::2] + b[0::2].double() - b[1::2].double()
            ok = (target > 0.01) & (target < 0.99)
            other = torch.log(target.clamp(0.01, 0.99) / (1 - target.clamp(0.01, 0.99)))
            z[:, 1::2] = torch.where(ok, other, z[:, 1::2].double()).float()
        else:
            b[1::2] = torch.nextafter(b[0::2], torch.full_like(b[0::2], 9.0))
            z[:, 1::2] = z[:, 0::2] - 1e-7 * torch.rand(T, E // 2, generator=g)
        ri = ref_forward(z, b, None, k, score, True, 1.0, 0.0)[0]
        got = moe.Router(T, E, k, score=score).forward(z.to(dev()), bias=b.to(dev()))[0].cpu().numpy()
        assert np.array_equal(got, ri)


@pytest.mark.parametrize("bias", [False, True])
def test_rows_do_not_depend_on_their_neighbours(moe, bias):
    """The bits of a row are the same alone and between rows of ties, of one value or of NaN."""
    import torch
    E, k, n = 256, 8, 40
    g = torch.Generator().manual_seed(71)
    rows = torch.randn(n, E, generator=g)
    b = (torch.randn(E, generator=g) * 0.05).to(dev()) if bias else None
    odd = torch.stack([torch.zeros(E), torch.randint(0, 2, (E,), generator=g).float(), torch.full((E,), float("nan"))])
    mixed = torch.cat([torch.cat([r[None], odd]) for r in rows])
    for score in (0, 1):
        a = moe.Router(n, E, k, score=score).forward(rows.to(dev()), bias=b, stats=False)
        c = moe.Router(4 * n, E, k, score=score).forward(mixed.to(dev()), bias=b, stats=False)
        assert torch.equal(a[0], c[0][::4]) and torch.equal(a[1], c[1][::4])
        one = moe.Router(1, E, k, score=score)
        for t in range(5):
            x = one.forward(rows[t:t + 1].to(dev()), bias=b, stats=False)
            assert torch.equal(x[0][0], a[0][t]) and torch.equal(x[1][0], a[1][t])


def test_nan_logits_are_chosen_last(moe):
    """Whole lanes of NaN (20 of 64 logits) with k = 12, sigmoid: the largest of the others are chosen."""
    import torch
    T, E, k = 8, 64, 12
    z, _, _ = make(T, E, torch.float32, 12)
    z[:, 8:28] = float("nan")
    ids = moe.Router(T, E, k, score=1).forward(z.to(dev()))[0].cpu().numpy()
    clean = z.clone()
    clean[:, 8:28] = float("-inf")
    assert np.array_equal(ids, ref_forward(clean, None, None, k, 1, True, 1.0, 0.0)[0])


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bias", [False, True])
def test_infinities_and_nan(moe, score, bias):
    import torch
    T, E, k = 20, 40, 4
    z, _, _ = make(T, E, torch.float32, 6)
    ninf = float("-inf")
    z[0] = ninf                                       # nothing to choose from
    z[1, 3:] = ninf                                   # fewer than k
    z[2] = torch.finfo(torch.float32).min             # masks of the lowest value
    z[3, 5] = float("nan")
    z[4, 7] = float("inf")
    b = torch.zeros(E) if bias else None
    d = dev()
    r = moe.Router(T, E, k, score=score, balance_coef=0.1)
    rows_ok = [t for t in range(T) if t not in (3, 4)]
    mask = torch.ones(T, dtype=torch.bool)
    mask[3] = mask[4] = False
    zd, bd = z.to(d), None if b is None else b.to(d)
    ids, w, counts, psum, loss = r.forward(zd, bias=bd)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert ((ids >= 0) & (ids < E)).all()
    assert all(len(set(row)) == k for row in ids.tolist())
    assert np.array_equal(ids[0], np.arange(k)) and (w[0] == 0).all()
    assert set(ids[1].tolist()) >= {0, 1, 2} and ids[1, 3] == 3 and w[1, 3] == 0
    assert abs(w[1].sum() - 1) < 1e-5
    assert np.array_equal(ids[2], np.arange(k))
    assert np.isfinite(w[2]).all()                    # softmax: equal; sigmoid: all 0
    if not bias:
        assert 5 not in ids[3].tolist()
        assert ids[4, 0] == 7
    if score == 0:
        assert np.isnan(w[3]).all() and np.isnan(w[4]).all() and math.isnan(float(loss))
    # the same rows masked: everything is finite, the other rows' results are as they were
    i2, w2, c2, p2, l2 = r.forward(zd, bias=bd, mask=mask.to(d))
    assert np.array_equal(i2.cpu().numpy()[rows_ok], ids[rows_ok])
    assert np.array_equal(w2.cpu().numpy()[rows_ok], w[rows_ok])
    assert (w2[[3, 4]] == 0).all() and torch.isfinite(p2).all() and math.isfinite(float(l2))
    assert int(c2.sum()) == k * (T - 2)
    g = r.backward(torch.ones(T, k, device=d), zd, i2, c2, dloss=torch.ones(1, device=d), mask=mask.to(d))
    assert torch.isfinite(g).all() and (g[[0, 3, 4]] == 0).all()


def test_empty_and_fully_masked_batches(moe):
    import torch
    d = dev()
    r = moe.Router(0, 16, 2, balance_coef=1.0)
    ids, w, counts, psum, loss = r.forward(torch.empty(0, 16, device=d))
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert (counts == 0).all() and (psum == 0).all() and float(loss) == 0
    assert r.backward(torch.empty(0, 2, device=d), torch.empty(0, 16, device=d), ids, counts,
                      dloss=torch.ones(1, device=d)).shape == (0, 16)
    for T in (5, 300):
        r = moe.Router(T, 16, 2, balance_coef=1.0)
        z = torch.randn(T, 16, device=d)
        mask = torch.zeros(T, dtype=torch.uint8, device=d)
        ids, w, counts, psum, loss = r.forward(z, mask=mask)
        assert (ids.cpu() == torch.arange(2)).all() and (w == 0).all()
        assert (counts == 0).all() and (psum == 0).all() and float(loss) == 0
        g = r.backward(torch.ones(T, 2, device=d), z, ids, counts, dloss=torch.ones(1, device=d), mask=mask)
        assert (g == 0).all()


def test_unaligned_rows(moe):
    """Logits that start 2 or 4 bytes behind a 16-byte line are read element by element."""
    import torch
    d = dev()
    for dt in (torch.float32, torch.bfloat16):
        T, E, k = 50, 64, 4
        flat = torch.randn(T * E + 1, device=d).to(dt)
        z = flat[1:].view(T, E)
        assert z.data_ptr() % 16 != 0
        r = moe.Router(T, E, k, balance_coef=0.1)
        a, b = r.forward(z), r.forward(z.clone())
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        ds = torch.randn(T, k, device=d)
        one = torch.ones((), device=d)
        out = torch.empty(T * E + 1, device=d, dtype=dt)[1:].view(T, E)
        ga = r.backward(ds, z, a[0], a[2], dloss=one, dlogits=out)
        gb = r.backward(ds, z.clone(), a[0], a[2], dloss=one)
        assert ga is out and torch.equal(ga, gb)


def test_bad_ids_in_the_backward_are_left_out(moe):
    import torch
    d = dev()
    T, E, k = 9, 16, 3
    z = torch.randn(T, E, device=d)
    r = moe.Router(T, E, k, normalize=False)
    ids = r.forward(z, stats=False)[0]
    ds = torch.randn(T, k, device=d)
    bad = ids.clone()
    bad[:, 1] = torch.tensor([-1, E, 1 << 30] * 3, dtype=torch.int32, device=d)
    ds0 = ds.clone()
    ds0[:, 1] = 0
    assert torch.equal(r.backward(ds, z, bad), r.backward(ds0, z, ids))


def test_refusals(moe):
    import torch
    d = dev()
    r = moe.Router(8, 16, 2)
    z = torch.randn(8, 16, device=d)
    ids = r.forward(z)[0]
    ds = torch.zeros(8, 2, device=d)
    for bad in (z[:7], z.half(), z.cpu(), torch.randn(16, 8, device=d).t()):
        with pytest.raises(ValueError):
            r.forward(bad)
    with pytest.raises(ValueError):
        r.forward(z, bias=torch.zeros(15, device=d))
    with pytest.raises(ValueError):
        r.forward(z, mask=torch.zeros(8, device=d))
    with pytest.raises(ValueError):
        r.backward(ds, z, ids.long())
    with pytest.raises(ValueError):
        r.backward(ds, z, ids, dloss=torch.ones(2, device=d))
    with pytest.raises(moe.MoeError):
        r.backward(ds, z, ids, dloss=torch.ones(1, device=d))          # a loss gradient without counts


def test_run_to_run_streams_and_graphs(moe):
    """Two routers on two streams at once, and a captured step replayed with other logits in
    between eager calls, give the eager bits."""
    import torch
    d = dev()
    T, E, k = 5000, 128, 8
    zs = [torch.randn(T, E, device=d) for _ in range(3)]
    ds = torch.randn(T, k, device=d)
    one = torch.ones((), device=d)
    r = moe.Router(T, E, k, balance_coef=0.01)

    def step(router, z):
        ids, w, counts, psum, loss = router.forward(z)
        return ids, w, counts, psum, loss, router.backward(ds, z, ids, counts, dloss=one)

    want = [step(r, z) for z in zs]
    torch.cuda.synchronize()
    others = [moe.Router(T, E, k, balance_coef=0.01) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for o, s, z in zip(others, streams, zs):
            ids, w, counts, psum, loss = o.forward(z, stream=s)
            got.append((ids, w, counts, psum, loss, o.backward(ds, z, ids, counts, dloss=one, stream=s)))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    buf = zs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(r, buf)
    for i in (0, 1, 2, 0):
        buf.copy_(zs[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        eager = step(r, zs[(i + 1) % 3])
        assert all(torch.equal(a, b) for a, b in zip(eager, want[(i + 1) % 3]))


@pytest.mark.parametrize("E", [20, 61, 96, 129, 136, 160, 200, 255, 256])
def test_choice_over_experts_and_k(moe, E):
    """Every way to the choice: all k around its borders, rows with and without many ties (BF16 and
    whole-number logits), with and without a bias, FP32 keys a rounding apart among them."""
    import torch
    T = 70
    for k in (1, 7, 8, 9, 12, 15, 16, 17, 20, 21, 24, 31, 32):
        if k > E:
            continue
        g = torch.Generator().manual_seed(100 * E + k)
        z = torch.randn(T, E, generator=g)
        z[1::4] = z[1::4].bfloat16().float()
        z[2::8] = torch.randint(-1, 2, (len(z[2::8]), E), generator=g).float()
        z[3::8] = z[3::8].sort(1, descending=True)[0]      # the largest side by side
        z[7::8] = z[7::8].sort(1)[0]
        z[4::8] = 0.3 + 1e-7 * torch.randn(len(z[4::8]), E, generator=g)
        b = torch.randn(E, generator=g) * 0.02
        b[::5] = 0.0
        for score in (0, 1):
            for bias in (None, b):
                ri = ref_forward(z, bias, None, k, score, True, 1.0, 0.0)[0]
                r = moe.Router(T, E, k, score=score)
                got = r.forward(z.to(dev()), bias=None if bias is None else bias.to(dev()), stats=False)[0].cpu().numpy()
                assert np.array_equal(got, ri), (E, k, score, bias is None)
