"""The router with groups (include/moe.h, router section) against float64 numpy: ids are whole numbers and have to
be equal; values are held to the bars of tests/test_gpu_router.py, derived there."""
import numpy as np
import pytest

from tests.gpu_util import dev, say
from tests.test_gpu_router import REL, make, scores64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    return moe


def ref_ids(z, b, k, score, groups, top_groups, group_top):
    """ids and the scores s in float64."""
    z = z.double().numpy()
    T, E = z.shape
    with np.errstate(all="ignore"):
        s, p = scores64(z, score)
        key = s if b is None else s + b.double().numpy()
        key = np.where((z == -np.inf) | np.isnan(key), -np.inf, key)
        order = np.where(np.isnan(z), -np.inf, z) if b is None else key
        of = order if b is None and group_top == 1 else key
        best = -np.sort(-of.reshape(T, groups, E // groups), axis=2)[:, :, :group_top].sum(2)
        best = np.where(np.isnan(best), -np.inf, best)
    chosen = np.argsort(-best, axis=1, kind="stable")[:, :top_groups]
    closed = np.ones((T, groups), bool)
    np.put_along_axis(closed, chosen, False, 1)
    closed = closed.repeat(E // groups, 1)
    # closed experts behind all others, keys of -inf included
    rank = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -order, closed), axis=1)
    return rank[:, :k], s, p


def forward(moe, z, b, m, k, score, groups, top_groups, group_top, normalize=True, scale=1.0, coef=0.0):
    r = moe.Router(*z.shape, k, score=score, normalize=normalize, scale=scale, balance_coef=coef, groups=groups,
                   top_groups=top_groups, group_top=group_top)
    out = r.forward(z.to(dev()), bias=None if b is None else b.to(dev()), mask=None if m is None else m.to(dev()))
    return r, [t.cpu().numpy() for t in out]


CASES = [  # T, E, k, groups, top_groups, group_top, score, normalize, dtype, bias, mask
    (1, 256, 8, 8, 4, 2, 1, 1, "f32", True, False),
    (1, 64, 6, 8, 3, 1, 0, 0, "bf16", False, False),
    (16, 160, 6, 8, 3, 1, 0, 1, "f32", False, True),
    (33, 256, 8, 8, 1, 2, 1, 1, "bf16", True, False),          # one group: 32 experts left
    (64, 256, 16, 8, 2, 2, 0, 1, "f32", True, True),
    (65, 128, 8, 4, 2, 2, 1, 0, "f32", False, False),
    (257, 60, 6, 6, 3, 2, 0, 1, "bf16", True, True),           # groups of 10
    (300, 96, 32, 3, 1, 1, 1, 1, "f32", True, False),          # every expert of the group
    (513, 7, 2, 7, 2, 1, 0, 1, "f32", False, False),           # groups of one
    (1000, 256, 20, 32, 7, 2, 1, 1, "bf16", False, True),
    (1031, 256, 31, 16, 2, 1, 0, 0, "f32", True, False),
    (2048, 250, 9, 10, 5, 2, 0, 1, "f32", False, False),       # groups of 25
    (4097, 130, 5, 2, 1, 2, 1, 1, "f32", True, True),          # groups of 65
    (4096, 32, 4, 4, 4, 2, 1, 1, "bf16", True, False),         # all groups
    (8192, 128, 8, 16, 5, 1, 0, 1, "f32", True, False),
    (16401, 256, 8, 8, 4, 2, 1, 1, "bf16", True, True),
    (16384, 256, 8, 8, 4, 1, 0, 1, "bf16", False, False),
]


@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top,score,normalize,dtype,bias,mask", CASES)
def test_forward_and_backward(moe, T, E, k, groups, top_groups, group_top, score, normalize, dtype, bias, mask):
    import torch
    say("router groups", T, E, k, groups, top_groups, group_top, score, dtype, bias, mask)
    z, b, m = make(T, E, torch.float32 if dtype == "f32" else torch.bfloat16, T + E, bias, mask)
    r, (ids, w, counts, psum, loss) = forward(moe, z, b, m, k, score, groups, top_groups, group_top, bool(normalize), 2.5, 0.01)
    ri, s, p = ref_ids(z, b, k, score, groups, top_groups, group_top)
    live = np.ones(T, bool) if m is None else m.numpy()
    ri[~live] = np.arange(k)
    bad = np.nonzero((ids != ri).any(1))[0]
    assert not len(bad), (bad[:5], ids[bad[:2]], ri[bad[:2]])
    rw = np.take_along_axis(s, ri, 1)
    rw = (rw / rw.sum(1, keepdims=True) if normalize else rw) * 2.5 * live[:, None]
    assert (np.abs(w - rw) <= REL * np.abs(rw)).all()
    rc = np.bincount(ri[live].ravel(), minlength=E)
    assert np.array_equal(counts, rc)
    rp = p[live].sum(0)
    assert (np.abs(psum - rp) <= 2 * REL * rp).all()
    n = max(int(live.sum()), 1)
    assert abs(loss - 0.01 * E / (k * n * n) * (rc * rp).sum()) <= 3 * REL * abs(loss)
    # the gradient is that of a router without groups at these ids, to the bit
    ds = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).to(dev())
    args = (ds, z.to(dev()), torch.from_numpy(ids).to(dev()), torch.from_numpy(counts).to(dev()), torch.ones((), device=dev()),
            None if m is None else m.to(dev()))
    free = moe.Router(T, E, k, score=score, normalize=bool(normalize), scale=2.5, balance_coef=0.01)
    assert torch.equal(r.backward(*args), free.backward(*args))
    # and without statistics the choice is the same
    a, c = r.forward(z.to(dev()), bias=None if b is None else b.to(dev()), mask=None if m is None else m.to(dev()), stats=False)[:2]
    assert np.array_equal(a.cpu().numpy(), ids) and np.array_equal(c.cpu().numpy(), w)


@pytest.mark.parametrize("E,k,groups,top_groups", [(256, 8, 8, 4), (64, 5, 8, 2), (60, 6, 6, 3), (128, 32, 4, 2)])
def test_all_groups_is_the_free_choice(moe, E, k, groups, top_groups):
    import torch
    for score in (0, 1):
        for bias in (False, True):
            z, b, m = make(777, E, torch.float32, E + score, bias, True)
            _, free = forward(moe, z, b, m, k, score, 0, 0, 0)
            for group_top in (1, 2):
                _, out = forward(moe, z, b, m, k, score, groups, groups, group_top)
                for x, y in zip(free[:3], out[:3]):
                    assert np.array_equal(x, y), (score, bias, group_top)


@pytest.mark.parametrize("E,groups,top_groups", [(256, 8, 4), (256, 8, 1), (48, 4, 2), (100, 10, 3), (256, 32, 9), (8, 4, 2)])
def test_near_and_equal_groups(moe, E, groups, top_groups):
    """Rows of one value, of values closer than FP32 keys tell apart, of BF16's few values, and groups that hold the same
    logits in another order: ties to the lowest group, everything else in the order of 64 bits."""
    import torch
    g = torch.Generator().manual_seed(E + groups)
    size = E // groups
    z = torch.randn(240, E, generator=g)
    z[0::6] = 0.25
    z[1::6] = 0.25 + 1e-7 * torch.randn(40, E, generator=g)
    z[2::6] = z[2::6].to(torch.bfloat16).float().round()
    z[3::6] = torch.stack([z[3::6, :size][:, torch.randperm(size, generator=g)] for _ in range(groups)], 1).flatten(1)
    z[4::6] = 3.0 + 3e-7 * torch.randint(-3, 4, (40, E), generator=g)
    k = min(top_groups * size, 8)
    small, wide = torch.randn(E, generator=g) * 0.05, torch.randn(E, generator=g) * 1000
    for b in (None, torch.zeros(E), small, wide, (small * 1e-6)):
        for score in (0, 1):
            for group_top in (1, 2):
                _, (ids, *_) = forward(moe, z, b, None, k, score, groups, top_groups, group_top)
                ri = ref_ids(z, b, k, score, groups, top_groups, group_top)[0]
                bad = np.nonzero((ids != ri).any(1))[0]
                assert not len(bad), (b is None, score, group_top, bad[:5] % 6, ids[bad[:2]], ri[bad[:2]])


@pytest.mark.parametrize("E,groups,top_groups", [(256, 8, 4), (64, 8, 3), (60, 6, 2), (6, 3, 1)])
def test_infinities_and_nan(moe, E, groups, top_groups):
    import torch
    g = torch.Generator().manual_seed(E)
    size = E // groups
    z = torch.randn(60, E, generator=g)
    for t in range(10, 60):
        n = int(torch.randint(0, E + 1, (1,), generator=g))
        z[t, torch.randperm(E, generator=g)[:n]] = -INF
    z[0] = -INF
    z[1, 3], z[2, 0], z[3] = NAN, INF, NAN
    z[4, :size] = -INF                                   # a whole group
    z[5, 1:] = -INF
    b = torch.randn(E, generator=g) * 0.05
    pinned, off = b.clone(), b.clone()
    pinned[E // 2], pinned[1] = INF, INF
    off[::3] = -INF
    for k in sorted({1, 2, min(top_groups * size, 9)}):
        for bias in (None, b, pinned, off):
            for score in (0, 1):
                for group_top in (1, 2):
                    _, (ids, w, *_) = forward(moe, z, bias, None, k, score, groups, top_groups, group_top)
                    ri = ref_ids(z, bias, k, score, groups, top_groups, group_top)[0]
                    bad = np.nonzero((ids != ri).any(1))[0]
                    assert not len(bad), (k, bias is None, score, group_top, bad[:5], ids[bad[:2]], ri[bad[:2]])


def test_unaligned_logits(moe):
    """Rows that do not start on a load's alignment."""
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        T, E = 50, 64
        z = torch.randn(T * E + 3, generator=torch.Generator().manual_seed(1)).to(dtype)
        b = torch.randn(E + 1, generator=torch.Generator().manual_seed(2)) * 0.05
        zd, bd = z.to(dev())[3:].view(T, E), b.to(dev())[1:]
        r = moe.Router(T, E, 4, score=1, groups=8, top_groups=3, group_top=2)
        ids = r.forward(zd, bias=bd)[0].cpu().numpy()
        assert np.array_equal(ids, ref_ids(z[3:].view(T, E), b[1:], 4, 1, 8, 3, 2)[0])
