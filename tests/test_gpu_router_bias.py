"""The router's choice with a selection bias at its edges (include/moe.h, router section), against the
float64 order of tests/test_gpu_router.py: ids are whole numbers and have to be equal; scores are held
to its REL, derived there."""
import numpy as np
import pytest

from tests.gpu_util import dev, say
from tests.test_gpu_router import REL, ref_backward, ref_forward, scores64

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available()
    from mixture_experts_routed_dispatch_amd import moe
    moe.lib()
    return moe


def compare(moe, z, b, k, score):
    """ids, scores and counts of all rows."""
    T, E = z.shape
    r = moe.Router(T, E, k, score=score)
    ids, w, counts, _, _ = r.forward(z.to(dev()), bias=b.to(dev()))
    ri, rw, rc, _, _ = ref_forward(z, b, None, k, score, True, 1.0, 0.0)
    ids = ids.cpu().numpy()
    assert np.array_equal(ids, ri), (E, k, score, np.nonzero((ids != ri).any(1))[0][:5])
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert (np.abs(w.cpu().numpy() - rw) <= REL * np.abs(rw)).all()


@pytest.mark.parametrize("E", [2, 3, 20, 32, 61, 128, 256])
def test_infinite_biases(moe, E):
    """+inf pins experts and -inf leaves them to the end, ties by index: as many pinned experts as
    places, more and fewer; nothing but infinite keys; rows of ties and of near keys among them."""
    import torch
    T = 37
    g = torch.Generator().manual_seed(E)
    for pinned in sorted({0, 1, 2, 3, 5, E // 2, E}):
        for out in sorted({0, 1, E // 2, E - pinned}):
            if pinned + out > E:
                continue
            order = torch.randperm(E, generator=g)
            b = torch.randn(E, generator=g) * 0.05
            b[order[:pinned]] = INF
            b[order[pinned:pinned + out]] = -INF
            z = torch.randn(T, E, generator=g)
            z[1::5] = 0.25
            z[2::5] = 0.25 + 1e-7 * torch.randn(len(z[2::5]), E, generator=g)
            say("router bias", E, pinned, out)
            for k in sorted({1, 2, 3, pinned, pinned + 1, pinned + 2, E - out, min(E, 21), min(E, 32)}):
                if not 1 <= k <= min(E, 32):
                    continue
                for score in (0, 1):
                    compare(moe, z, b, k, score)


def ref_keys(z, b, score):
    """Keys with a bias: s + b, -inf for logits of -inf, and NaN as -inf."""
    z, b = z.double().numpy(), b.double().numpy()
    with np.errstate(all="ignore"):
        key = scores64(z, score)[0] + b
    return np.where((z == -np.inf) | np.isnan(key), -np.inf, key)


@pytest.mark.parametrize("E,k", [(8, 3), (24, 4), (40, 4), (61, 20), (128, 8), (256, 8), (256, 32)])
def test_logits_of_minus_infinity_stay_behind_whatever_their_bias(moe, E, k):
    """Disabled experts have the largest biases, +inf among them; every number of live experts from
    none to all, in one piece or spread."""
    import torch
    g = torch.Generator().manual_seed(E + k)
    live = sorted({0, 1, 2, k - 1, k, k + 1, E // 4, E // 2, E - 1, E})
    z = torch.randn(2 * len(live), E, generator=g)
    for t, n in enumerate(live):
        z[2 * t, torch.randperm(E, generator=g)[n:]] = -INF
        z[2 * t + 1, n:] = -INF
    for biases in (torch.linspace(-1, 1, E), torch.linspace(1, -1, E), torch.randn(E, generator=g)):
        for pin in (False, True):
            b = biases.clone()
            if pin:
                b[E // 2] = INF
            for score in (0, 1):
                r = moe.Router(len(z), E, k, score=score)
                ids, w, counts, _, _ = r.forward(z.to(dev()), bias=b.to(dev()))
                ids, w = ids.cpu().numpy(), w.cpu().numpy()
                want = np.argsort(-ref_keys(z, b, score), axis=1, kind="stable")[:, :k]
                assert np.array_equal(ids, want), (E, k, score, pin)
                assert np.array_equal(counts.cpu().numpy(), np.bincount(want.ravel(), minlength=E))
                off = np.take_along_axis(z.numpy(), ids.astype(np.int64), 1) == -np.inf
                assert (w[off] == 0).all() and np.isfinite(w).all()
                assert (np.abs(w.sum(1)[1:] - 1)[~off[1:].all(1)] <= 1e-5).all()


@pytest.mark.parametrize("E", [24, 100, 256])
def test_nan_and_infinite_logits_with_a_bias(moe, E):
    """A NaN logit comes with those of -inf, by index; with softmax its row has no other keys, nor has a
    row with +inf: ids 0 .. k-1.  With sigmoid +inf has a score of 1."""
    import torch
    T, k = 12, 5
    g = torch.Generator().manual_seed(E)
    z = torch.randn(T, E, generator=g)
    b = torch.randn(E, generator=g)
    top = int(b.argmax())
    z[0, top] = float("nan")
    z[1, top], z[1, (top + 1) % E] = -INF, float("nan")
    z[2, k - 1:] = float("nan")
    z[3, k - 1:] = -INF
    z[4, 3:] = float("nan")
    z[4, 9::2] = -INF
    z[5, 7] = INF
    z[6, 7], z[6, top] = INF, float("nan")
    for score in (0, 1):
        r = moe.Router(T, E, k, score=score)
        ids = r.forward(z.to(dev()), bias=b.to(dev()), stats=False)[0].cpu().numpy()
        assert np.array_equal(ids, np.argsort(-ref_keys(z, b, score), axis=1, kind="stable")[:, :k]), score
        if score == 0:
            assert (ids[[0, 1, 2, 4, 5, 6]] == np.arange(k)).all()


@pytest.mark.parametrize("k", [2, 8, 24])
def test_scores_far_below_the_rows_maximum(moe, k):
    """Experts that the bias chose 40 to 80 below the maximum (sigmoid: below 0).  The logits are multiples
    of 2^-8 and the maximum is 0, so that differences are exact and what is left is e^x: with u = 2^-24,
    e^x by the hardware's exp2 (1 ulp, 2 u) with its argument's rounding made up for (2 u more), one
    factor (u; with sigmoid an addition and a reciprocal, 3 u), the sum of k of them (5 u and the terms'
    own 7 u) and the quotient (u): within 20 u.  With e^x from an argument rounded to 24 bits they are
    80 u off."""
    import torch
    T, E = 400, 64
    g = torch.Generator().manual_seed(k)
    z = torch.zeros(T, E)
    low = torch.randperm(E - 1, generator=g)[:k] + 1
    z[:, low] = -(40 * 256 + torch.randint(0, 40 * 256, (T, k), generator=g)) / 256.0
    b = torch.zeros(E)
    b[low] = 10.0
    for score in (0, 1):
        ids, w, _, _, _ = moe.Router(T, E, k, score=score).forward(z.to(dev()), bias=b.to(dev()), stats=False)
        ids = ids.cpu().numpy().astype(np.int64)
        assert (np.sort(ids, 1) == np.sort(low.numpy())).all()
        s = np.take_along_axis(scores64(z.double().numpy(), score)[0], ids, 1)
        want = s / s.sum(1, keepdims=True)
        off = (np.abs(w.cpu().numpy() - want) / want).max() * 2.0 ** 24
        print("  %s, k = %d: %.1f u" % (("softmax", "sigmoid")[score], k, off), flush=True)
        assert off <= 20


@pytest.mark.parametrize("k", [2, 8, 20])
def test_one_dominant_score_next_to_biased_small_ones(moe, k):
    """Rows whose sum loses the most to rounding (the lane of the score near 1 adds terms just under
    half a step), and biases that lift small scores to within 1e-6 of the large one, above and below."""
    import torch
    E, T = 256, 96
    g = torch.Generator().manual_seed(60 + k)
    z = torch.full((T, E), -80.0)
    z[:, 0] = 0.0
    share = 0.5 + 0.5 * torch.rand(T, 1, generator=g)
    z[:, [*range(1, 8), *range(128, 136)]] = torch.log(2.0 ** -24 * share)
    low = torch.arange(20, 20 + 2 * k)
    z[:, low] = -17 - torch.rand(T, len(low), generator=g)
    b = torch.zeros(E)
    b[low] = 1.0 + 1e-6 * (2 * torch.rand(len(low), generator=g) - 1)
    z[T // 2:] = torch.randn(T - T // 2, E, generator=g) * 3
    z[T // 2:, 0] = 16.0
    compare(moe, z, b, k, 0)


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_of_the_smallest_sigmoid_scores(moe, normalize):
    """Rows whose scores are all near FP32's smallest normal number, 2^-126: their reciprocal sums times a
    gradient of 100 pass its largest.  Bars as in tests/test_gpu_router.py: 2e-5 of the row's largest term."""
    import torch
    T, E, k = 200, 24, 4
    g = torch.Generator().manual_seed(5)
    z = -86.5 - 0.6 * torch.rand(T, E, generator=g)
    z[T // 2:] = -60 - 20 * torch.rand(T - T // 2, E, generator=g)
    ds = 100 * torch.randn(T, k, generator=g)
    r = moe.Router(T, E, k, score=1, normalize=normalize, balance_coef=20.0)
    ids, w, counts, _, _ = r.forward(z.to(dev()))
    ri, rw, rc, _, _ = ref_forward(z, None, None, k, 1, normalize, 1.0, 20.0)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert (np.abs(w.cpu().numpy() - rw) <= REL * np.abs(rw)).all()
    for dloss in (None, 3.0):
        got = r.backward(ds.to(dev()), z.to(dev()), ids, counts, dloss=None if dloss is None else torch.tensor(dloss, device=dev()))
        ref = ref_backward(z, None, ri.copy(), rc, ds, dloss, k, 1, normalize, 1.0, 20.0)
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all()
        top = 2 * np.abs(ds.numpy()).max(1, keepdims=True) * (1 if normalize else rw.max(1, keepdims=True))
        assert (np.abs(got - ref) <= 2e-5 * top + (0 if dloss is None else 2e-5 * 20.0)).all()
