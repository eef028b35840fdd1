"""The router's choice with a selection bias at its edges (include/moe.h, router section), against the
float64 order of tests/test_gpu_router.py: ids are whole numbers and have to be equal; scores are held
to its REL, derived there."""
import numpy as np
import pytest

from tests.gpu_util import dev, say
from tests.test_gpu_router import REL, ref_forward

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
