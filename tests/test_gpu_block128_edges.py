"""Weights in blocks of 128 at the edges of their use: empty batches, numbers that are not finite, outputs of
unlike size, arguments of wrong form, the status word, operands that end with their memory.  Layers are held to the
bounds that tests/test_gpu_block128.py derives."""
import pytest

from tests.gpu_util import dev
from tests.test_gpu_block128 import moe, randn  # noqa: F401

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
