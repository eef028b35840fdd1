"""Host checks of the products and of the layer on weights in blocks of 128 at the edges of their use."""
import pytest

from mixture_experts_routed_dispatch_amd import moe
from tests.test_block128_abi import BAD, L, OK, P, ROOM, STATE, product  # noqa: F401


def test_gradients_of_no_rows(L):
    """With no rows the input gradient is empty: its pointer, like those of dy, x and the weights, may be null.  Nothing is
    launched for it."""
    import ctypes
    call = lambda c, dx=None, dw=None, ws=None, nbytes=0: L.moe_product_backward(
        ctypes.byref(c), None, None, None, None, None, dx, dw, None, ws, nbytes, None)
    for E in (1, 2):
        for add in (0, 1):
            c = product(R=0, E=E, wgrad_accumulate=add)
            assert call(c) == OK and call(c, dx=P) == OK
            assert call(c, dw=P) == ROOM and call(c, dw=P + 8) == BAD
    assert call(product(R=0, training=0)) == STATE
    assert call(product(R=8)) == BAD and call(product(R=0, N=100)) != OK
