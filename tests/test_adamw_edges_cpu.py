"""Host checks of the optimiser's values: what its kernel could not compute is refused before any GPU work."""
import ctypes as C

import pytest

from helpers import ensure_built

OK, ARG = 0, 1


@pytest.mark.parametrize("eps, code", [(0.0, OK), (1e-8, OK), (2.0 ** -126, OK), (1.1e-38, ARG), (1e-40, ARG),
                                       (1e-60, ARG), (5e-324, ARG)])
def test_eps_below_the_normal_values(eps, code):
    """The quotient's reciprocal flushes them to 0, so an element without gradient would be 0 * infinity."""
    from pruned_expert_backward_gb300 import _lib as L
    h = L.AdamwHyper(1e-3, 0.9, 0.95, eps, 1, 0, 0.0, None, None, None)
    assert ensure_built().lrm_adamw(None, 0, 1, 1, 8, 0, C.byref(h), None) == code
