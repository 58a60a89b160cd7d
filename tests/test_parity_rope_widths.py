"""Every head width of the rotation and the norms, with halves at even and odd places (GPU)."""

import pytest

from tests import test_parity_rope as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", range(8, 257, 8))
def test_every_width(d, dt):
    for n in sorted({d // 2, d // 2 - 1, (d // 4 + 1) // 2 * 2, 1}):
        for adj in (False, True):
            base.test_rope(dt, 1, 5, 3, 2, d, n, 2, adj, False, adj)
            base.test_norm_forward_and_backward(dt, 1, 5, 3, 2, d, n, 2, adj, not adj, True)
