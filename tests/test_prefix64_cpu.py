"""The large-problem reference of the shared-prefix tests against the oracle (CPU)."""

import numpy as np
import pytest
import torch

import oracle
from tests._prefix64 import as_oracle, attention


@pytest.mark.parametrize("S_P,S_cap", [(7, 5), (0, 5), (7, 0)])
@pytest.mark.parametrize("S_Q", [1, 3])
def test_equals_the_oracle(S_P, S_cap, S_Q):
    g = torch.Generator().manual_seed(S_P + S_Q)
    t = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    pre = (t(S_P, 2, 8), t(S_P, 2, 8)) if S_P else (None, None)
    suf = (t(5, S_cap, 2, 8), t(5, S_cap, 2, 8), torch.tensor([0, 1, 2, 5, 99])) if S_cap else (None,) * 3
    args = (t(5, S_Q, 6, 8), *pre, *suf)
    for x, y in zip(attention(*args, scale=0.3), oracle.attention_prefix(*as_oracle(args), scale=0.3)):
        assert np.allclose(x.numpy(), y, rtol=1e-12, atol=1e-13)
