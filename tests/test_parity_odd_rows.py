"""Block forward with rows that have no number to go by, beside ordinary ones in the same warp (GPU)."""

import numpy as np
import pytest
import torch

import oracle
from blockwise_long_context_b200 import binding as lvx
from tests._parity import compare, to64

pytestmark = pytest.mark.gpu


def _make(d, S_Q=200, S_KV=1000):
    g = torch.Generator().manual_seed(d)
    t = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    return t(1, S_Q, 4, d), t(1, S_KV, 2, d), t(1, S_KV, 2, d)


@pytest.mark.parametrize("n_blocks", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_query_leaves_the_others(d, n_blocks):
    q, k, v = _make(d)
    q[0, 5, 1] = float("nan")
    q[0, 77, 2, 3] = float("nan")
    fine = torch.ones(1, 200, 4, dtype=torch.bool)
    fine[0, 5, 1] = fine[0, 77, 2] = False
    out, lse = lvx.attention_forward(q, k, v, n_blocks)
    lvx.lvx_last_device_error()
    q = q.nan_to_num(0)
    ref, ref_l = oracle.attention_fwd(to64(q), to64(k), to64(v))
    compare(out[fine.cuda()], ref[fine.numpy()], "bf16", "out")
    rows = fine.transpose(1, 2)
    compare(lse[rows.cuda()], ref_l[rows.numpy()], "f32", "lse")


@pytest.mark.parametrize("n_blocks", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_a_first_tile_of_minus_infinities_for_some_rows(d, n_blocks):
    """The first 128 keys' products overflow to -inf for every third row: weights of 0."""
    q, k, v = _make(d)
    q[..., 0] = 0
    q[:, ::3, :, 0] = 3
    k[..., 0] = 0
    k[:, :128, :, 0] = -3e38
    out, lse = lvx.attention_forward(q, k, v, n_blocks)
    lvx.lvx_last_device_error()
    with np.errstate(all="ignore"):
        ref, ref_l = oracle.attention_fwd(to64(q), to64(k), to64(v))
    compare(out, ref, "bf16", "out")
    compare(lse, ref_l, "f32", "lse")


@pytest.mark.parametrize("n_blocks", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_minus_infinities_see_no_key(d, n_blocks):
    q, k, v = _make(d)
    q[..., 0] = 0
    q[:, ::3, :, 0] = 3
    k[..., 0] = -3e38
    out, lse = lvx.attention_forward(q, k, v, n_blocks)
    lvx.lvx_last_device_error()
    assert (out[:, ::3] == 0).all() and torch.isneginf(lse[:, :, ::3]).all()
    fine = [i for i in range(200) if i % 3]
    ref, ref_l = oracle.attention_fwd(to64(q[:, fine]), to64(k), to64(v))
    compare(out[:, fine], ref, "bf16", "out")
    compare(lse[:, :, fine], ref_l, "f32", "lse")
