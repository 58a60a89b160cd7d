"""Shared-prefix attention kernel by kernel against 64 bits (GPU): each problem's plan is asked for, so that the
kernel that a test is about is the one that runs."""

import math

import pytest
import torch

from blockwise_long_context_b200 import binding as lvx
from tests._prefix64 import check

pytestmark = pytest.mark.gpu


def _plan(B, H, H_kv, S_Q, S_P, S_cap, d, dt=torch.bfloat16):
    return lvx.lvx_selftest_prefix_plan(B, H, H_kv, S_Q, S_P, S_cap, d,
                                        lvx.LVX_BF16 if dt is torch.bfloat16 else lvx.LVX_FP32)


def _make(B, H, H_kv, S_Q, S_P, S_cap, d, dt=torch.bfloat16, seed=0, lens=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    q = t(B, S_Q, H, d)
    kp, vp = (t(S_P, H_kv, d), t(S_P, H_kv, d)) if S_P else (None, None)
    if not S_cap:
        return [q, kp, vp, None, None, None]
    if lens is None:
        lens = torch.randint(0, S_cap + 1, (B,), generator=g, device="cuda").tolist()
    n = torch.tensor((lens * B)[:B], dtype=torch.int32, device="cuda")
    return [q, kp, vp, t(B, S_cap, H_kv, d), t(B, S_cap, H_kv, d), n]


def _rising(k, v, part):
    """Scores that rise by 6 (more than 2^8) nine times in every part of `part` keys, for queries whose first
    element is 8; the values fall as they rise, so that every stretch of keys counts in the output."""
    at = torch.arange(k.shape[-3], device="cuda") % part // -(-part // 10)
    level = 6.0 * at[:, None]
    k[..., 0] = level * math.sqrt(k.shape[-1]) / 8
    v.mul_(torch.exp(54 - level)[..., None].to(v.dtype))


@pytest.mark.parametrize("shape,prefix,suffix", [
    ((32, 32, 8, 1, 30000, 0, 96), "tc", None),
    ((32, 32, 8, 1, 20000, 300, 128), "tc", "rows"),
    ((100, 28, 4, 4, 8000, 300, 80), "tc", "tc"),
    ((40, 8, 8, 5, 9000, 0, 64), "tc", None),
    ((2, 8, 2, 1, 9000, 700, 64), "rows", "rows"),
])
def test_rising_scores(shape, prefix, suffix):
    plan = _plan(*shape)
    assert plan["prefix"] == prefix and suffix in (None, plan["suffix"]) and not plan["whole"], plan
    args = _make(*shape)
    q, kp, vp, ks, vs, n = args
    q[..., 0] = 8.0 * (torch.arange(q.shape[0] * q.shape[1] * q.shape[2], device="cuda") % 3 / 2).view(q.shape[:3])
    _rising(kp, vp, plan["pre_len"])
    if ks is not None:
        _rising(ks, vs, min(plan["suf_len"], ks.shape[1]))
    first = lvx.attention_prefix(*args)
    check(*first, args, what=str(plan))
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(lvx.attention_prefix(*args), first))
    lvx.lvx_last_device_error()
