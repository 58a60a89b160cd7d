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


def _garbage(args):
    """NaN and infinities behind every request's last key."""
    n = args[5].long().clamp(0, args[3].shape[1])
    behind = torch.arange(args[3].shape[1], device="cuda") >= n[:, None]
    args[3][behind] = float("nan")
    args[4][behind] = float("nan")
    args[4][:, ::2][behind[:, ::2]] = float("inf")


LENGTHS = [0, 1, 2, 63, 64, 65, 127, 129, 255, 256, 257, 511, 512, 513, 600, 1023, 1024, 1025, 2047, 2049, 9999, -3]


@pytest.mark.parametrize("shape,prefix,suffix", [
    # the tensor-core kernel's head widths, and heads a group that do and do not divide its 128 rows
    ((40, 8, 4, 50, 0, 65, 8), None, "tc"),
    ((8, 10, 2, 130, 65, 300, 8), "tc", "tc"),
    ((8, 66, 2, 9, 300, 513, 40), "tc", "tc"),         # 33 heads: 3 tokens a tile
    ((1, 65, 1, 50, 1000, 1100, 40), "tc", "tc"),      # one token a tile
    ((16, 7, 1, 50, 300, 513, 40), "tc", "tc"),
    ((16, 16, 4, 17, 300, 513, 64), "tc", "tc"),
    ((5, 4, 4, 130, 3000, 1100, 64), "tc", "tc"),      # two row tiles of a request
    ((16, 260, 4, 4, 0, 65, 64), None, "tc"),
    ((40, 4, 4, 130, 300, 65, 72), "tc", "tc"),
    ((24, 12, 4, 100, 0, 300, 72), None, "tc"),
    ((24, 4, 2, 64, 0, 1100, 80), None, "tc"),         # five parts
    ((40, 20, 4, 17, 300, 65, 80), "tc", "tc"),
    ((24, 12, 4, 17, 300, 1100, 96), "tc", "tc"),
    ((2, 256, 2, 17, 300, 130, 96), "tc", "tc"),       # 128 heads a group
    ((3, 12, 4, 130, 300, 513, 128), "tc", "tc"),
    ((2, 28, 4, 100, 65, 700, 128), "tc", "tc"),
    ((1, 100, 1, 50, 300, 513, 128), "tc", "tc"),
    # the few-row kernel beside it, and alone in parts
    ((6, 8, 2, 40, 2000, 800, 128), "tc", "rows"),
    ((3, 4, 1, 2, 5000, 700, 72), "rows", "rows"),
    # parts of more than 512 keys
    ((90, 16, 4, 1, 200, 6000, 64), "rows", "rows"),
    ((40, 32, 4, 16, 100, 9000, 128), "tc", "tc"),
])
def test_ragged_lengths_with_garbage_behind_them(shape, prefix, suffix):
    plan = _plan(*shape)
    assert prefix in (None, plan["prefix"]) and suffix in (None, plan["suffix"]) and not plan["whole"], plan
    cap = shape[5]
    for turn in (0, 7, 14):
        lens = [n for n in LENGTHS[turn:] + LENGTHS[:turn] if n <= cap or n == 9999] + [cap - 1, cap]
        args = _make(*shape, seed=turn, lens=lens)
        _garbage(args)
        first = lvx.attention_prefix(*args)
        check(*first, args, what=f"{plan} {lens}")
        for _ in range(3):
            assert all(torch.equal(x, y) for x, y in zip(lvx.attention_prefix(*args), first))
    lvx.lvx_last_device_error()


@pytest.mark.parametrize("shape", [(4, 32, 8, 64, 300, 9000, 64), (100, 8, 2, 1, 50, 20000, 72)])
def test_long_fp32_parts(shape):
    plan = _plan(*shape, dt=torch.float32)
    assert plan["suffix"] == "fp32" and plan["suf_len"] > 512, plan
    args = _make(*shape, dt=torch.float32, lens=[shape[5], 0, 1, plan["suf_len"] - 1, plan["suf_len"], plan["suf_len"] + 1])
    _garbage(args)
    check(*lvx.attention_prefix(*args), args, what=str(plan))


@pytest.mark.parametrize("shape,prefix,suffix", [((40, 20, 4, 17, 300, 65, 80), "tc", "tc"),
                                                 ((16, 16, 4, 17, 300, 513, 64), "tc", "tc"),
                                                 ((6, 8, 2, 40, 2000, 800, 128), "tc", "rows")])
def test_nan_queries_stay_in_their_rows(shape, prefix, suffix):
    plan = _plan(*shape)
    assert (plan["prefix"], plan["suffix"]) == (prefix, suffix), plan
    args = _make(*shape)
    q = args[0]
    clean = q.clone()
    fine = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
    for b, t, h in ((0, 0, 0), (1, 5, 3), (shape[0] - 1, shape[3] - 1, shape[1] - 1)):
        q[b, t, h, (b + t) % shape[6]] = float("nan")
        fine[b, t, h] = False
    out, lse = lvx.attention_prefix(*args)
    assert torch.isnan(out[~fine]).all() and torch.isnan(lse.transpose(1, 2)[~fine]).all()
    check(out, lse, [clean, *args[1:]], rows=fine, what=str(plan))


@pytest.mark.parametrize("shape,prefix,suffix", [((40, 20, 4, 17, 300, 65, 80), "tc", "tc"),
                                                 ((32, 32, 8, 1, 20000, 300, 128), "tc", "rows"),
                                                 ((3, 4, 1, 2, 5000, 700, 72), "rows", "rows")])
def test_first_keys_of_minus_infinity_for_some_rows(shape, prefix, suffix):
    """The first 100 prefix keys' products overflow to -inf for every third row: weights of 0."""
    plan = _plan(*shape)
    assert (plan["prefix"], plan["suffix"]) == (prefix, suffix), plan
    q, kp, vp, ks, vs, n = args = _make(*shape)
    rows = torch.arange(q.shape[0] * q.shape[1] * q.shape[2], device="cuda").view(q.shape[:3]) % 3 == 0
    q[..., 0] = 0
    longest = max(float(x.float().norm(dim=-1).max()) for x in (kp, ks))
    q[..., 0][rows] = 3
    kp[..., 0] = ks[..., 0] = 0
    kp[:100, :, 0] = -3e38
    check(*lvx.attention_prefix(*args), args, what=str(plan), kmax=longest)


@pytest.mark.parametrize("d", range(8, 129, 8))
def test_every_head_width(d):
    """Many parts of few rows in both types, and whole row tiles on the tensor cores."""
    few, tiles = (2, 4, 2, 1, 9000, 300, d), (24, 12, 4, 100, 300, 1100, d)
    for shape, dt, kernel in ((few, torch.bfloat16, "rows"), (few, torch.float32, "fp32"), (tiles, torch.bfloat16, "tc")):
        plan = _plan(*shape, dt=dt)
        assert plan["prefix"] == plan["suffix"] == kernel and not plan["whole"], plan
        args = _make(*shape, dt=dt, lens=[shape[5], 0, 77, 256, 299])
        _garbage(args)
        check(*lvx.attention_prefix(*args), args, what=f"{plan} {dt}")
    lvx.lvx_last_device_error()
