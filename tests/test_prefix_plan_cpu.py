"""How the shared-prefix attention cuts its keys, asked of the library (CPU: nothing is launched)."""

import random

import pytest

from blockwise_long_context_b200 import binding as lvx

TYPES = [lvx.LVX_BF16, lvx.LVX_FP32]


def _some(seed, count=300):
    r = random.Random(seed)
    log = lambda hi: int(round(2 ** r.uniform(0, hi)))  # noqa: E731
    for _ in range(count):
        H_kv, d = r.choice([1, 2, 3, 8]), r.choice([8, 40, 64, 72, 96, 128])
        S_P, S_cap = r.choice([0, log(17)]), r.choice([0, log(12)])
        yield log(7), H_kv * r.choice([1, 2, 4, 7, 16]), H_kv, log(7), S_P or (0 if S_cap else 1), S_cap, d


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("seed", range(3))
def test_the_parts_cover_the_keys_and_fill_the_workspace(seed, dt):
    for shape in _some(seed):
        B, H, H_kv, S_Q, S_P, S_cap, d = shape
        p = lvx.lvx_selftest_prefix_plan(*shape, dt)
        need = lvx.lvx_attn_prefix_workspace(*shape, dt)
        parts, rows = p["n_pre"] + p["n_suf"], B * S_Q * H
        up = lambda x: (x + 255) // 256 * 256  # noqa: E731
        assert need == max(up(parts * rows * d * 4) + up(parts * rows * 4), 256), (shape, p)
        if p["whole"]:
            assert parts == 0 and p["prefix"] != "tc", (shape, p)
        else:
            for n, keys, length in ((p["n_pre"], S_P, p["pre_len"]), (p["n_suf"], S_cap, p["suf_len"])):
                assert n * length >= keys > (n - 1) * length or n == keys == 0, (shape, p)
                assert length % 64 == 0, (shape, p)   # a part ends where a key tile does
        if dt == lvx.LVX_FP32:
            assert p["prefix"] == p["suffix"] == "fp32"
        else:
            assert "fp32" not in (p["prefix"], p["suffix"]), (shape, p)


def test_more_heads_a_group_than_a_row_tile():
    assert lvx.lvx_selftest_prefix_plan(1, 130, 1, 2, 100, 20, 64, lvx.LVX_BF16)["prefix"] == "fp32"


@pytest.mark.parametrize("shape,code", [((0, 4, 2, 1, 8, 8, 64), 1), ((1, 4, 3, 1, 8, 8, 64), 1),
                                        ((1, 4, 2, 1, 0, 0, 64), 1), ((1, 4, 2, 1, 8, 8, 136), 2)])
def test_refusals(shape, code):
    with pytest.raises(lvx.LvxError) as e:
        lvx.lvx_selftest_prefix_plan(*shape, lvx.LVX_BF16)
    assert e.value.status == code


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", [
    (1, 32, 8, 4096, 65536, 65536, 128), (8, 32, 8, 2048, 1000, 32768, 128), (1, 32, 8, 1024, 1000, 65536, 128),
    (128, 32, 8, 1, 1, 65536, 128), (16, 16, 16, 512, 0, 100000, 64), (64, 28, 4, 4, 100, 20000, 80)])
def test_long_caches_take_a_bounded_workspace(shape, dt):
    """The parts of many rows over long caches stay below what the caches themselves take."""
    B, H, H_kv, S_Q, S_P, S_cap, d = shape
    caches = 2 * B * S_cap * H_kv * d * (4 if dt == lvx.LVX_FP32 else 2)
    assert lvx.lvx_attn_prefix_workspace(*shape, dt) <= caches


@pytest.mark.parametrize("dt", TYPES)
def test_short_parts_where_there_are_few_blocks(dt):
    """One request over a long cache: its parts are what fills the machine."""
    p = lvx.lvx_selftest_prefix_plan(1, 32, 8, 1, 0, 65536, 128, dt)
    assert p["suf_len"] <= 512 and p["n_suf"] * 8 >= 148, p
