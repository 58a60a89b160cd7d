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
