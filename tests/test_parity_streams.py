"""Calls with an explicit stream and no workspace (GPU): the workspace that the binding takes belongs to the
stream of the launches, not to the current one."""

import pytest
import torch

from blockwise_long_context_b200 import binding as lvx

pytestmark = pytest.mark.gpu


def _prefix(seed):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q = t(6, 1, 8, 128)
    args = (q, t(3000, 2, 128), t(3000, 2, 128), t(6, 300, 2, 128), t(6, 300, 2, 128),
            torch.tensor([0, 1, 64, 65, 299, 300], dtype=torch.int32, device="cuda"))
    out = torch.empty_like(q), torch.empty(6, 8, 1, device="cuda")
    return args, out, lambda s: lvx.lvx_attn_prefix(*args, *out, stream=s)


def _norm(seed):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    args = t(2, 500, 8, 128), t(2, 500, 2, 128), t(128), t(128), t(2, 500, 8, 128), t(2, 500, 2, 128)
    out = torch.empty_like(args[0]), torch.empty_like(args[1]), *torch.empty(2, 128, device="cuda")
    return args, out, lambda s: lvx.lvx_head_norm_rope_bwd(*args, *out, stream=s)


def _handle(stream, raw):
    return stream.cuda_stream if raw else stream


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("make", [_prefix, _norm])
def test_the_workspace_belongs_to_the_launch_stream(make, raw, monkeypatch):
    """Nothing is launched: the memory that the call would have used is not given out again on the current
    stream when the call has returned."""
    _, _, call = make(0)
    used = []
    monkeypatch.setattr(lvx, "_launch", lambda name, dev, stream, *a: used.append((a[-2], a[-1])))
    call(_handle(torch.cuda.Stream(), raw))
    (at, size), = used
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() + size <= at or at + size <= x.data_ptr() for x in later)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("make", [_prefix, _norm])
def test_two_explicit_streams_with_other_allocations_in_between(make, raw):
    want, calls = [], []
    for seed in (1, 2):
        _, out, call = make(seed)
        call(None)
        want.append([x.clone() for x in out])
        calls.append((out, call))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for out, _call in calls:
            for x in out:
                x.fill_(7)
        torch.cuda.synchronize()
        for s, (_, call) in zip(streams, calls):
            with torch.cuda.stream(s):
                torch.cuda._sleep(5_000_000)   # the launches wait behind it
            call(_handle(s, raw))
            for n in (1 << 16, 1 << 20, 1 << 22):
                torch.full((n,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for (out, _call), ref in zip(calls, want):
            assert all(torch.equal(x, y) for x, y in zip(out, ref))


def _accumulate(dt):
    g = torch.Generator().manual_seed(3)
    t = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
    q, k, v, do = t(1, 300, 4, 64), t(1, 500, 2, 64), t(1, 500, 2, 64), t(1, 300, 4, 64)
    out, lse = lvx.attention_forward(q, k, v, 2)
    grads = [torch.zeros(x.shape, device="cuda") for x in (q, k, v)]
    return grads, lambda s: lvx.lvx_attn_bwd_accumulate(q, k, v, out, lse, do, *grads, stream=s)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_the_backward_s_workspace_belongs_to_the_launch_stream(dt, raw, monkeypatch):
    """Nothing is launched, as above."""
    _, call = _accumulate(dt)
    torch.cuda.synchronize()
    used = []

    class Recorder:
        def lvx_attn_bwd_workspace(self, *a):
            return real.lvx_attn_bwd_workspace(*a)

        def lvx_attn_bwd_accumulate(self, *a):
            used.append((a[-3], a[-2]))
            return 0

    real = lvx.lib()
    monkeypatch.setattr(lvx, "lib", Recorder)
    call(_handle(torch.cuda.Stream(), raw))
    (at, size), = used
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() + size <= at or at + size <= x.data_ptr() for x in later)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_accumulating_on_an_explicit_stream_with_other_allocations(dt, raw):
    grads, call = _accumulate(dt)
    call(None)
    want = [x.clone() for x in grads]
    side = torch.cuda.Stream()
    for _ in range(5):
        for x in grads:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        call(_handle(side, raw))
        for n in (1 << 16, 1 << 20, 1 << 22):
            torch.full((n,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for x, y in zip(grads, want):   # (the order of the atomic additions may differ)
            assert float((x - y).norm()) <= 1e-4 * float(y.norm())
