"""Calls with an explicit stream and no workspace (GPU): the workspace that the binding takes belongs to the
stream of the launches, not to the current one."""

import pytest
import torch

from blockwise_long_context_b200 import binding as lvx
from blockwise_long_context_b200 import distributed, ring

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


@pytest.mark.parametrize("raw", [False, True])
def test_the_sharded_calls_run_on_the_explicit_stream(raw):
    """One rank of each sharded call while the current stream is busy: what the call fills, computes and frees
    goes with the given stream."""
    g = torch.Generator().manual_seed(4)
    t = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v, do = t(1, 256, 4, 64), t(1, 512, 2, 64), t(1, 512, 2, 64), t(1, 256, 4, 64)
    out, lse = lvx.attention_forward(q, k, v, 1)
    calls = [lambda s: distributed.xattn_forward_sharded(q, k, v, n_local_blocks=2, stream=s),
             lambda s: distributed.xattn_forward_ring(q, k, v, n_local_blocks=2, stream=s),
             lambda s: ring.ring_attention_forward(q, k, v, stream=s),
             lambda s: distributed.xattn_backward_sharded(q, k, v, out, lse, do, stream=s),
             lambda s: distributed.xattn_backward_ring(q, k, v, out, lse, do, stream=s)]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        torch.cuda._sleep(50_000_000)   # the current stream's work ends after the call's
        got = call(_handle(side, raw))
        side.synchronize()
        torch.full((1 << 22,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for x, y in zip(got, want):   # (bf16 gradients of sums whose order may differ)
            assert float((x.float() - y.float()).norm()) <= 1e-2 * float(y.float().norm())


def test_a_partial_in_an_unaligned_place_on_an_explicit_stream():
    """The copy of a partial whose place is not 16-byte aligned goes with the kernel that writes it."""
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, s, 1, 64, generator=g).bfloat16().cuda() for s in (3, 512, 512))
    l_all = torch.zeros(2, 1, 1, 3, device="cuda")   # the second slice: 12 bytes from the first
    want_o, want_l = torch.zeros(1, 1, 1, 3, 64, device="cuda"), torch.zeros(1, 1, 1, 3, device="cuda")
    ring.kernel_partial()(q, k, v, want_o, want_l, False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = torch.zeros_like(want_o)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    ring.kernel_partial(stream=side)(q, k, v, o, l_all[1:], False)
    side.synchronize()
    assert torch.equal(o, want_o) and torch.equal(l_all[1:], want_l) and (l_all[0] == 0).all()
