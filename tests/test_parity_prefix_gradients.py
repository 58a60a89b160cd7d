"""Gradients over a shared prefix and ragged suffixes from the accumulating backward, as the header composes them
(GPU)."""

import pytest
import torch

from blockwise_long_context_b200 import binding as lvx

pytestmark = pytest.mark.gpu


def _accumulated(args, lens, out, lse, do):
    q, kp, vp, ks, vs, _ = args
    B, S, H, d = q.shape
    dq, dkp, dvp, dks, dvs = (torch.zeros(x.shape, device="cuda") for x in (q, kp, vp, ks, vs))
    flat = lambda x: x.reshape(1, B * S, H, d)  # noqa: E731
    lvx.lvx_attn_bwd_accumulate(flat(q), kp[None], vp[None], flat(out), lse.permute(1, 0, 2).reshape(1, H, B * S).contiguous(),
                                flat(do), dq.view(1, B * S, H, d), dkp[None], dvp[None])
    for b, n in enumerate(lens):
        def add(first, k0, k1, causal):
            rows, keys = slice(first, S), slice(k0, k1)
            one = lambda x, at: x[b:b + 1, at].contiguous()  # noqa: E731
            part = [torch.zeros_like(one(x, at)) for x, at in ((dq, rows), (dks, keys), (dvs, keys))]
            lvx.lvx_attn_bwd_accumulate(one(q, rows), one(ks, keys), one(vs, keys), one(out, rows),
                                        lse[b:b + 1, :, first:].contiguous(), one(do, rows), *part, causal=causal)
            dq[b, rows] += part[0][0]
            dks[b, keys] += part[1][0]
            dvs[b, keys] += part[2][0]
        if n > S:
            add(0, 0, n - S, False)
        if n > 0:
            m = min(n, S)
            add(S - m, n - m, n, True)
    return dq, dkp, dvp, dks, dvs


@pytest.mark.parametrize("dt,bar", [(torch.float32, 1e-5), (torch.bfloat16, 1e-2)])   # the framework's bars
@pytest.mark.parametrize("S", [1, 6])
def test_ragged_suffixes(dt, bar, S):
    lens = [0, 2, S, S + 1, 37]
    B, H, H_kv, d, S_P, cap = len(lens), 4, 2, 64, 130, 40
    g = torch.Generator().manual_seed(S)
    t = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = t(B, S, H, d), t(S_P, H_kv, d), t(S_P, H_kv, d), t(B, cap, H_kv, d), t(B, cap, H_kv, d), n
    do = t(B, S, H, d)
    out, lse = lvx.attention_prefix(*args)
    got = _accumulated(args, lens, out, lse, do)
    lvx.lvx_last_device_error()
    x = [a.double().cpu().requires_grad_() for a in args[:5]]   # in 64 bits on the host
    rep = lambda a: a.repeat_interleave(H // H_kv, -2)  # noqa: E731
    k = torch.cat((rep(x[1]).expand(B, S_P, H, d), rep(x[3])), 1)
    v = torch.cat((rep(x[2]).expand(B, S_P, H, d), rep(x[4])), 1)
    s = torch.einsum("bthd,bjhd->bhtj", x[0], k) * d ** -0.5
    j, at = torch.arange(S_P + cap), torch.arange(S)[:, None]
    seen = (j < S_P) | (j - S_P <= (n.cpu()[:, None, None] - S + at))
    s = s.masked_fill(~seen[:, None], -torch.inf)
    o = torch.einsum("bhtj,bjhd->bthd", torch.softmax(s, -1), v)
    for a, b, name in zip(got, torch.autograd.grad(o, x, do.double().cpu()), ("dq", "dkp", "dvp", "dks", "dvs")):
        assert float((a.double().cpu() - b).norm() / b.norm()) < bar, name
