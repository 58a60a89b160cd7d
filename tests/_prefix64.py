"""Shared-prefix attention in 64 bits with torch, for problems too large for the oracle's loops, and the bound of
the kernels' errors (derived in test_parity_prefix.py, whose numbers these are)."""

import math

import numpy as np
import torch

V = 2.0 ** -24


def attention(q, kp, vp, ks, vs, lens, scale=None):
    """(out, lse, sum p |v|) as oracle.attention_prefix has them; tensors of any type on one device."""
    B, S_Q, H, d = q.shape
    Hkv = (kp if kp is not None else ks).shape[-2]
    G, dev = H // Hkv, q.device
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(B, S_Q, H, d, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(out)
    lse = torch.full((B, H, S_Q), -math.inf, dtype=torch.float64, device=dev)
    none = torch.zeros(0, Hkv, d, dtype=torch.float64, device=dev)
    k0, v0 = (none if x is None else x.double() for x in (kp, vp))
    for b in range(B):
        n = 0 if ks is None else min(max(int(lens[b]), 0), ks.shape[1])
        k = torch.cat((k0, ks[b, :n].double())) if n else k0
        v = torch.cat((v0, vs[b, :n].double())) if n else v0
        if not len(k):
            continue
        x = torch.einsum("tgjd,kgd->gtjk", q[b].double().view(S_Q, Hkv, G, d), k) * scale
        j, t = torch.arange(len(k), device=dev), torch.arange(S_Q, device=dev)[:, None]
        seen = j < len(k0) + (n - S_Q + 1 + t).clamp(min=0)
        x = x.masked_fill(~seen[None, :, None], -math.inf)
        top = x.amax(-1, keepdim=True).clamp(min=-1e300)
        p = (x - top).exp()
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
        out[b] = torch.einsum("gtjk,kgd->tgjd", p, v).reshape(S_Q, H, d)
        mag[b] = torch.einsum("gtjk,kgd->tgjd", p, v.abs()).reshape(S_Q, H, d)
        lse[b] = (top + total.log())[..., 0].permute(0, 2, 1).reshape(H, S_Q)
    return out, lse, mag


def check(out, lse, args, scale=None, what="", rows=None, kmax=None):
    """The outputs against 64 bits; rows [B, S_Q, H]: those that count; kmax: norm of the longest key that does."""
    q, kp, vp, ks, vs, n = args
    ref, ref_l, mag = attention(*args, scale=scale)
    d = q.shape[-1]
    sc = d ** -0.5 if scale is None else scale
    longest = lambda x: float(x.float().nan_to_num(0, 0, 0).norm(dim=-1).max())  # noqa: E731
    kmax = kmax or max(longest(x) for x in (kp, ks) if x is not None and x.numel())
    keys = sum(x.shape[-3] for x in (kp, ks) if x is not None)
    e = (d + 2) * V * sc * q.double().norm(dim=-1) * kmax          # [B, S_Q, H]
    r = 2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0
    tol = (2 * (e[..., None] + 2.0 ** -21) + r + (keys + 64) * V) * mag + torch.finfo(q.dtype).eps / 2 * ref.abs()
    rows = torch.ones_like(e, dtype=torch.bool) if rows is None else rows
    worst = ((out.double() - ref).abs() - 1.01 * tol)[rows]
    assert torch.isfinite(out[rows]).all() and worst.max() <= 0, f"{what} out: {float(worst.max()):.3e} over the bound"
    fin = torch.isfinite(ref_l) & rows.transpose(1, 2)
    empty = torch.isneginf(ref_l) & rows.transpose(1, 2)
    assert torch.isneginf(lse[empty]).all() and (out.transpose(1, 2)[empty] == 0).all(), what
    tol = e.transpose(1, 2) + 2.0 ** -20 + (keys + 64) * V + 4 * V * ref_l.abs()
    worst = ((lse.double() - ref_l).abs() - 1.01 * tol)[fin]
    assert not fin.any() or worst.max() <= 0, f"{what} lse: {float(worst.max()):.3e} over the bound"


def as_oracle(args):
    """The same problem as numpy arrays in 64 bits."""
    return [None if x is None else np.asarray(x.double().cpu()) for x in args]
