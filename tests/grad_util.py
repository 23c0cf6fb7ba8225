"""Plain forms, in 64 bits, of the gradients of attention and of norm and rotation, with a bound for each value of the
kernels' results, derived from their arithmetic (not from what they give)."""
import math

import torch

F64 = torch.float64
# fp16 rounds by at most 2^-11 of a value; what lies below its normal range by at most 2^-25
H, SUB = 2.0 ** -11, 2.0 ** -25
TYPE_EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attention_forward(q, k, v, see, scale):
    """o, lse (fp32, as a forward call leaves them) of q [B, T, H, D] over k, v [B, n, Hk, D]; see: bool [B, T, n]."""
    B, T, Hq, D = q.shape
    G = Hq // k.shape[2]
    s = torch.einsum("bthd,bnhd->bhtn", q.to(F64), k.to(F64).repeat_interleave(G, 2)) * scale
    s = s.masked_fill(~see.unsqueeze(1), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.unsqueeze(-1)).nan_to_num(0.0)
    o = torch.einsum("bhtn,bnhd->bthd", p, v.to(F64).repeat_interleave(G, 2))
    return o.float().contiguous(), lse.permute(0, 2, 1).float().contiguous()


def attention_backward(q, k, v, see, scale, o, lse, d_o, d_lse=None):
    """(dq, dk, dv) and their bounds, from the definition with the given o and lse, head by head.

    Errors of the kernels' arithmetic, for one probability p and ds = p (dp - delta):
      p:  the scores' fp32 sums (cut off, not rounded: 2^-23 of the sum of magnitudes for each of D/16 steps),
          the rounding of score, lse and their difference (2^-22 of their sizes), exp2's 2^-22; then fp16: 2^-11, or
          2^-40 where 2^15 p lies below the normal range;
      dp, delta: fp32 sums of at most 128 products (2^-19 of the sums of magnitudes leaves room), and an fp32 d_o is
          rounded to fp16 first: 2^-11 of each value, 2^-25 2^-13 of the row's largest below the normal range;
      ds: the fp16 number that enters the product: 2^-11, or 2^-25 of its scale 2^(e - 15), e at most 3 above the
          largest possible |dp - delta| (a row's own for dq, the call's largest one for dk);
          What this takes from the terms of a row of dq is given back for the mean m of one tile's keys (of 128, those
          behind the last one that the row's tile sees counted as zeros): sum eps_k K_k - (sum eps_k) m, so |eps_k| |K_k - m|
          stands in the bound, with |m| at most the largest mean that the first keys of a tile have;
      sums over keys or rows: fp32, cut off every 16 terms within stretches of 16384: 2^-24 of the sum of magnitudes for
          each of at most 1024 steps.
    """
    B, T, Hq, D = q.shape
    n, Hk = k.shape[1], k.shape[2]
    G = Hq // Hk
    f32do = d_o.dtype == torch.float32
    dq, bq = (torch.zeros((B, T, Hq, D), dtype=F64, device=q.device) for _ in "ab")
    dk, dv, bk, bv = (torch.zeros((B, n, Hk, D), dtype=F64, device=q.device) for _ in "abcd")
    steps = 2.0 ** -24 * 1024
    for b in range(B):
        for h in range(Hq):
            live = see[b].any(1) & (lse[b, :, h] > -math.inf)
            sb = see[b] & live.unsqueeze(1)
            seen = sb.any(0)
            qq, dd, oo = (torch.where(live.unsqueeze(1), x[b, :, h].to(F64), 0.0) for x in (q, d_o, o))
            kk, vv = (torch.where(seen.unsqueeze(1), x[b, :, h // G].to(F64), 0.0) for x in (k, v))
            ll = torch.where(live, lse[b, :, h].to(F64), 0.0)
            s = qq @ kk.t() * scale
            sa = qq.abs() @ kk.abs().t() * abs(scale)
            p = torch.where(sb, torch.exp(s - ll.unsqueeze(1)), 0.0)
            dp = dd @ vv.t()
            delta = (dd * oo).sum(1, keepdim=True)
            da = dd.abs() @ vv.abs().t() + (dd * oo).abs().sum(1, keepdim=True)
            if d_lse is not None:
                dl = torch.where(live, d_lse[b, :, h].to(F64), 0.0).unsqueeze(1)
                delta, da = delta - dl, da + dl.abs()
            ds = p * (dp - delta)
            # |error of p| / p, then of ds
            ep = (sa * (D / 16) * 2.0 ** -23 + (s.abs() + ll.abs().unsqueeze(1)) * 2.0 ** -22 + 2.0 ** -21)
            top = dd.abs().amax(1, keepdim=True) if f32do else 0.0 * delta
            edp = da * (2.0 ** -19 + (H if f32do else 0.0)) + (top * 2.0 ** -38 * (vv.abs().sum(1) + oo.abs().sum(1, keepdim=True)) if f32do else 0.0)
            eds = ds.abs() * ep + p * edp
            size = torch.linalg.vector_norm(dd, dim=1, keepdim=True) * torch.linalg.vector_norm(vv, dim=1).max() + delta.abs()
            tiles = torch.nn.functional.pad(kk, (0, 0, 0, -n % 128)).view(-1, 128, D).cumsum(1) / 128
            mean = tiles.abs().amax((0, 1))
            sub_q, sub_k = size * 2.0 ** -40 * 8, size.max() * 2.0 ** -40 * 8
            dq[b, :, h] = ds @ kk * scale
            bq[b, :, h] = ((eds + ds.abs() * H + sub_q) * sb) @ kk.abs() * abs(scale) + ds.abs() @ kk.abs() * abs(scale) * steps
            bq[b, :, h] += ((ds.abs() * H + sub_q) * sb).sum(1, keepdim=True) * mean * abs(scale)
            dk[b, :, h // G] += ds.t() @ qq * scale
            bk[b, :, h // G] += ((eds + ds.abs() * H + sub_k) * sb).t() @ qq.abs() * abs(scale) + ds.abs().t() @ qq.abs() * abs(scale) * steps
            dv[b, :, h // G] += p.t() @ dd
            # an fp32 d_o's rows are taken against the largest one: 2^15 p of a small row may lie below fp16's normal range
            psub = 2.0 ** -40 * (dd.abs().max() / top.clamp_min(1e-300)).clamp_max(1e30) * 2 if f32do else 2.0 ** -40 + 0.0 * delta
            bv[b, :, h // G] += ((p * (ep + H + (H if f32do else 0.0)) + psub) * sb).t() @ dd.abs() + p.t() @ dd.abs() * steps
            if f32do:
                bv[b, :, h // G] += (p.t() @ top) * 2.0 ** -38
    return (dq, dk, dv), (bq, bk, bv)


def check(got, want, bound, what):
    """|got - want| within the bound and half a step of got's type (with that type's smallest step)."""
    eps = TYPE_EPS[got.dtype]
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}[got.dtype]
    g = got.to(F64)
    assert g.shape == want.shape, f"{what}: {tuple(g.shape)} instead of {tuple(want.shape)}"
    assert torch.isfinite(g).all(), f"{what}: {int((~torch.isfinite(g)).sum())} values are not finite"
    room = bound * (1 + eps) + want.abs() * eps + tiny
    off = (g - want).abs()
    bad = off > room
    if bad.any():
        at = int((off / room).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, the worst at {at}: got "
                             f"{g.flatten()[at]:.8g}, want {want.flatten()[at]:.8g} +- {room.flatten()[at]:.3g}")


def rope_forward(x, w, pos, freq, axis, interleaved, factor=1.0, eps=1e-6):
    """Norm and rotation of x [n, heads, D] in 64 bits; pos [axes, n], freq, axis [R/2]."""
    x, R = x.to(F64), 2 * freq.numel()
    y = x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.to(F64)
    th = (pos[axis.long()].to(F64) * freq.to(F64).unsqueeze(1)).t().unsqueeze(1)
    c, s = factor * th.cos(), factor * th.sin()
    i = torch.arange(R // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out
