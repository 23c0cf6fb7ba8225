"""More references of the calls over 8-bit pages, in 64 bits: scales of either
sign, and attention with a bound for each row from what that row sees."""
import math

import numpy as np

from q8_util import PAGE, code, visible


def append(c, k_new, v_new):
    """skv_q8_append on the host cache (lengths are not advanced), page by page as the header
    states it: d' = max(|d|, fp32(amax / 127)), and earlier codes are those nearest c d / d'
    where d' is another number than d."""
    S, n = k_new.shape[:2]
    for s in range(S):
        m = int(c.lens[s])
        for k in range(c.Hk):
            for b in range(m // PAGE, -(-(m + n) // PAGE)):
                p = int(c.ids[s, k, b])
                lo, hi = max(m - b * PAGE, 0), min(m + n - b * PAGE, PAGE)
                for x, codes, scale in ((k_new, c.k, c.ks), (v_new, c.v, c.vs)):
                    rows = x[s, b * PAGE + lo - m:b * PAGE + hi - m, k].astype(np.float32)
                    d0 = np.float32(scale[p]) if lo > 0 else np.float32(0)
                    d1 = max(abs(d0), np.float32(np.abs(rows).astype(np.float64).max() / 127.0))
                    if lo > 0 and d1 != d0:
                        codes[p, :lo] = np.rint(codes[p, :lo].astype(np.float64) * float(d0) / float(d1)).astype(np.int8)
                    codes[p, lo:hi] = code(rows, d1)
                    scale[p] = d1
                c.lo[p], c.hi[p] = c.k[p, :hi].min(0), c.k[p, :hi].max(0)


def select(c, q, n_sel, n_first, n_last, q_pos=None):
    """skv_q8_select: a page's bound is |k_scale| times the largest, over the head's queries, of
    fp32(dq * sum_d max(cq_d x_d, cq_d y_d)), x and y the extremes of sign(k_scale) k."""
    S, nq, H, D = q.shape
    G = H // c.Hk
    out = np.full((S, nq, c.Hk, n_sel), -1, np.int32)
    for s in range(S):
        for t in range(nq):
            nb = -(-visible(c, s, t, q_pos) // PAGE)
            for k in range(c.Hk):
                x = q[s, t, k * G:(k + 1) * G].astype(np.float32)
                dq = (np.abs(x).astype(np.float64).max(1) / 127.0).astype(np.float32)
                cq = np.stack([code(r, d) for r, d in zip(x, dq)]).astype(np.int64)
                rank = []
                for b in range(nb):
                    p = int(c.ids[s, k, b])
                    if p < 0 or p >= c.n_pages:
                        continue
                    sign = -1 if c.ks[p] < 0 else 1
                    lo, hi = sign * c.lo[p].astype(np.int64), sign * c.hi[p].astype(np.int64)
                    f = np.maximum(cq * lo, cq * hi).sum(1).astype(np.float32) * dq
                    must = b < n_first or b >= nb - n_last
                    rank.append((not must, -float(np.float32(f.max() * np.abs(c.ks[p]))), b))
                pick = sorted(b for _, _, b in sorted(rank)[:n_sel])
                out[s, t, k, :len(pick)] = pick
    return out


def attention(c, q, *, q_pos=None, sel=None):
    """(o, lse, tol_o, tol_lse, vmax) in 64 bits, the last three for each row: as in q8_util.attention, with
    the largest |v| and the largest sum |q_d k_d| of the keys that the row sees itself."""
    S, nq, H, D = q.shape
    Hk, G = c.Hk, H // c.Hk
    o = np.zeros((S, nq, H, D))
    lse = np.full((S, nq, H), -np.inf)
    tol, vmax = np.zeros((S, nq, H)), np.zeros((S, nq, H))
    for s in range(S):
        for k in range(Hk):
            for t in range(nq):
                m = visible(c, s, t, q_pos)
                blocks = range(-(-m // PAGE)) if sel is None else [b for b in map(int, sel[s, t, k]) if 0 <= b and b * PAGE < m]
                kk, vv = [], []
                for b in blocks:
                    p, n = int(c.ids[s, k, b]), min(PAGE, m - b * PAGE)
                    if 0 <= p < c.n_pages:
                        kk.append(c.k[p, :n].astype(np.float64) * float(c.ks[p]))
                        vv.append(c.v[p, :n].astype(np.float64) * float(c.vs[p]))
                if not kk:
                    continue
                kk, vv = np.concatenate(kk), np.concatenate(vv)
                rows = slice(k * G, (k + 1) * G)
                x = q[s, t, rows].astype(np.float64)
                w = x @ kk.T / math.sqrt(D)
                top = w.max(1, keepdims=True)
                e = np.exp(w - top)
                z = e.sum(1, keepdims=True)
                o[s, t, rows] = e / z @ vv
                lse[s, t, rows] = (top + np.log(z))[:, 0]
                tol[s, t, rows] = (D + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(kk).T).max(1) / math.sqrt(D) + 2.0 ** -19
                vmax[s, t, rows] = np.abs(vv).max()
    return o, lse, 2 * tol * vmax, tol + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0), vmax


def check(o, lse, ref, *, f16=False):
    """Every row within its own bound.  fp16: the result's rounding and one of each weight, half a step
    (2^-11) of each, and half a step of the smallest numbers (2^-25)."""
    ro, rl, tol_o, tol_l, vmax = ref
    assert str(o.dtype) == ("torch.float16" if f16 else "torch.float32")
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl)) and np.all(o[np.isneginf(rl)] == 0)
    if f16:
        tol_o = tol_o + 2.0 ** -11 * (np.abs(ro).max(-1) + vmax) + 2.0 ** -25
    off = np.abs(o - ro).max(-1) - tol_o
    at = np.unravel_index(off.argmax(), off.shape)
    assert off[at] <= 0, f"row {at}: max|do| = {off[at] + tol_o[at]:.3e} > {tol_o[at]:.3e}"
    on = np.isfinite(rl)
    assert np.all(np.abs(lse[on] - rl[on]) <= tol_l[on])
