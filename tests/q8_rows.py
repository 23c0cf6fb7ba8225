"""More references of the calls over 8-bit pages, in 64 bits: scales of either sign."""
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
