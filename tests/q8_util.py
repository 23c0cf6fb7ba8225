"""References of the calls over 8-bit pages, in 64 bits and page by page from
their definitions, and the tolerances that follow from the arithmetic."""
import math

import numpy as np

PAGE = 64


class Cache:
    """A pool, lists and lengths on the host (numpy), with values drawn to order."""

    def __init__(self, rng, lens, Hk, D, *, spare=3, extra=0, shuffle=True, cap=None):
        self.S, self.Hk, self.D = len(lens), Hk, D
        self.lens = np.asarray(lens, np.int32)
        held = [-(-(int(n) + extra) // PAGE) for n in lens]
        self.cap = max(held) + 2 if cap is None else cap
        self.n_pages = sum(held) * Hk + spare
        order = rng.permutation(self.n_pages) if shuffle else np.arange(self.n_pages)
        self.ids = np.full((self.S, Hk, self.cap), -1, np.int32)
        at = 0
        for s, n in enumerate(held):
            for k in range(Hk):
                self.ids[s, k, :n] = order[at:at + n]
                at += n
        self.k = np.clip(np.rint(rng.standard_normal((self.n_pages, PAGE, D)) * 30), -127, 127).astype(np.int8)
        self.v = np.clip(np.rint(rng.standard_normal((self.n_pages, PAGE, D)) * 30), -127, 127).astype(np.int8)
        self.ks = rng.uniform(0.02, 0.05, self.n_pages).astype(np.float32)
        self.vs = rng.uniform(0.005, 0.05, self.n_pages).astype(np.float32)
        self.lo = np.zeros((self.n_pages, D), np.int8)
        self.hi = np.zeros((self.n_pages, D), np.int8)
        self.extremes()

    def extremes(self):
        for s in range(self.S):
            for k in range(self.Hk):
                for b in range(-(-int(self.lens[s]) // PAGE)):
                    p = self.ids[s, k, b]
                    if p >= 0:
                        rows = self.k[p, :min(PAGE, int(self.lens[s]) - b * PAGE)]
                        self.lo[p], self.hi[p] = rows.min(0), rows.max(0)

    def on_gpu(self):
        import torch
        import split_kv_flash_attn_gb300 as skv
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()   # noqa: E731
        pool = skv.Q8Pool(dev(self.k), dev(self.v), dev(self.ks), dev(self.vs), dev(self.lo), dev(self.hi))
        return pool, dev(self.ids), dev(self.lens)


def visible(c, s, t, q_pos):
    n = int(c.lens[s])
    return n if q_pos is None else max(0, min(n, int(q_pos[s, t]) + 1))


def attention(c, q, *, q_pos=None, sel=None, scale=None):
    """(o, lse, mass, tol_o, tol_lse) in 64 bits.

    tol: a score is a sum of D exact products in fp32, each addition off by at
    most 2^-23 of the sums' magnitude (bounded by sum |q k|), and two more fp32
    products: off by (D + 4) 2^-23 A in all, A = scale * max sum |q_d k_d|.
    2^x (2^-22), the shift by the reference (2^-23 |x|), the split of a weight in two (2^-22)
    and the sums' rest add 2^-19 generously: each probability is off by e =
    (D + 4) 2^-23 A + 2^-19 relative, so o by 2 e max|v| and lse by e + 2^-22 |lse|."""
    S, nq, H, D = q.shape
    Hk, G = c.Hk, H // c.Hk
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = np.zeros((S, nq, H, D))
    lse = np.full((S, nq, H), -np.inf)
    mass = np.zeros((S, Hk, c.cap))
    A = vmax = 0.0
    for s in range(S):
        for k in range(Hk):
            for t in range(nq):
                m = visible(c, s, t, q_pos)
                blocks = range(-(-m // PAGE)) if sel is None else [b for b in map(int, sel[s, t, k]) if 0 <= b and b * PAGE < m]
                ks, vs, at = [], [], []
                for b in blocks:
                    p = int(c.ids[s, k, b])
                    if p < 0 or p >= c.n_pages:
                        continue
                    n = min(PAGE, m - b * PAGE)
                    ks.append(c.k[p, :n].astype(np.float64) * float(c.ks[p]))
                    vs.append(c.v[p, :n].astype(np.float64) * float(c.vs[p]))
                    at.append((b, n))
                if not ks:
                    continue
                kk, vv = np.concatenate(ks), np.concatenate(vs)
                vmax = max(vmax, np.abs(vv).max())
                qq = q[s, t, k * G:(k + 1) * G].astype(np.float64)
                w = qq @ kk.T * scale
                A = max(A, (np.abs(qq) @ np.abs(kk).T).max() * abs(scale))
                top = w.max(1, keepdims=True)
                e = np.exp(w - top)
                z = e.sum(1, keepdims=True)
                p = e / z
                o[s, t, k * G:(k + 1) * G] = p @ vv
                lse[s, t, k * G:(k + 1) * G] = (top + np.log(z))[:, 0]
                i = 0
                for b, n in at:
                    mass[s, k, b] += p[:, i:i + n].sum()
                    i += n
    err = (D + 4) * 2.0 ** -23 * A + 2.0 ** -19
    fin = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
    return o, lse, mass, 2 * err * vmax, err + 2.0 ** -22 * fin, vmax


def check(o, lse, ref, *, f16=False, what=""):
    ro, rl, _, tol_o, tol_l, vmax = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl)), f"{what}: rows without a key differ"
    on = np.isfinite(rl)
    assert np.all(o[~on] == 0.0), f"{what}: a row without a key has o != 0"
    assert np.all(np.isfinite(o))
    if not on.any():
        return
    if f16:   # the result's rounding, and one of each weight: 2^-11 relative; below 2^-14 half a step is 2^-25
        tol_o = tol_o + 2.0 ** -11 * np.abs(ro[on]).max() + 2.0 ** -11 * vmax + 2.0 ** -25
    d = np.abs(o[on] - ro[on]).max()
    assert d <= tol_o, f"{what}: max|do| = {d:.3e} > {tol_o:.3e}"
    d = np.abs(lse[on] - rl[on]).max()
    assert d <= tol_l, f"{what}: max|dlse| = {d:.3e} > {tol_l:.3e}"


def code(x, d):
    """The integer nearest x / d: the quotient of two fp32 numbers cannot be
    rounded onto a half-integer in 64 bits that it is not."""
    x = np.asarray(x, np.float32).astype(np.float64)
    if d == 0:
        return np.zeros(x.shape, np.int8)
    with np.errstate(invalid="ignore"):
        r = np.clip(np.rint(x / float(d)), -127, 127)
    return np.where(np.isnan(x), 0, r).astype(np.int8)


def append(c, k_new, v_new, n_new=None):
    """skv_q8_append on the host cache (lengths are not advanced)."""
    S, n_max = k_new.shape[:2]
    for s in range(S):
        n = n_max if n_new is None else min(n_max, max(0, int(n_new[s])))
        m = int(c.lens[s])
        for k in range(c.Hk):
            for b in range(m // PAGE, -(-(m + n) // PAGE) if n else 0):
                p = int(c.ids[s, k, b]) if b < c.cap else -1
                if p < 0 or p >= c.n_pages:
                    continue
                lo, hi = max(m - b * PAGE, 0), min(m + n - b * PAGE, PAGE)
                for x, codes, scale in ((k_new, c.k, c.ks), (v_new, c.v, c.vs)):
                    rows = x[s, b * PAGE + lo - m:b * PAGE + hi - m, k].astype(np.float32)
                    mag = np.abs(rows)
                    top = mag[np.isfinite(mag)].max(initial=0.0)
                    d0 = np.float32(scale[p]) if lo > 0 else np.float32(0)
                    d1 = max(d0, np.float32(np.float64(top) / 127.0))
                    if lo > 0 and d1 != d0:
                        codes[p, :lo] = np.rint(codes[p, :lo].astype(np.float64) * float(d0) / float(d1)).astype(np.int8)
                    codes[p, lo:hi] = code(rows, d1)
                    scale[p] = d1
                c.lo[p], c.hi[p] = c.k[p, :hi].min(0), c.k[p, :hi].max(0)


def select(c, q, n_sel, n_first, n_last, q_pos=None):
    S, nq, H, D = q.shape
    G = H // c.Hk
    out = np.full((S, nq, c.Hk, n_sel), -1, np.int32)
    for s in range(S):
        for t in range(nq):
            nb = -(-visible(c, s, t, q_pos) // PAGE)
            for k in range(c.Hk):
                rank = []
                for b in range(nb):
                    p = int(c.ids[s, k, b])
                    if p < 0 or p >= c.n_pages:
                        continue
                    best = None
                    for h in range(k * G, (k + 1) * G):
                        x = q[s, t, h].astype(np.float32)
                        dq = np.float32(np.float64(np.abs(x).max()) / 127.0)
                        cq = code(x, dq).astype(np.int64)
                        dot = int(np.maximum(cq * c.lo[p].astype(np.int64), cq * c.hi[p].astype(np.int64)).sum())
                        f = np.float32(np.float32(dot) * dq)
                        best = f if best is None else max(best, f)
                    must = b < n_first or b >= nb - n_last
                    rank.append((not must, -float(np.float32(best * c.ks[p])), b))
                pick = sorted(b for _, _, b in sorted(rank)[:n_sel])
                out[s, t, k, :len(pick)] = pick
    return out


def evict(ids, mass, lens, n_keep, n_first, n_last):
    S, Hk, cap = ids.shape
    oi, om = np.full_like(ids, -1), np.zeros_like(mass)
    fr, ol = np.full_like(ids, -1), np.array(lens, np.int32)
    for s in range(S):
        n = -(-int(lens[s]) // PAGE)
        out = max(0, n - n_keep)
        ol[s] -= out * PAGE
        for k in range(Hk):
            m = mass[s, k].astype(np.float64)
            m = np.where(np.isnan(m), np.inf, m)
            m = np.where(ids[s, k] < 0, -np.inf, m)      # absent pages go first, all alike
            rank = sorted(range(n), key=lambda b: (not (b < n_first or b >= n - n_last), ids[s, k, b] < 0, -m[b], b))
            keep = sorted(rank[:n_keep])
            gone = [b for b in range(n) if b not in set(keep) and ids[s, k, b] >= 0]
            row = [ids[s, k, b] for b in keep] + list(ids[s, k, n:])
            oi[s, k, :len(row)] = row
            om[s, k, :len(keep)] = mass[s, k, keep]
            fr[s, k, :len(gone)] = ids[s, k, gone]
    return oi, om, ol, fr
