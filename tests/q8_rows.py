"""More references of the calls over 8-bit pages, in 64 bits: scales of either sign."""
import numpy as np

from q8_util import PAGE, code


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
