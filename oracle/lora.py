"""Low-rank adapters of many requests beside a shared projection.

Oracle (test infrastructure only; see ``oracle/__init__.py``): y_r = base_r + s_a B_a (A_a x_r) in
float64, a = the row's adapter; an id outside [0, adapters) leaves the base (-1 says so, others are
bad data). The pages run one set of weights for all streams, so this is the library's own reading.
"""
import numpy as np


def lora(x, a, b, ids, base=None, scales=None):
    """(exact y [R][n], the magnitude |base| + |s| |B| (|A| |x|) that bounds its fp32 error, bad)."""
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    R, n = x.shape[0], b.shape[1]
    y = np.zeros((R, n)) if base is None else np.array(base, dtype=np.float64)
    mag, bad = np.abs(y), False
    for r in range(R):
        i = int(ids[r])
        if not 0 <= i < a.shape[0]:
            bad |= i != -1
            continue
        s = 1.0 if scales is None else float(scales[i])
        y[r] += s * (b[i] @ (a[i] @ x[r]))
        mag[r] += abs(s) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[r])))
    return y, mag, bad
