"""64-bit reference of the int8 operators (numpy), and the error bounds their kernels are
held to.  Shares no code with the library."""
import numpy as np

U32 = 2.0 ** -24  # unit roundoff of fp32


def quantize(x):
    """(codes, scales) of float32 rows by the definition: each of its operations is a
    single fp32 operation, so this is exact."""
    x = np.asarray(x, np.float32)
    fine = np.isfinite(x).all(1)
    v = np.where(fine[:, None], x, np.float32(0))
    a = np.maximum(np.abs(v).max(1), np.float32(2.0 ** -100)).astype(np.float32)
    q = np.rint(v * (np.float32(127) / a)[:, None]).astype(np.int8)
    return q, np.where(fine, a / np.float32(127), np.float32(np.nan))


def product(xq, xs, wq, ws):
    """Rows times one expert's weights in 64 bits, and the bound of the kernels' result.

    Sums of codes are whole numbers: exact here, and in the kernel where no partial sum
    can pass 2^24; beyond, each addition of 16 products to an fp32 sum is off by at most
    one fp32 ulp of a partial sum (a truncating adder).  Then the sum, the product of
    the scales and their product are rounded once each."""
    x, w = xq.astype(np.float64), wq.astype(np.float64)
    scale = xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    ref = (x @ w.T) * scale
    mag = np.abs(x) @ np.abs(w).T
    adds = -(-x.shape[1] // 16) + 8
    err = np.where(mag > 2.0 ** 24, mag * adds * 2 * U32, 0.0) * np.abs(scale)
    return ref, err + np.abs(ref) * 3 * U32
