"""Plain float64 definitions of the microscaled 4-bit operators and of the
routing from logits, shared by their CPU and GPU tests (numpy, no code of the
package)."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(x):
    """Scale byte of every block of 32 of x [..., K] (float64 holding the input values)."""
    b = np.abs(x).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        amax = b.max(-1)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, amax)
    e = np.frexp(amax)[1] - 3  # floor(log2) - 2
    e = np.where(amax == 0, -127, np.maximum(e, -127))
    return np.where(bad, 255, e + 127).astype(np.uint8)


def codes_under(x, s):
    """e2m1 codes of x [..., K] under given scale bytes [..., K/32] (255: zeros)."""
    e = s.astype(np.int64) - 127
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.ldexp(x.reshape(*x.shape[:-1], -1, 32), -e[..., None])
    v = np.where((s == 255)[..., None], 0.0, v)
    a = np.abs(v)
    d = np.abs(a[..., None] - LEVELS)
    near = d.argmin(-1)                       # the lower of two equal distances
    up = np.minimum(near + 1, 7)
    tie = (d[..., 0] < 0) | (np.take_along_axis(d, up[..., None], -1)[..., 0]
                             == np.take_along_axis(d, near[..., None], -1)[..., 0])
    code = np.where(tie & (up > near) & (near % 2 == 1), up, near)
    code = code + 8 * np.signbit(v)
    return code.reshape(x.shape).astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    out = np.empty((*codes.shape[:-1], codes.shape[-1] * 2), np.uint8)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def values(code, s):
    """float64 values of codes [..., K] under scale bytes [..., K/32]."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    unit = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v.reshape(*code.shape[:-1], -1, 32) * unit[..., None]).reshape(code.shape)


def quantised(x):
    s = scale_bytes(x)
    return values(codes_under(x, s), s)


def tile(s):
    """Scale bytes [rows, K/32] -> tiles [ceil(rows/128), ceil(K/128), 512], by the definition."""
    rows, cols = s.shape
    out = np.zeros(((rows + 127) // 128, (cols + 3) // 4, 512), np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    out[r // 128, c // 4, r % 32 * 16 + r % 128 // 32 * 4 + c % 4] = s
    return out


def slack(x, err):
    """Largest change of quantised(x) when every x moves by at most err
    (elementwise bound): the block's scale may be that of amax - err or amax +
    err, and under each scale the rounding is monotone."""
    q = quantised(x)
    out = np.zeros_like(q)
    b = np.abs(x).reshape(*x.shape[:-1], -1, 32)
    eb = err.reshape(b.shape)
    for hi in (False, True):
        amax = np.maximum((b + eb if hi else b - eb).max(-1), 0.0)
        ref = np.zeros_like(b)
        ref[..., 0] = amax
        s = scale_bytes(ref.reshape(x.shape))
        for sign in (-1, 1):
            out = np.maximum(out, np.abs(values(codes_under(x + sign * err, s), s) - q))
    return out


# --------------------------------------------------------------- routing ---

def route(logits, k, renorm, mask=None):
    """Routing from logits [T, E] (float64 holding the inputs): a dict."""
    T, E = logits.shape
    valid = np.ones(T, bool) if mask is None else mask.astype(bool)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        valid = valid & ~(np.isneginf(logits).all(1))
        m = logits.max(1, keepdims=True) if E else logits
        p = np.exp(logits - m)
        p = p / p.sum(1, keepdims=True)
    ids = np.sort(np.argsort(-logits, axis=1, kind="stable")[:, :k], axis=1)
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        with np.errstate(invalid="ignore"):
            w = w / w.sum(1, keepdims=True)
    w = np.where(valid[:, None], w, 0.0)
    p = np.where(valid[:, None], p, 0.0)
    counts = np.bincount(ids[valid].ravel(), minlength=E)
    n = max(int(valid.sum()), 1)
    loss = E * float((counts / (n * k) * (p.sum(0) / n)).sum())
    return {"ids": ids, "w": w, "p": p, "counts": counts, "prob_sums": p.sum(0), "loss": loss,
            "valid": valid}


def route_grad(logits, k, renorm, dw, dloss, mask=None, ids=None, counts=None):
    """d/dlogits of sum dw * w + dloss * loss, ids and counts held fixed."""
    r = route(logits, k, renorm, mask)
    ids = r["ids"] if ids is None else ids
    counts = r["counts"] if counts is None else counts
    T, E = logits.shape
    n = counts.sum() / k
    dp = np.zeros((T, E))
    if n > 0:
        dp += dloss * E * counts / (n * k) / n
    if dw is not None:
        chosen = np.take_along_axis(r["p"], ids, 1)
        g = dw
        if renorm:
            tot = chosen.sum(1, keepdims=True)
            tot = np.where(tot > 0, tot, 1.0)
            g = (dw - (dw * chosen / tot).sum(1, keepdims=True)) / tot
        np.add.at(dp, (np.arange(T)[:, None], ids), g)
    return r["p"] * (dp - (r["p"] * dp).sum(1, keepdims=True))
