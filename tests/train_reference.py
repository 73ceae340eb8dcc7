"""Float64 definitions of the operators that train the routed experts, shared by
their CPU and GPU tests (torch, no code of the package)."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# Below these a rounding is off by half of the type's smallest step instead.
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def group(ids, E, mask=None):
    """places [T, k] and offsets [E + 1]: slots sorted by expert, stable, -1 for none."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    keep = [True] * T if mask is None else [bool(m) for m in mask.tolist()]
    of = [[] for _ in range(E)]
    for f, e in enumerate(flat):
        if keep[f // k] and 0 <= e < E:
            of[e].append(f)
    places = torch.full((T * k,), -1, dtype=torch.int32)
    offsets = [0]
    for slots in of:
        for i, f in enumerate(slots):
            places[f] = offsets[-1] + i
        offsets.append(offsets[-1] + len(slots))
    return places.view(T, k), torch.tensor(offsets, dtype=torch.int32)


def combine(rows, places, w=None):
    """(out, the sum of the terms' magnitudes), float64."""
    T, k = places.shape
    r = rows.double()
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    mag = out.clone()
    for j in range(k):
        p = places[:, j].long()
        has = (p >= 0)[:, None]
        v = r[p.clamp_min(0)]
        if w is not None:
            v = v * w[:, j, None].double()
        out += torch.where(has, v, torch.zeros_like(v))
        mag += torch.where(has, v.abs(), torch.zeros_like(v))
    return out, mag


def product(x, w, offsets, way):
    """(result, the sum of the terms' magnitudes) in float64; rows outside the segments 0.
    way: "forward" (x, w), "dx" (dy, w), "dw" (w is x then, the first argument dy)."""
    off = offsets.tolist()
    E = len(off) - 1
    x, w = x.double(), w.double()
    if way == "dw":
        out = torch.zeros(E, x.shape[1], w.shape[1], dtype=torch.float64, device=x.device)
    else:
        out = torch.zeros(x.shape[0], w.shape[1 if way == "forward" else 2], dtype=torch.float64,
                          device=x.device)
    mag = out.clone()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if way == "dw":
            out[e] = x[a:b].T @ w[a:b]
            mag[e] = x[a:b].abs().T @ w[a:b].abs()
        else:
            m = w[e].T if way == "forward" else w[e]
            out[a:b] = x[a:b] @ m
            mag[a:b] = x[a:b].abs() @ m.abs()
    return out, mag


def _power(e):
    """2^e of whole numbers e, made from its bits: the functions' own powers can be a last
    bit off (2^-4 and 2^11 are, on a GPU), and a value half way between two codes then
    falls to the wrong one (97.5 to 97)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def encode(z):
    """8-bit integers and scale bytes of z [R, C] (any float type)."""
    b = z.double().reshape(z.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    amax = torch.where(bad, torch.ones((), dtype=torch.float64, device=z.device),
                       b.abs().amax(-1))
    e = torch.where(amax == 0, torch.full_like(amax, -127),
                    (torch.frexp(amax)[1] - 7).clamp_min(-127).double())
    q = (b * _power(-e[..., None])).nan_to_num(0, 0, 0).round().clamp(-127, 127)
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    s = torch.where(bad, torch.full_like(e, 255), e + 127)
    return q.reshape(z.shape).to(torch.int8), s.to(torch.uint8)


def decode(q, s):
    e = s.double() - 127
    unit = torch.where(s == 255, torch.full_like(e, float("nan")), _power(e))
    return (q.double().reshape(q.shape[0], -1, 32) * unit[..., None]).reshape(q.shape)


def swiglu(z):
    I = z.shape[1] // 2
    return z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]


def swiglu_grad(z, da, w=None):
    """(dz, act, d_row_w) by the formulas, float64."""
    I = z.shape[1] // 2
    g, u = z[:, :I].double(), z[:, I:].double()
    s = torch.sigmoid(g)
    a, d = g * s * u, da.double()
    wd = d if w is None else d * w.double()[:, None]
    dz = torch.cat((wd * u * s * (1 + g * (1 - s)), wd * g * s), 1)
    return dz, (a if w is None else a * w.double()[:, None]), (d * a).sum(1)


def experts(hidden, ids, w, w_gate_up, w_down, mask=None):
    """The layer's experts in float64, differentiable in every float argument."""
    T, k = ids.shape
    E, H, I = w_down.shape
    rows = []
    for t in range(T):
        y = torch.zeros(H, dtype=torch.float64)
        if mask is None or bool(mask[t]):
            for j in range(k):
                e = int(ids[t, j])
                z = w_gate_up[e] @ hidden[t]
                y = y + w[t, j] * (w_down[e] @ (z[:I] * torch.sigmoid(z[:I]) * z[I:]))
        rows.append(y)
    return torch.stack(rows)


# A sigmoid below 2^-126 is a subnormal number and may be taken as 0. That is g below
# -87.3; where e^-g is infinite (g below -88.8) it is 0 as well and smaller yet. So g
# sigma(g), and sigma (1 + g (1 - sigma)), are off by at most 90 times 2^-126.
FLUSH = 90 * 2.0 ** -126


def close(got, ref, mag, terms, what="", rounding=True, floor=0.0):
    """Every value within one rounding to its type plus what `terms` fp32 additions and
    products (2^-23 of the magnitudes each: the tensor cores cut, others round) leave, and
    `floor`."""
    t = got.dtype
    err = (got.double() - ref).abs()
    tol = terms * 2.0 ** -23 * mag + TINY[t] + floor
    if rounding:
        tol = tol + HALF[t] * (ref.abs() + tol)
    worst = (err - tol).max().item() if err.numel() else -1.0
    assert not (err > tol).any() and torch.isfinite(got).all(), f"{what}: beyond by {worst:.3e}"
