"""Measured calls of the operators that train the routed experts.

Three groups of calls, each in a plain form (elementary torch operations in 32
bits) and through the package:

  product   products grouped by expert over ragged segments of rows: rows
            offsets[e] .. offsets[e + 1] - 1 belong to expert e
              forward  y[r]  = W[e] x[r]
              dx       dx[r] = W[e]^T dy[r]
              dw       dW[e] = sum over the expert's rows of dy[r] x[r]^T
  pack      the SwiGLU between the experts' products, keeping what its
            backward pass needs in 8 bits: blocks of 32 columns of the
            pre-activations as 8-bit integers under one power of two
  unpack    its backward pass from those 8 bits: the gradient of the
            pre-activations, the activations again (weighted, for the
            gradient of the next weight) and the gradient of the row's weight
  rows      tokens to their experts' segments and the weighted sum back

A block of 32 values is stored as integers q in [-127, 127] and a byte s:
the values are q 2^(s - 127), with s - 127 = floor(log2 max|x|) - 6 (at least
-127), q to nearest, ties to even.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # A small step: 64 tokens of 8 slots over 128 experts, a few rows each;
        # the weights' bytes are the work (gate_up: 2 x 768 outputs).
        dict(name="forward_few_rows", op="product", way="forward", R=512, E=128, N=1536, K=2048,
             dtype="bf16", empty=0.0),
        # A training micro-batch of 4096 tokens through gate_up.
        dict(name="forward_train", op="product", way="forward", R=32768, E=128, N=1536, K=2048,
             dtype="bf16", empty=0.0),
        # Ragged in every size, experts without rows, fp16.
        dict(name="forward_odd", op="product", way="forward", R=5003, E=60, N=1000, K=1016,
             dtype="fp16", empty=0.2),
        # The gradient of the down product's input for that micro-batch.
        dict(name="dx_train", op="product", way="dx", R=32768, E=128, N=2048, K=768,
             dtype="bf16", empty=0.0),
        # The gradient of gate_up's weights: every expert's matrix is written.
        dict(name="dw_train", op="product", way="dw", R=32768, E=128, N=1536, K=2048,
             dtype="bf16", out="bf16", empty=0.0),
        # Few experts with long segments, small matrices, gradient in fp32.
        dict(name="dw_long", op="product", way="dw", R=20011, E=8, N=640, K=328,
             dtype="bf16", out="fp32", empty=0.0),
        # The SwiGLU of one small step: latency.
        dict(name="pack_small", op="pack", R=512, I=768, dtype="bf16"),
        # The micro-batch: the layer's largest activation goes to 8 bits.
        dict(name="pack_train", op="pack", R=32768, I=768, dtype="bf16"),
        # Its backward pass for odd sizes, without row weights, fp16.
        dict(name="unpack_odd", op="unpack", R=5003, I=352, dtype="fp16", weighted=False),
        # The micro-batch backwards, with the routing weights.
        dict(name="unpack_train", op="unpack", R=32768, I=768, dtype="bf16", weighted=True),
        # 64 tokens to their experts and back.
        dict(name="rows_small", op="rows", T=64, H=2048, E=128, k=8, dtype="bf16", masked=0.0),
        # The micro-batch with padded sequences, whose tokens have no rows.
        dict(name="rows_train", op="rows", T=4096, H=2048, E=128, k=8, dtype="bf16", masked=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "pack", "unpack", "rows"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "product":
        way = rng.choice(["forward", "dx", "dw"])
        E = rng.choice([1, 4, 8, 40, 60, 64, 128])
        N, K = 8 * _log(rng, 8, 256), 8 * _log(rng, 8, 256)
        while E * N * K > 128 * 1536 * 2048:
            E //= 2
        R = min(_log(rng, 1, 32768), 32768 * 1536 * 2048 // (N * K))
        c = dict(op=op, way=way, R=R, E=E, N=N, K=K, dtype=dtype,
                 empty=rng.choice([0.0, 0.0, 0.25]))
        if way == "dw":
            c["out"] = rng.choice([dtype, "fp32"])
        return c
    if op == "rows":
        T, E = _log(rng, 1, 4096), rng.choice([4, 8, 40, 60, 64, 128, 256])
        k = rng.randint(1, min(E, 10))
        H = min(8 * _log(rng, 8, 512), 4096 * 8 * 2048 // (T * k) // 8 * 8)
        return dict(op=op, T=T, H=H, E=E, k=k, dtype=dtype,
                    masked=rng.choice([0.0, 0.0, 0.1, 0.4]))
    R = _log(rng, 1, 32768)
    I = min(32 * _log(rng, 1, 64), max(32, 32768 * 768 // R // 32 * 32))
    c = dict(op=op, R=R, I=I, dtype=dtype)
    if op == "unpack":
        c["weighted"] = rng.random() < 0.6
    return c


def work(case):
    op = case["op"]
    if op == "product":
        R, E, N, K = (case[n] for n in ("R", "E", "N", "K"))
        used = E * (1 - (1 - 1 / E) ** R)  # experts that some row belongs to (expected)
        n = 2 * R * (N + K) + 4 * (E + 1)
        n += E * N * K * (4 if case["out"] == "fp32" else 2) if case["way"] == "dw" \
            else 2 * used * N * K
        return {"bytes": n, "flops": 2 * R * N * K}
    if op == "rows":
        T, H, k = case["T"], case["H"], case["k"]
        S = T * k * (1 - case["masked"])
        # tokens in, their rows out; rows in, tokens out; ids, weights, places, masks
        return {"bytes": 2 * H * (T + S + S + T) + 16 * T * k + T * (case["masked"] > 0),
                "flops": 2 * S * H}
    n = case["R"] * case["I"]
    # z in, activations out, 8-bit values and their scales out; or those and the
    # gradient in, the gradient of z and the activations out.
    if op == "pack":
        # (and the stored values read back: 2 bytes each)
        return {"bytes": n * (4 + 2) + 2 * n * 33 / 32 * 2 + 4 * n, "flops": 12 * n}
    return {"bytes": 2 * n * 33 / 32 + n * 2 + n * 4 + n * 2 + 8 * case["R"] * case["weighted"],
            "flops": 24 * n}


# ----------------------------------------------------------------- inputs ---

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _segments(g, R, E, empty):
    """Offsets [E + 1] of R rows over E experts of uneven load, some without rows."""
    p = torch.exp(0.5 * _normal(g, E))
    p = torch.where(torch.rand(E, generator=g, device="cuda") < empty, torch.zeros_like(p), p)
    p[0] += 1e-3
    e = torch.multinomial(p, R, replacement=True, generator=g)
    counts = torch.bincount(e, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, int(counts.max())


def _encode(z):
    """8-bit integers (int8) and block exponents (uint8) of z [R, C] float32."""
    b = z.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax == 0, torch.full_like(amax, -127),
                    (torch.frexp(amax)[1] - 7).clamp(-127, 127).float()).to(torch.int32)
    q = torch.ldexp(b, -e.unsqueeze(-1)).round().clamp(-127, 127)
    return q.flatten(-2).to(torch.int8), (e + 127).to(torch.uint8)


def _pre_activations(g, R, I):
    """Gate and up values as the gate_up product gives them: rows and columns
    of different sizes."""
    z = _normal(g, R, 2 * I)
    z *= torch.exp(0.4 * _normal(g, R, 1))
    z *= torch.exp(0.4 * _normal(g, 1, 2 * I))
    return z


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], _DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "product":
        R, E, N, K = (case[n] for n in ("R", "E", "N", "K"))
        s["offsets"], s["most"] = _segments(g, R, E, case["empty"])
        if case["way"] != "forward":
            s["dy"] = _normal(g, R, N).to(dt)
        if case["way"] != "dx":
            s["x"] = _normal(g, R, K).to(dt)
        if case["way"] != "dw":
            s["w"] = torch.empty(E, N, K, dtype=dt, device="cuda")
            for e in range(0, E, 16):
                s["w"][e:e + 16] = 0.02 * _normal(g, min(16, E - e), N, K)
    elif op == "pack":
        s["z"] = _pre_activations(g, case["R"], case["I"]).to(dt)
    elif op == "unpack":
        R, I = case["R"], case["I"]
        s["codes"], s["scales"] = _encode(_pre_activations(g, R, I).to(dt).float())
        s["da"] = _normal(g, R, I).to(dt)
        s["row_w"] = torch.rand(R, generator=g, device="cuda") if case["weighted"] else None
    else:
        T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
        logits = _normal(g, T, E) + 0.5 * _normal(g, 1, E)
        w, ids = torch.sort(torch.softmax(logits, -1), dim=-1, descending=True, stable=True)
        ids, order = torch.sort(ids[:, :k], -1)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["w"] = w[:, :k].gather(1, order).contiguous()
        s["x"] = _normal(g, T, H).to(dt)
        s["y"] = _normal(g, T * k, H).to(dt)  # the experts' outputs, one row a slot
        s["mask"] = None
        if case["masked"] > 0:
            s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"]
        # What a program keeps from step to step: the rows' buffers. Rows behind
        # the last segment stay as they are.
        s["rows"] = torch.zeros(T * k, H, dtype=dt, device="cuda")
        s["row_w"] = torch.zeros(T * k, device="cuda")
    return s


# ------------------------------------------------------------- plain form ---

def _plain_product(s):
    c = s["case"]
    R, E, N, K, most = c["R"], c["E"], c["N"], c["K"], s["most"]
    off = s["offsets"].long()
    r = torch.arange(R, device=off.device)
    e = torch.bucketize(r, off[1:], right=True)
    at = e * most + r - off[e]  # the row's place in [E, most]

    def padded(x):
        p = torch.zeros(E * most, x.shape[1], device=x.device)
        p[at] = x.float()
        return p.view(E, most, -1)

    if c["way"] == "forward":
        y = torch.bmm(padded(s["x"]), s["w"].float().transpose(1, 2))
    elif c["way"] == "dx":
        y = torch.bmm(padded(s["dy"]), s["w"].float())
    else:
        return torch.bmm(padded(s["dy"]).transpose(1, 2), padded(s["x"])).to(_DTYPES[c["out"]])
    return y.view(E * most, -1)[at].to(_DTYPES[c["dtype"]])


def _decode(q, s):
    v = q.float().unflatten(-1, (-1, 32))
    return torch.ldexp(v, (s.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _plain_pack(s):
    I, dt = s["case"]["I"], _DTYPES[s["case"]["dtype"]]
    z = s["z"].float()
    gate, up = z[:, :I], z[:, I:]
    act = gate / (1 + torch.exp(-gate)) * up
    return {"act": act.to(dt), "stored": _decode(*_encode(z)).to(torch.bfloat16)}


def _plain_unpack(s):
    I, dt = s["case"]["I"], _DTYPES[s["case"]["dtype"]]
    z = _decode(s["codes"], s["scales"])
    gate, up, da = z[:, :I], z[:, I:], s["da"].float()
    sig = 1 / (1 + torch.exp(-gate))
    act = gate * sig * up
    w = 1.0 if s["row_w"] is None else s["row_w"][:, None]
    dz = torch.cat((w * da * up * sig * (1 + gate * (1 - sig)), w * da * gate * sig), 1)
    out = {"dz": dz.to(dt), "act": (w * act).to(dt)}
    if s["row_w"] is not None:
        out["d_row_w"] = (da * act).sum(1)
    return out


def _plain_rows(s):
    c = s["case"]
    T, H, E, k, dt = c["T"], c["H"], c["E"], c["k"], _DTYPES[c["dtype"]]
    valid = torch.ones(T, 1, dtype=torch.bool, device=s["x"].device) if s["mask"] is None \
        else s["mask"][:, None]
    e = torch.where(valid, s["ids"].long(), torch.full_like(s["ids"].long(), E)).flatten()
    order = torch.sort(e, stable=True)[1]
    place = torch.empty_like(e)
    place[order] = torch.arange(T * k, device=e.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device).scatter_add_(
        0, e, torch.ones_like(e))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=e.device)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    used = (torch.arange(T * k, device=e.device) < offsets[E])[:, None]
    rows = torch.where(used, s["x"][order // k], s["rows"])
    row_w = torch.where(used[:, 0], s["w"].flatten()[order], s["row_w"])
    y = s["y"][place].view(T, k, H).float()
    out = (torch.where(valid[..., None], s["w"][..., None] * y, torch.zeros_like(y))).sum(1)
    place = torch.where(valid, place.view(T, k), torch.full_like(place.view(T, k), -1))
    return {"places": place.to(torch.int32), "offsets": offsets, "rows": rows, "row_w": row_w,
            "out": out.to(dt)}


# ------------------------------------------------------------------- run ---

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"product": _plain_product, "pack": _plain_pack, "unpack": _plain_unpack,
                "rows": _plain_rows}[op](s)
    import mixture_experts_layer_mm_gb300 as mm
    if op == "product":
        if c["way"] == "forward":
            return mm.mm_grouped_product(s["x"], s["w"], s["offsets"])
        if c["way"] == "dx":
            return mm.mm_grouped_product_dx(s["dy"], s["w"], s["offsets"])
        return mm.mm_grouped_product_dw(s["dy"], s["x"], s["offsets"],
                                        out_dtype=_DTYPES[c["out"]])
    if op == "pack":
        act, codes, scales = mm.mm_swiglu_pack(s["z"])
        return {"act": act, "stored": mm.mm_mxint8_dequantize(codes, scales)}
    if op == "unpack":
        dz, act, d_row_w = mm.mm_swiglu_pack_backward(s["codes"], s["scales"], s["da"],
                                                      row_w=s["row_w"])
        out = {"dz": dz, "act": act}
        if s["row_w"] is not None:
            out["d_row_w"] = d_row_w
        return out
    places, offsets = mm.mm_group_slots(s["ids"], c["E"], token_mask=s["mask"])
    rows, row_w = mm.mm_dispatch_rows(s["x"], places, w=s["w"], rows=s["rows"],
                                      row_w=s["row_w"])
    out = mm.mm_combine_rows(s["y"], places, w=s["w"])
    return {"places": places, "offsets": offsets, "rows": rows, "row_w": row_w, "out": out}


# ----------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        R, E, N, K = (case[n] for n in ("R", "E", "N", "K"))
        off = s["offsets"].tolist()
        way = case["way"]
        shape = {"forward": (R, N), "dx": (R, K), "dw": (E, N, K)}[way]
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            if way == "forward":
                out[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
            elif way == "dx":
                out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
            else:
                out[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
        return out
    if op == "pack":
        z, I = s["z"].double(), case["I"]
        b = z.reshape(-1, 32)
        amax = b.abs().amax(1, keepdim=True)
        unit = torch.exp2(torch.floor(torch.log2(amax.clamp_min(2.0 ** -121))) - 6)
        unit = torch.where(64 * unit > amax, unit / 2, unit)  # log2 rounded up
        unit = torch.where(128 * unit <= amax, unit * 2, unit).clamp_min(2.0 ** -127)
        stored = torch.round(b / unit).clamp(-127, 127) * unit
        return {"act": torch.nn.functional.silu(z[:, :I]) * z[:, I:],
                "stored": stored.reshape(z.shape)}
    if op == "unpack":
        I = case["I"]
        z = s["codes"].double() * torch.exp2(s["scales"].double() - 127).repeat_interleave(32, 1)
        z.requires_grad_(True)
        w = torch.ones(case["R"], dtype=torch.float64, device="cuda") if s["row_w"] is None \
            else s["row_w"].double()
        w.requires_grad_(True)
        act = w[:, None] * (z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:])
        dz, dw = torch.autograd.grad(act, (z, w), s["da"].double())
        out = {"dz": dz, "act": act.detach()}
        if s["row_w"] is not None:
            out["d_row_w"] = dw
        return out
    T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
    ids, w = s["ids"].cpu(), s["w"].double()
    keep = torch.ones(T, dtype=torch.bool) if s["mask"] is None else s["mask"].cpu()
    flat = torch.where(keep[:, None], ids.long(), torch.tensor(E)).flatten()
    places = torch.full((T * k,), -1, dtype=torch.int64)
    offsets = [0]
    for e in range(E):  # the expert's slots in their order
        f = torch.nonzero(flat == e).flatten()
        places[f] = offsets[-1] + torch.arange(f.numel())
        offsets.append(offsets[-1] + f.numel())
    slots = torch.nonzero(places >= 0).flatten()
    to = places[slots].cuda()
    rows, row_w = s["rows"].double(), s["row_w"].double()
    rows[to] = s["x"][(slots // k).cuda()].double()
    row_w[to] = w.flatten()[slots.cuda()]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    out.index_add_(0, (slots // k).cuda(), w.flatten()[slots.cuda()][:, None]
                   * s["y"][to].double())
    return {"places": places.view(T, k).to(torch.int32),
            "offsets": torch.tensor(offsets, dtype=torch.int32), "rows": rows, "row_w": row_w,
            "out": out}
