"""Measured cases of the 4-bit weight products, their quantiser and the expert router.

Five operations, each in a plain form (elementary torch operations in 32
bits) and as a call of the library's entry point:

  quant   bsmm_quant_w4: a weight to 4-bit codes with group scales
  mm      bsmm_w4_mm: activations times a 4-bit weight, one token to a prompt
  expert  bsmm_w4_expert_mm: routed tokens times their experts' 4-bit weights
  route   bsmm_route_topk: top-k experts, counts, slot order, balance loss
  back    bsmm_route_topk_backward: the logits' gradient of that

``own`` selects the form.  A 4-bit code is stored as 0..15 and stands for
code - zero (zero 8 where no zero points are kept), times its group's scale.
"""

import numpy as np
import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a small projection's weight quantised at load time: symmetric, fp32 scales
        dict(name="quant-1024x4096-bf16-sym-g128", op="quant", R=1024, K=4096, x="bf16", s="f32",
             group=128, sym=True),
        # a large fp32 weight with zero points, small groups and bf16 scales
        dict(name="quant-5120x8192-f32-asym-g32", op="quant", R=5120, K=8192, x="f32", s="bf16",
             group=32, sym=False),
        # one token through a large projection: the weight's bytes
        dict(name="mm-1x5120x8192-bf16-sym-g128", op="mm", M=1, N=5120, K=8192, x="bf16",
             s="bf16", o="bf16", group=128, sym=True),
        # a few sequences decoded together: fp32 activations, an odd width, small groups
        dict(name="mm-13x4099x7168-f32-asym-g32", op="mm", M=13, N=4099, K=7168, x="f32",
             s="f32", o="f32", group=32, sym=False),
        # a prompt of odd length
        dict(name="mm-2047x5120x8192-bf16-asym-g128", op="mm", M=2047, N=5120, K=8192, x="bf16",
             s="f32", o="bf16", group=128, sym=False),
        # one token through its eight of sixty-four experts, the layer's first product
        dict(name="expert-1-8of64-2048x4096-bf16", op="expert", T=1, k=8, E=64, N=2048, K=4096,
             x="bf16", s="bf16", o="bf16", group=128, sym=True, second=False),
        # a decode batch through the layer's second product: a row and a weight for every slot
        dict(name="expert-33-4of16-4096x1024-f32-second", op="expert", T=33, k=4, E=16, N=4096,
             K=1024, x="f32", s="f32", o="f32", group=64, sym=False, second=True),
        # a prompt through the experts, with uneven loads
        dict(name="expert-1021-8of32-2048x4096-bf16", op="expert", T=1021, k=8, E=32, N=2048,
             K=4096, x="bf16", s="bf16", o="bf16", group=128, sym=True, second=False),
        # one token's choice of experts in serving: no loss
        dict(name="route-1x64-top8-bf16", op="route", T=1, E=64, k=8, x="bf16", renorm=True,
             loss=False, masked=False),
        # a training batch with padding: choice, counts, order and balance loss
        dict(name="route-16384x256-top8-f32-loss", op="route", T=16384, E=256, k=8, x="f32",
             renorm=True, loss=True, masked=True),
        # an odd batch's gradient, weights taken from the softmax as they are
        dict(name="back-333x60-top6-bf16", op="back", T=333, E=60, k=6, x="bf16", renorm=False,
             loss=True, masked=True),
        # a training batch's gradient, weights that sum to one
        dict(name="back-16384x256-top8-f32", op="back", T=16384, E=256, k=8, x="f32",
             renorm=True, loss=True, masked=True),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quant", "mm", "mm", "expert", "expert", "route", "back"])
    c = dict(op=op, x=rng.choice(["bf16", "f32"]))
    if op in ("quant", "mm", "expert"):
        c["group"] = rng.choice([32, 64, 128])
        c["sym"] = rng.random() < 0.5
        c["s"] = rng.choice(["bf16", "f32"])
    if op == "quant":
        c["R"] = _log(rng, 16, 5120)
        c["K"] = c["group"] * max(1, _log(rng, 256, 8192) // c["group"])
    elif op == "mm":
        c["M"] = _log(rng, 1, 2047)
        c["N"] = _log(rng, 128, 5120)
        c["K"] = c["group"] * max(1, _log(rng, 256, 8192) // c["group"])
        c["o"] = rng.choice(["bf16", "f32"])
    elif op == "expert":
        c["T"] = _log(rng, 1, 1021)
        c["E"] = _log(rng, 4, 64)
        c["k"] = rng.randint(1, min(8, c["E"]))
        c["second"] = rng.random() < 0.5
        c["N"] = _log(rng, 128, 2048)
        c["K"] = c["group"] * max(1, _log(rng, 256, 4096) // c["group"])
        c["o"] = rng.choice(["bf16", "f32"])
    else:
        c["T"] = _log(rng, 1, 16384)
        c["E"] = _log(rng, 4, 256)
        c["k"] = rng.randint(1, min(8, c["E"]))
        c["renorm"] = rng.random() < 0.5
        c["masked"] = rng.random() < 0.5
        c["loss"] = op == "back" or rng.random() < 0.5
    return c


ALPHA = 0.01      # weight of the balance loss


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale)


def _weight(rows, K, g):
    """A weight as training leaves it: normal, rows of unequal size, a few
    outlier columns."""
    w = _normal((rows, K), g, 0.02)
    w *= torch.exp(_normal((rows, 1), g, 0.3))
    cols = torch.randint(K, (max(1, K // 256),), generator=g, device=DEV)
    w[:, cols] *= 4.0
    return w


def _activations(rows, K, g, dt):
    """Activations behind a norm: about unit size, with a few large channels."""
    x = _normal((rows, K), g)
    cols = torch.randint(K, (max(1, K // 128),), generator=g, device=DEV)
    x[:, cols] *= 8.0
    return x.to(dt)


def _logits(T, E, g, dt, masked):
    """Router outputs: some experts favoured; where masked, tokens whose
    experts are limited to the first half and a few with none at all."""
    x = _normal((T, E), g, 1.5) + _normal((1, E), g, 0.5)
    if masked:
        r = torch.rand((T,), generator=g, device=DEV)
        x[:, (E + 1) // 2:] = torch.where((r < 0.2)[:, None], -torch.inf, x[:, (E + 1) // 2:])
        x = torch.where((r > 0.99)[:, None], -torch.inf, x)
    return x.to(dt)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    st = {"case": c}
    op = c["op"]
    if op == "quant":
        st["w"] = _weight(c["R"], c["K"], g).to(DT[c["x"]])
    elif op == "mm":
        w = _weight(c["N"], c["K"], g)
        st["q"], st["scale"], st["zero"], _ = _plain_quant(w, c["group"], c["sym"], DT[c["s"]])
        st["x"] = _activations(c["M"], c["K"], g, DT[c["x"]])
    elif op == "expert":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        parts = [_plain_quant(_weight(N, K, g), c["group"], c["sym"], DT[c["s"]])
                 for _ in range(E)]
        st["q"] = torch.stack([p[0] for p in parts])
        st["scale"] = torch.stack([p[1] for p in parts])
        st["zero"] = None if c["sym"] else torch.stack([p[2] for p in parts])
        r = _plain_route(_logits(T, E, g, torch.float32, False), k, None, True, False)
        st["order"], st["offsets"] = r["order"], r["offsets"]
        st["ends"] = r["offsets"].tolist()          # the plain form loops over experts
        st["x"] = _activations(T * k if c["second"] else T, K, g, DT[c["x"]])
        st["weight"] = r["weight"].reshape(-1).contiguous() if c["second"] else None
    else:
        T, E, k = c["T"], c["E"], c["k"]
        st["logits"] = _logits(T, E, g, DT[c["x"]], c["masked"])
        st["mask"] = (torch.rand((T,), generator=g, device=DEV) < 0.9) if c["masked"] else None
        if op == "back":
            r = _plain_route(st["logits"], k, st["mask"], c["renorm"], True)
            st.update(index=r["index"], weight=r["weight"], counts=r["counts"], live=r["live"])
            st["dweight"] = _normal((T, k), g, 1.0 / T)
            st["dloss"] = torch.ones((1,), device=DEV)
    return st


# ------------------------------------------------------------- plain forms --

def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(q):
    return torch.stack([q & 15, q >> 4], dim=-1).reshape(q.shape[0], -1).to(torch.float32)


def _plain_quant(w, group, sym, scale_dtype):
    R, K = w.shape
    f = w.to(torch.float32).reshape(R, K // group, group)
    if sym:
        hi = f.abs().amax(2)
        s = hi / torch.full_like(hi, 7.0)      # by a tensor: a true division
    else:
        lo, hi = f.amin(2).clamp_max(0.0), f.amax(2).clamp_min(0.0)
        s = (hi - lo) / torch.full_like(hi, 15.0)
    s = s.to(scale_dtype)
    sf = s.to(torch.float32)
    none = sf == 0.0
    sf = torch.where(none, 1.0, sf)
    if sym:
        z = torch.full_like(sf, 8.0)
        code = torch.round(f / sf[..., None]).clamp(-8.0, 7.0) + 8.0
    else:
        z = torch.round(-lo / sf).clamp(0.0, 15.0)
        z = torch.where(none, 0.0, z)
        code = (torch.round(f / sf[..., None]) + z[..., None]).clamp(0.0, 15.0)
    code = torch.where(none[..., None], z[..., None], code)
    values = ((code - z[..., None]) * sf[..., None]).reshape(R, K).to(w.dtype)
    q = _pack(code.reshape(R, K).to(torch.uint8))
    return q, sf.to(scale_dtype), None if sym else z.to(torch.uint8), values


def _plain_weight(q, scale, zero):
    """A 4-bit weight as the 32-bit matrix it stands for."""
    G = scale.shape[1]
    v = _unpack(q).reshape(q.shape[0], G, -1)
    z = 8.0 if zero is None else zero.to(torch.float32)[..., None]
    return ((v - z) * scale.to(torch.float32)[..., None]).reshape(q.shape[0], -1)


def _plain_expert(st):
    c = st["case"]
    x = st["x"].to(torch.float32)
    order = st["order"].to(torch.int64)
    out = torch.zeros((order.numel(), c["N"]), device=DEV, dtype=torch.float32)
    for e in range(c["E"]):
        lo, hi = st["ends"][e], st["ends"][e + 1]
        if lo == hi:
            continue
        slots = order[lo:hi]
        rows = slots if c["second"] else slots // c["k"]
        w = _plain_weight(st["q"][e], st["scale"][e], None if st["zero"] is None else st["zero"][e])
        y = x[rows] @ w.t()
        if st["weight"] is not None:
            y = y * st["weight"][slots][:, None]
        out[slots] = y
    return out.to(DT[c["o"]])


def _softmax(l):
    m = l.amax(1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(l - m)
    s = p.sum(1, keepdim=True)
    return p / torch.where(s == 0.0, 1.0, s)


def _plain_route(logits, k, mask, renorm, loss):
    T, E = logits.shape
    l = logits.to(torch.float32)
    if mask is not None:
        l = torch.where(mask[:, None], l, -torch.inf)
    ids = torch.arange(E, device=DEV, dtype=torch.int32)
    p = _softmax(l)
    left = l.clone()
    index = torch.empty((T, k), device=DEV, dtype=torch.int32)
    weight = torch.empty((T, k), device=DEV, dtype=torch.float32)
    for j in range(k):
        best = left.amax(1, keepdim=True)
        first = torch.where(left == best, ids, E).amin(1, keepdim=True)
        found = best > -torch.inf
        at = first.to(torch.int64)
        index[:, j:j + 1] = torch.where(found, first, -1)
        weight[:, j:j + 1] = torch.where(found, p.gather(1, at), 0.0)
        left.scatter_(1, at, -torch.inf)
    if renorm:
        s = weight.sum(1, keepdim=True)
        weight = weight / torch.where(s == 0.0, 1.0, s)
    key = torch.where(index < 0, E, index).reshape(-1)
    by, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=DEV, dtype=torch.int32),
                                 out_int32=True)
    counts = offsets[1:] - offsets[:-1]
    r = dict(index=index, weight=weight, counts=counts, offsets=offsets,
             order=order.to(torch.int32))
    if loss:
        live = (index[:, 0] >= 0).sum().to(torch.int32).reshape(1)
        r["live"] = live
        r["prob_sum"] = p.sum(0)
        n = live.to(torch.float32).clamp_min(1.0)
        r["loss"] = (ALPHA * E / k) * ((counts.to(torch.float32) / n) * (r["prob_sum"] / n)
                                       ).sum().reshape(1)
    return r


def _plain_back(st):
    c = st["case"]
    l = st["logits"].to(torch.float32)
    if st["mask"] is not None:
        l = torch.where(st["mask"][:, None], l, -torch.inf)
    E, k = c["E"], c["k"]
    p = _softmax(l)
    n = st["live"].to(torch.float32).clamp_min(1.0)
    f = st["dloss"] * (ALPHA * E / k) * (st["counts"].to(torch.float32) / n) / n
    d = p * (f - (p * f).sum(1, keepdim=True))
    used = st["index"] >= 0
    at = st["index"].clamp_min(0).to(torch.int64)
    dw = torch.where(used, st["dweight"], 0.0)
    dot = (st["weight"] * dw).sum(1, keepdim=True)
    if c["renorm"]:
        d.scatter_add_(1, at, torch.where(used, st["weight"] * (dw - dot), 0.0))
    else:
        d -= p * dot
        d.scatter_add_(1, at, st["weight"] * dw)
    return d.to(st["logits"].dtype)


# --------------------------------------------------------------------- run --

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import block_scaled_precision_gemm_amd as bsmm
        if op == "quant":
            q, s, z, v = bsmm.bsmm_quant_w4(state["w"], group=c["group"], symmetric=c["sym"],
                                            scale_dtype=c["s"], values=True)
            return dict(q=q, scale=s, zero=z, values=v) if z is not None else \
                dict(q=q, scale=s, values=v)
        if op == "mm":
            return bsmm.bsmm_w4_mm(state["x"], state["q"], state["scale"], state["zero"],
                                   out_dtype=c["o"])
        if op == "expert":
            return bsmm.bsmm_w4_expert_mm(
                state["x"], state["q"], state["scale"], state["zero"], state["order"],
                state["offsets"], slots_per_row=1 if c["second"] else c["k"],
                row_scale=state["weight"], out_dtype=c["o"])
        if op == "route":
            r = bsmm.bsmm_route_topk(state["logits"], c["k"], mask=state["mask"],
                                     renorm=c["renorm"], alpha=ALPHA if c["loss"] else None)
            return {n: getattr(r, n) for n in _route_names(c)}
        return bsmm.bsmm_route_topk_backward(
            state["logits"], state["index"], state["weight"], state["counts"], state["live"],
            dweight=state["dweight"], dloss=state["dloss"], alpha=ALPHA, mask=state["mask"],
            renorm=c["renorm"])
    if op == "quant":
        q, s, z, v = _plain_quant(state["w"], c["group"], c["sym"], DT[c["s"]])
        return dict(q=q, scale=s, zero=z, values=v) if z is not None else \
            dict(q=q, scale=s, values=v)
    if op == "mm":
        w = _plain_weight(state["q"], state["scale"], state["zero"])
        return (state["x"].to(torch.float32) @ w.t()).to(DT[c["o"]])
    if op == "expert":
        return _plain_expert(state)
    if op == "route":
        r = _plain_route(state["logits"], c["k"], state["mask"], c["renorm"], c["loss"])
        return {n: r[n] for n in _route_names(c)}
    return _plain_back(state)


def _route_names(c):
    names = ["index", "weight", "counts", "offsets", "order"]
    return names + ["live", "prob_sum", "loss"] if c["loss"] else names


# -------------------------------------------------------------------- work --

def _weight_bytes(rows, c):
    return rows * (c["K"] // 2 + c["K"] // c["group"] * (SIZE[c["s"]] + (0 if c["sym"] else 1)))


def work(case):
    c = case
    op = c["op"]
    if op == "quant":
        n = c["R"] * c["K"]
        return {"bytes": 2 * n * SIZE[c["x"]] + _weight_bytes(c["R"], c), "flops": 4 * n}
    if op == "mm":
        return {"bytes": c["M"] * c["K"] * SIZE[c["x"]] + _weight_bytes(c["N"], c)
                + c["M"] * c["N"] * SIZE[c["o"]],
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    if op == "expert":
        slots = c["T"] * c["k"]
        # experts that some slot is expected to reach, were the choice even
        touched = min(c["E"], max(c["k"], round(c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"]))))
        rows = slots if c["second"] else c["T"]
        return {"bytes": rows * c["K"] * SIZE[c["x"]] + touched * _weight_bytes(c["N"], c)
                + slots * c["N"] * SIZE[c["o"]] + slots * (8 if c["second"] else 4),
                "flops": 2 * slots * c["N"] * c["K"]}
    n = c["T"] * c["E"]
    if op == "route":
        return {"bytes": n * SIZE[c["x"]] + c["T"] * c["k"] * 12 + c["T"] * c["masked"]
                + c["E"] * 12, "flops": 6 * n}
    return {"bytes": 2 * n * SIZE[c["x"]] + c["T"] * c["k"] * 12 + c["T"] * c["masked"]
            + c["E"] * 4, "flops": 10 * n}


# ------------------------------------------------------------------- exact --

def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _codes64(q):
    """uint8 [N, K/2] -> the codes as 64-bit floats [N, K] (low nibble first)."""
    out = torch.empty((q.shape[0], 2 * q.shape[1]), device=q.device, dtype=torch.float64)
    out[:, 0::2] = q.remainder(16)
    out[:, 1::2] = torch.div(q, 16, rounding_mode="floor")
    return out


def _product64(x, q, scale, zero, group):
    """sum over groups of scale * (x_g . (code_g - zero)), in 64 bits."""
    x = x.to(torch.float64)
    code = _codes64(q)
    y = torch.zeros((x.shape[0], q.shape[0]), device=x.device, dtype=torch.float64)
    for i in range(scale.shape[1]):
        cut = slice(i * group, (i + 1) * group)
        z = 8.0 if zero is None else zero[:, i:i + 1].to(torch.float64)
        y += (x[:, cut] @ (code[:, cut] - z).t().contiguous()) * scale[:, i].to(torch.float64)
    return y


def _bf16_64(a):
    """64-bit values to the nearest bf16 (even on ties), subnormals included."""
    m, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.where(a == 0.0, 0.0, np.rint(a / step) * step)


def _exact_quant(c, st):
    w = _np(st["w"]).reshape(c["R"], -1, c["group"])
    # a quotient of two binary32 values rounded to 64 bits and then to 32 is
    # the binary32 quotient of the definition
    if c["sym"]:
        s = (np.abs(w).max(2) / 7.0).astype(np.float32)
    else:
        lo, hi = np.minimum(w.min(2), 0.0), np.maximum(w.max(2), 0.0)
        s = ((hi - lo).astype(np.float32).astype(np.float64) / 15.0).astype(np.float32)
    s = s.astype(np.float64)
    if c["s"] == "bf16":
        s = _bf16_64(s)
    empty = s == 0.0
    s = np.where(empty, 1.0, s)
    n = np.rint((w / s[..., None]).astype(np.float32)).astype(np.int64)
    if c["sym"]:
        z = np.full(s.shape, 8, np.int64)
        code = np.clip(n, -8, 7) + 8
    else:
        z = np.clip(np.rint((-lo / s).astype(np.float32)), 0, 15).astype(np.int64)
        z = np.where(empty, 0, z)
        code = np.clip(n + z[..., None], 0, 15)
    code = np.where(empty[..., None], z[..., None], code)
    v = ((code - z[..., None]) * s[..., None]).reshape(c["R"], -1)
    code = code.reshape(c["R"], -1).astype(np.uint8)
    out = dict(q=code[:, 0::2] + 16 * code[:, 1::2], scale=s, values=v)
    if not c["sym"]:
        out["zero"] = z.astype(np.uint8)
    return out


def _route64(logits, mask, k, renorm):
    """Probabilities, indices and weights in 64 bits, from a sorted order."""
    l = _np(logits)
    if mask is not None:
        l = np.where(mask.cpu().numpy()[:, None], l, -np.inf)
    at = np.argsort(-l, axis=1, kind="stable")[:, :k]
    val = np.take_along_axis(l, at, 1)
    none = val == -np.inf
    top = np.where(none[:, :1], 0.0, val[:, :1])
    ex = np.exp(l - top)
    p = ex / np.where(none[:, :1], 1.0, ex.sum(1, keepdims=True))
    w = np.where(none, 0.0, np.take_along_axis(p, at, 1))
    if renorm:
        w = w / np.where(none[:, :1], 1.0, w.sum(1, keepdims=True))
    return p, np.where(none, -1, at), w


def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    op = c["op"]
    if op == "quant":
        return _exact_quant(c, st)
    if op == "mm":
        return _product64(st["x"], st["q"], st["scale"], st["zero"], c["group"]).cpu().numpy()
    if op == "expert":
        order = st["order"].cpu().numpy()
        out = np.zeros((order.size, c["N"]))
        for e in range(c["E"]):
            slots = order[st["ends"][e]:st["ends"][e + 1]]
            if slots.size == 0:
                continue
            rows = torch.from_numpy(slots // (1 if c["second"] else c["k"])).to(DEV).long()
            y = _product64(st["x"][rows], st["q"][e], st["scale"][e],
                           None if st["zero"] is None else st["zero"][e], c["group"])
            y = y.cpu().numpy()
            out[slots] = y * _np(st["weight"])[slots, None] if c["second"] else y
        return out
    p, index, w = _route64(st["logits"], st["mask"], c["k"], c["renorm"])
    T, E, k = c["T"], c["E"], c["k"]
    counts = np.bincount(index[index >= 0], minlength=E)
    live = int((index[:, 0] >= 0).sum())
    f = counts * (ALPHA * E / (k * max(live, 1) ** 2))
    if op == "route":
        key = np.where(index < 0, E, index).reshape(-1)
        out = dict(index=index.astype(np.int32), weight=w, counts=counts.astype(np.int32),
                   offsets=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
                   order=np.argsort(key, kind="stable").astype(np.int32))
        if c["loss"]:
            out.update(live=np.array([live], np.int32), prob_sum=p.sum(0),
                       loss=np.array([(f * p.sum(0)).sum()]))
        return {n: out[n] for n in _route_names(c)}
    # the loss and weights are functions of the softmax alone: collect the
    # derivative by each probability, then go through the softmax once
    dw = _np(st["dweight"])
    hit = index >= 0
    rows, cols = np.nonzero(hit)
    picked = index[rows, cols]
    gp = np.broadcast_to(f * float(st["dloss"].item()), (T, E)).copy()
    if c["renorm"]:
        tot = np.take_along_axis(p, np.maximum(index, 0), 1)
        tot = np.where(hit, tot, 0.0).sum(1)
        mean = np.where(hit, w * dw, 0.0).sum(1)
        gp[rows, picked] += (dw[rows, cols] - mean[rows]) / tot[rows]
    else:
        gp[rows, picked] += dw[rows, cols]
    return p * (gp - (p * gp).sum(1, keepdims=True))
