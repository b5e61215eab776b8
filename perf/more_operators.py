"""Measured cases of the experts' products in 16 and 32 bits, their weight
gradient, and 8-bit activation checkpoints with the gate that uses them.

Five operations, each in a plain form (elementary torch operations in 32
bits) and as a call of the library's entry point:

  mm      bsmm_expert_mm: routed rows times their experts' weights, forward
          or (back) times the transposed weights, the input's gradient
  wgrad   bsmm_expert_wgrad: the experts' weight gradients, from the layer's
          input or from its 8-bit checkpoint
  quant   bsmm_quant_int8_mx: activations to an 8-bit checkpoint
  gate    bsmm_swiglu: silu(first half) * second half, in training with the
          8-bit checkpoint of its input
  back    bsmm_swiglu_backward: its gradient from that checkpoint

``own`` selects the form.  A checkpoint holds int8 codes and one power of two
(its exponent + 127 as a byte) per 32 elements of a row: code * 2^(byte - 133).
"""

import numpy as np
import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "ckpt": 1 + 1 / 32}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one token through its eight of sixty-four experts: the weights' bytes
        dict(name="mm-1-8of64-2048x4096-bf16", op="mm", T=1, k=8, E=64, N=2048, K=4096, x="bf16",
             o="bf16", second=False, back=False, masked=False),
        # a decode batch through the layer's second product, in fp32: a row and a weight for
        # every slot, an odd width
        dict(name="mm-33-4of16-4099x1024-f32-second", op="mm", T=33, k=4, E=16, N=4099, K=1024,
             x="f32", o="f32", second=True, back=False, masked=False),
        # a prompt through the experts, with uneven loads
        dict(name="mm-1021-8of32-2048x4096-bf16", op="mm", T=1021, k=8, E=32, N=2048, K=4096,
             x="bf16", o="bf16", second=False, back=False, masked=False),
        # a training batch with padding: the gradient of the layer's input, a row per slot
        dict(name="mm-4096-8of64-2048x4096-bf16-back", op="mm", T=4096, k=8, E=64, N=2048, K=4096,
             x="bf16", o="bf16", second=True, back=True, masked=True),
        # a small batch's weight gradient in fp32, odd sizes
        dict(name="wgrad-333-2of6-1001x515-f32", op="wgrad", T=333, k=2, E=6, N=1001, K=515,
             y="f32", x="f32", o="f32", second=False, masked=True),
        # a training batch's weight gradient from the 8-bit checkpoint of the layer's input
        dict(name="wgrad-4096-8of32-2048x4096-ckpt", op="wgrad", T=4096, k=8, E=32, N=2048, K=4096,
             y="bf16", x="ckpt", o="f32", second=False, masked=True),
        # a decode-sized batch's activations, fp32
        dict(name="quant-33x4096-f32", op="quant", R=33, K=4096, x="f32"),
        # a training batch's activations
        dict(name="quant-16384x5120-bf16", op="quant", R=16384, K=5120, x="bf16"),
        # one token's eight slots in serving: no checkpoint
        dict(name="gate-8x2048-bf16", op="gate", S=8, F=2048, x="bf16", ckpt=False),
        # a training batch's slots with their checkpoint
        dict(name="gate-32768x2048-bf16-ckpt", op="gate", S=32768, F=2048, x="bf16", ckpt=True),
        # a small fp32 batch's gradient, no routing weights
        dict(name="back-1001x1024-f32", op="back", S=1001, F=1024, x="f32", weighted=False),
        # a training batch's gradient with the routing weights'
        dict(name="back-32768x2048-bf16", op="back", S=32768, F=2048, x="bf16", weighted=True),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return int(round(lo * (hi / lo) ** rng.random()))


def _size(rng, lo, hi):
    """A feature count: two in three are multiples of 32, the others any."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 1 / 3 else max(32, n // 32 * 32)


def draw(rng):
    op = rng.choice(["mm", "mm", "mm", "wgrad", "wgrad", "quant", "gate", "back"])
    c = dict(op=op)
    if op in ("mm", "wgrad"):
        c["T"] = _log(rng, 1, 4096)
        c["E"] = _log(rng, 2, 64 if op == "mm" else 32)
        c["k"] = rng.randint(1, min(8, c["E"]))
        c["N"] = _size(rng, 64, 2048)
        c["K"] = _size(rng, 64, 4096)
        c["second"] = rng.random() < 0.5
        c["masked"] = rng.random() < 0.5
        c["o"] = rng.choice(["bf16", "f32"])
    if op == "mm":
        c["x"] = rng.choice(["bf16", "bf16", "f32"])
        c["back"] = rng.random() < 0.5
        if c["x"] == "f32":             # six times the matrix work of bf16
            c["T"] = min(c["T"], 1 + c["T"] % 1024)
    elif op == "wgrad":
        c["y"] = rng.choice(["bf16", "bf16", "f32"])
        c["x"] = rng.choice([c["y"], "ckpt"])
        if c["x"] == "ckpt":
            c["K"] = max(64, c["K"] // 32 * 32)
        if c["y"] == "f32":
            c["T"] = min(c["T"], 1 + c["T"] % 1024)
    elif op == "quant":
        c["R"] = _log(rng, 1, 16384)
        c["K"] = 32 * _log(rng, 2, 160)
        c["x"] = rng.choice(["bf16", "f32"])
    else:
        c["S"] = _log(rng, 1, 32768)
        c["F"] = 32 * _log(rng, 2, 64)
        c["x"] = rng.choice(["bf16", "f32"])
        if c["x"] == "f32":
            c["S"] = (c["S"] + 1) // 2
        if op == "gate":
            c["ckpt"] = rng.random() < 0.5
        else:
            c["weighted"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale)


def _weights(E, N, K, g, dt):
    """Weights as training leaves them: normal, rows of unequal size."""
    w = torch.empty((E, N, K), device=DEV, dtype=dt)
    for e in range(E):
        w[e] = _normal((N, K), g, K ** -0.5) * torch.exp(_normal((N, 1), g, 0.3))
    return w


def _activations(rows, K, g, dt):
    """Activations behind a norm: about unit size, with a few large channels."""
    x = _normal((rows, K), g)
    cols = torch.randint(K, (max(1, K // 128),), generator=g, device=DEV)
    x[:, cols] *= 8.0
    return x.to(dt)


def _gradients(rows, N, g, dt):
    """Gradients of a mean loss: small, rows of very unequal size."""
    return (_normal((rows, N), g, 1e-3) * torch.exp(_normal((rows, 1), g, 1.0))).to(dt)


def _routes(T, E, k, g, masked):
    """Slots sorted by expert and each expert's start: k experts a token,
    some favoured; where masked, a tenth of the tokens have none."""
    logits = _normal((T, E), g, 1.5) + _normal((1, E), g, 0.5)
    expert = torch.topk(logits, k, dim=1).indices
    if masked:
        gone = torch.rand((T, 1), generator=g, device=DEV) < 0.1
        expert = torch.where(gone, E, expert)
    by, order = torch.sort(expert.reshape(-1), stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=DEV))
    return order.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    st = {"case": c}
    op = c["op"]
    if op in ("mm", "wgrad"):
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        st["order"], st["offsets"] = _routes(T, E, k, g, c["masked"])
        st["ends"] = st["offsets"].tolist()         # the plain form loops over experts
        rows = T * k if c["second"] else T
        if op == "mm":
            st["w"] = _weights(E, N, K, g, DT[c["x"]])
            if c["back"]:
                st["x"] = _gradients(rows, N, g, DT[c["x"]])
            else:
                st["x"] = _activations(rows, K, g, DT[c["x"]])
            # the routing weights belong to the forward pass's second product
            st["weight"] = None
            if c["second"] and not c["back"]:
                st["weight"] = torch.rand((T * k,), generator=g, device=DEV)
        else:
            # the first product's gradient has a row per slot and the token's input, the
            # second's the token's gradient and a row of the gate's output per slot
            st["dy"] = _gradients(T if c["second"] else T * k, N, g, DT[c["y"]])
            st["x"] = _activations(rows, K, g, DT[c["y"]])
            st["x_scale"] = None
            if c["x"] == "ckpt":
                st["x"], st["x_scale"], _ = _plain_quant(st["x"])
    elif op == "quant":
        st["x"] = _activations(c["R"], c["K"], g, DT[c["x"]])
    elif op == "gate":
        st["h"] = _activations(c["S"], 2 * c["F"], g, DT[c["x"]])
    else:
        st["q"], st["scale"], _ = _plain_quant(_activations(c["S"], 2 * c["F"], g, DT[c["x"]]))
        st["da"] = _gradients(c["S"], c["F"], g, DT[c["x"]])
        st["weight"] = torch.rand((c["S"],), generator=g, device=DEV) if c["weighted"] else None
    return st


# ------------------------------------------------------------- plain forms --

def _plain_quant(x):
    R, K = x.shape
    f = x.to(torch.float32).reshape(R, K // 32, 32)
    amax = f.abs().amax(2)
    power = torch.frexp(amax).exponent - 1              # amax = m 2^power, m in [1, 2)
    power = torch.where(amax == 0.0, 0, power).clamp_min(-127)
    q = torch.round(torch.ldexp(f, (6 - power)[..., None])).clamp(-127.0, 127.0)
    values = torch.ldexp(q, (power - 6)[..., None])
    return (q.reshape(R, K).to(torch.int8), (power + 127).to(torch.uint8),
            values.reshape(R, K).to(x.dtype))


def _plain_restore(q, scale):
    """A checkpoint as the 32-bit values it stands for."""
    R, K = q.shape
    f = q.to(torch.float32).reshape(R, K // 32, 32)
    return torch.ldexp(f, (scale.to(torch.int32) - 133)[..., None]).reshape(R, K)


def _runs(st):
    """(expert, its slots) of every expert that has some."""
    order = st["order"].to(torch.int64)
    for e, (lo, hi) in enumerate(zip(st["ends"], st["ends"][1:])):
        if hi > lo:
            yield e, order[lo:hi]


def _plain_mm(st):
    c = st["case"]
    x = st["x"].to(torch.float32)
    out = torch.zeros((c["T"] * c["k"], c["K"] if c["back"] else c["N"]), device=DEV,
                      dtype=torch.float32)
    for e, slots in _runs(st):
        rows = slots if c["second"] else slots // c["k"]
        w = st["w"][e].to(torch.float32)
        y = x[rows] @ (w if c["back"] else w.t())
        if st["weight"] is not None:
            y = y * st["weight"][slots][:, None]
        out[slots] = y
    return out.to(DT[c["o"]])


def _plain_wgrad(st):
    c = st["case"]
    dy = st["dy"].to(torch.float32)
    x = st["x"].to(torch.float32) if st["x_scale"] is None else \
        _plain_restore(st["x"], st["x_scale"])
    dw = torch.zeros((c["E"], c["N"], c["K"]), device=DEV, dtype=torch.float32)
    for e, slots in _runs(st):
        token = slots // c["k"]
        a, b = (token, slots) if c["second"] else (slots, token)
        torch.mm(dy[a].t(), x[b], out=dw[e])
    return dw.to(DT[c["o"]])


def _plain_gate(h):
    f = h.to(torch.float32)
    g, u = f.chunk(2, 1)
    return (g / (1.0 + torch.exp(-g)) * u).to(h.dtype)


def _plain_back(st):
    dt = st["da"].dtype
    g, u = _plain_restore(st["q"], st["scale"]).chunk(2, 1)
    da = st["da"].to(torch.float32)
    s = 1.0 / (1.0 + torch.exp(-g))
    a = g * s * u
    out = {}
    if st["weight"] is not None:
        out["drow"] = (da * a).sum(1)
        da = da * st["weight"][:, None]
        a = a * st["weight"][:, None]
    out["dh"] = torch.cat([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], 1).to(dt)
    out["act"] = a.to(dt)
    return out


# --------------------------------------------------------------------- run --

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import block_scaled_precision_gemm_amd as bsmm
        if op == "mm":
            w = state["w"].transpose(1, 2) if c["back"] else state["w"]
            return bsmm.bsmm_expert_mm(state["x"], w, state["order"], state["offsets"],
                                       slots_per_row=1 if c["second"] else c["k"],
                                       row_scale=state["weight"], out_dtype=c["o"])
        if op == "wgrad":
            return bsmm.bsmm_expert_wgrad(
                state["dy"], state["x"], state["order"], state["offsets"],
                x_scale=state["x_scale"], dy_slots_per_row=c["k"] if c["second"] else 1,
                x_slots_per_row=1 if c["second"] else c["k"], out_dtype=c["o"])
        if op == "quant":
            q, s, v = bsmm.bsmm_quant_int8_mx(state["x"], values=True)
            return dict(q=q, scale=s, values=v)
        if op == "gate":
            if not c["ckpt"]:
                return dict(a=bsmm.bsmm_swiglu(state["h"]))
            a, q, s = bsmm.bsmm_swiglu(state["h"], checkpoint=True)
            return dict(a=a, q=q, scale=s)
        dh, act, drow = bsmm.bsmm_swiglu_backward(state["da"], state["q"], state["scale"],
                                                  row_scale=state["weight"])
        return dict(dh=dh, act=act) if drow is None else dict(dh=dh, act=act, drow=drow)
    if op == "mm":
        return _plain_mm(state)
    if op == "wgrad":
        return _plain_wgrad(state)
    if op == "quant":
        q, s, v = _plain_quant(state["x"])
        return dict(q=q, scale=s, values=v)
    if op == "gate":
        if not c["ckpt"]:
            return dict(a=_plain_gate(state["h"]))
        q, s, _ = _plain_quant(state["h"])
        return dict(a=_plain_gate(state["h"]), q=q, scale=s)
    return _plain_back(state)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    op = c["op"]
    if op in ("mm", "wgrad"):
        slots = c["T"] * c["k"]
        n, K = c["N"], c["K"]
        flops = 2 * slots * n * K
        if op == "mm":
            # experts that some slot is expected to reach, were the choice even
            touched = min(c["E"], max(c["k"], round(c["E"] * (1 - (1 - c["k"] / c["E"])
                                                             ** c["T"]))))
            depth, width = (n, K) if c["back"] else (K, n)
            rows = slots if c["second"] else c["T"]
            return {"bytes": rows * depth * SIZE[c["x"]] + touched * n * K * SIZE[c["x"]]
                    + slots * width * SIZE[c["o"]] + slots * 4, "flops": flops}
        dy, x = (c["T"], slots) if c["second"] else (slots, c["T"])
        return {"bytes": int(dy * n * SIZE[c["y"]] + x * K * SIZE[c["x"]]
                             + c["E"] * n * K * SIZE[c["o"]] + slots * 4), "flops": flops}
    if op == "quant":
        n = c["R"] * c["K"]
        return {"bytes": int(n * (2 * SIZE[c["x"]] + SIZE["ckpt"])), "flops": 4 * n}
    n = c["S"] * c["F"]
    size = SIZE[c["x"]]
    if op == "gate":
        return {"bytes": int(n * (3 * size + (2 * SIZE["ckpt"] if c["ckpt"] else 0))),
                "flops": 6 * n}
    return {"bytes": int(n * (4 * size + 2 * SIZE["ckpt"]) + c["S"] * 8 * c["weighted"]),
            "flops": 16 * n}


# ------------------------------------------------------------------- exact --

def _codes64(x):
    """An 8-bit checkpoint of x (numpy, 64 bits): codes, bytes, values."""
    m = x.reshape(x.shape[0], -1, 32)
    top = np.abs(m).max(2)
    byte = np.where(top == 0.0, 127, np.maximum(np.frexp(top)[1] + 126, 0)).astype(np.int32)
    step = np.ldexp(1.0, byte - 133)[..., None]
    q = np.clip(np.rint(m / step), -127, 127)
    return (q.reshape(x.shape).astype(np.int8), byte.astype(np.uint8),
            (q * step).reshape(x.shape))


def _values64(q, byte):
    step = np.ldexp(1.0, byte.astype(np.int32) - 133)
    return q.astype(np.float64) * np.repeat(step, 32, axis=1)


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _experts64(st):
    """The expert of every slot, -1 for none (numpy)."""
    order, ends = st["order"].cpu().numpy(), st["offsets"].cpu().numpy()
    expert = np.full(order.size, -1)
    for e in range(ends.size - 1):
        expert[order[ends[e]:ends[e + 1]]] = e
    return expert


def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    op = c["op"]
    if op in ("mm", "wgrad"):
        expert = torch.from_numpy(_experts64(st)).to(DEV)
        slot = torch.arange(expert.numel(), device=DEV)
        if op == "mm":
            out = torch.zeros((expert.numel(), c["K"] if c["back"] else c["N"]), device=DEV,
                              dtype=torch.float64)
        else:
            out = torch.zeros((c["E"], c["N"], c["K"]), device=DEV, dtype=torch.float64)
            x = st["x"].to(torch.float64)
            if st["x_scale"] is not None:
                step = torch.pow(2.0, st["x_scale"].to(torch.float64) - 133.0)
                x = x * step.repeat_interleave(32, dim=1)
        for e in range(c["E"]):
            mine = slot[expert == e]
            if mine.numel() == 0:
                continue
            token = torch.div(mine, c["k"], rounding_mode="floor")
            if op == "mm":
                w = st["w"][e].to(torch.float64)
                w = w if c["back"] else w.t().contiguous()
                y = torch.mm(st["x"][mine if c["second"] else token].to(torch.float64), w)
                if st["weight"] is not None:
                    y *= st["weight"][mine].to(torch.float64)[:, None]
                out[mine] = y
            else:
                dy = st["dy"][token if c["second"] else mine].to(torch.float64)
                out[e] = torch.mm(dy.t().contiguous(), x[mine if c["second"] else token])
        return out.cpu().numpy()
    if op == "quant":
        q, byte, values = _codes64(_np(st["x"]))
        return dict(q=q, scale=byte, values=values)
    if op == "gate":
        h = st["h"].to(torch.float64)
        g, u = h[:, :c["F"]], h[:, c["F"]:]
        out = dict(a=(u * g * torch.sigmoid(g)).cpu().numpy())
        if c["ckpt"]:
            out["q"], out["scale"], _ = _codes64(h.cpu().numpy())
        return out
    h = torch.from_numpy(_values64(st["q"].cpu().numpy(), st["scale"].cpu().numpy())).to(DEV)
    g, u = h[:, :c["F"]], h[:, c["F"]:]
    da = st["da"].to(torch.float64)
    w = 1.0 if st["weight"] is None else st["weight"].to(torch.float64)[:, None]
    silu = g * torch.sigmoid(g)
    # silu' = sigma + silu (1 - sigma), with 1 - sigma(g) = sigma(-g)
    slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
    out = dict(dh=torch.cat([w * da * u * slope, w * da * silu], 1).cpu().numpy(),
               act=(w * silu * u).cpu().numpy())
    if st["weight"] is not None:
        out["drow"] = (da * silu * u).sum(1).cpu().numpy()
    return out
