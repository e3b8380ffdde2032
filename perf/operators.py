"""What is measured of the operators around the experts: the layer norm with
its gradient, activation checkpoints in 8 bits with their use in the backward
pass, and the experts' matrix-vector products with weights in 4 bits, for
tokens that are generated.

A case names one operator (or a forward with its backward, where the 8-bit
checkpoint that the one writes is what the other reads), its sizes and its
type. `own` chooses between the plain form, written with elementary torch
operations in 32 bits, and the library's calls.

The 8-bit format is OCP MXINT8: per 32 neighbouring elements of a row one
power-of-two scale X = 2^floor(log2 amax), and whole numbers c in [-127, 127]
that stand for c * X / 64, rounded to nearest even. A checkpoint is a uint8
tensor of the elements (two's complement) and one of the scales' exponents
(biased by 127). The 4-bit weights are OCP MXFP4: per 32 neighbouring elements
of a row one such exponent, and elements of one sign and three magnitude bits
that stand for 0, 1/2, 1, 3/2, 2, 3, 4, 6; two a byte, the first in the low half.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # the norm in front of the experts at the layer's own size: the forward
        # adds the sublayer before it to the residual stream and keeps the
        # stream in 8 bits, the backward reads it from there
        {"name": "norm_train_bf16", "op": "norm_train", "T": 16384, "d": 2048, "bf16": True, "bias": True, "stream": True, "act8": True},
        # the widest of the layer's sizes, the largest case
        {"name": "norm_train_wide", "op": "norm_train", "T": 32768, "d": 4096, "bf16": True, "bias": False, "stream": True, "act8": True},
        # one token while text is generated
        {"name": "norm_one_token", "op": "norm", "T": 1, "d": 2048, "bf16": True, "bias": True, "stream": True},
        # the gradient alone, fp32, odd sizes in both directions
        {"name": "norm_back_f32", "op": "norm_back", "T": 1003, "d": 4128, "bf16": False, "bias": True, "stream": False, "act8": False},
        # gate and up projections of all routed rows, stored and brought back
        {"name": "act8_bf16", "op": "act8", "rows": 65536, "cols": 2048, "bf16": True},
        # a few rows of an odd width in fp32
        {"name": "act8_f32_odd", "op": "act8", "rows": 77, "cols": 352, "bf16": False},
        # the backward's gate, up and hidden rows rebuilt from the checkpoint
        {"name": "swiglu_bf16", "op": "swiglu", "rows": 65536, "h": 1024, "bf16": True},
        {"name": "swiglu_f32_odd", "op": "swiglu", "rows": 1001, "h": 416, "bf16": False},
        # the combine that also keeps the experts' rows in 8 bits, and its
        # backward from them (with the router's), at the layer's own size
        {"name": "combine_train_bf16", "op": "combine_train", "T": 16384, "d": 2048, "E": 128, "k": 4, "bf16": True},
        # the combine's backward alone on a handful of tokens
        {"name": "combine_back_f32", "op": "combine_back", "T": 37, "d": 352, "E": 8, "k": 2, "bf16": False},
        # the experts of one generated token, of the layer's own widths
        {"name": "w4_one_token", "op": "w4", "T": 1, "d": 2048, "h": 1024, "E": 128, "k": 4, "bf16": True},
        # the experts of a batch of sequences that are generated together
        {"name": "w4_batch", "op": "w4", "T": 64, "d": 2048, "h": 1024, "E": 128, "k": 4, "bf16": True},
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return 32 * max(1, _size(rng, lo, hi) // 32)


def draw(rng):
    """One more case: rows from one to the largest listed count, widths in
    steps of 32, no more bytes than the largest listed case."""
    most = work(listed()[1])["bytes"]
    while True:
        op = rng.choice(["norm_train", "norm", "norm_back", "act8", "swiglu", "combine_train", "combine_back", "w4", "w4"])
        bf16 = rng.random() < 0.6
        if op.startswith("norm"):
            c = {"op": op, "T": _size(rng, 1, 65536), "d": _width(rng, 32, 16384), "bf16": bf16, "bias": rng.random() < 0.5, "stream": rng.random() < 0.5}
            if op != "norm":
                c["act8"] = rng.random() < 0.6
        elif op == "act8":
            c = {"op": op, "rows": _size(rng, 1, 131072), "cols": _width(rng, 32, 16384), "bf16": bf16}
        elif op == "swiglu":
            c = {"op": op, "rows": _size(rng, 1, 131072), "h": _width(rng, 32, 8192), "bf16": bf16}
        elif op == "w4":
            E = _size(rng, 2, 256)
            c = {"op": op, "T": _size(rng, 1, 256), "d": _width(rng, 32, 8192), "h": _width(rng, 32, 4096), "E": E, "k": rng.randint(1, min(8, E)), "bf16": True}
            if E * c["h"] * c["d"] > 128 * 2048 * 1024:
                continue
        else:
            E = _size(rng, 2, 256)
            c = {"op": op, "T": _size(rng, 1, 32768), "d": _width(rng, 32, 16384), "E": E, "k": rng.randint(1, min(8, E)), "bf16": bf16}
        if work(c)["bytes"] <= most:
            return c


def work(case):
    op, s = case["op"], 2 if case["bf16"] else 4
    q = 1 + 1 / 32  # bytes of a checkpointed element
    if op.startswith("norm"):
        T, d = case["T"], case["d"]
        n = T * d
        wb = 8 if case["bias"] else 4
        # x (and the rows added to it, and their sum) in, y out
        fwd = n * s * (4 if case["stream"] else 2) + d * wb
        # dy (and the stream's gradient) in, dx out, x or its checkpoint in, the weight's gradients out
        x = q if case.get("act8") else s
        bwd = n * (s * (3 if case["stream"] else 2) + x) + 8 * T + d * (4 + wb)
        if op == "norm":
            return {"bytes": fwd, "flops": 8 * n}
        if op == "norm_back":
            return {"bytes": bwd, "flops": 14 * n}
        return {"bytes": fwd + bwd + 8 * T + (n * q if case["act8"] else 0), "flops": 22 * n}
    if op == "act8":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * (s + q), "flops": 4 * n}
    if op == "swiglu":
        n = case["rows"] * case["h"]
        return {"bytes": n * (2 * q + 3 * s), "flops": 12 * n}
    T, d, E, k = case["T"], case["d"], case["E"], case["k"]
    if op == "w4":
        h = case["h"]
        # the experts that T tokens choose at random, their weights read once
        n = E * (1 - (1 - k / E) ** T) * 3 * h * d
        return {"bytes": n * (1 / 2 + 1 / 32) + 2 * T * d * s + 20 * T * k + 4 * E, "flops": 6 * T * k * h * d}
    n = T * k * d
    bwd = T * d * s + n * (q + s) + 12 * T * k + 4 * T * E + 4 * T * k
    if op == "combine_back":
        return {"bytes": bwd, "flops": 3 * n}
    return {"bytes": bwd + n * (s + q) + T * d * s + 8 * T * k, "flops": 6 * n}


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _channels(g, d):
    """Widths of a model's channels: most alike, some several times larger."""
    return torch.exp(0.5 * _randn(g, d))


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _weights4(g, E, rows, cols):
    """E matrices of normal weights in 4 bits (nearest element): bytes and scales' exponents."""
    w = (_randn(g, E, rows, cols) * cols ** -0.5).view(E, rows, cols // 32, 32)
    e = (w.abs().amax(3).view(torch.int32) >> 23) - 2  # the largest element, 6, is 1.5 * 2^2
    v = torch.ldexp(w.abs(), 127 - e[..., None])
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = torch.bucketize(v, mid, out_int32=True).to(torch.uint8) | (w < 0).to(torch.uint8) << 3
    c = c.view(E, rows, cols // 2, 2)
    return c[..., 0] | c[..., 1] << 4, e.to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], torch.bfloat16 if case["bf16"] else torch.float32
    st = dict(case)
    if op.startswith("norm"):
        T, d = case["T"], case["d"]
        st["weight"] = 1 + 0.1 * _randn(g, d)
        st["bias_v"] = 0.1 * _randn(g, d) if case["bias"] else None
        st["x"] = (_randn(g, T, d) * _channels(g, d) + 0.1).to(dt)
        st["res"] = _randn(g, T, d).to(dt) if case["stream"] and op != "norm_back" else None
        if op != "norm":
            st["dy"] = _randn(g, T, d).to(dt)
            st["dsum"] = _randn(g, T, d).to(dt) if case["stream"] else None
        if op == "norm_back":
            x = st["x"].double()
            st["mean"] = x.mean(1).float()
            st["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
            if case["act8"]:
                st["x8"], st["x8_scale"] = _encode(st["x"])
        if op == "norm":  # buffers that a decoding loop keeps
            st["out"] = {"y": torch.empty_like(st["x"])}
            if case["stream"]:
                st["out"]["sum"] = torch.empty_like(st["x"])
    elif op == "act8":
        st["x"] = (_randn(g, case["rows"], case["cols"]) * _channels(g, case["cols"])).to(dt)
    elif op == "swiglu":
        ab = (_randn(g, case["rows"], 2 * case["h"]) * _channels(g, 2 * case["h"])).to(dt)
        st["ab8"], st["ab8_scale"] = _encode(ab)
    else:
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        if op == "w4":
            h = case["h"]
            st["w1q"], st["w1s"] = _weights4(g, E, 2 * h, d)
            st["w2q"], st["w2s"] = _weights4(g, E, d, h)
            st["x"] = _randn(g, T, d).to(dt)
        top, idx = _randn(g, T, E).topk(k, dim=1)
        st["topk_gate"] = torch.softmax(top, 1).contiguous()
        st["topk_idx"] = idx.int().contiguous()
        order = torch.argsort(idx.reshape(-1), stable=True)  # rows by expert, then by token
        pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
        pos[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        st["token_pos"] = pos.view(T, k)
        if op == "w4":  # the rest of what the routing hands on
            st["sorted_token"] = torch.div(order, k, rounding_mode="floor").int()
            ends = torch.bincount(idx.reshape(-1), minlength=E).cumsum(0).int()
            st["offsets"] = torch.cat([ends.new_zeros(1), ends])
            return st
        y = (_randn(g, T * k, d) * _channels(g, d)).to(dt)
        st["dout"] = _randn(g, T, d).to(dt)
        if op == "combine_train":
            st["y"] = y
        else:
            st["y8"], st["y8_scale"] = _encode(y)
    return st


# ---------------------------------------------------------------------------
# the plain forms


def _encode(x):
    """The checkpoint of x: its elements and its scales' exponents, bytes."""
    b = x.float().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(2)
    e = (amax.view(torch.int32) >> 23) & 0xFF  # biased exponent of amax
    # 2^(133 - e), in two factors that are normal numbers
    half = (133 - e) // 2
    b = torch.ldexp(torch.ldexp(b, half[..., None]), (133 - e - half)[..., None])
    c = b.round().clamp(-127, 127).to(torch.int8)
    return c.reshape(x.shape).view(torch.uint8), e.to(torch.uint8)


def _decode(q, scale):
    """The values that a checkpoint stands for, in fp32."""
    c = q.view(torch.int8).float().reshape(q.shape[0], -1, 32)
    return torch.ldexp(c, scale[..., None].int() - 133).reshape(q.shape)


def _norm(x, weight, bias):
    f = x.float()
    mean = f.mean(1)
    m = f - mean[:, None]
    rstd = torch.rsqrt((m * m).mean(1) + EPS)
    y = m * rstd[:, None] * weight
    return (y if bias is None else y + bias).to(x.dtype), mean, rstd


def _norm_back(f, mean, rstd, dy, weight, dsum, has_bias):
    g = dy.float()
    xh = (f - mean[:, None]) * rstd[:, None]
    gw = g * weight
    dx = rstd[:, None] * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.float()
    return {"dx": dx.to(dy.dtype), "dweight": (g * xh).sum(0), "dbias": g.sum(0) if has_bias else None}


def _combine_back(y, st):
    """y: the experts' rows that the checkpoint stands for, in fp32."""
    gate, pos, go = st["topk_gate"], st["token_pos"].long(), st["dout"].float()
    dgate = (y[pos] * go[:, None]).sum(2)
    dy = torch.empty(y.shape, dtype=st["dout"].dtype, device=y.device)
    dy[pos.reshape(-1)] = (gate[..., None] * go[:, None]).to(dy.dtype).reshape(y.shape)
    # g_i sum_j g_j (dg_i - dg_j): the gates of a token sum to one
    rows = gate * ((dgate[:, :, None] - dgate[:, None, :]) * gate[:, None, :]).sum(2)
    dlogits = torch.zeros(gate.shape[0], st["E"], device=y.device)
    return {"dy_perm": dy, "dlogits": dlogits.scatter(1, st["topk_idx"].long(), rows), "dgate": dgate}


def _decode4(q, scale):
    """The weights that 4-bit elements [..., rows, cols/2] and scales stand for, in fp32."""
    both = torch.stack((q & 15, q >> 4), -1).reshape(*scale.shape, 32).int()
    v = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=q.device)[both]
    return torch.ldexp(v, scale[..., None].int() - 127).flatten(-2)


def _experts4(st):
    x, idx, E, T, k, h = st["x"].float(), st["topk_idx"].long(), st["E"], st["T"], st["k"], st["h"]
    if T * k < E:  # the chosen experts' weights for every token
        w1, w2 = (_decode4(st[q][idx.reshape(-1)], st[s][idx.reshape(-1)]) for q, s in (("w1q", "w1s"), ("w2q", "w2s")))
        ab = torch.bmm(w1, x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        a, b = ab[:, :h], ab[:, h:]
        y = torch.bmm(w2, (a / (1 + torch.exp(-a)) * b)[:, :, None]).view(T, k, -1)
    else:  # all experts for all tokens, then the chosen ones
        ab = torch.matmul(_decode4(st["w1q"], st["w1s"]), x.t())
        a, b = ab[:, :h], ab[:, h:]
        y = torch.bmm(_decode4(st["w2q"], st["w2s"]), a / (1 + torch.exp(-a)) * b)  # [E, d, T]
        y = y[idx, :, torch.arange(T, device=x.device)[:, None]]
    return (st["topk_gate"][..., None] * y).sum(1).to(st["x"].dtype)


def _plain(st):
    op = st["op"]
    if op == "w4":
        return _experts4(st)
    if op == "norm" or op == "norm_train":
        s = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(st["x"].dtype)
        y, mean, rstd = _norm(s, st["weight"], st["bias_v"])
        out = {"y": y, "sum": None if st["res"] is None else s}
        if op == "norm":
            return out
        f = _decode(*_encode(s)) if st["act8"] else s.float()
        return {**out, "mean": mean, "rstd": rstd,
                **_norm_back(f, mean, rstd, st["dy"], st["weight"], st["dsum"], st["bias"])}
    if op == "norm_back":
        f = _decode(st["x8"], st["x8_scale"]) if st["act8"] else st["x"].float()
        return _norm_back(f, st["mean"], st["rstd"], st["dy"], st["weight"], st["dsum"], st["bias"])
    if op == "act8":
        return _decode(*_encode(st["x"])).to(st["x"].dtype)
    if op == "swiglu":
        dt = torch.bfloat16 if st["bf16"] else torch.float32
        ab = _decode(st["ab8"], st["ab8_scale"])
        a, b = ab[:, :st["h"]], ab[:, st["h"]:]
        return {"ab": ab.to(dt), "hp": (a / (1 + torch.exp(-a)) * b).to(dt)}
    if op == "combine_train":
        y, pos = st["y"], st["token_pos"].long()
        out = (y.float()[pos] * st["topk_gate"][..., None]).sum(1).to(y.dtype)
        return {"out": out, **_combine_back(_decode(*_encode(y)), st)}
    return _combine_back(_decode(st["y8"], st["y8_scale"]), st)


# ---------------------------------------------------------------------------
# the library's calls


def _calls(st):
    import routing_grouped_gemm_router_amd as moe

    op = st["op"]
    if op == "norm":
        r = moe.moe_layer_norm(st["x"], st["weight"], st["bias_v"], EPS, residual=st["res"], stats=False, out=st["out"])
        return {"y": r["y"], "sum": r.get("sum")}
    if op == "norm_train":
        r = moe.moe_layer_norm(st["x"], st["weight"], st["bias_v"], EPS, residual=st["res"], act8=st["act8"])
        saved = dict(r, x=None if st["act8"] else (st["x"] if st["res"] is None else r["sum"]))
        b = moe.moe_layer_norm_backward(saved, st["dy"], st["weight"], dsum=st["dsum"], want_dbias=st["bias"])
        return {"y": r["y"], "sum": r.get("sum"), "mean": r["mean"], "rstd": r["rstd"],
                "dx": b["dx"], "dweight": b["dweight"], "dbias": b.get("dbias")}
    if op == "norm_back":
        saved = {"mean": st["mean"], "rstd": st["rstd"]}
        saved.update({"x8": st["x8"], "x8_scale": st["x8_scale"]} if st["act8"] else {"x": st["x"]})
        b = moe.moe_layer_norm_backward(saved, st["dy"], st["weight"], dsum=st["dsum"], want_dbias=st["bias"])
        return {"dx": b["dx"], "dweight": b["dweight"], "dbias": b.get("dbias")}
    if op == "act8":
        q, scale = moe.moe_act8_store(st["x"])
        return moe.moe_act8_load(q, scale, st["x"].dtype)
    if op == "swiglu":
        ab, hp = moe.moe_act8_swiglu(st["ab8"], st["ab8_scale"], torch.bfloat16 if st["bf16"] else torch.float32)
        return {"ab": ab, "hp": hp}
    if op == "w4":
        return moe.moe_w4_experts(st["x"], st, st["w1q"], st["w1s"], st["w2q"], st["w2s"])
    out = {}
    y8, scale = st.get("y8"), st.get("y8_scale")
    if op == "combine_train":
        out["out"], y8, scale = moe.moe_combine_act8(st["y"], st["topk_gate"], st["token_pos"])
    b = moe.moe_combine_backward_act8(st["dout"], y8, scale, st["topk_gate"], st["topk_idx"], st["token_pos"], st["E"])
    return {**out, "dy_perm": b["dy_perm"], "dlogits": b["dlogits"], "dgate": b["dgate"]}


def run(st):
    return _calls(st) if own else _plain(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_act8(x):
    """Every block of 32 rounded to multiples of its step, amax's power of two over 64."""
    v = x.double().view(x.shape[0], x.shape[1] // 32, 32)
    top = v.abs().max(dim=2, keepdim=True).values
    _, p = torch.frexp(top)  # top = m 2^p with m in [1/2, 1)
    step = torch.exp2(torch.where(top == 0, -133, (p - 7).clamp(min=-133)).double())
    return (torch.round(v / step).clamp(-127, 127) * step).view(x.shape)


def _exact_codes(q, scale):
    n = q.to(torch.int16)
    n = torch.where(n > 127, n - 256, n).double()
    return n * torch.exp2(scale.double() - 133).repeat_interleave(32, dim=1)


def _exact_weights4(q, scale):
    """Sign, two exponent bits, one mantissa bit: (1 + m/2) 2^(e-1), or m/2 where e is 0."""
    c = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
    c[:, 0::2], c[:, 1::2] = (q % 16).long(), (q // 16).long()
    e, m, sign = (c // 2) % 4, (c % 2).double(), 1 - 2 * (c // 8).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    return sign * v * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        w = st["weight"].double()
        out, x, mean, rstd = {}, st["x"], None, None
        if op != "norm_back":
            if st["res"] is not None:  # the stream is kept in the inputs' type
                x = (x.double() + st["res"].double()).to(x.dtype)
            v = x.double()
            var, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
            rstd = 1 / torch.sqrt(var + EPS)
            y = (v - mean) * rstd * w
            out = {"y": y if st["bias_v"] is None else y + st["bias_v"].double(), "sum": v if st["res"] is not None else None}
            if op == "norm":
                return out
            out.update(mean=mean[:, 0], rstd=rstd[:, 0])
            v = _exact_act8(x) if case["act8"] else v
        else:
            mean, rstd = st["mean"].double()[:, None], st["rstd"].double()[:, None]
            v = _exact_codes(st["x8"], st["x8_scale"]) if case["act8"] else x.double()
        dy, d = st["dy"].double(), case["d"]
        n = (v - mean) * rstd
        t = dy * w
        dx = (t - t.sum(1, keepdim=True) / d - n * ((t * n).sum(1, keepdim=True) / d)) * rstd
        if st["dsum"] is not None:
            dx += st["dsum"].double()
        return {**out, "dx": dx, "dweight": (n * dy).sum(0), "dbias": dy.sum(0) if case["bias"] else None}
    if op == "act8":
        return _exact_act8(st["x"])
    if op == "swiglu":
        ab = _exact_codes(st["ab8"], st["ab8_scale"])
        return {"ab": ab, "hp": torch.sigmoid(ab[:, :case["h"]]) * ab[:, :case["h"]] * ab[:, case["h"]:]}
    T, k = case["T"], case["k"]
    if op == "w4":
        x, h = st["x"].double(), case["h"]
        out = torch.zeros_like(x)
        for e in range(case["E"]):
            t, j = torch.nonzero(st["topk_idx"] == e, as_tuple=True)
            if len(t):
                ab = x[t] @ _exact_weights4(st["w1q"][e], st["w1s"][e]).T
                y = (torch.sigmoid(ab[:, :h]) * ab[:, :h] * ab[:, h:]) @ _exact_weights4(st["w2q"][e], st["w2s"][e]).T
                out[t] += st["topk_gate"][t, j].double()[:, None] * y
        return out
    gate, pos, out = st["topk_gate"].double(), st["token_pos"].long(), {}
    y = _exact_act8(st["y"]) if op == "combine_train" else _exact_codes(st["y8"], st["y8_scale"])
    go = st["dout"].double()
    dy = torch.zeros_like(y)
    dgate = torch.empty_like(gate)
    total = torch.zeros_like(go)
    for j in range(k):
        dgate[:, j] = torch.linalg.vecdot(go, y[pos[:, j]])
        dy[pos[:, j]] = gate[:, j:j + 1] * go
        if op == "combine_train":
            total += gate[:, j:j + 1] * st["y"][pos[:, j]].double()
    if op == "combine_train":
        out["out"] = total
    dlogits = torch.zeros(T, case["E"], dtype=torch.float64, device=y.device)
    # the gates' sum is one up to their rounding: the differences' form of the softmax's gradient
    dlogits.scatter_(1, st["topk_idx"].long(), gate * torch.stack([(gate * (dgate[:, i:i + 1] - dgate)).sum(1) for i in range(k)], 1))
    return {**out, "dy_perm": dy, "dlogits": dlogits, "dgate": dgate}
