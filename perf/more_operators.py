"""What is measured of the operators that the layer's training step and its
prompts need beside the experts' own: the root-mean-square norm with the
residual's addition and an output in 8 bits, the norm of many gradients
together with their clipping, and the experts' products of 8-bit rows with
4-bit weights.

A case names one operator (or a forward with its backward), its sizes and its
type. `own` chooses between the plain form, written with elementary torch
operations, and the library's calls.

The 8-bit rows are OCP MXFP8: per 32 neighbouring elements of a row one
power-of-two scale X = 2^(floor(log2 amax) - 8) (its exponent biased by 127 in
a byte, 0 at least) and E4M3 elements, nearest even, saturated to +-448. The
4-bit weights are OCP MXFP4: per 32 elements one such exponent, and elements of
one sign and three magnitude bits that stand for 0, 1/2, 1, 3/2, 2, 3, 4, 6;
two a byte, the first in the low half.
"""
import math
import random

import torch

own = False

EPS = 1e-6
MAX_NORM = 1.0


def listed():
    return [
        # the norm of a training step at the layer's own size: the forward adds
        # the sublayer before it to the residual stream and writes the rows
        # that the router reads in bf16 and the 8-bit experts in MXFP8
        {"name": "rms_train_bf16", "op": "rms_train", "T": 16384, "d": 2048, "bf16": True, "stream": True, "quant": True},
        # a prompt's norm that writes the 8-bit rows alone, wide rows
        {"name": "rms_prompt_8bit", "op": "rms", "T": 8192, "d": 4096, "bf16": True, "stream": True, "quant": True},
        # one token while text is generated
        {"name": "rms_one_token", "op": "rms", "T": 1, "d": 2048, "bf16": True, "stream": True, "quant": False},
        # the gradient alone, fp32, odd sizes in both directions
        {"name": "rms_back_f32", "op": "rms_back", "T": 1003, "d": 4128, "bf16": False, "stream": False},
        # the norm of the layer's own weight gradients (128 experts), as it is logged
        {"name": "grad_norm_layer", "op": "grad_norm", "kind": "layer", "E": 128, "d": 2048, "h": 1024, "type": "f32"},
        # and their clipping, the largest case
        {"name": "clip_layer", "op": "clip", "kind": "layer", "E": 128, "d": 2048, "h": 1024, "type": "f32"},
        # many tensors of a model's other parts, each at any place of one flat
        # buffer, in bf16 and fp32
        {"name": "clip_many_mixed", "op": "clip", "kind": "many", "count": 60, "most": 4000000, "sizes": 7, "type": "mixed"},
        # a norm's weight, a small router and its bias: latency alone
        {"name": "clip_few_small", "op": "clip", "kind": "many", "count": 4, "most": 20000, "sizes": 3, "type": "f32"},
        # the down projection of all routed rows of 16384 tokens
        {"name": "w4_down_e128", "op": "w4_gemm", "T": 16384, "K": 1024, "N": 2048, "E": 128, "k": 4, "skew": 0.0, "gather": False},
        # rows read through the routing's map, uneven experts, odd sizes
        {"name": "w4_gather_odd", "op": "w4_gemm", "T": 1003, "K": 640, "N": 416, "E": 7, "k": 2, "skew": 3.0, "gather": True},
        # the experts of a long prompt, of the layer's own widths
        {"name": "w4_prompt_e128", "op": "w4_experts", "T": 16384, "d": 2048, "h": 1024, "E": 128, "k": 4, "skew": 0.0},
        # the experts of a short prompt: some rows an expert, bound by the weights
        {"name": "w4_prompt_short", "op": "w4_experts", "T": 500, "d": 2048, "h": 1024, "E": 32, "k": 2, "skew": 0.5},
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    return step * max(1, _size(rng, lo, hi) // step)


def draw(rng):
    """One more case: rows from one to more than the listed ones, widths in
    the steps that the formats need, no more work than the largest listed."""
    top = {c["op"]: work(c) for c in listed()}
    most = max(w["bytes"] for w in top.values())
    most_flops = max(w["flops"] for w in top.values())
    while True:
        op = rng.choice(["rms", "rms_train", "rms_back", "grad_norm", "clip", "clip", "w4_gemm", "w4_gemm", "w4_experts", "w4_experts"])
        if op.startswith("rms"):
            c = {"op": op, "T": _size(rng, 1, 65536), "d": _width(rng, 32, 16384, 32), "bf16": rng.random() < 0.6, "stream": rng.random() < 0.5}
            if op != "rms_back":
                c["quant"] = rng.random() < 0.6
        elif op in ("grad_norm", "clip"):
            if rng.random() < 0.3:
                c = {"op": op, "kind": "layer", "E": _size(rng, 2, 128), "d": _width(rng, 32, 4096, 32), "h": _width(rng, 32, 2048, 32)}
            else:
                c = {"op": op, "kind": "many", "count": _size(rng, 1, 60), "most": _size(rng, 1, 20000000), "sizes": rng.randrange(1 << 30)}
            c["type"] = rng.choice(["f32", "f32", "bf16", "mixed"])
        else:
            E = _size(rng, 2, 256)
            c = {"op": op, "T": _size(rng, 1, 32768), "E": E, "k": rng.randint(1, min(8, E)), "skew": rng.choice([0.0, 0.0, 0.5, 1.5])}
            if op == "w4_gemm":
                c.update(K=_width(rng, 128, 8192, 128), N=_width(rng, 32, 8192, 32), gather=rng.random() < 0.5)
                weights = E * c["K"] * c["N"]
            else:
                c.update(d=_width(rng, 128, 8192, 128), h=_width(rng, 128, 4096, 128))
                weights = 3 * E * c["d"] * c["h"]
            # the plain form's padded groups and wide weights fit the card
            if weights > 3 * 128 * 2048 * 1024 or c["T"] * c["k"] > 131072 or c["T"] * c["k"] * max(c.get("N", 0), c.get("K", 0), c.get("d", 0), 2 * c.get("h", 0)) > 3 << 28:
                continue
        w = work(c)
        if w["bytes"] <= most and w["flops"] <= most_flops:
            return c


def _shapes(case):
    """The shapes of a case's gradients and whether each is bf16."""
    if case["kind"] == "layer":  # both projections, the router's weight, the norm's
        E, d, h = case["E"], case["d"], case["h"]
        shapes = [(E, 2 * h, d), (E, d, h), (E, d), (d,)]
    else:
        r = random.Random(case["sizes"])
        shapes = [(_size(r, 1, case["most"]),) for _ in range(case["count"])]
    t = case["type"]
    return [(s, t == "bf16" or (t == "mixed" and i % 3 != 0)) for i, s in enumerate(shapes)]


def work(case):
    op, q = case["op"], 1 + 1 / 32  # bytes of an 8-bit element with its scale
    if op.startswith("rms"):
        T, d, s = case["T"], case["d"], 2 if case["bf16"] else 4
        n = T * d
        quant = case.get("quant")
        # x (and the rows added to it, and their sum) in; y out, or its 8 bits
        # alone with the values that they stand for (in bf16, which holds them)
        fwd = n * s * (3 if case["stream"] else 1) + 4 * d + (n * (2 * q + 2) if quant else n * s)
        bwd = n * s * (4 if case["stream"] else 3) + 4 * T + 8 * d
        if op == "rms":
            return {"bytes": fwd, "flops": 8 * n}
        if op == "rms_back":
            return {"bytes": bwd, "flops": 11 * n}
        return {"bytes": fwd + bwd + 4 * T + (n * s if quant else 0), "flops": 19 * n}
    if op in ("grad_norm", "clip"):
        sizes = [(math.prod(s), 2 if b else 4) for s, b in _shapes(case)]
        n = sum(m * s for m, s in sizes)
        return {"bytes": (2 if op == "clip" else 1) * n + 4, "flops": (3 if op == "clip" else 2) * sum(m for m, _ in sizes)}
    T, E, k = case["T"], case["E"], case["k"]
    R, hit = T * k, E * (1 - (1 - k / E) ** T)  # the experts that T tokens choose
    if op == "w4_gemm":
        K, N = case["K"], case["N"]
        rows = T if case["gather"] else R
        return {"bytes": rows * K * q + hit * N * K * (1 / 2 + 1 / 32) + 2 * R * N + (4 * R if case["gather"] else 0), "flops": 2 * R * N * K}
    d, h = case["d"], case["h"]
    return {"bytes": T * d * (q + 2) + hit * 3 * h * d * (1 / 2 + 1 / 32) + 20 * R, "flops": 6 * R * h * d}


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


def _weights4(g, E, rows, cols):
    """E matrices of normal weights in 4 bits (nearest element): bytes and scales' exponents."""
    w = (_randn(g, E, rows, cols) * cols ** -0.5).view(E, rows, cols // 32, 32)
    e = (w.abs().amax(3).view(torch.int32) >> 23) - 2  # the largest element, 6, is 1.5 * 2^2
    v = torch.ldexp(w.abs(), 127 - e[..., None])
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = torch.bucketize(v, mid, out_int32=True).to(torch.uint8) | (w < 0).to(torch.uint8) << 3
    c = c.view(E, rows, cols // 2, 2)
    return c[..., 0] | c[..., 1] << 4, e.to(torch.uint8)


def _routing(g, case):
    """What the routing hands on for T tokens, its experts as uneven as `skew` says."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _randn(g, T, E) + case["skew"] * torch.linspace(1, -1, E, device="cuda")
    top, idx = logits.topk(k, dim=1)
    order = torch.argsort(idx.reshape(-1), stable=True)  # rows by expert, then by token
    pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    ends = counts.cumsum(0).int()
    return {"topk_gate": torch.softmax(top, 1).contiguous(), "topk_idx": idx.int().contiguous(), "token_pos": pos.view(T, k),
            "sorted_token": torch.div(order, k, rounding_mode="floor").int(), "offsets": torch.cat([ends.new_zeros(1), ends]),
            "most": int(counts.max())}  # rows of the largest group, known to the host


def prepare(case, seed):
    g = _gen(seed)
    op, st = case["op"], dict(case)
    if op.startswith("rms"):
        T, d, dt = case["T"], case["d"], torch.bfloat16 if case["bf16"] else torch.float32
        st["weight"] = 1 + 0.1 * _randn(g, d)
        st["x"] = (_randn(g, T, d) * _channels(g, d)).to(dt)
        st["res"] = _randn(g, T, d).to(dt) if case["stream"] and op != "rms_back" else None
        if op != "rms":
            st["dy"] = _randn(g, T, d).to(dt)
            st["dsum"] = _randn(g, T, d).to(dt) if case["stream"] else None
        if op == "rms_back":
            st["rstd"] = ((st["x"].double() ** 2).mean(1) + EPS).rsqrt().float()
        if op == "rms" and not case["quant"]:  # buffers that a decoding loop keeps
            st["out"] = {"y": torch.empty_like(st["x"])}
            if case["stream"]:
                st["out"]["sum"] = torch.empty_like(st["x"])
        return st
    if op in ("grad_norm", "clip"):
        shapes, st["grads"], st["out"] = _shapes(case), [], []
        for bf16 in (False, True):
            dt = torch.bfloat16 if bf16 else torch.float32
            if case["kind"] == "many":  # the tensors one after the other in a flat buffer
                flat = torch.empty(sum(math.prod(s) for s, b in shapes if b == bf16), dtype=dt, device="cuda")
                into = torch.empty_like(flat)
            at = 0
            for i, (shape, b) in enumerate(shapes):
                if b != bf16:
                    continue
                n = math.prod(shape)
                t = flat[at:at + n].view(shape) if case["kind"] == "many" else torch.empty(shape, dtype=dt, device="cuda")
                t.normal_(generator=g).mul_(10.0 ** (i % 4 - 3))
                if len(shape) == 3 and shape[0] > 1:
                    t[1] = 0  # an expert that no token chose
                st["grads"].append((i, t))
                st["out"].append((i, into[at:at + n].view(shape) if case["kind"] == "many" else torch.empty_like(t) if op == "clip" else None))
                at += n
        for name in ("grads", "out"):
            st[name] = [t for _, t in sorted(st[name], key=lambda p: p[0])]
        return st
    st.update(_routing(g, case))
    E, T = case["E"], case["T"]
    if op == "w4_gemm":
        rows, width = T if case["gather"] else T * case["k"], case["K"]
        st["wq"], st["ws"] = _weights4(g, E, case["N"], width)
    else:
        rows, width = T, case["d"]
        st["w1q"], st["w1s"] = _weights4(g, E, 2 * case["h"], width)
        st["w2q"], st["w2s"] = _weights4(g, E, width, case["h"])
    st["xq"], st["xs"] = _encode(_randn(g, rows, width) * _channels(g, width))
    return st


# ---------------------------------------------------------------------------
# the plain forms


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x):
    """x [..., cols] in MXFP8: E4M3 bytes and the scales' exponents."""
    b = x.float().reshape(-1, 32)
    amax = b.abs().amax(1)
    e = (((amax.view(torch.int32) >> 23) & 0xFF) - 8).clamp(min=0)
    # times 2^(127 - e), in two factors that are normal numbers
    half = (127 - e) // 2
    b = torch.ldexp(torch.ldexp(b, half[:, None]), (127 - e - half)[:, None])
    q = b.clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(x.shape), e.to(torch.uint8).reshape(*x.shape[:-1], -1)


def _decode(q, scale):
    """The values of MXFP8 bytes, in fp32."""
    v = q.view(torch.float8_e4m3fn).float().reshape(*scale.shape, 32)
    return torch.ldexp(v, scale[..., None].int() - 127).reshape(q.shape)


def _decode4(q, scale):
    """The weights that 4-bit elements [..., rows, cols/2] and scales stand for, in fp32."""
    both = torch.stack((q & 15, q >> 4), -1).reshape(*scale.shape, 32).int()
    v = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=q.device)[both]
    return torch.ldexp(v, scale[..., None].int() - 127).flatten(-2)


def _rms(st):
    s = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(st["x"].dtype)
    f = s.float()
    rstd = torch.rsqrt((f * f).mean(1) + EPS)
    y = (f * rstd[:, None] * st["weight"]).to(s.dtype)
    v = _decode(*_encode(y)).to(torch.bfloat16) if st["quant"] else None
    return s, y, v, rstd


def _rms_back(s, rstd, st):
    g, f = st["dy"].float(), s.float()
    xh = f * rstd[:, None]
    gw = g * st["weight"]
    dx = rstd[:, None] * (gw - xh * (gw * xh).mean(1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(s.dtype), "dweight": (g * xh).sum(0)}


def _grouped(a, w, st):
    """a [rows, K] in expert order times w [E, N, K], each row by its expert's
    matrix: the groups padded to the largest one for a batched product."""
    off, most, E = st["offsets"].long(), st["most"], w.shape[0]
    at = torch.arange(most, device=a.device)
    rows = (off[:-1, None] + at).clamp(max=a.shape[0] - 1)  # [E, most], past a group's end any row
    y = torch.bmm(w, a[rows].transpose(1, 2).contiguous())  # [E, N, most]
    e = torch.repeat_interleave(torch.arange(E, device=a.device), off[1:] - off[:-1], output_size=a.shape[0])
    return y.transpose(1, 2)[e, torch.arange(a.shape[0], device=a.device) - off[e]]


def _plain(st):
    op = st["op"]
    if op == "rms":
        s, y, v, _ = _rms(st)
        return {"sum": None if st["res"] is None else s, "y": None if st["quant"] else y, "v": v}
    if op == "rms_train":
        s, y, v, rstd = _rms(st)
        return {"sum": None if st["res"] is None else s, "y": y, "v": v, "rstd": rstd, **_rms_back(s, rstd, st)}
    if op == "rms_back":
        return _rms_back(st["x"], st["rstd"], st)
    if op in ("grad_norm", "clip"):
        norm = torch.stack([g.double().square().sum() for g in st["grads"]]).sum().sqrt()
        if op == "grad_norm":
            return {"norm": norm.float()}
        scale = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
        return {"norm": norm.float(), "grads": [(g.float() * scale).to(g.dtype) for g in st["grads"]]}
    x = _decode(st["xq"], st["xs"])
    if op == "w4_gemm":
        if st["gather"]:
            x = x[st["sorted_token"].long()]
        return _grouped(x, _decode4(st["wq"], st["ws"]), st).to(torch.bfloat16)
    ab = _grouped(x[st["sorted_token"].long()], _decode4(st["w1q"], st["w1s"]), st)
    a, b = ab[:, :st["h"]], ab[:, st["h"]:]
    hp = _decode(*_encode(a / (1 + torch.exp(-a)) * b))
    y = _grouped(hp, _decode4(st["w2q"], st["w2s"]), st)
    return (y[st["token_pos"].long()] * st["topk_gate"][..., None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the library's calls


def _calls(st):
    import routing_grouped_gemm_router_amd as moe

    op = st["op"]
    if op == "rms":
        r = moe.moe_rms_norm(st["x"], st["weight"], EPS, residual=st["res"], quantize=st["quant"], want_y=not st["quant"], stats=False, out=st.get("out"))
        v = moe.mxfp8_dequantize(r["yq"], r["yq_scale"]) if st["quant"] else None
        return {"sum": r.get("sum"), "y": r.get("y"), "v": v}
    if op == "rms_train":
        r = moe.moe_rms_norm(st["x"], st["weight"], EPS, residual=st["res"], quantize=st["quant"])
        v = moe.mxfp8_dequantize(r["yq"], r["yq_scale"]) if st["quant"] else None
        saved = {"rstd": r["rstd"], "x": st["x"] if st["res"] is None else r["sum"]}
        b = moe.moe_rms_norm_backward(saved, st["dy"], st["weight"], dsum=st["dsum"])
        return {"sum": r.get("sum"), "y": r["y"], "v": v, "rstd": r["rstd"], "dx": b["dx"], "dweight": b["dweight"]}
    if op == "rms_back":
        b = moe.moe_rms_norm_backward({"rstd": st["rstd"], "x": st["x"]}, st["dy"], st["weight"], dsum=st["dsum"])
        return {"dx": b["dx"], "dweight": b["dweight"]}
    if op == "grad_norm":
        return {"norm": moe.moe_grad_norm(st["grads"])}
    if op == "clip":
        return {"norm": moe.moe_clip_grad_norm(st["grads"], MAX_NORM, out=st["out"]), "grads": st["out"]}
    if op == "w4_gemm":
        return moe.moe_w4_gemm(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], a_rows=st["sorted_token"] if st["gather"] else None)
    return moe.moe_w4_experts8(st["xq"], st["xs"], st, st["w1q"], st["w1s"], st["w2q"], st["w2s"])


def run(st):
    return _calls(st) if own else _plain(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_e4m3(x):
    """Every block of 32 rounded to E4M3 elements of its scale, 2^(p - 9) with
    2^(p-1) <= amax < 2^p: a significand of 4 bits, steps of 2^-9 at least."""
    v = x.double().reshape(-1, 32)
    top = v.abs().max(dim=1, keepdim=True).values
    _, p = torch.frexp(top)
    unit = torch.exp2(torch.where(top == 0, -127, (p - 9).clamp(min=-127)).double())
    v = v / unit
    _, m = torch.frexp(v)
    step = torch.exp2((m - 4).clamp(min=-9).double())
    return ((torch.round(v / step) * step).clamp(-448, 448) * unit).reshape(x.shape)


def _exact_codes(q, scale):
    """Sign, four exponent bits biased by 7, three mantissa bits."""
    c = q.to(torch.int64)
    e, m, sign = (c >> 3) & 15, (c & 7).double() / 8, 1 - 2 * (c >> 7).double()
    v = torch.where(e == 0, m * 2.0 ** -6, (1 + m) * torch.exp2(e.double() - 7))
    return sign * v * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=-1)


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
    if op.startswith("rms"):
        w, x, out = st["weight"].double(), st["x"], {}
        if op == "rms_back":
            v, rstd = x.double(), st["rstd"].double()[:, None]
        else:
            if st["res"] is not None:  # the stream is kept in the inputs' type
                x = (x.double() + st["res"].double()).to(x.dtype)
            v = x.double()
            rstd = 1 / torch.sqrt(torch.linalg.vecdot(v, v)[:, None] / case["d"] + EPS)
            y = v * rstd * w
            out = {"sum": v if st["res"] is not None else None, "y": None if op == "rms" and case["quant"] else y,
                   "v": _exact_e4m3(y.to(x.dtype)) if case["quant"] else None}
            if op == "rms":
                return out
            out["rstd"] = rstd[:, 0]
        dy, n = st["dy"].double(), v * rstd
        t = dy * w
        dx = (t - n * (torch.linalg.vecdot(t, n)[:, None] / case["d"])) * rstd
        if st["dsum"] is not None:
            dx += st["dsum"].double()
        return {**out, "dx": dx, "dweight": (n * dy).sum(0)}
    if op in ("grad_norm", "clip"):
        norm = 0.0
        for g in st["grads"]:
            v = g.double().reshape(-1)
            norm += float(torch.dot(v, v))
        norm = math.sqrt(norm)
        out = {"norm": torch.tensor(norm, dtype=torch.float64)}
        if op == "clip":
            out["grads"] = [g.double() * min(1.0, MAX_NORM / (norm + 1e-6)) for g in st["grads"]]
        return out
    x, off = _exact_codes(st["xq"], st["xs"]), st["offsets"].tolist()
    gather = op == "w4_experts" or case["gather"]
    y = torch.empty(case["T"] * case["k"], case["d"] if op == "w4_experts" else case["N"], dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        a = x[st["sorted_token"][lo:hi].long()] if gather else x[lo:hi]
        if op == "w4_gemm":
            y[lo:hi] = a @ _exact_weights4(st["wq"][e], st["ws"][e]).T
        else:
            ab = a @ _exact_weights4(st["w1q"][e], st["w1s"][e]).T
            u = torch.sigmoid(ab[:, :case["h"]]) * ab[:, :case["h"]] * ab[:, case["h"]:]
            y[lo:hi] = _exact_e4m3(u) @ _exact_weights4(st["w2q"][e], st["w2s"][e]).T
    if op == "w4_gemm":
        return y
    out = torch.zeros(case["T"], case["d"], dtype=torch.float64, device=x.device)
    for j in range(case["k"]):
        out += st["topk_gate"][:, j:j + 1].double() * y[st["token_pos"][:, j].long()]
    return out
