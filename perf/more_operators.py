"""Cases of the matrix products with an epilogue, the residual norms and the clipped update, with their plain forms.

Each case is one pass through one operator as a training step (or, where it says so, a prediction) calls it:

  lin_fwd   : y = residual + scale act(x w^T + b), where asked with the pre-activation beside it
  lin_dgrad : dx = add + scale (dz w) act'(pre), with the derivative of the activation that made x
  lin_wgrad : dw = scale dz^T x and db = scale sum dz
  rn_fwd    : r = x + scale gate N_post(f), h = N_pre(r): the norms after one block and before the next with the gated sum between
  rn_bwd    : its backward: gradients of the stream, of the block's output and of every vector
  norm      : the global norm of a list of gradients and the factor that clips it
  adam      : that norm and the Adam step of the list with clipped gradients

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and the library's entry points.
"""
import math

import torch

own = False

NORM_EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 2e-4, 0.9, 0.999, 1e-8, 0.01, 7
CLIP_EPS = 1e-6
GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


# --------------------------------------------------------------------------------------------------------------------- cases
def _lin(name, kind, rows, k, n, act="none", slope=1.0, scale=1.0, dtype="bf16", bias=True, residual=False, pre=False, x_pitch=0,
         y_pitch=0):
    return {"name": name, "kind": kind, "rows": rows, "k": k, "n": n, "act": act, "slope": slope, "scale": scale, "dtype": dtype,
            "bias": bias, "residual": residual, "pre": pre, "x_pitch": x_pitch, "y_pitch": y_pitch}


def _rn(name, kind, rows, c, post, pre, dtype="bf16", f_dtype="bf16", samples=1, gate="shared", modulated=False, scale=1.0):
    return {"name": name, "kind": kind, "rows": rows, "c": c, "post": post, "pre": pre, "dtype": dtype, "f_dtype": f_dtype,
            "samples": samples, "gate": gate, "modulated": modulated, "scale": scale}


def listed():
    return [
        # the hidden layer of the head at the training batch: few rows, all of the time is reading the weights
        _lin("lin_fwd head 8x2048->2048", "lin_fwd", 8, 2048, 2048, act="gelu"),
        # the widening product on every voxel behind the five-block stack's second block, kept for the backward: stores bound it
        _lin("lin_fwd voxels 8x64^3 64->256", "lin_fwd", 8 * 64 ** 3, 64, 256, act="gelu", pre=True),
        # a wide block's projection back, added to a stream in 32 bits: the largest product
        _lin("lin_fwd 16384x8192->4096 residual f32", "lin_fwd", 16384, 8192, 4096, scale=0.5, dtype="f32", residual=True),
        # a cropped volume's voxels and layer widths that fit nothing, rows in slices of wider tensors
        _lin("lin_dgrad ragged 100003x515->130", "lin_dgrad", 100003, 130, 515, act="silu", residual=True, x_pitch=133, y_pitch=520),
        # the weights of the widening product on the voxels: a long sum for a small result
        _lin("lin_wgrad voxels 8x64^3 64x256", "lin_wgrad", 8 * 64 ** 3, 64, 256),
        # the weights of a wide head's hidden layer at a large batch of crops
        _lin("lin_wgrad 16384 2048x8192", "lin_wgrad", 16384, 2048, 8192),
        # a block's output added to the last feature map of one volume and the next block's norm: only the latency counts
        _rn("rn_fwd 64x256", "rn_fwd", 64, 256, "none", "rms", gate="none"),
        # between two blocks on 32^3 voxels of eight samples, the gate and the norm before modulated by each sample's conditions
        _rn("rn_fwd 8x32^3x128 modulated", "rn_fwd", 8 * 32 ** 3, 128, "layer", "layer", samples=8, gate="sample", modulated=True),
        # its backward
        _rn("rn_bwd 8x32^3x128 modulated", "rn_bwd", 8 * 32 ** 3, 128, "layer", "layer", samples=8, gate="sample", modulated=True),
        # the backward on a wide stream in 32 bits
        _rn("rn_bwd 16384x4096 f32", "rn_bwd", 16384, 4096, "rms", "rms", dtype="f32", scale=0.7),
        # every gradient of the five-block stack: the smallest list, ten tensors
        {"name": "norm five-block", "kind": "norm", "shapes": "32x108,32,64x864,64,128x1728,128,256x3456,256,256x6912,256",
         "dtype": "f32", "max_norm": 1.0},
        # every tensor of the seven-conv network with a wide head
        {"name": "adam seven-conv wide head", "kind": "adam", "dtype": "f32", "max_norm": 1.0,
         "shapes": "16x108,16,32x432,32,64x864,64,128x1728,128,256x3456,256,256x6912,256,256x6912,256,"
                   "2048x16384,2048,2048x2048,2048,256x2048,256,4x256,4"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    w = _log(rng, lo, hi)
    return rng.choice([w, max(8, w // 8 * 8), 2 ** max(3, round(math.log2(w)))])


def _draw_lin(rng, kind):
    while True:
        k, n = _width(rng, 8, 12000), _width(rng, 8, 12000)
        rows = _log(rng, 1, 1 << 21)
        if kind == "lin_wgrad" and rows < 4:
            continue
        if rows * k * n > 16384 * 8192 * 4096 or rows * (k + 2 * n) > (1 << 21) * 576 or k * n > 1 << 27:
            continue
        act = rng.choice(["none", "lrelu", "silu", "gelu"]) if kind != "lin_wgrad" else "none"
        case = _lin("", kind, rows, k, n, act, {"none": 1.0, "lrelu": rng.choice([0.3, 0.01, 0.0])}.get(act, 1.0),
                    rng.choice([1.0, 0.5, 1.7]), rng.choice(["bf16", "bf16", "f32"]) if kind != "lin_wgrad" else "f32",
                    rng.random() < 0.8, rng.random() < 0.5 and kind != "lin_wgrad", kind == "lin_fwd" and rng.random() < 0.4,
                    0 if rng.random() < 0.7 else k + rng.choice([8, 64, rng.randint(1, 40)]),
                    0 if rng.random() < 0.7 else n + rng.choice([8, 64, rng.randint(1, 40)]))
        del case["name"]
        return case


def _draw_rn(rng, kind):
    while True:
        c = _width(rng, 16, 12000)
        samples = rng.choice([1, 1, 2, 8, rng.randint(1, 40)])
        rows = samples * _log(rng, 1, 1 << 18)
        if not 1 << 10 <= rows * c <= 1 << 26:
            continue
        post, pre = rng.choice([("none", "rms"), ("none", "layer"), ("rms", "rms"), ("layer", "layer"), ("rms", "none")])
        dtype, f_dtype = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        gate = rng.choice(["none", "shared", "sample"])
        case = _rn("", kind, rows, c, post, pre, dtype, f_dtype, samples, gate, pre != "none" and rng.random() < 0.3,
                   rng.choice([1.0, 0.5]))
        del case["name"]
        return case


def _draw_list(rng, kind):
    shapes = []
    total = 0
    for _ in range(rng.choice([_log(rng, 1, 200), rng.randint(5, 30)])):
        rows = rng.choice([2 ** rng.randrange(4, 12), _log(rng, 2, 2500)])
        cols = rng.choice([1, 27 * 2 ** rng.randrange(2, 9), _log(rng, 4, 9000)])
        if total + rows * cols > 60 << 20:
            continue
        total += rows * cols
        shapes.append("%dx%d" % (rows, cols) if cols > 1 else "%d" % rows)
    return {"kind": kind, "shapes": ",".join(shapes), "dtype": rng.choice(["f32", "f32", "bf16", "mixed"]) if kind == "norm" else "f32",
            "max_norm": rng.choice([1.0, 0.1, 1e4])}


def draw(rng):
    kind = rng.choice(["lin_fwd", "lin_dgrad", "lin_wgrad", "rn_fwd", "rn_bwd", "norm", "adam"])
    return _draw_lin(rng, kind) if kind.startswith("lin") else _draw_rn(rng, kind) if kind.startswith("rn") else _draw_list(rng, kind)


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


# -------------------------------------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(gen, rows, width, pitch, dtype):
    """Rows of `width` values, `pitch` apart where they are a slice of a wider tensor."""
    return torch.empty(rows, pitch or width, device="cuda", dtype=dtype).normal_(generator=gen)[:, :width]


def _prepare_lin(s, gen):
    case = s["case"]
    rows, k, n, kind = case["rows"], case["k"], case["n"], case["kind"]
    bf, dt = torch.bfloat16, _TYPES[case["dtype"]]
    if kind != "lin_dgrad":
        s["x"] = _normal(gen, rows, k, case["x_pitch"], bf)  # normalised features
    if kind != "lin_fwd":
        s["dz"] = _normal(gen, rows, n, case["y_pitch"], bf)
        s["dz"] += 0.1 * torch.randn(n, device="cuda", generator=gen).to(bf)
    if kind != "lin_wgrad":
        s["w"] = (torch.randn(n, k, device="cuda", generator=gen) * math.sqrt(1.0 / k)).to(bf)
    if kind == "lin_fwd":
        s["bias"] = 0.3 * torch.randn(n, device="cuda", generator=gen) if case["bias"] else None
        s["residual"] = _normal(gen, rows, n, case["y_pitch"], dt) if case["residual"] else None
    if kind == "lin_dgrad":
        s["pre"] = _normal(gen, rows, k, case["x_pitch"], bf) if case["act"] != "none" else None
        s["add"] = _normal(gen, rows, k, case["x_pitch"], dt) if case["residual"] else None


def _stats_of(v, kind):
    """(mean, 1 / width) of each row, as the forward leaves them."""
    rows = v.shape[0]
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    for i in range(0, rows, 1 << 14):
        t = v[i:i + (1 << 14)].double()
        m = t.mean(1, keepdim=True) if kind == "layer" else 0.0
        if kind != "none":
            rstd[i:i + (1 << 14)] = ((t - m).square().mean(1) + NORM_EPS).rsqrt().float()
        if kind == "layer":
            mean[i:i + (1 << 14)] = m[:, 0].float()
    return mean, rstd


def _prepare_rn(s, gen):
    case = s["case"]
    rows, c = case["rows"], case["c"]
    dt, fdt = _TYPES[case["dtype"]], _TYPES[case["f_dtype"]]
    stream = _normal(gen, rows, c, 0, dt)
    stream *= 1.5
    stream += (0.5 * torch.randn(c, device="cuda", generator=gen)).to(dt)  # channels of different means
    s["f"] = _normal(gen, rows, c, 0, fdt)
    vec = lambda mean, width, *lead: mean + width * torch.randn(*lead, c, device="cuda", generator=gen)  # noqa: E731
    s["post_gamma"] = vec(1.0, 0.3) if case["post"] != "none" else None
    s["post_beta"] = vec(0.0, 0.3) if case["post"] == "layer" else None
    s["gate"] = {"none": lambda: None, "shared": lambda: vec(0.5, 0.3), "sample": lambda: vec(0.5, 0.3, case["samples"])}[case["gate"]]()
    lead = (case["samples"],) if case["modulated"] else ()
    s["pre_gamma"] = vec(1.0, 0.3, *lead) if case["pre"] != "none" else None
    s["pre_beta"] = vec(0.0, 0.3, *lead) if case["pre"] == "layer" else None
    if case["kind"] == "rn_fwd":
        s["x"] = stream
        return
    s["r"] = stream
    s["dr"] = _normal(gen, rows, c, 0, dt)
    s["dh"] = _normal(gen, rows, c, 0, fdt) if case["pre"] != "none" else None
    # the forward's statistics, which the backward is given
    s["stats"] = torch.stack(_stats_of(s["f"], case["post"]) + _stats_of(s["r"], case["pre"]), 1)


def _flat(s, name, matrices=False):
    """The optimizer's tensors of one kind in one buffer, each beginning at a multiple of 64 values."""
    dt, offset = torch.bfloat16 if matrices else torch.float32, 0
    places = []
    for shape in _shapes(s["case"]):
        places.append(None if matrices and len(shape) < 2 else offset)
        offset += 0 if places[-1] is None else -(-math.prod(shape) // 64) * 64
    s[name] = torch.zeros(offset, device="cuda", dtype=dt)
    for p, shape, at in zip(s["list"], _shapes(s["case"]), places):
        p[name] = None if at is None else s[name][at:at + math.prod(shape)].view(shape)


def _prepare_list(s, gen):
    case = s["case"]
    s["list"] = []
    for i, shape in enumerate(_shapes(case)):
        dt = torch.bfloat16 if case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 2) else torch.float32
        g = torch.empty(shape, device="cuda", dtype=dt).normal_(generator=gen)
        g *= 10.0 ** (-1 - i % 4)  # layers' gradients differ by orders of magnitude
        s["list"].append({"g": g})
    if case["kind"] == "adam":
        for name in ("w", "m", "v", "w16"):
            _flat(s, name, name == "w16")
        for p in s["list"]:
            p["w"].normal_(0, 0.05, generator=gen)
            p["m"].normal_(0, 1e-3, generator=gen)
            p["v"].uniform_(0, 1e-6, generator=gen)
            if p["w16"] is not None:
                p["w16"].copy_(p["w"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    {"lin": _prepare_lin, "rn_": _prepare_rn}.get(case["kind"][:3], _prepare_list)(s, gen)
    return s


# --------------------------------------------------------------------------------------------------------------- plain forms
def _act(z, case):
    if case["act"] == "gelu":
        return z * torch.sigmoid(2 * GELU_A * (z + GELU_B * z * z * z))
    if case["act"] == "silu":
        return z * torch.sigmoid(z)
    return torch.where(z > 0, z, case["slope"] * z) if case["act"] == "lrelu" else z


def _act_grad(z, case):
    if case["act"] == "gelu":
        e = torch.sigmoid(2 * GELU_A * (z + GELU_B * z * z * z))
        return e + z * e * (1 - e) * (2 * GELU_A * (1 + 3 * GELU_B * z * z))
    if case["act"] == "silu":
        e = torch.sigmoid(z)
        return e * (1 + z * (1 - e))
    return torch.where(z > 0, 1.0, case["slope"])


def _plain_lin(s):
    case, dt = s["case"], _TYPES[s["case"]["dtype"]]
    if case["kind"] == "lin_fwd":
        z = s["x"].float() @ s["w"].float().T
        if s["bias"] is not None:
            z += s["bias"]
        out = {"y": _act(z, case) * case["scale"]}
        if s["residual"] is not None:
            out["y"] += s["residual"]
        out["y"] = out["y"].to(dt)
        if case["pre"]:
            out["pre"] = z.to(torch.bfloat16)
        return out
    if case["kind"] == "lin_dgrad":
        dx = s["dz"].float() @ s["w"].float() * case["scale"]
        if s["pre"] is not None:
            dx *= _act_grad(s["pre"].float(), case)
        if s["add"] is not None:
            dx += s["add"]
        return {"dx": dx.to(dt)}
    dz = s["dz"].float()
    return {"dw": dz.T @ s["x"].float() * case["scale"], "db": dz.sum(0) * case["scale"]}


def _wide(v, case):
    """A vector, or one for each sample, beside rows."""
    return v if v is None or v.dim() == 1 else v.repeat_interleave(case["rows"] // case["samples"], 0)


def _plain_norm(v, kind, gamma, beta):
    if kind == "none":
        return v, torch.zeros_like(v[:, 0]), torch.ones_like(v[:, 0])
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    t = v - mean[:, None]
    rstd = 1 / torch.sqrt(t.square().mean(1) + NORM_EPS)
    t = t * rstd[:, None] * gamma
    return t + beta if beta is not None else t, mean, rstd


def _plain_rn_fwd(s):
    case = s["case"]
    p, mf, sf = _plain_norm(s["f"].float(), case["post"], s["post_gamma"], s["post_beta"])
    p = p * case["scale"]
    if s["gate"] is not None:
        p = p * _wide(s["gate"], case)
    r = s["x"].float() + p
    h, mr, sr = _plain_norm(r, case["pre"], _wide(s["pre_gamma"], case), _wide(s["pre_beta"], case))
    out = {"r": r.to(s["x"].dtype), "stats": torch.stack((mf, sf, mr, sr), 1)}
    if case["pre"] != "none":
        out["h"] = h.to(s["f"].dtype)
    return out


def _norm_back(u, vh, rstd, kind):
    d = u - vh * (u * vh).mean(1, keepdim=True)
    return rstd[:, None] * (d - u.mean(1, keepdim=True) if kind == "layer" else d)


def _per_sample(t, v, case):
    """Column sums, for each sample where the vector is each sample's."""
    return t.sum(0) if v is None or v.dim() == 1 else t.reshape(case["samples"], -1, t.shape[1]).sum(1)


def _plain_rn_bwd(s):
    case = s["case"]
    mf, sf, mr, sr = s["stats"].unbind(1)
    dr, f, out = s["dr"].float(), s["f"].float(), {}
    if case["pre"] != "none":
        dh = s["dh"].float()
        rh = (s["r"].float() - mr[:, None]) * sr[:, None]
        out["pre_gamma"] = _per_sample(dh * rh, s["pre_gamma"], case)
        if s["pre_beta"] is not None:
            out["pre_beta"] = _per_sample(dh, s["pre_beta"], case)
        dr = dr + _norm_back(dh * _wide(s["pre_gamma"], case), rh, sr, case["pre"])
    fh = (f - mf[:, None]) * sf[:, None]
    p = fh
    if case["post"] != "none":
        p = p * s["post_gamma"]
        if s["post_beta"] is not None:
            p = p + s["post_beta"]
    dp = dr * case["scale"]
    if s["gate"] is not None:
        out["gate"] = _per_sample(dp * p, s["gate"], case)
        dp = dp * _wide(s["gate"], case)
    if case["post"] != "none":
        out["post_gamma"] = (dp * fh).sum(0)
        if s["post_beta"] is not None:
            out["post_beta"] = dp.sum(0)
        dp = _norm_back(dp * s["post_gamma"], fh, sf, case["post"])
    out["dx"], out["df"] = dr.to(s["r"].dtype), dp.to(s["f"].dtype)
    return out


def _plain_factor(s):
    parts = torch.stack([p["g"].float().square().sum() for p in s["list"]])
    norm = torch.sqrt(parts.sum())
    return norm, torch.clamp(s["case"]["max_norm"] / (norm + CLIP_EPS), max=1.0)


def _plain_list(s):
    norm, factor = _plain_factor(s)
    out = {"norm": norm, "factor": factor}
    if s["case"]["kind"] == "adam":
        for p in s["list"]:
            g = p["g"] * factor
            p["m"].mul_(BETA1).add_((1 - BETA1) * g)
            p["v"].mul_(BETA2).add_((1 - BETA2) * g * g)
            step = p["m"] / (1 - BETA1 ** STEP) / (torch.sqrt(p["v"] / (1 - BETA2 ** STEP)) + ADAM_EPS)
            p["w"].mul_(1 - LR * DECAY).sub_(LR * step)
            if p["w16"] is not None:
                p["w16"].copy_(p["w"])
        out.update({name: s[name] for name in ("w", "m", "v", "w16")})
    return out


# ------------------------------------------------------------------------------------------------- the library's entry points
def _like_rows(rows, width, pitch, dtype):
    return torch.empty(rows, pitch or width, device="cuda", dtype=dtype)[:, :width]


def _plan(s):
    """What a program keeps between calls: descriptors, output buffers, the workspace and the stream."""
    from cnn_conv3d_gb300 import cfconv as cf

    case = s["case"]
    kind = case["kind"]
    p = {"cf": cf, "stream": torch.cuda.current_stream().cuda_stream}
    dtypes = {"bf16": cf.CF_DT_BF16, "f32": cf.CF_DT_F32}
    if kind.startswith("lin"):
        act = {"gelu": cf.CF_ACT_GELU, "silu": cf.CF_ACT_SILU}.get(case["act"], cf.CF_ACT_LRELU)
        rows, k, n = case["rows"], case["k"], case["n"]
        p["desc"] = cf.cf_linear_desc(rows, k, n, act, case["slope"], case["scale"], dtypes[case["dtype"]], case["x_pitch"],
                                      case["y_pitch"])
        if kind == "lin_fwd":
            p["y"] = _like_rows(rows, n, case["y_pitch"], _TYPES[case["dtype"]])
            p["pre"] = _like_rows(rows, n, case["y_pitch"], torch.bfloat16) if case["pre"] else None
            op = cf.CF_LINEAR_FWD
        elif kind == "lin_dgrad":
            p["dx"] = _like_rows(rows, k, case["x_pitch"], _TYPES[case["dtype"]])
            op = cf.CF_LINEAR_DGRAD
        else:
            p["dw"] = torch.empty(n, k, device="cuda")
            p["db"] = torch.empty(n, device="cuda")
            op = cf.CF_LINEAR_WGRAD
        size = cf.cf_linear_workspace_size(p["desc"], op)
    elif kind.startswith("rn"):
        norms = {"none": cf.CF_NORM_NONE, "rms": cf.CF_NORM_RMS, "layer": cf.CF_NORM_LAYER}
        per_sample = (cf.CF_PER_SAMPLE_GATE if case["gate"] == "sample" else 0) | (cf.CF_PER_SAMPLE_PRE if case["modulated"] else 0)
        p["desc"] = cf.cf_residual_norm_desc(case["rows"], case["c"], norms[case["post"]], norms[case["pre"]], NORM_EPS, case["scale"],
                                             dtypes[case["dtype"]], dtypes[case["f_dtype"]], per_sample,
                                             case["rows"] // case["samples"])
        names = ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")
        p["weights"] = cf.cf_residual_norm_vectors(*(s[v] for v in names))
        if kind == "rn_fwd":
            p["r"], p["h"] = torch.empty_like(s["x"]), torch.empty_like(s["f"]) if case["pre"] != "none" else None
            p["stats"] = torch.empty(case["rows"], 4, device="cuda")
        else:
            p["dx"], p["df"] = torch.empty_like(s["r"]), torch.empty_like(s["f"])
            p["vec"] = {v: torch.empty_like(s[v]) for v in names if s[v] is not None}
            p["grads"] = cf.cf_residual_norm_vectors(*(p["vec"].get(v) for v in names))
        size = cf.cf_residual_norm_workspace_size(p["desc"]) if kind == "rn_bwd" else 0
    else:
        p["out"] = torch.empty(2, device="cuda")  # the norm and the factor
        if kind == "norm":
            p["list"] = cf.cf_grads([t["g"] for t in s["list"]])
            size = cf.cf_grad_workspace_size(p["list"])
        else:
            p["list"] = cf.cf_adam_params([(t["w"], t["w16"], t["g"], t["m"], t["v"]) for t in s["list"]])
            p["hyper"] = cf.cf_adam_hyper(LR, BETA1, BETA2, ADAM_EPS, DECAY, case["max_norm"], STEP)
            size = cf.cf_clip_adam_workspace_size(p["list"])
    p["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    p["ws_bytes"] = size
    return p


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    cf, case, tail = p["cf"], s["case"], (p["ws"], p["ws_bytes"], p["stream"])
    kind = case["kind"]
    if kind == "lin_fwd":
        cf.cf_linear_fwd(p["desc"], s["x"], s["w"], s["bias"], s["residual"], p["y"], p["pre"], *tail)
        return {"y": p["y"], "pre": p["pre"]} if case["pre"] else {"y": p["y"]}
    if kind == "lin_dgrad":
        cf.cf_linear_dgrad(p["desc"], s["dz"], s["w"], s["pre"], s["add"], p["dx"], *tail)
        return {"dx": p["dx"]}
    if kind == "lin_wgrad":
        cf.cf_linear_wgrad(p["desc"], s["x"], s["dz"], p["dw"], p["db"], 0, *tail)
        return {"dw": p["dw"], "db": p["db"]}
    if kind == "rn_fwd":
        cf.cf_residual_norm_fwd(p["desc"], s["x"], s["f"], p["weights"], p["r"], p["h"], p["stats"], p["stream"])
        out = {"r": p["r"], "stats": p["stats"]}
        if case["pre"] != "none":
            out["h"] = p["h"]
        return out
    if kind == "rn_bwd":
        cf.cf_residual_norm_bwd(p["desc"], s["f"], s["r"], p["weights"], s["stats"], s["dh"], s["dr"], p["dx"], p["df"],
                                p["grads"], *tail)
        return dict(p["vec"], dx=p["dx"], df=p["df"])
    if kind == "norm":
        cf.cf_grad_norm(p["list"], case["max_norm"], p["out"], *tail)
        return {"norm": p["out"][0], "factor": p["out"][1]}
    cf.cf_clip_adam_step(p["list"], p["hyper"], p["out"], *tail)
    return {"norm": p["out"][0], "factor": p["out"][1], "w": s["w"], "m": s["m"], "v": s["v"], "w16": s["w16"]}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind.startswith("lin"):
        return _plain_lin(state)
    if kind.startswith("rn"):
        return _plain_rn_fwd(state) if kind == "rn_fwd" else _plain_rn_bwd(state)
    return _plain_list(state)


# ---------------------------------------------------------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    if kind.startswith("lin"):
        rows, k, n = case["rows"], case["k"], case["n"]
        size = 4 if case["dtype"] == "f32" else 2
        flops = 2.0 * rows * k * n
        if kind == "lin_fwd":
            return {"bytes": 2 * rows * k + 2 * n * k + rows * n * (size * (1 + case["residual"]) + 2 * case["pre"]) + 4 * n, "flops": flops}
        if kind == "lin_dgrad":
            return {"bytes": 2 * rows * n + 2 * n * k + rows * k * (size * (1 + case["residual"]) + 2 * (case["act"] != "none")), "flops": flops}
        return {"bytes": 2 * rows * (k + n) + 4 * n * k + 4 * n, "flops": flops + rows * n}
    if kind.startswith("rn"):
        size = {"bf16": 2, "f32": 4}
        a, b, pre = size[case["dtype"]], size[case["f_dtype"]], case["pre"] != "none"
        full = case["rows"] * case["c"]
        if kind == "rn_fwd":
            return {"bytes": full * (2 * a + b + b * pre) + 16 * case["rows"], "flops": 16 * full}
        return {"bytes": full * (2 * a + a * pre + 2 * b + b * pre) + 16 * case["rows"], "flops": 30 * full}
    count = sum(math.prod(t) for t in _shapes(case))
    if kind == "norm":
        size = {"f32": 4, "bf16": 2, "mixed": 3}[case["dtype"]]
        return {"bytes": size * count, "flops": 2 * count}
    return {"bytes": 28 * count + 2 * sum(math.prod(t) for t in _shapes(case) if len(t) == 2), "flops": 20 * count}


# --------------------------------------------------------------------------------------------------------------------- exact
def _exact_act(z, case):
    if case["act"] == "gelu":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if case["act"] == "silu":
        return z / (1 + torch.exp(-z))
    return torch.maximum(z, case["slope"] * z) if case["act"] == "lrelu" else z


def _exact_lin(case, s):
    """Row blocks in 64 bits; the activation's derivative by differentiating it."""
    rows = case["rows"]
    step = max(1, (1 << 28) // (case["k"] + case["n"]))
    out = {}
    w = s["w"].double() if "w" in s else None
    for i in range(0, rows, step):
        at = slice(i, i + step)
        if case["kind"] == "lin_fwd":
            z = torch.einsum("rk,nk->rn", s["x"][at].double(), w)
            if s["bias"] is not None:
                z = z + s["bias"].double()
            y = case["scale"] * _exact_act(z, case)
            out.setdefault("y", []).append(y if s["residual"] is None else s["residual"][at].double() + y)
            if case["pre"]:
                out.setdefault("pre", []).append(z)
        elif case["kind"] == "lin_dgrad":
            da = torch.einsum("rn,nk->rk", s["dz"][at].double(), w)
            if s["pre"] is not None:
                z = s["pre"][at].double().requires_grad_()
                if case["act"] == "lrelu":  # the slope at 0 itself
                    da = da * ((z > 0).double() + case["slope"] * (z <= 0).double()).detach()
                else:
                    with torch.enable_grad():
                        da = torch.autograd.grad(_exact_act(z, case), z, da)[0]
            dx = case["scale"] * da
            out.setdefault("dx", []).append(dx if s["add"] is None else s["add"][at].double() + dx)
        else:
            dz, x = s["dz"][at].double(), s["x"][at].double()
            for name, part in (("dw", torch.einsum("rn,rk->nk", dz, x)), ("db", torch.einsum("rn->n", dz))):
                out[name] = [out[name][0] + part * case["scale"]] if name in out else [part * case["scale"]]
    return {k: torch.cat(v) if len(v) > 1 else v[0] for k, v in out.items()}


def _exact_rn(case, s):
    """By the definition in 64 bits, sample by sample, row blocks at a time; gradients by differentiating it."""
    back = case["kind"] == "rn_bwd"
    names = [v for v in ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta") if s[v] is not None]
    vec = {v: s[v].double().requires_grad_(back) for v in names}
    per, step = case["rows"] // case["samples"], max(1, (1 << 24) // case["c"])
    got = {}

    def norm(v, kind, gamma, beta):
        if kind == "none":
            return v, torch.zeros(len(v), device="cuda").double(), torch.ones(len(v), device="cuda").double()
        mean = v.sum(1) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, 0])
        c = v - mean[:, None]
        rstd = ((c ** 2).sum(1) / v.shape[1] + NORM_EPS) ** -0.5
        t = c * rstd[:, None] * gamma
        return (t if beta is None else t + beta), mean, rstd

    with torch.set_grad_enabled(back):
        for n in range(case["samples"]):
            mine = lambda v: None if v not in vec else vec[v][n] if vec[v].dim() == 2 else vec[v]  # noqa: E731
            for i in range(n * per, (n + 1) * per, step):
                at = slice(i, min(i + step, (n + 1) * per))
                f = s["f"][at].double().requires_grad_(back)
                p, mf, sf = norm(f, case["post"], mine("post_gamma"), mine("post_beta"))
                p = case["scale"] * (p if mine("gate") is None else mine("gate") * p)
                if back:  # the stream is given; what comes to it goes on to x and to p
                    r = s["r"][at].double().requires_grad_()
                    h, _, _ = norm(r, case["pre"], mine("pre_gamma"), mine("pre_beta"))
                    dr = s["dr"][at].double()
                    if case["pre"] != "none":
                        (h * s["dh"][at].double()).sum().backward()
                        dr = dr + r.grad
                    (p * dr).sum().backward()
                    rows = {"dx": dr, "df": f.grad}
                else:
                    r = s["x"][at].double() + p
                    h, mr, sr = norm(r, case["pre"], mine("pre_gamma"), mine("pre_beta"))
                    rows = {"r": r, "stats": torch.stack((mf, sf, mr, sr), 1)}
                    if case["pre"] != "none":
                        rows["h"] = h
                for k, v in rows.items():
                    got.setdefault(k, []).append(v)
    out = {k: torch.cat(v) for k, v in got.items()}
    if back:
        out.update({v: vec[v].grad for v in names})
    return out


def _exact_list(case, s):
    norm = math.sqrt(math.fsum(float((p["g"].double() ** 2).sum()) for p in s["list"]))
    factor = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    scalar = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"norm": scalar(norm), "factor": scalar(factor)}
    if case["kind"] == "adam":
        out.update({name: s[name].double() for name in ("w", "m", "v")})
        out["w16"] = s["w16"].double()
        at = at16 = 0
        for p in s["list"]:
            g = p["g"].double() * factor
            m = BETA1 * p["m"].double() + (1 - BETA1) * g
            v = BETA2 * p["v"].double() + (1 - BETA2) * g ** 2
            w = p["w"].double() * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)) ** 0.5 + ADAM_EPS)
            size = g.numel()
            for name, t in (("w", w), ("m", m), ("v", v)):
                out[name][at:at + size] = t.reshape(-1)
            at += -(-size // 64) * 64
            if p["w16"] is not None:
                out["w16"][at16:at16 + size] = w.reshape(-1)
                at16 += -(-size // 64) * 64
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"lin": _exact_lin, "rn_": _exact_rn}.get(case["kind"][:3], _exact_list)(case, s)
