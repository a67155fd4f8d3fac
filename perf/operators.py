"""Cases of the group norm and the orthogonalised updates, with their plain forms.

Each case is one pass through one operator as a training step calls it:

  gn_fwd : group norm of a conv output, channels last, with its activation and, in a pooled block, the 2x2x2 max pooling
  gn_bwd : its backward: gradients of the input, of gamma and of beta
  orth   : the Newton-Schulz orthogonalisation of one or several matrices of one shape
  muon   : momentum, orthogonalisation and the decayed update of a list of weight matrices, with their bf16 copies

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and the library's entry points.
"""
import math

import torch

own = False

NS_STEPS, NS_A, NS_B, NS_C, NS_EPS = 5, 3.4445, -4.7750, 2.0315, 1e-7
LR, MOMENTUM, DECAY = 2e-4, 0.95, 0.01
GN_EPS = 1e-5


# --------------------------------------------------------------------------------------------------------------------- cases
def _gn(name, kind, n, dhw, c, groups, pool="none", act="lrelu", slope=0.3, dtype="bf16", pitch=0):
    d, h, w = dhw
    return {"name": name, "kind": kind, "n": n, "d": d, "h": h, "w": w, "c": c, "groups": groups, "pool": pool, "act": act,
            "slope": slope, "dtype": dtype, "pitch": pitch}


def _orth(name, rows, cols, batch=1, dtype="f32"):
    return {"name": name, "kind": "orth", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # the unpooled last block of the seven-conv network: 4^3 voxels a sample, where only the latency counts
        _gn("gn_fwd tail 8x4^3x256", "gn_fwd", 8, (4, 4, 4), 256, 32),
        # a pooled middle block of the five-block stack
        _gn("gn_fwd pool 8x32^3x128", "gn_fwd", 8, (32, 32, 32), 128, 16, pool="max"),
        # the pooled first block of the five-block stack at its full batch: larger than any cache
        _gn("gn_fwd pool 8x128^3x32", "gn_fwd", 8, (128, 128, 128), 32, 8, pool="max"),
        # a cropped volume of odd sizes in 32 bits, its channels a slice of a wider tensor
        _gn("gn_fwd odd f32 3x15x17x13x20", "gn_fwd", 3, (15, 17, 13), 20, 5, act="silu", dtype="f32", pitch=27),
        # the backward of a small unpooled block
        _gn("gn_bwd 2x8^3x128", "gn_bwd", 2, (8, 8, 8), 128, 16, act="silu"),
        # the backward of the pooled second block of the five-block stack
        _gn("gn_bwd pool 8x64^3x64", "gn_bwd", 8, (64, 64, 64), 64, 8, pool="max"),
        # one large sample whose channels are a slice of a concatenation with a skip connection
        _gn("gn_bwd slice 1x96x80x112x48", "gn_bwd", 1, (96, 80, 112), 48, 6, pitch=112),
        # the first filter of the seven-conv network: the smallest matrix that is orthogonalised
        _orth("orth 16x108", 16, 108),
        # tall matrices of odd sizes, gradients in 16 bits
        _orth("orth 3x1511x515 bf16", 1511, 515, batch=3, dtype="bf16"),
        # the first fully connected layer behind a wide feature map: the largest matrix
        _orth("orth 2048x8192", 2048, 8192),
        # the five filters of the five-block stack
        {"name": "muon five-block filters", "kind": "muon", "shapes": "32x108,64x864,128x1728,256x3456,256x6912", "nesterov": True},
        # every matrix of the seven-conv network with its fully connected layers
        {"name": "muon seven-conv network", "kind": "muon", "nesterov": True,
         "shapes": "16x108,32x432,64x864,128x1728,256x3456,256x6912,256x6912,2048x2048,256x2048,4x256"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_gn(rng, kind):
    while True:
        c = rng.choice([_log(rng, 4, 512), 8 * _log(rng, 1, 64), 2 ** rng.randrange(4, 9)])
        groups = rng.choice([g for g in range(1, min(c, 64) + 1) if c % g == 0])
        pool = rng.choice(["none", "max"])
        dtype = "bf16" if pool == "max" else rng.choice(["bf16", "bf16", "f32"])
        # a derivative with a jump is not drawn for the 32-bit gradients: the side a value within rounding of 0 falls on is no error
        act = "lrelu" if pool == "max" else "silu" if dtype == "f32" and kind == "gn_bwd" else rng.choice(["lrelu", "silu"])
        side = _log(rng, 2, 128)
        dhw = [max(1, min(144, int(round(side * rng.uniform(0.6, 1.5))))) for _ in range(3)]
        if pool == "max":
            dhw = [s + s % 2 for s in dhw]
        n = rng.randint(1, 8)
        pitch = 0 if rng.random() < 0.75 else c + rng.choice([8, 64, rng.randint(1, 40)])
        if not 2 ** 10 <= n * dhw[0] * dhw[1] * dhw[2] * c <= 2 ** 27:
            continue
        if dhw[0] * dhw[1] * dhw[2] * c < 32 * groups:  # with two or three values to a group the gradient is rounding alone
            continue
        case = _gn("", kind, n, dhw, c, groups, pool, act, rng.choice([0.3, 0.1, 0.01]), dtype, pitch)
        del case["name"]
        return case


def _draw_orth(rng):
    while True:
        rows, cols, batch = _log(rng, 4, 8192), _log(rng, 4, 8192), rng.choice([1, 1, 2, 3, 5])
        if rng.random() < 0.5:
            rows, cols = max(8, rows // 8 * 8), max(8, cols // 8 * 8)
        k, n = min(rows, cols), max(rows, cols)
        if batch * k * k * n > 2048 * 2048 * 6000 or k < 2:
            continue
        case = _orth("", rows, cols, batch, rng.choice(["f32", "bf16"]))
        del case["name"]
        return case


def _draw_muon(rng):
    while True:
        count = rng.randint(1, 9)
        shapes = []
        for _ in range(count):
            rows = rng.choice([2 ** rng.randrange(4, 11), _log(rng, 2, 1500)])
            cols = rng.choice([27 * 2 ** rng.randrange(2, 9), _log(rng, 4, 6000)])
            shapes.append((rows, cols))
        if sum(min(s) ** 2 * max(s) for s in shapes) <= 2048 ** 3 and sum(r * c for r, c in shapes) <= 2 ** 24:
            return {"kind": "muon", "shapes": ",".join("%dx%d" % s for s in shapes), "nesterov": rng.random() < 0.7}


def draw(rng):
    kind = rng.choice(["gn_fwd", "gn_bwd", "orth", "muon"])
    return _draw_gn(rng, kind) if kind.startswith("gn") else _draw_orth(rng) if kind == "orth" else _draw_muon(rng)


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


# -------------------------------------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _matrix(shape, gen, noise):
    """A gradient as products of few directions with noise: what sums over voxels or samples look like."""
    *lead, rows, cols = shape
    r = min(rows, cols, 16)
    left = torch.randn(*lead, rows, r, device="cuda", generator=gen)
    right = torch.randn(*lead, r, cols, device="cuda", generator=gen)
    return left @ right / r + noise * torch.randn(*shape, device="cuda", generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["kind"].startswith("gn"):
        dt, c = _TYPES[case["dtype"]], case["c"]
        dims = (case["n"], case["d"], case["h"], case["w"])
        # a conv output: channels of different means and widths; in a slice its neighbours are there too
        wide = torch.empty(dims + (case["pitch"] or c,), device="cuda", dtype=dt).normal_(generator=gen)
        x = wide[..., :c]
        x *= torch.rand(c, device="cuda", generator=gen).add_(0.5).to(dt)
        x += torch.randn(c, device="cuda", generator=gen).to(dt)
        s["x"] = x
        s["gamma"] = 1 + 0.3 * torch.randn(c, device="cuda", generator=gen)
        s["beta"] = 0.3 * torch.randn(c, device="cuda", generator=gen)
        if case["kind"] == "gn_bwd":
            p = 2 if case["pool"] == "max" else 1
            out = (dims[0], dims[1] // p, dims[2] // p, dims[3] // p, c)
            s["dy"] = torch.empty(out, device="cuda", dtype=dt).normal_(generator=gen)
            # the forward's statistics, which the backward is given
            x5 = x.reshape(dims[0], -1, case["groups"], c // case["groups"])
            mean = x5.mean((1, 3), dtype=torch.float32)
            var = torch.stack([(x5[i].float() - mean[i, None, :, None]).square_().mean((0, 2)) for i in range(dims[0])])
            s["mean"], s["rstd"] = mean, (var + GN_EPS).rsqrt()
    elif case["kind"] == "orth":
        s["g"] = _matrix((case["batch"], case["rows"], case["cols"]), gen, 0.1).mul_(1e-3).to(_TYPES[case["dtype"]])
    else:
        s["params"] = []
        for shape in _shapes(case):
            w = torch.randn(shape, device="cuda", generator=gen) * math.sqrt(2.0 / shape[1])
            g = _matrix(shape, gen, 0.1) * 1e-3
            m = _matrix(shape, gen, 0.1) * 1e-2
            s["params"].append({"w": w, "g": g, "m": m, "w16": w.to(torch.bfloat16), "scale": 0.2 * math.sqrt(max(shape))})
    return s


# --------------------------------------------------------------------------------------------------------------- plain forms
def _windows(t):
    """[n, d, h, w, c] as [n, d/2, h/2, w/2, 8, c], the voxels of a window in (dd, dh, dw) order."""
    n, d, h, w, c = t.shape
    return t.reshape(n, d // 2, 2, h // 2, 2, w // 2, 2, c).permute(0, 1, 3, 5, 2, 4, 6, 7).reshape(n, d // 2, h // 2, w // 2, 8, c)


def _unwindows(t):
    n, d, h, w, _, c = t.shape
    return t.reshape(n, d, h, w, 2, 2, 2, c).permute(0, 1, 4, 2, 5, 3, 6, 7).reshape(n, 2 * d, 2 * h, 2 * w, c)


def _act(u, case):
    return u * torch.sigmoid(u) if case["act"] == "silu" else torch.where(u > 0, u, case["slope"] * u)


def _act_grad(u, case):
    if case["act"] == "silu":
        e = torch.sigmoid(u)
        return e * (1 + u * (1 - e))
    return torch.where(u > 0, 1.0, case["slope"])


def _affine(s, mean, rstd):
    """a, b of u = a x + b, as [n, 1, 1, 1, c]."""
    case = s["case"]
    per = case["c"] // case["groups"]
    a = s["gamma"] * rstd.repeat_interleave(per, 1)
    b = s["beta"] - mean.repeat_interleave(per, 1) * a
    return a[:, None, None, None, :], b[:, None, None, None, :]


def _plain_gn_fwd(s):
    case, x = s["case"], s["x"].float()
    n, c, G = case["n"], case["c"], case["groups"]
    xg = x.reshape(n, -1, G, c // G)
    mean = xg.mean((1, 3))
    var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = 1 / torch.sqrt(var + GN_EPS)
    a, b = _affine(s, mean, rstd)
    u = x * a + b
    if case["pool"] == "max":
        d, h, w = case["d"] // 2, case["h"] // 2, case["w"] // 2
        u = u.reshape(n, d, 2, h, 2, w, 2, c).amax((2, 4, 6))
    return {"y": _act(u, case).to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_gn_bwd(s):
    case, x, dy = s["case"], s["x"].float(), s["dy"].float()
    n, c, G = case["n"], case["c"], case["groups"]
    per = c // G
    mean, rstd = s["mean"], s["rstd"]
    a, b = _affine(s, mean, rstd)
    u = x * a + b
    if case["pool"] == "max":
        win = _windows(u)
        m = win.amax(4, keepdim=True)
        hit = win == m
        first = hit & (hit.cumsum(4, dtype=torch.int8) == 1)
        du = _unwindows(torch.where(first, (dy[..., None, :] * _act_grad(m, case)), 0.0))
        del win, m, hit, first
    else:
        du = dy * _act_grad(u, case)
    del u
    shape = (n, 1, 1, 1, c)
    wide = lambda t: t.repeat_interleave(per, 1).reshape(shape)  # noqa: E731
    xh = (x - wide(mean)) * wide(rstd)
    dbeta, dgamma = du.sum((1, 2, 3)), (du * xh).sum((1, 2, 3))  # [n, c]
    count = case["d"] * case["h"] * case["w"] * per
    s1 = (dbeta * s["gamma"]).reshape(n, G, per).sum(2) / count
    s2 = (dgamma * s["gamma"]).reshape(n, G, per).sum(2) / count
    dx = wide(rstd) * (du * s["gamma"] - wide(s1) - xh * wide(s2))
    return {"dx": dx.to(s["x"].dtype), "dgamma": dgamma.sum(0), "dbeta": dbeta.sum(0)}


def _plain_ns(u):
    """Newton-Schulz products of [..., rows, cols] in 32 bits."""
    tall = u.shape[-2] > u.shape[-1]
    x = u.transpose(-1, -2) if tall else u
    x = x / (torch.sqrt(x.square().sum((-1, -2), keepdim=True)) + NS_EPS)
    for _ in range(NS_STEPS):
        a = x @ x.transpose(-1, -2)
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.transpose(-1, -2) if tall else x


def _plain_muon(s):
    for p in s["params"]:
        p["m"].mul_(MOMENTUM).add_(p["g"])
        u = p["g"] + MOMENTUM * p["m"] if s["case"]["nesterov"] else p["m"]
        p["w"].mul_(1 - LR * DECAY).sub_(LR * p["scale"] * _plain_ns(u))
        p["w16"].copy_(p["w"])
    return [[p["w"], p["m"], p["w16"]] for p in s["params"]]


# ------------------------------------------------------------------------------------------------- the library's entry points
def _plan(s):
    """What a program keeps between calls: descriptors, output buffers, the workspace and the stream."""
    from cnn_conv3d_gb300 import cfconv as cf

    case = s["case"]
    p = {"cf": cf, "stream": torch.cuda.current_stream().cuda_stream}
    if case["kind"].startswith("gn"):
        x, c = s["x"], case["c"]
        pool = cf.CF_POOL_MAX if case["pool"] == "max" else cf.CF_POOL_NONE
        act = cf.CF_ACT_SILU if case["act"] == "silu" else cf.CF_ACT_LRELU
        dtype = cf.CF_DT_F32 if case["dtype"] == "f32" else cf.CF_DT_BF16
        p["desc"] = cf.cf_gn_desc(case["n"], case["d"], case["h"], case["w"], c, case["groups"], pool, act, case["slope"], GN_EPS,
                                  dtype, case["pitch"], 0)
        back = case["kind"] == "gn_bwd"
        if back:
            p["dx"] = torch.empty_like(x) if not case["pitch"] else x.new_empty(x.shape[:-1] + (case["pitch"],))[..., :c]
            p["dgamma"], p["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
        else:
            q = 2 if case["pool"] == "max" else 1
            p["y"] = x.new_empty((case["n"], case["d"] // q, case["h"] // q, case["w"] // q, c))
            p["mean"] = torch.empty((case["n"], case["groups"]), device="cuda")
            p["rstd"] = torch.empty_like(p["mean"])
        size = cf.cf_group_norm_workspace_size(p["desc"], back)
    elif case["kind"] == "orth":
        dtype = cf.CF_DT_F32 if case["dtype"] == "f32" else cf.CF_DT_BF16
        p["desc"] = cf.cf_ns_desc(case["batch"], case["rows"], case["cols"], dtype, NS_STEPS, NS_A, NS_B, NS_C, NS_EPS)
        p["o"] = torch.empty(s["g"].shape, dtype=torch.bfloat16, device="cuda")
        size = cf.cf_orthogonalize_workspace_size(p["desc"])
    else:
        p["params"] = cf.cf_muon_params([(t["w"], t["w16"], t["g"], t["m"], t["scale"]) for t in s["params"]])
        p["hyper"] = cf.cf_muon_hyper(LR, MOMENTUM, DECAY, int(case["nesterov"]), NS_STEPS, NS_A, NS_B, NS_C, NS_EPS)
        size = cf.cf_muon_workspace_size(p["params"])
    p["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    p["ws_bytes"] = size
    return p


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    cf, kind = p["cf"], s["case"]["kind"]
    if kind == "gn_fwd":
        cf.cf_group_norm_fwd(p["desc"], s["x"], s["gamma"], s["beta"], p["y"], p["mean"], p["rstd"], p["ws"], p["ws_bytes"], p["stream"])
        return {"y": p["y"], "mean": p["mean"], "rstd": p["rstd"]}
    if kind == "gn_bwd":
        cf.cf_group_norm_bwd(p["desc"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], s["dy"], p["dx"], p["dgamma"], p["dbeta"],
                             p["ws"], p["ws_bytes"], p["stream"])
        return {"dx": p["dx"], "dgamma": p["dgamma"], "dbeta": p["dbeta"]}
    if kind == "orth":
        cf.cf_orthogonalize(p["desc"], s["g"], p["o"], p["ws"], p["ws_bytes"], p["stream"])
        return {"o": p["o"]}
    cf.cf_muon_step(p["params"], p["hyper"], p["ws"], p["ws_bytes"], p["stream"])
    return [[t["w"], t["m"], t["w16"]] for t in s["params"]]


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "gn_fwd":
        return _plain_gn_fwd(state)
    if kind == "gn_bwd":
        return _plain_gn_bwd(state)
    if kind == "orth":
        return {"o": _plain_ns(state["g"].float()).to(torch.bfloat16)}
    return _plain_muon(state)


# ---------------------------------------------------------------------------------------------------------------------- work
def _ns_flops(rows, cols):
    """The symmetric products counted once for each pair: k^2 n for X X^T, k^3 for its square, 2 k^2 n for B X, a step."""
    k, n = min(rows, cols), max(rows, cols)
    return NS_STEPS * (3.0 * k * k * n + 1.0 * k * k * k)


def work(case):
    if case["kind"].startswith("gn"):
        size = 4 if case["dtype"] == "f32" else 2
        full = case["n"] * case["d"] * case["h"] * case["w"] * case["c"]
        out = full // 8 if case["pool"] == "max" else full
        back = case["kind"] == "gn_bwd"
        return {"bytes": size * (full + out + (full if back else 0)) + 16 * case["c"], "flops": full * (20 if back else 9)}
    if case["kind"] == "orth":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["batch"] * case["rows"] * case["cols"] * (size + 2), "flops": case["batch"] * _ns_flops(case["rows"], case["cols"])}
    shapes = _shapes(case)
    return {"bytes": sum(22 * r * c for r, c in shapes), "flops": sum(_ns_flops(r, c) for r, c in shapes)}


# --------------------------------------------------------------------------------------------------------------------- exact
def _exact_gn(case, s):
    """By the definition in 64 bits, sample by sample; gradients by differentiating it, given the statistics' definition."""
    n, c, G = case["n"], case["c"], case["groups"]
    back = case["kind"] == "gn_bwd"
    gamma = s["gamma"].double().requires_grad_(back)
    beta = s["beta"].double().requires_grad_(back)
    got = {k: [] for k in (("dx",) if back else ("y", "mean", "rstd"))}
    with torch.set_grad_enabled(back):
        for i in range(n):
            x = s["x"][i].double().requires_grad_(back)
            v = x.reshape(-1, G, c // G)
            mean = v.sum((0, 2), keepdim=True) / (v.shape[0] * v.shape[2])
            centred = v - mean
            var = (centred ** 2).sum((0, 2), keepdim=True) / (v.shape[0] * v.shape[2])
            u = (centred / (var + GN_EPS) ** 0.5).reshape(x.shape) * gamma + beta
            if case["pool"] == "max":
                win = _windows(u[None])[0]
                with torch.no_grad():  # the first maximum: the highest of 8, 7, ... 1 among the equal ones
                    order = torch.arange(8, 0, -1, device="cuda", dtype=torch.int8)[:, None]
                    at = ((win == win.amax(3, keepdim=True)) * order).argmax(3, keepdim=True)
                u = torch.gather(win, 3, at).squeeze(3)
            y = torch.nn.functional.silu(u) if case["act"] == "silu" else torch.maximum(u, case["slope"] * u)
            if back:
                (y * s["dy"][i].double()).sum().backward()
                got["dx"].append(x.grad)
            else:
                got["y"].append(y)
                got["mean"].append(mean.reshape(G))
                got["rstd"].append(((var + GN_EPS) ** -0.5).reshape(G))
            del x, v, centred, u, y
    out = {k: torch.stack(v) for k, v in got.items()}
    if back:
        out["dgamma"], out["dbeta"] = gamma.grad, beta.grad
    return out


def _exact_ns(u):
    """From the singular values: X = U p(p(...p(S))) V^T with p(t) = a t + b t^3 + c t^5, S scaled by the Frobenius norm.  The values and
    the factors come from the eigenvectors of the smaller Gram matrix."""
    if u.shape[-2] > u.shape[-1]:
        return _exact_ns(u.mT).mT
    x = u / (torch.linalg.vector_norm(u, dim=(-1, -2), keepdim=True) + NS_EPS)
    lam, vec = torch.linalg.eigh(x @ x.mT)
    t, ratio = lam.clamp_min(0), torch.ones_like(lam)  # squared singular values; output over input of each
    for _ in range(NS_STEPS):
        f = NS_A + NS_B * t + NS_C * t * t
        ratio, t = ratio * f, t * f * f
    return (vec * ratio[..., None, :]) @ (vec.mT @ x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("gn"):
        return _exact_gn(case, s)
    if case["kind"] == "orth":
        return {"o": _exact_ns(s["g"].double())}
    out = []
    for p in s["params"]:
        g, m = p["g"].double(), p["m"].double() * MOMENTUM + p["g"].double()
        o = _exact_ns(g + MOMENTUM * m if case["nesterov"] else m)
        w = p["w"].double() * (1 - LR * DECAY) - LR * p["scale"] * o
        out.append([w, m, w])
    return out
