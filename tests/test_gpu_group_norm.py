"""Group norm with the block's activation and pooling, forward and backward, through the C ABI against the 64-bit oracle.

Tolerances, per element, from the arithmetic (eps24 = 2^-24, the fp32 unit roundoff; a bf16 store rounds by at most 2^-9 of
the value, taken twice as large):
  mean     2^-17 of the mean of |x| (sums of fp32 partials of at most a few hundred terms: 2^7 eps24)
  rstd     2^-17 relative, plus what a wrong mean adds: (mean error * rstd)^2
  u        2^-16 (|a x| + |mean a| + |beta|): the statistics' errors and three roundings
  y        2^-8 |y| for bf16 (2^-22 for fp32) plus the error of u (the activations' slopes are at most 1.1)
  dgamma, dbeta   2^-15 of the sum of their terms' magnitudes
  dx       2^-8 |dx| (bf16) plus 2^-14 of the sum of the magnitudes it is made of
Where u is within its error of 0, LReLU' may be either of its values; where two voxels of a window are, the gradient may go
to either: such places widen the tolerance by what they could move, and are few."""
import numpy as np
import pytest

from tests.gpu_util import guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cf():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def _desc(cf, shape, groups, pool, act, slope, eps, dtype, xp=0, yp=0):
    n, d, h, w, c = shape
    return cf.cf_gn_desc(n, d, h, w, c, groups, {"none": cf.CF_POOL_NONE, "max": cf.CF_POOL_MAX, "avg": cf.CF_POOL_AVG}[pool],
                         {"lrelu": cf.CF_ACT_LRELU, "silu": cf.CF_ACT_SILU}[act], slope, eps,
                         {"bf16": cf.CF_DT_BF16, "f32": cf.CF_DT_F32}[dtype], xp, yp)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _pitched(t, pitch):
    """The values of t in voxels `pitch` values apart; the values between are NaN."""
    import torch
    if not pitch:
        return t
    wide = torch.full(t.shape[:-1] + (pitch,), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _inputs(shape, pool, dtype, seed, offset=0.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    c = shape[-1]
    x = torch.randn(shape, device="cuda", generator=gen) * (0.5 + torch.rand(c, device="cuda", generator=gen))
    x = (x + torch.randn(c, device="cuda", generator=gen) + offset).to(dt)
    gamma = 1 + 0.4 * torch.randn(c, device="cuda", generator=gen)
    gamma[::5] *= -1
    beta = 0.4 * torch.randn(c, device="cuda", generator=gen)
    q = 1 if pool == "none" else 2
    out = (shape[0], shape[1] // q, shape[2] // q, shape[3] // q, c)
    dy = torch.randn(out, device="cuda", generator=gen).to(dt)
    return x, gamma, beta, dy


def _run_fwd(cf, shape, groups, pool, act, slope, eps, dtype, x, gamma, beta, xp=0, yp=0, stats=True, stream=None):
    import torch
    desc = _desc(cf, shape, groups, pool, act, slope, eps, dtype, xp, yp)
    q = 1 if pool == "none" else 2
    out = (shape[0], shape[1] // q, shape[2] // q, shape[3] // q, yp or shape[-1])
    y, check = guarded(out, x.dtype, fill=7.0)
    mean = torch.empty((shape[0], groups), device="cuda") if stats else None
    rstd = torch.empty_like(mean) if stats else None
    size = cf.cf_group_norm_workspace_size(desc, 0)
    ws, check_ws = guarded((max(size, 16),), torch.uint8, fill=0xEE)
    cf.cf_group_norm_fwd(desc, _pitched(x, xp), gamma, beta, y, mean, rstd, ws, size, stream)
    torch.cuda.synchronize()
    check("y")
    check_ws("workspace")
    if yp:
        assert bool((y[..., shape[-1]:] == 7.0).all()), "values between the voxels of y changed"
    assert cf.cf_last_device_status() == cf.CF_OK
    return y[..., :shape[-1]], mean, rstd


def _run_bwd(cf, shape, groups, pool, act, slope, eps, dtype, x, gamma, beta, mean, rstd, dy, xp=0, yp=0):
    import torch
    desc = _desc(cf, shape, groups, pool, act, slope, eps, dtype, xp, yp)
    dx, check = guarded(shape[:-1] + (xp or shape[-1],), x.dtype, fill=7.0)
    dgamma, check_g = guarded((shape[-1],), torch.float32)
    dbeta, check_b = guarded((shape[-1],), torch.float32)
    size = cf.cf_group_norm_workspace_size(desc, 1)
    ws, check_ws = guarded((max(size, 16),), torch.uint8, fill=0xEE)
    cf.cf_group_norm_bwd(desc, _pitched(x, xp), gamma, beta, mean, rstd, _pitched(dy, yp), dx, dgamma, dbeta, ws, size)
    torch.cuda.synchronize()
    for c, what in ((check, "dx"), (check_g, "dgamma"), (check_b, "dbeta"), (check_ws, "workspace")):
        c(what)
    if xp:
        assert bool((dx[..., shape[-1]:] == 7.0).all()), "values between the voxels of dx changed"
    assert cf.cf_last_device_status() == cf.CF_OK
    return dx[..., :shape[-1]], dgamma, dbeta


def _u_error(oracle, x, gamma, beta, mean, rstd):
    c = x.shape[-1]
    a = np.abs(gamma) * oracle._per_channel(rstd, c)
    return 2.0 ** -16 * (a * np.abs(x) + a * np.abs(oracle._per_channel(mean, c)) + np.abs(beta)) + 1e-30


def check_forward(cf, oracle, shape, groups, pool="none", act="lrelu", slope=0.3, eps=1e-5, dtype="bf16", xp=0, yp=0, seed=0,
                  offset=0.0, affine=True):
    x, gamma, beta, _ = _inputs(shape, pool, dtype, seed, offset)
    y, mean, rstd = _run_fwd(cf, shape, groups, pool, act, slope, eps, dtype, x, gamma if affine else None,
                             beta if affine else None, xp, yp)
    X = _f64(x)
    G, B = (_f64(gamma), _f64(beta)) if affine else (np.ones(shape[-1]), np.zeros(shape[-1]))
    ref, rm, rr = oracle.group_norm_fwd(X, G, B, groups, pool, act, slope, eps)
    mabs = np.abs(X).reshape(shape[0], -1, groups, shape[-1] // groups).mean(axis=(1, 3))
    merr = np.abs(_f64(mean) - rm)
    assert np.all(merr <= 2.0 ** -17 * mabs + 1e-30), merr.max()
    assert np.all(np.abs(_f64(rstd) - rr) <= rr * (2.0 ** -17 + (2.0 ** -17 * mabs * rr) ** 2)), np.max(np.abs(_f64(rstd) / rr - 1))
    ue = _u_error(oracle, X, G, B, rm, rr)
    ue = oracle._to_windows(ue).max(axis=4) if pool != "none" else ue
    tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22) * np.abs(ref) + 1.1 * ue
    err = np.abs(_f64(y) - ref)
    assert np.all(err <= tol), (err.max(), np.max(err / tol))
    return x, gamma, beta, mean, rstd, y


def check_backward(cf, oracle, shape, groups, pool="none", act="lrelu", slope=0.3, eps=1e-5, dtype="bf16", xp=0, yp=0, seed=0,
                   offset=0.0, affine=True):
    import torch
    x, gamma, beta, dy = _inputs(shape, pool, dtype, seed, offset)
    X, G, B, DY = _f64(x), _f64(gamma), _f64(beta), _f64(dy)
    if not affine:
        G, B = np.ones(shape[-1]), np.zeros(shape[-1])
    mean, rstd = (s.astype(np.float32) for s in oracle.group_norm_stats(X, groups, eps))
    tm, tr = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    dx, dgamma, dbeta = _run_bwd(cf, shape, groups, pool, act, slope, eps, dtype, x, gamma if affine else None,
                                 beta if affine else None, tm, tr, dy, xp, yp)
    stats = (mean.astype(np.float64), rstd.astype(np.float64))
    n, c = shape[0], shape[-1]
    rdx, rdg, rdb = oracle.group_norm_bwd(X, G, B, groups, DY, pool, act, slope, eps, stats)
    u, xh = oracle.group_norm_pre(X, G, B, *stats)
    du = oracle.group_norm_du(u, DY, pool, act, slope)
    ue = _u_error(oracle, X, G, B, *stats)
    # what an ambiguous derivative or maximum could move, per element of du
    if pool == "max":
        win, we = oracle._to_windows(u), oracle._to_windows(ue)
        top = np.sort(win, axis=4)
        xw = oracle._to_windows(X)
        first = np.argmax(win, axis=4)[..., None, :]
        xtop = np.take_along_axis(xw, first, 4)
        # equal x are equal u for the kernel too: only values that differ may be ordered either way
        near = (win >= top[..., -1:, :] - 2 * we) & (xw != xtop)
        edge = np.abs(top[..., -1, :]) <= we.max(axis=4)
        amb = np.where(near | (near.any(axis=4, keepdims=True) & (np.arange(8)[:, None] == first)), np.abs(DY)[..., None, :], 0.0)
        amb = amb + np.where(np.arange(8)[:, None] == first, (edge * np.abs(DY))[..., None, :], 0.0)
        amb = oracle._from_windows(amb)
    elif act == "lrelu":
        full = oracle._from_windows(np.repeat(np.abs(DY)[..., None, :], 8, axis=4)) / 8 if pool == "avg" else np.abs(DY)
        amb = np.where(np.abs(u) <= ue, full * abs(1 - slope), 0.0)
    else:
        amb = np.zeros_like(u)
    assert np.count_nonzero(amb) <= 1e-3 * amb.size + 8
    axes = (0, 1, 2, 3)
    tol_b = 2.0 ** -15 * np.abs(du).sum(axis=axes) + amb.sum(axis=axes) + 1e-30
    tol_g = 2.0 ** -15 * np.abs(du * xh).sum(axis=axes) + (amb * np.abs(xh)).sum(axis=axes) + 2.0 ** -15 * np.abs(du).sum(axis=axes)
    assert np.all(np.abs(_f64(dbeta) - rdb) <= tol_b), np.max(np.abs(_f64(dbeta) - rdb) / tol_b)
    assert np.all(np.abs(_f64(dgamma) - rdg) <= tol_g), np.max(np.abs(_f64(dgamma) - rdg) / tol_g)

    def gm(t):
        return oracle._per_channel(t.reshape(n, -1, groups, c // groups).mean(axis=(1, 3)), c)

    r = oracle._per_channel(stats[1], c)
    g = np.abs(G)
    parts = r * (g * np.abs(du) + gm(g * np.abs(du)) + np.abs(xh) * gm(g * np.abs(du * xh)))
    # xh is formed from fp32 x - mean: an error of its own where |mean| is large against the deviation
    parts = parts * (1 + np.abs(oracle._per_channel(stats[0], c)) * r)
    moved = r * (g * amb + gm(g * amb) + np.abs(xh) * gm(g * amb * np.abs(xh)))
    tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22) * np.abs(rdx) + 2.0 ** -14 * parts + 1.01 * moved
    err = np.abs(_f64(dx) - rdx)
    assert np.all(err <= tol), (err.max(), np.max(err / tol))


SHAPES = [
    # one voxel; one channel; a group per channel; one group; channels that fill no vector; more than a block's channels
    ((1, 1, 1, 1, 8), 1), ((2, 1, 1, 1, 64), 4), ((3, 1, 1, 1, 4), 4), ((1, 3, 5, 7, 1), 1), ((2, 3, 4, 5, 6), 3),
    ((2, 5, 3, 3, 12), 2), ((1, 7, 5, 3, 13), 13), ((2, 4, 4, 4, 20), 5), ((1, 2, 3, 2, 433), 1), ((1, 3, 2, 2, 520), 8),
    ((2, 6, 5, 4, 96), 6), ((5, 4, 6, 2, 32), 32), ((1, 9, 11, 13, 16), 2), ((2, 16, 16, 16, 64), 8), ((1, 33, 31, 29, 24), 3),
    ((9, 4, 4, 4, 256), 32), ((1, 2, 2, 2, 2056), 257), ((1, 17, 16, 15, 48), 1),
]
POOLED = [((1, 2, 2, 2, 8), 2), ((2, 4, 2, 6, 5), 5), ((2, 8, 6, 4, 32), 4), ((3, 2, 10, 4, 20), 2), ((1, 16, 16, 16, 64), 8),
          ((1, 14, 10, 22, 16), 16), ((2, 4, 4, 4, 264), 3), ((1, 32, 34, 30, 24), 3), ((4, 4, 4, 4, 433), 1)]


@pytest.mark.parametrize("shape,groups", SHAPES)
@pytest.mark.parametrize("act,dtype", [("lrelu", "bf16"), ("silu", "bf16"), ("silu", "f32")])
def test_forward(cf, oracle_mod, shape, groups, act, dtype):
    check_forward(cf, oracle_mod, shape, groups, act=act, dtype=dtype, seed=11)


@pytest.mark.parametrize("shape,groups", SHAPES)
@pytest.mark.parametrize("act,dtype", [("lrelu", "bf16"), ("silu", "bf16"), ("silu", "f32"), ("lrelu", "f32")])
def test_backward(cf, oracle_mod, shape, groups, act, dtype):
    check_backward(cf, oracle_mod, shape, groups, act=act, dtype=dtype, seed=12)


@pytest.mark.parametrize("shape,groups", POOLED)
@pytest.mark.parametrize("pool,act", [("max", "lrelu"), ("avg", "lrelu"), ("avg", "silu")])
def test_pooled(cf, oracle_mod, shape, groups, pool, act):
    check_forward(cf, oracle_mod, shape, groups, pool=pool, act=act, seed=13)
    check_backward(cf, oracle_mod, shape, groups, pool=pool, act=act, seed=14)


@pytest.mark.parametrize("c,xp,yp", [(16, 24, 40), (16, 16, 24), (16, 19, 0), (6, 11, 9), (20, 0, 21), (32, 160, 0), (12, 16, 20)])
@pytest.mark.parametrize("pool,dtype", [("none", "bf16"), ("none", "f32"), ("max", "bf16")])
def test_pitches(cf, oracle_mod, c, xp, yp, pool, dtype):
    shape = (2, 6, 4, 10, c)
    check_forward(cf, oracle_mod, shape, 2, pool=pool, dtype=dtype, xp=xp, yp=yp, seed=15)
    check_backward(cf, oracle_mod, shape, 2, pool=pool, dtype=dtype, act="lrelu" if pool == "max" else "silu", xp=xp, yp=yp, seed=16)


def test_slopes_and_missing_affine(cf, oracle_mod):
    for slope in (0.0, 0.01, 1.0):
        check_forward(cf, oracle_mod, (2, 4, 6, 8, 16), 4, pool="max", slope=slope, seed=17)
        check_backward(cf, oracle_mod, (2, 4, 6, 8, 16), 4, pool="max", slope=slope, seed=18)
    for pool in ("none", "max"):
        check_forward(cf, oracle_mod, (2, 4, 6, 8, 16), 4, pool=pool, affine=False, seed=19)
        check_backward(cf, oracle_mod, (2, 4, 6, 8, 16), 4, pool=pool, affine=False, seed=20)
    check_forward(cf, oracle_mod, (2, 5, 6, 7, 16), 2, slope=-0.5, seed=21)


def test_mean_far_from_zero(cf, oracle_mod):
    """Deviations of about 1 around 1000: the variance is not a difference of large sums."""
    check_forward(cf, oracle_mod, (2, 9, 10, 11, 24), 3, act="silu", dtype="f32", offset=1000.0, seed=22)
    check_backward(cf, oracle_mod, (2, 9, 10, 11, 24), 3, act="silu", dtype="f32", offset=1000.0, seed=23)


def test_outliers_first(cf, oracle_mod):
    """The first voxels of a sample a thousand times as large as the rest."""
    import torch
    shape, groups = (1, 16, 16, 16, 32), 4
    x, gamma, beta, _ = _inputs(shape, "none", "f32", 24)
    x.view(-1, 32)[:64] *= 1000.0
    y, mean, rstd = _run_fwd(cf, shape, groups, "none", "silu", 0.3, 1e-5, "f32", x, gamma, beta)
    rm, rr = oracle_mod.group_norm_stats(_f64(x), groups)
    mabs = np.abs(_f64(x)).reshape(1, -1, groups, 8).mean(axis=(1, 3))
    assert np.all(np.abs(_f64(mean) - rm) <= 2.0 ** -17 * mabs)
    assert np.all(np.abs(_f64(rstd) / rr - 1) <= 2.0 ** -16)


def test_constant_input(cf):
    import torch
    shape = (2, 4, 4, 4, 16)
    for dtype, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        x = torch.full(shape, 3.140625, device="cuda", dtype=dt)
        beta = torch.linspace(-1, 1, 16, device="cuda")
        y, mean, rstd = _run_fwd(cf, shape, 4, "none", "lrelu", 1.0, 1e-5, dtype, x, None, beta)
        assert torch.all((mean - 3.140625).abs() <= 1e-6) and torch.all((rstd * 1e-5 ** 0.5 - 1).abs() < 1e-4)
        assert torch.all((y.float() - beta).abs() <= 2.0 ** -8 + 1e-3)


def test_infinities_and_nans_stay_in_their_group(cf):
    import torch
    shape = (2, 4, 4, 6, 16)
    x, gamma, beta, dy = _inputs(shape, "none", "bf16", 25)
    clean, mean0, rstd0 = _run_fwd(cf, shape, 4, "none", "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta)
    x2 = x.clone()
    x2[1, 0, 0, 0, 5] = float("nan")
    x2[0, 3, 3, 5, 12] = float("inf")
    y, mean, rstd = _run_fwd(cf, shape, 4, "none", "lrelu", 0.3, 1e-5, "bf16", x2, gamma, beta)
    hit = torch.zeros((2, 4), dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[0, 3] = True
    assert torch.equal(rstd[~hit], rstd0[~hit]) and bool(torch.isnan(rstd[hit]).all())
    wide = hit.repeat_interleave(4, 1)[:, None, None, None, :].expand(shape)
    assert torch.equal(y[~wide], clean[~wide])
    assert bool(torch.isnan(y[wide]).all())


def test_inference_without_statistics_and_same_bits_again(cf):
    import torch
    for shape, groups, pool in (((2, 8, 8, 8, 32), 4, "max"), ((3, 5, 6, 7, 40), 5, "none"), ((1, 32, 32, 32, 64), 8, "none")):
        x, gamma, beta, dy = _inputs(shape, pool, "bf16", 26)
        y, mean, rstd = _run_fwd(cf, shape, groups, pool, "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta)
        y2, _, _ = _run_fwd(cf, shape, groups, pool, "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta, stats=False)
        assert torch.equal(y, y2)
        a = _run_bwd(cf, shape, groups, pool, "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta, mean, rstd, dy)
        b = _run_bwd(cf, shape, groups, pool, "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta, mean, rstd, dy)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_gradients_alone(cf):
    """dx without dgamma and dbeta, and those without dx, have the bits of the whole call."""
    import torch
    shape, groups = (2, 8, 6, 4, 32), 4
    x, gamma, beta, dy = _inputs(shape, "none", "bf16", 27)
    _, mean, rstd = _run_fwd(cf, shape, groups, "none", "silu", 0.3, 1e-5, "bf16", x, gamma, beta)
    desc = _desc(cf, shape, groups, "none", "silu", 0.3, 1e-5, "bf16")
    size = cf.cf_group_norm_workspace_size(desc, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    cf.cf_group_norm_bwd(desc, x, gamma, beta, mean, rstd, dy, dx, dg, db, ws, size)
    dx2, dg2, db2 = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    cf.cf_group_norm_bwd(desc, x, gamma, beta, mean, rstd, dy, dx2, None, None, ws, size)
    cf.cf_group_norm_bwd(desc, x, gamma, beta, mean, rstd, dy, None, dg2, db2, ws, size)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2) and torch.equal(db, db2)


def test_backward_by_differences(cf):
    """The gradient along a direction against the forward's difference quotient, fp32.  With h = 2^-6 the quotient's cut-off
    error is about h^2 / 6 of the third derivative (order 1: 1e-4 of the scale) and its rounding 2^-22 / h of the sums."""
    import torch
    shape, groups = (2, 6, 5, 7, 24), 4
    x, gamma, beta, dy = _inputs(shape, "none", "f32", 28)
    args = ("none", "silu", 0.3, 1e-5, "f32")
    _, mean, rstd = _run_fwd(cf, shape, groups, *args, x, gamma, beta)
    grads = _run_bwd(cf, shape, groups, *args, x, gamma, beta, mean, rstd, dy)
    gen = torch.Generator(device="cuda").manual_seed(29)
    h = 2.0 ** -6
    for i, grad in enumerate(grads):
        v = torch.randn((x, gamma, beta)[i].shape, device="cuda", generator=gen)
        val = []
        for s in (h, -h):
            a = [x, gamma, beta]
            a[i] = a[i] + s * v
            val.append((_run_fwd(cf, shape, groups, *args, *a)[0].double() * dy.double()).sum().item())
        want = (grad.double() * v.double()).sum().item()
        scale = (grad.double() ** 2).sum().sqrt().item()
        assert abs((val[0] - val[1]) / (2 * h) - want) <= 5e-3 * scale


def test_on_a_stream_of_its_own(cf):
    import torch
    shape, groups = (2, 8, 8, 8, 64), 8
    x, gamma, beta, _ = _inputs(shape, "none", "bf16", 30)
    y, _, _ = _run_fwd(cf, shape, groups, "none", "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, _, _ = _run_fwd(cf, shape, groups, "none", "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta, stream=s)
    assert torch.equal(y, y2)


def test_in_a_cuda_graph(cf):
    import torch
    shape, groups = (2, 16, 16, 16, 32), 4
    x, gamma, beta, dy = _inputs(shape, "max", "bf16", 31)
    desc = _desc(cf, shape, groups, "max", "lrelu", 0.3, 1e-5, "bf16")
    size = max(cf.cf_group_norm_workspace_size(desc, b) for b in (0, 1))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    y = torch.empty((2, 8, 8, 8, 32), dtype=torch.bfloat16, device="cuda")
    mean, rstd = torch.empty((2, 4), device="cuda"), torch.empty((2, 4), device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)

    def both(s):
        cf.cf_group_norm_fwd(desc, x, gamma, beta, y, mean, rstd, ws, size, s)
        cf.cf_group_norm_bwd(desc, x, gamma, beta, mean, rstd, dy, dx, dg, db, ws, size, s)

    both(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(torch.cuda.current_stream())
    x.copy_(x.flip(1))
    want_dx, want_dg, want_db = _run_bwd(cf, shape, groups, "max", "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta,
                                         *_run_fwd(cf, shape, groups, "max", "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta)[1:], dy)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want_dx) and torch.equal(dg, want_dg) and torch.equal(db, want_db)


def test_large_offsets(cf):
    """Samples far apart: offsets beyond 2^31 values, with the last sample against the same data at the front."""
    import torch
    shape, groups, pitch = (3, 64, 64, 64, 8), 2, 3200
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    wide = torch.zeros(shape[:-1] + (pitch,), dtype=torch.bfloat16, device="cuda")
    x, gamma, beta, dy = _inputs((1,) + shape[1:], "none", "bf16", 32)
    wide[2, ..., :8] = x[0]
    desc = _desc(cf, shape, groups, "none", "lrelu", 0.3, 1e-5, "bf16", pitch, 0)
    size = cf.cf_group_norm_workspace_size(desc, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    y = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    cf.cf_group_norm_fwd(desc, wide, gamma, beta, y, None, None, ws, size)
    one, mean, rstd = _run_fwd(cf, (1,) + shape[1:], groups, "none", "lrelu", 0.3, 1e-5, "bf16", x, gamma, beta)
    torch.cuda.synchronize()
    # the chunks of one sample and of three may differ, and with them the last bits of the statistics
    assert torch.all((y[2].float() - one[0].float()).abs() <= 2.0 ** -7 * one[0].float().abs() + 1e-4)


def test_workspace_too_small(cf):
    import torch
    shape = (2, 8, 8, 8, 32)
    x, gamma, beta, dy = _inputs(shape, "none", "bf16", 33)
    desc = _desc(cf, shape, 4, "none", "lrelu", 0.3, 1e-5, "bf16")
    stat = torch.empty((2, 4), device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for back in (0, 1):
        size = cf.cf_group_norm_workspace_size(desc, back)
        if size == 0:
            continue
        call = (lambda s: cf.cf_group_norm_bwd(desc, x, gamma, beta, stat, stat, dy, torch.empty_like(x), None, None, ws, s,
                                               check=False)) if back else \
            (lambda s: cf.cf_group_norm_fwd(desc, x, gamma, beta, torch.empty_like(x), None, None, ws, s, check=False))
        assert call(size - 1) == cf.CF_ERR_WORKSPACE


@pytest.mark.parametrize("shape,groups,xp,yp", [((2, 6, 4, 10, 10), 5, 0, 0), ((2, 6, 4, 10, 26), 2, 90, 30), ((1, 40, 32, 30, 58), 2, 0, 60),
                                                ((3, 50, 48, 46, 26), 13, 90, 0), ((1, 8, 8, 8, 1030), 5, 0, 0)])
@pytest.mark.parametrize("pool", ["none", "max", "avg"])
def test_channels_in_pairs(cf, oracle_mod, shape, groups, xp, yp, pool):
    """Channels and pitches that are even and no more."""
    act = "lrelu" if pool == "max" else "silu"
    check_forward(cf, oracle_mod, shape, groups, pool=pool, act=act, xp=xp, yp=yp, seed=31)
    check_backward(cf, oracle_mod, shape, groups, pool=pool, act=act, xp=xp, yp=yp, seed=32)


# one group of all channels, so that a cluster of 16 blocks takes a sample: of the blocks 9, 9, 11 and 9 have rows (or windows)
@pytest.mark.parametrize("shape,pool", [((2, 1, 3, 3, 2048), "none"), ((1, 1, 3, 6, 2048), "none"), ((3, 1, 3, 11, 1024), "none"),
                                        ((2, 2, 6, 6, 2048), "max")])
def test_clusters_whose_blocks_have_no_rows(cf, oracle_mod, shape, pool):
    """And the same bits each time, whatever order the blocks begin in."""
    import torch
    act = "lrelu" if pool == "max" else "silu"
    check_forward(cf, oracle_mod, shape, 1, pool=pool, act=act, seed=41)
    check_backward(cf, oracle_mod, shape, 1, pool=pool, act=act, seed=42)
    x, gamma, beta, dy = _inputs(shape, pool, "bf16", 43)
    first = None
    for _ in range(20):
        y, mean, rstd = _run_fwd(cf, shape, 1, pool, act, 0.3, 1e-5, "bf16", x, gamma, beta)
        got = (y, mean, rstd) + _run_bwd(cf, shape, 1, pool, act, 0.3, 1e-5, "bf16", x, gamma, beta, mean, rstd, dy)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def _windows(t):
    n, d, h, w, c = t.shape
    return t.reshape(n, d // 2, 2, h // 2, 2, w // 2, 2, c).permute(0, 1, 3, 5, 2, 4, 6, 7).reshape(n, d // 2, h // 2, w // 2, 8, c)


def _unwindows(t):
    n, d, h, w, _, c = t.shape
    return t.reshape(n, d, h, w, 2, 2, 2, c).permute(0, 1, 4, 2, 5, 3, 6, 7).reshape(n, 2 * d, 2 * h, 2 * w, c)


# more rows than one wave of blocks has in chunks of their longest: 75 million values in eights (forward and backward: two waves),
# 21 million one by one (three), 43 million in fours
@pytest.mark.parametrize("shape,groups", [((2, 128, 96, 96, 32), 8), ((3, 96, 82, 70, 13), 13), ((2, 128, 96, 88, 20), 4)])
@pytest.mark.parametrize("pool,act", [("none", "silu"), ("max", "lrelu"), ("avg", "silu")])
def test_several_waves_of_chunks(cf, shape, groups, pool, act):
    """Against the same formulas in 64 bits on the GPU, with the tolerances of the small shapes."""
    import torch
    n, c, per, eps = shape[0], shape[-1], shape[-1] // groups, 1e-5
    x, gamma, beta, dy = _inputs(shape, pool, "bf16", 51)
    y, mean, rstd = _run_fwd(cf, shape, groups, pool, act, 0.3, eps, "bf16", x, gamma, beta)
    X, G, B = x.double(), gamma.double(), beta.double()
    grouped = X.reshape(n, -1, groups, per)

    def wide(t):
        return t.repeat_interleave(per, 1)[:, None, None, None, :]

    rm = grouped.mean((1, 3))
    rr = ((grouped - rm[:, None, :, None]) ** 2).mean((1, 3)).add(eps).rsqrt()
    mabs = grouped.abs().mean((1, 3))
    assert bool(((mean - rm).abs() <= 2.0 ** -17 * mabs).all())
    assert bool(((rstd - rr).abs() <= rr * (2.0 ** -17 + (2.0 ** -17 * mabs * rr) ** 2)).all())
    xh = (X - wide(rm)) * wide(rr)
    u = G * xh + B
    ue = 2.0 ** -16 * (G.abs() * wide(rr) * (X.abs() + wide(rm).abs()) + B.abs())
    act_of = torch.nn.functional.silu if act == "silu" else lambda t: torch.where(t > 0, t, 0.3 * t)
    if pool == "max":
        ref = act_of(_windows(u).amax(4))
    else:
        ref = act_of(u) if pool == "none" else _windows(act_of(u)).mean(4)
    tol = 2.0 ** -8 * ref.abs() + 1.1 * (_windows(ue).amax(4) if pool != "none" else ue)
    assert bool(((y.double() - ref).abs() <= tol).all())
    del y, ref, tol, ue
    if pool == "max":  # its gradient may go to either of two voxels that are equal within rounding: small shapes look at that
        return
    sm, sr = rm.float(), rr.float()
    dx, dgamma, dbeta = _run_bwd(cf, shape, groups, pool, act, 0.3, eps, "bf16", x, gamma, beta, sm, sr, dy)
    xh = (X - wide(sm.double())) * wide(sr.double())
    u = G * xh + B
    s = torch.sigmoid(u)
    full = dy.double() if pool == "none" else _unwindows((dy.double() / 8)[..., None, :].expand(*dy.shape[:4], 8, c))
    du = full * s * (1 + u * (1 - s))
    del u, s, full

    def gm(t):
        return wide(t.reshape(n, -1, groups, per).mean((1, 3)))

    axes = (0, 1, 2, 3)
    assert bool(((dbeta - du.sum(axes)).abs() <= 2.0 ** -15 * du.abs().sum(axes)).all())
    assert bool(((dgamma - (du * xh).sum(axes)).abs() <= 2.0 ** -15 * ((du * xh).abs() + du.abs()).sum(axes)).all())
    r = wide(sr.double())
    ref = r * (G * du - gm(G * du) - xh * gm(G * du * xh))
    parts = r * ((G * du).abs() + gm((G * du).abs()) + xh.abs() * gm((G * du * xh).abs())) * (1 + wide(sm.double()).abs() * r)
    assert bool(((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * parts).all())


@pytest.mark.parametrize("pool,dtype", [("none", "bf16"), ("none", "f32"), ("max", "bf16"), ("avg", "bf16")])
@pytest.mark.parametrize("shape", [(2, 6, 4, 10, 24), (1, 48, 40, 36, 48)])
def test_slices_that_begin_inside_a_wider_tensor(cf, shape, pool, dtype):
    """Channels 16 .. 16 + c - 1 of 128, x and dx, and 8 .. of 80, y and dy, have the bits of tensors of their own, and the channels
    beside them stay as they are."""
    import torch
    act, c, groups, xp, yp = "lrelu" if pool == "max" else "silu", shape[-1], 4, 128, 80
    x, gamma, beta, dy = _inputs(shape, pool, dtype, 52)
    y, mean, rstd = _run_fwd(cf, shape, groups, pool, act, 0.3, 1e-5, dtype, x, gamma, beta)
    dx, dgamma, dbeta = _run_bwd(cf, shape, groups, pool, act, 0.3, 1e-5, dtype, x, gamma, beta, mean, rstd, dy)
    desc = _desc(cf, shape, groups, pool, act, 0.3, 1e-5, dtype, xp, yp)
    ws = torch.empty(max(cf.cf_group_norm_workspace_size(desc, b) for b in (0, 1)), dtype=torch.uint8, device="cuda")

    def inside(t, pitch, at):
        buf = torch.full(t.shape[:-1] + (pitch,), 7.0, dtype=t.dtype, device="cuda")
        return buf, buf[..., at:at + c]

    (_, xs), (yb, ys), (_, dys), (dxb, dxs) = inside(x, xp, 16), inside(y, yp, 8), inside(dy, yp, 8), inside(x, xp, 16)
    xs.copy_(x)
    dys.copy_(dy)
    m2, r2, dg2, db2 = (torch.empty_like(t) for t in (mean, rstd, dgamma, dbeta))
    cf.cf_group_norm_fwd(desc, xs, gamma, beta, ys, m2, r2, ws, ws.numel())
    cf.cf_group_norm_bwd(desc, xs, gamma, beta, mean, rstd, dys, dxs, dg2, db2, ws, ws.numel())
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    for a, b in ((y, ys), (mean, m2), (rstd, r2), (dx, dxs), (dgamma, dg2), (dbeta, db2)):
        assert torch.equal(a, b)
    for buf, at in ((yb, 8), (dxb, 16)):
        assert bool((buf[..., :at] == 7).all()) and bool((buf[..., at + c:] == 7).all())


@pytest.mark.parametrize("pool", ["none", "max", "avg"])
def test_large_offsets_both_ways(cf, pool):
    """The last of three samples, beyond 2^31 values, against the same sample alone: forward and backward.  The chunks of one sample
    and of three differ, and with them the last bits of sums: 2^-14 of terms of which dx has at most about ten, beside its rounding."""
    import torch
    shape, groups, pitch = (3, 64, 64, 64, 8), 2, 3200
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    one = (1,) + shape[1:]
    act = "lrelu" if pool == "max" else "silu"
    x, gamma, beta, dy = _inputs(one, pool, "bf16", 53)
    y, mean, rstd = _run_fwd(cf, one, groups, pool, act, 0.3, 1e-5, "bf16", x, gamma, beta)
    dx, dgamma, dbeta = _run_bwd(cf, one, groups, pool, act, 0.3, 1e-5, "bf16", x, gamma, beta, mean, rstd, dy)
    wide = torch.zeros(shape[:-1] + (pitch,), dtype=torch.bfloat16, device="cuda")
    wide[2, ..., :8] = x[0]
    desc = _desc(cf, shape, groups, pool, act, 0.3, 1e-5, "bf16", pitch, 0)
    ws = torch.empty(max(cf.cf_group_norm_workspace_size(desc, b) for b in (0, 1)), dtype=torch.uint8, device="cuda")
    y3 = torch.empty((3,) + y.shape[1:], dtype=torch.bfloat16, device="cuda")
    cf.cf_group_norm_fwd(desc, wide, gamma, beta, y3, None, None, ws, ws.numel())
    m3, r3, dy3 = (torch.zeros((3,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in (mean, rstd, dy))
    m3[2], r3[2], dy3[2] = mean[0], rstd[0], dy[0]
    dwide = torch.full_like(wide, 7.0)
    dg3, db3 = torch.empty_like(dgamma), torch.empty_like(dbeta)
    cf.cf_group_norm_bwd(desc, wide, gamma, beta, m3, r3, dy3, dwide, dg3, db3, ws, ws.numel())
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    for a, b in ((y[0], y3[2]), (dx[0], dwide[2, ..., :8])):
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 1e-3).all())
    assert bool((dwide[..., 8:] == 7).all()) and bool((dwide[:2, ..., :8] == 0).all())
    count = dy[..., 0].numel()
    for a, b in ((dgamma, dg3), (dbeta, db3)):
        assert bool(((a - b).abs() <= 2.0 ** -14 * count).all())


@pytest.mark.parametrize("shape,groups", [((2, 4, 4, 6, 16), 4), ((3, 48, 48, 48, 64), 8), ((2, 50, 48, 46, 20), 5)])
@pytest.mark.parametrize("pool", ["none", "max", "avg"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_finite_stays_in_its_group_both_ways(cf, shape, groups, pool, value):
    """Small and large samples: one value of one group of the last sample; every other group has the bits that it had before."""
    import torch
    per, act = shape[-1] // groups, "lrelu" if pool == "max" else "silu"
    x, gamma, beta, dy = _inputs(shape, pool, "bf16", 54)

    def both(x):
        y, mean, rstd = _run_fwd(cf, shape, groups, pool, act, 0.3, 1e-5, "bf16", x, gamma, beta)
        return (y, mean, rstd) + _run_bwd(cf, shape, groups, pool, act, 0.3, 1e-5, "bf16", x, gamma, beta, mean, rstd, dy)

    clean = both(x)
    x = x.clone()
    x[-1, -1, 1, 2, per + 1] = value  # the second group
    got = both(x)
    for i, (a, b) in enumerate(zip(clean, got)):
        if i in (1, 2):  # mean, rstd [n][groups]
            same = torch.ones_like(a, dtype=torch.bool)
            same[-1, 1] = False
            assert bool((~torch.isfinite(b[-1, 1])).all())
        else:  # y, dx of the last sample; dgamma, dbeta of the group's channels
            same = torch.ones_like(a, dtype=torch.bool)
            (same[-1] if a.dim() == 5 else same)[..., per:2 * per] = False
            # (dbeta sums LReLU'(u) dy, and LReLU' is the slope for any u that is not above 0, NaN too)
            assert bool(torch.isnan(b[~same]).all()) or (i == 5 and act == "lrelu"), i
        assert torch.equal(a[same], b[same]), i
