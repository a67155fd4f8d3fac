"""Matrix products with bias, activation and residual (cf_linear_*) against 64 bits, on the sizes, types, pitches and values where
they can go wrong."""
import numpy as np
import pytest

import oracle
from gpu_util import guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def f64(t):
    return t.detach().double().cpu().numpy()


def rows_of(rng, rows, width, pitch=0, dtype=BF, mean=0.0):
    """[rows][width] on the device, a slice of rows `pitch` apart whose gaps hold NaN."""
    t = torch.full((rows, pitch or width), float("nan"), dtype=dtype)
    t[:, :width] = torch.from_numpy(rng.normal(mean, 1.0, (rows, width))).to(dtype)
    return t.cuda()[:, :width]


def out_rows(rows, width, pitch, dtype):
    """An output with its guards: (tensor, check); the check looks at the gaps of its rows too."""
    t, guard = guarded((rows, pitch or width), dtype, fill=-7.0)

    def check():
        guard()
        assert bool((t[:, width:] == -7.0).all()), "values between the rows were written"
    return t[:, :width], check


def desc_of(cf, rows, k, n, act="none", slope=1.0, scale=1.0, dtype=BF, xp=0, yp=0):
    a = {"gelu": cf.CF_ACT_GELU, "silu": cf.CF_ACT_SILU}.get(act, cf.CF_ACT_LRELU)
    return cf.cf_linear_desc(rows, k, n, a, slope if act == "lrelu" else 1.0, scale, cf.CF_DT_F32 if dtype == F32 else cf.CF_DT_BF16, xp, yp)


def workspace(cf, d, op):
    size = cf.cf_linear_workspace_size(d, op)
    return torch.full((max(size, 16),), 0xA5, dtype=torch.uint8, device="cuda"), size


HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}  # a rounding's largest error, relative


def sum_bound(terms, s):
    """Error of an fp32 sum of `terms` exact products of total size s, in any order, were each step cut off instead of rounded."""
    return (terms + 8) * 2.0 ** -23 * s


def check_fwd(cf, rng, rows, k, n, act="none", slope=1.0, scale=1.0, dtype=BF, xp=0, yp=0, bias=True, residual=True, pre=True, stream=None):
    x, w = rows_of(rng, rows, k, xp), rows_of(rng, n, k) * (1.0 / np.sqrt(k))
    b = torch.from_numpy(rng.normal(0, 0.5, n)).float().cuda() if bias else None
    res = rows_of(rng, rows, n, yp, dtype) if residual else None
    y, ok_y = out_rows(rows, n, yp, dtype)
    z, ok_z = out_rows(rows, n, yp, BF) if pre else (None, lambda: None)
    d = desc_of(cf, rows, k, n, act, slope, scale, dtype, xp, yp)
    ws, size = workspace(cf, d, cf.CF_LINEAR_FWD)
    torch.cuda.synchronize()
    cf.cf_linear_fwd(d, x, w, b, res, y, z, ws, size, stream)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    ok_y(), ok_z()
    X, W = f64(x), f64(w)
    B = f64(b) if bias else None
    ry, rz = oracle.linear_fwd(X, W, B, f64(res) if residual else None, act, slope, scale)
    ez = sum_bound(k, np.abs(X) @ np.abs(W).T + (np.abs(B) if bias else 0.0))
    if pre:
        assert np.all(np.abs(f64(z) - rz) <= HALF[BF] * (np.abs(rz) + ez) + ez)
    # activations change by at most 1.13 of their argument's change; their own functions are good to 2^-20 of the value
    # (exponents up to 2^7 in an fp32 argument), and the value is rounded when it is scaled and when the residual is added
    a = np.abs(scale * oracle.linear_act(rz, act, slope))
    ey = 1.13 * abs(scale) * ez + (2.0 ** -16 if act in ("gelu", "silu") else 0.0) * a + 2.0 ** -22 * (a + np.abs(ry))
    assert np.all(np.abs(f64(y) - ry) <= HALF[dtype] * (np.abs(ry) + ey) + ey + 1e-37)
    return y, z


def check_dgrad(cf, rng, rows, k, n, act="none", slope=1.0, scale=1.0, dtype=BF, xp=0, yp=0, add=True, pre=True):
    dz, w = rows_of(rng, rows, n, yp), rows_of(rng, n, k) * (1.0 / np.sqrt(n))
    z = rows_of(rng, rows, k, xp) if pre else None
    res = rows_of(rng, rows, k, xp, dtype) if add else None
    dx, ok = out_rows(rows, k, xp, dtype)
    d = desc_of(cf, rows, k, n, act, slope, scale, dtype, xp, yp)
    ws, size = workspace(cf, d, cf.CF_LINEAR_DGRAD)
    cf.cf_linear_dgrad(d, dz, w, z, res, dx, ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    ok()
    DZ, W = f64(dz), f64(w)
    ref = oracle.linear_dgrad(DZ, W, f64(z) if pre else None, f64(res) if add else None, act, slope, scale)
    g = np.abs(oracle.linear_act_grad(f64(z), act, slope)) if pre else 1.0
    S = np.abs(DZ) @ np.abs(W)
    # derivatives are sums of values up to 8 that are good to 2^-20
    e = abs(scale) * (g * sum_bound(n, S) + 2.0 ** -16 * S) + 2.0 ** -22 * (np.abs(ref) + abs(scale) * S)
    assert np.all(np.abs(f64(dx) - ref) <= HALF[dtype] * (np.abs(ref) + e) + e)
    return dx


def check_wgrad(cf, rng, rows, k, n, scale=1.0, xp=0, yp=0, bias=True, accumulate=0):
    x, dz = rows_of(rng, rows, k, xp, mean=0.2), rows_of(rng, rows, n, yp, mean=0.1)
    dw, ok_w = out_rows(n, k, 0, F32)
    db, ok_b = guarded((n,), F32, fill=3.0)
    d = desc_of(cf, rows, k, n, scale=scale, xp=xp, yp=yp)
    ws, size = workspace(cf, d, cf.CF_LINEAR_WGRAD)
    cf.cf_linear_wgrad(d, x, dz, dw, db if bias else None, accumulate, ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    ok_w(), ok_b()
    X, DZ = f64(x), f64(dz)
    rw, rb = oracle.linear_wgrad(X, DZ, scale)
    S, Sb = np.abs(scale) * (np.abs(DZ).T @ np.abs(X)), np.abs(scale) * np.abs(DZ).sum(0)
    if accumulate:
        rw, rb, S, Sb = rw - 7.0, rb + 3.0, S + 7.0, Sb + 3.0
    assert np.all(np.abs(f64(dw) - rw) <= sum_bound(rows, S))
    if bias:
        assert np.all(np.abs(f64(db) - rb) <= sum_bound(rows, Sb))
    else:
        assert bool((db == 3.0).all())
    return dw, db


SIZES = [(1, 8, 8), (1, 1, 1), (2, 2048, 96), (8, 512, 2048), (33, 64, 40), (128, 64, 256), (129, 72, 264), (300, 32, 32), (257, 1000, 130),
         (5, 3, 7), (640, 515, 77), (1000, 130, 33), (2000, 256, 512), (77, 4100, 520), (16, 4096, 1024), (64, 96, 4096), (4096, 16, 48),
         # tiles that clusters share, more blocks than CTAs or as many, ends inside a tile
         (20, 200, 1000), (100, 1030, 500), (200, 2000, 1000), (260, 700, 150), (500, 4000, 520), (1000, 640, 320), (3, 130, 40)]


@pytest.mark.parametrize("rows,k,n", SIZES)
def test_forward_sizes(cf, rows, k, n):
    check_fwd(cf, np.random.default_rng(rows + k + n), rows, k, n, "gelu")


@pytest.mark.parametrize("rows,k,n", SIZES)
def test_backward_data_sizes(cf, rows, k, n):
    check_dgrad(cf, np.random.default_rng(rows + k + n), rows, k, n, "silu")


@pytest.mark.parametrize("rows,k,n", SIZES + [(30000, 64, 64), (50001, 40, 24), (20000, 520, 136)])
def test_backward_weight_sizes(cf, rows, k, n):
    check_wgrad(cf, np.random.default_rng(rows + k + n), rows, k, n)


# tiles of pairs, whole and cut, ends that fill neither half of a pair; many tiles of lone CTAs
LARGE = [(40, 3000, 10000), (1500, 3000, 1000), (5000, 520, 1290), (700, 9000, 400), (2048, 2048, 2048), (300, 20000, 272), (9000, 1032, 160), (50000, 64, 250),
         (150, 5000, 2600)]


@pytest.mark.parametrize("rows,k,n", LARGE)
def test_large_products(cf, rows, k, n):
    rng = np.random.default_rng(rows)
    check_fwd(cf, rng, rows, k, n, "silu", pre=False)
    check_dgrad(cf, rng, rows, n, k, "gelu", dtype=F32)
    check_wgrad(cf, rng, n, k, rows)
    check_wgrad(cf, rng, k, rows, n)


@pytest.mark.parametrize("rows,k,n", [(160001, 32, 32), (400100, 64, 16), (170000, 40, 48), (330000, 16, 128), (200003, 24, 21)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_narrow_products_of_many_rows(cf, rows, k, n, dtype):
    rng = np.random.default_rng(rows)
    check_fwd(cf, rng, rows, k, n, "gelu", dtype=dtype)
    check_dgrad(cf, rng, rows, n, k, "silu", dtype=dtype)


@pytest.mark.parametrize("act,slope", [("none", 1.0), ("lrelu", 0.3), ("lrelu", 0.0), ("silu", 1.0), ("gelu", 1.0)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [4, 300])
def test_activations_and_types(cf, act, slope, dtype, rows):
    rng = np.random.default_rng(11)
    check_fwd(cf, rng, rows, 96, 136, act, slope, 0.7, dtype)
    check_dgrad(cf, rng, rows, 96, 136, act, slope, 0.7, dtype)


@pytest.mark.parametrize("rows,k,n,op", [(200000, 64, 72, "wgrad"), (9000, 520, 264, "wgrad"), (300, 12000, 264, "fwd"), (40, 12000, 264, "fwd"),
                                         (700, 136, 9000, "dgrad")])
def test_long_sums_keep_fp32s_precision(cf, rows, k, n, op):
    """The tensor cores cut sums off, on average by 2^-24 of them, at each of at most 96 steps of 16 before they are added up in fp32
    that rounds; a sum of values of mixed signs is on average at most 0.7 of its end: 96 0.7 2^-24 = 4.0e-6 of the result."""
    rng = np.random.default_rng(20)
    x, w, dz = rows_of(rng, rows, k), rows_of(rng, n, k), rows_of(rng, rows, n)
    out = torch.empty({"wgrad": (n, k), "fwd": (rows, n), "dgrad": (rows, k)}[op], device="cuda")
    d = desc_of(cf, rows, k, n, dtype=F32)
    ws = workspace(cf, d, {"fwd": 0, "dgrad": 1, "wgrad": 2}[op])
    if op == "wgrad":
        cf.cf_linear_wgrad(d, x, dz, out, None, 0, *ws)
        ref = f64(dz).T @ f64(x)
    elif op == "fwd":
        cf.cf_linear_fwd(d, x, w, None, None, out, None, *ws)
        ref = f64(x) @ f64(w).T
    else:
        cf.cf_linear_dgrad(d, dz, w, None, None, out, *ws)
        ref = f64(dz) @ f64(w)
    assert np.linalg.norm(f64(out) - ref) <= 4.0e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("residual,pre,bias", [(0, 0, 0), (1, 0, 1), (0, 1, 0), (0, 0, 1)])
@pytest.mark.parametrize("rows,k,n", [(3, 256, 200), (520, 256, 200)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_may_be_left_out(cf, residual, pre, bias, rows, k, n, dtype):
    rng = np.random.default_rng(12)
    check_fwd(cf, rng, rows, k, n, "silu", dtype=dtype, bias=bool(bias), residual=bool(residual), pre=bool(pre))
    check_dgrad(cf, rng, rows, k, n, "silu", dtype=dtype, add=bool(residual), pre=bool(pre))
    check_wgrad(cf, rng, rows, k, n, -0.5, bias=bool(bias))


@pytest.mark.parametrize("rows,k,n,xp,yp", [(200, 64, 96, 72, 104), (200, 64, 96, 65, 97), (7, 130, 515, 133, 520), (7, 130, 515, 136, 517),
                                            (1000, 515, 130, 515, 133), (129, 24, 40, 1000, 41), (300, 33, 64, 40, 0), (300, 64, 33, 0, 48)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_are_slices(cf, rows, k, n, xp, yp, dtype):
    rng = np.random.default_rng(13)
    check_fwd(cf, rng, rows, k, n, "gelu", dtype=dtype, xp=xp, yp=yp)
    check_dgrad(cf, rng, rows, k, n, "gelu", dtype=dtype, xp=xp, yp=yp)
    check_wgrad(cf, rng, rows, k, n, xp=xp, yp=yp)


@pytest.mark.parametrize("rows,k,n", [(1, 64, 64), (700, 48, 80), (9000, 40, 33)])
def test_weight_gradients_add_to_what_is_there(cf, rows, k, n):
    check_wgrad(cf, np.random.default_rng(14), rows, k, n, 0.5, accumulate=1)


@pytest.mark.parametrize("accumulate", [0, 1])
def test_no_rows(cf, accumulate):
    d = desc_of(cf, 0, 40, 24)
    dw, db = torch.ones((24, 40), device="cuda"), torch.ones(24, device="cuda")
    ws, size = workspace(cf, d, cf.CF_LINEAR_WGRAD)
    cf.cf_linear_wgrad(d, None, None, dw, db, accumulate, ws, size)
    assert bool((dw == accumulate).all()) and bool((db == accumulate).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,n,yp", [(5, 200, 0), (500, 200, 0), (500, 201, 211)])
def test_in_place_on_the_stream(cf, dtype, rows, n, yp):
    """y over the residual and dx over add, with the bits of the call that writes elsewhere."""
    rng = np.random.default_rng(15)
    x, w = rows_of(rng, rows, 64), rows_of(rng, n, 64)
    res = rows_of(rng, rows, n, yp, dtype)
    d = desc_of(cf, rows, 64, n, "silu", dtype=dtype, yp=yp)
    ws, size = workspace(cf, d, cf.CF_LINEAR_FWD)
    y = torch.empty((rows, yp or n), dtype=dtype, device="cuda")[:, :n]
    cf.cf_linear_fwd(d, x, w, None, res, y, None, ws, size)
    cf.cf_linear_fwd(d, x, w, None, res, res, None, ws, size)
    assert torch.equal(y, res)
    dz, wt = rows_of(rng, rows, 64), rows_of(rng, 64, n)
    add = rows_of(rng, rows, n, yp, dtype)
    d = desc_of(cf, rows, n, 64, dtype=dtype, xp=yp)
    ws, size = workspace(cf, d, cf.CF_LINEAR_DGRAD)
    cf.cf_linear_dgrad(d, dz, wt, None, add, y, ws, size)
    cf.cf_linear_dgrad(d, dz, wt, None, add, add, ws, size)
    assert torch.equal(y, add)


@pytest.mark.parametrize("rows", [6, 400])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row_or_column(cf, rows, value):
    rng = np.random.default_rng(16)
    k, n = 72, 136
    x, w, dz = rows_of(rng, rows, k), rows_of(rng, n, k), rows_of(rng, rows, n)
    d = desc_of(cf, rows, k, n, "gelu")
    ws, size = workspace(cf, d, cf.CF_LINEAR_FWD)
    wsw, sizew = workspace(cf, d, cf.CF_LINEAR_WGRAD)
    y0, y1 = torch.empty((rows, n), dtype=BF, device="cuda"), torch.empty((rows, n), dtype=BF, device="cuda")
    dw0, dw1 = torch.empty((n, k), device="cuda"), torch.empty((n, k), device="cuda")
    cf.cf_linear_fwd(d, x, w, None, None, y0, None, ws, size)
    cf.cf_linear_wgrad(d, x, dz, dw0, None, 0, wsw, sizew)
    x[rows - 2, 5] = value
    cf.cf_linear_fwd(d, x, w, None, None, y1, None, ws, size)
    cf.cf_linear_wgrad(d, x, dz, dw1, None, 0, wsw, sizew)
    keep = torch.arange(rows, device="cuda") != rows - 2
    assert torch.equal(y0[keep], y1[keep]) and not bool(torch.isfinite(y1[rows - 2]).all())
    cols = torch.arange(k, device="cuda") != 5
    assert torch.equal(dw0[:, cols], dw1[:, cols]) and not bool(torch.isfinite(dw1[:, 5]).any())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_of_large_arguments(cf, act):
    """Far from 0 the activations are z and 0, their derivatives 1 and 0, with no overflow on the way."""
    z = torch.tensor([1e4, 1e20, 3e38, -1e4, -1e20, -3e38, 50.0, -200.0], device="cuda").to(BF).repeat(16, 1)
    eye = torch.eye(8, device="cuda", dtype=BF)
    y, dx = torch.empty_like(z), torch.empty_like(z)
    d = desc_of(cf, 16, 8, 8, act)
    ws, size = workspace(cf, d, cf.CF_LINEAR_FWD)
    cf.cf_linear_fwd(d, z, eye, None, None, y, None, ws, size)
    assert torch.equal(y, torch.where(z > 0, z, torch.zeros_like(z)))
    wsd, sized = workspace(cf, d, cf.CF_LINEAR_DGRAD)
    one = torch.ones_like(z)
    cf.cf_linear_dgrad(d, one, eye, z, None, dx, wsd, sized)
    assert torch.equal(dx, (z > 0).to(BF))
    cf.cf_linear_act_bwd(d, one, z, dx)
    assert torch.equal(dx, (z > 0).to(BF))


@pytest.mark.parametrize("rows,n,yp,dtype", [(1, 1, 0, BF), (33, 70, 0, BF), (200, 64, 72, F32), (50, 33, 41, F32), (1000, 256, 0, BF)])
@pytest.mark.parametrize("act", ["lrelu", "gelu"])
def test_activation_backward(cf, rows, n, yp, dtype, act):
    rng = np.random.default_rng(17)
    dy, z = rows_of(rng, rows, n, yp, dtype), rows_of(rng, rows, n, yp)
    dz, ok = out_rows(rows, n, yp, BF)
    cf.cf_linear_act_bwd(desc_of(cf, rows, 8, n, act, 0.3, 0.7, dtype, 0, yp), dy, z, dz)
    torch.cuda.synchronize()
    ok()
    ref = 0.7 * f64(dy) * oracle.linear_act_grad(f64(z), act, 0.3)
    e = 2.0 ** -16 * np.abs(f64(dy))
    assert np.all(np.abs(f64(dz) - ref) <= HALF[BF] * (np.abs(ref) + e) + e)


@pytest.mark.parametrize("rows,k,n", [(4, 1024, 512), (500, 128, 384), (30000, 64, 48)])
def test_the_same_bits_again_on_another_stream_and_in_a_graph(cf, rows, k, n):
    rng = np.random.default_rng(18)
    x, w, dz = rows_of(rng, rows, k), rows_of(rng, n, k), rows_of(rng, rows, n)
    z = rows_of(rng, rows, k)
    d = desc_of(cf, rows, k, n, "gelu")
    out = [[torch.empty((rows, n), dtype=BF, device="cuda"), torch.empty((rows, k), dtype=BF, device="cuda"),
            torch.empty((n, k), device="cuda"), torch.empty(n, device="cuda")] for _ in range(3)]
    ws = [workspace(cf, d, op) for op in range(3)]

    def calls(o, s):
        cf.cf_linear_fwd(d, x, w, None, None, o[0], None, *ws[0], s)
        cf.cf_linear_dgrad(d, dz, w, z, None, o[1], *ws[1], s)
        cf.cf_linear_wgrad(d, x, dz, o[2], o[3], 0, *ws[2], s)

    calls(out[0], torch.cuda.current_stream())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls(out[1], side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls(out[2], torch.cuda.current_stream())
    for _ in range(2):
        for t in out[2]:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    for o in out[1:]:
        for a, b in zip(out[0], o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("k,n", [(64, 64), (64, 40)])
def test_offsets_beyond_2_to_32(cf, k, n):
    """Rows far apart: the last one starts beyond 2^32 values."""
    rows, pitch = 140, 1 << 25
    rng = np.random.default_rng(19)
    big = torch.empty(((rows - 1) * pitch + max(k, n),), dtype=BF, device="cuda")
    x = torch.as_strided(big, (rows, k), (pitch, 1))
    x.copy_(torch.from_numpy(rng.normal(size=(rows, k))))
    w = rows_of(rng, n, k)
    d = desc_of(cf, rows, k, n, xp=pitch)
    y = torch.empty((rows, n), dtype=BF, device="cuda")
    ws, size = workspace(cf, d, cf.CF_LINEAR_FWD)
    cf.cf_linear_fwd(d, x, w, None, None, y, None, ws, size)
    xc, y2 = x.contiguous(), torch.empty_like(y)
    d2 = desc_of(cf, rows, k, n)
    cf.cf_linear_fwd(d2, xc, w, None, None, y2, None, ws, size)
    assert torch.equal(y, y2)
    dz = rows_of(rng, rows, n)
    ws, size = workspace(cf, d, cf.CF_LINEAR_WGRAD)
    dw, dw2 = torch.empty((n, k), device="cuda"), torch.empty((n, k), device="cuda")
    cf.cf_linear_wgrad(d, x, dz, dw, None, 0, ws, size)
    cf.cf_linear_wgrad(d2, xc, dz, dw2, None, 0, ws, size)
    assert torch.equal(dw, dw2)
    ws, size = workspace(cf, d, cf.CF_LINEAR_DGRAD)
    cf.cf_linear_dgrad(d2, dz, w, None, None, xc, ws, size)
    cf.cf_linear_dgrad(d, dz, w, None, None, x, ws, size)
    assert torch.equal(x, xc)
