"""Products of whole numbers (cf_linear_*), whose sums fp32 holds: every block of the contracted axis counts once, whichever way a product
is cut.  A bound for sums of random values does not see a lost block where the axis is long."""
import pytest

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


def whole(g, shape, most):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def rows_of(g, rows, width, pitch, most, dtype):
    """[rows][width] of rows `pitch` apart with NaN between."""
    t = torch.full((rows, pitch or width), float("nan"), device="cuda", dtype=dtype)
    t[:, :width] = whole(g, (rows, width), most).to(dtype)
    return t[:, :width]


def out_of(rows, width, pitch, dtype):
    t, guard = guarded((rows, pitch or width), dtype, fill=-7.0)

    def check():
        guard()
        assert bool((t[:, width:] == -7.0).all()), "values between the rows were written"
    return t[:, :width], check


# few rows (clusters, sides exchanged), long sums (cut tiles, segments), pairs and lone CTAs, narrow tiles side by side, rows that begin anywhere
SIZES = [(1, 20000, 72, 0, 0), (8, 2048, 2048, 0, 0), (40, 12000, 264, 0, 0), (40, 3000, 10000, 0, 0), (100, 1030, 500, 0, 0), (128, 4096, 4096, 0, 0),
         (200, 2000, 1000, 0, 0), (300, 20000, 272, 0, 0), (150, 5001, 2600, 0, 0), (700, 9000, 400, 0, 0), (2048, 2048, 2048, 0, 0), (5000, 520, 1290, 0, 0),
         (257, 1000, 130, 1003, 141), (9000, 1032, 160, 1040, 168), (160001, 32, 32, 0, 0), (200003, 24, 21, 0, 0), (50000, 64, 250, 0, 256)]


@pytest.mark.parametrize("rows,k,n,xp,yp", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(cf, rows, k, n, xp, yp, dtype):
    g = torch.Generator("cuda").manual_seed(rows + k + n)
    x, w, b, res = rows_of(g, rows, k, xp, 3, BF), whole(g, (n, k), 3).to(BF), whole(g, (n,), 50).float(), rows_of(g, rows, n, yp, 100, dtype)
    kind = cf.CF_DT_F32 if dtype == F32 else cf.CF_DT_BF16
    d = cf.cf_linear_desc(rows, k, n, cf.CF_ACT_LRELU, 1.0, 0.5, kind, xp, yp)
    size = cf.cf_linear_workspace_size(d, cf.CF_LINEAR_FWD)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    (y, ok_y), (z, ok_z) = out_of(rows, n, yp, dtype), out_of(rows, n, yp, BF)
    cf.cf_linear_fwd(d, x, w, b, res, y, z, ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    ok_y(), ok_z()
    want = x.double() @ w.double().T + b.double()
    assert torch.equal(z, want.float().to(BF))
    assert torch.equal(y, (0.5 * want + res.double()).float().to(dtype))


@pytest.mark.parametrize("rows,k,n,xp,yp", [(r, n, k, xp and yp, yp and xp) for r, k, n, xp, yp in SIZES])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_data(cf, rows, k, n, xp, yp, dtype):
    g = torch.Generator("cuda").manual_seed(rows + k + n)
    dz, w, add, pre = rows_of(g, rows, n, yp, 3, BF), whole(g, (n, k), 3).to(BF), rows_of(g, rows, k, xp, 100, dtype), rows_of(g, rows, k, xp, 3, BF)
    kind = cf.CF_DT_F32 if dtype == F32 else cf.CF_DT_BF16
    d = cf.cf_linear_desc(rows, k, n, cf.CF_ACT_LRELU, 0.5, 0.5, kind, xp, yp)
    size = cf.cf_linear_workspace_size(d, cf.CF_LINEAR_DGRAD)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, ok = out_of(rows, k, xp, dtype)
    cf.cf_linear_dgrad(d, dz, w, pre, add, dx, ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    ok()
    want = 0.5 * (dz.double() @ w.double()) * torch.where(pre > 0, 1.0, 0.5).double() + add.double()
    assert torch.equal(dx, want.float().to(dtype))
