"""Residual norms (cf_residual_norm_*) of rows in stages whose tensors end inside 16 bytes: the last values come to their stage one by
one, not by the copies that bring the others, and are there when the stage is."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


@pytest.mark.parametrize("dtype,f_dtype", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("rows,c", [(20003, 130), (20001, 129), (10007, 255), (2437, 515), (1301, 2045), (701, 4095), (600001, 3), (400003, 1)])
def test_last_values_every_time(cf, rows, c, dtype, f_dtype):
    """Twenty calls over refilled outputs give the bits that the last rows have in a call of their own, which has no stages."""
    g = torch.Generator("cuda").manual_seed(rows + c)
    x, dr = (torch.randn((rows, c), generator=g, device="cuda").to(dtype) for _ in range(2))
    f, dh = (torch.randn((rows, c), generator=g, device="cuda").to(f_dtype) for _ in range(2))
    few = 8  # rows, whose bytes are a multiple of 16 at any width
    kind = cf.CF_DT_F32 if dtype == F32 else cf.CF_DT_BF16, cf.CF_DT_F32 if f_dtype == F32 else cf.CF_DT_BF16

    def calls(n, x, f, dh, dr, out, ws, size):
        d = cf.cf_residual_norm_desc(n, c, cf.CF_NORM_RMS, cf.CF_NORM_LAYER, 1e-5, 0.7, *kind, 0, 0)
        r, h, st, dx, df = out
        cf.cf_residual_norm_fwd(d, x, f, None, r, h, st)
        cf.cf_residual_norm_bwd(d, f, r, None, st, dh, dr, dx, df, None, ws, size)

    def room(n):
        d = cf.cf_residual_norm_desc(n, c, cf.CF_NORM_RMS, cf.CF_NORM_LAYER, 1e-5, 0.7, *kind, 0, 0)
        size = cf.cf_residual_norm_workspace_size(d)
        return (torch.empty((n, c), dtype=dtype, device="cuda"), torch.empty((n, c), dtype=f_dtype, device="cuda"), torch.empty((n, 4), device="cuda"),
                torch.empty((n, c), dtype=dtype, device="cuda"), torch.empty((n, c), dtype=f_dtype, device="cuda")), \
            torch.empty((size,), dtype=torch.uint8, device="cuda"), size

    alone, ws, size = room(few)
    calls(few, *(t[-few:].clone() for t in (x, f, dh, dr)), alone, ws, size)
    out, ws, size = room(rows)
    for _ in range(20):
        for t in out:
            t.fill_(float("nan"))
        calls(rows, x, f, dh, dr, out, ws, size)
        assert all(torch.equal(t[-few:], a) for t, a in zip(out, alone))
    assert cf.cf_last_device_status() == cf.CF_OK
