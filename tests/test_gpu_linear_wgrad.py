"""The backward weight of the products (cf_linear_wgrad) where its sums are taken in many pieces: by CTAs with several tiles each, and
over many rows."""
import numpy as np
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


def call(cf, x, dz, dw, db, scale=1.0, accumulate=0):
    (rows, k), n = x.shape, dz.shape[1]
    d = cf.cf_linear_desc(rows, k, n, cf.CF_ACT_LRELU, 1.0, scale, cf.CF_DT_BF16, x.stride(0), dz.stride(0))
    size = cf.cf_linear_workspace_size(d, cf.CF_LINEAR_WGRAD)
    ws = torch.full((max(size, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    cf.cf_linear_wgrad(d, x, dz, dw, db, accumulate, ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK


def whole(g, shape, most):
    """Whole numbers from -most to most."""
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int32)


# more tiles than CTAs or pairs take at once, of few rows: what is added comes ahead of the products (pairs with several tiles of which
# some take the sums of dz, lone CTAs, tiles one across, ends inside a tile, rows that TMA does not take); the last: cut tiles
SEVERAL = [(8, 16384, 2048), (512, 2048, 8192), (1000, 4096, 4096), (256, 1024, 4096), (1000, 136, 40000), (512, 4096, 4096), (256, 2048, 11008),
           (300, 200, 20000), (40, 264, 30000), (1024, 8192, 8192), (70, 1001, 9000), (64, 20000, 136), (1100, 2056, 4100), (30000, 520, 264)]
# and long sums: cut and whole tiles of pairs and lone CTAs in segments, sides exchanged, rows that TMA does not take
LONG = [(16384, 2048, 2048), (9000, 4096, 4096), (9000, 1041, 4100), (100000, 64, 4096), (20000, 128, 38912), (200000, 64, 72), (50001, 40, 24),
        (200003, 33, 300)]


@pytest.mark.parametrize("rows,k,n", SEVERAL + LONG)
@pytest.mark.parametrize("with_db", [True, False])
@pytest.mark.parametrize("accumulate", [1, 0])
def test_sums_of_whole_numbers_are_exact(cf, rows, k, n, with_db, accumulate):
    """Products of whole numbers up to 3 stay below 2^24 over all rows, so that every fp32 sum holds them and no order or cut rounds; the
    gradients that are there differ from value to value."""
    g = torch.Generator("cuda").manual_seed(rows + k + n)
    x, dz = whole(g, (rows, k), 3).to(BF), whole(g, (rows, n), 3).to(BF)
    (dw, ok_w), (db, ok_b) = guarded((n, k), F32, fill=0.0), guarded((n,), F32, fill=0.0)
    dw.copy_(whole(g, (n, k), 1000)), db.copy_(whole(g, (n,), 1000))
    want_w, want_b = (0.5 * dz.double().T @ x.double(), 0.5 * dz.double().sum(0)) if not accumulate else \
        (dw.double() + 0.5 * dz.double().T @ x.double(), db.double() + 0.5 * dz.double().sum(0))
    left = db.clone()
    call(cf, x, dz, dw, db if with_db else None, 0.5, accumulate)
    ok_w(), ok_b()
    assert torch.equal(dw.double(), want_w)
    assert torch.equal(db.double(), want_b) if with_db else torch.equal(db, left)


# tiles of pairs, whole and cut, of lone CTAs with rows that TMA takes and does not, sides exchanged, cut and whole
@pytest.mark.parametrize("rows,k,n", [(16384, 4096, 4096), (16384, 2048, 2048), (9000, 1040, 4100), (16384, 200, 136), (100000, 64, 4096),
                                      (20000, 128, 38912), (200000, 72, 1000)])
def test_bias_sums_keep_fp32s_precision(cf, rows, k, n):
    """Sums of dz whose rows differ in size by e^3 each way, with a mean of their own.  The tensor cores cut sums off, on average by 2^-24 of
    them, at each of at most 96 steps of 16 rows before they are added up in fp32 that rounds, once for each 1536 rows and a few times where
    a tile is cut; on average a sum is at most 0.7 of its end on the way: (96 + rows / 1536 + 8) 0.7 2^-24 of the result."""
    g = torch.Generator("cuda").manual_seed(rows + k + n)
    size = torch.exp(6 * torch.rand((rows, 1), generator=g, device="cuda") - 3)
    dz = ((torch.randn((rows, n), generator=g, device="cuda") + 0.25) * size).to(BF)
    x = torch.randn((rows, k), generator=g, device="cuda").to(BF)
    dw, db = torch.empty((n, k), device="cuda"), torch.empty(n, device="cuda")
    call(cf, x, dz, dw, db)
    want = sum(dz[i:i + 8192].double().sum(0) for i in range(0, rows, 8192))
    error = float((db.double() - want).norm() / want.norm())
    assert error <= (96 + rows / 1536 + 8) * 0.7 * 2.0 ** -24, f"{error:.2e}"
    # and added to what is there, with the same bits before the addition
    again = torch.full_like(db, 3.0)
    call(cf, x, dz, dw, again, 1.0, 1)
    assert torch.equal(again, db + 3.0)
