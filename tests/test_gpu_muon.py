"""Orthogonalisation and the momentum step through the C ABI against the 64-bit oracle.

Tolerance of an orthogonalised matrix, in the Frobenius norm relative to the result: each of the five steps rounds operands to
11 bits (2^-12 of a value) and a step passes an error on with at most the polynomial's slope 3.45, three roundings a step that
add in squares over the steps: sqrt(3 * 5) * 3.45 * 2^-12 = 3.3e-3.  A bf16 output adds 2^-9 / sqrt(3) * sqrt(2): 1.6e-3.
Together at most 5e-3.  An fp32 weight is off by its own rounding and by 3.3e-3 of the update."""
import numpy as np
import pytest

from tests.gpu_util import guarded

pytestmark = pytest.mark.gpu

NS_TOL, OUT_TOL = 3.3e-3, 5e-3


@pytest.fixture(scope="module")
def cf():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _matrix(rng, shape, kind):
    g = rng.normal(size=shape)
    r = min(min(shape), 16)
    if kind == "directions":  # few directions and noise, as a gradient summed over voxels
        g = 0.1 * g + rng.normal(size=(shape[0], r)) @ rng.normal(size=(r, shape[1])) / r
    elif kind == "decay":  # singular values over four decades
        u, _, vt = np.linalg.svd(g, full_matrices=False)
        g = (u * np.logspace(0, -4, min(shape))) @ vt
    return g


def _orth(cf, g, dtype, steps=5, coef=None, eps=1e-7):
    import torch
    a, b, c = coef or (3.4445, -4.7750, 2.0315)
    batch, rows, cols = g.shape
    t = torch.from_numpy(np.asarray(g, np.float32)).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    desc = cf.cf_ns_desc(batch, rows, cols, cf.CF_DT_BF16 if dtype == "bf16" else cf.CF_DT_F32, steps, a, b, c, eps)
    size = cf.cf_orthogonalize_workspace_size(desc)
    assert size > 0
    o, check = guarded(g.shape, torch.bfloat16, fill=9.0)
    ws, check_ws = guarded((size,), torch.uint8, fill=0xFF)
    cf.cf_orthogonalize(desc, t, o, ws, size)
    torch.cuda.synchronize()
    check("o")
    check_ws("workspace")
    assert cf.cf_last_device_status() == cf.CF_OK
    return _f64(o), _f64(t)


def _check(oracle, o, g, tol=OUT_TOL, **kw):
    for i in range(len(g)):
        ref = oracle.newton_schulz(g[i], **kw)
        assert np.all(np.isfinite(o[i]))
        rel = np.linalg.norm(o[i] - ref) / np.linalg.norm(ref)
        assert rel <= tol, (i, rel)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (5, 3), (8, 8), (16, 108), (27, 16), (32, 432), (63, 65), (64, 864), (100, 37), (127, 129),
          (128, 128), (128, 1728), (129, 300), (130, 4000), (200, 256), (256, 108), (256, 3456), (257, 255), (300, 17), (384, 1000),
          (512, 512), (1000, 333), (640, 2049), (3, 9001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind,dtype", [("normal", "f32"), ("directions", "bf16"), ("decay", "f32")])
def test_orthogonalize(cf, oracle_mod, rows, cols, kind, dtype):
    rng = np.random.default_rng(rows * 10007 + cols)
    o, g = _orth(cf, _matrix(rng, (rows, cols), kind)[None], dtype)
    _check(oracle_mod, o, g)


@pytest.mark.parametrize("batch,rows,cols", [(2, 16, 108), (3, 45, 33), (7, 65, 130), (2, 300, 257), (40, 8, 24), (5, 130, 128)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_batches(cf, oracle_mod, batch, rows, cols, dtype):
    rng = np.random.default_rng(batch)
    g = np.stack([_matrix(rng, (rows, cols), "directions") * 10.0 ** (i - 2) for i in range(batch)])
    o, g = _orth(cf, g, dtype)
    _check(oracle_mod, o, g)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_and_coefficients(cf, oracle_mod, steps):
    rng = np.random.default_rng(3)
    for shape in ((40, 200), (150, 300), (70, 30)):
        o, g = _orth(cf, _matrix(rng, shape, "normal")[None], "f32", steps, (1.5, -0.5, 0.0))
        _check(oracle_mod, o, g, steps=steps, coef=(1.5, -0.5, 0.0))


def test_zero_and_extreme_scales(cf, oracle_mod):
    rng = np.random.default_rng(4)
    for shape in ((20, 50), (200, 400)):
        g = np.stack([np.zeros(shape), _matrix(rng, shape, "normal") * 1e-5, _matrix(rng, shape, "normal") * 1e12])
        o, g = _orth(cf, g, "f32")
        assert np.all(o[0] == 0)
        _check(oracle_mod, o[1:], g[1:])


def test_large_matrix(cf):
    """2048 x 4100 against 64-bit products on the GPU."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = torch.randn((2048, 16), device="cuda", generator=gen) @ torch.randn((16, 4100), device="cuda", generator=gen) / 16
    g += 0.1 * torch.randn((2048, 4100), device="cuda", generator=gen)
    desc = cf.cf_ns_desc(1, 2048, 4100, cf.CF_DT_F32, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    size = cf.cf_orthogonalize_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    o = torch.empty((2048, 4100), dtype=torch.bfloat16, device="cuda")
    cf.cf_orthogonalize(desc, g, o, ws, size)
    x = g.double() / g.double().norm()
    for _ in range(5):
        a = x @ x.T
        x = 3.4445 * x + (-4.7750 * a + 2.0315 * a @ a) @ x
    assert float((o.double() - x).norm() / x.norm()) <= OUT_TOL
    again = torch.empty_like(o)
    cf.cf_orthogonalize(desc, g, again, ws, size)
    torch.cuda.synchronize()
    assert torch.equal(o, again)
    assert cf.cf_last_device_status() == cf.CF_OK


def test_same_bits_again_and_alone_as_in_a_batch(cf):
    rng = np.random.default_rng(6)
    for shape in ((33, 70), (180, 260)):
        g = np.stack([_matrix(rng, shape, "directions") for _ in range(3)])
        a, _ = _orth(cf, g, "f32")
        b, _ = _orth(cf, g, "f32")
        c, _ = _orth(cf, g[1:2], "f32")
        assert np.array_equal(a, b) and np.array_equal(a[1], c[0])


def test_nan_stays_in_its_matrix(cf, oracle_mod):
    rng = np.random.default_rng(7)
    g = np.stack([_matrix(rng, (30, 60), "normal") for _ in range(3)])
    g[1, 3, 4] = np.nan
    o, g = _orth(cf, g, "f32")
    _check(oracle_mod, o[[0, 2]], g[[0, 2]])
    assert np.all(np.isnan(o[1]))


LISTS = [
    [(16, 108)],
    [(32, 108), (64, 864), (128, 1728)],
    [(4, 256), (1, 1), (300, 200), (16, 27), (129, 131)],
    [(256, 3456), (8, 8), (256, 108), (512, 640), (2, 900), (96, 96), (64, 576)],
    [(5 + i, 20 + 3 * i) for i in range(40)],
]


@pytest.mark.parametrize("shapes", LISTS, ids=[str(len(s)) for s in LISTS])
@pytest.mark.parametrize("nesterov,decay", [(True, 0.01), (False, 0.0)])
def test_muon_step(cf, oracle_mod, shapes, nesterov, decay):
    import torch
    rng = np.random.default_rng(len(shapes))
    lr, mu = 0.02, 0.95
    entries, host, checks = [], [], []
    for i, shape in enumerate(shapes):
        w = rng.normal(size=shape) * np.sqrt(2 / shape[1])
        m = _matrix(rng, shape, "directions")
        g = [_matrix(rng, shape, "normal") for _ in range(2)]
        scale = 0.2 * np.sqrt(max(shape))
        bufs = []
        for dt, v in ((torch.float32, w), (torch.bfloat16, w), (torch.float32, g[0]), (torch.float32, m)):
            t, check = guarded(shape, dt)
            t.copy_(torch.from_numpy(v))
            bufs.append(t)
            checks.append(check)
        if i % 3 == 2:
            bufs[1] = None
        entries.append((*bufs, scale))
        host.append([_f64(bufs[0]), _f64(bufs[3]), g, scale])
    params = cf.cf_muon_params(entries)
    hyper = cf.cf_muon_hyper(lr, mu, decay, int(nesterov), 5, 3.4445, -4.7750, 2.0315, 1e-7)
    size = cf.cf_muon_workspace_size(params)
    ws, check = guarded((size,), torch.uint8, fill=0xFF)
    checks.append(check)
    for step in range(2):
        for e, h in zip(entries, host):
            e[2].copy_(torch.from_numpy(h[2][step]))
        before = [(_f64(e[0]), _f64(e[3])) for e in entries]
        cf.cf_muon_step(params, hyper, ws, size)
        torch.cuda.synchronize()
        assert cf.cf_last_device_status() == cf.CF_OK
        for (w, w16, g, m, scale), (w0, m0) in zip(entries, before):
            rw, rm = oracle_mod.muon_step(w0, _f64(g), m0, lr, scale, mu, nesterov, decay)
            assert np.all(np.abs(_f64(m) - rm) <= 2.0 ** -22 * (np.abs(mu * m0) + np.abs(_f64(g))))
            o = (w0 * (1 - lr * decay) - rw) / (lr * scale)
            off = np.linalg.norm(_f64(w) - rw)
            assert off <= NS_TOL * lr * scale * np.linalg.norm(o) + 2.0 ** -22 * np.linalg.norm(w0), (w.shape, off)
            if w16 is not None:
                assert torch.equal(w16, w.to(torch.bfloat16))
    for check in checks:
        check("a tensor of the step")


def test_muon_in_a_cuda_graph_and_on_a_stream(cf):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(8)
    shapes = [(48, 200), (200, 300)]
    w0 = [torch.randn(s, device="cuda", generator=gen) for s in shapes]
    g = [torch.randn(s, device="cuda", generator=gen) for s in shapes]

    def fresh():
        return [t.clone() for t in w0], [torch.zeros_like(t) for t in w0]

    hyper = cf.cf_muon_hyper(0.01, 0.9, 0.1, 1, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    w, m = fresh()
    params = cf.cf_muon_params([(a, None, b, c, 1.0) for a, b, c in zip(w, g, m)])
    size = cf.cf_muon_workspace_size(params)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        cf.cf_muon_step(params, hyper, ws, size)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    w2, m2 = fresh()
    p2 = cf.cf_muon_params([(a, None, b, c, 1.0) for a, b, c in zip(w2, g, m2)])
    s.wait_stream(torch.cuda.current_stream())
    cf.cf_muon_step(p2, hyper, ws, size, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cf.cf_muon_step(p2, hyper, ws, size, torch.cuda.current_stream())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(w + m, w2 + m2):
        assert torch.equal(a, b)


def test_workspace_too_small(cf):
    import torch
    g = torch.randn((40, 50), device="cuda")
    desc = cf.cf_ns_desc(1, 40, 50, cf.CF_DT_F32, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    size = cf.cf_orthogonalize_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    o = torch.empty((40, 50), dtype=torch.bfloat16, device="cuda")
    assert cf.cf_orthogonalize(desc, g, o, ws, size - 1, check=False) == cf.CF_ERR_WORKSPACE
    params = cf.cf_muon_params([(g, None, g.clone(), g.clone(), 1.0)])
    size = cf.cf_muon_workspace_size(params)
    hyper = cf.cf_muon_hyper(0.01, 0.9, 0.0, 1, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    assert cf.cf_muon_step(params, hyper, ws, size - 1, check=False) == cf.CF_ERR_WORKSPACE


# where one way of taking a matrix ends and the next begins; shares of products that end inside tiles; pairs of CTAs
@pytest.mark.parametrize("rows,cols", [(16, 1408), (1409, 16), (17, 40), (512, 32), (32, 513), (64, 4096), (64, 4097), (128, 1536),
                                       (1537, 128), (100, 1500), (1024, 2500), (1200, 1201), (2048, 2600), (2300, 2050)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_orthogonalize_sizes_where_the_way_changes(cf, oracle_mod, rows, cols, dtype):
    rng = np.random.default_rng(rows * 31 + cols)
    o, g = _orth(cf, _matrix(rng, (rows, cols), "normal")[None], dtype)
    _check(oracle_mod, o, g)


def test_result_in_rows_that_start_anywhere(cf, oracle_mod):
    """Outputs whose rows start at 16 bytes, at 32, and at neither."""
    import torch
    rng = np.random.default_rng(12)
    for rows, cols in ((130, 264), (130, 272), (130, 271)):
        desc = cf.cf_ns_desc(1, rows, cols, cf.CF_DT_F32, 5, 3.4445, -4.7750, 2.0315, 1e-7)
        size = cf.cf_orthogonalize_workspace_size(desc)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        g = torch.from_numpy(rng.normal(size=(rows, cols)).astype(np.float32)).cuda()
        for skip in (0, 8, 16):  # 0, 16 and 32 bytes into a buffer
            buf = torch.full((rows * cols + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
            o = buf[skip:skip + rows * cols].view(rows, cols)
            cf.cf_orthogonalize(desc, g, o, ws, size)
            torch.cuda.synchronize()
            assert bool((buf[:skip] == 9).all()) and bool((buf[skip + rows * cols:] == 9).all())
            _check(oracle_mod, _f64(o)[None], _f64(g)[None])


@pytest.mark.parametrize("shapes", [[(2048, 2600), (130, 270), (7, 9)], [(32, 64), (30, 20), (9, 500)], [(1024, 1024), (512, 512), (256, 2304), (3, 5)]],
                         ids=["pairs", "tiny", "shares"])
def test_muon_step_over_the_ways(cf, oracle_mod, shapes):
    test_muon_step(cf, oracle_mod, shapes, True, 0.01)


@pytest.mark.parametrize("rows,cols", [(2048, 2600), (515, 1511), (128, 700), (16, 108)])
def test_same_bits_in_a_cuda_graph_and_again(cf, rows, cols):
    import torch
    rng = np.random.default_rng(rows)
    desc = cf.cf_ns_desc(1, rows, cols, cf.CF_DT_F32, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    size = cf.cf_orthogonalize_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    g = torch.from_numpy(rng.normal(size=(rows, cols)).astype(np.float32)).cuda()
    o = [torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    cf.cf_orthogonalize(desc, g, o[0], ws, size)
    cf.cf_orthogonalize(desc, g, o[1], ws, size)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cf.cf_orthogonalize(desc, g, o[2], ws, size, torch.cuda.current_stream())
    ws.fill_(0xFF)
    o[2].fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])


@pytest.mark.parametrize("rows,cols", [(130, 300), (515, 1511), (2048, 2600), (64, 864)])
def test_workspace_that_starts_at_any_16_bytes(cf, rows, cols):
    """The same bits from a workspace of exactly its size that starts 16, 32 or 240 bytes into a buffer, and nothing beyond its ends
    is written."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows)
    desc = cf.cf_ns_desc(1, rows, cols, cf.CF_DT_F32, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    size = cf.cf_orthogonalize_workspace_size(desc)
    g = torch.randn((rows, cols), device="cuda", generator=gen)
    out = []
    for skip in (0, 16, 32, 240):
        buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        o = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        assert buf.data_ptr() % 256 == 0
        cf.cf_orthogonalize(desc, g, o, buf[skip:skip + size], size)
        torch.cuda.synchronize()
        assert cf.cf_last_device_status() == cf.CF_OK
        assert bool((buf[:skip] == 0xA5).all()) and bool((buf[skip + size:] == 0xA5).all())
        out.append(o)
    assert all(torch.equal(out[0], o) for o in out[1:])


def test_muon_workspace_that_starts_at_any_16_bytes(cf):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(40)
    shapes = [(300, 200), (16, 27), (129, 131), (200, 512)]
    w0, g, m0 = ([torch.randn(s, device="cuda", generator=gen) for s in shapes] for _ in range(3))
    hyper = cf.cf_muon_hyper(0.01, 0.9, 0.1, 1, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    got = []
    for skip in (0, 16, 48):
        w, m = [t.clone() for t in w0], [t.clone() for t in m0]
        params = cf.cf_muon_params([(a, None, b, c, 0.5) for a, b, c in zip(w, g, m)])
        size = cf.cf_muon_workspace_size(params)
        buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        cf.cf_muon_step(params, hyper, buf[skip:skip + size], size)
        torch.cuda.synchronize()
        assert cf.cf_last_device_status() == cf.CF_OK
        assert bool((buf[:skip] == 0xA5).all()) and bool((buf[skip + size:] == 0xA5).all())
        got.append(w + m)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# a shape for each way that a matrix goes: one CTA, a cluster of one and of several CTAs, the whole GPU, pairs of CTAs
WAYS = [(20, 50), (60, 100), (100, 1200), (200, 400), (2048, 2600)]


@pytest.mark.parametrize("rows,cols", WAYS)
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-7, 4.0])
def test_values_whose_squares_underflow_or_overflow(cf, oracle_mod, rows, cols, eps):
    """The norm of values down to fp32's smallest normal ones and up to 1e30, and of zeros, beside an eps of any size.  Where eps is
    by far the larger, X is near 0 and its values are held to 2^-33 / tau, sqrt(k n) / tau being 4 to 8: over the steps, each of
    which passes that on with at most 3.45, sqrt(5) 8 3.45^5 2^-33 = 1e-6 in the Frobenius norm."""
    rng = np.random.default_rng(rows)
    base = rng.normal(size=(rows, cols))
    eps = float(np.float32(eps))
    scales = [1e-37, 1e-25, 1e-16, 1e30] if rows < 1000 else [1e-25]
    g = np.stack([np.zeros((rows, cols))] + [base * s for s in scales])
    o, g = _orth(cf, g, "f32", eps=eps)
    assert np.all(o[0] == 0)
    for i in range(1, len(g)):
        ref = oracle_mod.newton_schulz(g[i], eps=eps)
        assert np.linalg.norm(o[i] - ref) <= OUT_TOL * np.linalg.norm(ref) + 1e-6, scales[i - 1]


@pytest.mark.parametrize("rows,cols", WAYS[:-1])
def test_muon_step_of_tiny_and_zero_momenta(cf, oracle_mod, rows, cols):
    import torch
    rng = np.random.default_rng(cols)
    m0 = [np.zeros((rows, cols)), rng.normal(size=(rows, cols)) * 1e-26]
    w = [torch.zeros((rows, cols), device="cuda") for _ in m0]
    m = [torch.from_numpy(v.astype(np.float32)).cuda() for v in m0]
    g = [torch.zeros((rows, cols), device="cuda") for _ in m0]
    params = cf.cf_muon_params([(a, None, b, c, 1.0) for a, b, c in zip(w, g, m)])
    size = cf.cf_muon_workspace_size(params)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    m64 = _f64(m[1])
    cf.cf_muon_step(params, cf.cf_muon_hyper(1.0, 0.5, 0.0, 0, 5, 3.4445, -4.7750, 2.0315, 0.0), ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    assert bool((w[0] == 0).all()) and bool((m[0] == 0).all())
    ref = oracle_mod.newton_schulz(0.5 * m64, eps=0.0)
    assert np.linalg.norm(_f64(w[1]) + ref) <= NS_TOL * np.linalg.norm(ref)


def _precise(cf, shapes, kind, seed):
    """Orthogonalised matrices as fp32, as the step from weights of zero writes them, and the matrices."""
    import torch
    rng = np.random.default_rng(seed)
    g = [torch.from_numpy(_matrix(rng, s, kind).astype(np.float32)).cuda() for s in shapes]
    w, m = [torch.zeros_like(t) for t in g], [torch.zeros_like(t) for t in g]
    params = cf.cf_muon_params([(a, None, b, c, 1.0) for a, b, c in zip(w, g, m)])
    size = cf.cf_muon_workspace_size(params)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    cf.cf_muon_step(params, cf.cf_muon_hyper(1.0, 0.0, 0.0, 0, 5, 3.4445, -4.7750, 2.0315, 1e-7), ws, size)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    return [-_f64(t) for t in w], [_f64(t) for t in g]


# The stated precision.  fp16 operands and X to 2^-20: the roundings simulated in 64 bits give 4e-4 to 1.3e-3 over such shapes and
# kinds of matrices, and 5e-3 to 2e-2 for the third kind where X is carried as its operand alone; half as much again, 2e-3.  fp32
# throughout: roundings of sums of up to 1408 terms, at most about 2^-19 each, sqrt(3 * 5) * 3.45 * 2^-19 = 2.6e-5 as above, with
# room for the early steps' that several steps pass on, 1e-4.
@pytest.mark.parametrize("shape,tol", [((16, 108), 1e-4), ((20, 50), 1e-4), ((1408, 16), 1e-4), ((32, 512), 1e-4), ((32, 513), 2e-3),
                                       ((64, 864), 2e-3), ((128, 432), 2e-3), ((100, 1200), 2e-3), ((130, 300), 2e-3), ((515, 1511), 2e-3),
                                       ((2000, 300), 2e-3), ((2048, 2600), 2e-3)])
@pytest.mark.parametrize("kind", ["normal", "directions", "decay"])
def test_precision(cf, oracle_mod, shape, tol, kind):
    (o,), (g,) = _precise(cf, [shape], kind, shape[0] + shape[1])
    ref = oracle_mod.newton_schulz(g)
    assert np.linalg.norm(o - ref) <= tol * np.linalg.norm(ref), np.linalg.norm(o - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("shapes,tol", [([(16, 108), (12, 1400)], 1e-4), ([(16, 108), (31, 40), (512, 30)], 1e-4), ([(16, 108), (17, 600)], 2e-3),
                                        ([(16, 108), (300, 200)], 2e-3)])
def test_precision_of_a_list(cf, oracle_mod, shapes, tol):
    """A list is taken as a whole: its largest matrix says how."""
    for o, g in zip(*_precise(cf, shapes, "directions", len(shapes))):
        ref = oracle_mod.newton_schulz(g)
        assert np.linalg.norm(o - ref) <= tol * np.linalg.norm(ref), (o.shape, np.linalg.norm(o - ref) / np.linalg.norm(ref))


def test_more_matrices_than_a_launch_takes(cf, oracle_mod):
    """A batch of 100 in three launches, whose workspaces follow one another; the same bits as a few of them alone."""
    rng = np.random.default_rng(50)
    g = np.stack([_matrix(rng, (130, 140), "directions") for _ in range(100)])
    o, g = _orth(cf, g, "f32")
    _check(oracle_mod, o, g)
    few, _ = _orth(cf, g[46:50], "f32")
    assert np.array_equal(few, o[46:50])


MANY = {"one above 128 rows": [(20 + i, 30 + 2 * i) for i in range(59)] + [(150, 200)], "small": [(3 + i, 10 + 5 * i) for i in range(60)],
        "tiny": [(1 + i % 16, 16 + i) for i in range(60)], "large last": [(140, 150)] * 48 + [(300, 500), (2, 7)]}


@pytest.mark.parametrize("shapes", list(MANY.values()), ids=list(MANY))
def test_muon_step_of_more_matrices_than_a_launch_takes(cf, oracle_mod, shapes):
    test_muon_step(cf, oracle_mod, shapes, True, 0.01)


@pytest.mark.parametrize("batch,rows,cols", [(1, 130, 300), (2, 515, 1511), (1, 2048, 2600), (60, 130, 140)])
def test_laid_out_workspace_too_small(cf, batch, rows, cols):
    import torch
    g = torch.zeros((batch, rows, cols), device="cuda")
    o = torch.full((batch, rows, cols), 9.0, dtype=torch.bfloat16, device="cuda")
    desc = cf.cf_ns_desc(batch, rows, cols, cf.CF_DT_F32, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    size = cf.cf_orthogonalize_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert cf.cf_orthogonalize(desc, g, o, ws, size - 1, check=False) == cf.CF_ERR_WORKSPACE
    entries = [tuple(torch.zeros((rows, cols), device="cuda") for _ in range(3)) for _ in range(batch)]
    params = cf.cf_muon_params([(w, None, u, m, 1.0) for w, u, m in entries])
    size = cf.cf_muon_workspace_size(params)
    hyper = cf.cf_muon_hyper(0.01, 0.9, 0.0, 1, 5, 3.4445, -4.7750, 2.0315, 1e-7)
    assert cf.cf_muon_step(params, hyper, ws, size - 1, check=False) == cf.CF_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((o == 9).all()) and cf.cf_last_device_status() == cf.CF_OK


FEW = [(1, 1), (1, 3), (2, 2), (4, 2), (3, 3), (4, 8), (8, 8), (9, 100), (16, 108), (16, 512), (512, 5), (1, 512)]


@pytest.mark.parametrize("larger", [(17, 40), (64, 576), (16, 513), (300, 200), (2048, 2600)])
def test_matrices_of_few_values_beside_larger_ones(cf, oracle_mod, larger):
    """They run in fp32 whatever else is in the list: the 1e-4 of test_precision, and the bits of a list of their own."""
    shapes = FEW * 5 + [larger]
    o, g = _precise(cf, shapes, "normal", larger[1])
    for a, b in list(zip(o, g))[:-1]:
        ref = oracle_mod.newton_schulz(b)
        assert np.linalg.norm(a - ref) <= 1e-4 * np.linalg.norm(ref), (a.shape, np.linalg.norm(a - ref) / np.linalg.norm(ref))
    ref = oracle_mod.newton_schulz(g[-1])
    assert np.linalg.norm(o[-1] - ref) <= 2e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("larger", [(33, 40), (300, 200)])
def test_matrices_of_few_values_end_with_the_step(cf, larger):
    """What is enqueued after the step sees them done, on a stream and in a CUDA graph, and they have the bits of a list of their own."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(60)
    shapes = [(16, 512), (3, 40)] * 30 + [larger]
    w0, g, m0 = ([torch.randn(s, device="cuda", generator=gen) for s in shapes] for _ in range(3))
    hyper = cf.cf_muon_hyper(0.01, 0.9, 0.1, 1, 16, 1.5, -0.5, 0.0, 1e-7)

    def entries(w, m, count):
        return cf.cf_muon_params([(a, None, b, c, 0.5) for a, b, c in zip(w, g, m)][:count])

    def fresh():
        return [t.clone() for t in w0], [t.clone() for t in m0]

    w, m = fresh()
    alone = entries(w, m, len(shapes) - 1)
    size = cf.cf_muon_workspace_size(alone)
    cf.cf_muon_step(alone, hyper, torch.empty(size, dtype=torch.uint8, device="cuda"), size)
    want = w[:-1] + m[:-1]
    torch.cuda.synchronize()
    w, m = fresh()
    params = entries(w, m, len(shapes))
    size = cf.cf_muon_workspace_size(params)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cf.cf_muon_step(params, hyper, ws, size, s)
        got = [t.clone() for t in w[:-1] + m[:-1]]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cf.cf_muon_step(params, hyper, ws, size, torch.cuda.current_stream())
        got = [t.clone() for t in w[:-1] + m[:-1]]
    for a, b in zip(w + m, w0 + m0):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows,cols", WAYS)
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_what_is_not_finite_stays_in_its_matrix(cf, rows, cols, value):
    rng = np.random.default_rng(70)
    g = np.stack([_matrix(rng, (rows, cols), "normal") for _ in range(3)])
    clean, _ = _orth(cf, g, "f32")
    g[1, rows // 2, cols - 1] = value
    o, _ = _orth(cf, g, "f32")
    assert np.array_equal(o[[0, 2]], clean[[0, 2]])
    assert np.all(np.isnan(o[1]))
