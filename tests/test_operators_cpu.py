"""Pins of the 64-bit group norm, Newton-Schulz and momentum step that the GPU tests compare with, and the refusals of their
entry points (no GPU needed).  Each pin compares with something else: closed forms, invariances, finite differences, the
singular values."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _case(seed, shape, groups):
    rng = np.random.default_rng(seed)
    c = shape[-1]
    return rng, rng.normal(size=shape) * 2 + 0.5, rng.normal(1, 0.3, c), rng.normal(0, 0.3, c)


def test_group_norm_normalises_each_group():
    rng, x, _, _ = _case(1, (2, 3, 4, 5, 6), 3)
    y, mean, rstd = oracle.group_norm_fwd(x, np.ones(6), np.zeros(6), 3, slope=1.0, eps=0.0)
    for n in range(2):
        for g in range(3):
            v = y[n, ..., 2 * g:2 * g + 2]
            assert abs(v.mean()) < 1e-12 and abs(v.var() - 1) < 1e-12
    # shift and scale of a group's input change nothing but the statistics
    y2, _, _ = oracle.group_norm_fwd(3 * x + 7, np.ones(6), np.zeros(6), 3, slope=1.0, eps=0.0)
    np.testing.assert_allclose(y2, y, atol=1e-12)


def test_group_norm_of_one_voxel_is_a_norm_over_the_channels():
    rng, x, gamma, beta = _case(2, (3, 1, 1, 1, 8), 1)
    y, _, _ = oracle.group_norm_fwd(x, gamma, beta, 1, slope=1.0)
    v = x.reshape(3, 8)
    ref = (v - v.mean(1, keepdims=True)) / np.sqrt(v.var(1, keepdims=True) + 1e-5) * gamma + beta
    np.testing.assert_allclose(y.reshape(3, 8), ref, rtol=1e-12)


def test_group_norm_with_a_group_per_channel_and_one_sample_is_batch_norm():
    rng, x, gamma, beta = _case(3, (1, 3, 4, 2, 5), 5)
    u, _, _ = oracle.bn_fwd(x, gamma, beta)
    y, _, _ = oracle.group_norm_fwd(x, gamma, beta, 5, slope=0.3)
    np.testing.assert_allclose(y, np.where(u > 0, u, 0.3 * u), atol=1e-12)


@pytest.mark.parametrize("pool,act", [("none", "lrelu"), ("none", "silu"), ("max", "lrelu"), ("avg", "lrelu"), ("avg", "silu")])
def test_group_norm_backward_by_differences(pool, act):
    rng, x, gamma, beta = _case(4, (2, 2, 4, 2, 6), 2)
    y, _, _ = oracle.group_norm_fwd(x, gamma, beta, 2, pool, act)
    dy = rng.normal(size=y.shape)
    grads = oracle.group_norm_bwd(x, gamma, beta, 2, dy, pool, act)

    def loss(x, gamma, beta):
        return (oracle.group_norm_fwd(x, gamma, beta, 2, pool, act)[0] * dy).sum()

    args, h = [x, gamma, beta], 1e-6
    for i, grad in enumerate(grads):
        v = rng.normal(size=args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        np.testing.assert_allclose((loss(*up) - loss(*down)) / (2 * h), (grad * v).sum(), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (1, 1)])
def test_newton_schulz_maps_the_singular_values(shape):
    g = np.random.default_rng(5).normal(size=shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    t = s / (np.linalg.norm(g) + 1e-7)
    for _ in range(5):
        a, b, c = oracle.NS_COEFFICIENTS
        t = a * t + b * t ** 3 + c * t ** 5
    np.testing.assert_allclose(oracle.newton_schulz(g), (u * t) @ vt, atol=1e-10)
    assert np.array_equal(oracle.newton_schulz(np.zeros(shape)), np.zeros(shape))


def test_newton_schulz_is_invariant_to_scale_and_rotation():
    rng = np.random.default_rng(6)
    g = rng.normal(size=(5, 12))
    q, _ = np.linalg.qr(rng.normal(size=(5, 5)))
    np.testing.assert_allclose(oracle.newton_schulz(1e3 * g, eps=0.0), oracle.newton_schulz(g, eps=0.0), atol=1e-12)
    np.testing.assert_allclose(oracle.newton_schulz(q @ g), q @ oracle.newton_schulz(g), atol=1e-11)


def test_muon_step_closed_forms():
    rng = np.random.default_rng(7)
    w, g = rng.normal(size=(4, 7)), rng.normal(size=(4, 7))
    w1, m1 = oracle.muon_step(w, g, np.zeros_like(w), 0.1, 2.0, momentum=0.9, nesterov=False, weight_decay=0.5)
    np.testing.assert_allclose(m1, g)
    np.testing.assert_allclose(w1, 0.95 * w - 0.2 * oracle.newton_schulz(g))
    w2, m2 = oracle.muon_step(w, g, m1, 0.1, 2.0, momentum=0.9, nesterov=True)
    np.testing.assert_allclose(m2, 1.9 * g)
    np.testing.assert_allclose(w2, w - 0.2 * oracle.newton_schulz(g), atol=1e-7)  # any multiple of g has its update


# ------------------------------------------------------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def _gn(cf, **kw):
    d = dict(n=1, d=4, h=4, w=4, c=8, groups=2, pool=cf.CF_POOL_NONE, act=cf.CF_ACT_LRELU, slope=0.3, eps=1e-5,
             dtype=cf.CF_DT_BF16, x_pitch=0, y_pitch=0)
    d.update(kw)
    return cf.cf_gn_desc(*d.values())


def test_group_norm_refusals(cf):
    bad, un, ws = cf.CF_ERR_INVALID_ARG, cf.CF_ERR_UNSUPPORTED, cf.CF_ERR_WORKSPACE

    def both(desc, x=16, y=32, stat=48):
        f = cf.cf_group_norm_fwd(desc, x, None, None, y, None, None, check=False)
        b = cf.cf_group_norm_bwd(desc, x, None, None, stat, stat, y, 64, None, None, check=False)
        assert f == b
        return f

    for kw in (dict(n=0), dict(d=0), dict(c=0), dict(groups=0), dict(groups=3), dict(n=70000), dict(pool=5), dict(pool=-1),
               dict(act=2), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(slope=float("nan")), dict(x_pitch=7),
               dict(y_pitch=4), dict(x_pitch=-8), dict(h=1 << 21)):
        assert both(_gn(cf, **kw)) == bad, kw
        assert cf.cf_group_norm_workspace_size(_gn(cf, **kw), 0) == 0
    for kw in (dict(pool=cf.CF_POOL_MAX, d=3), dict(pool=cf.CF_POOL_AVG, w=5), dict(pool=cf.CF_POOL_MAX, dtype=cf.CF_DT_F32),
               dict(pool=cf.CF_POOL_MAX, act=cf.CF_ACT_SILU), dict(pool=cf.CF_POOL_MAX, slope=-0.1)):
        assert both(_gn(cf, **kw)) == un, kw
        assert cf.cf_group_norm_workspace_size(_gn(cf, **kw), 1) == 0
    assert both(None) == bad
    assert both(_gn(cf), x=None) == bad and both(_gn(cf), y=None) == bad
    assert both(_gn(cf), x=18) == bad and both(_gn(cf), y=40) == bad
    assert cf.cf_group_norm_bwd(_gn(cf), 16, None, None, None, 16, 32, 64, None, None, check=False) == bad
    assert cf.cf_group_norm_fwd(_gn(cf), 16, 20, None, 32, None, None, check=False) == bad
    assert ws == 3


def test_orthogonalize_refusals(cf):
    def call(batch=1, rows=4, cols=8, dtype=1, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, g=16, o=32, ws=None):
        return cf.cf_orthogonalize(cf.cf_ns_desc(batch, rows, cols, dtype, steps, a, b, c, eps), g, o, ws, 0, check=False)

    for kw in (dict(batch=0), dict(rows=0), dict(cols=-1), dict(dtype=3), dict(steps=0), dict(a=float("nan")),
               dict(b=float("inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(g=None), dict(o=None), dict(g=8), dict(o=33),
               dict(ws=8)):
        assert call(**kw) == cf.CF_ERR_INVALID_ARG, kw
    assert call(rows=70000) == cf.CF_ERR_UNSUPPORTED and call(steps=17) == cf.CF_ERR_UNSUPPORTED
    assert cf.cf_orthogonalize(None, 16, 32, check=False) == cf.CF_ERR_INVALID_ARG
    assert call() == cf.CF_ERR_WORKSPACE


class _Fake:
    """Something with an address and a shape, for argument checks that launch nothing."""

    def __init__(self, ptr, *shape):
        self.ptr, self.shape = ptr, shape

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return int(np.prod(self.shape))


def test_muon_refusals(cf):
    def entry(w=16, w16=32, g=48, m=64, shape=(4, 8), scale=1.0):
        return (_Fake(w, *shape), w16, g, m, scale)

    def hyper(lr=1e-3, mu=0.9, wd=0.0, steps=5, a=3.4):
        return cf.cf_muon_hyper(lr, mu, wd, 1, steps, a, -4.7, 2.0, 1e-7)

    def call(e, h, ws=None):
        return cf.cf_muon_step(cf.cf_muon_params(e), h, ws, 0, check=False)

    bad = cf.CF_ERR_INVALID_ARG
    assert call([], hyper()) == cf.CF_OK
    for e in (entry(w=0), entry(g=None), entry(m=None), entry(w=20), entry(w16=34), entry(m=65), entry(scale=float("nan"))):
        assert call([entry(), e], hyper()) == bad
    for h in (hyper(lr=float("nan")), hyper(mu=float("inf")), hyper(wd=float("nan")), hyper(steps=0), hyper(a=float("nan"))):
        assert call([entry()], h) == bad
    assert cf.cf_muon_step(cf.cf_muon_params([entry()]), None, check=False) == bad
    assert call([entry()], hyper(), ws=4) == bad
    assert call([entry(shape=(70000, 2))], hyper()) == cf.CF_ERR_UNSUPPORTED
    assert call([entry()], hyper(steps=20)) == cf.CF_ERR_UNSUPPORTED
    assert call([entry()], hyper()) == cf.CF_ERR_WORKSPACE
    p = cf.cf_muon_params([(_Fake(16, 8, 3, 3, 3, 4), None, 48, 64, 0.5)])
    assert (p[0].rows, p[0].cols, p[0].w_bf16, p[0].scale) == (8, 108, None, 0.5)


def _refused(cf, desc):
    """Whether all three entry points refuse the descriptor as unsupported."""
    status = [cf.cf_group_norm_fwd(desc, 16, None, None, 32, None, None, 48, 1 << 62, check=False),
              cf.cf_group_norm_bwd(desc, 16, None, None, 48, 48, 32, 64, None, None, 80, 1 << 62, check=False)]
    sizes = [cf.cf_group_norm_workspace_size(desc, b) for b in (0, 1)]
    return status == [cf.CF_ERR_UNSUPPORTED] * 2 and sizes == [0, 0]


def test_group_norm_refuses_samples_of_2_to_32_windows(cf):
    """A window's number is divided in 32 bits."""
    for pool in (cf.CF_POOL_MAX, cf.CF_POOL_AVG):
        for d, h, w in ((3300, 3300, 3300), (1 << 12, 1 << 12, 1 << 11), (1 << 20, 1 << 15, 2)):
            assert _refused(cf, _gn(cf, d=d, h=h, w=w, c=1, groups=1, pool=pool)), (d, h, w)
        assert cf.cf_group_norm_workspace_size(_gn(cf, d=1 << 12, h=1 << 12, w=(1 << 11) - 2, c=1, groups=1, pool=pool), 0) > 0
    assert cf.cf_group_norm_workspace_size(_gn(cf, d=3300, h=3300, w=3300, c=1, groups=1), 0) > 0


def test_group_norm_refuses_more_blocks_than_a_launch_has(cf):
    """2^60 voxels are 2^46 chunks, of which an int held none; 65535 x 65537 groups, and 2^27 chunks of 16 samples, wrapped too."""
    side = 1 << 20
    for kw in (dict(d=side, h=side, w=side, c=1, groups=1), dict(n=65535, d=1, h=1, w=1, c=65537, groups=65537),
               dict(n=16, d=1 << 14, h=1 << 14, w=1 << 13, c=1, groups=1), dict(n=1, d=1, h=1, w=1, c=1 << 30, groups=1)):
        assert _refused(cf, _gn(cf, **kw)), kw
    # as much as a device holds
    assert cf.cf_group_norm_workspace_size(_gn(cf, n=65535, d=128, h=128, w=128, c=1, groups=1), 1) > 0
    assert cf.cf_group_norm_workspace_size(_gn(cf, n=4096, d=1, h=1, w=1, c=8192, groups=32), 0) > 0


# ------------------------------------------------------------------------------------------------- launches that fail, by a fake runtime
# Stands in for the CUDA runtime's calls, with no GPU: counts launches, fails the one of a given number, and says how many blocks
# a device holds at once.
FAKE_RUNTIME = """
static int launches, fail_at, fit = 1, last;
int fake_launches(void) { return launches; }
void fake_set(int f, int at) { fit = f; fail_at = at; launches = 0; }
static int launch(void) { return ++launches == fail_at ? (last = 98) : 0; }
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int a, int d) { *v = 152; return 0; }
int cudaGetSymbolAddress(void** p, const void* s) { static int word; *p = &word; return 0; }
int cudaGetDriverEntryPointByVersion(const char* s, void** fn, unsigned v, unsigned long long f, int* q) { *fn = (void*)1; *q = 0; return 0; }
int cudaFuncSetAttribute(const void* f, int a, int v) { return 0; }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
int cudaLaunchKernelExC(const void* c, const void* f, void** a) { return launch(); }
int __cudaLaunchKernel() { return launch(); }
int __cudaGetKernel(void** k, const void* f) { *k = (void*)f; return 0; }
unsigned __cudaPushCallConfiguration() { return 0; }
int __cudaPopCallConfiguration() { return 0; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int t, unsigned long s, unsigned g) { *n = fit; return 0; }
int cudaOccupancyMaxActiveClusters(int* n, const void* f, const void* c) { *n = 76 * fit; return 0; }
"""


def _with_fake_runtime(tmp_path, script):
    """Runs the script with `cf` (the binding) and `fake` (the fake runtime's controls); returns what it prints."""
    from cnn_conv3d_gb300 import build
    build.build()
    src, lib = tmp_path / "fake.c", tmp_path / "fake.so"
    src.write_text(FAKE_RUNTIME)
    subprocess.run(["gcc", "-w", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    head = f"import ctypes, sys\nsys.path.insert(0, {ROOT!r})\nfake = ctypes.CDLL({str(lib)!r})\nfrom cnn_conv3d_gb300 import cfconv as cf\n"
    r = subprocess.run([sys.executable, "-c", head + textwrap.dedent(script)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, LD_PRELOAD=str(lib)))
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.split()


# 200 x 400 on single CTAs, 2048 x 2600 on pairs, the two in one list
MUON_CALL = """
def muon(shapes):
    params = (cf.cf_muon_param * len(shapes))()
    for p, (p.rows, p.cols) in zip(params, shapes):
        p.w, p.g, p.m, p.scale = 512, 1024, 2048, 1.0
    hyper = cf.cf_muon_hyper(1e-3, 0.9, 0.0, 1, 5, 3.4, -4.7, 2.0, 1e-7)
    return cf.cf_muon_step(params, hyper, 4096, cf.cf_muon_workspace_size(params), check=False)
"""


@pytest.mark.parametrize("shapes,launches", [([(200, 400)], 3), ([(2048, 2600)], 3), ([(200, 400)] * 50 + [(2048, 2600)], 6), ([(16, 108)], 1)])
def test_muon_step_enqueues_all_or_nothing(tmp_path, shapes, launches):
    """On a device that does not hold the cooperative launch nothing is enqueued: no momentum without its update."""
    call = MUON_CALL + f"fake.fake_set(%d, 0)\nprint(muon({shapes!r}), fake.fake_launches())"
    assert _with_fake_runtime(tmp_path, call % 1) == ["0", str(launches)]
    if launches > 1:
        assert _with_fake_runtime(tmp_path, call % 0) == ["4", "0"]


@pytest.mark.parametrize("shape,at", [((16, 108), 1), ((64, 864), 1), ((200, 400), 1), ((200, 400), 2), ((200, 400), 3), ((2048, 2600), 3)])
def test_a_launch_that_fails_is_reported_once(tmp_path, shape, at):
    """The call says CF_ERR_CUDA and enqueues nothing more, and the error is not left behind for the next one to report as its own."""
    call = MUON_CALL + f"""
gn = cf.cf_gn_desc(1, 4, 4, 4, 8, 2, cf.CF_POOL_NONE, cf.CF_ACT_LRELU, 0.3, 1e-5, cf.CF_DT_BF16, 0, 0)
fake.fake_set(1, {at})
print(muon([{shape!r}]), fake.fake_launches())
fake.fake_set(1, 0)
print(cf.cf_group_norm_fwd(gn, 16, None, None, 32, None, None, 256, 1 << 20, check=False))
print(muon([{shape!r}]))
"""
    assert _with_fake_runtime(tmp_path, call) == ["4", str(at), "0", "0"]


@pytest.mark.parametrize("shapes,launches", [([(16, 108), (200, 400)], 4), ([(2, 3)] * 50 + [(2048, 2600)], 5), ([(3, 3), (64, 576)], 2),
                                             ([(16, 512)], 1), ([(16, 512), (30, 30)], 1)])
def test_muon_step_with_matrices_of_few_values_enqueues_all_or_nothing(tmp_path, shapes, launches):
    call = MUON_CALL + f"fake.fake_set(%d, 0)\nprint(muon({shapes!r}), fake.fake_launches())"
    assert _with_fake_runtime(tmp_path, call % 1) == ["0", str(launches)]
    if max(min(s) for s in shapes) > 128:  # the cooperative launch, on a device that does not hold it
        assert _with_fake_runtime(tmp_path, call % 0) == ["4", "0"]
