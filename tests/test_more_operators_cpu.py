"""Pins of the 64-bit products with an epilogue, residual norms and clipped steps that the GPU tests compare with, and the
refusals of their entry points (no GPU needed)."""
import numpy as np
import pytest

import oracle


# ---------------------------------------------------------------------------------------------------------------------- pins
@pytest.mark.parametrize("act,slope", [("none", 1.0), ("lrelu", 0.3), ("silu", 1.0), ("gelu", 1.0)])
def test_linear_gradients_by_differences(act, slope):
    rng = np.random.default_rng(1)
    x, w, b, res, dy = (rng.normal(size=s) for s in ((5, 7), (6, 7), (6,), (5, 6), (5, 6)))

    def loss(x, w, b):
        return (oracle.linear_fwd(x, w, b, res, act, slope, 0.7)[0] * dy).sum()

    _, z = oracle.linear_fwd(x, w, b, res, act, slope, 0.7)
    dz = 0.7 * dy * oracle.linear_act_grad(z, act, slope)
    dw, db = oracle.linear_wgrad(x, dz)
    h = 1e-6
    for i, grad in enumerate((oracle.linear_dgrad(dz, w), dw, db)):
        args = [x, w, b]
        v = rng.normal(size=args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        np.testing.assert_allclose((loss(*up) - loss(*down)) / (2 * h), (grad * v).sum(), rtol=1e-6)


def test_linear_dgrad_passes_the_layer_below():
    """Two layers: the backward data with the pre-activation below is that layer's dz."""
    rng = np.random.default_rng(2)
    x, w1, w2, dy = (rng.normal(size=s) for s in ((4, 5), (6, 5), (3, 6), (4, 3)))

    def loss(w1):
        return (oracle.linear_fwd(oracle.linear_fwd(x, w1, act="gelu")[0], w2, scale=1.3)[0] * dy).sum()

    z = x @ w1.T
    dw, _ = oracle.linear_wgrad(x, oracle.linear_dgrad(dy, w2, z, None, "gelu", scale=1.3))
    v = rng.normal(size=w1.shape)
    np.testing.assert_allclose((loss(w1 + 1e-6 * v) - loss(w1 - 1e-6 * v)) / 2e-6, (dw * v).sum(), rtol=1e-6)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_agree_with_torch(act):
    import torch
    z = np.linspace(-8, 8, 101)
    t = torch.from_numpy(z)
    ref = torch.nn.functional.silu(t) if act == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    np.testing.assert_allclose(oracle.linear_act(z, act), ref.numpy(), atol=1e-12)


def _vectors(rng, c, post, pre, gate, samples, each):
    vec = {}
    if post != "none":
        vec["post_gamma"] = rng.normal(1, 0.3, c)
    if post == "layer":
        vec["post_beta"] = rng.normal(0, 0.3, c)
    if gate:
        vec["gate"] = rng.normal(0.5, 0.3, (samples, c) if each & 1 else c)
    if pre != "none":
        vec["pre_gamma"] = rng.normal(1, 0.3, (samples, c) if each & 2 else c)
    if pre == "layer":
        vec["pre_beta"] = rng.normal(0, 0.3, (samples, c) if each & 2 else c)
    return vec


@pytest.mark.parametrize("post,pre,gate,each", [("none", "rms", False, 0), ("rms", "layer", True, 0), ("layer", "layer", True, 3),
                                                ("layer", "rms", True, 2), ("rms", "none", True, 1), ("none", "none", True, 0)])
def test_residual_norm_gradients_by_differences(post, pre, gate, each):
    rng = np.random.default_rng(3)
    rows, c, per = 7, 6, 3
    x, f = rng.normal(size=(rows, c)) + 0.4, rng.normal(size=(rows, c)) - 0.2
    vec = _vectors(rng, c, post, pre, gate, 3, each)
    dr, dh = rng.normal(size=(rows, c)), rng.normal(size=(rows, c))
    kw = dict(post=post, pre=pre, scale=0.8, per=per)

    def loss(x, f, vec):
        r, h, _ = oracle.residual_norm_fwd(x, f, vec, **kw)
        return (r * dr).sum() + (0.0 if h is None else (h * dh).sum())

    r, _, _ = oracle.residual_norm_fwd(x, f, vec, **kw)
    dx, df, grads = oracle.residual_norm_bwd(f, r, vec, dh, dr, **kw)
    h = 1e-6
    for name, grad in [("x", dx), ("f", df)] + [(k, grads[k]) for k in vec]:
        v = rng.normal(size=grad.shape)
        e = lambda s: ((x + s * v, f, vec) if name == "x" else (x, f + s * v, vec) if name == "f"  # noqa: E731
                       else (x, f, dict(vec, **{name: vec[name] + s * v})))
        np.testing.assert_allclose((loss(*e(h)) - loss(*e(-h))) / (2 * h), (grad * v).sum(), rtol=2e-6, atol=1e-8, err_msg=name)


def test_residual_norm_closed_forms():
    x = np.array([[3.0, 4.0]])
    r, h, st = oracle.residual_norm_fwd(x, None, {}, pre="rms", eps=0.0)
    np.testing.assert_allclose(h, x / np.sqrt(12.5))
    r, h, st = oracle.residual_norm_fwd(x, np.array([[1.0, 3.0]]), {"gate": np.array([2.0, 10.0])}, post="layer", pre="layer", scale=0.5, eps=0.0)
    np.testing.assert_allclose(r, [[2.0, 9.0]])
    np.testing.assert_allclose(h, [[-1.0, 1.0]])
    np.testing.assert_allclose(st, [[2.0, 1.0, 5.5, 1 / 3.5]])


def test_clip_factor_and_adam_closed_forms():
    assert oracle.clip_factor([np.array([3.0]), np.array([4.0])], 10.0) == (5.0, 1.0)
    norm, f = oracle.clip_factor([np.array([3.0]), np.array([4.0])], 1.0)
    assert norm == 5.0 and abs(f * 5.0 - 1.0) < 1e-6
    w, m, v = oracle.adam_decay_step(np.array([2.0]), np.array([0.5]), 0.0, 0.0, 0.1, 1, eps=0.0, weight_decay=0.5)
    np.testing.assert_allclose([w[0], m[0], v[0]], [2.0 * 0.95 - 0.1, 0.05, 0.00025])


# ------------------------------------------------------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def _lin(cf, **kw):
    d = dict(rows=4, k=8, n=16, act=cf.CF_ACT_GELU, slope=1.0, scale=1.0, dtype=cf.CF_DT_BF16, x_pitch=0, y_pitch=0)
    d.update(kw)
    return cf.cf_linear_desc(*d.values())


def test_linear_refusals(cf):
    bad, un = cf.CF_ERR_INVALID_ARG, cf.CF_ERR_UNSUPPORTED

    def all_of(d):
        st = [cf.cf_linear_fwd(d, 16, 32, None, None, 64, None, check=False), cf.cf_linear_dgrad(d, 16, 32, None, None, 64, check=False),
              cf.cf_linear_wgrad(d, 16, 32, 64, None, check=False), cf.cf_linear_act_bwd(d, 16, 32, 64, check=False)]
        assert len(set(st)) == 1
        assert all(cf.cf_linear_workspace_size(d, op) == 0 for op in range(3))
        return st[0]

    nan, inf = float("nan"), float("inf")
    for kw in (dict(rows=-1), dict(k=0), dict(n=0), dict(k=-4), dict(act=3), dict(act=-1), dict(slope=nan), dict(scale=inf), dict(dtype=2),
               dict(x_pitch=7), dict(y_pitch=15), dict(x_pitch=-8)):
        assert all_of(_lin(cf, **kw)) == bad, kw
    for kw in (dict(rows=1 << 31), dict(k=(1 << 20) + 1), dict(n=1 << 21), dict(x_pitch=1 << 28), dict(y_pitch=1 << 28)):
        assert all_of(_lin(cf, **kw)) == un, kw
    assert all_of(None) == bad
    d = _lin(cf)
    for i in (0, 1, 4):  # a tensor missing; any pointer off 16 bytes
        a = [16, 32, None, None, 64, None]
        a[i] = None
        assert cf.cf_linear_fwd(d, *a, check=False) == bad
    for i in range(6):
        a = [16, 32, 48, 64, 80, 96]
        a[i] += 2
        assert cf.cf_linear_fwd(d, *a, check=False) == bad
    for i in range(5):
        a = [16, 32, 48, 64, 80]
        a[i] += 4
        assert cf.cf_linear_dgrad(d, *a, check=False) == bad
    assert cf.cf_linear_dgrad(d, 16, None, None, None, 64, check=False) == bad
    assert cf.cf_linear_wgrad(d, 16, 32, None, 48, check=False) == bad and cf.cf_linear_wgrad(d, None, 32, 64, None, check=False) == bad
    assert cf.cf_linear_wgrad(d, 16, 32, 64, 40, check=False) == bad
    assert cf.cf_linear_act_bwd(d, 16, None, 64, check=False) == bad
    assert cf.cf_linear_workspace_size(d, 3) == 0 and cf.cf_linear_workspace_size(d, -1) == 0
    for rows in (1, 8, 1000):  # a workspace that is too small
        for k in (8, 130, 4096):
            d = _lin(cf, rows=rows, k=k)
            for op, call in enumerate((lambda ws, n: cf.cf_linear_fwd(d, 16, 32, None, None, 64, None, ws, n, check=False),
                                       lambda ws, n: cf.cf_linear_dgrad(d, 16, 32, None, None, 64, ws, n, check=False),
                                       lambda ws, n: cf.cf_linear_wgrad(d, 16, 32, 64, None, 0, ws, n, check=False))):
                size = cf.cf_linear_workspace_size(d, op)
                if size:
                    assert call(16, size - 1) == cf.CF_ERR_WORKSPACE and call(None, size) == cf.CF_ERR_WORKSPACE
    assert cf.cf_linear_fwd(_lin(cf, rows=0), None, None, None, None, None, None, check=False) == cf.CF_OK
    assert cf.cf_linear_dgrad(_lin(cf, rows=0), None, None, None, None, None, check=False) == cf.CF_OK


def _rn(cf, **kw):
    d = dict(rows=4, c=8, post=cf.CF_NORM_NONE, pre=cf.CF_NORM_RMS, eps=1e-5, scale=1.0, dtype=cf.CF_DT_BF16, f_dtype=cf.CF_DT_BF16,
             per_sample=0, rows_per_sample=0)
    d.update(kw)
    return cf.cf_residual_norm_desc(*d.values())


def test_residual_norm_refusals(cf):
    bad, un = cf.CF_ERR_INVALID_ARG, cf.CF_ERR_UNSUPPORTED
    V = cf.cf_residual_norm_vectors

    def fwd(d, x=16, f=32, v=None, r=48, h=64, stats=80):
        return cf.cf_residual_norm_fwd(d, x, f, v, r, h, stats, check=False)

    def bwd(d, f=16, r=32, v=None, stats=48, dh=64, dr=80, dx=96, df=112, g=None, ws=128, size=1 << 40):
        return cf.cf_residual_norm_bwd(d, f, r, v, stats, dh, dr, dx, df, g, ws, size, check=False)

    for kw in (dict(rows=-1), dict(c=0), dict(post=3), dict(pre=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")),
               dict(dtype=2), dict(f_dtype=-1), dict(per_sample=4), dict(rows_per_sample=-1)):
        assert fwd(_rn(cf, **kw)) == bwd(_rn(cf, **kw)) == bad, kw
        assert cf.cf_residual_norm_workspace_size(_rn(cf, **kw)) == 0
    for kw in (dict(f_dtype=cf.CF_DT_F32), dict(c=65537), dict(rows=1 << 31), dict(rows=1 << 25, per_sample=1, rows_per_sample=1)):
        assert fwd(_rn(cf, **kw)) == bwd(_rn(cf, **kw)) == un, kw
    d = _rn(cf)
    assert fwd(None) == bad and bwd(None) == bad
    assert fwd(d, x=None) == bad and fwd(d, h=None) == bad and fwd(d, x=18) == bad and fwd(d, stats=84) == bad
    assert fwd(_rn(cf, pre=cf.CF_NORM_NONE)) == bad  # h without a norm
    assert fwd(_rn(cf, post=cf.CF_NORM_RMS), f=None) == bad and fwd(d, f=None, v=V(gate=16)) == bad
    assert fwd(d, v=V(post_gamma=16)) == bad and fwd(d, v=V(pre_beta=16)) == bad and fwd(d, v=V(pre_gamma=20)) == bad
    assert bwd(d, stats=None) == bad and bwd(d, dh=None) == bad and bwd(d, r=None) == bad and bwd(d, f=None) == bad
    assert bwd(d, dx=None, df=None) == bad and bwd(d, g=V(post_beta=16)) == bad and bwd(d, dr=81) == bad
    assert bwd(_rn(cf, pre=cf.CF_NORM_NONE), dh=None, dr=None) == bad
    assert bwd(d, ws=None) == cf.CF_ERR_WORKSPACE and bwd(d, size=cf.cf_residual_norm_workspace_size(d) - 1) == cf.CF_ERR_WORKSPACE
    assert fwd(_rn(cf, rows=0), x=None, r=None, h=None) == cf.CF_OK


def test_clip_refusals(cf):
    bad = cf.CF_ERR_INVALID_ARG

    def grads(*entries):
        out = (cf.cf_grad * len(entries))()
        for p, e in zip(out, entries):
            p.g, p.count, p.dtype = e
        return out

    ok = (16, 4, cf.CF_DT_F32)
    for call in (cf.cf_grad_norm, cf.cf_clip_grads):
        for e in ((None, 4, 1), (18, 4, 1), (17, 4, 0), (16, -1, 1), (16, 4, 2)):
            assert call(grads(ok, e), 1.0, 32, 64, 1 << 30, check=False) == bad, e
            assert cf.cf_grad_workspace_size(grads(ok, e)) == 0
        for kw in ((-1.0, 32, 64), (float("nan"), 32, 64), (1.0, None, 64), (1.0, 33, 64), (1.0, 32, 72)):
            assert call(grads(ok), *kw, 1 << 30, check=False) == bad, kw
        size = cf.cf_grad_workspace_size(grads(ok))
        assert call(grads(ok), 1.0, 32, 64, size - 1, check=False) == cf.CF_ERR_WORKSPACE
        assert call(grads(ok), 1.0, 32, None, size, check=False) == cf.CF_ERR_WORKSPACE

    def params(**kw):
        out = (cf.cf_adam_param * 1)()
        for k, v in dict(dict(w=16, w_bf16=None, g=32, m=48, v=64, count=4), **kw).items():
            setattr(out[0], k, v)
        return out

    def adam(p, out=32, ws=64, size=1 << 30, **kw):
        h = cf.cf_adam_hyper(*dict(dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_norm=1.0, t=1), **kw).values())
        return cf.cf_clip_adam_step(p, h, out, ws, size, check=False)

    for kw in (dict(w=None), dict(g=None), dict(m=None), dict(v=None), dict(w=18), dict(w_bf16=17), dict(count=-1)):
        assert adam(params(**kw)) == bad, kw
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(t=0), dict(max_norm=-1.0), dict(lr=float("nan")),
               dict(weight_decay=float("inf")), dict(max_norm=float("nan")), dict(out=None), dict(ws=8)):
        assert adam(params(), **kw) == bad, kw
    assert cf.cf_clip_adam_step(params(), None, 32, 64, 1 << 30, check=False) == bad
    assert adam(params(), size=cf.cf_clip_adam_workspace_size(params()) - 1) == cf.CF_ERR_WORKSPACE


# ------------------------------------------------------------------------------------------------- launches that fail, by a fake runtime
CALLS = """
def grads(n):
    out = (cf.cf_grad * n)()
    for p in out:
        p.g, p.count, p.dtype = 4096, 5000, cf.CF_DT_F32
    return out
def norm(n=3):
    g = grads(n)
    return cf.cf_grad_norm(g, 1.0, 256, 512, cf.cf_grad_workspace_size(g), check=False)
def clip(n=3):
    g = grads(n)
    return cf.cf_clip_grads(g, 1.0, 256, 512, cf.cf_grad_workspace_size(g), check=False)
def adam(n=3, max_norm=1.0):
    out = (cf.cf_adam_param * n)()
    for p in out:
        p.w, p.g, p.m, p.v, p.count = 4096, 8192, 12288, 16384, 3000
    h = cf.cf_adam_hyper(1e-3, 0.9, 0.999, 1e-8, 0.0, max_norm, 1)
    return cf.cf_clip_adam_step(out, h, 256, 512, cf.cf_clip_adam_workspace_size(out), check=False)
def rn(rows, c, back, each=0, per=0, sums=True):
    d = cf.cf_residual_norm_desc(rows, c, cf.CF_NORM_RMS, cf.CF_NORM_RMS, 1e-5, 1.0, 0, 0, each, per)
    if not back:
        return cf.cf_residual_norm_fwd(d, 256, 512, None, 768, 1024, None, check=False)
    g = cf.cf_residual_norm_vectors(gate=2048) if sums else None
    return cf.cf_residual_norm_bwd(d, 256, 512, None, 768, 1024, 1280, 1536, 1792, g, 4096, cf.cf_residual_norm_workspace_size(d), check=False)
"""


@pytest.mark.parametrize("call,launches", [("norm()", 2), ("clip()", 2), ("adam()", 2), ("adam(3, 0.0)", 1), ("norm(2000)", 3), ("clip(2000)", 4),
                                           ("adam(1000)", 4), ("norm(0)", 1), ("rn(64, 256, 0)", 1), ("rn(64, 256, 1)", 2), ("rn(64, 256, 1, sums=False)", 1),
                                           ("rn(64, 256, 1, 1, 32)", 3), ("rn(100000, 128, 0)", 1), ("rn(100000, 128, 1)", 2), ("rn(64, 9000, 0)", 1),
                                           ("rn(64, 9000, 1)", 3)])
def test_a_launch_that_fails_ends_the_call_and_is_reported_once(tmp_path, call, launches):
    """The call says CF_ERR_CUDA, enqueues nothing more, and does not leave the error behind for the next one."""
    from test_operators_cpu import _with_fake_runtime
    script = CALLS + f"fake.fake_set(1, 0)\nprint({call}, fake.fake_launches())\n"
    for at in range(1, launches + 1):
        script += f"fake.fake_set(1, {at})\nprint({call}, fake.fake_launches())\nfake.fake_set(1, 0)\nprint({call})\n"
    want = ["0", str(launches)]
    for at in range(1, launches + 1):
        want += ["4", str(at), "0"]
    assert _with_fake_runtime(tmp_path, script) == want
