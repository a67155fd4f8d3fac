"""Residual blocks of norms and products (VoxelMLP), and the training step of a CosmoFlowModel with them and with clipped gradients:
the library's calls one after another, each against 64 bits on the GPU's own inputs of it."""
import numpy as np
import pytest

import oracle
import synthdata

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
CHANNELS = (4, 32, 64)
SPECS = [(1, "max"), (1, "max", "gn")]
# A stored bf16 value is off by at most 2^-8 of itself, and so is a tensor of them in the 2-norm; what is summed from such values
# in fp32 before adds far less (a relative 1e-4 of sums of the sizes here).
BF16 = 2.0 ** -8 + 1e-4
# Gradients through a norm take its statistics from before the stream's rounding, the check from after it: values off by 2^-8 are a
# mean square, and so a width, off by at most 2^-7.
THROUGH = 2.0 ** -7 + BF16


@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    rel = np.linalg.norm(f64(got).reshape(want.shape) - want) / max(np.linalg.norm(want), 1e-30)
    assert rel <= tol, f"{what}: {rel:.2e}"


def fill(mix, seed):
    rng = np.random.default_rng(seed)
    for ts, mean, width in ((mix.w1, 0, 1 / np.sqrt(mix.c)), (mix.w2, 0, 1 / np.sqrt(mix.wide)), (mix.b1, 0, 0.2), (mix.b2, 0, 0.2),
                            (mix.gamma, 1, 0.2), (mix.post, 1, 0.2), (mix.gate, 0.5, 0.2)):
        for t in ts:
            t.copy_(torch.from_numpy(rng.normal(mean, width, tuple(t.shape))))
    mix.sync_master()
    return rng


def check_mixer(mix, x, dr, dx):
    """Every call of a forward and a backward, from the buffers that they left."""
    X, eps = f64(x).reshape(mix.rows, mix.c), mix.eps
    stream = X
    _, h, _ = oracle.residual_norm_fwd(X, None, {"pre_gamma": f64(mix.gamma[0])}, pre="rms", eps=eps)
    close(mix.h[0], h, BF16, "first norm")
    for l in range(mix.blocks):
        last = l + 1 == mix.blocks
        a, z = oracle.linear_fwd(f64(mix.h[l]), f64(mix.w1_16[l]), f64(mix.b1[l]), act="gelu")
        close(mix.z[l], z, BF16, f"z {l}")
        close(mix.a[l], a, BF16, f"a {l}")
        close(mix.f[l], oracle.linear_fwd(f64(mix.a[l]), f64(mix.w2_16[l]), f64(mix.b2[l]))[0], BF16, f"f {l}")
        vec = {"post_gamma": f64(mix.post[l]), "gate": f64(mix.gate[l])}
        if not last:
            vec["pre_gamma"] = f64(mix.gamma[l + 1])
        r, h, _ = oracle.residual_norm_fwd(stream, f64(mix.f[l]), vec, "rms", "none" if last else "rms", eps=eps)
        close(mix.r[l], r, BF16, f"stream {l}")
        if not last:
            close(mix.h[l + 1], h, BF16, f"norm {l + 1}")
        stream = f64(mix.r[l])
    # the backward, whole: each block's gradients from the stream's before it, which the GPU has rounded on the way
    dh, dr = None, f64(dr).reshape(mix.rows, mix.c)
    tol = THROUGH
    for l in range(mix.blocks - 1, -1, -1):
        last = l + 1 == mix.blocks
        vec = {"post_gamma": f64(mix.post[l]), "gate": f64(mix.gate[l])}
        if not last:
            vec["pre_gamma"] = f64(mix.gamma[l + 1])
        dr, df, g = oracle.residual_norm_bwd(f64(mix.f[l]), f64(mix.r[l]), vec, dh, dr, "rms", "none" if last else "rms", eps=eps)
        close(mix.dpost[l], g["post_gamma"], tol, f"dpost {l}")
        close(mix.dgate[l], g["gate"], tol, f"dgate {l}")
        if not last:
            close(mix.dgamma[l + 1], g["pre_gamma"], tol, f"dgamma {l + 1}")
        dw2, db2 = oracle.linear_wgrad(f64(mix.a[l]), df)
        dz = oracle.linear_dgrad(df, f64(mix.w2_16[l]), f64(mix.z[l]), act="gelu")
        dw1, db1 = oracle.linear_wgrad(f64(mix.h[l]), dz)
        tol += 4 * BF16  # df, dz and dh of this block and the stream's gradient before it are rounded
        for got, want, what in ((mix.dw2, dw2, "dw2"), (mix.db2, db2, "db2"), (mix.dw1, dw1, "dw1"), (mix.db1, db1, "db1")):
            close(got[l], want, tol, f"{what} {l}")
        dh = oracle.linear_dgrad(dz, f64(mix.w1_16[l]))
    dx_, _, g = oracle.residual_norm_bwd(None, X, {"pre_gamma": f64(mix.gamma[0])}, dh, dr, pre="rms", eps=eps)
    close(mix.dgamma[0], g["pre_gamma"], tol, "dgamma 0")
    close(dx, dx_, tol + BF16, "dx")


@pytest.mark.parametrize("rows,c,blocks,expansion", [(512, 64, 2, 4), (300, 40, 1, 3), (64, 256, 3, 4), (5000, 36, 2, 2)])
def test_blocks(cf, rows, c, blocks, expansion):
    from cnn_conv3d_gb300.mixer import VoxelMLP
    mix = VoxelMLP(rows, c, blocks, expansion)
    rng = fill(mix, rows)
    x, dr = (torch.from_numpy(rng.normal(size=(rows, c))).to(torch.bfloat16).cuda() for _ in range(2))
    dx = torch.empty_like(x)
    assert mix.forward(x) is mix.r[-1]
    mix.backward(x, dr, dx)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    check_mixer(mix, x, dr, dx)


def test_blocks_refuse_what_they_are_not():
    from cnn_conv3d_gb300.mixer import VoxelMLP
    for bad in ((0, 8, 1), (8, 0, 1), (8, 8, 0), (8, 8, 1, 0)):
        with pytest.raises(ValueError):
            VoxelMLP(*bad)


def model(optimizer, mixers=2, seed=91):
    from cnn_conv3d_gb300.model import CosmoFlowModel
    m = CosmoFlowModel(2, 32, CHANNELS, specs=SPECS, fc=(64, 16, 4), optimizer=optimizer, mixers=mixers, expansion=2)
    inp = synthdata.stack_inputs(2, 32, CHANNELS, seed=seed, with_dy=False)
    m.stack.load(inp["x"], inp["w"], inp["b"])
    rng = fill(m.mixer, seed) if mixers else np.random.default_rng(seed)
    m.sync_master()
    for w, b in zip(m.fw, m.fb):
        w.copy_(torch.from_numpy(rng.normal(0, np.sqrt(2.0 / w.shape[1]), size=tuple(w.shape))))
        b.copy_(torch.from_numpy(rng.normal(0, 0.05, size=tuple(b.shape))))
    m.set_masks([(rng.random(tuple(t.shape)) < 0.8).astype(np.uint8) for t in m.masks])
    m.target.copy_(torch.from_numpy(rng.uniform(-1, 1, size=tuple(m.target.shape))))
    return m


@pytest.mark.parametrize("optimizer", ["adam", "muon"])
@pytest.mark.parametrize("share", [0.1, 10.0])
def test_training_step_with_blocks_and_clipping(cf, optimizer, share):
    m = model(optimizer)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    x = m.stack.y[-1]
    check_mixer(m.mixer, x, m.dmix, m.dfeat)
    grads = [f64(g) for _, _, g in m.params()]
    assert all(np.isfinite(g).all() and g.any() for g in grads)
    norm, _ = oracle.clip_factor(grads, 1.0)
    clip = share * norm
    factor = oracle.clip_factor(grads, clip)[1]
    before = [f64(p) for p, _, _ in m.params()]
    m.update(1e-3, clip=clip)
    torch.cuda.synchronize()
    got = f64(m.grad_norm)
    assert abs(got[0] - norm) <= 1e-6 * norm and abs(got[1] - factor) <= 2e-6 * factor
    taken = {p.data_ptr() for p, _, _ in m.matrices()} if optimizer == "muon" else set()
    assert len(taken) == (0 if optimizer == "adam" else 2 + 4 + 2)
    for (p, p16, g), b, g0 in zip(m.params(), before, grads):
        if optimizer == "muon":
            np.testing.assert_allclose(f64(g), g0 * factor, rtol=4e-6, atol=1e-30)
        else:
            assert np.array_equal(f64(g), g0)
        if p.data_ptr() in taken:
            assert np.abs(f64(p) - b).max() > 0
        else:
            w, _, _ = oracle.adam_decay_step(b, g0 * factor, 0.0, 0.0, 1e-3, 1)
            # a first step is lr g / (|g| + eps): where g is not far above eps its relative error counts whole
            np.testing.assert_allclose(f64(p), w, rtol=1e-5, atol=1e-3 * 2e-4)
        if p16 is not None:
            assert torch.equal(p16.reshape(p.shape), p.to(torch.bfloat16))


def test_a_step_without_either_keeps_its_bits(cf):
    """mixers=0 and clip=0 are the model as it was, and a norm that nothing exceeds changes no gradient."""
    a, b = model("muon", mixers=0), model("muon", mixers=0)
    for m, clip in ((a, 0.0), (b, 1e30)):
        m.step(1e-3, clip=clip)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for (p, _, _), (q, _, _) in zip(a.params(), b.params()))
    with pytest.raises(ValueError):
        a.update(1e-3, clip=-1.0)


@pytest.mark.parametrize("optimizer", ["adam", "muon"])
def test_a_captured_step_gives_the_same_bits(cf, optimizer):
    a, b = model(optimizer), model(optimizer)
    for _ in range(2):
        a.step(1e-3, clip=0.5)
    b.step(1e-3, clip=0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(1e-3, clip=0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert a.t == b.t
    assert torch.equal(a.grad_norm, b.grad_norm) and torch.equal(a.loss, b.loss)
    for (p, p16, _), (q, q16, _) in zip(a.params(), b.params()):
        assert torch.equal(p, q) and (p16 is None or torch.equal(p16, q16))
