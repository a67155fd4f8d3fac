"""Group-normalised blocks and the Muon step where they are used: in a CosmoStack, whose kernels are each checked against the
64-bit oracle on the GPU's own inputs of that kernel, and in CosmoFlowModel's training step."""
import numpy as np
import pytest

import synthdata
from tests.gpu_util import assert_close

pytestmark = pytest.mark.gpu

SLOPE = 0.3
CHANNELS = (4, 32, 64, 64, 128)
SPECS = [(1, "max", "gn"), (1, "avg", "gn", 4), (2, "none", "gn", 16), (1, "none", "gn")]


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cnn_conv3d_gb300 import build
    build.build()
    return torch


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _bf16(a, torch):
    return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()


def test_stack_of_group_normalised_blocks(torch_cuda, oracle_mod):
    torch = torch_cuda
    from cnn_conv3d_gb300 import cfconv as cf
    from cnn_conv3d_gb300.stack import CosmoStack
    n, spatial = 2, 32
    inp = synthdata.stack_inputs(n, spatial, CHANNELS, seed=71, with_dy=False)
    rng = np.random.default_rng(71)
    inp["b"] = [rng.normal(0, 0.5, size=c).astype(np.float32) for c in CHANNELS[1:]]
    st = CosmoStack(n, spatial, CHANNELS, SLOPE, specs=SPECS)
    st.load(inp["x"], inp["w"], inp["b"])
    gammas = [rng.normal(1, 0.3, size=c) for c in CHANNELS[1:]]
    for l, g in enumerate(gammas):
        st.gamma[l].copy_(torch.from_numpy(g))
    dy = _bf16(synthdata.to_bf16_bits(rng.normal(size=tuple(st.y[-1].shape))), torch)
    st.step(dy)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    f = oracle_mod.bf16_bits_to_f64
    for l in range(st.L):
        x, w, z = _f64(st.block_input(l)), f(inp["w"][l]), _f64(st.zc[l])
        fwd = oracle_mod.conv3d_fwd if SPECS[l][0] == 1 else oracle_mod.conv3d_fwd_s2
        assert_close(z, fwd(x, w), fwd(np.abs(x), np.abs(w)), f"conv {l + 1}")
        gamma, beta, groups, pool = _f64(st.gamma[l]), _f64(st.b[l]), st.groups(l), SPECS[l][1]
        y, mean, rstd = oracle_mod.group_norm_fwd(z, gamma, beta, groups, pool, "lrelu", SLOPE)
        assert_close(_f64(st.stats[l][0]), mean, np.abs(mean) + 1e-2, f"mean {l + 1}")
        assert_close(_f64(st.stats[l][1]), rstd, rstd, f"rstd {l + 1}")
        assert_close(_f64(st.y[l]), y, np.abs(y) + 1e-1, f"block {l + 1}")
        g = _f64(dy if l == st.L - 1 else st.g[l])
        dz, dgamma, dbeta = oracle_mod.group_norm_bwd(z, gamma, beta, groups, g, pool, "lrelu", SLOPE)
        s = np.abs(g).reshape(-1, g.shape[-1]).sum(0)
        assert_close(_f64(st.dgamma[l]), dgamma, s, f"dgamma {l + 1}")
        assert_close(_f64(st.db[l]), dbeta, s, f"dbeta {l + 1}")
        rel = np.linalg.norm(_f64(st.dz[l]) - dz) / np.linalg.norm(dz)
        assert rel <= 5e-3, (l, rel)
        d = _f64(st.dz[l])
        wgrad = oracle_mod.conv3d_wgrad if SPECS[l][0] == 1 else oracle_mod.conv3d_wgrad_s2
        assert_close(_f64(st.dw[l]), wgrad(x, d), wgrad(np.abs(x), np.abs(d)), f"dW {l + 1}")
        if l > 0:  # the gradient at the block below's output, without its activation's derivative
            if SPECS[l][0] == 1:
                ref, S = oracle_mod.conv3d_dgrad(d, w), oracle_mod.conv3d_dgrad(np.abs(d), np.abs(w))
            else:
                ref = oracle_mod.conv3d_dgrad_s2(d, w, x.shape[1:4])
                S = oracle_mod.conv3d_dgrad_s2(np.abs(d), np.abs(w), x.shape[1:4])
            assert_close(_f64(st.g[l - 1]), ref, S, f"dX {l + 1}")


def test_graphed_and_host_buffer_steps_give_the_same_bits(torch_cuda):
    torch = torch_cuda
    from cnn_conv3d_gb300.stack import CosmoStack
    n, spatial = 2, 32
    inp = synthdata.stack_inputs(n, spatial, CHANNELS, seed=72, with_dy=False)
    st = CosmoStack(n, spatial, CHANNELS, SLOPE, specs=SPECS)
    st.load(inp["x"], inp["w"], inp["b"])
    gen = torch.Generator(device="cuda").manual_seed(72)
    dy = torch.randn(st.y[-1].shape, device="cuda", generator=gen).to(torch.bfloat16)
    st.step(dy)
    torch.cuda.synchronize()
    want = [t.clone() for t in st.dw + st.db + st.dgamma]
    graph = st.capture(dy)
    for t in st.dw + st.db + st.dgamma:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, st.dw + st.db + st.dgamma))


def _model(torch, optimizer, seed=73):
    from cnn_conv3d_gb300.model import CosmoFlowModel
    m = CosmoFlowModel(2, 32, CHANNELS, specs=SPECS, fc=(64, 16, 4), optimizer=optimizer)
    inp = synthdata.stack_inputs(2, 32, CHANNELS, seed=seed, with_dy=False)
    m.stack.load(inp["x"], inp["w"], inp["b"])
    m.sync_master()
    rng = np.random.default_rng(seed)
    for w, b in zip(m.fw, m.fb):
        w.copy_(torch.from_numpy(rng.normal(0, np.sqrt(2.0 / w.shape[1]), size=w.shape)))
        b.copy_(torch.from_numpy(rng.normal(0, 0.05, size=b.shape)))
    m.set_masks([(rng.random(t.shape) < 0.8).astype(np.uint8) for t in m.masks])
    m.target.copy_(torch.from_numpy(rng.uniform(-1, 1, size=m.target.shape)))
    return m


def test_muon_training_step(torch_cuda, oracle_mod):
    torch = torch_cuda
    from cnn_conv3d_gb300 import cfconv as cf
    m = _model(torch, "muon")
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    before = {p.data_ptr(): (_f64(p), _f64(g)) for p, _, g in m.params()}
    lr = 1e-3
    m.update(lr, weight_decay=0.1)
    torch.cuda.synchronize()
    assert cf.cf_last_device_status() == cf.CF_OK
    muon = {p.data_ptr() for p, _, _ in m.matrices()}
    assert len(muon) == len(CHANNELS) - 1 + 2
    for p, p16, _ in m.params():
        w0, g0 = before[p.data_ptr()]
        if p.data_ptr() in muon:
            w2, g2 = w0.reshape(w0.shape[0], -1), g0.reshape(g0.shape[0], -1)
            scale = 0.2 * max(w2.shape) ** 0.5
            ref, _ = oracle_mod.muon_step(w2, g2, np.zeros_like(w2), lr, scale, 0.95, True, 0.1)
            o = (w2 * (1 - lr * 0.1) - ref) / (lr * scale)
            off = np.linalg.norm(_f64(p).reshape(w2.shape) - ref)
            assert off <= 3.3e-3 * lr * scale * np.linalg.norm(o) + 2.0 ** -22 * np.linalg.norm(w2)
        else:
            ref, _, _ = oracle_mod.adam_step(w0, g0, np.zeros_like(w0), np.zeros_like(w0), lr=lr, t=1)
            np.testing.assert_allclose(_f64(p), ref, rtol=1e-6, atol=1e-7)
        if p16 is not None:
            assert torch.equal(p16, p.to(torch.bfloat16))


def test_training_reduces_the_loss(torch_cuda):
    torch = torch_cuda
    from cnn_conv3d_gb300 import cfconv as cf
    m = _model(torch, "muon", seed=74)
    losses = []
    for _ in range(15):
        m.step(2e-3)
        torch.cuda.synchronize()
        losses.append(float(m.loss[0]))
    assert cf.cf_last_device_status() == cf.CF_OK
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.7 * losses[0], losses


def test_unknown_optimizer_is_refused(torch_cuda):
    from cnn_conv3d_gb300.model import CosmoFlowModel
    with pytest.raises(ValueError):
        CosmoFlowModel(1, 32, CHANNELS, specs=SPECS, optimizer="sgd")


@pytest.mark.parametrize("optimizer", ["muon", "adam"])
@pytest.mark.parametrize("handle", [False, True])
def test_first_step_on_a_stream_of_its_own(torch_cuda, optimizer, handle):
    """The optimizer's state is zeroed in the order of the stream that the step is enqueued on, whatever another stream is busy with."""
    torch = torch_cuda
    from cnn_conv3d_gb300 import cfconv as cf
    runs = []
    for own in (False, True):
        m = _model(torch, optimizer, seed=75)
        m.forward()
        m.backward()
        torch.cuda.synchronize()
        s = torch.cuda.Stream() if own else torch.cuda.current_stream()
        if own:
            # memory that is handed out again does not hold zeros
            junk = [torch.full_like(p, 3.0) for p, _, _ in m.params() for _ in range(2)]
            torch.cuda.synchronize()
            del junk
            torch.cuda._sleep(100_000_000)  # the current stream is busy for some 50 ms
        for _ in range(2):
            m.update(1e-3, stream=s.cuda_stream if handle and own else s, weight_decay=0.1)
        torch.cuda.synchronize()
        assert cf.cf_last_device_status() == cf.CF_OK
        runs.append([p.clone() for p, _, _ in m.params()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_steps_from_host_buffers_give_the_same_bits(torch_cuda):
    """step_host and step_host_pipelined over group-normalised blocks, and step_host as a CUDA graph, against load + step."""
    torch = torch_cuda
    from cnn_conv3d_gb300 import cfconv as cf
    from cnn_conv3d_gb300.stack import CosmoStack
    n, spatial = 3, 32
    inp = synthdata.stack_inputs(n, spatial, CHANNELS, seed=76, with_dy=False)
    st = CosmoStack(n, spatial, CHANNELS, SLOPE, specs=SPECS)
    st.load(inp["x"], inp["w"], inp["b"])
    gen = torch.Generator(device="cuda").manual_seed(76)
    dy = torch.randn(st.y[-1].shape, device="cuda", generator=gen).to(torch.bfloat16)
    st.step(dy)
    torch.cuda.synchronize()
    outputs, want_dev = st.y + st.dgamma, [t.clone() for t in st.y + st.dgamma]
    want = [t.cpu() for t in st.dw + st.db]
    x_host, dy_host = st.x.cpu().pin_memory(), dy.cpu().pin_memory()
    dw_host, db_host = ([torch.empty(t.shape, dtype=t.dtype).pin_memory() for t in ts] for ts in (st.dw, st.db))

    def clear():
        torch.cuda.synchronize()
        for t in [st.x] + outputs + st.dw + st.db + dw_host + db_host:
            t.fill_(9.0)
        torch.cuda.synchronize()

    def check():
        torch.cuda.synchronize()
        assert cf.cf_last_device_status() == cf.CF_OK
        assert all(torch.equal(a, b) for a, b in zip(want, dw_host + db_host))
        assert all(torch.equal(a, b) for a, b in zip(want_dev, outputs))

    clear()
    st.step_host(x_host, dy_host, dw_host, db_host, chunks=2)
    check()
    graph = st.capture(None, host=(x_host, dy_host, dw_host, db_host))
    clear()
    graph.replay()
    check()
    clear()
    st.prefetch_host(x_host, dy_host)
    st.step_host_pipelined(x_host, dy_host, dw_host, db_host)
    check()
