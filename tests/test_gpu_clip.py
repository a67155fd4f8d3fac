"""The global gradient norm, clipping and the clipped Adam step (cf_grad_norm, cf_clip_grads, cf_clip_adam_step) against 64 bits."""
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


def grads_of(seed, counts, dtypes=(F32,), offsets=(0,), scale=1.0):
    """Gradients that start `offset` values into buffers of their own, between guards."""
    rng = np.random.default_rng(seed)
    out, checks = [], []
    for i, n in enumerate(counts):
        dt, off = dtypes[i % len(dtypes)], offsets[i % len(offsets)]
        t, check = guarded((off + n + 3,), dt, fill=-7.0)
        t = t[off:off + n]
        t.copy_(torch.from_numpy(rng.normal(size=n) * scale * 10.0 ** (-(i % 3))))
        out.append(t)
        checks.append(check)
    return out, checks


def call(cf, fn, grads, max_norm, stream=None):
    lst = cf.cf_grads(grads)
    size = cf.cf_grad_workspace_size(lst)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((2,), -1.0, device="cuda")
    torch.cuda.synchronize()
    fn(lst, max_norm, out, ws, size, stream)
    torch.cuda.synchronize()
    return f64(out)


# sums of 16 squares in fp32 (20 roundings at most, all of one sign of error), then 64 bits, a root and a rounding; the factor is
# a sum and a quotient on top
NORM_TOL, FACTOR_TOL = 16 * 2.0 ** -24, 20 * 2.0 ** -24

COUNTS = [[1], [5], [4096], [4097, 3], [100000], [1, 2, 3, 4, 5, 6, 7, 8, 9], [0, 17, 0, 12345], [32] * 40, [3456, 32, 55296, 64, 221184, 128],
          [1000] * 1500, [1 << 20, 7, (1 << 20) + 1], [0, 0]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{c[0]}")
@pytest.mark.parametrize("dtypes,offsets", [((F32,), (0,)), ((BF,), (0,)), ((F32, BF, BF), (1, 0, 3, 5))])
@pytest.mark.parametrize("max_norm", [0.01, 1e9])
def test_norm_and_clip(cf, counts, dtypes, offsets, max_norm):
    grads, checks = grads_of(len(counts), counts, dtypes, offsets)
    before = [f64(g) for g in grads]
    norm, factor = oracle.clip_factor(before, max_norm) if sum(counts) else (0.0, min(1.0, max_norm / 1e-6))
    got = call(cf, cf.cf_grad_norm, grads, max_norm)
    for b, g in zip(before, grads):
        assert np.array_equal(b, f64(g))
    again = call(cf, cf.cf_clip_grads, grads, max_norm)
    assert np.array_equal(got, again)
    assert abs(got[0] - norm) <= NORM_TOL * norm and abs(got[1] - factor) <= FACTOR_TOL * factor
    for b, g, check in zip(before, grads, checks):
        check()
        half = 2.0 ** -24 if g.dtype == F32 else 2.0 ** -8
        if got[1] == 1.0:
            assert np.array_equal(b, f64(g))
        else:
            assert np.all(np.abs(f64(g) - b * factor) <= (FACTOR_TOL + half) * np.abs(b * factor) * 1.01 + 1e-45)
    if sum(counts) and factor < 1:
        # (values around a tensor are the fill: guarded() left them)
        assert abs(np.sqrt(sum((f64(g) ** 2).sum() for g in grads)) - max_norm) <= 1e-2 * max_norm


@pytest.mark.parametrize("scale", [1e-30, 1e-38, 1e-42, 1e20, 1e36])
def test_squares_neither_overflow_nor_vanish(cf, scale):
    grads, _ = grads_of(3, [1000, 5000, 33], scale=scale)
    vals = [f64(g) for g in grads]
    norm, _ = oracle.clip_factor(vals, 1.0)
    got = call(cf, cf.cf_grad_norm, grads, 1.0)
    assert abs(got[0] - norm) <= NORM_TOL * norm + 1e-45
    # beside ordinary values the small ones are nothing and the large ones everything
    mixed, _ = grads_of(4, [4096 * 3])
    both = mixed + grads
    norm, factor = oracle.clip_factor([f64(g) for g in both], 1.0)
    got = call(cf, cf.cf_grad_norm, both, 1.0)
    assert abs(got[0] - norm) <= NORM_TOL * norm and abs(got[1] - factor) <= FACTOR_TOL * factor + 1e-45


@pytest.mark.parametrize("dtype", [F32, BF])
def test_zero_infinite_and_nan_gradients(cf, dtype):
    z = [torch.zeros(10000, device="cuda", dtype=dtype)]
    assert list(call(cf, cf.cf_clip_grads, z, 1.0)) == [0.0, 1.0] and not bool(z[0].any())
    g, _ = grads_of(5, [5000, 40], (dtype,))
    g[0][4321] = float("inf")
    out = call(cf, cf.cf_clip_grads, g, 1.0)
    assert np.isinf(out[0]) and out[1] == 0.0
    assert bool(torch.isnan(g[0][4321])) and not bool(g[0][:4321].any()) and not bool(g[1].any())
    g, _ = grads_of(6, [5000, 40], (dtype,))
    g[1][39] = float("nan")
    out = call(cf, cf.cf_clip_grads, g, 1.0)
    assert np.isnan(out).all() and all(bool(torch.isnan(t).all()) for t in g)


def test_no_gradients(cf):
    assert list(call(cf, cf.cf_grad_norm, [], 1.0)) == [0.0, 1.0]
    assert list(call(cf, cf.cf_clip_grads, [], 1.0)) == [0.0, 1.0]


def adam_list(seed, counts, offsets=(0,), w16=True):
    rng = np.random.default_rng(seed)
    out, checks = [], []
    for i, n in enumerate(counts):
        entry = []
        for kind in range(5):
            off = offsets[(i + kind) % len(offsets)] if len(offsets) > 1 else offsets[0]
            t, check = guarded((off + n + 2,), BF if kind == 1 else F32, fill=-7.0)
            t = t[off:off + n]
            v = rng.normal(size=n)
            if kind != 1:
                t.copy_(torch.from_numpy({0: v, 2: 0.1 * v, 3: 1e-2 * v, 4: 1e-4 * v * v}[kind]))
            entry.append(t)
            checks.append(check)
        if not w16 or i % 3 == 2:
            entry[1] = None
        out.append(entry)
    return out, checks


@pytest.mark.parametrize("counts", [[1], [7, 4096, 33], [100000, 5], [64] * 40, [300] * 1000, [0, 50], [(1 << 20) + 3]],
                         ids=lambda c: f"{len(c)}x{c[0]}")
@pytest.mark.parametrize("offsets", [(0,), (3,), (0, 1, 2)])
@pytest.mark.parametrize("max_norm", [0.0, 0.05, 1e6])
def test_clipped_adam_step(cf, counts, offsets, max_norm):
    lst, checks = adam_list(7, counts, offsets)
    b1, b2, eps, decay, lr, t = 0.9, 0.999, 1e-8, 0.02, 1e-3, 5
    before = [[None if v is None else f64(v) for v in e] for e in lst]
    norm, factor = oracle.clip_factor([e[2] for e in before], max_norm) if max_norm else (None, 1.0)
    params = cf.cf_adam_params(lst)
    size = cf.cf_clip_adam_workspace_size(params)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((2,), -1.0, device="cuda")
    cf.cf_clip_adam_step(params, cf.cf_adam_hyper(lr, b1, b2, eps, decay, max_norm, t), out, ws, size)
    torch.cuda.synchronize()
    for check in checks:
        check()
    got = f64(out)
    if max_norm:
        assert abs(got[0] - norm) <= NORM_TOL * norm and abs(got[1] - factor) <= FACTOR_TOL * factor
    else:
        assert list(got) == [-1.0, -1.0]
    for e, (w, _, g, m, v) in zip(lst, before):
        assert np.array_equal(f64(e[2]), g)
        rw, rm, rv = oracle.adam_decay_step(w, g * factor, m, v, lr, t, b1, b2, eps, decay)
        tol = FACTOR_TOL + 8 * 2.0 ** -24
        assert np.all(np.abs(f64(e[3]) - rm) <= tol * (np.abs(b1 * m) + np.abs((1 - b1) * g * factor)))
        assert np.all(np.abs(f64(e[4]) - rv) <= 2 * tol * rv + 1e-45)
        # the step: a quotient of m, which may cancel, and the root
        size_ = lr / (1 - b1 ** t) * (np.abs(b1 * m) + np.abs((1 - b1) * g * factor)) / (np.sqrt(rv / (1 - b2 ** t)) + eps)
        ew = 2.0 ** -23 * np.abs(w) + 4 * tol * size_
        assert np.all(np.abs(f64(e[0]) - rw) <= ew)
        if e[1] is not None:
            assert torch.equal(e[1], e[0].to(BF))


def test_an_adam_step_without_clipping_is_cf_adam_step(cf):
    """The same formula, to the roundings of its constants."""
    lst, _ = adam_list(8, [5000])
    w, w16, g, m, v = lst[0]
    w2, m2, v2 = w.clone(), m.clone(), v.clone()
    cf.cf_clip_adam_step(cf.cf_adam_params(lst), cf.cf_adam_hyper(1e-3, 0.9, 0.999, 1e-8, 0.0, 0.0, 3), None)
    cf.cf_adam_step(5000, w2, None, g, m2, v2, 1e-3, 0.9, 0.999, 1e-8, 3)
    assert torch.allclose(w, w2, rtol=1e-5, atol=1e-7) and torch.allclose(m, m2, rtol=1e-5, atol=1e-8) and torch.allclose(v, v2, rtol=1e-4)


@pytest.mark.parametrize("counts", [[3456, 32, 221184, 128], [700] * 1100])
def test_the_same_bits_again_on_another_stream_and_in_a_graph(cf, counts):
    lists = [adam_list(9, counts)[0] for _ in range(3)]
    grads = [grads_of(10, counts)[0] for _ in range(3)]
    hyper = cf.cf_adam_hyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 0.5, 2)
    state = []
    for l, g in zip(lists, grads):
        p, gl = cf.cf_adam_params(l), cf.cf_grads(g)
        size = max(cf.cf_clip_adam_workspace_size(p), cf.cf_grad_workspace_size(gl))
        state.append((p, gl, torch.empty(size, dtype=torch.uint8, device="cuda"), size, torch.empty(2, device="cuda"),
                      torch.empty(2, device="cuda")))

    def calls(s, stream):
        p, gl, ws, size, a, b = s
        cf.cf_clip_adam_step(p, hyper, a, ws, size, stream)
        cf.cf_clip_grads(gl, 0.1, b, ws, size, stream)

    torch.cuda.synchronize()
    calls(state[0], torch.cuda.current_stream())
    side = torch.cuda.Stream()
    calls(state[1], side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(state[2], torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(state[0][4], state[i][4]) and torch.equal(state[0][5], state[i][5])
        for a, b in zip(lists[0], lists[i]):
            assert all(torch.equal(s, t) for s, t in zip(a, b) if s is not None)
        assert all(torch.equal(s, t) for s, t in zip(grads[0], grads[i]))
