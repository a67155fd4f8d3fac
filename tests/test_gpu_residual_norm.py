"""The norms before and after a block with the gated sum between (cf_residual_norm_*) against 64 bits."""
import numpy as np
import pytest

import oracle
from gpu_util import guarded
from test_more_operators_cpu import _vectors

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
NAMES = ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")
KINDS = ("none", "rms", "layer")


@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


def f64(t):
    return t.detach().double().cpu().numpy()


def desc_of(cf, rows, c, post, pre, scale, dtype, f_dtype, each, per, eps=1e-5):
    t = {BF: cf.CF_DT_BF16, F32: cf.CF_DT_F32}
    return cf.cf_residual_norm_desc(rows, c, KINDS.index(post), KINDS.index(pre), eps, scale, t[dtype], t[f_dtype], each, per)


class Case:
    def __init__(self, cf, seed, rows, c, post="rms", pre="rms", dtype=BF, f_dtype=BF, gate=True, each=0, per=0, scale=0.8, with_f=True,
                 with_dr=True, shift=0.5):
        rng = np.random.default_rng(seed)
        self.cf, self.rows, self.c, self.dtype, self.f_dtype, self.post, self.pre = cf, rows, c, dtype, f_dtype, post, pre
        self.kw = dict(post=post, pre=pre, scale=scale, per=per)
        samples = -(-rows // per) if each else 1
        vec = _vectors(rng, c, post, pre, gate and with_f, samples, each)
        self.vec = {k: torch.from_numpy(v).float().cuda() for k, v in vec.items()}
        self.vec64 = {k: f64(v) for k, v in self.vec.items()}

        def rows_of(dt, mean):
            return torch.from_numpy(rng.normal(mean, 1.0, (rows, c)) * rng.uniform(0.5, 2.0, (rows, 1))).to(dt).cuda()
        self.x, self.r = rows_of(dtype, shift), rows_of(dtype, shift)
        self.f = rows_of(f_dtype, -shift) if with_f else None
        self.dh = rows_of(f_dtype, 0.1) if pre != "none" else None
        self.dr = rows_of(dtype, 0.1) if with_dr else None
        self.desc = desc_of(cf, rows, c, post, pre, scale, dtype, f_dtype, each, per)
        self.vectors = cf.cf_residual_norm_vectors(**self.vec)

    # A sum of c values of fp32 is off by at most (c + 8) 2^-24 of their sizes' sum, in any order; normalised values take two
    # such sums, a root and three roundings, and whatever is made of them some more.
    def eps(self):
        return (2 * self.c + 40) * 2.0 ** -24

    def stats(self, v, kind):
        _, mean, rstd = oracle._row_norm(v, kind, 1e-5)
        return np.abs(mean)[:, None], rstd[:, None]

    def forward(self, r=None, h=None, stats=True, stream=None, x=None):
        cf = self.cf
        ok = []
        if r is None:
            r, check = guarded((self.rows, self.c), self.dtype, fill=-7.0)
            ok.append(check)
        if h is None and self.pre != "none":
            h, check = guarded((self.rows, self.c), self.f_dtype, fill=-7.0)
            ok.append(check)
        st, check = guarded((self.rows, 4), F32, fill=-7.0)
        ok.append(check)
        cf.cf_residual_norm_fwd(self.desc, self.x if x is None else x, self.f, self.vectors, r, h, st if stats else None, stream)
        torch.cuda.synchronize()
        for check in ok:
            check()
        return r, h, st

    def check_forward(self):
        r, h, st = self.forward()
        v = self.vec64
        rr, hh, ss = oracle.residual_norm_fwd(f64(self.x), None if self.f is None else f64(self.f), v, **self.kw)
        per = lambda t: oracle._rows_of(t, self.rows, self.kw["per"]) if t is not None else 1.0  # noqa: E731
        p = np.zeros_like(rr)
        if self.f is not None:
            F = f64(self.f)
            mean, rstd = self.stats(F, self.post)
            p = abs(self.kw["scale"]) * np.abs(per(v.get("gate"))) * ((np.abs(F) + mean) * rstd * np.abs(v.get("post_gamma", 1.0))
                                                                       + np.abs(v.get("post_beta", 0.0)))
        er = self.eps() * (np.abs(f64(self.x)) + p)
        assert np.all(np.abs(f64(r) - rr) <= HALF[self.dtype] * (np.abs(rr) + er) + er)
        mean, rstd = self.stats(rr, self.pre)
        tot = np.abs(f64(st) - ss)
        # the width is a mean of squares of values that are off by er
        assert np.all(tot[:, :2] <= self.eps() * 8 * (np.abs(ss[:, :2]) + 1))
        rel = er.max(1) * rstd[:, 0] + self.eps()
        assert np.all(tot[:, 2:] <= (8 * rel * (1 + mean[:, 0] * rstd[:, 0]))[:, None] * (np.abs(ss[:, 2:]) + 1))
        if h is not None:
            g = np.abs(per(v.get("pre_gamma")))
            eh = 8 * rel[:, None] * g * ((np.abs(rr) + mean) * rstd + 1) + self.eps() * np.abs(per(v.get("pre_beta", np.zeros(self.c))))
            assert np.all(np.abs(f64(h) - hh) <= HALF[self.f_dtype] * (np.abs(hh) + eh) + eh)
        return r, h, st

    def given_stats(self):
        F = np.zeros((self.rows, self.c)) if self.f is None else f64(self.f)
        _, mf, sf = oracle._row_norm(F, self.post, 1e-5)
        _, mr, sr = oracle._row_norm(f64(self.r), self.pre, 1e-5)
        return torch.from_numpy(np.stack((mf, sf, mr, sr), 1)).float().cuda()

    def backward(self, dx=None, df=None, names=NAMES, stream=None, out=None):
        cf = self.cf
        ok = []
        if dx is None:
            dx, check = guarded((self.rows, self.c), self.dtype, fill=-7.0)
            ok.append(check)
        if df is None and self.f is not None:
            df, check = guarded((self.rows, self.c), self.f_dtype, fill=-7.0)
            ok.append(check)
        grads = {}
        for k, t in self.vec.items():
            if k in names:
                grads[k], check = guarded(tuple(t.shape), F32, fill=-7.0)
                ok.append(check)
        size = cf.cf_residual_norm_workspace_size(self.desc)
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
        cf.cf_residual_norm_bwd(self.desc, self.f, self.r, self.vectors, self.given_stats(), self.dh, self.dr, dx, df,
                                cf.cf_residual_norm_vectors(**grads), ws, size, stream)
        torch.cuda.synchronize()
        for check in ok:
            check()
        return dx, df, grads

    def check_backward(self):
        dx, df, grads = self.backward()
        v, eps, s = self.vec64, self.eps(), abs(self.kw["scale"])
        R, DR = f64(self.r), np.zeros((self.rows, self.c)) if self.dr is None else f64(self.dr)
        DH = None if self.dh is None else f64(self.dh)
        F = None if self.f is None else f64(self.f)
        rdx, rdf, rg = oracle.residual_norm_bwd(F, R, v, DH, None if self.dr is None else DR, **self.kw)
        per = lambda t: oracle._rows_of(t, self.rows, self.kw["per"]) if t is not None else 1.0  # noqa: E731
        # sizes of the terms that each value is the sum of
        total, rh = np.abs(DR), np.zeros_like(R)
        if DH is not None:
            mean, rstd = self.stats(R, self.pre)
            rh = (np.abs(R) + mean) * rstd
            u = np.abs(per(v.get("pre_gamma"))) * np.abs(DH)
            total = total + rstd * (u + u.mean(1, keepdims=True) + (rh + 1) * (u * (rh + 1)).mean(1, keepdims=True))
        ex = 4 * eps * total
        assert np.all(np.abs(f64(dx) - rdx) <= HALF[self.dtype] * (np.abs(rdx) + ex) + ex)
        sizes = {}
        rows = (self.rows + 40) * 2.0 ** -24 + 4 * eps
        if F is not None:
            mean, rstd = self.stats(F, self.post)
            fh = (np.abs(F) + mean) * rstd + 1 if self.post != "none" else np.abs(F)
            gate, pg, pb = np.abs(per(v.get("gate"))), np.abs(v.get("post_gamma", 1.0)), np.abs(v.get("post_beta", 0.0))
            dv = s * gate * pg * total
            if self.post != "none":
                dv = rstd * (dv + dv.mean(1, keepdims=True) + fh * (dv * fh).mean(1, keepdims=True))
            ef = 8 * eps * dv
            assert np.all(np.abs(f64(df) - rdf) <= HALF[self.f_dtype] * (np.abs(rdf) + ef) + ef)
            sizes = {"gate": s * total * (pg * fh + pb), "post_gamma": s * gate * total * fh, "post_beta": s * gate * total}
        if DH is not None:
            sizes.update(pre_gamma=np.abs(DH) * (rh + 1), pre_beta=np.abs(DH))
        for k, t in grads.items():
            shape = self.vec64[k].shape
            sz = sizes[k] * np.ones((self.rows, self.c))
            sz = sz.sum(0) if len(shape) == 1 else np.stack([sz[i * self.kw["per"]:(i + 1) * self.kw["per"]].sum(0) for i in range(shape[0])])
            assert np.all(np.abs(f64(t) - rg[k]) <= 2 * rows * sz), k
        return dx, df, grads


KINDS_CASES = [("none", "rms"), ("none", "layer"), ("rms", "rms"), ("layer", "layer"), ("rms", "layer"), ("layer", "rms"), ("rms", "none"),
               ("layer", "none"), ("none", "none")]
TYPES = [(BF, BF), (F32, BF), (F32, F32)]
WIDTHS = [1, 2, 7, 8, 16, 24, 31, 32, 33, 64, 100, 128, 200, 256, 257, 264, 512, 520, 1000, 1024, 2040, 4096, 4100, 8192, 8200, 12000]


@pytest.mark.parametrize("post,pre", KINDS_CASES)
@pytest.mark.parametrize("dtype,f_dtype", TYPES)
@pytest.mark.parametrize("c", [40, 129, 640])
def test_norms_and_types(cf, post, pre, dtype, f_dtype, c):
    case = Case(cf, c, 37, c, post, pre, dtype, f_dtype)
    case.check_forward()
    case.check_backward()


@pytest.mark.parametrize("c", WIDTHS)
@pytest.mark.parametrize("rows", [1, 19])
def test_widths(cf, c, rows):
    case = Case(cf, c + rows, rows, c, "layer" if c > 2 else "rms", "layer" if c > 2 else "rms", F32 if c % 3 else BF, BF)
    case.check_forward()
    case.check_backward()


@pytest.mark.parametrize("each", [1, 2, 3])
@pytest.mark.parametrize("rows,per,c", [(40, 10, 64), (41, 10, 130), (7, 1, 96), (2000, 400, 32), (300, 1000, 512), (65, 13, 8200), (3001, 100, 16)])
def test_vectors_of_each_sample(cf, each, rows, per, c):
    case = Case(cf, rows + c, rows, c, "layer", "layer", each=each, per=per)
    case.check_forward()
    case.check_backward()


@pytest.mark.parametrize("rows,c", [(20000, 32), (5000, 128), (3000, 1000), (1500, 2048), (70001, 8)])
def test_many_rows(cf, rows, c):
    case = Case(cf, rows, rows, c, "rms", "layer", F32, BF)
    case.check_forward()
    case.check_backward()


# enough rows for the kernels that copies feed: ends inside a stage, in a round of rows, samples that end inside a block's
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "none"), ("none", "rms")])
@pytest.mark.parametrize("dtype,f_dtype", TYPES)
@pytest.mark.parametrize("rows,c,each,per", [(19001, 128, 0, 0), (10007, 256, 3, 1000), (2003, 1000, 2, 333), (1300, 2048, 0, 0), (701, 4096, 1, 100)])
def test_rows_in_stages(cf, rows, c, each, per, post, pre, dtype, f_dtype):
    case = Case(cf, rows, rows, c, post, pre, dtype, f_dtype, each=each, per=per)
    case.check_forward()
    case.check_backward()


# rows that begin inside 16 bytes, whose tensors end inside 16 bytes too
@pytest.mark.parametrize("dtype,f_dtype", TYPES)
@pytest.mark.parametrize("rows,c,each,per", [(20003, 130, 0, 0), (10007, 255, 3, 1001), (2003, 1001, 2, 333), (1301, 2045, 0, 0), (701, 4095, 1, 101),
                                             (600001, 3, 0, 0), (400003, 1, 0, 0), (2437, 515, 0, 0)])
def test_rows_that_begin_anywhere_in_stages(cf, rows, c, each, per, dtype, f_dtype):
    case = Case(cf, rows, rows, c, "layer" if c > 3 else "rms", "rms", dtype, f_dtype, each=each, per=per)
    case.check_forward()
    case.check_backward()


@pytest.mark.parametrize("rows,c", [(300001, 8), (80003, 32), (38000, 56)])
def test_narrow_rows_in_stages(cf, rows, c):
    case = Case(cf, rows, rows, c, "layer", "rms", BF, BF, each=1, per=rows // 3)
    case.check_forward()
    case.check_backward()


@pytest.mark.parametrize("rows,c", [(20000, 128), (1300, 2048), (20001, 129), (1301, 2047)])
def test_stages_without_some_tensors(cf, rows, c):
    case = Case(cf, c, rows, c, "none", "layer", gate=False, with_f=False, with_dr=False)
    case.check_forward()
    case.check_backward()
    case = Case(cf, c, rows, c, "rms", "rms", F32, BF)
    dx, df, g = case.backward()
    dr, dh = case.dr, case.dh
    case.dr = dr.clone()
    dx2, df2, g2 = case.backward(dx=case.dr)
    assert torch.equal(dx, dx2) and torch.equal(df, df2) and all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("c", [48, 300, 9000])
def test_first_norm_and_parts_left_out(cf, c):
    case = Case(cf, c, 33, c, "none", "layer", gate=False, with_f=False, with_dr=False)
    case.check_forward()
    case.check_backward()
    case = Case(cf, c, 33, c, "rms", "rms", gate=False)
    r, h, st = case.forward()
    r2, h2, st2 = case.forward(stats=False)
    assert torch.equal(r, r2) and torch.equal(h, h2) and bool((st2 == -7.0).all())
    h3 = torch.empty_like(h)
    cf.cf_residual_norm_fwd(case.desc, case.x, case.f, case.vectors, None, h3, None)
    assert torch.equal(h, h3)
    dx, df, g = case.backward()
    dx2, df2, g2 = case.backward(names=("pre_gamma",))
    assert torch.equal(dx, dx2) and torch.equal(df, df2) and torch.equal(g["pre_gamma"], g2["pre_gamma"])


@pytest.mark.parametrize("c", [64, 96, 130, 2048, 9000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(cf, c, dtype):
    case = Case(cf, c, 50, c, "layer", "rms", dtype, dtype)
    r, h, _ = case.forward()
    x = case.x.clone()
    r2, h2, _ = case.forward(r=x, x=x)
    assert torch.equal(r, r2) and torch.equal(h, h2)
    dx, df, g = case.backward()
    dr, dh = case.dr, case.dh
    case.dr, case.dh = dr.clone(), dh.clone()
    dx2, df2, g2 = case.backward(dx=case.dr, df=case.dh)
    assert torch.equal(dx, dx2) and torch.equal(df, df2) and all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("c", [64, 1000, 9000])
def test_rows_far_from_zero_and_constant_rows(cf, c):
    """A width is taken about the row's mean: rows of a large mean keep it, constant ones give beta."""
    case = Case(cf, c, 24, c, "none", "layer", F32, F32, gate=False, with_f=False)
    case.x = case.x + 1000.0
    case.x[3] = 5.0
    r, h, st = oracle.residual_norm_fwd(f64(case.x), None, case.vec64, **case.kw)
    _, gh, gst = case.forward()
    # values of 1000 are held to 2^-14, so that a mean is off by at most some of those, and a value over the width by as much
    keep = np.arange(24) != 3
    assert np.abs(f64(gh) - h)[keep].max() <= (c + 40) * 2.0 ** -24 * 1000 * 16
    assert np.all(np.abs(f64(gh)[3] - f64(case.vec["pre_beta"])) <= (c + 40) * 2.0 ** -24 * 5 * 1e3)


@pytest.mark.parametrize("c", [32, 300, 9000])
def test_what_is_not_finite_stays_in_its_row(cf, c):
    case = Case(cf, c, 21, c, "layer", "layer")
    r0, h0, _ = case.forward()
    dx0, df0, _ = case.backward()
    case.f[4, c // 2] = float("nan")
    case.dh[9, 0] = float("inf")
    r1, h1, _ = case.forward()
    keep = torch.arange(21, device="cuda") != 4
    assert torch.equal(r0[keep], r1[keep]) and torch.equal(h0[keep], h1[keep]) and bool(torch.isnan(h1[4]).all())
    dx1, df1, _ = case.backward()
    keep &= torch.arange(21, device="cuda") != 9
    assert torch.equal(dx0[keep], dx1[keep]) and torch.equal(df0[keep], df1[keep]) and not bool(torch.isfinite(dx1[9]).all())


def test_no_rows(cf):
    d = desc_of(cf, 0, 40, "layer", "layer", 1.0, BF, BF, 0, 0)
    g = {k: torch.ones(40, device="cuda") for k in NAMES}
    cf.cf_residual_norm_bwd(d, None, None, None, None, None, None, None, None, cf.cf_residual_norm_vectors(**g))
    assert all(bool((t == 0).all()) for t in g.values())


@pytest.mark.parametrize("rows,c,each,per", [(64, 256, 0, 0), (4000, 64, 3, 500), (300, 4096, 0, 0), (100, 9000, 1, 30)])
def test_the_same_bits_again_on_another_stream_and_in_a_graph(cf, rows, c, each, per):
    case = Case(cf, 5, rows, c, "layer", "rms", each=each, per=per)
    st = case.given_stats()
    size = cf.cf_residual_norm_workspace_size(case.desc)
    ws = torch.empty((size,), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        g = {k: torch.empty_like(t) for k, t in case.vec.items()}
        outs.append(([torch.empty_like(case.x), torch.empty_like(case.f), torch.empty((rows, 4), device="cuda"), torch.empty_like(case.x),
                      torch.empty_like(case.f)] + list(g.values()), cf.cf_residual_norm_vectors(**g)))

    def calls(o, s):
        t, g = o
        cf.cf_residual_norm_fwd(case.desc, case.x, case.f, case.vectors, t[0], t[1], t[2], s)
        cf.cf_residual_norm_bwd(case.desc, case.f, case.r, case.vectors, st, case.dh, case.dr, t[3], t[4], g, ws, size, s)

    torch.cuda.synchronize()
    calls(outs[0], torch.cuda.current_stream())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls(outs[1], side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(outs[2], torch.cuda.current_stream())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        for a, b in zip(outs[0][0], o[0]):
            assert torch.equal(a, b)


def test_offsets_beyond_2_to_31(cf):
    """2^31 values and more: the last rows as alone."""
    c, rows = 4096, (1 << 19) + 40
    x = torch.empty((rows, c), dtype=BF, device="cuda").normal_()
    f = torch.empty((rows, c), dtype=BF, device="cuda").normal_()
    h = torch.empty_like(x)
    st = torch.empty((rows, 4), device="cuda")
    d = desc_of(cf, rows, c, "rms", "layer", 1.0, BF, BF, 0, 0)
    cf.cf_residual_norm_fwd(d, x, f, None, None, h, st)
    d2 = desc_of(cf, 50, c, "rms", "layer", 1.0, BF, BF, 0, 0)
    h2, st2 = torch.empty((50, c), dtype=BF, device="cuda"), torch.empty((50, 4), device="cuda")
    cf.cf_residual_norm_fwd(d2, x[-50:], f[-50:], None, None, h2, st2)
    assert torch.equal(h[-50:], h2) and torch.equal(st[-50:], st2)
    size = cf.cf_residual_norm_workspace_size(d)
    ws = torch.empty((size,), dtype=torch.uint8, device="cuda")
    dx, df = torch.empty_like(x), torch.empty_like(x)
    cf.cf_residual_norm_bwd(d, f, x, None, st, h, None, dx, df, None, ws, size)
    dx2, df2 = torch.empty_like(h2), torch.empty_like(h2)
    cf.cf_residual_norm_bwd(d2, f[-50:], x[-50:], None, st2, h[-50:], None, dx2, df2, None, ws, size)
    assert torch.equal(dx[-50:], dx2) and torch.equal(df[-50:], df2)
