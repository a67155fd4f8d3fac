"""The whole CosmoFlow network as one training step through the C ABI: the
conv stack (CosmoStack), the fully connected head, the mean squared error and
Adam (hybrid-parallelism page, section IV and Table I: fc1 2048 -> fc2 256 ->
fc3 4 outputs, leaky ReLU after every layer but the last, dropout with keep
probability 0.8 after the hidden fc layers, MSE loss, Adam with beta1 0.9,
beta2 0.999, eps 1e-8 and a linear learning-rate decay to 0.01x).

Python only owns buffers (torch allocations) and enqueues library calls; every
arithmetic step runs in libcfconv3d's kernels.  Conv weights keep an fp32
master copy that Adam updates; the bf16 copy the conv kernels read is written
by the same launch.  Dropout draws are inputs (keep masks), set per step by the
caller (set_masks).

With optimizer="muon" the weight matrices (conv filters as [c_out][27 c_in], the
hidden fc layers) take momentum steps with orthogonalised updates, one
cf_muon_step call for all of them, scaled so that an update has the root mean
square of 0.2 lr that Adam's typically has; vectors and the output layer stay
with Adam.
"""
from __future__ import annotations

import torch

from . import cfconv as cf
from .stack import CosmoStack


class CosmoFlowModel:
    def __init__(self, n: int, spatial: int, channels, specs=None, fc=(2048, 256, 4), slope: float = 0.3,
                 keep: float = 0.8, device: str = "cuda", optimizer: str = "adam"):
        if optimizer not in ("adam", "muon"):
            raise ValueError(f"optimizer {optimizer!r}: adam or muon")
        self.optimizer = optimizer
        self.n, self.slope, self.keep, self.device = n, float(slope), float(keep), device
        self.stack = CosmoStack(n, spatial, channels, slope, device, backward=True, specs=specs)
        st = self.stack
        f32, u8 = torch.float32, torch.uint8
        self.feat = int(st.y[-1][0].numel())  # flattened NDHWC top output per sample
        self.dims = [self.feat] + list(fc)
        D = self.dims
        self.fw = [torch.zeros((D[i + 1], D[i]), dtype=f32, device=device) for i in range(len(fc))]
        self.fb = [torch.zeros((D[i + 1],), dtype=f32, device=device) for i in range(len(fc))]
        # hidden outputs (after activation and dropout), predictions, keep masks
        self.h = [torch.empty((n, D[i + 1]), dtype=f32, device=device) for i in range(len(fc) - 1)]
        self.pred = torch.empty((n, D[-1]), dtype=f32, device=device)
        self.masks = [torch.ones((n, D[i + 1]), dtype=u8, device=device) for i in range(len(fc) - 1)]
        self.target = torch.zeros((n, D[-1]), dtype=f32, device=device)
        self.loss = torch.zeros((4,), dtype=f32, device=device)
        # gradients
        self.dpred = torch.empty_like(self.pred)
        self.dh = [torch.empty_like(t) for t in self.h]
        self.dfw = [torch.empty_like(t) for t in self.fw]
        self.dfb = [torch.empty_like(t) for t in self.fb]
        self.dfeat = torch.empty(tuple(st.y[-1].shape), dtype=torch.bfloat16, device=device)
        # conv weights' fp32 master copies (set by sync_master after loading)
        self.w32 = [torch.empty(w.shape, dtype=f32, device=device) for w in st.w]
        self._adam = None
        self._muon = None
        self.t = 0

    # ---------------------------------------------------------------- set-up
    def sync_master(self):
        """fp32 master copies of the conv weights from their bf16 values."""
        for m, w in zip(self.w32, self.stack.w):
            m.copy_(w.float())

    def set_masks(self, masks):
        for dst, src in zip(self.masks, masks):
            dst.copy_(torch.as_tensor(src, dtype=torch.uint8).reshape(dst.shape))

    def params(self):
        """(fp32 tensor, bf16 copy or None, gradient) of every trained parameter."""
        st = self.stack
        out = []
        for l in range(st.L):
            out.append((self.w32[l], st.w[l], st.dw[l]))
            out.append((st.b[l], None, st.db[l]))
            if st.normed(l):
                out.append((st.gamma[l], None, st.dgamma[l]))
        for i in range(len(self.fw)):
            out.append((self.fw[i], None, self.dfw[i]))
            out.append((self.fb[i], None, self.dfb[i]))
        return out

    # ------------------------------------------------------------------ step
    def forward(self, stream=None):
        """Conv stack, then the head: predictions in self.pred, loss in self.loss[0]."""
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = self.stack
        st.forward(s)
        n, D = self.n, self.dims
        x, xb = st.y[-1], 1
        for i in range(len(self.fw)):
            last = i == len(self.fw) - 1
            out = self.pred if last else self.h[i]
            cf.cf_fc_fwd(n, D[i], D[i + 1], x, xb, self.fw[i], self.fb[i], 0 if last else 1, self.slope,
                         None if last else self.masks[i], self.keep, out, s)
            x, xb = out, 0
        cf.cf_mse(self.pred.numel(), self.pred, self.target, self.loss, self.dpred, s)

    def backward(self, stream=None):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        n, D, L = self.n, self.dims, len(self.fw)
        g = self.dpred
        for i in range(L - 1, -1, -1):
            last = i == L - 1
            x, xb = (self.stack.y[-1], 1) if i == 0 else (self.h[i - 1], 0)
            dx, dxb = (self.dfeat, 1) if i == 0 else (self.dh[i - 1], 0)
            cf.cf_fc_bwd(n, D[i], D[i + 1], x, xb, self.fw[i], None if last else self.h[i], self.slope,
                         None if last else self.masks[i], self.keep, g, dx, dxb, self.dfw[i], self.dfb[i], s)
            g = dx if i > 0 else None
        self.stack.backward(self.dfeat, s)

    def matrices(self):
        """(fp32 tensor, bf16 copy or None, gradient) of the parameters that optimizer="muon" orthogonalises."""
        st = self.stack
        return [(self.w32[l], st.w[l], st.dw[l]) for l in range(st.L)] + \
            [(self.fw[i], None, self.dfw[i]) for i in range(len(self.fw) - 1)]

    def _on(self, stream):
        """Torch's own work of a first step (the optimizer's zeroed state) in the order of the step's stream."""
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int) else stream)

    def _muon_update(self, lr, momentum, weight_decay, stream):
        if self._muon is None:
            with self._on(stream):
                ms = [torch.zeros_like(p) for p, _, _ in self.matrices()]
                params = cf.cf_muon_params([(p, p16, g, m, 0.2 * max(p.shape[0], p.numel() // p.shape[0]) ** 0.5)
                                            for (p, p16, g), m in zip(self.matrices(), ms)])
                size = cf.cf_muon_workspace_size(params)
                self._muon = (ms, params, torch.empty((max(size, 16),), dtype=torch.uint8, device=self.device), size)
        _, params, ws, size = self._muon
        hyper = cf.cf_muon_hyper(lr, momentum, weight_decay, 1, 5, 3.4445, -4.7750, 2.0315, 1e-7)
        cf.cf_muon_step(params, hyper, ws, size, stream)

    def update(self, lr, beta1=0.9, beta2=0.999, eps=1e-8, stream=None, momentum=0.95, weight_decay=0.0):
        """One step of every parameter (step counter t advances): Adam, or with optimizer="muon" the orthogonalised
        momentum step (momentum, weight_decay) of matrices() and Adam for the rest."""
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        ps = self.params()
        if self.optimizer == "muon":
            self._muon_update(lr, momentum, weight_decay, s)
            taken = {p.data_ptr() for p, _, _ in self.matrices()}
            ps = [t for t in ps if t[0].data_ptr() not in taken]
        if self._adam is None:
            with self._on(s):
                self._adam = [(torch.zeros_like(p), torch.zeros_like(p)) for p, _, _ in ps]
        self.t += 1
        for (p, p16, g), (m, v) in zip(ps, self._adam):
            cf.cf_adam_step(p.numel(), p, p16, g, m, v, lr, beta1, beta2, eps, self.t, s)

    def step(self, lr, stream=None):
        self.forward(stream)
        self.backward(stream)
        self.update(lr, stream=stream)
