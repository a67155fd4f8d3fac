"""Residual blocks on the voxels of a feature map, through the C ABI: norm, widening product with GELU, product back, and the
gated sum on the stream (the pages have no such blocks; they stand between a CosmoStack and a head).

A block takes the stream x [rows][c] (rows: voxels of all samples, channels last) to

  h = N(x);  a = GELU(h W1^T + b1);  f = a W2^T + b2;  x' = x + gate N_post(f)

with root-mean-square norms.  The norm of one block and the sum of the one before are one call (cf_residual_norm_fwd), the products
carry their biases and the activation (cf_linear_fwd), and their backward data the activation's derivative (cf_linear_dgrad).

Python only owns buffers and enqueues library calls.  Weights are fp32 masters with bf16 copies (sync_master), as a CosmoFlowModel's
filters are."""
from __future__ import annotations

import torch

from . import cfconv as cf


class VoxelMLP:
    eps = 1e-6

    def __init__(self, rows: int, c: int, blocks: int, expansion: int = 4, device: str = "cuda", backward: bool = True):
        if rows < 1 or c < 1 or blocks < 1 or expansion < 1:
            raise ValueError(f"VoxelMLP of {blocks} blocks, {rows} rows of {c} channels, expansion {expansion}")
        self.rows, self.c, self.blocks, self.wide = rows, c, blocks, expansion * c
        f32, bf = torch.float32, torch.bfloat16
        B, n = range(blocks), self.wide
        new = lambda dt, *shape: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        # trained: masters, copies, biases, the norms' gammas and the gates
        self.w1, self.w2 = [torch.zeros((n, c), dtype=f32, device=device) for _ in B], [torch.zeros((c, n), dtype=f32, device=device) for _ in B]
        self.w1_16, self.w2_16 = [new(bf, n, c) for _ in B], [new(bf, c, n) for _ in B]
        self.b1, self.b2 = [torch.zeros((n,), dtype=f32, device=device) for _ in B], [torch.zeros((c,), dtype=f32, device=device) for _ in B]
        self.gamma, self.post, self.gate = ([torch.ones((c,), dtype=f32, device=device) for _ in B] for _ in range(3))
        # the stream after each block, what is kept for the backward
        self.r, self.h, self.f = ([new(bf, rows, c) for _ in B] for _ in range(3))
        self.z, self.a = ([new(bf, rows, n) for _ in B] for _ in range(2))
        self.stats = [new(f32, rows, 4) for _ in range(blocks + 1)]
        self.backward_enabled = backward
        rms, no, dt = cf.CF_NORM_RMS, cf.CF_NORM_NONE, cf.CF_DT_BF16
        norm = lambda post, pre: cf.cf_residual_norm_desc(rows, c, post, pre, self.eps, 1.0, dt, dt, 0, 0)  # noqa: E731
        # the norm before the first block, then what follows each block: its sum, and the next one's norm if there is one
        self.norms = [norm(no, rms)] + [norm(rms, rms if l + 1 < blocks else no) for l in B]
        vectors = lambda post, gate, gamma: [  # noqa: E731
            cf.cf_residual_norm_vectors(post_gamma=post[l - 1] if l else None, gate=gate[l - 1] if l else None,
                                        pre_gamma=gamma[l] if l < blocks else None) for l in range(blocks + 1)]
        self.vectors = vectors(self.post, self.gate, self.gamma)
        self.up = cf.cf_linear_desc(rows, c, n, cf.CF_ACT_GELU, 1.0, 1.0, dt, 0, 0)
        self.down = cf.cf_linear_desc(rows, n, c, cf.CF_ACT_LRELU, 1.0, 1.0, dt, 0, 0)
        # backward data of the product back with GELU's derivative in it, and of the widening one with none
        self.down_act = cf.cf_linear_desc(rows, n, c, cf.CF_ACT_GELU, 1.0, 1.0, dt, 0, 0)
        size = max(cf.cf_linear_workspace_size(d, op) for d in (self.up, self.down) for op in range(3))
        if backward:
            self.dw1, self.dw2 = [new(f32, n, c) for _ in B], [new(f32, c, n) for _ in B]
            self.db1, self.db2 = [new(f32, n) for _ in B], [new(f32, c) for _ in B]
            self.dgamma, self.dpost, self.dgate = ([new(f32, c) for _ in B] for _ in range(3))
            self.grads = vectors(self.dpost, self.dgate, self.dgamma)
            self.df, self.dh, self.dr = new(bf, rows, c), new(bf, rows, c), [new(bf, rows, c) for _ in range(2)]
            self.dz = new(bf, rows, n)
            size = max([size] + [cf.cf_residual_norm_workspace_size(d) for d in self.norms])
        self.ws, self.ws_bytes = torch.empty((max(size, 16),), dtype=torch.uint8, device=device), size

    def sync_master(self):
        """The products' bf16 copies from their masters."""
        for w, w16 in zip(self.w1 + self.w2, self.w1_16 + self.w2_16):
            w16.copy_(w)

    def params(self):
        """(fp32 tensor, bf16 copy or None, gradient) of every trained parameter."""
        out = []
        for l in range(self.blocks):
            out += [(self.w1[l], self.w1_16[l], self.dw1[l]), (self.b1[l], None, self.db1[l]), (self.w2[l], self.w2_16[l], self.dw2[l]),
                    (self.b2[l], None, self.db2[l]), (self.gamma[l], None, self.dgamma[l]), (self.post[l], None, self.dpost[l]),
                    (self.gate[l], None, self.dgate[l])]
        return out

    def matrices(self):
        return [t for t in self.params() if t[0].dim() == 2]

    def forward(self, x, stream=None):
        """The stream after the last block, from x [rows][c] bf16, which the backward reads again."""
        s, ws = stream, (self.ws, self.ws_bytes, stream)
        cf.cf_residual_norm_fwd(self.norms[0], x, None, self.vectors[0], None, self.h[0], self.stats[0], s)
        for l in range(self.blocks):
            cf.cf_linear_fwd(self.up, self.h[l], self.w1_16[l], self.b1[l], None, self.a[l], self.z[l], *ws)
            cf.cf_linear_fwd(self.down, self.a[l], self.w2_16[l], self.b2[l], None, self.f[l], None, *ws)
            last = l + 1 == self.blocks
            cf.cf_residual_norm_fwd(self.norms[l + 1], x, self.f[l], self.vectors[l + 1], self.r[l], None if last else self.h[l + 1],
                                    self.stats[l + 1], s)
            x = self.r[l]
        return x

    def backward(self, x, dr, dx, stream=None):
        """All gradients and dx, the gradient at x, from dr, the gradient at forward()'s result."""
        ws = (self.ws, self.ws_bytes, stream)
        dh = None
        for l in range(self.blocks - 1, -1, -1):
            to = self.dr[l & 1]
            cf.cf_residual_norm_bwd(self.norms[l + 1], self.f[l], self.r[l], self.vectors[l + 1], self.stats[l + 1], dh, dr, to, self.df,
                                    self.grads[l + 1], *ws)
            cf.cf_linear_wgrad(self.down, self.a[l], self.df, self.dw2[l], self.db2[l], 0, *ws)
            cf.cf_linear_dgrad(self.down_act, self.df, self.w2_16[l], self.z[l], None, self.dz, *ws)
            cf.cf_linear_wgrad(self.up, self.h[l], self.dz, self.dw1[l], self.db1[l], 0, *ws)
            cf.cf_linear_dgrad(self.up, self.dz, self.w1_16[l], None, None, self.dh, *ws)
            dh, dr = self.dh, to
        cf.cf_residual_norm_bwd(self.norms[0], None, x, self.vectors[0], self.stats[0], dh, dr, dx, None, self.grads[0], *ws)
