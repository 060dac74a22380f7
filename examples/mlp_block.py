"""A pre-norm MLP block trained with the block preconditioner.

    r = x + residual        the stream
    y = gamma r / rms(r)    layer_norm_forward(center=False)
    z = y W1^T,  h = max(z, 0)^2,  out = h W2^T

Between the two passes the block keeps no 16-bit activation: the norm leaves the 8-bit
checkpoint of its normalised rows, and h is compressed.  Both are read back where they are
used: the norm's backward pass and the weight gradients decode them on the way in, and the
activation's derivative 2 sqrt(h) comes from the restored h.  The weight gradients leave in
the (N, B, B) blocks that shampoo_accumulate takes, and the preconditioned step updates
the weights in the same blocks.

    python examples/mlp_block.py [--steps 30] [--tokens 4096] [--dim 2048] [--hidden 5632]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import matrix_inverse_roots_gb300 as dr  # noqa: E402


class Weight:
    """A (rows, cols) weight as fp32 blocks, its 16-bit copy and its Shampoo factors."""

    def __init__(self, value, block, beta=0.95, vectors=16):
        self.shape, self.beta, self.ridge = value.shape, beta, None
        self.blocks, self.vr, self.vc = dr.pack_blocks(value, block)
        n = self.blocks.shape[0]
        self.factors = torch.zeros((2 * n, block, block), device=value.device)
        self.start = torch.randn((2 * n, block, vectors), device=value.device)
        self._copy()

    def _copy(self):
        self.w16 = dr.unpack_blocks(self.blocks, *self.shape).to(torch.bfloat16)

    def step(self, grad, lr):
        """W -= lr L^(-1/4) G R^(-1/4) on the gradient's blocks."""
        dr.shampoo_accumulate(grad, self.factors, self.beta, self.vr, self.vc)
        if self.ridge is None:  # from the first gradient: 1e-4 of its factors' norm
            lam = dr.spectral_scale(self.factors, V0=self.start)
            self.ridge = 1e-4 * float(lam.max())
        lam = dr.spectral_scale(self.factors, V0=self.start, ridge=self.ridge)
        roots = dr.inv_root_cn(self.factors, lam, iters=12, ridge=self.ridge)
        dr.precondition_update(grad, roots, self.blocks, lr)
        self._copy()


class MlpBlock:
    def __init__(self, dim, hidden, block, device="cuda", generator=None):
        def draw(rows, cols):
            w = torch.randn((rows, cols), device=device, generator=generator)
            return w / cols ** 0.5

        self.block, self.dim, self.hidden = block, dim, hidden
        self.gamma = torch.ones(dim, device=device)
        self.w1 = Weight(draw(hidden, dim), block)
        self.w2 = Weight(draw(dim, hidden), block)

    def forward(self, x, residual, train=True):
        """(out, r).  In training the block keeps what its backward pass needs."""
        n = dr.layer_norm_forward(x, self.gamma, center=False, residual=residual, stats=train,
                                  ckpt="int8" if train else None)
        h = torch.relu(n.y @ self.w1.w16.T).square_()
        if train:
            # h is far from normal, with many small values: a floating-point code.
            self.kept = (n.rstd, n.q, n.scale) + dr.act_compress(h, "e4m3")
        return h @ self.w2.w16.T, n.r

    def backward(self, dout, dr_out):
        """(dx, dgamma, dW1 blocks, dW2 blocks) from the gradients of out and r.  dx is the
        gradient of x and of residual."""
        rstd, q, scale, hq, hscale = self.kept
        dw2, _ = dr.weight_grad(dout, hq, hscale, self.hidden, "e4m3", B=self.block)
        dz = dr.act_restore(hq, hscale, self.hidden, "e4m3", dout.dtype).sqrt_().mul_(2)
        dz *= dout @ self.w2.w16
        dw1, _ = dr.weight_grad(dz, q, scale, self.dim, "int8", gamma=self.gamma, B=self.block)
        dx, dgamma, _ = dr.layer_norm_backward(dz @ self.w1.w16, rstd, self.gamma, q=q,
                                               scale=scale, center=False, dres=dr_out,
                                               beta=False)
        return dx, dgamma, dw1, dw2


def train(steps=30, tokens=4096, dim=2048, hidden=5632, block=1024, lr=1e-2, seed=1, log=print):
    """Fits the block to a fixed random block of the same shape; the losses."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    teacher = MlpBlock(dim, hidden, block, generator=g)
    net = MlpBlock(dim, hidden, block, generator=g)
    losses = []
    for i in range(steps):
        x, res = (torch.randn((tokens, dim), device="cuda", generator=g).to(torch.bfloat16)
                  for _ in range(2))
        want, _ = teacher.forward(x, res, train=False)
        out, _ = net.forward(x, res)
        diff = out.float() - want.float()
        losses.append(float(diff.square().mean()))
        # The gradient of half the sum of squares over tokens, averaged over them.
        dout = (diff / tokens ** 0.5).to(torch.bfloat16)
        _, dgamma, dw1, dw2 = net.backward(dout, torch.zeros_like(dout))
        net.gamma -= 1e-3 * dgamma / tokens ** 0.5
        net.w1.step(dw1, lr)
        net.w2.step(dw2, lr)
        log("step %3d  loss %.4f" % (i, losses[-1]))
    # Serving: a single token, no statistics, nothing kept.
    one, _ = net.forward(x[:1], res[:1], train=False)
    many, _ = net.forward(x, res, train=False)
    log("one token against the batch: %.1e" % float((one - many[:1]).abs().max()))
    if dr.device_status() != 0:
        raise RuntimeError("device error %d" % dr.device_status())
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--dim", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=5632)
    ap.add_argument("--block", type=int, default=1024)
    ap.add_argument("--lr", type=float, default=1e-2)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.dim, a.hidden, a.block, a.lr)


if __name__ == "__main__":
    main()
