"""A layer that mixes tokens twice, by a gated linear recurrence and by causal
linear attention, trained and then run token by token.

    s1 = x                      y1 = LN(s1)
    h  = recurrence(y1 Wx, y1 Wg)          (sigmoid gate)
    s2 = s1 + h Wh              y2 = LN(s2)
    o  = linear attention(y2 Wq, y2 Wk, y2 Wv)
    s3 = s2 + o Wo              y3 = LN(s3)

The forward pass, the gradients by the chain rule, the clipping of them and
the decoding step call the library for everything but the plain matrix
products.  Run as a script it trains on a synthetic task (each token's target
is the running mean of the tokens so far, seen through a fixed matrix), then
decodes the same sequence from an empty state and compares.

    python examples/hybrid_layer.py [--steps 60] [--dtype f32|bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_recurrence_gb300 import la  # noqa: E402


class HybridLayer:
    """Weights are fp32; activations are of `dtype`, states fp32."""

    MATRICES = ("Wx", "Wg", "Wh", "Wq", "Wk", "Wv", "Wo")
    NORMS = ("w1", "b1", "w2", "b2", "w3", "b3")

    def __init__(self, C, heads, dtype=torch.float32, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.C, self.heads, self.dtype, self.device = C, heads, dtype, device
        self.p = {n: (torch.randn(C, C, generator=g) / C ** 0.5).to(device) for n in self.MATRICES}
        for n in self.NORMS:
            self.p[n] = (torch.ones(C) if n[0] == "w" else torch.zeros(C)).to(device)

    def _mm(self, x, name):
        return x @ self.p[name].to(self.dtype)

    def _split(self, x):   # [B, N, C] -> [B, H, N, C / H]
        B, N, C = x.shape
        return x.view(B, N, self.heads, C // self.heads).transpose(1, 2).contiguous()

    def _join(self, x):
        B, H, N, D = x.shape
        return x.transpose(1, 2).reshape(B, N, H * D)

    def forward(self, x):
        """y3 of x [B, N, C]; keeps what backward() needs."""
        p = self.p
        y1, s1, m1, r1 = la.la_layernorm_forward(x, p["w1"], p["b1"])
        u, g = self._mm(y1, "Wx"), self._mm(y1, "Wg")
        h = la.la_recurrence_forward(u, g, "sigmoid")
        y2, s2, m2, r2 = la.la_layernorm_forward(self._mm(h, "Wh"), p["w2"], p["b2"], res=s1)
        q, k, v = (self._split(self._mm(y2, n)) for n in ("Wq", "Wk", "Wv"))
        o = self._join(la.la_forward_causal(q, k, v))
        y3, s3, m3, r3 = la.la_layernorm_forward(self._mm(o, "Wo"), p["w3"], p["b3"], res=s2)
        self.saved = (y1, s1, m1, r1, u, g, h, y2, s2, m2, r2, q, k, v, o, s3, m3, r3)
        return y3

    def backward(self, dy3):
        """Gradients of every weight (fp32, by name) and of x, given dL/dy3."""
        y1, s1, m1, r1, u, g, h, y2, s2, m2, r2, q, k, v, o, s3, m3, r3 = self.saved
        p, d = self.p, {}

        def mm(dout, x, name):   # of x @ W: dW kept, dx returned
            d[name] = x.reshape(-1, self.C).T.float() @ dout.reshape(-1, self.C).float()
            return dout @ p[name].to(self.dtype).T
        ds3, d["w3"], d["b3"] = la.la_layernorm_backward(dy3, s3, p["w3"], m3, r3)
        dq, dk, dv = la.la_backward_causal(q, k, v, self._split(mm(ds3, o, "Wo")))
        dy2 = mm(self._join(dq), y2, "Wq") + mm(self._join(dk), y2, "Wk") + mm(self._join(dv), y2, "Wv")
        ds2, d["w2"], d["b2"] = la.la_layernorm_backward(dy2, s2, p["w2"], m2, r2, dsum=ds3)
        du, dg = la.la_recurrence_backward(u, g, h, mm(ds2, h, "Wh"), "sigmoid")
        dy1 = mm(du, y1, "Wx") + mm(dg, y1, "Wg")
        dx, d["w1"], d["b1"] = la.la_layernorm_backward(dy1, s1, p["w1"], m1, r1, dsum=ds2)
        return d, dx

    def update(self, d, rate, max_norm):
        """One clipped gradient step; returns the gradients' norm (on the device)."""
        names = list(d)
        norm = la.la_grad_clip([d[n] for n in names], max_norm)
        for n in names:
            self.p[n].sub_(d[n], alpha=rate)
        return norm

    def empty_state(self, B):
        D = self.C // self.heads
        z = dict(dtype=torch.float32, device=self.device)
        return (torch.zeros(B, self.C, **z), torch.zeros(B, self.heads, D, D, **z), torch.zeros(B, self.heads, D, **z))

    def step(self, x, state):
        """y3 of one token x [B, C]; the state (h, S, z) is updated in place."""
        h, S, z = state
        p, B = self.p, x.shape[0]
        y1, s1, _, _ = la.la_layernorm_forward(x, p["w1"], p["b1"], stats=False)
        y = la.la_recurrence_step(self._mm(y1, "Wx"), self._mm(y1, "Wg"), h, "sigmoid")
        y2, s2, _, _ = la.la_layernorm_forward(self._mm(y, "Wh"), p["w2"], p["b2"], res=s1, stats=False)
        q, k, v = (self._mm(y2, n).view(B, self.heads, -1) for n in ("Wq", "Wk", "Wv"))
        o = la.la_decode_step(q, k, v, S, z).reshape(B, self.C)
        return la.la_layernorm_forward(self._mm(o, "Wo"), p["w3"], p["b3"], res=s2, stats=False)[0]


def task(B, N, C, dtype, seed, device="cuda"):
    """x [B, N, C] and its targets."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, C, generator=g)
    fixed = torch.randn(C, C, generator=torch.Generator().manual_seed(99)) / C ** 0.5
    mean = x.cumsum(dim=1) / torch.arange(1, N + 1).sqrt()[None, :, None]
    return x.to(dtype).to(device), (mean @ fixed).to(device)


def train(steps=60, B=8, N=256, C=128, heads=2, dtype=torch.float32, rate=0.3, max_norm=1.0, verbose=False):
    """Losses of a training run, and the largest difference between the trained
    layer's outputs token by token and its forward pass."""
    layer = HybridLayer(C, heads, dtype)
    losses = []
    for i in range(steps):
        x, target = task(B, N, C, dtype, seed=i)
        off = layer.forward(x).float() - target
        losses.append((off * off).mean())
        norm = layer.update(layer.backward((2.0 / C / 8 * off).to(dtype))[0], rate, max_norm)
        if verbose and (i % 10 == 0 or i == steps - 1):
            print("step %3d   loss %.4f   gradient norm %.3f" % (i, losses[-1].item(), norm.item()))
    x, _ = task(B, N, C, dtype, seed=0)
    whole, state = layer.forward(x), layer.empty_state(B)
    each = torch.stack([layer.step(x[:, t].contiguous(), state) for t in range(N)], dim=1)
    return [v.item() for v in losses], float((each.float() - whole.float()).abs().max())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    losses, off = train(a.steps, dtype=torch.float32 if a.dtype == "f32" else torch.bfloat16, verbose=True)
    print("token by token against the whole sequence: largest difference %.3g" % off)
