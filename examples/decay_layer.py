"""A layer of linear attention with a decay for each head, with hand-written
gradients, a prompt of sequences of different lengths and decoding.

    q, k, v = x W                          (one projection, split into heads)
    q, k = norm and rotation of q, k       (positions; RMS norm of every head)
    o = decaying linear attention(q, k, v) (a decay for each head)
    y = LN(o) W_o                          (layer norm of every head's output)

The library's calls do everything but the plain matrix products.  Run as a
script it runs a batch of prompts, goes on token by token and compares with the
whole sequences.

    python examples/decay_layer.py [--dtype f32|bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_recurrence_gb300 import la  # noqa: E402


class DecayLayer:
    """Weights are fp32; activations are of `dtype`, states fp32."""

    def __init__(self, C, heads, dtype=torch.float32, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.C, self.H, self.D, self.dtype = C, heads, C // heads, dtype
        self.p = {"W": torch.randn(C, 3 * C, generator=g) / C ** 0.5, "Wo": torch.randn(C, C, generator=g) / C ** 0.5,
                  "wq": torch.ones(self.D), "wk": torch.ones(self.D), "wn": torch.ones(self.D), "bn": torch.zeros(self.D)}
        self.p = {n: t.to(device) for n, t in self.p.items()}
        # memories of 4 tokens to about a thousand
        self.log_decay = torch.log1p(-torch.exp2(-torch.linspace(2, 10, heads))).to(device)
        self.freq = (10000.0 ** (-torch.arange(self.D // 2) / (self.D // 2))).to(device)
        self.scale = self.D ** -0.5

    def _heads(self, x):     # [B, N, 3 C] -> three views [B, H, N, D]
        return x.unflatten(-1, (3, self.H, self.D)).permute(2, 0, 3, 1, 4)

    def forward(self, x, pos, lens=None, state=None):
        """y of x [B, N, C] at positions pos [B, N]; state [B, H, D, D] (or None), if given, is started from and left
        after each sequence's own length.  Keeps what backward() needs."""
        q0, k0, v = self._heads(x @ self.p["W"].to(self.dtype))
        q, k = la.la_qk_rotate_forward(q0, k0, pos, self.freq, self.p["wq"], self.p["wk"])
        start = None if state is None else state.clone()
        o = la.la_decay_forward(q, k, v, self.log_decay, self.scale, S0=start, SN=state, lens=lens)
        n, s, mean, rstd = la.la_layernorm_forward(o, self.p["wn"], self.p["bn"])
        joined = n.transpose(1, 2).flatten(2)
        self.saved = (x, pos, lens, start, q0, k0, q, k, v, s, mean, rstd, joined)
        return joined @ self.p["Wo"].to(self.dtype)

    def backward(self, dy):
        """Gradients of the weights (fp32, by name) and of x, given dL/dy."""
        x, pos, lens, start, q0, k0, q, k, v, s, mean, rstd, joined = self.saved
        d = {"Wo": joined.flatten(0, 1).T.float() @ dy.flatten(0, 1).float()}
        dn = (dy @ self.p["Wo"].to(self.dtype).T).unflatten(-1, (self.H, self.D)).transpose(1, 2).contiguous()
        do, d["wn"], d["bn"] = la.la_layernorm_backward(dn, s, self.p["wn"], mean, rstd)
        dqkv = torch.empty(x.shape[:2] + (3 * self.C,), dtype=self.dtype, device=x.device)
        dq, dk, dv = self._heads(dqkv)      # the gradients go where the projection's lie
        la.la_decay_backward(q, k, v, do, self.log_decay, self.scale, S0=start, lens=lens, dq=dq, dk=dk, dv=dv)
        _, _, d["wq"], d["wk"] = la.la_qk_rotate_backward(dq, dk, q0, k0, pos, self.freq, self.p["wq"], self.p["wk"],
                                                          dq=dq, dk=dk)
        d["W"] = x.flatten(0, 1).T.float() @ dqkv.flatten(0, 1).float()
        return d, dqkv @ self.p["W"].to(self.dtype).T

    def step(self, x, pos, state):
        """y of one token x [B, C] at positions pos [B]; the state is updated in place."""
        q, k, v = self._heads((x @ self.p["W"].to(self.dtype))[:, None])
        q, k = la.la_qk_rotate_forward(q, k, pos[:, None], self.freq, self.p["wq"], self.p["wk"])
        o = la.la_decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], state, self.log_decay, self.scale)
        n = la.la_layernorm_forward(o, self.p["wn"], self.p["bn"], stats=False)[0]
        return n.flatten(1) @ self.p["Wo"].to(self.dtype)


def prompts_then_tokens(B=4, N=300, extra=20, C=256, heads=4, dtype=torch.float32, seed=0):
    """Prompts of different lengths in one call, then tokens one by one; the largest
    difference of the tokens' outputs from those of the whole sequences."""
    layer = DecayLayer(C, heads, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(B, N + extra, C, generator=g).to(dtype).cuda()
    lens = torch.linspace(1, N, B).int().cuda()
    state = torch.zeros(B, heads, C // heads, C // heads, device="cuda")
    at = torch.arange(N + extra, device="cuda", dtype=torch.int32).expand(B, -1)
    layer.forward(x[:, :N], at[:, :N], lens, state)
    each = []
    for t in range(extra):
        here = lens + t
        each.append(layer.step(x[torch.arange(B), here.long()], here, state))
    whole = layer.forward(x, at)
    off = [each[t][b] - whole[b, int(lens[b]) + t] for t in range(extra) for b in range(B)]
    return float(torch.stack(off).float().abs().max()), float(whole.float().abs().max())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    off, size = prompts_then_tokens(dtype=torch.float32 if a.dtype == "f32" else torch.bfloat16)
    print("tokens after the prompts against the whole sequences: largest difference %.3g of %.3g" % (off, size))
