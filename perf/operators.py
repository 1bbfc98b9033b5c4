"""Cases of the operators around the attention: the gated linear recurrence
(forward, backward, single step), layer norm (forward, backward, residual sum)
and the global gradient norm with clipping.

``run`` computes a case in plain torch operations (``own`` false) or through
the library's entry points (``own`` true); ``exact`` computes it in 64 bits
from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one decoded token for a batch of 64 sequences: latency
        dict(name="rec_step_b64_d1024", op="rec_step", B=64, H=1, N=1, D=1024, dtype="bf16", gate="sigmoid",
             ragged=False, strided=False),
        # prefill of one long document, few channels: the time axis has to be split
        dict(name="rec_fwd_n65536_d1024", op="rec_fwd", B=1, H=1, N=65536, D=1024, dtype="bf16", gate="sigmoid",
             ragged=False, strided=False),
        # prompts of different lengths (one empty) in head layout, x and g two halves of one projection,
        # decays given, some of them 0 (a document starts)
        dict(name="rec_fwd_ragged_b7h5_f32", op="rec_fwd", B=7, H=5, N=1537, D=64, dtype="f32", gate="decay",
             ragged=True, strided=True),
        # a training batch
        dict(name="rec_train_b8n4096_d2048", op="rec_train", B=8, H=1, N=4096, D=2048, dtype="bf16", gate="sigmoid",
             ragged=False, strided=False),
        # odd sizes, log decays, state and its gradient carried between segments of a sequence
        dict(name="rec_train_odd_f32", op="rec_train", B=3, H=1, N=5001, D=333, dtype="f32", gate="log",
             ragged=False, strided=False),
        # the norm before a decoded token's next layer, with the residual sum
        dict(name="ln_fwd_r16_c2048", op="ln_fwd", R=16, C=2048, dtype="bf16", res=True),
        # per-head norm of the attention's outputs [2, 16, 8192, 64]
        dict(name="ln_fwd_heads_c64", op="ln_fwd", R=2 * 16 * 8192, C=64, dtype="bf16", res=False),
        # a training batch, residual stream
        dict(name="ln_train_r32768_c2048", op="ln_train", R=32768, C=2048, dtype="bf16", res=True),
        # odd sizes
        dict(name="ln_train_odd_f32", op="ln_train", R=4099, C=1001, dtype="f32", res=False),
        # a small layer's gradients: latency
        dict(name="clip_small_f32", op="clip", layers=2, width=64, vocab=0, dtype="f32"),
        # a language model's gradients, matrices bf16 and vectors fp32
        dict(name="clip_model_mixed", op="clip", layers=24, width=1024, vocab=32000, dtype="mixed"),
        # the norm alone (logged every step), odd sizes
        dict(name="norm_odd_f32", op="norm", layers=12, width=333, vocab=5003, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rec_step", "rec_fwd", "rec_train", "ln_fwd", "ln_train", "clip", "norm"])
    if op.startswith("rec"):
        heads = rng.random() < 0.4
        D = rng.choice([16, 32, 64, 128]) if heads else _log_int(rng, 16, 2048)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        H = rng.randint(1, 12) if heads else 1
        N = 1 if op == "rec_step" else _log_int(rng, 2, 65536)
        B = min(_log_int(rng, 1, 256 if op == "rec_step" else 32), max(1, (8 * 4096 * 2048) // (2 * H * N * D)))
        H = min(H, max(1, (8 * 4096 * 2048) // (2 * B * N * D)))
        return dict(op=op, B=B, H=H, N=N, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    gate=rng.choice(["sigmoid", "sigmoid", "decay", "log"]),
                    ragged=op != "rec_step" and rng.random() < 0.3, strided=rng.random() < 0.3)
    if op.startswith("ln"):
        C = rng.choice([64, 128, 256, 512, 1024, 2048, 4096, 8192]) if rng.random() < 0.6 else _log_int(rng, 16, 8192)
        R = min(_log_int(rng, 1, 262144), (32768 * 2048) // (2 * C))
        return dict(op=op, R=R, C=C, dtype=rng.choice(["bf16", "bf16", "f32"]), res=rng.random() < 0.5)
    width = _log_int(rng, 32, 1024)
    layers = rng.randint(1, 12)
    return dict(op=op, layers=layers, width=width, vocab=_log_int(rng, 100, 32000),
                dtype=rng.choice(["bf16", "f32", "mixed"]))


# ---------------------------------------------------------------- inputs

def _lens(case):
    """Lengths of a ragged batch: spread from an empty sequence to a full one."""
    B, N = case["B"], case["N"]
    return [N] if B == 1 else [N * i // (B - 1) for i in range(B)]


def _tensors(case):
    """(elements, dtype) of every gradient of a model: per layer four matrices,
    two vectors and a scalar-sized one; the embedding."""
    w, t = case["width"], case["dtype"]
    big = DTYPES["bf16" if t == "mixed" else t]
    small = DTYPES["f32" if t == "mixed" else t]
    one = [(w * w, big)] * 4 + [(w, small)] * 2 + [(1, small)]
    return one * case["layers"] + ([(case["vocab"] * w, big)] if case["vocab"] else [])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    st = dict(case=dict(case))
    if case["op"].startswith("rec"):
        B, H, N, D, dt = case["B"], case["H"], case["N"], case["D"], DTYPES[case["dtype"]]
        # time constants from about one token to about a thousand, by channel
        rate = torch.linspace(0.0, 6.9, D, device=DEV)
        n = normal(B, H, N, D)
        if case["gate"] == "sigmoid":
            gates = rate + n
        elif case["gate"] == "log":
            gates = -torch.exp(-rate) * (1.0 + torch.exp(n)).log()
        else:
            gates = torch.exp(-torch.exp(-rate) * n.abs())
            gates = gates * (torch.rand((B, H, N, 1), generator=g, device=DEV) > 1.0 / 256)
        x = normal(B, H, N, D)
        if case["strided"]:   # both from one projection, token-major: [B, N, H, 2D]
            both = torch.cat([x, gates], dim=-1).to(dt).transpose(1, 2).contiguous()
            st["x"], st["g"] = both[..., :D].transpose(1, 2), both[..., D:].transpose(1, 2)
        else:
            st["x"], st["g"] = x.to(dt), gates.to(dt)
        if case["op"] == "rec_step":
            st["x"], st["g"] = st["x"][:, :, 0], st["g"][:, :, 0]
        st["h0"] = normal(B, H, D)
        st["hN"] = torch.zeros_like(st["h0"])
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
        if case["op"] == "rec_train":
            st["dout"] = normal(B, H, N, D).to(dt)
            st["dhN"] = normal(B, H, D)
    elif case["op"].startswith("ln"):
        R, C, dt = case["R"], case["C"], DTYPES[case["dtype"]]
        st["x"] = (normal(R, C) + 0.5 * normal(R, 1)).to(dt)
        st["res"] = normal(R, C).to(dt) if case["res"] else None
        st["w"], st["b"] = 1.0 + 0.2 * normal(C), 0.2 * normal(C)
        if case["op"] == "ln_train":
            st["dy"] = normal(R, C).to(dt)
            st["dsum"] = normal(R, C).to(dt) if case["res"] else None
    else:
        scale = 0.01
        st["grads"] = [(scale * normal(n)).to(dt) for n, dt in _tensors(case)]
        # a tenth of the norm these values have, so that the factor is not 1
        st["max_norm"] = 0.1 * scale * math.sqrt(sum(n for n, _ in _tensors(case)))
        if case["op"] == "clip":   # the optimiser's flat buffer, each gradient on a 16-byte boundary
            st["flat"], st["dst"] = {}, [None] * len(st["grads"])
            for name, dt in DTYPES.items():
                at, off = [i for i, t in enumerate(st["grads"]) if t.dtype == dt], 0
                pad = [(st["grads"][i].numel() + 7) // 8 * 8 for i in at]
                if at:
                    st["flat"][name] = flat = torch.zeros(sum(pad), dtype=dt, device=DEV)
                for i, p in zip(at, pad):
                    st["dst"][i] = flat[off:off + st["grads"][i].numel()]
                    off += p
    return st


# ---------------------------------------------------------------- the plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 2 (h before the first is 0), by pairs:
    two neighbours are one affine map, so half as many positions remain."""
    n = a.shape[2]
    if n == 1:
        return b
    m = n // 2 * 2
    odd = _scan(a[:, :, 1:m:2] * a[:, :, 0:m:2], a[:, :, 1:m:2] * b[:, :, 0:m:2] + b[:, :, 1:m:2])
    h = torch.empty_like(b)
    h[:, :, 1:m:2] = odd
    h[:, :, 0] = b[:, :, 0]
    h[:, :, 2::2] = a[:, :, 2::2] * odd[:, :, :(n - 1) // 2] + b[:, :, 2::2]
    return h


def _gates(gate, x, g):
    """a, u of h = a h + u, and du/dx.  e^g of small g is next to 1 and enters a
    product over thousands of tokens, where a 32-bit exponential that is mostly
    off to one side shows: it is computed in 64 bits and rounded once."""
    if gate == "sigmoid":
        w = 1.0 / (1.0 + torch.exp(g))
        return 1.0 / (1.0 + torch.exp(-g)), w * x, w
    return (torch.exp(g.double()).float() if gate == "log" else g), x, 1.0


def _plain_rec(st):
    c = st["case"]
    gate, dt = c["gate"], DTYPES[c["dtype"]]
    if c["op"] == "rec_step":
        a, u, _ = _gates(gate, st["x"].float(), st["g"].float())
        h = a * st["h0"] + u
        st["h0"].copy_(h)
        return h.to(dt), st["h0"]
    x, g, h0 = st["x"].float(), st["g"].float(), st["h0"]
    a, u, w = _gates(gate, x, g)
    keep = None
    if st["lens"] is not None:
        keep = (torch.arange(c["N"], device=DEV) < st["lens"][:, None])[:, None, :, None]
        a, u = torch.where(keep, a, 1.0), torch.where(keep, u, 0.0)
    first = u.clone()
    first[:, :, 0] += a[:, :, 0] * h0
    h = _scan(a, first)
    st["hN"].copy_(h[:, :, -1])
    out = (h if keep is None else torch.where(keep, h, 0.0)).to(dt)
    if c["op"] == "rec_fwd":
        return out, st["hN"]
    dout = st["dout"].float()
    if keep is not None:
        dout = torch.where(keep, dout, 0.0)
    else:
        dout = dout.clone()
    dout[:, :, -1] += st["dhN"]
    after = torch.cat([a[:, :, 1:], torch.ones_like(a[:, :, :1])], dim=2)
    lam = _scan(after.flip(2), dout.flip(2)).flip(2)
    before = torch.cat([h0[:, :, None], h[:, :, :-1]], dim=2)
    dh0 = a[:, :, 0] * lam[:, :, 0]
    if gate == "sigmoid":
        dx, dg = lam * w, lam * (before - x) * a * w
    else:
        dx, dg = lam, lam * before * (a if gate == "log" else 1.0)
    if keep is not None:
        dx, dg = torch.where(keep, dx, 0.0), torch.where(keep, dg, 0.0)
    return out, st["hN"], dx.to(dt), dg.to(dt), dh0


def _plain_ln(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    s = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(dt)
    z = s.float()
    mid = z - z.mean(dim=1, keepdim=True)
    rstd = 1.0 / torch.sqrt((mid * mid).mean(dim=1, keepdim=True) + EPS)
    xh = mid * rstd
    y = (xh * st["w"] + st["b"]).to(dt)
    if c["op"] == "ln_fwd":
        return (y, s) if st["res"] is not None else (y,)
    dy = st["dy"].float()
    wdy = dy * st["w"]
    dx = rstd * (wdy - wdy.mean(dim=1, keepdim=True) - xh * (wdy * xh).mean(dim=1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    grads = dx.to(dt), (dy * xh).sum(dim=0), dy.sum(dim=0)
    return (y, s) + grads if st["res"] is not None else (y,) + grads


def _plain_clip(st):
    total = torch.stack([t.float().square().sum() for t in st["grads"]]).sum()
    norm = torch.sqrt(total)
    if st["case"]["op"] == "norm":
        return norm
    c = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    [d.copy_(t.float() * c) for d, t in zip(st["dst"], st["grads"])]
    return norm, st["flat"]


# ---------------------------------------------------------------- through the library

def _own_rec(st):
    from weight_recurrence_gb300 import la
    c = st["case"]
    gate = c["gate"]
    if c["op"] == "rec_step":
        return la.la_recurrence_step(st["x"], st["g"], st["h0"], gate), st["h0"]
    out = la.la_recurrence_forward(st["x"], st["g"], gate, h0=st["h0"], hN=st["hN"], lens=st["lens"])
    if c["op"] == "rec_fwd":
        return out, st["hN"]
    dh0 = torch.empty_like(st["h0"])
    dx, dg = la.la_recurrence_backward(st["x"], st["g"], out, st["dout"], gate, h0=st["h0"], dhN=st["dhN"], dh0=dh0,
                                       lens=st["lens"])
    return out, st["hN"], dx, dg, dh0


def _own_ln(st):
    from weight_recurrence_gb300 import la
    c = st["case"]
    train = c["op"] == "ln_train"
    y, s, mean, rstd = la.la_layernorm_forward(st["x"], st["w"], st["b"], eps=EPS, res=st["res"], stats=train)
    if not train:
        return (y, s) if st["res"] is not None else (y,)
    grads = la.la_layernorm_backward(st["dy"], s, st["w"], mean, rstd, dsum=st["dsum"])
    return (y, s) + grads if st["res"] is not None else (y,) + grads


def _own_clip(st):
    from weight_recurrence_gb300 import la
    if st["case"]["op"] == "norm":
        return la.la_grad_norm(st["grads"])
    return la.la_grad_clip(st["grads"], st["max_norm"], out=st["dst"]), st["flat"]


def run(state):
    op = state["case"]["op"]
    if op.startswith("rec"):
        return _own_rec(state) if own else _plain_rec(state)
    if op.startswith("ln"):
        return _own_ln(state) if own else _plain_ln(state)
    return _own_clip(state) if own else _plain_clip(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"].startswith("rec"):
        size = 2 if case["dtype"] == "bf16" else 4
        rows = sum(_lens(case)) if case["ragged"] else case["B"] * case["N"]
        full = case["B"] * case["N"] * case["H"] * case["D"]
        n, state = rows * case["H"] * case["D"], case["B"] * case["H"] * case["D"] * 4
        # x and g are read, out is written whole (0 past a sequence's end); a training pass also reads dout and writes dx and dg
        if case["op"] == "rec_train":
            return dict(bytes=(3 * n + 3 * full) * size + 4 * state, flops=12 * n)
        return dict(bytes=(2 * n + full) * size + 2 * state, flops=4 * n)
    if case["op"].startswith("ln"):
        size = 2 if case["dtype"] == "bf16" else 4
        n, rows = case["R"] * case["C"], 2 if case["res"] else 1
        if case["op"] == "ln_train":   # x, dy (res, dsum) in; y, dx (s) out
            return dict(bytes=(4 + (3 if case["res"] else 0)) * n * size + 16 * case["C"], flops=20 * n)
        return dict(bytes=2 * rows * n * size + 8 * case["C"], flops=8 * n)
    sizes = [(n, 2 if dt == torch.bfloat16 else 4) for n, dt in _tensors(case)]
    total = sum(n * b for n, b in sizes)
    return dict(bytes=(2 if case["op"] == "clip" else 1) * total + 4, flops=(3 if case["op"] == "clip" else 2) * sum(n for n, _ in sizes))


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rec(st):
    c = st["case"]
    gate, N = c["gate"], c["N"]
    step = c["op"] == "rec_step"
    x, g = (t.unsqueeze(2) if step else t for t in (st["x"], st["g"]))
    # token-major, so that one token of all sequences is one slice
    x, g = (t.permute(2, 0, 1, 3).double().contiguous() for t in (x, g))
    lens = st["lens"].tolist() if st["lens"] is not None else [N] * c["B"]
    length = torch.tensor(lens, device=DEV)[:, None, None]
    inside = [None if min(lens) > t else t < length for t in range(N)]
    a = torch.sigmoid(g) if gate == "sigmoid" else g.exp() if gate == "log" else g
    u = torch.sigmoid(-g) * x if gate == "sigmoid" else x
    h = torch.empty_like(x)
    now = st["h0"].double()
    zero = torch.zeros_like(now)
    before = torch.empty_like(x) if c["op"] == "rec_train" else None
    for t in range(N):
        if before is not None:
            before[t] = now
        new = torch.addcmul(u[t], a[t], now)
        now = new if inside[t] is None else torch.where(inside[t], new, now)
        h[t] = now if inside[t] is None else torch.where(inside[t], now, zero)
    out = h.permute(1, 2, 0, 3)
    if step:
        return out[:, :, 0], now
    if c["op"] == "rec_fwd":
        return out, now
    dout = st["dout"].permute(2, 0, 1, 3).double().contiguous()
    lam = torch.empty_like(dout)
    back = st["dhN"].double()
    for t in range(N - 1, -1, -1):
        here = dout[t] + back
        lam[t] = here if inside[t] is None else torch.where(inside[t], here, zero)
        back = a[t] * here if inside[t] is None else torch.where(inside[t], a[t] * here, back)
    if gate == "sigmoid":
        dx, dg = lam * torch.sigmoid(-g), lam * (before - x) * a * torch.sigmoid(-g)
    else:
        dx, dg = lam, lam * before * (a if gate == "log" else 1.0)
    return out, now, dx.permute(1, 2, 0, 3), dg.permute(1, 2, 0, 3), back


def _exact_ln(st):
    c = st["case"]
    s = st["x"].double()
    if st["res"] is not None:   # the stream is kept in its type, and what is kept is normalised
        s = (s + st["res"].double()).to(DTYPES[c["dtype"]]).double()
    var, mu = torch.var_mean(s, dim=1, unbiased=False, keepdim=True)
    xh = (s - mu) / (var + EPS).sqrt()
    w, b = st["w"].double(), st["b"].double()
    first = (xh * w + b, s) if st["res"] is not None else (xh * w + b,)
    if c["op"] == "ln_fwd":
        return first
    dy = st["dy"].double()
    v = dy * w
    dx = (v - v.mean(1, True) - xh * (v * xh).mean(1, True)) / (var + EPS).sqrt()
    if st["dsum"] is not None:
        dx = dx + st["dsum"].double()
    return first + (dx, torch.einsum("rc,rc->c", dy, xh), dy.sum(0))


def _exact_clip(st):
    total = 0.0
    for t in st["grads"]:
        total += float(torch.linalg.vector_norm(t.double()) ** 2)
    norm = torch.tensor(math.sqrt(total), dtype=torch.float64)
    if st["case"]["op"] == "norm":
        return norm
    c = min(1.0, st["max_norm"] / (math.sqrt(total) + 1e-6))
    flat = {}
    for name, dt in DTYPES.items():
        parts = [torch.nn.functional.pad(t.double() * c, (0, -t.numel() % 8)) for t in st["grads"] if t.dtype == dt]
        if parts:
            flat[name] = torch.cat(parts)
    return norm, flat


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("rec"):
        return _exact_rec(st)
    if case["op"].startswith("ln"):
        return _exact_ln(st)
    return _exact_clip(st)
