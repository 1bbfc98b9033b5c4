"""Cases of linear attention with a decay for each head (prompts, training,
single tokens) and of the norm and rotation of queries and keys in front of it
(forward, backward).

``run`` computes a case in plain torch operations (``own`` false) or through
the library's entry points (``own`` true); ``exact`` computes it in 64 bits
from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decoded token for a batch of 64 sequences, fewer key heads than query heads: latency
        dict(name="rot_step_b64", op="rot_fwd", B=64, N=1, Hq=16, Hk=4, D=64, P=32, axes=1, norm=True, pairs="half",
             dtype="bf16", strided=True),
        # a prompt of images and text: positions in time, height and width, queries and keys in one projection
        dict(name="rot_fwd_axes_n16384", op="rot_fwd", B=2, N=16384, Hq=16, Hk=16, D=128, P=64, axes=3, norm=True,
             pairs="half", dtype="bf16", strided=True),
        # a training batch
        dict(name="rot_train_b8n4096", op="rot_train", B=8, N=4096, Hq=16, Hk=16, D=64, P=32, axes=1, norm=True,
             pairs="half", dtype="bf16", strided=False),
        # odd sizes, a part of each head rotated, neighbouring channels paired
        dict(name="rot_train_odd_f32", op="rot_train", B=3, N=1001, Hq=6, Hk=3, D=80, P=20, axes=2, norm=True,
             pairs="adjacent", dtype="f32", strided=True),
        # one decoded token for the batch of the decode benchmark: the state is read and written
        dict(name="dec_step_b256h16", op="dec_step", B=256, H=16, N=1, D=64, M=64, dtype="bf16", ragged=False,
             strided=False),
        # a few sequences: latency
        dict(name="dec_step_b4h8", op="dec_step", B=4, H=8, N=1, D=128, M=128, dtype="bf16", ragged=False, strided=True),
        # a batch of prompts, the state kept for decoding
        dict(name="dec_fwd_b16h8n4096", op="dec_fwd", B=16, H=8, N=4096, D=64, M=64, dtype="bf16", ragged=False,
             strided=False),
        # one long document, few heads: the time axis has to be split
        dict(name="dec_fwd_n65536_d128", op="dec_fwd", B=1, H=16, N=65536, D=128, M=128, dtype="bf16", ragged=False,
             strided=False),
        # prompts of different lengths (one empty), token-major in one projection, 32 bits
        dict(name="dec_fwd_ragged_f32", op="dec_fwd", B=7, H=5, N=1537, D=64, M=64, dtype="f32", ragged=True,
             strided=True),
        # a training batch
        dict(name="dec_train_b16h8n2048", op="dec_train", B=16, H=8, N=2048, D=64, M=64, dtype="bf16", ragged=False,
             strided=False),
        # training on long sequences, state and its gradient carried between segments
        dict(name="dec_train_n16384_d128", op="dec_train", B=2, H=8, N=16384, D=128, M=128, dtype="bf16", ragged=False,
             strided=True),
        # odd sizes, 32 bits
        dict(name="dec_train_odd_f32", op="dec_train", B=3, H=5, N=1001, D=40, M=72, dtype="f32", ragged=True,
             strided=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rot_fwd", "rot_train", "dec_step", "dec_fwd", "dec_fwd", "dec_train", "dec_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("rot"):
        D = rng.choice([32, 64, 80, 96, 128]) if rng.random() < 0.7 else 2 * rng.randint(4, 64)
        P = D // 2 if rng.random() < 0.6 else rng.randint(1, D // 2)
        Hq, Hk = rng.randint(1, 24), rng.randint(1, 24)
        most = (2 * 16384 * 32 * 128) // ((2 if op == "rot_fwd" else 5) * (Hq + Hk) * D)
        N = min(_log_int(rng, 1, 32768), most)
        B = min(_log_int(rng, 1, 128), max(1, most // N))
        return dict(op=op, B=B, N=N, Hq=Hq, Hk=Hk, D=D, P=P, axes=min(P, rng.choice([1, 1, 2, 3])),
                    norm=rng.random() < 0.7, pairs=rng.choice(["half", "adjacent"]), dtype=dtype,
                    strided=rng.random() < 0.5)
    D, M = ((rng.choice([16, 32, 64, 64, 128]), rng.choice([16, 32, 64, 64, 128])) if rng.random() < 0.75
            else (rng.randint(3, 128), rng.randint(3, 128)))
    H = rng.randint(1, 16)
    if op == "dec_step":
        B = min(_log_int(rng, 1, 512), max(1, (256 * 16 * 64 * 64) // (H * D * M)))
        return dict(op=op, B=B, H=H, N=1, D=D, M=M, dtype=dtype, ragged=False, strided=rng.random() < 0.5)
    most = (16 * 65536 * 256) // ((2 if op == "dec_fwd" else 5) * H * (D + M) * (1 if dtype == "bf16" else 4))
    N = min(_log_int(rng, 1, 65536), most)
    B = min(_log_int(rng, 1, 32), max(1, most // N))
    return dict(op=op, B=B, H=H, N=N, D=D, M=M, dtype=dtype, ragged=rng.random() < 0.3, strided=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _lens(case):
    """Lengths of a ragged batch: spread from an empty sequence to a full one."""
    B, N = case["B"], case["N"]
    return [N] if B == 1 else [N * i // (B - 1) for i in range(B)]


def _axes(case):
    """The axis of each rotated pair: runs of nearly equal length."""
    return [i * case["axes"] // case["P"] for i in range(case["P"])]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def views(dt, *parts):
        """Tensors [B, H, N, D]: side by side in one token-major projection, or each by itself."""
        if not case["strided"]:
            return [p.to(dt) for p in parts]
        flat = [p.to(dt).transpose(1, 2).flatten(2) for p in parts]   # [B, N, H D]
        both = torch.cat(flat, dim=-1)
        out, at = [], 0
        for p in parts:
            B, H, N, D = p.shape
            out.append(both[..., at:at + H * D].unflatten(-1, (H, D)).transpose(1, 2))
            at += H * D
        return out

    st = dict(case=dict(case))
    dt = DTYPES[case["dtype"]]
    B, N, D = case["B"], case["N"], case["D"]
    if case["op"].startswith("rot"):
        st["q"], st["k"] = views(dt, normal(B, case["Hq"], N, D), 2.0 * normal(B, case["Hk"], N, D))
        # time goes on from a cache (far into it); the other axes are rows and columns of images
        first = torch.randint(0, 1 << 17, (1, B, 1), generator=g, device=DEV)
        pos = [first + torch.arange(N, device=DEV)]
        pos += [torch.randint(0, 512, (1, B, N), generator=g, device=DEV) for _ in range(1, case["axes"])]
        st["pos"] = torch.cat(pos).to(torch.int32)
        st["freq"] = 10000.0 ** (-torch.arange(case["P"], device=DEV, dtype=torch.float64) / case["P"])
        st["freq"] = st["freq"].float()
        st["axes"] = tuple(_axes(case))
        st["wq"], st["wk"] = (1.0 + 0.2 * normal(D), 1.0 + 0.2 * normal(D)) if case["norm"] else (None, None)
        if case["op"] == "rot_train":
            st["dqo"], st["dko"] = normal(B, case["Hq"], N, D).to(dt), normal(B, case["Hk"], N, D).to(dt)
        return st
    H, M = case["H"], case["M"]
    st["q"], st["k"], st["v"] = views(dt, normal(B, H, N, D), normal(B, H, N, D), normal(B, H, N, M))
    # memories of two tokens to some thousand, by head, as fixed decays of such models are; the last head forgets nothing
    span = torch.linspace(1.0, 12.0, H, device=DEV, dtype=torch.float64)
    st["log_decay"] = torch.log1p(-torch.exp2(-span))
    if H > 2:
        st["log_decay"][-1] = 0.0
    st["log_decay"] = st["log_decay"].float()
    st["scale"] = D ** -0.5
    st["S0"] = normal(B, H, D, M)
    if case["op"] == "dec_step":
        st["q"], st["k"], st["v"] = (st[n][:, :, 0] for n in "qkv")
        return st
    st["SN"] = torch.zeros_like(st["S0"])
    st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
    if case["op"] == "dec_train":
        st["dout"] = normal(B, H, N, M).to(dt)
        st["dSN"] = normal(B, H, D, M)
    return st


# ---------------------------------------------------------------- the plain forms

def _pair(x, pairs, P):
    """First and second value of the rotated pairs, and the channels behind them."""
    r = x[..., :2 * P]
    a, b = (r[..., :P], r[..., P:]) if pairs == "half" else (r[..., 0::2], r[..., 1::2])
    return a, b, x[..., 2 * P:]


def _unpair(a, b, rest, pairs):
    r = torch.cat([a, b], dim=-1) if pairs == "half" else torch.stack([a, b], dim=-1).flatten(-2)
    return torch.cat([r, rest], dim=-1)


def _turn(x, cos, sin, pairs):
    a, b, rest = _pair(x, pairs, cos.shape[-1])
    return _unpair(a * cos - b * sin, b * cos + a * sin, rest, pairs)


def _plain_rot(st):
    c = st["case"]
    dt, pairs = DTYPES[c["dtype"]], c["pairs"]
    axes = torch.tensor(st["axes"], device=DEV)
    # far positions: the angle in 64 bits
    angle = st["pos"][axes].double().movedim(0, -1) * st["freq"].double()   # [B, N, P]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w, dy):
        x = x.float()
        n, r = x, None
        if c["norm"]:
            r = 1.0 / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
            n = x * r * w
        y = _turn(n, cos, sin, pairs).to(dt)
        if dy is None:
            return (y,)
        dn = _turn(dy.float(), cos, -sin, pairs)
        if not c["norm"]:
            return y, dn.to(dt)
        xh = x * r
        wdn = dn * w
        dx = r * (wdn - xh * (wdn * xh).mean(dim=-1, keepdim=True))
        return y, dx.to(dt), (dn * xh).sum(dim=(0, 1, 2))

    return one(st["q"], st["wq"], st.get("dqo")), one(st["k"], st["wk"], st.get("dko"))


CHUNK = 64


def _sweep(x, y, z, g, count, S0, lead):
    """out_i = sum over j <= i of a^(c_i - c_j) (x_i . y_j) z_j + a^(c_i - 1 + lead) x_i S0 along dim 2, and the
    state after it, by chunks; a = e^g, c_i the number of tokens up to i that count."""
    B, H, N, D = x.shape
    C = min(CHUNK, N)
    pad = -N % C
    n = (N + pad) // C
    x, y, z = (torch.nn.functional.pad(t, (0, 0, 0, pad)).unflatten(2, (n, C)) for t in (x, y, z))
    count = torch.cat([count, count[:, -1:].expand(-1, pad)], dim=1).unflatten(1, (n, C)).double()[:, None]
    g = g.double()[:, None]                                       # [H, 1]
    ends = count[..., -1]                                         # [b, 1, n]
    base = torch.cat([torch.zeros_like(ends[..., :1]), ends], dim=-1)
    first = base[..., :-1, None]
    gap = count[..., :, None] - count[..., None, :]               # [b, 1, n, C, C]
    W = torch.exp(g[..., None, None] * gap).float().tril()
    out = ((x @ y.transpose(-1, -2)) * W) @ z
    into = torch.exp(g[..., None] * (ends[..., None] - count + 1 - lead)).float()
    dS = (y * into[..., None]).transpose(-1, -2) @ z              # [B, H, n, D, M]
    # T[c, c'] = a^(tokens between the end of chunk c' and the start of chunk c)
    between = (base[..., :, None] - ends[..., None, :]).clamp(min=0)
    T = torch.exp(g[..., None] * between).float().tril(-1)
    S = (T @ dS.flatten(3)).unflatten(3, (D, -1)) + torch.exp(g * base).float()[..., None, None] * S0[:, :, None]
    seen = torch.exp(g[..., None] * (count - first - 1 + lead)).float()
    out = out + seen[..., None] * (x @ S[:, :, :-1])
    return out.flatten(2, 3)[:, :, :N], S[:, :, -1]


def _plain_dec(st):
    c = st["case"]
    dt, g, scale = DTYPES[c["dtype"]], st["log_decay"], st["scale"]
    if c["op"] == "dec_step":
        q, k, v = (st[n].float() for n in "qkv")
        a = torch.exp(g.double()).float()
        S = a[:, None, None] * st["S0"] + k[..., :, None] * v[..., None, :]
        st["S0"].copy_(S)
        return (scale * (q[..., None, :] @ S)[..., 0, :]).to(dt), st["S0"]
    N = c["N"]
    at = torch.arange(N, device=DEV)
    keep, count = None, at[None] + 1
    back = count
    if st["lens"] is not None:
        keep = (at < st["lens"][:, None])[:, None, :, None]
        count = torch.minimum(at + 1, st["lens"][:, None])
        back = torch.clamp(at + 1 - (N - st["lens"][:, None]), min=0)

    def rows(name):
        t = st[name].float()
        return t if keep is None else torch.where(keep, t, 0.0)

    def done(t):
        return (t if keep is None else torch.where(keep, t, 0.0)).to(dt)

    q, k, v = rows("q"), rows("k"), rows("v")
    out, SN = _sweep(q, k, v, g, count, st["S0"], 1)
    st["SN"].copy_(SN)
    out = done(scale * out)
    if c["op"] == "dec_fwd":
        return out, st["SN"]
    dout = scale * rows("dout")
    dq, _ = _sweep(dout, v, k, g, count, st["S0"].transpose(-1, -2), 1)
    qr, kr, vr, dr = (t.flip(2) for t in (q, k, v, dout))
    dv, dS0 = _sweep(kr, qr, dr, g, back, st["dSN"], 0)
    dk, _ = _sweep(vr, dr, qr, g, back, st["dSN"].transpose(-1, -2), 0)
    return out, st["SN"], done(dq), done(dk.flip(2)), done(dv.flip(2)), dS0


# ---------------------------------------------------------------- through the library

def _own_rot(st):
    from weight_recurrence_gb300 import la
    c = st["case"]
    how = dict(wq=st["wq"], wk=st["wk"], eps=EPS, norm=c["norm"], pairs=c["pairs"], axes=st["axes"])
    q, k = la.la_qk_rotate_forward(st["q"], st["k"], st["pos"], st["freq"], **how)
    if c["op"] == "rot_fwd":
        return (q,), (k,)
    dq, dk, dwq, dwk = la.la_qk_rotate_backward(st["dqo"], st["dko"], st["q"], st["k"], st["pos"], st["freq"], **how)
    return ((q, dq, dwq), (k, dk, dwk)) if c["norm"] else ((q, dq), (k, dk))


def _own_dec(st):
    from weight_recurrence_gb300 import la
    c = st["case"]
    if c["op"] == "dec_step":
        return la.la_decay_step(st["q"], st["k"], st["v"], st["S0"], st["log_decay"], st["scale"]), st["S0"]
    out = la.la_decay_forward(st["q"], st["k"], st["v"], st["log_decay"], st["scale"], S0=st["S0"], SN=st["SN"],
                              lens=st["lens"])
    if c["op"] == "dec_fwd":
        return out, st["SN"]
    dS0 = torch.empty_like(st["S0"])
    dq, dk, dv = la.la_decay_backward(st["q"], st["k"], st["v"], st["dout"], st["log_decay"], st["scale"], S0=st["S0"],
                                      dSN=st["dSN"], dS0=dS0, lens=st["lens"])
    return out, st["SN"], dq, dk, dv, dS0


def run(state):
    if state["case"]["op"].startswith("rot"):
        return _own_rot(state) if own else _plain_rot(state)
    return _own_dec(state) if own else _plain_dec(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    B, N, D = case["B"], case["N"], case["D"]
    if case["op"].startswith("rot"):
        n = B * N * (case["Hq"] + case["Hk"]) * D
        small = 4 * (case["axes"] * B * N + case["P"])
        if case["op"] == "rot_train":   # q, k, their outputs' gradients in; outputs and gradients out
            return dict(bytes=4 * n * size + small, flops=20 * n)
        return dict(bytes=2 * n * size + small, flops=7 * n)
    H, M = case["H"], case["M"]
    rows = (sum(_lens(case)) if case["ragged"] else B * N) * H
    full, state = B * N * H, B * H * D * M
    if case["op"] == "dec_train":       # q, k, v, dout in; out, dq, dk, dv out (0 past a sequence's end), four states
        return dict(bytes=(rows + full) * 2 * (D + M) * size + 16 * state, flops=16 * rows * D * M)
    return dict(bytes=(rows * (2 * D + M) + full * M) * size + 8 * state, flops=4 * rows * D * M)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rot(st):
    c = st["case"]
    D, P, pairs = c["D"], c["P"], c["pairs"]
    angle = torch.stack([st["pos"][a].double() * f for a, f in zip(st["axes"], st["freq"].double())], dim=-1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]     # [B, 1, N, P]
    one = torch.arange(P, device=DEV) * (2 if pairs == "adjacent" else 1)
    two = one + (1 if pairs == "adjacent" else P)

    def rotate(x, by):
        z = torch.complex(x[..., one], x[..., two]) * by
        y = x.clone()
        y[..., one], y[..., two] = z.real, z.imag
        return y

    def side(x, w, dy):
        x = x.double()
        s = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        r = torch.rsqrt(s * s / D + EPS) if c["norm"] else 1.0
        w = w.double() if c["norm"] else 1.0
        y = rotate(x * r * w, turn)
        if dy is None:
            return (y,)
        u = rotate(dy.double(), turn.conj())
        if not c["norm"]:
            return y, u
        dot = torch.einsum("bhnd,bhnd->bhn", u * w, x)[..., None]
        return y, r * u * w - x * dot * r ** 3 / D, torch.einsum("bhnd,bhnd->d", u, x * r)

    return side(st["q"], st["wq"], st.get("dqo")), side(st["k"], st["wk"], st.get("dko"))


def _exact_dec(st):
    c = st["case"]
    N, scale = c["N"], st["scale"]
    a = st["log_decay"].double().exp()[:, None, None]
    step = c["op"] == "dec_step"

    def major(name):   # token-major, so that one token of all heads is one slice
        t = st[name].unsqueeze(2) if step else st[name]
        return t.permute(2, 0, 1, 3).double().contiguous()

    q, k, v = major("q"), major("k"), major("v")
    lens = None if step or st["lens"] is None else st["lens"]
    shortest = N if lens is None else int(lens.min())
    inside = [None if t < shortest else (t < lens)[:, None, None, None] for t in range(N)]
    train = c["op"] == "dec_train"
    S = st["S0"].double()
    out = torch.empty_like(v)
    dq = torch.empty_like(q) if train else None
    do = major("dout") if train else None
    for t in range(N):
        new = torch.addcmul(a * S, k[t][..., None], v[t][..., None, :])
        S = new if inside[t] is None else torch.where(inside[t], new, S)
        out[t] = (q[t][..., None] * S).sum(-2)
        if train:
            dq[t] = (S * do[t][..., None, :]).sum(-1)
    gone = None if lens is None else (torch.arange(N, device=DEV)[:, None] >= lens)[:, :, None, None]

    def back(t, by=scale):
        t = by * t
        t = t if gone is None else torch.where(gone, 0.0, t)
        return t.permute(1, 2, 0, 3)

    if step:
        return back(out)[:, :, 0], S
    if not train:
        return back(out), S
    G = st["dSN"].double()
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    for t in range(N - 1, -1, -1):
        here = torch.addcmul(G, scale * q[t][..., None], do[t][..., None, :])
        dk[t] = (here * v[t][..., None, :]).sum(-1)
        dv[t] = (here * k[t][..., None]).sum(-2)
        G = a * here if inside[t] is None else torch.where(inside[t], a * here, G)
    return back(out), S, back(dq), back(dk, 1.0), back(dv, 1.0), G


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("rot"):
        return _exact_rot(st)
    return _exact_dec(st)
