"""Cases that measure the gated linear recurrence, the block norm and the rotary positions.

Each case is one call a user's program makes: a prompt's recurrence, its gradients and
its single-token step; the norms around a block, with its gate and residual, and their
gradients; the rotation of queries and keys by their positions. `run` computes it in
elementary torch operations, or (`own`) with the library's kernels."""
import math

import torch

own = False

EPS = 1e-5
KEEP = 64  # tokens between the states that a forward pass keeps for its gradients


def listed():
    rec = dict(io="bf16", input_gate=True, h0=False, ragged=False, states=False)
    norm = dict(io="bf16", residual="bf16", post=True, gate=True, act="silu", scale=True)
    rot = dict(io="bf16", layout="half", positions="none", back=False)
    return [
        # a batch of prompts through a recurrent layer
        dict(rec, op="rec_fwd", name="recurrence prompt b8 4096", batch=8, seqlen=4096, channels=4096),
        # two long documents continued from a state: few chains, a long axis
        dict(rec, op="rec_fwd", name="recurrence long b2 32768", batch=2, seqlen=32768, channels=2560, h0=True),
        # one short prompt in fp32, where latency counts, of an odd width
        dict(rec, op="rec_fwd", name="recurrence short f32 b1 77", batch=1, seqlen=77, channels=1001, io="f32"),
        # a training step's gradients, with the states that its forward pass kept
        dict(rec, op="rec_bwd", name="recurrence grad b8 2048", batch=8, seqlen=2048, channels=4096, states=True),
        # gradients of a padded fp32 batch with an initial state, nothing kept by the forward pass
        dict(rec, op="rec_bwd", name="recurrence grad ragged f32", batch=3, seqlen=1001, channels=640, io="f32", h0=True,
             ragged=True),
        # one token for a full serving batch
        dict(op="rec_step", name="recurrence step b128", batch=128, channels=4096, io="bf16", input_gate=True),
        # behind one block and before the next, for a batch of prompts: norm, gate, scale, fp32 residual, norm
        dict(norm, op="block_fwd", name="block norm b8 4096", tokens=32768, channels=2048, residual="f32"),
        # its gradients in a training step
        dict(norm, op="block_bwd", name="block norm grad b4 4096", tokens=16384, channels=4096),
        # one token for a serving batch: the residual and the norm before the next block alone
        dict(norm, op="block_fwd", name="block norm decode b64", tokens=64, channels=2048, post=False, gate=False,
             scale=False),
        # queries and keys of a prompt, keys shared by eight heads
        dict(rot, op="rotary", name="rotary prompt b8 4096", batch=8, seqlen=4096, heads=64, kv_heads=8, dim=128, rotary=128),
        # one token each of a serving batch, at far positions
        dict(rot, op="rotary", name="rotary decode b128", batch=128, seqlen=1, heads=32, kv_heads=4, dim=128, rotary=128,
             positions="each"),
        # gradients of a prompt continued from offsets, half of an odd-sized head rotated, interleaved, in fp32
        dict(rot, op="rotary", name="rotary grad f32 partial", batch=2, seqlen=1999, heads=16, kv_heads=4, dim=80, rotary=40,
             layout="interleaved", io="f32", positions="offsets", back=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_fwd", "rec_bwd", "rec_bwd", "rec_step", "block_fwd", "block_bwd", "rotary", "rotary"])
    io = rng.choice(["bf16", "bf16", "f32"])
    width = rng.choice([_log_int(rng, 16, 8192), 8 * _log_int(rng, 2, 1024), 128 * rng.randint(1, 40)])
    if op == "rec_step":
        return dict(op=op, batch=_log_int(rng, 1, 1024), channels=width, io=io, input_gate=rng.random() < 0.7)
    if op.startswith("rec"):
        most = (100_000_000 if op == "rec_fwd" else 40_000_000) // (2 if io == "f32" else 1) // width
        seqlen = min(_log_int(rng, 1, 65536), most)
        return dict(op=op, batch=max(1, min(_log_int(rng, 1, 32), most // seqlen)), seqlen=seqlen, channels=width, io=io,
                    input_gate=rng.random() < 0.7, h0=rng.random() < 0.5, ragged=rng.random() < 0.4,
                    states=rng.random() < 0.5)
    if op.startswith("block"):
        post, gate = rng.random() < 0.6, rng.random() < 0.5
        return dict(op=op, tokens=_log_int(rng, 1, 40_000_000 // width), channels=width, io=io,
                    residual=rng.choice(["f32", io]), post=post, gate=gate, act=rng.choice(["silu", "sigmoid", "none"]),
                    scale=rng.random() < 0.5)
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    heads = kv * rng.choice([1, 1, 2, 3, 4, 8])
    dim = rng.choice([32, 64, 80, 96, 128, 128, 256, 2 * rng.randint(4, 128)])
    most = 200_000_000 // (heads + kv) // dim
    seqlen = min(_log_int(rng, 1, 32768), most)
    return dict(op=op, batch=max(1, min(_log_int(rng, 1, 64), most // seqlen)), seqlen=seqlen, heads=heads, kv_heads=kv, dim=dim,
                rotary=rng.choice([dim, dim, 2 * rng.randint(1, dim // 2)]), io=io,
                layout=rng.choice(["half", "interleaved"]), positions=rng.choice(["none", "each", "offsets"]),
                back=rng.random() < 0.3)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, to=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(to)

    def uniform(n, lo, hi):
        return lo + (hi - lo) * torch.rand(n, generator=gen, device=dev)

    c = dict(case)
    io = torch.bfloat16 if c["io"] == "bf16" else torch.float32
    s = {"case": c, "io": io}
    if c["op"].startswith("rec"):
        b, C = c["batch"], c["channels"]
        shape = (b, C) if c["op"] == "rec_step" else (b, c["seqlen"], C)
        s["x"], s["decay_gate"] = normal(*shape, to=io), normal(*shape, to=io)
        s["input_gate"] = normal(*shape, to=io) if c["input_gate"] else None
        # a state's decay a token, from 0.9 to 0.999 to the power 8 sigmoid(gate)
        s["log_decay"] = 8 * torch.log(uniform(C, 0.9, 0.999))
        if c["op"] == "rec_step":
            s["h"] = normal(b, C)
            return s
        s["h0"] = normal(b, C) if c["h0"] else None
        s["lengths"] = None
        if c["ragged"]:
            s["lengths"] = torch.randint(0, c["seqlen"] + 1, (b,), generator=gen, device=dev, dtype=torch.int32)
            s["lengths"][0] = c["seqlen"]
        s["states"] = None
        if c["op"] == "rec_bwd":
            s["dy"], s["dh_final"] = normal(*shape, to=io), normal(b, C)
            if c["states"]:  # what the forward pass of a training step left
                s["states"] = _kept(*_rec_states(s)[:2], s["h0"])
        return s
    if c["op"].startswith("block"):
        n, C = c["tokens"], c["channels"]
        res = torch.bfloat16 if c["residual"] == "bf16" else torch.float32
        s["x"] = (2 * normal(n, C)).to(io)
        s["z"] = normal(n, C, to=io) if c["gate"] else None
        s["post_weight"] = 1 + 0.2 * normal(C) if c["post"] else None
        s["pre_weight"] = 1 + 0.2 * normal(C)
        s["scale"] = 0.5 + 0.2 * normal(C) if c["scale"] else None
        s["residual_scale"] = 0.75
        # (of the gradients it is the stream behind the block, of the forward pass the one before it)
        s["residual"] = (3 * normal(n, C)).to(res)
        if c["op"] == "block_bwd":
            s["dy"], s["dresidual"] = normal(n, C, to=io), normal(n, C, to=res)
        return s
    b, L, H, G, D = c["batch"], c["seqlen"], c["heads"], c["kv_heads"], c["dim"]
    s["q"], s["k"] = normal(b, L, H, D, to=io), normal(b, L, G, D, to=io)
    half = c["rotary"] // 2
    # a base of 10^4 and positions divided by 4, as for a context longer than the one trained on
    s["freqs"] = (10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half) / 4).float()
    s["scale"] = 0.1 * math.log(4) + 1
    s["positions"] = s["offsets"] = None
    if c["positions"] == "each":
        s["positions"] = torch.randint(0, 1 << 20, (b, L), generator=gen, device=dev, dtype=torch.int32)
    elif c["positions"] == "offsets":
        s["offsets"] = torch.randint(0, 1 << 17, (b,), generator=gen, device=dev, dtype=torch.int32)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rec_fwd": _rec_fwd, "rec_bwd": _rec_bwd, "rec_step": _rec_step, "block_fwd": _block_fwd,
            "block_bwd": _block_bwd, "rotary": _rotary}[op](state)


def _own(s, op):
    from state_space_sequence_amd import m3

    c = s["case"]
    if op == "rotary":
        q, k = m3.rotary(s["q"], s["k"], s["freqs"], positions=s["positions"], offsets=s["offsets"], layout=c["layout"],
                         scale=s["scale"], backward=c["back"])
        return {"q": q, "k": k}
    if op.startswith("block"):
        kw = dict(z=s["z"], activation=c["act"], scale=s["scale"], post_norm=c["post"], post_weight=s["post_weight"],
                  pre_weight=s["pre_weight"], residual_scale=s["residual_scale"], eps=EPS)
        if op == "block_fwd":
            y, r = m3.block_norm_fwd(s["x"], s["residual"], **kw)
            return {"y": y, "residual": r}
        return m3.block_norm_bwd(s["x"], s["residual"], s["dy"], s["dresidual"], **kw)
    if op == "rec_step":
        y = m3.recurrence_step(s["x"], s["decay_gate"], s["log_decay"], s["h"], input_gate=s["input_gate"])
        return {"y": y, "h": s["h"]}
    kw = dict(input_gate=s["input_gate"], h0=s["h0"], lengths=s["lengths"])
    if op == "rec_fwd":
        if c["states"]:
            y, h, states = m3.recurrence_fwd(s["x"], s["decay_gate"], s["log_decay"], want_states=True, **kw)
            return {"y": y, "h": h, "states": states}
        y, h = m3.recurrence_fwd(s["x"], s["decay_gate"], s["log_decay"], **kw)
        return {"y": y, "h": h}
    return m3.recurrence_bwd(s["x"], s["decay_gate"], s["log_decay"], s["dy"], dh_final=s["dh_final"], states=s["states"], **kw)


# ------------------------------------------------------------ plain forms ---
def _chain(a, b):
    """h_t = a_t h_{t-1} + b_t from 0 along dim 1, and the products of a from the start, by doubling."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return a, b


def _rec_gates(s):
    f = lambda t: torch.sigmoid(t.float())  # noqa: E731
    sr = f(s["decay_gate"])
    g = f(s["input_gate"]) if s["input_gate"] is not None else torch.ones_like(sr)
    log_a = s["log_decay"] * sr
    return sr, g, torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))


def _live(s):
    L = s["x"].shape[1]
    at = torch.arange(L, device=s["x"].device)
    if s["lengths"] is None:
        return (at >= 0)[None, :, None]
    return (at[None] < s["lengths"][:, None])[..., None]


def _rec_states(s):
    """The products of the decays and the states from 0 at every token, [b, L, C]."""
    _, g, a, m = _rec_gates(s)
    live = _live(s)
    one, zero = torch.ones((), device=a.device), torch.zeros((), device=a.device)
    return _chain(torch.where(live, a, one), torch.where(live, m * g * s["x"].float(), zero))


def _from(decay, h, h0):
    return h if h0 is None else h + decay * h0[:, None]


def _before(h, h0):
    """The state before each token."""
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None]
    return torch.cat([first, h[:, :-1]], 1)


def _kept(decay, h, h0):
    return _before(_from(decay, h, h0), h0)[:, ::KEEP].contiguous()


def _rec_fwd(s):
    decay, h = _rec_states(s)
    kept = _kept(decay, h, s["h0"]) if s["case"]["states"] else None
    h = _from(decay, h, s["h0"])
    y = torch.where(_live(s), h, torch.zeros((), device=h.device)).to(s["io"])
    return {"y": y, "h": h[:, -1].contiguous()} if kept is None else {"y": y, "h": h[:, -1].contiguous(), "states": kept}


def _rec_bwd(s):
    sr, g, a, m = _rec_gates(s)
    live = _live(s)
    zero, one = torch.zeros((), device=a.device), torch.ones((), device=a.device)
    x, dy = torch.where(live, s["x"].float(), zero), torch.where(live, s["dy"].float(), zero)
    before = _before(_from(*_rec_states(s), s["h0"]), s["h0"])
    al = torch.where(live, a, one)
    # backwards: D_t = dy_t + a_{t+1} D_{t+1}, the last state's gradient behind the last token
    nxt = torch.cat([al[:, 1:], torch.ones_like(al[:, :1])], 1).flip(1)
    decay, D = _chain(nxt, dy.flip(1))
    D = (D + decay * s["dh_final"][:, None]).flip(1)
    dh0 = al[:, 0] * D[:, 0]
    D = torch.where(live, D, zero)
    dlog = D * (a * before - g * x * a * a / m)
    io = s["io"]
    r = {"x": (D * m * g).to(io), "decay_gate": (dlog * s["log_decay"] * sr * (1 - sr)).to(io),
         "log_decay": (dlog.double() * sr).sum((0, 1)).float(), "h0": dh0}
    if s["input_gate"] is not None:
        r["input_gate"] = (D * m * x * g * (1 - g)).to(io)
    return r


def _rec_step(s):
    _, g, a, m = _rec_gates(s)
    s["h"].copy_(a * s["h"] + m * g * s["x"].float())
    return {"y": s["h"].to(s["io"]), "h": s["h"]}


def _gate(s):
    """The gate's value and slope."""
    if s["z"] is None:
        return torch.ones((), device=s["x"].device), None
    z = s["z"].float()
    if s["case"]["act"] == "none":
        return z, torch.ones_like(z)
    g = torch.sigmoid(z)
    return (z * g, g * (1 + z * (1 - g))) if s["case"]["act"] == "silu" else (g, g * (1 - g))


def _rms(t):
    return torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)


def _block_parts(s):
    x = s["x"].float()
    rx = _rms(x) if s["case"]["post"] else torch.ones((), device=x.device)
    w = s["post_weight"] if s["case"]["post"] else torch.ones((), device=x.device)
    sc = s["scale"] if s["scale"] is not None else torch.ones((), device=x.device)
    return x, rx, w, sc


def _block_fwd(s):
    x, rx, w, sc = _block_parts(s)
    r = s["residual_scale"] * s["residual"].float() + sc * _gate(s)[0] * (x * rx * w)
    return {"y": (r * _rms(r) * s["pre_weight"]).to(s["io"]), "residual": r.to(s["residual"].dtype)}


def _rms_back(d, t, r):
    """Gradient of t * r, with r = rsqrt(mean t^2 + eps)."""
    return r * (d - t * r * (d * t * r).mean(-1, keepdim=True))


def _block_bwd(s):
    x, rx, w, sc = _block_parts(s)
    R, dy = s["residual"].float(), s["dy"].float()
    rr = _rms(R)
    dR = s["dresidual"].float() + _rms_back(dy * s["pre_weight"], R, rr)
    act, slope = _gate(s)
    v = x * rx * w
    dv = dR * sc * act
    r = {"residual": (s["residual_scale"] * dR).to(s["residual"].dtype), "pre_weight": (dy * R * rr).double().sum(0).float()}
    if s["scale"] is not None:
        r["scale"] = (dR * act * v).double().sum(0).float()
    if s["z"] is not None:
        r["z"] = (dR * sc * v * slope).to(s["io"])
    if s["case"]["post"]:
        r["post_weight"] = (dv * x * rx).double().sum(0).float()
        dv = _rms_back(dv * w, x, rx)
    r["x"] = dv.to(s["io"])
    return r


def _rotary(s):
    c = s["case"]
    b, L, n = c["batch"], c["seqlen"], c["rotary"]
    dev = s["q"].device
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(L, device=dev)[None] + (s["offsets"][:, None] if s["offsets"] is not None else 0)
    angle = pos.double()[..., None, None] * s["freqs"].double()
    cos, sin = (s["scale"] * torch.cos(angle)).float(), (s["scale"] * torch.sin(angle)).float()
    if c["back"]:
        sin = -sin

    def turn(x):
        t, rest = x[..., :n].float(), x[..., n:]
        if c["layout"] == "half":
            u, v = t[..., :n // 2], t[..., n // 2:]
            t = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
        else:
            u, v = t[..., 0::2], t[..., 1::2]
            t = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
        return torch.cat([t.to(x.dtype), rest], -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


# ----------------------------------------------------------------- counts ---
def work(case):
    c = dict(case)
    e = 2 if c["io"] == "bf16" else 4
    if c["op"] == "rotary":
        n = c["batch"] * c["seqlen"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 2 * n * c["dim"] * e, "flops": 3 * n * c["rotary"]}
    if c["op"].startswith("block"):
        n, r = c["tokens"] * c["channels"], 2 if c["residual"] == "bf16" else 4
        if c["op"] == "block_fwd":
            return {"bytes": n * (e * (3 if c["gate"] else 2) + 2 * r) + 12 * c["channels"], "flops": 16 * n}
        return {"bytes": n * (e * (5 if c["gate"] else 3) + 3 * r) + 24 * c["channels"], "flops": 36 * n}
    ins = 3 if c["input_gate"] else 2
    if c["op"] == "rec_step":
        n = c["batch"] * c["channels"]
        return {"bytes": n * (e * (ins + 1) + 8) + 4 * c["channels"], "flops": 30 * n}
    n, state = c["batch"] * c["seqlen"] * c["channels"], 4 * c["batch"] * c["channels"]
    kept = -(-c["seqlen"] // KEEP) * state if c["states"] else 0
    if c["op"] == "rec_fwd":
        return {"bytes": n * e * (ins + 1) + state * (2 if c["h0"] else 1) + kept, "flops": 30 * n}
    return {"bytes": n * e * (2 * ins + 1) + state * (3 if c["h0"] and not c["states"] else 2) + kept, "flops": 60 * n}


# ------------------------------------------------------------ 64-bit value ---
def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, its adjoint, the norms row sums, the angles."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rotary":
        return _exact_rotary(s, c)
    if c["op"].startswith("block"):
        return _exact_block(s, c)
    one = lambda t: 1 / (1 + torch.exp(-t.double()))  # noqa: E731
    ld = s["log_decay"].double()

    def token(t):
        """decay, input factor, both gates of token t (None: the only one)."""
        at = lambda n: s[n] if t is None else s[n][:, t]  # noqa: E731
        sr = one(at("decay_gate"))
        a = torch.exp(ld * sr)
        return a, torch.sqrt(1 - a * a), sr, one(at("input_gate")) if c["input_gate"] else torch.ones_like(a)

    if c["op"] == "rec_step":
        a, m, _, g = token(None)
        h = a * s["h"].double() + m * g * s["x"].double()
        return {"y": h, "h": h}
    b, L, C = s["x"].shape
    dev = s["x"].device
    new = lambda *n: torch.zeros(*n, device=dev, dtype=torch.float64)  # noqa: E731
    h = s["h0"].double() if c["h0"] else new(b, C)
    before, y = new(b, L, C), new(b, L, C)
    live = None if s["lengths"] is None else (torch.arange(L, device=dev)[:, None] < s["lengths"][None])[..., None]
    for t in range(L):
        a, m, _, g = token(t)
        before[:, t] = h
        n = a * h + m * g * s["x"][:, t].double()
        h = n if live is None else torch.where(live[t], n, h)
        y[:, t] = h if live is None else h * live[t]
    if c["op"] == "rec_fwd":
        r = {"y": y, "h": h}
        if c["states"]:
            r["states"] = before[:, ::KEEP].contiguous()
        return r
    r = {"x": new(b, L, C), "decay_gate": new(b, L, C), "log_decay": new(C)}
    if c["input_gate"]:
        r["input_gate"] = new(b, L, C)
    D = s["dh_final"].double()
    for t in reversed(range(L)):
        a, m, sr, g = token(t)
        x = s["x"][:, t].double()
        on = 1.0 if live is None else live[t].double()
        E = D + s["dy"][:, t].double()
        da = E * (before[:, t] - g * x * a / m) * on
        r["x"][:, t] = E * m * g * on
        if c["input_gate"]:
            r["input_gate"][:, t] = E * m * x * g * (1 - g) * on
        r["decay_gate"][:, t] = da * a * ld * sr * (1 - sr)
        r["log_decay"] += (da * a * sr).sum(0)
        D = a * E if live is None else torch.where(live[t], a * E, D)
    r["h0"] = D
    return r


def _exact_block(s, c):
    one = torch.ones((), device=s["x"].device, dtype=torch.float64)
    get = lambda n: one if s[n] is None else s[n].double()  # noqa: E731
    x, z, w, wp, sc = (get(n) for n in ("x", "z", "post_weight", "pre_weight", "scale"))
    C = x.shape[1]
    e = torch.exp(-z)
    act, slope = one, one
    if c["gate"]:
        act, slope = {"none": (z, torch.ones_like(z)), "sigmoid": (1 / (1 + e), e / (1 + e) ** 2),
                      "silu": (z / (1 + e), 1 / (1 + e) + z * e / (1 + e) ** 2)}[c["act"]]
    sd = (x.square().sum(1, keepdim=True) / C + EPS).sqrt() if c["post"] else one
    u = x / sd
    R = s["residual"].double()
    if c["op"] == "block_fwd":
        R = s["residual_scale"] * R + sc * act * u * w
        return {"y": R / (R.square().sum(1, keepdim=True) / C + EPS).sqrt() * wp, "residual": R}
    SD = (R.square().sum(1, keepdim=True) / C + EPS).sqrt()
    U, dy = R / SD, s["dy"].double()
    q = dy * wp
    dR = s["dresidual"].double() + (q - U * ((q * U).sum(1, keepdim=True) / C)) / SD
    r = {"residual": s["residual_scale"] * dR, "pre_weight": (dy * U).sum(0)}
    if c["scale"]:
        r["scale"] = (dR * act * u * w).sum(0)
    if c["gate"]:
        r["z"] = dR * sc * u * w * slope
    p = dR * sc * act
    if c["post"]:
        r["post_weight"] = (p * u).sum(0)
        p = p * w
        p = (p - u * ((p * u).sum(1, keepdim=True) / C)) / sd
    r["x"] = p
    return r


def _exact_rotary(s, c):
    n, f = c["rotary"], s["freqs"].double()
    r = {}
    for name in "qk":
        x = s[name].double()
        L = x.shape[1]
        p = torch.arange(L, device=x.device, dtype=torch.float64).expand(x.shape[0], L)
        if s["positions"] is not None:
            p = s["positions"].double()
        if s["offsets"] is not None:
            p = p + s["offsets"].double().unsqueeze(1)
        turn = torch.polar(torch.full_like(f, s["scale"]).expand(p.shape + f.shape), (-p if c["back"] else p).unsqueeze(-1) * f)
        i = torch.arange(n // 2, device=x.device)
        u, v = (i, i + n // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        w = torch.complex(x[..., u], x[..., v]) * turn[:, :, None]
        x[..., u], x[..., v] = w.real, w.imag
        r[name] = x
    return r
