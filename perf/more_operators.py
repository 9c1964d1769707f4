"""Cases of the gated linear recurrence (prompts, single tokens, training steps), of rotary positions for
queries and keys, and of the norms around a block with its gate and residual, each in a plain form of
elementary torch operations and as calls of the library's entry points.

Gated recurrence, per sequence and channel, with a gate r_t, an input gate i_t (or none) and a decay d:
    a_t = exp(-power softplus(d) sigmoid(r_t)),  w_t = sqrt(1 - a_t^2)       or with `lerp`
    a_t = sigmoid(r_t + d),                      w_t = 1 - a_t
    h_t = a_t h_{t-1} + w_t sigmoid(i_t) x_t     (h_{-1} = the initial state, fp32)
Packed sequences lie one behind the other in the rows of one tensor, sequence n in rows
[cu_seqlens[n], cu_seqlens[n + 1]); rows behind the last are no tokens.

Rotary positions: pair j of the first `rot` dimensions of a head, (j, j + rot / 2) or with `inter`
(2 j, 2 j + 1), is turned by the angle position * freq[j], all times a scale; the rest is copied. The
gradient is the turn back (`inverse`).

Block norm, per row of C channels, with the block's output y, the residual stream x, a gate z:
    h = x + alpha post(y) act(z),   out = pre(h)
post and pre: nothing, or a norm (layer: mean taken off; rms: not) times weight plus bias.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases

def listed():
    bf, f32 = "bfloat16", "float32"
    return [
        # the smallest prompt: 64 tokens of one head's 64 channels, fp32 (latency)
        dict(name="gs_b1_L64_C64_fp32", op="gs", b=1, L=64, C=64, dtype=f32, gate=True, decay=True, lerp=False,
             init=False, lens="", train=False),
        # a long context in one sequence, at the package's width of 64 heads of 64 channels
        dict(name="gs_b1_L65536_C4096", op="gs", b=1, L=65536, C=4096, dtype=bf, gate=True, decay=True, lerp=False,
             init=True, lens="", train=False),
        # a training step at the package's prefill sizes: forward and gradients
        dict(name="gst_b4_L2048_C4096", op="gs", b=4, L=2048, C=4096, dtype=bf, gate=True, decay=True, lerp=False,
             init=False, lens="", train=True),
        # a training step over documents of unequal lengths in one row of tokens, odd width, fp32, the
        # convex form without an input gate, states carried over, five spare rows
        dict(name="gst_packed_C1915_fp32", op="gs", b=1, L=4229, C=1915, dtype=f32, gate=False, decay=False, lerp=True,
             init=True, lens="1,777,0,2048,129,64,1000,205", train=True),
        # one token of 128 sequences, the states in a pool of slots
        dict(name="step_b128_C4096", op="step", b=128, C=4096, dtype=bf, gate=True, decay=True, lerp=False, slots=160),
        # queries and keys of a prefill for linear attention
        dict(name="rot_b4_L2048_H64", op="rot", b=4, L=2048, hq=64, hk=64, D=128, rot=128, dtype=bf, inter=False,
             inverse=False, scaling="", pos="", lens=""),
        # gradients of packed sequences' queries and shared keys, interleaved pairs in a quarter of the head, fp32
        dict(name="rot_packed_back_fp32", op="rot", b=1, L=4229, hq=16, hk=4, D=128, rot=32, dtype=f32, inter=True,
             inverse=True, scaling="", pos="", lens="1,777,0,2048,129,64,1000,205"),
        # one token of 128 sequences at positions of their own, far beyond the trained length
        dict(name="rot_step_b128_H64", op="rot", b=128, L=0, hq=64, hk=1, D=128, rot=64, dtype=bf, inter=False,
             inverse=False, scaling="yarn", pos="any", lens=""),
        # between two blocks of a prefill: norm of the block's output, gate, residual, norm before the next block
        dict(name="bn_T8192_C4096", op="bn", T=8192, C=4096, dtype=bf, res=bf, post="rms", pre="rms", gate="silu",
             affine=True),
        # the same for one decode step's 128 rows, the residual stream in fp32
        dict(name="bn_T128_C4096", op="bn", T=128, C=4096, dtype=bf, res=f32, post="rms", pre="rms", gate="silu",
             affine=True),
        # its gradients in training
        dict(name="bnb_T8192_C4096", op="bnb", T=8192, C=4096, dtype=bf, res=bf, post="rms", pre="rms", gate="silu",
             affine=True),
        # gradients at an odd row count and width, fp32, layer norms
        dict(name="bnb_T777_C1920_fp32", op="bnb", T=777, C=1920, dtype=f32, res=f32, post="layer", pre="layer",
             gate="sigmoid", affine=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _cut(rng, rows):
    n = min(rows, rng.randint(1, 12))
    cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
    return ",".join(str(y - x) for x, y in zip([0] + cuts, cuts + [rows]))


def draw(rng):
    op = rng.choice(("gs", "gs", "gs", "step", "rot", "rot", "bn", "bnb"))
    dtype = rng.choice(("bfloat16", "bfloat16", "bfloat16", "float32"))
    if op in ("bn", "bnb"):
        C = rng.choice((64, 128, 256, 512, 768, 1024, 1536, 1920, 2048, 2560, 4096, 5120, 8192, 37, 1001, 2050))
        return dict(op=op, T=_log_uniform(rng, 1, min(16384, (1 << 25) // C)), C=C, dtype=dtype,
                    res=rng.choice((dtype, "float32")), post=rng.choice(("", "rms", "rms", "layer")),
                    pre=rng.choice(("", "rms", "rms", "layer")), gate=rng.choice(("", "id", "sigmoid", "silu")),
                    affine=rng.random() < 0.75)
    if op == "rot":
        D = rng.choice((32, 64, 64, 80, 96, 128, 128, 160, 192, 256))
        rot = rng.choice((D, D, D // 2, D // 4, 10))
        hq = rng.choice((1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64))
        c = dict(op=op, hq=hq, hk=rng.choice([0] + [d for d in range(1, hq + 1) if hq % d == 0]), D=D, rot=rot,
                 dtype=dtype, inter=rng.random() < 0.4, inverse=rng.random() < 0.4,
                 scaling=rng.choice(("", "", "linear", "ntk", "yarn", "bands")))
        if rng.random() < 0.25:
            return dict(c, b=_log_uniform(rng, 1, 256), L=0, pos="any", lens="")
        rows = _log_uniform(rng, 1, min(65536, (1 << 25) // (hq * D)))
        if rng.random() < 0.3 and rows > 1:
            return dict(c, b=1, L=rows + rng.choice((0, 0, 3, 40)), pos="", lens=_cut(rng, rows))
        b = rng.randint(1, 4)
        return dict(c, b=b, L=max(1, rows // b), pos=rng.choice(("", "any")), lens="")
    C = (rng.choice((64, 128, 256, 512, 1024, 1536, 1920, 2048, 2560, 4096, 8192)) if rng.random() < 0.7
         else rng.randint(1, 4096))
    c = dict(op=op, C=C, dtype=dtype, gate=rng.random() < 0.75, lerp=rng.random() < 0.4)
    c["decay"] = rng.random() < 0.75 or not c["lerp"]
    if op == "step":
        b = _log_uniform(rng, 1, 256)
        return dict(c, b=b, slots=b + rng.randint(1, 40) if rng.random() < 0.5 else 0)
    c["train"] = rng.random() < 0.5
    rows = _log_uniform(rng, 1, min(65536, (1 << (24 if c["train"] else 26)) // C))
    c["init"] = rng.random() < 0.5
    if rng.random() < 0.4 and rows > 1:
        return dict(c, b=1, L=rows + rng.choice((0, 0, 3, 40)), lens=_cut(rng, rows))
    b = rng.randint(1, 4)
    return dict(c, b=b, L=max(1, rows // b), lens="")


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case.get("lens") else None


def _offsets(lens, dev):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


POWER = 8.0
TRAINED, FACTOR = 8192, 16.0        # tokens of the training contexts that the positions are scaled from, and how far


def _frequencies(case):
    """Radians per position of each pair, and the scale, in 64 bits: the published ways of reaching beyond
    the trained length (linear interpolation, a larger base, a ramp over the number of turns, bands of
    wavelengths)."""
    n, base, kind = case["rot"], 10000.0, case["scaling"]
    j = torch.arange(n // 2, dtype=torch.float64)
    if kind == "ntk":
        base = base * FACTOR ** (n / (n - 2)) if n > 2 else base
    f = base ** (-2 * j / n)
    if kind == "linear":
        f = f / FACTOR
    if kind == "yarn":      # pairs of over 32 turns in the trained length stay, those under one are interpolated
        at = [n * math.log(TRAINED / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / FACTOR * ramp + f * (1 - ramp), 0.1 * math.log(FACTOR) + 1.0
    if kind == "bands":     # four turns and more in the trained length stay, one and less are interpolated
        turns = TRAINED * f / (2 * math.pi)
        s = ((turns - 1.0) / 3.0).clamp(0, 1)
        f = f / FACTOR * (1 - s) + f * s
    return f, 1.0


def prepare(case, seed):
    dev, dt = torch.device("cuda"), getattr(torch, case["dtype"])
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = dict(case=case)
    if case["op"] in ("bn", "bnb"):
        T, C, rt = case["T"], case["C"], getattr(torch, case["res"])
        s.update(y=rn(T, C, dtype=dt), x=rn(T, C, dtype=rt), z=rn(T, C, dtype=dt) if case["gate"] else None,
                 alpha=0.5, eps=1e-5)
        for n in ("post", "pre"):
            on = case["affine"] and case[n]
            s.update({n + "_w": 1 + 0.1 * rn(C) if on else None,
                      n + "_b": 0.1 * rn(C) if on and case[n] == "layer" else None})
        if case["op"] == "bnb":
            s.update(dh=rn(T, C, dtype=rt), dout=rn(T, C, dtype=dt) if case["pre"] else None)
        return s
    if case["op"] == "rot":
        b, L, lens = case["b"], case["L"], _lens(case)
        f, scale = _frequencies(case)
        lead = (b, L) if L else (b,)
        s.update(q=rn(*lead, case["hq"], case["D"], dtype=dt), scale=scale, freq=f.to(dev), lens=lens,
                 k=rn(*lead, case["hk"], case["D"], dtype=dt) if case["hk"] else None,
                 pos=torch.randint(0, int(TRAINED * FACTOR), lead, generator=g, device=dev) if case["pos"] else None,
                 cu=_offsets(lens, dev) if lens is not None else None, offset=7)
        for n in "qk":
            s[n + "_out"] = torch.zeros_like(s[n]) if s[n] is not None else None
        return s
    b, C = case["b"], case["C"]
    # decays between 0.9 and 0.999 a token where the gate is open (the convex form: gates around one half)
    u = 0.9 + 0.099 * torch.rand(C, generator=g, device=dev)
    s["decay"] = None
    if case["decay"]:
        s["decay"] = torch.logit(u) if case["lerp"] else torch.log(torch.expm1(-torch.log(u) / POWER))
    if case["op"] == "step":
        n = case["slots"] or b
        s.update(x=rn(b, C, dtype=dt), r=rn(b, C, dtype=dt), i=rn(b, C, dtype=dt) if case["gate"] else None,
                 state=rn(n, C))
        s["out"] = s["state"].clone()      # the buffer that receives the new states
        s["slots"] = (torch.randperm(n, generator=g, device=dev)[:b].to(torch.int32) if case["slots"] else None)
        return s
    L, lens = case["L"], _lens(case)
    n = len(lens) if lens is not None else b
    s.update(x=rn(b, L, C, dtype=dt), r=rn(b, L, C, dtype=dt), i=rn(b, L, C, dtype=dt) if case["gate"] else None,
             lens=lens, cu=_offsets(lens, dev) if lens is not None else None, state=rn(n, C) if case["init"] else None,
             y=torch.zeros(b, L, C, dtype=dt, device=dev))
    if case["train"]:
        s.update(dy=rn(b, L, C, dtype=dt), dfinal=rn(n, C) if case["init"] else None,
                 dx=torch.zeros_like(s["x"]), dr=torch.zeros_like(s["r"]),
                 di=torch.zeros_like(s["i"]) if case["gate"] else None)
    return s


def work(case):
    e = 2 if case["dtype"] == "bfloat16" else 4
    if case["op"] in ("bn", "bnb"):
        n, er = case["T"] * case["C"], 2 if case["res"] == "bfloat16" else 4
        z, out = int(bool(case["gate"])), int(bool(case["pre"]))
        if case["op"] == "bn":
            return dict(bytes=n * (e * (1 + z + out) + 2 * er), flops=n * 20)
        return dict(bytes=n * (e * (2 + 2 * z + out) + 3 * er), flops=n * 50)
    if case["op"] == "rot":
        lens = _lens(case)
        tok = sum(lens) if lens is not None else case["b"] * max(1, case["L"])
        heads = tok * (case["hq"] + case["hk"])
        return dict(bytes=2 * e * heads * case["D"], flops=heads * case["rot"] * 3)
    ins = 2 + int(case["gate"])
    if case["op"] == "step":
        n = case["b"] * case["C"]
        return dict(bytes=n * (8 + e * (ins + 1)), flops=n * 20)
    lens = _lens(case)
    tok, seqs = (sum(lens), len(lens)) if lens is not None else (case["b"] * case["L"], case["b"])
    n, st = tok * case["C"], 4 * seqs * case["C"]
    got = dict(bytes=n * e * (ins + 1) + st * (1 + int(case["init"])), flops=n * 20)
    if case["train"]:       # the gradients begin when y is written: the inputs are read by both
        got = dict(bytes=got["bytes"] + n * e * (2 * ins + 1) + st * (1 + 2 * int(case["init"])), flops=n * 70)
    return got


# ------------------------------------------------------------------ plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 of [n, L, C] from zero: blocks side by side, then their ends."""
    n, L, C = a.shape
    T = max(1, int(math.sqrt(L)))
    m = -(-L // T)
    pad = m * T - L
    if pad:
        a = torch.cat([a, a.new_ones(n, pad, C)], 1)
        b = torch.cat([b, b.new_zeros(n, pad, C)], 1)
    a, b = a.reshape(n, m, T, C), b.reshape(n, m, T, C)
    h, p = torch.empty_like(b), torch.empty_like(a)
    h[:, :, 0], p[:, :, 0] = b[:, :, 0], a[:, :, 0]
    for t in range(1, T):
        h[:, :, t] = a[:, :, t] * h[:, :, t - 1] + b[:, :, t]
        p[:, :, t] = p[:, :, t - 1] * a[:, :, t]
    for j in range(1, m):       # the block before is complete
        h[:, j] += p[:, j] * h[:, j - 1, -1][:, None]
    return h.reshape(n, m * T, C)[:, :L]


def _gates(s, x, r, i):
    """a, w, u (the gated input), the gates' sigmoids and log a (with lerp None)."""
    si = torch.sigmoid(i.float()) if i is not None else None
    u = x.float() * si if i is not None else x.float()
    if s["case"]["lerp"]:
        v = r.float() + s["decay"] if s["decay"] is not None else r.float()
        return torch.sigmoid(v), torch.sigmoid(-v), u, torch.sigmoid(v), si, None
    sr = torch.sigmoid(r.float())
    la = sr * (torch.nn.functional.softplus(s["decay"]) * -POWER)
    return torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), u, sr, si, la


def _ends(s):
    """First rows and rows behind the last of the sequences that have tokens, and which these are."""
    cu = s["cu"].long()
    has = torch.tensor([i for i, n in enumerate(s["lens"]) if n], device=cu.device)
    return cu[has], cu[has + 1], has


def _gs(s):
    case = s["case"]
    a, w, u, sr, si, la = _gates(s, s["x"], s["r"], s["i"])
    if s["lens"] is not None:
        rows = sum(s["lens"])
        a, w, u, sr = (t[:, :rows] for t in (a, w, u, sr))
        si, la = (t[:, :rows] if t is not None else None for t in (si, la))
        first, end, has = _ends(s)
    f, f0 = a.clone(), w * u
    if s["lens"] is None:
        if s["state"] is not None:
            f0[:, 0] += a[:, 0] * s["state"]
    else:
        if s["state"] is not None:
            f0[0, first] += a[0, first] * s["state"][has]
        f[0, first] = 0
    h = _scan(f, f0)
    s["y"][:, :h.shape[1]] = h
    if s["lens"] is None:
        final = h[:, -1].clone()
    else:
        final = s["state"].clone() if s["state"] is not None else h.new_zeros(len(s["lens"]), case["C"])
        final[has] = h[0, end - 1]
    if not case["train"]:
        return s["y"], final
    # the adjoint of h_t, from the last token back
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    up = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    d = s["dy"][:, :h.shape[1]].to(torch.float32, copy=True)
    if s["lens"] is None:
        if s["state"] is not None:
            before[:, 0] = s["state"]
            d[:, -1] += s["dfinal"]
    else:
        before[0, first] = s["state"][has] if s["state"] is not None else 0.0
        up[0, end - 1] = 0
        if s["dfinal"] is not None:
            d[0, end - 1] += s["dfinal"][has]
    gr = _scan(up.flip(1), d.flip(1)).flip(1)
    if s["lens"] is None:
        dinit = a[:, 0] * gr[:, 0]
    else:
        dinit = s["dfinal"].clone() if s["dfinal"] is not None else h.new_zeros(len(s["lens"]), case["C"])
        dinit[has] = a[0, first] * gr[0, first]
    rows = h.shape[1]
    du = gr * w
    s["dx"][:, :rows] = du * si if si is not None else du
    if si is not None:
        s["di"][:, :rows] = du * u * (1 - si)
    if la is None:
        dv = gr * (before - u) * (a * w)
        s["dr"][:, :rows] = dv
        return s["y"], final, s["dx"], s["dr"], s["di"], dv.sum((0, 1)) if s["decay"] is not None else None, dinit
    over = torch.where(la == 0, torch.zeros_like(la), la / w)
    dl = gr * (before * (a * la) - u * (a * a * over))         # log a times its gradient
    s["dr"][:, :rows] = dl * (1 - sr)
    sp = torch.nn.functional.softplus(s["decay"])
    dd = dl.sum((0, 1)) * (torch.sigmoid(s["decay"]) / sp)
    return s["y"], final, s["dx"], s["dr"], s["di"], dd, dinit


def _step(s):
    a, w, u = _gates(s, s["x"], s["r"], s["i"])[:3]
    at = s["slots"]
    new = a * (s["state"] if at is None else s["state"][at.long()]) + w * u
    if at is None:
        s["out"].copy_(new)
    else:
        s["out"][at.long()] = new
    return new.to(s["x"].dtype), s["out"]


def _positions(s):
    """The position of every token, [b, L] (or [b])."""
    if s["pos"] is not None:
        return s["pos"]
    L, dev = s["case"]["L"], s["q"].device
    t = torch.arange(L, device=dev)
    if s["lens"] is not None:
        cu = s["cu"].long()
        seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device=dev), cu[1:] - cu[:-1],
                                      output_size=sum(s["lens"]))
        t = t[:sum(s["lens"])] - cu[seq]
    return (t + s["offset"])[None]


def _rot(s):
    case = s["case"]
    n, half = case["rot"], case["rot"] // 2
    ang = _positions(s).double()[..., None] * s["freq"]
    c, sn = (torch.cos(ang) * s["scale"]).float()[..., None, :], (torch.sin(ang) * s["scale"]).float()[..., None, :]
    if case["inverse"]:
        sn = -sn
    for name in "qk":
        if s[name] is None:
            continue
        out, rows = s[name + "_out"], slice(None)
        src = s[name]
        if s["lens"] is not None:
            rows = slice(0, sum(s["lens"]))
            src, out = src[:, rows], out[:, rows]
        x = src.float()
        lo, hi = (x[..., 0:n:2], x[..., 1:n:2]) if case["inter"] else (x[..., :half], x[..., half:n])
        a, b = lo * c - hi * sn, hi * c + lo * sn
        out[..., :n] = torch.stack([a, b], -1).flatten(-2) if case["inter"] else torch.cat([a, b], -1)
        out[..., n:] = src[..., n:]
    return s["q_out"], s["k_out"]


def _normed(x, kind, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, r


def _scaled(x, w, b):
    x = x * w if w is not None else x
    return x + b if b is not None else x


def _act(kind, z):
    """The gate and its slope."""
    if kind == "id":
        return z, torch.ones_like(z)
    sg = torch.sigmoid(z)
    return (sg, sg * (1 - sg)) if kind == "sigmoid" else (z * sg, sg * (1 + z * (1 - sg)))


def _bn_state(s):
    case = s["case"]
    y = s["y"].float()
    yh, ry = _normed(y, case["post"], s["eps"]) if case["post"] else (y, None)
    n = _scaled(yh, s["post_w"], s["post_b"])
    act, slope = _act(case["gate"], s["z"].float()) if case["gate"] else (None, None)
    h = s["x"].float() + s["alpha"] * (n * act if act is not None else n)
    return yh, ry, n, act, slope, h


def _bn(s):
    h = _bn_state(s)[-1]
    out = None
    if s["case"]["pre"]:
        out = _scaled(_normed(h, s["case"]["pre"], s["eps"])[0], s["pre_w"], s["pre_b"]).to(s["y"].dtype)
    return h.to(s["x"].dtype), out


def _norm_back(d, w, xh, r, kind):
    """Gradients of a norm's input, weight and bias from its output's."""
    g = d * w if w is not None else d
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    return dx * r, (d * xh).sum(0), d.sum(0)


def _bnb(s):
    case = s["case"]
    yh, ry, n, act, slope, h = _bn_state(s)
    d = s["dh"].float()
    w2 = b2 = dz = w1 = b1 = None
    if case["pre"]:
        hh, rh = _normed(h, case["pre"], s["eps"])
        dx, w2, b2 = _norm_back(s["dout"].float(), s["pre_w"], hh, rh, case["pre"])
        d = d + dx
    dn = d * s["alpha"]
    if act is not None:
        dz = (dn * n * slope).to(s["z"].dtype)
        dn = dn * act
    dy = dn
    if case["post"]:
        dy, w1, b1 = _norm_back(dn, s["post_w"], yh, ry, case["post"])
    keep = lambda g, p: g if p is not None else None  # noqa: E731
    return (dy.to(s["y"].dtype), d.to(s["x"].dtype), dz, keep(w1, s["post_w"]), keep(b1, s["post_b"]),
            keep(w2, s["pre_w"]), keep(b2, s["pre_b"]))


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from state_space_sequence_mamba_b200 import binding as m3
    case = s["case"]
    op = case["op"]
    if op in ("bn", "bnb"):
        args = dict(z=s["z"], gate={"": None, "id": None}.get(case["gate"], case["gate"]), alpha=s["alpha"],
                    post=case["post"] or None, post_weight=s["post_w"], post_bias=s["post_b"],
                    pre=case["pre"] or None, pre_weight=s["pre_w"], pre_bias=s["pre_b"], eps=s["eps"])
        if op == "bn":
            return m3.block_norm_fwd(s["y"], s["x"], **args)
        g = m3.block_norm_bwd(s["dh"], s["dout"], s["y"], s["x"], **args)
        return tuple(g[n] for n in ("dy", "dresidual", "dz", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"))
    if op == "rot":
        return m3.rotary(s["q"], s["k"], s["freq"], positions=s["pos"], offset=0 if s["pos"] is not None else s["offset"],
                         cu_seqlens=s["cu"], interleaved=case["inter"], inverse=case["inverse"], scale=s["scale"],
                         q_out=s["q_out"], k_out=s["k_out"])
    args = dict(i=s["i"], decay=s["decay"], power=POWER, lerp=case["lerp"])
    if op == "step":
        return m3.gated_scan_step(s["x"], s["r"], s["state"], state_out=s["out"], slots=s["slots"], **args)
    args.update(init=s["state"], cu_seqlens=s["cu"])
    y, final, marks = m3.gated_scan_fwd(s["x"], s["r"], y=s["y"], marks=case["train"], **args)
    if not case["train"]:
        return y, final
    g = m3.gated_scan_bwd(s["dy"], s["x"], s["r"], dfinal=s["dfinal"], marks=marks,
                          grads=(s["dx"], s["dr"], s["di"]), **args)
    return y, final, g["dx"], g["dr"], g["di"], g["ddecay"], g["dinit"]


def run(state):
    if own:
        return _own(state)
    return {"gs": _gs, "step": _step, "rot": _rot, "bn": _bn, "bnb": _bnb}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"gs": _exact_gs, "step": _exact_step, "rot": _exact_rot, "bn": _exact_bn, "bnb": _exact_bn}[case["op"]](s)


def _leaves(s, names, grad):
    got = {n: None if s[n] is None else s[n].double() for n in names}
    for t in got.values():
        if t is not None and grad:
            t.requires_grad_()
    return got


def _terms(s, t):
    """a_t and what token t adds, from the definition."""
    add = t["x"] / (1 + torch.exp(-t["i"])) if t["i"] is not None else t["x"]
    if s["case"]["lerp"]:
        e = torch.exp(-(t["r"] + t["decay"] if t["decay"] is not None else t["r"]))
        return 1 / (1 + e), add * (e / (1 + e))
    la = -POWER * torch.log1p(torch.exp(t["decay"])) / (1 + torch.exp(-t["r"]))
    return torch.exp(la), add * torch.sqrt(-torch.expm1(2 * la))


def _exact_step(s):
    a, add = _terms(s, _leaves(s, ("x", "r", "i", "decay"), False))
    at = torch.arange(s["case"]["b"], device=a.device) if s["slots"] is None else s["slots"].long()
    new = s["state"].double()
    new[at] = a * new[at] + add
    return new[at], new


def _exact_gs(s):
    case = s["case"]
    t = _leaves(s, ("x", "r", "i", "decay"), case["train"])
    a, add = _terms(s, t)
    av, bv = a.detach(), add.detach()
    b, L, C = av.shape
    lens = s["lens"]
    runs, at = [(slice(None), 0, L, slice(None))], 0
    if lens is not None:
        runs = []
        for i, n in enumerate(lens):
            runs.append((slice(0, 1), at, at + n, slice(i, i + 1)))
            at += n
    n = len(lens) if lens is not None else b
    h = torch.zeros_like(av)
    final = s["state"].double() if s["state"] is not None else av.new_zeros(n, C)
    start = final.clone()
    for rows, lo, hi, who in runs:      # the recurrence, a token at a time
        x = start[who]
        for p in range(lo, hi):
            x = torch.addcmul(bv[rows, p], av[rows, p], x)
            h[rows, p] = x
        final[who] = x
    if not case["train"]:
        return h, final
    g = s["dy"].double()
    if lens is not None:
        g[:, sum(lens):] = 0
    dinit = s["dfinal"].double() if s["dfinal"] is not None else av.new_zeros(n, C)
    prev = torch.zeros_like(h)
    for rows, lo, hi, who in runs:      # the adjoint of the state behind each token, from the last one back
        x = dinit[who]
        for p in range(hi - 1, lo - 1, -1):
            x = g[rows, p] + x
            g[rows, p] = x
            x = av[rows, p] * x
        dinit[who] = x
        if hi > lo:
            prev[rows, lo] = start[who]
            prev[rows, lo + 1:hi] = h[rows, lo:hi - 1]
    lead = [x for x in t.values() if x is not None]
    got = iter(torch.autograd.grad([a, add], lead, [g * prev, g]))
    dx, dr, di, dd = (None if t[k] is None else next(got) for k in ("x", "r", "i", "decay"))
    return h, final, dx, dr, di, dd, dinit


def _exact_rot(s):
    case = s["case"]
    n, got = case["rot"], []
    if s["pos"] is not None:
        at = s["pos"].double()
    else:
        at = torch.cat([torch.arange(m, dtype=torch.float64) for m in s["lens"] or [case["L"]]])[None] + s["offset"]
    ang = at.to(s["q"].device)[..., None, None] * s["freq"]
    turn = torch.polar(torch.full_like(ang, s["scale"]), -ang if case["inverse"] else ang)
    for name in "qk":
        if s[name] is None:
            got.append(None)
            continue
        x = s[name].double()
        rows = sum(s["lens"]) if s["lens"] is not None else None
        part = x[..., :n] if rows is None else x[:, :rows, :, :n]
        pairs = part.unflatten(-1, (-1, 2)) if case["inter"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = (z if case["inter"] else z.transpose(-1, -2)).flatten(-2)
        if rows is None:
            x[..., :n] = z
        else:
            x[:, :rows, :, :n] = z
            x[:, rows:] = 0
        got.append(x)
    return tuple(got)


def _exact_bn(s):
    case = s["case"]
    names = ("y", "x", "z", "post_w", "post_b", "pre_w", "pre_b")
    back = case["op"] == "bnb"
    t = _leaves(s, names, back)

    def norm(x, which):
        if not case[which]:
            return x
        if case[which] == "layer":
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            x = (x - mean) / torch.sqrt(var + s["eps"])
        else:
            x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + s["eps"])
        w, b = t[which + "_w"], t[which + "_b"]
        return x * (1.0 if w is None else w) + (0.0 if b is None else b)

    add = norm(t["y"], "post")
    if case["gate"]:
        z = t["z"]
        sg = 1 / (1 + torch.exp(-z))
        add = add * {"id": z, "sigmoid": sg, "silu": z * sg}[case["gate"]]
    h = t["x"] + s["alpha"] * add
    out = norm(h, "pre") if case["pre"] else None
    if not back:
        return h, out
    total = (h * s["dh"].double()).sum()
    if out is not None:
        total = total + (out * s["dout"].double()).sum()
    lead = [t[k] for k in names if t[k] is not None]
    got = iter(torch.autograd.grad(total, lead))
    return tuple(None if t[k] is None else next(got) for k in names)
