"""Cases of linear attention with a decay for each head (prompts, single tokens, gradients) and of
the grouped norm with a gate that follows it, each in a plain form of elementary torch operations
and as calls of the library's entry points.

Linear attention, per sequence and head h with decay a = exp(log_decay[h]):
    S_t = a S_{t-1} + k_t v_t^T            (S_{-1} = the initial state, K x V, fp32)
    o_t = scale S_t^T q_t
q, k and v may each have fewer heads than there are decays (a divisor): head h reads head
h // (H / heads) of the tensor. Packed sequences lie one behind the other in the rows of one
tensor, sequence i in rows [cu_seqlens[i], cu_seqlens[i + 1]); rows behind the last are no tokens.

Grouped norm over the channels of each row (channels last), with an activation:
    y = (x - mean) / sqrt(var + eps) * weight + bias      per row and group
    out = y * silu(z)   with a gate z,   silu(y) without
"""
import math

import torch

own = False

CHUNK = 128


# ------------------------------------------------------------------ the cases

def listed():
    bf, f32 = "bfloat16", "float32"
    return [
        # the smallest scan of the package's workloads: one head, 64 tokens, fp32 (latency)
        dict(name="fwd_b1_L64_H1_fp32", op="fwd", b=1, L=64, H=1, hq=1, hk=1, hv=1, K=16, V=16,
             dtype=f32, init=False, lens=""),
        # the package's prefill workload: 64 heads share one key and query head
        dict(name="fwd_b4_L2048_H64", op="fwd", b=4, L=2048, H=64, hq=1, hk=1, hv=64, K=128, V=64,
             dtype=bf, init=True, lens=""),
        # the package's long-context workload, every head with queries and keys of its own
        dict(name="fwd_b1_L65536_H64", op="fwd", b=1, L=65536, H=64, hq=64, hk=64, hv=64, K=128,
             V=64, dtype=bf, init=True, lens=""),
        # a server's prompts of unequal lengths in one packed tensor, grouped keys and values,
        # five spare rows at the end
        dict(name="fwd_packed_H16", op="fwd", b=1, L=4229, H=16, hq=16, hk=4, hv=4, K=96, V=128,
             dtype=bf, init=True, lens="1,777,0,2048,129,64,1000,205"),
        # one token of the package's decode workload: 128 sequences, 64 heads
        dict(name="step_b128_H64", op="step", b=128, H=64, hq=1, hk=1, hv=64, K=128, V=64,
             dtype=bf, slots=0),
        # one token of a single user (latency), the state kept in a pool of slots
        dict(name="step_b1_H64", op="step", b=1, H=64, hq=64, hk=64, hv=64, K=128, V=64,
             dtype=bf, slots=8),
        # a training step's gradients at the prefill workload's sizes
        dict(name="bwd_b4_L2048_H64", op="bwd", b=4, L=2048, H=64, hq=64, hk=64, hv=64, K=128,
             V=64, dtype=bf, init=False, lens=""),
        # gradients of packed sequences with grouped keys and values, and of their states
        dict(name="bwd_packed_H8", op="bwd", b=1, L=1501, H=8, hq=8, hk=2, hv=2, K=64, V=96,
             dtype=bf, init=True, lens="500,1,0,700,297"),
        # the norm of the prefill's 64 heads of 64 channels with a gate
        dict(name="gn_T8192_C4096_G64", op="gn", T=8192, C=4096, G=64, dtype=bf, gate=True,
             center=True, affine=True),
        # the same for one decode step's 128 rows
        dict(name="gn_T128_C4096_G64", op="gn", T=128, C=4096, G=64, dtype=bf, gate=True,
             center=True, affine=True),
        # its gradients in training
        dict(name="gnb_T8192_C4096_G64", op="gnb", T=8192, C=4096, G=64, dtype=bf, gate=True,
             center=True, affine=True),
        # gradients at an odd row count and group size, fp32, mean kept, no gate
        dict(name="gnb_T777_C1920_G16_fp32", op="gnb", T=777, C=1920, G=16, dtype=f32, gate=False,
             center=False, affine=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "step", "bwd", "gn", "gnb"))
    dtype = rng.choice(("bfloat16", "bfloat16", "bfloat16", "float32"))
    if op in ("gn", "gnb"):
        D = rng.choice((8, 24, 32, 48, 64, 96, 120, 128, 160, 256, 512))
        G = rng.choice((1, 2, 4, 8, 12, 16, 24, 32, 64))
        while D * G > 8192:
            G //= 2
        return dict(op=op, T=_log_uniform(rng, 1, 16384), C=D * G, G=G, dtype=dtype,
                    gate=rng.random() < 0.75, center=rng.random() < 0.5,
                    affine=rng.random() < 0.75)
    H = rng.choice((1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64))
    div = [d for d in range(1, H + 1) if H % d == 0]
    share = rng.random()
    if share < 0.5:
        hq = hk = hv = H                              # every head its own
    elif share < 0.8:
        hq, hk = H, rng.choice(div)                   # grouped keys and values
        hv = hk
    else:
        hq, hv = rng.choice(div), H                   # shared queries and keys
        hk = hq
    K = 8 * rng.randint(2, 16)
    V = 8 * rng.randint(2, 16) if rng.random() < 0.75 else 8 * rng.randint(17, 32)
    if op == "step":
        b = _log_uniform(rng, 1, 256)
        return dict(op=op, b=b, H=H, hq=hq, hk=hk, hv=hv, K=K, V=V, dtype=dtype,
                    slots=b + rng.randint(1, 40) if rng.random() < 0.5 else 0)
    rows = _log_uniform(rng, 1, (262144 if op == "fwd" else 131072) // (H if dtype == "bfloat16" else 4 * H))
    if rng.random() < 0.4 and rows > 1:
        n = min(rows, rng.randint(1, 12))
        cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
        lens = [y - x for x, y in zip([0] + cuts, cuts + [rows])]
        return dict(op=op, b=1, L=rows + rng.choice((0, 0, 3, 40)), H=H, hq=hq, hk=hk, hv=hv, K=K,
                    V=V, dtype=dtype, init=rng.random() < 0.5, lens=",".join(map(str, lens)))
    b = rng.randint(1, 4)
    return dict(op=op, b=b, L=max(1, rows // b), H=H, hq=hq, hk=hk, hv=hv, K=K, V=V, dtype=dtype,
                init=rng.random() < 0.5, lens="")


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case.get("lens") else None


def prepare(case, seed):
    dev, dt = torch.device("cuda"), getattr(torch, case["dtype"])
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = dict(case=case)
    if case["op"] in ("gn", "gnb"):
        T, C = case["T"], case["C"]
        s.update(x=rn(T, C, dtype=dt), z=rn(T, C, dtype=dt) if case["gate"] else None, eps=1e-5)
        s.update(w=1 + 0.1 * rn(C) if case["affine"] else None,
                 bias=0.1 * rn(C) if case["affine"] else None)
        if case["op"] == "gnb":
            s["dout"] = rn(T, C, dtype=dt)
        return s
    b, H, K, V = case["b"], case["H"], case["K"], case["V"]
    # decays between 1/2 and 1 - 2^-9 per token, another set per seed
    u = 1 + 8 * (torch.arange(H, device=dev) + torch.rand(H, generator=g, device=dev)) / H
    s.update(log_decay=torch.log1p(-torch.exp2(-u)), scale=K ** -0.5)
    if case["op"] == "step":
        n = case["slots"] or b
        s.update(q=rn(b, case["hq"], K, dtype=dt), k=rn(b, case["hk"], K, dtype=dt),
                 v=rn(b, case["hv"], V, dtype=dt), state=rn(n, H, K, V))
        s["out"] = s["state"].clone()      # the buffer that receives the new states
        s["slots"] = (torch.randperm(n, generator=g, device=dev)[:b].to(torch.int32)
                      if case["slots"] else None)
        return s
    L, lens = case["L"], _lens(case)
    n = len(lens) if lens is not None else b
    s.update(q=rn(b, L, case["hq"], K, dtype=dt), k=rn(b, L, case["hk"], K, dtype=dt),
             v=rn(b, L, case["hv"], V, dtype=dt), lens=lens, cu=None,
             state=rn(n, H, K, V) if case["init"] else None)
    if lens is not None:
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] == "fwd":
        s["o"] = torch.zeros(b, L, H, V, dtype=dt, device=dev)
    else:
        s.update(do=rn(b, L, H, V, dtype=dt), dfinal=rn(n, H, K, V) if case["init"] else None,
                 dq=torch.zeros_like(s["q"]), dk=torch.zeros_like(s["k"]),
                 dv=torch.zeros_like(s["v"]))
    return s


def work(case):
    e = 2 if case["dtype"] == "bfloat16" else 4
    if case["op"] in ("gn", "gnb"):
        n, z = case["T"] * case["C"], int(case["gate"])
        tensors = 2 + z if case["op"] == "gn" else 3 + 2 * z
        return dict(bytes=n * e * tensors + 4 * case["C"] * 2 * int(case["affine"]),
                    flops=n * (12 if case["op"] == "gn" else 30))
    H, K, V = case["H"], case["K"], case["V"]
    if case["op"] == "step":
        n = case["b"]
        return dict(bytes=n * (H * K * V * 8 + e * ((case["hq"] + case["hk"]) * K + (case["hv"] + H) * V)),
                    flops=n * H * K * V * 5)
    lens = _lens(case)
    tok, n = (sum(lens), len(lens)) if lens is not None else (case["b"] * case["L"], case["b"])
    ins = (case["hq"] + case["hk"]) * K + case["hv"] * V
    states = n * H * K * V * 4
    if case["op"] == "fwd":
        return dict(bytes=tok * e * (ins + H * V) + states * (1 + int(case["init"])),
                    flops=tok * H * 4 * K * V)
    return dict(bytes=tok * e * (2 * ins + H * V) + states * (1 + 2 * int(case["init"])),
                flops=tok * H * 10 * K * V)


# ------------------------------------------------------------------ plain forms

def _powers(log_decay, n):
    """a^n for every head: [H, *n.shape]."""
    e = log_decay.double().reshape(-1, *[1] * n.dim()) * n.double()
    return torch.exp(torch.where(n == 0, torch.zeros_like(e), e)).float()


def _heads(x, H):
    """[n, h, ...] with every head h repeated for the H / h heads that read it."""
    return x if x.shape[1] == H else x.repeat_interleave(H // x.shape[1], 1)


def _fold(x, h):
    """The sum over the heads that share one of h: [n, H, L, D] -> [n, h, L, D]."""
    n, H, L, D = x.shape
    return x if h == H else x.reshape(n, h, H // h, L, D).sum(2)


def _mix(q, k, v, log_decay):
    """sum over s <= t of a^(t - s) (q_t . k_s) v_s on [n, heads, L, D] in fp32, in chunks."""
    H, L = log_decay.shape[0], q.shape[2]
    C = min(CHUNK, L)
    m = -(-L // C)
    pad = m * C - L

    def cut(x):
        return torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(x.shape[0], x.shape[1], m, C, x.shape[3])

    qc, kc, vc = cut(q), cut(k), cut(v)
    hs = max(q.shape[1], k.shape[1])
    hs = hs if hs % q.shape[1] == 0 and hs % k.shape[1] == 0 else H
    score = _heads(_heads(qc, hs) @ _heads(kc, hs).transpose(-1, -2), H)
    i = torch.arange(C, device=q.device)
    mask = _powers(log_decay, (i[:, None] - i[None]).clamp(min=0)) * (i[:, None] >= i[None])
    vh = _heads(vc, H)
    o = (score * mask[:, None]) @ vh
    if m > 1:
        kd = _heads(kc, H) * _powers(log_decay, C - 1 - i)[:, None, :, None]
        inc = kd.transpose(-1, -2) @ vh                                    # [n, H, m, K, V]
        j = torch.arange(m, device=q.device)
        d = j[:, None] - 1 - j[None]
        carry = _powers(log_decay, C * d.clamp(min=0)) * (d >= 0)           # [H, m, m]
        before = (carry @ inc.flatten(3)).reshape(inc.shape)
        o = o + (_heads(qc, H) @ before) * _powers(log_decay, i + 1)[:, None, :, None]
    return o.reshape(o.shape[0], H, m * C, -1)[:, :, :L]


def _rows(s, x, flip=False):
    """[b, L, h, D] rows -> fp32 [n, h, Lmax, D]: each sequence from its first token on (or, with
    flip, from its last back), zeros behind its end."""
    if s["lens"] is None:
        y = x.float().transpose(1, 2)
        return y.flip(2) if flip else y
    at, live = _places(s, flip)
    return (x[0].float()[at] * live[..., None, None]).transpose(1, 2)


def _places(s, flip=False):
    cu = s["cu"].long()
    n, start = cu[1:] - cu[:-1], cu[:-1]
    i = torch.arange(max(1, max(s["lens"])), device=cu.device)
    live = i[None] < n[:, None]
    at = start[:, None] + (n[:, None] - 1 - i[None] if flip else i[None].expand(len(n), -1))
    return torch.where(live, at, 0), live


def _back(s, y, out, flip=False):
    """The inverse of _rows, rounded once, into `out` [b, L, h, D]."""
    y = y.transpose(1, 2)
    if s["lens"] is None:
        return out.copy_(y.flip(1) if flip else y)
    total, n = sum(s["lens"]), (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device=n.device), n, output_size=total)
    i = torch.arange(total, device=n.device) - s["cu"].long()[seq]
    out[0, :total] = y[seq, n[seq] - 1 - i if flip else i].to(out.dtype)
    return out


def _lengths(s, L):
    """Tokens of each sequence [n, 1, 1] (H and position broadcast)."""
    n = torch.tensor([L], device=s["q"].device) if s["lens"] is None else (s["cu"][1:] - s["cu"][:-1]).long()
    return n[:, None, None]


def _decay_to(s, n, i):
    """a^(n - 1 - i) per sequence, head and token, 0 behind a sequence's end: [n, H, L, 1]."""
    e = n - 1 - i
    p = torch.exp(s["log_decay"].double()[None, :, None] * e.clamp(min=0).double()) * (e >= 0)
    return p.float()[..., None]


def _fwd(s):
    g, H = s["log_decay"], s["log_decay"].shape[0]
    q, k, v = (_rows(s, s[x]) for x in "qkv")
    i = torch.arange(q.shape[2], device=q.device)
    n = _lengths(s, q.shape[2])
    o = _mix(q, k, v, g)
    final = (_heads(k, H) * _decay_to(s, n, i)).transpose(-1, -2) @ _heads(v, H)
    if s["state"] is not None:
        o = o + (_heads(q, H) @ s["state"]) * _powers(g, i + 1)[..., None]
        final = final + s["state"] * torch.exp(g.double()[None, :, None, None] * n[..., None]).float()
    return _back(s, o * s["scale"], s["o"]), final


def _bwd(s):
    g, H, sc = s["log_decay"], s["log_decay"].shape[0], s["scale"]
    q, k, v, do = (_rows(s, s[x]) for x in ("q", "k", "v", "do"))
    i = torch.arange(q.shape[2], device=q.device)
    n = _lengths(s, q.shape[2])
    dq = _mix(do, v, k, g)
    if s["state"] is not None:
        dq = dq + (do @ s["state"].transpose(-1, -2)) * _powers(g, i + 1)[..., None]
    dq = _back(s, _fold(dq * sc, s["q"].shape[2]), s["dq"])
    del q, k, v, do
    q, k, v, do = (_rows(s, s[x], True) for x in ("q", "k", "v", "do"))
    dk, dv = _mix(v, do, q, g) * sc, _mix(k, q, do, g) * sc
    # position i of the flipped order is token n - 1 - i, whose weight in S_0's gradient is a^(n - i)
    a = torch.exp(g)[:, None, None]
    dinit = (_heads(q, H) * (_decay_to(s, n, i) * a * sc)).transpose(-1, -2) @ do
    if s["dfinal"] is not None:
        p = _powers(g, i)[..., None]
        dk = dk + (_heads(v, H) @ s["dfinal"].transpose(-1, -2)) * p
        dv = dv + (_heads(k, H) @ s["dfinal"]) * p
        dinit = dinit + s["dfinal"] * torch.exp(g.double()[None, :, None, None] * n[..., None]).float()
    return (dq, _back(s, _fold(dk, s["k"].shape[2]), s["dk"], True),
            _back(s, _fold(dv, s["v"].shape[2]), s["dv"], True), dinit)


def _step(s):
    H = s["log_decay"].shape[0]
    q, k, v = (_heads(s[x].float(), H) for x in "qkv")
    at = s["slots"]
    old = s["state"] if at is None else s["state"][at.long()]
    new = old * torch.exp(s["log_decay"])[:, None, None] + k[..., None] * v[..., None, :]
    o = (q[..., None] * new).sum(-2) * s["scale"]
    if at is None:
        s["out"].copy_(new)
    else:
        s["out"][at.long()] = new
    return o.to(s["q"].dtype), s["out"]


def _normed(s):
    T, C, G = s["case"]["T"], s["case"]["C"], s["case"]["G"]
    x = s["x"].float().reshape(T, G, C // G)
    if s["case"]["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    return x * r, r


def _affine(s, xh):
    y = xh.reshape(s["x"].shape)
    if s["w"] is not None:
        y = y * s["w"] + s["bias"]
    return y


def _gn(s):
    y = _affine(s, _normed(s)[0])
    z = s["z"].float() if s["z"] is not None else y
    act = z * torch.sigmoid(z)
    return (y * act if s["z"] is not None else act).to(s["x"].dtype)


def _gnb(s):
    xh, r = _normed(s)
    y, d = _affine(s, xh), s["dout"].float()
    z = s["z"].float() if s["z"] is not None else y
    sg = torch.sigmoid(z)
    slope = sg * (1 + z * (1 - sg))
    dz = None
    if s["z"] is not None:
        dz = (d * y * slope).to(s["x"].dtype)
        dy = d * (z * sg)
    else:
        dy = d * slope
    dw = db = None
    dxh = dy
    if s["w"] is not None:
        dw, db = (dy * xh.reshape(dy.shape)).sum(0), dy.sum(0)
        dxh = dy * s["w"]
    dxh = dxh.reshape(xh.shape)
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if s["case"]["center"]:
        dx = dx - dxh.mean(-1, keepdim=True)
    return (dx * r).reshape(s["x"].shape).to(s["x"].dtype), dz, dw, db


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from state_space_sequence_mamba_b200 import binding as m3
    op = s["case"]["op"]
    if op == "fwd":
        return m3.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                              init=s["state"], o=s["o"], cu_seqlens=s["cu"])
    if op == "step":
        return m3.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                               state_out=s["out"], slots=s["slots"], scale=s["scale"])
    if op == "bwd":
        g = m3.linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                           init=s["state"], dfinal=s["dfinal"], cu_seqlens=s["cu"],
                           grads=(s["dq"], s["dk"], s["dv"]))
        return g["dq"], g["dk"], g["dv"], g["dinit"]
    args = dict(groups=s["case"]["G"], weight=s["w"], bias=s["bias"], z=s["z"],
                center=s["case"]["center"], eps=s["eps"])
    if op == "gn":
        return m3.group_norm_fwd(s["x"], **args)
    g = m3.group_norm_bwd(s["dout"], s["x"], **args)
    return g["dx"], g["dz"], g["dweight"], g["dbias"]


def run(state):
    if own:
        return _own(state)
    return {"fwd": _fwd, "bwd": _bwd, "step": _step, "gn": _gn, "gnb": _gnb}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gn" or case["op"] == "gnb":
        return _exact_norm(s)
    a = torch.exp(s["log_decay"].double())[:, None, None]
    H = a.shape[0]
    wide = lambda x, dim: x.double().repeat_interleave(H // x.shape[dim], dim)  # noqa: E731
    if case["op"] == "step":
        q, k, v = (wide(s[x], 1) for x in "qkv")
        at = torch.arange(case["b"], device=q.device) if s["slots"] is None else s["slots"].long()
        new = s["state"].double()
        new[at] = a * new[at] + torch.einsum("bhk,bhv->bhkv", k, v)
        return s["scale"] * torch.einsum("bhk,bhkv->bhv", q, new[at]), new
    seqs = _sequences(s)
    q, k, v = s["q"], s["k"], s["v"]
    n, K, V = len(seqs) if s["lens"] is not None else case["b"], case["K"], case["V"]
    zero = torch.zeros(n, H, K, V, dtype=torch.float64, device=q.device)
    S = s["state"].double() if s["state"] is not None else zero.clone()
    if case["op"] == "fwd":
        o = torch.zeros(*q.shape[:2], H, V, dtype=torch.float64, device=q.device)
        for rows, lo, hi, who in seqs:
            for t in range(lo, hi):     # the recurrence, a token at a time
                kt, vt, qt = (wide(x[rows, t], 1) for x in (k, v, q))
                S[who] = torch.addcmul(a * S[who], kt[..., None], vt[..., None, :])
                o[rows, t] = (qt[..., None, :] @ S[who]).squeeze(-2) * s["scale"]
        return o, S
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v))
    R = s["dfinal"].double() if s["dfinal"] is not None else zero.clone()

    def put(to, rows, t, x):            # the sum over the heads that read one head
        to[rows, t] = x.reshape(x.shape[0], to.shape[2], -1, x.shape[-1]).sum(2)

    for rows, lo, hi, who in seqs:
        for t in range(lo, hi):
            kt, vt, dt = (wide(x[rows, t], 1) for x in (k, v, s["do"]))
            S[who] = torch.addcmul(a * S[who], kt[..., None], vt[..., None, :])
            put(dq, rows, t, (S[who] @ dt[..., None]).squeeze(-1) * s["scale"])
        for t in range(hi - 1, lo - 1, -1):     # the adjoint of S_t, from the last token back
            kt, vt, qt, dt = (wide(x[rows, t], 1) for x in (k, v, q, s["do"]))
            R[who] = torch.addcmul(R[who], qt[..., None], dt[..., None, :], value=s["scale"])
            put(dk, rows, t, (R[who] @ vt[..., None]).squeeze(-1))
            put(dv, rows, t, (kt[..., None, :] @ R[who]).squeeze(-2))
            R[who] = a * R[who]
    return dq, dk, dv, R


def _sequences(s):
    """(batch rows, first token, end, states) of what the recurrence runs over at once."""
    if s["lens"] is None:
        return [(slice(None), 0, s["q"].shape[1], slice(None))]
    got, at = [], 0
    for i, n in enumerate(s["lens"]):
        got.append((slice(0, 1), at, at + n, slice(i, i + 1)))
        at += n
    return got


def _exact_norm(s):
    T, C, G = s["case"]["T"], s["case"]["C"], s["case"]["G"]
    lead = {k: None if s[k] is None else s[k].double() for k in ("x", "z", "w", "bias")}
    for v in lead.values():
        if v is not None:
            v.requires_grad_()
    x = lead["x"].view(T, G, C // G)
    if s["case"]["center"]:
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        x = (x - mean) / torch.sqrt(var + s["eps"])
    else:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + s["eps"])
    y = x.view(T, C)
    if lead["w"] is not None:
        y = y * lead["w"] + lead["bias"]
    gate = lead["z"] if lead["z"] is not None else y
    out = gate / (1 + torch.exp(-gate))
    out = out * y if lead["z"] is not None else out
    if s["case"]["op"] == "gn":
        return out.detach()
    out.backward(s["dout"].double())
    return tuple(None if lead[k] is None else lead[k].grad for k in ("x", "z", "w", "bias"))
