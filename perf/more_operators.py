"""How a Gaussian-predicting network's tokens get their content, as measured cases.

The feature maps of the input views go through group norms with an activation
(channels last); their pixels or patches are the encoder's states, and the
scene's tokens read them by cross attention before a head turns them into
Gaussians.  For training, the norm keeps its input in 8-bit blocks: feature
maps of all views are the largest activations of such a network.

Operators and the calls they are measured through
(gaussian_splatting_tile_amd.binding):
  attention_fwd, attention_bwd      attention_fwd, attention_bwd
  group_norm_fwd, group_norm_bwd    group_norm_fwd, group_norm_bwd

Attention layouts: q, out [batch][tokens][heads][d], k, v [batch][states]
[kv heads][d]; `heads / kv heads` neighbouring heads share a k and v.  States
from a batch element's length on, and those whose mask byte is 0, are not
attended.  8-bit tensors are blocks of 32 consecutive channels: e4m3 values and
one power-of-two scale (e8m0) per block, the smallest that leaves no value of
the block above 448.
"""

import math

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # serving: one camera token reads a scene's states, latency of a few small launches
        dict(name="attention one token, 4096 states", op="attention_fwd", batch=1, nq=1, nk=4096, heads=8, kv=8, d=64, dtype="bf16", states="all", train=False),
        # serving: a few camera tokens over the states of many views, heads sharing k and v, some views missing
        dict(name="attention 16 tokens, 65536 states shared", op="attention_fwd", batch=1, nq=16, nk=65536, heads=16, kv=2, d=128, dtype="bf16", states="masked", train=False),
        # training: 2048 scene tokens over 8 views of 2048 patches
        dict(name="attention 2048 tokens, 16384 states", op="attention_fwd", batch=1, nq=2048, nk=16384, heads=16, kv=16, d=64, dtype="bf16", states="all", train=True),
        # a batch of scenes with different numbers of views, one of them without any
        dict(name="attention fp16 ragged", op="attention_fwd", batch=4, nq=1000, nk=2777, heads=8, kv=4, d=128, dtype="f16", states="ragged", train=True),
        # the small head of a 1000-Gaussian scene in fp32, odd in every axis
        dict(name="attention fp32 odd", op="attention_fwd", batch=1, nq=257, nk=1001, heads=3, kv=3, d=40, dtype="f32", states="all", train=True),
        dict(name="attention backward 2048 tokens, 8192 states", op="attention_bwd", batch=1, nq=2048, nk=8192, heads=16, kv=16, d=64, dtype="bf16", states="all"),
        dict(name="attention backward fp16 ragged", op="attention_bwd", batch=4, nq=500, nk=1777, heads=8, kv=2, d=80, dtype="f16", states="ragged"),
        # serving: one small feature map
        dict(name="group norm 256 pixels x 64", op="group_norm_fwd", n=1, p=256, c=64, groups=8, dtype="bf16", act="silu", train=False, kept=False),
        # training: 8 views of 256 x 256 pixels, the input kept in 8 bits
        dict(name="group norm 8 x 65536 x 128", op="group_norm_fwd", n=8, p=65536, c=128, groups=32, dtype="bf16", act="silu", train=True, kept=True),
        # odd in every axis
        dict(name="group norm fp32 odd", op="group_norm_fwd", n=3, p=1001, c=90, groups=6, dtype="f32", act="gelu", train=True, kept=False),
        # training: 8 views of 128 x 128 pixels from their 8-bit checkpoint
        dict(name="group norm backward 8 x 16384 x 256 from 8 bits", op="group_norm_bwd", n=8, p=16384, c=256, groups=32, dtype="bf16", act="silu", kept=True),
        dict(name="group norm backward fp16 odd", op="group_norm_bwd", n=5, p=777, c=60, groups=12, dtype="f16", act="relu", kept=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention_fwd", "attention_fwd", "attention_bwd", "attention_bwd", "group_norm_fwd", "group_norm_bwd"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("attention"):
        kv = rng.choice([1, 2, 3, 4, 8])
        c = dict(op=op, batch=rng.choice([1, 1, 2, 3, 8]), nq=_log(rng, 1, 4096), nk=_log(rng, 1 if op == "attention_fwd" else 16, 32768), heads=kv * rng.choice([1, 1, 2, 4]), kv=kv,
                 d=rng.choice([32, 40, 64, 64, 80, 96, 128, 128, rng.randint(8, 128)]), dtype=t, states=rng.choice(["all", "all", "ragged", "masked"]))
        if op == "attention_fwd":
            c["train"] = rng.random() < 0.5
        most = (3.4e10 if op == "attention_fwd" else 1.7e10) / (6 if t == "f32" else 1)
        while c["batch"] * c["nq"] * c["nk"] * c["heads"] * c["d"] > most:
            if c["nk"] > c["nq"]:
                c["nk"] //= 2
            else:
                c["nq"] //= 2
        return c
    groups = rng.choice([1, 2, 4, 8, 16, 32, rng.randint(1, 32)])
    c = dict(op=op, n=rng.choice([1, 2, 3, 8, 16]), p=_log(rng, 16, 65536), c=groups * _log(rng, 1, 32), groups=groups, dtype=t,
             act=rng.choice(["none", "relu", "silu", "gelu"]), kept=rng.random() < 0.5)
    if c["kept"]:
        c["groups"] = rng.choice([1, 4, 8, 16, 32])
        c["c"] = 32 * rng.randint(1, 32)
    if op == "group_norm_fwd":
        c["train"] = c["kept"] or rng.random() < 0.5
    while c["n"] * c["p"] * c["c"] > (6e7 if op == "group_norm_fwd" else 3e7):
        c["p"] //= 2
    return c


def _lengths(c):
    """Attended states of every batch element: all, or (ragged) from all of
    them down to half, with none for the last of three or more."""
    if c["states"] != "ragged":
        return [c["nk"]] * c["batch"]
    n = [c["nk"] - i * c["nk"] // (2 * c["batch"]) for i in range(c["batch"])]
    if len(n) > 2:
        n[-1] = 0
    return n


def work(c):
    if c["op"].startswith("attention"):
        s = SIZES[c["dtype"]]
        states = sum(_lengths(c)) * (0.75 if c["states"] == "masked" else 1.0)
        rows = c["batch"] * c["nq"] * c["heads"]
        pairs = states * c["nq"] * c["heads"] * c["d"]
        mask = c["batch"] * c["nk"] if c["states"] == "masked" else 0
        if c["op"] == "attention_fwd":
            return {"bytes": 2 * rows * c["d"] * s + 2 * states * c["kv"] * c["d"] * s + (4 * rows if c["train"] else 0) + mask, "flops": 4 * pairs}
        # q, out, dout in, dq out; k and v in, dk and dv out (zeros where nothing is attended)
        return {"bytes": 4 * rows * c["d"] * s + 4 * rows + (2 * states + 2 * c["batch"] * c["nk"]) * c["kv"] * c["d"] * s + mask, "flops": 10 * pairs}
    m, s = c["n"] * c["p"] * c["c"], SIZES[c["dtype"]]
    if c["op"] == "group_norm_fwd":
        return {"bytes": m * (2 * s + (33 / 32 if c["kept"] else 0)) + 8 * c["c"] + (8 * c["n"] * c["groups"] if c["train"] else 0), "flops": 12 * m}
    return {"bytes": m * (2 * s + (33 / 32 if c["kept"] else s)) + 16 * c["c"] + 8 * c["n"] * c["groups"], "flops": 24 * m}


# ---- inputs -----------------------------------------------------------------
def _quantize(v):
    """fp32 [..][c] -> e4m3 values [..][c] and e8m0 scales [..][c / 32]."""
    b = v.unflatten(-1, (-1, 32))
    mant, e = torch.frexp(b.abs().amax(-1, keepdim=True) / 448.0)
    e = torch.where(mant == 0.5, e - 1, e).clamp(-127, 127)             # smallest e with amax <= 448 * 2^e
    e = torch.where(mant == 0, -127, e)
    q = torch.ldexp(b, -e).reshape(v.shape).to(torch.float8_e4m3fn)
    return q, (e[..., 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantize(q, scales):
    f = torch.ldexp(torch.ones((), device=q.device), scales.view(torch.uint8).int() - 127)
    return (q.float().unflatten(-1, (-1, 32)) * f[..., None]).reshape(q.shape)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def rand(*shape, scale=1.0, dtype="f32"):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(TYPES[dtype])

    def empty(*shape, dtype):
        return torch.empty(shape, device=dev, dtype=dtype)

    c = dict(case)
    s = {"case": c, "op": c["op"]}
    t = TYPES[c["dtype"]]
    if c["op"].startswith("attention"):
        b, nq, nk, h, kv, d = c["batch"], c["nq"], c["nk"], c["heads"], c["kv"], c["d"]
        s["q"] = rand(b, nq, h, d, scale=1.7, dtype=c["dtype"])
        # k and v are the two halves of one product's rows, as a network has them; channels have magnitudes of their own
        both = (rand(b, nk, 2, kv, d) * torch.exp(0.3 * rand(1, 1, 2, kv, d))).to(t)
        s["k"], s["v"] = both[:, :, 0], both[:, :, 1]
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev) if c["states"] == "ragged" else None
        s["mask"] = None
        if c["states"] == "masked":       # a quarter of the states missing, in runs
            run = max(1, nk // 64)
            s["mask"] = (torch.rand((b, -(-nk // run)), generator=gen, device=dev) < 0.75).repeat_interleave(run, 1)[:, :nk].to(torch.uint8).contiguous()
        s["scale"] = d ** -0.5
        s["out"] = empty(b, nq, h, d, dtype=t)
        if c["op"] == "attention_fwd":
            s["lse"] = empty(b, h, nq, dtype=torch.float32) if c["train"] else None
        else:
            kept = _plain_attention_fwd({**s, "lse": True})
            s["out"].copy_(kept["out"])
            s["lse"] = kept["lse"]
            s["dout"] = rand(b, nq, h, d, scale=1e-2, dtype=c["dtype"])
            s["dq"], s["dk"], s["dv"] = empty(b, nq, h, d, dtype=t), empty(b, nk, kv, d, dtype=t), empty(b, nk, kv, d, dtype=t)
        return s
    n, p, ch, g = c["n"], c["p"], c["c"], c["groups"]
    # features of a convolution: channels with offsets and magnitudes of their own, views of different contrast
    x = rand(1, 1, ch, scale=0.8) + torch.exp(0.4 * rand(n, 1, 1)) * torch.exp(0.5 * rand(1, 1, ch)) * rand(n, p, ch)
    s["x"] = x.to(t)
    s["gamma"], s["beta"] = 1.0 + 0.2 * rand(ch), 0.3 * rand(ch)
    s["scales"] = None
    if c["op"] == "group_norm_fwd":
        s["y"] = empty(n, p, ch, dtype=t)
        s["mean"], s["rstd"] = (empty(n, g, dtype=torch.float32), empty(n, g, dtype=torch.float32)) if c["train"] else (None, None)
        s["kept"], s["scales"] = (empty(n, p, ch, dtype=torch.float8_e4m3fn), empty(n, p, ch // 32, dtype=torch.float8_e8m0fnu)) if c["kept"] else (None, None)
    else:
        s["mean"], s["rstd"] = _moments(s["x"].float(), g)
        if c["kept"]:
            s["x"], s["scales"] = _quantize(s["x"].float())
        s["dy"] = rand(n, p, ch, scale=1e-2, dtype=c["dtype"])
        s["dx"] = empty(n, p, ch, dtype=t)
        s["dgamma"], s["dbeta"] = empty(ch, dtype=torch.float32), empty(ch, dtype=torch.float32)
    return s


# ---- one pass ---------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _attended(s):
    """[batch][1][1][states] truth values, or None: all of them."""
    c = s["case"]
    if s["lengths"] is not None:
        return (torch.arange(c["nk"], device=s["q"].device) < s["lengths"][:, None])[:, None, None]
    return None if s["mask"] is None else (s["mask"] != 0)[:, None, None]


def _heads(s):
    """q [b][h][nq][d], k and v [b][h][nk][d], all in fp32."""
    g = s["case"]["heads"] // s["case"]["kv"]
    return (s["q"].float().transpose(1, 2).contiguous(), s["k"].float().repeat_interleave(g, 2).transpose(1, 2).contiguous(),
            s["v"].float().repeat_interleave(g, 2).transpose(1, 2).contiguous())


def _plain_attention_fwd(s):
    q, k, v = _heads(s)
    z = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    seen = _attended(s)
    if seen is not None:
        z = torch.where(seen, z, -math.inf)
    top = z.amax(3, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(3, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    r = {"out": out.transpose(1, 2).to(s["q"].dtype).contiguous()}
    if s["lse"] is not None:
        r["lse"] = (top + torch.log(total))[..., 0]
    return r


def _plain_attention_bwd(s):
    c = s["case"]
    q, k, v = _heads(s)
    dout, out = s["dout"].float().transpose(1, 2).contiguous(), s["out"].float().transpose(1, 2)
    p = torch.exp(torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"] - s["lse"][..., None])
    seen = _attended(s)
    if seen is not None:
        p = torch.where(seen, p, 0.0)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), dout)
    ds = p * (torch.matmul(dout, v.transpose(2, 3).contiguous()) - (dout * out).sum(3, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    t, shared = s["q"].dtype, (c["kv"], c["heads"] // c["kv"])
    return {"dq": dq.transpose(1, 2).to(t).contiguous(), "dk": dk.unflatten(1, shared).sum(2).transpose(1, 2).to(t).contiguous(),
            "dv": dv.unflatten(1, shared).sum(2).transpose(1, 2).to(t).contiguous()}


def _moments(x, groups):
    """(mean, rstd) [n][groups] of fp32 [n][p][c]."""
    v = x.unflatten(2, (groups, -1))
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return mean, 1.0 / torch.sqrt(var + EPS)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    return torch.ones_like(z)


def _spread(v, channels):
    """[n][groups] -> [n][1][channels]"""
    return v.repeat_interleave(channels // v.shape[1], 1)[:, None]


def _plain_group_norm_fwd(s):
    c, x = s["case"], s["x"].float()
    mean, rstd = _moments(x, c["groups"])
    z = (x - _spread(mean, c["c"])) * _spread(rstd, c["c"]) * s["gamma"] + s["beta"]
    r = {"y": _act(z, c["act"]).to(s["x"].dtype)}
    if c["train"]:
        r["mean"], r["rstd"] = mean, rstd
    if c["kept"]:
        r["kept"], r["scales"] = _quantize(x)
    return r


def _plain_group_norm_bwd(s):
    c = s["case"]
    x = _dequantize(s["x"], s["scales"]) if c["kept"] else s["x"].float()
    rstd = _spread(s["rstd"], c["c"])
    h = (x - _spread(s["mean"], c["c"])) * rstd
    dz = s["dy"].float() * _act_slope(h * s["gamma"] + s["beta"], c["act"])
    g = dz * s["gamma"]
    mean_g = _spread(g.unflatten(2, (c["groups"], -1)).mean((1, 3)), c["c"])
    mean_gh = _spread((g * h).unflatten(2, (c["groups"], -1)).mean((1, 3)), c["c"])
    return {"dx": (rstd * (g - mean_g - h * mean_gh)).to(s["dy"].dtype), "dgamma": (dz * h).sum((0, 1)), "dbeta": dz.sum((0, 1))}


_plain = {"attention_fwd": _plain_attention_fwd, "attention_bwd": _plain_attention_bwd, "group_norm_fwd": _plain_group_norm_fwd,
          "group_norm_bwd": _plain_group_norm_bwd}


def _bytes(n, like):
    return torch.empty(n, dtype=torch.uint8, device=like.device)


def _own_attention_fwd(s):
    from gaussian_splatting_tile_amd import binding as B
    a = B.attention_struct(s["q"], s["k"], s["v"], s["out"], lse=s["lse"], kv_lengths=s["lengths"], kv_mask=s["mask"], scale=s["scale"])
    B.attention_fwd(a, _bytes(B.attention_fwd_workspace_bytes(a), s["q"]))
    return {k: s[k] for k in ("out", "lse") if s[k] is not None}


def _own_attention_bwd(s):
    from gaussian_splatting_tile_amd import binding as B
    a = B.attention_struct(s["q"], s["k"], s["v"], s["out"], lse=s["lse"], kv_lengths=s["lengths"], kv_mask=s["mask"], scale=s["scale"])
    g = B.attention_grads_struct(a, s["dout"], dq=s["dq"], dk=s["dk"], dv=s["dv"])
    B.attention_bwd(a, g, _bytes(B.attention_bwd_workspace_bytes(a, g), s["q"]))
    return {k: s[k] for k in ("dq", "dk", "dv")}


def _own_group_norm_fwd(s):
    from gaussian_splatting_tile_amd import binding as B
    c = s["case"]
    B.group_norm_fwd(s["x"], s["y"], c["groups"], gamma=s["gamma"], beta=s["beta"], act=c["act"], mean=s["mean"], rstd=s["rstd"], kept=s["kept"],
                     kept_scales=s["scales"], eps=EPS, workspace=_bytes(B.group_norm_fwd_workspace_bytes(c["n"], c["p"], c["c"], c["groups"]), s["x"]))
    return {k: s[k] for k in ("y", "mean", "rstd", "kept", "scales") if s[k] is not None}


def _own_group_norm_bwd(s):
    from gaussian_splatting_tile_amd import binding as B
    c = s["case"]
    B.group_norm_bwd(s["x"], s["mean"], s["rstd"], s["dy"], s["dx"], c["groups"], gamma=s["gamma"], beta=s["beta"], act=c["act"], dgamma=s["dgamma"],
                     dbeta=s["dbeta"], x_scales=s["scales"], workspace=_bytes(B.group_norm_bwd_workspace_bytes(c["n"], c["p"], c["c"], c["groups"]), s["x"]))
    return {k: s[k] for k in ("dx", "dgamma", "dbeta")}


_own = {"attention_fwd": _own_attention_fwd, "attention_bwd": _own_attention_bwd, "group_norm_fwd": _own_group_norm_fwd,
        "group_norm_bwd": _own_group_norm_bwd}


# ---- the definitions in 64 bits ---------------------------------------------
def _exact_attention(s):
    c, scale = s["case"], s["scale"]
    b, nq, nk, kv, d = c["batch"], c["nq"], c["nk"], c["kv"], c["d"]
    g = c["heads"] // kv
    # the heads that share a k are rows of one matrix: [b][kv][nq * g][d]
    rows = lambda t: t.double().reshape(b, nq, kv, g, d).permute(0, 2, 1, 3, 4).reshape(b, kv, nq * g, d)
    back = lambda t: t.reshape(b, kv, nq, g, d).permute(0, 2, 1, 3, 4).reshape(b, nq, kv * g, d)
    q, k, v = rows(s["q"]), s["k"].double().permute(0, 2, 1, 3), s["v"].double().permute(0, 2, 1, 3)
    z = q @ k.mT * scale
    for i, n in enumerate(_lengths(c)):
        z[i, :, :, n:] = -math.inf
    if s["mask"] is not None:
        z.masked_fill_((s["mask"] == 0)[:, None, None, :], -math.inf)
    if c["op"] == "attention_fwd":
        lse = torch.logsumexp(z, 3, keepdim=True)
        p = torch.exp(z - lse.clamp(min=-1e300))
        out = {"out": back(p @ v)}
        if c["train"]:
            out["lse"] = lse.reshape(b, kv, nq, g).permute(0, 1, 3, 2).reshape(b, kv * g, nq)
        return out
    lse = s["lse"].double().reshape(b, kv, g, nq).permute(0, 1, 3, 2).reshape(b, kv, nq * g, 1)
    p = torch.exp(z.sub_(lse.clamp(min=-1e300)))
    dout = rows(s["dout"])
    dv = p.mT @ dout
    ds = p.mul_(dout @ v.mT - torch.linalg.vecdot(dout, rows(s["out"]))[..., None])
    return {"dq": back(ds @ k * scale), "dk": (ds.mT @ q * scale).permute(0, 2, 1, 3), "dv": dv.permute(0, 2, 1, 3)}


def _round_e4m3(v):
    """Nearest value of 1 sign, 4 exponent and 3 mantissa bits, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"].startswith("attention"):
        return _exact_attention(s)
    n, p, ch, groups = c["n"], c["p"], c["c"], c["groups"]
    by_group = lambda t: t.reshape(n, p, groups, ch // groups).transpose(1, 2).reshape(n, groups, -1)
    flat = lambda t: t.reshape(n, groups, p, ch // groups).transpose(1, 2).reshape(n, p, ch)
    per_channel = lambda t: t.double().reshape(1, groups, 1, ch // groups).expand(n, groups, p, ch // groups).reshape(n, groups, -1)
    gamma, beta = per_channel(s["gamma"]), per_channel(s["beta"])
    if c["op"] == "group_norm_fwd":
        x = by_group(s["x"].double())
        var, mean = torch.var_mean(x, 2, correction=0, keepdim=True)
        rstd = (var + EPS).pow(-0.5)
        z = (x - mean) * rstd * gamma + beta
        y = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[c["act"]](z)
        out = {"y": flat(y)}
        if c["train"]:
            out["mean"], out["rstd"] = mean[..., 0], rstd[..., 0]
        if c["kept"]:
            v = s["x"].double()
            scale = torch.exp2(torch.ceil(torch.log2(v.unflatten(2, (ch // 32, 32)).abs().max(3).values / 448.0)).clamp(-127.0, 127.0))
            out["kept"], out["scales"] = _round_e4m3(v / scale.repeat_interleave(32, 2)), scale
        return out
    x = s["x"].double()
    if c["kept"]:
        x = x * torch.exp2(s["scales"].view(torch.uint8).double() - 127.0).repeat_interleave(32, 2)
    rstd = s["rstd"].double()[..., None]
    h = (by_group(x) - s["mean"].double()[..., None]) * rstd
    z = gamma * h + beta
    sig = torch.sigmoid(z)
    slope = {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(), "silu": lambda: sig + z * sig * (1 - sig),
             "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[c["act"]]()
    dz = by_group(s["dy"].double()) * slope
    u = dz * gamma
    dx = rstd * u - rstd * (u.sum(2, keepdim=True) + h * (u * h).sum(2, keepdim=True)) / u.shape[2]
    return {"dx": flat(dx), "dgamma": flat(dz * h).sum((0, 1)), "dbeta": flat(dz).sum((0, 1))}
