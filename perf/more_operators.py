"""Cases of the decoder layer's steps around its FP8 products, and their plain forms.

Two operators stand here, each with its backward pass:

* norms of queries and keys for each head with the rotation by positions in the same pass: what
  happens to the packed result of the query/key/value projection before attention. Positions have
  one axis (text) or several (time, height, width), each with its share of the rotated pairs.
* the FP8 product with bias, activation and residual in its epilogue: one linear layer's forward on
  E4M3 codes and block scales. The activation may be gated: the weight's first half of rows makes
  the gate, its second half what the gate multiplies. For training the value before the activation
  is kept, and the activation's backward makes its gradient and the bias's.

``own`` False computes them with elementary torch operations in 32 bits; True calls the framework.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------------------------------- cases
def _rope(name, op, tokens, heads_q, heads_k, head_dim, rotary=1.0, axes=1, order="blocked", interleaved=False,
          norm=True, wtype="bf16", offset=False, scale=1.0, base=1e6, far=40000, packed=True):
    pairs = max(axes, int(head_dim * rotary) // 2)
    rest = pairs - 2 * (pairs // 3) if axes == 3 else pairs - (axes - 1) * (pairs // axes)
    sections = [rest] + [pairs // axes] * (axes - 1)
    return {"name": name, "op": op, "tokens": tokens, "heads_q": heads_q, "heads_k": heads_k, "head_dim": head_dim,
            "pairs": pairs, "axes": axes, "sections": ",".join(map(str, sections)), "order": order,
            "interleaved": interleaved, "norm": norm, "wtype": wtype, "offset": offset, "scale": scale, "base": base,
            "far": far, "packed": packed}


def _product(name, m, n, k, act="none", gated=False, bias="none", residual=False, save_z=False):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "act": act, "gated": gated, "bias": bias,
            "residual": residual, "save_z": save_z}


def _act_bwd(name, rows, cols, act, gated=False, bias=False):
    return {"name": name, "op": "act_bwd", "rows": rows, "cols": cols, "act": act, "gated": gated, "bias": bias}


def listed():
    return [
        # one token of a decoding step, 16 query and 8 key heads of 128: latency
        _rope("rope_token", "rope", 1, 16, 8, 128),
        # a micro-batch of 2 x 4096 tokens of the same layer
        _rope("rope_tokens8192", "rope", 8192, 16, 8, 128),
        # video patches: three axes dealt in turn over neighbouring pairs, a ragged batch, odd heads, half rotated
        _rope("rope_video_odd", "rope", 1003, 14, 2, 80, rotary=0.5, axes=3, order="cycled", interleaved=True,
              wtype="f32", offset=True, scale=1.1, base=1e4),
        # backward of the micro-batch
        _rope("rope_bwd_tokens8192", "rope_bwd", 8192, 16, 8, 128),
        # backward of a short ragged image and text batch, one shared key head, far positions
        _rope("rope_bwd_image", "rope_bwd", 1537, 7, 1, 96, axes=3, wtype="f32", far=1000000, packed=False),
        # one token through the gated gate+up projection: latency
        _product("product_token", 1, 12288, 2048, "silu", gated=True),
        # a few sequences' tokens through the down projection onto the residual stream
        _product("product_tokens33", 33, 2048, 6144, bias="f32", residual=True),
        # the micro-batch through the gated gate+up projection, keeping what the backward needs
        _product("product_gateup8192", 8192, 12288, 2048, "silu", gated=True, save_z=True),
        # the micro-batch through the down projection onto the residual stream
        _product("product_down8192", 8192, 2048, 6144, bias="bf16", residual=True),
        # a ragged batch through a plain layer of a smaller model
        _product("product_odd", 1003, 1000, 1536, "gelu", bias="bf16"),
        # backward of the gated activation of the micro-batch
        _act_bwd("act_bwd_gated8192", 8192, 6144, "silu", gated=True),
        # backward of an activation and a bias over a ragged batch of odd width
        _act_bwd("act_bwd_odd", 1003, 5407, "gelu_tanh", bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]


def draw(rng):
    op = rng.choice(["rope", "rope", "rope_bwd", "rope_bwd", "product", "product", "product", "act_bwd", "act_bwd"])
    if op == "product":
        gated = rng.random() < 0.4
        m, k = _log_int(rng, 1, 8192), 128 * _log_int(rng, 1, 48)
        n = 128 * _log_int(rng, 1, 96) if gated else _log_int(rng, 16, 12288)
        if rng.random() < 0.5:
            n = -(-n // 128) * 128
        act = rng.choice(ACTS[1:] if gated else ACTS)
        c = _product("", min(m, int(2e11 // (n * k))), n, k, act, gated, rng.choice(["none", "bf16", "f32"]),
                     rng.random() < 0.5, rng.random() < 0.3)
    elif op == "act_bwd":
        gated = rng.random() < 0.5
        cols = _log_int(rng, 16, 6144)
        cols = cols if rng.random() < 0.4 else -(-cols // 8) * 8
        c = _act_bwd("", _log_int(rng, 1, 8192), cols, rng.choice(ACTS[1:]), gated, rng.random() < 0.5)
    else:
        dim = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128, 160, 192, 256, 2 * rng.randint(8, 128)])
        kv = rng.choice([1, 1, 2, 4, 5, 8])
        q = kv * rng.choice([1, 2, 4, 7, 8])
        axes = rng.choice([1, 1, 2, 3, 3])
        tokens = min(_log_int(rng, 1, 8192), int(2.5e7 // ((q + kv) * dim)))
        c = _rope("", op, tokens, q, kv, dim, rng.choice([1.0, 1.0, 0.5, 0.25]), axes,
                  rng.choice(["blocked", "cycled"]) if axes > 1 else "blocked", rng.random() < 0.3,
                  rng.random() < 0.8, rng.choice(["bf16", "f32"]), rng.random() < 0.3, rng.choice([1.0, 1.0, 1.25]),
                  rng.choice([1e4, 5e5, 1e6]), rng.choice([0, 4096, 40000, 1000000]), rng.random() < 0.7)
    c.pop("name")
    return c


# --------------------------------------------------------------------------------------- inputs
def _codes(x, rows):
    """E4M3 codes and power-of-two scales of a matrix: one scale for each 1 x 128 or 128 x 128 block."""
    n, k = x.shape
    full = -(-n // rows) * rows
    v = torch.zeros(full, k, device=x.device) if full != n else x
    if full != n:
        v[:n] = x
    v = v.view(full // rows, rows, k // 128, 128)
    man, ex = torch.frexp(v.abs().amax((1, 3), keepdim=True))
    e = torch.where(man == 0, torch.zeros_like(ex), torch.clamp(ex - 9 + (man > 0.875).int(), min=-126))
    s = torch.ldexp(torch.ones_like(man), e)
    q = (v / s).to(torch.float8_e4m3fn).view(full, k)[:n]
    return q.contiguous().view(torch.uint8), s.view(full // rows, k // 128)


def _sections(case):
    return [int(v) for v in case["sections"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    bf = torch.bfloat16
    st = {"case": case}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        wide = 1.0 + 20.0 * (torch.rand(k, generator=g, device=DEV) < 0.002).float()  # a few large channels
        qx, sx = _codes((rnd(m, k) * wide).to(bf).float(), 1)
        st["qx"], st["sx"] = qx, sx.t().contiguous()
        st["qw"], st["sw"] = _codes((rnd(n, k) / k ** 0.5).to(bf).float(), 128)
        no = n // 2 if case["gated"] else n
        st["bias"] = None if case["bias"] == "none" else (0.2 * rnd(n)).to(torch.float32 if case["bias"] == "f32" else bf)
        st["residual"] = (2.0 * rnd(m, no)).to(bf) if case["residual"] else None
        return st
    if case["op"] == "act_bwd":
        rows, cols = case["rows"], case["cols"]
        st["z"] = rnd(rows, 2 * cols if case["gated"] else cols).to(bf)
        st["dd"] = (1e-3 * rnd(rows, cols)).to(bf)
        return st
    t, hq, hk, dim = case["tokens"], case["heads_q"], case["heads_k"], case["head_dim"]
    wt = torch.float32 if case["wtype"] == "f32" else bf
    if case["packed"]:  # the projection's result holds queries, keys and values beside one another
        qkv = (3.0 * rnd(t, (hq + 2 * hk) * dim)).to(bf)
        st["q"] = qkv[:, : hq * dim].unflatten(1, (hq, dim))
        st["k"] = qkv[:, hq * dim: (hq + hk) * dim].unflatten(1, (hk, dim))
    else:
        st["q"], st["k"] = (3.0 * rnd(t, hq, dim)).to(bf), (3.0 * rnd(t, hk, dim)).to(bf)
    base = 0.0 if case["offset"] else 1.0
    st["w_q"] = (base + 0.2 * rnd(dim)).to(wt) if case["norm"] else None
    st["w_k"] = (base + 0.2 * rnd(dim)).to(wt) if case["norm"] else None
    pairs = case["pairs"]
    st["inv_freq"] = (float(case["base"]) ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(DEV)
    start = int(torch.randint(0, case["far"] + 1, (1,), generator=g, device=DEV))
    p = torch.arange(t, device=DEV)
    side = max(2, int(t ** 0.4))
    grid = [p // (side * side), p // side % side, p % side]
    st["positions"] = p + start if case["axes"] == 1 else torch.stack([start + v for v in grid[: case["axes"]]])
    if case["op"] == "rope_bwd":
        st["dq"], st["dk"] = (1e-2 * rnd(t, hq, dim)).to(bf), (1e-2 * rnd(t, hk, dim)).to(bf)
    return st


# ------------------------------------------------------------------------------------ own calls
def _own(st):
    import fp8_block_scaled_pf8_amd as pf8

    c = st["case"]
    act = None if c.get("act") == "none" else c.get("act")
    if c["op"] == "product":
        r = pf8.fprop_act(st["qx"], st["sx"], st["qw"], st["sw"], bias=st["bias"], activation=act, gated=c["gated"],
                          residual=st["residual"], save_z=c["save_z"])
        return {"d": r[0], "z": r[1]} if c["save_z"] else {"d": r}
    if c["op"] == "act_bwd":
        r = pf8.act_backward(st["dd"], st["z"], act, gated=c["gated"], bias_grad=c["bias"])
        return {"dz": r.dz, "dbias": r.dbias}
    kw = dict(w_q=st["w_q"], w_k=st["w_k"], sections=_sections(c) if c["axes"] > 1 else None, section_order=c["order"],
              interleaved=c["interleaved"], rotary_scale=c["scale"], eps=EPS, unit_offset=c["offset"])
    if c["op"] == "rope":
        q, k = pf8.qk_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], **kw)
        return {"q": q, "k": k}
    d = pf8.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["positions"], st["inv_freq"], **kw)
    return {"dq": d.dq, "dk": d.dk, "dw_q": d.dw_q, "dw_k": d.dw_k}


# ---------------------------------------------------------------------------------- plain forms
def _axis_of_pair(case, device):
    """The position axis of each rotated pair: runs of pairs, or the axes in turn with the rest left to the first."""
    sec, pairs = _sections(case), case["pairs"]
    if case["order"] == "blocked":
        axis = [a for a, s in enumerate(sec) for _ in range(s)]
    else:
        axis = [i % len(sec) if i < len(sec) * sec[i % len(sec)] else 0 for i in range(pairs)]
    return torch.tensor(axis, device=device)


def _cos_sin(st):
    c, pos = st["case"], st["positions"]
    if c["axes"] > 1:
        pos = pos[_axis_of_pair(c, pos.device)].t()
    else:
        pos = pos[:, None]
    angle = pos.double() * st["inv_freq"].double()  # far positions' angles need 64 bits
    return (torch.cos(angle) * c["scale"]).float()[:, None], (torch.sin(angle) * c["scale"]).float()[:, None]


def _pairs(x, case):
    """First and second elements of the rotated pairs, and the rest."""
    r = 2 * case["pairs"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., : r // 2], x[..., r // 2: r], x[..., r:]


def _unpairs(a, b, rest, case):
    if case["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _rotate(x, cos, sin, case):
    a, b, rest = _pairs(x, case)
    return _unpairs(a * cos - b * sin, a * sin + b * cos, rest, case)


def _rope_plain(st):
    c = st["case"]
    cos, sin = _cos_sin(st)
    off = 1.0 if c["offset"] else 0.0
    out = {}
    for n in ("q", "k"):
        x, w = st[n].float(), st["w_" + n]
        if w is not None:
            rho = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if c["op"] == "rope":
            y = x if w is None else x * rho * (w.float() + off)
            out[n] = _rotate(y, cos, sin, c).to(torch.bfloat16)
            continue
        d = _rotate(st["d" + n].float(), cos, -sin, c)  # the rotation's transpose
        dw = None
        if w is not None:
            xn = x * rho
            dw = (d * xn).sum((0, 1))
            t = d * (w.float() + off)
            d = rho * (t - xn * (t * xn).mean(-1, keepdim=True))
        out["d" + n], out["dw_" + n] = d.to(torch.bfloat16), dw
    return {k: out[k] for k in (("q", "k") if c["op"] == "rope" else ("dq", "dk", "dw_q", "dw_k"))}


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu2":
        return torch.clamp(z, min=0) ** 2
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "relu2":
        return 2 * torch.clamp(z, min=0)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi)
    t = torch.tanh(u * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * u * (1 + 3 * 0.044715 * z * z)


def _values(q, s, rows):
    """The values that codes and their blocks' scales stand for."""
    n, k = q.shape
    s = s.repeat_interleave(rows, 0)[:n] if rows > 1 else s
    return (q.view(torch.float8_e4m3fn).float().view(n, k // 128, 128) * s.unsqueeze(2)).view(n, k)


def _plain(st):
    c = st["case"]
    low = lambda t: t.to(torch.bfloat16)  # noqa: E731
    if c["op"] in ("rope", "rope_bwd"):
        return _rope_plain(st)
    if c["op"] == "product":
        z = torch.matmul(_values(st["qx"], st["sx"].t(), 1), _values(st["qw"], st["sw"], 128).t())
        z = z if st["bias"] is None else z + st["bias"].float()
        half = c["n"] // 2
        d = _act(z[:, :half], c["act"]) * z[:, half:] if c["gated"] else _act(z, c["act"])
        d = low(d if st["residual"] is None else d + st["residual"].float())
        return {"d": d, "z": low(z)} if c["save_z"] else {"d": d}
    dd, z = st["dd"].float(), st["z"].float()
    if c["gated"]:
        g, u = z[:, : c["cols"]], z[:, c["cols"]:]
        dz = torch.cat([dd * u * _slope(g, c["act"]), dd * _act(g, c["act"])], 1)
    else:
        dz = dd * _slope(z, c["act"])
    return {"dz": low(dz), "dbias": dz.sum(0) if c["bias"] else None}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- the work
def work(case):
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        no = n // 2 if case["gated"] else n
        read = m * k + 4 * m * k // 128 + n * k + 4 * (-(-n // 128)) * k // 128
        read += {"none": 0, "bf16": 2 * n, "f32": 4 * n}[case["bias"]] + (2 * m * no if case["residual"] else 0)
        return {"bytes": read + 2 * m * no + (2 * m * n if case["save_z"] else 0), "flops": 2 * m * n * k}
    if case["op"] == "act_bwd":
        n = case["rows"] * case["cols"]
        wide = 2 if case["gated"] else 1
        return {"bytes": n * (2 + 4 * wide) + (4 * case["cols"] * wide if case["bias"] else 0), "flops": 15 * n * wide}
    n = case["tokens"] * (case["heads_q"] + case["heads_k"]) * case["head_dim"]
    small = 8 * case["axes"] * case["tokens"] + 4 * case["pairs"]
    weights = 2 * case["head_dim"] * (4 if case["wtype"] == "f32" else 2) if case["norm"] else 0
    if case["op"] == "rope":
        return {"bytes": 4 * n + small + weights, "flops": 7 * n}
    return {"bytes": 6 * n + small + weights + (8 * case["head_dim"] if case["norm"] else 0), "flops": 15 * n}


# ------------------------------------------------------------------------------- 64-bit results
def _act64(z, act):
    F = torch.nn.functional
    return {"none": lambda v: v, "relu": torch.relu, "relu2": lambda v: torch.relu(v) * torch.relu(v), "silu": F.silu,
            "gelu": F.gelu, "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[act](z)


def exact(case, seed):
    """What run() returns, from the definitions in float64: rotations as products of complex numbers,
    gradients by automatic differentiation."""
    st = prepare(case, seed)
    D = lambda t: None if t is None else t.to(torch.float64)  # noqa: E731
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x = D(st["qx"].view(torch.float8_e4m3fn).float())
        w = D(st["qw"].view(torch.float8_e4m3fn).float())
        col = torch.arange(k, device=DEV) // 128
        x *= D(st["sx"])[col].t()
        w *= D(st["sw"])[torch.arange(n, device=DEV) // 128][:, col]
        z = torch.mm(x, w.t())
        if st["bias"] is not None:
            z += D(st["bias"])
        d = _act64(z[:, : n // 2], case["act"]) * z[:, n // 2:] if case["gated"] else _act64(z, case["act"])
        d = d if st["residual"] is None else d + D(st["residual"])
        return {"d": d, "z": z} if case["save_z"] else {"d": d}
    if case["op"] == "act_bwd":
        z = D(st["z"]).requires_grad_()
        with torch.enable_grad():
            n = case["cols"]
            d = _act64(z[:, :n], case["act"]) * z[:, n:] if case["gated"] else _act64(z, case["act"])
            (dz,) = torch.autograd.grad(d, z, D(st["dd"]))
        return {"dz": dz, "dbias": dz.sum(0) if case["bias"] else None}
    sec, pairs, r = _sections(case), case["pairs"], 2 * case["pairs"]
    pos = st["positions"].reshape(case["axes"], -1).to(torch.float64)
    angle = torch.empty(case["tokens"], pairs, dtype=torch.float64, device=DEV)
    first = 0
    for a, s in enumerate(sec):
        if case["order"] == "blocked":
            at = slice(first, first + s)
            first += s
        else:
            at = slice(a, len(sec) * s, len(sec)) if a else slice(0, pairs)  # the first axis keeps what others leave
        angle[:, at] = pos[a][:, None] * st["inv_freq"].double()[at]
    turn = torch.polar(torch.full_like(angle, case["scale"]), angle)[:, None]
    one = 1.0 if case["offset"] else 0.0
    out = {}
    for n in ("q", "k"):
        x, w = D(st[n]).requires_grad_(), D(st["w_" + n])
        w = None if w is None else w.requires_grad_()
        with torch.enable_grad():
            y = x if w is None else x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * (w + one)
            p = y[..., :r]
            p = p.unflatten(-1, (pairs, 2)) if case["interleaved"] else p.unflatten(-1, (2, pairs)).transpose(-2, -1)
            p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * turn)
            p = p.flatten(-2) if case["interleaved"] else p.transpose(-2, -1).flatten(-2)
            y = torch.cat([p, y[..., r:]], -1)
            if case["op"] == "rope":
                out[n] = y.detach()
                continue
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], D(st["d" + n]))
        out["d" + n], out["dw_" + n] = grads[0], None if w is None else grads[1]
    return {k: out[k] for k in (("q", "k") if case["op"] == "rope" else ("dq", "dk", "dw_q", "dw_k"))}
