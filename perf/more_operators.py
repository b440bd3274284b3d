"""Measured cases of a transformer's feed-forward half as a rank trains it:
the root-mean-square norm with the residual's addition, 16-bit linear layers
with bias, activation and residual, the gated block, and activations kept in
8 bits for the backward pass.

`run` computes a case with the library's entry points where `own` is true,
and otherwise in plain torch operations in 32 bits, rounded once at the end.
`exact` is the same in 64 bits, from the definitions.

The definitions, T() rounding to the case's type:

  norm     s = T(x + r), which is kept as the next residual; rstd = 1 / sqrt(mean
           of s^2 along the row + eps); y = s rstd w.  Backward: with n = s rstd,
           dx = ds + rstd (w dy - n mean(w dy n)), the gradient of x and of r;
           dw = sum over rows of dy n
  linear   z = x W^T + b, y = act(z) + r.  Backward: dz = dy act'(T(z)),
           dx = dz W, dW = dz^T x, db = sum over rows of dz
  gated    g = x Wg^T, u = x Wu^T, h = act(g) u.  Backward, at the kept
           T(g) and T(u): dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu,
           dWg = dg^T x, dWu = du^T x
  pack8    blocks of 32 along a row share the power of two 2^e, e the smallest
           with max|x| 2^-e <= 448 (not below -127); an element is x 2^-e rounded to the
           nearest e4m3 value (3 bits after the leading one, exponents from -6 on
           and subnormals below), ties to the even one
  keep8    gated or linear with what is kept for the backward pass (x, and z or
           g and u before any rounding) packed to 8 bits, whose values the
           backward pass takes in place of x, T(z), T(g) and T(u)

act is SiLU (v / (1 + exp(-v))), GELU (v times the normal distribution
function), its form with tanh, ReLU or none.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}
ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
EPS = 1e-5


def listed():
    return [
        # the next token of 48 sequences of GPT-2 small's width: latency
        dict(name="norm_token", op="norm", rows=48, dim=768, dtype="bf16", residual=True,
             q=False, train=False),
        # a ragged prompt at GPT-2 XL's width, the output in 8 bits only
        dict(name="norm_prompt8", op="norm", rows=333, dim=1600, dtype="f16", residual=True,
             q=True, train=False),
        # 16 sequences of 1024 at Llama-7B's width, both directions
        dict(name="norm_train", op="norm", rows=16 * 1024, dim=4096, dtype="bf16", residual=True,
             q=False, train=True),
        # one token through GPT-2 XL's MLP weight: latency, the weight's bytes
        dict(name="linear_token", op="linear", m=1, n=6400, k=1600, dtype="f16", bias=True,
             act="gelu_tanh", residual=False, train=False, keep8=False),
        # 100 rows of the small MLP's first layer (64 to 256), both directions: latency
        dict(name="linear_small", op="linear", m=100, n=256, k=64, dtype="bf16", bias=True,
             act="gelu", residual=False, train=True, keep8=False),
        # a ragged prompt through GPT-2 XL's second MLP weight, onto the residual
        dict(name="linear_prompt", op="linear", m=333, n=1600, k=6400, dtype="f16", bias=True,
             act="none", residual=True, train=False, keep8=False),
        # 8 sequences of 1024 through GPT-2 XL's first MLP weight, both directions
        dict(name="linear_train", op="linear", m=8 * 1024, n=6400, k=1600, dtype="bf16",
             bias=True, act="gelu_tanh", residual=False, train=True, keep8=False),
        # one token through Llama-7B's gated block: latency, the weights' bytes
        dict(name="gated_token", op="gated", m=1, n=11008, k=4096, dtype="bf16", act="silu",
             train=False, keep8=False),
        # a ragged prompt through the same
        dict(name="gated_prompt", op="gated", m=77, n=11008, k=4096, dtype="bf16", act="silu",
             train=False, keep8=False),
        # 8 sequences of 1024 through the same, both directions
        dict(name="gated_train", op="gated", m=8 * 1024, n=11008, k=4096, dtype="bf16",
             act="silu", train=True, keep8=False),
        # fp32 activations of an odd width, kept and taken back
        dict(name="pack_odd", op="pack", rows=1000, cols=1601, dtype="f32"),
        # two sequences of 1000 through the gated block, kept in 8 bits
        dict(name="gated_train8", op="gated", m=2000, n=11008, k=4096, dtype="bf16", act="silu",
             train=True, keep8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "gated", "gated", "pack"])
    low = rng.choice(["bf16", "f16"])
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 16384), dim=_log(rng, 64, 8192),
                    dtype=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.7,
                    q=rng.random() < 0.4, train=rng.random() < 0.6)
    if op == "pack":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 32, 8192),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    train = rng.random() < 0.6
    keep8 = train and rng.random() < 0.4
    # half of the widths whole eights, as models have them
    step = rng.choice([1, 8])
    n, k = (max(64, _log(rng, 64, hi) // step * step) for hi in (8192, 4096))
    m = _log(rng, 1, 8000)
    if op == "gated":
        return dict(op=op, m=m, n=n, k=k, dtype=low, act=rng.choice(["silu", "gelu_tanh"]),
                    train=train, keep8=keep8)
    return dict(op=op, m=m, n=n, k=k, dtype=low, bias=rng.random() < 0.6,
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                residual=rng.random() < 0.4, train=train, keep8=keep8)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)


def _normal(g, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _activations(g, rows, cols, dtype, sigma=1.0):
    """Normal values with a few columns much larger than the others, as the
    activations of large models have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * sigma
    big = torch.rand(cols, generator=g, device="cuda") < 0.01
    return torch.where(big, x * 12.0, x).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case, "stream": torch.cuda.current_stream().cuda_stream}
    t = DT[case["dtype"]]

    def room(*shape, dtype=t):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "norm":
        R, C = case["rows"], case["dim"]
        s["x"] = _activations(g, R, C, t)
        s["residual"] = _activations(g, R, C, t) if case["residual"] else None
        s["w"] = (1.0 + 0.1 * torch.randn(C, generator=g, device="cuda")).to(t)
        s["sum"] = room(R, C) if case["residual"] else None
        s["y"], s["rstd"] = room(R, C), room(R, dtype=torch.float32)
        s["values"] = room(R, C, dtype=torch.bfloat16)
        if case["train"]:
            s["dy"], s["ds"] = _normal(g, (R, C), t, 1e-2), _normal(g, (R, C), t, 1e-2)
            s["dx"], s["dw"] = room(R, C), room(C)
    elif op == "pack":
        R, C = case["rows"], case["cols"]
        s["x"] = _activations(g, R, C, t)
        s["values"] = room(R, C)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _activations(g, m, k, t)
        gated = op == "gated"
        for name in (("wg", "wu") if gated else ("w",)):
            s[name] = _normal(g, (n, k), t, 1.0 / math.sqrt(k))
            s["d" + name] = room(n, k)
        if not gated:
            s["b"] = _normal(g, (n,), t, 0.1) if case["bias"] else None
            s["residual"] = _normal(g, (m, n), t) if case["residual"] else None
        s["y"] = room(m, n)
        if case["train"]:
            s["dy"] = _normal(g, (m, n), t, 1e-1)
            s["dx"] = room(m, k)
            if not case["keep8"]:
                s["kept"] = [room(m, n) for _ in range(2 if gated else 1)]
            s["dz"] = [room(m, n) for _ in range(2 if gated else 1)]
            s["x8"] = room(m, k) if case["keep8"] else None
            s["db"] = room(n)
    return s


# ---------------------------------------------------------------- the passes

def run(state):
    return _own(state) if own else _plain(state)


def _bytes(s, name, count):
    """A buffer of so many bytes, made at the first pass."""
    if name not in s:
        s[name] = torch.empty(max(count, 16), dtype=torch.uint8, device="cuda")
    return s[name]


def _own(s):
    import zero_sharded_optimizer_step_gb300 as z
    c, st = s["case"], s["stream"]
    op, dt = c["op"], CODE[c["dtype"]]
    if op == "norm":
        R, C = c["rows"], c["dim"]
        q = _bytes(s, "q", z.zero_pack8_bytes(R, C)) if c["q"] else None
        y = None if c["q"] else s["y"]
        z.zero_rms_norm(s["x"], C, s["residual"], C, s["w"], dt, R, C, EPS, s["sum"], C, y, C, q,
                        s["rstd"], st)
        out = {"y": y}
        if c["q"]:
            z.zero_unpack8(q, R, C, s["values"], CODE["bf16"], C, st)
            out = {"y": s["values"]}
        if c["residual"]:
            out["sum"] = s["sum"]
        if c["train"]:
            need = z.zero_rms_norm_grad_workspace(R, C)
            z.zero_rms_norm_grad(s["dy"], C, s["ds"], C, s["sum"] if c["residual"] else s["x"], C,
                                 s["w"], s["rstd"], dt, R, C, s["dx"], C, s["dw"], dt, False,
                                 _bytes(s, "ws", need), need, st)
            out["dx"], out["dw"] = s["dx"], s["dw"]
        return out
    if op == "pack":
        R, C = c["rows"], c["cols"]
        q = _bytes(s, "q", z.zero_pack8_bytes(R, C))
        z.zero_pack8(s["x"], dt, R, C, C, q, st)
        z.zero_unpack8(q, R, C, s["values"], dt, C, st)
        return s["values"]
    m, n, k, act = c["m"], c["n"], c["k"], ACT[c["act"]]
    x, keep8, gated = s["x"], c["keep8"], op == "gated"

    def product(out, rows, cols, depth, a, a_cols, b, b_cols, a2=None, b2=None, bias=None,
                activation=0, residual=None, kept=None, kept_q=None):
        sa, sb = rows if a_cols else depth, cols if b_cols else depth
        need = z.zero_matmul_workspace(a, a_cols, sa, b, b_cols, sb, a2, sa, b2, sb, rows, cols,
                                       depth)
        ws = _bytes(s, ("ws", need), need) if need else None
        z.zero_matmul(a, a_cols, sa, b, b_cols, sb, a2, sa, b2, sb, dt, rows, cols, depth, bias,
                      activation, residual, cols, kept, cols, kept_q, out, dt, cols, False, ws,
                      need, st)

    kept, kept_q = [None, None], [None, None]
    if c["train"] and keep8:
        kept_q = [_bytes(s, "kept%d" % i, z.zero_pack8_bytes(m, n)) for i in (0, 1)]
        xq = _bytes(s, "xq", z.zero_pack8_bytes(m, k))
        z.zero_pack8(x, dt, m, k, k, xq, st)
    elif c["train"]:
        kept = s["kept"] + [None]
    if gated:
        need = z.zero_gated_workspace(x, k, s["wg"], k, s["wu"], k, m, n, k)
        ws = _bytes(s, "ws_gated", need) if need else None
        z.zero_gated(x, k, s["wg"], k, s["wu"], k, dt, m, n, k, act, kept[0], kept[1], n,
                     kept_q[0], kept_q[1], s["y"], n, ws, need, st)
    else:
        linear = act == 0               # its gradient needs nothing kept
        product(s["y"], m, n, k, x, False, s["w"], False, bias=s["b"], activation=act,
                residual=s["residual"], kept=None if linear else kept[0],
                kept_q=None if linear else kept_q[0])
    if not c["train"]:
        return {"y": s["y"]}
    if keep8:
        z.zero_unpack8(xq, m, k, s["x8"], dt, k, st)
        x = s["x8"]
    if gated:
        dg, du = s["dz"]
        z.zero_gated_grad(s["dy"], n, kept[0], kept[1], n, kept_q[0], kept_q[1], act, dt, m, n,
                          dg, du, n, None, n, st)
        product(s["dx"], m, k, n, dg, False, s["wg"], True, du, s["wu"])
        product(s["dwg"], n, k, m, dg, True, x, True)
        product(s["dwu"], n, k, m, du, True, x, True)
        return {"y": s["y"], "dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"]}
    dz = s["dy"] if act == 0 else s["dz"][0]
    out = {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    if act or c["bias"]:
        need = z.zero_activation_grad_workspace(m, n)
        z.zero_activation_grad(s["dy"], n, None if act == 0 else kept[0], n,
                               None if act == 0 else kept_q[0], act, dt, m, n,
                               None if act == 0 else dz, n, s["db"] if c["bias"] else None, dt,
                               False, _bytes(s, "ws_bias", need), need, st)
        if c["bias"]:
            out["db"] = s["db"]
    product(s["dx"], m, k, n, dz, False, s["w"], True)
    product(s["dw"], n, k, m, dz, True, x, True)
    return out


def _act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v.clamp(min=0.0) if act == "relu" else v


def _act_grad(v, act):
    if act == "silu":
        p = torch.sigmoid(v)
        return p * (1.0 + v * (1.0 - p))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
                + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * (1.0 + th) + 0.5 * v * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * v * v)
    return (v > 0).to(v.dtype) if act == "relu" else torch.ones_like(v)


def _plain_pack(x):
    """The values an fp32 matrix is packed to."""
    R, C = x.shape
    full = torch.nn.functional.pad(x, (0, -C % 32)).reshape(R, -1, 32)
    top = full.abs().amax(2).view(torch.int32)
    e = ((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000).int()).clamp_(min=0)
    down = (254 - e << 23).view(torch.float32)[:, :, None]
    up = torch.where(e > 0, e << 23, 1 << 22).int().view(torch.float32)[:, :, None]
    codes = (full * down).to(torch.float8_e4m3fn)
    return (codes.float() * up).reshape(R, -1)[:, :C]


def _plain(s):
    c = s["case"]
    op, t = c["op"], DT[c["dtype"]]
    if op == "pack":
        s["values"].copy_(_plain_pack(s["x"].float()))
        return s["values"]
    if op == "norm":
        out = {"y": s["values"] if c["q"] else s["y"]}
        x = s["x"].float()
        if c["residual"]:
            out["sum"] = s["sum"].copy_(x + s["residual"].float())
            x = s["sum"].float()
        w = s["w"].float()
        rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        y = x * rstd * w
        out["y"].copy_(_plain_pack(y) if c["q"] else y)
        if c["train"]:
            dy, n = s["dy"].float(), x * rstd
            wdy = dy * w
            out["dx"] = s["dx"].copy_(
                s["ds"].float() + rstd * (wdy - n * (wdy * n).mean(1, keepdim=True)))
            out["dw"] = s["dw"].copy_((dy * n).sum(0))
        return out
    act, x = c["act"], s["x"].float()
    if op == "gated":
        wg, wu = s["wg"].float(), s["wu"].float()
        g, u = x @ wg.t(), x @ wu.t()
        s["y"].copy_(_act(g, act) * u)
        if not c["train"]:
            return {"y": s["y"]}
        if c["keep8"]:
            x, g, u = _plain_pack(x), _plain_pack(g), _plain_pack(u)
        else:
            g, u = g.to(t).float(), u.to(t).float()
        dy = s["dy"].float()
        dg, du = dy * u * _act_grad(g, act), dy * _act(g, act)
        s["dx"].copy_(dg @ wg + du @ wu)
        s["dwg"].copy_(dg.t() @ x)
        s["dwu"].copy_(du.t() @ x)
        return {"y": s["y"], "dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"]}
    w = s["w"].float()
    v = x @ w.t()
    if c["bias"]:
        v += s["b"].float()
    y = _act(v, act)
    s["y"].copy_(y + s["residual"].float() if c["residual"] else y)
    if not c["train"]:
        return {"y": s["y"]}
    if c["keep8"]:
        x, v = _plain_pack(x), _plain_pack(v)
    else:
        v = v.to(t).float()
    dv = s["dy"].float() * _act_grad(v, act)
    s["dx"].copy_(dv @ w)
    s["dw"].copy_(dv.t() @ x)
    out = {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    if c["bias"]:
        out["db"] = s["db"].copy_(dv.sum(0))
    return out


# ------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    es = torch.finfo(DT[case["dtype"]]).bits // 8
    if op == "pack":
        e = case["rows"] * case["cols"]
        return {"bytes": int(e * (2 * es + 2 * (1 + 1 / 32))), "flops": 3 * e}
    if op == "norm":
        e = case["rows"] * case["dim"]
        b = e * es * (3 if case["residual"] else 1) + (e * 4 if case["q"] else e * es)
        if case["train"]:
            b += 4 * e * es                  # dy, ds and the sum again; dx
        return {"bytes": b, "flops": e * (14 if case["train"] else 5)}
    m, n, k = case["m"], case["n"], case["k"]
    w = 2 if op == "gated" else 1
    b = (m * k + w * n * k + m * n) * es
    if op == "linear" and case["residual"]:
        b += m * n * es
    if case["train"]:
        b += (m * n + m * k + w * n * k) * es
    return {"bytes": b, "flops": 2 * w * m * n * k * (3 if case["train"] else 1)}


# ------------------------------------------------- the definitions in 64 bits

def _power(e):
    """2^e for whole e, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_pack(x):
    """The values a float64 matrix is packed to: the element's own power of two
    gives its spacing, and the rounding to a whole number of spacings is to
    the even one."""
    R, C = x.shape
    out = torch.empty_like(x)
    for lo in range(0, R, 1024):
        part = x[lo:lo + 1024]
        b = torch.nn.functional.pad(part, (0, -C % 32)).reshape(part.shape[0], -1, 32)
        frac, ex = torch.frexp(b.abs().amax(2, keepdim=True))     # frac in [0.5, 1)
        e = torch.where(frac > 0, ex - 9 + (frac > 0.875).int(), -127).clamp(min=-127)
        unit = _power(e)
        v = b / unit
        step = _power((torch.frexp(v).exponent - 1).clamp(min=-6) - 3)
        out[lo:lo + 1024] = (torch.round(v / step) * step * unit).reshape(
            part.shape[0], -1)[:, :C]
    return out


def _exact_act(v, act):
    """act(v) and act'(v)."""
    if act == "silu":
        e = torch.exp(-v.abs())
        p = torch.where(v >= 0, 1.0, e) / (1.0 + e)
        return v * p, p + v * p * (1.0 - p)
    if act == "gelu":
        phi = torch.special.ndtr(v)
        return v * phi, phi + v * torch.exp(-v * v / 2) * 0.3989422804014327
    if act == "gelu_tanh":
        a = 0.7978845608028654
        w = 2.0 * a * (v + 0.044715 * v * v * v)       # (1 + tanh(w / 2)) / 2 = sigmoid(w)
        p = torch.sigmoid(w)
        return v * p, p + v * p * torch.sigmoid(-w) * 2.0 * a * (1.0 + 0.134145 * v * v)
    if act == "relu":
        return torch.where(v > 0, v, 0.0), torch.where(v > 0, 1.0, 0.0).to(v.dtype)
    return v, torch.ones_like(v)


def exact(case, seed):
    s = prepare(case, seed)
    op, t = case["op"], DT[case["dtype"]]
    if op == "pack":
        return _exact_pack(s["x"].double())
    if op == "norm":
        x, out = s["x"].double(), {}
        if case["residual"]:
            x = (x + s["residual"].double()).to(t).double()
            out["sum"] = x
        w = s["w"].double()
        rstd = (torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / case["dim"] + EPS) ** -0.5
        n = x * rstd
        out["y"] = _exact_pack(n * w) if case["q"] else n * w
        if case["train"]:
            dy = s["dy"].double()
            dn = dy * w
            share = torch.einsum("ij,ij->i", dn, n) / case["dim"]
            out["dx"] = s["ds"].double() + rstd * (dn - n * share[:, None])
            out["dw"] = torch.einsum("ij,ij->j", dy, n)
        return out
    act, x = case["act"], s["x"].double()

    def kept(v):
        return _exact_pack(v) if case["keep8"] else v.to(t).double()

    if op == "gated":
        wg, wu = s["wg"].double(), s["wu"].double()
        g, u = x @ wg.t(), x @ wu.t()
        out = {"y": _exact_act(g, act)[0] * u}
        if case["train"]:
            g, u = kept(g), kept(u)
            f, slope = _exact_act(g, act)
            dy = s["dy"].double()
            f *= dy
            slope *= dy * u
            out["dx"] = torch.addmm(f @ wu, slope, wg)
            if case["keep8"]:
                x = _exact_pack(x)
            out["dwg"], out["dwu"] = slope.t() @ x, f.t() @ x
        return out
    w = s["w"].double()
    z = x @ w.t()
    if case["bias"]:
        z += s["b"].double()
    out = {"y": _exact_act(z, act)[0]}
    if case["residual"]:
        out["y"] = out["y"] + s["residual"].double()
    if case["train"]:
        dz = s["dy"].double() * _exact_act(kept(z), act)[1]
        out["dx"] = dz @ w
        out["dw"] = dz.t() @ (_exact_pack(x) if case["keep8"] else x)
        if case["bias"]:
            out["db"] = dz.sum(0)
    return out
