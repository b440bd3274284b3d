"""Measured cases of the training operators beside the optimizer step: the
embedding lookup and its gradient, dropout from a counter-based generator,
and the microscaled 4-bit (MX FP4) quantisation and product.

`run` computes a case with the library's entry points where `own` is true,
and otherwise in plain torch operations in 32 bits, rounded once at the end.
`exact` is the same in 64 bits, from the definitions.

The definitions:

  embed       y[i] = scale * table[tok[i]]; a row of zeros where tok[i] is the
              padding token
  embed_grad  dtable[r] (+)= scale * sum of dy[i] over the i with tok[i] = r,
              the padding token's taking no part
  dropout     out[e] = residual[e] + (keep(e) ? x[e] / (1 - p) : 0); keep(e)
              where word e % 4 of Philox4x32-10 (Salmon et al. 2011) under the
              key `seed` at the counter (e / 4, offset) is at least p * 2^32.
              Its gradient is the same map of dy, without the residual
  quantize    blocks of 32 along a row share the power of two 2^(floor(log2
              max|x|) - 2); an element is the nearest of 0, .5, 1, 1.5, 2, 3,
              4, 6 (and their negatives) times it, ties to the even code
  linear      y = Q(x) Q(W)^T, W quantised once, x on every call
  linear_train  y as above, dx = Q(dy) Q(W^T)^T, dW = Q(dy^T) Q(x^T)^T

A quantised matrix is laid out as the library keeps it: records of 128 rows
by 256 columns, each the packed codes (128 rows of 128 bytes, whose 16-byte
pieces are exchanged by the row's low three bits) and then the 8 scale
exponents of every row.
"""
import math

import numpy as np
import torch

own = False

VOCAB = 50257          # the GPT-2 shapes' token table
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}


def listed():
    return [
        # the next token of 48 sequences being generated: latency
        dict(name="embed_token", op="embed", n=48, rows=VOCAB, dim=768, dtype="bf16",
             wide=True, scale=1.0, padded=0.0),
        # 16 sequences of 1024 tokens into GPT-2 XL's width, scaled by its root
        dict(name="embed_prompt", op="embed", n=16 * 1024, rows=VOCAB, dim=1600, dtype="f16",
             wide=True, scale=40.0, padded=0.05),
        # a short micro-batch added to the running fp32 gradient of the table
        dict(name="embed_grad_micro", op="embed_grad", n=1000, rows=VOCAB, dim=768, dtype="bf16",
             grad="f32", wide=False, scale=1.0, padded=0.1, accumulate=True),
        # one rank's batch of GPT-2 small: 8 sequences of 1024, into its bf16 grads
        dict(name="embed_grad_small", op="embed_grad", n=8 * 1024, rows=VOCAB, dim=768,
             dtype="bf16", grad="bf16", wide=True, scale=1.0, padded=0.02, accumulate=False),
        # a long batch at GPT-2 XL's width, one token short of a power of two
        dict(name="embed_grad_xl", op="embed_grad", n=131071, rows=VOCAB, dim=1600, dtype="f16",
             grad="f16", wide=True, scale=40.0, padded=0.05, accumulate=False),
        # fp32 activations of a few tokens: latency
        dict(name="dropout_small", op="dropout", n=33 * 768, dtype="f32", p=0.1, residual=False),
        # the residual branch of 16 sequences of 1024 at width 4096, both directions
        dict(name="dropout_residual", op="dropout", n=16 * 1024 * 4096, dtype="bf16", p=0.1,
             residual=True),
        # a ragged batch of tokens, along the rows only, as before a product
        dict(name="quantize_tokens", op="quantize", rows=77, cols=1600, dtype="bf16", both=False),
        # a Llama-7B MLP weight after an optimizer step, for both products
        dict(name="quantize_weight", op="quantize", rows=11008, cols=4096, dtype="bf16",
             both=True),
        # one token through a Llama-7B MLP weight: latency, the weight's bytes
        dict(name="linear_token", op="linear", m=1, n=11008, k=4096, dtype="bf16"),
        # a prompt of 333 tokens through GPT-2 XL's MLP weight: every size ragged
        dict(name="linear_prompt", op="linear", m=333, n=6400, k=1600, dtype="f16"),
        # forward and backward of a Llama-7B MLP weight over 8192 tokens
        dict(name="linear_train", op="linear_train", m=8192, n=11008, k=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "dropout", "quantize", "linear", "linear_train"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    low = rng.choice(["bf16", "f16"])
    if op == "embed":
        return dict(op=op, n=_log(rng, 1, 32768), rows=_log(rng, 1000, 65000),
                    dim=_log(rng, 64, 2000), dtype=dtype, wide=rng.random() < 0.5,
                    scale=rng.choice([1.0, 22.625, 40.0]), padded=rng.choice([0.0, 0.05, 0.5]))
    if op == "embed_grad":
        accumulate = rng.random() < 0.3
        return dict(op=op, n=_log(rng, 1, 130000), rows=_log(rng, 1000, 65000),
                    dim=_log(rng, 64, 1600), dtype=dtype, grad="f32" if accumulate else dtype,
                    wide=rng.random() < 0.5, scale=rng.choice([1.0, 22.625]),
                    padded=rng.choice([0.0, 0.05, 0.5]), accumulate=accumulate)
    if op == "dropout":
        return dict(op=op, n=_log(rng, 1000, 60_000_000), dtype=dtype,
                    p=rng.choice([0.0, 0.1, 0.25, 0.5]), residual=rng.random() < 0.5)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 10000), cols=_log(rng, 32, 4096), dtype=dtype,
                    both=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 4000), n=_log(rng, 64, 11008), k=_log(rng, 64, 8192),
                    dtype=low)
    return dict(op=op, m=_log(rng, 16, 8000), n=_log(rng, 64, 8192), k=_log(rng, 64, 4096),
                dtype=low)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)


def _normal(g, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _tokens(case, g):
    """Token ids whose frequencies fall as 1 / rank, as those of text do, with
    a share of padding (the table's last row)."""
    n, rows = case["n"], case["rows"]
    rank = torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
                     * math.log(rows)).long().clamp_(1, rows) - 1
    tok = (rank * 7919) % rows                   # the frequent ones not all side by side
    if case["padded"]:
        pad = torch.rand(n, generator=g, device="cuda") < case["padded"]
        tok = torch.where(pad, rows - 1, tok)
    return tok.to(torch.int64 if case["wide"] else torch.int32)


def _activations(g, rows, cols, dtype, sigma=1.0):
    """Normal values with a few columns much larger than the others, as the
    activations of large models have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * sigma
    big = torch.rand(cols, generator=g, device="cuda") < 0.01
    return torch.where(big, x * 12.0, x).to(dtype)


def _records(codes, exps):
    """Codes [R, C] and scale exponents [R, ceil(C / 32)] in the library's
    layout."""
    R, C = codes.shape
    rt, kt = -(-R // 128), -(-C // 256)
    full = torch.zeros(rt * 128, kt * 256, dtype=torch.uint8, device="cuda")
    full[:R, :C] = codes
    b = full[:, 0::2] | (full[:, 1::2] << 4)
    b = b.view(rt, 128, kt, 8, 16).permute(0, 2, 1, 3, 4)
    row = torch.arange(128, device="cuda")[:, None]
    piece = (torch.arange(8, device="cuda")[None, :] ^ (row & 7))
    b = torch.gather(b, 3, piece[None, None, :, :, None].expand(rt, kt, 128, 8, 16))
    s = torch.zeros(rt * 128, kt * 8, dtype=torch.uint8, device="cuda")
    s[:R, :exps.shape[1]] = exps
    s = s.view(rt, 4, 32, kt, 2, 4).permute(0, 3, 4, 2, 1, 5)
    return torch.cat([b.reshape(rt, kt, 16384), s.reshape(rt, kt, 1024)], 2).contiguous()


def _room(rows, cols):
    return torch.empty((-(-rows // 128), -(-cols // 256), 17408), dtype=torch.uint8,
                       device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case, "stream": torch.cuda.current_stream().cuda_stream}
    t = DT[case["dtype"]]
    if op == "embed":
        s["table"] = _normal(g, (case["rows"], case["dim"]), t, 0.02)
        s["tokens"] = _tokens(case, g)
        s["out"] = torch.empty(case["n"], case["dim"], dtype=t, device="cuda")
    elif op == "embed_grad":
        s["tokens"] = _tokens(case, g)
        s["dy"] = _normal(g, (case["n"], case["dim"]), t, 1e-2)
        gt = DT[case["grad"]]
        s["grad"] = (_normal(g, (case["rows"], case["dim"]), gt, 1e-2) if case["accumulate"] else
                     torch.empty(case["rows"], case["dim"], dtype=gt, device="cuda"))
    elif op == "dropout":
        n = case["n"]
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ (int(seed) * 2654435761), int(seed) * 64 + 5
        s["x"] = _normal(g, (n,), t)
        s["residual"] = _normal(g, (n,), t) if case["residual"] else None
        s["dy"] = _normal(g, (n,), t, 1e-2)
        s["out"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    elif op == "quantize":
        R, C = case["rows"], case["cols"]
        s["x"] = _activations(g, R, C, t)
        s["q"], s["v"] = _room(R, C), torch.empty_like(s["x"])
        if case["both"]:
            s["qt"] = _room(C, R)
            s["vt"] = torch.empty(C, R, dtype=t, device="cuda")
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _activations(g, m, k, t)
        w = torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)
        s["w_codes"], s["w_exps"] = _plain_quantize(w)
        s["wq"] = _records(s["w_codes"], s["w_exps"])
        s["xq"] = _room(m, k)
        s["y"] = torch.empty(m, n, dtype=t, device="cuda")
        if op == "linear_train":
            s["wt_codes"], s["wt_exps"] = _plain_quantize(w.t().contiguous())
            s["wtq"] = _records(s["wt_codes"], s["wt_exps"])
            s["dy"] = _normal(g, (m, n), t, 1e-2)
            s["xtq"], s["dyq"], s["dytq"] = _room(k, m), _room(m, n), _room(n, m)
            s["dx"] = torch.empty(m, k, dtype=t, device="cuda")
            s["dw"] = torch.empty(n, k, dtype=t, device="cuda")
    return s


# ---------------------------------------------------------------- the passes

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import zero_sharded_optimizer_step_gb300 as z
    c, st = s["case"], s["stream"]
    op, dt = c["op"], CODE[c["dtype"]]
    if op == "embed":
        z.zero_embed(s["table"], dt, c["rows"], c["dim"], c["dim"], s["tokens"],
                     8 if c["wide"] else 4, c["n"], c["rows"] - 1, c["scale"], s["out"],
                     c["dim"], None, st)
        return s["out"]
    if op == "embed_grad":
        if "ws" not in s:
            s["ws_bytes"] = z.zero_embed_grad_workspace(c["rows"], c["dim"], c["n"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        z.zero_embed_grad(s["dy"], dt, c["dim"], s["tokens"], 8 if c["wide"] else 4, c["n"],
                          c["rows"] - 1, c["scale"], s["grad"], CODE[c["grad"]], c["rows"],
                          c["dim"], c["dim"], c["accumulate"], s["ws"], s["ws_bytes"], st)
        return s["grad"]
    if op == "dropout":
        z.zero_dropout(s["x"], s["residual"], s["out"], dt, c["n"], c["p"], s["seed"],
                       s["offset"], 0, st)
        z.zero_dropout(s["dy"], None, s["dx"], dt, c["n"], c["p"], s["seed"], s["offset"], 0, st)
        return [s["out"], s["dx"]]
    if op == "quantize":
        R, C = c["rows"], c["cols"]
        if not c["both"]:
            z.zero_mx4_quantize(s["x"], dt, R, C, C, s["q"], None, st)
            z.zero_mx4_dequantize(s["q"], R, C, s["v"], dt, C, st)
            return [s["v"]]
        z.zero_mx4_quantize(s["x"], dt, R, C, C, s["q"], s["qt"], st)
        z.zero_mx4_dequantize(s["q"], R, C, s["v"], dt, C, st)
        z.zero_mx4_dequantize(s["qt"], C, R, s["vt"], dt, R, st)
        return [s["v"], s["vt"]]
    m, n, k = c["m"], c["n"], c["k"]
    if op == "linear":
        z.zero_mx4_quantize(s["x"], dt, m, k, k, s["xq"], None, st)
        z.zero_mx4_matmul(s["xq"], m, s["wq"], n, k, 1.0, False, s["y"], dt, n, st)
        return s["y"]
    z.zero_mx4_quantize(s["x"], dt, m, k, k, s["xq"], s["xtq"], st)
    z.zero_mx4_matmul(s["xq"], m, s["wq"], n, k, 1.0, False, s["y"], dt, n, st)
    z.zero_mx4_quantize(s["dy"], dt, m, n, n, s["dyq"], s["dytq"], st)
    z.zero_mx4_matmul(s["dyq"], m, s["wtq"], k, n, 1.0, False, s["dx"], dt, k, st)
    z.zero_mx4_matmul(s["dytq"], n, s["xtq"], k, m, 1.0, False, s["dw"], dt, k, st)
    return [s["y"], s["dx"], s["dw"]]


def _mulhilo(a, b):
    """High and low 32 bits of a * b, for a in [0, 2^32) held in int64."""
    lo = (a & 0xFFFF) * b
    hi = (a >> 16) * b + (lo >> 16)
    return hi >> 16, ((hi & 0xFFFF) << 16) | (lo & 0xFFFF)


def _plain_keep(n, p, seed, offset):
    c0 = torch.arange(-(-n // 4), device="cuda")
    c1 = c0 >> 32
    c0 = c0 & 0xFFFFFFFF
    c2 = torch.full_like(c0, offset & 0xFFFFFFFF)
    c3 = torch.full_like(c0, (offset >> 32) & 0xFFFFFFFF)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], 1).view(-1)[:n]
    return words >= int(p * 2.0 ** 32)


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_quantize(x):
    """Codes [R, C] (sign in bit 3) and scale exponents + 127 [R, ceil(C/32)]
    of an fp32 matrix, blocks along its rows."""
    R, C = x.shape
    blocks = -(-C // 32)
    full = x if C == 32 * blocks else torch.nn.functional.pad(x, (0, 32 * blocks - C))
    full = full.reshape(R, blocks, 32)
    top = full.abs().amax(2)
    e = ((top.view(torch.int32) >> 23) - 2).clamp_(min=0)
    inv = ((254 - e) << 23).view(torch.float32)
    v = (full * inv[:, :, None]).reshape(R, -1)[:, :C]
    a = v.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    return code + 8 * torch.signbit(v).byte(), e.byte()


def _plain_values(codes, exps):
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
    scale = torch.exp2(exps.float() - 127.0)
    C = codes.shape[1]
    return grid[codes.int()] * torch.repeat_interleave(scale, 32, 1)[:, :C]


def _plain(s):
    c = s["case"]
    op, t = c["op"], DT[c["dtype"]]
    if op == "embed":
        live = s["tokens"] != c["rows"] - 1
        y = s["table"][s["tokens"]].float() * c["scale"]
        s["out"].copy_(y * live[:, None])
        return s["out"]
    if op == "embed_grad":
        live = s["tokens"] != c["rows"] - 1
        acc = torch.zeros(c["rows"], c["dim"], device="cuda")
        acc.index_add_(0, s["tokens"], s["dy"].float() * live[:, None])
        acc *= c["scale"]
        if c["accumulate"]:
            acc += s["grad"].float()
        s["grad"].copy_(acc)
        return s["grad"]
    if op == "dropout":
        keep = _plain_keep(c["n"], c["p"], s["seed"], s["offset"])
        up = 1.0 / (1.0 - c["p"])
        y = torch.where(keep, s["x"].float() * up, 0.0)
        if c["residual"]:
            y += s["residual"].float()
        s["out"].copy_(y)
        s["dx"].copy_(torch.where(keep, s["dy"].float() * up, 0.0))
        return [s["out"], s["dx"]]
    if op == "quantize":
        x = s["x"].float()
        s["v"].copy_(_plain_values(*_plain_quantize(x)))
        if not c["both"]:
            return [s["v"]]
        s["vt"].copy_(_plain_values(*_plain_quantize(x.t().contiguous())))
        return [s["v"], s["vt"]]
    x = s["x"].float()
    xv = _plain_values(*_plain_quantize(x))
    s["y"].copy_(xv @ _plain_values(s["w_codes"], s["w_exps"]).t())
    if op == "linear":
        return s["y"]
    dy = s["dy"].float()
    dyv = _plain_values(*_plain_quantize(dy))
    s["dx"].copy_(dyv @ _plain_values(s["wt_codes"], s["wt_exps"]).t())
    xtv = _plain_values(*_plain_quantize(x.t().contiguous()))
    dytv = _plain_values(*_plain_quantize(dy.t().contiguous()))
    s["dw"].copy_(dytv @ xtv.t())
    return [s["y"], s["dx"], s["dw"]]


# ------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    es = torch.finfo(DT[case["dtype"]]).bits // 8
    if op in ("embed", "embed_grad"):
        n, d, ids = case["n"], case["dim"], 8 if case["wide"] else 4
        # rows that at least one of n tokens of such frequencies is expected to name
        h = math.log(case["rows"])
        r = np.arange(1, case["rows"] + 1)
        live = n * (1.0 - case["padded"])
        used = float(np.sum(1.0 - np.exp(-live * np.log1p(1.0 / r) / h)))
        if op == "embed":
            return {"bytes": int(n * ids + used * d * es + n * d * es), "flops": n * d}
        gs = torch.finfo(DT[case["grad"]]).bits // 8
        table = 2 * used * d * gs if case["accumulate"] else case["rows"] * d * gs
        return {"bytes": int(n * ids + live * d * es + table), "flops": int(live * d)}
    if op == "dropout":
        n = case["n"]
        return {"bytes": n * es * (5 if case["residual"] else 4), "flops": 4 * n}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        q = R * C // 2 + R * -(-C // 32)
        qt = R * C // 2 + C * -(-R // 32)
        b = R * C * es + 2 * q + R * C * es
        if case["both"]:
            b += 2 * qt + R * C * es
        return {"bytes": b, "flops": 2 * R * C * (2 if case["both"] else 1)}
    m, n, k = case["m"], case["n"], case["k"]
    w = n * k // 2 + n * k // 32
    if op == "linear":
        return {"bytes": m * k * es + w + m * n * es, "flops": 2 * m * n * k}
    return {"bytes": 2 * (m * k + m * n) * es + 2 * w + n * k * es, "flops": 6 * m * n * k}


# ------------------------------------------------- the definitions in 64 bits

def _power(e):
    """2^e for whole e, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(x):
    """The values a float64 matrix is quantised to, blocks along its rows: the
    element's own power of two gives its spacing, and the rounding to a whole
    number of spacings is to the even one."""
    R, C = x.shape
    out = torch.empty_like(x)
    for lo in range(0, C, 32 * 64):
        part = x[:, lo:lo + 32 * 64]
        w = part.shape[1]
        b = torch.nn.functional.pad(part, (0, -w % 32)).reshape(R, -1, 32)
        top = b.abs().amax(2, keepdim=True)
        shared = torch.where(top > 0, torch.frexp(top).exponent - 3, -127)
        unit = _power(shared.clamp(min=-127))
        v = b / unit
        step = _power((torch.frexp(v).exponent - 2).clamp(min=-1))
        v = torch.clamp(torch.round(v / step) * step, -6.0, 6.0) * unit
        out[:, lo:lo + w] = v.reshape(R, -1)[:, :w]
    return out


def _exact_keep(n, p, seed, offset):
    m32 = np.uint64(0xFFFFFFFF)
    c = [np.arange(-(-n // 4), dtype=np.uint64), None, None, None]
    c[1] = c[0] >> np.uint64(32)
    c[0] = c[0] & m32
    c[2] = np.full_like(c[0], offset & 0xFFFFFFFF)
    c[3] = np.full_like(c[0], (offset >> 32) & 0xFFFFFFFF)
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a = c[0] * np.uint64(0xD2511F53)
        b = c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(key[0]), b & m32,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(key[1]), a & m32]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).reshape(-1)[:n] >= np.uint64(math.floor(p * 2.0 ** 32))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        rows = s["table"].double().index_select(0, s["tokens"].long()) * case["scale"]
        rows[s["tokens"].long() == case["rows"] - 1] = 0.0
        return rows
    if op == "embed_grad":
        tok = s["tokens"].long()
        order = torch.argsort(tok, stable=True)
        order = order[tok[order] != case["rows"] - 1]
        out = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        out.index_add_(0, tok[order], s["dy"][order].double())
        out *= case["scale"]
        return out + s["grad"].double() if case["accumulate"] else out
    if op == "dropout":
        keep = torch.from_numpy(_exact_keep(case["n"], case["p"], s["seed"],
                                            s["offset"])).cuda().double()
        up = keep / (1.0 - case["p"])
        out = s["x"].double() * up
        if case["residual"]:
            out += s["residual"].double()
        return [out, s["dy"].double() * up]
    if op == "quantize":
        x = s["x"].double()
        v = _exact_values(x)
        return [v, _exact_values(x.t().contiguous())] if case["both"] else [v]
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")

    def of(codes, exps):
        v = grid[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3).double())
        return v * _power(exps.int() - 127).repeat_interleave(32, 1)[:, :codes.shape[1]]

    x = s["x"].double()
    y = _exact_values(x) @ of(s["w_codes"], s["w_exps"]).t()
    if op == "linear":
        return y
    dy = s["dy"].double()
    dx = _exact_values(dy) @ of(s["wt_codes"], s["wt_exps"]).t()
    dw = _exact_values(dy.t().contiguous()) @ _exact_values(x.t().contiguous()).t()
    return [y, dx, dw]
