"""Cases, plain forms and definitions of the 8-bit training and serving operators.

Six passes over three operators and their gradients:

  norm          residual addition, root-mean-square norm and an 8-bit output with a scale per 128 columns
  norm_grad     its gradients (input and gamma)
  project       matrix product of 8-bit operands with a scale per block of 128
  project_grad  the product's two gradients from bf16 dL/dy: quantise, dx and dW
  adamw         one AdamW step over many tensors, states in 8 or 32 bits
  adamw_rows    the same step over the touched rows of a table, from its sparse gradient

8-bit data is OCP E4M3 codes with E8M0 (power of two) scales.  A matrix of `rows` x `cols` holds its codes as
[rows][128 ceil(cols / 128)], zero past `cols`, and its scales as [rows or ceil(rows / 128)][4 ceil(blocks / 4)],
one byte for each block of 128 columns.  Codes and scales are returned in their own floating types.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
EPS = 1e-6
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
MASK64 = (1 << 64) - 1


# ---------------------------------------------------------------------------------------------------------------
# The cases.

def listed():
    return [
        # four sequences decoding one token each through the norm in front of an 8-bit product
        {"name": "norm_decode", "op": "norm", "n": 4, "d": 2560, "x": "bf16", "keep": False},
        # the prefill batch (8 x 4096 tokens) at the table's width
        {"name": "norm_prefill", "op": "norm", "n": 32768, "d": 2560, "x": "bf16", "keep": False},
        # a ragged training batch of fp32 sums at an odd width; the bf16 output and 1/rms are kept for the backward
        {"name": "norm_train_ragged", "op": "norm", "n": 5003, "d": 1032, "x": "f32", "keep": True},
        # the backward of the prefill-sized batch, with the gradient that comes down the residual stream
        {"name": "norm_grad_prefill", "op": "norm_grad", "n": 32768, "d": 2560, "dy": "bf16"},
        {"name": "norm_grad_ragged", "op": "norm_grad", "n": 777, "d": 520, "dy": "f32"},
        # decode: every weight read once for four tokens
        {"name": "project_decode", "op": "project", "n": 4, "d_in": 2560, "d_out": 2560, "y": "bf16"},
        # the projected path's product at prefill
        {"name": "project_prefill", "op": "project", "n": 32768, "d_in": 2560, "d_out": 2560, "y": "bf16"},
        # a short chunk of a prompt, odd in every direction
        {"name": "project_ragged", "op": "project", "n": 777, "d_in": 1032, "d_out": 4104, "y": "f32"},
        # both gradients of the product for a training batch
        {"name": "project_grad", "op": "project_grad", "n": 8192, "d_in": 2560, "d_out": 2560},
        # the dense parameters of a few blocks, bf16 with 8-bit states
        {"name": "adamw_8bit", "op": "adamw", "tensors": 96, "total": 200_000_000, "p": "bf16", "g": "bf16", "state": 8},
        # gates, norms and other small vectors: fp32 with fp32 states, where launches count
        {"name": "adamw_small", "op": "adamw", "tensors": 40, "total": 300_000, "p": "f32", "g": "f32", "state": 32},
        # the rows that a prefill-sized training batch touches in a bf16 table with 8-bit states
        {"name": "adamw_rows", "op": "adamw_rows", "rows": 260_000, "R": 1_000_000, "d": 2560, "p": "bf16", "state": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 8, often no multiple of 128."""
    w = _log(rng, lo, hi)
    w = max(lo, w // 128 * 128) if rng.random() < 0.4 else max(lo, w // 8 * 8)
    return w + 8 if w == 3072 else w


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "project", "project_grad", "adamw", "adamw_rows"])
    if op in ("norm", "norm_grad"):
        d = _width(rng, 64, 8192)
        n = _log(rng, 1, min(32768, 32768 * 2560 // d))
        n += n == 3072
        if op == "norm":
            return {"op": op, "n": n, "d": d, "x": rng.choice(["bf16", "f32"]), "keep": rng.random() < 0.5}
        return {"op": op, "n": n, "d": d, "dy": rng.choice(["bf16", "f32"])}
    if op == "project":
        d_in, d_out = _width(rng, 256, 8192), _width(rng, 256, 8192)
        n = _log(rng, 1, min(32768, 32768 * 2560 * 2560 // (d_in * d_out)))
        return {"op": op, "n": n + (n == 3072), "d_in": d_in, "d_out": d_out, "y": rng.choice(["bf16", "f32"])}
    if op == "project_grad":
        d_in, d_out = _width(rng, 256, 5120), _width(rng, 256, 5120)
        n = _log(rng, 16, min(16384, 8192 * 2560 * 2560 // (d_in * d_out)))
        return {"op": op, "n": n + (n == 3072), "d_in": d_in, "d_out": d_out}
    if op == "adamw":
        count = _log(rng, 1, 200)
        total = _log(rng, 2000 * count, max(100_000_000, 2000 * count))
        return {"op": op, "tensors": count, "total": total, "p": rng.choice(["bf16", "f32"]), "g": rng.choice(["bf16", "f32"]),
                "state": rng.choice([8, 32])}
    d = _width(rng, 64, 8192)
    rows = _log(rng, 1, 200_000 * 2560 // d)
    return {"op": op, "rows": rows, "R": rows * rng.randint(1, 3) + rng.randint(1, 1000), "d": d, "p": rng.choice(["bf16", "f32"]),
            "state": rng.choice([8, 32])}


# ---------------------------------------------------------------------------------------------------------------
# Layouts.

def _blocks(cols):
    return (cols + 127) // 128


def _scale_cols(cols):
    return (_blocks(cols) + 3) // 4 * 4


def _sizes(case):
    """The tensors' sizes of an adamw case (spread over their logarithm, odd ones among them) and their places in one
    buffer, each at a multiple of 128 elements."""
    rng = random.Random(case["tensors"] * 1_000_003 + case["total"])
    parts = [math.exp(rng.uniform(0.0, 5.0)) for _ in range(case["tensors"])]
    whole = sum(parts)
    sizes = [max(1, int(case["total"] * p / whole)) for p in parts]
    places, at = [], 0
    for s in sizes:
        places.append(at)
        at += _blocks(s) * 128
    return sizes, places, at


def work(case):
    op = case["op"]
    if op == "norm":
        n, d = case["n"], case["d"]
        x = 2 if case["x"] == "bf16" else 4
        out = 2 + 1 + 1 / 128 + (2 if case["keep"] else 0)
        return {"bytes": n * d * (x + 2 + out) + 4 * d + (4 * n if case["keep"] else 0), "flops": 0}
    if op == "norm_grad":
        n, d = case["n"], case["d"]
        return {"bytes": n * d * ((2 if case["dy"] == "bf16" else 4) + 2 + 2 + 2) + 4 * n + 8 * d, "flops": 0}
    if op == "project":
        n, k, o = case["n"], case["d_in"], case["d_out"]
        return {"bytes": n * k * 129 / 128 + o * k + n * o * (2 if case["y"] == "bf16" else 4), "flops": 2 * n * k * o}
    if op == "project_grad":
        n, k, o = case["n"], case["d_in"], case["d_out"]
        return {"bytes": 2 * n * o + 2 * n * k + o * k + 2 * n * k + 4 * o * k, "flops": 4 * n * k * o}
    p, g = (2 if case["p"] == "bf16" else 4), (2 if case.get("g", "f32") == "bf16" else 4)
    s = 4 * (1 + 1 / 128) if case["state"] == 8 else 16
    count = sum(_sizes(case)[0]) if op == "adamw" else case["rows"] * case["d"]
    return {"bytes": count * (2 * p + g + s), "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits.

def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, at least -126; 0 for a block of zeros."""
    bits = amax.view(torch.int32)
    e = ((bits >> 23) & 255) - 135 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return torch.where(amax > 0, e.clamp(min=-126), torch.zeros_like(e))


def _pow2(e):
    """2^e in fp32 for integer e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _scale_bytes(e, rows, cols):
    """Exponents [r][blocks] as E8M0 bytes in rows of 4 ceil(blocks / 4); the bytes past the blocks are 127 (a scale of 1)."""
    out = torch.full((rows, _scale_cols(cols)), 127, dtype=torch.uint8, device=e.device)
    out[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    return out


def _quant(x, tile=False):
    """fp32 [rows][cols] to codes and scale bytes: a scale for each row's 128 columns, or for each 128 x 128 tile."""
    rows, cols = x.shape
    nb = _blocks(cols)
    full = torch.zeros((_blocks(rows) * 128 if tile else rows, nb * 128), dtype=torch.float32, device=x.device)
    full[:rows, :cols] = x
    if tile:
        t = full.view(-1, 128, nb, 128)
        e = _exponent(t.abs().amax(dim=(1, 3)))
        codes = (t * _pow2(-e)[:, None, :, None]).view(-1, nb * 128)[:rows].to(E4M3)
    else:
        t = full.view(rows, nb, 128)
        e = _exponent(t.abs().amax(dim=2))
        codes = (t * _pow2(-e)[:, :, None]).view(rows, nb * 128).to(E4M3)
    return codes, _scale_bytes(e, e.shape[0], cols)


def _dequant(codes, scales, cols):
    """The values that codes [rows][ld] and scale bytes stand for, fp32 [rows][ld]; a row of scales may serve 128 rows."""
    rows, ld = codes.shape
    s = _pow2(scales[:, :ld // 128].to(torch.int32) - 127)
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, dim=0)[:rows]
    return (codes.to(torch.float32).view(rows, ld // 128, 128) * s[:, :, None]).view(rows, ld)


def _plain_norm(s):
    x = s["x"].float() + s["res"].float()
    total = x.to(torch.bfloat16)
    f = total.float()
    r = torch.rsqrt((f * f).sum(dim=1) / s["d"] + EPS)
    y = f * r[:, None] * s["gamma"]
    codes, scales = _quant(y)
    out = {"sum": total, "codes": codes, "scales": scales.view(E8M0)}
    if s["keep"]:
        out |= {"y": y.to(torch.bfloat16), "r": r}
    return out


def _plain_norm_grad(s):
    f, dy, r = s["sum"].float(), s["dy"].float(), s["r"][:, None]
    h = dy * s["gamma"]
    dot = (h * f).sum(dim=1, keepdim=True)
    dx = h * r - f * (dot * r * r * r / s["d"]) + s["dsum"].float()
    return {"dx": dx.to(torch.bfloat16), "dgamma": (dy * (f * r)).sum(dim=0)}


def _plain_project(s):
    a = _dequant(s["x_codes"], s["x_scales"], s["d_in"])
    b = _dequant(s["w_codes"], s["w_scales"], s["d_in"])
    return {"y": (a @ b.t()).to(s["y_dtype"])}


def _plain_project_grad(s):
    n, dy, x = s["n"], s["dy"].float(), s["x"].float()
    q = _dequant(*_quant(dy), s["d_out"])
    qt = _dequant(*_quant(dy.t()), n)
    xt = _dequant(*_quant(x.t()), n)
    w = _dequant(s["wt_codes"], s["wt_scales"], s["d_out"])
    return {"dx": (q @ w.t()).to(torch.bfloat16), "dw": qt @ xt.t()}


def _mix(z):
    """splitmix64's first output from each state of an int64 tensor (wrapping arithmetic, logical shifts)."""
    z = z + (0x9E3779B97F4A7C15 - (1 << 64))
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * (0xBF58476D1CE4E5B9 - (1 << 64))
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * (0x94D049BB133111EB - (1 << 64))
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _mix_int(x):
    z = (x + 0x9E3779B97F4A7C15) & MASK64
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK64
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK64
    return z ^ (z >> 31)


def _random_words(seed, step, index):
    """The 32 random bits of each element: its half of splitmix64(key + index / 2), even indexes the low one."""
    key = _mix_int((_mix_int(seed) + step) & MASK64)
    z = _mix(key - (1 << 64 if key >> 63 else 0) + (index >> 1))
    return torch.where((index & 1) == 1, (z >> 32) & 0xFFFFFFFF, z & 0xFFFFFFFF)


def _code_up(a, rand20, positive):
    """Codes of the scaled magnitudes a <= 448, rounded up with the chance that 20 random bits give; `positive`: a value
    above zero never becomes zero."""
    near = ((a.view(torch.int32).long() + rand20) >> 20) - 960
    low = (a * 512 + rand20.float() * 2.0 ** -20).long()
    code = torch.where(a >= 2.0 ** -6, near, low).clamp(max=126)
    return torch.where(a > 0, code.clamp(min=1), code) if positive else code


def _pack_state(x, rand20, positive):
    """fp32 [rows][ld] to codes and scale bytes with a scale for each 128 elements."""
    t = x.view(x.shape[0], -1, 128)
    e = _exponent(t.abs().amax(dim=2))
    code = _code_up((t * _pow2(-e)[:, :, None]).view(x.shape).abs(), rand20, positive)
    return torch.where(x < 0, code + 128, code).to(torch.uint8).view(E4M3), (e + 127).to(torch.uint8)


def _round_bf16(x, rand16):
    return ((x.view(torch.int32).long() + rand16) >> 16).to(torch.int16).view(torch.bfloat16)


def _plain_step(p, g, m, v, ms, vs, state, index, seed, step):
    """One AdamW step on [rows][ld] (ld a multiple of 128 where the states have 8 bits): the new p, m, v and scales.
    In 8 bits v holds the square root of the second moment."""
    h = HYPER
    b1, b2 = h["beta1"], h["beta2"]
    decay, rate = 1 - h["lr"] * h["weight_decay"], h["lr"] / (1 - b1 ** step)
    root = 1 / math.sqrt(1 - b2 ** step)
    g = g.float()
    if state == 8:
        m = _dequant(m, ms, m.shape[1])
        v = _dequant(v, vs, v.shape[1])
        v = v * v
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * (g * g)
    root_v = v.sqrt()
    new = p.float() * decay - rate * (m / (root_v * root + h["eps"]))
    if state == 8 or p.dtype == torch.bfloat16:
        word = _random_words(seed, step, index)
    if p.dtype == torch.bfloat16:
        new = _round_bf16(new, (word >> 8) & 0xFFFF)
    if state == 32:
        return new, m, v, None, None
    m, ms = _pack_state(m, word & 0xFFFFF, False)
    v, vs = _pack_state(root_v, word >> 12, True)
    return new, m, v, ms, vs


def _plain_adamw(s):
    index = torch.arange(s["p"].numel(), device=DEV).view(1, -1)
    names = ("p", "m", "v") + (("ms", "vs") if s["state"] == 8 else ())
    row = {k: s[k].view(1, -1) for k in names}
    new = _plain_step(row["p"], s["g"].view(1, -1), row["m"], row["v"], row.get("ms"), row.get("vs"), s["state"], index, s["seed"], s["step"])
    for k, t in zip(("p", "m", "v", "ms", "vs"), new):
        if t is not None:
            row[k].view(torch.uint8).copy_(t.view(torch.uint8))
    return _states(s)


def _plain_adamw_rows(s):
    rows, d = s["row_ids"].long(), s["d"]
    ld = _blocks(d) * 128 if s["state"] == 8 else d
    pad = lambda t: torch.nn.functional.pad(t.view(torch.uint8), (0, (ld - d) * t.element_size())).view(t.dtype)  # noqa: E731
    index = rows[:, None] * d + torch.arange(ld, device=DEV)
    take = lambda t: pad(t.view(torch.uint8)[rows].view(t.dtype))  # noqa: E731
    ms, vs = (s["ms"][rows], s["vs"][rows]) if s["state"] == 8 else (None, None)
    new = _plain_step(take(s["p"]), pad(s["g"]), take(s["m"]), take(s["v"]), ms, vs, s["state"], index, s["seed"], s["step"])
    for k, t in zip(("p", "m", "v"), new):
        s[k].view(torch.uint8)[rows] = t[:, :d].contiguous().view(torch.uint8)
    if s["state"] == 8:
        s["ms"][rows], s["vs"][rows] = new[3], new[4]
    return _states(s)


def _states(s):
    out = {"p": s["p"], "m": s["m"], "v": s["v"]}
    return out | ({"ms": s["ms"].view(E8M0), "vs": s["vs"].view(E8M0)} if s["state"] == 8 else {})


# ---------------------------------------------------------------------------------------------------------------
# Inputs.

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _activations(g, n, d):
    """Hidden states: a few columns far larger than the others, as a residual stream has them."""
    x = _normal(g, n, d)
    return x.mul_(torch.exp(0.5 * _normal(g, d)) * (1 + 20 * (torch.rand(d, generator=g, device=DEV) < 0.004)))


def _optimiser_state(g, p, state, rows, d):
    """Moments as after some hundred steps: sizes spread over several powers of ten within a tensor."""
    size = 1e-3 * torch.exp(_normal(g, rows, d))
    m = size * _normal(g, rows, d, std=0.3)
    v = size.square_()
    if state == 32:
        return {"m": m, "v": v}
    mc, ms = _quant(m)
    del m
    vc, vs = _quant(v.sqrt_())
    nb = _blocks(d)
    return {"m": mc[:, :d].contiguous(), "v": vc[:, :d].contiguous(), "ms": ms[:, :nb].contiguous(), "vs": vs[:, :nb].contiguous()}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op in ("norm", "norm_grad"):
        n, d = case["n"], case["d"]
        s |= {"d": d, "gamma": 1 + 0.2 * _normal(g, d)}
        if op == "norm":
            s |= {"x": _normal(g, n, d, std=0.1).to(_DT[case["x"]]), "res": _activations(g, n, d).to(torch.bfloat16), "keep": case["keep"]}
            s["sum_out"] = torch.empty((n, d), dtype=torch.bfloat16, device=DEV)
            return s
        total = _activations(g, n, d).to(torch.bfloat16)
        f = total.float()
        s |= {"sum": total, "r": torch.rsqrt((f * f).sum(dim=1) / d + EPS), "dy": _normal(g, n, d, std=1e-2).to(_DT[case["dy"]]),
              "dsum": _normal(g, n, d, std=1e-2).to(torch.bfloat16)}
        return s
    if op in ("project", "project_grad"):
        n, k, o = case["n"], case["d_in"], case["d_out"]
        s |= {"n": n, "d_in": k, "d_out": o}
        x, w = _activations(g, n, k), _normal(g, o, k, std=k ** -0.5)
        if op == "project":
            s["x_codes"], s["x_scales"] = _quant(x.to(torch.bfloat16).float())
            s["w_codes"], s["w_scales"] = _quant(w, tile=True)
            s["y_dtype"] = _DT[case["y"]]
            return s
        s["x"] = x.to(torch.bfloat16)
        s["wt_codes"], s["wt_scales"] = _quant(w.t().contiguous(), tile=True)
        s["dy"] = (_normal(g, n, o, std=1e-2) * torch.exp(_normal(g, n, 1))).to(torch.bfloat16)
        return s
    s |= {"state": case["state"], "seed": seed & MASK64, "step": 200}
    if op == "adamw":
        sizes, places, whole = _sizes(case)
        live = torch.zeros(whole, dtype=torch.bool, device=DEV)
        for at, size in zip(places, sizes):
            live[at:at + size] = True
        s |= {"sizes": sizes, "places": places}
        s["p"] = (_normal(g, whole, std=0.02) * live).to(_DT[case["p"]])
        s["g"] = (_normal(g, whole, std=1e-3) * live).to(_DT[case["g"]])
        st = _optimiser_state(g, s["p"], 32, 1, whole)
        m, v = st["m"].mul_(live), st["v"].mul_(live)
        if case["state"] == 8:
            (m, ms), (v, vs) = _quant(m), _quant(v.sqrt_())
            s |= {"ms": ms.view(-1)[:whole // 128].clone(), "vs": vs.view(-1)[:whole // 128].clone()}
        s |= {"m": m.view(-1), "v": v.view(-1)}
        return s
    rows, R, d = case["rows"], case["R"], case["d"]
    s |= {"d": d, "R": R, "p": _normal(g, R, d, std=0.02).to(_DT[case["p"]])}
    s |= _optimiser_state(g, s["p"], case["state"], R, d)
    s["row_ids"] = torch.randperm(R, generator=g, device=DEV)[:rows].sort().values.to(torch.int32)
    s["count"] = torch.tensor([rows], device=DEV)
    s["g"] = _normal(g, rows, d, std=1e-3)
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass.

def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "project": _plain_project, "project_grad": _plain_project_grad,
          "adamw": _plain_adamw, "adamw_rows": _plain_adamw_rows}


def _own_norm(s):
    import hashed_gram_embedding_ngram_amd as ng
    out = ng.ngram_add_norm(s["x"], s["gamma"], EPS, residual=s["res"], sum_out=s["sum_out"], keep_y=s["keep"], keep_r=s["keep"])
    got = {"sum": s["sum_out"], "codes": out.q.codes, "scales": out.q.scales.view(E8M0)}
    return got | ({"y": out.y, "r": out.r} if s["keep"] else {})


def _own_norm_grad(s):
    import hashed_gram_embedding_ngram_amd as ng
    dx, dgamma = ng.ngram_add_norm_grad(s["dy"], s["sum"], s["r"], s["gamma"], dsum=s["dsum"])
    return {"dx": dx, "dgamma": dgamma}


def _own_project(s):
    import hashed_gram_embedding_ngram_amd as ng
    x = ng.Fp8(s["x_codes"], s["x_scales"], s["x_codes"].shape[0], s["d_in"])
    w = ng.Fp8(s["w_codes"], s["w_scales"], s["w_codes"].shape[0], s["d_in"], block_rows=128)
    return {"y": ng.ngram_project_fp8(x, w, dtype=s["y_dtype"])}


def _own_project_grad(s):
    import hashed_gram_embedding_ngram_amd as ng
    wt = ng.Fp8(s["wt_codes"], s["wt_scales"], s["d_in"], s["d_out"], block_rows=128)
    q, qt = ng.ngram_quant_fp8(s["dy"], rows=True, transposed=True)
    _, xt = ng.ngram_quant_fp8(s["x"], rows=False, transposed=True)
    return {"dx": ng.ngram_project_fp8(q, wt, dtype=torch.bfloat16), "dw": ng.ngram_project_fp8(qt, xt, dtype=torch.float32)}


def _own_adamw(s):
    import hashed_gram_embedding_ngram_amd as ng
    if "handle" not in s:  # the parameter list that a training program builds once
        cut = lambda t, at, size: t[at:at + size]  # noqa: E731
        spans = list(zip(s["places"], s["sizes"]))
        parts = {k: [cut(s[k], at, size) for at, size in spans] for k in ("p", "g", "m", "v")}
        if s["state"] == 8:
            parts |= {k: [cut(s[k], at // 128, _blocks(size)) for at, size in spans] for k in ("ms", "vs")}
        s["handle"] = ng.AdamWTensors(parts["p"], parts["g"], parts["m"], parts["v"], m_scales=parts.get("ms"), v_scales=parts.get("vs"),
                                      rng_offsets=s["places"])
    ng.ngram_adamw(s["handle"], step=s["step"], seed=s["seed"], **HYPER)
    return _states(s)


def _own_adamw_rows(s):
    import hashed_gram_embedding_ngram_amd as ng
    ng.ngram_adamw_rows(s["p"], s["m"], s["v"], s["row_ids"], s["g"], s["count"], m_scale=s.get("ms"), v_scale=s.get("vs"),
                        step=s["step"], seed=s["seed"], **HYPER)
    return _states(s)


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "project": _own_project, "project_grad": _own_project_grad,
        "adamw": _own_adamw, "adamw_rows": _own_adamw_rows}


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits.

def _x_exponent(amax):
    f, k = torch.frexp(amax)
    e = torch.where(f <= 0.875, k - 9, k - 8).clamp(min=-126)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _x_pow2(e):
    """2^e in float64, exactly (torch.ldexp goes through pow, which is an ulp off on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _x_scale(e, rows, cols):
    out = torch.ones((rows, _scale_cols(cols)), dtype=torch.float64, device=e.device)
    out[:, :e.shape[1]] = _x_pow2(e)
    return out


def _x_grid(a, least=-6):
    """The spacing of E4M3 values at magnitude a."""
    _, k = torch.frexp(a)
    return _x_pow2(torch.where(a > 0, k - 4, k.new_full((), least - 3)).clamp(min=least - 3))


def _x_quant(x):
    """Codes (as the numbers they encode, unscaled) and scales of float64 rows, a scale for each 128 columns."""
    rows, cols = x.shape
    nb = _blocks(cols)
    full = torch.zeros((rows, nb * 128), dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    t = full.view(rows, nb, 128)
    e = _x_exponent(t.abs().amax(dim=2))
    t = t * _x_pow2(-e)[:, :, None]
    step = _x_grid(t.abs())
    return (torch.round(t / step) * step).view(rows, nb * 128), _x_scale(e, rows, cols)


def _x_values(codes, scales):
    rows, ld = codes.shape
    return (codes.view(rows, ld // 128, 128) * scales[:, :ld // 128, None]).view(rows, ld)


def _x_bytes(scales):
    return _x_pow2(scales.view(torch.uint8).int() - 127)


def _x_dequant(codes, scales):
    s = _x_bytes(scales)
    return _x_values(codes.double(), s if s.shape[0] == codes.shape[0] else s.repeat_interleave(128, dim=0)[:codes.shape[0]])


def _x_norm(s, case):
    total = (s["x"].double() + s["res"].double()).to(torch.bfloat16)
    f = total.double()
    r = (f.square().sum(dim=1) / s["d"] + EPS).rsqrt()
    y = f * r[:, None] * s["gamma"].double()
    codes, scales = _x_quant(y)
    return {"sum": total.double(), "codes": codes, "scales": scales} | ({"y": y, "r": r} if case["keep"] else {})


def _x_norm_grad(s, case):
    f, dy, r = s["sum"].double(), s["dy"].double(), s["r"].double()[:, None]
    hat, h = f * r, dy * s["gamma"].double()
    dx = r * (h - hat * (h * hat).mean(dim=1, keepdim=True)) + s["dsum"].double()
    return {"dx": dx, "dgamma": (dy * hat).sum(dim=0)}


def _x_project(s, case):
    return {"y": _x_dequant(s["x_codes"], s["x_scales"]) @ _x_dequant(s["w_codes"], s["w_scales"]).t()}


def _x_project_grad(s, case):
    dy, x = s["dy"].double(), s["x"].double()
    dx = _x_values(*_x_quant(dy)) @ _x_dequant(s["wt_codes"], s["wt_scales"]).t()
    return {"dx": dx, "dw": _x_values(*_x_quant(dy.t())) @ _x_values(*_x_quant(x.t())).t()}


def _x_up(x, rand, bits, step, positive=False):
    """x >= 0 to a multiple of `step`, up with the chance that `rand` of 2^bits gives."""
    q = torch.floor(x / step + rand.double() * 2.0 ** -bits)
    return (torch.where(x > 0, q.clamp(min=1), q) if positive else q) * step


def _x_state(x, rand, positive):
    t = x.view(x.shape[0], -1, 128)
    e = _x_exponent(t.abs().amax(dim=2))
    a = (t * _x_pow2(-e)[:, :, None]).view(x.shape)
    q = _x_up(a.abs(), rand, 20, _x_grid(a.abs()), positive).clamp(max=448.0)
    return torch.where(a < 0, -q, q), _x_pow2(e)


def _x_step(p, g, m, v, state, bf16, index, seed, step):
    h = HYPER
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    m_hat, v_hat = m / (1 - h["beta1"] ** step), v / (1 - h["beta2"] ** step)
    p = p - h["lr"] * h["weight_decay"] * p - h["lr"] * m_hat / (v_hat.sqrt() + h["eps"])
    word = _random_words(seed, step, index) if state == 8 or bf16 else None
    if bf16:
        _, k = torch.frexp(p.abs())
        grid = _x_pow2((k - 8).clamp(min=-133))
        p = torch.where(p < 0, -1.0, 1.0) * _x_up(p.abs(), (word >> 8) & 0xFFFF, 16, grid)
    if state == 32:
        return {"p": p, "m": m, "v": v}
    m, ms = _x_state(m, word & 0xFFFFF, False)
    v, vs = _x_state(v.sqrt(), word >> 12, True)
    return {"p": p, "m": m, "v": v, "ms": ms, "vs": vs}


def _x_moments(s, rows, d):
    """(m, second moment) in float64 [rows][d]."""
    take = (lambda t: t) if rows is None else (lambda t: t.view(torch.uint8)[rows].view(t.dtype))
    m, v = take(s["m"]).double(), take(s["v"]).double()
    if s["state"] == 32:
        return m, v
    ms, vs = (_x_bytes(take(s[k])) for k in ("ms", "vs"))
    wide = lambda t, b: t * b.repeat_interleave(128, dim=-1)[..., :d]  # noqa: E731
    return wide(m, ms), wide(v, vs).square()


def _x_adamw(s, case):
    whole = s["p"].numel()
    m, v = _x_moments(s, None, whole)
    one = lambda t: t.view(1, -1)  # noqa: E731
    new = _x_step(one(s["p"].double()), one(s["g"].double()), one(m), one(v), s["state"], case["p"] == "bf16",
                  one(torch.arange(whole, device=DEV)), s["seed"], s["step"])
    return {k: t.view(-1) for k, t in new.items()}


def _x_adamw_rows(s, case):
    d, R = s["d"], s["R"]
    ld = _blocks(d) * 128
    out = {"p": s["p"].double(), "m": s["m"].double(), "v": s["v"].double()}
    if s["state"] == 8:
        out |= {"ms": _x_bytes(s["ms"]), "vs": _x_bytes(s["vs"])}
    for at in range(0, s["row_ids"].numel(), 32768):
        rows = s["row_ids"][at:at + 32768].long()
        pad = lambda t: torch.nn.functional.pad(t, (0, ld - d))  # noqa: E731
        m, v = _x_moments(s, rows, d)
        p = s["p"].view(torch.uint8)[rows].view(s["p"].dtype).double()
        new = _x_step(pad(p), pad(s["g"][at:at + 32768].double()), pad(m), pad(v), s["state"], case["p"] == "bf16",
                      rows[:, None] * d + torch.arange(ld, device=DEV), s["seed"], s["step"])
        for k, t in new.items():
            out[k][rows] = t[:, :out[k].shape[1]]
    return out


_EXACT = {"norm": _x_norm, "norm_grad": _x_norm_grad, "project": _x_project, "project_grad": _x_project_grad, "adamw": _x_adamw,
          "adamw_rows": _x_adamw_rows}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)
