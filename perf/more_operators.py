"""Cases, plain forms and definitions of the operators over the vocabulary: 4-bit products, beam search, distillation.

Five operators:

  project_int4  product with 4-bit weights that have a scale (and a zero) for each group of columns: few rows, all weights
  quant_int4    weights rounded to that format and read back as the values they stand for
  beam_step     the next beams of each sequence from the logits: tokens, scores, parents, two-token histories, finished marks
  beam_reorder  per-beam state rows taken from the beams' parents, in place, in many tensors
  distill       loss against a teacher's top logits and its gradient, in one call or in two

4-bit codes lie two to a byte, the even column in the low nibble, in rows of 16 ceil(cols / 32) bytes; scales and zeros in rows
of 4 ceil(groups / 4), a group being 32, 64 or 128 columns.  Value = scale * (code - zero); without zeros, zero is 8.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
NEG = float("-inf")


# ---------------------------------------------------------------------------------------------------------------
# The cases.

def listed():
    return [
        # one token through a square projection of the layer's width: launch and one pass over 3 MB
        {"name": "project_one", "op": "project_int4", "n": 1, "d_in": 2560, "d_out": 2560, "group": 128, "zeros": False, "x": "bf16",
         "y": "bf16", "scale": "bf16"},
        # logits of 4 sequences with 8 beams each, the whole vocabulary
        {"name": "project_head", "op": "project_int4", "n": 32, "d_in": 2560, "d_out": 151936, "group": 64, "zeros": True, "x": "bf16",
         "y": "f32", "scale": "bf16"},
        # fp32 sums of the gather, odd in every direction, small groups with fp32 scales
        {"name": "project_ragged", "op": "project_int4", "n": 11, "d_in": 1032, "d_out": 4103, "group": 32, "zeros": True, "x": "f32",
         "y": "bf16", "scale": "f32"},
        # a vocabulary's weights quantised for serving, and the rounded values back for training through them
        {"name": "quant_head", "op": "quant_int4", "rows": 151936, "cols": 2560, "group": 64, "zeros": True, "x": "bf16", "y": "bf16",
         "scale": "bf16"},
        {"name": "quant_ragged", "op": "quant_int4", "rows": 777, "cols": 1032, "group": 32, "zeros": False, "x": "f32", "y": "f32",
         "scale": "f32"},
        # one prompt with four beams
        {"name": "beam_one", "op": "beam_step", "batch": 1, "beams": 4, "V": 151936, "logits": "bf16"},
        # a full serving batch with fp32 logits
        {"name": "beam_batch", "op": "beam_step", "batch": 64, "beams": 8, "V": 151936, "logits": "f32"},
        # the token lists and a hidden state of one prompt's beams
        {"name": "reorder_one", "op": "beam_reorder", "batch": 1, "beams": 4, "tensors": 3, "row_bytes": 5120},
        # per-layer states of a serving batch
        {"name": "reorder_batch", "op": "beam_reorder", "batch": 16, "beams": 8, "tensors": 24, "row_bytes": 262144},
        # a training batch at the table's vocabulary: loss and gradient in one call
        {"name": "distill_train", "op": "distill", "n": 4096, "V": 151936, "k": 64, "logits": "bf16", "T": 1.0, "tail": False, "fused": True},
        # forward and backward apart, with the teacher's mass off the list, at an odd vocabulary
        {"name": "distill_split", "op": "distill", "n": 1021, "V": 32003, "k": 100, "logits": "f32", "T": 2.0, "tail": True, "fused": False},
        # a short evaluation batch: fewer rows than compute units
        {"name": "distill_few", "op": "distill", "n": 24, "V": 151936, "k": 16, "logits": "bf16", "T": 1.5, "tail": True, "fused": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 8, often no multiple of 128."""
    w = _log(rng, lo, hi)
    return max(lo, w // 128 * 128) if rng.random() < 0.4 else max(lo, w // 8 * 8)


def draw(rng):
    op = rng.choice(["project_int4", "quant_int4", "beam_step", "beam_reorder", "distill"])
    kind = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op == "project_int4":
        d_in = _width(rng, 256, 8192)
        d_out = _log(rng, 256, min(152000, 151936 * 2560 // d_in))
        n = _log(rng, 1, 64)
        while n * d_in * d_out > 32 * 2560 * 151936:
            n -= 1
        return {"op": op, "n": n, "d_in": d_in, "d_out": d_out, "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "x": kind(), "y": kind(), "scale": kind()}
    if op == "quant_int4":
        cols = _width(rng, 64, 8192)
        return {"op": op, "rows": _log(rng, 1, 151936 * 1280 // cols), "cols": cols, "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.5, "x": kind(), "y": kind(), "scale": kind()}
    if op == "beam_step":
        V, beams = _log(rng, 1000, 152000), rng.randint(1, 16)
        return {"op": op, "batch": _log(rng, 1, max(1, min(64, 64 * 8 * 151936 // (V * beams)))), "beams": beams, "V": V, "logits": kind()}
    if op == "beam_reorder":
        beams, tensors = rng.randint(2, 16), rng.randint(1, 40)
        batch = _log(rng, 1, 64)
        most = 16 * 8 * 24 * 262144 // (batch * beams * tensors)
        return {"op": op, "batch": batch, "beams": beams, "tensors": tensors, "row_bytes": 4 * _log(rng, 1, min(262144, most // 4))}
    V = _log(rng, 1000, 152000)
    logits, fused = kind(), rng.random() < 0.5
    most = 4096 * 151936 * 4 // (V * _SIZE[logits] * (2 if fused else 3))
    return {"op": op, "n": _log(rng, 1, min(8192, most)), "V": V, "k": _log(rng, 1, 128), "logits": logits,
            "T": rng.choice([1.0, 1.5, 2.0, 4.0]), "tail": rng.random() < 0.5, "fused": fused}


# ---------------------------------------------------------------------------------------------------------------
# Sizes.

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def _code_ld(cols):
    return (cols + 31) // 32 * 16


def _groups(cols, group):
    return (cols + group - 1) // group


def _scale_ld(cols, group):
    return (_groups(cols, group) + 3) // 4 * 4


def work(case):
    op = case["op"]
    if op == "project_int4":
        n, k, o = case["n"], case["d_in"], case["d_out"]
        groups = o * _groups(k, case["group"])
        weights = o * k / 2 + groups * (_SIZE[case["scale"]] + (1 if case["zeros"] else 0))
        return {"bytes": weights + n * k * _SIZE[case["x"]] + n * o * _SIZE[case["y"]], "flops": 2 * n * k * o}
    if op == "quant_int4":
        r, c = case["rows"], case["cols"]
        groups = r * _groups(c, case["group"]) * (_SIZE[case["scale"]] + (1 if case["zeros"] else 0))
        return {"bytes": r * c * (_SIZE[case["x"]] + 0.5 + 0.5 + _SIZE[case["y"]]) + 2 * groups, "flops": 0}
    if op == "beam_step":
        rows = case["batch"] * case["beams"]
        return {"bytes": rows * case["V"] * _SIZE[case["logits"]] + rows * 42, "flops": 0}
    if op == "beam_reorder":
        rows, b = case["batch"] * case["beams"], case["beams"]
        # parents are uniform: a row changes unless it is its own parent, and is read if another row takes it
        moved = (1 - 1 / b) + (1 - (1 - 1 / b) ** (b - 1))
        return {"bytes": rows * moved * case["row_bytes"] * case["tensors"] + 4 * rows, "flops": 0}
    n, size = case["n"] * case["V"], _SIZE[case["logits"]]
    return {"bytes": n * size * (2 if case["fused"] else 3) + case["n"] * (8 * case["k"] + 12), "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits.

def _unpack(codes, rows, cols):
    q = torch.stack((codes & 15, codes >> 4), dim=2).view(rows, -1)
    return q[:, :cols]


def _spread(t, cols, group):
    """A value for each group to a value for each column."""
    return t[:, :_groups(cols, group)].repeat_interleave(group, dim=1)[:, :cols]


def _int4_values(s, rows, cols, group):
    q = _unpack(s["codes"], rows, cols).float()
    zero = _spread(s["zeros"], cols, group).float() if s["zeros"] is not None else 8.0
    return (q - zero) * _spread(s["scales"].float(), cols, group)


def _plain_project(s):
    w = _int4_values(s, s["o"], s["k"], s["group"])
    return {"y": (s["x"].float() @ w.t()).to(s["y_dtype"])}


def _plain_quant(s):
    rows, cols, group = s["rows"], s["cols"], s["group"]
    groups = _groups(cols, group)
    w = torch.nn.functional.pad(s["w"].float(), (0, groups * group - cols)).view(rows, groups, group)
    if s["asym"]:
        lo, hi = w.amin(dim=2).clamp(max=0.0), w.amax(dim=2).clamp(min=0.0)
        scale = (hi - lo) / lo.new_full((), 15.0)           # a tensor: division by a number goes by its reciprocal
    else:
        scale = w.abs().amax(dim=2) / w.new_full((), 7.0)
    scale = scale.to(s["scale_dtype"])
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    f = scale.float()
    if s["asym"]:
        zero = torch.round(-lo / f).clamp(0.0, 15.0)
        code = (torch.round(w / f[:, :, None]) + zero[:, :, None]).clamp(0.0, 15.0)
        value = (code - zero[:, :, None]) * f[:, :, None]
    else:
        value = torch.round(w / f[:, :, None]).clamp(-8.0, 7.0) * f[:, :, None]
    out = {"values": value.view(rows, -1)[:, :cols].to(s["y_dtype"]), "scales": scale}
    return out | ({"zeros": zero.to(torch.uint8)} if s["asym"] else {})


def _first_largest(x, k):
    """The k largest of each row of fp32 x and their indexes, ties to the lowest index."""
    x = x + 0.0                                         # -0 and 0 are equal
    bits = x.view(torch.int32).to(torch.int64)
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    last = x.shape[1] - 1
    key = order * (1 << 22) + (last - torch.arange(x.shape[1], device=x.device))
    best = key.topk(k, dim=1).values
    return last - (best & ((1 << 22) - 1))


def _plain_beam_step(s):
    batch, B, V, end = s["batch"], s["beams"], s["V"], s["end"]
    x = s["logits"].float()
    m = x.amax(dim=1, keepdim=True)
    lse = m.double() + (x - m).exp().sum(dim=1, keepdim=True).double().log()
    keep = min(B, V)
    index = _first_largest(x, keep)                                                         # [rows][keep]
    score = s["scores"].double()[:, None] + (x.gather(1, index).double() - lse)
    done = s["finished"]
    score[done] = NEG
    score[done, 0] = s["scores"][done].double()
    index[done, 0] = end
    score = torch.where(score > NEG, score, torch.full_like(score, NEG))
    flat = (torch.arange(B, device=x.device).repeat(batch)[:, None] * V + index).view(batch, B * keep)
    score = score.view(batch, B * keep)
    by_place = flat.argsort(dim=1)
    flat, score = flat.gather(1, by_place), score.gather(1, by_place)
    best = score.argsort(dim=1, descending=True, stable=True)[:, :B]
    flat, score = flat.gather(1, best), score.gather(1, best)
    parents, tokens = flat // V, flat % V
    row = parents + torch.arange(batch, device=x.device)[:, None] * B
    last = torch.stack((s["history"][row.view(-1), 1], s["tokens"][row.view(-1)]), dim=1)
    return {"scores": score.view(-1).float(), "tokens": tokens.view(-1).int(), "parents": parents.view(-1).int(), "history": last,
            "finished": done[row.view(-1)] | (tokens.view(-1) == end)}


def _plain_beam_reorder(s):
    B = s["beams"]
    rows = s["parents"].view(-1, B).long() + torch.arange(s["batch"], device=DEV)[:, None] * B
    for t in s["states"]:
        t.copy_(t[rows.view(-1)])
    return {f"state{i}": t for i, t in enumerate(s["states"])}


def _plain_distill(s):
    T, V = s["T"], s["V"]
    z = s["logits"].float() / T
    m = z.amax(dim=1, keepdim=True)
    e = (z - m).exp()
    lse = m + e.sum(dim=1, keepdim=True).log()
    on = (s["ids"] >= 0) & (s["ids"] < V)
    ids = torch.where(on, s["ids"], torch.zeros_like(s["ids"])).long()
    t = torch.where(on, s["teacher"].float() / T, torch.full_like(s["teacher"], NEG, dtype=torch.float32))
    any_on = on.any(dim=1, keepdim=True)
    log_q = z.gather(1, ids) - lse
    stats = torch.stack((s["logits"].float().amax(dim=1), e.sum(dim=1).log(), torch.zeros_like(lse[:, 0])), dim=1)
    if s["tail"]:
        log_p = t - s["teacher_lse"][:, None]
    else:
        tm = t.amax(dim=1, keepdim=True).clamp(min=-3e38)
        log_p = t - (tm + (t - tm).exp().sum(dim=1, keepdim=True).log())
        log_p = torch.where(any_on, log_p, torch.full_like(log_p, NEG))
    p = log_p.exp()
    loss = torch.where(p > 0, p * (log_p - log_q), torch.zeros_like(p)).sum(dim=1)
    q = (z - lse).exp()
    if s["tail"]:
        rest = (1.0 - p.double().sum(dim=1)).clamp(min=0.0).float()
        off = torch.ones_like(z, dtype=torch.bool)
        row = torch.arange(z.shape[0], device=z.device)[:, None].expand_as(ids)
        off[row[on], ids[on]] = False
        mass = torch.where(off, e, torch.zeros_like(e)).sum(dim=1)
        log_rest = (m[:, 0] + mass.log()) - lse[:, 0]
        stats[:, 2] = log_rest
        loss = loss + torch.where(rest > 0, rest * (rest.log() - log_rest), torch.zeros_like(rest))
        factor = torch.where(rest > 0, 1.0 - (rest.log() - log_rest).exp(), torch.ones_like(rest))
        g = torch.where(off, q * factor[:, None], q)
    else:
        g = torch.where(any_on, q, torch.zeros_like(q))
    g = g.scatter_add(1, ids, -p)
    w = s["weight"] * (s["scale"] * T)
    g = torch.where(w[:, None] != 0, g * w[:, None], torch.zeros_like(g))
    return {"loss": loss * (T * T), "dlogits": g.to(s["logits"].dtype)} | ({} if s["fused"] else {"stats": stats})


# ---------------------------------------------------------------------------------------------------------------
# Inputs.

def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _below(g, high, *shape, low=0):
    return torch.randint(low, high, shape, generator=g, device=DEV, dtype=torch.int32)


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _activations(g, n, d):
    """Hidden states: a few columns far larger than the others, as a residual stream has them."""
    x = _normal(g, n, d)
    return x.mul_(torch.exp(0.5 * _normal(g, d)) * (1 + 20 * (_uniform(g, d) < 0.004)))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "project_int4":
        n, k, o, group = case["n"], case["d_in"], case["d_out"], case["group"]
        s |= {"n": n, "k": k, "o": o, "group": group, "y_dtype": _DT[case["y"]]}
        s["x"] = _activations(g, n, k).to(_DT[case["x"]])
        ld, sld = _code_ld(k), _scale_ld(k, group)
        # codes as rounding normal weights gives them: all sixteen in use, the middle ones most
        s["codes"] = torch.zeros((o, ld), dtype=torch.uint8, device=DEV)
        for at in range(0, o, 32768):
            part = _normal(g, min(32768, o - at), 2 * ld, std=3.0).add_(8.0).round_().clamp_(0, 15).to(torch.uint8)
            part[:, k:] = 0
            s["codes"][at:at + 32768] = part[:, 0::2] | (part[:, 1::2] << 4)
        scales = torch.ones((o, sld), device=DEV)
        scales[:, :_groups(k, group)] = k ** -0.5 / 3 * torch.exp(0.3 * _normal(g, o, _groups(k, group)))
        s["scales"] = scales.to(_DT[case["scale"]])
        s["zeros"] = _below(g, 11, o, sld, low=6).to(torch.uint8) if case["zeros"] else None
        return s
    if op == "quant_int4":
        r, c = case["rows"], case["cols"]
        s |= {"rows": r, "cols": c, "group": case["group"], "asym": case["zeros"], "y_dtype": _DT[case["y"]], "scale_dtype": _DT[case["scale"]]}
        s["w"] = (_normal(g, r, c, std=c ** -0.5) * torch.exp(0.3 * _normal(g, r, 1))).to(_DT[case["x"]])
        return s
    if op == "beam_step":
        batch, B, V = case["batch"], case["beams"], case["V"]
        rows = batch * B
        s |= {"batch": batch, "beams": B, "V": V, "end": 2}
        x = _normal(g, rows, V, std=2.0)
        peaks = _below(g, V, rows, 12).long()
        x.scatter_(1, peaks, 6.0 + 2.0 * _normal(g, rows, 12))
        s["logits"] = x.to(_DT[case["logits"]])
        s["scores"] = -12.0 * _uniform(g, rows)
        s["tokens"] = _below(g, V, rows)
        s["history"] = _below(g, V, rows, 2)
        s["finished"] = _uniform(g, rows) < 0.1
        return s
    if op == "beam_reorder":
        batch, B = case["batch"], case["beams"]
        s |= {"batch": batch, "beams": B}
        words = case["row_bytes"] // 4
        s["states"] = [_below(g, 1 << 30, batch * B, words) for _ in range(case["tensors"])]
        s["parents"] = _below(g, B, batch * B)
        return s
    n, V, k, T = case["n"], case["V"], case["k"], case["T"]
    s |= {"n": n, "V": V, "k": k, "T": T, "tail": case["tail"], "fused": case["fused"]}
    # the teacher's most likely tokens: distinct, spread over the vocabulary, falling logits; short lists end in -1
    step = _below(g, max(2, V // k), n, 1, low=1)
    ids = (_below(g, V, n, 1) + step * torch.arange(k, device=DEV, dtype=torch.int32)) % V
    teacher = 9.0 - 1.5 * torch.log1p(torch.arange(k, device=DEV).float()) + 0.5 * _normal(g, n, k)
    z = _normal(g, n, V, std=1.5)
    z.scatter_(1, ids.long(), 0.7 * teacher + _normal(g, n, k))
    s["logits"] = z.to(_DT[case["logits"]])
    del z
    length = torch.where(_uniform(g, n, 1) < 0.1, _below(g, k + 1, n, 1), torch.full((n, 1), k, device=DEV, dtype=torch.int32))
    ids = torch.where(torch.arange(k, device=DEV) < length, ids, torch.full_like(ids, -1))
    s["ids"], s["teacher"] = ids.int().contiguous(), teacher.to(_DT[case["logits"]])
    if case["tail"]:
        t = s["teacher"].float() / T
        s["teacher_lse"] = torch.logsumexp(t, dim=1) + 0.02 + 0.4 * _uniform(g, n)
    # rows of padding weigh nothing
    s["weight"] = (_uniform(g, n) >= 0.05).float() * (0.5 + _uniform(g, n))
    s["scale"] = 1.0 / n
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass.

def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


_PLAIN = {"project_int4": _plain_project, "quant_int4": _plain_quant, "beam_step": _plain_beam_step, "beam_reorder": _plain_beam_reorder,
          "distill": _plain_distill}


def _own_project(s):
    import hashed_gram_embedding_ngram_amd as ng
    if "handle" not in s:  # the weights that a serving program holds
        s["handle"] = ng.Int4(s["codes"], s["scales"], s["o"], s["k"], s["group"], zeros=s["zeros"])
    return {"y": ng.ngram_project_int4(s["x"], s["handle"], dtype=s["y_dtype"])}


def _own_quant(s):
    import hashed_gram_embedding_ngram_amd as ng
    q = ng.ngram_quant_int4(s["w"], s["group"], zeros=s["asym"], scale_dtype=s["scale_dtype"])
    groups = _groups(s["cols"], s["group"])
    out = {"values": ng.ngram_dequant_int4(q, dtype=s["y_dtype"]), "scales": q.scales[:, :groups]}
    return out | ({"zeros": q.zeros[:, :groups]} if s["asym"] else {})


def _own_beam_step(s):
    import hashed_gram_embedding_ngram_amd as ng
    out = ng.ngram_beam_step(s["logits"], s["scores"], s["beams"], tokens=s["tokens"], history=s["history"], finished=s["finished"],
                             end_token=s["end"])
    return {"scores": out.scores, "tokens": out.tokens, "parents": out.parents, "history": out.history, "finished": out.finished}


def _own_beam_reorder(s):
    import hashed_gram_embedding_ngram_amd as ng
    if "handle" not in s:  # the list of states that a decoding program keeps
        s["handle"] = ng.BeamStates(s["states"])
    ng.ngram_beam_reorder(s["handle"], s["parents"], s["beams"])
    return {f"state{i}": t for i, t in enumerate(s["states"])}


def _own_distill(s):
    import hashed_gram_embedding_ngram_amd as ng
    a = {"temperature": s["T"], "teacher_lse": s.get("teacher_lse"), "weight": s["weight"], "scale": s["scale"]}
    if s["fused"]:
        out = ng.ngram_distill(s["logits"], s["teacher"], s["ids"], grad=True, **a)
        return {"loss": out.loss, "dlogits": out.dlogits}
    out = ng.ngram_distill(s["logits"], s["teacher"], s["ids"], keep_stats=True, temperature=s["T"], teacher_lse=s.get("teacher_lse"))
    return {"loss": out.loss, "dlogits": ng.ngram_distill_grad(s["logits"], s["teacher"], s["ids"], out.stats, **a), "stats": out.stats}


_OWN = {"project_int4": _own_project, "quant_int4": _own_quant, "beam_step": _own_beam_step, "beam_reorder": _own_beam_reorder,
        "distill": _own_distill}


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits.

def _x_project(s, case):
    k, group = s["k"], s["group"]
    groups = _groups(k, group)
    x = s["x"].double()
    parts = []
    for at in range(0, s["o"], 16384):
        codes = s["codes"][at:at + 16384]
        w = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = (codes % 16).double(), (codes // 16).double()
        y = torch.zeros((x.shape[0], codes.shape[0]), dtype=torch.float64, device=DEV)
        for i in range(groups):
            cut = slice(i * group, min((i + 1) * group, k))
            zero = s["zeros"][at:at + 16384, i].double() if s["zeros"] is not None else torch.full_like(w[:, 0], 8.0)
            y += (x[:, cut] @ (w[:, cut] - zero[:, None]).t().contiguous()) * s["scales"][at:at + 16384, i].double()
        parts.append(y)
    return {"y": torch.cat(parts, dim=1)}


def _x_quant(s, case):
    """The format's steps, each result rounded to the type that holds it, in float64."""
    rows, cols, group = s["rows"], s["cols"], s["group"]
    groups = _groups(cols, group)
    single = lambda t: t.float().double()  # noqa: E731
    values = torch.empty((rows, cols), dtype=torch.float64, device=DEV)
    scales = torch.empty((rows, groups), dtype=torch.float64, device=DEV)
    zeros = torch.empty_like(scales)
    for i in range(groups):
        w = s["w"][:, i * group:min((i + 1) * group, cols)].double()
        if s["asym"]:
            low, high = torch.clamp(w.min(dim=1).values, max=0), torch.clamp(w.max(dim=1).values, min=0)
            f = single(single(high - low) / 15)
        else:
            f = single(w.abs().max(dim=1).values / 7)
        f = f.to(s["scale_dtype"]).double()
        f[f == 0] = 1
        zero = torch.clamp(torch.round(single(-low / f)), 0, 15) if s["asym"] else torch.full_like(f, 8)
        code = torch.clamp(torch.round(single(w / f[:, None])) + zero[:, None], 0, 15)
        values[:, i * group:i * group + w.shape[1]] = f[:, None] * (code - zero[:, None])
        scales[:, i], zeros[:, i] = f, zero
    return {"values": values, "scales": scales} | ({"zeros": zeros.to(torch.uint8)} if s["asym"] else {})


def _x_beam_step(s, case):
    batch, B, V, end = s["batch"], s["beams"], s["V"], s["end"]
    out = {"scores": [], "tokens": [], "parents": [], "history": [], "finished": []}
    column = torch.arange(V, device=DEV)
    for e in range(batch):
        cut = slice(e * B, (e + 1) * B)
        x = s["logits"][cut].double()
        score = s["scores"][cut].double()[:, None] + x - torch.logsumexp(x, dim=1, keepdim=True)
        done = s["finished"][cut]
        held = torch.where(column[None] == end, s["scores"][cut].double()[:, None], torch.full_like(x, NEG))
        score = torch.where(done[:, None], held, score).reshape(-1)
        for _ in range(B):
            best = int(torch.nonzero(score == score.max())[0])
            b, t = best // V, best % V
            out["scores"].append(float(score[best]))
            out["tokens"].append(t)
            out["parents"].append(b)
            out["history"].append([int(s["history"][e * B + b, 1]), int(s["tokens"][e * B + b])])
            out["finished"].append(bool(done[b]) or t == end)
            score[best] = NEG
    types = {"scores": torch.float64, "finished": torch.bool}
    return {name: torch.tensor(v, dtype=types.get(name, torch.int32), device=DEV) for name, v in out.items()}


def _x_beam_reorder(s, case):
    B = s["beams"]
    out = {}
    for i, t in enumerate(s["states"]):
        new = torch.empty_like(t)
        for e in range(s["batch"]):
            new[e * B:(e + 1) * B] = torch.index_select(t[e * B:(e + 1) * B], 0, s["parents"][e * B:(e + 1) * B])
        out[f"state{i}"] = new
    return out


def _x_distill(s, case):
    T, V, n = s["T"], s["V"], s["n"]
    loss = torch.empty(n, dtype=torch.float64, device=DEV)
    stats = torch.zeros((n, 3), dtype=torch.float64, device=DEV)
    grad = torch.empty((n, V), dtype=torch.float64, device=DEV)
    for at in range(0, n, 256):
        cut = slice(at, min(at + 256, n))
        log_q = torch.log_softmax(s["logits"][cut].double() / T, dim=1)
        rows = log_q.shape[0]
        # the teacher over the whole vocabulary, what its list leaves out apart
        ids = s["ids"][cut].long()
        slot = torch.where(ids < 0, torch.full_like(ids, V), ids)
        t = s["teacher"][cut].double() / T
        t[ids < 0] = NEG
        live = (ids >= 0).any(dim=1)
        if s["tail"]:
            p = torch.exp(t - s["teacher_lse"][cut].double()[:, None])
        else:
            p = torch.nan_to_num(torch.softmax(t, dim=1), nan=0.0)
        P = torch.zeros((rows, V + 1), dtype=torch.float64, device=DEV).scatter_add_(1, slot, p)[:, :V]
        part = torch.xlogy(P, P) - P * log_q
        row_loss = part.sum(dim=1)
        g = torch.exp(log_q) * (live[:, None] if not s["tail"] else 1.0)
        if s["tail"]:
            listed_ = torch.zeros((rows, V + 1), dtype=torch.bool, device=DEV).scatter_(1, slot, True)[:, :V]
            log_rest = torch.logsumexp(log_q.masked_fill(listed_, NEG), dim=1)
            rest = torch.clamp(1 - p.sum(dim=1), min=0)
            row_loss = row_loss + torch.xlogy(rest, rest) - torch.where(rest > 0, rest * log_rest, torch.zeros_like(rest))
            ratio = torch.where(rest > 0, rest / torch.exp(log_rest), torch.zeros_like(rest))
            g = torch.where(listed_, g, g * (1 - ratio[:, None]))
            stats[cut, 2] = log_rest
        w = s["weight"][cut].double()[:, None]
        grad[cut] = (g - P) * w * (s["scale"] * T)
        loss[cut] = row_loss * T * T
        stats[cut, 0] = s["logits"][cut].double().max(dim=1).values
        stats[cut, 1] = torch.logsumexp((s["logits"][cut].double() - stats[cut, :1]) / T, dim=1)
    return {"loss": loss, "dlogits": grad} | ({} if s["fused"] else {"stats": stats})


_EXACT = {"project_int4": _x_project, "quant_int4": _x_quant, "beam_step": _x_beam_step, "beam_reorder": _x_beam_reorder,
          "distill": _x_distill}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)
