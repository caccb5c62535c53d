"""Plain float64 forms of the vocabulary's operators (4-bit weights, beam
search, distillation), from the formulas in include/ngram.h, in numpy and with
no code of the library."""
import numpy as np

U = 2.0 ** -24                  # half an ulp of fp32 at 1


def bf16(x):
    """x (fp32) rounded to bf16, nearest, ties to even, as fp32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32("nan"), r).astype(np.float32)


def half_step(x, bf):
    """Half the distance of neighbours at |x| in bf16 or fp32 (subnormals aside)."""
    _, e = np.frexp(np.abs(x))
    return 2.0 ** (np.maximum(e, -125) - (9 if bf else 25))


# 4 bits ------------------------------------------------------------------------------------------------------

def code_ld(cols):
    return -(-cols // 32) * 16


def groups_of(cols, group):
    return -(-cols // group)


def scale_ld(cols, group):
    return -(-groups_of(cols, group) // 4) * 4


def pack(q, cols):
    """Codes [rows][cols] to bytes; the places past cols hold 15."""
    full = np.full((q.shape[0], 2 * code_ld(cols)), 15, np.uint8)
    full[:, :cols] = q
    return full[:, 0::2] | (full[:, 1::2] << 4)


def unpack(codes, cols):
    q = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    return q[:, :cols]


def values4(codes, scales, zeros, cols, group):
    """What a 4-bit matrix stands for, float64; scales and zeros [rows][>= groups]."""
    g = np.arange(cols) // group
    z = 8.0 if zeros is None else zeros[:, g].astype(np.float64)
    return (unpack(codes, cols).astype(np.float64) - z) * scales[:, g].astype(np.float64)


def quant4(x, group, asym, bf):
    """(codes unpacked, scales, zeros or None): the format's fp32 steps."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    n = groups_of(cols, group)
    q, s, z = np.zeros((rows, cols), np.uint8), np.zeros((rows, n), np.float32), np.full((rows, n), 8, np.uint8)
    with np.errstate(all="ignore"):
        for g in range(n):
            w = x[:, g * group:(g + 1) * group]
            lo, hi = np.minimum(w, 0).min(axis=1), np.maximum(w, 0).max(axis=1)
            f = (hi - lo) / np.float32(15) if asym else np.abs(w).max(axis=1) / np.float32(7)
            f = bf16(f) if bf else f
            bad = ~np.isfinite(w).all(axis=1) | ~np.isfinite(f)
            f = np.where(f == 0, np.float32(1), f).astype(np.float32)
            zero = np.clip(np.rint(-lo / f), 0, 15) if asym else np.full(rows, 8, np.float32)
            code = np.clip(np.rint(w / f[:, None]) + zero[:, None], 0, 15)
            q[:, g * group:(g + 1) * group] = np.where(bad[:, None], 8, np.where(bad[:, None], 0, code)).astype(np.uint8)
            s[:, g], z[:, g] = np.where(bad, np.float32("nan"), f), np.where(bad, 8, zero).astype(np.uint8)
    return q, s, (z if asym else None)


# softmax error -----------------------------------------------------------------------------------------------

def sum_error(z, c, lanes=256):
    """A bound of the relative error of a row's sum of exp(c (z - max)), c = 1 / T, in fp32: per term the exponent's
    difference, its two products and 2 ulp of exp2; then additions, at most ceil(V / lanes) + 8 of a vector in a lane,
    each lane rescaled once a vector, and 16 to join."""
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        m = z.max(axis=-1, keepdims=True)
        a = np.where(np.isneginf(z), 0.0, (z - m) * c)
        e = np.where(np.isneginf(z), 0.0, np.exp(a))
    V = z.shape[-1]
    total = e.sum(axis=-1)
    term = np.where(total > 0, (e * (4 * np.abs(a) + 6)).sum(axis=-1) / np.where(total > 0, total, 1.0), 0.0)     # of nothing: none
    return U * (term + 3 * (V / lanes) + 40)


def log_softmax(z):
    """Relative to the largest value, so that rows of huge values keep their differences."""
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        d = z - z.max(axis=-1, keepdims=True)
        return d - np.log(np.exp(d).sum(axis=-1, keepdims=True))


def log_sum(z):
    z = np.asarray(z, np.float64)
    m = z.max(axis=-1, keepdims=True)
    with np.errstate(all="ignore"):
        return (m + np.log(np.exp(z - m).sum(axis=-1, keepdims=True)))[..., 0]


# beams -------------------------------------------------------------------------------------------------------

def beam_step(logits, scores, beams, tokens=None, history=None, finished=None, end=-1):
    """Dict of the outputs, and under "gap" the smallest distance of the scores of two candidates that were compared and
    decided (of different beams)."""
    rows, V = logits.shape
    x = np.asarray(logits, np.float64)
    out = {k: [] for k in ("scores", "tokens", "parents", "history", "finished")}
    gap = np.inf
    for e in range(rows // beams):
        cand = []
        for b in range(beams):
            r = e * beams + b
            if not scores[r] > -np.inf:
                continue
            if finished is not None and finished[r]:
                cand.append((float(scores[r]), b, end))
                continue
            if np.isnan(x[r]).any() or np.isposinf(x[r]).any() or np.isneginf(x[r]).all():
                continue
            s = float(scores[r]) + log_softmax(x[r])
            order = np.argsort(-x[r], kind="stable")[:beams + 1]
            cand += [(s[t], b, int(t)) for t in order if s[t] > -np.inf]
        cand.sort(key=lambda c: (-c[0], c[1] * V + c[2]))
        for i in range(min(beams, len(cand) - 1)):
            if cand[i][1] != cand[i + 1][1] and cand[i][0] != cand[i + 1][0]:
                gap = min(gap, cand[i][0] - cand[i + 1][0])
        for i in range(beams):
            s, b, t = cand[i] if i < len(cand) else (-np.inf, -1, -1)
            out["scores"].append(s)
            out["tokens"].append(t)
            out["parents"].append(b)
            r = e * beams + b
            out["history"].append((history[r][1], tokens[r]) if history is not None and b >= 0 else (-1, -1))
            out["finished"].append(b >= 0 and bool((finished is not None and finished[r]) or t == end))
    out = {k: np.array(v) for k, v in out.items()}
    out["gap"] = gap
    return out


# distillation ------------------------------------------------------------------------------------------------

def distill(z, t, ids, T, lse_t=None, weight=None, scale=1.0):
    """(loss, stats, gradient, pieces): float64; pieces has q, a, p spread over V, and the rest's ratio."""
    z, t = np.asarray(z, np.float64) / T, np.asarray(t, np.float64) / T
    n, V = z.shape
    loss, stats, grad = np.zeros(n), np.zeros((n, 3)), np.zeros((n, V))
    pieces = {"q": np.zeros((n, V)), "a": np.ones((n, V)), "p": np.zeros((n, V)), "ratio": np.zeros(n), "rest": np.zeros(n)}
    for i in range(n):
        with np.errstate(all="ignore"):
            log_q = log_softmax(z[i])
            q = np.exp(log_q)
            on = (ids[i] >= 0) & (ids[i] < V)
            idx, ti = ids[i][on], t[i][on]
            if lse_t is not None:
                log_p = ti - float(lse_t[i])
            else:
                log_p = log_softmax(ti) if on.any() and not np.isneginf(ti).all() else np.full(ti.shape, -np.inf)
            p = np.exp(log_p)
            part = np.where(p == 0, 0.0, p * (log_p - log_q[idx]))
            total, a, ratio, rest, log_rest = part.sum(), np.full(V, p.sum()), 0.0, 0.0, 0.0
            if lse_t is not None:
                off = np.ones(V, bool)
                off[idx] = False
                rest = 1.0 - p.sum()
                log_rest = log_sum(np.where(off, log_q, -np.inf)) if off.any() and not np.isneginf(log_q[off]).all() else -np.inf
                if rest > 0:
                    total += rest * (np.log(rest) - log_rest)
                    ratio = rest / np.exp(log_rest) if log_rest > -np.inf else 0.0
                a = np.where(off, 1.0 - ratio, 1.0)
            P = np.zeros(V)
            np.add.at(P, idx, p)
            w = (1.0 if weight is None else float(weight[i])) * scale * T
            loss[i] = total * T * T if not np.isnan(log_q).any() else np.nan
            stats[i] = z[i].max() * T, -log_q.max(), log_rest
            grad[i] = 0.0 if w == 0 else w * (a * q - P)
            for k, v in (("q", q), ("a", a), ("p", P), ("ratio", ratio), ("rest", rest)):
                pieces[k][i] = v
    return loss, stats, grad, pieces
