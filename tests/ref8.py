"""Plain float64 forms of the 8-bit norm, product and optimiser step, from the
formulas in include/ngram.h, in numpy and with no code of the library."""
import numpy as np

U = 2.0 ** -24                  # half an ulp of fp32 at 1
BLOCK = 128
MASK = (1 << 64) - 1


def ceil_div(a, b):
    return -(-a // b)


def code_shape(rows, cols):
    return rows, ceil_div(cols, BLOCK) * BLOCK


def scale_cols(cols):
    return ceil_div(ceil_div(cols, BLOCK), 4) * 4


def decode(codes):
    """The numbers that E4M3 bytes encode, float64."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7), m / 8.0 * 2.0 ** -6)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def exponent(amax):
    """Smallest e >= -126 with amax <= 448 * 2^e; 0 where amax is 0."""
    f, k = np.frexp(np.asarray(amax, dtype=np.float64))
    e = np.maximum(np.where(f <= 0.875, k - 9, k - 8), -126)
    return np.where(np.asarray(amax) > 0, e, 0)


def step_at(a):
    """The spacing of E4M3 values just above magnitude a (scaled)."""
    _, k = np.frexp(a)
    return 2.0 ** np.maximum(np.where(a > 0, k - 4, -9), -9)


def encode(x):
    """E4M3 bytes of |x| <= 448, nearest, ties to even; not finite: NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    s = step_at(a)
    q = np.rint(a / s) * s                          # rint: ties to even multiples, which are even codes
    return np.where(np.isfinite(x), code_of(q) | np.where(np.signbit(x), 0x80, 0), 0x7F).astype(np.uint8)


def code_of(q):
    """The byte of a non-negative E4M3 value."""
    f, k = np.frexp(q)
    return np.where(q >= 2.0 ** -6, ((k + 6) << 3) + np.rint((f * 2 - 1) * 8).astype(np.int64),
                    np.rint(q * 512).astype(np.int64)).astype(np.int64)


def block_max(x):
    """Largest finite magnitude of each row's blocks of 128 (x padded)."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    return a.reshape(x.shape[0], -1, BLOCK).max(axis=2)


def padded(x):
    out = np.zeros(code_shape(*x.shape))
    out[:, :x.shape[1]] = x
    return out


def quant(x, tile=False):
    """(codes, scale bytes) of float64 x [rows][cols] in the stored layout."""
    rows, cols = x.shape
    p = padded(x)
    am = block_max(p)
    if tile:
        full = np.zeros((ceil_div(rows, BLOCK) * BLOCK, am.shape[1]))
        full[:rows] = am
        am = full.reshape(-1, BLOCK, am.shape[1]).max(axis=1)
    e = exponent(am)
    scales = np.full((e.shape[0], scale_cols(cols)), 127, dtype=np.uint8)
    scales[:, :e.shape[1]] = e + 127
    per_row = np.repeat(e, BLOCK, axis=0)[:rows] if tile else e
    with np.errstate(invalid="ignore"):
        codes = encode(p / 2.0 ** np.repeat(per_row, BLOCK, axis=1))
    codes[:, cols:] = 0
    return codes, scales


def values(codes, scales, cols, tile=False):
    rows = codes.shape[0]
    s = 2.0 ** (scales[:, :ceil_div(cols, BLOCK)].astype(np.float64) - 127)
    if tile:
        s = np.repeat(s, BLOCK, axis=0)[:rows]
    return (decode(codes) * np.repeat(s, BLOCK, axis=1))[:, :cols]


def bf16(x):
    """fp32 rounded to bf16, nearest, ties to even, as fp32 (NaN stays NaN)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def bf16_half_step(x):
    """Half a bf16 ulp at |x|."""
    _, k = np.frexp(np.abs(x))
    return 2.0 ** (np.maximum(k, -125).astype(np.float64) - 9)


def add_norm(x, residual, gamma, eps):
    """(s, r, y) in float64 from fp32 x, residual and gamma; s exactly as stored."""
    s = bf16(x.astype(np.float32) + residual.astype(np.float32)).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        r = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
        return s, r, s * r[:, None] * gamma.astype(np.float64)


def add_norm_grad(dy, s, r, gamma, dsum):
    """(dx, dgamma, and the sums of absolute terms of each)."""
    h = dy * gamma
    r = r[:, None]
    d = dy.shape[1]
    dx = r * h - s * (r ** 3 / d) * (h * s).sum(axis=1, keepdims=True) + dsum
    size = np.abs(r * h) + np.abs(s) * (r ** 3 / d) * np.abs(h * s).sum(axis=1, keepdims=True) + np.abs(dsum)
    t = dy * s * r
    return dx, t.sum(axis=0), size, np.abs(t).sum(axis=0)


def splitmix64(x):
    with np.errstate(over="ignore"):
        z = np.asarray(x, dtype=np.uint64) + np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def random_words(seed, step, index):
    with np.errstate(over="ignore"):
        key = splitmix64(splitmix64(np.uint64(seed & MASK)) + np.uint64(step))
        z = splitmix64(key + np.asarray(index, dtype=np.uint64) // np.uint64(2))
    return np.where(np.asarray(index) % 2 == 1, z >> np.uint64(32), z & np.uint64(0xFFFFFFFF)).astype(np.int64)


def round_up(a, chance, step):
    """Multiples of `step` around a >= 0: the upper one where the fraction plus the chance in [0, 1) passes one."""
    return np.floor(a / step + chance) * step


def adamw(p, g, m, v, h, step):
    """Unrounded (p', m', v') in float64; v is the second moment."""
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    mh, vh = m / (1 - h["beta1"] ** step), v / (1 - h["beta2"] ** step)
    return p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * mh / (np.sqrt(vh) + h["eps"]), m, v


def pack_state(x, word20, positive):
    """(codes, scale bytes, values) of rows x [rows][128 nb], rounded by 20 random bits."""
    e = exponent(block_max(x))
    scale = np.repeat(2.0 ** e, BLOCK, axis=1)
    a = np.abs(x) / scale
    q = np.minimum(round_up(a, word20 * 2.0 ** -20, step_at(a)), 448.0)
    if positive:
        q = np.where(a > 0, np.maximum(q, 2.0 ** -9), q)
    return (code_of(q) | np.where(x < 0, 0x80, 0)).astype(np.uint8), (e + 127).astype(np.uint8), np.where(x < 0, -q, q) * scale


def bf16_random(p, word16):
    _, k = np.frexp(np.abs(p))
    step = 2.0 ** (np.maximum(k, -125).astype(np.float64) - 8)
    return np.where(p < 0, -1.0, 1.0) * round_up(np.abs(p), word16 * 2.0 ** -16, step)
