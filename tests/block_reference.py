"""Plain 64-bit forms of the 8-bit block operators, for the tests alone (numpy on the CPU;
nothing here is shared with the library). E4M3 codes are uint8, BF16 values are float64
numbers that BF16 holds."""
import numpy as np
import torch

BLOCK, E4M3_MAX = 128, 448.0


def bf16(a):
    """Rounded to BF16 (nearest even), as float64."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(torch.float32).to(torch.bfloat16).double().numpy()


def to_bf16_cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def _decode_table():
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = np.nan if (c & 0x7F) == 0x7F else (-v if s else v)
    return t


DECODE = _decode_table()
_GRID = DECODE[:0x7F]  # the non-negative finite values, ascending with the code


def nearest_e4m3(v):
    """Codes of the nearest E4M3 value, ties to the even code, saturated (finite float64 input)."""
    a = np.minimum(np.abs(v), E4M3_MAX)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | (np.signbit(v) * 0x80)).astype(np.uint8)


def nb(n):
    return -(-n // BLOCK)


def block_amax(x):
    return np.stack([np.abs(x[:, b * BLOCK:(b + 1) * BLOCK]).max(1) for b in range(nb(x.shape[1]))], 1)


def expand(scales, cols):
    """[rows, blocks] to [rows, cols]."""
    return np.repeat(scales, BLOCK, axis=1)[:, :cols]


def codes32(x, power=False):
    """(codes, FP32 scales) of finite rows whose values FP32 holds, the scale and the product with
    448 / amax rounded to FP32 as the operator's formula has them."""
    amax = block_amax(x).astype(np.float32)
    used = np.maximum(amax, np.float32(2.0 ** -110))
    if power:
        m, e = np.frexp(used.astype(np.float64) / 448.0)
        e = np.where(m == 0.5, e - 1, e)
        scale = (2.0 ** e.astype(np.float64)).astype(np.float32)
        mult = (2.0 ** (-e.astype(np.float64))).astype(np.float32)
    else:
        scale, mult = used / np.float32(448.0), np.float32(448.0) / used
    scale, mult = np.where(amax == 0, np.float32(1), scale), np.where(amax == 0, np.float32(1), mult)
    return nearest_e4m3((x.astype(np.float32) * expand(mult, x.shape[1])).astype(np.float64)), scale


def silu_up(x):
    f = x.shape[1] // 2
    with np.errstate(over="ignore"):
        return x[:, :f] / (1.0 + np.exp(-x[:, :f])) * x[:, f:]


def real_rows(q, s):
    return DECODE[q] * expand(s.astype(np.float64), q.shape[1])


def real_weights(q, s):
    return DECODE[q] * expand(np.repeat(s.astype(np.float64), BLOCK, axis=0)[: q.shape[0]], q.shape[1])


def random_codes(rng, *shape):
    """Finite codes of values about N(0, 60)."""
    return nearest_e4m3(rng.normal(0, 60, shape))


def route(x, bias, K, scoring, groups, kept, rule, renorm, scale):
    """(ids, weights) of one row of logits, in 64 bits."""
    x = x.astype(np.float64)
    nan = np.isnan(x)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-np.where(nan, 0.0, x)))
        s[nan] = 0.0
    else:
        m = np.max(np.where(nan, -np.inf, x))
        if m == -np.inf:
            s = np.zeros_like(x)
        elif m == np.inf:
            s = (x == np.inf).astype(np.float64)
            s /= s.sum()
        else:
            s = np.where(nan, 0.0, np.exp(np.where(nan, -np.inf, x) - m))
            s /= s.sum()
    key = s if bias is None else s + bias.astype(np.float64)
    key = np.where(nan | np.isnan(key), -np.inf, key)
    size = x.size // groups
    if groups > 1:
        by = -np.sort(-key.reshape(groups, size), axis=1)
        with np.errstate(invalid="ignore"):
            v = by[:, 0] + by[:, 1] if rule == "top2" and size > 1 else by[:, 0]
        v = np.where(np.isnan(v), -np.inf, v)
        order = sorted(range(groups), key=lambda g: (-v[g], g))[:kept]
        allowed = [g * size + i for g in sorted(order) for i in range(size)]
    else:
        allowed = list(range(x.size))
    ids = sorted(allowed, key=lambda e: (-key[e], e))[:K]
    w = s[ids]
    if renorm:
        w = w / w.sum() if w.sum() != 0 else np.zeros_like(w)
    return np.array(ids, np.int32), w * scale


def block_norm(y, r, post, gate, nxt, alpha, eps):
    """(h, n) before any rounding; gate broadcast to y's shape or None."""
    rms = lambda v: v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    u = y if post is None else rms(y) * post
    if gate is not None:
        u = gate * u
    h = r + alpha * u
    return h, rms(h) * nxt
