"""The AdamW step and its 8-bit states in float64, from their definitions: test infrastructure."""
import numpy as np

import oracle

BLOCK = 256


def step(p, g, m, v, t, lr, beta1, beta2, eps, wd, scale=1.0):
    """(p', m', v') of one step, all float64."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** t), v / (1 - beta2 ** t)
    return p - lr * wd * p - lr * mh / (np.sqrt(vh) + eps), m, v


def words(seed, offset, tensor, n):
    """The random word of each element of tensor number `tensor`."""
    return oracle.rand_words(seed, offset, tensor, 0, n).astype(np.uint64)


def exponent(x):
    """The biased fp32 exponent of |x| (0 for 0 and for values below 2^-126)."""
    _, e = np.frexp(np.abs(np.asarray(x, np.float64)))
    return np.where(np.abs(x) > 0, np.maximum(e + 126, 0), 0)


def base(x, span):
    """The exponent byte of every block."""
    e = exponent(x)
    pad = (-len(e)) % BLOCK
    top = np.pad(e, (0, pad)).reshape(-1, BLOCK).max(1)
    return np.maximum(top - span, 0)


def value(code, exps, signed):
    """What codes stand for: 2^(E - 127) (1 + f / 8), with E and f the upper and the lowest three bits of
    c + 8 b (E = 0: f 2^-129)."""
    code = np.asarray(code, np.int64)
    c = code & 127 if signed else code
    k = c + 8 * np.repeat(np.asarray(exps, np.int64), BLOCK)[:len(code)]
    E, f = k >> 3, k & 7
    x = np.where(E > 0, np.ldexp(1 + f / 8.0, (E - 127).astype(np.int32)), np.ldexp(f / 8.0, -126))
    x = np.where(c == 0, 0.0, x)
    return np.where(signed & (code > 127), -x, x)


def grid(x, exps, signed, rand=None):
    """The value that x is rounded to on its block's grid: by the 16 random bits upwards (unsigned), or to the
    nearest with ties to even (signed); values above 0 stay at or above the first code (unsigned)."""
    x = np.asarray(x, np.float64)
    mag = np.abs(x)
    E = np.maximum(exponent(mag), 1)
    ulp = np.ldexp(1.0, (E - 130).astype(np.int32))
    q = np.floor(mag / ulp + rand / 65536.0) if not signed else np.rint(mag / ulp)
    y = q * ulp
    low = value(np.ones(len(x), np.int64), exps, False)  # code 1
    y = np.where(y < low, 0.0 if signed else low, y)
    top = value(np.full(len(x), 127 if signed else 255, np.int64), exps, False)
    return np.where(mag == 0, 0.0, np.sign(x) * np.minimum(y, top))


def bf16_by_word(p, word):
    """p to bf16 with the word's upper 16 bits deciding upwards in magnitude."""
    p = np.asarray(p, np.float64)
    _, e = np.frexp(np.abs(p))
    ulp = np.ldexp(1.0, np.maximum(e, -125).astype(np.int32) - 8)
    q = np.floor(np.abs(p) / ulp + (word >> np.uint64(16)).astype(np.float64) / 65536.0)
    return np.where(p == 0, 0.0, np.sign(p) * q * ulp)
