"""Plain reference of the turbo4 cache type, in numpy: the format's fixed fp32 operation order
for the codes (numpy's fp32 operations round once each), 64-bit arithmetic for everything
computed from them, and bounds of what the kernels may differ by.

Block layout and definition: include/tq.h.
"""
import numpy as np

LEVELS = np.array([9, 26, 44, 64, 88, 112, 144, 192], np.float64)
STEP = 2619.0 / 2097152.0
CENT = np.concatenate([-LEVELS[::-1], LEVELS]) * STEP        # ascending
INV = np.float32(float.fromhex("0x1.6a09e6p-4"))             # fp32 nearest to 1 / sqrt(128)
SIGN_BIT = np.array([8 * k + 7 if k < 4 else 8 * (k - 4) + 3 for k in range(8)])


def hadamard():
    h = np.ones((1, 1))
    for _ in range(7):
        h = np.block([[h, h], [h, -h]])
    return h


H = hadamard() / np.sqrt(128.0)


def tree(x):
    """Sum over the last axis in fp32, element i with element i + half."""
    while x.shape[-1] > 1:
        h = x.shape[-1] // 2
        x = x[..., :h] + x[..., h:]
    return x[..., 0]


def butterflies32(x):
    shape, h = x.shape, 1
    while h < 128:
        x = x.reshape(-1, 128 // (2 * h), 2, h)
        x = np.stack((x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]), 2)
        h *= 2
    return x.reshape(shape)


def encode(x16, signs=None, correct=False):
    """fp16 [n, 128] -> (magnitude [n, 128], negative [n, 128], norm fp16 [n])."""
    x = x16.astype(np.float32)
    if signs is not None:
        x = np.where(np.asarray(signs, bool), -x, x)
    n = np.sqrt(tree(x * x))
    with np.errstate(divide="ignore", invalid="ignore"):
        k = np.where(n > 0, INV / n, np.float32(0)).astype(np.float32)
    y = butterflies32(x) * k[:, None]
    c = (LEVELS * STEP).astype(np.float32)
    t = (c[1:] + c[:-1]) * np.float32(0.5)
    mag = np.searchsorted(t, np.abs(y), side="left")          # thresholds strictly below
    if correct:
        n = n / np.sqrt(tree(c[mag] * c[mag]))
    return mag, np.signbit(y), np.minimum(n, np.float32(65504)).astype(np.float16)


def pack(mag, neg, norm, blocks):
    """Blocks of whole rows -> uint8 [rows, blocks * 66]."""
    rows = mag.shape[0] // blocks
    w = np.zeros((mag.shape[0], 16), np.uint32)
    m, s = mag.reshape(-1, 16, 8).astype(np.uint32), neg.reshape(-1, 16, 8).astype(np.uint32)
    for k in range(8):
        w |= (m[..., k] << np.uint32(4 * k)) | (s[..., k] << np.uint32(SIGN_BIT[k]))
    codes = np.ascontiguousarray(w.astype("<u4")).view(np.uint8).reshape(rows, blocks * 64)
    return np.concatenate([codes, np.ascontiguousarray(norm).view(np.uint8).reshape(rows, blocks * 2)], 1)


def encode_rows(x16, blocks, signs=None, correct=False):
    """fp16 [n, blocks * 128] -> packed rows."""
    return pack(*encode(x16.reshape(-1, 128), signs, correct), blocks)


def unpack(rows, blocks):
    """uint8 [n, blocks * 66] -> (64-bit levels [n, blocks, 128], norms [n, blocks])."""
    n = rows.shape[0]
    w = np.ascontiguousarray(rows[:, : blocks * 64]).view("<u4").reshape(n, blocks, 16)
    out = np.empty((n, blocks, 16, 8))
    for k in range(8):
        m = (w >> np.uint32(4 * k)) & np.uint32(7)
        neg = (w >> np.uint32(SIGN_BIT[k])) & np.uint32(1)
        out[..., k] = LEVELS[m] * STEP * (1.0 - 2.0 * neg)
    norm = np.ascontiguousarray(rows[:, blocks * 64:]).view(np.float16).astype(np.float64)
    return out.reshape(n, blocks, 128), norm.reshape(n, blocks)


def flip(signs):
    return 1.0 if signs is None else 1.0 - 2.0 * np.asarray(signs, np.float64)


def dequant(rows, blocks, signs=None):
    c, n = unpack(rows, blocks)
    return (c @ H) * n[..., None] * flip(signs)


def attention(kd, vd, q, see, scale, hkv):
    """kd / vd: 64-bit values [T, hkv * nb, 128] in the model's basis; q [n, hq, d];
    see [n, T].  Returns 64-bit [n, hq, d]; a query that sees nothing gets zeros."""
    n, hq, d = q.shape
    T = kd.shape[0]
    k, v = kd.reshape(T, hkv, d), vd.reshape(T, hkv, d)
    out = np.zeros((n, hq, d))
    G = hq // hkv
    for h in range(hq):
        s = q[:, h].astype(np.float64) @ k[:, h // G].T * scale
        s = np.where(see, s, -np.inf)
        top = s.max(-1, keepdims=True) if T else np.full((n, 1), -np.inf)
        top = np.where(np.isfinite(top), top, 0.0)
        p = np.exp(s - top)
        tot = p.sum(-1, keepdims=True)
        out[:, h] = np.where(tot > 0, (p @ v[:, h // G]) / np.where(tot > 0, tot, 1.0), 0.0)
    return out


def attention_bound(krows, vrows, q, see, scale, hkv, f16_out, v_rounded, signs_k=None):
    """2-norm bound of every (query, head) vector's error, [n, hq].

    In the rotated domain o = sum_t w_t |v_t| c_t.  The kernels round each product's factors:
    the weight p |v| to 11 bits (half a step, 2^-11 relative, from three 4-bit operands or one
    fp16 operand), a prompt chunk's |v| c to fp16 (2^-11 more: v_rounded), so coordinate j is
    off by at most e sum_t w_t |v_t| |c_tj|.  A score is off by ds = 2^-20 sum_j |q~_j c_j| |k|
    scale (the query keeps 22 bits and sums of 128 products in fp32 lose 7 bits of 24 at the
    worst; the levels are exact operands), and the exponent's own error (2^-22 of a value up to
    2^5 below its maximum, and an approximate exp2 of 2^-22) adds 2^-16: every weight and the
    sum that divides them are off by a factor within 1 +- (ds + 2^-16) each.  Weights below
    2^-25 of the largest p |v| may be flushed: T 2^-24 of the largest contribution bounds them.
    The fp16 output rounds once more, 2^-11.  W / sqrt(128) keeps 2-norms.
    """
    nb = krows.shape[1] // 66 // hkv
    kc, kn = unpack(krows, hkv * nb)
    vc, vn = unpack(vrows, hkv * nb)
    n, hq, d = q.shape
    G, T = hq // hkv, krows.shape[0]
    out = np.zeros((n, hq))
    for h in range(hq):
        g = h // G
        qr = (q[:, h].astype(np.float64).reshape(n, nb, 128) * flip(signs_k)) @ H
        s = np.zeros((n, T))
        ds = np.zeros((n, T))
        for b in range(nb):
            s += qr[:, b] @ kc[:, g * nb + b].T * kn[:, g * nb + b] * scale
            ds += np.abs(qr[:, b]) @ np.abs(kc[:, g * nb + b]).T * np.abs(kn[:, g * nb + b]) * scale
        s = np.where(see, s, -np.inf)
        some = see.any(-1)
        top = np.where(some, s.max(-1, initial=-np.inf), 0.0)
        w = np.exp(s - top[:, None])
        w = w / np.where(some, w.sum(-1), 1.0)[:, None]
        eps = (2.0 if v_rounded else 1.0) * 2.0 ** -11
        shift = 2.0 * (np.where(see, ds, 0.0).max(-1, initial=0.0) * 2.0 ** -20 + 2.0 ** -16)
        err = np.zeros(n)
        size = np.zeros(n)
        for b in range(nb):
            a = vn[:, g * nb + b, None] * np.abs(vc[:, g * nb + b])
            err += ((w @ a) ** 2).sum(-1)
            size += ((w @ (vn[:, g * nb + b, None] * vc[:, g * nb + b])) ** 2).sum(-1)
        flush = T * 2.0 ** -24 * (w[:, :] * vn[:, g * nb:(g + 1) * nb].max(-1)[None]).max(-1, initial=0.0) * np.sqrt(nb)
        out[:, h] = (eps + shift) * np.sqrt(err) + flush + (2.0 ** -11 * np.sqrt(size) if f16_out else 0.0)
    return out
