"""f64 numpy reference of the 4-bit cache: the row format, the attention over it, the rotation.

Written from the format's definition in ``include/oxd.h`` and sharing no code with the kernels.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MAX_SCALE = 10912.0


def f16(x):
    """f64 rounded once to f16 (numpy's own conversion rounds to nearest even)."""
    return np.asarray(x, np.float64).astype(np.float16)


def round_bf16(x):
    """f64 rounded once to 8 significant bits, ties to even (bf16's normal range)."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def hold(x):
    """Rows [..., 128] of bf16 values (f64) -> codes u8 [..., 64], scales f16 [..., 4]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (4, 32))
    scale = f16(np.minimum(np.abs(g).max(-1) / 6.0, MAX_SCALE))
    s = scale.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(g) / s, 0.0)
    # nearest level; at a midpoint the even code
    d = np.abs(np.minimum(y, 6.0)[..., None] - LEVELS)
    code = d.argmin(-1)
    second = np.where(np.arange(8) == code[..., None], np.inf, d)
    tie = second.min(-1) == d.min(-1)
    other = second.argmin(-1)
    code = np.where(tie & (code % 2 == 1), other, code)
    code = (code + 8 * (np.signbit(g) & (s > 0))).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def plain_zero(codes):
    """Codes with the sign of zeros dropped: a value that rounds to zero may keep its sign or not."""
    low, high = codes & 15, codes >> 4
    return np.where(low == 8, 0, low) | (np.where(high == 8, 0, high) << 4)


def values(codes, scales):
    """codes u8 [..., 64], scales f16 [..., 4] -> f64 [..., 128]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (128,))
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(scales.astype(np.float64), 32, -1)


def code_order(scales, layout):
    """Scales [pages, heads, page_size, 4] in the axis order of the codes."""
    return scales.swapaxes(1, 2) if layout == "NHD" else scales


def pool_values(codes, scales, layout):
    return values(codes, code_order(scales, layout))


def tokens(pool, pages, layout):
    """Rows of a page list of a pool of values: [heads, tokens, 128]."""
    x = pool[pages]
    x = x.transpose(2, 0, 1, 3) if layout == "NHD" else x.transpose(1, 0, 2, 3)
    return x.reshape(x.shape[0], -1, 128)


def decode(q, kv, vv, indptr, indices, lengths, layout, sm_scale):
    """(out, lse, spread, size, total) in f64: spread = sum w |v| bounds what relative errors of w
    and v move, size = the largest sum |q k| sm_scale of a row's logits, total = sum |v| bounds
    what an error of every weight by the same small number moves."""
    B, Hq, _ = q.shape
    Hkv = kv.shape[2] if layout == "NHD" else kv.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, 128)), np.zeros((B, Hq))
    spread, size, total = np.zeros((B, Hq, 128)), np.zeros((B, Hq)), np.zeros((B, Hq, 128))
    for b in range(B):
        pages = indices[indptr[b]:indptr[b + 1]]
        k = tokens(kv, pages, layout)[:, :lengths[b]]
        v = tokens(vv, pages, layout)[:, :lengths[b]]
        for h in range(Hkv):
            qh = q[b, h * G:(h + 1) * G]
            x = qh @ k[h].T * sm_scale
            m = x.max(-1, keepdims=True)
            w = np.exp(x - m)
            z = w.sum(-1, keepdims=True)
            rows = slice(h * G, (h + 1) * G)
            out[b, rows] = w @ v[h] / z
            lse[b, rows] = (m + np.log(z))[:, 0]
            spread[b, rows] = w @ np.abs(v[h]) / z
            total[b, rows] = np.abs(v[h]).sum(0)
            size[b, rows] = (np.abs(qh) @ np.abs(k[h]).T * abs(sm_scale)).max(-1)
    return out, lse, spread, size, total


def rotate(x, angle_positions, pair_axis, theta):
    """Split-half rotation in f64 of rows [T, H, 128]; angle_positions [axes][T]."""
    i = np.arange(64)
    a = np.asarray(angle_positions, np.float64)[np.asarray(pair_axis)].T * theta ** (-2.0 * i / 128)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo, hi = x[..., :64], x[..., 64:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)
