"""Plain fp64 CPU statement of the 4-bit latent cache and of rotary positions (numpy only).

No code is shared with the GPU path.  Rows are decoded value by value from the format's definition; the encoder
searches the format's values instead of computing a code.
"""
import math

import numpy as np

DIM, NOPE, ROT, ROW = 576, 512, 64, 320
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode_rows(rows):
    """[n, 320] uint8 -> [n, 576] fp64."""
    rows = np.asarray(rows, dtype=np.uint8)
    out = np.empty((rows.shape[0], DIM))
    for d in range(DIM):
        word, i = d // 8, d % 8
        w = sum(rows[:, 4 * word + b].astype(np.int64) << (8 * b) for b in range(4))
        mag = MAGS[(w >> (4 * i)) & 7]
        sign = (w >> (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)) & 1
        e = rows[:, 288 + d // 32].astype(np.int64)
        v = np.where(sign == 1, -mag, mag) * 2.0 ** (e - 127.0)
        # at exponent 14 code 7 is NaN (and every other code, like every other exponent, has no meaning)
        out[:, d] = np.where((e >= 114) & (e <= 140), v, np.nan)
    return out


def block_exponent(block):
    """Least e of [-13, 13] whose largest value 6 * 2^e covers the block (13 if none does)."""
    amax = np.max(np.abs(block))
    for e in range(-13, 14):
        if amax <= 6.0 * 2.0 ** e:
            return e
    return 13


def encode_rows(y):
    """[n, 576] fp32 -> [n, 320] uint8: nearest value of the block's grid, ties to the even code."""
    y = np.asarray(y, dtype=np.float32).astype(np.float64)
    out = np.zeros((y.shape[0], ROW), dtype=np.uint8)
    for r in range(y.shape[0]):
        words = [0] * 72
        for b in range(18):
            blk = y[r, 32 * b:32 * b + 32]
            if np.isnan(blk).any():
                out[r, 288 + b] = 141
                for w in range(4 * b, 4 * b + 4):
                    words[w] = 0x77777777
                continue
            e = block_exponent(blk)
            out[r, 288 + b] = e + 127
            for j, v in enumerate(blk):
                a = min(abs(v) / 2.0 ** e, 6.0)
                dist = np.abs(MAGS - a)
                near = np.flatnonzero(dist == dist.min())
                code = int(near[0] if len(near) == 1 else near[near % 2 == 0][0])
                d = 32 * b + j
                word, i = d // 8, d % 8
                words[word] |= code << (4 * i)
                if np.signbit(v):
                    words[word] |= 1 << (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)
        for w, x in enumerate(words):
            out[r, 4 * w:4 * w + 4] = [(x >> s) & 255 for s in (0, 8, 16, 24)]
    return out


def inv_freq(rot_dim, theta, scaling=None, factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """(angle per position of each pair, factor on the rotated values)."""
    base = theta * factor ** (rot_dim / (rot_dim - 2.0)) if scaling == "ntk" else theta
    f = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def dim_of(turns):
        return rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low, high = max(math.floor(dim_of(beta_fast)), 0), min(math.ceil(dim_of(beta_slow)), rot_dim - 1)
    g = np.clip((np.arange(rot_dim // 2) - low) / max(high - low, 0.001), 0, 1)
    return f * (1 - g) + f / factor * g, 0.1 * math.log(factor) + 1.0


def rotate(x, pos, freq, mscale, layout, backward=False):
    """x [T, H, rot] fp64 turned to pos [T]: each pair times m * exp(+-i angle)."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    out = np.empty_like(x)
    for i in range(d // 2):
        a, b = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
        angle = np.fmod(np.asarray(pos, dtype=np.float64) * freq[i], 2 * math.pi)
        turn = mscale * np.exp((-1j if backward else 1j) * angle)
        z = (x[..., a] + 1j * x[..., b]) * turn[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def latent_rows(x, gamma=None, eps=1e-6, pos=None, freq=None, mscale=1.0, layout="interleaved"):
    """The rows an append stores, before quantisation, rounded to fp32."""
    y = np.array(x, dtype=np.float64)
    if gamma is not None:
        y[:, :NOPE] *= gamma / np.sqrt((y[:, :NOPE] ** 2).mean(-1, keepdims=True) + eps)
    if freq is not None:
        y[:, NOPE:] = rotate(y[:, None, NOPE:], pos, freq, mscale, layout)[:, 0]
    return y.astype(np.float32)


def append(pool, y, block_table, seq, pos):
    """A copy of the 4-bit pool [n_pages, 64, 320] with rows y [n, 576] fp32 at their slots."""
    pool = pool.copy()
    rows = encode_rows(y)
    for r in range(len(y)):
        pool[block_table[seq[r]][pos[r] // 64], pos[r] % 64] = rows[r]
    return pool


def paged_rows(pool, block_table, b, n):
    """[n, 576] fp64: positions 0..n-1 of sequence b."""
    t = np.arange(n)
    return decode_rows(pool[block_table[b][t // 64], t % 64])
