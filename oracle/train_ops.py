"""Float64 oracle of the training-step operators around the optimizer: the
counter-based generator, dropout, embedding lookup and gradient. NumPy, plain
loops and formulas; shares no code with the library."""
import numpy as np

M32 = 0xFFFFFFFF


def philox4x32_10(counter, key):
    """One call of Philox4x32-10 (Salmon et al., 2011) in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & M32, (p >> 32) ^ c[3] ^ k[1], p & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def random16(n, seed, offset=0, first=0):
    """The 16-bit numbers of elements first .. first + n - 1."""
    g0, g1 = first // 8, (first + n + 7) // 8
    j = np.arange(g0, g1, dtype=np.uint64)
    m = np.uint64(M32)
    s = np.uint64(32)
    c = [j & m, j >> s, np.full_like(j, offset & M32), np.full_like(j, offset >> 32)]
    k = [seed & M32, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> s) ^ c[1] ^ np.uint64(k[0]), q & m, (p >> s) ^ c[3] ^ np.uint64(k[1]), p & m]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    h = np.empty((len(j), 8), dtype=np.int64)
    for w in range(4):
        h[:, 2 * w] = (c[w] & np.uint64(0xFFFF)).astype(np.int64)
        h[:, 2 * w + 1] = (c[w] >> np.uint64(16)).astype(np.int64)
    return h.reshape(-1)[first - 8 * g0:first - 8 * g0 + n]


def dropout_factors(shape, p, seed, offset=0):
    """Per element, 0 where dropped and 65536 / (65536 - T) where kept."""
    T = int(np.rint(65536.0 * float(np.float32(p))))
    u = random16(int(np.prod(shape)), seed, offset).reshape(shape)
    return np.where(u >= T, 65536.0 / (65536 - T) if T < 65536 else 0.0, 0.0)


def dropout(x, p, seed, offset=0, residual=None):
    f = dropout_factors(np.shape(x), p, seed, offset)
    y = np.where(f > 0, np.where(f > 0, x, 0.0) * f, 0.0)
    return y if residual is None else y + residual


def embed_lookup(table, tokens, scale=1.0, add=None, drop=None):
    """drop: (p, seed, offset) or None. An index outside the table reads zeros."""
    tokens = np.asarray(tokens).reshape(-1)
    ok = (tokens >= 0) & (tokens < table.shape[0])
    out = np.where(ok[:, None], table[np.where(ok, tokens, 0)] * scale, 0.0)
    if add is not None:
        out = out + add[np.arange(len(tokens)) % len(add)]
    return out if drop is None else dropout(out, *drop)


def embed_grad(dout, tokens, vocab, scale=1.0, padding_idx=-1, drop=None, so_far=None):
    tokens = np.asarray(tokens).reshape(-1)
    d = dout if drop is None else dropout(dout, *drop)
    g = np.zeros((vocab, dout.shape[1])) if so_far is None else so_far.copy()
    for t, v in enumerate(tokens):
        if 0 <= v < vocab and v != padding_idx:
            g[v] += scale * d[t]
    return g


# ---------------------------------------------------------------- 4-bit tensors

FP4_BLOCK = {"mx": 32, "nv": 16}
FP4_GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def fp4_scale_values(fmt):
    """Value of every scale byte, increasing: e8m0, or the finite e4m3 from 0."""
    if fmt == "mx":
        return np.ldexp(1.0, np.arange(-127, 128))
    i = np.arange(127)
    return np.where(i < 8, i / 512.0, np.ldexp(8.0 + i % 8, i // 8 - 10))


def fp4_tensor_scale(amax):
    """Smallest power of two g (from 2^-126) with amax <= 2688 g; 1 for 0."""
    if not (0 < amax < np.inf):
        return 1.0
    e = -126
    while 2688.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def fp4_quantize(x, fmt, stochastic=None, amax=None):
    """(codes [rows, k] 0-15, scale bytes [rows, blocks], values) of x (64 bits),
    blocks along its rows. stochastic: (seed, offset) or None."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    B = FP4_BLOCK[fmt]
    kp = (k + 31) // 32 * 32
    pad = np.zeros((rows, kp))
    pad[:, :k] = x
    v = pad.reshape(rows, kp // B, B)
    finite = np.isfinite(v)
    if amax is None:
        amax = np.abs(v[finite]).max() if finite.any() else 0.0
    g = fp4_tensor_scale(amax) if fmt == "nv" else 1.0
    sv = fp4_scale_values(fmt) * g
    bad = ~finite.all(axis=2)
    w = np.where(bad[..., None], 0.0, v)
    bits = np.minimum(np.searchsorted(6 * sv, np.abs(w).max(axis=2)), len(sv) - 1)
    s = sv[bits][..., None]
    y = np.minimum(np.where(s > 0, np.abs(w) / np.where(s > 0, s, 1), 0.0), 6.0)
    lo = np.searchsorted(FP4_GRID, y, side="right") - 1
    hi = np.minimum(lo + 1, 7)
    gap = np.where(hi > lo, FP4_GRID[hi] - FP4_GRID[lo], 1.0)
    if stochastic is None:
        part = (y - FP4_GRID[lo]) / gap
        up = (part > 0.5) | ((part == 0.5) & (lo % 2 == 1))
    else:
        u = random16(rows * kp, *stochastic).reshape(v.shape)
        up = np.floor(np.floor((y - FP4_GRID[lo]) * 131072) / (gap * 2)) + u >= 65536
    c = np.where(up, hi, lo)
    values = FP4_GRID[c] * s * np.where(np.signbit(w), -1.0, 1.0)
    codes = c + 8 * np.signbit(w)
    nb = (k + B - 1) // B
    bits = np.where(bad, 255 if fmt == "mx" else 127, bits)
    values = np.where(bad[..., None], np.nan, values)
    return codes.reshape(rows, kp)[:, :k], bits[:, :nb], values.reshape(rows, kp)[:, :k]


def fp4_pack(codes, bits, fmt):
    """(codes, scales) bytes in the library's storage order."""
    rows, k = codes.shape
    kp = (k + 31) // 32 * 32
    c = np.zeros((rows, kp), np.uint8)
    c[:, :k] = codes
    packed = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8).reshape(-1)
    per_tile = 4 * FP4_BLOCK[fmt]
    tk = (k + per_tile - 1) // per_tile
    s = np.zeros((rows + 127) // 128 * tk * 512, np.uint8)
    for r in range(rows):
        for b in range(bits.shape[1]):
            s[(r // 128 * tk + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = bits[r, b]
    return packed, s
