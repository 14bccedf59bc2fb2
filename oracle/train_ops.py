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
