"""The quantised KV cache in 64 bits, from its description in include/seer.h:
quantisation, the record's layout, and the operators on the values it holds.
Shares no code with the package; plain numpy on the CPU."""
import numpy as np

BLOCK = 64


def group(bits):
    return 32 if bits == 4 else 64


def record_bytes(bits, d):
    return 2 * 64 * (d * bits // 8 + 4 * d // group(bits))


def bf16_round(x):
    """float64 -> the nearest bf16 (ties to even), as float64 and as bits."""
    u = np.asarray(x, np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    b = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64), b


def quantise(x, bits):
    """x float64 [..., d] (bf16 values): codes int [..., d], s and z float64 [..., d / G]."""
    G, top = group(bits), 2 ** bits - 1
    g = x.reshape(*x.shape[:-1], -1, G)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        bad = ~(np.abs(g) < 2.0 ** 126).all(-1)
        lo, hi = np.where(bad, 0, g.min(-1)), np.where(bad, 0, g.max(-1))
        s, _ = bf16_round((hi - lo) / top)
        s = np.where(bad | (s < 2.0 ** -100), 0.0, s)
        q = np.where(s[..., None] > 0, (g - lo[..., None]) / np.where(s > 0, s, 1)[..., None], 0.0)
        n = np.where(bad[..., None], 0, np.minimum(np.rint(q), top))
    return n.reshape(x.shape).astype(np.int64), s, np.where(bad, np.nan, lo)


def values(n, s, z):
    G = n.shape[-1] // s.shape[-1]
    return np.repeat(z, G, -1) + np.repeat(s, G, -1) * n


def _row(bits, d, t):
    """Byte offsets of token t's K and V codes within a half, in element order."""
    R, NG = d * bits // 8, d // group(bits)
    k, v = [], []
    for m in range(R):
        if bits == 4:
            c, e = m // 4, 2 * m                   # word of elements 8c ..; the byte's first element
            k.append(t * R + 4 * ((c % 4) * NG + c // 4) + m % 4)
            g, r = e // 32, (e % 32) // 4
            place = r ^ (4 if d == 128 and t & 4 else 0)
            v.append(t * R + place * 2 * NG + 2 * g + (e % 4) // 2)
        else:
            c = m // 4
            p = c // 16
            if d == 128:
                p ^= t & 1
            k.append(t * R + 4 * (16 * p + 4 * (c % 4) + (c // 4) % 4) + m % 4)
            g, r = m // 64, (m % 64) // 8
            place = r ^ (2 * ((t >> 1) & 3) if d == 128 else 4 * ((t >> 2) & 1))
            v.append(t * R + place * 8 * NG + 8 * g + m % 8)
    return k, v


def _places(bits, d):
    """Per token of a record: byte places of the K codes, K params, V codes, V params."""
    R, P = d * bits // 8, 4 * d // group(bits)
    half = 64 * (R + P)
    out = []
    for tok in range(64):
        t, base = tok % 32, (tok // 32) * half
        k, v = _row(bits, d, t)
        vb = base + 32 * (R + P)
        out.append((base + np.array(k), base + 32 * R + t * P + np.arange(P),
                    vb + np.array(v), vb + 32 * R + t * P + np.arange(P)))
    return out


def unpack(pages, bits, d):
    """pages u8 [n_pages, Hkv, record] -> ((n, s, z) of K, of V), [n_pages, Hkv, 64, ...]."""
    res = []
    pl = _places(bits, d)
    for at in (0, 2):
        by = np.stack([pages[..., pl[t][at]] for t in range(64)], 2).astype(np.int64)
        n = by if bits == 8 else np.stack((by & 15, by >> 4), -1).reshape(*by.shape[:-1], d)
        par = np.ascontiguousarray(np.stack([pages[..., pl[t][at + 1]] for t in range(64)], 2))
        u = par.view(np.uint16).astype(np.uint32).reshape(*par.shape[:-1], -1, 2)
        with np.errstate(invalid="ignore"):
            f = (u << 16).view(np.float32).astype(np.float64)
        res.append((n, f[..., 0], f[..., 1]))
    return res


def pack(pages, page, kvh, tok, kq, vq, bits, d):
    """Write one token's (n, s, z) of K and V into pages."""
    pk = _places(bits, d)[tok]
    for (n, s, z), (cp, pp) in ((kq, pk[:2]), (vq, pk[2:])):
        pages[page, kvh, cp] = n if bits == 8 else n[0::2] | (n[1::2] << 4)
        pages[page, kvh, pp] = np.stack((bf16_round(s)[1], bf16_round(z)[1]), -1).reshape(-1).view(np.uint8)


def gather(pages, table, bits, d):
    """(value parts of K, of V) [B, Hkv, blocks * 64, ...] of the sequences of a block table."""
    out = []
    for parts in unpack(pages, bits, d):
        out.append(tuple(np.concatenate([p[table[:, j]] for j in range(table.shape[1])], 2) for p in parts))
    return out


def decode(q, k, v, mask, lens, scale=None):
    """q [B,Hq,d]; k, v: (n, s, z); returns o, lse and, for the tolerances, sum p (s n + |z|) of the output and the
    largest sum |q| (s n + |z|) * scale of a key."""
    B, Hq, d = q.shape
    Hkv = k[0].shape[1]
    scale = d ** -0.5 if scale is None else scale
    kx, vx = values(*k), values(*v)
    ka, va = values(k[0], k[1], np.abs(k[2])), values(v[0], v[1], np.abs(v[2]))
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    A, E = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            t = np.arange(max(0, min(int(lens[b]), kx.shape[2], 64 * mask.shape[2])))
            t = t[mask[b, h, t // BLOCK] != 0]
            if not len(t):
                continue
            x = kx[b, kv, t] @ q[b, h] * scale
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            o[b, h], lse[b, h] = p @ vx[b, kv, t] / l, m + np.log(l)
            A[b, h] = p @ va[b, kv, t] / l
            E[b, h] = (ka[b, kv, t] @ np.abs(q[b, h])).max() * scale
    return o, lse, A, E


def gate_keys(k, wk, lens, first, theta, maxmin):
    """Key rows [B,Hkv,nb,dg] of blocks first.. (0 below) and, for the tolerance, sum pool|x| |w| over both halves."""
    n, s, z = k
    x, xa = values(n, s, z), values(n, s, np.abs(z))
    B, H, T, d = x.shape
    dg, nb = wk.shape[-1], T // 64
    kt, A = np.zeros((B, H, nb, dg)), np.zeros((B, H, nb, dg))
    half = dg // 2
    freq = theta ** (-2.0 * np.arange(half) / dg)
    for b in range(B):
        for j in range(first, nb):
            hi = min(64 * j + 64, int(lens[b]))
            if hi <= 64 * j:
                continue
            blk, ba = x[b, :, 64 * j:hi], xa[b, :, 64 * j:hi]
            xp = np.concatenate((blk.max(1), blk.min(1)), -1) if maxmin else blk.mean(1)
            ap = np.concatenate((ba.max(1), ba.max(1)), -1) if maxmin else ba.mean(1)
            y = np.einsum("hc,hcg->hg", xp, wk)
            a = np.einsum("hc,hcg->hg", ap, np.abs(wk))
            c, sn = np.cos(freq * j), np.sin(freq * j)
            kt[b, :, j, :half] = y[:, :half] * c - y[:, half:] * sn
            kt[b, :, j, half:] = y[:, half:] * c + y[:, :half] * sn
            A[b, :, j] = np.tile(a[:, :half] + a[:, half:], 2)
    return kt, A
