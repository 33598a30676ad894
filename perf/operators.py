"""Cases for the operators of the quantised KV cache.

The cache holds K and V in 4 or 8 bits.  A token's row of one head is cut into
groups of G elements (32 at 4 bits, 64 at 8); a group is stored as
    z = min(x),  s = bf16((max(x) - min(x)) / (2^bits - 1)),
    n = nearest integer to (x - z) / s, ties to even, clamped to 2^bits - 1
and stands for z + s n.  s below 2^-100 is stored as 0 (n = 0); a group that
holds a NaN or a value of magnitude 2^126 or more is stored as s = 0, z = NaN.
A page holds the 64 tokens of a key block for every KV head: per head a record
of two halves of 32 tokens, each [K codes | K params | V codes | V params], a
param being (bf16 s, bf16 z).  `_layout` gives the place of each code.

Operators: "write" (rows quantised into the cache, then read back), "gate"
(the gate's key rows from the cache), "decode" (block-sparse attention of one
token per sequence over the cache).
"""
import math

import torch

own = False
BLOCK = 64
THETA = 5e5

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step appends a token to each of 8 sequences of different lengths; the block
        # that it lands in is read back
        dict(name="append_kv4_b8", op="write", bits=4, B=8, Hkv=8, d=128, L=8192, n=1, r=64, ragged=True, paged=True,
             token_major=True),
        # a 32k prompt of a Llama-3.1-8B layer goes into the cache at once and is read back
        dict(name="prompt_kv4_32k", op="write", bits=4, B=1, Hkv=8, d=128, L=32768, n=32768, r=32768, ragged=False,
             paged=False, token_major=False),
        # a chunk of a chunked prefill, padded to the longest of 5 sequences, rows as a projection writes them
        # ([B, tokens, heads, d]); head dim 64, odd sizes
        dict(name="chunk_kv8_d64_b5", op="write", bits=8, B=5, Hkv=4, d=64, L=3001, n=777, r=1500, ragged=True,
             paged=True, token_major=True),
        # the gate's key rows of a whole 32k cache, after its prefill
        dict(name="gate_kv4_32k", op="gate", bits=4, B=1, Hkv=8, d=128, dg=128, L=32768, first=0, maxmin=False,
             ragged=False, paged=False),
        # the refresh of a decode step: only the last block's key rows, max+min pooling
        dict(name="gate_kv8_last_block_b4", op="gate", bits=8, B=4, Hkv=8, d=128, dg=64, L=8000, first=124, maxmin=True,
             ragged=False, paged=True),
        # the shortest decode: a few hundred tokens, head dim 64, groups of two heads
        dict(name="decode_kv4_d64_l200", op="decode", bits=4, B=2, Hq=6, Hkv=3, d=64, L=200, density=0.5, ragged=False,
             paged=False),
        # the decode step of the 32k Llama layer at density 0.1
        dict(name="decode_kv4_32k_d0.1", op="decode", bits=4, B=1, Hq=32, Hkv=8, d=128, L=32768, density=0.1,
             ragged=False, paged=False),
        # the same with every block active
        dict(name="decode_kv4_32k_dense", op="decode", bits=4, B=1, Hq=32, Hkv=8, d=128, L=32768, density=1.0,
             ragged=False, paged=False),
        # a padded serving batch: 8 paged sequences from 32k tokens down to an idle slot
        dict(name="decode_kv4_b8_ragged", op="decode", bits=4, B=8, Hq=32, Hkv=8, d=128, L=32768, density=0.2,
             ragged=True, paged=True),
        # 128k context at the density that a threshold gives there, 8 bits
        dict(name="decode_kv8_128k_d0.17", op="decode", bits=8, B=1, Hq=32, Hkv=8, d=128, L=131072, density=0.17,
             ragged=False, paged=True),
        # a 40/8-head layer (groups of five), two sequences, odd length
        dict(name="decode_kv8_g5_64k", op="decode", bits=8, B=2, Hq=40, Hkv=8, d=128, L=65001, density=0.3,
             ragged=True, paged=False),
        # a large batch of short dense contexts, multi-query heads in groups of 16
        dict(name="decode_kv4_b16_mqa16", op="decode", bits=4, B=16, Hq=64, Hkv=4, d=128, L=16384, density=1.0,
             ragged=False, paged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "gate", "decode", "decode"))
    bits, d, Hkv = rng.choice((4, 8)), rng.choice((64, 128, 128)), rng.choice((1, 2, 3, 4, 8))
    B = rng.choice((1, 1, 2, 3, 4, 7, 8))
    ragged, paged = rng.random() < 0.5, rng.random() < 0.5
    L = _log(rng, 1, min(60000, (1 << (18 if op == "write" else 20)) // (B * Hkv)))
    c = dict(op=op, bits=bits, B=B, Hkv=Hkv, d=d, L=L, ragged=ragged, paged=paged)
    if op == "write":
        n = _log(rng, 1, L)
        return dict(c, n=n, r=min(L, rng.choice((n, 64, 2 * n + 5))), token_major=rng.random() < 0.5)
    if op == "gate":
        nb = -(-L // BLOCK)
        return dict(c, dg=rng.choice((32, 64, 128)), first=rng.choice((0, nb - 1, nb // 2)), maxmin=rng.random() < 0.3)
    g = rng.choice((1, 2, 3, 4, 4, 5, 7, 8, 12))
    return dict(c, Hq=Hkv * g, density=rng.choice((1.0, 0.5, 0.2, 0.1, 0.05)))


def _lens(c):
    """Tokens of each sequence: L, or from L down, with an idle slot at the end of a batch of four or more."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    lens = [max(1, L - (b * L * 6) // (7 * B)) for b in range(B)]
    if B >= 4:
        lens[-1] = 0
    return lens


def _group(bits):
    return 32 if bits == 4 else 64


def work(case):
    c = case
    d, Hkv, lens = c["d"], c["Hkv"], _lens(c)
    half = d * c["bits"] // 8 + d // _group(c["bits"]) * 4      # bytes of one token's K (or V) row of one head
    if c["op"] == "write":
        wrote, back = sum(min(c["n"], x) for x in lens), sum(min(c["r"], x) for x in lens)
        return {"bytes": Hkv * 2 * ((wrote + back) * (2 * d + half)), "flops": Hkv * 2 * d * (wrote * 8 + back * 2)}
    if c["op"] == "gate":
        nb = -(-c["L"] // BLOCK)
        rows = sum(max(0, -(-x // BLOCK) - c["first"]) for x in lens)
        toks = sum(max(0, x - BLOCK * c["first"]) for x in lens)
        dk = 2 * d if c["maxmin"] else d
        return {"bytes": Hkv * (toks * half + dk * c["dg"] * 2 + c["B"] * (nb - c["first"]) * c["dg"] * 4),
                "flops": Hkv * (toks * d * 3 + rows * 2 * dk * c["dg"])}
    g, tot, act = c["Hq"] // Hkv, 0.0, 0.0
    for x in lens:
        nb = -(-x // BLOCK)
        if nb == 0:
            continue
        k = min(nb, max(min(2, nb), math.ceil(c["density"] * nb)))
        free = max(1, nb - 2)
        share = max(0, k - 2) / free
        union = min(nb, 2 + (nb - 2) * (1 - (1 - share) ** g)) if nb > 2 else nb
        tot += union * x / nb
        act += k * x / nb
    nb = -(-c["L"] // BLOCK)
    return {"bytes": Hkv * tot * 2 * half + c["B"] * c["Hq"] * (4 * d + nb + 4), "flops": 4.0 * d * c["Hq"] * act}


# ------------------------------------------------------------------ the cache


def _layout(bits, d, device):
    """Row bytes R, groups, bytes of a half record, and for each token of a half and each byte of its row (two
    neighbouring elements at 4 bits, one at 8) the byte's place among the K codes and among the V codes."""
    R, NG = d * bits // 8, d // _group(bits)
    t = torch.arange(32, device=device)[:, None]
    m = torch.arange(R, device=device)[None]
    c, b = m // 4, m % 4                       # 32-bit words of the row in element order
    if bits == 4:
        kb = t * R + ((c % 4) * NG + c // 4) * 4 + b
        w = m % 16
        swz = ((t >> 2) & 1) * 4 if d == 128 else 0 * t
        vb = t * R + ((w // 2) ^ swz) * (2 * NG) + (m // 16) * 2 + w % 2
    else:
        p = (c // 16) ^ (t & 1) if d == 128 else c // 16 + 0 * t
        kb = t * R + (p * 16 + (c // 4 % 4) + (c % 4) * 4) * 4 + b
        swz = ((t >> 1) & 3) * 2 if d == 128 else ((t >> 2) & 1) * 4
        vb = t * R + (((m % 64) // 8) ^ swz) * (8 * NG) + (m // 64) * 8 + m % 8
    return R, NG, 2 * 32 * (R + 4 * NG), kb, vb


def _quantise(x, bits):
    """Codes (uint8) and scale, zero (bf16) of rows x [..., d], in 64 bits."""
    G, top = _group(bits), 2 ** bits - 1
    g = x.double().unflatten(-1, (-1, G))
    lo, hi = g.amin(-1), g.amax(-1)
    bad = ~((lo > -2.0 ** 126) & (hi < 2.0 ** 126))
    s = ((hi - lo) / top).to(torch.bfloat16)
    s = torch.where(bad | (s.float() < 2.0 ** -100), torch.zeros_like(s), s)
    z = torch.where(bad, torch.full_like(lo, float("nan")), lo).to(torch.bfloat16)
    sd = s.double()[..., None]
    n = torch.where(sd > 0, ((g - lo[..., None]) / torch.where(sd > 0, sd, 1.0)).round().clamp(0, top), 0.0)
    return torch.where(bad[..., None], 0.0, n).to(torch.uint8).flatten(-2), s, z


def _bytes(codes, bits):
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pack(c, kq, vq, n_pages, table):
    """Pages u8 [n_pages, Hkv, record] of whole blocks from the codes and params of K and V [B, Hkv, nb * 64, ...]."""
    bits, d, B, Hkv = c["bits"], c["d"], c["B"], c["Hkv"]
    dev = kq[0].device
    R, NG, H, kb, vb = _layout(bits, d, dev)
    nb = kq[0].shape[2] // BLOCK
    out = torch.zeros((B * nb, Hkv, 2, H), dtype=torch.uint8, device=dev)

    def blocks(x):                             # [B, Hkv, nb * 64, w] -> [B * nb, Hkv, 2, 32 * w]
        w = x.shape[-1]
        return x.view(B, Hkv, nb, 2, 32, w).permute(0, 2, 1, 3, 4, 5).reshape(B * nb, Hkv, 2, 32 * w)

    for (codes, s, z), place, at in ((kq, kb, 0), (vq, vb, 32 * (R + 4 * NG))):
        out[..., at + place.flatten()] = blocks(_bytes(codes, bits))
        par = torch.stack((s, z), -1).view(torch.uint8).flatten(-2)
        out[..., at + 32 * R: at + 32 * (R + 4 * NG)] = blocks(par)
    pages = torch.zeros((n_pages, Hkv, 2 * H), dtype=torch.uint8, device=dev)
    pages[table.flatten().long()] = out.view(B * nb, Hkv, 2 * H)
    return pages


def _unpack(state, want_v=True):
    """K and V in 32 bits [B, Hkv, nb * 64, d], as the pages hold them."""
    c = state["case"]
    bits, d, B, Hkv = c["bits"], c["d"], c["B"], c["Hkv"]
    pages, table = state["pages"], state["table"]
    R, NG, H, kb, vb = _layout(bits, d, pages.device)
    nb = table.shape[1]
    rec = pages[table.flatten().long()].view(B, nb, Hkv, 2, H)

    def rows(place, at):
        by = rec[..., at + place.flatten()].view(B, nb, Hkv, 64, R)
        n = by if bits == 8 else torch.stack((by & 15, by >> 4), -1).flatten(-2)
        par = rec[..., at + 32 * R: at + 32 * (R + 4 * NG)].contiguous().view(torch.bfloat16)
        par = par.view(B, nb, Hkv, 64, NG, 2).float()
        x = par[..., 1:] + par[..., :1] * n.view(B, nb, Hkv, 64, NG, -1).float()
        return x.flatten(-2).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nb * 64, d)

    return rows(kb, 0), rows(vb, 32 * (R + 4 * NG)) if want_v else None


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(c, n, g):
    """K, V rows bf16 [B, Hkv, n, d]: unit normal, K with a bias of each 64 tokens and a few strong channels."""
    shape = (c["B"], c["Hkv"], n, c["d"])
    k = torch.randn(shape, generator=g, device="cuda")
    bias = 0.5 * torch.randn((c["B"], c["Hkv"], -(-n // BLOCK), c["d"]), generator=g, device="cuda")
    k += bias.repeat_interleave(BLOCK, 2)[:, :, :n]
    k *= 1 + 2 * (torch.rand(c["d"], generator=g, device="cuda") < 0.05).float()
    v = torch.randn(shape, generator=g, device="cuda")
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _drawn(c, seed):
    """What prepare() and exact() both start from: the cache's codes before they are packed, and the inputs."""
    g = _generator(seed)
    B, Hkv, d, nb = c["B"], c["Hkv"], c["d"], -(-c["L"] // BLOCK)
    k, v = _rows(c, nb * BLOCK, g)
    x = {"kq": _quantise(k, c["bits"]), "vq": _quantise(v, c["bits"])}
    n_pages = B * nb + (3 if c["paged"] else 0)
    if c["paged"]:
        x["table"] = torch.randperm(n_pages, generator=g, device="cuda")[:B * nb].view(B, nb).to(torch.int32)
    else:
        x["table"] = torch.arange(B * nb, device="cuda", dtype=torch.int32).view(B, nb)
    x["n_pages"] = n_pages
    x["lens"] = torch.tensor(_lens(c), device="cuda", dtype=torch.int32)
    if c["op"] == "write":
        x["k"], x["v"] = _rows(c, c["n"], g)
        x["count"] = x["lens"].clamp(max=c["n"])
        x["start"] = x["lens"] - x["count"]
        x["rcount"] = x["lens"].clamp(max=c["r"])
        x["rstart"] = x["lens"] - x["rcount"]
    elif c["op"] == "gate":
        dk = 2 * d if c["maxmin"] else d
        w = (2 * torch.rand((Hkv, dk, c["dg"]), generator=g, device="cuda") - 1) * math.sqrt(6.0 / (dk + c["dg"]))
        x["wk"] = w.to(torch.bfloat16)
        x["kt"] = torch.randn((B, Hkv, nb, c["dg"]), generator=g, device="cuda")
    else:
        x["q"] = torch.randn((B, c["Hq"], d), generator=g, device="cuda").to(torch.bfloat16)
        own_nb = (x["lens"] + 63) // 64
        j = torch.arange(nb, device="cuda")
        r = torch.rand((B, c["Hq"], nb), generator=g, device="cuda")
        r = torch.where((j == 0) | (j == own_nb[:, None, None] - 1), 2.0, r)
        r = torch.where(j >= own_nb[:, None, None], -1.0, r)
        keep = (own_nb * c["density"]).ceil().clamp(min=2)
        rank = r.argsort(-1, descending=True).argsort(-1)
        x["mask"] = ((rank < keep[:, None, None]) & (r >= 0)).to(torch.uint8)
    return x


def prepare(case, seed):
    c = dict(case)
    x = _drawn(c, seed)
    s = {"case": c, "lens": x["lens"], "table": x["table"]}
    s["pages"] = _pack(c, x["kq"], x["vq"], x["n_pages"], x["table"])
    if c["op"] == "write":
        for n in ("k", "v"):                   # as the projections hand them over
            t = x[n]
            s[n] = t.transpose(1, 2).contiguous().transpose(1, 2) if c["token_major"] else t
        for n in ("start", "count", "rstart", "rcount"):
            s[n] = x[n]
        shape = (c["B"], c["Hkv"], c["r"], c["d"])
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif c["op"] == "gate":
        s["wk"], s["kt"] = x["wk"], x["kt"]
    else:
        s["q"], s["mask"] = x["q"], x["mask"]
    return s


# ------------------------------------------------------------------ plain forms


def _write_plain(s):
    c = s["case"]
    bits, d, B, Hkv, n, r = c["bits"], c["d"], c["B"], c["Hkv"], c["n"], c["r"]
    pages, table = s["pages"], s["table"]
    R, NG, H, kb, vb = _layout(bits, d, pages.device)
    t = torch.arange(n, device=pages.device)
    b_of, t_of = torch.nonzero(t[None] < s["count"][:, None], as_tuple=True)
    pos = s["start"][b_of].long() + t_of
    page = table[b_of, pos // BLOCK].long()
    tok = pos % 32
    base = ((page[:, None] * Hkv + torch.arange(Hkv, device=pages.device)) * 2 + (pos % 64 // 32)[:, None]) * H
    flat = pages.view(-1)
    for x, place, at in ((s["k"], kb, 0), (s["v"], vb, 32 * (R + 4 * NG))):
        codes, sc, z = _quantise(x[b_of, :, t_of], bits)                       # [rows, Hkv, ...]
        flat[base[..., None] + (at + place[tok])[:, None]] = _bytes(codes, bits)
        par = torch.stack((sc, z), -1).view(torch.uint8).flatten(-2)
        to = at + 32 * R + tok[:, None] * (4 * NG) + torch.arange(4 * NG, device=pages.device)
        flat[base[..., None] + to[:, None]] = par
    k, v = _unpack(s)
    t = torch.arange(r, device=pages.device)
    b_of, t_of = torch.nonzero(t[None] < s["rcount"][:, None], as_tuple=True)
    pos = s["rstart"][b_of].long() + t_of
    s["k_out"][b_of, :, t_of] = k[b_of, :, pos].to(torch.bfloat16)
    s["v_out"][b_of, :, t_of] = v[b_of, :, pos].to(torch.bfloat16)
    return s["k_out"], s["v_out"]


def _rope(y, first, dg):
    """y [..., blocks, dg] rotated at the positions first, first + 1, ...: pairs (t, t + dg / 2)."""
    pos = torch.arange(first, first + y.shape[-2], device=y.device, dtype=torch.float64)
    ang = pos[:, None] * THETA ** (-2.0 * torch.arange(dg // 2, device=y.device, dtype=torch.float64) / dg)
    c, s = ang.cos().to(y.dtype), ang.sin().to(y.dtype)
    a, b = y[..., :dg // 2], y[..., dg // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _gate_plain(s):
    c = s["case"]
    k, _ = _unpack(s, want_v=False)
    B, Hkv, T, d = k.shape
    k = k.view(B, Hkv, T // 64, 64, d)[:, :, c["first"]:]
    pos = torch.arange(64 * c["first"], T, device=k.device).view(1, 1, -1, 64, 1)
    ok = pos < s["lens"].view(B, 1, 1, 1, 1)
    some = ok.any(3)
    if c["maxmin"]:
        xp = torch.cat((k.masked_fill(~ok, -math.inf).amax(3), k.masked_fill(~ok, math.inf).amin(3)), -1)
    else:
        xp = k.masked_fill(~ok, 0).sum(3) / ok.sum(3).clamp(min=1)
    xp = torch.where(some, xp, 0.0)
    y = torch.einsum("bhjc,hcg->bhjg", xp, s["wk"].float())
    s["kt"][:, :, c["first"]:] = _rope(y, c["first"], c["dg"])
    return s["kt"]


def _decode_plain(s):
    c = s["case"]
    k, v = _unpack(s)
    B, Hkv, T, d = k.shape
    g = c["Hq"] // Hkv
    q = s["q"].float().view(B, Hkv, g, d)
    x = torch.einsum("bhgd,bhtd->bhgt", q, k) / math.sqrt(d)
    ok = s["mask"].view(B, Hkv, g, -1).bool().repeat_interleave(64, -1)
    ok &= torch.arange(T, device=k.device) < s["lens"].view(B, 1, 1, 1)
    x = x.masked_fill(~ok, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgt,bhtd->bhgd", p, v) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + l.log(), -math.inf)
    return o.view(B, c["Hq"], d).to(torch.bfloat16), lse.view(B, c["Hq"])


# ------------------------------------------------------------------ the framework's calls


def _run_own(s):
    import long_context_prefill_attngate_b200 as seer
    c = s["case"]
    cache = seer.SeerKVCache(s["pages"], c["d"], c["bits"], block_table=s["table"])
    if c["op"] == "write":
        seer.seer_kv_write(cache, s["k"], s["v"], start=s["start"], count=s["count"])
        return seer.seer_kv_read(cache, c["r"], start=s["rstart"], count=s["rcount"], k=s["k_out"], v=s["v_out"])
    if c["op"] == "gate":
        return seer.seer_gate_key_cache_quant(cache, s["wk"], c["L"], kt=s["kt"], first_block=c["first"],
                                              lens=s["lens"], rope_theta=THETA, k_maxmin=c["maxmin"])
    return seer.seer_block_sparse_decode_quant(s["q"], cache, s["mask"], c["L"], lens=s["lens"], return_lse=True)


def run(state):
    if own:
        return _run_own(state)
    return {"write": _write_plain, "gate": _gate_plain, "decode": _decode_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits


def _values64(codes, s, z, G):
    """z + s n of natural-order codes, in 64 bits."""
    n = codes.to(torch.float64)
    return torch.repeat_interleave(z.double(), G, -1) + torch.repeat_interleave(s.double(), G, -1) * n


def _nearest64(x, bits):
    """The value that each element of x [..., d] stands for in the cache, by the definition: the nearest of the
    group's 2^bits levels (the even one of two)."""
    G, top = _group(bits), 2 ** bits - 1
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for i in range(0, x.shape[-1], G):
        v = x[..., i:i + G].double()
        lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
        step = ((hi - lo) / top).bfloat16().double()
        step = torch.where(step < 2.0 ** -100, 0.0, step)
        q = (v - lo) / torch.where(step == 0, 1.0, step)
        low = q.floor()
        n = low + ((q - low > 0.5) | ((q - low == 0.5) & (low % 2 == 1))).double()
        y = lo + step * n.clamp(max=top)
        out[..., i:i + G] = torch.where((lo > -2.0 ** 126) & (hi < 2.0 ** 126), y, math.nan)
    return out


def exact(case, seed):
    c = dict(case)
    x = _drawn(c, seed)
    G, B, Hkv, d, lens = _group(c["bits"]), c["B"], c["Hkv"], c["d"], _lens(c)
    if c["op"] == "write":
        outs = []
        for old, new in ((x["kq"], x["k"]), (x["vq"], x["v"])):
            held = _values64(*old, G)
            fresh = _nearest64(new, c["bits"])
            out = torch.zeros((B, Hkv, c["r"], d), dtype=torch.float64, device="cuda")
            for b, ln in enumerate(lens):
                nw, nr = min(c["n"], ln), min(c["r"], ln)
                held[b, :, ln - nw:ln] = fresh[b, :, :nw]
                out[b, :, :nr] = held[b, :, ln - nr:ln]
            outs.append(out)
        return tuple(outs)
    k = _values64(*x["kq"], G)
    if c["op"] == "gate":
        kt = x["kt"].double()
        half = c["dg"] // 2
        freq = torch.tensor([THETA ** (-2.0 * t / c["dg"]) for t in range(half)], device="cuda", dtype=torch.float64)
        for b, ln in enumerate(lens):
            nb = kt.shape[2]
            kt[b, :, c["first"]:] = 0
            for j in range(c["first"], min(nb, -(-ln // BLOCK))):
                blk = k[b, :, 64 * j:min(ln, 64 * j + 64)]
                xp = torch.cat((blk.max(1).values, blk.min(1).values), -1) if c["maxmin"] else blk.mean(1)
                y = (xp[:, :, None] * x["wk"].double()).sum(1)
                cs, sn = (freq * j).cos(), (freq * j).sin()
                kt[b, :, j, :half] = y[:, :half] * cs - y[:, half:] * sn
                kt[b, :, j, half:] = y[:, half:] * cs + y[:, :half] * sn
        return kt
    v = _values64(*x["vq"], G)
    g = c["Hq"] // Hkv
    o = torch.zeros((B, c["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, ln in enumerate(lens):
        if ln == 0:
            continue
        for h in range(Hkv):
            seen = x["mask"][b, h * g:(h + 1) * g].bool()
            seen = seen[:, torch.arange(ln, device="cuda") // BLOCK]
            w = x["q"][b, h * g:(h + 1) * g].double() @ k[b, h, :ln].T * d ** -0.5
            w = torch.where(seen, w, -math.inf)
            l = torch.logsumexp(w, -1)
            lse[b, h * g:(h + 1) * g] = l
            w = torch.where(seen.any(-1, keepdim=True), (w - l[:, None]).exp(), 0.0)
            o[b, h * g:(h + 1) * g] = w @ v[b, h, :ln]
    return o, lse
