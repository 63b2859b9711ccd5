"""Cases of the paged 4-bit KV-cache operators: append, gather, attention, differential attention.

The cache holds 68-byte turbo4 records (fp32 norm, 128 4-bit codebook indices of the rotated
unit vector) in pages [n_pages][Hkv][page_size] that a block table lists per sequence.

  append     the new tokens' keys (position rotation applied) and values are quantized into
             their pages; the values the new rows then stand for are read back (gather)
  gather     whole sequences read back from their pages as dense rows
  attention  ragged causal attention of the last tokens of each sequence over its pages
  diff       the difference of two such maps per head pair, with a learned weight, an RMS
             norm per head and a scale

With ``own`` false every pass runs in elementary torch operations in fp32.
"""

import math
import random

import numpy as np
import torch

own = False

D = 128
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases

def listed():
    base = {"rot": "wht", "rope": 128, "inter": False, "pad": 0, "zero": False, "fused": False}

    def case(name, op, **kw):
        return {"name": name, "op": op, **base, **kw}

    return [
        # one decode step of a small batch: each sequence appends one token, taken from the
        # fused projection's output
        case("append_step_b8", "append", B=8, Hq=32, Hkv=8, page=64, lo=900, hi=4000, tlo=1, thi=1, dtype="bf16",
             mix=11, fused=True),
        # a prefill batch of 16K tokens over several prompts
        case("append_chunk_16k", "append", B=6, Hq=32, Hkv=8, page=64, lo=0, hi=0, tlo=1500, thi=4200, dtype="bf16",
             mix=12),
        # ragged chunks, three KV heads, half of each head rotated in adjacent pairs, padded batch
        case("append_ragged_f16", "append", B=9, Hq=3, Hkv=3, page=16, lo=1, hi=700, tlo=1, thi=403, dtype="f16",
             mix=13, rope=64, inter=True, pad=19),
        # prompts' prefixes handed to a program that wants them dense
        case("gather_prefix", "gather", B=4, Hq=8, Hkv=8, page=128, lo=3000, hi=12000, tlo=0, thi=0, dtype="bf16",
             mix=14, rot="dense"),
        case("gather_short_f16", "gather", B=5, Hq=2, Hkv=2, page=16, lo=1, hi=90, tlo=0, thi=0, dtype="f16", mix=15,
             zero=True),
        # the framework's long decode: 8 sequences towards 32K, 4 query heads per KV head
        case("decode_b8_32k", "attention", B=8, Hq=32, Hkv=8, page=64, lo=24000, hi=32768, tlo=1, thi=1,
             dtype="bf16", mix=16, rot="dense"),
        # a single user's short chat: latency counts
        case("decode_b1_short", "attention", B=1, Hq=32, Hkv=8, page=16, lo=733, hi=733, tlo=1, thi=1, dtype="bf16",
             mix=17, fused=True),
        # a server's mixed batch, an idle slot in it, 6 query heads per KV head
        case("decode_b64_mixed", "attention", B=64, Hq=12, Hkv=2, page=32, lo=16, hi=16000, tlo=1, thi=1,
             dtype="f16", mix=18, zero=True),
        # chunked prefill over long contexts
        case("prefill_chunk", "attention", B=4, Hq=32, Hkv=8, page=64, lo=4000, hi=16000, tlo=200, thi=512,
             dtype="bf16", mix=19, rot="dense"),
        # whole prompts, one KV head per query head, a padded batch
        case("prefill_prompt_f16", "attention", B=3, Hq=8, Hkv=8, page=16, lo=0, hi=0, tlo=129, thi=2047, dtype="f16",
             mix=20, pad=33),
        # differential decode of a batch, one weight per token and head pair
        case("diff_decode_b16", "diff", B=16, Hq=32, Hkv=8, page=64, lo=2000, hi=9000, tlo=1, thi=1, dtype="bf16",
             mix=21),
        # differential prefill chunks
        case("diff_chunk", "diff", B=2, Hq=16, Hkv=2, page=32, lo=1000, hi=5000, tlo=130, thi=400, dtype="bf16",
             mix=22, rot="dense"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "attention", "attention", "attention", "diff", "diff"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([2, 4, 6, 8] if op == "diff" else [1, 2, 3, 4, 6, 8, 12])
    c = {"op": op, "Hq": Hkv * g, "Hkv": Hkv, "page": rng.choice([16, 32, 64, 128]),
         "dtype": rng.choice(["bf16", "bf16", "f16"]), "rot": "wht" if op == "append" else rng.choice(["wht", "dense"]),
         "rope": rng.choice([128, 128, 64, 0]), "inter": rng.random() < 0.3, "pad": rng.choice([0, 0, 1, 17]),
         "zero": rng.random() < 0.25, "fused": rng.random() < 0.3, "mix": rng.randrange(1 << 30)}
    if op == "append":
        B = _log(rng, 1, 64)
        thi = _log(rng, 1, max(1, 16000 // B))
        c |= {"B": B, "lo": 1, "hi": _log(rng, 2, 3000), "tlo": max(1, thi // 3), "thi": thi}
    elif op == "gather":
        B = _log(rng, 1, 32)
        c |= {"B": B, "lo": 1, "hi": _log(rng, 2, 32000 // B), "tlo": 0, "thi": 0, "pad": 0, "fused": False}
    elif rng.random() < 0.6:  # single tokens
        B = _log(rng, 1, 128)
        hi = _log(rng, 40, max(64, min(32768, 1800000 // (B * Hkv))))
        c |= {"B": B, "lo": max(1, hi // rng.choice([1, 2, 30])), "hi": hi, "tlo": 1, "thi": 1, "pad": 0}
    else:
        B = _log(rng, 1, 5)
        thi = _log(rng, 2, 450 // B)
        c |= {"B": B, "lo": 1, "hi": _log(rng, 16, 8000), "tlo": max(1, thi // 2), "thi": thi}
    return c


def _sizes(case):
    """Per sequence: (length after the new tokens, new tokens); from the case alone."""
    rng = random.Random(case["mix"])
    out = []
    for b in range(case["B"]):
        ctx = _log(rng, case["lo"], case["hi"]) if case["lo"] > 0 else 0
        new = _log(rng, case["tlo"], case["thi"]) if case["tlo"] > 0 else 0
        if case["op"] in ("attention", "diff") and new == 1:  # a context of n tokens, the last one new
            ctx -= 1
        out.append((ctx + new, new))
    if case["zero"] and case["B"] > 1:  # an idle slot: no tokens (decode: its row has no key)
        out[case["B"] // 2] = (0, 1 if case["thi"] == 1 and case["op"] in ("attention", "diff") else 0)
    if case["op"] == "gather":  # whole sequences
        out = [(n, n) for n, _ in out]
    return out


# ------------------------------------------------------------------------------ inputs

def _splitmix(seed, n):
    i = np.arange(1, n + 1, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + i * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def _signs(seed):
    return np.where(_splitmix(seed, D) >> np.uint64(63), -1.0, 1.0)


def _rotation(kind, seed):
    """R of y = R u in fp64: the seeded +-1 diagonal and normalised Sylvester Hadamard matrix,
    or the Q factor (positive diagonal of R) of a seeded Gaussian matrix rounded to fp32."""
    if kind == "wht":
        i = np.arange(D)
        bits = i[:, None] & i[None, :]
        par = np.zeros_like(bits)
        for s in range(7):
            par ^= (bits >> s) & 1
        return (1.0 - 2.0 * par) * _signs(seed)[None, :] / math.sqrt(D)
    o = _splitmix(seed, D * D)
    u1 = ((o[0::2] >> np.uint64(11)).astype(np.float64) + 1.0) * 2.0 ** -53
    u2 = (o[1::2] >> np.uint64(11)).astype(np.float64) * 2.0 ** -53
    r = np.sqrt(-2.0 * np.log(u1))
    g = np.stack([r * np.cos(2 * math.pi * u2), r * np.sin(2 * math.pi * u2)], 1).reshape(D, D)
    q, t = np.linalg.qr(g)
    return (q * np.where(np.diag(t) < 0, -1.0, 1.0)[None, :]).astype(np.float32).astype(np.float64)


def _codebook():
    """16 centroids (conditional means of equal-probability cells of N(0, 1/128)) and the 15
    midpoints between the stored fp32 values."""
    t = torch.special.ndtri(torch.arange(17, dtype=torch.float64) / 16)
    pdf = torch.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    c = (16 * (pdf[:-1] - pdf[1:]) / math.sqrt(D)).to(torch.float32)
    b = (0.5 * (c[1:].double() + c[:-1].double())).to(torch.float32)
    return c, b


KSEED, VSEED = 7, 8  # rotation seeds of the key and value contexts


def prepare(case, seed):
    dev = "cuda"
    sizes = _sizes(case)
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["page"]
    dt = _DT[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)
    pages_of = [(n + P - 1) // P for n, _ in sizes]
    n_pages = sum(pages_of) + 3
    width = max(max(pages_of), 1)
    order = torch.randperm(n_pages, generator=gen, device=dev, dtype=torch.int32).cpu()
    table = torch.zeros((B, width), dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages_of):
        table[b, :k] = order[at:at + k]
        at += k
    lens = torch.tensor([n for n, _ in sizes], dtype=torch.int32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum([t for _, t in sizes])]), dtype=torch.int32)
    n = int(cu[-1])
    n_tok = n + case["pad"]
    # packed pages: equal-probability cells make the indices of Gaussian rows uniform; norms as
    # of unit-variance rows with a spread between tokens
    pages = []
    for _ in range(2):
        w = torch.randint(-2 ** 31, 2 ** 31, (n_pages, Hkv, P, 17), generator=gen, device=dev, dtype=torch.int64).to(
            torch.int32)
        norm = math.sqrt(D) * torch.exp(0.2 * torch.randn((n_pages, Hkv, P), generator=gen, device=dev))
        w[..., 0] = norm.view(torch.int32)
        pages.append(w.view(torch.uint8).view(n_pages, Hkv, P, 68))
    # rows of q, k, v, as slices of a fused projection's output or alone
    def rows(h):
        return torch.randn((max(n_tok, 1), h, D), generator=gen, device=dev).to(dt)

    if case["fused"]:
        qkv = rows(Hq + 2 * Hkv)
        q, k, v = qkv[:n_tok, :Hq], qkv[:n_tok, Hq:Hq + Hkv], qkv[:n_tok, Hq + Hkv:]
    else:
        q, k, v = rows(Hq)[:n_tok], rows(Hkv)[:n_tok], rows(Hkv)[:n_tok]
    c, bnd = _codebook()
    s = {"case": case, "lens": lens.to(dev), "cu": cu.to(dev), "table": table.to(dev), "kp": pages[0], "vp": pages[1],
         "q": q, "k": k, "v": v, "n": n, "max_q": max(t for _, t in sizes), "max_len": max(x for x, _ in sizes),
         "codes": c.to(dev), "bounds": bnd.to(dev),
         "kr": torch.from_numpy(_rotation(case["rot"], KSEED)).to(dev, torch.float32),
         "vr": torch.from_numpy(_rotation(case["rot"], VSEED)).to(dev, torch.float32),
         "ks": torch.from_numpy(_signs(KSEED)).to(dev, torch.float32),
         "vs": torch.from_numpy(_signs(VSEED)).to(dev, torch.float32)}
    if case["rope"]:
        half = case["rope"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        ang = (torch.arange(width * P, dtype=torch.float64)[:, None] * inv).to(dev)
        s["cos"], s["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
    if case["op"] in ("append", "gather"):
        s["out"] = [torch.zeros((n_tok, Hkv, D), dtype=dt, device=dev) for _ in range(2)]
    else:
        heads = Hq // 2 if case["op"] == "diff" else Hq
        s["out"] = torch.zeros((n_tok, heads, D), dtype=dt, device=dev)
    if case["op"] == "diff":
        s["lam"] = torch.rand((n_tok, Hq // 2), generator=gen, device=dev) * 0.6 + 0.2
        s["gain"] = 1.0 + 0.1 * torch.randn((D,), generator=gen, device=dev)
    if own:
        import compressed_attention_gb300 as tq
        s["tq"] = tq
        s["kc"] = tq.Ctx("turbo4", case["rot"], KSEED)
        s["vc"] = tq.Ctx("turbo4", case["rot"], VSEED)
        s["kv"] = tq.PagedKV(s["kp"], s["vp"], s["table"], P, Hkv)
        one = case["thi"] == 1 and s["max_q"] == 1 and n == B
        s["batch"] = (tq.PagedBatch(s["lens"], max_len=s["max_len"]) if one and not case["pad"] else
                      tq.PagedBatch(s["lens"], cu_q=s["cu"], max_q=s["max_q"], n_tokens=n_tok, max_len=s["max_len"]))
        s["rope"] = tq.Rope(s["cos"], s["sin"], interleaved=case["inter"]) if case["rope"] else None
        if case["op"] in ("attention", "diff"):
            s["ws"] = tq.alloc_workspace(tq.tq_paged_workspace_size(s["kc"], s["vc"], s["kv"], s["batch"], Hq))
        if case["op"] == "diff":
            s["mix"] = tq.DiffMix(s["lam"], norm_weight=s["gain"], eps=1e-5, out_scale=0.8)
    return s


# ------------------------------------------------------------------------------ passes

def run(s):
    op = s["case"]["op"]
    if own:
        tq, Hq = s["tq"], s["case"]["Hq"]
        if op == "append":
            tq.tq_paged_append(s["kc"], s["vc"], s["kv"], s["batch"], s["k"], s["v"], rope=s["rope"])
        if op in ("append", "gather"):
            tq.tq_paged_gather(s["kc"], s["vc"], s["kv"], s["batch"], s["out"][0], s["out"][1])
        elif op == "attention":
            tq.tq_paged_attention(s["kc"], s["vc"], s["kv"], s["batch"], s["q"], s["out"], s["ws"], rope=s["rope"])
        else:
            tq.tq_paged_diff_attention(s["kc"], s["vc"], s["kv"], s["batch"], s["q"], s["mix"], s["out"], s["ws"],
                                       rope=s["rope"])
        return s["out"]
    seq, pos = _places(s)
    if op == "append":
        _append(s, seq, pos)
    if op in ("append", "gather"):
        n = s["n"]
        s["out"][0][:n] = _values(s, s["kp"], seq, pos) @ s["kr"]
        s["out"][1][:n] = _values(s, s["vp"], seq, pos) @ s["vr"]
        return s["out"]
    att = _attend(s, seq, pos)
    if op == "diff":
        a = att[:, 0::2] - s["lam"][:s["n"], :, None] * att[:, 1::2]
        att = a * torch.rsqrt(torch.mean(a * a, -1, keepdim=True) + 1e-5) * s["gain"] * 0.8
    s["out"][:s["n"]] = att
    return s["out"]


def _places(s):
    """(sequence, position) of each new token: the last cu[b+1] - cu[b] of sequence b."""
    cu = s["cu"].long()
    i = torch.arange(s["n"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    pos = s["lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + (i - cu[seq])
    return seq, pos


def _turn(s, x, pos):
    """fp32 position rotation of rows x [n, heads, 128]; the rest of a head passes."""
    r = s["case"]["rope"]
    if not r:
        return x
    pos = pos.clamp(min=0)
    c, z = s["cos"][pos][:, None], s["sin"][pos][:, None]
    if s["case"]["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * z, a * z + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * z, a * z + b * c], -1)
    return torch.cat([y, x[..., r:]], -1)


def _stage(v, h):
    w = v.reshape(*v.shape[:-1], D // (2 * h), 2, h)
    a, b = w[..., 0, :], w[..., 1, :]
    return torch.stack([a + b, a - b], -2).reshape(v.shape)


def _fold(p):
    h = p.shape[-1] // 2
    return p[..., :h] + p[..., h:]


def _encode(s, x, signs):
    """The cache's canonical fp32 sequence: norm over a fixed tree, division, sign flips,
    butterflies 1, 2, ..., 64, scale, nearest centroid.  Returns 17 words a row."""
    w = (x * x).reshape(*x.shape[:-1], D // 4, 4)
    p = (w[..., 0] + w[..., 1]) + (w[..., 2] + w[..., 3])
    norm = torch.sqrt(_fold(_fold(_fold(_fold(_fold(p))))))
    u = torch.where(norm > 0, x / norm, torch.zeros_like(x))
    v = u * signs
    v = _stage(_stage(_stage(_stage(_stage(_stage(_stage(v, 1), 2), 4), 8), 16), 32), 64)
    y = v * torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32, device=v.device)
    idx = torch.searchsorted(s["bounds"], y.contiguous()).to(torch.uint8)  # #{k: y > b_k}
    packed = idx[..., 0::2] | (idx[..., 1::2] << 4)
    return torch.cat([norm.contiguous().view(torch.uint8), packed], -1)


def _append(s, seq, pos):
    P, n = s["case"]["page"], s["n"]
    page = s["table"][seq, pos // P].long()
    k = _turn(s, s["k"][:n].float(), pos)
    s["kp"][page, :, pos % P] = _encode(s, k, s["ks"])
    s["vp"][page, :, pos % P] = _encode(s, s["v"][:n].float(), s["vs"])


def _unpack(s, rows):
    """Packed rows [..., 68] -> norm * centroid in the rotated basis, fp32."""
    norm = rows[..., :4].contiguous().view(torch.float32)
    b = rows[..., 4:].int()
    idx = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return norm * s["codes"][idx]


def _values(s, pages, seq, pos):
    P = s["case"]["page"]
    return _unpack(s, pages[s["table"][seq, pos // P].long(), :, pos % P])


def _attend(s, seq, pos):
    """fp32 [n, Hq, 128]: sequences padded to the longest, keys after a token masked."""
    case, n = s["case"], s["n"]
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["page"]
    g, L, T = Hq // Hkv, max(s["max_len"], 1), s["max_q"]
    t = torch.arange(L, device=s["q"].device)
    page = s["table"][:, t // P].long()                               # [B, L]
    q = (_turn(s, s["q"][:n].float(), pos) @ s["kr"].T) / math.sqrt(D)
    row = torch.arange(n, device=q.device) - s["cu"].long()[seq]
    qp = torch.zeros((B, T, Hkv, g, D), device=q.device)
    qp[seq, row] = q.reshape(n, Hkv, g, D)
    pp = torch.full((B, T), -1, device=q.device)
    pp[seq, row] = pos
    kh = _unpack(s, s["kp"][page, :, t % P])                          # [B, L, Hkv, D]
    x = torch.einsum("bthgd,blhd->bhgtl", qp, kh)
    del kh
    seen = (t[None, None] <= pp[..., None])[:, None, None]            # [B, 1, 1, T, L]
    x = torch.where(seen, x, torch.full((), -math.inf, device=q.device))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = x.sum(-1)                                                 # 0 where nothing is seen
    vh = _unpack(s, s["vp"][page, :, t % P])
    o = torch.einsum("bhgtl,blhd->bthgd", x, vh)
    o = o / torch.where(total > 0, total, torch.ones_like(total)).permute(0, 3, 1, 2)[..., None]
    return (o[seq, row] @ s["vr"]).reshape(n, Hq, D)


# ------------------------------------------------------------------------------ work, exact

def work(case):
    sizes = _sizes(case)
    Hq, Hkv, e = case["Hq"], case["Hkv"], 2
    new = sum(t for _, t in sizes)
    angles = 4 * case["rope"] * new if case["op"] != "gather" else 0  # cos and sin of a position
    if case["op"] == "append":  # K and V rows in, records out and read back, rows out
        return {"bytes": new * Hkv * 2 * (D * e + 68 + 68 + D * e) + angles, "flops": new * Hkv * 2 * 12 * D}
    if case["op"] == "gather":
        per = 2 * D if case["rot"] == "dense" else 8
        return {"bytes": new * Hkv * 2 * (68 + D * e), "flops": new * Hkv * 2 * D * per}
    cache = sum(n for n, _ in sizes) * Hkv * 2 * 68
    pairs = sum(t * n - t * (t - 1) // 2 for n, t in sizes if n)
    heads = Hq // 2 if case["op"] == "diff" else Hq
    return {"bytes": cache + new * (Hq + heads) * D * e + angles, "flops": pairs * Hq * 4 * D}


def exact(case, seed):
    """The same outputs in 64 bits, one sequence at a time, from whole un-rotated rows."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    sizes = _sizes(case)
    if case["op"] in ("attention", "diff") and sum(n * t for n, t in sizes) * case["Hq"] > 4e9:
        return None
    f64 = torch.float64
    dev = s["q"].device
    codes, P = s["codes"].to(f64), case["page"]
    KR, VR = (torch.from_numpy(_rotation(case["rot"], z)).to(dev) for z in (KSEED, VSEED))

    def hat(pages, b, a, e, R):
        """Rows a..e of sequence b as the records stand for them, [e - a, Hkv, 128]."""
        at = torch.arange(a, e, device=dev)
        rec = pages[s["table"][b].long()[at // P], :, at % P]
        half = torch.empty((*rec.shape[:-1], D), dtype=f64, device=dev)
        half[..., 0::2], half[..., 1::2] = codes[(rec[..., 4:] % 16).long()], codes[(rec[..., 4:] // 16).long()]
        return rec[..., :4].contiguous().view(torch.float32).to(f64) * (half @ R)

    def turned(x, a):
        x = x.to(f64).clone()
        r = case["rope"]
        if r:
            first = torch.arange(0, r, 2, device=dev) if case["inter"] else torch.arange(r // 2, device=dev)
            second = first + (1 if case["inter"] else r // 2)
            at = torch.arange(a, a + x.shape[0], device=dev).clamp(min=0)
            z = torch.complex(s["cos"][at].to(f64), s["sin"][at].to(f64))[:, None]
            y = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = y.real, y.imag
        return x

    def stands_for(x, R):
        norm = x.norm(dim=-1, keepdim=True)
        y = (x / norm.clamp(min=1e-300)) @ R.T
        idx = torch.bucketize(y.contiguous(), s["bounds"].to(f64))
        return norm * (codes[idx] @ R)

    out = s["out"] if isinstance(s["out"], list) else [s["out"]]
    out = [o.to(f64) for o in out]
    for b, (n, t) in enumerate(sizes):
        a = int(s["cu"][b])
        if not n or not t:
            continue
        rows = slice(a, a + t)
        if case["op"] == "append":
            out[0][rows] = stands_for(turned(s["k"][rows], n - t), KR)
            out[1][rows] = stands_for(s["v"][rows].to(f64), VR)
        elif case["op"] == "gather":
            out[0][rows], out[1][rows] = hat(s["kp"], b, 0, n, KR), hat(s["vp"], b, 0, n, VR)
        else:
            K, V = hat(s["kp"], b, 0, n, KR), hat(s["vp"], b, 0, n, VR)
            q = turned(s["q"][rows], n - t)
            g = case["Hq"] // case["Hkv"]
            hidden = torch.arange(n, device=dev)[None] > torch.arange(n - t, n, device=dev)[:, None]
            att = torch.empty((t, case["Hq"], D), dtype=f64, device=dev)
            for h in range(case["Hq"]):
                x = (q[:, h] @ K[:, h // g].T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                att[:, h] = torch.softmax(x, -1) @ V[:, h // g]
            if case["op"] == "diff":
                d = att[:, 0::2] - s["lam"][rows, :, None].to(f64) * att[:, 1::2]
                att = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5) * s["gain"].to(f64) * 0.8
            out[0][rows] = att
    return out if case["op"] in ("append", "gather") else out[0]
