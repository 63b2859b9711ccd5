"""Cases of speculative decoding over the paged 4-bit KV cache: drafted tokens in a tree.

A step drafts a tree of tokens per sequence (node 0, the root, is the token chosen last; every
other node names its parent, an earlier node), runs the model on all nodes at once, keeps the
path that the target's probabilities accept, and goes on from the token drawn behind it.

  attention  the nodes attend to the cached context and to their own ancestors
  verify     the walk along the tree from given random numbers: accepted path and next token
  keep       the nodes' keys and values appended (keys turned by context + depth), the accepted
             path's records moved to the front of the tree's slots, the slots read back

The cache holds 68-byte turbo4 records (fp32 norm, 128 4-bit codebook indices of the rotated
unit vector) in pages [n_pages][Hkv][page_size] that a block table lists per sequence.

With ``own`` false every pass runs in elementary torch operations, in fp32 but for the verification's
weights and sums, which lie next to the border that a random number sets: those are fp64.
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
    base = {"rot": "wht", "rope": 128, "inter": False, "pad": 0, "zero": False, "fused": False, "wide": 4}

    def case(name, op, **kw):
        return {"name": name, "op": op, **base, **kw}

    def cached(name, op, **kw):
        return case(name, op, Hq=32, Hkv=8, page=64, dtype="bf16", **kw)

    return [
        # a single user's short chat, eight drafted tokens: latency counts
        cached("tree_b1_short", "attention", B=1, lo=733, hi=733, tlo=8, thi=8, mix=31, fused=True),
        # the framework's long decode with a tree of eight: 8 sequences towards 32K
        cached("tree_b8_32k", "attention", B=8, lo=24000, hi=32768, tlo=8, thi=8, mix=32, rot="dense"),
        # wide trees of a few sequences over long contexts
        cached("tree_b4_wide", "attention", B=4, lo=8000, hi=24000, tlo=40, thi=64, mix=33, wide=16),
        # a server's mixed batch of short drafts, an idle slot in it, 6 query heads per KV head
        case("tree_b32_mixed_f16", "attention", B=32, Hq=12, Hkv=2, page=32, lo=16, hi=8000, tlo=1, thi=20,
             dtype="f16", mix=34, zero=True, pad=5),
        # chains of drafted tokens, one KV head per query head
        case("chain_b16_f16", "attention", B=16, Hq=8, Hkv=8, page=16, lo=500, hi=4000, tlo=5, thi=5, dtype="f16",
             mix=35, wide=1, rope=64, inter=True),
        # one user's chain of four drafted tokens over the largest vocabulary
        case("verify_b1_chain", "verify", B=1, V=131072, tlo=5, thi=5, dtype="f32", draft=True, mix=36, wide=1),
        # a batch's chains
        case("verify_b64_chain", "verify", B=64, V=131072, tlo=8, thi=8, dtype="f32", draft=True, mix=37, wide=1),
        # trees with several tokens drawn at a node: residuals of residuals; odd vocabulary
        case("verify_b16_tree", "verify", B=16, V=50001, tlo=9, thi=16, dtype="f32", draft=True, mix=38, wide=3, pad=3),
        # trees of the likeliest tokens, without a draft's probabilities, 16-bit rows
        case("verify_b32_topk_bf16", "verify", B=32, V=65537, tlo=20, thi=32, dtype="bf16", draft=False, mix=39,
             wide=8),
        # one sequence's eight nodes, from the fused projection's output
        cached("keep_b1", "keep", B=1, lo=733, hi=733, tlo=8, thi=8, mix=40, fused=True),
        # a batch's trees
        cached("keep_b64", "keep", B=64, lo=900, hi=4000, tlo=24, thi=32, mix=41),
        # ragged trees, three KV heads, half of each head turned in adjacent pairs, padded batch
        case("keep_ragged_f16", "keep", B=9, Hq=3, Hkv=3, page=16, lo=1, hi=700, tlo=1, thi=64, dtype="f16", mix=42,
             rope=64, inter=True, pad=19, wide=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "verify", "verify", "keep"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "pad": rng.choice([0, 0, 1, 17]),
         "wide": rng.choice([1, 2, 4, 16]), "mix": rng.randrange(1 << 30)}
    if op == "verify":
        V = _log(rng, 100, 131072)
        thi = _log(rng, 1, 64)
        c |= {"dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "V": V, "draft": rng.random() < 0.6,
              "B": _log(rng, 1, max(1, min(64, 60000000 // (V * thi)))), "tlo": max(1, thi // 2), "thi": thi}
        return c
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c |= {"Hq": Hkv * rng.choice([1, 2, 3, 4, 6, 8, 12]), "Hkv": Hkv, "page": rng.choice([16, 32, 64, 128]),
          "rot": "wht" if op == "keep" else rng.choice(["wht", "dense"]), "rope": rng.choice([128, 128, 64, 0]),
          "inter": rng.random() < 0.3, "zero": op == "attention" and rng.random() < 0.25,
          "fused": rng.random() < 0.3}
    B = _log(rng, 1, 64)
    if op == "keep":
        thi = _log(rng, 1, max(1, min(128, 4000 // B)))
        c |= {"lo": 1, "hi": _log(rng, 2, 3000)}
    else:
        thi = _log(rng, 1, max(1, min(128, 1000 // B)))
        hi = _log(rng, 16, max(32, min(32768, 1800000 // (B * Hkv), 100000000 // (B * c["Hq"] * thi))))
        c |= {"lo": max(1, hi // rng.choice([1, 2, 30])), "hi": hi}
    return c | {"B": B, "tlo": max(1, thi // 2), "thi": thi}


def _sizes(case):
    """Per sequence: (length with the tree's nodes, nodes); from the case alone."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        ctx = _log(rng, case["lo"], case["hi"]) if "lo" in case else 0
        new = _log(rng, case["tlo"], case["thi"])
        out.append((ctx + new, new))
    if case.get("zero") and case["B"] > 1:  # an idle slot: its one row has no key
        out[case["B"] // 2] = (0, 1)
    return out


def _tree(case, b, n):
    """Parents of sequence b's n nodes: each node's is one of the `wide` nodes before it."""
    rng = random.Random(case["mix"] * 977 + b)
    return [-1] + [rng.randint(max(0, i - case["wide"]), i - 1) for i in range(1, n)]


def _path(parents, rng):
    """A root-to-node path of the tree, as verification accepts it."""
    at, path = rng.randrange(len(parents)), []
    while at >= 0:
        path.append(at)
        at = parents[at]
    return path[::-1]


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
        odd = np.array([bin(x).count("1") & 1 for x in range(D)])
        return (1.0 - 2.0 * odd[i[:, None] & i[None, :]]) * _signs(seed)[None, :] / math.sqrt(D)
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
    trees = [_tree(case, b, t) for b, (_, t) in enumerate(sizes)]
    cu = np.concatenate([[0], np.cumsum([t for _, t in sizes])])
    n = int(cu[-1])
    n_tok = n + case["pad"]
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 23)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": case, "cu": ints(cu), "n": n, "n_tok": n_tok, "max_q": max(t for _, t in sizes),
         "parents": ints([p for tree in trees for p in tree] + [-1] * case["pad"]),
         "lens": ints([m for m, _ in sizes]), "max_len": max(m for m, _ in sizes)}
    if case["op"] == "verify":
        _prepare_verify(s, gen)
    else:
        _prepare_cache(s, gen, sizes)
        if case["op"] == "keep":
            rng = random.Random(seed)
            paths = [_path(tree, rng) for tree in trees]
            s["path"] = ints([p + [-1] * (s["max_q"] - len(p)) for p in paths])
            s["n_path"], s["new_lens"] = ints([len(p) for p in paths]), torch.zeros_like(s["lens"])
    if own:
        import compressed_attention_gb300 as tq
        s["tq"] = tq
        s["kc"] = tq.Ctx("turbo4", case.get("rot", "wht"), KSEED)
        s["batch"] = tq.PagedBatch(s["lens"], cu_q=s["cu"], max_q=s["max_q"], n_tokens=n_tok, max_len=s["max_len"])
        if case["op"] != "verify":
            s["vc"] = tq.Ctx("turbo4", case["rot"], VSEED)
            s["kv"] = tq.PagedKV(s["kp"], s["vp"], s["table"], case["page"], case["Hkv"])
            s["turn"] = tq.Rope(s["cos"], s["sin"], interleaved=case["inter"]) if case["rope"] else None
        if case["op"] == "attention":
            s["ws"] = tq.alloc_workspace(
                tq.tq_paged_tree_workspace_size(s["kc"], s["vc"], s["kv"], s["batch"], case["Hq"]))
    return s


def _prepare_verify(s, gen):
    """Rows of the target's and the draft's probabilities (row v: of what follows node v), the nodes'
    tokens drawn from the draft's row of their parent (or its likeliest ones), and random numbers."""
    case, n = s["case"], s["n_tok"]
    dev, V, dt = "cuda", case["V"], _DT[case["dtype"]]
    logits = 2.5 * torch.randn((n, V), generator=gen, device=dev)
    near = logits + 0.7 * torch.randn((n, V), generator=gen, device=dev)
    s["target"] = torch.softmax(logits, -1).to(dt)
    q = torch.softmax(near, -1)
    del logits
    par = s["parents"].long()
    up = (s["cu"].long()[_rows(s)[0]] + par[:s["n"]]).clamp(min=0)  # the parent's row
    tokens = torch.zeros(n, dtype=torch.int64, device=dev)
    if case["draft"]:
        s["draft"] = q.to(dt)
        for i in range(0, s["n"], 64):  # the largest of log q plus Gumbel noise
            e = torch.rand((min(64, s["n"] - i), V), generator=gen, device=dev).clamp(min=1e-20)
            tokens[i:i + 64][:e.shape[0]] = (near[up[i:i + 64]] - torch.log(-torch.log(e))).argmax(-1)
    else:
        s["draft"] = None
        i = torch.arange(s["n"], device=dev)
        rank = ((up[:, None] == up[None]) & (par[None, :s["n"]] >= 0) & (i[None] < i[:, None])).sum(-1)
        k = min(V, case["wide"])
        tokens[:s["n"]] = near.topk(k, -1).indices[up].gather(1, rank.clamp(max=k - 1)[:, None])[:, 0]
    s["tokens"] = tokens.to(torch.int32)
    s["u"] = torch.rand(n, generator=gen, device=dev)
    s["u_next"] = torch.rand(case["B"], generator=gen, device=dev)
    s["path"] = torch.zeros((case["B"], s["max_q"]), dtype=torch.int32, device=dev)
    s["n_path"], s["next"] = (torch.zeros(case["B"], dtype=torch.int32, device=dev) for _ in range(2))


def _prepare_cache(s, gen, sizes):
    case, dev, n_tok = s["case"], "cuda", s["n_tok"]
    Hq, Hkv, P, dt = case["Hq"], case["Hkv"], case["page"], _DT[case["dtype"]]
    pages_of = [(n + P - 1) // P for n, _ in sizes]
    n_pages = sum(pages_of) + 3
    width = max(max(pages_of), 1)
    order = torch.randperm(n_pages, generator=gen, device=dev, dtype=torch.int32).cpu()
    table = torch.zeros((case["B"], width), dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages_of):
        table[b, :k] = order[at:at + k]
        at += k
    # packed pages: equal-probability cells make the indices of Gaussian rows uniform; norms as
    # of unit-variance rows with a spread between tokens
    pages = []
    for _ in range(2):
        w = torch.randint(-2 ** 31, 2 ** 31, (n_pages, Hkv, P, 17), generator=gen, device=dev, dtype=torch.int64).to(
            torch.int32)
        norm = math.sqrt(D) * torch.exp(0.2 * torch.randn((n_pages, Hkv, P), generator=gen, device=dev))
        w[..., 0] = norm.view(torch.int32)
        pages.append(w.view(torch.uint8).view(n_pages, Hkv, P, 68))

    def rows(h):
        return torch.randn((n_tok, h, D), generator=gen, device=dev).to(dt)

    # rows of q, k, v, as slices of a fused projection's output or alone
    if case["fused"]:
        qkv = rows(Hq + 2 * Hkv)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = rows(Hq), rows(Hkv), rows(Hkv)
    c, bnd = _codebook()
    s |= {"table": table.to(dev), "kp": pages[0], "vp": pages[1], "q": q, "k": k, "v": v, "codes": c.to(dev),
          "bounds": bnd.to(dev), "kr": torch.from_numpy(_rotation(case["rot"], KSEED)).to(dev, torch.float32),
          "vr": torch.from_numpy(_rotation(case["rot"], VSEED)).to(dev, torch.float32),
          "ks": torch.from_numpy(_signs(KSEED)).to(dev, torch.float32),
          "vs": torch.from_numpy(_signs(VSEED)).to(dev, torch.float32)}
    if case["rope"]:
        half = case["rope"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        ang = (torch.arange(width * P, dtype=torch.float64)[:, None] * inv).to(dev)
        s["cos"], s["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
    s["out"] = (torch.zeros((n_tok, Hq, D), dtype=dt, device=dev) if case["op"] == "attention" else
                [torch.zeros((n_tok, Hkv, D), dtype=dt, device=dev) for _ in range(2)])


# ------------------------------------------------------------------------------ passes

def run(s):
    op = s["case"]["op"]
    if own:
        tq = s["tq"]
        if op == "attention":
            tq.tq_paged_tree_attention(s["kc"], s["vc"], s["kv"], s["batch"], s["parents"], s["q"], s["out"], s["ws"],
                                       rope=s["turn"])
            return s["out"]
        if op == "verify":
            tq.tq_tree_verify(s["kc"], s["batch"], s["parents"], s["tokens"], s["target"], s["u"], s["u_next"],
                              s["path"], s["n_path"], s["next"], draft=s["draft"])
            return [s["path"], s["n_path"], s["next"]]
        tq.tq_paged_tree_append(s["kc"], s["vc"], s["kv"], s["batch"], s["parents"], s["k"], s["v"], rope=s["turn"])
        tq.tq_paged_tree_keep(s["kc"], s["vc"], s["kv"], s["batch"], s["path"], s["n_path"], s["new_lens"])
        tq.tq_paged_gather(s["kc"], s["vc"], s["kv"], s["batch"], s["out"][0], s["out"][1])
        return [*s["out"], s["new_lens"]]
    if op == "attention":
        s["out"][:s["n"]] = _attend(s)
        return s["out"]
    if op == "verify":
        return _verify(s)
    seq, slot = _rows(s)
    P, n = s["case"]["page"], s["n"]
    page = s["table"][seq, slot // P].long()
    s["kp"][page, :, slot % P] = _encode(s, _turn(s, s["k"][:n].float(), _positions(s)), s["ks"])
    s["vp"][page, :, slot % P] = _encode(s, s["v"][:n].float(), s["vs"])
    _keep(s)
    s["out"][0][:n] = _unpack(s, s["kp"][page, :, slot % P]) @ s["kr"]
    s["out"][1][:n] = _unpack(s, s["vp"][page, :, slot % P]) @ s["vr"]
    return [*s["out"], s["new_lens"]]


def _rows(s):
    """(sequence, slot) of each node: the last cu[b+1] - cu[b] slots of sequence b."""
    cu = s["cu"].long()
    i = torch.arange(s["n"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    return seq, s["lens"].long()[seq] - (cu[seq + 1] - i)


def _seen(s):
    """Bool [B, T, T]: node j is node i's ancestor or node i; from the parents by doubling."""
    cu, T = s["cu"].long(), s["max_q"]
    i = torch.arange(T, device=cu.device)
    row = cu[:-1, None] + i
    live = row < cu[1:, None]
    par = torch.where(live, s["parents"].long()[row.clamp(max=s["n"] - 1)], torch.full_like(row, -1))
    a = ((par[..., None] == i) | (i[:, None] == i)).float()
    for _ in range(max(T - 1, 1).bit_length()):  # paths of up to 1, 2, 4, ... edges
        a = ((a @ a) > 0).float()
    return a > 0


def _positions(s):
    """Context length plus depth of each node."""
    seq, slot = _rows(s)
    node = torch.arange(s["n"], device=slot.device) - s["cu"].long()[seq]
    return slot - node + _seen(s).sum(-1)[seq, node] - 1


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
    butterflies 1, 2, ..., 64, scale, nearest centroid.  Returns 68 bytes a row."""
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


def _keep(s):
    """Slot context + j takes the record of slot context + path[j]; past the path's end a slot keeps its own."""
    P = s["case"]["page"]
    nodes = s["cu"][1:] - s["cu"][:-1]
    base = (s["lens"] - nodes).long()[:, None]
    j = torch.minimum(torch.arange(s["max_q"], device=base.device), nodes.long()[:, None] - 1)
    src = base + torch.where(j < s["n_path"][:, None], s["path"].long().gather(1, j), j)
    dst = base + j
    src_page, dst_page = s["table"].gather(1, src // P).long(), s["table"].gather(1, dst // P).long()
    s["kp"][dst_page, :, dst % P] = s["kp"][src_page, :, src % P]
    s["vp"][dst_page, :, dst % P] = s["vp"][src_page, :, src % P]
    s["new_lens"].copy_(base[:, 0].int() + s["n_path"])


def _unpack(s, rows):
    """Packed rows [..., 68] -> norm * centroid in the rotated basis, fp32."""
    norm = rows[..., :4].contiguous().view(torch.float32)
    b = rows[..., 4:].int()
    idx = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return norm * s["codes"][idx]


def _attend(s):
    """fp32 [n, Hq, 128]: sequences padded to the longest; a node sees the context's keys, its
    ancestors' and its own."""
    case, n = s["case"], s["n"]
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["page"]
    g, L, T = Hq // Hkv, max(s["max_len"], 1), s["max_q"]
    seq, slot = _rows(s)
    t = torch.arange(L, device=s["q"].device)
    page = s["table"][:, t // P].long()                               # [B, L]
    q = (_turn(s, s["q"][:n].float(), _positions(s)) @ s["kr"].T) / math.sqrt(D)
    cu = s["cu"].long()
    node = torch.arange(n, device=q.device) - cu[seq]
    qp = torch.zeros((B, T, Hkv, g, D), device=q.device)
    qp[seq, node] = q.reshape(n, Hkv, g, D)
    kh = _unpack(s, s["kp"][page, :, t % P])                          # [B, L, Hkv, D]
    x = torch.einsum("bthgd,blhd->bhgtl", qp, kh)
    del kh
    end = s["lens"].long()[:, None]
    j = t - (end - (cu[1:] - cu[:-1])[:, None])                       # [B, L]: node of a slot
    tree = _seen(s).gather(2, j.clamp(0, T - 1)[:, None].expand(B, T, L))
    seen = ((j < 0)[:, None] | tree) & (t < end)[:, None]             # [B, T, L]
    x = torch.where(seen[:, None, None], x, torch.full((), -math.inf, device=q.device))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = x.sum(-1)                                                 # 0 where nothing is seen
    vh = _unpack(s, s["vp"][page, :, t % P])
    o = torch.einsum("bhgtl,blhd->bthgd", x, vh)
    o = o / torch.where(total > 0, total, torch.ones_like(total)).permute(0, 3, 1, 2)[..., None]
    return (o[seq, node] @ s["vr"]).reshape(n, Hq, D)


def _verify(s):
    """The walk of all sequences at once, in fp64: nodes in order, each tested where it is a child of
    the node that its sequence stands on."""
    cu, T, n = s["cu"].long(), s["max_q"], s["n"]
    i = torch.arange(T, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=n - 1)                        # [B, T]
    live = (cu[:-1, None] + i) < cu[1:, None]
    par = torch.where(live, s["parents"].long()[row], torch.full_like(row, -2))
    tok, u = s["tokens"].long()[row], s["u"].double()[row]
    on = torch.zeros_like(live)
    on[:, 0] = live[:, 0]
    if s["draft"] is None:
        # a child is taken with its share of what its earlier siblings left
        mine = s["target"][row.gather(1, par.clamp(min=0)), tok].double()                 # p(node | parent)
        before = (par[:, :, None] == par[:, None]) & (i[None] < i[:, None]) & (par >= 0)[:, None]  # [B, i, j]
        again = before & (tok[:, :, None] == tok[:, None])
        first = torch.where(again.any(-1), torch.zeros_like(mine), mine)  # a token again has nothing left
        take = (u * (1.0 - (before * first[:, None]).sum(-1)) < first) & (par >= 0)
        take &= ~(before & take[:, None]).any(-1)
        on = ((_seen(s) & ~(take | (i == 0))[:, None]).sum(-1) == 0) & live
        last = (on * (i + 1)).amax(-1) - 1
        r = s["target"][row.gather(1, last.clamp(min=0)[:, None])[:, 0]].double()
        gone = torch.zeros_like(r).scatter_add(1, tok, (par == last[:, None]).double())
        r = torch.where(gone > 0, torch.zeros_like(r), r)
    else:
        cur = torch.zeros_like(row[:, 0])
        r, q = s["target"][row[:, 0]].double(), s["draft"][row[:, 0]].double()
        z = torch.ones_like(r[:, 0])
        for k in range(1, T):
            child, x = (par[:, k] == cur), tok[:, k:k + 1]
            ok = child & (u[:, k] * q.gather(1, x)[:, 0] * z < r.gather(1, x)[:, 0])
            rest = torch.clamp(r - z[:, None] * q, min=0)
            left = rest.sum(-1)
            off = child & ~ok & (left > 0)
            cur = torch.where(ok, torch.full_like(cur, k), cur)
            on[:, k] = ok
            r = torch.where(off[:, None], rest, torch.where(ok[:, None], s["target"][row[:, k]].double(), r))
            q = torch.where(ok[:, None], s["draft"][row[:, k]].double(), q)
            z = torch.where(off, left, torch.where(ok, torch.ones_like(z), z))
    c = r.cumsum(-1)
    at = torch.searchsorted(c, s["u_next"].double()[:, None] * c[:, -1:], right=True)[:, 0]
    count = on.sum(-1)
    order = torch.where(on, i, torch.full_like(row, T)).sort(-1).values
    s["path"].copy_(torch.where(i < count[:, None], order, torch.full_like(order, -1)))
    s["n_path"].copy_(count)
    s["next"].copy_(at.clamp(max=c.shape[1] - 1))
    return [s["path"], s["n_path"], s["next"]]


# ------------------------------------------------------------------------------ work, exact

def work(case):
    sizes = _sizes(case)
    B, new = case["B"], sum(t for _, t in sizes)
    if case["op"] == "verify":  # a row of the weights that the next token is drawn from; the nodes' numbers
        e = 4 if case["dtype"] == "f32" else 2
        rows = 2 if case["draft"] else 1
        return {"bytes": B * case["V"] * e * rows + new * (12 + 2 * e) + B * 12, "flops": B * case["V"] * 3 * rows}
    Hq, Hkv, e = case["Hq"], case["Hkv"], 2
    angles = 4 * case["rope"] * new  # cos and sin of a position
    if case["op"] == "keep":  # K and V rows in, records out; the path's records moved; all read back, rows out
        return {"bytes": new * Hkv * 2 * (D * e + 68 + 68 + D * e) + angles, "flops": new * Hkv * 2 * 12 * D}
    cache = sum(n for n, _ in sizes) * Hkv * 2 * 68
    pairs = sum(t * (n - t) + t * min(t, 6) for n, t in sizes if n)
    return {"bytes": cache + new * 2 * Hq * D * e + angles, "flops": pairs * Hq * 4 * D}


def exact(case, seed):
    """The same outputs in 64 bits, one sequence at a time, from the definitions."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    sizes, dev, f64 = _sizes(case), s["cu"].device, torch.float64
    trees = [_tree(case, b, t) for b, (_, t) in enumerate(sizes)]
    if case["op"] == "verify":
        return _exact_verify(s, sizes, trees)
    if case["op"] == "attention" and sum(n * t for n, t in sizes) * case["Hq"] > 4e9:
        return None
    codes, P = s["codes"].to(f64), case["page"]
    KR, VR = (torch.from_numpy(_rotation(case["rot"], z)).to(dev) for z in (KSEED, VSEED))

    def depths(tree):
        d = []
        for p in tree:
            d.append(0 if p < 0 else d[p] + 1)
        return torch.tensor(d, device=dev)

    def hat(pages, b, n, R):
        """The n rows of sequence b as the records stand for them, [n, Hkv, 128]."""
        at = torch.arange(n, device=dev)
        rec = pages[s["table"][b].long()[at // P], :, at % P]
        half = torch.empty((*rec.shape[:-1], D), dtype=f64, device=dev)
        half[..., 0::2], half[..., 1::2] = codes[(rec[..., 4:] % 16).long()], codes[(rec[..., 4:] // 16).long()]
        return rec[..., :4].contiguous().view(torch.float32).to(f64) * (half @ R)

    def turned(x, at):
        x = x.to(f64).clone()
        r = case["rope"]
        if r:
            first = torch.arange(0, r, 2, device=dev) if case["inter"] else torch.arange(r // 2, device=dev)
            second = first + (1 if case["inter"] else r // 2)
            at = at.clamp(min=0)
            z = torch.complex(s["cos"][at].to(f64), s["sin"][at].to(f64))[:, None]
            y = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = y.real, y.imag
        return x

    def stands_for(x, R):
        norm = x.norm(dim=-1, keepdim=True)
        y = (x / norm.clamp(min=1e-300)) @ R.T
        idx = torch.bucketize(y.contiguous(), s["bounds"].to(f64))
        return norm * (codes[idx] @ R)

    out = [o.to(f64) for o in (s["out"] if isinstance(s["out"], list) else [s["out"]])]
    for b, (n, t) in enumerate(sizes):
        a = int(s["cu"][b])
        rows = slice(a, a + t)
        if not n:
            continue
        pos = n - t + depths(trees[b])
        if case["op"] == "keep":
            m = int(s["n_path"][b])
            for o, x, R in ((out[0], turned(s["k"][rows], pos), KR), (out[1], s["v"][rows].to(f64), VR)):
                o[rows] = stands_for(x, R)
                o[a:a + m] = o[a + s["path"][b, :m].long()]
            continue
        K, V = hat(s["kp"], b, n, KR), hat(s["vp"], b, n, VR)
        q = turned(s["q"][rows], pos)
        hidden = torch.zeros((t, n), dtype=torch.bool, device=dev)
        for i in range(t):
            line, at = [], i
            while at >= 0:
                line.append(at)
                at = trees[b][at]
            hidden[i, n - t:] = True
            hidden[i, [n - t + j for j in line]] = False
        for h in range(case["Hq"]):
            x = (q[:, h] @ K[:, h * case["Hkv"] // case["Hq"]].T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            out[0][rows, h] = torch.softmax(x, -1) @ V[:, h * case["Hkv"] // case["Hq"]]
    if case["op"] == "attention":
        return out[0]
    return [*out, torch.tensor([n - t for n, t in sizes], device=dev) + s["n_path"]]


def _exact_verify(s, sizes, trees):
    case = s["case"]
    path, count, nxt = s["path"].long(), s["n_path"].long(), s["next"].long()
    tokens, u, u_next = s["tokens"].tolist(), s["u"].tolist(), s["u_next"].tolist()
    for b, (_, t) in enumerate(sizes):
        a, at, line = int(s["cu"][b]), 0, [0]
        while True:
            left = s["target"][a + at].double()
            mass, taken = 1.0, None
            for c in [i for i in range(at + 1, t) if trees[b][i] == at]:
                x = tokens[a + c]
                if s["draft"] is not None:
                    q = s["draft"][a + at].double()
                    if u[a + c] * float(q[x]) * mass < float(left[x]):
                        taken = c
                        break
                    rest = (left - mass * q).clamp(min=0)
                    if float(rest.sum()) > 0:
                        left, mass = rest, float(rest.sum())
                else:
                    if u[a + c] * mass < float(left[x]):
                        taken = c
                        break
                    mass -= float(left[x])
                    left = left.clone()
                    left[x] = 0
            if taken is None:
                break
            at = taken
            line.append(at)
        total = left.cumsum(0)
        nxt[b] = min(int((total <= u_next[b] * total[-1]).sum()), case["V"] - 1)
        count[b] = len(line)
        path[b] = -1
        path[b, :len(line)] = torch.tensor(line, device=path.device)
    return [path, count, nxt]
