"""Operators that serving over the packed KV cache needs around its attention, as measured cases.

  attn    tq_decode_attn_shared: one decode step of a batch whose sequences share a prefix that is stored once
  rows    tq_qkv_norm_rope: the projection's rows of new tokens to normalised, position-rotated queries and keys, and values
  step    tq_pages_free then tq_pages_fork: finished sequences give up their pages, others start from a shared one or grow
  pack    tq_pages_compact: live pages to the front of the pool, tables rewritten

`run` computes them with elementary torch operations in 32 bits where `own` is false, and with the library's calls where
it is true."""
import math

import numpy as np
import torch

own = False

# Codec settings (block, bits) of keys and values by name, as the repository's workloads have them.
LAYOUTS = {
    "turbo3_d128": (128, (32, 3), (32, 3)),        # Qwen3-8B-shaped decode
    "turbo4k_turbo3v_d256": (256, (32, 4), (32, 3)),  # head_dim 256, long context
    "pervec4_d64": (64, (64, 4), (64, 4)),         # Llama-3.2-1B-shaped KV, one norm per vector
    "block4_d64": (64, (32, 4), (32, 4)),          # the same with a norm per 32 values
    "pervec2k_3v_d128": (128, (128, 2), (128, 3)),  # 2-bit keys, one norm per vector
}
SIGN_SEED = 1


def listed():
    return [
        # a chat server's small batch behind a short system prompt: launches and latency
        {"name": "attn_small", "op": "attn", "layout": "turbo3_d128", "B": 4, "Hq": 32, "Hkv": 8, "prefix": 1024,
         "own": 48, "page": 0},
        # a batch of samples over one long document, each with its own few hundred tokens
        {"name": "attn_doc_b32", "op": "attn", "layout": "turbo3_d128", "B": 32, "Hq": 32, "Hkv": 8, "prefix": 32768,
         "own": 512, "page": 0},
        # odd sizes, d 64, no grouping by 4, pages: a few-shot prompt shared by seven requests
        {"name": "attn_odd_paged", "op": "attn", "layout": "pervec4_d64", "B": 7, "Hq": 16, "Hkv": 8, "prefix": 2011,
         "own": 333, "page": 64},
        # the long-context model: 131072 shared tokens, eight questions about them
        {"name": "attn_long_d256", "op": "attn", "layout": "turbo4k_turbo3v_d256", "B": 8, "Hq": 16, "Hkv": 4,
         "prefix": 131072, "own": 256, "page": 0},
        # one decode step: eight tokens, keys and values into the fp16 window of recent tokens
        {"name": "rows_decode_b8", "op": "rows", "B": 8, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "pair": "half",
         "norm": True, "f32": False, "cap": 128, "ragged": False},
        # a speculative step: five drafts each for three sequences, fp32 projections, part of the head rotated
        {"name": "rows_draft_f32", "op": "rows", "B": 3, "T": 5, "Hq": 16, "Hkv": 4, "d": 256, "rot": 64, "pair": "next",
         "norm": True, "f32": True, "cap": 5, "ragged": False},
        # a padded batch of prompts of odd lengths, without norms
        {"name": "rows_ragged_d64", "op": "rows", "B": 5, "T": 701, "Hq": 16, "Hkv": 8, "d": 64, "rot": 64, "pair": "half",
         "norm": False, "f32": False, "cap": 701, "ragged": True},
        # a long prompt in one piece
        {"name": "rows_prompt_32k", "op": "rows", "B": 1, "T": 32768, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "pair": "half", "norm": True, "f32": False, "cap": 32768, "ragged": False},
        # a scheduler step of a small server, one layer's K and V
        {"name": "step_small", "op": "step", "layout": "turbo3_d128", "layers": 1, "Hkv": 8, "page": 32, "seqs": 16,
         "pages_per_seq": 64, "pages": 512, "frees": 3, "forks": 4, "grows": 4},
        # many samples forked from their prompts over all layers of a model, others growing
        {"name": "step_large", "op": "step", "layout": "pervec4_d64", "layers": 16, "Hkv": 8, "page": 64, "seqs": 256,
         "pages_per_seq": 128, "pages": 2000, "frees": 60, "forks": 150, "grows": 40},
        # a small pool with holes
        {"name": "pack_small", "op": "pack", "layout": "turbo3_d128", "layers": 1, "Hkv": 8, "page": 32, "seqs": 16,
         "pages_per_seq": 64, "pages": 512, "frees": 7},
        # a pool over all layers after a wave of requests has ended
        {"name": "pack_large", "op": "pack", "layout": "pervec4_d64", "layers": 16, "Hkv": 8, "page": 64, "seqs": 256,
         "pages_per_seq": 64, "pages": 2500, "frees": 130},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rows", "rows", "step", "pack"])
    if op == "attn":
        name = rng.choice(sorted(LAYOUTS))
        d = LAYOUTS[name][0]
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 64)
        most = int(min(65536, 4.0e9 / (Hkv * d * max(64, B * G))))
        return {"op": op, "layout": name, "B": B, "Hq": G * Hkv, "Hkv": Hkv, "prefix": _log(rng, 1, max(2, most)),
                "own": rng.choice([0, _log(rng, 1, 1024)]), "page": rng.choice([0, 32, 64, 96])}
    if op == "rows":
        d, B = rng.choice([64, 128, 256]), _log(rng, 1, 24)
        T = rng.choice([1, 1, min(_log(rng, 2, 4096), 1500000 // (B * d))])
        cap = T + rng.choice([0, 17])
        return {"op": op, "B": B, "T": T, "Hq": rng.choice([7, 8, 16, 24]), "Hkv": rng.choice([1, 4, 7]),
                "d": d, "rot": rng.choice([0, 32, d // 2, d]), "pair": rng.choice(["half", "next"]),
                "norm": rng.random() < 0.7, "f32": rng.random() < 0.4, "cap": cap, "ragged": rng.random() < 0.5}
    seqs = _log(rng, 12, 200)
    case = {"op": op, "layout": rng.choice(["turbo3_d128", "pervec4_d64", "block4_d64"]), "layers": _log(rng, 1, 8),
            "Hkv": rng.choice([1, 2, 8]), "page": rng.choice([32, 64, 128]), "seqs": seqs,
            "pages_per_seq": rng.choice([16, 33, 64]), "pages": seqs * 9 + _log(rng, 1, 400), "frees": seqs // 4}
    return case if op == "pack" else {**case, "forks": seqs // 4 + rng.randint(0, seqs // 8), "grows": rng.randint(1, seqs // 4)}


# ------------------------------------------------------------------ inputs
def _codebook(bits):
    """Lloyd-Max levels of N(0, 1) in 64 bits: boundaries at midpoints, levels at the means of their cells."""
    n = 1 << bits
    c = [-2.0 + 4.0 * (k + 0.5) / n for k in range(n)]
    pdf = lambda t: 0.0 if math.isinf(t) else math.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda t: 0.5 * math.erfc(-t / math.sqrt(2))  # noqa: E731
    for _ in range(20000):
        e = [-math.inf] + [0.5 * (a + b) for a, b in zip(c, c[1:])] + [math.inf]
        new = [(pdf(a) - pdf(b)) / (cdf(b) - cdf(a)) for a, b in zip(e, e[1:])]
        if max(abs(a - b) for a, b in zip(new, c)) < 1e-15:
            break
        c = new
    return [0.5 * (a - b) for a, b in zip(c, c[::-1])]


_BOOKS = {}


def _levels(bits, block):
    if bits not in _BOOKS:
        _BOOKS[bits] = _codebook(bits)
    return torch.tensor(_BOOKS[bits], dtype=torch.float64, device="cuda") / math.sqrt(block)


def _signs(seed, d):
    """+-1 from the top bits of splitmix64's outputs."""
    mask, out = (1 << 64) - 1, []
    for _ in range(d):
        seed = (seed + 0x9E3779B97F4A7C15) & mask
        z = ((seed ^ (seed >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return out


def _hadamard(n):
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(n)


def _pack(codes, bits):
    """Codes [N, d] to packed words: a nibble per code of a word, 8 codes a word, see the record of the C header."""
    n, d = codes.shape
    c = codes.to(torch.int64).view(n, d // 32, 4, 8)          # group, run of eight, place
    nib = (c << (4 * torch.arange(8, device=c.device))).sum(-1)  # [n, groups, 4]
    if bits == 4:
        w = nib
    elif bits == 3:
        last = c[:, :, 3]
        hi = [((((last >> k) & 1) << (4 * torch.arange(8, device=c.device) + 3)).sum(-1)) for k in range(3)]
        w = nib[:, :, :3] | torch.stack(hi, -1)
    elif bits == 2:
        w = nib[:, :, :2] | (nib[:, :, 2:] << 2)
    else:
        w = nib[:, :, :1] | (nib[:, :, 1:2] << 1) | (nib[:, :, 2:3] << 2) | (nib[:, :, 3:] << 3)
    return w.to(torch.int32).contiguous().view(torch.uint8).view(n, d * bits // 8)


def _cache(gen, lead, d, block, bits):
    """A packed cache of Gaussian rows: rotated, they are Gaussian again, so their codes are drawn there."""
    n = math.prod(lead)
    codes = torch.empty(n, d * bits // 8, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, d // block, dtype=torch.float16, device="cuda")
    lev = _levels(bits, block).float()
    edges = (0.5 * (lev[1:] + lev[:-1])).contiguous()
    step = max(1, (1 << 25) // d)
    for i in range(0, n, step):
        m = min(step, n - i)
        y = torch.randn(m, d // block, block, generator=gen, device="cuda")
        norm = y.norm(dim=-1, keepdim=True)
        codes[i:i + m] = _pack(torch.bucketize(y / norm, edges).view(m, d), bits)
        scales[i:i + m] = norm[..., 0].half()
    return codes.view(*lead, -1), scales.view(*lead, -1)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _prepare_attn(case, gen, rnd):
    d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
    B, Hkv, P, S, page = case["B"], case["Hkv"], case["prefix"], case["own"], case["page"]
    s = {"op": "attn", "case": case}
    cap = S + 9
    if page:  # one pool for everything: the prefix's pages, then every sequence's own, in shuffled places
        pp, po = -(-P // page), -(-cap // page)
        n = pp + B * po + 3
        place = torch.from_numpy(rnd.permutation(n).astype(np.int32)).cuda()
        lead_p = lead_o = (n, Hkv, page)
        s["table_p"], s["table_o"] = place[:pp].view(1, pp), place[pp:pp + B * po].view(B, po)
        cap, P_cap = po * page, pp * page
    else:
        P_cap = P + 5
        lead_p, lead_o = (1, Hkv, P_cap), (B, Hkv, cap)
        s["table_p"] = s["table_o"] = None
    s["kp"], s["vp"] = _cache(gen, lead_p, d, kb, kbits), _cache(gen, lead_p, d, vb, vbits)
    s["k"], s["v"] = (s["kp"], s["vp"]) if page else (_cache(gen, lead_o, d, kb, kbits), _cache(gen, lead_o, d, vb, vbits))
    # scores of twice the unit deviation: some tokens stand out, as a trained model's do
    s["q"] = (2.0 * torch.randn(B, case["Hq"], d, generator=gen, device="cuda")).half()
    lens = rnd.integers(max(0, S // 2), S + 1, size=B).astype(np.int32)
    lens[-1] = S
    s["len"] = torch.from_numpy(lens).cuda()
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        Lk, Lv = tb.make_layout(d, kb, kbits, sign_seed=SIGN_SEED), tb.make_layout(d, vb, vbits, sign_seed=SIGN_SEED)
        s["K_p"] = tb.PackedKV.of(Lk, *s["kp"], page_table=s["table_p"])
        s["V_p"] = tb.PackedKV.of(Lv, *s["vp"], page_table=s["table_p"])
        s["K_o"] = tb.PackedKV.of(Lk, *s["k"], page_table=s["table_o"])
        s["V_o"] = tb.PackedKV.of(Lv, *s["v"], page_table=s["table_o"])
        s["ws"] = torch.empty(max(16, tb.tq_decode_shared_workspace_bytes(B, case["Hq"], Hkv, d, P, S)), dtype=torch.uint8,
                              device="cuda")
    else:
        s["books"] = [(_levels(kbits, kb).float(), _hadamard(kb).float().cuda()),
                      (_levels(vbits, vb).float(), _hadamard(vb).float().cuda())]
        s["signs"] = torch.tensor(_signs(SIGN_SEED, d), device="cuda")
    return s


def _prepare_rows(case, gen, rnd):
    B, T, Hq, Hkv, d, rot, cap = (case[k] for k in ("B", "T", "Hq", "Hkv", "d", "rot", "cap"))
    width = (Hq + 2 * Hkv) * d
    x = torch.randn(B, T, width, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(width, generator=gen, device="cuda"))  # channels of unequal size
    s = {"op": "rows", "case": case, "x": x if case["f32"] else x.half()}
    w = 1.0 + 0.1 * torch.randn(2, d, generator=gen, device="cuda")
    s["wq"], s["wk"] = (w[0].contiguous(), w[1].contiguous()) if case["norm"] else (None, None)
    first = rnd.integers(0, 30000, size=B)
    n_pos = 30000 + T
    s["rope"] = None
    if rot:
        freq = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * freq
        s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    s["pos"] = torch.from_numpy(first.astype(np.int32)).cuda()
    lens = rnd.integers(T // 3, T + 1, size=B) if case["ragged"] else np.full(B, T)
    s["len"] = torch.from_numpy(lens.astype(np.int32)).cuda() if case["ragged"] else None
    slot = rnd.integers(0, cap - T + 1, size=B)
    s["slot"] = torch.from_numpy(slot.astype(np.int32)).cuda()
    s["q"] = torch.zeros(B, Hq, T, d, dtype=torch.float16, device="cuda")
    s["k"], s["v"] = (torch.zeros(B, Hkv, cap, d, dtype=torch.float16, device="cuda") for _ in range(2))
    return s


def _prepare_pool(case, gen, rnd):
    d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
    n, S, pps, page, L = case["pages"], case["seqs"], case["pages_per_seq"], case["page"], case["layers"]
    # random records: nothing here reads them, they are moved
    arrays = {}
    for name, block, bits in (("k", kb, kbits), ("v", vb, vbits)):
        arrays[name + "_codes"] = torch.randint(0, 256, (L, n, case["Hkv"], page, d * bits // 8), dtype=torch.uint8,
                                                generator=gen, device="cuda")
        arrays[name + "_scales"] = torch.rand(L, n, case["Hkv"], page, d // block, generator=gen, device="cuda").half()
    # sequences of a few pages each in shuffled places, some sharing their first pages; every fourth slot is empty
    table = np.zeros((S, pps), np.int32)
    held = np.zeros(S, np.int32)
    ref = np.zeros(n, np.int32)
    place = rnd.permutation(n).astype(np.int32)
    at, length = 0, np.zeros(S, np.int64)
    busy = [i for i in range(S) if i % 4]
    for k, i in enumerate(busy):
        room = (n - n // 4 - at) // (len(busy) - k)
        m = int(rnd.integers(1, max(2, min(pps - 1, 2 * room, n - n // 4 - at))))
        shared = 0
        if k and k % 3 == 0:
            p = busy[k - 1]
            shared = int(min(held[p] // 2, m))
            table[i, :shared] = table[p, :shared]
        table[i, shared:m] = place[at:at + m - shared]
        at += m - shared
        held[i] = m
        length[i] = (m - 1) * page + int(rnd.integers(1, page + 1))
        np.add.at(ref, table[i, :m], 1)
    flat = torch.from_numpy(np.concatenate([table.ravel(), held, ref])).cuda()
    s = {"op": case["op"], "case": case, "arrays": arrays, "start": flat, "book": flat.clone()}
    b = s["book"]
    s["table"], s["held"], s["ref"] = b[:S * pps].view(S, pps), b[S * pps:S * pps + S], b[S * pps + S:]
    order = [int(i) for i in rnd.permutation(busy)]
    done = order[:case["frees"]]
    s["done"] = torch.tensor(done, dtype=torch.int32, device="cuda")
    if case["op"] == "step":
        rest = order[case["frees"]:]
        grows, parents = rest[:case["grows"]], rest[case["grows"]:]
        slots = ([i for i in range(S) if i % 4 == 0] + done)[:case["forks"]]
        rows = []  # parent, child, tokens shared, tokens to hold
        for k, c in enumerate(slots):
            if k % 8 == 7 or not parents:  # a new sequence
                rows.append((-1, c, 0, int(rnd.integers(1, 2 * page))))
            else:
                p = parents[k % min(len(parents), 5)]
                cut = int(rnd.integers(1, length[p] + 1))
                rows.append((p, c, cut, min(cut + int(rnd.integers(1, page + 1)), pps * page)))
        for g in grows:
            rows.append((g, g, int(length[g]), min(int(length[g]) + int(rnd.integers(1, page + 1)), pps * page)))
        r = torch.tensor(rows, dtype=torch.int32, device="cuda")
        s["parent"], s["child"], s["share"], s["new"] = (r[:, k].contiguous() for k in range(4))
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        Lk, Lv = tb.make_layout(d, kb, kbits, sign_seed=SIGN_SEED), tb.make_layout(d, vb, vbits, sign_seed=SIGN_SEED)
        caches = []
        for i in range(L):
            caches += [tb.PackedKV.of(Lk, arrays["k_codes"][i], arrays["k_scales"][i]),
                       tb.PackedKV.of(Lv, arrays["v_codes"][i], arrays["v_scales"][i])]
        s["pool"] = tb.PagePool(s["table"], s["held"], s["ref"], page, caches)
        s["result"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        s["ws"] = torch.empty(tb.tq_pages_workspace_bytes(S, n, len(s["child"]) if case["op"] == "step" else 0),
                              dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen, rnd = _gen(seed), np.random.default_rng(int(seed))
    return {"attn": _prepare_attn, "rows": _prepare_rows, "step": _prepare_pool, "pack": _prepare_pool}[case["op"]](case, gen, rnd)


# ------------------------------------------------------------------ plain forms
def _unpack(words, bits):
    """Packed bytes [..., d bits / 8] to codes [..., d]."""
    w = words.view(torch.int32).unflatten(-1, (-1, bits))  # [..., groups, bits]
    place = 4 * torch.arange(8, device=w.device, dtype=torch.int32)
    nib = (w[..., None] >> place) & 15                      # [..., groups, bits, 8]
    if bits == 4:
        c = nib
    elif bits == 3:
        top = nib >> 3
        c = torch.cat([nib & 7, (top[..., 0:1, :] | (top[..., 1:2, :] << 1) | (top[..., 2:3, :] << 2))], -2)
    elif bits == 2:
        c = torch.cat([nib & 3, nib >> 2], -2)
    else:
        c = torch.cat([nib & 1, (nib >> 1) & 1, (nib >> 2) & 1, nib >> 3], -2)
    return c.flatten(-3)


def _decoded(cache, book, bits, block, signs):
    """The vectors that a packed cache stands for, in 32 bits: scale * D H c."""
    codes, scales = cache
    level, had = book
    y = level[_unpack(codes, bits)].unflatten(-1, (-1, block)) @ had
    return (y * scales.float()[..., None]).flatten(-2) * signs


def _by_table(cache, table):
    """Pages [n, H, page, ...] of a table [B, m] as [B, H, m page, ...]."""
    return tuple(a[table.long()].transpose(1, 2).flatten(2, 3) for a in cache)


def _attn_plain(s):
    c = s["case"]
    d, (kb, kbits), (vb, vbits) = LAYOUTS[c["layout"]]
    B, Hkv, G, P, S = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["prefix"], c["own"]
    kp, vp, k, v = s["kp"], s["vp"], s["k"], s["v"]
    if c["page"]:
        kp, vp = _by_table(kp, s["table_p"]), _by_table(vp, s["table_p"])
        k, v = _by_table(k, s["table_o"]), _by_table(v, s["table_o"])
    cut = lambda a, n: tuple(t[:, :, :n].contiguous() for t in a)  # noqa: E731
    q = s["q"].float().view(B, Hkv, G, d) / math.sqrt(d)
    bk, bv = s["books"]
    kp, vp = _decoded(cut(kp, P), bk, kbits, kb, s["signs"])[0], _decoded(cut(vp, P), bv, vbits, vb, s["signs"])[0]
    k, v = _decoded(cut(k, S), bk, kbits, kb, s["signs"]), _decoded(cut(v, S), bv, vbits, vb, s["signs"])
    rows = q.transpose(0, 1).reshape(Hkv, B * G, d)  # every query of a KV head against the one prefix
    sp = (rows @ kp.transpose(1, 2)).view(Hkv, B, G, P).transpose(0, 1)
    so = q @ k.transpose(2, 3)
    dead = torch.arange(S, device=q.device) >= s["len"][:, None]
    so = so.masked_fill(dead[:, None, None], -math.inf)
    m = torch.maximum(sp.amax(-1), so.amax(-1) if S else sp.amax(-1))[..., None]
    ep, eo = (sp - m).exp(), (so - m).exp()
    o = (ep.transpose(0, 1).reshape(Hkv, B * G, P) @ vp).view(Hkv, B, G, d).transpose(0, 1) + eo @ v
    o = o / (ep.sum(-1) + eo.sum(-1))[..., None]
    return o.reshape(B, c["Hq"], d).half()


def _turned(x, cos, sin, pair):
    """The first 2 n values of the last axis rotated by n angles, the rest as they are."""
    n = cos.shape[-1]
    if pair == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * n:]], -1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., 2 * n:]], -1)


EPS = 1e-6


def _rows_plain(s):
    c = s["case"]
    B, T, Hq, Hkv, d, cap = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "cap"))
    x = s["x"].float().view(B, T, Hq + 2 * Hkv, d).transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if s["wq"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["wq"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["wk"]
    j = torch.arange(T, device=x.device)
    if s["rope"] is not None:
        t = s["rope"][(s["pos"][:, None] + j).long()][:, None]  # [B, 1, T, rot]
        n = t.shape[-1] // 2
        q, k = (_turned(z, t[..., :n], t[..., n:], c["pair"]) for z in (q, k))
    n_new = s["len"][:, None] if s["len"] is not None else torch.full((B, 1), T, device=x.device)
    s["q"] = torch.where((j < n_new)[:, None, :, None], q.half(), s["q"])
    at = torch.arange(cap, device=x.device) - s["slot"][:, None]  # which token a slot gets
    live = ((at >= 0) & (at < n_new))[:, None, :, None]
    pick = at.clamp(0, T - 1)[:, None, :, None].expand(B, Hkv, cap, d)
    s["k"] = torch.where(live, k.half().gather(2, pick), s["k"])
    s["v"] = torch.where(live, v.half().gather(2, pick), s["v"])
    return s["q"], s["k"], s["v"]


def _free_plain(s):
    rows = s["done"].long()
    pps = s["table"].shape[1]
    held = torch.arange(pps, device=rows.device) < s["held"][rows][:, None]
    s["ref"].index_add_(0, torch.where(held, s["table"][rows], 0).flatten().long(), -held.int().flatten())
    s["held"][rows] = 0


def _fork_plain(s):
    page, n = s["case"]["page"], s["case"]["pages"]
    table, held, ref = s["table"], s["held"], s["ref"]
    par, kid, share, new = s["parent"].long(), s["child"].long(), s["share"].long(), s["new"].long()
    pps = table.shape[1]
    grow, has = par == kid, held[kid].long()
    src = table[par.clamp_min(0)]
    total, at = (new + page - 1) // page, share // page            # pages to hold, page that is written next
    old = src.gather(1, at.clamp_max(pps - 1)[:, None])[:, 0].long()
    cow = grow & (at < has) & (ref[old] > 1)                       # a shared page that would be written
    copied = (share % page > 0) & (~grow | cow)
    first = torch.where(grow, has, at)
    fresh = (total - first).clamp_min(0) + cow.long()
    off = fresh.cumsum(0) - fresh
    free = ref == 0
    page_of = torch.zeros(n + 1, dtype=torch.int64, device=ref.device)
    page_of.scatter_(0, torch.where(free, free.cumsum(0) - 1, n), torch.arange(n, device=ref.device))
    j = torch.arange(pps, device=ref.device)
    over = cow[:, None] & (j == at[:, None])
    take = over | ((j >= first[:, None]) & (j < total[:, None]))
    rank = off[:, None] + torch.where(over, 0, j - first[:, None] + cow.long()[:, None])
    shared = ~grow[:, None] & (j < at[:, None])
    rows = torch.where(take, page_of[rank.clamp(0, n)].int(), torch.where(shared, src, table[kid]))
    table[kid] = rows
    held[kid] = torch.where(grow, torch.maximum(has, total), total).int()
    ref.index_add_(0, torch.where(take | shared, rows, 0).flatten().long(), (take | shared).int().flatten())
    ref.index_add_(0, old, -cow.int())
    moved = copied.nonzero()[:, 0]
    a, b = old[moved], rows.gather(1, at.clamp_max(pps - 1)[:, None])[moved, 0].long()
    for x in s["arrays"].values():
        x[:, b] = x[:, a]
    return torch.stack([torch.zeros_like(fresh[0]), fresh.sum(), copied.sum(), torch.zeros_like(fresh[0])]).int()


def _pack_plain(s):
    table, held, ref = s["table"], s["held"], s["ref"]
    live = ref > 0
    n_live = live.sum()
    at = torch.arange(ref.numel(), device=ref.device)
    holes, movers = ((at < n_live) & ~live).nonzero()[:, 0], ((at >= n_live) & live).nonzero()[:, 0]
    to = at.clone()
    to[movers] = holes
    mine = torch.arange(table.shape[1], device=ref.device) < held[:, None]
    table.copy_(torch.where(mine, to[table.long()].int(), table))
    ref[holes] = ref[movers]
    ref[movers] = 0
    for x in s["arrays"].values():
        x[:, holes] = x[:, movers]
    return torch.stack([torch.zeros_like(n_live), n_live, (to != at).sum(), torch.zeros_like(n_live)]).int()


def _pool_out(s, result):
    return {"table": s["table"], "held": s["held"], "ref": s["ref"], "result": result, **s["arrays"]}


def _plain(s):
    if s["op"] == "attn":
        return _attn_plain(s)
    if s["op"] == "rows":
        return _rows_plain(s)
    s["book"].copy_(s["start"])
    if s["op"] == "pack":
        _free_plain(s)
        return _pool_out(s, _pack_plain(s))
    _free_plain(s)
    return _pool_out(s, _fork_plain(s))


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from turboquant_kv_cache_gb300 import binding as tb
    c = s["case"]
    if s["op"] == "attn":
        return tb.tq_decode_attn_shared(s["K_p"], s["V_p"], s["K_o"], s["V_o"], s["q"], prefix_ctx=c["prefix"], ctx=c["own"],
                                        kv_len=s["len"], workspace=s["ws"])
    if s["op"] == "rows":
        return tb.tq_qkv_norm_rope(s["x"], c["Hq"], c["Hkv"], c["d"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                   rope=s["rope"], interleaved=c["pair"] == "next", pos=s["pos"], new_len=s["len"],
                                   slot=s["slot"], q_out=s["q"], k_out=s["k"], v_out=s["v"])
    s["book"].copy_(s["start"])  # the pool as the step finds it
    tb.tq_pages_free(s["pool"], s["done"])
    if s["op"] == "pack":
        return _pool_out(s, tb.tq_pages_compact(s["pool"], workspace=s["ws"], result=s["result"]))
    return _pool_out(s, tb.tq_pages_fork(s["pool"], s["parent"], s["child"], s["share"], s["new"], workspace=s["ws"],
                                         result=s["result"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and exact values
def work(case):
    if case["op"] == "attn":
        d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
        rec = d * (kbits + vbits) / 8 + 2 * d // kb + 2 * d // vb
        tokens = case["prefix"] + 0.75 * case["own"] * case["B"]
        pairs = case["B"] * case["Hq"] * (case["prefix"] + 0.75 * case["own"])
        return {"bytes": tokens * case["Hkv"] * rec + 4 * case["B"] * case["Hq"] * d, "flops": 4.0 * d * pairs}
    if case["op"] == "rows":
        n = case["B"] * case["T"] * (0.67 if case["ragged"] else 1.0)
        width = (case["Hq"] + 2 * case["Hkv"]) * case["d"]
        return {"bytes": n * (width * ((4 if case["f32"] else 2) + 2) + 4 * case["rot"]), "flops": 8.0 * n * width}
    d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
    page = case["layers"] * case["Hkv"] * case["page"] * (d * (kbits + vbits) / 8 + 2 * d // kb + 2 * d // vb)
    book = 4.0 * (case["pages"] + case["seqs"] * (case["pages_per_seq"] + 1))
    moved = 0.8 * case["forks"] if case["op"] == "step" else 0.2 * case["pages"]
    return {"bytes": 3 * book + 2 * moved * page, "flops": 0.0}


def _exact_vectors(codes, scales, d, block, bits):
    """Records to vectors in 64 bits, code by code from the packed layout's definition."""
    w = codes.reshape(-1, d // 32, 4 * bits).to(torch.int64)
    w = (w.view(*w.shape[:2], bits, 4) << torch.tensor([0, 8, 16, 24], device=w.device)).sum(-1)
    bit = lambda word, at: (w[..., word] >> at) & 1  # noqa: E731
    out = []
    for i in range(32):
        run8, k = divmod(i, 8)
        if bits == 4:
            c = (w[..., run8] >> (4 * k)) & 15
        elif bits == 3:
            c = (w[..., run8] >> (4 * k)) & 7 if run8 < 3 else sum(bit(j, 4 * k + 3) << j for j in range(3))
        elif bits == 2:
            c = (w[..., run8 % 2] >> (4 * k + 2 * (run8 // 2))) & 3
        else:
            c = bit(0, 4 * k + run8)
        out.append(c)
    c = _levels(bits, block)[torch.stack(out, -1)].reshape(-1, d // block, block)
    h = 1
    while h < block:  # the transform as butterflies
        a, b = c.reshape(-1, block // (2 * h), 2, h).unbind(2)
        c = torch.stack([a + b, a - b], 2).reshape(-1, d // block, block)
        h *= 2
    c = c / math.sqrt(block) * scales.reshape(-1, d // block, 1).double()
    return c.reshape(*codes.shape[:-1], d) * torch.tensor(_signs(SIGN_SEED, d), dtype=torch.float64, device=c.device)


def _exact_attn(s):
    c = s["case"]
    d, (kb, kbits), (vb, vbits) = LAYOUTS[c["layout"]]
    B, Hq, Hkv, P = c["B"], c["Hq"], c["Hkv"], c["prefix"]
    lens = s["len"].tolist()
    out = torch.empty(B, Hq, d, dtype=torch.float64, device="cuda")

    def tokens(cache, table, b, h, n, block, bits):
        codes, scales = cache
        if table is not None:
            t = torch.arange(n, device="cuda")
            at = table[b, t // c["page"]].long()
            codes, scales = codes[at, h, t % c["page"]], scales[at, h, t % c["page"]]
        else:
            codes, scales = codes[b, h, :n], scales[b, h, :n]
        return _exact_vectors(codes, scales, d, block, bits)

    for h in range(Hkv):
        kp, vp = tokens(s["kp"], s["table_p"], 0, h, P, kb, kbits), tokens(s["vp"], s["table_p"], 0, h, P, vb, vbits)
        for b in range(B):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k, v = kp, vp
            if lens[b]:
                k = torch.cat([kp, tokens(s["k"], s["table_o"], b, h, lens[b], kb, kbits)])
                v = torch.cat([vp, tokens(s["v"], s["table_o"], b, h, lens[b], vb, vbits)])
            w = s["q"][b, heads].double() @ k.T / math.sqrt(d)
            out[b, heads] = torch.softmax(w, -1) @ v
    return out


def _exact_rows(s):
    c = s["case"]
    B, T, Hq, Hkv, d, rot = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "rot"))
    x = s["x"].double().reshape(B, T, Hq + 2 * Hkv, d)
    for lo, n, w in ((0, Hq, s["wq"]), (Hq, Hkv, s["wk"])):
        if w is not None:
            z = x[:, :, lo:lo + n]
            x[:, :, lo:lo + n] = z / ((z * z).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
    if rot:
        i = torch.arange(rot // 2, device="cuda")
        a, b = (i, i + rot // 2) if c["pair"] == "half" else (2 * i, 2 * i + 1)
        t = s["rope"].double()[s["pos"].long()[:, None] + torch.arange(T, device="cuda")]
        z = torch.complex(x[:, :, :Hq + Hkv, a], x[:, :, :Hq + Hkv, b]) * torch.complex(t[..., :rot // 2], t[..., rot // 2:])[:, :, None]
        x[:, :, :Hq + Hkv, a], x[:, :, :Hq + Hkv, b] = z.real.clone(), z.imag.clone()
    out = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (s["q"], s["k"], s["v"])]
    lens = s["len"].tolist() if s["len"] is not None else [T] * B
    for b, (n, at) in enumerate(zip(lens, s["slot"].tolist())):
        out[0][b, :, :n] = x[b, :n, :Hq].transpose(0, 1)
        out[1][b, :, at:at + n] = x[b, :n, Hq:Hq + Hkv].transpose(0, 1)
        out[2][b, :, at:at + n] = x[b, :n, Hq + Hkv:].transpose(0, 1)
    return tuple(out)


def exact(case, seed):
    if case["op"] in ("step", "pack"):  # whole numbers and moved bytes: nothing is computed
        return None
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_rows(s)
