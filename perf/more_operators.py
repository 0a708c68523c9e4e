"""Operators that a serving step needs around the packed KV cache, as measured cases.

  slots   tq_batch_slots: request lengths to the place of every row of a ragged batch (sequence, position, cache slot, block table)
  append  tq_append_kv_slots: the rows of a ragged batch quantised into their slots, keys and values
  beam    tq_beam_select: the best continuations over all beams and the whole vocabulary
  states  tq_states_reorder: caches, norms and token histories of beams follow their parents, in place
  tables  tq_pages_reorder: the same for a paged cache: rows of the page table and the pages' reference counts

`run` computes them with elementary torch operations where `own` is false, and with the library's calls where it is true."""
import math

import numpy as np
import torch

own = False

# Codec settings by name, as the repository's workloads have them: head_dim, then (block, bits) of keys and values.
LAYOUTS = {
    "turbo3_d128": (128, (32, 3), (32, 3)),           # Qwen3-8B-shaped cache
    "turbo4k_turbo3v_d256": (256, (32, 4), (32, 3)),  # head_dim 256, long context
    "pervec4_d64": (64, (64, 4), (64, 4)),            # Llama-3.2-1B-shaped cache, one norm per vector
    "pervec2k_3v_d128": (128, (128, 2), (128, 3)),    # 2-bit keys, one norm per vector
}
SIGN_SEED = 1


def listed():
    return [
        # a decode step beside two short prompts: 8 requests, their rows in a buffer of fixed size, a table row for each
        {"name": "slots_small", "op": "slots", "B": 8, "rows": 96, "fill": 0.8, "page": 32, "pages_per_seq": 64, "tables": True},
        # the whole queue of a large server: prompts of very unequal lengths
        {"name": "slots_large", "op": "slots", "B": 2048, "rows": 1000003, "fill": 0.97, "page": 64, "pages_per_seq": 256,
         "tables": False},
        # a decode step: one token of each of 8 requests
        {"name": "append_step", "op": "append", "layout": "turbo3_d128", "B": 8, "rows": 8, "Hkv": 8, "page": 32, "f32": False},
        # a ragged chunk of odd size, contiguous cache, a norm per vector, head_dim 64
        {"name": "append_odd", "op": "append", "layout": "pervec4_d64", "B": 5, "rows": 701, "Hkv": 7, "page": 0, "f32": False},
        # a prefill batch of many prompts into pages
        {"name": "append_prompts", "op": "append", "layout": "turbo3_d128", "B": 24, "rows": 32768, "Hkv": 8, "page": 64,
         "f32": False},
        # two requests with four beams, half-precision logits
        {"name": "beam_small", "op": "beam", "B": 2, "W": 4, "V": 32000, "n_out": 8, "f32": False, "done": False, "allowed": 0,
         "keep": False},
        # odd sizes: rows that start anywhere, a grammar that allows 40 tokens, finished beams
        {"name": "beam_grammar", "op": "beam", "B": 7, "W": 5, "V": 50021, "n_out": 5, "f32": True, "done": True, "allowed": 40,
         "keep": True},
        # a large batch with wide beams over a large vocabulary
        {"name": "beam_large", "op": "beam", "B": 32, "W": 16, "V": 128256, "n_out": 16, "f32": True, "done": True, "allowed": 0,
         "keep": True},
        # four beams of one request behind a short prompt, one layer
        {"name": "states_small", "op": "states", "layout": "turbo3_d128", "layers": 1, "groups": 1, "W": 4, "Hkv": 8, "cap": 1024,
         "len": 700, "dead": 2},
        # eight requests with eight beams, four layers of a cache with a norm per vector
        {"name": "states_large", "op": "states", "layout": "pervec4_d64", "layers": 4, "groups": 8, "W": 8, "Hkv": 8, "cap": 2048,
         "len": 1531, "dead": 4},
        # the same step over pages: a small server
        {"name": "tables_small", "op": "tables", "groups": 4, "W": 4, "pages_per_seq": 33, "shared": 8, "dead": 2},
        # 512 sequences of 8 beams each behind long prompts
        {"name": "tables_large", "op": "tables", "groups": 64, "W": 8, "pages_per_seq": 512, "shared": 300, "dead": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "append", "append", "beam", "beam", "beam", "states", "states", "tables"])
    if op == "slots":
        rows = _log(rng, 1, 500000)
        return {"op": op, "B": _log(rng, 1, 2048), "rows": rows, "fill": rng.choice([0.3, 0.8, 1.0]),
                "page": rng.choice([0, 32, 64, 96]), "pages_per_seq": rng.choice([33, 128, 256]), "tables": rows < 20000}
    if op == "append":
        name = rng.choice(sorted(LAYOUTS))
        Hkv = rng.choice([1, 2, 3, 4, 7, 8])
        return {"op": op, "layout": name, "B": _log(rng, 1, 64), "rows": min(_log(rng, 1, 32768), 33000000 // (Hkv * LAYOUTS[name][0])),
                "Hkv": Hkv, "page": rng.choice([0, 32, 64, 96]), "f32": rng.random() < 0.3}
    if op == "beam":
        W, V = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32]), _log(rng, 100, 200000)
        B = min(_log(rng, 1, 48), max(1, 60000000 // (W * V)))
        keep = rng.random() < 0.5
        return {"op": op, "B": B, "W": W, "V": V, "n_out": W if keep else rng.choice([1, W, 2 * W]), "f32": rng.random() < 0.5,
                "done": rng.random() < 0.5, "allowed": rng.choice([0, 0, 3, min(V, 90)]), "keep": keep}
    W = rng.choice([2, 3, 4, 5, 8, 16, 32])
    if op == "states":
        cap = _log(rng, 64, 4096)
        name, Hkv = rng.choice(sorted(LAYOUTS)), rng.choice([1, 2, 8])
        groups = min(_log(rng, 1, 16), max(1, 200000000 // (W * Hkv * cap * LAYOUTS[name][0])))
        return {"op": op, "layout": name, "layers": 1, "groups": groups, "W": W, "Hkv": Hkv, "cap": cap,
                "len": rng.randint(1, cap), "dead": rng.randint(1, W - 1)}
    pps = _log(rng, 8, 512)
    return {"op": op, "groups": _log(rng, 1, 64 if W < 16 else 16), "W": W, "pages_per_seq": pps, "shared": rng.randint(0, pps // 2),
            "dead": rng.randint(1, W - 1)}


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


_EDGES = {}


def _edges(bits):
    """Borders of the cells of N(0, 1)."""
    if bits not in _EDGES:
        c = _codebook(bits)
        _EDGES[bits] = [0.5 * (a + b) for a, b in zip(c, c[1:])]
    return torch.tensor(_EDGES[bits], dtype=torch.float64, device="cuda")


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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _ragged(rnd, B, rows, most):
    """Rows of each of B requests, `rows` in all where they fit: one token for most, prompts of unequal lengths for the others."""
    w = np.where(rnd.random(B) < 0.5, 0.0, rnd.pareto(1.2, B) + 0.1)
    if B * most < rows:
        rows = B * most
    if not w.any():
        w[rnd.integers(B)] = 1.0
    n = np.minimum((w / w.sum() * max(0, rows - B)).astype(np.int64) + (1 if rows >= B else 0), most)
    for i in rnd.permutation(B):  # what rounding and the longest allowed left over
        n[i] += min(most - n[i], rows - n.sum())
    return n


def _prepare_slots(case, gen, rnd):
    B, page, pps = case["B"], case["page"], case["pages_per_seq"]
    cap = pps * (page or 64)
    new = _ragged(rnd, B, int(case["rows"] * case["fill"]), cap)
    have = (rnd.random(B) * (cap - new + 1)).astype(np.int64)
    s = {"op": "slots", "case": case, "new": _i32(new), "have": _i32(have), "cap": cap, "table": None}
    if page:
        n = B * pps
        s["table"] = _i32(rnd.permutation(n).reshape(B, pps))
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        s["out"] = tb.BatchSlots.new(B, case["rows"], row_pages=pps if case["tables"] and page else 0)
    return s


def _keep_off(u, edges, room=0.01):
    """Coordinates within `room` of a cell's border moved away from it."""
    k = torch.bucketize(u, edges.to(u.dtype))
    lo = torch.cat([edges.new_full((1,), -math.inf), edges]).to(u.dtype)[k] + room
    hi = torch.cat([edges, edges.new_full((1,), math.inf)]).to(u.dtype)[k] - room
    return torch.minimum(torch.maximum(u, lo), hi)


def _vectors(gen, n, d, block, bits, dtype):
    """Gaussian vectors.  Codes are whole numbers, and a coordinate on the border of two cells could go to either in 32 bits:
    there is none within a hundredth of a deviation of one."""
    out = torch.empty(n, d, dtype=dtype, device="cuda")
    edges, had = _edges(bits).float(), _hadamard(block).float().cuda()
    sign = torch.tensor(_signs(SIGN_SEED, d), device="cuda")
    step = max(1, (1 << 25) // d)
    for i in range(0, n, step):
        m = min(step, n - i)
        y = torch.randn(m, d // block, block, generator=gen, device="cuda")
        size = y.norm(dim=-1, keepdim=True) / math.sqrt(block)
        y = _keep_off(y / size, edges) * size
        out[i:i + m] = ((y @ had).flatten(1) * sign).to(dtype)
    return out


def _prepare_append(case, gen, rnd):
    d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
    B, H, rows, page = case["B"], case["Hkv"], case["rows"], case["page"]
    dt = torch.float32 if case["f32"] else torch.float16
    s = {"op": "append", "case": case}
    s["k"] = _vectors(gen, rows * H, d, kb, kbits, dt).view(rows, H, d)
    s["v"] = _vectors(gen, rows * H, d, vb, vbits, dt).view(rows, H, d)
    most = min(rows, 4 * rows // B + 1)  # of one request
    new = _ragged(rnd, B, rows, most)
    have = rnd.integers(0, 65, size=B)
    if page:  # the sequences' pages in shuffled places, some spare
        pages = -(-(new + have) // page)
        n_pages = rows // page + 3 * B + 3
        lead, place, at = (n_pages, H, page), rnd.permutation(n_pages), 0
    else:
        cap = most + 67
        lead = (B, H, cap)
    slot = []
    for b in range(B):
        pos = have[b] + np.arange(new[b])
        if page:
            slot.append(place[at + pos // page] * page + pos % page)
            at += pages[b]
        else:
            slot.append(b * cap + pos)
    slot = np.concatenate(slot).astype(np.int64)
    slot = np.where(rnd.random(rows) < 0.02, -1, slot) if rows > 50 else slot  # rows of requests that were cancelled
    s["slot"] = torch.from_numpy(slot).cuda()
    for name, blk, bits in (("K", kb, kbits), ("V", vb, vbits)):
        s[name] = (torch.zeros(*lead, d * bits // 8, dtype=torch.uint8, device="cuda"),
                   torch.zeros(*lead, d // blk, dtype=torch.float16, device="cuda"))
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        Lk, Lv = tb.make_layout(d, kb, kbits, sign_seed=SIGN_SEED), tb.make_layout(d, vb, vbits, sign_seed=SIGN_SEED)
        s["cache"] = tb.PackedKV.of(Lk, *s["K"]), tb.PackedKV.of(Lv, *s["V"])
    else:
        s["books"] = {n: (_edges(b).float(), _hadamard(k).float().cuda()) for n, k, b in (("K", kb, kbits), ("V", vb, vbits))}
        s["signs"] = torch.tensor(_signs(SIGN_SEED, d), device="cuda")
    return s


EOS = 2


def _prepare_beam(case, gen, rnd):
    B, W, V = case["B"], case["W"], case["V"]
    # a few likely tokens and a long tail, as a trained model's; every row prefers others
    liked = torch.rand(B, 1, V, generator=gen, device="cuda").mul_(V).add_(1.0).log_().mul_(-1.2)
    x = torch.randn(B, W, V, generator=gen, device="cuda").mul_(1.5).add_(liked)
    if case["allowed"]:  # a grammar: all but a few tokens are shut out
        live = torch.rand(B, 1, V, generator=gen, device="cuda") < case["allowed"] / V
        live[:, :, rnd.integers(V, size=2)] = True
        x.masked_fill_(~live, -math.inf)
    x = x if case["f32"] else x.half()
    scores = -torch.rand(B, W, generator=gen, device="cuda").mul_(6.0)
    if W > 3:
        scores[0, 1:] = -math.inf  # a request at its first step: one beam lives
    done = torch.zeros(B, W, dtype=torch.uint8, device="cuda")
    if case["done"]:
        done = (torch.rand(B, W, generator=gen, device="cuda") < 0.2).to(torch.uint8)
    s = {"op": "beam", "case": case, "x": x, "scores": scores, "done": done}
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        s["ws"] = torch.empty(tb.tq_beam_workspace_bytes(B, W, V, case["n_out"]), dtype=torch.uint8, device="cuda")
    return s


def _parents(rnd, groups, W, dead):
    """Beams after a step that keeps survivors in place: `dead` of each group's W follow one of the others."""
    parent = np.arange(groups * W).reshape(groups, W)
    for g in range(groups):
        p = rnd.permutation(W)
        parent[g, p[:dead]] = g * W + rnd.choice(p[dead:], dead)
    return parent.ravel()


def _prepare_states(case, gen, rnd):
    d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
    n, H, cap = case["groups"] * case["W"], case["Hkv"], case["cap"]
    arrays = []
    for _ in range(case["layers"]):
        for blk, bits in ((kb, kbits), (vb, vbits)):
            arrays.append(torch.randint(0, 256, (n, H, cap, d * bits // 8), dtype=torch.uint8, generator=gen, device="cuda"))
            arrays.append(torch.rand(n, H, cap, d // blk, generator=gen, device="cuda").half())
    arrays.append(torch.randint(0, 30000, (n, 1, cap, 1), dtype=torch.int32, generator=gen, device="cuda"))  # token history
    lens = np.minimum(case["len"], case["len"] - rnd.integers(0, 1 + case["len"] // 20, size=n))
    s = {"op": "states", "case": case, "arrays": arrays, "len": _i32(lens),
         "parent": _i32(_parents(rnd, case["groups"], case["W"], case["dead"]))}
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        s["states"] = tb.StateArrays(arrays, s["len"])
    return s


def _prepare_tables(case, gen, rnd):
    W, pps, n = case["W"], case["pages_per_seq"], case["groups"] * case["W"]
    pages = case["groups"] * (case["shared"] + W * (pps - case["shared"])) + 7
    place, at = rnd.permutation(pages), 0
    table, held = rnd.integers(0, pages, size=(n, pps)), np.zeros(n, np.int64)
    ref = np.zeros(pages, np.int64)
    for g in range(case["groups"]):
        prompt = place[at:at + case["shared"]]
        at += case["shared"]
        for i in range(g * W, g * W + W):
            m = case["shared"] + int(rnd.integers(0, pps - case["shared"] + 1))
            table[i, :case["shared"]] = prompt
            table[i, case["shared"]:m] = place[at:at + m - case["shared"]]
            at += m - case["shared"]
            held[i] = m
            ref[table[i, :m]] += 1
    start = _i32(np.concatenate([table.ravel(), held, ref]))
    b = start.clone()
    s = {"op": "tables", "case": case, "start": start, "book": b, "table": b[:n * pps].view(n, pps), "held": b[n * pps:n * pps + n],
         "ref": b[n * pps + n:], "parent": _i32(_parents(rnd, case["groups"], W, case["dead"]))}
    if own:
        from turboquant_kv_cache_gb300 import binding as tb
        s["pool"] = tb.PagePool(s["table"], s["held"], s["ref"], 64)
        s["result"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        s["ws"] = torch.empty(tb.tq_pages_reorder_workspace_bytes(n, pps, n), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen, rnd = _gen(seed), np.random.default_rng(int(seed))
    return {"slots": _prepare_slots, "append": _prepare_append, "beam": _prepare_beam, "states": _prepare_states,
            "tables": _prepare_tables}[case["op"]](case, gen, rnd)


# ------------------------------------------------------------------ plain forms
def _slots_plain(s):
    c, new, have = s["case"], s["new"].long(), s["have"].long()
    end = new.cumsum(0)
    start = torch.cat([torch.zeros_like(end[:1]), end])
    r = torch.arange(c["rows"], device=end.device)
    live = r < end[-1]
    b = torch.searchsorted(end, r, right=True).clamp_max(c["B"] - 1)
    pos = have[b] + r - start[b]
    if s["table"] is not None:
        slot = s["table"][b, (pos // c["page"]).clamp_max(c["pages_per_seq"] - 1)].long() * c["page"] + pos % c["page"]
    else:
        slot = b * s["cap"] + pos
    none = torch.full_like(r, -1)
    out = {"row_start": start.int(), "seq": torch.where(live, b, none).int(), "pos": torch.where(live, pos, none).int(),
           "slot": torch.where(live, slot, none), "row_len": torch.where(live, pos + 1, 0).int(),
           "result": torch.stack([0 * end[-1], end[-1], 0 * end[-1], 0 * end[-1]]).int()}
    if c["tables"] and s["table"] is not None:
        out["row_table"] = torch.where(live[:, None], s["table"][b], 0)
    return out


def _pack(codes, bits):
    """Codes [N, d] to packed words: a nibble per code of a word, 8 codes a word, see the record of the C header."""
    n, d = codes.shape
    c = codes.view(n, d // 32, 4, 8)                             # group, run of eight, place
    at = 4 * torch.arange(8, device=c.device)
    nib = (c << at).sum(-1)                                      # [n, groups, 4]
    if bits == 4:
        w = nib
    elif bits == 3:
        w = nib[:, :, :3] | torch.stack([(((c[:, :, 3] >> k) & 1) << (at + 3)).sum(-1) for k in range(3)], -1)
    else:
        w = nib[:, :, :2] | (nib[:, :, 2:] << 2)
    return w.to(torch.int32).contiguous().view(torch.uint8).view(n, d * bits // 8)


def _append_plain(s):
    c = s["case"]
    d, (kb, kbits), (vb, vbits) = LAYOUTS[c["layout"]]
    live = s["slot"] >= 0
    for x, name, blk, bits in ((s["k"], "K", kb, kbits), (s["v"], "V", vb, vbits)):
        codes, scales = s[name]
        edges, had = s["books"][name]
        y = (x.float() * s["signs"]).unflatten(-1, (-1, blk))
        size = y.square().sum(-1).sqrt()
        code = ((y @ had) * (math.sqrt(blk) / size)[..., None] > edges[:, None, None, None, None]).sum(0)
        n, H, cap = codes.shape[:3]
        # a row that has no slot is written to a spare one, which is dropped
        at = torch.where(live, s["slot"], n * cap)
        rec = ((at // cap)[:, None] * H + torch.arange(H, device=x.device)) * cap + (at % cap)[:, None]
        rec = torch.where(live[:, None], rec, n * H * cap).flatten()
        for to, rows in ((codes, _pack(code.flatten(0, 1).flatten(1), bits)), (scales, size.half().flatten(0, 1))):
            all_rows = torch.cat([to.view(n * H * cap, -1), to.new_zeros(1, to.shape[-1])])
            all_rows[rec] = rows
            to.copy_(all_rows[:-1].view_as(to))
    return {"k_codes": s["K"][0], "k_scales": s["K"][1], "v_codes": s["V"][0], "v_scales": s["V"][1]}


def _beam_plain(s):
    c, x = s["case"], s["x"].float()
    B, W, V, n = c["B"], c["W"], c["V"], c["n_out"]
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    lse = m.double() + (x - m).exp().sum(-1, keepdim=True, dtype=torch.float64).log()  # a long sum
    # scores in 64 bits: two candidates next to each other are told apart
    score = s["scores"].double()[..., None] + (x.double() - lse)
    done = s["done"].bool()
    stay = torch.where(torch.arange(V, device=x.device) == EOS, s["scores"].double()[..., None], -math.inf)
    score = torch.where(done[..., None], stay, score)
    best, flat = score.view(B, W * V).sort(dim=-1, descending=True, stable=True)  # ties: the lowest place first
    best, flat = best[:, :n], flat[:, :n]
    beam, token = flat // V, flat % V
    ended = done.gather(1, beam) | (token == EOS)
    if c["keep"]:  # a beam's best child stays in its place, the others go to the places left, in order
        j = torch.arange(n, device=x.device)
        same = beam[:, :, None] == beam[:, None, :]
        first = ~(same & (j < j[:, None])).any(-1)
        used = torch.zeros(B, W, dtype=torch.int64, device=x.device).scatter_(1, beam, 1)
        free_at = (used * W + j).sort(dim=-1, stable=True).indices  # free places, then the others
        place = torch.where(first, beam, free_at.gather(1, ((~first).cumsum(1) - 1).clamp_min(0)))
        order = place.argsort(1)
        best, beam, token, ended = (t.gather(1, order) for t in (best, beam, token, ended))
    return {"scores": best.float(), "parent": (beam + W * torch.arange(B, device=x.device)[:, None]).int(), "token": token.int(),
            "done": ended.to(torch.uint8)}


def _states_plain(s):
    p, cap = s["parent"].long(), s["case"]["cap"]
    live = (torch.arange(cap, device=p.device) < s["len"][p][:, None])[:, None, :, None]
    for a in s["arrays"]:
        a.copy_(torch.where(live, a[p], a))
    return s["arrays"]


def _tables_plain(s):
    s["book"].copy_(s["start"])
    p, table, held, ref = s["parent"].long(), s["table"], s["held"], s["ref"]
    at = torch.arange(table.shape[1], device=p.device)
    rows, mine = table[p], at < held[:, None]
    theirs = at < held[p][:, None]
    ref.index_add_(0, torch.where(mine, table, 0).flatten().long(), -mine.int().flatten())
    ref.index_add_(0, torch.where(theirs, rows, 0).flatten().long(), theirs.int().flatten())
    table.copy_(torch.where(theirs, rows, table))
    held.copy_(held[p])
    moved = (p != torch.arange(p.numel(), device=p.device)).sum()
    return {"table": table, "held": held, "ref": ref, "result": torch.stack([0 * moved, moved, 0 * moved, 0 * moved]).int()}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from turboquant_kv_cache_gb300 import binding as tb
    c = s["case"]
    if s["op"] == "slots":
        o = tb.tq_batch_slots(s["new"], s["have"], S_cap=s["cap"], page_table=s["table"], page_size=c["page"], out=s["out"])
        got = {"row_start": o.row_start, "seq": o.seq, "pos": o.pos, "slot": o.slot, "row_len": o.row_len, "result": o.result}
        return {**got, "row_table": o.row_table} if o.row_table is not None else got
    if s["op"] == "append":
        K, V = s["cache"]
        tb.tq_append_kv_slots(K, s["k"], s["slot"])
        tb.tq_append_kv_slots(V, s["v"], s["slot"])
        return {"k_codes": K.codes, "k_scales": K.scales, "v_codes": V.codes, "v_scales": V.scales}
    if s["op"] == "beam":
        scores, parent, token, done = tb.tq_beam_select(s["x"], s["scores"], n_out=c["n_out"], done=s["done"], eos=EOS,
                                                        keep_place=c["keep"], workspace=s["ws"])
        return {"scores": scores, "parent": parent, "token": token, "done": done}
    if s["op"] == "states":
        tb.tq_states_reorder(s["states"], s["parent"], c["W"])
        return s["arrays"]
    s["book"].copy_(s["start"])  # the pool as the step finds it
    result = tb.tq_pages_reorder(s["pool"], s["parent"], workspace=s["ws"], result=s["result"])
    return {"table": s["table"], "held": s["held"], "ref": s["ref"], "result": result}


def run(state):
    if own:
        return _own(state)
    return {"slots": _slots_plain, "append": _append_plain, "beam": _beam_plain, "states": _states_plain,
            "tables": _tables_plain}[state["op"]](state)


# ------------------------------------------------------------------ work and exact values
def work(case):
    if case["op"] == "slots":
        table = 4.0 * case["rows"] * case["pages_per_seq"] if case["tables"] and case["page"] else 0.0
        return {"bytes": 12.0 * case["B"] + 20.0 * case["rows"] + table, "flops": 0.0}
    if case["op"] == "beam":
        read = case["B"] * case["W"] * case["V"] * (0.8 if case["done"] else 1.0)  # a finished beam's row need not be read
        return {"bytes": read * (4 if case["f32"] else 2), "flops": 4.0 * read}
    if case["op"] == "append":
        d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
        vec = 2 * d * (4 if case["f32"] else 2) + d * (kbits + vbits) / 8 + 2 * d // kb + 2 * d // vb
        n = float(case["rows"] * case["Hkv"])
        return {"bytes": n * vec + 16.0 * case["rows"], "flops": n * 2 * d * (math.log2(kb) + math.log2(vb) + 8)}
    alive = case["W"] - case["dead"]
    followed = alive * (1.0 - (1.0 - 1.0 / alive) ** case["dead"])  # survivors that some other beam follows, on average
    if case["op"] == "tables":
        entries = case["groups"] * (case["shared"] + 0.5 * (case["pages_per_seq"] - case["shared"]))
        own_pages = case["groups"] * 0.5 * (case["pages_per_seq"] - case["shared"])
        return {"bytes": 4.0 * entries * (2 * case["dead"] + followed) + 16.0 * own_pages * case["dead"], "flops": 0.0}
    d, (kb, kbits), (vb, vbits) = LAYOUTS[case["layout"]]
    token = case["layers"] * case["Hkv"] * (d * (kbits + vbits) / 8 + 2 * d // kb + 2 * d // vb) + 4
    return {"bytes": case["groups"] * (case["dead"] + followed) * 0.975 * case["len"] * token, "flops": 0.0}


def _exact_beam(s):
    """Scores in 64 bits, request by request: the best n by (score, place) in a sorted list."""
    c = s["case"]
    B, W, V, n = c["B"], c["W"], c["V"], c["n_out"]
    out = torch.empty(B, n, dtype=torch.float64, device="cuda")
    for b in range(B):
        x, sc, done = s["x"][b].double(), s["scores"][b].double(), s["done"][b].tolist()
        rows = []
        for w in range(W):
            if done[w]:
                row = torch.full((V,), -math.inf, dtype=torch.float64, device="cuda")
                row[EOS] = sc[w]
            else:
                row = sc[w] + (x[w] - torch.logsumexp(x[w], 0))
            rows.append(row)
        flat = torch.cat(rows)
        least = flat.topk(n).values[-1]
        at = (flat >= least).nonzero()[:, 0]
        at = at[: 4 * n + 64] if math.isinf(least) else at
        if math.isinf(least):
            fine = (flat > least).nonzero()[:, 0]
            at = torch.unique(torch.cat([fine, at]))
        best = sorted(zip((-flat[at]).tolist(), at.tolist()))[:n]
        if c["keep"]:
            place, left = {}, []
            for v, i in best:
                if i // V in place:
                    left.append(v)
                else:
                    place[i // V] = v
            for k in range(W):
                if k not in place:
                    place[k] = left.pop(0)
            best = [(place[k], 0) for k in range(W)]
        out[b] = torch.tensor([-v for v, _ in best], dtype=torch.float64)
    return {"scores": out, "parent": None, "token": None, "done": None}


def _exact_append(s):
    """Norms of the rotation blocks in 64 bits, slot by slot; codes are whole numbers."""
    c = s["case"]
    d, (kb, _), (vb, _) = LAYOUTS[c["layout"]]
    out = {}
    slots = s["slot"].cpu().numpy()
    keep = np.nonzero(slots >= 0)[0]
    for x, name, key, blk in ((s["k"], "K", "k", kb), (s["v"], "V", "v", vb)):
        scales = s[name][1]
        cap = scales.shape[2]
        to = torch.zeros(scales.shape, dtype=torch.float64, device="cuda")
        norm = torch.linalg.vector_norm(x.double().reshape(c["rows"], c["Hkv"], d // blk, blk), dim=-1)
        page, off = torch.from_numpy(slots[keep] // cap).cuda(), torch.from_numpy(slots[keep] % cap).cuda()
        to.permute(0, 2, 1, 3)[page, off] = norm[torch.from_numpy(keep).cuda()]
        out[key + "_codes"], out[key + "_scales"] = None, to
    return out


def exact(case, seed):
    if case["op"] not in ("beam", "append"):  # whole numbers and moved bytes: nothing is computed
        return None
    s = prepare(case, seed)
    return _exact_beam(s) if case["op"] == "beam" else _exact_append(s)
