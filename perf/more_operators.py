"""Timing cases of drafted tokens and of latent attention over paged caches.

Five operators, all over caches of pages that a table maps to sequences:

* tree: attention of a tree of drafted tokens over a key-value cache (K pages
  [page][kv head][token][dim], V pages [page][kv head][dim][token], fp16);
* keep: the accepted tokens of each tree moved together in that cache;
* append: new tokens' latent rows (norm, rotary part) into a latent cache (pages
  [page][token][latent + 64], fp16), and their queries;
* latent: attention over the latent rows themselves (absorbed form), of single
  tokens, chains and trees;
* prompt: keys and values of every head expanded from the latent rows by int4
  weights, and the prompt's attention over them (expanded form).

`run` computes them in elementary torch operations in float32, rounded once at
the end, or (own = True) through the library.  `exact` states the same results
in float64, one sequence at a time.
"""
import math
import random

import torch

own = False

ROPE_BASE = 10000.0
EPS = 1e-6
ROT = 64      # rotary columns of a latent row
GROUP = 128   # columns of an int4 group


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _tree(name, seqs, draft, length, heads, kv, dim, page, ragged=True, softcap=0.0, window=0, slopes=False):
    return {"name": name, "op": "tree", "seqs": seqs, "draft": draft, "length": length, "heads": heads, "kv": kv,
            "dim": dim, "page": page, "ragged": ragged, "softcap": softcap, "window": window, "slopes": slopes}


def _keep(name, seqs, draft, taken, length, kv, dim, page):
    return {"name": name, "op": "keep", "seqs": seqs, "draft": draft, "taken": taken, "length": length, "kv": kv,
            "dim": dim, "page": page, "ragged": True}


def _append(name, tokens, seqs, past, heads, main, latent, page, interleaved=True, norm=True, factor=1.0):
    return {"name": name, "op": "append", "tokens": tokens, "seqs": seqs, "past": past, "heads": heads, "main": main,
            "latent": latent, "page": page, "interleaved": interleaved, "norm": norm, "factor": factor}


def _latent(name, seqs, draft, length, heads, latent, page, tree=False, ragged=True):
    return {"name": name, "op": "latent", "seqs": seqs, "draft": draft, "length": length, "heads": heads,
            "latent": latent, "page": page, "tree": tree, "ragged": ragged}


def _prompt(name, tokens, seqs, past, heads, value, latent, page):
    return {"name": name, "op": "prompt", "tokens": tokens, "seqs": seqs, "past": past, "heads": heads,
            "value": value, "latent": latent, "page": page}


def listed():
    return [
        # one request whose next tokens were drafted as a small tree
        _tree("tree 1x8 on 700", 1, 8, 700, 16, 4, 128, 64),
        # a batch of requests of very different lengths, uneven trees, inside a sliding window with capped scores and a bias
        _tree("tree 9x13 ragged window cap bias", 9, 13, 3001, 12, 3, 64, 16, softcap=30.0, window=1025, slopes=True),
        # a server's batch with the widest trees on long contexts
        _tree("tree 16x64 on 16384", 16, 64, 16384, 32, 8, 128, 64, ragged=False),
        # the accepted path of one request's tree
        _keep("keep 1x5", 1, 16, 5, 700, 4, 128, 64),
        # the accepted paths of a full server's trees
        _keep("keep 256x12", 256, 48, 12, 600, 8, 128, 64),
        # one token of one request, its queries already multiplied into the latent space
        _append("append 1", 1, 1, 777, 16, 512, 512, 64),
        # uneven prompts, queries for the expanded form, positions scaled for a long context
        _append("append 4001", 4001, 3, 45, 128, 128, 512, 64, factor=4.0),
        # one request of a model of few heads
        _latent("latent 1x2000", 1, 1, 2000, 16, 512, 64),
        # trees of drafted tokens of a batch of uneven requests, small latent rows and pages
        _latent("latent 7x11 tree ragged", 7, 11, 5003, 12, 256, 16, tree=True),
        # a full server of a model of many heads
        _latent("latent 64x8192", 64, 1, 8192, 128, 512, 64, ragged=False),
        # a short follow-up of two requests on a cached context
        _prompt("prompt 77 on 900", 77, 2, 900, 16, 128, 512, 64),
        # one long prompt of a model of many heads
        _prompt("prompt 4096", 4096, 1, 0, 64, 128, 512, 64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "keep", "append", "latent", "latent", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    latent = rng.choice([512, 512, 256, 128])
    if op in ("tree", "keep"):
        dim = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 3, 4, 8])
        draft = _log_int(rng, 1, 64)
        if op == "keep":
            c = _keep("", _log_int(rng, 1, 300), draft, rng.randrange(0, draft // 2 + 2), _log_int(rng, draft, 600), kv,
                      dim, page)
        else:
            heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
            seqs = _log_int(rng, 1, 48)
            most = 16 * 64 * 16384 * 32 * 128 // (seqs * draft * heads * dim)
            fits = 64 * 16384 * 4 * 128 // (seqs * kv * dim)
            length = draft + _log_int(rng, 1, min(most, fits, 65536))
            c = _tree("", seqs, draft, length, heads, kv, dim, page, rng.random() < 0.7,
                      rng.choice([0.0, 0.0, 20.0, 50.0]), rng.choice([0, 0, _log_int(rng, 16, 4096)]),
                      rng.random() < 0.3)
    elif op == "append":
        heads = rng.choice([1, 7, 16, 32, 64, 128])
        main = rng.choice([64, 128, latent, latent])
        seqs = _log_int(rng, 1, 32)
        most = 4001 * 128 * 192 // (heads * (main + ROT))
        c = _append("", max(seqs, _log_int(rng, 1, min(most, 9000))), seqs, rng.randrange(0, 3000), heads, main, latent,
                    page, rng.random() < 0.5, rng.random() < 0.7, rng.choice([1.0, 1.0, 2.0, 8.0]))
    elif op == "latent":
        heads = rng.choice([1, 5, 12, 16, 20, 32, 64, 128])
        seqs, draft = _log_int(rng, 1, 64), rng.choice([1, 1, 1, _log_int(rng, 2, 64)])
        most = 64 * 8192 * 128 * 512 // (seqs * draft * heads * latent)
        fits = 64 * 8192 * 576 // (seqs * (latent + ROT))
        c = _latent("", seqs, draft, draft + _log_int(rng, 1, min(most, fits, 65536)), heads, latent, page,
                    rng.random() < 0.6, rng.random() < 0.7)
    else:
        heads = rng.choice([1, 3, 8, 16, 32, 64])
        seqs = _log_int(rng, 1, 5)
        tokens = max(seqs, _log_int(rng, 2, 4000))
        most = 4096 * 4096 * 64 // (2 * tokens * heads)
        past = rng.choice([0, 0, _log_int(rng, 1, max(1, min(9000, most - tokens)))])
        c = _prompt("", tokens, seqs, past, heads, rng.choice([128, 128, 64]), latent, page)
    del c["name"]
    return c


def _share(i):
    """A fixed, uneven share in (0, 1] for sequence i; the first has 1."""
    return 1.0 if i == 0 else (i * 0.6180339887498949) % 1.0


def _new_tokens(case):
    """New tokens of each sequence (at least one each)."""
    seqs = case["seqs"]
    if "draft" in case:
        return [max(1, int(case["draft"] * _share(i))) if case["ragged"] else case["draft"] for i in range(seqs)]
    shares = [_share(i) for i in range(seqs)]
    got = [1 + int((case["tokens"] - seqs) * s / sum(shares)) for s in shares]
    got[0] += case["tokens"] - sum(got)
    return got


def _lengths(case):
    """Cached positions of each sequence, the new tokens included."""
    new = _new_tokens(case)
    if "draft" in case:
        return [max(n, int(case["length"] * _share(3 * i))) if case["ragged"] else case["length"]
                for i, n in enumerate(new)]
    return [n + int(case["past"] * _share(i)) for i, n in enumerate(new)]


def _taken(case):
    """Accepted tokens of each tree: the first of the draft, and some from behind the path's own length."""
    got = []
    for i, n in enumerate(_new_tokens(case)):
        count = min(case["taken"], n)
        tail = max(0, min(count - 1, n - count))
        got.append(list(range(count - tail)) + [n - tail + j for j in range(tail)])
    return got


def _trees(case, seed):
    """Masks of the drafted tokens of all sequences: bit k of a token's mask is set if it sees token k."""
    rng = random.Random(seed)
    masks = []
    for n in _new_tokens(case):
        mine = []
        for i in range(n):
            parent = rng.randrange(max(-1, i - 6), i) if case.get("tree", True) else i - 1
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
        masks += [m - (1 << 64) if m >> 63 else m for m in mine]
    return masks


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    page = case["page"]
    lengths, new = _lengths(case), _new_tokens(case)
    used = [max(1, -(-n // page)) for n in lengths]
    cols, pages = max(used), sum(used) + 3

    def normal(*shape, dtype=torch.float16):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, device=dev, dtype=dtype)

    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    row = torch.arange(cols, device=dev)
    first = ints([sum(used[:i]) for i in range(len(used))], torch.int64)
    count = ints(used, torch.int64)
    table = torch.where(row < count[:, None], order[(first[:, None] + row).clamp(max=pages - 1)], -1)
    s = dict(case)
    s["table"] = table.to(torch.int32).contiguous()
    s["lengths"], s["max_length"] = ints(lengths), max(lengths)
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    s["q_starts"], s["rows"], s["max_new"] = ints(starts), starts[-1], max(new)
    seq = [i for i, n in enumerate(new) for _ in range(n)]
    at = [lengths[i] - n + j for i, n in enumerate(new) for j in range(n)]
    s["seq"], s["slots"] = ints(seq), ints(at)
    if case["op"] in ("tree", "keep"):
        s["k_cache"] = normal(pages, case["kv"], page, case["dim"])
        s["v_cache"] = normal(pages, case["kv"], case["dim"], page)
    else:
        s["cache"] = normal(pages, page, case["latent"] + ROT)
    if case["op"] == "tree":
        s["q"] = normal(s["rows"], case["heads"], case["dim"])
        s["scale"] = case["dim"] ** -0.5
        s["slope"] = torch.linspace(0.5, 0.01, case["heads"], device=dev) if case["slopes"] else None
        s["masks"] = ints(_trees(case, seed), torch.int64)
    elif case["op"] == "keep":
        taken = _taken(case)
        s["starts"] = ints([n - m for n, m in zip(lengths, new)])
        s["keep_starts"] = ints([sum(len(t) for t in taken[:i]) for i in range(len(taken) + 1)])
        s["keep"] = ints([i for t in taken for i in t])
    elif case["op"] == "append":
        s["kv_rows"] = normal(s["rows"], case["latent"] + ROT, dtype=torch.float32)
        # queries as their products leave them: for the expanded form both parts of a head lie in one row
        if case["main"] == case["latent"]:
            s["q_main"] = normal(s["rows"], case["heads"], case["main"], dtype=torch.float32)
            s["q_rot"] = normal(s["rows"], case["heads"], 128 + ROT, dtype=torch.float32)[:, :, 128:]
        else:
            both = normal(s["rows"], case["heads"], case["main"] + ROT, dtype=torch.float32)
            s["q_main"], s["q_rot"] = both[:, :, :case["main"]], both[:, :, case["main"]:]
        half = ROT // 2
        freq = ROPE_BASE ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        # long contexts: slow pairs are slowed by the factor, fast ones kept, with a ramp between
        ramp = torch.arange(half, device=dev, dtype=torch.float64) / half
        s["inv_freq"] = (freq * (1 - ramp + ramp / case["factor"])).float()
        s["mscale"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        s["norm_weight"] = normal(case["latent"]) * 0.1 + 1 if case["norm"] else None
    elif case["op"] == "latent":
        s["q"] = normal(s["rows"], case["heads"], case["latent"] + ROT)
        s["scale"] = (128 + ROT) ** -0.5
        s["masks"] = ints(_trees(case, seed), torch.int64) if case["tree"] else None
    else:
        heads, value, latent = case["heads"], case["value"], case["latent"]
        s["q"] = normal(s["rows"], heads, value + ROT)
        s["scale"] = (value + ROT) ** -0.5
        # weights whose products with unit rows are about one, in int4 groups
        wide = heads * 2 * value
        s["packed"] = torch.randint(0, 256, (wide, latent // 2), generator=gen, device=dev, dtype=torch.uint8)
        spread = torch.rand((wide, latent // GROUP), generator=gen, device=dev) * 0.4 + 0.8
        step = spread / (4.61 * latent ** 0.5)
        s["scales"], s["mins"] = step.half(), (step * -7.5).half()
        # the pages that the expanded keys and values go to, mapped as the latent rows are
        s["k_cache"] = torch.zeros((pages, heads, page, value + ROT), device=dev, dtype=torch.float16)
        s["v_cache"] = torch.zeros((pages, heads, value, page), device=dev, dtype=torch.float16)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _library(s)
    return {"tree": _plain_tree, "keep": _plain_keep, "append": _plain_append, "latent": _plain_latent,
            "prompt": _plain_prompt}[s["op"]](s)


def _library(s):
    import int4_group_quantized_amd as q4

    table = s["table"]
    if s["op"] == "tree":
        return {"out": q4.q4g128_attn_tree(s["q"], s["k_cache"], s["v_cache"], table, s["q_starts"], s["lengths"],
                                           s["masks"], scale=s["scale"], softcap=s["softcap"], window=s["window"],
                                           slopes=s["slope"], max_new=s["max_new"], max_length=s["max_length"])}
    if s["op"] == "keep":
        q4.q4g128_cache_keep(s["k_cache"], s["v_cache"], table, s["starts"], s["keep_starts"], s["keep"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "append":
        q = q4.q4g128_latent_append(s["kv_rows"], s["cache"], table, s["slots"], s["inv_freq"], seq=s["seq"],
                                    norm=s["norm_weight"], eps=EPS, interleaved=s["interleaved"], mscale=s["mscale"],
                                    q_main=s["q_main"], q_rot=s["q_rot"])
        return {"q": q, "cache": s["cache"]}
    if s["op"] == "latent":
        return {"out": q4.q4g128_latent_attn(s["q"], s["cache"], table, s["q_starts"], s["lengths"], s["scale"],
                                             masks=s["masks"], max_new=s["max_new"], max_length=s["max_length"])}
    q4.q4g128_latent_expand(s["cache"], table, s["lengths"], s["packed"], s["scales"], s["mins"], s["k_cache"],
                            s["v_cache"], table, max_length=s["max_length"])
    out = q4.q4g128_latent_prefill(s["q"], s["k_cache"], s["v_cache"], table, s["q_starts"], s["lengths"], s["scale"],
                                   max_length=s["max_length"])
    return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _padded(s, rows):
    """rows [T][...] as [S][max_new][...], zeros where a sequence has fewer."""
    within = torch.arange(s["rows"], device=rows.device) - s["q_starts"].long()[s["seq"].long()]
    out = rows.new_zeros((s["seqs"], s["max_new"]) + tuple(rows.shape[1:]))
    out[s["seq"].long(), within] = rows
    return out, within


def _seen(s, positions):
    """[S][max_new][positions]: the cached positions that each new token may see, and the tokens' and positions' places.

    A drafted token's place is the number of positions in front of the draft plus that of drafted tokens it sees,
    itself among them, less one; elsewhere place and position are the same.
    """
    dev = s["table"].device
    key = torch.arange(positions, device=dev)
    lengths = s["lengths"].long()[:, None]
    new = (s["q_starts"][1:] - s["q_starts"][:-1]).long()[:, None]
    base = lengths - new
    token = torch.arange(s["max_new"], device=dev)
    if s.get("masks") is None:
        here = base + token
        seen = key <= here[:, :, None]
        place = key.expand(s["seqs"], positions)
    else:
        masks, _ = _padded(s, s["masks"])
        bit = torch.arange(64, device=dev)
        bits = ((masks[:, :, None] >> bit) & 1) * (bit < new[:, :, None])
        here = base + bits.sum(-1) - 1
        k = key - base
        drafted = (k >= 0) & (key < lengths)
        k = k.clamp(0, 63)
        seen = (key < base)[:, None] | (drafted[:, None] & (bits.gather(2, k[:, None].expand(-1, s["max_new"], -1)) > 0))
        place = torch.where(drafted, here.gather(1, k.clamp(max=s["max_new"] - 1)), key)
    return seen & (key < lengths)[:, None] & (token < new)[:, :, None], here, place


def _softmax(score):
    score = (score - score.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    return score / score.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_tree(s):
    table = s["table"].clamp(min=0).long()
    seqs, cols = table.shape
    kv, dim, group = s["kv"], s["dim"], s["heads"] // s["kv"]
    positions = cols * s["page"]
    k = s["k_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(seqs, kv, positions, dim)
    v = s["v_cache"][table].float().permute(0, 2, 1, 4, 3).reshape(seqs, kv, positions, dim)
    q, within = _padded(s, s["q"].float())
    new = s["max_new"]
    rows = q.view(seqs, new, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * new, dim)
    score = (torch.matmul(rows, k.transpose(-1, -2).contiguous()) * s["scale"]).view(seqs, kv, group, new, positions)
    if s["softcap"]:
        score = torch.tanh(score / s["softcap"]) * s["softcap"]
    seen, here, place = _seen(s, positions)
    apart = place[:, None] - here[:, :, None]
    if s["slope"] is not None:
        score = score + s["slope"].view(1, kv, group, 1, 1) * apart[:, None, None].float()
    if s["window"]:
        seen = seen & (apart > -s["window"])
    weights = _softmax(score.masked_fill(~seen[:, None, None], -math.inf))
    out = torch.matmul(weights.view(seqs, kv, group * new, positions), v)
    out = out.view(seqs, kv, group, new, dim).permute(0, 3, 1, 2, 4).reshape(seqs, new, s["heads"], dim)
    return {"out": out[s["seq"].long(), within].half()}


def _plain_keep(s):
    page = s["page"]
    count = (s["keep_starts"][1:] - s["keep_starts"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device=count.device), count, output_size=s["keep"].shape[0])
    base = s["starts"].long()[seq]
    source = base + s["keep"].long()
    target = base + torch.arange(s["keep"].shape[0], device=count.device) - s["keep_starts"].long()[seq]
    from_page, to_page = s["table"][seq, source // page].long(), s["table"][seq, target // page].long()
    s["k_cache"][to_page, :, target % page] = s["k_cache"][from_page, :, source % page]
    s["v_cache"][to_page, :, :, target % page] = s["v_cache"][from_page, :, :, source % page]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _turned(s, x, angle):
    """x [T][...][ROT] with its pairs turned by angle [T][ROT / 2] and scaled, in float32 from 64-bit angles."""
    shape = (s["rows"],) + (1,) * (x.dim() - 2) + (ROT // 2,)
    cos, sin = (angle.cos() * s["mscale"]).float().view(shape), (angle.sin() * s["mscale"]).float().view(shape)
    if s["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x[..., :ROT // 2], x[..., ROT // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_append(s):
    latent, page = s["latent"], s["page"]
    angle = s["slots"].double()[:, None] * s["inv_freq"].double()
    rows = s["kv_rows"][:, :latent]
    if s["norm_weight"] is not None:
        rows = rows * torch.rsqrt(rows.square().mean(-1, keepdim=True) + EPS) * s["norm_weight"].float()
    rows = torch.cat([rows, _turned(s, s["kv_rows"][:, latent:], angle)], dim=-1)
    at = s["slots"].long()
    s["cache"][s["table"][s["seq"].long(), at // page].long(), at % page] = rows.half()
    return {"q": torch.cat([s["q_main"], _turned(s, s["q_rot"], angle)], dim=-1).half(), "cache": s["cache"]}


def _plain_latent(s):
    table = s["table"].clamp(min=0).long()
    seqs, cols = table.shape
    positions, heads, new = cols * s["page"], s["heads"], s["max_new"]
    rows = s["cache"][table].float().reshape(seqs, positions, s["latent"] + ROT)
    q, within = _padded(s, s["q"].float())
    score = torch.matmul(q.reshape(seqs, new * heads, -1), rows.transpose(-1, -2).contiguous()) * s["scale"]
    seen, _, _ = _seen(s, positions)
    weights = _softmax(score.view(seqs, new, heads, positions).masked_fill(~seen[:, :, None], -math.inf))
    out = torch.matmul(weights.view(seqs, new * heads, positions), rows[:, :, :s["latent"]].contiguous())
    return {"out": out.view(seqs, new, heads, s["latent"])[s["seq"].long(), within].half()}


def _weights(s, real):
    """The int4 weights as they enter the product: rounded once to fp16, [heads][2 value][latent]."""
    low, high = s["packed"] & 15, s["packed"] >> 4
    codes = torch.stack([low, high], dim=-1).flatten(1).view(-1, s["latent"] // GROUP, GROUP)
    w = codes.float() * s["scales"].float()[:, :, None] + s["mins"].float()[:, :, None]
    return w.half().to(real).view(s["heads"], 2 * s["value"], s["latent"])


def _plain_prompt(s):
    table = s["table"].clamp(min=0).long()
    seqs, cols = table.shape
    positions, heads, value, latent = cols * s["page"], s["heads"], s["value"], s["latent"]
    rows = s["cache"][table].float().reshape(seqs, positions, latent + ROT)
    both = torch.matmul(rows[:, :, :latent].reshape(seqs * positions, latent),
                        _weights(s, torch.float32).view(-1, latent).t().contiguous())
    both = both.view(seqs, positions, heads, 2 * value).permute(0, 2, 1, 3)
    k = torch.cat([both[..., :value], rows[:, None, :, latent:].expand(-1, heads, -1, -1)], dim=-1)
    at = torch.arange(positions, device=rows.device).expand(seqs, -1)
    there = at < s["lengths"][:, None]
    page, off = table.repeat_interleave(s["page"], 1)[there], at[there] % s["page"]
    s["k_cache"][page, :, off] = k.transpose(1, 2)[there].half()
    s["v_cache"][page, :, :, off] = both[..., value:].transpose(1, 2)[there].half()
    q, within = _padded(s, s["q"].float())
    score = torch.matmul(q.permute(0, 2, 1, 3).contiguous(), k.transpose(-1, -2).contiguous()) * s["scale"]
    seen, _, _ = _seen(s, positions)
    weights = _softmax(score.masked_fill_(~seen[:, None], -math.inf))
    out = torch.matmul(weights, both[..., value:].contiguous()).permute(0, 2, 1, 3)
    return {"out": out[s["seq"].long(), within].half(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "keep": _exact_keep, "append": _exact_append, "latent": _exact_latent,
            "prompt": _exact_prompt}[s["op"]](s)


def _sequences(s):
    """(sequence, first row, last row, length, page numbers, [rows][length] what each row sees, places of both)."""
    lengths, starts, words = s["lengths"].tolist(), s["q_starts"].tolist(), s.get("masks")
    for b, n in enumerate(lengths):
        a, e = starts[b], starts[b + 1]
        if a == e:
            continue
        place = list(range(n))
        see = torch.ones((e - a, n), dtype=torch.bool).tril_(n - (e - a))
        if words is not None:
            draft = [w & ((1 << 64) - 1) & ((1 << (e - a)) - 1) for w in words[a:e].tolist()]
            for i, w in enumerate(draft):
                place[n - (e - a) + i] = n - (e - a) + bin(w).count("1") - 1
                see[i, n - (e - a):] = torch.tensor([w >> j & 1 for j in range(e - a)], dtype=torch.bool)
        place = torch.tensor(place, device=s["table"].device)
        yield b, a, e, n, s["table"][b, :-(-n // s["page"])].long(), see.to(place.device), place


def _attend(q, k, v, bias, see):
    """softmax(q k^T + bias) v in 64 bits over what each row sees; rows that see nothing are zeros."""
    score = (q @ k.t() + bias).masked_fill(~see, -math.inf)
    return torch.nan_to_num(torch.softmax(score, -1), nan=0.0) @ v


def _exact_tree(s):
    kv, dim, group = s["kv"], s["dim"], s["heads"] // s["kv"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    for _, a, e, n, ids, see, place in _sequences(s):
        apart = place[None, :] - place[n - (e - a):, None]
        if s["window"]:
            see = see & (apart > -s["window"])
        for h in range(kv):
            k = s["k_cache"][ids, h].double().reshape(-1, dim)[:n]
            v = s["v_cache"][ids, h].double().transpose(1, 2).reshape(-1, dim)[:n]
            for i in range(h * group, (h + 1) * group):
                score = q[a:e, i] @ k.t() * s["scale"]
                if s["softcap"]:
                    score = s["softcap"] * torch.tanh(score / s["softcap"])
                if s["slope"] is not None:
                    score = score + s["slope"][i].double() * apart
                score = score.masked_fill(~see, -math.inf)
                out[a:e, i] = torch.nan_to_num(torch.softmax(score, -1), nan=0.0) @ v
    return {"out": out}


def _exact_keep(s):
    page = s["page"]
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    starts, keep, table, base = s["keep_starts"].tolist(), s["keep"].tolist(), s["table"].tolist(), s["starts"].tolist()
    for b in range(s["seqs"]):
        for i, j in enumerate(keep[starts[b]:starts[b + 1]]):
            there, here = base[b] + j, base[b] + i
            k[table[b][here // page], :, here % page] = s["k_cache"][table[b][there // page], :, there % page]
            v[table[b][here // page], :, :, here % page] = s["v_cache"][table[b][there // page], :, :, there % page]
    return {"k_cache": k.double(), "v_cache": v.double()}


def _exact_append(s):
    latent, page, half = s["latent"], s["page"], ROT // 2
    which = torch.arange(half, device=s["cache"].device)
    low, high = (2 * which, 2 * which + 1) if s["interleaved"] else (which, which + half)
    wheel = torch.polar(torch.full((s["rows"], half), s["mscale"], dtype=torch.float64, device=which.device),
                        s["slots"].double()[:, None] * s["inv_freq"].double())

    def turned(x, wheel):
        z = torch.complex(x[..., low], x[..., high]) * wheel
        y = torch.empty_like(x)
        y[..., low], y[..., high] = z.real, z.imag
        return y

    rows = s["kv_rows"].double()
    body = rows[:, :latent]
    if s["norm_weight"] is not None:
        body = body / (body.pow(2).sum(-1, keepdim=True) / latent + EPS).sqrt() * s["norm_weight"].double()
    rows = torch.cat([body, turned(rows[:, latent:].contiguous(), wheel)], -1)
    cache = s["cache"].double()
    at = s["slots"].long()
    slot = s["table"].long()[s["seq"].long(), at.div(page, rounding_mode="floor")] * page + at.remainder(page)
    cache.view(-1, latent + ROT)[slot] = rows
    q = torch.cat([s["q_main"].double(), turned(s["q_rot"].double().contiguous(), wheel[:, None])], -1)
    return {"q": q, "cache": cache}


def _exact_latent(s):
    heads, latent = s["heads"], s["latent"]
    q = s["q"].double()
    out = torch.zeros((s["rows"], heads, latent), dtype=torch.float64, device=q.device)
    for _, a, e, n, ids, see, _ in _sequences(s):
        rows = s["cache"][ids].double().reshape(-1, latent + ROT)[:n]
        mine = (q[a:e] * s["scale"]).reshape(-1, latent + ROT)
        seen = see[:, None].expand(-1, heads, -1).reshape(-1, n)
        out[a:e] = _attend(mine, rows, rows[:, :latent], 0.0, seen).view(e - a, heads, latent)
    return {"out": out}


def _exact_prompt(s):
    heads, value, latent = s["heads"], s["value"], s["latent"]
    weights = _weights(s, torch.float64)
    q = s["q"].double()
    out = torch.zeros((s["rows"], heads, value), dtype=torch.float64, device=q.device)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    for _, a, e, n, ids, see, _ in _sequences(s):
        rows = s["cache"][ids].double().reshape(-1, latent + ROT)[:n]
        slot = torch.arange(n, device=ids.device)
        page, off = ids[slot // s["page"]], slot % s["page"]
        for h in range(heads):
            k = torch.cat([rows[:, :latent] @ weights[h, :value].t(), rows[:, latent:]], -1)
            v = rows[:, :latent] @ weights[h, value:].t()
            k_cache[page, h, off], v_cache[page, h, :, off] = k, v
            out[a:e, h] = _attend(q[a:e, h] * s["scale"], k, v, 0.0, see)
    return {"out": out, "k_cache": k_cache, "v_cache": v_cache}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _pairs(case, lengths, new):
    """Keys read and query-key pairs, a chain's or a tree's drafted tokens taken as half of them seen."""
    window = case.get("window", 0)
    keys = pairs = 0
    for n, m in zip(lengths, new):
        past = n - m
        keys += min(n, window + m) if window else n
        pairs += m * (min(past, window) if window else past) + m * (m + 1) // 2
    return keys, pairs


def work(case):
    lengths, new = _lengths(case), _new_tokens(case)
    rows, op = sum(new), case["op"]
    if op == "keep":
        moved = sum(sum(1 for i, j in enumerate(t) if i != j) for t in _taken(case))
        return {"bytes": 2 * 2 * 2 * moved * case["kv"] * case["dim"], "flops": 0}
    if op == "append":
        wide = case["latent"] + ROT + case["heads"] * (case["main"] + ROT)
        return {"bytes": rows * (wide * 6 + 8), "flops": rows * (4 * case["latent"] + 6 * ROT * (1 + case["heads"]))}
    keys, pairs = _pairs(case, lengths, new)
    heads = case["heads"]
    if op == "tree":
        dim = case["dim"]
        return {"bytes": 2 * keys * case["kv"] * dim * 2 + 2 * rows * heads * dim * 2, "flops": 4 * pairs * heads * dim}
    latent = case["latent"]
    if op == "latent":
        return {"bytes": 2 * keys * (latent + ROT) + 2 * rows * heads * (2 * latent + ROT),
                "flops": 2 * pairs * heads * (2 * latent + ROT)}
    value = case["value"]
    wide = 2 * value * heads
    # latent rows and int4 weights read, keys and values written and read once, queries read and outputs written
    return {"bytes": 2 * keys * (latent + ROT) + wide * latent // 2 + 4 * wide * latent // GROUP
            + 2 * 2 * keys * heads * (2 * value + ROT) + 2 * rows * heads * (2 * value + ROT),
            "flops": 2 * keys * latent * wide + 2 * pairs * heads * (2 * value + ROT)}
