"""Timing cases of the attention operators between the fused projection and o_proj.

Three operators over one paged key-value cache (K pages [page][kv head][token][dim],
V pages [page][kv head][dim][token], fp16):

* append: head norm + rotary position + cache write of new tokens, from the
  fused projection's fp32 rows;
* decode: attention of one new token per sequence;
* prefill: attention of prompt tokens, packed over sequences.

`run` computes them in elementary torch operations in float32, rounded once at
the end, or (own = True) through the library.  `exact` states the same results
in float64, one sequence at a time.
"""
import math

import torch

own = False

ROPE_BASE = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, tokens, seqs, past, heads, kv, dim, page, rot, interleaved=False, norm=False, factor=1.0, extra=0):
    return {"name": name, "op": "append", "tokens": tokens, "seqs": seqs, "past": past, "heads": heads, "kv": kv,
            "dim": dim, "page": page, "rot": rot, "interleaved": interleaved, "norm": norm, "factor": factor,
            "extra": extra}


def _decode(name, seqs, length, heads, kv, dim, page, ragged=True, softcap=0.0, window=0, slopes=False):
    return {"name": name, "op": "decode", "seqs": seqs, "length": length, "heads": heads, "kv": kv, "dim": dim,
            "page": page, "ragged": ragged, "softcap": softcap, "window": window, "slopes": slopes}


def _prefill(name, tokens, seqs, past, heads, kv, dim, page, softcap=0.0, window=0, slopes=False, prefix=0):
    return {"name": name, "op": "prefill", "tokens": tokens, "seqs": seqs, "past": past, "heads": heads, "kv": kv,
            "dim": dim, "page": page, "softcap": softcap, "window": window, "slopes": slopes, "prefix": prefix}


def listed():
    return [
        # one token of one request: the step after the fused 25,088-row GEMV (16 + 4 + 4 heads of 128, then gate and up)
        _append("append 1", 1, 1, 777, 16, 4, 128, 64, 128, extra=22016),
        # a batch of 16 requests, one token each, with head norms and interleaved pairs
        _append("append 16 seqs norm", 16, 16, 2000, 16, 4, 128, 64, 128, interleaved=True, norm=True, extra=22016),
        # three uneven prompts after a cached part, a quarter of each head rotated, small pages
        _append("append 333 partial", 333, 3, 45, 12, 3, 64, 16, 16, norm=True),
        # one long prompt with positions scaled for a long context
        _append("append 8192 scaled", 8192, 1, 0, 32, 8, 128, 64, 128, norm=True, factor=4.0),
        # one request at the position where the write-up measures its attention
        _decode("decode 1x2000", 1, 2000, 16, 4, 128, 64, ragged=False),
        # a small batch of requests of very different lengths
        _decode("decode 16 ragged 4096", 16, 4096, 16, 4, 128, 64),
        # small heads, every head with its own keys, capped scores inside a sliding window
        _decode("decode 7x3001 cap window", 7, 3001, 10, 10, 64, 16, softcap=30.0, window=1025),
        # a full server: the step whose cache traffic passes the weights'
        _decode("decode 64x16384", 64, 16384, 16, 4, 128, 64, ragged=False),
        # the write-up's 34-token prompt
        _prefill("prefill 34", 34, 1, 0, 16, 4, 128, 64),
        # five uneven prompts of small heads: bidirectional over a prefix, with a distance bias
        _prefill("prefill 1501 prefix bias", 1501, 5, 0, 9, 3, 64, 32, slopes=True, prefix=40),
        # a short follow-up on a long cached context
        _prefill("prefill 34 on 8000", 34, 1, 8000, 16, 4, 128, 64),
        # one long prompt
        _prefill("prefill 8192", 8192, 1, 0, 32, 8, 128, 64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        seqs = _log_int(rng, 1, 32)
        most = 8192 * 48 * 128 // ((heads + 2 * kv) * dim)
        tokens = max(seqs, _log_int(rng, 1, min(most, 12000)))
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        c = _append("", tokens, seqs, rng.randrange(0, 3000), heads, kv, dim, page, rot, rng.random() < 0.4,
                    rng.random() < 0.5, rng.choice([1.0, 1.0, 2.0, 8.0]), 4 * rng.randrange(0, 500))
    else:
        options = {"softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "slopes": rng.random() < 0.3}
        window = rng.choice([0, 0, _log_int(rng, 16, 4096)])
        if op == "decode":
            seqs = _log_int(rng, 1, 96)
            most = 64 * 16384 * 4 * 128 // (seqs * kv * dim)
            length = _log_int(rng, 1, min(most, 65536))
            c = _decode("", seqs, length, heads, kv, dim, page, rng.random() < 0.7, window=window, **options)
        else:
            seqs = _log_int(rng, 1, 6)
            tokens = max(seqs, _log_int(rng, 2, 6000))
            most = 8192 * 8192 * 32 * 128 // (2 * tokens * heads * dim)
            past = rng.choice([0, 0, _log_int(rng, 1, max(2, min(20000, most - tokens)))])
            prefix = _log_int(rng, 1, 200) if window == 0 and rng.random() < 0.3 else 0
            c = _prefill("", tokens, seqs, past, heads, kv, dim, page, window=window, prefix=prefix, **options)
    del c["name"]
    return c


def _share(i):
    """A fixed, uneven share in (0, 1] for sequence i; the first has 1."""
    return 1.0 if i == 0 else (i * 0.6180339887498949) % 1.0


def _new_tokens(case):
    """New tokens of each sequence (at least one each), summing to case["tokens"]."""
    seqs, tokens = case["seqs"], case["tokens"]
    shares = [_share(i) for i in range(seqs)]
    got = [1 + int((tokens - seqs) * s / sum(shares)) for s in shares]
    got[0] += tokens - sum(got)
    return got


def _lengths(case):
    """Cached positions of each sequence, the new tokens included."""
    if case["op"] == "decode":
        return [max(1, int(case["length"] * _share(i))) if case["ragged"] else case["length"]
                for i in range(case["seqs"])]
    return [n + int(case["past"] * _share(i)) for i, n in enumerate(_new_tokens(case))]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    lengths = _lengths(case)
    used = [-(-n // page) for n in lengths]
    cols, pages = max(used), sum(used) + 3

    def normal(*shape, dtype=torch.float16):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    row = torch.arange(cols, device=dev)
    first = torch.tensor([sum(used[:i]) for i in range(len(used))], device=dev)
    count = torch.tensor(used, device=dev)
    table = torch.where(row < count[:, None], order[(first[:, None] + row).clamp(max=pages - 1)], -1).to(torch.int32)
    s = dict(case)
    s["k_cache"] = normal(pages, kv, page, dim)
    s["v_cache"] = normal(pages, kv, dim, page)
    s["table"] = table.contiguous()
    s["lengths"] = torch.tensor(lengths, device=dev, dtype=torch.int32)
    s["max_length"] = max(lengths)
    if case["op"] != "decode":
        new = torch.tensor(_new_tokens(case), device=dev)
        starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=dev), new)
        at = torch.arange(case["tokens"], device=dev) - starts[seq] + s["lengths"][seq] - new[seq]
        s["q_starts"], s["seq"], s["positions"] = (t.to(torch.int32) for t in (starts, seq, at))
        s["max_new"] = max(_new_tokens(case))
    if case["op"] == "append":
        width = (heads + 2 * kv) * dim + case["extra"]
        s["qkv"] = normal(case["tokens"], width, dtype=torch.float32)
        half = case["rot"] // 2
        freq = ROPE_BASE ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        # long contexts: slow pairs are slowed by the factor, fast ones kept, with a ramp between
        ramp = (torch.arange(half, device=dev, dtype=torch.float64) / half).clamp(0, 1)
        s["inv_freq"] = (freq * (1 - ramp + ramp / case["factor"])).float()
        s["mscale"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        s["q_norm"] = normal(dim) * 0.1 + 1 if case["norm"] else None
        s["k_norm"] = normal(dim) * 0.1 + 1 if case["norm"] else None
    else:
        rows = case["seqs"] if case["op"] == "decode" else case["tokens"]
        s["q"] = normal(rows, heads, dim)
        s["scale"] = dim ** -0.5
        s["slope"] = torch.linspace(0.5, 0.01, heads, device=dev) if case["slopes"] else None
        if case["op"] == "prefill":
            s["prefix_len"] = (torch.full((case["seqs"],), case["prefix"], device=dev, dtype=torch.int32)
                               if case["prefix"] else None)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _library(s)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[s["op"]](s)


def _library(s):
    import int4_group_quantized_amd as q4

    cache = (s["k_cache"], s["v_cache"], s["table"])
    if s["op"] == "append":
        q = q4.q4g128_rope_append(s["qkv"], *cache, s["positions"], s["inv_freq"], s["heads"], seq=s["seq"],
                                  q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, interleaved=s["interleaved"],
                                  mscale=s["mscale"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "decode":
        return {"out": q4.q4g128_attn_decode(s["q"], *cache, s["lengths"], scale=s["scale"], softcap=s["softcap"],
                                             window=s["window"], slopes=s["slope"], max_length=s["max_length"])}
    return {"out": q4.q4g128_attn_prefill(s["q"], *cache, s["q_starts"], s["lengths"], scale=s["scale"],
                                          softcap=s["softcap"], window=s["window"], slopes=s["slope"],
                                          prefix=s["prefix_len"], max_length=s["max_length"])}


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][H][D] with its first `rot` dims turned by the angles of cos / sin [T][1][rot/2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _head_norm(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)


def _append_in(s, real):
    """(q, k, v) of the new tokens in the given floating type."""
    tokens, heads, kv, dim, rot = s["tokens"], s["heads"], s["kv"], s["dim"], s["rot"]
    x = s["qkv"][:, :(heads + 2 * kv) * dim].to(real).view(tokens, heads + 2 * kv, dim)
    angle = s["positions"].to(real)[:, None] * s["inv_freq"].to(real)
    cos, sin = (angle.cos() * s["mscale"])[:, None], (angle.sin() * s["mscale"])[:, None]
    q = _rotate(_head_norm(x[:, :heads], s["q_norm"]), cos, sin, rot, s["interleaved"])
    k = _rotate(_head_norm(x[:, heads:heads + kv], s["k_norm"]), cos, sin, rot, s["interleaved"])
    return q, k, x[:, heads + kv:]


def _plain_append(s):
    q, k, v = _append_in(s, torch.float32)
    at = s["positions"].long()
    page = s["table"][s["seq"].long(), at // s["page"]].long()
    s["k_cache"][page, :, at % s["page"]] = k.half()
    s["v_cache"][page, :, :, at % s["page"]] = v.half()
    return {"q": q.half(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(s):
    """K and V of every sequence as float32 [S][kv][positions][dim], padded."""
    table = s["table"].clamp(min=0).long()
    seqs, cols = table.shape
    k = s["k_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(seqs, s["kv"], cols * s["page"], s["dim"])
    v = s["v_cache"][table].float().permute(0, 2, 1, 4, 3).reshape(seqs, s["kv"], cols * s["page"], s["dim"])
    return k, v


def _attend(s, q, k, v, at, prefix):
    """q [S][Q][H][D] at positions at [S][Q] (-1: none) over k, v -> [S][Q][H][D], float32."""
    seqs, width = q.shape[:2]
    kv, group, dim = s["kv"], s["heads"] // s["kv"], s["dim"]
    rows = q.view(seqs, width, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * width, dim)
    score = (torch.matmul(rows, k.transpose(-1, -2).contiguous()) * s["scale"]).view(seqs, kv, group, width, -1)
    if s["softcap"]:
        score = torch.tanh(score / s["softcap"]) * s["softcap"]
    key = torch.arange(k.shape[2], device=q.device)
    here = at[:, :, None]
    if s["slope"] is not None:
        score = score + s["slope"].view(1, kv, group, 1, 1) * (key - here)[:, None, None].float()
    seen = key <= here
    if s["window"]:
        seen = seen & (key > here - s["window"])
    if prefix is not None:
        seen = seen | ((key < prefix[:, None, None]) & (here >= 0))
    seen = (seen & (key < s["lengths"][:, None, None]))[:, None, None]
    score = score.masked_fill(~seen, -math.inf)
    score = score - score.amax(-1, keepdim=True).clamp(min=-1e30)
    score = score.exp()
    total = score.sum(-1, keepdim=True)
    score = (score / total.clamp(min=1e-30)).view(seqs, kv, group * width, -1)
    out = torch.matmul(score, v)
    return out.view(seqs, kv, group, width, dim).permute(0, 3, 1, 2, 4).reshape(seqs, width, s["heads"], dim)


def _plain_decode(s):
    k, v = _gathered(s)
    at = (s["lengths"].long() - 1)[:, None]
    return {"out": _attend(s, s["q"].float()[:, None], k, v, at, None)[:, 0].half()}


def _plain_prefill(s):
    k, v = _gathered(s)
    seq, within = s["seq"].long(), torch.arange(s["tokens"], device=s["q"].device) - s["q_starts"].long()[s["seq"].long()]
    q = torch.zeros((s["seqs"], s["max_new"], s["heads"], s["dim"]), device=s["q"].device)
    at = torch.full((s["seqs"], s["max_new"]), -1, device=s["q"].device)
    q[seq, within] = s["q"].float()
    at[seq, within] = s["positions"].long()
    return {"out": _attend(s, q, k, v, at, s["prefix_len"])[seq, within].half()}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        return _exact_append(s)
    return {"out": _exact_attention(s)}


def _exact_append(s):
    heads, kv, dim, page, half = s["heads"], s["kv"], s["dim"], s["page"], s["rot"] // 2
    x = s["qkv"].double()[:, :(heads + 2 * kv) * dim].reshape(s["tokens"], heads + 2 * kv, dim)
    turned = x.clone()
    for first, last, weight in ((0, heads, s["q_norm"]), (heads, heads + kv, s["k_norm"])):
        if weight is not None:
            part = x[:, first:last]
            turned[:, first:last] = part / (part.pow(2).sum(-1, keepdim=True) / dim + EPS).sqrt() * weight.double()
    which = torch.arange(half, device=x.device)
    low, high = (2 * which, 2 * which + 1) if s["interleaved"] else (which, which + half)
    wheel = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=x.device).expand(s["tokens"], half).contiguous(),
                        s["positions"].double()[:, None] * s["inv_freq"].double())[:, None]
    z = torch.complex(turned[:, :heads + kv, low], turned[:, :heads + kv, high]) * wheel
    turned[:, :heads + kv, low], turned[:, :heads + kv, high] = z.real, z.imag
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    at, seq = s["positions"].long(), s["seq"].long()
    slot = s["table"].long()[seq, at.div(page, rounding_mode="floor")] * page + at.remainder(page)
    for h in range(kv):
        k_cache[slot // page, h, slot % page] = turned[:, heads + h]
        v_cache[slot // page, h, :, slot % page] = turned[:, heads + kv + h]
    return {"q": turned[:, :heads], "k_cache": k_cache, "v_cache": v_cache}


def _exact_attention(s):
    heads, kv, dim, page = s["heads"], s["kv"], s["dim"], s["page"]
    group, decode = heads // kv, s["op"] == "decode"
    q = s["q"].double()
    out = torch.zeros_like(q)
    lengths = s["lengths"].tolist()
    starts = list(range(s["seqs"] + 1)) if decode else s["q_starts"].tolist()
    for b, n in enumerate(lengths):
        a, e = starts[b], starts[b + 1]
        if n == 0 or a == e:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        key = torch.arange(n, device=q.device)
        at = torch.arange(n - (e - a), n, device=q.device)[:, None]
        seen = key <= at
        if s["window"]:
            seen &= at - key < s["window"]
        if not decode and s["prefix_len"] is not None:
            seen |= key < int(s["prefix_len"][b])
        for h in range(kv):
            k = s["k_cache"][ids, h].double().reshape(-1, dim)[:n]
            v = s["v_cache"][ids, h].double().transpose(1, 2).reshape(-1, dim)[:n]
            for i in range(h * group, (h + 1) * group):
                w = q[a:e, i] @ k.t() * s["scale"]
                if s["softcap"]:
                    w = s["softcap"] * torch.tanh(w / s["softcap"])
                if s["slope"] is not None:
                    w = w + s["slope"][i].double() * (key - at)
                out[a:e, i] = torch.softmax(w.masked_fill(~seen, -math.inf), -1) @ v
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    if case["op"] == "append":
        n, wide = case["tokens"], (heads + 2 * kv) * dim
        # read fp32 rows, positions and sequence numbers; write q, k and v in fp16
        return {"bytes": n * wide * 6 + n * 8, "flops": n * wide * 6}
    lengths = _lengths(case)
    new = [1] * len(lengths) if case["op"] == "decode" else _new_tokens(case)
    window, prefix = case["window"], case.get("prefix", 0)
    keys = pairs = 0
    for n, m in zip(lengths, new):
        start = n - m  # position of the first query
        keys += min(n, m + window - 1) if window else n
        if window:
            full = max(0, min(m, window - start))  # queries that see all earlier positions
            pairs += full * start + full * (full + 1) // 2 + (m - full) * window
        else:
            pairs += m * start + m * (m + 1) // 2
            inside = max(0, min(prefix, n) - start)  # queries inside the prefix see the rest of it too
            pairs += inside * (inside - 1) // 2
    return {"bytes": 2 * keys * kv * dim * 2 + 2 * sum(new) * heads * dim * 2, "flops": 4 * pairs * heads * dim}
