"""GPU parity of the expanded form (q4g128_latent_expand, q4g128_latent_prefill)
against oracle/latent.py and oracle/attention.py's definition.

Bounds, from the arithmetic (u = 2^-24, one fp16 rounding = 2^-11 relative, or
2^-25 absolute below the normal range):
  * expand: weights are the oracle's, code * scale + min rounded once to fp16.  Sums
    of L products in fp32: |y - ref| <= 2^-11 |ref| + 2^-25 + (L + 8) u sum |w c|.
    Rotary columns are equal bit for bit.
  * attention over the keys and values as stored: scores err by ds = (K + 8) u scale
    max_j sum|q k|, weights by 2 ds plus 2^-11, a sum over n positions by n u, and a
    weight below 2^-14 of the largest by 2^-25 of it; with A = sum w |v|:
    |out - ref| <= 2^-11 |ref| + 2^-25 + (2^-11 + 2 ds + (n + 64) u) A + n 2^-25 max|v|.
"""
import numpy as np
import pytest

from oracle import latent as ref
from gpu_helpers import U32, device, note
from test_gpu_attention import H, TINY, i32
from test_gpu_latent import ROT, Rows

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


@pytest.fixture(scope="module")
def dev():
    return device()


def quantized(rng, rows, latent, dev):
    """int4 weights on the GPU, and their fp16 values in float64."""
    packed = rng.integers(0, 256, (rows, latent // 2), dtype=np.uint8)
    scales = (rng.uniform(0.8, 1.2, (rows, latent // 128)) / (4.61 * latent ** 0.5)).astype(np.float16)
    mins = (scales.astype(np.float64) * -7.4).astype(np.float16)
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(rows, latent).astype(np.float64)
    w = codes * np.repeat(scales.astype(np.float64), 128, 1) + np.repeat(mins.astype(np.float64), 128, 1)
    return [torch.from_numpy(a).to(dev) for a in (packed, scales, mins)], w.astype(np.float16).astype(np.float64)


def target(rng, lengths, heads, value, page, fill=7.0, absent=()):
    """Pages for keys and values, [k, v, table]."""
    used = [-(-max(0, n) // page) for n in lengths]
    pages = sum(used) + 2
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(1, max(used))), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    for s, i in absent:
        table[s, i] = (-1, pages, 2 ** 31 - 1)[(s + i) % 3]
    return (np.full((pages, heads, page, value + ROT), fill, np.float16), np.full((pages, heads, value, page), fill, np.float16),
            table)


def expand_case(dev, seed, lengths, heads, value, latent, page, to_page=None, firsts=None, absent=(), to_absent=(), **kw):
    rng = np.random.default_rng(seed)
    to_page = to_page or page
    pool = Rows(rng, lengths, latent, page, absent=absent)
    weights, w = quantized(rng, heads * 2 * value, latent, dev)
    k, v, table = target(rng, lengths, heads, value, to_page, absent=to_absent)
    got = [torch.from_numpy(a).to(dev) for a in (k, v, table)]
    q4.q4g128_latent_expand(*pool.on(dev), i32(lengths, dev), *weights, *got,
                            firsts=None if firsts is None else i32(firsts, dev), **kw)
    got_k, got_v = got[0].cpu().numpy(), got[1].cpu().numpy()
    want_k, want_v = k.copy(), v.copy()
    keys, values = ref.expanded(pool.rows, pool.table, lengths, w, heads)
    sums_k, sums_v = ref.expanded(np.abs(pool.rows), pool.table, lengths, np.abs(w), heads)
    most = kw.get("max_length", 10 ** 9)
    for s, n in enumerate(lengths):
        for j in range(0 if firsts is None else max(0, firsts[s]), min(n, most)):
            at, there = ref.slot(table, s, j, to_page, len(k)), ref.slot(pool.table, s, j, page, pool.pages)
            if at is None or there is None:
                continue
            p, o = at
            for got_x, x, mag in ((got_k[p, :, o], keys[s][j], sums_k[s][j]), (got_v[p, :, :, o], values[s][j], sums_v[s][j])):
                err = np.abs(got_x.astype(np.float64) - x)
                assert np.all(err <= H * np.abs(x) + TINY + (latent + 8) * U32 * mag), (s, j, err.max())
            assert np.array_equal(got_k[p, :, o, value:], np.broadcast_to(pool.rows[there[0], there[1], latent:], (heads, ROT)))
            want_k[p, :, o], want_v[p, :, :, o] = got_k[p, :, o], got_v[p, :, :, o]
    assert np.array_equal(got_k.view(np.uint16), want_k.view(np.uint16))  # nothing else is written
    assert np.array_equal(got_v.view(np.uint16), want_v.view(np.uint16))


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_expand_widths_and_pages(dev, latent, value, page):
    expand_case(dev, 1, [103, 30], 3, value, latent, page)


@pytest.mark.parametrize("page,to_page", [(16, 64), (64, 16), (32, 256), (256, 32)])
def test_expand_between_pages(dev, page, to_page):
    expand_case(dev, 2, [203, 7, 64], 2, 64, 128, page, to_page)


@pytest.mark.parametrize("length", [0, 1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 129])
def test_expand_lengths(dev, length):
    expand_case(dev, 3, [length], 2, 64, 128, 16)
    expand_case(dev, 4, [5, length, 0, 70], 1, 128, 128, 32)


@pytest.mark.parametrize("firsts", [[0, 0], [1, 63], [64, 70], [130, -5], [200, 99], [205, 66]])
def test_expand_from(dev, firsts):
    """A follow-up's positions only; what is there before them stays."""
    expand_case(dev, 5, [201, 100], 2, 64, 128, 16, firsts=firsts)


def test_expand_absent_pages_and_max_length(dev):
    expand_case(dev, 6, [150, 90], 2, 64, 128, 16, absent=[(0, 3), (1, 0)], to_absent=[(0, 5), (1, 4)])
    expand_case(dev, 7, [150, 90], 2, 64, 128, 16, max_length=100)


def test_expand_many_tiles_and_heads(dev):
    """Several tiles a workgroup, and more heads than CUs."""
    expand_case(dev, 8, [500 + 64 * i for i in range(3)], 90, 64, 128, 64)
    expand_case(dev, 9, [70, 3], 300, 64, 128, 64)
    expand_case(dev, 10, [1 + 13 * i % 40 for i in range(70)], 2, 64, 128, 16)


def attend(q, k, v, table, starts, lengths, scale):
    """(out, sum w |v|, largest sum |q k|), float64, of caches as stored."""
    tokens, heads, _ = q.shape
    value, page = v.shape[2], k.shape[2]
    out, mag, dots = np.zeros((tokens, heads, value)), np.zeros((tokens, heads, value)), np.zeros((tokens, heads))
    for s, n in enumerate(lengths):
        places = [ref.slot(table, s, j, page, len(k)) for j in range(n)]
        there = np.array([p is not None for p in places], dtype=bool)
        for t in range(int(starts[s]), int(starts[s + 1])):
            position = n - (int(starts[s + 1]) - t)
            at = [j for j in range(min(position + 1, n)) if there[j]]
            if not at:
                continue
            for h in range(heads):
                kk = np.array([k[places[j][0], h, places[j][1]] for j in at], dtype=np.float64)
                vv = np.array([v[places[j][0], h, :, places[j][1]] for j in at], dtype=np.float64)
                w = scale * (kk @ q[t, h].astype(np.float64))
                w = np.exp(w - w.max())
                w /= w.sum()
                out[t, h], mag[t, h] = w @ vv, w @ np.abs(vv)
                dots[t, h] = (np.abs(kk) @ np.abs(q[t, h].astype(np.float64))).max()
    return out, mag, dots


def prefill_case(dev, seed, new, lengths, heads, value, page, absent=(), junk=np.nan):
    rng = np.random.default_rng(seed)
    k, v, table = target(rng, lengths, heads, value, page, fill=junk, absent=absent)
    for s, n in enumerate(lengths):
        for j in range(n):
            at = ref.slot(table, s, j, page, len(k))
            if at:
                k[at[0], :, at[1]] = rng.standard_normal((heads, value + ROT))
                v[at[0], :, :, at[1]] = rng.standard_normal((heads, value))
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(starts[-1]), heads, value + ROT)).astype(np.float16)
    scale = (value + ROT) ** -0.5 * 1.5
    out = q4.q4g128_latent_prefill(torch.from_numpy(q).to(dev), *(torch.from_numpy(a).to(dev) for a in (k, v, table)),
                                   i32(starts, dev), i32(lengths, dev), scale)
    want, mag, dots = attend(q, k, v, table, starts, lengths, scale)
    n = max(1, max(lengths))
    ds = (value + ROT + 8) * U32 * scale * dots
    vmax = np.abs(v[np.isfinite(v)]).max()
    bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[..., None] * mag + n * TINY * vmax * (mag > 0)
    got = out.float().cpu().numpy()
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= bound), f"{int((err > bound).sum())} above the bound, worst {(err / bound).max():.3f}"


@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prefill_widths_and_pages(dev, value, page):
    prefill_case(dev, 11, [33, 7], [133, 40], 2, value, page)


@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("tokens", [1, 31, 64, 65, 128, 129, 200])
def test_prefill_lengths(dev, value, tokens):
    prefill_case(dev, 12, [tokens], [tokens], 1, value, 64)
    prefill_case(dev, 13, [tokens], [tokens + 130], 2, value, 16)


@pytest.mark.parametrize("value", [64, 128])
def test_prefill_forms(dev, value):
    """Many workgroups (128 rows each), few tokens on a long cache (split and joined), empty sequences, absent pages."""
    prefill_case(dev, 14, [40], [60], 260, value, 64)
    prefill_case(dev, 15, [3], [3000], 1, value, 64)
    prefill_case(dev, 16, [0, 5, 3, 9], [20, 0, 70, 4], 2, value, 16)
    prefill_case(dev, 17, [20, 9], [170, 100], 2, value, 16, absent=[(0, 0), (0, 6), (1, 5)])


@pytest.mark.parametrize("value", [64, 128])
def test_prompt_step_and_follow_up(dev, value):
    """Append, expand, attend; then a follow-up that expands its own positions only; all as the absorbed form has it."""
    rng = np.random.default_rng(18)
    heads, latent, page, lengths = 3, 128, 16, [50, 23]
    weights, w = quantized(rng, heads * 2 * value, latent, dev)
    w = w.reshape(heads, 2, value, latent)
    pages, cols = 12, 6
    table = i32([[3, 1, 5, 0, 7, 9], [2, 4, 6, 8, 10, 11]], dev)
    rows = torch.zeros((pages, page, latent + ROT), dtype=torch.float16, device=dev)
    k = torch.zeros((pages, heads, page, value + ROT), dtype=torch.float16, device=dev)
    v = torch.zeros((pages, heads, value, page), dtype=torch.float16, device=dev)
    freq = torch.from_numpy((1000.0 ** (-np.arange(32) / 32)).astype(np.float32)).to(dev)
    scale = (value + ROT) ** -0.5
    done = [0, 0]
    for new in ([50, 23], [9, 4], [1, 1]):
        total = sum(new)
        seq = np.repeat([0, 1], new)
        at = np.concatenate([np.arange(d, d + n) for d, n in zip(done, new)])
        kv = torch.from_numpy(rng.standard_normal((total, latent + ROT)).astype(np.float32)).to(dev)
        both = torch.from_numpy(rng.standard_normal((total, heads, value + ROT)).astype(np.float32)).to(dev)
        q = q4.q4g128_latent_append(kv, rows, table, i32(at, dev), freq, seq=i32(seq, dev), q_main=both[:, :, :value],
                                    q_rot=both[:, :, value:])
        starts, lengths = i32([0, new[0], total], dev), i32([d + n for d, n in zip(done, new)], dev)
        q4.q4g128_latent_expand(rows, table, lengths, *weights, k, v, table, firsts=i32(done, dev))
        out = q4.q4g128_latent_prefill(q, k, v, table, starts, lengths, scale).float().cpu().numpy()
        # absorbed: queries through the key weights, mixed rows through the value weights
        x = q.float().cpu().numpy().astype(np.float64)
        lat = np.concatenate([np.einsum("thv,hvl->thl", x[:, :, :value], w[:, 0]), x[:, :, value:]], -1).astype(np.float16)
        mixed = q4.q4g128_latent_attn(torch.from_numpy(lat).to(dev), rows, table, starts, lengths, scale)
        m = mixed.float().cpu().numpy().astype(np.float64)
        want = np.einsum("thl,hvl->thv", m, w[:, 1])
        # Against the exact result E of each form, with S = scale sum |q| |W_k| |c| over what a score is summed from and
        # A = sum_j w_j |W_v| |c_j|: rounded keys, or rounded absorbed queries, move scores by at most ds = (2^-11 +
        # (latent + 72) u) S, the normalised weights by a factor within e^(2 ds); the weights' own fp16 form, the rounded
        # values or mixed rows, the sums and the last rounding add 4 times 2^-11 of A, weights below fp16's normal
        # range n 2^-25 max |W_v| |c|.  The two forms differ by twice that at most.
        c = rows.float().cpu().numpy().astype(np.float64)
        tab = table.cpu().numpy()
        for s in range(2):
            n = done[s] + new[s]
            cs = np.stack([c[tab[s, p // page], p % page] for p in range(n)])
            far = np.abs(cs[:, :latent]) @ np.abs(w[:, 1]).transpose(0, 2, 1)                 # [heads][n][value]
            keys = np.concatenate([cs[:, :latent] @ w[:, 0].transpose(0, 2, 1),
                                   np.broadcast_to(cs[:, latent:], (heads, n, ROT))], -1)
            size = np.concatenate([np.abs(cs[:, :latent]) @ np.abs(w[:, 0]).transpose(0, 2, 1),
                                   np.broadcast_to(np.abs(cs[:, latent:]), (heads, n, ROT))], -1)
            for i in range(new[s]):
                r, sees = (0, new[0])[s] + i, done[s] + i + 1
                for h in range(heads):
                    dots = scale * keys[h, :sees] @ x[r, h]
                    e = np.exp(dots - dots.max())
                    ds = (H + (latent + 72) * U32) * scale * (size[h, :sees] @ np.abs(x[r, h])).max()
                    a = (e / e.sum()) @ far[h, :sees]
                    bound = 2 * ((np.expm1(2 * ds) + 4 * H) * a * (1 + 4 * H) + sees * TINY * far[h, :sees].max() + TINY)
                    assert np.all(np.abs(out[r, h] - want[r, h]) <= bound), (s, i, h)
        done = [d + n for d, n in zip(done, new)]


def test_prefill_repeats_and_replays(dev):
    rng = np.random.default_rng(19)
    heads, value, latent, page, length = 4, 128, 256, 64, 1500
    pool = Rows(rng, [length], latent, page)
    weights, _ = quantized(rng, heads * 2 * value, latent, dev)
    rows, table = pool.on(dev)
    k = torch.zeros((pool.pages, heads, page, value + ROT), dtype=torch.float16, device=dev)
    v = torch.zeros((pool.pages, heads, value, page), dtype=torch.float16, device=dev)
    q = torch.from_numpy(rng.standard_normal((9, heads, value + ROT)).astype(np.float16)).to(dev)
    n, starts = i32([length], dev), i32([0, 9], dev)

    def step():
        q4.q4g128_latent_expand(rows, table, n, *weights, k, v, table)
        return q4.q4g128_latent_prefill(q, k, v, table, starts, n, 0.07)

    first = step()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        again = step()
    other.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        held.fill_(7.0)
        k.zero_(), v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, held)
        assert torch.equal(first, step())
