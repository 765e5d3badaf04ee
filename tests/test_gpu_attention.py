"""GPU parity of the paged cache calls (q4g128_rope_append, q4g128_attn_decode,
q4g128_attn_prefill) against oracle/attention.py, through the C ABI.

Bounds, from the arithmetic (u = 2^-24, one fp16 rounding = 2^-11 relative, or
2^-25 absolute below the normal range):
  * append: |y - ref| <= 2^-11 |ref| + 2^-25 + (dim + 64) u mscale (|lo| + |hi|):
    the norm's sum has dim terms, sines and cosines and the turn a few roundings.
  * attention, per output: scores err by ds = (dim + 8) u scale max_j sum|q k|
    (+ 2^-21 softcap, + 2^-22 largest |slope * distance|), and a weight's
    relative error is 2 ds plus 2^-11 for its fp16 form; a sum over n positions
    adds n u; a weight below 2^-14 of the largest errs by 2^-25 of it.  With
    A = sum w |v|:
    |out - ref| <= 2^-11 |ref| + 2^-25 + (2^-11 + 2 ds + (n + 64) u) A + n 2^-25 max|v|.
"""
import numpy as np
import pytest

from oracle import attention as ref
from gpu_helpers import U32, device, note

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")

H = 2.0 ** -11
TINY = 2.0 ** -25


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


@pytest.fixture(scope="module")
def dev():
    return device()


class Pool:
    """A cache of random pages, its table a random choice of them; junk fills what no sequence holds."""

    def __init__(self, rng, lengths, kv, page, dim, cols=None, junk=np.nan, absent=()):
        used = [-(-max(0, n) // page) for n in lengths]
        self.page, self.kv, self.dim = page, kv, dim
        self.cols = cols or max(1, max(used))
        self.pages = sum(used) + 2
        order = rng.permutation(self.pages)
        self.k = rng.standard_normal((self.pages, kv, page, dim)).astype(np.float16)
        self.v = rng.standard_normal((self.pages, kv, dim, page)).astype(np.float16)
        held = np.zeros((self.pages, page), dtype=bool)
        self.table = np.full((len(lengths), self.cols), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(lengths):
            for i in range(used[s]):
                self.table[s, i] = order[at]
                held[order[at], :min(page, n - i * page)] = True
                at += 1
        if junk is not None:
            p, o = np.nonzero(~held)
            self.k[p, :, o] = junk
            self.v[p, :, :, o] = junk
        for s, i in absent:
            self.table[s, i] = (-1, self.pages, 2 ** 31 - 1)[(s + i) % 3]

    def on(self, dev):
        return tuple(torch.from_numpy(a).to(dev) for a in (self.k, self.v, self.table))


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def check_attention(got, q, pool, starts, lengths, scale, what, softcap=0.0, window=0, slopes=None, prefix=None):
    want, mag, dots = ref.attention(q, pool.k, pool.v, pool.table, starts, lengths, scale, softcap, window, slopes,
                                    prefix)
    n = max(1, max(lengths))
    ds = (q.shape[2] + 8) * U32 * scale * dots + 2.0 ** -21 * softcap
    if slopes is not None:
        ds = ds + 2.0 ** -22 * n * np.abs(slopes)[None]
    vmax = np.abs(pool.v[np.isfinite(pool.v)]).max() if np.isfinite(pool.v).any() else 0.0
    bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[..., None] * mag + n * TINY * vmax * (mag > 0)
    g = got.float().cpu().numpy().astype(np.float64)
    assert g.shape == want.shape
    assert np.all(np.isfinite(g)), f"{what}: {int((~np.isfinite(g)).sum())} outputs are not finite"
    err = np.abs(g - want)
    assert np.all(err <= bound), f"{what}: {int((err > bound).sum())} above the bound, worst {(err / bound).max():.3f}"


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def check_append(dev, rng, placed, heads, kv, dim, page, rot, interleaved=False, norm=False, mscale=1.0, extra=0,
                 seqs=None, absent=(), base=10000.0, cols=None):
    """placed: [(sequence, position)] of the tokens."""
    tokens = len(placed)
    seqs = seqs or max(1, max(s for s, _ in placed) + 1)
    lengths = [1 + max([p for s, p in placed if s == b] or [0]) for b in range(seqs)]
    pool = Pool(rng, [min(n, (cols or 10 ** 9) * page) for n in lengths], kv, page, dim, junk=7.0, cols=cols, absent=absent)
    width = (heads + 2 * kv) * dim + extra
    qkv = rng.standard_normal((tokens, width)).astype(np.float32) * 3
    freq = (base ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    wq = rng.uniform(0.5, 1.5, dim).astype(np.float16) if norm else None
    wk = rng.uniform(0.5, 1.5, dim).astype(np.float16) if norm else None
    k, v, table = pool.on(dev)
    q = q4.q4g128_rope_append(
        torch.from_numpy(qkv).to(dev), k, v, table, i32([p for _, p in placed], dev),
        torch.from_numpy(freq).to(dev) if rot else None, heads, seq=i32([s for s, _ in placed], dev),
        q_norm=None if wq is None else torch.from_numpy(wq).to(dev),
        k_norm=None if wk is None else torch.from_numpy(wk).to(dev), eps=1e-5, interleaved=interleaved, mscale=mscale)
    got_q, got_k, got_v = (t.cpu().numpy() for t in (q, k, v))
    want_k, want_v = pool.k.copy(), pool.v.copy()

    def bound(want, x):
        pair = np.abs(x)
        for i in range(rot // 2):
            lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            pair[lo] = pair[hi] = (np.abs(x[lo]) + np.abs(x[hi])) * abs(mscale)
        return H * np.abs(want) + TINY + (dim + 64) * U32 * pair

    for t, (s, p) in enumerate(placed):
        row = qkv[t].reshape(-1)[:(heads + 2 * kv) * dim].reshape(-1, dim).astype(np.float64)
        at = ref.slot(pool.table, s, p, page, pool.pages)
        for h in range(heads + kv):
            w = wq if h < heads else wk
            want = ref.rotated(row[h], p, freq, rot, interleaved, mscale, w, 1e-5)
            plain = ref.rotated(row[h], 0, freq, 0, False, 1.0, w, 1e-5)
            if h < heads:
                err = np.abs(got_q[t, h].astype(np.float64) - want)
                assert np.all(err <= bound(want, plain)), (t, h, err.max())
            elif at:
                err = np.abs(got_k[at[0], h - heads, at[1]].astype(np.float64) - want)
                assert np.all(err <= bound(want, plain)), (t, h, err.max())
                want_k[at[0], h - heads, at[1]] = got_k[at[0], h - heads, at[1]]
        if at:
            want_v[at[0], :, :, at[1]] = row[heads + kv:].astype(np.float16)
    # values are rounded only, and nothing else of the pools changes
    assert np.array_equal(got_v.view(np.uint16), want_v.view(np.uint16))
    assert np.array_equal(got_k.view(np.uint16), want_k.view(np.uint16))


def run_of(seq, start, n):
    return [(seq, start + i) for i in range(n)]


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_dims(dev, dim, interleaved, norm):
    rng = np.random.default_rng(dim + interleaved + 2 * norm)
    placed = run_of(0, 5, 11) + run_of(2, 60, 3) + run_of(1, 0, 1)
    check_append(dev, rng, placed, 6, 2, dim, 16, dim // 2, interleaved, norm, extra=12)


@pytest.mark.parametrize("rot", [0, 4, 20, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_part_of_the_head(dev, rot, interleaved):
    check_append(dev, np.random.default_rng(rot), run_of(0, 3, 9), 3, 1, 64, 32, rot, interleaved, True, mscale=1.25)


@pytest.mark.parametrize("tokens,start", [(1, 0), (1, 255), (63, 0), (64, 0), (65, 0), (130, 8), (130, 3), (200, 64)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_prompt_lengths(dev, tokens, start, page):
    check_append(dev, np.random.default_rng(tokens + start), run_of(0, start, tokens), 2, 1, 64, page, 64)


def test_append_many_heads(dev):
    check_append(dev, np.random.default_rng(8), run_of(0, 40, 70), 35, 5, 128, 64, 128, norm=True)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("tokens", [210, 420, 830])
def test_append_several_heads_of_a_token_together(dev, dim, tokens):
    """Enough tokens that 2, 4 or 8 heads share a token's sines, 45 heads that do not divide by them."""
    rng = np.random.default_rng(dim + tokens)
    check_append(dev, rng, run_of(0, 5, tokens), 40, 5, dim, 64, 16, interleaved=tokens == 420, norm=True)


def test_append_one_token_of_each_sequence(dev):
    rng = np.random.default_rng(3)
    check_append(dev, rng, [(s, int(p)) for s, p in enumerate(rng.integers(0, 700, 16))], 16, 4, 128, 64, 128,
                 extra=256)


def test_append_far_positions(dev):
    """Angles at position 2^20 and beyond come out as exactly as near ones."""
    cols = (1 << 21) // 256
    rng = np.random.default_rng(4)
    placed = [(0, (1 << 20) + 1), (0, (1 << 21) - 1)]
    pool_k = torch.zeros((1, 1, 256, 64), dtype=torch.float16, device=dev)
    pool_v = torch.zeros((1, 1, 64, 256), dtype=torch.float16, device=dev)
    table = torch.full((1, cols), -1, dtype=torch.int32, device=dev)
    qkv = rng.standard_normal((2, 3 * 64)).astype(np.float32)
    freq = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    q = q4.q4g128_rope_append(torch.from_numpy(qkv).to(dev), pool_k, pool_v, table, i32([p for _, p in placed], dev),
                              torch.from_numpy(freq).to(dev), 1, seq=i32([0, 0], dev)).cpu().numpy()
    for t, (_, p) in enumerate(placed):
        want = ref.rotated(qkv[t, :64], p, freq, 64)
        pair = np.tile(np.abs(qkv[t, :32]) + np.abs(qkv[t, 32:64]), 2)
        assert np.all(np.abs(q[t, 0] - want) <= H * np.abs(want) + TINY + 128 * U32 * pair)
    assert not pool_k.any() and not pool_v.any()  # both pages are absent


def test_append_tokens_without_a_place(dev):
    """Sequences and positions outside the table and absent pages write nothing; q is still computed."""
    rng = np.random.default_rng(5)
    placed = [(0, 0), (5, 3), (-1, 3), (0, -4), (1, 40), (1, 17), (0, 64), (0, 31)]
    check_append(dev, rng, placed, 2, 2, 64, 16, 64, seqs=2, cols=4, absent=[(1, 1)])


def test_append_without_sequence_numbers(dev):
    rng = np.random.default_rng(6)
    pool = Pool(rng, [40, 40, 40], 1, 16, 64, junk=1.0)
    qkv = torch.from_numpy(rng.standard_normal((3, 256)).astype(np.float32)).to(dev)
    k, v, table = pool.on(dev)
    k2, v2 = k.clone(), v.clone()
    pos = i32([3, 39, 20], dev)
    freq = torch.ones(16, device=dev)
    a = q4.q4g128_rope_append(qkv, k, v, table, pos, freq, 2)
    b = q4.q4g128_rope_append(qkv, k2, v2, table, pos, freq, 2, seq=i32([0, 1, 2], dev))
    assert torch.equal(a, b) and torch.equal(k, k2) and torch.equal(v, v2)


def test_append_into_a_slice_of_a_larger_pool(dev):
    """One allocation [pages][layers][2][...]: one layer's pools are strided, the other layers keep their bits."""
    rng = np.random.default_rng(7)
    pages, layers, kv, page, dim = 6, 3, 2, 16, 64
    big = torch.from_numpy(rng.standard_normal((pages, layers, 2, kv * page * dim)).astype(np.float16)).to(dev)
    before = big.clone()
    k = big[:, 1, 0].view(pages, kv, page, dim)
    v = big[:, 1, 1].view(pages, kv, dim, page)
    table = i32([[4, 0, 2]], dev)
    tokens = 41
    qkv = torch.from_numpy(rng.standard_normal((tokens, 4 * dim)).astype(np.float32)).to(dev)
    wide = torch.zeros((tokens, 6 * dim), device=dev)
    wide[:, :4 * dim] = qkv
    q_dense_k, q_dense_v = torch.zeros_like(k).contiguous(), torch.zeros_like(v).contiguous()
    args = dict(seq=torch.zeros(tokens, dtype=torch.int32, device=dev))
    pos = torch.arange(3, 3 + tokens, dtype=torch.int32, device=dev)
    freq = torch.linspace(1.0, 0.01, 32, device=dev)
    with pytest.raises(ValueError):
        q4.q4g128_rope_append(qkv, q_dense_k, q_dense_v, table, pos, freq, 2, **args)  # too few columns
    qkv = torch.from_numpy(rng.standard_normal((tokens, 6 * dim)).astype(np.float32)).to(dev)
    a = q4.q4g128_rope_append(qkv, k, v, table, pos, freq, 2, **args)
    b = q4.q4g128_rope_append(qkv, q_dense_k, q_dense_v, table, pos, freq, 2, **args)
    assert torch.equal(a, b)
    for p in range(tokens):
        page_no, off = int(table[0, (3 + p) // page]), (3 + p) % page
        assert torch.equal(k[page_no, :, off], q_dense_k[page_no, :, off])
        assert torch.equal(v[page_no, :, :, off], q_dense_v[page_no, :, :, off])
        k[page_no, :, off] = before[:, 1, 0].view(pages, kv, page, dim)[page_no, :, off]
        v[page_no, :, :, off] = before[:, 1, 1].view(pages, kv, dim, page)[page_no, :, :, off]
    assert torch.equal(big, before)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

def decode_case(dev, seed, lengths, heads, kv, dim, page, cols=None, absent=(), softcap=0.0, window=0, slopes=False,
                max_length=None, junk=np.nan):
    rng = np.random.default_rng(seed)
    pool = Pool(rng, lengths, kv, page, dim, cols=cols, absent=absent, junk=junk)
    q = rng.standard_normal((len(lengths), heads, dim)).astype(np.float16)
    slope = np.linspace(0.4, 0.01, heads).astype(np.float32) if slopes else None
    scale = dim ** -0.5 * 1.5
    out = q4.q4g128_attn_decode(torch.from_numpy(q).to(dev), *pool.on(dev), i32(lengths, dev), scale=scale,
                                softcap=softcap, window=window,
                                slopes=None if slope is None else torch.from_numpy(slope).to(dev),
                                max_length=max_length)
    check_attention(out, q, pool, range(len(lengths) + 1), lengths, scale, f"decode {lengths}", softcap, window, slope)
    return out


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_dims_and_pages(dev, dim, page):
    decode_case(dev, dim + page, [1, 300, 77, 0, 64], 6, 2, dim, page)


@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 5), (3, 1), (10, 2), (16, 1), (17, 1), (40, 1), (64, 1), (66, 2)])
def test_decode_groups(dev, heads, kv):
    decode_case(dev, heads, [70, 3], heads, kv, 64, 16)


@pytest.mark.parametrize("length", [0, 1, 2, 7, 8, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_decode_lengths(dev, length):
    decode_case(dev, length, [length], 4, 1, 128, 64)


def test_decode_long_and_split(dev):
    decode_case(dev, 1, [9001, 13, 5000, 0, 1], 2, 1, 64, 64)


def test_decode_joined_in_groups(dev):
    """Two sequences of more than 32 parts among short ones, two row blocks each; repeats find the counters at zero."""
    first = decode_case(dev, 40, [20000, 3, 0, 9000], 17, 1, 64, 64)
    assert torch.equal(first, decode_case(dev, 40, [20000, 3, 0, 9000], 17, 1, 64, 64))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 2900])
def test_decode_long_uneven(dev, dim, window):
    """More than eight tiles for each workgroup of a kv head: parts are evened out."""
    decode_case(dev, 14 + dim, [3000, 100, 0, 2500, 1, 4000, 64, 65], 32, 32, dim, 64, window=window)
    decode_case(dev, 15 + dim, [700] * 7 + [8000], 33, 33, dim, 16, window=window)


def test_decode_many_sequences(dev):
    rng = np.random.default_rng(2)
    decode_case(dev, 2, [int(n) for n in rng.integers(0, 40, 150)] + [3000], 2, 1, 64, 16)


@pytest.mark.parametrize("window", [1, 5, 64, 65, 130, 257, 4096])
def test_decode_window(dev, window):
    decode_case(dev, window, [1, 64, 129, 700, 0], 4, 2, 64, 16, window=window)


@pytest.mark.parametrize("softcap,slopes", [(5.0, False), (0.0, True), (20.0, True)])
def test_decode_capped_and_biased(dev, softcap, slopes):
    decode_case(dev, 9, [400, 33], 6, 2, 128, 32, softcap=softcap, slopes=slopes, window=300)


def test_decode_absent_pages(dev):
    decode_case(dev, 11, [400, 64, 33, 16], 4, 1, 64, 16, absent=[(0, 0), (0, 3), (0, 4), (0, 24), (1, 1), (3, 0)])


def test_decode_max_length_bounds_the_lengths(dev):
    """A length above max_length counts as max_length, one below zero as zero."""
    rng = np.random.default_rng(12)
    pool = Pool(rng, [200, 100, 50], 1, 16, 64)
    q = torch.from_numpy(rng.standard_normal((3, 4, 64)).astype(np.float16)).to(dev)
    c = pool.on(dev)
    a = q4.q4g128_attn_decode(q, *c, i32([200, 100, -3], dev), max_length=120)
    b = q4.q4g128_attn_decode(q, *c, i32([120, 100, 0], dev))
    check_attention(a, q.cpu().numpy(), pool, range(4), [120, 100, 0], 64 ** -0.5, "max_length")
    check_attention(b, q.cpu().numpy(), pool, range(4), [120, 100, 0], 64 ** -0.5, "lengths")


@pytest.mark.parametrize("junk", [np.nan, np.inf, -np.inf, -65504.0])
def test_decode_masked_positions_stay_out(dev, junk):
    """Positions before the window hold junk too."""
    rng = np.random.default_rng(13)
    lengths, window = [150, 90], 40
    pool = Pool(rng, lengths, 1, 16, 64, junk=junk)
    for s, n in enumerate(lengths):
        for j in range(n - window):
            p = pool.table[s, j // 16]
            pool.k[p, :, j % 16] = junk
            pool.v[p, :, :, j % 16] = junk
    q = rng.standard_normal((2, 4, 64)).astype(np.float16)
    out = q4.q4g128_attn_decode(torch.from_numpy(q).to(dev), *pool.on(dev), i32(lengths, dev), scale=0.2, window=window)
    check_attention(out, q, pool, range(3), lengths, 0.2, f"junk {junk}", window=window)


def test_decode_shapes_share_a_workspace(dev):
    """Calls of different shapes on one workspace, with prompt calls between them, leave its counters at zero."""
    rng = np.random.default_rng(15)
    cases = [([3000, 5], 4, 1, 64), ([700] * 9, 12, 3, 128), ([9000], 40, 1, 64), ([1, 0], 2, 2, 256)]
    need = max(max(q4.q4g128_attn_decode_workspace(len(n), h, d),
                   q4.q4g128_attn_prefill_workspace(len(n), len(n), h, kv, d, max(n))) for n, h, kv, d in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    ws[q4.ATTN_COUNTER_BYTES:] = 0xFF
    for lengths, heads, kv, dim in cases + cases[::-1]:
        pool = Pool(rng, lengths, kv, 64, dim)
        c = pool.on(dev)
        q = rng.standard_normal((len(lengths), heads, dim)).astype(np.float16)
        qd, n, starts = torch.from_numpy(q).to(dev), i32(lengths, dev), i32(range(len(lengths) + 1), dev)
        for out in (q4.q4g128_attn_decode(qd, *c, n, scale=0.1, max_length=max(lengths), workspace=ws),
                    q4.q4g128_attn_prefill(qd, *c, starts, n, scale=0.1, max_length=max(lengths), workspace=ws)):
            check_attention(out, q, pool, range(len(lengths) + 1), lengths, 0.1, f"shared workspace {lengths}")
        assert not ws[:q4.ATTN_COUNTER_BYTES].any()


def test_decode_repeats_bit_for_bit_and_on_another_stream(dev):
    rng = np.random.default_rng(14)
    lengths = [5000, 17, 1200]
    pool = Pool(rng, lengths, 2, 64, 128)
    c = pool.on(dev)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128)).astype(np.float16)).to(dev)
    n = i32(lengths, dev)
    first = q4.q4g128_attn_decode(q, *c, n)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(first, q4.q4g128_attn_decode(q, *c, n))
        out = q4.q4g128_attn_decode(q, *c, n, stream=other)
        other.synchronize()
        assert torch.equal(first, out)


# ---------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------

def prefill_case(dev, seed, new, lengths, heads, kv, dim, page, absent=(), softcap=0.0, window=0, slopes=False,
                 prefix=None, junk=np.nan):
    rng = np.random.default_rng(seed)
    pool = Pool(rng, lengths, kv, page, dim, absent=absent, junk=junk)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(starts[-1]), heads, dim)).astype(np.float16)
    slope = np.linspace(0.4, 0.01, heads).astype(np.float32) if slopes else None
    scale = dim ** -0.5 * 1.5
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev),
                                 scale=scale, softcap=softcap, window=window,
                                 slopes=None if slope is None else torch.from_numpy(slope).to(dev),
                                 prefix=None if prefix is None else i32(prefix, dev))
    check_attention(out, q, pool, starts, lengths, scale, f"prefill {new} of {lengths}", softcap, window, slope, prefix)
    return out


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prefill_dims_and_pages(dev, dim, page):
    prefill_case(dev, dim + page, [40, 1, 90], [40, 130, 200], 4, 2, dim, page)


@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 5), (3, 1), (10, 2), (7, 1), (17, 1), (64, 1)])
def test_prefill_groups(dev, heads, kv):
    prefill_case(dev, heads, [37, 5], [60, 5], heads, kv, 64, 16)


@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_prefill_lengths(dev, tokens):
    prefill_case(dev, tokens, [tokens], [tokens], 4, 1, 128, 64)
    prefill_case(dev, tokens, [tokens], [tokens + 37], 4, 4, 64, 32)


def test_prefill_empty_sequences(dev):
    """Sequences without new tokens, without positions, and with fewer positions than new tokens."""
    prefill_case(dev, 20, [0, 5, 0, 30, 3, 0], [50, 5, 0, 12, 0, 7], 4, 2, 64, 16)


@pytest.mark.parametrize("window", [1, 16, 63, 64, 65, 200, 4096])
def test_prefill_window(dev, window):
    prefill_case(dev, window, [150, 33], [260, 33], 4, 2, 64, 16, window=window)


@pytest.mark.parametrize("prefix", [[0, 0], [1, 300], [70, 5], [-4, 64]])
def test_prefill_prefix(dev, prefix):
    prefill_case(dev, 21, [130, 40], [150, 100], 6, 2, 64, 32, prefix=prefix, slopes=True)


@pytest.mark.parametrize("softcap,slopes", [(5.0, False), (0.0, True), (20.0, True)])
def test_prefill_capped_and_biased(dev, softcap, slopes):
    prefill_case(dev, 22, [100, 70], [100, 90], 4, 2, 128, 64, softcap=softcap, slopes=slopes, window=80)


def test_prefill_few_tokens_on_a_long_cache(dev):
    prefill_case(dev, 23, [9], [6000], 2, 1, 64, 64)
    prefill_case(dev, 24, [3, 20, 1], [2500, 40, 1300], 4, 2, 128, 16, softcap=10.0, slopes=True)


@pytest.mark.parametrize("window", [1, 100, 1000, 3000, 5990])
def test_prefill_few_tokens_on_a_long_cache_with_a_window(dev, window):
    prefill_case(dev, 30 + window, [9, 40], [6000, 2000], 4, 2, 64, 64, window=window)
    prefill_case(dev, 31 + window, [5], [6000], 8, 1, 256, 32, window=window)


def test_prefill_absent_pages(dev):
    prefill_case(dev, 25, [60, 20], [200, 20], 4, 1, 64, 16, absent=[(0, 0), (0, 3), (0, 12), (1, 0), (1, 1)])
    prefill_case(dev, 26, [5], [3000], 4, 1, 64, 64, absent=[(0, 0), (0, 20), (0, 46)])


@pytest.mark.parametrize("junk", [np.nan, np.inf, -np.inf])
def test_prefill_masked_positions_stay_out(dev, junk):
    """A later token's keys and values hold junk: earlier tokens' results are those without it, and a row
    that sees an infinite value has it."""
    rng = np.random.default_rng(27)
    n, bad = 100, (70, 99)
    pool = Pool(rng, [n], 1, 16, 64)
    q = rng.standard_normal((n, 4, 64)).astype(np.float16)
    clean_k, clean_v = pool.k.copy(), pool.v.copy()
    for j in bad:
        pool.v[pool.table[0, j // 16], :, 5:9, j % 16] = junk
    c = pool.on(dev)
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *c, i32([0, n], dev), i32([n], dev), scale=0.1)
    o = out.float().cpu().numpy()
    seen = o[70:, :, 5:9]
    assert np.all(np.isnan(seen) if np.isnan(junk) else seen == junk)
    pool.k, pool.v = clean_k, clean_v
    o[70:, :, 5:9] = 0
    want, mag, _ = ref.attention(q, pool.k, pool.v, pool.table, [0, n], [n], 0.1)
    want[70:, :, 5:9] = 0
    assert np.all(np.isfinite(o))
    assert np.all(np.abs(o - want) <= H * np.abs(want) + TINY + (2 * H) * mag + n * TINY * 8)


# Sequences without tokens count as possible workgroups: with 40 of them and 8 kv heads a call takes the form
# for many (128 rows each), without them the one for few (64 rows).
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("options", [{}, dict(softcap=20.0, slopes=True, window=150), dict(prefix=[30, 0, 420])])
def test_prefill_many_workgroups(dev, dim, page, options):
    empty = [0] * 40
    options = dict(options)
    if "prefix" in options:
        options["prefix"] = options["prefix"] + empty
    prefill_case(dev, dim + page + 1, [40, 1, 90] + empty, [40, 130, 500] + empty, 16, 8, dim, page,
                 absent=[(2, 1)], **options)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("empty", [0, 10])
def test_prefill_split_forms(dev, dim, empty):
    prefill_case(dev, dim + empty, [9, 7] + [0] * empty, [2500, 300] + [0] * empty, 16, 8, dim, 64)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("empty", [0, 40])
@pytest.mark.parametrize("rising", [True, False])
def test_prefill_scores_that_grow_or_shrink(dev, dim, empty, rising):
    """Maxima that move by far more than the weights' range, up to the last position or from the first."""
    rng = np.random.default_rng(dim + empty)
    n, kv = 460, 8 if empty else 1
    lengths = [n] + [0] * empty
    pool = Pool(rng, lengths, kv, 64, dim)
    for j in range(n):
        grown = 1 + (j if rising else n - 1 - j) / 12
        pool.k[pool.table[0, j // 64], :, j % 64] *= np.float16(grown)
    starts = [0] + [70] * (empty + 1)
    q = rng.standard_normal((70, 2 * kv, dim)).astype(np.float16)
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev),
                                 scale=0.3)
    check_attention(out, q, pool, starts, lengths, 0.3, "moving maxima")


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("empty", [0, 40])
@pytest.mark.parametrize("bad", [(70, 99), (3, 40), (63, 64)])
def test_prefill_masked_infinities_in_every_form(dev, dim, empty, bad):
    rng = np.random.default_rng(dim + empty + bad[0])
    n, kv = 100, 8 if empty else 1
    lengths = [n] + [0] * empty
    pool = Pool(rng, lengths, kv, 32, dim)
    starts = [0] + [n] * (empty + 1)
    q = rng.standard_normal((n, 2 * kv, dim)).astype(np.float16)
    clean_k, clean_v = pool.k.copy(), pool.v.copy()
    dims = [5, dim // 2 - 1, dim - 1]
    for j in bad:
        pool.v[pool.table[0, j // 32], :, dims, j % 32] = np.inf
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev),
                                 scale=0.1)
    o = out.float().cpu().numpy()
    assert np.all(o[bad[0]:, :, dims] == np.inf)
    pool.k, pool.v = clean_k, clean_v
    o[bad[0]:, :, dims] = 0
    want, mag, _ = ref.attention(q, pool.k, pool.v, pool.table, starts, lengths, 0.1)
    want[bad[0]:, :, dims] = 0
    assert np.all(np.isfinite(o))
    assert np.all(np.abs(o - want) <= H * np.abs(want) + TINY + (2 * H) * mag + n * TINY * 8)


def test_prefill_agrees_with_decode(dev):
    """The last token of a prompt is the same question to both calls."""
    rng = np.random.default_rng(28)
    pool = Pool(rng, [333, 90], 2, 32, 128)
    c = pool.on(dev)
    q = torch.from_numpy(rng.standard_normal((60, 8, 128)).astype(np.float16)).to(dev)
    n = i32([333, 90], dev)
    p = q4.q4g128_attn_prefill(q, *c, i32([0, 40, 60], dev), n)
    d = q4.q4g128_attn_decode(q[[39, 59]].contiguous(), *c, n)
    torch.cuda.synchronize()
    assert (p[[39, 59]].float() - d.float()).abs().max() < 4 * H * 4


def test_prefill_repeats_bit_for_bit(dev):
    rng = np.random.default_rng(29)
    pool = Pool(rng, [4000], 2, 64, 128)
    c = pool.on(dev)
    q = torch.from_numpy(rng.standard_normal((34, 8, 128)).astype(np.float16)).to(dev)
    first = q4.q4g128_attn_prefill(q, *c, i32([0, 34], dev), i32([4000], dev))
    for _ in range(3):
        assert torch.equal(first, q4.q4g128_attn_prefill(q, *c, i32([0, 34], dev), i32([4000], dev)))


# ---------------------------------------------------------------------------
# graphs
# ---------------------------------------------------------------------------

def test_step_in_a_graph(dev):
    """Append and both attention calls captured once, replayed on growing lengths: equal to the eager calls."""
    rng = np.random.default_rng(30)
    heads, kv, dim, page, b = 8, 2, 128, 64, 3
    pool = Pool(rng, [900, 300, 200], kv, page, dim, junk=0.0)
    k, v, table = pool.on(dev)
    qkv = torch.from_numpy(rng.standard_normal((b, (heads + 2 * kv) * dim)).astype(np.float32)).to(dev)
    freq = torch.from_numpy((10000.0 ** (-np.arange(64) / 64)).astype(np.float32)).to(dev)
    lengths = i32([700, 100, 5], dev)
    positions = lengths - 1
    starts = i32([0, 1, 2, 3], dev)
    q = torch.empty((b, heads, dim), dtype=torch.float16, device=dev)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    ws = torch.zeros(q4.q4g128_attn_decode_workspace(b, heads, dim), dtype=torch.uint8, device=dev)
    ws2 = torch.empty(q4.q4g128_attn_prefill_workspace(b, 3, heads, kv, dim, 900), dtype=torch.uint8, device=dev)

    def step():
        q4.q4g128_rope_append(qkv, k, v, table, positions, freq, heads, q=q)
        q4.q4g128_attn_decode(q, k, v, table, lengths, max_length=900, out=out, workspace=ws)
        q4.q4g128_attn_prefill(q, k, v, table, starts, lengths, max_length=900, out=out2, workspace=ws2)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        lengths += 7
        positions.copy_(lengths - 1)
        qkv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, out, out2, k, v)]
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (q, out, out2, k, v)):
            assert torch.equal(x, y), i


# ---------------------------------------------------------------------------
# the binding and the calls together
# ---------------------------------------------------------------------------

def test_pools_beyond_4_gb(dev):
    """Page offsets of more than 2^32 bytes, in both directions of both pools."""
    rng = np.random.default_rng(31)
    heads, kv, dim, page, n = 4, 2, 64, 16, 40
    stride = 3 << 30  # elements: page 1 starts 6 GB after page 0
    small = Pool(rng, [n], kv, page, dim)
    k_all = torch.empty(2 * stride + kv * page * dim, dtype=torch.float16, device=dev)
    v_all = torch.empty(2 * stride + kv * page * dim, dtype=torch.float16, device=dev)
    k = k_all.as_strided((3, kv, page, dim), (stride, page * dim, dim, 1))
    v = v_all.as_strided((3, kv, dim, page), (stride, page * dim, page, 1))
    order = [2, 0, 1]
    for i, p in enumerate(small.table[0]):
        k[order[i]] = torch.from_numpy(small.k[p]).to(dev)
        v[order[i]] = torch.from_numpy(small.v[p]).to(dev)
    table = i32([order], dev)
    q = rng.standard_normal((1, heads, dim)).astype(np.float16)
    qd = torch.from_numpy(q).to(dev)
    for out in (q4.q4g128_attn_decode(qd, k, v, table, i32([n], dev), scale=0.1),
                q4.q4g128_attn_prefill(qd, k, v, table, i32([0, 1], dev), i32([n], dev), scale=0.1)):
        check_attention(out, q, small, [0, 1], [n], 0.1, "large pool")
    qkv = torch.from_numpy(rng.standard_normal((n, (heads + 2 * kv) * dim)).astype(np.float32)).to(dev)
    q4.q4g128_rope_append(qkv, k, v, table, i32(range(n), dev), None, heads, seq=i32([0] * n, dev))
    for j in range(n):
        row = qkv[j].half().view(-1, dim)
        assert torch.equal(k[order[j // page], :, j % page], row[heads:heads + kv])
        assert torch.equal(v[order[j // page], :, :, j % page], row[heads + kv:])


def test_binding_refusals(dev):
    f16, i = dict(dtype=torch.float16, device=dev), dict(dtype=torch.int32, device=dev)
    k, v = torch.zeros(4, 2, 16, 64, **f16), torch.zeros(4, 2, 64, 16, **f16)
    table, n = torch.zeros(3, 4, **i), torch.ones(3, **i)
    q, qkv, pos = torch.zeros(3, 4, 64, **f16), torch.zeros(3, 512, device=dev), torch.zeros(3, **i)
    starts = torch.arange(4, **i)

    def append(**kw):
        a = dict(qkv=qkv, k_cache=k, v_cache=v, table=table, positions=pos, inv_freq=None, heads=4)
        a.update(kw)
        return q4.q4g128_rope_append(**a)

    def decode(**kw):
        a = dict(q=q, k_cache=k, v_cache=v, table=table, lengths=n)
        a.update(kw)
        return q4.q4g128_attn_decode(**a)

    def prefill(**kw):
        a = dict(q=q, k_cache=k, v_cache=v, table=table, q_starts=starts, lengths=n)
        a.update(kw)
        return q4.q4g128_attn_prefill(**a)

    append(), decode(), prefill()
    for call in (append, decode, prefill):
        for bad, error in ((dict(k_cache=k.float()), TypeError), (dict(v_cache=v.cpu()), ValueError),
                           (dict(k_cache=k[0]), ValueError), (dict(v_cache=k), ValueError),
                           (dict(k_cache=k.transpose(1, 2)), ValueError), (dict(table=table.long()), TypeError),
                           (dict(table=table[0]), ValueError), (dict(table=table.t()), ValueError),
                           (dict(table="table"), TypeError), (dict(k_cache=k[:0], v_cache=v[:0]), q4.Q4Error),
                           (dict(k_cache=torch.zeros(4, 2, 16, 80, **f16), v_cache=torch.zeros(4, 2, 80, 16, **f16)),
                            (ValueError, q4.Q4Error))):
            with pytest.raises(error):
                call(**bad)
    for bad, error in ((dict(qkv=qkv.half()), TypeError), (dict(qkv=qkv[:, :511]), ValueError),
                       (dict(qkv=qkv.t()), ValueError), (dict(qkv=qkv[0]), ValueError), (dict(heads=5), ValueError),
                       (dict(heads=3), q4.Q4Error), (dict(heads=-1), ValueError), (dict(positions=pos[:2]), ValueError),
                       (dict(inv_freq=torch.ones(3, device=dev)), q4.Q4Error),
                       (dict(inv_freq=torch.ones(40, device=dev)), q4.Q4Error),
                       (dict(inv_freq=torch.ones(2, 2, device=dev)), ValueError), (dict(q_norm=pos), TypeError),
                       (dict(q_norm=torch.ones(32, **f16)), ValueError), (dict(seq=pos.long()), TypeError),
                       (dict(eps=-1.0), q4.Q4Error), (dict(q=torch.zeros(3, 4, 32, **f16)), ValueError),
                       (dict(qkv=qkv[:0], positions=pos[:0]), q4.Q4Error)):
        with pytest.raises(error):
            append(**bad)
    for call in (decode, prefill):
        for bad, error in ((dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError), (dict(q=q[..., :32]), ValueError),
                           (dict(lengths=n.long()), TypeError), (dict(scale=0.0), q4.Q4Error),
                           (dict(softcap=-1.0), q4.Q4Error), (dict(window=-1), q4.Q4Error),
                           (dict(slopes=torch.ones(3, device=dev)), ValueError), (dict(max_length=0), q4.Q4Error),
                           (dict(max_length=65), q4.Q4Error), (dict(out=q), q4.Q4Error), (dict(out=n), TypeError),
                           (dict(workspace=n), ValueError), (dict(softcap="1"), TypeError)):
            with pytest.raises(error):
                call(**bad)
    with pytest.raises(q4.Q4Error):
        decode(workspace=torch.zeros(64, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        decode(lengths=n[:2])
    with pytest.raises(ValueError):
        prefill(q_starts=starts[:3])
    with pytest.raises(q4.Q4Error):
        prefill(prefix=n, window=3)
    with pytest.raises(ValueError):
        decode(q=torch.zeros(4, 4, 64, **f16), lengths=torch.ones(4, **i))  # more rows than the table
    torch.cuda.synchronize()


def test_calls_without_a_workspace_in_a_graph_and_on_streams(dev):
    """The workspaces that the binding keeps: one per stream, a graph's own."""
    rng = np.random.default_rng(32)
    pool = Pool(rng, [3000, 1500], 2, 64, 128)
    c = pool.on(dev)
    q = torch.from_numpy(rng.standard_normal((2, 8, 128)).astype(np.float16)).to(dev)
    n, starts = i32([3000, 1500], dev), i32([0, 1, 2], dev)

    def both(stream=None):
        return (q4.q4g128_attn_decode(q, *c, n, stream=stream), q4.q4g128_attn_prefill(q, *c, starts, n, stream=stream))

    want = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [both(s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for _ in range(3):
        for o in outs:
            o.zero_()
        eager = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, want))


def test_example_decodes_what_the_prompt_path_gives(dev):
    """Decoded tokens against the same tokens as a prompt.  Both paths round q, k, the weights and the
    attention outputs to fp16 once, each up to 2^-11 of values about their rms, and the products carry
    fp32 sums: within 16 such roundings of the outputs' rms."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(steps=5) < 16 * H
