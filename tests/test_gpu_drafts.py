"""GPU parity of the calls for drafted tokens (q4g128_attn_tree, q4g128_cache_keep,
slots of q4g128_rope_append) against oracle/drafts.py.

Bounds, from the arithmetic (u = 2^-24, one fp16 rounding = 2^-11 relative, or
2^-25 absolute below the normal range): scores err by ds = (dim + 8) u scale max_j
sum|q k| (+ 2^-21 softcap, + 2^-22 largest |slope * distance|), a weight's relative
error is 2 ds plus 2^-11 for its fp16 form, a sum over n positions adds n u, and a
weight below 2^-14 of the largest errs by 2^-25 of it.  With A = sum w |v|:
|out - ref| <= 2^-11 |ref| + 2^-25 + (2^-11 + 2 ds + (n + 64) u) A + n 2^-25 max|v|.
Moved tokens are equal bit for bit.
"""
import numpy as np
import pytest

from oracle import attention as ref
from oracle import drafts
from gpu_helpers import U32, device, note
from test_gpu_attention import H, TINY, Pool, i32

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


def trees(rng, new, kind="tree"):
    """Masks of the tokens of all sequences, as int64: trees, chains, or any bits (none and foreign ones among them)."""
    masks = []
    for n in new:
        mine = []
        for i in range(n):
            if kind == "any":
                m = int(rng.integers(0, 2 ** 63)) & int(rng.integers(0, 2 ** 63)) | int(rng.integers(0, 2)) << 63
                mine.append(0 if rng.random() < 0.2 else m)
            else:
                parent = i - 1 if kind == "chain" else int(rng.integers(max(-1, i - 5), i)) if i else -1
                mine.append((mine[parent] if parent >= 0 else 0) | (1 << i if i < 64 else 0))
        masks += mine
    return np.array([m - (1 << 64) if m >> 63 else m for m in masks], dtype=np.int64)


def check(got, q, pool, starts, lengths, scale, masks, what, softcap=0.0, window=0, slopes=None):
    want, mag, dots = drafts.attention(q, pool.k, pool.v, pool.table, starts, lengths, scale, masks, softcap, window,
                                       slopes)
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


def tree_case(dev, seed, new, lengths, heads, kv, dim, page, kind="tree", absent=(), softcap=0.0, window=0, slopes=False,
              junk=np.nan, **kw):
    rng = np.random.default_rng(seed)
    pool = Pool(rng, lengths, kv, page, dim, absent=absent, junk=junk)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(starts[-1]), heads, dim)).astype(np.float16)
    masks = None if kind is None else trees(rng, new, kind)
    slope = np.linspace(0.4, 0.01, heads).astype(np.float32) if slopes else None
    scale = dim ** -0.5 * 1.5
    args = (torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev),
            None if masks is None else torch.from_numpy(masks).to(dev))
    options = dict(scale=scale, softcap=softcap, window=window,
                   slopes=None if slope is None else torch.from_numpy(slope).to(dev), **kw)
    out = q4.q4g128_attn_tree(*args, **options)
    check(out, q, pool, starts, lengths, scale, masks, f"tree {new} of {lengths}", softcap, window, slope)
    return out, args, options


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_tree_dims_and_pages(dev, dim, page):
    tree_case(dev, 1, [7, 3], [203, 90], 4, 2, dim, page)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows", [(3, 5), (8, 4), (20, 3), (64, 2), (64, 5), (13, 64)])
def test_tree_row_blocks(dev, dim, rows):
    """One, two, four and more row blocks of 16 per kv head, the last one part filled."""
    n, group = rows
    tree_case(dev, 2, [n, max(1, n // 3)], [300, 150], group, 1, dim, 64)


@pytest.mark.parametrize("kind", ["tree", "chain", "any", None])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
def test_tree_masks(dev, kind, n):
    tree_case(dev, 3, [n], [n + 101], 4, 2, 64, 16, kind)


@pytest.mark.parametrize("before", [0, 1, 31, 32, 33, 63, 64, 65, 127, 200])
def test_tree_draft_across_tiles(dev, before):
    """Drafts that begin anywhere in a tile, over nothing too."""
    tree_case(dev, 4, [40], [before + 40], 2, 1, 64, 16, "any")
    tree_case(dev, 5, [5], [before + 5], 2, 1, 128, 32)


@pytest.mark.parametrize("window", [1, 2, 5, 17, 63, 64, 65, 100, 257, 4096])
@pytest.mark.parametrize("kind", ["tree", "any", None])
def test_tree_window(dev, window, kind):
    tree_case(dev, 6, [40, 9], [240, 30], 4, 2, 64, 32, kind, window=window)


@pytest.mark.parametrize("softcap,slopes", [(5.0, False), (0.0, True), (20.0, True), (200.0, False)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tree_capped_and_biased(dev, softcap, slopes, dim):
    tree_case(dev, 7, [23, 6], [190, 70], 6, 2, dim, 32, softcap=softcap, slopes=slopes)
    tree_case(dev, 8, [9], [300], 6, 2, dim, 64, "any", softcap=softcap, slopes=slopes, window=20)


def test_tree_empty_sequences_and_rows(dev):
    """Sequences without drafted tokens, with fewer positions than tokens, and without positions."""
    tree_case(dev, 9, [0, 5, 0, 7, 3], [40, 60, 0, 4, 0], 4, 1, 64, 16)
    tree_case(dev, 10, [0, 70 - 64, 8], [0, 3, 8], 4, 1, 64, 16, "any", window=3)


def test_tree_absent_pages(dev):
    tree_case(dev, 11, [9, 4], [300, 100], 4, 2, 64, 16, absent=[(0, 0), (0, 7), (1, 3)])
    tree_case(dev, 11, [9, 4], [300, 100], 4, 2, 64, 16, absent=[(0, i) for i in range(19)])


def test_tree_long_and_split(dev):
    """One sequence in many parts, which join in groups; uneven ones; many short ones."""
    tree_case(dev, 12, [3], [9000], 2, 1, 64, 64)
    tree_case(dev, 13, [12, 2, 7], [5000, 17, 1200], 8, 2, 128, 64)
    tree_case(dev, 14, [1 + i % 5 for i in range(70)], [1 + 37 * i % 400 + 5 for i in range(70)], 2, 1, 64, 16)


@pytest.mark.parametrize("junk", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dim,n,group", [(64, 4, 3), (128, 10, 3), (128, 30, 2), (256, 9, 3)])
def test_tree_masked_positions_stay_out(dev, junk, dim, n, group):
    """A drafted token that most do not see, and positions before a window, hold junk; who sees them may not be finite."""
    rng = np.random.default_rng(15)
    length, window = 170 + n, 50
    pool = Pool(rng, [length], 1, 16, dim, junk=junk)
    starts = [0, n]
    for j in list(range(0, length - n - window - 1)) + [length - 1]:
        pool.k[pool.table[0, j // 16], :, j % 16] = junk
        pool.v[pool.table[0, j // 16], :, :, j % 16] = junk
    masks = trees(rng, [n]) & ~np.int64(1 << (n - 1))  # no one sees the last
    q = rng.standard_normal((n, group, dim)).astype(np.float16)
    out = q4.q4g128_attn_tree(torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32([length], dev),
                              torch.from_numpy(masks).to(dev), scale=0.2, window=window)
    check(out, q, pool, starts, [length], 0.2, masks, f"junk {junk}", window=window)


def test_tree_seen_infinities_reach_their_rows_only(dev):
    rng = np.random.default_rng(16)
    pool = Pool(rng, [100], 1, 16, 64)
    pool.v[pool.table[0, 6], 0, 5, 1] = np.inf  # dimension 5 of drafted token 1
    masks = np.array([1, 3, 5, 11], dtype=np.int64)  # tokens 1 and 3 see token 1
    q = rng.standard_normal((4, 2, 64)).astype(np.float16)
    c = pool.on(dev)
    out = q4.q4g128_attn_tree(torch.from_numpy(q).to(dev), *c, i32([0, 4], dev), i32([100], dev),
                              torch.from_numpy(masks).to(dev), scale=0.2).cpu().numpy()
    assert np.all(np.isinf(out[[1, 3], :, 5]))
    out[[1, 3], :, 5] = 0
    assert np.all(np.isfinite(out))
    pool.v[pool.table[0, 6], 0, 5, 1] = 0
    want, mag, _ = drafts.attention(q, pool.k, pool.v, pool.table, [0, 4], [100], 0.2, masks)
    want[[1, 3], :, 5] = 0
    assert np.all(np.abs(out - want) <= 2e-3 * mag + 1e-6)


def test_tree_max_new_and_rows_of_no_sequence(dev):
    """Rows past max_new and rows of no sequence are left as they were."""
    rng = np.random.default_rng(17)
    pool = Pool(rng, [80, 60], 1, 16, 64)
    q = torch.from_numpy(rng.standard_normal((20, 2, 64)).astype(np.float16)).to(dev)
    out = torch.full_like(q, 7.0)
    args = (q, *pool.on(dev), i32([2, 10, 15], dev), i32([80, 60], dev))
    q4.q4g128_attn_tree(*args, scale=0.1, max_new=6, out=out)
    whole = q4.q4g128_attn_tree(*args, scale=0.1)
    for rows, kept in ((range(0, 2), True), (range(2, 8), False), (range(8, 10), True), (range(10, 15), False),
                       (range(15, 20), True)):
        for t in rows:
            assert torch.equal(out[t], torch.full_like(out[t], 7.0) if kept else whole[t]), t


@pytest.mark.parametrize("options", [dict(), dict(softcap=30.0, slopes=True), dict(window=300), dict(window=40, slopes=True)])
def test_tree_options_in_parts(dev, options):
    """Windows, caps and biases where the positions are split, and many sequences beside a long one."""
    tree_case(dev, 18, [20, 3], [6000, 900], 4, 2, 128, 64, "any", **options)
    tree_case(dev, 19, [i % 4 for i in range(70)], [3000 if i == 33 else 4 + 11 * i % 90 for i in range(70)], 2, 1, 64, 16, "any",
              **options)


def test_tree_max_new_in_parts(dev):
    """The join leaves rows past max_new and rows of no sequence as they were."""
    rng = np.random.default_rng(20)
    lengths, starts = [5000, 2500] + [40] * 68, [2, 10, 15] + list(range(16, 84))
    pool = Pool(rng, lengths, 1, 64, 64)
    q = rng.standard_normal((90, 2, 64)).astype(np.float16)
    args = (torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev))
    out = torch.full((90, 2, 64), 7.0, dtype=torch.float16, device=dev)
    q4.q4g128_attn_tree(*args, scale=0.1, max_new=6, out=out)
    left = [0, 1, 8, 9] + list(range(83, 90))
    assert torch.all(out[left] == 7.0)
    whole = q4.q4g128_attn_tree(*args, scale=0.1, out=torch.zeros_like(out))
    out[left] = whole[left]
    check(out, q, pool, starts, lengths, 0.1, None, "max_new in parts", 0.0, 0, None)


def test_tree_is_decode_for_one_token_and_prompt_for_a_chain(dev):
    """Within the two calls' bounds of each other, from the same definition."""
    rng = np.random.default_rng(18)
    lengths, new = [700, 64, 9], [1, 1, 1]
    pool = Pool(rng, lengths, 2, 64, 128)
    c, n = pool.on(dev), i32(lengths, dev)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128)).astype(np.float16)).to(dev)
    a = q4.q4g128_attn_tree(q, *c, i32([0, 1, 2, 3], dev), n)
    b = q4.q4g128_attn_decode(q, *c, n)
    assert torch.allclose(a, b, rtol=2e-3, atol=2e-3)
    q = torch.from_numpy(rng.standard_normal((60, 8, 128)).astype(np.float16)).to(dev)
    starts = i32([0, 40, 51, 60], dev)
    assert torch.allclose(q4.q4g128_attn_tree(q, *c, starts, n), q4.q4g128_attn_prefill(q, *c, starts, n), rtol=2e-3,
                          atol=2e-3)


def test_tree_repeats_on_other_streams_and_in_graphs(dev):
    """Bit for bit the same on another stream, with a shared workspace, and replayed between eager calls."""
    out, args, options = tree_case(dev, 19, [12, 3, 7], [5000, 17, 1200], 8, 2, 128, 64)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = q4.q4g128_attn_tree(*args, **options, stream=other)
    other.synchronize()
    assert torch.equal(out, got)
    ws = torch.zeros(max(q4.q4g128_attn_tree_workspace(22, 3, 8, 2, 128, 22, 5056), q4.q4g128_attn_decode_workspace(3, 8, 128)),
                     dtype=torch.uint8, device=dev)
    for _ in range(2):
        assert torch.equal(out, q4.q4g128_attn_tree(*args, **options, workspace=ws))
        q4.q4g128_attn_decode(args[0][:3], *args[1:4], args[5], workspace=ws)
        assert not ws[:q4.ATTN_COUNTER_BYTES].any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = q4.q4g128_attn_tree(*args, **options)
    for _ in range(3):
        held.fill_(7.0)
        graph.replay()
        eager = q4.q4g128_attn_tree(*args, **options)
        torch.cuda.synchronize()
        assert torch.equal(out, held) and torch.equal(out, eager)


# ---------------------------------------------------------------------------
# keep
# ---------------------------------------------------------------------------

def keep_case(dev, seed, starts, kept, kv, dim, page, draft=70, absent=()):
    rng = np.random.default_rng(seed)
    pool = Pool(rng, [n + draft for n in starts], kv, page, dim, absent=absent, junk=3.0)
    k, v, table = pool.on(dev)
    keep_starts = np.concatenate([[0], np.cumsum([len(a) for a in kept])]).astype(int)
    flat = np.array([i for a in kept for i in a], dtype=np.int32)
    q4.q4g128_cache_keep(k, v, table, i32(starts, dev), i32(keep_starts, dev), i32(flat, dev))
    want_k, want_v = drafts.keep(pool.k, pool.v, pool.table, starts, keep_starts, flat)
    assert np.array_equal(k.cpu().numpy().view(np.uint16), want_k.view(np.uint16))
    assert np.array_equal(v.cpu().numpy().view(np.uint16), want_v.view(np.uint16))


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_keep_dims_and_pages(dev, dim, page):
    keep_case(dev, 20, [30, 0, 61], [[0, 2, 3, 9], [1], [5, 6, 7, 31, 63]], 2, dim, page)


@pytest.mark.parametrize("taken", [0, 1, 2, 31, 32, 33, 63, 64])
def test_keep_counts(dev, taken):
    """Paths that overlap the places they move to, longer than a workgroup moves at a time."""
    rng = np.random.default_rng(taken)
    keep_case(dev, 21, [77, 10], [sorted(rng.choice(64, taken, replace=False)), list(range(taken))], 3, 64, 16)
    keep_case(dev, 22, [5], [list(range(64 - taken, 64))], 1, 128, 32)


def test_keep_tokens_without_a_place(dev):
    """Absent pages, numbers below zero and beyond the table: not moved, nothing else touched."""
    keep_case(dev, 23, [30, 30], [[1, 2, 40, 5000], [-40, 3, 10 ** 9, 2 ** 31 - 1]], 2, 64, 16, absent=[(0, 1), (1, 3)])


def test_slots_apart_from_rotary_positions(dev):
    """A head is turned by its position and written to its slot."""
    rng = np.random.default_rng(24)
    heads, kv, dim, page = 4, 2, 64, 16
    positions, slots, seq = [40, 41, 41, 42, 42, 7, 8, 8, 8], [40, 41, 42, 43, 44, 7, 8, 9, 10], [0] * 5 + [1] * 4
    pool = Pool(rng, [50, 20], kv, page, dim, junk=7.0)
    qkv = torch.from_numpy(rng.standard_normal((9, (heads + 2 * kv) * dim)).astype(np.float32)).to(dev)
    freq = torch.from_numpy((100.0 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32)).to(dev)
    k, v, table = pool.on(dev)
    q = q4.q4g128_rope_append(qkv, k, v, table, i32(positions, dev), freq, heads, seq=i32(seq, dev),
                              slots=i32(slots, dev)).cpu().numpy()
    want_k, want_v = pool.k.copy(), pool.v.copy()
    k, v = k.cpu().numpy(), v.cpu().numpy()
    for t in range(9):
        p, o = pool.table[seq[t], slots[t] // page], slots[t] % page
        rows = qkv[t].cpu().numpy().reshape(-1, dim)
        for h in range(heads + kv):
            want = ref.rotated(rows[h], positions[t], freq.cpu().numpy(), dim)
            got = q[t, h] if h < heads else k[p, h - heads, o]
            assert np.all(np.abs(got - want) <= 2 ** -11 * np.abs(want) + 1e-4), (t, h)
        want_k[p, :, o], want_v[p, :, :, o] = k[p, :, o], rows[heads + kv:].astype(np.float16)
    assert np.array_equal(k, want_k) and np.array_equal(v, want_v)


def test_drafting_step(dev):
    """Append a tree, attend, keep a path, go on with one token: the same as the path appended as a chain."""
    rng = np.random.default_rng(25)
    heads, kv, dim, page, base = 8, 2, 128, 16, 37
    freq = torch.from_numpy((1000.0 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32)).to(dev)
    rows = torch.from_numpy(rng.standard_normal((base + 12, (heads + 2 * kv) * dim)).astype(np.float32)).to(dev)
    parents = [-1, 0, 0, 1, 2, 2, 4, 5, 5, 6]
    path = [0, 2, 4, 6, 9]
    masks, depth = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)

    def cache():
        k = torch.zeros((6, kv, page, dim), dtype=torch.float16, device=dev)
        v = torch.zeros((6, kv, dim, page), dtype=torch.float16, device=dev)
        table = i32([[3, 1, 5, 0]], dev)
        q4.q4g128_rope_append(rows[:base], k, v, table, i32(range(base), dev), freq, heads, seq=i32([0] * base, dev))
        return k, v, table

    tree, chain = cache(), cache()
    n = len(parents)
    q = q4.q4g128_rope_append(rows[base:base + n], *tree, i32([base + d for d in depth], dev), freq, heads,
                              seq=i32([0] * n, dev), slots=i32(range(base, base + n), dev))
    got = q4.q4g128_attn_tree(q, *tree, i32([0, n], dev), i32([base + n], dev),
                              torch.tensor(masks, device=dev, dtype=torch.int64))
    picked = rows[base:base + n][path].contiguous()
    m = len(path)
    qc = q4.q4g128_rope_append(picked, *chain, i32(range(base, base + m), dev), freq, heads, seq=i32([0] * m, dev))
    want = q4.q4g128_attn_prefill(qc, *chain, i32([0, m], dev), i32([base + m], dev))
    assert torch.equal(q[path], qc)
    # Either call errs by 2^-11 of the result for its last rounding and by 2^-11 of sum w |v| for its weights', both at
    # most 2^-11 max |v|; sums of these few positions add less than a hundredth of that.
    assert (got[path].float() - want.float()).abs().max() <= 4.04 * H * tree[1].abs().max()
    q4.q4g128_cache_keep(*tree, i32([base], dev), i32([0, m], dev), i32(path, dev))
    outs = []
    for c in (tree, chain):
        qn = q4.q4g128_rope_append(rows[base + n:base + n + 1], *c, i32([base + m], dev), freq, heads)
        outs.append(q4.q4g128_attn_decode(qn, *c, i32([base + m + 1], dev)))
    assert torch.equal(outs[0], outs[1])
