"""GPU parity of the latent calls (q4g128_latent_append, q4g128_latent_keep,
q4g128_latent_attn) against oracle/latent.py.

Bounds, from the arithmetic (u = 2^-24, one fp16 rounding = 2^-11 relative, or
2^-25 absolute below the normal range):
  * append: |y - ref| <= 2^-11 |ref| + 2^-25 + (latent + 64) u mscale (|lo| + |hi|).
  * attention: scores err by ds = (latent + 72) u scale max_j sum|q c|, a weight's
    relative error is 2 ds plus 2^-11 for its fp16 form, a sum over n positions adds
    n u, and a weight below 2^-14 of the largest errs by 2^-25 of it; with A = sum w
    |c|: |out - ref| <= 2^-11 |ref| + 2^-25 + (2^-11 + 2 ds + (n + 64) u) A + n 2^-25 max|c|.
"""
import numpy as np
import pytest

from oracle import attention as heads_ref
from oracle import drafts
from oracle import latent as ref
from gpu_helpers import U32, device, note
from test_gpu_attention import H, TINY, i32
from test_gpu_drafts import trees

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")

ROT = ref.ROT


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


@pytest.fixture(scope="module")
def dev():
    return device()


class Rows:
    """A latent cache of random pages, its table a random choice of them; junk fills what no sequence holds."""

    def __init__(self, rng, lengths, latent, page, junk=np.nan, absent=(), cols=None):
        used = [-(-max(0, n) // page) for n in lengths]
        self.page, self.pages = page, sum(used) + 2
        cols = cols or max(1, max(used))
        order = rng.permutation(self.pages)
        self.rows = rng.standard_normal((self.pages, page, latent + ROT)).astype(np.float16)
        held = np.zeros((self.pages, page), dtype=bool)
        self.table = np.full((len(lengths), cols), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(lengths):
            for i in range(used[s]):
                self.table[s, i] = order[at]
                held[order[at], :min(page, n - i * page)] = True
                at += 1
        if junk is not None:
            self.rows[~held] = junk
        for s, i in absent:
            self.table[s, i] = (-1, self.pages, 2 ** 31 - 1)[(s + i) % 3]

    def on(self, dev):
        return torch.from_numpy(self.rows).to(dev), torch.from_numpy(self.table).to(dev)


def check(got, q, pool, starts, lengths, scale, masks, what):
    want, mag, dots = ref.attention(q, pool.rows, pool.table, starts, lengths, scale, masks)
    n = max(1, max(lengths))
    ds = (q.shape[2] + 8) * U32 * scale * dots
    finite = pool.rows[np.isfinite(pool.rows)]
    cmax = np.abs(finite).max() if len(finite) else 0.0
    bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[..., None] * mag + n * TINY * cmax * (mag > 0)
    g = got.float().cpu().numpy().astype(np.float64)
    assert g.shape == want.shape
    assert np.all(np.isfinite(g)), f"{what}: {int((~np.isfinite(g)).sum())} outputs are not finite"
    err = np.abs(g - want)
    assert np.all(err <= bound), f"{what}: {int((err > bound).sum())} above the bound, worst {(err / bound).max():.3f}"


def attn_case(dev, seed, new, lengths, heads, latent, page, kind=None, absent=(), junk=np.nan, rising=0.0, **kw):
    rng = np.random.default_rng(seed)
    pool = Rows(rng, lengths, latent, page, absent=absent, junk=junk)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(starts[-1]), heads, latent + ROT)).astype(np.float16)
    if rising:
        # scores that rise along the sequence, so that the running maximum moves again and again
        for s, n in enumerate(lengths):
            for j in range(n):
                p = pool.table[s, j // page]
                if 0 <= p < pool.pages:
                    pool.rows[p, j % page, -1] = rising * j
        q[:, :, -1] = 1.0
    masks = None if kind is None else trees(rng, new, kind)
    scale = 0.06
    args = (torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev), scale)
    kw["masks"] = None if masks is None else torch.from_numpy(masks).to(dev)
    out = q4.q4g128_latent_attn(*args, **kw)
    check(out, q, pool, starts, lengths, scale, masks, f"latent {new} of {lengths}")
    return out, args, kw


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attn_widths_and_pages(dev, latent, page):
    attn_case(dev, 1, [1, 1, 1], [203, 90, 64], 6, latent, page)


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("heads", [1, 5, 16, 17, 20, 32, 33, 48, 64, 65, 128])
def test_attn_heads(dev, latent, heads):
    """One row block, two, 64 rows and more, the last one part filled."""
    attn_case(dev, 2, [1, 1], [150, 77], heads, latent, 32)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 193, 300])
@pytest.mark.parametrize("heads", [4, 40])
def test_attn_lengths(dev, length, heads):
    attn_case(dev, 3, [1], [length], heads, 512, 16)


@pytest.mark.parametrize("kind", ["tree", "any", "chain", None])
@pytest.mark.parametrize("n", [2, 7, 31, 64])
@pytest.mark.parametrize("latent,heads", [(512, 3), (256, 10), (128, 1)])
def test_attn_drafts(dev, kind, n, latent, heads):
    attn_case(dev, 4, [n, 1, max(1, n // 2)], [n + 101, 1, 200], heads, latent, 16, kind)


@pytest.mark.parametrize("before", [0, 1, 31, 33, 63, 64, 65, 127, 200])
def test_attn_draft_across_tiles(dev, before):
    attn_case(dev, 5, [40], [before + 40], 2, 128, 16, "any")


@pytest.mark.parametrize("new", [[70], [130, 3], [1, 200, 64]])
def test_attn_prompts(dev, new):
    """More tokens than a mask could name, without masks."""
    attn_case(dev, 6, new, [n + 37 for n in new], 5, 128, 32)
    attn_case(dev, 7, new, new, 3, 512, 64)


def test_attn_empty_sequences_and_rows(dev):
    attn_case(dev, 8, [0, 5, 0, 7, 3], [40, 60, 0, 4, 0], 4, 128, 16)
    attn_case(dev, 9, [0, 6, 8], [0, 3, 8], 20, 256, 16, "any")


def test_attn_absent_pages(dev):
    attn_case(dev, 10, [9, 4], [300, 100], 4, 512, 16, "tree", absent=[(0, 0), (0, 7), (1, 3)])
    attn_case(dev, 10, [1, 1], [300, 100], 40, 512, 16, absent=[(0, 0), (0, 7), (1, 3)])
    attn_case(dev, 10, [9, 4], [300, 100], 4, 256, 32, "tree", absent=[(0, i) for i in range(10)])


@pytest.mark.parametrize("heads", [2, 24, 40])
def test_attn_long_and_split(dev, heads):
    attn_case(dev, 11, [1], [9000], heads, 128, 64)
    attn_case(dev, 12, [1, 1, 1], [5000, 17, 1200], heads, 256, 64)
    attn_case(dev, 13, [1 + i % 3 for i in range(70)], [3 + 37 * i % 400 for i in range(70)], heads, 128, 16)


@pytest.mark.parametrize("heads", [3, 20, 40])
@pytest.mark.parametrize("kind", ["any", None])
def test_attn_many_sequences_below_a_loose_bound(dev, heads, kind):
    """Far fewer rows than max_new would allow, sequences without any, one in many parts."""
    new = [i % 4 for i in range(150)]
    lengths = [n + 29 * i % 90 for i, n in enumerate(new)]
    lengths[77] = 3000
    attn_case(dev, 33, new, lengths, heads, 128, 16, kind, max_new=64)


@pytest.mark.parametrize("heads", [3, 30, 64])
@pytest.mark.parametrize("rising", [0.05, 2.0])
def test_attn_moving_maximum(dev, heads, rising):
    """Maxima that differ from wave to wave and tile to tile, by little and by more than fp16 weights span."""
    attn_case(dev, 14, [1, 1], [500, 260], heads, 512, 64, rising=rising)
    attn_case(dev, 15, [5], [300], heads, 128, 64, "tree", rising=rising)


@pytest.mark.parametrize("junk", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("latent,n,heads", [(512, 4, 3), (512, 10, 7), (256, 9, 3), (128, 30, 2)])
def test_attn_masked_positions_stay_out(dev, junk, latent, n, heads):
    """Drafted tokens that most do not see hold junk."""
    rng = np.random.default_rng(16)
    length = 170 + n
    pool = Rows(rng, [length], latent, 16, junk=junk)
    for k in (n - 1, n - 2):
        j = length - n + k
        pool.rows[pool.table[0, j // 16], j % 16, ::3] = junk
    masks = trees(rng, [n]) & ~np.int64(3 << (n - 2))
    q = rng.standard_normal((n, heads, latent + ROT)).astype(np.float16)
    out = q4.q4g128_latent_attn(torch.from_numpy(q).to(dev), *pool.on(dev), i32([0, n], dev), i32([length], dev), 0.06,
                                masks=torch.from_numpy(masks).to(dev))
    check(out, q, pool, [0, n], [length], 0.06, masks, f"junk {junk}")


def test_attn_max_new_and_rows_of_no_sequence(dev):
    rng = np.random.default_rng(17)
    pool = Rows(rng, [80, 60], 128, 16)
    q = torch.from_numpy(rng.standard_normal((20, 2, 128 + ROT)).astype(np.float16)).to(dev)
    out = torch.full((20, 2, 128), 7.0, dtype=torch.float16, device=dev)
    args = (q, *pool.on(dev), i32([2, 10, 15], dev), i32([80, 60], dev), 0.1)
    q4.q4g128_latent_attn(*args, max_new=6, out=out)
    whole = q4.q4g128_latent_attn(*args)
    for rows, kept in ((range(0, 2), True), (range(2, 8), False), (range(8, 10), True), (range(10, 15), False),
                       (range(15, 20), True)):
        for t in rows:
            assert torch.equal(out[t], torch.full_like(out[t], 7.0) if kept else whole[t]), t


@pytest.mark.parametrize("heads", [2, 5, 20])
def test_attn_max_new_in_parts(dev, heads):
    rng = np.random.default_rng(34)
    lengths, starts = [5000, 2500] + [40] * 68, [2, 10, 15] + list(range(16, 84))
    pool = Rows(rng, lengths, 128, 64)
    q = rng.standard_normal((90, heads, 128 + ROT)).astype(np.float16)
    args = (torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev), 0.06)
    out = torch.full((90, heads, 128), 7.0, dtype=torch.float16, device=dev)
    q4.q4g128_latent_attn(*args, max_new=6, out=out)
    left = [0, 1, 8, 9] + list(range(83, 90))
    assert torch.all(out[left] == 7.0)
    whole = q4.q4g128_latent_attn(*args, out=torch.zeros_like(out))
    out[left] = whole[left]
    check(out, q, pool, starts, lengths, 0.06, None, "max_new in parts")


def test_attn_cache_in_a_larger_pool(dev):
    rng = np.random.default_rng(18)
    pool = Rows(rng, [300], 256, 32)
    rows, table = pool.on(dev)
    wide = torch.full((pool.pages, 3, 32, 256 + ROT), float("nan"), dtype=torch.float16, device=dev)
    wide[:, 1] = rows
    q = torch.from_numpy(rng.standard_normal((1, 8, 256 + ROT)).astype(np.float16)).to(dev)
    args = (table, i32([0, 1], dev), i32([300], dev), 0.06)
    assert torch.equal(q4.q4g128_latent_attn(q, rows, *args), q4.q4g128_latent_attn(q, wide[:, 1], *args))


@pytest.mark.parametrize("heads", [5, 40])
def test_attn_repeats_on_other_streams_and_in_graphs(dev, heads):
    out, args, kw = attn_case(dev, 19, [3, 1, 7], [5000, 17, 1200], heads, 128, 64, "tree")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = q4.q4g128_latent_attn(*args, **kw, stream=other)
    other.synchronize()
    assert torch.equal(out, got)
    ws = torch.zeros(q4.q4g128_latent_attn_workspace(heads, 128, 11), dtype=torch.uint8, device=dev)
    for _ in range(2):
        assert torch.equal(out, q4.q4g128_latent_attn(*args, **kw, workspace=ws))
        assert not ws[:q4.ATTN_COUNTER_BYTES].any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = q4.q4g128_latent_attn(*args, **kw)
    for _ in range(3):
        held.fill_(7.0)
        graph.replay()
        eager = q4.q4g128_latent_attn(*args, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, held) and torch.equal(out, eager)


# ---------------------------------------------------------------------------
# append and keep
# ---------------------------------------------------------------------------

def append_case(dev, seed, placed, latent, page, heads=0, main=128, interleaved=False, norm=False, mscale=1.0, extra=0,
                slots=None, joint=True, turn=True, absent=(), cols=None):
    """placed: [(sequence, position)] of the tokens; slots: the positions written, if others."""
    rng = np.random.default_rng(seed)
    tokens = len(placed)
    slots = [p for _, p in placed] if slots is None else slots
    seqs = max(s for s, _ in placed) + 1
    lengths = [1 + max([p for (s, _), p in zip(placed, slots) if s == b] or [0]) for b in range(seqs)]
    pool = Rows(rng, [min(n, (cols or 10 ** 9) * page) for n in lengths], latent, page, junk=7.0, absent=absent, cols=cols)
    kv = rng.standard_normal((tokens, latent + ROT + extra)).astype(np.float32) * 3
    freq = (10000.0 ** (-np.arange(ROT // 2) / (ROT // 2))).astype(np.float32) if turn else None
    weight = rng.uniform(0.5, 1.5, latent).astype(np.float16) if norm else None
    both = torch.from_numpy(rng.standard_normal((tokens, max(heads, 1), main + ROT)).astype(np.float32)).to(dev)
    qm, qr = both[:, :, :main], both[:, :, main:]
    if not joint:
        qm, qr = qm.transpose(0, 1).contiguous().transpose(0, 1), qr.contiguous()
    rows, table = pool.on(dev)
    q = q4.q4g128_latent_append(
        torch.from_numpy(kv).to(dev), rows, table, i32([p for _, p in placed], dev),
        None if freq is None else torch.from_numpy(freq).to(dev), seq=i32([s for s, _ in placed], dev),
        slots=i32(slots, dev), norm=None if weight is None else torch.from_numpy(weight).to(dev), eps=1e-5,
        interleaved=interleaved, mscale=mscale, q_main=qm if heads else None, q_rot=qr if heads else None)
    got, want = rows.cpu().numpy(), pool.rows.copy()

    def bound(want, x, first):
        pair = np.abs(x)
        for i in range(ROT // 2):
            lo, hi = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + i + ROT // 2)
            pair[lo] = pair[hi] = (np.abs(x[lo]) + np.abs(x[hi])) * abs(mscale)
        return H * np.abs(want) + TINY + (latent + 64) * U32 * pair

    for t, (s, p) in enumerate(placed):
        at = ref.slot(pool.table, s, slots[t], page, pool.pages)
        if at:
            w = ref.row(kv[t], p, freq, latent, interleaved, mscale, weight, 1e-5)
            plain = ref.row(kv[t], p, None, latent, norm=weight, eps=1e-5)
            err = np.abs(got[at].astype(np.float64) - w)
            assert np.all(err <= bound(w, plain, latent)), (t, err.max())
            want[at] = got[at]
        for h in range(heads):
            x = both[t, h].cpu().numpy().astype(np.float64)
            w = np.concatenate([x[:main], ref.turned(x[main:], p, freq, interleaved, mscale)])
            err = np.abs(q[t, h].cpu().numpy().astype(np.float64) - w)
            assert np.all(err <= bound(w, x, main)), (t, h, err.max())
    assert (q is None) == (heads == 0)
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))  # nothing else changes


@pytest.mark.parametrize("latent", [128, 256, 512])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_widths(dev, latent, interleaved, norm):
    append_case(dev, 20, [(0, 5), (1, 40), (0, 6), (2, 17), (0, 7)], latent, 32, 3, latent, interleaved, norm, mscale=1.3,
                extra=12)


@pytest.mark.parametrize("heads,main", [(0, 128), (1, 8), (1, 512), (7, 64), (128, 128), (60, 72), (33, 1024)])
@pytest.mark.parametrize("joint", [True, False])
def test_append_queries(dev, heads, main, joint):
    append_case(dev, 21, [(0, 3), (1, 9)], 256, 16, heads, main, joint=joint)


def test_append_without_rotation_and_far(dev):
    append_case(dev, 22, [(0, 3), (0, 4)], 128, 16, 2, 64, turn=False, mscale=2.0)
    append_case(dev, 23, [(0, 131071), (0, 100003)], 128, 256, 2, 64, interleaved=True)


def test_append_many_tokens_and_slots(dev):
    append_case(dev, 24, [(0, p) for p in range(3, 133)] + [(1, p) for p in range(50)], 512, 64, 2, 128, norm=True)
    append_case(dev, 25, [(0, 20), (0, 21), (0, 21), (0, 22)], 128, 16, 2, 64, slots=[20, 21, 22, 23])


def test_append_tokens_without_a_place(dev):
    append_case(dev, 26, [(0, 5), (0, 40), (1, 3), (1, 100)], 128, 16, 1, 64, absent=[(0, 2)], cols=3)


@pytest.mark.parametrize("latent", [128, 256, 512])
def test_keep(dev, latent):
    rng = np.random.default_rng(27)
    starts, kept = [30, 0, 61], [[0, 2, 3, 9], [1], list(range(5, 44))]
    pool = Rows(rng, [n + 70 for n in starts], latent, 32, junk=3.0)
    rows, table = pool.on(dev)
    keep_starts = np.concatenate([[0], np.cumsum([len(a) for a in kept])]).astype(int)
    flat = [i for a in kept for i in a]
    q4.q4g128_latent_keep(rows, table, i32(starts, dev), i32(keep_starts, dev), i32(flat, dev))
    want, _ = drafts.keep(pool.rows, None, pool.table, starts, keep_starts, flat)
    assert np.array_equal(rows.cpu().numpy().view(np.uint16), want.view(np.uint16))


def test_one_token_through_the_absorbed_products(dev):
    """Queries by the heads' key weights, latent attention, values by the heads' value weights, all int4 products of one
    token, against attention over the keys and values that the rows stand for."""
    rng = np.random.default_rng(28)
    heads, own, value, latent, page, length = 4, 128, 128, 256, 16, 70
    pool = Rows(rng, [length], latent, page)
    w_key = rng.standard_normal((heads, latent, own)).astype(np.float32) / 16      # q in the latent space = w_key q
    w_value = rng.standard_normal((heads, value, latent)).astype(np.float32) / 16
    quantized = [[q4.q4g128_quantize(torch.from_numpy(w[h]).to(dev)) for h in range(heads)] for w in (w_key, w_value)]
    q_own = torch.from_numpy(rng.standard_normal((heads, own)).astype(np.float16)).to(dev)
    q_rot = torch.from_numpy(rng.standard_normal((1, heads, ROT)).astype(np.float32)).to(dev)
    kv = torch.from_numpy(rng.standard_normal((1, latent + ROT)).astype(np.float32)).to(dev)
    freq = torch.from_numpy((1000.0 ** (-np.arange(32) / 32)).astype(np.float32)).to(dev)
    rows, table = pool.on(dev)
    q_main = torch.empty((1, heads, latent), dtype=torch.float32, device=dev)
    q4.q4g128_gemv_grouped([(*quantized[0][h], q_own[h]) for h in range(heads)], [q_main[0, h] for h in range(heads)])
    q = q4.q4g128_latent_append(kv, rows, table, i32([length - 1], dev), freq, q_main=q_main, q_rot=q_rot)
    scale = (own + ROT) ** -0.5
    mixed = q4.q4g128_latent_attn(q, rows, table, i32([0, 1], dev), i32([length], dev), scale)
    out = torch.stack(q4.q4g128_gemv_grouped([(*quantized[1][h], mixed[0, h]) for h in range(heads)])).cpu().numpy()

    def weights(packed, scales, mins):
        p = packed.cpu().numpy()
        codes = np.stack([p & 15, p >> 4], -1).reshape(p.shape[0], -1)
        s, m = (np.repeat(t.cpu().numpy().astype(np.float64), 128, 1) for t in (scales, mins))
        return codes * s + m

    c, _ = ref.rows_of(rows.cpu().numpy(), pool.table[0], length)
    turned = q[0, :, latent:].cpu().numpy().astype(np.float64)
    for h in range(heads):
        k = np.concatenate([c[:, :latent] @ weights(*quantized[0][h]), c[:, latent:]], -1)
        v = c[:, :latent] @ weights(*quantized[1][h]).T
        x = np.concatenate([q_own[h].cpu().numpy().astype(np.float64), turned[h]])
        w = heads_ref.weights(x, k, length - 1, np.ones(length, dtype=bool), scale)
        wv = weights(*quantized[1][h])
        # The query in the latent space is rounded to fp16: scores err by ds, normalised weights by a factor within
        # e^(2 ds) and their own rounding; so is the mixed row before its product with the value weights (fp32 sums,
        # as the query's); below fp16's normal range weights and mixed row err by 2^-25 of the largest value each.
        ds = (H + (own + latent + 72) * U32) * scale * (np.abs(weights(*quantized[0][h]) @ x[:own]) @ np.abs(c[:, :latent]).T).max()
        far = np.abs(c[:, :latent]) @ np.abs(wv).T
        bound = ((np.expm1(2 * ds) + 2 * H + 2 * (latent + 72) * U32) * (1 + 2 * H) * (w @ far)
                 + TINY * (length * far.max(0) + np.abs(wv).sum(1)))
        assert np.all(np.abs(out[h] - w @ v) <= bound), h


def test_binding_refusals(dev):
    f16, i = dict(dtype=torch.float16, device=dev), dict(dtype=torch.int32, device=dev)
    rows, table, n, starts = torch.zeros(4, 16, 192, **f16), torch.zeros(3, 4, **i), torch.ones(3, **i), torch.arange(4, **i)
    pos, kv = torch.zeros(3, **i), torch.zeros(3, 192, device=dev)
    kc, vc = torch.zeros(4, 2, 16, 128, **f16), torch.zeros(4, 2, 64, 16, **f16)
    packed, sm = torch.zeros(256, 64, dtype=torch.uint8, device=dev), torch.zeros(256, 1, **f16)
    calls = {
        "append": (q4.q4g128_latent_append, dict(kv=kv, cache=rows, table=table, positions=pos, inv_freq=None)),
        "keep": (q4.q4g128_latent_keep, dict(cache=rows, table=table, starts=n, keep_starts=starts, keep=pos)),
        "attn": (q4.q4g128_latent_attn, dict(q=torch.zeros(3, 2, 192, **f16), cache=rows, table=table, q_starts=starts,
                                             lengths=n, scale=0.1)),
        "expand": (q4.q4g128_latent_expand, dict(cache=rows, table=table, lengths=n, packed=packed, scales=sm, mins=sm.clone(),
                                                 k_cache=kc, v_cache=vc, expanded_table=table.clone())),
        "prefill": (q4.q4g128_latent_prefill, dict(q=torch.zeros(3, 2, 128, **f16), k_cache=kc, v_cache=vc, table=table,
                                                   q_starts=starts, lengths=n, scale=0.1)),
        "tree": (q4.q4g128_attn_tree, dict(q=torch.zeros(3, 2, 64, **f16), k_cache=torch.zeros(4, 2, 16, 64, **f16),
                                           v_cache=vc, table=table, q_starts=starts, lengths=n)),
    }
    for call, good in calls.values():
        call(**good)
        for name, x in good.items():
            if not isinstance(x, torch.Tensor):
                continue
            for bad, error in ((x.cpu(), (ValueError,)), (x.double(), (TypeError,)), (x[None], (ValueError, q4.Q4Error)),
                               ("x", (TypeError,))):
                with pytest.raises(error):
                    call(**dict(good, **{name: bad}))
    for name, bad, error in (("append", dict(kv=kv[:, :191]), ValueError), ("append", dict(kv=kv.t()), ValueError),
                             ("append", dict(q_main=torch.zeros(3, 2, 64, device=dev)), ValueError),
                             ("append", dict(norm=torch.zeros(64, **f16)), ValueError),
                             ("append", dict(inv_freq=torch.zeros(16, device=dev)), ValueError),
                             ("attn", dict(masks=pos), TypeError), ("attn", dict(lengths=n[:2]), ValueError),
                             ("attn", dict(max_new=0), q4.Q4Error), ("attn", dict(scale=0.0), q4.Q4Error),
                             ("attn", dict(max_length=65), q4.Q4Error), ("attn", dict(workspace=pos), ValueError),
                             ("attn", dict(cache=rows.transpose(1, 2)), ValueError),
                             ("attn", dict(masks=pos.long(), max_new=65), q4.Q4Error),
                             ("keep", dict(keep_starts=starts[:3]), ValueError),
                             ("expand", dict(packed=packed[:128]), ValueError),
                             ("expand", dict(expanded_table=table[:2]), (ValueError, q4.Q4Error)),
                             ("expand", dict(v_cache=kc), ValueError), ("prefill", dict(k_cache=vc), ValueError),
                             ("tree", dict(masks=pos.long()[:2]), ValueError), ("tree", dict(max_new=65), q4.Q4Error)):
        with pytest.raises(error):
            calls[name][0](**dict(calls[name][1], **bad))
    torch.cuda.synchronize()
