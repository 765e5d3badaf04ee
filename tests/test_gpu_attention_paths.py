"""Forms of the cache and attention kernels that only larger calls take: wide groups
of values in the append, table entries beyond the 64 that a workgroup of the prompt
kernel holds, and launches beyond one dimension of a grid.
"""
import numpy as np
import pytest

from oracle import attention as ref
from gpu_helpers import U32, note
from test_gpu_attention import H, TINY, Pool, check_append, dev, i32, run_of  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


# ---------------------------------------------------------------------------
# append: values of 64, 32 or 16 tokens together, from 256 workgroups on
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,kv,page,together", [(300, 64, 16, 64), (260, 64, 64, 64), (200, 40, 16, 32),
                                                     (150, 64, 64, 32), (131, 32, 16, 16), (70, 64, 64, 16)])
@pytest.mark.parametrize("start", [0, 3, 7])
def test_append_values_together(dev, tokens, kv, page, together, start):  # noqa: F811
    """As many tokens together as give 256 workgroups of values: aligned and unaligned runs, across pages, with a
    ragged tail."""
    wide = 64
    while wide > 8 and -(-tokens // wide) * kv < 256:
        wide //= 2
    assert wide == together
    check_append(dev, np.random.default_rng(tokens + start), run_of(0, start, tokens), kv, kv, 64, page, 0)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_append_values_of_several_sequences_together(dev, dim):  # noqa: F811
    """64 tokens together that belong to several sequences, some of them on absent pages or without a place."""
    rng = np.random.default_rng(dim)
    placed = (run_of(0, 5, 37) + run_of(1, 16, 24) + run_of(3, 0, 3) + run_of(2, 9, 61) + [(4, 40), (-1, 0), (2, 1 << 20)] +
              run_of(1, 40, 80) + run_of(4, 47, 60))
    assert -(-len(placed) // 64) * 64 >= 256
    check_append(dev, rng, placed, 64, 64, dim, 16, 0, seqs=5, cols=8, absent=[(0, 1), (2, 2), (4, 3), (1, 7)])


# ---------------------------------------------------------------------------
# prompt: more than 64 table entries per workgroup
# ---------------------------------------------------------------------------

def check_rows(got, q, pool, starts, lengths, scale, rows):
    """Some rows of the prompt call, each against the oracle as a prompt of one token."""
    for s, t in rows:
        n = lengths[s] - (starts[s + 1] - starts[s]) + t + 1  # what this token's sequence holds up to it
        at = starts[s] + t
        want, mag, dots = ref.attention(q[at:at + 1], pool.k, pool.v, pool.table[s:s + 1], [0, 1], [n], scale)
        ds = (q.shape[2] + 8) * U32 * scale * dots
        vmax = np.abs(pool.v[np.isfinite(pool.v)]).max()
        bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[..., None] * mag + n * TINY * vmax * (mag > 0)
        err = np.abs(got[at:at + 1].float().cpu().numpy().astype(np.float64) - want)
        assert np.all(err <= bound), f"sequence {s}, token {t}: worst {(err / bound).max():.3f} of the bound"


@pytest.mark.parametrize("page,past", [(16, 0), (16, 1500), (32, 1900), (64, 4300)])
@pytest.mark.parametrize("several", [False, True])
def test_prompt_walks_many_pages(dev, page, past, several):  # noqa: F811
    """A workgroup of the last tokens walks 66 to more than 128 table entries, which it holds 64 at a time; the page
    after the first 64 is absent.  1,100 tokens of 32 heads are enough workgroups to leave the positions whole."""
    rng = np.random.default_rng(page + past)
    new = [1100, 40] if several else [1100]
    lengths = [1100 + past, 70] if several else [1100 + past]
    assert lengths[0] > 64 * page
    heads, kv, dim, scale = 32, 32, 64, 0.2
    assert q4.q4g128_attn_prefill_workspace(sum(new), len(new), heads, kv, dim, max(lengths)) == 0
    pool = Pool(rng, lengths, kv, page, dim, absent=[(0, 64)])
    starts = [0] + [int(x) for x in np.cumsum(new)]
    q = rng.standard_normal((starts[-1], heads, dim)).astype(np.float16)
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32(lengths, dev),
                                 scale=scale, max_length=max(lengths))
    assert torch.isfinite(out).all()
    rows = [(0, t) for t in (0, 500, 1090, 1099)] + ([(1, 0), (1, 39)] if several else [])
    check_rows(out, q, pool, starts, lengths, scale, rows)


# ---------------------------------------------------------------------------
# launches beyond one dimension of a grid
# ---------------------------------------------------------------------------

def test_decode_of_more_parts_than_a_grid_dimension(dev):  # noqa: F811
    """33,000 sequences, which share their pages: parts beyond the 32,768th lie in the grid's third dimension."""
    rng = np.random.default_rng(1)
    b, page, dim = 33000, 16, 64
    pool = Pool(rng, [160], 1, page, dim, junk=None)
    lengths = rng.integers(0, 161, b).astype(np.int32)
    table = np.broadcast_to(pool.table[0], (b, pool.table.shape[1]))
    q = rng.standard_normal((b, 2, dim)).astype(np.float16)
    k, v, _ = pool.on(dev)
    out = q4.q4g128_attn_decode(torch.from_numpy(q).to(dev), k, v, torch.from_numpy(table.copy()).to(dev),
                                i32(lengths, dev), scale=0.2)
    assert torch.isfinite(out).all()
    for s in [0, 1, 511, 16000, 32255, 32256, 32767, 32768, 32769, 32999] + [int(x) for x in rng.integers(32000, b, 10)]:
        n = int(lengths[s])
        want, mag, dots = ref.attention(q[s:s + 1], pool.k, pool.v, pool.table, [0, 1], [n], 0.2)
        ds = (dim + 8) * U32 * 0.2 * dots
        bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[..., None] * mag + 160 * TINY * 8 * (mag > 0)
        assert np.all(np.abs(out[s:s + 1].float().cpu().numpy() - want) <= bound), (s, n)


def test_prompt_of_more_tiles_than_a_grid_dimension(dev):  # noqa: F811
    """65,536 sequences of one to 140 tokens, which share their pages: more than 65,535 tiles take two launches."""
    rng = np.random.default_rng(2)
    count, page, dim = 65536, 64, 64
    new = np.ones(count, dtype=np.int64)
    new[[0, 7, 40000, 65000, 65535]] = [129, 140, 64, 130, 135]
    starts = np.concatenate([[0], np.cumsum(new)])
    past = rng.integers(0, 60, count)
    lengths = (new + past).astype(np.int32)
    pool = Pool(rng, [int(lengths.max())], 1, page, dim, junk=None)
    table = np.broadcast_to(pool.table[0], (count, pool.table.shape[1]))
    assert np.sum(-(-new // 128)) > 65535
    q = rng.standard_normal((int(starts[-1]), 1, dim)).astype(np.float16)
    k, v, _ = pool.on(dev)
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), k, v, torch.from_numpy(table.copy()).to(dev),
                                 i32(starts, dev), i32(lengths, dev), scale=0.2)
    assert torch.isfinite(out).all()
    shared = Pool.__new__(Pool)
    shared.k, shared.v, shared.table = pool.k, pool.v, table
    rows = [(0, 0), (0, 128), (7, 139), (1, 0), (40000, 63), (65000, 129), (65000, 0), (65534, 0), (65535, 0), (65535, 134)]
    check_rows(out, q, shared, starts, lengths, 0.2, rows)
