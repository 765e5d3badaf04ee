"""Workgroups of the latent kernels that walk more table entries than the 64 they hold at a time: attention over a whole
sequence or a long part of it in every height of workgroup, and expansion of many tiles, with small pages on either
side and an absent page behind the first 64.  Sequences share pages, so the caches stay small.

Bounds as in test_gpu_latent.py and test_gpu_latent_expanded.py.
"""
import numpy as np
import pytest

from gpu_helpers import U32, device, note
from test_gpu_attention import H, TINY, i32
from test_gpu_latent import ROT
from test_gpu_latent_expanded import quantized

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


def held(rows, entries, page, length):
    """The rows of positions 0 .. length - 1, float64, and whether they have a page."""
    j = np.arange(length)
    p = entries[j // page]
    return rows[np.clip(p, 0, len(rows) - 1), j % page].astype(np.float64), (p >= 0) & (p < len(rows))


def attn_walk(dev, seed, heads, lengths, latent, page, max_new, absent, checked):
    """One token per sequence; those of `checked` are compared."""
    rng = np.random.default_rng(seed)
    pages, scale, count = 150, 0.06, len(lengths)
    rows = rng.standard_normal((pages, page, latent + ROT)).astype(np.float16)
    table = rng.integers(0, pages, (count, -(-max(lengths) // page))).astype(np.int32)
    table[:, absent] = -1
    q = rng.standard_normal((count, heads, latent + ROT)).astype(np.float16)
    out = q4.q4g128_latent_attn(torch.from_numpy(q).to(dev), torch.from_numpy(rows).to(dev), torch.from_numpy(table).to(dev),
                                i32(range(count + 1), dev), i32(lengths, dev), scale,
                                max_new=max_new).float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(out))
    for s in checked:
        n = lengths[s]
        c, there = held(rows, table[s], page, n)
        x = q[s].astype(np.float64)
        w = scale * (x @ c.T)
        w[:, ~there] = -np.inf
        w = np.exp(w - w.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        want, mag = w @ c[:, :latent], w @ np.abs(c[:, :latent])
        dots = (np.abs(x) @ np.abs(c[there]).T).max(1)
        ds = (latent + 72) * U32 * scale * dots
        bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[:, None] * mag + n * TINY * np.abs(c).max()
        err = np.abs(out[s] - want)
        assert np.all(err <= bound), f"sequence {s}: worst {(err / bound).max():.3f} of the bound"


@pytest.mark.parametrize("page,length", [(16, 4700), (32, 4700), (64, 9000)])
@pytest.mark.parametrize("latent", [128, 512])
def test_attention_of_one_sequence_in_one_part(dev, page, length, latent):
    """A bound of 200 new tokens of 64 heads asks for one part per row block."""
    attn_walk(dev, 1, 64, [length], latent, page, 200, [64, 65], [0])


@pytest.mark.parametrize("heads", [5, 20])
@pytest.mark.parametrize("page", [16, 32])
def test_attention_of_one_sequence_in_long_parts(dev, heads, page):
    """256 parts of 23 tiles or 41, which begin anywhere in the table."""
    attn_walk(dev, 2, heads, [256 * 64 * (23 if page == 16 else 41) - 100], 128, page, 1, [64, 70, 5000], [0])


@pytest.mark.parametrize("heads", [5, 20, 40])
@pytest.mark.parametrize("page,length", [(16, 1700), (32, 2900)])
def test_attention_of_many_sequences(dev, heads, page, length):
    """More tiles than parts, so that most sequences are walked whole."""
    lengths = [length + 13 * i % 300 for i in range(300)]
    attn_walk(dev, 3, heads, lengths, 128, page, 1, [64], [0, 1, 63, 64, 150, 299])


@pytest.mark.parametrize("page,to_page", [(16, 16), (16, 64), (64, 16), (32, 256), (256, 32)])
@pytest.mark.parametrize("lengths,firsts", [([1500], None), ([2300], [300]), ([1500, 30, 1290], None)])
def test_expansion(dev, page, to_page, lengths, firsts):
    """300 heads leave one workgroup per head, which walks all tiles."""
    rng = np.random.default_rng(4)
    heads, value, latent, pages, count = 300, 64, 128, 60, len(lengths)
    rows = rng.standard_normal((pages, page, latent + ROT)).astype(np.float16)
    table = rng.integers(0, pages, (count, -(-max(lengths) // page))).astype(np.int32)
    used = [-(-n // to_page) for n in lengths]
    order = rng.permutation(sum(used) + 1)
    to = np.full((count, max(used)), -1, np.int32)
    at = 0
    for s, n in enumerate(used):
        to[s, :n] = order[at:at + n]
        at += n
    for t in (table, to):
        if t.shape[1] > 64:
            t[0, 64] = -1
    weights, w = quantized(rng, heads * 2 * value, latent, dev)
    w = w.reshape(heads, 2, value, latent)
    k = torch.full((len(order), heads, to_page, value + ROT), 7.0, dtype=torch.float16, device=dev)
    v = torch.full((len(order), heads, value, to_page), 7.0, dtype=torch.float16, device=dev)
    q4.q4g128_latent_expand(torch.from_numpy(rows).to(dev), torch.from_numpy(table).to(dev), i32(lengths, dev), *weights, k, v,
                            torch.from_numpy(to).to(dev), firsts=None if firsts is None else i32(firsts, dev))
    picked = [0, 1, 2, 77, 150, 298, 299]
    got_k, got_v = k[:, picked].cpu().numpy().astype(np.float64), v[:, picked].cpu().numpy().astype(np.float64)
    written = np.zeros((len(order), to_page), dtype=bool)
    for s, n in enumerate(lengths):
        c, there = held(rows, table[s], page, n)
        j = np.arange(firsts[s] if firsts else 0, n)
        j = j[there[j] & (to[s, j // to_page] >= 0)]
        p, o = to[s, j // to_page], j % to_page
        written[p, o] = True
        x = c[j, :latent]
        for i, h in enumerate(picked):
            for got, wh in ((got_k[p, i, o, :value], w[h, 0]), (got_v[p, i, :, o], w[h, 1])):
                want, mag = x @ wh.T, np.abs(x) @ np.abs(wh).T
                err = np.abs(got - want)
                assert np.all(err <= H * np.abs(want) + TINY + (latent + 8) * U32 * mag), (s, h, err.max())
            assert np.array_equal(got_k[p, i, o, value:], c[j, latent:]), (s, h)
    left = torch.from_numpy(~written).to(dev)
    assert torch.all(k.transpose(1, 2)[left] == 7.0) and torch.all(v.permute(0, 3, 1, 2)[left] == 7.0)
