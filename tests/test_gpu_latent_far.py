"""Pages far apart in memory: offsets past 32 bits, in bytes and in elements, give the results of a dense pool, bit by bit."""
import numpy as np
import pytest

from gpu_helpers import device, note
from test_gpu_attention import i32
from test_gpu_drafts import trees
from test_gpu_latent import ROT, Rows
from test_gpu_latent_expanded import quantized, target

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


def far(dense, stride=3 * 10 ** 8):
    """The same pages, `stride` elements from one to the next."""
    pool = torch.empty((dense.shape[0] - 1) * stride + dense[0].numel(), dtype=dense.dtype, device=dense.device)
    wide = pool.as_strided(dense.shape, (stride,) + dense.stride()[1:])
    wide.copy_(dense)
    return wide


def same(a, b):
    return torch.equal(a.view(torch.int16), b.contiguous().view(torch.int16))


def test_latent_rows(dev):
    rng = np.random.default_rng(1)
    pool = Rows(rng, [300, 200], 256, 64, junk=1.0)
    rows, table = pool.on(dev)
    wide = far(rows)
    new = [5, 3]
    masks = torch.from_numpy(trees(rng, new)).to(dev)
    for heads in (2, 12, 40):
        q = torch.from_numpy(rng.standard_normal((8, heads, 256 + ROT)).astype(np.float16)).to(dev)
        args = (table, i32([0, 5, 8], dev), i32([300, 200], dev), 0.06)
        assert same(q4.q4g128_latent_attn(q, rows, *args, masks=masks), q4.q4g128_latent_attn(q, wide, *args, masks=masks))
    kv = torch.from_numpy(rng.standard_normal((3, 256 + ROT)).astype(np.float32)).to(dev)
    for r in (rows, wide):
        q4.q4g128_latent_append(kv, r, table, i32([10, 290, 199], dev), None, seq=i32([0, 0, 1], dev))
        q4.q4g128_latent_keep(r, table, i32([60, 3], dev), i32([0, 4, 6], dev), i32([0, 2, 70, 200, 1, 190], dev))
    assert same(rows, wide)


def test_expanded_rows(dev):
    rng = np.random.default_rng(2)
    heads, lengths = 3, [300, 200]
    pool = Rows(rng, lengths, 128, 64, junk=1.0)
    rows, table = pool.on(dev)
    weights, _ = quantized(rng, heads * 2 * 64, 128, dev)
    k, v, to = (torch.from_numpy(a).to(dev) for a in target(rng, lengths, heads, 64, 64))
    n = i32(lengths, dev)
    far_k, far_v = far(k), far(v)
    q4.q4g128_latent_expand(rows, table, n, *weights, k, v, to)
    q4.q4g128_latent_expand(far(rows), table, n, *weights, far_k, far_v, to)
    assert same(k, far_k) and same(v, far_v)
    q = torch.from_numpy(rng.standard_normal((9, heads, 64 + ROT)).astype(np.float16)).to(dev)
    args = (to, i32([0, 5, 9], dev), n, 0.1)
    assert same(q4.q4g128_latent_prefill(q, k, v, *args), q4.q4g128_latent_prefill(q, far_k, far_v, *args))


def test_drafted_tokens(dev):
    rng = np.random.default_rng(3)
    k = torch.from_numpy(rng.standard_normal((9, 2, 64, 128)).astype(np.float16)).to(dev)
    v = torch.from_numpy(rng.standard_normal((9, 2, 128, 64)).astype(np.float16)).to(dev)
    far_k, far_v, table = far(k), far(v), i32([[8, 1, 6, 3, 0], [2, 7, 4, 5, -1]], dev)
    masks = torch.from_numpy(trees(rng, [5, 3])).to(dev)
    q = torch.from_numpy(rng.standard_normal((8, 6, 128)).astype(np.float16)).to(dev)
    args = (table, i32([0, 5, 8], dev), i32([300, 200], dev), masks)
    assert same(q4.q4g128_attn_tree(q, k, v, *args), q4.q4g128_attn_tree(q, far_k, far_v, *args))
    for a, b in ((k, v), (far_k, far_v)):
        q4.q4g128_cache_keep(a, b, table, i32([60, 3], dev), i32([0, 4, 6], dev), i32([0, 2, 70, 200, 1, 190], dev))
    assert same(k, far_k) and same(v, far_v)
