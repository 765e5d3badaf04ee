"""Caches given as views: sizes of one have no next element, so their strides mean nothing."""
import numpy as np
import pytest

from gpu_helpers import note
from test_gpu_attention import dev, i32  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


def one_head_views(pages, page, dim, dev):  # noqa: F811
    """Contiguous pages of one kv head whose head strides are those of a transposition."""
    k = torch.zeros((pages, page, 1, dim), dtype=torch.float16, device=dev).transpose(1, 2)
    v = torch.zeros((pages, dim, 1, page), dtype=torch.float16, device=dev).transpose(1, 2)
    return k, v


def one_page_views(page, dim, dev):  # noqa: F811
    """One page of two kv heads whose page stride is zero."""
    k = torch.zeros((2, page, dim), dtype=torch.float16, device=dev).expand(1, 2, page, dim)
    v = torch.zeros((2, dim, page), dtype=torch.float16, device=dev).expand(1, 2, dim, page)
    return k, v.as_strided(v.shape, (0,) + v.stride()[1:])


@pytest.mark.parametrize("kind", ["one head", "one page"])
def test_strides_of_sizes_of_one(dev, kind):  # noqa: F811
    rng = np.random.default_rng(1)
    page, dim, n = 32, 64, 30
    k, v = one_head_views(3, page, dim, dev) if kind == "one head" else one_page_views(page, dim, dev)
    kv = k.shape[1]
    assert k.is_contiguous() and v.is_contiguous()
    plain_k, plain_v = torch.zeros(k.shape, dtype=k.dtype, device=dev), torch.zeros(v.shape, dtype=v.dtype, device=dev)
    qkv = torch.from_numpy(rng.standard_normal((n, (4 + 2 * kv) * dim)).astype(np.float32)).to(dev)
    table, pos, seq = i32([[0]], dev), i32(range(n), dev), i32([0] * n, dev)
    got = []
    for c in ((k, v), (plain_k, plain_v)):
        q = q4.q4g128_rope_append(qkv, *c, table, pos, None, 4, seq=seq)
        got.append((q, q4.q4g128_attn_prefill(q, *c, table, i32([0, n], dev), i32([n], dev)),
                    q4.q4g128_attn_decode(q[-1:], *c, table, i32([n], dev))))
    assert torch.equal(k, plain_k) and torch.equal(v, plain_v)
    assert all(torch.equal(a, b) for a, b in zip(*got))
