"""Latent rows and expanded keys and values side by side in the pages of one allocation: the results of pools of their
own, bit by bit, and nothing else written.
"""
import numpy as np
import pytest

from gpu_helpers import device, note
from test_gpu_attention import i32
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


@pytest.mark.parametrize("order", ["rkv", "kvr", "krv"])
@pytest.mark.parametrize("gap", [0, 24])
def test_one_allocation(dev, order, gap):
    rng = np.random.default_rng(1)
    heads, value, latent, page, lengths = 3, 64, 128, 32, [150, 70]
    pool = Rows(rng, lengths, latent, page, junk=1.0)
    weights, _ = quantized(rng, heads * 2 * value, latent, dev)
    rows, table = pool.on(dev)
    own = dict(r=rows)
    own["k"], own["v"], _ = (torch.from_numpy(a).to(dev) for a in target(rng, lengths, heads, value, page))
    width = gap + sum(own[c][0].numel() for c in order)
    whole = torch.full((pool.pages, width), 3.0, dtype=torch.float16, device=dev)
    parts, at = {}, gap
    for c in order:
        size = own[c][0].numel()
        parts[c] = whole[:, at:at + size].view(own[c].shape)
        parts[c].copy_(own[c])
        at += size
    n = i32(lengths, dev)
    for p in (own, parts):
        q4.q4g128_latent_expand(p["r"], table, n, *weights, p["k"], p["v"], table)
    for c in order:
        assert torch.equal(parts[c].contiguous().view(torch.int16), own[c].view(torch.int16)), c
    assert torch.all(whole[:, :gap] == 3.0)
    q = torch.from_numpy(rng.standard_normal((9, heads, value + ROT)).astype(np.float16)).to(dev)
    args = (table, i32([0, 5, 9], dev), n, 0.1)
    assert torch.equal(q4.q4g128_latent_prefill(q, parts["k"], parts["v"], *args),
                       q4.q4g128_latent_prefill(q, own["k"], own["v"], *args))
