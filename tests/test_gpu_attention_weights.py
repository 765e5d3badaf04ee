"""The softmax weights' own arithmetic: what they sum to."""
import numpy as np
import pytest

from gpu_helpers import note
from test_gpu_attention import Pool, dev, i32  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("value", [1.0, -1.3330078125, 65504.0])
@pytest.mark.parametrize("lengths", [[1, 5, 60], [300, 64, 2000]])
def test_equal_values_come_back(dev, dim, value, lengths):  # noqa: F811
    """The mean of equal values is that value.  The weights are fp16 numbers and are summed as such, so what
    remains are fp32 roundings, (n + 64) 2^-24 < 2^-12 of the value: less than half a step of fp16."""
    rng = np.random.default_rng(dim)
    pool = Pool(rng, lengths, 2, 64, dim, junk=None)
    pool.v[:] = value
    q = rng.standard_normal((len(lengths), 6, dim)).astype(np.float16)
    qd, c, n = torch.from_numpy(q).to(dev), pool.on(dev), i32(lengths, dev)
    for out in (q4.q4g128_attn_decode(qd, *c, n),
                q4.q4g128_attn_prefill(qd, *c, i32(range(len(lengths) + 1), dev), n)):
        assert torch.all(out == np.float16(value)), (out.float() - value).abs().max()


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("value", [1.0, -1.3330078125, 65504.0])
@pytest.mark.parametrize("off", [0.9, 1.1])
@pytest.mark.parametrize("length", [64, 700])
def test_equal_values_under_weights_rounded_alike(dev, dim, value, off, length):  # noqa: F811
    """All weights but one are 1/2 + off * 2^-12 of the largest, between two fp16 numbers 2^-11 apart: all of them
    are rounded the same way, by nearly 2^-11 of themselves.  The mean of equal values stays that value."""
    pool = Pool(np.random.default_rng(dim), [length], 2, 64, dim, junk=None)
    pool.k[:] = 0
    pool.v[:] = value
    for j in range(length):
        if j != 7:
            p = pool.table[0, j // 64]
            pool.k[p, :, j % 64, 0] = -1
            pool.k[p, :, j % 64, 1] = 2.0 ** 10 * (np.log2(0.5 + off * 2.0 ** -12) + 1)
    q = np.zeros((1, 4, dim), dtype=np.float16)
    q[:, :, 0], q[:, :, 1] = 1, 2.0 ** -10
    qd, c, n = torch.from_numpy(q).to(dev), pool.on(dev), i32([length], dev)
    for out in (q4.q4g128_attn_decode(qd, *c, n, scale=float(np.log(2.0))),
                q4.q4g128_attn_prefill(qd, *c, i32([0, 1], dev), n, scale=float(np.log(2.0)))):
        assert torch.all(out == np.float16(value)), (out.float() - value).abs().max()
