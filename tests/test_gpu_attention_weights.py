"""The softmax weights' own arithmetic: what they sum to, and what small ones keep."""
import numpy as np
import pytest

from gpu_helpers import note
from test_gpu_attention import H, TINY, Pool, dev, i32  # noqa: F401  (dev: fixture)

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


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("tokens,many", [(5, False), (5, True), (40, True)])
@pytest.mark.parametrize("low_half", [0, 1])
def test_small_weights_beside_a_jump_of_the_maximum(dev, dim, tokens, many, low_half):  # noqa: F811
    """One half of a tile's keys lies 2^7.75 above the running maximum, the other 2^24.9: the first half's weights,
    2^-17.15 of the largest, stay (weights are rounded to 2^-25 of it), for the output dimensions of either wave
    where two share the rows.  40 tokens beside many empty sequences: the form of 128 rows."""
    rng = np.random.default_rng(dim)
    empty = [0] * (80 if many else 0)
    page, kv = 64, 8 if many else 1
    n = 128 + tokens  # a tile of zeros, the tile with the jump, and the tokens themselves
    score = np.full(n, -60.0)
    score[:64] = 0.0
    half = slice(64, 96) if low_half == 0 else slice(96, 128)
    score[64:128] = 24.9
    score[half] = 7.75
    value = np.zeros((n, dim))
    value[half] = rng.uniform(20000, 60000, (32, dim))
    pool = Pool(rng, [n] + empty, kv, page, dim)
    for j in range(n):
        pool.k[pool.table[0, j // page], :, j % page] = 0
        pool.k[pool.table[0, j // page], :, j % page, 0] = score[j]
        pool.v[pool.table[0, j // page], :, :, j % page] = value[j]
    q = np.zeros((tokens, kv, dim), dtype=np.float16)
    q[:, :, 0] = 1
    scale = np.log(2.0)
    starts = [0] + [tokens] * (len(empty) + 1)
    s = np.float64(score.astype(np.float16))
    v = np.float64(value.astype(np.float16))
    w = 2.0 ** (s[:128] - s[:128].max())  # the tokens' own positions weigh 2^-85
    want = w @ v[:128] / w.sum()
    err = H * want + 2 * H * want + n * TINY * v.max() / w.sum()
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *pool.on(dev), i32(starts, dev), i32([n] + empty, dev),
                                 scale=float(scale)).float().cpu().numpy()
    assert np.all(np.abs(out - want) <= err), (np.abs(out - want) / err).max()
