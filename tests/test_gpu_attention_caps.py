"""Capped scores over the whole range of caps: softcap * tanh(s / softcap) has an
error relative to s, so a cap far above the scores leaves them as they are.

The bound is that of test_gpu_attention.py with the cap's term relative to the
scores.  tanh's error is about three roundings of 2^-23 where it is formed as
1 - 2 / (e^2x + 1), which it is from |x| = 0.114 on, so 26 * 2^-23 < 2^-18 of
it there; below, the series up to x^5 is off by less than 2^-22 of it.
"""
import numpy as np
import pytest

from oracle import attention as ref
from gpu_helpers import U32, note
from test_gpu_attention import H, TINY, Pool, dev, i32  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _announce(request):
    note(f"[gpu-test] {request.node.nodeid}")
    yield


def check(got, q, pool, starts, lengths, scale, softcap, slopes=None):
    want, mag, dots = ref.attention(q, pool.k, pool.v, pool.table, starts, lengths, scale, softcap, 0, slopes)
    n = max(lengths)
    ds = ((q.shape[2] + 8) * U32 + 2.0 ** -18) * scale * dots
    if slopes is not None:
        ds = ds + 2.0 ** -22 * n * np.abs(slopes)[None]
    vmax = np.abs(pool.v[np.isfinite(pool.v)]).max()
    bound = H * np.abs(want) + TINY + (H + 2 * ds + (n + 64) * U32)[..., None] * mag + n * TINY * vmax * (mag > 0)
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= bound), f"softcap {softcap}: worst {(err / bound).max():.3f} of the bound"


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 0.5, 4.0, 30.0, 1e3, 1e5, 1e6, 1e12, 3e38])
@pytest.mark.parametrize("slopes", [False, True])
def test_caps(dev, dim, softcap, slopes):  # noqa: F811
    rng = np.random.default_rng(dim)
    lengths, new, heads, kv = [150, 70], [40, 70], 4, 2
    pool = Pool(rng, lengths, kv, 32, dim)
    # a key of zeros: its score is zero under every cap
    pool.k[pool.table[0, 0], :, 3] = 0
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(starts[-1]), heads, dim)).astype(np.float16)
    slope = np.linspace(0.4, 0.01, heads).astype(np.float32) if slopes else None
    sd = None if slope is None else torch.from_numpy(slope).to(dev)
    scale = dim ** -0.5 * 3
    c, n = pool.on(dev), i32(lengths, dev)
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *c, i32(starts, dev), n, scale=scale, softcap=softcap,
                                 slopes=sd)
    check(out, q, pool, starts, lengths, scale, softcap, slope)
    last = np.ascontiguousarray(q[starts[1:] - 1])
    out = q4.q4g128_attn_decode(torch.from_numpy(last).to(dev), *c, n, scale=scale, softcap=softcap, slopes=sd)
    check(out, last, pool, [0, 1, 2], lengths, scale, softcap, slope)
