"""Scores far beyond the weights' range, of either sign: the best position takes all.

Queries are +-2^14 and keys 2^12 times whole numbers up to 7, so that every product and sum is exact in fp32 (a whole
number below 2^24 times 2^26) and two different scores are at least 2^26 apart: 2^26 log2(e) of them in base 2, where a
rounding of the largest (below 2^39) is 2^14 at most.  All weights but the best ones' are 0, those are equal, and the
result is their values' mean, rounded once: |out - ref| <= 2^-11 |ref| + 2^-25.
"""
import numpy as np
import pytest

from gpu_helpers import device, note
from oracle import latent as lref
from test_gpu_attention import H, TINY, Pool, i32
from test_gpu_drafts import check as check_heads
from test_gpu_drafts import trees
from test_gpu_latent import ROT, Rows
from test_gpu_latent import check as check_latent
from test_gpu_latent_expanded import target

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


def queries(rng, shape):
    return (16384.0 * rng.choice([-1, 1], shape)).astype(np.float16)


def keys(rng, n, width, sign, q):
    """[n][width]; position 3 n / 4 has the middle one's, whose scores therefore tie.  sign: of all scores with query q (0:
    either)."""
    k = rng.integers(-7, 8, (n, width)).astype(np.float64)
    if sign:
        k = sign * np.abs(k) * np.sign(q.astype(np.float64))
    k[3 * n // 4] = k[n // 2]
    return (4096.0 * k).astype(np.float16)


def close(got, k, v, q, sees):
    """One token and head: its result against the mean of the best positions' values."""
    s = k.astype(np.float64) @ q.astype(np.float64)
    s[~sees] = -np.inf
    want = v[s == s.max()].astype(np.float64).mean(0)
    return np.all(np.abs(got.astype(np.float64) - want) <= H * np.abs(want) + TINY)


def filled(rng, length, kv, dim, page, sign, q):
    """A cache of one sequence, as kept and as rows [kv][length][dim]; q: the query that signs go by."""
    pool = Pool(rng, [length], kv, page, dim)
    k = np.stack([keys(rng, length, dim, sign, q) for _ in range(kv)])
    v = rng.standard_normal((kv, length, dim)).astype(np.float16)
    for j in range(length):
        p = pool.table[0, j // page]
        pool.k[p, :, j % page], pool.v[p, :, :, j % page] = k[:, j], v[:, j]
    return pool, k, v


# 64 rows a workgroup whole and split, 128 rows, and two waves to the same rows at 192 and 256.
@pytest.mark.parametrize("dim,tokens,length,heads,kv", [(64, 40, 150, 4, 2), (128, 3, 4000, 4, 2), (96, 60, 200, 4, 2),
                                                        (128, 70, 130, 130, 65), (192, 40, 170, 4, 2), (256, 9, 200, 3, 1),
                                                        (256, 70, 130, 260, 130)])
@pytest.mark.parametrize("sign", [0, 1, -1])
@pytest.mark.parametrize("call", ["prompt", "tree", "decode"])
def test_heads(dev, dim, tokens, length, heads, kv, sign, call):
    rng = np.random.default_rng(dim + tokens + sign)
    tokens = 1 if call == "decode" else min(tokens, 64) if call == "tree" else tokens
    q = queries(rng, (tokens, heads, dim))
    q[:] = q[:1, :1] if sign else q
    pool, k, v = filled(rng, length, kv, dim, 64, sign, q[0, 0])
    base = length - tokens
    t, n, starts = torch.from_numpy(q).to(dev), i32([length], dev), i32([0, tokens], dev)
    masks = trees(rng, [tokens]) if call == "tree" else None
    if call == "decode":
        out = q4.q4g128_attn_decode(t, *pool.on(dev), n, scale=1.0)
    elif call == "tree":
        out = q4.q4g128_attn_tree(t, *pool.on(dev), starts, n, torch.from_numpy(masks).to(dev), scale=1.0)
    else:
        out = q4.q4g128_attn_prefill(t, *pool.on(dev), starts, n, scale=1.0)
    out = out.float().cpu().numpy()
    assert np.all(np.isfinite(out))
    for i in range(tokens):
        sees = np.arange(length) <= base + i
        if masks is not None:
            sees[base:] = (int(masks[i]) % (1 << 64)) >> np.arange(tokens, dtype=object) & 1 != 0
        for h in sorted({0, 1 % heads, heads // 2, heads - 1}):
            g = h // (heads // kv)
            assert close(out[i, h], k[g], v[g], q[i, h], sees), (i, h)


@pytest.mark.parametrize("latent", [128, 512])
@pytest.mark.parametrize("heads", [4, 20, 40, 130])
@pytest.mark.parametrize("length", [50, 700])
@pytest.mark.parametrize("sign", [0, 1, -1])
def test_latent_rows(dev, latent, heads, length, sign):
    rng = np.random.default_rng(latent + heads + sign)
    pool = Rows(rng, [length], latent, 64)
    q = queries(rng, (2, heads, latent + ROT))
    q[:] = q[:1, :1] if sign else q
    c = keys(rng, length, latent + ROT, sign, q[0, 0])
    for j in range(length):
        pool.rows[pool.table[0, j // 64], j % 64] = c[j]
    out = q4.q4g128_latent_attn(torch.from_numpy(q).to(dev), *pool.on(dev), i32([0, 2], dev), i32([length], dev),
                                1.0).float().cpu().numpy()
    assert np.all(np.isfinite(out))
    for i in range(2):
        for h in range(heads):
            assert close(out[i, h], c, c[:, :latent], q[i, h], np.arange(length) <= length - 2 + i), (i, h)


@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("tokens,length,heads", [(40, 150, 2), (3, 3000, 1), (40, 60, 260)])
@pytest.mark.parametrize("sign", [0, 1, -1])
def test_expanded_rows(dev, value, tokens, length, heads, sign):
    rng = np.random.default_rng(value + tokens + sign)
    k, v, table = target(rng, [length], heads, value, 64)
    q = queries(rng, (tokens, heads, value + ROT))
    q[:] = q[:1, :1] if sign else q
    ks = np.stack([keys(rng, length, value + ROT, sign, q[0, 0]) for _ in range(heads)])
    vs = rng.standard_normal((heads, length, value)).astype(np.float16)
    for j in range(length):
        p, o = lref.slot(table, 0, j, 64, len(k))
        k[p, :, o], v[p, :, :, o] = ks[:, j], vs[:, j]
    out = q4.q4g128_latent_prefill(torch.from_numpy(q).to(dev), *(torch.from_numpy(a).to(dev) for a in (k, v, table)),
                                   i32([0, tokens], dev), i32([length], dev), 1.0).float().cpu().numpy()
    assert np.all(np.isfinite(out))
    for i in range(tokens):
        for h in sorted({0, heads // 2, heads - 1}):
            assert close(out[i, h], ks[h], vs[h], q[i, h], np.arange(length) <= length - tokens + i), (i, h)


# Scores of 2^33 to 2^18 in base 2, on either side of where the kernels take another way (2^26).
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -4, 2.0 ** -6, 2.0 ** -7, 2.0 ** -8, 2.0 ** -9, 2.0 ** -15])
@pytest.mark.parametrize("sign", [0, 1, -1])
def test_any_size_of_scores(dev, scale, sign):
    rng = np.random.default_rng(7 + sign)
    length, latent, dim = 330, 128, 64
    q = queries(rng, (2, 20, latent + ROT))
    q[:] = q[:1, :1] if sign else q
    rows = Rows(rng, [length], latent, 64)
    c = keys(rng, length, latent + ROT, sign, q[0, 0])
    for j in range(length):
        rows.rows[rows.table[0, j // 64], j % 64] = c[j]
    starts, n = i32([0, 2], dev), i32([length], dev)
    for heads in (3, 20):
        out = q4.q4g128_latent_attn(torch.from_numpy(q[:, :heads].copy()).to(dev), *rows.on(dev), starts, n,
                                    scale).float().cpu().numpy()
        for i in range(2):
            for h in range(heads):
                assert close(out[i, h], c, c[:, :latent], q[i, h], np.arange(length) <= length - 2 + i), (heads, i, h)
    pool, k, v = filled(rng, length, 1, dim, 64, sign, q[0, 0, :dim])
    q = q[:, :, :dim].copy()
    out = q4.q4g128_attn_prefill(torch.from_numpy(q).to(dev), *pool.on(dev), starts, n, scale=scale).float().cpu().numpy()
    for i in range(2):
        for h in range(20):
            assert close(out[i, h], k[0], v[0], q[i, h], np.arange(length) <= length - 2 + i), (i, h)


@pytest.mark.parametrize("heads", [4, 20, 40])
@pytest.mark.parametrize("length", [90, 3000])
def test_far_rows_beside_others(dev, heads, length):
    """Rows of one workgroup, every third far: the others stay within their bounds.  The far ones' queries are 2^28 times the
    others'."""
    rng = np.random.default_rng(heads)
    latent, dim, scale = 128, 64, 2.0 ** -7
    far = np.arange(heads) % 3 == 0
    size = np.where(far, 1.0, 2.0 ** -28)[None, :, None]
    rows = Rows(rng, [length], latent, 64)
    c = keys(rng, length, latent + ROT, 0, None)
    for j in range(length):
        rows.rows[rows.table[0, j // 64], j % 64] = c[j]
    starts, n = i32([0, 2], dev), i32([length], dev)
    q = (queries(rng, (2, heads, latent + ROT)) * size).astype(np.float16)
    out = q4.q4g128_latent_attn(torch.from_numpy(q).to(dev), *rows.on(dev), starts, n, scale)
    check_latent(out[:, ~far], q[:, ~far], rows, [0, 2], [length], scale, None, "beside far rows")
    got = out.float().cpu().numpy()
    pool, k, v = filled(rng, length, 1, dim, 64, 0, None)
    qh = q[:, :, :dim].copy()
    out = q4.q4g128_attn_prefill(torch.from_numpy(qh).to(dev), *pool.on(dev), starts, n, scale=scale)
    check_heads(out[:, ~far], qh[:, ~far], pool, [0, 2], [length], scale, None, "beside far rows")
    out = out.float().cpu().numpy()
    for i in range(2):
        sees = np.arange(length) <= length - 2 + i
        for h in np.flatnonzero(far):
            assert close(got[i, h], c, c[:, :latent], q[i, h], sees) and close(out[i, h], k[0], v[0], qh[i, h], sees), (i, h)
