"""Infinities and NaN in positions of an expanded cache that a sequence holds and most of its tokens do not see: they reach
the tokens that see them and no other.  Every form of the prompt call with keys wider than values: 64 and 128 rows a
workgroup, whole and split over the positions.

Bound of the other tokens as in test_gpu_latent_expanded.py.
"""
import numpy as np
import pytest

from gpu_helpers import U32, device, note
from oracle import latent as ref
from test_gpu_attention import H, TINY, i32
from test_gpu_latent import ROT
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


def check(got, q, k, v, base, scale, what):
    """One sequence: got, q [n][heads][...], its keys and values [positions][heads][...], token i sees positions up to
    base + i."""
    k, v, q = k.astype(np.float64), v.astype(np.float64), q.astype(np.float64)
    positions = base + len(q)
    for i in range(len(q)):
        n = base + i + 1
        s = scale * np.einsum("jhd,hd->hj", k[:n], q[i])
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        want, mag = np.einsum("hj,jhd->hd", w, v[:n]), np.einsum("hj,jhd->hd", w, np.abs(v[:n]))
        dots = np.einsum("jhd,hd->hj", np.abs(k[:n]), np.abs(q[i])).max(1)
        ds = (k.shape[2] + 8) * U32 * scale * dots
        bound = H * np.abs(want) + TINY + (H + 2 * ds + (positions + 64) * U32)[:, None] * mag + positions * TINY * np.abs(v[:n]).max()
        err = np.abs(got[i] - want)
        assert np.all(np.isfinite(got[i])), f"{what}, token {i}: {int((~np.isfinite(got[i])).sum())} outputs are not finite"
        assert np.all(err <= bound), f"{what}, token {i}: worst {(err / bound).max():.3f} of the bound"


def masked_case(dev, seed, new, lengths, heads, value, page, where, junk, splits):
    rng = np.random.default_rng(seed)
    k, v, table = target(rng, lengths, heads, value, page, fill=np.nan)
    ks = [rng.standard_normal((n, heads, value + ROT)).astype(np.float16) for n in lengths]
    vs = [rng.standard_normal((n, heads, value)).astype(np.float16) for n in lengths]
    for s, n in enumerate(lengths):
        for j in range(n):
            p, o = ref.slot(table, s, j, page, len(k))
            k[p, :, o], v[p, :, :, o] = ks[s][j], vs[s][j]
        # The last position, which the last token alone sees.
        p, o = ref.slot(table, s, n - 1, page, len(k))
        if where in ("keys", "both"):
            k[p, :, o] = junk
        if where in ("values", "both"):
            v[p, :, :, o] = junk
        if where == "one dimension":
            v[p, :, 5, o] = junk
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(starts[-1]), heads, value + ROT)).astype(np.float16)
    most = table.shape[1] * page
    if splits is not None:
        assert (q4.q4g128_latent_prefill_workspace(len(q), len(new), heads, value, most) > 0) == splits
    scale = (value + ROT) ** -0.5 * 1.5
    out = q4.q4g128_latent_prefill(torch.from_numpy(q).to(dev), *(torch.from_numpy(a).to(dev) for a in (k, v, table)),
                                   i32(starts, dev), i32(lengths, dev), scale).float().cpu().numpy().astype(np.float64)
    for s, n in enumerate(lengths):
        rows, base, last = slice(starts[s], starts[s + 1] - 1), n - new[s], starts[s + 1] - 1
        check(out[rows], q[rows], ks[s], vs[s], base, scale, f"sequence {s}")
        if where == "one dimension":
            assert not np.any(np.isfinite(out[last, :, 5]))
            seen = vs[s].copy()
            seen[n - 1, :, 5] = out[last, :, 5] = 0
            # Dimension 5 is left out on both sides.
            seen[:, :, 5] = 0
            check(out[last:last + 1], q[last:last + 1], ks[s], seen, n - 1, scale, f"sequence {s}, the last token")
        else:
            assert not np.any(np.isfinite(out[last]))


FORMS = {"64 rows": ([33, 7], [133, 40], 2, False), "128 rows": ([40], [60], 260, False),
         "128 rows, several tiles": ([200], [230], 130, False), "64 rows, split": ([3], [3000], 1, True),
         "128 rows, split": ([9], [2000], 70, True)}


@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("where,junk", [("both", np.nan), ("both", np.inf), ("values", -np.inf), ("keys", np.nan),
                                        ("one dimension", np.inf), ("one dimension", np.nan)])
def test_masked_positions_stay_out(dev, value, form, where, junk):
    new, lengths, heads, splits = FORMS[form]
    masked_case(dev, 1, new, lengths, heads, value, 16 if form == "64 rows" else 64, where, junk, splits)


@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128, 256])
def test_masked_positions_in_all_pages(dev, value, page):
    masked_case(dev, 2, [70, 1, 5], [170, 65, 5], 3, value, page, "both", np.nan, None)
