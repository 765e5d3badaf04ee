"""Latent and expanded pages that interleave in one allocation, without a GPU.  Pointers are fake addresses, so a call that
is not refused must find no device; where there is one, such calls are left to the GPU tests.
"""
import pytest

from test_abi_attention import EINVAL, q4, torch
from test_abi_latent import ROWS, expand

# Halves of a page: 64 positions of 512 + 64 latent columns, of 16 heads' 192 key and of their 128 value columns.
LATENT, KEYS, VALUES = 64 * 576, 16 * 64 * 192, 16 * 64 * 128
STRIDE = LATENT + KEYS + VALUES


def interleaved(k=LATENT, v=LATENT + KEYS, rows=0, stride=STRIDE, k_stride=None, v_stride=None, **kw):
    """The call over three parts of pages `stride` apart, given by where they begin, in halves."""
    return expand(rows=ROWS + 2 * rows, stride=stride,
                  to=dict(k=ROWS + 2 * k, v=ROWS + 2 * v, k_stride=k_stride or stride, v_stride=v_stride or stride), **kw)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are fake")
@pytest.mark.parametrize("parts", [dict(), dict(rows=KEYS + VALUES, k=0, v=KEYS), dict(rows=KEYS, k=0, v=KEYS + LATENT),
                                   dict(rows=8, k=8 + LATENT, v=24 + LATENT + KEYS, stride=STRIDE + 24),
                                   dict(rows=3 * STRIDE), dict(k=LATENT + 5 * STRIDE), dict(v=LATENT + KEYS + 99 * STRIDE)])
def test_interleaved_pages_are_taken(parts):
    assert interleaved(**parts) == q4.Q4_EDEVICE


@pytest.mark.parametrize("parts", [dict(k=LATENT - 8), dict(rows=8), dict(v=STRIDE - VALUES + 8), dict(k=0), dict(v=0),
                                   dict(k=LATENT - 8 + 7 * STRIDE), dict(rows=STRIDE - 8), dict(v=LATENT + KEYS - 8),
                                   dict(k_stride=STRIDE + 8), dict(v_stride=STRIDE + 8),
                                   dict(stride=STRIDE + 8, k_stride=STRIDE, v_stride=STRIDE)])
def test_pages_that_share_elements_are_refused(parts):
    assert interleaved(**parts) == EINVAL
