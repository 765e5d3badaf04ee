"""Refusals of the calls for drafted tokens and latent rows, without a GPU: every invalid argument gives its documented
status before any HIP call.  Pointers are fake addresses that are never dereferenced.
"""
import ctypes

import pytest

from test_abi_attention import (A, EALIGN, EINVAL, ESHAPE, FREQ, K, LEN, NORM, OUT, POS, Q, QKV, SEQ, SLOPES, STARTS,
                                TABLE, V, WS, cache, options, q4, torch)

MASKS, SLOTS, KEEP, ROWS, MAIN, ROT, PACKED, SCALES, MINS, FIRSTS, TO = (A + (20 + i) * (1 << 36) for i in range(11))
NAN = float("nan")


def latent_cache(**kw):
    d = dict(rows=ROWS, table=TABLE, pages=100, stride=64 * 576, sequences=8, table_cols=16, latent=512, page=64)
    d.update(kw)
    return q4.LatentCache(**d)


def expanded_cache(**kw):
    d = dict(kv_heads=16, k_stride=16 * 64 * 192, v_stride=16 * 64 * 128)
    d.update(kw)
    return cache(**d)


def ref(c):
    return None if c is None else ctypes.byref(c)


def append(tokens=5, heads=16, slots=SLOTS, qkv=QKV, pos=POS, freq=FREQ, q=Q, eps=1e-6, ld=24 * 128, **kw):
    return q4.library().q4g128_rope_append_slots(qkv, ld, tokens, heads, ref(cache(**kw)), SEQ, pos, slots, freq, 128, 0,
                                                 1.0, NORM, NORM, eps, q, None)


def tree(q=Q, starts=STARTS, lengths=LEN, masks=MASKS, max_new=16, max_length=1024, tokens=100, count=8, heads=16, opt=None,
         out=OUT, ws=WS, ws_bytes=1 << 30, c=True, o=True, **kw):
    return q4.library().q4g128_attn_tree(q, ref(cache(**kw)) if c else None, starts, lengths, masks, max_new, max_length,
                                         tokens, count, heads, ref(options(**(opt or {}))) if o else None, out, ws,
                                         ws_bytes, None)


def keep(starts=POS, keep_starts=STARTS, keep=KEEP, total=9, count=8, c=True, **kw):
    return q4.library().q4g128_cache_keep(ref(cache(**kw)) if c else None, starts, keep_starts, keep, total, count, None)


def latent_keep(starts=POS, keep_starts=STARTS, keep=KEEP, total=9, count=8, c=True, **kw):
    return q4.library().q4g128_latent_keep(ref(latent_cache(**kw)) if c else None, starts, keep_starts, keep, total, count,
                                           None)


def latent_append(kv=QKV, ld=576, tokens=5, seq=SEQ, pos=POS, slots=SLOTS, freq=FREQ, norm=NORM, eps=1e-6, qm=MAIN,
                  main_ld=16 * 128, main_head=128, main=128, qr=ROT, rot_ld=16 * 64, rot_head=64, heads=16, q=Q, c=True,
                  **kw):
    return q4.library().q4g128_latent_append(kv, ld, tokens, ref(latent_cache(**kw)) if c else None, seq, pos, slots, freq, 0,
                                             1.0, norm, eps, qm, main_ld, main_head, main, qr, rot_ld, rot_head, heads, q,
                                             None)


def latent_attn(q=Q, starts=STARTS, lengths=LEN, masks=MASKS, max_new=16, max_length=1024, tokens=100, count=8, heads=16,
                scale=0.1, out=OUT, ws=WS, ws_bytes=1 << 32, c=True, **kw):
    return q4.library().q4g128_latent_attn(q, ref(latent_cache(**kw)) if c else None, starts, lengths, masks, max_new,
                                           max_length, tokens, count, heads, scale, out, ws, ws_bytes, None)


def expand(lengths=LEN, firsts=FIRSTS, max_length=1024, count=8, packed=PACKED, scales=SCALES, mins=MINS, c=True, to=None,
           **kw):
    return q4.library().q4g128_latent_expand(ref(latent_cache(**kw)) if c else None, lengths, firsts, max_length, count,
                                             packed, scales, mins, None if to is False else ref(expanded_cache(**(to or {}))),
                                             None)


def prefill(q=Q, starts=STARTS, lengths=LEN, max_length=1024, tokens=3, count=1, scale=0.1, out=OUT, ws=WS,
            ws_bytes=1 << 30, c=True, **kw):
    return q4.library().q4g128_latent_prefill(q, ref(expanded_cache(**kw)) if c else None, starts, lengths, max_length,
                                              tokens, count, scale, out, ws, ws_bytes, None)


LATENT = [latent_append, latent_keep, latent_attn, expand]
KEEPS = [keep, latent_keep]
ATTENTION = [tree, latent_attn, prefill]


@pytest.mark.parametrize("call", LATENT)
def test_latent_cache(call):
    for bad in (dict(c=False), dict(rows=None), dict(table=None), dict(pages=0), dict(sequences=0), dict(table_cols=0)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(latent=64), dict(latent=384), dict(latent=1024), dict(page=8), dict(page=48), dict(page=512),
                dict(stride=64 * 576 - 8), dict(stride=64 * 576 + 4), dict(stride=1 << 62), dict(pages=1 << 31),
                dict(sequences=1 << 31), dict(table_cols=1 << 26)):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(rows=ROWS + 8), dict(table=TABLE + 2)):
        assert call(**bad) == EALIGN, bad


@pytest.mark.parametrize("call", [tree, keep])
def test_head_cache(call):
    for bad in (dict(c=False), dict(k=None), dict(v=None), dict(table=None), dict(pages=0), dict(kv_heads=0)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dim=80), dict(page=8), dict(k_stride=4 * 64 * 128 - 8), dict(v_stride=4 * 64 * 128 + 4)):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(k=K + 8), dict(v=V + 2), dict(table=TABLE + 2)):
        assert call(**bad) == EALIGN, bad


@pytest.mark.parametrize("call,wrap", [(prefill, lambda d: d), (expand, lambda d: dict(to=d))])
def test_expanded_cache(call, wrap):
    for bad in (dict(k=None), dict(v=None), dict(table=None), dict(pages=0), dict(sequences=0), dict(table_cols=0),
                dict(kv_heads=0)):
        assert call(**wrap(bad)) == EINVAL, bad
    for bad in (dict(dim=96), dict(dim=192), dict(dim=256), dict(kv_heads=1025), dict(page=8), dict(page=512),
                dict(k_stride=16 * 64 * 192 - 8), dict(k_stride=16 * 64 * 128), dict(v_stride=16 * 64 * 128 - 8),
                dict(k_stride=16 * 64 * 192 + 4), dict(k_stride=1 << 62), dict(table_cols=1 << 26)):
        assert call(**wrap(bad)) == ESHAPE, bad
    for bad in (dict(k=K + 8), dict(v=V + 8), dict(table=TABLE + 1)):
        assert call(**wrap(bad)) == EALIGN, bad


def test_slots():
    assert append(slots=None) == EINVAL
    assert append(slots=SLOTS + 2) == EALIGN
    for bad in (dict(slots=Q), dict(slots=K + 64), dict(slots=V), dict(q=SLOTS), dict(pos=None), dict(eps=NAN)):
        assert append(**bad) == EINVAL, bad


@pytest.mark.parametrize("call", KEEPS)
def test_keep_refusals(call):
    pool = K if call is keep else ROWS
    for bad in (dict(starts=None), dict(keep_starts=None), dict(keep=None), dict(total=-1), dict(count=0),
                dict(starts=pool + 64), dict(keep_starts=pool), dict(keep=pool + 4), dict(table=pool + 128)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(count=9), dict(count=65537, sequences=65537), dict(total=(1 << 20) + 1)):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(starts=POS + 2), dict(keep_starts=STARTS + 1), dict(keep=KEEP + 3)):
        assert call(**bad) == EALIGN, bad
    assert call(total=0) == q4.Q4_OK and call(total=0, keep=None) == q4.Q4_OK  # nothing to move, nothing launched


def test_keep_pools_that_meet():
    for bad in (dict(v=K), dict(v=K + 4096, v_stride=4 * 64 * 128 + 8)):
        assert keep(**bad) == EINVAL, bad


@pytest.mark.parametrize("call", ATTENTION)
def test_attention_refusals(call):
    pool = ROWS if call is latent_attn else K
    for bad in (dict(q=None), dict(starts=None), dict(lengths=None), dict(out=None), dict(tokens=0), dict(count=0),
                dict(max_length=0), dict(ws=None), dict(ws_bytes=0), dict(out=Q), dict(out=pool + 256), dict(out=TABLE),
                dict(out=LEN), dict(out=STARTS), dict(ws=Q), dict(ws=OUT), dict(ws=pool), dict(ws=LEN), dict(ws=STARTS),
                dict(c=False)):
        # a short call on a long table needs a workspace
        assert call(**dict(dict(tokens=3, count=1), **bad)) == EINVAL, bad
    for bad in (dict(count=9), dict(tokens=(1 << 20) + 1), dict(max_length=16 * 64 + 1), dict(count=65537, sequences=65537)):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(q=Q + 8), dict(out=OUT + 8), dict(starts=STARTS + 2), dict(lengths=LEN + 2), dict(ws=WS + 8)):
        assert call(**bad) == EALIGN, bad
    for scale in (0.0, -1.0, NAN, float("inf")):
        bad = dict(opt=dict(scale=scale)) if call is tree else dict(scale=scale)
        assert call(**bad) == EINVAL, bad


@pytest.mark.parametrize("call", [tree, latent_attn])
def test_masks_and_bounds(call):
    assert call(masks=MASKS + 4) == EALIGN
    assert call(max_new=0) == EINVAL
    assert call(max_new=65) == ESHAPE
    for bad in (dict(out=MASKS), dict(ws=MASKS)):
        assert call(**dict(dict(tokens=3, count=1), **bad)) == EINVAL, bad
    assert call(max_new=(1 << 20) + 1, masks=None) == ESHAPE


def test_tree_refusals():
    assert tree(o=False) == EINVAL
    for bad in (dict(softcap=NAN), dict(window=-1), dict(prefix=LEN), dict(slopes=OUT), dict(softcap=-1.0)):
        assert tree(opt=bad) == EINVAL, bad
    assert tree(opt=dict(slopes=SLOPES + 2)) == EALIGN
    for bad in (dict(heads=15), dict(kv_heads=1, heads=65), dict(heads=2048, kv_heads=1024)):
        assert tree(**bad) == ESHAPE, bad
    assert tree(heads=0) == EINVAL
    need = q4.q4g128_attn_tree_workspace(3, 1, 16, 4, 128, 16, 1024)
    assert need > 0 and tree(tokens=3, count=1, ws_bytes=need - 1) == EINVAL


def test_latent_append_refusals():
    for bad in (dict(kv=None), dict(pos=None), dict(slots=None), dict(tokens=0), dict(heads=-1), dict(qm=None),
                dict(qr=None), dict(q=None), dict(eps=-1.0), dict(eps=NAN), dict(q=MAIN), dict(q=ROT + 64), dict(q=QKV),
                dict(q=ROWS), dict(q=TABLE), dict(q=POS), dict(q=FREQ), dict(q=NORM), dict(kv=ROWS + 64),
                dict(slots=ROWS), dict(norm=ROWS + 32), dict(table=ROWS + 64), dict(qm=ROWS + 16)):
        assert latent_append(**bad) == EINVAL, bad
    for bad in (dict(ld=572), dict(ld=578), dict(tokens=(1 << 20) + 1), dict(heads=1025), dict(main=4), dict(main=100),
                dict(main=1032, main_ld=1 << 15, main_head=1032), dict(main_ld=120), dict(main_head=120),
                dict(main_head=130), dict(rot_ld=60), dict(rot_head=32), dict(rot_head=66), dict(main_ld=1 << 62),
                dict(rot_head=1 << 62), dict(ld=1 << 62)):
        assert latent_append(**bad) == ESHAPE, bad
    for bad in (dict(kv=QKV + 8), dict(seq=SEQ + 2), dict(pos=POS + 1), dict(slots=SLOTS + 2), dict(freq=FREQ + 2),
                dict(norm=NORM + 1), dict(qm=MAIN + 4), dict(qr=ROT + 8), dict(q=Q + 2)):
        assert latent_append(**bad) == EALIGN, bad


def test_latent_attn_refusals():
    assert latent_attn(heads=0) == EINVAL
    assert latent_attn(heads=1025) == ESHAPE
    need = q4.q4g128_latent_attn_workspace(16, 512, 16)
    assert need > 0 and latent_attn(ws_bytes=need - 1) == EINVAL


def test_expand_refusals():
    for bad in (dict(lengths=None), dict(packed=None), dict(scales=None), dict(mins=None), dict(count=0),
                dict(max_length=0), dict(to=False), dict(lengths=K), dict(firsts=V + 64), dict(packed=K + 4096),
                dict(scales=V), dict(mins=K), dict(rows=K), dict(rows=V + 4096), dict(table=K),
                dict(to=dict(table=V + 4096)), dict(to=dict(v=K)), dict(to=dict(v=K + 4096)),
                dict(to=dict(v=K + 100 * 16 * 64 * 192)), dict(to=dict(k=ROWS)), dict(to=dict(v=ROWS + 4096))):
        assert expand(**bad) == EINVAL, bad
    for bad in (dict(count=9), dict(count=9, sequences=9), dict(max_length=16 * 64 + 1),
                dict(max_length=16 * 64 + 1, table_cols=17), dict(count=65537, sequences=65537, to=dict(sequences=65537))):
        assert expand(**bad) == ESHAPE, bad
    for bad in (dict(lengths=LEN + 2), dict(firsts=FIRSTS + 1), dict(packed=PACKED + 8), dict(scales=SCALES + 1),
                dict(mins=MINS + 1)):
        assert expand(**bad) == EALIGN, bad


def test_workspaces():
    for args, status in (((0, 1, 16, 4, 128, 16, 64), EINVAL), ((4, 0, 16, 4, 128, 16, 64), EINVAL),
                         ((4, 1, 0, 4, 128, 16, 64), EINVAL), ((4, 1, 16, 0, 128, 16, 64), EINVAL),
                         ((4, 1, 16, 4, 128, 0, 64), EINVAL), ((4, 1, 16, 4, 128, 16, 0), EINVAL),
                         ((4, 1, 16, 3, 128, 16, 64), ESHAPE), ((4, 1, 16, 4, 72, 16, 64), ESHAPE),
                         ((4, 1, 16, 4, 128, 65, 64), ESHAPE), ((4, 1, 128, 1, 128, 16, 64), ESHAPE)):
        assert q4.q4g128_attn_tree_workspace(*args) == status, args
    for args, status in (((0, 512, 1), EINVAL), ((16, 512, 0), EINVAL), ((1025, 512, 1), ESHAPE), ((16, 500, 1), ESHAPE),
                         ((16, 512, (1 << 20) + 1), ESHAPE)):
        assert q4.q4g128_latent_attn_workspace(*args) == status, args
    for args, status in (((0, 1, 16, 128, 64), EINVAL), ((4, 0, 16, 128, 64), EINVAL), ((4, 1, 0, 128, 64), EINVAL),
                         ((4, 1, 16, 128, 0), EINVAL), ((4, 1, 16, 96, 64), ESHAPE), ((4, 1, 1025, 128, 64), ESHAPE),
                         ((4, 65537, 16, 128, 64), ESHAPE), (((1 << 20) + 1, 1, 16, 128, 64), ESHAPE)):
        assert q4.q4g128_latent_prefill_workspace(*args) == status, args


def test_binding_refuses_host_tensors():
    f16, i32 = dict(dtype=torch.float16), dict(dtype=torch.int32)
    k, v, table = torch.zeros(2, 1, 16, 64, **f16), torch.zeros(2, 1, 64, 16, **f16), torch.zeros(1, 2, **i32)
    rows, one, two = torch.zeros(2, 16, 192, **f16), torch.ones(1, **i32), torch.tensor([0, 1], **i32)
    q = torch.zeros(1, 2, 64, **f16)
    for call in (lambda: q4.q4g128_attn_tree(q, k, v, table, two, one),
                 lambda: q4.q4g128_cache_keep(k, v, table, one, two, one),
                 lambda: q4.q4g128_rope_append(torch.zeros(1, 256), k, v, table, one, None, 2, slots=one),
                 lambda: q4.q4g128_latent_keep(rows, table, one, two, one),
                 lambda: q4.q4g128_latent_append(torch.zeros(1, 192), rows, table, one, None),
                 lambda: q4.q4g128_latent_attn(torch.zeros(1, 2, 192, **f16), rows, table, two, one, 0.1),
                 lambda: q4.q4g128_latent_prefill(torch.zeros(1, 1, 128, **f16), torch.zeros(2, 1, 16, 128, **f16), v, table,
                                                  two, one, 0.1),
                 lambda: q4.q4g128_latent_expand(rows, table, one, torch.zeros(128, 64, dtype=torch.uint8),
                                                 torch.zeros(128, 1, **f16), torch.zeros(128, 1, **f16),
                                                 torch.zeros(2, 1, 16, 128, **f16), v, table)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        q4.q4g128_latent_attn(q, None, table, two, one, 0.1)
