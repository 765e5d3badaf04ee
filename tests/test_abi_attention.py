"""Refusals of the cache and attention calls, without a GPU: every invalid
argument gives its documented status before any HIP call.  Pointers are fake
addresses that are never dereferenced.
"""
import ctypes

import pytest

q4 = pytest.importorskip("int4_group_quantized_amd")
torch = pytest.importorskip("torch")

EINVAL, ESHAPE, EALIGN = q4.Q4_EINVAL, q4.Q4_ESHAPE, q4.Q4_EALIGN

A = 0x7F0000000000
(QKV, K, V, TABLE, SEQ, POS, FREQ, NORM, Q, OUT, LEN, STARTS, SLOPES, PREFIX, WS) = (A + i * (1 << 36) for i in range(15))


def cache(**kw):
    d = dict(k=K, v=V, table=TABLE, pages=100, k_stride=4 * 64 * 128, v_stride=4 * 64 * 128, sequences=8,
             table_cols=16, kv_heads=4, dim=128, page=64)
    d.update(kw)
    return q4.KvCache(**d)


def append(qkv=QKV, ld=24 * 128, tokens=5, heads=16, c=None, seq=SEQ, pos=POS, freq=FREQ, rot=128, inter=0, mscale=1.0,
           qn=NORM, kn=NORM, eps=1e-6, q=Q, **kw):
    c = cache(**kw) if c is None else c
    return q4.library().q4g128_rope_append(qkv, ld, tokens, heads, ctypes.byref(c) if c else None, seq, pos, freq, rot,
                                           inter, mscale, qn, kn, eps, q, None)


def options(scale=0.1, softcap=0.0, window=0, slopes=None, prefix=None):
    return q4.AttnOptions(scale, softcap, window, slopes, prefix)


def decode(q=Q, lengths=LEN, max_length=1024, batch=8, heads=16, o=None, out=OUT, ws=WS, ws_bytes=1 << 30, no_cache=False,
           no_options=False, opt=None, **kw):
    c, o = cache(**kw), options(**(opt or {}))
    return q4.library().q4g128_attn_decode(q, None if no_cache else ctypes.byref(c), lengths, max_length, batch, heads,
                                           None if no_options else ctypes.byref(o), out, ws, ws_bytes, None)


def prefill(q=Q, starts=STARTS, lengths=LEN, max_length=1024, tokens=100, count=8, heads=16, out=OUT, ws=WS,
            ws_bytes=1 << 30, no_cache=False, no_options=False, opt=None, **kw):
    c, o = cache(**kw), options(**(opt or {}))
    return q4.library().q4g128_attn_prefill(q, None if no_cache else ctypes.byref(c), starts, lengths, max_length,
                                            tokens, count, heads, None if no_options else ctypes.byref(o), out, ws,
                                            ws_bytes, None)


ALL = [append, decode, prefill]
BOTH = [decode, prefill]


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(table=None), dict(q=None), dict(pages=0),
                                 dict(sequences=0), dict(table_cols=0), dict(kv_heads=0), dict(heads=0)])
def test_einval_cache(call, bad):
    assert call(**bad) == EINVAL


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("bad", [dict(dim=80), dict(dim=0), dict(dim=512), dict(page=8), dict(page=48), dict(page=512),
                                 dict(heads=15), dict(kv_heads=1, heads=65), dict(heads=2048, kv_heads=1024),
                                 dict(k_stride=4 * 64 * 128 - 8), dict(v_stride=4 * 64 * 128 + 4),
                                 dict(k_stride=1 << 62), dict(table_cols=1 << 26), dict(pages=1 << 31),
                                 dict(sequences=1 << 31)])
def test_eshape_cache(call, bad):
    assert call(**bad) == ESHAPE


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("bad", [dict(k=K + 8), dict(v=V + 2), dict(table=TABLE + 2), dict(q=Q + 8)])
def test_ealign_cache(call, bad):
    assert call(**bad) == EALIGN


def test_append_refusals():
    assert append(c=False) == EINVAL
    for bad in (dict(qkv=None), dict(pos=None), dict(tokens=0), dict(tokens=-1), dict(freq=None), dict(eps=-1.0),
                dict(eps=float("nan")), dict(q=K + 256), dict(q=TABLE), dict(q=QKV + 1024), dict(q=POS), dict(q=FREQ),
                dict(qkv=K + 64), dict(seq=V), dict(qn=V + 64), dict(v=K), dict(v=K + 4 * 64 * 128),
                dict(v=K + 4096, v_stride=4 * 64 * 128 + 8), dict(table=K + 64)):
        assert append(**bad) == EINVAL, bad
    for bad in (dict(rot=130), dict(rot=-4), dict(rot=2), dict(rot=132), dict(ld=24 * 128 - 4), dict(ld=24 * 128 + 2),
                dict(tokens=q4.library() and (1 << 20) + 1)):
        assert append(**bad) == ESHAPE, bad
    for bad in (dict(qkv=QKV + 4), dict(seq=SEQ + 1), dict(pos=POS + 2), dict(freq=FREQ + 2), dict(qn=NORM + 1),
                dict(kn=NORM + 1)):
        assert append(**bad) == EALIGN, bad


@pytest.mark.parametrize("call", BOTH)
def test_attention_refusals(call):
    assert call(no_cache=True) == EINVAL
    assert call(no_options=True) == EINVAL
    for bad in (dict(lengths=None), dict(out=None), dict(max_length=0), dict(ws=None), dict(ws_bytes=0),
                dict(out=Q), dict(out=K + 256), dict(out=V), dict(out=TABLE), dict(out=LEN), dict(ws=Q), dict(ws=OUT),
                dict(ws=K), dict(ws=LEN), dict(opt=dict(scale=0.0)), dict(opt=dict(scale=-1.0)),
                dict(opt=dict(scale=float("nan"))), dict(opt=dict(softcap=-1.0)), dict(opt=dict(softcap=float("nan"))),
                dict(opt=dict(window=-1)), dict(opt=dict(window=5, prefix=PREFIX)), dict(opt=dict(slopes=OUT)),
                dict(opt=dict(slopes=WS))):
        # one short prompt on a long table needs a workspace; the decode call always does
        if call is prefill:
            bad = dict(tokens=3, count=1, **bad)
        assert call(**bad) == EINVAL, bad
    for bad in (dict(max_length=16 * 64 + 1),):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(out=OUT + 8), dict(lengths=LEN + 2), dict(ws=WS + 8), dict(opt=dict(slopes=SLOPES + 2))):
        assert call(**bad) == EALIGN, bad


def test_decode_refusals():
    assert decode(batch=0) == EINVAL
    assert decode(batch=9) == ESHAPE  # the table has 8 sequences
    assert decode(batch=65537, sequences=65537) == ESHAPE
    assert decode(opt=dict(prefix=PREFIX)) == EINVAL
    need = q4.q4g128_attn_decode_workspace(8, 16, 128)
    assert need > 0 and decode(ws_bytes=need - 1) == EINVAL
    for args, status in (((0, 16, 128), EINVAL), ((8, 0, 128), EINVAL), ((8, 16, 100), ESHAPE), ((8, 1025, 128), ESHAPE),
                         ((65537, 16, 128), ESHAPE)):
        assert q4.q4g128_attn_decode_workspace(*args) == status


def test_prefill_refusals():
    assert prefill(starts=None) == EINVAL
    assert prefill(starts=STARTS + 2) == EALIGN
    assert prefill(tokens=0) == EINVAL
    assert prefill(count=0) == EINVAL
    assert prefill(count=9) == ESHAPE
    assert prefill(tokens=(1 << 20) + 1) == ESHAPE
    assert prefill(out=STARTS) == EINVAL
    assert prefill(opt=dict(prefix=OUT)) == EINVAL
    assert prefill(opt=dict(prefix=PREFIX + 1)) == EALIGN
    need = q4.q4g128_attn_prefill_workspace(3, 1, 16, 4, 128, 1024)
    assert need > 0 and prefill(tokens=3, count=1, ws_bytes=need - 1) == EINVAL
    assert prefill(tokens=3, count=1, ws=STARTS) == EINVAL
    assert q4.q4g128_attn_prefill_workspace(1 << 16, 1, 16, 4, 128, 1 << 16) == 0
    for args, status in (((0, 1, 16, 4, 128, 64), EINVAL), ((4, 0, 16, 4, 128, 64), EINVAL),
                         ((4, 1, 16, 3, 128, 64), ESHAPE), ((4, 1, 16, 4, 72, 64), ESHAPE),
                         ((4, 1, 128, 1, 128, 64), ESHAPE), ((4, 1, 16, 4, 128, 0), EINVAL)):
        assert q4.q4g128_attn_prefill_workspace(*args) == status


def test_binding_refuses_host_tensors():
    f16 = dict(dtype=torch.float16)
    k, v = torch.zeros(2, 1, 16, 64, **f16), torch.zeros(2, 1, 64, 16, **f16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    one = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        q4.q4g128_rope_append(torch.zeros(1, 256), k, v, table, one, None, 2)
    with pytest.raises(ValueError):
        q4.q4g128_attn_decode(torch.zeros(1, 2, 64, **f16), k, v, table, one)
    with pytest.raises(ValueError):
        q4.q4g128_attn_prefill(torch.zeros(1, 2, 64, **f16), k, v, table, torch.tensor([0, 1], dtype=torch.int32), one)
    with pytest.raises(TypeError):
        q4.q4g128_attn_decode(torch.zeros(1, 2, 64, **f16), None, v, table, one)
