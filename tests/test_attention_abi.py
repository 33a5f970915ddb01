"""The attention entry points' host side, without a GPU: refusals (every call
below is rejected before anything is launched) and the rotary frequencies,
which are computed on the host."""
import ctypes
import math

import numpy as np
import pytest

import trellis_quantized_gb300 as tq

FAKE = ctypes.c_void_p(0x10000)       # 16-byte aligned, never dereferenced
FAKE_MIS = ctypes.c_void_p(0x10008)   # 8-byte aligned
FAKE_ODD = ctypes.c_void_p(0x10002)   # not even 4-byte aligned


def _err():
    return tq.lib().exl3_last_error().decode()


def _transform(**kw):
    d = dict(q_norm=FAKE.value, k_norm=FAKE.value, eps=1e-6, inv_freq=FAKE.value, rotary_dim=128, layout=0,
             magnitude=1.0)
    d.update(kw)
    return tq.HeadTransform(*[d[n] for n, _ in tq.HeadTransform._fields_])


def _cache(**kw):
    d = dict(k=FAKE.value, v=FAKE.value, num_pages=10, page_size=16, heads_kv=8, head_dim=128,
             stride_page=16 * 8 * 128, stride_token=8 * 128, stride_head=128)
    d.update(kw)
    return tq.KvCache(*[d[n] for n, _ in tq.KvCache._fields_])


def _batch(**kw):
    d = dict(q_start=FAKE.value, kv_len=FAKE.value, page_table=FAKE.value, batch=2, max_pages=4)
    d.update(kw)
    return tq.PagedBatch(*[d[n] for n, _ in tq.PagedBatch._fields_])


ref = lambda s: None if s is None else ctypes.byref(s)


def _rope(t="default", **kw):
    g = lambda n, v: kw.get(n, v)
    t = _transform() if t == "default" else t
    return tq.lib().exl3_qk_norm_rope(g("q", FAKE), g("qs", 40 * 128), g("k", FAKE), g("ks", 8 * 128), g("idt", 0),
                                      g("T", 3), g("hq", 40), g("hkv", 8), g("D", 128), ref(t), g("pos", FAKE),
                                      g("qo", FAKE), g("ko", FAKE), g("odt", 0), None)


def _append(t="default", b="default", c="default", **kw):
    g = lambda n, v: kw.get(n, v)
    t = _transform() if t == "default" else t
    b = _batch() if b == "default" else b
    c = _cache() if c == "default" else c
    return tq.lib().exl3_qkv_append(g("q", FAKE), g("qs", 40 * 128), g("k", FAKE), g("ks", 8 * 128), g("v", FAKE),
                                    g("vs", 8 * 128), g("idt", 0), g("T", 3), g("hq", 40), ref(t), g("pos", None),
                                    ref(b), ref(c), g("qo", FAKE), g("ws", FAKE), g("wsb", 256), None)


def _attend(b="default", c="default", **kw):
    g = lambda n, v: kw.get(n, v)
    b = _batch() if b == "default" else b
    c = _cache() if c == "default" else c
    return tq.lib().exl3_paged_attention(g("q", FAKE), g("qs", 40 * 128), g("T", 3), g("hq", 40), ref(b), ref(c),
                                         g("scale", 0.1), g("causal", 1), g("window", 0), g("y", FAKE), g("odt", 0),
                                         g("lse", None), g("ws", FAKE), g("wsb", 1 << 40), None)


ROPE_REFUSALS = [
    (dict(q=None), tq.EXL3_ERR_ARG, "q is NULL"), (dict(q=FAKE_MIS), tq.EXL3_ERR_ARG, "q"),
    (dict(k=None), tq.EXL3_ERR_ARG, "k is NULL"), (dict(qo=None), tq.EXL3_ERR_ARG, "q_out"),
    (dict(ko=FAKE_MIS), tq.EXL3_ERR_ARG, "k_out"), (dict(pos=None), tq.EXL3_ERR_ARG, "positions"),
    (dict(pos=FAKE_ODD), tq.EXL3_ERR_ARG, "positions"), (dict(idt=2), tq.EXL3_ERR_ARG, "in_dtype"),
    (dict(odt=-1), tq.EXL3_ERR_ARG, "out_dtype"), (dict(D=96), tq.EXL3_ERR_SHAPE, "head_dim"),
    (dict(T=-1), tq.EXL3_ERR_SHAPE, "T ="), (dict(hq=0), tq.EXL3_ERR_SHAPE, "heads_q"),
    (dict(qs=40 * 128 - 8), tq.EXL3_ERR_SHAPE, "stride"), (dict(qs=40 * 128 + 4), tq.EXL3_ERR_SHAPE, "stride"),
    (dict(ks=0), tq.EXL3_ERR_SHAPE, "stride"),
]
TRANSFORM_REFUSALS = [
    (dict(rotary_dim=129), tq.EXL3_ERR_SHAPE, "rotary_dim"), (dict(rotary_dim=130), tq.EXL3_ERR_SHAPE, "rotary_dim"),
    (dict(rotary_dim=-2), tq.EXL3_ERR_SHAPE, "rotary_dim"), (dict(inv_freq=None), tq.EXL3_ERR_ARG, "inv_freq"),
    (dict(layout=2), tq.EXL3_ERR_ARG, "layout"), (dict(eps=-1.0), tq.EXL3_ERR_ARG, "eps"),
    (dict(eps=math.nan), tq.EXL3_ERR_ARG, "eps"), (dict(magnitude=math.inf), tq.EXL3_ERR_ARG, "magnitude"),
    (dict(q_norm=FAKE_MIS.value), tq.EXL3_ERR_ARG, "q_norm"), (dict(k_norm=FAKE_MIS.value), tq.EXL3_ERR_ARG, "k_norm"),
]
CACHE_REFUSALS = [
    (dict(k=None), tq.EXL3_ERR_ARG, "cache.k"), (dict(v=FAKE_MIS.value), tq.EXL3_ERR_ARG, "cache.v"),
    (dict(num_pages=0), tq.EXL3_ERR_SHAPE, "num_pages"), (dict(page_size=8), tq.EXL3_ERR_SHAPE, "page_size"),
    (dict(page_size=24), tq.EXL3_ERR_SHAPE, "page_size"), (dict(head_dim=80), tq.EXL3_ERR_SHAPE, "head_dim"),
    (dict(heads_kv=0), tq.EXL3_ERR_SHAPE, "heads_kv"), (dict(stride_page=4), tq.EXL3_ERR_SHAPE, "stride"),
    (dict(stride_token=-1024), tq.EXL3_ERR_SHAPE, "stride"), (dict(stride_head=64), tq.EXL3_ERR_SHAPE, "overlap"),
    (dict(stride_page=1 << 39), tq.EXL3_ERR_SHAPE, "stride"),
]
BATCH_REFUSALS = [
    (dict(q_start=None), tq.EXL3_ERR_ARG, "q_start"), (dict(kv_len=FAKE_ODD.value), tq.EXL3_ERR_ARG, "kv_len"),
    (dict(page_table=None), tq.EXL3_ERR_ARG, "page_table"), (dict(batch=0), tq.EXL3_ERR_SHAPE, "batch"),
    (dict(max_pages=0), tq.EXL3_ERR_SHAPE, "max_pages"), (dict(max_pages=1 << 27), tq.EXL3_ERR_SHAPE, "2^30"),
]


@pytest.mark.parametrize("kw,code,text", ROPE_REFUSALS)
def test_qk_norm_rope_refuses(kw, code, text):
    assert _rope(**kw) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", TRANSFORM_REFUSALS)
def test_transform_refusals(kw, code, text):
    assert _rope(_transform(**kw)) == code and text in _err()
    assert _append(_transform(**kw)) == code and text in _err()


def test_null_descriptors_are_refused():
    for rc in (_rope(None), _append(None), _append(b=None), _append(c=None), _attend(b=None), _attend(c=None)):
        assert rc == tq.EXL3_ERR_ARG


@pytest.mark.parametrize("kw,code,text", CACHE_REFUSALS)
def test_cache_refusals(kw, code, text):
    assert _append(c=_cache(**kw)) == code and text in _err()
    assert _attend(c=_cache(**kw)) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", BATCH_REFUSALS)
def test_batch_refusals(kw, code, text):
    assert _append(b=_batch(**kw)) == code and text in _err()
    assert _attend(b=_batch(**kw)) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", [
    (dict(q=None), tq.EXL3_ERR_ARG, "q is NULL"), (dict(v=FAKE_MIS), tq.EXL3_ERR_ARG, "v is"),
    (dict(vs=8), tq.EXL3_ERR_SHAPE, "v: stride"), (dict(qo=None), tq.EXL3_ERR_ARG, "q_out"),
    (dict(pos=FAKE_ODD), tq.EXL3_ERR_ARG, "positions"), (dict(T=-1), tq.EXL3_ERR_SHAPE, "T ="),
    (dict(ws=None), tq.EXL3_ERR_WORKSPACE, "workspace"), (dict(wsb=255), tq.EXL3_ERR_WORKSPACE, "workspace"),
])
def test_append_refuses(kw, code, text):
    assert _append(**kw) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", [
    (dict(q=FAKE_MIS), tq.EXL3_ERR_ARG, "q is"), (dict(y=None), tq.EXL3_ERR_ARG, "y is NULL"),
    (dict(odt=7), tq.EXL3_ERR_ARG, "out_dtype"), (dict(hq=44), tq.EXL3_ERR_SHAPE, "multiple of heads_kv"),
    (dict(hq=4), tq.EXL3_ERR_SHAPE, "multiple of heads_kv"), (dict(hq=8 * 129, qs=8 * 129 * 128), tq.EXL3_ERR_SHAPE, "128 times"), (dict(T=1 << 30), tq.EXL3_ERR_SHAPE, "2^31"),
    (dict(scale=0.0), tq.EXL3_ERR_ARG, "scale"), (dict(scale=math.inf), tq.EXL3_ERR_ARG, "scale"),
    (dict(scale=math.nan), tq.EXL3_ERR_ARG, "scale"), (dict(causal=2), tq.EXL3_ERR_ARG, "causal"),
    (dict(window=-1), tq.EXL3_ERR_ARG, "window"), (dict(lse=FAKE_ODD), tq.EXL3_ERR_ARG, "lse"),
    (dict(qs=8), tq.EXL3_ERR_SHAPE, "stride"), (dict(ws=None), tq.EXL3_ERR_WORKSPACE, "workspace"),
    (dict(wsb=1000), tq.EXL3_ERR_WORKSPACE, "workspace"), (dict(ws=FAKE_MIS), tq.EXL3_ERR_WORKSPACE, "aligned"),
])
def test_attention_refuses(kw, code, text):
    assert _attend(**kw) == code and text in _err()


def test_no_rows_enqueue_nothing():
    assert _rope(T=0) == _append(T=0) == _attend(T=0) == tq.EXL3_OK


def test_workspace_sizes():
    size = tq.exl3_paged_attention_workspace_size(1, 40, 8, 128, 1)
    assert size > 0 and size % 256 == 0
    for bad in ((1, 40, 8, 96, 1), (1, 44, 8, 128, 1), (1, 4, 8, 128, 1), (-1, 40, 8, 128, 1), (1, 40, 8, 128, 0),
                (1, 40, 0, 128, 1)):
        assert tq.exl3_paged_attention_workspace_size(*bad) == 0
    assert tq.exl3_qkv_append_workspace_size() >= 4


# ---------------------------------------------------------------- frequencies

def _reference(R, base, kind, factor, orig, low, high):
    i = np.arange(R // 2, dtype=np.float64)
    if kind == tq.EXL3_ROPE_NTK:
        base = base * factor ** (R / (R - 2))
    f = 1.0 / base ** (2 * i / R)
    if kind == tq.EXL3_ROPE_LINEAR:
        return f / factor, 1.0
    if kind == tq.EXL3_ROPE_BANDS:
        wavelength = 2 * np.pi / f
        s = (orig / wavelength - low) / (high - low)
        mid = (1 - s) * f / factor + s * f
        return np.where(wavelength < orig / high, f, np.where(wavelength > orig / low, f / factor, mid)), 1.0
    if kind == tq.EXL3_ROPE_YARN:
        dim = lambda n: R * np.log(orig / (n * 2 * np.pi)) / (2 * np.log(base))
        a, b = max(0, math.floor(dim(high))), min(R - 1, math.ceil(dim(low)))
        ramp = np.clip((i - a) / max(b - a, 1e-3), 0, 1)
        return f / factor * ramp + f * (1 - ramp), (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)
    return f, 1.0


@pytest.mark.parametrize("R", [4, 64, 128, 256, 20])
@pytest.mark.parametrize("kind,factor", [(0, 1.0), (1, 4.0), (2, 8.0), (3, 8.0), (4, 16.0), (4, 0.5)])
@pytest.mark.parametrize("base,orig,low,high", [(10000.0, 4096, 1.0, 4.0), (1e6, 32768, 1.0, 32.0)])
def test_rope_frequencies(R, kind, factor, base, orig, low, high):
    f, mag = tq.exl3_rope_frequencies(R, base, kind, factor, orig, low, high)
    want, want_mag = _reference(R, base, kind, factor, orig, low, high)
    assert f.shape == (R // 2,)
    # one rounding to fp32, and double-precision arithmetic before it
    np.testing.assert_allclose(f.numpy().astype(np.float64), want, rtol=2.0 ** -24 + 1e-12, atol=0)
    assert abs(mag - want_mag) <= 2.0 ** -24 * want_mag


def test_rope_frequencies_refuse():
    L = tq.lib()
    buf, mag = (ctypes.c_float * 64)(), ctypes.c_float(0)
    call = lambda R=64, base=1e4, kind=4, factor=2.0, orig=4096, low=1.0, high=32.0, out=buf, m=ctypes.byref(mag): \
        L.exl3_rope_frequencies(R, base, kind, factor, orig, low, high, out, m)
    assert call() == tq.EXL3_OK
    for kw in (dict(R=0), dict(R=7), dict(R=-2), dict(R=2, kind=2)):
        assert call(**kw) == tq.EXL3_ERR_SHAPE
    for kw in (dict(out=None), dict(m=None), dict(kind=5), dict(kind=-1), dict(base=1.0), dict(base=math.nan),
               dict(factor=0.0), dict(factor=math.inf), dict(orig=0), dict(low=0.0), dict(low=32.0),
               dict(high=math.inf), dict(kind=3, high=0.5)):
        assert call(**kw) == tq.EXL3_ERR_ARG
    assert call(kind=0, factor=0.0, orig=0, low=0.0) == tq.EXL3_OK      # not read without scaling


def test_bindings_refuse_other_tensors():
    import torch
    f = torch.zeros(8, dtype=torch.float64)
    with pytest.raises(TypeError):
        tq.head_transform(inv_freq=f)
    with pytest.raises(ValueError):
        tq.head_transform(q_norm=torch.zeros(128, dtype=torch.float16))        # a host tensor
    with pytest.raises(ValueError):
        tq.kv_cache(torch.zeros(2, 16, 8, 128, dtype=torch.float16), torch.zeros(2, 16, 8, 128, dtype=torch.float16))
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        tq.paged_batch(i, i[:1], torch.zeros((1, 3), dtype=torch.int32))
