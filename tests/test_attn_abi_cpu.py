"""CPU tests of the attention entry points: arguments are validated before any HIP call, workspaces are sized by
the split, and the binding refuses tensors that do not fit. No kernel is launched."""

import ctypes

import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from bit_weight_quantized_qgemm_amd import attention
from bit_weight_quantized_qgemm_amd.attention import _CacheStruct

OK, NULL, SHAPE, ALIGN, WS, RANGE, ALIAS, HIP, DEV = 0, -1, -2, -3, -4, -6, -7, -8, -9
F16, BF16, FP8 = qg.DT_F16, qg.DT_BF16, qg.DT_FP8
Q, K, V, OUT, TABLE, LENS, START, WSP, KC, VC, ROPE, POS, NORM = (0x10000000 * i for i in range(1, 14))


def _cache(**kw):
    f = dict(k=KC, v=VC, num_pages=100, page_stride=8 * 16 * 128, token_stride=128, head_stride=16 * 128, page_size=16,
             kv_heads=8, head_dim=128, dtype=F16, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return _CacheStruct(*(f[n] for n, _ in _CacheStruct._fields_))


def _decode(cache=None, **kw):
    a = dict(q=Q, qts=64 * 128, qhs=128, table=TABLE, cols=64, lens=LENS, seqs=4, max_len=1000, heads=64, act=F16,
             scale=0.1, window=0, sinks=0, out=OUT, ots=64 * 128, ohs=128, ws=WSP, wsb=1 << 30)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return qg.lib().qgemm_attn_decode(a["q"], a["qts"], a["qhs"], ctypes.byref(c), a["table"], a["cols"], a["lens"],
                                      a["seqs"], a["max_len"], a["heads"], a["act"], a["scale"], a["window"],
                                      a["sinks"], a["out"], a["ots"], a["ohs"], a["ws"], a["wsb"], None)


def _prefill(cache=None, **kw):
    a = dict(q=Q, qts=64 * 128, qhs=128, table=TABLE, cols=64, start=START, lens=LENS, seqs=4, tokens=40, max_q=20,
             max_len=1000, heads=64, act=F16, scale=0.1, window=0, sinks=0, out=OUT, ots=64 * 128, ohs=128, ws=WSP,
             wsb=1 << 30)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return qg.lib().qgemm_attn_prefill(a["q"], a["qts"], a["qhs"], ctypes.byref(c), a["table"], a["cols"], a["start"],
                                       a["lens"], a["seqs"], a["tokens"], a["max_q"], a["max_len"], a["heads"],
                                       a["act"], a["scale"], a["window"], a["sinks"], a["out"], a["ots"], a["ohs"],
                                       a["ws"], a["wsb"], None)


def _append(cache=None, **kw):
    a = dict(q=Q, qts=80 * 128, qhs=128, k=K, kts=80 * 128, khs=128, v=V, vts=80 * 128, vhs=128, qn=NORM, kn=None,
             eps=1e-6, rope=ROPE, rows=4096, rot=128, inter=0, pos=POS, seq=None, table=TABLE, cols=64, seqs=4,
             tokens=10, heads=64, act=F16, out=OUT, ots=64 * 128, ohs=128)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return qg.lib().qgemm_qk_rope_append(a["q"], a["qts"], a["qhs"], a["k"], a["kts"], a["khs"], a["v"], a["vts"],
                                         a["vhs"], a["qn"], a["kn"], a["eps"], a["rope"], a["rows"], a["rot"],
                                         a["inter"], a["pos"], a["seq"], a["table"], a["cols"], a["seqs"],
                                         a["tokens"], a["heads"], a["act"], ctypes.byref(c), a["out"], a["ots"],
                                         a["ohs"], None)


# Every call below is refused before any HIP call, or (OK) launches nothing.
CACHE_FAULTS = [
    (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE), (dict(head_dim=120), SHAPE), (dict(head_dim=272), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=65552), SHAPE), (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 31), SHAPE),
    (dict(dtype=0), RANGE), (dict(dtype=4), RANGE), (dict(dtype=BF16), RANGE),
    (dict(k_scale=0.5), RANGE), (dict(v_scale=2.0), RANGE), (dict(dtype=FP8, k_scale=0.0), RANGE),
    (dict(dtype=FP8, v_scale=float("nan")), RANGE), (dict(dtype=FP8, k_scale=float("inf")), RANGE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=KC + 8), ALIGN), (dict(v=VC + 4), ALIGN),
    (dict(token_stride=120), ALIGN), (dict(token_stride=132), ALIGN), (dict(token_stride=(1 << 25) + 8), ALIGN),
    (dict(head_stride=64), ALIGN), (dict(head_stride=2044), ALIGN), (dict(head_stride=-2048), ALIGN),
    (dict(page_stride=-16), ALIGN), (dict(page_stride=12), ALIGN), (dict(page_stride=1 << 31), ALIGN),
    (dict(dtype=FP8, token_stride=136), ALIGN),
]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_faults(fault, status):
    for call in (_decode, _prefill, _append):
        assert call(_cache(**fault)) == status, call


ATTN_FAULTS = [
    (dict(seqs=-1), SHAPE), (dict(seqs=65536), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_len=(1 << 24) + 1), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=60), SHAPE), (dict(heads=8 * 129), SHAPE), (dict(max_len=1025), SHAPE),
    (dict(cols=-1), SHAPE), (dict(act=0), RANGE), (dict(act=FP8), RANGE), (dict(window=-1), RANGE),
    (dict(sinks=-1), RANGE), (dict(scale=0.0), RANGE), (dict(scale=-1.0), RANGE), (dict(scale=float("nan")), RANGE),
    (dict(scale=float("inf")), RANGE), (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(q=Q + 8), ALIGN), (dict(out=OUT + 2), ALIGN), (dict(lens=LENS + 2), ALIGN),
    (dict(table=TABLE + 1), ALIGN), (dict(qts=64 * 128 + 4), ALIGN), (dict(qhs=120), ALIGN), (dict(qts=-8), ALIGN),
    (dict(ots=128), ALIGN), (dict(ohs=64), ALIGN), (dict(ots=64 * 128 - 8), ALIGN),
    (dict(out=Q), ALIAS), (dict(out=Q + 4096), ALIAS), (dict(out=KC + 256), ALIAS), (dict(out=VC), ALIAS),
    (dict(out=TABLE), ALIAS), (dict(out=LENS), ALIAS), (dict(out=WSP), ALIAS), (dict(ws=Q), ALIAS),
    (dict(ws=KC), ALIAS), (dict(ws=None), NULL), (dict(ws=WSP + 8), ALIGN), (dict(wsb=4096), WS),
]


@pytest.mark.parametrize("fault,status", ATTN_FAULTS)
def test_attention_faults(fault, status):
    for call in (_decode, _prefill):
        assert call(**fault) == status, call


PREFILL_FAULTS = [(dict(tokens=-1), SHAPE), (dict(tokens=(1 << 20) + 1), SHAPE), (dict(max_q=-1), SHAPE),
                  (dict(max_q=(1 << 20) + 1), SHAPE), (dict(start=None), NULL), (dict(start=START + 2), ALIGN),
                  (dict(out=START), ALIAS), (dict(tokens=0), OK), (dict(max_q=0), OK), (dict(seqs=0), OK)]


@pytest.mark.parametrize("fault,status", PREFILL_FAULTS)
def test_prefill_faults(fault, status):
    assert _prefill(**fault) == status


APPEND_FAULTS = [
    (dict(act=FP8), RANGE), (dict(inter=2), RANGE), (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE),
    (dict(seqs=65536), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 20) + 1), SHAPE), (dict(heads=12), SHAPE),
    (dict(rot=8), SHAPE), (dict(rot=144), SHAPE), (dict(rot=-16), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=(1 << 24) + 1), SHAPE), (dict(cols=(1 << 24) + 1), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL), (dict(pos=None), NULL),
    (dict(table=None), NULL), (dict(rope=None), NULL), (dict(q=Q + 2), ALIGN), (dict(k=K + 8), ALIGN),
    (dict(v=V + 8), ALIGN), (dict(qn=NORM + 2), ALIGN), (dict(kn=NORM + 2), ALIGN), (dict(rope=ROPE + 4), ALIGN),
    (dict(out=OUT + 8), ALIGN), (dict(pos=POS + 2), ALIGN), (dict(seq=LENS + 2), ALIGN), (dict(kts=84), ALIGN),
    (dict(vhs=64), ALIGN), (dict(ots=128), ALIGN), (dict(out=Q + 256), ALIAS), (dict(out=Q), ALIAS),
    (dict(out=K), ALIAS), (dict(out=V), ALIAS), (dict(out=POS), ALIAS), (dict(out=KC), ALIAS), (dict(q=VC), ALIAS),
    (dict(k=KC), ALIAS), (dict(rope=VC), ALIAS), (dict(tokens=0), OK),
]


@pytest.mark.parametrize("fault,status", APPEND_FAULTS)
def test_append_faults(fault, status):
    assert _append(**fault) == status


def test_append_task_numbers_stay_in_32_bits():
    # 2^20 tokens of 1024 + 2 * 1024 heads
    c = _cache(kv_heads=1024, head_stride=128, token_stride=1024 * 128, page_stride=1 << 21)
    assert _append(c, tokens=1 << 20, heads=1024, qts=3072 * 128, kts=3072 * 128, vts=3072 * 128,
                   ots=1024 * 128) == SHAPE


def test_null_cache_and_null_results():
    L = qg.lib()
    assert L.qgemm_attn_decode(Q, 8, 8, None, TABLE, 1, LENS, 1, 1, 1, F16, 1.0, 0, 0, OUT, 8, 8, None, 0, None) == NULL
    assert L.qgemm_attn_decode_workspace_bytes(1, 1, 1, 1, 16, 0, 0, None) == NULL
    assert L.qgemm_attn_prefill_workspace_bytes(1, 1, 1, 1, 1, 16, 0, 0, None) == NULL


def test_valid_calls_reach_the_device_check():
    for call in (_decode, _prefill, _append):
        if not torch.cuda.is_available():
            assert call() in (HIP, DEV)
            assert len(qg.lib().qgemm_last_error()) > 0
    # in place: q_out is q, inside a fused product that also holds k and v
    if not torch.cuda.is_available():
        assert _append(k=Q + 64 * 128 * 2, v=Q + 72 * 128 * 2, out=Q, ots=80 * 128) in (HIP, DEV)


def test_workspace_sizes_follow_the_split():
    dec, pre = qg.attn_decode_workspace_bytes, qg.attn_prefill_workspace_bytes
    try:
        qg.set_attn_splits(1)
        assert dec(1, 1 << 20, 64, 8, 128) == 0 and pre(1, 4096, 1 << 20, 64, 8, 128) == 0
        qg.set_attn_splits(4)
        # counters, then per part and row (max, sum) and head_dim sums of 4 bytes
        assert dec(2, 4096, 64, 8, 128) == 65536 + 2 * 8 * 4 * 8 * (8 + 512)
        assert pre(2, 5, 4096, 64, 8, 128) == 65536 + 2 * 8 * 4 * 40 * (8 + 512)
        qg.set_attn_splits(0)
        assert dec(1, 1 << 20, 64, 8, 128) > 0 and pre(1, 4, 1 << 20, 64, 8, 128) > 0
        # a window bounds the tokens that are worth splitting
        assert dec(1, 1 << 20, 64, 8, 128, 64, 4) < dec(1, 1 << 20, 64, 8, 128)
        # more row tiles than the workspace has counters: unsplit
        assert dec(65535, 4096, 8, 8, 128) == 0
        assert dec(0, 4096, 8, 8, 128) == 0 and pre(3, 0, 4096, 8, 8, 128) == 0
    finally:
        qg.set_attn_splits(0)
    for bad in (-1, 1025):
        with pytest.raises(qg.QgemmError):
            qg.set_attn_splits(bad)
    for args in ((-1, 1, 1, 1, 16), (1, -1, 1, 1, 16), (1, 1, 3, 2, 16), (1, 1, 1, 1, 8)):
        with pytest.raises(qg.QgemmError):
            dec(*args)


def test_rope_table():
    t = qg.rope_table(5, 4, theta=100.0)
    assert t.shape == (5, 4) and t.dtype == torch.float32
    a = torch.tensor([[p * 1.0, p * 0.1] for p in range(5)], dtype=torch.float64)
    assert torch.allclose(t.double(), torch.cat([a.cos(), a.sin()], dim=1), atol=1e-7)


def test_cache_binding_refuses_tensors_that_do_not_fit():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    for bad in (lambda: qg.KVCache(k, k), lambda: qg.KVCache(k[0], k[0]), lambda: qg.KVCache(k, k.bfloat16()),
                lambda: qg.KVCache(k, k[:2]), lambda: qg.KVCache(k.float(), k.float()),
                lambda: qg.KVCache(k, k.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            bad()


def _attn_struct(cache=None, **kw):
    a = dict(q=Q, qts=64 * 128, qhs=128, table=TABLE, cols=64, start=START, lens=LENS, seqs=4, tokens=40, max_q=20,
             max_len=1000, heads=64, act=F16, scale=0.1, window=0, sinks=0, out=OUT, ots=64 * 128, ohs=128, ws=WSP,
             wsb=1 << 30)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return c, attention._attn_call(
        a["q"] or 0, a["qts"], a["qhs"], ctypes.addressof(c), a["table"] or 0, a["cols"], a["start"] or 0,
        a["lens"] or 0, a["seqs"], a["tokens"], a["max_q"], a["max_len"], a["window"], a["out"] or 0, a["ots"],
        a["ohs"], a["ws"] or 0, a["wsb"], 0, a["heads"], a["act"], a["sinks"], a["scale"])


def _append_struct(cache=None, **kw):
    a = dict(q=Q, qts=80 * 128, qhs=128, k=K, kts=80 * 128, khs=128, v=V, vts=80 * 128, vhs=128, qn=NORM, kn=None,
             eps=1e-6, rope=ROPE, rows=4096, rot=128, inter=0, pos=POS, seq=None, table=TABLE, cols=64, seqs=4,
             tokens=10, heads=64, act=F16, out=OUT, ots=64 * 128, ohs=128)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return c, attention._append_call(
        a["q"] or 0, a["qts"], a["qhs"], a["k"] or 0, a["kts"], a["khs"], a["v"] or 0, a["vts"], a["vhs"],
        a["qn"] or 0, a["kn"] or 0, a["rope"] or 0, a["rows"], a["pos"] or 0, a["seq"] or 0, a["table"] or 0,
        a["cols"], a["seqs"], a["tokens"], ctypes.addressof(c), a["out"] or 0, a["ots"], a["ohs"], 0, a["rot"],
        a["inter"], a["heads"], a["act"], a["eps"])


# The calls by struct refuse what the calls by argument refuse: every field is where the library reads it.
@pytest.mark.parametrize("fault,status", ATTN_FAULTS)
def test_attention_faults_by_struct(fault, status):
    c, call = _attn_struct(**fault)
    for name in ("qgemm_attn_decode_call", "qgemm_attn_prefill_call"):
        assert getattr(qg.lib(), name)(call) == status, name


@pytest.mark.parametrize("fault,status", PREFILL_FAULTS)
def test_prefill_faults_by_struct(fault, status):
    c, call = _attn_struct(**fault)
    assert qg.lib().qgemm_attn_prefill_call(call) == status


def test_decode_by_struct_ignores_what_belongs_to_prefill():
    c, call = _attn_struct(start=START + 2, tokens=-1, max_q=-1, seqs=0)
    assert qg.lib().qgemm_attn_decode_call(call) == OK


@pytest.mark.parametrize("fault,status", APPEND_FAULTS)
def test_append_faults_by_struct(fault, status):
    c, call = _append_struct(**fault)
    assert qg.lib().qgemm_qk_rope_append_call(call) == status


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_faults_by_struct(fault, status):
    c, call = _attn_struct(_cache(**fault))
    assert qg.lib().qgemm_attn_decode_call(call) == status
    assert qg.lib().qgemm_attn_prefill_call(call) == status
    c, call = _append_struct(_cache(**fault))
    assert qg.lib().qgemm_qk_rope_append_call(call) == status


def test_null_structs():
    for name in ("qgemm_attn_decode_call", "qgemm_attn_prefill_call", "qgemm_qk_rope_append_call"):
        assert getattr(qg.lib(), name)(None) == NULL
