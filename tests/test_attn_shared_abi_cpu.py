"""CPU tests of the entry points for shared tokens: arguments are validated before any HIP call, and workspaces hold every
part that the kernels may write. No kernel is launched."""

import ctypes

import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from bit_weight_quantized_qgemm_amd.attention import _attn_call, _shared_call
from test_attn_abi_cpu import (ALIAS, ALIGN, ATTN_FAULTS, CACHE_FAULTS, DEV, HIP, NULL, OK, OUT, PREFILL_FAULTS, Q, RANGE, SHAPE,
                               START, TABLE, LENS, WS, WSP, F16, _cache)

GROUPS, SHARED = 0xE0000000, 0xF0000000


@pytest.fixture(autouse=True)
def _modes():
    qg.set_attn_splits(0)
    qg.set_attn_sharing(1)
    yield
    qg.set_attn_splits(0)
    qg.set_attn_sharing(0)


def _call(prefill, cache=None, **kw):
    a = dict(q=Q, qts=64 * 128, qhs=128, table=TABLE, cols=64, start=START, lens=LENS, seqs=4, tokens=40, max_q=20,
             max_len=1000, heads=64, act=F16, scale=0.1, window=0, sinks=0, out=OUT, ots=64 * 128, ohs=128, ws=WSP,
             wsb=1 << 40, groups=GROUPS, shared=SHARED, n=2, max_shared=512)
    a.update(kw)
    c = cache if cache is not None else _cache()
    z = {k: 0 if v is None else v for k, v in a.items()}
    fn = qg.lib().qgemm_attn_prefill_shared if prefill else qg.lib().qgemm_attn_decode_shared
    return fn(_shared_call(z["q"], z["qts"], z["qhs"], ctypes.addressof(c), z["table"], z["cols"], z["start"], z["lens"], z["seqs"],
                           z["tokens"], z["max_q"], z["max_len"], z["window"], z["out"], z["ots"], z["ohs"], z["ws"],
                           z["wsb"], 0, z["heads"], z["act"], z["sinks"], z["scale"], z["groups"], z["shared"], z["n"],
                           z["max_shared"]))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are good: with a GPU the call would run")
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_good_arguments_reach_the_device_check(mode):
    qg.set_attn_sharing(mode)
    for prefill in (False, True):
        assert _call(prefill) in (DEV, HIP)
        assert _call(prefill, n=0, groups=0, shared=0) in (DEV, HIP)
        assert _call(prefill, max_shared=0) in (DEV, HIP)
        assert _call(prefill, max_shared=1 << 62) in (DEV, HIP)


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_faults(fault, status):
    for prefill in (False, True):
        assert _call(prefill, _cache(**fault)) == status


@pytest.mark.parametrize("fault,status", ATTN_FAULTS)
def test_attention_faults(fault, status):
    for prefill in (False, True):
        assert _call(prefill, **fault) == status


@pytest.mark.parametrize("fault,status", PREFILL_FAULTS)
def test_prefill_faults(fault, status):
    assert _call(True, **fault) == status


GROUP_FAULTS = [(dict(n=-1), SHAPE), (dict(n=65536), SHAPE), (dict(max_shared=-1), SHAPE), (dict(groups=0), NULL),
                (dict(shared=0), NULL), (dict(groups=GROUPS + 2), ALIGN), (dict(shared=SHARED + 1), ALIGN),
                (dict(out=GROUPS), ALIAS), (dict(out=SHARED), ALIAS), (dict(ws=GROUPS), ALIAS), (dict(ws=SHARED), ALIAS),
                (dict(seqs=0), OK)]


@pytest.mark.parametrize("fault,status", GROUP_FAULTS)
def test_group_faults(fault, status):
    for prefill in (False, True):
        assert _call(prefill, **fault) == status


def test_null_struct_and_modes():
    assert qg.lib().qgemm_attn_decode_shared(None) == NULL
    assert qg.lib().qgemm_attn_prefill_shared(None) == NULL
    for mode in (-1, 3):
        assert qg.lib().qgemm_attn_set_sharing(mode) == RANGE


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
@pytest.mark.parametrize("splits", [0, 1, 7, 1024])
@pytest.mark.parametrize("seqs,groups,max_shared,max_len,H,KV,D,new", [
    (4, 1, 768, 898, 32, 32, 128, 5), (64, 1, 8192, 8704, 64, 8, 128, 1), (101, 4, 4096, 4800, 32, 8, 128, 3),
    (1, 1, 16, 16, 1, 1, 16, 1), (300, 150, 1 << 20, 1 << 24, 128, 1, 256, 40), (65535, 65535, 64, 128, 8, 8, 64, 1)])
def test_workspaces_hold_every_part(seqs, groups, max_shared, max_len, H, KV, D, new, splits, window, sinks):
    """Counters; statistics and sums of every row (token and head) for each part of the shared tokens, all parts of whole
    tiles of keys, and for at least one part of the own ones; the plain call's own parts."""
    qg.set_attn_splits(splits)
    for prefill in (False, True):
        tokens = seqs * new if prefill else seqs
        if tokens > 1 << 20:
            continue
        args = (seqs, tokens, new, max_len) if prefill else (seqs, max_len)
        size = qg.attn_prefill_shared_workspace_bytes if prefill else qg.attn_decode_shared_workspace_bytes
        got = size(*args, H, KV, D, window, sinks, groups, max_shared)
        blocks = max_shared // 16
        parts = min(splits or 1, blocks)
        step = 4 if D <= 128 else 2
        per = -(-(-(-blocks // parts)) // step) * step
        parts = -(-blocks // per)
        least = 65536 + tokens * H * (parts + 1) * (D + 2) * 4
        assert got >= least
        assert qg.lib().qgemm_attn_set_sharing(2) == OK
        plain = size(*args, H, KV, D, window, sinks, groups, max_shared)
        without = (qg.attn_prefill_workspace_bytes(seqs, new, max_len, H, KV, D, window, sinks) if prefill else
                   qg.attn_decode_workspace_bytes(seqs, max_len, H, KV, D, window, sinks))
        assert plain == without
        qg.set_attn_sharing(1)


@pytest.mark.parametrize("seqs,new,max_len,max_shared", [(32, 4096, 12400, 8192), (64, 8192, 40000, 32000),
                                                         (1000, 4096, 70000, 65536), (500, 1, 9000, 8192)])
@pytest.mark.parametrize("mode", [0, 1], ids=["automatic", "shared"])
def test_one_long_prompt_among_single_tokens(mode, seqs, new, max_len, max_shared):
    """Memory goes by the rows that there are, not by the longest prompt times the sequences, nor by tiles of groups with few
    rows: one place per row, with sums and statistics, in each of at most 64 parts (of 256 workgroups' worth of tiles) of the
    shared and as many of the own tokens."""
    H, KV, D, tokens = 64, 8, 128, seqs - 1 + new
    qg.set_attn_sharing(mode)
    got = qg.attn_prefill_shared_workspace_bytes(seqs, tokens, new, max_len, H, KV, D, 0, 0, seqs // 2, max_shared)
    one = tokens * H * (D + 2) * 4
    tiles = (seqs // 2 + tokens * H // KV // 128) * KV
    parts = max(1, -(-8 * 256 // tiles))
    assert got <= 65536 + 4 * 256 + 2 * parts * one


def test_small_workspaces_are_refused():
    for prefill in (False, True):
        size = (qg.attn_prefill_shared_workspace_bytes(4, 40, 20, 1000, 64, 8, 128, 0, 0, 2, 512) if prefill else
                qg.attn_decode_shared_workspace_bytes(4, 1000, 64, 8, 128, 0, 0, 2, 512))
        assert _call(prefill, wsb=size - 1) == WS
        if not torch.cuda.is_available():
            assert _call(prefill, wsb=size) in (DEV, HIP)


def test_struct_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qgemm.h"\nint main(void) { printf("%zu %zu %zu",'
                   ' sizeof(qgemm_attn_call), offsetof(qgemm_attn_shared_call, group_start), sizeof(qgemm_attn_shared_call));'
                   ' return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    plain = len(_attn_call(*[0] * 23))
    assert got == [plain, plain, len(_shared_call(*[0] * 27))]
