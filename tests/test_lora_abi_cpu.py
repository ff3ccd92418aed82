"""CPU tests of the low-rank adapters' entry points: arguments are validated before any HIP call, plans and workspaces are
sized for the largest case, and the binding refuses tensors that do not fit. No kernel is launched."""

import ctypes

import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from bit_weight_quantized_qgemm_amd.lora import MAX_SLICES, _AdaptersStruct, _lora_call

OK, NULL, SHAPE, ALIGN, WS, RANGE, ALIAS, HIP, DEV, SIZE = 0, -1, -2, -3, -4, -6, -7, -8, -9, -10
X, A, B, BASE, OUT, PLAN, WSP, SC, RK, IDS = (0x100000000 * i for i in range(1, 11))


def plan_bytes(T, n):
    got = ctypes.c_size_t(0)
    assert qg.lib().qgemm_lora_plan_bytes(T, n, ctypes.byref(got)) == OK
    return got.value


def _call(w=None, **kw):
    f = dict(a=A, b=B, a_stride=16 * 1024, b_stride=512 * 16, scales=SC, ranks=RK, K=1024, N=512,
             widths=[256, 128, 128], num_adapters=10, rank=16, slices=3, dtype=qg.DT_F16)
    f["a_stride"] = 3 * 16 * 1024
    f.update(w or {})
    widths = (ctypes.c_int64 * MAX_SLICES)(*f.pop("widths"))
    st = _AdaptersStruct(*(widths if n == "widths" else f[n] for n, _ in _AdaptersStruct._fields_))
    g = dict(x=X, xs=1024, plan=PLAN, pb=None, base=BASE, bs=512, out=OUT, os=512, T=100, ws=WSP, wsb=1 << 30)
    g.update(kw)
    if g["pb"] is None:
        g["pb"] = plan_bytes(g["T"], st.num_adapters) if 0 <= g["T"] <= 65535 and 1 <= st.num_adapters <= 4096 else 64
    return qg.lib().qgemm_lora(_lora_call(ctypes.addressof(st), g["x"], g["xs"], g["plan"], g["pb"], g["base"], g["bs"],
                                          g["out"], g["os"], g["T"], g["ws"], g["wsb"], 0))


NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are good: with a GPU the call would run")


@NO_GPU
def test_good_arguments_reach_the_device_check():
    assert _call() in (DEV, HIP)
    assert _call(base=0) in (DEV, HIP)
    assert _call(out=BASE) in (DEV, HIP)   # in place
    assert _call(w=dict(scales=0, ranks=0)) in (DEV, HIP)
    assert _call(T=1, xs=7, os=3, base=0) in (DEV, HIP)   # one row: its stride is not used
    assert _call(w=dict(num_adapters=1, a_stride=0, b_stride=0)) in (DEV, HIP)


ADAPTER_FAULTS = [
    (dict(K=0), SHAPE), (dict(K=1020), SHAPE), (dict(K=(1 << 20) + 8), SHAPE), (dict(N=0), SHAPE), (dict(N=516), SHAPE),
    (dict(rank=0), SHAPE), (dict(rank=12), SHAPE), (dict(rank=264), SHAPE), (dict(slices=0), SHAPE), (dict(slices=9), SHAPE),
    (dict(widths=[256, 128, 120]), SHAPE), (dict(widths=[260, 124, 128]), SHAPE), (dict(widths=[512, 0, 0]), SHAPE),
    (dict(widths=[520, -8, 0]), SHAPE), (dict(num_adapters=0), SHAPE), (dict(num_adapters=4097), SHAPE),
    (dict(num_adapters=-1), SHAPE), (dict(dtype=0), RANGE), (dict(dtype=qg.DT_FP8), RANGE), (dict(a=0), NULL), (dict(b=0), NULL),
    (dict(a=A + 8), ALIGN), (dict(b=B + 8), ALIGN), (dict(scales=SC + 2), ALIGN), (dict(ranks=RK + 2), ALIGN),
    (dict(a_stride=3 * 16 * 1024 - 8), ALIGN), (dict(a_stride=3 * 16 * 1024 + 4), ALIGN), (dict(b_stride=512 * 16 - 8), ALIGN),
    (dict(b_stride=-512 * 16), ALIGN), (dict(b_stride=(1 << 32) + 8), ALIGN),
]


@pytest.mark.parametrize("fault,status", ADAPTER_FAULTS)
def test_adapter_faults(fault, status):
    assert _call(w=fault) == status


CALL_FAULTS = [
    (dict(T=-1), SHAPE), (dict(T=65536), SHAPE), (dict(x=0), NULL), (dict(out=0), NULL), (dict(plan=0), NULL), (dict(ws=0), NULL),
    (dict(x=X + 8), ALIGN), (dict(out=OUT + 2), ALIGN), (dict(base=BASE + 4), ALIGN), (dict(plan=PLAN + 4), ALIGN),
    (dict(ws=WSP + 8), ALIGN), (dict(xs=1020), ALIGN), (dict(xs=1016), ALIGN), (dict(os=504), ALIGN), (dict(bs=508), ALIGN),
    (dict(xs=(1 << 32) + 8), ALIGN), (dict(xs=-1024), ALIGN), (dict(pb=64), SIZE), (dict(wsb=4096), WS),
    (dict(out=X), ALIAS), (dict(out=A), ALIAS), (dict(out=B + 512), ALIAS), (dict(out=SC), ALIAS), (dict(out=RK), ALIAS),
    (dict(out=PLAN), ALIAS), (dict(out=WSP + (1 << 16)), ALIAS), (dict(out=BASE + 16), ALIAS), (dict(out=BASE, os=520), ALIAS),
    (dict(ws=X), ALIAS), (dict(ws=BASE), ALIAS), (dict(ws=A), ALIAS), (dict(ws=PLAN), ALIAS), (dict(T=0), OK),
]


@pytest.mark.parametrize("fault,status", CALL_FAULTS)
def test_call_faults(fault, status):
    assert _call(**fault) == status


def test_null_struct():
    assert qg.lib().qgemm_lora(None) == NULL
    assert _lora_call(0, *[0] * 12) and qg.lib().qgemm_lora(_lora_call(0, *[0] * 12)) == NULL


PLAN_FAULTS = [(dict(T=-1), SHAPE), (dict(T=65536), SHAPE), (dict(n=0), SHAPE), (dict(n=4097), SHAPE), (dict(ids=0), NULL),
               (dict(plan=0), NULL), (dict(ids=IDS + 2), ALIGN), (dict(plan=PLAN + 8), ALIGN), (dict(pb=16), SIZE),
               (dict(plan=IDS), ALIAS), (dict(T=0), OK)]


@pytest.mark.parametrize("fault,status", PLAN_FAULTS)
def test_plan_faults(fault, status):
    a = dict(ids=IDS, T=100, n=10, plan=PLAN, pb=plan_bytes(100, 10))
    a.update(fault)
    assert qg.lib().qgemm_lora_plan(a["ids"], a["T"], a["n"], a["plan"], a["pb"], None) == status


@pytest.mark.parametrize("T", [1, 15, 16, 64, 100, 256, 257, 5000, 65535])
@pytest.mark.parametrize("n", [1, 2, 63, 4096])
def test_plans_hold_the_most_tiles(T, n):
    # the worst case: as many runs of one row as there are adapters (and rows without one), the rest in one run
    buckets = min(T, n + 1)
    tiles = {r: (buckets - 1) + -(-(T - (buckets - 1)) // r) for r in (16, 64)}
    words = plan_bytes(T, n) // 4
    assert words >= 16 + T + 4 * (tiles[16] + tiles[64])
    assert words <= 16 + T + 3 + 4 * (T // 16 + T // 64 + 2 * buckets)


def test_workspace_sizes():
    for args in ((1, 8, 4096, 4096, 16, 1), (64, 66, 8192, 10240, 16, 3), (1003, 7, 4096, 11008, 64, 1),
                 (8192, 5, 8192, 8192, 16, 1), (65535, 4096, 8192, 8192, 256, 8)):
        T, n, K, N, r, s = args
        got = qg.lora_workspace_bytes(*args)
        y = 4 * T * s * -(-r // 16) * 16
        assert got >= 65536 + y
        # parts of K: whole fragments for every tile, at most 1024 workgroups' worth of 16 KB
        assert got <= 65536 + y + 256 + 1024 * 16384
    assert qg.lora_workspace_bytes(0, 1, 64, 64, 8, 1) == 0
    for bad in ((-1, 1, 64, 64, 8, 1), (1, 0, 64, 64, 8, 1), (1, 1, 60, 64, 8, 1), (1, 1, 64, 60, 8, 1), (1, 1, 64, 64, 9, 1),
                (1, 1, 64, 64, 8, 9)):
        with pytest.raises(qg.QgemmError):
            qg.lora_workspace_bytes(*bad)


def test_binding_refuses_what_does_not_fit():
    half = torch.zeros((4, 16, 64), dtype=torch.float16)
    for a, b in ((half.float(), half.float()), (half, half.bfloat16()), (half, half)):   # the last: not on a GPU
        with pytest.raises(ValueError):
            qg.LoraAdapters(a, b)
    with pytest.raises(ValueError):
        qg.LoraBatch(torch.zeros(4, dtype=torch.int32), 4)


def test_struct_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qgemm.h"\nint main(void) { printf("%zu %zu %zu %zu",'
                   ' sizeof(qgemm_lora_adapters), offsetof(qgemm_lora_adapters, widths),'
                   ' sizeof(qgemm_lora_call), offsetof(qgemm_lora_call, stream)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    size = len(_lora_call(*[0] * 13))
    assert got == [ctypes.sizeof(_AdaptersStruct), _AdaptersStruct.widths.offset, size, size - 8]
