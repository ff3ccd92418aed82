"""The low-rank adapters against the fp64 oracle: sizes, types, orders of the ids, ranks, slices, strides, and the calls
around them (in place, updates, streams, graphs). Bounds are the oracle's, from the roundings of the formula."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import NAN, to_bits, to_torch
from lora_problem import Pool, check, guarded, untouched, values
from oracle import attention as oa
from oracle import lora as lora_oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


def _say(*a):
    print("[case]", *a, flush=True)


def _ids(rng, T, n, kind):
    if kind == "one":
        return np.full(T, n - 1)
    if kind == "none":
        return np.full(T, -1)
    if kind == "sorted":
        return np.sort(rng.integers(0, n, T))
    if kind == "own":   # a different one for each row, as far as they go
        return np.arange(T) % n
    ids = rng.integers(0, n, T)
    out = [-1, n, n + 5, INT_MIN, INT_MAX]
    for i, bad in enumerate(out):
        ids[rng.random(T) < 0.04] = bad
    return ids


def _batch(ids, n):
    return qg.LoraBatch(torch.tensor(ids, dtype=torch.int32, device=DEV), n)


def _run(rng, T, K, widths, rank, n, fmt, kind, ranks=None, gap=0, with_base=True, **pool):
    _say(T, K, widths, rank, n, fmt, kind, ranks, gap)
    p = Pool(rng, n, K, widths, rank, fmt, DEV, ranks=ranks, gap=gap, **pool)
    ids = _ids(rng, T, n, kind)
    x_bits, x = values(rng, (T, K), fmt)
    base_bits, base = values(rng, (T, p.N), fmt)
    xd, _ = guarded(T, K, fmt, DEV, gap, x_bits, NAN[fmt])
    bd, _ = guarded(T, p.N, fmt, DEV, gap, base_bits, NAN[fmt])
    od, buf = guarded(T, p.N, fmt, DEV, gap)
    got = qg.lora(xd, p.adapters, _batch(ids, n), base=bd if with_base else None, out=od)
    torch.cuda.synchronize()
    assert got is od
    ref, bound = p.expected(x, ids, base if with_base else None)
    check(od, ref, bound, fmt, (T, K, widths, rank, n, fmt, kind))
    assert untouched(buf, T, p.N, gap)
    return p, ids, (x_bits, xd), (base_bits, bd), od


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65])
def test_small_batches(T, fmt):
    rng = np.random.default_rng(T)
    _run(rng, T, 256, [192], 16, 5, fmt, "mixed")
    _run(rng, T, 128, [64], 8, 70, fmt, "own", with_base=False)


@pytest.mark.parametrize("T", [255, 256, 257, 300, 517])
def test_the_change_to_tall_tiles(T):
    rng = np.random.default_rng(T)
    _run(rng, T, 160, [136], 24, 3, "f16", "mixed")
    _run(rng, T, 96, [72], 8, 2, "bf16", "sorted")
    _run(rng, T, 64, [64], 16, 300, "f16", "own")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("T,rank", [(769, 40), (800, 64), (1025, 16), (1100, 72), (1030, 128), (1040, 136), (1025, 256),
                                    (2561, 8), (2600, 32), (2700, 24)])
def test_tall_tiles(T, rank, fmt):
    """Tiles of 64 rows in the first product, the second, and both; the last ones part empty."""
    rng = np.random.default_rng(T + rank)
    _run(rng, T, 104, [72, 136], rank, 5, fmt, "sorted", gap=8)


def test_tall_tiles_of_many_kinds():
    rng = np.random.default_rng(77)
    _run(rng, 1200, 64, [64], 64, 7, "bf16", "mixed", ranks=[64, 8, 0, 17, 33, 64, 1])
    _run(rng, 2600, 32, [16, 40], 16, 900, "f16", "mixed")
    _run(rng, 1300, 2056, [24], 48, 3, "f16", "one")
    _run(rng, 2570, 1032, [8] * 8, 8, 4, "bf16", "none")
    _run(rng, 1500, 40, [32, 32, 32, 32, 32, 32, 32, 32], 40, 6, "f16", "own", with_base=False)


@pytest.mark.parametrize("K", [8, 24, 32, 40, 120, 128, 136, 1000, 2056, 4096])
def test_inner_lengths(K):
    rng = np.random.default_rng(K)
    _run(rng, 5, K, [64], 16, 3, "f16", "mixed")
    _run(rng, 270, K, [64], 8, 2, "bf16", "mixed")


@pytest.mark.parametrize("widths", [[8], [16], [56], [64], [72], [120, 8, 200], [64, 64], [1000, 8, 8, 8, 136, 64, 24, 40]],
                         ids=str)
def test_column_ranges(widths):
    rng = np.random.default_rng(sum(widths))
    _run(rng, 7, 64, widths, 16, 3, "bf16", "mixed")
    _run(rng, 261, 64, widths, 24, 3, "f16", "mixed")


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128, 136, 256])
def test_ranks(rank):
    rng = np.random.default_rng(rank)
    _run(rng, 9, 128, [136], rank, 3, "f16", "mixed")
    _run(rng, 260, 64, [72, 64], rank, 3, "bf16", "mixed")


@pytest.mark.parametrize("rank,ranks", [(64, [64, 8, 0, 17, 33, 64, 1]), (16, [16, 8, 0, -5]), (256, [8, 200, 256, 1000]),
                                        (40, [40, 24, 7])], ids=str)
@pytest.mark.parametrize("T", [20, 290])
def test_adapters_of_different_ranks(T, rank, ranks):
    rng = np.random.default_rng(rank + T)
    _run(rng, T, 96, [64, 40], rank, len(ranks), "f16", "mixed", ranks=ranks)
    _run(rng, T, 64, [64], rank, len(ranks), "bf16", "own", ranks=ranks)


@pytest.mark.parametrize("kind", ["one", "none", "sorted", "own", "mixed"])
@pytest.mark.parametrize("T", [40, 400])
def test_orders_of_the_ids_and_strides(T, kind):
    rng = np.random.default_rng(T)
    _run(rng, T, 72, [88], 16, 6, "bf16", kind, gap=24)
    _run(rng, T, 72, [88], 16, 6, "f16", kind, gap=8, with_base=False, scaled=False)


def test_many_adapters():
    rng = np.random.default_rng(1)
    _run(rng, 600, 16, [16], 8, 4096, "f16", "mixed")
    _run(rng, 30, 16, [16], 8, 4096, "f16", "mixed")


def test_a_long_projection_in_parts():
    # few rows: K is split over workgroups and waves; the sums' order is the kernel's, within the bound
    rng = np.random.default_rng(2)
    _run(rng, 1, 28672, [1024], 16, 2, "f16", "one")
    _run(rng, 3, 11008, [64], 64, 2, "bf16", "own")
    _run(rng, 1003, 4096, [128], 64, 5, "f16", "sorted")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("a_dev,b_dev", [(3e3, 1e-6), (1e-6, 3e2), (1e-7, 1e-3)])
def test_products_beyond_16_bits(fmt, a_dev, b_dev):
    """A x lies far outside fp16's range, or far below its smallest values, on the way to an ordinary result."""
    rng = np.random.default_rng(3)
    _run(rng, 20, 512, [64], 16, 3, fmt, "mixed", a_dev=a_dev, b_dev=b_dev, with_base=False)


def test_in_place_equals_out_of_place():
    rng = np.random.default_rng(4)
    for T in (13, 300, 2600):
        p, ids, (_, xd), (base_bits, bd), od = _run(rng, T, 128, [64, 72], 16, 4, "f16", "mixed")
        y, buf = guarded(T, p.N, "f16", DEV, 16, base_bits)
        assert qg.lora(xd, p.adapters, _batch(ids, 4), base=y, out=y) is y
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), od.view(torch.int16)) and untouched(buf, T, p.N, 16)
        fresh = qg.lora(xd, p.adapters, _batch(ids, 4), base=bd)
        assert fresh.is_contiguous() and torch.equal(fresh.view(torch.int16), od.view(torch.int16))


def test_rows_without_an_adapter_keep_every_bit_of_their_base():
    rng = np.random.default_rng(5)
    for T in (9, 400):
        p = Pool(rng, 2, 64, [72], 8, "f16", DEV)
        base = to_torch(rng.integers(0, 65536, (T, 72)).astype(np.uint16), "f16", DEV)   # any bits, NaN and infinities too
        x = to_torch(oa.encode(rng.standard_normal((T, 64)), "f16"), "f16", DEV)
        ids = np.where(np.arange(T) % 3 == 0, 0, -1)
        out = qg.lora(x, p.adapters, _batch(ids, 2), base=base)
        keep = ids < 0
        assert np.array_equal(to_bits(out)[keep], to_bits(base)[keep])
        none = qg.lora(x, p.adapters, _batch(np.full(T, -1), 2))
        assert not to_bits(none).any()


def test_rows_do_not_influence_each_other():
    rng = np.random.default_rng(6)
    for T in (24, 330, 2700):
        p = Pool(rng, 3, 192, [136], 24, "bf16", DEV)
        ids = rng.integers(-1, 3, T)
        x_bits, _ = values(rng, (T, 192), "bf16")
        x = to_torch(x_bits, "bf16", DEV)
        want = to_bits(qg.lora(x, p.adapters, _batch(ids, 3)))
        # the same rows in another order
        order = rng.permutation(T)
        moved = to_bits(qg.lora(x[torch.from_numpy(order).to(DEV)].contiguous(), p.adapters, _batch(ids[order], 3)))
        assert np.array_equal(moved, want[order])
        # NaN and infinity in one row
        x_bits[T // 2, 5], x_bits[T // 3, 7] = NAN["bf16"], 0x7F80
        got = to_bits(qg.lora(to_torch(x_bits, "bf16", DEV), p.adapters, _batch(ids, 3)))
        rest = np.ones(T, dtype=bool)
        rest[[T // 2, T // 3]] = False
        assert np.array_equal(got[rest], want[rest])


@pytest.mark.parametrize("T", [3, 1100])
@pytest.mark.parametrize("rank", [8, 16, 24, 72])
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_infinite_sums_stay_infinite(T, rank, fmt):
    """Where every term of a sum has one sign the formula gives an infinity, not NaN; zeros times it give NaN."""
    _say("infinite", T, rank, fmt)
    dtype = torch.float16 if fmt == "f16" else torch.bfloat16
    K, N = 72, 24
    x = torch.ones(T, K, dtype=dtype, device=DEV)
    x[0, 3], x[2, 5] = float("inf"), -float("inf")
    a = torch.full((1, rank, K), 0.5, dtype=dtype, device=DEV)
    b = torch.full((1, N, rank), 0.25, dtype=dtype, device=DEV)
    b[0, 1::3], b[0, 2::3] = -0.25, 0.0
    out = qg.lora(x, qg.LoraAdapters(a, b), _batch(np.zeros(T, np.int64), 1)).float().cpu()
    part = K * 0.5 * 0.25 * rank   # exact in both formats
    ref = torch.tensor([part, -part, 0.0]).repeat(N // 3).expand(T, N).clone()
    ref[0] = torch.tensor([float("inf"), -float("inf"), float("nan")]).repeat(N // 3)
    ref[2] = torch.tensor([-float("inf"), float("inf"), float("nan")]).repeat(N // 3)
    assert torch.equal(torch.nan_to_num(out, nan=123.0), torch.nan_to_num(ref, nan=123.0))


def test_other_adapters_are_not_read():
    rng = np.random.default_rng(7)
    p = Pool(rng, 4, 64, [64], 16, "f16", DEV, gap=8)
    p.adapters.a[2].fill_(float("nan"))
    p.adapters.b[2].fill_(float("nan"))
    for T in (12, 280, 2590):
        ids = rng.choice([0, 1, 3, -1], T)
        x_bits, x = values(rng, (T, 64), "f16")
        out = qg.lora(to_torch(x_bits, "f16", DEV), p.adapters, _batch(ids, 4))
        check(out, *p.expected(x, ids), "f16", T)


def test_repeated_calls_give_the_same_bits_and_leave_the_workspace_usable():
    rng = np.random.default_rng(8)
    ws = qg.Workspace()
    p = Pool(rng, 5, 1024, [256], 16, "f16", DEV)
    ids = rng.integers(0, 5, 50)
    x = to_torch(values(rng, (50, 1024), "f16")[0], "f16", DEV)
    first = qg.lora(x, p.adapters, _batch(ids, 5), workspace=ws)
    for _ in range(3):
        assert torch.equal(qg.lora(x, p.adapters, _batch(ids, 5), workspace=ws), first)
    counters = ws.get(1, DEV)[0][:65536]
    assert not counters.any()


def test_update_and_graphs():
    """A captured step of an update, a product on 4-bit weights and its adapters follows new ids and inputs."""
    rng = np.random.default_rng(9)
    T, K, N, n = 19, 256, 192, 4
    p = Pool(rng, n, K, [N], 16, "f16", DEV)
    codes = torch.from_numpy(rng.integers(0, 2 ** 32, (K // 8, N), dtype=np.uint64).astype(np.uint32).view(np.int32)).to(DEV)
    blob = qg.repack_w4a16(codes, torch.full((K // 128, N), 0.01, dtype=torch.float16, device=DEV))
    ids = torch.zeros(T, dtype=torch.int32, device=DEV)
    x = torch.zeros((T, K), dtype=torch.float16, device=DEV)
    y = torch.zeros((T, N), dtype=torch.float16, device=DEV)
    batch, ws, side = qg.LoraBatch(ids, n), qg.Workspace(), torch.cuda.Stream()

    def step(batch, out):
        qg.w4a16(x, blob, K, N, out=out, workspace=ws)
        return qg.lora(x, p.adapters, batch.update(ids), base=out, out=out, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(batch, y)
    for i in range(4):
        new = rng.integers(-1, n, T)
        ids.copy_(torch.from_numpy(new.astype(np.int32)))
        x.copy_(to_torch(values(rng, (T, K), "f16")[0], "f16", DEV))
        want = step(qg.LoraBatch(ids, n), torch.zeros_like(y))
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_another_stream():
    rng = np.random.default_rng(10)
    p = Pool(rng, 3, 512, [256], 16, "bf16", DEV)
    ids = rng.integers(0, 3, 70)
    x = to_torch(values(rng, (70, 512), "bf16")[0], "bf16", DEV)
    want = qg.lora(x, p.adapters, _batch(ids, 3))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = qg.lora(x, p.adapters, _batch(ids, 3))
    s.synchronize()
    assert torch.equal(got, want)


def test_calls_on_two_streams_at_once():
    """One batch and pool in two streams, whose calls overlap: each stream has a workspace of its own."""
    rng = np.random.default_rng(15)
    p = Pool(rng, 6, 4096, [2048], 16, "f16", DEV)
    ids = rng.integers(-1, 6, 96)
    xs = [to_torch(values(rng, (96, 4096), "f16")[0], "f16", DEV) for _ in range(2)]
    batch = _batch(ids, 6)
    want = [qg.lora(x, p.adapters, batch) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(qg.lora(xs[i], p.adapters, batch))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_one_row_against_every_adapter_of_a_batch():
    """The same row and adapter many times give the same bits wherever they stand."""
    rng = np.random.default_rng(16)
    p = Pool(rng, 3, 320, [200], 24, "bf16", DEV)
    for T in (37, 1290):
        row, _ = values(rng, (1, 320), "bf16")
        out = to_bits(qg.lora(to_torch(np.repeat(row, T, axis=0), "bf16", DEV), p.adapters, _batch(np.arange(T) % 3, 3)))
        for i in range(3):
            assert (out[i::3] == out[i]).all()


def test_empty_batches():
    rng = np.random.default_rng(11)
    p = Pool(rng, 3, 64, [64], 8, "f16", DEV)
    out = qg.lora(torch.empty((0, 64), dtype=torch.float16, device=DEV), p.adapters, _batch([], 3))
    assert out.shape == (0, 64)


def test_offsets_beyond_32_bits():
    """Adapters 4 GiB apart, and rows of x and out 2 GiB."""
    n, K, N, R, far = 2, 64, 64, 8, 1 << 31   # elements
    rng = np.random.default_rng(12)

    def spread(shape, stride, step):
        size = (shape[0] - 1) * stride + int(np.prod(shape[1:]))
        return torch.zeros(size, dtype=torch.float16, device=DEV).as_strided(shape, (stride, *step))

    a_bits, a = values(rng, (n, 1, R, K), "f16", 0.1)
    b_bits, b = values(rng, (n, N, R), "f16", 0.5)
    x_bits, x = values(rng, (4, K), "f16")
    av, bv = spread((n, 1, R, K), far, (R * K, K, 1)), spread((n, N, R), far, (R, 1))
    xv, out = (spread((4, 64), far // 2, (1,)) for _ in range(2))
    for t, bits in ((av, a_bits), (bv, b_bits), (xv, x_bits)):
        t.copy_(to_torch(bits, "f16", DEV))
    ids = [1, 0, -1, 1]
    got = qg.lora(xv, qg.LoraAdapters(av, bv), _batch(ids, n), out=out)
    check(got, *lora_oracle.lora(x, a, b, ids, "f16"), "f16", "far")


REFUSALS = [
    (lambda k: k.update(x=k["x"].float()), "x must be"), (lambda k: k.update(x=k["x"][:, :32]), "x must be"),
    (lambda k: k.update(x=k["x"].t().contiguous().t()), "contiguous"), (lambda k: k.update(x=k["x"].cpu()), "x must be"),
    (lambda k: k.update(base=k["x"][:5]), "base must be"), (lambda k: k.update(out=k["x"]), "out must be"),
    (lambda k: k.update(batch=_batch([0, 1], 3)), "rows"), (lambda k: k.update(batch=_batch([0] * 6, 2)), "adapters"),
    (lambda k: k.update(out=k["out"].view(torch.bfloat16)), "out must be"),
]


@pytest.mark.parametrize("fault,text", REFUSALS)
def test_refusals_of_the_binding(fault, text):
    rng = np.random.default_rng(13)
    p = Pool(rng, 3, 64, [72], 8, "f16", DEV)
    kw = dict(x=torch.zeros((6, 64), dtype=torch.float16, device=DEV), adapters=p.adapters, batch=_batch([0] * 6, 3),
              out=torch.zeros((6, 72), dtype=torch.float16, device=DEV))
    qg.lora(**kw)
    fault(kw)
    with pytest.raises(ValueError, match=text):
        qg.lora(**kw)


def test_overlaps_and_small_workspaces_are_refused():
    rng = np.random.default_rng(14)
    p = Pool(rng, 3, 64, [64], 8, "f16", DEV)
    buf = torch.zeros((8, 64), dtype=torch.float16, device=DEV)
    batch = _batch([0] * 6, 3)
    x = torch.zeros((6, 64), dtype=torch.float16, device=DEV)
    with pytest.raises(qg.QgemmError, match="ALIAS"):
        qg.lora(x, p.adapters, batch, base=buf[:6], out=buf[1:7])
    with pytest.raises(qg.QgemmError, match="ALIAS"):
        qg.lora(x, p.adapters, batch, out=x)
    with pytest.raises(qg.QgemmError, match="ALIGN"):
        qg.lora(buf.flatten()[4:4 + 6 * 64].view(6, 64), p.adapters, batch)

    class Small(qg.Workspace):
        def get(self, nbytes, device):
            return super().get(nbytes, device)[0], nbytes - 1
    with pytest.raises(qg.QgemmError, match="WORKSPACE"):
        qg.lora(x, p.adapters, batch, workspace=Small())
