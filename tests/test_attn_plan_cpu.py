"""CPU tests of the attention planner over the whole range of the arguments that the entry points accept: windows and
sinks beyond the context mean what the context's length means, whatever their size. No kernel is launched."""

import pytest

import bit_weight_quantized_qgemm_amd as qg

WINDOW_MAX, SINKS_MAX = 2 ** 63 - 1, 2 ** 31 - 1
# seqs, max_q, max_len, q heads, kv heads, head_dim
SHAPES = [(1, 1, 131072, 64, 8, 128), (1, 5, 131072, 64, 8, 128), (4, 128, 6001, 32, 32, 64), (2, 300, 1 << 24, 8, 1, 256),
          (1, 1 << 20, 1 << 20, 8, 8, 128), (3, 7, 129, 4, 2, 128), (2, 3, 1, 4, 2, 128), (2, 3, 0, 4, 2, 128)]


@pytest.fixture(autouse=True)
def _automatic_splits():
    qg.set_attn_splits(0)
    yield
    qg.set_attn_splits(0)


def _sizes(shape, window, sinks):
    seqs, max_q, max_len, heads, kv_heads, dim = shape
    return (qg.attn_decode_workspace_bytes(seqs, max_len, heads, kv_heads, dim, window, sinks),
            qg.attn_prefill_workspace_bytes(seqs, max_q, max_len, heads, kv_heads, dim, window, sinks))


@pytest.mark.parametrize("splits", [0, 4, 1024])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_window_beyond_the_context_is_none(shape, splits):
    qg.set_attn_splits(splits)
    plain = _sizes(shape, 0, 0)
    for window in [max(1, shape[2]), shape[2] + 1] + [WINDOW_MAX - n for n in (0, 1, 29, 30, 31, 157, 158, 1 << 20)]:
        for sinks in (0, 4, SINKS_MAX):
            assert _sizes(shape, window, sinks) == plain, (window, sinks)


@pytest.mark.parametrize("splits", [0, 4, 1024])
@pytest.mark.parametrize("shape", SHAPES)
def test_sinks_beyond_the_context_are_all_of_it(shape, splits):
    qg.set_attn_splits(splits)
    for window in (1, 100, 4096):
        whole = _sizes(shape, window, shape[2])
        for sinks in [shape[2] + 1] + [SINKS_MAX - n for n in (0, 1, 14, 15, 16, 1 << 20)]:
            assert _sizes(shape, window, sinks) == whole, (window, sinks)


def test_long_contexts_stay_split_under_any_mask_that_shows_them():
    for window, sinks in ((0, 0), (131072, 0), (WINDOW_MAX, 0), (4096, 131072), (4096, SINKS_MAX), (1, SINKS_MAX)):
        dec, pre = _sizes(SHAPES[0], window, sinks)
        assert dec > 0 and pre > 0, (window, sinks)


def test_strides_along_one_token_head_or_page_are_not_used():
    import torch
    from test_attn_abi_cpu import DEV, FP8, HIP, _append, _cache, _decode, _prefill

    if torch.cuda.is_available():
        pytest.skip("the addresses are not a device's")
    one = dict(num_pages=1, page_stride=-3, kv_heads=1, head_stride=1)
    for cache in (_cache(**one), _cache(**one, dtype=FP8)):
        for odd in (1, -1, 7, (1 << 40) + 1):
            assert _decode(cache, seqs=1, heads=1, cols=1, max_len=16, qts=odd, qhs=odd, ots=odd, ohs=odd) in (HIP, DEV)
            assert _prefill(cache, seqs=1, tokens=1, heads=1, cols=1, max_len=16, qts=odd, qhs=odd, ots=odd,
                            ohs=odd) in (HIP, DEV)
            assert _append(cache, tokens=1, heads=1, cols=1, qts=odd, qhs=odd, kts=odd, khs=odd, vts=odd, vhs=odd,
                           ots=odd, ohs=odd) in (HIP, DEV)
