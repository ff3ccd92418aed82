"""CPU tests of how shared-prefix decodes cut the tokens that a sequence does not share, as far as the workspace tells."""

import pytest

import bit_weight_quantized_qgemm_amd as qg


@pytest.fixture(autouse=True)
def _modes():
    qg.set_attn_splits(0)
    qg.set_attn_sharing(1)
    yield
    qg.set_attn_splits(0)
    qg.set_attn_sharing(0)


def _parts(seqs, max_len, max_shared, H=64, KV=8, D=128, window=0, groups=1):
    """Parts per row that the workspace has places for, shared and own ones: statistics and sums in fp32 behind the counters
    (up to four roundings to 256 bytes)."""
    size = qg.attn_decode_shared_workspace_bytes(seqs, max_len, H, KV, D, window, 0, groups, max_shared) - 65536
    one = seqs * H * (D + 2) * 4
    assert size % one <= 4 * 255
    return size // one


@pytest.mark.parametrize("seqs,KV,H", [(2, 8, 64), (3, 4, 4), (2, 32, 32), (4, 8, 64)])
def test_a_sequence_of_no_group_has_more_than_a_part(seqs, KV, H):
    """A bound of 64 tokens past the shared ones is one part for the sequences of the groups. One of no group has the whole
    context for itself, in as many parts as eight waves per compute unit (256 here) allow for all tiles of heads; the shared
    tokens have one part at least and at most one per unit, of one tile of rows per head."""
    got = _parts(seqs, 16384 + 64, 16384, H, KV, groups=1)
    own = min(8 * 256 // (seqs * KV), 128)
    assert own > 256 // KV
    assert 1 + own <= got <= 256 // KV + own + 1


def test_parts_have_128_tokens_at_least():
    for max_len in (128, 500, 1000, 5000):
        assert _parts(2, max_len, 64, groups=1) <= 1 + -(-max_len // 128)


def test_a_window_bounds_the_parts():
    # 200 tokens of a window are in at most 15 blocks of 16 (both ends cut), two parts
    assert _parts(2, 16384 + 64, 16384, window=200) <= 256 // 8 + 2


@pytest.mark.parametrize("seqs,new,KV,H", [(8, 16, 8, 64), (4, 32, 8, 64), (12, 10, 8, 64), (6, 16, 8, 64), (3, 32, 8, 64)])
def test_several_tokens_of_a_sequence_of_no_group_have_the_plain_parts(seqs, new, KV, H):
    """The same for several new tokens: own tokens have as many parts as the plain call makes of the whole context, next to
    a part of the shared ones at least; those have at most one workgroup per unit in all."""
    tokens, one, shared, bound = seqs * new, seqs * new * H * (128 + 2) * 4, 16384, 16384 + 64
    plain = (qg.attn_prefill_workspace_bytes(seqs, new, bound, H, KV, 128) - 65536) // one
    tiles = -(-tokens * H // KV // 128) * KV
    assert plain > 256 // tiles
    got = (qg.attn_prefill_shared_workspace_bytes(seqs, tokens, new, bound, H, KV, 128, 0, 0, 1, shared) - 65536) // one
    assert plain + 1 <= got <= plain + 256 // tiles
