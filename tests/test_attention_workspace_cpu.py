"""What the backward pass of attention needs beside its tensors, where a bias's partial sums are kept for many sequences, heads and distances."""
import ctypes

import pytest

import matrix_aware_optimizer_amd as mao


def _need(sequences, tokens, heads, reach, width=64, dtype=mao.MUON_BF16):
    at = [k << 44 for k in range(1, 24)]
    ld = heads * width
    a = mao.MuonAttentionBackwardArgs(*at[:16], tokens, tokens, sequences, *[ld, width] * 9, 0, 0.125, heads, heads, width, 8, reach, 1, dtype)
    need = mao.load().muon_attention_backward_workspace_bytes(ctypes.byref(a))
    assert need > 0, mao.muon_last_error_message()
    return need


@pytest.mark.parametrize("sequences,tokens,heads,reach", [(4000, 160000, 16, 1024), (4000, 160000, 16, 4096), (1 << 20, 1 << 22, 64, 4096), (12, 8192, 16, 4096),
                                                          (1, 1 << 20, 32, 4096)])
def test_the_biass_partial_sums_stay_within_half_a_gigabyte(sequences, tokens, heads, reach):
    # beside them: delta, sums of the distances, and parts of a split walk (none where there are this many units)
    rest = tokens * heads * 4 + heads * (2 * reach + 1) * 8 + 1024
    assert _need(sequences, tokens, heads, reach) <= (1 << 29) + rest


def test_they_take_what_they_need_where_that_is_less():
    small = _need(12, 8192, 16, 128)
    units = (8192 // 128 + 12 + 3) | 1
    assert small <= units * 4 * 16 * 257 * 4 + 8192 * 16 * 4 + 16 * 257 * 8 + 1024
