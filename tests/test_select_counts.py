"""CPU: page counts that 32 bits do not hold are refused before they are cut to 32 bits
(2^32 + 1 would be one page)."""
import pytest
import torch

import head_aware_paged_gb300 as H


class Reached(Exception):
    pass


@pytest.mark.parametrize("counts", [(1 << 32, 1, 1), (1, (1 << 32) + 1, 1), (1, 1, (1 << 33) + 7), (1 << 31, 0, 1),
                                    (-(1 << 31) - 1, 0, 1), (1, 0, -(1 << 32) + 1)])
def test_counts_past_32_bits(monkeypatch, counts):
    def load():
        raise Reached
    monkeypatch.setattr(H, "load", load)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(OverflowError):
        H.sp_attention_decode_select(0, 0, [0], q, *counts, q, stream=0)
    with pytest.raises(Reached):                                 # (others are the library's to refuse)
        H.sp_attention_decode_select(0, 0, [0], q, (1 << 31) - 1, -(1 << 31), 1, q, stream=0)
