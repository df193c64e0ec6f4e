"""What the calls after a context refuse, without a GPU."""
import pytest
import torch

import context_zigzag_cp_b200 as cz

bf16, i32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2.5])
def test_windows_that_32_bits_do_not_hold(window):
    """Refused by name, not cut to 32 bits (2^32 + 5 would be a window of 5)."""
    pages = torch.zeros(4, 2, cz.kv4_page_bytes(32, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="window"):
        cz.attn_kv4(torch.zeros(3, 4, 1, 64, dtype=bf16), pages, torch.zeros(3, 2, dtype=i32),
                    torch.zeros(3, dtype=i32), window=window)
