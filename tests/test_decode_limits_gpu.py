"""The calls after a context at the ends of their ranges."""
import pytest
import torch

import context_zigzag_cp_b200 as cz
from test_kv4_gpu import check_attn, filled, i32, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,T", [([500], 1024), ([1], 4), ([3, 0, 90], 8), ([700], 2)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 1024])
def test_windows_that_reach_beyond_every_key(lens, T, window):
    """A window that is written for "no limit", over sequences that may be shorter than their query tokens: bit for
    bit the call without a window."""
    pages, table = filled(lens, 1, 64, 32, 1)
    q = rows(len(lens), 1, T, 64, 2)
    got = cz.attn_kv4(q.cuda(), pages, table, i32(lens), window=window)
    want = cz.attn_kv4(q.cuda(), pages, table, i32(lens))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_attn(q, pages, table, lens, *got, window=window)
    assert cz.get_device_status() == 0
