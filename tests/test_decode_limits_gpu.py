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


@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (3, 1, 1), (3, 4, 1), (3, 1, 5), (1, 1, 5), (1, 4, 1), (1, 4, 5)])
def test_in_place_where_an_extent_is_one(B, H, N):
    """A contiguous tensor is rotated in place whatever its extents: a step's token, one KV head."""
    D = 128
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    pos = torch.arange(7, 7 + N, dtype=torch.int32, device="cuda")[None]
    x, k = rows(B, H, N, D, 1).cuda(), rows(B, 2 * H, N, D, 2).cuda()
    for kw in (dict(), dict(stream=torch.cuda.current_stream())):
        want = cz.rope([x, k], f, positions=pos, **kw)
        y, z = x.clone(), k.clone()
        back = cz.rope([y, z], f, positions=pos, outs=[y, z], **kw)
        assert back[0] is y and back[1] is z
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    # not the same rows: an output that begins one token on, which a tensor of one row (D values) does not reach
    flat = torch.zeros(B * H * N * D + D, dtype=torch.bfloat16, device="cuda")
    call = lambda: cz.rope([flat[:-D].view(B, H, N, D)], f, positions=pos, outs=[flat[D:].view(B, H, N, D)])
    if B * H * N == 1:
        call()
    else:
        with pytest.raises(cz.CPError):
            call()


def test_keys_and_values_read_into_one_tensor():
    """Refused: rows of both would go to the same place."""
    pages, table = filled([40], 2, 64, 32, 1)
    out = torch.zeros(2, 2, 40, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(), dict(stream=torch.cuda.current_stream())):
        with pytest.raises(cz.CPError):
            cz.kv4_read(pages, table, i32([0]), 40, 64, k=out[:1], v=out[:1], **kw)
        k, v = cz.kv4_read(pages, table, i32([0]), 40, 64, k=out[:1], v=out[1:], **kw)
        assert torch.equal(k, cz.kv4_read(pages, table, i32([0]), 40, 64)[0])
        assert torch.equal(v, cz.kv4_read(pages, table, i32([0]), 40, 64)[1])


@pytest.mark.parametrize("B,T", [(1, 1), (3, 4), (200, 1)])
def test_a_table_without_pages(B, T):
    """Sequences that hold nothing yet: O = 0, LSE = -inf; a token has no place there."""
    pages, _ = filled([16], 2, 64, 16, 1)
    before = pages.clone()
    table = torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(causal=False), dict(window=3)):
        o, lse = cz.attn_kv4(rows(B, 4, T, 64, 2).cuda(), pages, table, i32([0] * B), **kw)
        assert (o == 0).all() and (lse == float("-inf")).all()
    assert cz.get_device_status() == 0
    k = rows(B, 2, T, 64, 3).cuda()
    cz.kv4_write(pages, table, i32([0] * B), k, k)
    assert cz.get_device_status() == 1 and torch.equal(pages, before)
    got = cz.kv4_read(pages, table, i32([0] * B), T, 64, k=k.clone(), v=k.clone())
    assert cz.get_device_status() == 1 and torch.equal(got[0], k) and torch.equal(got[1], k)


@pytest.mark.parametrize("B,Hq,Hkv,D,most,window", [(1, 4, 1, 128, 1023, 0), (1, 4, 1, 128, 1024, 0), (18, 16, 8, 64, 1023, 0),
                                                    (19, 16, 8, 64, 1023, 0), (3, 8, 2, 256, 1008, 0),
                                                    (2, 16, 1, 128, 3000, 1020), (2, 16, 1, 128, 3000, 1023)])
def test_tables_and_windows_around_what_one_cta_takes_alone(B, Hq, Hkv, D, most, window):
    lens = [most - 37 * b for b in range(B)]
    lens[-1] = max(lens[-1], 1)
    pages, table = filled(lens, Hkv, D, 16, 5)
    q = rows(B, Hq, 1, D, 6)
    o, lse = cz.attn_kv4(q.cuda(), pages, table, i32(lens), window=window)
    check_attn(q, pages, table, lens, o, lse, window=window)
    assert cz.get_device_status() == 0
