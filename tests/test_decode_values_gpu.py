"""Attention over a 4-bit cache whose values have very different sizes, or are not numbers."""
import pytest
import torch

import context_zigzag_cp_b200 as cz
from test_kv4_gpu import check_attn, i32, paged, rows

pytestmark = pytest.mark.gpu

SIZES = 2.0 ** 30


def spread_cache(B, Hkv, D, n, seed, change):
    """K, V drawn on the GPU, changed, and written; -> pages, table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages, table = paged(B, Hkv, D, 64, n, seed)
    k, v = (torch.randn(B, Hkv, n, D, generator=g, device="cuda") for _ in range(2))
    change(k, v)
    cz.kv4_write(pages, table, i32([0] * B), k.bfloat16(), v.bfloat16())
    return pages, table


def check_few(q, pages, table, n, o, lse, which, **kw):
    for b in which:
        order = torch.arange(table.shape[1], dtype=torch.int32, device="cuda")[None]
        check_attn(q[b:b + 1], pages[table[b].long()], order, [n], o[b:b + 1], lse[b:b + 1], **kw)


@pytest.mark.parametrize("D,Hq,Hkv,B,n", [(128, 4, 1, 2, 3000), (128, 32, 8, 64, 2048), (128, 64, 8, 16, 1024), (256, 4, 1, 2, 700),
                                          (256, 16, 2, 40, 1024), (128, 16, 1, 64, 1024), (64, 4, 1, 2, 300),
                                          (128, 3, 1, 48, 1024), (64, 5, 1, 48, 1024), (256, 7, 1, 48, 700), (64, 9, 1, 2, 300)])
def test_values_of_very_different_sizes(D, Hq, Hkv, B, n):
    """Groups of 64 dims some 2^30 apart; keys with values 2^30 times the others' that no row gives weight (far below in
    score); such keys among the first ones, left behind by the rows' maximum later; and sizes that change
    from key to key and group to group.  The bound of check_attn is
    relative to what a group's own weighed values are."""
    q = rows(B, Hq, 1, D, 5).abs()

    def groups(k, v):
        v[..., :64] *= SIZES

    def unseen(k, v):
        for at in (0, 1, 70, n // 2, n - 1):
            k[:, :, at], v[:, :, at, :64] = -16.0, v[:, :, at, :64] * SIZES

    def left_behind(k, v):
        v[:, :, :3] *= SIZES
        k[:, :, n // 3:] += 10.0

    def mixed(k, v):
        g = torch.Generator(device="cuda").manual_seed(9)
        size = torch.rand(B, Hkv, n, D // 64, generator=g, device="cuda") * 20 - 10
        v *= torch.exp2(size).repeat_interleave(64, -1)

    for seed, change in enumerate((groups, unseen, left_behind, mixed)):
        pages, table = spread_cache(B, Hkv, D, n, 10 + seed, change)
        o, lse = cz.attn_kv4(q.cuda(), pages, table, i32([n] * B), partial=True)
        check_few(q, pages, table, n, o, lse, (0, B - 1), partial=True)
    assert cz.get_device_status() == 0


@pytest.mark.parametrize("D,T,Hq", [(64, 1, 1), (64, 2, 8), (128, 1, 4), (128, 2, 3), (256, 1, 2)])
@pytest.mark.parametrize("at", [0, 5, 70, 150, 199])
def test_a_value_that_is_not_a_number_under_no_weight(D, T, Hq, at):
    """0 times NaN is NaN for every row that sees the key, wherever it stands; rows that do not see it are clean."""
    n = 200
    k, v = rows(1, 1, n, D, 1), rows(1, 1, n, D, 2)
    k[0, 0, at] = -128.0                              # some 128 0.8 sqrt(D) below the others: its weight is 0
    v[0, 0, at, D - 1] = float("nan")
    q = rows(1, Hq, T, D, 3).abs()
    pages, table = paged(1, 1, D, 16, n, 4)
    cz.kv4_write(pages, table, i32([0]), k.cuda(), v.cuda())
    o, lse = cz.attn_kv4(q.cuda(), pages, table, i32([n]))
    assert torch.isfinite(lse).all()
    for t in range(T):
        sees = at <= n - T + t
        assert torch.isnan(o[0, :, t, D - 64:]).all() == sees
        assert torch.isfinite(o[0, :, t, :D - 64]).all()
        if not sees:
            assert torch.isfinite(o[0, :, t]).all()
    o, lse = cz.attn_kv4(q.cuda(), pages, table, i32([n]), window=n - 100)
    assert torch.isnan(o[..., D - 64:]).any() == (at > 100 - T)


@pytest.mark.parametrize("D,Hq,B,n", [(64, 4, 2, 300), (128, 3, 48, 1024), (256, 8, 2, 700), (128, 16, 2, 3000)])
def test_values_at_the_ends_of_their_type(D, Hq, B, n):
    """Small values beside keys with the largest ones that bf16 has, which no row gives weight."""
    def change(k, v):
        v *= 2.0 ** -12
        for at in (3, n // 2, n - 2):
            k[:, :, at] = -64.0
            v[:, :, at] = v[:, :, at].sign() * 2.0 ** 126
    q = rows(B, Hq, 1, D, 5).abs()
    pages, table = spread_cache(B, 1, D, n, 20, change)
    o, lse = cz.attn_kv4(q.cuda(), pages, table, i32([n] * B), partial=True)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    check_few(q, pages, table, n, o, lse, (0, B - 1), partial=True)
