"""Partials that are not a number, joined by cp_lse_merge."""
import pytest
import torch

import context_zigzag_cp_b200 as cz
from test_kv4_gpu import i32, paged, rows

pytestmark = pytest.mark.gpu


def test_parts_that_are_not_a_number_stay_so():
    """lse_merge: a NaN part makes its row NaN, beside parts without a key and beside ordinary ones."""
    nan, inf = float("nan"), float("inf")
    lse = torch.tensor([[nan, nan, 0.5, -inf, -inf, 1.0, nan], [nan, -inf, nan, nan, -inf, 2.0, 3.0]])
    for n in (2, 5, 40):
        for D in (64, 256):
            full = torch.full((n, lse.shape[1]), -inf)
            full[0], full[n - 1] = lse
            o = torch.randn(n, lse.shape[1], D, generator=torch.Generator().manual_seed(n))
            oo, ol = cz.lse_merge(o.cuda(), full.cuda())
            oo, ol = oo.float().cpu(), ol.cpu()
            assert torch.isnan(oo[[0, 1, 2, 3, 6]]).all() and torch.isnan(ol[[0, 1, 2, 3, 6]]).all()
            assert (oo[4] == 0).all() and ol[4] == -inf
            assert torch.isfinite(oo[5]).all() and torch.isfinite(ol[5])


@pytest.mark.parametrize("bad", ["query", "keys"])
def test_joined_parts_of_rows_that_are_not_finite(bad):
    """A context in two caches: joined, the rows are NaN that are NaN over one cache."""
    D, Hq, Hkv, n, cut = 64, 4, 2, 200, 120
    k, v, q = rows(1, Hkv, n, D, 1), rows(1, Hkv, n, D, 2), rows(1, Hq, 1, D, 3)
    if bad == "query":
        q[0, 1, 0, 5], q[0, 2, 0, 6] = float("inf"), float("nan")
    else:
        k[0, 1, 20, 3] = float("nan")                 # KV head 1: query heads 2 and 3
    parts, whole = [], None
    for a, b, last in ((0, cut, False), (cut, n, True), (0, n, True)):
        pages, table = paged(1, Hkv, D, 32, b - a, 4)
        cz.kv4_write(pages, table, i32([0]), k[:, :, a:b].cuda(), v[:, :, a:b].cuda())
        whole = cz.attn_kv4(q.cuda(), pages, table, i32([b - a]), causal=last, partial=True)
        parts.append(whole)
    o, lse = cz.lse_merge(torch.stack([x[0].view(-1, D) for x in parts[:2]]), torch.stack([x[1].view(-1) for x in parts[:2]]))
    rowsbad = [1, 2] if bad == "query" else [2, 3]
    for h in range(Hq):
        if h in rowsbad:
            assert torch.isnan(o[h]).all() and torch.isnan(lse[h]) and torch.isnan(whole[1][0, h]).all()
        else:
            assert torch.isfinite(o[h]).all() and torch.isfinite(lse[h])
