"""ContextParallel.decode attends the whole of every rank's part of a cache: problems whose mask would leave keys out
are refused, on every rank and before any collective."""
import datetime

import pytest
import torch

import context_zigzag_cp_b200 as cz
from context_zigzag_cp_b200.dist import ContextParallel
from test_decode_dist import B, D, HKV, HQ, PlainKernels, T, _free_port, lengths, part, queries


@pytest.fixture(scope="module")
def group():
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{_free_port()}", rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=60))
    yield dist
    dist.destroy_process_group()


def decode(**kw):
    cu = kw.pop("cu_seqlens", None)
    prob = cz.Problem(B, 128, 1, HQ, HKV, D, **kw)
    prob.cu_seqlens = cu                              # a Problem itself takes documents on a GPU only
    ctx = ContextParallel(prob, kernels=PlainKernels(), plan=object())
    pages, table, _ = part(0, 1)
    return ctx.decode(queries(), torch.from_numpy(pages), torch.from_numpy(table),
                      torch.tensor(lengths(1)[0], dtype=torch.int32), 0)


@pytest.mark.parametrize("kw,what", [(dict(window=16), "window"), (dict(causal=False), "causal"),
                                     (dict(cu_seqlens=torch.tensor([0, 100, 128], dtype=torch.int32)), "cu_seqlens")])
def test_masks_that_leave_keys_out(group, kw, what):
    with pytest.raises(ValueError, match="decode: the problem has " + what):
        decode(**kw)


def test_the_causal_mask(group):
    o, lse = decode()
    assert o.shape == (B, HQ, T, D) and torch.isfinite(lse).all()
