"""Steps of decoding in a row, every input another one at every step, never waited for: what each kernel reads is what
the kernel before it wrote, not what lay there a step ago."""
import pytest
import torch

import context_zigzag_cp_b200 as cz
from test_kv4_gpu import filled, rows

pytestmark = pytest.mark.gpu


def run(wait, B, T, D, page, steps, given):
    """Rotate, write, attend and read, each from the buffers that the call before filled; -> every step's outputs."""
    pages, table, inv_freq, ins = given
    pages = pages.clone()
    q, k = (torch.full_like(x, float("nan")) for x in ins[0][:2])
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    ko, vo = (torch.full_like(k, float("nan")) for _ in range(2))
    pos, start, lens = (torch.zeros_like(x) for x in ins[0][3:])
    got = []
    torch.cuda.synchronize()
    for x in ins:
        for to, new in zip((pos, start, lens), x[3:]):
            to.copy_(new)
        calls = [lambda: cz.rope(list(x[:2]), inv_freq, positions=pos, outs=[q, k]),
                 lambda: cz.kv4_write(pages, table, start, k, x[2]),
                 lambda: cz.attn_kv4(q, pages, table, lens, o=o, lse=lse),
                 lambda: cz.kv4_read(pages, table, start, T, D, k=ko, v=vo),
                 # the outputs turned back in place: reads what the attention has just written
                 lambda: cz.rope([o], inv_freq, positions=pos, inverse=True, outs=[o])]
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()
        got.append([y.clone() for y in (q, k, o, lse, ko, vo)])
    torch.cuda.synchronize()
    return got, pages


@pytest.mark.parametrize("B,Hq,Hkv,T,D,n", [(2, 8, 2, 2, 128, 3000), (48, 8, 2, 1, 64, 300), (3, 4, 1, 1, 256, 900)])
def test_every_step_reads_what_it_was_given(B, Hq, Hkv, T, D, n):
    page, steps = 64, 40
    pages, table = filled([n + steps * T] * B, Hkv, D, page, 1)
    inv_freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    ins = []
    for i in range(steps):
        at = torch.tensor([n + i * T - (b % 3) for b in range(B)], dtype=torch.int32, device="cuda")
        pos = (at[:, None, None] + torch.arange(T, dtype=torch.int32, device="cuda")).contiguous()
        ins.append((rows(B, Hq, T, D, 10 * i).cuda(), rows(B, Hkv, T, D, 10 * i + 1).cuda(),
                    rows(B, Hkv, T, D, 10 * i + 2).cuda(), pos, at, at + T))
    given = (pages, table, inv_freq, ins)
    want, end = run(True, B, T, D, page, steps, given)
    for _ in range(5):
        got, last = run(False, B, T, D, page, steps, given)
        for i, (a, b) in enumerate(zip(want, got)):
            for x, y in zip(a, b):
                assert torch.equal(x, y), i
        assert torch.equal(end, last)
    assert not torch.equal(want[0][2], want[1][2])
    assert cz.get_device_status() == 0
