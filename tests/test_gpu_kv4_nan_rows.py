"""Decode attention of rows that attend, or are, something that is not a number:
NaN and a report, never the zeros of a row that attends nothing."""
import numpy as np
import pytest
import torch

from test_gpu_kv4_nonfinite import case, dev, q3, spoil  # noqa: F401

pytestmark = pytest.mark.gpu


# n_q, n_kv, the rows' contexts, the row and position that is spoilt
DECODE = [(32, 8, [70, 90], 0, 33), (40, 8, [700, 64], 0, 3), (16, 8, [1, 5], 0, 0), (64, 8, [3000], 0, 2999), (8, 8, [257, 33], 1, 32),
          (4, 4, [33, 64], 0, 32)]


@pytest.mark.parametrize("which", ["K", "V", "q", "all K"])
@pytest.mark.parametrize("qt", [torch.float16, torch.float32])
@pytest.mark.parametrize("c", DECODE, ids=str)
def test_decode_rows_of_numbers_that_are_not(q3,  # noqa: F811
                                              c, qt, which):
    n_q, n_kv, lens, row, p = c
    q, kv, tables, _, _ = case(n_q, n_kv, [(1, n - 1) for n in lens], 71 + n_q)
    q = q.to(qt)
    bad, qq = kv, q
    if which == "all K":
        for b in tables[row]:
            for r in range(32):
                bad = spoil(bad, b, r, 0)
    elif which == "q":
        qq = q.clone()
        qq[row, :, 5] = float("nan")
    else:
        bad = spoil(kv, tables[row, p // 32], p % 32, "KV".index(which))
    pos, slot = dev(np.array(lens, np.int32) - 1), dev(np.arange(len(lens), dtype=np.int32))
    clean = q3.op_kv4_decode_attention(q, pos, slot, dev(tables), dev(kv))
    for dt in (torch.float16, torch.float32):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.empty(q.shape, dtype=dt, device="cuda")
        got = q3.op_kv4_decode_attention(qq, pos, slot, dev(tables), dev(bad), out=out, status=status)
        assert torch.isnan(got[row]).all()
        if dt == torch.float16:
            others = [i for i in range(len(lens)) if i != row]
            assert status.item() == 0x8 and torch.equal(got[others], clean[others])
