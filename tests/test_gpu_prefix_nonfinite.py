"""Queries that are not finite, in a batch that shares a prefix: their rows are NaN, as the softmax of their scores is,
and no other row changes by a bit."""
import pytest
import torch

import synth
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("columns", [0, 80])                 # own tokens joined with the merge, or split before it
@pytest.mark.parametrize("bits", [0, 2, 4])
def test_rows_of_queries_that_are_not_finite(kvlib, bits, columns, qdt):
    kv, B, P = kvlib, 32, 150
    lens = [70, 0, 64, 3, 40, 0] * 8
    s = Shared(kv, 23, P, lens, 8, 2, B, bits)
    if columns:
        narrow = s.table
        s.table = torch.full((len(lens), columns), -1, dtype=torch.int32, device="cuda")
        s.table[:, :narrow.shape[1]] = narrow
    pl = [(P, P, 0, 1, 149, 0)[b % 6] for b in range(len(lens))]
    clean = synth.queries(synth.make_gen(6), len(lens), 8).to(qdt).cuda()
    want = s.run(clean, pl)
    q = clean.clone()
    q[0:6, 1, 5] = float("nan")
    q[6:12, 2] = float("nan")
    q[12:18, 7, 127] = float("inf")
    q[18:24, 4] = float("-inf")
    bad = ~torch.isfinite(q).all(-1)
    for odt in (torch.float32, torch.bfloat16):
        got = s.run(q, pl, out_dtype=odt)
        for b in range(len(lens)):
            if pl[b] == 0 and lens[b] == 0:
                assert torch.all(got[b] == 0)                # no token at all
            else:
                assert torch.isnan(got[b][bad[b]]).all()
        assert torch.equal(got[~bad], want[~bad].to(odt))
