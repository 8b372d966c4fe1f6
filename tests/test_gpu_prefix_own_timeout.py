"""Own tokens of a shared-prefix call over the packed cache whose copy waits give up (the test switch: at once, nothing
hangs): with no prefix, so that the flag comes from them alone, and with one. The flag is raised, the copies land, and
the workspace serves the next call with the same bits."""
import pytest
import torch

import synth
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,B", [(2, 32), (2, 64), (3, 64), (4, 32)])
@pytest.mark.parametrize("batch,columns", [(4, 0), (4, 80), (80, 0)])   # joined with the merge; split: a wide table, many units
def test_own_waits_that_give_up(kvlib, bits, B, batch, columns):
    kv, P = kvlib, 300
    lens = [(9 * B + 5, 3 * B, B - 1, 5 * B + 1)[b % 4] for b in range(batch)]
    s = Shared(kv, 41, P, lens, 8, 2, B, bits)
    if columns:
        narrow = s.table
        s.table = torch.full((batch, columns), -1, dtype=torch.int32, device="cuda")
        s.table[:, :narrow.shape[1]] = narrow
    q = synth.queries(synth.make_gen(2), batch, 8).to(torch.bfloat16).cuda()
    ws = kv.alloc_prefix_workspace(s.cfg, batch, len(s.prefix_np))
    for pl in ([0] * batch, [P] * batch):
        good = s.run(q, pl, ws=ws)
        s.cfg.flags |= kv.FLAG_TEST_WAIT_TIMEOUT
        for _ in range(3):
            s.run(q, pl, ws=ws, check=False)
            assert kv.read_error(ws) == kv.DEVERR_WAIT_TIMEOUT
            kv.clear_error(ws)
        s.cfg.flags &= ~kv.FLAG_TEST_WAIT_TIMEOUT
        assert torch.equal(s.run(q, pl, ws=ws), good)
