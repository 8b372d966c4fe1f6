"""Ragged rotary appends whose offsets or lengths do not fit: the header's faults, the same into bf16 pages and the
packed cache, and nothing written for the sequence at fault."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(params=[False, True], ids=["bf16", "packed"])
def call(request, kvlib):
    """call(cu, pos, n_tokens) -> (error word, pool, staging, q_out); token rows of bf16 noise, outputs preset to 7."""
    kv, n_q, n_kv, B, nb = kvlib, 4, 2, 32, 2
    cfg = kv.make_config(n_q, n_kv, B, 2, synth.sign_bits(0))
    rope, ws = kv.make_rope(kv.rope_frequencies(128)[0]), kv.alloc_workspace(cfg, 0, 0)
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(200, n_q + 2 * n_kv, D, generator=g).to(torch.bfloat16).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(cu, pos, T):
        batch = len(pos)
        table = torch.arange(batch * nb, dtype=torch.int32, device="cuda").view(batch, nb)
        stage = torch.full((batch, n_kv, 2, B, D), 7.0, dtype=torch.bfloat16, device="cuda")
        out = torch.full((T, n_q, D), 7.0, device="cuda")
        q, k, v = rows[:T, :n_q], rows[:T, n_q:n_q + n_kv], rows[:T, n_q + n_kv:]
        kv.clear_error(ws)
        if request.param:
            pool = kv.alloc_pool(cfg, batch * nb) + 7
            kv.append_rope(cfg, rope, pool, stage, table, i32(pos), q, k, v, out, ws, cu_tokens=i32(cu))
        else:
            pool = torch.full((batch * nb, n_kv, 2, B, D), 7.0, dtype=torch.bfloat16, device="cuda")
            kv.append_rope_bf16(cfg, rope, pool, table, i32(pos), q, k, v, out, ws, cu_tokens=i32(cu))
        return kv.read_error(ws), pool.view(batch, nb, *pool.shape[1:]), stage, out

    run.kv = kv
    return run


def _untouched(got, b, lo, hi):
    _, pool, stage, out = got
    assert torch.all(pool[b] == 7) and torch.all(stage[b] == 7) and torch.all(out[lo:hi] == 7)


def _written(got, want, b, lo, hi):
    assert torch.equal(got[1][b], want[1][b]) and torch.equal(got[2][b], want[2][b])
    assert torch.equal(got[3][lo:hi], want[3][lo:hi]) and torch.all(got[3][lo:hi] != 7)


def test_rows_before_the_first_sequence_are_left_alone(call):
    got = call([3, 40, 44], [0, 30], 50)
    assert got[0] == 0
    assert torch.all(got[3][:3] == 7) and torch.all(got[3][44:] == 7) and torch.all(got[3][3:44] != 7)


def test_a_last_run_beyond_the_rows_is_flagged_and_skipped(call):
    want = call([0, 5, 9], [30, 31], 9)
    assert want[0] == 0
    for T in (9, 8, 6, 5):                  # the last run's 4 rows, some of them, none of them there
        got = call([0, 5, 10 if T == 9 else 9], [30, 31], T)
        assert got[0] == call.kv.DEVERR_POSITION
        _written(got, want, 0, 0, 5)
        _untouched(got, 1, 5, T)


def test_a_run_beyond_the_block_table_is_skipped_whole(call):
    want = call([0, 5, 12, 15], [0, 57, 3], 15)          # 57 + 7 = 64: fits
    assert want[0] == 0
    for pos in (58, 63, 64, 2 ** 31 - 1, -1, -2 ** 31):
        got = call([0, 5, 12, 15], [0, pos, 3], 15)
        assert got[0] == call.kv.DEVERR_POSITION
        _untouched(got, 1, 5, 12)
        for b, lo, hi in ((0, 0, 5), (2, 12, 15)):
            _written(got, want, b, lo, hi)
    assert call([0, 5, 5, 8], [0, 2 ** 31 - 1, 3], 8)[0] == 0      # (no token: nothing to place)


@pytest.mark.parametrize("cu", [[5, 0], [9, 9, 4], [0, 7, 6, 9], [0, 9, 9, 2], [-1, 3], [0, 2, -3, 9], [9, 4, 0]])
def test_offsets_that_descend_are_flagged_whatever_rows_there_are(call, cu):
    assert call(cu, [0] * (len(cu) - 1), 9)[0] == call.kv.DEVERR_POSITION


def test_more_sequences_than_the_grid_has_threads(call):
    """One token row, and offsets that descend at the last of 3000 sequences without tokens."""
    cu = [0] * 3000 + [1]
    assert call(cu, [0] * 3000, 1)[0] == 0
    cu[2999] = 2
    assert call(cu, [0] * 3000, 1)[0] == call.kv.DEVERR_POSITION
