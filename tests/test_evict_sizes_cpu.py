"""Sizes of an eviction that do not fit the C entry point's 32 bits: refused before anything is looked at."""
import pytest
import torch

import bit_kv_cache_08_gb300 as kv


@pytest.fixture(scope="module", autouse=True)
def built():
    kv.build()


@pytest.mark.parametrize("bits", [0, 2])
@pytest.mark.parametrize("budget,recent", [(64, (1 << 32) + 32), (64, (1 << 31) + 32), (64, -(1 << 32) + 32), ((1 << 32) + 64, 32),
                                           ((1 << 31), 32), (-(1 << 32) + 64, 0)])
def test_sizes_beyond_32_bits(bits, budget, recent):
    """(recent = 2^32 + 32 was taken as 32.)"""
    cfg = kv.make_config(2, 2, 32, 2, [0] * 4)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros(4, kv.block_bytes(cfg), dtype=torch.uint8) if bits else torch.zeros(4, 2, 2, 32, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        (kv.evict if bits else kv.evict_bf16)(cfg, pool, i(1, 4), i(1), torch.zeros(1, 2, 128), i(1, 3), i(1), torch.zeros(1, 2, 96),
                                              i(1, 2, 2 if bits else 64), torch.zeros(256, dtype=torch.uint8), budget=budget, recent=recent)
