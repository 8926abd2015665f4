"""The fp8b attention kernels where values are of very different sizes or where what
surrounds them was never written, against fp64 on the same codes (block_ref.py).
"""
import numpy as np
import pytest
import torch

import quantized_kv_cache_17_b200 as kvq
from tests import block_ref as br
from tests.test_gpu_block import (DT, built, check_decode, check_prefill, decode, dev, i32, make_pool, page_table,  # noqa: F401
                                  prefill, random_cache)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,hkv,n_ctas", [([9000], 4, 148), ([3000, 9000], 8, 148), ([2000] * 60, 1, 148), ([20000], 1, 600)])
def test_decode_merge_gives_the_same_bits_every_time(lens, hkv, n_ctas):
    """One, four and sixteen CTAs a merge, and more than 128 units in one: every head's sum is there in every run."""
    rng = np.random.default_rng(200)
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, 8, hkv)                       # the pages are the same few, over and over
    table = np.where(table >= 0, table % 8, table).astype(np.int32)
    q = rng.standard_normal((len(lens), 8 * hkv, 256)).astype(np.float32)
    pool, qd, td = make_pool(cache, 8 * hkv), dev(q), dev(table)
    plan, info = kvq.decode_plan(pool.desc, lens, table.shape[1], n_ctas)
    assert info.n_units > len(lens) * hkv
    pd, ws = dev(plan), torch.empty(info.workspace_bytes // 4, device="cuda")
    out, of = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape, device="cuda")
    first = None
    for _ in range(300):
        of.fill_(float("nan"))
        kvq.paged_decode_attn_combined(pool, 0, qd, td, pd, info, ws, out, of)
        first = of.clone() if first is None else first
        assert torch.equal(of, first)
    check_decode(cache, table[:1], lens[:1], q[:1], out[:1], of[:1])
