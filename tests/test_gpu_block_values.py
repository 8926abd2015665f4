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


def spoil_with(rng, cache, table, lens, scale):
    """What lies past a sequence's last token in its last page: codes of every kind, and `scale` (or any bits) for its scales."""
    for b, n in enumerate(lens):
        page = table[b, (n - 1) // 256]
        if n % 256:
            stale = cache.codes[page, :, :, n % 256:]
            stale[:] = rng.integers(0, 256, stale.shape, dtype=np.uint8)
        for blk in range(-(-n // 64), -(-n // 256) * 4):
            to = cache.scales[page, :, blk % 4]
            to[:] = rng.integers(0, 1 << 32, to.shape, dtype=np.uint32).view(np.float32) if scale is None else scale


@pytest.mark.parametrize("scale", [-1.0, -np.inf, np.inf, np.nan, -0.0, 3e38, None])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stale_scales_past_the_end_count_for_nothing(scale, dtype):
    """Sequences that end in the first or the second tile of a step of 128 keys, in each quarter of a page."""
    rng = np.random.default_rng(210)
    pos0, toks = [0, 100, 300, 129, 30, 500], [40, 60, 30, 63, 90, 12]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    spoil_with(rng, cache, table, lens, scale)
    q = dev(rng.standard_normal((sum(toks), 12, 256)).astype(np.float32), DT[dtype])
    for n_ctas in (1, 148):
        out, of = prefill(make_pool(cache, 12), q, dev(table), pos0, toks, n_ctas=n_ctas)
        check_prefill(cache, table, pos0, toks, q, out, of, DT[dtype])
    last = q[torch.tensor(toks).cumsum(0).cuda() - 1].float()
    out, of = decode(make_pool(cache, 12), last, dev(table), lens)
    check_decode(cache, table, lens, last.cpu().numpy(), out, of)
