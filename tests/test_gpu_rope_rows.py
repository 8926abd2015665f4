"""kv_append_rope: which rows belong to which sequence, for every pool format."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_17_b200 as kvq
from tests import block_ref as br
from tests.test_gpu_block import built, dev, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def one_page_each(fmt, n_seq, hkv=1, hq=2):
    return kvq.KVPool.allocate(kvq.make_desc(1, hkv, hq, n_seq, fmt)), torch.arange(n_seq, dtype=torch.int32, device="cuda")[:, None]


@pytest.mark.parametrize("fmt", ["fp8b", "q4_0", "nvfp4"])
@pytest.mark.parametrize("part", ["all", "q", "kv"])
def test_a_row_start_that_is_not_one_is_flagged(fmt, part):
    rng = np.random.default_rng(300)
    n = 20
    x = dev(rng.standard_normal((n, 4, 256)).astype(np.float32))
    many = np.arange(701) // 40
    fell, passed = many.copy(), many.copy()
    fell[650], passed[700] = 3, n + 1
    good = [[0, 10, 10, 20], [3, 4, 9, 9], [0, 0, 0, 0], [20, 20, 20, 20], many]
    bad = [[0, 10, 5, 20], [0, 5, 9, n + 1], [-1, 0, 5, 9], [0, 30, 20, 20], [9, 8, 9, 20], fell, passed]
    for start, want in [(s, 0) for s in good] + [(s, kvq.STATUS_BAD_PLAN) for s in bad]:
        n_seq = len(start) - 1
        pool, table = one_page_each(fmt, n_seq)
        status = i32([0])
        k, v, q = (x[:, 2:3], x[:, 3:], x[:, :2]) if part == "all" else (None, None, x[:, :2]) if part == "q" else (x[:, 2:3], x[:, 3:], None)
        kvq.kv_append_rope(pool, 0, k, v, dev(np.asarray(start, np.int32)), i32([0] * n_seq), table, q=q, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == want, list(start)[:5]


@pytest.mark.parametrize("fmt", ["fp8b", "int8", "k8v4", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (12, 2)])
@pytest.mark.parametrize("before,toks,after", [(7, [3, 0, 65], 5), (70, [1, 1, 0, 2], 0), (130, [130, 1], 1), (1, [1] * 40, 3),
                                               (200, [0, 2] * 20, 9), (5, [1400], 3)])
def test_rows_before_the_first_sequence_are_padding(fmt, hq, hkv, before, toks, after):
    """As the rows behind the last: the same pool and queries as without them, status 0."""
    rng = np.random.default_rng(310)
    n, total = sum(toks), before + sum(toks) + after
    x = rng.standard_normal((total, hq + 2 * hkv, 256)).astype(np.float32)
    x[:before], x[before + n:] = np.nan, np.nan
    x = dev(x, torch.bfloat16)
    pages = -(-max(toks) // 256) + 1
    table = torch.arange(len(toks) * pages, dtype=torch.int32, device="cuda").view(-1, pages)
    start = np.concatenate([[0], np.cumsum(toks)]).astype(np.int32)
    pos0 = i32([3 * i % 60 for i in range(len(toks))])
    cs, status = dev(br.rope_table(2000, 64)), i32([0])
    got = []
    for y, s in ((x, start + before), (x[before:before + n].contiguous(), start)):
        pool = kvq.KVPool.allocate(kvq.make_desc(1, hkv, hq, table.numel(), fmt))
        out = torch.full((len(y), hq, 256), 7.0, device="cuda")
        kvq.kv_append_rope(pool, 0, y[:, hq:hq + hkv], y[:, hq + hkv:], dev(s), pos0, table, cos_sin=cs, q=y[:, :hq], q_out=out, status=status)
        got.append((pool.buf, out))
    assert int(status.item()) == 0
    assert torch.equal(got[0][0], got[1][0])
    assert torch.equal(got[0][1][before:before + n], got[1][1])
    assert (got[0][1][:before] == 7).all() and (got[0][1][before + n:] == 7).all()
