"""The fp8b attention kernels where values are of very different sizes or where what
surrounds them was never written, against fp64 on the same codes (block_ref.py).

Where values differ in size, a row answers for the keys it attends to and no others.
With p the softmax of a row, d a key's V scale, B = max over dims of sum p |v|, T the
row's largest p d, and A and K of test_gpu_block.py over the row's own keys:
 a score that is off by ds changes the output by at most 2 ds B, a weight rounded by
   the factor 1 + w by w B (2 w B where the sum of weights is not the rounded ones');
 a weight is stored so that the row's largest p d lies in [2^9, 2^15] (prefill) or the
   largest of a warp's keys in [2^6, 2^15] (decode).  Three E5M2 terms of a weight,
   the last of them cut off, are within 2^-16 of it (over all fp16, 0.875 of that); a
   pair of fp16 within 2^-25.  A code is at most 448: 448 T 2^-25 and 448 T 2^-31 a key.
 prefill: 2 B ((2^-15 + e) A + 2^-17 qmax K + 2^-9) + 448 n T 2^-25, e = 2^-12 unless bf16
 decode:  2 B (2^-15 A + 2^-19) + 448 n T 2^-31
"""
import numpy as np
import pytest
import torch

import oracle
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


def check_rows(cache, table, pos0, toks, q, of, dtype=None):
    """of against fp64, each row by the keys below its limit.  dtype None: decode, one row a sequence over all its tokens."""
    hq, hkv, row = q.shape[1], cache.codes.shape[1], 0
    G, qf, got = hq // hkv, q.float().cpu().numpy().astype(np.float64), of.cpu().numpy().astype(np.float64)
    for b, (p0, n) in enumerate(zip(pos0, toks)):
        for h in range(hkv if n else 0):
            k, v = cache.values(table[b], p0 + n, h)
            d = np.repeat(cache.scales[table[b, :-(-(p0 + n) // 256)], h, :, 1].astype(np.float64).ravel(), 64)[:p0 + n]
            x = qf[row:row + n, h * G:(h + 1) * G].reshape(n * G, 256)
            limit = np.repeat(np.arange(p0 + 1, p0 + n + 1), G)
            hidden = np.arange(p0 + n)[None] >= limit[:, None]
            s = np.where(hidden, -np.inf, x @ k.T / 16)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            B, T = (w @ np.abs(v)).max(1), (w * d).max(1)
            A = np.where(hidden, 0, np.abs(x) @ np.abs(k).T / 16).max(1)
            K = np.where(hidden, 0, np.abs(k).sum(1)[None] / 16).max(1)
            if dtype is None:
                tol = 2 * B * (2.0 ** -15 * A + 2.0 ** -19) + 448 * limit * T * 2.0 ** -31
            else:
                e = 0.0 if dtype == torch.bfloat16 else 2.0 ** -12
                tol = 2 * B * ((2.0 ** -15 + e) * A + 2.0 ** -17 * np.abs(x).max(1) * K + 2.0 ** -9) + 448 * limit * T * 2.0 ** -25
            err = np.abs(got[row:row + n, h * G:(h + 1) * G].reshape(n * G, 256) - w @ v).max(1)
            assert (err <= tol + 1e-37).all(), f"seq {b} head {h}: row {np.argmax(err / (tol + 1e-37))}, {(err / (tol + 1e-37)).max()} of the tolerance"
        row += n


def tiles_cache(rng, n_slots, heads):
    """Keys below 2^-3 but for dim 0, which is 0; scales of 1."""
    c = random_cache(rng, n_slots, heads)
    c.codes[:, :, 0] &= 0x9F
    c.codes[:, :, 0, :, 0] = 0
    c.scales[:] = 1.0
    return c


def set_tile(cache, slots, i, score=None, exponent=None):
    """Tile i of a sequence: scores (natural units, by dim 0 where queries have 16) and the exponent of its V scale."""
    page, blk = slots[i // 4], i % 4
    if score is not None:
        cache.codes[page, :, 0, blk * 64:(blk + 1) * 64, 0] = oracle.f32_to_e4m3(np.array([score], np.float32))[0]
    if exponent is not None:
        cache.scales[page, :, blk, 1] = 0.0 if exponent == "zero" else 2.0 ** exponent


def value_queries(rng, rows, heads, dtype):
    q = rng.standard_normal((rows, heads, 256)).astype(np.float32)
    q[:, :, 0] = 16.0
    return dev(q, DT[dtype])


@pytest.mark.parametrize("up", [12, 20, 28, 60, 118])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_that_a_row_does_not_see_leave_it_alone(dtype, up):
    """The tile behind each row tile's first one, hidden from its first rows, has values 2^up larger."""
    rng = np.random.default_rng(220)
    pos0, toks = [0, 128, 320], [100, 90, 128]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = tiles_cache(rng, n_slots, 1)
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            if i * 64 >= max(pos0[b], 1) + 8:
                set_tile(cache, table[b], i, exponent=up)
    q = value_queries(rng, sum(toks), 2, dtype)
    for n_ctas in (1, 148):
        _, of = prefill(make_pool(cache, 2), q, dev(table), pos0, toks, n_ctas=n_ctas)
        check_rows(cache, table, pos0, toks, q, of, DT[dtype])


# per tile: score and V exponent.  A large value of no weight before (or behind) the ones that count; values and scores that
# balance; a reference that climbs while the values fall, so that what is stored has to follow by both; scales of 0
LADDERS = {
    "large_first": [(-80, 60), (0, 0), (0, 0), (1, 0), (0, -1)],
    "large_last": [(0, 0), (0, 0), (1, 1), (-80, 60), (-96, 80)],
    "balanced": [(-20, 29), (0, 0), (-10, 14), (-13, 19), (-26, 37), (0, 0)],
    "climbing": [(0.625 * i, 40 - 3 * i) for i in range(24)],
    "climbing_slowly": [(0.5 * i, 24 - i) for i in range(48)],
    "falling": [(16 - i, i) for i in range(24)],
    "zero_scales": [(120, "zero"), (110, 3), (112, 0), (120, "zero")],
    "only_zero": [(3, "zero"), (1, "zero")],
    "far_apart": [(-224, 118), (0, -90), (-20, -61), (1, -100), (-160, 100)],
    "tiny_then_large": [(8, -60), (0, 30), (-30, 60), (8, -60)],
}


def ladder_cache(rng, ladder):
    tiles = LADDERS[ladder]
    end = 64 * len(tiles)
    table, n_slots = page_table(rng, [end, end])
    cache = tiles_cache(rng, n_slots, 1)
    for slots in table:
        for i, (score, exponent) in enumerate(tiles):
            set_tile(cache, slots, i, score, exponent)
    return cache, table


def random_sizes_cache(rng, spread, lens):
    table, n_slots = page_table(rng, lens)
    cache = tiles_cache(rng, n_slots, 2)
    for slots, n in zip(table, lens):
        for i in range(-(-n // 64)):
            up = int(rng.integers(-spread, spread + 1))
            set_tile(cache, slots, i, float(np.round(-0.69 * up + 2 * rng.standard_normal())), up)
    return cache, table


@pytest.mark.parametrize("ladder", list(LADDERS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_of_values_of_very_different_sizes(dtype, ladder):
    rng = np.random.default_rng(230)
    end = 64 * len(LADDERS[ladder])
    pos0, toks = [end - 50, 0], [47, min(end, 330)]
    cache, table = ladder_cache(rng, ladder)
    q = value_queries(rng, sum(toks), 4, dtype)
    for n_ctas in (1, 148):
        _, of = prefill(make_pool(cache, 4), q, dev(table), pos0, toks, n_ctas=n_ctas)
        check_rows(cache, table, pos0, toks, q, of, DT[dtype])


@pytest.mark.parametrize("spread", [20, 60])
def test_prefill_of_values_of_random_sizes(spread):
    rng = np.random.default_rng(240)
    pos0, toks = [2000, 0, 777], [70, 400, 200]
    cache, table = random_sizes_cache(rng, spread, [p + t for p, t in zip(pos0, toks)])
    q = value_queries(rng, sum(toks), 12, "bf16")
    _, of = prefill(make_pool(cache, 12), q, dev(table), pos0, toks)
    check_rows(cache, table, pos0, toks, q, of, torch.bfloat16)


@pytest.mark.parametrize("n_ctas", [1, 148])
@pytest.mark.parametrize("ladder", list(LADDERS))
def test_decode_of_values_of_very_different_sizes(ladder, n_ctas):
    rng = np.random.default_rng(250)
    end = 64 * len(LADDERS[ladder])
    cache, table = ladder_cache(rng, ladder)
    lens = [end - 3, max(64, end - 64)]
    q = value_queries(rng, 2, 4, "f32")
    _, of = decode(make_pool(cache, 4), q, dev(table), lens, n_ctas=n_ctas)
    for b, n in enumerate(lens):
        check_rows(cache, table[b:b + 1], [n - 1], [1], q[b:b + 1], of[b:b + 1])


@pytest.mark.parametrize("spread", [20, 60])
def test_decode_of_values_of_random_sizes(spread):
    rng = np.random.default_rng(260)
    lens = [2070, 400, 977]
    cache, table = random_sizes_cache(rng, spread, lens)
    q = value_queries(rng, 3, 12, "f32")
    for n_ctas in (3, 148):
        _, of = decode(make_pool(cache, 12), q, dev(table), lens, n_ctas=n_ctas)
        for b, n in enumerate(lens):
            check_rows(cache, table[b:b + 1], [n - 1], [1], q[b:b + 1], of[b:b + 1])


def test_decode_takes_the_query_of_an_append():
    """fp32 when asked for; the append's default for 16-bit rows, which the prefill takes, is refused."""
    rng = np.random.default_rng(270)
    x = dev(rng.standard_normal((2, 16, 256)).astype(np.float32), torch.bfloat16)
    q, k, v = x[:, :12], x[:, 12:14], x[:, 14:]
    table = np.array([[1], [0]], np.int32)
    cs, td = br.rope_table(10, 64), dev(table)
    pool = kvq.KVPool.allocate(kvq.make_desc(1, 2, 12, 2, "fp8b"))
    args = (pool, 0, k, v, i32([0, 1, 2]), i32([0, 0]), td)
    default = kvq.kv_append_rope(*args, cos_sin=dev(cs), q=q)
    plan, info = kvq.decode_plan(pool.desc, [1, 1], 1)
    ws, out = torch.empty(info.workspace_bytes // 4, device="cuda"), torch.empty((2, 12, 256), dtype=torch.bfloat16, device="cuda")
    assert default.dtype == torch.bfloat16
    with pytest.raises(kvq.KVQError, match="float32"):
        kvq.paged_decode_attn_combined(pool, 0, default, td, dev(plan), info, ws, out)
    with pytest.raises(kvq.KVQError, match="float32"):
        kvq.paged_decode_attn_fp8b(pool, 0, default, td, dev(plan), info, ws)
    qf = kvq.kv_append_rope(*args, cos_sin=dev(cs), q=q, q_out_dtype=torch.float32)
    kvq.paged_decode_attn_combined(pool, 0, qf, td, dev(plan), info, ws, out)
    cache = br.Cache.unpack(pool.buf.view(2, 2, br.PAGE_BYTES).cpu().numpy())
    for b in range(2):                                       # one key: its value
        for h in range(2):
            want = torch.from_numpy(cache.values(table[b], 1, h)[1].astype(np.float32)).to(torch.bfloat16)
            assert torch.equal(out[b, 6 * h:6 * h + 6].cpu(), want.expand(6, 256))


@pytest.mark.parametrize("n_ctas", [1, 148])
def test_a_sequence_without_pages(n_ctas):
    """Zeros from the combined decode, NaN where attn_combine divides by no weight at all, and the other sequence as alone."""
    rng = np.random.default_rng(280)
    lens = [700, 300]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    q = rng.standard_normal((2, 12, 256)).astype(np.float32)
    gone = table.copy()
    gone[0] = -1
    for mode in ("combined", "split"):
        status = i32([0])
        _, of = decode(make_pool(cache, 12), dev(q), dev(gone), lens, n_ctas=n_ctas, mode=mode, status=status)
        assert int(status.item()) == kvq.STATUS_BAD_SLOT
        assert (of[0] == 0).all() if mode == "combined" else torch.isnan(of[0]).all()
        check_rows(cache, table[1:], [299], [1], dev(q[1:]), of[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rounding_of_the_weights(dtype):
    """kvq.h: about 2^-12 of the sum of |weight v|.  Keys of 0 make every weight the same, 1 / n, whatever q is."""
    rng = np.random.default_rng(290)
    pos0, toks = [900], [200]
    table, n_slots = page_table(rng, [1100])
    cache = random_cache(rng, n_slots, 1)
    cache.codes[:, :, 0] = 0
    q = dev(rng.standard_normal((200, 4, 256)).astype(np.float32), DT[dtype])
    _, of = prefill(make_pool(cache, 4), q, dev(table), pos0, toks)
    v = cache.values(table[0], 1100, 0)[1]
    n = np.arange(901, 1101)[:, None]
    want, B = np.cumsum(v, 0)[900:] / n, np.cumsum(np.abs(v), 0)[900:] / n
    err = np.abs(of.cpu().numpy().astype(np.float64) - want[:, None])
    assert (err <= 1.01 * 2.0 ** -12 * B[:, None] + 1e-30).all()
