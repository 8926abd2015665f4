"""The fp8b cache on the GPU: kv_append_rope (all formats), the single-token
attention and the ragged prefill, against the model in block_ref.py.

Appended bytes are compared whole (codes, scales and everything that must stay as
it was).  Attention is compared with fp64 on the same codes.  Tolerances, with
A = max_j sum_d |q_d k_jd| / 16 of the row and V = max |v|: a score that is off by
ds changes the output by at most 2 ds V, a weight rounded by the factor 1 + w by at
most w V (2 w V where the sum of weights is not the rounded ones').
 decode: the products keep 22 bits of q and are summed in fp32 over 256 terms, at
   most 2^-16 A with every rounding of the sum (256 of 2^-24); the exponential is
   good to 2^-21 and the score's conversion to base 2 to 2^-23 A; weights are pairs
   of fp16, 2^-21.  f32: 2 V (2^-15 A + 2^-19).
 prefill: q as two E4M3 terms under a power of two per row holds bf16 exactly down to 2^-10 of a code
   of the row's largest value in [2^7, 2^8), 2^-17 of it; as three terms fp16 and fp32 to 2^-12 besides; weights
   as three terms of 3 bits, 2^-9, and nothing below 2^-27 of the row's reference (half
   the smallest E5M2 number, 2^-17, of weights made 2^10 times larger; n keys: n 2^-27).  f32: 2 V (2^-15 A + e A + 2^-17 qmax K + 2^-9 + n 2^-27) with e = 0 or 2^-12
   and K = max_j sum_d |k_jd| / 16.
 bf16: half a step more, 2^-9 of the value.
"""
import numpy as np
import pytest
import torch

import oracle
import quantized_kv_cache_17_b200 as kvq
from tests import block_ref as br

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_17_b200 import build
    build.build()
    oracle.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_pool(cache, hq, layers=1, layer=0):
    n, h = cache.codes.shape[:2]
    desc = kvq.make_desc(layers, h, hq, n, "fp8b")
    pool = kvq.KVPool.allocate(desc)
    pool.buf.view(layers, n, h, br.PAGE_BYTES)[layer] = dev(cache.pack())
    return pool


def pool_bytes_of(pool, layer=0):
    d = pool.desc
    return pool.buf.view(d.n_layers, d.n_pages, d.n_kv_heads, br.PAGE_BYTES)[layer].cpu().numpy()


def page_table(rng, lens, extra=1, n_slots=None):
    need = [max(1, -(-n // 256)) for n in lens]
    n_slots = n_slots or sum(need) + 2
    slots = rng.permutation(n_slots)[:sum(need)]
    t = np.full((len(lens), max(need) + extra), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = slots[at:at + n]
        at += n
    return t, n_slots


def random_cache(rng, n_slots, heads, spread=2.0, stale_nan=None):
    """Codes of every kind but NaN under scales of very different sizes."""
    c = br.Cache(n_slots, heads)
    c.codes[:] = rng.integers(0, 256, c.codes.shape, dtype=np.uint8)
    c.codes[(c.codes & 0x7F) == 0x7F] = 0
    c.codes[:] = np.where(rng.random(c.codes.shape) < 0.9, c.codes & 0xBF, c.codes)      # most of them small
    c.scales[:] = 2.0 ** rng.integers(-9 - int(spread), -8 + int(spread), c.scales.shape).astype(np.float32)
    return c


def spoil_after(cache, table, lens):
    """What lies past a sequence's last token in its last page: NaN codes."""
    for b, n in enumerate(lens):
        if n % 256:
            cache.codes[table[b, n // 256], :, :, n % 256:] = 0x7F
        for blk in range(-(-n // 64), -(-n // 256) * 4):
            cache.scales[table[b, n // 256], :, blk % 4] = np.nan


def rows_of(x, seq_rows, dtype, pad=0, stride_extra=0):
    """[rows, heads, 256] fp32 -> a device tensor of the type whose rows are strided."""
    t = dev(x).to(dtype)
    if stride_extra:
        wide = torch.full((t.shape[0], t.shape[1] + stride_extra, 256), float("nan"), dtype=dtype, device="cuda")
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    return t


# ---- append ----------------------------------------------------------------
def run_appends(calls, hq, hkv, dtype, rot, inter, q_f32, lens, seed, mul=1.0, stride_extra=0, pad=0, layers=1, layer=0):
    """calls: lists of new tokens per sequence, from empty sequences.  Checks pool bytes and rotated queries after each."""
    rng = np.random.default_rng(seed)
    table, n_slots = page_table(rng, lens)
    model = br.Cache(n_slots, hkv)
    model.codes[:] = rng.integers(0, 256, model.codes.shape, dtype=np.uint8)          # whatever lay there before
    model.scales[:] = rng.random(model.scales.shape, dtype=np.float32)
    pool = make_pool(model, hq, layers, layer)
    other = [pool_bytes_of(pool, x) for x in range(layers)]
    cs = br.rope_table(max(lens) + 1, rot)
    status = i32([0])
    pos = [0] * len(lens)
    for step, toks in enumerate(calls):
        n = sum(toks)
        k = rng.standard_normal((n + pad, hkv, 256)) * np.exp(rng.standard_normal((n + pad, 1, 1)) * 2) * mul
        v = rng.standard_normal((n + pad, hkv, 256)) * (1 + step)
        v[rng.random((n + pad, 1, 1)).repeat(hkv, 1)[..., 0] < 0.2] = 0.0
        k, v = k.astype(np.float32), v.astype(np.float32)
        q = rng.standard_normal((n + pad, hq, 256)).astype(np.float32)
        if pad:
            k[n:], v[n:], q[n:] = np.nan, np.nan, np.nan
        kd, vd, qd = (rows_of(x, None, dtype, stride_extra=stride_extra) for x in (k, v, q))
        start = np.concatenate([[0], np.cumsum(toks)]).astype(np.int32)
        q_out = torch.full((n + pad, hq, 256), 7.0, dtype=torch.float32 if q_f32 else dtype, device="cuda")
        got = kvq.kv_append_rope(pool, layer, kd, vd, dev(start), i32(pos), dev(table), cos_sin=dev(cs) if rot else None,
                                 interleaved=inter, q=qd, q_out=q_out, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and got is q_out
        kf, vf, qf = (x.float().cpu().numpy() for x in (kd, vd, qd))
        want_q = np.full((n + pad, hq, 256), 7.0, np.float32)
        for b, t in enumerate(toks):
            sl, p = slice(start[b], start[b] + t), np.arange(pos[b], pos[b] + t)
            model.append(table[b], pos[b], br.rotate(kf[sl], p, cs, inter) if rot else kf[sl], vf[sl])
            want_q[sl] = br.rotate(qf[sl], p, cs, inter) if rot else qf[sl]
            pos[b] += t
        want_q = torch.from_numpy(want_q).to(q_out.dtype)
        assert torch.equal(want_q.float(), q_out.cpu().float()), f"q of call {step}"
        assert np.array_equal(pool_bytes_of(pool, layer), model.pack()), f"pool after call {step}"
    for x in range(layers):
        if x != layer:
            assert np.array_equal(pool_bytes_of(pool, x), other[x])
    return pool, model, table, pos


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (64, True), (96, False), (256, False), (256, True)])
def test_append_bytes(dtype, rot, inter):
    run_appends([[70, 1, 0], [1, 63, 300], [1, 1, 1], [0, 65, 2]], 6, 2, DT[dtype], rot, inter, dtype == "f32", [80, 140, 310], 1)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (24, 4), (5, 5)])
def test_append_head_layouts_strides_and_padding(hq, hkv):
    run_appends([[3, 130, 64], [64, 1, 1]], hq, hkv, torch.bfloat16, 128, False, True, [70, 140, 70], 2, stride_extra=3, pad=5,
                layers=3, layer=1)


@pytest.mark.parametrize("mul", [1e-30, 3e4, 1e-41])
def test_append_extreme_sizes(mul):
    """Scales at the ends of their range, subnormal inputs among them."""
    run_appends([[40], [30], [1]], 2, 1, torch.float32, 64, False, True, [80], 3, mul=mul)


def test_append_one_token_at_a_time_rescales():
    """Every token larger than the last: the tile's scale grows and its codes move down."""
    rng = np.random.default_rng(5)
    table, n_slots = page_table(rng, [130])
    model = br.Cache(n_slots, 2)
    pool = make_pool(model, 4)
    for p in range(130):
        k = (rng.standard_normal((1, 2, 256)) * 1.3 ** (p % 64)).astype(np.float32)
        v = (rng.standard_normal((1, 2, 256)) * (0 if p < 3 else 1.2 ** (p % 50))).astype(np.float32)
        kvq.kv_append_rope(pool, 0, dev(k), dev(v), i32([0, 1]), i32([p]), dev(table))
        model.append(table[0], p, k, v)
    assert np.array_equal(pool_bytes_of(pool), model.pack())


def test_append_many_sequences():
    """More sequences than one warp's search covers at once, most of them with nothing or one token."""
    rng = np.random.default_rng(8)
    toks = [int(x) for x in rng.integers(0, 3, 1100)]
    toks[500], toks[1099] = 150, 70
    run_appends([toks], 2, 1, torch.bfloat16, 64, False, False, [max(t, 1) for t in toks], 9)


def test_append_decoding_batch_with_padding():
    """Fewer rows than tiles they could touch (a tile belongs to its first row), sequences without rows, padding behind."""
    run_appends([[1, 0, 2, 1, 70], [1, 1, 0, 63, 1], [1, 1, 1, 1, 1]], 6, 2, torch.bfloat16, 64, False, True, [9, 9, 9, 80, 90], 12, pad=6)
    run_appends([[1] * 40, [2] * 40], 4, 1, torch.float16, 32, True, False, [3] * 40, 13, pad=2)


@pytest.mark.parametrize("hq,hkv,toks,dtype,inter,q_f32", [
    (24, 4, [0, 1701, 40, 0, 660], "bf16", False, False), (7, 1, [8200], "f16", True, False), (24, 3, [2400], "f32", False, False),
    (16, 2, [3600], "bf16", True, True), (1, 1, [57000, 3], "f16", False, False), (8, 1, [200] * 36, "bf16", False, True)])
def test_append_of_many_query_rows(hq, hkv, toks, dtype, inter, q_f32):
    """As many query rows as make a warp take eight, of one row and of several, of sequences that end between them."""
    run_appends([toks], hq, hkv, DT[dtype], 64, inter, q_f32, [max(t, 1) for t in toks], 14, pad=5, stride_extra=1)


def test_append_that_starts_past_the_rotation_table():
    """The place lies in a tile that the table still reaches: nothing is read or written for it."""
    rng = np.random.default_rng(15)
    model = br.Cache(2, 1)
    model.codes[:], model.scales[:] = rng.integers(0, 256, model.codes.shape, dtype=np.uint8), 1.0
    pool, status = make_pool(model, 1), i32([0])
    k, q = dev(rng.standard_normal((9, 1, 256)).astype(np.float32)), torch.zeros((9, 1, 256), device="cuda")
    out = torch.full((9, 1, 256), 5.0, device="cuda")
    kvq.kv_append_rope(pool, 0, k, k, i32([0, 9]), i32([25]), i32([[0, 1]]), cos_sin=dev(br.rope_table(22, 64)), q=q, q_out=out,
                       status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.STATUS_BAD_SLOT and (out == 5).all()
    assert np.array_equal(pool_bytes_of(pool), model.pack())


def test_append_of_no_rows():
    pool = make_pool(br.Cache(2, 2), 4)
    before = pool.buf.clone()
    k, q = torch.empty((0, 2, 256), device="cuda"), torch.empty((0, 4, 256), device="cuda")
    out = kvq.kv_append_rope(pool, 0, k, k, i32([0, 0, 0]), i32([5, 0]), i32([[0], [1]]), q=q)
    torch.cuda.synchronize()
    assert tuple(out.shape) == (0, 4, 256) and torch.equal(pool.buf, before)


def test_append_q_only_and_kv_only_and_in_place():
    rng = np.random.default_rng(4)
    table, n_slots = page_table(rng, [300])
    model = br.Cache(n_slots, 2)
    pool = make_pool(model, 8)
    cs = br.rope_table(400, 128)
    x = dev(rng.standard_normal((20, 12, 256)).astype(np.float32), torch.bfloat16)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    before = pool.buf.clone()
    a = kvq.kv_append_rope(pool, 0, None, None, i32([0, 20]), i32([33]), dev(table), cos_sin=dev(cs), q=q)
    assert torch.equal(before, pool.buf) and a.dtype == torch.bfloat16
    assert kvq.kv_append_rope(pool, 0, k, v, i32([0, 20]), i32([33]), dev(table), cos_sin=dev(cs)) is None
    p = np.arange(33, 53)
    want = torch.from_numpy(br.rotate(q.float().cpu().numpy(), p, cs, False)).bfloat16()
    assert torch.equal(a.cpu(), want)
    qc = q.contiguous()
    assert kvq.kv_append_rope(pool, 0, None, None, i32([0, 20]), i32([33]), dev(table), cos_sin=dev(cs), q=qc, q_out=qc) is qc
    assert torch.equal(qc.cpu(), want)


def test_append_nonfinite_values_are_flagged_and_kept_out():
    rng = np.random.default_rng(6)
    table, n_slots = page_table(rng, [100])
    model = br.Cache(n_slots, 1)
    pool = make_pool(model, 2)
    k = rng.standard_normal((70, 1, 256)).astype(np.float32)
    v = k[::-1].copy()
    k[3, 0, 7], k[69, 0, 255], v[5, 0, 0] = np.nan, np.inf, -np.inf
    status = i32([0])
    kvq.kv_append_rope(pool, 0, dev(k), dev(v), i32([0, 70]), i32([0]), dev(table), status=status)
    model.append(table[0], 0, k, v)
    assert int(status.item()) == kvq.STATUS_NONFINITE and model.nonfinite
    raw = pool_bytes_of(pool)
    assert np.array_equal(raw, model.pack())
    c = br.Cache.unpack(raw)
    assert not ((c.codes & 0x7F) == 0x7F).any()


def test_append_bad_places_are_flagged_and_skipped():
    rng = np.random.default_rng(7)
    model = br.Cache(3, 1)
    table = np.array([[0, 99], [1, -1], [2, 2]], np.int32)
    k = rng.standard_normal((400, 1, 256)).astype(np.float32)

    def call(toks, pos0, rows=None, cs=None, start=None):
        pool, status = make_pool(model, 1), i32([0])
        st = np.concatenate([[0], np.cumsum(toks)]).astype(np.int32) if start is None else np.array(start, np.int32)
        q = torch.zeros((400, 1, 256), device="cuda")
        out = torch.full((400, 1, 256), 5.0, device="cuda")
        kvq.kv_append_rope(pool, 0, dev(k), dev(k), dev(st), i32(pos0), dev(table), cos_sin=cs, q=q, q_out=out, status=status)
        torch.cuda.synchronize()
        return br.Cache.unpack(pool_bytes_of(pool)), int(status.item()), out.cpu().numpy()

    c, st, _ = call([10, 1, 1], [250, 0, 0])                 # six tokens fit, four fall into a slot past the pool
    assert st == kvq.STATUS_BAD_SLOT and (c.codes[0, 0, 0, 250:256] != 0).any() and (c.scales[0, 0, 3] > 0).all()
    c, st, _ = call([1, 2, 1], [0, 255, 0])                  # a slot of -1
    assert st == kvq.STATUS_BAD_SLOT and (c.codes[1, 0, 0, 255] != 0).any()
    c, st, out = call([1, 1, 10], [0, 0, 506])               # past the page table
    assert st == kvq.STATUS_BAD_SLOT and (c.codes[2, 0, 0, 250:256] != 0).any()
    assert (out[:8] != 5).all() and (out[8:] == 5).all()
    c, st, out = call([1, 1, 10], [0, 0, -3])                # before the start
    assert st == kvq.STATUS_BAD_SLOT and (c.codes[2] == 0).all()
    cs = dev(br.rope_table(20, 64))
    c, st, out = call([1, 30, 1], [0, 5, 0], cs=cs)          # past the rotation table: 15 tokens fit
    assert st == kvq.STATUS_BAD_SLOT and (c.codes[1, 0, 0, 5:20] != 0).any(1).all() and (c.codes[1, 0, :, 20:] == 0).all()
    assert (out[1:16] != 5).all() and (out[16:31] == 5).all()
    c, st, _ = call(None, [0, 0, 0], start=[0, 300, 100, 401])       # decreases, then passes n_rows
    assert st & kvq.STATUS_BAD_PLAN
    c, st, _ = call(None, [0, 0, 0], start=[-70, -60, -50, -40])
    assert (c.codes == 0).all()


@pytest.mark.parametrize("fmt", ["int8", "q4_0", "k8v4", "fp8", "nvfp4"])
@pytest.mark.parametrize("dtype,rot,inter", [("bf16", 64, False), ("f32", 256, True), ("f16", 0, False)])
def test_append_other_formats_equal_kv_append_of_rotated_rows(fmt, dtype, rot, inter):
    rng = np.random.default_rng(11)
    toks, pos0, hq, hkv = [5, 0, 260, 1], [250, 3, 0, 40], 12, 2
    table, n_slots = page_table(rng, [p + t for p, t in zip(pos0, toks)])
    desc = kvq.make_desc(2, hkv, hq, n_slots, fmt)
    a, b = kvq.KVPool.allocate(desc), kvq.KVPool.allocate(desc)
    x = dev(rng.standard_normal((sum(toks) + 3, hq + 2 * hkv, 256)).astype(np.float32), DT[dtype])
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    start = np.concatenate([[0], np.cumsum(toks)]).astype(np.int32)
    cs = br.rope_table(600, rot)
    status = i32([0])
    q_out = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
    kvq.kv_append_rope(a, 1, k, v, dev(start), i32(pos0), dev(table), cos_sin=dev(cs) if rot else None, interleaved=inter, q=q,
                       q_out=q_out, status=status)
    n = sum(toks)
    seq = np.repeat(np.arange(4), toks).astype(np.int32)
    pos = np.concatenate([np.arange(p, p + t) for p, t in zip(pos0, toks)]).astype(np.int32)
    turn = (lambda y: br.rotate(y[:n].float().cpu().numpy(), pos, cs, inter)) if rot else (lambda y: y[:n].float().cpu().numpy())
    kvq.kv_append(b, 1, dev(turn(k)), v[:n].float().contiguous(), dev(pos), dev(table), row_seq=dev(seq), status=status)
    want = dev(turn(q))
    if kvq.rotated_q(fmt):
        want = kvq.q_rotate(want)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(a.buf, b.buf)
    assert torch.equal(q_out[:n], want) and (q_out[n:] == 7).all()


# ---- decode ----------------------------------------------------------------
def decode(pool, q, table, lens, n_ctas=0, mode="combined", status=None, f32=True):
    plan, info = kvq.decode_plan(pool.desc, lens, table.shape[1], n_ctas)
    ws = torch.full((info.workspace_bytes // 4,), float("nan"), device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    of = torch.full(q.shape, float("nan"), device="cuda") if f32 else None
    own = status is None
    status = i32([0]) if own else status
    if mode == "combined":
        kvq.paged_decode_attn_combined(pool, 0, q, table, dev(plan), info, ws, out, of, status)
    else:
        kvq.paged_decode_attn_fp8b(pool, 0, q, table, dev(plan), info, ws, status)
        kvq.attn_combine(ws, dev(plan), info, False, out, of)
    torch.cuda.synchronize()
    assert not own or int(status.item()) == 0
    return out, of


def check_decode(cache, table, lens, q, out, of):
    hq, hkv = q.shape[1], cache.codes.shape[1]
    G = hq // hkv
    for b, n in enumerate(lens):
        for h in range(hkv):
            k, v = cache.values(table[b], n, h)
            want, a = br.attend(q[b, h * G:(h + 1) * G].astype(np.float64), k, v, [n] * G)
            V = np.abs(v).max()
            tol = 2 * V * (2.0 ** -15 * a + 2.0 ** -19)
            got = of[b, h * G:(h + 1) * G].cpu().numpy().astype(np.float64)
            err = np.abs(got - want).max(1)
            assert (err <= tol).all(), f"seq {b} head {h}: {err} over {tol}"
    assert torch.equal(of.to(torch.bfloat16), out)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("mode", ["combined", "split"])
def test_decode_parity(G, mode):
    rng = np.random.default_rng(20 + G)
    lens = [1, 2, 16, 17, 63, 64, 65, 255, 257, 700]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    spoil_after(cache, table, lens)
    q = rng.standard_normal((len(lens), 2 * G, 256)).astype(np.float32)
    status = i32([0])
    out, of = decode(make_pool(cache, 2 * G), dev(q), dev(table), lens, mode=mode, status=status)
    assert int(status.item()) == 0
    check_decode(cache, table, lens, q, out, of)


@pytest.mark.parametrize("n_ctas", [1, 3, 40, 148, 1000])
def test_decode_splits(n_ctas):
    rng = np.random.default_rng(31)
    lens = [5000, 1, 2111]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    spoil_after(cache, table, lens)
    q = rng.standard_normal((3, 12, 256)).astype(np.float32)
    out, of = decode(make_pool(cache, 12), dev(q), dev(table), lens, n_ctas=n_ctas)
    check_decode(cache, table, lens, q, out, of)
    out2, of2 = decode(make_pool(cache, 12), dev(q), dev(table), lens, n_ctas=n_ctas)
    assert torch.equal(of, of2)                                    # the same bits on every run


@pytest.mark.parametrize("case", ["wide_scales", "zero_blocks", "one_key", "large_q", "zero_q", "tiny_v"])
def test_decode_values(case):
    rng = np.random.default_rng(40)
    lens = [1000, 130]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1, spread=2.0)
    q = rng.standard_normal((2, 4, 256)).astype(np.float32)
    if case == "wide_scales":
        cache.scales[:] = 2.0 ** rng.integers(-24, 6, cache.scales.shape).astype(np.float32)
        q /= 64
    elif case == "zero_blocks":
        cache.scales[:, :, 1:3] = 0
    elif case == "one_key":
        cache.codes[table[0, 1], 0, 0, 77] = (np.sign(q[0, 0]) < 0) * 0x80 + 0x70        # q.k far above all others
    elif case == "large_q":
        q *= 30
    elif case == "zero_q":
        q[:] = 0
    elif case == "tiny_v":
        cache.scales[..., 1] = 2.0 ** -100
    out, of = decode(make_pool(cache, 4), dev(q), dev(table), lens)
    check_decode(cache, table, lens, q, out, of)


def test_decode_bad_slots_and_plans():
    rng = np.random.default_rng(50)
    lens = [600, 300]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1)
    q = rng.standard_normal((2, 4, 256)).astype(np.float32)
    pool = make_pool(cache, 4)
    bad = table.copy()
    bad[0, 1], bad[1, :] = n_slots, -1
    status = i32([0])
    out, of = decode(pool, dev(q), dev(bad), lens, status=status)
    assert int(status.item()) == kvq.STATUS_BAD_SLOT
    k, v = cache.values(table[0], 600, 0)
    keep = np.r_[0:256, 512:600]
    want, a = br.attend(q[0].astype(np.float64), k[keep], v[keep], [len(keep)] * 4)
    assert np.abs(of[0].cpu().numpy() - want).max() <= (2 * np.abs(v).max() * (2.0 ** -15 * a.max() + 2.0 ** -19))
    assert (of[1] == 0).all()
    plan, info = kvq.decode_plan(pool.desc, lens, table.shape[1])
    ws = torch.zeros(info.workspace_bytes // 4, device="cuda")
    o = torch.zeros((2, 4, 256), dtype=torch.bfloat16, device="cuda")
    for at, value in ((0, 1), (8, 2), (8, -1), (9, 1), (10, 32), (11, 0), (11, 1 << 20), (3, 2)):
        p = plan.copy()
        p[at] = value
        status.zero_()
        kvq.paged_decode_attn_combined(pool, 0, dev(q), dev(table), dev(p), info, ws, o, None, status)
        torch.cuda.synchronize()
        assert int(status.item()) & kvq.STATUS_BAD_PLAN, (at, value)


# ---- prefill ---------------------------------------------------------------
def prefill(pool, q, table, pos0, toks, n_ctas=0, status=None):
    plan, info = kvq.prefill_plan(pool.desc, pos0, toks, table.shape[1], n_ctas)
    ws = torch.full((max(1, info.workspace_bytes // 4),), float("nan"), device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    of = torch.full(q.shape, 7.0, device="cuda")
    own = status is None
    status = i32([0]) if own else status
    kvq.paged_prefill_attn_fp8b(pool, 0, q, table, dev(plan), info, ws, out, of, status)
    torch.cuda.synchronize()
    assert not own or int(status.item()) == 0
    return out, of


def check_prefill(cache, table, pos0, toks, q, out, of, dtype):
    hq, hkv = q.shape[1], cache.codes.shape[1]
    G, row = hq // hkv, 0
    qf = q.float().cpu().numpy().astype(np.float64)
    e = 0.0 if dtype == torch.bfloat16 else 2.0 ** -12
    for b, (p, n) in enumerate(zip(pos0, toks)):
        for h in range(hkv):
            if not n:
                continue
            k, v = cache.values(table[b], p + n, h)
            x = qf[row:row + n, h * G:(h + 1) * G].reshape(n * G, 256)
            limits = np.repeat(np.arange(p + 1, p + n + 1), G)
            want, a = br.attend(x, k, v, limits)
            V, K = np.abs(v).max(), np.abs(k).sum(1).max() / 16
            tol = 2 * V * ((2.0 ** -15 + e) * a + 2.0 ** -17 * np.abs(x).max(1) * K + 2.0 ** -9 + (p + n) * 2.0 ** -27)
            got = of[row:row + n, h * G:(h + 1) * G].cpu().numpy().reshape(n * G, 256).astype(np.float64)
            err = np.abs(got - want).max(1)
            assert (err <= tol).all(), f"seq {b} head {h}: row {np.argmax(err / tol)}, {(err / tol).max()} of the tolerance"
            # and as a whole far closer: the roundings are independent
            assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want) + 1e-30
        row += n
    assert torch.equal(of[:row].to(torch.bfloat16), out[:row])
    assert (out[row:] == 7).all() and (of[row:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(24, 4), (7, 1), (3, 3), (16, 2), (5, 1)])
def test_prefill_parity(dtype, hq, hkv):
    rng = np.random.default_rng(60)
    pos0, toks = [0, 100, 511, 64, 3], [130, 1, 67, 0, 20]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, hkv)
    spoil_after(cache, table, lens)
    q = rows_of(rng.standard_normal((sum(toks) + 4, hq, 256)).astype(np.float32), None, DT[dtype], stride_extra=2)
    status = i32([0])
    out, of = prefill(make_pool(cache, hq), q, dev(table), pos0, toks, status=status)
    assert int(status.item()) == 0
    check_prefill(cache, table, pos0, toks, q, out, of, DT[dtype])


@pytest.mark.parametrize("n_ctas", [1, 2, 7, 148])
@pytest.mark.parametrize("pos0,toks", [([4000], [33]), ([0], [700]), ([2047, 0, 900], [2, 300, 128])])
def test_prefill_splits(n_ctas, pos0, toks):
    rng = np.random.default_rng(70)
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1)
    spoil_after(cache, table, lens)
    q = dev(rng.standard_normal((sum(toks), 6, 256)).astype(np.float32), torch.bfloat16)
    pool = make_pool(cache, 6)
    out, of = prefill(pool, q, dev(table), pos0, toks, n_ctas=n_ctas)
    check_prefill(cache, table, pos0, toks, q, out, of, torch.bfloat16)
    out2, of2 = prefill(pool, q, dev(table), pos0, toks, n_ctas=n_ctas)
    assert torch.equal(of, of2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefill_of_whole_tiles(dtype):
    """More row tiles than CTAs and none of them cut: the plan deals them out of order, several to a CTA."""
    rng = np.random.default_rng(75)
    pos0, toks = [0, 333, 5], [1300, 400, 1]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    spoil_after(cache, table, lens)
    q = rows_of(rng.standard_normal((sum(toks) + 3, 16, 256)).astype(np.float32), None, DT[dtype], stride_extra=2)
    pool = make_pool(cache, 16)
    _, info = kvq.prefill_plan(pool.desc, pos0, toks, table.shape[1], 148)
    assert info.n_units > 148 and info.n_merges == 0
    out, of = prefill(pool, q, dev(table), pos0, toks, n_ctas=148)
    check_prefill(cache, table, pos0, toks, q, out, of, DT[dtype])


@pytest.mark.parametrize("case", ["wide_scales", "zero_blocks", "one_key", "large_q", "zero_q", "tiny_v", "growing", "sink"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_values(case, dtype):
    rng = np.random.default_rng(80)
    pos0, toks = [700, 0], [60, 200]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1)
    q = rng.standard_normal((sum(toks), 4, 256)).astype(np.float32)
    if case == "wide_scales":
        cache.scales[..., 0] = 2.0 ** rng.integers(-24, 6, cache.scales.shape[:-1]).astype(np.float32)
        cache.scales[..., 1] = 2.0 ** rng.integers(-14, -4, cache.scales.shape[:-1]).astype(np.float32)
        q /= 64
    elif case == "zero_blocks":
        cache.scales[:, :, 1:3] = 0
    elif case == "one_key":
        cache.codes[table[0, 1], 0, 0, 77] = (np.sign(q[0, 0]) < 0) * 0x80 + 0x70
    elif case == "large_q":
        q *= 30
    elif case == "zero_q":
        q[:] = 0
    elif case == "tiny_v":
        cache.scales[..., 1] = 2.0 ** -100
    elif case == "growing":                       # each tile's scores and values larger than the last: every step rescales
        for b in range(2):
            for i in range(lens[b] // 64 + 1):
                cache.scales[table[b, i // 4], :, i % 4] = 2.0 ** (i - 16)
    elif case == "sink":                          # one key far above the rest, whose weights still add up
        cache.codes[:, :, 0] = 0
        cache.codes[table[0, 0], 0, 0, 0, :64] = 0x38
        cache.scales[..., 0] = 1.0
        q[:, :, :64] = 2.0
    q = dev(q, DT[dtype])
    out, of = prefill(make_pool(cache, 4), q, dev(table), pos0, toks)
    check_prefill(cache, table, pos0, toks, q, out, of, DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("e", [-90, 115, 125])
def test_queries_near_the_ends_of_the_range(dtype, e):
    """q of 2^e or so against keys that bring the scores back to ordinary sizes."""
    rng = np.random.default_rng(85)
    pos0, toks = [200, 0], [30, 70]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1)
    cache.codes[:, :, 0] &= 0x9F                  # |k| below 2^-3 under a scale of 1
    cache.scales[..., 0] = 2.0 ** -min(e, 120)
    q = np.clip(rng.standard_normal((sum(toks), 4, 256)), -3.9, 3.9)
    q = dev((q * 2.0 ** e / (32 if e > 120 else 1)).astype(np.float32), DT[dtype])
    if e > 120:
        q[:, :, 5] = 1.5 * 2.0 ** e
    out, of = prefill(make_pool(cache, 4), q, dev(table), pos0, toks)
    check_prefill(cache, table, pos0, toks, q, out, of, DT[dtype])
    last = torch.stack([q[29], q[99]]).float()
    out, of = decode(make_pool(cache, 4), last, dev(table), lens)
    check_decode(cache, table, lens, last.cpu().numpy(), out, of)


def test_prefill_bad_slots_and_plans():
    rng = np.random.default_rng(90)
    lens, pos0, toks = [900], [890], [10]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1)
    pool = make_pool(cache, 4)
    q = dev(rng.standard_normal((10, 4, 256)).astype(np.float32), torch.bfloat16)
    bad = table.copy()
    bad[0, 1] = -1
    status = i32([0])
    out, of = prefill(pool, q, dev(bad), pos0, toks, status=status)
    assert int(status.item()) == kvq.STATUS_BAD_SLOT
    k, v = cache.values(table[0], 900, 0)
    keep = np.r_[0:256, 512:900]
    x = q.float().cpu().numpy().astype(np.float64).reshape(40, 256)
    want, a = br.attend(x, k[keep], v[keep], np.repeat(np.arange(891 - 256, 901 - 256), 4))
    assert np.linalg.norm(of.cpu().numpy().reshape(40, 256) - want) <= 2.0 ** -8 * np.linalg.norm(want)
    status.zero_()
    out, of = prefill(pool, q, torch.full_like(dev(table), 1 << 20), pos0, toks, status=status)
    assert int(status.item()) == kvq.STATUS_BAD_SLOT and (of == 0).all()
    plan, info = kvq.prefill_plan(pool.desc, pos0, toks, table.shape[1])
    ws = torch.zeros(max(1, info.workspace_bytes // 4), device="cuda")
    for at, value in ((0, 0), (1, 99), (8, 1), (9, -1), (10, 40), (10, -128), (11, 64), (12, 0), (12, 4000), (13, 1 << 20), (14, 1),
                      (15, -2), (16, 11)):
        p = plan.copy()
        p[at] = value
        status.zero_()
        kvq.paged_prefill_attn_fp8b(pool, 0, q, dev(table), dev(p), info, ws, out, None, status)
        torch.cuda.synchronize()
        assert int(status.item()) & kvq.STATUS_BAD_PLAN, (at, value)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_queries_stay_in_their_rows(bad):
    rng = np.random.default_rng(95)
    lens, pos0, toks = [700], [660], [40]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 1)
    pool = make_pool(cache, 4)
    q = rng.standard_normal((40, 4, 256)).astype(np.float32)
    spoilt = q.copy()
    spoilt[7, 2, 100] = bad
    for n_ctas in (1, 148):
        out, of = prefill(pool, dev(spoilt, torch.bfloat16), dev(table), pos0, toks, n_ctas=n_ctas)
        want, wf = prefill(pool, dev(q, torch.bfloat16), dev(table), pos0, toks, n_ctas=n_ctas)
        assert torch.isnan(of[7, 2]).all() and torch.isnan(out[7, 2]).all()
        # the rows of a warp move their references together, so the others are as near, not the same bits
        of[7, 2], out[7, 2] = wf[7, 2], want[7, 2]
        check_prefill(cache, table, pos0, toks, dev(q, torch.bfloat16), out, of, torch.bfloat16)
        a, af = decode(pool, dev(spoilt[7:8]), dev(table), lens, n_ctas=n_ctas)
        b, bf = decode(pool, dev(q[7:8]), dev(table), lens, n_ctas=n_ctas)
        assert torch.isnan(af[0, 2]).all()
        af[0, 2] = bf[0, 2]
        assert torch.equal(af, bf)


# ---- together --------------------------------------------------------------
def test_serving_run_of_the_operators():
    """Prompts in two chunks, then decoding steps: append (rotated), prefill and decode as a server calls them, in one captured
    graph per decode step, on a side stream, checked against fp64 over the cache that the calls left."""
    rng = np.random.default_rng(100)
    hq, hkv, G = 12, 2, 6
    chunks = [[200, 37, 0], [61, 300, 5]]
    lens = [sum(c[b] for c in chunks) + 3 for b in range(3)]
    table, n_slots = page_table(rng, lens)
    td, cs = dev(table), dev(br.rope_table(400, 128))
    pool = kvq.KVPool.allocate(kvq.make_desc(1, hkv, hq, n_slots, "fp8b"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pos = [0, 0, 0]
    status = i32([0])

    def cache_now():
        return br.Cache.unpack(pool_bytes_of(pool))

    for toks in chunks:
        n = sum(toks)
        x = dev(rng.standard_normal((n, hq + 2 * hkv, 256)).astype(np.float32), torch.bfloat16)
        plan, info = kvq.prefill_plan(pool.desc, pos, toks, table.shape[1])
        pd, ws = dev(plan), torch.empty(max(1, info.workspace_bytes // 4), device="cuda")
        start, p0 = dev(np.concatenate([[0], np.cumsum(toks)]).astype(np.int32)), i32(pos)
        out = torch.full((n, hq, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        of = torch.full((n, hq, 256), 7.0, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q = kvq.kv_append_rope(pool, 0, x[:, hq:hq + hkv], x[:, hq + hkv:], start, p0, td, cos_sin=cs, q=x[:, :hq], status=status)
            kvq.paged_prefill_attn_fp8b(pool, 0, q, td, pd, info, ws, out, of, status)
        side.synchronize()
        check_prefill(cache_now(), table, pos, toks, q, out, of, torch.bfloat16)
        pos = [p + t for p, t in zip(pos, toks)]
    # decode: static buffers, one graph a step
    x = torch.empty((3, hq + 2 * hkv, 256), dtype=torch.bfloat16, device="cuda")
    start = i32([0, 1, 2, 3])
    for step in range(3):
        now = [p + 1 for p in pos]
        plan, info = kvq.decode_plan(pool.desc, now, table.shape[1])
        pd, ws, p0 = dev(plan), torch.empty(info.workspace_bytes // 4, device="cuda"), i32(pos)
        qf = torch.empty((3, hq, 256), device="cuda")
        out = torch.empty((3, hq, 256), dtype=torch.bfloat16, device="cuda")
        of = torch.empty((3, hq, 256), device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            kvq.kv_append_rope(pool, 0, x[:, hq:hq + hkv], x[:, hq + hkv:], start, p0, td, cos_sin=cs, q=x[:, :hq], q_out=qf,
                               status=status)
            kvq.paged_decode_attn_combined(pool, 0, qf, td, pd, info, ws, out, of, status)
        for _ in range(2):                                     # replayed with other inputs: the second ones stand
            x.copy_(dev(rng.standard_normal(tuple(x.shape)).astype(np.float32), torch.bfloat16))
            graph.replay()
        torch.cuda.synchronize()
        check_decode(cache_now(), table, now, qf.cpu().numpy(), out, of)
        pos = now
    assert int(status.item()) == 0


def test_calls_side_by_side_on_two_streams():
    """Two batches with workspaces of their own, on two streams at once, give what they give alone."""
    rng = np.random.default_rng(120)
    state = []
    for lens in ([3000, 40], [1234]):
        table, n_slots = page_table(rng, lens)
        cache = random_cache(rng, n_slots, 2)
        pool = make_pool(cache, 12)
        plan, info = kvq.decode_plan(pool.desc, lens, table.shape[1])
        pplan, pinfo = kvq.prefill_plan(pool.desc, [n - 30 for n in lens], [30] * len(lens), table.shape[1])
        state.append(dict(pool=pool, table=dev(table), q=dev(rng.standard_normal((len(lens), 12, 256)).astype(np.float32)),
                          pq=dev(rng.standard_normal((30 * len(lens), 12, 256)).astype(np.float32), torch.bfloat16), plan=dev(plan), info=info,
                          pplan=dev(pplan), pinfo=pinfo, stream=torch.cuda.Stream()))

    def go(s):
        ws = torch.empty(s["info"].workspace_bytes // 4, device="cuda")
        pws = torch.empty(max(1, s["pinfo"].workspace_bytes // 4), device="cuda")
        o, po = (torch.empty(s[n].shape, dtype=torch.bfloat16, device="cuda") for n in ("q", "pq"))
        for _ in range(4):
            kvq.paged_decode_attn_combined(s["pool"], 0, s["q"], s["table"], s["plan"], s["info"], ws, o)
            kvq.paged_prefill_attn_fp8b(s["pool"], 0, s["pq"], s["table"], s["pplan"], s["pinfo"], pws, po)
        return o, po

    alone = [go(s) for s in state]
    torch.cuda.synchronize()
    both = []
    for s in state:
        with torch.cuda.stream(s["stream"]):
            both.append(go(s))
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_32_bits():
    """A pool of 5.5 GB whose last pages hold the sequence, in its second layer."""
    rng = np.random.default_rng(130)
    slots, lens = 10500, [600]
    table = np.array([[slots - 1, slots - 3, slots - 2]], np.int32)
    cs = dev(br.rope_table(700, 64))
    pool = kvq.KVPool.allocate(kvq.make_desc(2, 2, 12, slots, "fp8b"))
    assert kvq.pool_bytes(pool.desc) > 5 << 30
    x = dev(rng.standard_normal((600, 16, 256)).astype(np.float32), torch.bfloat16)
    q = kvq.kv_append_rope(pool, 1, x[:, 12:14], x[:, 14:], i32([0, 600]), i32([0]), dev(table), cos_sin=cs, q=x[:, :12])
    view = pool.buf.view(2, slots, 2, br.PAGE_BYTES)
    assert not view[0].any() and not view[1, :slots - 3].any()
    cache = br.Cache.unpack(view[1, slots - 3:].cpu().numpy())
    near = table - (slots - 3)
    model = br.Cache(3, 2)
    model.append(near[0], 0, br.rotate(x[:, 12:14].float().cpu().numpy(), np.arange(600), br.rope_table(700, 64), False),
                 x[:, 14:].float().cpu().numpy())
    assert np.array_equal(model.pack(), cache.pack())
    plan, info = kvq.prefill_plan(pool.desc, [590], [10], 3)
    ws = torch.empty(max(1, info.workspace_bytes // 4), device="cuda")
    out, of = torch.empty((10, 12, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((10, 12, 256), device="cuda")
    kvq.paged_prefill_attn_fp8b(pool, 1, q[590:], dev(table), dev(plan), info, ws, out, of)
    check_prefill(cache, near, [590], [10], q[590:], out, of, torch.bfloat16)
    plan, info = kvq.decode_plan(pool.desc, lens, 3)
    ws = torch.empty(info.workspace_bytes // 4, device="cuda")
    out, of = torch.empty((1, 12, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 12, 256), device="cuda")
    kvq.paged_decode_attn_combined(pool, 1, q[599:].float(), dev(table), dev(plan), info, ws, out, of)
    check_decode(cache, near, lens, q[599:].float().cpu().numpy(), out, of)


def test_prefill_replayed_from_a_graph():
    """Captured once, replayed with other queries and another page order."""
    rng = np.random.default_rng(140)
    pos0, toks = [300, 0], [70, 150]
    lens = [p + t for p, t in zip(pos0, toks)]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    pool = make_pool(cache, 12)
    plan, info = kvq.prefill_plan(pool.desc, pos0, toks, table.shape[1])
    pd, ws, td = dev(plan), torch.empty(max(1, info.workspace_bytes // 4), device="cuda"), dev(table)
    q = torch.zeros((sum(toks), 12, 256), dtype=torch.bfloat16, device="cuda")
    out, of = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.paged_prefill_attn_fp8b(pool, 0, q, td, pd, info, ws, out, of)
    for seed in range(2):
        q.copy_(dev(rng.standard_normal(tuple(q.shape)).astype(np.float32), torch.bfloat16))
        table = np.where(table >= 0, (table + 1) % n_slots, table).astype(np.int32)
        td.copy_(dev(table))
        graph.replay()
        torch.cuda.synchronize()
        check_prefill(cache, table, pos0, toks, q, out, of, torch.bfloat16)


def test_fp8b_pages_move_through_the_resident_cache():
    """The page cache copies fp8b pages like any other, and the decode over the cache pool gives the same bits."""
    rng = np.random.default_rng(110)
    lens = [700, 300]
    table, n_slots = page_table(rng, lens)
    cache = random_cache(rng, n_slots, 2)
    desc = kvq.make_desc(1, 2, 12, n_slots, "fp8b")
    host = kvq.KVPool.allocate(desc, device="pinned")
    host.buf.copy_(torch.from_numpy(cache.pack().reshape(-1)))
    dpool = make_pool(cache, 12)
    small = kvq.KVPool.allocate(kvq.make_desc(1, 2, 12, 5, "fp8b"))
    rc = kvq.ResidentCache(host, small)
    cpt, loads = rc.map(0, np.where(table < 0, 0, table), lens)
    rc.load(0, loads)
    q = dev(rng.standard_normal((2, 12, 256)).astype(np.float32))
    a = decode(dpool, q, dev(table), lens)
    b = decode(small, q, dev(cpt), lens)
    assert torch.equal(a[1], b[1])
