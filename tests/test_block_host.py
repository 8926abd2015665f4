"""fp8b on the host: sizes and layout, the prefill plan, and the refusals of the
new entry points.  Nothing here reaches a GPU."""
import ctypes

import numpy as np
import pytest

import quantized_kv_cache_17_b200 as kvq
from tests import block_ref as br


@pytest.fixture(scope="module", autouse=True)
def built():
    import oracle
    from quantized_kv_cache_17_b200 import build
    build.build()
    oracle.build()


def test_pool_bytes_and_layout():
    d = kvq.make_desc(3, 2, 12, 5, "fp8b")
    L = kvq.pool_layout(d)
    assert (L.tile_bytes, L.k_codes_off, L.v_codes_off, L.k_scales_off, L.v_scales_off) == (32768, 0, 16384, 131072, 131076)
    assert L.page_bytes == br.PAGE_BYTES and L.bytes_per_token_head == 512
    assert kvq.pool_bytes(d) == 3 * 5 * 2 * br.PAGE_BYTES


def test_layout_is_a_bijection():
    both = np.concatenate([br.K_MAP.ravel(), br.V_MAP.ravel()])
    assert np.array_equal(np.sort(both), np.arange(br.TILE_BYTES))


@pytest.mark.parametrize("amax,want", [(0.0, 0.0), (448.0, 1.0), (np.nextafter(np.float32(448.0), np.float32(500.0)), 2.0), (447.9, 1.0), (1.0, 2.0 ** -8),
                                       (0.875, 2.0 ** -9), (0.876, 2.0 ** -8), (1e-40, 2.0 ** -120), (3.4e38, 2.0 ** 118)])
def test_scale_rule(amax, want):
    assert br.pow2_scale(float(np.float32(amax))) == want


def _units(plan, info):
    n, m = info.n_units, info.n_merges
    u = plan[8:8 + 12 * n].reshape(n, 12)
    g = plan[8 + 12 * n:8 + 12 * n + 8 * m].reshape(m, 8)
    return u, g, plan[8 + 12 * n + 8 * m:]


@pytest.mark.parametrize("pos0,toks,n_ctas", [([0], [1], 148), ([0], [777], 148), ([32256], [512], 148), ([5, 0, 900], [1, 0, 300], 7),
                                              ([100] * 64, [1] * 64, 148), ([0, 200000], [2049, 3], 148), ([7] * 9, [0] * 9, 20),
                                              ([262143], [1], 148), ([0], [2000], 1)])
@pytest.mark.parametrize("heads", [(24, 4), (4, 1), (7, 7), (16, 2)])
def test_prefill_plan_covers_every_row_and_key_once(pos0, toks, n_ctas, heads):
    hq, hkv = heads
    G = hq // hkv
    d = kvq.make_desc(1, hkv, hq, 8, "fp8b")
    plan, info = kvq.prefill_plan(d, pos0, toks, max_pages=1024, n_ctas=n_ctas)
    u, merges, start = _units(plan, info)
    assert list(plan[:8]) == [0x4B565150, info.n_units, len(pos0), sum(toks), hkv, G, info.n_merges, info.n_ctas]
    assert len(start) == info.n_ctas + 1 and start[0] == 0 and info.n_ctas <= n_ctas
    if info.n_units:
        assert start[-1] == info.n_units and (np.diff(start) >= 1).all()
    assert info.n_rows == sum(toks) and info.workspace_bytes == info.n_slots * 128 * 258 * 4
    assert sorted(u[u[:, 5] >= 0, 5]) == list(range(info.n_slots))
    row = 0
    by_tile = {}
    for x in u:
        by_tile.setdefault((x[0], x[1], x[2]), []).append(x)
    merged = {(int(m[4]), int(m[0]), int(m[1])): m for m in merges}
    for b, (p, n) in enumerate(zip(pos0, toks)):
        for h in range(hkv):
            for r0 in range(0, n * G, 128):
                parts = by_tile.pop((b, h, r0))
                end = p + min(n, (r0 + 127) // G + 1)
                assert parts[0][3] == 0 and parts[-1][4] == end
                for a, c in zip(parts, parts[1:]):
                    assert a[4] == c[3] and a[4] % 128 == 0 and c[5] == a[5] + 1
                for x in parts:
                    assert tuple(x[6:9]) == (row, p, n) and x[3] < x[4]
                if len(parts) > 1:
                    m = merged.pop((row, h, r0))
                    assert (m[2], m[3], m[5]) == (parts[0][5], len(parts), n)
                else:
                    assert parts[0][5] == -1
        row += n
    assert not by_tile and not merged


def test_prefill_plan_is_even():
    """A chunk at the end of a long prompt: no CTA gets over a tenth more than the mean (in steps of 128 keys)."""
    d = kvq.make_desc(1, 4, 24, 8, "fp8b")
    plan, info = kvq.prefill_plan(d, [32256], [512], max_pages=1024, n_ctas=148)
    u, _, start = _units(plan, info)
    steps = (u[:, 4] - u[:, 3] + 127) // 128
    per = np.add.reduceat(steps, start[:-1])
    assert info.n_ctas == 148 and per.max() <= 1.1 * per.mean()


@pytest.mark.parametrize("pos0,toks,whole", [([0], [7777], True), ([0, 901], [1025, 2047], True), ([32256], [512], False),
                                             ([5604, 0], [873, 568], False)])
def test_prefill_plan_cuts_tiles_only_where_whole_ones_are_uneven(pos0, toks, whole):
    d = kvq.make_desc(1, 4, 24, 8, "fp8b")
    plan, info = kvq.prefill_plan(d, pos0, toks, max_pages=1024, n_ctas=148)
    u, _, start = _units(plan, info)
    tiles = 4 * sum(-(-6 * n // 128) for n in toks)
    if whole:
        per = np.add.reduceat((u[:, 4] - u[:, 3] + 127) // 128 + 8, start[:-1])
        assert info.n_units == tiles and info.n_merges == info.n_slots == 0 and info.workspace_bytes == 0
        assert info.n_ctas == min(148, tiles) and per.max() <= 1.1 * per.mean() + 10
    else:
        assert info.n_units > tiles and info.n_merges > 0


def test_prefill_plan_does_not_depend_on_the_room_for_it():
    d = kvq.make_desc(1, 2, 16, 8, "fp8b")
    for pos0, toks in (([0, 0, 7], [900, 3, 400]), ([9000], [64])):
        plan, info = kvq.prefill_plan(d, pos0, toks, max_pages=1024, n_ctas=148)
        a, b = np.array(pos0, np.int32), np.array(toks, np.int32)
        exact, again = np.empty(info.plan_len, np.int32), kvq.PrefillInfo()
        args = (ctypes.byref(d), len(a), a.ctypes.data, b.ctypes.data, 1024, 148)
        assert kvq.lib().kvq_prefill_plan(*args, exact.ctypes.data, info.plan_len - 1, ctypes.byref(again)) == -5
        assert again.plan_len == info.plan_len
        assert kvq.lib().kvq_prefill_plan(*args, exact.ctypes.data, info.plan_len, ctypes.byref(again)) == 0
        assert np.array_equal(plan, exact) and bytes(info) == bytes(again)


def _pool(fmt="fp8b", hq=24, hkv=4):
    return kvq.Pool(0x10000, kvq.make_desc(1, hkv, hq, 8, fmt))


def test_refusals_of_the_append():
    L = kvq.lib()

    def call(pool=None, layer=0, cs=0x1000, n_pos=100, rot=64, inter=0, q=0x2000, k=0x3000, v=0x4000, dt=1, qs=6144, ks=1024,
             vs=1024, n_rows=4, rs=0x5000, p0=0x6000, pt=0x7000, mp=8, ns=1, qo=0x8000, qd=0):
        return L.kv_append_rope(ctypes.byref(pool or _pool()), layer, cs, n_pos, rot, inter, q, k, v, dt, qs, ks, vs, n_rows, rs, p0,
                                pt, mp, ns, qo, qd, None, None)

    assert call(layer=1) == -1 and call(n_rows=-1) == -1 and call(ns=0) == -1 and call(mp=0) == -1
    assert call(mp=1 << 24) == -1                                             # positions past 32 bits
    for rot in (-16, 8, 24, 272):
        assert call(rot=rot) == -1
    assert call(inter=2) == -1 and call(dt=3) == -1 and call(dt=-1) == -1
    assert call(k=None) == -1 and call(v=None) == -1 and call(q=None) == -1 and call(qo=None) == -1
    assert call(q=None, qo=None, k=None, v=None) == -1
    assert call(qd=2) == -1                                                   # neither fp32 nor the input's type
    assert call(pool=_pool("q4_0"), qd=1) == -2                               # the decode of q4_0 takes fp32
    assert call(cs=None) == -1 and call(n_pos=0) == -1
    assert call(ks=1023) == -1 and call(vs=1000) == -1 and call(qs=6143) == -1
    assert call(n_rows=(1 << 26) + 1) == -1
    assert call(rs=None) == -1 and call(p0=None) == -1 and call(pt=None) == -1
    assert call(k=0x3008) == -3 and call(q=0x2002) == -3 and call(qo=0x8004) == -3 and call(cs=0x1004) == -3
    assert call(ks=1028) == -3 and call(qs=6148) == -3                        # rows off the 16-byte grid
    assert call(n_rows=0) == 0
    assert call(pool=kvq.Pool(0x10008, kvq.make_desc(1, 4, 24, 8, "fp8b"))) == -3


def test_refusals_of_entry_points_that_do_not_take_fp8b():
    L = kvq.lib()
    p = ctypes.byref(_pool())
    assert L.kv_append(p, 0, 0x1000, 0x1000, 1, None, 0x1000, 0x1000, 8, 1, None, None) == -2
    assert L.kv_append_q_rotate(p, 0, 0x1000, 0x1000, 1, None, 0x1000, 0x1000, 8, 1, 0x1000, 0x1000, 1, None, None) == -2
    assert L.paged_prefill_attn(p, 0, 0x1000, 0, 256, 4, 0x2000, 8, 1, 1, None, 0, 0x3000, None, None, None) == -2
    plan, info = kvq.decode_plan(_pool().desc, [1000], max_pages=8, n_ctas=148)
    args = (p, 0, 0x1000, 0x2000, 8, 0x3000, ctypes.byref(info), 0x4000, info.workspace_bytes)
    assert L.paged_decode_attn_cudacore(8, *args, None, None) == -2
    assert L.paged_decode_attn_fp8(*args, None, None) == -1                    # another format's entry point
    assert L.paged_decode_attn_fp8b(*args[:-1], info.workspace_bytes - 1, None, None) == -5
    assert L.paged_decode_attn_fp8b_combined(*args, None, None, None, None) == -1
    with pytest.raises(kvq.KVQError, match="KVQ_EUNSUPPORTED"):
        kvq.paged_decode_step(kvq.KVPool(_pool().desc, None), 0, None, None, None, None, None, None, None, None)


def test_refusals_of_the_prefill():
    L = kvq.lib()
    d = _pool().desc
    info = kvq.PrefillInfo()

    def plan_rc(pos0, toks, desc=d, mp=8, n_ctas=148):
        a, b = np.array(pos0, np.int32), np.array(toks, np.int32)
        return L.kvq_prefill_plan(ctypes.byref(desc), len(a), a.ctypes.data, b.ctypes.data, mp, n_ctas, None, 0, ctypes.byref(info))

    assert plan_rc([-1], [4]) == -1 and plan_rc([0], [-1]) == -1 and plan_rc([2045], [4]) == -1 and plan_rc([0], [4], mp=0) == -1
    assert plan_rc([0], [4], n_ctas=-1) == -1 and plan_rc([0], [4], desc=kvq.make_desc(1, 4, 24, 8, "fp8")) == -2
    assert plan_rc([2044], [4]) == -5
    plan, info = kvq.prefill_plan(d, [1500], [4], max_pages=8, n_ctas=148)
    assert info.workspace_bytes > 0

    def call(pool=None, q=0x1000, dt=1, qs=6144, pt=0x2000, mp=8, pl=0x3000, ws=0x4000, wb=1 << 40, out=0x5000, of=None, inf=info):
        return L.paged_prefill_attn_fp8b(ctypes.byref(pool or _pool()), 0, q, dt, qs, pt, mp, pl, ctypes.byref(inf), ws, wb, out, of, None, None)

    assert call(pool=_pool("fp8")) == -1 and call(pool=_pool(hq=16, hkv=2)) == -1
    assert call(q=None) == -1 and call(dt=3) == -1 and call(qs=6143) == -1 and call(pt=None) == -1 and call(pl=None) == -1
    assert call(out=None) == -1 and call(ws=None) == -1 and call(wb=info.workspace_bytes - 1) == -5
    assert call(q=0x1008) == -3 and call(out=0x5008) == -3 and call(of=0x6004) == -3 and call(ws=0x4008) == -3 and call(qs=6148) == -3
    for field, value in (("n_units", info.n_units + 1), ("n_slots", 0), ("group", 5), ("n_kv_heads", 2), ("plan_len", 3)):
        bad = kvq.PrefillInfo.from_buffer_copy(info)
        setattr(bad, field, value)
        assert call(inf=bad) == -1
    empty, einfo = kvq.prefill_plan(d, [10, 20], [0, 0], max_pages=8, n_ctas=148)
    assert einfo.n_units == 0 and einfo.workspace_bytes == 0 and call(inf=einfo, q=None, ws=None) == 0


def test_binding_refuses_wrong_tensors():
    import torch
    pool = kvq.KVPool(_pool().desc, torch.zeros(16, dtype=torch.uint8))
    k = torch.zeros((3, 4, 256), dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    rs, p0, pt = torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros((1, 8), **i32)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k.double(), k.double(), rs, p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k, k[:2], rs, p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k, k.half(), rs, p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k, None, rs, p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k.transpose(0, 1), k.transpose(0, 1), rs, p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k, k, rs.long(), p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k, k, rs[:1], p0, pt)
    with pytest.raises(kvq.KVQError):
        kvq.kv_append_rope(pool, 0, k, k, rs, p0, pt, cos_sin=torch.zeros((8, 64), dtype=torch.float64))
    plan, info = kvq.prefill_plan(pool.desc, [0], [4], max_pages=8, n_ctas=148)
    q = torch.zeros((3, 24, 256), dtype=torch.bfloat16)
    with pytest.raises(kvq.KVQError):
        kvq.paged_prefill_attn_fp8b(pool, 0, q, pt, None, info, None, q)


def _decode_call(**kw):
    """A decode through the binding with CPU tensors: what it refuses before it looks at the device."""
    import torch
    desc = _pool().desc
    plan, info = kvq.decode_plan(desc, [1000, 70], max_pages=8, n_ctas=148)
    a = dict(q=torch.zeros((2, 24, 256)), page_table=torch.zeros((2, 8), dtype=torch.int32), plan_dev=torch.from_numpy(plan),
             workspace=torch.zeros(info.workspace_bytes // 4), out_bf16=torch.zeros((2, 24, 256), dtype=torch.bfloat16), out_f32=None,
             status=torch.zeros(1, dtype=torch.int32))
    a.update(kw)
    pool = kvq.KVPool(desc, torch.zeros(16, dtype=torch.uint8))
    outs = (a.pop("out_bf16"), a.pop("out_f32"))
    for call in (lambda: kvq.paged_decode_attn_combined(pool, 0, a["q"], a["page_table"], a["plan_dev"], info, a["workspace"], *outs,
                                                        a["status"]),
                 lambda: kvq.paged_decode_attn_fp8b(pool, 0, a["q"], a["page_table"], a["plan_dev"], info, a["workspace"], a["status"])):
        try:
            call()
        except kvq.KVQError as e:
            yield str(e)


def test_binding_refuses_wrong_tensors_of_a_decode():
    import torch
    assert all("the current device" in m for m in _decode_call())              # nothing else is wrong with these
    for t in (torch.bfloat16, torch.float16, torch.float64):                   # a 16-bit query is not read as fp32, past its end
        msgs = list(_decode_call(q=torch.zeros((2, 24, 256), dtype=t)))
        assert len(msgs) == 2 and all("float32" in m for m in msgs)
    for kw, word in ((dict(q=torch.zeros((1, 24, 256))), "q is not"), (dict(q=torch.zeros((2, 24, 512))[..., :256]), "q is not"),
                     (dict(page_table=torch.zeros((1, 8), dtype=torch.int32)), "page_table"),
                     (dict(page_table=torch.zeros((2, 8), dtype=torch.int64)), "page_table"),
                     (dict(plan_dev=torch.zeros(20, dtype=torch.int32)), "plan_dev"),
                     (dict(plan_dev=torch.zeros(4096, dtype=torch.float32)), "plan_dev"),
                     (dict(workspace=torch.zeros(1 << 20)[::2]), "workspace"), (dict(status=torch.zeros(1)), "status")):
        msgs = list(_decode_call(**kw))
        assert len(msgs) == 2 and all(word in m for m in msgs), (kw.keys(), msgs)
    for kw in (dict(out_bf16=torch.zeros((2, 24, 256))), dict(out_bf16=torch.zeros((2, 24, 256), dtype=torch.float16)),
               dict(out_bf16=torch.zeros((1, 24, 256), dtype=torch.bfloat16)), dict(out_f32=torch.zeros((2, 24, 256), dtype=torch.bfloat16)),
               dict(out_f32=torch.zeros((2, 24, 128)))):
        assert "shaped as q" in list(_decode_call(**kw))[0]
