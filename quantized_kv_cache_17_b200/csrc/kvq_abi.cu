// C ABI of the library: argument validation, pool layout, split plan, and the
// launches.  See include/kvq.h for the contract of every entry point.
#include <algorithm>
#include <cstring>
#include <functional>
#include <memory>
#include <new>
#include <vector>

#include "kvq_block.cuh"

using namespace kvq;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_desc(const kvq_pool_desc *d) {
    if (!d) return KVQ_EINVAL;
    if (d->n_layers <= 0 || d->n_kv_heads <= 0 || d->n_q_heads <= 0 || d->n_pages <= 0) return KVQ_EINVAL;
    if (!host_valid_format(d->fmt)) return KVQ_EINVAL;
    if (d->head_dim != KVQ_HEAD_DIM || d->page_tokens != KVQ_PAGE_TOKENS) return KVQ_EUNSUPPORTED;
    if (d->n_q_heads % d->n_kv_heads != 0) return KVQ_EINVAL;
    if (d->n_q_heads / d->n_kv_heads > KVQ_MAX_GROUP) return KVQ_EUNSUPPORTED;
    return KVQ_OK;
}

int64_t tile_bytes_for(int fmt) {
    const int kp = host_part_k(fmt), vp = host_part_v(fmt);
    return part_code_bytes(kp) + part_scale_bytes(kp) + part_code_bytes(vp) + part_scale_bytes(vp);
}

void fill_layout(const kvq_pool_desc *d, kvq_layout *L) {
    const int kp = host_part_k(d->fmt), vp = host_part_v(d->fmt);
    L->k_codes_off = 0;
    if (d->fmt == KVQ_FP8B) {
        L->tile_bytes = BT_BYTES;
        L->v_codes_off = BT_K_BYTES;
        L->k_scales_off = B_SCALES_OFF;
        L->v_scales_off = B_SCALES_OFF + 4;
        L->page_bytes = B_PAGE_BYTES;
    } else {
        L->tile_bytes = tile_bytes_for(d->fmt);
        L->k_scales_off = part_code_bytes(kp);
        L->v_codes_off = L->k_scales_off + part_scale_bytes(kp);
        L->v_scales_off = L->v_codes_off + part_code_bytes(vp);
        L->page_bytes = L->tile_bytes * TILES_PER_PAGE;
    }
    L->head_stride = L->page_bytes;
    L->slot_stride = (int64_t)d->n_kv_heads * L->page_bytes;
    L->layer_stride = (int64_t)d->n_pages * L->slot_stride;
    L->total_bytes = (int64_t)d->n_layers * L->layer_stride;
    L->bytes_per_token_head = L->tile_bytes / (d->fmt == KVQ_FP8B ? BT : TILE);
}

int check_pool(const kvq_pool *pool, int layer, PoolGeom *geo) {
    if (!pool || !pool->base) return KVQ_EINVAL;
    const int rc = check_desc(&pool->desc);
    if (rc) return rc;
    if (!aligned16(pool->base)) return KVQ_EALIGN;
    if (layer < 0 || layer >= pool->desc.n_layers) return KVQ_EINVAL;
    kvq_layout L;
    fill_layout(&pool->desc, &L);
    geo->layer_stride = L.layer_stride;
    geo->slot_stride = L.slot_stride;
    geo->page_bytes = L.page_bytes;
    geo->n_pages = pool->desc.n_pages;
    geo->n_kv_heads = pool->desc.n_kv_heads;
    return KVQ_OK;
}

// Prefill plan: what a part of a row tile costs beyond its steps of 128 keys, in
// steps (its query, its output and the rescaling of its first steps; prompts of 568,
// 873 and 170 tokens, the second at 5,604, took 156, 146, 142.5 and 146 us planned
// with 4, 5, 6 and 8, 512 tokens at 32,768 340, 341.5, 340.5 and 339.5), the shortest
// part worth a partial result (8 x 5 tokens at 64 to 4,095 keys: 27.3, 28.7, 29.0,
// 31.8 and 34.4 us with 1, 2, 3, 4 and 6), and how much longer than the cut plan's
// the longest CTA may be with whole tiles, which need no partial results and no merge:
// with more tiles than CTAs, where cuts are units on top of the tiles (us cut and
// whole: 4 steps longer 67.0 and 62.0, 8 longer 394 and 389, 10 longer 320 and 319.5,
// 13 longer 369 and 372, 16 longer 154 and 173), and with fewer, where a part is all
// that a CTA has (2 longer 18.2 and 18.4, 4 longer 18.0 and 21.2, 6 longer 18.3 and 23.9).
constexpr int64_t PFB_TILE_COST = 8, PFB_MIN_PART = 2, PFB_CUT_COST = 10, PFB_CUT_COST_FEW = 2;

// Decode plan of fp8b: what a unit costs beyond its steps of 64 tokens, in steps
// (its query, the merge of its warps, its result and its share of the units' merge;
// 48 ragged sequences took 50, 48, 45, 41, 39.6, 40.2 and 41 us planned with 1, 2,
// 3, 4, 6, 8 and 10, 32,768 tokens 21.1, 20.1, 19.7 and from 4 on 19.2), and the
// shortest unit worth cutting off.
constexpr int64_t BD_UNIT_COST = 6, BD_MIN_PART = 2;

// The (sequence, KV head) ranges one after another, cut where a CTA has its share,
// so that a CTA takes consecutive units and all CTAs about the same; the units
// start table is followed by the CTAs' (n_ctas + 1 entries, header entry 6 holds
// n_ctas).  Ranges that are longer or shorter than a share need no CTA of their
// own: four sequences of 8,192 to 262,144 tokens differ by 1 % between CTAs, where
// whole CTAs per range leave 13 %.
int block_decode_plan(int n_seq, int n_kv, int G, const int32_t *seq_len, int n_ctas, int32_t *plan, int plan_capacity,
                      kvq_plan_info *info) {
    const int64_t groups = (int64_t)n_seq * n_kv;
    auto steps_of = [&](int b) { return ((int64_t)seq_len[b] + STEP_TOKENS - 1) / STEP_TOKENS; };
    int64_t total = 0, longest = 0;
    for (int b = 0; b < n_seq; ++b) total += (steps_of(b) + BD_UNIT_COST) * n_kv;
    if (groups > (1 << 24)) return KVQ_EUNSUPPORTED;
    struct Count {
        int64_t units = 0, ctas = 0;
    };
    auto walk = [&](int64_t share, int32_t *U, int32_t *start, int32_t *cta) {
        Count c;
        int64_t used = 0;
        if (cta) cta[0] = 0;
        auto close = [&]() {
            ++c.ctas;
            used = 0;
            if (cta) cta[c.ctas] = (int32_t)c.units;
        };
        longest = 0;
        for (int b = 0; b < n_seq; ++b)
            for (int g = 0; g < n_kv; ++g) {
                if (start) start[(int64_t)b * n_kv + g] = (int32_t)c.units;
                const int64_t steps = steps_of(b);
                for (int64_t s0 = 0; s0 < steps;) {
                    const int64_t room = share - used - BD_UNIT_COST, rest = steps - s0;
                    if (room < BD_MIN_PART && rest > room && used > 0) {
                        close();
                        continue;
                    }
                    const int64_t n = rest < room + BD_MIN_PART ? rest : std::max(room, BD_MIN_PART);
                    if (U) {
                        int32_t *u = U + 4 * c.units;
                        u[0] = b;
                        u[1] = g;
                        u[2] = (int32_t)(s0 * STEP_TOKENS);
                        u[3] = (int32_t)std::min<int64_t>((s0 + n) * STEP_TOKENS, seq_len[b]);
                    }
                    ++c.units;
                    s0 += n;
                    used += n + BD_UNIT_COST;
                    longest = std::max(longest, n);
                    if (used >= share) close();
                }
            }
        if (used > 0) close();
        if (start) start[groups] = (int32_t)c.units;
        return c;
    };
    int64_t lo = std::max<int64_t>(BD_MIN_PART + BD_UNIT_COST, (total + n_ctas - 1) / n_ctas), hi = std::max(lo, total);
    while (lo < hi) {                      // a share of the whole total needs one CTA
        const int64_t mid = lo + (hi - lo) / (hi > 2 * lo ? 16 : 2);
        if (walk(mid, nullptr, nullptr, nullptr).ctas <= n_ctas) hi = mid;
        else lo = mid + 1;
    }
    const Count c = walk(lo, nullptr, nullptr, nullptr);
    if (c.units > (1 << 24)) return KVQ_EUNSUPPORTED;
    const int64_t len = (int64_t)plan_len_for((int)c.units, n_seq, n_kv) + c.ctas + 1;
    info->n_units = (int32_t)c.units;
    info->n_seq = n_seq;
    info->n_kv_heads = n_kv;
    info->group = G;
    info->plan_len = (int32_t)len;
    info->chunk_tokens = (int32_t)(longest * STEP_TOKENS);
    info->workspace_bytes = ws_bytes_for((int)c.units, G, (int)groups);
    if (!plan || plan_capacity < len) return KVQ_ESIZE;
    const int32_t head[PLAN_HEADER] = {PLAN_MAGIC, (int32_t)c.units, n_seq, n_kv, G, info->chunk_tokens, (int32_t)c.ctas, 0};
    std::copy(head, head + PLAN_HEADER, plan);
    int32_t *U = plan + PLAN_HEADER, *start = U + 4 * c.units;
    walk(lo, U, start, start + groups + 1);
    return KVQ_OK;
}

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA; }

}  // namespace

// Host-side checks of a decode call, shared by every decode entry point (and
// by the workspace-free one, which must run them before it touches its
// scratch array).  Fills geo on success.
int kvq::check_decode_args(int fmt, const kvq_pool *pool, int layer, const float *q, const int32_t *page_table,
                           int max_pages, const int32_t *plan, const kvq_plan_info *info, uint64_t workspace_bytes,
                           const uint16_t *out_bf16, const float *out_f32, PoolGeom *geo) {
    int rc = check_pool(pool, layer, geo);
    if (rc) return rc;
    if (pool->desc.fmt != fmt) return KVQ_EINVAL;
    if (!q || !page_table || !plan || !info || max_pages <= 0) return KVQ_EINVAL;
    if (!aligned16(q)) return KVQ_EALIGN;
    const int G = pool->desc.n_q_heads / pool->desc.n_kv_heads;
    if (info->group != G || info->n_kv_heads != pool->desc.n_kv_heads || info->n_units <= 0 || info->n_seq <= 0)
        return KVQ_EINVAL;
    if ((int64_t)max_pages * PAGE > INT32_MAX) return KVQ_EINVAL;
    if (info->workspace_bytes != ws_bytes_for(info->n_units, G, info->n_seq * info->n_kv_heads)) return KVQ_EINVAL;
    if (workspace_bytes < info->workspace_bytes) return KVQ_ESIZE;
    if ((out_bf16 && !aligned16(out_bf16)) || (out_f32 && !aligned16(out_f32))) return KVQ_EALIGN;
    if (!out_bf16 && out_f32) return KVQ_EINVAL;
    return KVQ_OK;
}

namespace {

int decode_common(int fmt, bool tc, const kvq_pool *pool, int layer, const float *q, const int32_t *page_table,
                  int max_pages, const int32_t *plan, const kvq_plan_info *info, float *workspace,
                  uint64_t workspace_bytes, int32_t *status, void *stream, uint16_t *out_bf16 = nullptr,
                  float *out_f32 = nullptr, const float *k_new = nullptr, const float *v_new = nullptr) {
    PoolGeom geo;
    if (!workspace) return KVQ_EINVAL;
    if (!aligned16(workspace)) return KVQ_EALIGN;
    const int rc = check_decode_args(fmt, pool, layer, q, page_table, max_pages, plan, info, workspace_bytes,
                                     out_bf16, out_f32, &geo);
    if (rc) return rc;
    if (fmt == KVQ_FP8B) {
        const int64_t n_ctas = (int64_t)info->plan_len - plan_len_for(info->n_units, info->n_seq, info->n_kv_heads) - 1;
        if (n_ctas < 1 || n_ctas > info->n_units) return KVQ_EINVAL;      // another format's plan
        return cuda_rc(launch_block_decode(static_cast<const uint8_t *>(pool->base), geo, layer, q, page_table, max_pages,
                                           plan, *info, (int)n_ctas, workspace, status, out_bf16, out_f32,
                                           static_cast<cudaStream_t>(stream)));
    }
    const int inverse = host_rotated_v(fmt) ? 1 : 0;
    return cuda_rc(launch_decode(fmt, tc, static_cast<const uint8_t *>(pool->base), geo, layer, q, page_table,
                                 max_pages, plan, *info, workspace, status, inverse, out_bf16, out_f32,
                                 static_cast<cudaStream_t>(stream), k_new, v_new));
}

}  // namespace

extern "C" {

const char *kvq_version(void) { return "kvq 0.1 (sm_100a)"; }

int kvq_pool_bytes(const kvq_pool_desc *desc, uint64_t *bytes) {
    const int rc = check_desc(desc);
    if (rc) return rc;
    if (!bytes) return KVQ_EINVAL;
    kvq_layout L;
    fill_layout(desc, &L);
    *bytes = (uint64_t)L.total_bytes;
    return KVQ_OK;
}

int kvq_pool_layout(const kvq_pool_desc *desc, kvq_layout *out) {
    const int rc = check_desc(desc);
    if (rc) return rc;
    if (!out) return KVQ_EINVAL;
    fill_layout(desc, out);
    return KVQ_OK;
}

int q_rotate(const float *q, float *q_rot, int64_t n_vec, void *stream) {
    if (n_vec < 0) return KVQ_EINVAL;
    if (n_vec == 0) return KVQ_OK;
    if (!q || !q_rot) return KVQ_EINVAL;
    if (!aligned16(q) || !aligned16(q_rot)) return KVQ_EALIGN;
    if (n_vec > ((int64_t)1 << 36)) return KVQ_EINVAL;
    return cuda_rc(launch_q_rotate(q, q_rot, n_vec, static_cast<cudaStream_t>(stream)));
}

int kv_append(const kvq_pool *pool, int layer, const float *k, const float *v, int64_t n_rows,
              const int32_t *row_seq, const int32_t *row_pos, const int32_t *page_table, int max_pages, int n_seq,
              int32_t *status, void *stream) {
    PoolGeom geo;
    int rc = check_pool(pool, layer, &geo);
    if (rc) return rc;
    if (pool->desc.fmt == KVQ_FP8B) return KVQ_EUNSUPPORTED;   // rows in any order cannot share a tile's scale
    if (n_rows < 0 || max_pages <= 0 || n_seq <= 0) return KVQ_EINVAL;
    if (n_rows == 0) return KVQ_OK;
    if (!k || !v || !row_pos || !page_table) return KVQ_EINVAL;
    if (!aligned16(k) || !aligned16(v)) return KVQ_EALIGN;
    if ((int64_t)max_pages * PAGE > INT32_MAX || n_rows * geo.n_kv_heads > ((int64_t)1 << 34)) return KVQ_EINVAL;
    return cuda_rc(launch_append(pool->desc.fmt, static_cast<uint8_t *>(pool->base), geo, layer, k, v, n_rows,
                                 row_seq, row_pos, page_table, max_pages, n_seq, status,
                                 static_cast<cudaStream_t>(stream)));
}

int kv_append_q_rotate(const kvq_pool *pool, int layer, const float *k, const float *v, int64_t n_rows,
                       const int32_t *row_seq, const int32_t *row_pos, const int32_t *page_table, int max_pages,
                       int n_seq, const float *q, float *q_rot, int64_t n_vec, int32_t *status, void *stream) {
    PoolGeom geo;
    int rc = check_pool(pool, layer, &geo);
    if (rc) return rc;
    if (pool->desc.fmt == KVQ_FP8B) return KVQ_EUNSUPPORTED;
    if (n_rows < 0 || n_vec < 0 || max_pages <= 0 || n_seq <= 0) return KVQ_EINVAL;
    if (n_rows == 0 && n_vec == 0) return KVQ_OK;
    if (n_rows > 0 && (!k || !v || !row_pos || !page_table)) return KVQ_EINVAL;
    if (n_vec > 0 && (!q || !q_rot)) return KVQ_EINVAL;
    if ((n_rows > 0 && (!aligned16(k) || !aligned16(v))) || (n_vec > 0 && (!aligned16(q) || !aligned16(q_rot))))
        return KVQ_EALIGN;
    if ((int64_t)max_pages * PAGE > INT32_MAX || n_rows * geo.n_kv_heads > ((int64_t)1 << 34) ||
        n_vec > ((int64_t)1 << 34))
        return KVQ_EINVAL;
    return cuda_rc(launch_append_rotate(pool->desc.fmt, static_cast<uint8_t *>(pool->base), geo, layer, k, v, n_rows,
                                        row_seq, row_pos, page_table, max_pages, n_seq, status, q, q_rot, n_vec,
                                        static_cast<cudaStream_t>(stream)));
}

int kvq_decode_plan(const kvq_pool_desc *desc, int n_seq, const int32_t *seq_len, int max_pages, int n_ctas,
                    int32_t *plan, int plan_capacity, kvq_plan_info *info) {
    int rc = check_desc(desc);
    if (rc) return rc;
    if (n_seq <= 0 || !seq_len || !info || max_pages <= 0 || n_ctas < 0) return KVQ_EINVAL;
    if ((int64_t)max_pages * PAGE > INT32_MAX) return KVQ_EINVAL;
    const int n_kv = desc->n_kv_heads, G = desc->n_q_heads / desc->n_kv_heads;
    std::vector<int64_t> steps(n_seq);
    int64_t total = 0;
    for (int b = 0; b < n_seq; ++b) {
        if (seq_len[b] <= 0 || (int64_t)seq_len[b] > (int64_t)max_pages * PAGE) return KVQ_EINVAL;
        steps[b] = (seq_len[b] + STEP_TOKENS - 1) / STEP_TOKENS;
        total += steps[b] * n_kv;
    }
    if (n_ctas == 0) {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return KVQ_ECUDA;
        n_ctas = sms;   // one decode CTA per SM
    }
    if (desc->fmt == KVQ_FP8B) return block_decode_plan(n_seq, n_kv, G, seq_len, n_ctas, plan, plan_capacity, info);
    auto units_for = [&](int64_t c) {
        int64_t n = 0;
        for (int b = 0; b < n_seq; ++b) n += n_kv * ((steps[b] + c - 1) / c);
        return n;
    };
    int64_t maxsteps = *std::max_element(steps.begin(), steps.end());
    int64_t c = std::max<int64_t>(1, (total + n_ctas - 1) / n_ctas);
    if (c > maxsteps) c = maxsteps;
    while (c < maxsteps && units_for(c) > n_ctas) ++c;
    const int64_t n_units = units_for(c);
    if (n_units > (1 << 24)) return KVQ_EUNSUPPORTED;
    const int len = plan_len_for((int)n_units, n_seq, n_kv);
    info->n_units = (int32_t)n_units;
    info->n_seq = n_seq;
    info->n_kv_heads = n_kv;
    info->group = G;
    info->plan_len = len;
    info->chunk_tokens = (int32_t)(c * STEP_TOKENS);
    info->workspace_bytes = ws_bytes_for((int)n_units, G, n_seq * n_kv);
    if (!plan || plan_capacity < len) return KVQ_ESIZE;
    plan[0] = PLAN_MAGIC;
    plan[1] = (int32_t)n_units;
    plan[2] = n_seq;
    plan[3] = n_kv;
    plan[4] = G;
    plan[5] = (int32_t)(c * STEP_TOKENS);
    plan[6] = plan[7] = 0;
    int32_t *units = plan + PLAN_HEADER;
    int32_t *start = units + 4 * n_units;
    int u = 0;
    for (int b = 0; b < n_seq; ++b) {
        const int64_t nu = (steps[b] + c - 1) / c;
        const int64_t base = steps[b] / nu, rem = steps[b] % nu;
        for (int g = 0; g < n_kv; ++g) {
            start[b * n_kv + g] = u;
            int64_t s0 = 0;
            for (int64_t k = 0; k < nu; ++k) {
                const int64_t ns = base + (k < rem ? 1 : 0);
                units[4 * u + 0] = b;
                units[4 * u + 1] = g;
                units[4 * u + 2] = (int32_t)(s0 * STEP_TOKENS);
                units[4 * u + 3] = (int32_t)std::min<int64_t>((s0 + ns) * STEP_TOKENS, seq_len[b]);
                s0 += ns;
                ++u;
            }
        }
    }
    start[n_seq * n_kv] = u;
    return KVQ_OK;
}

int paged_decode_attn_int8(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,
                           const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,
                           int32_t *status, void *stream) {
    return decode_common(KVQ_INT8, true, pool, layer, q, page_table, max_pages, plan, info, workspace,
                         workspace_bytes, status, stream);
}

int paged_decode_attn_q4_0(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,
                           const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,
                           int32_t *status, void *stream) {
    return decode_common(KVQ_Q4_0, true, pool, layer, q, page_table, max_pages, plan, info, workspace,
                         workspace_bytes, status, stream);
}

int paged_decode_attn_k8v4(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,
                           const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,
                           int32_t *status, void *stream) {
    return decode_common(KVQ_K8V4, true, pool, layer, q, page_table, max_pages, plan, info, workspace,
                         workspace_bytes, status, stream);
}

int paged_decode_attn_fp8(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,
                          const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,
                          int32_t *status, void *stream) {
    return decode_common(KVQ_FP8, true, pool, layer, q, page_table, max_pages, plan, info, workspace,
                         workspace_bytes, status, stream);
}

int paged_decode_attn_nvfp4(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,
                            const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,
                            int32_t *status, void *stream) {
    return decode_common(KVQ_NVFP4, true, pool, layer, q, page_table, max_pages, plan, info, workspace,
                         workspace_bytes, status, stream);
}

int paged_decode_attn_fp8b(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,
                           const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,
                           int32_t *status, void *stream) {
    return decode_common(KVQ_FP8B, true, pool, layer, q, page_table, max_pages, plan, info, workspace,
                         workspace_bytes, status, stream);
}

int paged_decode_attn_cudacore(int fmt, const kvq_pool *pool, int layer, const float *q, const int32_t *page_table,
                               int max_pages, const int32_t *plan, const kvq_plan_info *info, float *workspace,
                               uint64_t workspace_bytes, int32_t *status, void *stream) {
    if (!host_valid_format(fmt)) return KVQ_EINVAL;
    if (fmt == KVQ_FP8 || fmt == KVQ_NVFP4 || fmt == KVQ_FP8B) return KVQ_EUNSUPPORTED;   // the control covers the three 2-part formats
    if (pool) {
        const int G = pool->desc.n_kv_heads > 0 ? pool->desc.n_q_heads / pool->desc.n_kv_heads : 0;
        if (G != 4 && G != 6 && G != 8) return KVQ_EUNSUPPORTED;
    }
    return decode_common(fmt, false, pool, layer, q, page_table, max_pages, plan, info, workspace, workspace_bytes,
                         status, stream);
}

#define KVQ_COMBINED(NAME, FMT)                                                                                 \
    int NAME(const kvq_pool *pool, int layer, const float *q, const int32_t *page_table, int max_pages,              \
             const int32_t *plan, const kvq_plan_info *info, float *workspace, uint64_t workspace_bytes,             \
             uint16_t *out_bf16, float *out_f32, int32_t *status, void *stream) {                                    \
        if (!out_bf16) return KVQ_EINVAL;                                                                            \
        return decode_common(FMT, true, pool, layer, q, page_table, max_pages, plan, info, workspace,               \
                             workspace_bytes, status, stream, out_bf16, out_f32);                                   \
    }
KVQ_COMBINED(paged_decode_attn_int8_combined, KVQ_INT8)
KVQ_COMBINED(paged_decode_attn_q4_0_combined, KVQ_Q4_0)
KVQ_COMBINED(paged_decode_attn_k8v4_combined, KVQ_K8V4)
KVQ_COMBINED(paged_decode_attn_fp8_combined, KVQ_FP8)
KVQ_COMBINED(paged_decode_attn_nvfp4_combined, KVQ_NVFP4)
KVQ_COMBINED(paged_decode_attn_fp8b_combined, KVQ_FP8B)
#undef KVQ_COMBINED

#define KVQ_STEP(NAME, FMT)                                                                                     \
    int NAME(const kvq_pool *pool, int layer, const float *q, const float *k_new, const float *v_new,              \
             const int32_t *page_table, int max_pages, const int32_t *plan, const kvq_plan_info *info,            \
             float *workspace, uint64_t workspace_bytes, uint16_t *out_bf16, float *out_f32, int32_t *status,      \
             void *stream) {                                                                                       \
        if (!out_bf16 || !k_new || !v_new) return KVQ_EINVAL;                                                      \
        if (!aligned16(k_new) || !aligned16(v_new)) return KVQ_EALIGN;                                             \
        return decode_common(FMT, true, pool, layer, q, page_table, max_pages, plan, info, workspace,             \
                             workspace_bytes, status, stream, out_bf16, out_f32, k_new, v_new);                   \
    }
KVQ_STEP(paged_decode_step_int8, KVQ_INT8)
KVQ_STEP(paged_decode_step_q4_0, KVQ_Q4_0)
KVQ_STEP(paged_decode_step_k8v4, KVQ_K8V4)
KVQ_STEP(paged_decode_step_fp8, KVQ_FP8)
KVQ_STEP(paged_decode_step_nvfp4, KVQ_NVFP4)
#undef KVQ_STEP

int kvq_prefill_split(const kvq_pool_desc *desc, int pos0, int n_tok, int n_sms, int *n_split,
                      uint64_t *workspace_bytes) {
    uint64_t pb = 0;
    if (!desc || !n_split || !workspace_bytes) return KVQ_EINVAL;
    const int rc = kvq_pool_bytes(desc, &pb);
    if (rc) return rc;
    if (n_tok <= 0 || pos0 < 0 || (int64_t)pos0 + n_tok > INT32_MAX || n_sms < 0) return KVQ_EINVAL;
    const int sms = n_sms ? n_sms : 148;
    const int G = desc->n_q_heads / desc->n_kv_heads;
    const int64_t n_rows = (int64_t)n_tok * G;
    const int64_t ctas = (n_rows + 63) / 64 * desc->n_kv_heads;    // CTAs of one part (64 rows each)
    const int64_t t_end = (int64_t)pos0 + n_tok;
    // cost of a choice: waves of CTAs times the longest part
    int best = 1;
    int64_t best_cost = (ctas + sms - 1) / sms * t_end;
    for (int s = 2; s <= PF_MAX_SPLIT; ++s) {
        const int st = prefill_split_tokens(pos0, n_tok, s);
        if (!st) break;
        const int64_t longest = std::max<int64_t>(st, t_end - (int64_t)(s - 1) * st);
        const int64_t cost = (ctas * s + sms - 1) / sms * longest;
        if (cost < best_cost) {
            best = s;
            best_cost = cost;
        }
    }
    *n_split = best;
    *workspace_bytes = best > 1 ? (uint64_t)best * desc->n_kv_heads * n_rows * PF_WS_STRIDE * sizeof(float) : 0;
    return KVQ_OK;
}

int paged_prefill_attn(const kvq_pool *pool, int layer, const float *q, int seq, int pos0, int n_tok,
                       const int32_t *page_table, int max_pages, int n_seq, int n_split, float *workspace,
                       uint64_t workspace_bytes, uint16_t *out_bf16, float *out_f32, int32_t *status, void *stream) {
    PoolGeom geo;
    const int rc = check_pool(pool, layer, &geo);
    if (rc) return rc;
    if (pool->desc.fmt == KVQ_FP8B) return KVQ_EUNSUPPORTED;   // paged_prefill_attn_fp8b
    if (!q || !page_table || !out_bf16 || n_tok <= 0 || pos0 < 0 || max_pages <= 0 || seq < 0 || seq >= n_seq)
        return KVQ_EINVAL;
    if ((int64_t)max_pages * PAGE > INT32_MAX || (int64_t)pos0 + n_tok > (int64_t)max_pages * PAGE) return KVQ_EINVAL;
    if ((int64_t)n_tok * pool->desc.n_q_heads > ((int64_t)1 << 28)) return KVQ_EINVAL;
    if (n_split < 1 || n_split > PF_MAX_SPLIT) return KVQ_EINVAL;
    const int split_tokens = prefill_split_tokens(pos0, n_tok, n_split);
    if (n_split > 1) {
        if (!split_tokens || !workspace) return KVQ_EINVAL;
        const uint64_t need = (uint64_t)n_split * pool->desc.n_kv_heads * ((uint64_t)n_tok * pool->desc.n_q_heads /
                                                                            pool->desc.n_kv_heads) *
                              PF_WS_STRIDE * sizeof(float);
        if (workspace_bytes < need) return KVQ_ESIZE;
        if (!aligned16(workspace)) return KVQ_EALIGN;
    }
    if (!aligned16(q) || !aligned16(out_bf16) || (out_f32 && !aligned16(out_f32))) return KVQ_EALIGN;
    return cuda_rc(launch_prefill(pool->desc.fmt, static_cast<const uint8_t *>(pool->base), geo, layer, q, seq, pos0,
                                  n_tok, page_table, max_pages, pool->desc.n_q_heads, n_split, split_tokens,
                                  workspace, host_rotated_v(pool->desc.fmt) ? 1 : 0, out_bf16, out_f32, status,
                                  static_cast<cudaStream_t>(stream)));
}

int kv_append_rope(const kvq_pool *pool, int layer, const float *cos_sin, int n_pos, int rot_dim, int interleaved,
                   const void *q, const void *k, const void *v, int dtype, int64_t q_stride, int64_t k_stride,
                   int64_t v_stride, int64_t n_rows, const int32_t *row_start, const int32_t *pos0,
                   const int32_t *page_table, int max_pages, int n_seq, void *q_out, int q_dtype, int32_t *status,
                   void *stream) {
    PoolGeom geo;
    const int rc = check_pool(pool, layer, &geo);
    if (rc) return rc;
    if (n_rows < 0 || n_seq <= 0 || max_pages <= 0 || (int64_t)max_pages * PAGE > INT32_MAX) return KVQ_EINVAL;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1)) return KVQ_EINVAL;
    if (dtype < KVQ_F32 || dtype > KVQ_F16) return KVQ_EINVAL;
    if (n_rows == 0) return KVQ_OK;
    if (!k != !v || (!k && !q) || !q != !q_out) return KVQ_EINVAL;
    if (q && q_dtype != KVQ_F32 && q_dtype != dtype) return KVQ_EINVAL;
    if (q && q_dtype != KVQ_F32 && pool->desc.fmt != KVQ_FP8B) return KVQ_EUNSUPPORTED;   // those decodes take fp32
    if (rot_dim && (!cos_sin || n_pos <= 0)) return KVQ_EINVAL;
    const int n_q = pool->desc.n_q_heads;
    // keeps the grid and the row arithmetic in range; row_start is int32
    if (n_rows > (1 << 26) || n_seq > (1 << 24) || n_rows * n_q > ((int64_t)1 << 31) ||
        (n_rows / 64 + 2 * (int64_t)n_seq) * geo.n_kv_heads * 2 + (n_rows * n_q + 63) / 64 >= INT32_MAX)
        return KVQ_EINVAL;
    if ((k && (k_stride < (int64_t)geo.n_kv_heads * D || v_stride < (int64_t)geo.n_kv_heads * D)) ||
        (q && q_stride < (int64_t)n_q * D))
        return KVQ_EINVAL;
    if (!row_start || !pos0 || !page_table) return KVQ_EINVAL;
    const int64_t esize = dtype == KVQ_F32 ? 4 : 2;
    if ((rot_dim && !aligned16(cos_sin)) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        (k && (k_stride * esize % 16 || v_stride * esize % 16)) || (q && q_stride * esize % 16))
        return KVQ_EALIGN;
    RopeArgs R{layer, cos_sin, n_pos, rot_dim, interleaved, q, k, v, q_stride, k_stride, v_stride, n_rows,
               row_start, pos0, page_table, max_pages, n_seq, n_q, q_out, status};
    return cuda_rc(launch_rope_append(pool->desc.fmt, static_cast<uint8_t *>(pool->base), geo, R, dtype, q ? q_dtype : KVQ_F32,
                                      static_cast<cudaStream_t>(stream)));
}

int kvq_prefill_plan(const kvq_pool_desc *desc, int n_seq, const int32_t *pos0, const int32_t *n_tok, int max_pages,
                     int n_ctas, int32_t *plan, int plan_capacity, kvq_prefill_info *info) {
    const int rc = check_desc(desc);
    if (rc) return rc;
    if (desc->fmt != KVQ_FP8B) return KVQ_EUNSUPPORTED;
    if (n_seq <= 0 || !pos0 || !n_tok || !info || max_pages <= 0 || n_ctas < 0 || n_ctas > (1 << 16)) return KVQ_EINVAL;
    if ((int64_t)max_pages * PAGE > INT32_MAX) return KVQ_EINVAL;
    const int n_kv = desc->n_kv_heads, G = desc->n_q_heads / n_kv;
    if (n_ctas == 0) {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return KVQ_ECUDA;
        n_ctas = sms;   // one prefill CTA per SM
    }
    // Work in steps of 128 keys; every row tile costs PFB_TILE_COST more, for its
    // query and its output.
    int64_t rows = 0, total = 0, tiles = 0;
    for (int b = 0; b < n_seq; ++b) {
        if (pos0[b] < 0 || n_tok[b] < 0 || (int64_t)pos0[b] + n_tok[b] > (int64_t)max_pages * PAGE) return KVQ_EINVAL;
        rows += n_tok[b];
    }
    if (rows * G > INT32_MAX || rows * desc->n_q_heads > ((int64_t)1 << 31)) return KVQ_EUNSUPPORTED;
    auto steps_of = [&](int b, int64_t r0) {
        const int64_t last = std::min<int64_t>(n_tok[b], (r0 + PFB_ROWS - 1) / G + 1);   // tokens up to the tile's last
        return (pos0[b] + last + PFB_KEYS - 1) / PFB_KEYS;
    };
    for (int b = 0; b < n_seq; ++b)
        for (int64_t r0 = 0; r0 < (int64_t)n_tok[b] * G; r0 += PFB_ROWS) {
            total += (steps_of(b, r0) + PFB_TILE_COST) * n_kv;
            tiles += n_kv;
        }
    if (tiles > (1 << 24)) return KVQ_EUNSUPPORTED;
    if (plan_capacity < 0) return KVQ_EINVAL;
    // Walk the row tiles in order and cut where a CTA has its share.  Parts shorter
    // than PFB_MIN_PART steps are not made, and a part costs PFB_TILE_COST whether
    // it is a whole tile or not, so the share that n_ctas CTAs need is searched for.
    struct Count {
        int64_t units = 0, merges = 0, slots = 0, ctas = 0;
    };
    auto walk = [&](int64_t share, int32_t *U, int32_t *M, int32_t *S) {
        Count c;
        int64_t used = 0, row_start = 0;
        if (S) S[0] = 0;
        auto close = [&]() {
            ++c.ctas;
            used = 0;
            if (S) S[c.ctas] = (int32_t)c.units;
        };
        for (int b = 0; b < n_seq; ++b) {
            for (int g = 0; g < n_kv; ++g)
                for (int64_t r0 = 0; r0 < (int64_t)n_tok[b] * G; r0 += PFB_ROWS) {
                    const int64_t steps = steps_of(b, r0), slot0 = c.slots;
                    int64_t s0 = 0, parts = 0;
                    while (s0 < steps) {
                        const int64_t room = share - used - PFB_TILE_COST, rest = steps - s0;
                        if (room < PFB_MIN_PART && rest > room && used > 0) {     // nothing worth starting here
                            close();
                            continue;
                        }
                        const int64_t n = rest < room + PFB_MIN_PART ? rest : std::max(room, PFB_MIN_PART);
                        const bool cut = n < rest || s0 > 0;
                        if (U) {
                            const int64_t keys = std::min<int64_t>(n_tok[b], (r0 + PFB_ROWS - 1) / G + 1) + pos0[b];
                            const int32_t u[PFB_UNIT] = {b, g, (int32_t)r0, (int32_t)(s0 * PFB_KEYS),
                                                         (int32_t)std::min<int64_t>((s0 + n) * PFB_KEYS, keys),
                                                         cut ? (int32_t)c.slots : -1, (int32_t)row_start, pos0[b], n_tok[b], 0, 0, 0};
                            std::copy(u, u + PFB_UNIT, U + c.units * PFB_UNIT);
                        }
                        ++c.units;
                        if (cut) ++c.slots, ++parts;
                        s0 += n;
                        used += n + PFB_TILE_COST;
                        if (used >= share) close();
                    }
                    if (parts) {
                        if (M) {
                            const int32_t m[PFB_MERGE] = {g, (int32_t)r0, (int32_t)slot0, (int32_t)parts, (int32_t)row_start, n_tok[b], 0, 0};
                            std::copy(m, m + PFB_MERGE, M + c.merges * PFB_MERGE);
                        }
                        ++c.merges;
                    }
                }
            row_start += n_tok[b];
        }
        if (used > 0) close();
        return c;
    };
    int64_t lo = std::max<int64_t>(PFB_MIN_PART + PFB_TILE_COST, (total + n_ctas - 1) / n_ctas), hi = std::max(lo, total);
    while (lo < hi) {                      // a share of the whole total needs one CTA
        const int64_t mid = lo + (hi - lo) / (hi > 2 * lo ? 16 : 2);   // the answer is near the mean
        if (walk(mid, nullptr, nullptr, nullptr).ctas <= n_ctas) hi = mid;
        else lo = mid + 1;
    }
    Count c = walk(lo, nullptr, nullptr, nullptr);
    // Where whole tiles, the longest first, each to the CTA with the least, come out
    // about as even, nothing is cut.  (Not tried for so many that cuts are a small
    // share of the work.)
    struct Tile {
        int64_t steps, row_start;
        int32_t b, g, r0, cta;
    };
    using Load = std::pair<int64_t, int32_t>;
    const int32_t n_whole = (int32_t)std::min<int64_t>(n_ctas, tiles);
    const int64_t limit = lo + (tiles > n_ctas ? PFB_CUT_COST : PFB_CUT_COST_FEW);
    const bool try_whole = c.merges > 0 && tiles <= (1 << 18);
    std::unique_ptr<Tile[]> whole(try_whole ? new (std::nothrow) Tile[tiles] : nullptr);
    std::unique_ptr<Load[]> least(try_whole ? new (std::nothrow) Load[n_whole] : nullptr);
    if (whole && least) {
        int64_t row_start = 0, longest = 0, n = 0;
        for (int b = 0; b < n_seq; row_start += n_tok[b], ++b)
            for (int g = 0; g < n_kv; ++g)
                for (int64_t r0 = 0; r0 < (int64_t)n_tok[b] * G; r0 += PFB_ROWS)
                    whole[n++] = {steps_of(b, r0), row_start, b, g, (int32_t)r0, 0};
        auto in_order = [](const Tile &x, const Tile &y) {
            return x.b != y.b ? x.b < y.b : x.g != y.g ? x.g < y.g : x.r0 < y.r0;
        };
        std::sort(whole.get(), whole.get() + n, [&](const Tile &x, const Tile &y) { return x.steps != y.steps ? x.steps > y.steps : in_order(x, y); });
        for (int32_t i = 0; i < n_whole; ++i) least[i] = {0, i};         // a heap already
        for (int64_t i = 0; i < n && longest <= limit; ++i) {
            std::pop_heap(least.get(), least.get() + n_whole, std::greater<Load>());
            Load &x = least[n_whole - 1];
            whole[i].cta = x.second;
            x.first += whole[i].steps + PFB_TILE_COST;
            longest = std::max(longest, x.first);
            std::push_heap(least.get(), least.get() + n_whole, std::greater<Load>());
        }
        if (longest <= limit) {
            c = Count{tiles, 0, 0, n_whole};
            std::sort(whole.get(), whole.get() + n, [&](const Tile &x, const Tile &y) {
                return x.cta != y.cta ? x.cta < y.cta : x.steps != y.steps ? x.steps > y.steps : in_order(x, y);
            });
        } else {
            whole.reset();
        }
    } else {
        whole.reset();
    }
    const int64_t len = pfb_plan_len(c.units, c.merges, c.ctas);
    if (len > INT32_MAX) return KVQ_EUNSUPPORTED;
    info->n_units = (int32_t)c.units;
    info->n_ctas = (int32_t)c.ctas;
    info->n_merges = (int32_t)c.merges;
    info->n_slots = (int32_t)c.slots;
    info->n_seq = n_seq;
    info->n_rows = (int32_t)rows;
    info->n_kv_heads = n_kv;
    info->group = G;
    info->plan_len = (int32_t)len;
    info->reserved = 0;
    info->workspace_bytes = (uint64_t)c.slots * PFB_SLOT * sizeof(float);
    if (!plan || plan_capacity < len) return KVQ_ESIZE;
    const int32_t head[PLAN_HEADER] = {PFB_MAGIC, (int32_t)c.units, n_seq, (int32_t)rows, n_kv, G, (int32_t)c.merges, (int32_t)c.ctas};
    std::copy(head, head + PLAN_HEADER, plan);
    int32_t *U = plan + PLAN_HEADER, *M = U + c.units * PFB_UNIT;
    if (!whole) {
        walk(lo, U, M, M + c.merges * PFB_MERGE);
        return KVQ_OK;
    }
    int32_t *S = M;                        // no merges
    S[0] = 0;
    for (int64_t i = 0; i < tiles; ++i) {
        const Tile &t = whole[i];
        const int64_t keys = std::min<int64_t>(n_tok[t.b], ((int64_t)t.r0 + PFB_ROWS - 1) / G + 1) + pos0[t.b];
        const int32_t u[PFB_UNIT] = {t.b, t.g, t.r0, 0, (int32_t)keys, -1, (int32_t)t.row_start, pos0[t.b], n_tok[t.b], 0, 0, 0};
        std::copy(u, u + PFB_UNIT, U + i * PFB_UNIT);
        S[t.cta + 1] = (int32_t)i + 1;
    }
    return KVQ_OK;
}

int paged_prefill_attn_fp8b(const kvq_pool *pool, int layer, const void *q, int q_dtype, int64_t q_stride,
                            const int32_t *page_table, int max_pages, const int32_t *plan,
                            const kvq_prefill_info *info, float *workspace, uint64_t workspace_bytes,
                            uint16_t *out_bf16, float *out_f32, int32_t *status, void *stream) {
    PoolGeom geo;
    const int rc = check_pool(pool, layer, &geo);
    if (rc) return rc;
    if (pool->desc.fmt != KVQ_FP8B) return KVQ_EINVAL;
    if (!info || max_pages <= 0 || (int64_t)max_pages * PAGE > INT32_MAX) return KVQ_EINVAL;
    const int n_q = pool->desc.n_q_heads;
    if (info->group != n_q / geo.n_kv_heads || info->n_kv_heads != geo.n_kv_heads || info->n_seq <= 0 ||
        info->n_units < 0 || info->n_ctas < 0 || info->n_merges < 0 || info->n_slots < 0 || info->n_rows < 0 ||
        info->plan_len != pfb_plan_len(info->n_units, info->n_merges, info->n_ctas) ||
        info->workspace_bytes != (uint64_t)info->n_slots * PFB_SLOT * sizeof(float))
        return KVQ_EINVAL;
    if (q_dtype < KVQ_F32 || q_dtype > KVQ_F16) return KVQ_EINVAL;
    if (info->n_units == 0) return KVQ_OK;
    if (!q || !page_table || !plan || !out_bf16 || q_stride < (int64_t)n_q * D || info->n_ctas == 0) return KVQ_EINVAL;
    if (info->workspace_bytes > 0) {
        if (!workspace) return KVQ_EINVAL;
        if (workspace_bytes < info->workspace_bytes) return KVQ_ESIZE;
    }
    if (!aligned16(q) || !aligned16(plan) || !aligned16(workspace) || !aligned16(out_bf16) || !aligned16(out_f32) ||
        q_stride * (q_dtype == KVQ_F32 ? 4 : 2) % 16)
        return KVQ_EALIGN;
    return cuda_rc(launch_block_prefill(static_cast<const uint8_t *>(pool->base), geo, layer, q, q_dtype, q_stride,
                                        page_table, max_pages, plan, *info, workspace, status, out_bf16, out_f32,
                                        static_cast<cudaStream_t>(stream)));
}

int attn_combine(const float *workspace, const int32_t *plan, const kvq_plan_info *info, int inverse_fwht,
                 uint16_t *out_bf16, float *out_f32, void *stream) {
    if (!workspace || !plan || !info || !out_bf16) return KVQ_EINVAL;
    if (!aligned16(workspace) || !aligned16(out_bf16) || (out_f32 && !aligned16(out_f32))) return KVQ_EALIGN;
    if (info->n_seq <= 0 || info->n_kv_heads <= 0 || info->group <= 0 || info->group > KVQ_MAX_GROUP ||
        info->n_units <= 0)
        return KVQ_EINVAL;
    return cuda_rc(launch_combine(workspace, plan, *info, inverse_fwht, out_bf16, out_f32,
                                  static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
