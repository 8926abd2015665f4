// paged_prefill_attn_fp8b: causal attention of a ragged batch's new tokens over
// the fp8b pool.
#include <mutex>

#include "kvq_block.cuh"

namespace kvq {
namespace {

struct PfbArgs {
    const uint8_t *pool;
    PoolGeom geo;
    int layer;
    const void *q;
    int64_t q_stride;
    const int32_t *page_table;
    int max_pages;
    const int32_t *plan;
    int n_units, n_seq, n_rows, n_merges, n_slots, n_ctas, G, n_q_heads;
    float *ws;
    int32_t *status;
    uint16_t *out_bf16;
    float *out_f32;
};

struct Unit {
    int seq, head, r0, k0, k1, slot, row_start, pos0, n_tok;
};

// Reads unit i of the plan; false (with a status bit) when it does not fit the call.
__device__ __forceinline__ bool load_unit(const PfbArgs &A, int i, Unit &u) {
    const int4 *p = reinterpret_cast<const int4 *>(A.plan + PLAN_HEADER + (int64_t)i * PFB_UNIT);
    const int4 a = __ldg(p), b = __ldg(p + 1), c = __ldg(p + 2);
    u = Unit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x};
    const bool ok = u.seq >= 0 && u.seq < A.n_seq && u.head >= 0 && u.head < A.geo.n_kv_heads && u.pos0 >= 0 &&
                    u.n_tok > 0 && (int64_t)u.pos0 + u.n_tok <= (int64_t)A.max_pages * PAGE && u.r0 >= 0 &&
                    u.r0 < (int64_t)u.n_tok * A.G && u.row_start >= 0 && (int64_t)u.row_start + u.n_tok <= A.n_rows &&
                    u.k0 >= 0 && u.k0 % PFB_KEYS == 0 && u.k0 < u.k1 && u.k1 <= u.pos0 + u.n_tok && u.slot < A.n_slots;
    if (!ok && threadIdx.x == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
    return ok;
}

__device__ __forceinline__ bool plan_ok(const PfbArgs &A) {
    const int4 a = __ldg(reinterpret_cast<const int4 *>(A.plan)), b = __ldg(reinterpret_cast<const int4 *>(A.plan) + 1);
    const bool ok = a.x == PFB_MAGIC && a.y == A.n_units && a.z == A.n_seq && a.w == A.n_rows &&
                    b.x == A.geo.n_kv_heads && b.y == A.G && b.z == A.n_merges && b.w == A.n_ctas;
    if (!ok && threadIdx.x == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
    return ok;
}

__device__ __forceinline__ float load_q(const void *q, int dtype, int64_t i) {
    if (dtype == KVQ_F32) return static_cast<const float *>(q)[i];
    if (dtype == KVQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(q)[i]);
    return __half2float(static_cast<const __half *>(q)[i]);
}

// One CTA per plan CTA; each warp takes four rows of a unit at a time, a lane two
// keys of a 64-token tile for the scores and eight dims for the values, in fp32.
constexpr int PS_WARPS = 8;
__global__ void __launch_bounds__(PS_WARPS * 32) block_prefill_kernel(PfbArgs A, int q_dtype) {
    __shared__ float qs[PS_WARPS][4][D];
    __shared__ float ps[PS_WARPS][4][BT];
    grid_dependency_wait();
    if (!plan_ok(A)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t *start = A.plan + PLAN_HEADER + (int64_t)A.n_units * PFB_UNIT + (int64_t)A.n_merges * PFB_MERGE;
    const int i0 = max(0, start[blockIdx.x]), i1 = min(A.n_units, start[blockIdx.x + 1]);
    for (int i = i0; i < i1; ++i) {
        Unit u;
        if (!load_unit(A, i, u)) continue;
        const int n_rows = u.n_tok * A.G;
        for (int rr = warp * 4; rr < PFB_ROWS; rr += PS_WARPS * 4) {
            const int r = u.r0 + rr;
            if (r >= n_rows) break;
            int limit[4];
            float m[4], l[4], o[4][8];
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int ri = min(r + x, n_rows - 1), tok = ri / A.G, h = u.head * A.G + ri % A.G;
                limit[x] = min(u.k1, u.pos0 + tok + 1);
                m[x] = -INFINITY;
                l[x] = 0.0f;
                for (int d = lane; d < D; d += 32)
                    qs[warp][x][d] = load_q(A.q, q_dtype, (u.row_start + tok) * A.q_stride + h * D + d);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[x][e] = 0.0f;
            }
            __syncwarp();
            for (int t0 = u.k0; t0 < limit[3]; t0 += BT) {
                const int slot = __ldg(A.page_table + (int64_t)u.seq * A.max_pages + (t0 >> 8));
                if (slot < 0 || slot >= A.geo.n_pages) {
                    if (lane == 0) status_or(A.status, KVQ_STATUS_BAD_SLOT);
                    continue;
                }
                const uint8_t *page = A.pool + A.layer * A.geo.layer_stride + (int64_t)slot * A.geo.slot_stride + (int64_t)u.head * A.geo.page_bytes;
                const uint8_t *tile = page + ((t0 >> 6) & 3) * BT_BYTES;
                const float *sc = reinterpret_cast<const float *>(page + B_SCALES_OFF) + 2 * ((t0 >> 6) & 3);
                float s[4][2] = {};
                for (int c = 0; c < 16; ++c)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(tile + block_k_off(lane + 32 * j, 16 * c));
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const float2 k = __half22float2(u32_as_h2(e4m3x2_to_h2((ww[b >> 1] >> (16 * (b & 1))) & 0xFFFFu)));
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[x][j] = fmaf(qs[warp][x][16 * c + 2 * b + 1], k.y, fmaf(qs[warp][x][16 * c + 2 * b], k.x, s[x][j]));
                        }
                    }
                const float f = sc[0] * (1.4426950408889634f / 16.0f), dv = sc[1];
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float a = t0 + lane < limit[x] ? s[x][0] * f : -INFINITY;
                    const float b = t0 + lane + 32 < limit[x] ? s[x][1] * f : -INFINITY;
                    float mx = fmaxf(a, b);
#pragma unroll
                    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    const float mn = fmaxf(m[x], mx), ref = mn == -INFINITY ? 0.0f : mn;
                    const float fac = exp2f(m[x] - ref), pa = exp2f(a - ref), pb = exp2f(b - ref);
                    m[x] = mn;
                    l[x] = l[x] * fac + pa + pb;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[x][e] *= fac;
                    ps[warp][x][lane] = pa * dv;
                    ps[warp][x][lane + 32] = pb * dv;
                }
                __syncwarp();
                for (int k = 0; k < BT && t0 + k < limit[3]; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t code = tile[BT_K_BYTES + block_v_off(k, lane * 8 + e)];
                        const float v = __low2float(u32_as_h2(e4m3x2_to_h2(code)));
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (t0 + k < limit[x]) o[x][e] = fmaf(ps[warp][x][k], v, o[x][e]);
                    }
                __syncwarp();
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (r + x >= n_rows) continue;
#pragma unroll
                for (int d = 16; d; d >>= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
                if (u.slot >= 0) {
                    float *w = A.ws + (int64_t)u.slot * PFB_SLOT;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[(rr + x) * D + lane * 8 + e] = o[x][e];
                    if (lane == 0) w[PFB_ROWS * D + rr + x] = m[x], w[PFB_ROWS * (D + 1) + rr + x] = l[x];
                } else {
                    const float inv = l[x] > 0.0f ? 1.0f / l[x] : 0.0f;
                    const int tok = (r + x) / A.G, h = u.head * A.G + (r + x) % A.G;
                    const int64_t at = ((int64_t)(u.row_start + tok) * A.n_q_heads + h) * D + lane * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        A.out_bf16[at + e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[x][e] * inv));
                        if (A.out_f32) A.out_f32[at + e] = o[x][e] * inv;
                    }
                }
            }
        }
    }
}

// The parts of a cut row tile: M = max m, L = sum l 2^(m - M), o = sum o 2^(m - M) / L.
// One warp per row, eight dims a lane.
__global__ void __launch_bounds__(256) block_prefill_merge_kernel(PfbArgs A) {
    grid_dependency_wait();
    if (!plan_ok(A)) return;
    const int lane = threadIdx.x & 31, mi = blockIdx.x >> 4, rr = (blockIdx.x & 15) * 8 + (threadIdx.x >> 5);
    const int4 *p = reinterpret_cast<const int4 *>(A.plan + PLAN_HEADER + (int64_t)A.n_units * PFB_UNIT + (int64_t)mi * PFB_MERGE);
    const int4 a = __ldg(p), b = __ldg(p + 1);
    const int head = a.x, r0 = a.y, slot0 = a.z, parts = a.w, row_start = b.x, n_tok = b.y;
    if (head < 0 || head >= A.geo.n_kv_heads || r0 < 0 || slot0 < 0 || parts < 1 || parts > A.n_slots - slot0 || n_tok <= 0 ||
        row_start < 0 || (int64_t)row_start + n_tok > A.n_rows) {
        if (threadIdx.x == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
        return;
    }
    if ((int64_t)r0 + rr >= (int64_t)n_tok * A.G) return;
    const float *ws = A.ws + (int64_t)slot0 * PFB_SLOT;
    float M = -INFINITY;
    for (int x = lane; x < parts; x += 32) M = fmaxf(M, ws[(int64_t)x * PFB_SLOT + PFB_ROWS * D + rr]);
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float o[8] = {}, L = 0.0f;
#pragma unroll 4
    for (int x = 0; x < parts; ++x) {
        const float *w = ws + (int64_t)x * PFB_SLOT;
        const float m = w[PFB_ROWS * D + rr], f = m == -INFINITY ? 0.0f : exp2f(m - M);
        const float4 v0 = *reinterpret_cast<const float4 *>(w + rr * D + lane * 8);
        const float4 v1 = *reinterpret_cast<const float4 *>(w + rr * D + lane * 8 + 4);
        L = fmaf(w[PFB_ROWS * (D + 1) + rr], f, L);
        o[0] = fmaf(v0.x, f, o[0]); o[1] = fmaf(v0.y, f, o[1]); o[2] = fmaf(v0.z, f, o[2]); o[3] = fmaf(v0.w, f, o[3]);
        o[4] = fmaf(v1.x, f, o[4]); o[5] = fmaf(v1.y, f, o[5]); o[6] = fmaf(v1.z, f, o[6]); o[7] = fmaf(v1.w, f, o[7]);
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    const int tok = (r0 + rr) / A.G, h = head * A.G + (r0 + rr) % A.G;
    const int64_t at = ((int64_t)(row_start + tok) * A.n_q_heads + h) * D + lane * 8;
    uint32_t pk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
        pk[e] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(A.out_bf16 + at) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    if (A.out_f32) {
        *reinterpret_cast<float4 *>(A.out_f32 + at) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        *reinterpret_cast<float4 *>(A.out_f32 + at + 4) = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
    }
}

}  // namespace

cudaError_t launch_block_prefill(const uint8_t *pool, const PoolGeom &geo, int layer, const void *q, int q_dtype,
                                 int64_t q_stride, const int32_t *page_table, int max_pages, const int32_t *plan,
                                 const kvq_prefill_info &info, float *ws, int32_t *status, uint16_t *out_bf16,
                                 float *out_f32, cudaStream_t s) {
    const PfbArgs a{pool, geo, layer, q, q_stride, page_table, max_pages, plan, info.n_units, info.n_seq, info.n_rows,
                    info.n_merges, info.n_slots, info.n_ctas, info.group, info.group * info.n_kv_heads, ws, status,
                    out_bf16, out_f32};
    cudaError_t e = launch_ex(block_prefill_kernel, dim3((unsigned)info.n_ctas), dim3(PS_WARPS * 32), 0, s, false, a, q_dtype);
    if (e != cudaSuccess || info.n_merges == 0) return e;
    return launch_ex(block_prefill_merge_kernel, dim3((unsigned)info.n_merges * 16), dim3(256), 0, s, false, a);
}

}  // namespace kvq
