// paged_decode_attn_fp8b: single-token attention over the fp8b pool (E4M3 codes,
// one power-of-two scale for K and one for V per 64 tokens of a KV head).
//
// Per unit of the split plan, one CTA streams the unit's tiles (64 tokens, 32 KB
// of codes, contiguous) through a ring of bulk copies.  A tile goes to four of
// the eight compute warps, 16 of its tokens each; even tiles to warps 0-3, odd
// ones to warps 4-7.  A warp does scores, softmax and values of its 16 tokens
// with nothing exchanged between warps until the unit ends:
//   S[8 heads][16 tokens] = Q K^T, m16n8k16 in fp16.  Codes are exact in fp16.
//     The query rows are fp16 high parts (rows 0-7) and low parts (rows 8-15) of
//     q 2^kq, so the product keeps 22 bits of q at no extra instruction.
//   softmax in base 2 with a running maximum per head that moves only when a
//     score passes it by 2^8 (the weights then stay below 2^8).
//   O[256 dims][8 heads] += V^T W, W = p d_v as an fp16 pair (high, low): V codes
//     are the A operand as they are, and d_v, a power of two, goes into W relative
//     to the largest d_v the warp has met.
// The scores' C fragment is the values' B fragment: with column n of score tile j
// holding token 4 (n >> 1) + 2 j + (n & 1), lane (g, t) ends up with the tokens
// 4t .. 4t + 3 of head g, four adjacent bytes of a V row.
#include <mutex>

#include "kvq_block.cuh"

namespace kvq {
namespace {

constexpr int BD_STAGES = 6;
constexpr int BD_WARPS = 8;                       // compute warps
constexpr int BD_THREADS = (BD_WARPS + 1) * 32;   // and the copy warp
constexpr uint64_t BD_WAIT_NS = 2000000000ull;
constexpr int BD_OSTRIDE = 260;                   // floats of a head's row in the merge: heads 2t, 2t+1 of a store fall on their own banks
constexpr int BD_RING = BD_STAGES * BT_BYTES;
// after the ring: the query (8 x 256 fp32), scales, barriers, softmax state
struct BdTail {
    float q[8][D];
    float scale[BD_STAGES][4];                    // the 16 bytes that hold the tile's scales
    float m[BD_WARPS][8], l[BD_WARPS][8];
    float e[BD_WARPS];
    float w[BD_WARPS][8];
    float L[8];
    uint64_t full[BD_STAGES], empty[BD_STAGES];
    int slot_ok[BD_STAGES];
};
constexpr int BD_SMEM = BD_RING + (int)sizeof(BdTail) + 1024;   // 1,024: the ring starts on an atom's boundary
static_assert(BD_WARPS * 8 * BD_OSTRIDE * 4 <= BD_RING, "merge buffers fit in the ring");

struct BdArgs {
    const uint8_t *pool;
    PoolGeom geo;
    int layer;
    const float *q;
    const int32_t *page_table;
    int max_pages;
    const int32_t *plan;
    int n_units, n_seq, n_q_heads, G;
    float *ws;
    int32_t *status;
    uint16_t *out_bf16;       // null: every unit leaves a partial
    float *out_f32;
};

__device__ __forceinline__ float pow2i(int e) { return e < -126 ? 0.0f : __uint_as_float((uint32_t)(min(e, 127) + 127) << 23); }

__device__ __forceinline__ void write_out(const BdArgs &A, int64_t row, int dim, float x) {
    const __nv_bfloat16 b = __float2bfloat16_rn(x);
    A.out_bf16[row * D + dim] = __bfloat16_as_ushort(b);
    if (A.out_f32) A.out_f32[row * D + dim] = x;
}

__global__ void __launch_bounds__(BD_THREADS, 1) block_decode_kernel(BdArgs A) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    BdTail &T = *reinterpret_cast<BdTail *>(ring + BD_RING);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int G = A.G, unit = blockIdx.x;
    grid_dependency_wait();
    const int32_t *u = A.plan + PLAN_HEADER + 4 * unit;
    const int seq = u[0], kvh = u[1], t0 = u[2], t1 = u[3];
    float *wsu = A.ws + (int64_t)unit * ws_unit_floats(G);
    if (A.plan[0] != PLAN_MAGIC || A.plan[1] != A.n_units || A.plan[2] != A.n_seq || A.plan[3] != A.geo.n_kv_heads ||
        seq < 0 || seq >= A.n_seq || kvh < 0 || kvh >= A.geo.n_kv_heads || t0 < 0 || t0 >= t1 || t0 % BT != 0 ||
        t1 > A.max_pages * PAGE) {
        if (tid == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
        for (int i = tid; i < G * D; i += BD_THREADS) wsu[i] = 0.0f;
        if (tid < 8) wsu[G * D + tid] = -INFINITY, wsu[G * D + 8 + tid] = 0.0f;
        return;
    }
    const int n_tiles = (t1 - t0 + BT - 1) / BT;
    if (tid < BD_STAGES) {
        mbar_init(&T.full[tid], 1);
        mbar_init(&T.empty[tid], 4);
    }
    fence_mbar_init();
    __syncthreads();

    if (warp == BD_WARPS) {                        // ---- copy warp ----
        const uint64_t policy = policy_evict_first();
        const int32_t *row = A.page_table + (int64_t)seq * A.max_pages;
        const uint8_t *base = A.pool + A.layer * A.geo.layer_stride + (int64_t)kvh * A.geo.page_bytes;
        const int page0 = t0 >> 8, page_end = (t1 + PAGE - 1) >> 8;
        int held = -1, held_from = page0 - 32, i = 0;
        for (; i < n_tiles; ++i) {
            const int tile = (t0 >> 6) + i, page = tile >> 2, s = i % BD_STAGES, use = i / BD_STAGES;
            if (page >= held_from + 32) {          // 32 page-table entries at a time
                held_from = page;
                held = page + lane < page_end ? __ldg(row + page + lane) : -1;
            }
            const int slot = __shfl_sync(0xffffffffu, held, page - held_from);
            if (use > 0 && !mbar_wait_bounded(&T.empty[s], (use - 1) & 1, BD_WAIT_NS)) {
                if (lane == 0) status_or(A.status, KVQ_STATUS_TIMEOUT);
                break;
            }
            __syncwarp();
            if (lane == 0) {
                const bool ok = slot >= 0 && slot < A.geo.n_pages;
                T.slot_ok[s] = ok;
                if (ok) {
                    const uint8_t *blk = base + (int64_t)slot * A.geo.slot_stride;
                    mbar_arrive_expect_tx(&T.full[s], BT_BYTES + 16);
                    bulk_g2s(T.scale[s], blk + B_SCALES_OFF + ((tile & 3) >> 1) * 16, 16, &T.full[s], policy);
                    bulk_g2s(ring + s * BT_BYTES, blk + (tile & 3) * BT_BYTES, BT_BYTES, &T.full[s], policy);
                } else {
                    status_or(A.status, KVQ_STATUS_BAD_SLOT);
                    mbar_arrive(&T.full[s]);
                }
            }
            __syncwarp();
        }
        // no copy is left in flight
        for (int o = max(0, i - BD_STAGES); o < i; ++o) mbar_wait_bounded(&T.full[o % BD_STAGES], (o / BD_STAGES) & 1, BD_WAIT_NS);
    } else {
        // ---- query: head `warp` to shared memory, then fragments ----
        {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (warp < G) {
                const float4 *p = reinterpret_cast<const float4 *>(A.q + ((int64_t)seq * A.n_q_heads + kvh * G + warp) * D);
                a = __ldg(p + lane);
                b = __ldg(p + 32 + lane);
            }
            reinterpret_cast<float4 *>(T.q[warp])[lane] = a;
            reinterpret_cast<float4 *>(T.q[warp])[lane + 32] = b;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(BD_WARPS * 32) : "memory");
        // k-step (h, i, x): lane t holds the dims 128 h + 16 (2 t + i) + 4 x + 0 .. 3
        uint32_t qf[16][4];
        float qscale;
        {
            float mx = 0.0f;
            for (int i = 0; i < 64; ++i) mx = fmaxf(mx, fabsf(T.q[g][(i * 4 + t) & 255]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // 2^kq puts the head's largest |q| into [2^12, 2^13)
            const int kq = mx > 0.0f ? max(-114, min(114, 12 - ((int)(__float_as_uint(mx) >> 23) - 127))) : 0;
            const float up = pow2i(kq);
            qscale = pow2i(-kq) * (1.4426950408889634f / 16.0f);
#pragma unroll
            for (int s = 0; s < 16; ++s) {
                const float4 v = *reinterpret_cast<const float4 *>(&T.q[g][128 * (s >> 3) + 16 * (2 * t + ((s >> 2) & 1)) + 4 * (s & 3)]);
                const float f[4] = {v.x * up, v.y * up, v.z * up, v.w * up};
                __half2 hi[2], lo[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    hi[j] = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
                    const float2 r = __half22float2(hi[j]);
                    lo[j] = __floats2half2_rn(f[2 * j] - r.x, f[2 * j + 1] - r.y);
                }
                qf[s][0] = h2_as_u32(hi[0]);
                qf[s][1] = h2_as_u32(lo[0]);
                qf[s][2] = h2_as_u32(hi[1]);
                qf[s][3] = h2_as_u32(lo[1]);
            }
        }
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m = -INFINITY, l = 0.0f;             // of head g; l over this lane's tokens
        int E = -10000;                            // o is in units of 2^(E - 7)
        const int set = warp >> 2, w4 = warp & 3;
        for (int i = set; i < n_tiles; i += 2) {
            const int s = i % BD_STAGES;
            if (!mbar_wait_bounded(&T.full[s], (i / BD_STAGES) & 1, BD_WAIT_NS)) {
                if (lane == 0) status_or(A.status, KVQ_STATUS_TIMEOUT);
                break;
            }
            const int tok = t0 + i * BT + 16 * w4 + 4 * t;      // this lane's four tokens
            const int valid = min(4, max(0, t1 - tok));
            if (T.slot_ok[s] && t0 + i * BT + 16 * w4 < t1) {
                const uint8_t *kt = ring + s * BT_BYTES, *vt = kt + BT_K_BYTES;
                const int half = ((t0 >> 6) + i) & 1;
                const float dk = T.scale[s][2 * half], dv = T.scale[s][2 * half + 1];
                float sc[2][2][4];                 // [score tile][accumulator of the dim half]
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = 16 * w4 + 4 * (g >> 1) + 2 * j + (g & 1);
                    const uint8_t *kr = kt + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float (&c)[4] = sc[j][h];
                        c[0] = c[1] = c[2] = c[3] = 0.0f;
#pragma unroll
                        for (int ii = 0; ii < 2; ++ii) {
                            const uint4 w = lds128(kr + h * 8192 + (((2 * t + ii) ^ (row & 7)) << 4));
                            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                mma16816(c, qf[8 * h + 4 * ii + x], e4m3x2_to_h2(ws[x] & 0xFFFFu), e4m3x2_to_h2(ws[x] >> 16));
                        }
                    }
                }
                // scores of head g, tokens 4t .. 4t + 3: high and low rows, both dim halves
                const float f = dk * qscale;
                float p[4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float v = (sc[j][0][x] + sc[j][1][x] + (sc[j][0][x + 2] + sc[j][1][x + 2])) * f;
                        p[2 * j + x] = 2 * j + x < valid ? v : -INFINITY;
                    }
                float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int ev = dv > 0.0f ? (int)(__float_as_uint(dv) >> 23) - 127 : -10000;
                if (__any_sync(0xffffffffu, mx > m + 8.0f) || ev > E) {
                    const float mn = fmaxf(m, mx), fm = m == -INFINITY ? 0.0f : exp2f(m - mn);
                    const float fe = ev > E ? pow2i(E - ev) : 1.0f;
                    m = mn;
                    E = max(E, ev);
                    l *= fm;
                    const float f0 = __shfl_sync(0xffffffffu, fm, 8 * t) * fe, f1 = __shfl_sync(0xffffffffu, fm, 8 * t + 4) * fe;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        o[x][0] *= f0;
                        o[x][1] *= f1;
                        o[x][2] *= f0;
                        o[x][3] *= f1;
                    }
                }
                const float mref = m == -INFINITY ? 0.0f : m;
                const float wv = ev < -5000 ? 0.0f : pow2i(ev - E + 7);
                uint32_t whi[2], wlo[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p0 = ex2(p[2 * j] - mref), p1 = ex2(p[2 * j + 1] - mref);
                    l += p0 + p1;
                    const __half2 h = __floats2half2_rn(p0 * wv, p1 * wv);
                    const float2 r = __half22float2(h);
                    whi[j] = h2_as_u32(h);
                    wlo[j] = h2_as_u32(__floats2half2_rn(p0 * wv - r.x, p1 * wv - r.y));
                }
                const uint32_t keep = valid == 4 ? 0xFFFFFFFFu : (1u << (8 * valid)) - 1u;   // codes past the end may be NaN
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    // dims 16 x + g and + 8: rows of V; (dim >> 1) & 3 = (g >> 1) & 3 for both
                    const uint8_t *vr = vt + x * 1024 + g * 64 + ((w4 ^ ((g >> 1) & 3)) << 4) + 4 * t;
                    const uint32_t va = lds32(vr) & keep, vb = lds32(vr + 512) & keep;
                    const uint32_t a[4] = {e4m3x2_to_h2(va & 0xFFFFu), e4m3x2_to_h2(vb & 0xFFFFu), e4m3x2_to_h2(va >> 16), e4m3x2_to_h2(vb >> 16)};
                    mma16816(o[x], a, whi[0], whi[1]);
                    mma16816(o[x], a, wlo[0], wlo[1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&T.empty[s]);
        }
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) T.m[warp][g] = m, T.l[warp][g] = l;
        // o in true units would be o 2^(E - 7): the exponent goes into the warp's weight
        if (lane == 0) T.e[warp] = E > -5000 ? exp2f((float)(E - 7)) : 0.0f;
        asm volatile("bar.sync 1, %0;" ::"n"(BD_WARPS * 32) : "memory");
        // ---- merge of the eight warps ----
        float *buf = reinterpret_cast<float *>(ring);
        if (tid < 64) {
            const int w = tid >> 3, h = tid & 7;
            float M = -INFINITY;
            for (int x = 0; x < BD_WARPS; ++x) M = fmaxf(M, T.m[x][h]);
            T.w[w][h] = T.m[w][h] == -INFINITY ? 0.0f : exp2f(T.m[w][h] - M);
        }
#pragma unroll
        for (int x = 0; x < 16; ++x)
#pragma unroll
            for (int c = 0; c < 4; ++c) buf[(warp * 8 + 2 * t + (c & 1)) * BD_OSTRIDE + 16 * x + g + 8 * (c >> 1)] = o[x][c];
        asm volatile("bar.sync 1, %0;" ::"n"(BD_WARPS * 32) : "memory");
        const int32_t *start = A.plan + PLAN_HEADER + 4 * A.n_units + seq * A.geo.n_kv_heads + kvh;
        const bool whole = A.out_bf16 && start[0] == unit && start[1] == unit + 1;
        for (int h = 0; h < G; ++h) {
            float acc = 0.0f, L = 0.0f;
#pragma unroll
            for (int w = 0; w < BD_WARPS; ++w) {
                acc = fmaf(buf[(w * 8 + h) * BD_OSTRIDE + tid], T.w[w][h] * T.e[w], acc);
                L = fmaf(T.l[w][h], T.w[w][h], L);
            }
            if (whole) {
                write_out(A, (int64_t)seq * A.n_q_heads + kvh * G + h, tid, L > 0.0f ? acc / L : 0.0f);
            } else {
                wsu[h * D + tid] = acc;
                if (tid == 0) {
                    float M = -INFINITY;
                    for (int x = 0; x < BD_WARPS; ++x) M = fmaxf(M, T.m[x][h]);
                    wsu[G * D + h] = M;
                    wsu[G * D + 8 + h] = L;
                }
            }
        }
    }
}

// Merge of the units of one (sequence, query head): M = max m_u, L = sum l_u
// 2^(m_u - M), o = sum 2^(m_u - M) o_u / L, a head of four 64-lane parts.
__global__ void __launch_bounds__(256) block_merge_kernel(BdArgs A) {
    __shared__ float4 part[4][64];
    __shared__ float s_l[8], s_m[8];
    grid_dependency_wait();
    const int tid = threadIdx.x, G = A.G;
    const int row = blockIdx.x, seq = row / A.n_q_heads, hq = row - seq * A.n_q_heads, kvh = hq / G, h = hq - kvh * G;
    const int32_t *start = A.plan + PLAN_HEADER + 4 * A.n_units + seq * A.geo.n_kv_heads + kvh;
    const int u0 = start[0], u1 = start[1];
    if (u0 < 0 || u1 > A.n_units || u1 <= u0) {
        if (tid == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
        return;
    }
    if (u1 - u0 == 1 && A.plan[1] == A.n_units) return;      // the unit wrote the output itself
    const int stride = ws_unit_floats(G);
    const float *ws = A.ws;
    float M = -INFINITY;
    for (int x = u0 + tid; x < u1; x += 256) M = fmaxf(M, ws[(int64_t)x * stride + G * D + h]);
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if ((tid & 31) == 0) s_m[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 8; ++x) M = fmaxf(M, s_m[x]);
    const int c = tid & 63, pt = tid >> 6;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.0f;
#pragma unroll 8
    for (int x = u0 + pt; x < u1; x += 4) {
        const float *p = ws + (int64_t)x * stride;
        const float mu = p[G * D + h], f = mu == -INFINITY ? 0.0f : exp2f(mu - M);
        const float4 v = *reinterpret_cast<const float4 *>(p + h * D + 4 * c);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
        L = fmaf(p[G * D + 8 + h], f, L);
    }
    part[pt][c] = acc;
    if (c == 0) s_l[pt] = L;
    __syncthreads();
    if (tid < 64) {
        L = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = part[i][c];
            x[0] += v.x;
            x[1] += v.y;
            x[2] += v.z;
            x[3] += v.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) write_out(A, row, 4 * c + i, x[i] * inv);
    }
}

}  // namespace

cudaError_t launch_block_decode(const uint8_t *pool, const PoolGeom &geo, int layer, const float *q,
                                const int32_t *page_table, int max_pages, const int32_t *plan,
                                const kvq_plan_info &info, float *ws, int32_t *status, uint16_t *out_bf16,
                                float *out_f32, cudaStream_t s) {
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(block_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BD_SMEM);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    const int n_q = info.n_kv_heads * info.group;
    const BdArgs a{pool, geo, layer, q, page_table, max_pages, plan, info.n_units, info.n_seq, n_q, info.group, ws,
                   status, out_bf16, out_f32};
    cudaError_t e = launch_ex(block_decode_kernel, dim3((unsigned)info.n_units), dim3(BD_THREADS), BD_SMEM, s, false, a);
    if (e != cudaSuccess || !out_bf16 || info.n_units == info.n_seq * info.n_kv_heads) return e;
    return launch_ex(block_merge_kernel, dim3((unsigned)(info.n_seq * n_q)), dim3(256), 0, s, false, a);
}

}  // namespace kvq
