// paged_decode_attn_fp8b: single-token attention over the fp8b pool (E4M3 codes,
// one power-of-two scale for K and one for V per 64 tokens of a KV head).
//
// A CTA takes consecutive units of the plan and streams their tiles (64 tokens,
// 32 KB of codes, contiguous) through a ring of bulk copies that runs on from unit
// to unit.  A tile goes to four of the twelve compute warps, 16 of its tokens
// each; the three sets of four take turns.  A warp does scores, softmax and
// values of its 16 tokens with nothing exchanged between warps until the unit ends:
//   S[8 heads][16 tokens] = Q K^T, m16n8k16 in fp16.  Codes are exact in fp16.
//     The query rows are fp16 high parts (rows 0-7) and low parts (rows 8-15) of
//     q 2^kq, so the product keeps 22 bits of q at no extra instruction.
//   softmax in base 2 with a running maximum m per head that moves only when a
//     score passes it by 2^8.
//   O[256 dims][8 heads] += V^T W, W = p d_v 2^(7 - E) as an fp16 pair (high, low):
//     V codes are the A operand as they are, and d_v, a power of two, goes into W.
//     E is the head's own: the largest log2(p d_v) that the warp has met, rounded
//     up, which moves as m does.  Large values without weight take no bits from the
//     others.
// The scores' C fragment is the values' B fragment: with column n of score tile j
// holding token 4 (n >> 1) + 2 j + (n & 1), lane (g, t) ends up with the tokens
// 4t .. 4t + 3 of head g, four adjacent bytes of a V row.
#include <mutex>

#include "kvq_block.cuh"

namespace kvq {
namespace {

constexpr int BD_SETS = 3, BD_WARPS = 4 * BD_SETS;    // compute warps, four to a tile
constexpr int BD_THREADS = (BD_WARPS + 4) * 32;       // and a warpgroup whose first warp copies
constexpr int BD_REGS = 128, BD_REGS_COMPUTE = 152, BD_REGS_REST = 56;   // a thread's registers at launch and after setmaxnreg
static_assert(BD_SETS * BD_REGS_COMPUTE + BD_REGS_REST <= 4 * BD_REGS, "the compute warps take what the others give back");
// A multiple of the sets, and a tile's set goes by its place in the CTA's stream, so that a stage always belongs to the same
// four warps: a set that skipped uses of a stage could take an older phase of its barrier, of the same parity, for the one it
// waits for.
constexpr int BD_STAGES = 6;
static_assert(BD_STAGES % BD_SETS == 0, "stages per set");
constexpr float BD_ZERO_V = -1000.0f;                 // the exponent of a V scale of 0, whose codes are 0 too
constexpr uint64_t BD_WAIT_NS = 2000000000ull;
constexpr int BD_RING = BD_STAGES * BT_BYTES;
struct BdTail {                                   // after the ring
    union {
        uint4 q[16][32];                          // query fragments [k-step][lane], until a unit's last tile
        float o[4][D][8];                         // merge of the warps [tile quarter][dim][head], after it
    };
    float scale[BD_STAGES][4];                    // the 16 bytes that hold the tile's scales
    float m[BD_WARPS][8], l[BD_WARPS][8], M[8], L[8], qscale[8];
    uint64_t full[BD_STAGES], empty[BD_STAGES];
    int slot_ok[BD_STAGES];
};
constexpr int BD_SMEM = BD_RING + (int)sizeof(BdTail) + 1024;   // 1,024: the ring starts on an atom's boundary
static_assert(BD_SMEM <= 232448, "227 KB a CTA");

struct BdArgs {
    const uint8_t *pool;
    PoolGeom geo;
    int layer;
    const float *q;
    const int32_t *page_table;
    int max_pages;
    const int32_t *plan;
    int n_units, n_ctas, n_seq, n_q_heads, G;
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

struct BdUnit {
    int seq, kvh, t0, t1;
};
// Unit i of the plan; false when it does not fit the call.
__device__ __forceinline__ bool load_unit(const BdArgs &A, int i, BdUnit &u) {
    const int32_t *p = A.plan + PLAN_HEADER + 4 * (int64_t)i;
    u = BdUnit{__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3)};
    return u.seq >= 0 && u.seq < A.n_seq && u.kvh >= 0 && u.kvh < A.geo.n_kv_heads && u.t0 >= 0 && u.t0 < u.t1 &&
           u.t0 % BT == 0 && u.t1 <= A.max_pages * PAGE;
}

__global__ void __launch_bounds__(BD_THREADS, 1) block_decode_kernel(BdArgs A) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    BdTail &T = *reinterpret_cast<BdTail *>(ring + BD_RING);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int G = A.G;
    if (tid < BD_STAGES) {
        mbar_init(&T.full[tid], 1);
        mbar_init(&T.empty[tid], 4);
    }
    fence_mbar_init();
    __syncthreads();
    grid_dependency_wait();
    const int32_t *start = A.plan + PLAN_HEADER + 4 * (int64_t)A.n_units;
    const int32_t *cta = start + A.n_seq * A.geo.n_kv_heads + 1 + blockIdx.x;
    const int first = __ldg(cta), last = __ldg(cta + 1);             // together with the header: one wait
    const bool good = __ldg(A.plan) == PLAN_MAGIC && __ldg(A.plan + 1) == A.n_units && __ldg(A.plan + 2) == A.n_seq &&
                      __ldg(A.plan + 3) == A.geo.n_kv_heads && __ldg(A.plan + 6) == A.n_ctas;
    if (!good && tid == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
    const int i0 = good ? max(0, first) : 0, i1 = good ? min(A.n_units, last) : 0;

    if (warp >= BD_WARPS) {                        // ---- copies ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(BD_REGS_REST));
        if (warp > BD_WARPS) return;
        const uint64_t policy = policy_evict_first();
        int it = 0;
        bool ok = true;
        for (int i = i0; i < i1 && ok; ++i) {
            BdUnit u;
            if (!load_unit(A, i, u)) continue;
            const int n_tiles = (u.t1 - u.t0 + BT - 1) / BT;
            const int32_t *row = A.page_table + (int64_t)u.seq * A.max_pages;
            const uint8_t *base = A.pool + A.layer * A.geo.layer_stride + (int64_t)u.kvh * A.geo.page_bytes;
            const int page_end = (u.t1 + PAGE - 1) >> 8;
            int held = -1, held_from = (u.t0 >> 8) - 32;
            for (int j = 0; j < n_tiles; ++j, ++it) {
                const int tile = (u.t0 >> 6) + j, page = tile >> 2, s = it % BD_STAGES, use = it / BD_STAGES;
                if (page >= held_from + 32) {      // 32 page-table entries at a time
                    held_from = page;
                    held = page + lane < page_end ? __ldg(row + page + lane) : -1;
                }
                const int slot = __shfl_sync(0xffffffffu, held, page - held_from);
                if (use > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(&T.empty[s], (use - 1) & 1, BD_WAIT_NS))) {
                    if (lane == 0) status_or(A.status, KVQ_STATUS_TIMEOUT);
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const bool there = slot >= 0 && slot < A.geo.n_pages;
                    T.slot_ok[s] = there;
                    if (there) {
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
        }
        // no copy is left in flight
        for (int o = max(0, it - BD_STAGES); o < it; ++o) mbar_wait_bounded(&T.full[o % BD_STAGES], (o / BD_STAGES) & 1, BD_WAIT_NS);
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(BD_REGS_COMPUTE));
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(BD_WARPS * 32) : "memory"); };
    // head `warp` of a unit's query
    auto load_query = [&](const BdUnit &u, float4 &a, float4 &b) {
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (warp < G) {
            const float4 *p = reinterpret_cast<const float4 *>(A.q + ((int64_t)u.seq * A.n_q_heads + u.kvh * G + warp) * D);
            a = __ldg(p + lane);
            b = __ldg(p + 32 + lane);
        }
    };
    const int set = warp >> 2, w4 = warp & 3;
    int it = 0;                                    // tiles of the units before
    bool alive = true;
    BdUnit u;
    bool fits = i0 < i1 && load_unit(A, i0, u);
    float4 qa, qb;
    if (fits) load_query(u, qa, qb);
    for (int i = i0; i < i1; ++i) {
        float *wsu = A.ws + (int64_t)i * ws_unit_floats(G);
        BdUnit next;
        const bool next_fits = i + 1 < i1 && load_unit(A, i + 1, next);
        if (!fits) {                               // an empty partial, which the merge ignores
            if (tid == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
            for (int x = tid; x < G * D; x += BD_WARPS * 32) wsu[x] = 0.0f;
            if (tid < 8) wsu[G * D + tid] = -INFINITY, wsu[G * D + 8 + tid] = 0.0f;
            u = next;
            fits = next_fits;
            if (fits) load_query(u, qa, qb);
            continue;
        }
        const int seq = u.seq, kvh = u.kvh, t0 = u.t0, t1 = u.t1, n_tiles = (t1 - t0 + BT - 1) / BT;
        // ---- query fragments, head `warp`.  k-step s = (h, i, x): lane (g, t) takes the dims 128 h + 16 (2 t + i) + 4 x + 0 .. 3
        // of head g, which are four floats of one lane here ----
        if (warp < 8) {
            const float4 v[2] = {qa, qb};
            float mx = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) mx = fmaxf(fmaxf(mx, fmaxf(fabsf(v[h].x), fabsf(v[h].y))), fmaxf(fabsf(v[h].z), fabsf(v[h].w)));
            mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));       // not negative: the bits order as the values
            // 2^kq puts the head's largest |q| into [2^12, 2^13)
            const int kq = mx > 0.0f ? max(-114, min(114, 12 - ((int)(__float_as_uint(mx) >> 23) - 127))) : 0;
            const float up = pow2i(kq);
            if (lane == 0) T.qscale[warp] = pow2i(-kq) * (1.4426950408889634f / 16.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f[4] = {v[h].x * up, v[h].y * up, v[h].z * up, v[h].w * up};
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __half2 a = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
                    const float2 r = __half22float2(a);
                    hi[j] = h2_as_u32(a);
                    lo[j] = h2_as_u32(__floats2half2_rn(f[2 * j] - r.x, f[2 * j + 1] - r.y));
                }
                T.q[8 * h + 4 * ((lane >> 2) & 1) + (lane & 3)][4 * warp + (lane >> 3)] = make_uint4(hi[0], lo[0], hi[1], lo[1]);
            }
        }
        sync();
        const float qscale = T.qscale[g];
        float o[16][4];
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.0f;
        float m = -INFINITY, l = 0.0f;             // of head g; l over this lane's tokens
        float R = -INFINITY, E = 0.0f;             // the largest score and V exponent together, and ceil(R - m); o is in units of 2^(E - 7)
        for (int j = (set + BD_SETS - it % BD_SETS) % BD_SETS; j < n_tiles && alive; j += BD_SETS) {
            const int s = (it + j) % BD_STAGES;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&T.full[s], ((it + j) / BD_STAGES) & 1, BD_WAIT_NS))) {
                if (lane == 0) status_or(A.status, KVQ_STATUS_TIMEOUT);
                alive = false;                     // this warp computes no more, but keeps the barriers
                break;
            }
            const int tok = t0 + j * BT + 16 * w4 + 4 * t;      // this lane's four tokens
            const int valid = min(4, max(0, t1 - tok));
            if (T.slot_ok[s] && t0 + j * BT + 16 * w4 < t1) {
                const uint8_t *kt = ring + s * BT_BYTES, *vt = kt + BT_K_BYTES;
                const int half = ((t0 >> 6) + j) & 1;
                const float dk = T.scale[s][2 * half], dv = T.scale[s][2 * half + 1];
                float sc[2][2][4];                 // [score tile][accumulator of the dim half]
                const uint8_t *kr[2];
                int row7[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int row = 16 * w4 + 4 * (g >> 1) + 2 * y + (g & 1);
                    kr[y] = kt + (row >> 3) * 1024 + (row & 7) * 128;
                    row7[y] = row & 7;
#pragma unroll
                    for (int h = 0; h < 2; ++h) sc[y][h][0] = sc[y][h][1] = sc[y][h][2] = sc[y][h][3] = 0.0f;
                }
#pragma unroll
                for (int ii = 0; ii < 2; ++ii) {
                    uint32_t kw[2][2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 w = lds128(kr[y] + h * 8192 + (((2 * t + ii) ^ row7[y]) << 4));
                            kw[y][h][0] = w.x; kw[y][h][1] = w.y; kw[y][h][2] = w.z; kw[y][h][3] = w.w;
                        }
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 w = lds128(&T.q[8 * h + 4 * ii + x][lane]);
                            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                uint32_t b0, b1;
                                e4m3x4_to_h2(kw[y][h][x], b0, b1);
                                mma16816(sc[y][h], q, b0, b1);
                            }
                        }
                }
                // scores of head g, tokens 4t .. 4t + 3: high and low rows, both dim halves
                const float f = dk * qscale;
                float p[4];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float v = (sc[y][0][x] + sc[y][1][x] + (sc[y][0][x + 2] + sc[y][1][x + 2])) * f;
                        p[2 * y + x] = 2 * y + x < valid ? v : -INFINITY;
                    }
                float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float ev = dv > 0.0f ? (float)((int)(__float_as_uint(dv) >> 23) - 127) : BD_ZERO_V;
                const bool ask = mx > fminf(m, R - ev) + 8.0f;
                if (__any_sync(0xffffffffu, ask)) {
                    float fo = 1.0f;
                    if (ask) {                                    // only heads that ask move
                        const float mn = fmaxf(m, mx), Rn = fmaxf(R, mx + ev), En = ceilf(Rn - mn);
                        fo = m == -INFINITY ? 0.0f : exp2f((m - mn) + (E - En));
                        l *= m == -INFINITY ? 0.0f : exp2f(m - mn);
                        m = mn;
                        R = Rn;
                        E = En;
                    }
                    const float f0 = __shfl_sync(0xffffffffu, fo, 8 * t), f1 = __shfl_sync(0xffffffffu, fo, 8 * t + 4);
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        o[x][0] *= f0;
                        o[x][1] *= f1;
                        o[x][2] *= f0;
                        o[x][3] *= f1;
                    }
                }
                const float mref = m == -INFINITY ? 0.0f : m, c = ev - E + 7.0f;
                uint32_t whi[2], wlo[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float s0 = p[2 * y] - mref, s1 = p[2 * y + 1] - mref;
                    l += ex2(s0) + ex2(s1);
                    const float w0 = ex2(s0 + c), w1 = ex2(s1 + c);      // not 2^s0 2^c: 2^s0 alone may be too small to hold
                    const __half2 h = __floats2half2_rn(w0, w1);
                    const float2 r = __half22float2(h);
                    whi[y] = h2_as_u32(h);
                    wlo[y] = h2_as_u32(__floats2half2_rn(w0 - r.x, w1 - r.y));
                }
                const uint32_t keep = valid == 4 ? 0xFFFFFFFFu : (1u << (8 * valid)) - 1u;   // codes past the end may be NaN
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    // dims 16 x + g and + 8: rows of V; (dim >> 1) & 3 = (g >> 1) & 3 for both
                    const uint8_t *vr = vt + x * 1024 + g * 64 + ((w4 ^ ((g >> 1) & 3)) << 4) + 4 * t;
                    const uint32_t va = lds32(vr) & keep, vb = lds32(vr + 512) & keep;
                    uint32_t a[4];
                    e4m3x4_to_h2(va, a[0], a[2]);
                    e4m3x4_to_h2(vb, a[1], a[3]);
                    mma16816(o[x], a, whi[0], whi[1]);
                    mma16816(o[x], a, wlo[0], wlo[1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&T.empty[s]);
        }
        it += n_tiles;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) T.m[warp][g] = m, T.l[warp][g] = l;
        if (next_fits) load_query(next, qa, qb);
        sync();
        // ---- merge of the warps: each brings its o to the unit's reference (true units: 2^(E - 7)) ----
        {
            float f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float M = T.m[0][2 * t + x];
#pragma unroll
                for (int w = 1; w < BD_WARPS; ++w) M = fmaxf(M, T.m[w][2 * t + x]);
                const float mine = T.m[warp][2 * t + x];
                const float eo = __shfl_sync(0xffffffffu, E, 8 * t + 4 * x) - 7.0f;
                f[x] = mine == -INFINITY ? 0.0f : exp2f(mine - M + eo);
            }
            if (tid < 8) {                         // head tid: the reference and the sum, for later
                float M = T.m[0][tid], L = 0.0f;
#pragma unroll
                for (int w = 1; w < BD_WARPS; ++w) M = fmaxf(M, T.m[w][tid]);
#pragma unroll
                for (int w = 0; w < BD_WARPS; ++w) L = fmaf(T.l[w][tid], T.m[w][tid] == -INFINITY ? 0.0f : ex2(T.m[w][tid] - M), L);
                T.M[tid] = M;
                T.L[tid] = L;
            }
#pragma unroll
            for (int turn = BD_SETS - 1; turn >= 0; --turn) {       // the sets add theirs one after another
                if (set == turn)
#pragma unroll
                    for (int x = 0; x < 16; ++x)
#pragma unroll
                        for (int c = 0; c < 4; c += 2) {     // heads 2t, 2t + 1 of a dim
                            float2 &to = *reinterpret_cast<float2 *>(&T.o[w4][16 * x + g + 4 * c][2 * t]);
                            float2 v = turn == BD_SETS - 1 ? make_float2(0.f, 0.f) : to;
                            v.x = fmaf(o[x][c], f[0], v.x);
                            v.y = fmaf(o[x][c + 1], f[1], v.y);
                            to = v;
                        }
                sync();
            }
        }
        const int32_t *st = start + seq * A.geo.n_kv_heads + kvh;
        const bool whole = A.out_bf16 && __ldg(st) == i && __ldg(st + 1) == i + 1;
        if (tid < D) {
            float acc[8];
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
                float4 v[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) v[w] = *reinterpret_cast<const float4 *>(&T.o[w][tid][h]);
                acc[h] = (v[0].x + v[1].x) + (v[2].x + v[3].x);
                acc[h + 1] = (v[0].y + v[1].y) + (v[2].y + v[3].y);
                acc[h + 2] = (v[0].z + v[1].z) + (v[2].z + v[3].z);
                acc[h + 3] = (v[0].w + v[1].w) + (v[2].w + v[3].w);
            }
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                if (h >= G) break;
                if (whole) {
                    const float L = T.L[h];
                    write_out(A, (int64_t)seq * A.n_q_heads + kvh * G + h, tid, L == 0.0f ? 0.0f : acc[h] / L);   // NaN stays NaN
                } else {
                    wsu[h * D + tid] = acc[h];
                }
            }
        }
        if (!whole && tid < G) wsu[G * D + tid] = T.M[tid], wsu[G * D + 8 + tid] = T.L[tid];
        sync();                                    // the next query goes where o was
        u = next;
        fits = next_fits;
    }
}

// Merge of the units of one (sequence, KV head): M = max m_u, L = sum l_u
// 2^(m_u - M), o = sum 2^(m_u - M) o_u / L for each of its heads.  A CTA takes
// 256 / SPLIT dims of all eight heads; a thread four dims of one head and every
// PARTS-th unit.  It asks for its first units' partials before it knows their
// weights, so a merge is two loads deep (the unit range, then everything else).
constexpr int BM_THREADS = 512;
constexpr int BM_BATCH = 5;                        // units of a thread loaded together
template <int SPLIT> __global__ void __launch_bounds__(BM_THREADS) block_merge_kernel(BdArgs A) {
    constexpr int COLS = D / SPLIT / 4, PARTS = BM_THREADS / 8 / COLS, CHUNK = 128;
    static_assert(PARTS * COLS * 8 == BM_THREADS, "threads");
    __shared__ float4 part[PARTS][8][COLS];
    __shared__ float s_f[CHUNK][8], s_M[8], s_L[8], s_old[8];
    grid_dependency_wait();
    const int tid = threadIdx.x, G = A.G, lane = tid & 31, warp = tid >> 5;
    const int grp = blockIdx.x / SPLIT, seq = grp / A.geo.n_kv_heads, kvh = grp - seq * A.geo.n_kv_heads;
    const int32_t *start = A.plan + PLAN_HEADER + 4 * (int64_t)A.n_units + grp;
    const int u0 = __ldg(start), u1 = __ldg(start + 1), n = u1 - u0;
    if (u0 < 0 || u1 > A.n_units || n <= 0) {
        if (tid == 0) status_or(A.status, KVQ_STATUS_BAD_PLAN);
        return;
    }
    if (n == 1) return;                            // the unit wrote the output itself
    const int c = tid % COLS, h = tid / COLS % 8, pt = tid / COLS / 8;
    const int64_t stride = ws_unit_floats(G);
    const float *ws = A.ws + u0 * stride, *mine = ws + min(h, G - 1) * D + (blockIdx.x % SPLIT) * (D / SPLIT) + 4 * c;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < n; c0 += CHUNK) {        // 128 units at a time
        const int nc = min(CHUNK, n - c0);
        float4 v[BM_BATCH];
#pragma unroll
        for (int b = 0; b < BM_BATCH; ++b) {
            const int x = pt + PARTS * b;
            v[b] = x < nc ? *reinterpret_cast<const float4 *>(mine + (c0 + x) * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // head `warp`: the reference, the units' factors, the sum.  Nothing is set before the first chunk: these warps have no
        // barrier behind them yet, so a value another thread stored could land on top of theirs
        if (warp < G) {
            float m[CHUNK / 32], l[CHUNK / 32];
#pragma unroll
            for (int x = 0; x < CHUNK / 32; ++x) {
                const float *p = ws + (c0 + lane + 32 * x) * stride + G * D + warp;
                m[x] = lane + 32 * x < nc ? p[0] : -INFINITY;
                l[x] = lane + 32 * x < nc ? p[8] : 0.0f;
            }
            __syncwarp();
            const float M0 = c0 ? s_M[warp] : -INFINITY;
            float M = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
#pragma unroll
            for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
            M = fmaxf(M, M0);
            float L = 0.0f;
#pragma unroll
            for (int x = 0; x < CHUNK / 32; ++x) {
                const float f = m[x] == -INFINITY ? 0.0f : exp2f(m[x] - M);
                if (lane + 32 * x < nc) s_f[lane + 32 * x][warp] = f;
                L = fmaf(l[x], f, L);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
            if (lane == 0) {
                const float old = M0 == -INFINITY ? 0.0f : exp2f(M0 - M);
                s_old[warp] = old;
                s_L[warp] = fmaf(c0 ? s_L[warp] : 0.0f, old, L);
                s_M[warp] = M;
            }
        }
        __syncthreads();
        if (c0 > 0 && h < G) {
            const float old = s_old[h];
            acc.x *= old;
            acc.y *= old;
            acc.z *= old;
            acc.w *= old;
        }
        for (int b0 = 0; b0 < nc; b0 += PARTS * BM_BATCH) {
            if (b0 > 0)
#pragma unroll
                for (int b = 0; b < BM_BATCH; ++b) {
                    const int x = b0 + pt + PARTS * b;
                    v[b] = x < nc ? *reinterpret_cast<const float4 *>(mine + (c0 + x) * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int b = 0; b < BM_BATCH; ++b) {
                const int x = b0 + pt + PARTS * b;
                const float w = x < nc && h < G ? s_f[x][h] : 0.0f;
                acc.x = fmaf(v[b].x, w, acc.x);
                acc.y = fmaf(v[b].y, w, acc.y);
                acc.z = fmaf(v[b].z, w, acc.z);
                acc.w = fmaf(v[b].w, w, acc.w);
            }
        }
        __syncthreads();
    }
    if (PARTS > 1) {
        part[pt][h][c] = acc;
        __syncthreads();
        if (pt > 0) return;
#pragma unroll
        for (int x = 1; x < PARTS; ++x) {          // the parts in order
            const float4 v = part[x][h][c];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
    }
    if (h >= G) return;
    const float inv = s_L[h] == 0.0f ? 0.0f : 1.0f / s_L[h];
    const int64_t at = ((int64_t)seq * A.n_q_heads + kvh * G + h) * D + (blockIdx.x % SPLIT) * (D / SPLIT) + 4 * c;
    const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2 *>(A.out_bf16 + at) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    if (A.out_f32) *reinterpret_cast<float4 *>(A.out_f32 + at) = o;
}

}  // namespace

cudaError_t launch_block_decode(const uint8_t *pool, const PoolGeom &geo, int layer, const float *q,
                                const int32_t *page_table, int max_pages, const int32_t *plan,
                                const kvq_plan_info &info, int n_ctas, float *ws, int32_t *status, uint16_t *out_bf16,
                                float *out_f32, cudaStream_t s) {
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            cudaFuncAttributes fa;
            cudaError_t e = cudaFuncGetAttributes(&fa, block_decode_kernel);
            if (e != cudaSuccess) return e;
            if (fa.numRegs != BD_REGS) return cudaErrorInvalidConfiguration;    // setmaxnreg.inc would wait for good
            e = cudaFuncSetAttribute(block_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BD_SMEM);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    const int n_q = info.n_kv_heads * info.group;
    const BdArgs a{pool, geo, layer, q, page_table, max_pages, plan, info.n_units, n_ctas, info.n_seq, n_q, info.group, ws,
                   status, out_bf16, out_f32};
    cudaError_t e = launch_ex(block_decode_kernel, dim3((unsigned)n_ctas), dim3(BD_THREADS), BD_SMEM, s, false, a);
    if (e != cudaSuccess || !out_bf16 || info.n_units == info.n_seq * info.n_kv_heads) return e;
    // few ranges, each cut into many units, are merged by 16 or 4 CTAs each, many by one: as many as fit the SMs at once
    // (1 x 32,768 tokens of four KV heads: 21.3 us with 4, 20.1 with 16; 48 ragged sequences of two: 54 us with 4, 48 with 1)
    const int groups = info.n_seq * info.n_kv_heads, sms = device_sms();
    if (groups <= sms / 16) return launch_ex(block_merge_kernel<16>, dim3((unsigned)groups * 16), dim3(BM_THREADS), 0, s, false, a);
    if (groups <= sms / 4) return launch_ex(block_merge_kernel<4>, dim3((unsigned)groups * 4), dim3(BM_THREADS), 0, s, false, a);
    return launch_ex(block_merge_kernel<1>, dim3((unsigned)groups), dim3(BM_THREADS), 0, s, false, a);
}

}  // namespace kvq
