// paged_prefill_attn_fp8b: causal attention of a ragged batch's new tokens over
// the fp8b pool.
#include <cfloat>
#include <mutex>
#include <type_traits>

#include "kvq_block.cuh"
#include "kvq_tcgen05.cuh"

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

// ---------------------------------------------------------------------------
// The kernel: one CTA per SM, 384 threads, walking its units.
//   warps 0-7  softmax.  Warp w and warp w + 4 share the 32 rows 32 (w % 4) ..; a
//              thread has one row and 64 of a step's 128 keys, one 64-token tile
//              and so one K and one V scale.
//   warps 8, 9    bulk copies of K and of V codes, each into a ring of 32 KB slots
//   warps 10, 11  one lane issues the scores' products, one the values': each waits
//                 for its own operands while the other's are in the tensor cores
// The copy and product warps' warpgroup gives registers to the softmax's two
// (setmaxnreg): at the 168 that 384 threads get, the softmax loop spilled.
// Both products take the codes as they lie in the pool (kind::f8f6f4, B operand):
//   S[128 rows][128 keys] = sum over terms of Q_i K^T: a row of Q, scaled so that
//     its largest value lies in [2^7, 2^8), is a sum of E4M3 terms, each the
//     rounding of what the earlier ones leave.  Two terms hold bf16's 8 bits (4
//     each) down to 2^-10, which is 2^-17 of the row's largest; three hold fp16's 11,
//     and fp32 is rounded to those.
//   O[128 rows][256 dims] += sum over three terms of W_i V: a weight as fp16 (11
//     bits), then three E5M2 terms of 3 bits each: E5M2 is the upper byte of fp16,
//     so a term is an integer rounding of the bits and what it leaves an exact fp16
//     difference.  E5M2 and not E4M3, for range: weights from 2^15 down to 2^-16.
// The five 8-bit passes cost 1.25 times two 16-bit ones; what they save is the
// conversion of every K and V code to 16 bits, which would move as many bytes
// through shared memory as the products themselves.
// Weights: W = 2^(s - m) 2^(e_v - E) 2^10, with s the score in base 2, m the row's
// reference, e_v the exponent of the tile's V scale, so V scales cost nothing, and
// E the row's own: the largest s - m + e_v of the keys it attends to, rounded up.
// So what a weight is measured by is the largest product of weight and V scale in
// its row; large values that the row does not see, or that have no weight in it,
// take no bits from the others.  References move only when a score, or a score and
// its V exponent, pass theirs by 2^5: the row's O is then multiplied in TMEM.
// TMEM: O 0-255, S 256-383, weights 384-479 (term i of the 32 keys c at
// 384 + 24 c + 8 i); all 512 columns are allocated.  The scores of step j + 1 are
// made as soon as the softmax has step j's in registers, behind the values of step
// j - 1 in the tensor cores' queue, so the softmax runs from step to step.  (Two
// score buffers with the weights over the scores need as many columns and make
// the scores of step j + 2 wait for the values of step j: 3,610 cycles a step.)
// ---------------------------------------------------------------------------
constexpr int PF_SOFT = 8;                       // softmax warps
constexpr int PF_THREADS = (PF_SOFT + 4) * 32;     // three warpgroups
constexpr int PF_REGS = 168;                     // a thread's registers at launch: what 384 threads can have
constexpr int PF_REGS_SOFT = 208, PF_REGS_REST = 88;
static_assert(2 * PF_REGS_SOFT + PF_REGS_REST <= 3 * PF_REGS, "the softmax warps take what the others give back");
constexpr int PF_SLOT_BYTES = 32768;
constexpr uint64_t PF_WAIT_NS = 2000000000ull;
constexpr int PF_S_COL = 256, PF_P_COL = 384;
// References move when they are passed by 2^PF_LAZY; weights are made 2^PF_SHIFT times larger, up to fp16's 2^15.  At 3 and 12 the
// first steps of a unit rescaled O about twice as often.
constexpr int PF_LAZY = 5, PF_SHIFT = 10;
static_assert(PF_LAZY + PF_SHIFT == 15, "the largest weight");
constexpr float PF_NO_E = -10000.0f;             // no key seen
constexpr float PF_ZERO_V = -1000.0f;            // the exponent of a V scale of 0, whose codes are 0 too

template <int TERMS> struct PfCfg {
    static constexpr int K_SLOTS = 2, V_SLOTS = TERMS == 2 ? 3 : 2;
    static constexpr int Q_BYTES = TERMS * 32768;
    static constexpr int RING = Q_BYTES;
    static constexpr int TAIL = RING + (K_SLOTS + V_SLOTS) * PF_SLOT_BYTES;
    static constexpr int SMEM = TAIL + 2048 + 1024;         // the tail; the ring starts on an atom's boundary
};
struct PfTail {
    uint64_t k_full[2], k_empty[2], v_full[3], v_empty[3], s_full, s_free, p_full, o_done, q_full, drained;
    uint32_t tmem;
    int abort;
    float qscale[PFB_ROWS];
    float red[2][PFB_ROWS], ev[PF_SOFT];
};
static_assert(sizeof(PfTail) <= 2048, "tail");
static_assert(PfCfg<2>::SMEM <= 232448 && PfCfg<3>::SMEM <= 232448, "227 KB a CTA");

__device__ __forceinline__ float pow2f(int e) { return e < -126 ? 0.0f : __uint_as_float((uint32_t)(min(e, 127) + 127) << 23); }

__device__ __forceinline__ uint32_t h2_to_e4m3x2(uint32_t h) {       // nearest even, saturating
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}

// The whole pair of warps (64 threads, barrier id) agrees on whether any thread asks.
__device__ __forceinline__ bool pair_any(bool ask, int id) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)ask), "r"(id)
                 : "memory");
    return r != 0;
}

// The 16 query rows of a warp (rows 16 warp .. of the tile, zeros past the last), eight dims a lane.  16-bit rows are
// held as they are, all 16 loaded at once (kept from before the unit before's result was written they were spilled, one
// wait each: 8,000 cycles a unit against 1,000); fp32 rows would need twice the registers and are read when they are used.
__device__ __forceinline__ int64_t query_row(const PfbArgs &A, const Unit &u, int r) {
    if (r >= u.n_tok * A.G) return -1;
    const int tok = r / A.G;
    return (int64_t)(u.row_start + tok) * A.q_stride + (u.head * A.G + r - tok * A.G) * D;
}
template <typename T> struct QueryRows {
    uint4 raw[16];
    __device__ __forceinline__ void load(const PfbArgs &A, const Unit &u, int warp, int lane) {
        const int64_t mine = query_row(A, u, u.r0 + 16 * warp + (lane & 15));
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            const int64_t at = __shfl_sync(0xffffffffu, mine, y);
            raw[y] = at < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(A.q) + at) + lane);
        }
    }
    __device__ __forceinline__ float largest(const PfbArgs &, int, int y) const {
        const uint32_t a = raw[y].x & 0x7FFF7FFFu, b = raw[y].y & 0x7FFF7FFFu, c = raw[y].z & 0x7FFF7FFFu, d = raw[y].w & 0x7FFF7FFFu;
        if constexpr (std::is_same_v<T, __half>) {
            const float2 f = __half22float2(__hmax2(__hmax2(u32_as_h2(a), u32_as_h2(b)), __hmax2(u32_as_h2(c), u32_as_h2(d))));
            return fmaxf(f.x, f.y);
        } else {
            auto bf = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
            const __nv_bfloat162 m = __hmax2(__hmax2(bf(a), bf(b)), __hmax2(bf(c), bf(d)));
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
    __device__ __forceinline__ void get(const PfbArgs &, int, int y, float (&x)[8]) const {
        const uint32_t w[4] = {raw[y].x, raw[y].y, raw[y].z, raw[y].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same_v<T, __half>) {
                const float2 f = __half22float2(u32_as_h2(w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
};
template <> struct QueryRows<float> {
    int64_t mine;
    __device__ __forceinline__ void load(const PfbArgs &A, const Unit &u, int warp, int lane) { mine = query_row(A, u, u.r0 + 16 * warp + (lane & 15)); }
    __device__ __forceinline__ float largest(const PfbArgs &A, int lane, int y) const {
        float x[8], m = 0.0f;
        get(A, lane, y, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
        return m;
    }
    __device__ __forceinline__ void get(const PfbArgs &A, int lane, int y, float (&x)[8]) const {
        const int64_t at = __shfl_sync(0xffffffffu, mine, y);
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(A.q) + at) + 2 * lane;
        const float4 a = at < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldg(p), b = at < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldg(p + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Loads that stay where they are written: a plain load was moved to its use, a
// step later, and cost every step its latency (1,200 cycles).
__device__ __forceinline__ float4 ld_now(const float4 *p) {
    float4 v;
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ int ld_now(const int32_t *p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two pairs of weights (fp16) to three words of four E5M2 bytes.
__device__ __forceinline__ void split_weights(uint32_t a, uint32_t b, uint32_t &t1, uint32_t &t2, uint32_t &t3) {
    const uint32_t a1 = a + 0x00800080u, b1 = b + 0x00800080u;
    t1 = __byte_perm(a1, b1, 0x7531);
    const uint32_t ra = h2_as_u32(__hsub2(u32_as_h2(a), u32_as_h2(a1 & 0xFF00FF00u)));
    const uint32_t rb = h2_as_u32(__hsub2(u32_as_h2(b), u32_as_h2(b1 & 0xFF00FF00u)));
    const uint32_t a2 = ra + 0x00800080u, b2 = rb + 0x00800080u;
    t2 = __byte_perm(a2, b2, 0x7531);
    const uint32_t sa = h2_as_u32(__hsub2(u32_as_h2(ra), u32_as_h2(a2 & 0xFF00FF00u)));
    const uint32_t sb = h2_as_u32(__hsub2(u32_as_h2(rb), u32_as_h2(b2 & 0xFF00FF00u)));
    t3 = __byte_perm(sa, sb, 0x7531);                // what is left of 11 bits has 3 at most: nothing to round above 2^-6
}

template <typename T, int TERMS>
__global__ void __launch_bounds__(PF_THREADS, 1) block_prefill_kernel(PfbArgs A) {
    using C = PfCfg<TERMS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    PfTail &X = *reinterpret_cast<PfTail *>(sm + C::TAIL);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < C::K_SLOTS; ++i) {
            mbar_init(&X.k_full[i], 1);
            mbar_init(&X.k_empty[i], 1);
        }
        for (int i = 0; i < C::V_SLOTS; ++i) {
            mbar_init(&X.v_full[i], 1);
            mbar_init(&X.v_empty[i], 1);
        }
        mbar_init(&X.s_full, 1);
        mbar_init(&X.s_free, PF_SOFT);
        mbar_init(&X.p_full, PF_SOFT);
        mbar_init(&X.o_done, 1);
        mbar_init(&X.drained, 2);
        mbar_init(&X.q_full, PF_SOFT);
        X.abort = 0;
        fence_mbar_init();
    }
    if (warp == PF_SOFT) tmem_alloc(&X.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = X.tmem;
    grid_dependency_wait();
    const int32_t *start = A.plan + PLAN_HEADER + (int64_t)A.n_units * PFB_UNIT + (int64_t)A.n_merges * PFB_MERGE + blockIdx.x;
    const int first = __ldg(start), last = __ldg(start + 1);         // together with the header: one wait
    const bool good = plan_ok(A);
    const int i0 = good ? max(0, first) : 0, i1 = good ? min(A.n_units, last) : 0;
    // A wait that gives up (2 s, or another role's did) raises the CTA's flag and the call's status.  From then on
    // nothing is copied or multiplied and no wait waits, but every role walks its loop to the end: the warps' own
    // barriers always find their partners.  Called by whole warps.
    volatile int *abort_flag = &X.abort;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        bool ok = mbar_try_wait(bar, parity);
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            while (!(ok = mbar_try_wait_sleep(bar, parity, 20000u))) {
                if (*abort_flag) break;
                if (globaltimer_ns() - t0 > PF_WAIT_NS) {
                    *abort_flag = 1;
                    status_or(A.status, KVQ_STATUS_TIMEOUT);
                    break;
                }
            }
        }
        return __all_sync(0xffffffffu, ok) && !*abort_flag;
    };

    if (warp >= PF_SOFT) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PF_REGS_REST));
        const bool is_v = warp & 1;                          // warps 8 and 10: K; 9 and 11: V
        const int slots = is_v ? C::V_SLOTS : C::K_SLOTS;
        uint64_t *full = is_v ? X.v_full : X.k_full, *empty = is_v ? X.v_empty : X.k_empty;
        uint8_t *ring = sm + C::RING + (is_v ? C::K_SLOTS * PF_SLOT_BYTES : 0);
        int slot = 0, it = 0, un = 0;
        uint32_t phase = 0;                                  // of the ring
        bool ok = true;
        auto next_slot = [&]() {
            if (++slot == slots) slot = 0, phase ^= 1;
        };
        if (warp < PF_SOFT + 2) {                            // ---- copies ----
            const uint8_t *base = A.pool + A.layer * A.geo.layer_stride;
            for (int i = i0; i < i1 && ok; ++i) {
                Unit u;
                if (!load_unit(A, i, u)) continue;
                const int nt = (u.k1 - u.k0 + PFB_KEYS - 1) / PFB_KEYS, kv_end = u.pos0 + u.n_tok;
                const int32_t *row = A.page_table + (int64_t)u.seq * A.max_pages;
                const int page_end = (u.k1 + PAGE - 1) >> 8;
                int held = -1, from = (u.k0 >> 8) - 32;      // entries of 32 pages at a time
                for (int j = 0; j < nt; ++j, ++it) {
                    const int key = u.k0 + j * PFB_KEYS, page = key >> 8;
                    if (page >= from + 32) {
                        from = page;
                        held = page + lane < page_end ? __ldg(row + page + lane) : -1;
                    }
                    const int at = __shfl_sync(0xffffffffu, held, page - from);
                    if (it >= slots && !wait(&empty[slot], phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        uint8_t *dst = ring + slot * PF_SLOT_BYTES;
                        if (at >= 0 && at < A.geo.n_pages) {
                            const uint8_t *src = base + (int64_t)at * A.geo.slot_stride + (int64_t)u.head * A.geo.page_bytes +
                                                 ((key >> 6) & 3) * BT_BYTES;
                            const int blocks = key + BT < kv_end ? 2 : 1;
                            mbar_arrive_expect_tx(&full[slot], blocks * BT_K_BYTES);
                            for (int b = 0; b < blocks; ++b) {
                                if (is_v) {
                                    bulk_g2s_plain(dst + b * BT_K_BYTES, src + b * BT_BYTES + BT_K_BYTES, BT_K_BYTES, &full[slot]);
                                } else {         // a dim half of both tiles lies together: 16 atoms, 1,024 bytes apart
                                    bulk_g2s_plain(dst + b * 8192, src + b * BT_BYTES, 8192, &full[slot]);
                                    bulk_g2s_plain(dst + 16384 + b * 8192, src + b * BT_BYTES + 8192, 8192, &full[slot]);
                                }
                            }
                        } else {
                            status_or(A.status, KVQ_STATUS_BAD_SLOT);
                            mbar_arrive(&full[slot]);
                        }
                    }
                    __syncwarp();
                    next_slot();
                }
            }
            for (int o = max(0, it - slots); o < it; ++o)    // no copy is left in flight
                mbar_wait_bounded(&full[o % slots], (o / slots) & 1, PF_WAIT_NS);
        } else if (lane == 0) {                              // ---- products: one lane, a warp for each of the two ----
            constexpr uint32_t ID_QK = umma_idesc_f8(128, 128, 0, 0), ID_PV = umma_idesc_f8(128, 256, 1, 0);
            const uint64_t q_desc = umma_desc(smem_u32(sm), 1024, 2), k_desc = umma_desc(smem_u32(ring), 1024, 2),
                           v_desc = umma_desc(smem_u32(ring), 512, 4);
            auto wait1 = [&](uint64_t *bar, uint32_t parity) {
                if (mbar_try_wait(bar, parity)) return true;
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
                    if (*abort_flag) return false;
                    if (globaltimer_ns() - t0 > PF_WAIT_NS) {
                        *abort_flag = 1;
                        status_or(A.status, KVQ_STATUS_TIMEOUT);
                        return false;
                    }
                }
                return true;
            };
            for (int i = i0; i < i1 && ok; ++i) {
                Unit u;
                if (!load_unit(A, i, u)) continue;
                const int nt = (u.k1 - u.k0 + PFB_KEYS - 1) / PFB_KEYS;
                if (!is_v) ok = wait1(&X.q_full, un & 1);
                ++un;
                for (int j = 0; j < nt && ok; ++j, ++it) {
                    ok = wait1(&full[slot], phase);
                    if (is_v) {                              // values: the weights are written
                        if (!ok || !wait1(&X.p_full, it & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t v = v_desc + slot * (PF_SLOT_BYTES >> 4);
#pragma unroll
                        for (int x = 0; x < 12; ++x) {
                            const int c = x / 3, term = x % 3;
                            umma_f8_ts(tmem, tmem + PF_P_COL + 24 * c + 8 * term, v + (((c >> 1) * BT_K_BYTES + (c & 1) * 32) >> 4), ID_PV,
                                       j > 0 || x > 0);
                        }
                        tc_commit(&X.o_done);
                    } else {                                 // scores: the ones before have been read
                        if (!ok || (it > 0 && !wait1(&X.s_free, (it - 1) & 1))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t k = k_desc + slot * (PF_SLOT_BYTES >> 4);
#pragma unroll
                        for (int x = 0; x < TERMS * 8; ++x) {
                            const uint64_t off = (((x >> 2) & 1) * 16384 + (x & 3) * 32) >> 4;
                            umma_f8_ss(tmem + PF_S_COL, q_desc + ((x >> 3) * 32768 >> 4) + off, k + off, ID_QK, x > 0);
                        }
                        tc_commit(&X.s_full);
                    }
                    tc_commit(&empty[slot]);
                    next_slot();
                }
            }
            tc_commit(&X.drained);                           // every product is complete before TMEM goes back
            mbar_wait_bounded(&X.drained, 0, PF_WAIT_NS);
        }
        __syncwarp();
    } else {                                     // ---- softmax ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PF_REGS_SOFT));
        const int part = warp >> 2, row = 32 * (warp & 3) + lane, bar = 1 + (warp & 3);
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        int it = 0;
        auto wait_s = [&](uint64_t *bar, uint32_t parity) {     // as wait, without its answer
            if (!mbar_try_wait(bar, parity)) {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait_sleep(bar, parity, 20000u) && !*abort_flag) {
                    if (globaltimer_ns() - t0 > PF_WAIT_NS) {
                        *abort_flag = 1;
                        status_or(A.status, KVQ_STATUS_TIMEOUT);
                    }
                }
            }
            __syncwarp();
        };
        for (int i = i0; i < i1; ++i) {
            Unit u;
            if (!load_unit(A, i, u)) continue;
            const int n_rows = u.n_tok * A.G, nt = (u.k1 - u.k0 + PFB_KEYS - 1) / PFB_KEYS, kv_end = u.pos0 + u.n_tok;
            // ---- query terms: rows 16 warp .. + 15, eight dims a lane ----
            QueryRows<T> rows;
            rows.load(A, u, warp, lane);
            float top[16];                               // the rows' largest magnitudes, all reductions under way at once
#pragma unroll
            for (int y = 0; y < 16; ++y)                 // not negative: the bits order as the values
                top[y] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rows.largest(A, lane, y))));
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                const int r = 16 * warp + y;
                const int kq = top[y] > 0.0f ? min(114, 7 - ((int)(__float_as_uint(top[y]) >> 23) - 127)) : 0;
                const float up = top[y] <= FLT_MAX ? pow2f(kq) : __uint_as_float(0x7FC00000u);     // an infinity makes its row NaN
                if (lane == 0) X.qscale[r] = pow2f(-kq) * (1.4426950408889634f / 16.0f);
                // scaled as fp16: exact for 16-bit types down to what E4M3 terms reach, the 11 bits of three terms for fp32
                float x[8];
                rows.get(A, lane, y, x);
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = h2_as_u32(__floats2half2_rn(x[2 * e] * up, x[2 * e + 1] * up));
                // dims 8 lane ..: half lane / 16, chunk (lane / 2) % 8, its low or high 8 bytes
                uint8_t *dst = sm + (lane >> 4) * 16384 + (r >> 3) * 1024 + (r & 7) * 128 + ((((lane >> 1) & 7) ^ (r & 7)) << 4) + (lane & 1) * 8;
#pragma unroll
                for (int t = 0; t < TERMS; ++t) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = h2_to_e4m3x2(h[e]);
                        if (t + 1 < TERMS) h[e] = h2_as_u32(__hsub2(u32_as_h2(h[e]), u32_as_h2(e4m3x2_to_h2(w[e]))));   // exact
                    }
                    *reinterpret_cast<uint2 *>(dst + t * 32768) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&X.q_full);
            asm volatile("bar.sync 5, %0;" ::"n"(PF_SOFT * 32) : "memory");      // qscale of every row
            if (i + 1 < i1) {                            // the next unit's rows come to L2 meanwhile
                Unit v;
                if (load_unit(A, i + 1, v)) {
                    const int64_t at = query_row(A, v, v.r0 + 16 * warp + (lane & 15));
                    if (at >= 0)
                        for (int x = lane >> 4; x < 2 * (int)sizeof(T); x += 2)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t *>(static_cast<const T *>(A.q) + at) + 128 * x));
                }
            }
            const float qs = X.qscale[row];
            const int r = u.r0 + row;
            const int limit = r < n_rows ? min(u.k1, u.pos0 + r / A.G + 1) : u.k1;
            const int low = min(u.k1, u.pos0 + u.r0 / A.G + 1);                  // keys below it are seen by every row
            const int32_t *pt = A.page_table + (int64_t)u.seq * A.max_pages;
            const uint8_t *kv = A.pool + A.layer * A.geo.layer_stride + (int64_t)u.head * A.geo.page_bytes + B_SCALES_OFF;
            // What a step needs of its tiles' scales is the same for every row: lane i works it out for step i of 32, and a
            // step takes it from there.  rec_k: this half's K scale, -1 where the page is not there and 0 past the sequence's
            // end, where the pool may hold anything (a sign of its own for one half's page would clear the other's V).  rec_v: the
            // exponent of this half's V scale.  The next 32 steps' page slots and scales are loaded while these are used.
            auto load_slot = [&](int j) { return j < nt ? ld_now(pt + ((u.k0 + j * PFB_KEYS) >> 8)) : -1; };
            auto load_scales = [&](int slot, int j) {
                if (slot < 0 || slot >= A.geo.n_pages) return make_float4(0.f, 0.f, 0.f, 0.f);
                return ld_now(reinterpret_cast<const float4 *>(kv + (int64_t)slot * A.geo.slot_stride + (((u.k0 >> 7) + j) & 1) * 16));
            };
            int slot = load_slot(lane);
            float4 sc = load_scales(slot, lane);
            float rec_k = 0.0f, rec_v = 0.0f;
            float m = -INFINITY, l = 0.0f;               // the score's reference, and the sum of 2^(s - m)
            float R = -INFINITY, E = PF_NO_E;            // the largest s + e_v, and ceil(R - m)
            for (int j = 0; j < nt; ++j, ++it) {
                const int key0 = u.k0 + j * PFB_KEYS, mine = key0 + 64 * part;
                if ((j & 31) == 0) {
                    const int step = j + lane;
                    const bool second = u.k0 + step * PFB_KEYS + BT < kv_end;
                    const float dk = part ? (second ? sc.z : 0.0f) : sc.x, dv = part ? (second ? sc.w : 0.0f) : sc.y;
                    rec_k = slot >= 0 && slot < A.geo.n_pages ? fmaxf(dk, 0.0f) : -1.0f;
                    rec_v = dv > 0.0f ? (float)((int)(__float_as_uint(dv) >> 23) - 127) : PF_ZERO_V;
                    slot = load_slot(step + 32);
                }
                if ((j & 31) == 16) sc = load_scales(slot, (j & ~31) + 32 + lane);
                const float dk = __shfl_sync(0xffffffffu, rec_k, j & 31);
                const float ev = __shfl_sync(0xffffffffu, rec_v, j & 31);
                const bool there = !(dk < 0.0f);
                wait_s(&X.s_full, it & 1);
                tc_fence_after();
                const uint32_t scol = tl + PF_S_COL + 64 * part, pcol = tl + PF_P_COL + 48 * part;
                uint32_t s[64];
                tmem_ld32<0>(scol, s);
                tmem_ld32<32>(scol + 32, s);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&X.s_free);
                // masked keys: past the row's limit, or in a page that is not there (their scores, and the scale of a
                // tile that has no tokens, can be anything); a scale of 0 makes every score 0
                const bool nonzero = dk > 0.0f;
                if (!there || key0 + PFB_KEYS > low || !nonzero) {
                    const int n = there ? limit - mine : 0;
#pragma unroll
                    for (int x = 0; x < 64; ++x) s[x] = x < n ? (nonzero ? s[x] : 0u) : 0xFF800000u;
                }
                const float f = nonzero ? fmaxf(qs * dk, FLT_MIN) : 1.0f;
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < 64; x += 2) mx4[(x >> 1) & 3] = max3(mx4[(x >> 1) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                float mx = max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
                mx *= f;                                                         // f > 0
                if (pair_any(mx > fminf(m, R - ev) + (float)PF_LAZY, bar)) {
                    X.red[part][row] = mx;
                    if (lane == 0) X.ev[warp] = ev;
                    asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
                    // every row of the warp moves when one asks: moved alone, the others ask more often (3 to 6 % of a call)
                    const float other = X.red[part ^ 1][row], mn = fmaxf(m, fmaxf(mx, other));
                    const float fm = m == -INFINITY ? 0.0f : ex2(m - mn);
                    R = fmaxf(R, fmaxf(mx + ev, other + X.ev[warp ^ 4]));
                    const float En = mn == -INFINITY ? E : ceilf(R - mn);        // no key yet: as it was
                    if (j > 0) {
                        wait_s(&X.o_done, (it - 1) & 1);
                        tc_fence_after();
                        const float fo = m == -INFINITY ? 0.0f : ex2((m - mn) + (E - En));
                        uint32_t o[32];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_ld32<0>(tl + 128 * part + 32 * c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fo);
                            tmem_st32<0>(tl + 128 * part + 32 * c, o);
                        }
                    }
                    l *= fm;
                    m = mn;
                    E = En;
                }
                // The sum takes what the weights are made of.  A V scale so small (or 0) that the weights vanish beside the
                // row's others would take the sum with it: it is made first then.
                const float ref = m == -INFINITY ? 0.0f : m, c0 = ev - E + (float)PF_SHIFT;
                if (c0 < -28.0f) {
#pragma unroll
                    for (int x = 0; x < 64; ++x) l += ex2(fmaf(__uint_as_float(s[x]), f, -ref));
                }
                const uint64_t f2 = pack_f2(f, f), b2 = pack_f2(c0 - ref, c0 - ref);
                uint64_t sum[2] = {0, 0};
                uint32_t t[48];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        uint32_t h[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int at = 32 * c + 4 * x + 2 * y;
                            float w0, w1;
                            unpack_f2(fma_f2(pack_f2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), f2, b2), w0, w1);
                            w0 = ex2(w0);
                            w1 = ex2(w1);
                            sum[y] = add_f2(sum[y], pack_f2(w0, w1));
                            h[y] = h2_as_u32(__floats2half2_rn(w0, w1));
                        }
                        split_weights(h[0], h[1], t[24 * c + x], t[24 * c + 8 + x], t[24 * c + 16 + x]);
                    }
                }
                if (c0 >= -28.0f) {
                    float a0, a1;
                    unpack_f2(add_f2(sum[0], sum[1]), a0, a1);
                    l = fmaf(a0 + a1, ex2(-c0), l);
                }
                if (j > 0) {                             // the weights before have been used
                    wait_s(&X.o_done, (it - 1) & 1);
                    tc_fence_after();
                }
                tmem_st32<0>(pcol, t);
                tmem_st16<32>(pcol + 32, t);
                // V codes that belong to no token (past the sequence's end, or of a page that is not there) may be
                // NaN: they become zeros before the product
                if (!there || key0 + PFB_KEYS > kv_end) {
                    const int vs = it % C::V_SLOTS;
                    wait_s(&X.v_full[vs], (it / C::V_SLOTS) & 1);
                    uint8_t *v = sm + C::RING + (C::K_SLOTS + vs) * PF_SLOT_BYTES + tid * 64;        // dim tid of the first tile
                    const int n = there ? kv_end - key0 : 0;
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        const int have = n - 16 * c;
                        if (have >= 16) continue;
                        uint4 *p = reinterpret_cast<uint4 *>(v + (c >> 2) * BT_K_BYTES + (((c & 3) ^ ((tid >> 1) & 3)) << 4));
                        uint4 w = *p;
                        uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int k = have - 4 * y;
                            b[y] = k <= 0 ? 0u : (k >= 4 ? b[y] : b[y] & ((1u << (8 * k)) - 1u));
                        }
                        *p = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                    fence_async_shared();
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&X.p_full);
            }
            // ---- the unit's result ----
            wait_s(&X.o_done, (it - 1) & 1);
            tc_fence_after();
            X.red[part][row] = l;
            asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
            l = X.red[0][row] + X.red[1][row];
            const bool cut = u.slot >= 0;
            const float unit_o = E == PF_NO_E ? 0.0f : exp2f(E - (float)PF_SHIFT);
            const float fo = cut ? unit_o : (l == 0.0f ? 0.0f : unit_o / l);   // NaN stays NaN
            const int tok = r / A.G;
            const int64_t at = r < n_rows ? ((int64_t)(u.row_start + tok) * A.n_q_heads + u.head * A.G + (r - tok * A.G)) * D : -1;
            float *ws = A.ws + (int64_t)u.slot * PFB_SLOT;
            if (cut && part == 0) {
                ws[PFB_ROWS * D + row] = m;
                ws[PFB_ROWS * (D + 1) + row] = l;
            }
            // Through the query's shared memory (its products are complete), so that a warp stores 512 bytes of one row at
            // a time: a row's 16-byte chunks are XORed with the row, which keeps both sides free of bank conflicts.
            auto put = [&](int chunk, const uint4 &v) { *reinterpret_cast<uint4 *>(sm + row * 512 + ((chunk ^ (row & 7)) << 4)) = v; };
            auto rows_out = [&](auto store) {            // the pair's 32 rows, 16 a warp; lane = chunk
                asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
#pragma unroll 4
                for (int y = 16 * part; y < 16 * part + 16; ++y) {
                    const int rr = 32 * (warp & 3) + y;
                    const int64_t to = __shfl_sync(0xffffffffu, at, y);
                    const uint4 v = *reinterpret_cast<const uint4 *>(sm + rr * 512 + ((lane ^ (rr & 7)) << 4));
                    if (to >= 0) store(rr, to, v);
                }
                asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
            };
            if (cut || A.out_f32) {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {            // 64 columns of each half a round
                    uint32_t o[64];
                    tmem_ld32<0>(tl + 128 * part + 64 * h, o);
                    tmem_ld32<32>(tl + 128 * part + 64 * h + 32, o);
                    tc_wait_ld();
#pragma unroll
                    for (int x = 0; x < 64; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fo);
#pragma unroll
                    for (int x = 0; x < 16; ++x) put(16 * part + x, make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
                    rows_out([&](int rr, int64_t to, const uint4 &v) {
                        float *dst = (cut ? ws + rr * D : A.out_f32 + to) + 128 * (lane >> 4) + 64 * h + 4 * (lane & 15);
                        *reinterpret_cast<uint4 *>(dst) = v;
                    });
                }
            }
            if (!cut) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tmem_ld32<0>(tl + 128 * part + 32 * c, o);
                    tc_wait_ld();
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * x]) * fo, __uint_as_float(o[2 * x + 1]) * fo);
                        pk[x] = *reinterpret_cast<const uint32_t *>(&b);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) put(16 * part + 4 * c + x, make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]));
                }
                rows_out([&](int, int64_t to, const uint4 &v) { *reinterpret_cast<uint4 *>(A.out_bf16 + to + 8 * lane) = v; });
            }
            asm volatile("bar.sync 5, %0;" ::"n"(PF_SOFT * 32) : "memory");      // the next query goes where the rows were
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == PF_SOFT) tmem_dealloc(tmem, 512);
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
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
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

template <typename T, int TERMS> cudaError_t launch_prefill_typed(const PfbArgs &a, cudaStream_t s) {
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            cudaFuncAttributes fa;
            cudaError_t e = cudaFuncGetAttributes(&fa, block_prefill_kernel<T, TERMS>);
            if (e != cudaSuccess) return e;
            if (fa.numRegs != PF_REGS) return cudaErrorInvalidConfiguration;    // setmaxnreg.inc would wait for good
            e = cudaFuncSetAttribute(block_prefill_kernel<T, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, PfCfg<TERMS>::SMEM);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    return launch_ex(block_prefill_kernel<T, TERMS>, dim3((unsigned)a.n_ctas), dim3(PF_THREADS), PfCfg<TERMS>::SMEM, s, false, a);
}

}  // namespace

cudaError_t launch_block_prefill(const uint8_t *pool, const PoolGeom &geo, int layer, const void *q, int q_dtype,
                                 int64_t q_stride, const int32_t *page_table, int max_pages, const int32_t *plan,
                                 const kvq_prefill_info &info, float *ws, int32_t *status, uint16_t *out_bf16,
                                 float *out_f32, cudaStream_t s) {
    const PfbArgs a{pool, geo, layer, q, q_stride, page_table, max_pages, plan, info.n_units, info.n_seq, info.n_rows,
                    info.n_merges, info.n_slots, info.n_ctas, info.group, info.group * info.n_kv_heads, ws, status,
                    out_bf16, out_f32};
    cudaError_t e = q_dtype == KVQ_BF16  ? launch_prefill_typed<__nv_bfloat16, 2>(a, s)
                    : q_dtype == KVQ_F16 ? launch_prefill_typed<__half, 3>(a, s)
                                         : launch_prefill_typed<float, 3>(a, s);
    if (e != cudaSuccess || info.n_merges == 0) return e;
    return launch_ex(block_prefill_merge_kernel, dim3((unsigned)info.n_merges * 16), dim3(256), 0, s, false, a);
}

}  // namespace kvq
