// kv_append_rope: new K and V rows of a ragged batch go into the paged cache with
// the position rotation applied on the way, and the query rows are rotated in the
// same launch.
//
// Rotation of a pair (a, b) with the table's c, s of its angle at the row's
// position: (rn(rn(a c) - rn(b s)), rn(rn(b c) + rn(a s))), every operation a
// single fp32 rounding (explicit intrinsics, no contraction), so the rotated row,
// and with it the codes, are bit-exact functions of the input and the table.
#include <cfloat>
#include <type_traits>

#include "kvq_append_dev.cuh"
#include "kvq_block.cuh"

namespace kvq {
namespace {

// Lane l's elements 8l .. 8l+7 of one row of 256.
template <typename T> __device__ __forceinline__ void load_row8(const T *row, int lane, float (&x)[8]);
template <> __device__ __forceinline__ void load_row8<float>(const float *row, int lane, float (&x)[8]) {
    load8(row + lane * 8, x);
}
template <> __device__ __forceinline__ void load_row8<__nv_bfloat16>(const __nv_bfloat16 *row, int lane, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row) + lane);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <> __device__ __forceinline__ void load_row8<__half>(const __half *row, int lane, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row) + lane);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) { return h2_as_u32(__floats2half2_rn(a, b)); }

template <typename T> __device__ __forceinline__ void store_row8(T *row, int lane, const float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        float4 *o = reinterpret_cast<float4 *>(row) + 2 * lane;
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        reinterpret_cast<uint4 *>(row)[lane] = make_uint4(pack2(x[0], x[1], T{}), pack2(x[2], x[3], T{}),
                                                          pack2(x[4], x[5], T{}), pack2(x[6], x[7], T{}));
    }
}

// A position's cosines and sines as the lane needs them: of its four (interleaved)
// or eight pairs, the sine negated where it is subtracted (a c - b s and
// a c + b (-s) are the same roundings).  rot_dim is a multiple of 16, so a split
// pair's partner is the same element of another lane, rot_dim / 16 lanes away.
struct Angles {
    float c[8], s[8];
    __device__ __forceinline__ void load(const RopeArgs &R, int pos, int lane) {
        if (lane * 8 >= R.rot_dim) return;
        const int half = R.rot_dim >> 1, hl = half >> 3;
        const float *cs = R.cos_sin + (int64_t)pos * R.rot_dim;
        if (R.interleaved) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(cs) + lane), b = __ldg(reinterpret_cast<const float4 *>(cs + half) + lane);
            c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
            s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
        } else {
            const int at = (lane >= hl ? lane - hl : lane) * 8;
            load8(cs + at, c);
            load8(cs + half + at, s);
            if (lane < hl)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
    }
};

// The warp rotates one row.
__device__ __forceinline__ void rope_row(float (&x)[8], const RopeArgs &R, const Angles &a, int lane) {
    if (R.interleaved) {
        if (lane * 8 < R.rot_dim)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(u, a.c[i]), __fmul_rn(v, a.s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(v, a.c[i]), __fmul_rn(u, a.s[i]));
            }
    } else {
        const int hl = R.rot_dim >> 4;
        const bool in = lane < 2 * hl;
        const int src = in ? (lane >= hl ? lane - hl : lane + hl) : lane;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], src);
        if (in)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], a.c[i]), __fmul_rn(o[i], a.s[i]));
    }
}

// The last block of a launch looks at row_start as a whole: no other block sees
// more of it than its own rows need.
__device__ __forceinline__ void check_row_start(const RopeArgs &R) {
    bool bad = false;
    for (int s = threadIdx.x; s <= R.n_seq; s += blockDim.x) {
        const int at = __ldg(R.row_start + s);
        bad |= at < (s > 0 ? __ldg(R.row_start + s - 1) : 0) || at > R.n_rows;
    }
    if (bad) status_or(R.status, KVQ_STATUS_BAD_PLAN);
}

// Sequence and position of a row (by the whole warp).  False outside all
// sequences' rows, and with a status bit where row_start or the position is bad.
__device__ __forceinline__ bool row_place(const RopeArgs &R, int64_t row, int lane, int &seq, int &pos) {
    if (row >= __ldg(R.row_start + R.n_seq)) return false;
    seq = warp_find_last(R.n_seq, row, lane, [&](int s) { return (int64_t)__ldg(R.row_start + s); });
    if (seq < 0) return false;
    if (row >= __ldg(R.row_start + seq + 1)) {
        if (lane == 0) status_or(R.status, KVQ_STATUS_BAD_PLAN);
        return false;
    }
    const int64_t p = (int64_t)__ldg(R.pos0 + seq) + (row - __ldg(R.row_start + seq));
    if (p < 0 || p >= (int64_t)R.max_pages * PAGE || (R.rot_dim && p >= R.n_pos)) {
        if (lane == 0) status_or(R.status, KVQ_STATUS_BAD_SLOT);
        return false;
    }
    pos = (int)p;
    return true;
}

// One query row of one head: rotate, rotate once more by H/16 where the format
// keeps K that way, store.
template <bool FWHT, typename T, typename TQ>
__device__ __forceinline__ void rope_query(const RopeArgs &R, int64_t item, int lane) {
    const int64_t row = item / R.n_q_heads;
    const int head = (int)(item - row * R.n_q_heads);
    if (row >= R.n_rows) return;
    float x[8];
    load_row8<T>(static_cast<const T *>(R.q) + row * R.q_stride + head * D, lane, x);
    int seq, pos;
    if (!row_place(R, row, lane, seq, pos)) return;
    if (R.rot_dim) {
        Angles a;
        a.load(R, pos, lane);
        rope_row(x, R, a, lane);
    }
    if (FWHT) fwht256_lane(x, lane);
    store_row8<TQ>(static_cast<TQ *>(R.q_out) + (row * R.n_q_heads + head) * D, lane, x);
}

// Formats whose scales are a token's own: one warp per (row, KV head), then one
// per (row, query head).
template <int FMT, typename T>
__global__ void __launch_bounds__(128) rope_append_kernel(uint8_t *pool, PoolGeom geo, RopeArgs R, unsigned kv_blocks) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == gridDim.x - 1) return check_row_start(R);
    if (blockIdx.x >= kv_blocks) {
        rope_query<Fmt<FMT>::KROT, T, float>(R, (int64_t)(blockIdx.x - kv_blocks) * 4 + (threadIdx.x >> 5), lane);
        return;
    }
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t row = item / geo.n_kv_heads;
    const int head = (int)(item - row * geo.n_kv_heads);
    if (row >= R.n_rows) return;
    float xk[8], xv[8];
    load_row8<T>(static_cast<const T *>(R.k) + row * R.k_stride + head * D, lane, xk);
    load_row8<T>(static_cast<const T *>(R.v) + row * R.v_stride + head * D, lane, xv);
    int seq, pos;
    if (!row_place(R, row, lane, seq, pos)) return;
    const int slot = __ldg(R.page_table + (int64_t)seq * R.max_pages + (pos >> 8));
    uint8_t *tile = token_tile<FMT>(pool, geo, R.layer, slot, head, pos, R.status, lane);
    if (!tile) return;
    if (R.rot_dim) {
        Angles a;
        a.load(R, pos, lane);
        rope_row(xk, R, a, lane);
    }
    TokenCodes t;
    quant_token<FMT>(xk, xv, lane, t);
    store_token<FMT>(t, lane, pos & 7, tile);
}

// ---- fp8b ------------------------------------------------------------------
constexpr int BA_WARPS = 16, BA_THREADS = BA_WARPS * 32;
constexpr int BA_ROWS = 4;             // rows of a warp, all loaded before the first is used
constexpr int BA_MANY = 8;             // query items of a warp where there are many (16-bit types: fp32 ones would be spilled)
constexpr int BA_DIRECT = 4;           // tokens of a tile up to which their V codes are stored byte by byte
static_assert(BA_WARPS * BA_ROWS == BT && BA_ROWS == 4, "a CTA holds a tile's rows, a warp the tokens of one word of V codes");

// Which eight dims of a row a lane holds: a .. a + 3 and b .. b + 3.  With split
// pairs the lanes of the rotated part hold both halves of their pairs, so nothing
// moves between lanes; everywhere else the eight are adjacent.
struct Dims {
    int a, b;
    bool split;                        // of the warp: not all lanes' dims are adjacent
    bool turns;                        // this lane's dims are rotated
    __device__ __forceinline__ Dims(int rot_dim, int interleaved, int lane) {
        const int half = rot_dim >> 1;
        split = rot_dim > 0 && !interleaved;
        turns = split ? lane < (half >> 2) : lane * 8 < rot_dim;
        a = split ? (turns ? 4 * lane : rot_dim + 8 * (lane - (half >> 2))) : 8 * lane;
        b = split && turns ? half + 4 * lane : a + 4;
    }
};

__device__ __forceinline__ void unpack4(const uint2 &u, float *x, __nv_bfloat16) {
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack4(const uint2 &u, float *x, __half) {
    const float2 p = __half22float2(u32_as_h2(u.x)), q = __half22float2(u32_as_h2(u.y));
    x[0] = p.x;
    x[1] = p.y;
    x[2] = q.x;
    x[3] = q.y;
}

// A row's eight values as they are in memory.
template <typename T> struct Raw {
    uint2 a, b;
    __device__ __forceinline__ void load(const T *row, const Dims &m) {
        if (m.split) {
            a = __ldg(reinterpret_cast<const uint2 *>(row + m.a));
            b = __ldg(reinterpret_cast<const uint2 *>(row + m.b));
        } else {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row + m.a));
            a = make_uint2(u.x, u.y);
            b = make_uint2(u.z, u.w);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        unpack4(a, x, T{});
        unpack4(b, x + 4, T{});
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *row, const Dims &m) {
        a = __ldg(reinterpret_cast<const float4 *>(row + m.a));
        b = __ldg(reinterpret_cast<const float4 *>(row + m.b));
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

template <typename TQ> __device__ __forceinline__ void store_dims(TQ *row, const Dims &m, const float (&x)[8]) {
    if constexpr (sizeof(TQ) == 4) {
        *reinterpret_cast<float4 *>(row + m.a) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(row + m.b) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        const uint2 u = make_uint2(pack2(x[0], x[1], TQ{}), pack2(x[2], x[3], TQ{})), v = make_uint2(pack2(x[4], x[5], TQ{}), pack2(x[6], x[7], TQ{}));
        if (m.split) {
            *reinterpret_cast<uint2 *>(row + m.a) = u;
            *reinterpret_cast<uint2 *>(row + m.b) = v;
        } else {
            *reinterpret_cast<uint4 *>(row + m.a) = make_uint4(u.x, u.y, v.x, v.y);
        }
    }
}

// Two fp32 values in one 64-bit register, one instruction for both, each result
// rounded once.
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void un2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The sums of two products each, added one by one: an add.rn.f32x2 of two
// mul.rn.f32x2 came out fused, rounded once (the last bit of q differed).
__device__ __forceinline__ void sum2(uint64_t a, uint64_t b, float &x, float &y) {
    float a0, a1, b0, b1;
    un2(a, a0, a1);
    un2(b, b0, b1);
    x = __fadd_rn(a0, b0);
    y = __fadd_rn(a1, b1);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The cosines and sines of a lane's four pairs at one position.
struct Turn {
    float4 c, s;
    __device__ __forceinline__ void load(const RopeArgs &R, int pos, int lane, const Dims &m) {
        if (!m.turns) return;
        const float *cs = R.cos_sin + (int64_t)pos * R.rot_dim + 4 * lane;
        c = __ldg(reinterpret_cast<const float4 *>(cs));
        s = __ldg(reinterpret_cast<const float4 *>(cs + (R.rot_dim >> 1)));
    }
    // a c - b s as a c + b (-s): the same roundings
    __device__ __forceinline__ void apply(float (&x)[8], const Dims &m) const {
        if (!m.turns) return;
        const uint64_t c0 = f2(c.x, c.y), c1 = f2(c.z, c.w), s0 = f2(s.x, s.y), s1 = f2(s.z, s.w), n0 = f2(-s.x, -s.y), n1 = f2(-s.z, -s.w);
        if (m.split) {
            const uint64_t a0 = f2(x[0], x[1]), a1 = f2(x[2], x[3]), b0 = f2(x[4], x[5]), b1 = f2(x[6], x[7]);
            sum2(mul2(a0, c0), mul2(b0, n0), x[0], x[1]);
            sum2(mul2(a1, c1), mul2(b1, n1), x[2], x[3]);
            sum2(mul2(b0, c0), mul2(a0, s0), x[4], x[5]);
            sum2(mul2(b1, c1), mul2(a1, s1), x[6], x[7]);
        } else {
            const uint64_t a0 = f2(x[0], x[2]), a1 = f2(x[4], x[6]), b0 = f2(x[1], x[3]), b1 = f2(x[5], x[7]);
            sum2(mul2(a0, c0), mul2(b0, n0), x[0], x[2]);
            sum2(mul2(a1, c1), mul2(b1, n1), x[4], x[6]);
            sum2(mul2(b0, c0), mul2(a0, s0), x[1], x[3]);
            sum2(mul2(b1, c1), mul2(a1, s1), x[5], x[7]);
        }
    }
};

// row_start and pos0 of a batch of fewer than 32 sequences, an entry a lane: one
// load where a search and what it finds are two or three.
struct Batch {
    int start, pos0, n_seq;
    __device__ __forceinline__ Batch(const RopeArgs &R, bool few, int lane) : start(0), pos0(0), n_seq(R.n_seq) {
        if (few && lane <= R.n_seq) start = __ldg(R.row_start + lane);
        if (few && lane < R.n_seq) pos0 = __ldg(R.pos0 + lane);
    }
    // the last sequence that starts at or below row, -1 if none (by the whole warp)
    __device__ __forceinline__ int last_below(int row) const {
        return 31 - __clz(__ballot_sync(0xffffffffu, (int)(threadIdx.x & 31) < n_seq && start <= row));
    }
    // the last sequence whose tile items start at or below item
    __device__ __forceinline__ int last_tiles_below(int item) const {
        const int lane = threadIdx.x & 31;
        return 31 - __clz(__ballot_sync(0xffffffffu, lane < n_seq && (start >> 6) + 2 * lane <= item));
    }
};

// Query rows: a warp takes n <= N consecutive (row, head) items, mostly of one or
// two rows, whose angles it loads once.
template <typename T, typename TQ, int N> __device__ __forceinline__ void rope_queries(const RopeArgs &R, uint32_t item0, int n, int lane) {
    const uint32_t n_items = (uint32_t)(R.n_rows * R.n_q_heads), n_q = (uint32_t)R.n_q_heads;   // at most 2^31
    if (item0 >= n_items) return;
    n = (int)min((uint32_t)n, n_items - item0);
    const uint32_t row0 = item0 / n_q, head0 = item0 - row0 * n_q;
    const Dims m(R.rot_dim, R.interleaved, lane);
    Raw<T> raw[N];
    {
        uint32_t h = head0;
        const T *src = static_cast<const T *>(R.q) + (int64_t)row0 * R.q_stride;
#pragma unroll
        for (int y = 0; y < N; ++y) {
            if (y < n) raw[y].load(src + h * D, m);
            if (++h == n_q) h = 0, src += R.q_stride;
        }
    }
    // positions: lane y < n has item y's, -1 where it has none
    int seq = warp_find_last(R.n_seq, row0, lane, [&](int s) { return (int64_t)__ldg(R.row_start + s); });   // -1: before all of them
    int pos = -1;
    if (lane < n) {
        const int row = (int)((item0 + lane) / n_q);
        if (row < __ldg(R.row_start + R.n_seq)) {
            while (seq < R.n_seq && row >= __ldg(R.row_start + seq + 1)) ++seq;
            if (seq >= R.n_seq || (seq >= 0 && row < __ldg(R.row_start + seq))) {
                status_or(R.status, KVQ_STATUS_BAD_PLAN);
            } else if (seq >= 0) {
                const int64_t p = (int64_t)__ldg(R.pos0 + seq) + (row - __ldg(R.row_start + seq));
                if (p < 0 || p >= (int64_t)R.max_pages * PAGE || (R.rot_dim && p >= R.n_pos)) status_or(R.status, KVQ_STATUS_BAD_SLOT);
                else pos = (int)p;
            }
        }
    }
    __syncwarp();
    Turn turn;
    int held = -1;
    TQ *dst = static_cast<TQ *>(R.q_out) + (int64_t)item0 * D;
#pragma unroll
    for (int y = 0; y < N; ++y) {
        const int p = __shfl_sync(0xffffffffu, pos, y);
        if (p < 0) continue;
        float x[8];
        raw[y].get(x);
        if (R.rot_dim) {
            if (p != held) turn.load(R, p, lane, m);
            held = p;
            turn.apply(x, m);
        }
        store_dims<TQ>(dst + y * D, m, x);
    }
}

// 16 codes times the power of two f (0 clears them); bytes whose token is not
// below keep (bit i of keep: byte i is an old token's) stay as they are.
__device__ __forceinline__ uint4 rescale16(uint4 u, float f, uint32_t keep) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 v = __half22float2(u32_as_h2(e4m3x2_to_h2((w[i] >> (16 * h)) & 0xFFFFu)));
            r |= f32x2_to_e4m3x2(__fmul_rn(v.x, f), __fmul_rn(v.y, f)) << (16 * h);
        }
        uint32_t m = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) m |= (keep >> (4 * i + b) & 1u) ? 0xFFu << (8 * b) : 0u;
        w[i] = (r & m) | (w[i] & ~m);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per (sequence, tile it appends to, KV head, K or V); the CTAs after those
// take the query rows.  Item i belongs to the sequence s whose range
// [row_start[s] / 64 + 2 s, row_start[s+1] / 64 + 2 (s+1)) holds it: n rows touch
// at most n / 64 + 2 tiles, so the ranges are found from row_start alone and a
// surplus item has no rows.  Where the rows are fewer than those items (by_row:
// decoding batches), item i is row i, and a tile is taken by its first row.
// Warp w holds the rows of tokens 4 w .. 4 w + 3 in
// registers between the tile's scale and its codes, so each row is read once.
// Bound by HBM for long prompts (K, V and Q once in, codes and Q once out) and by
// the chain of loads item -> rows and page slot -> scale for a few tokens.
template <typename T, typename TQ>
__global__ void __launch_bounds__(BA_THREADS, 2) block_append_kernel(uint8_t *pool, PoolGeom geo, RopeArgs R,
                                                                     unsigned kv_blocks, int by_row, int q_rows) {
    __shared__ float s_max[BA_WARPS];
    __shared__ __align__(16) uint8_t s_v[32 * 528];     // V codes: 512 bytes a dim group, 16 of padding
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == gridDim.x - 1) return check_row_start(R);
    if (blockIdx.x >= kv_blocks) {
        const uint32_t item0 = ((blockIdx.x - kv_blocks) * BA_WARPS + warp) * q_rows;
        if (q_rows <= BA_ROWS) rope_queries<T, TQ, BA_ROWS>(R, item0, q_rows, lane);
        else if constexpr (sizeof(T) == 2) rope_queries<T, TQ, BA_MANY>(R, item0, q_rows, lane);
        return;
    }
    const bool is_v = blockIdx.x & 1;
    const int item = (blockIdx.x >> 1) / (unsigned)geo.n_kv_heads, head = (int)(blockIdx.x >> 1) - item * geo.n_kv_heads;
    const bool few = R.n_seq < 32;
    const Batch all(R, few, lane);
    const int seq = few      ? (by_row ? all.last_below(item) : all.last_tiles_below(item))
                    : by_row ? warp_find_last(R.n_seq, item, lane, [&](int s) { return (int64_t)__ldg(R.row_start + s); })
                             : warp_find_last(R.n_seq, item, lane, [&](int s) { return (int64_t)(__ldg(R.row_start + s) >> 6) + 2 * (int64_t)s; });
    if (seq < 0) return;                                 // before the first sequence's rows
    const int row0 = few ? __shfl_sync(0xffffffffu, all.start, seq) : __ldg(R.row_start + seq);
    const int row1 = few ? __shfl_sync(0xffffffffu, all.start, seq + 1) : __ldg(R.row_start + seq + 1);
    const int p0 = few ? __shfl_sync(0xffffffffu, all.pos0, seq) : __ldg(R.pos0 + seq);
    if (row0 < 0 || row1 < row0 || row1 > R.n_rows) {
        if (threadIdx.x == 0) status_or(R.status, KVQ_STATUS_BAD_PLAN);
        return;
    }
    if (by_row ? item >= row1 : row1 == row0) return;    // padding, or no rows
    int64_t end = (int64_t)p0 + (row1 - row0);
    const int64_t room = R.rot_dim ? min((int64_t)R.max_pages * PAGE, (int64_t)R.n_pos) : (int64_t)R.max_pages * PAGE;
    if (p0 < 0 || end > room) {
        if (threadIdx.x == 0) status_or(R.status, KVQ_STATUS_BAD_SLOT);
        if (p0 < 0) return;
        end = min(end, room);
    }
    const int64_t tile_i = by_row ? ((int64_t)p0 + (item - row0)) >> 6
                                  : (int64_t)(p0 >> 6) + (item - ((int64_t)(row0 >> 6) + 2 * (int64_t)seq));
    const int64_t first = tile_i * BT;
    if (first >= end) return;
    if (by_row && item > row0 && (int64_t)p0 + (item - row0) != first) return;   // not the tile's first row
    const int slot = __ldg(R.page_table + (int64_t)seq * R.max_pages + (first >> 8));
    const int t0 = first >= p0 ? 0 : (int)(p0 - first), t1 = (int)min((int64_t)BT, end - first);
    if (t0 >= t1) return;                                // the sequence starts past its room
    // the rows; the tile's token 0 would be row rbase (it may lie before row0)
    const int64_t rbase = row0 + (first - p0);
    const int tok0 = BA_ROWS * warp;
    const Dims m(is_v ? 0 : R.rot_dim, R.interleaved, lane);
    Raw<T> raw[BA_ROWS];
    Turn turn[BA_ROWS];
    float x[BA_ROWS][8];
    const bool turned = !is_v && R.rot_dim;
    const bool any = tok0 < t1 && tok0 + BA_ROWS > t0;   // the warp has rows; a token of its four that is not the call's stands for
                                                         // one that is, so that nothing below has to ask
    if (any) {
        const T *src = (is_v ? static_cast<const T *>(R.v) : static_cast<const T *>(R.k)) + head * D;
        const int64_t stride = is_v ? R.v_stride : R.k_stride;
#pragma unroll
        for (int i = 0; i < BA_ROWS; ++i) {              // the angles with the values: asked for one by one they cost a wait each
            const int tok = min(max(tok0 + i, t0), t1 - 1);
            raw[i].load(src + (rbase + tok) * stride, m);
            if (turned) turn[i].load(R, (int)first + tok, lane, m);
        }
    }
    if (slot < 0 || slot >= geo.n_pages) {
        if (threadIdx.x == 0) status_or(R.status, KVQ_STATUS_BAD_SLOT);
        return;
    }
    uint8_t *page = pool + R.layer * geo.layer_stride + (int64_t)slot * geo.slot_stride + (int64_t)head * geo.page_bytes;
    uint8_t *codes = page + (tile_i & 3) * BT_BYTES + (is_v ? BT_K_BYTES : 0);
    float *scale = reinterpret_cast<float *>(page + B_SCALES_OFF) + 2 * (tile_i & 3) + is_v;
    const float d0 = t0 > 0 ? *scale : 0.0f;

    float amax = 0.0f;
    uint64_t odd2 = 0;                                   // NaN once a value is not finite
    if (any) {
#pragma unroll
        for (int i = 0; i < BA_ROWS; ++i) {
            raw[i].get(x[i]);
            if (turned) turn[i].apply(x[i], m);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                asm("max.f32 %0, %1, %2, %3;" : "=f"(amax) : "f"(amax), "f"(fabsf(x[i][e])), "f"(fabsf(x[i][e + 1])));
                odd2 = fma2(f2(x[i][e], x[i][e + 1]), 0, odd2);
            }
        }
    }
    float odd, odd1;
    un2(odd2, odd, odd1);
    if (__any_sync(0xffffffffu, odd + odd1 != 0.0f)) {   // NaN is kept out of the cache, infinity saturates
        if (lane == 0) status_or(R.status, KVQ_STATUS_NONFINITE);
        amax = 0.0f;
#pragma unroll
        for (int i = 0; i < BA_ROWS; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (!(fabsf(x[i][e]) <= FLT_MAX)) x[i][e] = x[i][e] != x[i][e] ? 0.0f : copysignf(FLT_MAX, x[i][e]);
                    amax = fmaxf(amax, fabsf(x[i][e]));
                }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));      // not negative: the bits order as the values
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();                                     // also: every thread has read the old scale
#pragma unroll
    for (int w = 0; w < BA_WARPS; ++w) amax = fmaxf(amax, s_max[w]);
    const float d = fmaxf(d0, block_scale(amax));
    if (threadIdx.x == 0) *scale = d;
    // 1 / d of a power of two with exponent within -120 .. 118: x * inv is x / d, and d0 / d is exact too
    const float inv = d > 0.0f ? __uint_as_float((254u << 23) - __float_as_uint(d)) : 0.0f;
    const float f = d > 0.0f ? d0 * inv : 1.0f;
    const bool grown = t0 > 0 && f != 1.0f;
    const bool staged = is_v && (grown || t1 - t0 > BA_DIRECT);
    if (!is_v) {
        if (grown)
            for (int c = threadIdx.x; c < t0 * 16; c += BA_THREADS) {
                uint4 *p = reinterpret_cast<uint4 *>(codes + block_k_off(c >> 4, (c & 15) * 16));
                *p = rescale16(*p, f, 0xFFFFu);
            }
    } else if (staged && (t0 > 0 || t1 < BT)) {          // the tile's bytes, rescaled, come to shared memory first
        for (int c = threadIdx.x; c < 1024; c += BA_THREADS) {
            uint4 u = reinterpret_cast<const uint4 *>(codes)[c];
            const int row = c >> 2, tok = ((c & 3) ^ ((row >> 1) & 3)) * 16;
            if (grown && t0 > tok) u = rescale16(u, f, t0 - tok >= 16 ? 0xFFFFu : (1u << (t0 - tok)) - 1u);
            *reinterpret_cast<uint4 *>(s_v + (c >> 5) * 528 + (c & 31) * 16) = u;
        }
        __syncthreads();
    }
    const bool whole = tok0 >= t0 && tok0 + BA_ROWS <= t1;
    uint32_t c[BA_ROWS][4];                              // two codes a word
    const uint64_t inv2 = f2(inv, inv);
#pragma unroll
    for (int i = 0; i < BA_ROWS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            un2(mul2(f2(x[i][2 * j], x[i][2 * j + 1]), inv2), lo, hi);
            c[i][j] = f32x2_to_e4m3x2(lo, hi);
        }
    if (!(d > 0.0f))                                     // all values are 0, some of them perhaps -0
#pragma unroll
        for (int i = 0; i < BA_ROWS; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0;
    if (staged && whole) {                               // the warp's tokens of a dim are adjacent bytes
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t sel = e & 1 ? 0x0051u : 0x0040u;
            const uint32_t w = __byte_perm(__byte_perm(c[0][e >> 1], c[1][e >> 1], sel), __byte_perm(c[2][e >> 1], c[3][e >> 1], sel), 0x5410);
            *reinterpret_cast<uint32_t *>(s_v + lane * 528 + e * 64 + (((warp >> 2) ^ ((e >> 1) & 3)) << 4) + (warp & 3) * 4) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < BA_ROWS; ++i) {
            const int t = tok0 + i;
            if (t < t0 || t >= t1) continue;
            if (!is_v) {
                *reinterpret_cast<uint32_t *>(codes + block_k_off(t, m.a)) = c[i][0] | c[i][1] << 16;
                *reinterpret_cast<uint32_t *>(codes + block_k_off(t, m.b)) = c[i][2] | c[i][3] << 16;
            } else {
                uint8_t *to = staged ? s_v + lane * 528 : codes + lane * 512;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    to[e * 64 + (((t >> 4) ^ ((e >> 1) & 3)) << 4) + (t & 15)] = (uint8_t)(c[i][e >> 1] >> (8 * (e & 1)));
            }
        }
    }
    if (!staged) return;
    __syncthreads();
    for (int k = threadIdx.x; k < 1024; k += BA_THREADS)
        reinterpret_cast<uint4 *>(codes)[k] = *reinterpret_cast<const uint4 *>(s_v + (k >> 5) * 528 + (k & 31) * 16);
}

template <typename T, typename TQ>
cudaError_t launch_typed(int fmt, uint8_t *pool, const PoolGeom &geo, const RopeArgs &R, cudaStream_t s) {
    const int64_t q_items = R.q ? R.n_rows * R.n_q_heads : 0;
    if (fmt == KVQ_FP8B) {
        const int64_t by_tiles = (R.n_rows >> 6) + 2 * (int64_t)R.n_seq;
        const int by_row = R.n_rows < by_tiles ? 1 : 0;
        const int64_t kv = R.k ? (by_row ? R.n_rows : by_tiles) * geo.n_kv_heads * 2 : 0;
        // a few query rows are spread over as many warps, 2 CTAs of them an SM; more are taken BA_ROWS at a time, for the loads in flight and
        // the angles they share, and very many BA_MANY at a time, for the instructions around them (4 and 8 a warp, 24
        // heads: 2,000 rows 15.6 and 15.7 us, 3,000 rows 22.2 and 21.7, 8,917 rows 60.7 and 55)
        const int64_t warps = (int64_t)device_sms() * 2 * BA_WARPS;
        const int q_rows = q_items <= warps ? 1 : sizeof(T) == 2 && q_items > 12 * warps ? BA_MANY : BA_ROWS;
        const int64_t qb = (q_items + BA_WARPS * q_rows - 1) / (BA_WARPS * q_rows);
        return launch_ex(block_append_kernel<T, TQ>, dim3((unsigned)(kv + qb + 1)), dim3(BA_THREADS), 0, s, false, pool, geo,
                         R, (unsigned)kv, by_row, q_rows);
    }
    if constexpr (std::is_same_v<TQ, float>) {           // the decodes of these formats take fp32 queries
        const int64_t kv = R.k ? (R.n_rows * geo.n_kv_heads + 3) / 4 : 0, qb = (q_items + 3) / 4;
        auto kern = fmt == KVQ_INT8    ? rope_append_kernel<KVQ_INT8, T>
                    : fmt == KVQ_Q4_0  ? rope_append_kernel<KVQ_Q4_0, T>
                    : fmt == KVQ_K8V4  ? rope_append_kernel<KVQ_K8V4, T>
                    : fmt == KVQ_FP8   ? rope_append_kernel<KVQ_FP8, T>
                                       : rope_append_kernel<KVQ_NVFP4, T>;
        return launch_ex(kern, dim3((unsigned)(kv + qb + 1)), dim3(128), 0, s, false, pool, geo, R, (unsigned)kv);
    } else {
        return cudaErrorNotSupported;
    }
}

}  // namespace

cudaError_t launch_rope_append(int fmt, uint8_t *pool, const PoolGeom &geo, const RopeArgs &R, int dtype, int q_dtype,
                               cudaStream_t s) {
    if (dtype == KVQ_F32) return launch_typed<float, float>(fmt, pool, geo, R, s);
    if (dtype == KVQ_BF16)
        return q_dtype == KVQ_F32 ? launch_typed<__nv_bfloat16, float>(fmt, pool, geo, R, s)
                                  : launch_typed<__nv_bfloat16, __nv_bfloat16>(fmt, pool, geo, R, s);
    return q_dtype == KVQ_F32 ? launch_typed<__half, float>(fmt, pool, geo, R, s)
                              : launch_typed<__half, __half>(fmt, pool, geo, R, s);
}

}  // namespace kvq
