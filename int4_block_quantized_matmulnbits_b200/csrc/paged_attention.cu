// paged_attention.cu -- attention of one new token per request over a paged
// key-value cache (mnb_paged_attention).
//
// For request b, query head i of KV head h = i / G and the n = seq_lens[b] rows
// of the cache that the block table names:
//   s_j = scale * q_i . k_j,  lse = log sum_j exp(s_j),  o_i = sum_j exp(s_j - lse) v_j.
// One pass over K and V with the running maximum m and sum l of the softmax:
// on a new maximum, l and the accumulated o are scaled by exp(m_old - m_new).
// Two such (m, l, o) over disjoint keys join the same way, so the cache's
// length may be cut anywhere.
//
// Work split.  The keys of a segment -- a (request, KV head, row tile of query
// heads) -- are cut into tiles of TK keys: first over P groups, then over the S
// CTAs of each group's thread-block cluster, then every W-th tile to each of a
// CTA's W warps.  The parts are joined in that order's reverse: the warps' in
// shared memory, the cluster's through distributed shared memory behind one
// cluster barrier, the groups' (P > 1 only where a few long segments would leave
// most SMs idle) through the workspace, by the group that arrives last, in group
// order, so that no result depends on which group that is.
//
// Each warp owns a ring of tiles in shared memory that it fills with 16-byte
// cp.async (rows behind the length and rows of page ids outside the pool are
// zero-filled and masked, never read) and drains by itself: the main loop has no
// CTA barrier, and a warp waits for its own copies only.
//
// Bound by the cache's bytes where there are many (64 requests of up to 8192 tokens
// in 8 heads of 128: 162 to 166 us in a graph, 6600 GB/s; 173 us as calls from
// Python), by latency where there are few (one request of 390 tokens: 5.9 us).  A
// tile is one warp's alone because its chain of products and exponentials, about
// 0.65 us, is what a warp's rate is made of: more warps hide it, more copies in
// flight do not.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mnb_tune.h"

namespace mnb {
namespace {

constexpr int kMaxSplit = 8;    // CTAs of a cluster
constexpr int kMaxWarps = 12;   // of a CTA
constexpr int kMaxStages = 6;   // of a warp's ring
constexpr int kMaxGroups = 64;  // of a call that has more than one per segment
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    int *counters;      // workspace: a segment's groups that have arrived, zero between calls
    float *partials;    // workspace: the groups' partial results
    int *status;
    int64_t q_bs, q_hs, o_bs, o_hs;                             // elements
    int64_t table_stride, page_stride, slot_stride, head_stride;
    int G, Hkv, D, rows, row_tiles, page, num_pages, cap;       // cap: rows the table has room for
    int one_page;          // a tile's keys are in one page: page % TK == 0
    int split, groups, stages;
    int least;             // fewest tiles that a CTA of a cluster takes
    Div by_page, by_split, by_groups;
    float scale;
};

// Element type, padded head size and whether D fills it, rows of query heads per
// segment.  A tile is 8 KB of K and V (16 KB for heads of 256): 16 keys of 128
// fp16 entries.  Rows are swizzled in shared memory (chunk ^ row % 8), so that
// reads of eight rows' same chunk meet no bank twice.
template <typename T_, int DP_, int ROWS_, bool WHOLE_>
struct Cfg {
    using T = T_;
    static constexpr bool F16 = std::is_same<T, half>::value;
    static constexpr int DP = DP_, ROWS = ROWS_;
    static constexpr bool WHOLE = WHOLE_;                            // D == DP
    static constexpr int TK = (F16 ? 16 : 8) * (DP <= 64 ? 2 : 1);   // keys per tile
    static constexpr int NCH = DP * (int)sizeof(T) / 16;             // 16-byte chunks per row
    static constexpr int ROW_BYTES = DP * (int)sizeof(T);
    static constexpr int TILE_BYTES = TK * ROW_BYTES;
    static __device__ __forceinline__ uint32_t at(int row, int chunk) { return row * ROW_BYTES + (chunk ^ (row & 7)) * 16; }
    static constexpr int kWarpsMost = DP > 128 ? 6 : kMaxWarps;      // on an SM, two stages each in shared memory
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(a)
                 : "memory");
}
// Four fp32 values as two pairs, for the instructions that take two at a time
// (each value rounded as by the scalar instruction).
struct Quad {
    unsigned long long lo, hi;
};
__device__ __forceinline__ Quad lds_quad(uint32_t a) {
    Quad r;
    asm volatile("ld.shared.v2.u64 {%0,%1}, [%2];" : "=l"(r.lo), "=l"(r.hi) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ unsigned long long pair(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1,%2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(unsigned long long p) {
    float2 r;
    asm("mov.b64 {%0,%1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two numbers of 0 or above (or NaN) as sums of two fp16 numbers each, within 2^-21
// of them and 2^-25: the first rounded towards zero, `lo` the rest.  Where the first
// is above 0 so is the rest (at least 2^-24), so that products of both with an
// infinity are that infinity and not 0 times it.
__device__ __forceinline__ uint32_t split2(float x, float y, uint32_t &lo) {
    uint32_t hi;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    const half2 h = u32_as_h2(hi);
    const float2 f = __half22float2(h);
    const half2 least = __hmin2(h, u32_as_h2(0x00010001u));
    lo = h2_as_u32(__hmax2(__floats2half2_rn(x - f.x, y - f.y), least));
    return hi;
}
__device__ __forceinline__ void fma4(float4 &c, float s, float4 v) {
    c.x = fmaf(s, v.x, c.x), c.y = fmaf(s, v.y, c.y), c.z = fmaf(s, v.z, c.z), c.w = fmaf(s, v.w, c.w);
}

// Two neighbouring outputs of one row; c is even and below D (a multiple of 8).
__device__ __forceinline__ void store2(half *p, float a, float b) { *reinterpret_cast<half2 *>(p) = __floats2half2_rn(a, b); }
__device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }

// The transpose of an 8x8 matrix of 16-bit values, one packed pair per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// log sum exp from a maximum in log2 units and a sum relative to it (0: no key; NaN where a score was NaN).
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : m * kLn2 + logf(l); }

// The running softmax of one segment in a warp's registers.  The maximum m is a
// reference, not the exact maximum: it moves, and o and l are rescaled, only
// when a score exceeds it by more than 2^LAZY (in most tiles one vote says that
// none does, and no maximum is taken across lanes).
constexpr float LAZY = 5.0f;

template <typename C, bool F16>
struct Acc;

// fp16: S^T = K Q^T and O^T += V^T P^T as m16n8k16 products: keys, then head
// entries are the 16 rows, up to 8 query heads the 8 columns (the grouped heads
// of one KV head seldom fill more).  P enters the second product as two fp16
// numbers, which keep 21 of fp32's bits, scaled so that the reference maximum is
// at 2^SHIFT: its largest values stay below 2^15, and what is lost of any term is
// below 2^-34 of the largest.  l is summed from the unrounded fp32 values.  Up to
// four query heads stand in the columns twice, and the second four take the rest
// of P: then both parts are one product (32 requests of up to 4096 in 8 heads of
// 80: 42.5 us, 44.0 with two products, 42.0 with P rounded to fp16; 16 heads on a
// KV head of 256, 24 requests of up to 4001, two products: 40.8 us, 37.3 rounded).
template <typename C>
struct Acc<C, true> {
    static constexpr bool TWICE = C::ROWS == 4;
    static constexpr int NT = TWICE ? 1 : C::ROWS / 8, KB = C::TK / 16, KS = C::DP / 16;
    static constexpr float SHIFT = 10.0f;
    static constexpr float kSumScale = 1.0f / 1024.0f;   // 2^-SHIFT
    float o[KS][NT][4];        // entry 16 i + lane / 4 (+ 8), heads 2 (lane % 4) and the next
    float m[NT][2], l[NT][2];
    uint32_t q[KS][NT][2];     // B fragments of the segment's query rows

    // The segment's query rows are at `qs`.
    __device__ __forceinline__ void open(uint32_t qs, int rows) {
        const int lane = threadIdx.x & 31, i = lane >> 3;
        if constexpr (NT == 1) {
            const int r = min(lane & (TWICE ? 3 : 7), rows - 1);
#pragma unroll
            for (int kk = 0; kk < KS; kk += 2)
                ldsm4(qs + C::at(r, kk * 2 + i), q[kk][0][0], q[kk][0][1], q[kk + 1][0][0],
                      q[kk + 1][0][1]);
        } else {
            const int r = min((lane & 7) + (i >> 1) * 8, rows - 1);
#pragma unroll
            for (int kk = 0; kk < KS; kk++)
                ldsm4(qs + C::at(r, kk * 2 + (i & 1)), q[kk][0][0], q[kk][0][1],
                      q[kk][NT - 1][0], q[kk][NT - 1][1]);
        }
#pragma unroll
        for (int t = 0; t < NT; t++) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; k++)
                o[k][t][0] = o[k][t][1] = o[k][t][2] = o[k][t][3] = 0.0f;
        }
    }

    // One tile: K and V in shared memory, `valid` one bit per key.
    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, uint32_t, int, int D, uint32_t valid, float scale2) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        float s[KB][NT][4];
        {
            float h[2][KB][NT][4] = {};   // even and odd steps: two chains of products
            const int kr = (lane & 7) + ((lane >> 3) & 1) * 8, kc = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < KS; kk++) {
                if (!C::WHOLE && kk * 16 >= D)
                    break;
#pragma unroll
                for (int b = 0; b < KB; b++) {
                    uint32_t a0, a1, a2, a3;
                    ldsm4(ks + C::at(b * 16 + kr, kk * 2 + kc), a0, a1, a2, a3);
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        mma16816(h[kk & 1][b][t], a0, a1, a2, a3, q[kk][t][0], q[kk][t][1]);
                }
            }
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        s[b][t][c] = h[0][b][t][c] + h[1][b][t][c];
        }
        bool over = false;
#pragma unroll
        for (int b = 0; b < KB; b++)
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const bool ok = (valid >> (b * 16 + g + (c >> 1) * 8)) & 1;
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    s[b][t][c] = ok ? s[b][t][c] * scale2 : -INFINITY;
                    over |= s[b][t][c] > m[t][c & 1] + LAZY;
                }
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    float mn = m[t][c];
#pragma unroll
                    for (int b = 0; b < KB; b++)
                        mn = fmaxf(mn, fmaxf(s[b][t][c], s[b][t][c + 2]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
                    const float alpha = mn > m[t][c] ? ex2(m[t][c] - mn) : 1.0f;   // 0 after m = -inf
                    m[t][c] = mn;
                    l[t][c] *= alpha;
#pragma unroll
                    for (int k = 0; k < KS; k++)
                        o[k][t][c] *= alpha, o[k][t][c + 2] *= alpha;
                }
        }
        uint32_t p[KB][NT][2], p_lo[KB][NT][2];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const float b0 = m[t][0] == -INFINITY ? 0.0f : m[t][0] - SHIFT;
            const float b1 = m[t][1] == -INFINITY ? 0.0f : m[t][1] - SHIFT;
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float x = ex2(s[b][t][2 * h] - b0), y = ex2(s[b][t][2 * h + 1] - b1);
                    l[t][0] += x, l[t][1] += y;
                    uint32_t lo;
                    const uint32_t hi = split2(x, y, lo);
                    p[b][t][h] = transpose8(TWICE && (lane & 2) ? lo : hi);
                    if constexpr (!TWICE)
                        p_lo[b][t][h] = transpose8(lo);
                }
        }
        const int vr = (lane & 7) + (lane >> 4) * 8, vc = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < KS; k++) {
            if (!C::WHOLE && k * 16 >= D)
                break;
#pragma unroll
            for (int b = 0; b < KB; b++) {
                uint32_t a0, a1, a2, a3;
                ldsm4t(vs + C::at(b * 16 + vr, k * 2 + vc), a0, a1, a2, a3);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    mma16816(o[k][t], a0, a1, a2, a3, p[b][t][0], p[b][t][1]);
                    if constexpr (!TWICE)
                        mma16816(o[k][t], a0, a1, a2, a3, p_lo[b][t][0], p_lo[b][t][1]);
                }
            }
        }
    }

    // Sums over the lanes' keys, and over P's two halves where they have columns of their own.
    __device__ __forceinline__ void finish() {
        if constexpr (TWICE)
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int c = 0; c < 4; c++)
                    o[k][0][c] += __shfl_xor_sync(0xffffffffu, o[k][0][c], 2);
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    l[t][c] += __shfl_xor_sync(0xffffffffu, l[t][c], x);
    }

    // A partial result: rows x D outputs, maxima, sums.
    __device__ __forceinline__ void to_slot(float *sl, int rows, int D) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int r = t * 8 + (lane & 3) * 2 + c;
                if (r < rows) {
#pragma unroll
                    for (int k = 0; k < 2 * KS; k++)
                        if (k * 8 < D)
                            sl[r * D + k * 8 + g] = o[k / 2][t][c + 2 * (k & 1)];
                    if (g == 0) {
                        sl[rows * D + r] = m[t][c];
                        sl[rows * D + rows + r] = l[t][c];
                    }
                }
            }
    }
};

// fp32: every product and sum in fp32 on the CUDA cores, two at a time, eight keys
// at a time.
// Scores: a lane holds key lane % 8 and a quarter of the chunks, two shuffles
// add the quarters.  Output: a lane holds whole columns; a row's probabilities
// come by shuffle.
template <typename C>
struct Acc<C, false> {
    static constexpr int LPR = C::NCH < 32 ? C::NCH : 32;   // lanes per row of V
    static constexpr int PER = C::NCH / LPR;                // chunks a lane holds
    static constexpr int KSPLIT = 32 / LPR;                 // keys taken at a time
    static constexpr float kSumScale = 1.0f;
    static constexpr int QC = C::NCH / 4;                   // chunks of a query row that a lane needs
    static constexpr bool QREG = C::ROWS * QC <= 16;        // they stay in registers
    Quad o[C::ROWS][PER];
    Quad q[QREG ? C::ROWS : 1][QREG ? QC : 1];
    float m[C::ROWS], l[C::ROWS];

    __device__ __forceinline__ void open(uint32_t qs, int rows) {
        const int quarter = (threadIdx.x & 31) >> 3;
        if constexpr (QREG)
#pragma unroll
            for (int r = 0; r < C::ROWS; r++)
#pragma unroll
                for (int c = 0; c < QC; c++)
                    q[r][c] = lds_quad(qs + C::at(min(r, rows - 1), c * 4 + quarter));
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
#pragma unroll
            for (int c = 0; c < PER; c++)
                o[r][c] = {0, 0};
            m[r] = -INFINITY;
            l[r] = 0.0f;
        }
    }

    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, uint32_t qs, int rows, int D, uint32_t valid, float scale2) {
#pragma unroll 1
        for (int j = 0; j < C::TK / 8; j++)
            eight(ks + j * 8 * C::ROW_BYTES, vs + j * 8 * C::ROW_BYTES, qs, rows, D, valid >> (8 * j), scale2);
    }

    __device__ __forceinline__ void eight(uint32_t ks, uint32_t vs, uint32_t qs, int rows, int D, uint32_t valid, float scale2) {
        const int lane = threadIdx.x & 31, key = lane & 7, quarter = lane >> 3;
        float s[C::ROWS];
        unsigned long long s2[C::ROWS] = {};   // even and odd entries
#pragma unroll(QREG ? QC : 4)
        for (int c = 0; c < QC; c++) {
            if (!C::WHOLE && c * 16 >= D)
                break;
            const int ch = c * 4 + quarter;
            Quad k = lds_quad(ks + C::at(key, ch));
            if (!C::WHOLE && ch * 4 >= D)   // columns that nothing has written
                k = {0, 0};
#pragma unroll
            for (int r = 0; r < C::ROWS; r++) {
                const Quad qr = QREG ? q[QREG ? r : 0][QREG ? c : 0] : lds_quad(qs + C::at(min(r, rows - 1), ch));
                s2[r] = fma2(k.hi, qr.hi, fma2(k.lo, qr.lo, s2[r]));
            }
        }
        const bool ok = (valid >> key) & 1;
        bool over = false;
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
            const float2 both = unpair(s2[r]);
            s[r] = both.x + both.y;
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 8);
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 16);
            s[r] = ok ? s[r] * scale2 : -INFINITY;
            over |= s[r] > m[r] + LAZY;
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int r = 0; r < C::ROWS; r++) {
                float mn = fmaxf(m[r], s[r]);
#pragma unroll
                for (int x = 1; x < 8; x <<= 1)
                    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
                const float alpha = mn > m[r] ? ex2(m[r] - mn) : 1.0f;
                m[r] = mn;
                l[r] *= alpha;
#pragma unroll
                for (int c = 0; c < PER; c++)
                    o[r][c] = {mul2(o[r][c].lo, pair(alpha, alpha)), mul2(o[r][c].hi, pair(alpha, alpha))};
            }
        }
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
            s[r] = ex2(s[r] - (m[r] == -INFINITY ? 0.0f : m[r]));   // NaN stays NaN, whatever m is
            l[r] += s[r];   // this lane's key; the eight keys are added in finish()
        }
        const int col = lane % LPR, sub = lane / LPR;
#pragma unroll
        for (int j = 0; j < 8; j += KSPLIT) {
            const int kj = j + sub;
            Quad v[PER];
#pragma unroll
            for (int c = 0; c < PER; c++)
                v[c] = lds_quad(vs + C::at(kj, col + c * 32));
#pragma unroll
            for (int r = 0; r < C::ROWS; r++) {
                const float pr = __shfl_sync(0xffffffffu, s[r], kj);
                const unsigned long long p2 = pair(pr, pr);
#pragma unroll
                for (int c = 0; c < PER; c++)
                    o[r][c] = {fma2(p2, v[c].lo, o[r][c].lo), fma2(p2, v[c].hi, o[r][c].hi)};
            }
        }
    }

    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
#pragma unroll
            for (int x = 1; x < 8; x <<= 1)
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
#pragma unroll
            for (int c = 0; c < PER; c++)
#pragma unroll
                for (int x = LPR; x < 32; x <<= 1) {
                    float2 a = unpair(o[r][c].lo), b = unpair(o[r][c].hi);
                    a.x += __shfl_xor_sync(0xffffffffu, a.x, x), a.y += __shfl_xor_sync(0xffffffffu, a.y, x);
                    b.x += __shfl_xor_sync(0xffffffffu, b.x, x), b.y += __shfl_xor_sync(0xffffffffu, b.y, x);
                    o[r][c] = {pair(a.x, a.y), pair(b.x, b.y)};
                }
        }
    }

    __device__ __forceinline__ void to_slot(float *sl, int rows, int D) {
        const int lane = threadIdx.x & 31, col = lane % LPR;
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
            if (r >= rows)
                break;
#pragma unroll
            for (int c = 0; c < PER; c++)
                if (lane < LPR && (col + c * 32) * 4 < D) {
                    const float2 a = unpair(o[r][c].lo), b = unpair(o[r][c].hi);
                    *reinterpret_cast<float4 *>(sl + r * D + (col + c * 32) * 4) = make_float4(a.x, a.y, b.x, b.y);
                }
            if (lane == 0) {
                sl[rows * D + r] = m[r];
                sl[rows * D + rows + r] = l[r];
            }
        }
    }
};

// A warp's copies into its ring: lane i holds the table entry of key i of the
// next tile, loaded while earlier tiles are under way.
template <typename C>
struct Feed {
    using T = typename C::T;
    static constexpr int EPC = 16 / (int)sizeof(T);                 // entries per chunk
    static constexpr int RPI = C::NCH >= 32 ? 1 : 32 / C::NCH;      // rows per instruction
    static constexpr int CPL = C::NCH > 32 ? C::NCH / 32 : 1;       // chunks of a row per lane
    static constexpr uint32_t kAll = C::TK == 32 ? 0xffffffffu : (1u << C::TK % 32) - 1;
    const AttnParams &p;
    uint32_t ring;
    int ent, ent_off;    // page and offset in it of this lane's key; of the tile's first key where page % TK == 0
    uint32_t want;       // keys of the tile, a bit each

    __device__ __forceinline__ Feed(const AttnParams &p_, uint32_t ring_) : p(p_), ring(ring_) {}

    // Starts loading the entries of a tile of `n` (at most TK) keys from `key0` on; row: the request's table.
    __device__ __forceinline__ void fetch(const int32_t *row, int key0, int n) {
        const int lane = threadIdx.x & 31;
        want = n < 32 ? (1u << n) - 1 : 0xffffffffu;
        ent = -1;
        if (p.one_page || lane < n) {
            const int key = p.one_page ? key0 : key0 + lane;
            const int blk = quotient(key, p.by_page);
            ent_off = key - blk * p.page;
            ent = row[blk];
        }
    }

    // Starts the copies of the fetched tile into a stage; returns its valid keys.
    __device__ __forceinline__ uint32_t tile(int stage, int64_t head_off) {
        const int lane = threadIdx.x & 31;
        const int sub = C::NCH >= 32 ? 0 : lane / C::NCH, ch0 = C::NCH >= 32 ? lane : lane % C::NCH;
        // row j RPI + sub, chunk ch0 + 32 c: its swizzle is that of row sub but for the bits of j RPI
        const uint32_t dst = ring + stage * 2 * C::TILE_BYTES + sub * C::ROW_BYTES;
        const uint32_t sw = (ch0 ^ sub) << 4;
        const bool has = ent >= 0 && ent < p.num_pages;
        uint32_t valid = has ? want : 0u;
        int64_t off = has ? ent * p.page_stride + ent_off * p.slot_stride + head_off : 0;
        if (!p.one_page)
            valid = __ballot_sync(0xffffffffu, has) & want;
        if (valid != want && p.status)
            atomicOr(p.status, 1);
        if (p.one_page && valid == kAll) {   // one page, every key: the rows are slot_stride apart
            const T *k = (const T *)p.k + off + sub * p.slot_stride + ch0 * EPC;
            const T *v = (const T *)p.v + off + sub * p.slot_stride + ch0 * EPC;
            const int64_t step = RPI * p.slot_stride;
#pragma unroll
            for (int j = 0; j < C::TK / RPI; j++) {
                const uint32_t d = dst + j * RPI * C::ROW_BYTES + (sw ^ ((j * RPI & 7) << 4));
#pragma unroll
                for (int c = 0; c < CPL; c++)
                    if (C::WHOLE || (ch0 + c * 32) * EPC < p.D) {
                        cp_async16(d + c * 512, k + c * 32 * EPC);
                        cp_async16(d + c * 512 + C::TILE_BYTES, v + c * 32 * EPC);
                    }
                k += step, v += step;
            }
            return valid;
        }
#pragma unroll
        for (int j = 0; j < C::TK / RPI; j++) {
            const int row = j * RPI + sub;
            const int64_t ro = (p.one_page ? off + row * p.slot_stride : __shfl_sync(0xffffffffu, off, row)) + ch0 * EPC;
            const bool ok = (valid >> row) & 1;
            const uint32_t d = dst + j * RPI * C::ROW_BYTES + (sw ^ ((j * RPI & 7) << 4));
            const T *k = (const T *)p.k + (ok ? ro : 0), *v = (const T *)p.v + (ok ? ro : 0);
            const int n = ok ? 16 : 0;
#pragma unroll
            for (int c = 0; c < CPL; c++)
                if (C::WHOLE || (ch0 + c * 32) * EPC < p.D) {
                    cp_async16(d + c * 512, k + c * 32 * EPC, n);
                    cp_async16(d + c * 512 + C::TILE_BYTES, v + c * 32 * EPC, n);
                }
        }
        return valid;
    }
};

// A partial result in memory: rows x D outputs, then rows maxima, then rows sums
// (relative to the maximum, as o is), to a multiple of 16 bytes.
__host__ __device__ __forceinline__ int partial_floats(int rows, int D) { return (rows * (D + 2) + 3) / 4 * 4; }

// Counts an arrival: what the CTA has written is visible to the CTA that counts
// the last one (called by one thread, behind a barrier of its CTA).
__device__ __forceinline__ uint32_t arrive(int *counter) {
    uint32_t n;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
    return n;
}

__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

// Waits until at most n (1 .. kMaxStages - 1) groups of this thread's copies are on their way.
__device__ __forceinline__ void cp_wait_rt(int n) {
    switch (n) {
    case 1: cp_wait<1>(); break;
    case 2: cp_wait<2>(); break;
    case 3: cp_wait<3>(); break;
    case 4: cp_wait<4>(); break;
    default: cp_wait<5>(); break;
    }
}

// Joins partial results of a row for four outputs a lane: ml(i) is the maximum and
// sum of part i, out(i) the lane's outputs of it.  Four parts are on their way at a
// time and every lane works out every weight: no lane waits for another (16
// requests of 128 tokens: 5.15 us, 5.4 with weights by shuffle, 5.5 with eight).
template <typename MaxSum, typename Out>
__device__ __forceinline__ float4 merge(int parts, float &M, float &L, MaxSum ml, Out out) {
    constexpr int N = 4;
    float4 o = make_float4(0, 0, 0, 0);
    M = -INFINITY, L = 0.0f;
    for (int i = 0; i < parts; i += N) {
        float2 s[N];
        float4 v[N];
#pragma unroll
        for (int u = 0; u < N; u++)
            if (i + u < parts)
                s[u] = ml(i + u), v[u] = out(i + u);
        float mn = M;
#pragma unroll
        for (int u = 0; u < N; u++)
            mn = i + u < parts ? fmaxf(mn, s[u].x) : mn;
        const float base = mn == -INFINITY ? 0.0f : mn, old = ex2(M - base);
        M = mn, L *= old;
        o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
        for (int u = 0; u < N; u++)
            if (i + u < parts) {
                const float w = ex2(s[u].x - base);
                L = fmaf(w, s[u].y, L);
                fma4(o, w, v[u]);
            }
    }
    return o;
}

template <typename C>
__global__ void __launch_bounds__(C::kWarpsMost * 32) paged_attention_kernel(const __grid_constant__ AttnParams p) {
    using T = typename C::T;
    using A = Acc<C, C::F16>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t vmask[kMaxWarps][kMaxStages];    // valid keys of the tile in each stage
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int kRing = p.stages * 2 * C::TILE_BYTES;   // bytes a warp
    uint8_t *my_ring = smem + (size_t)warp * kRing;
    const uint32_t ring = smem_u32(my_ring);
    uint8_t *q_rows = smem + (size_t)W * kRing;   // then the CTA's partial result
    const int S = p.split, P = p.groups, seg = blockIdx.y, b = blockIdx.z;
    const int group = P == 1 ? 0 : quotient(blockIdx.x, p.by_split), rank = blockIdx.x - group * S;
    const int h = p.row_tiles == 1 ? seg : seg / p.row_tiles, r0 = (seg - h * p.row_tiles) * C::ROWS;
    auto head_of = [&](int r) { return r0 + r < p.G ? h * p.G + r0 + r : -1; };   // of row r of the segment

    // half a step of 16 entries is beyond D: K's there, which no copy writes, must be finite
    if (C::F16 && !C::WHOLE && p.D % 16)
        for (int i = lane; i < p.stages * C::TK; i += 32)
            *reinterpret_cast<uint4 *>(my_ring + i / C::TK * 2 * C::TILE_BYTES + C::at(i % C::TK, p.D / 8)) =
                make_uint4(0, 0, 0, 0);

    pdl_wait();
    pdl_launch_dependents();
    const int given = p.lens[b], len = min(max(given, 0), p.cap);
    if (given != len && blockIdx.x == 0 && seg == 0 && threadIdx.x == 0 && p.status)
        atomicOr(p.status, 2);
    const int tiles = (int)(((uint32_t)len + C::TK - 1) / C::TK);
    // the group's tiles [g0, g1), the CTA's [t0, t1)
    const int per_group = P == 1 ? tiles : quotient(tiles + P - 1, p.by_groups);
    const int g0 = group * per_group, g1 = min(tiles, g0 + per_group);
    if (group > 0 && g0 >= tiles)
        return;
    const int used_groups = P == 1 || tiles == 0 ? 1 : (tiles + per_group - 1) / per_group;
    // a segment too short for all S CTAs leaves the last of them idle; one for a single CTA needs no cluster
    const int per = S == 1 ? g1 - g0 : max(quotient(g1 - g0 + S - 1, p.by_split), p.least);
    const bool joined = per < g1 - g0;
    if (!joined && rank > 0)
        return;
    const int t0 = g0 + rank * per, t1 = min(g1, t0 + per);

    const int32_t *row = p.table + b * p.table_stride;
    const int64_t head_off = h * p.head_stride;
    int t = t0 + warp, load = t;   // tile to compute, tile to issue
    Feed<C> feed(p, ring);
    auto issue = [&](int stage) {
        if (load < t1) {
            const uint32_t valid = feed.tile(stage, head_off);
            if (lane == 0)
                vmask[warp][stage] = valid;
            load += W;
            if (load < t1)
                feed.fetch(row, load * C::TK, min(C::TK, len - load * C::TK));
        }
        cp_commit();
    };
    if (load < t1)
        feed.fetch(row, load * C::TK, min(C::TK, len - load * C::TK));
    for (int s = 0; s + 1 < p.stages; s++)
        issue(s);
    // the segment's query rows, for all warps
    for (int i0 = threadIdx.x; i0 < p.rows * C::NCH; i0 += 4 * blockDim.x) {
        uint4 v[4];   // four chunks a thread on their way at a time
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int i = i0 + u * blockDim.x, head = head_of(i / C::NCH), e = i % C::NCH * (16 / (int)sizeof(T));
            v[u] = make_uint4(0, 0, 0, 0);
            if (i < p.rows * C::NCH && head >= 0 && e < p.D)
                v[u] = ldg_v4((const T *)p.q + b * p.q_bs + head * p.q_hs + e);
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int i = i0 + u * blockDim.x;
            if (i < p.rows * C::NCH)
                *reinterpret_cast<uint4 *>(q_rows + C::at(i / C::NCH, i % C::NCH)) = v[u];
        }
    }
    __syncthreads();

    const int part_at = p.rows * p.D;   // of a partial result's maxima; the sums follow
    if (t < t1) {
        A acc;
        const uint32_t qs = smem_u32(q_rows);
        acc.open(qs, p.rows);
        int stage = 0;
        for (; t < t1; t += W) {
            __syncwarp();   // every lane has read the stage that the last tile left: it takes the next one
            issue(stage == 0 ? p.stages - 1 : stage - 1);
            cp_wait_rt(p.stages - 1);
            __syncwarp();
            const uint32_t ks = ring + stage * 2 * C::TILE_BYTES;
            acc.tile(ks, ks + C::TILE_BYTES, qs, p.rows, p.D, vmask[warp][stage], p.scale * kLog2e);
            stage = stage + 1 == p.stages ? 0 : stage + 1;
        }
        acc.finish();
        __syncwarp();   // every lane has read the last tile of a ring that is written over
        acc.to_slot(reinterpret_cast<float *>(my_ring), p.rows, p.D);
    }
    __syncthreads();

    // The joins: a warp per row and 128 outputs.
    const int chunks = (p.D + 127) >> 7, tasks = p.rows * chunks;
    const int pf = partial_floats(p.rows, p.D), id = b * gridDim.y + seg;
    auto row_of = [&](int task) { return chunks == 1 ? task : task >> 1; };
    auto col_of = [&](int task) { return (chunks == 1 ? 0 : (task & 1) * 128) + lane * 4; };
    auto keep = [&](float *part, int r, int c, float4 o, float M, float L) {
        if (c < p.D)
            *reinterpret_cast<float4 *>(part + r * p.D + c) = o;
        if (c == 0)
            part[part_at + r] = M, part[part_at + p.rows + r] = L;
    };
    auto write = [&](int r, int c, float4 o, float M, float L) {
        const int head = head_of(r);
        if (head < 0)
            return;
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        if (c < p.D) {
            T *d = (T *)p.out + b * p.o_bs + head * p.o_hs + c;
            store2(d, o.x * inv, o.y * inv);
            store2(d + 2, o.z * inv, o.w * inv);
        }
        if (c == 0 && p.lse)
            p.lse[(int64_t)b * p.Hkv * p.G + head] = lse_of(M, L * A::kSumScale);
    };
    float *group_part = p.partials + ((int64_t)id * P + group) * pf;

    // of the CTA's warps
    float *cta_part = reinterpret_cast<float *>(q_rows);   // every warp is done with the query rows
    {
        const int parts = min(max(t1 - t0, 0), W);
        for (int task = warp; task < tasks; task += W) {
            const int r = row_of(task), c = col_of(task);
            float M, L;
            const float *at = reinterpret_cast<const float *>(smem) + part_at + r;
            const float *from = reinterpret_cast<const float *>(smem) + r * p.D + (c < p.D ? c : 0);
            const float4 o = merge(
                parts, M, L, [&](int i) { return make_float2(at[i * (kRing / 4)], at[i * (kRing / 4) + p.rows]); },
                [&](int i) { return *reinterpret_cast<const float4 *>(from + i * (kRing / 4)); });
            if (joined)
                keep(cta_part, r, c, o, M, L);
            else if (used_groups > 1)
                keep(group_part, r, c, o, M, L);
            else
                write(r, c, o, M, L);
        }
    }
    // of the cluster's CTAs
    if (joined) {
        cluster_sync();
        const int parts = (g1 - g0 + per - 1) / per;   // CTAs with a tile
        const uint32_t at = smem_u32(cta_part);
        for (int task = warp * S + rank; task < tasks; task += W * S) {
            const int r = row_of(task), c = col_of(task);
            const uint32_t ml = at + (part_at + r) * 4, from = at + (r * p.D + (c < p.D ? c : 0)) * 4;
            float M, L;
            const float4 o = merge(
                parts, M, L,
                [&](int i) {
                    const uint32_t m = cluster_map(ml, i);
                    return make_float2(ld_cluster(m), ld_cluster(m + p.rows * 4));
                },
                [&](int i) { return ld_cluster4(cluster_map(from, i)); });
            if (used_groups > 1)
                keep(group_part, r, c, o, M, L);
            else
                write(r, c, o, M, L);
        }
        if (used_groups > 1)
            __threadfence();
        cluster_sync();   // no CTA leaves while another reads its part
    }
    // of the segment's groups
    if (used_groups > 1 && rank == 0) {
        __syncthreads();
        if (threadIdx.x == 0) {
            last = arrive(p.counters + id) == (uint32_t)used_groups - 1;
            if (last)
                p.counters[id] = 0;
        }
        __syncthreads();
        if (!last)
            return;
        const float *first = p.partials + (int64_t)id * P * pf;
        for (int task = warp; task < tasks; task += W) {
            const int r = row_of(task), c = col_of(task);
            float M, L;
            const float4 o = merge(
                used_groups, M, L,
                [&](int i) {
                    const float *ml = first + (int64_t)i * pf + part_at + r;
                    return make_float2(__ldcg(ml), __ldcg(ml + p.rows));
                },
                [&](int i) {
                    return __ldcg(reinterpret_cast<const float4 *>(first + (int64_t)i * pf + r * p.D + (c < p.D ? c : 0)));
                });
            write(r, c, o, M, L);
        }
    }
}

constexpr size_t kSmemMax = 227 * 1024 - 512;   // of a CTA, besides its static shared memory
constexpr size_t kSmemSm = 228 * 1024;          // of an SM, 1 KB of it for each CTA

__global__ void occupancy_kernel() {}

// Clusters of `split` CTAs that run at once on the current device with `per_sm`
// CTAs on an SM, as the driver counts them: a cluster's CTAs share one of the
// GPU's parts, whose SMs differ in number from GPU to GPU (15 clusters of 8 CTAs
// with an SM each on one, 14 on another; one more waits for a whole round: 7
// against 8 requests of 4096 tokens in two heads took 11.9 and 20.5 us).
int64_t clusters_at_once(int per_sm, int split) {
    static int known[kMaxDevices][kMaxWarps + 1][kMaxSplit + 1] = {};   // threads that race here write the same
    static int smem_cache[kMaxDevices] = {};
    const int guess = device_sm_count() * per_sm / split;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return guess;
    int &n = known[dev][per_sm][split];
    if (n == 0) {
        const size_t share = kSmemSm / per_sm - 1024 - 512, smem = share < kSmemMax ? share : kSmemMax;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3((unsigned)split);
        cfg.blockDim = dim3(32);
        cfg.dynamicSmemBytes = smem;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int got = 0;
        const void *kernel = reinterpret_cast<const void *>(occupancy_kernel);
        if (ensure_dynamic_smem(kernel, (int)kSmemMax, smem_cache) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&got, kernel, &cfg) != cudaSuccess || got < 1) {
            (void)cudaGetLastError();   // a failed query is no error of the call's
            got = guess;
        }
        n = got;
    }
    return n;
}

// Tuning hook: what is not 0 replaces the rule's choice.
int g_split = 0, g_warps = 0, g_groups = 0;

template <typename C>
int launch_cfg(AttnParams p, int B, unsigned flags, cudaStream_t s) {
    static int cache[kMaxDevices] = {};
    const int segs = p.Hkv * p.row_tiles, sms = device_sm_count();
    const int64_t all = (int64_t)B * segs;
    const int tiles = (p.cap - 1) / C::TK + 1;   // of the longest request that the table has room for
    p.one_page = p.page % C::TK == 0;
    // The shape, CTAs of a cluster x warps of a CTA: an SM has room for kWarpsMost
    // warps' rings.  Of the shapes whose CTAs all run at once, the one with the most
    // warps; of those, where a warp's ring is 16 KB, the one with the most CTAs, as
    // shorter CTAs even out ragged lengths (16 requests of up to 16384: 97 us as 4 x 3
    // against 101 us as 1 x 12; heads of 256 keep three warps or more for the joins of
    // their longer rows).  More CTAs than 1.5 per SM only for work: 4 tiles a warp (16
    // requests of 128 tokens in 8 heads: 5.4 us as 1 x 4, 9.8 as 4 x 4).
    const int most = C::kWarpsMost;
    int split = 1, warps = 0;
    for (int S = 1; S <= kMaxSplit && S <= tiles; S++) {
        int k = 1;
        while (k <= 6 && all > clusters_at_once(k, S))
            k++;
        const int W = most / k;
        if (k > 6 || W < most / 6 || (most < kMaxWarps && W < 3) ||
            (S > 1 && 2 * all * S > 3 * sms && (int64_t)4 * S * W > tiles))
            continue;
        if (S * W > split * warps || (S * W == split * warps && most == kMaxWarps && W >= 3))
            split = S, warps = W;
    }
    // More segments than that, or long work for each warp: CTAs of a third of an SM,
    // about 32 tiles a warp, in turn (64 requests of up to 8192: 164 us as 4 x 4,
    // 176 as 1 x 4); short segments as CTAs of two warps (256 requests of 100: 27.8
    // us as 1 x 2, 32 as 1 x 4).  The lengths are on the device, and no edge between
    // two and four warps is right for all: even lengths gain from two at any length,
    // ragged ones from four behind about 24 tiles (40 requests in 16 heads of 64, as
    // 1 x 2 and 1 x 4: of 1000 tokens 31.5 and 36.1 us, of up to 1000 25.6 and 21.5;
    // of 1500 45.8 and 51.2, of up to 1500 34.9 and 25.1; of 1600 48.0 and 54.0, of up
    // to 1600 36.6 and 27.5; 256 requests in 8 heads of 128: of 1000 158 and 156, of up
    // to 1000 87 and 84).
    if (warps == 0 || (split < kMaxSplit && tiles > 32 * split * warps) || (warps < 3 && tiles > 24 * warps)) {
        const int W = tiles <= 48 ? 2 : most == kMaxWarps ? 4 : 3, long_split = (tiles - 1) / (32 * W) + 1;
        split = long_split > split ? long_split : split;
        split = split < kMaxSplit ? split : kMaxSplit;
        warps = W;
    }
    split = g_split ? g_split : split;
    // no more warps than tiles, or than rows to join (one key of 16 heads of 256: 25.9 us with one warp)
    const int joins = p.rows * ((p.D + 127) / 128), useful = (tiles - 1) / split + 1 > joins ? (tiles - 1) / split + 1 : joins;
    warps = useful < warps ? useful : warps;
    warps = g_warps ? g_warps < C::kWarpsMost ? g_warps : C::kWarpsMost : warps;
    // Groups: where the clusters of a few long segments would leave SMs idle, until a warp has 4 tiles.
    int64_t groups = 1;
    if (all <= clusters_at_once(1, kMaxSplit) && tiles > 6 * split * warps) {
        const int64_t want = (tiles - 1) / (4 * split * warps) + 1, room = clusters_at_once(1, split) / all;
        groups = want < room ? want : room;
    }
    groups = g_groups ? g_groups : groups;
    groups = groups < 32 ? groups : 32;
    groups = all * groups > kMaxGroups || groups < 1 ? 1 : groups;
    // A deeper ring where the CTAs leave room for one.
    const size_t stage = (size_t)warps * 2 * C::TILE_BYTES, q_bytes = (size_t)p.rows * C::ROW_BYTES;
    const size_t part_bytes = (size_t)partial_floats(p.rows, p.D) * 4, tail = q_bytes > part_bytes ? q_bytes : part_bytes;
    static_assert(2 * 2 * C::TILE_BYTES >= (C::ROWS * (C::DP + 2) + 3) / 4 * 16, "a ring holds its warp's partial result");
    int per_sm = 1;
    while (per_sm < C::kWarpsMost / warps && all * groups > clusters_at_once(per_sm, split))
        per_sm++;
    size_t room = kSmemSm / per_sm - 1024 - 512;
    room = room < kSmemMax ? room : kSmemMax;
    const size_t fit = (room - tail) / stage;
    p.stages = fit < 2 ? 2 : fit > kMaxStages ? kMaxStages : (int)fit;
    // few CTAs: every one for the shortest way; many: none for less than two tiles a warp
    p.least = all * split <= 2 * sms ? 1 : 2 * warps;
    p.split = split, p.groups = (int)groups;
    p.by_page = div_by((uint32_t)p.page), p.by_split = div_by((uint32_t)split), p.by_groups = div_by((uint32_t)groups);

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(split * groups), (unsigned)segs, (unsigned)B);
    cfg.blockDim = dim3((unsigned)warps * 32);
    cfg.dynamicSmemBytes = p.stages * stage + tail;
    cfg.stream = s;
    cfg.attrs = attr;
    if (split > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    if (flags & MNB_FLAG_PDL) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    auto *kernel = paged_attention_kernel<C>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)cfg.dynamicSmemBytes, cache);
    if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess)
        return fail(MNB_ERR_CUDA, "mnb_paged_attention: launch: %s", cudaGetErrorString(e));
    return MNB_OK;
}

template <typename T, int DP, int ROWS>
int launch_rows(const AttnParams &p, int B, unsigned flags, cudaStream_t s) {
    return p.D == DP ? launch_cfg<Cfg<T, DP, ROWS, true>>(p, B, flags, s)
                     : launch_cfg<Cfg<T, DP, ROWS, false>>(p, B, flags, s);
}

template <typename T, int DP>
int launch_dp(const AttnParams &p, int B, unsigned flags, cudaStream_t s) {
    if constexpr (std::is_same<T, half>::value)
        return p.rows > 8   ? launch_rows<T, DP, 16>(p, B, flags, s)
               : p.rows > 4 ? launch_rows<T, DP, 8>(p, B, flags, s)
                            : launch_rows<T, DP, 4>(p, B, flags, s);
    else
        return p.rows > 4   ? launch_rows<T, DP, 8>(p, B, flags, s)
               : p.rows > 2 ? launch_rows<T, DP, 4>(p, B, flags, s)
               : p.rows > 1 ? launch_rows<T, DP, 2>(p, B, flags, s)
                            : launch_rows<T, DP, 1>(p, B, flags, s);
}

int rows_per_segment(int G, int f16) { return G < (f16 ? 16 : 8) ? G : (f16 ? 16 : 8); }
constexpr size_t kCounterBytes = kMaxGroups * 4;

}  // namespace

int set_paged_attention_shape(int split, int warps, int groups) {
    if (split < 0 || split > kMaxSplit || warps < 0 || warps > kMaxWarps || groups < 0 || groups > 32)
        return MNB_ERR_INVALID_ARG;
    g_split = split, g_warps = warps, g_groups = groups;
    return MNB_OK;
}

size_t paged_attention_workspace_bytes(int Hq, int Hkv, int D, int f16) {
    return kCounterBytes + (size_t)kMaxGroups * partial_floats(rows_per_segment(Hq / Hkv, f16), D) * 4;
}

int launch_paged_attention(const void *q, int64_t q_bs, int64_t q_hs, const mnb_paged_cache *c, const int32_t *table,
                           int64_t table_stride, int max_blocks, const int32_t *lens, int B, int Hq, float scale,
                           void *out, int64_t o_bs, int64_t o_hs, float *lse, void *workspace, int *status,
                           unsigned flags, cudaStream_t s) {
    const int f16 = c->dtype == MNB_F16;
    AttnParams p;
    p.q = q, p.k = c->k, p.v = c->v, p.out = out, p.lse = lse, p.table = table, p.lens = lens, p.status = status;
    p.q_bs = q_bs, p.q_hs = q_hs, p.o_bs = o_bs, p.o_hs = o_hs, p.table_stride = table_stride;
    p.page_stride = c->page_stride, p.slot_stride = c->slot_stride, p.head_stride = c->head_stride;
    p.Hkv = (int)c->num_heads, p.G = Hq / p.Hkv, p.D = (int)c->head_dim;
    p.rows = rows_per_segment(p.G, f16);
    p.row_tiles = (p.G + p.rows - 1) / p.rows;
    p.page = (int)c->page_size, p.num_pages = (int)c->num_pages, p.cap = max_blocks * p.page, p.scale = scale;
    p.counters = (int *)workspace;
    p.partials = (float *)((uint8_t *)workspace + kCounterBytes);
    if (f16)
        return p.D <= 64    ? launch_dp<half, 64>(p, B, flags, s)
               : p.D <= 128 ? launch_dp<half, 128>(p, B, flags, s)
                            : launch_dp<half, 256>(p, B, flags, s);
    return p.D <= 64    ? launch_dp<float, 64>(p, B, flags, s)
           : p.D <= 128 ? launch_dp<float, 128>(p, B, flags, s)
                        : launch_dp<float, 256>(p, B, flags, s);
}

}  // namespace mnb

extern "C" MNB_API int mnb_tune_paged_attention(int split, int warps, int groups) {
    return mnb::set_paged_attention_shape(split, warps, groups);
}
