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
// Work split.  The keys of every (request, KV head, row tile of query heads) --
// a segment -- are cut into tiles of TK keys.  All tiles of the call, in the
// order (request, segment, tile), form one list that is cut into equal
// contiguous ranges, one per CTA, and each CTA's range again into one per warp:
// every warp streams the same number of tiles (+-1) whatever the lengths are.
// A segment inside one warp's range is finished there; one that crosses warps
// is joined in shared memory, one that crosses CTAs through the workspace, by
// the CTA that arrives last, in CTA order (the result does not depend on which
// CTA that is).
//
// Each warp owns a ring of STAGES tiles in shared memory that it fills with
// 16-byte cp.async (rows behind the length and rows of page ids outside the
// pool are zero-filled and masked, never read) and drains by itself: the main
// loop has no CTA barrier, and the next segment's query rows (a stage of their
// own) and first tiles are in flight while the current one ends.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mnb_tune.h"

namespace mnb {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 3;   // per SM
constexpr int kMaxWarps = 12; // of a CTA of the cluster kernel
constexpr int kClusterTiles = 16;   // most tiles a warp of the cluster kernel may have
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    int *counters;      // workspace: arrivals for the one segment that crosses the end of a CTA's range and
                        // begins inside it, one count per CTA, zero between calls
    float *partials;    // workspace: two partial results per CTA
    int *status;
    int64_t q_bs, q_hs, o_bs, o_hs;                        // elements
    int64_t table_stride, page_stride, slot_stride, head_stride;
    int B, G, Hkv, D, rows, row_tiles, page, num_pages, cap;   // cap: rows the table has room for
    int page_shift;                                        // log2(page), -1 if it is no power of two
    int one_page, whole;                                   // a tile's keys are in one page: page % TK == 0; and D == DP
    int min_tiles;                                         // fewest tiles worth a CTA
    float join_cost;                                       // of a partial result in the last join, in tiles
    uint32_t split_magic;                                  // cluster kernel: ceil(2^32 / CTAs per segment)
    int stages;                                            // cluster kernel: of each warp's ring
    float scale;
};

// Element type, padded head size, rows of query heads per segment.  A tile is
// 8 KB of K and V (16 KB for heads of 256): 16 keys of 128 fp16 entries.
// Rows are swizzled in shared memory (chunk ^ row % 8), so that reads of eight
// rows' same chunk meet no bank twice.
template <typename T_, int DP_, int ROWS_>
struct Cfg {
    using T = T_;
    static constexpr bool F16 = std::is_same<T, half>::value;
    static constexpr int DP = DP_, ROWS = ROWS_, STAGES = 2;
    static constexpr int TK = (F16 ? 16 : 8) * (DP <= 64 ? 2 : 1);   // keys per tile
    static constexpr int NCH = DP * (int)sizeof(T) / 16;             // 16-byte chunks per row
    static constexpr int ROW_BYTES = DP * (int)sizeof(T);
    static constexpr int TILE_BYTES = TK * ROW_BYTES;
    static __device__ __forceinline__ uint32_t at(int row, int chunk) { return row * ROW_BYTES + (chunk ^ (row & 7)) * 16; }
    static constexpr int kWarpsMost = DP > 128 ? 6 : kMaxWarps;      // as far as shared memory goes
    static constexpr int kCtas = DP > 128 ? 1 : !F16 && ROWS > 4 ? 2 : kMaxCtas;                          // CTAs on an SM, as far as registers go
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
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float dot(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ void fma4(float4 &c, float s, float4 v) {
    c.x = fmaf(s, v.x, c.x), c.y = fmaf(s, v.y, c.y), c.z = fmaf(s, v.z, c.z), c.w = fmaf(s, v.w, c.w);
}

// A position in the list of tiles (32 bits: the host refuses longer lists).
struct Cursor {
    int b, seg;              // request, segment in it
    uint32_t tile, tiles;    // tile in the segment, tiles per segment of b
};

struct Shared {
    const uint32_t *prefix;    // [B + 1] tiles (of one segment) before request b
    int B, NS;                 // NS = segments per request
};

__device__ __forceinline__ Cursor cursor_at(const Shared &sh, uint32_t t) {
    Cursor c;
    const uint32_t u = t / (uint32_t)sh.NS;   // among the requests' tiles of one segment each
    int lo = 0, hi = sh.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sh.prefix[mid + 1] > u)
            hi = mid;
        else
            lo = mid + 1;
    }
    c.b = lo;
    c.tiles = sh.prefix[lo + 1] - sh.prefix[lo];
    const uint32_t r = t - sh.prefix[lo] * (uint32_t)sh.NS;
    c.seg = (int)(r / c.tiles);
    c.tile = r - (uint32_t)c.seg * c.tiles;
    return c;
}

// The next tile; the caller knows that there is one.
__device__ __forceinline__ void advance(const Shared &sh, Cursor &c) {
    if (++c.tile < c.tiles)
        return;
    c.tile = 0;
    if (++c.seg < sh.NS)
        return;
    c.seg = 0;
    do {
        c.b++;
        c.tiles = sh.prefix[c.b + 1] - sh.prefix[c.b];
    } while (c.tiles == 0);
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

// log sum exp from a maximum in log2 units and a sum relative to it.
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.0f ? m * kLn2 + logf(l) : -INFINITY; }

// The running softmax of one segment in a warp's registers.  The maximum m is a
// reference, not the exact maximum: it moves, and o and l are rescaled, only
// when a score exceeds it by more than 2^LAZY (in most tiles one vote says that
// none does, and no maximum is taken across lanes).
constexpr float LAZY = 5.0f;

template <typename C, bool F16>
struct Acc;

// fp16: S^T = K Q^T and O^T += V^T P^T as m16n8k16 products: keys, then head
// entries are the 16 rows, up to 8 query heads the 8 columns (the grouped heads
// of one KV head seldom fill more).  P is rounded to fp16 for the second
// product, scaled so that the reference maximum is at 2^SHIFT: its largest
// values stay below 2^15, and terms down to 2^-24 of the largest keep their 11
// bits.  l is summed from the unrounded fp32 values.
template <typename C>
struct Acc<C, true> {
    static constexpr int NT = C::ROWS / 8, KB = C::TK / 16, KS = C::DP / 16;
    static constexpr float SHIFT = 10.0f;
    static constexpr float kSumScale = 1.0f / 1024.0f;   // 2^-SHIFT
    float o[KS][NT][4];        // entry 16 i + lane / 4 (+ 8), heads 2 (lane % 4) and the next
    float m[NT][2], l[NT][2];
    uint32_t q[KS][NT][2];     // B fragments of the segment's query rows

    // The segment's query rows, just landed at `qs`.
    __device__ __forceinline__ void open(uint32_t qs, uint32_t, int rows) {
        const int lane = threadIdx.x & 31, i = lane >> 3;
        if constexpr (NT == 1) {
            const int r = min(lane & 7, rows - 1);
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
    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, uint32_t, int, uint32_t valid, float scale2) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        float s[KB][NT][4];
        {
            float h[2][KB][NT][4] = {};   // even and odd steps: two chains of products
            const int kr = (lane & 7) + ((lane >> 3) & 1) * 8, kc = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < KS; kk++)
#pragma unroll
                for (int b = 0; b < KB; b++) {
                    uint32_t a0, a1, a2, a3;
                    ldsm4(ks + C::at(b * 16 + kr, kk * 2 + kc), a0, a1, a2, a3);
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        mma16816(h[kk & 1][b][t], a0, a1, a2, a3, q[kk][t][0], q[kk][t][1]);
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
        uint32_t p[KB][NT][2];
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
                    p[b][t][h] = transpose8(h2_as_u32(__floats2half2_rn(x, y)));
                }
        }
        const int vr = (lane & 7) + (lane >> 4) * 8, vc = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < KS; k++)
#pragma unroll
            for (int b = 0; b < KB; b++) {
                uint32_t a0, a1, a2, a3;
                ldsm4t(vs + C::at(b * 16 + vr, k * 2 + vc), a0, a1, a2, a3);
#pragma unroll
                for (int t = 0; t < NT; t++)
                    mma16816(o[k][t], a0, a1, a2, a3, p[b][t][0], p[b][t][1]);
            }
    }

    // Sums over the lanes' keys.
    __device__ __forceinline__ void finish() {
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

    // The finished rows: row(r) is the query head of row r, or -1.
    template <typename F>
    __device__ __forceinline__ void to_out(half *out, int64_t hs, float *lse, int D, F row) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const float i0 = l[t][0] > 0.0f ? 1.0f / l[t][0] : 0.0f, i1 = l[t][1] > 0.0f ? 1.0f / l[t][1] : 0.0f;
            const int head = row(t * 8 + g);
            half *p = out + head * hs + t2;
#pragma unroll
            for (int k = 0; k < 2 * KS; k++) {
                const int h = 2 * (k & 1);
                const uint32_t v = transpose8(h2_as_u32(__floats2half2_rn(o[k / 2][t][h] * i0, o[k / 2][t][h + 1] * i1)));
                if (head >= 0 && k * 8 < D)
                    *reinterpret_cast<uint32_t *>(p + k * 8) = v;
            }
            if (lse && g < 2) {
                const int hl = row(t * 8 + t2 + g);
                if (hl >= 0)
                    lse[hl] = lse_of(g ? m[t][1] : m[t][0], (g ? l[t][1] : l[t][0]) * kSumScale);
            }
        }
    }
};

// fp32: every product and sum in fp32 on the CUDA cores, eight keys at a time.
// Scores: a lane holds key lane % 8 and a quarter of the chunks, two shuffles
// add the quarters.  Output: a lane holds whole columns; a row's probabilities
// come by shuffle.
template <typename C>
struct Acc<C, false> {
    static constexpr int LPR = C::NCH < 32 ? C::NCH : 32;   // lanes per row of V
    static constexpr int PER = C::NCH / LPR;                // chunks a lane holds
    static constexpr int KSPLIT = 32 / LPR;                 // keys taken at a time
    static constexpr float kSumScale = 1.0f;
    float4 o[C::ROWS][PER];
    float m[C::ROWS], l[C::ROWS];

    // The segment's query rows, just landed at `land`: kept at `qs` (which may be `land`).
    __device__ __forceinline__ void open(uint32_t land, uint32_t qs, int rows) {
        __syncwarp();   // the last segment's rows have been read
        for (int i = threadIdx.x & 31; land != qs && i < rows * C::NCH; i += 32) {
            const float4 v = lds4(land + i * 16);
            asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(qs + i * 16), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                         : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
#pragma unroll
            for (int c = 0; c < PER; c++)
                o[r][c] = make_float4(0, 0, 0, 0);
            m[r] = -INFINITY;
            l[r] = 0.0f;
        }
    }

    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, uint32_t qs, int rows, uint32_t valid, float scale2) {
#pragma unroll 1
        for (int j = 0; j < C::TK / 8; j++)
            eight(ks + j * 8 * C::ROW_BYTES, vs + j * 8 * C::ROW_BYTES, qs, rows, valid >> (8 * j), scale2);
    }

    __device__ __forceinline__ void eight(uint32_t ks, uint32_t vs, uint32_t qs, int rows, uint32_t valid, float scale2) {
        const int lane = threadIdx.x & 31, key = lane & 7, quarter = lane >> 3;
        float s[C::ROWS] = {};
#pragma unroll 4
        for (int c = 0; c < C::NCH / 4; c++) {
            const int ch = c * 4 + quarter;
            const float4 k = lds4(ks + C::at(key, ch));
#pragma unroll
            for (int r = 0; r < C::ROWS; r++) {
                const int qr = min(r, rows - 1);
                s[r] = dot(k, lds4(qs + C::at(qr, ch)), s[r]);
            }
        }
        const bool ok = (valid >> key) & 1;
        bool over = false;
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
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
                    o[r][c].x *= alpha, o[r][c].y *= alpha, o[r][c].z *= alpha, o[r][c].w *= alpha;
            }
        }
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
            s[r] = m[r] == -INFINITY ? 0.0f : ex2(s[r] - m[r]);
            l[r] += s[r];   // this lane's key; the eight keys are added in finish()
        }
        const int col = lane % LPR, sub = lane / LPR;
#pragma unroll
        for (int j = 0; j < 8; j += KSPLIT) {
            const int kj = j + sub;
            float4 v[PER];
#pragma unroll
            for (int c = 0; c < PER; c++)
                v[c] = lds4(vs + C::at(kj, col + c * 32));
#pragma unroll
            for (int r = 0; r < C::ROWS; r++) {
                const float pr = __shfl_sync(0xffffffffu, s[r], kj);
#pragma unroll
                for (int c = 0; c < PER; c++)
                    fma4(o[r][c], pr, v[c]);
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
                    o[r][c].x += __shfl_xor_sync(0xffffffffu, o[r][c].x, x);
                    o[r][c].y += __shfl_xor_sync(0xffffffffu, o[r][c].y, x);
                    o[r][c].z += __shfl_xor_sync(0xffffffffu, o[r][c].z, x);
                    o[r][c].w += __shfl_xor_sync(0xffffffffu, o[r][c].w, x);
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
                if (lane < LPR && (col + c * 32) * 4 < D)
                    *reinterpret_cast<float4 *>(sl + r * D + (col + c * 32) * 4) = o[r][c];
            if (lane == 0) {
                sl[rows * D + r] = m[r];
                sl[rows * D + rows + r] = l[r];
            }
        }
    }

    template <typename F>
    __device__ __forceinline__ void to_out(float *out, int64_t hs, float *lse, int D, F row) {
        const int lane = threadIdx.x & 31, col = lane % LPR;
#pragma unroll
        for (int r = 0; r < C::ROWS; r++) {
            const int head = row(r);
            if (head < 0)
                continue;
            const float inv = l[r] > 0.0f ? 1.0f / l[r] : 0.0f;
#pragma unroll
            for (int c = 0; c < PER; c++)
                if (lane < LPR && (col + c * 32) * 4 < D)
                    *reinterpret_cast<float4 *>(out + head * hs + (col + c * 32) * 4) =
                        make_float4(o[r][c].x * inv, o[r][c].y * inv, o[r][c].z * inv, o[r][c].w * inv);
            if (lane == 0 && lse)
                lse[head] = lse_of(m[r], l[r]);
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
            const int blk = p.page_shift >= 0 ? key >> p.page_shift : key / p.page;
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
        if (p.whole && valid == kAll) {   // one page, every key, every column
            const T *k = (const T *)p.k + off + sub * p.slot_stride + ch0 * EPC;
            const T *v = (const T *)p.v + off + sub * p.slot_stride + ch0 * EPC;
            const int64_t step = RPI * p.slot_stride;
#pragma unroll
            for (int j = 0; j < C::TK / RPI; j++) {
                const uint32_t d = dst + j * RPI * C::ROW_BYTES + (sw ^ ((j * RPI & 7) << 4));
#pragma unroll
                for (int c = 0; c < CPL; c++) {
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
#pragma unroll
            for (int c = 0; c < CPL; c++) {
                const bool in = ok && (ch0 + c * 32) * EPC < p.D;
                const int64_t at = in ? ro + c * 32 * EPC : 0;
                cp_async16(d + c * 512, (const T *)p.k + at, in ? 16 : 0);
                cp_async16(d + c * 512 + C::TILE_BYTES, (const T *)p.v + at, in ? 16 : 0);
            }
        }
        return valid;
    }

    // Starts the copies of a segment's query rows into a stage; head(r) is row r's query head, or -1.
    template <typename F>
    __device__ __forceinline__ void query(int stage, int b, F head) {
        const uint32_t qs = ring + stage * 2 * C::TILE_BYTES;
        for (int i = threadIdx.x & 31; i < p.rows * C::NCH; i += 32) {
            const int r = i / C::NCH, ch = i % C::NCH, h = head(r);
            const bool in = h >= 0 && ch * EPC < p.D;
            const T *src = (const T *)p.q + (in ? b * p.q_bs + h * p.q_hs + ch * EPC : 0);
            cp_async16(qs + C::at(r, ch), src, in ? 16 : 0);
        }
    }
};

// A partial result in memory: rows x D outputs, then rows maxima, then rows sums
// (relative to the maximum, as o is), to a multiple of 16 bytes.
__host__ __device__ __forceinline__ int partial_floats(int rows, int D) { return (rows * (D + 2) + 3) / 4 * 4; }

// First tile of the i-th of n equal ranges of `total` tiles.
__device__ __forceinline__ uint32_t range_at(uint32_t total, uint32_t n, uint32_t i) {
    const uint32_t q = total / n;
    return q * i + min(i, total - q * n);
}
// The range that holds tile t (0 <= t < total).
__device__ __forceinline__ uint32_t range_of(uint32_t total, uint32_t n, uint32_t t) {
    const uint32_t q = total / n, r = total - q * n, cut = r * (q + 1);
    return t < cut ? t / (q + 1) : r + (t - cut) / q;
}

// Counts an arrival: what the CTA has written is visible to the CTA that counts
// the last one (called by one thread, behind a barrier of its CTA).
__device__ __forceinline__ uint32_t arrive(int *counter) {
    uint32_t n;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
    return n;
}

// A segment that more than one warp or CTA works on, as one CTA sees it.
struct Chain {
    int warp, parts;         // its first warp here and the number of warps; parts = 0: none
    int b, seg;
    uint32_t first, end;     // its tiles in the list
};

template <typename C>
__global__ void __launch_bounds__(kThreads, C::kCtas) paged_attention_kernel(const __grid_constant__ AttnParams p) {
    using T = typename C::T;
    using A = Acc<C, C::F16>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kRing = C::STAGES * 2 * C::TILE_BYTES;   // bytes a warp
    uint8_t *ring = smem + (size_t)warp * kRing;
    const int q_bytes = C::F16 ? 0 : p.rows * C::ROW_BYTES;   // fp32 only: the current query rows
    const uint32_t q_keep = smem_u32(smem) + kWarps * kRing + warp * q_bytes;
    const int pf = partial_floats(p.rows, p.D);
    // a warp's partial results: [0] of the segment that its range begins inside
    // of, [1] of the one that it opens and does not end, in its drained ring
    float *heads = reinterpret_cast<float *>(smem + kWarps * (kRing + q_bytes));   // [kWarps][pf]
    auto slot_of = [&](int w, bool opened) {
        return opened ? reinterpret_cast<float *>(smem + (size_t)w * kRing) : heads + w * pf;
    };
    uint32_t *prefix = reinterpret_cast<uint32_t *>(heads + kWarps * pf);          // [B + 1]
    __shared__ uint32_t warp_sums[kWarps];
    __shared__ Chain chains[kWarps + 1];   // [0] the segment that the CTA's range begins inside of, [1 + w] opened by warp w
    __shared__ int last[2];
    __shared__ int2 joins[2];

    pdl_wait();
    pdl_launch_dependents();

    // tiles of each request, and their sums; up to 32 requests: by every warp for itself, to the same words
    uint32_t carry = 0;
    bool bad_len = false;
    const bool alone = p.B <= 32;
    for (int b0 = 0; b0 < p.B; b0 += alone ? 32 : kThreads) {
        const int b = b0 + (alone ? lane : (int)threadIdx.x);
        uint32_t v = 0;
        if (b < p.B) {
            const int n = p.lens[b];
            bad_len |= n < 0 || n > p.cap;
            v = ((uint32_t)min(max(n, 0), p.cap) + C::TK - 1) / C::TK;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += u;
        }
        if (alone) {
            carry = __shfl_sync(0xffffffffu, v, 31);
        } else {
            __syncthreads();
            if (lane == 31)
                warp_sums[warp] = v;
            __syncthreads();
            v += carry;
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                v += w < warp ? warp_sums[w] : 0u;
                carry += warp_sums[w];
            }
        }
        if (b < p.B)
            prefix[b + 1] = v;
    }
    if (lane == 0)
        prefix[0] = 0;
    if (threadIdx.x <= kWarps)
        chains[threadIdx.x].parts = 0;
    if (bad_len && blockIdx.x == 0 && p.status)
        atomicOr(p.status, 2);
    __syncthreads();

    Shared sh;
    sh.prefix = prefix, sh.B = p.B, sh.NS = p.Hkv * p.row_tiles;
    const int Hq = p.Hkv * p.G;

    // requests without a key: zero rows
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
        if (prefix[b + 1] == prefix[b]) {
            for (int i = threadIdx.x; i < Hq * (p.D / 2); i += kThreads)
                store2((T *)p.out + b * p.o_bs + (i / (p.D / 2)) * p.o_hs + (i % (p.D / 2)) * 2, 0.0f, 0.0f);
            if (p.lse)
                for (int i = threadIdx.x; i < Hq; i += kThreads)
                    p.lse[(int64_t)b * Hq + i] = -INFINITY;
        }

    const uint32_t total = carry * (uint32_t)sh.NS;
    // CTAs at work: at least min_tiles tiles each, and few enough for the joins
    // (splits of an average segment x join_cost <= tiles of a CTA)
    const uint32_t least = max((float)p.min_tiles, sqrtf((float)carry / p.B * p.join_cost));
    const uint32_t nc = min(gridDim.x, max(total / least, 1u));
    if (blockIdx.x >= nc || total == 0)
        return;
    const uint32_t c0 = range_at(total, nc, blockIdx.x), c1 = range_at(total, nc, blockIdx.x + 1);
    const uint32_t w0 = c0 + range_at(c1 - c0, kWarps, warp), w1 = c0 + range_at(c1 - c0, kWarps, warp + 1);
    const float scale2 = p.scale * kLog2e;

    // the query head of row r of a segment, or -1 past the group
    auto head_of = [&](int seg, int r) -> int {
        if (p.row_tiles == 1)
            return r < p.G ? seg * p.G + r : -1;   // G = rows
        const int h = seg / p.row_tiles, i = (seg - h * p.row_tiles) * C::ROWS + r;
        return r < p.rows && i < p.G ? h * p.G + i : -1;
    };

    if (w0 < w1) {
        uint32_t left = w1 - w0, todo = left;     // tiles to issue, tiles to compute
        Cursor load = cursor_at(sh, w0), cur = load;
        if (load.tile != 0 && warp == 0 && lane == 0) {
            const uint32_t end = c0 - load.tile + load.tiles;
            chains[0] = {0, (int)range_of(c1 - c0, kWarps, min(end, c1) - 1 - c0) + 1, load.b, load.seg, c0 - load.tile, end};
        }
        bool load_q = true, cur_q = true;         // the segment's query rows come first
        int len = min(p.lens[load.b], p.cap);
        int64_t head_off = (p.row_tiles == 1 ? load.seg : load.seg / p.row_tiles) * p.head_stride;
        Feed<C> feed(p, smem_u32(ring));
        auto fetch = [&]() {
            int n = C::TK;
            if (load.tile + 1 == load.tiles)
                n = len - (int)load.tile * C::TK;
            feed.fetch(p.table + load.b * p.table_stride, (int)load.tile * C::TK, n);
        };
        // Starts the copies of the next item (query rows or a tile) into a stage; the tile's valid keys.
        auto issue = [&](int stage) -> uint32_t {
            if (load_q) {
                load_q = false;
                feed.query(stage, load.b, [&](int r) { return head_of(load.seg, r); });
                return 0;
            }
            const uint32_t valid = feed.tile(stage, head_off);
            if (--left > 0) {
                const int b = load.b;
                advance(sh, load);
                load_q = load.tile == 0;
                if (load_q)
                    head_off = (p.row_tiles == 1 ? load.seg : load.seg / p.row_tiles) * p.head_stride;
                if (load.b != b)
                    len = min(p.lens[load.b], p.cap);
                fetch();
            }
            return valid;
        };
        A acc;
        uint32_t vmask[C::STAGES - 1];   // valid keys of the items in flight
        fetch();
#pragma unroll
        for (int s = 0; s < C::STAGES - 1; s++) {
            vmask[s] = left > 0 ? issue(s) : 0u;
            cp_commit();
        }
        bool opened = cur.tile == 0;   // the segment's first tile is this warp's
        int stage = 0;
        while (todo > 0) {
            __syncwarp();   // every lane has read the stage that the last item left: it takes the next one
            const int ahead = stage == 0 ? C::STAGES - 1 : stage - 1;
            const uint32_t nv = left > 0 ? issue(ahead) : 0u;
            cp_commit();
            cp_wait<C::STAGES - 1>();
            __syncwarp();
            const uint32_t ks = smem_u32(ring) + stage * 2 * C::TILE_BYTES;
            const uint32_t valid = vmask[0];
#pragma unroll
            for (int s = 0; s + 1 < C::STAGES - 1; s++)
                vmask[s] = vmask[s + 1];
            vmask[C::STAGES - 2] = nv;
            stage = stage + 1 == C::STAGES ? 0 : stage + 1;
            if (cur_q) {
                cur_q = false;
                acc.open(ks, q_keep, p.rows);
                continue;
            }
            acc.tile(ks, ks + C::TILE_BYTES, q_keep, p.rows, valid, scale2);
            todo--;
            const bool ends = cur.tile + 1 == cur.tiles;
            if (ends || todo == 0) {
                acc.finish();
                if (opened && ends) {
                    acc.to_out((T *)p.out + cur.b * p.o_bs, p.o_hs, p.lse ? p.lse + (int64_t)cur.b * Hq : nullptr, p.D,
                               [&](int r) { return head_of(cur.seg, r); });
                } else {
                    __syncwarp();   // every lane has read the last tile of a ring that is written over
                    acc.to_slot(slot_of(warp, opened), p.rows, p.D);
                    if (opened && lane == 0) {   // and todo == 0: the segment goes on in the next warp
                        const uint32_t first = w1 - 1 - cur.tile, end = first + cur.tiles;
                        chains[1 + warp] = {warp, (int)range_of(c1 - c0, kWarps, min(end, c1) - 1 - c0) - warp + 1,
                                            cur.b, cur.seg, first, end};
                    }
                }
                opened = true;
                cur_q = true;
            }
            if (todo > 0)
                advance(sh, cur);
        }
    }
    __syncthreads();

    auto write4 = [&](int b, int head, int c, float4 o, float inv) {
        T *d = (T *)p.out + b * p.o_bs + head * p.o_hs + c;
        store2(d, o.x * inv, o.y * inv);
        store2(d + 2, o.z * inv, o.w * inv);
    };

    // segments that cross warps: finished here, or this CTA's part of them to the workspace; a warp per row
    bool wrote = false;
    for (int k = 0; k <= kWarps; k++) {
        const Chain ch = chains[k];
        if (ch.parts == 0)
            continue;
        const bool whole = ch.first >= c0 && ch.end <= c1;
        float *dst = p.partials + ((int64_t)blockIdx.x * 2 + (k > 0)) * pf;
        wrote |= !whole;
        for (int r = warp; r < p.rows; r += kWarps) {
            const float *part[kWarps];
            float w[kWarps], M = -INFINITY, l = 0.0f;
#pragma unroll
            for (int j = 0; j < kWarps; j++) {
                part[j] = slot_of(ch.warp + min(j, ch.parts - 1), k > 0 && j == 0);
                w[j] = j < ch.parts ? part[j][p.rows * p.D + r] : -INFINITY;
                M = fmaxf(M, w[j]);
            }
            const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int j = 0; j < kWarps; j++) {
                w[j] = ex2(w[j] - base);
                l = fmaf(w[j], part[j][p.rows * p.D + p.rows + r], l);
            }
            const int head = whole ? head_of(ch.seg, r) : 0;
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            for (int c = lane * 4; c < p.D; c += 128) {
                float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < kWarps; j++)
                    if (j < ch.parts)
                        fma4(o, w[j], *reinterpret_cast<const float4 *>(part[j] + r * p.D + c));
                if (!whole)
                    *reinterpret_cast<float4 *>(dst + r * p.D + c) = o;
                else if (head >= 0)
                    write4(ch.b, head, c, o, inv);
            }
            if (lane == 0) {
                if (!whole) {
                    dst[p.rows * p.D + r] = M;
                    dst[p.rows * p.D + p.rows + r] = l;
                } else if (head >= 0 && p.lse) {
                    p.lse[(int64_t)ch.b * Hq + head] = lse_of(M, l * A::kSumScale);
                }
            }
        }
    }
    if (!wrote)   // the same in every thread
        return;

    // segments that cross CTAs: the CTA that arrives last joins the parts, in CTA order
    __syncthreads();
    if (threadIdx.x < 2) {
        int mine = -1;
        for (int k = threadIdx.x; k <= (threadIdx.x ? kWarps : 0); k++) {
            const Chain &ch = chains[k];
            if (ch.parts == 0 || (ch.first >= c0 && ch.end <= c1))
                continue;
            const uint32_t cf = range_of(total, nc, ch.first), cl = range_of(total, nc, ch.end - 1);
            if (arrive(p.counters + cf) == cl - cf) {
                p.counters[cf] = 0;
                mine = k;
                joins[threadIdx.x] = make_int2((int)cf, (int)(cl - cf) + 1);
            }
        }
        last[threadIdx.x] = mine;
    }
    __syncthreads();
    float *wm = reinterpret_cast<float *>(smem);   // the rings are free now; the host bounds nc so that this fits them
    for (int kind = 0; kind < 2; kind++) {
        if (last[kind] < 0)
            continue;
        const Chain ch = chains[last[kind]];
        const int cf = joins[kind].x, np = joins[kind].y;
        const float *first = p.partials + ((int64_t)cf * 2 + 1) * pf;             // part 0; part i at rest + (i - 1) * 2 pf
        const float *rest = p.partials + ((int64_t)cf + 1) * 2 * pf;
        auto part = [&](int i) { return i == 0 ? first : rest + (int64_t)(i - 1) * 2 * pf; };
        // fewer rows than warps: 2^sh warps share a row and take every 2^sh-th part each
        const int sh = p.rows == 1 ? 2 : p.rows == 2 ? 1 : 0, sets = 1 << sh;
        static_assert(kWarps == 4, "sets of warps");
        float *red = wm + (p.rows * (np + kWarps) + 3) / 4 * 4;                    // [sets][rows][D]
        for (int r = warp >> sh; r < p.rows; r += kWarps >> sh) {
            const int set = warp & (sets - 1);
            float *w = wm + r * (np + kWarps) + set * ((np + sets - 1) >> sh);     // this set's weights
            // the row's maximum and sum
            float M = -INFINITY, l = 0.0f;
            for (int i = lane; i < np; i += 32) {
                const float mi = __ldcg(part(i) + p.rows * p.D + r), li = __ldcg(part(i) + p.rows * p.D + p.rows + r);
                const float mn = fmaxf(M, mi), at = mn == -INFINITY ? 0.0f : mn;
                l = l * ex2(M - at) + li * ex2(mi - at);
                M = mn;
                if ((i & (sets - 1)) == set)
                    w[i >> sh] = mi;
            }
            const float mine = M;
#pragma unroll
            for (int x = 16; x; x >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
            const float base = M == -INFINITY ? 0.0f : M;
            l *= ex2(mine - base);
            for (int i = lane; i < np; i += 32)   // the lane's own entries again
                if ((i & (sets - 1)) == set)
                    w[i >> sh] = ex2(w[i >> sh] - base);
#pragma unroll
            for (int x = 16; x; x >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, x);
            __syncwarp();
            const int head = head_of(ch.seg, r);
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            for (int c = lane * 4; c < p.D; c += 128) {
                float4 o = make_float4(0, 0, 0, 0);
                for (int i0 = set; i0 < np; i0 += 8 * sets) {
                    float4 v[8];   // eight loads on their way at a time
#pragma unroll
                    for (int u = 0; u < 8; u++)
                        if (i0 + u * sets < np)
                            v[u] = __ldcg(reinterpret_cast<const float4 *>(part(i0 + u * sets) + r * p.D + c));
#pragma unroll
                    for (int u = 0; u < 8; u++)
                        if (i0 + u * sets < np)
                            fma4(o, w[(i0 >> sh) + u], v[u]);
                }
                if (sets > 1)
                    *reinterpret_cast<float4 *>(red + (set * p.rows + r) * p.D + c) = o;
                else if (head >= 0)
                    write4(ch.b, head, c, o, inv);
            }
            if (lane == 0 && set == 0 && head >= 0 && p.lse)
                p.lse[(int64_t)ch.b * Hq + head] = lse_of(M, l * A::kSumScale);
            if (sets > 1) {   // one or two rows: every warp is here once
                __syncthreads();
                if (set == 0 && head >= 0)
                    for (int c = lane * 4; c < p.D; c += 128) {
                        float4 o = make_float4(0, 0, 0, 0);
                        for (int x = 0; x < sets; x++)
                            fma4(o, 1.0f, *reinterpret_cast<const float4 *>(red + (x * p.rows + r) * p.D + c));
                        write4(ch.b, head, c, o, inv);
                    }
            }
        }
        __syncthreads();
    }
}

__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

// Waits until at most n (1 .. kMaxStages - 1) groups of this thread's copies are on their way.
constexpr int kMaxStages = 6;
__device__ __forceinline__ void cp_wait_rt(int n) {
    switch (n) {
    case 1: cp_wait<1>(); break;
    case 2: cp_wait<2>(); break;
    case 3: cp_wait<3>(); break;
    case 4: cp_wait<4>(); break;
    default: cp_wait<5>(); break;
    }
}

// The same attention with one cluster of S CTAs per segment: a CTA has an S-th
// of the segment's tiles, W warps take every W-th of them.  No list, no
// workspace and no second pass over memory: the parts are joined in shared
// memory, then through distributed shared memory behind one cluster barrier.
template <typename C>
__global__ void __launch_bounds__(C::kWarpsMost * 32) paged_attention_cluster_kernel(const __grid_constant__ AttnParams p) {
    using T = typename C::T;
    using A = Acc<C, C::F16>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t vmask[kMaxWarps][kMaxStages];    // valid keys of the tile in each stage
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int kRing = p.stages * 2 * C::TILE_BYTES;   // bytes a warp
    uint8_t *my_ring = smem + (size_t)warp * kRing;
    const uint32_t ring = smem_u32(my_ring);
    uint8_t *q_rows = smem + (size_t)W * kRing;
    const int rank = blockIdx.x, S = gridDim.x, seg = blockIdx.y, b = blockIdx.z;
    const int h = p.row_tiles == 1 ? seg : seg / p.row_tiles, r0 = (seg - h * p.row_tiles) * C::ROWS;
    auto head_of = [&](int r) { return r0 + r < p.G ? h * p.G + r0 + r : -1; };

    pdl_wait();
    pdl_launch_dependents();
    const int given = p.lens[b], len = min(max(given, 0), p.cap);
    if (given != len && rank == 0 && seg == 0 && threadIdx.x == 0 && p.status)
        atomicOr(p.status, 2);
    const int tiles = (int)(((uint32_t)len + C::TK - 1) / C::TK);
    const int per = S == 1 ? tiles : (int)__umulhi((uint32_t)(tiles + S - 1), p.split_magic);   // ceil(tiles / S)
    const int end = min(tiles, (rank + 1) * per);
    T *out = (T *)p.out + b * p.o_bs;
    float *lse = p.lse ? p.lse + (int64_t)b * p.Hkv * p.G : nullptr;

    const int32_t *row = p.table + b * p.table_stride;
    const int64_t head_off = h * p.head_stride;
    int t = rank * per + warp, load = t;   // tile to compute, tile to issue
    Feed<C> feed(p, ring);
    auto issue = [&](int stage) {
        if (load < end) {
            const uint32_t valid = feed.tile(stage, head_off);
            if (lane == 0)
                vmask[warp][stage] = valid;
            load += W;
            if (load < end)
                feed.fetch(row, load * C::TK, min(C::TK, len - load * C::TK));
        }
        cp_commit();
    };
    if (load < end)
        feed.fetch(row, load * C::TK, min(C::TK, len - load * C::TK));
    for (int s = 0; s + 1 < p.stages; s++)
        issue(s);
    // the segment's query rows, for all warps
    for (int i = threadIdx.x; i < p.rows * C::NCH; i += blockDim.x) {
        const int r = i / C::NCH, ch = i % C::NCH, head = head_of(r);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (head >= 0 && ch * (16 / (int)sizeof(T)) < p.D)
            v = ldg_v4((const T *)p.q + b * p.q_bs + head * p.q_hs + ch * (16 / (int)sizeof(T)));
        *reinterpret_cast<uint4 *>(q_rows + C::at(r, ch)) = v;
    }
    __syncthreads();

    A acc;
    if (t < end) {
        const uint32_t qs = smem_u32(q_rows);
        acc.open(qs, qs, p.rows);
        int stage = 0;
        for (; t < end; t += W) {
            __syncwarp();   // every lane has read the stage that the last tile left: it takes the next one
            issue(stage == 0 ? p.stages - 1 : stage - 1);
            cp_wait_rt(p.stages - 1);
            __syncwarp();
            const uint32_t ks = ring + stage * 2 * C::TILE_BYTES;
            acc.tile(ks, ks + C::TILE_BYTES, qs, p.rows, vmask[warp][stage], p.scale * kLog2e);
            stage = stage + 1 == p.stages ? 0 : stage + 1;
        }
        acc.finish();
        __syncwarp();
        acc.to_slot(reinterpret_cast<float *>(my_ring), p.rows, p.D);
    }
    __syncthreads();

    // The CTA's warps joined: a warp per row and 128 outputs, lane i looks after warp i.
    const int chunks = (p.D + 127) >> 7, tasks = p.rows * chunks;
    const int parts = min(max(end - rank * per, 0), W);
    float *cta_part = reinterpret_cast<float *>(smem) + partial_floats(p.rows, p.D);   // in warp 0's ring, behind its part
    for (int task = warp; task < tasks; task += W) {
        const int r = chunks == 1 ? task : task >> 1, c = (chunks == 1 ? 0 : (task & 1) * 128) + lane * 4;
        const float *ml = reinterpret_cast<const float *>(smem + (size_t)lane * kRing) + p.rows * p.D + r;
        const float m = lane < parts ? ml[0] : -INFINITY;
        float l = lane < parts ? ml[p.rows] : 0.0f, M = m;
#pragma unroll
        for (int x = 16; x; x >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        const float w = ex2(m - (M == -INFINITY ? 0.0f : M));
        l *= w;
#pragma unroll
        for (int x = 16; x; x >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, x);
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int i = 0; i < parts; i++) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (c < p.D)
                fma4(o, wi, *reinterpret_cast<const float4 *>(smem + (size_t)i * kRing + (r * p.D + c) * 4));
        }
        if (S > 1) {
            if (c < p.D)
                *reinterpret_cast<float4 *>(cta_part + r * p.D + c) = o;
            if (c == 0) {
                cta_part[p.rows * p.D + r] = M;
                cta_part[p.rows * p.D + p.rows + r] = l;
            }
        } else {
            const int head = head_of(r);
            if (head >= 0) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                if (c < p.D) {
                    T *d = out + head * p.o_hs + c;
                    store2(d, o.x * inv, o.y * inv);
                    store2(d + 2, o.z * inv, o.w * inv);
                }
                if (c == 0 && lse)
                    lse[head] = lse_of(M, l * A::kSumScale);
            }
        }
    }
    if (S > 1) {
        cluster_sync();
        // the ranks joined, the same way; lane i looks after rank i
        const int used = per > 0 ? (tiles + per - 1) / per : 0;   // ranks with a tile
        const uint32_t mine = cluster_map(smem_u32(cta_part), lane < used ? lane : rank);
        for (int task = warp * S + rank; task < tasks; task += W * S) {
            const int r = chunks == 1 ? task : task >> 1, c = (chunks == 1 ? 0 : (task & 1) * 128) + lane * 4;
            const uint32_t ml = mine + (p.rows * p.D + r) * 4;
            const float m = lane < used ? ld_cluster(ml) : -INFINITY;
            float l = lane < used ? ld_cluster(ml + p.rows * 4) : 0.0f, M = m;
            float4 v[8];
            const uint32_t at = (r * p.D + (c < p.D ? c : 0)) * 4;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint32_t part = __shfl_sync(0xffffffffu, mine, i);
                v[i] = i < used ? ld_cluster4(part + at) : make_float4(0, 0, 0, 0);
            }
#pragma unroll
            for (int x = 16; x; x >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
            const float w = ex2(m - (M == -INFINITY ? 0.0f : M));
            l *= w;
#pragma unroll
            for (int x = 16; x; x >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, x);
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; i++)
                fma4(o, __shfl_sync(0xffffffffu, w, i), v[i]);
            for (int i = 8; i < used; i++)
                fma4(o, __shfl_sync(0xffffffffu, w, i), ld_cluster4(__shfl_sync(0xffffffffu, mine, i) + at));
            const int head = head_of(r);
            if (head >= 0) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                if (c < p.D) {
                    T *d = out + head * p.o_hs + c;
                    store2(d, o.x * inv, o.y * inv);
                    store2(d + 2, o.z * inv, o.w * inv);
                }
                if (c == 0 && lse)
                    lse[head] = lse_of(M, l * A::kSumScale);
            }
        }
        cluster_sync();   // no CTA leaves while another reads its part
    }
}

constexpr size_t kSmemMax = 227 * 1024 - 256;
constexpr size_t kSmemSm = 228 * 1024;

// Tuning hook: 0 = the rule in launch_cfg, 1 = always the list, 2 = always clusters.
int g_mode = 0, g_split = 0, g_warps = 0;

template <typename C>
int launch_cfg(AttnParams p, unsigned flags, cudaStream_t s) {
    static int caches[2][kMaxDevices] = {};
    const int segs = p.Hkv * p.row_tiles;
    p.one_page = p.page % C::TK == 0;
    p.whole = p.one_page && p.D == C::DP;
    p.page_shift = (p.page & (p.page - 1)) == 0 ? __builtin_ctz((unsigned)p.page) : -1;
    const int64_t most_tiles = (p.cap - 1) / C::TK + 1, tiles = most_tiles * p.B * segs;
    if (tiles > 0x7fffffff)
        return fail(MNB_ERR_SHAPE, "mnb_paged_attention: B=%d requests of up to %d tokens in %d heads are 2^31 tiles or more",
                    p.B, p.cap, segs);
    const size_t ring = (size_t)kWarps * (C::STAGES * 2 * C::TILE_BYTES + (C::F16 ? 0 : p.rows * C::ROW_BYTES));
    const size_t list = ring + (size_t)kWarps * partial_floats(p.rows, p.D) * 4 + (size_t)(p.B + 1) * 4;
    if (list > kSmemMax)
        return fail(MNB_ERR_UNSUPPORTED, "mnb_paged_attention: %zu bytes of shared memory needed", list);
    auto resident = [&](size_t smem) {
        const int fit = (int)(kSmemSm / (smem + 1024 + 512));
        return device_sm_count() * (fit < C::kCtas ? fit : C::kCtas);
    };

    // Clusters.
    const int64_t all = (int64_t)p.B * segs;
    const size_t per_warp = (size_t)C::TILE_BYTES * 2, q_bytes = (size_t)p.rows * C::ROW_BYTES;
    int split = (int)(resident(kWarps * 2 * per_warp + q_bytes) / all < 8 ? resident(kWarps * 2 * per_warp + q_bytes) / all : 8);
    const int64_t by_tiles = (most_tiles - 1) / kWarps + 1;
    split = split < by_tiles ? split : (int)by_tiles;
    split = g_split ? g_split : split < 1 ? 1 : split;
    int warps = g_warps ? g_warps : kWarps;
    const int fit_warps = (int)((kSmemMax - q_bytes) / (2 * per_warp));
    warps = warps < fit_warps ? warps : fit_warps;
    warps = warps < C::kWarpsMost ? warps : C::kWarpsMost;
    p.split_magic = split > 1 ? (uint32_t)((((uint64_t)1 << 32) + split - 1) / split) : 0;
    const int64_t warp_tiles = (most_tiles - 1) / (warps * split) + 1;
    const bool clusters = g_mode == 2 || (g_mode == 0 && warp_tiles <= kClusterTiles);

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    if (clusters) {
        // a deeper ring where the SMs have room for one
        const int64_t ctas = all * split, sms = device_sm_count();
        const int most_ctas = kMaxWarps / warps;
        const int per_sm = ctas > sms * (most_ctas - 1) ? most_ctas : (int)((ctas - 1) / sms) + 1;
        const size_t room = kSmemSm / per_sm - 1024 - 1024;
        const size_t fit = ((room < kSmemMax ? room : kSmemMax) - q_bytes) / (warps * per_warp);
        p.stages = fit < 2 ? 2 : fit > kMaxStages ? kMaxStages : (int)fit;
        cfg.blockDim = dim3((unsigned)warps * 32);
        cfg.gridDim = dim3((unsigned)split, (unsigned)segs, (unsigned)p.B);
        cfg.dynamicSmemBytes = p.stages * warps * per_warp + q_bytes;
        if (split > 1) {
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)split;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.numAttrs = 1;
        }
    } else {
        // CTAs worth the table's width; the last join keeps a float per row and part, and an output row per warp,
        // in the rings
        const int64_t want = (tiles - 1) / p.min_tiles + 1;
        const int joinable = (kWarps * (C::STAGES * 2 * C::TILE_BYTES - p.D * 4) - 32) / (4 * p.rows) - kWarps;
        int grid = resident(list);
        grid = grid < joinable ? grid : joinable;
        cfg.gridDim = dim3((unsigned)(want < grid ? want : grid));
        cfg.dynamicSmemBytes = list;
    }
    if (flags & MNB_FLAG_PDL) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    auto *kernel = clusters ? paged_attention_cluster_kernel<C> : paged_attention_kernel<C>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)cfg.dynamicSmemBytes, caches[clusters]);
    if (e == cudaSuccess && clusters && split > 8)
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess)
        return fail(MNB_ERR_CUDA, "mnb_paged_attention: launch: %s", cudaGetErrorString(e));
    return MNB_OK;
}

template <typename T, int DP, int ROWS>
int launch_rows(const AttnParams &p, unsigned flags, cudaStream_t s) {
    return launch_cfg<Cfg<T, DP, ROWS>>(p, flags, s);
}

template <typename T, int DP>
int launch_dp(const AttnParams &p, unsigned flags, cudaStream_t s) {
    if constexpr (std::is_same<T, half>::value)
        return p.rows > 8 ? launch_rows<T, DP, 16>(p, flags, s) : launch_rows<T, DP, 8>(p, flags, s);
    else
        return p.rows > 4   ? launch_rows<T, DP, 8>(p, flags, s)
               : p.rows > 2 ? launch_rows<T, DP, 4>(p, flags, s)
               : p.rows > 1 ? launch_rows<T, DP, 2>(p, flags, s)
                            : launch_rows<T, DP, 1>(p, flags, s);
}

int rows_per_segment(int G, int f16) { return G < (f16 ? 16 : 8) ? G : (f16 ? 16 : 8); }
int grid_of() { return device_sm_count() * kMaxCtas; }
size_t counters_bytes() { return ((size_t)grid_of() * 4 + 127) / 128 * 128; }

}  // namespace

int set_paged_attention_mode(int mode, int split, int warps) {
    if (mode < 0 || mode > 2 || split < 0 || split > 16 || warps < 0 || warps > kMaxWarps)
        return MNB_ERR_INVALID_ARG;
    g_mode = mode, g_split = split, g_warps = warps;
    return MNB_OK;
}

size_t paged_attention_workspace_bytes(int Hq, int Hkv, int D, int f16) {
    return counters_bytes() + (size_t)grid_of() * 2 * partial_floats(rows_per_segment(Hq / Hkv, f16), D) * 4;
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
    p.B = B, p.Hkv = (int)c->num_heads, p.G = Hq / p.Hkv, p.D = (int)c->head_dim;
    p.rows = rows_per_segment(p.G, f16);
    p.row_tiles = (p.G + p.rows - 1) / p.rows;
    p.page = (int)c->page_size, p.num_pages = (int)c->num_pages, p.cap = max_blocks * p.page, p.scale = scale;
    p.min_tiles = kWarps;
    p.join_cost = (float)(p.rows * (p.D + 2) * 4) / (2 * (f16 ? 16 * 2 : 8 * 4) * p.D);   // bytes over bytes
    p.counters = (int *)workspace;
    p.partials = (float *)((uint8_t *)workspace + counters_bytes());
    if (f16)
        return p.D <= 64    ? launch_dp<half, 64>(p, flags, s)
               : p.D <= 128 ? launch_dp<half, 128>(p, flags, s)
                            : launch_dp<half, 256>(p, flags, s);
    return p.D <= 64    ? launch_dp<float, 64>(p, flags, s)
           : p.D <= 128 ? launch_dp<float, 128>(p, flags, s)
                        : launch_dp<float, 256>(p, flags, s);
}

}  // namespace mnb

extern "C" MNB_API int mnb_tune_paged_attention(int mode, int split, int warps) {
    return mnb::set_paged_attention_mode(mode, split, warps);
}
