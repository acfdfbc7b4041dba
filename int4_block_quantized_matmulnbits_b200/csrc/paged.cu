// paged.cu -- bookkeeping and writes of a paged key-value cache: block tables,
// slots and positions of a step's new tokens (mnb_paged_tables), and the
// RMS norm + rotary embedding + append of those tokens (mnb_rope_append).
#include "common.cuh"
#include "internal.h"

namespace mnb {
namespace {

// ------------------------------------------------------------- paged tables

constexpr int kTabThreads = 512;
constexpr uint32_t kRefused = 0x80000000u;   // a request's page offset: it was granted nothing

// Sum of counts that stops at 2^31 - 1 (associative for operands below 2^31).
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// Inclusive saturating scan over the CTA; `total` gets the CTA's sum.  Two
// barriers; `warp_sums` must not be reused before the next barrier.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v = sat_add(v, u);
    }
    __syncthreads();   // the sums of an earlier scan have been read
    if (lane == 31)
        warp_sums[warp] = v;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; w++) {
        const uint32_t s = warp_sums[w];
        if (w < warp)
            before = sat_add(before, s);
        total = sat_add(total, s);
    }
    return sat_add(v, before);
}

struct TabParams {
    const int32_t *ctx, *neu, *free_pages, *free_start;
    int32_t *table, *seq, *cu, *slots, *pos, *free_next;
    int *status;
    int64_t table_stride;
    int B, page, max_blocks, T, num_free, num_pages;
};

__device__ __forceinline__ int blocks_of(int64_t tokens, int page) { return (int)((tokens + page - 1) / page); }

// Every CTA scans all B requests (B <= 4096: two scans of one integer each, in
// shared memory), so no CTA waits for another; requests and tokens are then
// spread over the grid.  A new token's page is found in shared memory too: its
// request by binary search over the token offsets, its page in the block table
// if the request held it before the call and in the free list otherwise, so
// nothing that this launch writes is read back.  Bound by latency: the lengths'
// load, the scans and the page's load follow one another.
__global__ void __launch_bounds__(kTabThreads) paged_tables_kernel(const __grid_constant__ TabParams p) {
    extern __shared__ uint32_t sh[];
    uint32_t *cu = sh;                    // [B + 1] tokens before request b
    uint32_t *pg = sh + p.B + 1;          // [B] pages taken before request b, kRefused when it gets none
    __shared__ uint32_t warp_sums[kTabThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int start = *p.free_start;
    const uint32_t avail = (start >= 0 && start <= p.num_free) ? (uint32_t)(p.num_free - start) : 0u;
    int bad = (start < 0 || start > p.num_free) ? 4 : 0;
    uint32_t tok0 = 0, pg0 = 0, granted = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTabThreads) {
        const int b = b0 + (int)threadIdx.x;
        int c = 0, n = 0, need = 0;
        bool ok = true;
        if (b < p.B) {
            c = p.ctx[b];
            n = p.neu[b];
            ok = c >= 0 && n >= 0;
        }
        const uint32_t cnt = n > 0 ? (uint32_t)n : 0u;
        uint32_t tot;
        const uint32_t incl = sat_add(block_scan(cnt, warp_sums, tot), tok0);
        tok0 = sat_add(tok0, tot);
        if (b < p.B) {
            cu[b + 1] = incl;
            const int64_t len = (int64_t)c + n;
            ok = ok && incl <= (uint32_t)p.T && len <= (int64_t)p.max_blocks * p.page;
            if (!ok)
                bad |= 2;
            else
                need = blocks_of(len, p.page) - blocks_of(c, p.page);
        }
        const uint32_t pincl = sat_add(block_scan((uint32_t)need, warp_sums, tot), pg0);
        pg0 = sat_add(pg0, tot);
        if (b < p.B) {
            // the list runs out at one request; a later one passes only if it needs no page
            const bool fits = need == 0 || pincl <= avail;
            if (!fits)
                bad |= 4;
            pg[b] = ok && fits ? pincl - (uint32_t)need : kRefused;
            if (fits && need > 0)
                granted = max(granted, pincl);
        }
    }
    if (threadIdx.x == 0)
        cu[0] = 0;
    __syncthreads();
    const uint32_t total = cu[p.B];
    // free_next: the largest granted offset over the CTA (granted prefixes grow with b)
    if (blockIdx.x == 0) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            granted = max(granted, __shfl_xor_sync(0xffffffffu, granted, o));
        if ((threadIdx.x & 31) == 0)
            warp_sums[threadIdx.x >> 5] = granted;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kTabThreads / 32; w++)
                granted = max(granted, warp_sums[w]);
            *p.free_next = start + (int)granted;
            p.cu[0] = 0;
        }
        if (bad && p.status)
            atomicOr(p.status, bad);
    }
    // requests: one warp each
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kTabThreads / 32);
    for (int b = blockIdx.x * (kTabThreads / 32) + (threadIdx.x >> 5); b < p.B; b += warps) {
        const int c = max(p.ctx[b], 0), n = max(p.neu[b], 0);
        const uint32_t first = pg[b];
        const bool ok = first != kRefused;
        if (lane == 0) {
            p.seq[b] = ok ? c + n : c;
            p.cu[b + 1] = (int)cu[b + 1];
        }
        if (ok) {
            const int had = blocks_of(c, p.page), need = blocks_of((int64_t)c + n, p.page) - had;
            for (int j = lane; j < need; j += 32)
                p.table[b * p.table_stride + had + j] = p.free_pages[start + first + j];
        }
    }
    // tokens: one thread each
    for (int64_t t64 = (int64_t)blockIdx.x * kTabThreads + threadIdx.x; t64 < p.T;
         t64 += (int64_t)gridDim.x * kTabThreads) {
        const uint32_t t = (uint32_t)t64;
        int slot = -1, pos = 0;
        if (t < total) {
            int lo = 0, hi = p.B - 1;   // the request with cu[b] <= t < cu[b + 1]
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid + 1] > t)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            const uint32_t first = pg[lo];
            if (first != kRefused) {
                const int c = p.ctx[lo];
                pos = c + (int)(t - cu[lo]);
                const int blk = pos / p.page, had = blocks_of(c, p.page);
                const int page = blk < had ? p.table[lo * p.table_stride + blk] : p.free_pages[start + first + (blk - had)];
                if (page >= 0 && page < p.num_pages)
                    slot = page * p.page + (pos - blk * p.page);
                else if (p.status)
                    atomicOr(p.status, 1);
            }
        }
        p.slots[t] = slot;
        p.pos[t] = pos;
    }
}

// ---------------------------------------------------------- norm, rotary, append

struct AppendParams {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    const int32_t *slots, *pos;
    const float *cos, *sin, *qw, *kw;
    int *status;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;   // token and head strides, elements
    int64_t page_stride, slot_stride, head_stride;
    int64_t items;                                            // T * (Hq + 2 Hkv)
    int Hq, Hkv, D, R, page, num_pos, num_slots;
    float eps;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4(const half *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(u32_as_h2(u.x)), b = __half22float2(u32_as_h2(u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(half *p, float4 v) {
    uint2 u;
    u.x = h2_as_u32(__floats2half2_rn(v.x, v.y));
    u.y = h2_as_u32(__floats2half2_rn(v.z, v.w));
    *reinterpret_cast<uint2 *>(p) = u;
}

__device__ __forceinline__ float dot4(float4 a) { return a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w; }
__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }
__device__ __forceinline__ float4 mul4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }

// One group of LPH lanes per (token, head), eight entries a lane: a rotary lane
// holds four entries of the first half and their four partners of the second,
// so norm, rotation and store stay in registers.  One rounding, at the store.
template <typename T, int LPH>
__global__ void __launch_bounds__(256) rope_append_kernel(const __grid_constant__ AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int l = threadIdx.x % LPH;
    const unsigned mask = LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1) << ((threadIdx.x & 31) / LPH * LPH);
    const int heads = p.Hq + 2 * p.Hkv;
    const int64_t step = (int64_t)gridDim.x * (256 / LPH);
    const bool live = l * 8 < p.D;
    const bool rot = l * 8 < p.R;
    const int e0 = rot ? 4 * l : 8 * l, e1 = rot ? p.R / 2 + 4 * l : 8 * l + 4;
    for (int64_t i = (int64_t)blockIdx.x * (256 / LPH) + threadIdx.x / LPH; i < p.items; i += step) {
        const int64_t t = i / heads;
        int h = (int)(i - t * heads);
        const T *src;
        T *dst = nullptr;
        const float *w = nullptr;
        bool turn = p.R > 0;
        const int slot = p.slots[t];
        const int pos = p.R > 0 ? p.pos[t] : 0;
        const bool pos_ok = p.R == 0 || (pos >= 0 && pos < p.num_pos);
        if (h < p.Hq) {
            src = (const T *)p.q + t * p.q_ts + h * p.q_hs;
            dst = (T *)p.q_out + t * p.o_ts + h * p.o_hs;
            w = p.qw;
        } else {
            h -= p.Hq;
            const bool is_v = h >= p.Hkv;
            if (is_v)
                h -= p.Hkv;
            src = is_v ? (const T *)p.v + t * p.v_ts + h * p.v_hs : (const T *)p.k + t * p.k_ts + h * p.k_hs;
            w = is_v ? nullptr : p.kw;
            turn = turn && !is_v;
            if (slot >= 0 && slot < p.num_slots && pos_ok) {
                const int page = slot / p.page;
                dst = (T *)(is_v ? p.v_cache : p.k_cache) + page * p.page_stride +
                      (int64_t)(slot - page * p.page) * p.slot_stride + h * p.head_stride;
            }
            if (l == 0 && p.status && (slot < -1 || slot >= p.num_slots || !pos_ok))
                atomicOr(p.status, 1);
        }
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (live) {
            a = load4(src + e0);
            b = load4(src + e1);
        }
        if (w) {
            float ss = dot4(a) + dot4(b);
#pragma unroll
            for (int o = LPH / 2; o; o >>= 1)
                ss += __shfl_xor_sync(mask, ss, o);
            const float r = 1.0f / sqrtf(ss / (float)p.D + p.eps);
            if (live) {
                a = mul4(mul4(a, r), load4(w + e0));
                b = mul4(mul4(b, r), load4(w + e1));
            }
        }
        if (!dst || !live)
            continue;
        if (turn && rot) {
            if (pos_ok) {
                const float4 c = load4(p.cos + (int64_t)pos * (p.R / 2) + 4 * l);
                const float4 s = load4(p.sin + (int64_t)pos * (p.R / 2) + 4 * l);
                const float4 x = a, y = b;
                a = make_float4(x.x * c.x - y.x * s.x, x.y * c.y - y.y * s.y, x.z * c.z - y.z * s.z,
                                x.w * c.w - y.w * s.w);
                b = make_float4(y.x * c.x + x.x * s.x, y.y * c.y + x.y * s.y, y.z * c.z + x.z * s.z,
                                y.w * c.w + x.w * s.w);
            }
        }
        if (!pos_ok)
            a = b = make_float4(0, 0, 0, 0);   // only a q row: a k or v row has no dst then
        store4(dst + e0, a);
        store4(dst + e1, b);
    }
}

template <typename P>
int launch(const char *fn, void (*kernel)(P), const P &p, int grid, int threads, size_t smem, unsigned flags,
           cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (flags & MNB_FLAG_PDL) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
        cfg.attrs = attr;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess)
        return fail(MNB_ERR_CUDA, "%s: launch: %s", fn, cudaGetErrorString(e));
    return MNB_OK;
}

template <typename T>
int launch_append(const AppendParams &p, unsigned flags, cudaStream_t s) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    const int64_t ctas = (p.items * lanes + 255) / 256;
    const int grid = (int)(ctas < device_sm_count() * 64 ? ctas : device_sm_count() * 64);
    auto *k = lanes == 8 ? rope_append_kernel<T, 8> : lanes == 16 ? rope_append_kernel<T, 16> : rope_append_kernel<T, 32>;
    return launch("mnb_rope_append", k, p, grid, 256, 0, flags, s);
}

}  // namespace

int launch_paged_tables(const int32_t *ctx, const int32_t *neu, int B, int page, int num_pages,
                        const int32_t *free_pages, int num_free, const int32_t *free_start, int32_t *table,
                        int64_t table_stride, int max_blocks, int32_t *seq, int32_t *cu, int32_t *slots, int32_t *pos,
                        int T, int32_t *free_next, int *status, unsigned flags, cudaStream_t s) {
    TabParams p;
    p.ctx = ctx, p.neu = neu, p.free_pages = free_pages, p.free_start = free_start;
    p.table = table, p.seq = seq, p.cu = cu, p.slots = slots, p.pos = pos, p.free_next = free_next;
    p.status = status, p.table_stride = table_stride;
    p.B = B, p.page = page, p.max_blocks = max_blocks, p.T = T, p.num_free = num_free, p.num_pages = num_pages;
    const int by_tokens = (T + kTabThreads - 1) / kTabThreads, by_rows = (B + kTabThreads / 32 - 1) / (kTabThreads / 32);
    int grid = by_tokens > by_rows ? by_tokens : by_rows;
    const int most = device_sm_count() * 2;
    grid = grid < 1 ? 1 : grid > most ? most : grid;
    return launch("mnb_paged_tables", paged_tables_kernel, p, grid, kTabThreads, (size_t)(2 * B + 1) * 4, flags, s);
}

int launch_rope_append(const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs,
                       const void *v, int64_t v_ts, int64_t v_hs, const mnb_paged_cache *c, const int32_t *slots,
                       const int32_t *pos, int64_t T, int Hq, const float *cos, const float *sin, int R, int num_pos,
                       const float *qw, const float *kw, float eps, void *q_out, int64_t o_ts, int64_t o_hs,
                       int *status, unsigned flags, cudaStream_t s) {
    AppendParams p;
    p.q = q, p.k = k, p.v = v, p.q_out = q_out, p.k_cache = c->k, p.v_cache = c->v;
    p.slots = slots, p.pos = pos, p.cos = cos, p.sin = sin, p.qw = qw, p.kw = kw, p.status = status;
    p.q_ts = q_ts, p.q_hs = q_hs, p.k_ts = k_ts, p.k_hs = k_hs, p.v_ts = v_ts, p.v_hs = v_hs, p.o_ts = o_ts, p.o_hs = o_hs;
    p.page_stride = c->page_stride, p.slot_stride = c->slot_stride, p.head_stride = c->head_stride;
    p.items = T * (Hq + 2 * c->num_heads);
    p.Hq = Hq, p.Hkv = (int)c->num_heads, p.D = (int)c->head_dim, p.R = R, p.page = (int)c->page_size;
    p.num_pos = num_pos, p.num_slots = (int)(c->num_pages * c->page_size), p.eps = eps;
    return c->dtype == MNB_F16 ? launch_append<half>(p, flags, s) : launch_append<float>(p, flags, s);
}

}  // namespace mnb
