// paged.cu -- bookkeeping and writes of a paged key-value cache: block tables,
// slots and positions of a step's new tokens (mnb_paged_tables), and the
// RMS norm + rotary embedding + append of those tokens (mnb_rope_append).
#include "common.cuh"
#include "internal.h"

namespace mnb {
namespace {

// ------------------------------------------------------------- paged tables

constexpr uint32_t kRefused = 0x80000000u;   // a request's page offset: it was granted nothing

// Sum of counts that stops at 2^31 - 1 (associative for operands below 2^31).
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// Inclusive saturating scan over the CTA; `total` gets the CTA's sum.  Two
// barriers; `warp_sums` must not be reused before the next barrier.
template <int NT>
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
    for (int w = 0; w < NT / 32; w++) {
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
template <int NT>
__global__ void __launch_bounds__(NT) paged_tables_kernel(const __grid_constant__ TabParams p) {
    extern __shared__ uint32_t sh[];
    uint32_t *cu = sh;                    // [B + 1] tokens before request b
    uint32_t *pg = sh + p.B + 1;          // [B] pages taken before request b, kRefused when it gets none
    __shared__ uint32_t warp_sums[NT / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int start = *p.free_start;
    const uint32_t avail = (start >= 0 && start <= p.num_free) ? (uint32_t)(p.num_free - start) : 0u;
    int bad = (start < 0 || start > p.num_free) ? 4 : 0;
    uint32_t tok0 = 0, pg0 = 0, granted = 0;
    for (int b0 = 0; b0 < p.B; b0 += NT) {
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
        const uint32_t incl = sat_add(block_scan<NT>(cnt, warp_sums, tot), tok0);
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
        const uint32_t pincl = sat_add(block_scan<NT>((uint32_t)need, warp_sums, tot), pg0);
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
            for (int w = 1; w < NT / 32; w++)
                granted = max(granted, warp_sums[w]);
            *p.free_next = start + (int)granted;
            p.cu[0] = 0;
        }
        if (bad && p.status)
            atomicOr(p.status, bad);
    }
    // requests: one warp each
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (NT / 32);
    for (int b = blockIdx.x * (NT / 32) + (threadIdx.x >> 5); b < p.B; b += warps) {
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
    for (int64_t t64 = (int64_t)blockIdx.x * NT + threadIdx.x; t64 < p.T;
         t64 += (int64_t)gridDim.x * NT) {
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
    uint32_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;   // token and head strides, elements (at most 2^31)
    uint32_t page_stride, slot_stride, head_stride;
    int64_t T;
    int Hq, Hkv, D, R, page, num_pos, num_slots;
    int lph, gpt, tpc;   // lanes a head, groups a token, tokens a CTA
    float eps, inv_D;
    Div by_page, by_gpt;
};

// V neighbouring entries in fp32 (V = 4, or 8 of fp16: 16-byte accesses but for 4 of fp16).
template <int V>
__device__ __forceinline__ void load_v(const float *p, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + i);
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
}
// The same as they lie in memory (16 bytes, or 8 for four of fp16), and their fp32 values.
template <typename T, int V>
struct Raw {
    uint32_t u[V * (int)sizeof(T) / 4];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(u) == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            u[0] = v.x, u[1] = v.y;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (sizeof(u) == 16)
            *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(u) / 4); i++)
            u[i] = 0;
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(u) / 4); i++)
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(u[i]);
            } else {
                const float2 f = __half22float2(u32_as_h2(u[i]));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            }
    }
};
template <int V>
__device__ __forceinline__ void store_v(float *p, const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int V>
__device__ __forceinline__ void store_v(half *p, const float (&x)[V]) {
    uint32_t u[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; i++)
        u[i] = h2_as_u32(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
}

// n x stride in 64 bits, one instruction.
__device__ __forceinline__ int64_t wide(int n, uint32_t stride) { return (int64_t)((uint64_t)(uint32_t)n * stride); }

constexpr int kAppendThreads = 256;

// A group of `lph` lanes (a power of two, up to a warp) per head, 2 V entries a
// lane: a rotary lane holds V entries of the first half and their V partners of
// the second, so norm, rotation and store stay in registers; one rounding, at the
// store.  A token's heads are spread over `gpt` groups of one CTA, so its slot,
// position, cosines and sines are loaded once for the heads that a group takes.
// Bound by the chain slot / position -> cosines -> store for few tokens (2.5 us for
// one), by instruction issue and DRAM for many (8191 fp32 tokens: 5200 GB/s, 8000
// fp16 tokens: 4000 GB/s).
template <typename T, int V>
__global__ void __launch_bounds__(kAppendThreads, V == 8 ? 4 : 6) rope_append_kernel(const __grid_constant__ AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int l = threadIdx.x & (p.lph - 1), group = threadIdx.x / p.lph;
    const unsigned mask = (p.lph == 32 ? 0xffffffffu : (1u << p.lph) - 1) << (threadIdx.x & 31 & ~(p.lph - 1));
    const int tok = quotient(group, p.by_gpt), h0 = group - tok * p.gpt;
    const int t = blockIdx.x * p.tpc + tok;   // below 2^30 + 256
    if (tok >= p.tpc || t >= p.T)
        return;
    const int heads = p.Hq + 2 * p.Hkv;
    const bool live = l * 2 * V < p.D, rot = l * 2 * V < p.R;
    const int e0 = rot ? V * l : 2 * V * l, e1 = rot ? p.R / 2 + V * l : 2 * V * l + V;
    // What no other load decides on is requested first: slot, position and the first head.
    const int slot = p.slots[t];
    const int pos = p.R > 0 ? p.pos[t] : 0;
    Raw<T, V> ra, rb;   // of the next head to work on
    auto load = [&](int i) {
        const bool q = i < p.Hq, k = i < p.Hq + p.Hkv;
        const uint32_t ts = q ? p.q_ts : k ? p.k_ts : p.v_ts, hs = q ? p.q_hs : k ? p.k_hs : p.v_hs;
        const T *src = (const T *)(q ? p.q : k ? p.k : p.v) + wide(t, ts) + wide(q ? i : k ? i - p.Hq : i - p.Hq - p.Hkv, hs);
        if (live)
            ra.load(src + e0), rb.load(src + e1);
        else
            ra.zero(), rb.zero();
    };
    load(h0);
    const bool pos_ok = p.R == 0 || (pos >= 0 && pos < p.num_pos);
    float c[V], s[V];
    if (rot && pos_ok) {
        load_v<V>(p.cos + (int64_t)pos * (p.R / 2) + V * l, c);
        load_v<V>(p.sin + (int64_t)pos * (p.R / 2) + V * l, s);
    }
    const bool slot_ok = slot >= 0 && slot < p.num_slots && pos_ok;
    if (h0 == 0 && l == 0 && p.status && (slot < -1 || slot >= p.num_slots || !pos_ok))
        atomicOr(p.status, 1);
    int64_t cache_at = 0;
    if (slot_ok) {
        const int page = quotient(slot, p.by_page);
        cache_at = wide(page, p.page_stride) + wide(slot - page * p.page, p.slot_stride);
    }
    for (int i = h0;;) {
        const int kind = i < p.Hq ? 0 : i < p.Hq + p.Hkv ? 1 : 2;   // q, k, v
        const int h = kind == 0 ? i : kind == 1 ? i - p.Hq : i - p.Hq - p.Hkv;
        T *dst = kind == 0 ? (T *)p.q_out + wide(t, p.o_ts) + wide(h, p.o_hs)
                           : (T *)(kind == 1 ? p.k_cache : p.v_cache) + cache_at + wide(h, p.head_stride);
        if (kind == 2) {   // as it is
            if (live && slot_ok)
                ra.store(dst + e0), rb.store(dst + e1);
            if ((i += p.gpt) >= heads)
                return;
            load(i);
            continue;
        }
        const float *w = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
        float a[V], b[V];
        ra.get(a), rb.get(b);
        if (w) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < V; j++)
                ss += a[j] * a[j] + b[j] * b[j];
            for (int o = p.lph / 2; o; o >>= 1)
                ss += __shfl_xor_sync(mask, ss, o);
            const float r = rsqrtf(fmaf(ss, p.inv_D, p.eps));
            if (live) {
                float x[V], y[V];
                load_v<V>(w + e0, x);
                load_v<V>(w + e1, y);
#pragma unroll
                for (int j = 0; j < V; j++)
                    a[j] = a[j] * r * x[j], b[j] = b[j] * r * y[j];
            }
        }
        if (rot && pos_ok) {
#pragma unroll
            for (int j = 0; j < V; j++) {
                const float x = a[j], y = b[j];
                a[j] = x * c[j] - y * s[j];
                b[j] = y * c[j] + x * s[j];
            }
        }
        if (!pos_ok) {   // a zero q row; k and v are dropped
#pragma unroll
            for (int j = 0; j < V; j++)
                a[j] = b[j] = 0.0f;
        }
        if (live && (kind == 0 || slot_ok)) {
            store_v<V>(dst + e0, a);
            store_v<V>(dst + e1, b);
        }
        i += p.gpt;
        if (i >= heads)
            return;
        load(i);
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

template <typename T, int V>
int launch_append(AppendParams p, unsigned flags, cudaStream_t s) {
    const int heads = p.Hq + 2 * p.Hkv, units = (p.D + 2 * V - 1) / (2 * V);
    p.lph = 1;
    while (p.lph < units)
        p.lph *= 2;
    const int groups = kAppendThreads / p.lph;
    // With tokens for every SM a group takes two heads of 16-byte pairs, or three of
    // 8-byte (fp16) or fp32 ones: what the lanes work out per token is then shared
    // (1024 fp16 tokens: 7.0 us, 7.9 with one head; 8191 fp32 tokens: 28 us, 30).
    const int rounds = max((heads + groups - 1) / groups, p.T < 2 * device_sm_count() ? 1 : V == 8 ? 2 : 3);
    p.gpt = (heads + rounds - 1) / rounds;   // as many heads a group for all groups, or one fewer
    p.by_gpt = div_by((uint32_t)p.gpt);
    p.tpc = groups / p.gpt;
    if (p.T < p.tpc)
        p.tpc = (int)p.T;
    const int threads = (p.tpc * p.gpt * p.lph + 31) / 32 * 32;
    return launch("mnb_rope_append", rope_append_kernel<T, V>, p, (int)((p.T + p.tpc - 1) / p.tpc), threads, 0, flags, s);
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
    // a short barrier for a decode step's few requests, wide scans for many
    const int nt = B <= 128 && T <= 1024 ? 128 : 512;
    const int by_tokens = (T + nt - 1) / nt, by_rows = (B + nt / 32 - 1) / (nt / 32);
    int grid = by_tokens > by_rows ? by_tokens : by_rows;
    const int most = device_sm_count() * 2;
    grid = grid < 1 ? 1 : grid > most ? most : grid;
    return launch("mnb_paged_tables", nt == 128 ? paged_tables_kernel<128> : paged_tables_kernel<512>, p, grid, nt,
                  (size_t)(2 * B + 1) * 4, flags, s);
}

int launch_rope_append(const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs,
                       const void *v, int64_t v_ts, int64_t v_hs, const mnb_paged_cache *c, const int32_t *slots,
                       const int32_t *pos, int64_t T, int Hq, const float *cos, const float *sin, int R, int num_pos,
                       const float *qw, const float *kw, float eps, void *q_out, int64_t o_ts, int64_t o_hs,
                       int *status, unsigned flags, cudaStream_t s) {
    AppendParams p;
    p.q = q, p.k = k, p.v = v, p.q_out = q_out, p.k_cache = c->k, p.v_cache = c->v;
    p.slots = slots, p.pos = pos, p.cos = cos, p.sin = sin, p.qw = qw, p.kw = kw, p.status = status;
    p.q_ts = (uint32_t)q_ts, p.q_hs = (uint32_t)q_hs, p.k_ts = (uint32_t)k_ts, p.k_hs = (uint32_t)k_hs;
    p.v_ts = (uint32_t)v_ts, p.v_hs = (uint32_t)v_hs, p.o_ts = (uint32_t)o_ts, p.o_hs = (uint32_t)o_hs;
    p.page_stride = (uint32_t)c->page_stride, p.slot_stride = (uint32_t)c->slot_stride;
    p.head_stride = (uint32_t)c->head_stride;
    p.T = T;
    p.Hq = Hq, p.Hkv = (int)c->num_heads, p.D = (int)c->head_dim, p.R = R, p.page = (int)c->page_size;
    p.inv_D = 1.0f / (float)p.D, p.by_page = div_by((uint32_t)c->page_size);
    p.num_pos = num_pos, p.num_slots = (int)(c->num_pages * c->page_size), p.eps = eps;
    if (c->dtype == MNB_F32)
        return launch_append<float, 4>(p, flags, s);
    return p.D % 16 == 0 && R % 16 == 0 ? launch_append<half, 8>(p, flags, s) : launch_append<half, 4>(p, flags, s);
}

}  // namespace mnb
