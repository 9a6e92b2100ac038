// kvcache.cu -- the paged NVFP4 cache: a step's block tables and slots (nvfp4_kv_plan), and new
// keys and values quantized into it (nvfp4_kv_append).
#include <cuda_bf16.h>

#include "kvcache.cuh"

namespace nvq {

// ------------------------------------------------------------------ checks of a cache
nvq_status check_cache(const nvq_kv_cache* c, const char* who)
{
    NVQ_CHECK_ARG(c && c->k_codes && c->k_sf && c->v_codes && c->v_sf && c->k_tscale && c->v_tscale, NVQ_ERR_ARG,
                  "%s: null cache or cache pointer", who);
    NVQ_CHECK_ARG(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, NVQ_ERR_SHAPE,
                  "%s: head_dim %d is not 64, 128 or 256", who, (int)c->head_dim);
    NVQ_CHECK_ARG(c->page_size >= 16 && c->page_size <= 65536 && c->page_size % 16 == 0, NVQ_ERR_SHAPE,
                  "%s: page_size %d is not a multiple of 16 in [16, 65536]", who, (int)c->page_size);
    NVQ_CHECK_ARG(c->pages >= 1 && c->pages < (1ll << 31) && c->pages * c->page_size < (1ll << 31) && c->kv_heads >= 1 &&
                      c->kv_heads <= 1024,
                  NVQ_ERR_SHAPE, "%s: pages * page_size outside [1, 2^31) or kv_heads outside [1, 1024]", who);
    const int64_t code_rows = (int64_t)c->page_size * (c->head_dim / 2), sf_rows = (int64_t)c->page_size * (c->head_dim / 16);
    NVQ_CHECK_ARG((c->head_stride >= code_rows || c->kv_heads == 1) && (c->page_stride >= code_rows || c->pages == 1) &&
                      (c->sf_head_stride >= sf_rows || c->kv_heads == 1) && (c->sf_page_stride >= sf_rows || c->pages == 1),
                  NVQ_ERR_SHAPE, "%s: a stride shorter than a page's rows", who);
    NVQ_CHECK_ARG(c->head_stride % 16 == 0 && c->page_stride % 16 == 0 && c->sf_head_stride % 16 == 0 &&
                      c->sf_page_stride % 16 == 0 && aligned(c->k_codes, 16) && aligned(c->k_sf, 16) &&
                      aligned(c->v_codes, 16) && aligned(c->v_sf, 16) && aligned(c->k_tscale, 4) && aligned(c->v_tscale, 4),
                  NVQ_ERR_ALIGN, "%s: cache pointers and strides must be multiples of 16 bytes", who);
    return NVQ_OK;
}

// ------------------------------------------------------------------ plan
// One launch.  Every CTA owns kPlanTokens consecutive entries of the slot list and scans all
// requests by itself (two sums: new tokens and new pages), so no CTA waits for another: a request
// costs 8 bytes that L2 serves, a second launch would cost more than the scan of a batch.  Each
// request that has a token in the CTA's range marks its first one; a maximum-scan over the range
// then tells every token its request.  A new page's table entry is written by the thread of the
// page's first token (that token is in the step: the page was not there before).
// kPlanTokens is 512, a token a thread, while that is a block an SM at most, else 2048, as each block
// pays for the scan: 4096 decoding requests 6.0 us with 512 and 9.7 with 2048, with prompts among them
// (211k tokens) 11.9 and 8.2.  512 threads: 4096 requests took 9.2 us with 256 and 9.0 with 1024, where
// these took 7.3.  Measured: 256 decoding requests in 3.7 us, bound by the launch and two loads' latencies.
constexpr int kPlanThreads = 512;

struct PlanArgs {
    const int32_t* new_tokens;
    const int32_t* kv_len;
    int32_t B;
    FastDiv page;
    int32_t* table;
    int64_t ld_table;
    int32_t max_blocks;
    const int32_t* free_pages;
    int64_t free_cap;
    const int32_t* free_count;
    int32_t* kv_len_out;
    int32_t* free_count_out;
    int32_t* q_off;
    int64_t* slots;
    int32_t* positions;
    int64_t room;
    bool vectors;  // kv_len and new_tokens lie on 16-byte boundaries
    DeviceStatus* status;
};

struct Need {
    uint32_t len, n;  // below 2^31
    uint32_t held;    // pages that it holds
    uint32_t pages;   // pages beyond those
    bool bad;
};

__device__ __forceinline__ Need plan_need(const PlanArgs& a, int len, int n)
{
    Need r;
    r.len = max(len, 0);
    r.n = max(n, 0);
    r.bad = len < 0 || n < 0 || r.len + r.n > 0x7fffffffu;  // the new length is an int32
    if (r.len + r.n > 0x7fffffffu) r.n = 0;
    const uint32_t up = a.page.d - 1;
    r.held = a.page(r.len + up);
    r.pages = a.page(r.len + r.n + up) - r.held;
    return r;
}

// use(b, need) for the requests [b0, b1) in order.  Eight requests' loads go out together: one at a
// time each would cost a latency (4096 requests, then 16 a thread: 13.7 us against 9.7).
template <class F>
__device__ __forceinline__ void for_requests(const PlanArgs& a, int b0, int b1, F&& use)
{
    for (int b = b0; b < b1; b += 8) {
        int len[8], n[8];
        if (a.vectors && b + 8 <= b1) {  // b is a multiple of 4
#pragma unroll
            for (int q = 0; q < 8; q += 4) {
                *reinterpret_cast<int4*>(len + q) = *reinterpret_cast<const int4*>(a.kv_len + b + q);
                *reinterpret_cast<int4*>(n + q) = *reinterpret_cast<const int4*>(a.new_tokens + b + q);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                len[q] = b + q < b1 ? a.kv_len[b + q] : 0;
                n[q] = b + q < b1 ? a.new_tokens[b + q] : 0;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (b + q < b1) use(b + q, plan_need(a, len[q], n[q]));
    }
}

template <int kPlanTokens>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a)
{
    __shared__ int64_t warp_tok[kPlanThreads / 32], warp_pag[kPlanThreads / 32];
    __shared__ int32_t owner[kPlanTokens];       // request + 1 at its first token of the range, else 0
    __shared__ int32_t warp_max[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * kPlanTokens;
    const int64_t t1 = min(t0 + kPlanTokens, a.room);
    for (int i = tid; i < kPlanTokens; i += kPlanThreads) owner[i] = 0;

    // sums of this thread's consecutive requests
    const int per = a.B > kPlanThreads ? (a.B + kPlanThreads * 4 - 1) / (kPlanThreads * 4) * 4 : 1;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int64_t tok = 0, pag = 0;
    bool bad = false;
    for_requests(a, b0, b1, [&](int, const Need& r) {
        tok += r.n;
        pag += r.pages;
        bad |= r.bad;
    });
    if (bad) report_status(a.status, NVQ_ERR_ARG, kWherePlan);
    int64_t tok_in = tok, pag_in = pag;  // inclusive over the warp's threads
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t u = __shfl_up_sync(~0u, tok_in, d), v = __shfl_up_sync(~0u, pag_in, d);
        if (lane >= d) {
            tok_in += u;
            pag_in += v;
        }
    }
    if (lane == 31) {
        warp_tok[warp] = tok_in;
        warp_pag[warp] = pag_in;
    }
    __syncthreads();
    int64_t tok_off = tok_in - tok, tok_all = 0, pag_off = pag_in - pag, pag_all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            tok_off += warp_tok[w];
            pag_off += warp_pag[w];
        }
        tok_all += warp_tok[w];
        pag_all += warp_pag[w];
    }
    const int64_t have = min((int64_t)max(*a.free_count, 0), a.free_cap);
    if (blockIdx.x == 0 && tid == 0) {
        a.q_off[a.B] = (int32_t)min(tok_all, (int64_t)0x7fffffff);
        *a.free_count_out = (int32_t)max(have - pag_all, (int64_t)0);
        if (pag_all > have || tok_all > a.room || *a.free_count < 0 || *a.free_count > a.free_cap)
            report_status(a.status, NVQ_ERR_ARG, kWherePlan);
    }
    // the requests again, with their offsets: outputs per request (spread over the CTAs by thread),
    // marks in this CTA's range, and the pages taken before the request kept for its tokens
    const bool mine = tid % gridDim.x == blockIdx.x;
    __shared__ int64_t first_tok[kPlanTokens], first_pag[kPlanTokens];
    int64_t to = tok_off, po = pag_off;
    for_requests(a, b0, b1, [&](int b, const Need& r) {
        if (mine) {
            a.kv_len_out[b] = r.len + r.n;
            a.q_off[b] = (int32_t)min(to, (int64_t)0x7fffffff);
        }
        if (r.n > 0 && to < t1 && to + r.n > t0) {
            const int at = (int)(max(to, t0) - t0);
            owner[at] = b + 1;
            first_tok[at] = to;
            first_pag[at] = po;
        }
        to += r.n;
        po += r.pages;
    });
    __syncthreads();
    // position of the last mark at or before each token of the range (marks ascend with the request)
    constexpr int kPer = kPlanTokens / kPlanThreads;
    int best = -1, marks[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = tid * kPer + i;
        if (owner[at]) best = at;
        marks[i] = best;
    }
    int run = best;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(~0u, run, d);
        if (lane >= d) run = max(run, u);
    }
    if (lane == 31) warp_max[warp] = run;
    int before = __shfl_up_sync(~0u, run, 1);
    if (lane == 0) before = -1;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = max(before, warp_max[w]);
    bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t t = t0 + tid * kPer + i;
        if (t >= t1) break;
        const int at = max(marks[i], before);
        int64_t slot = -1;
        int32_t place = -1;
        if (at >= 0 && t < tok_all) {
            const int b = owner[at] - 1;
            const uint32_t len = max(a.kv_len[b], 0), pos = len + (uint32_t)(t - first_tok[at]);
            const uint32_t blk = a.page(pos), held = a.page(len + a.page.d - 1), in = pos - blk * a.page.d;
            int32_t page = -1;
            place = (int32_t)pos;
            if (blk < (uint32_t)a.max_blocks) {
                if (blk < held) {
                    page = a.table[(int64_t)b * a.ld_table + blk];
                } else {
                    const int64_t f = have - 1 - (first_pag[at] + blk - held);
                    if (f >= 0) {
                        page = a.free_pages[f];
                        if (in == 0) a.table[(int64_t)b * a.ld_table + blk] = page;
                    }
                }
            }
            if (page >= 0) slot = (int64_t)page * a.page.d + in;
            bad |= page < 0;
        }
        a.slots[t] = slot;
        if (a.positions) a.positions[t] = place;
    }
    if (bad) report_status(a.status, NVQ_ERR_ARG, kWherePlan);
}

// ------------------------------------------------------------------ append
// One thread per block of 16 keys' values and the same block of the values: 64 bytes read, twice 8
// code bytes and a scale byte written (and 64 bytes of the values held, if asked for).  A pure
// stream: bound by HBM for a prompt's tokens, by the launch for a decode batch.
// Measured: 16384 tokens of 4 heads of 128 values in 13.7 us = 5.6 TB/s, 0.82 of a copy; 64 tokens in
// 2.6 us.
struct AppendArgs {
    nvq_kv_cache c;
    const __nv_bfloat16 *k, *v;
    int64_t ks_t, ks_h, vs_t, vs_h;
    const int64_t* slots;
    uint32_t rows;  // tokens x heads
    FastDiv heads, page;
    __nv_bfloat16 *k_hat, *v_hat;
    DeviceStatus* status;
};

template <int kDim>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr uint32_t kBlocks = kDim / 16;
    const uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const uint32_t blk = (uint32_t)i % kBlocks, row = (uint32_t)(i / kBlocks);
    if (row >= a.rows) return;
    const uint32_t t = a.heads(row), head = row - t * a.heads.d;
    const uint4* pk = reinterpret_cast<const uint4*>(a.k + t * a.ks_t + head * a.ks_h + blk * 16);
    const uint4* pv = reinterpret_cast<const uint4*>(a.v + t * a.vs_t + head * a.vs_h + blk * 16);
    const uint4 in[2][2] = {{__ldcs(pk), __ldcs(pk + 1)}, {__ldcs(pv), __ldcs(pv + 1)}};
    const int64_t slot = a.slots[t];
    const bool kept = slot >= 0 && slot < a.c.pages * a.c.page_size;
    if (slot >= 0 && !kept) report_status(a.status, NVQ_ERR_ARG, kWhereAppend);
    const uint32_t page = kept ? a.page((uint32_t)slot) : 0, at = kept ? (uint32_t)slot - page * a.page.d : 0;
    const int64_t code_at = page * a.c.page_stride + head * a.c.head_stride + at * (kDim / 2) + blk * 8;
    const int64_t sf_at = page * a.c.sf_page_stride + head * a.c.sf_head_stride + at * kBlocks + blk;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint32_t w[8] = {in[side][0].x, in[side][0].y, in[side][0].z, in[side][0].w,
                               in[side][1].x, in[side][1].y, in[side][1].z, in[side][1].w};
        float v[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[2 * e] = bf16lo(w[e]);
            v[2 * e + 1] = bf16hi(w[e]);
        }
        const nvq_tensor_scale* ts = side ? a.c.v_tscale : a.c.k_tscale;
        const BlockOut o = quantize16(v, ts->s_enc, ts->s_dec);
        if (kept) {
            *reinterpret_cast<uint2*>((side ? a.c.v_codes : a.c.k_codes) + code_at) = make_uint2(o.code_lo, o.code_hi);
            (side ? a.c.v_sf : a.c.k_sf)[sf_at] = (uint8_t)o.sb;
        }
        __nv_bfloat16* hat = side ? a.v_hat : a.k_hat;
        if (hat) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 x = e2m1x2_value(((e < 4 ? o.code_lo : o.code_hi) >> (8 * (e & 3))) & 0xffu);
                const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(x.x, o.d_b), __fmul_rn(x.y, o.d_b));
                h[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            uint4* dst = reinterpret_cast<uint4*>(hat + ((int64_t)row * kDim + blk * 16));
            __stcs(dst, make_uint4(h[0], h[1], h[2], h[3]));
            __stcs(dst + 1, make_uint4(h[4], h[5], h[6], h[7]));
        }
    }
}

}  // namespace nvq

using namespace nvq;

extern "C" nvq_status nvfp4_kv_plan(const int32_t* new_tokens, const int32_t* kv_len, int32_t B, int32_t page_size,
                                    int32_t* block_table, int64_t ld_table, int32_t max_blocks, const int32_t* free_pages,
                                    int64_t free_cap, const int32_t* free_count, int32_t* kv_len_out, int32_t* free_count_out,
                                    int32_t* q_off, int64_t* slots, int32_t* positions, int64_t room, void* stream)
{
    NVQ_TRACE("nvfp4_kv_plan");
    NVQ_CHECK_ARG(new_tokens && kv_len && block_table && free_pages && free_count && kv_len_out && free_count_out && q_off && slots,
                  NVQ_ERR_ARG, "nvfp4_kv_plan: null pointer argument");
    NVQ_CHECK_ARG(kv_len_out != kv_len && kv_len_out != new_tokens && free_count_out != free_count, NVQ_ERR_ARG,
                  "nvfp4_kv_plan: an output is its own input");
    NVQ_CHECK_ARG(B >= 1 && B <= (1 << 20), NVQ_ERR_SHAPE, "nvfp4_kv_plan: B outside [1, 2^20]");
    NVQ_CHECK_ARG(page_size >= 1 && page_size <= 65536, NVQ_ERR_SHAPE, "nvfp4_kv_plan: page_size outside [1, 65536]");
    NVQ_CHECK_ARG(max_blocks >= 1 && ld_table >= max_blocks && free_cap >= 1, NVQ_ERR_SHAPE,
                  "nvfp4_kv_plan: max_blocks < 1, ld_table < max_blocks or free_cap < 1");
    NVQ_CHECK_ARG(room >= 1 && room < (1ll << 31), NVQ_ERR_SHAPE, "nvfp4_kv_plan: room outside [1, 2^31)");
    NVQ_CHECK_ARG(aligned(slots, 8) && aligned(new_tokens, 4) && aligned(kv_len, 4) && aligned(block_table, 4) &&
                      aligned(free_pages, 4) && aligned(free_count, 4) && aligned(kv_len_out, 4) && aligned(free_count_out, 4) &&
                      aligned(q_off, 4) && aligned(positions, 4),
                  NVQ_ERR_ALIGN, "nvfp4_kv_plan: a pointer is not aligned to its elements");
    DeviceStatus* dst = device_status_ptr();
    NVQ_CHECK_ARG(dst, NVQ_ERR_CUDA, "nvfp4_kv_plan: device status word unavailable");
    set_error("");
    PlanArgs a{new_tokens, kv_len, B, FastDiv::by((uint32_t)page_size), block_table, ld_table, max_blocks, free_pages, free_cap, free_count,
               kv_len_out, free_count_out, q_off, slots, positions, room, aligned(kv_len, 16) && aligned(new_tokens, 16), dst};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e, "nvfp4_kv_plan: device attributes");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (room <= (int64_t)sms * 512)
        plan_kernel<512><<<(unsigned)((room + 511) / 512), kPlanThreads, 0, st>>>(a);
    else
        plan_kernel<2048><<<(unsigned)((room + 2047) / 2048), kPlanThreads, 0, st>>>(a);
    NVQ_LAUNCH_CHECK("plan_kernel");
    return NVQ_OK;
}

extern "C" nvq_status nvfp4_kv_append(const nvq_kv_cache* cache, const void* k, int64_t k_stride_t, int64_t k_stride_h,
                                      const void* v, int64_t v_stride_t, int64_t v_stride_h, const int64_t* slots,
                                      int64_t tokens, void* k_hat, void* v_hat, void* stream)
{
    NVQ_TRACE("nvfp4_kv_append");
    const nvq_status s = check_cache(cache, "nvfp4_kv_append");
    if (s != NVQ_OK) return s;
    NVQ_CHECK_ARG(k && v && slots && !k_hat == !v_hat, NVQ_ERR_ARG,
                  "nvfp4_kv_append: null pointer argument, or one of k_hat and v_hat without the other");
    NVQ_CHECK_ARG(tokens >= 1 && tokens * cache->kv_heads < (1ll << 31) && tokens < (1ll << 31), NVQ_ERR_SHAPE,
                  "nvfp4_kv_append: tokens < 1, or 2^31 rows (tokens x heads) or more");
    NVQ_CHECK_ARG(k_stride_t >= 0 && k_stride_h >= 0 && v_stride_t >= 0 && v_stride_h >= 0, NVQ_ERR_SHAPE,
                  "nvfp4_kv_append: a negative stride");
    NVQ_CHECK_ARG(k_stride_t % 8 == 0 && k_stride_h % 8 == 0 && v_stride_t % 8 == 0 && v_stride_h % 8 == 0 && aligned(k, 16) &&
                      aligned(v, 16) && aligned(slots, 8) && aligned(k_hat, 16) && aligned(v_hat, 16),
                  NVQ_ERR_ALIGN, "nvfp4_kv_append: k, v and the hats need 16-byte aligned rows");
    DeviceStatus* dst = device_status_ptr();
    NVQ_CHECK_ARG(dst, NVQ_ERR_CUDA, "nvfp4_kv_append: device status word unavailable");
    set_error("");
    AppendArgs a{*cache, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), k_stride_t, k_stride_h,
                 v_stride_t, v_stride_h, slots, (uint32_t)(tokens * cache->kv_heads), FastDiv::by((uint32_t)cache->kv_heads),
                 FastDiv::by((uint32_t)cache->page_size), static_cast<__nv_bfloat16*>(k_hat), static_cast<__nv_bfloat16*>(v_hat), dst};
    const int64_t blocks = (tokens * cache->kv_heads * (cache->head_dim / 16) + 255) / 256;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (cache->head_dim) {
        case 64: append_kernel<64><<<(unsigned)blocks, 256, 0, st>>>(a); break;
        case 128: append_kernel<128><<<(unsigned)blocks, 256, 0, st>>>(a); break;
        default: append_kernel<256><<<(unsigned)blocks, 256, 0, st>>>(a); break;
    }
    NVQ_LAUNCH_CHECK("append_kernel");
    return NVQ_OK;
}
