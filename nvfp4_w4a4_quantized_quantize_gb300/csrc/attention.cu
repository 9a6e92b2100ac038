// attention.cu -- attention of new queries over the paged NVFP4 cache (nvfp4_kv_attention).
//
//   s_j = sm_scale * S_dec(K) * sum_d q_d V[k_jd] sb(k)_{j, d/16},  p = softmax(s),
//   out_d = S_dec(V) * sum_j p_j V[v_jd] sb(v)_{j, d/16}
//
// One pass over the keys with a running maximum and sum.  A decode step's floor is the cache
// read once (0.5625 bytes a value); the work on a value is its expansion to 16 bits and 8 or 16
// rows of products, so the design keeps both in registers:
//   - a warp works on 32 keys at a time (of 64 values a key it fetches two such tiles at a time).
//     S^T = K Q^T and O^T = V^T P^T put the keys' and the values' tiles in the 16-row operand of
//     mma.m16n8k16 and the queries (the heads of a group, times the new tokens) in its 8 columns, so
//     a group of 8 heads wastes nothing.
//   - the products' inner index may be permuted: a lane reads the head dimension (or the keys) in
//     the order in which the bytes lie, expands two codes an instruction to f16 and multiplies
//     by the block's scale.  A code times its E4M3 scale has at most 6 significant bits and lies
//     in [2^-10, 2688] in magnitude, so the f16 value is exact.
//   - queries are scaled per row by a power of two into f16's range: exact, except that a component
//     below 2^-32 of its row's largest is rounded at 2^-39 of that.
//   - weights enter the second product as f16 of 2^13 p relative to the running maximum (11
//     significant bits down to 2^-27 of it; a tile that holds smaller weights takes further
//     passes for them, each 2^28 lower, so none is lost); sums stay fp32.  The maximum is moved
//     only when a score passes it by a factor of 4, which keeps 2^13 p within f16 and leaves
//     most tiles without a reduction over lanes or a rescaling.
//   - tiles arrive by asynchronous 16-byte copies into a ring per warp, a part of the warp for each
//     16 keys (which are sure to share a page), so no barrier joins the warps while they stream.  (Bulk
//     copies, one elected lane each, cost more: a step's eight small copies are issued one after the
//     other, 107 us against 82 for 64 requests of up to 16k keys as the kernel then was.)
// Work is cut into equal runs of steps of 64 or 32 keys over all requests, heads and row tiles, one run per
// resident block, whatever the lengths; beginning a row tile counts as kBeginKeys keys.  A row tile
// whose keys are spread over several blocks is joined by the block that finishes last, always in
// the order of the keys.
//
// Measured (this kernel alone, replayed; 32 query and 4 key heads of 128 values, against a copy's 6.78
// TB/s): 64 requests of 65536 keys, 2.4 GB, in 441 us = 5.48 TB/s, 0.81; 64 of 1 to 16384 keys, 292 MB, in
// 64 us = 0.67, of which about 12 us are the beginning and the join; 8 of up to 100k keys of 64 values with 4
// new tokens each (16-row tiles, pages of 16), 119 MB, in 57 us; one request of 1000 keys in 9 us.  Instruction issue
// bounds it: 605 instructions of a warp per 32 keys of 128 values, 2.2 of 4 issued a cycle, the
// integer pipe (which expands the codes) 46 % busy, tensor cores 23 %.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

#include "kvcache.cuh"

namespace nvq {

constexpr int kAttnMaxCtas = 640;    // bound of the grid, which sizes the workspace
constexpr int kPieceFloats = 2048 + 32;  // accumulators (rows x head_dim) and two statistics a row
constexpr float kShift = 13.0f;      // weights are held times 2^kShift
constexpr float kSlack = 2.0f;       // how far (log2) a score may pass the running maximum
constexpr float kLevel = 268435456.0f;      // 2^28: a pass for smaller weights covers as much
constexpr float kNormalLog2 = -14.0f, kNormal = 6.103515625e-5f;  // the least f16 with all its bits
constexpr int kBeginKeys = 384;      // keys that a segment's beginning and end cost as much as
constexpr double kMaxUnits = 9007199254740992.0;  // 2^53 units of work: times the blocks they stay within 64 bits

struct AttnArgs {
    nvq_kv_cache c;
    const __nv_bfloat16* q;
    int64_t q_t, q_h, rows;
    int32_t heads, group;
    const int32_t* q_off;
    int32_t B, max_q;
    const int32_t* kv_len;
    const int32_t* table;
    int64_t ld_table;
    int32_t max_blocks;
    float sm_scale;
    int32_t window;
    __nv_bfloat16* out;
    int64_t o_t, o_h;
    float* lse;
    float* pieces;       // [grid][2][kPieceFloats]
    uint32_t* arrived;   // [grid]
    int32_t page_shift;  // log2(page_size / 16), or -1
    DeviceStatus* status;
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t attn_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes from global to shared memory, asynchronously; zeros where `there` is false (src stays valid).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Eight E2M1 codes of a word -> four f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* o)
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// Two E4M3 bytes (low half of w) -> an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// An f16 pair times one half (low or high) of another.
__device__ __forceinline__ uint32_t mul_f16_half(uint32_t a, uint32_t s, int high)
{
    const __half2 h = *reinterpret_cast<const __half2*>(&s);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), high ? __high2half2(h) : __low2half2(h));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The key (of 16) behind row r of a tile: pairs of rows at odd distance, so that neither the rows
// (8 at a time) nor every second row (4 at a time) of a tile fall on the same shared-memory banks.
__device__ __forceinline__ int key_of_row(int r) { return r ^ ((r >> 1) & 1); }

// ------------------------------------------------------------------ a request's share of the work
struct Request {
    int first, n;     // query rows [first, first + n)
    int lo, hi;       // keys read: [lo, hi), lo a multiple of 16
    int steps, segs;  // steps of a segment; segments: kv heads x row tiles
    int cost, begin;  // units of work of a step and of a segment's beginning
    __device__ __forceinline__ int units() const { return begin + steps * cost; }
};

template <int kRows, int kStep>
__device__ __forceinline__ Request request(const AttnArgs& a, int b, bool& bad)
{
    Request r;
    const int64_t first = a.q_off ? a.q_off[b] : b, end = a.q_off ? a.q_off[b + 1] : b + 1;
    int64_t len = a.kv_len[b];
    const int64_t most = (int64_t)a.max_blocks * a.c.page_size;
    const bool bad_rows = first < 0 || end < first || end > a.rows || end - first > a.max_q;
    bad |= bad_rows || len < 0 || len > most;
    len = min(max(len, (int64_t)0), most);
    r.first = (int)first;
    r.n = bad_rows ? 0 : (int)(end - first);
    r.hi = (int)len;
    // the first query's oldest key; queries before the sequence's start see nothing
    const int64_t oldest = a.window > 0 ? max((int64_t)0, len - r.n + 1 - a.window) : 0;
    r.lo = (int)min(oldest, len) & ~15;
    r.steps = max(1, (r.hi - r.lo + kStep - 1) / kStep);
    // of 16-row tiles a step on 8 rows costs three quarters
    r.cost = kRows == 8 ? 1 : r.n * a.group <= 8 ? 3 : 4;
    r.begin = kBeginKeys / kStep * (kRows == 8 ? 1 : 4);
    r.segs = a.c.kv_heads * ((r.n * a.group + kRows - 1) / kRows);
    return r;
}

// Every block finds its run by itself: a scan of all requests (12 bytes each, served by L2), which
// costs less than a launch that would prepare it.
template <int kThreads>
__device__ __forceinline__ int64_t block_scan(int64_t mine, uint32_t mine2, int64_t& all, uint32_t& all2, int64_t* part, uint32_t* part2)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t in = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t u = __shfl_up_sync(~0u, in, d);
        if (lane >= d) in += u;
    }
    mine2 = __reduce_add_sync(~0u, mine2);
    if (lane == 31) {
        part[warp] = in;
        part2[warp] = mine2;
    }
    __syncthreads();
    int64_t off = in - mine;
    all = 0;
    all2 = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) off += part[w];
        all += part[w];
        all2 += part2[w];
    }
    return off;
}

// ------------------------------------------------------------------ the kernel
// kDim: head dimension; kRows: query rows of a tile (8 or 16); kStep: keys of a step, which a stage
// holds; kWarps a block, kStages a warp.
template <int kDim, int kRows, int kStep_, int kWarps, int kStages>
struct Attn {
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTiles = kRows / 8;              // 8-column tiles of the products
    static constexpr int kStep = kStep_;
    static constexpr int kSub = kRows == 8 ? kStep : 32;  // keys of a tile
    static constexpr int kCodeBytes = kStep * kDim / 2, kSfBytes = kStep * kDim / 16;
    static constexpr int kStageBytes = 2 * (kCodeBytes + kSfBytes);
    static constexpr int kJoinBytes = kWarps * (kRows * kDim + 2 * kRows) * 4;
    static constexpr int kRing = kWarps * kStages * kStageBytes > kJoinBytes ? kWarps * kStages * kStageBytes : kJoinBytes;
    static constexpr int kSmem = kRing;
    static constexpr int kPairs = kRows * kDim / 2 / kThreads;  // pairs of a thread in the join
    static constexpr int kBatch = 16 / kPairs;                  // pieces whose loads go out together
    static_assert(kPairs * kThreads == kRows * kDim / 2 && kPairs <= 8);
    static constexpr int kWords = kDim / 32;              // words of codes a lane has of a key (4 lanes a key)
    static_assert(kRows * kDim + 2 * kRows <= kPieceFloats, "a piece fits its slot");
    static_assert(kAttnMaxCtas * kRows * 4 <= kRing, "all pieces' factors fit");
};

template <int kDim, int kRows, int kStep, int kWarps, int kStages, int kMinCtas>
__global__ void __launch_bounds__(kWarps * 32, kMinCtas) attention_kernel(const __grid_constant__ AttnArgs a)
{
    using T = Attn<kDim, kRows, kStep, kWarps, kStages>;
    constexpr int kTiles = T::kTiles, kWords = T::kWords, kThreads = T::kThreads;
    constexpr int kOut = kDim / 16;  // 16-row tiles of O^T
    constexpr int kSub = T::kSub, kM = kSub / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t part[kWarps];
    __shared__ uint32_t part2[kWarps];
    __shared__ int64_t run_base;
    __shared__ int run_b, last_piece;
    __shared__ float row_top[kRows], row_sum[kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

    // ---- this block's run of steps
    const int per = (a.B + kThreads - 1) / kThreads;
    const int rb0 = min((int)threadIdx.x * per, a.B), rb1 = min(rb0 + per, a.B);
    int64_t mine = 0, total;
    uint32_t my_tiles = 0, tiles;
    bool bad = false;
    for (int b = rb0; b < rb1; ++b) {
        const Request r = request<kRows, T::kStep>(a, b, bad);
        mine += (int64_t)r.units() * r.segs;
        my_tiles += min(r.segs, 1 << 10);  // capped: below they matter only while few, and their sum stays in 32 bits
    }
    my_tiles = min(my_tiles, 1u << 20);
    const int64_t before = block_scan<kThreads>(mine, my_tiles, total, tiles, part, part2);
    if (bad && blockIdx.x == 0) report_status(a.status, NVQ_ERR_ARG, kWhereAttention);
    if (total == 0) return;  // no queries
    // A step for every warp: fewer, fuller blocks have fewer pieces to join.  (At least: a run is then
    // longer than a step, so a block within a segment has a piece of it, which the join counts on.)
    constexpr int kLeast = kWarps * (kRows == 8 ? 1 : 2);
    static_assert(kLeast >= 4);
    // And no more than pay: a row tile of S steps in n pieces takes about S / (kWarps n) steps and n / kBatch
    // loads of the join one after the other, least for n near the root of S.  (Measured: 1.1 sqrt(S).  One
    // request of 100k keys of one KV head in 456 blocks took 71 us, in 110 27; 4 new tokens after 10000 keys
    // 43 and 30.)  The first few loads of the join are nearly free.
    const float spread = fmaxf(1.1f * sqrtf((float)tiles * (float)total * (kRows == 8 ? 1.0f : 0.25f)), 3.0f * T::kBatch * (float)tiles);
    const int64_t blocks = min((int64_t)gridDim.x, max(min(total / kLeast, (int64_t)spread), (int64_t)1));
    if ((int64_t)blockIdx.x >= blocks) return;
    // units are counted in 64 bits over the batch (below kMaxUnits, which the host sees to), in 32 within a segment
    const int64_t begin = total * blockIdx.x / blocks, end = total * (blockIdx.x + 1) / blocks;
    if (before <= begin && begin < before + mine) {
        int64_t base = before;
        for (int b = rb0; b < rb1; ++b) {
            const Request r = request<kRows, T::kStep>(a, b, bad);
            const int64_t s = (int64_t)r.units() * r.segs;
            if (begin < base + s) {
                run_b = b;
                run_base = base;
                break;
            }
            base += s;
        }
    }
    __syncthreads();
    int b = run_b;
    Request rq = request<kRows, T::kStep>(a, b, bad);
    int seg = (int)((begin - run_base) / rq.units());
    int64_t seg_at = run_base + (int64_t)seg * rq.units();  // the segment's first unit
    int from = (int)(begin - seg_at);                       // where the run is in it

    // the sign of sm_scale goes into the queries, so that the largest product is the largest score; a
    // scale of 0 becomes the least that keeps -inf times it -inf
    const float z_sign = a.sm_scale < 0.0f ? -1.0f : 1.0f;
    const float z_scale = fabsf(a.sm_scale) * a.c.k_tscale->s_dec * 1.4426950408889634f;
    const float v_scale = a.c.v_tscale->s_dec;
    const uint32_t ring = attn_smem(smem) + warp * kStages * T::kStageBytes;
    uint32_t fill = 0, turn = 0;  // stage filled next, stage read next

    while (true) {
        // ---- the run's portion, steps [pbeg, pend), of one segment
        while (seg >= rq.segs) {
            rq = request<kRows, T::kStep>(a, ++b, bad);
            seg = 0;
        }
        // a step belongs to the run that its first unit falls in
        auto step_at = [&](int u) { return u <= rq.begin ? 0 : min((u - rq.begin + rq.cost - 1) / rq.cost, rq.steps); };
        const int pbeg = step_at(from), pend = step_at((int)min(end - seg_at, (int64_t)rq.units()));
        if (pend <= pbeg) {
            seg_at += rq.units();
            if (seg_at >= end) break;
            ++seg;
            from = 0;
            continue;
        }
        const int kvh = seg % a.c.kv_heads, row0 = seg / a.c.kv_heads * kRows;
        const int rows = rq.n * a.group;

        // kLanes lanes copy the codes and scales of 16 keys
        constexpr int kLanes = 32 * 16 / T::kStep, kPieces = kDim / 16;  // 16-byte pieces of 16 keys' scales
        const int group = lane / kLanes, li = lane % kLanes;
        const int32_t* table = a.table + (int64_t)b * a.ld_table;
        const int gran = a.c.page_size >> 4;
        const uint8_t* kc = a.c.k_codes + kvh * a.c.head_stride + li * 16;
        const uint8_t* vc = a.c.v_codes + kvh * a.c.head_stride + li * 16;
        const uint8_t* ks = a.c.k_sf + kvh * a.c.sf_head_stride;
        const uint8_t* vs = a.c.v_sf + kvh * a.c.sf_head_stride;
        const uint8_t* sf = (kLanes >= 2 * kPieces && li >= kPieces ? vs : ks) + (li % kPieces) * 16;
        auto group_of = [&](int step) { return (rq.lo >> 4) + step * (T::kStep / 16) + group; };  // of 16 keys
        auto page_of = [&](int step) {
            const int t = group_of(step);
            return t * 16 < rq.hi ? __ldg(table + (a.page_shift >= 0 ? t >> a.page_shift : t / gran)) : 0;
        };
        auto issue = [&](int step, int page) {
            const int t = group_of(step);
            if ((unsigned)page >= (unsigned)a.c.pages) {
                report_status(a.status, NVQ_ERR_ARG, kWhereAttention);
                page = 0;
            }
            const bool there = t * 16 < rq.hi;
            const int in = a.page_shift >= 0 ? t & (gran - 1) : t % gran;
            const int64_t off = page * a.c.page_stride + in * (8 * kDim), soff = page * a.c.sf_page_stride + in * kDim;
            const uint32_t dst = ring + fill * T::kStageBytes + group * (8 * kDim) + li * 16;
            const uint32_t sdst = ring + fill * T::kStageBytes + 2 * T::kCodeBytes + group * kDim + (li % kPieces) * 16;
#pragma unroll
            for (int i = 0; i < kDim / 2 / kLanes; ++i) {
                copy16(dst + i * (kLanes * 16), kc + off + i * (kLanes * 16), there);
                copy16(dst + T::kCodeBytes + i * (kLanes * 16), vc + off + i * (kLanes * 16), there);
            }
            if constexpr (kLanes >= 2 * kPieces) {
                static_assert(kLanes == 2 * kPieces);
                copy16(sdst + (li < kPieces ? 0 : T::kSfBytes), sf + soff, there);
            } else {
                static_assert(kLanes == kPieces);
                copy16(sdst, sf + soff, there);
                copy16(sdst + T::kSfBytes, vs + li * 16 + soff, there);
            }
            fill = fill + 1 == kStages ? 0 : fill + 1;
        };
        auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

        // ---- queries: lane (g, c) holds row g of each tile, the dimensions of its bytes of a key
        uint32_t q[kTiles][kWords * 4];
        float zs[kTiles][2];  // score scale (log2) of columns 2c, 2c + 1
        const int first_s = pbeg + warp;
        turn = fill;
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            if (first_s + i * kWarps < pend) issue(first_s + i * kWarps, page_of(first_s + i * kWarps));
            commit();
        }
        int page_next = first_s + kStages * kWarps < pend ? page_of(first_s + kStages * kWarps) : 0;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const int r = row0 + t * 8 + g;
            uint4 w[kWords];
            const bool there = r < rows;
            const int i = r / a.group;
            const __nv_bfloat16* qp = a.q + (int64_t)(rq.first + (there ? i : 0)) * a.q_t +
                                      (int64_t)(kvh * a.group + (there ? r - i * a.group : 0)) * a.q_h + c * (kDim / 4);
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                w[k] = there ? *reinterpret_cast<const uint4*>(qp + k * 8) : make_uint4(0, 0, 0, 0);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[k].x & 0x7fff7fffu, w[k].y & 0x7fff7fffu),
                                             __vmaxu2(w[k].z & 0x7fff7fffu, w[k].w & 0x7fff7fffu)));
            }
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            // largest magnitude into [2^14, 2^15)
            const int shift = min(14 - ((int)(top >> 7) - 127), 126);
            const float up = __uint_as_float((uint32_t)(shift + 127) << 23), down = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) q[t][k * 4 + e] = pack_f16(bf16lo(u[e]) * (z_sign * up), bf16hi(u[e]) * (z_sign * up));
            }
            const float s = fmaxf(z_scale * down, 1e-37f);
            zs[t][0] = __shfl_sync(~0u, s, (2 * c) * 4);
            zs[t][1] = __shfl_sync(~0u, s, (2 * c + 1) * 4);
        }
        // keys seen by columns 2c, 2c + 1
        int see_lo[kTiles][2], see_hi[kTiles][2], all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int p = rq.hi - rq.n + min(row0 + t * 8 + 2 * c + e, rows - 1) / a.group;
                see_hi[t][e] = p + 1;
                see_lo[t][e] = a.window > 0 ? p + 1 - a.window : 0;
                all_lo = max(all_lo, see_lo[t][e]);
                all_hi = min(all_hi, see_hi[t][e]);
            }

        all_lo = __reduce_max_sync(~0u, all_lo);
        all_hi = __reduce_min_sync(~0u, all_hi);

        float o[kOut][kTiles][4], m[kTiles][2], l[kTiles][2];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            m[t][0] = m[t][1] = -CUDART_INF_F;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < kOut; ++j) o[j][t][0] = o[j][t][1] = o[j][t][2] = o[j][t][3] = 0.0f;
        }

        // ---- a tile of 32 keys, the first of them tok, at `codes` and `scales` of a stage; for the
        // first kUsed tiles of rows
        auto attend = [&](auto used, const uint8_t* codes, const uint8_t* scales, int tok) {
            constexpr int kUsed = decltype(used)::value;
            const bool whole = tok >= all_lo && tok + kSub <= all_hi;

            // scores
            float z[kM][kUsed][4];
#pragma unroll
            for (int mt = 0; mt < kM; ++mt) {
#pragma unroll
                for (int t = 0; t < kUsed; ++t) z[mt][t][0] = z[mt][t][1] = z[mt][t][2] = z[mt][t][3] = 0.0f;
                uint32_t ka[kWords], kb[kWords];
                const int ta = mt * 16 + key_of_row(g), tb = mt * 16 + 8 + key_of_row(g);
                const uint8_t* pa = codes + ta * (kDim / 2) + c * (kDim / 8);
                const uint8_t* pb = codes + tb * (kDim / 2) + c * (kDim / 8);
                const uint8_t* sa = scales + ta * (kDim / 16) + c * (kDim / 64);
                const uint8_t* sb = scales + tb * (kDim / 16) + c * (kDim / 64);
                uint32_t fa, fb;
                if constexpr (kDim == 64) {
                    *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(pa);
                    *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(pb);
                    fa = *sa;
                    fb = *sb;
                } else {
#pragma unroll
                    for (int k = 0; k < kWords; k += 4) {
                        *reinterpret_cast<uint4*>(ka + k) = *reinterpret_cast<const uint4*>(pa + k * 4);
                        *reinterpret_cast<uint4*>(kb + k) = *reinterpret_cast<const uint4*>(pb + k * 4);
                    }
                    if constexpr (kDim == 128) {
                        fa = *reinterpret_cast<const uint16_t*>(sa);
                        fb = *reinterpret_cast<const uint16_t*>(sb);
                    } else {
                        fa = *reinterpret_cast<const uint32_t*>(sa);
                        fb = *reinterpret_cast<const uint32_t*>(sb);
                    }
                }
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    // words 2i and 2i + 1 share the scale byte i
                    const uint32_t fa2 = e4m3x2_f16(k >> 2 ? fa >> 16 : fa), fb2 = e4m3x2_f16(k >> 2 ? fb >> 16 : fb);
                    const int high = k >> 1 & 1;
                    uint32_t xa[4], xb[4];
                    e2m1x8_f16(ka[k], xa);
                    e2m1x8_f16(kb[k], xb);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        xa[e] = mul_f16_half(xa[e], fa2, high);
                        xb[e] = mul_f16_half(xb[e], fb2, high);
                    }
#pragma unroll
                    for (int t = 0; t < kUsed; ++t) {
                        mma16816(z[mt][t], xa[0], xb[0], xa[1], xb[1], q[t][k * 4], q[t][k * 4 + 1]);
                        mma16816(z[mt][t], xa[2], xb[2], xa[3], xb[3], q[t][k * 4 + 2], q[t][k * 4 + 3]);
                    }
                }
            }
            // keys a row does not see get -inf
            float low[kUsed][2];  // least score seen
            if (!whole) {
#pragma unroll
                for (int t = 0; t < kUsed; ++t) {
                    low[t][0] = low[t][1] = CUDART_INF_F;
#pragma unroll
                    for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = tok + mt * 16 + (e >> 1) * 8 + key_of_row(g);
                            const bool sees = j >= see_lo[t][e & 1] && j < see_hi[t][e & 1];
                            if (sees) low[t][e & 1] = fminf(low[t][e & 1], z[mt][t][e]);
                            if (!sees) z[mt][t][e] = -CUDART_INF_F;
                        }
                }
            } else {
#pragma unroll
                for (int t = 0; t < kUsed; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        low[t][e] = fminf(z[0][t][e], z[0][t][e + 2]);
#pragma unroll
                        for (int mt = 1; mt < kM; ++mt) low[t][e] = fminf(low[t][e], fminf(z[mt][t][e], z[mt][t][e + 2]));
                    }
            }
            // running maximum (of scores in units of log2)
            float top[kUsed][2];
            bool move = false;
#pragma unroll
            for (int t = 0; t < kUsed; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[t][e] = fmaxf(z[0][t][e], z[0][t][e + 2]);
#pragma unroll
                    for (int mt = 1; mt < kM; ++mt) top[t][e] = fmaxf(top[t][e], fmaxf(z[mt][t][e], z[mt][t][e + 2]));
                    top[t][e] *= zs[t][e];
                    move |= top[t][e] > m[t][e] + kSlack;
                }
            if (__any_sync(~0u, move)) {
#pragma unroll
                for (int t = 0; t < kUsed; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[t][e];
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                        const float mn = fmaxf(m[t][e], x);
                        const float keep = mn == -CUDART_INF_F ? 1.0f : exp2_fast(m[t][e] - mn);
                        m[t][e] = mn;
                        l[t][e] *= keep;
#pragma unroll
                        for (int j = 0; j < kOut; ++j) {
                            o[j][t][e] *= keep;
                            o[j][t][e + 2] *= keep;
                        }
                    }
            }
            // values: lane (g, c) has dimensions [g * kDim / 8, ...) of the keys behind rows 2c, 2c + 1,
            // 2c + 8, 2c + 9; with each 16 x 16 tile of V^T: use(mt, tile of O^T, operand)
            auto for_values = [&](auto&& use) {
#pragma unroll
                for (int mt = 0; mt < kM; ++mt) {
                    constexpr int kVWords = kDim / 64;  // words of codes a lane has of a key (8 lanes a key)
                    uint32_t v[4][kVWords], f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = mt * 16 + (e >> 1) * 8 + key_of_row(2 * c + (e & 1));
                        const uint8_t* pv = codes + T::kCodeBytes + t * (kDim / 2) + g * (kDim / 16);
                        const uint8_t* sv = scales + T::kSfBytes + t * (kDim / 16) + (kDim == 64 ? g >> 1 : g * (kDim / 128));
                        if constexpr (kDim == 64) {
                            v[e][0] = *reinterpret_cast<const uint32_t*>(pv);
                            f[e] = *sv;
                        } else if constexpr (kDim == 128) {
                            *reinterpret_cast<uint2*>(v[e]) = *reinterpret_cast<const uint2*>(pv);
                            f[e] = *sv;
                        } else {
                            *reinterpret_cast<uint4*>(v[e]) = *reinterpret_cast<const uint4*>(pv);
                            f[e] = *reinterpret_cast<const uint16_t*>(sv);
                        }
                        // bytes of keys that no row sees may hold anything: a scale of 0 makes them 0
                        if (!whole && tok + t >= rq.hi) f[e] = 0;
                    }
#pragma unroll
                    for (int k = 0; k < kVWords; ++k) {
                        const uint32_t sel = 0x40 + (k >> 1) * 0x11;  // the scale byte of words 2i, 2i + 1 of both keys
                        const uint32_t f01 = e4m3x2_f16(__byte_perm(f[0], f[1], sel)), f23 = e4m3x2_f16(__byte_perm(f[2], f[3], sel));
                        // nibbles of two keys side by side, even dimensions first: a byte then expands
                        // to one dimension of both
                        constexpr uint32_t kLow = 0x0f0f0f0fu;
                        const uint32_t w01[2] = {(v[0][k] & kLow) | ((v[1][k] * 16) & ~kLow), ((v[0][k] >> 4) & kLow) | (v[1][k] & ~kLow)};
                        const uint32_t w23[2] = {(v[2][k] & kLow) | ((v[3][k] * 16) & ~kLow), ((v[2][k] >> 4) & kLow) | (v[3][k] & ~kLow)};
                        uint32_t x01[2][4], x23[2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            e2m1x8_f16(w01[e], x01[e]);
                            e2m1x8_f16(w23[e], x23[e]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t op[4] = {mul_f16x2(x01[0][e], f01), mul_f16x2(x01[1][e], f01), mul_f16x2(x23[0][e], f23),
                                                    mul_f16x2(x23[1][e], f23)};
                            use(mt, k * 4 + e, op);
                        }
                    }
                }
            };
            // weights, transposed into the second product's column operand
            uint32_t p[kM][kUsed][2];
            bool tiny = false;
#pragma unroll
            for (int t = 0; t < kUsed; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float base = kShift - (m[t][e] == -CUDART_INF_F ? 0.0f : m[t][e]);
                    tiny |= fmaf(low[t][e], zs[t][e], base) < kNormalLog2;
#pragma unroll
                    for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float& x = z[mt][t][2 * h + e];
                            x = exp2_fast(fmaf(x, zs[t][e], base));
                            l[t][e] += x;
                        }
                }
            if (__any_sync(~0u, tiny)) {
                float up = kLevel, down = 1.0f / kLevel;
                for (int level = 1; level <= 4; ++level, up *= kLevel, down *= 1.0f / kLevel) {
                    bool any = false;
#pragma unroll
                    for (int t = 0; t < kUsed; ++t)
#pragma unroll
                        for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float x = z[mt][t][2 * h] * up, y = z[mt][t][2 * h + 1] * up;
                                x = x < kNormal || x >= kNormal * kLevel ? 0.0f : x;
                                y = y < kNormal || y >= kNormal * kLevel ? 0.0f : y;
                                any |= x != 0.0f || y != 0.0f;
                                p[mt][t][h] = transpose8x8(pack_f16(x, y));
                            }
                    if (!__any_sync(~0u, any)) continue;
                    for_values([&](int mt, int j, const uint32_t* op) {
#pragma unroll
                        for (int t = 0; t < kUsed; ++t) {
                            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816(part, op[0], op[1], op[2], op[3], p[mt][t][0], p[mt][t][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[j][t][e] += part[e] * down;
                        }
                    });
                }
#pragma unroll
                for (int t = 0; t < kUsed; ++t)
#pragma unroll
                    for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (z[mt][t][e] < kNormal) z[mt][t][e] = 0.0f;
            }
#pragma unroll
            for (int t = 0; t < kUsed; ++t)
#pragma unroll
                for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) p[mt][t][h] = transpose8x8(pack_f16(z[mt][t][2 * h], z[mt][t][2 * h + 1]));
            for_values([&](int mt, int j, const uint32_t* op) {
#pragma unroll
                for (int t = 0; t < kUsed; ++t) mma16816(o[j][t], op[0], op[1], op[2], op[3], p[mt][t][0], p[mt][t][1]);
            });
        };

        // ---- the steps
        for (int s = first_s; s < pend; s += kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();  // the stage has arrived for all lanes
            const uint8_t* st = smem + (warp * kStages + turn) * T::kStageBytes;
#pragma unroll 1
            for (int k = 0; k < T::kStep; k += kSub) {
                const int tok = rq.lo + s * T::kStep + k;
                if (tok >= rq.hi) break;
                const uint8_t *codes = st + k * (kDim / 2), *scales = st + 2 * T::kCodeBytes + k * (kDim / 16);
                if (kTiles == 1 || rows - row0 > 8)
                    attend(std::integral_constant<int, kTiles>{}, codes, scales, tok);
                else
                    attend(std::integral_constant<int, 1>{}, codes, scales, tok);
            }
            turn = turn + 1 == kStages ? 0 : turn + 1;
            __syncwarp();  // all lanes have left the stage
            const int ahead = s + kStages * kWarps;
            if (ahead < pend) {
                issue(ahead, page_next);
                page_next = ahead + kWarps < pend ? page_of(ahead + kWarps) : 0;
            }
            commit();
        }

        // ---- join the warps: [warp][tile of 16 dims][row][g][2] accumulators, then maxima and sums
        __syncthreads();
        float* js = reinterpret_cast<float*>(smem);
        float* jm = js + kWarps * kRows * kDim;
        float* jl = jm + kWarps * kRows;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[t][e];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                const int r = t * 8 + 2 * c + e;
                if (g == 0) {
                    jm[warp * kRows + r] = m[t][e];
                    jl[warp * kRows + r] = x;
                }
#pragma unroll
                for (int j = 0; j < kOut; ++j)
                    *reinterpret_cast<float2*>(js + warp * kRows * kDim + ((j * kRows + r) * 8 + g) * 2) = make_float2(o[j][t][e], o[j][t][e + 2]);
            }
        __syncthreads();
        const bool starts = pbeg == 0, ends = pend == rq.steps;
        auto piece_of = [&](int k, int c0) { return a.pieces + ((int64_t)k * 2 + (k == c0 ? 1 : 0)) * kPieceFloats; };
        float* piece = a.pieces + ((int64_t)blockIdx.x * 2 + (starts ? 1 : 0)) * kPieceFloats;
        // a thread's pair: dimensions 2 * j ... of row r; out dimension d = g * kDim / 8 + 2 * j
        auto finish = [&](int i, float x, float y, float top, float sum) {
            const int gg = i & 7, r = (i >> 3) % kRows, j = (i >> 3) / kRows;
            if (row0 + r >= rows) return;
            const int qi = (row0 + r) / a.group, h = kvh * a.group + (row0 + r) - qi * a.group;
            const float s = sum == 0.0f ? 0.0f : 1.0f / sum;  // times v_scale last: their product may lie below fp32's range
            const __nv_bfloat162 pair = __floats2bfloat162_rn(x * s * v_scale, y * s * v_scale);
            *reinterpret_cast<__nv_bfloat162*>(a.out + (int64_t)(rq.first + qi) * a.o_t + (int64_t)h * a.o_h + gg * (kDim / 8) + 2 * j) = pair;
            if (a.lse && gg == 0 && j == 0)
                a.lse[(int64_t)(rq.first + qi) * a.heads + h] =
                    sum == 0.0f ? -CUDART_INF_F : ((top == -CUDART_INF_F ? 0.0f : top) + log2f(sum) - kShift) * 0.6931471805599453f;
        };
        for (int i = threadIdx.x; i < kRows * kDim / 2; i += kThreads) {
            const int r = (i >> 3) % kRows;
            float top = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, jm[w * kRows + r]);
            float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = top == -CUDART_INF_F ? 1.0f : exp2_fast(jm[w * kRows + r] - top);
                const float2 v = *reinterpret_cast<const float2*>(js + w * kRows * kDim + i * 2);
                x += v.x * f;
                y += v.y * f;
                sum += jl[w * kRows + r] * f;
            }
            if (starts && ends) {
                finish(i, x, y, top, sum);
            } else {
                __stcg(reinterpret_cast<float2*>(piece + i * 2), make_float2(x, y));
                if ((i & 7) == 0 && (i >> 3) / kRows == 0) {
                    __stcg(piece + kRows * kDim + r, top);
                    __stcg(piece + kRows * kDim + kRows + r, sum);
                }
            }
        }
        if (!(starts && ends)) {
            // the blocks of the segment, by the runs its first and last step fall in
            auto block_of = [&](int64_t u) { return (int)(((u + 1) * blocks - 1) / total); };
            const int c0 = block_of(seg_at + rq.begin), c1 = block_of(seg_at + rq.begin + (rq.steps - 1) * rq.cost);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                last_piece = atomicAdd(a.arrived + c0, 1u) == (uint32_t)(c1 - c0);
                if (last_piece) a.arrived[c0] = 0;  // ready for the next call
            }
            __syncthreads();
            if (last_piece) {
                __threadfence();
                // the pieces' factors relative to the largest maximum, then sums in the order of the
                // keys, several pieces' loads at a time (one after another each costs a latency)
                const int n = c1 - c0 + 1;
                float* factor = reinterpret_cast<float*>(smem);  // [row][piece]: maxima, then factors
                constexpr int kPairs = T::kPairs, kBatch = T::kBatch;
                float2 v[kBatch][kPairs];
                auto fetch = [&](int k0) {
#pragma unroll
                    for (int q = 0; q < kBatch; ++q)
#pragma unroll
                        for (int j = 0; j < kPairs; ++j)
                            if (k0 + q < n) v[q][j] = __ldcg(reinterpret_cast<const float2*>(piece_of(c0 + k0 + q, c0)) + threadIdx.x + j * kThreads);
                };
                fetch(0);
                constexpr int kMine = kRows / kWarps;  // rows of a warp
                float top[kMine], sum[kMine], sum0[kMine];
                auto stat = [&](int k, int q) { return __ldcg(piece_of(c0 + k, c0) + kRows * kDim + warp + q * kWarps); };
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
                    top[q] = -CUDART_INF_F;
                    sum[q] = 0.0f;
                    sum0[q] = lane < n ? stat(lane, q + kMine) : 0.0f;
                }
                for (int k = lane; k < n; k += 32)
#pragma unroll
                    for (int q = 0; q < kMine; ++q) {
                        const float m = stat(k, q);
                        factor[(warp + q * kWarps) * n + k] = m;
                        top[q] = fmaxf(top[q], m);
                    }
#pragma unroll
                for (int q = 0; q < kMine; ++q)
#pragma unroll
                    for (int d = 16; d; d >>= 1) top[q] = fmaxf(top[q], __shfl_xor_sync(~0u, top[q], d));
                for (int k = lane; k < n; k += 32)
#pragma unroll
                    for (int q = 0; q < kMine; ++q) {
                        const float f = top[q] == -CUDART_INF_F ? 1.0f : exp2_fast(factor[(warp + q * kWarps) * n + k] - top[q]);
                        factor[(warp + q * kWarps) * n + k] = f;
                        sum[q] += (k < 32 ? sum0[q] : stat(k, q + kMine)) * f;
                    }
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
#pragma unroll
                    for (int d = 16; d; d >>= 1) sum[q] += __shfl_xor_sync(~0u, sum[q], d);
                    if (lane == 0) {
                        row_top[warp + q * kWarps] = top[q];
                        row_sum[warp + q * kWarps] = sum[q];
                    }
                }
                __syncthreads();
                float2 x[kPairs];
#pragma unroll
                for (int j = 0; j < kPairs; ++j) x[j] = make_float2(0.0f, 0.0f);
                for (int k0 = 0; k0 < n; k0 += kBatch) {
                    if (k0) fetch(k0);
#pragma unroll
                    for (int q = 0; q < kBatch; ++q)
#pragma unroll
                        for (int j = 0; j < kPairs; ++j)
                            if (k0 + q < n) {
                                const float f = factor[((threadIdx.x + j * kThreads) >> 3) % kRows * n + k0 + q];
                                x[j].x = fmaf(v[q][j].x, f, x[j].x);
                                x[j].y = fmaf(v[q][j].y, f, x[j].y);
                            }
                }
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const int i = threadIdx.x + j * kThreads, r = (i >> 3) % kRows;
                    finish(i, x[j].x, x[j].y, row_top[r], row_sum[r]);
                }
            }
        }
        seg_at += rq.units();
        if (seg_at >= end) break;
        ++seg;
        from = 0;
        __syncthreads();  // the ring is free again
    }
}

template <int kDim, int kRows, int kStep, int kWarps, int kStages, int kMinCtas>
static cudaError_t launch_attention(const AttnArgs& a, int sms, cudaStream_t st)
{
    using T = Attn<kDim, kRows, kStep, kWarps, kStages>;
    auto kernel = attention_kernel<kDim, kRows, kStep, kWarps, kStages, kMinCtas>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return e;
    // no more blocks than can have a step each (an upper bound that the host knows)
    int64_t most = (int64_t)a.B * a.c.kv_heads * (((int64_t)a.max_q * a.group + kRows - 1) / kRows);
    const int64_t steps = kBeginKeys / T::kStep + ((int64_t)a.max_blocks * a.c.page_size + T::kStep - 1) / T::kStep;
    const int64_t units = 2 * steps;  // 16-row tiles: 4 a step, of which a warp's least is 2
    most = most > kAttnMaxCtas || most * units > (int64_t)kAttnMaxCtas * kWarps ? kAttnMaxCtas : (most * units + kWarps - 1) / kWarps;
    const int64_t full = sms * kMinCtas < kAttnMaxCtas ? sms * kMinCtas : kAttnMaxCtas;
    kernel<<<(unsigned)(most < full ? most : full), kWarps * 32, T::kSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace nvq

using namespace nvq;

extern "C" size_t nvfp4_kv_attention_workspace_size(void) 
{
    return (size_t)kAttnMaxCtas * (2 * kPieceFloats * sizeof(float) + sizeof(uint32_t));
}

extern "C" nvq_status nvfp4_kv_attention(const nvq_kv_cache* cache, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                                         int64_t rows, int32_t heads, const int32_t* q_off, int32_t B, int32_t max_q,
                                         const int32_t* kv_len, const int32_t* block_table, int64_t ld_table,
                                         int32_t max_blocks, float sm_scale, int32_t window, void* out,
                                         int64_t out_stride_t, int64_t out_stride_h, float* lse, void* workspace,
                                         size_t workspace_bytes, void* stream)
{
    NVQ_TRACE("nvfp4_kv_attention");
    const nvq_status s = check_cache(cache, "nvfp4_kv_attention");
    if (s != NVQ_OK) return s;
    NVQ_CHECK_ARG(q && kv_len && block_table && out && workspace, NVQ_ERR_ARG, "nvfp4_kv_attention: null pointer argument");
    NVQ_CHECK_ARG(isfinite(sm_scale) && window >= 0, NVQ_ERR_ARG, "nvfp4_kv_attention: sm_scale not finite or window < 0");
    NVQ_CHECK_ARG(heads >= 1 && heads <= 65535 && heads % cache->kv_heads == 0, NVQ_ERR_SHAPE,
                  "nvfp4_kv_attention: heads must be a multiple of kv_heads, at most 65535");
    NVQ_CHECK_ARG(B >= 1 && B <= (1 << 20) && max_q >= 1 && max_q <= 65535 && rows >= 1 && rows < (1ll << 31), NVQ_ERR_SHAPE,
                  "nvfp4_kv_attention: B outside [1, 2^20], max_q outside [1, 65535] or rows outside [1, 2^31)");
    NVQ_CHECK_ARG(q_off || B <= rows, NVQ_ERR_SHAPE, "nvfp4_kv_attention: more requests than query rows without q_off");
    NVQ_CHECK_ARG(max_blocks >= 1 && ld_table >= max_blocks && (int64_t)max_blocks * cache->page_size < (1ll << 31), NVQ_ERR_SHAPE,
                  "nvfp4_kv_attention: max_blocks < 1, ld_table < max_blocks, or max_blocks * page_size >= 2^31");
    // a row tile has 8 rows at least if there are as many, a step 32 keys and 4 units at most
    NVQ_CHECK_ARG((int64_t)max_q * heads <= (1 << 30) &&
                      (double)B * cache->kv_heads * ((int64_t)max_q * (heads / cache->kv_heads) / 8 + 1) *
                              ((double)max_blocks * cache->page_size / 8 + 64) < kMaxUnits,
                  NVQ_ERR_SHAPE, "nvfp4_kv_attention: heads * max_q above 2^30, or B * heads * max_q * max_blocks * page_size beyond the units of work");
    NVQ_CHECK_ARG(q_stride_t >= 0 && q_stride_h >= 0 && out_stride_t >= 0 && out_stride_h >= cache->head_dim, NVQ_ERR_SHAPE,
                  "nvfp4_kv_attention: a negative stride, or heads of out that overlap");
    NVQ_CHECK_ARG(q_stride_t % 8 == 0 && q_stride_h % 8 == 0 && out_stride_t % 8 == 0 && out_stride_h % 8 == 0 && aligned(q, 16) &&
                      aligned(out, 16) && aligned(lse, 4) && aligned(q_off, 4) && aligned(kv_len, 4) && aligned(block_table, 4),
                  NVQ_ERR_ALIGN, "nvfp4_kv_attention: q and out need 16-byte aligned rows");
    NVQ_CHECK_ARG(workspace_bytes >= nvfp4_kv_attention_workspace_size() && aligned(workspace, 16), NVQ_ERR_SHAPE,
                  "nvfp4_kv_attention: workspace of %zu bytes, or not 16-byte aligned: %zu are needed", workspace_bytes,
                  nvfp4_kv_attention_workspace_size());
    DeviceStatus* dst = device_status_ptr();
    NVQ_CHECK_ARG(dst, NVQ_ERR_CUDA, "nvfp4_kv_attention: device status word unavailable");
    set_error("");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e, "nvfp4_kv_attention: device attributes");
    const int gran = cache->page_size / 16;
    float* pieces = static_cast<float*>(workspace);
    AttnArgs a{*cache, static_cast<const __nv_bfloat16*>(q), q_stride_t, q_stride_h, rows, heads, heads / cache->kv_heads, q_off, B,
               max_q, kv_len, block_table, ld_table, max_blocks, sm_scale, window, static_cast<__nv_bfloat16*>(out), out_stride_t,
               out_stride_h, lse, pieces, reinterpret_cast<uint32_t*>(pieces + (size_t)kAttnMaxCtas * 2 * kPieceFloats),
               (gran & (gran - 1)) == 0 ? __builtin_ctz(gran) : -1, dst};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // 8-row tiles where a request's heads and new tokens fit them.  Steps of 64 keys cost fewer
    // instructions a key; of 128 values a key they halve the blocks' number of steps, so they are
    // taken where the tables allow 32 steps a warp (64 requests of 65536 keys 488 -> 452 us as they
    // were; a single request of 1000 keys takes 9 us in steps of 32, 11 in steps of 64).  16-row tiles
    // of 128 values have registers for two blocks an SM: a request of 100k keys with 4 new tokens 54 us
    // so, 76 with three blocks that spill; 64 requests of 16384 keys and 16 heads a group 192 and 185.
    const bool narrow = (int64_t)max_q * a.group <= 8;
    const int64_t keys = (int64_t)B * cache->kv_heads * max_blocks * cache->page_size;
    switch (cache->head_dim) {
        case 64: e = narrow ? launch_attention<64, 8, 64, 4, 3, 3>(a, sms, st) : launch_attention<64, 16, 64, 4, 3, 3>(a, sms, st); break;
        case 128:
            e = !narrow                                   ? launch_attention<128, 16, 64, 4, 2, 2>(a, sms, st)
                : keys >= (int64_t)sms * 12 * 32 * 64 ? launch_attention<128, 8, 64, 4, 2, 3>(a, sms, st)
                                                          : launch_attention<128, 8, 32, 4, 3, 3>(a, sms, st);
            break;
        default: e = launch_attention<256, 8, 32, 4, 2, 2>(a, sms, st); break;
    }
    if (e != cudaSuccess) return cuda_status(e, "attention_kernel");
    return NVQ_OK;
}
