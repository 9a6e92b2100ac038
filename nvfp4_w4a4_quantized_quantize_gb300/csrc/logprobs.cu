// logprobs.cu -- log-probabilities of given tokens with entropy and top alternatives
// (token_logprobs), and the gradient of the first two (token_logprobs_backward).
//
// With z = scale * logits of a row, m = max z, s = sum exp(z - m), u = sum exp(z - m) (z - m):
//   lse = m + log s,  entropy = log s - u / s,  logprob = z_target - lse,
//   d/dlogit_j = scale * (g_lp [j = target] - p_j (g_lp + g_H (z_j - lse + entropy))).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "common.cuh"

namespace nvq {

constexpr int kWhereTarget = 50;
constexpr int kMaxTop = 32;

struct LogprobArgs {
    const void* logits;
    int64_t rows, V, ld;
    const int64_t* targets;
    float scale;
    int32_t top_n;
    float *logprob, *entropy, *lse;
    int32_t* top_ids;
    float* top_lp;
    DeviceStatus* status;
};

struct LogprobGradArgs {
    const void* logits;
    int64_t rows, V, ld;
    const int64_t* targets;
    float scale;
    const float *lse, *entropy, *g_logprob, *g_entropy;
    void* grad;
    int64_t ld_grad;
    DeviceStatus* status;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A total order of (logit, index): larger logits first, then lower indices.  The logit's bits as
// an unsigned number that ascends with it (-0 and +0 alike), above the complement of the index.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t j)
{
    uint32_t u = x == x ? __float_as_uint(x + 0.0f) : 0x7fffffffu;  // NaN above everything
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)u << 32) | (uint32_t)~j;
}

// Logits from which the one-pass form takes a row, and what masked logits count as in it: low enough
// that their weight is 0 beside any logit above -kMaxLogit, high enough that nothing overflows.
constexpr float kMaxLogit = 1208925819614629174706176.0f, kClamp = -8.0f * kMaxLogit;  // 2^80, -2^83

// ------------------------------------------------------------------ vectors of a row
// A row is read in 16-byte vectors that lie on 16-byte boundaries: vector i holds elements
// [i * kWidth - head, ...) of the row, head = elements between the boundary below and the row.
template <class T>
struct Vec {
    static constexpr int kWidth = 16 / sizeof(T);
    uint32_t u[4];
    __device__ __forceinline__ float at(int e) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(u[e]);
        return (e & 1) ? bf16hi(u[e >> 1]) : bf16lo(u[e >> 1]);
    }
    __device__ __forceinline__ float largest() const  // NaNs left out, unless all are
    {
        if constexpr (sizeof(T) == 4) return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3)));
        uint32_t m;
        asm("{\n\t.reg .b32 p, q;\n\tmax.bf16x2 p, %1, %2;\n\tmax.bf16x2 q, %3, %4;\n\tmax.bf16x2 %0, p, q;\n\t}"
            : "=r"(m)
            : "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]));
        return fmaxf(bf16lo(m), bf16hi(m));
    }
    // Elements below kClamp (masked logits) become kClamp; NaNs stay.
    __device__ __forceinline__ Vec clamped() const
    {
        Vec v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4)
                asm("max.NaN.f32 %0, %1, %2;" : "=f"(reinterpret_cast<float&>(v.u[k])) : "f"(__uint_as_float(u[k])), "f"(kClamp));
            else
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(v.u[k]) : "r"(u[k]), "r"((__float_as_uint(kClamp) & 0xffff0000u) | (__float_as_uint(kClamp) >> 16)));
        }
        return v;
    }
};

template <class T>
struct Row {
    static constexpr int kWidth = Vec<T>::kWidth;
    const T* x;       // first element
    int head;         // elements of vector 0 before it
    int V;
    int lo, hi;       // vectors that lie within the row
    __device__ __forceinline__ Row(const void* logits, int64_t t, int64_t ld, int64_t V_) : x(static_cast<const T*>(logits) + t * ld), V((int)V_)
    {
        head = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
        lo = head ? 1 : 0;
        hi = (int)((V_ + head) / kWidth);
    }
    __device__ __forceinline__ int vectors() const { return (int)(((int64_t)V + head + kWidth - 1) / kWidth); }
    __device__ __forceinline__ bool inside(int i) const { return i >= lo && i < hi; }
    __device__ __forceinline__ int64_t element(int i, int e) const { return (int64_t)i * kWidth + e - head; }
    __device__ __forceinline__ Vec<T> load_whole(int i) const
    {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(x - head) + i);
        return {{w.x, w.y, w.z, w.w}};
    }
    // A vector of the row; of one that reaches beyond it its own elements, and -inf for the others.
    __device__ __forceinline__ Vec<T> load(int i) const
    {
        if (inside(i)) return load_whole(i);
        Vec<T> v;
        constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80u;
        v.u[0] = v.u[1] = v.u[2] = v.u[3] = 0;
#pragma unroll
        for (int e = 0; e < kWidth; ++e) {
            const int64_t j = element(i, e);
            uint32_t b = none;
            if (j >= 0 && j < V) {
                if constexpr (sizeof(T) == 4)
                    b = reinterpret_cast<const uint32_t*>(x)[j];
                else
                    b = reinterpret_cast<const uint16_t*>(x)[j];
            }
            if constexpr (sizeof(T) == 4)
                v.u[e] = b;
            else
                v.u[e >> 1] |= b << (16 * (e & 1));
        }
        return v;
    }
};

// ------------------------------------------------------------------ forward
constexpr int kMaxThreads = 512;
constexpr int kUnroll = 4;
constexpr int kCandidates = 1024;
constexpr float kHuge = 2147483648.0f;  // 2^31: an fp32 lse from here on cannot hold the logarithm of a sum
__device__ __forceinline__ float key_value(uint64_t key)  // the logit of an order_key (+0 for -0)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// Sums of a part of a row, in units of log2 relative to a whole number: s = sum 2^(z' - ref),
// u = sum 2^(z' - ref) (z' - ref), z' = scale * log2(e) * logit.
struct Sums {
    float ref, s, u;
};

__device__ __forceinline__ float pow2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ Sums join(const Sums& a, const Sums& b)
{
    // a part without elements has ref = -inf and s = u = 0
    const float ref = fmaxf(a.ref, b.ref);
    if (ref == -CUDART_INF_F) return {ref, a.s + b.s, a.u + b.u};
    const float da = a.ref - ref, db = b.ref - ref, fa = pow2(da), fb = pow2(db);
    const float ua = a.ref == -CUDART_INF_F ? 0.0f : (a.u + da * a.s) * fa, ub = b.ref == -CUDART_INF_F ? 0.0f : (b.u + db * b.s) * fb;
    return {ref, a.s * fa + b.s * fb, ua + ub};
}

__device__ __forceinline__ Sums warp_join(Sums v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const Sums o = {__shfl_xor_sync(~0u, v.ref, d), __shfl_xor_sync(~0u, v.s, d), __shfl_xor_sync(~0u, v.u, d)};
        v = join(v, o);
    }
    return v;
}

__device__ __forceinline__ uint64_t key_max(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t warp_key_max(uint64_t k)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) k = key_max(k, __shfl_xor_sync(~0u, k, d));
    return k;
}

struct alignas(16) ForwardShared {
    uint64_t cand[kCandidates];
    uint64_t top[kMaxTop];            // the part's alternatives, largest first
    int32_t count, readers;
    uint32_t least;
    uint32_t first[kMaxTop + kMaxThreads / 32];
    uint16_t reader[kMaxThreads];
    Sums warp_sums[kMaxThreads / 32];
    Sums sums;
    uint64_t warp_key[kMaxThreads / 32];
    uint64_t best;                    // the part's largest logit, as a key
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// An address of this block's shared memory as it is in block `rank` of the cluster.
template <class P>
__device__ __forceinline__ uint32_t peer(const P* p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint64_t peer_u64(uint32_t a)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float peer_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// use(key, rank) for each of `count` keys in shared memory, equal ones in their order; four lanes compare one.
template <class F>
__device__ __forceinline__ void for_ranks(const uint64_t* keys, int count, F&& use)
{
    for (int i = threadIdx.x; (i & ~31) < 4 * count; i += blockDim.x) {
        const int k = min(i >> 2, count - 1);
        const uint64_t key = keys[k];
        int rank = 0;
        for (int o = i & 3; o < count; o += 4) rank += keys[o] > key || (keys[o] == key && o < k);
        rank += __shfl_xor_sync(~0u, rank, 1);
        rank += __shfl_xor_sync(~0u, rank, 2);
        if ((i & 3) == 0 && i < 4 * count) use(key, rank);
    }
}

// The n largest keys of this block's vectors [v0, v1); thread t has read vectors v0 + t + k * threads
// and brings the largest of its logits.  The warps' k largest of those, k * warps >= n, hold n
// logits of at least their n-th largest, `least`; so the n largest of all are among the logits not
// below it, which lie in the vectors of the few threads whose largest is not.  Those are read
// again (by all threads, one vector each) and ranked against each other.
template <class T>
__device__ void part_top(ForwardShared& sh, const Row<T>& row, int v0, int v1, int n, uint64_t mine)
{
    constexpr int kWidth = Vec<T>::kWidth;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x, warps = threads >> 5;
    const uint32_t value = (uint32_t)(mine >> 32);
    uint32_t left = value;
    int firsts = 0;
    for (; firsts < n; firsts += warps) {
        const uint32_t m = __reduce_max_sync(~0u, left);
        const uint32_t who = __ballot_sync(~0u, left == m);
        if (lane == __ffs(who) - 1) left = 0;
        if (lane == 0) sh.first[firsts + warp] = m;
    }
    if (threadIdx.x == 0) sh.count = sh.readers = 0;
    if ((int)threadIdx.x < n) sh.top[threadIdx.x] = 0;
    __syncthreads();
    if ((int)threadIdx.x < firsts) {
        const uint32_t m = sh.first[threadIdx.x];
        int rank = 0;
        for (int o = 0; o < firsts; ++o) rank += sh.first[o] > m || (sh.first[o] == m && o < (int)threadIdx.x);
        if (rank == n - 1) sh.least = m;
    }
    __syncthreads();
    const uint32_t least = sh.least;
    if (value >= least) sh.reader[atomicAdd(&sh.readers, 1)] = (uint16_t)threadIdx.x;
    __syncthreads();
    const int readers = sh.readers;
    int shift = 0;  // a reader's vectors, rounded up to a power of two
    while ((threads << shift) < v1 - v0) ++shift;
    for (int f = threadIdx.x; f < readers << shift; f += threads) {
        const int i = v0 + sh.reader[f >> shift] + (f & ((1 << shift) - 1)) * threads;
        if (i >= v1) continue;
        const Vec<T> v = row.load(i);
#pragma unroll
        for (int e = 0; e < kWidth; ++e) {
            const int64_t j = row.element(i, e);
            const uint64_t key = order_key(v.at(e), (uint32_t)j);
            if ((uint32_t)(key >> 32) >= least && j >= 0 && j < row.V) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCandidates) sh.cand[at] = key;
            }
        }
    }
    __syncthreads();
    const int count = sh.count;
    if (count <= kCandidates) {
        for_ranks(sh.cand, count, [&](uint64_t key, int rank) {
            if (rank < n) sh.top[rank] = key;
        });
    } else {
        // Many equal logits (most of a row masked, say): one alternative at a time.  The warp of the
        // thread that has the largest left reads that thread's vectors again for its next.
        uint64_t next = 0;
        auto rescan = [&](int thread, uint64_t below) {  // by the whole warp: the largest key under `below`
            uint64_t best = 0;
            for (int i = v0 + thread + lane * threads; i < v1; i += 32 * threads) {
                const Vec<T> v = row.load(i);
#pragma unroll
                for (int e = 0; e < kWidth; ++e) {
                    const int64_t j = row.element(i, e);
                    const uint64_t key = order_key(v.at(e), (uint32_t)j);
                    if (key < below && j >= 0 && j < row.V) best = key_max(best, key);
                }
            }
            return warp_key_max(best);
        };
        for (int l = 0; l < 32; ++l) {  // the threads' exact keys (so far they name a vector)
            const uint64_t k = rescan(warp * 32 + l, ~0ull);
            if (lane == l) next = k;
        }
        for (int i = 0; i < n; ++i) {
            const uint64_t w = warp_key_max(next);
            __syncthreads();
            if (lane == 0) sh.warp_key[warp] = w;
            __syncthreads();
            const uint64_t best = warp_key_max(lane < warps ? sh.warp_key[lane] : 0);
            if (threadIdx.x == 0) sh.top[i] = best;
            const uint32_t who = __ballot_sync(~0u, next == best && best);
            if (who) {
                const int l = __ffs(who) - 1;
                const uint64_t k = rescan(warp * 32 + l, best);
                if (lane == l) next = k;
            }
        }
    }
    __syncthreads();
}

// A cluster per row, each of its blocks a part (1 block when there are rows enough).  One pass:
// every thread keeps sums relative to a whole power of two at or above its first vector's
// maximum, moved only when a logit passes it by 2^60 (fp32 sums have the range), so that an
// element costs one multiply-add, one exp2 and two accumulations.
// Measured: 4096 rows of 131072 bf16 logits (1.07 GB) in 159 us = 6.75 TB/s, a copy's rate, so bound by
// HBM; 64 rows of 131072 fp32 logits with the 20 largest (34 MB) in 12.9 us, bound by latency (a pass of
// 5 us, the join in the cluster and the choice of the largest).
template <class T, bool kTop>
__global__ void __launch_bounds__(kMaxThreads, kTop ? 2 : 4) logprob_kernel(const __grid_constant__ LogprobArgs a, int parts, int wide)
{
    constexpr int kWidth = Vec<T>::kWidth;
    __shared__ ForwardShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x, warps = threads >> 5;
    const int64_t t = blockIdx.x / (unsigned)parts;
    const uint32_t rank = parts > 1 ? cluster_rank() : 0;
    const int n = a.top_n;
    int64_t target = a.targets ? a.targets[t] : 0;
    if (target >= a.V) {
        if (threadIdx.x == 0 && rank == 0) report_status(a.status, NVQ_ERR_ARG, kWhereTarget);
        target = -1;
    }
    if (target < 0) {  // the whole cluster leaves
        if (rank == 0) {
            if (threadIdx.x == 0) {
                if (a.logprob) a.logprob[t] = 0.0f;
                if (a.entropy) a.entropy[t] = 0.0f;
                if (a.lse) a.lse[t] = 0.0f;
            }
            if ((int)threadIdx.x < n) {
                a.top_ids[t * n + threadIdx.x] = -1;
                a.top_lp[t * n + threadIdx.x] = -CUDART_INF_F;
            }
        }
        return;
    }
    const Row<T> row(a.logits, t, a.ld, a.V);
    const int64_t all = row.vectors();
    const int v0 = (int)(all * rank / parts), v1 = (int)(all * (rank + 1) / parts);
    const float c = a.scale * 1.4426950408889634f;

    const float x_target = to_f32(row.x[target]);

    Sums sum = {-CUDART_INF_F, 0.0f, 0.0f};
    float best = -CUDART_INF_F;
    int best_at = -1;
    auto note = [&](float top, int i) {
        if constexpr (kTop) {
            if (top > best || best_at < 0) {
                best = top;
                best_at = i;
            }
        } else {
            best = fmaxf(best, top);
            best_at = 0;
        }
    };
    auto take = [&](const Vec<T>& v, int i) {
        const float top = v.largest();
        note(top, i);
        if (!(fmaf(top, c, -sum.ref) <= 60.0f)) {  // the first vector too, whatever it holds
            const float ref = ceilf(fminf(fmaxf(top, kClamp), kMaxLogit) * c);
            if (sum.ref > -CUDART_INF_F) {
                const float d = sum.ref - ref, f = pow2(d);
                sum.u = (sum.u + d * sum.s) * f;
                sum.s *= f;
            }
            sum.ref = ref;
        }
        const Vec<T> x = v.clamped();
#pragma unroll
        for (int e = 0; e < kWidth; ++e) {
            const float y = fmaf(x.at(e), c, -sum.ref), p = pow2(y);
            sum.s += p;
            sum.u = fmaf(p, y, sum.u);
        }
    };
    int i = v0 + threadIdx.x;
    if (!wide) {
        if (i < row.lo && i < v1) {
            take(row.load(i), i);
            i += threads;
        }
        const int whole = min(v1, row.hi);
        for (; i + (kUnroll - 1) * threads < whole; i += kUnroll * threads) {
            Vec<T> v[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) v[k] = row.load_whole(i + k * threads);
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) take(v[k], i + k * threads);
        }
        for (; i < v1; i += threads) take(row.load(i), i);
    } else {
        for (; i < v1; i += threads) note(row.load(i).largest(), i);
    }

    // ---- join the threads, then the blocks
    const uint64_t my_key = best_at < 0 ? 0 : order_key(best, (uint32_t)max(row.element(best_at, 0), (int64_t)0));
    const uint64_t wk = warp_key_max(my_key);
    const Sums ws = warp_join(sum);
    if (lane == 0) {
        sh.warp_key[warp] = wk;
        sh.warp_sums[warp] = ws;
    }
    __syncthreads();
    if (warp == 0) {
        const uint64_t k = warp_key_max(lane < warps ? sh.warp_key[lane] : 0);
        const Sums v = warp_join(lane < warps ? sh.warp_sums[lane] : Sums{-CUDART_INF_F, 0.0f, 0.0f});
        if (lane == 0) {
            sh.sums = v;
            sh.best = k;
        }
    }
    __syncthreads();
    uint64_t row_key = sh.best;
    if (kTop) part_top(sh, row, v0, v1, n, my_key);
    if (parts > 1) {
        cluster_sync();
        row_key = 0;
        for (int r = 0; r < parts; ++r) row_key = key_max(row_key, peer_u64(peer(&sh.best, r)));
    }
    // the row's largest logit, from its key
    const float top = key_value(row_key);
    // Rows outside the one-pass form's range (nothing but masks, or huge logits), and every row where
    // scale is: a second pass over differences, which are exact where they matter.
    const bool again = wide || !(fabsf(top) < kMaxLogit && fabsf(top * a.scale) < kHuge / 2);
    if (again) {
        Sums v = {0.0f, 0.0f, 0.0f};
        const float base = top == -CUDART_INF_F ? 0.0f : top;
        for (int k = v0 + threadIdx.x; k < v1; k += threads) {
            const Vec<T> w = row.load(k);
#pragma unroll
            for (int e = 0; e < kWidth; ++e) {
                const float y = (w.at(e) - base) * a.scale * 1.4426950408889634f, p = pow2(y);
                v.s += p;
                v.u += p == 0.0f ? 0.0f : p * y;
            }
        }
        v = warp_join(v);
        __syncthreads();
        if (lane == 0) sh.warp_sums[warp] = v;
        __syncthreads();
        if (warp == 0) {
            v = warp_join(lane < warps ? sh.warp_sums[lane] : Sums{0.0f, 0.0f, 0.0f});
            if (lane == 0) sh.sums = v;
        }
        __syncthreads();
        if (parts > 1) cluster_sync();  // the whole cluster is here: all see the same largest logit
    }
    if (rank == 0) {
        Sums v = sh.sums;
        for (int r = 1; r < parts; ++r) {
            const uint32_t p = peer(&sh.sums, r);
            v = join(v, Sums{peer_f32(p), peer_f32(p + 4), peer_f32(p + 8)});
        }
        const bool none = top == -CUDART_INF_F && v.s == 0.0f;
        const float ls = log2f(v.s);
        // logits relative to lse, in units of log2: the reference is a whole number or the row's maximum
        auto relative = [&](float x) {
            const float z = again ? (x - top) * a.scale * 1.4426950408889634f : fmaf(x, c, -v.ref);
            return (z - ls) * 0.6931471805599453f;
        };
        if (threadIdx.x == 0) {
            const float z = __fmul_rn(top, a.scale);  // beyond kHuge the lse rounds to the largest logit: made exact for the gradient
            const float lse = !again ? (v.ref + ls) * 0.6931471805599453f : fabsf(z) >= kHuge && ls == ls ? z : fmaf(top, a.scale, ls * 0.6931471805599453f);
            if (a.lse) a.lse[t] = none ? -CUDART_INF_F : lse;
            if (a.entropy) a.entropy[t] = none ? 0.0f : fmaxf((ls - v.u / v.s), v.s != v.s ? CUDART_NAN_F : 0.0f) * 0.6931471805599453f;
            if (a.logprob) a.logprob[t] = none ? -CUDART_INF_F : relative(x_target);
        }
        if (kTop) {
            // rank the parts' alternatives against each other
            for (int i = threadIdx.x; i < parts * n; i += threads) sh.cand[i] = parts > 1 ? peer_u64(peer(&sh.top[i % n], i / n)) : sh.top[i];
            __syncthreads();
            for_ranks(sh.cand, parts * n, [&](uint64_t mine, int before) {
                if (before < n) {
                    const int64_t j = min((int64_t)(uint32_t)~(uint32_t)mine, a.V - 1);
                    a.top_ids[t * n + before] = (int32_t)j;
                    a.top_lp[t * n + before] = none ? -CUDART_INF_F : relative(key_value(mine));
                }
            });
        }
    }
    if (parts > 1) cluster_sync();  // no block ends while another reads its shared memory
}

// ------------------------------------------------------------------ gradient
// A stream: p_j from the row's lse, two multiply-adds, one write.  blockIdx.y takes a stretch of the
// row's vectors.  Where the gradient's rows do not lie on the same 16-byte grid as the logits',
// elements are written one by one.
// An lse far from zero is rounded by more than the weights may be off: fp32 holds it to 2^-23 of its
// size (with the forward's roundings), 2 at 2^24.  From kRounded on, where that is 2^-15, the row's weights
// are made independent of it: p = exp(z - lse) / sum exp(z - lse), whose differences are exact where
// they matter.  One block then takes the whole row, as grad may be logits: it has read all of the row
// before it writes.
// Measured: 4096 rows of 131072 bf16 logits (1.07 GB read, as much written) in 325 us = 6.6 TB/s, 0.97 of
// a copy; 2000 rows of 50003 in 62 us = 6.4 TB/s (odd rows begin off the 16-byte grid).  With 1000 added to
// every logit (the row read twice, by one block): 4096 rows 496 us for 338 with cold caches, 64 fp32 rows of
// 131072 66 for 19.
constexpr int kGradThreads = 256, kGradUnroll = 4, kGradPerThread = 16;
constexpr float kRounded = 256.0f;

// z = scale * logit relative to lse.  A masked logit goes far below all others: weight 0, and no 0 * inf.
__device__ __forceinline__ float grad_relative(float x, float scale, float lse, bool huge)
{
    float z = huge ? __fmul_rn(x, scale) - lse : fmaf(x, scale, -lse);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(z) : "f"(kClamp));
    return z;
}

// log sum exp(scale * logit - lse) of a row, by the whole block: sums relative to the largest term so far, as the
// terms are off by lse's rounding, up to 2^7 near kHuge.  (Not inlined: its registers would cost the stream a tenth.)
template <class T>
__device__ __noinline__ float row_correction(const T* x, int64_t V, float scale, float lse)
{
    __shared__ float maxima[kGradThreads / 32], sums[kGradThreads / 32];
    const Row<T> row(x, 0, 0, V);
    constexpr int kWidth = Vec<T>::kWidth;
    constexpr float kLog2e = 1.4426950408889634f;
    float m = -CUDART_INF_F, s = 0.0f;
    auto take = [&](const Vec<T>& v) {
        const float top = grad_relative(v.largest(), scale, lse, false);
        if (top > m) {
            s *= pow2((m - top) * kLog2e);
            m = top;
        }
        float part = 0.0f;
#pragma unroll
        for (int e = 0; e < kWidth; ++e) part += pow2((grad_relative(v.at(e), scale, lse, false) - m) * kLog2e);
        s += part;
    };
    const int all = row.vectors();
    int i = threadIdx.x;
    if (i < row.lo && i < all) {
        take(row.load(i));
        i += kGradThreads;
    }
    for (; i + (kGradUnroll - 1) * kGradThreads < row.hi; i += kGradUnroll * kGradThreads) {
        Vec<T> v[kGradUnroll];
#pragma unroll
        for (int k = 0; k < kGradUnroll; ++k) v[k] = row.load_whole(i + k * kGradThreads);
#pragma unroll
        for (int k = 0; k < kGradUnroll; ++k) take(v[k]);
    }
    for (; i < all; i += kGradThreads) take(row.load(i));
    auto join = [](float& m, float& s, float om, float os) {  // of parts without vectors m is -inf, s 0
        const float top = fmaxf(m, om);
        s = (m == top ? s : s * pow2((m - top) * kLog2e)) + (om == top ? os : os * pow2((om - top) * kLog2e));
        m = top;
    };
#pragma unroll
    for (int d = 16; d; d >>= 1) join(m, s, __shfl_xor_sync(~0u, m, d), __shfl_xor_sync(~0u, s, d));
    if (threadIdx.x % 32 == 0) {
        maxima[threadIdx.x / 32] = m;
        sums[threadIdx.x / 32] = s;
    }
    __syncthreads();
    m = maxima[0];
    s = sums[0];
    for (int w = 1; w < kGradThreads / 32; ++w) join(m, s, maxima[w], sums[w]);
    return m + logf(s);
}

template <class T>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const __grid_constant__ LogprobGradArgs a)
{
    constexpr int kWidth = Vec<T>::kWidth;
    const int64_t t = blockIdx.x;
    const Row<T> row(a.logits, t, a.ld, a.V);
    T* g = static_cast<T*>(a.grad) + t * a.ld_grad;
    const bool same_grid = reinterpret_cast<uintptr_t>(g) % 16 == reinterpret_cast<uintptr_t>(row.x) % 16;
    int64_t target = a.targets ? a.targets[t] : 0;
    if (target >= a.V) {
        if (threadIdx.x == 0 && blockIdx.y == 0) report_status(a.status, NVQ_ERR_ARG, kWhereTarget);
        target = -1;
    }
    const float lse = a.lse[t], h = a.entropy[t];
    const bool skip = target < 0 || lse == -CUDART_INF_F;
    const float glp = a.g_logprob ? a.g_logprob[t] : 0.0f, gh = a.g_entropy ? a.g_entropy[t] : 0.0f;
    // From kHuge on the lse is the largest logit itself: the weights are even over the logits equal
    // to it, and the entropy is the logarithm of their number.
    const bool huge = fabsf(lse) >= kHuge;
    float bias = huge ? h : 0.0f;
    // the row's vectors in even stretches
    const int all = row.vectors();
    int first = (int)((int64_t)all * blockIdx.y / gridDim.y), last = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y);
    if (!skip && !huge && fabsf(lse) >= kRounded) {
        if (blockIdx.y) return;
        first = 0;
        last = all;
        bias = row_correction(row.x, a.V, a.scale, lse);
    }
    // weights are formed times 2^24, the slope times 2^-24: exp2 flushes what is below 2^-126
    const float bias2 = 24.0f - bias * 1.4426950408889634f;
    const float c1 = -gh * a.scale * 5.9604644775390625e-8f, c0 = -(glp + gh * (h - bias)) * a.scale * 5.9604644775390625e-8f;
    auto slope = [&](float x) {
        const float z = grad_relative(x, a.scale, lse, huge), p = pow2(fmaf(z, 1.4426950408889634f, bias2));
        return p * fmaf(c1, z, c0);
    };
    const int64_t tv = a.targets && !skip ? (target + row.head) / kWidth : -1;  // the target's vector
    auto put = [&](const Vec<T>& v, int i) {
        float d[kWidth];
#pragma unroll
        for (int e = 0; e < kWidth; ++e) d[e] = skip ? 0.0f : slope(v.at(e));
        if (i == tv) {
#pragma unroll
            for (int e = 0; e < kWidth; ++e)
                if (row.element(i, e) == target) d[e] += glp * a.scale;
        }
        if (same_grid && row.inside(i)) {
            uint4 w;
            if constexpr (sizeof(T) == 4) {
                w = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
            } else {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(d[2 * e], d[2 * e + 1]);
                    u[e] = *reinterpret_cast<const uint32_t*>(&b);
                }
                w = make_uint4(u[0], u[1], u[2], u[3]);
            }
            __stcs(reinterpret_cast<uint4*>(g - row.head) + i, w);
        } else {
#pragma unroll
            for (int e = 0; e < kWidth; ++e) {
                const int64_t j = row.element(i, e);
                if (j >= 0 && j < a.V) from_f32(g + j, d[e]);
            }
        }
    };
    // a thread's loads go out together, before its first write (grad may be logits)
    for (int i0 = first + threadIdx.x; i0 < last; i0 += kGradThreads * kGradUnroll) {
        Vec<T> v[kGradUnroll];
        const bool whole = i0 >= row.lo && i0 + (kGradUnroll - 1) * kGradThreads < min(last, row.hi);
        if (whole && !skip) {
#pragma unroll
            for (int k = 0; k < kGradUnroll; ++k) v[k] = row.load_whole(i0 + k * kGradThreads);
        } else {
#pragma unroll
            for (int k = 0; k < kGradUnroll; ++k)
                if (i0 + k * kGradThreads < last && !skip) v[k] = row.load(i0 + k * kGradThreads);
        }
#pragma unroll
        for (int k = 0; k < kGradUnroll; ++k)
            if (whole || i0 + k * kGradThreads < last) put(v[k], i0 + k * kGradThreads);
    }
}

template <class T>
static cudaError_t launch_forward(const LogprobArgs& a, int sms, cudaStream_t st)
{
    // Parts: blocks of a cluster per row, doubled while all are resident at once (two an SM) and a part
    // keeps 128 KB, or 64 KB if every block has an SM to itself: 64 rows of 131072 fp32 logits took
    // 9.4 us in 4 parts, 10.3 in 2 and 13.3 in 8; 24 of 50000 with the 20 largest 9.4 us in one, 13.7 in 8.
    int parts = 1;
    while (parts < 4 && a.rows * parts <= sms && a.V * (int64_t)sizeof(T) / (2 * parts) >= (a.rows * 2 * parts <= sms ? 65536 : 131072)) parts *= 2;
    // Threads: enough vectors each for the unrolled loop.  Of many rows, more and smaller blocks an SM,
    // whose joins overlap the others' loads: 4000 rows of 50000 bf16 logits with the 20 largest 118 us
    // with 256 threads, 145 with 512 (up to 3 rows an SM of long rows 512 keep more of the SM busy: 306 of
    // 131072 fp32 logits 27.8 us, 32.6 with 256).  Where rows are longer the choice of the largest, whose second
    // reading grows with a thread's vectors, turns it round: 2000 rows of 131072 fp32 logits 249 and 200.
    const int64_t vectors = (a.V + Vec<T>::kWidth - 1) / Vec<T>::kWidth / parts + 2;
    const bool many = a.rows * parts > (a.top_n || vectors < 8192 ? 2 : 3) * sms;
    const int most = many && !(a.top_n && vectors > 14336) ? kMaxThreads / 2 : kMaxThreads;
    int threads = 128;
    while (threads < most && vectors > threads * (many ? 2 * kUnroll : kUnroll)) threads *= 2;
    const float c = a.scale * 1.4426950408889634f;
    const int wide = !(c > 1e-12f && c < 1e3f);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)(a.rows * parts));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)parts;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return a.top_n ? cudaLaunchKernelEx(&cfg, logprob_kernel<T, true>, a, parts, wide) : cudaLaunchKernelEx(&cfg, logprob_kernel<T, false>, a, parts, wide);
}

}  // namespace nvq

using namespace nvq;

static nvq_status check_logits(const char* who, const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t ld, float scale)
{
    NVQ_CHECK_ARG(logits, NVQ_ERR_ARG, "%s: null pointer argument", who);
    NVQ_CHECK_ARG(dtype == NVQ_BF16 || dtype == NVQ_F32, NVQ_ERR_ARG, "%s: unknown logits type %d", who, (int)dtype);
    NVQ_CHECK_ARG(isfinite(scale) && scale > 0.0f, NVQ_ERR_ARG, "%s: scale must be finite and positive", who);
    NVQ_CHECK_ARG(rows >= 1 && rows < (1ll << 31) && V >= 1 && V < (1ll << 31) && ld >= V, NVQ_ERR_SHAPE,
                  "%s: rows or V outside [1, 2^31), or ld < V", who);
    NVQ_CHECK_ARG(aligned(logits, dtype == NVQ_F32 ? 4 : 2), NVQ_ERR_ALIGN, "%s: logits not aligned to their type", who);
    return NVQ_OK;
}

extern "C" nvq_status token_logprobs(const void* logits, int32_t logits_dtype, int64_t rows, int64_t V, int64_t ld,
                                     const int64_t* targets, float scale, int32_t top_n, float* logprob, float* entropy,
                                     float* lse, int32_t* top_ids, float* top_logprobs, void* stream)
{
    NVQ_TRACE("token_logprobs");
    const nvq_status s = check_logits("token_logprobs", logits, logits_dtype, rows, V, ld, scale);
    if (s != NVQ_OK) return s;
    NVQ_CHECK_ARG(targets || !logprob, NVQ_ERR_ARG, "token_logprobs: logprob without targets");
    NVQ_CHECK_ARG(top_n >= 0 && top_n <= kMaxTop && top_n <= V, NVQ_ERR_SHAPE, "token_logprobs: top_n outside [0, min(%d, V)]", kMaxTop);
    NVQ_CHECK_ARG((top_n > 0) == (top_ids != nullptr) && (top_n > 0) == (top_logprobs != nullptr), NVQ_ERR_ARG,
                  "token_logprobs: top_ids and top_logprobs go with top_n > 0");
    NVQ_CHECK_ARG(aligned(targets, 8) && aligned(logprob, 4) && aligned(entropy, 4) && aligned(lse, 4) && aligned(top_ids, 4) &&
                      aligned(top_logprobs, 4),
                  NVQ_ERR_ALIGN, "token_logprobs: a pointer is not aligned to its elements");
    DeviceStatus* dst = device_status_ptr();
    NVQ_CHECK_ARG(dst, NVQ_ERR_CUDA, "token_logprobs: device status word unavailable");
    set_error("");
    LogprobArgs a{logits, rows, V, ld, targets, scale, top_n, logprob, entropy, lse, top_ids, top_logprobs, dst};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e, "token_logprobs: device attributes");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = logits_dtype == NVQ_F32 ? launch_forward<float>(a, sms, st) : launch_forward<__nv_bfloat16>(a, sms, st);
    if (e != cudaSuccess) return cuda_status(e, "logprob_kernel");
    NVQ_LAUNCH_CHECK("logprob_kernel");
    return NVQ_OK;
}

extern "C" nvq_status token_logprobs_backward(const void* logits, int32_t logits_dtype, int64_t rows, int64_t V, int64_t ld,
                                              const int64_t* targets, float scale, const float* lse, const float* entropy,
                                              const float* g_logprob, const float* g_entropy, void* grad, int64_t ld_grad,
                                              void* stream)
{
    NVQ_TRACE("token_logprobs_backward");
    const nvq_status s = check_logits("token_logprobs_backward", logits, logits_dtype, rows, V, ld, scale);
    if (s != NVQ_OK) return s;
    NVQ_CHECK_ARG(lse && entropy && grad, NVQ_ERR_ARG, "token_logprobs_backward: null pointer argument");
    NVQ_CHECK_ARG(targets || !g_logprob, NVQ_ERR_ARG, "token_logprobs_backward: g_logprob without targets");
    NVQ_CHECK_ARG(ld_grad >= V && (grad != logits || ld_grad == ld), NVQ_ERR_SHAPE,
                  "token_logprobs_backward: ld_grad < V, or a gradient in place with another leading dimension");
    NVQ_CHECK_ARG(aligned(targets, 8) && aligned(lse, 4) && aligned(entropy, 4) && aligned(g_logprob, 4) && aligned(g_entropy, 4) &&
                      aligned(grad, logits_dtype == NVQ_F32 ? 4 : 2),
                  NVQ_ERR_ALIGN, "token_logprobs_backward: a pointer is not aligned to its elements");
    DeviceStatus* dst = device_status_ptr();
    NVQ_CHECK_ARG(dst, NVQ_ERR_CUDA, "token_logprobs_backward: device status word unavailable");
    set_error("");
    LogprobGradArgs a{logits, rows, V, ld, targets, scale, lse, entropy, g_logprob, g_entropy, grad, ld_grad, dst};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t width = logits_dtype == NVQ_F32 ? 4 : 8, vectors = (V + width - 1) / width + 1;
    const int64_t stretches = (vectors + kGradThreads * kGradPerThread - 1) / (kGradThreads * kGradPerThread);
    NVQ_CHECK_ARG(stretches <= 65535, NVQ_ERR_SHAPE, "token_logprobs_backward: V of %lld is too large", (long long)V);
    const dim3 grid((unsigned)rows, (unsigned)stretches);
    if (logits_dtype == NVQ_F32)
        logprob_grad_kernel<float><<<grid, kGradThreads, 0, st>>>(a);
    else
        logprob_grad_kernel<__nv_bfloat16><<<grid, kGradThreads, 0, st>>>(a);
    NVQ_LAUNCH_CHECK("logprob_grad_kernel");
    return NVQ_OK;
}
