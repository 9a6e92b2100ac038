// gemv.cu -- a few bf16 rows times NVFP4 weights (nvfp4_gemv, W4A16):
//   Y[r, n] = S_dec[g] * sum_k x[r / x_div, k] V[b_nk] sb_{n, k/16},  g = ids[r].
//
// The floor is the weights read once: 9/16 byte each.  What stands between is their expansion, so:
//   - a code times its block scale has at most 6 significant bits within [2^-10, 2688]: f16 holds it
//     exactly, two codes an instruction; bf16 would need four more operations a pair.
//   - the rows of x are brought into f16's range by a power of two each (undone at the end): exact,
//     except that a component below 2^-32 of its row's largest is rounded at 2^-39 of that.
//   - the weights are the 16-row operand of mma.m16n8k16 and up to 8 rows of x its columns, so the
//     products cost the same for 1 row and for 8; the inner index is permuted so that a lane takes
//     its 16 bytes of a weight row as they lie.
//   - the unit is a set of 32 weight rows, those whose scales share 16-byte pieces of the blocked
//     layout.  A block's warps form teams that take a set each and share its columns in stretches
//     of 128; each lane has a ring of two to four stretches' bytes of its own in shared memory, filled by
//     asynchronous copies ahead and over the borders between sets (loads into registers instead
//     were waited for in groups and reached 3.6 TB/s where this reaches 4.8).
//   - blocks (one an SM) take equal runs of sets over the groups that have rows (listed by each
//     block from ids), so idle experts cost nothing and x is brought in once for a run within one.
//
// Measured: one row of 4096 columns to 14336 (33 MB) in 12.9 us, to 131072 (302 MB) in 62.6 us =
// 4.8 TB/s, 0.71 of a copy; 16 tokens through 8 of 128 experts, 1536 x 2048 each (146 MB), in 40.5 us =
// 3.6 TB/s.  The small ones are bound by latency (2.4 us until x is in, 3 us of launch, the last join);
// the long ones by the issue of instructions at 16 warps an SM: 263 a stretch of a warp, 2.0 a cycle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace nvq {

constexpr int kWhereGemv = 49;
constexpr int kGemvStage = 5 * 32 * 16;  // a stretch: 5 pieces of 16 bytes a lane
constexpr int kGemvRows = 1024;    // rows of a launch
constexpr int kGemvGroups = 1024;
constexpr int kBegin = 4;
constexpr int kGemvSmem = 217 * 1024;

struct GemvArgs {
    const __nv_bfloat16* x;
    int64_t ldx;
    int32_t row0, rows;   // output rows [row0, row0 + rows) of this launch
    int32_t x_div;
    const int32_t* ids;
    int32_t groups;
    const uint8_t* codes;
    int64_t ldb;
    const uint8_t* sf;
    int64_t sf_cols;
    const nvq_tensor_scale* ts;
    int32_t N, K;
    int32_t cols;         // output columns: N, or N / 2 with SwiGLU
    int32_t epilogue;
    const float* row_w;
    void* out;
    int64_t ldo;
    int32_t pass;         // rows of x in shared memory at a time
    DeviceStatus* status;
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ void gemv_expand(uint32_t w, uint32_t* o)  // eight E2M1 codes -> four f16 pairs
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

__device__ __forceinline__ __half2 gemv_scale(uint32_t w)  // two E4M3 bytes -> an f16 pair
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return *reinterpret_cast<const __half2*>(&r);
}

// An f16 pair times one half (low or high) of another.
__device__ __forceinline__ uint32_t gemv_mul(uint32_t a, __half2 s, int high)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), high ? __high2half2(s) : __low2half2(s));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void gemv_mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t gemv_f16(uint32_t w, float up)  // a bf16 pair times `up` -> an f16 pair
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(bf16hi(w) * up), "f"(bf16lo(w) * up));
    return r;
}

// 16 or 4 bytes from global to shared memory, asynchronously; zeros where `there` is false.
__device__ __forceinline__ void gemv_copy(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void gemv_copy(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void gemv_copy4(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

__device__ __forceinline__ void gemv_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float gemv_of(uint32_t at, int rank)  // a float in the shared memory of the cluster's block `rank`
{
    uint32_t there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
}

// kTiles: 8-row tiles of x; kGlu: sets of gate rows, each followed by its up rows; kSplit: a cluster's
// blocks take the same run of sets, each a part of the columns, and join their sums through shared memory.
constexpr int kGemvMaxWarps = 16;
constexpr int kSplitBlocks = 2;
constexpr int kChunk = 8;  // sets between two joins of a cluster (2 us each)

template <int kTiles, bool kGlu, bool kSplit, int kGemvStages>
__global__ void __launch_bounds__(kGemvMaxWarps * 32, 1) gemv_kernel(const __grid_constant__ GemvArgs a)
{
    constexpr int kHalves = kGlu ? 2 : 1;
    constexpr int kPart = kTiles * 256;  // sums of a set: [tile of x][j][g][8 rows of x]
    extern __shared__ __align__(16) uint8_t smem[];
    const int threads = blockDim.x, warps = threads >> 5;
    float* parts = reinterpret_cast<float*>(smem + warps * kGemvStages * kGemvStage);  // [warp][kPart], behind the rings
    float* gates = parts + warps * kPart;                                              // [team][kPart], SwiGLU only
    float* store = parts + (kSplit ? 1 : kHalves) * warps * kPart;                     // [set of a chunk][half][row][32], clusters only
    uint4* xs = reinterpret_cast<uint4*>(store + (kSplit ? kChunk * kHalves * 32 * a.pass : 0));
    __shared__ int first[kGemvGroups + 1];      // a group's first place in `member`
    __shared__ uint16_t member[kGemvRows];      // rows by group
    __shared__ uint16_t active[kGemvGroups];    // groups that have rows
    __shared__ int n_active, scan_part[32];
    __shared__ uint32_t x_top[8 * kTiles];
    __shared__ float x_down[8 * kTiles];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

    // ---- rows by group
    if (a.groups == 1 && !a.ids) {
        if (tid == 0) {
            n_active = 1;
            active[0] = 0;
            first[0] = 0;
            first[1] = a.rows;
        }
        for (int r = tid; r < a.rows; r += threads) member[r] = (uint16_t)r;
        __syncthreads();
    } else {
        for (int i = tid; i < a.groups; i += threads) first[i] = 0;
        if (tid == 0) n_active = 0;
        __syncthreads();
        for (int r = tid; r < a.rows; r += threads) {
            const int id = a.ids ? a.ids[a.row0 + r] : 0;
            if ((unsigned)id < (unsigned)a.groups) atomicAdd(&first[id], 1);
        }
        __syncthreads();
        // exclusive sums of the counts, four groups a thread; active groups in order
        int n[4], sum = 0, act = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int id = tid * 4 + i;
            n[i] = id < a.groups ? first[id] : 0;
            sum += n[i];
            act += n[i] > 0;
        }
        int both = sum | act << 16, in = both;  // at most 1024 each
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(~0u, in, d);
            if (lane >= d) in += u;
        }
        if (lane == 31) scan_part[warp] = in;
        __syncthreads();
        int off = in - both;
        for (int w = 0; w < warp; ++w) off += scan_part[w];
        int at = off & 0xffff, ai = off >> 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int id = tid * 4 + i;
            if (id < a.groups) {
                first[id] = at;
                if (n[i]) active[ai++] = (uint16_t)id;
            }
            at += n[i];
        }
        if (tid == threads - 1) n_active = ai;
        __syncthreads();
        for (int r = tid; r < a.rows; r += threads) {
            const int id = a.ids ? a.ids[a.row0 + r] : 0;
            if ((unsigned)id < (unsigned)a.groups) {
                member[atomicAdd(&first[id], 1)] = (uint16_t)r;  // first[id] ends as the group's end
            } else if (blockIdx.x == 0) {
                report_status(a.status, NVQ_ERR_ARG, kWhereGemv);
                for (int n0 = 0; n0 < a.cols; ++n0) {
                    if (a.epilogue == NVQ_EPI_STORE_F32)
                        static_cast<float*>(a.out)[(a.row0 + r) * a.ldo + n0] = 0.0f;
                    else
                        static_cast<__nv_bfloat16*>(a.out)[(a.row0 + r) * a.ldo + n0] = __float2bfloat16_rn(0.0f);
                }
            }
        }
        __syncthreads();
    }
    const bool listed = !(a.groups == 1 && !a.ids);
    const int sets = (a.cols + 127) / 128 * 4;  // row sets of a group
    // a run's part in a group costs as much as kBegin sets to begin (x, and the rings run dry)
    const int begin = n_active > 1 ? kBegin : 0;
    const int64_t units = (int64_t)n_active * (sets + begin);
    constexpr int split = kSplit ? kSplitBlocks : 1;
    const int rank = kSplit ? blockIdx.x % split : 0;
    const int run = kSplit ? blockIdx.x / split : blockIdx.x, runs = kSplit ? gridDim.x / split : gridDim.x;
    const int64_t u0 = units * run / runs, u1 = units * (run + 1) / runs;
    const int stretches = (a.K + 127) / 128, k8 = a.K / 8;
    const int kf = kSplit ? stretches * rank / split : 0, kt = kSplit ? stretches * (rank + 1) / split : stretches;  // the block's

    const int64_t row_step = 32 * a.ldb;                      // bytes from a lane's row to its next
    const int64_t sf_block = a.sf_cols * 128;                 // bytes of a 128-row block of scales
    const bool turned = a.cols % 128 != 0;                    // the up rows do not begin a block of scales
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kGemvStages * kGemvStage + lane * 16;
    int fill = 0, turn = 0;  // stage filled next, stage read next
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    for (int64_t run0 = u0; run0 < u1;) {
        // ---- the part of the run within one group
        const int which = (int)(run0 / (sets + begin)), grp = active[which];
        const int from = (int)(run0 - (int64_t)which * (sets + begin)), to = (int)min((int64_t)(sets + begin), from + (u1 - run0));
        run0 += to - from;
        const int s0 = max(from - begin, 0), s1 = to - begin;
        if (s1 <= s0) continue;
        // first[] holds ends after the listing (begins without it)
        const int mend = listed ? first[grp] : a.rows, mbeg = listed ? (which ? first[active[which - 1]] : 0) : 0;
        const float s_dec = a.ts[grp].s_dec;
        // Warps of a team: the least number of stretches that the busiest warp takes, a join counted
        // as one.  Three sets of 4096 columns on 16 warps: one round of 7 stretches for three teams of
        // 5, three rounds of 2 for a team of 16.  (Lane t weighs teams of t + 1.)
        int size;
        {
            const int t = lane + 1, teams_t = max(1, warps / t);
            const int most = kSplit ? (stretches + split - 1) / split : stretches;
            const unsigned cost = t > warps || (kSplit && teams_t > kChunk)
                                      ? ~0u
                                      : (unsigned)((s1 - s0 + teams_t - 1) / teams_t * kHalves * ((most + t - 1) / t + 1));
            const unsigned least = __reduce_min_sync(~0u, cost);
            size = __ffs(__ballot_sync(~0u, cost == least));  // of equals the smallest: the fewest joins
        }
        const int teams = warps / size, team = warp / size, in_team = warp % size;
        const bool idle = team >= teams;  // a warp left over
        auto join = [&] {
            if (size == 1)
                __syncwarp();
            else
                asm volatile("barrier.sync %0, %1;" ::"r"(team + 1), "r"(size * 32) : "memory");
        };

        for (int m0 = mbeg; m0 < mend; m0 += a.pass) {
            const int nx = min(a.pass, mend - m0);
            // ---- what is loaded next: stretch lk of half lh of set ls
            int ls = s0 + team, lh = 0, lk = kf + in_team;
            const uint8_t *lcodes = nullptr, *lsf = nullptr;
            int lrows = 0;    // of the lane's four rows, those that exist
            int64_t lrow = 0;
            bool lfull = false;  // all rows of the set exist, their scales in one piece
            const int whole = a.K / 128;
            auto aim = [&] {
                const int n = (ls >> 2) * 128 + (ls & 3) * 8 + g;
                lrow = (int64_t)grp * a.N + n + (lh ? a.cols : 0);
                lcodes = a.codes + lrow * a.ldb + c * 16;
                lrows = n < a.cols ? min(4, (a.cols - n + 31) >> 5) : 0;
                lsf = a.sf + (lrow >> 7) * sf_block + (lrow & 31) * 16 + (c >> 1) * 512;
                lfull = (ls >> 2) * 128 + 128 <= a.cols && !(kGlu && lh && turned);
            };
            auto load = [&] {
                const int at = lk * 64;  // bytes along a row
                const bool there = at + c * 16 < a.K / 2;
                const uint32_t dst = ring + fill * kGemvStage;
                if (lk < whole && lfull) {  // the usual case: no row or column ends here
                    const uint8_t* p = lcodes + at;
#pragma unroll
                    for (int j = 0; j < 4; ++j, p += row_step) gemv_copy(dst + j * 512, p);
                    gemv_copy(dst + 4 * 512, lsf + lk * 1024);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool row = there && j < lrows;
                        gemv_copy(dst + j * 512, row ? lcodes + j * row_step + at : a.codes, row);
                    }
                    if (kGlu && lh && turned) {
                        for (int j = 0; j < 4; ++j) {
                            const bool row = there && j < lrows;
                            const int64_t r = lrow + 32 * j;
                            const int64_t o = (r >> 7) * sf_block + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (int64_t)(lk * 2 + (c >> 1)) * 512;
                            gemv_copy4(dst + 4 * 512 + j * 4, row ? a.sf + o : a.sf, row);
                        }
                    } else {
                        const bool any = there && lrows > 0;
                        gemv_copy(dst + 4 * 512, any ? lsf + (int64_t)lk * 1024 : a.sf, any);
                    }
                }
                fill = fill + 1 == kGemvStages ? 0 : fill + 1;
                lk += size;
                if (lk >= kt) {
                    lk = kf + in_team;
                    if (kGlu && !lh) {
                        lh = 1;
                    } else {
                        lh = 0;
                        ls += teams;
                    }
                    if (ls < s1) aim();
                }
            };
            const bool works = !idle && kf + in_team < kt && ls < s1;
            if (works) aim();
            turn = fill;
#pragma unroll
            for (int i = 0; i < kGemvStages; ++i) {
                if (works && ls < s1) load();
                commit();
            }
            // ---- rows of x into shared memory as f16, [stretch][word][row][c] of 8 values
            __syncthreads();  // the last pass has read them
            if (tid < 8 * kTiles) x_top[tid] = 0;
            __syncthreads();
            const int share = max(1, warps / nx);  // warps of a row
            constexpr int kKeep = 4;
            const int x0 = kf * 16, nk = min(kt * 16, k8) - x0;  // the block's columns, in eights
            const int kb = x0 + nk * (warp % share) / share, ke = x0 + nk * (warp % share + 1) / share;
            for (int r0 = 0; r0 < nx; r0 += warps / share) {
                const int r = r0 + warp / share;
                const uint4* src = reinterpret_cast<const uint4*>(a.x + (int64_t)((a.row0 + member[m0 + min(r, nx - 1)]) / a.x_div) * a.ldx);
                uint4 keep[kKeep];
                uint32_t top = 0;
                if (r < nx) {
                    for (int k0 = kb + lane; k0 < ke; k0 += 32 * kKeep) {
#pragma unroll
                        for (int q = 0; q < kKeep; ++q)
                            if (k0 + 32 * q < ke) keep[q] = __ldg(src + k0 + 32 * q);
#pragma unroll
                        for (int q = 0; q < kKeep; ++q)
                            if (k0 + 32 * q < ke)
                                top = __vmaxu2(top, __vmaxu2(__vmaxu2(keep[q].x & 0x7fff7fffu, keep[q].y & 0x7fff7fffu),
                                                             __vmaxu2(keep[q].z & 0x7fff7fffu, keep[q].w & 0x7fff7fffu)));
                    }
                    top = __reduce_max_sync(~0u, max(top & 0xffffu, top >> 16));
                    if (lane == 0 && share > 1) atomicMax(&x_top[r], top);
                }
                if (share > 1) __syncthreads();
                if (r >= nx) continue;
                if (share > 1) top = x_top[r];
                const int shift = min(14 - ((int)(top >> 7) - 127), 126);  // largest into [2^14, 2^15)
                const float up = __uint_as_float((uint32_t)(shift + 127) << 23);
                if (lane == 0 && warp % share == 0) x_down[r] = __uint_as_float((uint32_t)(127 - shift) << 23);
                for (int k0 = kb + lane; k0 < ke; k0 += 32 * kKeep)
#pragma unroll
                    for (int q = 0; q < kKeep; ++q) {
                        const int k = k0 + 32 * q;
                        if (k < ke) {
                            const uint4 v = ke - kb <= 32 * kKeep ? keep[q] : __ldg(src + k);
                            xs[((((k >> 4) - kf) * 4 + (k & 3)) * nx + r) * 4 + ((k >> 2) & 3)] =
                                make_uint4(gemv_f16(v.x, up), gemv_f16(v.y, up), gemv_f16(v.z, up), gemv_f16(v.w, up));
                        }
                    }
                for (int k = k8 + lane; k < kt * 16 && warp % share == 0; k += 32)  // zeros up to the last stretch's end
                    xs[((((k >> 4) - kf) * 4 + (k & 3)) * nx + r) * 4 + ((k >> 2) & 3)] = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();

            // ---- the sets
            float acc[kTiles][2][4];
            auto clear = [&] {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int p = 0; p < 2; ++p) acc[t][p][0] = acc[t][p][1] = acc[t][p][2] = acc[t][p][3] = 0.0f;
            };
            clear();
            // the stretch's last columns beyond K (a RAC tail, or nothing) have scale 0
            const int tail_k = a.K / 2 % 64 ? stretches - 1 : stretches;
            const uint32_t sel = (c & 1) ? 0x32 : 0x10;  // the lane's two scale bytes of a word
            auto multiply = [&](int k) {
                const uint4* st = reinterpret_cast<const uint4*>(smem + (warp * kGemvStages + turn) * kGemvStage) + lane;
                const uint4 sfw = st[4 * 32];
                const uint32_t sf[4] = {sfw.x, sfw.y, sfw.z, sfw.w};
                uint4 codes[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) codes[j] = st[j * 32];
                const bool cut = k == tail_k && c * 16 + 8 >= a.K / 2 - k * 64;
                __half2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = gemv_scale(__byte_perm(sf[j], 0, cut ? sel & 0x0f | 0x40 : sel));
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint4 b[kTiles];
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) b[t] = t * 8 + g < nx ? xs[(((k - kf) * 4 + w) * nx + t * 8 + g) * 4 + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint4 &lo = codes[2 * p], &hi = codes[2 * p + 1];
                        uint32_t x0[4], x1[4];
                        gemv_expand(w == 0 ? lo.x : w == 1 ? lo.y : w == 2 ? lo.z : lo.w, x0);
                        gemv_expand(w == 0 ? hi.x : w == 1 ? hi.y : w == 2 ? hi.z : hi.w, x1);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x0[e] = gemv_mul(x0[e], f[2 * p], w >> 1);
                            x1[e] = gemv_mul(x1[e], f[2 * p + 1], w >> 1);
                        }
#pragma unroll
                        for (int t = 0; t < kTiles; ++t) {
                            gemv_mma(acc[t][p], x0[0], x1[0], x0[1], x1[1], b[t].x, b[t].y);
                            gemv_mma(acc[t][p], x0[2], x1[2], x0[3], x1[3], b[t].z, b[t].w);
                        }
                    }
                }
            };
            auto put = [&](int s, int i, float y) {  // element i of set s: 32 weight rows of each row of x
                const int n = (s >> 2) * 128 + (s & 3) * 8 + (i & 7) + 32 * ((i >> 3) & 3);
                if (n >= a.cols) return;
                const int64_t row = a.row0 + member[m0 + (i >> 5)];
                if (a.epilogue == NVQ_EPI_ROW_SCALE) y *= a.row_w[row];
                if (a.epilogue == NVQ_EPI_STORE_F32)
                    static_cast<float*>(a.out)[row * a.ldo + n] = y;
                else
                    static_cast<__nv_bfloat16*>(a.out)[row * a.ldo + n] = __float2bfloat16_rn(y);
            };
            // the team's sums of half h of set s, in the warps' order; `nth` counts the chunk's sets
            auto finish = [&](int s, int h, int nth) {
                float* mine = parts + warp * kPart;
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int e = 0; e < 2; ++e)  // weight row 2 p + e of the lane's four, rows 2c, 2c + 1 of x
                            if (t * 8 + 2 * c < nx)
                                *reinterpret_cast<float2*>(mine + (t * 4 + 2 * p + e) * 64 + g * 8 + 2 * c) = make_float2(acc[t][p][2 * e], acc[t][p][2 * e + 1]);
                clear();
                join();
                const float* in = parts + team * size * kPart;
                // (row of x, weight row) pairs of the set; neighbouring threads take neighbouring weight rows
                for (int i = in_team * 32 + lane; i < nx * 32; i += size * 32) {
                    const int r = i >> 5, at = ((r >> 3) * 4 + ((i >> 3) & 3)) * 64 + (i & 7) * 8 + (r & 7);
                    float y = 0.0f;
                    for (int w = 0; w < size; ++w) y += in[w * kPart + at];
                    // x's power of two before the weights' scale where it is small, after it where it is large:
                    // rows near fp32's ends stay within its range on the way
                    const float down = x_down[r];
                    y = y * fminf(down, 1.0f) * s_dec * fmaxf(down, 1.0f);
                    if constexpr (kSplit) {
                        store[(nth * kHalves + h) * nx * 32 + i] = y;
                        continue;
                    }
                    if constexpr (kGlu) {
                        if (!h) {
                            gates[team * kPart + at] = silu(y);
                            continue;
                        }
                        y *= gates[team * kPart + at];
                    }
                    put(s, i, y);
                }
                join();
            };
            const int chunk = kSplit ? kChunk / teams * teams : s1 - s0;
            for (int c0 = s0; c0 < s1; c0 += chunk) {
                const int c1 = min(c0 + chunk, s1);
                for (int s = idle ? c1 : c0 + team; s < c1; s += teams)
#pragma unroll 1
                    for (int h = 0; h < kHalves; ++h) {
                        for (int k = kf + in_team; k < kt; k += size) {
                            // a lane reads what it copied itself: its own groups are all it waits for
                            asm volatile("cp.async.wait_group %0;" ::"n"(kGemvStages - 1) : "memory");
                            multiply(k);
                            turn = turn + 1 == kGemvStages ? 0 : turn + 1;
                            if (ls < s1) load();  // into the stage just read
                            commit();
                        }
                        finish(s, h, s - c0);
                    }
                if constexpr (kSplit) {
                    // the blocks' sums of the chunk, in the blocks' order; each block writes a share
                    gemv_cluster_sync();
                    const uint32_t base = (uint32_t)__cvta_generic_to_shared(store);
                    for (int i = rank * threads + tid; i < (c1 - c0) * nx * 32; i += split * threads) {
                        const int nth = i / (nx * 32), e = i - nth * nx * 32;
                        float y[kHalves] = {};
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            for (int q = 0; q < split; ++q) y[h] += gemv_of(base + ((nth * kHalves + h) * nx * 32 + e) * 4, q);
                        put(c0 + nth, e, kGlu ? silu(y[0]) * y[kHalves - 1] : y[0]);
                    }
                    gemv_cluster_sync();  // read before they are written again, or before their block ends
                }
            }
        }
    }
}

template <int kTiles, bool kGlu, bool kSplit, int kStages>
static cudaError_t launch_gemv(const GemvArgs& a, int warps, int smem, int sms, cudaStream_t st)
{
    constexpr int blocks = kSplit ? kSplitBlocks : 1;
    auto kernel = gemv_kernel<kTiles, kGlu, kSplit, kStages>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)(a.groups < a.rows ? a.groups : a.rows) * ((a.cols + 127) / 128 * 4);
    const int runs = (int)(units < sms / blocks ? units : sms / blocks);
    if constexpr (kSplit) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[1];
        cfg.gridDim = dim3((unsigned)(runs * blocks));
        cfg.blockDim = dim3((unsigned)(warps * 32));
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = st;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = blocks;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, a);
    } else {
        kernel<<<(unsigned)runs, warps * 32, smem, st>>>(a);
        return cudaGetLastError();
    }
}

// Shared memory of a block: rings, sums (and gates, or a cluster's chunk), x.
static int gemv_smem(int tiles, bool glu, int blocks, int warps, int stages, int rows, int K)
{
    return warps * (stages * kGemvStage + (glu && blocks == 1 ? 2 : 1) * tiles * 1024) +
           (blocks > 1 ? kChunk * (glu ? 2 : 1) * rows * 128 : 0) + rows * (((K + 127) / 128 + blocks - 1) / blocks * 256);
}

// Shared memory goes to x first: all rows of the tiles at a time if they fit beside 8 warps and their
// rings (else as many as do); then to warps, up to 16; then to the rings' stages.  With two tiles, two
// stages and more warps are better than three and fewer: 16 rows of 4096 columns to 14336 took 21.0 us
// with 12 warps of two stages, 25.0 with 8 of three.
template <int kTiles, bool kGlu, bool kSplit>
static cudaError_t launch_gemv(GemvArgs a, int sms, cudaStream_t st)
{
    auto smem = [&](int warps, int stages) { return gemv_smem(kTiles, kGlu, kSplit ? kSplitBlocks : 1, warps, stages, a.pass, a.K); };
    a.pass = a.rows < 8 * kTiles ? a.rows : 8 * kTiles;
    constexpr int least = kTiles > 1 ? 2 : 3;
    while (a.pass > 1 && smem(8, least) > kGemvSmem) --a.pass;
    int warps = 16;
    while (warps > 8 && smem(warps, least) > kGemvSmem) --warps;
    if constexpr (kTiles > 1)
        if (smem(warps, 3) > kGemvSmem) return launch_gemv<kTiles, kGlu, kSplit, 2>(a, warps, smem(warps, 2), sms, st);
    if constexpr (!kSplit)  // a pair that had room for four would not have been split
        if (smem(warps, 4) <= kGemvSmem) return launch_gemv<kTiles, kGlu, kSplit, 4>(a, warps, smem(warps, 4), sms, st);
    return launch_gemv<kTiles, kGlu, kSplit, 3>(a, warps, smem(warps, 3), sms, st);
}

// Pairs of blocks share the columns where whole rows leave no room for 16 warps: the 16 rows above
// take 18.7 us so (SwiGLU 20.6 for 41.0), 32 rows in two passes 34.8 for 39.7, 8 rows of 14336 columns to
// 4096 21.8 for 45.0.  12 rows of 4096, whose rings fit, take 17.6 us unsplit and 19.1 split, for the
// join; clusters of four take 23 us for 16.  Not with ids: each block lists a group's rows in an order of its own.
template <bool kGlu>
static cudaError_t launch_gemv(const GemvArgs& a, bool two, int sms, cudaStream_t st)
{
    const int tiles = two ? 2 : 1, rows = a.rows < 8 * tiles ? a.rows : 8 * tiles;
    if (!a.ids && gemv_smem(tiles, kGlu, 1, 16, two ? 2 : 3, rows, a.K) > kGemvSmem)
        return two ? launch_gemv<2, kGlu, true>(a, sms, st) : launch_gemv<1, kGlu, true>(a, sms, st);
    return two ? launch_gemv<2, kGlu, false>(a, sms, st) : launch_gemv<1, kGlu, false>(a, sms, st);
}

}  // namespace nvq

using namespace nvq;

extern "C" nvq_status nvfp4_gemv(const void* x, int64_t ldx, int64_t rows, int32_t x_div, const int32_t* ids, int32_t groups,
                                 const uint8_t* b_codes, int64_t ldb, const uint8_t* b_sf, int64_t b_sf_cols,
                                 const nvq_tensor_scale* b_tscale, int64_t N, int64_t K, int32_t epilogue, const float* row_w,
                                 void* out, int64_t ldo, void* stream)
{
    NVQ_TRACE("nvfp4_gemv");
    NVQ_CHECK_ARG(x && b_codes && b_sf && b_tscale && out, NVQ_ERR_ARG, "nvfp4_gemv: null pointer argument");
    NVQ_CHECK_ARG(epilogue == NVQ_EPI_STORE || epilogue == NVQ_EPI_SWIGLU || epilogue == NVQ_EPI_ROW_SCALE ||
                      epilogue == NVQ_EPI_STORE_F32,
                  NVQ_ERR_ARG, "nvfp4_gemv: unknown epilogue %d", (int)epilogue);
    NVQ_CHECK_ARG((epilogue == NVQ_EPI_ROW_SCALE) == (row_w != nullptr), NVQ_ERR_ARG,
                  "nvfp4_gemv: row_w goes with NVQ_EPI_ROW_SCALE and with nothing else");
    NVQ_CHECK_ARG(rows >= 1 && rows <= 32768 && x_div >= 1, NVQ_ERR_SHAPE, "nvfp4_gemv: rows outside [1, 32768] or x_div < 1");
    NVQ_CHECK_ARG(groups >= 1 && groups <= 1024 && (groups == 1 || ids), NVQ_ERR_SHAPE,
                  "nvfp4_gemv: groups outside [1, 1024], or several groups without ids");
    NVQ_CHECK_ARG(K >= 16 && K % 16 == 0 && K <= 65536, NVQ_ERR_SHAPE, "nvfp4_gemv: K must be a multiple of 16 in [16, 65536]");
    NVQ_CHECK_ARG(N >= 1 && N <= (1ll << 24) && groups * N <= (1ll << 31) - 1 && (groups == 1 || N % 128 == 0), NVQ_ERR_SHAPE,
                  "nvfp4_gemv: N outside [1, 2^24], too many weight rows, or not a multiple of 128 with several groups");
    NVQ_CHECK_ARG(epilogue != NVQ_EPI_SWIGLU || N % 64 == 0, NVQ_ERR_SHAPE, "nvfp4_gemv: SwiGLU needs N / 2 to be a multiple of 32");
    NVQ_CHECK_ARG(ldb >= K / 2 && b_sf_cols >= nvq_sf_cols(K) && b_sf_cols % 4 == 0 && ldx >= K &&
                      ldo >= (epilogue == NVQ_EPI_SWIGLU ? N / 2 : N),
                  NVQ_ERR_SHAPE, "nvfp4_gemv: a leading dimension or b_sf_cols is too small");
    NVQ_CHECK_ARG(ldb % 16 == 0 && aligned(b_codes, 16) && aligned(b_sf, 16) && ldx % 8 == 0 && aligned(x, 16) && aligned(out, 4) &&
                      aligned(b_tscale, 4) && aligned(row_w, 4) && aligned(ids, 4),
                  NVQ_ERR_ALIGN, "nvfp4_gemv: x and codes need 16-byte aligned rows, the scales 16 bytes, out 4");
    DeviceStatus* dst = device_status_ptr();
    NVQ_CHECK_ARG(dst, NVQ_ERR_CUDA, "nvfp4_gemv: device status word unavailable");
    set_error("");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e, "nvfp4_gemv: device attributes");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool glu = epilogue == NVQ_EPI_SWIGLU;
    for (int64_t r0 = 0; r0 < rows; r0 += kGemvRows) {
        const int n = (int)(rows - r0 < kGemvRows ? rows - r0 : kGemvRows);
        GemvArgs a{static_cast<const __nv_bfloat16*>(x), ldx, (int)r0, n, x_div, ids, groups, b_codes, ldb, b_sf, b_sf_cols, b_tscale,
                   (int)N, (int)K, (int)(glu ? N / 2 : N), epilogue, row_w, out, ldo, 0, dst};
        // a second tile of 8 rows by the rows a group has (on average, where ids say); a third and a
        // fourth cost more registers than reading the weights again: 32 rows of 4096 columns 39.7 us
        const bool two = (n + groups - 1) / groups > 8;
        e = glu ? launch_gemv<true>(a, two, sms, st) : launch_gemv<false>(a, two, sms, st);
        if (e != cudaSuccess) return cuda_status(e, "gemv_kernel");
    }
    return NVQ_OK;
}
