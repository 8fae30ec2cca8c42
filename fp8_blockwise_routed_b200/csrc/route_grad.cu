// route_grad.cu -- the router's balance loss with per-expert counts, and the
// gradient of the routing in the logits.
//
// Balance and z loss of a batch of logits z [T, E] that moe_route routed into
// counts c_e (differences of expert_offsets), P = sum c_e pairs:
//   p_te = softmax over the selectable logits of row t (not NaN, not -Inf),
//   N    = tokens with at least one of them,
//   L_b  = E * sum_e (c_e / P) * (1/N sum_t p_te),   L_z = 1/N sum_t lse_t^2.
// Gradient of d0*L_b + d1*L_z + <dout, combine(y)> in z (counts held fixed):
//   s_j   = rs * <dout_t, y_tj>                      (y_tj = w_j * expert row)
//   dz_e  = sum_{j: id_j = e} (s_j - w_j * sum_i s_i)
//         + p_te * (g_e - sum_e' p_te' g_e' + 2 d1 lse_t / N),  g_e = d0 E c_e / (P N).
// The first line is w_j (dw_j - sum_i w_i dw_i) with w_j dw_j = s_j, so the
// weight that y already carries is never divided out.
//
// Bounds: the loss reads each logit once (4 T E bytes) and is HBM-bound once
// the logits exceed L2, launch-bound below; the gradient reads every filled
// slot row once (4 T k H bytes) and is HBM-bound.  All sums are FP32 in a
// fixed order (FP64 across blocks): no atomics, the same bits every run on a
// given GPU.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <climits>

#include "internal.h"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace fp8moe {
namespace {

__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A row of E <= VPL * LPR logits in the registers of LPR lanes: register i of
// lane l holds expert 4 (l % LPR) + 4 LPR (i / 4) + i % 4, so that a lane's
// four neighbours are one 16-byte access where E is a multiple of four.
template <int LPR>
__device__ __forceinline__ int expert_of(int lane, int i)
{
    return 4 * (lane % LPR) + 4 * LPR * (i / 4) + i % 4;
}

template <int VPL, int LPR>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, bool ok, float (&v)[VPL])
{
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
        const int e = expert_of<LPR>(lane, i);
        if (E % 4 == 0) {
            const float4 t = (ok && e < E) ? __ldg(reinterpret_cast<const float4*>(row + e))
                                           : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            v[i] = t.x;
            v[i + 1] = t.y;
            v[i + 2] = t.z;
            v[i + 3] = t.w;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) v[i + u] = (ok && e + u < E) ? __ldg(row + e + u) : -INFINITY;
        }
    }
}

__device__ __forceinline__ float lg2_approx(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

template <int LPR>
__device__ __forceinline__ float row_max(float v)
{
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// a * b + c and a + b on two neighbours at once.
__device__ __forceinline__ void fma2(float& x, float& y, float a0, float a1, float b, float c0, float c1)
{
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(x), "=f"(y)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& x, float& y, float a0, float a1)
{
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a0), "f"(a1));
}

// Softmax of a row over its selectable entries (fmaxf drops NaN): v becomes
// the exponentials, 0 where not selectable, and inv what they are to be
// multiplied by; returns whether there is any, and log(sum exp) in lse.
// 2^(v L - mL), L = log2 e, mL = m L rounded: the rounding of mL is the same
// for the whole row, so it cancels in the probabilities, and its effect on
// the sum is known exactly (delta) and taken out of the logarithm.  That holds
// while the rounding is small: below kOffsetMax it is at most 2^-11, so the
// sum lies in [0.999, 1.001 E], where lg2.approx is within 2^-22 (relative to
// values beyond 1) and one Newton step makes rcp.approx good to an ulp.  From
// there on (half a step of mL reaches 126, FP32's whole range of exponents, at
// |m| = 1.5e9) the maximum is subtracted first, one instruction more per
// logit.  A +Inf logit gives NaN (Inf - Inf), as in the router's weights.
constexpr float kOffsetMax = 16384.0f;
template <int VPL, int LPR>
__device__ __forceinline__ bool softmax_row(float (&v)[VPL], float& inv, float& lse)
{
    constexpr float kL = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        v[i] = fmaxf(v[i], -INFINITY);
        m = fmaxf(m, v[i]);
    }
    m = row_max<LPR>(m);
    const bool any = m != -INFINITY;
    const float mL = m * kL;
    float s0 = 0.0f, s1 = 0.0f, delta = 0.0f;
    if (fabsf(mL) < kOffsetMax) {
        delta = fmaf(m, kL, -mL);
#pragma unroll
        for (int i = 0; i < VPL; i += 2) {
            fma2(v[i], v[i + 1], v[i], v[i + 1], kL, -mL, -mL);
            v[i] = sm100::ex2_approx_ftz(v[i]);
            v[i + 1] = sm100::ex2_approx_ftz(v[i + 1]);
            add2(s0, s1, v[i], v[i + 1]);
        }
    } else {  // a maximum far out, an infinite one, or none
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = any ? sm100::ex2_approx_ftz((v[i] - m) * kL) : 0.0f;
            s0 += v[i];
        }
    }
    const float sum = row_sum<LPR>(s0 + s1);
    inv = sm100::rcp_approx_ftz(sum);
    inv = any ? fmaf(inv, fmaf(-sum, inv, 1.0f), inv) : 0.0f;
    lse = any ? m + (lg2_approx(sum) - delta) * kLn2 : 0.0f;
    return any;
}

// ------------------------------------------------------------------- losses

constexpr int kLossWarps = 16;

// What a warp gathers over its rows.
template <int VPL>
struct WarpSums {
    float acc[VPL];  // probabilities
    double z = 0.0;  // lse^2 (short FP32 sums, FP64 beyond)
    float zf = 0.0f;
    int n = 0;       // counted rows

    __device__ __forceinline__ WarpSums()
    {
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
    }
    template <int LPR>
    __device__ __forceinline__ void add(float (&v)[VPL])
    {
        float inv, lse;
        if (softmax_row<VPL, LPR>(v, inv, lse)) {
            // 16 squares stay within FP32
            const float near = fabsf(lse) < 0x1p60f ? lse : 0.0f;
            zf = fmaf(near, near, zf);
            const bool last = (++n & 15) == 0;
            if (last || near != lse) {
                z += zf;
                zf = 0.0f;
                if (near != lse) z += static_cast<double>(lse) * lse;
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; i += 2) fma2(acc[i], acc[i + 1], v[i], v[i + 1], inv, acc[i], acc[i + 1]);
    }
};

// A block's sums from its warps', in warp order: probabilities into s_sum [E],
// lse^2 and the number of counted rows to every thread.
struct LossSums {
    double z;
    int n;
};
template <int VPL, int LPR>
__device__ __forceinline__ LossSums join_warps(WarpSums<VPL>& w, int E, float* s_sum)
{
    __shared__ __align__(16) float red[kLossWarps][256];
    __shared__ double red_z[kLossWarps];
    __shared__ int red_n[kLossWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double z = w.z + w.zf;
    // the groups of a warp, then the warps, 256 experts at a time
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) w.acc[i] += __shfl_xor_sync(0xFFFFFFFFu, w.acc[i], off);
        z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
        w.n += __shfl_xor_sync(0xFFFFFFFFu, w.n, off);
    }
    if (lane == 0) {
        red_z[warp] = z;
        red_n[warp] = w.n;
    }
    constexpr int kPart = VPL * LPR < 256 ? VPL * LPR : 256;
#pragma unroll
    for (int e0 = 0; e0 < VPL * LPR; e0 += kPart) {
        __syncthreads();
        if (lane < LPR) {
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                const int e = expert_of<LPR>(lane, i);
                if (e >= e0 && e < e0 + kPart)
                    *reinterpret_cast<float4*>(&red[warp][e - e0]) =
                        make_float4(w.acc[i], w.acc[i + 1], w.acc[i + 2], w.acc[i + 3]);
            }
        }
        __syncthreads();
        const int e = e0 + threadIdx.x;
        if (threadIdx.x < kPart && e < E) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kLossWarps; ++q) s += red[q][threadIdx.x];
            s_sum[e] = s;
        }
    }
    __syncthreads();
    LossSums out{0.0, 0};
#pragma unroll
    for (int q = 0; q < kLossWarps; ++q) {
        out.z += red_z[q];
        out.n += red_n[q];
    }
    return out;
}

// Rows dealt to the blocks' warps (and to the 32 / LPR groups of a warp) one at
// a time, read straight into registers, the next while one is summed: for few
// rows, and for row lengths that bulk copies cannot take.
template <int VPL, int LPR>
__device__ __forceinline__ LossSums loss_sums(const float* __restrict__ logits, int64_t T, int E, int block, int blocks,
                                              float* s_sum)
{
    constexpr int kRows = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    WarpSums<VPL> sums;
    const int64_t step = static_cast<int64_t>(blocks) * kLossWarps * kRows;
    int64_t t = (static_cast<int64_t>(block) * kLossWarps + warp) * kRows;  // the warp's first row
    const int64_t mine = lane / LPR;
    float next[VPL];
    load_row<VPL, LPR>(logits + (t + mine) * E, E, lane, t + mine < T, next);
    for (; t < T; t += step) {
        float v[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = next[i];
        load_row<VPL, LPR>(logits + (t + step + mine) * E, E, lane, t + step + mine < T, next);
        sums.template add<LPR>(v);
    }
    return join_warps<VPL, LPR>(sums, E, s_sum);
}

__device__ __forceinline__ double block_sum(double v, double* s_red)  // kLossWarps warps, every thread gets it
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kLossWarps; ++w) s += s_red[w];
    return s;
}

// Few rows: one cluster of up to eight blocks does the whole loss in one
// launch.  Each block sums the experts of its share over the cluster, in
// block order.
constexpr int kSmallBlocks = 8;
template <int VPL, int LPR>
__global__ void __launch_bounds__(kLossWarps * 32)
    balance_small_kernel(const float* __restrict__ logits, int64_t T, int E, const int32_t* __restrict__ offsets,
                         float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob_mean)
{
    __shared__ float s_sum[VPL * LPR];
    __shared__ LossSums s_all;
    __shared__ double s_term[kSmallBlocks];
    __shared__ double s_red[kLossWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const LossSums own = loss_sums<VPL, LPR>(logits, T, E, rank, nc, s_sum);
    if (threadIdx.x == 0) s_all = own;
    cluster.sync();
    LossSums all{0.0, 0};
    for (int b = 0; b < nc; ++b) {
        const LossSums* o = cluster.map_shared_rank(&s_all, b);
        all.z += o->z;
        all.n += o->n;
    }
    const double inv_n = 1.0 / (all.n > 0 ? all.n : 1);
    const int share = (E + nc - 1) / nc;
    double term = 0.0;
    for (int e = rank * share + threadIdx.x; e < E && e < (rank + 1) * share; e += kLossWarps * 32) {
        double s = 0.0;
        for (int b = 0; b < nc; ++b) s += cluster.map_shared_rank(s_sum, b)[e];
        const int32_t c = __ldg(offsets + e + 1) - __ldg(offsets + e);
        s *= inv_n;
        term += s * c;
        prob_mean[e] = static_cast<float>(s);
        counts[e] = c;
    }
    term = block_sum(term, s_red);
    if (threadIdx.x == 0) cluster.map_shared_rank(s_term, 0)[rank] = term;
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
        double sum = 0.0;
        for (int b = 0; b < nc; ++b) sum += s_term[b];
        const int32_t P = __ldg(offsets + E);
        loss[0] = static_cast<float>(E * sum / (P > 0 ? P : 1));
        loss[1] = static_cast<float>(all.z * inv_n);
        counts[E] = all.n;
    }
}

// Many rows: per-block sums part [gridDim.x][E], part_z, part_n ...  A block
// that lacks rows (a wait ran out) writes NaN and a count below any sum of the
// others'.
constexpr int kLostRows = INT_MIN;
// Counted tokens of a loss that lacks rows: negative, also once other ranks'
// counts are added to it.
constexpr int kNoCount = -(1 << 30);
template <int VPL, int LPR>
__device__ __forceinline__ void write_part(const LossSums& own, const float* s_sum, bool lost, int E,
                                           float* __restrict__ part, double* __restrict__ part_z,
                                           int* __restrict__ part_n)
{
    for (int e = threadIdx.x; e < E; e += kLossWarps * 32)
        part[static_cast<int64_t>(blockIdx.x) * E + e] = lost ? NAN : s_sum[e];
    if (threadIdx.x == 0) {
        part_z[blockIdx.x] = lost ? NAN : own.z;
        part_n[blockIdx.x] = lost ? kLostRows : own.n;
    }
}

template <int VPL, int LPR>
__global__ void __launch_bounds__(kLossWarps * 32)
    balance_partial_kernel(const float* __restrict__ logits, int64_t T, int E, float* __restrict__ part,
                           double* __restrict__ part_z, int* __restrict__ part_n)
{
    __shared__ float s_sum[VPL * LPR];
    allow_next();
    const LossSums own = loss_sums<VPL, LPR>(logits, T, E, blockIdx.x, gridDim.x, s_sum);
    write_part<VPL, LPR>(own, s_sum, false, E, part, part_z, part_n);
}

// The same by bulk copies, for rows of whole 16-byte pieces: every warp has a
// ring of its own, chunks of `rows` consecutive rows (4 KB at most), of which
// up to two are on their way while one is summed.  (With the next row in
// registers instead, a warp has 1 KB on its way at 256 experts and waits for
// it: 131072 x 256 in 40 us against 35.)
constexpr int kLossRing = 3;
constexpr int kLossChunk = 4096;  // bytes

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int VPL>
constexpr int rows_at_once()  // rows that a lane works on side by side
{
    return VPL <= 8 ? 2 : 1;
}

// (One block fits an SM.  Saying so for the short rows keeps the compiler from
// spilling to 40 registers; for the long ones it changed nothing or, at 512
// experts, cost 2 %.)
template <int VPL, int LPR>
__global__ void __launch_bounds__(kLossWarps * 32, VPL <= 8 ? 1 : 0)
    balance_bulk_kernel(const float* __restrict__ logits, int64_t T, int E, int rows, float* __restrict__ part,
                        double* __restrict__ part_z, int* __restrict__ part_n, Waits waits)
{
    constexpr int kGroups = 32 / LPR, kOnce = rows_at_once<VPL>();
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float s_sum[VPL * LPR];
    __shared__ __align__(8) uint64_t s_bar[kLossWarps][kLossRing];
    __shared__ int s_abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    allow_next();
    if (lane == 0) {
        for (int i = 0; i < kLossRing; ++i) sm100::mbar_init(sm100::smem_u32(&s_bar[warp][i]), 1 + waits.extra(kHoldLoss));
        sm100::fence_barrier_init();
    }
    if (threadIdx.x == 0) s_abort = 0;
    __syncthreads();
    uint8_t* const mine = ring + warp * kLossRing * kLossChunk;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLossWarps * rows;
    const int64_t t0 = (static_cast<int64_t>(warp) * gridDim.x + blockIdx.x) * rows;
    auto fetch = [&](int64_t t, int slot) {
        if (lane == 0 && t < T) {
            const uint32_t bytes = static_cast<uint32_t>(min(static_cast<int64_t>(rows), T - t)) * E * 4;
            const uint32_t bar = sm100::smem_u32(&s_bar[warp][slot]);
            sm100::mbar_arrive_expect_tx(bar, bytes);
            bulk_load(sm100::smem_u32(mine) + slot * kLossChunk, logits + t * E, bytes, bar);
        }
    };
#pragma unroll
    for (int i = 0; i < kLossRing; ++i) fetch(t0 + i * step, i);
    WarpSums<VPL> sums;
    int slot = 0, turn = 0;
    bool ok = true;
    for (int64_t t = t0; t < T; t += step) {
        ok = ok && sm100::mbar_wait_bounded(sm100::smem_u32(&s_bar[warp][slot]), turn & 1, &s_abort, waits.ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        const int have = static_cast<int>(min(static_cast<int64_t>(rows), T - t));
        const float* const chunk = reinterpret_cast<const float*>(mine + slot * kLossChunk);
        for (int r0 = 0; r0 < have; r0 += kGroups * kOnce) {
            float v[kOnce][VPL];
#pragma unroll
            for (int o = 0; o < kOnce; ++o) {
                const int r = r0 + o * kGroups + lane / LPR;
#pragma unroll
                for (int i = 0; i < VPL; i += 4) {
                    const int e = expert_of<LPR>(lane, i);
                    const float4 q = (r < have && e < E)
                                         ? *reinterpret_cast<const float4*>(chunk + r * E + e)
                                         : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    v[o][i] = q.x;
                    v[o][i + 1] = q.y;
                    v[o][i + 2] = q.z;
                    v[o][i + 3] = q.w;
                }
            }
#pragma unroll
            for (int o = 0; o < kOnce; ++o) sums.template add<LPR>(v[o]);
        }
        __syncwarp();
        fetch(t + kLossRing * step, slot);
        if (++slot == kLossRing) {
            slot = 0;
            ++turn;
        }
    }
    const LossSums own = join_warps<VPL, LPR>(sums, E, s_sum);
    const bool lost = s_abort != 0;  // (every warp is past its waits)
    write_part<VPL, LPR>(own, s_sum, lost, E, part, part_z, part_n);
    if (lost) sm100::settle();
}

// ... summed by one cluster of eight blocks, which share the experts; the
// threads of a block take every kGroups-th partial row of one expert, and the
// groups are added in order.
constexpr int kFinalThreads = kLossWarps * 32;
constexpr int kFinalBlocks = 8;
__global__ void __launch_bounds__(kFinalThreads)
    balance_final_kernel(const float* __restrict__ part, const double* __restrict__ part_z,
                         const int* __restrict__ part_n, int nb, int E, const int32_t* __restrict__ offsets,
                         float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob_mean)
{
    __shared__ double s_group[kFinalThreads];
    __shared__ double s_term[kFinalBlocks];
    __shared__ double s_red[kLossWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    cluster_arrive();  // this block has started: waited for before a peer's memory is written
    const int share = (E + kFinalBlocks - 1) / kFinalBlocks;  // at most 128 experts a block
    int width = 1;                                            // experts side by side, a power of two
    while (width < share) width *= 2;
    const int groups = kFinalThreads / width;
    const int col = threadIdx.x % width, grp = threadIdx.x / width;
    const int e = rank * share + col;
    const bool in = col < share && e < E;
    const int32_t c = in ? __ldg(offsets + e + 1) - __ldg(offsets + e) : 0;
    const int32_t P = __ldg(offsets + E);
    wait_previous();  // the partial sums
    double z = 0.0, nd = 0.0, s = 0.0;
    for (int b = threadIdx.x; b < nb; b += kFinalThreads) {
        z += __ldcg(part_z + b);
        nd += __ldcg(part_n + b);
    }
    if (in) {
#pragma unroll 8
        for (int b = grp; b < nb; b += groups) s += __ldcg(part + static_cast<int64_t>(b) * E + e);
    }
    z = block_sum(z, s_red);
    nd = block_sum(nd, s_red);
    s_group[threadIdx.x] = s;
    __syncthreads();
    const double inv_n = 1.0 / (nd > 0.0 ? nd : 1.0);
    double term = 0.0;
    if (grp == 0 && in) {
        s = 0.0;
        for (int q = 0; q < groups; ++q) s += s_group[q * width + col];
        s *= inv_n;
        term = s * c;
        prob_mean[e] = static_cast<float>(s);
        counts[e] = c;
    }
    term = block_sum(term, s_red);
    __syncwarp();
    cluster_wait();  // every block of the cluster has started
    if (threadIdx.x == 0) cluster.map_shared_rank(s_term, 0)[rank] = term;
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
        double sum = 0.0;
        for (int b = 0; b < kFinalBlocks; ++b) sum += s_term[b];
        loss[0] = static_cast<float>(E * sum / (P > 0 ? P : 1));
        loss[1] = static_cast<float>(z * inv_n);
        counts[E] = nd < 0.0 ? kNoCount : static_cast<int32_t>(nd);
    }
}

// ----------------------------------------------------------------- gradient

// g_e = d0 E c_e / (P N) of the lane's experts, and 2 d1 / N.
template <int VPL, int LPR>
__device__ __forceinline__ float balance_slopes(const int32_t* __restrict__ counts, const float* __restrict__ d_loss,
                                                int E, int lane, float (&g)[VPL])
{
    if (!d_loss) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) g[i] = 0.0f;
        return 0.0f;
    }
    double P = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = expert_of<LPR>(lane, i);
        const int c = (e < E) ? __ldg(counts + e) : 0;
        g[i] = static_cast<float>(c);
        P += c;
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) P += __shfl_xor_sync(0xFFFFFFFFu, P, off);
    const int n = __ldg(counts + E);
    const double inv_n = n < 0 ? NAN : 1.0 / (n > 0 ? n : 1);  // negative: not counted (kNoCount)
    const float f = static_cast<float>(__ldg(d_loss) * E * inv_n / (P > 0.0 ? P : 1.0));
#pragma unroll
    for (int i = 0; i < VPL; ++i) g[i] *= f;
    return static_cast<float>(2.0 * __ldg(d_loss + 1) * inv_n);
}

// A row's gradient from its logits v: balance and z terms (if losses), plus
// slot_d of lane j at expert slot_id of lane j for the k slots.
template <int VPL, int LPR>
__device__ __forceinline__ void grad_row(float (&v)[VPL], bool losses, const float (&g)[VPL], float zc, int E, int k,
                                         int slot_id, float slot_d, float* __restrict__ dst, int lane, bool ok)
{
    if (losses) {
        float inv, lse, inner = 0.0f;
        softmax_row<VPL, LPR>(v, inv, lse);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] *= inv;
            inner += v[i] * g[i];
        }
        inner = row_sum<LPR>(inner);
        const float slope = zc * lse;
        if (fabsf(slope) < INFINITY) {
            inner -= slope;
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] *= g[i] - inner;
        } else {  // times the probability first: in range where the product is, 0 where p is
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = fmaf(v[i] * zc, lse, v[i] * (g[i] - inner));
        }
    } else {  // 0 times the softmax would pass on the NaN of a +Inf logit
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = 0.0f;
    }
    for (int j = 0; j < k; ++j) {
        const int id = __shfl_sync(0xFFFFFFFFu, slot_id, j);
        const float d = __shfl_sync(0xFFFFFFFFu, slot_d, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (id == expert_of<LPR>(lane, i)) v[i] += d;
    }
    if (!ok) return;
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
        const int e = expert_of<LPR>(lane, i);
        if (E % 4 == 0) {
            if (e < E) *reinterpret_cast<float4*>(dst + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (e + u < E) dst[e + u] = v[i + u];
        }
    }
}

// With slot rows.  Persistent blocks, one per SM, tokens dealt round: a
// producer warp streams the filled slot rows and dout in chunks of 1024
// columns by bulk copies, as far ahead as the ring holds (up to about 200 KB,
// across tokens), eight warps take the dots out of shared memory, and four
// more finish the tokens (sum of the warps' dots, softmax gradient, the row's
// write), so that no load waits for a token's end.  (One block per token with
// direct loads: 137 us against 113 at T = 4096, H = 5120, k = 8.)
constexpr int kDotWarps = 8;
constexpr int kTailWarps = 4;
constexpr int kGradThreads = (kDotWarps + 1 + kTailWarps) * 32;
constexpr int kChunk = 1024;     // columns: one float4 per thread of the dot warps
constexpr int kSlotBatch = 8;    // slots per stage
constexpr int kMaxStages = 16;
constexpr int kDotBufs = 8;      // tokens between dots and tails
constexpr int kGradRing = 200 * 1024;

template <int VPL>
__global__ void __launch_bounds__(kGradThreads, 1)
    route_grad_kernel(const float* __restrict__ logits, int64_t T, int E, const int32_t* __restrict__ ids,
                      const float* __restrict__ w, int k, const float* __restrict__ y,
                      const uint16_t* __restrict__ dout, int H, float rs, const int32_t* __restrict__ counts,
                      const float* __restrict__ d_loss, float* __restrict__ d_logits, int stages, int stage_bytes,
                      Waits waits)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_dots[kDotBufs], s_done[kDotBufs];
    __shared__ float s_red[kDotBufs][kDotWarps][32];
    __shared__ int s_abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            sm100::mbar_init(sm100::smem_u32(&s_full[i]), 1 + waits.extra(kHoldGradFull));
            sm100::mbar_init(sm100::smem_u32(&s_empty[i]), kDotWarps + waits.extra(kHoldGradEmpty));
        }
        for (int i = 0; i < kDotBufs; ++i) {
            sm100::mbar_init(sm100::smem_u32(&s_dots[i]), kDotWarps);
            sm100::mbar_init(sm100::smem_u32(&s_done[i]), 1);
        }
        sm100::fence_barrier_init();
        s_abort = 0;
    }
    __syncthreads();
    auto wait = [&](uint64_t* b, int phase) {
        return sm100::mbar_wait_bounded(sm100::smem_u32(b), phase & 1, &s_abort, waits.ns);
    };
    // slots of a token that hold an expert, as a mask
    auto load_id = [&](int64_t t) { return (t < T && lane < k) ? __ldg(ids + t * k + lane) : -1; };
    auto mask_of = [&](int id) { return __ballot_sync(0xFFFFFFFFu, id >= 0 && id < E); };
    if (warp < kDotWarps) {
        int st = 0, turn = 0, buf = 0, pass = 0;
        bool ok = true;
        int id = load_id(blockIdx.x);
        for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
            const uint32_t mask = mask_of(id);
            id = load_id(t + gridDim.x);
            if (pass > 0) ok = ok && wait(&s_done[buf], pass - 1);
            for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
                const uint32_t m = (mask >> j0) & 0xFFu;
                if (m == 0) continue;
                float acc[kSlotBatch];
#pragma unroll
                for (int u = 0; u < kSlotBatch; ++u) acc[u] = 0.0f;
                for (int c0 = 0; c0 < H; c0 += kChunk) {
                    ok = __all_sync(0xFFFFFFFFu, ok && wait(&s_full[st], turn));
                    if (!ok) break;
                    const uint8_t* s = ring + st * stage_bytes;
                    const int c = threadIdx.x * 4;
                    if (c0 + c < H) {
                        const uint2 d2 = *reinterpret_cast<const uint2*>(s + c * 2);
                        const float2 d01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&d2.x));
                        const float2 d23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&d2.y));
#pragma unroll
                        for (int u = 0; u < kSlotBatch; ++u) {
                            if (!((m >> u) & 1u)) continue;
                            const float4 r =
                                *reinterpret_cast<const float4*>(s + kChunk * 2 + u * kChunk * 4 + c * 4);
                            acc[u] += d01.x * r.x + d01.y * r.y + d23.x * r.z + d23.y * r.w;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) sm100::mbar_arrive(sm100::smem_u32(&s_empty[st]));
                    if (++st == stages) {
                        st = 0;
                        ++turn;
                    }
                }
                // sums over the warp, halving the slots a lane carries: lane l
                // ends with slot (l / 4) % 8
#pragma unroll
                for (int half = 4; half > 0; half >>= 1) {
                    const bool up = lane & (half * 4);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (u >= half) continue;
                        const float keep = up ? acc[u + half] : acc[u], give = up ? acc[u] : acc[u + half];
                        acc[u] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, half * 4);
                    }
                }
                acc[0] += __shfl_xor_sync(0xFFFFFFFFu, acc[0], 2);
                acc[0] += __shfl_xor_sync(0xFFFFFFFFu, acc[0], 1);
                // NaN once a wait ran out: columns, or the tail's leave to write, are
                // missing.  (The warp arrives below all the same, also out of turn, but
                // never before its NaN is in every token that the arrival can complete.)
                if ((lane & 3) == 0) s_red[buf][warp][j0 + lane / 4] = ok ? acc[0] : NAN;
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sm100::smem_u32(&s_dots[buf]));
            if (++buf == kDotBufs) {
                buf = 0;
                ++pass;
            }
        }
    } else if (warp == kDotWarps) {
        int st = 0, turn = 0;
        bool ok = true;
        int id = load_id(blockIdx.x);
        for (int64_t t = blockIdx.x; t < T && ok; t += gridDim.x) {
            const uint32_t mask = mask_of(id);
            id = load_id(t + gridDim.x);
            for (int j0 = 0; j0 < k && ok; j0 += kSlotBatch) {
                const uint32_t m = (mask >> j0) & 0xFFu;
                if (m == 0) continue;
                for (int c0 = 0; c0 < H; c0 += kChunk) {
                    if (turn > 0) ok = wait(&s_empty[st], turn - 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const uint32_t cols = min(kChunk, H - c0);
                    const uint32_t s = sm100::smem_u32(ring) + st * stage_bytes;
                    const uint32_t bar = sm100::smem_u32(&s_full[st]);
                    if (lane == 0) sm100::mbar_arrive_expect_tx(bar, cols * (2 + 4 * __popc(m)));
                    __syncwarp();
                    if (lane < kSlotBatch) {
                        if ((m >> lane) & 1u)
                            bulk_load(s + kChunk * 2 + lane * kChunk * 4, y + (t * k + j0 + lane) * H + c0, cols * 4, bar);
                    } else if (lane == kSlotBatch) {
                        bulk_load(s, dout + t * H + c0, cols * 2, bar);
                    }
                    if (++st == stages) {
                        st = 0;
                        ++turn;
                    }
                }
            }
        }
    } else {
        // every kTailWarps-th token of the block
        const int tail = warp - kDotWarps - 1;
        float g[VPL];
        const float zc = balance_slopes<VPL, 32>(counts, d_loss, E, lane, g);
        int64_t n = tail;
        bool ok = true;
        for (int64_t t = blockIdx.x + n * gridDim.x; t < T; n += kTailWarps, t = blockIdx.x + n * gridDim.x) {
            float v[VPL];
            load_row<VPL, 32>(logits + t * E, E, lane, true, v);
            int id = load_id(t);
            if (id < 0 || id >= E) id = -1;
            const float wj = id >= 0 ? __ldg(w + t * k + lane) : 0.0f;
            const int buf = static_cast<int>(n % kDotBufs);
            ok = ok && wait(&s_dots[buf], static_cast<int>(n / kDotBufs));
            float s = 0.0f;
            if (id >= 0) {
#pragma unroll
                for (int q = 0; q < kDotWarps; ++q) s += s_red[buf][q][lane];
                s *= rs;
            }
            if (!ok) s = NAN;  // a wait that ran out
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sm100::smem_u32(&s_done[buf]));
            const float total = row_sum<32>(s);
            grad_row<VPL, 32>(v, d_loss != nullptr, g, zc, E, k, id, s - wj * total, d_logits + t * E, lane, true);
        }
    }
    __syncthreads();
    if (s_abort) sm100::settle();
}

// Without slot rows: the balance and z gradients alone, 32 / LPR rows per warp.
constexpr int kBalanceGradThreads = 256;
template <int VPL, int LPR>
__global__ void __launch_bounds__(kBalanceGradThreads)
    balance_grad_kernel(const float* __restrict__ logits, int64_t T, int E, const int32_t* __restrict__ counts,
                        const float* __restrict__ d_loss, float* __restrict__ d_logits)
{
    constexpr int kRows = 32 / LPR;
    const int lane = threadIdx.x & 31;
    float g[VPL];
    const float zc = balance_slopes<VPL, LPR>(counts, d_loss, E, lane, g);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kBalanceGradThreads / 32) * kRows;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kBalanceGradThreads / 32) + (threadIdx.x >> 5)) * kRows;
         t0 < T; t0 += step) {
        const int64_t t = t0 + lane / LPR;
        float v[VPL];
        load_row<VPL, LPR>(logits + t * E, E, lane, t < T, v);
        grad_row<VPL, LPR>(v, true, g, zc, E, 0, -1, 0.0f, d_logits + t * E, lane, t < T);
    }
}

// Blocks of the two-launch loss.
int64_t loss_blocks(int64_t T)
{
    const int64_t want = ceil_div64(T > 0 ? T : 1, kLossWarps);
    return want < kLossMaxBlocks ? want : kLossMaxBlocks;
}

// One cluster while the logits take no longer to read through eight SMs than
// a second launch costs.
bool loss_small(int64_t T, int E) { return T * E <= (1 << 18); }

template <int VPL, int LPR>
cudaError_t balance(const float* logits, int64_t T, int E, const int32_t* offsets, float* loss, int32_t* counts,
                    float* prob_mean, float* part, double* pz, int* pn, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    cfg.blockDim = dim3(kLossWarps * 32);
    cfg.stream = s;
    cfg.attrs = at;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    if (loss_small(T, E)) {
        unsigned nc = 1;  // blocks with four rows per warp or more
        while (nc < kSmallBlocks && T > static_cast<int64_t>(nc) * kLossWarps * 4 * (32 / LPR)) nc *= 2;
        at[0].val.clusterDim.x = nc;
        cfg.numAttrs = nc > 1 ? 1 : 0;  // (a cluster of one needs none, and launches faster)
        cfg.gridDim = dim3(nc);
        return cudaLaunchKernelEx(&cfg, balance_small_kernel<VPL, LPR>, logits, T, E, offsets, loss, counts, prob_mean);
    }
    const int nb = static_cast<int>(loss_blocks(T));
    cudaError_t err;
    if (E % 4 == 0) {
        // rows per chunk: as many as fit, but no more than give every warp one
        const int once = 32 / LPR * rows_at_once<VPL>();
        int64_t rows = ceil_div64(T, static_cast<int64_t>(nb) * kLossWarps);
        rows = ceil_div64(rows, once) * once;
        const int most = kLossChunk / (4 * E) / once * once;
        err = allow_smem<balance_bulk_kernel<VPL, LPR>>(kLossWarps * kLossRing * kLossChunk);
        if (err != cudaSuccess) return err;
        balance_bulk_kernel<VPL, LPR><<<nb, kLossWarps * 32, kLossWarps * kLossRing * kLossChunk, s>>>(
            logits, T, E, rows < most ? static_cast<int>(rows) : most, part, pz, pn, waits());
        err = cudaGetLastError();
    } else {
        balance_partial_kernel<VPL, LPR><<<nb, kLossWarps * 32, 0, s>>>(logits, T, E, part, pz, pn);
        err = cudaGetLastError();
    }
    if (err != cudaSuccess) return err;
    at[0].val.clusterDim.x = kFinalBlocks;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(kFinalBlocks);
    return cudaLaunchKernelEx(&cfg, balance_final_kernel, static_cast<const float*>(part),
                              static_cast<const double*>(pz), static_cast<const int*>(pn), nb, E, offsets, loss, counts,
                              prob_mean);
}

template <int VPL, int LPR>
cudaError_t balance_grad(const RouteGradArgs& a, int sm_count, cudaStream_t s)
{
    const int64_t want = ceil_div64(a.T, kBalanceGradThreads / 32 * (32 / LPR));
    const int64_t cap = static_cast<int64_t>(sm_count) * 8;
    balance_grad_kernel<VPL, LPR><<<static_cast<unsigned>(want < cap ? want : cap), kBalanceGradThreads, 0, s>>>(
        a.logits, a.T, a.E, a.counts, a.d_loss, a.d_logits);
    return cudaGetLastError();
}

template <int VPL>
cudaError_t route_grad(const RouteGradArgs& a, int sm_count, cudaStream_t s)
{
    const int slots = a.k < kSlotBatch ? a.k : kSlotBatch;
    const int stage_bytes = kChunk * (2 + 4 * slots);
    const int stages = kGradRing / stage_bytes < kMaxStages ? kGradRing / stage_bytes : kMaxStages;
    cudaError_t err = allow_smem<route_grad_kernel<VPL>>(kGradRing);
    if (err != cudaSuccess) return err;
    const unsigned grid = static_cast<unsigned>(a.T < sm_count ? a.T : sm_count);
    route_grad_kernel<VPL><<<grid, kGradThreads, stages * stage_bytes, s>>>(
        a.logits, a.T, a.E, a.ids, a.w, a.k, a.y, a.dout, a.H, a.rs, a.counts, a.d_loss, a.d_logits, stages,
        stage_bytes, waits());
    return cudaGetLastError();
}

}  // namespace

size_t balance_ws_layout(int64_t T, int E, size_t* off_n, size_t* off_part)
{
    const int64_t nb = loss_blocks(T);
    size_t o = align_up(static_cast<size_t>(nb) * 8, 256);
    *off_n = o;
    o = align_up(o + static_cast<size_t>(nb) * 4, 256);
    *off_part = o;
    return align_up(o + static_cast<size_t>(nb) * (E > 0 ? E : 1) * 4, 256);
}

cudaError_t launch_balance_loss(const float* logits, int64_t T, int E, const int32_t* offsets, float* loss,
                                int32_t* counts, float* prob_mean, void* ws, cudaStream_t s)
{
    size_t off_n, off_part;
    balance_ws_layout(T, E, &off_n, &off_part);
    uint8_t* w8 = static_cast<uint8_t*>(ws);
    double* pz = reinterpret_cast<double*>(w8);
    int* pn = reinterpret_cast<int*>(w8 + off_n);
    float* part = reinterpret_cast<float*>(w8 + off_part);
    if (E <= 32) return balance<4, 8>(logits, T, E, offsets, loss, counts, prob_mean, part, pz, pn, s);
    if (E <= 64) return balance<4, 16>(logits, T, E, offsets, loss, counts, prob_mean, part, pz, pn, s);
    if (E <= 128) return balance<4, 32>(logits, T, E, offsets, loss, counts, prob_mean, part, pz, pn, s);
    if (E <= 256) return balance<8, 32>(logits, T, E, offsets, loss, counts, prob_mean, part, pz, pn, s);
    if (E <= 512) return balance<16, 32>(logits, T, E, offsets, loss, counts, prob_mean, part, pz, pn, s);
    return balance<32, 32>(logits, T, E, offsets, loss, counts, prob_mean, part, pz, pn, s);
}

cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    DeviceInfo di;
    if (!device_info(&di)) return cudaErrorUnknown;
    const int sms = di.sm_count;
    if (a.y) {
        if (a.E <= 128) return route_grad<4>(a, sms, s);
        if (a.E <= 256) return route_grad<8>(a, sms, s);
        if (a.E <= 512) return route_grad<16>(a, sms, s);
        return route_grad<32>(a, sms, s);
    }
    if (a.E <= 32) return balance_grad<4, 8>(a, sms, s);
    if (a.E <= 64) return balance_grad<4, 16>(a, sms, s);
    if (a.E <= 128) return balance_grad<4, 32>(a, sms, s);
    if (a.E <= 256) return balance_grad<8, 32>(a, sms, s);
    if (a.E <= 512) return balance_grad<16, 32>(a, sms, s);
    return balance_grad<32, 32>(a, sms, s);
}

}  // namespace fp8moe
