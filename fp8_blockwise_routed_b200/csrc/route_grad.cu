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
#include <cuda_bf16.h>

#include "internal.h"

namespace fp8moe {
namespace {

constexpr int kLossWarps = 16;   // tokens in flight per block of the loss kernel
constexpr int kGradThreads = 256;
constexpr int kSlotBatch = 8;    // slot rows read together per thread

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

template <int VPL>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float (&v)[VPL])
{
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        v[i] = (e < E) ? __ldg(row + e) : -INFINITY;
    }
}

// Softmax of a row over its selectable entries, in place (0 where not
// selectable); returns whether there is any, and log(sum exp) in lse.  A +Inf
// logit gives NaN (Inf - Inf), as in the router's weights.
template <int VPL>
__device__ __forceinline__ bool softmax_row(float (&v)[VPL], float& lse)
{
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (isnan(v[i])) v[i] = -INFINITY;
        m = fmaxf(m, v[i]);
    }
    m = warp_max(m);
    if (m == -INFINITY) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = 0.0f;
        lse = 0.0f;
        return false;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        v[i] = (v[i] == -INFINITY) ? 0.0f : expf(v[i] - m);
        sum += v[i];
    }
    sum = warp_sum(sum);
    const float inv = __fdiv_rn(1.0f, sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] *= inv;
    lse = m + logf(sum);
    return true;
}

// Per-block sums of the probabilities, of lse^2 and of the counted tokens:
// part [gridDim.x][E] FP32, part_z [gridDim.x] FP64, part_n [gridDim.x].
template <int VPL>
__global__ void __launch_bounds__(kLossWarps * 32)
    balance_partial_kernel(const float* __restrict__ logits, int64_t T, int E, float* __restrict__ part,
                           double* __restrict__ part_z, int* __restrict__ part_n)
{
    __shared__ float red[kLossWarps][256];
    __shared__ double red_z[kLossWarps];
    __shared__ int red_n[kLossWarps];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    float acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
    double z = 0.0;
    int n = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLossWarps;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kLossWarps + warp;
    float next[VPL];
    if (t < T) load_row<VPL>(logits + t * E, E, lane, next);
    for (; t < T; t += step) {
        float v[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = next[i];
        if (t + step < T) load_row<VPL>(logits + (t + step) * E, E, lane, next);
        float lse;
        if (softmax_row<VPL>(v, lse)) {
            z += static_cast<double>(lse) * lse;
            ++n;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += v[i];
    }
    if (lane == 0) {
        red_z[warp] = z;
        red_n[warp] = n;
    }
    // warps summed in order, 256 experts at a time
#pragma unroll
    for (int i0 = 0; i0 < VPL; i0 += 8) {
        __syncthreads();
#pragma unroll
        for (int i = i0; i < VPL && i < i0 + 8; ++i) red[warp][lane + 32 * (i - i0)] = acc[i];
        __syncthreads();
        const int e = 32 * i0 + threadIdx.x;
        if (threadIdx.x < 256 && threadIdx.x < 32 * (VPL - i0) && e < E) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kLossWarps; ++w) s += red[w][threadIdx.x];
            part[static_cast<int64_t>(blockIdx.x) * E + e] = s;
        }
    }
    if (threadIdx.x == 0) {
        double sz = 0.0;
        int sn = 0;
        for (int w = 0; w < kLossWarps; ++w) {
            sz += red_z[w];
            sn += red_n[w];
        }
        part_z[blockIdx.x] = sz;
        part_n[blockIdx.x] = sn;
    }
}

// One block: sums the partials in block order and writes the losses.
__global__ void __launch_bounds__(1024)
    balance_final_kernel(const float* __restrict__ part, const double* __restrict__ part_z,
                         const int* __restrict__ part_n, int nb, int E, const int32_t* __restrict__ offsets,
                         float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob_mean)
{
    __shared__ double red[32];
    __shared__ int s_n;
    __shared__ double s_z;
    if (threadIdx.x < 32) {
        double z = 0.0;
        int n = 0;
        for (int b = threadIdx.x; b < nb; b += 32) {
            z += part_z[b];
            n += part_n[b];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
            n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
        }
        if (threadIdx.x == 0) {
            s_n = n;
            s_z = z;
        }
    }
    __syncthreads();
    const int n = s_n;
    const double inv_n = 1.0 / (n > 0 ? n : 1);
    double term = 0.0;
    const int e = threadIdx.x;
    if (e < E) {
        double s = 0.0;
        for (int b = 0; b < nb; ++b) s += part[static_cast<int64_t>(b) * E + e];
        const int32_t c = offsets[e + 1] - offsets[e];
        s *= inv_n;
        term = s * c;
        prob_mean[e] = static_cast<float>(s);
        counts[e] = c;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int w = 0; w < 32; ++w) sum += red[w];
        const int32_t P = offsets[E];
        loss[0] = static_cast<float>(E * sum / (P > 0 ? P : 1));
        loss[1] = static_cast<float>(s_z * inv_n);
        counts[E] = n;
    }
}

// The balance and z gradients of one token's row by one warp, plus the
// routing part that the caller gives per slot: slot_id / slot_d of lane j.
template <int VPL>
__device__ __forceinline__ void grad_row(float (&v)[VPL], const float (&g)[VPL], float zc, int E, int k,
                                         int slot_id, float slot_d, float* __restrict__ dst, int lane)
{
    float lse, inner = 0.0f;
    softmax_row<VPL>(v, lse);
#pragma unroll
    for (int i = 0; i < VPL; ++i) inner += v[i] * g[i];
    inner = warp_sum(inner) - zc * lse;
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] *= g[i] - inner;
    for (int j = 0; j < k; ++j) {
        const int id = __shfl_sync(0xFFFFFFFFu, slot_id, j);
        const float d = __shfl_sync(0xFFFFFFFFu, slot_d, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (id == lane + 32 * i) v[i] += d;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) dst[lane + 32 * i] = v[i];
}

// g_e = d0 E c_e / (P N) of the lane's experts, and 2 d1 / N.
template <int VPL>
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
        const int e = lane + 32 * i;
        const int c = (e < E) ? __ldg(counts + e) : 0;
        g[i] = static_cast<float>(c);
        P += c;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) P += __shfl_xor_sync(0xFFFFFFFFu, P, off);
    const int n = __ldg(counts + E);
    const double inv_n = 1.0 / (n > 0 ? n : 1);
    const float f = static_cast<float>(__ldg(d_loss) * E * inv_n / (P > 0.0 ? P : 1.0));
#pragma unroll
    for (int i = 0; i < VPL; ++i) g[i] *= f;
    return static_cast<float>(2.0 * __ldg(d_loss + 1) * inv_n);
}

// One block per token: its warps take the dots of dout with the filled slot
// rows, its first warp the softmax gradient and the row's write.
template <int VPL>
__global__ void __launch_bounds__(kGradThreads)
    route_grad_kernel(const float* __restrict__ logits, int64_t T, int E, const int32_t* __restrict__ ids,
                      const float* __restrict__ w, int k, const float4* __restrict__ y,
                      const uint2* __restrict__ dout, int H4, float rs, const int32_t* __restrict__ counts,
                      const float* __restrict__ d_loss, float* __restrict__ d_logits)
{
    __shared__ float red[kGradThreads / 32][32];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    float v[VPL], g[VPL];
    if (warp == 0) load_row<VPL>(logits + t * E, E, lane, v);
    for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
        float acc[kSlotBatch];
        bool ok[kSlotBatch];
        bool any = false;
#pragma unroll
        for (int u = 0; u < kSlotBatch; ++u) {
            const int id = (j0 + u < k) ? __ldg(ids + t * k + j0 + u) : -1;
            ok[u] = id >= 0 && id < E;
            any |= ok[u];
            acc[u] = 0.0f;
        }
        if (any) {
            for (int c = threadIdx.x; c < H4; c += kGradThreads) {
                const uint2 d2 = __ldg(dout + t * H4 + c);
                const float2 d01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&d2.x));
                const float2 d23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&d2.y));
                float4 r[kSlotBatch];
#pragma unroll
                for (int u = 0; u < kSlotBatch; ++u)
                    r[u] = ok[u] ? __ldcs(y + (t * k + j0 + u) * H4 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int u = 0; u < kSlotBatch; ++u)
                    if (ok[u]) acc[u] += d01.x * r[u].x + d01.y * r[u].y + d23.x * r[u].z + d23.y * r[u].w;
            }
        }
#pragma unroll
        for (int u = 0; u < kSlotBatch; ++u) {
            const float s = warp_sum(acc[u]);
            if (lane == 0) red[warp][j0 + u] = s;
        }
    }
    __syncthreads();
    if (warp != 0) return;
    float s = 0.0f, wj = 0.0f;
    int id = -1;
    if (lane < k) {
        id = __ldg(ids + t * k + lane);
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) {
            wj = __ldg(w + t * k + lane);
            for (int q = 0; q < kGradThreads / 32; ++q) s += red[q][lane];
            s *= rs;
        }
    }
    const float total = warp_sum(s);
    const float zc = balance_slopes<VPL>(counts, d_loss, E, lane, g);
    grad_row<VPL>(v, g, zc, E, k, id, s - wj * total, d_logits + t * E, lane);
}

// Without slot rows: the balance and z gradients alone, one warp per token.
template <int VPL>
__global__ void __launch_bounds__(kGradThreads)
    balance_grad_kernel(const float* __restrict__ logits, int64_t T, int E, const int32_t* __restrict__ counts,
                        const float* __restrict__ d_loss, float* __restrict__ d_logits)
{
    const int lane = threadIdx.x & 31;
    float g[VPL];
    const float zc = balance_slopes<VPL>(counts, d_loss, E, lane, g);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + (threadIdx.x >> 5); t < T;
         t += static_cast<int64_t>(gridDim.x) * (kGradThreads / 32)) {
        float v[VPL];
        load_row<VPL>(logits + t * E, E, lane, v);
        grad_row<VPL>(v, g, zc, E, 0, -1, 0.0f, d_logits + t * E, lane);
    }
}

int64_t loss_blocks(int64_t T)
{
    const int64_t want = ceil_div64(T > 0 ? T : 1, kLossWarps);
    return want < kLossMaxBlocks ? want : kLossMaxBlocks;
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
    const int nb = static_cast<int>(loss_blocks(T));
    if (E <= 64)
        balance_partial_kernel<2><<<nb, kLossWarps * 32, 0, s>>>(logits, T, E, part, pz, pn);
    else if (E <= 256)
        balance_partial_kernel<8><<<nb, kLossWarps * 32, 0, s>>>(logits, T, E, part, pz, pn);
    else
        balance_partial_kernel<32><<<nb, kLossWarps * 32, 0, s>>>(logits, T, E, part, pz, pn);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    balance_final_kernel<<<1, 1024, 0, s>>>(part, pz, pn, nb, E, offsets, loss, counts, prob_mean);
    return cudaGetLastError();
}

namespace {

template <int VPL>
cudaError_t route_grad(const RouteGradArgs& a, int sm_count, cudaStream_t s)
{
    if (a.y) {
        route_grad_kernel<VPL><<<static_cast<unsigned>(a.T), kGradThreads, 0, s>>>(
            a.logits, a.T, a.E, a.ids, a.w, a.k, reinterpret_cast<const float4*>(a.y),
            reinterpret_cast<const uint2*>(a.dout), a.H / 4, a.rs, a.counts, a.d_loss, a.d_logits);
    } else {
        const int64_t want = ceil_div64(a.T, kGradThreads / 32);
        const int64_t cap = static_cast<int64_t>(sm_count) * 8;
        balance_grad_kernel<VPL><<<static_cast<unsigned>(want < cap ? want : cap), kGradThreads, 0, s>>>(
            a.logits, a.T, a.E, a.counts, a.d_loss, a.d_logits);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    DeviceInfo di;
    if (!device_info(&di)) return cudaErrorUnknown;
    if (a.E <= 64) return route_grad<2>(a, di.sm_count, s);
    if (a.E <= 256) return route_grad<8>(a, di.sm_count, s);
    return route_grad<32>(a, di.sm_count, s);
}

}  // namespace fp8moe
