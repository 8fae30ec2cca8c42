// lora.cu -- low-rank adapters of many requests beside a shared projection,
// forward and backward.
//
// Adapter a holds A_a [R, C_in] and B_a [R, C_out] (both rank-major: a rank
// row is contiguous) and a scale f_a.  For a token t of adapter a, at place p
// of the tokens sorted by adapter:
//   v_p   = A_a x_t                         (shrink)
//   out_t = base_t + f_a B_a^T v_p          (expand)
// and, for dout the gradient of out,
//   dv_p  = f_a B_a dout_t                  (shrink)
//   dx_t  = dx_base_t + A_a^T dv_p          (expand)
//   dA_a  = sum_p dv_p x_t^T,  dB_a = f_a sum_p v_p dout_t^T   (outer)
// so three kernels carry both directions; the rank-major B is what makes the
// backward shrink and expand the same products as the forward ones.
//
// Precision: x, dout, A and B are BF16 and their products exact in FP32; v
// and dv stay FP32.  Where v or dv meets the tensor cores it is split into
// three BF16 terms (8 + 8 + 8 mantissa bits, h + m + l = v exactly), so the
// products carry FP32's precision; the small terms are summed first.
//
// Everything is bound by moving rows (2 C bytes of x or dout, 8 C of base and
// out) and the adapters in use; the products fit under that on the tensor
// cores.  No atomics: every sum has a fixed order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "internal.h"

namespace cg = cooperative_groups;

namespace fp8moe {
namespace {

// D += A B, m16n8k16, BF16 inputs, FP32 accumulation.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// a = h + m + l in BF16 terms; h alone where a is not finite or rounds to
// infinity, so that no Inf - Inf turns an infinity into NaN.
struct Split {
    float h, m, l;
};
__device__ __forceinline__ Split split3(float a)
{
    Split s;
    s.h = __bfloat162float(__float2bfloat16_rn(a));
    const bool fin = fabsf(s.h) <= 3.4028234e38f;
    const float r = fin ? a - s.h : 0.0f;
    s.m = __bfloat162float(__float2bfloat16_rn(r));
    s.l = r - s.m;
    return s;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// The `tile`-th group of at most BT sorted tokens of one adapter, adapters in
// order.  Called by the whole block; offsets are clamped to [0, T], so a
// tile never leaves the token list whatever they hold.
struct Tile {
    int a;     // adapter, -1: past the last tile
    int p0;    // first sorted place
    int count;
};
template <int THREADS>
__device__ __forceinline__ Tile find_tile(const LoraRows& rows, int bt, int64_t tile)
{
    __shared__ int s_warp[THREADS / 32];
    __shared__ Tile s_tile;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int T = static_cast<int>(rows.T);
    constexpr int kMaxPer = 1024 / THREADS;  // n <= 1024
    if (threadIdx.x == 0) s_tile.a = -1;
    int lo[kMaxPer], cnt[kMaxPer];
    int mine = 0;
    const int per = (rows.n + THREADS - 1) / THREADS;
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) {
        const int a = threadIdx.x * per + i;
        lo[i] = cnt[i] = 0;
        if (i < per && a < rows.n) {
            lo[i] = min(max(__ldg(rows.offsets + a), 0), T);
            cnt[i] = min(max(__ldg(rows.offsets + a + 1), lo[i]), T) - lo[i];
            mine += (cnt[i] + bt - 1) / bt;
        }
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) {
        const int nt = (cnt[i] + bt - 1) / bt;
        if (tile >= before && tile < before + nt) {
            const int skip = static_cast<int>(tile - before) * bt;
            s_tile = Tile{static_cast<int>(threadIdx.x * per + i), lo[i] + skip, min(bt, cnt[i] - skip)};
        }
        before += nt;
    }
    __syncthreads();
    return s_tile;
}

// Tiles of bt tokens that T tokens over n adapters can need at most.
int64_t max_tiles(int64_t T, int n, int bt) { return ceil_div64(T, bt) + (T < n ? T : n); }

// ------------------------------------------------------------------ shrink
//
// v[p, r] = f_a sum_c x[tok, c] w[a, r, c], 8 tokens and 16 MR ranks per
// cluster.  Ranks are the rows of the MMA and tokens its columns; both
// operands go from global memory to registers in 16-byte pieces, which the
// free choice of the order of the sum allows: lane q of a quad takes columns
// 8q .. 8q+7 of a 32-column step as its K indices of two MMAs.  The columns
// are dealt to the warps of all blocks of the cluster; their sums are joined
// in shared memory and across the cluster in a fixed order.
constexpr int kShrinkThreads = 256;
constexpr int kShrinkTokens = 8;

template <int MR>
__global__ void __launch_bounds__(kShrinkThreads)
    lora_shrink_kernel(LoraRows rows, const uint16_t* __restrict__ x, int64_t ldx, int C,
                       const uint16_t* __restrict__ w, int R, int rblocks, const float* __restrict__ scales,
                       float* __restrict__ v)
{
    __shared__ float red[kShrinkThreads / 32][MR * 16 * kShrinkTokens];
    __shared__ float part[MR * 16 * kShrinkTokens];
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int64_t unit = blockIdx.x / nc;
    const Tile tile = find_tile<kShrinkThreads>(rows, kShrinkTokens, unit / rblocks);
    if (tile.a < 0) return;  // the whole cluster
    const int r0 = static_cast<int>(unit % rblocks) * MR * 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const uint16_t* xr = nullptr;
    if (g < tile.count) {
        const int tok = __ldg(rows.tokens + tile.p0 + g);
        if (tok >= 0 && tok < rows.T) xr = x + tok * ldx;
    }
    const uint16_t* wa = w + (static_cast<int64_t>(tile.a) * R + r0) * C;
    float acc[MR][4], sum[MR][4];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = sum[m][i] = 0.0f;
    const int chunks = (C + 31) / 32;
    int since = 0;
    for (int c = rank * (kShrinkThreads / 32) + warp; c < chunks; c += nc * (kShrinkThreads / 32)) {
        const int k = c * 32 + q * 8;
        const bool in = k < C;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 b = (in && xr) ? ldg16(xr + k) : zero;
        uint4 lo[MR], hi[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const int r = m * 16 + g;
            lo[m] = (in && r0 + r < R) ? ldg16(wa + static_cast<int64_t>(r) * C + k) : zero;
            hi[m] = (in && r0 + r + 8 < R) ? ldg16(wa + static_cast<int64_t>(r + 8) * C + k) : zero;
        }
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            mma_bf16(acc[m], lo[m].x, hi[m].x, lo[m].y, hi[m].y, b.x, b.y);
            mma_bf16(acc[m], lo[m].z, hi[m].z, lo[m].w, hi[m].w, b.z, b.w);
        }
        if (++since == 8) {  // short chains on the tensor core, joined in FP32
            since = 0;
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[m][i] += acc[m][i];
                    acc[m][i] = 0.0f;
                }
        }
    }
    // element (rank m*16 + g [+8], token 2q [+1]) of the tile
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[warp][(m * 16 + g + (i >> 1) * 8) * kShrinkTokens + 2 * q + (i & 1)] = sum[m][i] + acc[m][i];
    __syncthreads();
    constexpr int kElems = MR * 16 * kShrinkTokens;
    for (int e = threadIdx.x; e < kElems; e += kShrinkThreads) {
        float s = 0.0f;
#pragma unroll
        for (int wi = 0; wi < kShrinkThreads / 32; ++wi) s += red[wi][e];
        part[e] = s;
    }
    cluster.sync();
    const float f = scales ? __ldg(scales + tile.a) : 1.0f;
    for (int e = rank * kShrinkThreads + threadIdx.x; e < kElems; e += nc * kShrinkThreads) {
        float s = 0.0f;
        for (int b = 0; b < nc; ++b) s += cluster.map_shared_rank(part, b)[e];
        const int tk = e % kShrinkTokens, r = r0 + e / kShrinkTokens;
        if (tk < tile.count && r < R) v[static_cast<int64_t>(tile.p0 + tk) * R + r] = f * s;
    }
    cluster.sync();  // the peers have read this block's part
}

// ------------------------------------------------------------------ expand
//
// out[t, c] = base[t, c] + f_a sum_r v[p, r] w[a, r, c].  A warp keeps the
// adapter's ranks of 8 NW columns in registers (the B operand, two rank rows
// interleaved per register) and walks over the tile's tokens, 16 at a time:
// tokens are the rows of the MMA, so that a lane ends up with 2 NW
// consecutive columns of two rows, read and written in 16-byte pieces.  The
// split terms of v wait in shared memory in the order of the A operand.
constexpr int kExpandThreads = 128;

template <int KS, int NW, int BT>
__global__ void __launch_bounds__(kExpandThreads)
    lora_expand_kernel(LoraRows rows, const float* __restrict__ v, int R, const uint16_t* __restrict__ w, int C,
                       int cblocks, const float* __restrict__ scales, const float* base, int64_t ld_base, float* out,
                       int64_t ld_out, uint16_t* __restrict__ out_bf16)
{
    __shared__ __align__(16) uint32_t frag[BT / 16][3][KS][32 * 4];
    __shared__ int s_tok[BT];
    const Tile tile = find_tile<kExpandThreads>(rows, BT, blockIdx.x / cblocks);
    if (tile.a < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int c0 = (static_cast<int>(blockIdx.x % cblocks) * (kExpandThreads / 32) + warp) * 8 * NW;
    // the adapter's slab: ranks 16 s + 4 q + i, columns c0 + NW g + j
    uint32_t b[KS][NW][2];
    {
        const int c = c0 + NW * g;
        const uint16_t* wa = w + static_cast<int64_t>(tile.a) * R * C + c;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint32_t rr[4][NW / 2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * s + 4 * q + i;
                const bool in = r < R && c < C;
                if (NW == 8) {
                    const uint4 u = in ? ldg16(wa + static_cast<int64_t>(r) * C) : make_uint4(0, 0, 0, 0);
                    rr[i][0] = u.x;
                    rr[i][1] = u.y;
                    rr[i][NW / 2 - 2] = u.z;
                    rr[i][NW / 2 - 1] = u.w;
                } else {
                    const uint2 u = in ? __ldg(reinterpret_cast<const uint2*>(wa + static_cast<int64_t>(r) * C))
                                       : make_uint2(0, 0);
                    rr[i][0] = u.x;
                    rr[i][1] = u.y;
                }
            }
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                b[s][j][0] = __byte_perm(rr[0][j / 2], rr[1][j / 2], sel);
                b[s][j][1] = __byte_perm(rr[2][j / 2], rr[3][j / 2], sel);
            }
        }
    }
    // split terms of v, four ranks of one token at a time
    for (int idx = threadIdx.x; idx < BT * KS * 4; idx += kExpandThreads) {
        const int i = idx / (KS * 4), r4 = idx % (KS * 4);
        Split t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = r4 * 4 + u;
            const bool in = i < tile.count && r < R;
            t[u] = split3(in ? __ldg(v + static_cast<int64_t>(tile.p0 + i) * R + r) : 0.0f);
        }
        const int at = (((i & 7) * 4 + (r4 & 3)) << 2) + ((i >> 3) & 1);
        uint32_t* d = &frag[i >> 4][0][r4 >> 2][at];
        d[0] = pack_bf16(t[0].h, t[1].h);
        d[2] = pack_bf16(t[2].h, t[3].h);
        d[KS * 128] = pack_bf16(t[0].m, t[1].m);
        d[KS * 128 + 2] = pack_bf16(t[2].m, t[3].m);
        d[2 * KS * 128] = pack_bf16(t[0].l, t[1].l);
        d[2 * KS * 128 + 2] = pack_bf16(t[2].l, t[3].l);
    }
    for (int i = threadIdx.x; i < BT; i += kExpandThreads) {
        int tok = (i < tile.count) ? __ldg(rows.tokens + tile.p0 + i) : -1;
        s_tok[i] = (tok >= 0 && tok < rows.T) ? tok : -1;
    }
    __syncthreads();
    const float f = scales ? __ldg(scales + tile.a) : 1.0f;
    const int cl = c0 + 2 * NW * q;  // the lane's 2 NW columns
    for (int i0 = 0; i0 < tile.count; i0 += 16) {
        const int tok[2] = {s_tok[i0 + g], s_tok[i0 + 8 + g]};
        float4 old[2][NW / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < NW / 2; ++u)
                old[h][u] = (base && tok[h] >= 0 && cl + 4 * u < C)
                                ? *reinterpret_cast<const float4*>(base + tok[h] * ld_base + cl + 4 * u)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        float acc[NW][4];
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
        for (int sp = 2; sp >= 0; --sp)  // the small terms first
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint4 a = *reinterpret_cast<const uint4*>(&frag[i0 >> 4][sp][s][lane * 4]);
#pragma unroll
                for (int j = 0; j < NW; ++j) mma_bf16(acc[j], a.x, a.y, a.z, a.w, b[s][j][0], b[s][j][1]);
            }
        // acc[j][0], [1]: row g, columns cl + j and cl + NW + j; [2], [3]: row g + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (tok[h] < 0) continue;
            float o[2 * NW];
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                o[j] = acc[j][2 * h];
                o[NW + j] = acc[j][2 * h + 1];
            }
#pragma unroll
            for (int u = 0; u < NW / 2; ++u) {
                if (cl + 4 * u >= C) continue;
                const float4 r = make_float4(fmaf(f, o[4 * u], old[h][u].x), fmaf(f, o[4 * u + 1], old[h][u].y),
                                             fmaf(f, o[4 * u + 2], old[h][u].z), fmaf(f, o[4 * u + 3], old[h][u].w));
                *reinterpret_cast<float4*>(out + tok[h] * ld_out + cl + 4 * u) = r;
                if (out_bf16)
                    *reinterpret_cast<uint2*>(out_bf16 + static_cast<int64_t>(tok[h]) * C + cl + 4 * u) =
                        make_uint2(pack_bf16(r.x, r.y), pack_bf16(r.z, r.w));
            }
        }
    }
}

// ------------------------------------------------------------------- outer
//
// d[a, r, c] = f_a sum_p v[p, r] x[tok, c].  A block holds 16 MR ranks times
// 256 columns of one adapter in registers (a warp 64 columns) and walks over
// the adapter's tokens.  Ranks are the rows of the MMA, tokens its K; two
// token rows of x are interleaved into the B operand as in the expand.  Each
// 16-token product of the three terms starts from zero and is added in FP32,
// so no long sum is left to the tensor core's rounding.
constexpr int kOuterThreads = 128;
constexpr int kOuterTokens = 64;
constexpr int kOuterCols = 256;

template <int MR>
__global__ void __launch_bounds__(kOuterThreads)
    lora_outer_kernel(LoraRows rows, int R, int rblocks, LoraOuter pa, LoraOuter pb, int ablocks)
{
    __shared__ __align__(16) uint32_t frag[kOuterTokens / 16][3][MR][32 * 4];
    __shared__ int s_tok[kOuterTokens];
    const bool first = static_cast<int>(blockIdx.x) < ablocks;
    const LoraOuter& pr = first ? pa : pb;
    const int cblk = first ? blockIdx.x : blockIdx.x - ablocks;
    const int a = blockIdx.y / rblocks;
    const int r0 = (blockIdx.y % rblocks) * 16 * MR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int T = static_cast<int>(rows.T);
    const int p_lo = min(max(__ldg(rows.offsets + a), 0), T);
    const int p_hi = min(max(__ldg(rows.offsets + a + 1), p_lo), T);
    const int C = pr.C;
    const int c0 = cblk * kOuterCols + warp * 64;
    const int c = c0 + 8 * g;
    float sum[MR][8][4];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[m][j][i] = 0.0f;
    for (int p0 = p_lo; p0 < p_hi; p0 += kOuterTokens) {
        const int count = min(kOuterTokens, p_hi - p0);
        __syncthreads();
        for (int i = threadIdx.x; i < kOuterTokens; i += kOuterThreads) {
            const int tok = (i < count) ? __ldg(rows.tokens + p0 + i) : -1;
            s_tok[i] = (tok >= 0 && tok < T) ? tok : -1;
        }
        for (int idx = threadIdx.x; idx < (kOuterTokens / 2) * MR * 16; idx += kOuterThreads) {
            const int r = idx % (MR * 16), i = (idx / (MR * 16)) * 2;
            Split t[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool in = i + u < count && r0 + r < R;
                t[u] = split3(in ? __ldg(pr.v + static_cast<int64_t>(p0 + i + u) * R + r0 + r) : 0.0f);
            }
            // tokens 4 q + 2 h, + 1 of a group; ranks g and g + 8 of a 16-rank tile
            const int at = ((((r & 7) * 4 + ((i & 15) >> 2)) << 2) | (((i >> 1) & 1) << 1) | ((r >> 3) & 1));
            uint32_t* d = &frag[i >> 4][0][r >> 4][at];
            d[0] = pack_bf16(t[0].h, t[1].h);
            d[MR * 128] = pack_bf16(t[0].m, t[1].m);
            d[2 * MR * 128] = pack_bf16(t[0].l, t[1].l);
        }
        __syncthreads();
        for (int i0 = 0; i0 < count; i0 += 16) {
            uint4 xr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = s_tok[i0 + 4 * q + i];
                xr[i] = (tok >= 0 && c < C) ? ldg16(pr.x + tok * pr.ldx + c) : make_uint4(0, 0, 0, 0);
            }
            uint32_t b[8][2];
            const uint32_t(&w0)[4] = reinterpret_cast<const uint32_t(&)[4]>(xr[0]);
            const uint32_t(&w1)[4] = reinterpret_cast<const uint32_t(&)[4]>(xr[1]);
            const uint32_t(&w2)[4] = reinterpret_cast<const uint32_t(&)[4]>(xr[2]);
            const uint32_t(&w3)[4] = reinterpret_cast<const uint32_t(&)[4]>(xr[3]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                b[j][0] = __byte_perm(w0[j / 2], w1[j / 2], sel);
                b[j][1] = __byte_perm(w2[j / 2], w3[j / 2], sel);
            }
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                float t[8][4];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[j][i] = 0.0f;
#pragma unroll
                for (int sp = 2; sp >= 0; --sp) {
                    const uint4 av = *reinterpret_cast<const uint4*>(&frag[i0 >> 4][sp][m][lane * 4]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) mma_bf16(t[j], av.x, av.y, av.z, av.w, b[j][0], b[j][1]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[m][j][i] += t[j][i];
            }
        }
    }
    // sum[m][j][0], [1]: rank g, columns c0 + 16 q + j and + 8 + j; [2], [3]: rank g + 8
    const float f = pr.scales ? __ldg(pr.scales + a) : 1.0f;
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + m * 16 + g + 8 * h;
            if (r >= R) continue;
            float* d = pr.d + (static_cast<int64_t>(a) * R + r) * C;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int cc = c0 + 16 * q + 8 * half;
                if (cc >= C) continue;
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    *reinterpret_cast<float4*>(d + cc + 4 * u) =
                        make_float4(f * sum[m][4 * u][2 * h + half], f * sum[m][4 * u + 1][2 * h + half],
                                    f * sum[m][4 * u + 2][2 * h + half], f * sum[m][4 * u + 3][2 * h + half]);
            }
        }
}

template <int MR>
cudaError_t shrink(const LoraRows& rows, const uint16_t* x, int64_t ldx, int C, const uint16_t* w, int R,
                   const float* scales, float* v, int sm_count, cudaStream_t s)
{
    const int rblocks = (R + 16 * MR - 1) / (16 * MR);
    const int64_t units = max_tiles(rows.T, rows.n, kShrinkTokens) * rblocks;
    // as many blocks per cluster (they share the columns) as it takes to give
    // every SM two blocks, while each warp keeps two column steps
    int nc = 1;
    while (nc < 8 && units * nc < 2 * sm_count && (C + 31) / 32 >= nc * 2 * (kShrinkThreads / 32) * 2) nc *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * nc));
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nc;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_shrink_kernel<MR>, rows, x, ldx, C, w, R, rblocks, scales, v);
}

template <int KS, int NW, int BT>
cudaError_t expand(const LoraRows& rows, const float* v, int R, const uint16_t* w, int C, const float* scales,
                   const float* base, int64_t ld_base, float* out, int64_t ld_out, uint16_t* out_bf16, cudaStream_t s)
{
    const int cols = kExpandThreads / 32 * 8 * NW;
    const int cblocks = (C + cols - 1) / cols;
    const int64_t grid = max_tiles(rows.T, rows.n, BT) * cblocks;
    lora_expand_kernel<KS, NW, BT><<<static_cast<unsigned>(grid), kExpandThreads, 0, s>>>(
        rows, v, R, w, C, cblocks, scales, base, ld_base, out, ld_out, out_bf16);
    return cudaGetLastError();
}

template <int MR>
cudaError_t outer(const LoraRows& rows, int R, const LoraOuter& a, const LoraOuter& b, cudaStream_t s)
{
    const int rblocks = (R + 16 * MR - 1) / (16 * MR);
    const int ab = (a.C + kOuterCols - 1) / kOuterCols, bb = (b.C + kOuterCols - 1) / kOuterCols;
    const dim3 grid(static_cast<unsigned>(ab + bb), static_cast<unsigned>(rows.n * rblocks));
    lora_outer_kernel<MR><<<grid, kOuterThreads, 0, s>>>(rows, R, rblocks, a, b, ab);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraRows& rows, const uint16_t* x, int64_t ldx, int C, const uint16_t* w, int R,
                               const float* scales, float* v, cudaStream_t s)
{
    DeviceInfo di;
    if (!device_info(&di)) return cudaErrorUnknown;
    if (R <= 16) return shrink<1>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
    if (R <= 32) return shrink<2>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
    return shrink<4>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
}

cudaError_t launch_lora_expand(const LoraRows& rows, const float* v, int R, const uint16_t* w, int C,
                               const float* scales, const float* base, int64_t ld_base, float* out, int64_t ld_out,
                               uint16_t* out_bf16, cudaStream_t s)
{
    if (R <= 16) return expand<1, 8, 64>(rows, v, R, w, C, scales, base, ld_base, out, ld_out, out_bf16, s);
    if (R <= 32) return expand<2, 8, 64>(rows, v, R, w, C, scales, base, ld_base, out, ld_out, out_bf16, s);
    if (R <= 64) return expand<4, 8, 64>(rows, v, R, w, C, scales, base, ld_base, out, ld_out, out_bf16, s);
    return expand<8, 4, 32>(rows, v, R, w, C, scales, base, ld_base, out, ld_out, out_bf16, s);
}

cudaError_t launch_lora_outer(const LoraRows& rows, int R, const LoraOuter& a, const LoraOuter& b, cudaStream_t s)
{
    if (R <= 16) return outer<1>(rows, R, a, b, s);
    if (R <= 32) return outer<2>(rows, R, a, b, s);
    return outer<4>(rows, R, a, b, s);
}

}  // namespace fp8moe
