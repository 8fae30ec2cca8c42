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
#include "sm100.cuh"

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

// a = h + m + l in BF16 terms, two neighbours at a time; h alone where a is
// not finite or rounds to infinity, so that no Inf - Inf makes a NaN of it.
__device__ __forceinline__ void split3_pair(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l)
{
    h = pack_bf16(a, b);
    const float ha = __uint_as_float(h << 16), hb = __uint_as_float(h & 0xFFFF0000u);
    float ra = fabsf(ha) <= 3.4028234e38f ? a - ha : 0.0f;
    float rb = fabsf(hb) <= 3.4028234e38f ? b - hb : 0.0f;
    m = pack_bf16(ra, rb);
    ra -= __uint_as_float(m << 16);
    rb -= __uint_as_float(m & 0xFFFF0000u);
    l = pack_bf16(ra, rb);
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// 16 bytes from global to shared memory without registers; zeros if !in
// (then nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Programmatic launch: a kernel of a call lets the next one start its blocks
// (which load what does not depend on it) and that one waits here until
// everything before it in the stream is complete and visible.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
    allow_next();
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
    const int step = nc * (kShrinkThreads / 32);
    for (int c = rank * (kShrinkThreads / 32) + warp; c < chunks; c += 2 * step) {
        uint4 b[2], lo[2][MR], hi[2][MR];
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // two column steps' loads in flight
            const int k = (c + u * step) * 32 + q * 8;
            const bool in = k < C;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            b[u] = (in && xr) ? ldg16(xr + k) : zero;
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const int r = m * 16 + g;
                lo[u][m] = (in && r0 + r < R) ? ldg16(wa + static_cast<int64_t>(r) * C + k) : zero;
                hi[u][m] = (in && r0 + r + 8 < R) ? ldg16(wa + static_cast<int64_t>(r + 8) * C + k) : zero;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                mma_bf16(acc[m], lo[u][m].x, hi[u][m].x, lo[u][m].y, hi[u][m].y, b[u].x, b[u].y);
                mma_bf16(acc[m], lo[u][m].z, hi[u][m].z, lo[u][m].w, hi[u][m].w, b[u].z, b[u].w);
            }
        if (++since == 4) {  // short chains on the tensor core, joined in FP32
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

// The same product for adapters with many tokens: 128 tokens times all ranks
// per cluster on tcgen05, the columns dealt to the cluster's blocks 64 at a
// time.  A stage holds the 128 token rows and the RP rank rows of 64 columns
// (128-byte rows, 128-byte swizzle, filled by cp.async, which gathers the
// token rows and zero-fills what is missing); one thread issues the four MMAs
// of a stage.  The accumulator is moved from TMEM to FP32 registers every
// four stages (two TMEM buffers in turn), so a chain on the tensor core stays
// 256 columns long.  At the end the blocks' sums are joined in block order.
constexpr int kTileTokens = 128;
constexpr int kTileThreads = 128;
constexpr int kTileChain = 4;  // stages per accumulation chain
constexpr uint64_t kTileWaitNs = 2000000000ull;

constexpr int tile_stages(int RP) { return RP <= 64 ? 4 : 3; }
constexpr int tile_stage_bytes(int RP) { return (kTileTokens + RP) * 128; }
constexpr int tile_smem(int RP)
{
    return 1024 + tile_stages(RP) * tile_stage_bytes(RP);
}
constexpr uint32_t tile_acc(int RP) { return RP <= 32 ? 32 : RP; }  // TMEM columns of one accumulator
constexpr uint32_t tile_tmem(int RP) { return 2 * tile_acc(RP); }

__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor, kind::f16: D FP32, A and B BF16, dense, M x N;
// a_mn / b_mn: that operand is MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, int a_mn, int b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

template <int RP>
__global__ void __launch_bounds__(kTileThreads)
    lora_shrink_tile_kernel(LoraRows rows, const uint16_t* __restrict__ x, int64_t ldx, int C,
                            const uint16_t* __restrict__ w, int R, const float* __restrict__ scales,
                            float* __restrict__ v)
{
    constexpr int S = tile_stages(RP);
    constexpr int kStage = tile_stage_bytes(RP);
    constexpr int RL = (RP + 31) / 32 * 32;  // accumulator columns read
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t s_bar[S];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_tok[kTileTokens];
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    allow_next();
    const Tile tile = find_tile<kTileThreads>(rows, kTileTokens, blockIdx.x / nc);
    if (tile.a < 0) return;  // the whole cluster
    uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_s = sm100::smem_u32(ring);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) sm100::mbar_init(sm100::smem_u32(&s_bar[i]), 1);
        sm100::fence_barrier_init();
        s_abort = 0;
    }
    if (warp == 0) {
        sm100::tmem_alloc(sm100::smem_u32(&s_tmem), tile_tmem(RP));
        sm100::tmem_relinquish();
    }
    {
        int tok = (tid < tile.count) ? __ldg(rows.tokens + tile.p0 + tid) : -1;
        s_tok[tid] = (tok >= 0 && tok < rows.T) ? tok : -1;
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint16_t* wa = w + static_cast<int64_t>(tile.a) * R * C;
    const int ch = tid & 7, row0 = tid >> 3;
    const int chunks = (C + 63) / 64;
    const int mine = (chunks - rank + nc - 1) / nc;  // this block's: rank, rank + nc, ...
    const uint32_t swz = (static_cast<uint32_t>(ch ^ (row0 & 7)) << 4);
    auto load = [&](int i) {
        if (i < mine) {
            const int k = (rank + i * nc) * 64 + ch * 8;
            const bool in = k < C;
            const uint32_t dst = ring_s + (i % S) * kStage + row0 * 128 + swz;
#pragma unroll
            for (int j = 0; j < kTileTokens / 16; ++j) {
                const int tok = s_tok[row0 + 16 * j];
                const bool ok = in && tok >= 0;
                cp_async16(dst + j * 2048, ok ? x + tok * ldx + k : x, ok);
            }
#pragma unroll
            for (int j = 0; j < RP / 16; ++j) {
                const int r = row0 + 16 * j;
                const bool ok = in && r < R;
                cp_async16(dst + kTileTokens * 128 + j * 2048, ok ? wa + static_cast<int64_t>(r) * C + k : w, ok);
            }
        }
        cp_async_commit();
    };
    float sum[RL];
#pragma unroll
    for (int r = 0; r < RL; ++r) sum[r] = 0.0f;
    bool alive = true;
    auto wait_stage = [&](int i) {  // the MMAs of this block's i-th step are complete
        alive = alive && sm100::mbar_wait_bounded(sm100::smem_u32(&s_bar[i % S]), (i / S) & 1,
                                                  reinterpret_cast<volatile int*>(&s_abort), kTileWaitNs);
    };
    auto promote = [&](int chain) {
        sm100::tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < RL; c0 += 32) {
            uint32_t t[32];
            sm100::tmem_ld32_issue(tmem + (static_cast<uint32_t>(warp) << 21) + (chain & 1) * tile_acc(RP) + c0, t);
            sm100::tmem_ld_wait(t);
#pragma unroll
            for (int u = 0; u < 32; ++u) sum[c0 + u] += __uint_as_float(t[u]);
        }
        sm100::tc_fence_before();
    };
    for (int i = 0; i < S - 1; ++i) load(i);
    constexpr uint32_t idesc = idesc_bf16_f32(kTileTokens, RP, 0, 0);
    for (int i = 0; i < mine; ++i) {
        cp_async_wait<S - 2>();
        sm100::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0 && alive) {
            sm100::tc_fence_after();
            const uint32_t st = ring_s + (i % S) * kStage;
            const uint64_t da = sm100::sw128_kmajor_desc(st), db = sm100::sw128_kmajor_desc(st + kTileTokens * 128);
            const uint32_t d = tmem + ((i / kTileChain) & 1) * tile_acc(RP);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f16_ss(d, da + 2 * kk, db + 2 * kk, idesc, (i % kTileChain != 0 || kk != 0) ? 1u : 0u);
            sm100::mma_commit(sm100::smem_u32(&s_bar[i % S]));
        }
        if (i > 0) {
            wait_stage(i - 1);
            if (i % kTileChain == 0) promote(i / kTileChain - 1);
        }
        load(i + S - 1);
    }
    wait_stage(mine - 1);
    promote((mine - 1) / kTileChain);
    cp_async_wait<0>();
    __syncthreads();
    if (warp == 0) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, tile_tmem(RP));
    }
    // the block's sums, rank-minor; a wait that ran out leaves NaN
    constexpr int kPitch = RP + 1;
    float* const part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int r = 0; r < RP; ++r) part[tid * kPitch + r] = alive ? sum[r] : NAN;
    cluster.sync();
    const float f = scales ? __ldg(scales + tile.a) : 1.0f;
    const int per = kTileTokens / nc;  // this block's token rows
    for (int e = tid; e < per * RP; e += kTileThreads) {
        const int row = rank * per + e / RP, r = e % RP;
        if (row >= tile.count || r >= R) continue;
        float s = 0.0f;
        for (int b = 0; b < nc; ++b) s += cluster.map_shared_rank(part, b)[row * kPitch + r];
        v[static_cast<int64_t>(tile.p0 + row) * R + r] = f * s;
    }
    cluster.sync();  // the peers have read this block's sums
}

// ------------------------------------------------------------------ expand
//
// out[t, c] = base[t, c] + f_a sum_r v[p, r] w[a, r, c].  A warp keeps the
// adapter's ranks of 8 NW columns in registers (the B operand, two rank rows
// interleaved per register) and walks over the tile's tokens, 16 at a time.
// Tokens are the rows of the MMA; column g of its j-th tile is column
// 32 (j / 4) + 4 g + j % 4, so that a lane ends up with 8 consecutive columns
// per row.  The base rows of the next two groups are on their way to a
// per-warp ring in shared memory meanwhile; the sum is formed there in place
// and written out in whole row segments.  v waits in shared memory in FP32 and
// is split as it is read (each warp for itself: the splits hide under the
// MMAs, where preparing them once per block stood in front of them).
constexpr int kExpandThreads = 128;
constexpr int kExpandRing = 3;

template <int NW>
constexpr int expand_pitch()  // bytes of a ring row: 16 past a multiple of 128, so fragment reads do not collide
{
    return 32 * NW + 16;
}
template <int KS>
constexpr int expand_v_pitch()  // bytes of a row of v: 64 past a multiple of 128, as two rows are read at once
{
    return KS == 1 ? 64 : 64 * KS + 64;
}
template <int KS, int NW, int BT>
constexpr int expand_smem()
{
    return BT * expand_v_pitch<KS>() + (kExpandThreads / 32) * kExpandRing * 16 * expand_pitch<NW>();
}

template <int KS, int NW, int BT>
__global__ void __launch_bounds__(kExpandThreads)
    lora_expand_kernel(LoraRows rows, const float* v, int R, const uint16_t* __restrict__ w, int C, int cblocks,
                       const float* __restrict__ scales, const float* base, int64_t ld_base, float* out,
                       int64_t ld_out, uint16_t* __restrict__ out_bf16)
{
    constexpr int P = expand_pitch<NW>();
    constexpr int kPieces = 2 * NW;         // 16-byte pieces of a row segment
    constexpr int kRowsAt = 32 / kPieces;   // rows a warp moves per instruction
    extern __shared__ __align__(16) uint8_t dyn[];
    constexpr int VP = expand_v_pitch<KS>();
    __shared__ int s_tok[BT];
    allow_next();
    const Tile tile = find_tile<kExpandThreads>(rows, BT, blockIdx.x / cblocks);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int c0 = (static_cast<int>(blockIdx.x % cblocks) * (kExpandThreads / 32) + warp) * 8 * NW;
    if (tile.a < 0) return;
    for (int i = threadIdx.x; i < BT; i += kExpandThreads) {
        const int tok = (i < tile.count) ? __ldg(rows.tokens + tile.p0 + i) : -1;
        s_tok[i] = (tok >= 0 && tok < rows.T) ? tok : -1;
    }
    // the adapter's slab: ranks 16 s + 4 q + i, columns c0 + 32 h + 4 g + 0..3
    uint32_t b[KS][NW][2];
    {
        const uint16_t* wa = w + static_cast<int64_t>(tile.a) * R * C + c0 + 4 * g;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < NW / 4; ++h) {
                uint2 rr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * s + 4 * q + i;
                    rr[i] = (r < R && c0 + 32 * h + 4 * g < C)
                                ? __ldg(reinterpret_cast<const uint2*>(wa + static_cast<int64_t>(r) * C + 32 * h))
                                : make_uint2(0, 0);
                }
                b[s][4 * h][0] = __byte_perm(rr[0].x, rr[1].x, 0x5410);
                b[s][4 * h][1] = __byte_perm(rr[2].x, rr[3].x, 0x5410);
                b[s][4 * h + 1][0] = __byte_perm(rr[0].x, rr[1].x, 0x7632);
                b[s][4 * h + 1][1] = __byte_perm(rr[2].x, rr[3].x, 0x7632);
                b[s][4 * h + 2][0] = __byte_perm(rr[0].y, rr[1].y, 0x5410);
                b[s][4 * h + 2][1] = __byte_perm(rr[2].y, rr[3].y, 0x5410);
                b[s][4 * h + 3][0] = __byte_perm(rr[0].y, rr[1].y, 0x7632);
                b[s][4 * h + 3][1] = __byte_perm(rr[2].y, rr[3].y, 0x7632);
            }
    }
    __syncthreads();  // s_tok
    // ring of base row segments: piece `lane % kPieces` of rows lane / kPieces + kRowsAt * i
    uint8_t* const ring = dyn + BT * VP + warp * kExpandRing * 16 * P;
    const uint32_t ring_s = sm100::smem_u32(ring);
    const int pc = lane % kPieces, pr = lane / kPieces;
    const int cp = c0 + 4 * pc;
    auto fetch = [&](int i0) {
        if (base && i0 < tile.count && cp < C) {
            const uint32_t dst = ring_s + ((i0 >> 4) % kExpandRing) * 16 * P + pr * P + pc * 16;
#pragma unroll
            for (int i = 0; i < 16 / kRowsAt; ++i) {
                const int tok = s_tok[i0 + pr + kRowsAt * i];
                if (tok >= 0) cp_async16(dst + kRowsAt * i * P, base + tok * ld_base + cp, true);
            }
        }
        cp_async_commit();
    };
    fetch(0);
    fetch(16);
    wait_previous();  // v
    // v rows, four ranks at a time, zeros past the rank and the tile
    {
        const uint32_t v_s = sm100::smem_u32(dyn);
        const float* vt = v + static_cast<int64_t>(tile.p0) * R;
        for (int idx = threadIdx.x; idx < BT * KS * 4; idx += kExpandThreads) {
            const int i = idx / (KS * 4), r = idx % (KS * 4) * 4;
            const uint32_t dst = v_s + i * VP + r * 4;
            if (R % 4 == 0) {
                const bool in = i < tile.count && r < R;
                cp_async16(dst, in ? vt + static_cast<int64_t>(i) * R + r : v, in);
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool in = i < tile.count && r + u < R;
                    cp_async4(dst + 4 * u, in ? vt + static_cast<int64_t>(i) * R + r + u : v, in);
                }
            }
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    const float f = scales ? __ldg(scales + tile.a) : 1.0f;
    for (int i0 = 0; i0 < tile.count; i0 += 16) {
        fetch(i0 + 32);
        float acc[NW][4];
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
        // rows g and g + 8, ranks 16 s + 4 q + 0..3: A operands of the terms h, m, l
        uint32_t hi[KS][4], mid[KS][4];
        const uint8_t* vr = dyn + (i0 + g) * VP + q * 16;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const float4 v0 = *reinterpret_cast<const float4*>(vr + s * 64);
            const float4 v1 = *reinterpret_cast<const float4*>(vr + 8 * VP + s * 64);
            uint32_t lo[4];
            split3_pair(v0.x, v0.y, hi[s][0], mid[s][0], lo[0]);
            split3_pair(v1.x, v1.y, hi[s][1], mid[s][1], lo[1]);
            split3_pair(v0.z, v0.w, hi[s][2], mid[s][2], lo[2]);
            split3_pair(v1.z, v1.w, hi[s][3], mid[s][3], lo[3]);
#pragma unroll
            for (int j = 0; j < NW; ++j) mma_bf16(acc[j], lo[0], lo[1], lo[2], lo[3], b[s][j][0], b[s][j][1]);
        }
        // the small terms first
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < NW; ++j)
                mma_bf16(acc[j], mid[s][0], mid[s][1], mid[s][2], mid[s][3], b[s][j][0], b[s][j][1]);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < NW; ++j)
                mma_bf16(acc[j], hi[s][0], hi[s][1], hi[s][2], hi[s][3], b[s][j][0], b[s][j][1]);
        cp_async_wait<2>();
        __syncwarp();
        // acc[4 h + u][0], [1]: row g, columns 32 h + 8 q + u and + 4 + u; [2], [3]: row g + 8
        uint8_t* const slot = ring + ((i0 >> 4) % kExpandRing) * 16 * P;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr)
#pragma unroll
            for (int h = 0; h < NW / 4; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4* at = reinterpret_cast<float4*>(slot + (g + 8 * hr) * P + (32 * h + 8 * q + 4 * e) * 4);
                    const float4 o = base ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                    const int n = 2 * hr + e;
                    *at = make_float4(fmaf(f, acc[4 * h][n], o.x), fmaf(f, acc[4 * h + 1][n], o.y),
                                      fmaf(f, acc[4 * h + 2][n], o.z), fmaf(f, acc[4 * h + 3][n], o.w));
                }
        __syncwarp();
        if (cp < C) {
#pragma unroll
            for (int i = 0; i < 16 / kRowsAt; ++i) {
                const int tok = s_tok[i0 + pr + kRowsAt * i];
                if (tok < 0) continue;
                const float4 r = *reinterpret_cast<const float4*>(slot + (pr + kRowsAt * i) * P + pc * 16);
                *reinterpret_cast<float4*>(out + tok * ld_out + cp) = r;
                if (out_bf16)
                    *reinterpret_cast<uint2*>(out_bf16 + static_cast<int64_t>(tok) * C + cp) =
                        make_uint2(pack_bf16(r.x, r.y), pack_bf16(r.z, r.w));
            }
        }
        __syncwarp();  // the slot is free for the fetch of the next round
    }
}

// ------------------------------------------------------------------- outer
//
// d[a, r, c] = f_a sum_p v[p, r] x[tok, c], 64 ranks times 256 columns per
// cluster on tcgen05; tokens are the K of the product, dealt in equal runs to
// the cluster's blocks.  Both operands lie in shared memory token by token,
// 64 values (128 bytes, 128-byte swizzle) per token and panel, so they are
// MN-major: x comes in by cp.async (gathered rows), the three terms of v are
// written by the threads, which split them on the way.  The three products
// share the accumulator; it is moved to FP32 registers every kOuterChain
// stages, so no long sum is left to the tensor core's rounding.  Two blocks
// per SM cover each other's waits.  The blocks' sums are joined in block
// order.
constexpr int kOuterThreads = 128;
constexpr int kOuterRanks = 64;
constexpr int kOuterCols = 256;
constexpr int kOuterTokens = 32;   // per stage
constexpr int kOuterStages = 3;
constexpr int kOuterChain = 8;
constexpr int kOuterPanel = kOuterTokens * 128;
constexpr int kOuterStageBytes = (kOuterCols / 64 + 3) * kOuterPanel;  // four panels of x, three of v
constexpr int kOuterPitch = kOuterCols + 4;                            // floats per rank row of the block's sums
constexpr int kOuterSmem = 1024 + kOuterStages * kOuterStageBytes;
static_assert(kOuterRanks * kOuterPitch * 4 <= kOuterStages * kOuterStageBytes, "the sums reuse the ring");

// Shared-memory matrix descriptor of an MN-major operand in the 128-byte
// swizzle: panels of 64 MN values (128-byte rows, one per K index), 8 K rows
// per 1024-byte atom (stride offset), panels `panel` bytes apart (leading
// offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t panel)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(panel >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__global__ void __launch_bounds__(kOuterThreads)
    lora_outer_kernel(LoraRows rows, int R, int rblocks, LoraOuter pa, LoraOuter pb, int ablocks)
{
    constexpr int S = kOuterStages;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t s_bar[S];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int blk = static_cast<int>(blockIdx.x) / nc;
    const bool first = blk < ablocks;
    const float* const pv = first ? pa.v : pb.v;
    const uint16_t* const px = first ? pa.x : pb.x;
    const int64_t ldx = first ? pa.ldx : pb.ldx;
    const int C = first ? pa.C : pb.C;
    const int c0 = (first ? blk : blk - ablocks) * kOuterCols;
    const int a = blockIdx.y / rblocks;
    const int r0 = (blockIdx.y % rblocks) * kOuterRanks;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_s = sm100::smem_u32(ring);
    if (tid == 0) {
        for (int i = 0; i < S; ++i) sm100::mbar_init(sm100::smem_u32(&s_bar[i]), 1);
        sm100::fence_barrier_init();
        s_abort = 0;
    }
    if (warp == 0) {
        sm100::tmem_alloc(sm100::smem_u32(&s_tmem), kOuterCols);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = s_tmem;
    // this block's run of the adapter's tokens, in whole stages
    const int T = static_cast<int>(rows.T);
    const int lo = min(max(__ldg(rows.offsets + a), 0), T);
    const int hi = min(max(__ldg(rows.offsets + a + 1), lo), T);
    const int stages = (hi - lo + kOuterTokens - 1) / kOuterTokens;
    const int s_lo = static_cast<int>(static_cast<int64_t>(stages) * rank / nc);
    const int mine = static_cast<int>(static_cast<int64_t>(stages) * (rank + 1) / nc) - s_lo;
    const int p0 = lo + s_lo * kOuterTokens;
    // x: piece ch (8 columns) of panel j, token rows row0 and row0 + 16
    const int ch = tid & 7, row0 = tid >> 3;
    const uint32_t swz = static_cast<uint32_t>(ch ^ (row0 & 7)) << 4;
    auto load_x = [&](int i) {
        if (i < mine) {
            const uint32_t dst = ring_s + (i % S) * kOuterStageBytes + row0 * 128 + swz;
#pragma unroll
            for (int h = 0; h < kOuterTokens / 16; ++h) {
                const int p = p0 + i * kOuterTokens + row0 + 16 * h;
                const int tok = p < hi ? __ldg(rows.tokens + p) : -1;
                const bool row = tok >= 0 && tok < T;
                const uint16_t* src = px + (row ? tok * ldx : 0) + c0 + ch * 8;
#pragma unroll
                for (int j = 0; j < kOuterCols / 64; ++j) {
                    const bool ok = row && c0 + j * 64 + ch * 8 < C;
                    cp_async16(dst + j * kOuterPanel + h * 2048, ok ? src + j * 64 : px, ok);
                }
            }
        }
        cp_async_commit();
    };
    // v: token vt, ranks vr .. vr + 15 of the block's 64
    const int vt = tid >> 2, vr = (tid & 3) * 16;
    float va[16];
    auto load_v = [&](int i) {
        const int p = p0 + i * kOuterTokens + vt;
        const bool row = i < mine && p < hi;
        const float* src = pv + static_cast<int64_t>(p) * R + r0 + vr;
        if (R % 4 == 0) {
#pragma unroll
            for (int u = 0; u < 16; u += 4) {
                const float4 t = (row && r0 + vr + u < R) ? __ldcg(reinterpret_cast<const float4*>(src + u))
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                va[u] = t.x;
                va[u + 1] = t.y;
                va[u + 2] = t.z;
                va[u + 3] = t.w;
            }
        } else {
#pragma unroll
            for (int u = 0; u < 16; ++u) va[u] = (row && r0 + vr + u < R) ? __ldcg(src + u) : 0.0f;
        }
    };
    auto store_v = [&](int i) {
        uint8_t* const dst = ring + (i % S) * kOuterStageBytes + (kOuterCols / 64) * kOuterPanel + vt * 128;
#pragma unroll
        for (int u = 0; u < 16; u += 8) {
            uint4 h, m, l;
            split3_pair(va[u], va[u + 1], h.x, m.x, l.x);
            split3_pair(va[u + 2], va[u + 3], h.y, m.y, l.y);
            split3_pair(va[u + 4], va[u + 5], h.z, m.z, l.z);
            split3_pair(va[u + 6], va[u + 7], h.w, m.w, l.w);
            const int at = (((vr + u) >> 3) ^ (vt & 7)) << 4;
            *reinterpret_cast<uint4*>(dst + at) = h;
            *reinterpret_cast<uint4*>(dst + kOuterPanel + at) = m;
            *reinterpret_cast<uint4*>(dst + 2 * kOuterPanel + at) = l;
        }
    };
    float sum[kOuterCols / 64][32];
#pragma unroll
    for (int j = 0; j < kOuterCols / 64; ++j)
#pragma unroll
        for (int u = 0; u < 32; ++u) sum[j][u] = 0.0f;
    bool alive = true;
    auto wait_stage = [&](int i) {  // the MMAs of stage i are complete
        alive = alive && sm100::mbar_wait_bounded(sm100::smem_u32(&s_bar[i % S]), (i / S) & 1,
                                                  reinterpret_cast<volatile int*>(&s_abort), kTileWaitNs);
    };
    auto promote = [&]() {
        sm100::tc_fence_after();
#pragma unroll
        for (int j = 0; j < kOuterCols / 64; ++j) {
            uint32_t t[32];
            sm100::tmem_ld16x256_x8_issue(tmem + (static_cast<uint32_t>(warp) << 21) + j * 64, t);
            sm100::tmem_ld_wait(t);
#pragma unroll
            for (int u = 0; u < 32; ++u) sum[j][u] += __uint_as_float(t[u]);
        }
        sm100::tc_fence_before();
    };
    constexpr uint32_t idesc = idesc_bf16_f32(kOuterRanks, kOuterCols, 1, 1);
    load_x(0);
    load_x(1);
    wait_previous();  // dv
    load_v(0);
    for (int i = 0; i < mine; ++i) {
        store_v(i);
        load_v(i + 1);
        if (i > 0 && i % kOuterChain == 0) {
            wait_stage(i - 1);
            promote();
        }
        cp_async_wait<1>();
        sm100::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0 && alive) {
            sm100::tc_fence_after();
            const uint32_t st = ring_s + (i % S) * kOuterStageBytes;
            const uint64_t dx = sw128_mnmajor_desc(st, kOuterPanel);
            const uint64_t dv = sw128_mnmajor_desc(st + (kOuterCols / 64) * kOuterPanel, kOuterPanel);
#pragma unroll
            for (int kk = 0; kk < kOuterTokens / 16; ++kk)
#pragma unroll
                for (int sp = 2; sp >= 0; --sp)  // 16 token rows are 2048 bytes
                    mma_f16_ss(tmem, dv + (sp * kOuterPanel + kk * 2048) / 16, dx + kk * 2048 / 16, idesc,
                               (i % kOuterChain != 0 || kk != 0 || sp != 2) ? 1u : 0u);
            sm100::mma_commit(sm100::smem_u32(&s_bar[i % S]));
        }
        if (i > 0) wait_stage(i - 1);
        load_x(i + 2);
    }
    if (mine > 0) {
        wait_stage(mine - 1);
        promote();
    }
    cp_async_wait<0>();
    __syncthreads();
    if (warp == 0) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, kOuterCols);
    }
    // the block's sums: lane l holds ranks 16 warp + l / 4 (+ 8), columns
    // 64 j + 8 i + 2 (l % 4) and + 1; a wait that ran out leaves NaN
    float* const part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int j = 0; j < kOuterCols / 64; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float2 t = make_float2(sum[j][4 * i + 2 * h], sum[j][4 * i + 2 * h + 1]);
                if (!alive) t = make_float2(NAN, NAN);
                *reinterpret_cast<float2*>(part + (16 * warp + lane / 4 + 8 * h) * kOuterPitch + 64 * j + 8 * i +
                                           2 * (lane % 4)) = t;
            }
    cluster.sync();
    const float* const scales = first ? pa.scales : pb.scales;
    const float f = scales ? __ldg(scales + a) : 1.0f;
    float* const d = (first ? pa.d : pb.d) + static_cast<int64_t>(a) * R * C;
    const int per = kOuterRanks / nc;  // this block's rank rows
    for (int e = tid; e < per * (kOuterCols / 4); e += kOuterThreads) {
        const int row = rank * per + e / (kOuterCols / 4), c = e % (kOuterCols / 4) * 4;
        if (r0 + row >= R || c0 + c >= C) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = 0; b < nc; ++b) {
            const float4 t = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, b) + row * kOuterPitch + c);
            s.x += t.x;
            s.y += t.y;
            s.z += t.z;
            s.w += t.w;
        }
        *reinterpret_cast<float4*>(d + static_cast<int64_t>(r0 + row) * C + c0 + c) =
            make_float4(f * s.x, f * s.y, f * s.z, f * s.w);
    }
    cluster.sync();  // the peers have read this block's sums
}

// A launch with up to two attributes: cluster size along x (0: none), and
// programmatic launch after the kernel before it.
struct Launch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    Launch(int64_t grid, int threads, size_t smem, cudaStream_t s, int cluster, bool programmatic)
    {
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = at;
        if (cluster) {
            at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            at[cfg.numAttrs].val.clusterDim.x = cluster;
            at[cfg.numAttrs].val.clusterDim.y = 1;
            at[cfg.numAttrs++].val.clusterDim.z = 1;
        }
        if (programmatic) {
            at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
        }
    }
};

// Dynamic shared memory beyond 48 KB is a per-device attribute of a kernel.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes)
{
    return bytes <= 48 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(bytes));
}

// Blocks per cluster (they share the columns): enough to give every SM two
// blocks, while each block keeps `least` column steps.
int cluster_size(int64_t units, int steps, int least, int sm_count)
{
    int nc = 1;
    while (nc < 8 && units * nc < 2 * sm_count && steps >= 2 * nc * least) nc *= 2;
    return nc;
}

template <int MR>
cudaError_t shrink(const LoraRows& rows, const uint16_t* x, int64_t ldx, int C, const uint16_t* w, int R,
                   const float* scales, float* v, int sm_count, cudaStream_t s)
{
    const int rblocks = (R + 16 * MR - 1) / (16 * MR);
    const int64_t units = max_tiles(rows.T, rows.n, kShrinkTokens) * rblocks;
    const int nc = cluster_size(units, (C + 31) / 32, 2 * (kShrinkThreads / 32), sm_count);
    Launch l(units * nc, kShrinkThreads, 0, s, nc, false);
    return cudaLaunchKernelEx(&l.cfg, lora_shrink_kernel<MR>, rows, x, ldx, C, w, R, rblocks, scales, v);
}

template <int RP>
cudaError_t shrink_tile(const LoraRows& rows, const uint16_t* x, int64_t ldx, int C, const uint16_t* w, int R,
                        const float* scales, float* v, int sm_count, cudaStream_t s)
{
    const int64_t units = max_tiles(rows.T, rows.n, kTileTokens);
    const int nc = cluster_size(units, (C + 63) / 64, 4, sm_count);
    cudaError_t err = allow_smem(lora_shrink_tile_kernel<RP>, tile_smem(RP));
    if (err != cudaSuccess) return err;
    Launch l(units * nc, kTileThreads, tile_smem(RP), s, nc, false);
    return cudaLaunchKernelEx(&l.cfg, lora_shrink_tile_kernel<RP>, rows, x, ldx, C, w, R, scales, v);
}

template <int KS, int NW, int BT>
cudaError_t expand(const LoraRows& rows, const float* v, int R, const uint16_t* w, int C, const float* scales,
                   const float* base, int64_t ld_base, float* out, int64_t ld_out, uint16_t* out_bf16, cudaStream_t s)
{
    const int cols = kExpandThreads / 32 * 8 * NW;
    const int cblocks = (C + cols - 1) / cols;
    constexpr int smem = expand_smem<KS, NW, BT>();
    cudaError_t err = allow_smem(lora_expand_kernel<KS, NW, BT>, smem);
    if (err != cudaSuccess) return err;
    Launch l(max_tiles(rows.T, rows.n, BT) * cblocks, kExpandThreads, smem, s, 0, true);
    return cudaLaunchKernelEx(&l.cfg, lora_expand_kernel<KS, NW, BT>, rows, v, R, w, C, cblocks, scales, base, ld_base,
                              out, ld_out, out_bf16);
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraRows& rows, const uint16_t* x, int64_t ldx, int C, const uint16_t* w, int R,
                               const float* scales, float* v, cudaStream_t s)
{
    DeviceInfo di;
    if (!device_info(&di)) return cudaErrorUnknown;
    if (rows.T >= 256 && rows.T >= 16 * static_cast<int64_t>(rows.n)) {
        if (R <= 16) return shrink_tile<16>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
        if (R <= 32) return shrink_tile<32>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
        if (R <= 64) return shrink_tile<64>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
        return shrink_tile<128>(rows, x, ldx, C, w, R, scales, v, di.sm_count, s);
    }
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
    const int rblocks = (R + kOuterRanks - 1) / kOuterRanks;
    const int ab = (a.C + kOuterCols - 1) / kOuterCols, bb = (b.C + kOuterCols - 1) / kOuterCols;
    // blocks per cluster (they share an adapter's tokens): about 128 tokens
    // each, so that an adapter with many tokens does not outlast the others
    int nc = 1;
    while (nc < 8 && rows.T >= 2 * static_cast<int64_t>(nc) * rows.n * 128) nc *= 2;
    cudaError_t err = allow_smem(lora_outer_kernel, kOuterSmem);
    if (err != cudaSuccess) return err;
    Launch l(static_cast<int64_t>(ab + bb) * nc, kOuterThreads, kOuterSmem, s, nc, true);
    l.cfg.gridDim.y = static_cast<unsigned>(rows.n * rblocks);
    return cudaLaunchKernelEx(&l.cfg, lora_outer_kernel, rows, R, rblocks, a, b, ab);
}

}  // namespace fp8moe
