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
// so three products carry both directions; the rank-major B is what makes the
// backward shrink and expand the same as the forward ones.  Few tokens take
// shrink and expand in one launch (lora_small_kernel), many a kernel for each
// (launch_lora has the rule).
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

#include "../../include/fp8moe.h"
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

__device__ __forceinline__ float4 add4(const float4& a, const float4& b)
{
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// 16 bytes from global to shared memory without registers; zeros if !in
// (then nothing is read).  No memory clobber: the waits that make the copies
// visible have it, and with one here each copy's address would wait for the
// copy before it (a stage of the tiled shrink took 0.55 us to issue so).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Arrives on the barrier once this thread's earlier cp.async are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Column group of 16 FP32 accumulators of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 16 TMEM lanes x 32 FP32 columns (.16x256b four times): lane t receives, for
// repetition i, r[4 i], r[4 i + 1] = row t / 4, columns 8 i + 2 (t % 4) and + 1,
// and r[4 i + 2], r[4 i + 3] the same of row t / 4 + 8.
__device__ __forceinline__ void tmem_ld16x256_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Programmatic launch: a kernel of a call lets the next one start its blocks
// (which load what does not depend on it) and that one waits until everything
// before it in the stream is complete and visible.  The expand lets the next
// kernel start only once its own wait is over, so the outer product behind it
// starts with the shrink complete: it needs nothing of the expand, runs beside
// its end, and waits for it before its own.
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
struct Tiles {
    static constexpr int kPer = (1024 + THREADS - 1) / THREADS;  // n <= 1024
    int lo[kPer], cnt[kPer];  // this thread's adapters
    int64_t before;           // tiles of the adapters before them
    int64_t total;            // all tiles
    int per, bt;

    __device__ __forceinline__ void scan(const LoraRows& rows, int bt_)
    {
        __shared__ int s_warp[THREADS / 32];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int T = static_cast<int>(rows.T);
        bt = bt_;
        per = (rows.n + THREADS - 1) / THREADS;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
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
        before = incl - mine;
        total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += s_warp[w];
            total += s_warp[w];
        }
    }

    // The whole block calls it; barriers before and after the result is set.
    __device__ __forceinline__ Tile find(int64_t tile) const
    {
        __shared__ Tile s_tile;
        if (threadIdx.x == 0) s_tile.a = -1;
        __syncthreads();
        int64_t first = before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int nt = (cnt[i] + bt - 1) / bt;
            if (tile >= first && tile < first + nt) {
                const int skip = static_cast<int>(tile - first) * bt;
                s_tile = Tile{static_cast<int>(threadIdx.x * per + i), lo[i] + skip, min(bt, cnt[i] - skip)};
            }
            first += nt;
        }
        __syncthreads();
        return s_tile;
    }
};

template <int THREADS>
__device__ __forceinline__ Tile find_tile(const LoraRows& rows, int bt, int64_t tile)
{
    Tiles<THREADS> t;
    t.scan(rows, bt);
    return t.find(tile);
}

// The three BF16 terms of FP32 rows [T, R], as the gradient product reads
// them: [3][T][R8], R8 = R rounded up to 8, zeros past R.
struct Terms {
    uint16_t* at;  // null: not wanted
    int64_t plane;
    int R8;

    __device__ __forceinline__ void put4(int64_t p, int r, float a, float b, float c, float d) const
    {
        uint2 h, m, l;
        split3_pair(a, b, h.x, m.x, l.x);
        split3_pair(c, d, h.y, m.y, l.y);
        uint16_t* q = at + p * R8 + r;
        *reinterpret_cast<uint2*>(q) = h;
        *reinterpret_cast<uint2*>(q + plane) = m;
        *reinterpret_cast<uint2*>(q + 2 * plane) = l;
    }
};

// Splits rows p_lo .. p_hi - 1 of src [T, R]; threads tid of n.
__device__ __forceinline__ void split_rows(const float* __restrict__ src, int R, const Terms& t, int p_lo, int p_hi,
                                           int tid, int n)
{
    const int quads = t.R8 / 4;
    for (int e = tid; e < (p_hi - p_lo) * quads; e += n) {
        const int64_t p = p_lo + e / quads;
        const int r = e % quads * 4;
        const float* s = src + p * R + r;
        float a[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = r + u < R ? __ldg(s + u) : 0.0f;
        t.put4(p, r, a[0], a[1], a[2], a[3]);
    }
}

// Tiles of bt tokens that T tokens over n adapters can need at most.
int64_t max_tiles(int64_t T, int n, int bt) { return ceil_div64(T, bt) + (T < n ? T : n); }

// ------------------------------------------------- few tokens: one launch
//
// Both products for 8 tokens of one adapter, per cluster.  First v: ranks are
// the rows of the MMA and tokens its columns; both operands go from global
// memory to registers in 16-byte pieces, which the free choice of the order of
// the sum allows: lane q of a quad takes columns 8q .. 8q+7 of a 32-column step
// as its K indices of two MMAs.  The columns are dealt to the warps of all
// blocks of the cluster, whose sums are joined in a fixed order in every
// block, through the cluster's shared memory.  Then the output columns, a
// slice per block and 64 per warp: columns are the rows of the MMA, two rank
// rows interleaved per register, and the three terms of v its columns.  A
// decode batch is bound by bringing the adapters in (64 tokens on 34 adapters
// of rank 64, 5120 to 5120: 24.5 us); a single token by the steps in a row, where
// the wait in the middle is a cluster barrier and not a launch.
constexpr int kSmallThreads = 256;
constexpr int kSmallTokens = 8;
constexpr int kSmallVPitch = 132;  // floats per token of v, off the bank period

// The first product's side and the second's (w2 null: only v is wanted).
struct SmallArgs {
    const uint16_t* x;
    int64_t ldx;
    int C1;
    const uint16_t* w1;
    const float* f1;  // null: 1
    float* v;
    Terms terms;
    const float* u;
    Terms u_terms;
    const uint16_t* w2;
    int C2;
    const float* f2;
    const float* base;
    int64_t ld_base;
    float* out;
    int64_t ld_out;
    uint16_t* out_bf16;
};

template <int MR>
__global__ void __launch_bounds__(kSmallThreads, 2) lora_small_kernel(LoraRows rows, int R, SmallArgs p)
{
    constexpr int kWarps = kSmallThreads / 32;
    __shared__ __align__(16) float red[kWarps][MR * 16 * kSmallTokens];
    __shared__ __align__(16) float part[MOE_MAX_LORA_RANK * kSmallTokens];
    __shared__ __align__(16) float s_v[kSmallTokens * kSmallVPitch];
    __shared__ int s_tok[kSmallTokens];
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const Tile tile = find_tile<kSmallThreads>(rows, kSmallTokens, blockIdx.x / nc);
    if (tile.a < 0) return;  // the whole cluster
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    int tok = (g < tile.count) ? __ldg(rows.tokens + tile.p0 + g) : -1;
    if (tok < 0 || tok >= rows.T) tok = -1;
    if (warp == 0 && q == 0) s_tok[g] = tok;
    // this block's columns of the second product, dealt evenly to its warps
    const int slice = ((p.C2 / 8 + nc - 1) / nc) * 8;
    const int per = ((slice / 8 + kWarps - 1) / kWarps) * 8;
    const int c_lo = min(rank * slice + warp * per, min((rank + 1) * slice, p.C2));
    const int c_hi = min(c_lo + per, min((rank + 1) * slice, p.C2));
    const uint16_t* const w2 = p.w2 ? p.w2 + static_cast<int64_t>(tile.a) * R * p.C2 : nullptr;
    const int chunks = (p.C1 + 31) / 32, step = nc * kWarps;
    for (int r0 = 0; r0 < R; r0 += MR * 16) {
        const uint16_t* const wa = p.w1 + (static_cast<int64_t>(tile.a) * R + r0) * p.C1;
        float acc[MR][4], sum[MR][4];
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = sum[m][i] = 0.0f;
        int since = 0;
        for (int c = rank * kWarps + warp; c < chunks; c += 2 * step) {
            uint4 b[2], lo[2][MR], hi[2][MR];
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // two column steps' loads in flight
                const int k = (c + u * step) * 32 + q * 8;
                const bool in = k < p.C1;
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    const int r = m * 16 + g;
                    lo[u][m] = (in && r0 + r < R) ? ldg16(wa + static_cast<int64_t>(r) * p.C1 + k) : zero;
                    hi[u][m] = (in && r0 + r + 8 < R) ? ldg16(wa + static_cast<int64_t>(r + 8) * p.C1 + k) : zero;
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // (their address comes later than the weights')
                const int k = (c + u * step) * 32 + q * 8;
                b[u] = (k < p.C1 && tok >= 0) ? ldg16(p.x + tok * p.ldx + k) : make_uint4(0, 0, 0, 0);
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
        if (r0 > 0) __syncthreads();
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[warp][(m * 16 + g + (i >> 1) * 8) * kSmallTokens + 2 * q + (i & 1)] = sum[m][i] + acc[m][i];
        __syncthreads();
        for (int e = tid * 4; e < MR * 16 * kSmallTokens; e += kSmallThreads * 4) {
            float4 s = *reinterpret_cast<const float4*>(&red[0][e]);
#pragma unroll
            for (int w = 1; w < kWarps; ++w) s = add4(s, *reinterpret_cast<const float4*>(&red[w][e]));
            *reinterpret_cast<float4*>(part + r0 * kSmallTokens + e) = s;
        }
    }
    // the warp's first weights of the second product are under way during the join
    uint2 ra[MR][4], rb[MR][4];
    auto load_w2 = [&](int c0, int s0) {  // 64 columns, MR steps of 16 ranks
        const int ca = c0 + 4 * g, cb = ca + 32;
#pragma unroll
        for (int s = 0; s < MR; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * (s0 + s) + 4 * q + i;
                const uint16_t* w = w2 + static_cast<int64_t>(r) * p.C2;
                ra[s][i] = (r < R && ca < c_hi) ? __ldg(reinterpret_cast<const uint2*>(w + ca)) : make_uint2(0, 0);
                rb[s][i] = (r < R && cb < c_hi) ? __ldg(reinterpret_cast<const uint2*>(w + cb)) : make_uint2(0, 0);
            }
    };
    if (w2) load_w2(c_lo, 0);
    cluster.sync();
    const float f1 = p.f1 ? __ldg(p.f1 + tile.a) : 1.0f;
    const int ranks = (R + MR * 16 - 1) / (MR * 16) * MR * 16;  // with the zeros past R
    for (int e = tid * 4; e < ranks * kSmallTokens; e += kSmallThreads * 4) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int b = 0; b < nc; ++b)
            s = add4(s, *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, b) + e));
        const int r = e / kSmallTokens;
        const bool in = r < R;
        float* const d = s_v + e % kSmallTokens * kSmallVPitch + r;
        d[0] = in ? f1 * s.x : 0.0f;
        d[kSmallVPitch] = in ? f1 * s.y : 0.0f;
        d[2 * kSmallVPitch] = in ? f1 * s.z : 0.0f;
        d[3 * kSmallVPitch] = in ? f1 * s.w : 0.0f;
    }
    __syncwarp();
    cluster_arrive();  // the peers' sums are read
    __syncthreads();
    // v itself, and its terms, by the blocks in turn
    for (int e = rank * kSmallThreads + tid; e < tile.count * (ranks / 4); e += nc * kSmallThreads) {
        const int tk = e / (ranks / 4), r = e % (ranks / 4) * 4;
        const int64_t at = tile.p0 + tk;
        const float* s = s_v + tk * kSmallVPitch + r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r + i < R) p.v[at * R + r + i] = s[i];
        if (p.terms.at && r < p.terms.R8) p.terms.put4(at, r, s[0], s[1], s[2], s[3]);
    }
    if (p.u_terms.at && rank == 0) split_rows(p.u, R, p.u_terms, tile.p0, tile.p0 + tile.count, tid, kSmallThreads);
    if (w2) {
        const float f2 = p.f2 ? __ldg(p.f2 + tile.a) : 1.0f;
        const int tk[2] = {s_tok[2 * q], s_tok[2 * q + 1]};
        const int steps = ranks / 16;
        for (int c0 = c_lo; c0 < c_hi; c0 += 64) {
            // tile j: row g is column c0 + 4 g + j, row g + 8 column c0 + 32 + 4 g + j
            const int ca = c0 + 4 * g, cb = ca + 32;
            float4 old[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int c = z ? cb : ca;
                    old[t][z] = (p.base && tk[t] >= 0 && c < c_hi)
                                    ? *reinterpret_cast<const float4*>(p.base + tk[t] * p.ld_base + c)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
            for (int s0 = 0; s0 < steps; s0 += MR) {
                if (c0 != c_lo || s0 != 0) load_w2(c0, s0);
#pragma unroll
                for (int s = 0; s < MR; ++s) {
                    const float4 vv =
                        *reinterpret_cast<const float4*>(s_v + g * kSmallVPitch + 16 * (s0 + s) + 4 * q);
                    uint32_t h[2], m[2], l[2];
                    split3_pair(vv.x, vv.y, h[0], m[0], l[0]);
                    split3_pair(vv.z, vv.w, h[1], m[1], l[1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                        const bool up = j >= 2;
                        const uint32_t a0 = __byte_perm(up ? ra[s][0].y : ra[s][0].x, up ? ra[s][1].y : ra[s][1].x, sel);
                        const uint32_t a1 = __byte_perm(up ? rb[s][0].y : rb[s][0].x, up ? rb[s][1].y : rb[s][1].x, sel);
                        const uint32_t a2 = __byte_perm(up ? ra[s][2].y : ra[s][2].x, up ? ra[s][3].y : ra[s][3].x, sel);
                        const uint32_t a3 = __byte_perm(up ? rb[s][2].y : rb[s][2].x, up ? rb[s][3].y : rb[s][3].x, sel);
                        mma_bf16(acc[j], a0, a1, a2, a3, l[0], l[1]);  // the small terms first
                        mma_bf16(acc[j], a0, a1, a2, a3, m[0], m[1]);
                        mma_bf16(acc[j], a0, a1, a2, a3, h[0], h[1]);
                    }
                }
            }
            // acc[j][2 z + t]: column (z ? cb : ca) + j of token 2 q + t
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int c = z ? cb : ca;
                    if (tk[t] < 0 || c >= c_hi) continue;
                    const float4 o = old[t][z];
                    const float4 r = make_float4(fmaf(f2, acc[0][2 * z + t], o.x), fmaf(f2, acc[1][2 * z + t], o.y),
                                                 fmaf(f2, acc[2][2 * z + t], o.z), fmaf(f2, acc[3][2 * z + t], o.w));
                    *reinterpret_cast<float4*>(p.out + tk[t] * p.ld_out + c) = r;
                    if (p.out_bf16)
                        *reinterpret_cast<uint2*>(p.out_bf16 + static_cast<int64_t>(tk[t]) * p.C2 + c) =
                            make_uint2(pack_bf16(r.x, r.y), pack_bf16(r.z, r.w));
                }
        }
    }
    __syncwarp();
    cluster_wait();  // no block ends while a peer reads its sums
}

// ------------------------------------------------------------------ shrink
//
// v[p, r] = f_a sum_c x[tok, c] w[a, r, c] for adapters with many tokens: 128
// tokens times all ranks per cluster on tcgen05, the columns dealt to the
// cluster's blocks 64 at a time.  A stage holds the 128 token rows and the RP rank rows of 64 columns
// (128-byte rows, 128-byte swizzle); four producer warps bring in the token
// rows by cp.async, which gathers them and zero-fills what is missing, one TMA
// box the rank rows (cp.async sustains about 40 bytes per clock and SM, which
// these rows would share), and one thread issues the four MMAs.  Four more
// warps move the accumulator to FP32 registers every four stages (two TMEM
// buffers in turn), so a chain on the tensor core stays 256 columns long (unbroken, 16384 columns come out 2e-6
// off; so, 2.4e-7).  The producers neither fence nor read TMEM: both wait for
// a thread's copies in flight, which kept one stage in flight instead of S
// (16384 x 6144, rank 64: 72 us against 48, 4.3 TB/s of x and A).  The proxy
// fence is the issuer's, behind the barrier that the copies arrive on.  At the
// end the blocks' sums are joined in block order.
constexpr int kTileTokens = 128;
constexpr int kTileThreads = 288;  // four warps of sums, four producers, the issuer
constexpr int kTileChain = 4;      // stages per accumulation chain

constexpr int tile_stages(int RP) { return RP <= 32 ? 5 : RP <= 64 ? 4 : 6; }
constexpr int tile_blocks(int RP) { return RP <= 64 ? 2 : 1; }  // per SM
constexpr int tile_stage_bytes(int RP) { return (kTileTokens + RP) * 128; }
constexpr int tile_smem(int RP) { return 1024 + tile_stages(RP) * tile_stage_bytes(RP); }
constexpr uint32_t tile_acc(int RP) { return RP <= 32 ? 32 : RP; }  // TMEM columns of one accumulator
constexpr uint32_t tile_tmem(int RP) { return 2 * tile_acc(RP); }

// Issued by one elected lane; the whole warp calls them, so that descriptors
// and addresses stay in uniform registers.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_warp(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
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

// K-major operand of 128 token rows in panels of 64 columns: its descriptor
// from column `col` on (a multiple of 16).
__device__ __forceinline__ uint64_t sw128_kmajor_desc_at(uint32_t smem_addr, int col)
{
    return sm100::sw128_kmajor_desc(smem_addr + (col >> 6) * kTileTokens * 128) + (col & 63) * 2 / 16;
}

template <int RP>
__global__ void __launch_bounds__(kTileThreads, tile_blocks(RP))
    lora_shrink_tile_kernel(const __grid_constant__ CUtensorMap wmap, LoraRows rows, const uint16_t* __restrict__ x,
                            int64_t ldx, int C, int R, const float* __restrict__ scales, float* __restrict__ v,
                            Terms terms, const float* __restrict__ u, Terms u_terms, Waits waits)
{
    constexpr int S = tile_stages(RP);
    constexpr int kStage = tile_stage_bytes(RP);
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t s_full[S], s_empty[S], s_ready[2], s_read[2];
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
        for (int i = 0; i < S; ++i) {
            // the copies of x, the box of w
            sm100::mbar_init(sm100::smem_u32(&s_full[i]), 128 + 1 + waits.extra(kHoldShrinkFull));
            sm100::mbar_init(sm100::smem_u32(&s_empty[i]), 1 + waits.extra(kHoldShrinkEmpty));
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(sm100::smem_u32(&s_ready[i]), 1);
            sm100::mbar_init(sm100::smem_u32(&s_read[i]), 128);
        }
        sm100::fence_barrier_init();
        s_abort = 0;
    }
    if (warp == 8) {
        sm100::tmem_alloc(sm100::smem_u32(&s_tmem), tile_tmem(RP));
        sm100::tmem_relinquish();
    }
    if (tid < kTileTokens) {
        const int tok = (tid < tile.count) ? __ldg(rows.tokens + tile.p0 + tid) : -1;
        s_tok[tid] = (tok >= 0 && tok < rows.T) ? tok : -1;
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int chunks = (C + 63) / 64;
    const int mine = (chunks - rank + nc - 1) / nc;  // this block's: rank, rank + nc, ...
    auto wait = [&](uint64_t* b, int phase) {
        return sm100::mbar_wait_bounded(sm100::smem_u32(b), phase & 1, &s_abort, waits.ns);
    };
    // For the roles that go on with collective instructions: a warp goes one way
    // (lanes may see a late arrival and the abort flag in either order).
    auto wait_warp = [&](uint64_t* b, int phase) { return __all_sync(0xFFFFFFFFu, wait(b, phase)) != 0; };
    constexpr int kPitch = RP + 4;
    float* const part = reinterpret_cast<float*>(ring);
    float sum[RP];
    if (warp < 4) {
#pragma unroll
        for (int r = 0; r < RP; ++r) sum[r] = 0.0f;
        const int chains = (mine + kTileChain - 1) / kTileChain;
        for (int c = 0; c < chains; ++c) {
            if (!wait_warp(&s_ready[c & 1], c >> 1)) break;
            sm100::tc_fence_after();
#pragma unroll
            for (int c0 = 0; c0 < RP; c0 += 16) {
                uint32_t t[16];
                tmem_ld16(tmem + (static_cast<uint32_t>(warp) << 21) + (c & 1) * tile_acc(RP) + c0, t);
#pragma unroll
                for (int u = 0; u < 16; ++u) sum[c0 + u] += __uint_as_float(t[u]);
            }
            sm100::tc_fence_before();
            sm100::mbar_arrive(sm100::smem_u32(&s_read[c & 1]));
        }
    } else if (warp < 8) {
        const int ch = tid & 7, row0 = (tid >> 3) & 15;
        const uint32_t swz = static_cast<uint32_t>(ch ^ (row0 & 7)) << 4;
        const uint16_t* xr[kTileTokens / 16];
        uint32_t have = 0;
#pragma unroll
        for (int j = 0; j < kTileTokens / 16; ++j) {
            const int tok = s_tok[row0 + 16 * j];
            xr[j] = x + (tok >= 0 ? tok * ldx : 0);
            have |= (tok >= 0 ? 1u : 0u) << j;
        }
        for (int i = 0; i < mine; ++i) {
            if (i >= S && !wait(&s_empty[i % S], i / S - 1)) break;
            const int k = (rank + i * nc) * 64 + ch * 8;
            const bool in = k < C;
            const int kc = in ? k : 0;
            const uint32_t dst = ring_s + (i % S) * kStage + row0 * 128 + swz;
#pragma unroll
            for (int j = 0; j < kTileTokens / 16; ++j) cp_async16(dst + j * 2048, xr[j] + kc, in && ((have >> j) & 1u));
            cp_async_arrive(sm100::smem_u32(&s_full[i % S]));
            if (tid == 128) {  // rank rows past R come in as zeros
                const uint32_t bar = sm100::smem_u32(&s_full[i % S]);
                sm100::mbar_arrive_expect_tx(bar, RP * 128);
                sm100::tma_load_3d(ring_s + (i % S) * kStage + kTileTokens * 128, &wmap, (rank + i * nc) * 128, 0,
                                   tile.a, bar);
            }
        }
        cp_async_wait_all();
    } else {
        constexpr uint32_t idesc = idesc_bf16_f32(kTileTokens, RP, 0, 0);
        {
            const uint64_t da0 = sm100::sw128_kmajor_desc(ring_s);
            const uint64_t db0 = sm100::sw128_kmajor_desc(ring_s + kTileTokens * 128);
            int st = 0, turn = 0, step = 0, c = 0;
            for (int i = 0; i < mine; ++i) {
                if (step == 0 && c >= 2 && !wait_warp(&s_read[c & 1], (c >> 1) - 1)) break;
                if (!wait_warp(&s_full[st], turn)) break;
                sm100::fence_proxy_async_smem();
                sm100::tc_fence_after();
                const uint64_t da = da0 + st * (kStage / 16), db = db0 + st * (kStage / 16);
                const uint32_t d = tmem + (c & 1) * tile_acc(RP);
                mma_f16_ss(d, da, db, idesc, step != 0 ? 1u : 0u);
                mma_f16_ss(d, da + 2, db + 2, idesc, 1u);
                mma_f16_ss(d, da + 4, db + 4, idesc, 1u);
                mma_f16_ss(d, da + 6, db + 6, idesc, 1u);
                mma_commit_warp(sm100::smem_u32(&s_empty[st]));
                if (++step == kTileChain || i == mine - 1) {
                    mma_commit_warp(sm100::smem_u32(&s_ready[c & 1]));
                    step = 0;
                    ++c;
                }
                if (++st == S) {
                    st = 0;
                    ++turn;
                }
            }
        }
        __syncwarp();
    }
    __syncthreads();  // every chain is read: the MMAs and the ring are done with
    if (s_abort) sm100::settle();
    if (warp == 8) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, tile_tmem(RP));
    }
    // the block's sums, rank-minor; a wait that ran out leaves NaN
    if (warp < 4) {
        const bool bad = s_abort != 0;
#pragma unroll
        for (int r = 0; r < RP; r += 4)
            *reinterpret_cast<float4*>(part + tid * kPitch + r) =
                bad ? make_float4(NAN, NAN, NAN, NAN) : make_float4(sum[r], sum[r + 1], sum[r + 2], sum[r + 3]);
    }
    cluster.sync();
    const float f = scales ? __ldg(scales + tile.a) : 1.0f;
    const int per = kTileTokens / nc;  // this block's token rows
#pragma unroll 4
    for (int e = tid; e < per * (RP / 4); e += kTileThreads) {
        const int row = rank * per + e / (RP / 4), r = e % (RP / 4) * 4;
        if (row >= tile.count || r >= R) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = 0; b < nc; ++b) {
            const float4 t = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, b) + row * kPitch + r);
            s.x += t.x;
            s.y += t.y;
            s.z += t.z;
            s.w += t.w;
        }
        s = make_float4(f * s.x, r + 1 < R ? f * s.y : 0.0f, r + 2 < R ? f * s.z : 0.0f, r + 3 < R ? f * s.w : 0.0f);
        const int64_t p = tile.p0 + row;
        float* const d = v + p * R + r;
        if (R % 4 == 0) {
            *reinterpret_cast<float4*>(d) = s;
        } else {
            d[0] = s.x;
            if (r + 1 < R) d[1] = s.y;
            if (r + 2 < R) d[2] = s.z;
            if (r + 3 < R) d[3] = s.w;
        }
        if (terms.at) {
            terms.put4(p, r, s.x, s.y, s.z, s.w);
            if (r + 4 >= R && r + 4 < terms.R8) terms.put4(p, r + 4, 0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    if (u_terms.at)
        split_rows(u, R, u_terms, tile.p0 + min(rank * per, tile.count), tile.p0 + min((rank + 1) * per, tile.count), tid,
                   kTileThreads);
    cluster.sync();  // the peers have read this block's sums
}

// ------------------------------------------------------------------ expand
//
// out[t, c] = base[t, c] + f_a sum_r v[p, r] w[a, r, c], behind the tiled shrink.
// A warp keeps the
// adapter's ranks of 8 NW columns in registers (the B operand, two rank rows
// interleaved per register) and walks over the tile's tokens, 16 at a time.
// Tokens are the rows of the MMA; column g of its j-th tile is column
// 32 (j / 4) + 4 g + j % 4, so that a lane ends up with 8 consecutive columns
// per row.  The base rows of the next two groups are on their way to a
// per-warp ring in shared memory meanwhile; the sum is formed there in place
// and written out in whole row segments.  The split
// terms of v wait in shared memory in the order of the A operand.
constexpr int kExpandThreads = 128;

template <int NW>
constexpr int expand_pitch()  // bytes of a ring row: 16 past a multiple of 128, so fragment reads do not collide
{
    return 32 * NW + 16;
}
template <int KS, int NW, int BT, int RING>
constexpr int expand_smem()
{
    return (BT / 16) * 3 * KS * 512 + (kExpandThreads / 32) * RING * 16 * expand_pitch<NW>();
}

template <int KS, int NW, int BT, int RING>
__global__ void __launch_bounds__(kExpandThreads)
    lora_expand_kernel(LoraRows rows, const float* v, int R, const uint16_t* __restrict__ w, int C, int cblocks,
                       const float* __restrict__ scales, const float* base, int64_t ld_base, float* out,
                       int64_t ld_out, uint16_t* __restrict__ out_bf16)
{
    constexpr int P = expand_pitch<NW>();
    constexpr int kPieces = 2 * NW;         // 16-byte pieces of a row segment
    constexpr int kRowsAt = 32 / kPieces;   // rows a warp moves per instruction
    extern __shared__ __align__(16) uint8_t dyn[];
    uint32_t* const frag = reinterpret_cast<uint32_t*>(dyn);  // [BT / 16][3][KS][32 * 4]
    __shared__ int s_tok[BT];
    const Tile tile = find_tile<kExpandThreads>(rows, BT, blockIdx.x / cblocks);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int c0 = (static_cast<int>(blockIdx.x % cblocks) * (kExpandThreads / 32) + warp) * 8 * NW;
    if (tile.a < 0) {
        wait_previous();  // so that this kernel never ends before the one it follows
        return;
    }
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
    uint8_t* const ring = dyn + (BT / 16) * 3 * KS * 512 + warp * RING * 16 * P;
    const uint32_t ring_s = sm100::smem_u32(ring);
    const int pc = lane % kPieces, pr = lane / kPieces;
    const int cp = c0 + 4 * pc;
    auto fetch = [&](int i0) {
        if (base && i0 < tile.count && cp < C) {
            const uint32_t dst = ring_s + ((i0 >> 4) % RING) * 16 * P + pr * P + pc * 16;
#pragma unroll
            for (int i = 0; i < 16 / kRowsAt; ++i) {
                const int tok = s_tok[i0 + pr + kRowsAt * i];
                if (tok >= 0) cp_async16(dst + kRowsAt * i * P, base + tok * ld_base + cp, true);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) fetch(16 * i);
    wait_previous();  // v
    allow_next();
    // the terms of v, four ranks of one token at a time, in the order of the A
    // operand: lane 4 g + q holds rows g, g + 8 and ranks 16 s + 4 q + 0..3
    {
        constexpr int kEach = BT * KS * 4 / kExpandThreads;
        float t[kEach][4];  // all loads before the first use
        const float* vt = v + static_cast<int64_t>(tile.p0) * R;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int idx = threadIdx.x + e * kExpandThreads;
            const int i = idx / (KS * 4), r = idx % (KS * 4) * 4;
            if (R % 4 == 0) {
                const float4 u = (i < tile.count && r < R)
                                     ? __ldcg(reinterpret_cast<const float4*>(vt + static_cast<int64_t>(i) * R + r))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                t[e][0] = u.x;
                t[e][1] = u.y;
                t[e][2] = u.z;
                t[e][3] = u.w;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    t[e][u] = (i < tile.count && r + u < R) ? __ldcg(vt + static_cast<int64_t>(i) * R + r + u) : 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int idx = threadIdx.x + e * kExpandThreads;
            const int i = idx / (KS * 4), r4 = idx % (KS * 4);
            uint2 h, m, l;
            split3_pair(t[e][0], t[e][1], h.x, m.x, l.x);
            split3_pair(t[e][2], t[e][3], h.y, m.y, l.y);
            uint32_t* d = frag + ((i >> 4) * 3 * KS + (r4 >> 2)) * 128 + ((i & 7) * 4 + (r4 & 3)) * 4 +
                          ((i >> 3) & 1) * 2;
            *reinterpret_cast<uint2*>(d) = h;
            *reinterpret_cast<uint2*>(d + KS * 128) = m;
            *reinterpret_cast<uint2*>(d + 2 * KS * 128) = l;
        }
    }
    __syncthreads();
    const float f = scales ? __ldg(scales + tile.a) : 1.0f;
    for (int i0 = 0; i0 < tile.count; i0 += 16) {
        fetch(i0 + 16 * (RING - 1));
        float acc[NW][4];
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
        for (int sp = 2; sp >= 0; --sp)  // the small terms first
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint4 a =
                    *reinterpret_cast<const uint4*>(frag + (((i0 >> 4) * 3 + sp) * KS + s) * 128 + lane * 4);
#pragma unroll
                for (int j = 0; j < NW; ++j) mma_bf16(acc[j], a.x, a.z, a.y, a.w, b[s][j][0], b[s][j][1]);
            }
        cp_async_wait<RING - 1>();
        __syncwarp();
        // acc[4 h + u][0], [1]: row g, columns 32 h + 8 q + u and + 4 + u; [2], [3]: row g + 8
        uint8_t* const slot = ring + ((i0 >> 4) % RING) * 16 * P;
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

// The same product for adapters with many tokens, on tcgen05: 128 tokens times
// W columns at a time, one persistent block per SM over an equal run of
// (tile, column block) items.  The split terms of a tile's v rows lie in
// shared memory as one K-major operand [h | m | l] (3 RP wide) and stay for
// all its columns; the adapter's rank rows of W columns are the other,
// MN-major, by TMA, used once per term.  Base rows come in by cp.async; a
// thread of the epilogue owns one row (TMEM lane), forms its sums in place, and
// its warp writes the rows out whole.  (One bulk copy per row and direction
// instead: 206 us against 164 us for 16384 x 6144, rank 64; the copy engine
// takes a request about every 32 clocks, whatever its size.)  Two
// row buffers, each with its own four epilogue warps, take turns; the products
// run up to four blocks ahead of them (four accumulators in TMEM, two slabs),
// so a buffer only waits for its base rows.
constexpr int kWideThreads = 416;  // two epilogue groups of 128, the issuer's warp, four producer warps
constexpr int wide_cols(int RP) { return RP <= 64 ? 128 : 64; }
constexpr int wide_panels(int RP) { return (3 * RP + 63) / 64; }
constexpr int wide_pitch(int RP) { return wide_cols(RP) * 4 + 16; }  // bytes of a base row, off the bank period
constexpr int wide_slab(int RP) { return RP * wide_cols(RP) * 2; }
constexpr int wide_smem(int RP)
{
    return 1024 + wide_panels(RP) * kTileTokens * 128 + 2 * (wide_slab(RP) + kTileTokens * wide_pitch(RP));
}

template <int RP>
__global__ void __launch_bounds__(kWideThreads, 1)
    lora_expand_tile_kernel(const __grid_constant__ CUtensorMap wmap, LoraRows rows, const float* v, int R, int C,
                            const float* __restrict__ scales, const float* base, int64_t ld_base, float* out,
                            int64_t ld_out, uint16_t* __restrict__ out_bf16, Waits waits)
{
    constexpr int W = wide_cols(RP);
    constexpr int NP = wide_panels(RP);
    constexpr int P = wide_pitch(RP);
    constexpr uint32_t kSlab = wide_slab(RP);
    extern __shared__ uint8_t dyn[];
    // barriers: base rows in and buffer free (2 buffers), slab in and used
    // (2 slabs), sums ready and read (4 accumulators)
    __shared__ __align__(8) uint64_t s_bar[16];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_tok[kTileTokens];
    uint8_t* const mem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint8_t* const slabs = mem + NP * kTileTokens * 128;
    uint8_t* const bufs = slabs + 2 * kSlab;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* const abort = &s_abort;
    enum { kBaseIn = 0, kFree = 2, kSlabIn = 4, kSlabUsed = 6, kReady = 8, kRead = 12 };
    auto bar = [&](int kind, int i) { return sm100::smem_u32(&s_bar[kind + i]); };
    auto wait = [&](uint32_t b, uint32_t phase) {
        return sm100::mbar_wait_bounded(b, phase & 1, abort, waits.ns);
    };
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            sm100::mbar_init(bar(kBaseIn, b), 128);
            sm100::mbar_init(bar(kFree, b), 128 + waits.extra(kHoldExpandFree));
            sm100::mbar_init(bar(kSlabIn, b), 1 + waits.extra(kHoldExpandSlab));
            sm100::mbar_init(bar(kSlabUsed, b), 1);
        }
        for (int d = 0; d < 4; ++d) {
            sm100::mbar_init(bar(kReady, d), 1);
            sm100::mbar_init(bar(kRead, d), 128);
        }
        sm100::fence_barrier_init();
        s_abort = 0;
    }
    if (warp == 8) {
        sm100::tmem_alloc(sm100::smem_u32(&s_tmem), 4 * W);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    Tiles<kWideThreads> tiles;
    tiles.scan(rows, kTileTokens);
    sm100::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int nblk = (C + W - 1) / W;
    const int64_t items = tiles.total * nblk;
    const int64_t it_lo = items * blockIdx.x / gridDim.x, it_hi = items * (blockIdx.x + 1) / gridDim.x;
    uint32_t use = 0;      // column blocks this CTA has been through: buffer use & 1, phase use / 2
    bool waited = false;
    bool alive = true;
    for (int64_t it = it_lo; it < it_hi;) {
        const Tile tile = tiles.find(it / nblk);
        const int b_lo = static_cast<int>(it % nblk);
        const int b_hi = static_cast<int>(min(static_cast<int64_t>(nblk), b_lo + (it_hi - it)));
        const int nb = b_hi - b_lo;
        if (tid < kTileTokens) {
            const int tok = (tid < tile.count) ? __ldg(rows.tokens + tile.p0 + tid) : -1;
            s_tok[tid] = (tok >= 0 && tok < rows.T) ? tok : -1;
        }
        __syncthreads();
        if (warp > 8) {
            // producers: a column block's base rows, W / 4 pieces each
            constexpr int kAt = 128 / W;  // rows per warp and instruction
            const int pc = lane % (W / 4) * 4;
            for (int j = 0; j < nb && alive; ++j) {
                const uint32_t u = use + j;
                const int b = u & 1;
                if (u >= 2) alive = wait(bar(kFree, b), (u >> 1) - 1);
                if (!alive) break;  // the rows' barrier stays open, so the sums are not formed either
                const int c = (b_lo + j) * W + pc;
                if (base && c < C) {
#pragma unroll 8
                    for (int r = (warp - 9) * kAt + lane / (W / 4); r < kTileTokens; r += 4 * kAt) {
                        const int tok = s_tok[r];
                        if (tok >= 0)
                            cp_async16(sm100::smem_u32(bufs + (b * kTileTokens + r) * P + pc * 4),
                                       base + tok * ld_base + c, true);
                    }
                }
                cp_async_arrive(bar(kBaseIn, b));
            }
        } else {
            if (warp < 8) {
                // the terms of v: row tid % 128, every other 8 ranks
                if (!waited) {
                    wait_previous();
                    allow_next();
                }
                waited = true;
                const int row = tid & 127;
                const bool in = row < tile.count;
                const float* src = v + static_cast<int64_t>(tile.p0 + row) * R;
                float t[RP / 16][8];  // all loads before the first use
#pragma unroll
                for (int i = 0; i < RP / 16; ++i) {
                    const int r = (tid >> 7) * 8 + 16 * i;
#pragma unroll
                    for (int u = 0; u < 8; u += 4) {
                        if (R % 4 == 0) {
                            const float4 q4 = (in && r + u < R) ? __ldcg(reinterpret_cast<const float4*>(src + r + u))
                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
                            t[i][u] = q4.x;
                            t[i][u + 1] = q4.y;
                            t[i][u + 2] = q4.z;
                            t[i][u + 3] = q4.w;
                        } else {
#pragma unroll
                            for (int w4 = 0; w4 < 4; ++w4)
                                t[i][u + w4] = (in && r + u + w4 < R) ? __ldcg(src + r + u + w4) : 0.0f;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < RP / 16; ++i) {
                    uint4 term[3];
                    split3_pair(t[i][0], t[i][1], term[0].x, term[1].x, term[2].x);
                    split3_pair(t[i][2], t[i][3], term[0].y, term[1].y, term[2].y);
                    split3_pair(t[i][4], t[i][5], term[0].z, term[1].z, term[2].z);
                    split3_pair(t[i][6], t[i][7], term[0].w, term[1].w, term[2].w);
#pragma unroll
                    for (int sp = 0; sp < 3; ++sp) {
                        const int col = sp * RP + (tid >> 7) * 8 + 16 * i;
                        *reinterpret_cast<uint4*>(mem + (col >> 6) * kTileTokens * 128 + row * 128 +
                                                  ((((col & 63) >> 3) ^ (row & 7)) << 4)) = term[sp];
                    }
                }
                sm100::fence_proxy_async_smem();
            }
            auto load_slab = [&](int j) {
                if (lane != 0 || j >= nb) return;
                const int sl = (use + j) & 1;
                sm100::mbar_arrive_expect_tx(bar(kSlabIn, sl), kSlab);
                for (int h = 0; h < W / 64; ++h)
                    sm100::tma_load_3d(sm100::smem_u32(slabs + sl * kSlab + h * RP * 128), &wmap,
                                       ((b_lo + j) * W + 64 * h) * 2, 0, tile.a, bar(kSlabIn, sl));
            };
            if (warp == 8 && alive) {  // the slabs of the tile before are all used
                load_slab(0);
                load_slab(1);
            }
            asm volatile("bar.sync 1, 288;" ::: "memory");  // epilogue groups and issuer: v is in place
            if (warp == 8) {
                constexpr uint32_t idesc = idesc_bf16_f32(kTileTokens, W, 0, 1);
                for (int j = 0; j < nb && alive; ++j) {
                    const uint32_t u = use + j;
                    const int sl = u & 1, d = u & 3;
                    if (u >= 4) alive = wait(bar(kRead, d), (u >> 2) - 1);
                    alive = alive && wait(bar(kSlabIn, sl), u >> 1);
                    alive = __all_sync(0xFFFFFFFFu, alive);
                    if (!alive) break;
                    {
                        sm100::tc_fence_after();
                        const uint64_t dw = sw128_mnmajor_desc(sm100::smem_u32(slabs + sl * kSlab), RP * 128);
#pragma unroll
                        for (int sp = 2; sp >= 0; --sp)  // the small terms first
#pragma unroll
                            for (int k = 0; k < RP / 16; ++k) {
                                const uint64_t dv = sw128_kmajor_desc_at(sm100::smem_u32(mem), sp * RP + k * 16);
                                mma_f16_ss(tmem + d * W, dv, dw + k * 2048 / 16, idesc, (sp != 2 || k != 0) ? 1u : 0u);
                            }
                        mma_commit_warp(bar(kReady, d));
                        mma_commit_warp(bar(kSlabUsed, sl));
                    }
                    __syncwarp();
                    if (j > 0) {  // the slab before is free: fetch the one after this
                        alive = __all_sync(0xFFFFFFFFu, wait(bar(kSlabUsed, sl ^ 1), (u - 1) >> 1));
                        if (alive) load_slab(j + 1);
                    }
                }
                if (alive)
                    alive = __all_sync(0xFFFFFFFFu, wait(bar(kSlabUsed, (use + nb - 1) & 1), (use + nb - 1) >> 1));
            } else {
                const int b = warp >> 2;
                const int row = tid & 127;
                const int tok = s_tok[row];
                const float f = scales ? __ldg(scales + tile.a) : 1.0f;
                uint8_t* const mine = bufs + (b * kTileTokens + row) * P;
                int j = (b ^ use) & 1;
                for (; j < nb; j += 2) {
                    const uint32_t u = use + j;
                    const int c0 = (b_lo + j) * W;
                    const int width = min(W, C - c0);
                    const int d = u & 3;
                    alive = alive && wait(bar(kReady, d), u >> 2);
                    alive = alive && wait(bar(kBaseIn, b), u >> 1);
                    // lanes may see a late arrival and the abort flag in either
                    // order; what follows needs the whole warp
                    alive = __all_sync(0xFFFFFFFFu, alive);
                    if (!alive) break;
                    sm100::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < W; c += 32) {
                        uint32_t t[32];
                        sm100::tmem_ld32_issue(tmem + (static_cast<uint32_t>(warp & 3) << 21) + d * W + c, t);
                        sm100::tmem_ld_wait(t);
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4) {
                            float4* at = reinterpret_cast<float4*>(mine + (c + 4 * q4) * 4);
                            const float4 o = base ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                            *at = make_float4(fmaf(f, __uint_as_float(t[4 * q4]), o.x),
                                              fmaf(f, __uint_as_float(t[4 * q4 + 1]), o.y),
                                              fmaf(f, __uint_as_float(t[4 * q4 + 2]), o.z),
                                              fmaf(f, __uint_as_float(t[4 * q4 + 3]), o.w));
                        }
                    }
                    sm100::tc_fence_before();
                    sm100::mbar_arrive(bar(kRead, d));
                    __syncwarp();
                    constexpr int kAt = 128 / W;  // rows per instruction
                    const int c = lane % (W / 4) * 4;
                    if (c < width) {
#pragma unroll 4
                        for (int r = (warp & 3) * 32 + lane / (W / 4); r < (warp & 3) * 32 + 32; r += kAt) {
                            const int tk = s_tok[r];
                            if (tk < 0) continue;
                            const float4 o = *reinterpret_cast<const float4*>(bufs + (b * kTileTokens + r) * P + c * 4);
                            *reinterpret_cast<float4*>(out + tk * ld_out + c0 + c) = o;
                            if (out_bf16)
                                *reinterpret_cast<uint2*>(out_bf16 + static_cast<int64_t>(tk) * C + c0 + c) =
                                    make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
                        }
                    }
                    sm100::mbar_arrive(bar(kFree, b));
                }
                // after a wait that ran out the rest of the row says so (behind
                // the loop: inside it these stores slow the loop by 4 %)
                for (; j < nb && tok >= 0; j += 2)
                    for (int c = (b_lo + j) * W; c < min((b_lo + j + 1) * W, C); ++c) {
                        out[tok * ld_out + c] = NAN;
                        if (out_bf16) out_bf16[static_cast<int64_t>(tok) * C + c] = 0x7FFF;
                    }
            }
        }
        __syncthreads();  // the tile's v and token list are free
        use += nb;
        it += nb;
    }
    if (!waited) wait_previous();  // this kernel never ends before the one it follows
    if (warp > 8) cp_async_wait_all();
    __syncthreads();
    if (s_abort) sm100::settle();
    if (warp == 8) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, 4 * W);
    }
}

// ------------------------------------------------------------------- outer
//
// d[a, r, c] = f_a sum_p v[p, r] x[tok, c], an item being 64 ranks times 128
// columns of one adapter, on tcgen05 with the tokens as the K of the product.
// Both operands lie in shared memory token by token, 64 values (128 bytes,
// 128-byte swizzle) per token and panel, so they are MN-major: x comes in by
// cp.async (gathered rows), the three terms of v, which the shrink before left
// split, by TMA (by cp.async in an item's last stage, whose rows past the
// adapter's tokens have to be zeros).  One thread issues the MMAs, three per
// 16 tokens into one accumulator; four warps move it to FP32 registers every
// kOuterChain stages (two TMEM buffers in turn), so no long sum is left to the
// tensor core's rounding, and write an item out.  Blocks are persistent, two
// per SM, and the ring runs on from item to item: an item is a few stages,
// shorter than a block's start and end (one item per block: the whole
// gradient of 4096 x 5120, rank 64, 16 adapters took 38 us more).  Items go from the adapter with most
// tokens to the one with fewest, dealt to the blocks there and back, so that
// uneven adapters even out.  With few adapters there are too few items for
// that; then the blocks of a cluster share one item's tokens and join their
// sums in block order.
constexpr int kOuterThreads = 288;
constexpr int kOuterRanks = 64;
constexpr int kOuterCols = 128;
constexpr int kOuterTokens = 32;   // per stage
constexpr int kOuterStages = 5;
constexpr int kOuterChain = 4;
constexpr int kOuterPanel = kOuterTokens * 128;
constexpr int kOuterV = (kOuterCols / 64) * kOuterPanel;  // panels of x, then three of v
constexpr int kOuterStageBytes = kOuterV + 3 * kOuterPanel;
constexpr int kOuterPitch = kOuterCols + 4;  // floats per rank row of the block's sums
constexpr int kOuterSmem = 1024 + kOuterStages * kOuterStageBytes;
static_assert(kOuterRanks * kOuterPitch * 4 <= kOuterStages * kOuterStageBytes, "the sums reuse the ring");

// One of the two products, its terms of v and where they lie.
struct OuterSide {
    Terms v;
    const uint16_t* x;
    int64_t ldx;
    int C;
    const float* scales;
    float* d;
};

// The item's part of the problem: which product, adapter, ranks and columns,
// and this block's run of the adapter's tokens in whole stages.
struct OuterItem {
    bool first;
    int a, r0, c0, C;
    int p0, hi, stages;
};
__device__ __forceinline__ OuterItem outer_item(const LoraRows& rows, const int16_t* order, int64_t item, int ablocks,
                                                int blocks, int rblocks, int Ca, int Cb, int rank, int nc)
{
    OuterItem o;
    const int blk = static_cast<int>(item % blocks);
    const int ar = static_cast<int>(item / blocks);
    o.first = blk < ablocks;
    o.C = o.first ? Ca : Cb;
    o.c0 = (o.first ? blk : blk - ablocks) * kOuterCols;
    o.a = order[ar / rblocks];
    o.r0 = ar % rblocks * kOuterRanks;
    const int T = static_cast<int>(rows.T);
    const int lo = min(max(__ldg(rows.offsets + o.a), 0), T);
    o.hi = min(max(__ldg(rows.offsets + o.a + 1), lo), T);
    const int all = (o.hi - lo + kOuterTokens - 1) / kOuterTokens;
    const int s_lo = static_cast<int>(static_cast<int64_t>(all) * rank / nc);
    o.stages = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) / nc) - s_lo;
    o.p0 = lo + s_lo * kOuterTokens;
    return o;
}

__global__ void __launch_bounds__(kOuterThreads, 2)
    lora_outer_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      LoraRows rows, int R, int rblocks, OuterSide pa, OuterSide pb, int ablocks, int blocks,
                      bool behind_expand, Waits waits)
{
    constexpr int S = kOuterStages;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t s_full[S], s_empty[S], s_ready[2], s_read[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_count[kOuterThreads];
    __shared__ int16_t s_order[1024];  // n <= 1024
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int64_t items = static_cast<int64_t>(blocks) * rblocks * rows.n;
    const int64_t item0 = blockIdx.x / nc, step_items = gridDim.x / nc;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_s = sm100::smem_u32(ring);
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            // the copies of x, the terms of v
            sm100::mbar_init(sm100::smem_u32(&s_full[i]), 128 + 1 + waits.extra(kHoldOuterFull));
            sm100::mbar_init(sm100::smem_u32(&s_empty[i]), 1 + waits.extra(kHoldOuterEmpty));
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(sm100::smem_u32(&s_ready[i]), 1);
            sm100::mbar_init(sm100::smem_u32(&s_read[i]), 128);
        }
        sm100::fence_barrier_init();
        s_abort = 0;
    }
    if (warp == 8) {
        sm100::tmem_alloc(sm100::smem_u32(&s_tmem), 2 * kOuterCols);
        sm100::tmem_relinquish();
    }
    // adapters by falling number of tokens; with more adapters than threads
    // there are items enough to even out in any order
    const bool sorted = nc == 1 && rows.n <= kOuterThreads;
    int count = 0;
    if (sorted && tid < rows.n) {
        count = __ldg(rows.offsets + tid + 1) - __ldg(rows.offsets + tid);
        s_count[tid] = count;
    }
    __syncthreads();
    if (!sorted) {
        for (int i = tid; i < rows.n; i += kOuterThreads) s_order[i] = static_cast<int16_t>(i);
    } else if (tid < rows.n) {
        int at = 0;
        for (int b = 0; b < rows.n; ++b) at += s_count[b] > count || (s_count[b] == count && b < tid);
        s_order[at] = static_cast<int16_t>(tid);
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](uint64_t* b, int phase) {
        return sm100::mbar_wait_bounded(sm100::smem_u32(b), phase & 1, &s_abort, waits.ns);
    };
    // this block's item of a round (there in even rounds, back in odd ones)
    auto item_of = [&](int64_t round) {
        return round * step_items + ((round & 1) ? step_items - 1 - item0 : item0);
    };
    auto item_at = [&](int64_t item) {
        return outer_item(rows, s_order, item, ablocks, blocks, rblocks, pa.C, pb.C, rank, nc);
    };
    float sum[kOuterCols / 32][16];
    if (warp < 4) {
        int c = 0;  // chains so far
        bool ok = true;
        for (int64_t round = 0; round * step_items < items; ++round) {
            if (item_of(round) >= items) continue;
            const OuterItem o = item_at(item_of(round));
#pragma unroll
            for (int j = 0; j < kOuterCols / 32; ++j)
#pragma unroll
                for (int u = 0; u < 16; ++u) sum[j][u] = 0.0f;
            for (int i = 0; i < o.stages; i += kOuterChain, ++c) {
                // a warp goes one way (lanes may see a late arrival and the abort flag in either order)
                ok = __all_sync(0xFFFFFFFFu, ok && wait(&s_ready[c & 1], c >> 1));
                if (!ok) break;
                sm100::tc_fence_after();
#pragma unroll
                for (int j = 0; j < kOuterCols / 32; ++j) {
                    uint32_t t[16];
                    tmem_ld16x256_x4(tmem + (static_cast<uint32_t>(warp) << 21) + (c & 1) * kOuterCols + j * 32, t);
#pragma unroll
                    for (int u = 0; u < 16; ++u) sum[j][u] += __uint_as_float(t[u]);
                }
                sm100::tc_fence_before();
                sm100::mbar_arrive(sm100::smem_u32(&s_read[c & 1]));
            }
            if (nc > 1) break;  // one item per cluster: joined below
            // lane l holds ranks 16 warp + l / 4 (+ 8), columns 32 j + 8 i +
            // 2 (l % 4) and + 1; a wait that ran out leaves NaN
            const float* const scales = o.first ? pa.scales : pb.scales;
            const float f = !ok ? NAN : scales ? __ldg(scales + o.a) : 1.0f;
            float* const d = (o.first ? pa.d : pb.d) + (static_cast<int64_t>(o.a) * R + o.r0) * o.C + o.c0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 16 * warp + lane / 4 + 8 * h;
                if (o.r0 + row >= R) continue;
#pragma unroll
                for (int j = 0; j < kOuterCols / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int col = 32 * j + 8 * i + 2 * (lane % 4);
                        if (o.c0 + col < o.C)
                            *reinterpret_cast<float2*>(d + static_cast<int64_t>(row) * o.C + col) =
                                make_float2(f * sum[j][4 * i + 2 * h], f * sum[j][4 * i + 2 * h + 1]);
                    }
            }
        }
    } else if (warp < 8) {
        const int pt = tid - 128;
        // piece ch (8 values) of the panels, token rows row0 and row0 + 16
        const int ch = pt & 7, row0 = pt >> 3;
        const uint32_t swz = static_cast<uint32_t>(ch ^ (row0 & 7)) << 4;
        const int T = static_cast<int>(rows.T);
        int st = 0, turn = 0;
        bool ok = true, waited = false;
        for (int64_t round = 0; round * step_items < items && ok; ++round) {
            if (item_of(round) >= items) continue;
            const OuterItem o = item_at(item_of(round));
            const uint16_t* const px = o.first ? pa.x : pb.x;
            const int64_t ldx = o.first ? pa.ldx : pb.ldx;
            const Terms pv = o.first ? pa.v : pb.v;
            int next[2];  // token rows of the next stage
            auto load_tokens = [&](int i) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = o.p0 + i * kOuterTokens + row0 + 16 * h;
                    next[h] = at < o.hi ? __ldg(rows.tokens + at) : -1;
                }
            };
            load_tokens(0);
            for (int i = 0; i < o.stages; ++i) {
                const int cur[2] = {next[0], next[1]};
                load_tokens(i + 1);
                ok = ok && (turn == 0 || wait(&s_empty[st], turn - 1));
                if (!ok) break;
                const uint32_t at = ring_s + st * kOuterStageBytes;
                const uint32_t bar = sm100::smem_u32(&s_full[st]);
                const int p = o.p0 + i * kOuterTokens;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool row = cur[h] >= 0 && cur[h] < T;
                    const uint16_t* src = px + (row ? cur[h] * ldx : 0) + o.c0 + ch * 8;
#pragma unroll
                    for (int j = 0; j < kOuterCols / 64; ++j) {
                        const bool in = row && o.c0 + j * 64 + ch * 8 < o.C;
                        cp_async16(at + j * kOuterPanel + (row0 + 16 * h) * 128 + swz, in ? src + j * 64 : px, in);
                    }
                }
                if (!waited && !behind_expand) wait_previous();  // the terms of dv
                waited = true;
                if (p + kOuterTokens <= o.hi) {
                    if (pt == 0) {
                        sm100::mbar_arrive_expect_tx(bar, 3 * kOuterPanel);
                        for (int sp = 0; sp < 3; ++sp)
                            sm100::tma_load_3d(at + kOuterV + sp * kOuterPanel, o.first ? &map_a : &map_b, o.r0 * 2, p,
                                               sp, bar);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int sp = 0; sp < 3; ++sp) {
                            const int row = p + row0 + 16 * h;
                            const bool in = row < o.hi && o.r0 + ch * 8 < pv.R8;
                            cp_async16(
                                at + kOuterV + sp * kOuterPanel + (row0 + 16 * h) * 128 + swz,
                                in ? pv.at + sp * pv.plane + static_cast<int64_t>(row) * pv.R8 + o.r0 + ch * 8 : pv.at,
                                in);
                        }
                    if (pt == 0) sm100::mbar_arrive(bar);
                }
                cp_async_arrive(bar);
                if (++st == S) {
                    st = 0;
                    ++turn;
                }
            }
        }
        cp_async_wait_all();
    } else {
        constexpr uint32_t idesc = idesc_bf16_f32(kOuterRanks, kOuterCols, 1, 1);
        const uint64_t dx0 = sw128_mnmajor_desc(ring_s, kOuterPanel);
        const uint64_t dv0 = sw128_mnmajor_desc(ring_s + kOuterV, kOuterPanel);
        int st = 0, turn = 0, c = 0;
        bool ok = true;
        for (int64_t round = 0; round * step_items < items && ok; ++round) {
            if (item_of(round) >= items) continue;
            const OuterItem o = item_at(item_of(round));
            int step = 0;
            for (int i = 0; i < o.stages; ++i) {
                if (step == 0 && c >= 2) ok = ok && wait(&s_read[c & 1], (c >> 1) - 1);
                ok = __all_sync(0xFFFFFFFFu, ok && wait(&s_full[st], turn));
                if (!ok) break;
                sm100::fence_proxy_async_smem();
                sm100::tc_fence_after();
                const uint64_t dx = dx0 + st * (kOuterStageBytes / 16), dv = dv0 + st * (kOuterStageBytes / 16);
                const uint32_t d = tmem + (c & 1) * kOuterCols;
#pragma unroll
                for (int kk = 0; kk < kOuterTokens / 16; ++kk)
#pragma unroll
                    for (int sp = 2; sp >= 0; --sp)  // 16 token rows are 2048 bytes
                        mma_f16_ss(d, dv + (sp * kOuterPanel + kk * 2048) / 16, dx + kk * 2048 / 16, idesc,
                                   (step != 0 || kk != 0 || sp != 2) ? 1u : 0u);
                mma_commit_warp(sm100::smem_u32(&s_empty[st]));
                if (++step == kOuterChain || i == o.stages - 1) {
                    mma_commit_warp(sm100::smem_u32(&s_ready[c & 1]));
                    step = 0;
                    ++c;
                }
                if (++st == S) {
                    st = 0;
                    ++turn;
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();  // every chain is read: the MMAs and the ring are done with
    if (s_abort) sm100::settle();
    wait_previous();  // (blocks without a stage) never end before the kernel they follow
    if (warp == 8) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, 2 * kOuterCols);
    }
    if (nc == 1) return;
    // a cluster's sums
    const OuterItem o = item_at(item0);
    float* const part = reinterpret_cast<float*>(ring);
    if (warp < 4) {
        const bool bad = s_abort != 0;
#pragma unroll
        for (int j = 0; j < kOuterCols / 32; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2*>(part + (16 * warp + lane / 4 + 8 * h) * kOuterPitch + 32 * j + 8 * i +
                                               2 * (lane % 4)) =
                        bad ? make_float2(NAN, NAN)
                            : make_float2(sum[j][4 * i + 2 * h], sum[j][4 * i + 2 * h + 1]);
    }
    cluster.sync();
    const float* const scales = o.first ? pa.scales : pb.scales;
    const float f = scales ? __ldg(scales + o.a) : 1.0f;
    float* const d = (o.first ? pa.d : pb.d) + (static_cast<int64_t>(o.a) * R + o.r0) * o.C + o.c0;
    const int per = kOuterRanks / nc;  // this block's rank rows
#pragma unroll 4
    for (int e = tid; e < per * (kOuterCols / 4); e += kOuterThreads) {
        const int row = rank * per + e / (kOuterCols / 4), c = e % (kOuterCols / 4) * 4;
        if (o.r0 + row >= R || o.c0 + c >= o.C) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = 0; b < nc; ++b) {
            const float4 t = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, b) + row * kOuterPitch + c);
            s.x += t.x;
            s.y += t.y;
            s.z += t.z;
            s.w += t.w;
        }
        *reinterpret_cast<float4*>(d + static_cast<int64_t>(row) * o.C + c) =
            make_float4(f * s.x, f * s.y, f * s.z, f * s.w);
    }
    cluster.sync();  // the peers have read this block's sums
}

// A launch with up to two attributes: cluster size along x, and
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
        if (cluster > 1) {  // (a cluster of one needs none, and launches faster)
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

// Blocks per cluster (they share the columns): enough to give every SM two
// blocks, while each block keeps `least` column steps.
int cluster_size(int64_t units, int steps, int least, int sm_count)
{
    int nc = 1;
    while (nc < 8 && units * 2 * nc <= 2 * sm_count && steps >= 2 * nc * least) nc *= 2;
    return nc;
}

// Rank rows [n, R, C] BF16 as bytes, boxes of 64 columns times RP ranks of one
// adapter (zeros past R and C).
bool rank_map(CUtensorMap* map, const LoraRows& rows, const uint16_t* w, int R, int C, int RP)
{
    const uint64_t dims[3] = {static_cast<uint64_t>(C) * 2, static_cast<uint64_t>(R), static_cast<uint64_t>(rows.n)};
    const uint64_t strides[2] = {static_cast<uint64_t>(C) * 2, static_cast<uint64_t>(R) * C * 2};
    return make_tmap_u8(map, w, 3, dims, strides, RP);
}

template <int MR>
cudaError_t small(const LoraRows& rows, int R, const SmallArgs& p, int sm_count, cudaStream_t s)
{
    const int64_t units = max_tiles(rows.T, rows.n, kSmallTokens);
    const int nc = cluster_size(units, (p.C1 + 31) / 32, 2 * (kSmallThreads / 32), sm_count);
    Launch l(units * nc, kSmallThreads, 0, s, nc, false);
    return cudaLaunchKernelEx(&l.cfg, lora_small_kernel<MR>, rows, R, p);
}

template <int RP>
cudaError_t shrink_tile(const LoraRows& rows, const uint16_t* x, int64_t ldx, int C, const uint16_t* w, int R,
                        const float* scales, float* v, const Terms& t, const float* u, const Terms& ut, int sm_count,
                        cudaStream_t s)
{
    const int64_t units = max_tiles(rows.T, rows.n, kTileTokens);
    const int nc = cluster_size(units, (C + 63) / 64, 4, sm_count);
    CUtensorMap map;
    if (!rank_map(&map, rows, w, R, C, RP)) return cudaErrorNotSupported;
    cudaError_t err = allow_smem<lora_shrink_tile_kernel<RP>>(tile_smem(RP));
    if (err != cudaSuccess) return err;
    Launch l(units * nc, kTileThreads, tile_smem(RP), s, nc, false);
    return cudaLaunchKernelEx(&l.cfg, lora_shrink_tile_kernel<RP>, map, rows, x, ldx, C, R, scales, v, t, u, ut,
                              waits());
}

template <int RP>
cudaError_t expand_tile(const LoraRows& rows, const float* v, int R, const uint16_t* w, int C, const float* scales,
                        const float* base, int64_t ld_base, float* out, int64_t ld_out, uint16_t* out_bf16,
                        int sm_count, cudaStream_t s)
{
    CUtensorMap map;
    if (!rank_map(&map, rows, w, R, C, RP)) return cudaErrorNotSupported;
    cudaError_t err = allow_smem<lora_expand_tile_kernel<RP>>(wide_smem(RP));
    if (err != cudaSuccess) return err;
    Launch l(sm_count, kWideThreads, wide_smem(RP), s, 0, true);
    return cudaLaunchKernelEx(&l.cfg, lora_expand_tile_kernel<RP>, map, rows, v, R, C, scales, base, ld_base, out,
                              ld_out, out_bf16, waits());
}

template <int KS, int NW, int BT, int RING>
cudaError_t expand(const LoraRows& rows, const float* v, int R, const uint16_t* w, int C, const float* scales,
                   const float* base, int64_t ld_base, float* out, int64_t ld_out, uint16_t* out_bf16, cudaStream_t s)
{
    const int cols = kExpandThreads / 32 * 8 * NW;
    const int cblocks = (C + cols - 1) / cols;
    constexpr int smem = expand_smem<KS, NW, BT, RING>();
    cudaError_t err = allow_smem<lora_expand_kernel<KS, NW, BT, RING>>(smem);
    if (err != cudaSuccess) return err;
    Launch l(max_tiles(rows.T, rows.n, BT) * cblocks, kExpandThreads, smem, s, 0, true);
    return cudaLaunchKernelEx(&l.cfg, lora_expand_kernel<KS, NW, BT, RING>, rows, v, R, w, C, cblocks, scales, base, ld_base,
                              out, ld_out, out_bf16);
}

int round8(int R) { return (R + 7) / 8 * 8; }

Terms terms_at(uint16_t* at, int64_t T, int R) { return Terms{at, T * round8(R), round8(R)}; }

}  // namespace

size_t lora_terms_bytes(int64_t T, int R) { return static_cast<size_t>(T) * round8(R) * 3 * 2; }

cudaError_t launch_lora(const LoraRows& rows, int R, const LoraProduct& p, bool* two_kernels, cudaStream_t s)
{
    *two_kernels = false;
    DeviceInfo di;
    if (!device_info(&di)) return cudaErrorUnknown;
    const Terms t = terms_at(p.v_terms, rows.T, R), ut = terms_at(p.u_terms, rows.T, R);
    const int sms = di.sm_count;
    // Few tokens, or few for each adapter: one launch over tiles of 8 tokens.
    // Measured, this one / the two kernels: 256 tokens on 16 adapters of rank 64,
    // 2048 to 2048, 11 / 15 us; 400 on 4, 5120 to 1536, 14 / 16.5; 512 on one,
    // 5120 to 5120, 23 / 19.5, of rank 32 on six 16 / 18; 4096 on 256 of rank 16,
    // 2048 to 2048, 31.5 / 41.5; 2048 on 200 of rank 64, 5120 to 5120, 128 / 113
    // (two tiles of 8 tokens each read an adapter's ranks).  All with the adapters
    // in use: n counts the resident ones, the host does not know the others
    // (8000 tokens on 4 of 1024 of rank 64 take 256 us here, 101 with n = 4).
    if (rows.T <= (R <= 32 ? 512 : 384) || rows.T < (R <= 32 ? 24 : 8) * static_cast<int64_t>(rows.n)) {
        const SmallArgs a{p.x,    p.ldx, p.C1,   p.w1,      p.f1,  p.v,      t,         p.u, ut, p.w2,
                          p.C2, p.f2,  p.base, p.ld_base, p.out, p.ld_out, p.out_bf16};
        if (R <= 16) return small<1>(rows, R, a, sms, s);
        if (R <= 32) return small<2>(rows, R, a, sms, s);
        return small<4>(rows, R, a, sms, s);
    }
    cudaError_t err;
    if (R <= 16)
        err = shrink_tile<16>(rows, p.x, p.ldx, p.C1, p.w1, R, p.f1, p.v, t, p.u, ut, sms, s);
    else if (R <= 32)
        err = shrink_tile<32>(rows, p.x, p.ldx, p.C1, p.w1, R, p.f1, p.v, t, p.u, ut, sms, s);
    else if (R <= 64)
        err = shrink_tile<64>(rows, p.x, p.ldx, p.C1, p.w1, R, p.f1, p.v, t, p.u, ut, sms, s);
    else
        err = shrink_tile<128>(rows, p.x, p.ldx, p.C1, p.w1, R, p.f1, p.v, t, p.u, ut, sms, s);
    if (err != cudaSuccess || !p.w2) return err;
    *two_kernels = true;
    // Ranks above 32 with many tokens per adapter and rows enough to fill the
    // GPU: the tcgen05 kernel.  Both measured, rank 64, register kernel / this
    // one: 16384 x 6144 220 / 164 us, 4096 x 5120 64 / 48, 2000 x 5120 36 / 35,
    // 2048 x 2048 20 / 23; 4096 x 5120 with 32 tokens per adapter 76 / 102.  Up
    // to rank 32 the register kernel is ahead (16384 x 6144, rank 16: 136 / 153).
    if (R > 32 && rows.T >= 64 * static_cast<int64_t>(rows.n) && rows.T * p.C2 >= (int64_t(1) << 23)) {
        if (R <= 64)
            return expand_tile<64>(rows, p.v, R, p.w2, p.C2, p.f2, p.base, p.ld_base, p.out, p.ld_out, p.out_bf16, sms,
                                   s);
        return expand_tile<128>(rows, p.v, R, p.w2, p.C2, p.f2, p.base, p.ld_base, p.out, p.ld_out, p.out_bf16, sms, s);
    }
    if (R <= 16)
        return expand<1, 8, 64, 3>(rows, p.v, R, p.w2, p.C2, p.f2, p.base, p.ld_base, p.out, p.ld_out, p.out_bf16, s);
    if (R <= 32)
        return expand<2, 8, 64, 3>(rows, p.v, R, p.w2, p.C2, p.f2, p.base, p.ld_base, p.out, p.ld_out, p.out_bf16, s);
    if (R <= 64)
        return expand<4, 8, 64, 2>(rows, p.v, R, p.w2, p.C2, p.f2, p.base, p.ld_base, p.out, p.ld_out, p.out_bf16, s);
    return expand<8, 4, 32, 3>(rows, p.v, R, p.w2, p.C2, p.f2, p.base, p.ld_base, p.out, p.ld_out, p.out_bf16, s);
}

cudaError_t launch_lora_outer(const LoraRows& rows, int R, const LoraOuter& a, const LoraOuter& b, bool behind_expand,
                              cudaStream_t s)
{
    const int rblocks = (R + kOuterRanks - 1) / kOuterRanks;
    const int ab = (a.C + kOuterCols - 1) / kOuterCols, bb = (b.C + kOuterCols - 1) / kOuterCols;
    DeviceInfo di;
    if (!device_info(&di)) return cudaErrorUnknown;
    // Persistent blocks, one item after the other, or clusters of nc blocks that
    // share an item's tokens: whichever takes fewer stages in a row, a cluster's
    // start, end and join counted as ten (a stage takes about 0.6 us).
    const int64_t items = static_cast<int64_t>(ab + bb) * rblocks * rows.n, resident = 2 * di.sm_count;
    const int64_t each = ceil_div64(rows.T, static_cast<int64_t>(kOuterTokens) * rows.n);
    int nc = 1;
    int64_t best = ceil_div64(items, resident) * each + 8;
    for (int n = 2; n <= 8; n *= 2) {
        const int64_t cost = ceil_div64(items * n, resident) * (ceil_div64(each, n) + 10);
        if (cost < best) {
            best = cost;
            nc = n;
        }
    }
    const int64_t grid = nc > 1 ? items * nc : items < resident ? items : resident;
    OuterSide side[2];
    CUtensorMap map[2];
    for (int i = 0; i < 2; ++i) {
        const LoraOuter& o = i == 0 ? a : b;
        side[i] = OuterSide{terms_at(const_cast<uint16_t*>(o.v_terms), rows.T, R), o.x, o.ldx, o.C, o.scales, o.d};
        const uint64_t row = static_cast<uint64_t>(side[i].v.R8) * 2, t1 = rows.T > 0 ? rows.T : 1;
        const uint64_t dims[3] = {row, t1, 3}, strides[2] = {row, t1 * row};
        if (!make_tmap_u8(&map[i], o.v_terms, 3, dims, strides, kOuterTokens)) return cudaErrorNotSupported;
    }
    cudaError_t err = allow_smem<lora_outer_kernel>(kOuterSmem);
    if (err != cudaSuccess) return err;
    // Without tokens no kernel of this call runs before this one, and the one
    // before it in the stream may be the expand of another call, which lets a
    // programmatic launch start while it still writes.
    Launch l(grid, kOuterThreads, kOuterSmem, s, nc, rows.T > 0);
    return cudaLaunchKernelEx(&l.cfg, lora_outer_kernel, map[0], map[1], rows, R, rblocks, side[0], side[1], ab,
                              ab + bb, behind_expand, waits());
}

}  // namespace fp8moe
