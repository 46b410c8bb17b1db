// experts.cu -- products grouped by expert with ragged row counts
// (md_expert_gemm, md_expert_wgrad, md_expert_gated).
//
// The rows are the conventional, expert-grouped rows of md_dispatch_layout:
// expert e owns rows [offsets[e], offsets[e] + counts[e]).
//   gemm   y[r, n]     = sum_k x[r, k] w[e, n, k]    (or w[e, k, n])
//   gated  a[r, f]     = silu(g) u,  g = w[e, f] . x[r],  u = w[e, F + f] . x[r]
//   wgrad  dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]
//
// One persistent kernel body.  The tensor cores' M axis (128 rows per CTA) holds weight
// rows n, their N axis holds the ragged rows r (for the weight gradient: the
// columns k).  The N extent of an MMA is free in steps of 16, so an expert's
// ragged remainder costs what it holds: an expert's c rows are split into
// ceil(c / BN) equal tiles, and each tile's MMAs are issued with its own N.
// Putting the rows on the M axis instead would pay for 128 rows per remainder,
// which at a few rows per expert (decoding) is nearly all of the work.
//
// Warps 0-3 drain accumulators (TMEM -> registers -> shared -> global), warp 4
// issues the TMA loads, warp 5 the MMAs; accumulators are double-buffered in
// TMEM, so a tile's epilogue runs under the next tile's products.  Every wait
// is bounded: the role whose wait runs out raises the CTA's abort flag and
// MD_ERR_TIMEOUT, all roles leave their loops, copies and MMAs in flight are
// awaited (bounded again), TMEM is freed, and the kernel returns.
#include "tcgen05.cuh"

namespace {

enum { kNK, kKN, kGated, kWgrad };

constexpr int kTileM = 128;  // weight rows per CTA
constexpr int kTileK = 64;   // 128 bytes of bf16: one swizzled line
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kABytes = kTileM * kTileK * 2;
constexpr int kBlock = 32;   // columns that share a scale of the 8-bit checkpoint
constexpr long long kPolls = 1ll << 22;
constexpr long long kDrainPolls = 1ll << 20;

struct Args {
    const int32_t *offsets, *counts;
    int64_t rows;
    int E;
    int n;        // weight rows per expert that tiles cover (gemm: N, gated: F, wgrad: N)
    int k;        // extent of the contraction (gemm, gated: K); wgrad: columns of dw
    int pitch;    // columns of y, or of a
    void *y;      // gemm: bf16 [rows, N]; gated: bf16 [rows, F]
    uint8_t *codes, *scales;  // gated: checkpoint or NULL
    int out_bf16, accumulate; // wgrad
    int32_t *status;
    long long polls;
};

template <int MODE, int CG, int BN>
struct Plan {
    static constexpr bool kWg = MODE == kWgrad;
    static constexpr int kGran = 16 * CG;             // step of an MMA's N
    static constexpr int kBRows = BN / CG;            // N-side lines per CTA
    static constexpr int kBBytes = kBRows * kTileK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kBox = BN >= 256 ? 64 : 16;  // x rows per TMA box
    static constexpr int kStaging = MODE == kNK || MODE == kKN ? 2 * 32 * 256 : 2 * 32 * 512;
    static constexpr int kFit = (212 * 1024 - kStaging) / kStageBytes;  // leaves 12 KB for 1024 experts' table
    static constexpr int kStages = kFit > 10 ? 10 : kFit;
    static constexpr int kCols = 2 * BN < 32 ? 32 : 2 * BN;  // TMEM columns: two accumulators
    static constexpr int kMWidth = MODE == kGated ? 64 : kTileM;  // output columns per CTA
    static size_t smem(int E) { return 1024 + (size_t)kStages * kStageBytes + kStaging + 12 * (size_t)E + 16; }
};

struct Bars {
    uint64_t full[10], empty[10], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int abort;
    int tiles;  // ragged tiles of all experts
};

// Bounded wait of one thread; on run-out raises the CTA's abort flag.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, Bars *b, const Args &a)
{
    if (md::mbar_try_wait(bar, parity)) return true;
    volatile int *ab = &b->abort;
    for (long long i = 1; i < a.polls; ++i) {
        if (*ab) return false;
        if (md::mbar_try_wait(bar, parity)) return true;
    }
    *ab = 1;
    md::report(a.status, MD_ERR_TIMEOUT);
    return false;
}

// The same for a whole warp: lane 0 waits, all lanes get its answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Bars *b, const Args &a)
{
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = wait_for(bar, parity, b, a);
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Whether all of the epilogue's warps say yes (they share barriers, so they
// leave together).
__device__ __forceinline__ bool all_warps(bool ok)
{
    int r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.and.pred q, 2, %2, p;\n"
                 " selp.s32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((int)ok), "n"(kEpiWarps * 32)
                 : "memory");
    return r != 0;
}

struct Tile {
    int e, m0;       // expert, first weight row of the CTA (pair: of its half)
    int64_t r0;      // gemm: first x row; wgrad: first row of the expert
    int count;       // gemm: rows of the tile; wgrad: rows of the expert
    int c0;          // wgrad: first dw column
    int n;           // MMA N
};

// A place in the ring of stages: the stage and the parity of its turn.
template <int STAGES>
struct Turn {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++s == STAGES) {
            s = 0;
            parity ^= 1u;
        }
    }
};

// experts' starts, counts and the running number of tiles, in shared memory
struct Table {
    int *off, *cnt, *pre;
};

template <int MODE, int CG, int BN>
__device__ __forceinline__ Tile tile_at(int t, const Table &tab, const Args &a, int mt, int rank)
{
    using P = Plan<MODE, CG, BN>;
    Tile q;
    if (P::kWg) {
        const int ct = (a.k + BN - 1) / BN;
        const int per = mt * ct;
        q.e = t / per;
        const int i = t - q.e * per;
        const int ci = i / mt;
        q.m0 = ((i - ci * mt) * CG + rank) * kTileM;
        q.c0 = ci * BN;
        q.r0 = tab.off[q.e];
        q.count = tab.cnt[q.e];
        const int left = a.k - q.c0;
        const int w = left < BN ? left : BN;
        q.n = (w + P::kGran - 1) / P::kGran * P::kGran;
        return q;
    }
    const int rt = t / mt;
    const int mi = t - rt * mt;
    int lo = 0, hi = a.E;  // last expert whose first tile is at or before rt
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.pre[mid] <= rt) lo = mid;
        else hi = mid;
    }
    const int c = tab.cnt[lo], nt = (c + BN - 1) / BN;
    const int each = ((c + nt - 1) / nt + P::kGran - 1) / P::kGran * P::kGran;
    const int at = (rt - tab.pre[lo]) * each;
    q.e = lo;
    q.m0 = (mi * CG + rank) * P::kMWidth;
    q.r0 = (int64_t)tab.off[lo] + at;
    q.count = c - at < each ? c - at : each;
    q.c0 = 0;
    q.n = (q.count + P::kGran - 1) / P::kGran * P::kGran;
    return q;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight columns of one row and one half of the checkpoint.  The four lanes of
// a 32-column block share its scale: the smallest 2^s with amax <= 448 * 2^s.
// 448 = 1.75 * 2^8, so s follows from amax's exponent and whether its fraction
// passes 1.75.  Inf and NaN are left out of amax and stored as NaN.
__device__ __forceinline__ void pack_block(const float (&v)[8], bool valid, bool store, uint8_t *code,
                                           uint8_t *scale, bool owner)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        if (u < 0x7f800000u && valid) m = m > u ? m : u;
    }
    uint32_t o = __shfl_xor_sync(0xffffffffu, m, 1);
    m = m > o ? m : o;
    o = __shfl_xor_sync(0xffffffffu, m, 2);
    m = m > o ? m : o;
    int s = (int)(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    s = s < 0 ? 0 : s;  // biased by 127
    if (!store) return;
    const float inv = __uint_as_float((uint32_t)(254 - s) << 23);  // 2^(127 - s), s <= 247
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = v[4 * h + i];
            q[i] = (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : x * inv;
        }
        w[h] = e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
    }
    *reinterpret_cast<uint2 *>(code) = make_uint2(w[0], w[1]);
    if (owner) *scale = (uint8_t)s;
}

template <int MODE, int CG, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_expert(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
             const __grid_constant__ CUtensorMap map_d, const __grid_constant__ Args a)
{
    using P = Plan<MODE, CG, BN>;
    static_assert(!P::kWg || CG == 1, "the pair's second CTA does not clear its share of a last block");
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(16) Bars bars;
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *staging = base + P::kStages * P::kStageBytes;
    Table tab;
    tab.off = reinterpret_cast<int *>(staging + P::kStaging);
    tab.cnt = tab.off + a.E;
    tab.pre = tab.cnt + a.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 1 ? 0 : (int)md::cluster_rank();
    Bars *b = &bars;

    // ---- setup: barriers, TMEM, the experts' ranges and tile counts
    if (threadIdx.x == 0) {
        for (int i = 0; i < P::kStages; ++i) {
            md::mbar_init(&b->full[i], 1);
            md::mbar_init(&b->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            md::mbar_init(&b->tfull[i], 1);
            md::mbar_init(&b->tempty[i], kEpiWarps * CG);
        }
        md::mbar_init(&b->drain, 1);
        b->abort = 0;
        md::fence_mbar_init();
    }
    if (warp == 4) {
        if (lane == 0) {
            md::prefetch_map(&map_a);
            md::prefetch_map(&map_b);
        }
    }
    if (warp == 5) md::tmem_alloc<CG>(&b->tmem, P::kCols);
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        int o = __ldg(a.offsets + e), c = __ldg(a.counts + e);
        if (c < 0 || (c > 0 && (o < 0 || (int64_t)o + c > a.rows))) {
            md::report(a.status, MD_ERR_DATA);
            c = 0;
        }
        tab.off[e] = c > 0 ? o : 0;
        tab.cnt[e] = c;
    }
    __syncthreads();
    if (!P::kWg && warp == 0) {  // exclusive running sum of the experts' row tiles
        int run = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int own = e < a.E ? (tab.cnt[e] + BN - 1) / BN : 0;
            int v = own;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += o;
            }
            if (e < a.E) tab.pre[e] = run + v - own;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) b->tiles = run;
    }
    md::tmem_fence_before();
    if (CG == 2) md::cluster_sync();
    __syncthreads();
    md::tmem_fence_after();
    const uint32_t tmem = b->tmem;

    const int mt = (a.n + P::kMWidth * CG - 1) / (P::kMWidth * CG);  // tiles along the weight rows
    const int total = P::kWg ? a.E * mt * ((a.k + BN - 1) / BN) : b->tiles * mt;  // the host keeps it below 2^31
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const uint32_t sbase = md::smem_addr(base);

    if (warp == 4) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            Turn<P::kStages> at;
            int used = 0;  // stages loaded at least once
            bool ok = true;
            for (int t = first; ok && t < total; t += step) {
                const Tile q = tile_at<MODE, CG, BN>(t, tab, a, mt, rank);
                const int kb = P::kWg ? (q.count + kTileK - 1) / kTileK : (a.k + kTileK - 1) / kTileK;
                const int half = q.n / CG;  // N-side lines of this CTA
                const int boxes = P::kWg ? (half + 63) / 64 : (half + P::kBox - 1) / P::kBox;
                const uint32_t bytes = (kABytes + boxes * (P::kWg ? 8192 : P::kBox * 128)) * CG;
                const int r0 = (int)q.r0 + (P::kWg ? 0 : rank * half), c0 = q.c0 + rank * half;
                for (int i = 0; i < kb; ++i) {
                    const int s = at.s;
                    if (!wait_for(&b->empty[s], at.parity ^ 1u, b, a)) {
                        ok = false;
                        break;
                    }
                    uint32_t bar = md::smem_addr(&b->full[s]);
                    if (rank == 0) md::mbar_expect_tx(&b->full[s], bytes);
                    if (CG == 2) bar = md::map_rank(bar, 0);
                    const uint32_t sa = sbase + s * P::kStageBytes, sb = sa + kABytes;
                    const int k0 = i * kTileK;
                    if (MODE == kNK) {
                        md::tma_load_3d<CG>(sa, &map_a, k0, q.m0, q.e, bar);
                    } else if (MODE == kGated) {
                        md::tma_load_3d<CG>(sa, &map_a, k0, q.m0, q.e, bar);
                        md::tma_load_3d<CG>(sa + 8192, &map_a, k0, a.n + q.m0, q.e, bar);
                    } else if (MODE == kKN) {
                        md::tma_load_3d<CG>(sa, &map_a, q.m0, k0, q.e, bar);
                        md::tma_load_3d<CG>(sa + 8192, &map_a, q.m0 + 64, k0, q.e, bar);
                    } else {
                        md::tma_load_2d<CG>(sa, &map_a, q.m0, r0 + k0, bar);
                        md::tma_load_2d<CG>(sa + 8192, &map_a, q.m0 + 64, r0 + k0, bar);
                    }
                    for (int j = 0; j < boxes; ++j) {
                        if (P::kWg) md::tma_load_2d<CG>(sb + j * 8192, &map_b, c0 + j * 64, r0 + k0, bar);
                        else md::tma_load_2d<CG>(sb + j * P::kBox * 128, &map_b, k0, r0 + j * P::kBox, bar);
                    }
                    if (used < P::kStages) ++used;
                    at.next();
                }
            }
            // await the copies in flight, whoever gave up: the last load of every stage
            if (rank == 0) {
                for (int j = 0; j < used; ++j) {  // backwards from the last stage loaded
                    at.parity ^= at.s == 0 ? 1u : 0u;
                    at.s = at.s == 0 ? P::kStages - 1 : at.s - 1;
                    md::mbar_wait_bounded(&b->full[at.s], at.parity, kDrainPolls);
                }
            } else if (!ok) {
                for (int j = 0; j < 2000; ++j) __nanosleep(500);
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------ products
        if (rank == 0 && (P::kWg || lane == 0)) {
            constexpr bool kAKMajor = MODE == kNK || MODE == kGated;
            const uint64_t da0 = kAKMajor ? md::operand_desc(sbase, 16, 1024) : md::operand_desc(sbase, 8192, 1024);
            const uint64_t db0 = P::kWg ? md::operand_desc(sbase + kABytes, 8192, 1024)
                                        : md::operand_desc(sbase + kABytes, 16, 1024);
            constexpr int kAStep = (kAKMajor ? 32 : 2048) >> 4, kBStep = (P::kWg ? 2048 : 32) >> 4;
            Turn<P::kStages> at;
            int acc = 0;
            bool ok = true;
            for (int t = first; ok && t < total; t += step) {
                const Tile q = tile_at<MODE, CG, BN>(t, tab, a, mt, rank);
                const int kb = P::kWg ? (q.count + kTileK - 1) / kTileK : (a.k + kTileK - 1) / kTileK;
                if (kb == 0) continue;
                const int buf = acc & 1;
                const uint32_t idesc = md::mma_desc(kTileM * CG, q.n, !kAKMajor, P::kWg);
                const uint32_t d = tmem + buf * BN;
                const uint32_t tparity = (uint32_t)((acc >> 1) & 1) ^ 1u;
                if (P::kWg ? !warp_wait(&b->tempty[buf], tparity, b, a) : !wait_for(&b->tempty[buf], tparity, b, a))
                    break;
                md::tmem_fence_after();
                ++acc;
                for (int i = 0; i < kb; ++i) {
                    const int s = at.s;
                    int steps = kTileK / 16;
                    if (P::kWg) {
                        if (!warp_wait(&b->full[s], at.parity, b, a)) {
                            ok = false;
                            break;
                        }
                        // the last block reaches into the next expert's rows: rows past the end
                        // are cleared on both sides (zero times a stray NaN or Inf is not zero)
                        const int v = q.count - i * kTileK;
                        if (v < kTileK) {
                            steps = (v + 15) / 16;
                            const int boxes = 2 + (q.n / CG + 63) / 64;
                            const int lines = steps * 16 - v, n16 = lines * 8 * boxes;
                            for (int z = lane; z < n16; z += 32) {
                                const int box = z / (lines * 8), w = z - box * (lines * 8);
                                *reinterpret_cast<uint4 *>(base + s * P::kStageBytes + box * 8192 + (v + (w >> 3)) * 128 +
                                                           (w & 7) * 16) = make_uint4(0, 0, 0, 0);
                            }
                            md::fence_async_shared();
                            __syncwarp();
                        }
                    } else if (!wait_for(&b->full[s], at.parity, b, a)) {
                        ok = false;
                        break;
                    }
                    md::tmem_fence_after();
                    if (lane == 0) {
                        const uint64_t da = da0 + (uint32_t)(s * (P::kStageBytes >> 4));
                        const uint64_t db = db0 + (uint32_t)(s * (P::kStageBytes >> 4));
#pragma unroll
                        for (int j = 0; j < kTileK / 16; ++j)
                            if (!P::kWg || j < steps)
                                md::mma_bf16<CG>(d, da + j * kAStep, db + j * kBStep, idesc, i > 0 || j > 0);
                        md::mma_commit<CG>(&b->empty[s]);
                        if (i == kb - 1) md::mma_commit<CG>(&b->tfull[buf]);
                    }
                    if (P::kWg) __syncwarp();
                    at.next();
                }
            }
            if (lane == 0) {  // await the MMAs in flight, whoever gave up
                md::mma_commit<CG>(&b->drain);
                md::mbar_wait_bounded(&b->drain, 0, kDrainPolls);
            }
        }
    } else {
        // ------------------------------------------------ results
        int acc = 0, chunk = 0;
        const uint32_t quarter = (uint32_t)(warp * 32) << 16;
        for (int t = first; t < total; t += step) {
            const Tile q = tile_at<MODE, CG, BN>(t, tab, a, mt, rank);
            const bool zero = P::kWg && q.count == 0;
            if (zero && a.accumulate) continue;
            const int buf = acc & 1;
            if (!zero) {
                if (!all_warps(warp_wait(&b->tfull[buf], (uint32_t)((acc >> 1) & 1), b, a))) break;
                md::tmem_fence_after();
                ++acc;
            }
            const uint32_t d = tmem + quarter + buf * BN;
            if (P::kWg) {
                // this warp's 32 rows of dw, 128 bytes of columns at a time
                const int wide = a.out_bf16 ? 64 : 32;
                const int left = a.k - q.c0, cols = left < BN ? left : BN;
                const int n0 = q.m0 + warp * 32;
                for (int c = 0; c < cols; c += wide, ++chunk) {
                    uint32_t v[32], w[32];
                    if (!zero) {
                        md::tmem_ld32(v, d + c);
                        if (a.out_bf16) md::tmem_ld32(w, d + c + 32);
                        md::tmem_ld_wait();
                        if (a.out_bf16) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                v[i] = md::pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                                w[i] = md::pack_bf16x2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[16 + i] = w[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0;
                    }
                    unsigned char *st = staging + warp * 8192 + (chunk & 1) * 4096;
                    if (lane == 0) md::bulk_wait_read<1>();  // the store that read this buffer
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // the map's 128-byte swizzle
                        *reinterpret_cast<uint4 *>(st + lane * 128 + ((i ^ (lane & 7)) * 16)) =
                            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    md::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (n0 < a.n) {
                            if (a.accumulate) md::tma_add_3d(&map_d, md::smem_addr(st), q.c0 + c, n0, q.e);
                            else md::tma_store_3d(&map_d, md::smem_addr(st), q.c0 + c, n0, q.e);
                        }
                        md::bulk_commit();
                    }
                }
            } else {
                for (int c = 0; c < q.count; c += 32, ++chunk) {
                    uint32_t v[32];
                    md::tmem_ld32(v, d + c);
                    md::tmem_ld_wait();
                    const int live = q.count - c < 32 ? q.count - c : 32;
                    if (MODE != kGated) {
                        // lane = weight row: lines of 32 x rows by 128 weight rows
                        __nv_bfloat16 *st = reinterpret_cast<__nv_bfloat16 *>(staging + (chunk & 1) * 8192);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            st[i * kTileM + threadIdx.x] = __float2bfloat16_rn(__uint_as_float(v[i]));
                        md::named_barrier(1, kEpiWarps * 32);
                        const uint4 *src = reinterpret_cast<const uint4 *>(st);
                        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y);
                        const int n0 = q.m0 + (threadIdx.x & 15) * 8;
                        if (n0 < a.n)
                            for (int i = threadIdx.x >> 4; i < live; i += 8)
                                *reinterpret_cast<uint4 *>(y + (q.r0 + c + i) * a.pitch + n0) =
                                    src[i * 16 + (threadIdx.x & 15)];
                    } else {
                        // lanes 0-63 of the tile hold g, 64-127 hold u of the same columns
                        float *st = reinterpret_cast<float *>(staging + (chunk & 1) * 16384);
#pragma unroll
                        for (int i = 0; i < 32; ++i) st[i * kTileM + threadIdx.x] = __uint_as_float(v[i]);
                        md::named_barrier(1, kEpiWarps * 32);
                        const int j = threadIdx.x & 7, f0 = q.m0 + j * 8;
                        const bool valid = f0 < a.n;
                        for (int i0 = warp * 4; i0 < live; i0 += 16) {  // four rows to a warp
                            const bool in = i0 + (lane >> 3) < live;
                            const int ii = in ? i0 + (lane >> 3) : i0;
                            float g[8], u[8];
                            *reinterpret_cast<float4 *>(g) = *reinterpret_cast<const float4 *>(st + ii * kTileM + j * 8);
                            *reinterpret_cast<float4 *>(g + 4) = *reinterpret_cast<const float4 *>(st + ii * kTileM + j * 8 + 4);
                            *reinterpret_cast<float4 *>(u) = *reinterpret_cast<const float4 *>(st + ii * kTileM + 64 + j * 8);
                            *reinterpret_cast<float4 *>(u + 4) = *reinterpret_cast<const float4 *>(st + ii * kTileM + 64 + j * 8 + 4);
                            const int64_t r = q.r0 + c + ii;
                            if (a.codes) {
                                const int blocks = (a.n + kBlock - 1) / kBlock;
                                uint8_t *cr = a.codes + r * 2 * a.n + f0, *sr = a.scales + r * 2 * blocks + f0 / kBlock;
                                pack_block(g, valid, valid && in, cr, sr, (j & 3) == 0);
                                pack_block(u, valid, valid && in, cr + a.n, sr + blocks, (j & 3) == 0);
                            }
                            if (valid && in) {
                                uint32_t w[4];
#pragma unroll
                                for (int p = 0; p < 4; ++p) {
                                    const float x0 = g[2 * p] / (1.0f + expf(-g[2 * p])) * u[2 * p];
                                    const float x1 = g[2 * p + 1] / (1.0f + expf(-g[2 * p + 1])) * u[2 * p + 1];
                                    w[p] = md::pack_bf16x2(x0, x1);
                                }
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + r * a.pitch + f0) =
                                    make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                }
            }
            if (!zero) {
                md::tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 1) md::mbar_arrive(&b->tempty[buf]);
                    else md::mbar_arrive_cluster(md::map_rank(md::smem_addr(&b->tempty[buf]), 0));
                }
            }
        }
        if (P::kWg && lane == 0) md::bulk_wait_all();
    }

    // ---- end: nobody leaves while its pair may still read its shared memory
    __syncwarp();
    md::tmem_fence_before();
    __syncthreads();
    if (CG == 2) md::cluster_sync();
    md::tmem_fence_after();
    if (warp == 5) md::tmem_free<CG>(tmem, P::kCols);
}

// ------------------------------------------------------------------ host

// One launch; the caller has made the maps.
template <int MODE, int CG, int BN>
int launch(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md_, Args &a, int64_t tiles,
           cudaStream_t s)
{
    using P = Plan<MODE, CG, BN>;
    if (tiles > (int64_t)1 << 30) return MD_ERR_UNSUPPORTED;
    static std::atomic<uint64_t> setup{0};
    md::once_per_device(setup, [] {
        if (cudaFuncSetAttribute(k_expert<MODE, CG, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)P::smem(MD_MAX_EXPERTS)) != cudaSuccess)
            cudaGetLastError();  // the launch then fails and reports MD_ERR_CUDA
    });
    const int64_t most = md::sm_count() / CG;
    const int64_t grid = (tiles < 1 ? 1 : tiles < most ? tiles : most) * CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::smem(a.E);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_expert<MODE, CG, BN>, ma, mb, md_, a) != cudaSuccess) {
        cudaGetLastError();
        return MD_ERR_CUDA;
    }
    md::count_launches(1);
    return md::launch_status();
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapDataType kF32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;

bool bad_sizes(int64_t rows, int E, int N, int K)
{
    return rows < 0 || E < 1 || N < 8 || K < 8 || N % 8 != 0 || K % 8 != 0;
}

// Row coordinates are 32-bit with room for a tile past the end; a tensor
// map's strides stay below 2^40 bytes.
bool too_large(int64_t rows, int E, int64_t N, int64_t K)
{
    return rows > (int64_t)INT32_MAX - 4096 || E > MD_MAX_EXPERTS || N > (1 << 20) || K > (1 << 20) ||
           N * K > ((int64_t)1 << 37);
}

// gemm (w_layout) and gated share everything but the A operand's boxes.
template <int MODE, int CG, int BN>
int run_rows(const void *x, const void *w, int64_t rows, Args &a, int64_t d0, int64_t d1, cudaStream_t s)
{
    using P = Plan<MODE, CG, BN>;
    CUtensorMap ma, mb;
    if (!md::make_map(&ma, w, kBf16, 2, d0, d1, a.E, 64, MODE == kNK ? kTileM : 64) ||
        !md::make_map(&mb, x, kBf16, 2, a.k, rows, 0, 64, P::kBox))
        return MD_ERR_CUDA;
    const int mt = (a.n + P::kMWidth * CG - 1) / (P::kMWidth * CG);
    const int64_t tiles = (rows / BN + (rows < a.E ? rows : a.E)) * mt;  // at most
    return launch<MODE, CG, BN>(ma, mb, mb, a, tiles, s);
}

// Few rows to an expert: narrow tiles leave shared memory for a deep ring,
// since such a call is bound by reading the weights.  Many: 256-row tiles.
bool few_rows(int64_t rows, int E) { return rows <= (int64_t)48 * E; }

}  // namespace

extern "C" int md_expert_gemm(const void *x, int64_t rows, int K, const void *w, int E, int N, int w_layout,
                              const int32_t *expert_offsets, const int32_t *expert_counts, void *y,
                              int32_t *dev_status, void *stream)
{
    if (bad_sizes(rows, E, N, K) || (w_layout != MD_W_NK && w_layout != MD_W_KN)) return MD_ERR_ARG;
    if (!w || !md::aligned16(w) || !expert_offsets || !expert_counts) return MD_ERR_ARG;
    if (rows > 0 && (!x || !y || !md::aligned16(x) || !md::aligned16(y))) return MD_ERR_ARG;
    if (too_large(rows, E, N, K)) return MD_ERR_UNSUPPORTED;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK || rows == 0) return rc;
    Args a = {};
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.rows = rows;
    a.E = E;
    a.n = N;
    a.k = K;
    a.pitch = N;
    a.y = y;
    a.status = dev_status;
    a.polls = md::hook_poll_limit(kPolls);
    if (w_layout == MD_W_NK)
        return few_rows(rows, E) ? run_rows<kNK, 1, 64>(x, w, rows, a, K, N, s)
                                 : run_rows<kNK, 2, 256>(x, w, rows, a, K, N, s);
    return few_rows(rows, E) ? run_rows<kKN, 1, 64>(x, w, rows, a, N, K, s)
                             : run_rows<kKN, 2, 256>(x, w, rows, a, N, K, s);
}

extern "C" int md_expert_gated(const void *x, int64_t rows, int K, const void *w, int E, int F,
                               const int32_t *expert_offsets, const int32_t *expert_counts, void *act,
                               void *codes, uint8_t *scales, int32_t *dev_status, void *stream)
{
    if (bad_sizes(rows, E, F, K) || (codes == nullptr) != (scales == nullptr)) return MD_ERR_ARG;
    if (!w || !md::aligned16(w) || !expert_offsets || !expert_counts) return MD_ERR_ARG;
    if (rows > 0 && (!x || !act || !md::aligned16(x) || !md::aligned16(act))) return MD_ERR_ARG;
    if (codes && !md::aligned16(codes)) return MD_ERR_ARG;
    if (too_large(rows, E, 2 * (int64_t)F, K)) return MD_ERR_UNSUPPORTED;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK || rows == 0) return rc;
    Args a = {};
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.rows = rows;
    a.E = E;
    a.n = F;
    a.k = K;
    a.pitch = F;
    a.y = act;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales;
    a.status = dev_status;
    a.polls = md::hook_poll_limit(kPolls);
    return few_rows(rows, E) ? run_rows<kGated, 1, 64>(x, w, rows, a, K, 2 * (int64_t)F, s)
                             : run_rows<kGated, 2, 256>(x, w, rows, a, K, 2 * (int64_t)F, s);
}

extern "C" int md_expert_wgrad(const void *dy, const void *x, int64_t rows, int E, int N, int K,
                               const int32_t *expert_offsets, const int32_t *expert_counts, int out_type,
                               int accumulate, void *dw, int32_t *dev_status, void *stream)
{
    if (bad_sizes(rows, E, N, K) || (out_type != MD_F32 && out_type != MD_BF16)) return MD_ERR_ARG;
    if (accumulate && out_type != MD_F32) return MD_ERR_ARG;
    if (!dw || !md::aligned16(dw) || !expert_offsets || !expert_counts) return MD_ERR_ARG;
    if (rows > 0 && (!dy || !x || !md::aligned16(dy) || !md::aligned16(x))) return MD_ERR_ARG;
    if (too_large(rows, E, N, K)) return MD_ERR_UNSUPPORTED;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK) return rc;
    const int size = out_type == MD_F32 ? 4 : 2;
    if (rows == 0) {
        if (accumulate) return MD_OK;
        md::count_memsets(1);
        return cudaMemsetAsync(dw, 0, (size_t)E * N * K * size, s) == cudaSuccess ? MD_OK : MD_ERR_CUDA;
    }
    Args a = {};
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.rows = rows;
    a.E = E;
    a.n = N;
    a.k = K;
    a.out_bf16 = out_type == MD_BF16;
    a.accumulate = accumulate != 0;
    a.status = dev_status;
    a.polls = md::hook_poll_limit(kPolls);
    CUtensorMap ma, mb, mo;
    if (!md::make_map(&ma, dy, kBf16, 2, N, rows, 0, 64, 64) || !md::make_map(&mb, x, kBf16, 2, K, rows, 0, 64, 64) ||
        !md::make_map(&mo, dw, a.out_bf16 ? kBf16 : kF32, size, K, N, E, 128 / size, 32))
        return MD_ERR_CUDA;
    const int64_t tiles = (int64_t)E * ((N + kTileM - 1) / kTileM) * ((K + 255) / 256);
    return launch<kWgrad, 1, 256>(ma, mb, mo, a, tiles, s);
}
