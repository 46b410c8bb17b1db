// experts.cu -- products grouped by expert with ragged row counts
// (md_expert_gemm, md_expert_wgrad, md_expert_gated).
//
// The rows are the conventional, expert-grouped rows of md_dispatch_layout:
// expert e owns rows [offsets[e], offsets[e] + counts[e]).
//   gemm   y[r, n]     = sum_k x[r, k] w[e, n, k]    (or w[e, k, n])
//   gated  a[r, f]     = silu(g) u,  g = w[e, f] . x[r],  u = w[e, F + f] . x[r]
//   wgrad  dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]
//
// Two persistent kernels: k_expert_few for calls with few rows to an expert, which
// are bound by reading the weights, and k_expert_wide for many, which are bound by
// the tensor cores and by the path from L2.  In both, the tensor cores' M axis
// (128 rows per CTA) holds weight rows n, their N axis the ragged rows r (weight
// gradient: the columns k).  The N extent of an MMA is free in steps of 16 (32 for
// a pair of CTAs), so an expert's ragged remainder costs what it holds: its c rows
// are split into ceil(c / BN) equal tiles, and each tile's MMAs are issued with
// its own N.  Rows on the M axis would pay for 128 rows per remainder, which at a
// few rows per expert (decoding) is nearly all of the work.
//
// Warps 0-7 drain accumulators (TMEM -> registers -> shared -> global; two
// groups of four, one warp for each quarter of TMEM's lanes); one warp issues
// the MMAs and one or two the TMA loads.  Every wait is bounded: the role whose
// wait runs out raises the CTA's abort flag and MD_ERR_TIMEOUT, all roles leave
// their loops, copies and MMAs in flight are awaited (bounded again), TMEM is
// freed, and the kernel returns.
#include "activation.cuh"
#include "ragged.cuh"
#include "tcgen05.cuh"

namespace {

enum { kNK, kKN, kGated, kWgrad };

constexpr int kTileM = 128;  // weight rows per CTA
constexpr int kTileK = 64;   // 128 bytes of bf16: one swizzled line
constexpr int kEpiWarps = 8;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLoadXWarp = 10;
constexpr int kABytes = kTileM * kTileK * 2;
constexpr int kBlock = 32;   // columns that share a scale of the 8-bit checkpoint
constexpr int kMaxSplit = 4; // CTAs that share a contraction (few rows)
constexpr long long kWaitCycles = 1ll << 32;  // a wait's limit while its CTA loads nothing: some two seconds
constexpr long long kDrainPolls = 1ll << 14;  // each may sleep for some microseconds

// Division by a number fixed at launch: exact for 0 <= x < 2^31 (d >= 1), by the
// round-up reciprocal of Granlund and Montgomery, with x below 2^31 in 33 bits.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t by) : d(by), mul(0), shift(0)
    {
        while (((uint64_t)1 << shift) < d) ++shift;  // ceil(log2 d)
        // mul = ceil(2^(31 + shift) / d) <= 2^32 - 1 for d >= 2; x mul < 2^63
        mul = d == 1 ? 0 : (uint32_t)((((uint64_t)1 << (31 + shift)) + d - 1) / d);
    }
    __host__ __device__ __forceinline__ int div(int x) const
    {
        return d == 1 ? x : (int)(((uint64_t)(uint32_t)x * mul) >> (31 + shift));
    }
};

struct Args {
    const int32_t *offsets, *counts;
    int64_t rows;
    int E;
    int64_t row_tiles;  // gemm, gated: as many as ranges that do not overlap can make
    int n;        // weight rows per expert that tiles cover (gemm: N, gated: F, wgrad: N)
    int k;        // extent of the contraction (gemm, gated: K); wgrad: columns of dw
    int pitch;    // columns of y, or of a
    void *y;      // gemm: bf16 [rows, N]; gated: bf16 [rows, F]; wgrad: dw
    uint8_t *codes, *scales;  // gated: checkpoint or NULL
    int out_bf16, accumulate; // wgrad
    int subs;     // k_expert_wide: M = 256 products to a tile, at most
    FastDiv mt;   // tiles along the weight rows
    FastDiv per;  // wgrad: tiles of an expert
    int split;    // k_expert_few: CTAs (a cluster) that share each tile's contraction; each cluster has one tile
    int32_t *status;
    long long polls;  // a wait's looks at most (test hook)
};

// What the roles of a CTA share, besides their barriers.
struct Shared {
    uint32_t tmem;
    int abort;
    unsigned loads;  // counts up as the loading warp goes on: a sign of life for the other roles' waits
    int tiles;  // ragged row tiles of all experts; -1: more than there can be
    int sums[12];
};

// Bounded wait of a converged warp; all lanes get the same answer.  The first look
// does not sleep, the others may.  A wait may be as long as its tile, so the limit
// is on the time without a load; on run-out the CTA's abort flag is raised.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Shared *sh, const Args &a)
{
    if (__all_sync(0xffffffffu, md::mbar_test_wait(bar, parity))) return true;
    volatile int *ab = &sh->abort;
    volatile unsigned *loads = &sh->loads;
    long long since = clock64();
    unsigned seen = *loads;
    for (long long i = 1; i < a.polls; ++i) {
        if (__any_sync(0xffffffffu, *ab)) return false;
        if (__all_sync(0xffffffffu, md::mbar_try_wait(bar, parity))) return true;
        const unsigned now = *loads;
        if (__any_sync(0xffffffffu, now != seen)) {
            seen = now;
            since = clock64();
        } else if (__any_sync(0xffffffffu, clock64() - since > kWaitCycles)) {
            break;
        }
    }
    *ab = 1;
    if ((threadIdx.x & 31) == 0) md::report(a.status, MD_ERR_TIMEOUT);
    __syncwarp();
    return false;
}

// By the loading warp, every 64 blocks of a tile.
__device__ __forceinline__ void sign_of_life(Shared *sh, unsigned n)
{
    if ((threadIdx.x & 31) == 0) *(volatile unsigned *)&sh->loads = n;
    __syncwarp();
}

// Wait of the epilogue's warps: the first polls, the others sleep at a barrier,
// and all get its answer (they share barriers, so they leave together).
__device__ __forceinline__ bool epilogue_wait(uint64_t *bar, uint32_t parity, Shared *sh, const Args &a)
{
    const bool ok = threadIdx.x >= 32 || warp_wait(bar, parity, sh, a);
    int r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n"
                 " selp.s32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((int)ok), "n"(kEpiWarps * 32)
                 : "memory");
    return r != 0;
}

struct Tile {
    int e, m0;       // expert, first weight row of the CTA (pair: of its half)
    int64_t r0;      // first x row (wgrad: of the expert)
    int count;       // rows (wgrad: of the expert)
    int c0;          // wgrad: first dw column
    int n;           // MMA N
    int subs;        // k_expert_wide: M = 256 products
};

// A place in the ring of stages: the stage and the parity of its turn.
struct Turn {
    int stages;
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ explicit Turn(int n) : stages(n) {}
    __device__ __forceinline__ void next()
    {
        if (++s == stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ void back()
    {
        if (s-- == 0) {
            s = stages - 1;
            parity ^= 1u;
        }
    }
};

// Await the copies in flight, whoever gave up: the last load of each stage (or, by `empty`, its last use).
__device__ __forceinline__ void drain_loads(Turn at, int used, uint64_t *bars)
{
    for (int j = 0; j < used; ++j) {
        at.back();
        md::mbar_wait_bounded(&bars[at.s], at.parity, kDrainPolls);
    }
}

// Experts' starts and counts, the running number of row tiles, and the
// experts in the order of their tiles; in shared memory.
struct Table {
    int *base;
    int E;
    __device__ __forceinline__ Table(void *at, int n) : base(static_cast<int *>(at)), E(n) {}
    __device__ __forceinline__ int &off(int e) const { return base[e]; }
    __device__ __forceinline__ int &cnt(int e) const { return base[E + e]; }
    __device__ __forceinline__ int &pre(int i) const { return base[2 * E + i]; }
    __device__ __forceinline__ int &order(int i) const { return base[3 * E + i]; }
    static size_t bytes(int E) { return 16 * (size_t)E; }
};

// The experts' ranges, checked, by all threads.
__device__ __forceinline__ void read_ranges(const Table &tab, const Args &a)
{
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int o = __ldg(a.offsets + e), c = __ldg(a.counts + e);
        if (c < 0 || (c > 0 && (o < 0 || (int64_t)o + c > a.rows))) {
            md::report(a.status, MD_ERR_DATA);
            c = 0;
        }
        tab.off(e) = c > 0 ? o : 0;
        tab.cnt(e) = c;
        tab.order(e) = e;
    }
}

// Rows of a row tile of an expert with c rows: equal tiles of at most BN.
template <int CG, int BN>
__device__ __forceinline__ int tile_rows(int c)
{
    return md::ragged_rows(c, BN, 16 * CG);
}

// Order the experts by the cost of their tiles, falling (equal: by number), by
// all threads; a barrier follows.  Tiles are dealt to the clusters back and
// forth, so that the clusters' sums stay within a tile of each other and
// the cheapest tiles come last.
template <int MODE>
__device__ __forceinline__ void sort_experts(const Table &tab, const Args &a)
{
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        tab.pre(e) = MODE == kWgrad ? tab.cnt(e) : tile_rows<2, 256>(tab.cnt(e));
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        const int c = tab.pre(e);
        int before = 0;
        for (int o = 0; o < a.E; ++o) before += tab.pre(o) > c || (tab.pre(o) == c && o < e);
        tab.order(before) = e;
    }
    __syncthreads();
}

// Exclusive running sum of the experts' row tiles, by all threads; barriers inside.  Ranges that
// overlap so far that they make more tiles than the rows can (and more than the host
// has allowed for) leave -1: no tiles, and a report at the kernel's end (here it
// would cost a one-token call 0.1 us).
template <int BN>
__device__ __forceinline__ void count_tiles(const Table &tab, Shared *sh, const Args &a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t run = 0;
    for (int e0 = 0; e0 < a.E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        const int own = e < a.E ? md::ragged_tiles(tab.cnt(tab.order(e)), BN) : 0;
        int v = own;  // an expert has 2^25 tiles at most, 32 of them 2^30
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) sh->sums[warp] = v;
        __syncthreads();
        int64_t before = run;
        for (int w = 0; w < warps; ++w) {
            before += w < warp ? sh->sums[w] : 0;
            run += sh->sums[w];
        }
        if (e < a.E) tab.pre(e) = (int)(before + v - own);
        __syncthreads();
    }
    if (threadIdx.x == 0) sh->tiles = run > a.row_tiles ? -1 : (int)run;
}

// Rows of row tile rt; a converged warp, which looks at 32 places of the order at once.
template <int CG, int BN>
__device__ __forceinline__ Tile rows_at(int rt, const Table &tab, const Args &a)
{
    constexpr int kGran = 16 * CG;
    // the last place in the order whose first tile is at or before rt: every `stride`-th first
    const int lane = threadIdx.x & 31, stride = (a.E + 31) >> 5;
    int at_place = lane * stride;
    unsigned m = __ballot_sync(0xffffffffu, at_place < a.E && tab.pre(at_place) <= rt);
    const int from = (__popc(m) - 1) * stride;
    at_place = from + lane;
    m = __ballot_sync(0xffffffffu, lane < stride && at_place < a.E && tab.pre(at_place) <= rt);
    const int lo = from + __popc(m) - 1;
    Tile q;
    q.e = tab.order(lo);
    const int c = tab.cnt(q.e), each = tile_rows<CG, BN>(c), at = (rt - tab.pre(lo)) * each;
    q.m0 = 0;
    q.r0 = (int64_t)tab.off(q.e) + at;
    q.count = c - at < each ? c - at : each;
    q.c0 = 0;
    q.n = (q.count + kGran - 1) / kGran * kGran;
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
// passes 1.75.  Inf and NaN are left out of amax and stored as NaN: a maximum drops
// NaN by itself and the conversion keeps it; blocks with Inf (or nothing but NaN)
// are looked through again.
__device__ __forceinline__ void pack_block(const float (&v)[8], bool valid, bool store, uint8_t *code,
                                           uint8_t *scale, bool owner)
{
    auto of_block = [](float m) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    };
    float m = fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
                    fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
    m = of_block(valid ? m : 0.0f);
    const bool odd = __any_sync(0xffffffffu, !(m < INFINITY));
    if (odd) {
        float f = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f = fabsf(v[i]) < INFINITY && valid ? fmaxf(f, fabsf(v[i])) : f;
        m = of_block(f);
    }
    const uint32_t bits = __float_as_uint(m);
    int s = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    s = s < 0 ? 0 : s;  // biased by 127
    if (!store) return;
    const float inv = __uint_as_float((uint32_t)(254 - s) << 23);  // 2^(127 - s), s <= 247
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = e4m3x2(v[4 * h] * inv, v[4 * h + 1] * inv) | (e4m3x2(v[4 * h + 2] * inv, v[4 * h + 3] * inv) << 16);
    if (odd) {  // the conversion would keep Inf as 448
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(v[i]) == INFINITY) w[i >> 2] |= 0x7fu << (i & 3) * 8;
    }
    *reinterpret_cast<uint2 *>(code) = make_uint2(w[0], w[1]);
    if (owner) *scale = (uint8_t)s;
}

// Output of 32 accumulator columns (x rows c .. c + 31 of the tile): v[i] is column c + i of
// this thread's TMEM lane.  The group of four warps turns them around in its 8 KB staging
// buffer (32 rows of 128 bf16, or twice 16 rows of 128 floats), so that global
// stores are rows of 16-byte pieces.
constexpr int kStagingBytes = 2 * 8192;

template <int MODE>
__device__ __forceinline__ void emit(const uint32_t (&v)[32], int c, const Tile &q, unsigned char *staging,
                                     const Args &a)
{
    const int lane = threadIdx.x & 31, gw = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
    const int row = threadIdx.x & 127;  // TMEM lane: weight row of the tile
    const int live = q.count - c < 32 ? q.count - c : 32;
    if (MODE != kGated) {
        __nv_bfloat16 *st = reinterpret_cast<__nv_bfloat16 *>(staging + group * 8192);
#pragma unroll
        for (int i = 0; i < 32; ++i) st[i * kTileM + row] = __float2bfloat16_rn(__uint_as_float(v[i]));
        md::named_barrier(2 + group, 128);
        const uint4 *src = reinterpret_cast<const uint4 *>(st);
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y);
        const int n0 = q.m0 + (row & 15) * 8;
        if (n0 < a.n)
            for (int i = row >> 4; i < live; i += 8)
                *reinterpret_cast<uint4 *>(y + (q.r0 + c + i) * a.pitch + n0) = src[i * 16 + (row & 15)];
        md::named_barrier(2 + group, 128);  // the buffer is free again
        return;
    }
    // lanes 0-63 of the tile hold g, 64-127 hold u of the same columns
    float *st = reinterpret_cast<float *>(staging + group * 8192);
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        if (h >= live) break;
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i * kTileM + row] = __uint_as_float(v[h + i]);
        md::named_barrier(2 + group, 128);
        const int j = lane & 7, f0 = q.m0 + j * 8;
        const bool valid = f0 < a.n;
        const int i0 = gw * 4 + h;  // four rows to a warp
        if (i0 < live) {
            const bool in = i0 + (lane >> 3) < live;
            const int ii = in ? i0 + (lane >> 3) : i0;
            float g[8], u[8];
            const float *at = st + (ii - h) * kTileM + j * 8;
            const int64_t r = q.r0 + c + ii;
            const int blocks = (a.n + kBlock - 1) / kBlock;
            *reinterpret_cast<float4 *>(g) = *reinterpret_cast<const float4 *>(at);
            *reinterpret_cast<float4 *>(g + 4) = *reinterpret_cast<const float4 *>(at + 4);
            if (a.codes)
                pack_block(g, valid, valid && in, a.codes + r * 2 * a.n + f0, a.scales + r * 2 * blocks + f0 / kBlock,
                           (j & 3) == 0);
#pragma unroll
            for (int p = 0; p < 8; ++p) g[p] *= md::sigmoid(g[p]);
            *reinterpret_cast<float4 *>(u) = *reinterpret_cast<const float4 *>(at + 64);
            *reinterpret_cast<float4 *>(u + 4) = *reinterpret_cast<const float4 *>(at + 68);
            if (a.codes)
                pack_block(u, valid, valid && in, a.codes + r * 2 * a.n + a.n + f0,
                           a.scales + r * 2 * blocks + blocks + f0 / kBlock, (j & 3) == 0);
            if (valid && in) {
                uint32_t w[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) w[p] = md::pack_bf16x2(g[2 * p] * u[2 * p], g[2 * p + 1] * u[2 * p + 1]);
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + r * a.pitch + f0) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        md::named_barrier(2 + group, 128);  // the buffer is free again
    }
}

// ------------------------------------------------------- few rows to an expert
//
// Tiles of 128 weight rows by up to 64 x rows, one CTA each.  The time is that of
// reading every chosen expert's weights once, so what counts is bytes in
// flight: a ring of 8 stages keeps 128 KB of weights on the way to each SM.
// Where there are too few tiles for the GPU (one token's eight experts), a cluster
// of CTAs shares each tile's contraction: every CTA leaves its float32 part in its
// ring's memory, and the first adds them in their order.
template <int MODE>
struct Few {
    static constexpr int BN = 64, kStages = 8, kBox = 16;  // x rows per TMA box
    static constexpr int kStageBytes = kABytes + BN * kTileK * 2;
    static constexpr int kThreads = 32 * 10;
    static constexpr int kWidth = MODE == kGated ? 64 : kTileM;  // output columns of a tile
    static constexpr int kCols = 2 * BN;                         // TMEM columns: two accumulators
    static size_t smem(int E) { return 1024 + (size_t)kStages * kStageBytes + kStagingBytes + Table::bytes(E); }
};

struct FewBars {
    uint64_t full[8], empty[8], tfull[2], tempty[2], drain;
};

template <int MODE>
__global__ void __launch_bounds__(Few<MODE>::kThreads, 1)
    k_expert_few(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ Args a)
{
    using P = Few<MODE>;
    constexpr int BN = P::BN;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared shared;
    __shared__ __align__(16) FewBars bars;
    Shared *sh = &shared;
    FewBars *b = &bars;
    // an offset, not a rounded address: the compiler then knows shared memory as such
    unsigned char *base = smem_raw + (-md::smem_addr(smem_raw) & 1023u);
    unsigned char *staging = base + P::kStages * P::kStageBytes;
    const Table tab(staging + kStagingBytes, a.E);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int share = a.split > 1 ? (int)md::cluster_rank() : 0;  // of the contraction

    if (threadIdx.x == 0) {
        for (int i = 0; i < P::kStages; ++i) {
            md::mbar_init(&b->full[i], 1);
            md::mbar_init(&b->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            md::mbar_init(&b->tfull[i], 1);
            md::mbar_init(&b->tempty[i], kEpiWarps);
        }
        md::mbar_init(&b->drain, 1);
        sh->abort = 0;
        sh->loads = 0;
        md::fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        md::prefetch_map(&map_a);
        md::prefetch_map(&map_b);
    }
    if (warp == kMmaWarp) md::tmem_alloc<1>(&sh->tmem, P::kCols);
    read_ranges(tab, a);
    __syncthreads();
    count_tiles<BN>(tab, sh, a);
    md::tmem_fence_before();
    __syncthreads();
    md::tmem_fence_after();
    const uint32_t tmem = sh->tmem;

    const int first = blockIdx.x / a.split, step = gridDim.x / a.split;
    const int total = max(sh->tiles, 0) * (int)a.mt.d;  // the host keeps it below 2^30
    const uint32_t sbase = md::smem_addr(base);
    // blocks of the contraction: [kb0, kb1) in this CTA
    const int kblocks = (a.k + kTileK - 1) / kTileK;
    const int kb0 = kblocks * share / a.split, kb1 = kblocks * (share + 1) / a.split;
    auto tile_of = [&](int t) {
        const int rt = a.mt.div(t);
        Tile q = rows_at<1, BN>(rt, tab, a);
        q.m0 = (t - rt * (int)a.mt.d) * P::kWidth;
        return q;
    };

    if (warp == kLoadWarp) {
        // ------------------------------------------------ loads
        Turn at(P::kStages);
        int used = 0;        // stages loaded at least once
        unsigned begun = 0;  // signs of life
        bool ok = true;
        for (int t = first; ok && t < total; t += step) {
            const Tile q = tile_of(t);
            const int boxes = (q.n + P::kBox - 1) / P::kBox, r0 = (int)q.r0;
            const uint32_t bytes = kABytes + boxes * P::kBox * 128;
            for (int i = kb0; i < kb1; ++i) {
                const int s = at.s;
                if (!(ok = warp_wait(&b->empty[s], at.parity ^ 1u, sh, a))) break;
                const uint32_t bar = md::smem_addr(&b->full[s]);
                if (i % 64 == 0) sign_of_life(sh, ++begun);
                md::expect_tx_one(&b->full[s], bytes);
                const uint32_t sa = sbase + s * P::kStageBytes, sb = sa + kABytes;
                const int k0 = i * kTileK;
                if (MODE == kNK) {
                    md::tma_load_3d<1>(sa, &map_a, k0, q.m0, q.e, bar);
                } else if (MODE == kGated) {
                    md::tma_load_3d<1>(sa, &map_a, k0, q.m0, q.e, bar);
                    md::tma_load_3d<1>(sa + 8192, &map_a, k0, a.n + q.m0, q.e, bar);
                } else {
                    md::tma_load_3d<1>(sa, &map_a, q.m0, k0, q.e, bar);
                    md::tma_load_3d<1>(sa + 8192, &map_a, q.m0 + 64, k0, q.e, bar);
                }
                for (int j = 0; j < boxes; ++j)
                    md::tma_load_2d<1>(sb + j * P::kBox * 128, &map_b, k0, r0 + j * P::kBox, bar);
                if (used < P::kStages) ++used;
                at.next();
            }
        }
        drain_loads(at, used, b->full);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ products
        constexpr bool kAKMajor = MODE != kKN;
        const uint64_t da0 = kAKMajor ? md::operand_desc(sbase, 16, 1024) : md::operand_desc(sbase, 8192, 1024);
        const uint64_t db0 = md::operand_desc(sbase + kABytes, 16, 1024);
        constexpr int kAStep = (kAKMajor ? 32 : 2048) >> 4;
        Turn at(P::kStages);
        int acc = 0;
        bool ok = true;
        for (int t = first; ok && t < total; t += step, ++acc) {
            const Tile q = tile_of(t);
            const int buf = acc & 1;
            const uint32_t idesc = md::mma_desc(kTileM, q.n, !kAKMajor, false), d = tmem + buf * BN;
            if (!warp_wait(&b->tempty[buf], (uint32_t)((acc >> 1) & 1) ^ 1u, sh, a)) break;
            md::tmem_fence_after();
            for (int i = kb0; i < kb1; ++i) {
                const int s = at.s;
                if (!(ok = warp_wait(&b->full[s], at.parity, sh, a))) break;
                md::tmem_fence_after();
                const uint64_t da = da0 + (uint32_t)(s * (P::kStageBytes >> 4));
                const uint64_t db = db0 + (uint32_t)(s * (P::kStageBytes >> 4));
#pragma unroll
                for (int j = 0; j < kTileK / 16; ++j)
                    md::mma_bf16<1>(d, da + j * kAStep, db + j * 2, idesc, i > kb0 || j > 0);
                md::mma_commit<1>(&b->empty[s]);
                if (i == kb1 - 1) md::mma_commit<1>(&b->tfull[buf]);
                at.next();
            }
        }
        md::mma_commit<1>(&b->drain);  // await the MMAs in flight, whoever gave up
        md::mbar_wait_bounded(&b->drain, 0, kDrainPolls);
    } else {
        // ------------------------------------------------ results
        int acc = 0;
        const int group = warp >> 2;
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        for (int t = first; t < total; t += step, ++acc) {
            const Tile q = tile_of(t);
            const int buf = acc & 1;
            if (!epilogue_wait(&b->tfull[buf], (uint32_t)((acc >> 1) & 1), sh, a)) break;
            md::tmem_fence_after();
            const int c = group * 32;
            uint32_t v[32];
            if (c < q.count) {
                md::tmem_ld32(v, tmem + quarter + buf * BN + c);
                md::tmem_ld_wait();
            }
            md::tmem_fence_before();
            __syncwarp();
            if (lane == 0) md::mbar_arrive(&b->tempty[buf]);
            if (c >= q.count) continue;
            if (a.split > 1) {  // left in the ring's memory, which this cluster's one tile is done with
                float *pt = reinterpret_cast<float *>(base);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i < q.count) pt[(c + i) * kTileM + (threadIdx.x & 127)] = __uint_as_float(v[i]);
            } else {
                emit<MODE>(v, c, q, staging, a);
            }
        }
    }

    if (a.split > 1) {
        __syncwarp();
        __syncthreads();
        md::cluster_sync();
        if (share == 0 && warp < kEpiWarps && first < total) {
            const Tile q = tile_of(first);
            const int c = (warp >> 2) * 32;
            if (c < q.count) {
                uint32_t v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
                for (int p = 0; p < a.split; ++p) {
                    const uint32_t from = md::map_rank(sbase + (c * kTileM + (threadIdx.x & 127)) * 4, p);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < q.count)
                            v[i] = __float_as_uint(__uint_as_float(v[i]) + md::ld_cluster(from + i * kTileM * 4));
                }
                emit<MODE>(v, c, q, staging, a);
            }
        }
    }

    if (threadIdx.x == 0 && sh->tiles < 0) md::report(a.status, MD_ERR_DATA);
    // ---- end: nobody leaves while its cluster may still read its shared memory
    __syncwarp();
    md::tmem_fence_before();
    __syncthreads();
    if (a.split > 1) md::cluster_sync();
    md::tmem_fence_after();
    if (warp == kMmaWarp) md::tmem_free<1>(tmem, P::kCols);
}

// ------------------------------------------------------ many rows to an expert
//
// A pair of CTAs makes 512 weight rows by up to 256 x rows (weight gradient: by 256
// columns): two M = 256 products ("subs") that share each block of x.  Every block of 64 of
// the contraction then brings 48 KB into an SM for 1024 tensor-core cycles.  What
// bounds this form is that path: about 45 bytes a cycle reach an SM from L2 when
// all of them load, and one 256 x 256 product per block needs 64 (it measured 70%
// of the tensor cores' rate; two need 47).  Calls with too few such tiles for the
// GPU take one sub.
//
// A stage holds a block of sub 0's A, of x, and of sub 1's A, on one barrier, and
// A and x have a loading warp each: the instructions around a barrier and its copies
// took longer than the products when one thread did it all.
//
// The two accumulators of 256 columns fill TMEM and are used in turn, one for
// each (tile, sub).  The epilogue's warps take an accumulator into registers and
// free it before most of it is written out, and at a tile's first and last blocks
// the subs go two blocks at a time, so that each accumulator has 1024 cycles to be
// freed while the other sub works.  For that the epilogue's warps hold up to 216
// registers: 12 warps of 168 at launch, 8 x 216 + 4 x 72 after.
//
// Weight gradient.  The contraction runs over an expert's rows, and its last block
// reaches into the next expert's: rows past the end are cleared in shared memory
// on both sides (zero times a stray NaN or Inf is not zero), by the MMA warp of
// each CTA.  For such a block the second CTA awaits its loads on a barrier of
// its own, clears, and tells the first; passing every stage on this way took a
// quarter of the loads' rate.  The tensor cores drop low bits at each
// addition, and a sum of n rows summed whole is off by some 1.2e-9 n (2-norm, normal data):
// 5.3e-5 for an expert of 46080 rows.  float32 results are therefore summed in TMEM over
// kSegment blocks at most, in equal shares, and then added in dw, in order: 1.1e-6 there.
// Of 131072 skewed rows over 128 experts 1.6e-6 becomes 0.9e-6, for 5% of the time (32
// blocks: 1.1e-6).
constexpr int kSegment = 18;

constexpr int kLaunchRegisters = 168;  // 12 warps of them: the sum of the split 8 x 216 + 4 x 72

template <int MODE>
struct Wide {
    static constexpr int kPart = 128 * kTileK * 2;  // 16 KB: 128 rows of A, or half of the tile's x rows
    // 4 stages of three parts, or 6 of two (one sub).  Weight gradient: 3 or 4, and two buffers of
    // 4 KB a warp for dw in the rest.
    static constexpr int kParts = MODE == kWgrad ? 9 : 12;
    static constexpr int kStaging = MODE == kWgrad ? kEpiWarps * 8192 : kStagingBytes;
    static constexpr int kThreads = 32 * 12;
    static constexpr int kSub = MODE == kGated ? 128 : 256;  // output columns of a sub
    static size_t smem(int E) { return 1024 + (size_t)kParts * kPart + kStaging + Table::bytes(E); }
};

struct WideBars {
    uint64_t full[6], empty[6], tfull[2], tempty[2], drain;
    // Weight gradient, a tile's last block in stage s: loaded (second CTA's barrier), and cleared
    // there (first CTA's).  One for each stage, since the loads run tiles ahead of
    // the products where tiles are short; roles keep their parities in a bit for each.
    uint64_t tail[6], cleared[6];
};

// Blocks that the subs take at a time from block i on.
__device__ __forceinline__ int blocks_at(int i, int kb, int subs)
{
    return subs == 2 && kb - i >= 2 && (i == 0 || i == kb - 2) ? 2 : 1;
}

// 32 columns of dw's rows, one row in each lane of the warp, into one of the warp's two
// 4 KB buffers: 32 rows of 128 bytes in the map's swizzle, which hold 32 float32
// columns or two runs of bf16 ones.
__device__ __forceinline__ void fill_rows(const uint32_t (&v)[32], const Args &a, bool odd, unsigned char *st)
{
    const int lane = threadIdx.x & 31, sw = (lane & 7) * 16;
    unsigned char *row = st + lane * 128;
    if (a.out_bf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                w[h] = md::pack_bf16x2(__uint_as_float(v[8 * i + 2 * h]), __uint_as_float(v[8 * i + 2 * h + 1]));
            *reinterpret_cast<uint4 *>(row + ((i * 16 + (odd ? 64 : 0)) ^ sw)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4 *>(row + (i * 16 ^ sw)) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// The filled buffer to dw, stored or added by TMA: the map cuts the box at dw's edges, and the
// warp goes on to the next columns.  Rows of 128 bytes: where dw's rows are not a multiple
// of 32 bytes long, each box row ends in parts of sectors, and with 64-byte rows the
// stores took twice the time.  Plain stores, from registers (32 lines each) or
// turned around in shared memory, were slower: the warp's own time.
__device__ __forceinline__ void send_rows(const CUtensorMap *map, int c, int row0, int e, bool add, const unsigned char *st)
{
    md::fence_async_shared();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        if (add) md::tma_add_3d(map, md::smem_addr(st), c, row0, e);
        else md::tma_store_3d(map, md::smem_addr(st), c, row0, e);
        md::bulk_commit();
    }
}

template <int MODE>
__global__ void __launch_bounds__(Wide<MODE>::kThreads, 1)
    k_expert_wide(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_d, const __grid_constant__ Args a)
{
    using W = Wide<MODE>;
    constexpr int BN = 256;
    constexpr bool kWg = MODE == kWgrad;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared shared;
    __shared__ __align__(16) WideBars bars;
    Shared *sh = &shared;
    WideBars *b = &bars;
    // an offset, not a rounded address: the compiler then knows shared memory as such
    unsigned char *base = smem_raw + (-md::smem_addr(smem_raw) & 1023u);
    unsigned char *staging = base + W::kParts * W::kPart;
    const Table tab(staging + W::kStaging, a.E);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)md::cluster_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < 6; ++i) {
            md::mbar_init(&b->full[i], 2);  // the first CTA's two loading threads
            md::mbar_init(&b->empty[i], 1);
            md::mbar_init(&b->tail[i], 2);
            md::mbar_init(&b->cleared[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            md::mbar_init(&b->tfull[i], 1);
            md::mbar_init(&b->tempty[i], kEpiWarps * 2);
        }
        md::mbar_init(&b->drain, 1);
        sh->abort = 0;
        sh->loads = 0;
        md::fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0) md::prefetch_map(&map_a);
    if (warp == kLoadXWarp && lane == 0) md::prefetch_map(&map_b);
    if (warp == kMmaWarp) md::tmem_alloc<2>(&sh->tmem, 512);
    read_ranges(tab, a);
    __syncthreads();
    sort_experts<MODE>(tab, a);
    if (!kWg) count_tiles<BN>(tab, sh, a);
    md::tmem_fence_before();
    md::cluster_sync();
    __syncthreads();
    md::tmem_fence_after();
    const uint32_t tmem = sh->tmem;

    const int width = a.subs * W::kSub;  // output columns (weight gradient: rows of dw) of a tile
    const int mt = (int)a.mt.d;
    const int total = kWg ? a.E * (int)a.per.d : max(sh->tiles, 0) * mt;  // the host keeps it below 2^30
    const int step = gridDim.x / 2, place = blockIdx.x / 2, rounds = (total + step - 1) / step;
    // the cluster's tile of a round, dealt back and forth; `total` or more: none
    auto deal = [&](int round) { return round * step + (round & 1 ? step - 1 - place : place); };
    const uint32_t sbase = md::smem_addr(base);
    const int stages = W::kParts / (a.subs + 1), stage_bytes = (a.subs + 1) * W::kPart;
    auto tile_of = [&](int t) {
        Tile q;
        int mi;  // tile along the weight rows
        if (kWg) {
            const int at = a.per.div(t), i = t - at * (int)a.per.d, ci = a.mt.div(i);
            mi = i - ci * mt;
            q.e = tab.order(at);
            q.r0 = tab.off(q.e);
            q.count = tab.cnt(q.e);
            q.c0 = ci * BN;
            q.n = (min(a.k - q.c0, BN) + 31) / 32 * 32;
        } else {
            const int rt = a.mt.div(t);
            mi = t - rt * mt;
            q = rows_at<2, BN>(rt, tab, a);
        }
        q.m0 = mi * width + rank * (W::kSub / 2);
        // the last tile along the weight rows may have one sub where others have two
        q.subs = a.subs == 2 && mi * width + W::kSub < a.n ? 2 : 1;
        return q;
    };
    // blocks of the tile's contraction
    auto blocks_of = [&](const Tile &q) { return ((kWg ? q.count : a.k) + kTileK - 1) / kTileK; };
    // blocks that one accumulator sums: all, or an equal share of kSegment at most
    auto segment_of = [&](int blocks) {
        if (!kWg || a.out_bf16 || blocks <= kSegment) return blocks;
        const int parts = (blocks + kSegment - 1) / kSegment;
        return (blocks + parts - 1) / parts;
    };

    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kLoadWarp || warp == kLoadXWarp) {
            // ------------------------------------------------ loads
            Turn at(stages);
            int used = 0;        // stages loaded at least once
            unsigned begun = 0;  // signs of life
            uint32_t tails = 0, used_tails = 0;
            bool ok = true;
            for (int round = 0; ok && round < rounds; ++round) {
                const int t = deal(round);
                if (t >= total) continue;
                const Tile q = tile_of(t);
                const int subs = q.subs, kb = blocks_of(q);
                const int half = q.n / 2, boxes = (half + 63) / 64;  // N-side lines of this CTA
                const int r0 = (int)q.r0 + (kWg ? 0 : rank * half), c0 = q.c0 + rank * half;
                const uint32_t bytes = warp == kLoadWarp ? subs * W::kPart : boxes * 8192;
                for (int i = 0; i < kb; ++i) {
                    if (!(ok = warp_wait(&b->empty[at.s], at.parity ^ 1u, sh, a))) break;
                    if (i % 64 == 0 && warp == kLoadWarp) sign_of_life(sh, ++begun);
                    // the first CTA's barrier counts both CTAs' bytes, but for a block to be cleared
                    const bool tail = kWg && i == kb - 1 && q.count % kTileK != 0;
                    uint32_t bar = md::map_rank(md::smem_addr(&b->full[at.s]), 0);
                    if (rank == 0) {
                        md::expect_tx_one(&b->full[at.s], tail ? bytes : 2 * bytes);
                    } else if (tail) {
                        md::expect_tx_one(&b->tail[at.s], bytes);
                        bar = md::map_rank(md::smem_addr(&b->tail[at.s]), 1);
                        used_tails |= 1u << at.s;
                        tails ^= 1u << at.s;
                    }
                    const uint32_t to = sbase + at.s * stage_bytes;
                    const int k0 = i * kTileK;
                    if (warp == kLoadXWarp) {
                        for (int j = 0; j < boxes; ++j) {
                            const uint32_t tx = to + W::kPart + j * 8192;
                            if (kWg) md::tma_load_2d<2>(tx, &map_b, c0 + j * 64, r0 + k0, bar);
                            else md::tma_load_2d<2>(tx, &map_b, k0, r0 + j * 64, bar);
                        }
                    } else {
                        for (int sub = 0; sub < subs; ++sub) {
                            const uint32_t ta = to + sub * 2 * W::kPart;
                            const int m = q.m0 + sub * W::kSub;
                            if (MODE == kNK) {
                                md::tma_load_3d<2>(ta, &map_a, k0, m, q.e, bar);
                            } else if (MODE == kGated) {
                                md::tma_load_3d<2>(ta, &map_a, k0, m, q.e, bar);
                                md::tma_load_3d<2>(ta + 8192, &map_a, k0, a.n + m, q.e, bar);
                            } else if (MODE == kKN) {
                                md::tma_load_3d<2>(ta, &map_a, m, k0, q.e, bar);
                                md::tma_load_3d<2>(ta + 8192, &map_a, m + 64, k0, q.e, bar);
                            } else {
                                md::tma_load_2d<2>(ta, &map_a, m, r0 + k0, bar);
                                md::tma_load_2d<2>(ta + 8192, &map_a, m + 64, r0 + k0, bar);
                            }
                        }
                    }
                    if (used < stages) ++used;
                    at.next();
                }
            }
            if (rank == 0) drain_loads(at, used, b->full);
            else
                for (int i = 0; i < stages; ++i)
                    if (used_tails >> i & 1u) md::mbar_wait_bounded(&b->tail[i], (tails >> i & 1u) ^ 1u, kDrainPolls);
            if (rank == 1 && !ok)
                for (int j = 0; j < 2000; ++j) __nanosleep(500);
            // nor may the products' last arrivals, which come from the first CTA, be still on their
            // way when this CTA's shared memory is given up
            if (ok && rank == 1) drain_loads(at, used, b->empty);
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------ products
            // Clears the lines from v on, up to the last of `steps` sixteenths, of every box of a stage.
            auto clear = [&](int s, int v, int steps, int xboxes, int subs) {
                const int boxes = 2 + xboxes + (subs == 2 ? 2 : 0), lines = steps * 16 - v;
                for (int z = lane; z < lines * 8 * boxes; z += 32) {
                    int box = z / (lines * 8);
                    const int w = z - box * (lines * 8);
                    if (box >= 2 + xboxes) box += 2 - xboxes;  // sub 1's A, behind x's two boxes
                    *reinterpret_cast<uint4 *>(base + s * stage_bytes + box * 8192 + (v + (w >> 3)) * 128 + (w & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                md::fence_async_shared();
                __syncwarp();
            };
            uint32_t tails = 0;
            if (kWg && rank == 1) {
                Turn at(stages);
                for (int round = 0; round < rounds; ++round) {
                    const int t = deal(round);
                    if (t >= total) continue;
                    const Tile q = tile_of(t);
                    for (int i = 0; i < blocks_of(q); ++i) at.next();
                    const int v = q.count % kTileK;
                    if (v == 0) continue;
                    at.back();
                    if (!warp_wait(&b->tail[at.s], tails >> at.s & 1u, sh, a)) break;
                    tails ^= 1u << at.s;
                    clear(at.s, v, (v + 15) / 16, (q.n / 2 + 63) / 64, q.subs);
                    if (lane == 0) md::mbar_arrive_cluster(md::map_rank(md::smem_addr(&b->cleared[at.s]), 0));
                    at.next();
                }
            } else if (rank == 0) {
                constexpr bool kAKMajor = MODE == kNK || MODE == kGated;
                const uint64_t da0 = kAKMajor ? md::operand_desc(sbase, 16, 1024) : md::operand_desc(sbase, 8192, 1024);
                const uint64_t db0 = kWg ? md::operand_desc(sbase, 8192, 1024) : md::operand_desc(sbase, 16, 1024);
                constexpr int kAStep = (kAKMajor ? 32 : 2048) >> 4, kBStep = (kWg ? 2048 : 32) >> 4;
                auto await = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, sh, a); };
                Turn at(stages);
                uint32_t opened = 0;  // accumulators taken so far
                bool ok = true;
                for (int round = 0; ok && round < rounds; ++round) {
                    const int t = deal(round);
                    if (t >= total) continue;
                    const Tile q = tile_of(t);
                    const int subs = q.subs, blocks = blocks_of(q);
                    const uint32_t idesc = md::mma_desc(256, q.n, !kAKMajor, kWg);
                    const int segment = segment_of(blocks);
                    for (int from = 0, kb; ok && from < blocks; from += kb, opened += subs) {
                        kb = min(blocks - from, segment);
                        // block i of one sub, in stage s; of a last block as many sixteenths as hold rows
                        auto product = [&](int sub, int i, int s) {
                            const uint32_t acc = opened + sub;
                            if (i == 0) {
                                if (!await(&b->tempty[acc & 1], ((acc >> 1) & 1u) ^ 1u)) return false;
                                md::tmem_fence_after();
                            }
                            const uint32_t off = (uint32_t)(s * stage_bytes) >> 4;
                            const uint64_t da = da0 + off + (sub ? 2 * W::kPart >> 4 : 0), db = db0 + off + (W::kPart >> 4);
                            const int v = q.count - (from + i) * kTileK;
                            if (!kWg || v > kTileK - 16) {
#pragma unroll
                                for (int j = 0; j < kTileK / 16; ++j)
                                    md::mma_bf16<2>(tmem + (acc & 1) * BN, da + j * kAStep, db + j * kBStep, idesc, i > 0 || j > 0);
                            } else {
#pragma unroll 1
                                for (int j = 0; j * 16 < v; ++j)
                                    md::mma_bf16<2>(tmem + (acc & 1) * BN, da + j * kAStep, db + j * kBStep, idesc, i > 0 || j > 0);
                            }
                            if (sub == subs - 1) md::mma_commit<2>(&b->empty[s]);
                            if (i == kb - 1) md::mma_commit<2>(&b->tfull[acc & 1]);
                            return true;
                        };
                        for (int i = 0, g; ok && i < kb; i += g) {
                            g = blocks_at(i, kb, subs);
                            const int s0 = at.s;
                            for (int j = 0; ok && j < g; ++j) {
                                if (!(ok = await(&b->full[at.s], at.parity))) break;
                                const int v = q.count - (from + i + j) * kTileK;  // weight gradient: rows left
                                if (kWg && v < kTileK) {
                                    clear(at.s, v, (v + 15) / 16, (q.n / 2 + 63) / 64, subs);
                                    if (!(ok = await(&b->cleared[at.s], tails >> at.s & 1u))) break;
                                    tails ^= 1u << at.s;
                                }
                                md::tmem_fence_after();
                                ok = product(0, i + j, at.s);
                                at.next();
                            }
                            if (subs == 2)
                                for (int j = 0, st = s0; ok && j < g; ++j, st = st + 1 == stages ? 0 : st + 1)
                                    ok = product(1, i + j, st);
                        }
                    }
                }
                md::mma_commit<2>(&b->drain);  // await the MMAs in flight, whoever gave up
                md::mbar_wait_bounded(&b->drain, 0, kDrainPolls);
            }
        }
    } else {
        // ------------------------------------------------ results
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int group = warp >> 2;
        // a group's runs of 32 columns: every other one, so that a short tile's are shared;
        // weight gradient: adjacent ones, which are adjacent in dw
        constexpr int kRun = kWg ? 32 : 64;
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + group * (kWg ? 128 : 32);
        uint32_t acc = 0;
        int buffer = 0;  // weight gradient: of the warp's two
        bool ok = true;
        // Accumulators are taken in turn: wait for the next, read this warp's columns in runs of 32,
        // give it back.  (All runs are read, the tile's or not: a register that is loaded on a
        // condition stays taken throughout.)
        auto await = [&]() {
            ok = epilogue_wait(&b->tfull[acc & 1], (acc >> 1) & 1u, sh, a);
            md::tmem_fence_after();
            return ok;
        };
        auto read = [&](uint32_t (&v)[32], int run) __attribute__((always_inline)) {
            md::tmem_ld32(v, mine + (acc & 1) * BN + run * kRun);
        };
        auto give_back = [&]() {
            md::tmem_ld_wait();
            md::tmem_fence_before();
            __syncwarp();
            // relaxed: what must be done are the reads of TMEM, and those are waited for; a release
            // would wait for this warp's stores to global memory too
            if (lane == 0) md::mbar_arrive_cluster_relaxed(md::map_rank(md::smem_addr(&b->tempty[acc & 1]), 0));
            ++acc;
        };
        auto take = [&](uint32_t (&v)[4][32]) __attribute__((always_inline)) {
            if (!await()) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) read(v[i], i);
            give_back();
        };
        // the subs' accumulators, out through put(values, sub, run).  Sub 1's is taken when half of sub
        // 0's is out, as soon as the registers allow (one run later: 1 to 4% slower).
        constexpr int kBefore = 2;
        auto results = [&](int subs, auto put) __attribute__((always_inline)) {
            uint32_t v[4][32];
            take(v);
            if (!ok) return;
#pragma unroll
            for (int i = 0; i < kBefore; ++i) put(v[i], 0, i);
            if (subs == 2) {
                uint32_t w[4][32];
                take(w);
                if (!ok) return;
#pragma unroll
                for (int i = kBefore; i < 4; ++i) put(v[i], 0, i);
#pragma unroll
                for (int i = 0; i < 4; ++i) put(w[i], 1, i);
            } else {
#pragma unroll
                for (int i = kBefore; i < 4; ++i) put(v[i], 0, i);
            }
        };
        for (int round = 0; ok && round < rounds; ++round) {
            const int t = deal(round);
            if (t >= total) continue;
            const Tile q = tile_of(t);
            const int subs = q.subs;
            if (kWg) {
                const int blocks = blocks_of(q), cols = min(a.k - q.c0, BN);
                if (blocks == 0 && a.accumulate) continue;
                const int segment = max(segment_of(blocks), 1);
                for (int from = 0; from == 0 || (ok && from < blocks); from += segment) {  // once if empty
                    const bool add = a.accumulate || from > 0;
                    if (from > 0) md::bulk_wait_all();  // what this adds to is written
                    auto put = [&](const uint32_t (&x)[32], int sub, int i) __attribute__((always_inline)) {
                        const int c = group * 128 + i * 32, row0 = q.m0 + sub * W::kSub + (warp & 3) * 32;
                        if (c >= cols || row0 >= a.n) return;
                        unsigned char *st = staging + warp * 8192 + buffer;
                        const bool pair = a.out_bf16, odd = pair && (i & 1);
                        if (!odd) {  // the buffer's last store has read it (lane 0's group; the others have none)
                            md::bulk_wait_read<1>();
                            __syncwarp();
                        }
                        fill_rows(x, a, odd, st);
                        if (pair && !odd && c + 32 < cols) return;  // with the next run
                        send_rows(&map_d, q.c0 + c - (odd ? 32 : 0), row0, q.e, add, st);
                        buffer ^= 4096;  // with each store made: a tile's edge may leave some out
                    };
                    if (blocks == 0) {  // an expert without rows
                        uint32_t none[32] = {};
#pragma unroll 1
                        for (int i = 0; i < 4 * subs; ++i) put(none, i >> 2, i & 3);
                        break;
                    }
                    results(subs, put);
                }
            } else {
                auto put = [&](const uint32_t (&x)[32], int sub, int i) __attribute__((always_inline)) {
                    Tile at = q;
                    at.m0 += sub * W::kSub;
                    if (group * 32 + i * 64 < q.count) emit<MODE>(x, group * 32 + i * 64, at, staging, a);
                };
                results(subs, put);
            }
        }
    }

    if (kWg) md::bulk_wait_all();
    if (!kWg && threadIdx.x == 0 && sh->tiles < 0) md::report(a.status, MD_ERR_DATA);
    // ---- end: nobody leaves while its pair may still read its shared memory
    __syncwarp();
    md::tmem_fence_before();
    __syncthreads();
    md::cluster_sync();
    md::tmem_fence_after();
    if (warp == kMmaWarp) {
        // The first CTA has seen its last commit arrive at home; the same commit's arrival here
        // is awaited too, whoever gave up.
        if (md::cluster_rank() == 1) md::mbar_wait_bounded(&bars.drain, 0, kDrainPolls);
        __syncwarp();
        md::tmem_free<2>(tmem, 512);
    }
}

// ------------------------------------------------------------------ host

// One launch in clusters of `members` CTAs of a kernel that needs `registers` a thread.
template <class Kernel, class... Params>
int launch(Kernel kernel, int threads, int registers, size_t smem, size_t most_smem, std::atomic<uint64_t> &setup, int64_t clusters,
           int members, cudaStream_t s, const Params &...params)
{
    md::once_per_device(setup, [&] {
        // the wide form's register split draws on what the block is launched with: fewer registers
        // than the split's sum would never be granted, so such a build is not launched
        cudaFuncAttributes at = {};
        const bool enough = cudaFuncGetAttributes(&at, kernel) == cudaSuccess && at.numRegs >= registers;
        if (!enough || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most_smem) != cudaSuccess)
            cudaGetLastError();  // without its shared memory the launch fails and reports MD_ERR_CUDA
    });
    const int64_t most = md::sm_count() / members;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((clusters < most ? clusters : most) * members));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = members;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, params...) != cudaSuccess) {
        cudaGetLastError();
        return MD_ERR_CUDA;
    }
    md::count_launches(1);
    return md::launch_status();
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

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

constexpr int64_t kMostTiles = (int64_t)1 << 30;

template <int MODE>
int run_few(const void *x, const void *w, int64_t rows, Args &a, int64_t d0, int64_t d1, cudaStream_t s)
{
    using P = Few<MODE>;
    CUtensorMap ma, mb;
    if (!md::make_map(&ma, w, kBf16, 2, d0, d1, a.E, 64, MODE == kNK ? kTileM : 64) ||
        !md::make_map(&mb, x, kBf16, 2, a.k, rows, 0, 64, P::kBox))
        return MD_ERR_CUDA;
    const int mt = (a.n + P::kWidth - 1) / P::kWidth;
    a.mt = FastDiv((uint32_t)mt);
    a.row_tiles = md::ragged_most_tiles(rows, a.E, P::BN);
    const int64_t tiles = a.row_tiles * mt;
    if (tiles > kMostTiles) return MD_ERR_UNSUPPORTED;
    // Few tiles leave SMs idle and each tile streams its weights through one SM: clusters of
    // CTAs share a tile's contraction, as long as all of them are resident and each has
    // four blocks or more.
    a.split = 1;
    while (a.split < kMaxSplit && tiles * a.split * 2 <= md::sm_count() && a.k >= a.split * 2 * 4 * kTileK)
        a.split *= 2;
    static std::atomic<uint64_t> setup{0};
    return launch(k_expert_few<MODE>, P::kThreads, 0, P::smem(a.E), P::smem(MD_MAX_EXPERTS), setup, tiles, a.split, s, ma,
                  mb, a);
}

// Two subs to a tile where that still gives the pairs of SMs several tiles each: from four
// tiles of one sub to a pair (16 experts of 384 rows, 2048 x 2048, one sub / two: 53 / 48 us; of
// 256 rows 37 / 37; 8 experts of 512 rows, 2048 x 1024: 19 / 28), for the weight gradient
// from eight (8 experts of 256 rows, 2048 x 2048: 32 / 38; 16 of 512 rows 88 / 82).
inline int subs_for(int64_t tiles_of_one, int to_a_pair)
{
    const int path = md::expert_path();
    if (path == MD_EXPERT_ONE || path == MD_EXPERT_TWO) return path == MD_EXPERT_TWO ? 2 : 1;
    return tiles_of_one >= (int64_t)to_a_pair * (md::sm_count() / 2) ? 2 : 1;
}

template <int MODE>
int run_wide(const void *x, const void *w, int64_t rows, Args &a, int64_t d0, int64_t d1, cudaStream_t s)
{
    using W = Wide<MODE>;
    CUtensorMap ma, mb;
    if (!md::make_map(&ma, w, kBf16, 2, d0, d1, a.E, 64, MODE == kNK ? kTileM : 64) ||
        !md::make_map(&mb, x, kBf16, 2, a.k, rows, 0, 64, 64))
        return MD_ERR_CUDA;
    a.row_tiles = md::ragged_most_tiles(rows, a.E, 256);
    a.subs = subs_for(a.row_tiles * ((a.n + W::kSub - 1) / W::kSub), 4);
    const int mt = (a.n + a.subs * W::kSub - 1) / (a.subs * W::kSub);
    a.mt = FastDiv((uint32_t)mt);
    if (a.row_tiles * mt > kMostTiles) return MD_ERR_UNSUPPORTED;
    static std::atomic<uint64_t> setup{0};
    return launch(k_expert_wide<MODE>, W::kThreads, kLaunchRegisters, W::smem(a.E), W::smem(MD_MAX_EXPERTS), setup, a.row_tiles * mt, 2, s, ma,
                  mb, mb, a);
}

// Which form: few, or wide (ragged_few has the rule).
bool few_rows(int64_t rows, int E, int64_t columns, int sub)
{
    const int path = md::expert_path();
    if (path != MD_EXPERT_AUTO) return path == MD_EXPERT_FEW;
    return md::ragged_few(rows, E, columns, sub, md::sm_count());
}

}  // namespace

extern "C" int md_expert_gemm(const void *x, int64_t rows, int K, const void *w, int E, int N, int w_layout,
                              const int32_t *expert_offsets, const int32_t *expert_counts, void *y,
                              int32_t *dev_status, void *stream)
{
    if (bad_sizes(rows, E, N, K) || (w_layout != MD_W_NK && w_layout != MD_W_KN)) return MD_ERR_ARG;
    if (!w || !md::aligned16(w) || !expert_offsets || !expert_counts) return MD_ERR_ARG;
    if (rows > 0 && (!x || !y || !md::aligned16(x) || !md::aligned16(y))) return MD_ERR_ARG;
    if (too_large(rows, E, N, K)) return MD_ERR_UNSUPPORTED;
    if (md::overlap(y, rows * N * 2, x, rows * K * 2) || md::overlap(y, rows * N * 2, w, (int64_t)E * N * K * 2)) return MD_ERR_ARG;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK || rows == 0) return rc;
    Args a = {};
    a.split = 1;
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.rows = rows;
    a.E = E;
    a.n = N;
    a.k = K;
    a.pitch = N;
    a.y = y;
    a.status = dev_status;
    a.polls = md::hook_poll_limit(INT64_MAX);
    if (w_layout == MD_W_NK)
        return few_rows(rows, E, N, Wide<kNK>::kSub) ? run_few<kNK>(x, w, rows, a, K, N, s)
                                                     : run_wide<kNK>(x, w, rows, a, K, N, s);
    return few_rows(rows, E, N, Wide<kKN>::kSub) ? run_few<kKN>(x, w, rows, a, N, K, s)
                                                 : run_wide<kKN>(x, w, rows, a, N, K, s);
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
    const int64_t wide = rows * F * 2, kept = rows * 2 * ((F + kBlock - 1) / kBlock);  // act and codes; scales
    const struct { const void *at; int64_t bytes; } in[2] = {{x, rows * K * 2}, {w, (int64_t)E * F * K * 4}};
    for (const auto &i : in)
        if (md::overlap(act, wide, i.at, i.bytes) || md::overlap(codes, wide, i.at, i.bytes) ||
            md::overlap(scales, kept, i.at, i.bytes))
            return MD_ERR_ARG;
    if (md::overlap(act, wide, codes, wide) || md::overlap(act, wide, scales, kept) || md::overlap(codes, wide, scales, kept))
        return MD_ERR_ARG;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK || rows == 0) return rc;
    Args a = {};
    a.split = 1;
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
    a.polls = md::hook_poll_limit(INT64_MAX);
    return few_rows(rows, E, F, Wide<kGated>::kSub) ? run_few<kGated>(x, w, rows, a, K, 2 * (int64_t)F, s)
                                                    : run_wide<kGated>(x, w, rows, a, K, 2 * (int64_t)F, s);
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
    const int size = out_type == MD_F32 ? 4 : 2;
    const int64_t bytes = (int64_t)E * N * K * size;
    if (md::overlap(dw, bytes, dy, rows * N * 2) || md::overlap(dw, bytes, x, rows * K * 2)) return MD_ERR_ARG;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK) return rc;
    if (rows == 0) {
        if (accumulate) return MD_OK;
        md::count_memsets(1);
        return cudaMemsetAsync(dw, 0, (size_t)bytes, s) == cudaSuccess ? MD_OK : MD_ERR_CUDA;
    }
    Args a = {};
    a.split = 1;
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.rows = rows;
    a.E = E;
    a.n = N;
    a.k = K;
    a.out_bf16 = out_type == MD_BF16;
    a.accumulate = accumulate != 0;
    a.status = dev_status;
    a.polls = md::hook_poll_limit(INT64_MAX);
    a.y = dw;
    using W = Wide<kWgrad>;
    CUtensorMap ma, mb, mo;
    if (!md::make_map(&ma, dy, kBf16, 2, N, rows, 0, 64, 64) || !md::make_map(&mb, x, kBf16, 2, K, rows, 0, 64, 64) ||
        !md::make_map(&mo, dw, a.out_bf16 ? kBf16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, size, K, N, E, 128 / size, 32))
        return MD_ERR_CUDA;
    const int64_t across = (K + 255) / 256;
    a.subs = subs_for(E * across * ((N + W::kSub - 1) / W::kSub), 8);
    const int64_t mt = (N + a.subs * W::kSub - 1) / (a.subs * W::kSub), tiles = E * across * mt;
    if (tiles > kMostTiles) return MD_ERR_UNSUPPORTED;
    a.mt = FastDiv((uint32_t)mt);
    a.per = FastDiv((uint32_t)(mt * across));
    static std::atomic<uint64_t> setup{0};
    return launch(k_expert_wide<kWgrad>, W::kThreads, kLaunchRegisters, W::smem(E), W::smem(MD_MAX_EXPERTS), setup, tiles, 2, s, ma, mb,
                  mo, a);
}
