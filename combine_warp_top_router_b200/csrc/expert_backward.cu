// expert_backward.cu -- the row-wise gradients around the expert products:
// md_expert_gated_backward (from the 8-bit checkpoint) and md_combine_backward.
//
// Both read every input once and write every output once, in 16-byte pieces
// (the checkpoint's codes in 8-byte ones); they are bound by HBM.
#include <cuda_fp16.h>

#include "activation.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 32;  // columns that share a scale

// a thread or warp for each item, as far as a grid reaches
unsigned grid_for(int64_t items, int per_block)
{
    const int64_t blocks = (items + per_block - 1) / per_block;
    return (unsigned)(blocks < 1 ? 1 : blocks < INT32_MAX ? blocks : INT32_MAX);
}

// four e4m3 codes -> floats, exact
__device__ __forceinline__ void from_e4m3(uint32_t w, float scale, float *v)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t f16x2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f16x2) : "h"((uint16_t)(w >> (16 * h))));
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&f16x2));
        v[2 * h] = f.x * scale;
        v[2 * h + 1] = f.y * scale;
    }
}

// 2^(s - 127), s = 0..254 (s = 0: the subnormal 2^-127)
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x00400000u); }

// With s = 1 / (1 + exp(-g)):  dg = da u s (1 + g (1 - s)), du = da g s,
// a = g s u.  Float32 throughout, one rounding to bf16 per output.
// One piece of 8 columns to a thread, and as many threads as pieces: kept threads
// with a loop ran 14% slower, two pieces at a time as fast.
// 131072 rows of 1024: 228 us, 5.9 TB/s (60% of it writes).
__global__ void __launch_bounds__(kThreads)
    k_gated_backward(const uint4 *__restrict__ da, const uint8_t *__restrict__ codes,
                     const uint8_t *__restrict__ scales, int64_t rows, int F, uint4 *__restrict__ dh,
                     uint4 *__restrict__ act)
{
    const int C = F / 8, blocks = (F + kBlock - 1) / kBlock;
    const int64_t n = rows * C;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = n <= INT32_MAX ? (int32_t)i / C : i / C;
        const int c = (int)(i - r * C);
        const uint8_t *cr = codes + r * 2 * F + c * 8, *sr = scales + r * 2 * blocks + c * 8 / kBlock;
        const uint4 d4 = md::ld_stream(da + i);
        const uint2 cg = __ldg(reinterpret_cast<const uint2 *>(cr)), cu = __ldg(reinterpret_cast<const uint2 *>(cr + F));
        const float sg = scale_of(__ldg(sr)), su = scale_of(__ldg(sr + blocks));
        float g[8], u[8];
        from_e4m3(cg.x, sg, g);
        from_e4m3(cg.y, sg, g + 4);
        from_e4m3(cu.x, su, u);
        from_e4m3(cu.y, su, u + 4);
        const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
        uint32_t og[4], ou[4], oa[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            float vg[2], vu[2], va[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float d = h ? md::bf16hi(dw[p]) : md::bf16lo(dw[p]);
                const float x = g[2 * p + h], y = u[2 * p + h];
                const float s = md::sigmoid(x);
                vg[h] = d * y * s * (1.0f + x * (1.0f - s));
                vu[h] = d * x * s;
                va[h] = x * s * y;
            }
            og[p] = md::pack_bf16x2(vg[0], vg[1]);
            ou[p] = md::pack_bf16x2(vu[0], vu[1]);
            oa[p] = md::pack_bf16x2(va[0], va[1]);
        }
        uint4 *to = dh + r * 2 * C + c;
        md::st_stream(to, make_uint4(og[0], og[1], og[2], og[3]));
        md::st_stream(to + C, make_uint4(ou[0], ou[1], ou[2], ou[3]));
        if (act) md::st_stream(act + i, make_uint4(oa[0], oa[1], oa[2], oa[3]));
    }
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t v, float w)
{
    return md::pack_bf16x2(md::bf16lo(v) * w, md::bf16hi(v) * w);
}

__device__ __forceinline__ void dot_pair(float &acc, uint32_t a, uint32_t b)
{
    acc = fmaf(md::bf16lo(a), md::bf16lo(b), acc);
    acc = fmaf(md::bf16hi(a), md::bf16hi(b), acc);
}

// One warp per slot (t, j): its y row is read and its dy row written in one pass,
// against the token's dout row, which the warps of a token's slots find in L1 or L2 after
// the first.  A lane has 4 pieces of 16 bytes of each row on the way (8: 5% slower), and
// warps are not kept for further slots as long as the grid reaches: with a token's
// slots in a row in one kept warp it ran 10% slower, and at 509 tokens, where
// that left SMs idle, at half the speed.  dw is summed in float32: a fixed order
// per lane, then a fixed butterfly, so it does not vary from run to run.
// 32768 tokens x 6 slots of 4096: 534 us, 6.5 TB/s.
template <bool DOT>
__global__ void __launch_bounds__(kThreads)
    k_combine_backward(const uint4 *__restrict__ dout, const uint4 *__restrict__ y, int64_t y_rows,
                       const int32_t *__restrict__ assign_row, const float *__restrict__ w, int64_t slots, int k,
                       int C, uint4 *__restrict__ dy, float *__restrict__ dw, int32_t *status)
{
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t s = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); s < slots; s += nw) {
        const int r = __ldg(assign_row + s);
        const float g = __ldg(w + s);
        float acc[U] = {};
        if (r >= 0 && r < y_rows) {
            const uint4 *src = dout + s / k * C, *yr = y + (int64_t)r * C;
            uint4 *dst = dy + (int64_t)r * C;
            for (int c0 = lane; c0 < C; c0 += 32 * U) {
                uint4 d[U], v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + 32 * u;
                    d[u] = c < C ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                    if (DOT) v[u] = c < C ? md::ld_stream(yr + c) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + 32 * u;
                    if (DOT) {
                        dot_pair(acc[u], d[u].x, v[u].x);
                        dot_pair(acc[u], d[u].y, v[u].y);
                        dot_pair(acc[u], d[u].z, v[u].z);
                        dot_pair(acc[u], d[u].w, v[u].w);
                    }
                    if (c < C)
                        md::st_stream(dst + c, make_uint4(scale_pair(d[u].x, g), scale_pair(d[u].y, g),
                                                          scale_pair(d[u].z, g), scale_pair(d[u].w, g)));
                }
            }
        } else if (lane == 0) {
            md::report(status, MD_ERR_DATA);
        }
        if (DOT) {
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) sum += acc[u];
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) dw[s] = sum;
        }
    }
}

}  // namespace

extern "C" int md_expert_gated_backward(const void *da, const void *codes, const uint8_t *scales, int64_t rows,
                                        int F, void *dh, void *act, void *stream)
{
    if (rows < 0 || F < 8 || F % 8 != 0) return MD_ERR_ARG;
    if (rows == 0) return MD_OK;
    if (!da || !codes || !scales || !dh || !md::aligned16(da) || !md::aligned16(codes) || !md::aligned16(dh) ||
        !md::aligned16(act))
        return MD_ERR_ARG;
    const int64_t n = rows * F * 2;  // bytes of da, of the codes, of act, and half of dh's
    const int64_t m = rows * 2 * ((F + kBlock - 1) / kBlock);
    if (md::overlap(dh, 2 * n, da, n) || md::overlap(dh, 2 * n, codes, n) || md::overlap(dh, 2 * n, scales, m) ||
        md::overlap(act, n, da, n) || md::overlap(act, n, codes, n) || md::overlap(act, n, scales, m) ||
        md::overlap(dh, 2 * n, act, n))
        return MD_ERR_ARG;
    cudaStream_t s = md::as_stream(stream);
    k_gated_backward<<<grid_for(rows * (F / 8), kThreads), kThreads, 0, s>>>(
        static_cast<const uint4 *>(da), static_cast<const uint8_t *>(codes), scales, rows, F,
        static_cast<uint4 *>(dh), static_cast<uint4 *>(act));
    md::count_launches(1);
    return md::launch_status();
}

extern "C" int md_combine_backward(const void *dout, const void *y, int64_t y_rows, const int32_t *assign_row,
                                   const float *topk_w, int64_t T, int k, int H, void *dy, float *dw,
                                   int32_t *dev_status, void *stream)
{
    if (T < 0 || H < 8 || H % 8 != 0 || k < 1 || k > MD_MAX_TOPK || y_rows < 0) return MD_ERR_ARG;
    if (T > 0 && (!dout || !md::aligned16(dout) || !assign_row || !topk_w)) return MD_ERR_ARG;
    if (y_rows > 0 && (!dy || !md::aligned16(dy))) return MD_ERR_ARG;
    if (dw && y_rows > 0 && (!y || !md::aligned16(y))) return MD_ERR_ARG;
    const int64_t row = (int64_t)H * 2;
    if (T > 0 && (md::overlap(dy, y_rows * row, dout, T * row) || (dw && md::overlap(dy, y_rows * row, y, y_rows * row))))
        return MD_ERR_ARG;
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK || T == 0) return rc;
    const unsigned grid = grid_for(T * k, kThreads / 32);
    if (dw)
        k_combine_backward<true><<<grid, kThreads, 0, s>>>(
            static_cast<const uint4 *>(dout), static_cast<const uint4 *>(y), y_rows, assign_row, topk_w, T * k, k, H / 8,
            static_cast<uint4 *>(dy), dw, dev_status);
    else
        k_combine_backward<false><<<grid, kThreads, 0, s>>>(static_cast<const uint4 *>(dout), nullptr, y_rows,
                                                            assign_row, topk_w, T * k, k, H / 8,
                                                            static_cast<uint4 *>(dy), nullptr, dev_status);
    md::count_launches(1);
    return md::launch_status();
}
