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

unsigned grid_for(int64_t items, int per_block, int per_sm)
{
    const int64_t blocks = (items + per_block - 1) / per_block, cap = (int64_t)md::sm_count() * per_sm;
    return (unsigned)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
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
__global__ void __launch_bounds__(kThreads)
    k_gated_backward(const uint4 *__restrict__ da, const uint8_t *__restrict__ codes,
                     const uint8_t *__restrict__ scales, int64_t rows, int F, uint4 *__restrict__ dh,
                     uint4 *__restrict__ act)
{
    const int C = F / 8, blocks = (F + kBlock - 1) / kBlock;
    const int64_t n = rows * C, step = (int64_t)gridDim.x * kThreads;
    // two pieces of 8 columns at a time: all their loads are on the way before the first is used
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < n; i0 += 2 * step) {
        int64_t r[2];
        int c[2];
        uint4 d4[2];
        uint2 cg[2], cu[2];
        uint32_t sg[2], su[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t i = i0 + q * step < n ? i0 + q * step : i0;
            r[q] = i / C;
            c[q] = (int)(i - r[q] * C);
            const uint8_t *cr = codes + r[q] * 2 * F + c[q] * 8, *sr = scales + r[q] * 2 * blocks + c[q] * 8 / kBlock;
            d4[q] = md::ld_stream(da + i);
            cg[q] = __ldg(reinterpret_cast<const uint2 *>(cr));
            cu[q] = __ldg(reinterpret_cast<const uint2 *>(cr + F));
            sg[q] = __ldg(sr);
            su[q] = __ldg(sr + blocks);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (i0 + q * step >= n) break;
            float g[8], u[8];
            from_e4m3(cg[q].x, scale_of(sg[q]), g);
            from_e4m3(cg[q].y, scale_of(sg[q]), g + 4);
            from_e4m3(cu[q].x, scale_of(su[q]), u);
            from_e4m3(cu[q].y, scale_of(su[q]), u + 4);
            const uint32_t dw[4] = {d4[q].x, d4[q].y, d4[q].z, d4[q].w};
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
            uint4 *to = dh + r[q] * 2 * C + c[q];
            md::st_stream(to, make_uint4(og[0], og[1], og[2], og[3]));
            md::st_stream(to + C, make_uint4(ou[0], ou[1], ou[2], ou[3]));
            if (act) md::st_stream(act + r[q] * C + c[q], make_uint4(oa[0], oa[1], oa[2], oa[3]));
        }
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

// One warp per token.  The token's dout row comes from HBM once (slots after
// the first find it in L1); each slot's y row is read and its dy row written
// in the same pass.  dw is summed in float32: a fixed order per lane, then a
// fixed butterfly, so it does not vary from run to run.
template <bool DOT>
__global__ void __launch_bounds__(kThreads)
    k_combine_backward(const uint4 *__restrict__ dout, const uint4 *__restrict__ y, int64_t y_rows,
                       const int32_t *__restrict__ assign_row, const float *__restrict__ w, int64_t T, int k,
                       int C, uint4 *__restrict__ dy, float *__restrict__ dw, int32_t *status)
{
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < T; t += nw) {
        int rl = -1;
        float wl = 0.f;
        if (lane < k) {
            rl = __ldg(assign_row + t * k + lane);
            wl = __ldg(w + t * k + lane);
            if (rl < 0 || rl >= y_rows) {
                md::report(status, MD_ERR_DATA);
                rl = -1;
            }
        }
        float mine = 0.f;
        for (int j = 0; j < k; ++j) {
            const int r = __shfl_sync(0xffffffffu, rl, j);
            const float g = __shfl_sync(0xffffffffu, wl, j);
            if (r < 0) continue;
            const uint4 *src = dout + t * C, *yr = y + (int64_t)r * C;
            uint4 *dst = dy + (int64_t)r * C;
            float acc[U] = {};
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
            if (DOT) {
                float s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == j) mine = s;
            }
        }
        if (DOT && lane < k) dw[t * k + lane] = mine;
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
    cudaStream_t s = md::as_stream(stream);
    k_gated_backward<<<grid_for(rows * (F / 8), kThreads, 8), kThreads, 0, s>>>(
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
    cudaStream_t s = md::as_stream(stream);
    const int rc = md::clear_status(dev_status, s);
    if (rc != MD_OK || T == 0) return rc;
    const unsigned grid = grid_for(T, kThreads / 32, 8);
    if (dw)
        k_combine_backward<true><<<grid, kThreads, 0, s>>>(
            static_cast<const uint4 *>(dout), static_cast<const uint4 *>(y), y_rows, assign_row, topk_w, T, k, H / 8,
            static_cast<uint4 *>(dy), dw, dev_status);
    else
        k_combine_backward<false><<<grid, kThreads, 0, s>>>(static_cast<const uint4 *>(dout), nullptr, y_rows,
                                                            assign_row, topk_w, T, k, H / 8,
                                                            static_cast<uint4 *>(dy), nullptr, dev_status);
    md::count_launches(1);
    return md::launch_status();
}
