// Attention of queries to an encoder's states of another length (cross
// attention): what the forward and backward kernels need around them when they
// run in their CROSS form.
//
//   fa_cross_combine_kernel  joins the parts of a forward whose key range was split;
//   fa_cross_prep_kernel     D_i = dO_i . O_i, L_i log2 e and the zeroed dQ sums;
//   fa_cross_dq_kernel       dQ = bf16(scale * sums), and dK, dV where their sums came in parts.
//
// The latter two are the backward's, over views of any strides.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "fa_bwd_kernel.cuh"
#include "fa_fwd_kernel.cuh"
#include "ptx.cuh"

namespace fa {
namespace cross {

constexpr int THREADS = 256;

// Place of query row `row` (b, head, i) of a view with strides sb, sh, sn.
struct Rows {
    int64_t sb, sh, sn;
    int heads, n;
    __device__ __forceinline__ int64_t at(int64_t row) const
    {
        const int64_t bh = row / n, b = bh / heads;
        return b * sb + (bh - b * heads) * sh + (row - bh * n) * sn;
    }
};

// A warp a row: out = sum_s w_s O_s / sum_s w_s with w_s = 2^(L_s - max L), over
// the parts that hold keys (the others were not written).  Lane l takes channels
// D/32 l and the next ones.
template <int D>
__global__ void __launch_bounds__(THREADS)
    fa_cross_combine_kernel(const float* __restrict__ part, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                            const int32_t* __restrict__ lens, const Rows view, int64_t rows, int nk, int splits, int d)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int b = (int)(row / ((int64_t)view.n * view.heads));
    const int tiles = (cross_length(lens, b, nk) + BN - 1) / BN;
    const float* const plse = part + (int64_t)splits * rows * D;
    constexpr int PER = D / 32;
    float mx = -INFINITY, l = 0.f, acc[PER] = {};
    auto first = [&](int s) { return (int)((int64_t)tiles * s / splits); };
    for (int s = lane; s < splits; s += 32)
        if (first(s + 1) > first(s)) mx = fmaxf(mx, plse[s * rows + row]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
    const float top = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        if (first(s + 1) == first(s)) continue;
        const float w = ptx::ex2(plse[s * rows + row] - top);
        const float* const f = part + (s * rows + row) * D + lane * PER;
        l += w;
        if constexpr (PER == 4) {
            const float4 v = *reinterpret_cast<const float4*>(f);
            acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
            acc[2] = fmaf(w, v.z, acc[2]), acc[3] = fmaf(w, v.w, acc[3]);
        } else {
            const float2 v = *reinterpret_cast<const float2*>(f);
            acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
        }
    }
    const float inv = l > 0.f || !(l == l) ? 1.0f / l : 0.f;
    __nv_bfloat16* const out = o + view.at(row) + lane * PER;
    if (lane * PER < d) {
        uint32_t w[PER / 2];
#pragma unroll
        for (int c = 0; c < PER / 2; ++c) w[c] = ptx::pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
        if constexpr (PER == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(out) = w[0];
    }
    if (lane == 0) lse[row] = l > 0.f || !(l == l) ? (mx + ptx::lg2(l)) * 0.69314718055994530942f : -INFINITY;
}

// As fa_bwd_prep_kernel, over views: rows i < np of every (b, head).
__global__ void __launch_bounds__(THREADS, 4)
    fa_cross_prep_kernel(const __nv_bfloat16* __restrict__ o, const Rows ov, const __nv_bfloat16* __restrict__ dout,
                         const Rows dv, const float* __restrict__ lse, float* __restrict__ lse2,
                         float* __restrict__ dsum, float* __restrict__ dq_acc, int np, int d, int dp, int64_t rows)
{
    constexpr int PER = bwd::PREP_ROWS;
    const int64_t row0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * PER;
    const int lane = threadIdx.x & 31;
    if (row0 >= rows) return;
    const int64_t bh = row0 / np;
    const int i0 = (int)(row0 - bh * np), n = ov.n;
    const int c = lane * 8;
    const int64_t b = bh / ov.heads, h = bh - b * ov.heads;
    const __nv_bfloat16* const po = o + b * ov.sb + h * ov.sh + i0 * ov.sn + c;
    const __nv_bfloat16* const pd = dout + b * dv.sb + h * dv.sh + i0 * dv.sn + c;
    uint4 x[PER], y[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        x[r] = y[r] = make_uint4(0u, 0u, 0u, 0u);
        if (i0 + r < n && c < d) {
            x[r] = *reinterpret_cast<const uint4*>(po + r * ov.sn);
            y[r] = *reinterpret_cast<const uint4*>(pd + r * dv.sn);
        }
    }
    float acc[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const uint32_t xw[4] = {x[r].x, x[r].y, x[r].z, x[r].w}, yw[4] = {y[r].x, y[r].y, y[r].z, y[r].w};
        acc[r] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 xf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xw[j]));
            const float2 yf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&yw[j]));
            acc[r] = fmaf(xf.x, yf.x, acc[r]);
            acc[r] = fmaf(xf.y, yf.y, acc[r]);
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], m);
    }
    if (lane < PER) {
        float v = acc[0];
#pragma unroll
        for (int r = 1; r < PER; ++r)
            if (lane == r) v = acc[r];
        const int i = i0 + lane;
        dsum[row0 + lane] = i < n ? v : 0.f;
        lse2[row0 + lane] = i < n ? lse[bh * n + i] * 1.4426950408889634074f : __int_as_float(0x7f800000);
    }
    float4* const z = reinterpret_cast<float4*>(dq_acc + row0 * dp);
    for (int k = lane; k < PER * dp / 4; k += 32) z[k] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Where the query blocks of a key block were cut into parts: their sums of dV and dK.
struct Parts {
    const float* part;  // dV, then dK: [part][b][kv head][key][dp]
    int parts;          // 1: none
    int64_t rows;       // b, kv head, key
    __nv_bfloat16 *dv, *dk;
    Rows vv, kv;
    const int32_t* lens;
};

// 8 elements a thread: those at src, times mul, to dst.
__device__ __forceinline__ void put8(__nv_bfloat16* dst, const float4 a, const float4 b, float mul)
{
    ptx::st_global_v4(dst, ptx::pack_bf16x2(a.x * mul, a.y * mul), ptx::pack_bf16x2(a.z * mul, a.w * mul),
                      ptx::pack_bf16x2(b.x * mul, b.y * mul), ptx::pack_bf16x2(b.z * mul, b.w * mul));
}

// As fa_bwd_dq_kernel, over a view.  With PARTS, dV's and dK's elements come behind
// dQ's: their parts are joined (in order, so that results repeat); rows behind the last
// key are zero.
template <bool PARTS>
__global__ void __launch_bounds__(THREADS)
    fa_cross_dq_kernel(const float* __restrict__ dq_acc, __nv_bfloat16* __restrict__ dq, const Rows view, int np, int d,
                       int dp, int64_t n8, float scale, const Parts x)
{
    int64_t e8 = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (e8 < n8) {
        const int64_t row = e8 / (d / 8);
        const int col = (int)(e8 - row * (d / 8)) * 8;
        const int64_t bh = row / view.n;
        const float4* const src = reinterpret_cast<const float4*>(dq_acc + (bh * np + (row - bh * view.n)) * dp + col);
        put8(dq + view.at(row) + col, src[0], src[1], scale);
    } else if (PARTS) {
        e8 -= n8;
        const int64_t line = e8 / (d / 8), which = line / x.rows, row = line - which * x.rows;
        if (which > 1) return;
        const int col = (int)(e8 - line * (d / 8)) * 8;
        const int64_t b = row / ((int64_t)x.kv.n * x.kv.heads), key = row % x.kv.n, step = x.rows * dp;
        const float* const src = x.part + which * x.parts * step + row * dp + col;
        const int parts = key < cross_length(x.lens, (int)b, x.kv.n) ? x.parts : 0;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float4 u = *reinterpret_cast<const float4*>(src + s * step), v = *reinterpret_cast<const float4*>(src + s * step + 4);
            lo.x += u.x, lo.y += u.y, lo.z += u.z, lo.w += u.w;
            hi.x += v.x, hi.y += v.y, hi.z += v.z, hi.w += v.w;
        }
        put8((which ? x.dk + x.kv.at(row) : x.dv + x.vv.at(row)) + col, lo, hi, which ? scale : 1.0f);
    }
}

}  // namespace cross
}  // namespace fa
