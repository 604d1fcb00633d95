// Rotary positions for sm_103a: the channels of a query or key row are taken
// in pairs (a, b), and pair i of the row at position t is turned by the angle
// t * f_i:
//
//   a' = factor * (a cos - b sin),   b' = factor * (b cos + a sin)
//
// Pair i is channels (i, i + rot/2) in the half layout and (2i, 2i + 1) in the
// interleaved one; channels from rot on pass through.  The map is linear, so
// its gradient is the same map with the angle negated (the transpose).
//
// Angles.  f_i comes as turns per position in 64-bit fixed point (units of
// 2^-64 of a turn), so t * f_i modulo one turn is the low 64 bits of one
// integer product, exact for any position (an fp32 product t * f_i is off by 0.03
// rad at t = 10^6); what remains is t times the word's own rounding.  The product
// is taken to the nearest quarter turn and its distance from there becomes fp32,
// so that cosine and sine come out to 2^-22 of themselves however small.
//
// The work is bound by memory: 4 bytes moved per element against 3 flops.  A
// thread owns one unit of channels (two 16-byte vectors holding 8 whole
// pairs) of one position and U = 4 heads, whose loads are in flight while it
// computes the 8 angles that they share.  Queries and keys go in one launch.
// Measured at B8 H32 + 32 N4096 d128 (a forward and a gradient, 2.15 GB): 318 us,
// 6744 GB/s, 1.00 of the measured copy bandwidth.  What brought it there: 4
// blocks an SM instead of 3 (349 -> 328 us; 5 spill, 409 us) and, for results
// larger than L2, streaming stores (328 -> 318 us); with 2 heads in flight 404
// us, with the angles computed before the loads 383 us.  Where the results go is
// worked out after the angles: 64 registers hold no more beside the loads in flight
// (worked out before, 19 words spill: 328 us).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fa {
namespace rope {

constexpr int THREADS = 256;
constexpr int U = 4;  // heads in flight per thread

struct View {
    __nv_bfloat16* p;
    int64_t sb, sh, sn;  // elements between batches, heads, positions
};

struct Params {
    View in[2], out[2];   // queries, keys
    int heads[2];
    const uint64_t* freqs;
    const void* positions;  // (B, N) int32 or int64, or null
    int64_t pos_sb;         // elements between the batches' positions (0: shared)
    const int32_t* lens;    // (B), or null
    int wide;               // positions are int64
    int64_t n;
    int d, rot, interleaved;
    int tiles;              // position tiles of a sequence
    int head_tiles;         // groups of U * blockDim.z heads
    int stream;
    float factor;
    float sign;             // -1 turns the angle round (gradient)
};

__device__ __forceinline__ int64_t position_of(const Params& p, int b, int64_t i)
{
    if (p.positions) {
        const int64_t at = b * p.pos_sb + i;
        return p.wide ? static_cast<const int64_t*>(p.positions)[at] : (int64_t) static_cast<const int32_t*>(p.positions)[at];
    }
    return (p.lens ? (int64_t)p.lens[b] - p.n : 0) + i;
}

// The angle of a pair, from its nearest quarter turn: z in [-1, 1], in units of an
// eighth of a turn, to fp32's rounding of itself, and the quarter.
__device__ __forceinline__ void angle(int64_t pos, uint64_t freq, float& z, uint32_t& quarter)
{
    const uint64_t a = (uint64_t)pos * freq;
    z = (float)(int64_t)(a << 2) * 0x1p-63f;
    quarter = ((uint32_t)(a >> 32) + (1u << 29)) >> 30;
}

// Cosine and sine of an angle z of at most an eighth of a turn, by their power
// series up to z^8 and z^9, which leave out at most 2^-25 and 2^-28 of the value: good
// to fp32's rounding of themselves, however small they are.  (The special-function
// unit's are good to 2^-21 of 1, which was 1 % of a slow pair's sine.)
constexpr double EIGHTH = 0.78539816339744830962, E2 = EIGHTH * EIGHTH, E4 = E2 * E2;
__device__ __forceinline__ void cos_sin(float z, float& c, float& s)
{
    const float w = z * z;
    c = fmaf(w, (float)(E4 * E4 / 40320), (float)(-E4 * E2 / 720));
    s = fmaf(w, (float)(EIGHTH * E4 * E4 / 362880), (float)(-EIGHTH * E4 * E2 / 5040));
    c = fmaf(w, c, (float)(E4 / 24));
    s = fmaf(w, s, (float)(EIGHTH * E4 / 120));
    c = fmaf(w, c, (float)(-E2 / 2));
    s = fmaf(w, s, (float)(-EIGHTH * E2 / 6));
    c = fmaf(w, c, 1.0f);
    s = z * fmaf(w, s, (float)EIGHTH);
}

// cos and sin of one pair's angle, scaled: those of its distance from the nearest
// quarter turn, then turned by the quarters: (c, s), (-s, c), (-c, -s), (s, -c).
__device__ __forceinline__ void turn(int64_t pos, uint64_t freq, float factor, float signed_factor, float& c, float& s)
{
    float z, x, y;
    uint32_t quarter;
    angle(pos, freq, z, quarter);
    cos_sin(z, x, y);
    c = (quarter & 1u ? y : x) * __uint_as_float(__float_as_uint(factor) ^ ((quarter + 1u) & 2u) << 30);
    s = (quarter & 1u ? x : y) * __uint_as_float(__float_as_uint(signed_factor) ^ (quarter & 2u) << 30);
}

// W elements.  Not .nc: an output may be its input.
template <int W, int N>
__device__ __forceinline__ void ld(uint32_t (&r)[N], const __nv_bfloat16* p)
{
    if constexpr (W == 8)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
    else if constexpr (W == 2)
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    else
        r[0] = *reinterpret_cast<const unsigned short*>(p);
}

// stream: the results are larger than L2 and will not be found there by the next reader.
template <int W, int N>
__device__ __forceinline__ void st(__nv_bfloat16* p, const uint32_t (&r)[N], int stream)
{
    if constexpr (W == 8) {
        if (stream)
            asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
        else
            ptx::st_global_v4(p, r[0], r[1], r[2], r[3]);
    } else if constexpr (W == 2) {
        *reinterpret_cast<uint32_t*>(p) = r[0];
    } else {
        *reinterpret_cast<unsigned short*>(p) = (unsigned short)r[0];
    }
}

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Pairs split over two words: word a holds two pairs' first channels, b their
// second ones; c, s: the two pairs' cosines and sines.
__device__ __forceinline__ void turn_half(uint32_t& a, uint32_t& b, uint64_t c, uint64_t s, uint64_t minus_s)
{
    const uint64_t x = ptx::f2_pack(lo(a), hi(a)), y = ptx::f2_pack(lo(b), hi(b));
    float u, v;
    ptx::f2_unpack(ptx::f2_fma(y, minus_s, ptx::f2_mul(x, c)), u, v);
    a = ptx::pack_bf16x2(u, v);
    ptx::f2_unpack(ptx::f2_fma(x, s, ptx::f2_mul(y, c)), u, v);
    b = ptx::pack_bf16x2(u, v);
}

// A pair within one word.
__device__ __forceinline__ void turn_word(uint32_t& w, float c, float s)
{
    const float a = lo(w), b = hi(w);
    w = ptx::pack_bf16x2(a * c - b * s, b * c + a * s);
}

// W = 8: units of two 16-byte vectors (every vector wholly turned or wholly
// passed through, rows and strides 16-byte aligned).  W = 2 and 1 do the same in
// two 4-byte and two 2-byte accesses, for turned parts and strides that 16
// bytes do not divide.  Block (units, positions, head lanes).
template <int W>
__global__ void __launch_bounds__(THREADS, 4) fa_rope_kernel(const Params p)
{
    ptx::griddep_wait();  // a programmatic dependent: the inputs are complete
    ptx::griddep_launch_dependents();
    unsigned blk = blockIdx.x;
    const int ht = blk % p.head_tiles;
    blk /= p.head_tiles;
    const int64_t i = (int64_t)(blk % p.tiles) * blockDim.y + threadIdx.y;
    const int b = blk / p.tiles;
    if (i >= p.n) return;
    const int u = threadIdx.x;

    // The unit's two places (channels) and its pairs' first index; pass: not turned.
    const int turned = p.rot / (2 * W);  // units of whole pairs (interleaved: maybe one half unit more)
    int ca, cb, f0;
    bool pass_a = false, pass_b = false;
    if (!p.interleaved && u < turned) {
        ca = u * W;
        cb = p.rot / 2 + u * W;
        f0 = u * W;
    } else {
        ca = u * 2 * W;
        cb = ca + W;
        f0 = u * W;
        pass_a = ca >= p.rot;
        pass_b = cb >= p.rot;
    }
    const bool have_b = cb < p.d;

    // The vectors of the thread's heads, in flight while the angles are computed.
    constexpr int WORDS = W / 2 > 0 ? W / 2 : 1;
    uint32_t va[U][WORDS], vb[U][WORDS];
#pragma unroll
    for (int e = 0; e < U; ++e) {
        const int h = (ht * U + e) * (int)blockDim.z + threadIdx.z;
        if (h >= p.heads[0] + p.heads[1]) continue;
        const int t = h >= p.heads[0];
        const int64_t hl = t ? h - p.heads[0] : h;
        const __nv_bfloat16* const src = p.in[t].p + b * p.in[t].sb + hl * p.in[t].sh + i * p.in[t].sn;
        ld<W>(va[e], src + ca);
        if (have_b) ld<W>(vb[e], src + cb);
    }
    const int64_t pos = position_of(p, b, i);
    float c[W], s[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
        if (f0 + e < p.rot / 2 && !pass_a) turn(pos, p.freqs[f0 + e], p.factor, p.factor * p.sign, c[e], s[e]);
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
        const int h = (ht * U + e) * (int)blockDim.z + threadIdx.z;
        if (h >= p.heads[0] + p.heads[1]) continue;
        const int t = h >= p.heads[0];
        const int64_t hl = t ? h - p.heads[0] : h;
        __nv_bfloat16* const dst = p.out[t].p + b * p.out[t].sb + hl * p.out[t].sh + i * p.out[t].sn;
        if constexpr (W == 1) {
            if (!pass_a) {
                const float a = lo(va[e][0]), bb = lo(vb[e][0]);
                va[e][0] = ptx::pack_bf16x2(a * c[0] - bb * s[0], 0.f);
                vb[e][0] = ptx::pack_bf16x2(bb * c[0] + a * s[0], 0.f);
            }
        } else if (!p.interleaved) {  // pairs lie across the two places
            if (!pass_a) {
#pragma unroll
                for (int k = 0; k < WORDS; ++k)
                    turn_half(va[e][k], vb[e][k], ptx::f2_pack(c[2 * k], c[2 * k + 1]), ptx::f2_pack(s[2 * k], s[2 * k + 1]),
                              ptx::f2_pack(-s[2 * k], -s[2 * k + 1]));
            }
        } else {
#pragma unroll
            for (int k = 0; k < WORDS; ++k) {
                if (!pass_a) turn_word(va[e][k], c[k], s[k]);
                if (!pass_b) turn_word(vb[e][k], c[WORDS + k], s[WORDS + k]);
            }
        }
        st<W>(dst + ca, va[e], p.stream);
        if (have_b) st<W>(dst + cb, vb[e], p.stream);
    }
}

}  // namespace rope
}  // namespace fa
