// A paged key/value cache held in 4 bits, for decode on sm_103a: rows are
// appended and read back, and a few query rows attend to it.
//
// A stored value is  e2m1 * e4m3 * scale:  a sign, two exponent bits and one
// mantissa bit a value (0, .5, 1, 1.5, 2, 3, 4, 6), one e4m3 scale for 16
// channels of a row and one fp32 scale a tensor.  That is 9/16 byte a value
// against bf16's 2, and decode, bound by reading the cache, can run 3.6 times
// as fast.  The product e2m1 * e4m3 has at most 6 significant bits and lies
// between 2^-10 and 2688, so it is exact in fp16: the tensor cores' operands
// are the stored values, not roundings of them.  (Measured: 2.9 times the bf16
// cache's speed at 8 x 32 heads x 32768 keys.)
//
// A page holds PAGE = 64 keys of one kv head in one block of 72 * D bytes,
// D = 64 or 128 stored channels (smaller head sizes are padded with zeros).
// Rows are laid out so that a lane's share of a tensor-core operand is 16
// consecutive bytes (8 at D = 64), neighbouring lanes' shares adjoin, and one
// cvt turns a byte into a register of the operand:
//   K codes   at 0:     byte x*D/2 + c/2 of key x, low nibble the even channel;
//   K scales  at 32*D:  byte ((x%8)*4 + b/p)*8*p + (x/8)*p + b%p of channel
//                       block b, p = D/64 (a lane's 8 keys are together);
//   V codes   at 36*D:  byte (x/2)*D + c, low nibble the even key (the
//                       contraction over keys wants pairs of keys);
//   V scales  at 68*D:  byte (((x/2)%4)*D/16 + b)*16 + (x/8)*2 + x%2.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fa {

constexpr uint32_t STATUS_BAD_PAGE = 4u;  // a page table entry outside the pool: its keys were skipped

namespace qc {

constexpr int PAGE = 64;
constexpr int MAX_B = 2048;   // sequences of a call (their page counts' prefix sums sit in shared memory)
constexpr int MAX_NQ = 8;
constexpr float LN2 = 0.69314718055994530942f;

template <int D>
struct Block {
    static_assert(D == 64 || D == 128, "stored channels");
    static constexpr int P = D / 64;             // channel blocks per lane of a key row
    static constexpr int NB = D / 16;            // channel blocks
    static constexpr int KS = 32 * D, VC = 36 * D, VS = 68 * D, BYTES = 72 * D;
    __host__ __device__ static constexpr int kcode(int x) { return x * (D / 2); }
    __host__ __device__ static constexpr int kscale(int x, int b)
    {
        return KS + ((x % 8) * 4 + b / P) * 8 * P + (x / 8) * P + b % P;
    }
    __host__ __device__ static constexpr int vcode(int x) { return VC + (x / 2) * D; }
    __host__ __device__ static constexpr int vscale(int x, int b)
    {
        return VS + (((x / 2) % 4) * NB + b) * 16 + (x / 8) * 2 + x % 2;
    }
};

// Two e2m1 values (byte `i` of w, low nibble first) as exact fp16.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t w)
{
    uint32_t r;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Two e4m3 values as exact fp16.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two_bytes)
{
    uint32_t r;
    const uint16_t h = (uint16_t)two_bytes;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What packing (lo, hi) as fp16 left of them, as fp16.
__device__ __forceinline__ uint32_t rest_h2(float lo, float hi, uint32_t packed)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
    return pack_h2(lo - f.x, hi - f.y);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// d += A (16 x 16, rows) * B (16 x 8, columns), fp16 operands, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// As mma from zero sums.
__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ----------------------------------------------------------------- rounding

// Scales for two blocks of 16 channels from their largest magnitudes:
// amax / (6 scale) in e4m3, to nearest (halves to even), at most 448.  Returns
// their bytes, lo first.  The quotient (by a reciprocal, within 2^-23) is rounded to
// 17 bits first, which brings one beside a half (5 bits) onto it.  Where the scale is
// a power of two (POW2) that moves no other across a half: the quotient of bf16's 8-bit
// significand that is not half way differs from there by 2^-8 of itself.  With
// any other scale it is then moved by a last place to the side that the remainder
// 6 * quotient * scale - amax tells: six halves are exact, and the sign of a fused
// multiply-add's result is the exact one's, so only what is half way stays there.
template <bool POW2>
__device__ __forceinline__ uint32_t scale_bytes(float amax_lo, float amax_hi, float inv_six, float scale)
{
    auto quotient = [&](float amax) {
        const uint32_t q = (__float_as_uint(amax * inv_six) + 0x40u) & 0xFFFFFF80u;
        if constexpr (POW2) return __uint_as_float(q);
        const float left = fmaf(6.0f * __uint_as_float(q), scale, -amax);
        return __uint_as_float(left > 0.f ? q - 1u : left < 0.f ? q + 1u : q);
    };
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(quotient(amax_hi)), "f"(quotient(amax_lo)));
    return r;
}

__device__ __forceinline__ float scale_value(uint32_t byte)
{
    const uint32_t h = e4m3x2(byte & 0xFFu);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

// The reciprocal of a block's scale, to 2^-23 (0 for a scale of 0).
__device__ __forceinline__ float reciprocal(float s)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s > 0.f ? r : 0.f;
}

// x * y + 1/2, held within 0 and 1 (0 for NaN).
__device__ __forceinline__ float half_more_saturated(float x, float y)
{
    float r;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(0.5f));
    return r;
}

// Two quotients x / (e4m3 * scale) as e2m1, to nearest, halves to even,
// magnitudes above 6 to 6: the first in the low nibble.  x, the reciprocals inv of
// e4m3 * scale and the e4m3 values, negated, come as pairs.  A product with a
// reciprocal lies up to 2^-19 off a quotient that is half way between two codes; adding
// and subtracting 1.5 * 2^9 rounds to a multiple of 2^-14 first, which brings it back.
// Where the scale is a power of two (POW2) bf16 inputs meet exact halves often, and
// a quotient of an 8-bit and a 4-bit significand that is not half way differs from
// there by 2^-10 at least, so nothing else is moved.  With any other scale quotients
// lie as near to a half as they like: the rounded quotient is moved off by 2^-15, half
// way to the next multiple, to the side that the sign of x - quotient * e4m3 * scale
// tells (exact where the quotient is a half: 7 bits before the fused multiply-add).
template <bool POW2>
__device__ __forceinline__ uint32_t codes2(uint64_t x, uint64_t inv, uint64_t minus_e4m3, float scale)
{
    constexpr float C = 768.0f, FAR = 0x1p127f, STEP = 0x1p-15f;
    uint64_t q = ptx::f2_add(ptx::f2_fma(x, inv, ptx::f2_pack(C, C)), ptx::f2_pack(-C, -C));
    float a, b;
    if constexpr (!POW2) {
        ptx::f2_unpack(ptx::f2_fma(ptx::f2_mul(q, minus_e4m3), ptx::f2_pack(scale, scale), x), a, b);
        const uint64_t side = ptx::f2_pack(half_more_saturated(a, FAR), half_more_saturated(b, FAR));  // 0, 1/2 or 1
        q = ptx::f2_fma(side, ptx::f2_pack(2 * STEP, 2 * STEP), ptx::f2_add(q, ptx::f2_pack(-STEP, -STEP)));
    }
    ptx::f2_unpack(q, a, b);
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b32 %0, {t, t, t, t};\n\t}" : "=r"(r) : "f"(b), "f"(a));
    return r & 0xFFu;
}

__device__ __forceinline__ void unpack8(const uint4 w, float* f)
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

// ------------------------------------------------------------ append, read

struct RowParams {
    const __nv_bfloat16 *k, *v;    // append: new rows, (B, Hkv, N, d) by strides
    __nv_bfloat16 *ko, *vo;        // read: contiguous (B, Hkv, N, d)
    int64_t ksb, ksh, ksn, vsb, vsh, vsn;
    uint8_t* pool;
    const int32_t *table, *lens;
    int64_t n;
    int hkv, d, max_pages, num_pages;
    int newest;                    // row i is position lens - N + i (else i)
    float k_scale, v_scale, k_inv_six, v_inv_six;  // 1 / (6 scale)
};

// The 16 channels of block b of row p (d of them exist), zeros past d or when !have.
struct Raw16 {
    uint4 w0, w1;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int b, int d, bool have)
    {
        w0 = w1 = make_uint4(0, 0, 0, 0);
        if (have && b * 16 < d) w0 = __ldg(reinterpret_cast<const uint4*>(p + b * 16));
        if (have && b * 16 + 8 < d) w1 = __ldg(reinterpret_cast<const uint4*>(p + b * 16 + 8));
    }
    __device__ __forceinline__ void unpack(float (&f)[16]) const
    {
        unpack8(w0, f);
        unpack8(w1, f + 8);
    }
    // The largest magnitude (NaN does not count).
    __device__ __forceinline__ float amax() const
    {
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
};

// The page of position x of sequence b, or -1 (and the status bit).
__device__ __forceinline__ int page_of(const int32_t* table, int max_pages, int num_pages, int b, int slot)
{
    int id = -1;
    if (slot < max_pages) id = table[(int64_t)b * max_pages + slot];
    return id >= 0 && id < num_pages ? id : -1;
}

constexpr int ROW_THREADS = 256;

// Append: block (tile, kv head, sequence) writes one page's share of the new
// rows.  New keys are positions lens - N .. lens - 1; rows of negative
// position are padding and go nowhere.  A byte of V holds two keys: where
// only one of them is new, the other nibble is kept.  One block writes all
// of a page's new rows, so no two blocks share a byte.
//
// Bound by memory for prompts (4d bytes read and 9d/8 written a key), by its
// launch for single keys.  Appending and reading back 4 x 8 heads x up to 4096
// keys at d = 128: 24.8 us, about half of it here; 64 x 8 heads x 1 key: 6.2 us.
// Appending 4 x 8 x 4096 keys alone: 17.4 us, 0.73 of the measured copy bandwidth;
// what is between is the rounding's integer and conversion instructions (that
// pipe is 0.63 busy).
template <int D, bool POW2>
__global__ void __launch_bounds__(ROW_THREADS) fa_qcache_append_kernel(const RowParams p)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    using L = Block<D>;
    const int b = blockIdx.z, h = blockIdx.y;
    const int64_t len = min((int64_t)max(p.lens[b], 0), (int64_t)p.max_pages * PAGE);
    const int64_t first = max((int64_t)p.lens[b] - p.n, (int64_t)0);  // first new position
    const int64_t shift = p.n - p.lens[b];                           // row of position x: x + shift
    const int64_t page0 = first / PAGE + blockIdx.x;
    const int x0 = (int)max(first - page0 * PAGE, (int64_t)0);
    const int x1 = (int)min(len - page0 * PAGE, (int64_t)PAGE);
    if (p.lens[b] > len && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(&g_status, STATUS_BAD_PAGE);  // longer than its page table
    if (x0 >= x1) return;
    const int id = page_of(p.table, p.max_pages, p.num_pages, b, (int)page0);
    if (id < 0) {
        if (threadIdx.x == 0) atomicOr(&g_status, STATUS_BAD_PAGE);
        return;
    }
    uint8_t* const blk = p.pool + ((int64_t)id * p.hkv + h) * L::BYTES;
    const __nv_bfloat16* const kr = p.k + b * p.ksb + h * p.ksh + (page0 * PAGE + shift) * p.ksn;
    const __nv_bfloat16* const vr = p.v + b * p.vsb + h * p.vsh + (page0 * PAGE + shift) * p.vsn;
    // A channel block of some key rows and of one pair of value rows to a
    // thread, all its loads in flight before the first is used.
    constexpr int STEP = ROW_THREADS / L::NB, PER = PAGE / STEP;
    const int c = threadIdx.x % L::NB, r0 = threadIdx.x / L::NB;
    const bool pair = r0 < PAGE / 2;
    const bool even = pair && 2 * r0 >= x0 && 2 * r0 < x1, odd = pair && 2 * r0 + 1 >= x0 && 2 * r0 + 1 < x1;
    Raw16 kr_[PER], vr_[2];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = r0 + i * STEP;
        kr_[i].load(kr + x * p.ksn, c, p.d, x >= x0 && x < x1);
    }
    vr_[0].load(vr + 2 * r0 * p.vsn, c, p.d, even);
    vr_[1].load(vr + (2 * r0 + 1) * p.vsn, c, p.d, odd);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = r0 + i * STEP;
        if (x < x0 || x >= x1) continue;
        float f[16];
        kr_[i].unpack(f);
        const uint32_t sb = scale_bytes<POW2>(kr_[i].amax(), 0.f, p.k_inv_six, p.k_scale) & 0xFFu;
        const float unit = scale_value(sb), inv = reciprocal(unit * p.k_scale);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e / 4] |= codes2<POW2>(ptx::f2_pack(f[2 * e], f[2 * e + 1]), ptx::f2_pack(inv, inv), ptx::f2_pack(-unit, -unit), p.k_scale)
                        << (8 * (e % 4));
        *reinterpret_cast<uint2*>(blk + L::kcode(x) + c * 8) = make_uint2(w[0], w[1]);
        blk[L::kscale(x, c)] = (uint8_t)sb;
    }
    if (!even && !odd) return;
    float f[16], g[16];
    vr_[0].unpack(f);
    vr_[1].unpack(g);
    const uint32_t both = scale_bytes<POW2>(vr_[0].amax(), vr_[1].amax(), p.v_inv_six, p.v_scale), sf = both & 0xFFu, sg = both >> 8;
    const float uf = scale_value(sf), ug = scale_value(sg);
    const uint64_t inv = ptx::f2_pack(reciprocal(uf * p.v_scale), reciprocal(ug * p.v_scale)), minus_units = ptx::f2_pack(-uf, -ug);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)  // channel i of both keys
        w[i / 4] |= codes2<POW2>(ptx::f2_pack(f[i], g[i]), inv, minus_units, p.v_scale) << (8 * (i % 4));
    uint4* const at = reinterpret_cast<uint4*>(blk + L::vcode(2 * r0) + c * 16);
    if (!(even && odd)) {
        const uint4 old = *at;
        const uint32_t mine = even ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
        w[0] = (w[0] & mine) | (old.x & ~mine);
        w[1] = (w[1] & mine) | (old.y & ~mine);
        w[2] = (w[2] & mine) | (old.z & ~mine);
        w[3] = (w[3] & mine) | (old.w & ~mine);
        *at = make_uint4(w[0], w[1], w[2], w[3]);
        if (even) blk[L::vscale(2 * r0, c)] = (uint8_t)sf;
        else blk[L::vscale(2 * r0 + 1, c)] = (uint8_t)sg;
        return;
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint16_t*>(blk + L::vscale(2 * r0, c)) = (uint16_t)both;
}

__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h2, float s)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    return ptx::pack_bf16x2(f.x * s, f.y * s);
}

// 32 consecutive bytes of global memory in one store (or two of 16).
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&w)[8], bool aligned)
{
    if (aligned)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        ptx::st_global_v4(p, w[0], w[1], w[2], w[3]);
        ptx::st_global_v4(static_cast<char*>(p) + 16, w[4], w[5], w[6], w[7]);
    }
}

// Read: rows 0 .. N - 1 (or the newest N) of every sequence as bf16 (rounded
// once: the stored value times the tensor's scale); rows where no key is are
// zero.  Block (tile of 64 rows, kv head, sequence): the rows' pages are looked
// up once, then a thread takes a channel block of some rows with all its loads
// in flight before the first is used.  Bound by memory: 64 heads x 4096 rows at
// d = 128 (38 MB read, 134 MB written) in 26 us, 6.6 TB/s; row by row, each
// load waited for, it took 38.
template <int D>
__global__ void __launch_bounds__(ROW_THREADS) fa_qcache_read_kernel(const RowParams p)
{
    using L = Block<D>;
    constexpr int STEP = ROW_THREADS / L::NB, PER = PAGE / STEP;  // rows apart, rows of a thread
    __shared__ int src_blk[PAGE], src_row[PAGE];
    const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t i0 = (int64_t)blockIdx.x * PAGE;
    const int rows = (int)min(p.n - i0, (int64_t)PAGE);
    if (tid < PAGE) {
        const int given = p.lens[b];
        const int64_t len = min((int64_t)max(given, 0), (int64_t)p.max_pages * PAGE);
        if (given > len && tid == 0 && h == 0 && blockIdx.x == 0) atomicOr(&g_status, STATUS_BAD_PAGE);
        const int64_t pos = i0 + tid + (p.newest ? (int64_t)given - p.n : 0);
        int blk = -1;
        if (tid < rows && pos >= 0 && pos < len) {
            const int id = page_of(p.table, p.max_pages, p.num_pages, b, (int)(pos / PAGE));
            if (id >= 0) blk = id * p.hkv + h;
            else atomicOr(&g_status, STATUS_BAD_PAGE);
        }
        src_blk[tid] = blk;
        src_row[tid] = (int)(pos & (PAGE - 1));
    }
    __syncthreads();
    const int c = tid % L::NB, r0 = tid / L::NB;
    if (c * 16 >= p.d) return;
    uint2 kc[PER];
    uint4 vc[PER];
    uint8_t ksc[PER], vsc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = r0 + i * STEP;
        kc[i] = make_uint2(0, 0);
        vc[i] = make_uint4(0, 0, 0, 0);
        ksc[i] = vsc[i] = 0;
        if (src_blk[r] >= 0) {
            const uint8_t* const blk = p.pool + (int64_t)src_blk[r] * L::BYTES;
            const int x = src_row[r];
            kc[i] = __ldg(reinterpret_cast<const uint2*>(blk + L::kcode(x) + c * 8));
            vc[i] = __ldg(reinterpret_cast<const uint4*>(blk + L::vcode(x) + c * 16));
            ksc[i] = __ldg(blk + L::kscale(x, c));
            vsc[i] = __ldg(blk + L::vscale(x, c));
        }
    }
    const int64_t out0 = (((int64_t)b * p.hkv + h) * p.n + i0) * p.d + c * 16;
    const bool aligned = p.d % 16 == 0 && ((reinterpret_cast<uintptr_t>(p.ko) | reinterpret_cast<uintptr_t>(p.vo)) & 31u) == 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = r0 + i * STEP;
        if (r >= rows) break;
        const float ks = scale_value(ksc[i]) * p.k_scale, vs = scale_value(vsc[i]) * p.v_scale;
        uint32_t kw[8], vw[8];
        kw[0] = scaled_bf16x2(e2m1x2<0>(kc[i].x), ks);
        kw[1] = scaled_bf16x2(e2m1x2<1>(kc[i].x), ks);
        kw[2] = scaled_bf16x2(e2m1x2<2>(kc[i].x), ks);
        kw[3] = scaled_bf16x2(e2m1x2<3>(kc[i].x), ks);
        kw[4] = scaled_bf16x2(e2m1x2<0>(kc[i].y), ks);
        kw[5] = scaled_bf16x2(e2m1x2<1>(kc[i].y), ks);
        kw[6] = scaled_bf16x2(e2m1x2<2>(kc[i].y), ks);
        kw[7] = scaled_bf16x2(e2m1x2<3>(kc[i].y), ks);
        const uint32_t v4[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
        const int nibble = src_row[r] % 2 * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // 4 channels' bytes: this key's nibbles, packed two to a byte
            const uint32_t n = v4[e] >> nibble & 0x0F0F0F0Fu;
            const uint32_t two = n | (n >> 4);  // bytes 0 and 2 hold channels (0, 1) and (2, 3)
            vw[2 * e] = scaled_bf16x2(e2m1x2<0>(two), vs);
            vw[2 * e + 1] = scaled_bf16x2(e2m1x2<2>(two), vs);
        }
        __nv_bfloat16* const ko = p.ko + out0 + (int64_t)r * p.d;
        __nv_bfloat16* const vo = p.vo + out0 + (int64_t)r * p.d;
        if (c * 16 + 8 < p.d) {
            st_global_32(ko, kw, aligned);
            st_global_32(vo, vw, aligned);
        } else {
            ptx::st_global_v4(ko, kw[0], kw[1], kw[2], kw[3]);
            ptx::st_global_v4(vo, vw[0], vw[1], vw[2], vw[3]);
        }
    }
}

// ---------------------------------------------------------- the work's division

// The calls over whole caches (decode, weights) divide a list of units: all
// pages of sequence 0's first (kv head, row block), of its second one, and so
// on, then sequence 1's.  The list's length follows from the lengths in
// device memory, so every block builds the page counts' prefix sums itself
// and takes an equal run of units: unequal sequences cost no idle blocks, and
// no plan is made on the host.
struct Work {
    const int* prefix;  // B + 1 sums of page counts (shared memory)
    int B, hr;          // hr: kv heads x row blocks

    struct Unit {
        int b, hr, page, pages;
    };
    __device__ __forceinline__ int total() const { return prefix[B] * hr; }
    __device__ __forceinline__ Unit at(int x) const
    {
        const int y = x / hr;
        int lo = 0, hi = B;  // prefix[lo] <= y < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= y) lo = mid;
            else hi = mid;
        }
        Unit u;
        u.b = lo;
        u.pages = prefix[lo + 1] - prefix[lo];
        const int rem = x - prefix[lo] * hr;
        u.hr = rem / u.pages;
        u.page = rem - u.hr * u.pages;
        return u;
    }
};

// A sequence's length, at most what its page table holds.
__device__ __forceinline__ int clamp_length(int len, int max_pages) { return (int)min((int64_t)max(len, 0), (int64_t)max_pages * PAGE); }
__device__ __forceinline__ int length_of(const int32_t* lens, int b, int max_pages) { return clamp_length(lens[b], max_pages); }

// prefix[0 .. B] by a block of NTHREADS threads (scratch: one int per warp).
// Up to 32 sequences every warp computes them all and waits for no other.
template <int NTHREADS>
__device__ __forceinline__ void page_prefix(const int32_t* lens, int B, int max_pages, int* prefix, int* scratch)
{
    constexpr int W = NTHREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto scan = [&](int b) {
        int v = b < B ? (length_of(lens, b, max_pages) + PAGE - 1) / PAGE : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += n;
        }
        return v;
    };
    if (B <= 32) {
        const int v = scan(lane);
        if (lane == 0) prefix[0] = 0;
        if (lane < B) prefix[lane + 1] = v;
        __syncwarp();
        return;
    }
    int base = 0;
    if (tid == 0) prefix[0] = 0;
    for (int b0 = 0; b0 < B; b0 += NTHREADS) {
        const int b = b0 + tid, v = scan(b);
        if (lane == 31) scratch[warp] = v;
        __syncthreads();
        int before = base, all = base;
#pragma unroll 4
        for (int w = 0; w < W; ++w) {
            const int n = scratch[w];
            if (w < warp) before += n;
            all += n;
        }
        if (b < B) prefix[b + 1] = before + v;
        base = all;
        __syncthreads();
    }
}

// Brings the small tensors of a call to L2, every block a share, before the
// work that this launch depends on has ended: their later reads, which
// follow one another, then cost an L2 access each instead of a DRAM one.  A
// page table with room for far more than its sequences hold is left alone.
__device__ __forceinline__ void prefetch_l2(const void* p, int64_t bytes)
{
    if (bytes > (1 << 20)) return;
    const char* const c = static_cast<const char*>(p);
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 128; i < bytes; i += (int64_t)gridDim.x * blockDim.x * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(c + i));
}

// ------------------------------------------------------------------- decode

struct DecParams {
    const __nv_bfloat16* q;       // (B, H, nq, d): the rows of a kv head's group adjoin
    const uint8_t* pool;          // (num_pages, hkv, 72 * D)
    const int32_t *table, *lens;  // (B, max_pages), (B)
    __nv_bfloat16* o;             // (B, H, nq, d)
    float* lse;                   // (B, H, nq)
    float* ws;                    // 2 partial results a block
    int* desc;                    // 2 ints a block: the split segment that begins there (or -1), its last block
    int B, hkv, nq, rows, rb;     // rows: query rows of a kv head; rb: blocks of them
    int d, max_pages, num_pages, causal;
    float scale_log2;             // scale * log2(e) * k_scale
    float v_scale;
    uint64_t wait_limit_ns;
    int debug_skip;               // test hook: block 0's first warp never copies this one of its pages (-1: off)
    const float* lse_in;          // weights: (B, H, nq)
    const float* w_in;            // (B, hkv, w_len)
    float* w_out;
    int64_t w_len;
};

// A probability 2^(x - max + SHIFT) is held as the sum of two fp16 numbers, its
// rounding and what that left: 22 bits, fp32's own errors (one alone has 11, and
// results that nearly cancel lost 2^-12 of sum p |v|).  1 becomes 2^15, within
// fp16's range, and what lies below fp16's smallest steps is under 2^-40 of the
// largest weight, so that a long cache of small weights is not rounded away.
constexpr float SHIFT = 15.0f;
constexpr uint32_t WAIT_CODE = 900;  // fa_check_device_status's wait code of the cache kernels' copies

template <int NBYTES>
struct Chunk {  // a lane's share of a row: 16 or 8 bytes
    uint32_t w[NBYTES / 4];
    __device__ __forceinline__ void load(const uint8_t* p)
    {
        if constexpr (NBYTES == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        }
    }
    __device__ __forceinline__ void store(uint8_t* p) const
    {
        if constexpr (NBYTES == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
};

// a * (half `HI` of f, twice): the multiply reads either half of its operand.
template <int HI>
__device__ __forceinline__ uint32_t hmul2_by(uint32_t a, uint32_t f)
{
    const __half2 x = *reinterpret_cast<const __half2*>(&a), y = *reinterpret_cast<const __half2*>(&f);
    const __half2 r = __hmul2(x, HI ? __high2half2(y) : __low2half2(y));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Query rows of one (sequence, kv head, row block), as the B operand of the
// score product, and what a lane needs of them: lane (g, t) = (lane / 4,
// lane % 4) holds row g's channels D/4 t .. and, of the columns 2t and
// 2t + 1 whose scores it gets, the factor to base-2 scores and the count of
// keys they see.  Rows are scaled by a power of two so that their largest
// entry lies in [2^14, 2^15): bf16 entries down to 2^-31 of it are exact in
// fp16 whatever the row's size.  FOLD: at most 4 rows, and the tile's rows 4 to 7 are
// rows 0 to 3 again (decode uses them for the second halves of probabilities).
template <int D, int NT, bool FOLD = false>
struct Rows {
    static_assert(!FOLD || NT == 1, "one tile, folded");
    // The query row of a tile's row.
    static __device__ __forceinline__ int row_of(int r) { return FOLD ? r & 3 : r; }
    uint32_t q[NT][D / 16][2];
    float sc[NT][2];
    int lim[NT][2];
    int len, min_lim;

    // The rows' raw entries: issued before a warp's first copies, so that they
    // do not wait behind them.
    struct Raw {
        uint4 w[NT][D / 32];
        int len;
    };
    static __device__ __forceinline__ void fetch(Raw& raw, const DecParams& p, int b, int hr)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int h = p.rb == 1 ? hr : hr / p.rb, r0 = (hr - h * p.rb) * (8 * NT);
        const int64_t row0 = ((int64_t)b * p.hkv + h) * p.rows;
        raw.len = p.lens[b];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = r0 + nt * 8 + row_of(g);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const int c = D / 4 * t + 8 * e;
                raw.w[nt][e] = make_uint4(0, 0, 0, 0);
                if (row < p.rows && c < p.d) raw.w[nt][e] = *reinterpret_cast<const uint4*>(p.q + (row0 + row) * p.d + c);
            }
        }
    }

    __device__ __forceinline__ void load(const Raw& raw, const DecParams& p, int hr)
    {
        const int lane = threadIdx.x & 31, t = lane & 3;
        const int r0 = p.rb == 1 ? 0 : hr % p.rb * (8 * NT);
        len = clamp_length(raw.len, p.max_pages);
        // A causal query stands at its place in the sequence, which a length beyond the page table does not move.
        const int end = max(raw.len, 0) - p.nq + 1;
        min_lim = p.causal ? min(len, end) : len;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[D / 4];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) unpack8(raw.w[nt][e], f + 8 * e);
            float am = 0.f;
#pragma unroll
            for (int e = 0; e < D / 4; ++e) am = fmaxf(am, fabsf(f[e]));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int ex = (int)(__float_as_uint(am) >> 23) - 127;
            const int k = am > 0.f && ex < 128 ? min(126, max(-126, 14 - ex)) : 0;
            const float up = __uint_as_float((uint32_t)(127 + k) << 23);
            const float down = p.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                q[nt][c][0] = pack_h2(f[4 * c] * up, f[4 * c + 1] * up);
                q[nt][c][1] = pack_h2(f[4 * c + 2] * up, f[4 * c + 3] * up);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sc[nt][j] = __shfl_sync(0xffffffffu, down, (2 * t + j) * 4);
                const int r = r0 + nt * 8 + row_of(2 * t + j);
                lim[nt][j] = p.causal && r < p.rows ? min(len, end + (p.nq == 1 ? 0 : r % p.nq)) : len;
            }
        }
    }
};

// Scores of a page, transposed: S^T = K Q^T, 16 keys by 8 query rows a
// product, so that few rows waste no tensor work.  Lane (g, t) of s[r][nt]
// holds keys 16r + g (entries 0, 1) and 16r + 8 + g (2, 3) against rows 2t and
// 2t + 1.  blk: a page's block in shared or global memory.
template <int D, int NT, int TOGETHER, bool FOLD>
__device__ __forceinline__ void page_scores(const uint8_t* blk, const Rows<D, NT, FOLD>& rows, float (&s)[4][NT][4])
{
    using L = Block<D>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    Chunk<8 * L::P> sc;
    sc.load(blk + L::KS + lane * (8 * L::P));
    // TOGETHER groups of 16 keys at a time: a product waits for the one before it
    // on the same sums, and another group's fill the wait.
#pragma unroll
    for (int r0 = 0; r0 < 4; r0 += TOGETHER) {
        Chunk<D / 8> k[TOGETHER][2];
        uint32_t f[TOGETHER][2];
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) {
            const int r = r0 + i;
            k[i][0].load(blk + L::kcode(16 * r + g) + t * (D / 8));
            k[i][1].load(blk + L::kcode(16 * r + 8 + g) + t * (D / 8));
            // Scales: at D = 128 those of rows g and g + 8, each of the lane's two
            // channel blocks; at D = 64 one of each row.
            f[i][0] = e4m3x2(D == 128 ? sc.w[r] : sc.w[r / 2] >> (16 * (r % 2)));
            f[i][1] = D == 128 ? e4m3x2(sc.w[r] >> 16) : f[i][0];
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int i = 0; i < TOGETHER; ++i) {
                const uint32_t w0 = k[i][0].w[c / 2], w1 = k[i][1].w[c / 2];
                auto by0 = [&](uint32_t a) { return D == 128 && c >= 4 ? hmul2_by<1>(a, f[i][0]) : hmul2_by<0>(a, f[i][0]); };
                auto by1 = [&](uint32_t a) { return D == 64 || c >= 4 ? hmul2_by<1>(a, f[i][1]) : hmul2_by<0>(a, f[i][1]); };
                const uint32_t a0 = by0(c % 2 ? e2m1x2<2>(w0) : e2m1x2<0>(w0));
                const uint32_t a1 = by1(c % 2 ? e2m1x2<2>(w1) : e2m1x2<0>(w1));
                const uint32_t a2 = by0(c % 2 ? e2m1x2<3>(w0) : e2m1x2<1>(w0));
                const uint32_t a3 = by1(c % 2 ? e2m1x2<3>(w1) : e2m1x2<1>(w1));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float(&d)[4] = s[r0 + i][nt];
                    if (c == 0) mma_zero(d, a0, a1, a2, a3, rows.q[nt][c][0], rows.q[nt][c][1]);
                    else mma(d, a0, a1, a2, a3, rows.q[nt][c][0], rows.q[nt][c][1]);
                }
            }
    }
}

// Running softmax of a warp over a segment's pages, O transposed: lane (g, t)
// of o[m][nt] holds channels D/8 g + 2m (entries 0, 1) and D/8 g + 2m + 1
// (2, 3) of rows 2t and 2t + 1.
//
// A probability is two fp16 numbers, and so V meets two operands.  At most 4 rows
// (FOLD) take one product for both: the tile's rows 0 to 3 carry the roundings, rows
// 4 to 7 what those left, and close() adds them up.  (8 x 32 heads x 32768 keys, one
// row, d = 128: 226 us with two products, 205 folded;
// More rows take two: 8 x 8 heads x 32768 keys, 8 rows 67.4 us (62.2 with one fp16
// number a probability), 16 rows 111.8 (92.6); 48 x 4 heads x 0 to 5000 keys, 16 rows,
// d = 64, 28.7 (27.2).)
template <int D, int NT, bool FOLD>
struct State {
    using R = Rows<D, NT, FOLD>;
    float o[D / 16][NT][4];
    // Largest unscaled score (differences to it are scaled, so that the
    // largest key's weight is 1 however large the scores are); this lane's
    // share of the sum (times 2^SHIFT).
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) m[nt][j] = -INFINITY, l[nt][j] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][nt][e] = 0.f;
        }
    }

    // A page's probabilities as B operands (keys 2t, 2t + 1 and 2t + 8, 2t + 9 of
    // row g): their fp16 roundings, then what those left.
    static constexpr int HALVES = FOLD ? 1 : 2;
    struct Probs {
        uint32_t w[4][NT][HALVES][2];
    };

    // Takes a page's scores in: the running maxima and sums, and the probabilities.
    __device__ __forceinline__ void add_scores(float (&s)[4][NT][4], const R& rows, int page, Probs& pb)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        const bool second = FOLD && (lane & 2);  // its columns carry the rests
        const int key0 = page * PAGE;
        const bool whole = key0 + PAGE <= rows.min_lim;  // every row sees every key
        bool rises = false;
        float mm[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (!whole) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (key0 + 16 * r + g >= rows.lim[nt][j]) s[r][nt][j] = -INFINITY;
                        if (key0 + 16 * r + 8 + g >= rows.lim[nt][j]) s[r][nt][2 + j] = -INFINITY;
                    }
                }
                float x = fmaxf(s[0][nt][j], s[0][nt][2 + j]);
#pragma unroll
                for (int r = 1; r < 4; ++r) x = ptx::fmax3(x, s[r][nt][j], s[r][nt][2 + j]);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                mm[nt][j] = fmaxf(m[nt][j], x);
                rises |= mm[nt][j] > m[nt][j];
            }
        if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f[j] = m[nt][j] == -INFINITY ? 0.f : ptx::ex2((m[nt][j] - mm[nt][j]) * rows.sc[nt][j]);
                    l[nt][j] *= f[j];
                    m[nt][j] = mm[nt][j];
                }
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    o[c][nt][0] *= f[0];
                    o[c][nt][1] *= f[1];
                    o[c][nt][2] *= f[0];
                    o[c][nt][3] *= f[1];
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float top[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) top[j] = m[nt][j] == -INFINITY ? 0.f : m[nt][j];
            // Pairs of columns in packed fp32 arithmetic.
            const uint64_t neg = ptx::f2_pack(-top[0], -top[1]), sc = ptx::f2_pack(rows.sc[nt][0], rows.sc[nt][1]);
            const uint64_t shift = ptx::f2_pack(SHIFT, SHIFT);
            uint64_t sum = ptx::f2_pack(l[nt][0], l[nt][1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    float x0 = s[r][nt][e], x1 = s[r][nt][e + 1], p0, p1;
                    ptx::f2_unpack(ptx::f2_fma(ptx::f2_add(ptx::f2_pack(x0, x1), neg), sc, shift), p0, p1);
                    p0 = ptx::ex2(p0);
                    p1 = ptx::ex2(p1);
                    if (!whole && x0 == -INFINITY) p0 = 0.f;
                    if (!whole && x1 == -INFINITY) p1 = 0.f;
                    sum = ptx::f2_add(sum, ptx::f2_pack(p0, p1));
                    s[r][nt][e] = p0;
                    s[r][nt][e + 1] = p1;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = s[r][nt][2 * e], b = s[r][nt][2 * e + 1];
                    const uint32_t h = pack_h2(a, b);
                    if constexpr (FOLD) {
                        pb.w[r][nt][0][e] = transpose8x8(second ? rest_h2(a, b, h) : h);
                    } else {
                        pb.w[r][nt][0][e] = transpose8x8(h);
                        pb.w[r][nt][1][e] = transpose8x8(rest_h2(a, b, h));
                    }
                }
            }
            ptx::f2_unpack(sum, l[nt][0], l[nt][1]);
        }
    }

    // O^T += V^T P^T: a scale belongs to a key and a block of channels, so it
    // multiplies the operand (exactly), two keys at a time.  vblk: the V half
    // of a page's block.
    __device__ __forceinline__ void add_values(const uint8_t* vblk, const R& rows, int page, const Probs& pb)
    {
        using L = Block<D>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint8_t* const blk = vblk - L::VC;
        const int key0 = page * PAGE;
        const bool whole = key0 + PAGE <= rows.len;
        const int b = g * (D / 8) / 16;
        Chunk<16> sc;
        sc.load(blk + L::VS + (t * L::NB + b) * 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            Chunk<D / 8> v0, v1;
            v0.load(blk + L::vcode(16 * r + 2 * t) + g * (D / 8));
            v1.load(blk + L::vcode(16 * r + 8 + 2 * t) + g * (D / 8));
            uint32_t w = sc.w[r];
            if (!whole) {  // places of no key hold anything: their weight is 0, and 0 * NaN must not be formed
                const int left = rows.len - (key0 + 16 * r + 2 * t);
                if (left < 10) w &= left <= 0 ? 0u : left == 1 ? 0xFFu : left <= 8 ? 0xFFFFu : 0xFFFFFFu;
            }
            const uint32_t f0 = e4m3x2(w), f1 = e4m3x2(w >> 16);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const uint32_t w0 = v0.w[c / 2], w1 = v1.w[c / 2];
                const uint32_t a0 = hmul2(c % 2 ? e2m1x2<2>(w0) : e2m1x2<0>(w0), f0);
                const uint32_t a1 = hmul2(c % 2 ? e2m1x2<3>(w0) : e2m1x2<1>(w0), f0);
                const uint32_t a2 = hmul2(c % 2 ? e2m1x2<2>(w1) : e2m1x2<0>(w1), f1);
                const uint32_t a3 = hmul2(c % 2 ? e2m1x2<3>(w1) : e2m1x2<1>(w1), f1);
#pragma unroll
                for (int half = 0; half < HALVES; ++half)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(o[c][nt], a0, a1, a2, a3, pb.w[r][nt][half][0], pb.w[r][nt][half][1]);
            }
        }
    }

    // The end of a segment: base-2 maxima, and the sums over the warp's lanes
    // that share a row.
    __device__ __forceinline__ void close(const R& rows)
    {
        if constexpr (FOLD) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][0][e] += __shfl_xor_sync(0xffffffffu, o[c][0][e], 2);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
                m[nt][j] = m[nt][j] == -INFINITY ? m[nt][j] : m[nt][j] * rows.sc[nt][j];
            }
    }
};

// A partial result: R rows of D unnormalised outputs, then their maxima and sums.
template <int D, int R>
struct Partial {
    static constexpr int FLOATS = R * (D + 2);
    static __device__ __forceinline__ int o(int row) { return row * D; }
    static __device__ __forceinline__ int m(int row) { return R * D + row; }
    static __device__ __forceinline__ int l(int row) { return R * D + R + row; }
};

// The same in shared memory, as the warps write it: pairs of channels by rows,
// a pair's rows adjoining and one place left free, which spreads a store of
// the lanes (8 pairs by 4 rows) over the banks.
template <int D, int R>
struct Piece {
    static constexpr int FLOATS = D * (R + 1) + 2 * R;
    // Channels D/8 g + 2c and the next.
    static __device__ __forceinline__ int o(int g, int c, int row) { return ((c * 8 + g) * (R + 1) + row) * 2; }
    static __device__ __forceinline__ int m(int row) { return D * (R + 1) + row; }
    static __device__ __forceinline__ int l(int row) { return D * (R + 1) + R + row; }
};

__device__ __forceinline__ float natural_lse(float m, float l)
{
    return l > 0.f || !(l == l) ? (m + ptx::lg2(l) - SHIFT) * LN2 : -INFINITY;
}

// Shared memory of the decode kernel: a ring of half pages for each warp, one
// partial result for each (its first piece; its last one takes the ring's
// place when the ring is done), and the page counts' prefix sums.
// One block an SM, of as many warps as registers and shared memory allow: a
// warp's chain through a page (scores, maximum, exponentials, transposes,
// products) is long, and it takes many to keep the SM's pipes fed (16 x 8 heads x
// 16384 keys, 4 rows, d = 64: 47.3 us with 12 warps, 45.2 with 16).
template <int D, int NT>
struct DecLayout {
    static constexpr int WARPS = D == 128 ? (NT == 1 ? 12 : 8) : (NT == 1 ? 16 : 12);
    static constexpr int THREADS = WARPS * 32;
    // A slot holds half a page (K or V) at 128 channels and a whole one at 64:
    // copies of 4608 bytes either way.
    static constexpr int SLOTS = D == 128 || NT == 2 ? 3 : 2;
    static constexpr bool WHOLE = D == 64;
    static constexpr int HALF = 36 * 128;
    static constexpr int PART = Piece<D, 8 * NT>::FLOATS * 4;
    static constexpr int RING = SLOTS * HALF;
    static constexpr int PREFIX = WARPS * (RING + PART);
    static_assert(PART <= RING && HALF % 16 == 0 && PART % 16 == 0, "layout");
    static constexpr int bytes(int B) { return PREFIX + (B + 1) * 4; }
    static_assert(bytes(MAX_B) + 2048 <= 232448, "shared memory");
    static __device__ __forceinline__ int ring(int warp) { return warp * RING; }
    static __device__ __forceinline__ float* partial(uint8_t* smem, int slot)
    {
        return reinterpret_cast<float*>(slot % 2 ? smem + ring(slot / 2) : smem + WARPS * RING + slot / 2 * PART);
    }
};

// A warp's copies of its run of pages into its ring.  SLOTS halves (K, then V;
// or K alone; or WHOLE pages) are in flight; the warp waits for one, reads it and refills its
// slot.  The places of 32 units are looked up at once, one a lane, the next
// 32 ahead of their use.
template <int D, int SLOTS, bool WITH_V, bool WHOLE>
struct Feed {
    static constexpr int HALF = WHOLE ? 72 * D : 36 * D, PER = WITH_V && !WHOLE ? 2 : 1;
    const DecParams& p;
    const Work& work;
    uint8_t* ring;
    uint32_t bar;
    int x1, base;             // end of the run; first unit of `now`
    int next_unit, next_half; // what is copied next
    int fill, use;            // slots
    uint32_t parity;
    int flying;
    bool due;                 // `ahead` is to be looked up
    // This lane's unit of the current 32 and of the next: its segment, and the
    // page's block in the pool (-1 where the table's entry is none of its pages;
    // until begin(), the entry itself, so that nothing waits for it yet).
    int now_seg, now_blk, ahead_seg, ahead_blk;
    int first_page;           // of the run's first unit (a later unit's page follows from its segment's first)
    const uint8_t* src;       // the block that is being copied

    // The segment and page of unit x, and the page table's entry.
    __device__ __forceinline__ int look(int x, int& seg, int& id) const
    {
        seg = id = -1;
        if (x >= x1) return 0;
        const Work::Unit u = work.at(x);
        seg = u.b * work.hr + u.hr;
        id = p.table[(int64_t)u.b * p.max_pages + u.page];
        return u.page;
    }
    __device__ __forceinline__ int block_of(int seg, int id) const
    {
        if (seg < 0) return -1;
        if ((unsigned)id >= (unsigned)p.num_pages) {
            atomicOr(&g_status, STATUS_BAD_PAGE);
            return -1;
        }
        const int hr = seg % work.hr;
        return id * p.hkv + (work.hr == p.hkv ? hr : hr / p.rb);
    }
    __device__ __forceinline__ Feed(uint8_t* ring_, uint32_t bar_, const DecParams& p_, const Work& work_)
        : p(p_), work(work_), ring(ring_), bar(bar_), fill(0), use(0), parity(0), flying(0), src(nullptr)
    {
    }
    // Takes up units x0 .. x1_ - 1 (nothing is in flight).
    __device__ __forceinline__ void start(int x0, int x1_)
    {
        x1 = x1_;
        base = next_unit = x0;
        next_half = 0;
        first_page = __shfl_sync(0xffffffffu, look(base + (int)(threadIdx.x & 31), now_seg, now_blk), 0);
        ahead_seg = ahead_blk = -1;
        due = x1 - base > 32;
    }
    // Starts the first copies, a lane a slot.
    __device__ __forceinline__ void begin()
    {
        now_blk = block_of(now_seg, now_blk);
        const int lane = threadIdx.x & 31;
        const int blk = __shfl_sync(0xffffffffu, now_blk, lane / PER);
        flying = min(SLOTS, (x1 - base) * PER);
        if (lane < flying) copy(fill + lane < SLOTS ? fill + lane : fill + lane - SLOTS, lane / PER, lane % PER, source(blk));
        fill = fill + flying < SLOTS ? fill + flying : fill + flying - SLOTS;
        next_unit = base + flying / PER;
        next_half = flying % PER;
        if (next_half != 0) src = source(__shfl_sync(0xffffffffu, now_blk, next_unit - base));
    }
    // A page's block; any block for a page that does not exist (it is not used).
    __device__ __forceinline__ const uint8_t* source(int blk) const { return p.pool + (int64_t)max(0, blk) * Block<D>::BYTES; }
    __device__ __forceinline__ void copy(int slot, int unit, int half, const uint8_t* from) const
    {
        ptx::mbar_arrive_expect_tx(bar + 8 * slot, HALF);
        if (!(p.debug_skip == unit && base == 0 && blockIdx.x == 0))
            ptx::bulk_load(ptx::smem_addr(ring) + slot * HALF, from + (PER == 2 ? half * HALF : 0), HALF, bar + 8 * slot);
    }
    // Starts the next copy, if one is left.
    __device__ __forceinline__ void issue()
    {
        if (next_unit >= x1) return;
        const int i = next_unit - base;
        if (next_half == 0) src = source(i < 32 ? __shfl_sync(0xffffffffu, now_blk, i) : __shfl_sync(0xffffffffu, ahead_blk, i - 32));
        if ((threadIdx.x & 31) == 0) copy(fill, i, next_half, src);
        fill = fill + 1 == SLOTS ? 0 : fill + 1;
        ++flying;
        if (++next_half == PER) {
            next_half = 0;
            ++next_unit;
        }
    }
    // The segment of unit x, the units in turn.
    __device__ __forceinline__ int place(int x)
    {
        if (x - base == 32) {
            now_seg = ahead_seg;
            now_blk = ahead_blk;
            base += 32;
            due = x1 - base > 32;
        }
        if (due && x - base >= 4) {  // well before the copies need it, and not among a run's first steps
            due = false;
            look(base + 32 + (int)(threadIdx.x & 31), ahead_seg, ahead_blk);
            ahead_blk = block_of(ahead_seg, ahead_blk);
        }
        return __shfl_sync(0xffffffffu, now_seg, x - base);
    }
    // Whether the page of the unit that place() gave last exists.
    __device__ __forceinline__ bool there(int x) const { return __shfl_sync(0xffffffffu, now_blk, x - base) >= 0; }
    // The oldest half in flight, or null when the wait gave up.
    __device__ __forceinline__ const uint8_t* wait(volatile uint32_t* abort_flag)
    {
        const bool ok = wait_bar(bar + 8 * use, parity, p.wait_limit_ns, abort_flag, WAIT_CODE);
        return __all_sync(0xffffffffu, ok) ? ring + use * HALF : nullptr;
    }
    // The warp has read it: refill its slot.
    __device__ __forceinline__ void next()
    {
        __syncwarp();
        if (++use == SLOTS) {
            use = 0;
            parity ^= 1u;
        }
        --flying;
        issue();
    }
    // Copies still in flight after a wait gave up must land before the block leaves.
    __device__ __forceinline__ void drain(volatile uint32_t* abort_flag)
    {
        for (; flying > 0; --flying) {
            drain_bar(bar + 8 * use, parity, p.wait_limit_ns, abort_flag, WAIT_CODE);
            if (++use == SLOTS) {
                use = 0;
                parity ^= 1u;
            }
        }
        __syncwarp();
    }
};

// Decode.  Block c takes units [c T / G, (c + 1) T / G) of the T pages, and its
// warps equal runs of those.  A segment (all pages of one sequence, kv head
// and row block) that lies within a warp's run is written out at once; the
// pieces of others go to shared memory, where the block joins neighbouring
// warps' pieces of a segment; pieces of segments that cross blocks go to the
// workspace (two a block at most) for the combine kernel.
//
// Bound by reading the cache: 8 x 32 heads x 32768 keys at d = 128 (1.21 GB) in
// 206 us with the combine kernel, 5870 GB/s, 0.87 of the measured copy
// bandwidth; the same attention over a bf16 cache takes 590 us.  In the loop a
// page (9216 bytes) takes an SM 430 cycles where the copy bandwidth alone gives
// about 400; the conversions (280 a page, 2 a clock) need 140 of them, the fp16
// multiplies 128 and the products 128, on pipes of their own.  The rest is the
// start (lengths, page table, query rows: 7 us) and the join.
template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(DecLayout<D, NT>::THREADS, 1) fa_qcache_decode_kernel(const DecParams p)
{
    using Y = DecLayout<D, NT>;
    constexpr int R = 8 * NT, WARPS = Y::WARPS, THREADS = Y::THREADS;
    using PS = Partial<D, R>;
    using PC = Piece<D, R>;
    extern __shared__ __align__(128) uint8_t smem[];
    int* const prefix = reinterpret_cast<int*>(smem + Y::PREFIX);
    __shared__ int scratch[WARPS];
    __shared__ __align__(8) uint64_t bars[WARPS * Y::SLOTS];
    __shared__ uint32_t abort_flags[WARPS];
    __shared__ int slot_seg[32];                 // segment of each slot, or -1
    __shared__ int slot_ends[2 * WARPS];         // bit 0: the segment begins in it, bit 1: ends
    __shared__ float slot_weight[2 * WARPS][R];  // of each slot's row in the joined one
    struct Run {
        uint32_t mask;    // its slots
        int begins, ends; // whether the segment does in this block
        int rows;         // query rows from its row block's first
        int64_t row;      // that one, of all
    };
    __shared__ Run runs[2 * WARPS];
    __shared__ int run_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    static_assert(2 * WARPS <= 32, "a lane a slot");
    if (lane < Y::SLOTS) ptx::mbar_init(ptx::smem_addr(&bars[warp * Y::SLOTS + lane]), 1);
    if (lane < 2) slot_seg[warp * 2 + lane] = -1;
    if (warp == 0 && lane >= 2 * WARPS) slot_seg[lane] = -1;
    if (lane == 0) abort_flags[warp] = 0;
    volatile uint32_t* const abort_flag = &abort_flags[warp];
    ptx::fence_barrier_init();
    __syncwarp();
    prefetch_l2(p.table, (int64_t)p.B * p.max_pages * 4);
    prefetch_l2(p.q, (int64_t)p.B * p.hkv * p.rows * p.d * 2);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    page_prefix<THREADS>(p.lens, p.B, p.max_pages, prefix, scratch);
    Work work{prefix, p.B, p.hkv * p.rb};

    // Sequences of no key: nothing is seen.
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (lane == 0 && warp == 0 && p.lens[b] > p.max_pages * (int64_t)PAGE) atomicOr(&g_status, STATUS_BAD_PAGE);
        if (prefix[b + 1] != prefix[b]) continue;
        const int64_t n = (int64_t)p.hkv * p.rows, at = b * n;
        for (int64_t e = tid; e < n * (p.d / 8); e += THREADS) ptx::st_global_v4(p.o + at * p.d + e * 8, 0, 0, 0, 0);
        for (int64_t e = tid; e < n; e += THREADS) p.lse[at + e] = -INFINITY;
    }

    const int T = work.total();
    const int G = min((int)gridDim.x, T);
    const int cta = blockIdx.x;
    if (cta >= G) {
        if (tid == 0) p.desc[2 * cta] = -1;
        return;
    }
    const int lo = (int)((int64_t)cta * T / G), hi = (int)((int64_t)(cta + 1) * T / G);
    const int nw = min(WARPS, hi - lo);
    int slot = 0;
    if (warp < nw) {
        const int x0 = lo + (int)((int64_t)(hi - lo) * warp / nw), x1 = lo + (int)((int64_t)(hi - lo) * (warp + 1) / nw);
        Rows<D, NT, FOLD> rows;
        State<D, NT, FOLD> st;
        int seg = -1, begins = 0, page = 0;
        auto finish = [&] {
            st.close(rows);
            const int ends = (page + 1) * PAGE >= rows.len;
            if (begins && ends) {
                const int b = seg / work.hr, hr = seg - b * work.hr, h = hr / p.rb;
                const int r0 = (hr - h * p.rb) * R;
                const int64_t row0 = ((int64_t)b * p.hkv + h) * p.rows;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int row = r0 + nt * 8 + 2 * t + j;
                        if (row >= p.rows) continue;
                        const float f = st.l[nt][j] == 0.f ? 0.f : p.v_scale / st.l[nt][j];
                        uint32_t w[D / 16];
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) w[c] = ptx::pack_bf16x2(st.o[c][nt][j] * f, st.o[c][nt][2 + j] * f);
                        __nv_bfloat16* const out = p.o + (row0 + row) * p.d + g * (D / 8);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            if (g * (D / 8) + 8 * c < p.d) ptx::st_global_v4(out + 8 * c, w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                        if (g == 0) p.lse[row0 + row] = natural_lse(st.m[nt][j], st.l[nt][j]);
                    }
                return;
            }
            const int at = warp * 2 + slot++;
            float* const f = Y::partial(smem, at);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = nt * 8 + 2 * t + j;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
                        *reinterpret_cast<float2*>(f + PC::o(g, c, row)) = make_float2(st.o[c][nt][j], st.o[c][nt][2 + j]);
                    if (g == 0) {
                        f[PC::m(row)] = st.m[nt][j];
                        f[PC::l(row)] = st.l[nt][j];
                    }
                }
            if (lane == 0) {
                slot_seg[at] = seg;
                slot_ends[at] = begins | (ends << 1);
            }
        };
        // Copies run ahead of the arithmetic by the ring's slots: K and V halves
        // of the pages in turn, each slot refilled as soon as the warp has read it.
        Feed<D, Y::SLOTS, true, Y::WHOLE> feed(smem + Y::ring(warp), ptx::smem_addr(&bars[warp * Y::SLOTS]), p, work);
        feed.start(x0, x1);
        typename Rows<D, NT, FOLD>::Raw raw;
        for (int x = x0; x < x1; ++x) {
            const int next_seg = feed.place(x);
            ++page;
            if (next_seg != seg) {
                const int b = next_seg / work.hr, hr = next_seg - b * work.hr;
                rows.fetch(raw, p, b, hr);
                if (seg >= 0) {
                    --page;
                    finish();
                } else {
                    feed.begin();
                }
                page = seg < 0 ? feed.first_page : 0;
                seg = next_seg;
                begins = page == 0;
                rows.load(raw, p, hr);
                st.clear();
            }
            const bool there = feed.there(x);
            float s[4][NT][4];
            typename State<D, NT, FOLD>::Probs pb;
            const uint8_t* blk = feed.wait(abort_flag);
            if (!blk) break;
            page_scores<D, NT, 1>(blk, rows, s);
            if constexpr (!Y::WHOLE) feed.next();
            if (there) st.add_scores(s, rows, page, pb);
            if constexpr (Y::WHOLE) {
                blk += Block<D>::VC;
            } else {
                blk = feed.wait(abort_flag);
                if (!blk) break;
            }
            if (there) st.add_values(blk, rows, page, pb);
            feed.next();
        }
        feed.drain(abort_flag);
        finish();
    }
    __syncthreads();

    // Join the warps' pieces: runs of slots of one segment.  A lane a slot finds
    // the runs, a thread a run's row weighs its slots (the first one takes the
    // joined maximum and sum), a thread four channels of a row adds them up.
    if (warp == 0) {
        const int seg = slot_seg[lane];
        const uint32_t mask = __match_any_sync(0xffffffffu, seg);
        const int a = __ffs(mask) - 1, z = 31 - __clz(mask);
        const bool leads = seg >= 0 && a == lane;
        const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
        if (lane == 0) {
            run_count = __popc(leaders);
            p.desc[2 * cta] = -1;
        }
        __syncwarp();
        if (leads) {
            Run& run = runs[__popc(leaders & ((1u << lane) - 1u))];
            const int b = seg / work.hr, hr = seg - b * work.hr, h = p.rb == 1 ? hr : hr / p.rb;
            run.mask = mask;
            run.begins = slot_ends[a] & 1;
            run.ends = slot_ends[z] & 2;
            run.row = ((int64_t)b * p.hkv + h) * p.rows + (hr - h * p.rb) * R;
            run.rows = p.rows - (hr - h * p.rb) * R;
            if (run.begins && !run.ends) {
                // The block that holds the segment's last unit x: the c with c T / G <= x < (c + 1) T / G.
                const int x = prefix[b] * work.hr + (hr + 1) * (prefix[b + 1] - prefix[b]) - 1;
                p.desc[2 * cta] = seg;
                p.desc[2 * cta + 1] = (int)(((int64_t)(x + 1) * G - 1) / T);
            }
        }
    }
    __syncthreads();
    const int n_runs = run_count;
    for (int e = tid; e < n_runs * R; e += THREADS) {
        const uint32_t mask = runs[e / R].mask;
        const int r = e % R, a = __ffs(mask) - 1, z = 31 - __clz(mask);
        float mx = -INFINITY, l = 0.f;
#pragma unroll 4
        for (int k = a; k <= z; ++k)
            if (mask >> k & 1u) mx = fmaxf(mx, Y::partial(smem, k)[PC::m(r)]);
#pragma unroll 4
        for (int k = a; k <= z; ++k)
            if (mask >> k & 1u) {
                const float* const f = Y::partial(smem, k);
                const float m = f[PC::m(r)], w = m == -INFINITY ? 0.f : ptx::ex2(m - mx);
                slot_weight[k][r] = w;
                l = fmaf(w, f[PC::l(r)], l);
            }
        float* const f = Y::partial(smem, a);
        f[PC::m(r)] = mx;
        f[PC::l(r)] = l;
    }
    __syncthreads();
    constexpr int QUADS = R * D / 4;
    for (int e = tid; e < n_runs * QUADS; e += THREADS) {
        const Run run = runs[e / QUADS];
        const int r = e % QUADS / (D / 4), c = e % (D / 4) * 4;
        if (r >= run.rows) continue;
        const int a = __ffs(run.mask) - 1, z = 31 - __clz(run.mask);
        const int at = PC::o(c / (D / 8), c % (D / 8) / 2, r), next = PC::o(c / (D / 8), c % (D / 8) / 2 + 1, r);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = a; k <= z; ++k)
            if (run.mask >> k & 1u) {
                const float* const f = Y::partial(smem, k);
                const float w = slot_weight[k][r];
                const float2 u = *reinterpret_cast<const float2*>(f + at), v = *reinterpret_cast<const float2*>(f + next);
                s.x = fmaf(u.x, w, s.x);
                s.y = fmaf(u.y, w, s.y);
                s.z = fmaf(v.x, w, s.z);
                s.w = fmaf(v.y, w, s.w);
            }
        const float m = Y::partial(smem, a)[PC::m(r)], l = Y::partial(smem, a)[PC::l(r)];
        if (run.begins && run.ends) {
            const float f = l == 0.f ? 0.f : p.v_scale / l;
            if (c < p.d)
                *reinterpret_cast<uint2*>(p.o + (run.row + r) * p.d + c) =
                    make_uint2(ptx::pack_bf16x2(s.x * f, s.y * f), ptx::pack_bf16x2(s.z * f, s.w * f));
            if (c == 0) p.lse[run.row + r] = natural_lse(m, l);
        } else {
            float* const part = p.ws + ((int64_t)cta * 2 + (run.begins ? 1 : 0)) * PS::FLOATS;
            *reinterpret_cast<float4*>(part + PS::o(r) + c) = s;
            if (c == 0) {
                part[PS::m(r)] = m;
                part[PS::l(r)] = l;
            }
        }
    }
}

// Joins the pieces of the segment that begins in block blockIdx.x and ends in
// a later one: its own second piece and the first pieces of the blocks after.
// Every row is one block's; 8 groups of 32 threads take every eighth piece.
// Bound by its launch and two round trips to L2 (about 3 us); one block of 1024
// threads for all of a segment's rows saved 1 us where segments have two or
// three pieces and cost 8 us for one sequence in 152 pieces.
template <int D, int NT>
__global__ void __launch_bounds__(256) fa_qcache_combine_kernel(const DecParams p)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    constexpr int R = 8 * NT, V = D / 32;
    using PS = Partial<D, R>;
    const int cta = blockIdx.x, r = blockIdx.y;
    const int seg = p.desc[2 * cta];
    if (seg < 0) return;
    const int parts = p.desc[2 * cta + 1] - cta + 1;
    const int HR = p.hkv * p.rb;
    const int b = seg / HR, hr = seg - b * HR, h = hr / p.rb;
    const int row = (hr - h * p.rb) * R + r;
    if (row >= p.rows) return;
    const int grp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float mx = -INFINITY, l = 0.f, o[V] = {};
    for (int k = grp; k < parts; k += 8) {
        const float* const f = p.ws + ((int64_t)(cta + k) * 2 + (k == 0 ? 1 : 0)) * PS::FLOATS;
        const float mk = f[PS::m(r)], lk = f[PS::l(r)];
        const float mn = fmaxf(mx, mk);
        const float wa = mx == -INFINITY ? 0.f : ptx::ex2(mx - mn), wb = mk == -INFINITY ? 0.f : ptx::ex2(mk - mn);
        l = l * wa + lk * wb;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = o[e] * wa + f[PS::o(r) + lane * V + e] * wb;
        mx = mn;
    }
    __shared__ float sm[8], sl[8], so[8][D];
    if (lane == 0) sm[grp] = mx, sl[grp] = l;
#pragma unroll
    for (int e = 0; e < V; ++e) so[grp][lane * V + e] = o[e];
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= D) return;
    mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, sm[k]);
    float x = 0.f;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float w = sm[k] == -INFINITY ? 0.f : ptx::ex2(sm[k] - mx);
        l += sl[k] * w;
        x += so[k][c] * w;
    }
    const int64_t at = ((int64_t)b * p.hkv + h) * p.rows + row;
    if (c < p.d) p.o[at * p.d + c] = __float2bfloat16_rn(l == 0.f ? 0.f : x * (p.v_scale / l));
    if (c == 0) p.lse[at] = natural_lse(mx, l);
}

// ------------------------------------------------------------------ weights

// w_out[key] = w_in[key] + sum over the rows of the key's kv head of
// exp(scale q.k - lse): the attention weight that the rows gave each key,
// from the logsumexps that decode returned.  Only K is read.  Two blocks of 8
// warps an SM, a page a warp as in decode, but every unit is a page of a kv head
// with all its query rows, so a key's sum is one warp's and needs no atomics.
// 8 x 8 heads x 30000 to 32768 keys, 8 rows each, d = 128 (161 MB): 34.5 us, 0.69
// of the measured copy bandwidth; 5 us are the start, the rest is bound by
// instructions (about 700 a page with the warp's start spread over 13 pages).
template <int D>
struct WeightLayout {
    static constexpr int WARPS = 8, THREADS = WARPS * 32;
    static constexpr int SLOTS = D == 128 ? 2 : 4;
    static constexpr int RING = SLOTS * 36 * D;
    static constexpr int PREFIX = WARPS * RING;
    static constexpr int bytes(int B) { return PREFIX + (B + 1) * 4; }
    static_assert(2 * (bytes(MAX_B) + 2048) <= 232448, "shared memory of two blocks an SM");
};

template <int D, int NT>
__global__ void __launch_bounds__(WeightLayout<D>::THREADS, 2) fa_qcache_weights_kernel(const DecParams p)
{
    using Y = WeightLayout<D>;
    constexpr int WARPS = Y::WARPS, THREADS = Y::THREADS;
    extern __shared__ __align__(128) uint8_t smem[];
    int* const prefix = reinterpret_cast<int*>(smem + Y::PREFIX);
    __shared__ int scratch[WARPS];
    __shared__ __align__(8) uint64_t bars[WARPS * Y::SLOTS];
    __shared__ uint32_t abort_flags[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    if (lane < Y::SLOTS) ptx::mbar_init(ptx::smem_addr(&bars[warp * Y::SLOTS + lane]), 1);
    if (lane == 0) abort_flags[warp] = 0;
    volatile uint32_t* const abort_flag = &abort_flags[warp];
    ptx::fence_barrier_init();
    __syncwarp();
    prefetch_l2(p.table, (int64_t)p.B * p.max_pages * 4);
    prefetch_l2(p.q, (int64_t)p.B * p.hkv * p.rows * p.d * 2);
    prefetch_l2(p.lse_in, (int64_t)p.B * p.hkv * p.rows * 4);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    page_prefix<THREADS>(p.lens, p.B, p.max_pages, prefix, scratch);
    // One unit is a page of a kv head: all its row blocks, so that every key's weight is one warp's.
    Work work{prefix, p.B, p.hkv};
    // Places behind the sequences' ends.
    for (int64_t bh = blockIdx.x; bh < (int64_t)p.B * p.hkv; bh += gridDim.x) {
        const int b = (int)(bh / p.hkv);
        if (tid == 0 && bh % p.hkv == 0 && p.lens[b] > p.max_pages * (int64_t)PAGE) atomicOr(&g_status, STATUS_BAD_PAGE);
        if (p.w_out == p.w_in) continue;
        for (int64_t e = length_of(p.lens, b, p.max_pages) + tid; e < p.w_len; e += THREADS)
            p.w_out[bh * p.w_len + e] = p.w_in[bh * p.w_len + e];
    }
    const int T = work.total();
    const int all = gridDim.x * WARPS, G = min(all, T), me = blockIdx.x + gridDim.x * warp;
    if (me >= G) return;
    const int x0 = (int)((int64_t)me * T / G), x1 = (int)((int64_t)(me + 1) * T / G);
    Rows<D, NT> rows;
    uint64_t off[NT], sc[NT];  // of the lane's two columns: scores' factors, and -lse in base 2
    int have = -1;             // segment (with row block) whose rows are loaded
    Feed<D, Y::SLOTS, false, false> feed(smem + warp * Y::RING, ptx::smem_addr(&bars[warp * Y::SLOTS]), p, work);
    typename Rows<D, NT>::Raw raw;
    // A lane's part of the weights: keys 16t + g and 16t + 8 + g of a page,
    // fetched while the page before is worked on.
    auto weights_at = [&](int seg_, int page_) { return (int64_t)seg_ * p.w_len + page_ * PAGE + 16 * t + g; };
    float w_next[2] = {0.f, 0.f};
    auto fetch_weights = [&](int rbi, int seg_, int page_) {
        const float* const w = (rbi == 0 ? p.w_in : p.w_out) + weights_at(seg_, page_);
        const int64_t left = p.w_len - (page_ * PAGE + 16 * t + g);
        if (left > 0) w_next[0] = w[0];
        if (left > 8) w_next[1] = w[8];
    };
    // With one row block the warp goes through its run once.  With more, it goes
    // through one segment's pages once a row block, adding to what the last time
    // wrote (its own lanes did): a row block's query rows stay in registers.
    bool ok = true;
    for (int xa = x0, xb; ok && xa < x1; xa = xb) {
        xb = x1;
        if (p.rb > 1) {
            const Work::Unit u = work.at(xa);
            xb = min(x1, xa + u.pages - u.page);
        }
        for (int rbi = 0; ok && rbi < p.rb; ++rbi) {
            feed.start(xa, xb);
            int seg = feed.place(xa), page = feed.first_page;
            fetch_weights(rbi, seg, page);
            feed.begin();
            bool there = feed.there(xa);
            for (int x = xa; x < xb; ++x) {
                const float w_now[2] = {w_next[0], w_next[1]};
                bool there_next = false;
                int seg_next = seg, page_next = page;
                if (x + 1 < xb) {
                    seg_next = feed.place(x + 1);
                    there_next = feed.there(x + 1);
                    page_next = seg_next == seg ? page + 1 : 0;
                    fetch_weights(rbi, seg_next, page_next);
                }
                if (seg * p.rb + rbi != have) {
                    have = seg * p.rb + rbi;
                    const int b = seg / p.hkv, hr = (seg - b * p.hkv) * p.rb + rbi;
                    rows.fetch(raw, p, b, hr);
                    const float* const lse = p.lse_in + (int64_t)seg * p.rows;
                    float e[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = rbi * 8 * NT + nt * 8 + 2 * t + j;
                            // A row that saw nothing (or is none) gives nothing: 2^-inf.
                            e[nt][j] = r < p.rows ? lse[r] : -INFINITY;
                        }
                    rows.load(raw, p, hr);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) e[nt][j] = e[nt][j] == -INFINITY ? e[nt][j] : -e[nt][j] * 1.4426950408889634f;
                        off[nt] = ptx::f2_pack(e[nt][0], e[nt][1]);
                        sc[nt] = ptx::f2_pack(rows.sc[nt][0], rows.sc[nt][1]);
                    }
                }
                const uint8_t* const blk = feed.wait(abort_flag);
                if (!blk) {
                    ok = false;
                    break;
                }
                float sum[8] = {};
                if (there) {
                    // (8 x 8 heads x 32768 keys, 8 rows: 35.3 us with two groups together, 36.9 with one; decode and
                    // more rows have products of their own to fill the waits and lose registers.)
                    float s[4][NT][4];
                    page_scores<D, NT, NT == 1 ? 2 : 1>(blk, rows, s);
                    const bool whole = (page + 1) * PAGE <= rows.min_lim;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float x0_, x1_;
                                ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[r][nt][2 * half], s[r][nt][2 * half + 1]), sc[nt], off[nt]), x0_, x1_);
                                if (!whole) {
                                    const int key = page * PAGE + 16 * r + 8 * half + g;
                                    if (key >= rows.lim[nt][0]) x0_ = -INFINITY;
                                    if (key >= rows.lim[nt][1]) x1_ = -INFINITY;
                                }
                                sum[2 * r + half] += ptx::ex2(x0_) + ptx::ex2(x1_);
                            }
                        }
                }
                feed.next();
                // Sums over the four lanes that share a key's columns, each lane ending
                // with the two keys it writes: half of the keys change hands, then half
                // of those left.
                const bool up2 = t & 2, up1 = t & 1;
                float four[4], two[2];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    four[e] = (up2 ? sum[4 + e] : sum[e]) + __shfl_xor_sync(0xffffffffu, up2 ? sum[e] : sum[4 + e], 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    two[e] = (up1 ? four[2 + e] : four[e]) + __shfl_xor_sync(0xffffffffu, up1 ? four[e] : four[2 + e], 1);
                float* const w = p.w_out + weights_at(seg, page);
                const int64_t left = min((int64_t)rows.len, p.w_len) - (page * PAGE + 16 * t + g);
                if (left > 0) w[0] = w_now[0] + two[0];
                if (left > 8) w[8] = w_now[1] + two[1];
                seg = seg_next;
                page = page_next;
                there = there_next;
            }
        }
    }
    feed.drain(abort_flag);
}

// ----------------------------------------------------------------- eviction

struct EvictParams {
    uint8_t* pool;
    const int32_t *table, *lens, *table_out;
    const float* w_in;   // (B, hkv, w_len)
    float* w_out;
    int32_t *kept, *lens_out;
    int64_t w_len;
    int hkv, max_pages, max_pages_out, num_pages;
    int keep, sink, recent;
    int held;            // weights a block of the selection keeps in shared memory
    int move_blocks;     // blocks of a head's move (a cluster)
};

// Floats in the order of their values as unsigned integers: equal values
// (-0 and 0 among them) are equal, NaN comes last.
__device__ __forceinline__ uint32_t order_of(float w)
{
    if (!(w == w)) return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Thread-block clusters: the C blocks of one kv head of one sequence.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same in two halves, ordering no memory: for leaving shared memory that others read.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Reads an int of block `rank`'s shared memory.
__device__ __forceinline__ int cluster_read(const int* mine, int rank)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_addr(mine)), "r"(rank));
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

constexpr int SEL_THREADS = 512;
constexpr int SEL_BINS = 256;
// Weights that a block keeps in shared memory over its passes, at most (the
// rest are read again).
constexpr int SEL_HELD_MOST = 32768;

// Chooses the keys that stay: the first `sink`, the last `recent`, and of those
// between the keep - sink - recent with the largest weights (of equal weights
// the lowest places), found by radix selection: four histograms of 8 bits of
// order_of, largest digit first, give the smallest weight that stays and how
// many of that weight do.  A cluster of C blocks shares a kv head of a
// sequence, each block a run of the places and each warp a run of its block's;
// the histograms and the counts before a block's run are read from the other
// blocks' shared memory, so the result does not depend on timing.
//
// Bound by latency: a pass is a sweep over the block's weights, a cluster
// barrier and a look at 256 counts, about 2.5 us.  64 heads of 32768 keys: 22 us
// in clusters of 4 (of 8 and of 2, 5 us more).  Three digits of 11 bits need a
// pass less but 8 times as many counts of the other blocks: 109 us.
template <int C>
__global__ void __launch_bounds__(SEL_THREADS) fa_qcache_select_kernel(const EvictParams p)
{
    constexpr int W = SEL_THREADS / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t* const held = reinterpret_cast<uint32_t*>(smem);
    __shared__ int hist[2][SEL_BINS];  // two, in turn: one is read by the cluster while the other is cleared
    __shared__ int found[2];
    __shared__ int sums[W];
    __shared__ int counts[2];          // this block's larger and equal ones
    __shared__ int warp_gt[W], warp_eq[W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? blockIdx.x % C : 0, h = blockIdx.x / C, b = blockIdx.y;
    for (int e = tid; e < 2 * SEL_BINS; e += SEL_THREADS) (&hist[0][0])[e] = 0;
    if (tid < 2) counts[tid] = 0;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t bh = (int64_t)b * p.hkv + h;
    const int len = length_of(p.lens, b, p.max_pages);
    const int count = min(len, p.keep);
    const float* const w = p.w_in + bh * p.w_len;
    float* const wo = p.w_out + bh * p.w_len;
    int32_t* const kept = p.kept + bh * p.keep;
    auto weight = [&](int x) { return x < p.w_len ? w[x] : 0.f; };
    auto put = [&](int at, int x, float v) {
        kept[at] = x;
        if (at < p.w_len) wo[at] = v;
    };
    // The weight that order_of made u of (NaN and the zeros, whose bits it does not keep, are read again).
    auto weight_of = [&](uint32_t u, int x) {
        return u == 0u || u == 0x80000000u ? weight(x) : __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
    };
    const int all = C * SEL_THREADS, me = rank * SEL_THREADS + tid;
    if (h == 0 && me == 0) {
        p.lens_out[b] = count;
        if (p.lens[b] > p.max_pages * (int64_t)PAGE) atomicOr(&g_status, STATUS_BAD_PAGE);
    }
    const bool cut = len > p.keep;
    const int first = p.sink, last = len - p.recent;  // the choice lies between
    int need = p.keep - p.sink - p.recent;
    // What needs no choice, written last: a barrier would wait for the stores.
    auto rest = [&] {
        for (int64_t e = count + me; e < p.w_len; e += all) wo[e] = 0.f;
        for (int e = count + me; e < p.keep; e += all) kept[e] = -1;
        for (int e = me; e < (cut ? p.sink : len); e += all) put(e, e, weight(e));
        if (!cut) return;
        for (int e = me; e < p.recent; e += all) put(p.keep - p.recent + e, last + e, weight(last + e));
    };
    if (cut && need > 0) {  // (the whole cluster)
        // This block's run of places, and each of its threads' view of their order.
        const int n = last - first;
        const int lo = first + (int)((int64_t)n * rank / C), hi = first + (int)((int64_t)n * (rank + 1) / C), size = hi - lo;
        auto order = [&](int e) { return e < p.held ? held[e] : order_of(weight(lo + e)); };
        for (int e0 = tid; e0 < min(size, p.held); e0 += 8 * SEL_THREADS) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = e0 + i * SEL_THREADS < size ? weight(lo + e0 + i * SEL_THREADS) : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i * SEL_THREADS < min(size, p.held)) held[e0 + i * SEL_THREADS] = order_of(x[i]);
        }
        __syncthreads();

        uint32_t prefix = 0, mask = 0;
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            int* const mine = hist[pass & 1];
            auto add = [&](uint32_t u) {
                if ((u & mask) == prefix) atomicAdd(&mine[u >> shift & 255u], 1);
            };
#pragma unroll 4
            for (int e = tid; e < min(size, p.held); e += SEL_THREADS) add(held[e]);
            for (int e = p.held + tid; e < size; e += SEL_THREADS) add(order_of(weight(lo + e)));
            if constexpr (C > 1) cluster_sync();
            else __syncthreads();
            // A pair of threads a digit, from the largest down, half of the blocks each.
            const int digit = 255 - tid / 2;
            int c = 0;
            if constexpr (C > 1) {
#pragma unroll
                for (int k = 0; k < C / 2; ++k) c += cluster_read(&mine[digit], tid % 2 * (C / 2) + k);
            } else {
                c = tid % 2 ? 0 : mine[digit];
            }
            c += __shfl_xor_sync(0xffffffffu, c, 1);
            int upto = tid % 2 ? 0 : c;  // sums over the digits, each once
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) sums[warp] = upto;
            __syncthreads();
            int before = 0;
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (k < warp) before += sums[k];
            const int above = before + upto - c;
            if (tid % 2 == 0 && above < need && need <= above + c) {
                found[0] = digit;
                found[1] = need - above;
            }
            // The other histogram is read by no block any more: all have passed this pass's cluster barrier.
            for (int e = tid; e < SEL_BINS; e += SEL_THREADS) hist[~pass & 1][e] = 0;
            __syncthreads();
            prefix |= (uint32_t)found[0] << shift;
            mask |= 255u << shift;
            need = found[1];
        }
        // Everything above `prefix` stays, and the first `need` equal to it.  Each
        // warp counts its run, then places it.
        const int wlo = (int)((int64_t)size * warp / W), whi = (int)((int64_t)size * (warp + 1) / W);
        int gt = 0, eq = 0;
#pragma unroll 4
        for (int e = wlo + lane; e < whi; e += 32) {
            const uint32_t u = order(e);
            gt += u > prefix;
            eq += u == prefix;
        }
        gt = __reduce_add_sync(0xffffffffu, gt);
        eq = __reduce_add_sync(0xffffffffu, eq);
        if (lane == 0) {
            warp_gt[warp] = gt, warp_eq[warp] = eq;
            atomicAdd(&counts[0], gt);
            atomicAdd(&counts[1], eq);
        }
        __syncthreads();
        int base = 0, base_eq = 0;
        if constexpr (C > 1) {
            cluster_sync();
            for (int k = 0; k < rank; ++k) {
                base += cluster_read(&counts[0], k);
                base_eq += cluster_read(&counts[1], k);
            }
        }
        for (int k = 0; k < warp; ++k) {
            base += warp_gt[k];
            base_eq += warp_eq[k];
        }
        for (int e0 = wlo; e0 < whi; e0 += 32) {
            const int e = e0 + lane;
            const uint32_t u = e < whi ? order(e) : 0u;
            const bool is_gt = e < whi && u > prefix, is_eq = e < whi && u == prefix;
            const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me_ = __ballot_sync(0xffffffffu, is_eq);
            const uint32_t below = (1u << lane) - 1u;
            const int ng = base + __popc(mg & below), ne = base_eq + __popc(me_ & below);
            if (is_gt || (is_eq && ne < need)) put(p.sink + ng + min(ne, need), lo + e, weight_of(u, lo + e));
            base += __popc(mg);
            base_eq += __popc(me_);
        }
        if constexpr (C > 1) cluster_arrive_relaxed();
    }
    rest();
    if constexpr (C > 1) {  // no block leaves while its shared memory may be read
        if (cut && p.keep - p.sink - p.recent > 0) cluster_wait();
    }
}

// Moves the kept rows to the front.  A cluster of up to 8 blocks shares a kv
// head of a sequence; in a round each block gathers up to MOVE_PAGES pages of
// the destination into shared memory, the cluster meets, and all write.  The
// destination's pages may be the sequence's own: row j comes from place
// kept[j] >= j, so what a round writes no later round reads, and what it
// overwrites has been read by then (its own and earlier rounds' rows).
// Bound by memory: a row touches 384 bytes of sectors for its 144; 64 heads cut
// to 4096 of 32768 keys (d = 128, 100 MB of sectors read, 38 MB written) in 25 us.
constexpr int MOVE_PAGES = 4, MOVE_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(MOVE_THREADS) fa_qcache_move_kernel(const EvictParams p)
{
    using L = Block<D>;
    constexpr int ROWS = MOVE_PAGES * PAGE;
    static_assert(ROWS == MOVE_THREADS, "a thread looks up a row");
    extern __shared__ __align__(128) uint8_t smem[];  // MOVE_PAGES blocks
    __shared__ int src_blk[ROWS], src_row[ROWS];
    __shared__ int out_blk[MOVE_PAGES];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int blocks = p.move_blocks, rank = blockIdx.x % blocks, h = blockIdx.x / blocks, b = blockIdx.y, tid = threadIdx.x;
    const int64_t bh = (int64_t)b * p.hkv + h;
    const int len = length_of(p.lens, b, p.max_pages), count = min(len, p.keep);
    // (The whole cluster.)  One table, rows of one pitch: nothing moves.
    if (len <= p.keep && p.table_out == p.table && p.max_pages_out == p.max_pages) return;
    const int pages = (count + PAGE - 1) / PAGE;
    // Pages of the block in a round: rank, rank + blocks, ... of the round's.
    for (int r0 = 0; r0 < pages; r0 += blocks * MOVE_PAGES) {
        {
            const int page = r0 + rank + blocks * (tid / PAGE), x = page * PAGE + tid % PAGE;
            int blk = -1, row = 0;
            if (x < count) {
                const int s = p.kept[bh * p.keep + x];
                const int id = page_of(p.table, p.max_pages, p.num_pages, b, s / PAGE);
                if (id >= 0) blk = id * p.hkv + h, row = s % PAGE;
                else atomicOr(&g_status, STATUS_BAD_PAGE);
            }
            src_blk[tid] = blk;
            src_row[tid] = row;
            if (tid % PAGE == 0) {
                int out = -1;
                if (page < pages) {
                    const int id = page_of(p.table_out, p.max_pages_out, p.num_pages, b, page);
                    if (id >= 0) out = id * p.hkv + h;
                    else atomicOr(&g_status, STATUS_BAD_PAGE);
                }
                out_blk[tid / PAGE] = out;
            }
        }
        __syncthreads();
        auto block = [&](int i) { return p.pool + (int64_t)i * L::BYTES; };
        // All of a thread's loads before its first store.
        // K: a quarter of a row and its scales to a thread.
        constexpr int NK = ROWS * 4 / MOVE_THREADS, NV = ROWS / 2 * L::NB / MOVE_THREADS;
        {
            Chunk<D / 8> code[NK];
            uint16_t sc[NK];
            const int t = tid % 4;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int r = (i * MOVE_THREADS + tid) / 4, from = src_blk[r], x = src_row[r];
                sc[i] = 0;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) code[i].w[k] = 0;
                if (from >= 0) {
                    const uint8_t* const blk = block(from);
                    code[i].load(blk + L::kcode(x) + t * (D / 8));
                    const uint8_t* const at = blk + L::kscale(x, t * L::P);
                    sc[i] = D == 128 ? *reinterpret_cast<const uint16_t*>(at) : *at;
                }
            }
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int r = (i * MOVE_THREADS + tid) / 4, x = r % PAGE;
                uint8_t* const buf = smem + r / PAGE * L::BYTES;
                code[i].store(buf + L::kcode(x) + t * (D / 8));
                if (D == 128) *reinterpret_cast<uint16_t*>(buf + L::kscale(x, t * L::P)) = sc[i];
                else buf[L::kscale(x, t)] = (uint8_t)sc[i];
            }
        }
        // V: a channel block of two rows to a thread.
        {
            uint4 v[NV][2];
            uint8_t sc[NV][2];
            const int c = tid % L::NB;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const int r = 2 * ((i * MOVE_THREADS + tid) / L::NB) + odd, from = src_blk[r], x = src_row[r];
                    v[i][odd] = make_uint4(0, 0, 0, 0);
                    sc[i][odd] = 0;
                    if (from >= 0) {
                        const uint8_t* const blk = block(from);
                        v[i][odd] = *reinterpret_cast<const uint4*>(blk + L::vcode(x) + c * 16);
                        sc[i][odd] = blk[L::vscale(x, c)];
                    }
                }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int r = 2 * ((i * MOVE_THREADS + tid) / L::NB), x = r % PAGE;
                const int s0 = src_row[r] % 2 * 4, s1 = src_row[r + 1] % 2 * 4;
                auto both = [&](uint32_t a, uint32_t e) { return (a >> s0 & 0x0F0F0F0Fu) | (e >> s1 & 0x0F0F0F0Fu) << 4; };
                const uint4 &a = v[i][0], &e = v[i][1];
                uint8_t* const buf = smem + r / PAGE * L::BYTES;
                *reinterpret_cast<uint4*>(buf + L::vcode(x) + c * 16) = make_uint4(both(a.x, e.x), both(a.y, e.y), both(a.z, e.z), both(a.w, e.w));
                *reinterpret_cast<uint16_t*>(buf + L::vscale(x, c)) = (uint16_t)(sc[i][0] | sc[i][1] << 8);
            }
        }
        cluster_sync();  // every block's rows are read
        for (int i = tid; i < MOVE_PAGES * L::BYTES / 16; i += MOVE_THREADS) {
            const int q = i / (L::BYTES / 16), at = i % (L::BYTES / 16);
            if (out_blk[q] >= 0) reinterpret_cast<uint4*>(block(out_blk[q]))[at] = reinterpret_cast<const uint4*>(smem)[i];
        }
        __syncthreads();  // out_blk and smem are free
    }
}

}  // namespace qc
}  // namespace fa
