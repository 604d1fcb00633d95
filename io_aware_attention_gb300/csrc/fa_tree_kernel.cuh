// Attention of many query rows over the 4-bit cache for sm_103a: the rows of a
// tree of drafted tokens (T drafts times the heads of a group) against one kv head.
//
// Everything is computed transposed, so that the stored values reach the tensor
// cores without passing through shared memory again and few rows waste no tensor
// work.  For a tile of 128 keys (two pages) and N query rows:
//
//   S^T = K Q^T     M = 128 keys (TMEM lanes), N rows, K = D     A = K from TMEM, B = Q in shared memory
//   P   = 2^(S * scale - max + SHIFT)                            one thread a key and N / 2 rows
//   O^T += V^T P^T  M = D channels (TMEM lanes), N rows, K = 128 A = V^T from TMEM, B = P^T in shared memory
//
// K codes of one key are neighbours in a page, and V codes of one channel come as
// pairs of keys, so a thread turns a key's codes (a few channels' of some pairs) into
// 16-bit operands in registers and stores them to TMEM lanes.  e2m1 * e4m3 is exact in
// fp16.  The maximum over keys runs across TMEM lanes and threads, which is dear:
// the reference of a row is kept until a score exceeds it by more than 2^RISE, which one
// barrier with a reduction (128 threads) tells; only then is the maximum taken and
// what has been summed scaled.
//
// A probability is one fp16 number (11 bits) of at most 2^(SHIFT + RISE) = 2^15, its sum
// fp32 over the unrounded ones: a result is off by at most 2^-11 of sum p |v|, an eighth
// of its own rounding to bf16 where terms do not cancel.  A row's largest probability is
// 2^SHIFT at least, so those below 2^-21 of it are fp16 subnormals, off by up to half a
// step, 2^-25, which is 2^-32 of the largest, and below that they are 0: another
// 2^-32 max p sum |v|, which shows where the heaviest keys hold 0 in a channel.  (Two numbers a
// probability, as with few rows, would double the products and the traffic of P in
// shared memory.  The form of the decode kernel that had them took 217 us where this one
// takes 139, 16 rows x 8 x 32 heads x 16384 keys, and 962 for 244 with 256 rows x 16 x 8
// heads x 3000 to 16384 keys.)
//
// Softmax of a tile is a long chain of short steps (waits, loads from TMEM, the vote,
// stores), so four groups of warps are at it at once: with many rows they share a tile's
// rows, with few rows they take tiles in turn, each with references, sums and an O^T of
// its own, which meet at a segment's end.  (N rows: tiles in flight x rows of a thread.
// 16: 4 x 16, 32: 4 x 32, 64: 2 x 32, 128: 1 x 32.  Two groups that shared the rows of
// every tile took 1740 cycles a tile of 16 rows and 4200 of 128.)
//
// Warps (1024 threads, one block an SM):
//   0-15      softmax, four groups: a thread a key; at a segment's end they write its result.
//   16-27     codes: three sets that take tiles in turn, from shared memory to fp16 in TMEM,
//             K a thread a key, then V.  (4 warps for K and 8 for V, every tile: V's, busy
//             for 1100 cycles a tile, held up the rest; 16 rows x 8 x 32 heads x 16384 keys
//             149 us, 139 with the sets.)
//   28        pages from the cache into a ring (bulk copies), and what the other roles
//             need to know of each tile.
//   29, 30    the two products (an elected lane each); 29 also allocates TMEM.
//   31        query rows of the next segment: from TMA to fp16 in place, all scaled by the
//             power of two that puts their largest entry into [2^14, 2^15): bf16 entries
//             down to 2^-31 of it stay exact, smaller ones are off by at most 2^-39 of it
//             (half of fp16's smallest step, 2^-25, against 2^14).
//             Where a row's own largest entry is more than 2^15 times smaller, every row
//             gets a power of its own (APART), and the softmax warps bring its scores back; they
//             also do the first segment's rows.
//
// TMEM columns: [0, 128) two K tiles, [128, 256) two V tiles, then the tiles of S^T in
// flight and their O^T.  At D = 64 V^T has 64 rows: the upper lanes hold anything, and
// their results are not read.
//
// The tiles of all sequences, kv heads and row blocks are one list (see Work), of
// which every block takes an equal run (see Units); segments that cross
// blocks leave partial results that the combine kernel joins.  A block's pipeline runs on across segments.
//
// The roles' loops share the SM's instruction caches: what does not fit is fetched at
// some 20 cycles an instruction, and the first form of this kernel, with everything
// unrolled and inlined, spent most of its time on that (16 rows x 8 x 32 heads x 16384
// keys: 485 us).  So hot loops are short, rare paths are rolled up and branched
// around.
//
// Every wait is bounded in time (see fa_fwd_kernel.cuh); after an abort the roles
// leave their loops, the softmax warps that share barriers together, which agree on it
// where they vote.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fa_fwd_kernel.cuh"
#include "fa_qcache_kernel.cuh"
#include "ptx.cuh"

namespace fa {
namespace tree {

using qc::DecParams;
using qc::PAGE;

constexpr int TILE = 2 * PAGE;
constexpr int THREADS = 1024, GROUPS = 4, SOFTMAX_WARPS = 4 * GROUPS;
constexpr int WARP_CODES = 16, SETS = 3, WARP_COPY = 28, WARP_S = 29, WARP_O = 30, WARP_Q = 31;
constexpr int NOTES = 16;
constexpr float SHIFT = 7.0f, RISE = 8.0f;
constexpr int APART = 15, TOGETHER = 1 << 20;  // binades; "power" of rows that share one
constexpr float UNSET = 3e38f;  // added to a row's scores before it has a reference: any finite one exceeds it
constexpr uint32_t TM_K = 0, TM_V = 128, TM_S = 256, TM_COLS = 512;
constexpr uint32_t NB_VOTE = 1, NB_GROUP = 5, NB_END = 9, NB_ALL = 13;  // + group, group, rows' share
// Registers a thread after the split; launched with 64 (65536 / 1024).
constexpr uint32_t REGS_SOFTMAX = 88, REGS_CODES = 40, REGS_OTHER = 32;
static_assert(512 * REGS_SOFTMAX + 128 * SETS * REGS_CODES + 128 * REGS_OTHER <= 65536, "register split");

template <int D, int N>
struct Layout {
    static_assert((D == 64 || D == 128) && (N == 16 || N == 32 || N == 64 || N == 128), "sizes");
    static constexpr int TURNS = N <= 32 ? 4 : N == 64 ? 2 : 1;  // tiles in flight
    static constexpr int SHARES = GROUPS / TURNS;                // groups that share a tile's rows
    static constexpr int NC = N / SHARES;                        // rows of a thread
    static constexpr int NO = NC / TURNS;                        // rows whose results a group writes
    // Where a tile has all groups' rows, the products are made in two streams of half
    // the rows each, which need not keep step: one's exponentials run beside the other's
    // loads and waits.
    static constexpr int STREAMS = TURNS == 1 ? 2 : 1, NM = N / STREAMS;  // rows of a product
    static constexpr int PBUFS = TURNS == 1 ? 2 : TURNS;
    static constexpr int EXTRA = TURNS == 1 ? 2 : 4;
    // Tiles' codes on their way: as many for each set of warps that takes them, so that
    // a stage's next tile is waited for by the warps that emptied it.
    static constexpr int RAW_STAGES = N == 128 ? SETS : 2 * SETS;
    static_assert(NOTES >= RAW_STAGES + 2 + SETS, "notes");
    // Tiles whose products are done, told of in turn by EMPTIES barriers: a set that
    // waits for tile g - 2 left tile g - 3 when the products of g - 5 were done, so of
    // the barrier's earlier tiles (g - 2 - EMPTIES) none is out, and its parity is clear.
    static constexpr int EMPTIES = 2 * SETS;
    static constexpr uint32_t TM_O = TM_S + TURNS * N;
    static_assert(TM_O + TURNS * N <= TM_COLS && NO % 4 == 0, "TMEM");
    static constexpr uint32_t QBLK = N * 128;              // 64 channels of the rows
    static constexpr uint32_t Q_BYTES = QBLK * (D / 64);
    static constexpr uint32_t PBLK = TILE * 128;           // 64 rows of a tile's probabilities
    static constexpr uint32_t P_BYTES = PBLK * (N == 128 ? 2 : 1);
    static constexpr uint32_t PAGE_BYTES = 72 * D, RAW_BYTES = 2 * PAGE_BYTES;
    static constexpr uint32_t OFF_P = 0;
    static constexpr uint32_t OFF_Q = OFF_P + PBUFS * P_BYTES;
    static constexpr uint32_t OFF_RAW = OFF_Q + 2 * Q_BYTES;
    // Per group: what is added to the rows' scores; their words, references, sums and
    // corrections; of every warp its maxima or sums.
    static constexpr uint32_t OFF_PAR = OFF_RAW + RAW_STAGES * RAW_BYTES;
    static constexpr uint32_t OFF_WORD = OFF_PAR + GROUPS * NC * 4;  // the rows' words
    static constexpr uint32_t OFF_REF = OFF_WORD + GROUPS * NC * 8;
    static constexpr uint32_t OFF_SUM = OFF_REF + GROUPS * NC * 4;
    static constexpr uint32_t OFF_CORR = OFF_SUM + GROUPS * NC * 4;
    static constexpr uint32_t OFF_WARP = OFF_CORR + GROUPS * NC * 4;
    static constexpr uint32_t OFF_APART = OFF_WARP + GROUPS * NC * 16;  // exponents, where rows have powers of their own
    static constexpr uint32_t OFF_LARGEST = OFF_APART + GROUPS * NC * 4;  // the two query blocks' rows' largest entries
    static constexpr uint32_t OFF_QSC = OFF_LARGEST + 2 * N * 4;  // their factors to base-2 scores and powers
    static constexpr uint32_t OFF_FACTORS = OFF_QSC + 16;      // the V warps' scales
    static constexpr uint32_t OFF_NOTES = OFF_FACTORS + 4 * SETS * 512;
    static constexpr uint32_t OFF_BAR = OFF_NOTES + NOTES * 8;
    static constexpr int B_RAWFULL = 0, B_RAWEMPTY = B_RAWFULL + RAW_STAGES, B_KFULL = B_RAWEMPTY + RAW_STAGES, B_KEMPTY = B_KFULL + 2,
                         B_VFULL = B_KEMPTY + EMPTIES, B_VEMPTY = B_VFULL + 2, B_QRAW = B_VEMPTY + EMPTIES, B_QFULL = B_QRAW + 2, B_QEMPTY = B_QFULL + 2,
                         B_SFULL = B_QEMPTY + 2, B_SREAD = B_SFULL + 4, B_PFULL = B_SREAD + 4, B_PDONE = B_PFULL + 4,
                         B_OFREE = B_PDONE + 4, B_DRAIN = B_OFREE + 1, NUM_BARS = B_DRAIN + 2;
    static constexpr uint32_t OFF_MISC = OFF_BAR + NUM_BARS * 8;  // TMEM base, abort
    static constexpr uint32_t OFF_PREFIX = OFF_MISC + 16;
    static_assert(OFF_Q % 1024 == 0 && OFF_RAW % 16 == 0 && OFF_PAR % 16 == 0 && OFF_WORD % 16 == 0 && OFF_FACTORS % 16 == 0 && OFF_NOTES % 8 == 0 && OFF_BAR % 8 == 0 && OFF_MISC % 8 == 0,
                  "alignment");
    __host__ __device__ static constexpr uint32_t bytes(int B) { return OFF_PREFIX + (uint32_t)(B + 1) * 4; }
    static_assert(OFF_PREFIX + (qc::MAX_B + 1) * 4 <= 232448, "shared memory");
};

// kind::f16 with fp16 A and B, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major)
{
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Meets the `count` threads of barrier `id`; whether any of them said yes.
__device__ __forceinline__ bool any_of(uint32_t id, uint32_t count, bool yes)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id), "r"(count)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// As warp_wait_bar, the usual case first: five roles of straight-line code share the
// instruction caches.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort_flag, uint32_t code)
{
    if (__builtin_expect(__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)), 1)) return true;
    uint64_t t0 = 0;
    for (uint32_t polls = 1;; ++polls) {
        if (__builtin_expect(__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, WAIT_SLEEP_NS)), 1)) return true;
        if (__builtin_expect((polls & 255u) == 0u, 0)) {
            if (__any_sync(0xffffffffu, *abort_flag != 0u)) return false;
            const uint64_t t = ptx::globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (__any_sync(0xffffffffu, t - t0 > limit_ns)) {
                record_timeout(code, abort_flag);
                return false;
            }
        }
    }
}

// C columns of this warp's lanes and their largest, as tcgen05.ld.red gives it (valid
// after load_cols_end).
template <int C>
__device__ __forceinline__ void load_cols_max(uint32_t taddr, uint32_t (&r)[C], float& red)
{
    static_assert(C == 16 || C == 32, "columns");
    if constexpr (C == 32)
        asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                     "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                       "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
                       "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
                       "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(red)
                     : "r"(taddr));
    else
        asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
                     "%16, [%17];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                       "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(red)
                     : "r"(taddr));
}

// TMEM <-> registers, C columns of this warp's lanes.
template <int C>
__device__ __forceinline__ void load_cols_begin(uint32_t taddr, uint32_t (&r)[C])
{
    if constexpr (C == 32) ptx::tmem_ld32(taddr, r);
    else if constexpr (C == 16) ptx::tmem_ld16(taddr, r);
    else ptx::tmem_ld8(taddr, r);
}
template <int C>
__device__ __forceinline__ void load_cols_end(uint32_t (&r)[C])
{
    if constexpr (C == 32) {
        ptx::tmem_wait_ld(r);
    } else {
        ptx::tmem_wait_ld_only();
        if constexpr (C == 16) ptx::reg_fence16(r);
        else ptx::reg_fence8(r);
    }
}
template <int C>
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&r)[C])
{
    load_cols_begin<C>(taddr, r);
    load_cols_end<C>(r);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }

// The keys of a tile in the order of TMEM lanes, rows of P^T and columns of V^T: lane
// r of a page's 64 holds key 8 (r / 2 % 8) + 2 (r / 16) + r % 2, which makes the pairs
// of keys whose V scales adjoin in a page (pairs q, q + 4, ...) neighbouring columns.
__device__ __forceinline__ int key_of(int r) { return (r >> 1 & 7) * 8 + (r >> 4 & 3) * 2 + (r & 1); }

// The channel, of a warp's 32, that TMEM lane r of V^T (and of O^T) holds.
__device__ __forceinline__ int channel_of(int r) { return (r & 7) * 4 + (r >> 3); }

// x, the same in every lane, by an instruction whose result the compiler knows to be:
// loops and addresses made of it run on the uniform datapath, and the products'
// operands need no moves there (8 products of a loop that lacked it took 690 cycles
// to issue, 120 with it).
__device__ __forceinline__ int uniform(int x) { return (int)__reduce_max_sync(0xffffffffu, (unsigned)x); }

// A block's run of tiles is cut into segments: tiles of one sequence, kv head and row
// block.  What the roles need to know of a tile, as the copying warp leaves it.
struct Note {
    enum : uint32_t { PAGE0 = 1, PAGE1 = 2, FIRST = 4, LAST = 8, INDEX = 4 };  // from bit INDEX on: its place in the segment, up to 15
    uint32_t what;  // which pages are there; first and last tile of its segment
    int left;       // keys of the sequence from the tile's first on
};

// The work's division.  A segment counts `extra` units more than its tiles, for its rows,
// first maxima and result, which cost about as much; none where blocks have few tiles
// anyway.  The list: sequence 0's (kv heads x row blocks), each its extra units, then its
// tiles, and so on.
struct Units {
    const int* prefix;  // sums of the sequences' tiles
    int B, hr, extra;
    __device__ __forceinline__ int before(int b) const { return prefix[b] + extra * b; }  // a (kv head, row block)'s units
    __device__ __forceinline__ int total() const { return before(B) * hr; }
    struct Place {
        int b, hr, at, tiles;  // at: unit of the segment
    };
    __device__ __forceinline__ Place find(int x) const
    {
        const int y = x / hr;
        int lo = 0, hi = B;  // before(lo) <= y < before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before(mid) <= y) lo = mid;
            else hi = mid;
        }
        Place u;
        u.b = lo;
        u.tiles = prefix[lo + 1] - prefix[lo];
        const int rem = x - before(lo) * hr, units = u.tiles + extra;
        u.hr = rem / units;
        u.at = rem - u.hr * units;
        return u;
    }
    // Tiles before unit x.
    __device__ __forceinline__ int tiles_before(int x) const
    {
        if (x >= total()) return prefix[B] * hr;
        const Place u = find(x);
        return prefix[u.b] * hr + u.hr * u.tiles + max(0, u.at - extra);
    }
};
// The next segment with tiles of a run x .. end - 1 of units; x moves behind it.
struct Run {
    int b, hr, tile0, n, tiles;
};
__device__ __forceinline__ bool next_run(const Units& work, int& x, int end, Run& r)
{
#pragma unroll 1
    while (x < end) {
        const Units::Place u = work.find(x);
        const int at = uniform(u.at), tiles = uniform(u.tiles), units = min(end - x, tiles + work.extra - at);
        const int tile0 = max(0, at - work.extra), tile1 = max(0, at + units - work.extra);
        x += units;
        if (tile1 == tile0) continue;
        r.b = uniform(u.b), r.hr = uniform(u.hr), r.tile0 = tile0, r.n = tile1 - tile0, r.tiles = tiles;
        return true;
    }
    return false;
}

// What the softmax warps need to know of a query block's scaling.
__device__ __forceinline__ void set_scaling(uint32_t at, float scale_log2, int power, bool apart)
{
    sts_f32(at, scale_log2 * __uint_as_float((uint32_t)(127 - power) << 23));
    sts_f32(at + 4, __int_as_float(apart ? power : TOGETHER));
}

// Query rows in shared memory (K-major, 128-byte swizzle), BATCH rows at a time, every
// step-th such batch: each row's largest magnitude (bf16 bits), and the rows to fp16 in place.
template <int D, int N>
struct QueryRows {
    static constexpr int PER = D / 32, BATCH = 4;  // channels a lane
    uint32_t q, largest_at;
    int first, step;
    __device__ __forceinline__ uint32_t at(int r) const
    {
        const int c = (threadIdx.x & 31) * PER;
        return q + (uint32_t)(c >> 6) * (N * 128) + (uint32_t)r * 128 + (uint32_t)((((c & 63) >> 3) ^ (r & 7)) * 16 + (c & 7) * 2);
    }
    __device__ __forceinline__ void load(int r, uint32_t (&w)[PER / 2]) const
    {
        if constexpr (PER == 4) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at(r)));
        else asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at(r)));
    }
    __device__ __forceinline__ uint32_t row_largest(int r) const
    {
        uint32_t am;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(am) : "r"(largest_at + (uint32_t)r * 4));
        return am;
    }
    __device__ __forceinline__ void measure() const
    {
#pragma unroll 1
        for (int r0 = first * BATCH; r0 < N; r0 += step * BATCH) {
            uint32_t w[BATCH][PER / 2], am[BATCH];
#pragma unroll
            for (int e = 0; e < BATCH; ++e) load(r0 + e, w[e]);
#pragma unroll
            for (int e = 0; e < BATCH; ++e) {
                am[e] = 0;
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) am[e] = max(am[e], max(w[e][i] & 0x7FFFu, w[e][i] >> 16 & 0x7FFFu));
            }
#pragma unroll
            for (int e = 0; e < BATCH; ++e) am[e] = __reduce_max_sync(0xffffffffu, am[e]);
            if ((threadIdx.x & 31) == 0)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(largest_at + (uint32_t)r0 * 4), "r"(am[0]), "r"(am[1]), "r"(am[2]),
                             "r"(am[3])
                             : "memory");
        }
        __syncwarp();
    }
    // The power of two that puts a largest entry (bits am) into [2^14, 2^15).
    static __device__ __forceinline__ int power(uint32_t am)
    {
        const int ex = (int)(am >> 7) - 127;
        return am > 0 && ex < 128 ? min(126, max(-126, 14 - ex)) : 0;
    }
    // The power of all rows' largest finite entry, and whether a row's is too far below it.
    // (Rows that are zero count for neither, and rows with infinities or NaN, whose results
    // are NaN in any scaling.)
    __device__ __forceinline__ int power_of_all(bool& apart) const
    {
        uint32_t high = 0, low = 0x7F80u;
#pragma unroll
        for (int e = 0; e < (N + 31) / 32; ++e) {
            const uint32_t am = row_largest((e * 32 + (int)(threadIdx.x & 31)) % N);
            if (am > 0 && am < 0x7F80u) high = max(high, am), low = min(low, am);
        }
        high = __reduce_max_sync(0xffffffffu, high);
        low = __reduce_min_sync(0xffffffffu, low);
        apart = (int)(high >> 7) - (int)(low >> 7) > APART;
        return power(high);
    }
    __device__ __forceinline__ void convert(int power_, bool apart) const
    {
        float up = __uint_as_float((uint32_t)(127 + power_) << 23);
#pragma unroll 1
        for (int r0 = first * BATCH; r0 < N; r0 += step * BATCH) {
            uint32_t w[BATCH][PER / 2];
#pragma unroll
            for (int e = 0; e < BATCH; ++e) load(r0 + e, w[e]);
#pragma unroll
            for (int e = 0; e < BATCH; ++e) {
                if (apart) up = __uint_as_float((uint32_t)(127 + power(row_largest(r0 + e))) << 23);
#pragma unroll
                for (int i = 0; i < PER / 2; ++i)
                    w[e][i] = qc::pack_h2(__uint_as_float(w[e][i] << 16) * up, __uint_as_float(w[e][i] & 0xFFFF0000u) * up);
                if constexpr (PER == 4) asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at(r0 + e)), "r"(w[e][0]), "r"(w[e][1]) : "memory");
                else asm volatile("st.shared.b32 [%0], %1;" ::"r"(at(r0 + e)), "r"(w[e][0]) : "memory");
            }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
    }
};

// The sums of C columns over a warp's lanes, to lane l that of column l % C: every step
// hands half of the columns to the lane across.
template <int C>
__device__ __forceinline__ float spread_sum(float (&v)[C])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = C / 2; m > 0; m >>= 1) {
#pragma unroll
        for (int c = 0; c < C / 2; ++c) {
            if (c >= m) continue;
            const bool up = lane & m;
            const float give = up ? v[c] : v[c + m], keep = up ? v[c + m] : v[c];
            v[c] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
#pragma unroll
    for (int m = C; m < 32; m <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
    return v[0];  // of column lane % C
}

// Joins the pieces of the segment that begins in block blockIdx.x and ends in a later
// one: its own second piece and the first pieces of the blocks after.  A warp a row,
// its lanes D / 32 channels each.
constexpr int JOIN_ROWS = 8;

template <int D, int N>
__global__ void __launch_bounds__(32 * JOIN_ROWS) fa_tree_combine_kernel(const DecParams p)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    using PS = qc::Partial<D, N>;
    constexpr int PER = D / 32;
    const int cta = blockIdx.x, r = blockIdx.y * JOIN_ROWS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int seg = p.desc[2 * cta];
    if (seg < 0) return;
    const int parts = p.desc[2 * cta + 1] - cta + 1;
    const int hr_all = p.hkv * p.rb, b = seg / hr_all, hr = seg - b * hr_all, h = hr / p.rb;
    const int row = (hr - h * p.rb) * N + r;
    if (row >= p.rows) return;
    auto piece = [&](int k) { return p.ws + ((int64_t)(cta + k) * 2 + (k == 0 ? 1 : 0)) * PS::FLOATS; };
    float mx = -INFINITY;
    for (int k = lane; k < parts; k += 32) mx = fmaxf(mx, piece(k)[PS::m(r)]);
    mx = warp_max(mx);
    float l = 0.f, o[PER] = {};
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
        const float* const f = piece(k);
        const float m = f[PS::m(r)], w = m == -INFINITY ? 0.f : ptx::ex2(m - mx);
        l = fmaf(w, f[PS::l(r)], l);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = fmaf(w, f[PS::o(r) + lane * PER + e], o[e]);
    }
    const int64_t at = ((int64_t)b * p.hkv + h) * p.rows + row;
    const float f = l == 0.f ? 0.f : p.v_scale / l;
    if (lane * PER < p.d) {
        uint32_t* const out = reinterpret_cast<uint32_t*>(p.o + at * p.d + lane * PER);
#pragma unroll
        for (int e = 0; e < PER / 2; ++e) out[e] = ptx::pack_bf16x2(o[2 * e] * f, o[2 * e + 1] * f);
    }
    if (lane == 0) p.lse[at] = qc::natural_lse(mx, l, SHIFT);
}

template <int D, int N>
__global__ void __launch_bounds__(THREADS, 1) fa_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const DecParams p)
{
    using L = Layout<D, N>;
    using PB = qc::Block<D>;
    constexpr int NC = L::NC, TURNS = L::TURNS, SHARES = L::SHARES, NO = L::NO, STREAMS = L::STREAMS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_status, STATUS_BAD_SMEM);
        return;
    }
    volatile uint32_t* const misc = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC);
    volatile uint32_t* const abort_flag = misc + 1;
    Note* const notes = reinterpret_cast<Note*>(smem + L::OFF_NOTES);
    int* const prefix = reinterpret_cast<int*>(smem + L::OFF_PREFIX);
    int* const scratch = reinterpret_cast<int*>(smem + L::OFF_WARP);  // (before the softmax warps use it)
    static_assert(GROUPS * NC * 16 >= THREADS / 32 * 4, "scratch");
    auto bar = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::RAW_STAGES; ++s) {
            ptx::mbar_init(bar(L::B_RAWFULL + s), 1);
            ptx::mbar_init(bar(L::B_RAWEMPTY + s), 4);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(bar(L::B_KFULL + s), 4);
            ptx::mbar_init(bar(L::B_VFULL + s), 4);
            ptx::mbar_init(bar(L::B_QRAW + s), 1);
            ptx::mbar_init(bar(L::B_QFULL + s), SOFTMAX_WARPS);
            ptx::mbar_init(bar(L::B_QEMPTY + s), 1 + SOFTMAX_WARPS);
            ptx::mbar_init(bar(L::B_DRAIN + s), 1);
        }
        for (int s = 0; s < L::EMPTIES; ++s) {
            ptx::mbar_init(bar(L::B_KEMPTY + s), 1);
            ptx::mbar_init(bar(L::B_VEMPTY + s), 1);
        }
        for (int s = 0; s < 4; ++s) {
            ptx::mbar_init(bar(L::B_SFULL + s), 1);
            ptx::mbar_init(bar(L::B_SREAD + s), 4 * SHARES / STREAMS);
            ptx::mbar_init(bar(L::B_PFULL + s), 4 * SHARES / STREAMS);
            ptx::mbar_init(bar(L::B_PDONE + s), 1);
        }
        ptx::mbar_init(bar(L::B_OFREE), SOFTMAX_WARPS);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == WARP_Q && lane == 0) ptx::prefetch_tensormap(&tm_q);
    qc::prefetch_l2(p.table, (int64_t)p.B * p.max_pages * 4);
    qc::prefetch_l2(p.q, (int64_t)p.B * p.hkv * p.rows * p.d * 2);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    qc::page_prefix<THREADS, TILE>(p.lens, p.B, p.max_pages, prefix, scratch);
    const int hr_all = p.hkv * p.rb;
    const Units work{prefix, p.B, hr_all, uniform(prefix[p.B]) * hr_all >= 4 * (int)gridDim.x ? L::EXTRA : 0};

    // Sequences of no key: nothing is seen.
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (threadIdx.x == 0 && p.lens[b] > p.max_pages * (int64_t)PAGE) atomicOr(&g_status, STATUS_BAD_PAGE);
        if (prefix[b + 1] != prefix[b]) continue;
        const int64_t n = (int64_t)p.hkv * p.rows, at = b * n;
        for (int64_t e = threadIdx.x; e < n * (p.d / 8); e += THREADS) ptx::st_global_v4(p.o + at * p.d + e * 8, 0, 0, 0, 0);
        for (int64_t e = threadIdx.x; e < n; e += THREADS) p.lse[at + e] = -INFINITY;
    }
    const int T = uniform(work.total()), G = min((int)gridDim.x, T), cta = blockIdx.x;
    if (threadIdx.x == 0) p.desc[2 * cta] = -1;
    if (cta >= G) return;
    const int lo = (int)((int64_t)cta * T / G), hi = (int)((int64_t)(cta + 1) * T / G);
    const int n_tiles = uniform(work.tiles_before(hi) - work.tiles_before(lo));
    if (n_tiles == 0) return;

    if (warp == WARP_S) {
        ptx::tmem_alloc(sbase + L::OFF_MISC, TM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = (uint32_t)uniform((int)misc[0]);

    if (warp >= WARP_COPY) {
        ptx::setmaxnreg_dec<REGS_OTHER>();
        if (warp == WARP_COPY) {
            // ------------------------------------------------------------ pages
            int g = 0;
            bool ok = true;
#pragma unroll 1
            for (int x = lo; ok;) {
                Run run;
                if (!next_run(work, x, hi, run)) break;
                const int b = run.b, h = run.hr / p.rb, tile0 = run.tile0, n = run.n;
                const int len = uniform(qc::length_of(p.lens, b, p.max_pages));
                const int pages = (len + PAGE - 1) / PAGE;
                int id = -1;
#pragma unroll 1
                for (int i = 0; ok && i < n; ++i, ++g) {
                    // The page table's entries of 16 tiles, one a lane.
                    if (i % 16 == 0) {
                        const int slot = 2 * (tile0 + i) + lane;
                        id = -1;
                        if (slot < pages && lane < 2 * (n - i)) {
                            id = p.table[(int64_t)b * p.max_pages + slot];
                            if ((unsigned)id >= (unsigned)p.num_pages) {
                                id = -1;
                                atomicOr(&g_status, STATUS_BAD_PAGE);
                            }
                        }
                    }
                    const int id0 = __shfl_sync(0xffffffffu, id, 2 * (i % 16)), id1 = __shfl_sync(0xffffffffu, id, 2 * (i % 16) + 1);
                    const int st = (int)((uint32_t)g % L::RAW_STAGES);
                    if (!(ok = warp_wait(bar(L::B_RAWEMPTY + st), ((uint32_t)g / L::RAW_STAGES & 1u) ^ 1u, limit, abort_flag,
                                         0x2100 + L::B_RAWEMPTY + st)))
                        break;
                    if (ptx::elect_one()) {
                        // The note's place held tile g - NOTES, which no one reads any more: this
                        // stage is free because the values of tile g - RAW_STAGES are in TMEM,
                        // so the products of the tile 2 before it are done, and all before.
                        Note note;
                        note.what = (id0 >= 0 ? Note::PAGE0 : 0u) | (id1 >= 0 ? Note::PAGE1 : 0u) | (i == 0 ? Note::FIRST : 0u) |
                                    (i == n - 1 ? Note::LAST : 0u) | (uint32_t)min(i, 15) << Note::INDEX;
                        note.left = len - (tile0 + i) * TILE;
                        notes[(uint32_t)g % NOTES] = note;
                        const uint32_t fb = bar(L::B_RAWFULL + st), dst = sbase + L::OFF_RAW + st * L::RAW_BYTES;
                        ptx::mbar_arrive_expect_tx(fb, ((id0 >= 0) + (id1 >= 0)) * L::PAGE_BYTES);
                        if (!(g == p.debug_skip && blockIdx.x == 0)) {
                            if (id0 >= 0) ptx::bulk_load(dst, p.pool + ((int64_t)id0 * p.hkv + h) * L::PAGE_BYTES, L::PAGE_BYTES, fb);
                            if (id1 >= 0)
                                ptx::bulk_load(dst + L::PAGE_BYTES, p.pool + ((int64_t)id1 * p.hkv + h) * L::PAGE_BYTES, L::PAGE_BYTES, fb);
                        }
                    }
                    __syncwarp();
                }
            }
            // Every copy lands before the block leaves.
#pragma unroll 1
            for (int e = max(0, g - L::RAW_STAGES); e < g; ++e)
                if (!(e == p.debug_skip && blockIdx.x == 0))
                    drain_bar(bar(L::B_RAWFULL + e % L::RAW_STAGES), (uint32_t)(e / L::RAW_STAGES) & 1u, limit, abort_flag, 0x2180);
        } else if (warp == WARP_S) {
            // ------------------------------------------------------------ S^T
            constexpr uint32_t ID = idesc_f16(128, L::NM, false);
            const uint64_t q_desc = ptx::sdesc_sw128(sbase + L::OFF_Q, 16, 1024);
            int k = 0;
            bool ok = true;
#pragma unroll 1
            for (int g = 0; ok && g < n_tiles; ++g) {
                const int kb = g & 1, turn = (int)((uint32_t)g % TURNS);
                ok = warp_wait(bar(L::B_KFULL + kb), (uint32_t)(g >> 1) & 1u, limit, abort_flag, 0x2200 + L::B_KFULL + kb);
                const uint32_t what = (uint32_t)uniform((int)notes[(uint32_t)g % NOTES].what);
                const int qb = k & 1;
                if ((what & Note::FIRST) && ok)
                    ok = warp_wait(bar(L::B_QFULL + qb), (uint32_t)(k >> 1) & 1u, limit, abort_flag, 0x2200 + L::B_QFULL + qb);
                const uint64_t q_at = q_desc + (uint64_t)(((uint32_t)qb * L::Q_BYTES) >> 4);
#pragma unroll 1
                for (int st = 0; st < STREAMS; ++st) {
                    const int sb = STREAMS > 1 ? st : turn;
                    if (ok) ok = warp_wait(bar(L::B_SREAD + sb), ((uint32_t)g / TURNS & 1u) ^ 1u, limit, abort_flag, 0x2200 + L::B_SREAD + sb);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint64_t q_rows = q_at + (uint64_t)(((uint32_t)st * L::NM * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        if (ptx::elect_one())
                            ptx::mma_ts(tmem + TM_S + (uint32_t)(turn * N + st * L::NM), tmem + TM_K + (uint32_t)(kb * 64 + kk * 8),
                                        q_rows + (uint64_t)(((uint32_t)(kk >> 2) * L::QBLK + (uint32_t)(kk & 3) * 32) >> 4), ID, kk > 0 ? 1u : 0u);
                    if (ptx::elect_one()) ptx::tc_commit(bar(L::B_SFULL + sb));
                }
                if (!ok) break;
                if (ptx::elect_one()) {
                    ptx::tc_commit(bar(L::B_KEMPTY + (int)((uint32_t)g % L::EMPTIES)));
                    if (what & Note::LAST) ptx::tc_commit(bar(L::B_QEMPTY + qb));
                }
                if (what & Note::LAST) ++k;
            }
            if (ptx::elect_one()) ptx::tc_commit(bar(L::B_DRAIN));
            drain_bar(bar(L::B_DRAIN), 0, limit, abort_flag, 0x2280);
        } else if (warp == WARP_O) {
            // ------------------------------------------------------------ O^T
            constexpr uint32_t ID = idesc_f16(128, L::NM, true);
            const uint64_t p_desc = ptx::sdesc_sw128(sbase + L::OFF_P, L::PBLK, 1024);
            int k = 0;
            bool ok = true;
#pragma unroll 1
            for (int g = 0; ok && g < n_tiles; ++g) {
                const int vb = g & 1, pb = (int)((uint32_t)g % L::PBUFS);
                ok = warp_wait(bar(L::B_VFULL + vb), (uint32_t)(g >> 1) & 1u, limit, abort_flag, 0x2300 + L::B_VFULL + vb);
                const uint32_t what = (uint32_t)uniform((int)notes[(uint32_t)g % NOTES].what);
                // A segment's first products overwrite O^T: what was there has been read.
                if ((what & Note::FIRST) && ok)
                    ok = warp_wait(bar(L::B_OFREE), (uint32_t)(k & 1) ^ 1u, limit, abort_flag, 0x2300 + L::B_OFREE);
                const uint32_t keep = (what >> Note::INDEX) < TURNS ? 0u : 1u;
#pragma unroll 1
                for (int st = 0; st < STREAMS; ++st) {
                    const int ps = st * L::PBUFS + pb;
                    if (ok) ok = warp_wait(bar(L::B_PFULL + ps), (uint32_t)g / L::PBUFS & 1u, limit, abort_flag, 0x2300 + L::B_PFULL + ps);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint64_t p_at = p_desc + (uint64_t)(((uint32_t)pb * L::P_BYTES + (uint32_t)st * L::PBLK) >> 4);
#pragma unroll
                    for (int kk = 0; kk < TILE / 16; ++kk)
                        if (ptx::elect_one())
                            ptx::mma_ts(tmem + L::TM_O + ((uint32_t)g % TURNS * N + (uint32_t)(st * L::NM)), tmem + TM_V + (uint32_t)(vb * 64 + kk * 8),
                                        p_at + (uint64_t)(((uint32_t)kk * 2048) >> 4), ID, kk > 0 ? 1u : keep);
                    if (ptx::elect_one()) ptx::tc_commit(bar(L::B_PDONE + ps));
                }
                if (!ok) break;
                if (ptx::elect_one()) ptx::tc_commit(bar(L::B_VEMPTY + (int)((uint32_t)g % L::EMPTIES)));
                if (what & Note::LAST) ++k;
            }
            if (ptx::elect_one()) ptx::tc_commit(bar(L::B_DRAIN + 1));
            drain_bar(bar(L::B_DRAIN + 1), 0, limit, abort_flag, 0x2281);
        } else {
            // ------------------------------------------------------- query rows
            int k = 0, loads = 0;
            bool ok = true;
#pragma unroll 1
            for (int x = lo; ok; ++k) {
                Run run;
                if (!next_run(work, x, hi, run)) break;
                const int b = run.b, hr = run.hr, h = hr / p.rb, qb = k & 1;
                if (!(ok = warp_wait(bar(L::B_QEMPTY + qb), ((uint32_t)(k >> 1) & 1u) ^ 1u, limit, abort_flag, 0x2400 + L::B_QEMPTY + qb)))
                    break;
                const uint32_t q = sbase + L::OFF_Q + (uint32_t)qb * L::Q_BYTES;
                if (ptx::elect_one()) {  // (rows and channels that do not exist come as zeros)
                    ptx::mbar_arrive_expect_tx(bar(L::B_QRAW + qb), L::Q_BYTES);
                    for (int c = 0; c < D / 64; ++c)
                        ptx::tma_load_3d(q + (uint32_t)c * L::QBLK, &tm_q, bar(L::B_QRAW + qb), c * 64, (hr - h * p.rb) * N, b * p.hkv + h);
                }
                __syncwarp();
                ++loads;
                if (k == 0) continue;  // (the softmax warps')
                if (!(ok = warp_wait(bar(L::B_QRAW + qb), (uint32_t)(k >> 1) & 1u, limit, abort_flag, 0x2400 + L::B_QRAW + qb))) break;
                const QueryRows<D, N> rows{q, sbase + L::OFF_LARGEST + (uint32_t)qb * (N * 4), 0, 1};
                rows.measure();
                bool apart;
                const int power = rows.power_of_all(apart);
                rows.convert(power, apart);
                if (lane == 0) set_scaling(sbase + L::OFF_QSC + (uint32_t)qb * 8, p.scale_log2, power, apart);
                __syncwarp();
                if (lane < SOFTMAX_WARPS) ptx::mbar_arrive(bar(L::B_QFULL + qb));  // (as those for the first)
            }
            // The last two loads land before the block leaves.
#pragma unroll 1
            for (int e = max(0, loads - 2); e < loads; ++e) drain_bar(bar(L::B_QRAW + (e & 1)), (uint32_t)(e >> 1) & 1u, limit, abort_flag, 0x2480);
        }
    } else if (warp >= WARP_CODES) {
        ptx::setmaxnreg_dec<REGS_CODES>();
        // --------------------------------------------------------------- codes
        // Three sets of warps take tiles in turn: first the keys, then the values.
        const int quarter = warp & 3, set = (warp - WARP_CODES) >> 2;
        // Of the keys, key x of page `page`.
        const int page = quarter >> 1, x = key_of((quarter & 1) * 32 + lane);
        const bool other = D == 128 ? (lane >> 1) & 1 : (lane >> 2) & 1;
        // Of the values 32 channels; a byte is a pair of keys.  A thread takes four channels
        // of every fourth pair at a time: a word of codes, whose bytes go to four TMEM
        // lanes (16x128b: the fragment of a product's operand; see channel_of).
        const int fourth = lane & 3;
        const uint32_t factors = sbase + L::OFF_FACTORS + (uint32_t)(warp - WARP_CODES) * 512;
        bool ok = true;
#pragma unroll 1
        for (int g = set, turn = 0; ok && g < n_tiles; g += SETS, ++turn) {  // (g = set + SETS * turn)
            constexpr int OWN = L::RAW_STAGES / SETS;  // stages of a set, 1 or 2
            const int st = set + SETS * (turn & (OWN - 1)), buf = g & 1;
            ok = warp_wait(bar(L::B_RAWFULL + st), (uint32_t)turn / OWN & 1u, limit, abort_flag, 0x2500 + L::B_RAWFULL + st);
            const int before = g - 2;
            const uint32_t empty = (uint32_t)max(before, 0) % L::EMPTIES, turns = (uint32_t)max(before, 0) / L::EMPTIES & 1u;
            if (ok && before >= 0) ok = warp_wait(bar(L::B_KEMPTY + empty), turns, limit, abort_flag, 0x2500 + L::B_KEMPTY + empty);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            const uint32_t raw = sbase + L::OFF_RAW + (uint32_t)st * L::RAW_BYTES;
            // (A page that is not there, and places of no key, leave anything: their
            // scores are not used.)
#pragma unroll 1
            for (int part = 0; part < D / 64; ++part) {
                // 64 channels: two pieces of 16 bytes, the second one first in every other
                // lane of those whose rows share banks.
                const uint32_t blk = raw + (uint32_t)page * L::PAGE_BYTES, row = blk + (uint32_t)PB::kcode(x);
                const uint4 first = lds128(row + (uint32_t)(part * 32 + (other ? 16 : 0)));
                const uint4 then = lds128(row + (uint32_t)(part * 32 + (other ? 0 : 16)));
                uint32_t sc[2];  // scales of two channel blocks each
                if constexpr (D == 128) {
                    sc[0] = lds_u16(blk + (uint32_t)PB::kscale(x, 0) + (uint32_t)part * 32);
                    sc[1] = lds_u16(blk + (uint32_t)PB::kscale(x, 2) + (uint32_t)part * 32);
                } else {
                    sc[0] = lds_u8(blk + PB::kscale(x, 0)) | lds_u8(blk + PB::kscale(x, 1)) << 8;
                    sc[1] = lds_u8(blk + PB::kscale(x, 2)) | lds_u8(blk + PB::kscale(x, 3)) << 8;
                }
                const uint32_t w[8] = {other ? then.x : first.x, other ? then.y : first.y, other ? then.z : first.z, other ? then.w : first.w,
                                       other ? first.x : then.x, other ? first.y : then.y, other ? first.z : then.z, other ? first.w : then.w};
                const uint32_t to = tmem + ((uint32_t)(quarter * 32) << 16) + TM_K + (uint32_t)(buf * 64 + part * 32);
#pragma unroll
                for (int half = 0; half < 4; ++half) {
                    const uint32_t f = qc::e4m3x2(sc[half >> 1]);
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        auto by = [&](uint32_t a) { return half % 2 == 0 ? qc::hmul2_by<0>(a, f) : qc::hmul2_by<1>(a, f); };
                        o[4 * j + 0] = by(qc::e2m1x2<0>(w[2 * half + j]));
                        o[4 * j + 1] = by(qc::e2m1x2<1>(w[2 * half + j]));
                        o[4 * j + 2] = by(qc::e2m1x2<2>(w[2 * half + j]));
                        o[4 * j + 3] = by(qc::e2m1x2<3>(w[2 * half + j]));
                    }
                    ptx::tmem_st8(to + (uint32_t)(half * 8), o);
                }
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(L::B_KFULL + buf));
            if (quarter * 32 < D) {
                // The scales of the warp's 2 channel blocks to fp16, pairs of keys: [page][block]
                // [column % 4][column / 4], column 8 q + r being pair q + 4 r, a lane two of a
                // page's 64.  Places of no key hold anything: their scale becomes 0 (their weight
                // is 0, and 0 * NaN must not be formed).
                const Note note = notes[(uint32_t)g % NOTES];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = (e & 1) * 32 + lane, b = e & 1, q = i >> 3 & 3, r = i & 7, pair = q + 4 * r, pg = e >> 1;
                    const int left = note.what >> pg & 1u ? note.left - pg * PAGE : 0;
                    uint32_t two = lds_u16(raw + (uint32_t)(pg * L::PAGE_BYTES + PB::VS + (q * PB::NB + quarter * 2 + b) * 16 + 2 * r));
                    two &= left > 2 * pair + 1 ? 0xFFFFu : left > 2 * pair ? 0xFFu : 0u;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(factors + (uint32_t)(pg * 64 + b * 32 + (i & 3) * 8 + (i >> 2 & 7)) * 4), "r"(qc::e4m3x2(two)) : "memory");
                }
                __syncwarp();
            }
            if (before >= 0) ok = warp_wait(bar(L::B_VEMPTY + empty), turns, limit, abort_flag, 0x2500 + L::B_VEMPTY + empty);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            if (quarter * 32 < D) {
                const uint32_t codes = raw + PB::VC + (uint32_t)(fourth * 4 * D + quarter * 32 + (lane >> 2) * 4);
                const uint32_t mine = factors + (uint32_t)((lane >> 4) * 32 + fourth * 8) * 4;
                const uint32_t to = tmem + ((uint32_t)(quarter * 32) << 16) + TM_V + (uint32_t)(buf * 64);
#pragma unroll 1
                for (int half = 0; half < 4; ++half) {  // columns 16 half + 4 e + fourth
                    uint32_t w[4], low[8], high[8];
                    const uint32_t at = codes + (uint32_t)((half >> 1) * L::PAGE_BYTES + (half & 1) * 2 * D);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = lds_u32(at + (uint32_t)((e / 2 + 16 * (e & 1)) * D));
                    const uint4 f4 = lds128(mine + (uint32_t)((half >> 1) * 256 + (half & 1) * 16));
                    const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        low[2 * e] = qc::hmul2(qc::e2m1x2<0>(w[e]), f[e]);
                        low[2 * e + 1] = qc::hmul2(qc::e2m1x2<1>(w[e]), f[e]);
                        high[2 * e] = qc::hmul2(qc::e2m1x2<2>(w[e]), f[e]);
                        high[2 * e + 1] = qc::hmul2(qc::e2m1x2<3>(w[e]), f[e]);
                    }
                    ptx::tmem_st_16x128b_x4(to + (uint32_t)(half * 16), low);
                    ptx::tmem_st_16x128b_x4(to + (16u << 16) + (uint32_t)(half * 16), high);
                }
                ptx::tmem_wait_st();
            }
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(bar(L::B_RAWEMPTY + st));
                ptx::mbar_arrive(bar(L::B_VFULL + buf));
            }
        }
    } else {
        ptx::setmaxnreg_inc<REGS_SOFTMAX>();
        // ------------------------------------------------------------- softmax
        const int group = warp >> 2, quarter = warp & 3, mine = quarter * 32 + lane;  // this thread's lane of a tile
        const int turn = group / SHARES, share = group % SHARES;  // its tiles, and its rows of them
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const int stream = share / (SHARES / STREAMS), c0 = share * NC;
        const int sb = STREAMS > 1 ? stream : turn;  // its barriers of S^T
        const uint32_t par = sbase + L::OFF_PAR + (uint32_t)(group * NC) * 4, refs = sbase + L::OFF_REF + (uint32_t)(group * NC) * 4;
        const uint32_t sums = sbase + L::OFF_SUM + (uint32_t)(group * NC) * 4, corr = sbase + L::OFF_CORR + (uint32_t)(group * NC) * 4;
        const uint32_t exps = sbase + L::OFF_APART + (uint32_t)(group * NC) * 4;
        const uint32_t warps = sbase + L::OFF_WARP + (uint32_t)(group * NC) * 16, word = sbase + L::OFF_WORD + (uint32_t)(group * NC) * 8;
        const uint32_t s_cols = tmem + lane_off + TM_S + (uint32_t)(turn * N + c0);
        const uint32_t o_cols = tmem + lane_off + L::TM_O + (uint32_t)(turn * N + c0);
        const int t = (int)threadIdx.x & 127;  // thread of the group
        // The first of its pieces of a row of P^T; the others differ in the bits that e8 has
        // (c0 / 8 is a multiple of NC / 8, a row starts on 128 bytes).
        const uint32_t p_row = sbase + L::OFF_P + (uint32_t)(c0 >> 6) * L::PBLK + (uint32_t)mine * 128 + (uint32_t)((((c0 >> 3) & 7) ^ (mine & 7)) * 16);
        bool ok = warp_wait(bar(L::B_QRAW), 0, limit, abort_flag, 0x2700 + L::B_QRAW);
        {
            const QueryRows<D, N> rows{sbase + L::OFF_Q, sbase + L::OFF_LARGEST, warp, SOFTMAX_WARPS};
            if (ok) rows.measure();
            ptx::named_barrier_sync(NB_ALL, 32 * SOFTMAX_WARPS);
            bool apart;
            const int power = rows.power_of_all(apart);
            if (ok) rows.convert(power, apart);
            if (warp == 0 && lane == 0) set_scaling(sbase + L::OFF_QSC, p.scale_log2, power, apart);
            if (lane == 0) ptx::mbar_arrive(bar(L::B_QFULL));
        }
        int g0 = 0;  // the segment's first tile, of the block's
#pragma unroll 1
        for (int k = 0, x = lo;; ++k) {
            Run run;
            if (!next_run(work, x, hi, run)) break;
            const int b = run.b, hr = run.hr, tile0 = run.tile0, tiles = run.tiles, n = run.n, h = hr / p.rb, row0 = (hr - h * p.rb) * N + c0;
            const int raw_len = uniform(max(p.lens[b], 0)), len = qc::clamp_length(raw_len, p.max_pages), draft0 = raw_len - p.nq;
            const int qb = k & 1;
            const uint64_t mine_word = t < NC ? __ldg(p.words + (int64_t)b * p.nq + (row0 + t) % p.nq) : 0;
            if (ok) ok = warp_wait(bar(L::B_QFULL + qb), (uint32_t)(k >> 1) & 1u, limit, abort_flag, 0x2700 + L::B_QFULL + qb);
            if (t < NC) {
                asm volatile("st.shared.b64 [%0], %1;" ::"r"(word + (uint32_t)t * 8), "l"(mine_word) : "memory");
                sts_f32(par + (uint32_t)t * 4, UNSET);
                sts_f32(refs + (uint32_t)t * 4, -INFINITY);
            }
            const float factor = lds_f32(sbase + L::OFF_QSC + (uint32_t)qb * 8);
            const int power = __float_as_int(lds_f32(sbase + L::OFF_QSC + (uint32_t)qb * 8 + 4));
            const bool apart = power != TOGETHER;
            if (apart && t < NC) {
                const uint32_t own = __float_as_uint(lds_f32(sbase + L::OFF_LARGEST + (uint32_t)(qb * N + c0 + t) * 4));
                sts_f32(exps + (uint32_t)t * 4, __int_as_float(own > 0 && own < 0x7F80u ? power - QueryRows<D, N>::power(own) : 0));
            }
            ptx::named_barrier_sync(NB_GROUP + group, 128);
            if (lane == 0) ptx::mbar_arrive(bar(L::B_QEMPTY + qb));
            uint64_t l[NC / 2];
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) l[c] = 0ull;

            bool dead = false;
            float lowest = UNSET;  // what is added to the scores of the row with the lowest reference
            int last = -1;  // the group's last tile of the segment
#pragma unroll 1
            for (int g = g0 + (turn + TURNS - g0 % TURNS) % TURNS; g < g0 + n; g += TURNS) {
                static_assert(L::PBUFS == (TURNS > 1 ? TURNS : 2), "a group that takes tiles in turn has a buffer of its own");
                const int pb = TURNS > 1 ? turn : g & 1, ps = stream * L::PBUFS + pb;
                if (ok) ok = warp_wait(bar(L::B_SFULL + sb), (uint32_t)g / TURNS & 1u, limit, abort_flag, 0x2700 + L::B_SFULL + sb);
                ptx::tc_fence_after_sync();
                const int key0 = (tile0 + g - g0) * TILE;
                // y = score - reference + SHIFT in base-2 units.
                uint32_t y[NC];
                float red;  // the largest score of this thread's key
                // Once more where references rise: the same code, as it is there already.
#pragma unroll 1
                for (bool settled = false;; settled = true) {
                    load_cols_max<NC>(s_cols, y, red);
                    const uint32_t what = notes[(uint32_t)g % NOTES].what;
                    load_cols_end<NC>(y);
                    asm volatile("" : "+f"(red));
                    if (__builtin_expect(!settled && ((what & 3u) != 3u || key0 + TILE > min(len, draft0) || apart), 0)) {
                        // Rows that do not see this thread's key: -inf in S^T itself; rows with a
                        // power of their own: the common one (in two steps, each a power of two that exists).
                        const int key = key0 + (quarter >> 1) * PAGE + key_of(mine % PAGE), bit = key - draft0;
                        const bool there = key < len && (what >> (quarter >> 1) & 1u), named = bit >= 0;
                        const uint64_t mask = named && bit < p.nq ? 1ull << bit : 0ull;
#pragma unroll 1
                        for (int c = 0; c < NC; c += 8) {
                            uint32_t r[8];
                            load_cols<8>(s_cols + (uint32_t)c, r);
                            if (apart) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const int down = -__float_as_int(lds_f32(exps + (uint32_t)(c + e) * 4)), half = down >> 1;
                                    r[e] = __float_as_uint(__uint_as_float(r[e]) * __uint_as_float((uint32_t)(127 - half) << 23) *
                                                           __uint_as_float((uint32_t)(127 - (down - half)) << 23));
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const uint4 w = lds128(word + (uint32_t)(c + e) * 8);
                                const uint64_t w0 = (uint64_t)w.y << 32 | w.x, w1 = (uint64_t)w.w << 32 | w.z;
                                if (!there || (named && !(w0 & mask))) r[e] = 0xFF800000u;
                                if (!there || (named && !(w1 & mask))) r[e + 1] = 0xFF800000u;
                            }
                            ptx::tmem_st8(s_cols + (uint32_t)c, r);
                        }
                        ptx::tmem_wait_st();
                        load_cols<NC>(s_cols, y);
                        red = INFINITY;
                    }
                    auto refer = [&] {
#pragma unroll
                        for (int c = 0; c < NC; c += 4) {
                            const uint4 a = lds128(par + (uint32_t)(c * 4));
                            const uint64_t f = ptx::f2_pack(factor, factor);
                            float v[4];
                            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), f,
                                                       ptx::f2_pack(__uint_as_float(a.x), __uint_as_float(a.y))), v[0], v[1]);
                            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(y[c + 2]), __uint_as_float(y[c + 3])), f,
                                                       ptx::f2_pack(__uint_as_float(a.z), __uint_as_float(a.w))), v[2], v[3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[c + e] = __float_as_uint(v[e]);
                        }
                    };
                    refer();
                    if (settled) break;
                    // Whether a score exceeds its row's reference.  Seldom a look at each: none can
                    // where the key's largest score does not exceed the lowest reference.
                    bool exceeds = !(fmaf(red, factor, lowest) <= SHIFT + RISE);
                    if (__builtin_expect(__any_sync(0xffffffffu, exceeds), 0)) {
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < NC; c += 2) top[c / 2 % 4] = ptx::fmax3(top[c / 2 % 4], __uint_as_float(y[c]), __uint_as_float(y[c + 1]));
                        exceeds = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > SHIFT + RISE;
                    }
                    if (__builtin_expect(!any_of(NB_VOTE + group, 128, !ok || exceeds), 1)) break;
                    // An abort that one warp of the group has met: all four leave here together.
                    dead = any_of(NB_VOTE + group, 128, !ok);
                    if (dead) break;
                    // The rows' maxima over this tile become their references.
#pragma unroll 1
                    for (int c = 0; c < NC; c += 8) {
                        uint32_t r[8];
                        load_cols<8>(s_cols + (uint32_t)c, r);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float m = warp_max(__uint_as_float(r[e]));
                            if (lane == e) sts_f32(warps + (uint32_t)(quarter * NC + c + e) * 4, m);
                        }
                    }
                    ptx::named_barrier_sync(NB_GROUP + group, 128);
                    if (t < NC) {
                        float m = -INFINITY;
#pragma unroll
                        for (int w = 0; w < 4; ++w) m = fmaxf(m, lds_f32(warps + (uint32_t)(w * NC + t) * 4));
                        const float old = lds_f32(refs + (uint32_t)t * 4), now = fmaxf(old, m == -INFINITY ? m : m * factor);
                        sts_f32(refs + (uint32_t)t * 4, now);
                        sts_f32(par + (uint32_t)t * 4, now == -INFINITY ? UNSET : SHIFT - now);
                        sts_f32(corr + (uint32_t)t * 4, old == -INFINITY ? 0.f : ptx::ex2(old - now));
                    }
                    ptx::named_barrier_sync(NB_GROUP + group, 128);
                    if (last >= 0) {
#pragma unroll
                        for (int c = 0; c < NC / 2; ++c)
                            l[c] = ptx::f2_mul(l[c], ptx::f2_pack(lds_f32(corr + (uint32_t)c * 8), lds_f32(corr + (uint32_t)c * 8 + 4)));
                    }
                    if (last >= 0 && ok) {  // what the products have summed
                        ok = warp_wait(bar(L::B_PDONE + stream * L::PBUFS + last % L::PBUFS), (uint32_t)(last / L::PBUFS) & 1u, limit, abort_flag,
                                       0x2700 + L::B_PDONE + last % L::PBUFS);
                        ptx::tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; ok && c < NC; c += 8) {
                            uint32_t r[8];
                            load_cols<8>(o_cols + (uint32_t)c, r);
#pragma unroll
                            for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * lds_f32(corr + (uint32_t)(c + e) * 4));
                            ptx::tmem_st8(o_cols + (uint32_t)c, r);
                        }
                        ptx::tmem_wait_st();
                    }
                    lowest = lds_f32(par + (uint32_t)(lane % NC) * 4);
                    lowest = warp_max(lowest);
                }
                if (dead) break;
                // S^T of this tile is in registers.
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(L::B_SREAD + sb));
                // P^T: a row of 128 bytes a key (64 query rows), 16-byte pieces swizzled.
                if (ok) ok = warp_wait(bar(L::B_PDONE + ps), ((uint32_t)g / L::PBUFS & 1u) ^ 1u, limit, abort_flag, 0x2700 + L::B_PDONE + ps);
                const uint32_t row = p_row + (uint32_t)pb * L::P_BYTES;
#pragma unroll
                for (int e8 = 0; e8 < NC / 8; ++e8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = e8 * 8 + 2 * e;
                        const float a = ptx::ex2(__uint_as_float(y[c])), b2 = ptx::ex2(__uint_as_float(y[c + 1]));
                        l[c / 2] = ptx::f2_add(l[c / 2], ptx::f2_pack(a, b2));
                        w[e] = qc::pack_h2(a, b2);
                    }
                    ptx::st_shared_v4(row ^ (uint32_t)(e8 * 16), w[0], w[1], w[2], w[3]);
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(L::B_PFULL + ps));
                last = g;
            }

            // -------------------------------------------------- a segment's end
            // Sums over the keys: the lanes, then the warps.
            {
                float v[NC];
#pragma unroll
                for (int c = 0; c < NC / 2; ++c) ptx::f2_unpack(l[c], v[2 * c], v[2 * c + 1]);
                const float sum = spread_sum<NC>(v);
                if (lane < NC) sts_f32(warps + (uint32_t)(quarter * NC + lane) * 4, sum);
            }
            ptx::named_barrier_sync(NB_GROUP + group, 128);
            if (t < NC) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) sum += lds_f32(warps + (uint32_t)(w * NC + t) * 4);
                sts_f32(sums + (uint32_t)t * 4, sum);
            }
            if (ok && last >= 0)
                ok = warp_wait(bar(L::B_PDONE + stream * L::PBUFS + last % L::PBUFS), (uint32_t)(last / L::PBUFS) & 1u, limit, abort_flag,
                               0x2700 + L::B_PDONE + last % L::PBUFS);
            ptx::tc_fence_before_sync();
            // All groups of these rows are here, their products done (or none goes on).
            if (any_of(NB_END + share, 128 * TURNS, dead || !ok)) break;
            ptx::tc_fence_after_sync();
            const bool begins = tile0 == 0, joined = begins && tile0 + n == tiles;
            const int out0 = turn * NO;  // of this group's share of the rows, those that it writes
            const int64_t at = ((int64_t)b * p.hkv + h) * p.rows + row0 + out0;
            const int rows = min(NO, p.rows - row0 - out0);
            float* const part = p.ws + ((int64_t)cta * 2 + (begins ? 1 : 0)) * qc::Partial<D, N>::FLOATS;
            if (t < NO) {
                // The weights of the groups' results in the joined one.
                const uint32_t c = (uint32_t)(out0 + t) * 4, step = SHARES * NC * 4;
                const uint32_t ref = sbase + L::OFF_REF + (uint32_t)(share * NC) * 4 + c, sum = sbase + L::OFF_SUM + (uint32_t)(share * NC) * 4 + c;
                float m = -INFINITY, total = 0.f, w[TURNS];
#pragma unroll
                for (int i = 0; i < TURNS; ++i) m = fmaxf(m, lds_f32(ref + i * step));
#pragma unroll
                for (int i = 0; i < TURNS; ++i) {
                    const float r = lds_f32(ref + i * step);
                    w[i] = r == -INFINITY ? 0.f : ptx::ex2(r - m);
                    total = fmaf(w[i], lds_f32(sum + i * step), total);
                }
                const float f = joined ? (total == 0.f ? 0.f : p.v_scale / total) : 1.f;
#pragma unroll
                for (int i = 0; i < TURNS; ++i) sts_f32(corr + (uint32_t)(i * NO + t) * 4, w[i] * f);
                if (t < rows) {
                    if (joined) {
                        p.lse[at + t] = qc::natural_lse(m, total, SHIFT);
                    } else {
                        part[qc::Partial<D, N>::m(c0 + out0 + t)] = m;
                        part[qc::Partial<D, N>::l(c0 + out0 + t)] = total;
                    }
                }
            }
            // (All groups have read the others' references before any begins the next segment.)
            ptx::named_barrier_sync(NB_END + share, 128 * TURNS);
            if (quarter * 32 < D) {  // O^T: this thread's channel
                const int ch = quarter * 32 + channel_of(lane);
#pragma unroll 1
                for (int c = 0; c < rows; c += 4) {
                    float v[4] = {};
#pragma unroll
                    for (int i = 0; i < TURNS; ++i) {
                        if (TURNS > 1 && n < TURNS && (i + TURNS - g0 % TURNS) % TURNS >= n) continue;  // this one had no tile
                        uint32_t r[4];
                        ptx::tmem_ld4(tmem + lane_off + L::TM_O + (uint32_t)(i * N + c0 + out0 + c), r);
                        ptx::tmem_wait_ld_only();
                        ptx::reg_fence4(r);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = fmaf(__uint_as_float(r[e]), lds_f32(corr + (uint32_t)(i * NO + c + e) * 4), v[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (c + e >= rows) continue;
                        if (!joined) part[qc::Partial<D, N>::o(c0 + out0 + c + e) + ch] = v[e];
                        else if (ch < p.d) p.o[(at + c + e) * p.d + ch] = __float2bfloat16_rn(v[e]);
                    }
                }
            }
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_relaxed(bar(L::B_OFREE));
            if (threadIdx.x == 0 && begins && !joined) {
                // The block that holds the segment's last unit x: the c with c T / G <= x < (c + 1) T / G.
                const int end = work.before(b) * hr_all + (hr + 1) * (tiles + work.extra) - 1;
                p.desc[2 * cta] = b * hr_all + hr;
                p.desc[2 * cta + 1] = (int)(((int64_t)(end + 1) * G - 1) / T);
            }
            g0 += n;
        }
    }

    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == WARP_S) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, TM_COLS);
    }
}

}  // namespace tree
}  // namespace fa
