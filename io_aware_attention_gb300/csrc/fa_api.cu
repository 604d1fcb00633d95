// C ABI of the attention-forward library: argument checks, TMA descriptors,
// kernel selection and launch.  Declarations and the contract: include/fa.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <utility>

#include "fa.h"
#include "fa_bwd_kernel.cuh"
#include "fa_decode_kernel.cuh"
#include "fa_ew_kernel.cuh"
#include "fa_fwd_kernel.cuh"
#include "fa_qcache_kernel.cuh"
#include "fa_rope_kernel.cuh"

namespace {

constexpr int FA_VERSION = 100;  // 0.1.0
constexpr uint64_t DEFAULT_WAIT_LIMIT_NS = 1000000000ull;
constexpr int MAX_DEVICES = 64;

std::atomic<uint64_t> g_wait_limit_ns{DEFAULT_WAIT_LIMIT_NS};
std::atomic<int> g_debug_skip_k{-1};
std::atomic<int> g_debug_schedule{-1};  // causal item order: -1 by size, 0 pairs, 1 cost order

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// (B*H, N, d) bf16 viewed as a 3-D tensor (d innermost); box = 64 columns x
// `rows` rows x 1 head, 128-byte swizzle.  Rows past N read as zero on loads
// and are dropped on stores.
bool make_map(CUtensorMap* map, const void* base, int64_t BH, int64_t N, int64_t d, uint32_t rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)(d * 2), (cuuint64_t)(N * d * 2)};
    cuuint32_t box[3] = {64, rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// make_map through a small per-thread cache of recent encodes.  The encode is
// a pure function of its arguments (address, sizes, box rows; the data type,
// swizzle and fill are fixed), so a hit returns exactly the map a fresh
// encode would.  Repeated calls on the same buffers then skip the driver's
// encode (three per forward call).
bool cached_map(CUtensorMap* map, const void* base, int64_t BH, int64_t N, int64_t d, uint32_t rows)
{
    struct Entry {
        CUtensorMap map;
        const void* base;
        int64_t BH, N, d;
        uint32_t rows;
        bool valid;
    };
    constexpr int SLOTS = 8;
    thread_local Entry cache[SLOTS] = {};
    thread_local unsigned next = 0;
    for (int i = 0; i < SLOTS; ++i) {
        const Entry& e = cache[i];
        if (e.valid && e.base == base && e.BH == BH && e.N == N && e.d == d && e.rows == rows) {
            *map = e.map;
            return true;
        }
    }
    if (!make_map(map, base, BH, N, d, rows)) return false;
    Entry& e = cache[next++ % SLOTS];
    e.map = *map;
    e.base = base;
    e.BH = BH;
    e.N = N;
    e.d = d;
    e.rows = rows;
    e.valid = true;
    return true;
}

// The backward's fp32 dQ accumulator (B*H, Np, d) as a 3-D tensor; box = 32
// columns x 64 rows x 1 head, no swizzle (the reduce-add source is a plain
// row-major 64 x 32 block).
bool make_acc_map(CUtensorMap* map, void* base, int64_t BH, int64_t Np, int64_t d)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Np, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)(d * 4), (cuuint64_t)(Np * d * 4)};
    cuuint32_t box[3] = {32, (cuuint32_t)fa::bwd::BQ, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Head sizes the forward and backward take: multiples of 8 up to 128.  They
// run in the kernel instance for 64 (d <= 64) or 128 columns; the TMA loads
// fill the columns past d with zeros.  Rows stay 16-byte aligned.
bool head_size_ok(int64_t d) { return d >= 8 && d <= 128 && d % 8 == 0; }
int64_t padded_head_size(int64_t d) { return d <= 64 ? 64 : 128; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Launches `kernel` as a programmatic dependent of the work before it on the
// stream (cudaLaunchAttributeProgrammaticStreamSerialization): its blocks may
// start, and set up, while that work's last blocks run.  The kernels launched
// this way (forward, decode, elementwise chain) wait (griddepcontrol.wait)
// for the work before them to complete before they touch global memory.  The
// backward's three kernels are launched plainly: measured, their chain ran
// 1% slower as programmatic dependents.
template <typename... KParams, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KParams...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Per-device, per-kernel one-time set-up (opt-in shared memory size).
template <int D, bool CAUSAL, bool PAD, bool SNAKE>
cudaError_t prepare_kernel(int dev)
{
    static std::atomic<int> done[MAX_DEVICES];
    if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(fa::fa_fwd_kernel<D, CAUSAL, PAD, SNAKE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)fa::Layout<D>::SMEM_BYTES);
    if (e == cudaSuccess) done[dev].store(1, std::memory_order_release);
    return e;
}

template <int D, bool CAUSAL, bool PAD, bool SNAKE>
fa_status launch_one(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                     const fa::Params& p, unsigned grid, int dev, cudaStream_t stream)
{
    if (prepare_kernel<D, CAUSAL, PAD, SNAKE>(dev) != cudaSuccess) return FA_ERR_CUDA;
    const cudaError_t e = launch_pdl(fa::fa_fwd_kernel<D, CAUSAL, PAD, SNAKE>, dim3(grid), dim3(fa::NUM_THREADS),
                                     fa::Layout<D>::SMEM_BYTES, stream, mq, mk, mv, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Causal problems run in cost order (snake) when `snake`; see item_of.
template <int D, bool CAUSAL, bool PAD = false>
fa_status launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                 const fa::Params& p, unsigned grid, int dev, cudaStream_t stream, bool snake)
{
    if constexpr (CAUSAL) {
        if (snake) return launch_one<D, true, PAD, true>(mq, mk, mv, p, grid, dev, stream);
    }
    return launch_one<D, CAUSAL, PAD, false>(mq, mk, mv, p, grid, dev, stream);
}

// Properties of a device that every call needs, queried once per device.
struct DevInfo {
    int sms;    // SMs: the persistent kernels run one CTA per SM
    int l2;     // L2 bytes: picks the causal item order
    bool sm103; // compute capability 10.3
};

std::atomic<int> g_devinfo_ready[MAX_DEVICES];
DevInfo g_devinfo[MAX_DEVICES];
std::mutex g_devinfo_lock;

// The current device (-1 if it cannot be queried) and its cached properties.
bool current_device(int* dev_out, DevInfo* info)
{
    int dev = -1;
    *dev_out = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return false;
    if (!g_devinfo_ready[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> guard(g_devinfo_lock);
        if (!g_devinfo_ready[dev].load(std::memory_order_relaxed)) {
            int major = 0, minor = 0, sms = 0, l2 = 0;
            if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev) != cudaSuccess || sms <= 0)
                return false;
            g_devinfo[dev] = DevInfo{sms, l2, major == 10 && minor == 3};
            g_devinfo_ready[dev].store(1, std::memory_order_release);
        }
    }
    *dev_out = dev;
    *info = g_devinfo[dev];
    return true;
}

// FA_OK when the current device is an sm_103 (its properties in *info),
// FA_ERR_CUDA when it cannot be queried, FA_ERR_UNSUPPORTED otherwise.
fa_status sm103_device(int* dev, DevInfo* info)
{
    if (!current_device(dev, info)) return FA_ERR_CUDA;
    return info->sm103 ? FA_OK : FA_ERR_UNSUPPORTED;
}

// -------------------------------------------------------------- backward

template <int D, bool CAUSAL>
cudaError_t prepare_bwd_kernel(int dev)
{
    static std::atomic<int> done[MAX_DEVICES];
    if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(fa::bwd::fa_bwd_kernel<D, CAUSAL>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)fa::bwd::Layout<D>::SMEM_BYTES);
    if (e == cudaSuccess) done[dev].store(1, std::memory_order_release);
    return e;
}

struct BwdShape {
    int64_t BH, Np, num_kb, Dp;  // Dp: the kernel instance's (padded) head size
    size_t ws_bytes;
};

// Resident CTAs per SM of the elementwise kernel (cached per device).
template <bool WIDE>
int ew_ctas_per_sm(int dev)
{
    static std::atomic<int> cache[MAX_DEVICES];
    if (dev < 0 || dev >= MAX_DEVICES) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0 && cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fa::ew::fa_bias_gelu_dropout_kernel<WIDE>,
                                                               fa::ew::THREADS, 0) == cudaSuccess)
        cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

fa_status bwd_check(int64_t B, int64_t H, int64_t N, int64_t d, BwdShape* sh)
{
    if (B < 1 || H < 1 || N < 1 || d < 1) return FA_ERR_INVALID_ARG;
    if (!head_size_ok(d)) return FA_ERR_UNSUPPORTED;
    const int64_t Dp = padded_head_size(d);
    const int64_t LIM = (int64_t)1 << 60;
    if (B > LIM / H || B * H > LIM / N || B * H * N > LIM / (Dp + 2)) return FA_ERR_INVALID_ARG;
    const int64_t BH = B * H;
    const int64_t Np = (N + fa::bwd::BQ - 1) / fa::bwd::BQ * fa::bwd::BQ;
    const int64_t num_kb = (N + fa::bwd::BKV - 1) / fa::bwd::BKV;
    // BH is the dQ conversion's grid.y; items are int
    if (Np > INT32_MAX / 2 || BH > 65535 || BH > (int64_t)(INT32_MAX / 2) / num_kb) return FA_ERR_INVALID_ARG;
    if (BH * Np > LIM / (Dp + 2)) return FA_ERR_INVALID_ARG;
    sh->BH = BH;
    sh->Np = Np;
    sh->num_kb = num_kb;
    sh->Dp = Dp;
    sh->ws_bytes = (size_t)(BH * Np) * (size_t)(Dp + 2) * sizeof(float);
    return FA_OK;
}

template <int D, bool CAUSAL>
fa_status launch_bwd_main(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                          const CUtensorMap& mdo, const CUtensorMap& mdq, const fa::bwd::Params& p, unsigned grid,
                          int dev, cudaStream_t st)
{
    if (prepare_bwd_kernel<D, CAUSAL>(dev) != cudaSuccess) return FA_ERR_CUDA;
    fa::bwd::fa_bwd_kernel<D, CAUSAL>
        <<<grid, fa::bwd::NUM_THREADS, fa::bwd::Layout<D>::SMEM_BYTES, st>>>(mq, mk, mv, mdo, mdq, p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ---------------------------------------------------------------- decode

// Query slots of the kernel instance serving nq query rows.
int decode_slots(int64_t nq) { return nq <= 1 ? 1 : nq <= 2 ? 2 : nq <= 4 ? 4 : 8; }

struct DecodePlan {
    int slots, splits, chunk;
    size_t ws_bytes;  // 0 when splits == 1 (the partial kernel writes the output)
};

// Splits of the key range.  Each CTA of the partial kernel streams one chunk
// (a whole number of rounds, at least 4) of one head's keys, and `wave` CTAs
// are resident at once.  All chunks cost about the same, so the cache is read
// in about (waves) x (chunk) time, waves = ceil(CTAs / wave): a last wave
// holding a few CTAs costs a whole chunk while most of the GPU idles.  Split
// results add traffic: the partial outputs are written and read back once.
// In bytes at the full bandwidth:
//   cost = waves * chunk * (K and V bytes a key) * wave + 2 * (partials' bytes).
// Candidates: 1 to 16 splits, and for k = 1 .. 8 the most splits that fill k
// waves.  The plan takes the candidate of least cost, or the smallest one
// within 2% of it.  A round is what the kernel instance for head size Dp
// (64 or 128) takes in one pass; the workspace holds d columns per partial
// output.
DecodePlan decode_plan(int64_t BH, int64_t nq, int64_t nk, int64_t d, int64_t wave)
{
    DecodePlan pl;
    pl.slots = decode_slots(nq);
    const int64_t Dp = padded_head_size(d);
    const int64_t round = fa::dec::WARPS * fa::dec::loads_in_flight(pl.slots) * (32 / (int)(Dp / 8));
    const int64_t max_splits = std::max<int64_t>(1, (nk + 4 * round - 1) / (4 * round));
    wave = std::max<int64_t>(1, wave);
    int64_t cand[24];
    int nc = 0;
    for (int64_t s = 1; s <= std::min<int64_t>(16, max_splits); ++s) cand[nc++] = s;
    for (int64_t k = 1; k <= 8; ++k) {
        const int64_t s = std::min<int64_t>(max_splits, k * wave / BH);
        if (s > cand[nc - 1]) cand[nc++] = s;  // ascending, no repeats
    }
    auto chunk_of = [&](int64_t s) { return ((nk + s - 1) / s + round - 1) / round * round; };
    double cost[24];
    double best = 0.0;
    for (int i = 0; i < nc; ++i) {
        const int64_t chunk = chunk_of(cand[i]), splits = (nk + chunk - 1) / chunk;
        const double partials = splits > 1 ? 2.0 * (double)(BH * nq * splits) * (double)(d + 1) * 4.0 : 0.0;
        cost[i] = (double)((BH * splits + wave - 1) / wave) * (double)chunk * (double)(4 * d) * (double)wave + partials;
        best = i == 0 ? cost[i] : std::min(best, cost[i]);
    }
    int pick = 0;
    while (cost[pick] > 1.02 * best) ++pick;
    const int64_t chunk = chunk_of(cand[pick]);
    const int64_t splits = (nk + chunk - 1) / chunk;
    pl.splits = (int)splits;
    pl.chunk = (int)chunk;
    pl.ws_bytes = splits > 1 ? (size_t)(BH * nq * splits) * (size_t)(d + 1) * sizeof(float) : 0;
    return pl;
}

// Checks of the sizes alone (no pointer, no device).
fa_status decode_check(int64_t B, int64_t H, int64_t Nq, int64_t Nk, int64_t d, int causal)
{
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || d < 1) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (causal && Nq > Nk) return FA_ERR_INVALID_ARG;
    if (!head_size_ok(d)) return FA_ERR_UNSUPPORTED;
    if (Nq > fa::dec::MAX_NQ) return FA_ERR_UNSUPPORTED;
    const int64_t LIM = (int64_t)1 << 62;
    if (B > LIM / H || B * H > LIM / Nk || B * H * Nk > LIM / d) return FA_ERR_INVALID_ARG;
    if (B * H > 65535 || Nk > INT32_MAX / 2) return FA_ERR_INVALID_ARG;  // grid.y, key indices
    return FA_OK;
}

// Every check that needs no device: sizes, scale, null and misaligned
// pointers, outputs overlapping inputs.  The workspace is checked against
// the plan later (its size depends on the device).
fa_status decode_args(const void* q, const void* k, const void* v, const void* o, const float* lse, int64_t B,
                      int64_t H, int64_t Nq, int64_t Nk, int64_t d, int causal, float scale, const void* ws)
{
    if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
    const fa_status st = decode_check(B, H, Nq, Nk, d, causal);
    if (st != FA_OK) return st;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
    const uintptr_t mis = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                          reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o) |
                          reinterpret_cast<uintptr_t>(ws);
    if ((mis & 15u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_UNSUPPORTED;
    const int64_t BH = B * H;
    const size_t qb = (size_t)(BH * Nq * d * 2), kb = (size_t)(BH * Nk * d * 2), lb = (size_t)(BH * Nq * 4);
    if (overlaps(o, qb, q, qb) || overlaps(o, qb, k, kb) || overlaps(o, qb, v, kb) || overlaps(o, qb, lse, lb) ||
        overlaps(lse, lb, q, qb) || overlaps(lse, lb, k, kb) || overlaps(lse, lb, v, kb))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Resident CTAs per SM of the partial kernel instance serving `slots` query
// rows at head size d (cached per device); 0 if the query fails.
template <int D, int QM, bool PAD>
int dec_ctas_per_sm(int dev)
{
    static std::atomic<int> cache[MAX_DEVICES];
    if (dev < 0 || dev >= MAX_DEVICES) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0 && cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fa::dec::fa_decode_partial_kernel<D, QM, PAD>,
                                                               fa::dec::THREADS, 0) == cudaSuccess)
        cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int D, bool PAD>
int dec_ctas_per_sm_d(int dev, int slots)
{
    switch (slots) {
    case 1: return dec_ctas_per_sm<D, 1, PAD>(dev);
    case 2: return dec_ctas_per_sm<D, 2, PAD>(dev);
    case 4: return dec_ctas_per_sm<D, 4, PAD>(dev);
    default: return dec_ctas_per_sm<D, 8, PAD>(dev);
    }
}

// The split plan on this device: one wave is the partial kernel's resident
// CTAs per SM times the SMs.  FA_ERR_CUDA if the occupancy query fails.
fa_status device_decode_plan(int dev, const DevInfo& info, int64_t BH, int64_t nq, int64_t nk, int64_t d,
                             DecodePlan* pl)
{
    const int slots = decode_slots(nq);
    const int per_sm = d == 128 ? dec_ctas_per_sm_d<128, false>(dev, slots)
                       : d == 64 ? dec_ctas_per_sm_d<64, false>(dev, slots)
                       : d > 64  ? dec_ctas_per_sm_d<128, true>(dev, slots)
                                 : dec_ctas_per_sm_d<64, true>(dev, slots);
    if (per_sm <= 0) return FA_ERR_CUDA;
    *pl = decode_plan(BH, nq, nk, d, (int64_t)per_sm * info.sms);
    return FA_OK;
}

template <int D, int QM, bool PAD>
fa_status launch_decode(const fa::dec::Params& p, int64_t BH, cudaStream_t st)
{
    if (launch_pdl(fa::dec::fa_decode_partial_kernel<D, QM, PAD>, dim3((unsigned)p.splits, (unsigned)BH),
                   dim3(fa::dec::THREADS), 0, st, p) != cudaSuccess)
        return FA_ERR_CUDA;
    if (p.splits > 1 &&
        launch_pdl(fa::dec::fa_decode_combine_kernel<D>, dim3((unsigned)(BH * p.nq)), dim3(D), 0, st, p) != cudaSuccess)
        return FA_ERR_CUDA;
    return FA_OK;
}

template <int D, bool PAD>
fa_status launch_decode_d(const fa::dec::Params& p, int slots, int64_t BH, cudaStream_t st)
{
    switch (slots) {
    case 1: return launch_decode<D, 1, PAD>(p, BH, st);
    case 2: return launch_decode<D, 2, PAD>(p, BH, st);
    case 4: return launch_decode<D, 4, PAD>(p, BH, st);
    default: return launch_decode<D, 8, PAD>(p, BH, st);
    }
}

// Decode with an explicit workspace (ws, ws_bytes >= the plan's), once the
// arguments have passed decode_args.
fa_status decode_run(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B,
                     int64_t H, int64_t Nq, int64_t Nk, int64_t d, int causal, float scale, void* ws,
                     size_t ws_bytes, fa_stream_t stream)
{
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    const int64_t BH = B * H;
    const size_t qb = (size_t)(BH * Nq * d * 2), kb = (size_t)(BH * Nk * d * 2), lb = (size_t)(BH * Nq * 4);
    DecodePlan pl;
    const fa_status ps = device_decode_plan(dev, info, BH, Nq, Nk, d, &pl);
    if (ps != FA_OK) return ps;
    if (pl.ws_bytes > 0) {
        if (!ws || ws_bytes < pl.ws_bytes) return FA_ERR_INVALID_ARG;
        if (overlaps(ws, pl.ws_bytes, o, qb) || overlaps(ws, pl.ws_bytes, lse, lb) || overlaps(ws, pl.ws_bytes, q, qb) ||
            overlaps(ws, pl.ws_bytes, k, kb) || overlaps(ws, pl.ws_bytes, v, kb))
            return FA_ERR_INVALID_ARG;
    }

    fa::dec::Params p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.ws_o = static_cast<float*>(ws);
    p.ws_lse = pl.ws_bytes > 0 ? static_cast<float*>(ws) + (size_t)(BH * Nq * pl.splits) * (size_t)d : nullptr;
    p.nq = (int)Nq;
    p.nk = (int)Nk;
    p.d = (int)d;
    p.splits = pl.splits;
    p.chunk = pl.chunk;
    p.causal = causal;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // Head sizes below 64 or 128 run in that instance with the columns past d
    // read as zeros (PAD).
    if (d == 128) return launch_decode_d<128, false>(p, pl.slots, BH, st);
    if (d == 64) return launch_decode_d<64, false>(p, pl.slots, BH, st);
    return d > 64 ? launch_decode_d<128, true>(p, pl.slots, BH, st) : launch_decode_d<64, true>(p, pl.slots, BH, st);
}

// Scratch of fa_decode_static: compiled into the library, one per device.
static __device__ __align__(256) unsigned char g_decode_scratch[FA_DECODE_STATIC_SCRATCH_BYTES];

// Device address of g_decode_scratch on device `dev` (the current device),
// looked up once per device.
void* static_scratch(int dev)
{
    static std::atomic<void*> cache[MAX_DEVICES];
    static std::mutex lock;
    if (dev < 0 || dev >= MAX_DEVICES) return nullptr;
    void* p = cache[dev].load(std::memory_order_acquire);
    if (p) return p;
    std::lock_guard<std::mutex> guard(lock);
    p = cache[dev].load(std::memory_order_relaxed);
    if (!p) {
        if (cudaGetSymbolAddress(&p, g_decode_scratch) != cudaSuccess) return nullptr;
        cache[dev].store(p, std::memory_order_release);
    }
    return p;
}

// ---------------------------------------------------------- rotary positions

// Extent in elements of a (B, heads, N, d) view with element strides s.
int64_t extent(const int64_t s[3], int64_t B, int64_t H, int64_t N, int64_t d)
{
    return (B - 1) * s[0] + (H - 1) * s[1] + (N - 1) * s[2] + d;
}

// Strides of a view: non-negative, small enough that extents fit.
bool strides_ok(const int64_t s[3], int64_t B, int64_t H, int64_t N)
{
    const int64_t LIM = (int64_t)1 << 59;
    const int64_t n[3] = {B, H, N};
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || (n[i] > 1 && s[i] > LIM / (n[i] - 1))) return false;
    return true;
}

// No two elements of the view share a place: taken by rising stride, each
// dimension steps over all that the ones before it span.
bool no_overlap_within(const int64_t s[3], int64_t B, int64_t H, int64_t N, int64_t d)
{
    int64_t st[3] = {s[0], s[1], s[2]}, n[3] = {B, H, N};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) std::swap(st[i], st[j]), std::swap(n[i], n[j]);
    int64_t span = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (st[i] < span) return false;
        span += (n[i] - 1) * st[i];
    }
    return true;
}

struct RopeView {
    const void* p;
    int64_t s[3], H;
};

// Whether two views may share a place.  They cannot where their extents do not
// meet, nor where some pitch keeps them apart: strides that are multiples of it
// leave a place's remainder as it is, the others spread it over a run, and two runs
// that do not meet on the pitch's circle hold no common place.  That lets through the
// queries and keys of one buffer, by positions (a fused projection), by heads or by
// batches, with one position or many; a stride over one element means nothing.
bool may_overlap(const RopeView& x, const RopeView& y, int64_t B, int64_t N, int64_t d)
{
    if (!overlaps(x.p, (size_t)extent(x.s, B, x.H, N, d) * 2, y.p, (size_t)extent(y.s, B, y.H, N, d) * 2)) return false;
    const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p));
    if (bytes % 2) return true;
    const RopeView* const v[2] = {&x, &y};
    for (int k = 0; k < 6; ++k) {
        const int64_t n[2][3] = {{B, x.H, N}, {B, y.H, N}}, pitch = v[k / 3]->s[k % 3];
        if (pitch < 1 || n[k / 3][k % 3] == 1) continue;
        int64_t run[2] = {d, d};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 3; ++j)
                if (n[i][j] > 1 && v[i]->s[j] % pitch) run[i] += (n[i][j] - 1) * v[i]->s[j];
        const int64_t at = ((bytes / 2) % pitch + pitch) % pitch;  // y's run after x's
        if (run[0] <= at && run[1] <= pitch - at) return false;
    }
    return true;
}

template <int W>
fa_status launch_rope(const fa::rope::Params& p, dim3 block, int64_t blocks, cudaStream_t st)
{
    return launch_pdl(fa::rope::fa_rope_kernel<W>, dim3((unsigned)blocks), block, 0, st, p) == cudaSuccess ? FA_OK
                                                                                                           : FA_ERR_CUDA;
}

// --------------------------------------------------------------- 4-bit cache

// The sizes of a cache, as every call on one gives them.
fa_status qcache_check(const void* pool, int64_t num_pages, const int32_t* table, int64_t max_pages,
                       const int32_t* lens, int64_t B, int64_t Hkv, int64_t d)
{
    if (!pool || !table || !lens) return FA_ERR_INVALID_ARG;
    if (B < 1 || Hkv < 1 || d < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
    if (!head_size_ok(d)) return FA_ERR_UNSUPPORTED;
    if (B > 65535 || Hkv > 65535 || num_pages > INT32_MAX / Hkv || max_pages > INT32_MAX / fa::qc::PAGE / B)
        return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(pool) & 15u) != 0 ||
        ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lens)) & 3u) != 0)
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

size_t qcache_block_bytes(int64_t d) { return (size_t)(72 * padded_head_size(d)); }

bool scale_ok(float s) { return std::isfinite(s) && s > 0.0f; }

// A tensor's scale: times any e4m3 scale its reciprocal is a normal number, and
// so is a result's factor, scale / sum of probabilities.
bool tensor_scale_ok(float s) { return s >= 0x1p-60f && s <= 0x1p60f; }

// A written range of `n` bytes at p may overlap none of the cache's tensors.
bool hits_cache(const void* p, size_t n, const void* pool, int64_t num_pages, int64_t Hkv, int64_t d,
                const int32_t* table, int64_t max_pages, const int32_t* lens, int64_t B)
{
    return overlaps(p, n, pool, (size_t)(num_pages * Hkv) * qcache_block_bytes(d)) ||
           overlaps(p, n, table, (size_t)(B * max_pages) * 4) || overlaps(p, n, lens, (size_t)B * 4);
}

// Query rows of a kv head and how the kernels take them: NT column tiles of 8
// rows at a time.
struct QRows {
    int64_t rows, rb;
    int nt;
};
QRows qcache_rows(int64_t group, int64_t Nq)
{
    QRows r;
    r.rows = group * Nq;
    r.nt = r.rows <= 8 ? 1 : 2;
    r.rb = (r.rows + 8 * r.nt - 1) / (8 * r.nt);
    return r;
}

size_t qcache_part_bytes(int64_t Dp, int nt) { return (size_t)(8 * nt) * (size_t)(Dp + 2) * 4; }

// Blocks of the decode kernel: one an SM, no more than there can be pages.
int64_t qcache_decode_blocks(int sms, int64_t B, int64_t Hkv, int64_t rb, int64_t max_pages)
{
    return std::min<int64_t>(sms, B * Hkv * rb * max_pages);
}

size_t qcache_decode_ws(int64_t blocks, int64_t Dp, int nt)
{
    return (size_t)blocks * (2 * qcache_part_bytes(Dp, nt) + 8);
}

template <typename K>
fa_status allow_smem(K kernel, size_t bytes, std::atomic<int>* done, int dev)
{
    if (dev < 0 || dev >= MAX_DEVICES) return FA_ERR_CUDA;
    if (done[dev].load(std::memory_order_acquire)) return FA_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return FA_ERR_CUDA;
    done[dev].store(1, std::memory_order_release);
    return FA_OK;
}

template <int D, int NT, bool FOLD>
fa_status launch_qcache_decode(const fa::qc::DecParams& p, int64_t blocks, int dev, cudaStream_t st)
{
    using Y = fa::qc::DecLayout<D, NT>;
    static std::atomic<int> done[MAX_DEVICES];
    const fa_status as = allow_smem(fa::qc::fa_qcache_decode_kernel<D, NT, FOLD>, (size_t)Y::bytes(fa::qc::MAX_B), done, dev);
    if (as != FA_OK) return as;
    if (launch_pdl(fa::qc::fa_qcache_decode_kernel<D, NT, FOLD>, dim3((unsigned)blocks), dim3(Y::THREADS),
                   (size_t)Y::bytes(p.B), st, p) != cudaSuccess ||
        launch_pdl(fa::qc::fa_qcache_combine_kernel<D, NT>,
                   dim3((unsigned)blocks, (unsigned)std::min(p.rows, 8 * NT)), dim3(256), 0, st, p) != cudaSuccess)
        return FA_ERR_CUDA;
    return FA_OK;
}

template <int D, int NT>
fa_status launch_qcache_weights(const fa::qc::DecParams& p, int64_t blocks, int dev, cudaStream_t st)
{
    using Y = fa::qc::WeightLayout<D>;
    static std::atomic<int> done[MAX_DEVICES];
    const fa_status as = allow_smem(fa::qc::fa_qcache_weights_kernel<D, NT>, (size_t)Y::bytes(fa::qc::MAX_B), done, dev);
    if (as != FA_OK) return as;
    return launch_pdl(fa::qc::fa_qcache_weights_kernel<D, NT>, dim3((unsigned)blocks), dim3(Y::THREADS),
                      (size_t)Y::bytes(p.B), st, p) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

// Launches `kernel` like launch_pdl, in clusters of `cluster` blocks along x.
template <typename... KParams, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KParams...), dim3 grid, dim3 block, size_t smem, int cluster,
                            cudaStream_t st, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int C>
fa_status launch_qcache_select(fa::qc::EvictParams p, int64_t Hkv, int64_t B, int dev, cudaStream_t st)
{
    static std::atomic<int> done[MAX_DEVICES];
    const fa_status as = allow_smem(fa::qc::fa_qcache_select_kernel<C>, (size_t)fa::qc::SEL_HELD_MOST * 4, done, dev);
    if (as != FA_OK) return as;
    p.held = (int)std::min<int64_t>(((int64_t)p.max_pages * fa::qc::PAGE + C - 1) / C, fa::qc::SEL_HELD_MOST);
    return launch_clusters(fa::qc::fa_qcache_select_kernel<C>, dim3((unsigned)(Hkv * C), (unsigned)B),
                           dim3(fa::qc::SEL_THREADS), (size_t)p.held * 4, C, st, p) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

template <int D>
fa_status launch_qcache_move(const fa::qc::EvictParams& p, int64_t Hkv, int64_t B, int dev, cudaStream_t st)
{
    static std::atomic<int> done[MAX_DEVICES];
    constexpr size_t bytes = (size_t)fa::qc::MOVE_PAGES * fa::qc::Block<D>::BYTES;
    const fa_status as = allow_smem(fa::qc::fa_qcache_move_kernel<D>, bytes, done, dev);
    if (as != FA_OK) return as;
    return launch_clusters(fa::qc::fa_qcache_move_kernel<D>, dim3((unsigned)(Hkv * p.move_blocks), (unsigned)B),
                           dim3(fa::qc::MOVE_THREADS), bytes, p.move_blocks, st, p) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

// What decode and weights share: the query side.
fa_status qcache_query_check(const void* q, int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t max_pages,
                             int causal, float scale, float k_scale)
{
    if (!q) return FA_ERR_INVALID_ARG;
    if (H < 1 || Nq < 1 || H % Hkv != 0 || (causal != 0 && causal != 1) || !scale_ok(scale) || !tensor_scale_ok(k_scale) ||
        !scale_ok((float)((double)scale * 1.4426950408889634074 * (double)k_scale)))
        return FA_ERR_INVALID_ARG;
    if (Nq > fa::qc::MAX_NQ || B > fa::qc::MAX_B) return FA_ERR_UNSUPPORTED;
    if (H > INT32_MAX / 8 / B) return FA_ERR_INVALID_ARG;
    const QRows r = qcache_rows(H / Hkv, Nq);
    if (B * Hkv * r.rb > INT32_MAX / max_pages) return FA_ERR_INVALID_ARG;  // units are counted in 32 bits
    if ((reinterpret_cast<uintptr_t>(q) & 15u) != 0) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// Clears the status bits a check has read (and the wait code, if it is still
// the one read), leaving bits that kernels on other streams set since.
__global__ void fa_clear_status_kernel(unsigned int bits, unsigned int where)
{
    atomicAnd(&fa::g_status, ~bits);
    atomicCAS(&fa::g_status_where, where, 0u);
}

}  // namespace

extern "C" {

fa_status fa_decode_static(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B,
                           int64_t H, int64_t Nq, int64_t Nk, int64_t d, int causal, float scale,
                           fa_stream_t stream)
{
    // The argument checks come first, so that a call fa_decode would refuse
    // gets the same status here, whatever its sizes.
    const fa_status st = decode_args(q, k, v, o, lse, B, H, Nq, Nk, d, causal, scale, nullptr);
    if (st != FA_OK) return st;
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    DecodePlan pl;
    const fa_status ps = device_decode_plan(dev, info, B * H, Nq, Nk, d, &pl);
    if (ps != FA_OK) return ps;
    if (pl.ws_bytes > FA_DECODE_STATIC_SCRATCH_BYTES) return FA_ERR_TOO_LARGE;
    void* scratch = static_scratch(dev);
    if (!scratch) return FA_ERR_CUDA;
    return decode_run(q, k, v, o, lse, B, H, Nq, Nk, d, causal, scale, scratch, FA_DECODE_STATIC_SCRATCH_BYTES,
                      stream);
}

fa_status fa_decode_workspace_bytes(int64_t B, int64_t H, int64_t Nq, int64_t Nk, int64_t d, int causal,
                                    size_t* bytes)
{
    if (!bytes) return FA_ERR_INVALID_ARG;
    const fa_status st = decode_check(B, H, Nq, Nk, d, causal);
    if (st != FA_OK) return st;
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    DecodePlan pl;
    const fa_status ps = device_decode_plan(dev, info, B * H, Nq, Nk, d, &pl);
    if (ps != FA_OK) return ps;
    *bytes = pl.ws_bytes;
    return FA_OK;
}

fa_status fa_decode(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                    int64_t Nq, int64_t Nk, int64_t d, int causal, float scale, void* workspace,
                    size_t workspace_bytes, fa_stream_t stream)
{
    const fa_status st = decode_args(q, k, v, o, lse, B, H, Nq, Nk, d, causal, scale, workspace);
    if (st != FA_OK) return st;
    return decode_run(q, k, v, o, lse, B, H, Nq, Nk, d, causal, scale, workspace, workspace_bytes, stream);
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B,
                 int64_t H, int64_t N, int64_t d, int causal, float scale, fa_stream_t stream)
{
    // ---- argument checks (no CUDA call before these pass)
    if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || N < 1 || d < 1) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
    if (!head_size_ok(d)) return FA_ERR_UNSUPPORTED;
    const int64_t LIM = (int64_t)1 << 62;
    if (B > LIM / H || B * H > LIM / N || B * H * N > LIM / d) return FA_ERR_INVALID_ARG;
    const int64_t BH = B * H;
    const int64_t m_blocks = (N + fa::BM - 1) / fa::BM;
    if (BH > (((int64_t)1 << 31) - 1) / m_blocks) return FA_ERR_INVALID_ARG;
    if (N > INT32_MAX || BH > INT32_MAX) return FA_ERR_INVALID_ARG;
    const uintptr_t mis = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                          reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o);
    if ((mis & 15u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_UNSUPPORTED;
    const size_t tb = (size_t)(BH * N * d * 2), lb = (size_t)(BH * N * 4);
    if (overlaps(o, tb, q, tb) || overlaps(o, tb, k, tb) || overlaps(o, tb, v, tb) ||
        overlaps(o, tb, lse, lb) || overlaps(lse, lb, q, tb) || overlaps(lse, lb, k, tb) ||
        overlaps(lse, lb, v, tb))
        return FA_ERR_INVALID_ARG;

    // ---- device
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;

    CUtensorMap mq, mk, mv;
    if (!cached_map(&mq, q, BH, N, d, fa::BM) || !cached_map(&mk, k, BH, N, d, fa::BN) ||
        !cached_map(&mv, v, BH, N, d, fa::BN))
        return FA_ERR_CUDA;

    fa::Params p;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.N = (int)N;
    p.d = (int)d;
    p.num_m_blocks = (int)m_blocks;
    p.num_bh = (int)BH;
    p.num_items = (int)(BH * m_blocks);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.debug_skip_k = g_debug_skip_k.load(std::memory_order_relaxed);
    // Causal items differ in cost.  Heavy/light pairs of a head keep its K/V
    // in L2 while its blocks run; when all heads' K and V fit in L2 anyway,
    // ordering the items by cost balances the CTAs better (see item_of).
    // (fa_debug_set_schedule may force either order for tests.)
    const double kv_bytes = 2.0 * (double)BH * (double)N * (double)d * 2.0;
    const int forced = g_debug_schedule.load(std::memory_order_relaxed);
    const bool snake = causal && (forced < 0 ? kv_bytes <= 0.6 * (double)info.l2 : forced == 1);
    // One CTA per SM, at most one per work item (per pair of items in pair order).
    const unsigned grid = (unsigned)std::min<int64_t>(snake ? BH * m_blocks : (BH * m_blocks + 1) / 2, info.sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

    if (d == 128)
        return causal ? launch<128, true>(mq, mk, mv, p, grid, dev, st, snake)
                      : launch<128, false>(mq, mk, mv, p, grid, dev, st, snake);
    if (d == 64)
        return causal ? launch<64, true>(mq, mk, mv, p, grid, dev, st, snake)
                      : launch<64, false>(mq, mk, mv, p, grid, dev, st, snake);
    if (d > 64)
        return causal ? launch<128, true, true>(mq, mk, mv, p, grid, dev, st, snake)
                      : launch<128, false, true>(mq, mk, mv, p, grid, dev, st, snake);
    return causal ? launch<64, true, true>(mq, mk, mv, p, grid, dev, st, snake)
                  : launch<64, false, true>(mq, mk, mv, p, grid, dev, st, snake);
}

fa_status fa_bwd_workspace_bytes(int64_t B, int64_t H, int64_t N, int64_t d, size_t* bytes)
{
    if (!bytes) return FA_ERR_INVALID_ARG;
    BwdShape sh;
    const fa_status st = bwd_check(B, H, N, d, &sh);
    if (st != FA_OK) return st;
    *bytes = sh.ws_bytes;
    return FA_OK;
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                 void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t N, int64_t d, int causal, float scale,
                 void* workspace, size_t workspace_bytes, fa_stream_t stream)
{
    // ---- argument checks (no CUDA call before these pass)
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
    BwdShape sh;
    const fa_status chk = bwd_check(B, H, N, d, &sh);
    if (chk != FA_OK) return chk;
    if (workspace_bytes < sh.ws_bytes) return FA_ERR_INVALID_ARG;
    const uintptr_t mis = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                          reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o) |
                          reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(dq) |
                          reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv) |
                          reinterpret_cast<uintptr_t>(workspace);
    if ((mis & 15u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_UNSUPPORTED;
    const int64_t BH = sh.BH;
    const size_t tb = (size_t)(BH * N * d * 2), lb = (size_t)(BH * N * 4);
    // Outputs and the workspace may overlap no input and no other output.
    const void* ins[6] = {q, k, v, o, lse, dout};
    const size_t in_b[6] = {tb, tb, tb, tb, lb, tb};
    const void* outs[4] = {dq, dk, dv, workspace};
    const size_t out_b[4] = {tb, tb, tb, sh.ws_bytes};
    for (int a = 0; a < 4; ++a) {
        for (int b = 0; b < 6; ++b)
            if (overlaps(outs[a], out_b[a], ins[b], in_b[b])) return FA_ERR_INVALID_ARG;
        for (int b = a + 1; b < 4; ++b)
            if (overlaps(outs[a], out_b[a], outs[b], out_b[b])) return FA_ERR_INVALID_ARG;
    }

    // ---- device
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    const int sms = info.sms;
    float* const lse2 = static_cast<float*>(workspace);
    float* const dsum = lse2 + BH * sh.Np;
    float* const acc = dsum + BH * sh.Np;
    CUtensorMap mq, mk, mv, mdo, mdq;
    if (!cached_map(&mq, q, BH, N, d, fa::bwd::BQ) || !cached_map(&mk, k, BH, N, d, fa::bwd::BKV) ||
        !cached_map(&mv, v, BH, N, d, fa::bwd::BKV) || !cached_map(&mdo, dout, BH, N, d, fa::bwd::BQ) ||
        !make_acc_map(&mdq, acc, BH, sh.Np, sh.Dp))
        return FA_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

    // 1. D, L * log2 e, zeroed dQ accumulator.
    const int64_t rows = BH * sh.Np;
    fa::bwd::fa_bwd_prep_kernel<<<(unsigned)((rows + 8 * fa::bwd::PREP_ROWS - 1) / (8 * fa::bwd::PREP_ROWS)), 256, 0,
                                   st>>>(
        static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, lse2, dsum, acc,
        (int)N, (int)sh.Np, (int)d, (int)sh.Dp, rows);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;

    // 2. dK, dV and the dQ accumulator.
    fa::bwd::Params p;
    p.dk = static_cast<__nv_bfloat16*>(dk);
    p.dv = static_cast<__nv_bfloat16*>(dv);
    p.lse2 = lse2;
    p.dsum = dsum;
    p.dq_acc = acc;
    p.N = (int)N;
    p.d = (int)d;
    p.Np = (int)sh.Np;
    p.num_kb = (int)sh.num_kb;
    p.num_items = (int)(BH * sh.num_kb);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    p.scale = scale;
    p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.debug_skip_q = g_debug_skip_k.load(std::memory_order_relaxed);
    const unsigned grid = (unsigned)std::min<int64_t>((BH * sh.num_kb + 1) / 2, sms);
    fa_status ms;
    if (sh.Dp == 128)
        ms = causal ? launch_bwd_main<128, true>(mq, mk, mv, mdo, mdq, p, grid, dev, st)
                    : launch_bwd_main<128, false>(mq, mk, mv, mdo, mdq, p, grid, dev, st);
    else
        ms = causal ? launch_bwd_main<64, true>(mq, mk, mv, mdo, mdq, p, grid, dev, st)
                    : launch_bwd_main<64, false>(mq, mk, mv, mdo, mdq, p, grid, dev, st);
    if (ms != FA_OK) return ms;

    // 3. dQ = scale * accumulator, bf16.
    const int64_t n8 = BH * N * d / 8;
    fa::bwd::fa_bwd_dq_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, st>>>(
        acc, static_cast<__nv_bfloat16*>(dq), (int)N, (int)sh.Np, (int)d, (int)sh.Dp, n8, scale);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bias_gelu_dropout(const void* x, const void* bias, const uint32_t* keep, void* y, int64_t rows,
                               int64_t cols, float p, fa_stream_t stream)
{
    // ---- argument checks (no CUDA call before these pass)
    if (!x || !bias || !y) return FA_ERR_INVALID_ARG;
    if (rows < 1 || cols < 1 || !(p >= 0.0f && p < 1.0f)) return FA_ERR_INVALID_ARG;
    if (cols % 8 != 0) return FA_ERR_UNSUPPORTED;
    if (rows > ((int64_t)1 << 62) / cols || cols / 8 > INT32_MAX) return FA_ERR_INVALID_ARG;
    const uintptr_t mis = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(bias) |
                          reinterpret_cast<uintptr_t>(y);
    if ((mis & 15u) != 0 || (reinterpret_cast<uintptr_t>(keep) & 3u) != 0) return FA_ERR_UNSUPPORTED;
    const int64_t n = rows * cols;
    const size_t tb = (size_t)n * 2, bb = (size_t)cols * 2, kb = (size_t)((n + 31) / 32) * 4;
    if (overlaps(y, tb, x, tb) || overlaps(y, tb, bias, bb) || (keep && overlaps(y, tb, keep, kb)))
        return FA_ERR_INVALID_ARG;

    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    const int sms = info.sms;

    fa::ew::Params prm;
    prm.x = static_cast<const __nv_bfloat16*>(x);
    prm.bias = static_cast<const __nv_bfloat16*>(bias);
    prm.keep = reinterpret_cast<const uint8_t*>(keep);
    prm.y = static_cast<__nv_bfloat16*>(y);
    prm.n8 = n / 8;
    prm.cols8 = (int)(cols / 8);
    // Division by the invariant cols8 (Granlund and Montgomery's round-up
    // method for 31-bit numerators): magic = floor(2^(31+l) / cols8) + 1.
    int l = 0;
    while (((int64_t)1 << l) < (int64_t)prm.cols8) ++l;
    prm.magic = (uint32_t)((((uint64_t)1) << (31 + l)) / (uint64_t)prm.cols8 + 1);
    prm.shift = 31 + l;
    prm.scale = 1.0f / (1.0f - p);
    // Exactly the CTAs that are resident at once (one wave), each thread
    // keeping UNROLL 16-byte loads in flight, walking the tensor grid-stride.
    const bool wide = prm.n8 >= ((int64_t)1 << 31);
    const int per_sm = wide ? ew_ctas_per_sm<true>(dev) : ew_ctas_per_sm<false>(dev);
    if (per_sm <= 0) return FA_ERR_CUDA;
    const int64_t per_cta = (int64_t)fa::ew::THREADS * fa::ew::UNROLL;
    const unsigned grid =
        (unsigned)std::max<int64_t>(1, std::min<int64_t>((prm.n8 + per_cta - 1) / per_cta, (int64_t)per_sm * sms));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        wide ? launch_pdl(fa::ew::fa_bias_gelu_dropout_kernel<true>, dim3(grid), dim3(fa::ew::THREADS), 0, st, prm)
             : launch_pdl(fa::ew::fa_bias_gelu_dropout_kernel<false>, dim3(grid), dim3(fa::ew::THREADS), 0, st, prm);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_rope(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, void* q_out,
                  const int64_t* q_out_strides, void* k_out, const int64_t* k_out_strides, int64_t B, int64_t Hq,
                  int64_t Hk, int64_t N, int64_t d, const uint64_t* freqs, int64_t rot, int interleaved, float factor,
                  int inverse, const void* positions, int position_bytes, int64_t position_stride,
                  const int32_t* lens, fa_stream_t stream)
{
    // ---- argument checks (no CUDA call before these pass)
    if (!q || !q_out || !freqs || (k == nullptr) != (k_out == nullptr)) return FA_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || Hk < 0 || N < 1 || d < 1 || (k ? Hk < 1 : Hk != 0)) return FA_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) || !std::isfinite(factor))
        return FA_ERR_INVALID_ARG;
    if (rot < 2 || rot > d || rot % 2 != 0) return FA_ERR_INVALID_ARG;
    if (positions && ((position_bytes != 4 && position_bytes != 8) || position_stride < 0)) return FA_ERR_INVALID_ARG;
    if (positions && lens) return FA_ERR_INVALID_ARG;
    if (!head_size_ok(d)) return FA_ERR_UNSUPPORTED;
    const int64_t LIM = (int64_t)1 << 59;
    if (Hq > INT32_MAX / 2 || Hk > INT32_MAX / 2 || B > LIM / (Hq + Hk) || B * (Hq + Hk) > LIM / N ||
        B * (Hq + Hk) * N > LIM / d || (positions && position_stride > LIM / B))
        return FA_ERR_INVALID_ARG;
    RopeView v[4] = {{q, {}, Hq}, {k, {}, Hk}, {q_out, {}, Hq}, {k_out, {}, Hk}};
    const int64_t* given[4] = {q_strides, k_strides, q_out_strides, k_out_strides};
    const int count = k ? 2 : 1;
    uintptr_t places = 0;  // the low bits that any row's address can have
    for (int i = 0; i < 4; ++i) {
        if (i % 2 >= count) continue;
        v[i].s[0] = given[i] ? given[i][0] : v[i].H * N * d;
        v[i].s[1] = given[i] ? given[i][1] : N * d;
        v[i].s[2] = given[i] ? given[i][2] : d;
        if (!strides_ok(v[i].s, B, v[i].H, N)) return FA_ERR_INVALID_ARG;
        const int64_t n[3] = {B, v[i].H, N};
        for (int j = 0; j < 3; ++j)
            if (n[j] > 1) places |= (uintptr_t)v[i].s[j] * 2;
        places |= reinterpret_cast<uintptr_t>(v[i].p);
        if ((reinterpret_cast<uintptr_t>(v[i].p) & 1u) != 0) return FA_ERR_UNSUPPORTED;
    }
    const uintptr_t pos_mask = positions ? (uintptr_t)position_bytes - 1 : 0;
    if ((reinterpret_cast<uintptr_t>(freqs) & 7u) != 0 || (reinterpret_cast<uintptr_t>(positions) & pos_mask) != 0 ||
        (reinterpret_cast<uintptr_t>(lens) & 3u) != 0)
        return FA_ERR_UNSUPPORTED;
    for (int i = 0; i < count; ++i) {
        const RopeView& out = v[2 + i];
        if (!no_overlap_within(out.s, B, out.H, N, d)) return FA_ERR_INVALID_ARG;
        const size_t nb = (size_t)extent(out.s, B, out.H, N, d) * 2;
        if (overlaps(out.p, nb, freqs, (size_t)rot * 4) || (lens && overlaps(out.p, nb, lens, (size_t)B * 4)) ||
            (positions &&
             overlaps(out.p, nb, positions, (size_t)((B - 1) * position_stride + N) * (size_t)position_bytes)))
            return FA_ERR_INVALID_ARG;
        for (int j = 0; j < count; ++j) {
            const RopeView& in = v[j];
            const bool in_place = i == j && out.p == in.p && (B == 1 || out.s[0] == in.s[0]) &&
                                  (out.H == 1 || out.s[1] == in.s[1]) && (N == 1 || out.s[2] == in.s[2]);
            if (!in_place && may_overlap(out, in, B, N, d)) return FA_ERR_INVALID_ARG;
        }
    }
    if (count == 2 && may_overlap(v[2], v[3], B, N, d)) return FA_ERR_INVALID_ARG;

    // ---- device
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;

    fa::rope::Params p = {};
    for (int i = 0; i < 2; ++i) {
        p.in[i] = {static_cast<__nv_bfloat16*>(const_cast<void*>(v[i].p)), v[i].s[0], v[i].s[1], v[i].s[2]};
        p.out[i] = {static_cast<__nv_bfloat16*>(const_cast<void*>(v[2 + i].p)), v[2 + i].s[0], v[2 + i].s[1], v[2 + i].s[2]};
    }
    p.heads[0] = (int)Hq;
    p.heads[1] = (int)Hk;
    p.freqs = freqs;
    p.positions = positions;
    p.pos_sb = position_stride;
    p.lens = lens;
    p.wide = position_bytes == 8;
    p.n = N;
    p.d = (int)d;
    p.rot = (int)rot;
    p.interleaved = interleaved;
    p.stream = (double)B * (double)(Hq + Hk) * (double)N * (double)d * 2.0 > (double)info.l2;
    p.factor = factor;
    p.sign = inverse ? -1.0f : 1.0f;
    // Whole 16-byte vectors turn together when the halves (or the end of the
    // turned part) fall on vector borders, else whole words, else single pairs.
    // B4 16 + 4 heads N2048 d80: 64 turned channels (16 bytes) 14.4 us, 36 (4
    // bytes) 17.6 us, 38 (2 bytes) 28.8 us.
    auto fits = [&](int64_t w) { return places % (uintptr_t)(2 * w) == 0 && rot % (interleaved ? w : 2 * w) == 0; };
    const int64_t w = fits(8) ? 8 : fits(2) ? 2 : 1;
    const int64_t units = interleaved ? (d + 2 * w - 1) / (2 * w) : rot / (2 * w) + (d - rot + 2 * w - 1) / (2 * w);
    const int64_t room = fa::rope::THREADS / units;
    // (A block's z is at most 64 on any device; ny <= THREADS is within y's 1024.)
    const int64_t ny = std::min<int64_t>(N, room), nz = std::max<int64_t>(1, std::min<int64_t>({room / ny, Hq + Hk, 64}));
    const int64_t total = Hq + Hk, tiles = (N + ny - 1) / ny;
    const int64_t head_tiles = (total + nz * fa::rope::U - 1) / (nz * fa::rope::U);
    if (tiles > INT32_MAX || B * head_tiles > INT32_MAX / tiles) return FA_ERR_INVALID_ARG;
    p.tiles = (int)tiles;
    p.head_tiles = (int)head_tiles;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 block((unsigned)units, (unsigned)ny, (unsigned)nz);
    const int64_t blocks = B * tiles * head_tiles;
    return w == 8   ? launch_rope<8>(p, block, blocks, st)
           : w == 2 ? launch_rope<2>(p, block, blocks, st)
                    : launch_rope<1>(p, block, blocks, st);
}

fa_status fa_qcache_append(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides, int64_t B,
                           int64_t Hkv, int64_t N, int64_t d, float k_scale, float v_scale, void* pool,
                           int64_t num_pages, const int32_t* table, int64_t max_pages, const int32_t* lens,
                           fa_stream_t stream)
{
    if (!k || !v) return FA_ERR_INVALID_ARG;
    const fa_status cs = qcache_check(pool, num_pages, table, max_pages, lens, B, Hkv, d);
    if (cs != FA_OK) return cs;
    if (N < 1 || N > INT32_MAX / 2 || !tensor_scale_ok(k_scale) || !tensor_scale_ok(v_scale)) return FA_ERR_INVALID_ARG;
    const int64_t LIM = (int64_t)1 << 59;
    if (B * Hkv > LIM / N || B * Hkv * N > LIM / d) return FA_ERR_INVALID_ARG;
    int64_t s[2][3];
    const int64_t* given[2] = {k_strides, v_strides};
    const void* rows[2] = {k, v};
    for (int i = 0; i < 2; ++i) {
        s[i][0] = given[i] ? given[i][0] : Hkv * N * d;
        s[i][1] = given[i] ? given[i][1] : N * d;
        s[i][2] = given[i] ? given[i][2] : d;
        if (!strides_ok(s[i], B, Hkv, N)) return FA_ERR_INVALID_ARG;
        const int64_t n[3] = {B, Hkv, N};
        for (int j = 0; j < 3; ++j)
            if (n[j] > 1 && s[i][j] % 8 != 0) return FA_ERR_UNSUPPORTED;
        if ((reinterpret_cast<uintptr_t>(rows[i]) & 15u) != 0) return FA_ERR_UNSUPPORTED;
        const size_t nb = (size_t)extent(s[i], B, Hkv, N, d) * 2;
        if (overlaps(pool, (size_t)(num_pages * Hkv) * qcache_block_bytes(d), rows[i], nb)) return FA_ERR_INVALID_ARG;
    }
    if (overlaps(pool, (size_t)(num_pages * Hkv) * qcache_block_bytes(d), table, (size_t)(B * max_pages) * 4) ||
        overlaps(pool, (size_t)(num_pages * Hkv) * qcache_block_bytes(d), lens, (size_t)B * 4))
        return FA_ERR_INVALID_ARG;

    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    fa::qc::RowParams p = {};
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.ksb = s[0][0], p.ksh = s[0][1], p.ksn = s[0][2];
    p.vsb = s[1][0], p.vsh = s[1][1], p.vsn = s[1][2];
    p.pool = static_cast<uint8_t*>(pool);
    p.table = table;
    p.lens = lens;
    p.n = N;
    p.hkv = (int)Hkv;
    p.d = (int)d;
    p.max_pages = (int)max_pages;
    p.num_pages = (int)num_pages;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_inv_six = (float)(1.0 / (6.0 * (double)k_scale));
    p.v_inv_six = (float)(1.0 / (6.0 * (double)v_scale));
    // Pages that N keys can touch, wherever they begin.
    const int64_t pages = std::min<int64_t>((N - 1 + fa::qc::PAGE - 1) / fa::qc::PAGE + 1, max_pages);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)pages, (unsigned)Hkv, (unsigned)B);
    // Powers of two (1 is the usual one) need no look at remainders: 4 x 8 heads x 4096
    // keys at d = 128 in 17.4 us, with other scales 21.6 (8 x 16 x 8192 keys: 109, 137).
    auto pow2 = [](float x) {
        int ex;
        return std::frexp(x, &ex) == 0.5f;
    };
    auto launch = [&](auto* kernel) { return launch_pdl(kernel, grid, dim3(fa::qc::ROW_THREADS), 0, st, p); };
    const bool easy = pow2(k_scale) && pow2(v_scale);
    const cudaError_t e =
        padded_head_size(d) == 128
            ? (easy ? launch(fa::qc::fa_qcache_append_kernel<128, true>) : launch(fa::qc::fa_qcache_append_kernel<128, false>))
            : (easy ? launch(fa::qc::fa_qcache_append_kernel<64, true>) : launch(fa::qc::fa_qcache_append_kernel<64, false>));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_qcache_read(const void* pool, int64_t num_pages, const int32_t* table, int64_t max_pages,
                         const int32_t* lens, void* k, void* v, int64_t B, int64_t Hkv, int64_t N, int64_t d,
                         int newest, float k_scale, float v_scale, fa_stream_t stream)
{
    if (!k || !v) return FA_ERR_INVALID_ARG;
    const fa_status cs = qcache_check(pool, num_pages, table, max_pages, lens, B, Hkv, d);
    if (cs != FA_OK) return cs;
    if (N < 1 || N > INT32_MAX / 2 || (newest != 0 && newest != 1) || !tensor_scale_ok(k_scale) ||
        !tensor_scale_ok(v_scale))
        return FA_ERR_INVALID_ARG;
    const int64_t LIM = (int64_t)1 << 59;
    if (B * Hkv > LIM / N || B * Hkv * N > LIM / d) return FA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) != 0) return FA_ERR_UNSUPPORTED;
    const size_t nb = (size_t)(B * Hkv * N * d) * 2;
    if (overlaps(k, nb, v, nb) || hits_cache(k, nb, pool, num_pages, Hkv, d, table, max_pages, lens, B) ||
        hits_cache(v, nb, pool, num_pages, Hkv, d, table, max_pages, lens, B))
        return FA_ERR_INVALID_ARG;

    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    fa::qc::RowParams p = {};
    p.ko = static_cast<__nv_bfloat16*>(k);
    p.vo = static_cast<__nv_bfloat16*>(v);
    p.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
    p.table = table;
    p.lens = lens;
    p.n = N;
    p.hkv = (int)Hkv;
    p.d = (int)d;
    p.max_pages = (int)max_pages;
    p.num_pages = (int)num_pages;
    p.newest = newest;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)((N + fa::qc::PAGE - 1) / fa::qc::PAGE), (unsigned)Hkv, (unsigned)B);
    const cudaError_t e =
        padded_head_size(d) == 128
            ? launch_pdl(fa::qc::fa_qcache_read_kernel<128>, grid, dim3(fa::qc::ROW_THREADS), 0, st, p)
            : launch_pdl(fa::qc::fa_qcache_read_kernel<64>, grid, dim3(fa::qc::ROW_THREADS), 0, st, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_qcache_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t d, int64_t max_pages,
                                           size_t* bytes)
{
    if (!bytes || B < 1 || H < 1 || Hkv < 1 || Nq < 1 || d < 1 || max_pages < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (!head_size_ok(d) || Nq > fa::qc::MAX_NQ || B > fa::qc::MAX_B) return FA_ERR_UNSUPPORTED;
    if (H > INT32_MAX / 8 / B) return FA_ERR_INVALID_ARG;
    const QRows r = qcache_rows(H / Hkv, Nq);
    if (max_pages > INT32_MAX / fa::qc::PAGE / B || B * Hkv * r.rb > INT32_MAX / max_pages) return FA_ERR_INVALID_ARG;
    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    *bytes = qcache_decode_ws(qcache_decode_blocks(info.sms, B, Hkv, r.rb, max_pages), padded_head_size(d), r.nt);
    return FA_OK;
}

fa_status fa_qcache_decode(const void* q, const void* pool, int64_t num_pages, const int32_t* table, int64_t max_pages,
                           const int32_t* lens, void* o, float* lse, int64_t B, int64_t H, int64_t Hkv, int64_t Nq,
                           int64_t d, int causal, float scale, float k_scale, float v_scale, void* workspace,
                           size_t workspace_bytes, fa_stream_t stream)
{
    if (!o || !lse || !workspace) return FA_ERR_INVALID_ARG;
    const fa_status cs = qcache_check(pool, num_pages, table, max_pages, lens, B, Hkv, d);
    if (cs != FA_OK) return cs;
    const fa_status qs = qcache_query_check(q, B, H, Hkv, Nq, max_pages, causal, scale, k_scale);
    if (qs != FA_OK) return qs;
    if (!tensor_scale_ok(v_scale)) return FA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(workspace)) & 15u) != 0 ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
        return FA_ERR_UNSUPPORTED;
    const size_t qb = (size_t)(B * H * Nq * d) * 2, lb = (size_t)(B * H * Nq) * 4;
    if (overlaps(o, qb, q, qb) || overlaps(o, qb, lse, lb) || overlaps(lse, lb, q, qb) ||
        hits_cache(o, qb, pool, num_pages, Hkv, d, table, max_pages, lens, B) ||
        hits_cache(lse, lb, pool, num_pages, Hkv, d, table, max_pages, lens, B))
        return FA_ERR_INVALID_ARG;

    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    const QRows r = qcache_rows(H / Hkv, Nq);
    const int64_t Dp = padded_head_size(d);
    const int64_t blocks = qcache_decode_blocks(info.sms, B, Hkv, r.rb, max_pages);
    const size_t need = qcache_decode_ws(blocks, Dp, r.nt);
    if (workspace_bytes < need || overlaps(workspace, need, q, qb) || overlaps(workspace, need, o, qb) ||
        overlaps(workspace, need, lse, lb) ||
        hits_cache(workspace, need, pool, num_pages, Hkv, d, table, max_pages, lens, B))
        return FA_ERR_INVALID_ARG;
    fa::qc::DecParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.pool = static_cast<const uint8_t*>(pool);
    p.table = table;
    p.lens = lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.ws = static_cast<float*>(workspace);
    p.desc = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + (size_t)blocks * 2 * qcache_part_bytes(Dp, r.nt));
    p.B = (int)B;
    p.hkv = (int)Hkv;
    p.nq = (int)Nq;
    p.rows = (int)r.rows;
    p.rb = (int)r.rb;
    p.d = (int)d;
    p.max_pages = (int)max_pages;
    p.num_pages = (int)num_pages;
    p.causal = causal;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074 * (double)k_scale);
    p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.debug_skip = g_debug_skip_k.load(std::memory_order_relaxed);
    p.v_scale = v_scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (Dp == 128)
        return r.rows <= 4 ? launch_qcache_decode<128, 1, true>(p, blocks, dev, st)
               : r.nt == 1 ? launch_qcache_decode<128, 1, false>(p, blocks, dev, st)
                           : launch_qcache_decode<128, 2, false>(p, blocks, dev, st);
    return r.rows <= 4 ? launch_qcache_decode<64, 1, true>(p, blocks, dev, st)
           : r.nt == 1 ? launch_qcache_decode<64, 1, false>(p, blocks, dev, st)
                       : launch_qcache_decode<64, 2, false>(p, blocks, dev, st);
}

fa_status fa_qcache_weights(const void* q, const float* lse, const void* pool, int64_t num_pages, const int32_t* table,
                            int64_t max_pages, const int32_t* lens, const float* weights, float* weights_out,
                            int64_t W, int64_t B, int64_t H, int64_t Hkv, int64_t Nq, int64_t d, int causal,
                            float scale, float k_scale, fa_stream_t stream)
{
    if (!lse || !weights || !weights_out) return FA_ERR_INVALID_ARG;
    const fa_status cs = qcache_check(pool, num_pages, table, max_pages, lens, B, Hkv, d);
    if (cs != FA_OK) return cs;
    const fa_status qs = qcache_query_check(q, B, H, Hkv, Nq, max_pages, causal, scale, k_scale);
    if (qs != FA_OK) return qs;
    if (W < 1 || W > INT32_MAX) return FA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(weights) |
          reinterpret_cast<uintptr_t>(weights_out)) & 3u) != 0)
        return FA_ERR_UNSUPPORTED;
    const size_t qb = (size_t)(B * H * Nq * d) * 2, lb = (size_t)(B * H * Nq) * 4, wb = (size_t)(B * Hkv * W) * 4;
    if ((weights != weights_out && overlaps(weights_out, wb, weights, wb)) || overlaps(weights_out, wb, q, qb) ||
        overlaps(weights_out, wb, lse, lb) ||
        hits_cache(weights_out, wb, pool, num_pages, Hkv, d, table, max_pages, lens, B))
        return FA_ERR_INVALID_ARG;

    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    const QRows r = qcache_rows(H / Hkv, Nq);
    fa::qc::DecParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.pool = static_cast<const uint8_t*>(pool);
    p.table = table;
    p.lens = lens;
    p.lse_in = lse;
    p.w_in = weights;
    p.w_out = weights_out;
    p.w_len = W;
    p.B = (int)B;
    p.hkv = (int)Hkv;
    p.nq = (int)Nq;
    p.rows = (int)r.rows;
    p.rb = (int)r.rb;
    p.d = (int)d;
    p.max_pages = (int)max_pages;
    p.num_pages = (int)num_pages;
    p.causal = causal;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074 * (double)k_scale);
    p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.debug_skip = g_debug_skip_k.load(std::memory_order_relaxed);
    const int64_t blocks = std::min<int64_t>((int64_t)info.sms * 2, B * Hkv * max_pages);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (padded_head_size(d) == 128)
        return r.nt == 1 ? launch_qcache_weights<128, 1>(p, blocks, dev, st) : launch_qcache_weights<128, 2>(p, blocks, dev, st);
    return r.nt == 1 ? launch_qcache_weights<64, 1>(p, blocks, dev, st) : launch_qcache_weights<64, 2>(p, blocks, dev, st);
}

fa_status fa_qcache_evict(void* pool, int64_t num_pages, const int32_t* table, int64_t max_pages, const int32_t* lens,
                          const int32_t* table_out, int64_t max_pages_out, const float* weights, float* weights_out,
                          int64_t W, int32_t* kept, int32_t* lens_out, int64_t B, int64_t Hkv, int64_t d, int64_t keep,
                          int64_t sink, int64_t recent, fa_stream_t stream)
{
    if (!table_out || !weights || !weights_out || !kept || !lens_out) return FA_ERR_INVALID_ARG;
    const fa_status cs = qcache_check(pool, num_pages, table, max_pages, lens, B, Hkv, d);
    if (cs != FA_OK) return cs;
    if (W < 1 || W > INT32_MAX || keep < 1 || keep > INT32_MAX / 2 || sink < 0 || recent < 0 || sink > keep ||
        recent > keep - sink)
        return FA_ERR_INVALID_ARG;
    const int64_t need = (keep + fa::qc::PAGE - 1) / fa::qc::PAGE;
    if (max_pages_out < std::min(need, max_pages) || max_pages_out > INT32_MAX / fa::qc::PAGE / B) return FA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(table_out) | reinterpret_cast<uintptr_t>(weights) |
          reinterpret_cast<uintptr_t>(weights_out) | reinterpret_cast<uintptr_t>(kept) |
          reinterpret_cast<uintptr_t>(lens_out)) & 3u) != 0)
        return FA_ERR_UNSUPPORTED;
    const size_t wb = (size_t)(B * Hkv * W) * 4, kb = (size_t)(B * Hkv * keep) * 4, lb = (size_t)B * 4;
    const size_t tb = (size_t)(B * max_pages_out) * 4;
    const void* outs[3] = {weights_out, kept, lens_out};
    const size_t out_b[3] = {wb, kb, lb};
    for (int i = 0; i < 3; ++i) {
        if (overlaps(outs[i], out_b[i], weights, wb) || overlaps(outs[i], out_b[i], table_out, tb) ||
            hits_cache(outs[i], out_b[i], pool, num_pages, Hkv, d, table, max_pages, lens, B))
            return FA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], out_b[i], outs[j], out_b[j])) return FA_ERR_INVALID_ARG;
    }
    const size_t pb = (size_t)(num_pages * Hkv) * qcache_block_bytes(d);
    if (overlaps(pool, pb, table, (size_t)(B * max_pages) * 4) || overlaps(pool, pb, lens, lb) ||
        overlaps(pool, pb, table_out, tb) || overlaps(pool, pb, weights, wb))
        return FA_ERR_INVALID_ARG;

    int dev = -1;
    DevInfo info;
    const fa_status ds = sm103_device(&dev, &info);
    if (ds != FA_OK) return ds;
    fa::qc::EvictParams p = {};
    p.pool = static_cast<uint8_t*>(pool);
    p.table = table;
    p.lens = lens;
    p.table_out = table_out;
    p.w_in = weights;
    p.w_out = weights_out;
    p.kept = kept;
    p.lens_out = lens_out;
    p.w_len = W;
    p.hkv = (int)Hkv;
    p.max_pages = (int)max_pages;
    p.max_pages_out = (int)max_pages_out;
    p.num_pages = (int)num_pages;
    p.keep = (int)keep;
    p.sink = (int)sink;
    p.recent = (int)recent;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // A cluster of 4 blocks a head pays where heads are long and few; one block
    // a head where they fill the SMs anyway.  (The lengths are on the device: the
    // rule goes by the table's room, and the figures are of full tables.)  Whole
    // call in us, cluster against one block, cutting 64-channel heads back to 64
    // keys: 8 heads of 2048 keys 10.4 / 9.2, of 8192 11.5 / 13.8; 64 heads of 8192
    // 20.5 / 16.4, of 32768 30.0 / 35.4; 256 heads of 16384 51.8 / 33.6, of 65536
    // 112 / 330.
    const int64_t heads = B * Hkv, most = max_pages * fa::qc::PAGE;
    const bool wide = most > (heads * 4 <= info.sms ? 4096 : heads <= info.sms ? 16384 : 32768);
    const fa_status ss = wide ? launch_qcache_select<4>(p, Hkv, B, dev, st) : launch_qcache_select<1>(p, Hkv, B, dev, st);
    if (ss != FA_OK) return ss;
    // Blocks of a head's move: one for each kept page, at most 8, and where there
    // are heads enough one for every 4 pages.
    const int64_t pages = std::min(need, max_pages);
    int blocks = 1;
    while (blocks < 8 && blocks < pages) blocks *= 2;
    while (blocks > 1 && heads * blocks > 4 * info.sms && blocks / 2 * fa::qc::MOVE_PAGES >= pages) blocks /= 2;
    p.move_blocks = blocks;
    return padded_head_size(d) == 128 ? launch_qcache_move<128>(p, Hkv, B, dev, st)
                                      : launch_qcache_move<64>(p, Hkv, B, dev, st);
}

fa_status fa_check_device_status(fa_stream_t stream, uint32_t* where)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    unsigned int h[2] = {0u, 0u};
    if (cudaMemcpyFromSymbolAsync(&h[0], fa::g_status, sizeof(unsigned int), 0,
                                  cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&h[1], fa::g_status_where, sizeof(unsigned int), 0,
                                  cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return FA_ERR_CUDA;
    if (where) *where = h[1];
    if (h[0] != 0u) {
        const fa_status st_code = (h[0] & fa::STATUS_TIMEOUT)    ? FA_ERR_TIMEOUT
                                  : (h[0] & fa::STATUS_BAD_SMEM) ? FA_ERR_CUDA
                                                                 : FA_ERR_INVALID_ARG;  // STATUS_BAD_PAGE
        // Clear what was read, atomically on the device: a bit that a kernel
        // on another stream set in between stays for the next check.
        fa_clear_status_kernel<<<1, 1, 0, st>>>(h[0], h[1]);
        if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) return FA_ERR_CUDA;
        return st_code;
    }
    return FA_OK;
}

fa_status fa_get_device_status(fa_stream_t stream) { return fa_check_device_status(stream, nullptr); }

fa_status fa_set_wait_limit_ns(uint64_t ns)
{
    g_wait_limit_ns.store(ns ? ns : DEFAULT_WAIT_LIMIT_NS, std::memory_order_relaxed);
    return FA_OK;
}

fa_status fa_debug_skip_k_tile(int tile)
{
    if (tile < -1) return FA_ERR_INVALID_ARG;
    g_debug_skip_k.store(tile, std::memory_order_relaxed);
    return FA_OK;
}

fa_status fa_debug_decode_plan(int64_t B, int64_t H, int64_t Nq, int64_t Nk, int64_t d, int64_t wave, int* splits,
                               int* chunk)
{
    if (!splits || !chunk || wave < 1) return FA_ERR_INVALID_ARG;
    const fa_status st = decode_check(B, H, Nq, Nk, d, 0);
    if (st != FA_OK) return st;
    const DecodePlan pl = decode_plan(B * H, Nq, Nk, d, wave);
    *splits = pl.splits;
    *chunk = pl.chunk;
    return FA_OK;
}

fa_status fa_debug_set_schedule(int order)
{
    if (order < -1 || order > 1) return FA_ERR_INVALID_ARG;
    g_debug_schedule.store(order, std::memory_order_relaxed);
    return FA_OK;
}

const char* fa_status_string(fa_status s)
{
    switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported (head size, alignment or device)";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "kernel pipeline wait timed out";
    case FA_ERR_TOO_LARGE: return "the sizes need more scratch than the library's static array holds";
    }
    return "unknown status";
}

int fa_version(void) { return FA_VERSION; }

#ifdef FA_TRACE
// Trace builds only: points the kernels' event trace at a device buffer.
int fa_debug_set_trace(void* device_buffer)
{
    unsigned long long* p = static_cast<unsigned long long*>(device_buffer);
    return cudaMemcpyToSymbol(fa::g_trace, &p, sizeof p) == cudaSuccess ? 0 : 1;
}
#endif

}  // extern "C"
