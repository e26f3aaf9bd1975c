// C ABI of the paged GQA decode library (declared in include/pgd.h):
// argument validation, the partition scheduler, TMA descriptor encoding,
// scratch management and the kernel launches.  Nothing here runs any part
// of the attention arithmetic on the host.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <algorithm>
#include <atomic>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>
#include <unordered_map>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pgd.h"
#include "pgd_internal.h"

// Scratch of paged_gqa_decode_noalloc: a fixed array in this library's
// device image, so that entry point never allocates.  Every GPU on which the
// library is used holds these PGD_NOALLOC_SCRATCH_BYTES until the process
// exits.  All calls of paged_gqa_decode_noalloc on a device share it.
static __device__ __align__(256) unsigned char pgd_noalloc_scratch[PGD_NOALLOC_SCRATCH_BYTES];

namespace pgd {
namespace {

thread_local std::string t_last_error;
thread_local int t_last_partition = 0;
thread_local cudaEvent_t t_ev_before = nullptr;
thread_local cudaEvent_t t_ev_after = nullptr;
thread_local const unsigned *t_stall_flag = nullptr;  // pgd_test_stall_next_decode
thread_local bool t_skip_reduce = false;               // pgd_test_fail_next_reduce
thread_local bool t_fail_set_up = false;               // pgd_test_fail_next_set_up

pgd_status fail(pgd_status st, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    t_last_error = buf;
    return st;
}

pgd_status cuda_fail(cudaError_t e, const char *what)
{
    return fail(PGD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// ------------------------------------------------------------------ per-device state
constexpr int kMaxDevices = 64;

struct DeviceState {
    std::once_flag once;
    cudaError_t init_error = cudaSuccess;
    int num_sms = 0;
    int ctas[3][3][5] = {};         // [kind: fp16, quantised, MQ][head_dim 64/128/256][block size]
    // set up by the first call that needs them, so that no other call pays for
    // them or fails with them
    std::atomic<int> tree_runs[3][2] = {};       // [head_dim][pairs]: resident runs, 0: not set up
    std::atomic<bool> prefill_ready[3] = {};     // [head_dim]
    std::atomic<int> latent_runs[3] = {};        // [latent_dim 128/256/512]: resident pairs
    std::atomic<bool> latent_prefill_ready[2] = {};  // [head_dim 64/128]
    unsigned *err_word = nullptr;   // address of g_device_error on this device
    std::mutex pool_mu;             // the pool is made on first library-owned scratch
    cudaMemPool_t pool = nullptr;   //   (and again after pgd_release): stream-ordered scratch
};

DeviceState g_dev[kMaxDevices];

__device__ unsigned g_device_error;

constexpr int kBlockSizes[5] = {8, 16, 32, 64, 128};

bool supported_head_dim(int D) { return D == 64 || D == 128 || D == 256; }
bool supported_block_size(int BS)
{
    for (int b : kBlockSizes)
        if (b == BS)
            return true;
    return false;
}
int d_index(int D) { return D == 64 ? 0 : D == 128 ? 1 : 2; }
int bs_index(int bs) { return bs == 8 ? 0 : bs == 16 ? 1 : bs == 32 ? 2 : bs == 64 ? 3 : 4; }
// Tokens per pipeline stage of the partition kernel for head_dim D.
int stage_tokens(int D)
{
    return D == 64 ? Shape<64>::T : D == 128 ? Shape<128>::T : Shape<256>::T;
}

cudaError_t init_device(int dev, DeviceState &st)
{
    cudaError_t e = cudaDeviceGetAttribute(&st.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    for (int kind = 0; kind < 3; ++kind)
        for (int i = 0; i < 5; ++i) {
            if ((e = occupancy_d64(kBlockSizes[i], kind, &st.ctas[kind][0][i])) != cudaSuccess)
                return e;
            if ((e = occupancy_d128(kBlockSizes[i], kind, &st.ctas[kind][1][i])) != cudaSuccess)
                return e;
            if ((e = occupancy_d256(kBlockSizes[i], kind, &st.ctas[kind][2][i])) != cudaSuccess)
                return e;
        }
    return cudaGetSymbolAddress(reinterpret_cast<void **>(&st.err_word), g_device_error);
}

cudaError_t create_pool(int dev, DeviceState &st)
{
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaError_t e = cudaMemPoolCreate(&st.pool, &props);
    if (e != cudaSuccess)
        return e;
    uint64_t keep = ~0ull;  // keep freed scratch in the pool between calls
    return cudaMemPoolSetAttribute(st.pool, cudaMemPoolAttrReleaseThreshold, &keep);
}

cudaError_t init_pool(int dev, DeviceState &st)
{
    // The call that needs it first may be captured into a graph.  A pool is no part
    // of any stream's work, so its creation is allowed there.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess)
        return e;
    e = create_pool(dev, st);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    return e != cudaSuccess ? e : back;
}

pgd_status device_state(DeviceState **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(PGD_ERR_UNSUPPORTED, "device ordinal %d beyond %d", dev, kMaxDevices);
    DeviceState &st = g_dev[dev];
    std::call_once(st.once, [&] { st.init_error = init_device(dev, st); });
    if (st.init_error != cudaSuccess)
        return cuda_fail(st.init_error, "device set-up");
    *out = &st;
    return PGD_OK;
}

// Sets a kernel up on the current device by `f` (which a test may have fail).  A
// failure is this call's alone: the next one tries again.
template <class F> pgd_status set_up(const char *what, F &&f)
{
    const bool withheld = t_fail_set_up;
    t_fail_set_up = false;
    if (withheld)
        return fail(PGD_ERR_CUDA, "%s: withheld by pgd_test_fail_next_set_up", what);
    const cudaError_t e = f();
    if (e == cudaSuccess)
        return PGD_OK;
    cudaGetLastError();  // no later call's launch is to find it
    return cuda_fail(e, what);
}

pgd_status tree_runs(DeviceState &st, int D, bool pair, int *runs)
{
    std::atomic<int> &known = st.tree_runs[d_index(D)][pair];
    if ((*runs = known.load(std::memory_order_acquire)) > 0)
        return PGD_OK;
    const pgd_status s =
        set_up("set-up of the tree kernel", [&] { return tree_resident(D, pair, runs); });
    if (!s)
        known.store(*runs, std::memory_order_release);
    return s;
}

pgd_status prefill_ready(DeviceState &st, int D)
{
    std::atomic<bool> &known = st.prefill_ready[d_index(D)];
    if (known.load(std::memory_order_acquire))
        return PGD_OK;
    const pgd_status s = set_up("set-up of the prompt kernel", [&] { return prefill_set_up(D); });
    if (!s)
        known.store(true, std::memory_order_release);
    return s;
}

pgd_status latent_prefill_ready(DeviceState &st, int D)
{
    std::atomic<bool> &known = st.latent_prefill_ready[D == 64 ? 0 : 1];
    if (known.load(std::memory_order_acquire))
        return PGD_OK;
    const pgd_status s =
        set_up("set-up of the latent prompt kernel", [&] { return latent_prefill_set_up(D); });
    if (!s)
        known.store(true, std::memory_order_release);
    return s;
}

pgd_status latent_runs(DeviceState &st, int R, int *runs)
{
    std::atomic<int> &known = st.latent_runs[R == 128 ? 0 : R == 256 ? 1 : 2];
    if ((*runs = known.load(std::memory_order_acquire)) > 0)
        return PGD_OK;
    const pgd_status s =
        set_up("set-up of the latent kernel", [&] { return latent_resident(R, runs); });
    if (!s)
        known.store(*runs, std::memory_order_release);
    return s;
}

// The library's scratch pool on the current device, created on first use
// (a failed creation is retried by the next call that needs it).
pgd_status device_pool(DeviceState &st, cudaMemPool_t *pool)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lock(st.pool_mu);
    if (!st.pool && (e = init_pool(dev, st)) != cudaSuccess) {
        if (st.pool)
            cudaMemPoolDestroy(st.pool);
        st.pool = nullptr;
        return cuda_fail(e, "scratch pool set-up");
    }
    *pool = st.pool;
    return PGD_OK;
}

// ------------------------------------------------------------------ tensor maps
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

pgd_status encode_fn(EncodeTiledFn *fn)
{
    static std::once_flag once;
    static EncodeTiledFn f = nullptr;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                               cudaEnableDefault, &q);
        if (err == cudaSuccess && q == cudaDriverEntryPointSuccess)
            f = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    if (!f)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)",
                    cudaGetErrorString(err));
    *fn = f;
    return PGD_OK;
}

// Geometry of one cache array: NB pages x Hkv heads x BS token rows of D
// contiguous halves, at the given strides (in halves).
struct CacheGeom {
    int NB, Hkv, BS, D;
    long long page_stride, head_stride, token_stride;
    bool operator==(const CacheGeom &o) const
    {
        return NB == o.NB && Hkv == o.Hkv && BS == o.BS && D == o.D &&
               page_stride == o.page_stride && head_stride == o.head_stride &&
               token_stride == o.token_stride;
    }
};

// One cache array viewed as a 5-D tensor, innermost first:
//   64 halves within a 128-byte slab  x  BS token rows (token stride)
//   x D/64 slabs (128 bytes)  x  Hkv heads (head stride)  x  NB pages (page stride),
// so one copy box of 64 x box_rows x D/64 x 1 x 1 brings box_rows whole rows
// of one (page, head) and lands in shared memory as [slab][row][128 B], each
// slab 128-byte swizzled (the span the tensor-core operand loads read
// without bank conflicts), whatever the layout of the array.
pgd_status encode_cache_map(CUtensorMap *map, const void *base, const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    cuuint64_t dims[5] = {64, (cuuint64_t)g.BS, (cuuint64_t)(g.D / 64), (cuuint64_t)g.Hkv,
                          (cuuint64_t)g.NB};
    cuuint64_t strides[4] = {(cuuint64_t)g.token_stride * 2, 128, (cuuint64_t)g.head_stride * 2,
                             (cuuint64_t)g.page_stride * 2};
    cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)(g.D / 64), 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return PGD_OK;
}

// Quantised pages (head-major): the 8-bit codes [NB][Hkv][BS][D] viewed as
// 128 bytes x BS rows x D/128 slabs x Hkv x NB (same box and landing order
// as the fp16 rows), and their (scale, bias) pairs [NB][Hkv][BS][D/64] as
// 32-bit elements: BS*D/64 per (page, head) x Hkv x NB, a box being the
// pairs of box_rows rows.
pgd_status encode_code_map(CUtensorMap *map, const void *base, const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    cuuint64_t dims[5] = {128, (cuuint64_t)g.BS, (cuuint64_t)(g.D / 128), (cuuint64_t)g.Hkv,
                          (cuuint64_t)g.NB};
    cuuint64_t strides[4] = {(cuuint64_t)g.token_stride, 128, (cuuint64_t)g.head_stride,
                             (cuuint64_t)g.page_stride};  // bytes (the cache's strides)
    cuuint32_t box[5] = {128, (cuuint32_t)box_rows, (cuuint32_t)(g.D / 128), 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(base), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (codes) failed (CUresult %d)", (int)r);
    return PGD_OK;
}

// Both quantised code arrays in one map (head-major caches): 128 bytes x rows
// x D/128 slabs x (page, head) blocks (page * Hkv + head) x 2 arrays, the
// array stride being the distance between them (`lo` the lower one); a box
// of 128 x rows x slabs x 1 x 2 lands a page's codes of both arrays as
// [array][slab][row][128 B] (128-byte swizzle).
pgd_status encode_code_pair_map(CUtensorMap *map, const void *lo, long long pair_stride,
                                const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    cuuint64_t dims[5] = {128, (cuuint64_t)g.BS, (cuuint64_t)(g.D / 128),
                          (cuuint64_t)g.NB * g.Hkv, 2};
    cuuint64_t strides[4] = {(cuuint64_t)g.D, 128, (cuuint64_t)g.BS * g.D,
                             (cuuint64_t)pair_stride};
    cuuint32_t box[5] = {128, (cuuint32_t)box_rows, (cuuint32_t)(g.D / 128), 1, 2};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(lo), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (code pair) failed (CUresult %d)", (int)r);
    return PGD_OK;
}

pgd_status encode_meta_map(CUtensorMap *map, const void *base, const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    const int ng = g.D / kQuantGroup;
    cuuint64_t dims[3] = {(cuuint64_t)g.BS * ng, (cuuint64_t)g.Hkv, (cuuint64_t)g.NB};
    cuuint64_t strides[2] = {(cuuint64_t)g.BS * ng * 4, (cuuint64_t)g.Hkv * g.BS * ng * 4};
    cuuint32_t box[3] = {(cuuint32_t)(box_rows * ng), 1, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (scales) failed (CUresult %d)", (int)r);
    return PGD_OK;
}

// (scale, bias) pairs at any strides where a row's pairs are 16 bytes
// (head_dim 256; strides are multiples of a row's pairs, so of 16 bytes):
// 32-bit elements viewed as D/64 pairs x BS rows (token stride) x Hkv heads
// (head stride) x NB pages (page stride), strides in bf16 elements, and
// with pair_stride > 0 both arrays (`lo` the lower one) as a fifth
// dimension; a box of D/64 x box_rows x 1 x 1 (x 2) lands box_rows rows of
// one (page, head) as [array][row][pair], the layout of the head-major
// copies.
pgd_status encode_meta_rows_map(CUtensorMap *map, const void *lo, long long pair_stride,
                                const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    const int ng = g.D / kQuantGroup;
    const cuuint32_t rank = pair_stride > 0 ? 5 : 4;
    cuuint64_t dims[5] = {(cuuint64_t)ng, (cuuint64_t)g.BS, (cuuint64_t)g.Hkv, (cuuint64_t)g.NB, 2};
    cuuint64_t strides[4] = {(cuuint64_t)g.token_stride * 2, (cuuint64_t)g.head_stride * 2,
                             (cuuint64_t)g.page_stride * 2, (cuuint64_t)pair_stride};
    cuuint32_t box[5] = {(cuuint32_t)ng, (cuuint32_t)box_rows, 1, 1, 2};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, rank, const_cast<void *>(lo), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (strided scales) failed (CUresult %d)",
                    (int)r);
    return PGD_OK;
}

// Both quantised code arrays in one map where a row's D codes and the KV
// heads of a token are adjacent (head stride D bytes, e.g. token-major
// caches): 128 bytes x rows (token stride) x (head, slab) pairs (head * D/128
// + slab, 128 bytes apart) x NB pages (page stride) x 2 arrays; a box of 128
// x rows x D/128 x 1 x 2 lands a page's codes of both arrays as
// [array][slab][row][128 B] (128-byte swizzle), like the head-major pair map.
pgd_status encode_code_pair_rows_map(CUtensorMap *map, const void *lo, long long pair_stride,
                                     const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    cuuint64_t dims[5] = {128, (cuuint64_t)g.BS, (cuuint64_t)g.Hkv * (g.D / 128),
                          (cuuint64_t)g.NB, 2};
    cuuint64_t strides[4] = {(cuuint64_t)g.token_stride, 128, (cuuint64_t)g.page_stride,
                             (cuuint64_t)pair_stride};  // bytes
    cuuint32_t box[5] = {128, (cuuint32_t)box_rows, (cuuint32_t)(g.D / 128), 1, 2};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(lo), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (code rows pair) failed (CUresult %d)",
                    (int)r);
    return PGD_OK;
}

// Both (scale, bias) pair arrays in one map (head-major): the pairs of a
// (page, head) block x blocks (page * Hkv + head) x 2 arrays, the array
// stride being the distance between them (`lo` the lower one); a box of
// box_rows rows x 1 x 2 lands a piece's pairs of both arrays side by side.
pgd_status encode_meta_pair_map(CUtensorMap *map, const void *lo, long long pair_stride,
                                const CacheGeom &g, int box_rows)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    const int ng = g.D / kQuantGroup;
    cuuint64_t dims[3] = {(cuuint64_t)g.BS * ng, (cuuint64_t)g.NB * g.Hkv, 2};
    cuuint64_t strides[2] = {(cuuint64_t)g.BS * ng * 4, (cuuint64_t)pair_stride};
    cuuint32_t box[3] = {(cuuint32_t)(box_rows * ng), 1, 2};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(lo), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (scale pair) failed (CUresult %d)",
                    (int)r);
    return PGD_OK;
}

// The cache viewed for the multi-token kernel, innermost first:
//   64 halves x 8 token rows (token stride) x D/64 slabs (128 bytes)
//   x BS/8 row groups (8 token strides) x blocks (u halves),
// where u = gcd(page stride, head stride) and (page b, head g) is block
// b * page_stride/u + g * head_stride/u.  A box of 64 x 8 x D/64 x groups x 1
// lands a page's rows as [group][slab][row][128 B] (128-byte swizzle): the
// layout the tensor cores read K (K-major) and V (MN-major) in.
long long gcd_ll(long long a, long long b)
{
    while (b) {
        const long long t = a % b;
        a = b;
        b = t;
    }
    return a;
}

pgd_status group_blocks(const CacheGeom &g, long long *u, long long *blocks)
{
    *u = gcd_ll(g.page_stride, g.head_stride);
    *blocks = (g.NB - 1) * (g.page_stride / *u) + (g.Hkv - 1) * (g.head_stride / *u) + 1;
    if (*blocks >= (1ll << 31))
        return fail(PGD_ERR_UNSUPPORTED,
                    "cache strides (%lld, %lld) give %lld page/head blocks (limit 2^31)",
                    g.page_stride, g.head_stride, *blocks);
    return PGD_OK;
}

pgd_status encode_cache_map_groups(CUtensorMap *map, const void *base, const CacheGeom &g,
                                   int box_groups, int box_slabs = 0)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    long long u, blocks;
    if ((st = group_blocks(g, &u, &blocks)))
        return st;
    cuuint64_t dims[5] = {64, 8, (cuuint64_t)(g.D / 64), (cuuint64_t)(g.BS / 8), (cuuint64_t)blocks};
    cuuint64_t strides[4] = {(cuuint64_t)g.token_stride * 2, 128, (cuuint64_t)g.token_stride * 16,
                             (cuuint64_t)u * 2};
    cuuint32_t box[5] = {64, 8, (cuuint32_t)(box_slabs ? box_slabs : g.D / 64),
                         (cuuint32_t)box_groups, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (page groups) failed (CUresult %d)",
                    (int)r);
    return PGD_OK;
}

// ------------------------------------------------------------------ claim counters
// The partition kernel hands out work units with a 4-byte counter that must
// read 0 at launch; the reduce kernel zeroes it at the end of every call.
// The library keeps one counter per (device, stream) it has run on: calls on
// one stream are serialised and can reuse it, calls on different streams
// never share one.  A counter whose call failed to launch is zeroed in
// stream order before its next use.  The counters are allocated by the
// first call on a device that needs one (again after pgd_release).
constexpr int kCounterSlots = 1024;
constexpr int kCounterStride = 32;  // unsigned words: 128 bytes apart

struct CounterPool {
    std::mutex mu;                 // guards everything below
    unsigned *base = nullptr;
    std::unordered_map<uintptr_t, int> slot_of;
    std::vector<char> dirty;
};

CounterPool g_counters[kMaxDevices];

// Allocates and zeroes the counters (cp.mu held); leaves cp.base null on failure.
cudaError_t init_counters(CounterPool &cp)
{
    unsigned *base = nullptr;
    const size_t bytes = sizeof(unsigned) * kCounterSlots * kCounterStride;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&base), bytes);
    if (e != cudaSuccess)
        return e;
    if ((e = cudaMemset(base, 0, bytes)) != cudaSuccess ||
        (e = cudaDeviceSynchronize()) != cudaSuccess) {
        cudaFree(base);
        return e;
    }
    cp.base = base;
    cp.slot_of.clear();
    cp.dirty.assign(kCounterSlots, 0);
    return cudaSuccess;
}

// The counter of `stream` on the current device (null when all slots are
// taken); *reset tells the caller to zero it in stream order first.
pgd_status stream_counter(cudaStream_t stream, unsigned **counter, int *slot, bool *reset)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(PGD_ERR_UNSUPPORTED, "device ordinal %d beyond %d", dev, kMaxDevices);
    CounterPool &cp = g_counters[dev];
    std::lock_guard<std::mutex> lock(cp.mu);
    if (!cp.base && (e = init_counters(cp)) != cudaSuccess)
        return cuda_fail(e, "claim-counter set-up");
    const uintptr_t key = reinterpret_cast<uintptr_t>(stream);
    auto it = cp.slot_of.find(key);
    int i;
    if (it != cp.slot_of.end()) {
        i = it->second;
    } else if ((int)cp.slot_of.size() < kCounterSlots) {
        i = (int)cp.slot_of.size();
        cp.slot_of.emplace(key, i);
    } else {
        *counter = nullptr;
        *slot = -1;
        *reset = false;
        return PGD_OK;
    }
    *counter = cp.base + (size_t)i * kCounterStride;
    *slot = i;
    *reset = cp.dirty[i] != 0;
    cp.dirty[i] = 0;
    return PGD_OK;
}

void mark_counter_dirty(int slot)
{
    int dev = 0;
    if (slot < 0 || cudaGetDevice(&dev) != cudaSuccess)
        return;
    std::lock_guard<std::mutex> lock(g_counters[dev].mu);
    if (slot < (int)g_counters[dev].dirty.size())
        g_counters[dev].dirty[slot] = 1;
}

// Descriptors of the last few (k_cache, v_cache) pairs used by this thread:
// encoding them is the largest host cost of a call, and a decode loop calls
// with the same caches every step.
struct MapCacheEntry {
    const void *k, *v;
    CacheGeom geom;
    int box, kind, dev;
    alignas(64) CUtensorMap tk;
    alignas(64) CUtensorMap tv;
};
constexpr int kMapCache = 8;
thread_local MapCacheEntry t_maps[kMapCache];
thread_local int t_maps_used = 0, t_maps_next = 0;

// kind 0: the decode view (box = rows per copy); kind 1: the page-group view
// (box = 8-row groups per copy); kind 2: quantised codes, kind 3: their
// (scale, bias) pairs (box = rows per copy); kind 4: both code arrays in one
// map, kind 5: both pair arrays in one map (*tk = *tv, based at the lower
// array).
pgd_status cache_maps(const void *k, const void *v, const CacheGeom &geom, int box, int kind,
                      const CUtensorMap **tk, const CUtensorMap **tv)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    for (int i = 0; i < t_maps_used; ++i) {
        MapCacheEntry &c = t_maps[i];
        if (c.k == k && c.v == v && c.geom == geom && c.box == box && c.kind == kind &&
            c.dev == dev) {
            *tk = &c.tk;
            *tv = &c.tv;
            return PGD_OK;
        }
    }
    MapCacheEntry &c = t_maps[t_maps_next];
    pgd_status st;
    // kinds: 0 fp16 rows, 1 fp16 8-row groups, 2 codes, 3 head-major pairs,
    // 6 pairs of 16-byte rows at any strides; both arrays in one map: 4
    // codes (head-major), 5 head-major pairs, 7 pairs of 16-byte rows, 8
    // codes with adjacent heads; 9 fp16 8-row groups, K and V in pieces of their own
    if (kind == 4 || kind == 5 || kind == 7 || kind == 8) {
        const uintptr_t ka = reinterpret_cast<uintptr_t>(k), va = reinterpret_cast<uintptr_t>(v);
        const long long stride = (long long)(ka < va ? va - ka : ka - va);
        const void *lo = ka < va ? k : v;
        if ((st = kind == 4   ? encode_code_pair_map(&c.tk, lo, stride, geom, box)
                  : kind == 5 ? encode_meta_pair_map(&c.tk, lo, stride, geom, box)
                  : kind == 7 ? encode_meta_rows_map(&c.tk, lo, stride, geom, box)
                              : encode_code_pair_rows_map(&c.tk, lo, stride, geom, box))) {
            c.k = c.v = nullptr;
            return st;
        }
        c.tv = c.tk;
    }
    auto enc = [&](CUtensorMap *m, const void *base) -> pgd_status {
        switch (kind) {
        case 0:
            return encode_cache_map(m, base, geom, box);
        case 1:
            return encode_cache_map_groups(m, base, geom, box);
        case 2:
            return encode_code_map(m, base, geom, box);
        case 6:
            return encode_meta_rows_map(m, base, 0, geom, box);
        case 9:  // (slabs of a K and a V copy, 8-row groups of a K and a V copy)
            return m == &c.tk
                       ? encode_cache_map_groups(m, base, geom, (box >> 8) & 255, box & 15)
                       : encode_cache_map_groups(m, base, geom, box >> 16, (box >> 4) & 15);
        default:
            return encode_meta_map(m, base, geom, box);
        }
    };
    if (kind != 4 && kind != 5 && kind != 7 && kind != 8 &&
        ((st = enc(&c.tk, k)) || (st = enc(&c.tv, v)))) {
        c.k = c.v = nullptr;
        return st;
    }
    c.k = k;
    c.v = v;
    c.geom = geom;
    c.box = box;
    c.kind = kind;
    c.dev = dev;
    t_maps_next = (t_maps_next + 1) % kMapCache;
    if (t_maps_used < kMapCache)
        ++t_maps_used;
    *tk = &c.tk;
    *tv = &c.tv;
    return PGD_OK;
}

// ------------------------------------------------------------------ validation & plan
struct Plan {
    int P;             // partition size
    int NPmax;         // partitions of the longest possible sequence
    size_t ws_bytes;   // scratch bytes (0 when NPmax == 1)
    size_t off_l, off_o;
    int grid;          // partition-kernel CTAs
    int reduce_blocks;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Scratch of the partition partials: m [S][Hq][NPmax], l [S][Hq][NPmax] and
// o [S][Hq][NPmax][D] fp32, each region 256-byte aligned; none when no
// sequence can span two partitions (NPmax == 1).
size_t partials_bytes(int S, int Hq, int D, int NPmax, size_t *off_l, size_t *off_o)
{
    if (NPmax <= 1) {
        *off_l = *off_o = 0;
        return 0;
    }
    const size_t rows = (size_t)S * Hq * NPmax;
    *off_l = align256(rows * 4);
    *off_o = *off_l + align256(rows * 4);
    return *off_o + align256(rows * D * 4);
}

pgd_status check_sizes(int S, int Hq, int Hkv, int D, int BS, int P, int MB)
{
    if (S < 0)
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d < 0", S);
    if (Hq <= 0 || Hkv <= 0)
        return fail(PGD_ERR_INVALID_ARG, "head counts must be positive (%d, %d)", Hq, Hkv);
    if (Hq % Hkv != 0)
        return fail(PGD_ERR_INVALID_ARG, "num_q_heads %d not a multiple of num_kv_heads %d", Hq,
                    Hkv);
    if (Hq / Hkv > kMaxGroup)
        return fail(PGD_ERR_UNSUPPORTED, "GQA group of %d query heads exceeds %d", Hq / Hkv,
                    kMaxGroup);
    if (!supported_head_dim(D))
        return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", D);
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (P != 0 && P != kPartitionSmall && P != kPartitionLarge)
        return fail(PGD_ERR_INVALID_ARG, "partition_size %d not in {0, 256, 512}", P);
    if (MB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "max_blocks_per_seq %d <= 0", MB);
    if ((long long)MB * BS > (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "length bound %lld above 2^30", (long long)MB * BS);
    return PGD_OK;
}

// Partition scheduler (the pages' "Dispatch layer": try 512 first, then
// 256, counting only full partitions, against a work budget scaled by the
// GPU's core count).  Here the budget is four units per resident CTA of the
// persistent kernel, and full partitions are counted at the length bound
// MB*BS because the lengths themselves stay on the device.
int choose_partition(int S, int Hkv, int maxlen, int num_sms, int ctas_per_sm)
{
    const long long target = 4ll * num_sms * (ctas_per_sm > 0 ? ctas_per_sm : 1);
    const long long full512 = (long long)S * Hkv * (maxlen / kPartitionLarge);
    return full512 >= target ? kPartitionLarge : kPartitionSmall;
}

// kind: 0 fp16 pages, 1 quantised pages, 2 several query tokens per sequence
// (the MQ form, whose partials are kept per query row: prow rows instead of S)
pgd_status make_plan(int S, int Hq, int Hkv, int D, int BS, int P, int MB, Plan *plan,
                     int kind = 0, int prow = -1)
{
    pgd_status st = check_sizes(S, Hq, Hkv, D, BS, P, MB);
    if (st)
        return st;
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    if (prow < 0)
        prow = S;
    const int ctas = ds->ctas[kind][d_index(D)][bs_index(BS)];
    if (ctas < 1)
        return fail(PGD_ERR_UNSUPPORTED, "partition kernel does not fit on an SM");
    const int maxlen = MB * BS;
    if (P == 0)
        P = choose_partition(S, Hkv, maxlen, ds->num_sms, ctas);
    plan->P = P;
    plan->NPmax = (maxlen + P - 1) / P;
    // the kernels count pipeline stages in 32-bit integers
    const long long stage_bound =
        (long long)S * Hkv * ((long long)maxlen / 32 + plan->NPmax);
    if (stage_bound >= (1ll << 31))
        return fail(PGD_ERR_UNSUPPORTED, "batch of %d sequences x %d KV heads x %d tokens too large",
                    S, Hkv, maxlen);
    plan->ws_bytes = partials_bytes(prow, Hq, D, plan->NPmax, &plan->off_l, &plan->off_o);
    if (plan->ws_bytes > kMaxWorkspaceBytes)
        return fail(PGD_ERR_WORKSPACE,
                    "partials need %zu bytes, above the %zu-byte cap (lower the length bound "
                    "or the batch)",
                    plan->ws_bytes, kMaxWorkspaceBytes);
    const long long units = (long long)S * Hkv * plan->NPmax;
    const long long slots = (long long)ds->num_sms * ctas;
    plan->grid = (int)(units < slots ? (units > 0 ? units : 1) : slots);
    plan->reduce_blocks = (int)((long long)prow * Hq);
    if (plan->reduce_blocks < 1)
        plan->reduce_blocks = 1;
    return PGD_OK;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Strides (in halves) of the default layout [NB][Hkv][BS][D].
struct Strides {
    long long page, head, token;
};
Strides head_major(int Hkv, int BS, int D)
{
    return {(long long)Hkv * BS * D, (long long)BS * D, (long long)D};
}

pgd_status check_strides(const Strides &x, int D)
{
    const long long limit = 1ll << 39;  // the tensor copies take strides below 2^40 bytes
    const long long v[3] = {x.page, x.head, x.token};
    for (long long e : v)
        if (e <= 0 || e % 8 != 0 || e >= limit)
            return fail(PGD_ERR_INVALID_ARG,
                        "cache strides (%lld, %lld, %lld) must be positive multiples of 8 "
                        "halves below 2^39",
                        x.page, x.head, x.token);
    if (x.token < D)
        return fail(PGD_ERR_INVALID_ARG, "token stride %lld below head_dim %d", x.token, D);
    return PGD_OK;
}

// Several query tokens per sequence on the decode kernel (its MQ form):
// the query rows of each sequence (cu_q), their total and bound.
struct MultiQuery {
    const int32_t *cu_q;
    int total_q, max_q;
};

// A claim counter the caller provides (paged_gqa_decode_noalloc's, in its
// static array) with its flag: set when a call failed after its partition
// kernel may have moved the counter, so the next call zeroes it first.
struct GivenCounter {
    unsigned *word;
    std::atomic<bool> *dirty;
};

// q8: the caches hold 8-bit codes (head-major) and k_meta / v_meta their
// (scale, bias) pairs.
pgd_status run(float *out, const uint16_t *q, const void *k_cache, const void *v_cache,
               const int32_t *block_tables, const int32_t *seq_lens, float scale, int S, int Hq,
               int Hkv, int D, int BS, int P, int MB, int NB, const Strides &kv_strides,
               void *workspace, size_t ws_bytes, bool own_workspace, int32_t *page_trace,
               void *stream_v, const GivenCounter *given = nullptr,
               const uint16_t *k_new = nullptr,
               const uint16_t *v_new = nullptr, bool q8 = false, const void *k_meta = nullptr,
               const void *v_meta = nullptr, const Strides *meta_strides = nullptr,
               const MultiQuery *mq = nullptr)
{
    if (q8 && D % 128 != 0)
        return fail(PGD_ERR_UNSUPPORTED, "quantised pages need head_dim 128 or 256, not %d", D);
    const int kind = mq ? 2 : q8 ? 1 : 0;
    const int prow = mq ? mq->total_q : S;
    if (S == 0) {  // nothing to read or write: only the sizes are checked
        Plan plan;
        pgd_status st0 = make_plan(S, Hq, Hkv, D, BS, P, MB, &plan, kind, prow);
        if (st0)
            return st0;
        t_last_partition = plan.P;
        t_last_error.clear();
        return PGD_OK;
    }
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens ||
        (q8 && (!k_meta || !v_meta)))
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (q8 && (!aligned(k_meta, 16) || !aligned(v_meta, 16)))
        return fail(PGD_ERR_INVALID_ARG, "k_meta and v_meta must be 16-byte aligned");
    if (!std::isfinite(scale))
        return fail(PGD_ERR_INVALID_ARG, "scale is not finite");
    if (NB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_blocks %d <= 0", NB);
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return fail(PGD_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    if (!aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        (page_trace && !aligned(page_trace, 4)))
        return fail(PGD_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    pgd_status st = check_sizes(S, Hq, Hkv, D, BS, P, MB);
    if (st)
        return st;
    if ((st = check_strides(kv_strides, D)))
        return st;
    // quantised pages: code strides in bytes (multiples of 16, the tensor
    // copies' rule), the pairs' strides in bf16 elements (multiples of a
    // row's pairs, so each row's pairs are one aligned 8- or 16-byte copy)
    const int NM = (D / kQuantGroup) * 2;
    const Strides ms = meta_strides ? *meta_strides
                                    : Strides{(long long)Hkv * BS * NM, (long long)BS * NM, NM};
    // q8_rows: the pairs are not head-major; 1: the kernel copies them row by
    // row, 2: by a tensor copy of 16-byte rows (head_dim 256: the strides,
    // multiples of a row's pairs, are multiples of 16 bytes)
    int q8_rows = 0;
    bool codes_head_major = true;
    if (q8) {
        if (kv_strides.page % 16 || kv_strides.head % 16 || kv_strides.token % 16)
            return fail(PGD_ERR_INVALID_ARG,
                        "code strides (%lld, %lld, %lld) must be multiples of 16 bytes",
                        kv_strides.page, kv_strides.head, kv_strides.token);
        const long long mv[3] = {ms.page, ms.head, ms.token};
        for (long long x : mv)
            if (x <= 0 || x % NM != 0 || x >= (1ll << 38))
                return fail(PGD_ERR_INVALID_ARG,
                            "pair strides (%lld, %lld, %lld) must be positive multiples of %d "
                            "elements below 2^38",
                            ms.page, ms.head, ms.token, NM);
        const Strides hm = head_major(Hkv, BS, D);
        codes_head_major = kv_strides.page == hm.page && kv_strides.head == hm.head &&
                           kv_strides.token == hm.token;
        const bool rows = !codes_head_major || ms.page != (long long)Hkv * BS * NM ||
                          ms.head != (long long)BS * NM || ms.token != NM;
        q8_rows = !rows ? 0 : (NM * 2 == 16 ? 2 : 1);
    }
    if (!own_workspace && workspace && !aligned(workspace, 256))
        return fail(PGD_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (mq && (!mq->cu_q || D > 128 || mq->total_q < 0 || mq->max_q < 1 ||
               (long long)mq->max_q * (Hq / Hkv) > kMaxCols || q8 || k_new || page_trace))
        return fail(PGD_ERR_UNSUPPORTED, "several query tokens on the decode kernel: head_dim "
                                         "<= 128, max_q_len * group <= %d, fp16 pages only",
                    kMaxCols);
    Plan plan;
    if ((st = make_plan(S, Hq, Hkv, D, BS, P, MB, &plan, kind, prow)))
        return st;
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    t_last_partition = plan.P;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    cudaError_t e;

    char *ws = static_cast<char *>(workspace);
    if (plan.ws_bytes) {
        if (own_workspace) {
            cudaMemPool_t pool;
            if ((st = device_pool(*ds, &pool)))
                return st;
            if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), plan.ws_bytes, pool,
                                             stream)) != cudaSuccess)
                return cuda_fail(e, "scratch allocation");
        } else {
            if (!ws || ws_bytes < plan.ws_bytes)
                return fail(PGD_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed",
                            ws ? ws_bytes : (size_t)0, plan.ws_bytes);
        }
    }

    const int stage_t = q8 ? (D == 128 ? Shape<128>::T8 : Shape<256>::T8) : stage_tokens(D);
    const int box = BS < stage_t ? BS : stage_t;
    const CacheGeom geom = {NB, Hkv, BS, D, kv_strides.page, kv_strides.head, kv_strides.token};
    const CUtensorMap *tk = nullptr, *tv = nullptr, *tkm = nullptr, *tvm = nullptr;
    // quantised pages with page pieces of up to 4 KB (the kernel then keeps a
    // piece's K and V codes side by side): one copy per page for both code
    // arrays when their distance fits a tensor-map stride (a multiple of 16
    // bytes below 2^40) and the (page, head) blocks fit a coordinate
    const uintptr_t k_at = reinterpret_cast<uintptr_t>(k_cache),
                    v_at = reinterpret_cast<uintptr_t>(v_cache);
    const long long code_gap = !q8 ? 0
                               : v_at >= k_at ? (long long)(v_at - k_at)
                                              : -(long long)(k_at - v_at);
    const long long gap_abs = code_gap < 0 ? -code_gap : code_gap;
    // (1: head-major codes; 2: a token's heads adjacent, head stride D bytes,
    // as token-major caches have them)
    const bool gap_ok = gap_abs > 0 && gap_abs % 16 == 0 && gap_abs < (1ll << 40);
    const int q8_pair = !q8 || box * D > 4096 || !gap_ok ? 0
                        : codes_head_major                ? ((long long)NB * Hkv < (1ll << 31) ? 1 : 0)
                        : kv_strides.head == D            ? 2
                                                          : 0;
    // One copy for both pair arrays under the same conditions, where a
    // piece's pairs fill whole 128-byte runs (the kernel then keeps a piece's
    // K and V pairs side by side): head-major pairs, or 16-byte rows at any
    // strides (q8_rows 2); the kernel copies other pairs row by row
    const uintptr_t km_at = reinterpret_cast<uintptr_t>(k_meta),
                    vm_at = reinterpret_cast<uintptr_t>(v_meta);
    const long long meta_gap = km_at < vm_at ? (long long)(vm_at - km_at) : (long long)(km_at - vm_at);
    const int q8_meta_pair = q8 && q8_rows != 1 && (box * (D / kQuantGroup) * 4) % 128 == 0 &&
                                     meta_gap > 0 && meta_gap % 16 == 0 && meta_gap < (1ll << 40) &&
                                     (q8_rows || (long long)NB * Hkv < (1ll << 31))
                                 ? (km_at < vm_at ? 1 : 2)
                                 : 0;
    const CacheGeom meta_geom = {NB, Hkv, BS, D, ms.page, ms.head, ms.token};
    const int code_kind = !q8 ? 0 : q8_pair == 1 ? 4 : q8_pair == 2 ? 8 : 2;
    if ((st = cache_maps(k_cache, v_cache, geom, box, code_kind, &tk, &tv)) ||
        (q8 && !q8_rows &&
         (st = cache_maps(k_meta, v_meta, geom, box, q8_meta_pair ? 5 : 3, &tkm, &tvm))) ||
        (q8 && q8_rows == 2 &&
         (st = cache_maps(k_meta, v_meta, meta_geom, box, q8_meta_pair ? 7 : 6, &tkm, &tvm)))) {
        if (own_workspace && ws)
            cudaFreeAsync(ws, stream);
        return st;
    }
    const KVMaps maps = {tk, tv, q8 && q8_rows != 1 ? tkm : tk, q8 && q8_rows != 1 ? tvm : tv};

    // claim counter: given (static scratch), this stream's, or a per-call one
    auto release_ws = [&] {
        if (own_workspace && ws)
            cudaFreeAsync(ws, stream);
    };
    unsigned *counter = given ? given->word : nullptr;
    int slot = -1;
    unsigned *own_counter = nullptr;
    if (given) {
        // an earlier call on it failed after its partition kernel may have
        // started: zero it in stream order first (allocates nothing)
        if (given->dirty->load()) {
            if ((e = cudaMemsetAsync(counter, 0, sizeof(unsigned), stream)) != cudaSuccess) {
                release_ws();
                return cuda_fail(e, "counter reset");
            }
            given->dirty->store(false);
        }
    } else {
        bool reset = false;
        if ((st = stream_counter(stream, &counter, &slot, &reset))) {
            release_ws();
            return st;
        }
        if (!counter) {  // every slot taken: a zeroed counter for this call only
            cudaMemPool_t pool;
            if ((st = device_pool(*ds, &pool))) {
                release_ws();
                return st;
            }
            if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&own_counter), 256, pool,
                                             stream)) != cudaSuccess) {
                release_ws();
                return cuda_fail(e, "counter allocation");
            }
            counter = own_counter;
            reset = true;
        }
        if (reset && (e = cudaMemsetAsync(counter, 0, sizeof(unsigned), stream)) != cudaSuccess) {
            if (slot >= 0)
                mark_counter_dirty(slot);
            if (own_counter)
                cudaFreeAsync(own_counter, stream);
            release_ws();
            return cuda_fail(e, "counter reset");
        }
    }

    DecodeParams p = {};
    p.out = out;
    p.q = reinterpret_cast<const __half *>(q);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    const bool partials = plan.NPmax > 1;
    p.ws_m = partials ? reinterpret_cast<float *>(ws) : nullptr;
    p.ws_l = partials ? reinterpret_cast<float *>(ws + plan.off_l) : nullptr;
    p.ws_o = partials ? reinterpret_cast<float *>(ws + plan.off_o) : nullptr;
    p.page_trace = page_trace;
    p.counter = counter;
    p.k_new = reinterpret_cast<const __half *>(k_new);
    p.v_new = reinterpret_cast<const __half *>(v_new);
    p.k_cache = reinterpret_cast<__half *>(const_cast<void *>(k_cache));
    p.v_cache = reinterpret_cast<__half *>(const_cast<void *>(v_cache));
    p.k_meta = q8 ? static_cast<uint16_t *>(const_cast<void *>(k_meta)) : nullptr;
    p.v_meta = q8 ? static_cast<uint16_t *>(const_cast<void *>(v_meta)) : nullptr;
    p.q8_pair = q8_pair;
    p.q8_meta_pair = q8_meta_pair;
    p.q8_rows = q8_rows;
    p.meta_page_stride = ms.page;
    p.meta_head_stride = ms.head;
    p.meta_token_stride = ms.token;
    p.q8_koff = q8_pair && code_gap < 0 ? box * D : 0;  // the lower array lands first
    p.q8_voff = q8_pair && code_gap < 0 ? 0 : box * D;   // (used for pieces of <= 4 KB)
    p.kv_page_stride = kv_strides.page;
    p.kv_head_stride = kv_strides.head;
    p.kv_token_stride = kv_strides.token;
    p.err = ds->err_word;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e) folded into the scale
    p.S = S;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.P = plan.P;
    p.logP = plan.P == kPartitionLarge ? 9 : 8;
    p.MB = MB;
    p.NB = NB;
    p.NPmax = plan.NPmax;
    p.wait_budget_ns = kWaitBudgetNs;
    p.stall_flag = t_stall_flag;  // one call only
    t_stall_flag = nullptr;
    p.cu_q = mq ? mq->cu_q : nullptr;
    p.max_q = mq ? mq->max_q : 0;
    p.total_q = mq ? mq->total_q : 0;

    LaunchConfig lc;
    lc.grid = plan.grid;
    lc.reduce_blocks = plan.reduce_blocks;
    lc.stream = stream;
    lc.ev_before = t_ev_before;
    lc.ev_after = t_ev_after;
    lc.skip_reduce = t_skip_reduce;  // one call only
    t_skip_reduce = false;
    const bool trace = page_trace != nullptr;
    e = D == 64    ? launch_decode_d64(BS, trace, q8, maps, p, lc)
        : D == 128 ? launch_decode_d128(BS, trace, q8, maps, p, lc)
                   : launch_decode_d256(BS, trace, q8, maps, p, lc);
    if (own_workspace && ws) {
        cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (own_counter) {
        cudaError_t e2 = cudaFreeAsync(own_counter, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (e != cudaSuccess || lc.skip_reduce) {
        // the reduce may not have zeroed the counter
        mark_counter_dirty(slot);
        if (given)
            given->dirty->store(true);
        if (e != cudaSuccess)
            return cuda_fail(e, "kernel launch");
        return fail(PGD_ERR_CUDA, "reduce launch withheld by pgd_test_fail_next_reduce (the "
                                  "call's output is undefined)");
    }
    t_last_error.clear();
    return PGD_OK;
}

// ------------------------------------------------------------------ several query tokens
// q [total_q][Hq][D] viewed as a 4-D tensor, innermost first: 64 halves x Hq
// heads (D*2 bytes apart) x total_q tokens (Hq*D*2 apart) x D/64 slabs (128
// bytes apart); a box of 64 x G x TQ x 1 is one slab of a 128-row tile (TQ
// tokens x the G heads of a group), landing row-major as [token][head][128 B].
pgd_status encode_q_map(CUtensorMap *map, const void *q, int total_q, int Hq, int D, int G,
                        int TQ)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    cuuint64_t dims[4] = {64, (cuuint64_t)Hq, (cuuint64_t)total_q, (cuuint64_t)(D / 64)};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2, 128};
    cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)TQ, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(q), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (queries) failed (CUresult %d)", (int)r);
    return PGD_OK;
}

struct VarlenPlan {
    int G, TQ, QT, QP, PK, NP, NT;
    bool mq;       // few query rows per (sequence, KV head): the decode kernel's MQ form
    bool pairs;    // two query tiles per CTA
    bool ordered;  // units sorted longest first on the device (more than one wave)
    long long grid;
    size_t ws_bytes, off_l, off_o, off_order;
};

int varlen_tokens_per_stage(int D) { return D == 64 ? VShape<64>::NT : D == 128 ? VShape<128>::NT : VShape<256>::NT; }

// Work split of the multi-token path: 128-row tiles of (query token, head)
// per (sequence, KV head); the KV range is cut into partitions of PK tokens
// only when the tiles alone (counted at max_q_len) would not give every SM
// two units.  Scratch (partials) only when some row spans two partitions.
pgd_status make_varlen_plan(int S, int total_q, int max_q, int Hq, int Hkv, int D, int BS,
                            int MB, int kv_partition, VarlenPlan *vp)
{
    pgd_status st;
    if (S < 0)
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d < 0", S);
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return fail(PGD_ERR_INVALID_ARG, "head counts %d / %d", Hq, Hkv);
    if (Hq / Hkv > 128)
        return fail(PGD_ERR_UNSUPPORTED, "GQA group of %d query heads exceeds 128", Hq / Hkv);
    if (!supported_head_dim(D))
        return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", D);
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (MB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "max_blocks_per_seq %d <= 0", MB);
    if ((long long)MB * BS > (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "length bound %lld above 2^30", (long long)MB * BS);
    if (total_q < 0 || max_q < 0 || (total_q > 0 && max_q < 1))
        return fail(PGD_ERR_INVALID_ARG, "total_q %d / max_q_len %d", total_q, max_q);
    vp->NT = varlen_tokens_per_stage(D);
    if (kv_partition < 0 || (kv_partition > 0 && kv_partition % vp->NT != 0))
        return fail(PGD_ERR_INVALID_ARG, "kv_partition %d: 0 or a positive multiple of %d",
                    kv_partition, vp->NT);
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    vp->G = Hq / Hkv;
    // Calls with at most kMaxCols (query token, head) rows per (sequence, KV
    // head) — decode steps, the verification step of speculative decoding —
    // read each K/V byte for only a few rows: an HBM-bound scan, which the
    // decode kernel's MQ form does (one n8 column tile of mma.sync, partitions of
    // 256 / 512 tokens chosen as for the decode, partials per query row).
    vp->mq = D <= 128 && vp->G <= kMaxGroup && max_q >= 1 &&
             (long long)max_q * vp->G <= kMaxCols &&
             (kv_partition == 0 || kv_partition == kPartitionSmall ||
              kv_partition == kPartitionLarge);
    if (vp->mq) {
        Plan plan;
        if ((st = make_plan(S, Hq, Hkv, D, BS, kv_partition, MB, &plan, 2, total_q)))
            return st;
        vp->TQ = vp->QT = vp->QP = 1;
        vp->PK = plan.P;
        vp->NP = plan.NPmax;
        vp->pairs = vp->ordered = false;
        vp->grid = plan.grid;
        vp->ws_bytes = plan.ws_bytes;
        vp->off_l = plan.off_l;
        vp->off_o = plan.off_o;
        vp->off_order = 0;
        return PGD_OK;
    }
    vp->TQ = 128 / vp->G;
    vp->QT = (max_q + vp->TQ - 1) / vp->TQ;
    // two query tiles per CTA where they fit in tensor memory and the
    // sequences can have more than one tile of query rows
    vp->pairs = (D == 64 ? varlen_pairs<64>() : D == 128 ? varlen_pairs<128>() : varlen_pairs<256>()) &&
                vp->QT >= 2;
    vp->QP = vp->pairs ? (vp->QT + 1) / 2 : vp->QT;  // query-tile units per (sequence, KV head)
    const long long maxlen = (long long)MB * BS;
    const long long whole = (maxlen + vp->NT - 1) / vp->NT * vp->NT;
    const long long tiles = (long long)S * Hkv * vp->QP;
    const size_t rows = (size_t)total_q * Hq;
    auto ws_for = [&](int NP) -> size_t {
        if (NP <= 1)
            return 0;
        return align256(rows * NP * 4) * 2 + align256(rows * NP * D * 4);
    };
    long long PK;
    if (kv_partition > 0) {
        PK = kv_partition;
    } else {
        const long long target = 2ll * ds->num_sms;
        PK = whole;
        if (tiles > 0 && tiles < target) {
            const long long want = (target + tiles - 1) / tiles;
            PK = std::max<long long>(4ll * vp->NT, ((maxlen + want - 1) / want + vp->NT - 1) /
                                                       vp->NT * vp->NT);
        }
        while (PK < whole && ws_for((int)((maxlen + PK - 1) / PK)) > kMaxWorkspaceBytes)
            PK *= 2;
    }
    if (PK > whole)
        PK = whole > 0 ? whole : vp->NT;
    vp->PK = (int)PK;
    vp->NP = (int)((maxlen + PK - 1) / PK);
    if (vp->NP < 1)
        vp->NP = 1;
    vp->off_l = align256(rows * vp->NP * 4);
    vp->off_o = 2 * vp->off_l;
    vp->grid = tiles * vp->NP;
    if (vp->grid >= (1ll << 31))
        return fail(PGD_ERR_UNSUPPORTED, "%lld work units", vp->grid);
    // pairs of query tiles (compute-bound) and more units than SMs: a unit
    // order (longest first) after the partials.  One-tile calls (decode and
    // speculative verification: HBM-bound, units of similar cost per byte)
    // measured slower with the extra sorting launch.
    vp->ordered = vp->pairs && vp->grid > ds->num_sms;
    vp->off_order = ws_for(vp->NP);
    vp->ws_bytes = vp->off_order + (vp->ordered ? align256((size_t)vp->grid * 4) : 0);
    if (vp->ws_bytes > kMaxWorkspaceBytes)
        return fail(PGD_ERR_WORKSPACE, "scratch of %zu bytes needed, above the %zu-byte cap",
                    vp->ws_bytes, kMaxWorkspaceBytes);
    return PGD_OK;
}

pgd_status run_varlen(float *out, const uint16_t *q, const int32_t *cu_q, const uint16_t *k_cache,
                      const uint16_t *v_cache, const int32_t *block_tables,
                      const int32_t *seq_lens, float scale, int S, int total_q, int max_q, int Hq,
                      int Hkv, int D, int BS, int MB, int NB, const Strides &kv_strides,
                      int kv_partition, void *workspace, size_t ws_bytes, void *stream_v)
{
    VarlenPlan vp;
    pgd_status st = make_varlen_plan(S, total_q, max_q, Hq, Hkv, D, BS, MB, kv_partition, &vp);
    if (st)
        return st;
    if (S == 0 || total_q == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    if (!out || !q || !cu_q || !k_cache || !v_cache || !block_tables || !seq_lens)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (!std::isfinite(scale))
        return fail(PGD_ERR_INVALID_ARG, "scale is not finite");
    if (NB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_blocks %d <= 0", NB);
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return fail(PGD_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    if (!aligned(cu_q, 4) || !aligned(block_tables, 4) || !aligned(seq_lens, 4))
        return fail(PGD_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    if ((st = check_strides(kv_strides, D)))
        return st;
    if (vp.mq) {  // the decode kernel's MQ form (its scratch, tensor maps and launches)
        const MultiQuery mq = {cu_q, total_q, max_q};
        return run(out, q, k_cache, v_cache, block_tables, seq_lens, scale, S, Hq, Hkv, D, BS,
                   vp.PK, MB, NB, kv_strides, workspace, ws_bytes, workspace == nullptr, nullptr,
                   stream_v, nullptr, nullptr, nullptr, false, nullptr, nullptr, nullptr, &mq);
    }
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    cudaError_t e;
    char *ws = static_cast<char *>(workspace);
    const bool own = workspace == nullptr;
    if (vp.ws_bytes) {
        if (own) {
            cudaMemPool_t pool;
            if ((st = device_pool(*ds, &pool)))
                return st;
            if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), vp.ws_bytes, pool,
                                             stream)) != cudaSuccess)
                return cuda_fail(e, "scratch allocation");
        } else if (ws_bytes < vp.ws_bytes || !aligned(ws, 256)) {
            return fail(PGD_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) given, %zu needed",
                        ws_bytes, vp.ws_bytes);
        }
    }
    CUtensorMap tq;
    const CacheGeom geom = {NB, Hkv, BS, D, kv_strides.page, kv_strides.head, kv_strides.token};
    const CUtensorMap *tk = nullptr, *tv = nullptr;
    long long blk_u, blk_n;
    const int box_groups = (BS <= vp.NT ? BS : vp.NT) / 8;
    if ((st = group_blocks(geom, &blk_u, &blk_n)) ||
        (st = encode_q_map(&tq, q, total_q, Hq, D, vp.G, vp.TQ)) ||
        (st = cache_maps(k_cache, v_cache, geom, box_groups, 1, &tk, &tv))) {
        if (own && ws)
            cudaFreeAsync(ws, stream);
        return st;
    }
    VarlenParams p = {};
    p.out = out;
    p.cu_q = cu_q;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.ws_m = vp.NP > 1 ? reinterpret_cast<float *>(ws) : nullptr;
    p.ws_l = vp.NP > 1 ? reinterpret_cast<float *>(ws + vp.off_l) : nullptr;
    p.ws_o = vp.NP > 1 ? reinterpret_cast<float *>(ws + vp.off_o) : nullptr;
    p.order = vp.ordered ? reinterpret_cast<const int *>(ws + vp.off_order) : nullptr;
    p.err = ds->err_word;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S = S;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = vp.G;
    p.TQ = vp.TQ;
    p.QT = vp.QT;
    p.QP = vp.QP;
    p.NP = vp.NP;
    p.PK = vp.PK;
    p.MB = MB;
    p.NB = NB;
    p.BS = BS;
    p.log2BS = BS == 8 ? 3 : BS == 16 ? 4 : BS == 32 ? 5 : BS == 64 ? 6 : 7;
    p.blk_page = (int)(kv_strides.page / blk_u);
    p.blk_head = (int)(kv_strides.head / blk_u);
    p.max_q = max_q;
    p.wait_budget_ns = kWaitBudgetNs;
    e = launch_varlen(D, vp.pairs, tq, *tk, *tv, p, (int)vp.grid, vp.NP > 1 ? total_q * Hq : 0,
                      stream);
    if (own && ws) {
        cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_partition = vp.PK;
    t_last_error.clear();
    return PGD_OK;
}

// Device address of pgd_noalloc_scratch on each device, looked up (with
// that device current) by the first paged_gqa_decode_noalloc call there;
// a failed lookup is not kept, the next call tries again.  `dirty` marks
// the array's claim counter (its first word) as possibly non-zero after a
// call that failed once its partition kernel could have started.
struct NoAllocScratch {
    std::mutex mu;
    void *ptr = nullptr;
    std::atomic<bool> dirty{false};
};

NoAllocScratch g_noalloc[kMaxDevices];

pgd_status noalloc_scratch(void **ptr, std::atomic<bool> **dirty)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(PGD_ERR_UNSUPPORTED, "device ordinal %d beyond %d", dev, kMaxDevices);
    NoAllocScratch &st = g_noalloc[dev];
    std::lock_guard<std::mutex> lock(st.mu);
    if (!st.ptr) {
        void *p = nullptr;
        if ((e = cudaGetSymbolAddress(&p, pgd_noalloc_scratch)) != cudaSuccess)
            return cuda_fail(e, "address of the static scratch");
        st.ptr = p;
    }
    *ptr = st.ptr;
    *dirty = &st.dirty;
    return PGD_OK;
}

// Device staging of paged_gqa_decode_host: q [S][Hq][D] fp16, block_tables
// [S][MB] int32, seq_lens [S] int32, out [S][Hq][D] fp32, each region
// 256-byte aligned.
struct HostStaging {
    size_t q, bt, sl, out, bytes;
};

HostStaging host_staging(int S, int Hq, int D, int MB)
{
    HostStaging h;
    h.q = 0;
    h.bt = align256((size_t)S * Hq * D * 2);
    h.sl = h.bt + align256((size_t)S * MB * 4);
    h.out = h.sl + align256((size_t)S * 4);
    h.bytes = h.out + align256((size_t)S * Hq * D * 4);
    return h;
}

// ------------------------------------------------------------------ trees of drafted tokens
struct TreePlan {
    int G, TQ, cs, runs;
    size_t ws_bytes, off_ml, off_cut;  // pieces' outputs, (maximum, exp-sum)s, cuts
};

// Trees of more than one 128-row tile are worked on by pairs of CTAs (head_dim 128
// and 256; tiles past the second are further units); as many runs of the work as
// are resident at once, or as there can be stages.
pgd_status make_tree_plan(int S, int total_q, int max_q, int Hq, int Hkv, int D, int BS, int MB,
                          TreePlan *tp)
{
    if (S < 0 || total_q < 0 || max_q < 0 || (total_q > 0 && max_q < 1))
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d, total_q %d, max_q_len %d", S, total_q, max_q);
    if (max_q > kTreeMaxNodes)
        return fail(PGD_ERR_UNSUPPORTED, "max_q_len %d: trees of up to %d nodes", max_q,
                    kTreeMaxNodes);
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return fail(PGD_ERR_INVALID_ARG, "head counts %d / %d", Hq, Hkv);
    if (Hq / Hkv > 128)
        return fail(PGD_ERR_UNSUPPORTED, "GQA group of %d query heads exceeds 128", Hq / Hkv);
    if (!supported_head_dim(D))
        return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", D);
    if (Hq > 65536)  // (a tile's rows span 128 / G tokens of Hq heads)
        return fail(PGD_ERR_UNSUPPORTED, "num_q_heads %d above 65536", Hq);
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (MB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "max_blocks_per_seq %d <= 0", MB);
    if ((long long)MB * BS > (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "length bound %lld above 2^30", (long long)MB * BS);
    DeviceState *ds;
    pgd_status st;
    if ((st = device_state(&ds)))
        return st;
    tp->G = Hq / Hkv;
    tp->TQ = 128 / tp->G;
    const int tiles = std::max(1, (max_q + tp->TQ - 1) / tp->TQ);
    int resident;
    tp->cs = tiles > 1 && D > 64 ? 2 : 1;
    if ((st = tree_runs(*ds, D, tp->cs == 2, &resident)))
        return st;
    if (resident < 1)
        return fail(PGD_ERR_UNSUPPORTED, "the tree kernel does not fit on this device");
    const long long stages = (long long)S * Hkv * ((tiles + tp->cs - 1) / tp->cs) *
                             (((long long)MB * BS + kTreeNT - 1) / kTreeNT);
    // (the kernel counts stages, and two more per unit, in 32-bit integers)
    if (3 * stages >= (1ll << 31))
        return fail(PGD_ERR_UNSUPPORTED, "batch of %d sequences x %d KV heads x %lld tokens too large",
                    S, Hkv, (long long)MB * BS);
    tp->runs = (int)std::max(1ll, std::min<long long>(resident, stages));
    const size_t rows = (size_t)2 * tp->runs * tp->cs * 128;
    tp->off_ml = align256(rows * D * 4);
    tp->off_cut = tp->off_ml + align256(rows * 8);
    tp->ws_bytes = S && total_q ? tp->off_cut + align256((size_t)tp->runs * 16) : 0;
    return PGD_OK;
}

// What a copy of the tree kernel's brings: tokens at most and slabs, of K and V.
struct TreeCopies {
    int k_keys, k_slabs, v_keys, v_slabs;
};
template <int D, bool PAIR> TreeCopies tree_copies_of()
{
    using T = TreePieces<D, PAIR>;
    return {T::KKEYS, T::KSLABS, T::VKEYS, T::VSLABS};
}
TreeCopies tree_copies(int D, bool pair)
{
    return D == 64    ? tree_copies_of<64, false>()
           : D == 128 ? (pair ? tree_copies_of<128, true>() : tree_copies_of<128, false>())
                      : (pair ? tree_copies_of<256, true>() : tree_copies_of<256, false>());
}

// The page-group views of K and V that the tree kernel copies from, kept with
// the other kinds' (kind 9: `box` holds the four sizes).
pgd_status tree_maps(const void *k, const void *v, const CacheGeom &geom, const TreeCopies &copies,
                     int k_groups, int v_groups, const CUtensorMap **tk, const CUtensorMap **tv)
{
    return cache_maps(k, v, geom,
                      copies.k_slabs | copies.v_slabs << 4 | k_groups << 8 | v_groups << 16, 9, tk,
                      tv);
}

pgd_status run_tree(void *out, bool half, const uint16_t *q, const int32_t *cu_q,
                    const int32_t *parents, const uint16_t *k_cache, const uint16_t *v_cache,
                    const int32_t *block_tables, const int32_t *seq_lens, float scale, int S,
                    int total_q, int max_q, int Hq, int Hkv, int D, int BS, int MB, int NB,
                    const Strides &kv_strides, void *workspace, size_t ws_bytes, void *stream_v)
{
    TreePlan tp;
    pgd_status st = make_tree_plan(S, total_q, max_q, Hq, Hkv, D, BS, MB, &tp);
    if (st)
        return st;
    if (S == 0 || total_q == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    if (!out || !q || !cu_q || !parents || !k_cache || !v_cache || !block_tables || !seq_lens)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (!std::isfinite(scale))
        return fail(PGD_ERR_INVALID_ARG, "scale is not finite");
    if (NB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_blocks %d <= 0", NB);
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return fail(PGD_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    if (!aligned(cu_q, 4) || !aligned(parents, 4) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4))
        return fail(PGD_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    if ((st = check_strides(kv_strides, D)))
        return st;
    char *ws = static_cast<char *>(workspace);
    const bool own = workspace == nullptr;
    if (!own && (ws_bytes < tp.ws_bytes || !aligned(ws, 256)))
        return fail(PGD_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) given, %zu needed",
                    ws_bytes, tp.ws_bytes);
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    CUtensorMap tq;
    const CacheGeom geom = {NB, Hkv, BS, D, kv_strides.page, kv_strides.head, kv_strides.token};
    const CUtensorMap *tk = nullptr, *tv = nullptr;
    long long blk_u, blk_n;
    // a copy is a page of a piece (or the piece, where pages are longer)
    const TreeCopies copies = tree_copies(D, tp.cs == 2);
    const int k_rows = std::min(BS, copies.k_keys), v_rows = std::min(BS, copies.v_keys);
    if ((st = group_blocks(geom, &blk_u, &blk_n)) ||
        (st = encode_q_map(&tq, q, total_q, Hq, D, tp.G, tp.TQ)) ||
        (st = tree_maps(k_cache, v_cache, geom, copies, k_rows / 8, v_rows / 8, &tk, &tv)))
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    cudaError_t e;
    if (own) {
        cudaMemPool_t pool;
        if ((st = device_pool(*ds, &pool)))
            return st;
        if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), tp.ws_bytes, pool,
                                         stream)) != cudaSuccess)
            return cuda_fail(e, "scratch allocation");
    }
    TreeParams p = {};
    p.out = out;
    p.out_half = half;
    p.wide_rows = aligned(out, 32);
    p.cu_q = cu_q;
    p.parents = parents;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + tp.off_ml);
    p.cut = reinterpret_cast<int4 *>(ws + tp.off_cut);
    p.err = ds->err_word;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S = S;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = tp.G;
    p.TQ = tp.TQ;
    p.total_q = total_q;
    p.max_q = max_q;
    p.MB = MB;
    p.NB = NB;
    p.BS = BS;
    p.log2BS = 3 + bs_index(BS);
    p.cs = tp.cs;
    p.runs = tp.runs;
    p.k_rows = k_rows;
    p.v_rows = v_rows;
    p.blk_page = (int)(kv_strides.page / blk_u);
    p.blk_head = (int)(kv_strides.head / blk_u);
    p.wait_budget_ns = kWaitBudgetNs;
    e = launch_tree(D, tq, *tk, *tv, p, stream);
    if (own) {
        const cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

// ------------------------------------------------------------------ the step around the cache
pgd_status run_slots(int32_t *slots, int32_t *positions, int32_t *cu_seqlens_q, int32_t *seq_lens,
                     int32_t *free_end, int32_t *block_tables, const int32_t *context_lens,
                     const int32_t *query_lens, const int32_t *free_pages,
                     const int32_t *free_start, int S, int N, int num_free, int BS, int MB, int NB,
                     void *stream)
{
    if (S < 0 || N < 0 || num_free < 0)
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d, num_rows %d, num_free %d", S, N, num_free);
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (MB <= 0 || NB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "max_blocks_per_seq %d / num_blocks %d", MB, NB);
    if ((long long)MB * BS > (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "length bound %lld above 2^30", (long long)MB * BS);
    if ((long long)NB * BS > (1ll << 31))
        return fail(PGD_ERR_UNSUPPORTED, "%d pages of %d rows: slots above 2^31", NB, BS);
    if (S > kSlotMaxSeqs)
        return fail(PGD_ERR_UNSUPPORTED, "num_seqs %d above %d", S, kSlotMaxSeqs);
    if (N >= kSlotCountCap || num_free >= kSlotCountCap)
        return fail(PGD_ERR_UNSUPPORTED, "num_rows %d / num_free %d: below 2^30", N, num_free);
    if (!cu_seqlens_q || !free_end || (N > 0 && !slots) || (num_free > 0 && !free_pages) ||
        (S > 0 && (!seq_lens || !block_tables || !context_lens || !query_lens)))
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    for (const void *a : {(const void *)slots, (const void *)positions, (const void *)cu_seqlens_q,
                          (const void *)seq_lens, (const void *)free_end,
                          (const void *)block_tables, (const void *)context_lens,
                          (const void *)query_lens, (const void *)free_pages,
                          (const void *)free_start})
        if (!aligned(a, 4))
            return fail(PGD_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    // every thread block reads its inputs while others write: no array that is
    // written (the first six) shares memory with another
    const struct {
        const void *at;
        long long values;
        const char *name;
    } arrays[] = {{slots, N, "slots"},
                  {positions, positions ? N : 0, "positions"},
                  {cu_seqlens_q, S + 1ll, "cu_seqlens_q"},
                  {seq_lens, S, "seq_lens"},
                  {free_end, 1, "free_end"},
                  {block_tables, (long long)S * MB, "block_tables"},
                  {context_lens, S, "context_lens"},
                  {query_lens, S, "query_lens"},
                  {free_pages, num_free, "free_pages"},
                  {free_start, free_start ? 1 : 0, "free_start"}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 10; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(arrays[i].at),
                            b = reinterpret_cast<uintptr_t>(arrays[j].at);
            if (a < b + 4 * arrays[j].values && b < a + 4 * arrays[i].values)
                return fail(PGD_ERR_INVALID_ARG, "%s overlaps %s", arrays[i].name, arrays[j].name);
        }
    DeviceState *ds;
    pgd_status st;
    if ((st = device_state(&ds)))
        return st;
    SlotParams p = {};
    p.slots = slots;
    p.positions = positions;
    p.cu_seqlens_q = cu_seqlens_q;
    p.seq_lens = seq_lens;
    p.free_end = free_end;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_lens = query_lens;
    p.free_pages = free_pages;
    p.free_start = free_start;
    p.err = ds->err_word;
    p.S = S;
    p.N = N;
    p.num_free = num_free;
    p.log2BS = 3 + bs_index(BS);
    p.MB = MB;
    p.NB = NB;
    p.vector_slots = aligned(slots, 16);
    p.vector_positions = aligned(positions, 16);
    const cudaError_t e = launch_kv_slots(p, ds->num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

pgd_status run_write(uint16_t *k_cache, uint16_t *v_cache, const uint16_t *k_new,
                     const uint16_t *v_new, const int32_t *slots, int rows, int Hkv, int D, int BS,
                     int NB, const Strides &kv, long long k_token, long long k_head,
                     long long v_token, long long v_head, void *stream)
{
    if (rows < 0 || Hkv <= 0 || NB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_rows %d, num_kv_heads %d, num_blocks %d", rows, Hkv,
                    NB);
    if (!supported_head_dim(D))
        return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", D);
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (Hkv > 65536)
        return fail(PGD_ERR_UNSUPPORTED, "num_kv_heads %d above 65536", Hkv);
    pgd_status st;
    if ((st = check_strides(kv, D)))
        return st;
    for (long long x : {k_token, k_head, v_token, v_head})
        if (x <= 0 || x % 8 != 0 || x >= (1ll << 39))
            return fail(PGD_ERR_INVALID_ARG,
                        "source strides (%lld, %lld; %lld, %lld) must be positive multiples of 8 "
                        "halves below 2^39",
                        k_token, k_head, v_token, v_head);
    if (rows == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    if (!k_cache || !v_cache || !k_new || !v_new || !slots)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_new, 16) ||
        !aligned(v_new, 16) || !aligned(slots, 4))
        return fail(PGD_ERR_INVALID_ARG, "k_cache, v_cache, k_new and v_new must be 16-byte "
                                         "aligned, slots 4");
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    WriteParams p = {};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_new = k_new;
    p.v_new = v_new;
    p.slots = slots;
    p.err = ds->err_word;
    p.rows = rows;
    p.Hkv = Hkv;
    p.vec = D / 8;
    p.log2BS = 3 + bs_index(BS);
    p.NB = NB;
    p.page_stride = kv.page;
    p.head_stride = kv.head;
    p.token_stride = kv.token;
    p.k_token_stride = k_token;
    p.k_head_stride = k_head;
    p.v_token_stride = v_token;
    p.v_head_stride = v_head;
    const cudaError_t e = launch_kv_write(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

// ------------------------------------------------------------------ packed prompts
// One of q, k, v of a packed batch: rows [total][heads][D] at any token and head
// strides (halves), as a 4-D tensor.  Keys (box_heads 0): 64 halves x tokens x
// D/64 slabs (128 bytes apart) x heads, a box being `box_tokens` tokens of
// `box_slabs` slabs of one head, landing as [slab][token][128 B].  Queries: 64
// halves x heads x tokens x slabs, a box being `box_heads` heads of
// `box_tokens` tokens of one slab, landing as [token][head][128 B].
pgd_status encode_packed_map(CUtensorMap *map, const void *base, int total, int heads, int D,
                             long long token_stride, long long head_stride, int box_tokens,
                             int box_slabs, int box_heads)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    const bool keys = box_heads == 0;
    const cuuint64_t T = (cuuint64_t)total, H = (cuuint64_t)heads, L = (cuuint64_t)(D / 64);
    const cuuint64_t ts = (cuuint64_t)token_stride * 2, hs = (cuuint64_t)head_stride * 2;
    cuuint64_t dims[4] = {64, keys ? T : H, keys ? L : T, keys ? H : L};
    cuuint64_t strides[3] = {keys ? ts : hs, keys ? 128 : ts, keys ? hs : 128};
    cuuint32_t box[4] = {64, (cuuint32_t)(keys ? box_tokens : box_heads),
                         (cuuint32_t)(keys ? box_slabs : box_tokens), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (packed rows) failed (CUresult %d)", (int)r);
    return PGD_OK;
}

struct PrefillPlan {
    int G, TQ, span, max_units;
    size_t ws_bytes;  // [256 B: unit count][units]
};

pgd_status make_prefill_plan(int S, int total, int Hq, int Hkv, int D, PrefillPlan *pp)
{
    if (S < 0 || total < 0)
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d, total %d", S, total);
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return fail(PGD_ERR_INVALID_ARG, "head counts %d / %d", Hq, Hkv);
    if (Hq / Hkv > 128)
        return fail(PGD_ERR_UNSUPPORTED, "GQA group of %d query heads exceeds 128", Hq / Hkv);
    if (!supported_head_dim(D))
        return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", D);
    if (Hq > 65536)  // (a tile's rows span 128 / G tokens of Hq heads)
        return fail(PGD_ERR_UNSUPPORTED, "num_q_heads %d above 65536", Hq);
    pp->G = Hq / Hkv;
    pp->TQ = 128 / pp->G;
    pp->span = D == 256 ? pp->TQ : 2 * pp->TQ;
    // disjoint prompts: whole spans of all rows, and one begun per prompt
    const long long units = ((long long)total / pp->span + S) * Hkv;
    if (units >= (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "%lld work units", units);
    pp->max_units = (int)units;
    pp->ws_bytes = total && S ? 256 + align256((size_t)units * 16) : 0;
    if (pp->ws_bytes > kMaxWorkspaceBytes)
        return fail(PGD_ERR_WORKSPACE, "scratch of %zu bytes needed, above the %zu-byte cap",
                    pp->ws_bytes, kMaxWorkspaceBytes);
    return PGD_OK;
}

struct PackedStrides {
    long long q_token, q_head, k_token, k_head, v_token, v_head;
};

pgd_status run_prefill(float *out, uint16_t *out_half, const uint16_t *q, const uint16_t *k,
                       const uint16_t *v, const int32_t *cu_seqlens, float scale, int S, int total,
                       int max_len, int Hq, int Hkv, int D, const PackedStrides &x,
                       void *workspace, size_t ws_bytes, void *stream_v)
{
    PrefillPlan pp;
    pgd_status st = make_prefill_plan(S, total, Hq, Hkv, D, &pp);
    if (st)
        return st;
    if (max_len < 0)
        return fail(PGD_ERR_INVALID_ARG, "max_len %d < 0", max_len);
    for (long long s : {x.q_token, x.q_head, x.k_token, x.k_head, x.v_token, x.v_head})
        if (s <= 0 || s % 8 != 0 || s >= (1ll << 39))
            return fail(PGD_ERR_INVALID_ARG,
                        "stride %lld: positive multiples of 8 halves below 2^39", s);
    if (!std::isfinite(scale))
        return fail(PGD_ERR_INVALID_ARG, "scale is not finite");
    if (S == 0 || total == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    const void *dst = out_half ? static_cast<const void *>(out_half) : out;
    if (!dst || !q || !k || !v || !cu_seqlens)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (!aligned(dst, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(cu_seqlens, 4))
        return fail(PGD_ERR_INVALID_ARG, "out, q, k and v must be 16-byte aligned, cu_seqlens 4");
    char *ws = static_cast<char *>(workspace);
    const bool own = workspace == nullptr;
    if (!own && (ws_bytes < pp.ws_bytes || !aligned(ws, 256)))
        return fail(PGD_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) given, %zu needed",
                    ws_bytes, pp.ws_bytes);
    DeviceState *ds;
    if ((st = device_state(&ds)) || (st = prefill_ready(*ds, D)))
        return st;
    CUtensorMap tq, tk, tv;
    const bool wide = D == 256;  // K by slabs of 128 keys, V by 32 keys of all slabs
    if ((st = encode_packed_map(&tq, q, total, Hq, D, x.q_token, x.q_head, pp.TQ, 1, pp.G)) ||
        (st = encode_packed_map(&tk, k, total, Hkv, D, x.k_token, x.k_head, 128, wide ? 1 : D / 64,
                                0)) ||
        (st = encode_packed_map(&tv, v, total, Hkv, D, x.v_token, x.v_head, wide ? 32 : 128, D / 64,
                                0)))
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    cudaError_t e;
    if (own) {
        cudaMemPool_t pool;
        if ((st = device_pool(*ds, &pool)))
            return st;
        if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), pp.ws_bytes, pool,
                                         stream)) != cudaSuccess)
            return cuda_fail(e, "scratch allocation");
    }
    PrefillParams p = {};
    p.out = out;
    p.out_half = reinterpret_cast<__half *>(out_half);
    p.cu_seqlens = cu_seqlens;
    p.num_units = reinterpret_cast<int *>(ws);
    p.units = reinterpret_cast<int4 *>(ws + 256);
    p.err = ds->err_word;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S = S;
    p.total = total;
    p.max_len = max_len;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = pp.G;
    p.TQ = pp.TQ;
    p.span = pp.span;
    p.max_units = pp.max_units;
    p.wide_rows = aligned(dst, 32);
    p.wait_budget_ns = kWaitBudgetNs;
    const int grid = std::min(ds->num_sms, pp.max_units);
    e = launch_prefill(D, tq, tk, tv, p, grid, stream);
    if (own) {
        const cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

// ------------------------------------------------------------------ rotary positions, latent caches
bool stride_ok(long long x) { return x > 0 && x % 8 == 0 && x < (1ll << 39); }

pgd_status check_row_strides(std::initializer_list<long long> strides)
{
    for (long long x : strides)
        if (!stride_ok(x))
            return fail(PGD_ERR_INVALID_ARG,
                        "stride %lld: positive multiples of 8 halves below 2^39", x);
    return PGD_OK;
}

pgd_status check_latent_dims(int R, int P)
{
    if (R != 128 && R != 256 && R != 512)
        return fail(PGD_ERR_UNSUPPORTED, "latent_dim %d not in {128, 256, 512}", R);
    if (P != 32 && P != 64)
        return fail(PGD_ERR_UNSUPPORTED, "rope_dim %d not in {32, 64}", P);
    return PGD_OK;
}

pgd_status check_latent_cache(int R, int P, int BS, int NB, long long page, long long token)
{
    pgd_status st;
    if ((st = check_latent_dims(R, P)))
        return st;
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (NB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_blocks %d <= 0", NB);
    if (!stride_ok(page) || !stride_ok(token))
        return fail(PGD_ERR_INVALID_ARG,
                    "cache strides (%lld, %lld) must be positive multiples of 8 halves below 2^39",
                    page, token);
    if (token < R + P)
        return fail(PGD_ERR_INVALID_ARG, "token stride %lld below latent_dim + rope_dim %d", token,
                    R + P);
    return PGD_OK;
}

// Runs of `width` bytes from `at` on, `rows` x `heads` of them at two strides: an array as a
// call reads or writes it.  (128 bits: strides and counts may come to more than 64.)
using wide_int = __int128;
struct ByteRuns {
    long long at, width, row, head, rows, heads;

    ByteRuns(const void *base, long long halves, long long n = 1, long long row_halves = 0,
             long long h = 1, long long head_halves = 0)
        : at((long long)reinterpret_cast<uintptr_t>(base)), width(2 * halves), row(2 * row_halves),
          head(2 * head_halves), rows(n), heads(h)
    {
    }
    // heads (then rows) that follow one another as one run
    ByteRuns joined() const
    {
        ByteRuns r = *this;
        if (r.heads > 1 && r.head == r.width) {
            r.width *= r.heads;
            r.heads = 1;
        }
        if (r.heads == 1 && r.rows > 1 && r.row == r.width) {
            r.width *= r.rows;
            r.rows = 1;
        }
        return r;
    }
    wide_int end() const { return at + (wide_int)(rows - 1) * row + (wide_int)(heads - 1) * head + width; }
};

wide_int floor_div(wide_int a, wide_int b)  // b > 0
{
    return a / b - (a % b < 0);
}

// Is low < x + k step < high for a whole k in [first, last]?  (low < 0 < high; first <= 0 <=
// last; step > 0, or first = last)
bool steps_into(wide_int x, wide_int step, long long first, long long last, wide_int low, wide_int high)
{
    auto in = [&](wide_int y) { return low < y && y < high; };
    if (first == last)
        return in(x);
    // (rows that lie within a step of one another, as slices of a row do: no division)
    if (-step <= low && high <= step && -step < x && x < step)
        return in(x) || (first < 0 && in(x - step)) || (last > 0 && in(x + step));
    const wide_int from = floor_div(low - x, step) + 1, to = floor_div(high - x - 1, step);
    return std::max<wide_int>(from, first) <= std::min<wide_int>(to, last);
}

// Do two arrays share a byte?  Exactly, so that slices of one projection's output, whose
// address ranges interleave, are told from arrays that overlap: run (n, h) of a meets run
// (m, g) of b where -b.width < b's place - a's place < a.width.  Equal strides count by their
// differences alone.
bool share_memory(const ByteRuns &one, const ByteRuns &other)
{
    if (one.end() <= other.at || other.end() <= one.at)
        return false;
    const ByteRuns a = one.joined(), b = other.joined();
    const bool by_head = a.heads == 1 || b.heads == 1 || a.head == b.head;
    const bool by_row = a.rows == 1 || b.rows == 1 || a.row == b.row;
    const long long row = b.rows > 1 ? b.row : a.row, head = b.heads > 1 ? b.head : a.head;
    auto heads_apart = [&](wide_int x) {  // x: b's head 0 from a's head 0
        if (by_row)
            return steps_into(x, row, 1 - a.rows, b.rows - 1, -b.width, a.width);
        for (long long n = 0; n < a.rows; ++n)
            if (steps_into(x - (wide_int)n * a.row, b.row, 0, b.rows - 1, -b.width, a.width))
                return true;
        return false;
    };
    if (by_head) {
        for (long long h = 1 - a.heads; h < b.heads; ++h)
            if (heads_apart(b.at - a.at + (wide_int)h * head))
                return true;
        return false;
    }
    for (long long h = 0; h < a.heads; ++h)
        for (long long g = 0; g < b.heads; ++g)
            if (heads_apart(b.at - a.at + (wide_int)g * b.head - (wide_int)h * a.head))
                return true;
    return false;
}

// Do two runs of one array share a byte?
bool overlaps_itself(const ByteRuns &a)
{
    if (a.rows > 1 && a.row < a.width)
        return true;
    if (a.head >= a.width && (a.rows == 1 || a.row >= (wide_int)(a.heads - 1) * a.head + a.width))
        return false;
    for (long long h = 1; h < a.heads; ++h)
        if (steps_into((wide_int)h * a.head, a.row, 1 - a.rows, a.rows - 1, -a.width, a.width))
            return true;
    return false;
}

// The turned queries are written while other threads read the call's arrays and write the
// cache: they share no memory with one of them, but for q itself, which the thread that
// turns a pair has read, nor with one another.
pgd_status check_turned_queries(const RopeParams &p)
{
    const long long N = p.rows;
    const int qw = 16 << p.log2q, kw = 16 << p.log2k, vw = 16 << p.log2v;
    const ByteRuns out(p.q_out, qw, N, p.qo_token, p.Hq, p.qo_head);
    if (overlaps_itself(out))
        return fail(PGD_ERR_INVALID_ARG, "rows of q_out overlap one another");
    const struct {
        ByteRuns at;
        const char *name;
    } reads[] = {{{p.k_new, kw, N, p.k_token, p.Hkv, p.k_head}, "the new keys"},
                 {{p.v_new, vw, N, p.v_token, p.Hkv, p.v_head}, "the new values"},
                 {{p.slots, 2 * N}, "slots"},
                 {{p.positions, 2 * N}, "positions"},
                 {{p.inv_freq, p.rot}, "inv_freq"}};
    for (const auto &x : reads)
        if (share_memory(out, x.at))
            return fail(PGD_ERR_INVALID_ARG, "q_out overlaps %s", x.name);
    if (!p.in_place && share_memory(out, ByteRuns(p.q, qw, N, p.q_token, p.Hq, p.q_head)))
        return fail(PGD_ERR_INVALID_ARG, "q_out overlaps q without being q");
    for (const bool v : {false, true}) {
        const uint16_t *const cache = v ? p.v_cache : p.k_cache;
        const int width = v ? vw : kw, BS = 1 << p.log2BS;
        const ByteRuns all(cache, (p.Hkv - 1) * p.head_stride + (BS - 1) * p.token_stride + width, p.NB,
                           p.page_stride);
        if (out.end() <= all.at || all.end() <= out.at)
            continue;
        for (int h = 0; h < p.Hkv; ++h)
            if (share_memory(out, ByteRuns(cache + h * p.head_stride, width, p.NB, p.page_stride, BS,
                                           p.token_stride)))
                return fail(PGD_ERR_INVALID_ARG, "q_out overlaps the cache");
    }
    return PGD_OK;
}

// What paged_rope_write and paged_latent_write share: `p` is filled but for the
// error word.
pgd_status run_rope(RopeParams &p, void *stream)
{
    if (!std::isfinite(p.magnitude))
        return fail(PGD_ERR_INVALID_ARG, "magnitude is not finite");
    if (p.rows >= 1 << 30)
        return fail(PGD_ERR_UNSUPPORTED, "num_rows %d: below 2^30", p.rows);
    if (p.rows == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    if (!p.k_cache || !p.v_cache || !p.k_new || !p.v_new || !p.slots || !p.positions ||
        !p.inv_freq || (p.Hq > 0 && (!p.q || !p.q_out)))
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    for (const void *a : {(const void *)p.k_cache, (const void *)p.v_cache, (const void *)p.k_new,
                          (const void *)p.v_new, (const void *)p.q, (const void *)p.q_out})
        if (!aligned(a, 16))
            return fail(PGD_ERR_INVALID_ARG, "fp16 arrays must be 16-byte aligned");
    if (!aligned(p.slots, 4) || !aligned(p.positions, 4) || !aligned(p.inv_freq, 4))
        return fail(PGD_ERR_INVALID_ARG, "slots, positions and inv_freq must be 4-byte aligned");
    p.in_place = p.Hq > 0 && p.q == p.q_out;
    if (p.in_place && ((p.rows > 1 && p.q_token != p.qo_token) || (p.Hq > 1 && p.q_head != p.qo_head)))
        return fail(PGD_ERR_INVALID_ARG, "q_out is q with other strides");
    DeviceState *ds;
    pgd_status st;
    if ((p.Hq > 0 && (st = check_turned_queries(p))) || (st = device_state(&ds)))
        return st;
    p.err = ds->err_word;
    const cudaError_t e = launch_rope_write(p, ds->num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

int log2_of(int x)
{
    int n = 0;
    while ((1 << n) < x)
        ++n;
    return n;
}

pgd_status run_rope_frequencies(float *inv_freq, float *magnitude, int rot, double base, int scaling,
                                double factor, double original_len, double beta_fast,
                                double beta_slow)
{
    if (!inv_freq)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (rot < 4 || rot % 2 != 0 || rot > 65536)
        return fail(PGD_ERR_INVALID_ARG, "rotary_dim %d: an even number from 4 on", rot);
    if (!(base > 1.0) || !std::isfinite(base))
        return fail(PGD_ERR_INVALID_ARG, "base %g", base);
    if (scaling < PGD_ROPE_PLAIN || scaling > PGD_ROPE_BY_PARTS)
        return fail(PGD_ERR_INVALID_ARG, "scaling %d", scaling);
    if (scaling != PGD_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
        return fail(PGD_ERR_INVALID_ARG, "factor %g: 1 or more", factor);
    const int pairs = rot / 2;
    double low = 0.0, high = 0.0;
    if (scaling == PGD_ROPE_BY_PARTS) {
        if (!(original_len > 0.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
            !std::isfinite(original_len) || !std::isfinite(beta_fast))
            return fail(PGD_ERR_INVALID_ARG, "original_len %g, beta_fast %g, beta_slow %g",
                        original_len, beta_fast, beta_slow);
        // the pair that turns `beta` times in original_len tokens
        auto index = [&](double beta) {
            return rot * std::log(original_len / (beta * 6.283185307179586)) / (2.0 * std::log(base));
        };
        low = std::max(std::floor(index(beta_fast)), 0.0);
        high = std::min(std::ceil(index(beta_slow)), rot - 1.0);
        if (high <= low)
            high = low + 0.001;  // a step
    }
    if (scaling == PGD_ROPE_BASE)
        base *= std::pow(factor, rot / (rot - 2.0));
    for (int i = 0; i < pairs; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == PGD_ROPE_LINEAR)
            f /= factor;
        if (scaling == PGD_ROPE_BY_PARTS) {
            const double shrunk = std::min(std::max((i - low) / (high - low), 0.0), 1.0);
            f = f / factor * shrunk + f * (1.0 - shrunk);
        }
        inv_freq[i] = (float)f;
    }
    if (magnitude)
        *magnitude = scaling == PGD_ROPE_BY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    t_last_error.clear();
    return PGD_OK;
}

struct LatentPlan {
    int hb, TQ, HB, runs;
    bool check_cost;
    size_t ws_bytes, off_ml, off_cut, off_allowed;  // pieces' outputs, (maximum, exp-sum)s, cuts
};

pgd_status make_latent_plan(int S, int total_q, int max_q, int H, int R, int P, int BS, int MB,
                            LatentPlan *lp)
{
    if (S < 0 || total_q < 0 || max_q < 0 || (total_q > 0 && max_q < 1))
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d, total_q %d, max_q_len %d", S, total_q, max_q);
    if (H <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_heads %d", H);
    if (H > 65536)
        return fail(PGD_ERR_UNSUPPORTED, "num_heads %d above 65536", H);
    pgd_status st;
    if ((st = check_latent_dims(R, P)))
        return st;
    if (!supported_block_size(BS))
        return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}", BS);
    if (MB <= 0)
        return fail(PGD_ERR_INVALID_ARG, "max_blocks_per_seq %d <= 0", MB);
    if ((long long)MB * BS > (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "length bound %lld above 2^30", (long long)MB * BS);
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    int resident;
    if ((st = latent_runs(*ds, R, &resident)))
        return st;
    if (resident < 1)
        return fail(PGD_ERR_UNSUPPORTED, "the latent kernel does not fit on this device");
    lp->hb = std::min(H, kLatentRows);
    lp->HB = (H + kLatentRows - 1) / kLatentRows;
    lp->TQ = H <= kLatentRows ? kLatentRows / H : 1;
    const long long most_q = std::min(max_q, total_q);
    const long long stages = ((long long)MB * BS + kLatentNT - 1) / kLatentNT;
    // tiles of one sequence, and of all: a sequence has no more than that, and all of them
    // together whole tiles of their rows and one begun in each that has any
    auto tiles_of = [&](long long q, long long begun) {
        return lp->HB == 1 ? (q + begun * (2 * lp->TQ - 1)) / (2 * lp->TQ)
                           : (q * lp->HB + begun * (lp->HB & 1)) / 2;
    };
    const long long one = tiles_of(most_q, 1);
    // (the kernel counts stages, and a unit's start and end, in 32-bit integers; a unit
    // has one stage at least.  Where rows that overlap could ask for more, a kernel in front
    // adds it up.)
    constexpr long long most = (1ll << 31) / (1 + kLatentUnitCost);
    const long long all =
        one >= most ? one : std::min(S * one, tiles_of(total_q, std::min(S, total_q)));
    if (all >= most || all * stages >= most)
        return fail(PGD_ERR_UNSUPPORTED,
                    "%d sequences of %d rows (up to %lld each) x %d heads, %lld tokens: too large", S,
                    total_q, most_q, H, (long long)MB * BS);
    // (the table's bound, however few rows the call has: the division of a batch's work does
    // not change with total_q)
    lp->check_cost = S * one >= most || S * one * stages >= most;
    const long long units = std::min<long long>(resident, S * one);
    lp->runs = (int)std::max(1ll, std::min<long long>(resident, units * stages));
    const size_t rows = (size_t)2 * lp->runs * 2 * kLatentRows;
    lp->off_ml = align256(rows * R * 4);
    lp->off_cut = lp->off_ml + align256(rows * 8);
    lp->off_allowed = lp->off_cut + align256((size_t)lp->runs * 16);
    lp->ws_bytes = S && total_q ? lp->off_allowed + (lp->check_cost ? 256 : 0) : 0;
    return PGD_OK;
}

// The views of a call: the queries' two parts [tokens][heads][64-wide slabs], a
// box being one slab of a half tile's rows; the cache's pages by groups of 8 rows
// (as encode_cache_map_groups), its latent part for K and V in copies of their own,
// its rotary keys.  Where rope_dim is 32 the slab's other half reads as zeros.
struct LatentViews {
    const void *q, *q_rope, *cache;
    long long q_token, q_head, qr_token, qr_head, page, token;
    int total_q, H, R, P, NB, BS, hb, TQ, k_slabs, k_rows, v_slabs, v_rows;
};

pgd_status encode_view(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box)
{
    EncodeTiledFn fn;
    pgd_status st = encode_fn(&fn);
    if (st)
        return st;
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void *>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PGD_ERR_CUDA, "cuTensorMapEncodeTiled (latent rows) failed (CUresult %d)", (int)r);
    return PGD_OK;
}

pgd_status encode_latent_maps(const LatentViews &v, LatentMaps *m)
{
    using u64 = cuuint64_t;
    using u32 = cuuint32_t;
    const u64 T = (u64)v.total_q, H = (u64)v.H, slabs = (u64)v.R / 64, groups = (u64)v.BS / 8,
              NB = (u64)v.NB;
    const u64 tok = (u64)v.token * 2, page = (u64)v.page * 2;
    const u64 q_dims[4] = {64, H, T, slabs}, q_str[3] = {(u64)v.q_head * 2, (u64)v.q_token * 2, 128};
    const u64 r_dims[4] = {(u64)v.P, H, T, 1},
              r_str[3] = {(u64)v.qr_head * 2, (u64)v.qr_token * 2, 128};
    const u32 q_box[4] = {64, (u32)v.hb, (u32)v.TQ, 1};
    const u64 c_dims[5] = {64, 8, slabs, groups, NB}, c_str[4] = {tok, 128, tok * 8, page};
    const u32 k_box[5] = {64, 8, (u32)v.k_slabs, (u32)v.k_rows / 8, 1};
    const u32 v_box[5] = {64, 8, (u32)v.v_slabs, (u32)v.v_rows / 8, 1};
    const u64 kr_dims[4] = {(u64)v.P, 8, groups, NB}, kr_str[3] = {tok, tok * 8, page};
    const u32 kr_box[4] = {64, 8, (u32)v.k_rows / 8, 1};
    pgd_status st;
    if ((st = encode_view(&m->q, v.q, 4, q_dims, q_str, q_box)) ||
        (st = encode_view(&m->qr, v.q_rope, 4, r_dims, r_str, q_box)) ||
        (st = encode_view(&m->k, v.cache, 5, c_dims, c_str, k_box)) ||
        (st = encode_view(&m->v, v.cache, 5, c_dims, c_str, v_box)) ||
        (st = encode_view(&m->kr, static_cast<const uint16_t *>(v.cache) + v.R, 4, kr_dims, kr_str,
                          kr_box)))
        return st;
    return PGD_OK;
}

struct LatentStrides {
    long long page, token, q_token, q_head, qr_token, qr_head;
};

pgd_status run_latent(void *out, bool half, const uint16_t *q, const uint16_t *q_rope,
                      const int32_t *cu_q, const uint16_t *cache, const int32_t *block_tables,
                      const int32_t *seq_lens, float scale, int S, int total_q, int max_q, int H,
                      int R, int P, int BS, int MB, int NB, const LatentStrides &x, void *workspace,
                      size_t ws_bytes, void *stream_v)
{
    pgd_status st;
    if ((st = check_latent_cache(R, P, BS, NB, x.page, x.token)) ||
        (st = check_row_strides({x.q_token, x.q_head, x.qr_token, x.qr_head})))
        return st;
    if (!std::isfinite(scale))
        return fail(PGD_ERR_INVALID_ARG, "scale is not finite");
    if (!cu_q && total_q != S)
        return fail(PGD_ERR_INVALID_ARG, "total_q %d for %d sequences of one row", total_q, S);
    if (!cu_q)
        max_q = 1;
    LatentPlan lp;
    if ((st = make_latent_plan(S, total_q, max_q, H, R, P, BS, MB, &lp)))
        return st;
    if (S == 0 || total_q == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    if (!out || !q || !q_rope || !cache || !block_tables || !seq_lens)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (!aligned(q, 16) || !aligned(q_rope, 16) || !aligned(cache, 16) || !aligned(out, 16))
        return fail(PGD_ERR_INVALID_ARG, "q, q_rope, cache and out must be 16-byte aligned");
    if (!aligned(cu_q, 4) || !aligned(block_tables, 4) || !aligned(seq_lens, 4))
        return fail(PGD_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    char *ws = static_cast<char *>(workspace);
    const bool own = workspace == nullptr;
    if (!own && (ws_bytes < lp.ws_bytes || !aligned(ws, 256)))
        return fail(PGD_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) given, %zu needed",
                    ws_bytes, lp.ws_bytes);
    DeviceState *ds;
    if ((st = device_state(&ds)))
        return st;
    const int v_keys = 128 / (R / 128);  // of a piece (LatentShape)
    const LatentViews views = {q,        q_rope,     cache,      x.q_token, x.q_head, x.qr_token,
                               x.qr_head, x.page,    x.token,    total_q,   H,        R,
                               P,        NB,         BS,         lp.hb,     lp.TQ,    2,
                               std::min(BS, kLatentRows), R / 128, std::min(BS, v_keys)};
    LatentMaps maps;
    if ((st = encode_latent_maps(views, &maps)))
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    cudaError_t e;
    if (own) {
        cudaMemPool_t pool;
        if ((st = device_pool(*ds, &pool)))
            return st;
        if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), lp.ws_bytes, pool,
                                         stream)) != cudaSuccess)
            return cuda_fail(e, "scratch allocation");
    }
    LatentParams p = {};
    p.out = out;
    p.out_half = half;
    p.wide_rows = aligned(out, 32);
    p.cu_q = cu_q;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + lp.off_ml);
    p.cut = reinterpret_cast<int4 *>(ws + lp.off_cut);
    p.allowed = lp.check_cost ? reinterpret_cast<int *>(ws + lp.off_allowed) : nullptr;
    p.err = ds->err_word;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S = S;
    p.total_q = total_q;
    p.max_q = max_q;
    p.H = H;
    p.R = R;
    p.MB = MB;
    p.NB = NB;
    p.BS = BS;
    p.log2BS = 3 + bs_index(BS);
    p.hb = lp.hb;
    p.TQ = lp.TQ;
    p.HB = lp.HB;
    p.k_rows = views.k_rows;
    p.v_rows = views.v_rows;
    p.runs = lp.runs;
    p.wait_budget_ns = kWaitBudgetNs;
    e = launch_latent(maps, p, stream);
    if (own) {
        const cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

struct LatentPrefillPlan {
    int max_units;
    size_t ws_bytes;  // [256 B: unit count][units]
};

pgd_status make_latent_prefill_plan(int S, int total, int H, int D, int P, LatentPrefillPlan *pp)
{
    if (S < 0 || total < 0)
        return fail(PGD_ERR_INVALID_ARG, "num_seqs %d, total %d", S, total);
    if (H <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_heads %d", H);
    if (H > 65536)
        return fail(PGD_ERR_UNSUPPORTED, "num_heads %d above 65536", H);
    if (D != 64 && D != 128)
        return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", D);
    if (P != 32 && P != 64)
        return fail(PGD_ERR_UNSUPPORTED, "rope_dim %d not in {32, 64}", P);
    // disjoint prompts: whole pairs of tiles of all rows, and one begun per prompt
    const long long units = ((long long)total / 256 + S) * H;
    if (units >= (1ll << 30))
        return fail(PGD_ERR_UNSUPPORTED, "%lld work units", units);
    pp->max_units = (int)units;
    pp->ws_bytes = total && S ? 256 + align256((size_t)units * 16) : 0;
    if (pp->ws_bytes > kMaxWorkspaceBytes)
        return fail(PGD_ERR_WORKSPACE, "scratch of %zu bytes needed, above the %zu-byte cap",
                    pp->ws_bytes, kMaxWorkspaceBytes);
    return PGD_OK;
}

struct ExpandedStrides {
    long long q_token, q_head, k_token, k_head, kr_token, v_token, v_head;
};

pgd_status run_latent_prefill(float *out, uint16_t *out_half, const uint16_t *q, const uint16_t *k,
                              const uint16_t *k_rope, const uint16_t *v, const int32_t *cu_seqlens,
                              float scale, int S, int total, int max_len, int H, int D, int P,
                              const ExpandedStrides &x, void *workspace, size_t ws_bytes,
                              void *stream_v)
{
    LatentPrefillPlan pp;
    pgd_status st = make_latent_prefill_plan(S, total, H, D, P, &pp);
    if (st)
        return st;
    if (max_len < 0)
        return fail(PGD_ERR_INVALID_ARG, "max_len %d < 0", max_len);
    if ((st = check_row_strides({x.q_token, x.q_head, x.k_token, x.k_head, x.kr_token, x.v_token,
                                 x.v_head})))
        return st;
    if (!std::isfinite(scale))
        return fail(PGD_ERR_INVALID_ARG, "scale is not finite");
    if (S == 0 || total == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    const void *dst = out_half ? static_cast<const void *>(out_half) : out;
    if (!dst || !q || !k || !k_rope || !v || !cu_seqlens)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    for (const void *a : {dst, (const void *)q, (const void *)k, (const void *)k_rope, (const void *)v})
        if (!aligned(a, 16))
            return fail(PGD_ERR_INVALID_ARG, "out, q, k, k_rope and v must be 16-byte aligned");
    if (!aligned(cu_seqlens, 4))
        return fail(PGD_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
    char *ws = static_cast<char *>(workspace);
    const bool own = workspace == nullptr;
    if (!own && (ws_bytes < pp.ws_bytes || !aligned(ws, 256)))
        return fail(PGD_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) given, %zu needed",
                    ws_bytes, pp.ws_bytes);
    DeviceState *ds;
    if ((st = device_state(&ds)) || (st = latent_prefill_ready(*ds, D)))
        return st;
    // rows of one head (of all heads: rope) as 64 halves x tokens x slabs x heads, a box
    // being 128 tokens of Q with all slabs, of K with one, 64 or 128 of V with all
    using u64 = cuuint64_t;
    using u32 = cuuint32_t;
    const u64 T = (u64)total, heads = (u64)H, slabs = (u64)D / 64;
    const u32 v_keys = D == 64 ? kLatentVKeys64 : kLatentVKeys128;
    LatentPrefillMaps maps;
    auto view = [&](CUtensorMap *map, const uint16_t *base, u64 width, u64 n_slabs, u64 n_heads,
                    long long token, long long head, u32 box_tokens, u32 box_slabs) -> pgd_status {
        const u64 dims[4] = {width, T, n_slabs, n_heads};
        const u64 strides[3] = {(u64)token * 2, 128, (u64)head * 2};
        const u32 box[4] = {64, box_tokens, box_slabs, 1};
        return encode_view(map, base, 4, dims, strides, box);
    };
    if ((st = view(&maps.q, q, 64, slabs, heads, x.q_token, x.q_head, 128, (u32)slabs)) ||
        (st = view(&maps.qr, q + D, (u64)P, 1, heads, x.q_token, x.q_head, 128, 1)) ||
        (st = view(&maps.k, k, 64, slabs, heads, x.k_token, x.k_head, 128, 1)) ||
        (st = view(&maps.kr, k_rope, (u64)P, 1, 1, x.kr_token, 8, 128, 1)) ||
        (st = view(&maps.v, v, 64, slabs, heads, x.v_token, x.v_head, v_keys, (u32)slabs)))
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    cudaError_t e;
    if (own) {
        cudaMemPool_t pool;
        if ((st = device_pool(*ds, &pool)))
            return st;
        if ((e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), pp.ws_bytes, pool,
                                         stream)) != cudaSuccess)
            return cuda_fail(e, "scratch allocation");
    }
    PrefillParams p = {};
    p.out = out;
    p.out_half = reinterpret_cast<__half *>(out_half);
    p.cu_seqlens = cu_seqlens;
    p.num_units = reinterpret_cast<int *>(ws);
    p.units = reinterpret_cast<int4 *>(ws + 256);
    p.err = ds->err_word;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S = S;
    p.total = total;
    p.max_len = max_len;
    p.Hq = p.Hkv = H;
    p.G = 1;
    p.TQ = 128;
    p.span = 256;
    p.max_units = pp.max_units;
    p.wide_rows = aligned(dst, 32);
    p.wait_budget_ns = kWaitBudgetNs;
    e = launch_latent_prefill(D, maps, p, std::min(ds->num_sms, pp.max_units), stream);
    if (own) {
        const cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess)
            e = e2;
    }
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

// Runs a C entry's body: nothing it throws (an allocation of the host's that
// failed) leaves the library.
template <class F> pgd_status guarded(F &&body) noexcept
{
    try {
        return body();
    } catch (...) {
        return PGD_ERR_CUDA;
    }
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" {

pgd_status paged_gqa_decode(float *out, const uint16_t *q, const uint16_t *k_cache,
                            const uint16_t *v_cache, const int32_t *block_tables,
                            const int32_t *seq_lens, float scale, int num_seqs, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int partition_size,
                            int max_blocks_per_seq, int num_blocks, void *stream)
{
    return run(out, q, k_cache, v_cache, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, head_major(num_kv_heads, block_size, head_dim), nullptr, 0, true,
               nullptr, stream);
}

pgd_status paged_gqa_decode_ex(float *out, const uint16_t *q, const uint16_t *k_cache,
                               const uint16_t *v_cache, const int32_t *block_tables,
                               const int32_t *seq_lens, float scale, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               int partition_size, int max_blocks_per_seq, int num_blocks,
                               void *workspace, size_t workspace_bytes, int32_t *page_trace,
                               void *stream)
{
    return run(out, q, k_cache, v_cache, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, head_major(num_kv_heads, block_size, head_dim), workspace,
               workspace_bytes, false, page_trace, stream);
}

pgd_status paged_gqa_decode_append(float *out, const uint16_t *q, const uint16_t *k_new,
                                   const uint16_t *v_new, uint16_t *k_cache, uint16_t *v_cache,
                                   const int32_t *block_tables, const int32_t *seq_lens,
                                   float scale, int num_seqs, int num_q_heads, int num_kv_heads,
                                   int head_dim, int block_size, int partition_size,
                                   int max_blocks_per_seq, int num_blocks, void *stream)
{
    if (num_seqs > 0 && (!k_new || !v_new))
        return fail(PGD_ERR_INVALID_ARG, "null k_new / v_new");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(PGD_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    return run(out, q, k_cache, v_cache, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, head_major(num_kv_heads, block_size, head_dim), nullptr, 0, true,
               nullptr, stream, nullptr, k_new, v_new);
}

pgd_status paged_gqa_decode_strided(float *out, const uint16_t *q, const uint16_t *k_new,
                                    const uint16_t *v_new, uint16_t *k_cache, uint16_t *v_cache,
                                    const int32_t *block_tables, const int32_t *seq_lens,
                                    float scale, int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_dim, int block_size, int partition_size,
                                    int max_blocks_per_seq, int num_blocks, int64_t page_stride,
                                    int64_t head_stride, int64_t token_stride, void *workspace,
                                    size_t workspace_bytes, int32_t *page_trace, void *stream)
{
    if ((k_new == nullptr) != (v_new == nullptr))
        return fail(PGD_ERR_INVALID_ARG, "give both k_new and v_new or neither");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(PGD_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    const bool own = workspace == nullptr;
    return run(out, q, k_cache, v_cache, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, Strides{page_stride, head_stride, token_stride}, workspace,
               workspace_bytes, own, page_trace, stream, nullptr, k_new, v_new);
}

pgd_status paged_gqa_decode_noalloc(float *out, const uint16_t *q, const uint16_t *k_cache,
                                    const uint16_t *v_cache, const int32_t *block_tables,
                                    const int32_t *seq_lens, float scale, int num_seqs,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int partition_size, int max_blocks_per_seq,
                                    int num_blocks, void *stream)
{
    Plan plan;
    pgd_status st = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              partition_size, max_blocks_per_seq, &plan);
    if (st)
        return st;
    if (plan.ws_bytes > PGD_NOALLOC_SCRATCH_BYTES - 256)
        return fail(PGD_ERR_WORKSPACE,
                    "these sizes need %zu bytes of scratch, more than the %zu bytes of static "
                    "scratch of paged_gqa_decode_noalloc; use paged_gqa_decode or "
                    "paged_gqa_decode_ex",
                    plan.ws_bytes, (size_t)PGD_NOALLOC_SCRATCH_BYTES - 256);
    void *scratch = nullptr;
    std::atomic<bool> *dirty = nullptr;
    if ((st = noalloc_scratch(&scratch, &dirty)))
        return st;
    // [256 B: claim counter, zero at load and after every call][partials]
    const GivenCounter counter = {static_cast<unsigned *>(scratch), dirty};
    return run(out, q, k_cache, v_cache, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, head_major(num_kv_heads, block_size, head_dim),
               static_cast<char *>(scratch) + 256, PGD_NOALLOC_SCRATCH_BYTES - 256, false,
               nullptr, stream, &counter);
}

size_t pgd_host_staging_bytes(int num_seqs, int num_q_heads, int head_dim,
                              int max_blocks_per_seq)
{
    if (num_seqs < 0 || num_q_heads <= 0 || head_dim <= 0 || max_blocks_per_seq <= 0) {
        fail(PGD_ERR_INVALID_ARG, "num_seqs %d, num_q_heads %d, head_dim %d, max_blocks_per_seq %d",
             num_seqs, num_q_heads, head_dim, max_blocks_per_seq);
        return ~(size_t)0;
    }
    t_last_error.clear();
    return host_staging(num_seqs, num_q_heads, head_dim, max_blocks_per_seq).bytes;
}

pgd_status paged_gqa_decode_host(float *out_host, const uint16_t *q_host,
                                 const int32_t *block_tables_host, const int32_t *seq_lens_host,
                                 const uint16_t *k_cache, const uint16_t *v_cache, float scale,
                                 int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int partition_size, int max_blocks_per_seq,
                                 int num_blocks, void *staging, size_t staging_bytes,
                                 void *stream_v)
{
    const int S = num_seqs, Hq = num_q_heads, D = head_dim, MB = max_blocks_per_seq;
    pgd_status st = check_sizes(S, Hq, num_kv_heads, D, block_size, partition_size, MB);
    if (st)
        return st;
    if (S == 0)
        return run(nullptr, nullptr, k_cache, v_cache, nullptr, nullptr, scale, S, Hq,
                   num_kv_heads, D, block_size, partition_size, MB, num_blocks,
                   head_major(num_kv_heads, block_size, D), nullptr, 0, true, nullptr, stream_v);
    if (!out_host || !q_host || !block_tables_host || !seq_lens_host || !staging)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    const HostStaging hs = host_staging(S, Hq, D, MB);
    if (!aligned(staging, 256) || staging_bytes < hs.bytes)
        return fail(PGD_ERR_WORKSPACE, "staging of %zu bytes (256-byte aligned) given, %zu needed",
                    staging_bytes, hs.bytes);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    char *dev = static_cast<char *>(staging);
    uint16_t *q = reinterpret_cast<uint16_t *>(dev + hs.q);
    int32_t *bt = reinterpret_cast<int32_t *>(dev + hs.bt);
    int32_t *sl = reinterpret_cast<int32_t *>(dev + hs.sl);
    float *out = reinterpret_cast<float *>(dev + hs.out);
    cudaError_t e;
    if ((e = cudaMemcpyAsync(q, q_host, (size_t)S * Hq * D * 2, cudaMemcpyHostToDevice,
                             stream)) != cudaSuccess ||
        (e = cudaMemcpyAsync(bt, block_tables_host, (size_t)S * MB * 4, cudaMemcpyHostToDevice,
                             stream)) != cudaSuccess ||
        (e = cudaMemcpyAsync(sl, seq_lens_host, (size_t)S * 4, cudaMemcpyHostToDevice,
                             stream)) != cudaSuccess)
        return cuda_fail(e, "copy of the step's inputs to the device");
    if ((st = run(out, q, k_cache, v_cache, bt, sl, scale, S, Hq, num_kv_heads, D, block_size,
                  partition_size, MB, num_blocks, head_major(num_kv_heads, block_size, D),
                  nullptr, 0, true, nullptr, stream_v)))
        return st;
    if ((e = cudaMemcpyAsync(out_host, out, (size_t)S * Hq * D * 4, cudaMemcpyDeviceToHost,
                             stream)) != cudaSuccess)
        return cuda_fail(e, "copy of the output to the host");
    if ((e = cudaStreamSynchronize(stream)) != cudaSuccess)
        return cuda_fail(e, "stream synchronize");
    t_last_error.clear();
    return PGD_OK;
}

pgd_status paged_gqa_decode_q8(float *out, const uint16_t *q, const uint8_t *k_codes,
                               const uint16_t *k_meta, const uint8_t *v_codes,
                               const uint16_t *v_meta, const int32_t *block_tables,
                               const int32_t *seq_lens, float scale, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               int partition_size, int max_blocks_per_seq, int num_blocks,
                               void *workspace, size_t workspace_bytes, int32_t *page_trace,
                               void *stream)
{
    if (num_seqs > 0 && (!k_meta || !v_meta))
        return fail(PGD_ERR_INVALID_ARG, "null k_meta / v_meta");
    const bool own = workspace == nullptr;
    // the codes' strides in elements (bytes): head-major [NB][Hkv][BS][D]
    return run(out, q, k_codes, v_codes, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, head_major(num_kv_heads, block_size, head_dim), workspace,
               workspace_bytes, own, page_trace, stream, nullptr, nullptr, nullptr, true, k_meta,
               v_meta);
}

pgd_status paged_gqa_decode_q8_append(float *out, const uint16_t *q, const uint16_t *k_new,
                                      const uint16_t *v_new, uint8_t *k_codes, uint16_t *k_meta,
                                      uint8_t *v_codes, uint16_t *v_meta,
                                      const int32_t *block_tables, const int32_t *seq_lens,
                                      float scale, int num_seqs, int num_q_heads,
                                      int num_kv_heads, int head_dim, int block_size,
                                      int partition_size, int max_blocks_per_seq, int num_blocks,
                                      void *stream)
{
    if (num_seqs > 0 && (!k_new || !v_new || !k_meta || !v_meta))
        return fail(PGD_ERR_INVALID_ARG, "null k_new / v_new / k_meta / v_meta");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(PGD_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    return run(out, q, k_codes, v_codes, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, head_major(num_kv_heads, block_size, head_dim), nullptr, 0, true,
               nullptr, stream, nullptr, k_new, v_new, true, k_meta, v_meta);
}

pgd_status paged_gqa_decode_q8_strided(
    float *out, const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new, uint8_t *k_codes,
    uint16_t *k_meta, uint8_t *v_codes, uint16_t *v_meta, const int32_t *block_tables,
    const int32_t *seq_lens, float scale, int num_seqs, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, int partition_size, int max_blocks_per_seq, int num_blocks,
    int64_t code_page_stride, int64_t code_head_stride, int64_t code_token_stride,
    int64_t meta_page_stride, int64_t meta_head_stride, int64_t meta_token_stride,
    void *workspace, size_t workspace_bytes, void *stream)
{
    if ((k_new == nullptr) != (v_new == nullptr))
        return fail(PGD_ERR_INVALID_ARG, "give both k_new and v_new or neither");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(PGD_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    if (num_seqs > 0 && (!k_meta || !v_meta))
        return fail(PGD_ERR_INVALID_ARG, "null k_meta / v_meta");
    const Strides ms = {meta_page_stride, meta_head_stride, meta_token_stride};
    return run(out, q, k_codes, v_codes, block_tables, seq_lens, scale, num_seqs, num_q_heads,
               num_kv_heads, head_dim, block_size, partition_size, max_blocks_per_seq,
               num_blocks, {code_page_stride, code_head_stride, code_token_stride}, workspace,
               workspace_bytes, workspace == nullptr, nullptr, stream, nullptr, k_new, v_new,
               true, k_meta, v_meta, &ms);
}

pgd_status paged_kv_quantize(uint8_t *codes, uint16_t *meta, const uint16_t *src,
                             const int32_t *slots, int num_rows, int num_kv_heads, int head_dim,
                             int block_size, int num_blocks, void *stream)
{
    if (num_rows < 0 || num_kv_heads <= 0 || num_blocks <= 0 || block_size <= 0)
        return fail(PGD_ERR_INVALID_ARG, "num_rows %d, num_kv_heads %d, num_blocks %d, block_size %d",
                    num_rows, num_kv_heads, num_blocks, block_size);
    if (head_dim != 128 && head_dim != 256)
        return fail(PGD_ERR_UNSUPPORTED, "quantised pages need head_dim 128 or 256, not %d",
                    head_dim);
    if ((long long)num_blocks * num_kv_heads * block_size >= (1ll << 40))
        return fail(PGD_ERR_UNSUPPORTED, "cache of %lld rows", (long long)num_blocks * num_kv_heads * block_size);
    if (num_rows == 0) {
        t_last_error.clear();
        return PGD_OK;
    }
    if (!codes || !meta || !src || !slots)
        return fail(PGD_ERR_INVALID_ARG, "null array argument");
    if (!aligned(codes, 16) || !aligned(meta, 16) || !aligned(src, 16) || !aligned(slots, 4))
        return fail(PGD_ERR_INVALID_ARG, "codes, meta and src must be 16-byte aligned, slots 4");
    DeviceState *ds;
    pgd_status st;
    if ((st = device_state(&ds)))
        return st;
    const cudaError_t e = launch_quantize(head_dim, codes, meta, src, slots, num_rows,
                                          num_kv_heads, block_size, num_blocks, ds->err_word,
                                          static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "kernel launch");
    t_last_error.clear();
    return PGD_OK;
}

pgd_status paged_gqa_varlen(float *out, const uint16_t *q, const int32_t *cu_seqlens_q,
                            const uint16_t *k_cache, const uint16_t *v_cache,
                            const int32_t *block_tables, const int32_t *seq_lens, float scale,
                            int num_seqs, int total_q, int max_q_len, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size,
                            int max_blocks_per_seq, int num_blocks, int64_t page_stride,
                            int64_t head_stride, int64_t token_stride, int kv_partition,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    return run_varlen(out, q, cu_seqlens_q, k_cache, v_cache, block_tables, seq_lens, scale,
                      num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads, head_dim,
                      block_size, max_blocks_per_seq, num_blocks,
                      Strides{page_stride, head_stride, token_stride}, kv_partition, workspace,
                      workspace_bytes, stream);
}

pgd_status pgd_varlen_plan(int num_seqs, int total_q, int max_q_len, int num_q_heads,
                           int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                           int kv_partition, int *chosen_kv_partition, size_t *workspace_bytes)
{
    VarlenPlan vp;
    pgd_status st = make_varlen_plan(num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads,
                                     head_dim, block_size, max_blocks_per_seq, kv_partition, &vp);
    if (st)
        return st;
    if (chosen_kv_partition)
        *chosen_kv_partition = vp.PK;
    if (workspace_bytes)
        *workspace_bytes = vp.ws_bytes;
    return PGD_OK;
}

pgd_status paged_gqa_tree(void *out, int out_type, const uint16_t *q, const int32_t *cu_seqlens_q,
                          const int32_t *parents, const uint16_t *k_cache, const uint16_t *v_cache,
                          const int32_t *block_tables, const int32_t *seq_lens, float scale,
                          int num_seqs, int total_q, int max_q_len, int num_q_heads,
                          int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                          int num_blocks, int64_t page_stride, int64_t head_stride,
                          int64_t token_stride, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    return guarded([&]() -> pgd_status {
        if (out_type != PGD_OUT_F32 && out_type != PGD_OUT_F16)
            return fail(PGD_ERR_INVALID_ARG, "out_type %d: PGD_OUT_F32 or PGD_OUT_F16", out_type);
        return run_tree(out, out_type == PGD_OUT_F16, q, cu_seqlens_q, parents, k_cache, v_cache,
                        block_tables, seq_lens, scale, num_seqs, total_q, max_q_len, num_q_heads,
                        num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                        Strides{page_stride, head_stride, token_stride}, workspace,
                        workspace_bytes, stream);
    });
}

pgd_status pgd_tree_plan(int num_seqs, int total_q, int max_q_len, int num_q_heads,
                         int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                         size_t *workspace_bytes)
{
    return guarded([&]() -> pgd_status {
        TreePlan tp;
        const pgd_status st = make_tree_plan(num_seqs, total_q, max_q_len, num_q_heads,
                                             num_kv_heads, head_dim, block_size,
                                             max_blocks_per_seq, &tp);
        if (st)
            return st;
        if (workspace_bytes)
            *workspace_bytes = tp.ws_bytes;
        return PGD_OK;
    });
}

pgd_status packed_gqa_prefill(void *out, int out_type, const uint16_t *q, const uint16_t *k,
                              const uint16_t *v, const int32_t *cu_seqlens, float scale,
                              int num_seqs, int total, int max_len, int num_q_heads,
                              int num_kv_heads, int head_dim, int64_t q_token_stride,
                              int64_t q_head_stride, int64_t k_token_stride,
                              int64_t k_head_stride, int64_t v_token_stride,
                              int64_t v_head_stride, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    return guarded([&]() -> pgd_status {
        if (out_type != PGD_OUT_F32 && out_type != PGD_OUT_F16)
            return fail(PGD_ERR_INVALID_ARG, "out_type %d: PGD_OUT_F32 or PGD_OUT_F16", out_type);
        const bool half = out_type == PGD_OUT_F16;
        return run_prefill(half ? nullptr : static_cast<float *>(out),
                           half ? static_cast<uint16_t *>(out) : nullptr, q, k, v, cu_seqlens,
                           scale, num_seqs, total, max_len, num_q_heads, num_kv_heads, head_dim,
                           {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                            v_token_stride, v_head_stride},
                           workspace, workspace_bytes, stream);
    });
}

pgd_status pgd_prefill_plan(int num_seqs, int total, int num_q_heads, int num_kv_heads,
                            int head_dim, size_t *workspace_bytes)
{
    return guarded([&]() -> pgd_status {
        PrefillPlan pp;
        const pgd_status st =
            make_prefill_plan(num_seqs, total, num_q_heads, num_kv_heads, head_dim, &pp);
        if (st)
            return st;
        if (workspace_bytes)
            *workspace_bytes = pp.ws_bytes;
        return PGD_OK;
    });
}

pgd_status paged_kv_slots(int32_t *slots, int32_t *positions, int32_t *cu_seqlens_q,
                          int32_t *seq_lens, int32_t *free_end, int32_t *block_tables,
                          const int32_t *context_lens, const int32_t *query_lens,
                          const int32_t *free_pages, const int32_t *free_start, int num_seqs,
                          int num_rows, int num_free, int block_size, int max_blocks_per_seq,
                          int num_blocks, void *stream)
{
    return guarded([&]() -> pgd_status {
        return run_slots(slots, positions, cu_seqlens_q, seq_lens, free_end, block_tables,
                         context_lens, query_lens, free_pages, free_start, num_seqs, num_rows,
                         num_free, block_size, max_blocks_per_seq, num_blocks, stream);
    });
}

pgd_status paged_kv_write(uint16_t *k_cache, uint16_t *v_cache, const uint16_t *k_new,
                          const uint16_t *v_new, const int32_t *slots, int num_rows,
                          int num_kv_heads, int head_dim, int block_size, int num_blocks,
                          int64_t page_stride, int64_t head_stride, int64_t token_stride,
                          int64_t src_token_stride, int64_t src_head_stride, void *stream)
{
    return paged_kv_write_strided(k_cache, v_cache, k_new, v_new, slots, num_rows, num_kv_heads,
                                  head_dim, block_size, num_blocks, page_stride, head_stride,
                                  token_stride, src_token_stride, src_head_stride,
                                  src_token_stride, src_head_stride, stream);
}

pgd_status paged_kv_write_strided(uint16_t *k_cache, uint16_t *v_cache, const uint16_t *k_new,
                                  const uint16_t *v_new, const int32_t *slots, int num_rows,
                                  int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                  int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                  int64_t k_token_stride, int64_t k_head_stride,
                                  int64_t v_token_stride, int64_t v_head_stride, void *stream)
{
    return guarded([&]() -> pgd_status {
        return run_write(k_cache, v_cache, k_new, v_new, slots, num_rows, num_kv_heads, head_dim,
                         block_size, num_blocks, Strides{page_stride, head_stride, token_stride},
                         k_token_stride, k_head_stride, v_token_stride, v_head_stride, stream);
    });
}

pgd_status paged_rope_write(uint16_t *k_cache, uint16_t *v_cache, uint16_t *q_out,
                            const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                            const int32_t *slots, const int32_t *positions,
                            const float *inv_freq, float magnitude, int interleaved, int num_rows,
                            int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                            int block_size, int num_blocks, int64_t page_stride,
                            int64_t head_stride, int64_t token_stride, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, int64_t q_token_stride,
                            int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                            int64_t v_token_stride, int64_t v_head_stride, void *stream)
{
    return guarded([&]() -> pgd_status {
        if (num_rows < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0)
            return fail(PGD_ERR_INVALID_ARG,
                        "num_rows %d, num_q_heads %d, num_kv_heads %d, num_blocks %d", num_rows,
                        num_q_heads, num_kv_heads, num_blocks);
        if (!supported_head_dim(head_dim))
            return fail(PGD_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", head_dim);
        if (!supported_block_size(block_size))
            return fail(PGD_ERR_UNSUPPORTED, "block_size %d not in {8, 16, 32, 64, 128}",
                        block_size);
        if (num_q_heads > 65536 || num_kv_heads > 65536)
            return fail(PGD_ERR_UNSUPPORTED, "head counts %d / %d above 65536", num_q_heads,
                        num_kv_heads);
        if (rotary_dim <= 0 || rotary_dim % 16 != 0 || rotary_dim > head_dim)
            return fail(PGD_ERR_INVALID_ARG, "rotary_dim %d: a multiple of 16 up to head_dim %d",
                        rotary_dim, head_dim);
        pgd_status st;
        if ((st = check_strides(Strides{page_stride, head_stride, token_stride}, head_dim)) ||
            (st = check_row_strides({k_token_stride, k_head_stride, v_token_stride,
                                     v_head_stride})) ||
            (num_q_heads && (st = check_row_strides({q_out_token_stride, q_out_head_stride,
                                                     q_token_stride, q_head_stride}))))
            return st;
        RopeParams p = {};
        p.k_cache = k_cache;
        p.v_cache = v_cache;
        p.q_out = q_out;
        p.q = q;
        p.k_new = k_new;
        p.v_new = v_new;
        p.slots = slots;
        p.positions = positions;
        p.inv_freq = inv_freq;
        p.magnitude = magnitude;
        p.interleaved = interleaved != 0;
        p.rows = num_rows;
        p.Hq = num_q_heads;
        p.Hkv = num_kv_heads;
        p.rot = rotary_dim;
        p.log2BS = 3 + bs_index(block_size);
        p.NB = num_blocks;
        p.log2q = p.log2k = p.log2v = log2_of(head_dim / 16);
        p.page_stride = page_stride;
        p.head_stride = head_stride;
        p.token_stride = token_stride;
        p.qo_token = q_out_token_stride;
        p.qo_head = q_out_head_stride;
        p.q_token = q_token_stride;
        p.q_head = q_head_stride;
        p.k_token = k_token_stride;
        p.k_head = k_head_stride;
        p.v_token = v_token_stride;
        p.v_head = v_head_stride;
        return run_rope(p, stream);
    });
}

pgd_status pgd_rope_frequencies(float *inv_freq, float *magnitude, int rotary_dim, double base,
                                int scaling, double factor, double original_len, double beta_fast,
                                double beta_slow)
{
    return guarded([&]() -> pgd_status {
        return run_rope_frequencies(inv_freq, magnitude, rotary_dim, base, scaling, factor,
                                    original_len, beta_fast, beta_slow);
    });
}

pgd_status paged_latent_write(uint16_t *cache, uint16_t *q_out, const uint16_t *q_rope,
                              const uint16_t *latent, const uint16_t *k_rope,
                              const int32_t *slots, const int32_t *positions,
                              const float *inv_freq, float magnitude, int interleaved,
                              int num_rows, int num_heads, int latent_dim, int rope_dim,
                              int block_size, int num_blocks, int64_t page_stride,
                              int64_t token_stride, int64_t q_out_token_stride,
                              int64_t q_out_head_stride, int64_t q_token_stride,
                              int64_t q_head_stride, int64_t latent_token_stride,
                              int64_t k_rope_token_stride, void *stream)
{
    return guarded([&]() -> pgd_status {
        if (num_rows < 0 || num_heads < 0)
            return fail(PGD_ERR_INVALID_ARG, "num_rows %d, num_heads %d", num_rows, num_heads);
        if (num_heads > 65536)
            return fail(PGD_ERR_UNSUPPORTED, "num_heads %d above 65536", num_heads);
        pgd_status st;
        if ((st = check_latent_cache(latent_dim, rope_dim, block_size, num_blocks, page_stride,
                                     token_stride)) ||
            (st = check_row_strides({latent_token_stride, k_rope_token_stride})) ||
            (num_heads && (st = check_row_strides({q_out_token_stride, q_out_head_stride,
                                                   q_token_stride, q_head_stride}))))
            return st;
        // one head of keys, rope_dim wide, and one of "values", latent_dim wide
        RopeParams p = {};
        p.k_cache = cache ? cache + latent_dim : nullptr;
        p.v_cache = cache;
        p.q_out = q_out;
        p.q = q_rope;
        p.k_new = k_rope;
        p.v_new = latent;
        p.slots = slots;
        p.positions = positions;
        p.inv_freq = inv_freq;
        p.magnitude = magnitude;
        p.interleaved = interleaved != 0;
        p.rows = num_rows;
        p.Hq = num_heads;
        p.Hkv = 1;
        p.rot = rope_dim;
        p.log2BS = 3 + bs_index(block_size);
        p.NB = num_blocks;
        p.log2q = p.log2k = log2_of(rope_dim / 16);
        p.log2v = log2_of(latent_dim / 16);
        p.page_stride = page_stride;
        p.token_stride = token_stride;
        p.qo_token = q_out_token_stride;
        p.qo_head = q_out_head_stride;
        p.q_token = q_token_stride;
        p.q_head = q_head_stride;
        p.k_token = k_rope_token_stride;
        p.v_token = latent_token_stride;
        return run_rope(p, stream);
    });
}

pgd_status paged_latent_attention(void *out, int out_type, const uint16_t *q,
                                  const uint16_t *q_rope, const int32_t *cu_seqlens_q,
                                  const uint16_t *cache, const int32_t *block_tables,
                                  const int32_t *seq_lens, float scale, int num_seqs, int total_q,
                                  int max_q_len, int num_heads, int latent_dim, int rope_dim,
                                  int block_size, int max_blocks_per_seq, int num_blocks,
                                  int64_t page_stride, int64_t token_stride,
                                  int64_t q_token_stride, int64_t q_head_stride,
                                  int64_t q_rope_token_stride, int64_t q_rope_head_stride,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> pgd_status {
        if (out_type != PGD_OUT_F32 && out_type != PGD_OUT_F16)
            return fail(PGD_ERR_INVALID_ARG, "out_type %d: PGD_OUT_F32 or PGD_OUT_F16", out_type);
        return run_latent(out, out_type == PGD_OUT_F16, q, q_rope, cu_seqlens_q, cache,
                          block_tables, seq_lens, scale, num_seqs, total_q, max_q_len, num_heads,
                          latent_dim, rope_dim, block_size, max_blocks_per_seq, num_blocks,
                          {page_stride, token_stride, q_token_stride, q_head_stride,
                           q_rope_token_stride, q_rope_head_stride},
                          workspace, workspace_bytes, stream);
    });
}

pgd_status pgd_latent_plan(int num_seqs, int total_q, int max_q_len, int num_heads,
                           int latent_dim, int rope_dim, int block_size, int max_blocks_per_seq,
                           size_t *workspace_bytes)
{
    return guarded([&]() -> pgd_status {
        LatentPlan lp;
        const pgd_status st = make_latent_plan(num_seqs, total_q, max_q_len, num_heads, latent_dim,
                                               rope_dim, block_size, max_blocks_per_seq, &lp);
        if (st)
            return st;
        if (workspace_bytes)
            *workspace_bytes = lp.ws_bytes;
        return PGD_OK;
    });
}

pgd_status packed_latent_prefill(void *out, int out_type, const uint16_t *q, const uint16_t *k,
                                 const uint16_t *k_rope, const uint16_t *v,
                                 const int32_t *cu_seqlens, float scale, int num_seqs, int total,
                                 int max_len, int num_heads, int head_dim, int rope_dim,
                                 int64_t q_token_stride, int64_t q_head_stride,
                                 int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t k_rope_token_stride, int64_t v_token_stride,
                                 int64_t v_head_stride, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    return guarded([&]() -> pgd_status {
        if (out_type != PGD_OUT_F32 && out_type != PGD_OUT_F16)
            return fail(PGD_ERR_INVALID_ARG, "out_type %d: PGD_OUT_F32 or PGD_OUT_F16", out_type);
        const bool half = out_type == PGD_OUT_F16;
        return run_latent_prefill(half ? nullptr : static_cast<float *>(out),
                                  half ? static_cast<uint16_t *>(out) : nullptr, q, k, k_rope, v,
                                  cu_seqlens, scale, num_seqs, total, max_len, num_heads, head_dim,
                                  rope_dim,
                                  {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                                   k_rope_token_stride, v_token_stride, v_head_stride},
                                  workspace, workspace_bytes, stream);
    });
}

pgd_status pgd_latent_prefill_plan(int num_seqs, int total, int num_heads, int head_dim,
                                   int rope_dim, size_t *workspace_bytes)
{
    return guarded([&]() -> pgd_status {
        LatentPrefillPlan pp;
        const pgd_status st =
            make_latent_prefill_plan(num_seqs, total, num_heads, head_dim, rope_dim, &pp);
        if (st)
            return st;
        if (workspace_bytes)
            *workspace_bytes = pp.ws_bytes;
        return PGD_OK;
    });
}

pgd_status pgd_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                    int block_size, int partition_size, int max_blocks_per_seq,
                    int *chosen_partition_size, size_t *workspace_bytes)
{
    Plan plan;
    pgd_status st = make_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              partition_size, max_blocks_per_seq, &plan);
    if (st)
        return st;
    if (chosen_partition_size)
        *chosen_partition_size = plan.P;
    if (workspace_bytes)
        *workspace_bytes = plan.ws_bytes;
    return PGD_OK;
}

size_t pgd_workspace_size(int num_seqs, int num_q_heads, int head_dim, int block_size,
                          int partition_size, int max_blocks_per_seq)
{
    const size_t bad = ~(size_t)0;
    if (num_seqs < 0 || num_q_heads <= 0) {
        fail(PGD_ERR_INVALID_ARG, "num_seqs %d / num_q_heads %d", num_seqs, num_q_heads);
        return bad;
    }
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size)) {
        fail(PGD_ERR_UNSUPPORTED, "no kernel for head_dim %d, block_size %d", head_dim,
             block_size);
        return bad;
    }
    if (partition_size != 0 && partition_size != kPartitionSmall &&
        partition_size != kPartitionLarge) {
        fail(PGD_ERR_INVALID_ARG, "partition_size %d not in {0, 256, 512}", partition_size);
        return bad;
    }
    if (max_blocks_per_seq <= 0 || (long long)max_blocks_per_seq * block_size > (1ll << 30)) {
        fail(PGD_ERR_INVALID_ARG, "max_blocks_per_seq %d (length bound up to 2^30)",
             max_blocks_per_seq);
        return bad;
    }
    // partition_size 0: the scheduler picks 512 or 256 at call time; 256
    // needs at least as many partials, so its bytes cover either choice
    const int P = partition_size ? partition_size : kPartitionSmall;
    const long long maxlen = (long long)max_blocks_per_seq * block_size;
    const int NPmax = (int)((maxlen + P - 1) / P);
    size_t off_l, off_o;
    t_last_error.clear();
    return partials_bytes(num_seqs, num_q_heads, head_dim, NPmax, &off_l, &off_o);
}

pgd_status pgd_release(void)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(PGD_ERR_UNSUPPORTED, "device ordinal %d beyond %d", dev, kMaxDevices);
    // calls already queued on this device may still use the scratch and counters
    if ((e = cudaDeviceSynchronize()) != cudaSuccess)
        return cuda_fail(e, "device synchronize");
    DeviceState &ds = g_dev[dev];
    {
        std::lock_guard<std::mutex> lock(ds.pool_mu);
        if (ds.pool) {
            if ((e = cudaMemPoolTrimTo(ds.pool, 0)) != cudaSuccess ||
                (e = cudaMemPoolDestroy(ds.pool)) != cudaSuccess)
                return cuda_fail(e, "scratch pool release");
            ds.pool = nullptr;
        }
    }
    {
        CounterPool &cp = g_counters[dev];
        std::lock_guard<std::mutex> lock(cp.mu);
        if (cp.base) {
            if ((e = cudaFree(cp.base)) != cudaSuccess)
                return cuda_fail(e, "claim-counter release");
            cp.base = nullptr;
            cp.slot_of.clear();
            cp.dirty.clear();
        }
    }
    t_maps_used = t_maps_next = 0;
    t_last_error.clear();
    return PGD_OK;
}

int pgd_last_partition_size(void) { return t_last_partition; }

const char *pgd_last_error(void) { return t_last_error.c_str(); }

pgd_status pgd_test_stall_next_decode(const void *device_flag)
{
    if (device_flag && !aligned(device_flag, 4))
        return fail(PGD_ERR_INVALID_ARG, "stall flag not 4-byte aligned");
    t_stall_flag = static_cast<const unsigned *>(device_flag);
    t_last_error.clear();
    return PGD_OK;
}

pgd_status pgd_test_fail_next_reduce(int enable)
{
    t_skip_reduce = enable != 0;
    t_last_error.clear();
    return PGD_OK;
}

pgd_status pgd_test_fail_next_set_up(int enable)
{
    t_fail_set_up = enable != 0;
    t_last_error.clear();
    return PGD_OK;
}

pgd_status pgd_check_device_error(void *stream, unsigned *bits)
{
    DeviceState *ds;
    pgd_status st = device_state(&ds);
    if (st)
        return st;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "stream synchronize");
    unsigned v = 0, zero = 0;
    if ((e = cudaMemcpy(&v, ds->err_word, sizeof v, cudaMemcpyDeviceToHost)) != cudaSuccess ||
        (e = cudaMemcpy(ds->err_word, &zero, sizeof zero, cudaMemcpyHostToDevice)) !=
            cudaSuccess)
        return cuda_fail(e, "device error word");
    if (bits)
        *bits = v;
    if (v)
        return fail(PGD_ERR_DEVICE, "device-side checks flagged 0x%x", v);
    return PGD_OK;
}

pgd_status pgd_set_timing_events(void *before, void *after)
{
    if ((before == nullptr) != (after == nullptr))
        return fail(PGD_ERR_INVALID_ARG, "give both timing events or neither");
    t_ev_before = static_cast<cudaEvent_t>(before);
    t_ev_after = static_cast<cudaEvent_t>(after);
    return PGD_OK;
}

pgd_status pgd_device_info(int head_dim, int block_size, int *num_sms, int *ctas_per_sm)
{
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size))
        return fail(PGD_ERR_UNSUPPORTED, "no kernel for head_dim %d, block_size %d", head_dim,
                    block_size);
    DeviceState *ds;
    pgd_status st = device_state(&ds);
    if (st)
        return st;
    if (num_sms)
        *num_sms = ds->num_sms;
    if (ctas_per_sm)
        *ctas_per_sm = ds->ctas[0][d_index(head_dim)][bs_index(block_size)];
    return PGD_OK;
}

int pgd_version(void) { return 10600; }

}  // extern "C"
