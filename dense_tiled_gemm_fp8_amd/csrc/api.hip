/*
 * api.hip -- the C ABI of libgemm355 (declared in include/gemm355.h).
 *
 * A call validates and plans on the host (plans are cached per argument
 * shape), then enqueues on the caller's stream: optional operand repacks,
 * the main MFMA kernel over the plan's work units, and for split-K (or a
 * split tail of a persistent grid) the combine kernel.  Nothing here blocks
 * the host except the first use of a device (property query), the growth
 * of library-owned scratch, and waiting for another thread that is
 * enqueueing on the same stream with that stream's scratch.
 */
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <map>
#include <memory>
#include <mutex>
#include <thread>
#include <tuple>
#include <unordered_map>

#include "../../include/gemm355.h"
#include "block.h"
#include "kernels.h"
#include "plan.h"
#include "serve.h"
#include "tiles.h"

using namespace g355;

namespace {

std::mutex g_mu;

int32_t device_cus()
{
    static std::map<int, int32_t> cache;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = cache.find(dev);
    if (it != cache.end()) return it->second;
    hipDeviceProp_t prop;
    int32_t cus = 256;
    if (hipGetDeviceProperties(&prop, dev) == hipSuccess && prop.multiProcessorCount > 0)
        cus = prop.multiProcessorCount;
    cache[dev] = cus;
    return cus;
}

int32_t planning_cus(const gemm355_args &a)
{
    if (a.cus > 0) return a.cus;
    if (a.cus < 0) return -1;
    int n = 0;
    if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) {
        (void)hipGetLastError();
        return 256;
    }
    return device_cus();
}

/* Plan cache: the plan depends on the shape arguments, the knobs and the
 * 16-byte alignment of A and B, never on the data. */
struct PlanKey {
    int64_t v[32];
    bool operator==(const PlanKey &o) const { return memcmp(v, o.v, sizeof v) == 0; }
};
struct PlanKeyHash {
    size_t operator()(const PlanKey &k) const
    {
        uint64_t h = 1469598103934665603ull;
        for (int64_t x : k.v) {
            h ^= (uint64_t)x;
            h *= 1099511628211ull;
        }
        return (size_t)h;
    }
};
std::unordered_map<PlanKey, Plan, PlanKeyHash> g_plans;

PlanKey key_of(const gemm355_args &a, int32_t S, const ConvShape *conv)
{
    PlanKey k;
    memset(&k, 0, sizeof k);
    if (conv) {
        const int64_t *f = &conv->N;
        for (int i = 0; i < 14; ++i) k.v[16 + i] = f[i];
        k.v[30] = 1;
    }
    k.v[0] = a.M;
    k.v[1] = a.N;
    k.v[2] = a.K;
    k.v[3] = a.lda;
    k.v[4] = a.ldb;
    k.v[5] = a.ldc;
    k.v[6] = a.stride_a;
    k.v[7] = a.stride_b;
    k.v[8] = a.stride_c;
    k.v[9] = a.batch;
    k.v[10] = ((int64_t)a.dtype << 8) | (int64_t)a.layout;
    k.v[11] = ((int64_t)a.split_k << 32) | (uint32_t)(a.persistent + 1);
    k.v[12] = ((int64_t)a.tile << 32) | (uint32_t)S;
    k.v[13] = (int64_t)(((uintptr_t)a.A & 15u) | (((uintptr_t)a.B & 15u) << 4) |
                        (((uintptr_t)a.C & 15u) << 8) | (((uintptr_t)a.scale_a & 3u) << 12) |
                        (((uintptr_t)a.scale_b & 3u) << 14));
    /* null-ness matters for validation */
    k.v[14] = (a.A ? 1 : 0) | (a.B ? 2 : 0) | (a.C ? 4 : 0) | (a.block_scale_a ? 8 : 0) |
              (a.block_scale_b ? 16 : 0);
    return k;
}

gemm355_status get_plan(const gemm355_args &a, Plan &out, const ConvShape *conv = nullptr)
{
    const int32_t S = planning_cus(a);
    if (S < 1) return GEMM355_EINVAL;
    const PlanKey k = key_of(a, S, conv);
    {
        std::lock_guard<std::mutex> lk(g_mu);
        auto it = g_plans.find(k);
        if (it != g_plans.end()) {
            out = it->second;
            return check_pointers(a, conv);
        }
    }
    gemm355_status st = make_plan(a, S, out, conv);
    if (st != GEMM355_OK) return st;
    /* pointer overlap is not part of the key: check_pointers runs on hits */
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_plans.size() > 4096) g_plans.clear();
    g_plans.emplace(k, out);
    return GEMM355_OK;
}

/* Library-owned scratch, one buffer per (device, stream), grown on demand.
 *
 * A call that uses the buffer holds its lock from the lookup until its last
 * kernel is enqueued.  Calls on one stream therefore enqueue their kernels
 * as whole groups, never interleaved (one call's main pass cannot overwrite
 * partial sums another call's combine pass has yet to read), and the stream
 * runs the groups in enqueue order.  A buffer is replaced (after the stream
 * has drained the work of earlier calls) only by a call holding the lock,
 * so no call can be handed a buffer that is then freed under it.  The
 * per-thread default stream is one handle for many streams, so its buffers
 * are kept per thread as well. */
struct Scratch {
    std::mutex mu;
    void *ptr = nullptr;
    size_t bytes = 0;
};
struct ScratchKey {
    int dev;
    void *stream;
    std::thread::id thread;
    bool operator<(const ScratchKey &o) const
    {
        return std::tie(dev, stream, thread) < std::tie(o.dev, o.stream, o.thread);
    }
};
std::map<ScratchKey, std::unique_ptr<Scratch>> g_scratch;
/* largest library-owned buffer a call may hold (gemm355_set_scratch_limit) */
std::atomic<uint64_t> g_scratch_limit{UINT64_MAX};

gemm355_status library_scratch(size_t need, void *stream, void **out, std::unique_lock<std::mutex> &hold)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return GEMM355_EHIP;
    Scratch *s;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const ScratchKey key{dev, stream,
                             (hipStream_t)stream == hipStreamPerThread ? std::this_thread::get_id() : std::thread::id()};
        std::unique_ptr<Scratch> &slot = g_scratch[key];
        if (!slot) slot.reset(new Scratch);
        s = slot.get();
    }
    /* entries are never erased before unload, so s stays valid */
    hold = std::unique_lock<std::mutex>(s->mu);
    const uint64_t limit = g_scratch_limit.load();
    /* over the cap: refused like a failed allocation, before the buffer
     * that earlier calls may still read is touched */
    if (need > limit) return GEMM355_ENOMEM;
    if (s->bytes < need) {
        if (s->ptr) {
            /* earlier calls on this stream may still read the old buffer */
            if (hipStreamSynchronize((hipStream_t)stream) != hipSuccess) return GEMM355_EHIP;
            (void)hipFree(s->ptr);
            s->ptr = nullptr;
            s->bytes = 0;
        }
        size_t grow = need + need / 4;
        if (grow > limit) grow = (size_t)limit;
        if (hipMalloc(&s->ptr, grow) != hipSuccess) {
            (void)hipGetLastError();
            s->ptr = nullptr;
            return GEMM355_ENOMEM;
        }
        s->bytes = grow;
    }
    *out = s->ptr;
    return GEMM355_OK;
}

struct ScratchReaper {
    ~ScratchReaper()
    {
        for (auto &kv : g_scratch)
            if (kv.second && kv.second->ptr) (void)hipFree(kv.second->ptr);
    }
} g_reaper;

/* Scratch of gemm355_gemm_noalloc: a fixed array in every device's memory,
 * held from the library's load until the process ends.  Host code never
 * passes `scratch` itself to a kernel (on the host the name denotes a
 * stand-in, not a device address): the device address is looked up once
 * per device, with that device current, and kept per device. */
constexpr size_t kNoAllocScratchBytes = (size_t)64 << 20;
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];

struct NoAllocScratch {
    std::mutex mu;          /* held by a call until its last enqueue */
    void *ptr = nullptr;    /* the array's address on this device */
};
std::mutex g_noalloc_mu;
std::map<int, std::unique_ptr<NoAllocScratch>> g_noalloc;

gemm355_status noalloc_scratch(void **out, std::unique_lock<std::mutex> &hold)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return GEMM355_EHIP;
    }
    NoAllocScratch *s;
    {
        std::lock_guard<std::mutex> lk(g_noalloc_mu);
        std::unique_ptr<NoAllocScratch> &slot = g_noalloc[dev];
        if (!slot) {
            void *ptr = nullptr;
            if (hipGetSymbolAddress((void **)&ptr, HIP_SYMBOL(scratch)) != hipSuccess || ptr == nullptr) {
                (void)hipGetLastError();
                return GEMM355_EHIP;
            }
            slot.reset(new NoAllocScratch);
            slot->ptr = ptr;
        }
        s = slot.get();
    }
    /* calls from several threads on one stream enqueue call by call */
    hold = std::unique_lock<std::mutex>(s->mu);
    *out = s->ptr;
    return GEMM355_OK;
}

/* no_alloc: take scratch from the fixed per-device array instead of the
 * caller's workspace or library-owned memory (nothing is allocated). */
gemm355_status run(const gemm355_args &a, void *stream, const ConvShape *conv = nullptr, bool no_alloc = false)
{
    Plan P;
    gemm355_status st = get_plan(a, P, conv);
    if (st != GEMM355_OK) return st;
    if (a.M == 0 || a.N == 0) return GEMM355_OK;
    hipStream_t hs = (hipStream_t)stream;

    if (a.K == 0) {
        if (launch_zero(a.C, (int32_t)a.M, (int32_t)a.N, a.ldc, a.stride_c, (int32_t)a.batch,
                        P.out_esize, hs) != hipSuccess)
            return GEMM355_EHIP;
        return GEMM355_OK;
    }

    uint8_t *ws = nullptr;
    /* held until this call's last launch is enqueued (library scratch) */
    std::unique_lock<std::mutex> hold;
    if (P.pub.workspace_bytes) {
        if (no_alloc) {
            /* every kernel writes the scratch it later reads (partial slots,
             * repacked rows, regrouped scales), so nothing needs clearing */
            if (P.pub.workspace_bytes > kNoAllocScratchBytes) return GEMM355_ETOOBIG;
            void *p = nullptr;
            st = noalloc_scratch(&p, hold);
            if (st != GEMM355_OK) return st;
            ws = (uint8_t *)p;
        } else if (a.workspace) {
            if (a.workspace_bytes < P.pub.workspace_bytes) return GEMM355_ENOMEM;
            if (((uintptr_t)a.workspace & 255u) != 0) return GEMM355_EALIGN;
            ws = (uint8_t *)a.workspace;
        } else {
            void *p = nullptr;
            st = library_scratch(P.pub.workspace_bytes, stream, &p, hold);
            if (st != GEMM355_OK) return st;
            ws = (uint8_t *)p;
        }
    }

    const uint8_t *Aop = (const uint8_t *)a.A;
    const uint8_t *Bop = (const uint8_t *)a.B;
    const bool a_row = a.layout == GEMM355_A_ROW_B_COL || a.layout == GEMM355_A_ROW_B_ROW;
    const bool b_col = a.layout == GEMM355_A_ROW_B_COL || a.layout == GEMM355_A_COL_B_COL;
    PackParams pks[2];
    int npk = 0;
    if (P.pack_a) {
        PackParams &pk = pks[npk++];
        pk.src = a.A;
        pk.dst = ws + P.ws_pack_a_off;
        pk.ld = a.lda;
        pk.stride = a.stride_a;
        pk.ldd_bytes = P.lda_b;
        pk.dst_stride_bytes = P.stride_a_b;
        pk.rows = (int32_t)a.M;
        pk.K = (int32_t)a.K;
        pk.batch = (int32_t)a.batch;
        pk.esize = P.esize;
        pk.kmajor = a_row ? 1 : 0;
        Aop = pk.dst;
    }
    if (P.pack_b) {
        PackParams &pk = pks[npk++];
        pk.src = a.B;
        pk.dst = ws + P.ws_pack_b_off;
        pk.ld = a.ldb;
        pk.stride = a.stride_b;
        pk.ldd_bytes = P.ldb_b;
        pk.dst_stride_bytes = P.stride_b_b;
        pk.rows = (int32_t)a.N;
        pk.K = (int32_t)a.K;
        pk.batch = (int32_t)a.batch;
        pk.esize = P.esize;
        pk.kmajor = b_col ? 1 : 0;
        Bop = pk.dst;
    }
    if (npk && launch_pack(pks, npk, hs) != hipSuccess) return GEMM355_EHIP;

    GemmParams gp;
    gp.A = Aop;
    gp.B = Bop;
    gp.C = a.C;
    gp.ws = (float *)(ws ? ws + P.ws_partial_off : nullptr);
    gp.lda = P.lda_b;
    gp.ldb = P.ldb_b;
    gp.stride_a = P.stride_a_b;
    gp.stride_b = P.stride_b_b;
    gp.ldc = a.ldc;
    gp.stride_c = a.stride_c;
    gp.scale_a = a.scale_a;
    gp.scale_b = a.scale_b;
    gp.M = (int32_t)a.M;
    gp.N = (int32_t)a.N;
    gp.Kb = P.Kb;
    gp.Kv = P.Kv;
    gp.out_bf16 = P.out_esize == 2 ? 1 : 0;
    gp.c_vec = ((uintptr_t)a.C % 16 == 0) && (a.ldc * P.out_esize) % 16 == 0 &&
               (a.batch <= 1 || (a.stride_c * P.out_esize) % 16 == 0);
    gp.stamps = a.unit_stamps;
    gp.bsa = gp.bsb = nullptr;
    gp.ktp_a = a.M * 4;
    gp.ktp_b = a.N * 4;
    gp.stride_bsa = a.M * (a.K / 32);
    gp.stride_bsb = a.N * (a.K / 32);
    if (P.ws_scale_a_bytes) {
        /* regroup the block scales K-tile-major so that one direct-to-LDS
         * dword copy of 64 rows reads 256 contiguous bytes */
        ScalePackParams sp;
        sp.src = a.block_scale_a;
        sp.dst = (uint32_t *)(ws + P.ws_scale_a_off);
        sp.rows = (int32_t)a.M;
        sp.nK = (int32_t)(a.K / 128);
        sp.batch = (int32_t)a.batch;
        if (launch_pack_scales(sp, hs) != hipSuccess) return GEMM355_EHIP;
        gp.bsa = (const uint8_t *)sp.dst;
        sp.src = a.block_scale_b;
        sp.dst = (uint32_t *)(ws + P.ws_scale_b_off);
        sp.rows = (int32_t)a.N;
        if (launch_pack_scales(sp, hs) != hipSuccess) return GEMM355_EHIP;
        gp.bsb = (const uint8_t *)sp.dst;
    }
    gp.cv_H = gp.cv_W = gp.cv_C = gp.cv_S = gp.cv_P = gp.cv_Q = 0;
    gp.cv_ph = gp.cv_pw = gp.cv_sh = gp.cv_sw = gp.cv_dh = gp.cv_dw = 0;
    if (conv) {
        gp.cv_H = (int32_t)conv->H;
        gp.cv_W = (int32_t)conv->W;
        gp.cv_C = (int32_t)conv->C;
        gp.cv_S = (int32_t)conv->S;
        gp.cv_P = (int32_t)conv->P;
        gp.cv_Q = (int32_t)conv->Q;
        gp.cv_ph = (int32_t)conv->pad_h;
        gp.cv_pw = (int32_t)conv->pad_w;
        gp.cv_sh = (int32_t)conv->stride_h;
        gp.cv_sw = (int32_t)conv->stride_w;
        gp.cv_dh = (int32_t)conv->dil_h;
        gp.cv_dw = (int32_t)conv->dil_w;
    }
    gp.s = P.s;
    /* operand-format pair of an 8-bit product: 0 E4M3 x E4M3, 1 E5M2 x E5M2,
     * 2 E4M3 x E5M2 */
    const int32_t fmt = !(dtype_fp8(a.dtype) || dtype_fp6(a.dtype)) ? 0
                        : dtype_fmt_a(a.dtype) ? 1 : dtype_fmt_b(a.dtype) ? 2 : 0;
    if (P.s.grid > 0 && launch_gemm(P.pub.tile, fmt, gp, hs) != hipSuccess) return GEMM355_EHIP;

    if (P.reduce_tiles > 0) {
        ReduceParams rp;
        rp.ws = gp.ws;
        rp.C = a.C;
        rp.ldc = a.ldc;
        rp.stride_c = a.stride_c;
        rp.scale_a = a.scale_a;
        rp.scale_b = a.scale_b;
        rp.M = (int32_t)a.M;
        rp.N = (int32_t)a.N;
        rp.TM = P.pub.T_M;
        rp.TN = P.pub.T_N;
        rp.out_bf16 = gp.out_bf16;
        rp.tail = P.reduce_tail;
        rp.s = P.s;
        if (launch_reduce(rp, P.reduce_tiles, hs) != hipSuccess) return GEMM355_EHIP;
    }
    return GEMM355_OK;
}

/* A convolution's implicit product: validation, output size, the product's
 * arguments and the shape the main loop gathers A with. */
gemm355_status conv_setup(const gemm355_conv_args *c, gemm355_args &a, ConvShape &cs)
{
    if (!c) return GEMM355_EINVAL;
    if (c->N < 1 || c->H < 1 || c->W < 1 || c->C < 1 || c->K < 1 || c->R < 1 || c->S < 1) return GEMM355_EINVAL;
    if (c->stride_h < 1 || c->stride_w < 1 || c->dil_h < 1 || c->dil_w < 1 || c->pad_h < 0 || c->pad_w < 0)
        return GEMM355_EINVAL;
    const int64_t lim = (int64_t)1 << 30;
    if (c->N > lim || c->H > lim || c->W > lim || c->C > lim || c->K > lim || c->R > lim || c->S > lim ||
        c->pad_h > lim || c->pad_w > lim || c->stride_h > lim || c->stride_w > lim || c->dil_h > lim ||
        c->dil_w > lim)
        return GEMM355_EUNSUPPORTED;
    const int64_t ph = c->H + 2 * c->pad_h - c->dil_h * (c->R - 1) - 1;
    const int64_t pw = c->W + 2 * c->pad_w - c->dil_w * (c->S - 1) - 1;
    if (ph < 0 || pw < 0) return GEMM355_EINVAL;
    if ((int)c->dtype < 0 || (int)c->dtype >= kNumDtypes) return GEMM355_EINVAL;
    if (c->dtype != GEMM355_BF16_F32 && c->dtype != GEMM355_BF16_BF16) return GEMM355_EUNSUPPORTED;
    cs.N = c->N;
    cs.H = c->H;
    cs.W = c->W;
    cs.C = c->C;
    cs.R = c->R;
    cs.S = c->S;
    cs.P = ph / c->stride_h + 1;
    cs.Q = pw / c->stride_w + 1;
    cs.pad_h = c->pad_h;
    cs.pad_w = c->pad_w;
    cs.stride_h = c->stride_h;
    cs.stride_w = c->stride_w;
    cs.dil_h = c->dil_h;
    cs.dil_w = c->dil_w;
    if (cs.N * cs.P * cs.Q > lim || cs.R * cs.S * cs.C > lim) return GEMM355_EUNSUPPORTED;
    memset(&a, 0, sizeof a);
    a.M = cs.N * cs.P * cs.Q;
    a.N = c->K;
    a.K = cs.R * cs.S * cs.C;
    a.A = c->x;
    a.lda = a.K;
    a.B = c->w;
    a.ldb = a.K;
    a.C = c->y;
    a.ldc = c->K;
    a.batch = 1;
    a.dtype = c->dtype;
    a.layout = GEMM355_A_ROW_B_COL;
    a.split_k = c->split_k;
    a.persistent = c->persistent;
    a.tile = c->tile;
    a.cus = c->cus;
    a.workspace = c->workspace;
    a.workspace_bytes = c->workspace_bytes;
    return GEMM355_OK;
}

/* ---- serving operators: argument checks ---- */

const int64_t kMaxDim = (int64_t)1 << 30;
const int64_t kMaxWide = (int64_t)1 << 23;
const int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;

/* Extent in bytes of `rows` rows of `cols` elements, ld elements apart.  Rows of
 * one pitch that lie beside each other, as columns of one buffer, do not meet. */
struct Span {
    uintptr_t lo, hi;
    uint64_t pitch, width;        /* of several rows; 0: one run of bytes     */
    Span(const void *ptr, uint64_t bytes) : lo((uintptr_t)ptr), hi((uintptr_t)ptr + (ptr ? bytes : 0)), pitch(0), width(0) {}
    Span(const void *ptr, int64_t rows, int64_t cols, int64_t ld, int64_t es)
        : Span(ptr, rows > 0 && cols > 0 ? ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * (uint64_t)es : 0)
    {
        if (rows > 1) {
            pitch = (uint64_t)(ld * es);
            width = (uint64_t)(cols * es);
        }
    }
    bool meets(const Span &o) const
    {
        if (!(lo < o.hi && o.lo < hi && lo < hi && o.lo < o.hi)) return false;
        if (!pitch || pitch != o.pitch) return true;
        /* where the other's rows begin, counted from the beginnings of these */
        const uint64_t at = o.lo >= lo ? (o.lo - lo) % pitch : (pitch - (lo - o.lo) % pitch) % pitch;
        return at < width || at + o.width > pitch;
    }
};

bool aligned(const void *ptr, uintptr_t to) { return ((uintptr_t)ptr & (to - 1)) == 0; }

gemm355_status check_w4(const gemm355_w4_matrix *q, W4Params &w)
{
    if (!q || q->N < 0 || q->K < 0) return GEMM355_EINVAL;
    if (q->fmt != GEMM355_W4_INT && q->fmt != GEMM355_W4_MXFP4) return GEMM355_EINVAL;
    const bool mx = q->fmt == GEMM355_W4_MXFP4;
    if (mx ? q->group != 32 : q->group != 32 && q->group != 64 && q->group != 128) return GEMM355_EINVAL;
    if (mx && q->zeros) return GEMM355_EINVAL;
    if (q->N > kMaxDim || q->K > kMaxDim || q->N * q->K > ((int64_t)1 << 40)) return GEMM355_EUNSUPPORTED;
    const int64_t ldw = q->ldw ? q->ldw : (q->K + 31) / 32 * 32;
    if (ldw < q->K || ldw % 32 != 0) return GEMM355_EINVAL;
    if (ldw > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (q->N > 0 && q->K > 0 && (!q->codes || !q->scales)) return GEMM355_EINVAL;
    if (!aligned(q->codes, 16) || (!mx && !aligned(q->scales, 2))) return GEMM355_EALIGN;
    w.codes = q->codes;
    w.ldb = ldw / 2;
    w.scales = q->scales;
    w.zeros = q->zeros;
    w.N = (int32_t)q->N;
    w.K = (int32_t)q->K;
    w.group = q->group;
    w.ng = (int32_t)((q->K + q->group - 1) / q->group);
    w.mx = mx ? 1 : 0;
    return GEMM355_OK;
}

/* Whether any part of the matrix lies in s. */
bool w4_meets(const W4Params &w, const Span &s)
{
    const int64_t groups = (int64_t)w.N * w.ng;
    return s.meets(Span(w.codes, w.N, ((int64_t)w.K + 31) / 32 * 16, w.ldb, 1)) ||
           s.meets(Span(w.scales, (uint64_t)groups * (w.mx ? 1 : 2))) || s.meets(Span(w.zeros, (uint64_t)groups));
}

gemm355_status w4_convert(const gemm355_w4_matrix *q, const void *dense, int64_t ld, gemm355_src type, W4QuantParams &p)
{
    gemm355_status st = check_w4(q, p.w);
    if (st != GEMM355_OK) return st;
    if (type != GEMM355_SRC_F32 && type != GEMM355_SRC_BF16) return GEMM355_EINVAL;
    const int64_t es = type == GEMM355_SRC_F32 ? 4 : 2;
    p.ld = ld ? ld : q->K;
    if (p.ld < q->K) return GEMM355_EINVAL;
    if (p.ld > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (q->N > 0 && q->K > 0 && !dense) return GEMM355_EINVAL;
    if (!aligned(dense, (uintptr_t)es)) return GEMM355_EALIGN;
    if (w4_meets(p.w, Span(dense, q->N, q->K, p.ld, es))) return GEMM355_EINVAL;
    p.x = dense;
    p.y = const_cast<void *>(dense);
    p.f32 = es == 4 ? 1 : 0;
    p.vec = aligned(dense, 16) && p.ld * es % 16 == 0 ? 1 : 0;
    return GEMM355_OK;
}

gemm355_status check_kv(const gemm355_kv_cache &c, KvParams &k)
{
    if (c.pages < 1 || c.heads < 1 || c.batch < 0 || c.tokens < 0 || c.max_new < 1 || c.max_len < 0 || c.table_ld < 0)
        return GEMM355_EINVAL;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return GEMM355_EUNSUPPORTED;
    if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) return GEMM355_EUNSUPPORTED;
    if (c.pages > 0x7FFFFFFF || c.tokens > kMaxDim || c.max_new > kMaxDim || c.max_len > kMaxDim || c.table_ld > kMaxDim ||
        c.batch > 65528 || c.batch * c.heads > 65528)
        return GEMM355_EUNSUPPORTED;
    const int64_t ld = c.table_ld ? c.table_ld : (c.max_len + c.page - 1) / c.page;
    if (c.max_len > ld * c.page) return GEMM355_EINVAL;
    if (!c.q_start && c.tokens != c.batch * c.max_new) return GEMM355_EINVAL;
    if (!c.k || !c.v || !c.k_scale || !c.v_scale) return GEMM355_EINVAL;
    if (c.batch > 0 && ((!c.table && c.max_len > 0) || !c.lens)) return GEMM355_EINVAL;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.table, 4) || !aligned(c.lens, 4) || !aligned(c.q_start, 4))
        return GEMM355_EALIGN;
    k.k = c.k;
    k.v = c.v;
    k.k_scale = c.k_scale;
    k.v_scale = c.v_scale;
    k.table = c.table;
    k.lens = c.lens;
    k.q_start = c.q_start;
    k.pages = c.pages;
    k.table_ld = ld;
    k.H = c.heads;
    k.page = c.page;
    k.page_log2 = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
    k.B = (int32_t)c.batch;
    k.tokens = (int32_t)c.tokens;
    /* no sequence has more new rows than the step has */
    k.max_new = (int32_t)std::min(c.max_new, std::max<int64_t>(c.tokens, 1));
    k.max_len = (int32_t)c.max_len;
    return GEMM355_OK;
}

/* Whether any buffer of the cache, or of the step's indices, lies in s. */
bool kv_meets(const gemm355_kv_cache &c, const Span &s, bool indices)
{
    const uint64_t blocks = (uint64_t)c.pages * (uint64_t)c.heads, bytes = blocks * (uint64_t)c.page * (uint64_t)c.head_dim;
    if (s.meets(Span(c.k, bytes)) || s.meets(Span(c.v, bytes)) || s.meets(Span(c.k_scale, blocks)) || s.meets(Span(c.v_scale, blocks)))
        return true;
    const int64_t ld = c.table_ld ? c.table_ld : (c.max_len + c.page - 1) / c.page;
    return indices && (s.meets(Span(c.table, (uint64_t)(c.batch * ld * 4))) || s.meets(Span(c.lens, (uint64_t)c.batch * 4)) ||
                       s.meets(Span(c.q_start, (uint64_t)(c.batch + 1) * 4)));
}

/* A step's bf16 rows of `heads` heads. */
gemm355_status check_rows(const void *ptr, int64_t &ld, int64_t tokens, int64_t heads, int32_t dim)
{
    const int64_t width = heads * dim;
    if (!ld) ld = width;
    if (heads < 1 || ld < width || ld % 8 != 0) return GEMM355_EINVAL;
    if (width > kMaxDim || ld > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (tokens > 0 && !ptr) return GEMM355_EINVAL;
    return aligned(ptr, 16) ? GEMM355_OK : GEMM355_EALIGN;
}

gemm355_status append_setup(const gemm355_kv_append_args *a, KvAppendParams &p)
{
    if (!a) return GEMM355_EINVAL;
    const gemm355_kv_cache &c = a->cache;
    gemm355_status st = check_kv(c, p.c);
    if (st != GEMM355_OK) return st;
    p.ldk = a->ldk;
    p.ldv = a->ldv;
    p.ldq = a->ldq;
    p.ldqo = a->ldqo;
    if ((st = check_rows(a->k, p.ldk, c.tokens, c.heads, c.head_dim)) != GEMM355_OK) return st;
    if ((st = check_rows(a->v, p.ldv, c.tokens, c.heads, c.head_dim)) != GEMM355_OK) return st;
    if ((a->q == nullptr) != (a->q_out == nullptr)) return GEMM355_EINVAL;
    if (a->q) {
        if ((st = check_rows(a->q, p.ldq, c.tokens, a->q_heads, c.head_dim)) != GEMM355_OK) return st;
        if ((st = check_rows(a->q_out, p.ldqo, c.tokens, a->q_heads, c.head_dim)) != GEMM355_OK) return st;
    }
    if (a->rot_dim < 0 || a->rot_dim > c.head_dim || a->rot_dim % 2 != 0) return GEMM355_EINVAL;
    if (a->rot_dim) {
        if (a->rot_len < c.max_len || (c.max_len > 0 && (!a->cos || !a->sin))) return GEMM355_EINVAL;
        if (!aligned(a->cos, 4) || !aligned(a->sin, 4)) return GEMM355_EALIGN;
    }
    const int64_t kw = (int64_t)c.heads * c.head_dim, qw = (int64_t)a->q_heads * c.head_dim;
    const Span k(a->k, c.tokens, kw, p.ldk, 2), v(a->v, c.tokens, kw, p.ldv, 2), q(a->q, c.tokens, qw, p.ldq, 2);
    const Span out(a->q_out, c.tokens, qw, p.ldqo, 2);
    const uint64_t table = a->rot_dim ? (uint64_t)c.max_len * (uint64_t)(a->rot_dim / 2) * 4 : 0;
    const Span cs(a->cos, table), sn(a->sin, table);
    const int64_t ld = p.c.table_ld;
    const Span idx[3] = {Span(c.table, (uint64_t)(c.batch * ld * 4)), Span(c.lens, (uint64_t)c.batch * 4),
                         Span(c.q_start, (uint64_t)(c.batch + 1) * 4)};
    if (out.meets(k) || out.meets(v) || out.meets(q) || out.meets(cs) || out.meets(sn) || kv_meets(c, out, true)) return GEMM355_EINVAL;
    if (kv_meets(c, k, false) || kv_meets(c, v, false) || kv_meets(c, q, false) || kv_meets(c, cs, false) || kv_meets(c, sn, false) ||
        kv_meets(c, idx[0], false) || kv_meets(c, idx[1], false) || kv_meets(c, idx[2], false))
        return GEMM355_EINVAL;
    /* a grid holds under 2^32 threads a dimension */
    const int64_t kv_units = (((int64_t)p.c.max_new + c.page - 2) / c.page + 1) * c.heads * 2;
    const int64_t q_blocks = a->q ? ((int64_t)p.c.max_new * a->q_heads * (c.head_dim / 8) + 255) / 256 : 0;
    if (kv_units > kMaxBlocks || q_blocks > kMaxBlocks - kv_units) return GEMM355_EUNSUPPORTED;
    p.xk = (const uint16_t *)a->k;
    p.xv = (const uint16_t *)a->v;
    p.q = (const uint16_t *)a->q;
    p.q_out = (uint16_t *)a->q_out;
    p.cos = a->cos;
    p.sin = a->sin;
    p.Hq = a->q_heads;
    p.D = c.head_dim;
    p.rot = a->rot_dim;
    p.interleaved = a->interleaved ? 1 : 0;
    p.whole = a->rot_dim % 16 == 0 && aligned(a->cos, 16) && aligned(a->sin, 16) ? 1 : 0;
    return GEMM355_OK;
}

/* Compute units of the current device, 256 without one. */
int32_t present_cus()
{
    int n = 0;
    if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) {
        (void)hipGetLastError();
        return 256;
    }
    return device_cus();
}

/* Checks, the split of the key axis and the scratch of an attention call. */
gemm355_status attention_setup(const gemm355_attention_args *a, AttnParams &p, size_t &bytes)
{
    if (!a) return GEMM355_EINVAL;
    const gemm355_kv_cache &c = a->cache;
    gemm355_status st = check_kv(c, p.c);
    if (st != GEMM355_OK) return st;
    if (a->q_heads < 1 || a->q_heads % c.heads != 0 || a->window < 0 || a->sinks < 0 || a->splits < 0) return GEMM355_EINVAL;
    /* scale * log2(e) stays finite */
    if (!(a->scale >= 0.0f) || !(a->scale <= 0x1p127f)) return GEMM355_EINVAL;
    p.ldq = a->ldq;
    p.ldo = a->ldo;
    if ((st = check_rows(a->q, p.ldq, c.tokens, a->q_heads, c.head_dim)) != GEMM355_OK) return st;
    if ((st = check_rows(a->o, p.ldo, c.tokens, a->q_heads, c.head_dim)) != GEMM355_OK) return st;
    if (!aligned(a->lse, 4)) return GEMM355_EALIGN;
    const int64_t qw = (int64_t)a->q_heads * c.head_dim;
    const Span q(a->q, c.tokens, qw, p.ldq, 2), o(a->o, c.tokens, qw, p.ldo, 2), lse(a->lse, (uint64_t)(c.tokens * a->q_heads * 4));
    if (o.meets(q) || o.meets(lse) || lse.meets(q) || kv_meets(c, o, true) || kv_meets(c, lse, true)) return GEMM355_EINVAL;
    p.q = (const uint16_t *)a->q;
    p.o = (uint16_t *)a->o;
    p.lse = a->lse;
    p.scale_log2 = (float)((a->scale > 0.0f ? (double)a->scale : 1.0 / sqrt((double)c.head_dim)) * 1.4426950408889634);
    p.Hq = a->q_heads;
    p.group = a->q_heads / c.heads;
    p.by_group = divider(p.group);
    p.D = c.head_dim;
    p.window = a->window >= c.max_len ? 0 : (int32_t)a->window;
    p.sinks = (int32_t)std::min<int64_t>(a->sinks, c.max_len);
    const int64_t rows = (int64_t)p.c.max_new * p.group;
    if (rows > (int64_t)16 * 65535) return GEMM355_EUNSUPPORTED;
    const int32_t cus = present_cus();
    /* Rows a workgroup: 16 while that makes no more workgroups than compute
     * units (heads of 256, whose 32 rows fill the registers: two a unit), else
     * 32, for which a chunk's codes are converted once; us with 16 and 32:
     *   heads of 64:   128 tokens of 4 x 4 heads, 2000 held 12.0, 18.9;
     *                  500 held, 2 x 160 of 8 x 4  11.4, 9.8
     *   heads of 128:  16.6, 27.5;  16.7, 14.8;  4 x 512 of 4 x 4 with a window
     *                  of 2048  96, 62
     *   heads of 256:  300 tokens of 8 x 1 13.0, 20.3;  500 held, 2 x 160 of
     *                  8 x 4  32.3, 26.5 */
    const int64_t pairs = c.batch * c.heads;
    p.tile_rows = rows <= 16 || pairs * ((rows + 15) / 16) <= (p.D == 256 ? 2 : 1) * cus ? 16 : 32;
    p.row_tiles = (int32_t)((rows + p.tile_rows - 1) / p.tile_rows);
    const int64_t tiles = std::max<int64_t>(1, pairs * p.row_tiles);
    int64_t seen = c.max_len;
    if (p.window) seen = std::min(seen, (int64_t)p.window + p.c.max_new + p.sinks + 128);
    /* Wavefronts a workgroup of 16 rows: as many as fill a compute unit's LDS
     * where there are at most as many workgroups as units, half of them (so that
     * two workgroups share a unit) where there are more: heads of 128, 8 against
     * 4 wavefronts, us: 8 x 2000 tokens 15.0, 16.3; 64 x 128 tokens 13.9, 9.4;
     * 64 x 500 19.6, 16.0; but 64 x 3000 62.2, 61.5 and 64 x 8192 148.1, 153.4.
     * Heads of 64 leave room for two either way.
     * Of 32 rows, 4 up to three workgroups a unit (heads of 128, of which two
     * fit: two and a half), else 2.  us with 4 and 2, heads of 128: 384 new of 8 x
     * 4 heads, 2000 held 31.1, 47.7; 2 x 300, 3000 held 60.7, 66.8; 700 new, 2000
     * held 50.1, 46.8; 4 x 512 with a window 70, 62; heads of 64: 700 new, 2000
     * held 24.9, 31.8; 2 x 512, 700 held 18.7, 17.0. */
    if (p.tile_rows == 32)
        p.waves = p.D < 256 && 2 * tiles <= (p.D == 64 ? 6 : 5) * (int64_t)cus ? 4 : 2;
    else
        p.waves = (p.D == 256 ? 4 : 8) / (p.D == 64 || tiles <= cus || seen > 4096 ? 1 : 2);
    /* Parts: as many as stay within one pass of workgroups over the device (18 x
     * 3000 tokens of 8 heads of 128: one part 21.7 us, two, of which the second
     * begins when the first is done, 31.8), and two chunks or more a wavefront,
     * as each part costs its share of a second kernel (one sequence, heads of
     * 128: 8000 tokens 16.1 us so, 20.7 with four chunks or more; heads of 256:
     * 19.8 us, 24.6 with four chunks a wavefront). */
    p.part_chunks = a->splits ? 4 : p.tile_rows == 32 ? 16 : 2 * p.waves;
    const int64_t most = std::max<int64_t>(1, (seen + 64 * p.part_chunks - 1) / (64 * p.part_chunks));
    const int64_t want = a->splits ? a->splits : std::max<int64_t>(1, (p.D == 64 ? 2 : 1) * (int64_t)cus / tiles);
    p.splits = (int32_t)std::min(want, most);
    const int64_t slots = tiles * p.splits;
    if (p.splits > 1 && slots > ((int64_t)1 << 31)) return GEMM355_EUNSUPPORTED;   /* bytes stay in 64 bits */
    bytes = p.splits > 1 ? (size_t)slots * (size_t)p.tile_rows * (size_t)(p.D + 2) * sizeof(float) : 0;
    p.part = p.stat = nullptr;
    return GEMM355_OK;
}

/* Whether work enqueued on the stream goes into a graph. */
bool capturing(void *stream)
{
    if (!stream) return false;
    hipStreamCaptureStatus state = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing((hipStream_t)stream, &state) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return state != hipStreamCaptureStatusNone;
}

/* ---- block-scaled operators: argument checks ---- */

/* 256 rows of a tile stay within the 32-bit offsets of its copies */
const int64_t kMaxRow = (int64_t)1 << 22;

gemm355_status check_block(const gemm355_block_matrix &q, BlockMat &b)
{
    if (q.rows < 0 || q.K < 0 || (q.block_rows != 1 && q.block_rows != 128)) return GEMM355_EINVAL;
    if (q.rows > ((int64_t)1 << 26) || q.K > kMaxRow) return GEMM355_EUNSUPPORTED;
    const int64_t nk = (q.K + 127) / 128, least = q.block_rows == 1 ? q.rows : nk;
    b.ld = q.ld ? q.ld : (q.K + 15) / 16 * 16;
    b.lds = q.ld_scale ? q.ld_scale : least;
    if (b.ld < q.K || b.ld % 16 != 0 || b.lds < least) return GEMM355_EINVAL;
    if (b.ld > kMaxRow || b.lds > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (q.rows > 0 && q.K > 0 && (!q.codes || !q.scales)) return GEMM355_EINVAL;
    if (!aligned(q.codes, 16) || !aligned(q.scales, 4)) return GEMM355_EALIGN;
    b.codes = q.codes;
    b.scales = q.scales;
    return GEMM355_OK;
}

Span block_codes(const gemm355_block_matrix &q, const BlockMat &b) { return Span(b.codes, q.rows, (q.K + 15) / 16 * 16, b.ld, 1); }

Span block_scales(const gemm355_block_matrix &q, const BlockMat &b)
{
    const int64_t nk = (q.K + 127) / 128;
    return q.block_rows == 1 ? Span(b.scales, nk, q.rows, b.lds, 4) : Span(b.scales, (q.rows + 127) / 128, nk, b.lds, 4);
}

bool block_meets(const gemm355_block_matrix &q, const BlockMat &b, const Span &s)
{
    return s.meets(block_codes(q, b)) || s.meets(block_scales(q, b));
}

bool known(gemm355_src t) { return t == GEMM355_SRC_F32 || t == GEMM355_SRC_BF16; }

/* Rows of one type in device memory: extent, and what may be written in place. */
struct Rows {
    const void *ptr;
    int64_t ld, es;
    Span span;
    Rows(const void *p, int64_t rows, int64_t cols, int64_t pitch, gemm355_src type)
        : ptr(p), ld(pitch ? pitch : cols), es(type == GEMM355_SRC_F32 ? 4 : 2), span(p, rows, cols, ld, es)
    {
    }
    bool same(const Rows &o) const { return ptr == o.ptr && ld == o.ld && es == o.es; }
};

gemm355_status norm_setup(const gemm355_rmsnorm_args *a, NormParams &p)
{
    if (!a || a->rows < 0 || a->width < 0) return GEMM355_EINVAL;
    if (!known(a->x_type) || !known(a->r_type) || !known(a->w_type) || !known(a->y_type)) return GEMM355_EINVAL;
    if (!(a->eps > 0.0f) || !(a->eps < INFINITY)) return GEMM355_EINVAL;
    /* a workgroup of 1024 threads a row, fewer than 2^32 of them */
    if (a->rows >= ((int64_t)1 << 22) || a->width > ((int64_t)1 << 15)) return GEMM355_EUNSUPPORTED;
    const int64_t n = a->rows, k = a->width;
    const Rows x(a->x, n, k, a->ldx, a->x_type), r(a->residual, n, k, a->ldr, a->r_type), h(a->sum, n, k, a->lds, a->r_type),
        y(a->y, n, k, a->ldy, a->y_type);
    const Span w(a->weight, (uint64_t)k * (a->w_type == GEMM355_SRC_F32 ? 4 : 2));
    for (const Rows *t : {&x, &r, &h, &y}) {
        if (t->ld < k) return GEMM355_EINVAL;
        if (t->ld > kMaxDim) return GEMM355_EUNSUPPORTED;
        if (!aligned(t->ptr, (uintptr_t)t->es)) return GEMM355_EALIGN;
    }
    if (!aligned(a->weight, a->w_type == GEMM355_SRC_F32 ? 4 : 2)) return GEMM355_EALIGN;
    p.q = BlockMat{};
    if (a->q) {
        if (a->q->rows != n || a->q->K != k || a->q->block_rows != 1) return GEMM355_EINVAL;
        const gemm355_status st = check_block(*a->q, p.q);
        if (st != GEMM355_OK) return st;
    }
    if (n == 0 || k == 0) return GEMM355_OK;
    if (!a->x || (a->sum && !a->residual) || (!a->y && !a->q)) return GEMM355_EINVAL;
    for (const Rows *in : {&x, &r}) {
        if (h.span.meets(in->span) && !h.same(*in)) return GEMM355_EINVAL;
        if (y.span.meets(in->span) && !y.same(*in)) return GEMM355_EINVAL;
    }
    if (h.span.meets(y.span) || h.span.meets(w) || y.span.meets(w)) return GEMM355_EINVAL;
    if (a->q) {
        for (const Span *s : {&x.span, &r.span, &h.span, &y.span, &w})
            if (block_meets(*a->q, p.q, *s)) return GEMM355_EINVAL;
        if (block_codes(*a->q, p.q).meets(block_scales(*a->q, p.q))) return GEMM355_EINVAL;
    }
    p.x = a->x;
    p.residual = a->residual;
    p.weight = a->weight;
    p.sum = a->sum;
    p.y = a->y;
    p.ldx = x.ld;
    p.ldr = r.ld;
    p.lds = h.ld;
    p.ldy = y.ld;
    p.rows = (int32_t)n;
    p.width = (int32_t)k;
    p.x_f32 = x.es == 4;
    p.r_f32 = r.es == 4;
    p.w_f32 = a->w_type == GEMM355_SRC_F32;
    p.y_f32 = y.es == 4;
    p.eps = a->eps;
    return GEMM355_OK;
}

/* Of the two kinds of products; up and q null for one. */
struct BlockCall {
    const gemm355_block_matrix *x, *w, *up, *q;
    void *y;
    int64_t ldy;
    gemm355_src out;
    int32_t splits;
    void *workspace;
    size_t workspace_bytes;
};

BlockCall block_call(const gemm355_block_gemm_args &a)
{
    return BlockCall{&a.x, &a.w, nullptr, nullptr, a.y, a.ldy, a.out, a.splits, a.workspace, a.workspace_bytes};
}

BlockCall block_call(const gemm355_block_gated_args &a)
{
    return BlockCall{&a.x, &a.gate, &a.up, &a.q, a.y, a.ldy, a.out, a.splits, a.workspace, a.workspace_bytes};
}

/* Checks, plan and scratch of a product.  Of a call with nothing to do p.M or p.N
 * is 0. */
gemm355_status block_setup(const BlockCall &c, BlockGemmParams &p, size_t &bytes)
{
    BlockMat x, w, up{};
    gemm355_status st = check_block(*c.x, x);
    if (st != GEMM355_OK || (st = check_block(*c.w, w)) != GEMM355_OK) return st;
    if (c.up && (st = check_block(*c.up, up)) != GEMM355_OK) return st;
    const int64_t M = c.x->rows, N = c.w->rows, K = c.x->K;
    if (c.x->block_rows != 1 || c.w->block_rows != 128 || c.w->K != K) return GEMM355_EINVAL;
    if (c.up && (c.up->block_rows != 128 || c.up->K != K || c.up->rows != N)) return GEMM355_EINVAL;
    if (!known(c.out) || c.splits < 0) return GEMM355_EINVAL;
    if (M > ((int64_t)1 << 21)) return GEMM355_EUNSUPPORTED;
    const bool codes = c.q && c.q->codes;
    p.q = BlockMat{};
    if (codes) {
        if (c.q->rows != M || c.q->K != N || c.q->block_rows != 1) return GEMM355_EINVAL;
        if ((st = check_block(*c.q, p.q)) != GEMM355_OK) return st;
    }
    const Rows y(c.y, M, N, c.ldy, c.out);
    if (y.ld < N) return GEMM355_EINVAL;
    if (y.ld > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (!aligned(c.y, (uintptr_t)y.es)) return GEMM355_EALIGN;
    bytes = 0;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    if (M == 0 || N == 0) return GEMM355_OK;
    if (c.up ? codes == (c.y != nullptr) : !c.y) return GEMM355_EINVAL;
    auto meets = [&](const Span &s) {
        return block_meets(*c.x, x, s) || block_meets(*c.w, w, s) || (c.up && block_meets(*c.up, up, s));
    };
    if (meets(y.span)) return GEMM355_EINVAL;
    if (codes && (meets(block_codes(*c.q, p.q)) || meets(block_scales(*c.q, p.q)) ||
                  block_codes(*c.q, p.q).meets(block_scales(*c.q, p.q))))
        return GEMM355_EINVAL;
    p.x = x.codes;
    p.w = w.codes;
    p.up = up.codes;
    p.xs = x.scales;
    p.ws = w.scales;
    p.us = up.scales;
    p.ldx = x.ld;
    p.ldw = w.ld;
    p.ldu = up.ld;
    p.lxs = x.lds;
    p.lws = w.lds;
    p.lus = up.lds;
    p.K = (int32_t)K;
    p.nk = (int32_t)((K + 127) / 128);
    p.two = c.up != nullptr;
    p.act = 0;
    p.y = c.y;
    p.ldy = y.ld;
    p.y_f32 = y.es == 4;
    const int64_t groups = block_plan(p, c.splits, present_cus());
    if (groups > kMaxBlocks) return GEMM355_EUNSUPPORTED;
    const double need = (double)p.part_planes * p.splits * (double)M * (double)p.ldp * 4.0;
    if (need > 0x1p40) return GEMM355_EUNSUPPORTED;
    bytes = (size_t)p.part_planes * (size_t)p.splits * (size_t)M * (size_t)p.ldp * sizeof(float);
    if (bytes && c.workspace) {
        const Span s(c.workspace, (uint64_t)bytes);
        if (meets(s) || s.meets(y.span) || (codes && block_meets(*c.q, p.q, s))) return GEMM355_EINVAL;
    }
    return GEMM355_OK;
}

template <class Args>
gemm355_status block_scratch(const Args *args, size_t *bytes)
{
    if (!args || !bytes) return GEMM355_EINVAL;
    try {
        BlockGemmParams p;
        size_t need = 0;
        const gemm355_status st = block_setup(block_call(*args), p, need);
        if (st != GEMM355_OK) return st;
        *bytes = need;
        return GEMM355_OK;
    } catch (...) {
        return GEMM355_ENOMEM;
    }
}

gemm355_status block_run(const BlockCall &c, int32_t act, void *stream)
{
    try {
        BlockGemmParams p;
        size_t need = 0;
        gemm355_status st = block_setup(c, p, need);
        if (st != GEMM355_OK || p.M == 0 || p.N == 0) return st;
        p.act = act;
        void *ws = nullptr;
        std::unique_lock<std::mutex> hold;
        if (need && c.workspace) {
            if (c.workspace_bytes < need) return GEMM355_ENOMEM;
            if (!aligned(c.workspace, 256)) return GEMM355_EALIGN;
            ws = c.workspace;
        } else if (need) {
            if (capturing(stream)) return GEMM355_ENOMEM;
            st = library_scratch(need, stream, &ws, hold);
            if (st != GEMM355_OK) return st;
        }
        p.part = (float *)ws;
        return launch_block_gemm(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
    } catch (...) {
        return GEMM355_ENOMEM;   /* the maps of scratch buffers could not grow */
    }
}

} /* namespace */

extern "C" {

gemm355_status gemm355_block_quantize(const void *x, int64_t ld, gemm355_src src, const gemm355_block_matrix *q, void *stream)
{
    if (!q || !known(src)) return GEMM355_EINVAL;
    BlockQuantParams p;
    const gemm355_status st = check_block(*q, p.q);
    if (st != GEMM355_OK) return st;
    const Rows rows(x, q->rows, q->K, ld, src);
    if (rows.ld < q->K) return GEMM355_EINVAL;
    if (rows.ld > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (!aligned(x, (uintptr_t)rows.es)) return GEMM355_EALIGN;
    if (q->rows == 0 || q->K == 0) return GEMM355_OK;
    if (!x || block_meets(*q, p.q, rows.span) || block_codes(*q, p.q).meets(block_scales(*q, p.q))) return GEMM355_EINVAL;
    const int64_t per = q->block_rows == 1 ? 16 : 128;
    if ((q->rows + per - 1) / per * ((q->K + 127) / 128) > kMaxBlocks) return GEMM355_EUNSUPPORTED;
    p.x = x;
    p.ldx = rows.ld;
    p.rows = (int32_t)q->rows;
    p.K = (int32_t)q->K;
    p.f32 = rows.es == 4;
    p.block_rows = q->block_rows;
    return launch_block_quantize(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
}

gemm355_status gemm355_rmsnorm(const gemm355_rmsnorm_args *args, void *stream)
{
    NormParams p;
    const gemm355_status st = norm_setup(args, p);
    if (st != GEMM355_OK || args->rows == 0 || args->width == 0) return st;
    return launch_rmsnorm(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
}

gemm355_status gemm355_block_gemm_workspace(const gemm355_block_gemm_args *args, size_t *bytes) { return block_scratch(args, bytes); }

gemm355_status gemm355_block_gated_workspace(const gemm355_block_gated_args *args, size_t *bytes)
{
    if (args && args->act != GEMM355_ACT_SILU && args->act != GEMM355_ACT_GELU_TANH) return GEMM355_EINVAL;
    return block_scratch(args, bytes);
}

gemm355_status gemm355_block_gemm(const gemm355_block_gemm_args *args, void *stream)
{
    if (!args) return GEMM355_EINVAL;
    return block_run(block_call(*args), 0, stream);
}

gemm355_status gemm355_block_gated(const gemm355_block_gated_args *args, void *stream)
{
    if (!args || (args->act != GEMM355_ACT_SILU && args->act != GEMM355_ACT_GELU_TANH)) return GEMM355_EINVAL;
    return block_run(block_call(*args), args->act == GEMM355_ACT_SILU ? 0 : 1, stream);
}

gemm355_status gemm355_w4_quantize(const void *w, int64_t ld, gemm355_src src, const gemm355_w4_matrix *q, void *stream)
{
    W4QuantParams p;
    const gemm355_status st = w4_convert(q, w, ld, src, p);
    if (st != GEMM355_OK || q->N == 0 || q->K == 0) return st;
    /* what is written lies in three places */
    const uint64_t groups = (uint64_t)p.w.N * (uint64_t)p.w.ng;
    const Span codes(q->codes, p.w.N, ((int64_t)p.w.K + 31) / 32 * 16, p.w.ldb, 1), zeros(q->zeros, groups);
    const Span scales(q->scales, groups * (p.w.mx ? 1 : 2));
    if (codes.meets(scales) || codes.meets(zeros) || scales.meets(zeros)) return GEMM355_EINVAL;
    return launch_w4_quantize(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
}

gemm355_status gemm355_w4_dequantize(const gemm355_w4_matrix *q, void *w, int64_t ld, gemm355_src dst, void *stream)
{
    W4QuantParams p;
    const gemm355_status st = w4_convert(q, w, ld, dst, p);
    if (st != GEMM355_OK || q->N == 0 || q->K == 0) return st;
    return launch_w4_dequantize(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
}

gemm355_status gemm355_w4_gemm(int64_t M, const void *x, int64_t ldx, const gemm355_w4_matrix *w, void *y, int64_t ldy,
                               gemm355_src out, void *stream)
{
    W4GemmParams p;
    const gemm355_status st = check_w4(w, p.w);
    if (st != GEMM355_OK) return st;
    if (M < 0 || (out != GEMM355_SRC_F32 && out != GEMM355_SRC_BF16)) return GEMM355_EINVAL;
    if (M > ((int64_t)1 << 19) || w->N > ((int64_t)1 << 26)) return GEMM355_EUNSUPPORTED;
    const int64_t N = w->N, K = w->K, es = out == GEMM355_SRC_F32 ? 4 : 2;
    p.ldx = ldx ? ldx : K;
    p.ldy = ldy ? ldy : N;
    if (p.ldx < K || p.ldy < N) return GEMM355_EINVAL;
    /* the kernel's 32-bit offsets span 64 rows */
    if (p.ldx > kMaxWide || p.w.ldb > kMaxWide / 2 || p.ldy > kMaxDim) return GEMM355_EUNSUPPORTED;
    if (M > 0 && N > 0 && (!y || (K > 0 && !x))) return GEMM355_EINVAL;
    if (!aligned(x, 2) || !aligned(y, (uintptr_t)es)) return GEMM355_EALIGN;
    const Span ys(y, M, N, p.ldy, es);
    if (ys.meets(Span(x, M, K, p.ldx, 2)) || w4_meets(p.w, ys)) return GEMM355_EINVAL;
    if (M == 0 || N == 0) return GEMM355_OK;
    if (K == 0)
        return launch_zero(y, (int32_t)M, (int32_t)N, p.ldy, 0, 1, (int32_t)es, (hipStream_t)stream) == hipSuccess ? GEMM355_OK
                                                                                                                  : GEMM355_EHIP;
    p.x = (const uint16_t *)x;
    p.y = y;
    p.M = (int32_t)M;
    p.out_bf16 = es == 2 ? 1 : 0;
    /* scales and zero points are read by whole dwords */
    const int64_t groups = N * p.w.ng;
    p.even = aligned(x, 16) && p.ldx % 8 == 0 && K % 128 == 0 && aligned(w->scales, 4) && aligned(w->zeros, 4) &&
                     groups % (p.w.zeros ? 4 : p.w.mx ? 1 : 2) == 0
                 ? 1
                 : 0;
    p.tiny = K < 8 || groups * (p.w.mx ? 1 : 2) < 4 || (p.w.zeros && groups < 4) ? 1 : 0;
    return launch_w4_gemm(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
}

gemm355_status gemm355_kv_append(const gemm355_kv_append_args *args, void *stream)
{
    KvAppendParams p;
    const gemm355_status st = append_setup(args, p);
    if (st != GEMM355_OK || p.c.B == 0 || p.c.tokens == 0) return st;
    return launch_kv_append(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
}

gemm355_status gemm355_attention_workspace(const gemm355_attention_args *args, size_t *bytes)
{
    if (!bytes) return GEMM355_EINVAL;
    AttnParams p;
    size_t need = 0;
    try {
        const gemm355_status st = attention_setup(args, p, need);
        if (st != GEMM355_OK) return st;
    } catch (...) {
        return GEMM355_ENOMEM;
    }
    *bytes = need;
    return GEMM355_OK;
}

gemm355_status gemm355_attention(const gemm355_attention_args *args, void *stream)
{
    try {
        AttnParams p;
        size_t need = 0;
        gemm355_status st = attention_setup(args, p, need);
        if (st != GEMM355_OK || p.c.B == 0 || p.c.tokens == 0) return st;
        void *ws = nullptr;
        std::unique_lock<std::mutex> hold;
        if (need && args->workspace) {
            if (args->workspace_bytes < need) return GEMM355_ENOMEM;
            if (!aligned(args->workspace, 256)) return GEMM355_EALIGN;
            const gemm355_kv_cache &c = args->cache;
            const Span s(args->workspace, (uint64_t)need);
            const int64_t width = (int64_t)args->q_heads * c.head_dim;
            if (s.meets(Span(args->q, c.tokens, width, p.ldq, 2)) || s.meets(Span(args->o, c.tokens, width, p.ldo, 2)) ||
                s.meets(Span(args->lse, (uint64_t)(c.tokens * args->q_heads * 4))) || kv_meets(c, s, true))
                return GEMM355_EINVAL;
            ws = args->workspace;
        } else if (need) {
            if (capturing(stream)) return GEMM355_ENOMEM;
            st = library_scratch(need, stream, &ws, hold);
            if (st != GEMM355_OK) return st;
        }
        if (need) {
            const int64_t slots = (int64_t)p.c.B * p.c.H * p.row_tiles * p.splits;
            p.part = (float *)ws;
            p.stat = p.part + slots * p.tile_rows * p.D;
        }
        return launch_attention(p, (hipStream_t)stream) == hipSuccess ? GEMM355_OK : GEMM355_EHIP;
    } catch (...) {
        return GEMM355_ENOMEM;   /* the maps of scratch buffers could not grow */
    }
}

gemm355_status gemm355_conv2d(const gemm355_conv_args *args, void *stream)
{
    gemm355_args a;
    ConvShape cs;
    const gemm355_status st = conv_setup(args, a, cs);
    if (st != GEMM355_OK) return st;
    return run(a, stream, &cs);
}

gemm355_status gemm355_conv2d_plan(const gemm355_conv_args *args, gemm355_plan_t *out)
{
    if (!out) return GEMM355_EINVAL;
    gemm355_args a;
    ConvShape cs;
    gemm355_status st = conv_setup(args, a, cs);
    if (st != GEMM355_OK) return st;
    Plan P;
    st = get_plan(a, P, &cs);
    if (st != GEMM355_OK) return st;
    *out = P.pub;
    return GEMM355_OK;
}

gemm355_status gemm355_conv2d_out_size(const gemm355_conv_args *args, int64_t *P, int64_t *Q)
{
    if (!P || !Q) return GEMM355_EINVAL;
    gemm355_args a;
    ConvShape cs;
    const gemm355_status st = conv_setup(args, a, cs);
    if (st != GEMM355_OK) return st;
    *P = cs.P;
    *Q = cs.Q;
    return GEMM355_OK;
}

gemm355_status gemm355_gemm(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                            const void *B, int64_t ldb, void *C, int64_t ldc, gemm355_dtype dtype,
                            gemm355_layout layout, int32_t split_k, int32_t persistent,
                            void *stream)
{
    gemm355_args a;
    memset(&a, 0, sizeof a);
    a.M = M;
    a.N = N;
    a.K = K;
    a.A = A;
    a.lda = lda;
    a.B = B;
    a.ldb = ldb;
    a.C = C;
    a.ldc = ldc;
    a.batch = 1;
    a.dtype = dtype;
    a.layout = layout;
    a.split_k = split_k;
    a.persistent = persistent;
    a.tile = -1;
    return run(a, stream);
}

gemm355_status gemm355_gemm_ex(const gemm355_args *args, void *stream)
{
    if (!args) return GEMM355_EINVAL;
    return run(*args, stream);
}

gemm355_status gemm355_gemm_noalloc(const gemm355_args *args, void *stream)
{
    if (!args) return GEMM355_EINVAL;
    if (args->workspace || args->workspace_bytes) return GEMM355_EINVAL;
    return run(*args, stream, nullptr, true);
}

gemm355_status gemm355_plan(const gemm355_args *args, gemm355_plan_t *out)
{
    if (!args || !out) return GEMM355_EINVAL;
    Plan P;
    gemm355_status st = get_plan(*args, P);
    if (st != GEMM355_OK) return st;
    *out = P.pub;
    return GEMM355_OK;
}

double gemm355_eta_wave(int64_t G, int32_t S, int32_t b)
{
    if (G < 1 || S < 1 || b < 1) return NAN;
    const uint64_t cap = (uint64_t)S * (uint64_t)b;
    const uint64_t waves = ((uint64_t)G + cap - 1) / cap;
    const uint64_t den = waves * cap;
    uint64_t num = (uint64_t)G, d = den, x = num, y = d;
    while (y) {
        const uint64_t t = x % y;
        x = y;
        y = t;
    }
    return rational_to_double(num / x, d / x);
}

double gemm355_eta_pad(int64_t M, int64_t N, int64_t K, int64_t T_M, int64_t T_N, int64_t T_K)
{
    if (M < 1 || N < 1 || K < 1 || T_M < 1 || T_N < 1 || T_K < 1) return NAN;
    if (M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > 0x7FFFFFFF) return NAN;
    /* reduce each factor, then cross-reduce, to keep the rational in 64 bits */
    uint64_t num[3] = {(uint64_t)M, (uint64_t)N, (uint64_t)K};
    uint64_t den[3] = {(uint64_t)((M + T_M - 1) / T_M * T_M), (uint64_t)((N + T_N - 1) / T_N * T_N),
                       (uint64_t)((K + T_K - 1) / T_K * T_K)};
    auto gcd = [](uint64_t x, uint64_t y) {
        while (y) {
            const uint64_t t = x % y;
            x = y;
            y = t;
        }
        return x;
    };
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            const uint64_t g = gcd(num[i], den[j]);
            num[i] /= g;
            den[j] /= g;
        }
    unsigned __int128 n = (unsigned __int128)num[0] * num[1] * num[2];
    unsigned __int128 d = (unsigned __int128)den[0] * den[1] * den[2];
    /* exact (nearest binary64) whenever the reduced denominator fits in 64
     * bits, i.e. always when M'N'K' < 2^64; beyond that within one ulp */
    if (d >> 64) return (double)((long double)n / (long double)d);
    return rational_to_double((uint64_t)n, (uint64_t)d);
}

gemm355_status gemm355_kslice(int64_t nK, int32_t s, int32_t i, int64_t *begin, int64_t *end)
{
    if (!begin || !end || nK < 0 || s < 1 || i < 0 || i >= s) return GEMM355_EINVAL;
    *begin = (int64_t)(((unsigned __int128)i * (uint64_t)nK) / (uint64_t)s);
    *end = (int64_t)(((unsigned __int128)(i + 1) * (uint64_t)nK) / (uint64_t)s);
    return GEMM355_OK;
}

gemm355_status gemm355_unit(const gemm355_args *args, int64_t u, int64_t *batch, int64_t *tile_m,
                            int64_t *tile_n, int64_t *kt_begin, int64_t *kt_end)
{
    if (!args || !batch || !tile_m || !tile_n || !kt_begin || !kt_end) return GEMM355_EINVAL;
    Plan P;
    gemm355_status st = get_plan(*args, P);
    if (st != GEMM355_OK) return st;
    if (u < 0 || u >= P.s.units) return GEMM355_EINVAL;
    const Unit un = decode_unit(P.s, (int32_t)u);
    *batch = un.batch;
    *tile_m = un.tile_m;
    *tile_n = un.tile_n;
    *kt_begin = un.kt_begin;
    *kt_end = un.kt_end;
    return GEMM355_OK;
}

int32_t gemm355_num_tiles(void) { return kNumTiles; }

gemm355_status gemm355_tile_info(int32_t tile, int32_t *dtype_class, int32_t *T_M, int32_t *T_N,
                                 int32_t *T_K, int32_t *stages, int32_t *waves, int32_t *lds_bytes,
                                 int32_t *b_max, int32_t *op, int32_t *schedule)
{
    if (tile < 0 || tile >= kNumTiles) return GEMM355_EINVAL;
    const TileCfg &c = kTiles[tile];
    if (dtype_class) *dtype_class = c.dtype_class;
    if (T_M) *T_M = c.TM;
    if (T_N) *T_N = c.TN;
    if (T_K) *T_K = c.TK;
    if (stages) *stages = c.stages;
    if (waves) *waves = tile_waves(c);
    if (lds_bytes) *lds_bytes = c.lds_bytes;
    if (b_max) *b_max = resident_workgroups(tile);
    if (op) *op = c.op;
    if (schedule) *schedule = c.spread;
    return GEMM355_OK;
}

gemm355_status gemm355_set_scratch_limit(uint64_t bytes, uint64_t *previous)
{
    const uint64_t old = g_scratch_limit.exchange(bytes);
    if (previous) *previous = old;
    return GEMM355_OK;
}

gemm355_status gemm355_tile_occupancy(int32_t tile, int32_t *blocks_per_cu)
{
    if (tile < 0 || tile >= kNumTiles || !blocks_per_cu) return GEMM355_EINVAL;
    int n = 0;
    const int threads = tile_waves(kTiles[tile]) * kWaveSize;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, gemm_kernel_symbol(tile), threads, 0) !=
        hipSuccess) {
        (void)hipGetLastError();
        return GEMM355_EHIP;
    }
    *blocks_per_cu = n;
    return GEMM355_OK;
}

gemm355_status gemm355_quantize(const void *x, int64_t n, int64_t batch, gemm355_src src, gemm355_fp8 fmt,
                                void *q, float *scale, void *stream)
{
    if (n < 0 || batch < 1) return GEMM355_EINVAL;
    if ((int)src < 0 || (int)src > 1 || (int)fmt < 0 || (int)fmt > 1) return GEMM355_EINVAL;
    if (!scale || (n > 0 && (!x || !q))) return GEMM355_EINVAL;
    const int64_t es = src == GEMM355_SRC_F32 ? 4 : 2;
    if (((uintptr_t)scale & 3u) != 0) return GEMM355_EALIGN;
    if (n > 0 && ((uintptr_t)x % (uintptr_t)es) != 0) return GEMM355_EALIGN;
    if (n > 0 && (n >= ((int64_t)1 << 40) || batch >= ((int64_t)1 << 40) / n)) return GEMM355_EUNSUPPORTED;
    const int64_t total = n * batch;
    /* blocks per tensor: one per 16 Ki elements, at most 4096 */
    const int32_t parts = (int32_t)std::min<int64_t>(4096, std::max<int64_t>(1, (n + 16383) / 16384));
    if (batch * parts > ((int64_t)1 << 30)) return GEMM355_EUNSUPPORTED;
    /* no overlap between the input, the codes and the scales */
    auto overlap = [](uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a0 < b1 && b0 < a1; };
    const uintptr_t x0 = (uintptr_t)x, x1 = x0 + (uintptr_t)(total * es);
    const uintptr_t q0 = (uintptr_t)q, q1 = q0 + (uintptr_t)total;
    const uintptr_t s0 = (uintptr_t)scale, s1 = s0 + (uintptr_t)(batch * 4);
    if (total > 0 && (overlap(x0, x1, q0, q1) || overlap(x0, x1, s0, s1) || overlap(q0, q1, s0, s1)))
        return GEMM355_EINVAL;
    void *scr = nullptr;
    std::unique_lock<std::mutex> hold;
    gemm355_status st = library_scratch((size_t)(batch * parts) * sizeof(float), stream, &scr, hold);
    if (st != GEMM355_OK) return st;
    QuantParams qp;
    qp.x = x;
    qp.q = (uint8_t *)q;
    qp.scale = scale;
    qp.maxima = (float *)scr;
    qp.n = n;
    qp.batch = batch;
    qp.parts = parts;
    qp.src = src == GEMM355_SRC_F32 ? 0 : 1;
    qp.fmt = fmt == GEMM355_FP8_E4M3 ? 0 : 1;
    qp.vec = (x0 % 16 == 0) && (q0 % 8 == 0) && (n % 8 == 0);
    if (launch_quantize(qp, (hipStream_t)stream) != hipSuccess) return GEMM355_EHIP;
    return GEMM355_OK;
}

const char *gemm355_status_string(gemm355_status status)
{
    switch (status) {
    case GEMM355_OK: return "ok";
    case GEMM355_EINVAL: return "invalid argument";
    case GEMM355_EALIGN: return "misaligned pointer";
    case GEMM355_EUNSUPPORTED: return "unsupported size";
    case GEMM355_ENOMEM: return "workspace too small, scratch over its cap, or allocation failed";
    case GEMM355_EHIP: return "HIP runtime error";
    case GEMM355_ETOOBIG: return "needs more scratch than the allocation-free entry point's fixed buffer";
    default: return "unknown status";
    }
}

} /* extern "C" */
