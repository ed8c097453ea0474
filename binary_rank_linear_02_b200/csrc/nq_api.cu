// nq_api.cu -- the C ABI of libnq (declared in include/nq.h): argument checks, the
// per-device workspace, host-memory staging and the decode / prefill dispatch.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <vector>
#include <float.h>
#include <string.h>

#include "nq_internal.cuh"
#include "nq_sm100.cuh"

namespace nq {

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxRank = 65536;
constexpr int64_t kMaxElems = int64_t(1) << 40;  // element-wise helpers: elements per call
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;  // one CTA per row
constexpr int64_t kMaxListed = 1024;                  // teacher entries per token
constexpr int64_t kMaxXentTokens = int64_t(1) << 24;
std::atomic<unsigned long long> g_head_wait_ns{kWaitLimitNs};
// From this many tokens the factor gradients take the prefill GEMM for t and u and the
// tensor cores for the sums over the tokens; below, the decode stage 1 and a SIMT kernel.
constexpr int64_t kFactorTcMinBatch = 64;

std::mutex g_mutex;
Workspace g_ws[kMaxDevices];
int g_sm_count[kMaxDevices];
uint64_t g_ws_generation = 1;  // bumped (under g_mutex) whenever a workspace buffer is replaced

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Memory kind of a pointer: kDeviceMem = memory this call's kernels may read (device
// memory of the current device, or managed memory), kHostMem = host memory (pageable or
// pinned), kForeignMem = device memory of another GPU, which a kernel launched on the
// current device must not be given (without peer access it faults): every entry point
// rejects it with NQ_ERR_PTRKIND before anything is enqueued.  Without a usable device
// every pointer is a host pointer.
constexpr int kHostMem = 0, kDeviceMem = 1, kForeignMem = -1;

int classify(const cudaPointerAttributes& attr) {
    if (attr.type == cudaMemoryTypeManaged) return kDeviceMem;
    if (attr.type != cudaMemoryTypeDevice) return kHostMem;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return kForeignMem;
    }
    return attr.device == dev ? kDeviceMem : kForeignMem;
}

int pointer_kind(const void* p) {
    cudaPointerAttributes attr;
    cudaError_t err = cudaPointerGetAttributes(&attr, p);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return kHostMem;
    }
    return classify(attr);
}

// One query for x or y: the kind as pointer_kind, and for page-locked (pinned) host memory
// the device address of it in *pinned (nullptr for pageable memory or anything else).
int pointer_kind_pinned(const void* p, void** pinned) {
    *pinned = nullptr;
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return kHostMem;
    }
    const int kind = classify(attr);
    if (kind == kHostMem && attr.type == cudaMemoryTypeHost) *pinned = attr.devicePointer;
    return kind;
}

}  // namespace

unsigned long long head_wait_ns() { return g_head_wait_ns.load(std::memory_order_relaxed); }

int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    if (g_sm_count[dev] == 0) {
        int c = 0;
        cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev);
        g_sm_count[dev] = c > 0 ? c : 148;
    }
    return g_sm_count[dev];
}

Workspace* workspace_for(int64_t m, int64_t n, int64_t r, int64_t batch, const DecodeNeed& dec, int* status) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        *status = NQ_ERR_CUDA;
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(g_mutex);
    Workspace& w = g_ws[dev];
    const int64_t pbatch = batch > NQ_DECODE_MAX_BATCH ? batch : 0;  // prefill buffers only for prefill
    auto fits = [&](const Workspace& c) {
        return c.base && r <= c.r_cap && n <= c.n_cap && m <= c.m_cap && pbatch <= c.batch_cap &&
               (size_t)dec.t <= c.t_cap && (size_t)dec.tgmax <= c.tgmax_cap && (size_t)dec.partials <= c.partial_cap &&
               (size_t)dec.counters <= c.counter_cap;
    };
    if (fits(w)) {
        *status = NQ_OK;
        return &w;
    }
    // grow: keep the larger of old and new capacities
    auto mx = [](int64_t a, int64_t b) { return a > b ? a : b; };
    const int64_t r_cap = mx(r, w.r_cap), n_cap = mx(n, w.n_cap), m_cap = mx(m, w.m_cap);
    const int64_t b_cap = mx(pbatch, w.batch_cap);
    const size_t t_cap = (size_t)mx(dec.t, (int64_t)w.t_cap), g_cap = (size_t)mx(dec.tgmax, (int64_t)w.tgmax_cap);
    const size_t p_cap = (size_t)mx(dec.partials, (int64_t)w.partial_cap);
    const size_t c_cap = (size_t)mx(dec.counters, (int64_t)w.counter_cap);
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaStreamIsCapturing(0, &cs);  // legacy stream: errors if a global capture is active
    if (cudaGetLastError() != cudaSuccess) {
        *status = NQ_ERR_NOMEM;
        return nullptr;
    }
    if (w.base) cudaDeviceSynchronize();  // old buffers may still be in use
    size_t off = 0;
    const size_t o_t = off;        off = align_up(off + sizeof(float) * (t_cap + 1), 256);
    const size_t o_tgmax = off;    off = align_up(off + sizeof(float) * (g_cap + 1), 256);
    const size_t o_part = off;     off = align_up(off + sizeof(float) * (p_cap + 1), 256);
    const size_t o_cnt = off;      off = align_up(off + sizeof(int) * (c_cap + 1), 256);
    const size_t o_status = off;   off = align_up(off + sizeof(unsigned) * 64, 256);
    const size_t o_xp = off;       off = align_up(off + sizeof(uint16_t) * (size_t)b_cap * n_cap, 256);
    const size_t o_T = off;        off = align_up(off + sizeof(uint16_t) * (size_t)b_cap * r_cap, 256);
    const size_t o_xs = off;       off = align_up(off + sizeof(float) * (size_t)(b_cap + 1), 256);
    char* base = nullptr;
    if (cudaMalloc(&base, off) != cudaSuccess) {
        cudaGetLastError();
        *status = NQ_ERR_NOMEM;
        return nullptr;
    }
    if (cudaMemset(base, 0, off) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        cudaFree(base);
        *status = NQ_ERR_CUDA;
        return nullptr;
    }
    if (w.base) cudaFree(w.base);
    w.device = dev;
    w.bytes = off;
    w.base = base;
    ++g_ws_generation;
    w.t = reinterpret_cast<float*>(base + o_t);
    w.tgmax = reinterpret_cast<float*>(base + o_tgmax);
    w.partials = reinterpret_cast<float*>(base + o_part);
    w.counters = reinterpret_cast<int*>(base + o_cnt);
    w.status = reinterpret_cast<unsigned*>(base + o_status);
    w.xprime = reinterpret_cast<uint16_t*>(base + o_xp);
    w.T = reinterpret_cast<uint16_t*>(base + o_T);
    w.xscale = reinterpret_cast<float*>(base + o_xs);
    w.t_cap = t_cap;
    w.tgmax_cap = g_cap;
    w.partial_cap = p_cap;
    w.counter_cap = c_cap;
    w.r_cap = r_cap;
    w.n_cap = n_cap;
    w.m_cap = m_cap;
    w.batch_cap = b_cap;
    *status = NQ_OK;
    return &w;
}

// Scratch a call needs: the decode launch's (batch <= 8), or the largest of the prefill
// layers' split-K partials and counters.
DecodeNeed decode_need(const DecodeCall* calls, int count, int64_t batch) {
    DecodeNeed d;
    if (batch >= 1 && batch <= NQ_DECODE_MAX_BATCH) {
        decode_workspace_need(calls, count, batch, kDecodeMaxSplits, &d.t, &d.tgmax, &d.partials, &d.counters);
    } else if (batch > NQ_DECODE_MAX_BATCH) {
        for (int i = 0; i < count; ++i) {
            int64_t pf = 0, ci = 0;
            prefill_workspace_need(calls[i].m, calls[i].n, calls[i].r, batch, &pf, &ci);
            d.partials = pf > d.partials ? pf : d.partials;
            d.counters = ci > d.counters ? ci : d.counters;
        }
    }
    return d;
}

// Host-memory x / y are staged through device buffers of the workspace.
static int ensure_staging(Workspace* w, size_t xbytes, size_t ybytes) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (xbytes > w->xstage_bytes) {
        if (w->xstage) { cudaDeviceSynchronize(); cudaFree(w->xstage); w->xstage = nullptr; w->xstage_bytes = 0; }
        if (cudaMalloc(&w->xstage, xbytes) != cudaSuccess) { cudaGetLastError(); return NQ_ERR_NOMEM; }
        w->xstage_bytes = xbytes;
        ++g_ws_generation;
    }
    if (ybytes > w->ystage_bytes) {
        if (w->ystage) { cudaDeviceSynchronize(); cudaFree(w->ystage); w->ystage = nullptr; w->ystage_bytes = 0; }
        void* p = nullptr;
        if (cudaMalloc(&p, ybytes) != cudaSuccess) { cudaGetLastError(); return NQ_ERR_NOMEM; }
        w->ystage = static_cast<float*>(p);
        w->ystage_bytes = ybytes;
        ++g_ws_generation;
    }
    return NQ_OK;
}

// Scratch of the scale gradients: a vector of fp16 ones (the layer evaluated without one
// of its scales) and the batch x max(m, n) fp32 output of that evaluation.
static int ensure_grad_scratch(Workspace* w, size_t ones, size_t outs_bytes, cudaStream_t stream) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (ones > w->ones_count) {
        if (w->ones) { cudaDeviceSynchronize(); cudaFree(w->ones); w->ones = nullptr; w->ones_count = 0; }
        void* p = nullptr;
        if (cudaMalloc(&p, sizeof(uint16_t) * ones) != cudaSuccess) { cudaGetLastError(); return NQ_ERR_NOMEM; }
        w->ones = static_cast<uint16_t*>(p);
        if (fill_u16_device(w->ones, (int64_t)ones, 0x3C00, stream) != NQ_OK) return NQ_ERR_CUDA;  // fp16 1.0
        w->ones_count = ones;
        ++g_ws_generation;
    }
    if (outs_bytes > w->gstage_bytes) {
        if (w->gstage) { cudaDeviceSynchronize(); cudaFree(w->gstage); w->gstage = nullptr; w->gstage_bytes = 0; }
        void* p = nullptr;
        if (cudaMalloc(&p, outs_bytes) != cudaSuccess) { cudaGetLastError(); return NQ_ERR_NOMEM; }
        w->gstage = static_cast<float*>(p);
        w->gstage_bytes = outs_bytes;
        ++g_ws_generation;
    }
    return NQ_OK;
}

// Scratch of the envelope's terms 1 .. l-1.
static int ensure_env_scratch(Workspace* w, size_t bytes) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (bytes > w->env_bytes) {
        if (w->env) { cudaDeviceSynchronize(); cudaFree(w->env); w->env = nullptr; w->env_bytes = 0; }
        void* p = nullptr;
        if (cudaMalloc(&p, bytes) != cudaSuccess) { cudaGetLastError(); return NQ_ERR_NOMEM; }
        w->env = static_cast<float*>(p);
        w->env_bytes = bytes;
        ++g_ws_generation;
    }
    return NQ_OK;
}

// Scratch of the tensor-core factor gradients (the transposed, split operands).
static int ensure_dense_scratch(Workspace* w, size_t bytes) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (bytes > w->dense_bytes) {
        if (w->dense) { cudaDeviceSynchronize(); cudaFree(w->dense); w->dense = nullptr; w->dense_bytes = 0; }
        if (cudaMalloc(&w->dense, bytes) != cudaSuccess) { cudaGetLastError(); w->dense = nullptr; return NQ_ERR_NOMEM; }
        w->dense_bytes = bytes;
        ++g_ws_generation;
    }
    return NQ_OK;
}

// ---------------------------------------------------------------- launch cache
// A call with host x or y synchronises before it returns, so its kernels never overlap the
// next call's, and the host cost of its launches (microseconds each) adds to its latency.
// Such calls are replayed from an executable CUDA graph when the identical call (every
// pointer, size and staging buffer alike, same workspace generation) was made before: its
// first occurrence launches directly (and sizes the workspace, sets kernel attributes), the
// second captures the same launches on a private stream into a graph that is kept, and later
// ones launch that graph alone.  Workspace growth changes the generation, so a graph is
// never replayed against freed scratch.  Calls on a stream that is itself being captured,
// and calls with pageable host buffers (copies through the staging buffers), launch directly.
constexpr size_t kGraphCacheEntries = 32;  // per device; least recently used out first

struct GraphEntry {
    std::vector<uint64_t> key;
    cudaGraphExec_t exec = nullptr;  // nullptr: seen once, not captured yet
    uint64_t stamp = 0;
};
struct GraphCache {
    std::vector<GraphEntry> entries;
    uint64_t clock = 0;
    cudaStream_t capture = nullptr;  // private stream the launches are captured on
};
std::mutex g_graph_mutex;
GraphCache* g_graphs[kMaxDevices];  // never freed: the driver releases the graphs at exit

uint64_t ws_generation() {
    std::lock_guard<std::mutex> lock(g_mutex);
    return g_ws_generation;
}

// Runs `launch` (which enqueues kernels on the stream it is given and nothing else) for the
// call identified by `key` on stream s, through the cache as described above.
template <typename Launch>
int launch_cached(int dev, const std::vector<uint64_t>& key, cudaStream_t s, Launch&& launch) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (dev < 0 || dev >= kMaxDevices || cudaStreamIsCapturing(s, &cs) != cudaSuccess ||
        cs != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return launch(s);
    }
    std::lock_guard<std::mutex> lock(g_graph_mutex);
    if (!g_graphs[dev]) g_graphs[dev] = new GraphCache();
    GraphCache& c = *g_graphs[dev];
    ++c.clock;
    GraphEntry* e = nullptr;
    for (GraphEntry& x : c.entries)
        if (x.key == key) e = &x;
    if (!e) {  // first occurrence: remember it, launch directly
        if (c.entries.size() >= kGraphCacheEntries) {
            auto old = std::min_element(c.entries.begin(), c.entries.end(),
                                        [](const GraphEntry& a, const GraphEntry& b) { return a.stamp < b.stamp; });
            if (old->exec) cudaGraphExecDestroy(old->exec);
            c.entries.erase(old);
        }
        c.entries.push_back(GraphEntry{key, nullptr, c.clock});
        return launch(s);
    }
    e->stamp = c.clock;
    if (!e->exec) {  // second occurrence: capture
        if (!c.capture && cudaStreamCreateWithFlags(&c.capture, cudaStreamNonBlocking) != cudaSuccess) {
            cudaGetLastError();
            c.capture = nullptr;
            return launch(s);
        }
        if (cudaStreamBeginCapture(c.capture, cudaStreamCaptureModeThreadLocal) != cudaSuccess) {
            cudaGetLastError();
            return launch(s);
        }
        const int st = launch(c.capture);
        cudaGraph_t g = nullptr;
        const cudaError_t end = cudaStreamEndCapture(c.capture, &g);
        cudaGraphExec_t exec = nullptr;
        const bool ok = st == NQ_OK && end == cudaSuccess && g && cudaGraphInstantiate(&exec, g, 0) == cudaSuccess;
        if (g) cudaGraphDestroy(g);
        if (!ok) {
            cudaGetLastError();
            return launch(s);
        }
        e->exec = exec;
    }
    return cudaGraphLaunch(e->exec, s) == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace nq

using namespace nq;

// The grouped forward over `count` descriptors `stride` bytes apart; `ex` (may be NULL)
// adds the optional bf16 outputs of nq_linear_desc_ex.  Without `ex`, a layer's x and y may
// be host memory: pinned x are gathered into the workspace by one kernel, pinned y written
// by the kernels through their device address, pageable x and y copied through the
// workspace; then the call synchronises the stream.  The scratch of every launch is sized
// before the first is enqueued, so that the launches can be captured (launch cache above).
static int grouped_run(const nq_linear_desc* first, size_t stride, const nq_linear_desc_ex* ex, int count,
                       int64_t batch, void* stream) {
    auto desc = [&](int i) -> const nq_linear_desc& {
        return *reinterpret_cast<const nq_linear_desc*>(reinterpret_cast<const char*>(first) + stride * i);
    };
    if (batch < 0) return NQ_ERR_BATCH;
    if (count < 0) return NQ_ERR_SHAPE;
    if (count == 0 || batch == 0) return NQ_OK;
    if (!first) return NQ_ERR_NULL;
    int64_t m_max = 0, n_max = 0, r_max = 0;
    for (int i = 0; i < count; ++i) {
        const nq_linear_desc& L = desc(i);
        if (L.m <= 0 || L.n <= 0 || L.r <= 0 || L.m % 128 || L.n % 128 || L.r % 128 || L.m > kMaxDim ||
            L.n > kMaxDim || L.r > kMaxRank)
            return NQ_ERR_SHAPE;
        if (batch > (int64_t(1) << 40) / (L.m > L.n ? L.m : L.n)) return NQ_ERR_SHAPE;
        if (!L.x || !L.Upk || !L.Vpk || !L.s1 || !L.s2 || !L.y) return NQ_ERR_NULL;
        if (!aligned16(L.x) || !aligned16(L.Upk) || !aligned16(L.Vpk) || !aligned16(L.s1) || !aligned16(L.s2) ||
            !aligned16(L.y))
            return NQ_ERR_ALIGN;
        if (ex && (!aligned16(ex[i].y_bf16) || !aligned16(ex[i].y_rmsnorm_bf16))) return NQ_ERR_ALIGN;
        m_max = L.m > m_max ? L.m : m_max;
        n_max = L.n > n_max ? L.n : n_max;
        r_max = L.r > r_max ? L.r : r_max;
    }
    // memory kinds: weights on the device; x and y on the device, or (plain call) on the host.
    // Pinned host x are gathered into the workspace by one kernel; pinned host y are written
    // by the kernels through their device address; pageable x / y go through copies.
    std::vector<char> x_host(count, 0), y_host(count, 0);
    std::vector<void*> x_pin(count, nullptr), y_pin(count, nullptr);
    size_t xbytes = 0, ybytes = 0;
    for (int i = 0; i < count; ++i) {
        const nq_linear_desc& L = desc(i);
        if (pointer_kind(L.Upk) != kDeviceMem || pointer_kind(L.Vpk) != kDeviceMem ||
            pointer_kind(L.s1) != kDeviceMem || pointer_kind(L.s2) != kDeviceMem)
            return NQ_ERR_PTRKIND;
        void *xp = nullptr, *yp = nullptr;
        const int kx = pointer_kind_pinned(L.x, &xp), ky = pointer_kind_pinned(L.y, &yp);
        if (kx == kForeignMem || ky == kForeignMem) return NQ_ERR_PTRKIND;
        x_host[i] = kx == kHostMem;
        y_host[i] = ky == kHostMem;
        if (ex && (x_host[i] || y_host[i] || (ex[i].y_bf16 && pointer_kind(ex[i].y_bf16) != kDeviceMem) ||
                   (ex[i].y_rmsnorm_bf16 && pointer_kind(ex[i].y_rmsnorm_bf16) != kDeviceMem)))
            return NQ_ERR_PTRKIND;
        if (x_host[i]) {
            x_pin[i] = xp;
            xbytes += align_up(sizeof(uint16_t) * (size_t)batch * L.n, 256);
        }
        if (y_host[i]) {
            y_pin[i] = yp;
            if (!y_pin[i]) ybytes += align_up(sizeof(float) * (size_t)batch * L.m, 256);
        }
    }
    const bool any_host = xbytes || std::find(y_host.begin(), y_host.end(), 1) != y_host.end();
    bool pageable = ybytes > 0;
    for (int i = 0; i < count; ++i) pageable = pageable || (x_host[i] && !x_pin[i]);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int st = NQ_OK;
    // Path.  Up to NQ_DECODE_MAX_BATCH tokens: the decode kernels, up to 16 layers per launch
    // pair.  More tokens: each layer's prefill GEMMs, one layer after another; or, for a group
    // of layers and a few dozen tokens, the decode kernels over token chunks of at most
    // NQ_DECODE_MAX_BATCH, whichever a cost estimate fitted to B200 timings (microseconds)
    // finds faster: a decode launch pair of 5..8 tokens ~ 29.4 + 0.53 per MB of the group's
    // packed signs (1..4 tokens: half that); one layer's prefill below 64 tokens ~ 28 + 0.2
    // per token + 1.0 per MB of its packed signs (latency-bound).
    bool use_decode = batch <= NQ_DECODE_MAX_BATCH;
    if (!use_decode && count > 1 && batch <= 64) {
        double mb = 0.0, t_pre = 0.0;
        for (int i = 0; i < count; ++i) {
            const nq_linear_desc& L = desc(i);
            const double mb_i = (double)L.r * (double)(L.m + L.n) / 8e6;
            mb += mb_i;
            t_pre += 28.0 + 0.2 * (double)batch + mb_i;
        }
        const double pair = 29.4 + 0.53 * mb;
        const int64_t full = batch / NQ_DECODE_MAX_BATCH, rest = batch % NQ_DECODE_MAX_BATCH;
        const double t_dec = (double)full * pair + (rest == 0 ? 0.0 : rest <= 4 ? 0.5 * pair : pair);
        use_decode = t_dec < t_pre;
    }
    // token chunks of the decode path: full ones of NQ_DECODE_MAX_BATCH, then the rest
    const int64_t chunk = batch < NQ_DECODE_MAX_BATCH ? batch : NQ_DECODE_MAX_BATCH;
    const int64_t tail = batch % chunk;
    // the scratch of every launch of the call, sized once before anything is enqueued
    DecodeNeed need;
    for (int i0 = 0; i0 < count; i0 += (use_decode ? kMaxGroup : 1)) {
        const int cnt = !use_decode ? 1 : (count - i0 < kMaxGroup ? count - i0 : kMaxGroup);
        DecodeCall calls[kMaxGroup];
        for (int i = 0; i < cnt; ++i) {
            const nq_linear_desc& L = desc(i0 + i);
            calls[i] = DecodeCall{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, L.m, L.n, L.r};
            if (ex) calls[i].y_norm = static_cast<uint16_t*>(ex[i0 + i].y_rmsnorm_bf16);
        }
        for (const int64_t b : {use_decode ? chunk : batch, use_decode ? tail : int64_t(0)}) {
            if (b == 0) continue;
            const DecodeNeed d = decode_need(calls, cnt, b);
            need.t = d.t > need.t ? d.t : need.t;
            need.tgmax = d.tgmax > need.tgmax ? d.tgmax : need.tgmax;
            need.partials = d.partials > need.partials ? d.partials : need.partials;
            need.counters = d.counters > need.counters ? d.counters : need.counters;
        }
    }
    Workspace* ws = workspace_for(m_max, n_max, r_max, use_decode ? chunk : batch, need, &st);
    if (!ws) return st;
    if (xbytes || ybytes) {
        st = ensure_staging(ws, xbytes, ybytes);
        if (st != NQ_OK) return st;
    }
    // where each layer reads x and writes y
    std::vector<const void*> xs(count);
    std::vector<float*> ys(count);
    size_t xo = 0, yo = 0;
    for (int i = 0; i < count; ++i) {
        const nq_linear_desc& L = desc(i);
        xs[i] = L.x;
        ys[i] = L.y;
        if (x_host[i]) {
            xs[i] = static_cast<char*>(ws->xstage) + xo;
            xo += align_up(sizeof(uint16_t) * (size_t)batch * L.n, 256);
        }
        if (y_host[i]) {
            if (y_pin[i]) {
                ys[i] = static_cast<float*>(y_pin[i]);
            } else {
                ys[i] = reinterpret_cast<float*>(reinterpret_cast<char*>(ws->ystage) + yo);
                yo += align_up(sizeof(float) * (size_t)batch * L.m, 256);
            }
        }
    }
    // every launch of the call on stream q: x staging, then the layers
    auto launch = [&](cudaStream_t q) -> int {
        GatherList gl;
        gl.count = 0;
        for (int i = 0; i < count; ++i) {
            if (!x_host[i]) continue;
            const nq_linear_desc& L = desc(i);
            const size_t b = sizeof(uint16_t) * (size_t)batch * L.n;
            void* dst = const_cast<void*>(xs[i]);
            if (x_pin[i]) {
                gl.seg[gl.count++] = GatherSeg{x_pin[i], dst, b};
                if (gl.count == kMaxGather) {
                    if (gather_device(gl, q) != NQ_OK) return NQ_ERR_CUDA;
                    gl.count = 0;
                }
            } else if (cudaMemcpyAsync(dst, L.x, b, cudaMemcpyHostToDevice, q) != cudaSuccess) {
                return NQ_ERR_CUDA;
            }
        }
        if (gl.count > 0 && gather_device(gl, q) != NQ_OK) return NQ_ERR_CUDA;
        int rc = NQ_OK;
        if (!use_decode) {
            for (int i = 0; i < count && rc == NQ_OK; ++i) {
                const nq_linear_desc& L = desc(i);
                rc = prefill_forward(static_cast<const uint16_t*>(xs[i]), L.Upk, L.Vpk,
                                     static_cast<const uint16_t*>(L.s1), static_cast<const uint16_t*>(L.s2), L.m, L.n,
                                     L.r, batch, ys[i], ws, q);
                // the optional outputs by the stand-alone kernels, after the layer
                if (rc == NQ_OK && ex && ex[i].y_bf16)
                    rc = cast_f32_bf16_device(ys[i], batch * L.m, static_cast<uint16_t*>(ex[i].y_bf16), q);
                if (rc == NQ_OK && ex && ex[i].y_rmsnorm_bf16)
                    rc = rms_normalize_bf16_device(ys[i], batch, L.m, static_cast<uint16_t*>(ex[i].y_rmsnorm_bf16), q);
            }
        } else {
            for (int64_t b0 = 0; b0 < batch && rc == NQ_OK; b0 += chunk) {
                const int64_t bc = batch - b0 < chunk ? batch - b0 : chunk;
                for (int i0 = 0; i0 < count && rc == NQ_OK; i0 += kMaxGroup) {
                    const int cnt = count - i0 < kMaxGroup ? count - i0 : kMaxGroup;
                    DecodeCall calls[kMaxGroup];
                    for (int i = 0; i < cnt; ++i) {
                        const nq_linear_desc& L = desc(i0 + i);
                        calls[i] = DecodeCall{static_cast<const uint16_t*>(xs[i0 + i]) + b0 * L.n, L.Upk, L.Vpk,
                                              static_cast<const uint16_t*>(L.s1), static_cast<const uint16_t*>(L.s2),
                                              ys[i0 + i] + b0 * L.m, L.m, L.n, L.r};
                        if (ex) {
                            if (ex[i0 + i].y_bf16) calls[i].y_bf16 = static_cast<uint16_t*>(ex[i0 + i].y_bf16) + b0 * L.m;
                            if (ex[i0 + i].y_rmsnorm_bf16)
                                calls[i].y_norm = static_cast<uint16_t*>(ex[i0 + i].y_rmsnorm_bf16) + b0 * L.m;
                        }
                    }
                    rc = decode_forward_group(calls, cnt, bc, ws, q);
                }
            }
        }
        return rc;
    };
    if (any_host && !pageable) {
        int dev = -1;
        if (cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            return NQ_ERR_CUDA;
        }
        std::vector<uint64_t> key;
        key.reserve(8 + 13 * (size_t)count);
        auto u = [](const void* p) { return (uint64_t)reinterpret_cast<uintptr_t>(p); };
        key.insert(key.end(), {(uint64_t)dev, ws_generation(), (uint64_t)batch, (uint64_t)count, ex ? 1ull : 0ull,
                               u(ws->base), u(ws->xstage), u(ws->ystage)});
        for (int i = 0; i < count; ++i) {
            const nq_linear_desc& L = desc(i);
            key.insert(key.end(), {u(L.x), u(L.Upk), u(L.Vpk), u(L.s1), u(L.s2), u(L.y), (uint64_t)L.m, (uint64_t)L.n,
                                   (uint64_t)L.r, u(x_pin[i]), u(y_pin[i]), u(ex ? ex[i].y_bf16 : nullptr),
                                   u(ex ? ex[i].y_rmsnorm_bf16 : nullptr)});
        }
        st = launch_cached(dev, key, s, launch);
    } else {
        st = launch(s);
    }
    if (st != NQ_OK) return st;
    if (ybytes) {
        for (int i = 0; i < count; ++i) {
            if (!y_host[i] || y_pin[i]) continue;
            const nq_linear_desc& L = desc(i);
            if (cudaMemcpyAsync(L.y, ys[i], sizeof(float) * (size_t)batch * L.m, cudaMemcpyDeviceToHost, s) !=
                cudaSuccess)
                return NQ_ERR_CUDA;
        }
    }
    if (any_host) {
        if (cudaStreamSynchronize(s) != cudaSuccess) return NQ_ERR_CUDA;
    }
    return NQ_OK;
}

extern "C" {

int nq_version(void) { return 100; }

const char* nq_status_string(int status) {
    switch (status) {
        case NQ_OK: return "NQ_OK";
        case NQ_ERR_NULL: return "NQ_ERR_NULL: a required pointer is NULL";
        case NQ_ERR_SHAPE: return "NQ_ERR_SHAPE: a size is out of range or not a supported multiple";
        case NQ_ERR_ALIGN: return "NQ_ERR_ALIGN: a pointer is not 16-byte aligned";
        case NQ_ERR_BATCH: return "NQ_ERR_BATCH: batch is negative";
        case NQ_ERR_VALUE: return "NQ_ERR_VALUE: an input value is outside its domain";
        case NQ_ERR_CUDA: return "NQ_ERR_CUDA: a CUDA call or kernel launch failed";
        case NQ_ERR_TIMEOUT: return "NQ_ERR_TIMEOUT: a bounded device-side wait gave up";
        case NQ_ERR_NOMEM: return "NQ_ERR_NOMEM: workspace allocation failed (or was needed during stream capture)";
        case NQ_ERR_PTRKIND:
            return "NQ_ERR_PTRKIND: pointers of mixed or unsupported memory kinds (or device memory of another GPU)";
        case NQ_ERR_NOALLOC_LIMIT:
            return "NQ_ERR_NOALLOC_LIMIT: nq_lowrank_linear_fwd_noalloc takes 1 <= batch <= 8 and r <= 4096 "
                   "(its scratch is a fixed array)";
        default: return "unknown nq status";
    }
}

double nq_bits_per_weight(int64_t m, int64_t n, int64_t r) {
    if (m <= 0 || n <= 0 || r <= 0) return -1.0;
    // r(m+n) one-bit sign entries + 16(m+n) bits of fp16 scales, over the m*n dense weights
    return ((double)r * (double)(m + n) + 16.0 * (double)(m + n)) / ((double)m * (double)n);
}

int nq_pack_signs(const int8_t* signs, int64_t rows, int64_t cols, uint32_t* out, void* stream) {
    if (rows < 0 || cols < 0) return NQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return NQ_OK;
    if (!signs || !out) return NQ_ERR_NULL;
    if (rows > (int64_t(1) << 40) / cols) return NQ_ERR_SHAPE;
    const int ks = pointer_kind(signs), ko = pointer_kind(out);
    if (ks != ko || ks == kForeignMem) return NQ_ERR_PTRKIND;
    const int64_t wpr = (cols + 31) / 32;
    if (ks == kHostMem) {
        for (int64_t i = 0; i < rows * cols; ++i)
            if (signs[i] < -1 || signs[i] > 1) return NQ_ERR_VALUE;
        for (int64_t row = 0; row < rows; ++row) {
            const int8_t* src = signs + row * cols;
            for (int64_t w = 0; w < wpr; ++w) {
                uint32_t word = 0;
                const int64_t c0 = 32 * w;
                const int nb = (int)((cols - c0) < 32 ? (cols - c0) : 32);
                for (int b = 0; b < nb; ++b) word |= (src[c0 + b] >= 0 ? 1u : 0u) << b;
                out[row * wpr + w] = word;
            }
        }
        return NQ_OK;
    }
    int st = NQ_OK;
    Workspace* ws = workspace_for(128, 128, 128, 0, DecodeNeed(), &st);
    if (!ws) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(ws->status, 0, sizeof(unsigned), s) != cudaSuccess) return NQ_ERR_CUDA;
    st = pack_device(signs, rows, cols, out, ws->status, s);
    if (st != NQ_OK) return st;
    unsigned flag = 0;
    if (cudaMemcpyAsync(&flag, ws->status, sizeof(unsigned), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return NQ_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return NQ_ERR_CUDA;
    return flag ? NQ_ERR_VALUE : NQ_OK;
}

int nq_unpack_signs(const uint32_t* packed, int64_t rows, int64_t cols, int8_t* out, void* stream) {
    if (rows < 0 || cols < 0) return NQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return NQ_OK;
    if (!packed || !out) return NQ_ERR_NULL;
    if (rows > (int64_t(1) << 40) / cols) return NQ_ERR_SHAPE;
    const int kp = pointer_kind(packed), ko = pointer_kind(out);
    if (kp != ko || kp == kForeignMem) return NQ_ERR_PTRKIND;
    const int64_t wpr = (cols + 31) / 32;
    if (kp == kHostMem) {
        for (int64_t row = 0; row < rows; ++row)
            for (int64_t c = 0; c < cols; ++c)
                out[row * cols + c] = ((packed[row * wpr + c / 32] >> (c % 32)) & 1u) ? 1 : -1;
        return NQ_OK;
    }
    return unpack_device(packed, rows, cols, out, static_cast<cudaStream_t>(stream));
}

int nq_transpose_signs(const uint32_t* packed, int64_t rows, int64_t cols, uint32_t* out, void* stream) {
    if (rows < 0 || cols < 0) return NQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return NQ_OK;
    if (!packed || !out) return NQ_ERR_NULL;
    if (rows > (int64_t(1) << 40) / cols) return NQ_ERR_SHAPE;
    const int kp = pointer_kind(packed), ko = pointer_kind(out);
    if (kp != ko || kp == kForeignMem) return NQ_ERR_PTRKIND;
    const int64_t wpr_in = (cols + 31) / 32, wpr_out = (rows + 31) / 32;
    if (kp == kHostMem) {
        memset(out, 0, sizeof(uint32_t) * (size_t)(cols * wpr_out));
        for (int64_t row = 0; row < rows; ++row)
            for (int64_t c = 0; c < cols; ++c)
                if ((packed[row * wpr_in + c / 32] >> (c % 32)) & 1u) out[c * wpr_out + row / 32] |= 1u << (row % 32);
        return NQ_OK;
    }
    return transpose_device(packed, rows, cols, out, static_cast<cudaStream_t>(stream));
}

int nq_lowrank_linear_bwd_input(const void* dy, const uint32_t* UpkT, const uint32_t* VpkT, const void* s1,
                                const void* s2, int64_t m, int64_t n, int64_t r, int64_t batch, float* dx,
                                void* stream) {
    // the forward pass with the factors' roles exchanged: dx = s2 (.) (V (U^T (s1 (.) dy)))
    return nq_lowrank_linear_fwd(dy, VpkT, UpkT, s2, s1, n, m, r, batch, dx, stream);
}

int nq_lowrank_linear_bwd_scales(const void* x, const void* dy, const uint32_t* Upk, const uint32_t* Vpk,
                                 const uint32_t* UpkT, const uint32_t* VpkT, const void* s1, const void* s2,
                                 int64_t m, int64_t n, int64_t r, int64_t batch, float* ds1, float* ds2,
                                 void* stream) {
    if (batch < 0) return NQ_ERR_BATCH;
    if (m <= 0 || n <= 0 || r <= 0 || m % 128 || n % 128 || r % 128 || m > kMaxDim || n > kMaxDim ||
        r > kMaxRank)
        return NQ_ERR_SHAPE;
    if (batch > (int64_t(1) << 40) / (m > n ? m : n)) return NQ_ERR_SHAPE;
    if (!ds1 && !ds2) return NQ_OK;
    if (!x || !dy || !Upk || !Vpk || !UpkT || !VpkT || !s1 || !s2) return NQ_ERR_NULL;
    const void* ptrs[] = {x, dy, Upk, Vpk, UpkT, VpkT, s1, s2, ds1, ds2};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return NQ_ERR_ALIGN;
    for (const void* p : ptrs)
        if (p && pointer_kind(p) != kDeviceMem) return NQ_ERR_PTRKIND;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (batch == 0) {  // empty sums
        if (ds1 && cudaMemsetAsync(ds1, 0, sizeof(float) * (size_t)m, s) != cudaSuccess) return NQ_ERR_CUDA;
        if (ds2 && cudaMemsetAsync(ds2, 0, sizeof(float) * (size_t)n, s) != cudaSuccess) return NQ_ERR_CUDA;
        return NQ_OK;
    }
    int st = NQ_OK;
    const DecodeCall c{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, m > n ? m : n, m > n ? m : n, r};
    Workspace* ws = workspace_for(m > n ? m : n, m > n ? m : n, r, batch, decode_need(&c, 1, batch), &st);
    if (!ws) return st;
    const int64_t wmax = m > n ? m : n;
    st = ensure_grad_scratch(ws, (size_t)wmax,
                             sizeof(float) * ((size_t)batch * (size_t)wmax + (size_t)col_dot_scratch_floats(batch, wmax)),
                             s);
    if (st != NQ_OK) return st;
    float* dot_scratch = ws->gstage + (size_t)batch * (size_t)wmax;
    if (ds1) {  // z = U (V^T (s2 (.) x)): the forward with s1 = 1; ds1 = sum_b dy (.) z
        st = nq_lowrank_linear_fwd(x, Upk, Vpk, ws->ones, s2, m, n, r, batch, ws->gstage, stream);
        if (st != NQ_OK) return st;
        st = col_dot_device(static_cast<const uint16_t*>(dy), ws->gstage, batch, m, ds1, dot_scratch, s);
        if (st != NQ_OK) return st;
    }
    if (ds2) {  // w = V (U^T (s1 (.) dy)): the input gradient with s2 = 1; ds2 = sum_b x (.) w
        st = nq_lowrank_linear_fwd(dy, VpkT, UpkT, ws->ones, s1, n, m, r, batch, ws->gstage, stream);
        if (st != NQ_OK) return st;
        st = col_dot_device(static_cast<const uint16_t*>(x), ws->gstage, batch, n, ds2, dot_scratch, s);
        if (st != NQ_OK) return st;
    }
    return NQ_OK;
}

int nq_lowrank_linear_bwd_factors(const void* x, const void* dy, const uint32_t* Vpk, const uint32_t* UpkT,
                                  const void* s1, const void* s2, int64_t m, int64_t n, int64_t r, int64_t batch,
                                  float* dU, float* dV, void* stream) {
    if (batch < 0) return NQ_ERR_BATCH;
    if (m <= 0 || n <= 0 || r <= 0 || m % 128 || n % 128 || r % 128 || m > kMaxDim || n > kMaxDim ||
        r > kMaxRank)
        return NQ_ERR_SHAPE;
    if (batch > (int64_t(1) << 40) / (m > n ? m : n) || (m > n ? m : n) > (int64_t(1) << 40) / r) return NQ_ERR_SHAPE;
    if (!dU && !dV) return NQ_OK;
    if (!x || !dy || !Vpk || !UpkT || !s1 || !s2) return NQ_ERR_NULL;
    const void* ptrs[] = {x, dy, Vpk, UpkT, s1, s2, dU, dV};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return NQ_ERR_ALIGN;
    for (const void* p : ptrs)
        if (p && pointer_kind(p) != kDeviceMem) return NQ_ERR_PTRKIND;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (batch == 0) {  // empty sums
        if (dU && cudaMemsetAsync(dU, 0, sizeof(float) * (size_t)(m * r), s) != cudaSuccess) return NQ_ERR_CUDA;
        if (dV && cudaMemsetAsync(dV, 0, sizeof(float) * (size_t)(n * r), s) != cudaSuccess) return NQ_ERR_CUDA;
        return NQ_OK;
    }
    int st = NQ_OK;
    const int64_t w = m > n ? m : n;
    const uint16_t* xb = static_cast<const uint16_t*>(x);
    const uint16_t* dyb = static_cast<const uint16_t*>(dy);
    const uint16_t* s1b = static_cast<const uint16_t*>(s1);
    const uint16_t* s2b = static_cast<const uint16_t*>(s2);
    if (batch >= kFactorTcMinBatch) {
        // calibration-sized batches: t and u from the prefill GEMM, the sums over the tokens on
        // the tensor cores (nq_dense.cu)
        const DecodeCall c{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 128, w, r};
        Workspace* ws = workspace_for(128, w, r, batch, decode_need(&c, 1, batch), &st);
        if (!ws) return st;
        if ((st = ensure_grad_scratch(ws, (size_t)r, sizeof(float) * 2 * (size_t)batch * (size_t)r, s)) != NQ_OK ||
            (st = ensure_dense_scratch(ws, (size_t)outer_tc_scratch_bytes(batch, w, r))) != NQ_OK)
            return st;
        float* t = ws->gstage;                       // batch x r: V^T (s2 (.) x)
        float* u = ws->gstage + (size_t)batch * r;   // batch x r: U^T (s1 (.) dy)
        if (dU) {
            st = prefill_rank_vector(xb, Vpk, s2b, n, r, batch, t, ws->ones, ws, s);
            if (st == NQ_OK) st = outer_tc(dyb, s1b, t, batch, m, r, dU, ws->dense, ws->status + 1, s);
            if (st != NQ_OK) return st;
        }
        if (dV) {
            st = prefill_rank_vector(dyb, UpkT, s1b, m, r, batch, u, ws->ones, ws, s);
            if (st == NQ_OK) st = outer_tc(xb, s2b, u, batch, n, r, dV, ws->dense, ws->status + 1, s);
            if (st != NQ_OK) return st;
        }
        return NQ_OK;
    }
    const int64_t bc = batch < NQ_DECODE_MAX_BATCH ? batch : NQ_DECODE_MAX_BATCH;
    const DecodeCall c{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 128, w, r};
    Workspace* ws = workspace_for(128, w, r, bc, decode_need(&c, 1, bc), &st);
    if (!ws) return st;
    st = ensure_grad_scratch(ws, 0, sizeof(float) * 2 * (size_t)batch * (size_t)r, s);
    if (st != NQ_OK) return st;
    float* t = ws->gstage;                       // batch x r: V^T (s2 (.) x)
    float* u = ws->gstage + (size_t)batch * r;   // batch x r: U^T (s1 (.) dy)
    if (dU) {
        st = decode_rank_vector(xb, Vpk, s2b, n, r, batch, t, ws, s);
        if (st == NQ_OK) st = outer_device(dyb, s1b, t, batch, m, r, dU, s);
        if (st != NQ_OK) return st;
    }
    if (dV) {
        st = decode_rank_vector(dyb, UpkT, s1b, m, r, batch, u, ws, s);
        if (st == NQ_OK) st = outer_device(xb, s2b, u, batch, n, r, dV, s);
        if (st != NQ_OK) return st;
    }
    return NQ_OK;
}

int nq_cast_f32_to_bf16(const float* src, int64_t count, void* dst, void* stream) {
    if (count < 0 || count > kMaxElems) return NQ_ERR_SHAPE;
    if (count == 0) return NQ_OK;
    if (!src || !dst) return NQ_ERR_NULL;
    if (!aligned16(src) || !aligned16(dst)) return NQ_ERR_ALIGN;
    if (pointer_kind(src) != kDeviceMem || pointer_kind(dst) != kDeviceMem) return NQ_ERR_PTRKIND;
    return cast_f32_bf16_device(src, count, static_cast<uint16_t*>(dst), static_cast<cudaStream_t>(stream));
}

int nq_rms_normalize_bf16(const float* src, int64_t rows, int64_t cols, void* dst, void* stream) {
    if (rows < 0 || cols <= 0 || rows > kMaxRows || cols > kMaxElems / (rows > 0 ? rows : 1)) return NQ_ERR_SHAPE;
    if (rows == 0) return NQ_OK;
    if (!src || !dst) return NQ_ERR_NULL;
    if (!aligned16(src) || !aligned16(dst)) return NQ_ERR_ALIGN;
    if (pointer_kind(src) != kDeviceMem || pointer_kind(dst) != kDeviceMem) return NQ_ERR_PTRKIND;
    return rms_normalize_bf16_device(src, rows, cols, static_cast<uint16_t*>(dst), static_cast<cudaStream_t>(stream));
}

int nq_lowrank_linear_fwd_grouped(const nq_linear_desc* layers, int count, int64_t batch, void* stream) {
    return grouped_run(layers, sizeof(nq_linear_desc), nullptr, count, batch, stream);
}

int nq_lowrank_linear_fwd_grouped_ex(const nq_linear_desc_ex* layers, int count, int64_t batch, void* stream) {
    return grouped_run(layers ? &layers[0].base : nullptr, sizeof(nq_linear_desc_ex), layers, count, batch, stream);
}

int nq_device_status(void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return NQ_ERR_CUDA;
    int st = NQ_OK;
    Workspace* ws = workspace_for(128, 128, 128, 0, DecodeNeed(), &st);
    if (!ws) return st;
    unsigned word = 0;
    if (cudaMemcpy(&word, ws->status + 1, sizeof(unsigned), cudaMemcpyDeviceToHost) != cudaSuccess) return NQ_ERR_CUDA;
    // a kernel that gave up may have left arrival counters part-way: start them from zero again
    if (word != 0 && (cudaMemset(ws->status + 1, 0, sizeof(unsigned)) != cudaSuccess ||
                      cudaMemset(ws->counters, 0, sizeof(int) * (ws->counter_cap + 1)) != cudaSuccess))
        return NQ_ERR_CUDA;
    // the kernels of the output head have words of their own, and no counters: the workspace may be in
    // use on another stream
    for (auto take : {q4_take_status, distill_take_status, xent_take_status}) {
        unsigned head = 0;
        if (take(&head) != NQ_OK) return NQ_ERR_CUDA;
        if (word == 0) word = head;
    }
    return word == 0 ? NQ_OK : -(int)word;
}

int nq_selftest_wait_timeout(int64_t limit_ns, void* stream) {
    if (limit_ns < 1000 || limit_ns > 10000000000ll) return NQ_ERR_VALUE;
    int st = NQ_OK;
    Workspace* ws = workspace_for(128, 128, 128, 0, DecodeNeed(), &st);
    if (!ws) return st;
    return selftest_wait_timeout(limit_ns, ws, static_cast<cudaStream_t>(stream));
}

int nq_selftest_head_wait_limit(int64_t limit_ns) {
    if (limit_ns < 0 || limit_ns > 10000000000ll) return NQ_ERR_VALUE;
    g_head_wait_ns.store(limit_ns ? (unsigned long long)limit_ns : kWaitLimitNs, std::memory_order_relaxed);
    return NQ_OK;
}

int nq_workspace_reserve(int64_t m, int64_t n, int64_t r, int64_t batch) {
    if (m <= 0 || n <= 0 || r <= 0 || m % 128 || n % 128 || r % 128 || m > kMaxDim || n > kMaxDim ||
        r > kMaxRank)
        return NQ_ERR_SHAPE;
    if (batch < 0) return NQ_ERR_BATCH;
    int st = NQ_OK;
    const DecodeCall c{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, m, n, r};
    Workspace* ws = workspace_for(m, n, r, batch, decode_need(&c, 1, batch), &st);
    return ws ? NQ_OK : st;
}

double nq_bits_per_weight_envelope(int64_t m, int64_t n, int64_t r, int64_t l) {
    if (m <= 0 || n <= 0 || r <= 0 || l <= 0) return -1.0;
    // r(m+n) one-bit sign entries + l pairs of fp16 scale vectors (16 l (m+n) bits)
    return ((double)r * (double)(m + n) + 16.0 * (double)l * (double)(m + n)) / ((double)m * (double)n);
}

int nq_lowrank_linear_fwd_envelope(const void* x, const uint32_t* Upk, const uint32_t* Vpk, const void* a,
                                   const void* b, int64_t l, int64_t m, int64_t n, int64_t r, int64_t batch, float* y,
                                   void* stream) {
    if (batch < 0) return NQ_ERR_BATCH;
    if (l < 1 || l > kMaxGroup) return NQ_ERR_VALUE;
    if (m <= 0 || n <= 0 || r <= 0 || m % 128 || n % 128 || r % 128 || m > kMaxDim || n > kMaxDim ||
        r > kMaxRank)
        return NQ_ERR_SHAPE;
    if (batch > (int64_t(1) << 40) / (m > n ? m : n)) return NQ_ERR_SHAPE;
    if (batch == 0) return NQ_OK;
    if (!x || !Upk || !Vpk || !a || !b || !y) return NQ_ERR_NULL;
    const void* ptrs[] = {x, Upk, Vpk, a, b, y};
    for (const void* p : ptrs)
        if (!aligned16(p)) return NQ_ERR_ALIGN;
    for (const void* p : ptrs)
        if (pointer_kind(p) != kDeviceMem) return NQ_ERR_PTRKIND;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* terms = nullptr;
    if (l > 1) {
        int st = NQ_OK;
        Workspace* ws = workspace_for(m, n, r, 0, DecodeNeed(), &st);
        if (!ws) return st;
        if ((st = ensure_env_scratch(ws, sizeof(float) * (size_t)(l - 1) * (size_t)(batch * m))) != NQ_OK) return st;
        terms = ws->env;
    }
    // term q: the layer with (s1, s2) = (a_q, b_q); term 0 into y, the others into scratch
    nq_linear_desc d[kMaxGroup];
    for (int64_t q = 0; q < l; ++q) {
        d[q].x = x;
        d[q].Upk = Upk;
        d[q].Vpk = Vpk;
        d[q].s1 = static_cast<const uint16_t*>(a) + q * m;
        d[q].s2 = static_cast<const uint16_t*>(b) + q * n;
        d[q].y = q == 0 ? y : terms + (q - 1) * batch * m;
        d[q].m = m;
        d[q].n = n;
        d[q].r = r;
    }
    int st = grouped_run(d, sizeof(nq_linear_desc), nullptr, (int)l, batch, stream);
    if (st != NQ_OK || l == 1) return st;
    return envelope_sum_device(y, terms, (int)(l - 1), batch * m, s);
}

int nq_lowrank_linear_fwd(const void* x, const uint32_t* Upk, const uint32_t* Vpk, const void* s1,
                          const void* s2, int64_t m, int64_t n, int64_t r, int64_t batch, float* y,
                          void* stream) {
    if (batch < 0) return NQ_ERR_BATCH;
    if (m <= 0 || n <= 0 || r <= 0 || m % 128 || n % 128 || r % 128 || m > kMaxDim || n > kMaxDim ||
        r > kMaxRank)
        return NQ_ERR_SHAPE;
    if (batch > (int64_t(1) << 40) / (m > n ? m : n)) return NQ_ERR_SHAPE;
    if (batch == 0) return NQ_OK;
    if (!x || !Upk || !Vpk || !s1 || !s2 || !y) return NQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(Upk) || !aligned16(Vpk) || !aligned16(s1) || !aligned16(s2) ||
        !aligned16(y))
        return NQ_ERR_ALIGN;
    if (pointer_kind(Upk) != kDeviceMem || pointer_kind(Vpk) != kDeviceMem || pointer_kind(s1) != kDeviceMem ||
        pointer_kind(s2) != kDeviceMem)
        return NQ_ERR_PTRKIND;
    // one layer of the grouped path, which also handles host x / y
    nq_linear_desc d;
    d.x = x;
    d.Upk = Upk;
    d.Vpk = Vpk;
    d.s1 = s1;
    d.s2 = s2;
    d.y = y;
    d.m = m;
    d.n = n;
    d.r = r;
    return grouped_run(&d, sizeof(d), nullptr, 1, batch, stream);
}

// ---------------------------------------------------------------- the output head

// The head's entry points take device pointers alone, 16-byte aligned; null ones are optional.
// (One query of the current device for all: these calls cost about as much as they compute.)
static int check_device_pointers(const void* const* ptrs, int count) {
    for (int i = 0; i < count; ++i)
        if (ptrs[i] && !aligned16(ptrs[i])) return NQ_ERR_ALIGN;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return NQ_ERR_PTRKIND;
    }
    for (int i = 0; i < count; ++i) {
        if (!ptrs[i]) continue;
        cudaPointerAttributes attr;
        if (cudaPointerGetAttributes(&attr, ptrs[i]) != cudaSuccess) {
            cudaGetLastError();
            return NQ_ERR_PTRKIND;
        }
        if (attr.type != cudaMemoryTypeManaged && (attr.type != cudaMemoryTypeDevice || attr.device != dev))
            return NQ_ERR_PTRKIND;
    }
    return NQ_OK;
}

int nq_pack_q4(const uint8_t* codes, int64_t rows, int64_t cols, uint32_t* out, void* stream) {
    if (rows < 0 || cols < 0) return NQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return NQ_OK;
    if (!codes || !out) return NQ_ERR_NULL;
    if (rows > (int64_t(1) << 40) / cols) return NQ_ERR_SHAPE;
    const int kc = pointer_kind(codes), ko = pointer_kind(out);
    if (kc != ko || kc == kForeignMem) return NQ_ERR_PTRKIND;
    const int64_t wpr = (cols + 7) / 8;
    if (kc == kHostMem) {
        for (int64_t i = 0; i < rows * cols; ++i)
            if (codes[i] > 15) return NQ_ERR_VALUE;
        for (int64_t row = 0; row < rows; ++row) {
            for (int64_t w = 0; w < wpr; ++w) {
                uint32_t word = 0;
                for (int64_t b = 0; b < 8 && 8 * w + b < cols; ++b)
                    word |= (uint32_t)codes[row * cols + 8 * w + b] << (4 * b);
                out[row * wpr + w] = word;
            }
        }
        return NQ_OK;
    }
    int st = NQ_OK;
    Workspace* ws = workspace_for(128, 128, 128, 0, DecodeNeed(), &st);
    if (!ws) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(ws->status, 0, sizeof(unsigned), s) != cudaSuccess) return NQ_ERR_CUDA;
    st = q4_pack_device(codes, rows, cols, out, ws->status, s);
    if (st != NQ_OK) return st;
    unsigned flag = 0;
    if (cudaMemcpyAsync(&flag, ws->status, sizeof(unsigned), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return NQ_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return NQ_ERR_CUDA;
    return flag ? NQ_ERR_VALUE : NQ_OK;
}

int nq_q4_linear_fwd(const void* x, const uint32_t* Wq, const void* scales, const void* zeros, int64_t m, int64_t n,
                     int64_t group, int64_t batch, float* y, void* stream) {
    if (batch < 0 || batch > kQ4MaxBatch) return NQ_ERR_BATCH;
    if (m <= 0 || n <= 0 || n % 128 || m > kMaxDim || n > kMaxDim) return NQ_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return NQ_ERR_SHAPE;
    if (batch == 0) return NQ_OK;
    if (!x || !Wq || !scales || !y) return NQ_ERR_NULL;
    const void* ptrs[] = {x, Wq, scales, zeros, y};
    const int st = check_device_pointers(ptrs, 5);
    if (st != NQ_OK) return st;
    return q4_forward(static_cast<const uint16_t*>(x), Wq, static_cast<const uint16_t*>(scales),
                      static_cast<const uint16_t*>(zeros), m, n, (int)group, batch, y,
                      static_cast<cudaStream_t>(stream));
}

static int check_distill(int logits_type, int64_t ld, int64_t tokens, int64_t vocab, int64_t k, float temperature) {
    if (tokens < 0 || tokens > kMaxRows) return NQ_ERR_BATCH;
    if (vocab <= 0 || vocab > kMaxDim || ld < vocab || ld > 2 * kMaxDim || k <= 0 || k > kMaxListed) return NQ_ERR_SHAPE;
    if (logits_type != NQ_F32 && logits_type != NQ_BF16) return NQ_ERR_VALUE;
    if (!(temperature >= FLT_MIN && temperature <= FLT_MAX)) return NQ_ERR_VALUE;  // (below, 1 / temperature overflows)
    return NQ_OK;
}

int nq_distill_topk_fwd(const void* logits, int logits_type, int64_t ld, const int32_t* ids, const float* teacher,
                        const float* teacher_lse, int64_t tokens, int64_t vocab, int64_t k, float temperature,
                        float* loss, void* stream) {
    int st = check_distill(logits_type, ld, tokens, vocab, k, temperature);
    if (st != NQ_OK) return st;
    if (tokens == 0) return NQ_OK;
    if (!logits || !ids || !teacher || !loss) return NQ_ERR_NULL;
    const void* ptrs[] = {logits, ids, teacher, teacher_lse, loss};
    if ((st = check_device_pointers(ptrs, 5)) != NQ_OK) return st;
    return distill_device(logits, logits_type == NQ_BF16, ld, ids, teacher, teacher_lse, nullptr, tokens, vocab, k,
                          temperature, loss, nullptr, false, static_cast<cudaStream_t>(stream));
}

int nq_distill_topk_bwd(const void* logits, int logits_type, int64_t ld, const int32_t* ids, const float* teacher,
                        const float* teacher_lse, const float* dloss, int64_t tokens, int64_t vocab, int64_t k,
                        float temperature, float* loss, void* dlogits, int grad_type, void* stream) {
    int st = check_distill(logits_type, ld, tokens, vocab, k, temperature);
    if (st != NQ_OK) return st;
    if (grad_type != NQ_F32 && grad_type != NQ_BF16) return NQ_ERR_VALUE;
    if (tokens == 0) return NQ_OK;
    if (!logits || !ids || !teacher || !dloss || !dlogits) return NQ_ERR_NULL;
    const void* ptrs[] = {logits, ids, teacher, teacher_lse, dloss, loss, dlogits};
    if ((st = check_device_pointers(ptrs, 7)) != NQ_OK) return st;
    return distill_device(logits, logits_type == NQ_BF16, ld, ids, teacher, teacher_lse, dloss, tokens, vocab, k,
                          temperature, loss, dlogits, grad_type == NQ_BF16, static_cast<cudaStream_t>(stream));
}

static int check_xent(int64_t tokens, int64_t vocab, int64_t d) {
    if (tokens < 0 || tokens > kMaxXentTokens) return NQ_ERR_BATCH;
    if (vocab <= 0 || vocab > kMaxDim || d <= 0 || d % 8 || d > kMaxDim) return NQ_ERR_SHAPE;
    return NQ_OK;
}

int64_t nq_linear_cross_entropy_scratch_bytes(int64_t tokens, int64_t vocab, int64_t d, int backward) {
    if (check_xent(tokens, vocab, d) != NQ_OK) return -1;
    if (tokens == 0) return 0;
    return backward ? xent_bwd_scratch_bytes(tokens, vocab, d) : xent_fwd_scratch_bytes(tokens, vocab);
}

int nq_linear_cross_entropy_fwd(const void* h, const void* W, const int32_t* labels, int64_t tokens, int64_t vocab,
                                int64_t d, float* loss, float* lse, void* scratch, int64_t scratch_bytes, void* stream) {
    int st = check_xent(tokens, vocab, d);
    if (st != NQ_OK) return st;
    if (tokens == 0) return NQ_OK;
    if (!h || !W || !labels || !loss || !lse || !scratch) return NQ_ERR_NULL;
    const void* ptrs[] = {h, W, labels, loss, lse, scratch};
    if ((st = check_device_pointers(ptrs, 6)) != NQ_OK) return st;
    if (scratch_bytes < xent_fwd_scratch_bytes(tokens, vocab)) return NQ_ERR_NOMEM;
    return xent_forward(static_cast<const uint16_t*>(h), static_cast<const uint16_t*>(W), labels, tokens, vocab, d, loss,
                        lse, scratch, static_cast<cudaStream_t>(stream));
}

int nq_linear_cross_entropy_bwd(const void* h, const void* W, const int32_t* labels, const float* lse,
                                const float* dloss, int64_t tokens, int64_t vocab, int64_t d, void* dh, void* dW,
                                void* scratch, int64_t scratch_bytes, void* stream) {
    int st = check_xent(tokens, vocab, d);
    if (st != NQ_OK) return st;
    if (!dh && !dW) return NQ_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {  // empty sums
        if (!dW) return NQ_OK;
        const void* out[] = {dW};
        if ((st = check_device_pointers(out, 1)) != NQ_OK) return st;
        return cudaMemsetAsync(dW, 0, sizeof(uint16_t) * (size_t)vocab * (size_t)d, s) == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
    }
    if (!h || !W || !labels || !lse || !dloss || !scratch) return NQ_ERR_NULL;
    const void* ptrs[] = {h, W, labels, lse, dloss, dh, dW, scratch};
    if ((st = check_device_pointers(ptrs, 8)) != NQ_OK) return st;
    if (scratch_bytes < xent_bwd_scratch_bytes(tokens, vocab, d)) return NQ_ERR_NOMEM;
    return xent_backward(static_cast<const uint16_t*>(h), static_cast<const uint16_t*>(W), labels, lse, dloss, tokens,
                         vocab, d, static_cast<uint16_t*>(dh), static_cast<uint16_t*>(dW), scratch, s);
}

}  // extern "C"
