// nq_distill.cu -- the distillation loss of a token against its teacher's top logits, and the
// gradient of the student's logits (the output gradient that starts the refinement's backward).
//
// For one token with student logits z_v (v < vocab), teacher entries (id_k, u_k) and
// temperature T, with p = softmax(z / T):
//     q_k   = exp(u_k / T) / sum_j exp(u_j / T)            (the teacher restricted to its list), or
//     q_k   = exp(u_k / T - teacher_lse), q_rest = max(0, 1 - sum_k q_k)   (its whole vocabulary),
//     loss  = T^2 (sum_k q_k (log q_k - log p_k) + q_rest (log q_rest - log p_rest)),
//     dz_v  = dloss T (p_v tot - sum_{k: id_k = v} q_k - [v not listed] q_rest p_v / p_rest),
// p_rest = the sum of p over the ids outside the list and tot = sum_k q_k + q_rest.
//
// Two or three CTAs per SM go from token to token, with the steps of a token hidden behind
// another's.  One warp streams the rows through a ring of 16 KB pieces in shared memory, by bulk
// copies (loads into registers did not get past 4 TB/s, whatever was in flight); eight go through
// the pieces; one works for them.  In the first pass over a row the eight keep a running maximum and
// sum per thread (fp32) over the classes outside the list where the list matters (bits in shared
// memory mark it), so p_rest is a sum of its own and never a difference.  The second pass writes the
// gradient as one exponential times one factor per class.  It takes the row from L2 again: three CTAs
// per SM where that many rows stay there, and the next row's first pass before this one's second
// where twice as many do (see launch()).
//
// The one warp has, in between, the list of the row after next (its bits, q, the listed classes'
// exponentials) and the sums of the last one: what the loss is made of (logarithms and the
// differences between them, which nearly cancel when the student is close) is fp64, for the listed
// classes alone.  It also takes the classes of a row that lie outside its 16-byte boundaries, and
// writes the listed classes' gradient, last, over the others'.
//
// What bounds it: HBM.  (Times in calls in a row.)  777 x 50257 fp32 forward: 33 us (4.7 TB/s of logits).
// 1024 x 32000 fp32 to bf16 gradients: 54 us, the logits and the gradient at 3.6 TB/s; 1024 rows are 2.3
// rounds of the 444 CTAs.  4096 x 128000 bf16: 517 to 548 us, where rows of 256 KB do not all stay in L2: HBM
// carries the logits almost twice (1024 such rows: 1.66 times) and the gradient once.  Where rows are short the teacher's warp bounds it:
// 4096 x 1000 fp32 forward, 64 listed: 40 us, some 4 us a row.  Ways around the second reading lost: a cluster
// that keeps a row in its shared memory (its reductions, 20 us of a row's life, left HBM idle), and
// one CTA of 16 warps per SM that keeps what its ring holds (on the device, by itself, 484 us where this
// took 503, but 62 in place of 50 for the smaller rows: the time between the passes is filled by nothing);
// nor did half a row to each CTA of a cluster, which leaves L2 half as many rows to keep, gain anything
// (541 us).  A second warp
// for the teacher (lists by one, sums by the other) made a call by itself 4% faster and calls in a
// row 1% slower.
#include <cuda_bf16.h>
#include <type_traits>

#include "nq_internal.cuh"
#include "nq_sm100.cuh"

namespace nq {
namespace {

constexpr int kDtWarps = 8;                        // that go through the rows
constexpr int kDtFetch = kDtWarps, kDtTeacher = kDtWarps + 1;  // the warps that fetch them, and that read the teacher
constexpr int kDtThreads = 32 * (kDtWarps + 2);
constexpr int kDtPiece = 16384;                    // bytes
constexpr int kDtMaxSlots = 8;
constexpr int kDtRows = 3;                         // rows a CTA has something of
constexpr size_t kDtMost = 226 * 1024;             // shared memory of an SM's CTAs
constexpr int64_t kDtStays = int64_t(64) << 20;    // of L2, for the rows that are in work

// A device-side wait that gave up (NQ_ERR_TIMEOUT) is recorded here; nq_device_status reads it.
__device__ unsigned g_distill_status;

struct DistillArgs {
    const void* logits;
    int64_t ld;
    const int32_t* ids;        // tokens x k
    const float* teacher;      // tokens x k
    const float* teacher_lse;  // tokens or null
    const float* dloss;        // tokens (gradient)
    float* loss;               // tokens or null
    void* dlogits;             // tokens x ld
    int vocab, k;
    float temperature;
    int64_t tokens;
    int slots, rows;           // pieces of shared memory; rows of lists in it
    int lag;                   // first passes ahead of the second ones (0, 1)
    unsigned long long wait_ns;  // kTimed: how long a wait lasts
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
// 8 values of a row as four pairs of floats.
__device__ __forceinline__ void load8(const float* p, float2 (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void load8(const uint16_t* p, float2 (&v)[4]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
// A group of 8 lies on a 16-byte boundary of the logits: in the gradient on one too, except that
// bf16 beside fp32 logits may lie between two.  (Stores that leave L2 first: the logits are to stay.)
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4], bool) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
}
__device__ __forceinline__ void store8(uint16_t* p, const float2 (&v)[4], bool aligned) {
    const uint4 w = make_uint4(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y), pack2(v[2].x, v[2].y), pack2(v[3].x, v[3].y));
    if (aligned) {
        __stcs(reinterpret_cast<uint4*>(p), w);
    } else {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(w.x, w.y));
        __stcs(reinterpret_cast<uint2*>(p) + 1, make_uint2(w.z, w.w));
    }
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A maximum m and a sum s of exponentials relative to it, exactly: the sum of 2^(v c) over what
// was taken is s 2^ref(m).  ref(m) is the float at(m), m c rounded (0 without values, m = -inf):
// one FMA per value; what at() and c round away is made up for in fp64 at the end.  It grows with
// m c, though, and from |m c| = 2^20 on (a mask of -1e10 or the type's lowest value, a tiny
// temperature) ref(m) is the number m c itself, and only differences (v - m) c are formed: a group
// of masked classes has that maximum, and at -1e10 the FMA's rest would be 2^439.
struct MaxSum {
    float m, s;
};
// (a product of its own: an FMA that took it in would be another reference)
__device__ __forceinline__ float at(float m, float c) { return m == -INFINITY ? 0.f : __fmul_rn(m, c); }
__device__ __forceinline__ bool far(float m, float c) { return m > -INFINITY && !(fabsf(m * c) < 0x1p20f); }
__device__ __forceinline__ float ex2_from(float v, float m, float c) {  // 2^(v c - ref(m))
    return ex2(far(m, c) ? (v - m) * c : fmaf(v, c, -at(m, c)));
}
__device__ __forceinline__ float ex2_between(float a, float b, float c) {  // 2^(ref(a) - ref(b)), a <= b; 0 for a = -inf
    if (a == -INFINITY) return 0.f;
    if (!far(a, c) && !far(b, c)) return ex2(at(a, c) - at(b, c));
    const float rest_a = far(a, c) ? 0.f : fmaf(a, c, -at(a, c)), rest_b = far(b, c) ? 0.f : fmaf(b, c, -at(b, c));
    return ex2((a - b) * c - rest_a + rest_b);
}
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m);
    return MaxSum{m, a.s * ex2_between(a.m, m, c) + b.s * ex2_between(b.m, m, c)};
}

// Two floats at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Shared memory of a row's list: q (fp64), ids, logits and owner marks, then a bit per class.
__host__ __device__ constexpr size_t distill_list_bytes(int64_t vocab, int64_t k) {
    return (8 * k + 4 * k + 4 * k + (k + 3) / 4 * 4 + (vocab + 24 + 31) / 32 * 4 + 15) / 16 * 16;
}

// A row of the CTA: where its logits lie, and the classes before and after its 16-byte boundaries.
template <typename TL>
struct DistillRow {
    int64_t row;
    const TL* z;
    int head, groups, tail, edge;
    __device__ __forceinline__ DistillRow(const DistillArgs& p, int i) {
        row = blockIdx.x + (int64_t)i * gridDim.x;
        z = static_cast<const TL*>(p.logits) + row * p.ld;
        const int head0 = (int)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(TL));
        head = head0 < p.vocab ? head0 : p.vocab;
        groups = (p.vocab - head) / 8;
        tail = head + 8 * groups;
        edge = head + p.vocab - tail;
    }
    __device__ __forceinline__ int edge_class(int i) const { return i < head ? i : tail + i - head; }
    __device__ __forceinline__ int bit(int v) const { return v - head + 8; }  // of class v: a group of 8 is a byte
};

// After a wait for a piece that was given up: the piece lands, or the fetching warp has stopped (which it
// does when it next waits).  So a place of the ring is given back only when nothing is under way to it,
// or nothing more will be.  (A look at the abort flag before each fetch cost 1% in place of this.)
__device__ __noinline__ void outlast(uint32_t bar, uint32_t parity, volatile int* ended) {
    const unsigned long long t0 = global_ns();
    while (!mbar_try(bar, parity) && !*ended && global_ns() - t0 < kWaitLimitNs) {
    }
}

// (kTimed: a kernel of its own, since a limit that is not a constant costs the others 1%)
template <typename TL, typename TG, bool kGrad, bool kTimed>
__global__ void __launch_bounds__(kDtThreads, 3) distill_kernel(const DistillArgs p) {
    const unsigned long long limit_ns = kTimed ? p.wait_ns : kWaitLimitNs;
    constexpr int kGroupBytes = 8 * sizeof(TL), kPieceGroups = kDtPiece / kGroupBytes;
    constexpr int kRowThreads = 32 * kDtWarps;               // threads that go through the rows
    constexpr int kPerThread = kPieceGroups / kRowThreads;   // groups of 8 classes a thread has of a piece
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ MaxSum warp_part[kDtRows][kDtWarps];
    __shared__ unsigned long long full[kDtMaxSlots], empty[kDtMaxSlots];
    // of a row: its list's bits are there; its first pass is done; its factors are there; its second pass is done
    __shared__ unsigned long long listed_bar[kDtRows], summed_bar[kDtRows], factors_bar[kDtRows], graded_bar[kDtRows];
    __shared__ float factor_of[kDtRows], mr_of[kDtRows], scale_of[kDtRows], m_of[kDtRows], edge_z[kDtRows][16];
    __shared__ double qsum_of[kDtRows], cross_of[kDtRows], sl_of[kDtRows];
    __shared__ float ml_of[kDtRows], origin_of[kDtRows];
    __shared__ int any_of[kDtRows], dups_of[kDtRows], abort_word, stopped_word;
    volatile int* abort_flag = &abort_word;
    const int V = p.vocab, K = p.k, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float c = 1.4426950408889634f / p.temperature;
    const bool whole = p.teacher_lse != nullptr;
    const int n = (int)((p.tokens - blockIdx.x + gridDim.x - 1) / gridDim.x);  // rows of this CTA
    const size_t list_bytes = distill_list_bytes(V, K);
    unsigned char* lists = smem + p.slots * kDtPiece;
    auto mask_of = [&](int b) {
        return reinterpret_cast<uint32_t*>(lists + b * list_bytes + 8 * K + 4 * K + 4 * K + (K + 3) / 4 * 4);
    };
    auto pieces_of = [&](int groups) { return (groups + kPieceGroups - 1) / kPieceGroups; };

    if (tid == 0) {
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), kDtWarps);
        }
        for (int b = 0; b < kDtRows; ++b) {
            mbar_init(smem_u32(&listed_bar[b]), 1);
            mbar_init(smem_u32(&summed_bar[b]), kDtWarps);
            mbar_init(smem_u32(&factors_bar[b]), 1);
            mbar_init(smem_u32(&graded_bar[b]), kDtWarps);
        }
        abort_word = stopped_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < p.rows * (int)(list_bytes / 16); i += kDtThreads)
        reinterpret_cast<uint4*>(lists)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    if (warp == kDtFetch) {
        if (lane == 0) {
            bool ok = true;
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            auto stream = [&](int i) {
                const DistillRow<TL> r(p, i);
                for (int first = 0; first < r.groups && ok; first += kPieceGroups) {
                    ok = mbar_wait(smem_u32(&empty[slot]), phase ^ 1u, abort_flag, &g_distill_status, limit_ns);
                    if (!ok) break;
                    const uint32_t bytes = (uint32_t)((r.groups - first < kPieceGroups ? r.groups - first : kPieceGroups) * kGroupBytes);
                    const uint32_t bar = smem_u32(&full[slot]);
                    mbar_expect_tx(bar, bytes);
                    bulk_load(smem_u32(smem + slot * kDtPiece), r.z + r.head + 8 * first, bytes, bar);
                    ++issued;
                    if (++slot == p.slots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            };
            for (int s = 0; s < n + p.lag && ok; ++s) {
                if (s < n) stream(s);
                if (kGrad && s >= p.lag) stream(s - p.lag);
            }
            *const_cast<volatile int*>(&stopped_word) = 1;
            // whoever gave up, if any: what is in flight lands before the CTA leaves
            for (int i = issued - p.slots < 0 ? 0 : issued - p.slots; i < issued; ++i)
                mbar_drain(smem_u32(&full[i % p.slots]), (uint32_t)(i / p.slots) & 1u);
        }
        __syncthreads();
        return;
    }

    if (warp == kDtTeacher) {
        const double T = p.temperature, invT = 1.0 / T;
        auto rounded = [&](float m) { return m > -INFINITY && !far(m, c) ? exp2((double)at(m, c) - (double)m * c) : 1.0; };
        // ---- the list of row i: bits, owners of a class (its first entry), q, what it comes to
        auto read_list = [&](int i) {
            const DistillRow<TL> r(p, i);
            const int b = i % kDtRows;
            double* sq = reinterpret_cast<double*>(lists + b * list_bytes);
            int32_t* sid = reinterpret_cast<int32_t*>(sq + K);
            float* sz = reinterpret_cast<float*>(sid + K);
            unsigned char* owner = reinterpret_cast<unsigned char*>(sz + K);
            uint32_t* mask = mask_of(b);
            const float* u = p.teacher + r.row * K;
            const double lse = whole ? (double)p.teacher_lse[r.row] : 0.0;
            if (lane < r.edge) edge_z[b][lane] = load1(r.z + r.edge_class(lane));
            bool any = false, twice = false;
            double umax = -INFINITY;
            float zmax = -INFINITY;
            constexpr int kBatch = 4;
            for (int k0 = lane; k0 < K + lane; k0 += 32 * kBatch) {
                int id[kBatch];
                float zk[kBatch], uk[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int k = k0 + 32 * j;
                    id[j] = k < K ? p.ids[r.row * K + k] : -1;
                    uk[j] = k < K ? u[k] : 0.f;
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (id[j] < 0 || id[j] >= V) id[j] = -1;
                    zk[j] = id[j] >= 0 ? load1(r.z + id[j]) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int k = k0 + 32 * j;
                    if (k >= K) continue;
                    bool own = false;
                    if (id[j] >= 0) {
                        const int bit = r.bit(id[j]);
                        own = !(atomicOr(&mask[bit >> 5], 1u << (bit & 31)) >> (bit & 31) & 1u);
                        twice |= !own;
                        any = true;
                        umax = fmax(umax, (double)uk[j]);
                        zmax = fmaxf(zmax, zk[j]);
                    }
                    sid[k] = id[j];
                    sz[k] = zk[j];
                    owner[k] = own;
                    sq[k] = uk[j];
                }
            }
            any = __any_sync(0xffffffffu, any);
            twice = __any_sync(0xffffffffu, twice);
            __syncwarp();
            // An id listed again belongs to its first entry, whichever lane was faster (the order of the
            // sum over the classes goes by it): the entries take the bits away in turn, and put them back.
            if (twice) {
                for (int k = lane; k < K + lane; k += 32) {
                    const int id = k < K ? sid[k] : -1, bit = r.bit(id);
                    const bool first = !(__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1u));
                    if (id >= 0) owner[k] = first && (atomicAnd(&mask[bit >> 5], ~(1u << (bit & 31))) >> (bit & 31) & 1u);
                    __syncwarp();
                }
                for (int k = lane; k < K; k += 32)
                    if (sid[k] >= 0) atomicOr(&mask[r.bit(sid[k]) >> 5], 1u << (r.bit(sid[k]) & 31));
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(smem_u32(&listed_bar[b]));
            double qsum = 0.0, cross = 0.0, sl = 0.0, shift = lse, esum = 0.0;  // q_k = exp(u_k / T - shift) (/ esum)
            if (!whole) {
                umax = warp_max(umax);
                shift = umax * invT;
            }
            // the logits' part of the loss is taken from the largest listed one on: where a whole row
            // is at -1e20, log p is what is left when that goes
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) zmax = fmaxf(zmax, __shfl_xor_sync(0xffffffffu, zmax, o));
            const float origin = fabsf(zmax) < INFINITY ? zmax : 0.f;
            for (int k = lane; k < K; k += 32) {
                const double lq = sq[k] * invT - shift, q = sid[k] >= 0 ? exp(lq) : 0.0;
                sq[k] = q;
                qsum += q;
                if (q > 0.0) cross += q * (lq - ((double)sz[k] - origin) * invT);
            }
            qsum = warp_sum(qsum);
            cross = warp_sum(cross);
            if (!whole) {  // to sum 1
                esum = 1.0 / qsum;
                cross = cross * esum - log(qsum);
                for (int k = lane; k < K; k += 32) sq[k] *= esum;
                qsum = any ? 1.0 : 0.0;
            } else {  // the listed classes, each once
                for (int k = lane; k < K; k += 32)
                    if (owner[k] && zmax > -INFINITY) sl += exp(((double)sz[k] - zmax) * invT);
                sl = warp_sum(sl);
            }
            if (lane == 0) {
                qsum_of[b] = qsum;
                cross_of[b] = cross;
                sl_of[b] = sl;
                ml_of[b] = whole ? zmax : -INFINITY;  // (of the listed classes, where these are apart)
                origin_of[b] = origin;
                any_of[b] = any;
                dups_of[b] = twice;
            }
            __syncwarp();
        };
        // ---- after row i's first pass: its loss, and the factors of its gradient
        auto put_together = [&](int i) {
            const DistillRow<TL> r(p, i);
            const int b = i % kDtRows;
            const double dloss = kGrad ? (double)p.dloss[r.row] : 0.0;
            mbar_wait(smem_u32(&summed_bar[b]), (uint32_t)(i / kDtRows) & 1u, abort_flag, &g_distill_status, limit_ns);
            MaxSum s = lane < kDtWarps ? warp_part[b][lane] : MaxSum{-INFINITY, 0.f};
            if (lane >= kDtWarps && lane - kDtWarps < r.edge) {
                const int bit = r.bit(r.edge_class(lane - kDtWarps));
                if (!whole || !(mask_of(b)[bit >> 5] >> (bit & 31) & 1u)) s = MaxSum{edge_z[b][lane - kDtWarps], 1.f};
                if (s.m != s.m) s = MaxSum{-INFINITY, s.m};  // a NaN is in every sum
            }
            float mr = s.m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
            // (in fp64: one exponential's error would shift every logarithm below; an edge class's sum
            // of 1 is relative to its own value, not to at() of it)
            const bool single = lane >= kDtWarps;
            const double between = (single || far(s.m, c) ? (double)s.m * c : (double)at(s.m, c)) -
                                   (far(mr, c) ? (double)mr * c : (double)at(mr, c));
            const double off = rounded(mr), sr = off * warp_sum(s.s * (s.m > -INFINITY ? exp2(between) : 0.0));
            const float ml = ml_of[b], m = fmaxf(mr, ml);
            const double qsum = qsum_of[b];
            // (two exponentials side by side in the lanes)
            const float mine = lane == 0 ? mr : ml;
            const double e = mine > -INFINITY ? exp(((double)mine - m) * invT) : 0.0;
            const double er = __shfl_sync(0xffffffffu, e, 0), el = __shfl_sync(0xffffffffu, e, 1);
            const double sum = (mr > -INFINITY ? sr * er : sr) + (ml > -INFINITY ? sl_of[b] * el : 0.0);
            const double qrest = whole && mr > -INFINITY ? fmax(0.0, 1.0 - qsum) : 0.0;
            if (kGrad && lane == 0) {
                // outside the list dz_v = exp((z_v - mr) / T) (tot exp((mr - m) / T) / sum - qrest / sr) T dloss
                // (the two nearly cancel when the student is close: in fp64)
                const double gT = T * dloss;
                scale_of[b] = (float)((qsum + qrest) * gT / sum);
                factor_of[b] = mr > -INFINITY ? (float)((er * (qsum + qrest) / sum - qrest / sr) * gT * off) : 0.f;
                mr_of[b] = mr;
                m_of[b] = m;
                mbar_arrive(smem_u32(&factors_bar[b]));
            }
            if (lane == 0 && p.loss) {
                double loss = 0.0;  // with nothing to learn from, whatever the logits are
                if (any_of[b]) {
                    const double logsum = log(sum);  // log p_v = (z_v - m) / T - logsum
                    loss = cross_of[b] + qsum * (((double)m - origin_of[b]) * invT + logsum);
                    if (qrest > 0.0) loss += qrest * (log(qrest) - (((double)mr - m) * invT + log(sr) - logsum));
                }
                p.loss[r.row] = (float)(loss * T * T);
            }
            __syncwarp();
        };
        // ---- after row i's second pass: the classes outside its groups, then the listed ones; and the
        // bits are cleared for the row that comes into their place
        auto finish = [&](int i) {
            const DistillRow<TL> r(p, i);
            const int b = i % kDtRows;
            const double* sq = reinterpret_cast<const double*>(lists + b * list_bytes);
            const int32_t* sid = reinterpret_cast<const int32_t*>(sq + K);
            const float* sz = reinterpret_cast<const float*>(sid + K);
            const unsigned char* owner = reinterpret_cast<const unsigned char*>(sz + K);
            if constexpr (kGrad) {
                TG* dz = static_cast<TG*>(p.dlogits) + r.row * p.ld;
                const float gT = p.temperature * p.dloss[r.row];
                mbar_wait(smem_u32(&graded_bar[b]), (uint32_t)(i / kDtRows) & 1u, abort_flag, &g_distill_status, limit_ns);
                if (lane < r.edge)
                    store1(dz + r.edge_class(lane), any_of[b] ? ex2_from(edge_z[b][lane], mr_of[b], c) * factor_of[b] : 0.f);
                __syncwarp();
                for (int k = lane; k < K; k += 32) {
                    if (!owner[k]) continue;
                    double q = sq[k];
                    if (dups_of[b]) {  // the class may be listed again: its masses add, in the list's order
                        q = 0.0;
                        for (int j = 0; j < K; ++j)
                            if (sid[j] == sid[k]) q += sq[j];
                    }
                    store1(dz + sid[k], ex2((sz[k] - m_of[b]) * c) * scale_of[b] - (float)q * gT);
                }
            }
            uint32_t* mask = mask_of(b);
            for (int k = lane; k < K; k += 32)
                if (sid[k] >= 0) mask[r.bit(sid[k]) >> 5] = 0;
            __syncwarp();
        };
        // The row after next's list is read while the eight are in the rows before it.
        read_list(0);
        if (n > 1) read_list(1);
        for (int i = 0; i < n; ++i) {
            put_together(i);
            if (kGrad && i > 0) finish(i - 1);
            if (!kGrad) finish(i);
            if (i + 2 < n) read_list(i + 2);
        }
        if (kGrad) finish(n - 1);
        __syncthreads();
        return;
    }

    int slot = 0;
    uint32_t phase = 0;
    // Takes the pieces of a row: fn(the place of the thread's first group in shared memory, its
    // number, how many groups there are, a constant where all are).
    auto through = [&](const DistillRow<TL>& r, auto&& fn) {
        for (int first = 0; first < r.groups; first += kPieceGroups) {
            if (!mbar_wait(smem_u32(&full[slot]), phase, abort_flag, &g_distill_status, limit_ns))
                outlast(smem_u32(&full[slot]), phase, &stopped_word);
            const TL* mine = reinterpret_cast<const TL*>(smem + slot * kDtPiece) + 8 * tid;
            const int left = r.groups - first - tid;
            if (r.groups - first >= kPieceGroups) {
#pragma unroll
                for (int q = 0; q < kPerThread; q += 2)
                    fn(mine + 8 * q * kRowThreads, first + tid + q * kRowThreads, std::integral_constant<int, 2>());
            } else
                for (int q = 0; q < kPerThread && q * kRowThreads < left; ++q)
                    fn(mine + 8 * q * kRowThreads, first + tid + q * kRowThreads, std::integral_constant<int, 1>());
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
            if (++slot == p.slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
    };
    const float2 cc = make_float2(c, c);
    auto first_pass = [&](int s) {
        const DistillRow<TL> r(p, s);
        const int b = s % kDtRows;
        const unsigned char* bytes = reinterpret_cast<const unsigned char*>(mask_of(b)) + 1;
        auto listed_yet = [&]() {
            mbar_wait(smem_u32(&listed_bar[b]), (uint32_t)(s / kDtRows) & 1u, abort_flag, &g_distill_status, limit_ns);
        };
        if (whole) listed_yet();
        MaxSum sum{-INFINITY, 0.f};
        through(r, [&](const TL* at8, int i, auto count) {
            constexpr int kCount = decltype(count)::value;
            float2 v[kCount][4];
#pragma unroll
            for (int q = 0; q < kCount; ++q) load8(at8 + 8 * q * kRowThreads, v[q]);
            if (whole) {
                unsigned listed[kCount], any = 0;
#pragma unroll
                for (int q = 0; q < kCount; ++q) any |= listed[q] = bytes[i + q * kRowThreads];
                if (any) {
#pragma unroll
                    for (int q = 0; q < kCount; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (listed[q] >> (2 * j) & 1u) v[q][j].x = -INFINITY;
                            if (listed[q] >> (2 * j + 1) & 1u) v[q][j].y = -INFINITY;
                        }
                }
            }
            float m = sum.m;
#pragma unroll
            for (int q = 0; q < kCount; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(v[q][j].x, v[q][j].y));
            if (m != sum.m) sum = MaxSum{m, sum.s * ex2_between(sum.m, m, c)};
            float2 e[2] = {make_float2(sum.s, 0.f), make_float2(0.f, 0.f)};
            if (far(m, c)) {
#pragma unroll
                for (int q = 0; q < kCount; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        e[j & 1] = add2(e[j & 1], make_float2(ex2((v[q][j].x - m) * c), ex2((v[q][j].y - m) * c)));
            } else {
                const float to = -at(m, c);
                const float2 to2 = make_float2(to, to);
#pragma unroll
                for (int q = 0; q < kCount; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = fma2(v[q][j], cc, to2);
                        e[j & 1] = add2(e[j & 1], make_float2(ex2(x.x), ex2(x.y)));
                    }
            }
            e[0] = add2(e[0], e[1]);
            sum.s = e[0].x + e[0].y;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum = join(sum, MaxSum{__shfl_xor_sync(0xffffffffu, sum.m, o), __shfl_xor_sync(0xffffffffu, sum.s, o)}, c);
        // Only this holds a forward back behind the teacher's warp (a gradient's second passes do as
        // well): row s's list is read after row s - 2's sums were put together, so the place of row
        // s - 3's sums is free, and its barrier has been looked at.  Without the list's bits it is
        // enough to wait here, when the row has been gone through.
        if (!whole) listed_yet();
        if (lane == 0) {
            warp_part[b][warp] = sum;
            mbar_arrive(smem_u32(&summed_bar[b]));
        }
    };
    auto second_pass = [&](int s) {
        const DistillRow<TL> r(p, s);
        const int b = s % kDtRows;
        TG* dz = static_cast<TG*>(p.dlogits) + r.row * p.ld;
        for (int64_t v = (int64_t)V + tid; v < p.ld; v += kRowThreads) store1(dz + v, 0.f);
        mbar_wait(smem_u32(&factors_bar[b]), (uint32_t)(s / kDtRows) & 1u, abort_flag, &g_distill_status, limit_ns);
        const float mr = mr_of[b], from = -at(mr, c), factor = factor_of[b];
        const float2 from2 = make_float2(from, from), factor2 = make_float2(factor, factor);
        TG* out = dz + r.head;
        const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const bool plain = any_of[b] && !far(mr, c);
        through(r, [&](const TL* at8, int i, auto count) {
            constexpr int kCount = decltype(count)::value;
            float2 v[kCount][4];
#pragma unroll
            for (int q = 0; q < kCount; ++q) load8(at8 + 8 * q * kRowThreads, v[q]);
            if (plain) {
#pragma unroll
                for (int q = 0; q < kCount; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = fma2(v[q][j], cc, from2);
                        v[q][j] = mul2(make_float2(ex2(x.x), ex2(x.y)), factor2);
                    }
            } else {  // nothing to learn from: no gradient, whatever the logits are
                const bool learns = any_of[b];
#pragma unroll
                for (int q = 0; q < kCount; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[q][j] = learns ? make_float2(ex2((v[q][j].x - mr) * c) * factor, ex2((v[q][j].y - mr) * c) * factor)
                                         : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int q = 0; q < kCount; ++q) store8(out + 8 * (i + q * kRowThreads), v[q], aligned);
        });
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&graded_bar[b]));
    };
    for (int s = 0; s < n + p.lag; ++s) {
        if (s < n) first_pass(s);
        if (kGrad && s >= p.lag) second_pass(s - p.lag);
    }
    __syncthreads();
}

template <typename TL, typename TG, bool kGrad, bool kTimed>
int launch_as(DistillArgs a, cudaStream_t stream) {
    static unsigned long long init_mask = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&init_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(distill_kernel<TL, TG, kGrad, kTimed>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kDtMost) != cudaSuccess)
            return NQ_ERR_CUDA;
        __atomic_fetch_or(&init_mask, bit, __ATOMIC_RELEASE);
    }
    // CTAs per SM: three, or two where that many rows leave L2 between their passes
    const size_t list = distill_list_bytes(a.vocab, a.k);
    const int64_t row_bytes = (int64_t)a.vocab * (int64_t)sizeof(TL);
    int per_sm = !kGrad || 3 * sm_count() * row_bytes <= kDtStays ? 3 : 2;
    // the lists of three rows beside four pieces at least; of one row, and one row per CTA, where the
    // bits of the vocabulary are too many
    a.rows = kDtRows;
    while (per_sm > 1 && kDtRows * list + 3 * kDtPiece > kDtMost / per_sm - 2048) --per_sm;
    if (kDtRows * list + 3 * kDtPiece > kDtMost / per_sm - 2048) a.rows = 1;
    const int64_t slots = (int64_t)((kDtMost / per_sm - 2048 - a.rows * list) / kDtPiece);
    a.slots = (int)(slots < kDtMaxSlots ? slots : kDtMaxSlots);
    // a row's second pass after the next row's first, where twice the rows stay in L2
    a.lag = kGrad && 2 * per_sm * sm_count() * row_bytes <= kDtStays;
    const int64_t at_once = (int64_t)per_sm * sm_count(), ctas = a.rows == 1 || a.tokens < at_once ? a.tokens : at_once;
    return launch_pdl(distill_kernel<TL, TG, kGrad, kTimed>, dim3((unsigned)ctas), dim3(kDtThreads),
                      (size_t)a.slots * kDtPiece + a.rows * list, stream, a) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

template <typename TL, typename TG, bool kGrad>
int launch(const DistillArgs& a, cudaStream_t stream) {
    return a.wait_ns == kWaitLimitNs ? launch_as<TL, TG, kGrad, false>(a, stream) : launch_as<TL, TG, kGrad, true>(a, stream);
}

}  // namespace

int distill_device(const void* logits, bool logits_bf16, int64_t ld, const int32_t* ids, const float* teacher,
                   const float* teacher_lse, const float* dloss, int64_t tokens, int64_t vocab, int64_t k,
                   float temperature, float* loss, void* dlogits, bool grad_bf16, cudaStream_t stream) {
    const DistillArgs a{logits, ld, ids, teacher, teacher_lse, dloss, loss, dlogits, (int)vocab, (int)k, temperature, tokens, 0, 0, 0,
                        head_wait_ns()};
    if (!dlogits)
        return logits_bf16 ? launch<uint16_t, float, false>(a, stream)
                           : launch<float, float, false>(a, stream);
    if (logits_bf16)
        return grad_bf16 ? launch<uint16_t, uint16_t, true>(a, stream)
                         : launch<uint16_t, float, true>(a, stream);
    return grad_bf16 ? launch<float, uint16_t, true>(a, stream) : launch<float, float, true>(a, stream);
}

// The recorded status of the current device, cleared (after the caller's synchronisation).
int distill_take_status(unsigned* word) {
    if (cudaMemcpyFromSymbol(word, g_distill_status, sizeof(unsigned)) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned zero = 0;
    if (*word != 0 && cudaMemcpyToSymbol(g_distill_status, &zero, sizeof(unsigned)) != cudaSuccess) return NQ_ERR_CUDA;
    return NQ_OK;
}

}  // namespace nq
