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
// One CTA per token.  The first pass over the row keeps a running maximum and sum per thread
// (fp32) over the classes outside the list where the list matters (bits in shared memory mark
// it), so p_rest is a sum of its own and never a difference; the listed classes, a handful,
// are added from their own logits.  What the loss is made of (logarithms and the differences
// between them, which nearly cancel when the student is close) is computed in fp64 for the
// listed classes alone.  The second pass reads the row again (from L2, it was just read) and
// writes the gradient as one exponential times one factor per class; the listed classes are
// written last, over it.
#include <cuda_bf16.h>

#include "nq_internal.cuh"

namespace nq {
namespace {

constexpr int kDtThreads = 512;
constexpr int kDtWarps = kDtThreads / 32;
constexpr int kDtMaxK = 1024;

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
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], bool aligned) {
    if (aligned) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = v[i];
    }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], bool aligned) {
    if (aligned) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) store1(p + i, v[i]);
    }
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// (m, s) stands for s 2^(m c); m = -inf: nothing.
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ float or_zero(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m), f = or_zero(m);
    return MaxSum{m, a.s * ex2((a.m - f) * c) + b.s * ex2((b.m - f) * c)};
}

template <typename V, typename Op>
__device__ __forceinline__ V block_reduce(V v, V* shared, V identity, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < kDtWarps ? shared[threadIdx.x & 31] : identity;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;  // the same in every thread
}

template <typename TL, typename TG, bool kGrad>
__global__ void __launch_bounds__(kDtThreads) distill_kernel(const DistillArgs p) {
    extern __shared__ uint32_t mask[];  // bit v - head + 8: class v is listed
    __shared__ double red_d[32];
    __shared__ float red_f[32], red_f2[32];
    __shared__ int32_t sid[kDtMaxK];
    __shared__ float sq[kDtMaxK], sz[kDtMaxK];
    __shared__ unsigned char owner[kDtMaxK];
    __shared__ int dups;
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const TL* z = static_cast<const TL*>(p.logits) + row * p.ld;
    TG* dz = static_cast<TG*>(p.dlogits) + row * p.ld;
    const int V = p.vocab, K = p.k, tid = threadIdx.x;
    const float c = 1.4426950408889634f / p.temperature;
    const bool whole = p.teacher_lse != nullptr;

    const int head0 = (int)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(TL));
    const int head = head0 < V ? head0 : V;  // classes before the row's first 16-byte boundary
    const int groups = (V - head) / 8, tail = head + 8 * groups;
    const int words = (groups * 8 + 8 + 8 + 31) / 32;

    for (int i = tid; i < words; i += kDtThreads) mask[i] = 0;
    if (tid == 0) dups = 0;
    __syncthreads();
    // ---- the teacher's list: bits, owners of a class (its first marker), logits
    double umax = -INFINITY;
    int valid = 0;
    for (int k = tid; k < K; k += kDtThreads) {
        int id = p.ids[row * K + k];
        if (id < 0 || id >= V) id = -1;
        sid[k] = id;
        bool own = false;
        if (id >= 0) {
            const int bit = id - head + 8;
            own = !(atomicOr(&mask[bit >> 5], 1u << (bit & 31)) >> (bit & 31) & 1u);
            if (!own) dups = 1;
            sz[k] = load1(z + id);
            ++valid;
            umax = fmax(umax, (double)p.teacher[row * K + k]);
        }
        owner[k] = own;
    }
    valid = __syncthreads_or(valid);
    if (!valid) {  // nothing to learn from: no loss and no gradient, whatever the logits are
        if (p.loss && tid == 0) p.loss[row] = 0.f;
        if (kGrad)
            for (int64_t v = tid; v < p.ld; v += kDtThreads) store1(dz + v, 0.f);
        return;
    }
    const double invT = 1.0 / (double)p.temperature;
    double shift;  // log q_k = u_k / T - shift
    if (whole) {
        shift = p.teacher_lse[row];
    } else {
        umax = block_reduce(umax, red_d, -(double)INFINITY, [](double a, double b) { return fmax(a, b); });
        double e = 0.0;
        for (int k = tid; k < K; k += kDtThreads)
            if (sid[k] >= 0) e += exp(((double)p.teacher[row * K + k] - umax) * invT);
        e = block_reduce(e, red_d, 0.0, [](double a, double b) { return a + b; });
        shift = umax * invT + log(e);
    }
    double qsum = 0.0;
    for (int k = tid; k < K; k += kDtThreads) {
        double q = 0.0;
        if (sid[k] >= 0) q = exp((double)p.teacher[row * K + k] * invT - shift);
        sq[k] = (float)q;
        qsum += q;
    }
    qsum = block_reduce(qsum, red_d, 0.0, [](double a, double b) { return a + b; });

    // ---- pass 1: running maximum and sum over the classes outside the list
    MaxSum r{-INFINITY, 0.f};
    auto add1 = [&](int v) {
        const int bit = v - head + 8;
        if (mask[bit >> 5] >> (bit & 31) & 1u) return;
        r = join(r, MaxSum{load1(z + v), 1.f}, c);
    };
    if (tid < head) add1(tid);
    if (tail + tid < V) add1(tail + tid);
    const unsigned char* bytes = reinterpret_cast<const unsigned char*>(mask);
    for (int i = tid; i < groups; i += kDtThreads) {
        float v[8];
        load8(z + head + 8 * i, v);
        const unsigned listed = bytes[i + 1];
        if (listed) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (listed >> j & 1u) v[j] = -INFINITY;
        }
        float m = r.m;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, v[j]);
        const float f = or_zero(m);
        float s = r.s * ex2((r.m - f) * c);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += ex2((v[j] - f) * c);
        r = MaxSum{m, s};
    }
    const float mr = block_reduce(r.m, red_f, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
    const float sr = block_reduce(r.s * ex2((r.m - or_zero(mr)) * c), red_f2, 0.f, [](float a, float b) { return a + b; });
    // the listed classes, each once
    MaxSum l{-INFINITY, 0.f};
    for (int k = tid; k < K; k += kDtThreads)
        if (owner[k]) l = join(l, MaxSum{sz[k], 1.f}, c);
    const float ml = block_reduce(l.m, red_f, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
    const float sl = block_reduce(l.s * ex2((l.m - or_zero(ml)) * c), red_f2, 0.f, [](float a, float b) { return a + b; });
    // their union: in fp64, since one exponential's error would shift every logarithm below
    const float m = fmaxf(mr, ml);
    const double sum = (mr > -INFINITY ? sr * exp(((double)mr - m) * invT) : 0.0) +
                       (ml > -INFINITY ? sl * exp(((double)ml - m) * invT) : 0.0);

    const double qrest = whole && mr > -INFINITY ? fmax(0.0, 1.0 - qsum) : 0.0;
    if (p.loss) {
        const double logsum = log(sum);  // log p_v = (z_v - m) / T - logsum
        double part = 0.0;
        for (int k = tid; k < K; k += kDtThreads) {
            const double lq = (double)p.teacher[row * K + k] * invT - shift;
            if (sid[k] >= 0 && sq[k] > 0.f) part += exp(lq) * (lq - (((double)sz[k] - m) * invT - logsum));
        }
        part = block_reduce(part, red_d, 0.0, [](double a, double b) { return a + b; });
        if (tid == 0) {
            if (qrest > 0.0) part += qrest * (log(qrest) - (((double)mr - m) * invT + log((double)sr) - logsum));
            p.loss[row] = (float)(part * (double)p.temperature * (double)p.temperature);
        }
    }
    if constexpr (kGrad) {
        // outside the list dz_v = 2^((z_v - mr) c) (tot 2^((mr - m) c) / sum - qrest / sr) T dloss
        const float gT = p.temperature * p.dloss[row];
        // (the two nearly cancel when the student is close: in fp64)
        const float base = or_zero(mr), scale = (float)((qsum + qrest) * gT / sum);
        const float factor =
            mr > -INFINITY ? (float)((exp(((double)mr - m) * invT) * (qsum + qrest) / sum - qrest / sr) * gT) : 0.f;
        const bool aligned = (reinterpret_cast<uintptr_t>(dz + head) & 15) == 0;
        auto put1 = [&](int v) { store1(dz + v, ex2((load1(z + v) - base) * c) * factor); };
        if (tid < head) put1(tid);
        if (tail + tid < V) put1(tail + tid);
        for (int64_t v = (int64_t)V + tid; v < p.ld; v += kDtThreads) store1(dz + v, 0.f);
        for (int i = tid; i < groups; i += kDtThreads) {
            float v[8];
            load8(z + head + 8 * i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = ex2((v[j] - base) * c) * factor;
            store8(dz + head + 8 * i, v, aligned);
        }
        __syncthreads();
        for (int k = tid; k < K; k += kDtThreads) {
            if (!owner[k]) continue;
            float q = sq[k];
            if (dups) {  // the class may be listed again: its masses add, in the list's order
                q = 0.f;
                for (int j = 0; j < K; ++j)
                    if (sid[j] == sid[k]) q += sq[j];
            }
            store1(dz + sid[k], ex2((sz[k] - m) * c) * scale - q * gT);
        }
    }
}

template <typename TL, typename TG, bool kGrad>
int launch(const DistillArgs& a, int64_t tokens, cudaStream_t stream) {
    static unsigned long long init_mask = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&init_mask, __ATOMIC_ACQUIRE) & bit)) {
        // the mask of the largest vocabulary (2^20 classes)
        if (cudaFuncSetAttribute(distill_kernel<TL, TG, kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (1 << 20) / 8 + 64) != cudaSuccess)
            return NQ_ERR_CUDA;
        __atomic_fetch_or(&init_mask, bit, __ATOMIC_RELEASE);
    }
    const size_t smem = ((size_t)a.vocab + 16 + 31) / 32 * 4 + 16;
    return launch_pdl(distill_kernel<TL, TG, kGrad>, dim3((unsigned)tokens), dim3(kDtThreads), smem, stream, a) ==
                   cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

}  // namespace

int distill_device(const void* logits, bool logits_bf16, int64_t ld, const int32_t* ids, const float* teacher,
                   const float* teacher_lse, const float* dloss, int64_t tokens, int64_t vocab, int64_t k,
                   float temperature, float* loss, void* dlogits, bool grad_bf16, cudaStream_t stream) {
    const DistillArgs a{logits, ld, ids, teacher, teacher_lse, dloss, loss, dlogits, (int)vocab, (int)k, temperature};
    if (!dlogits)
        return logits_bf16 ? launch<uint16_t, float, false>(a, tokens, stream)
                           : launch<float, float, false>(a, tokens, stream);
    if (logits_bf16)
        return grad_bf16 ? launch<uint16_t, uint16_t, true>(a, tokens, stream)
                         : launch<uint16_t, float, true>(a, tokens, stream);
    return grad_bf16 ? launch<float, uint16_t, true>(a, tokens, stream) : launch<float, float, true>(a, tokens, stream);
}

}  // namespace nq
