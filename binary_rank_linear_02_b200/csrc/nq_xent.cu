// nq_xent.cu -- cross entropy of a dense output head without its logits in memory, and its
// gradients.  For tokens h (N x d, bfloat16), head W (V x d, bfloat16) and labels:
//     z = h W^T,  lse_i = log sum_v exp(z_iv),  loss_i = lse_i - z_i,label(i),
//     dz_iv = dloss_i (exp(z_iv - lse_i) - [v = label(i)]),  dh = dz W,  dW = dz^T h.
//
// The logits exist only as accumulators in tensor memory.  Forward: each 128 x 128 tile of z
// is reduced in its epilogue to a maximum and a sum of exponentials per row (fp32), and a
// second kernel joins a row's tiles in order.  Backward: the vocabulary is taken in pieces;
// a piece's z is computed again, its epilogue writes dz as bfloat16 into a scratch of bounded
// size, and two products read it: the piece's rows of dW (complete, since they sum over the
// tokens) and its share of dh (summed over the pieces in fp32, in order).  dz in bfloat16 is
// what lets both products run on the bf16 tensor cores (an operand pair has one type): its
// rounding is 2^-9 of each term, of the same size as the rounding of the bfloat16 results.
//
// All four products are the same tcgen05 kernel (kind::f16, bf16 operands, fp32 accumulators)
// with other operand orders and epilogues: dW reads dz and h token-major (MN-major tiles), dh
// reads W's rows as MN-major tiles, so nothing is transposed in memory.  Sizes need not be
// multiples of the tile: TMA fills with zeros outside, epilogues mask.
#include <cuda.h>
#include <cuda_bf16.h>

#include "nq_internal.cuh"
#include "nq_sm100.cuh"

namespace nq {
namespace {

constexpr int kXM = 128, kXN = 128, kXK = 64;
constexpr int kXStages = 3;
constexpr int kXTileBytes = kXM * kXK * 2;
constexpr int kXStageBytes = 2 * kXTileBytes;
constexpr int kXHalf = kXTileBytes / 2;  // one TMA box of an MN-major tile: 64 rows x 64 elements
constexpr int kXThreads = 192;
constexpr int kXSmem = kXStages * kXStageBytes + 1024 + 1024;
constexpr int64_t kXPieceBytes = int64_t(256) << 20;  // scratch for dz

// A device-side wait that gave up (NQ_ERR_TIMEOUT) is recorded here; nq_device_status reads it.
__device__ unsigned g_xent_status;

__host__ __device__ constexpr uint32_t xent_idesc(bool amn, bool bmn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((amn ? 1u : 0u) << 15) | ((bmn ? 1u : 0u) << 16) |
           ((uint32_t)(kXN >> 3) << 17) | ((uint32_t)(kXM >> 4) << 24);
}

// SW128 MN-major operand descriptor: rows of 64 elements along K, 8-row groups 1024 B apart,
// the next 64 elements of M (or N) one box further.
__device__ __forceinline__ uint64_t xent_desc_mn(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(kXHalf >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

struct XentBarriers {
    unsigned long long full[kXStages], empty[kXStages];
    unsigned long long tmem_full, drain;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ float xent_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

enum { kStats = 0, kDz = 1, kToBf16 = 2, kAccumulate = 3 };

struct XentEpilogue {
    int64_t rows, cols;     // of the product (unpadded)
    const int32_t* labels;  // kStats, kDz: per row
    int64_t label0, vocab;  // first class of the columns; all classes
    float2* stats;          // kStats: [column tile][row]: maximum, sum of exp(z - maximum)
    float* picked;          // kStats: z of the label, per row
    const float* lse;       // kDz
    const float* dloss;     // kDz
    uint16_t* out;          // kDz, kToBf16, kAccumulate's last piece: bf16
    float* acc;             // kAccumulate: fp32 sums, pitch = cols
    int64_t ldo;
    int first, last;        // kAccumulate
};

__device__ __forceinline__ uint32_t xent_pack(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// 32 values of a row as bf16 at out[0 .. 31], the first n of them (out 16-byte aligned when whole).
__device__ __forceinline__ void xent_store32(uint16_t* out, const float (&v)[32], int n) {
    if (n >= 32 && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4*>(out + j) = make_uint4(xent_pack(v[j], v[j + 1]), xent_pack(v[j + 2], v[j + 3]),
                                                            xent_pack(v[j + 4], v[j + 5]), xent_pack(v[j + 6], v[j + 7]));
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n) out[j] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
    }
}

template <int kEpi, bool AMN, bool BMN>
__global__ void __launch_bounds__(kXThreads, 2)
xent_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, int nkb,
                 const XentEpilogue e) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    XentBarriers& bar = *reinterpret_cast<XentBarriers*>(smem_raw + (base - raw) + kXStages * kXStageBytes);
    volatile int* abort_flag = &bar.abort_flag;
    unsigned* status = &g_xent_status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = blockIdx.x * kXM, n0 = blockIdx.y * kXN;

    if (threadIdx.x == 0) {
        for (int st = 0; st < kXStages; ++st) {
            mbar_init(smem_u32(&bar.full[st]), 1);
            mbar_init(smem_u32(&bar.empty[st]), 1);
        }
        mbar_init(smem_u32(&bar.tmem_full), 1);
        mbar_init(smem_u32(&bar.drain), 1);
        bar.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&bar.tmem_base)), "r"((uint32_t)kXN));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int kb = 0; kb < nkb; ++kb) {
                const int st = kb % kXStages;
                const uint32_t ph = (uint32_t)(kb / kXStages) & 1u;
                if (!mbar_wait(smem_u32(&bar.empty[st]), ph ^ 1u, abort_flag, status)) break;
                const uint32_t full = smem_u32(&bar.full[st]);
                mbar_expect_tx(full, (uint32_t)kXStageBytes);
                const uint32_t dst = base + (uint32_t)(st * kXStageBytes);
                if constexpr (AMN) {
                    tma_load_2d(dst, &amap, m0, kb * kXK, full);
                    tma_load_2d(dst + kXHalf, &amap, m0 + 64, kb * kXK, full);
                } else {
                    tma_load_2d(dst, &amap, kb * kXK, m0, full);
                }
                if constexpr (BMN) {
                    tma_load_2d(dst + kXTileBytes, &bmap, n0, kb * kXK, full);
                    tma_load_2d(dst + kXTileBytes + kXHalf, &bmap, n0 + 64, kb * kXK, full);
                } else {
                    tma_load_2d(dst + kXTileBytes, &bmap, kb * kXK, n0, full);
                }
                ++issued;
            }
            if (*abort_flag) {
                for (int kb = issued - kXStages < 0 ? 0 : issued - kXStages; kb < issued; ++kb)
                    mbar_drain(smem_u32(&bar.full[kb % kXStages]), (uint32_t)(kb / kXStages) & 1u);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = xent_idesc(AMN, BMN);
            int kb = 0;
            for (; kb < nkb; ++kb) {
                const int st = kb % kXStages;
                const uint32_t ph = (uint32_t)(kb / kXStages) & 1u;
                if (!mbar_wait(smem_u32(&bar.full[st]), ph, abort_flag, status)) break;
                tc_fence_after();
                const uint32_t aaddr = base + (uint32_t)(st * kXStageBytes), baddr = aaddr + kXTileBytes;
                const uint64_t ad = AMN ? xent_desc_mn(aaddr) : sw128_desc(aaddr);
                const uint64_t bd = BMN ? xent_desc_mn(baddr) : sw128_desc(baddr);
                constexpr uint64_t astep = AMN ? 2048 / 16 : 32 / 16, bstep = BMN ? 2048 / 16 : 32 / 16;
#pragma unroll
                for (int k = 0; k < kXK / 16; ++k)
                    umma_f16(tmem, ad + (uint64_t)k * astep, bd + (uint64_t)k * bstep, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                umma_commit(smem_u32(&bar.empty[st]));
            }
            if (kb == nkb) {
                umma_commit(smem_u32(&bar.tmem_full));
            } else {
                umma_commit(smem_u32(&bar.drain));
                mbar_drain(smem_u32(&bar.drain), 0);
            }
        }
    } else {
        if (mbar_wait(smem_u32(&bar.tmem_full), 0, abort_flag, status)) {
            tc_fence_after();
            pdl_trigger();
            const int quad = warp & 3;
            const int64_t row = m0 + quad * 32 + lane;
            const bool there = row < e.rows;
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16);
            int64_t label = -1;
            float lse2 = 0.f, dl = 0.f;
            if constexpr (kEpi == kStats || kEpi == kDz) {
                label = there ? (int64_t)e.labels[row] : -1;
                if (label >= e.vocab) label = -1;
            }
            if constexpr (kEpi == kDz) {
                lse2 = there ? e.lse[row] * kLog2e : 0.f;
                dl = there && label >= 0 ? e.dloss[row] : 0.f;
            }
            float m = -INFINITY, s = 0.f;
#pragma unroll 1
            for (int c0 = 0; c0 < kXN; c0 += 32) {
                uint32_t w[32];
                tmem_ld32(taddr + (uint32_t)c0, w);
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
                const int64_t left = e.cols - n0 - c0;
                const int n = left < 32 ? (int)(left < 0 ? 0 : left) : 32;
                const int64_t at = label - e.label0 - n0 - c0;  // the label's column in this block, if it is in it
                if constexpr (kEpi == kStats) {
                    float mm = m;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j >= n) v[j] = -INFINITY;
                        mm = fmaxf(mm, v[j]);
                        if (j == at && label >= 0) e.picked[row] = v[j];
                    }
                    const float f = mm == -INFINITY ? 0.f : mm;
                    s *= xent_ex2((m - f) * kLog2e);
#pragma unroll
                    for (int j = 0; j < 32; ++j) s += xent_ex2((v[j] - f) * kLog2e);
                    m = mm;
                } else if constexpr (kEpi == kDz) {
                    if (there) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float q = xent_ex2(fmaf(v[j], kLog2e, -lse2)) - (j == at && label >= 0 ? 1.f : 0.f);
                            v[j] = dl != 0.f ? q * dl : 0.f;
                        }
                        xent_store32(e.out + row * e.ldo + n0 + c0, v, n);
                    }
                } else if constexpr (kEpi == kToBf16) {
                    if (there) xent_store32(e.out + row * e.ldo + n0 + c0, v, n);
                } else {
                    if (there) {
                        float* a = e.acc + row * e.cols + n0 + c0;
                        if (!e.first) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j < n) v[j] += a[j];
                        }
                        if (e.last) {
                            xent_store32(e.out + row * e.ldo + n0 + c0, v, n);
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j < n) a[j] = v[j];
                        }
                    }
                }
            }
            if constexpr (kEpi == kStats) {
                if (there) e.stats[(int64_t)blockIdx.y * e.rows + row] = make_float2(m, s);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)kXN));
    }
}

// A warp per token joins the tiles' (maximum, sum) pairs: lane l takes tiles l, l + 32, ... in
// order, then the lanes join in a tree (a fixed order).
__global__ void __launch_bounds__(256) xent_join_kernel(const float2* __restrict__ stats, const float* __restrict__ picked,
                                                        const int32_t* __restrict__ labels, int64_t tokens,
                                                        int64_t vocab, int tiles, float* __restrict__ loss,
                                                        float* __restrict__ lse) {
    pdl_wait();
    const int64_t row = blockIdx.x * (int64_t)(blockDim.x / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= tokens) return;
    float m = -INFINITY, s = 0.f;
    for (int t = lane; t < tiles; t += 32) {
        const float2 p = stats[(int64_t)t * tokens + row];
        const float mm = fmaxf(m, p.x), f = mm == -INFINITY ? 0.f : mm;
        s = s * xent_ex2((m - f) * kLog2e) + p.y * xent_ex2((p.x - f) * kLog2e);
        m = mm;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        const float mm = fmaxf(m, m2), f = mm == -INFINITY ? 0.f : mm;
        s = s * xent_ex2((m - f) * kLog2e) + s2 * xent_ex2((m2 - f) * kLog2e);
        m = mm;
    }
    if (lane == 0) {
        const float logs = logf(s);
        lse[row] = m + logs;
        const int32_t label = labels[row];
        // (m - z) + log s: exact difference first
        loss[row] = label >= 0 && label < vocab ? (m - picked[row]) + logs : 0.f;
    }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Boxes of 64 elements x box_rows of a row-major bf16 matrix, 128-byte swizzle, zeros outside.
bool xent_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
    static EncodeFn fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        fn = reinterpret_cast<EncodeFn>(p);
    }
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(pitch * 2)};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kEpi, bool AMN, bool BMN>
int xent_launch(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, int64_t M, int64_t N, int64_t K,
                const XentEpilogue& e, cudaStream_t stream) {
    static unsigned long long init_mask = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&init_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(xent_gemm_kernel<kEpi, AMN, BMN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmem) !=
            cudaSuccess)
            return NQ_ERR_CUDA;
        __atomic_fetch_or(&init_mask, bit, __ATOMIC_RELEASE);
    }
    CUtensorMap amap, bmap;
    if (!(AMN ? xent_map(&amap, A, K, M, lda, 64) : xent_map(&amap, A, M, K, lda, kXM)) ||
        !(BMN ? xent_map(&bmap, B, K, N, ldb, 64) : xent_map(&bmap, B, N, K, ldb, kXN)))
        return NQ_ERR_CUDA;
    const dim3 grid((unsigned)((M + kXM - 1) / kXM), (unsigned)((N + kXN - 1) / kXN));
    return launch_pdl(xent_gemm_kernel<kEpi, AMN, BMN>, grid, dim3(kXThreads), (size_t)kXSmem, stream, amap, bmap,
                      (int)((K + kXK - 1) / kXK), e) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t tiles_n(int64_t v) { return (v + kXN - 1) / kXN; }

// Classes per piece of the backward: as many whole column tiles as dz's scratch holds.
int64_t piece_classes(int64_t tokens, int64_t vocab) {
    const int64_t fit = kXPieceBytes / (2 * tokens) / kXN * kXN;
    const int64_t all = round_up(vocab, kXN);
    return fit < kXN ? kXN : fit < all ? fit : all;
}

}  // namespace

int64_t xent_fwd_scratch_bytes(int64_t tokens, int64_t vocab) {
    return round_up(8 * tokens * tiles_n(vocab), 256) + round_up(4 * tokens, 256);
}

int64_t xent_bwd_scratch_bytes(int64_t tokens, int64_t vocab, int64_t d) {
    const int64_t piece = piece_classes(tokens, vocab);
    return round_up(2 * tokens * piece, 256) + (piece < vocab ? round_up(4 * tokens * d, 256) : 0);
}

int xent_forward(const uint16_t* h, const uint16_t* W, const int32_t* labels, int64_t tokens, int64_t vocab, int64_t d,
                 float* loss, float* lse, void* scratch, cudaStream_t stream) {
    XentEpilogue e = {};
    e.rows = tokens;
    e.cols = e.vocab = vocab;
    e.labels = labels;
    e.stats = static_cast<float2*>(scratch);
    e.picked = reinterpret_cast<float*>(static_cast<char*>(scratch) + round_up(8 * tokens * tiles_n(vocab), 256));
    const int rc = xent_launch<kStats, false, false>(h, d, W, d, tokens, vocab, d, e, stream);
    if (rc != NQ_OK) return rc;
    return launch_pdl(xent_join_kernel, dim3((unsigned)((tokens + 7) / 8)), dim3(256), 0, stream,
                      (const float2*)e.stats, (const float*)e.picked, labels, tokens, vocab, (int)tiles_n(vocab), loss,
                      lse) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

int xent_backward(const uint16_t* h, const uint16_t* W, const int32_t* labels, const float* lse, const float* dloss,
                  int64_t tokens, int64_t vocab, int64_t d, uint16_t* dh, uint16_t* dW, void* scratch,
                  cudaStream_t stream) {
    const int64_t piece = piece_classes(tokens, vocab);
    uint16_t* dz = static_cast<uint16_t*>(scratch);
    float* acc = reinterpret_cast<float*>(static_cast<char*>(scratch) + round_up(2 * tokens * piece, 256));
    for (int64_t v0 = 0; v0 < vocab; v0 += piece) {
        const int64_t nv = vocab - v0 < piece ? vocab - v0 : piece;
        XentEpilogue e = {};
        e.rows = tokens;
        e.cols = nv;
        e.labels = labels;
        e.label0 = v0;
        e.vocab = vocab;
        e.lse = lse;
        e.dloss = dloss;
        e.out = dz;
        e.ldo = piece;
        int rc = xent_launch<kDz, false, false>(h, d, W + v0 * d, d, tokens, nv, d, e, stream);
        if (rc != NQ_OK) return rc;
        if (dW) {
            XentEpilogue g = {};
            g.rows = nv;
            g.cols = d;
            g.out = dW + v0 * d;
            g.ldo = d;
            rc = xent_launch<kToBf16, true, true>(dz, piece, h, d, nv, d, tokens, g, stream);
            if (rc != NQ_OK) return rc;
        }
        if (dh) {
            XentEpilogue g = {};
            g.rows = tokens;
            g.cols = d;
            g.out = dh;
            g.ldo = d;
            g.acc = acc;
            g.first = v0 == 0;
            g.last = v0 + piece >= vocab;
            rc = xent_launch<kAccumulate, false, true>(dz, piece, W + v0 * d, d, tokens, d, nv, g, stream);
            if (rc != NQ_OK) return rc;
        }
    }
    return NQ_OK;
}

// The recorded status of the current device, cleared (after the caller's synchronisation).
int xent_take_status(unsigned* word) {
    if (cudaMemcpyFromSymbol(word, g_xent_status, sizeof(unsigned)) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned zero = 0;
    if (*word != 0 && cudaMemcpyToSymbol(g_xent_status, &zero, sizeof(unsigned)) != cudaSuccess) return NQ_ERR_CUDA;
    return NQ_OK;
}

}  // namespace nq
