// nq_q4.cu -- products of a few tokens with a matrix kept at 4 bits per weight:
//     w[i][j] = s[i][j / g] * (c[i][j] - z[i][j / g]),   y[b][i] = sum_j w[i][j] x[b][j],
// codes c in 0 .. 15 (eight to a 32-bit word, row-major), fp16 scales and zero points per
// group of g columns (z = 8 without zero points).  The layers of a decoder that are not
// factorised (a head, a projection that loses too much) are kept in this form.
//
// The product is exact up to its sums: a code minus 8 and an activation are bfloat16
// numbers, so mma.sync m16n8k16 (bf16, fp32 accumulators) multiplies 16 rows x 16 columns
// by up to 8 tokens without rounding, and the scale and zero point are applied in fp32 to
// the accumulators of a finished group: y += s (acc - (z - 8) sum_j x_j), the sum of x over
// the group by one more MMA with a row of ones (only with zero points).
//
// What bounds it: the codes, n / 2 bytes a row, come from HBM once.  A warp owns 16 rows and
// a share of the columns and brings the codes of 256 columns at a time (16 rows x 128 bytes,
// whole cache lines) into its own ring in shared memory with cp.async, so that a CTA keeps
// tens of kilobytes in flight without holding them in registers and no warp waits for
// another before the final sum.  The 16-byte pieces of a row are XOR-swizzled by the row, so
// that the fragment loads (eight rows x four words) touch 32 banks.  The k order inside an
// MMA is free as long as both operands agree: a lane takes word t of a 32-column piece, whose
// nibble pairs (0,4), (1,5), (2,6), (3,7) come out with one LOP3 each, and permutes x to it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nq_internal.cuh"
#include "nq_sm100.cuh"

namespace nq {
namespace {

constexpr int kQWarps = 8;
constexpr int kQThreads = 32 * kQWarps;
constexpr int kQStages = 4;
constexpr int kQCols = 256;                     // columns per stage: one 128-byte line of a row
constexpr int kQStageBytes = 16 * kQCols / 2;   // 16 rows
constexpr int kQSmem = kQWarps * kQStages * kQStageBytes;
constexpr int kQTokens = 8;                     // tokens per CTA (the n of the MMA)

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word (shifted right by 4 i) as two bfloat16 numbers c - 8: the bits
// 0x4300 | c are 128 + c (one unit in the last place at 128 is 1), and 128 + c - 136 is exact.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w) {
    const uint32_t biased = (w & 0x000F000Fu) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x43084308u));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

struct Q4Args {
    const uint16_t* x;       // batch x n bf16
    const uint32_t* W;       // m x n/8
    const uint16_t* scales;  // m x n/g fp16
    const uint16_t* zeros;   // m x n/g fp16 or null
    float* y;                // batch x m
    int64_t m, n, batch;
    int group, ngroups;      // columns per group, groups per row
};

template <bool kZeros>
__global__ void __launch_bounds__(kQThreads) q4_kernel(const Q4Args p) {
    extern __shared__ __align__(128) unsigned char q4_smem[];
    unsigned char(*ring)[kQStages][kQStageBytes] = reinterpret_cast<unsigned char(*)[kQStages][kQStageBytes]>(q4_smem);
    __shared__ float part[kQWarps][16][kQTokens];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int64_t tok0 = (int64_t)blockIdx.y * kQTokens;
    const int nchunks = (int)((p.n + kQCols - 1) / kQCols);
    const int64_t row_bytes = p.n / 2;
    const char* wbase = reinterpret_cast<const char*>(p.W);

    // the warp's chunks are warp, warp + 8, ...: the CTA walks along its rows
    const int mine = warp < nchunks ? (nchunks - warp + kQWarps - 1) / kQWarps : 0;
    auto fetch = [&](int i) {
        if (i < mine) {
            const int chunk = warp + i * kQWarps;
            const uint32_t dst = smem_u32(ring[warp][i % kQStages]);
            const int piece = lane & 7;
            const int64_t byte = (int64_t)chunk * (kQCols / 2) + 16 * piece;
            if (byte < row_bytes) {  // n is a multiple of 128: pieces are whole
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int r = 4 * q + (lane >> 3);
                    const int64_t row = row0 + r < p.m ? row0 + r : p.m - 1;
                    cp_async16(dst + r * 128 + ((piece ^ (r & 7)) << 4), wbase + row * row_bytes + byte);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kQStages - 1; ++i) fetch(i);

    const int64_t ra = row0 + g < p.m ? row0 + g : p.m - 1, rb = row0 + g + 8 < p.m ? row0 + g + 8 : p.m - 1;
    const bool has_token = tok0 + g < p.batch;
    const uint16_t* xrow = p.x + (has_token ? tok0 + g : 0) * p.n;
    const int per_chunk = kQCols / p.group;  // groups in a whole chunk: 8, 4 or 2
    const int pieces_per_group = p.group / 32;

    float out[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < mine; ++i) {
        const int chunk = warp + i * kQWarps;
        const int col0 = chunk * kQCols;
        const int npieces = (int)(p.n - col0 < kQCols ? (p.n - col0) / 32 : kQCols / 32);
        // lane t of a quad holds the scales of the chunk's groups t and t + 4, rows g and g + 8
        float sa[2], sb[2], za[2], zb[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int grp = chunk * per_chunk + t + 4 * q;
            const bool there = t + 4 * q < per_chunk && grp < p.ngroups;
            sa[q] = there ? __half2float(__ushort_as_half(p.scales[ra * p.ngroups + grp])) : 0.f;
            sb[q] = there ? __half2float(__ushort_as_half(p.scales[rb * p.ngroups + grp])) : 0.f;
            if (kZeros) {
                za[q] = there ? __half2float(__ushort_as_half(p.zeros[ra * p.ngroups + grp])) - 8.f : 0.f;
                zb[q] = there ? __half2float(__ushort_as_half(p.zeros[rb * p.ngroups + grp])) - 8.f : 0.f;
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kQStages - 2) : "memory");
        __syncwarp();
        const unsigned char* st = ring[warp][i % kQStages];
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, sx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kQCols / 32; ++j) {
            if (j < npieces) {
                const uint32_t off = (uint32_t)(((j ^ g) << 4) + 4 * t);
                const uint32_t wa = *reinterpret_cast<const uint32_t*>(st + g * 128 + off);
                const uint32_t wb = *reinterpret_cast<const uint32_t*>(st + (g + 8) * 128 + off);
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (has_token) xv = __ldg(reinterpret_cast<const uint4*>(xrow + col0 + 32 * j + 8 * t));
                const uint32_t b04 = __byte_perm(xv.x, xv.z, 0x5410), b15 = __byte_perm(xv.x, xv.z, 0x7632);
                const uint32_t b26 = __byte_perm(xv.y, xv.w, 0x5410), b37 = __byte_perm(xv.y, xv.w, 0x7632);
                mma_bf16(acc, codes_bf16x2(wa), codes_bf16x2(wb), codes_bf16x2(wa >> 4), codes_bf16x2(wb >> 4), b04, b15);
                mma_bf16(acc, codes_bf16x2(wa >> 8), codes_bf16x2(wb >> 8), codes_bf16x2(wa >> 12),
                         codes_bf16x2(wb >> 12), b26, b37);
                if (kZeros) {
                    constexpr uint32_t one = 0x3F803F80u;
                    mma_bf16(sx, one, one, one, one, b04, b15);
                    mma_bf16(sx, one, one, one, one, b26, b37);
                }
                if ((j + 1) % pieces_per_group == 0) {  // the group is complete
                    const int q = j / pieces_per_group, src = (lane & ~3) | (q & 3);
                    const float s0 = __shfl_sync(0xffffffffu, q < 4 ? sa[0] : sa[1], src);
                    const float s1 = __shfl_sync(0xffffffffu, q < 4 ? sb[0] : sb[1], src);
                    if (kZeros) {
                        const float z0 = __shfl_sync(0xffffffffu, q < 4 ? za[0] : za[1], src);
                        const float z1 = __shfl_sync(0xffffffffu, q < 4 ? zb[0] : zb[1], src);
                        acc[0] = fmaf(-z0, sx[0], acc[0]);
                        acc[1] = fmaf(-z0, sx[1], acc[1]);
                        acc[2] = fmaf(-z1, sx[2], acc[2]);
                        acc[3] = fmaf(-z1, sx[3], acc[3]);
                    }
                    out[0] = fmaf(s0, acc[0], out[0]);
                    out[1] = fmaf(s0, acc[1], out[1]);
                    out[2] = fmaf(s1, acc[2], out[2]);
                    out[3] = fmaf(s1, acc[3], out[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = sx[e] = 0.f;
                }
            }
        }
        __syncwarp();  // the stage is free for the fetch below
        fetch(i + kQStages - 1);
    }
    pdl_trigger();

    // the warps' shares of the columns, added in warp order
    part[warp][g][2 * t] = out[0];
    part[warp][g][2 * t + 1] = out[1];
    part[warp][g + 8][2 * t] = out[2];
    part[warp][g + 8][2 * t + 1] = out[3];
    __syncthreads();
    const int e = threadIdx.x;
    if (e < 16 * kQTokens) {
        const int r = e & 15, b = e >> 4;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kQWarps; ++w) sum += part[w][r][b];
        if (row0 + r < p.m && tok0 + b < p.batch) p.y[(tok0 + b) * p.m + row0 + r] = sum;
    }
}

// Eight codes (one byte each) to a word: code j of a row in bits 4 (j % 8) of word j / 8.
__global__ void __launch_bounds__(256) q4_pack_kernel(const uint8_t* __restrict__ codes, int64_t words, int64_t wpr,
                                                      int64_t cols, uint32_t* __restrict__ out, unsigned* flag) {
    bool bad = false;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / wpr, c0 = (i % wpr) * 8;
        uint32_t word = 0;
        for (int b = 0; b < 8 && c0 + b < cols; ++b) {
            const uint32_t c = codes[row * cols + c0 + b];
            bad |= c > 15;
            word |= (c & 15u) << (4 * b);
        }
        out[i] = word;
    }
    if (bad) atomicOr(flag, 1u);
}

// The ring is larger than the shared memory a kernel gets by default: once per device.
template <bool kZeros>
int q4_prepare() {
    static unsigned long long init_mask = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&init_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(q4_kernel<kZeros>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSmem) != cudaSuccess)
            return NQ_ERR_CUDA;
        __atomic_fetch_or(&init_mask, bit, __ATOMIC_RELEASE);
    }
    return NQ_OK;
}

template <bool kZeros>
int q4_launch(const Q4Args& p, cudaStream_t stream) {
    const int rc = q4_prepare<kZeros>();
    if (rc != NQ_OK) return rc;
    const dim3 grid((unsigned)((p.m + 15) / 16), (unsigned)((p.batch + kQTokens - 1) / kQTokens));
    return launch_pdl(q4_kernel<kZeros>, grid, dim3(kQThreads), (size_t)kQSmem, stream, p) == cudaSuccess ? NQ_OK
                                                                                                    : NQ_ERR_CUDA;
}

}  // namespace

int q4_forward(const uint16_t* x, const uint32_t* W, const uint16_t* scales, const uint16_t* zeros, int64_t m,
               int64_t n, int group, int64_t batch, float* y, cudaStream_t stream) {
    const Q4Args p{x, W, scales, zeros, y, m, n, batch, group, (int)(n / group)};
    return zeros ? q4_launch<true>(p, stream) : q4_launch<false>(p, stream);
}

int q4_pack_device(const uint8_t* codes, int64_t rows, int64_t cols, uint32_t* out, unsigned* flag,
                   cudaStream_t stream) {
    const int64_t wpr = (cols + 7) / 8, words = rows * wpr;
    const int64_t blocks = (words + 255) / 256, cap = 16 * (int64_t)sm_count();
    q4_pack_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, stream>>>(codes, words, wpr, cols, out, flag);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace nq
