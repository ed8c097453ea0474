// nq_q4.cu -- products of a few tokens with a matrix kept at 4 bits per weight:
//     w[i][j] = s[i][j / g] * (c[i][j] - z[i][j / g]),   y[b][i] = sum_j w[i][j] x[b][j],
// codes c in 0 .. 15 (eight to a 32-bit word, row-major), fp16 scales and zero points per
// group of g columns (z = 8 without zero points).  The layers of a decoder that are not
// factorised (a head, a projection that loses too much) are kept in this form.
//
// The products are exact, the sums fp32: mma.sync m16n8k16 (bf16, fp32 accumulators)
// multiplies 16 rows x 16 columns by up to 8 tokens, and scale and zero point are applied in
// fp32 to a finished group: y += s (sum_j c_j x_j - z sum_j x_j).
//
// What bounds it: the codes, n / 2 bytes a row, come from HBM once; next to that, the
// instructions that make operands of them.  A code needs one AND: the 8 low bits of a bfloat16
// number with nothing above them are its value times 2^-133 (the subnormal numbers and the
// first normal ones lie on one line, and the tensor cores honour both), so of a word's nibble
// pairs (0,4), (1,5), (2,6), (3,7) the first two are operands as they lie under a mask, the
// second two after one shift by 8, and nibbles 1 and 3 count 16 times their code, for which x
// is divided by 16.  (Codes moved into normal numbers and centred took 11 instructions a word
// in place of 5, and the kernel 57 us in place of ~25 at 28672 x 8192, 8 tokens.)  The factor
// 2^-133 is met by x: each group of a token carries a power of two that brings its largest
// value near the top of bfloat16's range; multiplying by it is exact, and undone in fp32.
//
// Everything else is kept out of the inner loop.  x is brought to shared memory once per CTA,
// scaled and in the order of the codes' bits, with its sums per group, and stays there for all
// rows of the CTA (one per SM).  The codes come in stages of 16 rows x 2048 columns (or some 16
// rows of a narrow matrix), each by one TMA instruction: a three-dimensional map whose box is
// 64 bytes x 16 rows x 16 such pieces of the rows, 64-byte swizzle, which lands as 16 blocks of
// 16 rows x 128 columns, two for each of 8 warps, whose fragment loads then touch 32 banks; two
// such teams of warps take the stages in turn (one block a warp and stage cost 5 to 10% of the time,
// in waits and addresses).
// (Loads into registers, from the same rows, stayed at 3 to 3.9 TB/s however many were in
// flight, bulk copies of 1 KB at 3.4; these reach 6.1 with four stages.)  Scales and zero points
// come beside them by the fetching warp's cp.async, as wide as the rows' alignment allows.
// (Loaded by the warps that use them, a block ahead, they cost 8 to 10 us at the sizes below: a
// block's time is less than DRAM's latency.)  A tile's shares are
// added up by four of the warps, in turns, a tile later, when all have long been written: a
// meeting of the warps after every tile took half of the kernel's time.  Where the tokens' x is
// more than the shared memory holds, the columns are taken in panels and the rows' sums are
// kept between them.
//
// Measured: 32001 x 4096 (groups of 64 with zero points), 1 token: 24 us, 3.05 TB/s; 28672 x 8192
// (groups of 128), 8 tokens: 37 us, 3.3 TB/s.  Of these a third does not grow with the matrix (x, launch, the
// pipeline's start: twice the rows take 27 us more under a profiler where the first take 41); in between it is
// 4.5 TB/s and some 145 instructions, waits' polling included, per 16 x 128 weights, 2.3 of 4 a clock: not HBM,
// not issue, not shared memory (half of its wavefronts) but the latency of dependent instructions, which four
// warps a scheduler do not cover.  Every 8 tokens read and expand the codes again: 16 tokens 61 us, 1024
// 3.6 ms.  Small matrices take 5 us on the device.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nq_internal.cuh"
#include "nq_sm100.cuh"

namespace nq {
namespace {

constexpr int kQWarps = 16;                      // that multiply; one more fetches
constexpr int kQThreads = 32 * (kQWarps + 1);
constexpr int kQCols = 128;                      // columns of a warp's block of a stage
constexpr int kQBlockBytes = 16 * kQCols / 2;    // 16 rows x 64 bytes
constexpr int kQStageCols = kQWarps * kQCols;
constexpr int kQCodeBytes = kQWarps * kQBlockBytes;
constexpr int kQMaxStages = 8, kQMinStages = 4;  // an even number: a place of the ring is always the same team's
constexpr int kQParts = 3;                       // sets whose shares wait to be added
constexpr int kQTeam = kQWarps / 2;              // warps that share a stage, two blocks each
constexpr int kQAdders = 4;                      // warps that add a set's shares
constexpr int kQTokens = 8;                      // tokens per CTA (the n of the MMA)
constexpr int kQSpace = 201 * 1024;              // dynamic shared memory, at most
constexpr int kQPanelSets = 24;                  // sets per CTA whose sums are kept between panels

// A device-side wait that gave up (NQ_ERR_TIMEOUT) is recorded here; nq_device_status reads it.
__device__ unsigned g_q4_status;

// d = a b, and d += a b
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float low_half(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)v)); }
__device__ __forceinline__ float high_half(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)(v >> 16))); }
__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ float sum_bf16(uint32_t v) { return fmaf(high_bf16(v), 0x1p-16f, low_bf16(v) * 0x1p-16f); }  // 2^-16 of it

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 1, 2 or 4 consecutive halves in shared memory, and one of them as a float.
template <int kCount>
__device__ __forceinline__ uint2 lds_halves(uint32_t addr) {
    uint2 v = make_uint2(0, 0);
    if constexpr (kCount == 1) {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
        v.x = h;
    } else if constexpr (kCount == 2) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.x) : "r"(addr));
    } else {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    }
    return v;
}
__device__ __forceinline__ float one_half(uint2 v, int q) {
    const uint32_t w = q < 2 ? v.x : v.y;
    return q % 2 ? high_half(w) : low_half(w);
}

struct Q4Args {
    const uint16_t* x;       // batch x n bf16
    const uint16_t* scales;  // m x n/g fp16
    const uint16_t* zeros;   // m x n/g fp16 or null
    float* y;                // batch x m
    int64_t m, n, batch;
    int tps, blocks;         // tiles of 16 rows in a stage (a set), blocks of 128 columns of each
    int stages;              // of the ring
    int scale_copy;          // bytes of a copy of scales: 16, 8 or 4 (2: rows of an odd number of them, in fours)
    int scale_pitch;         // bytes between rows of a stage's scales
    int panel;               // columns whose x is in shared memory at a time (all, or a multiple of 2048)
    unsigned long long wait_ns;  // how long a wait lasts
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int width) {
    if (width == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (width == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// A stage's scales where the plain copies do not do: the last rows, the end of a row, rows of an
// odd number of scales (every second one begins between two 4-byte boundaries).  In copies of 4
// bytes, the array's last one of 2 where that is all there is.
__device__ __noinline__ void copy_scales_clipped(const uint16_t* scales, uint32_t dst, int row0, int group0, int stage_groups,
                                                 int rows, int ngroups, const Q4Args& p, int lane) {
    const int here = ngroups - group0 < stage_groups ? ngroups - group0 : stage_groups;
    const int words = here / 2 + 1;
    const char* base = reinterpret_cast<const char*>(scales);
    const int64_t end = 2 * p.m * ngroups;
    for (int e = lane; e < rows * words; e += 32) {
        const int r = e / words, w = e - r * words;
        if (row0 + r >= p.m) break;
        const int64_t start = 2 * ((int64_t)(row0 + r) * ngroups + group0), at = (start & ~(int64_t)3) + 4 * w;
        if (at >= start + 2 * here) continue;
        const int size = end - at < 4 ? 2 : 4;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                     ::"r"(dst + (uint32_t)(r * p.scale_pitch + 4 * w)), "l"(base + at), "r"(size) : "memory");
    }
}

template <int kGroup, bool kZeros>
__global__ void __launch_bounds__(kQThreads, 1)
q4_kernel(const __grid_constant__ CUtensorMap wmap, const Q4Args p) {
    constexpr int kPerBlock = kQCols / kGroup;  // groups in a block: 4, 2 or 1
    constexpr int kPieces = kGroup / 32;        // 32-column pieces per group
    extern __shared__ unsigned char smem_raw[];
    __shared__ float part[kQParts][kQWarps][16][kQTokens];
    __shared__ unsigned long long full[kQMaxStages], empty[kQMaxStages], written[kQParts], added[kQParts];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&full[i]), 33);  // the codes' bytes, and the fetching lanes' copies of scales
            mbar_init(smem_u32(&empty[i]), kQTeam);
        }
        for (int i = 0; i < kQParts; ++i) {
            mbar_init(smem_u32(&written[i]), kQWarps);
            mbar_init(smem_u32(&added[i]), kQAdders);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&wmap)) : "memory");
    }
    __syncthreads();
    pdl_wait();
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const int scale_bytes = 16 * p.tps * p.scale_pitch;  // of a stage; as many zero points follow
    const uint32_t scales_at = base + (uint32_t)(p.stages * kQCodeBytes), scale_stage = (uint32_t)(kZeros ? 2 : 1) * scale_bytes;
    unsigned char* xs = smem_raw + (base - raw) + p.stages * (kQCodeBytes + (int)scale_stage);
    const int64_t tok0 = (int64_t)blockIdx.y * kQTokens;
    const int ntok = p.batch - tok0 < kQTokens ? (int)(p.batch - tok0) : kQTokens, pairs = (ntok + 1) / 2;
    const int ngroups = (int)(p.n / kGroup), blocks_all = (int)(p.n / kQCols), set_rows = 16 * p.tps;
    const int all_sets = (int)((p.m + set_rows - 1) / set_rows);
    const int sets = (all_sets - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // blockIdx.x, + gridDim.x, ...
    const int panels = (int)((p.n + p.panel - 1) / p.panel), panel_blocks = p.panel / kQCols;
    const int pitch = 2 * p.panel + 64;  // bytes of a token's x: two tokens' 64 bytes hit different banks
    float4* sums = reinterpret_cast<float4*>(xs + ntok * pitch);  // [group of the panel][pair of tokens]: scale, sum, scale, sum
    float* kept = reinterpret_cast<float*>(sums + p.panel / kGroup * pairs);  // panels > 1: [set][row][token]
    auto stages_in = [&](int panel) {  // of a set
        const int left = blocks_all - panel * panel_blocks;
        return ((left < panel_blocks ? left : panel_blocks) + p.blocks - 1) / p.blocks;
    };

    if (warp == kQWarps) {
        // A lane's copies of a whole stage's scales: from where in the rows, to where.
        constexpr int kCopies = 8;
        const int row_bytes = 2 * ngroups, stage_groups = (p.blocks < blocks_all ? p.blocks : blocks_all) * kPerBlock, width = p.scale_copy;
        const int per_row = width == 2 ? 1 : 2 * stage_groups / width, copies = set_rows * per_row;
        int from[kCopies], to[kCopies];
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int e = lane + 32 * i, r = e / per_row, w = e - r * per_row;
            from[i] = r * row_bytes + w * width;
            to[i] = r * p.scale_pitch + w * width;
        }
        int it = 0, st = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int panel = 0; panel < panels && ok; ++panel) {
            const int per_set = stages_in(panel);
            for (int set = 0; set < sets && ok; ++set) {
                const int row = (int)(blockIdx.x + set * gridDim.x) * set_rows;
                for (int k = 0; k < per_set; ++k, ++it) {
                    // the stage is free, and (a lane sees to it) what was last fetched into it has landed: a
                    // warp that gave up frees stages without having waited for them
                    ok = mbar_wait(smem_u32(lane == 31 ? &full[st] : &empty[st]), phase ^ 1u, abort_flag, &g_q4_status, p.wait_ns);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&full[st]);
                    if (lane == 0) {
                        mbar_expect_tx(bar, (uint32_t)(p.tps * p.blocks * kQBlockBytes));
                        tma_load_3d(base + (uint32_t)(st * kQCodeBytes), &wmap, 0, row, panel * panel_blocks + k * p.blocks, bar);
                    }
                    const int group0 = (panel * panel_blocks + k * p.blocks) * kPerBlock;
                    const int64_t at = (int64_t)row * row_bytes + 2 * group0;
                    const uint32_t dst = scales_at + (uint32_t)st * scale_stage;
                    if (row + set_rows <= p.m && group0 + stage_groups <= ngroups && width > 2 && copies <= 32 * kCopies) {
                        const char* s = reinterpret_cast<const char*>(p.scales) + at;
                        const char* z = reinterpret_cast<const char*>(p.zeros) + at;
#pragma unroll
                        for (int i = 0; i < kCopies; ++i) {
                            if (32 * i >= copies) break;
                            if (lane + 32 * i < copies) {
                                copy_async(dst + to[i], s + from[i], width);
                                if constexpr (kZeros) copy_async(dst + scale_bytes + to[i], z + from[i], width);
                            }
                        }
                    } else {
                        copy_scales_clipped(p.scales, dst, row, group0, stage_groups, set_rows, ngroups, p, lane);
                        if constexpr (kZeros)
                            copy_scales_clipped(p.zeros, dst + scale_bytes, row, group0, stage_groups, set_rows, ngroups, p, lane);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
                    if (++st == p.stages) {
                        st = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        // whoever gave up, if any: what is in flight lands before the CTA leaves
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0)
            for (int i = it < p.stages ? 0 : it - p.stages; i < it; ++i)
                mbar_drain(smem_u32(&full[i % p.stages]), (uint32_t)(i / p.stages) & 1u);
        __syncthreads();
        return;
    }

    // Two teams take the stages in turn.  The warp's two blocks of a stage (neighbours; one barrier
    // and one set of addresses for both): blocks `block` and the next of tile `sub` of the set.
    const int g = lane >> 2, t = lane & 3;
    const int team = warp / kQTeam, slot = 2 * (warp % kQTeam);
    const int sub = p.tps == 1 ? 0 : slot / p.blocks, block = p.tps == 1 ? slot : slot % p.blocks;
    const bool placed = sub < p.tps && block < p.blocks;
    const uint32_t frag = base + (uint32_t)(block * p.tps * kQBlockBytes + sub * kQBlockBytes + g * 64 +
                                            ((g >> 1 & 3) << 4) + 4 * t);  // piece j: XOR j << 4
    // (rows of an odd number of scales are copied from the 4-byte boundary before an odd one)
    const uint32_t scale_at = scales_at + (uint32_t)((16 * sub + g) * p.scale_pitch + 2 * block * kPerBlock +
                                                     (p.scale_copy == 2 && (g & 1) ? 2 : 0));
    const uint32_t scale_down = (uint32_t)(8 * p.scale_pitch);  // to row g + 8
    const unsigned char* xrow = xs + (g < ntok ? g : 0) * pitch + 16 * t;  // an absent token's columns are not read out
    const float4* srow = sums + (t < pairs ? t : 0);

    // The shares of a set (number `no` of all panels'), added in the order of the warps by four of
    // them.
    auto add_up = [&](int no) {
        const int buf = no % kQParts, panel = no / sets, set = no - panel * sets;
        if (warp / kQAdders != set % (kQWarps / kQAdders)) return;  // (a set's sums are the same threads' in all panels)
        mbar_wait(smem_u32(&written[buf]), (uint32_t)(no / kQParts) & 1u, abort_flag, &g_q4_status, p.wait_ns);
        for (int e = threadIdx.x % (32 * kQAdders); e < p.tps * 16 * kQTokens; e += 32 * kQAdders) {
            const int r = e & 15, b = e / 16 % kQTokens, tile = e / (16 * kQTokens);
            float sum = 0.f;
            if (p.tps == 1) {
#pragma unroll
                for (int w = 0; w < kQWarps; ++w) sum += part[buf][w][r][b];
            } else {
                for (int w = 0; w < p.blocks / 2; ++w)
                    sum += part[buf][tile * p.blocks / 2 + w][r][b] + part[buf][kQTeam + tile * p.blocks / 2 + w][r][b];
            }
            if (panels > 1) {  // (then a set is one tile)
                float* kp = kept + set * (16 * kQTokens) + e;
                if (panel > 0) sum += *kp;
                *kp = sum;
            }
            const int64_t row = ((int64_t)blockIdx.x + (int64_t)set * gridDim.x) * set_rows + 16 * tile + r;
            if (panel == panels - 1 && row < p.m && b < ntok) p.y[(tok0 + b) * p.m + row] = 65536.f * sum;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&added[buf]));
    };

    int st = team, no = 0, first = team;  // the team's next stage, and which of the next set's that is
    uint32_t phase = 0;
    for (int panel = 0; panel < panels; ++panel) {
        const int64_t pcol = (int64_t)panel * p.panel;
        const int width = (int)(p.n - pcol < p.panel ? p.n - pcol : p.panel), nblocks = width / kQCols, per_set = stages_in(panel);
        if (panel > 0) asm volatile("barrier.sync 1, %0;" ::"n"(32 * kQWarps) : "memory");  // the place of x is free again
        // x, 8 columns a lane; a tree over a group's lanes gives its largest value and its sum.  A
        // group's values are multiplied by 2^shift; what undoes it (and 2^-133) is kept as
        // 2^(117 - shift), 2^-16 of it, and so is 2^-16 of the sum: a group's sums of the largest
        // bfloat16 numbers, 15 times them and more, stay finite (and 2^-16 of the smallest is exact).
        const int units = width / 8;  // a multiple of 16, a group of its divisors
        constexpr int kBatch = 8;
        int next_tok = 0, next_unit = warp * 32 + lane;
        auto settle = [&]() {
            for (; next_unit >= units && next_tok < ntok; ++next_tok) next_unit -= units;
        };
        settle();
        while (__any_sync(0xffffffffu, next_tok < ntok)) {
            uint4 v[kBatch];
            int tok[kBatch], unit[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                tok[i] = next_tok;
                unit[i] = next_unit;
                v[i] = make_uint4(0, 0, 0, 0);
                if (next_tok < ntok)
                    v[i] = *reinterpret_cast<const uint4*>(p.x + (tok0 + next_tok) * p.n + pcol + 8 * next_unit);
                next_unit += 32 * kQWarps;
                settle();
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t top2 = max_bf16x2(max_bf16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                                 max_bf16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
                uint32_t top = max(top2 >> 16, top2 & 0xFFFFu);
                float s = (sum_bf16(v[i].x) + sum_bf16(v[i].y)) + (sum_bf16(v[i].z) + sum_bf16(v[i].w));
#pragma unroll
                for (int o = 1; o < kGroup / 8; o <<= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                }
                const int exponent = (int)(top >> 7), shift = exponent < 126 ? 127 : 253 - exponent;
                const uint32_t f0 = (uint32_t)(127 + shift) * 0x00800080u, f1 = (uint32_t)(123 + shift) * 0x00800080u;
                if (tok[i] < ntok) {
                    *reinterpret_cast<uint4*>(xs + tok[i] * pitch + 16 * unit[i]) =
                        make_uint4(mul_bf16x2(__byte_perm(v[i].x, v[i].z, 0x5410), f0),
                                   mul_bf16x2(__byte_perm(v[i].x, v[i].z, 0x7632), f1),
                                   mul_bf16x2(__byte_perm(v[i].y, v[i].w, 0x5410), f0),
                                   mul_bf16x2(__byte_perm(v[i].y, v[i].w, 0x7632), f1));
                    if (unit[i] % (kGroup / 8) == 0)
                        reinterpret_cast<float2*>(sums + unit[i] / (kGroup / 8) * pairs)[tok[i]] =
                            make_float2(__uint_as_float((uint32_t)(244 - shift) << 23), s * (kZeros ? 1.f : 8.f));
                }
            }
        }
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * kQWarps) : "memory");

        for (int set = 0; set < sets; ++set) {
            float out[4] = {0.f, 0.f, 0.f, 0.f};
            int k = first;
            for (; k < per_set; k += 2) {
                // (a wait that gives up is recorded and ends the others: the CTA runs out in bounded time)
                mbar_wait(smem_u32(&full[st]), phase, abort_flag, &g_q4_status, p.wait_ns);
                const int at_block = k * p.blocks + block;
                const uint32_t at0 = frag + (uint32_t)(st * kQCodeBytes), h_at0 = scale_at + (uint32_t)st * scale_stage;
                const unsigned char* xat0 = xrow + 2 * kQCols * at_block;
                const float4* sat0 = srow + kPerBlock * pairs * at_block;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!placed || at_block + i >= nblocks) break;
                    const uint32_t at = at0 + (uint32_t)(i * p.tps * kQBlockBytes), h_at = h_at0 + 2 * kPerBlock * i;
                    const uint2 ha = lds_halves<kPerBlock>(h_at), hb = lds_halves<kPerBlock>(h_at + scale_down);
                    uint2 za = ha, zb = hb;
                    if constexpr (kZeros) {
                        za = lds_halves<kPerBlock>(h_at + scale_bytes);
                        zb = lds_halves<kPerBlock>(h_at + scale_bytes + scale_down);
                    }
                    const unsigned char* xat = xat0 + 2 * kQCols * i;
                    const float4* sat = sat0 + kPerBlock * pairs * i;
                    float acc[4];
#pragma unroll
                    for (int j = 0; j < kQCols / 32; ++j) {
                        const uint32_t wa = lds32(at ^ (j << 4)), wb = lds32((at ^ (j << 4)) + 512);
                        const uint4 b = *reinterpret_cast<const uint4*>(xat + 64 * j);
                        constexpr uint32_t low = 0x000F000Fu, high = 0x00F000F0u;
                        if (j % kPieces == 0)
                            mma_first(acc, wa & low, wb & low, wa & high, wb & high, b.x, b.y);
                        else
                            mma_add(acc, wa & low, wb & low, wa & high, wb & high, b.x, b.y);
                        const uint32_t va = wa >> 8, vb = wb >> 8;
                        mma_add(acc, va & low, vb & low, va & high, vb & high, b.z, b.w);
                        if ((j + 1) % kPieces == 0) {  // the group is complete
                            const int q = j / kPieces;
                            const float4 f = sat[q * pairs];
                            const float s0 = one_half(ha, q), s1 = one_half(hb, q);
                            if constexpr (kZeros) {
                                const float z0 = one_half(za, q), z1 = one_half(zb, q);
                                acc[0] = fmaf(acc[0], f.x, -z0 * f.y);
                                acc[1] = fmaf(acc[1], f.z, -z0 * f.w);
                                acc[2] = fmaf(acc[2], f.x, -z1 * f.y);
                                acc[3] = fmaf(acc[3], f.z, -z1 * f.w);
                            } else {  // the sums come 8 times as large
                                acc[0] = fmaf(acc[0], f.x, -f.y);
                                acc[1] = fmaf(acc[1], f.z, -f.w);
                                acc[2] = fmaf(acc[2], f.x, -f.y);
                                acc[3] = fmaf(acc[3], f.z, -f.w);
                            }
                            out[0] = fmaf(s0, acc[0], out[0]);
                            out[1] = fmaf(s0, acc[1], out[1]);
                            out[2] = fmaf(s1, acc[2], out[2]);
                            out[3] = fmaf(s1, acc[3], out[3]);
                        }
                    }
                }
                __syncwarp();  // the blocks were read by all lanes
                if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
                st += 2;
                if (st >= p.stages) {
                    st -= p.stages;
                    phase ^= 1u;
                }
            }
            first = k - per_set;
            // the warps' shares of the set's tiles
            if (no >= kQParts) mbar_wait(smem_u32(&added[no % kQParts]), (uint32_t)(no / kQParts - 1) & 1u, abort_flag, &g_q4_status, p.wait_ns);
            float(&mine)[16][kQTokens] = part[no % kQParts][warp];
            *reinterpret_cast<float2*>(&mine[g][2 * t]) = make_float2(out[0], out[1]);
            *reinterpret_cast<float2*>(&mine[g + 8][2 * t]) = make_float2(out[2], out[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&written[no % kQParts]));
            if (no > 0) add_up(no - 1);
            ++no;
        }
    }
    add_up(no - 1);
    __syncthreads();  // with the fetching warps
    pdl_trigger();
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

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The codes as (16 words, row, 64-byte block of the row); boxes of 16 words x rows x blocks,
// 64-byte swizzle, zeros outside.
bool q4_map(CUtensorMap* map, const uint32_t* W, int64_t m, int64_t n, int rows, int blocks) {
    static EncodeFn fn = nullptr;
    if (!fn) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        fn = reinterpret_cast<EncodeFn>(f);
    }
    const cuuint64_t dims[3] = {16, (cuuint64_t)m, (cuuint64_t)(n / kQCols)};
    const cuuint64_t strides[2] = {(cuuint64_t)(n / 2), 64};
    const cuuint32_t box[3] = {16, (cuuint32_t)rows, (cuuint32_t)blocks}, estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint32_t*>(W), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kGroup, bool kZeros>
int q4_launch(Q4Args p, const uint32_t* W, cudaStream_t stream) {
    // more shared memory than a kernel gets by default: once per device
    static unsigned long long init_mask = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&init_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(q4_kernel<kGroup, kZeros>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSpace) !=
            cudaSuccess)
            return NQ_ERR_CUDA;
        __atomic_fetch_or(&init_mask, bit, __ATOMIC_RELEASE);
    }
    const int64_t tokens = p.batch < kQTokens ? p.batch : kQTokens;
    auto bytes = [&](int64_t panel, bool panels) {
        return 1024 + tokens * (2 * panel + 64) + panel / kGroup * ((tokens + 1) / 2) * 16 +
               (panels ? kQPanelSets * 16 * kQTokens * 4 : 0);
    };
    const int64_t row_blocks = p.n / kQCols;
    p.blocks = (int)(row_blocks < kQWarps ? (row_blocks + 1) / 2 * 2 : kQWarps);
    const int64_t tiles = (p.m + 15) / 16;
    const int64_t token_groups = (p.batch + kQTokens - 1) / kQTokens;
    const int64_t at_once = sm_count() / token_groups > 0 ? sm_count() / token_groups : 1;
    // a stage holds several tiles of a narrow matrix, but not so many that fewer CTAs have work
    int64_t tps = kQWarps / p.blocks;
    while (tps > 1 && (tiles + tps - 1) / tps < at_once) --tps;
    p.tps = (int)tps;
    const int64_t scale_row = 2 * (p.n / kGroup), stage_row = 2 * p.blocks * (kQCols / kGroup);
    p.scale_copy = scale_row % 16 == 0 ? 16 : scale_row % 8 == 0 ? 8 : scale_row % 4 == 0 ? 4 : 2;
    p.scale_pitch = (int)(p.scale_copy > 2 ? stage_row : (stage_row + 2 + 3) / 4 * 4);
    const int64_t stage = kQCodeBytes + (kZeros ? 2 : 1) * 16 * tps * p.scale_pitch;
    // all columns of x, or panels of them
    const int64_t room = kQSpace - kQMinStages * stage;
    const bool panels = bytes(p.n, false) > room;
    int64_t panel = p.n;
    if (panels)
        for (panel = p.n / kQStageCols * kQStageCols; panel > kQStageCols && bytes(panel, true) > room;) panel -= kQStageCols;
    p.panel = (int)panel;
    const int64_t fixed = bytes(panel, panels), fit = (kQSpace - fixed) / stage;
    p.stages = (int)(fit < kQMaxStages ? fit / 2 * 2 : kQMaxStages);
    const int64_t sets = (tiles + tps - 1) / tps;
    // the sets evenly over the CTAs that fit at a time
    int64_t per_cta = (sets + at_once - 1) / at_once;
    if (panels && per_cta > kQPanelSets) per_cta = kQPanelSets;
    const int64_t ctas = (sets + per_cta - 1) / per_cta;
    CUtensorMap wmap;
    if (!q4_map(&wmap, W, p.m, p.n, 16 * p.tps, p.blocks)) return NQ_ERR_CUDA;
    return launch_pdl(q4_kernel<kGroup, kZeros>, dim3((unsigned)ctas, (unsigned)token_groups), dim3(kQThreads),
                      (size_t)(p.stages * stage + fixed), stream, wmap, p) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

template <int kGroup>
int q4_zeros(const Q4Args& p, const uint32_t* W, cudaStream_t stream) {
    return p.zeros ? q4_launch<kGroup, true>(p, W, stream) : q4_launch<kGroup, false>(p, W, stream);
}

}  // namespace

int q4_forward(const uint16_t* x, const uint32_t* W, const uint16_t* scales, const uint16_t* zeros, int64_t m,
               int64_t n, int group, int64_t batch, float* y, cudaStream_t stream) {
    const Q4Args p{x, scales, zeros, y, m, n, batch, 0, 0, 0, 0, 0, 0, head_wait_ns()};
    return group == 32   ? q4_zeros<32>(p, W, stream)
           : group == 64 ? q4_zeros<64>(p, W, stream)
                         : q4_zeros<128>(p, W, stream);
}

int q4_pack_device(const uint8_t* codes, int64_t rows, int64_t cols, uint32_t* out, unsigned* flag,
                   cudaStream_t stream) {
    const int64_t wpr = (cols + 7) / 8, words = rows * wpr;
    const int64_t blocks = (words + 255) / 256, cap = 16 * (int64_t)sm_count();
    q4_pack_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, stream>>>(codes, words, wpr, cols, out, flag);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

// The recorded status of the current device, cleared (after the caller's synchronisation).
int q4_take_status(unsigned* word) {
    if (cudaMemcpyFromSymbol(word, g_q4_status, sizeof(unsigned)) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned zero = 0;
    if (*word != 0 && cudaMemcpyToSymbol(g_q4_status, &zero, sizeof(unsigned)) != cudaSuccess) return NQ_ERR_CUDA;
    return NQ_OK;
}

}  // namespace nq
