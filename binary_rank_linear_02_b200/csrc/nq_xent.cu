// nq_xent.cu -- cross entropy of a dense output head without its logits in memory, and its
// gradients.  For tokens h (N x d, bfloat16), head W (V x d, bfloat16) and labels:
//     z = h W^T,  lse_i = log sum_v exp(z_iv),  loss_i = lse_i - z_i,label(i),
//     dz_iv = dloss_i (exp(z_iv - lse_i) - [v = label(i)]),  dh = dz W,  dW = dz^T h.
//
// The logits exist only as accumulators in tensor memory.  Forward: each 256 x 256 tile of z
// is reduced in its epilogue to a maximum and a sum of exponentials per row (fp32), and a
// second kernel joins a row's tiles in order.  Backward: the vocabulary is taken in pieces;
// a piece's z is computed again, its epilogue writes dz as bfloat16 into a scratch of bounded
// size, and two products read it: the piece's rows of dW (complete, since they sum over the
// tokens) and its share of dh (summed over the pieces in fp32, in order).  dz in bfloat16 is
// what lets both products run on the bf16 tensor cores (an operand pair has one type).  Its rounding,
// at most 2^-8 of each term, would be as large as that of the bfloat16 results, and nearly all of it
// at the labels, whose terms are the large ones: what bfloat16 leaves there is kept in fp32, a number
// a token, and added to dh and dW in the products' epilogues (their error in the norm is then the
// results' own rounding, 1.66e-3, where it was 2.4e-3; 1000 tokens x 50257 x 2048 backward: 524 to 544 us,
// 4096 x 32000 x 4096: 2% more).  With few tokens, where the others' roundings do not average out, dz is
// two bfloat16 parts; for dW also with many tokens per class, see many_per_class().
//
// All four products are the same tcgen05 kernel (kind::f16, bf16 operands, fp32 accumulators)
// with other operand orders and epilogues: dW reads dz and h token-major (MN-major tiles), dh
// reads W's rows as MN-major tiles, so nothing is transposed in memory.  Sizes need not be
// multiples of the tile: TMA fills with zeros outside, epilogues mask.
//
// What bounds it: the tensor cores, from some 256 tokens on.  4096 tokens x 32000 classes x 4096:
// forward 780 to 811 us (1376 to 1324 TFLOP/s; cuBLAS, kept busy for seconds, reaches 1407 under the power
// cap), backward, with z computed again, 2430 to 2550 us (1325 to 1263).  Hence pairs of CTAs (half of B's traffic in
// shared memory) and two accumulators (one CTA with a 128 x 256 tile took 1029 and 3756 us).  The
// epilogue has to be done within a tile's MMAs, some 13 us at d = 4096: eight warps a CTA, label
// and ignored tokens outside the loop over the columns, results written by way of shared memory
// as rows of 128 bytes (from the lanes, each its own row, they came in pieces of 16 bytes: four
// such warps took 556 us where these took 525, 1000 tokens x 50257 x 2048 backward).
// With few tokens HBM bounds it, W's bytes: see kXFewTokens.
//
// The tensor cores round an accumulator toward zero at each step of 16 products, so a sum of
// d = 4096 is low by some 1e-6 of its size.  The forward's epilogue therefore takes the logits in
// parts of about 32 K blocks (2048 products) and adds these in fp32.
#include <cuda.h>
#include <cuda_bf16.h>

#include "nq_internal.cuh"
#include "nq_sm100.cuh"

namespace nq {
namespace {

// A cluster of two CTAs computes a tile of 256 rows and up to 256 columns: each holds 128 rows
// of A, half of B's columns and the accumulators of its 128 rows.
constexpr int kXHalfTile = 128, kXTile = 256, kXK = 64;
constexpr int kXABytes = kXHalfTile * kXK * 2;      // 16 KB of A per CTA and stage; B: 64 bytes per column of the tile
constexpr int kXBox = 64 * kXK * 2;                 // one TMA box of an MN-major tile: 64 rows x 64 elements
constexpr int kXMaxStages = 13;
constexpr int kXEpilogueWarps = 8;                  // two for each 32 rows of a CTA
constexpr int kXThreads = 128 + 32 * kXEpilogueWarps;
constexpr int kXStagingBytes = 4096;                // of an epilogue warp: 32 rows x 128 bytes
constexpr int kXStaging = kXEpilogueWarps * kXStagingBytes;
constexpr int kXSpace = 224 * 1024;                 // stages, and behind them the staging where it is used
constexpr int kXSmem = kXSpace + 1024 + 1024;
// The forward's epilogue keeps 128 sums a thread: its two warpgroups take over registers of the
// first one, which hardly needs any (launched with 384 x 168 = 128 x 56 + 256 x 224).
constexpr int kXLaunchRegs = 168, kXFewRegs = 56, kXManyRegs = 224;
static_assert(128 * kXFewRegs + 32 * kXEpilogueWarps * kXManyRegs <= kXThreads * kXLaunchRegs, "more than launched with");
constexpr int kXPart = 32;                          // K blocks of a logit's sum in tensor memory, about
constexpr uint32_t kXTmemCols = 512;                // two accumulators of 256 columns
constexpr int64_t kXPieceBytes = int64_t(256) << 20;  // scratch for dz
constexpr int64_t kXSumBytes = int64_t(256) << 20;    // scratch for dh's partial sums

// A device-side wait that gave up (NQ_ERR_TIMEOUT) is recorded here; nq_device_status reads it.
__device__ unsigned g_xent_status;

__device__ __forceinline__ uint32_t xent_idesc(bool amn, bool bmn, int columns) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((amn ? 1u : 0u) << 15) | ((bmn ? 1u : 0u) << 16) |
           ((uint32_t)(columns >> 3) << 17) | ((uint32_t)(kXTile >> 4) << 24);
}

// SW128 MN-major operand descriptor: rows of 64 elements along K, 8-row groups 1024 B apart,
// the next 64 elements of M (or N) one box further.
__device__ __forceinline__ uint64_t xent_desc_mn(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(kXBox >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

struct XentBarriers {
    unsigned long long full[kXMaxStages], empty[kXMaxStages];
    unsigned long long acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    int issued[2], taken;  // K blocks that the pair's CTAs have loads of, and that the MMAs were given (in both CTAs)
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of this CTA's shared-memory location in the cluster's CTA `rank`, and in its first one.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) { return in_cta(addr, 0); }
__device__ __forceinline__ void store_in_both(int* p, int v) {
    for (uint32_t rank = 0; rank < 2; ++rank)
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(in_cta(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// A load into this CTA's shared memory that reports its bytes to a barrier of the pair.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Arrives on this barrier in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ float xent_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// (kMadeUp: as bf16 too, dW with what bf16 left of dz at the labels added; apart, since dW of few tokens is
// all epilogue and loses 4% to the registers for it)
enum { kStats = 0, kDz = 1, kToBf16 = 2, kPartial = 3, kMadeUp = 4 };

// "Token" and "class" in a transposed product (kT) change places: rows are classes (or
// elements of d), columns are tokens.
struct XentEpilogue {
    int64_t rows, cols;     // of the product (unpadded)
    const int32_t* labels;  // per token
    int64_t label0;         // first class of the product
    union {
        int64_t vocab;      // all classes (kPartial: those up to the product's end)
        int64_t tokens;     // kMadeUp: how many labels there are
    };
    // rest, not kStats: what bf16 leaves of dz at each token's label, fp32 (null: it is not kept apart).
    // kDz writes it; kPartial (dh) adds it times the label's row of W, kMadeUp (dW) times the token's row
    // of h, to the class's row.
    union {
        float2* stats;      // kStats: [token][slot]: maximum, sum of exp(z - maximum)
        float* rest;
    };
    union {
        int slots;
        int rest_pitch;     // floats from one token's rest to the next
    };
    union {
        float* picked;      // kStats: z of the label, per token
        const uint16_t* other;  // the rows that rest is multiplied by, as long as the product's
    };
    const float* lse;       // kDz, per token
    const float* dloss;     // kDz, per token
    uint16_t* out;          // kDz, kToBf16, kMadeUp: bf16, [row][column] with pitch ldo (kT: [column][row])
    int64_t ldo;
    int low;                // kDz: what bf16 leaves of dz goes this many rows (kT: columns) on (0: nowhere)
    float* part;            // kPartial: [split][row][column] fp32 (kT: [split][column][row]), added to unless first
    int first;
};

__device__ __forceinline__ uint32_t xent_pack(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// What a lane needs to know of a token: its label (-1: it does not count), the softmax's norm
// (times log2 e) and the loss's weight.
struct XentToken {
    int label;
    float lse2, dl;
};
template <int kEpi>
__device__ __forceinline__ XentToken xent_token(const XentEpilogue& e, int64_t token, bool there) {
    XentToken t{-1, INFINITY, 0.f};  // (exp(z - infinity) = 0: dz = 0)
    if constexpr (kEpi == kStats || kEpi == kDz) {
        if (there) {
            t.label = e.labels[token];
            if (t.label < 0 || t.label >= e.vocab) t.label = -1;
            if constexpr (kEpi == kDz) {
                if (t.label >= 0) {
                    t.dl = e.dloss[token];
                    t.lse2 = t.dl != 0.f ? e.lse[token] * kLog2e : INFINITY;
                }
            }
        }
    }
    if constexpr (kEpi == kPartial) {  // the label's row in `other` and what its dz is to be made up by
        if (there && e.rest) {
            const int64_t label = e.labels[token];
            if (label >= e.label0 && label < e.vocab) {
                t.label = (int)(label - e.label0);
                t.dl = e.rest[token * e.rest_pitch];
            }
        }
    }
    return t;
}

// Two floats at a time.
__device__ __forceinline__ float2 xent_fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}

// 32 rows (lane = row) x 128 bytes, 16 bytes at a time from the lanes into the warp's staging and
// out of it row by row, so that 8 lanes write 128 consecutive bytes: put(piece, value), then
// write(fn), fn(row of the 32, piece, value).  The pieces are XOR-swizzled over the banks.
__device__ __forceinline__ void staging_put(uint32_t buffer, int lane, int piece, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                 ::"r"(buffer + (uint32_t)(lane * 128 + ((piece ^ (lane & 7)) << 4))), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
template <int kPieces = 8, typename Fn>
__device__ __forceinline__ void staging_write(uint32_t buffer, int lane, Fn&& fn) {
    __syncwarp();
    const int piece = lane % kPieces;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int r = 32 / kPieces * i + lane / kPieces;
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(buffer + (uint32_t)(r * 128 + ((piece ^ (r & 7)) << 4))));
        fn(r, piece, v);
    }
    __syncwarp();
}

// Lane j's result: op over the lanes' v[j] (the lanes trade halves of what they hold: 31 shuffles).
template <typename Op>
__device__ __forceinline__ float across_lanes(const float (&values)[32], int lane, Op op) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = values[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + o], o);
            v[i] = op(upper ? v[i + o] : v[i], other);
        }
    }
    return v[0];
}

// The first 32 columns' worth of accumulators from `taddr` on.
__device__ __forceinline__ void xent_load32(uint32_t taddr, float (&v)[32]) {
    uint32_t w[32];
    tmem_ld32(taddr, w);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
}

// A row's 128 logits from col0 on: their maximum and sum of exponentials, and the label's logit.
__device__ __forceinline__ void xent_stats(const XentEpilogue& e, float (&z)[128], int64_t row, int64_t col0, int slot,
                                           const XentToken& tok) {
    const int64_t left = e.cols - col0, a = (int64_t)tok.label - col0;
    if (left < 128) {
#pragma unroll
        for (int j = 0; j < 128; ++j)
            if (j >= left) z[j] = -INFINITY;
    }
    if (tok.label >= 0 && a >= 0 && a < 128 && a < left) {
        float picked = z[0];
#pragma unroll
        for (int j = 1; j < 128; ++j) picked = j == (int)a ? z[j] : picked;
        e.picked[row] = picked;
    }
    float top[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = z[j];
#pragma unroll
    for (int j = 8; j < 128; ++j) top[j & 7] = fmaxf(top[j & 7], z[j]);
    const float m = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
    const float f = m == -INFINITY ? 0.f : m;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 128; ++j) sum[j & 7] += xent_ex2((z[j] - f) * kLog2e);
    const float s = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
    if (row < e.rows) e.stats[row * e.slots + slot] = make_float2(m, s);
}

// dz of a row's 32 columns; at: the label's column among them, if it is.
__device__ __forceinline__ void xent_dz32(float (&v)[32], int at, const XentToken& tok) {
    const float2 scale = make_float2(kLog2e, kLog2e), shift = make_float2(-tok.lse2, -tok.lse2);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 x = xent_fma2(make_float2(v[j], v[j + 1]), scale, shift);
        v[j] = xent_ex2(x.x);
        v[j + 1] = xent_ex2(x.y);
    }
    if ((unsigned)at < 32u) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j == at) v[j] -= 1.f;
    }
    if (tok.dl == 0.f) {  // whatever its logits are
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= tok.dl;
}

// What bf16 leaves of a number (nothing of an infinity).
__device__ __forceinline__ float xent_rest(float x) {
    const float rest = x - __bfloat162float(__float2bfloat16_rn(x));
    return fabsf(rest) < INFINITY ? rest : 0.f;
}
__device__ __forceinline__ float xent_float(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }

// What a warp needs to find the tokens whose labels are among its 32 classes (lane = class).
struct XentLabels {
    const int32_t* labels;
    const float* rest;
    const uint16_t* h;  // tokens' rows
    int64_t cols;
    int tokens, rest_pitch, first, limit;  // limit: how many of the 32 there are
};
__device__ __forceinline__ XentLabels xent_labels(const XentEpilogue& e, int64_t row0) {
    const int64_t rows = e.rows - row0;
    return XentLabels{e.labels, e.rest, e.other, e.cols, (int)e.tokens, e.rest_pitch, (int)(e.label0 + row0),
                      rows < 32 ? (int)(rows > 0 ? rows : 0) : 32};
}
// Goes through the labels from token `from` on, in order: fn(token, class), the same in all lanes, for those
// found; before a group of 32 tokens in which `room` has none left it stops, and returns where.
// `label` holds those of the 256 tokens from `from` on.
__device__ __forceinline__ void xent_load_labels(const int32_t* labels, int tokens, int from, int lane, int (&label)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int i = from + 32 * u + lane;
        label[u] = i < tokens ? labels[i] : -1;
    }
}
template <typename Room, typename Fn>
__device__ __forceinline__ int xent_search(const XentLabels& e, int (&label)[8], int from, int lane, Room&& room, Fn&& fn) {
    while (from < e.tokens) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int at = label[u] - e.first;
            unsigned hits = __ballot_sync(0xffffffffu, label[u] >= 0 && at >= 0 && at < e.limit);
            if (hits) {
                if (!room(__popc(hits))) return from + 32 * u;
                for (; hits; hits &= hits - 1) {
                    const int l = __ffs(hits) - 1;
                    fn(from + 32 * u + l, __shfl_sync(0xffffffffu, at, l));
                }
            }
        }
        from += 256;
        if (from < e.tokens) xent_load_labels(e.labels, e.tokens, from, lane, label);
    }
    return e.tokens;
}
// The tokens of a lane's class, if no class of the warp has more than kXOwn.
constexpr int kXOwn = 4;
struct XentMatches {
    int most;          // that a class has
    int token[kXOwn];  // of this lane's (-1: none)
    float rest[kXOwn];
};
__device__ __forceinline__ XentMatches xent_matches(const XentLabels& e, const int (&first)[8], int64_t col0, int lane) {
    XentMatches m;
#pragma unroll
    for (int k = 0; k < kXOwn; ++k) {
        m.token[k] = -1;
        m.rest[k] = 0.f;
    }
    int mine = 0, label[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) label[u] = first[u];
    xent_search(e, label, 0, lane, [](int) { return true; }, [&](int token, int row) {
        if (lane == row) {
#pragma unroll
            for (int k = 0; k < kXOwn; ++k)
                if (mine == k) m.token[k] = token;
            ++mine;
        }
    });
    m.most = __reduce_max_sync(0xffffffffu, mine);
#pragma unroll
    for (int k = 0; k < kXOwn; ++k) {
        if (m.token[k] < 0) break;
        m.rest[k] = e.rest[(int64_t)m.token[k] * e.rest_pitch];
        // the lines of h that the epilogue is to read, on their way while the sums are
        const uint16_t* h = e.h + (int64_t)m.token[k] * e.cols;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int64_t at = col0 + (i < 2 ? 64 * i : 127);
            asm volatile("{\n.reg .b16 t;\nld.global.ca.b16 t, [%0];\n}" ::"l"(h + (at < e.cols ? at : e.cols - 1)) : "memory");
        }
    }
    return m;
}

// Adds up, for a warp's 32 x 32 part of dW, what its classes' tokens are to be made up by, in the order of the
// tokens: in shared memory, a column to a lane (element (r, c) in place c ^ r of row r).  For classes that
// are many tokens' labels; 32 tokens at a time.
__device__ __noinline__ void xent_make_up(const XentLabels& e, int64_t col, uint32_t buffer, int lane) {
    for (int r = 0; r < 32; ++r) asm volatile("st.shared.f32 [%0], %1;" ::"r"(buffer + (uint32_t)(128 * r + 4 * lane)), "f"(0.f) : "memory");
    const bool there = col + lane < e.cols;
    const uint16_t* h = e.h + col + lane;
    for (int from = 0; from < e.tokens;) {
        int count = 0, token = 0, row = 0;  // (one to a lane)
        int label[8];
        xent_load_labels(e.labels, e.tokens, from, lane, label);
        from = xent_search(e, label, from, lane, [&](int more) { return count + more <= 32; }, [&](int t, int r) {
            if (lane == count) {
                token = t;
                row = r;
            }
            ++count;
        });
        const float rest = lane < count ? e.rest[(int64_t)token * e.rest_pitch] : 0.f;
        float x[32];
#pragma unroll
        for (int u = 0; u < 32; ++u) {
            const int t = __shfl_sync(0xffffffffu, token, u);
            x[u] = there && u < count ? xent_float(h[(int64_t)t * e.cols]) : 0.f;
        }
        // (a class that comes again at once is added up in a register: one that most tokens have costs their loads)
        int at_row = -1;
        uint32_t at = 0;
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 32; ++u) {
            const int r = __shfl_sync(0xffffffffu, row, u);
            const float part = __shfl_sync(0xffffffffu, rest, u);
            if (u >= count) break;
            if (r != at_row) {
                if (at_row >= 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(sum) : "memory");
                at_row = r;
                at = buffer + (uint32_t)(128 * r + 4 * (lane ^ r));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sum) : "r"(at) : "memory");
            }
            sum = fmaf(part, x[u], sum);
        }
        if (at_row >= 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(sum) : "memory");
    }
    __syncwarp();
}

// v += a times 32 bf16 numbers (left of them; a multiple of 8).
__device__ __forceinline__ void xent_add32(float (&v)[32], float a, const uint16_t* row, int left) {
    uint4 x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x[q] = 8 * q < left ? *reinterpret_cast<const uint4*>(row + 8 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t two[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * q + 2 * i] = fmaf(a, __uint_as_float(two[i] << 16), v[8 * q + 2 * i]);
            v[8 * q + 2 * i + 1] = fmaf(a, __uint_as_float(two[i] & 0xFFFF0000u), v[8 * q + 2 * i + 1]);
        }
    }
}

// The transposed product's 32 columns (tokens, from `col` on, n of them) of the warp's 32 rows
// (classes, or elements of d; lane = row); tok: of token col + lane.
template <int kEpi>
__device__ __forceinline__ void xent_columns_t(const XentEpilogue& e, float (&v)[32], int64_t row, int64_t col, int n,
                                               int64_t split, int slot, const XentToken& tok) {
    const bool there = row < e.rows;
    const int lane = threadIdx.x & 31;
    const int cls = (int)(e.label0 + row);
    if constexpr (kEpi == kStats) {
        // the warp's 32 classes: per token a maximum and a sum
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= n || !there) v[j] = -INFINITY;
            if (__shfl_sync(0xffffffffu, tok.label, j) == cls && there && j < n) e.picked[col + j] = v[j];
        }
        const float top = across_lanes(v, lane, [](float a, float b) { return fmaxf(a, b); });
        const float f = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = xent_ex2((v[j] - __shfl_sync(0xffffffffu, f, j)) * kLog2e);
        const float sum = across_lanes(v, lane, [](float a, float b) { return a + b; });
        if (lane < n) e.stats[(col + lane) * e.slots + slot] = make_float2(top, sum);
    } else {
        if constexpr (kEpi == kPartial) {
            if (e.rest) {  // what bf16 left of dz at the tokens' labels
                uint16_t w[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int label = __shfl_sync(0xffffffffu, tok.label, j);
                    w[j] = label >= 0 && there ? e.other[(int64_t)label * e.rows + row] : 0;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = fmaf(__shfl_sync(0xffffffffu, tok.dl, j), xent_float(w[j]), v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float x = v[j];
            if constexpr (kEpi == kDz) {
                const float p = xent_ex2(fmaf(x, kLog2e, -__shfl_sync(0xffffffffu, tok.lse2, j)));
                const float dl = __shfl_sync(0xffffffffu, tok.dl, j);
                const bool labelled = __shfl_sync(0xffffffffu, tok.label, j) == cls;
                x = (p - (labelled ? 1.f : 0.f)) * dl;
                x = dl == 0.f || j >= n ? 0.f : x;
                if (e.rest && labelled && there && j < n) e.rest[(col + j) * (int64_t)e.rest_pitch] = xent_rest(x);
                if (e.low && there && col + j < e.low) {  // (columns after the last: zeros)
                    const __nv_bfloat16 high = __float2bfloat16_rn(x);
                    e.out[(col + j) * e.ldo + row] = __bfloat16_as_ushort(high);
                    e.out[(e.low + col + j) * e.ldo + row] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(xent_rest(x)));
                }
            }
            if (j < n && there && (kEpi != kDz || !e.low)) {
                if constexpr (kEpi == kPartial) {
                    float* a = e.part + (split * e.cols + col + j) * e.rows + row;
                    *a = e.first ? x : x + *a;
                } else {
                    e.out[(col + j) * e.ldo + row] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
                }
            }
        }
    }
}

// An epilogue warp's share of a tile: its 32 rows (from row0 on), 128 columns from col0 on.
template <int kEpi>
__device__ __forceinline__ void xent_rows(const XentEpilogue& e, uint32_t taddr, int64_t row0, int64_t col0, int split, int splits,
                                          const XentToken& tok, const XentMatches& matches, uint32_t buffer, int lane) {
    const int left = (int)(e.cols - col0 < 128 ? e.cols - col0 : 128);
    int at = -1 << 20;  // the label's column from col0 on
    if constexpr (kEpi == kDz) {
        const int64_t a = (int64_t)tok.label - e.label0 - col0;
        if (tok.label >= 0 && a >= 0 && a < left) at = (int)a;
    }
    if constexpr (kEpi == kPartial) {
#pragma unroll 1
        for (int c0 = 0; c0 < left; c0 += 32) {
            float v[32];
            xent_load32(taddr + (uint32_t)c0, v);
            if (tok.label >= 0 && ((col0 + c0) >> 5) % splits == split)  // (what bf16 left of dz there: by one share of the sum)
                xent_add32(v, tok.dl, e.other + (int64_t)tok.label * e.cols + col0 + c0, left - c0);
#pragma unroll
            for (int p = 0; p < 8; ++p)
                staging_put(buffer, lane, p, make_uint4(__float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]),
                                                        __float_as_uint(v[4 * p + 2]), __float_as_uint(v[4 * p + 3])));
            staging_write(buffer, lane, [&](int r, int p, uint4 w) {
                if (row0 + r >= e.rows || c0 + 4 * p >= left) return;  // (cols is a multiple of 8)
                float4* a = reinterpret_cast<float4*>(e.part + ((int64_t)split * e.rows + row0 + r) * e.cols + col0 + c0 + 4 * p);
                float4 x = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
                if (!e.first) {
                    const float4 o = *a;
                    x.x += o.x;
                    x.y += o.y;
                    x.z += o.z;
                    x.w += o.w;
                }
                *a = x;
            });
        }
    } else {
        if constexpr (kEpi == kMadeUp) {
            if (matches.most > kXOwn) {  // (the staging serves the sums first, then half as wide rows of results)
#pragma unroll 1
                for (int c0 = 0; c0 < left; c0 += 32) {
                    xent_make_up(xent_labels(e, row0), col0 + c0, buffer, lane);
                    float v[32];
                    xent_load32(taddr + (uint32_t)c0, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float x;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(buffer + (uint32_t)(128 * lane + 4 * (j ^ lane))) : "memory");
                        v[j] += x;
                    }
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        staging_put(buffer, lane, p,
                                    make_uint4(xent_pack(v[8 * p], v[8 * p + 1]), xent_pack(v[8 * p + 2], v[8 * p + 3]),
                                               xent_pack(v[8 * p + 4], v[8 * p + 5]), xent_pack(v[8 * p + 6], v[8 * p + 7])));
                    staging_write<4>(buffer, lane, [&](int r, int p, uint4 w) {
                        if (row0 + r < e.rows && c0 + 8 * p < left)
                            *reinterpret_cast<uint4*>(e.out + (row0 + r) * e.ldo + col0 + c0 + 8 * p) = w;
                    });
                }
                return;
            }
        }
        // (dz in two parts: its second one by going through the tile again)
        const bool two = kEpi == kDz && e.low != 0;
#pragma unroll 1
        for (int c = 0; c < (two ? 256 : 128); c += 64) {
            const int c0 = c & 127;
            if (c0 >= left) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[32];
                xent_load32(taddr + (uint32_t)(c0 + 32 * half), v);
                if constexpr (kEpi == kDz) {
                    const int a = at - c0 - 32 * half;
                    xent_dz32(v, a, tok);
                    if (e.rest && (unsigned)a < 32u) {
                        float x = v[0];
#pragma unroll
                        for (int j = 1; j < 32; ++j) x = j == a ? v[j] : x;
                        e.rest[(row0 + lane) * e.rest_pitch] = xent_rest(x);
                    }
                    if (c >= 128) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = xent_rest(v[j]);
                    }
                }
                if constexpr (kEpi == kMadeUp) {
#pragma unroll
                    for (int k = 0; k < kXOwn; ++k) {
                        if (k >= matches.most) break;
                        if (matches.token[k] >= 0)
                            xent_add32(v, matches.rest[k], e.other + (int64_t)matches.token[k] * e.cols + col0 + c0 + 32 * half,
                                       left - c0 - 32 * half);
                    }
                }
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    staging_put(buffer, lane, 4 * half + p,
                                make_uint4(xent_pack(v[8 * p], v[8 * p + 1]), xent_pack(v[8 * p + 2], v[8 * p + 3]),
                                           xent_pack(v[8 * p + 4], v[8 * p + 5]), xent_pack(v[8 * p + 6], v[8 * p + 7])));
            }
            staging_write(buffer, lane, [&](int r, int p, uint4 w) {
                // (dz: whole tiles, its rows are as long; dW, dh: cols is a multiple of 8)
                if (row0 + r >= e.rows || (kEpi != kDz && c0 + 8 * p >= left)) return;
                *reinterpret_cast<uint4*>(e.out + (row0 + r + (c >= 128 ? e.low : 0)) * e.ldo + col0 + c0 + 8 * p) = w;
            });
        }
    }
}

// How the work is cut: tiles of the product, K blocks per share of the sum, shares.
struct XentPlan {
    int tm, tn, nkb, per_split, splits;
    int bn, stages;  // columns of a tile (256; transposed a multiple of 16); stages of the ring
    int accs;        // accumulators of a transposed tile, which its K blocks go to in turn
    int low;         // kT: the second half of a tile's columns is added to the first; not kT: where the second half
                     // of A's K blocks begins (both 0: no such halves)
    int part;        // K blocks that are summed in tensor memory before the epilogue takes them
    int n_fastest;  // the order of the tiles: neighbours in the first index run at the same time
    unsigned long long wait_ns;  // how long a wait lasts
};

// Waits (the first CTA) for the loads of the pair that no MMA waited for, all of which report to the
// first CTA's barriers: to each at most one use that is not complete.  Where only one of the CTAs
// loads a block, the other's bytes, or the first one's announcement, are made up for.
__device__ __noinline__ void xent_land(XentBarriers& bar, int stages, uint32_t stage_bytes) {
    const int both = bar.issued[0] < bar.issued[1] ? bar.issued[0] : bar.issued[1];
    const int last = bar.issued[0] + bar.issued[1] - both;
    for (int i = bar.taken; i < last; ++i) {
        const uint32_t full = smem_u32(&bar.full[i % stages]);
        if (i >= both && bar.issued[0] == both) mbar_expect_tx(full, stage_bytes);
        if (i >= both && bar.issued[1] == both)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(full), "r"(stage_bytes) : "memory");
        mbar_drain(full, (uint32_t)(i / stages) & 1u);
    }
}

// A persistent pair of CTAs per two SMs walks over the tiles.  Warp 0 loads (each CTA its own
// halves of A and B, reporting to the first CTA's barriers), warp 1 of the first CTA issues the
// MMAs of both, warps 4-11 of each CTA take the accumulators of its 128 rows out of tensor
// memory (two warps for the same 32 rows, each half of the columns) while the next tile's are
// being summed in the other 256 columns.
template <int kEpi, bool AMN, bool BMN, bool kT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXThreads, 1)
xent_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                 const XentPlan plan, const XentEpilogue e) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    XentBarriers& bar = *reinterpret_cast<XentBarriers*>(smem_raw + (base - raw) + kXSpace);
    volatile int* abort_flag = &bar.abort_flag;
    unsigned* status = &g_xent_status;
    constexpr bool kKeeps = kEpi == kStats && !kT;  // (see kXLaunchRegs)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int tiles = plan.tm * plan.tn, items = tiles * plan.splits;
    const int stages = plan.stages, half_bn = plan.bn / 2;
    const uint32_t stage_bytes = kXABytes + (uint32_t)half_bn * 128;

    if (threadIdx.x == 0) {
        for (int st = 0; st < stages; ++st) {
            mbar_init(smem_u32(&bar.full[st]), 1);
            mbar_init(smem_u32(&bar.empty[st]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar.acc_full[i]), 1);
            mbar_init(smem_u32(&bar.acc_empty[i]), 2 * kXEpilogueWarps);  // of both CTAs
        }
        mbar_init(smem_u32(&bar.drain), 1);
        bar.abort_flag = bar.issued[0] = bar.issued[1] = bar.taken = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&bar.tmem_base)), "r"(kXTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    pdl_wait();
    pdl_trigger();

    auto tile_of = [&](int item, int& tm, int& tn, int& kb0, int& kb1) {
        const int split = item / tiles, tile = item % tiles;
        if (plan.n_fastest) {
            tm = tile / plan.tn;
            tn = tile % plan.tn;
        } else {
            tn = tile / plan.tm;
            tm = tile % plan.tm;
        }
        kb0 = split * plan.per_split;
        kb1 = kb0 + plan.per_split < plan.nkb ? kb0 + plan.per_split : plan.nkb;
        return split;
    };

    if (warp < 4) {
        if constexpr (kKeeps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kXFewRegs));
        if (warp == 0 && lane == 0) {
            fence_proxy_async_global();  // dz was written by ordinary stores of the kernel before
            int it = 0, st = 0;  // K blocks so far, and the ring's stage and phase
            uint32_t ph = 0;
            bool ok = true;
            for (int item = pair; item < items && ok; item += pairs) {
                int tm, tn, kb0, kb1;
                tile_of(item, tm, tn, kb0, kb1);
                const int m0 = tm * kXTile + (int)rank * kXHalfTile, n0 = tn * plan.bn + (int)rank * half_bn;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    if (!mbar_wait(smem_u32(&bar.empty[st]), ph ^ 1u, abort_flag, status, plan.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = in_leader(smem_u32(&bar.full[st]));
                    if (rank == 0) mbar_expect_tx(smem_u32(&bar.full[st]), 2u * stage_bytes);
                    const uint32_t dst = base + (uint32_t)st * stage_bytes;
                    int ak = kb * kXK, bk = ak;  // (the second half of A meets B again)
                    if (AMN && BMN && plan.low && 2 * kb >= plan.nkb) {
                        bk = (kb - plan.nkb / 2) * kXK;
                        ak = plan.low + bk;
                    }
                    if constexpr (AMN) {
                        pair_load_2d(dst, &amap, m0, ak, full);
                        pair_load_2d(dst + kXBox, &amap, m0 + 64, ak, full);
                    } else {
                        pair_load_2d(dst, &amap, ak, m0, full);
                    }
                    if constexpr (BMN) {
                        pair_load_2d(dst + kXABytes, &bmap, n0, bk, full);
                        pair_load_2d(dst + kXABytes + kXBox, &bmap, n0 + 64, bk, full);
                    } else {
                        pair_load_2d(dst + kXABytes, &bmap, bk, n0, full);
                    }
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            store_in_both(&bar.issued[rank], it);
        }
        if (warp == 1 && lane == 0 && rank == 0) {
            const uint32_t idesc = xent_idesc(AMN, BMN, plan.bn);
            int n = 0, st = 0, taken = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int item = pair; item < items && ok; item += pairs) {
                int tm, tn, kb0, kb1;
                tile_of(item, tm, tn, kb0, kb1);
                for (int p0 = kb0; p0 < kb1 && ok; p0 += plan.part, ++n) {
                    const int p1 = p0 + plan.part < kb1 ? p0 + plan.part : kb1;
                    const int acc = n & 1;
                    if (!mbar_wait(smem_u32(&bar.acc_empty[acc]), ((uint32_t)(n >> 1) & 1u) ^ 1u, abort_flag, status, plan.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d0 = tmem + (uint32_t)(acc * kXTile);
                    for (int kb = p0, turn = 0; kb < p1; ++kb) {
                        const uint32_t d = kT ? d0 + (uint32_t)(turn * plan.bn) : d0;
                        const int before = kT ? plan.accs : 1;  // K blocks that begin an accumulator
                        if (kT && ++turn == plan.accs) turn = 0;
                        if (!mbar_wait(smem_u32(&bar.full[st]), ph, abort_flag, status, plan.wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t aaddr = base + (uint32_t)st * stage_bytes, baddr = aaddr + kXABytes;
                        const uint64_t ad = AMN ? xent_desc_mn(aaddr) : sw128_desc(aaddr);
                        const uint64_t bd = BMN ? xent_desc_mn(baddr) : sw128_desc(baddr);
                        constexpr uint64_t astep = AMN ? 2048 / 16 : 32 / 16, bstep = BMN ? 2048 / 16 : 32 / 16;
#pragma unroll
                        for (int k = 0; k < kXK / 16; ++k)
                            pair_mma(d, ad + (uint64_t)k * astep, bd + (uint64_t)k * bstep, idesc,
                                     (kb >= p0 + before || k > 0) ? 1u : 0u);
                        pair_commit(smem_u32(&bar.empty[st]));
                        ++taken;
                        if (++st == stages) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                    if (ok) pair_commit(smem_u32(&bar.acc_full[acc]));
                }
            }
            // whoever gave up, if any: the MMAs are done with both CTAs' memory before either leaves
            store_in_both(&bar.taken, taken);
            pair_commit(smem_u32(&bar.drain));
            mbar_drain(smem_u32(&bar.drain), 0);
        }
    } else {
        if constexpr (kKeeps) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kXManyRegs));
        const int quad = warp & 3, half = (warp - 4) / 4;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t buffer = base + (uint32_t)(kXSpace - kXStaging + (warp - 4) * kXStagingBytes);
        int n = 0;
        bool ok = true;
        [[maybe_unused]] int first_labels[8];  // (looked through for every tile)
        if constexpr (kEpi == kMadeUp) xent_load_labels(e.labels, (int)e.tokens, 0, lane, first_labels);
        for (int item = pair; item < items && ok; item += pairs) {
            int tm, tn, kb0, kb1;
            const int split = tile_of(item, tm, tn, kb0, kb1);
            const int64_t row0 = (int64_t)tm * kXTile + (int)rank * kXHalfTile + quad * 32;
            const int64_t col0 = (int64_t)tn * kXTile + 128 * half;  // (not transposed)
            XentToken tok = xent_token<kEpi>(e, row0 + lane, !kT && row0 + lane < e.rows);
            XentMatches matches;
            matches.most = 0;
            if constexpr (kEpi == kMadeUp) matches = xent_matches(xent_labels(e, row0), first_labels, col0, lane);  // (while the sums are under way)
            [[maybe_unused]] float z[128];  // (the sum of a tile's parts, where it may have several)
            if constexpr (kKeeps) {
#pragma unroll
                for (int j = 0; j < 128; ++j) z[j] = 0.f;
            }
#pragma unroll 1
            for (int p0 = kb0; p0 < kb1 && ok; p0 += plan.part, ++n) {
                const int acc = n & 1;
                // (the warp goes on, or gives up, as one)
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar.acc_full[acc]), (uint32_t)(n >> 1) & 1u, abort_flag, status, plan.wait_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t taddr = tmem + lanes + (uint32_t)(acc * kXTile);
                if constexpr (kT) {
                    const int accs = kb1 - kb0 < plan.accs ? kb1 - kb0 : plan.accs;
                    const int columns = plan.low ? plan.low : plan.bn;
#pragma unroll 1
                    for (int c0 = 32 * half; c0 < columns; c0 += 64) {
                        const int64_t col = (int64_t)tn * columns + c0, left = e.cols - col;
                        const int room = columns - c0 < 32 ? columns - c0 : 32, here = left < room ? (int)left : room;
                        if (here <= 0) break;
                        // (dh: what bf16 left of dz is added by one of the sum's shares, of 32 columns at a time)
                        tok = xent_token<kEpi>(e, col + lane, lane < here && (kEpi != kPartial || (c0 >> 5) % plan.splits == split));
                        float v[32];
                        xent_load32(taddr + (uint32_t)c0, v);
                        for (int i = 1; i < accs; ++i) {
                            float w[32];
                            xent_load32(taddr + (uint32_t)(i * plan.bn + c0), w);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] += w[j];
                        }
                        if (plan.low)
                            for (int i = 0; i < accs; ++i) {
                                float w[32];
                                xent_load32(taddr + (uint32_t)(i * plan.bn + plan.low + c0), w);
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[j] += w[j];
                            }
                        xent_columns_t<kEpi>(e, v, row0 + lane, col, here, split, (tm * 2 + (int)rank) * 4 + quad, tok);
                    }
                } else if constexpr (kKeeps) {
#pragma unroll
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        float v[32];
                        xent_load32(taddr + (uint32_t)(128 * half + c0), v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[c0 + j] += v[j];
                    }
                } else {
                    xent_rows<kEpi>(e, taddr + (uint32_t)(128 * half), row0, col0, split, plan.splits, tok, matches, buffer, lane);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(in_leader(smem_u32(&bar.acc_empty[acc])));
            }
            if constexpr (kKeeps) {
                if (ok) xent_stats(e, z, row0 + lane, col0, 2 * tn + half, tok);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal it
    if (bar.issued[0] != bar.taken || bar.issued[1] != bar.taken) {  // somewhere a wait gave up
        if (threadIdx.x == 0 && cluster_rank() == 0) xent_land(bar, plan.stages, kXABytes + 64u * (uint32_t)plan.bn);
        __syncthreads();
        cluster_sync();
    }
    if (threadIdx.x == 32 && rank == 1) mbar_drain(smem_u32(&bar.drain), 0);  // (the last of the MMAs' signals to this CTA)
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kXTmemCols));
    }
}

// dh = the shares' sums, added in order, as bf16 (four at a time: cols is a multiple of 8).
__global__ void __launch_bounds__(256) xent_sum_kernel(const float* __restrict__ part, int splits, int64_t count,
                                                       uint16_t* __restrict__ out) {
    pdl_wait();
    for (int64_t i = 4 * (blockIdx.x * (int64_t)blockDim.x + threadIdx.x); i < count;
         i += 4 * (int64_t)gridDim.x * blockDim.x) {
        float4 a = *reinterpret_cast<const float4*>(part + i);
        for (int q = 1; q < splits; ++q) {
            const float4 b = *reinterpret_cast<const float4*>(part + q * count + i);
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
        }
        *reinterpret_cast<uint2*>(out + i) = make_uint2(xent_pack(a.x, a.y), xent_pack(a.z, a.w));
    }
}

// A CTA per token joins the (maximum, sum) pairs of its slots: thread i takes slots i, i + 128,
// ... in order, then the threads join in a tree (a fixed order).
constexpr int kXJoinThreads = 128;

__device__ __forceinline__ float2 xent_join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), f = m == -INFINITY ? 0.f : m;
    return make_float2(m, a.y * xent_ex2((a.x - f) * kLog2e) + b.y * xent_ex2((b.x - f) * kLog2e));
}

__global__ void __launch_bounds__(kXJoinThreads)
xent_join_kernel(const float2* __restrict__ stats, const float* __restrict__ picked, const int32_t* __restrict__ labels,
                 int64_t tokens, int64_t vocab, int slots, float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ float2 warps[kXJoinThreads / 32];
    pdl_wait();
    const int64_t row = blockIdx.x;
    float2 r = make_float2(-INFINITY, 0.f);
    for (int t = threadIdx.x; t < slots; t += kXJoinThreads) r = xent_join(r, stats[row * slots + t]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        r = xent_join(r, make_float2(__shfl_xor_sync(0xffffffffu, r.x, o), __shfl_xor_sync(0xffffffffu, r.y, o)));
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = r;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kXJoinThreads / 32; ++w) r = xent_join(r, warps[w]);
        const float logs = logf(r.y);
        lse[row] = r.x + logs;
        const int32_t label = labels[row];
        // (m - z) + log s: exact difference first
        loss[row] = label >= 0 && label < vocab ? (r.x - picked[row]) + logs : 0.f;
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

int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t cut(int64_t v, int64_t a) { return (v + a - 1) / a; }

template <int kEpi, bool AMN, bool BMN, bool kT>
int xent_launch(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, int64_t M, int64_t N, int64_t K, int bn,
                int splits, bool n_fastest, const XentEpilogue& e, cudaStream_t stream, int low = 0) {
    static unsigned long long init_mask = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&init_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cudaFuncSetAttribute(xent_gemm_kernel<kEpi, AMN, BMN, kT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmem) !=
            cudaSuccess)
            return NQ_ERR_CUDA;
        if (kEpi == kStats && !kT) {  // what its warpgroups ask for has to be there, or they would wait for it
            cudaFuncAttributes attr;
            if (cudaFuncGetAttributes(&attr, xent_gemm_kernel<kEpi, AMN, BMN, kT>) != cudaSuccess) return NQ_ERR_CUDA;
            if (attr.numRegs < kXLaunchRegs) return NQ_ERR_CUDA;
        }
        __atomic_fetch_or(&init_mask, bit, __ATOMIC_RELEASE);
    }
    CUtensorMap amap, bmap;
    if (!(AMN ? xent_map(&amap, A, AMN && BMN && low ? 2 * low : K, M, lda, kXK) : xent_map(&amap, A, M, K, lda, kXHalfTile)) ||
        !(BMN ? xent_map(&bmap, B, K, N, ldb, kXK) : xent_map(&bmap, B, N, K, ldb, bn / 2)))
        return NQ_ERR_CUDA;
    XentPlan plan;
    plan.tm = (int)cut(M, kXTile);
    plan.tn = (int)cut(N, bn);
    plan.bn = bn;
    plan.stages = (kT ? kXSpace : kXSpace - kXStaging) / (kXABytes + 64 * bn);
    plan.accs = bn <= 64 ? 4 : bn <= 128 ? 2 : 1;
    if (plan.stages > kXMaxStages) plan.stages = kXMaxStages;
    plan.nkb = (int)cut(K, kXK) * (AMN && BMN && low ? 2 : 1);
    plan.low = low;
    plan.per_split = (int)cut(plan.nkb, splits);
    const int parts = (plan.nkb + kXPart / 2) / kXPart;
    plan.part = kEpi == kStats && !kT && parts > 1 ? (int)cut(plan.nkb, parts) : plan.per_split;
    plan.splits = splits;
    plan.n_fastest = n_fastest;
    plan.wait_ns = head_wait_ns();
    const int64_t items = (int64_t)plan.tm * plan.tn * splits, pairs = sm_count() / 2;
    return launch_pdl(xent_gemm_kernel<kEpi, AMN, BMN, kT>, dim3((unsigned)(2 * (items < pairs ? items : pairs))),
                      dim3(kXThreads), (size_t)kXSmem, stream, amap, bmap, plan, e) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

// Up to this many tokens the products with W are transposed: W's rows (or columns) are the
// tile's 256 rows, and all tokens fit its columns, of which only as many as needed are summed.
// (8 tokens x 32000 x 4096: 53 us, W at 4.9 TB/s, where tiles of 256 tokens took 73.)  Where the
// columns leave room, a tile has two or four accumulators: the tensor cores round a sum down
// after each step, and shorter sums lose less (a few 1e-7 of a loss in place of 1e-6).
constexpr int64_t kXFewTokens = 256;
int few_columns(int64_t tokens) { return (int)round_up(tokens, 16); }
// Up to this many, dz is kept as two bf16 parts, the second so many rows after the first (16
// bits of it: with few tokens the rounding of a token's large terms would not average out).  It
// costs next to nothing, since HBM bounds the products that read it: dh has twice the columns
// per tile of W, dW twice the K blocks.
constexpr int64_t kXTwoParts = 128;
int low_rows(int64_t tokens) { return tokens <= kXTwoParts ? few_columns(tokens) : 0; }
// Above, dW's epilogue looks for the tokens of its classes, to add what bfloat16 left of dz there.  With more
// tokens than half the classes it would find too many (4096 tokens x 500 x 4096: 456 us, 4096 x 2000 x 2048:
// 243, where the calls take 68 and 90 with nothing added): there dz is two parts for dW too, whose K blocks
// double (122 and 134 us); with fewer, hardly a warp has a class of more than the four that it keeps in
// registers.  Two parts of 256 classes have to fit dz's scratch; with more tokens than that dW is without.
constexpr int64_t kXTwoPartsMost = kXPieceBytes / (2 * 2 * kXTile);
bool many_per_class(int64_t tokens, int64_t vocab) { return tokens > kXTwoParts && 2 * tokens > vocab; }
// Rows (of tokens) after which dz's second part begins (0: it has none).
int dz_low(int64_t tokens, int64_t vocab) {
    if (!many_per_class(tokens, vocab)) return low_rows(tokens);
    return tokens > kXTwoPartsMost ? 0 : tokens <= kXFewTokens ? few_columns(tokens) : (int)tokens;
}
int64_t dz_rows(int64_t tokens, int64_t vocab) {
    const int low = dz_low(tokens, vocab);
    return low ? 2 * low : tokens;
}

// Classes per piece of the backward: as many whole column tiles as dz's scratch holds.
int64_t piece_classes(int64_t tokens, int64_t vocab) {
    const int64_t fit = kXPieceBytes / (2 * dz_rows(tokens, vocab)) / kXTile * kXTile;
    const int64_t all = round_up(vocab, kXTile);
    return fit < kXTile ? kXTile : fit < all ? fit : all;
}

// Shares of dh's sum over the classes of a piece: the count whose waves of tiles over the pairs
// of SMs take the least time, a K block (64 classes) being the unit and the traffic of the
// shares' sums (4 bytes written and read again per element, about 1.2 MB in the time of a K
// block) added; no share is empty and all fit their scratch.
int dh_splits(int64_t tokens, int64_t classes, int64_t d) {
    const int64_t tiles = (tokens <= kXFewTokens ? 1 : cut(tokens, kXTile)) * cut(d, kXTile), nkb = cut(classes, kXK);
    const int64_t pairs = sm_count() / 2;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int64_t s = 1; s <= 64 && s <= nkb; ++s) {
        if (s > 1 && 4 * s * tokens * d > kXSumBytes) break;
        const int64_t per = cut(nkb, s);
        if (cut(nkb, per) != s) continue;
        const int64_t time = cut(tiles * s, pairs) * (per + 8) + (s > 1 ? 8 * s * tokens * d / 1200000 : 0);
        if (time < least) {
            least = time;
            best = (int)s;
        }
    }
    return best;
}

struct BackwardPlan {
    int64_t piece;
    int splits;
    bool direct;  // one piece and one share: dh straight to bf16
};
BackwardPlan plan_backward(int64_t tokens, int64_t vocab, int64_t d) {
    BackwardPlan p;
    p.piece = piece_classes(tokens, vocab);
    p.splits = dh_splits(tokens, p.piece < vocab ? p.piece : vocab, d);
    p.direct = p.piece >= vocab && p.splits == 1 && tokens <= kXTwoParts;  // (else made up: see rest)
    return p;
}

// Pairs per token that the forward leaves to be joined: one per half of a column tile, or one
// per 32 classes of the transposed product.
int64_t stat_slots(int64_t tokens, int64_t vocab) {
    return (tokens <= kXFewTokens ? 8 : 2) * cut(vocab, kXTile);
}

}  // namespace

int64_t xent_fwd_scratch_bytes(int64_t tokens, int64_t vocab) {
    return round_up(8 * tokens * stat_slots(tokens, vocab), 256) + round_up(4 * tokens, 256);
}

int64_t xent_bwd_scratch_bytes(int64_t tokens, int64_t vocab, int64_t d) {
    const BackwardPlan p = plan_backward(tokens, vocab, d);
    return round_up(2 * dz_rows(tokens, vocab) * p.piece, 256) + (p.direct ? 0 : round_up(4 * p.splits * tokens * d, 256));
}

// z of tokens and classes (nv rows of W), its epilogue kEpi: stats or dz.
template <int kEpi>
static int xent_logits(const uint16_t* h, const uint16_t* W, int64_t tokens, int64_t nv, int64_t d, XentEpilogue e,
                       cudaStream_t stream) {
    if (tokens <= kXFewTokens) {
        e.rows = nv;
        e.cols = tokens;
        return xent_launch<kEpi, false, false, true>(W, d, h, d, nv, tokens, d, few_columns(tokens), 1, false, e, stream);
    }
    e.rows = tokens;
    e.cols = nv;
    return xent_launch<kEpi, false, false, false>(h, d, W, d, tokens, nv, d, kXTile, 1, false, e, stream);
}

// dz W: shares of the sum over the classes, or the whole as bf16.
template <int kEpi>
static int xent_dh(const uint16_t* dz, int64_t piece, const uint16_t* W, int64_t tokens, int64_t nv, int64_t d, int splits,
                   XentEpilogue e, cudaStream_t stream) {
    if (tokens <= kXFewTokens) {
        e.rows = d;
        e.cols = tokens;
        const int low = low_rows(tokens);  // (B: the rows of both parts)
        return xent_launch<kEpi, true, false, true>(W, d, dz, piece, d, low ? 2 * low : tokens, nv,
                                                    low ? 2 * low : few_columns(tokens), splits, false, e, stream, low);
    }
    if constexpr (kEpi == kPartial) {
        e.rows = tokens;
        e.cols = d;
        return xent_launch<kEpi, false, true, false>(dz, piece, W, d, tokens, d, nv, kXTile, splits, false, e, stream);
    }
    return NQ_ERR_SHAPE;  // (as bf16 at once: few tokens alone)
}

int xent_forward(const uint16_t* h, const uint16_t* W, const int32_t* labels, int64_t tokens, int64_t vocab, int64_t d,
                 float* loss, float* lse, void* scratch, cudaStream_t stream) {
    const int64_t slots = stat_slots(tokens, vocab);
    XentEpilogue e = {};
    e.slots = (int)slots;
    e.vocab = vocab;
    e.labels = labels;
    e.stats = static_cast<float2*>(scratch);
    e.picked = reinterpret_cast<float*>(static_cast<char*>(scratch) + round_up(8 * tokens * slots, 256));
    const int rc = xent_logits<kStats>(h, W, tokens, vocab, d, e, stream);
    if (rc != NQ_OK) return rc;
    return launch_pdl(xent_join_kernel, dim3((unsigned)tokens), dim3(kXJoinThreads), 0, stream, (const float2*)e.stats,
                      (const float*)e.picked, labels, tokens, vocab, (int)slots, loss, lse) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

int xent_backward(const uint16_t* h, const uint16_t* W, const int32_t* labels, const float* lse, const float* dloss,
                  int64_t tokens, int64_t vocab, int64_t d, uint16_t* dh, uint16_t* dW, void* scratch,
                  cudaStream_t stream) {
    const BackwardPlan plan = plan_backward(tokens, vocab, d);
    const int64_t piece = plan.piece;
    uint16_t* dz = static_cast<uint16_t*>(scratch);
    float* part = reinterpret_cast<float*>(static_cast<char*>(scratch) + round_up(2 * dz_rows(tokens, vocab) * piece, 256));
    for (int64_t v0 = 0; v0 < vocab; v0 += piece) {
        const int64_t nv = vocab - v0 < piece ? vocab - v0 : piece;
        XentEpilogue e = {};
        e.labels = labels;
        e.label0 = v0;
        e.vocab = vocab;
        e.lse = lse;
        e.dloss = dloss;
        e.out = dz;
        e.ldo = piece;
        e.low = dz_low(tokens, vocab);
        // above kXTwoParts tokens what bf16 leaves of dz at the labels: in dh's rows, which are written last,
        // or, with dW alone, where dh's sums would be
        if (tokens > kXTwoParts) {
            e.rest = dh ? reinterpret_cast<float*>(dh) : part;
            e.rest_pitch = dh ? (int)(d / 2) : 1;
        }
        int rc = xent_logits<kDz>(h, W + v0 * d, tokens, nv, d, e, stream);
        if (rc != NQ_OK) return rc;
        if (dW) {
            XentEpilogue g = {};
            g.rows = nv;
            g.cols = d;
            g.out = dW + v0 * d;
            g.ldo = d;
            if (!many_per_class(tokens, vocab)) {
                g.labels = labels;
                g.label0 = v0;
                g.rest = e.rest;
                g.rest_pitch = e.rest_pitch;
                g.other = h;
                g.tokens = tokens;
            }
            rc = g.rest ? xent_launch<kMadeUp, true, true, false>(dz, piece, h, d, nv, d, tokens, kXTile, 1, true, g, stream, e.low)
                        : xent_launch<kToBf16, true, true, false>(dz, piece, h, d, nv, d, tokens, kXTile, 1, true, g, stream, e.low);
            if (rc != NQ_OK) return rc;
        }
        if (dh) {
            XentEpilogue g = {};
            if (plan.direct) {
                g.out = dh;
                g.ldo = d;
                rc = xent_dh<kToBf16>(dz, piece, W + v0 * d, tokens, nv, d, 1, g, stream);
            } else {
                // the last piece may have fewer K blocks than shares: then it adds to the first ones
                g.part = part;
                g.first = v0 == 0;
                g.labels = labels;
                g.label0 = v0;
                g.vocab = v0 + nv;
                g.rest = e.rest;
                g.rest_pitch = e.rest_pitch;
                g.other = W + v0 * d;
                const int64_t nkb = cut(nv, kXK), per = cut(nkb, plan.splits);
                rc = xent_dh<kPartial>(dz, piece, W + v0 * d, tokens, nv, d, (int)cut(nkb, per), g, stream);
            }
            if (rc != NQ_OK) return rc;
        }
    }
    if (dh && !plan.direct) {
        const int64_t count = tokens * d, blocks = cut(count, 1024), cap = 16 * (int64_t)sm_count();
        if (launch_pdl(xent_sum_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, stream,
                       (const float*)part, plan.splits, count, dh) != cudaSuccess)
            return NQ_ERR_CUDA;
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
