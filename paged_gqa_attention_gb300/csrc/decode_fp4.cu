// decode_fp4.cu -- batched single-token GQA attention over the 4-bit KV cache, with an optional
// sliding window.
//
// The attention is that of decode.cu (page "扔掉 vLLM！从零构建 Qwen3-8B 推理引擎，C++/CUDA 实现性能追平
// 98%" §4.4.2: the four query heads of a group share every KV read; split-K over the context with a
// log-sum-exp merge); the cache is one step below the 8 bits of page "从零搭建AI工程能力：手写KV Cache与
// 动态批处理实战" §3.2 (format: fp4.cuh): 146 bytes per token and KV head instead of 512.
//
// What bounds it is the work a byte asks for, two values to convert and scale: 620 warp instructions for 32
// tokens, 128 of them conversions, at half rate on a pipe that is 60 % busy (64 sequences of 8192 to 16384 tokens,
// unsplit).  Hence:
//   * a stage is a whole 256-token block of K and V (16 KiB of codes each, TMA, 64-byte swizzle; 2 KiB of
//     scales and 256 exponents each, bulk copies), consumed by 8 warps of 32 tokens; three stages, two
//     CTAs per SM.  Two 16-token tiles a warp give every step of the chain (scores, softmax, output) two
//     independent halves, and share the votes and the rescaling;
//   * products in f16 (mma.sync), whose 8 columns are twice the 4 heads: code * scale has 6 bits and is exact.
//     S: ldmatrix on the codes gives a lane 8 consecutive dims of a token, two k16 steps once Q is loaded in
//     that order, all 8 in one scale group, and the two steps hold both groups of a 32-dim piece side by
//     side.  Columns 0..3 have Q in the first group's rows and zeros in the other's, columns 4..7 the
//     reverse: a product is a group's sum, which takes its scale in fp32 (one multiply-add for 16 codes and a
//     head instead of a multiply for every pair), and an exchange between lanes adds the halves up;
//   * O: the transposed ldmatrix gives a lane 4 dims of two tokens, and a converted byte is two dims of one token.
//     So the k16 step takes 8 tokens twice: columns 0..3 have (P, 0) and sum the even dims, columns 4..7 (0, P)
//     the odd ones.  No operand is permuted and no column idle; the accumulator of piece c holds dims
//     32c + 4r (rows r < 8), 32c + 4(r - 8) + 2, and one more in columns 4..7;
//   * the row's power of two enters S in fp32, and for V through P: each warp accumulates
//     P * 2^(e - sigma) in f16, sigma the largest exponent it has seen (of rows that are not zero), and rescales its
//     accumulator when sigma grows, as the online softmax does for its maximum.  A lane looks a token up and hands
//     on what the others need of it;
//   * tokens that are not attended to get scale 0 in V (every code is finite) and score -infinity.
// Measured: 64 sequences of 8192 to 16384 tokens 191 us (933 MB: 4.9 TB/s; with a multiply and a permute for
// every pair 274), 64 of 16384 227 us (5.3 TB/s), 32 of 128 to 4096 28.6, one of 9001 10.0, one tile 5.0.
#include <cuda_fp16.h>

#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "window.cuh"

namespace pa {
namespace {

constexpr int kTile = kDecodeFp4TileTokens;   // 256 tokens per stage: a cache block
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kWarpTokens = 32;
constexpr int kConsumerWarps = kTile / kWarpTokens;   // 8
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr int kCodeBytes = kTile * kFp4RowCodes;      // 16 KiB
constexpr int kScaleBytes = kTile * kFp4Groups;       // 2 KiB
constexpr uint32_t kSideTx = 2 * (kScaleBytes + kTile);
constexpr float kLn2 = 0.693147180559945309f;
constexpr int kNoSigma = -1000;

struct MergeArrays {                          // the warps' partial results, after the stages
    float o[kConsumerWarps][kGroup][kD];
    float m[kConsumerWarps][kGroup];
    float l[kConsumerWarps][kGroup];
    int sigma[kConsumerWarps];
};

struct DecodeFp4Smem {
    union {
        uint8_t codes[kStages][2][kCodeBytes];  // [stage][K, V], each 1 KiB aligned
        MergeArrays mg;                         // reused once every stage is consumed
    };
    uint8_t scales[kStages][2][kScaleBytes];
    uint8_t exps[kStages][2][kTile];
    uint64_t full[kStages];
    uint64_t empty[kStages];
    int last_cta;
    int poison;
    float cl_ml[kGroup][2];                    // cluster merge: this split's (m, l) per head
};

constexpr size_t kSmemBytes = sizeof(DecodeFp4Smem) + 1024;
static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");

__device__ __forceinline__ void store_out4(__nv_bfloat16 *dst, const float (&v)[4], float inv) {
    uint2 w;
    w.x = pack_bf16x2(v[0] * inv, v[1] * inv);
    w.y = pack_bf16x2(v[2] * inv, v[3] * inv);
    *reinterpret_cast<uint2 *>(dst) = w;
}

// Byte offset of 16-byte piece `piece` (0..3) of row `row` of a tile of 64-byte rows written by TMA with
// 64-byte swizzling.
__device__ __forceinline__ uint32_t sw64(int row, int piece) {
    return (uint32_t)(row * kFp4RowCodes + ((piece ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two E4M3 bytes -> f16x2 (the lower byte in the low half)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t d;
    asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}" : "=r"(d) : "r"(two));
    return d;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t a) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&a));
}

// One half of an f16x2, twice
__device__ __forceinline__ uint32_t low_f16x2(uint32_t a) {
    uint32_t d;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n mov.b32 %0, {l, l};\n}" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t high_f16x2(uint32_t a) {
    uint32_t d;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n mov.b32 %0, {h, h};\n}" : "=r"(d) : "r"(a));
    return d;
}

// 2^n for n <= 127, 0 below the normal range.
__device__ __forceinline__ float pow2_or_0(int n) { return n < -126 ? 0.f : __uint_as_float((uint32_t)(n + 127) << 23); }

template <bool kCluster>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
decode_fp4_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const __grid_constant__ CUtensorMap k16_map, const __grid_constant__ CUtensorMap v16_map,
                  const DecodeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    DecodeFp4Smem &sm = *reinterpret_cast<DecodeFp4Smem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    const int pair = blockIdx.x;          // sequence * 8 + kv head
    const int b = pair / kHkv;
    const int g = pair % kHkv;
    // the highest splits start first (longest work first, as in decode.cu)
    const int split = kCluster ? (int)blockIdx.y : (int)(gridDim.y - 1 - blockIdx.y);
    // a CTA without work: with a cluster, all of its threads meet the others at both barriers
    const auto leave = [] {
        if constexpr (kCluster) {
            __syncwarp();
            cluster_sync_all();
            cluster_sync_all();
        }
    };
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    const int32_t *bt = a.block_table + (size_t)b * a.max_blocks_per_seq;
    if (warp == kConsumerWarps && lane == 0) {
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
        tma_prefetch_map(&k16_map);
        tma_prefetch_map(&v16_map);
    }
    const int seq_len = __ldg(a.seq_lens + b);
    // an empty sequence (a padded row of the batch) has nothing to see: zeros, lse -inf
    if (seq_len == 0) {
        if (split == 0 && warp < kGroup) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            const int qh = g * kGroup + warp;
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            store_out4(static_cast<__nv_bfloat16 *>(a.out) + ((size_t)b * kHq + qh) * kD + lane * 4, zero, 0.f);
            if (a.lse && lane == 0) a.lse[(size_t)b * kHq + qh] = -INFINITY;
        }
        leave();
        return;
    }
    if (seq_len < 1 || seq_len > a.max_blocks_per_seq * kBlock) {
        if (split == 0 && g == 0 && threadIdx.x == 0) record_error(a.err, kErrDevice | kErrBadSeqLen);
        // (a kernel whose CTAs all left here must not complete before the one it depends on)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        leave();
        return;
    }
    const WindowTiles<kTile> wt(a.window, a.sinks, seq_len - 1, seq_len - 1);
    const int per_split = a.split_tokens / kTile;
    const int nsplit_b = (wt.n + per_split - 1) / per_split;
    if (split >= nsplit_b) {              // past the context
        leave();
        return;
    }
    // tiles v_begin .. v_begin + n_tiles - 1 of the list of visible ones
    const int v_len = (wt.n + nsplit_b - 1) / nsplit_b;
    const int v_begin = split * v_len;
    const int n_tiles = min(v_len, wt.n - v_begin);

    if (threadIdx.x == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), kConsumerWarps);
        }
        sm.poison = 0;
        fence_barrier_init();
    }
    __syncthreads();

    if (warp == kConsumerWarps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            // the cache may be written by the kernel just before this one on the stream
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int issued = 0;
            for (int i = 0; i < n_tiles; ++i) {
                const int st = i % kStages;
                if (i >= kStages && !mbar_wait(smem_u32(&sm.empty[st]), ((i / kStages) - 1) & 1)) {
                    record_error(a.err, kErrTimeout);
                    break;
                }
                const int tok = wt.tile(v_begin + i) * kTile;
                int blk = __ldg(bt + tok / kBlock);
                if (blk < 0 || blk >= a.num_blocks) {
                    record_error(a.err, kErrDevice | kErrBadBlock);
                    sm.poison = 1;
                    blk = 0;
                }
                const uint32_t bar = smem_u32(&sm.full[st]);
                const size_t srow = ((size_t)blk * kHkv + g) * kBlock;
                // the stage's 16-row groups that hold a visible token
                uint32_t need = 0;
#pragma unroll
                for (int r = 0; r < kTile / 16; ++r)
                    if (tok + 16 * r < seq_len && wt.sees_any(tok + 16 * r, 16)) need |= 1u << r;
                if (need == (1u << (kTile / 16)) - 1) {
                    mbar_arrive_expect_tx(bar, 2 * kCodeBytes + kSideTx);
                    tma_load_4d(smem_u32(sm.codes[st][0]), &k_map, bar, 0, g, 0, blk);
                    tma_load_4d(smem_u32(sm.codes[st][1]), &v_map, bar, 0, g, 0, blk);
                } else {
                    mbar_arrive_expect_tx(bar, __popc(need) * 16 * 2 * kFp4RowCodes + kSideTx);
                    for (int r = 0; r < kTile / 16; ++r) {
                        if (!(need >> r & 1u)) continue;
                        tma_load_4d(smem_u32(sm.codes[st][0] + r * 16 * kFp4RowCodes), &k16_map, bar, 0, g, 16 * r, blk);
                        tma_load_4d(smem_u32(sm.codes[st][1] + r * 16 * kFp4RowCodes), &v16_map, bar, 0, g, 16 * r, blk);
                    }
                }
                bulk_load(smem_u32(sm.scales[st][0]), a.k_scale4 + srow * kFp4Groups, kScaleBytes, bar);
                bulk_load(smem_u32(sm.exps[st][0]), a.k_exp + srow, kTile, bar);
                bulk_load(smem_u32(sm.scales[st][1]), a.v_scale4 + srow * kFp4Groups, kScaleBytes, bar);
                bulk_load(smem_u32(sm.exps[st][1]), a.v_exp + srow, kTile, bar);
                issued = i + 1;
            }
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(smem_u32(&sm.full[i % kStages]), (i / kStages) & 1);
        }
        leave();
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int w = warp;
    const int gq = lane >> 2;   // fragment row group
    const int tq = lane & 3;    // fragment column pair
    const int mi = lane >> 3;   // ldmatrix: which 8x8 matrix this lane addresses
    const int ri = lane & 7;    // ldmatrix: row within it

    // q may come from the kernel just before this one on the stream
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Q^T as the B operand of S^T = K Q^T, f16: of 32-dim piece c, k16 step u holds dims 32c + 8tq + 4u ..
    // + 3 of head gq & 3 (the order the code fragments arrive in); columns 0..3 have the piece's first 16
    // dims (tq < 2) and zeros, columns 4..7 the other 16.
    uint32_t qb[4][2][2];
    {
        const uint4 *qrow = reinterpret_cast<const uint4 *>(
            static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * kHq + g * kGroup + (gq & 3)) * kD);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 v = (gq >> 2) == (tq >> 1) ? __ldg(qrow + c * 4 + tq) : make_uint4(0u, 0u, 0u, 0u);
            qb[c][0][0] = bf16x2_to_f16x2(v.x);
            qb[c][0][1] = bf16x2_to_f16x2(v.y);
            qb[c][1][0] = bf16x2_to_f16x2(v.z);
            qb[c][1][1] = bf16x2_to_f16x2(v.w);
        }
    }

    float m0 = -INFINITY, m1 = -INFINITY;   // running max (log2 units) of heads 2tq, 2tq+1 (mod 4)
    float l0 = 0.f, l1 = 0.f;               // this thread's share of the running sums
    int sigma = kNoSigma;                   // exponent that the accumulator is in units of
    float acc[4][4];                        // O^T tiles
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;

    const int row = w * kWarpTokens + ri + ((mi & 1) << 3);   // token row addressed by this lane (+ 16 u)
    const uint32_t pick_k = tq & 2 ? 0x7531u : 0x6420u;       // odd or even bytes of a token's 8 scales
    const uint32_t pick_v = gq & 4 ? 0x7531u : 0x6420u;
    // P of a token beside a zero: even dims (columns 0..3) take it in the lower half, odd ones in the upper
    const uint32_t pick_p0 = gq & 4 ? 0x1044u : 0x4410u, pick_p1 = gq & 4 ? 0x3244u : 0x4432u;

    for (int i = 0; i < n_tiles; ++i) {
        const int st = i % kStages;
        if (!mbar_wait(smem_u32(&sm.full[st]), (i / kStages) & 1)) {
            if (lane == 0) record_error(a.err, kErrTimeout);
            break;
        }
        // this warp's 32 rows hold positions p_w .. p_w + 31
        const int p_w = wt.tile(v_begin + i) * kTile + w * kWarpTokens;
        if (p_w < seq_len && wt.sees_any(p_w, kWarpTokens)) {
            const uint32_t kc = smem_u32(sm.codes[st][0]);
            const uint32_t vc = smem_u32(sm.codes[st][1]);
            const uint8_t *ksc = sm.scales[st][0] + w * kWarpTokens * kFp4Groups;
            const uint8_t *vsc = sm.scales[st][1] + w * kWarpTokens * kFp4Groups;

            // lane l's token is p_w + l: whether it is attended to, K's factor, V's exponent
            const bool ok = p_w + lane < seq_len && wt.sees(p_w + lane);
            const uint32_t seen = __ballot_sync(0xffffffffu, ok);
            const float kf = fp4_unit(sm.exps[st][0][w * kWarpTokens + lane]) * a.scale_log2;
            const uint32_t ev = sm.exps[st][1][w * kWarpTokens + lane];
            int ve = !ok || ev == 0 ? kNoSigma : (int)ev - 127;   // 128: NaN

            // S^T[2 x 16 tokens x 8 columns] = K . Q^T, 64 dims per ldmatrix
            float x[2][4];
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // scales of tokens gq and gq + 8, one byte per 32-dim piece (this column's 16-dim half of it)
                uint32_t sc[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(ksc + (16 * u + 8 * h + gq) * kFp4Groups);
                    sc[h] = __byte_perm(y.x, y.y, pick_k);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[u][e] = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t r[4];
                    ldsm_x4(r, kc + sw64(row + 16 * u, 2 * j + (mi >> 1)));
                    float2 f[2];   // per token: scales of pieces 2j and 2j + 1
#pragma unroll
                    for (int h = 0; h < 2; ++h) f[h] = f16x2_to_f32x2(e4m3x2_to_f16x2(sc[h] >> (16 * j)));
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t lo[4], hi[4];
                        e2m1x8_to_f16x2x4(r[2 * c], lo);        // token gq, dims 32(2j+c) + 8tq ..
                        e2m1x8_to_f16x2x4(r[2 * c + 1], hi);    // token gq + 8
                        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const uint32_t af[4] = {lo[2 * v], hi[2 * v], lo[2 * v + 1], hi[2 * v + 1]};
                            mma_16816_f16(s, af, qb[2 * j + c][v][0], qb[2 * j + c][v][1]);
                        }
                        const float f_lo = c ? f[0].y : f[0].x, f_hi = c ? f[1].y : f[1].x;
                        x[u][0] = fmaf(s[0], f_lo, x[u][0]);
                        x[u][1] = fmaf(s[1], f_lo, x[u][1]);
                        x[u][2] = fmaf(s[2], f_hi, x[u][2]);
                        x[u][3] = fmaf(s[3], f_hi, x[u][3]);
                    }
                }
                // the other half of every piece; then x[u][2h + e]: (token 16u + 8h + gq, head 2tq + e mod 4)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = 16 * u + 8 * h + gq;
                    const float k = __shfl_sync(0xffffffffu, kf, t);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &y = x[u][2 * h + e];
                        y = (y + __shfl_xor_sync(0xffffffffu, y, 2)) * k;
                        if (seen != 0xffffffffu && !(seen >> t & 1u)) y = -INFINITY;
                    }
                    mx0 = fmaxf(mx0, x[u][2 * h]);
                    mx1 = fmaxf(mx1, x[u][2 * h + 1]);
                }
            }
            // lazy rescaling, as in decode_fp8.cu: one vote finds the tiles in which a maximum has grown by
            // more than 2^8 or a V exponent is the largest so far, and only they reduce over the warp
            if (__any_sync(0xffffffffu, mx0 > m0 + 8.f || mx1 > m1 + 8.f || (ve > sigma && ve < 128))) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
                }
                const bool up0 = mx0 > m0 + 8.f, up1 = mx1 > m1 + 8.f;   // also when m == -inf
                const float mn0 = up0 ? mx0 : m0, mn1 = up1 ? mx1 : m1;
                const float alpha0 = up0 ? fast_exp2(m0 - mn0) : 1.f, alpha1 = up1 ? fast_exp2(m1 - mn1) : 1.f;
                m0 = mn0;
                m1 = mn1;
                l0 *= alpha0;
                l1 *= alpha1;
                // a zero row (every scale 0) has the exponent 2^0, far above rows of ordinary size: it sets no unit
                // (and needs none; rows at or below sigma do not matter)
                if (ve > sigma && ve < 128) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(vsc + lane * kFp4Groups);
                    if ((y.x | y.y) == 0u) ve = kNoSigma;
                }
                const int top = __reduce_max_sync(0xffffffffu, ve < 128 ? ve : kNoSigma);
                const float grow = top > sigma ? pow2_or_0(sigma - top) : 1.f;
                sigma = max(sigma, top);
                const float f0 = alpha0 * grow, f1 = alpha1 * grow;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[c][0] *= f0;
                    acc[c][1] *= f1;
                    acc[c][2] *= f0;
                    acc[c][3] *= f1;
                }
            }
            const float vf = ve == 128 ? __int_as_float(0x7fc00000) : pow2_or_0(ve - sigma);
            uint32_t pb[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = fast_exp2(x[u][2 * h] - m0), p1 = fast_exp2(x[u][2 * h + 1] - m1);
                    l0 += p0;
                    l1 += p1;
                    const float r = __shfl_sync(0xffffffffu, vf, 16 * u + 8 * h + gq);
                    // P^T as the B operand of O^T += V^T P^T: transpose the 8x8 16-bit blocks
                    pb[u][h] = movmatrix_trans(pack_f16x2(p0 * r, p1 * r));
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // scales of tokens 2tq, 2tq + 1 of both halves, one byte per 32-dim piece
                uint32_t sc[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = 16 * u + 8 * h + 2 * tq;
                    const uint4 y = *reinterpret_cast<const uint4 *>(vsc + t * kFp4Groups);
                    sc[h][0] = __byte_perm(y.x, y.y, pick_v);
                    sc[h][1] = __byte_perm(y.z, y.w, pick_v);
                    if (seen != 0xffffffffu) {
                        if (!(seen >> t & 1u)) sc[h][0] = 0u;
                        if (!(seen >> t & 2u)) sc[h][1] = 0u;
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // matrices: tokens 0-7 / 8-15 of the tile x pieces 2j / 2j + 1
                    uint32_t r[4];
                    ldsm_x4_trans(r, vc + sw64(row + 16 * u, 2 * j + (mi >> 1)));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t b0 = __byte_perm(pb[u][h], 0u, pick_p0), b1 = __byte_perm(pb[u][h], 0u, pick_p1);
                        const uint32_t f0 = e4m3x2_to_f16x2(sc[h][0] >> (16 * j)), f1 = e4m3x2_to_f16x2(sc[h][1] >> (16 * j));
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t d[4];   // {token 2tq: dims 4gq, +1; +2, +3; token 2tq + 1: ..}
                            e2m1x8_to_f16x2x4(r[2 * c + h], d);
                            const uint32_t s0 = c ? high_f16x2(f0) : low_f16x2(f0), s1 = c ? high_f16x2(f1) : low_f16x2(f1);
                            const uint32_t af[4] = {mul_f16x2(d[0], s0), mul_f16x2(d[1], s0), mul_f16x2(d[2], s1),
                                                    mul_f16x2(d[3], s1)};
                            mma_16816_f16(acc[2 * j + c], af, b0, b1);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.empty[st]));
    }

    // ------------------------------------------------------------ merge the warps
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    // the merge arrays overlay the stages: every consumer warp must be done with them
    named_barrier(1, kConsumerWarps * 32);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int d = c * 32 + 4 * gq + (tq >> 1), hd = 2 * (tq & 1);
        sm.mg.o[w][hd][d] = acc[c][0];
        sm.mg.o[w][hd + 1][d] = acc[c][1];
        sm.mg.o[w][hd][d + 2] = acc[c][2];
        sm.mg.o[w][hd + 1][d + 2] = acc[c][3];
    }
    if (tq < 2 && gq == 0) {
        sm.mg.m[w][2 * tq] = m0;
        sm.mg.m[w][2 * tq + 1] = m1;
        sm.mg.l[w][2 * tq] = l0;
        sm.mg.l[w][2 * tq + 1] = l1;
    }
    if (lane == 0) sm.mg.sigma[w] = sigma;
    named_barrier(1, kConsumerWarps * 32);
    const bool bad = *reinterpret_cast<volatile int *>(&sm.poison) != 0;

    // the first 128 consumer threads merge (4 heads x 32 threads x 4 dims)
    const int c = threadIdx.x;
    if (c >= kGroup * 32) {
        // the others only take part in the partials' barriers below
        if (kCluster) {
            leave();
        } else if (nsplit_b > 1) {
            named_barrier(2, kConsumerWarps * 32);
            named_barrier(2, kConsumerWarps * 32);
        }
        return;
    }
    const int h = c >> 5;               // query head within the group
    const int d0 = (c & 31) * 4;        // 4 dims per thread
    float M = -INFINITY;
#pragma unroll
    for (int ww = 0; ww < kConsumerWarps; ++ww) M = fmaxf(M, sm.mg.m[ww][h]);
    float L = 0.f, o4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ww = 0; ww < kConsumerWarps; ++ww) {
        const float e = fast_exp2(sm.mg.m[ww][h] - M);
        L += sm.mg.l[ww][h] * e;
        const float eo = e * pow2_or_0(sm.mg.sigma[ww]);
#pragma unroll
        for (int k = 0; k < 4; ++k) o4[k] += sm.mg.o[ww][h][d0 + k] * eo;
    }
    if (bad) {
        M = L = __int_as_float(0x7fc00000);
#pragma unroll
        for (int k = 0; k < 4; ++k) o4[k] = __int_as_float(0x7fc00000);
    }
    const int qh = g * kGroup + h;      // query head
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + ((size_t)b * kHq + qh) * kD + d0;

    if constexpr (kCluster) {
        // this split's partial into its own shared memory: thread c alone read entries
        // [.][h][d0 .. d0+3] of the merge arrays, so it may overwrite warp 0's
        *reinterpret_cast<float4 *>(&sm.mg.o[0][h][d0]) = make_float4(o4[0], o4[1], o4[2], o4[3]);
        if ((c & 31) == 0) {
            sm.cl_ml[h][0] = M;
            sm.cl_ml[h][1] = L;
        }
        cluster_sync_all();   // every split's partial is in place
        if (split == 0) {
            float GM = M;
            for (int k = 1; k < nsplit_b; ++k)
                GM = fmaxf(GM, ld_cluster_f32(peer_addr(smem_u32(&sm.cl_ml[h][0]), (uint32_t)k)));
            float GL = 0.f, go[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < nsplit_b; ++k) {
                const float mk = ld_cluster_f32(peer_addr(smem_u32(&sm.cl_ml[h][0]), (uint32_t)k));
                const float lk = ld_cluster_f32(peer_addr(smem_u32(&sm.cl_ml[h][1]), (uint32_t)k));
                const float4 ok = ld_cluster_f4(peer_addr(smem_u32(&sm.mg.o[0][h][d0]), (uint32_t)k));
                const float e = fast_exp2(mk - GM);
                GL += lk * e;
                go[0] += ok.x * e;
                go[1] += ok.y * e;
                go[2] += ok.z * e;
                go[3] += ok.w * e;
            }
            if (nsplit_b > 1 && !(GL == GL)) GM = GL;   // a poisoned split (its NaN maximum loses in fmaxf)
            store_out4(out, go, 1.f / GL);
            if (a.lse && (c & 31) == 0) a.lse[(size_t)b * kHq + qh] = (GM + __log2f(GL)) * kLn2;
        }
        cluster_sync_all();   // the peers' shared memory stays until split 0 has read it
        return;
    }

    if (nsplit_b == 1) {
        store_out4(out, o4, 1.f / L);
        if (a.lse && (c & 31) == 0) a.lse[(size_t)b * kHq + qh] = (M + __log2f(L)) * kLn2;
        return;
    }

    // ------------------------------------------------------------ split-K partials
    const size_t entry = (size_t)pair * a.nsplit + split;
    *reinterpret_cast<float4 *>(a.part_o + (entry * kGroup + h) * kD + d0) =
        make_float4(o4[0], o4[1], o4[2], o4[3]);
    if ((c & 31) == 0) {
        a.part_ml[(entry * kGroup + h) * 2 + 0] = M;
        a.part_ml[(entry * kGroup + h) * 2 + 1] = L;
    }
    __threadfence();
    named_barrier(2, kConsumerWarps * 32);
    if (c == 0) {
        const int prev = atomicAdd(a.counters + pair, 1);
        sm.last_cta = (prev == nsplit_b - 1);
    }
    named_barrier(2, kConsumerWarps * 32);
    if (!sm.last_cta) return;

    // The last CTA of this (sequence, KV head) merges every split by log-sum-exp.
    __threadfence();
    if (c == 0) a.counters[pair] = 0;   // ready for the next call
    const size_t e0 = (size_t)pair * a.nsplit;
    float GM = -INFINITY;
    for (int k = 0; k < nsplit_b; ++k) GM = fmaxf(GM, __ldcg(a.part_ml + ((e0 + k) * kGroup + h) * 2));
    float GL = 0.f, go[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < nsplit_b; ++k) {
        const float mk = __ldcg(a.part_ml + ((e0 + k) * kGroup + h) * 2);
        const float lk = __ldcg(a.part_ml + ((e0 + k) * kGroup + h) * 2 + 1);
        const float e = fast_exp2(mk - GM);
        const float4 ok = __ldcg(reinterpret_cast<const float4 *>(a.part_o + ((e0 + k) * kGroup + h) * kD + d0));
        GL += lk * e;
        go[0] += ok.x * e;
        go[1] += ok.y * e;
        go[2] += ok.z * e;
        go[3] += ok.w * e;
    }
    if (!(GL == GL)) GM = GL;
    store_out4(out, go, 1.f / GL);
    if (a.lse && (c & 31) == 0) a.lse[(size_t)b * kHq + qh] = (GM + __log2f(GL)) * kLn2;
}

// As much shared memory as lets one CTA alone onto an SM
constexpr size_t kLoneBytes = 131072;
static_assert(kLoneBytes >= kSmemBytes && 2 * (kLoneBytes + 1024) > 233472, "one CTA per SM");

}  // namespace

cudaError_t decode_fp4_clusters(ClusterRoom &room) {
    static std::atomic<int> known[64][2][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    for (int c = 2; c <= 8; ++c) {
        for (int two = 0; two < 2; ++two) {
            int &out = two ? room.fit[c] : room.lone[c];
            out = known[dev][two][c].load();
            if (out != 0) continue;
            e = cudaFuncSetAttribute(decode_fp4_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLoneBytes);
            if (e != cudaSuccess) return e;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1;
            attr[0].val.clusterDim.y = (unsigned)c;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1, (unsigned)c);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = two ? kSmemBytes : kLoneBytes;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, decode_fp4_kernel<true>, &cfg) != cudaSuccess) {
                cudaGetLastError();   // none this time; asked again next time
                continue;
            }
            out = n > 0 ? n : -1;
            known[dev][two][c].store(out);
        }
    }
    return cudaSuccess;
}

cudaError_t launch_decode_fp4(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                              const CUtensorMap &k16_map, const CUtensorMap &v16_map, cudaStream_t stream) {
    if (a.batch == 0) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> configured[64] = {};
    if (dev < 0 || dev >= 64 || !configured[dev].load()) {
        e = cudaFuncSetAttribute(decode_fp4_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        // (as decode_fp4_clusters sets it)
        e = cudaFuncSetAttribute(decode_fp4_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLoneBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * kHkv, a.nsplit);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.cluster_merge) {
        if (a.nsplit < 1 || a.nsplit > 8) return cudaErrorInvalidValue;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = (unsigned)a.nsplit;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, decode_fp4_kernel<true>, k_map, v_map, k16_map, v16_map, a);
        if (e != cudaErrorLaunchOutOfResources && e != cudaErrorInvalidClusterSize && e != cudaErrorNotSupported &&
            e != cudaErrorCooperativeLaunchTooLarge)
            return e;
        cudaGetLastError();   // the cluster was refused: merge through the workspace instead
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, decode_fp4_kernel<false>, k_map, v_map, k16_map, v16_map, a);
}

}  // namespace pa
