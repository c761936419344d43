// kv_read.cu -- rows of the 8-bit or the 4-bit cache read back as bf16.
//
// Page "从零搭建AI工程能力：手写KV Cache与动态批处理实战" §3.2 stores the KV cache in 8 bits; what is
// stored has to come out again where a sequence moves to another cache or to a consumer of plain
// rows.  Row i of sequence s (row cu_rows[s] + i of the outputs) is the token at position first[s] + i:
// slot p % 256 of block block_table[s][p / 256], all 8 KV heads.  A value is code * scale in fp32 (8 bits),
// or code * scale * 2^(e - 127), exact (4 bits), rounded to bf16.
//
// The pass reads 132 or 73 bytes a row and writes 256: it is bound by HBM.  A warp takes 4 consecutive
// rows of K or of V; a lane 16 codes (16 or 8 bytes) at a time, whose 32 bytes of output make the warp's
// stores whole lines, and every load of the 4 rows goes out before the first is used.  The scales of the
// 4 x 8 (row, head) pairs come a pair a lane and are handed round (a load for every 16 codes kept the load
// queues full).  The CTA's 8 warps take 16 rows of K and of V, so that the scales, which lie 256 slots a
// head, come in whole sectors.
// Measured: 94311 tokens from 8 bits 86.8 us (585 MB: 6.75 TB/s, the copy rate), 25078 from 4 bits 20.3 us
// (6.5 TB/s); with a scale load for every 16 codes 100 and 30.9, with 16-byte stores 93 and 29.
#include <cuda_fp16.h>

#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kRowsPerWarp = 4;
constexpr int kRowsPerCta = kRowsPerWarp * kWarps / 2;   // half of the warps read K, half V
constexpr int kChunks = kHkv * kD / 16;                  // 16-value pieces of a token: 64, two a lane

// Where row t of the outputs is in the cache: block * 256 + slot; -1: nowhere (NaN), -2: behind the last
// sequence (left alone).
__device__ __forceinline__ long long place_of(const ReadArgs &a, int t, bool report) {
    int lo = 0, hi = a.num_seqs;   // the last sequence that begins at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu_rows + mid) <= t) lo = mid;
        else hi = mid;
    }
    const int r0 = __ldg(a.cu_rows + lo), r1 = __ldg(a.cu_rows + lo + 1);
    if (t >= r1 && lo == a.num_seqs - 1) return -2;
    if (r0 < 0 || r1 > a.total_rows || t < r0 || t >= r1) {
        if (report) record_error(a.err, kErrDevice | kErrBadCuQ);
        return -1;
    }
    const int first = __ldg(a.first + lo), limit = a.max_blocks_per_seq * kBlock;
    if (first < 0 || first > limit || t - r0 >= limit - first) {
        if (report) record_error(a.err, kErrDevice | kErrBadSeqLen);
        return -1;
    }
    const int p = first + (t - r0);
    const int blk = __ldg(a.block_table + (size_t)lo * a.max_blocks_per_seq + p / kBlock);
    if (blk < 0 || blk >= a.num_blocks) {
        if (report) record_error(a.err, kErrDevice | kErrBadBlock);
        return -1;
    }
    return (long long)blk * kBlock + p % kBlock;
}

template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const ReadArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float group_scale[kBits == 4 ? kWarps : 1][32][kFp4Groups];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool is_v = warp & 1;
    const long long t0 = (long long)blockIdx.x * kRowsPerCta + (warp >> 1) * kRowsPerWarp;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        const int end = __ldg(a.cu_rows + a.num_seqs);
        if (__ldg(a.cu_rows) != 0 || end < 0 || end > a.total_rows) record_error(a.err, kErrDevice | kErrBadCuQ);
    }
    if (t0 >= a.total_rows) return;
    const int rows = (int)min((long long)kRowsPerWarp, a.total_rows - t0);
    const long long mine = lane < rows ? place_of(a, (int)t0 + lane, !is_v) : -2;
    long long place[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) place[r] = __shfl_sync(0xffffffffu, mine, r);

    // the cache may be written, and the outputs still read, by the kernel just before this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint8_t *codes = static_cast<const uint8_t *>(is_v ? a.v_codes : a.k_codes);
    const void *scales = is_v ? a.v_scale : a.k_scale;
    const uint8_t *exps = is_v ? a.v_exp : a.k_exp;
    uint4 c[kRowsPerWarp][2];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            c[r][u] = make_uint4(0u, 0u, 0u, 0u);
            if (place[r] < 0) continue;
            const int chunk = u * 32 + lane;
            if constexpr (kBits == 8) {
                c[r][u] = *(reinterpret_cast<const uint4 *>(codes + place[r] * (kHkv * kD)) + chunk);
            } else {
                const uint2 w = *(reinterpret_cast<const uint2 *>(codes + place[r] * (kHkv * kFp4RowCodes)) + chunk);
                c[r][u].x = w.x;
                c[r][u].y = w.y;
            }
        }
    }
    // what scales KV head l % 8 of row l / 8, in lane l: one load (4 bits: two) for the warp's 32
    const long long at = __shfl_sync(0xffffffffu, mine, lane >> 3);
    const size_t row = at < 0 ? 0 : ((size_t)(at / kBlock) * kHkv + (lane & 7)) * kBlock + (size_t)(at % kBlock);
    float head_scale = __int_as_float(0x7fc00000);   // (of a row that is nowhere)
    if constexpr (kBits == 8) {
        if (at >= 0) head_scale = static_cast<const float *>(scales)[row];
    } else {
        uint2 w = make_uint2(0u, 0u);
        if (at >= 0) {
            w = static_cast<const uint2 *>(scales)[row];
            head_scale = fp4_unit(exps[row]);
        }
        uint32_t h[4];
        e4m3x4_to_f16x2x2(w.x, h[0], h[1]);
        e4m3x4_to_f16x2x2(w.y, h[2], h[3]);
        float4 f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&h[2 * i]));
            const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&h[2 * i + 1]));
            f[i] = make_float4(lo.x * head_scale, lo.y * head_scale, hi.x * head_scale, hi.y * head_scale);
            *reinterpret_cast<float4 *>(&group_scale[warp][lane][4 * i]) = f[i];
        }
        __syncwarp();
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(is_v ? a.v_out : a.k_out);
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        if (place[r] == -2) continue;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t h[8];   // f16 pairs of the codes
            const int from = r * kHkv + u * 4 + (lane >> 3);   // the lane of this chunk's row and head
            float scale;
            if constexpr (kBits == 8) {
                e4m3x4_to_f16x2x2(c[r][u].x, h[0], h[1]);
                e4m3x4_to_f16x2x2(c[r][u].y, h[2], h[3]);
                e4m3x4_to_f16x2x2(c[r][u].z, h[4], h[5]);
                e4m3x4_to_f16x2x2(c[r][u].w, h[6], h[7]);
                scale = __shfl_sync(0xffffffffu, head_scale, from);
            } else {
                uint32_t lo[4], hi[4];
                e2m1x8_to_f16x2x4(c[r][u].x, lo);
                e2m1x8_to_f16x2x4(c[r][u].y, hi);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = lo[e];
                    h[4 + e] = hi[e];
                }
                scale = group_scale[warp][from][lane & 7];
            }
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                w[e] = pack_bf16x2(f.x * scale, f.y * scale);
            }
            st_global_32b(out + (t0 + r) * (kHkv * kD) + (u * 32 + lane) * 16, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
        }
    }
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t stream) {
    if (a.total_rows == 0) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)a.total_rows + kRowsPerCta - 1) / kRowsPerCta));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.k_exp ? cudaLaunchKernelEx(&cfg, kv_read_kernel<4>, a) : cudaLaunchKernelEx(&cfg, kv_read_kernel<8>, a);
}

static_assert(kChunks == 64, "two pieces a lane");

}  // namespace pa
