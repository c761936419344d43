// kv_append.cu -- scatter of new K/V rows into their cache blocks.
//
// Page "扔掉 vLLM！从零构建 Qwen3-8B 推理引擎，C++/CUDA 实现性能追平 98%" §4.3.1
// (KVBlockManager::append): tokens fill a sequence's last 256-token block in order,
// a new block is taken when it is full.  Here the host has already extended the
// block table; the bf16 kernel only moves bytes.  New token i of sequence s lands at
// absolute position p = seq_lens[s] - q_len + i, slot p % 256 of block
// block_table[s][p / 256].  In the pool layout [block][slot][kv_head][dim] one
// token's K (or V) for all 8 KV heads is 2 KiB contiguous, so each copy is one
// contiguous 2 KiB move: one warp per (token, K|V), 16-byte vector accesses.
//
// The 8-bit cache variant (k_scale set) quantises instead of copying: each (token, KV
// head) row of 128 values gets scale = amax / 448 (fp32, 1 for an all-zero row) and codes
// E4M3(x / scale) (fp32 division, round to nearest even, saturating at 448), one half-
// warp per row; the codes keep the pool layout (128 bytes per row) and the scale goes to
// [block][head][slot].  Page "从零搭建AI工程能力：手写KV Cache与动态批处理实战" §3.2: an 8-bit
// KV cache halves its memory.
//
// The 4-bit variant (k_exp set; the format and its rule: fp4.cuh) gives a lane the 16 values of a group:
// the group's maximum, found among the packed bf16 bits, needs no other lane, the row's three shuffles.  Eight
// ragged chunks, 11093 tokens (58 MB): 15.2 us under the profiler, a half-warp per row and 8 values a lane 4 us more.
//
// The kernel is a chain of dependent loads (which sequence owns the token, its
// length, its block id, then the data), so its time is latency: the owner is first
// guessed in proportion (exact for one token per sequence and for one sequence) and
// only on a miss found by a warp-wide 32-way search.  It lets the next kernel on the
// stream start its own prologue early (programmatic dependent launch); that kernel
// waits for this one to finish before it reads the pools.
// The 4-bit form is launched as such a dependent as well: 128 rows back to back 2.4 us a call, 4.1 without.
#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "tokens.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;  // 4 tokens x {K, V} per CTA

// The larger 16-bit halves, unsigned
__device__ __forceinline__ uint32_t umax_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// kBits: 16 (copied), 8 or 4
template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) kv_append_kernel(AppendArgs a) {
    // The pools are this kernel's only output: a dependent kernel may launch now and
    // run its prologue; it waits for our completion before touching the pools.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kWarps / 2) + (warp >> 1);
    const bool is_v = warp & 1;
    // a programmatic dependent itself: the rows and the pools may belong to the kernel before
    if constexpr (kBits == 4) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.total_tokens) return;
    // The row's 2 KiB does not depend on where it goes: its loads are issued first, so they
    // overlap the chain that finds the destination.  2 KiB = 128 x 16 B: four 16-byte vectors
    // per lane.
    const uint4 *src = reinterpret_cast<const uint4 *>(
        static_cast<const char *>(is_v ? a.v_new : a.k_new) + (size_t)t * kTokenBytes);
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __ldg(src + (kBits == 4 ? 2 * lane + 64 * (k >> 1) + (k & 1) : lane + 32 * k));

    if (blockIdx.x == 0 && threadIdx.x == 0) {
        // cu_q_lens must start at 0 and end at total_tokens
        if (__ldg(a.cu_q_lens) != 0 || __ldg(a.cu_q_lens + a.num_seqs) != a.total_tokens)
            record_error(a.err, kErrDevice | kErrBadCuQ);
    }
    int s = (int)((long long)t * a.num_seqs / a.total_tokens);
    int q0 = __ldg(a.cu_q_lens + s);
    int q1 = __ldg(a.cu_q_lens + s + 1);
    int seq_len = __ldg(a.seq_lens + s);
    if (!(q0 <= t && t < q1)) {
        s = warp_find_sequence(a.cu_q_lens, a.num_seqs, t, lane);
        q0 = __ldg(a.cu_q_lens + s);
        q1 = __ldg(a.cu_q_lens + s + 1);
        seq_len = __ldg(a.seq_lens + s);
    }
    const int q_len = q1 - q0;
    const int i = t - q0;
    if (i < 0 || i >= q_len) {
        if (lane == 0 && !is_v) record_error(a.err, kErrDevice | kErrBadCuQ);
        return;
    }
    if (seq_len < q_len || seq_len > a.max_blocks_per_seq * kBlock) {
        if (lane == 0 && !is_v) record_error(a.err, kErrDevice | kErrBadSeqLen);
        return;
    }
    const int p = seq_len - q_len + i;
    const int blk = __ldg(a.block_table + (size_t)s * a.max_blocks_per_seq + p / kBlock);
    if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0 && !is_v) record_error(a.err, kErrDevice | kErrBadBlock);
        return;
    }
    const int slot = p % kBlock;
    if constexpr (kBits == 16) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(is_v ? a.v_pool : a.k_pool) +
                                               ((size_t)blk * kBlock + slot) * kTokenBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[lane + 32 * k] = v[k];
    } else if constexpr (kBits == 4) {
        // vectors 2k, 2k + 1 of lane l: KV head 4k + l/8, group l%8
        uint8_t *codes = static_cast<uint8_t *>(is_v ? a.v_pool : a.k_pool) +
                         ((size_t)blk * kBlock + slot) * (kHkv * kFp4RowCodes);
        const size_t row0 = (size_t)blk * kHkv * kBlock + slot;   // + head * 256
        uint8_t *scales = is_v ? a.v_scale4 : a.k_scale4;
        uint8_t *exps = is_v ? a.v_exp : a.k_exp;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w[8] = {v[2 * k].x,     v[2 * k].y,     v[2 * k].z,     v[2 * k].w,
                                   v[2 * k + 1].x, v[2 * k + 1].y, v[2 * k + 1].z, v[2 * k + 1].w};
            uint32_t pair = 0;   // magnitudes as bits, of the even and of the odd values
#pragma unroll
            for (int e = 0; e < 8; ++e) pair = umax_u16x2(pair, w[e] & 0x7fff7fffu);
            const uint32_t top = max(pair & 0xffffu, pair >> 16);
            uint32_t amax = top;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) amax = umax_xor(amax, o);
            const uint32_t exp = fp4_row_exp(amax << 16);
            const float unit = fp4_unit_inverse(exp);
            const uint32_t scale = fp4_group_scale(__uint_as_float(top << 16) * unit);
            uint2 c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ffma2(y[2 * e], y[2 * e + 1], bf16_lo(w[4 * h + e]), bf16_hi(w[4 * h + e]), unit, unit, -0.f, -0.f);
                (h ? c.y : c.x) = fp4_codes(y, scale);
            }
            const int head = 4 * k + (lane >> 3), group = lane & 7;
            *reinterpret_cast<uint2 *>(codes + head * kFp4RowCodes + group * 8) = c;
            const size_t row = row0 + (size_t)head * kBlock;
            scales[row * kFp4Groups + group] = (uint8_t)scale;
            if (group == 0) exps[row] = (uint8_t)exp;
        }
    } else {
        // vector k of lane l: KV head 2k + l/16, dims 8 (l%16) .. 8 (l%16) + 7
        uint8_t *codes = static_cast<uint8_t *>(is_v ? a.v_pool : a.k_pool) +
                         ((size_t)blk * kBlock + slot) * (kHkv * kD);
        float *scales = is_v ? a.v_scale : a.k_scale;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = bf16_lo(w[e]);
                x[2 * e + 1] = bf16_hi(w[e]);
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
            uint2 c;
            c.x = f32x2_to_e4m3x2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
                  f32x2_to_e4m3x2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16;
            c.y = f32x2_to_e4m3x2(__fdiv_rn(x[4], scale), __fdiv_rn(x[5], scale)) |
                  f32x2_to_e4m3x2(__fdiv_rn(x[6], scale), __fdiv_rn(x[7], scale)) << 16;
            const int head = 2 * k + (lane >> 4), chunk = lane & 15;
            *reinterpret_cast<uint2 *>(codes + head * kD + chunk * 8) = c;
            if (chunk == 0) scales[((size_t)blk * kHkv + head) * kBlock + slot] = scale;
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream) {
    if (a.total_tokens == 0) return cudaSuccess;
    const int tokens_per_cta = kWarps / 2;
    const int grid = (a.total_tokens + tokens_per_cta - 1) / tokens_per_cta;
    if (a.k_exp) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kWarps * 32);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kv_append_kernel<4>, a);
    }
    if (a.k_scale)
        kv_append_kernel<8><<<grid, kWarps * 32, 0, stream>>>(a);
    else
        kv_append_kernel<16><<<grid, kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pa
