// rope_append.cu -- the new tokens' q, k and v on their way into attention: per-head norm and
// rotary position embedding of q and k, k and v into their cache slots (bf16 or 8 bits), in
// one pass.
//
// Page "扔掉 vLLM！从零构建 Qwen3-8B 推理引擎，C++/CUDA 实现性能追平 98%" §4.3.1 appends a new
// token's K and V to its cache block; the pages name no position encoding or norm.  Those are
// RoFormer's rotation (Su et al. 2021, §3.4), in the pairing of Qwen3: dims d and d + 64 of a
// head turn by an angle a_d, and RMSNorm (Zhang and Sennrich 2019, §3).  For a head x:
//     y[d] = g[d] x[d] / sqrt(mean(x^2) + eps)                       (when gains are given)
//     z[d] = y[d] cos(a_d) - y[d+64] sin(a_d),  z[d+64] = y[d+64] cos(a_d) + y[d] sin(a_d)
//     a_d  = p[axis_d] * theta^(-d/64),  d < 64
// with p the token's position in the cache, or the caller's positions of up to three axes
// (time, height, width), axis_d naming the axis that pair d turns with.  All of it is fp32;
// q and the bf16 cache take one rounding, the 8-bit cache takes its codes and scale straight
// from the fp32 values (one rounding, not bf16 and then 8 bits).
//
// The pass reads each operand once and writes each result once: 8 KiB + 4 KiB a token in, as
// much out, so it is bound by HBM (by latency when there are few tokens).  Design:
//   * a head's row is held by 8 lanes of a warp, lane j the dims 8j .. 8j+7 and 64+8j .. 64+8j+7:
//     both dims of 8 rotation pairs, so only the sum of squares (and the 8-bit row's maximum)
//     crosses lanes, in 3 shuffles for the 4 heads that a warp instruction covers, and every
//     access is 16 bytes a lane, 128 contiguous bytes a row half;
//   * a token's 48 heads are 6 groups of 8 (4 of q, k, v).  The batch's groups, in token order,
//     are cut into one even run per resident warp: a warp looks its token up and computes its
//     angles when the run enters it, so few tokens spread over warps group by group, and many
//     leave no SM idle at the end.  (A warp per token took 26.1 us for 4096 tokens into the 8-bit
//     cache, 4096 tokens on 3648 warps being two rounds; even runs take 19.5 us.)
// Measured in a graph of calls: 1 token 2.0 us (three dependent loads and a launch), 128 tokens
// into the 8-bit cache 2.8 us, 4096 tokens into it 19.3 us (92 MB: 4.8 TB/s), 16381 tokens into the
// bf16 cache 65.1 us (403 MB: 6.2 TB/s, 93 % of the measured copy rate).  What the 8-bit rows wait for
// is a chain (row maximum, scale, reciprocal, quotients, codes) with one group's rows on their way
// meanwhile and 16 warps an SM at 124 registers to cover it; that is where this form stands, not
// shown to be a limit (the one form tried with more warps spilled its prefetched rows).
#include "common.cuh"
#include "launch.h"
#include "tokens.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 2;          // up to 128 registers a thread; 3 (80, spilling) was slower
constexpr int kQGroups = kHq / 8;      // groups of 8 heads: 0-3 q, 4 k, 5 v
constexpr int kGroups = kQGroups + 2;
constexpr float kPosLimit = 16777216.f;   // positions are exact in fp32 below 2^24

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// The fp32 quotient x / s, correctly rounded, from r = 1 / s (correctly rounded): an approximate
// quotient and one correction by its exact remainder (Markstein 1990, IBM J. Res. Dev. 34(1)).
// The signs are arranged so that a zero keeps x's.  For s far from overflow and underflow; where
// the remainder underflows, x / s is far below half the smallest code.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(q, s, -x), -r, q);
}

// E4M3 codes of 8 values: the fp32 quotient by the row's scale, rounded to nearest even (the
// rule of kv_append_fp8).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float r) {
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = quotient(x[e], s, r);
    uint2 c;
    c.x = f32x2_to_e4m3x2(q[0], q[1]) | f32x2_to_e4m3x2(q[2], q[3]) << 16;
    c.y = f32x2_to_e4m3x2(q[4], q[5]) | f32x2_to_e4m3x2(q[6], q[7]) << 16;
    return c;
}

// One K or V row half-pair of this lane into the 8-bit cache.
__device__ __forceinline__ void store_row8(uint8_t *codes, float *scale_slot, int j, float (&lo)[8], float (&hi)[8]) {
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmax3(amax, fabsf(lo[e]), fabsf(hi[e]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // (a normalised k row of at most 2^-141.2 would get the scale 0, and NaN codes: it gets the
    // smallest scale there is, by which its values are at most 224)
    const float scale = amax > 0.f ? fmaxf(__fdiv_rn(amax, 448.f), 0x1p-149f) : 1.f;
    // a row of extreme values is brought to the middle of the exponents first, which changes no
    // quotient; by an infinite scale every finite value gives 0 (s = r = 0 below), inf gives NaN
    float s = scale;
    if (!(scale >= 0x1p-100f && scale <= 0x1p100f)) {
        const float k = scale < 1.f ? 0x1p64f : 0x1p-64f;
        s *= k;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo[e] *= k;
            hi[e] *= k;
        }
    }
    const float r = __frcp_rn(s);
    if (r == 0.f) s = 0.f;
    *reinterpret_cast<uint2 *>(codes + 8 * j) = codes8(lo, s, r);
    *reinterpret_cast<uint2 *>(codes + kD / 2 + 8 * j) = codes8(hi, s, r);
    if (j == 0) *scale_slot = scale;
}

// Where token t of the batch goes.
struct Place {
    bool live;        // a sequence's token (false: behind the last sequence, left alone)
    int pos;          // absolute position, -1 when the sequence's data are inconsistent
    long long row;    // block * 256 + slot in the cache, -1: no K/V row is written
};

__device__ __forceinline__ Place place_of(const RopeAppendArgs &a, int t, int lane, bool report) {
    Place pl = {true, -1, -1};
    // the owner is first guessed in proportion: exact for one token per sequence and for one
    // sequence, so that the loads below go out together
    int s = (int)((long long)t * a.num_seqs / a.total_tokens);
    int q0 = __ldg(a.cu_q_lens + s), q1 = __ldg(a.cu_q_lens + s + 1), seq_len = __ldg(a.seq_lens + s);
    if (!(q0 <= t && t < q1)) {
        const int end = __ldg(a.cu_q_lens + a.num_seqs);
        if (t >= end) {
            pl.live = false;
            return pl;
        }
        s = warp_find_sequence(a.cu_q_lens, a.num_seqs, t, lane);
        q0 = __ldg(a.cu_q_lens + s);
        q1 = __ldg(a.cu_q_lens + s + 1);
        seq_len = __ldg(a.seq_lens + s);
    }
    // (offsets outside the batch first: with q0 near -2^31 the differences below would wrap)
    if (q0 < 0 || q1 > a.total_tokens || t < q0 || t >= q1) {
        if (report) record_error(a.err, kErrDevice | kErrBadCuQ);
        return pl;
    }
    const int q_len = q1 - q0;
    if (seq_len < q_len || seq_len > a.max_blocks_per_seq * kBlock) {
        if (report) record_error(a.err, kErrDevice | kErrBadSeqLen);
        return pl;
    }
    pl.pos = seq_len - q_len + (t - q0);
    const int blk = __ldg(a.block_table + (size_t)s * a.max_blocks_per_seq + pl.pos / kBlock);
    if (blk < 0 || blk >= a.num_blocks) {
        if (report) record_error(a.err, kErrDevice | kErrBadBlock);
        return pl;
    }
    pl.row = (long long)blk * kBlock + pl.pos % kBlock;
    return pl;
}

template <bool kFp8, bool kNorm>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
    // The next kernel on the stream may start its prologue; it waits for this one to complete
    // before it reads q_out or the cache.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int j = lane & 7;        // this lane's 16-byte piece of a row half
    const int hs = lane >> 3;      // which of the 4 heads of a warp access

    // frequencies and axes of the pairs, copied out of the argument space once (read there at
    // an index that differs between lanes, every read would be serialised)
    __shared__ float2 freq[kRopePairs];
    __shared__ uint8_t axis[kRopePairs];
    if (threadIdx.x < kRopePairs) {
        freq[threadIdx.x] = make_float2(a.freq_hi[threadIdx.x], a.freq_lo[threadIdx.x]);
        axis[threadIdx.x] = a.pair_axis[threadIdx.x];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        const int end = __ldg(a.cu_q_lens + a.num_seqs);
        if (__ldg(a.cu_q_lens) != 0 || end < 0 || end > a.total_tokens) record_error(a.err, kErrDevice | kErrBadCuQ);
    }
    __syncthreads();

    const long long groups = (long long)a.total_tokens * kGroups;
    const long long warps = (long long)gridDim.x * kWarps;
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long run_end = groups * (w + 1) / warps;
    long long at = groups * w / warps;
    bool waited = false;
    while (at < run_end) {
        const int tok = (int)(at / kGroups);
        const int g0 = (int)(at - (long long)tok * kGroups);
        const int g1 = (int)min((long long)kGroups, run_end - (long long)tok * kGroups);
        at = (long long)tok * kGroups + g1;
        const Place pl = place_of(a, tok, lane, lane == 0);
        // q, k_new, v_new, positions and gains may come from the kernel just before this one,
        // which may also still read the cache rows and q_out written here
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
        if (!pl.live) continue;

        // heads hs and 4 + hs of group g: the next group's rows are on their way while one is
        // computed, the first one's while the angles are
        uint4 n_lo[2], n_hi[2];
        const auto fetch = [&](int g) {
            const bool is_v = g == kGroups - 1;
            const __nv_bfloat16 *src =
                g < kQGroups ? static_cast<const __nv_bfloat16 *>(a.q) + (size_t)tok * a.q_stride + g * 8 * kD
                             : static_cast<const __nv_bfloat16 *>(is_v ? a.v_new : a.k_new) +
                                   (size_t)tok * (is_v ? a.v_stride : a.k_stride);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint4 *r = reinterpret_cast<const uint4 *>(src + (4 * u + hs) * kD) + j;
                n_lo[u] = r[0];
                n_hi[u] = r[kD / 16];
            }
        };
        fetch(g0);

        // cos and sin of this lane's 8 pairs (8j .. 8j+7).  The positions are checked for every run,
        // also one that begins at v: v's row goes with k's.
        float c[8], s[8];
        bool known = true;            // the rotation's positions are known and in range
        if (a.rope) {
            float p[kMaxRopeAxes];
#pragma unroll
            for (int x = 0; x < kMaxRopeAxes; ++x)
                p[x] = a.positions ? (x < a.axes ? (float)a.positions[(size_t)x * a.total_tokens + tok] : 0.f)
                                   : (float)pl.pos;
            if (a.positions) {
                known = fabsf(p[0]) < kPosLimit && fabsf(p[1]) < kPosLimit && fabsf(p[2]) < kPosLimit;
                if (!known && lane == 0) record_error(a.err, kErrDevice | kErrBadPosition);
            } else {
                known = pl.pos >= 0;
            }
            if (g0 <= kQGroups) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = freq[8 * j + e];
                    const int ax = axis[8 * j + e];
                    angle_cos_sin(ax == 0 ? p[0] : ax == 1 ? p[1] : p[2], f.x, f.y, c[e], s[e]);
                }
            }
        }
        if (!known) {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = s[e] = __int_as_float(0x7fc00000);
        }
        const bool store_kv = pl.row >= 0 && known;

        for (int g = g0; g < g1; ++g) {
            const bool is_q = g < kQGroups, is_v = g == kGroups - 1;
            if (!is_q && !store_kv) break;
            const uint4 w_lo[2] = {n_lo[0], n_lo[1]}, w_hi[2] = {n_hi[0], n_hi[1]};
            if (g + 1 < g1) fetch(g + 1);
            __nv_bfloat16 *dst =
                is_q ? static_cast<__nv_bfloat16 *>(a.q_out) + ((size_t)tok * kHq + g * 8) * kD
                     : static_cast<__nv_bfloat16 *>(is_v ? a.v_pool : a.k_pool) + pl.row * (kHkv * kD);
            uint8_t *codes = nullptr;
            float *scales = nullptr;
            if (kFp8 && !is_q) {
                codes = static_cast<uint8_t *>(is_v ? a.v_pool : a.k_pool) + pl.row * (kHkv * kD);
                scales = (is_v ? a.v_scale : a.k_scale) +
                         ((pl.row / kBlock) * kHkv * kBlock + pl.row % kBlock);   // + head * 256
            }
            uint4 gain_lo = {}, gain_hi = {};
            if (kNorm && !is_v) {
                const uint4 *gw = static_cast<const uint4 *>(is_q ? a.q_norm : a.k_norm) + j;
                gain_lo = gw[0];
                gain_hi = gw[kD / 16];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int h = 4 * u + hs;
                if (!kFp8 && is_v) {      // v: the row as it is
                    uint4 *d = reinterpret_cast<uint4 *>(dst + h * kD) + j;
                    d[0] = w_lo[u];
                    d[kD / 16] = w_hi[u];
                    continue;
                }
                float lo[8], hi[8];
                unpack8(w_lo[u], lo);
                unpack8(w_hi[u], hi);
                if (kFp8 && is_v) {
                    store_row8(codes + h * kD, scales + h * kBlock, j, lo, hi);
                    continue;
                }
                if constexpr (kNorm) {
                    float p = 0.f, q = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        ffma2(p, q, lo[e], lo[e + 1], lo[e], lo[e + 1], p, q);
                        ffma2(p, q, hi[e], hi[e + 1], hi[e], hi[e + 1], p, q);
                    }
                    float ss = p + q;
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = rsqrtf(fmaf(ss, 1.0f / kD, a.norm_eps));
                    float gl[8], gh[8];
                    unpack8(gain_lo, gl);
                    unpack8(gain_hi, gh);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        ffma2(lo[e], lo[e + 1], lo[e], lo[e + 1], inv, inv, 0.f, 0.f);
                        ffma2(hi[e], hi[e + 1], hi[e], hi[e + 1], inv, inv, 0.f, 0.f);
                        ffma2(lo[e], lo[e + 1], lo[e], lo[e + 1], gl[e], gl[e + 1], 0.f, 0.f);
                        ffma2(hi[e], hi[e + 1], hi[e], hi[e + 1], gh[e], gh[e + 1], 0.f, 0.f);
                    }
                }
                float zl[8], zh[8];
                if (a.rope) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        float t0, t1;
                        ffma2(t0, t1, hi[e], hi[e + 1], -s[e], -s[e + 1], 0.f, 0.f);
                        ffma2(zl[e], zl[e + 1], lo[e], lo[e + 1], c[e], c[e + 1], t0, t1);
                        ffma2(t0, t1, lo[e], lo[e + 1], s[e], s[e + 1], 0.f, 0.f);
                        ffma2(zh[e], zh[e + 1], hi[e], hi[e + 1], c[e], c[e + 1], t0, t1);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        zl[e] = lo[e];
                        zh[e] = hi[e];
                    }
                }
                if (kFp8 && !is_q) {
                    store_row8(codes + h * kD, scales + h * kBlock, j, zl, zh);
                } else {
                    uint4 *d = reinterpret_cast<uint4 *>(dst + h * kD) + j;
                    d[0] = pack8(zl);
                    d[kD / 16] = pack8(zh);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs &a, int num_sms, cudaStream_t stream) {
    if (a.total_tokens == 0) return cudaSuccess;
    const long long ctas = (long long)num_sms * kCtasPerSm;
    const long long need = ((long long)a.total_tokens * kGroups + kWarps - 1) / kWarps;   // a warp per group
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(need < ctas ? need : ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.k_scale)
        return a.q_norm ? cudaLaunchKernelEx(&cfg, rope_append_kernel<true, true>, a)
                        : cudaLaunchKernelEx(&cfg, rope_append_kernel<true, false>, a);
    return a.q_norm ? cudaLaunchKernelEx(&cfg, rope_append_kernel<false, true>, a)
                    : cudaLaunchKernelEx(&cfg, rope_append_kernel<false, false>, a);
}

}  // namespace pa
