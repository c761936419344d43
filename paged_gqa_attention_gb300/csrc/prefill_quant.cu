// prefill_quant.cu -- causal (chunked) prefill attention over the 8-bit or the 4-bit KV cache, with an
// optional sliding window, on the 5th-generation tensor cores.
//
// Page "从零搭建AI工程能力：手写KV Cache与动态批处理实战" §3.2 stores the KV cache in 8 bits, §3.3 cuts
// long prompts into chunks that attend to the cached context before them; here both at once.  The
// attention, its work units, key lists, tiles and tensor memory are those of the windowed form of
// prefill.cu (a window as long as the context is plain causal attention); what differs is how a key
// tile comes into being.
//
// Codes are not operands: their row scales run along the keys, and a 4-bit row has a scale for every 16
// dimensions besides.  So the products run in f16, and converter warps turn code tiles into f16 tiles in
// shared memory while the tensor cores work on the tiles before:
//   K' = code * s / 2^E,      E the exponent of the tile's largest scale: a magnitude of at most 448 (2688
//                             in 4 bits); the scores are multiplied by 2^E together with the softmax scale
//   V' = code * s / sigma,    sigma the power of two above the first tile's largest scale, taken anew only
//                             when a tile's V' could leave f16; O is then rescaled, as it is for the
//                             running maximum, and the epilogue multiplies by sigma
// with one rounding to f16 (8 bits: the scale is split into a sum of two f16, so that code * scale is rounded
// once, by 2^-11 of the value at most; 4 bits: exact).  Quotients under 2^-14 lose bits one by one.
// Q is converted to f16 in place (|q| < 65504, as for the decode over these caches), P is f16.
//
// What bounds it is not the products (4 x 128 x 128 x 256 operations a tile, 2048 clk at the tensor cores' rate)
// but what else a tile asks for: the softmax of 256 rows and the conversion of 2 x 16384 values share the
// issue slots, and a converter's visit to a tile (waits, scales, fence, arrival) costs as much as its
// arithmetic.  Hence pairs of CTAs (clusters of two, a sequence's adjacent 64 positions each) walk one list of keys:
// each converts 64 rows of every tile and copies them to the other's shared memory (bulk copies that
// complete on the barrier the other's products wait for), so that a row is converted once for 128 positions.
// Measured, 8192 new tokens after 8192 in 8 bits: 2012 us with the conversion unrolled for K and V apart, 1570
// in one rolled loop, 1555 with six converters, 1455 in pairs whose converters made the copies (400 clk a
// visit), 1239 with the copies in the producer, 1224 with the loads of V and the copies in a warp of their own and the
// tiles' exponents in the producer (1.35 PFLOP/s; the vote on small scales has since added 1 %; 4 chunks of up to 1024
// in 4 bits with a window of 2048, which the producer's 2400 clk of issuing loads a tile had held at 132 us: 120).  One
// CTA alone walking its list, 1555
// and 129, is left where a sequence has 64 positions at most (there is nobody to share with) and where few
// units share the GPU, whose keys are split instead.  Products over the pair (tcgen05 with two CTAs' operands) halve
// the same conversion without copies, but every step then waits for the peer: 1382.
//
// CTA = 16 warps, persistent, one per SM:
//   warps 0-3, 4-7    softmax + epilogue of query tiles A and B (thread = row = TMEM lane)
//   warps 8-11, 15    converters; without a pair 14 too
//   warp 12           TMA producer: Q, and the ring of code tiles in the order K(0) V(0) K(1) V(1) ...; in a pair of
//                     K alone, and of what the tiles are scaled by
//   warp 13           TMEM allocator and tcgen05.mma issuer
//   warp 14           in a pair: V's code tiles, and the copies of converted halves to the peer
// Every wait is bounded; on expiry the CTA records PA_ERR_TIMEOUT, unwinds, waits (bounded) for its own
// copies and MMAs, frees tensor memory and exits.
#include <atomic>
#include <cstddef>

#include <cuda_fp16.h>

#include "cluster.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "prefill_common.cuh"
#include "window.cuh"

namespace pa {
namespace {

template <bool kPair>
constexpr int kConvertWarps = kPair ? 5 : 6;  // 8-11, 15 and without a pair 14
constexpr int kProducerWarp = 12;
constexpr int kMmaWarp = 13;
constexpr int kPairWarp = 14;                 // a pair's V loads, and copies to the peer
constexpr int kThreads = 16 * 32;
// registers a thread, warpgroup by warpgroup: together the 512 x 128 that the block is launched with (8192 tokens
// after 8192 with 168 and 88 1300 us, 160 and 96 1224, 152 and 104 1314)
constexpr int kSoftmaxRegs = 160, kOtherRegs = 96;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs == 4 * 128, "register split");
constexpr uint32_t kTileBytes = 2 * kHalf;    // a 128 x 128 f16 tile
constexpr int kStages = 2;                    // f16 tiles of K and of V
constexpr int kPairPos = 2 * kUnitPos;        // query positions of a pair's unit
constexpr int kParams = 8;                    // see TileParams
constexpr int kReady = 4;                     // see scaled in QuantSmem

// f16 operands and fp32 accumulation: formats 0 where idesc_bf16 has 1
constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
    return idesc_bf16(m, n, b_mn_major) & ~((1u << 7) | (1u << 10));
}
constexpr uint32_t kIdescQK = idesc_f16(kRows, kKT, false);
constexpr uint32_t kIdescPV = idesc_f16(kRows, kD, true);

// Code tiles on their way in, with their scales: a ring of slots, K and V in turn.  A K tile brings along
// the V scales of the same rows (in 4 bits their exponents), from which sigma is chosen before the softmax
// needs it.  A slot of a pair holds the codes of the 64 rows that this CTA converts, and the scales of all.
template <int kBits, bool kPair>
struct CodeRing;
template <bool kPair>
struct CodeRing<8, kPair> {
    static constexpr int kSlots = kPair ? 3 : 2, kRow = kD, kRows = kPair ? 64 : kKT;
    uint8_t codes[kSlots][kRows * kRow];
    float scale[kSlots][kKT];
    float v_scale[kPair ? kSlots : 1][kKT];   // (with two slots those of K are all the first one's)
    __device__ __forceinline__ float *v_scales(int st) { return v_scale[kPair ? st : 0]; }
};
template <bool kPair>
struct CodeRing<4, kPair> {
    static constexpr int kSlots = kPair ? 6 : 3, kRow = kFp4RowCodes, kRows = kPair ? 64 : kKT;
    uint8_t codes[kSlots][kRows * kRow];
    uint8_t scale[kSlots][kKT * kFp4Groups];
    uint8_t exp[kSlots][kKT];
    uint8_t v_exp[kSlots][kKT];
};

// What key tile `it` is scaled by, in entry it % 8.  An entry is written when the tile's K is in the ring, at the earliest
// (six slots) when K(it - 3) is converted, which needs the slot of K(it - 5), so S_B(it - 5); that was issued after
// O_B += P_B(it - 6) V, so both query tiles' softmax have read entry it - 6 by then: 7 entries are enough.
struct TileParams {
    float k_unit;             // 2^E
    float sigma;
    float grow;               // the factor that brings O to units of sigma (1, or sigma has just grown)
    int unit, sigma_exp;      // E, and sigma's exponent
};

template <int kBits, bool kPair>
struct QuantSmem {
    uint8_t q[2][2][kHalf];          // [tile A|B][dims 0-63 | 64-127]
    uint8_t k[kStages][2][kHalf];
    uint8_t v[kStages][2][kHalf];
    union {
        CodeRing<kBits, kPair> ring;
        float ml[2 * kRows][2];      // kSplit, at the end: running maximum and sum of every row
    };
    uint64_t q_full, q_ready, q_empty;
    uint64_t c_full[CodeRing<kBits, kPair>::kSlots], c_empty[CodeRing<kBits, kPair>::kSlots];
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t v_full[kStages], v_empty[kStages];
    uint64_t half_done[2][kStages];                // a pair: this CTA's half of K, V is converted
    // a pair: tile it's entry is written, on it % 4 (that of it + 4 waits, at the earliest, for the conversion of
    // K(it + 1), so nobody waits for it any more)
    uint64_t scaled[kReady];
    uint64_t s_full[2], p_half[2][2], o_done[2];   // per query tile (P in two key halves)
    uint64_t mma_idle;
    TileParams params[kParams];
    uint32_t tmem_base;
    int abort;
};
using SplitSmem = QuantSmem<8, false>;
static_assert(offsetof(SplitSmem, k) == sizeof(SplitSmem::q) &&
                  sizeof(SplitSmem::q) + sizeof(SplitSmem::k) == 2 * kRows * kD * sizeof(float),
              "split merge area");

template <int kBits, bool kPair>
constexpr size_t kSmemBytes = sizeof(QuantSmem<kBits, kPair>) + 1024;
static_assert(kSmemBytes<8, false> <= 232448 && kSmemBytes<4, false> <= 232448 && kSmemBytes<8, true> <= 232448 &&
                  kSmemBytes<4, true> <= 232448,
              "shared memory");

__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// Two fp32 sums in one packed instruction: (d0, d1) += (a0, a1)
__device__ __forceinline__ void fadd2(float &d0, float &d1, float a0, float a1) {
    asm("{\n .reg .b64 ra, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rd, {%0, %1};\n add.rn.f32x2 rd, rd, ra;\n"
        " mov.b64 {%0, %1}, rd;\n}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// ---------------------------------------------------------------- a pair of CTAs
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Arrive on the barrier at this offset in both CTAs once every tcgen05 operation this thread issued has completed.
__device__ __forceinline__ void umma_commit_both(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"((uint16_t)3)
                 : "memory");
}

// Shared memory of this CTA -> of the peer, completing there.
__device__ __forceinline__ void copy_to_peer(uint32_t cluster_dst, uint32_t src, uint32_t bytes, uint32_t cluster_bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(cluster_dst), "r"(src), "r"(bytes), "r"(cluster_bar)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 ld_shared_8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The work unit dealt as the r-th of this CTA.  A pair's unit is 128 positions: one list of keys for both
// CTAs, the first 64 positions rank 0's, the others (none: computed all the same, and not stored) rank 1's.
template <bool kPlanned, bool kSplit, bool kPair>
__device__ __forceinline__ Unit unit_for(const PrefillArgs &a, int idx, int qblocks, int rank) {
    if constexpr (kPair) {
        Unit t = unit_at<false, true, kPairPos>(a, kPlanned ? __ldg(a.order + idx) : idx, qblocks);
        t.tok0 += rank * kUnitPos;
        t.pos0 += rank * kUnitPos;
        t.positions = min(kUnitPos, t.positions - rank * kUnitPos);
        return t;
    }
    if constexpr (kSplit) {
        // this CTA's run of the unit's key tiles (none: it only takes part in the merge)
        Unit t = unit_at<false, true>(a, idx, qblocks);
        if (!t.run) return t;
        const int len = (t.n_kt + a.unit_ctas - 1) / a.unit_ctas;
        t.kt0 = (int)(blockIdx.x % a.unit_ctas) * len;
        t.n_kt = min(len, t.n_kt - t.kt0);
        if (t.n_kt <= 0) t.run = false;
        return t;
    }
    return unit_at<false, true>(a, kPlanned ? __ldg(a.order + idx) : idx, qblocks);
}

// Fetch rows c0 .. c0 + 127 of the unit's key list (load_list_tile's rule in prefill.cu): codes in
// boxes of 64 and 16 rows, their scales beside them a run at a time.  Block ids are reported by K.  A CTA of
// a pair converts rows first .. first + 63 and fetches the codes of no others.
template <int kBits, bool kPair>
__device__ __forceinline__ void load_codes(const PrefillArgs &a, const Unit &t, const int32_t *bt, int c0, bool is_k,
                                           CodeRing<kBits, kPair> &ring, int st, uint32_t bar, const CUtensorMap *map64,
                                           const CUtensorMap *map16, int first) {
    constexpr int kRow = CodeRing<kBits, kPair>::kRow;
    constexpr int kScales = kBits == 8 ? 4 : kFp4Groups + 1;
    const int rows = min(kKT, ((t.win.rows + 15) & ~15) - c0);
    const int coded = kPair ? max(0, min(64, rows - first)) : rows;
    mbar_arrive_expect_tx(bar, (uint32_t)(coded * kRow + rows * (kScales + (is_k ? (kBits == 8 ? 4 : 1) : 0))));
    for (int r = 0; r < rows;) {
        const int p = t.win.position(c0 + r);
        int run = min(rows - r, kBlock - p % kBlock);
        if (c0 + r < t.win.s16) run = min(run, t.win.s16 - c0 - r);
        int blk = __ldg(bt + p / kBlock);
        if (blk < 0 || blk >= a.num_blocks) {
            if (is_k) record_error(a.err, kErrDevice | kErrBadBlock);
            blk = 0;   // stay inside the pool; the result is flagged as invalid
        }
        int off = p % kBlock;
        const size_t row = ((size_t)blk * kHkv + t.g) * kBlock + off;   // (off and run are multiples of 16)
        if constexpr (kBits == 8) {
            const void *scale = is_k ? a.k_scale : a.v_scale;
            bulk_load(smem_u32(ring.scale[st] + r), static_cast<const float *>(scale) + row, run * 4, bar);
            if (is_k) bulk_load(smem_u32(ring.v_scales(st) + r), static_cast<const float *>(a.v_scale) + row, run * 4, bar);
        } else {
            bulk_load(smem_u32(ring.scale[st] + r * kFp4Groups),
                      static_cast<const uint8_t *>(is_k ? a.k_scale : a.v_scale) + row * kFp4Groups, run * kFp4Groups, bar);
            bulk_load(smem_u32(ring.exp[st] + r), (is_k ? a.k_exp : a.v_exp) + row, run, bar);
            if (is_k) bulk_load(smem_u32(ring.v_exp[st] + r), a.v_exp + row, run, bar);
        }
        while (run > 0) {
            const bool big = run >= 64 && (!kPair || (r & 63) == 0);
            const int n = big ? 64 : 16;
            if (!kPair || (r & 64) == first)
                tma_load_4d(smem_u32(ring.codes[st] + (r - first) * kRow), big ? map64 : map16, bar, 0, t.g, off, blk);
            r += n;
            off += n;
            run -= n;
        }
    }
}

// ---------------------------------------------------------------- conversion (one warp's share)

// What a lane converts at a time: 2 x 16 codes of one row, dims 16c .. 16c + 15 and 64 + 16c .., with what scales
// them; then their f16 values code * scale * unit, `unit` a power of two.
template <int kBits>
struct Piece;
template <>
struct Piece<8> {
    uint4 c[2];
    float s;

    // lo, hi: addresses of the codes in the ring; row: of the tile
    template <bool kPair>
    __device__ __forceinline__ void read(const CodeRing<8, kPair> &ring, int st, uint32_t lo, uint32_t hi, int row, int) {
        c[0] = ld_shared_16(lo);
        c[1] = ld_shared_16(hi);
        s = ring.scale[st][row];
    }
    __device__ __forceinline__ void convert(float unit, uint32_t (&h)[2][8]) const {
        // the scale as hi + lo, so that code * scale is rounded once (code * lo is far below the last place).  A scale under
        // 2^-8, whose hi or lo would leave f16's normal range, is taken 2^14 times as large and the products brought
        // back: they round where they are under 2^-14 themselves, not 2^9 before.  The vote takes 15 us of 1290 (8192 tokens
        // after 8192); a flag a tile, from the least scale, 55.
        const float at = s * unit;
        const bool small = fabsf(at) < 0x1p-8f;
        const float x = small ? at * 0x1p14f : at;
        const uint32_t hi = pack_f16x2(x, x);
        const float rest = x - __half2float(__ushort_as_half((unsigned short)hi));
        const uint32_t lo = pack_f16x2(rest, rest);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            e4m3x4_to_f16x2x2(c[u].x, h[u][0], h[u][1]);
            e4m3x4_to_f16x2x2(c[u].y, h[u][2], h[u][3]);
            e4m3x4_to_f16x2x2(c[u].z, h[u][4], h[u][5]);
            e4m3x4_to_f16x2x2(c[u].w, h[u][6], h[u][7]);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[u][e] = fma_f16x2(h[u][e], hi, mul_f16x2(h[u][e], lo));
        }
        if (__any_sync(0xffffffffu, small)) {    // (rare: a row 2^-8 of the largest)
            const uint32_t back = small ? 0x04000400u : 0x3c003c00u;   // 2^-14, or 1
#pragma unroll
            for (int e = 0; e < 16; ++e) h[e >> 3][e & 7] = mul_f16x2(h[e >> 3][e & 7], back);
        }
    }
};
template <>
struct Piece<4> {
    uint2 c[2];
    uint32_t s[2], exp;

    template <bool kPair>
    __device__ __forceinline__ void read(const CodeRing<4, kPair> &ring, int st, uint32_t lo, uint32_t hi, int row, int chunk) {
        c[0] = ld_shared_8(lo);
        c[1] = ld_shared_8(hi);
        const uint8_t *scale = ring.scale[st] + row * kFp4Groups + chunk;
        s[0] = scale[0];
        s[1] = scale[4];
        exp = ring.exp[st][row];
    }
    __device__ __forceinline__ void convert(float unit, uint32_t (&h)[2][8]) const {
        const float power = fp4_unit(exp) * unit;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float x = e4m3_value(s[u]) * power;
            const uint32_t x2 = pack_f16x2(x, x);
            uint32_t lo[4], hi[4];
            e2m1x8_to_f16x2x4(c[u].x, lo);
            e2m1x8_to_f16x2x4(c[u].y, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[u][e] = mul_f16x2(lo[e], x2);
                h[u][4 + e] = mul_f16x2(hi[e], x2);
            }
        }
    }
};

// Exponent n of the power of two that the live rows' largest scale is below (8 bits; scales that are zero,
// negative, infinite or NaN leave it out) or at (4 bits, without NaN); kNone: there is none.  `x`: what rows 4 lane ..
// 4 lane + 3 have.
constexpr int kNone = -1000;
__device__ __forceinline__ bool is_dead(const DeadRows &dead, int r) { return (r >= dead.lo && r < dead.hi) || r >= dead.tail; }
__device__ __forceinline__ int top_of(int4 x, bool any_dead, const DeadRows &dead, int lane) {   // 8 bits: floats
    if (any_dead) {
        if (is_dead(dead, 4 * lane)) x.x = 0;
        if (is_dead(dead, 4 * lane + 1)) x.y = 0;
        if (is_dead(dead, 4 * lane + 2)) x.z = 0;
        if (is_dead(dead, 4 * lane + 3)) x.w = 0;
    }
    // as integers positive floats are in order, with infinities and NaN on top
    const auto finite = [](int v) { return v < 0x7f800000 ? v : 0; };
    return max(max(finite(x.x), finite(x.y)), max(finite(x.z), finite(x.w)));
}
__device__ __forceinline__ int top_of(uint32_t x, bool any_dead, const DeadRows &dead, int lane) {   // 4 bits: bytes
    if (any_dead) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (is_dead(dead, 4 * lane + i)) x &= ~(0xffu << (8 * i));
    }
    x &= ~__vcmpeq4(x, 0xffffffffu);         // without NaN
    const uint32_t y = __vmaxu4(x, x >> 16);
    return (int)max(y & 0xffu, y >> 8 & 0xffu);
}
template <int kBits>
__device__ __forceinline__ int exponent_of(int top) {   // of the largest of all lanes
    const int n = kBits == 8 ? (top >> 23) + 1 - 127 : top - 127;
    return top > 0 ? min(max(n, -126), 126) : kNone;
}

// 2^n as a float for n in -126 .. 127 (clamped).
__device__ __forceinline__ float exp2_int(int n) { return __uint_as_float((uint32_t)(min(max(n, -126), 127) + 127) << 23); }

// What the tile whose K is in slot st is scaled by (a warp's work); sigma: its exponent after the tile before, kNone at first.
template <int kBits, bool kPair>
__device__ __forceinline__ TileParams scale_tile(CodeRing<kBits, kPair> &ring, int st, const DeadRows &dead, int &sigma,
                                                 int lane) {
    // V' stays below 65504: codes reach 448 (2688 with their group's scale), so the tile's largest scale
    // may be this many powers of two above sigma
    constexpr int kHeadroom = kBits == 8 ? 7 : 4;
    const bool any_dead = dead.any();
    int top, v_top;                              // (read and reduced side by side)
    if constexpr (kBits == 8) {
        const int4 s = *reinterpret_cast<const int4 *>(ring.scale[st] + 4 * lane);
        const int4 v = *reinterpret_cast<const int4 *>(ring.v_scales(st) + 4 * lane);
        top = top_of(s, any_dead, dead, lane);
        v_top = top_of(v, any_dead, dead, lane);
    } else {
        const uint32_t s = *reinterpret_cast<const uint32_t *>(ring.exp[st] + 4 * lane);
        const uint32_t v = *reinterpret_cast<const uint32_t *>(ring.v_exp[st] + 4 * lane);
        top = top_of(s, any_dead, dead, lane);
        v_top = top_of(v, any_dead, dead, lane);
    }
    top = exponent_of<kBits>(__reduce_max_sync(0xffffffffu, top));
    v_top = exponent_of<kBits>(__reduce_max_sync(0xffffffffu, v_top));
    TileParams p;
    p.grow = 1.f;
    if (v_top != kNone && (sigma == kNone || v_top > sigma + kHeadroom)) {
        if (sigma != kNone) p.grow = exp2_int(sigma - v_top);
        sigma = v_top;
    }
    p.unit = top == kNone ? 0 : top;
    p.sigma_exp = sigma == kNone ? 0 : sigma;
    p.k_unit = exp2_int(p.unit);
    p.sigma = exp2_int(p.sigma_exp);
    return p;
}

// This warp's share of rows row0 .. end - 1 of a code tile into an f16 tile: rounds of 8 rows, `first` and every 6th (a
// pair: 5th) from there on, the next round's read ahead.  Dead rows are zeros: their codes and scales may be anything,
// and 0 * NaN is not 0.
// Lanes 8q .. 8q + 3 have row q of the 8, lanes 8q + 4 .. 8q + 7 row q ^ 5, so that with the swizzles below neither
// a load (whose rows must differ in bit 2) nor a store (in bit 0) meets a bank twice, and no lane has to exchange its
// pieces first.
// The loop stays rolled, and K and V share it: the roles of this kernel run different code at the same time, and
// unrolled, once for K and once for V, warps waited for instructions more than for anything else (2.3 of 10
// warp-cycles an instruction).  A round takes a warp some 265 clk on its own: 48 half-rate instructions and their
// latencies.
template <int kBits, bool kPair>
__device__ __forceinline__ void convert_tile(const CodeRing<kBits, kPair> &ring, int st, uint32_t dst, float unit,
                                             bool any_dead, const DeadRows &dead, int row0, int end, int first, int lane) {
    constexpr int kRow = CodeRing<kBits, kPair>::kRow, kStep = 8 * kConvertWarps<kPair>;
    const int c = lane & 3;
    int row = row0 + 8 * first + ((lane >> 3) ^ ((lane & 4) ? 5 : 0));
    // 8 bits: 128-byte rows, 128-byte swizzle (sw128); 4 bits: 64-byte rows, 64-byte swizzle, in which 16-byte
    // piece p of row r is at p ^ (r / 2 % 4).  Either repeats every 8 rows; 64 dims on flip one bit of the address.
    const int from = kPair ? row - row0 : row;   // row of the slot
    uint32_t src = smem_u32(ring.codes[st]) +
                   (kBits == 8 ? sw128(from, c) : from * kRow + (((c >> 1) ^ ((from >> 1) & 3)) << 4) + ((c & 1) << 3));
    constexpr uint32_t kFlip = kBits == 8 ? 64 : 32;
    uint32_t at = dst + sw128(row, 2 * c);
    Piece<kBits> x;
    x.read(ring, st, src, src ^ kFlip, row, c);
#pragma unroll 1
    while (true) {
        const bool more = row + kStep < end;
        Piece<kBits> next = x;
        src += kStep * kRow;
        if (more) next.read(ring, st, src, src ^ kFlip, row + kStep, c);
        uint32_t h[2][8];
        x.convert(unit, h);
        if (any_dead && is_dead(dead, row)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) h[e >> 3][e & 7] = 0u;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            st_shared_16(at + u * kHalf, h[u][0], h[u][1], h[u][2], h[u][3]);
            st_shared_16((at ^ 16u) + u * kHalf, h[u][4], h[u][5], h[u][6], h[u][7]);
        }
        if (!more) break;      // (alike in the whole warp: rounds do not cross the tile's end)
        x = next;
        at += kStep * 128;
        row += kStep;
    }
}

// Q in place, bf16 -> f16: this warp's share.
template <int kWarps>
__device__ __forceinline__ void convert_q(uint8_t *q, int w, int lane) {
    uint4 *p = reinterpret_cast<uint4 *>(q) + lane;
#pragma unroll 2
    for (int i = w; i < 4 * kHalf / 16 / 32; i += kWarps) {
        uint4 x = p[i * 32];
        x.x = bf16x2_to_f16x2(x.x);
        x.y = bf16x2_to_f16x2(x.y);
        x.z = bf16x2_to_f16x2(x.z);
        x.w = bf16x2_to_f16x2(x.w);
        p[i * 32] = x;
    }
}

template <int kBits, bool kPlanned, bool kSplit, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
prefill_quant_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap k16_map,
                     const __grid_constant__ CUtensorMap v16_map, const PrefillArgs a) {
    using Smem = QuantSmem<kBits, kPair>;
    constexpr int kRing = CodeRing<kBits, kPair>::kSlots;
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int *abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    static_assert(!(kPair && kSplit), "forms");
    constexpr int kPos = kPair ? kPairPos : kUnitPos;
    constexpr int kCtas = kPair ? 2 : 1;
    constexpr int kConv = kConvertWarps<kPair>;
    const int qblocks = (a.max_q_len + kPos - 1) / kPos;
    const int total = a.num_seqs * kHkv * qblocks;
    const int rank = kPair ? (int)cluster_rank() : 0;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sm.q_full), 1);
        mbar_init(smem_u32(&sm.q_ready), kConv);
        mbar_init(smem_u32(&sm.q_empty), 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&sm.c_full[i]), 1);
            mbar_init(smem_u32(&sm.c_empty[i]), kConv);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.k_full[i]), kPair ? 1 : kConv);   // pair: its pair warp, and the peer's copies
            mbar_init(smem_u32(&sm.k_empty[i]), kCtas);   // both CTAs' products are done with it
            mbar_init(smem_u32(&sm.v_full[i]), kPair ? 1 : kConv);
            mbar_init(smem_u32(&sm.v_empty[i]), kCtas);
            mbar_init(smem_u32(&sm.half_done[0][i]), kConv);
            mbar_init(smem_u32(&sm.half_done[1][i]), kConv);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&sm.s_full[x]), 1);
            mbar_init(smem_u32(&sm.p_half[x][0]), 4);   // the 4 warps of the tile's softmax
            mbar_init(smem_u32(&sm.p_half[x][1]), 4);
            mbar_init(smem_u32(&sm.o_done[x]), 1);
        }
        for (int i = 0; i < kReady; ++i) mbar_init(smem_u32(&sm.scaled[i]), 1);
        mbar_init(smem_u32(&sm.mma_idle), 1);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    // (a pair: both CTAs' barriers exist before either reaches for the other's)
    if constexpr (kPair) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_or_abort(smem_u32(bar), parity, abort_flag, a.err));
    };

    if (warp >= kSoftmaxWarps) {
        regs_dec<kOtherRegs>();
        if (warp == kProducerWarp) {
            // ---------------------------------------------------------------- TMA producer
            const bool leader = elect_one();
            if (leader) {
                tma_prefetch_map(&q_map);
                tma_prefetch_map(&k_map);
                tma_prefetch_map(&v_map);
                tma_prefetch_map(&k16_map);
                tma_prefetch_map(&v16_map);
            }
            // the cache and q may be written by the kernel just before this one on the stream
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int units = 0, it = 0;               // units, code tiles (K and V) issued
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit, kCtas>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit, kPair>(a, idx, qblocks, rank);
                if (leader && rank == 0 && t.error) record_error(a.err, kErrDevice | kErrQLen);
                if (!t.run) continue;
                const int32_t *bt = a.block_table + (size_t)t.s * a.max_blocks_per_seq;
                // Q behind the first K tile, which does not wait for the unit before
                const auto load_q = [&]() -> bool {
                    if (units >= 1 && !wait_all(&sm.q_empty, (units - 1) & 1)) return false;
                    if (leader) {
                        const uint32_t qbar = smem_u32(&sm.q_full);
                        mbar_arrive_expect_tx(qbar, 2 * kTileBytes);
                        for (int x = 0; x < 2; ++x) {
                            tma_load_3d(smem_u32(sm.q[x][0]), &q_map, qbar, 0, t.g * kGroup, t.tok0 + x * kTilePos);
                            tma_load_3d(smem_u32(sm.q[x][1]), &q_map, qbar, 64, t.g * kGroup, t.tok0 + x * kTilePos);
                        }
                    }
                    __syncwarp();
                    ++units;
                    return true;
                };
                // code tile i of the unit, `it` of the CTA
                const auto load_tile = [&](int i) -> bool {
                    const int st = it % kRing;
                    if (it >= kRing && !wait_all(&sm.c_empty[st], ((it / kRing) - 1) & 1)) return false;
                    const bool is_k = !(i & 1);
                    if (leader)
                        load_codes<kBits, kPair>(a, t, bt, (t.kt0 + (i >> 1)) * kKT, is_k, sm.ring, st,
                                                 smem_u32(&sm.c_full[st]), is_k ? &k_map : &v_map,
                                                 is_k ? &k16_map : &v16_map, 64 * rank);
                    __syncwarp();
                    return true;
                };
                if constexpr (kPair) {
                    // K alone, and what its tiles are scaled by: the tile's entry, before the next one's load
                    int sigma = kNone;
                    if (!(ok = load_tile(0))) break;
                    for (int j = 0; j < t.n_kt; ++j) {
                        const int kt = it >> 1, st = it % kRing;
                        if (!(ok = wait_all(&sm.c_full[st], (it / kRing) & 1))) { it += 2; break; }
                        const TileParams p = scale_tile(sm.ring, st, DeadRows(t.win, j * kKT), sigma, lane);
                        if (leader) {
                            sm.params[kt % kParams] = p;
                            mbar_arrive(smem_u32(&sm.scaled[kt % kReady]));
                        }
                        __syncwarp();
                        it += 2;
                        if (j == 0 && !(ok = load_q())) break;
                        if (j + 1 < t.n_kt && !(ok = load_tile(2 * (j + 1)))) break;
                    }
                } else {
                    for (int i = 0; i < 2 * t.n_kt; ++i) {
                        if (!(ok = load_tile(i))) break;
                        ++it;
                        if (i == 0 && !(ok = load_q())) break;
                    }
                }
            }
            // Drain: no TMA copy may still be landing when the CTA exits.  In the normal path every load has
            // been consumed and these waits return at once.
            if (units > 0) mbar_wait(smem_u32(&sm.q_full), (units - 1) & 1);
            for (int i = max(0, it - kRing); i < it; ++i)
                if (!kPair || !(i & 1)) mbar_wait(smem_u32(&sm.c_full[i % kRing]), (i / kRing) & 1);
        } else if (kPair && warp == kPairWarp) {
            // ---------------------------------------------------------------- V loads, and a pair's exchange
            const bool leader = elect_one();
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int kt = 0;                          // key tiles
            bool ok = true;
            // This CTA's half of key tile k to the peer, from where the other comes
            const auto send = [&](int k) -> bool {
                const int ks = k % kStages;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (!wait_all(&sm.half_done[v][ks], (k / kStages) & 1)) return false;
                    if (leader) {
                        const uint32_t half = smem_u32(v ? sm.v[ks] : sm.k[ks]) + (uint32_t)(64 * rank * 128);
                        const uint32_t full = smem_u32(v ? &sm.v_full[ks] : &sm.k_full[ks]);
                        const uint32_t dst = peer_addr(half, rank ^ 1), bar = peer_addr(full, rank ^ 1);
                        copy_to_peer(dst, half, kHalf / 2, bar);
                        copy_to_peer(dst + kHalf, half + kHalf, kHalf / 2, bar);
                        mbar_arrive_expect_tx(full, kHalf);
                    }
                    __syncwarp();
                }
                return true;
            };
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit, kCtas>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit, kPair>(a, idx, qblocks, rank);
                if (!t.run) continue;
                const int32_t *bt = a.block_table + (size_t)t.s * a.max_blocks_per_seq;
                for (int j = 0; j < t.n_kt; ++j, ++kt) {
                    const int it = 2 * kt + 1, st = it % kRing;
                    if (it >= kRing && !(ok = wait_all(&sm.c_empty[st], ((it / kRing) - 1) & 1))) break;
                    if (leader)
                        load_codes<kBits, kPair>(a, t, bt, j * kKT, false, sm.ring, st, smem_u32(&sm.c_full[st]), &v_map,
                                                 &v16_map, 64 * rank);
                    __syncwarp();
                    if (kt > 0 && !(ok = send(kt - 1))) {
                        ++kt;
                        break;
                    }
                }
            }
            if (ok && kt > 0) ok = send(kt - 1);
            // Copies to the peer have landed when the peer's products are done, which the end waits for.  Where something
            // gave up, those of the last moment are given a hundred times what they take.
            if (!ok) __nanosleep(100000);
            for (int i = max(0, 2 * kt - kRing); i < 2 * kt; ++i)
                if (i & 1) mbar_wait(smem_u32(&sm.c_full[i % kRing]), (i / kRing) & 1);
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- MMA issuer (as in prefill.cu)
            const bool leader = elect_one();
            if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
            const auto commit_tile = [&](uint64_t *bar) {   // a tile of K or V has been read
                if constexpr (kPair) umma_commit_both(smem_u32(bar));
                else umma_commit(smem_u32(bar));
            };
            const uint64_t qd0 = sdesc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
            const uint64_t kd0 = sdesc_sw128(smem_u32(sm.k[0][0]), 16, 1024);
            const uint64_t vd0 = sdesc_sw128(smem_u32(sm.v[0][0]), (uint32_t)kHalf, 1024);
            int units = 0, it = 0;
            int pend_it = -1, pend_j = 0;   // O_B += P_B V still to issue for key tile pend_it
            bool ok = true;
            auto issue_s = [&](int x, int ks) {
                const uint64_t qa = qd0 + (uint64_t)(x * 2048);
                const uint64_t kb = kd0 + (uint64_t)(ks * 2048);
                const uint32_t sd = tmem + col_s(x);
                if (leader) {
                    umma_ss_c<false>(sd, qa, kb, kIdescQK);
#pragma unroll
                    for (int kk = 1; kk < kD / 16; ++kk) {
                        const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
                        umma_ss_c<true>(sd, qa + off, kb + off, kIdescQK);
                    }
                    umma_commit(smem_u32(&sm.s_full[x]));
                }
                __syncwarp();
            };
            auto issue_pv = [&](int x, int pit, int pj) -> bool {
                const int vs = pit % kStages;
                if (x == 0 && !wait_all(&sm.v_full[vs], (pit / kStages) & 1)) return false;
                const uint64_t vb = vd0 + (uint64_t)(vs * 2048);
                const uint32_t pa = tmem + col_s(x);
                if (!wait_all(&sm.p_half[x][x], pit & 1)) return false;
                tc_fence_after();
                if (leader) {
                    umma_ts(tmem + col_o(x), pa, vb, kIdescPV, pj > 0 ? 1u : 0u);
#pragma unroll
                    for (int kk = 1; kk < kKT / 32; ++kk)
                        umma_ts_c<true>(tmem + col_o(x), pa + kk * 8, vb + (uint64_t)(kk * 128), kIdescPV);
                }
                __syncwarp();
                if (x == 0) {
                    if (!wait_all(&sm.p_half[x][1], pit & 1)) return false;
                    tc_fence_after();
                }
                if (leader) {
#pragma unroll
                    for (int kk = kKT / 32; kk < kKT / 16; ++kk)
                        umma_ts_c<true>(tmem + col_o(x), pa + kk * 8, vb + (uint64_t)(kk * 128), kIdescPV);
                    umma_commit(smem_u32(&sm.o_done[x]));
                    if (x == 1) commit_tile(&sm.v_empty[vs]);   // B is the V tile's last reader
                }
                __syncwarp();
                return true;
            };
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit, kCtas>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit, kPair>(a, idx, qblocks, rank);
                if (!t.run) continue;
                if (!(ok = wait_all(&sm.q_ready, units & 1))) break;
                for (int j = 0; j < t.n_kt; ++j, ++it) {
                    const int ks = it % kStages;
                    if (!(ok = wait_all(&sm.k_full[ks], (it / kStages) & 1))) break;
                    tc_fence_after();
                    issue_s(0, ks);                                        // S_A(j)
                    if (pend_it >= 0 && !(ok = issue_pv(1, pend_it, pend_j))) break;   // O_B, tile j-1
                    issue_s(1, ks);                                        // S_B(j)
                    if (leader) {
                        commit_tile(&sm.k_empty[ks]);
                        if (j == t.n_kt - 1) umma_commit(smem_u32(&sm.q_empty));
                    }
                    __syncwarp();
                    if (!(ok = issue_pv(0, it, j))) break;                 // O_A, tile j
                    pend_it = it;
                    pend_j = j;
                }
                // the unit's last O_B += P_B V now, not behind the next unit's Q and first S_A
                if (ok && pend_it >= 0) ok = issue_pv(1, pend_it, pend_j);
                pend_it = -1;
                ++units;
            }
            // Every MMA issued must have finished before tensor memory is released.
            if (leader) umma_commit(smem_u32(&sm.mma_idle));
            __syncwarp();
            mbar_wait(smem_u32(&sm.mma_idle), 0);
        } else {
            // ---------------------------------------------------------------- converters
            if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
            const int w = warp < kProducerWarp ? warp - kSoftmaxWarps : warp - (16 - kConv);
            int units = 0, it = 0;               // units, code tiles (K and V)
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit, kCtas>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit, kPair>(a, idx, qblocks, rank);
                if (!t.run) continue;
                int sigma = kNone;               // exponent of sigma
                DeadRows dead(t.win, t.kt0 * kKT);
                bool any_dead = false;
                TileParams par = {};
                for (int i = 0; i < 2 * t.n_kt; ++i, ++it) {     // K(0), V(0), K(1), ...
                    const bool is_k = !(i & 1);
                    const int st = it % kRing, kt = it >> 1, ks = kt % kStages;
                    if (!(ok = wait_all(&sm.c_full[st], (it / kRing) & 1))) break;
                    if (is_k) {
                        dead = DeadRows(t.win, (t.kt0 + (i >> 1)) * kKT);
                        any_dead = dead.any();
                        if constexpr (kPair) {
                            if (!(ok = wait_all(&sm.scaled[kt % kReady], (kt / kReady) & 1))) break;
                            par = sm.params[kt % kParams];
                        } else {
                            par = scale_tile(sm.ring, st, dead, sigma, lane);
                        }
                    }
                    const int unit = is_k ? par.unit : par.sigma_exp;   // exponent of what the tile is divided by
                    if (kt >= kStages &&
                        !(ok = wait_all(is_k ? &sm.k_empty[ks] : &sm.v_empty[ks], ((kt / kStages) - 1) & 1)))
                        break;
                    if (!kPair && is_k && w == 0 && lane == 0) sm.params[kt % kParams] = par;
                    const uint32_t dst = smem_u32(is_k ? sm.k[ks] : sm.v[ks]);
                    // (V starts two warps on, so that over both the rounds are nearly even)
                    const int first = is_k ? w : w < 2 ? w + kConv - 2 : w - 2;
                    const int row0 = 64 * rank, end = kPair ? row0 + 64 : kKT;
                    convert_tile<kBits, kPair>(sm.ring, st, dst, exp2_int(-unit), any_dead, dead, row0, end, first, lane);
                    fence_proxy_async_smem();    // generic writes -> visible to the MMA's reads, and the copies'
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&sm.c_empty[st]));
                        mbar_arrive(smem_u32(kPair ? &sm.half_done[!is_k][ks] : is_k ? &sm.k_full[ks] : &sm.v_full[ks]));
                    }
                    if (i == 0) {                // Q, which has been on its way meanwhile
                        if (!(ok = wait_all(&sm.q_full, units & 1))) { ++it; break; }
                        convert_q<kConv>(sm.q[0][0], w, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sm.q_ready));
                        ++units;
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax warps
        // Warpgroup x (= warp / 4) owns query tile x; thread = one row = one TMEM lane.
        regs_inc();
        if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + lane;    // MMA row == TMEM lane
        const int pl = row >> 2;                   // query position within the tile
        const int hl = row & 3;                    // query head within the group
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_col = col_s(x), o_col = col_o(x);
        int it = 0;
        bool ok = true;
        float split_m = -INFINITY, split_l = 0.f, split_sigma = 1.f;   // kSplit: no key seen so far
        bool split_done = false;
        // (a unit's lengths are looked up before the epilogue of the one before it, whose stores they would
        // otherwise queue behind)
        [[maybe_unused]] Unit next;
        [[maybe_unused]] bool fetched = false;
        next.run = false;
        for (int r = 0; ok; ++r) {
            const int idx = snake<kSplit, kCtas>(a, r, total);
            if (idx < 0) break;
            const Unit t = [&]() -> Unit {
                if constexpr (!kSplit) {
                    const bool have = fetched;
                    fetched = false;
                    return have ? next : unit_for<kPlanned, kSplit, kPair>(a, idx, qblocks, rank);
                } else {
                    return unit_for<kPlanned, kSplit, kPair>(a, idx, qblocks, rank);
                }
            }();
            if (!t.run) continue;
            const int pos_first = t.pos0 + x * kTilePos;
            const int pos = pos_first + pl;
            float m = -INFINITY;                   // running max, log2 units (scaled)
            float l = 0.f;                         // running sum of the weights
            float sigma = 1.f;                     // what O is in units of
            for (int j = 0; j < t.n_kt; ++j, ++it) {
                ok = wait_or_abort(smem_u32(&sm.s_full[x]), it & 1, abort_flag, a.err);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + s_col + c * 32, s[c]);
                const TileParams par = sm.params[it % kParams];
                const float sl2 = a.scale_log2 * par.k_unit;
                const float grow = par.grow;
                sigma = par.sigma;
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);

                // the tile's rows that some query of this MMA tile may not see lie past its first position, or
                // before its last one's window and behind the sinks: a bit per column, 32 columns at a time
                const int base = (t.kt0 + j) * kKT;
                const int shift = t.win.shift;     // list row r beyond the sinks holds position r + shift
                if (base + kKT - 1 > pos_first - shift ||
                    (base + shift <= pos_first + kTilePos - 1 - a.window && base + kKT > a.sinks)) {
                    const int hi = pos - shift - base + 1;       // columns below hi
                    const int lo = hi - min(a.window, hi + kKT);   // columns from lo on
                    const int sk = a.sinks - base;               // or below sk
                    const auto below = [](int n) {               // bits 0 .. n-1
                        return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
                    };
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t see = below(hi - c * 32) & (~below(lo - c * 32) | below(sk - c * 32));
                        // (a warp's 8 positions differ in few columns: most chunks are all seen)
                        if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see >> e & 1u)) s[c][e] = __float_as_uint(-INFINITY);
                    }
                }
                float cmax[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float r0 = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
                    float r1 = fmaxf(__uint_as_float(s[c][16]), __uint_as_float(s[c][17]));
#pragma unroll
                    for (int e = 2; e < 16; e += 2) {
                        r0 = fmax3(r0, __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                        r1 = fmax3(r1, __uint_as_float(s[c][e + 16]), __uint_as_float(s[c][e + 17]));
                    }
                    cmax[c] = fmaxf(r0, r1);
                }
                const float rmax = fmaxf(fmaxf(cmax[0], cmax[1]), fmaxf(cmax[2], cmax[3]));
                const float m_new = fmaxf(m, rmax * sl2);
                const bool rescale = m_new > m + kRescaleThreshold;   // also when m == -inf
                const float m_use = rescale ? m_new : m;
                const float alpha = rescale ? fast_exp2(m - m_new) : 1.f;
                // a row with every key so far masked keeps m = -inf; its weights are 0
                const float m_sub = m_use == -INFINITY ? 0.f : m_use;
                if (j > 0 && __any_sync(0xffffffffu, rescale || grow != 1.f)) {
                    // O must hold O += P V of the previous tile before it is rescaled (that product was
                    // issued before this tile's S, so it has completed).
                    ok = wait_or_abort(smem_u32(&sm.o_done[x]), (it - 1) & 1, abort_flag, a.err);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                    const float f = alpha * grow;
                    // 8 columns at a time: the scores of this tile are still live in registers
#pragma unroll 1
                    for (int c = 0; c < 16; ++c) {
                        uint32_t o[8];
                        tmem_ld8(lane_base + o_col + c * 8, o);
                        tmem_wait_ld8(o);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st8(lane_base + o_col + c * 8, o);
                    }
                }
                float part[4] = {0.f, 0.f, 0.f, 0.f};   // 4 partial row sums
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int c = 2 * h; c < 2 * h + 2; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float x0, x1;
                            ffma2(x0, x1, __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]), sl2, sl2,
                                  -m_sub, -m_sub);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            // weights are at most 2^8 (the lazy maximum); in f16 those under 2^-14 lose bits one by
                            // one.  The row sum takes them before that rounding (2^-12 of a weight at most): the sum of
                            // the rounded ones costs three instructions a pair more, 2000 of 10000 a tile.
                            pk[e / 2] = pack_f16x2(p0, p1);
                            const int k = (e >> 1) & 1;
                            fadd2(part[2 * k], part[2 * k + 1], p0, p1);
                        }
                        // P columns 16c..16c+15 go over S columns already read into registers
                        tmem_st16(lane_base + s_col + 16 * c, pk);
                    }
                    // P of keys 64h..64h+63 is in tensor memory: release that half of O += P V
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.p_half[x][h]));
                }
                const float rsum = (part[0] + part[1]) + (part[2] + part[3]);
                l = l * alpha + rsum;
                m = m_use;
            }
            if (!ok) break;

            // ------------------------------------------------------------ epilogue
            if constexpr (!kSplit) {
                const int idx_next = snake<kSplit, kCtas>(a, r + 1, total);
                if (idx_next >= 0) {
                    next = unit_for<kPlanned, kSplit, kPair>(a, idx_next, qblocks, rank);
                    fetched = true;
                }
            }
            ok = wait_or_abort(smem_u32(&sm.o_done[x]), (it - 1) & 1, abort_flag, a.err);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            if constexpr (kSplit) {
                split_m = m;
                split_l = l;
                split_sigma = sigma;
                split_done = true;
                continue;
            }
            const float inv_l = sigma / l;
            const bool row_ok = x * kTilePos + pl < t.positions;
            const size_t orow = (size_t)(t.tok0 + x * kTilePos + pl) * kHq + t.g * kGroup + hl;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld32(lane_base + o_col + c * 32, o);
                tmem_wait_ld(o);
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    w[e / 2] = pack_bf16x2(__uint_as_float(o[e]) * inv_l, __uint_as_float(o[e + 1]) * inv_l);
                // 32-byte stores: each writes whole sectors (out is 32-byte aligned, rows are 256 bytes)
                if (row_ok) {
                    __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(a.out) + orow * kD + c * 32;
                    st_global_32b(d, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
                    st_global_32b(d + 16, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
                }
            }
            if (row_ok && a.lse) a.lse[orow] = (m + __log2f(l)) * kLn2;
            tc_fence_before();
        }
        if constexpr (kSplit) {
            // Once both tiles' products are done, their reads of Q and K are too, and this CTA's O goes
            // over them, row by row, the 16-byte pieces of a row permuted by its low bits so that neither
            // these stores nor the merge's loads meet on a bank.  (All softmax warps come to this barrier,
            // also those that gave up.)
            named_barrier(1, kSoftmaxWarps * 32);
            const int rr = x * kRows + row;
            if (split_done) {
                uint8_t *dst = sm.q[0][0] + rr * (kD * 4);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + o_col + c * 32, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * split_sigma);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        *reinterpret_cast<uint4 *>(dst + (((c * 8 + v) ^ (rr & 7)) << 4)) =
                            make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                }
                tc_fence_before();
            }
            sm.ml[rr][0] = split_m;
            sm.ml[rr][1] = split_l;
        }
    }

    if constexpr (kSplit) {
        // every CTA's part is in its shared memory, merged by all, and stays until all have read it
        // (after an abort too: every wait above is bounded, so every CTA comes here)
        __syncwarp();
        cluster_sync_all();
        if (warp < kSoftmaxWarps) {
            const Unit t = unit_at<false, true>(a, (int)(blockIdx.x / a.unit_ctas), qblocks);
            if (t.run) merge_rows(a, t, smem_u32(sm.q), smem_u32(sm.ml), warp, lane);
        }
        __syncwarp();
        cluster_sync_all();
    }

    // ---------------------------------------------------------------- teardown
    __syncthreads();
    // (a pair: neither exits while the other may write into its memory or arrive on its barriers; every wait above
    // is bounded, so both come here)
    if constexpr (kPair) cluster_sync_all();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int kBits, bool kPlanned, bool kSplit, bool kPair>
cudaError_t launch_mode(const PrefillArgs &a, const CUtensorMap &q_map, const CUtensorMap &k_map,
                        const CUtensorMap &v_map, const CUtensorMap &k16_map, const CUtensorMap &v16_map, int num_sms,
                        cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto kernel = prefill_quant_kernel<kBits, kPlanned, kSplit, kPair>;
    static std::atomic<bool> configured[64] = {};
    if (dev < 0 || dev >= 64 || !configured[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<kBits, kPair>);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true);
    }
    constexpr int kPos = kPair ? kPairPos : kUnitPos;
    const long long qblocks = (a.max_q_len + kPos - 1) / kPos;
    const long long units = (long long)a.num_seqs * kHkv * qblocks;
    // Programmatic dependent launch: the producer waits (griddepcontrol.wait) before its first load, so the
    // launch and prologue may overlap the previous kernel on the stream.
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;   // kSplit and kPair only
    attr[1].val.clusterDim.x = kSplit ? (unsigned)a.unit_ctas : kPair ? 2u : 1u;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (kPlanned) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kPlanThreads);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, prefill_plan_kernel<false, true, kPos>, a, (int)qblocks, (int)units, plan_keys(a));
        if (e != cudaSuccess) return e;
    }
    cfg.numAttrs = kSplit || kPair ? 2 : 1;
    cfg.gridDim = dim3(kSplit  ? (unsigned)(units * a.unit_ctas)
                       : kPair ? 2 * (unsigned)std::min<long long>(units, num_sms / 2)
                               : (unsigned)std::min<long long>(units, num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<kBits, kPair>;
    return cudaLaunchKernelEx(&cfg, kernel, q_map, k_map, v_map, k16_map, v16_map, a);
}

// How many clusters of c CTAs of the split kernel fit on the current device at once, c = 2 .. 8
// (looked up once per device; a lookup that failed counts as none and is made again next time).
template <int kBits>
cudaError_t split_clusters(int (&out)[9]) {
    static std::atomic<int> known[64][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = prefill_quant_kernel<kBits, false, true, false>;
    for (int c = 2; c <= 8; ++c) {
        int n = known[dev][c].load();
        if (n == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<kBits, false>);
            if (e != cudaSuccess) return e;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)c;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)c);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kSmemBytes<kBits, false>;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                out[c] = 0;
                continue;
            }
            n = n > 0 ? n : -1;
            known[dev][c].store(n);
        }
        out[c] = n;
    }
    return cudaSuccess;
}

template <int kBits>
cudaError_t launch_bits(PrefillArgs a, long long tiles, const CUtensorMap &q_map, const CUtensorMap &k_map,
                        const CUtensorMap &v_map, const CUtensorMap &k16_map, const CUtensorMap &v16_map, int num_sms,
                        cudaStream_t stream) {
    const long long units = (long long)a.num_seqs * kHkv * ((a.max_q_len + kUnitPos - 1) / kUnitPos);
    a.unit_ctas = 1;
    if (units * 2 <= num_sms) {
        int clusters[9] = {};
        const cudaError_t e = split_clusters<kBits>(clusters);
        if (e != cudaSuccess) return e;
        a.unit_ctas = unit_ctas_for(units, tiles, std::min(a.max_q_len, kUnitPos), num_sms, clusters);
    }
    const auto refused = [](cudaError_t e) {   // a cluster that this device will not run
        return e == cudaErrorLaunchOutOfResources || e == cudaErrorInvalidClusterSize || e == cudaErrorNotSupported ||
               e == cudaErrorCooperativeLaunchTooLarge;
    };
    if (a.unit_ctas > 1) {
        const cudaError_t e =
            launch_mode<kBits, false, true, false>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
        if (!refused(e)) return e;
        cudaGetLastError();   // one CTA a unit, or a pair, instead
        a.unit_ctas = 1;
    }
    // Pairs where a sequence may have more than one CTA's positions: 20 chunks of 65 tokens over contexts of 4000 190 us (one
    // CTA a unit 234), of 128 191 (234), of 129 310 (310), 10 of 256 over 8000 347 (437), 4 of 1024 over 4096 226 (274),
    // 12 of 65 over 1000 45 (49), in 8 bits; in 4 bits 2 to 4 % less each.
    if (a.max_q_len > kUnitPos) {
        const long long pairs = (long long)a.num_seqs * kHkv * ((a.max_q_len + kPairPos - 1) / kPairPos);
        // (units that all start at once need no order)
        const cudaError_t e =
            a.order && pairs > num_sms / 2
                ? launch_mode<kBits, true, false, true>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream)
                : launch_mode<kBits, false, false, true>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
        if (!refused(e)) return e;
        cudaGetLastError();
    }
    if (a.order && units > num_sms)
        return launch_mode<kBits, true, false, false>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
    return launch_mode<kBits, false, false, false>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
}

}  // namespace

cudaError_t launch_prefill_quant(PrefillArgs a, long long tiles, const CUtensorMap &q_map, const CUtensorMap &k_map,
                                 const CUtensorMap &v_map, const CUtensorMap &k16_map, const CUtensorMap &v16_map,
                                 int num_sms, cudaStream_t stream) {
    if (a.num_seqs == 0 || a.max_q_len == 0 || a.total_tokens == 0) return cudaSuccess;
    return a.k_exp ? launch_bits<4>(a, tiles, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream)
                   : launch_bits<8>(a, tiles, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
}

}  // namespace pa
