// prefill_quant.cu -- causal (chunked) prefill attention over the 8-bit or the 4-bit KV cache, with an
// optional sliding window, on the 5th-generation tensor cores.
//
// Page "从零搭建AI工程能力：手写KV Cache与动态批处理实战" §3.2 stores the KV cache in 8 bits, §3.3 cuts
// long prompts into chunks that attend to the cached context before them; here both at once.  The
// attention, its work units, key lists, tiles and tensor memory are those of the windowed form of
// prefill.cu (a window as long as the context is plain causal attention); what differs is how the codes
// of a key tile become operands:
//   K, 8 bits  E4M3 codes are operands as they are (kind::f8f6f4).  A query row q, divided by the power of two
//              that brings its largest magnitude to 224 .. 448, is a sum hi + lo of two E4M3 rows: 4 + 4
//              significant bits, all that bf16 has, down to 2^-10 (2^-18 of the row's largest).  S = hi K^T +
//              lo K^T takes as long as one f16 product, and K needs no conversion and half the shared memory.
//   K, 4 bits  code * scale, 6 bits and exact in f16; q in f16 (|q| < 65504).
//   V          V' = code * s / sigma in f16, sigma a power of two above the first tile's largest scale, taken anew
//              only when a tile's V' could leave f16; O is then rescaled, as it is for the running maximum, and
//              the epilogue multiplies by sigma.  8 bits: s is split into a sum of two f16, so that code *
//              scale is rounded once; 4 bits: exact.  V' below 2^-14 loses bits one by one.
// A key's own factor (8 bits: its scale, 4 bits: its power of two) multiplies its column of the scores in fp32.
// The conversions run on warps of their own next to the softmax, 128 x 128 values an operand tile; with both
// operands converted by four warps they set the pace (4500 clk a tile, 2048 of products).
//
// CTA, persistent, one per SM:
//   warps 0-3, 4-7   softmax + epilogue of query tiles A and B (thread = row = TMEM lane)
//   warps 8-11       converters of V and of Q
//   warps 12-15      4 bits only: converters of K
//   then             a warp as TMA producer, one as TMEM allocator and tcgen05.mma issuer, two idle ones that
//                    complete the warpgroup (a warpgroup gives up or takes registers as a whole)
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

constexpr int kConvertWarps = 4;
constexpr int kVWarp = 8;                     // 8-11
constexpr int kKWarp = 12;                    // 12-15, 4 bits
constexpr uint32_t kTileBytes = 2 * kHalf;    // a 128 x 128 f16 tile
constexpr int kStages = 2;                    // f16 tiles of V, and in 4 bits of K
constexpr int kParams = 4;                    // see TileParams

template <int kBits>
struct Config;
template <>
struct Config<8> {
    static constexpr int kProducerWarp = 12, kThreads = 16 * 32;
    // registers a thread, warpgroup by warpgroup: together what the block is launched with
    static constexpr int kSoftmaxRegs = 176, kConvertRegs = 80, kControlRegs = 80;
    static_assert(2 * kSoftmaxRegs + kConvertRegs + kControlRegs <= 4 * 128, "register split");
    static constexpr int kRow = kD;           // bytes of a row's codes
    static constexpr int kKTiles = 3;         // K tiles ready for the products (the codes themselves)
    static constexpr int kSlotRows = kKT;     // rows of a slot of the V ring
    static constexpr int kVSlots = 2;
    static constexpr int kCols = 4;           // see QuantSmem::col
};
template <>
struct Config<4> {
    static constexpr int kProducerWarp = 16, kThreads = 20 * 32;
    static constexpr int kSoftmaxRegs = 160, kConvertRegs = 56, kControlRegs = 48;
    static_assert(2 * kSoftmaxRegs + 2 * kConvertRegs + kControlRegs <= 5 * 96, "register split");
    static constexpr int kRow = kFp4RowCodes;
    static constexpr int kKTiles = kStages;
    static constexpr int kSlotRows = kKT / 2;
    static constexpr int kKSlots = 3, kVSlots = 4;
    static constexpr int kCols = 3;
};

constexpr uint32_t idesc(int format, int m, int n, bool b_mn_major) {   // as idesc_bf16, A and B of that format
    return (idesc_bf16(m, n, b_mn_major) & ~((7u << 7) | (7u << 10))) | (uint32_t)format << 7 | (uint32_t)format << 10;
}
// format 0: f16 under kind::f16, E4M3 under kind::f8f6f4
constexpr uint32_t kIdescQK = idesc(0, kRows, kKT, false);
constexpr uint32_t kIdescPV = idesc(0, kRows, kD, true);

// D[tmem] (+)= A[smem] * B[smem], 8-bit operands, 32 deep
template <bool kAcc>
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(kAcc ? 1 : 0)
        : "memory");
}

// What the softmax needs of V tile `it`, in entry it % 4, announced on u_full.  Entry it is written after V(it - 1)
// was converted, which needed the tile of V(it - 3), so both query tiles' softmax have read entry it - 3 by then.
struct TileParams {
    float sigma;
    float grow;               // the factor that brings O to units of sigma (1, or sigma has just grown)
};

struct Barriers {
    uint64_t q_full, q_ready, q_empty;
    uint64_t k_full[3], k_empty[3];           // operand tiles
    uint64_t v_full[kStages], v_empty[kStages];
    uint64_t kc_full[3], kc_empty[3];         // code slots
    uint64_t vc_full[4], vc_empty[4];
    uint64_t u_full[kParams];
    uint64_t s_full[2], p_half[2][2], o_done[2];   // per query tile (P in two key halves)
    uint64_t mma_idle;
    uint32_t tmem_base;
    int abort;
};

template <int kBits>
struct QuantSmem;
template <>
struct QuantSmem<8> {
    uint8_t q[2][2][kHalf];          // [tile A|B][bf16: dims 0-63 | 64-127, then E4M3: hi | lo]
    uint8_t k[3][kKT * kD];          // operand tiles: the codes
    uint8_t v_codes[2][kKT * kD];
    uint8_t v[kStages][2][kHalf];
    // Factors of the score columns.  Entry it % 4 is loaded with K(it), into the tile of K(it - 3): S_B(it - 3) is
    // done then, and O_B += P_B(it - 4) V was issued before it, so the softmax have read entry it - 4.
    float col[4][kKT];
    float v_scale[2][kKT];
    // Powers of two of the query rows, two units in turn (Q of the unit after next is converted when S of the
    // next one is done, so when P of this one's last tile was there).
    float q_unit[2][2 * kRows];
    TileParams params[kParams];
    float ml[2 * kRows][2];          // kSplit: running maximum and sum of every row
    Barriers b;
};
template <>
struct QuantSmem<4> {
    uint8_t q[2][2][kHalf];          // bf16, then f16
    uint8_t k[kStages][2][kHalf];
    uint8_t v[kStages][2][kHalf];
    union {
        struct {                     // slots of half a tile
            uint8_t k_codes[3][kKT / 2 * kFp4RowCodes], v_codes[4][kKT / 2 * kFp4RowCodes];
            uint8_t k_scale[3][kKT / 2 * kFp4Groups], v_scale[4][kKT / 2 * kFp4Groups];
            uint8_t k_exp[3][kKT / 2], v_exp[4][kKT / 2];
        };
        float ml[2 * kRows][2];      // kSplit, at the end
    };
    // Entry it % 3 is written with K(it), into the tile of K(it - 2): S_B(it - 2) is done then, and O_B += P_B(it - 3) V
    // was issued before it.
    float col[3][kKT];
    TileParams params[kParams];
    Barriers b;
};
// kSplit: O of the 256 rows, fp32, over q and what follows it
static_assert(offsetof(QuantSmem<8>, k) == sizeof(QuantSmem<8>::q) &&
                  offsetof(QuantSmem<8>, v) >= 2 * kRows * kD * sizeof(float) &&
                  offsetof(QuantSmem<4>, v) >= 2 * kRows * kD * sizeof(float),
              "split merge area");

template <int kBits>
constexpr size_t kSmemBytes = sizeof(QuantSmem<kBits>) + 1024;
static_assert(kSmemBytes<8> <= 232448 && kSmemBytes<4> <= 232448, "shared memory");

template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// Two fp32 sums in one packed instruction: (d0, d1) += (a0, a1)
__device__ __forceinline__ void fadd2(float &d0, float &d1, float a0, float a1) {
    asm("{\n .reg .b64 ra, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rd, {%0, %1};\n add.rn.f32x2 rd, rd, ra;\n"
        " mov.b64 {%0, %1}, rd;\n}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}
// (d0, d1) = (a0 * b0, a1 * b1)
__device__ __forceinline__ void fmul2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n"
        " mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
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

// The work unit dealt as the r-th of this CTA.
template <bool kPlanned, bool kSplit>
__device__ __forceinline__ Unit unit_for(const PrefillArgs &a, int idx, int qblocks) {
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

// Where a slot's codes, scales and exponents go (8 bits: `scale` are floats, and no exponents).
struct SlotAt {
    uint32_t codes, scale, exp, bar;
};

// Fetch rows c0 .. c0 + kRowsMax - 1 of the unit's key list (load_list_tile's rule in prefill.cu): codes in boxes of
// 64 and 16 rows, their scales beside them a run at a time.  Block ids are reported by K.
template <int kBits, int kRowsMax>
__device__ __forceinline__ void load_codes(const PrefillArgs &a, const Unit &t, const int32_t *bt, int c0, bool is_k,
                                           const SlotAt &to, const CUtensorMap *map64, const CUtensorMap *map16) {
    constexpr int kRow = Config<kBits>::kRow;
    const int rows = max(0, min(kRowsMax, ((t.win.rows + 15) & ~15) - c0));
    mbar_arrive_expect_tx(to.bar, (uint32_t)rows * (kRow + (kBits == 8 ? 4 : kFp4Groups + 1)));
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
            bulk_load(to.scale + r * 4, static_cast<const float *>(is_k ? a.k_scale : a.v_scale) + row, run * 4, to.bar);
        } else {
            bulk_load(to.scale + r * kFp4Groups,
                      static_cast<const uint8_t *>(is_k ? a.k_scale : a.v_scale) + row * kFp4Groups, run * kFp4Groups, to.bar);
            bulk_load(to.exp + r, (is_k ? a.k_exp : a.v_exp) + row, run, to.bar);
        }
        while (run > 0) {
            const int n = run >= 64 ? 64 : 16;
            tma_load_4d(to.codes + r * kRow, run >= 64 ? map64 : map16, to.bar, 0, t.g, off, blk);
            r += n;
            off += n;
            run -= n;
        }
    }
}

// ---------------------------------------------------------------- conversion (one warp's share)

// 2^n as a float for n in -126 .. 127 (clamped).
__device__ __forceinline__ float exp2_int(int n) { return __uint_as_float((uint32_t)(min(max(n, -126), 127) + 127) << 23); }

// Rows 8b .. 8b + 7 of a slot are converted in one round of a warp: lanes 8q .. 8q + 3 have row q of the 8, lanes 8q +
// 4 .. 8q + 7 row q ^ 5, so that with the swizzles below neither a load (whose rows must differ in bit 2) nor a
// store (in bit 0) meets a bank twice; lane c of four has dims 16c .. 16c + 15 and 64 + 16c ...
__device__ __forceinline__ int round_row(int lane) { return (lane >> 3) ^ ((lane & 4) ? 5 : 0); }

// What a lane reads for that, and its f16 values code * scale * unit, `unit` a power of two.
template <int kBits>
struct Piece;
template <>
struct Piece<8> {
    uint4 c[2];
    float s;

    // (128-byte rows, 128-byte swizzle: sw128; 64 dims on flip bit 6 of the address)
    __device__ __forceinline__ void read(uint32_t codes, const float *scale, const uint8_t *, int row, int chunk) {
        const uint32_t at = codes + sw128(row, chunk);
        c[0] = ld_shared_16(at);
        c[1] = ld_shared_16(at ^ 64u);
        s = scale[row];
    }
    __device__ __forceinline__ void convert(float unit, uint32_t (&h)[2][8]) const {
        // the scale as hi + lo, so that code * scale is rounded once (code * lo is far below the last place)
        const float x = s * unit;
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
    }
};
template <>
struct Piece<4> {
    uint2 c[2];
    uint32_t s[2], exp;

    // (64-byte rows, 64-byte swizzle: 16-byte piece p of row r is at p ^ (r / 2 % 4); 64 dims on flip bit 5)
    __device__ __forceinline__ void read(uint32_t codes, const uint8_t *scale, const uint8_t *exps, int row, int chunk) {
        const uint32_t at = codes + row * kFp4RowCodes + (((chunk >> 1) ^ ((row >> 1) & 3)) << 4) + ((chunk & 1) << 3);
        c[0] = ld_shared_8(at);
        c[1] = ld_shared_8(at ^ 32u);
        s[0] = scale[row * kFp4Groups + chunk];
        s[1] = scale[row * kFp4Groups + chunk + 4];
        exp = exps ? exps[row] : 127;
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

// kRounds x 8 rows of a slot, from `row0` on, into an f16 tile (its rows from dst_row0 on), the next round read
// ahead.  Rows of the tile in [dead_lo, dead_hi) and from dead_tail on become zeros: their codes and scales may be anything,
// and 0 * NaN is not 0.
// The loop stays rolled: the roles of this kernel run different code at the same time, and with the rounds
// unrolled, once for K and once for V, warps waited for instructions more than for anything else (2.3 of 10
// warp-cycles an instruction).
template <int kBits, typename Scale>
__device__ __forceinline__ void convert_rows(uint32_t codes, const Scale *scale, const uint8_t *exps, int row0, int rounds,
                                             uint32_t dst, int dst_row0, float unit, bool any_dead, const DeadRows &dead,
                                             int lane) {
    const int c = lane & 3;
    int row = row0 + round_row(lane), to = dst_row0 + round_row(lane);
    uint32_t at = dst + sw128(to, 2 * c);
    Piece<kBits> x;
    x.read(codes, scale, exps, row, c);
#pragma unroll 1
    for (int b = 0; b < rounds; ++b) {
        Piece<kBits> next = x;
        row += 8;
        if (b + 1 < rounds) next.read(codes, scale, exps, row, c);
        uint32_t h[2][8];
        x.convert(unit, h);
        if (any_dead && ((to >= dead.lo && to < dead.hi) || to >= dead.tail)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) h[e >> 3][e & 7] = 0u;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            st_shared_16(at + u * kHalf, h[u][0], h[u][1], h[u][2], h[u][3]);
            st_shared_16((at ^ 16u) + u * kHalf, h[u][4], h[u][5], h[u][6], h[u][7]);
        }
        x = next;
        at += 1024;
        to += 8;
    }
}

// Exponent n of the power of two that the largest scale of the tile's live rows is below (8 bits) or at (4 bits);
// kNone: every one is zero or no number.  top4: of rows 4 lane .. 4 lane + 3, biased as below.
constexpr int kNone = -1000;
__device__ __forceinline__ int top_exponent(const int (&top4)[4], const DeadRows &dead, int lane) {
    int top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * lane + i;
        if (!(r >= dead.lo && r < dead.hi) && r < dead.tail) top = max(top, top4[i]);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    return top ? min(max(top - 127, -126), 126) : kNone;
}
// biased exponent + 1 of a scale, 0 for a zero, an infinity and a NaN
__device__ __forceinline__ int scale_exponent(float x) {
    const uint32_t bits = __float_as_uint(x) & 0x7fffffffu;
    return bits < 0x7f800000u && bits ? (int)(bits >> 23) + 1 : 0;
}

// Q in place, bf16 -> f16 (4 bits): this warp's quarter.
__device__ __forceinline__ void convert_q_f16(uint8_t *q, int w, int lane) {
    uint4 *p = reinterpret_cast<uint4 *>(q) + w * (4 * kHalf / 16 / kConvertWarps) + lane;
#pragma unroll 2
    for (int i = 0; i < 4 * kHalf / 16 / kConvertWarps / 32; ++i) {
        uint4 x = p[i * 32];
        x.x = bf16x2_to_f16x2(x.x);
        x.y = bf16x2_to_f16x2(x.y);
        x.z = bf16x2_to_f16x2(x.z);
        x.w = bf16x2_to_f16x2(x.w);
        p[i * 32] = x;
    }
}

// Q in place, bf16 -> E4M3 hi | lo (8 bits): this warp's 64 rows, four at a time, 8 lanes a row with 16 dims each.  A
// row's two 128-byte pieces, dims 0-63 and 64-127, become its hi and its lo row.
__device__ __forceinline__ void convert_q_e4m3(uint8_t *q, float *q_unit, int w, int lane) {
    const int c = lane & 7;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
        const int row = w * 64 + 4 * i + (lane >> 3), r = row & (kRows - 1);
        uint8_t *tile = q + (row >> 7) * (2 * kHalf);
        const uint8_t *src = tile + (c >> 2) * kHalf;
        const uint4 a = *reinterpret_cast<const uint4 *>(src + sw128(r, 2 * (c & 3)));
        const uint4 b = *reinterpret_cast<const uint4 *>(src + sw128(r, 2 * (c & 3) + 1));
        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t top = 0;     // largest magnitude as bits of an fp32 (NaN above infinity)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, max(x[e] << 16 & 0x7fffffffu, x[e] & 0x7fff0000u));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = umax_xor(top, o);
        // q = m 2^E <= 1.75 * 2^8 * 2^n: n = E - 8, one more when m > 1.75 (at least -119, so that 2^-n is a float)
        const int n = top ? max((int)((top + 0x7fffffu - 0x600000u) >> 23) - 127 - 8, -119) : 0;
        const float inv = exp2_int(-n);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y[4] = {bf16_lo(x[2 * e]) * inv, bf16_hi(x[2 * e]) * inv, bf16_lo(x[2 * e + 1]) * inv,
                                bf16_hi(x[2 * e + 1]) * inv};
            hi[e] = f32x2_to_e4m3x2(y[0], y[1]) | f32x2_to_e4m3x2(y[2], y[3]) << 16;
            uint32_t h[2];
            e4m3x4_to_f16x2x2(hi[e], h[0], h[1]);
            const float2 z0 = __half22float2(*reinterpret_cast<const __half2 *>(&h[0]));
            const float2 z1 = __half22float2(*reinterpret_cast<const __half2 *>(&h[1]));
            lo[e] = f32x2_to_e4m3x2(y[0] - z0.x, y[1] - z0.y) | f32x2_to_e4m3x2(y[2] - z1.x, y[3] - z1.y) << 16;
        }
        __syncwarp();   // every lane of the row has read it
        *reinterpret_cast<uint4 *>(tile + sw128(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(tile + kHalf + sw128(r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        // (an infinite or NaN q has no E4M3 form: its row's scores are NaN)
        if (c == 0) q_unit[row] = top >= 0x7f800000u ? __int_as_float(0x7fc00000) : exp2_int(n);
    }
}

template <int kBits, bool kPlanned, bool kSplit>
__global__ void __launch_bounds__(Config<kBits>::kThreads, 1)
prefill_quant_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap k16_map,
                     const __grid_constant__ CUtensorMap v16_map, const PrefillArgs a) {
    using Smem = QuantSmem<kBits>;
    using C = Config<kBits>;
    constexpr int kMmaWarp = C::kProducerWarp + 1;
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Barriers &bar = sm.b;
    volatile int *abort_flag = &bar.abort;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int qblocks = (a.max_q_len + kUnitPos - 1) / kUnitPos;
    const int total = a.num_seqs * kHkv * qblocks;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar.q_full), 1);
        mbar_init(smem_u32(&bar.q_ready), kConvertWarps);
        mbar_init(smem_u32(&bar.q_empty), 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(smem_u32(&bar.k_full[i]), kBits == 8 ? 1 : kConvertWarps);
            mbar_init(smem_u32(&bar.k_empty[i]), 1);
            mbar_init(smem_u32(&bar.kc_full[i]), 1);
            mbar_init(smem_u32(&bar.kc_empty[i]), kConvertWarps);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&bar.v_full[i]), kConvertWarps);
            mbar_init(smem_u32(&bar.v_empty[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&bar.vc_full[i]), 1);
            mbar_init(smem_u32(&bar.vc_empty[i]), kConvertWarps);
        }
        for (int i = 0; i < kParams; ++i) mbar_init(smem_u32(&bar.u_full[i]), 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&bar.s_full[x]), 1);
            mbar_init(smem_u32(&bar.p_half[x][0]), 4);   // the 4 warps of the tile's softmax
            mbar_init(smem_u32(&bar.p_half[x][1]), 4);
            mbar_init(smem_u32(&bar.o_done[x]), 1);
        }
        mbar_init(smem_u32(&bar.mma_idle), 1);
        bar.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&bar.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    const auto wait_all = [&](uint64_t *b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_or_abort(smem_u32(b), parity, abort_flag, a.err));
    };

    if (warp >= C::kProducerWarp) {
        regs_dec<C::kControlRegs>();
        if (warp == C::kProducerWarp) {
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
            int units = 0, kt = 0, ks = 0, vs = 0;   // units, key tiles, slots of K and of V issued
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit>(a, idx, qblocks);
                if (leader && t.error) record_error(a.err, kErrDevice | kErrQLen);
                if (!t.run) continue;
                const int32_t *bt = a.block_table + (size_t)t.s * a.max_blocks_per_seq;
                for (int j = 0; ok && j < t.n_kt; ++j, ++kt) {
                    const int c0 = (t.kt0 + j) * kKT;
                    if constexpr (kBits == 8) {
                        const int st = ks % C::kKTiles;
                        if (ks >= C::kKTiles && !(ok = wait_all(&bar.k_empty[st], ((ks / C::kKTiles) - 1) & 1))) break;
                        const SlotAt to = {smem_u32(sm.k[st]), smem_u32(sm.col[kt % C::kCols]), 0, smem_u32(&bar.k_full[st])};
                        if (leader) load_codes<8, kKT>(a, t, bt, c0, true, to, &k_map, &k16_map);
                        __syncwarp();
                        ++ks;
                    } else {
                        for (int h = 0; h < 2; ++h, ++ks) {
                            const int st = ks % C::kKSlots;
                            if (ks >= C::kKSlots && !(ok = wait_all(&bar.kc_empty[st], ((ks / C::kKSlots) - 1) & 1))) break;
                            const SlotAt to = {smem_u32(sm.k_codes[st]), smem_u32(sm.k_scale[st]), smem_u32(sm.k_exp[st]),
                                               smem_u32(&bar.kc_full[st])};
                            if (leader) load_codes<4, kKT / 2>(a, t, bt, c0 + h * (kKT / 2), true, to, &k_map, &k16_map);
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                    if (j == 0) {   // Q behind the first K tile, which does not wait for the unit before
                        if (units >= 1 && !(ok = wait_all(&bar.q_empty, (units - 1) & 1))) break;
                        if (leader) {
                            const uint32_t qbar = smem_u32(&bar.q_full);
                            mbar_arrive_expect_tx(qbar, 2 * kTileBytes);
                            for (int x = 0; x < 2; ++x) {
                                tma_load_3d(smem_u32(sm.q[x][0]), &q_map, qbar, 0, t.g * kGroup, t.tok0 + x * kTilePos);
                                tma_load_3d(smem_u32(sm.q[x][1]), &q_map, qbar, 64, t.g * kGroup, t.tok0 + x * kTilePos);
                            }
                        }
                        __syncwarp();
                        ++units;
                    }
                    for (int h = 0; h < kKT / C::kSlotRows; ++h, ++vs) {
                        const int st = vs % C::kVSlots;
                        if (vs >= C::kVSlots && !(ok = wait_all(&bar.vc_empty[st], ((vs / C::kVSlots) - 1) & 1))) break;
                        SlotAt to = {0, 0, 0, smem_u32(&bar.vc_full[st])};
                        if constexpr (kBits == 8) {
                            to.codes = smem_u32(sm.v_codes[st]);
                            to.scale = smem_u32(sm.v_scale[st]);
                        } else {
                            to.codes = smem_u32(sm.v_codes[st]);
                            to.scale = smem_u32(sm.v_scale[st]);
                            to.exp = smem_u32(sm.v_exp[st]);
                        }
                        if (leader)
                            load_codes<kBits, C::kSlotRows>(a, t, bt, c0 + h * C::kSlotRows, false, to, &v_map, &v16_map);
                        __syncwarp();
                    }
                }
            }
            // Drain: no TMA copy may still be landing when the CTA exits.  In the normal path every load has
            // been consumed and these waits return at once.
            if (units > 0) mbar_wait(smem_u32(&bar.q_full), (units - 1) & 1);
            constexpr int kK = kBits == 8 ? C::kKTiles : 3;
            for (int i = max(0, ks - kK); i < ks; ++i)
                mbar_wait(smem_u32(kBits == 8 ? &bar.k_full[i % kK] : &bar.kc_full[i % kK]), (i / kK) & 1);
            for (int i = max(0, vs - C::kVSlots); i < vs; ++i)
                mbar_wait(smem_u32(&bar.vc_full[i % C::kVSlots]), (i / C::kVSlots) & 1);
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- MMA issuer (as in prefill.cu)
            const bool leader = elect_one();
            if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
            const uint64_t qd0 = sdesc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
            const uint64_t kd0 = sdesc_sw128(smem_u32(&sm.k[0]), 16, 1024);
            const uint64_t vd0 = sdesc_sw128(smem_u32(sm.v[0][0]), (uint32_t)kHalf, 1024);
            int units = 0, it = 0;
            int pend_it = -1, pend_j = 0;   // O_B += P_B V still to issue for key tile pend_it
            bool ok = true;
            auto issue_s = [&](int x, int ks) {
                const uint64_t qa = qd0 + (uint64_t)(x * 2048);
                const uint32_t sd = tmem + col_s(x);
                if (leader) {
                    if constexpr (kBits == 8) {
                        // hi K^T + lo K^T, 4 steps of 32 dims each (+2 in a descriptor; lo 16 KiB behind hi)
                        const uint64_t kb = kd0 + (uint64_t)(ks * 1024);
                        umma_f8_ss<false>(sd, qa, kb, kIdescQK);
#pragma unroll
                        for (int kk = 1; kk < 2 * kD / 32; ++kk)
                            umma_f8_ss<true>(sd, qa + (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2), kb + (uint64_t)((kk & 3) * 2),
                                             kIdescQK);
                    } else {
                        const uint64_t kb = kd0 + (uint64_t)(ks * 2048);
                        umma_ss_c<false>(sd, qa, kb, kIdescQK);
#pragma unroll
                        for (int kk = 1; kk < kD / 16; ++kk) {
                            const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
                            umma_ss_c<true>(sd, qa + off, kb + off, kIdescQK);
                        }
                    }
                    umma_commit(smem_u32(&bar.s_full[x]));
                }
                __syncwarp();
            };
            auto issue_pv = [&](int x, int pit, int pj) -> bool {
                const int vs = pit % kStages;
                if (x == 0 && !wait_all(&bar.v_full[vs], (pit / kStages) & 1)) return false;
                const uint64_t vb = vd0 + (uint64_t)(vs * 2048);
                const uint32_t pa = tmem + col_s(x);
                if (!wait_all(&bar.p_half[x][x], pit & 1)) return false;
                tc_fence_after();
                if (leader) {
                    umma_ts(tmem + col_o(x), pa, vb, kIdescPV, pj > 0 ? 1u : 0u);
    #pragma unroll
                    for (int kk = 1; kk < kKT / 32; ++kk)
                        umma_ts_c<true>(tmem + col_o(x), pa + kk * 8, vb + (uint64_t)(kk * 128), kIdescPV);
                }
                __syncwarp();
                if (x == 0) {
                    if (!wait_all(&bar.p_half[x][1], pit & 1)) return false;
                    tc_fence_after();
                }
                if (leader) {
    #pragma unroll
                    for (int kk = kKT / 32; kk < kKT / 16; ++kk)
                        umma_ts_c<true>(tmem + col_o(x), pa + kk * 8, vb + (uint64_t)(kk * 128), kIdescPV);
                    umma_commit(smem_u32(&bar.o_done[x]));
                    if (x == 1) umma_commit(smem_u32(&bar.v_empty[vs]));   // B is the V tile's last reader
                }
                __syncwarp();
                return true;
            };
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit>(a, idx, qblocks);
                if (!t.run) continue;
                if (!(ok = wait_all(&bar.q_ready, units & 1))) break;
                for (int j = 0; j < t.n_kt; ++j, ++it) {
                    const int ks = it % C::kKTiles;
                    if (!(ok = wait_all(&bar.k_full[ks], (it / C::kKTiles) & 1))) break;
                    tc_fence_after();
                    issue_s(0, ks);                                        // S_A(j)
                    if (pend_it >= 0 && !(ok = issue_pv(1, pend_it, pend_j))) break;   // O_B, tile j-1
                    issue_s(1, ks);                                        // S_B(j)
                    if (leader) {
                        umma_commit(smem_u32(&bar.k_empty[ks]));
                        if (j == t.n_kt - 1) umma_commit(smem_u32(&bar.q_empty));
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
            if (leader) umma_commit(smem_u32(&bar.mma_idle));
            __syncwarp();
            mbar_wait(smem_u32(&bar.mma_idle), 0);
        }
    } else if (kBits == 4 && warp >= kKWarp) {
        // ---------------------------------------------------------------- converters of K (4 bits)
        regs_dec<C::kConvertRegs>();
        if constexpr (kBits == 4) {
            if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
            const int w = warp - kKWarp;
            int kt = 0, ks = 0;              // key tiles, slots
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int idx = snake<kSplit>(a, r, total);
                if (idx < 0) break;
                const Unit t = unit_for<kPlanned, kSplit>(a, idx, qblocks);
                if (!t.run) continue;
                for (int j = 0; ok && j < t.n_kt; ++j, ++kt) {
                    const int st = kt % kStages;
                    if (kt >= kStages && !(ok = wait_all(&bar.k_empty[st], ((kt / kStages) - 1) & 1))) break;
                    for (int h = 0; h < 2; ++h, ++ks) {
                        const int sl = ks % C::kKSlots;
                        if (!(ok = wait_all(&bar.kc_full[sl], (ks / C::kKSlots) & 1))) break;
                        // this warp's 16 rows of the half; its columns' factors.  (Rows that are no keys may become
                        // anything: their columns are masked.)
                        if (lane < 16)
                            sm.col[kt % C::kCols][h * 64 + w * 16 + lane] = fp4_unit(sm.k_exp[sl][w * 16 + lane]);
                        convert_rows<4>(smem_u32(sm.k_codes[sl]), sm.k_scale[sl], nullptr, w * 16, 2, smem_u32(sm.k[st]),
                                        h * 64 + w * 16, 1.f, false, DeadRows(t.win, 0), lane);
                        fence_proxy_async_smem();    // generic writes -> visible to the MMA's reads
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&bar.kc_empty[sl]));
                            if (h == 1) mbar_arrive(smem_u32(&bar.k_full[st]));
                        }
                    }
                }
            }
        }
    } else if (warp >= kVWarp) {
        // ---------------------------------------------------------------- converters of V and Q
        regs_dec<C::kConvertRegs>();
        if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int w = warp - kVWarp;
        // V' stays below 65504: codes reach 448 (2688 with their group's scale), so the tile's largest scale
        // may be this many powers of two above sigma
        constexpr int kHeadroom = kBits == 8 ? 7 : 4;
        int units = 0, kt = 0, vs = 0;       // units, key tiles, slots
        bool ok = true;
        for (int r = 0; ok; ++r) {
            const int idx = snake<kSplit>(a, r, total);
            if (idx < 0) break;
            const Unit t = unit_for<kPlanned, kSplit>(a, idx, qblocks);
            if (!t.run) continue;
            int sigma = kNone;               // exponent of sigma
            for (int j = 0; j < t.n_kt; ++j, ++kt) {
                const DeadRows dead(t.win, (t.kt0 + j) * kKT);
                const int st = kt % kStages;
                int top4[4];
                if constexpr (kBits == 8) {
                    const int sl = vs % C::kVSlots;
                    if (!(ok = wait_all(&bar.vc_full[sl], (vs / C::kVSlots) & 1))) break;
                    const float4 x = *reinterpret_cast<const float4 *>(sm.v_scale[sl] + 4 * lane);
                    top4[0] = scale_exponent(x.x), top4[1] = scale_exponent(x.y);
                    top4[2] = scale_exponent(x.z), top4[3] = scale_exponent(x.w);
                } else {
                    const int s0 = vs % C::kVSlots, s1 = (vs + 1) % C::kVSlots;
                    if (!(ok = wait_all(&bar.vc_full[s0], (vs / C::kVSlots) & 1))) break;
                    if (!(ok = wait_all(&bar.vc_full[s1], ((vs + 1) / C::kVSlots) & 1))) break;
                    const uint32_t x = *reinterpret_cast<const uint32_t *>(sm.v_exp[lane < 16 ? s0 : s1] + 4 * (lane & 15));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = (int)(x >> (8 * i) & 0xffu);
                        top4[i] = e < (int)kFp4NanExp ? e : 0;
                    }
                }
                const int top = top_exponent(top4, dead, lane);
                float grow = 1.f;
                if (top != kNone && (sigma == kNone || top > sigma + kHeadroom)) {
                    if (sigma != kNone) grow = exp2_int(sigma - top);
                    sigma = top;
                }
                const int unit = sigma == kNone ? 0 : sigma;
                if (w == 0 && lane == 0) {
                    sm.params[kt % kParams] = TileParams{exp2_int(unit), grow};
                    mbar_arrive(smem_u32(&bar.u_full[kt % kParams]));
                }
                __syncwarp();
                if (kt >= kStages && !(ok = wait_all(&bar.v_empty[st], ((kt / kStages) - 1) & 1))) break;
                constexpr int kWarpRows = C::kSlotRows / kConvertWarps;
                for (int h = 0; h < kKT / C::kSlotRows; ++h, ++vs) {
                    const int sl = vs % C::kVSlots;
                    if constexpr (kBits == 8)
                        convert_rows<8>(smem_u32(sm.v_codes[sl]), sm.v_scale[sl], nullptr, w * kWarpRows, kWarpRows / 8,
                                        smem_u32(sm.v[st]), w * kWarpRows, exp2_int(-unit), dead.any(), dead, lane);
                    else
                        convert_rows<4>(smem_u32(sm.v_codes[sl]), sm.v_scale[sl], sm.v_exp[sl], w * kWarpRows, kWarpRows / 8,
                                        smem_u32(sm.v[st]), h * C::kSlotRows + w * kWarpRows, exp2_int(-unit), dead.any(),
                                        dead, lane);
                    fence_proxy_async_smem();        // generic writes -> visible to the MMA's reads
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar.vc_empty[sl]));
                }
                if (lane == 0) mbar_arrive(smem_u32(&bar.v_full[st]));
                if (j == 0) {                // Q, which has been on its way meanwhile
                    if (!(ok = wait_all(&bar.q_full, units & 1))) break;
                    if constexpr (kBits == 8)
                        convert_q_e4m3(sm.q[0][0], sm.q_unit[units & 1], w, lane);
                    else
                        convert_q_f16(sm.q[0][0], w, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar.q_ready));
                    ++units;
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax warps
        // Warpgroup x (= warp / 4) owns query tile x; thread = one row = one TMEM lane.
        regs_inc<C::kSoftmaxRegs>();
        if constexpr (kPlanned) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + lane;    // MMA row == TMEM lane
        const int pl = row >> 2;                   // query position within the tile
        const int hl = row & 3;                    // query head within the group
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_col = col_s(x), o_col = col_o(x);
        int it = 0, units = 0;
        bool ok = true;
        float split_m = -INFINITY, split_l = 0.f, split_sigma = 1.f;   // kSplit: no key seen so far
        bool split_done = false;
        // (a unit's lengths are looked up before the epilogue of the one before it, whose stores they would
        // otherwise queue behind)
        [[maybe_unused]] Unit next;
        [[maybe_unused]] bool fetched = false;
        next.run = false;
        for (int r = 0; ok; ++r) {
            const int idx = snake<kSplit>(a, r, total);
            if (idx < 0) break;
            const Unit t = [&]() -> Unit {
                if constexpr (!kSplit) {
                    const bool have = fetched;
                    fetched = false;
                    return have ? next : unit_for<kPlanned, kSplit>(a, idx, qblocks);
                } else {
                    return unit_for<kPlanned, kSplit>(a, idx, qblocks);
                }
            }();
            if (!t.run) continue;
            const int pos_first = t.pos0 + x * kTilePos;
            const int pos = pos_first + pl;
            float m = -INFINITY;                   // running max, log2 units (scaled)
            float l = 0.f;                         // running sum of the weights
            float sigma = 1.f;                     // what O is in units of
            float sl2 = a.scale_log2;
            for (int j = 0; j < t.n_kt; ++j, ++it) {
                ok = wait_or_abort(smem_u32(&bar.s_full[x]), it & 1, abort_flag, a.err);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + s_col + c * 32, s[c]);
                ok = wait_or_abort(smem_u32(&bar.u_full[it % kParams]), (it / kParams) & 1, abort_flag, a.err);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const TileParams par = sm.params[it % kParams];
                const float grow = par.grow;
                sigma = par.sigma;
                if constexpr (kBits == 8) {
                    if (j == 0) sl2 = a.scale_log2 * sm.q_unit[units & 1][x * kRows + row];
                }
                const float4 *col = reinterpret_cast<const float4 *>(sm.col[it % C::kCols]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
                // every column by its key's factor
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 f = col[c * 8 + e / 4];
                        float y[4];
                        fmul2(y[0], y[1], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]), f.x, f.y);
                        fmul2(y[2], y[3], __uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3]), f.z, f.w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[c][e + i] = __float_as_uint(y[i]);
                    }

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
                    ok = wait_or_abort(smem_u32(&bar.o_done[x]), (it - 1) & 1, abort_flag, a.err);
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
                    if (lane == 0) mbar_arrive(smem_u32(&bar.p_half[x][h]));
                }
                const float rsum = (part[0] + part[1]) + (part[2] + part[3]);
                l = l * alpha + rsum;
                m = m_use;
            }
            if (!ok) break;
            ++units;

            // ------------------------------------------------------------ epilogue
            if constexpr (!kSplit) {
                const int idx_next = snake<kSplit>(a, r + 1, total);
                if (idx_next >= 0) {
                    next = unit_for<kPlanned, kSplit>(a, idx_next, qblocks);
                    fetched = true;
                }
            }
            ok = wait_or_abort(smem_u32(&bar.o_done[x]), (it - 1) & 1, abort_flag, a.err);
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
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int kBits, bool kPlanned, bool kSplit>
cudaError_t launch_mode(const PrefillArgs &a, const CUtensorMap &q_map, const CUtensorMap &k_map,
                        const CUtensorMap &v_map, const CUtensorMap &k16_map, const CUtensorMap &v16_map, int num_sms,
                        cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto kernel = prefill_quant_kernel<kBits, kPlanned, kSplit>;
    static std::atomic<bool> configured[64] = {};
    if (dev < 0 || dev >= 64 || !configured[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<kBits>);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true);
    }
    const long long qblocks = (a.max_q_len + kUnitPos - 1) / kUnitPos;
    const long long units = (long long)a.num_seqs * kHkv * qblocks;
    // Programmatic dependent launch: the producer waits (griddepcontrol.wait) before its first load, so the
    // launch and prologue may overlap the previous kernel on the stream.
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;   // kSplit only
    attr[1].val.clusterDim.x = kSplit ? (unsigned)a.unit_ctas : 1u;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = kSplit ? 2 : 1;
    if constexpr (kPlanned) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kPlanThreads);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, prefill_plan_kernel<false, true>, a, (int)qblocks, (int)units, plan_keys(a));
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(kSplit ? (unsigned)(units * a.unit_ctas) : (unsigned)std::min<long long>(units, num_sms));
    cfg.blockDim = dim3(Config<kBits>::kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<kBits>;
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
    const auto kernel = prefill_quant_kernel<kBits, false, true>;
    for (int c = 2; c <= 8; ++c) {
        int n = known[dev][c].load();
        if (n == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<kBits>);
            if (e != cudaSuccess) return e;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)c;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)c);
            cfg.blockDim = dim3(Config<kBits>::kThreads);
            cfg.dynamicSmemBytes = kSmemBytes<kBits>;
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
    if (a.unit_ctas > 1) {
        const cudaError_t e =
            launch_mode<kBits, false, true>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
        if (e != cudaErrorLaunchOutOfResources && e != cudaErrorInvalidClusterSize && e != cudaErrorNotSupported &&
            e != cudaErrorCooperativeLaunchTooLarge)
            return e;
        cudaGetLastError();   // the clusters were refused: one CTA a unit instead
        a.unit_ctas = 1;
    }
    if (a.order && units > num_sms)   // (units that all start at once need no order)
        return launch_mode<kBits, true, false>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
    return launch_mode<kBits, false, false>(a, q_map, k_map, v_map, k16_map, v16_map, num_sms, stream);
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
