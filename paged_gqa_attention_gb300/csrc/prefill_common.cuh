// prefill_common.cuh -- what the prefill kernels share: work units and how they are dealt, the
// planning kernel, bounded waits between the roles, and the merge of a cluster's shares.
#pragma once

#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "window.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                    // MMA M (one query tile)
constexpr int kKT = kPrefillKvTile;           // keys per K/V tile (MMA N of S, K of PV)
constexpr int kTilePos = kPrefillQPositions;  // query positions per MMA tile (32)
constexpr int kUnitPos = 2 * kTilePos;        // query positions per work unit (64)
constexpr int kSoftmaxWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kHalf = kRows * 128;            // 128 rows x 64 dims x 2 B = 16 KiB
constexpr uint32_t kParkNs = 20000;           // longest hardware park per wait attempt
constexpr float kRescaleThreshold = 8.0f;     // log2 units: rescale O when the max grows > 2^8
constexpr float kLn2 = 0.693147180559945309f;

// TMEM columns of query tile x (0 = A, 1 = B): S_A 0-127, S_B 128-255, O_A 256-383, O_B 384-511
__device__ __forceinline__ uint32_t col_s(int x) { return x ? 128u : 0u; }
__device__ __forceinline__ uint32_t col_o(int x) { return x ? 384u : 256u; }

struct Unit {
    bool run;       // has work
    bool error;     // inconsistent lengths (recorded once, then skipped)
    int s, g;
    int tok0;       // row of q/out holding the unit's first query position
    int positions;  // real positions in this unit (1..64)
    int pos0;       // absolute position of the unit's first query
    int seq_len;    // context length (keys 0 .. seq_len-1 exist)
    int kt0;        // first key tile visited (0 unless the keys are split)
    int n_kt;       // key tiles to visit: kt0 .. kt0 + n_kt - 1
    int ks;         // key split of the unit (shared-prefix mode)
    // Key tiles 0 .. n_old-1 hold positions 128j .. 128j+127 of the cache, only those below c0
    // being keys; with a fused append the tiles after them hold the new positions from c0 on,
    // 128 a tile (c0 + 128(j - n_old) + r), read from k_new rows tok_base + 128(j - n_old) + r.
    // Without one, c0 = seq_len and every tile is a cache tile.
    int c0;
    int n_old;
    int tok_base;
    // Sliding window: key tile j holds rows 128j .. 128j + 127 of this list.
    WindowRows win;
};

// Unit idx of the batch; kPos: query positions per unit
template <bool kAppend, bool kWindow, int kPos = kUnitPos>
__device__ __forceinline__ Unit unit_at(const PrefillArgs &a, int idx, int qblocks) {
    Unit t;
    const int per_qb = a.num_seqs * kHkv;
    const int qb = qblocks - 1 - idx / per_qb;   // latest query block first
    const int rem = idx - (idx / per_qb) * per_qb;
    t.s = rem / kHkv;
    t.g = rem % kHkv;
    t.run = false;
    t.error = false;
    const int c0 = __ldg(a.cu_q_lens + t.s);
    const int c1 = __ldg(a.cu_q_lens + t.s + 1);
    const int q_len = c1 - c0;
    const int seq_len = __ldg(a.seq_lens + t.s);
    if (q_len < 0 || q_len > a.max_q_len || c0 < 0 || c1 > a.total_tokens ||
        (q_len > 0 && (seq_len < q_len || seq_len > a.max_blocks_per_seq * kBlock))) {
        t.error = true;
        return t;
    }
    if (qb * kPos >= q_len) return t;
    t.run = true;
    t.tok0 = c0 + qb * kPos;
    t.positions = min(kPos, q_len - qb * kPos);
    t.pos0 = seq_len - q_len + qb * kPos;
    t.seq_len = seq_len;
    t.kt0 = 0;
    t.ks = 0;
    t.tok_base = c0;
    if constexpr (kAppend) {
        t.c0 = seq_len - q_len;
        t.n_old = (t.c0 + kKT - 1) / kKT;
        t.n_kt = t.n_old + (t.pos0 + t.positions - 1 - t.c0) / kKT + 1;
    } else {
        t.c0 = seq_len;
        t.n_kt = (t.pos0 + t.positions - 1) / kKT + 1;
        t.n_old = t.n_kt;
    }
    if constexpr (kWindow) {
        t.win.set(a.window, a.sinks, t.pos0, t.pos0 + t.positions - 1);
        t.n_kt = (t.win.rows + kKT - 1) / kKT;
    }
    return t;
}

// Key tiles of unit idx (the unit_at rule; 0 for a unit without work, which sorts last).
template <bool kAppend, bool kWindow, int kPos>
__device__ __forceinline__ int plan_key(const PrefillArgs &a, int idx, int qblocks) {
    const Unit t = unit_at<kAppend, kWindow, kPos>(a, idx, qblocks);
    return t.run ? t.n_kt : 0;
}

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxKeys = 12288;   // histogram buckets in shared memory (48 KiB)
// key buckets: a unit visits at most 2 * max_blocks_per_seq key tiles
inline int plan_keys(const PrefillArgs &a) { return 2 * a.max_blocks_per_seq + 2; }

// Planning kernel for several sequences: a counting sort of the units by key tiles, most
// first (longest processing time first), written as order[rank] = unit.  Units with equal
// keys take their ranks in whatever order the atomics resolve; every unit is computed by
// one CTA on its own, so the outputs do not depend on that order.  nk = key buckets.
template <bool kAppend, bool kWindow, int kPos = kUnitPos>
__global__ void __launch_bounds__(kPlanThreads, 1) prefill_plan_kernel(const PrefillArgs a, int qblocks, int total,
                                                                       int nk) {
    __shared__ int hist[kPlanMaxKeys];
    __shared__ int warp_sum[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // The prefill may start its prologue now; it waits for this kernel before it reads the order.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the key of this thread's first unit is needed twice and kept
    const int key0 = tid < total ? min(plan_key<kAppend, kWindow, kPos>(a, tid, qblocks), nk - 1) : 0;
    for (int k = tid; k < nk; k += kPlanThreads) hist[k] = 0;
    __syncthreads();
    for (int idx = tid; idx < total; idx += kPlanThreads)
        atomicAdd(&hist[idx == tid ? key0 : min(plan_key<kAppend, kWindow, kPos>(a, idx, qblocks), nk - 1)], 1);
    __syncthreads();
    // hist[k] <- first rank of key k = number of units with more key tiles.  Thread t owns
    // the keys hi, hi - 1, ..., hi - per + 1 counted from the top.
    const int per = (nk + kPlanThreads - 1) / kPlanThreads;
    const int hi = nk - 1 - tid * per;
    int sum = 0;
    for (int i = 0; i < per; ++i)
        if (hi - i >= 0) sum += hist[hi - i];
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += n;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += n;
        }
        warp_sum[lane] = w;   // inclusive over warps
    }
    __syncthreads();
    int run = incl - sum + (warp > 0 ? warp_sum[warp - 1] : 0);
    for (int i = 0; i < per; ++i) {
        const int k = hi - i;
        if (k >= 0) {
            const int v = hist[k];
            hist[k] = run;
            run += v;
        }
    }
    __syncthreads();
    for (int idx = tid; idx < total; idx += kPlanThreads) {
        const int key = idx == tid ? key0 : min(plan_key<kAppend, kWindow, kPos>(a, idx, qblocks), nk - 1);
        const int rank = atomicAdd(&hist[key], 1);
        a.order[rank] = idx;
    }
    // Complete only after the kernel before this one on the stream (kv_append lets its
    // dependents start early): the prefill launched after this kernel relies on it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Index of this CTA's r-th unit in the snake order (or -1 past the end); kSplit: the cluster's one; kCtas: of
// so many CTAs that take a unit together.
template <bool kSplit, int kCtas = 1>
__device__ __forceinline__ int snake(const PrefillArgs &a, int r, int total) {
    if constexpr (kSplit) return r == 0 ? (int)(blockIdx.x / a.unit_ctas) : -1;
    const int G = gridDim.x / kCtas, cta = (int)blockIdx.x / kCtas;
    const int idx = r * G + ((r & 1) ? (G - 1 - cta) : cta);
    return idx < total ? idx : -1;
}

// Bounded wait shared by all roles: gives up when another role has aborted or after
// the time limit (then raises the abort flag and records the timeout).
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                              uint32_t *err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_parked(bar, parity, kParkNs)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            record_error(err, kErrTimeout);
            return false;
        }
    }
}

// The rows of a tile of the list that no position of the unit sees: from `tail` on (past the last
// position), and lo .. hi - 1 (behind the sinks and before every position's window).  Their V rows
// may hold anything, NaN included; P is 0 there, but 0 * NaN is not.
struct DeadRows {
    int lo, hi, tail;

    __device__ __forceinline__ DeadRows(const WindowRows &w, int c0) {
        lo = max(w.s - c0, 0);
        hi = min(w.lo - w.shift - c0, kKT);
        tail = min(w.rows - c0, kKT);
    }
    __device__ __forceinline__ bool any() const { return lo < hi || tail < kKT; }
};

// kSplit: merge a share of the unit's rows from the O, m and l that every CTA of the cluster left
// in its shared memory (a row whose l is 0 saw no key there), and write their outputs.  Warp w takes
// rows rank + ctas (w + 8i); a lane 4 dims.
// o_base, ml_base: where in shared memory O [256][128] fp32 and (m, l) [256][2] are.
__device__ __forceinline__ void merge_rows(const PrefillArgs &a, const Unit &t, uint32_t o_base, uint32_t ml_base, int warp,
                                           int lane) {
    const int ctas = a.unit_ctas, rank = (int)(blockIdx.x % ctas);
    for (int row = rank + ctas * warp; row < 2 * kRows; row += ctas * kSoftmaxWarps) {
        const int x = row >> 7, pl = (row & (kRows - 1)) >> 2, hl = row & 3;   // tile, position, head
        if (x * kTilePos + pl >= t.positions) continue;
        const uint32_t o_at = o_base + (uint32_t)(row * kD * 4 + ((lane ^ (row & 7)) << 4));
        float m[8], l[8], M = -INFINITY;
        float4 o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= ctas) break;
            m[k] = ld_cluster_f32(peer_addr(ml_base + row * 8, (uint32_t)k));
            l[k] = ld_cluster_f32(peer_addr(ml_base + row * 8 + 4, (uint32_t)k));
            o[k] = ld_cluster_f4(peer_addr(o_at, (uint32_t)k));
            M = fmaxf(M, m[k]);
        }
        float L = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= ctas) break;
            if (l[k] == 0.f) continue;
            const float e = fast_exp2(m[k] - M);
            L = __fmaf_rn(l[k], e, L);
            v[0] = __fmaf_rn(o[k].x, e, v[0]);
            v[1] = __fmaf_rn(o[k].y, e, v[1]);
            v[2] = __fmaf_rn(o[k].z, e, v[2]);
            v[3] = __fmaf_rn(o[k].w, e, v[3]);
        }
        const float inv = 1.f / L;
        const size_t orow = (size_t)(t.tok0 + x * kTilePos + pl) * kHq + t.g * kGroup + hl;
        uint2 w;
        w.x = pack_bf16x2(v[0] * inv, v[1] * inv);
        w.y = pack_bf16x2(v[2] * inv, v[3] * inv);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * kD + lane * 4) = w;
        if (a.lse && lane == 0) a.lse[orow] = (M + __log2f(L)) * kLn2;
    }
}

// CTAs that share a unit (a cluster) in a windowed prefill of `units` units of up to `tiles` key
// tiles and `positions` query positions: 1 unless all clusters fit on the GPU at once.  Of the
// sizes that do, the one whose run of tiles (1.5 us each) and merge take least.
int unit_ctas_for(long long units, long long tiles, int positions, int num_sms, const int (&max_clusters)[9]) {
    const double merge_us = 1.6 + 5.2 * positions / kUnitPos;
    int best = 1;
    double best_us = 1.5 * (double)tiles;
    for (int c = 2; c <= 8 && units * c <= num_sms; ++c) {
        if (max_clusters[c] < units) continue;
        const double us = 1.5 * (double)((tiles + c - 1) / c) + merge_us;
        if (us < best_us) {
            best = c;
            best_us = us;
        }
    }
    return best;
}

}  // namespace
}  // namespace pa
