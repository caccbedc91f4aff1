// Softmax attention for bf16 storage on the tensor cores (sm_100a: TMA,
// tcgen05, TMEM).
#pragma once

#include <cuda.h>

#include "softmax.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace sm {
namespace tcf {

constexpr int TILE = 16384;  // one 128 x 64 bf16 tile
constexpr long long kWaitBudget = 4000000000LL;  // clock cycles (about 2 s)

// [B][H][L][64] bf16 with strides; boxes of `rows` tokens x `heads` heads, one
// row of 128 bytes each, 128-byte swizzle, zeros outside the tensor.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
        : "memory");
}

// Barriers whose waits are bounded: one that runs out records SA_ERR_TIMEOUT
// and makes every role of the block unwind.
struct Ctl {
    uint64_t* bar;
    volatile int* abort;
    int* status;
    __device__ bool wait(int slot, uint32_t parity) {
        if (tc::mbar_try_wait(bar + slot, parity)) return true;
        if (*abort) return false;
        if (tc::mbar_wait(bar + slot, parity, kWaitBudget)) return true;
        *abort = 1;
        if (status) atomicCAS(status, 0, (int)SA_ERR_TIMEOUT);
        return false;
    }
    // the same for a whole warp: one answer for all lanes
    __device__ bool wait_warp(int slot, uint32_t parity) { return __all_sync(~0u, wait(slot, parity)); }
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Items in the order of falling work (a causal band grows with the position),
// dealt to the blocks there and back so that their sums are alike.
struct Walk {
    int n, r = 0;
    __device__ explicit Walk(int items) : n(items) {}
    __device__ bool next(int& idx) {
        const int g = (int)gridDim.x;
        while (r * g < n) {
            idx = r * g + ((r & 1) ? g - 1 - (int)blockIdx.x : (int)blockIdx.x);
            ++r;
            if (idx < n) return true;
        }
        return false;
    }
};

// 2^x on the FMA pipe for a pair of arguments, x <= 8 or so: round to nearest by
// adding 1.5 * 2^23, then a polynomial of degree 4 for 2^f on [-1/2, 1/2]
// (least squares on Chebyshev nodes, reweighted towards the largest relative
// error, which is 2.7e-6: a probability is rounded to 2^-9 after it, and the row
// sums' duals keep 1e-5).
__device__ __forceinline__ void exp2_poly2(uint64_t x, float& e0, float& e1) {
    float x0, x1;
    tc::upk2(x, x0, x1);
    const uint64_t xx = tc::pk2(fmaxf(x0, -126.f), fmaxf(x1, -126.f));
    const uint64_t t = tc::add2(xx, tc::pk2(12582912.f, 12582912.f));
    const uint64_t f = tc::sub2(xx, tc::add2(t, tc::pk2(-12582912.f, -12582912.f)));
    uint64_t p = tc::fma2(tc::pk2(9.570101276040077e-3f, 9.570101276040077e-3f), f,
                          tc::pk2(5.591785907745361e-2f, 5.591785907745361e-2f));
    p = tc::fma2(p, f, tc::pk2(2.40247443318367e-1f, 2.40247443318367e-1f));
    p = tc::fma2(p, f, tc::pk2(6.931217908859253e-1f, 6.931217908859253e-1f));
    p = tc::fma2(p, f, tc::pk2(9.999992847442627e-1f, 9.999992847442627e-1f));
    float p0, p1, t0, t1;
    tc::upk2(p, p0, p1);
    tc::upk2(t, t0, t1);
    e0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
    e1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
}

// Bits x of a word for 32 consecutive positions with a <= x <= b.
__device__ __forceinline__ uint32_t range_bits(int a, int b) {
    if (b < 0 || a > 31 || b < a) return 0u;
    return (~0u << max(a, 0)) & (~0u >> (31 - min(b, 31)));
}

// ---------------------------------------------------------------------------
// Forward.  An item is a pair of tiles of 128 packed query rows (sub-tiles 0 and
// 1) of one key head and a part of their keys, walked in chunks of 128 keys that
// both sub-tiles share.  Eight softmax warps, four per sub-tile, one row per
// thread; a loader, a mask warp, and one issuing warp per product:
//   S_t = Q_t K^T    128 x 128 x 64 into TMEM, read by the rows' threads
//   O_t += P_t V     128 x 64 x 128, P_t bf16 from TMEM
// A row's scores leave TMEM at once, so S of the next chunk is formed while the
// exponentials of this one are taken.  The running maximum is only moved when
// it has grown by more than 8 (in log2 units): until then probabilities are at
// most 2^8, which the fp32 sums and bf16's exponent hold without loss, and O
// needs no rescaling.  The mask warp turns the token mask and the ends of the
// item's keys into one word per 32 columns, and zeroes the rows of V that no
// query of the item may read (0 times whatever they hold).
// ALT (few query rows): both sub-tiles hold the same rows and take the chunks in
// turn, each its own part.

namespace fwd {
constexpr int NST = 4;           // key chunk stages
constexpr int THREADS = 384;
constexpr int W_LOAD = 8, W_MASK = 9, W_S = 10, W_PV = 11;
constexpr int OFF_Q = 0;                       // two buffers of two tiles
constexpr int OFF_ST = OFF_Q + 4 * TILE;       // stages of K and V
constexpr int OFF_WORDS = OFF_ST + NST * 2 * TILE;
constexpr int OFF_BAR = OFF_WORDS + NST * 16;
enum { B_QFULL = 0, B_QEMPTY = 2, B_FULL = 4, B_READY = B_FULL + NST, B_EMPTY = B_READY + NST,
       B_SFULL = B_EMPTY + NST, B_SEMPTY = B_SFULL + 2, B_PFULL = B_SEMPTY + 2, B_PVDONE = B_PFULL + 2,
       B_DRAIN = B_PVDONE + 2, NBAR = B_DRAIN + 1 };
constexpr int OFF_END = OFF_BAR + NBAR * 8 + 16;
constexpr int SMEM = OFF_END + 1024;
static_assert(SMEM <= 227 * 1024, "shared memory");

struct Maps {
    CUtensorMap Q, K, V;
};

// What every role derives from an item's number.
template <bool ALT>
struct Item {
    int b, hk, i0, part, c0, c1, jlo, vlo, vhi, s0[2], s1[2];
    long long first;
    __device__ Item(const Args& a, int idx) {
        part = idx % a.nsplit;
        int x = idx / a.nsplit;
        const int BH = a.B * a.Hk, qt = a.ntile - 1 - x / BH;
        x %= BH;
        hk = x % a.Hk;
        b = x / a.Hk;
        first = a.first(b);
        i0 = qt * (ALT ? a.nq : 2 * a.nq);
        int lo[2], hi[2];
        tile_keys(a, first, i0, min(i0 + a.nq, a.Lq) - 1, lo[0], hi[0]);
        lo[1] = 0;
        hi[1] = -1;
        if (!ALT && i0 + a.nq < a.Lq) tile_keys(a, first, i0 + a.nq, min(i0 + 2 * a.nq, a.Lq) - 1, lo[1], hi[1]);
        vlo = 0;
        vhi = -1;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            if (hi[t] >= lo[t]) {
                vlo = vhi < vlo ? lo[t] : min(vlo, lo[t]);
                vhi = max(vhi, hi[t]);
            }
        const int n = (vhi - vlo + 128) / 128;  // 0 when empty
        jlo = vlo;
        c0 = (int)((long long)n * part / a.nsplit);
        c1 = (int)((long long)n * (part + 1) / a.nsplit);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s0[t] = c0;
            s1[t] = ALT ? c1 : c0;
            if (!ALT && hi[t] >= lo[t]) {
                s0[t] = max(c0, (lo[t] - jlo) / 128);
                s1[t] = min(c1, (hi[t] - jlo) / 128 + 1);
            }
        }
    }
    __device__ __forceinline__ bool uses(int c, int t) const {
        return ALT ? ((c - c0) & 1) == t : c >= s0[t] && c < s1[t];
    }
};

template <bool ALT>
__global__ void __launch_bounds__(THREADS, 1) tc_fwd(const Args a, const __grid_constant__ Maps maps, int nitems) {
    extern __shared__ uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tbase = reinterpret_cast<uint32_t*>(sm + OFF_BAR + NBAR * 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tbase + 1);
    uint32_t* words = reinterpret_cast<uint32_t*>(sm + OFF_WORDS);
    Ctl ctl{bar, abort_flag, a.status};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar + B_QFULL + i, 1);
            tc::mbar_init(bar + B_QEMPTY + i, 1);
            tc::mbar_init(bar + B_SFULL + i, 1);
            tc::mbar_init(bar + B_SEMPTY + i, 4);
            tc::mbar_init(bar + B_PFULL + i, 4);
            tc::mbar_init(bar + B_PVDONE + i, 1);
        }
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bar + B_FULL + s, 1);
            tc::mbar_init(bar + B_READY + s, 1);
            tc::mbar_init(bar + B_EMPTY + s, 1);
        }
        tc::mbar_init(bar + B_DRAIN, 2);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(tbase, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    // TMEM columns: S_t at 128 t, P_t (128 bf16 per row) at 256 + 64 t, O_t at 384 + 64 t
    const uint32_t tm = *tbase, tS = tm, tP = tm + 256, tO = tm + 384;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;

    Walk walk(nitems);
    int idx;
    if (warp == W_LOAD) {
        // ------------------------------------------------------------ loader (one lane)
        if (lane == 0) {
            int it = 0, gc = 0;
            bool ok = true;
            for (; ok && walk.next(idx); ++it) {
                const Item<ALT> w(a, idx);
                const int qb = it & 1;
                if (it >= 2 && !ctl.wait(B_QEMPTY + qb, ((it >> 1) - 1) & 1)) break;
                const uint32_t qbytes = (uint32_t)(a.nq * a.G) * 128u;
                tc::mbar_expect_tx(bar + B_QFULL + qb, ALT ? qbytes : 2 * qbytes);
                for (int t = 0; t < (ALT ? 1 : 2); ++t)
                    tma_load_4d(sm + OFF_Q + (2 * qb + t) * TILE, &maps.Q, bar + B_QFULL + qb, w.i0 + t * a.nq,
                                w.hk * a.G, w.b);
                for (int c = w.c0; c < w.c1; ++c, ++gc) {
                    const int s = gc % NST;
                    if (gc >= NST && !ctl.wait(B_EMPTY + s, ((gc / NST) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = sm + OFF_ST + s * 2 * TILE;
                    tc::mbar_expect_tx(bar + B_FULL + s, 2 * TILE);
                    tma_load_4d(st, &maps.K, bar + B_FULL + s, w.jlo + 128 * c, w.hk, w.b);
                    tma_load_4d(st + TILE, &maps.V, bar + B_FULL + s, w.jlo + 128 * c, w.hk, w.b);
                }
            }
            // the last loads have landed before the block ends, whatever the others do
            for (int x = max(0, it - 2); x < it; ++x) tc::mbar_wait(bar + B_QFULL + (x & 1), (x >> 1) & 1, kWaitBudget);
            for (int x = max(0, gc - NST); x < gc; ++x)
                tc::mbar_wait(bar + B_FULL + x % NST, (x / NST) & 1, kWaitBudget);
        }
        __syncwarp();
    } else if (warp == W_MASK) {
        // ------------------------------------------------------------ mask words, unused rows of V
        int gc = 0;
        bool ok = true;
        for (; ok && walk.next(idx);) {
            const Item<ALT> w(a, idx);
            for (int c = w.c0; c < w.c1; ++c, ++gc) {
                const int s = gc % NST, j0 = w.jlo + 128 * c;
                uint32_t bits[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = j0 + 32 * k + lane;
                    bits[k] = __ballot_sync(~0u, j >= w.vlo && j <= w.vhi && a.live(w.b, j));
                }
                if (!ctl.wait_warp(B_FULL + s, (gc / NST) & 1)) {
                    ok = false;
                    break;
                }
                if (lane < 4) words[4 * s + lane] = lane == 0 ? bits[0] : lane == 1 ? bits[1] : lane == 2 ? bits[2] : bits[3];
                if ((bits[0] & bits[1] & bits[2] & bits[3]) != ~0u) {
                    uint8_t* v = sm + OFF_ST + s * 2 * TILE + TILE;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t off = ~bits[k];
                        while (off) {  // four rows at a time, eight lanes of 16 bytes each
                            uint32_t m = off;
                            for (int x = 0; x < (lane >> 3); ++x) m &= m - 1;
                            if (m)
                                *reinterpret_cast<uint4*>(v + (32 * k + __ffs(m) - 1) * 128 + (lane & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                            for (int x = 0; x < 4; ++x) off &= off - 1;
                        }
                    }
                    tc::fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + B_READY + s);
            }
        }
    } else if (warp == W_S) {
        // ------------------------------------------------------------ S = Q K^T
        const uint32_t id = tc::idesc_bf16(128, 128, false, false);
        const uint64_t dQ = tc::sdesc_sw128(tc::smem_u32(sm + OFF_Q), 16, 1024);
        const uint64_t dK = tc::sdesc_sw128(tc::smem_u32(sm + OFF_ST), 16, 1024);
        int it = 0, gc = 0, n[2] = {0, 0};
        bool ok = true;
        for (; ok && walk.next(idx); ++it) {
            const Item<ALT> w(a, idx);
            const int qb = it & 1;
            if (!ctl.wait_warp(B_QFULL + qb, (it >> 1) & 1)) break;
            for (int c = w.c0; ok && c < w.c1; ++c, ++gc) {
                const int s = gc % NST;
                if (!ctl.wait_warp(B_READY + s, (gc / NST) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!w.uses(c, t)) continue;
                    if (n[t] >= 1 && !ctl.wait_warp(B_SEMPTY + t, (n[t] - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    ++n[t];
                    tc::tc_fence_after();
                    const uint64_t dA = tc::sdesc_add(dQ, (2 * qb + (ALT ? 0 : t)) * TILE);
                    const uint64_t dB = tc::sdesc_add(dK, s * 2 * TILE);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_bf16(tS + 128 * t, tc::sdesc_add(dA, 32 * k), tc::sdesc_add(dB, 32 * k), id, k > 0);
                        tc::tc_commit(bar + B_SFULL + t);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (tc::elect_one()) tc::tc_commit(bar + B_QEMPTY + qb);
            __syncwarp();
        }
        if (tc::elect_one()) tc::tc_commit(bar + B_DRAIN);
        __syncwarp();
        tc::mbar_wait(bar + B_DRAIN, 0, kWaitBudget);
    } else if (warp == W_PV) {
        // ------------------------------------------------------------ O += P V
        const uint32_t id = tc::idesc_bf16(128, 64, false, true);
        const uint64_t dV = tc::sdesc_sw128(tc::smem_u32(sm + OFF_ST + TILE), TILE, 1024);
        int gc = 0, n[2] = {0, 0};
        bool ok = true;
        for (; ok && walk.next(idx);) {
            const Item<ALT> w(a, idx);
            bool some[2] = {false, false};
            for (int c = w.c0; ok && c < w.c1; ++c, ++gc) {
                const int s = gc % NST;
                if (!ctl.wait_warp(B_READY + s, (gc / NST) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!w.uses(c, t)) continue;
                    if (!ctl.wait_warp(B_PFULL + t, n[t] & 1)) {
                        ok = false;
                        break;
                    }
                    ++n[t];
                    tc::tc_fence_after();
                    const uint64_t dB = tc::sdesc_add(dV, s * 2 * TILE);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma_bf16_ts(tO + 64 * t, tP + 64 * t + 8 * k, tc::sdesc_add(dB, k * 2048), id,
                                            (some[t] || k > 0) ? 1u : 0u);
                        tc::tc_commit(bar + B_PVDONE + t);
                    }
                    __syncwarp();
                    some[t] = true;
                }
                if (!ok) break;
                if (tc::elect_one()) tc::tc_commit(bar + B_EMPTY + s);
                __syncwarp();
            }
        }
        if (tc::elect_one()) tc::tc_commit(bar + B_DRAIN);
        __syncwarp();
        tc::mbar_wait(bar + B_DRAIN, 0, kWaitBudget);
    } else {
        // ------------------------------------------------------------ softmax rows
        const int t = warp >> 2, qd = warp & 3;
        const int r = qd * 32 + lane;  // row of the sub-tile
        const int g = r / a.nq, iq = r % a.nq;
        const uint32_t lanebase = (uint32_t)(qd * 32) << 16;
        const uint64_t c2p = tc::pk2(a.c2, a.c2);
        int gc = 0, n = 0;
        bool ok = true;
        for (; ok && walk.next(idx);) {
            const Item<ALT> w(a, idx);
            const int i = w.i0 + (ALT ? 0 : t * a.nq) + iq;
            const bool row = g < a.G && i < a.Lq;
            int lo = 0, hi = -1;
            {
                const long long p = w.first + i;
                if (row && p >= 0 && p < a.Lk && a.live(w.b, (int)p)) a.keys(p, lo, hi);
            }
            const bool dead = __all_sync(~0u, hi < lo);  // no row of this warp attends anything
            float m = -INFINITY;  // running maximum (log2 units), moved in steps of more than 8
            uint64_t l2[2] = {0, 0};
            float l = 0.f;
            bool some = false;
            for (int c = w.c0; c < w.c1; ++c, ++gc) {
                if (!w.uses(c, t)) continue;
                const int s = gc % NST;
                if (!ctl.wait_warp(B_READY + s, (gc / NST) & 1) || !ctl.wait_warp(B_SFULL + t, n & 1)) {
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
                if (dead) {  // its rows of P and O are never read
                    // the P barrier's last phase is over once its P V is
                    if (n > 0 && !ctl.wait_warp(B_PVDONE + t, (n - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        tc::mbar_arrive(bar + B_SEMPTY + t);
                        tc::mbar_arrive(bar + B_PFULL + t);
                    }
                    ++n;
                    continue;
                }
                uint32_t sv[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::tmem_ld32(tS + 128 * t + lanebase + 32 * k, sv[k]);
                const int j0 = w.jlo + 128 * c;
                uint32_t on[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) on[k] = words[4 * s + k] & range_bits(lo - j0 - 32 * k, hi - j0 - 32 * k);
                const bool full = __all_sync(~0u, (on[0] & on[1] & on[2] & on[3]) == ~0u);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + B_SEMPTY + t);
                if (!full) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((on[k] >> j) & 1u)) sv[k][j] = 0xff800000u;  // -inf
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        top[k] = max_nan(top[k], max_nan(__uint_as_float(sv[k][j]), __uint_as_float(sv[k][j + 1])));
                const float mx = max_nan(max_nan(top[0], top[1]), max_nan(top[2], top[3])) * a.c2;
                const bool move = mx > m + 8.f || (m == -INFINITY && mx > -INFINITY);
                // the last P V has read P and added to O
                if (n > 0 && !ctl.wait_warp(B_PVDONE + t, (n - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (__any_sync(~0u, move)) {
                    const float f = move ? ex2(m - mx) : 1.f;  // 0 from an empty row
                    if (move) m = mx;
                    float x, y;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        tc::upk2(l2[e], x, y);
                        l2[e] = tc::pk2(x * f, y * f);
                    }
                    if (some) {
                        tc::tc_fence_after();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t o[16];
                            tc::tmem_ld16(tO + 64 * t + lanebase + 16 * e, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tc::tmem_st16(tO + 64 * t + lanebase + 16 * e, o);
                        }
                    }
                }
                if (!(mx < INFINITY)) {  // NaN or +inf among the scores: so is the row
                    l2[0] = tc::pk2(NAN, NAN);
                    if (m == -INFINITY) m = 0.f;
                }
                const float use = m == -INFINITY ? 0.f : -m;
                const uint64_t mp = tc::pk2(use, use);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t pw[16];
                    // a word of 32 columns is in use for all rows, for none, or for some
                    const bool all = full || __all_sync(~0u, on[k] == ~0u);
                    if (all) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint64_t x = tc::fma2(
                                tc::pk2(__uint_as_float(sv[k][2 * j]), __uint_as_float(sv[k][2 * j + 1])), c2p, mp);
                            float e0, e1;
                            if (j % 4 == 3) {
                                exp2_poly2(x, e0, e1);
                            } else {
                                tc::upk2(x, e0, e1);
                                e0 = ex2(e0);
                                e1 = ex2(e1);
                            }
                            l2[j & 1] = tc::add2(l2[j & 1], tc::pk2(e0, e1));
                            pw[j] = tc::pack_bf16(e0, e1);
                        }
                    } else if (__any_sync(~0u, on[k] != 0u)) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint64_t x = tc::fma2(
                                tc::pk2(__uint_as_float(sv[k][2 * j]), __uint_as_float(sv[k][2 * j + 1])), c2p, mp);
                            float e0, e1;
                            tc::upk2(x, e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            l2[j & 1] = tc::add2(l2[j & 1], tc::pk2(e0, e1));
                            pw[j] = tc::pack_bf16(e0, e1);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) pw[j] = 0u;
                    }
                    tc::tmem_st16(tP + 64 * t + lanebase + 16 * k, pw);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + B_PFULL + t);
                ++n;
                some = true;
            }
            if (!ok) break;
            {
                float x0, x1, x2, x3;
                tc::upk2(l2[0], x0, x1);
                tc::upk2(l2[1], x2, x3);
                l = (x0 + x1) + (x2 + x3);
            }
            const long long at = ((long long)w.b * a.Hq + w.hk * a.G + g) * a.Lq + i;
            uint32_t o[2][32];
            if (some) {  // false where this warp formed no P
                if (!ctl.wait_warp(B_PVDONE + t, (n - 1) & 1)) break;
                tc::tc_fence_after();
                tc::tmem_ld32(tO + 64 * t + lanebase, o[0]);
                tc::tmem_ld32(tO + 64 * t + lanebase + 32, o[1]);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) o[0][j] = o[1][j] = 0u;
            }
            if (!row) continue;
            if (a.nparts > 1) {
                const long long pa = at * a.nparts + (ALT ? 2 * w.part + t : w.part);
                a.part_ml[pa] = make_float2(m, l);
                if (m > -INFINITY) {
                    float4* po = reinterpret_cast<float4*>(a.part_o + pa * 64);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            po[8 * k + j] = make_float4(__uint_as_float(o[k][4 * j]), __uint_as_float(o[k][4 * j + 1]),
                                                        __uint_as_float(o[k][4 * j + 2]), __uint_as_float(o[k][4 * j + 3]));
                }
            } else {
                const bool none = m == -INFINITY;  // nothing attended
                const float inv = none ? 0.f : 1.f / l;
                uint4* out = reinterpret_cast<uint4*>(a.o.at<__nv_bfloat16>(w.b, w.hk * a.G + g, i));
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = tc::pack_bf16(__uint_as_float(o[k][8 * j + 2 * e]) * inv,
                                                 __uint_as_float(o[k][8 * j + 2 * e + 1]) * inv);
                        out[4 * k + j] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                a.u[at] = none ? 0.f : -(m + lg2(l)) * kLn2;
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

}  // namespace fwd
}  // namespace tcf
}  // namespace sm
}  // namespace sa
