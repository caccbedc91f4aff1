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

// The largest of three; NaN if any is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Eight consecutive TMEM columns of this warp's lane quadrant.
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Registers per thread of the calling warpgroup from here on.
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
// error, which is 2.7e-6).  Degree 4, where the row-sum sweeps of the Sinkhorn
// iteration have 5: these exponentials enter one sum, not 2 T of them, a quarter of
// them at that, so u is off by 2.7e-6 at most of the 1e-5 that duals keep; P is
// rounded to bf16 next, off by up to 2^-8.
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
// Forward.  An item is NR tiles of 128 packed query rows of one key head and a
// part of their keys, walked in chunks of 64 keys that all tiles share.  Four
// groups of four softmax warps, one row per thread, each run one softmax: NR row
// tiles times KS = 4 / NR subsets of the chunks (every KS-th), whose results are
// joined through TMEM at the item's end.  Beside them a loader, a mask warp and
// two warps that issue both products:
//   S = Q K^T    128 x 64 x 64 into TMEM, read by the rows' threads
//   O += P V     128 x 64 x 64, P bf16 in TMEM over the S it came from
// Four chains (S, exponentials, P V) in flight hide each other's latency: the
// same kernel with two groups on chunks of 128 keys spent half its time in the
// hand-overs.  8192 dense tokens of 8 heads take 235 us (tensor cores and the
// exponentials alone 85 and 115): the exponential unit is 57 % busy, the tensor
// cores 38 %, DRAM 1 %; the rest is a chain's hand-overs, S to P to O, and issue.
// P is rounded to bf16 for P V: one MMA takes both operands in one type, V is bf16, and
// P in two parts would double these products.  The sum of a row is that of the unrounded P in
// fp32.  Against 64 bits O is off by 2.1e-3 to 2.4e-3 of its norm, 1.7e-3 of it the rounding of
// O itself (which is all that is off where P stays fp32).
// The running maximum is only moved when it has grown by more than 8 (in log2
// units): until then probabilities are at most 2^8, which the fp32 sums and bf16's
// exponent hold without loss, and O needs no rescaling.  The mask warp turns the
// token mask and the ends of the item's keys into one word per 32 columns, and
// zeroes the rows of V that no query of the item may read (0 times whatever they
// hold).
namespace fwd {
constexpr int THREADS = 640;
constexpr int W_LOAD = 16, W_MASK = 17, W_MMA = 18;  // 18: groups 0 and 1, 19: groups 2 and 3
// registers per thread: the block is launched with 96 x 640 = 61440
constexpr int REG_SOFTMAX = 104, REG_OTHER = 64;
static_assert(512 * REG_SOFTMAX + 128 * REG_OTHER <= 61440, "register split");
constexpr int KT = TILE / 2;  // one 64 x 64 bf16 tile of keys or values
constexpr int NIT = 4;        // items in flight between the loader and the other warps
// fma(S, c2, -m) takes m's rounding, half a step, into every exponent of a row: it
// cancels between P and its sum while it is at most 1/2.  From kRound on a row's
// products are rounded as m was and then subtracted, so that the largest gives 1,
// whatever its size.  (By row: the groups that share its keys then do the same.)
// A warp that holds such a row takes kBig for the first key that all its rows
// attend, and with it none of its words for a whole one: the test stands where masks
// are looked at (beside the unmasked words it took 4 to 9 % of the kernel's time).
constexpr float kRound = 0x1p24f;
constexpr int kBig = 0x7fffffff;

// What every role needs of an item; the loader writes it, once per block.
struct Item {
    int b, hk, i0, part, c0, c1, jlo, vlo, vhi, pad;  // b < 0: no more items
    int s0[4], s1[4];                                // chunks of each row tile
    long long first;
};

template <int NR>
struct Lay {
    static constexpr int KS = 4 / NR;
    static constexpr int NST = NR == 4 ? 5 : NR == 2 ? 8 : 10;  // key chunk stages
    static constexpr int Q = 0;                                 // two buffers of NR tiles
    static constexpr int ST = Q + 2 * NR * TILE;                // stages of K and V
    static constexpr int ITEM = ST + NST * 2 * KT;
    static constexpr int ML = ITEM + NIT * (int)sizeof(Item);   // maxima and sums of the joined subsets
    static constexpr int WORDS = ML + (4 - NR) * 128 * 8;
    static constexpr int BAR = WORDS + NST * 8;
    // barriers
    static constexpr int QFULL = 0, QEMPTY = 2, IFULL = 4, IEMPTY = IFULL + NIT, SFULL = IEMPTY + NIT,
                         PFULL = SFULL + 4, OFULL = PFULL + 4, MFULL = OFULL + 4, MEMPTY = MFULL + NR,
                         DRAIN = MEMPTY + NR, FULL = DRAIN + 1, READY = FULL + NST, EMPTY = READY + NST,
                         NBAR = EMPTY + NST;
    static constexpr int END = BAR + NBAR * 8 + 16;
    static constexpr int SMEM = END + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(sizeof(Item) % 16 == 0 && BAR % 8 == 0, "alignment");
};

struct Maps {
    CUtensorMap Q, K, V;
};

template <int NR>
__device__ __forceinline__ void make_item(const Args& a, int idx, Item& w) {
    w.part = idx % a.nsplit;
    int x = idx / a.nsplit;
    const int BH = a.B * a.Hk, qt = a.ntile - 1 - x / BH;
    x %= BH;
    w.hk = x % a.Hk;
    w.b = x / a.Hk;
    w.first = a.first(w.b);
    w.i0 = qt * NR * a.nq;
    int lo[NR], hi[NR], vlo = 0, vhi = -1;
#pragma unroll
    for (int t = 0; t < NR; ++t) {
        const int i = w.i0 + t * a.nq;
        lo[t] = 0;
        hi[t] = -1;
        if (i < a.Lq) tile_keys(a, w.b, i, min(i + a.nq, a.Lq) - 1, lo[t], hi[t]);
        if (hi[t] >= lo[t]) {
            vlo = vhi < vlo ? lo[t] : min(vlo, lo[t]);
            vhi = max(vhi, hi[t]);
        }
    }
    w.vlo = w.jlo = vlo;
    w.vhi = vhi;
    const int n = (vhi - vlo + 64) / 64;  // 0 when empty
    w.c0 = (int)((long long)n * w.part / a.nsplit);
    w.c1 = (int)((long long)n * (w.part + 1) / a.nsplit);
#pragma unroll
    for (int t = 0; t < NR; ++t) {
        w.s0[t] = w.s1[t] = w.c0;
        if (hi[t] >= lo[t]) {
            w.s0[t] = max(w.c0, (lo[t] - vlo) / 64);
            w.s1[t] = min(w.c1, (hi[t] - vlo) / 64 + 1);
        }
    }
}

template <int NR>
__global__ void __launch_bounds__(THREADS, 1) tc_fwd(const Args a, const __grid_constant__ Maps maps, int nitems) {
    using Y = Lay<NR>;
    constexpr int KS = Y::KS, NST = Y::NST;
    extern __shared__ uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Y::BAR);
    uint32_t* tbase = reinterpret_cast<uint32_t*>(sm + Y::BAR + Y::NBAR * 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tbase + 1);
    uint32_t* words = reinterpret_cast<uint32_t*>(sm + Y::WORDS);
    Item* items = reinterpret_cast<Item*>(sm + Y::ITEM);
    Ctl ctl{bar, abort_flag, a.status};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar + Y::QFULL + i, 1);
            tc::mbar_init(bar + Y::QEMPTY + i, 2);
        }
        for (int i = 0; i < NIT; ++i) {
            tc::mbar_init(bar + Y::IFULL + i, 1);
            tc::mbar_init(bar + Y::IEMPTY + i, 19);  // every warp but the loader
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(bar + Y::SFULL + i, 1);
            tc::mbar_init(bar + Y::PFULL + i, 4);
            tc::mbar_init(bar + Y::OFULL + i, 1);
        }
        for (int i = 0; i < NR; ++i) {
            tc::mbar_init(bar + Y::MFULL + i, KS > 1 ? 4 * (KS - 1) : 1);
            tc::mbar_init(bar + Y::MEMPTY + i, 4);
        }
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bar + Y::FULL + s, 1);
            tc::mbar_init(bar + Y::READY + s, 1);
            tc::mbar_init(bar + Y::EMPTY + s, 2);
        }
        tc::mbar_init(bar + Y::DRAIN, 2);
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
    // TMEM columns of group x = t * KS + ks: S (and P, 64 bf16 per row) at 64 x, O at 256 + 64 x
    const uint32_t tm = *tbase, tS = tm, tO = tm + 256;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;

    // An item's slot is read in place and handed back to the loader at the item's
    // end.  (Nothing of it is indexed by a runtime value in registers: local memory
    // would go to L2, as the shared memory leaves no L1 to speak of.  ptxas spills one
    // register of a thread all the same.)
    auto begin_item = [&](int it) -> bool {
        return ctl.wait_warp(Y::IFULL + it % NIT, (it / NIT) & 1) && items[it % NIT].b >= 0;
    };
    auto end_item = [&](int it) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + Y::IEMPTY + it % NIT);
    };

    if (warp >= 16) {
        reg_dec<REG_OTHER>();
        if (warp == W_LOAD) {
            // -------------------------------------------------------- loader (one lane)
            if (lane == 0) {
                Walk walk(nitems);
                int idx, nq = 0, gc = 0;
                bool ok = true;
                for (int it = 0; ok; ++it) {
                    const int e = it % NIT;
                    if (it >= NIT && !ctl.wait(Y::IEMPTY + e, ((it / NIT) - 1) & 1)) break;
                    const bool more = walk.next(idx);
                    Item& w = items[e];
                    if (more) make_item<NR>(a, idx, w);
                    else w.b = -1;
                    tc::mbar_arrive(bar + Y::IFULL + e);
                    if (!more) break;
                    const int qb = nq & 1;
                    if (nq >= 2 && !ctl.wait(Y::QEMPTY + qb, ((nq >> 1) - 1) & 1)) break;
                    tc::mbar_expect_tx(bar + Y::QFULL + qb, (uint32_t)(NR * a.nq * a.G) * 128u);
                    for (int t = 0; t < NR; ++t)
                        tma_load_4d(sm + Y::Q + (NR * qb + t) * TILE, &maps.Q, bar + Y::QFULL + qb, w.i0 + t * a.nq,
                                    w.hk * a.G, w.b);
                    ++nq;
                    const int jlo = w.jlo, hk = w.hk, b = w.b, c1 = w.c1;
                    for (int c = w.c0; c < c1; ++c, ++gc) {
                        const int s = gc % NST;
                        if (gc >= NST && !ctl.wait(Y::EMPTY + s, ((gc / NST) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        uint8_t* st = sm + Y::ST + s * 2 * KT;
                        tc::mbar_expect_tx(bar + Y::FULL + s, 2 * KT);
                        tma_load_4d(st, &maps.K, bar + Y::FULL + s, jlo + 64 * c, hk, b);
                        tma_load_4d(st + KT, &maps.V, bar + Y::FULL + s, jlo + 64 * c, hk, b);
                    }
                }
                // the last loads have landed before the block ends, whatever the others do
                for (int x = max(0, nq - 2); x < nq; ++x)
                    tc::mbar_wait(bar + Y::QFULL + (x & 1), (x >> 1) & 1, kWaitBudget);
                for (int x = max(0, gc - NST); x < gc; ++x)
                    tc::mbar_wait(bar + Y::FULL + x % NST, (x / NST) & 1, kWaitBudget);
            }
            __syncwarp();
        } else if (warp == W_MASK) {
            // -------------------------------------------------------- mask words, unused rows of V
            int gc = 0;
            bool ok = true;
            for (int it = 0; ok && begin_item(it); ++it) {
                const Item& w = items[it % NIT];
                for (int c = w.c0; c < w.c1; ++c, ++gc) {
                    const int s = gc % NST, j0 = w.jlo + 64 * c;
                    uint32_t bits[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = j0 + 32 * k + lane;
                        bits[k] = __ballot_sync(~0u, j >= w.vlo && j <= w.vhi && a.live(w.b, j));
                    }
                    if (!ctl.wait_warp(Y::FULL + s, (gc / NST) & 1)) {
                        ok = false;
                        break;
                    }
                    if (lane < 2) words[2 * s + lane] = lane ? bits[1] : bits[0];
                    if ((bits[0] & bits[1]) != ~0u) {
                        uint8_t* v = sm + Y::ST + s * 2 * KT + KT;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int e = 0; e < 8; ++e)  // four rows at a time, eight lanes of 16 bytes each
                                if (!((bits[k] >> (4 * e + (lane >> 3))) & 1u))
                                    *reinterpret_cast<uint4*>(v + (32 * k + 4 * e + (lane >> 3)) * 128 + (lane & 7) * 16) =
                                        make_uint4(0, 0, 0, 0);
                        tc::fence_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar + Y::READY + s);
                }
                end_item(it);
            }
        } else {
            // -------------------------------------------------------- S = Q K^T, O += P V
            // One lane issues both of a group, the P V of a chunk directly before the
            // S of the group's next chunk, which overwrites P: MMAs of one thread
            // execute in order, so neither waits for the other.  Two warps, as eight
            // MMAs and their hand-over take one warp longer than the exponentials.
            const int half = warp - W_MMA;
            const uint32_t id_s = tc::idesc_bf16(128, 64, false, false);
            const uint32_t id_o = tc::idesc_bf16(128, 64, false, true);
            const uint64_t dQ = tc::sdesc_sw128(tc::smem_u32(sm + Y::Q), 16, 1024);
            const uint64_t dK = tc::sdesc_sw128(tc::smem_u32(sm + Y::ST), 16, 1024);
            const uint64_t dV = tc::sdesc_sw128(tc::smem_u32(sm + Y::ST + KT), KT, 1024);
            int gc = 0;
            uint32_t n = 0;  // phases of the four P barriers
            bool ok = true;
            for (int it = 0; ok && begin_item(it); ++it) {
                const Item& w = items[it % NIT];
                const int qb = it & 1, c0 = w.c0, c1 = w.c1, g0 = gc - c0;
                int s0[NR], s1[NR];
#pragma unroll
                for (int t = 0; t < NR; ++t) {
                    s0[t] = w.s0[t];
                    s1[t] = w.s1[t];
                }
                if (!ctl.wait_warp(Y::QFULL + qb, it >> 1 & 1)) break;
                for (int c = c0 - KS; ok && c < c1; ++c) {
                    const int cn = c + KS, ks = cn % KS;  // the chunk whose S is formed
                    const int s = (g0 + c + NST) % NST, sn = (g0 + cn) % NST;
                    if (cn < c1 && !ctl.wait_warp(Y::READY + sn, ((g0 + cn) / NST) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint64_t dBv = tc::sdesc_add(dV, s * 2 * KT), dBk = tc::sdesc_add(dK, sn * 2 * KT);
#pragma unroll
                    for (int t = 0; t < NR; ++t) {
                        const int x = t * KS + ks;
                        if ((x >> 1) != half) continue;
                        const bool pv = c >= s0[t] && c < s1[t], sc = cn >= s0[t] && cn < s1[t];
                        if (pv) {
                            if (!ctl.wait_warp(Y::PFULL + x, (n >> x) & 1)) {
                                ok = false;
                                break;
                            }
                            n ^= 1u << x;
                        }
                        tc::tc_fence_after();
                        if (tc::elect_one()) {
                            if (pv) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tc::mma_bf16_ts(tO + 64 * x, tS + 64 * x + 8 * k, tc::sdesc_add(dBv, k * 2048), id_o,
                                                    (c - KS >= s0[t] || k > 0) ? 1u : 0u);
                                if (!sc) tc::tc_commit(bar + Y::OFULL + x);  // the group's last
                            }
                            if (sc) {
                                const uint64_t dA = tc::sdesc_add(dQ, (NR * qb + t) * TILE);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tc::mma_bf16(tS + 64 * x, tc::sdesc_add(dA, 32 * k), tc::sdesc_add(dBk, 32 * k), id_s,
                                                 k > 0);
                                tc::tc_commit(bar + Y::SFULL + x);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (c >= c0 && tc::elect_one()) tc::tc_commit(bar + Y::EMPTY + s);
                    __syncwarp();
                }
                if (!ok) break;
                gc += c1 - c0;
                if (tc::elect_one()) tc::tc_commit(bar + Y::QEMPTY + qb);
                end_item(it);
            }
            if (tc::elect_one()) tc::tc_commit(bar + Y::DRAIN);
            __syncwarp();
            tc::mbar_wait(bar + Y::DRAIN, 0, kWaitBudget);
        }
    } else {
        // ------------------------------------------------------------ softmax rows
        reg_inc<REG_SOFTMAX>();
        const int x = warp >> 2, qd = warp & 3, t = x / KS, ks = x % KS;
        const int r = qd * 32 + lane;  // row of the tile
        const int g = r / a.nq, iq = r % a.nq;
        const uint32_t lanebase = (uint32_t)(qd * 32) << 16;
        const uint32_t mS = tS + 64 * x + lanebase, mO = tO + 64 * x + lanebase;
        const uint64_t c2p = tc::pk2(a.c2, a.c2);
        float2* mls = reinterpret_cast<float2*>(sm + Y::ML) + (t * (KS - 1)) * 128 + r;
        int gc = 0;
        uint32_t n = 0, no = 0;  // chunks, and items with any
        bool ok = true, lent = false;  // lent: O is being read by the group that joins
        for (int it = 0; ok && begin_item(it); ++it) {
            const Item& w = items[it % NIT];
            // this row's keys, relative to the item's first chunk
            int lo = 0, hi = -1;
            {
                const int i = w.i0 + t * a.nq + iq;
                const long long p = w.first + i;
                if (g < a.G && i < a.Lq && p >= 0 && p < a.Lk && a.live(w.b, (int)p)) {
                    a.keys(p, lo, hi);
                    lo -= w.jlo;
                    hi -= w.jlo;
                }
            }
            const bool dead = __all_sync(~0u, hi < lo);  // no row of this warp attends anything
            // keys that every row of the warp attends, masks aside
            const int whi = __reduce_min_sync(~0u, hi);
            int wlo = __reduce_max_sync(~0u, lo);  // (kBig: see below)
            float m = -INFINITY;  // running maximum (log2 units), moved in steps of more than 8
            uint64_t l2[2] = {0, 0};
            bool some = false, used = false;
            const int g0 = gc - w.c0, c1 = w.s1[t];  // chunk c is the block's chunk g0 + c
            for (int c = w.s0[t] + (ks + 4 - w.s0[t] % KS) % KS; c < c1; c += KS) {
                const int s = (g0 + c) % NST;
                // (the words are written for a mask alone)
                if ((a.mask && !ctl.wait_warp(Y::READY + s, ((g0 + c) / NST) & 1)) ||
                    !ctl.wait_warp(Y::SFULL + x, n & 1)) {
                    ok = false;
                    break;
                }
                ++n;
                used = true;
                tc::tc_fence_after();
                if (!dead) {  // a dead warp's rows of P and O are never read
                    // Scores are read twice, 32 at a time, first for the maximum: held all
                    // at once they would not fit the registers of sixteen warps.
                    const int j0 = 64 * c;
                    uint32_t on[2] = {~0u, ~0u};
                    if (a.mask) {
                        const uint2 wd = *reinterpret_cast<const uint2*>(words + 2 * s);
                        on[0] = wd.x;
                        on[1] = wd.y;
                    }
                    const bool live[2] = {on[0] == ~0u, on[1] == ~0u};
                    bool full = j0 >= wlo && j0 + 63 <= whi && live[0] && live[1];
                    if (!full) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) on[k] &= range_bits(lo - j0 - 32 * k, hi - j0 - 32 * k);
                    }
                    uint32_t sv[32];
                    auto load = [&](int k) {
                        tc::tmem_ld32(mS + 32 * k, sv);
                        tc::tmem_wait_ld();
                        if (!full) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((on[k] >> j) & 1u)) sv[j] = 0xff800000u;  // -inf
                        }
                    };
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        load(k);
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float& y = top[(j >> 1) & 3];
                            y = max_nan(y, __uint_as_float(sv[j]), __uint_as_float(sv[j + 1]));
                        }
                    }
                    const float mx = max_nan(max_nan(top[0], top[1], top[2]), top[3], top[3]) * a.c2;
                    const bool move = mx > m + 8.f || (m == -INFINITY && mx > -INFINITY);
                    if (__any_sync(~0u, move)) {
                        const float f = move ? ex2(m - mx) : 1.f;  // 0 from an empty row
                        if (move) m = mx;
                        if (__any_sync(~0u, fabsf(m) >= kRound && fabsf(m) < INFINITY)) {
                            wlo = kBig;  // no word is taken as a whole from here on
                            full = false;
                        }
                        float y, z;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            tc::upk2(l2[e], y, z);
                            l2[e] = tc::pk2(y * f, z * f);
                        }
                        if (some) {  // the last P V was issued before this S: it has added to O
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t o[16];
                                tc::tmem_ld16(mO + 16 * e, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tc::tmem_st16(mO + 16 * e, o);
                            }
                        }
                    }
                    if (!(mx < INFINITY)) {  // NaN or +inf among the scores: so is the row
                        l2[0] = tc::pk2(NAN, NAN);
                        if (!(fabsf(m) < INFINITY)) m = 0.f;
                    }
                    const float use = m == -INFINITY ? 0.f : -m;
                    const uint64_t mp = tc::pk2(use, use);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t pw[16];
                        load(k);
                        // a word of 32 columns is in use for all rows, for none, or for some
                        const bool all =
                            full || (live[k] && j0 + 32 * k >= wlo && j0 + 32 * k + 31 <= whi);
                        if (all) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint64_t y = tc::fma2(
                                    tc::pk2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), c2p, mp);
                                float e0, e1;
                                if (j % 4 == 3) {
                                    exp2_poly2(y, e0, e1);
                                } else {
                                    tc::upk2(y, e0, e1);
                                    e0 = ex2(e0);
                                    e1 = ex2(e1);
                                }
                                l2[j & 1] = tc::add2(l2[j & 1], tc::pk2(e0, e1));
                                pw[j] = tc::pack_bf16(e0, e1);
                            }
                        } else if (wlo == kBig) {
                            const bool round = fabsf(use) >= kRound;
                            const float pre = round ? a.c2 : 1.f, post = round ? 1.f : a.c2;
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float e0 = ex2(fmaf(__uint_as_float(sv[2 * j]) * pre, post, use));
                                const float e1 = ex2(fmaf(__uint_as_float(sv[2 * j + 1]) * pre, post, use));
                                l2[j & 1] = tc::add2(l2[j & 1], tc::pk2(e0, e1));
                                pw[j] = tc::pack_bf16(e0, e1);
                            }
                        } else if (__any_sync(~0u, on[k] != 0u)) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint64_t y = tc::fma2(
                                    tc::pk2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), c2p, mp);
                                float e0, e1;
                                tc::upk2(y, e0, e1);
                                e0 = ex2(e0);
                                e1 = ex2(e1);
                                l2[j & 1] = tc::add2(l2[j & 1], tc::pk2(e0, e1));
                                pw[j] = tc::pack_bf16(e0, e1);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) pw[j] = 0u;
                        }
                        tc::tmem_st16(mS + 16 * k, pw);
                    }
                    tc::tmem_wait_st();
                    some = true;
                }
                // the joining group has read this group's O of the item before
                if (lent && !ctl.wait_warp(Y::MEMPTY + t, (it - 1) & 1)) {
                    ok = false;
                    break;
                }
                lent = false;
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + Y::PFULL + x);
            }
            if (!ok) break;
            gc += w.c1 - w.c0;
            float l;
            {
                float x0, x1, x2, x3;
                tc::upk2(l2[0], x0, x1);
                tc::upk2(l2[1], x2, x3);
                l = (x0 + x1) + (x2 + x3);
            }
            if (used) {
                if (!ctl.wait_warp(Y::OFULL + x, no & 1)) break;
                ++no;
            }
            tc::tc_fence_after();
            if (KS > 1 && ks > 0) {  // hand O, the maximum and the sum to the group of subset 0
                if (lent && !ctl.wait_warp(Y::MEMPTY + t, (it - 1) & 1)) break;
                mls[(ks - 1) * 128] = make_float2(m, l);
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + Y::MFULL + t);
                lent = true;
                end_item(it);
                continue;
            }
            float f = 1.f;                    // weights of the subsets' O
            float fs[KS > 1 ? KS - 1 : 1];
            if (KS > 1) {
                if (!ctl.wait_warp(Y::MFULL + t, it & 1)) break;
                tc::tc_fence_after();
                float mm = m, ms[KS > 1 ? KS - 1 : 1], ls[KS > 1 ? KS - 1 : 1];
#pragma unroll
                for (int e = 0; e < KS - 1; ++e) {
                    const float2 y = mls[e * 128];
                    ms[e] = y.x;
                    ls[e] = y.y;
                    mm = fmaxf(mm, y.x);
                }
                const float use = mm == -INFINITY ? 0.f : mm;
                f = ex2(m - use);
                l = m == -INFINITY ? 0.f : l * f;
#pragma unroll
                for (int e = 0; e < KS - 1; ++e) {
                    fs[e] = ex2(ms[e] - use);
                    if (ms[e] != -INFINITY) l = fmaf(ls[e], fs[e], l);
                }
                m = mm;
            }
            const bool none = m == -INFINITY;  // nothing attended
            const bool parts = a.nparts > 1;
            const float inv = parts ? 1.f : none ? 0.f : 1.f / l;
            const int i = w.i0 + t * a.nq + iq;
            const bool row = g < a.G && i < a.Lq;
            const long long at = ((long long)w.b * a.Hq + w.hk * a.G + g) * a.Lq + i;
            const long long pa = at * a.nparts + w.part;
            if (row) {
                if (parts) a.part_ml[pa] = make_float2(m, l);
                else a.u[at] = none ? 0.f : -(m + lg2(l)) * kLn2;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t o[16];
                tc::tmem_ld16(mO + 16 * k, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    // without a chunk, or for a row that attends none, O holds anything
                    const float y = f * inv * __uint_as_float(o[j]);
                    o[j] = some && f > 0.f ? __float_as_uint(y) : 0u;
                }
                if (KS > 1) {
#pragma unroll
                    for (int e = 0; e < KS - 1; ++e) {
                        uint32_t o2[16];
                        tc::tmem_ld16(mO + 64 * (e + 1) + 16 * k, o2);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (fs[e] > 0.f)
                                o[j] = __float_as_uint(fmaf(fs[e] * inv, __uint_as_float(o2[j]), __uint_as_float(o[j])));
                    }
                }
                if (row && parts && !none) {
                    float4* po = reinterpret_cast<float4*>(a.part_o + pa * 64 + 16 * k);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        po[j] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                            __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
                } else if (row && !parts) {
                    uint4* out = reinterpret_cast<uint4*>(a.o.at<__nv_bfloat16>(w.b, w.hk * a.G + g, i) + 16 * k);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = tc::pack_bf16(__uint_as_float(o[8 * j + 2 * e]), __uint_as_float(o[8 * j + 2 * e + 1]));
                        out[j] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                __syncwarp();
            }
            if (KS > 1) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + Y::MEMPTY + t);
            }
            end_item(it);
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
