// The softmax attention's backward for bf16 storage on the tensor cores.
//
// Two sweeps, so that every gradient is summed in one place and in one order:
//   DQ    rows: 128 packed query rows;  chunks: 64 keys
//         S = Q K^T, G = dO V^T, dS = P (G - D),  dQ += dS K, X += P K
//   DKV   rows: 128 keys;  chunks: 64 queries of one head after another
//         S^T = K Q^T, G^T = V dO^T,  dV += P^T dO,  dK += dS^T Q
// with P = 2^(c2 S + u2).  (One sweep that also added into dQ would save two of
// the products but needs atomics, whose order changes results.)
//
// D = dO . O from the rounded O lacks r, |r| up to 2^-8 |D|: where few keys hold a
// row's weight as much as the dS it is subtracted in.  As the rows of P sum to 1,
// r is the sum of dS; it is summed in DQ beside the products, dQ is set right by
// r X at the item's end, and DKV takes D + r.
//
// A unit is one row tile times one chunk.  S and G of a unit go to one of three
// slots of TMEM; a team of eight warps (two per lane quadrant, 32 columns each)
// reads them, forms P and dS and writes them as bf16 over the S and G they came
// from, 16 columns at a time (32 at once spilled: 0.55 ms for 0.48 at 32768 tokens
// of 16 heads, W = 256), from where the second products read them as their A
// operand.  Two teams take the units in turn; in DQ they ask for their rows of the
// next item while one ends (0.53 -> 0.51 ms), in DKV one writes an item's gradients
// while the other begins the next (0.51 -> 0.49 ms; DQ's teams form D together, and
// apart took longer).  One warp issues S and G, another the second products (one
// thread for all that add into an accumulator); a loader brings the tiles, and an
// aux warp prepares each chunk's columns (mask words; zeroed operand rows of tokens
// that are not in use, as 0 times what they hold need not be 0).  In DKV u and D
// belong to columns: they enter S and G in the products themselves, as 16 more
// channels, u / c and -D in three bf16 parts each (2^-24 of them) against ones
// (read by every thread from shared memory they cost the teams twice the time).
// dO . O is formed by the teams' warps at an item's start, a quarter of the channels
// each.
//
// P and dS are rounded to bf16 for the second products (their other operands are
// bf16; see softmax_tc.cuh); u, D, the sum of dS and all accumulators are fp32.  Gradients
// are off by 2.4e-3 of their norm against 64 bits, 1.7e-3 of it their own rounding.
//
// 8192 dense tokens of 8 heads take 661 us for the eight products, 0.51 of the
// matrix rate.  A banded item is bound by its start and its end, where the products
// drain, a long one by the hand-overs.  (The row tiles' operands in TMEM as well
// made the MMAs shorter but left five buffers of S or G in DKV: 3 % slower.)
#pragma once

#include "softmax_tc.cuh"

namespace sa {
namespace sm {
namespace tcf {
namespace bwd {

enum { DQ = 0, DKV = 1 };
constexpr int THREADS = 640;
constexpr int W_LOAD = 16, W_AUX = 17, W_SG = 18, W_AC = 19;
constexpr int REG_TEAM = 104, REG_OTHER = 64;  // launched with 96 x 640 = 61440
static_assert(512 * REG_TEAM + 128 * REG_OTHER <= 61440, "register split");
constexpr int KT = TILE / 2;
constexpr int NST = 7, NIT = 4, NSLOT = 3;

struct Item {
    int b, hk, r0, n, c0, vlo, vhi, pad;  // b < 0: no more; r0: first query or key; c0: column of chunk 0
    // columns vlo .. vhi (absolute) are in some row's band; n chunks per head
    long long first;
};

constexpr int OFF_R = 0;                        // two buffers of two row tiles
constexpr int OFF_ST = OFF_R + 4 * TILE;        // stages of two chunk tiles
constexpr int AUG = 64 * 32;                    // DKV: a chunk's columns as 16 more channels
constexpr int OFF_AUG = OFF_ST + NST * 2 * KT;  // one per stage
constexpr int OFF_ONE = OFF_AUG + NST * AUG;    // and the rows' side, 128 x 32 bytes for S, for G
constexpr int OFF_ITEM = OFF_ONE + 2 * 4096;
constexpr int OFF_XD = OFF_ITEM + NIT * (int)sizeof(Item);  // two buffers of shares of D, [4][128]
constexpr int OFF_WORDS = OFF_XD + 4096;
constexpr int OFF_BAR = OFF_WORDS + NST * 8;
enum { RFULL = 0, REMPTY = 2, IFULL = 4, IEMPTY = IFULL + NIT, SGFULL = IEMPTY + NIT, DSFULL = SGFULL + NSLOT, SLOT = DSFULL + NSLOT, ACCFULL = SLOT + NSLOT,
       ACCEMPTY = ACCFULL + 2, XDSUM = ACCEMPTY + 1, DRAIN = XDSUM + 1, FULL = DRAIN + 1, READY = FULL + NST,
       EMPTY = READY + NST, NBAR = EMPTY + NST };
constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
static_assert(SMEM <= 227 * 1024, "shared memory");
static_assert(sizeof(Item) % 8 == 0 && OFF_BAR % 8 == 0, "alignment");

struct Maps {
    CUtensorMap R1, R2, C1, C2;  // DQ: Q, dO, K, V;  DKV: K, V, Q, dO
    CUtensorMap X;               // DKV: the queries' 16 further channels
};

// Byte offset of 16-byte piece c (0, 1) of row r in a tile of 32-byte rows, 32-byte swizzle.
__device__ __forceinline__ uint32_t aug_off(int r, int c) { return r * 32 + ((c ^ ((r >> 2) & 1)) << 4); }
// x as hi + mid + lo, the bits of three bf16 numbers.
__device__ __forceinline__ void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    const float y = x - __bfloat162float(h);
    const __nv_bfloat16 m = __float2bfloat16_rn(y);
    const __nv_bfloat16 l = __float2bfloat16_rn(y - __bfloat162float(m));
    hi = __bfloat16_as_ushort(h);
    mid = __bfloat16_as_ushort(m);
    lo = __bfloat16_as_ushort(l);
}

template <int MODE>
__device__ __forceinline__ void make_item(const Args& a, int idx, Item& w) {
    const int BH = a.B * a.Hk, x = idx % BH, rt = idx / BH;
    w.hk = x % a.Hk;
    w.b = x / a.Hk;
    w.first = a.first(w.b);
    int lo = 0, hi = -1;
    if (MODE == DQ) {  // the later the query, the more keys a causal band holds
        w.r0 = (a.ntile - 1 - rt) * a.nq;
        tile_keys(a, w.b, w.r0, min(w.r0 + a.nq, a.Lq) - 1, lo, hi);
    } else {  // queries whose position lies in [k0 - R, k1 + W], and in the span
        w.r0 = rt * 128;
        const int2 s = span(a, w.b);
        const int k0 = max(w.r0, s.x), k1 = min(w.r0 + 127, s.y);
        long long p0 = (long long)k0 - a.R, p1 = (long long)k1 + a.W;
        p0 = p0 > s.x ? p0 : s.x;
        p1 = k1 < k0 ? -1 : p1 < s.y ? p1 : s.y;
        p0 -= w.first;
        p1 -= w.first;
        if (p0 < 0) p0 = 0;
        if (p1 > a.Lq - 1) p1 = a.Lq - 1;
        if (p0 <= p1) {
            lo = (int)p0;
            hi = (int)p1;
        }
    }
    w.c0 = w.vlo = lo;
    w.vhi = hi;
    w.n = (hi - lo + 64) / 64;  // 0 when empty
}

template <int MODE>
__global__ void __launch_bounds__(THREADS, 1) tc_bwd(const Args a, const __grid_constant__ Maps maps, int nitems) {
    extern __shared__ uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tbase = reinterpret_cast<uint32_t*>(sm + OFF_BAR + NBAR * 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tbase + 1);
    uint32_t* words = reinterpret_cast<uint32_t*>(sm + OFF_WORDS);
    Item* items = reinterpret_cast<Item*>(sm + OFF_ITEM);
    float* xd = reinterpret_cast<float*>(sm + OFF_XD);
    Ctl ctl{bar, abort_flag, a.status};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar + RFULL + i, 1);
            tc::mbar_init(bar + REMPTY + i, MODE == DQ ? 17 : 1);  // the MMAs, and the warps that read dO
            tc::mbar_init(bar + ACCFULL + i, 1);
        }
        for (int i = 0; i < NIT; ++i) {
            tc::mbar_init(bar + IFULL + i, 1);
            tc::mbar_init(bar + IEMPTY + i, 19);  // every warp but the loader
        }
        for (int i = 0; i < NSLOT; ++i) {
            tc::mbar_init(bar + SGFULL + i, 1);
            tc::mbar_init(bar + DSFULL + i, 8);
            tc::mbar_init(bar + SLOT + i, 1);
        }
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bar + FULL + s, 1);
            tc::mbar_init(bar + READY + s, 1);
            tc::mbar_init(bar + EMPTY + s, 1);
        }
        tc::mbar_init(bar + ACCEMPTY, MODE == DQ ? 16 : 8);
        tc::mbar_init(bar + XDSUM, 16);
        tc::mbar_init(bar + DRAIN, 2);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (MODE == DKV) {  // the constant rows: 1 in slots 0-2 (S) or 3-5 (G) of 16
        for (int x = threadIdx.x; x < 512; x += THREADS) {
            const int r = x & 127, c = (x >> 7) & 1, t = x >> 8;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (c == 0) w = t == 0 ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0x3f800000u, 0x3f803f80u, 0u);
            *reinterpret_cast<uint4*>(sm + OFF_ONE + t * 4096 + aug_off(r, c)) = w;
        }
        tc::fence_async_smem();
    }
    if (warp == 0) {
        tc::tmem_alloc(tbase, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    // TMEM columns: slot x: S at 128 x, G at 128 x + 64; accumulators from 384
    const uint32_t tm = *tbase, tA = tm + 384;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (MODE == DQ && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;

    auto begin_item = [&](int it) -> bool {
        return ctl.wait_warp(IFULL + it % NIT, (it / NIT) & 1) && items[it % NIT].b >= 0;
    };
    auto end_item = [&](int it) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + IEMPTY + it % NIT);
    };
    // units of an item: its chunks, for each head of the group in DKV
    const int passes = MODE == DKV ? a.G : 1;

    if (warp >= 16) {
        reg_dec<REG_OTHER>();
        if (warp == W_LOAD) {
            // -------------------------------------------------------- loader (one lane)
            if (lane == 0) {
                Walk walk(nitems);
                int idx, nr = 0, gu = 0;
                bool ok = true;
                for (int it = 0; ok; ++it) {
                    const int e = it % NIT;
                    if (it >= NIT && !ctl.wait(IEMPTY + e, ((it / NIT) - 1) & 1)) break;
                    const bool more = walk.next(idx);
                    Item& w = items[e];
                    if (more) make_item<MODE>(a, idx, w);
                    else w.b = -1;
                    tc::mbar_arrive(bar + IFULL + e);
                    if (!more) break;
                    const int rb = nr & 1, n = w.n, hk = w.hk, b = w.b, c0 = w.c0, r0 = w.r0;
                    if (nr >= 2 && !ctl.wait(REMPTY + rb, ((nr >> 1) - 1) & 1)) break;
                    const int h0 = MODE == DQ ? hk * a.G : hk;
                    tc::mbar_expect_tx(bar + RFULL + rb, MODE == DQ ? (uint32_t)(2 * a.nq * a.G) * 128u : 2u * TILE);
                    tma_load_4d(sm + OFF_R + 2 * rb * TILE, &maps.R1, bar + RFULL + rb, r0, h0, b);
                    tma_load_4d(sm + OFF_R + (2 * rb + 1) * TILE, &maps.R2, bar + RFULL + rb, r0, h0, b);
                    ++nr;
                    for (int p = 0; ok && p < passes; ++p) {
                        const int h = MODE == DQ ? hk : hk * a.G + p;
                        for (int c = 0; c < n; ++c, ++gu) {
                            const int s = gu % NST;
                            if (gu >= NST && !ctl.wait(EMPTY + s, ((gu / NST) - 1) & 1)) {
                                ok = false;
                                break;
                            }
                            uint8_t* st = sm + OFF_ST + s * 2 * KT;
                            tc::mbar_expect_tx(bar + FULL + s, 2 * KT + (MODE == DKV ? AUG : 0));
                            if (MODE == DKV)
                                tc::tma_load_3d(sm + OFF_AUG + s * AUG, &maps.X, bar + FULL + s, 0, c0 + 64 * c, b * a.Hq + h);
                            tma_load_4d(st, &maps.C1, bar + FULL + s, c0 + 64 * c, h, b);
                            tma_load_4d(st + KT, &maps.C2, bar + FULL + s, c0 + 64 * c, h, b);
                        }
                    }
                }
                // the last loads have landed before the block ends, whatever the others do
                for (int x = max(0, nr - 2); x < nr; ++x)
                    tc::mbar_wait(bar + RFULL + (x & 1), (x >> 1) & 1, kWaitBudget);
                for (int x = max(0, gu - NST); x < gu; ++x)
                    tc::mbar_wait(bar + FULL + x % NST, (x / NST) & 1, kWaitBudget);
            }
            __syncwarp();
        } else if (warp == W_AUX) {
            // -------------------------------------------------------- columns
            int gu = 0;
            bool ok = true;
            for (int it = 0; ok && begin_item(it); ++it) {
                const Item& w = items[it % NIT];
                const int n = w.n, last = w.vhi - w.c0;  // columns 0 .. last, from c0 on
                // mask of column 0
                const uint8_t* pm = a.mask ? a.mask + (long long)w.b * a.Lk + w.c0 + (MODE == DKV ? w.first : 0) : nullptr;
                uint32_t bits[2];
                auto fetch = [&](int c) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = 64 * c + 32 * k + lane;
                        bits[k] = __ballot_sync(~0u, j <= last && (pm == nullptr || pm[j] != 0));
                    }
                };
                if (n > 0) fetch(0);
                for (int p = 0; ok && p < passes; ++p) {
                    for (int c = 0; c < n; ++c, ++gu) {
                        const int s = gu % NST;
                        if (!ctl.wait_warp(FULL + s, (gu / NST) & 1)) {
                            ok = false;
                            break;
                        }
                        if (lane < 2) words[2 * s + lane] = lane ? bits[1] : bits[0];
                        if ((bits[0] & bits[1]) != ~0u) {
                            uint8_t* x = sm + OFF_ST + s * 2 * KT;
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int e = 0; e < 8; ++e)  // four rows at a time, eight lanes of 16 bytes each
                                    if (!((bits[k] >> (4 * e + (lane >> 3))) & 1u)) {
                                        uint4* q = reinterpret_cast<uint4*>(x + (32 * k + 4 * e + (lane >> 3)) * 128 +
                                                                            (lane & 7) * 16);
                                        q[0] = make_uint4(0, 0, 0, 0);
                                        if (MODE == DKV) q[KT / 16] = make_uint4(0, 0, 0, 0);
                                    }
                            tc::fence_async_smem();
                        }
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(bar + READY + s);
                        fetch(c + 1 < n ? c + 1 : 0);
                    }
                }
                end_item(it);
            }
        } else if (warp == W_SG) {
            // -------------------------------------------------------- S and G
            const uint32_t id = tc::idesc_bf16(128, 64, false, false);
            const uint64_t dR = tc::sdesc_sw128(tc::smem_u32(sm + OFF_R), 16, 1024);
            const uint64_t dC = tc::sdesc_sw128(tc::smem_u32(sm + OFF_ST), 16, 1024);
            const uint64_t dOne = tc::sdesc_sw32(tc::smem_u32(sm + OFF_ONE));
            const uint64_t dAug = tc::sdesc_sw32(tc::smem_u32(sm + OFF_AUG));
            int gu = 0;
            bool ok = true;
            for (int it = 0; ok && begin_item(it); ++it) {
                const int rb = it & 1, nu = items[it % NIT].n * passes;
                if (!ctl.wait_warp(RFULL + rb, (it >> 1) & 1)) break;
                const uint64_t dA = tc::sdesc_add(dR, 2 * rb * TILE);
                for (int u = 0; u < nu; ++u, ++gu) {
                    const int s = gu % NST, x = gu % NSLOT;
                    if (!ctl.wait_warp(READY + s, (gu / NST) & 1) ||
                        (gu >= NSLOT && !ctl.wait_warp(SLOT + x, ((gu / NSLOT) - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint64_t dB = tc::sdesc_add(dC, s * 2 * KT);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_bf16(tm + 128 * x, tc::sdesc_add(dA, 32 * k), tc::sdesc_add(dB, 32 * k), id, k > 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_bf16(tm + 128 * x + 64, tc::sdesc_add(dA, TILE + 32 * k),
                                         tc::sdesc_add(dB, KT + 32 * k), id, k > 0);
                        if (MODE == DKV) {  // S + u / c, G - D
                            tc::mma_bf16(tm + 128 * x, dOne, tc::sdesc_add(dAug, s * AUG), id, 1u);
                            tc::mma_bf16(tm + 128 * x + 64, tc::sdesc_add(dOne, 4096), tc::sdesc_add(dAug, s * AUG), id, 1u);
                        }
                        tc::tc_commit(bar + SGFULL + x);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (tc::elect_one()) tc::tc_commit(bar + REMPTY + rb);
                end_item(it);
            }
            if (tc::elect_one()) tc::tc_commit(bar + DRAIN);
            __syncwarp();
            tc::mbar_wait(bar + DRAIN, 0, kWaitBudget);
        } else {
            // -------------------------------------------------------- the second products
            const uint32_t id = tc::idesc_bf16(128, 64, false, true);
            const uint64_t dC = tc::sdesc_sw128(tc::smem_u32(sm + OFF_ST), KT, 1024);
            int gu = 0, na = 0;  // units, items with any
            bool ok = true;
            for (int it = 0; ok && begin_item(it); ++it) {
                const int nu = items[it % NIT].n * passes;
                for (int u = 0; u < nu; ++u, ++gu) {
                    const int s = gu % NST, x = gu % NSLOT;
                    if ((u == 0 && na > 0 && !ctl.wait_warp(ACCEMPTY, (na - 1) & 1)) ||
                        !ctl.wait_warp(DSFULL + x, (gu / NSLOT) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint64_t dB = tc::sdesc_add(dC, s * 2 * KT);
                    const uint32_t slot = tm + 128 * x;
                    if (tc::elect_one()) {
                        // 16 columns of the chunk are 8 of TMEM; each half of a
                        // slot's S (or G) keeps the columns it was formed from
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // P times K, dO
                            tc::mma_bf16_ts(tA, slot + 32 * (k >> 1) + 8 * (k & 1),
                                            tc::sdesc_add(dB, (MODE == DQ ? 0 : KT) + k * 2048), id,
                                            (u > 0 || k > 0) ? 1u : 0u);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // dS times K, Q
                            tc::mma_bf16_ts(tA + 64, slot + 64 + 32 * (k >> 1) + 8 * (k & 1),
                                            tc::sdesc_add(dB, k * 2048), id, (u > 0 || k > 0) ? 1u : 0u);
                        tc::tc_commit(bar + SLOT + x);
                        tc::tc_commit(bar + EMPTY + s);
                        if (u == nu - 1) tc::tc_commit(bar + ACCFULL + (MODE == DQ ? 0 : gu & 1));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (nu > 0) ++na;
                end_item(it);
            }
            if (tc::elect_one()) tc::tc_commit(bar + DRAIN);
            __syncwarp();
            tc::mbar_wait(bar + DRAIN, 0, kWaitBudget);
        }
    } else {
        // ------------------------------------------------------------ P and dS
        reg_inc<REG_TEAM>();
        const int qd = warp & 3, hf = (warp >> 2) & 1, team = warp >> 3, q4 = warp >> 2;
        const int r = qd * 32 + lane;
        const int g = MODE == DQ ? r / a.nq : 0, iq = MODE == DQ ? r % a.nq : r;
        const uint32_t lanebase = (uint32_t)(qd * 32) << 16;
        const uint64_t c2p = tc::pk2(a.c2, a.c2);
        const float uscale = 1.f / a.c;
        int gu = 0, na = 0, nx = 0;  // units, items whose accumulators this team read, sums of D
        bool ok = true;
        // The sum over the four warps that hold a row's columns.  Two buffers: to
        // reach the one after the next, every warp has read this one.
        auto put = [&](float x) {
            xd[(nx & 1) * 512 + q4 * 128 + r] = x;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar + XDSUM);
        };
        auto get = [&](float& total) -> bool {
            const float* sh = xd + (nx & 1) * 512;
            if (!ctl.wait_warp(XDSUM, nx & 1)) return false;
            ++nx;
            total = (sh[r] + sh[128 + r]) + (sh[256 + r] + sh[384 + r]);
            return true;
        };
        // DQ: u and O of this thread's row of an item, asked for while the item before ends.
        float un = 0.f;
        uint4 orow[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        bool in = false;
        auto ask = [&](const Item& w) {
            const int i = w.r0 + iq;
            const long long p = w.first + i;
            in = g < a.G && i < a.Lq && p >= 0 && p < a.Lk && a.live(w.b, (int)p);
            if (!in) return;
            const int h = w.hk * a.G + g;
            un = a.u[((long long)w.b * a.Hq + h) * a.Lq + i];
            const uint4* po = reinterpret_cast<const uint4*>(a.o.at<__nv_bfloat16>(w.b, h, i) + 16 * q4);
            orow[0] = po[0];
            orow[1] = po[1];
        };
        if (MODE == DQ && begin_item(0)) ask(items[0]);
        for (int it = 0; ok && begin_item(it); ++it) {
            const Item& w = items[it % NIT];
            const int rb = it & 1, n = w.n, nu = n * passes;
            // this row: its columns in the band, relative to chunk 0
            float ur = 0.f, D = 0.f;  // u in units of <q, k>, as the scores
            int lo = 0, hi = -1;
            const int i = w.r0 + iq;  // query or key
            const bool exists = MODE == DQ ? g < a.G && i < a.Lq : i < a.Lk;
            const long long at = MODE == DQ ? ((long long)w.b * a.Hq + w.hk * a.G + g) * a.Lq + i : 0;
            if (MODE == DQ) {
                if (in) {
                    a.keys(w.first + i, lo, hi);
                    lo -= w.c0;
                    hi -= w.c0;
                    ur = un * uscale;
                }
                if (!ctl.wait_warp(RFULL + rb, (it >> 1) & 1)) break;
                {  // dO . O, a quarter of the channels here
                    const uint8_t* dO = sm + OFF_R + (2 * rb + 1) * TILE;
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 y = *reinterpret_cast<const uint4*>(dO + tc::sw128_off(r, 2 * q4 + e));
                        const __nv_bfloat162* po = reinterpret_cast<const __nv_bfloat162*>(&orow[e]);
                        const __nv_bfloat162* py = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float2 f = __bfloat1622float2(po[z]), k = __bfloat1622float2(py[z]);
                            x = fmaf(f.x, k.x, fmaf(f.y, k.y, x));
                        }
                    }
                    put(in ? x : 0.f);
                    if (!get(D)) break;
                }
                if (lane == 0) tc::mbar_arrive(bar + REMPTY + rb);
            } else if (exists && a.live(w.b, i)) {
                // queries i - R .. i + W of the item's vlo .. vhi
                const long long l = (long long)i - a.R - w.first - w.c0, h = (long long)i + a.W - w.first - w.c0;
                const int last = w.vhi - w.c0;
                lo = (int)(l < 0 ? 0 : l > last ? last + 1 : l);
                hi = (int)(h < -1 ? -1 : h > last ? last : h);
            }
            // columns that every row of the warp attends, and any
            const int wlo = __reduce_max_sync(~0u, lo), whi = __reduce_min_sync(~0u, hi);
            const int alo = __reduce_min_sync(~0u, hi < lo ? 0x7fffffff : lo);
            const int ahi = __reduce_max_sync(~0u, hi < lo ? -1 : hi);
            // This team's units: every second one of the block's.  c: the unit's chunk.
            uint64_t sum2 = 0;  // DQ: of P (G - D), two columns apart
            int c = (gu ^ team) & 1;
            for (int u = c; u < nu; u += 2, c += 2) {
                while (c >= n) c -= n;
                const int gv0 = gu + u, s = gv0 % NST, x = gv0 % NSLOT;
                if ((a.mask && !ctl.wait_warp(READY + s, (gv0 / NST) & 1)) ||
                    !ctl.wait_warp(SGFULL + x, (gv0 / NSLOT) & 1)) {
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
                const uint32_t mS = tm + 128 * x + lanebase + 32 * hf, mG = mS + 64;
                const int j0 = 64 * c + 32 * hf;
                uint32_t on = a.mask ? words[2 * s + hf] : ~0u;
                const bool full = j0 >= wlo && j0 + 31 <= whi && on == ~0u;
                const bool any = j0 <= ahi && j0 + 31 >= alo;
                if (!any) {
                    const uint32_t zero[16] = {};
                    tc::tmem_st16(mS, zero);
                    tc::tmem_st16(mG, zero);
                } else {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {  // 16 columns at a time
                        uint32_t sv[16], gv[16], pw[8], dw[8];
                        tc::tmem_ld16(mS + 16 * z, sv);
                        tc::tmem_ld16(mG + 16 * z, gv);
                        tc::tmem_wait_ld();
                        if (!full) {
                            // scores of -inf give P = 0; G must be finite for dS = 0
                            const uint32_t m = on & range_bits(lo - j0, hi - j0);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (!((m >> (16 * z + j)) & 1u)) {
                                    sv[j] = 0xff800000u;
                                    gv[j] = 0u;
                                }
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint64_t x2 = tc::pk2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1]));
                            uint64_t d2 = tc::pk2(__uint_as_float(gv[2 * j]), __uint_as_float(gv[2 * j + 1]));
                            if (MODE == DQ) {  // in DKV the products have u and D in them
                                x2 = mul2(tc::add2(x2, tc::pk2(ur, ur)), c2p);
                                d2 = tc::sub2(d2, tc::pk2(D, D));
                            } else {
                                x2 = mul2(x2, c2p);
                            }
                            float e0, e1, d0, d1;
                            tc::upk2(x2, e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            d2 = mul2(d2, tc::pk2(e0, e1));
                            if (MODE == DQ) sum2 = tc::add2(sum2, d2);
                            tc::upk2(d2, d0, d1);
                            dw[j] = tc::pack_bf16(d0, d1);
                            pw[j] = tc::pack_bf16(e0, e1);
                        }
                        // over columns that this thread has read
                        tmem_st8(mS + 8 * z, pw);
                        tmem_st8(mG + 8 * z, dw);
                    }
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar + DSFULL + x);
            }
            if (!ok) break;
            gu += nu;
            float rest = 0.f;  // DQ: what D lacked
            if (MODE == DQ) {
                float x0, x1;
                tc::upk2(sum2, x0, x1);
                put(x0 + x1);
                if (begin_item(it + 1)) ask(items[(it + 1) % NIT]);
            }
            // The accumulators, this warp's lanes.  DQ: 16 columns.  DKV: 32 of each,
            // by the team that had the last unit; the other is at the next item.
            const bool mine = MODE == DQ || (((nu > 0 ? gu - 1 : 0) ^ team) & 1) == 0;
            if (nu > 0 && mine) {  // DKV: a barrier per team
                if (!ctl.wait_warp(ACCFULL + (MODE == DQ ? 0 : team), na & 1)) break;
                ++na;
                tc::tc_fence_after();
            }
            if (MODE == DQ) {
                if (!get(rest)) break;
                if (exists && q4 == 0) {  // for the key sweep: u / c and -D
                    uint32_t u0, u1, u2, d0, d1, d2;
                    split3(ur, u0, u1, u2);
                    split3(-(D + rest), d0, d1, d2);
                    a.aug[2 * at] = make_uint4(u0 | u1 << 16, u2 | d0 << 16, d1 | d2 << 16, 0u);
                    a.aug[2 * at + 1] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            if (mine) {
#pragma unroll
                for (int k = 0; k < (MODE == DQ ? 1 : 4); ++k) {
                    const int col = MODE == DQ ? 16 * q4 : 32 * hf + 16 * (k & 1);
                    uint32_t o[16], pk[MODE == DQ ? 16 : 1];
                    if (nu > 0) {
                        tc::tmem_ld16(tA + (MODE == DQ || k > 1 ? 64 : 0) + lanebase + col, o);
                        if constexpr (MODE == DQ) tc::tmem_ld16(tA + lanebase + col, pk);
                        tc::tmem_wait_ld();
                        if constexpr (MODE == DQ) {
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                o[j] = __float_as_uint(fmaf(-rest, __uint_as_float(pk[j]), __uint_as_float(o[j])));
                        }
                    }
                    const float f = MODE == DKV && k < 2 ? 1.f : a.c;
                    if (exists) {
                        uint4* p = reinterpret_cast<uint4*>(
                            (MODE == DQ ? a.dq.at<__nv_bfloat16>(w.b, w.hk * a.G + g, i)
                                        : (k < 2 ? a.dv : a.dk).at<__nv_bfloat16>(w.b, w.hk, i)) + col);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = nu > 0 ? tc::pack_bf16(__uint_as_float(o[8 * j + 2 * e]) * f,
                                                              __uint_as_float(o[8 * j + 2 * e + 1]) * f)
                                              : 0u;
                            p[j] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                    __syncwarp();
                }
                if (nu > 0) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar + ACCEMPTY);
                }
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

}  // namespace bwd
}  // namespace tcf
}  // namespace sm
}  // namespace sa
