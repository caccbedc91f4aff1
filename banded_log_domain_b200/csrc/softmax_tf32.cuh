// Softmax attention in fp32 on warp matrix instructions (the larger problems; see
// softmax_simt.cuh for the few small tiles).
//
// Every fp32 operand is split in two tf32 numbers, x = hi + lo, hi rounded to
// nearest and lo, of either sign, cut to 11 bits (at most 2^-21 of x is lost).
// Every product is hi lo' + lo hi' + hi hi' with fp32 sums, the cross terms summed
// apart; the term left out is 2^-22 of a product.  (hi of a magnitude from
// 2^128 (1 - 2^-12) on rounds to infinity: such values count as infinite.)  Against 64 bits the results are
// off by 3e-7 to 7e-7, as on the FMA pipe (6e-7).
// mma.sync takes 508 tf32 FMA per clock and SM, a third of that here; two warps a
// scheduler and the splitting keep it half busy.  Measured against 64 x 64 tiles on
// the FMA pipe, which shared-memory reads hold at 45 % of its rate: masked2k's
// training step 0.59 ms (0.66), 4096 dense tokens of 4 heads 0.49 + 1.56 ms (0.55 +
// 1.87).  (tcgen05 takes tf32 operands from shared memory: the splits would have to
// be written back there first, four tiles for two.)
//
// Blocks of four warps, 16 rows each, on tiles of 64 rows x 64 columns.  A lane
// holds rows g and g + 8, columns 2t and 2t + 1 of every eight (g = lane / 4, t =
// lane % 4).  As the A operand of the second product these entries serve as they
// are, with the columns of an eight counted 0 2 4 6 1 3 5 7 on both sides.
#pragma once

#include "softmax_simt.cuh"

namespace sa {
namespace sm {
namespace tf32 {

using simt::LD;
using simt::TILE;
using simt::copy_commit;
using simt::copy_wait;
constexpr int THREADS = 128;
// bytes: `tiles` of 64 rows
__host__ __device__ constexpr int smem_bytes(int tiles) { return tiles * TILE * 4; }

struct Two {
    uint32_t hi, lo;
};
__device__ __forceinline__ Two split(float x) {
    Two s;
    s.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    s.lo = __float_as_uint(x - __uint_as_float(s.hi));  // the instruction reads its upper 19 bits
    return s;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c (main), x (cross terms) += a b for four tiles of columns, one kind of product
// after the other: an accumulator's next use lies four instructions on.
__device__ __forceinline__ void mma3(float (&c)[4][4], float (&x)[4][4], const uint32_t (&ah)[4],
                                     const uint32_t (&al)[4], const float (&b0)[4], const float (&b1)[4]) {
    Two p[4], q[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        p[n] = split(b0[n]);
        q[n] = split(b1[n]);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) mma(x[n], al, p[n].hi, q[n].hi);
#pragma unroll
    for (int n = 0; n < 4; ++n) mma(c[n], ah, p[n].hi, q[n].hi);
#pragma unroll
    for (int n = 0; n < 4; ++n) mma(x[n], ah, p[n].lo, q[n].lo);
}

// s[n] = A B^T for this warp's 16 rows (A at its first) and the 64 rows of B
__device__ __forceinline__ void mm_abt(const float* A, const float* B, int g, int t, float (&s)[8][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float c[4][4], x[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[n][e] = x[n][e] = 0.f;
#pragma unroll 2
        for (int k = 0; k < 64; k += 8) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Two y = split(A[(g + 8 * (e & 1)) * LD + k + t + 4 * (e >> 1)]);
                ah[e] = y.hi;
                al[e] = y.lo;
            }
            float b0[4], b1[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float* b = B + (32 * h + 8 * n + g) * LD + k + t;
                b0[n] = b[0];
                b1[n] = b[4];
            }
            mma3(c, x, ah, al, b0, b1);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[4 * h + n][e] = c[n][e] + x[n][e];
    }
}

// o += P X, P this warp's 16 x 64 entries as mm_abt leaves them, X 64 rows
__device__ __forceinline__ void mm_ab(const float (&p)[8][4], const float* X, int g, int t, float (&o)[8][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float c[4][4], x[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[n][e] = x[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Two y = split(p[k][2 * (e & 1) + (e >> 1)]);
                ah[e] = y.hi;
                al[e] = y.lo;
            }
            float b0[4], b1[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float* b = X + (8 * k + 2 * t) * LD + 32 * h + 8 * n + g;
                b0[n] = b[0];
                b1[n] = b[LD];
            }
            mma3(c, x, ah, al, b0, b1);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[4 * h + n][e] += c[n][e] + x[n][e];
    }
}

// A tile of 64 rows base(r) (nullptr: zeros) by cp.async.
template <typename F>
__device__ __forceinline__ void copy_tile(float* dst, const float* any, F base) {
#pragma unroll
    for (int x = threadIdx.x; x < 64 * 16; x += THREADS) {
        const int r = x >> 4, c = (x & 15) * 4;
        const float* p = base(r);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + r * LD + c)),
                     "l"(p ? p + c : any), "r"(p ? 16 : 0)
                     : "memory");
    }
}

__device__ __forceinline__ float sum4(float x) {  // over the lanes of a row
    x += __shfl_xor_sync(~0u, x, 1);
    return x + __shfl_xor_sync(~0u, x, 2);
}
__device__ __forceinline__ float max4(float x) {
    x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
    return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}

// A tile of query rows; this lane's are g and g + 8 of its warp's 16.
struct RowTile {
    int b, hk, i0, part, jlo, jhi, lo[2], hi[2];
    long long first;

    __device__ void init(const Args& a, int r0) {
        int x = blockIdx.x;
        part = x % a.nsplit;
        x /= a.nsplit;
        const int qt = x % a.ntile;
        x /= a.ntile;
        hk = x % a.Hk;
        b = x / a.Hk;
        i0 = qt * a.nq;
        first = a.first(b);
        tile_keys(a, b, i0, min(i0 + a.nq, a.Lq) - 1, jlo, jhi);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int h, t;
            lo[i] = 0;
            hi[i] = -1;
            if (!row(a, r0 + 8 * i, h, t)) continue;
            const long long p = first + t;
            if (p >= 0 && p < a.Lk && a.live(b, (int)p)) a.keys(p, lo[i], hi[i]);
        }
    }
    __device__ __forceinline__ bool row(const Args& a, int r, int& h, int& t) const {
        const int g = r / a.nq;
        t = i0 + r % a.nq;
        h = hk * a.G + g;
        return g < a.G && t < a.Lq;
    }
    // the row's part of a query tensor, nullptr where it is not in use
    __device__ __forceinline__ const float* in_use(const Args& a, const View& x, int r) const {
        int h, t;
        if (!row(a, r, h, t)) return nullptr;
        const long long p = first + t;
        return p >= 0 && p < a.Lk && a.live(b, (int)p) ? x.at<float>(b, h, t) : nullptr;
    }
};

// Two words of which of a chunk's 64 keys exist and are unmasked.
using simt::live_bit;
using simt::live_keys;

__global__ void __launch_bounds__(THREADS, 2) k_fwd(const Args a) {
    extern __shared__ __align__(16) float sh[];
    __shared__ uint32_t words[2][2];
    float *Q = sh, *K0 = Q + TILE;
    const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    RowTile rt;
    rt.init(a, 16 * warp + g);
    const int n = (rt.jhi - rt.jlo + 64) / 64;  // 0 when empty
    const int n0 = (int)((long long)n * rt.part / a.nsplit), n1 = (int)((long long)n * (rt.part + 1) / a.nsplit);
    copy_tile(Q, a.q.at<float>(0, 0, 0), [&](int r) { return rt.in_use(a, a.q, r); });
    auto fetch = [&](int ch) {
        const int c0 = rt.jlo + 64 * ch;
        float* K = K0 + 2 * (ch & 1) * TILE;
        auto row = [&](const View& x, int r) -> const float* {
            const int j = c0 + r;
            return j <= rt.jhi && a.live(rt.b, j) ? x.at<float>(rt.b, rt.hk, j) : nullptr;
        };
        copy_tile(K, a.k.at<float>(0, 0, 0), [&](int r) { return row(a.k, r); });
        copy_tile(K + TILE, a.k.at<float>(0, 0, 0), [&](int r) { return row(a.v, r); });
        copy_commit();
    };
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    if (n0 < n1) fetch(n0);
    for (int ch = n0; ch < n1; ++ch) {
        const int c0 = rt.jlo + 64 * ch;
        const float *K = K0 + 2 * (ch & 1) * TILE, *V = K + TILE;
        live_keys(a, rt.b, c0, words[ch & 1]);
        copy_wait();
        __syncthreads();
        if (ch + 1 < n1) fetch(ch + 1);
        float s[8][4];
        mm_abt(Q + 16 * warp * LD, K, g, t, s);
        const uint32_t* w = words[ch & 1];
        const bool full = w[0] == ~0u && w[1] == ~0u;
        float top[2] = {m[0], m[1]};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int jj = 8 * i + 2 * t + (e & 1), key = c0 + jj;
                const bool on = key >= rt.lo[e >> 1] && key <= rt.hi[e >> 1] && (full || live_bit(w, jj));
                s[i][e] = on ? s[i][e] * a.c2 : -INFINITY;
                top[e >> 1] = fmaxf(top[e >> 1], s[i][e]);
            }
        float use[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top[r] = max4(top[r]);
            use[r] = top[r] == -INFINITY ? 0.f : top[r];
            const float f = ex2(m[r] - use[r]);
            m[r] = top[r];
            l[r] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][2 * r] *= f;
                o[i][2 * r + 1] *= f;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i][e] = ex2(s[i][e] - use[e >> 1]);
                l[e >> 1] += s[i][e];
            }
        mm_ab(s, V, g, t, o);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float total = sum4(l[r]);
        int h, tt;
        if (!rt.row(a, 16 * warp + g + 8 * r, h, tt)) continue;
        const long long row = ((long long)rt.b * a.Hq + h) * a.Lq + tt;
        const long long at = row * a.nparts + rt.part;
        const float inv = a.nsplit > 1 ? 1.f : total == 0.f ? 0.f : 1.f / total;  // a NaN stays one
        float* out = a.nsplit > 1 ? a.part_o + at * 64 : a.o.at<float>(rt.b, h, tt);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float2*>(out + 8 * i + 2 * t) = make_float2(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
        if (t != 0) continue;
        // a NaN among the scores stays one when the parts are joined
        if (a.nsplit > 1) a.part_ml[at] = make_float2(total != total && m[r] == -INFINITY ? 0.f : m[r], total);
        else a.u[row] = total == 0.f ? 0.f : -(m[r] + lg2(total)) * kLn2;
    }
}

// dQ by query rows; also D, for the key sweep.
__global__ void __launch_bounds__(THREADS, 2) k_bwd_q(const Args a) {
    extern __shared__ __align__(16) float sh[];
    __shared__ uint32_t words[2][2];
    float *Q = sh, *dO = Q + TILE, *K0 = dO + TILE;
    const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    RowTile rt;
    rt.init(a, 16 * warp + g);
    const int nc = (rt.jhi - rt.jlo + 64) / 64;
    const int n0 = (int)((long long)nc * rt.part / a.nsplit), n1 = (int)((long long)nc * (rt.part + 1) / a.nsplit);
    copy_tile(Q, a.q.at<float>(0, 0, 0), [&](int r) { return rt.in_use(a, a.q, r); });
    copy_tile(dO, a.q.at<float>(0, 0, 0), [&](int r) { return rt.in_use(a, a.dO, r); });
    auto fetch = [&](int ch) {
        const int c0 = rt.jlo + 64 * ch;
        float* K = K0 + 2 * (ch & 1) * TILE;
        auto row = [&](const View& x, int r) -> const float* {
            const int j = c0 + r;
            return j <= rt.jhi && a.live(rt.b, j) ? x.at<float>(rt.b, rt.hk, j) : nullptr;
        };
        copy_tile(K, a.k.at<float>(0, 0, 0), [&](int r) { return row(a.k, r); });
        copy_tile(K + TILE, a.k.at<float>(0, 0, 0), [&](int r) { return row(a.v, r); });
        copy_commit();
    };
    if (n0 < n1) fetch(n0);
    else copy_commit();
    // D = dO . O, 16 channels in each of a row's lanes
    float u2[2], D[2], acc[8][4];
    float4 o[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        u2[r] = 0.f;
        int h, tt;
        if (rt.row(a, 16 * warp + g + 8 * r, h, tt)) u2[r] = a.u[((long long)rt.b * a.Hq + h) * a.Lq + tt] * kLog2e;
        const float* x = rt.in_use(a, a.o, 16 * warp + g + 8 * r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[r][i] = x ? reinterpret_cast<const float4*>(x + 16 * t)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    copy_wait();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(dO + (16 * warp + g + 8 * r) * LD + 16 * t + 4 * i);
            dot = fmaf(o[r][i].x, x.x, fmaf(o[r][i].y, x.y, fmaf(o[r][i].z, x.z, fmaf(o[r][i].w, x.w, dot))));
        }
        D[r] = sum4(dot);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    for (int ch = n0; ch < n1; ++ch) {
        const int c0 = rt.jlo + 64 * ch;
        const float *K = K0 + 2 * (ch & 1) * TILE, *V = K + TILE;
        live_keys(a, rt.b, c0, words[ch & 1]);
        copy_wait();
        __syncthreads();
        if (ch + 1 < n1) fetch(ch + 1);
        float s[8][4], gg[8][4];
        mm_abt(Q + 16 * warp * LD, K, g, t, s);
        mm_abt(dO + 16 * warp * LD, V, g, t, gg);
        const uint32_t* w = words[ch & 1];
        const bool full = w[0] == ~0u && w[1] == ~0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int jj = 8 * i + 2 * t + (e & 1), key = c0 + jj, r = e >> 1;
                const bool on = key >= rt.lo[r] && key <= rt.hi[r] && (full || live_bit(w, jj));
                s[i][e] = on ? ex2(fmaf(s[i][e], a.c2, u2[r])) * (gg[i][e] - D[r]) : 0.f;
            }
        mm_ab(s, K, g, t, acc);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        int h, tt;
        if (!rt.row(a, 16 * warp + g + 8 * r, h, tt)) continue;
        const long long row = ((long long)rt.b * a.Hq + h) * a.Lq + tt;
        float* out = a.nsplit > 1 ? a.part_o + (row * a.nsplit + rt.part) * 64 : a.dq.at<float>(rt.b, h, tt);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float2*>(out + 8 * i + 2 * t) = make_float2(acc[i][2 * r] * a.c, acc[i][2 * r + 1] * a.c);
        if (t == 0 && rt.part == 0) a.D[row] = D[r];
    }
}

// dK and dV by key rows: the queries of every head of the group whose band holds the keys.
__global__ void __launch_bounds__(THREADS, 2) k_bwd_kv(const Args a) {
    extern __shared__ __align__(16) float sh[];
    __shared__ uint32_t words[2][2];
    __shared__ float u2[2][64], D[2][64];
    float *K = sh, *V = K + TILE, *Q0 = V + TILE;
    const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int x = blockIdx.x;
    const int part = x % a.nsplit;
    x /= a.nsplit;
    const int j0 = (x % a.ntile) * 64;
    x /= a.ntile;
    const int hk = x % a.Hk, b = x / a.Hk;
    const long long first = a.first(b);
    // queries whose position lies in [j0 - R, j0 + 63 + W] and in the span
    const int2 sp = span(a, b);
    const long long pl = j0 - (long long)a.R > sp.x ? j0 - (long long)a.R : sp.x;
    const long long ph = (long long)j0 + 63 + a.W < sp.y ? (long long)j0 + 63 + a.W : sp.y;
    const long long il = pl - first > 0 ? pl - first : 0;
    const long long ih = ph - first < a.Lq - 1 ? ph - first : a.Lq - 1;
    const int n = ih < il || j0 > sp.y || j0 + 63 < sp.x ? 0 : (int)((ih - il) / 64 + 1);
    auto krow = [&](const View& y, int r) -> const float* {
        const int j = j0 + r;
        return j < a.Lk && a.live(b, j) ? y.at<float>(b, hk, j) : nullptr;
    };
    copy_tile(K, a.k.at<float>(0, 0, 0), [&](int r) { return krow(a.k, r); });
    copy_tile(V, a.k.at<float>(0, 0, 0), [&](int r) { return krow(a.v, r); });
    const int ny0 = (int)((long long)n * a.G * part / a.nsplit), ny1 = (int)((long long)n * a.G * (part + 1) / a.nsplit);
    auto fetch = [&](int y) {
        const int h = hk * a.G + y / n, t0 = (int)il + 64 * (y % n), bf = y & 1;
        if (threadIdx.x < 64) {
            const int i = t0 + threadIdx.x;
            const bool on = i <= ih && a.live(b, (int)(first + i));
            const uint32_t w = __ballot_sync(~0u, on);
            if ((threadIdx.x & 31) == 0) words[bf][threadIdx.x >> 5] = w;
            const long long at = ((long long)b * a.Hq + h) * a.Lq + i;
            u2[bf][threadIdx.x] = on ? a.u[at] * kLog2e : 0.f;
            D[bf][threadIdx.x] = on ? a.D[at] : 0.f;
        }
        auto row = [&](const View& z, int r) -> const float* {
            const int i = t0 + r;
            return i <= ih && a.live(b, (int)(first + i)) ? z.at<float>(b, h, i) : nullptr;
        };
        float* Q = Q0 + 2 * bf * TILE;
        copy_tile(Q, a.q.at<float>(0, 0, 0), [&](int r) { return row(a.q, r); });
        copy_tile(Q + TILE, a.q.at<float>(0, 0, 0), [&](int r) { return row(a.dO, r); });
        copy_commit();
    };
    // this lane's keys, and their queries' positions
    bool ok[2];
    float dk[8][4], dv[8][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) ok[r] = krow(a.k, 16 * warp + g + 8 * r) != nullptr;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[i][e] = dv[i][e] = 0.f;
    if (ny0 < ny1) fetch(ny0);
    else copy_commit();
    for (int y = ny0; y < ny1; ++y) {
        const int t0 = (int)il + 64 * (y % n), bf = y & 1;
        const float *Q = Q0 + 2 * bf * TILE, *dO = Q + TILE;
        copy_wait();
        __syncthreads();
        if (y + 1 < ny1) fetch(y + 1);
        float s[8][4], gg[8][4];
        mm_abt(K + 16 * warp * LD, Q, g, t, s);
        mm_abt(V + 16 * warp * LD, dO, g, t, gg);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int jj = 8 * i + 2 * t + (e & 1), r = e >> 1;
                const long long gap = first + t0 + jj - (j0 + 16 * warp + g + 8 * r);  // query's position less the key's
                const bool on = ok[r] && live_bit(words[bf], jj) && gap <= a.W && gap >= -(long long)a.R;
                const float p = on ? ex2(fmaf(s[i][e], a.c2, u2[bf][jj])) : 0.f;
                s[i][e] = p;
                gg[i][e] = on ? p * (gg[i][e] - D[bf][jj]) : 0.f;
            }
        mm_ab(s, dO, g, t, dv);
        mm_ab(gg, Q, g, t, dk);
    }
    copy_wait();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int j = j0 + 16 * warp + g + 8 * r;
        if (j >= a.Lk) continue;
        const long long row = ((long long)b * a.Hk + hk) * a.Lk + j;
        float* pv = a.nsplit > 1 ? a.part_o + (row * a.nsplit + part) * 128 : a.dv.at<float>(b, hk, j);
        float* pk = a.nsplit > 1 ? pv + 64 : a.dk.at<float>(b, hk, j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            *reinterpret_cast<float2*>(pv + 8 * i + 2 * t) = make_float2(dv[i][2 * r], dv[i][2 * r + 1]);
            *reinterpret_cast<float2*>(pk + 8 * i + 2 * t) = make_float2(dk[i][2 * r] * a.c, dk[i][2 * r + 1] * a.c);
        }
    }
}

}  // namespace tf32
}  // namespace sm
}  // namespace sa
