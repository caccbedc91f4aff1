// Softmax attention on the FP32 pipe, for fp32 problems of few small tiles: 16 RPT
// rows x 64 columns (RPT 1 or 2), 256 threads of RPT x 4 entries.  All products are
// packed f32x2 FMAs on operands in shared memory, bound by the shared-memory
// reads; what counts here is the latency of a tile's short chain of chunks (512
// tokens of one head, W = 64, backward: 72 us with 64 rows a tile, 39 with 16).
#pragma once

#include "softmax.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace sm {
namespace simt {

constexpr int LD = 68;            // floats per tile row: 16-byte aligned, rows 4 banks apart
constexpr int THREADS = 256;

// floats of tiles of 16 RPT rows and of the 64-row tiles of a chunk
constexpr int TILE = 64 * LD;
__host__ __device__ constexpr int rtile(int rpt) { return 16 * rpt * LD; }
// bytes of `r` row tiles and `c` chunk tiles
__host__ __device__ constexpr int smem_bytes(int rpt, int r, int c) { return (r * rtile(rpt) + c * TILE) * 4; }

// s[i][j] = sum_k A[ty * RPT + i][k] B[tx + 16 j][k] (even and odd k apart, then together)
template <int RPT>
__device__ __forceinline__ void mm_abt(const float* A, const float* B, int ty, int tx, float (&s)[RPT][4]) {
    uint64_t acc[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll 4
    for (int k = 0; k < 64; k += 4) {
        ulonglong2 x[RPT], y[4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(A + (ty * RPT + i) * LD + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * j) * LD + k);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = tc::fma2(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = tc::fma2(x[i].y, y[j].y, acc[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            tc::upk2(acc[i][j], lo, hi);
            s[i][j] = lo + hi;
        }
}

// acc[i] (two packed pairs) += sum_j P[ty * RPT + i][j] X[j][tx * 4 ..]
template <int RPT>
__device__ __forceinline__ void mm_ab(const float* P, const float* X, int ty, int tx, uint64_t (&acc)[RPT][2]) {
#pragma unroll 4
    for (int j = 0; j < 64; j += 4) {
        float4 p[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * RPT + i) * LD + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(X + (j + jj) * LD + tx * 4);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float e = reinterpret_cast<const float*>(&p[i])[jj];
                const uint64_t ee = tc::pk2(e, e);
                acc[i][0] = tc::fma2(ee, x.x, acc[i][0]);
                acc[i][1] = tc::fma2(ee, x.y, acc[i][1]);
            }
        }
    }
}

// A tile of ROWS rows base(r) (nullptr: zeros) into shared memory by cp.async, 16
// bytes at a time.
template <int ROWS, typename F>
__device__ __forceinline__ void copy_tile(float* dst, const float* any, F base) {
#pragma unroll
    for (int x = threadIdx.x; x < ROWS * 16; x += THREADS) {
        const int r = x >> 4, c = (x & 15) * 4;
        const float* p = base(r);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + r * LD + c)),
                     "l"(p ? p + c : any), "r"(p ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int m = 8; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
    return x;
}
__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int m = 8; m; m >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, m));
    return x;
}

// A tile of query rows: which query and head a row is, and the keys it attends.
template <int RPT>
struct RowTile {
    int b, hk, i0, part;
    long long first;
    int lo[RPT], hi[RPT];  // this thread's rows (hi < lo: none)
    int jlo, jhi;      // the tile's keys

    __device__ void init(const Args& a, int ty) {
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
        for (int i = 0; i < RPT; ++i) {
            int h, t;
            lo[i] = 0;
            hi[i] = -1;
            if (!row(a, ty * RPT + i, h, t)) continue;
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
};

// Which of the chunk's 64 keys exist and are unmasked, as two words.
__device__ __forceinline__ void live_keys(const Args& a, int b, int c0, uint32_t* words) {
    if (threadIdx.x < 64) {
        const int j = c0 + threadIdx.x;
        const bool ok = j < a.Lk && a.live(b, j);
        const uint32_t w = __ballot_sync(~0u, ok);
        if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = w;
    }
}
__device__ __forceinline__ bool live_bit(const uint32_t* words, int j) { return (words[j >> 5] >> (j & 31)) & 1u; }

// One pass over the keys with the running maximum and sum of each row.
template <int RPT>
__global__ void __launch_bounds__(THREADS, 2) k_fwd(const Args a) {
    using T = float;
    extern __shared__ __align__(16) float sh[];
    __shared__ uint32_t words[2][2];
    float *Q = sh, *P = Q + rtile(RPT), *K0 = P + rtile(RPT);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    RowTile<RPT> rt;
    rt.init(a, ty);
    const int n = (rt.jhi - rt.jlo + 64) / 64;  // 0 when empty
    const int n0 = (int)((long long)n * rt.part / a.nsplit), n1 = (int)((long long)n * (rt.part + 1) / a.nsplit);
    copy_tile<16 * RPT>(Q, a.q.at<T>(0, 0, 0), [&](int r) -> const T* {
        int h, t;
        return rt.row(a, r, h, t) ? a.q.at<T>(rt.b, h, t) : nullptr;
    });
    float m[RPT], l[RPT];
    uint64_t o[RPT][2];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        o[i][0] = o[i][1] = 0;
    }
    auto fetch = [&](int ch) {
        const int c0 = rt.jlo + 64 * ch, bf = ch & 1;
        auto row = [&](const View& x, int r) -> const T* {
            const int j = c0 + r;
            return j <= rt.jhi && a.live(rt.b, j) ? x.at<T>(rt.b, rt.hk, j) : nullptr;
        };
        copy_tile<64>(K0 + 2 * bf * TILE, a.k.at<T>(0, 0, 0), [&](int r) { return row(a.k, r); });
        copy_tile<64>(K0 + (2 * bf + 1) * TILE, a.v.at<T>(0, 0, 0), [&](int r) { return row(a.v, r); });
        copy_commit();
    };
    if (n0 < n1) fetch(n0);
    for (int ch = n0; ch < n1; ++ch) {
        const int c0 = rt.jlo + 64 * ch, bf = ch & 1;
        const float *K = K0 + 2 * bf * TILE, *V = K + TILE;
        live_keys(a, rt.b, c0, words[ch & 1]);
        copy_wait();
        __syncthreads();
        if (ch + 1 < n1) fetch(ch + 1);
        float s[RPT][4];
        mm_abt<RPT>(Q, K, ty, tx, s);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int jj = tx + 16 * j, key = c0 + jj;
                const bool on = key >= rt.lo[i] && key <= rt.hi[i] && live_bit(words[ch & 1], jj);
                s[i][j] = on ? s[i][j] * a.c2 : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            top = max16(top);
            const float use = top == -INFINITY ? 0.f : top;
            const float f = ex2(m[i] - use);
            m[i] = top;
            float add = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = ex2(s[i][j] - use);
                add += p;
                P[(ty * RPT + i) * LD + tx + 16 * j] = p;
            }
            l[i] = l[i] * f + add;  // this thread's share of the sum
            const uint64_t ff = tc::pk2(f, f);
            o[i][0] = tc::fma2(o[i][0], ff, 0);
            o[i][1] = tc::fma2(o[i][1], ff, 0);
        }
        __syncwarp();  // a warp writes and reads the same rows of P
        mm_ab<RPT>(P, V, ty, tx, o);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float total = sum16(l[i]);
        int h, t;
        if (!rt.row(a, ty * RPT + i, h, t)) continue;
        float x[4];
        tc::upk2(o[i][0], x[0], x[1]);
        tc::upk2(o[i][1], x[2], x[3]);
        const long long row = ((long long)rt.b * a.Hq + h) * a.Lq + t;
        if (a.nsplit > 1) {
            const long long at = row * a.nparts + rt.part;
            store4(a.part_o + at * 64 + tx * 4, x[0], x[1], x[2], x[3]);
            // a NaN among the scores stays one when the parts are joined
            if (tx == 0) a.part_ml[at] = make_float2(total != total && m[i] == -INFINITY ? 0.f : m[i], total);
            continue;
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;  // a NaN stays one
        store4(a.o.at<T>(rt.b, h, t) + tx * 4, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        if (tx == 0) a.u[row] = total == 0.f ? 0.f : -(m[i] + lg2(total)) * kLn2;
    }
}

// dQ by query rows; also D, for the key sweep.
template <int RPT>
__global__ void __launch_bounds__(THREADS, 2) k_bwd_q(const Args a) {
    using T = float;
    extern __shared__ __align__(16) float sh[];
    __shared__ uint32_t words[2][2];
    float *Q = sh, *dO = Q + rtile(RPT), *S = dO + rtile(RPT), *K0 = S + rtile(RPT);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    RowTile<RPT> rt;
    rt.init(a, ty);
    const int nc = (rt.jhi - rt.jlo + 64) / 64;
    const int n0 = (int)((long long)nc * rt.part / a.nsplit), n = (int)((long long)nc * (rt.part + 1) / a.nsplit);
    auto qrow = [&](const View& x, int r) -> const T* {
        int h, t;
        if (!rt.row(a, r, h, t)) return nullptr;
        const long long p = rt.first + t;
        return p >= 0 && p < a.Lk && a.live(rt.b, (int)p) ? x.at<T>(rt.b, h, t) : nullptr;
    };
    uint64_t acc[RPT][2];
#pragma unroll
    for (int i = 0; i < RPT; ++i) acc[i][0] = acc[i][1] = 0;
    auto fetch = [&](int ch) {
        const int c0 = rt.jlo + 64 * ch, bf = ch & 1;
        auto row = [&](const View& x, int r) -> const T* {
            const int j = c0 + r;
            return j <= rt.jhi && a.live(rt.b, j) ? x.at<T>(rt.b, rt.hk, j) : nullptr;
        };
        copy_tile<64>(K0 + 2 * bf * TILE, a.k.at<T>(0, 0, 0), [&](int r) { return row(a.k, r); });
        copy_tile<64>(K0 + (2 * bf + 1) * TILE, a.v.at<T>(0, 0, 0), [&](int r) { return row(a.v, r); });
        copy_commit();
    };
    copy_tile<16 * RPT>(Q, a.q.at<T>(0, 0, 0), [&](int r) { return qrow(a.q, r); });
    copy_tile<16 * RPT>(dO, a.q.at<T>(0, 0, 0), [&](int r) { return qrow(a.dO, r); });
    if (n0 < n) fetch(n0);
    else copy_commit();
    float u2[RPT], D[RPT];
    float4 o[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        u2[i] = 0.f;
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        int h, t;
        if (rt.row(a, ty * RPT + i, h, t)) u2[i] = a.u[((long long)rt.b * a.Hq + h) * a.Lq + t] * kLog2e;
        if (const T* x = qrow(a.o, ty * RPT + i)) o[i] = *reinterpret_cast<const float4*>(x + tx * 4);
    }
    copy_wait();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {  // D = dO . O
        const float4 g = *reinterpret_cast<const float4*>(dO + (ty * RPT + i) * LD + tx * 4);
        D[i] = sum16(fmaf(o[i].x, g.x, fmaf(o[i].y, g.y, fmaf(o[i].z, g.z, o[i].w * g.w))));
    }
    for (int ch = n0; ch < n; ++ch) {
        const int c0 = rt.jlo + 64 * ch, bf = ch & 1;
        const float *K = K0 + 2 * bf * TILE, *V = K + TILE;
        live_keys(a, rt.b, c0, words[ch & 1]);
        copy_wait();
        __syncthreads();
        if (ch + 1 < n) fetch(ch + 1);
        float s[RPT][4], g[RPT][4];
        mm_abt<RPT>(Q, K, ty, tx, s);
        mm_abt<RPT>(dO, V, ty, tx, g);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int jj = tx + 16 * j, key = c0 + jj;
                const bool on = key >= rt.lo[i] && key <= rt.hi[i] && live_bit(words[ch & 1], jj);
                S[(ty * RPT + i) * LD + jj] = on ? ex2(fmaf(s[i][j], a.c2, u2[i])) * (g[i][j] - D[i]) : 0.f;
            }
        __syncwarp();  // a warp writes and reads the same rows of S
        mm_ab<RPT>(S, K, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        int h, t;
        if (!rt.row(a, ty * RPT + i, h, t)) continue;
        float x[4];
        tc::upk2(acc[i][0], x[0], x[1]);
        tc::upk2(acc[i][1], x[2], x[3]);
        const long long row = ((long long)rt.b * a.Hq + h) * a.Lq + t;
        T* out = a.nsplit > 1 ? a.part_o + (row * a.nsplit + rt.part) * 64 : a.dq.at<T>(rt.b, h, t);
        store4(out + tx * 4, x[0] * a.c, x[1] * a.c, x[2] * a.c, x[3] * a.c);
        if (tx == 0 && rt.part == 0) a.D[row] = D[i];
    }
}

// dK and dV by key rows: the queries of every head of the group whose band holds the keys.
template <int RPT>
__global__ void __launch_bounds__(THREADS, 2) k_bwd_kv(const Args a) {
    using T = float;
    extern __shared__ __align__(16) float sh[];
    __shared__ uint32_t words[2][2];
    __shared__ float u2[2][64], D[2][64];
    float *K = sh, *V = K + rtile(RPT), *P = V + rtile(RPT), *S = P + rtile(RPT), *Q0 = S + rtile(RPT);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int x = blockIdx.x;
    const int part = x % a.nsplit;
    x /= a.nsplit;
    constexpr int M = 16 * RPT;
    const int j0 = (x % a.ntile) * M;
    x /= a.ntile;
    const int hk = x % a.Hk, b = x / a.Hk;
    const long long first = a.first(b);
    // queries whose position lies in [j0 - R, j0 + M - 1 + W] and in the span
    const int2 sp = span(a, b);
    const long long pl = j0 - (long long)a.R > sp.x ? j0 - (long long)a.R : sp.x;
    const long long ph = (long long)j0 + M - 1 + a.W < sp.y ? (long long)j0 + M - 1 + a.W : sp.y;
    const long long il = pl - first > 0 ? pl - first : 0;
    const long long ih = ph - first < a.Lq - 1 ? ph - first : a.Lq - 1;
    const int n = ih < il || j0 > sp.y || j0 + M - 1 < sp.x ? 0 : (int)((ih - il) / 64 + 1);
    auto krow = [&](const View& y, int r) -> const T* {
        const int j = j0 + r;
        return j < a.Lk && a.live(b, j) ? y.at<T>(b, hk, j) : nullptr;
    };
    copy_tile<16 * RPT>(K, a.k.at<T>(0, 0, 0), [&](int r) { return krow(a.k, r); });
    copy_tile<16 * RPT>(V, a.k.at<T>(0, 0, 0), [&](int r) { return krow(a.v, r); });
    bool ok[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) ok[i] = krow(a.k, ty * RPT + i) != nullptr;
    uint64_t dk[RPT][2], dv[RPT][2];
#pragma unroll
    for (int i = 0; i < RPT; ++i) dk[i][0] = dk[i][1] = dv[i][0] = dv[i][1] = 0;
    // chunks of queries, head after head: this part's
    const int y0 = (int)((long long)n * a.G * part / a.nsplit), ny = (int)((long long)n * a.G * (part + 1) / a.nsplit);
    auto fetch = [&](int y) {
        const int h = hk * a.G + y / n, t0 = (int)il + 64 * (y % n), bf = y & 1;
        if (threadIdx.x < 64) {
            const int t = t0 + threadIdx.x;
            const bool on = t <= ih && a.live(b, (int)(first + t));
            const uint32_t w = __ballot_sync(~0u, on);
            if ((threadIdx.x & 31) == 0) words[bf][threadIdx.x >> 5] = w;
            const long long at = ((long long)b * a.Hq + h) * a.Lq + t;
            u2[bf][threadIdx.x] = on ? a.u[at] * kLog2e : 0.f;
            D[bf][threadIdx.x] = on ? a.D[at] : 0.f;
        }
        auto row = [&](const View& z, int r) -> const T* {
            const int t = t0 + r;
            return t <= ih && a.live(b, (int)(first + t)) ? z.at<T>(b, h, t) : nullptr;
        };
        copy_tile<64>(Q0 + 2 * bf * TILE, a.q.at<T>(0, 0, 0), [&](int r) { return row(a.q, r); });
        copy_tile<64>(Q0 + (2 * bf + 1) * TILE, a.dO.at<T>(0, 0, 0), [&](int r) { return row(a.dO, r); });
        copy_commit();
    };
    if (y0 < ny) fetch(y0);
    for (int y = y0; y < ny; ++y) {
        const int t0 = (int)il + 64 * (y % n), bf = y & 1;
        const float *Q = Q0 + 2 * bf * TILE, *dO = Q + TILE;
        copy_wait();
        __syncthreads();
        if (y + 1 < ny) fetch(y + 1);
        float s[RPT][4], g[RPT][4];
        mm_abt<RPT>(K, Q, ty, tx, s);
        mm_abt<RPT>(V, dO, ty, tx, g);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int jj = tx + 16 * j;
                const long long gap = first + t0 + jj - (j0 + ty * RPT + i);  // query's position less the key's
                const bool on = ok[i] && live_bit(words[bf], jj) && gap <= a.W && gap >= -(long long)a.R;
                const float p = on ? ex2(fmaf(s[i][j], a.c2, u2[bf][jj])) : 0.f;
                P[(ty * RPT + i) * LD + jj] = p;
                S[(ty * RPT + i) * LD + jj] = on ? p * (g[i][j] - D[bf][jj]) : 0.f;
            }
        __syncwarp();
        mm_ab<RPT>(P, dO, ty, tx, dv);
        mm_ab<RPT>(S, Q, ty, tx, dk);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int j = j0 + ty * RPT + i;
        if (j >= a.Lk) continue;
        float z[4];
        tc::upk2(dv[i][0], z[0], z[1]);
        tc::upk2(dv[i][1], z[2], z[3]);
        const long long row = ((long long)b * a.Hk + hk) * a.Lk + j;
        T* out = a.part_o + (row * a.nsplit + part) * 128;
        store4((a.nsplit > 1 ? out : a.dv.at<T>(b, hk, j)) + tx * 4, z[0], z[1], z[2], z[3]);
        tc::upk2(dk[i][0], z[0], z[1]);
        tc::upk2(dk[i][1], z[2], z[3]);
        store4((a.nsplit > 1 ? out + 64 : a.dk.at<T>(b, hk, j)) + tx * 4, z[0] * a.c, z[1] * a.c, z[2] * a.c, z[3] * a.c);
    }
}

// The parts' gradients added up in their order, one warp per row: dQ, or dV and dK.
__global__ void __launch_bounds__(128) k_sum(const Args a, int kv) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, H = kv ? a.Hk : a.Hq, L = kv ? a.Lk : a.Lq;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (row >= (long long)a.B * H * L) return;
    const int t = (int)(row % L), h = (int)(row / L % H), b = (int)(row / L / H);
    for (int z = 0; z < (kv ? 2 : 1); ++z) {
        const float2* p = reinterpret_cast<const float2*>(a.part_o + row * a.nsplit * (kv ? 128 : 64) + 64 * z) + lane;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < a.nsplit; ++i) {
            const float2 x = p[i * (kv ? 64 : 32)];
            s.x += x.x;
            s.y += x.y;
        }
        reinterpret_cast<float2*>((!kv ? a.dq : z == 0 ? a.dv : a.dk).at<float>(b, h, t))[lane] = s;
    }
}

}  // namespace simt
}  // namespace sm
}  // namespace sa
