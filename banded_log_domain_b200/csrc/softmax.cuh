// What the softmax attention kernels share: the arguments, the band of a tile
// of query rows, and the kernel that joins the parts of split rows.
//
// Query rows are packed: a tile of M rows holds the same nq queries of all G
// query heads that share a key head, row r = g * nq + i, so that the group reads
// each key tile once.  With G == 1 that is M consecutive queries.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace sm {

struct View {
    void* p;
    long long s[3];  // element strides: batch, head, token
    template <typename T>
    __device__ __forceinline__ T* at(int b, int h, long long t) const {
        return reinterpret_cast<T*>(p) + b * s[0] + h * s[1] + t * s[2];
    }
};

struct Args {
    int B, Hq, Hk, G, Lq, Lk;
    int W, R;             // keys p - W .. p + R
    float c, c2;          // 1 / (sqrt(d) eps), and that times log2(e)
    const int* q_pos;     // [B], or NULL: Lk - Lq
    const uint8_t* mask;  // [B][Lk], or NULL
    int2* span;           // [B]: first and last unmasked token, with a mask
    View q, k, v, o, dO, dq, dk, dv;
    float* u;             // [B][Hq][Lq]
    float* D;             // [B][Hq][Lq], backward, fp32
    uint4* aug;           // [B][Hq][Lq][2], bf16: u / c and -D as 16 more channels of a query
    int* status;
    int nq;               // queries per tile and head
    int ntile;            // query (dK, dV: key) tiles per sequence and key head
    int nsplit;           // forward: parts of a tile's keys
    float* part_o;        // [row][part][64], then
    float2* part_ml;      // [row][part]: running maximum (log2 units) and sum
    int nparts;

    // position of query 0 of sequence b
    __device__ __forceinline__ long long first(int b) const { return q_pos ? q_pos[b] : Lk - Lq; }
    __device__ __forceinline__ bool live(int b, int j) const {
        return mask == nullptr || mask[(long long)b * Lk + j] != 0;
    }
    // keys [lo, hi] that the query at position p attends, mask aside
    __device__ __forceinline__ void keys(long long p, int& lo, int& hi) const {
        lo = (int)(p - W > 0 ? p - W : 0);
        hi = (int)(p + R < Lk - 1 ? p + R : Lk - 1);
    }
};

// Sequence b's tokens [x, y] outside of which all are masked.
__device__ __forceinline__ int2 span(const Args& a, int b) {
    return a.mask ? a.span[b] : make_int2(0, a.Lk - 1);
}

// The keys [lo, hi] that any of queries i0 .. i1 (inclusive) of sequence b may
// attend; empty (hi < lo) when none may.
__device__ __forceinline__ void tile_keys(const Args& a, int b, int i0, int i1, int& lo, int& hi) {
    const int2 s = span(a, b);
    long long p0 = a.first(b) + i0, p1 = a.first(b) + i1;
    if (p0 < s.x) p0 = s.x;
    if (p1 > s.y) p1 = s.y;
    lo = 0;
    hi = -1;
    if (p1 < p0) return;
    int x;
    a.keys(p0, lo, x);
    a.keys(p1, x, hi);
    lo = max(lo, s.x);
    hi = min(hi, s.y);
}

// The spans, one block per sequence: padding at either end then costs no tiles.
__global__ void __launch_bounds__(1024) k_span(const Args a) {
    __shared__ int lo[32], hi[32];
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const uint8_t* m = a.mask + (long long)blockIdx.x * a.Lk;
    int x = 0x7fffffff, y = -1;
#pragma unroll 8
    for (int j = threadIdx.x; j < a.Lk; j += 1024)
        if (m[j]) {
            x = min(x, j);
            y = j;
        }
    x = __reduce_min_sync(~0u, x);
    y = __reduce_max_sync(~0u, y);
    if ((threadIdx.x & 31) == 0) {
        lo[threadIdx.x >> 5] = x;
        hi[threadIdx.x >> 5] = y;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        x = __reduce_min_sync(~0u, lo[threadIdx.x]);
        y = __reduce_max_sync(~0u, hi[threadIdx.x]);
        if (threadIdx.x == 0) a.span[blockIdx.x] = make_int2(y < 0 ? 0 : x, y);
    }
}

// Joins the parts of split rows: o = sum_s 2^(m_s - m) o_s / l, one warp per row,
// two channels per lane.  Reads each part once (bound by latency: few rows).
template <typename T>
__global__ void __launch_bounds__(128) k_join(const Args a) {
    const long long rows = (long long)a.B * a.Hq * a.Lq;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::grid_dep_wait();
    if (row >= rows) return;
    const float2* ml = a.part_ml + row * a.nparts;
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < a.nparts; s += 32) lse_merge(m, l, ml[s].x, ml[s].y);
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        const float m2 = __shfl_xor_sync(~0u, m, x), l2 = __shfl_xor_sync(~0u, l, x);
        lse_merge(m, l, m2, l2);
    }
    float2 o = make_float2(0.f, 0.f);
    for (int s = 0; s < a.nparts; ++s) {
        const float2 x = ml[s];
        if (x.x == -INFINITY) continue;
        const float w = ex2(x.x - m);
        const float2 y = reinterpret_cast<const float2*>(a.part_o + (row * a.nparts + s) * 64)[lane];
        o.x = fmaf(w, y.x, o.x);
        o.y = fmaf(w, y.y, o.y);
    }
    const float inv = m == -INFINITY ? 0.f : 1.f / l;  // no part holds a key: zeros
    const int t = (int)(row % a.Lq);
    const long long bh = row / a.Lq;
    T* out = a.o.at<T>((int)(bh / a.Hq), (int)(bh % a.Hq), t) + 2 * lane;
    store_elem(out, o.x * inv);
    store_elem(out + 1, o.y * inv);
    if (lane == 0) a.u[row] = m == -INFINITY ? 0.f : -(m + lg2(l)) * kLn2;
}

// dK = dV = 0, one warp per key.
template <typename T>
__global__ void __launch_bounds__(128) k_zero(const Args a) {
    const long long key = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    tc::grid_dep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    if (key >= (long long)a.B * a.Hk * a.Lk) return;
    const int j = (int)(key % a.Lk), lane = threadIdx.x & 31;
    const long long bh = key / a.Lk;
    for (const View* x : {&a.dk, &a.dv}) {
        T* out = x->at<T>((int)(bh / a.Hk), (int)(bh % a.Hk), j) + 2 * lane;
        store_elem(out, 0.f);
        store_elem(out + 1, 0.f);
    }
}

}  // namespace sm
}  // namespace sa
