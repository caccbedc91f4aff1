// Softmax attention of single new tokens over their caches: a key head's query
// rows (query heads of its group times queries) are few, so the pass is bound by
// reading K and V once.
//
// The 64-key chunks of all sequences and key heads are laid end to end and every
// block takes an equal share, whatever the sequences' lengths; a share is walked
// in segments, one per (sequence, key head) that it touches.  Each warp brings its
// keys by cp.async into a ring of its own in shared memory and runs a softmax of
// its own, whose maximum is only moved when it has grown by more than 8 (in log2
// units); the warps' are joined at the segment's end, the blocks' by a second
// kernel.
//   bf16: warp-wide matrix instructions, S^T = K Q^T for 16 keys and 8 rows at a
//     time and O^T += V^T P.  (tcgen05's 128 rows would be mostly empty, and its
//     hand-overs took 1.5 times as long per byte.)  P is rounded to bf16 for its
//     product, as V is (see softmax_tc.cuh); the sum takes it unrounded.
//   fp32: eight lanes hold a key's 64 channels, so a warp takes four keys at once,
//     each with a softmax of its own; the sums of a score over eight lanes end
//     each in one row's lanes, which alone go through that row's softmax.
#pragma once

#include "softmax.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace sm {
namespace token {

constexpr int THREADS = 256;     // fp32
constexpr int THREADS_MMA = 128; // bf16
// Sequences: a loop over them finds a block's share, and a warp's sum over them where they
// lie.  The limit is a choice and not where the kernel stops paying: with it raised, 128
// sequences of 8192 tokens took 168 us (tiled 377), 1024 of 1024 tokens 315 (394).
constexpr int MAXB = 64;
// Query rows per key head: what two tiles of eight (bf16), or four rows of eight lanes'
// sums (fp32), hold.  The tiled forward takes more: 8 sequences of 8192 tokens, 8 key heads
// of 8 heads, bf16: 16 rows 42 us here, 58 tiled; 24 rows 57 tiled.
__host__ __device__ constexpr int max_rows(bool bf16) { return bf16 ? 16 : 4; }

// Whether the sequences' chunks differ in number.
__device__ __forceinline__ bool ragged(const Args& a) { return a.q_pos != nullptr || a.mask != nullptr; }

// Where the chunks of the (sequence, key head) pairs lie in the line of all.
struct Line {
    // chunks of sequence b, of each of its key heads
    static __device__ __forceinline__ int chunks(const Args& a, int b, int& lo, int& hi) {
        tile_keys(a, b, 0, a.Lq - 1, lo, hi);
        return (hi - lo + 64) / 64;
    }
    static __device__ __forceinline__ int chunks(const Args& a, int b) {
        int lo, hi;
        return chunks(a, b, lo, hi);
    }
    // chunks of the sequences before b; the whole warp calls
    static __device__ __forceinline__ long long before(const Args& a, int b) {
        if (!ragged(a)) return (long long)chunks(a, 0) * b;
        int n = 0;
        for (int x = threadIdx.x & 31; x < b; x += 32) n += chunks(a, x);
        return __reduce_add_sync(~0u, n);
    }
};
// Block i of n takes chunks [total i / n, total (i + 1) / n); n is the number of
// blocks, or of chunks where there are fewer (no share is then empty, and every
// block between a pair's first and last has written its part).
__device__ __forceinline__ int share_count(long long total, int blocks) {
    return (int)(total < blocks ? total : blocks);
}
__device__ __forceinline__ long long share_begin(long long total, int i, int n) { return total * i / n; }
__device__ __forceinline__ int share_of(long long chunk, long long total, int n) {
    return (int)(((chunk + 1) * n - 1) / total);
}

// Pair i of 8 fp32 channels.
__device__ __forceinline__ uint64_t pair(const uint4 (&r)[2], int i) {
    const uint4& q = r[i >> 1];
    return (i & 1) ? tc::pk2(__uint_as_float(q.z), __uint_as_float(q.w))
                   : tc::pk2(__uint_as_float(q.x), __uint_as_float(q.y));
}
// 16 bytes global -> shared, asynchronously; zeros when not `valid`.
__device__ __forceinline__ void cp16(void* dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

// A block's share, segment by segment: keys k0 .. k1 - 1 of key head hk of
// sequence b; whole: those are all of them.
struct Share {
    long long at, end, start = 0;  // chunks; start: of sequence b's first
    int b = 0, hk = 0, k0 = 0, k1 = 0;
    bool whole = false;
    __device__ explicit Share(const Args& a) {  // the whole block calls
        const long long total = Line::before(a, a.B) * a.Hk;
        const int n = share_count(total, gridDim.x), i = blockIdx.x;
        at = i < n ? share_begin(total, i, n) : 0;
        end = i < n ? share_begin(total, i + 1, n) : 0;
        if (at < end && !ragged(a)) {
            const long long len = (long long)Line::chunks(a, 0) * a.Hk;
            b = (int)(at / len);
            start = b * len;
        }
    }
    __device__ bool next(const Args& a) {
        if (at >= end) return false;
        int lo, hi, n;
        while (at >= start + (long long)(n = Line::chunks(a, b, lo, hi)) * a.Hk) {
            start += (long long)n * a.Hk;
            ++b;
        }
        hk = (int)((at - start) / n);
        const int c0 = (int)((at - start) - (long long)hk * n);
        const int c1 = (int)(end - at < n - c0 ? c0 + (end - at) : n);
        k0 = lo + 64 * c0;
        k1 = min(hi + 1, lo + 64 * c1);
        whole = c0 == 0 && c1 == n;
        at += c1 - c0;
        return true;
    }
};

constexpr int NV = 2;                           // 16-byte pieces of 8 fp32 channels
constexpr int STAGES = 4;                       // groups of four keys in flight, and values
constexpr int RING_WARP = STAGES * 2 * NV * 512;  // bytes
constexpr int SMEM = 8 * RING_WARP;

// ROWS: the rows of a key head, rounded up to 1, 2 or 4.
template <int ROWS>
__global__ void __launch_bounds__(THREADS, 2) k_token(const Args a) {
    using T = float;
    constexpr int ST = STAGES;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float so[8][ROWS][64];
    __shared__ float2 sml[8][ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = lane >> 3, ch = 8 * (lane & 7);
    // the row whose scores this lane ends up with, and the lane that has row r's
    const int rr = ROWS == 4 ? (lane >> 1) & 3 : ROWS == 2 ? (lane >> 2) & 1 : 0;
    auto holder = [&](int r) { return (lane & 24) + (ROWS == 4 ? 2 * r : ROWS == 2 ? 4 * r : 0); };
    uint4* mine = reinterpret_cast<uint4*>(ring + warp * RING_WARP) + lane;  // stage st, piece e: [(st * 2 NV + e) * 32]
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    Share sh(a);
    const int rows = a.G * a.Lq;
    while (sh.next(a)) {
        const int b = sh.b, hk = sh.hk, k0 = sh.k0, k1 = sh.k1;
        // the rows: r = g * Lq + t; their queries (this lane's channels)
        uint64_t q[ROWS][4], o[ROWS][4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            uint4 x[NV];
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                x[e] = make_uint4(0, 0, 0, 0);
                if (r < rows) x[e] = reinterpret_cast<const uint4*>(a.q.at<T>(b, hk * a.G + r / a.Lq, r % a.Lq) + ch)[e];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[r][i] = pair(x, i);
                o[r][i] = 0;
            }
        }
        // this lane's row: its band, running maximum and sum
        int lo = 0, hi = -1;
        if (rr < rows) {
            const long long p = a.first(b) + rr % a.Lq;
            if (p >= 0 && p < a.Lk && a.live(b, (int)p)) a.keys(p, lo, hi);
        }
        float m = -INFINITY, l = 0.f;
        const T* kp = a.k.at<T>(b, hk, 0) + ch;
        const T* vp = a.v.at<T>(b, hk, 0) + ch;
        // group g of this warp: keys k0 + 4 warp + 32 g + slot
        const int ng = (k1 - (k0 + 4 * warp) + 31) / 32;
        auto fetch = [&](int g) {
            const int j = k0 + 4 * warp + 32 * g + slot;
            const bool on = g < ng && j < k1 && a.live(b, j);
            const long long jj = on ? j : 0;  // an address that is not read, inside the tensor
            uint4* d = mine + (g % ST) * 2 * NV * 32;
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                cp16(d + e * 32, reinterpret_cast<const uint4*>(kp + jj * a.k.s[2]) + e, on);
                cp16(d + (NV + e) * 32, reinterpret_cast<const uint4*>(vp + jj * a.v.s[2]) + e, on);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int g = 0; g < ST - 1; ++g) fetch(g);
        for (int g = 0; g < ng; ++g) {
            fetch(g + ST - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
            const uint4* d = mine + (g % ST) * 2 * NV * 32;
            uint4 x[NV];
#pragma unroll
            for (int e = 0; e < NV; ++e) x[e] = d[e * 32];
            float s[ROWS];
            {
                uint64_t kk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) kk[i] = pair(x, i);
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    uint64_t y = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y = tc::fma2(q[r][i], kk[i], y);
                    float y0, y1;
                    tc::upk2(y, y0, y1);
                    s[r] = y0 + y1;
                }
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) x[e] = d[(NV + e) * 32];
            // sum over eight lanes, handing half of the rows over at every step
            float sc;
            if (ROWS == 4) {
                const bool up = lane & 4;
                float y0 = up ? s[2 % ROWS] : s[0], y1 = up ? s[3 % ROWS] : s[1 % ROWS];
                y0 += __shfl_xor_sync(~0u, up ? s[0] : s[2 % ROWS], 4);
                y1 += __shfl_xor_sync(~0u, up ? s[1 % ROWS] : s[3 % ROWS], 4);
                const bool up2 = lane & 2;
                sc = up2 ? y1 : y0;
                sc += __shfl_xor_sync(~0u, up2 ? y0 : y1, 2);
            } else {
                const bool up = lane & 4;
                sc = ROWS == 2 && up ? s[1 % ROWS] : s[0];
                sc += __shfl_xor_sync(~0u, ROWS == 2 && !up ? s[1 % ROWS] : s[0], 4);
                sc += __shfl_xor_sync(~0u, sc, 2);
            }
            sc += __shfl_xor_sync(~0u, sc, 1);
            const int j = k0 + 4 * warp + 32 * g + slot;
            sc = j >= lo && j <= hi && j < k1 && a.live(b, j) ? sc * a.c2 : -INFINITY;
            const bool move = sc > m + 8.f;
            if (__any_sync(~0u, move)) {
                const float f = move ? ex2(m - sc) : 1.f;  // 0 at the first key
                if (move) m = sc;
                l *= f;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const float fr = __shfl_sync(~0u, f, holder(r));
                    const uint64_t ff = tc::pk2(fr, fr);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r][i] = tc::fma2(o[r][i], ff, 0);
                }
            }
            if (!(sc < INFINITY)) {  // NaN or +inf: so is the row
                l = NAN;
                if (!(fabsf(m) < INFINITY)) m = 0.f;
            }
            const float p = m == -INFINITY ? 0.f : ex2(sc - m);
            l += p;
            uint64_t vv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) vv[i] = pair(x, i);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float pr = ROWS == 1 ? p : __shfl_sync(~0u, p, holder(r));
                const uint64_t pp = tc::pk2(pr, pr);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][i] = tc::fma2(pp, vv[i], o[r][i]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // the warp's four softmaxes, then the block's eight warps
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float mr = __shfl_sync(~0u, m, holder(r)), lr = __shfl_sync(~0u, l, holder(r));
            float mm = mr;
            mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, 8));
            mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, 16));
            const float f = mr == -INFINITY ? 0.f : ex2(mr - mm);
            float ll = mr == -INFINITY ? 0.f : lr * f;
            ll += __shfl_xor_sync(~0u, ll, 8);
            ll += __shfl_xor_sync(~0u, ll, 16);
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::upk2(o[r][i], y[2 * i], y[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] *= f;
                y[i] += __shfl_xor_sync(~0u, y[i], 8);
                y[i] += __shfl_xor_sync(~0u, y[i], 16);
            }
            if (slot == 0) {
                *reinterpret_cast<float4*>(&so[warp][r][ch]) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(&so[warp][r][ch + 4]) = make_float4(y[4], y[5], y[6], y[7]);
                if (ch == 0) sml[warp][r] = make_float2(mm, ll);
            }
        }
        __syncthreads();
        const int r = threadIdx.x >> 6, d = threadIdx.x & 63;
        if (r < ROWS && r < rows) {
            float mm = -INFINITY, ll = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sml[w][r].x);
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float2 z = sml[w][r];
                if (z.x == -INFINITY) continue;
                const float f = ex2(z.x - mm);
                ll = fmaf(z.y, f, ll);
                y = fmaf(so[w][r][d], f, y);
            }
            const int bh = b * a.Hk + hk;
            if (sh.whole) {  // all of the row's keys: the result itself
                const bool none = mm == -INFINITY;
                const int h = hk * a.G + r / a.Lq, t = r % a.Lq;
                store_elem(a.o.at<T>(b, h, t) + d, none ? 0.f : y / ll);
                if (d == 0) a.u[((long long)b * a.Hq + h) * a.Lq + t] = none ? 0.f : -(mm + lg2(ll)) * kLn2;
            } else {
                const long long part = ((long long)blockIdx.x + bh) * rows + r;
                a.part_o[part * 64 + d] = y;
                if (d == 0) a.part_ml[part] = make_float2(mm, ll);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// bf16
namespace mma {
constexpr int STAGES = 6;                   // groups of 16 keys and values in flight, per warp
constexpr int STAGE = 2 * 16 * 128;         // bytes
constexpr int WARPS = THREADS_MMA / 32;
constexpr int SMEM = WARPS * STAGES * STAGE;

__device__ __forceinline__ void ldm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose(uint32_t x) {  // of an 8 x 8 tile of 16-bit elements
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// NT: tiles of eight rows.
template <int NT>
__global__ void __launch_bounds__(THREADS_MMA, 2) k_token(const Args a) {
    using T = __nv_bfloat16;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float so[WARPS][NT * 8][64];
    __shared__ float2 sml[WARPS][NT * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;  // of the fragments: S^T[key g, g + 8][row 2t, 2t + 1]
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const int rows = a.G * a.Lq;
    const uint32_t mine = tc::smem_u32(ring) + warp * STAGES * STAGE;
    // a group's row (key) r keeps its 16-byte piece c at c ^ (r & 7): eight rows of
    // a matrix then lie in eight different banks' quadruples
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t ka = (mr + 8 * (mi & 1)) * 128, va = (mr + 8 * (mi >> 1)) * 128;
    Share sh(a);
    while (sh.next(a)) {
        const int b = sh.b, hk = sh.hk, k0 = sh.k0, k1 = sh.k1;
        // Q^T as the B operand: row n = g of each tile, channels 16 kk + 2t (+ 8)
        uint32_t qf[NT][4][2];
        int lo[NT][2], hi[NT][2], wlo = 0, whi = 0x7fffffff;
        float m[NT][2], l[NT][2], o[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            const uint32_t* q =
                r < rows ? reinterpret_cast<const uint32_t*>(a.q.at<T>(b, hk * a.G + r / a.Lq, r % a.Lq)) : nullptr;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                qf[n][kk][0] = q ? q[8 * kk + t] : 0u;
                qf[n][kk][1] = q ? q[8 * kk + 4 + t] : 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][kk][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // this lane's rows: their bands, running maxima and sums
                const int x = 8 * n + 2 * t + e;
                lo[n][e] = 0;
                hi[n][e] = -1;
                if (x < rows) {
                    const long long p = a.first(b) + x % a.Lq;
                    if (p >= 0 && p < a.Lk && a.live(b, (int)p)) a.keys(p, lo[n][e], hi[n][e]);
                    wlo = max(wlo, lo[n][e]);
                    whi = min(whi, hi[n][e]);
                }
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
            }
        }
        wlo = __reduce_max_sync(~0u, wlo);
        whi = __reduce_min_sync(~0u, whi);
        const uint8_t* pm = a.mask ? a.mask + (long long)b * a.Lk : nullptr;
        const T* kp = a.k.at<T>(b, hk, 0) + 8 * mr;
        const T* vp = a.v.at<T>(b, hk, 0) + 8 * mr;
        // group i of this warp: keys k0 + 16 warp + 64 i ..; a lane brings piece mr
        // of keys mi, mi + 4, mi + 8, mi + 12
        const int ng = (k1 - (k0 + 16 * warp) + 63) / 64;
        auto fetch = [&](int i) {
            const uint32_t d = mine + (i % STAGES) * STAGE;
            const int j0 = k0 + 16 * warp + 64 * i + mi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = mi + 4 * e, j = j0 + 4 * e;
                const bool on = i < ng && j < k1 && (pm == nullptr || pm[j] != 0);
                const long long jj = on ? j : 0;  // an address inside the tensor, not read
                const uint32_t w = d + r * 128 + ((mr ^ (r & 7)) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(w), "l"(kp + jj * a.k.s[2]),
                             "r"(on ? 16 : 0)
                             : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(w + 2048), "l"(vp + jj * a.v.s[2]),
                             "r"(on ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = 0; i < STAGES - 1; ++i) fetch(i);
        for (int i = 0; i < ng; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncwarp();  // every lane's pieces of this group; and all have read the one before
            fetch(i + STAGES - 1);
            const uint32_t st = mine + (i % STAGES) * STAGE;
            const int j0 = k0 + 16 * warp + 64 * i;
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t x[4];
                ldm(x, st + ka + (((2 * kk + (mi >> 1)) ^ mr) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(s[n], x, qf[n][kk][0], qf[n][kk][1]);
            }
            const bool full = j0 >= wlo && j0 + 15 <= whi && j0 + 15 < k1 && pm == nullptr;
            uint32_t pf[NT][2];
            bool move = false;
            float mx[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // key g + 8 (e >> 1), row 2t + (e & 1)
                    s[n][e] *= a.c2;
                    if (!full) {
                        const int j = j0 + g + 8 * (e >> 1);
                        if (!(j >= lo[n][e & 1] && j <= hi[n][e & 1] && j < k1 && (pm == nullptr || pm[j] != 0)))
                            s[n][e] = -INFINITY;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[n][e] = fmaxf(s[n][e], s[n][e + 2]);
                    move = move || mx[n][e] > m[n][e] + 8.f;
                }
            }
            if (__any_sync(~0u, move)) {  // all rows' maxima to what they are now
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(mx[n][e], m[n][e]);
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                        const float f = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - x);
                        m[n][e] = x;
                        l[n][e] *= f;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            o[n][kk][e] *= f;
                            o[n][kk][e + 2] *= f;
                        }
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float mm = m[n][e & 1];
                    p[e] = ex2(s[n][e] - (mm == -INFINITY ? 0.f : mm));
                    l[n][e & 1] += p[e];
                }
                // P[key][row] of the accumulator's layout as the B operand's
                pf[n][0] = transpose(tc::pack_bf16(p[0], p[1]));
                pf[n][1] = transpose(tc::pack_bf16(p[2], p[3]));
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // channels 16 kk ..
                uint32_t x[4];
                ldm_t(x, st + 2048 + va + (((2 * kk + (mi & 1)) ^ mr) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(o[n][kk], x, pf[n][0], pf[n][1]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[n][e];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                const int r = 8 * n + 2 * t + e;
                // NaN among the scores: the sum is one, and the maximum must not say "none"
                if (g == 0) sml[warp][r] = make_float2(x != x && m[n][e] == -INFINITY ? 0.f : m[n][e], x);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    so[warp][r][16 * kk + g] = o[n][kk][e];
                    so[warp][r][16 * kk + g + 8] = o[n][kk][e + 2];
                }
            }
        __syncthreads();
        for (int x = threadIdx.x; x < rows * 64; x += THREADS_MMA) {
            const int r = x >> 6, d = x & 63;
            float mm = -INFINITY, ll = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, sml[w][r].x);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 z = sml[w][r];
                if (z.x == -INFINITY) continue;
                const float f = ex2(z.x - mm);
                ll = fmaf(z.y, f, ll);
                y = fmaf(so[w][r][d], f, y);
            }
            const int bh = b * a.Hk + hk;
            if (sh.whole) {  // all of the row's keys: the result itself
                const bool none = mm == -INFINITY;
                const int h = hk * a.G + r / a.Lq, tt = r % a.Lq;
                store_elem(a.o.at<T>(b, h, tt) + d, none ? 0.f : y / ll);
                if (d == 0) a.u[((long long)b * a.Hq + h) * a.Lq + tt] = none ? 0.f : -(mm + lg2(ll)) * kLn2;
            } else {
                const long long part = ((long long)blockIdx.x + bh) * rows + r;
                a.part_o[part * 64 + d] = y;
                if (d == 0) a.part_ml[part] = make_float2(mm, ll);
            }
        }
        __syncthreads();
    }
}
}  // namespace mma

// The rows whose keys several blocks (of nblocks) shared, and those without a
// key; one warp per row, two channels per lane.  Part i + bh is block i's of the
// pair bh: no two blocks and pairs share a number along the line.
template <typename T>
__global__ void __launch_bounds__(128) k_token_join(const Args a, int nblocks) {
    const int rows = a.G * a.Lq, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    tc::grid_dep_wait();
    if (row >= (long long)a.B * a.Hk * rows) return;
    const int r = (int)(row % rows), bh = (int)(row / rows), b = bh / a.Hk, hk = bh % a.Hk;
    const int h = hk * a.G + r / a.Lq, t = r % a.Lq;
    const long long total = Line::before(a, a.B) * a.Hk;
    const int n = Line::chunks(a, b);
    int i0 = 0, i1 = -1;
    if (n > 0) {
        const long long s = Line::before(a, b) * a.Hk + (long long)hk * n;
        const int shares = share_count(total, nblocks);
        i0 = share_of(s, total, shares);
        i1 = share_of(s + n - 1, total, shares);
        if (i0 == i1) return;  // one block had all of it
    }
    float m = -INFINITY, l = 0.f;
    for (int i = i0 + lane; i <= i1; i += 32) {
        const float2 x = a.part_ml[((long long)i + bh) * rows + r];
        lse_merge(m, l, x.x, x.y);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        const float m2 = __shfl_xor_sync(~0u, m, x), l2 = __shfl_xor_sync(~0u, l, x);
        lse_merge(m, l, m2, l2);
    }
    float2 o = make_float2(0.f, 0.f);
    for (int i = i0; i <= i1; i += 32) {  // a part's weight in each lane, then their rows
        float w = 0.f;
        if (i + lane <= i1) {
            const float x = a.part_ml[((long long)i + lane + bh) * rows + r].x;
            w = x == -INFINITY ? 0.f : ex2(x - m);
        }
        const int c = min(32, i1 - i + 1);
#pragma unroll 8
        for (int e = 0; e < c; ++e) {
            const float we = __shfl_sync(~0u, w, e);
            const float2 y = reinterpret_cast<const float2*>(a.part_o + (((long long)i + e + bh) * rows + r) * 64)[lane];
            o.x = fmaf(we, y.x, o.x);
            o.y = fmaf(we, y.y, o.y);
        }
    }
    const bool none = m == -INFINITY;
    const float inv = none ? 0.f : 1.f / l;
    T* out = a.o.at<T>(b, h, t) + 2 * lane;
    store_elem(out, o.x * inv);
    store_elem(out + 1, o.y * inv);
    if (lane == 0) a.u[((long long)b * a.Hq + h) * a.Lq + t] = none ? 0.f : -(m + lg2(l)) * kLn2;
}

}  // namespace token
}  // namespace sm
}  // namespace sa
