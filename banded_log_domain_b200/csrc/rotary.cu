// Rotary positions of queries and keys (sinkhorn_attn_rotary_*).
//
// A thread owns one 16-byte piece of a token's rotated channels (two pieces, x_a
// and x_b, in the half layout) or of its copied ones, forms the piece's
// cosines and sines once, and applies them to the same piece of several heads:
// the angle p * f is reduced in double, so far positions lose nothing.
// Bound by HBM: every element is read and written once (262144 tokens, 8 + 8 heads,
// bf16, backward: 188-194 us, 5.5-5.7 TB/s of the 6.5 that a copy reaches; 32768 tokens of
// 16 + 16 heads from a [B][L][H][d] projection 57 us, 4.7 TB/s, of which the kernel is 54:
// a warp's loads there lie 2 KB apart, 64 to 128 bytes at a time).
#include <cmath>
#include <algorithm>

#include "common.cuh"
#include "host_util.cuh"

namespace sa {
namespace {

struct RotArgs {
    const void *q, *k;
    void *qo, *ko;
    long long qs[3], ks[3], qos[3], kos[3];  // element strides: batch, head, token
    const double* freqs;
    const int* pos;
    int Hq, H, L, rot, hc;  // H = Hq + Hk; hc heads per thread
    int nrot;               // pieces of the rotated channels; the others are copied
    float scale;
    int inverse;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Piece {
    T x[N];
};

// Sine and cosine of the angle p f.  For fp32 results the product is held in two
// doubles and reduced by n turns with 2 pi in two parts (Cody and Waite), so that
// nothing is lost for |p f| up to 2^31 and beyond, and what the remainder loses as a
// float, 2^-23.4 of a radian near half a turn, is put back by the first term of the
// sums' formulas (results off by 2.9e-8; with the short form 3.7e-8 and, at positions
// near 2^31, 3e-7).  bf16 rounds the result at 2^-9: the short form, off by less than
// 2^-20, saves 2 % of the kernel's time there.
template <bool FULL>
__device__ __forceinline__ void sincos_of(double p, double f, float& s, float& c) {
    const double x = p * f;
    if (!FULL) {
        const double turns = x * 0.15915494309189533577;  // 1 / (2 pi)
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        return;
    }
    const double n = rint(x * 0.15915494309189533577);
    double r = fma(-n, 6.283185307179586232, x);
    r = fma(-n, 2.449293598294706414e-16, r) + fma(p, f, -x);
    const float h = (float)(r * 0.31830988618379067154);  // half turns
    const float d = (float)fma(-(double)h, 3.14159265358979323846, r);
    float s0, c0;
    sincospif(h, &s0, &c0);
    s = fmaf(c0, d, s0);
    c = fmaf(-s0, d, c0);
}

// NP pairs per thread; HALF: the pair's channels are two pieces of NP elements,
// else one piece of 2 NP.  The heads are taken U at a time, all their loads first;
// the sines are formed while the first ones are on their way.
template <typename T, int NP, bool HALF>
__global__ void __launch_bounds__(256) k_rotary(const RotArgs a) {
    constexpr int NV = HALF ? NP : 2 * NP;  // elements of a piece
    // bf16 has twice the pairs, and sines, in a thread (there 4 heads took 2 % longer)
    constexpr int U = sizeof(T) == 4 ? 4 : 1;
    const int t = blockIdx.x * blockDim.y + threadIdx.y, unit = threadIdx.x, b = blockIdx.z;
    if (t >= a.L) return;
    const int h0 = blockIdx.y * a.hc, h1 = min(a.H, h0 + a.hc);
    const bool turn = unit < a.nrot;
    // first channel of the piece (of its x_a in the half layout)
    const int ch = turn ? unit * NV : a.rot + (unit - a.nrot) * NV;
    const int half = turn && HALF ? a.rot / 2 : 0;  // x_b's distance
    float cs[NP], sn[NP];
    for (int h = h0; h < h1; h += U) {
        Piece<T, NV> x[U], y[HALF ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u >= h1) break;
            const bool isq = h + u < a.Hq;
            const int hh = isq ? h + u : h + u - a.Hq;
            const long long* is = isq ? a.qs : a.ks;
            const T* in = (const T*)(isq ? a.q : a.k) + b * is[0] + hh * is[1] + t * is[2] + ch;
            x[u] = *reinterpret_cast<const Piece<T, NV>*>(in);
            if (HALF) y[HALF ? u : 0] = *reinterpret_cast<const Piece<T, NV>*>(in + half);
        }
        if (h == h0 && turn) {
            const double p = a.pos ? (double)a.pos[(long long)b * a.L + t] : (double)t;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float s, c;
                sincos_of<sizeof(T) == 4>(p, a.freqs[unit * NP + i], s, c);
                cs[i] = c * a.scale;
                sn[i] = (a.inverse ? -s : s) * a.scale;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u >= h1) break;
            if (turn) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    T* pa = HALF ? &x[u].x[i % NV] : &x[u].x[2 * i % NV];
                    T* pb = HALF ? &y[HALF ? u : 0].x[i % NV] : &x[u].x[(2 * i + 1) % NV];
                    const float xa = to_f32(*pa), xb = to_f32(*pb);
                    store_elem(pa, xa * cs[i] - xb * sn[i]);
                    store_elem(pb, xa * sn[i] + xb * cs[i]);
                }
            }
            const bool isq = h + u < a.Hq;
            const int hh = isq ? h + u : h + u - a.Hq;
            const long long* os = isq ? a.qos : a.kos;
            T* out = (T*)(isq ? a.qo : a.ko) + b * os[0] + hh * os[1] + t * os[2] + ch;
            *reinterpret_cast<Piece<T, NV>*>(out) = x[u];
            if (HALF && turn) *reinterpret_cast<Piece<T, NV>*>(out + half) = y[HALF ? u : 0];
        }
    }
}

template <typename T, int NP, bool HALF>
cudaError_t launch_rotary(RotArgs a, int B, int d, cudaStream_t st) {
    constexpr int NV = HALF ? NP : 2 * NP;
    a.nrot = a.rot / (2 * NP);
    const int units = a.nrot + (d - a.rot) / NV;
    const int ty = std::max(1, 128 / units);
    // Heads per thread: up to 8 share one set of sines, as long as about half
    // the threads that the GPU holds remain.
    const long long all = (long long)B * a.L * units * a.H;
    a.hc = (int)std::min<long long>(8, std::max<long long>(1, all / (148LL * 1024)));
    const dim3 grid((unsigned)((a.L + ty - 1) / ty), (unsigned)((a.H + a.hc - 1) / a.hc), (unsigned)B);
    k_rotary<T, NP, HALF><<<grid, dim3(units, ty), 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rotary_t(const RotArgs& a, int B, int d, bool half, cudaStream_t st) {
    // 16-byte pieces where they fit the rotated channels, else pair by pair
    constexpr int V = 16 / sizeof(T);
    if (half) {
        if (a.rot % (2 * V) == 0) return launch_rotary<T, V, true>(a, B, d, st);
        return launch_rotary<T, 1, true>(a, B, d, st);
    }
    if (a.rot % V == 0) return launch_rotary<T, V / 2, false>(a, B, d, st);
    return launch_rotary<T, 1, false>(a, B, d, st);
}

// The strides of a [B][H][L][d] tensor (three zeros: contiguous); false unless
// each is a positive multiple of 16 bytes (extents of 1 are not looked at).
bool strides(const long long s[3], int B, int H, int L, int d, int size, long long out[3]) {
    const long long n[3] = {B, H, L};
    if (!s[0] && !s[1] && !s[2]) {
        out[2] = d;
        out[1] = (long long)L * d;
        out[0] = (long long)H * L * d;
        return true;
    }
    for (int i = 0; i < 3; ++i) {
        out[i] = n[i] > 1 ? s[i] : 0;
        if (n[i] > 1 && (s[i] <= 0 || (s[i] * size) % 16 != 0 || s[i] > (1LL << 38))) return false;
    }
    return true;
}

sa_status rotary_call(const sa_rotary_params* p, const double* freqs, const int* pos, const void* q,
                      const void* k, void* qo, void* ko, void* stream, int inverse) {
    if (!p) return SA_ERR_INVALID_ARG;
    if (p->B < 0 || p->Hq < 0 || p->Hk < 0 || p->L < 0 || p->d <= 0) return SA_ERR_INVALID_ARG;
    if (p->rot < 2 || p->rot % 2 || p->rot > p->d) return SA_ERR_INVALID_ARG;
    if (p->interleaved != 0 && p->interleaved != 1) return SA_ERR_INVALID_ARG;
    if (p->dtype != SA_F32 && p->dtype != SA_BF16) return SA_ERR_INVALID_ARG;
    if (!std::isfinite(p->scale)) return SA_ERR_INVALID_ARG;
    if (p->d % 8 || p->d > 256 || p->B > 65535 || (long long)p->Hq + p->Hk > 65535 || p->L > (1 << 30))
        return SA_ERR_UNSUPPORTED;  // (token indices stay clear of 2^31 with a block's rows added)
    const int size = p->dtype == SA_F32 ? 4 : 2;
    RotArgs a;
    if (!strides(p->q_stride, p->B, p->Hq, p->L, p->d, size, a.qs) ||
        !strides(p->k_stride, p->B, p->Hk, p->L, p->d, size, a.ks) ||
        !strides(p->q_out_stride, p->B, p->Hq, p->L, p->d, size, a.qos) ||
        !strides(p->k_out_stride, p->B, p->Hk, p->L, p->d, size, a.kos))
        return SA_ERR_INVALID_ARG;
    if (p->B == 0 || p->L == 0 || p->Hq + p->Hk == 0) return SA_OK;
    if ((p->Hq > 0 && (!device_ok(q) || !device_ok(qo))) || (p->Hk > 0 && (!device_ok(k) || !device_ok(ko))))
        return SA_ERR_INVALID_ARG;
    if (!freqs || ((uintptr_t)freqs & 7) || !on_current_device(freqs)) return SA_ERR_INVALID_ARG;
    if (pos && (((uintptr_t)pos & 3) || !on_current_device(pos))) return SA_ERR_INVALID_ARG;
    a.q = q;
    a.k = k;
    a.qo = qo;
    a.ko = ko;
    a.freqs = freqs;
    a.pos = pos;
    a.Hq = p->Hq;
    a.H = p->Hq + p->Hk;
    a.L = p->L;
    a.rot = p->rot;
    a.scale = p->scale;
    a.inverse = inverse;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p->dtype == SA_F32
                              ? launch_rotary_t<float>(a, p->B, p->d, !p->interleaved, st)
                              : launch_rotary_t<__nv_bfloat16>(a, p->B, p->d, !p->interleaved, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace
}  // namespace sa

extern "C" {

sa_status sinkhorn_attn_rotary_fwd(const sa_rotary_params* p, const double* freqs, const int* pos,
                                   const void* q, const void* k, void* q_out, void* k_out, void* stream) {
    return sa::rotary_call(p, freqs, pos, q, k, q_out, k_out, stream, 0);
}

sa_status sinkhorn_attn_rotary_bwd(const sa_rotary_params* p, const double* freqs, const int* pos,
                                   const void* dq, const void* dk, void* dq_in, void* dk_in, void* stream) {
    return sa::rotary_call(p, freqs, pos, dq, dk, dq_in, dk_in, stream, 1);
}

sa_status sinkhorn_attn_rotary_freqs(int rot, double base, sa_rotary_scaling kind, double factor,
                                     double train_len, double turns_hi, double turns_lo, double* freqs,
                                     float* scale) {
    if (rot < 2 || rot % 2 || !freqs) return SA_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor)) return SA_ERR_INVALID_ARG;
    if (kind < SA_ROTARY_PLAIN || kind > SA_ROTARY_BY_PARTS) return SA_ERR_INVALID_ARG;
    const int n = rot / 2;
    double lo = 0.0, hi = 0.0;
    if (kind == SA_ROTARY_BY_PARTS) {
        if (!(train_len > 0.0) || !std::isfinite(train_len) || !(turns_lo > 0.0) || !(turns_hi > turns_lo) ||
            !std::isfinite(turns_hi))
            return SA_ERR_INVALID_ARG;
        // the pair index at which train_len tokens make `turns` whole turns
        auto at = [&](double turns) {
            return n * std::log(train_len / (turns * 2.0 * 3.14159265358979323846)) / std::log(base);
        };
        // The ramp starts at the first pair at the earliest, but may end behind the
        // last (YaRN's bound is rot - 1): pairs that still turn more than turns_lo
        // times are mixed, not divided by the whole factor.
        lo = std::max(0.0, std::floor(at(turns_hi)));
        hi = std::min(rot - 1.0, std::ceil(at(turns_lo)));
    }
    if (kind == SA_ROTARY_NTK && n > 1) base *= std::pow(factor, (double)n / (n - 1));
    for (int i = 0; i < n; ++i) {
        double f = std::pow(base, -(double)i / n);
        if (kind == SA_ROTARY_LINEAR) f /= factor;
        if (kind == SA_ROTARY_BY_PARTS) {
            // (hi <= lo: every pair lies on one side of the ramp)
            const double ramp = hi > lo ? std::min(1.0, std::max(0.0, (i - lo) / (hi - lo))) : i >= hi ? 1.0 : 0.0;
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        freqs[i] = f;
    }
    if (scale) *scale = kind == SA_ROTARY_BY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return SA_OK;
}

}  // extern "C"
