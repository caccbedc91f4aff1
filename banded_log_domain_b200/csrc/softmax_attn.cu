// C ABI of the softmax attention (sinkhorn_attn_softmax_*): argument
// validation, the launch plan and the launches.
#include <cmath>
#include <algorithm>
#include <cstring>

#include "host_util.cuh"
#include "softmax.cuh"
#include "softmax_simt.cuh"
#include "softmax_tf32.cuh"
#include "softmax_tc.cuh"
#include "softmax_tc_bwd.cuh"
#include "softmax_token.cuh"

namespace sa {
namespace {

constexpr int kD = 64;
constexpr int kMaxGroup = 64;   // query heads per key head (they share a tile's rows)

// How a call is cut: tiles of `nq` queries x the group's heads, `nr` tiles (`per`
// queries) to a forward item, its keys in `nsplit` parts.
struct Plan {
    bool tc;
    int G, nq, rpt, nr, per, ntile, nktile, nsplit, nparts;
    int token;  // blocks of the single-token forward, 0 where it does not apply
    long long rows;  // B * Hq * Lq
    int qsplit, ksplit;  // parts of the fp32 backward's tiles
    size_t fwd_bytes, bwd_bytes, bwd_part, part_ml, span;  // span: in either workspace
};

sa_status make_plan(const sa_softmax_params* p, Plan* pl) {
    if (!p) return SA_ERR_INVALID_ARG;
    if (p->B < 0 || p->Hq < 0 || p->Hk < 0 || p->Lq < 0 || p->Lk < 0 || p->d <= 0 || p->W < 0)
        return SA_ERR_INVALID_ARG;
    if (!(p->eps > 0.f) || !std::isfinite(p->eps)) return SA_ERR_INVALID_ARG;
    if (p->causal != 0 && p->causal != 1) return SA_ERR_INVALID_ARG;
    if (p->dtype != SA_F32 && p->dtype != SA_BF16) return SA_ERR_INVALID_ARG;
    if (p->Lq > p->Lk) return SA_ERR_INVALID_ARG;
    if (p->Hk == 0 ? p->Hq != 0 : p->Hq % p->Hk != 0) return SA_ERR_INVALID_ARG;
    if (p->d != kD) return SA_ERR_UNSUPPORTED;
    // u / c and 1 / c stay far from fp32's ends (the backward forms both)
    if (p->eps < 0x1p-100f || p->eps > 0x1p100f) return SA_ERR_UNSUPPORTED;
    pl->G = p->Hk ? std::max(1, p->Hq / p->Hk) : 1;
    if (pl->G > kMaxGroup) return SA_ERR_UNSUPPORTED;
    // token indices stay clear of 2^31 with a tile's rows added
    if (p->Lk > (1 << 30) || (long long)p->B * p->Hq > 65535) return SA_ERR_UNSUPPORTED;
    pl->rows = (long long)p->B * p->Hq * p->Lq;
    pl->tc = p->dtype == SA_BF16;
    const int sms = sm_count();
    const long long BH = (long long)p->B * p->Hk;
    const long long W = std::min(p->W, p->Lk), span = W + (p->causal ? 0 : W);
    // fp32 tiles of 64 rows on matrix instructions (softmax_tf32.cuh); of 32 or 16
    // on the FMA pipe (softmax_simt.cuh) where even those leave half of the SMs free
    // (one kernel's blocks are placed while the last one's are there: twice as many
    // share SMs and take twice as long) and a row's keys are too few to be cut into
    // parts instead.  Backward with tiles of 16, 32, 64 rows, W = 64: 512 tokens of a
    // head 39, 46, 72 us; 1024 of two 64, 46, 72; 2048 of two 65, 75, 74.
    const long long t64 = BH * ((p->Lq + 64 / pl->G - 1) / (64 / pl->G));
    const bool few = span <= 384;
    pl->rpt = few && pl->G <= 16 && 8 * t64 <= sms ? 1 : few && pl->G <= 32 && 4 * t64 <= sms ? 2 : 4;
    pl->nq = (pl->tc ? 128 : 16 * pl->rpt) / pl->G;
    const long long RT = (p->Lq + pl->nq - 1) / pl->nq;  // row tiles
    // The tensor-core forward's items are 4, 2 or 1 row tiles (see softmax_tc.cuh).
    // One leaves the fewest SMs idle where all tiles fit them at once; of many, two
    // share the key chunks (32768 tokens of 16 heads, W = 256: 187 us, four 191, one
    // 237).  Four on long bands of many tiles: us with four and two on 8192 dense
    // tokens 439, 465; 32768 with W = 4096 1436, 1469; 32768 causal ones of 4 key heads
    // 2919, 2980.  Not everywhere: there are half as many items to share out (16384 dense
    // tokens of 4 key heads 1664, 1529; 8191 causal ones 254, 235).
    pl->nr = 1;
    if (pl->tc && BH * RT > sms) pl->nr = W >= 4096 && BH * RT >= 6LL * sms ? 4 : 2;
    pl->per = pl->nr * pl->nq;
    pl->ntile = (int)((RT + pl->nr - 1) / pl->nr);
    pl->nktile = (p->Lk + 16 * pl->rpt - 1) / (16 * pl->rpt);
    const long long tiles = BH * pl->ntile;
    if (std::max(tiles, BH * pl->nktile) > (1LL << 30)) return SA_ERR_UNSUPPORTED;
    // A few query rows over many keys (single new tokens) would leave most SMs
    // idle: then every tile's keys are cut into parts for about two blocks an
    // SM, of at least four (bf16: eight) chunks each, joined by a second kernel.
    // 64 query tokens of 8 heads over 32768: 32 us, not cut 199; 2048 dense fp32
    // tokens of one head: 44 us, not cut 208.
    const long long keys = std::min<long long>(p->Lk, span + pl->per);
    const long long chunks = (keys + 63) / 64;
    pl->nsplit = 1;
    if (tiles > 0 && tiles < sms)
        pl->nsplit = (int)std::max<long long>(1, std::min(2LL * sms / tiles, chunks / (pl->tc ? 8 : 4)));
    pl->nparts = pl->nsplit;
    long long parts = pl->nparts > 1 ? pl->rows * pl->nparts : 0;
    // Few query rows per key head are bound by reading the keys and
    // values: a kernel without tiles, whose blocks (two per SM, of two chunks or
    // more) share all sequences' chunks evenly (4 key heads of 4 heads each, us here
    // and tiled: 8 sequences of up to 32768 tokens, bf16 61, 86, fp32 152, 422; 64 of
    // 8192, bf16 98, 199, fp32 244, 944).  Its limits on rows and sequences: see there.
    pl->token = 0;
    if ((long long)pl->G * p->Lq <= sm::token::max_rows(pl->tc) && p->B <= sm::token::MAXB && BH <= 4096 && BH > 0) {
        pl->token = (int)std::max<long long>(1, std::min<long long>(2LL * sms, BH * chunks / 2));
        parts = (pl->token + BH) * pl->G * p->Lq;
    }
    pl->span = kHeader;
    const size_t head = kHeader + align_up((size_t)p->B * 8);
    pl->part_ml = head + align_up((size_t)parts * kD * 4);
    pl->fwd_bytes = pl->part_ml + align_up((size_t)parts * 8);
    // the fp32 backward's tiles, where few, are cut likewise (2048 dense tokens of
    // one head: 122 us, not cut 596; the sums take two short kernels)
    const long long kchunks = (std::min<long long>(p->Lq, span + 64) + 63) / 64 * pl->G, kt = BH * pl->nktile;
    pl->qsplit = pl->ksplit = 1;
    if (!pl->tc && pl->rows > 0 && tiles < sms)
        pl->qsplit = (int)std::max<long long>(1, std::min(2LL * sms / tiles, chunks / 3));
    if (!pl->tc && pl->rows > 0 && kt < sms)
        pl->ksplit = (int)std::max<long long>(1, std::min(2LL * sms / kt, kchunks / 3));
    const long long qparts = pl->qsplit > 1 ? pl->rows * pl->qsplit * 64 : 0;
    const long long kparts = pl->ksplit > 1 ? BH * p->Lk * pl->ksplit * 128 : 0;
    pl->bwd_part = head + align_up((size_t)pl->rows * (pl->tc ? 32 : 4));
    pl->bwd_bytes = pl->bwd_part + align_up((size_t)std::max(qparts, kparts) * 4);
    return SA_OK;
}

// A [B][H][L][64] tensor's strides (three zeros: contiguous); false unless each
// is a positive multiple of 16 bytes (extents of 1 are not looked at).
bool view(sm::View* v, const void* ptr, const long long s[3], int B, int H, int L, int size) {
    v->p = const_cast<void*>(ptr);
    if (!s[0] && !s[1] && !s[2]) {
        v->s[2] = kD;
        v->s[1] = (long long)L * kD;
        v->s[0] = (long long)H * L * kD;
        return true;
    }
    const long long n[3] = {B, H, L};
    for (int i = 0; i < 3; ++i) {
        v->s[i] = n[i] > 1 ? s[i] : 0;
        if (n[i] > 1 && (s[i] <= 0 || (s[i] * size) % 16 != 0 || s[i] > (1LL << 38))) return false;
    }
    return true;
}

// A call with nothing to do launches no kernel that would reset the status word.
sa_status reset_status(void* ws, void* stream) {
    if (!device_ok(ws)) return SA_OK;  // an empty call needs no workspace
    return cudaMemsetAsync(ws, 0, 4, (cudaStream_t)stream) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

bool ints_ok(const int* x) { return !x || (((uintptr_t)x & 3u) == 0 && on_current_device(x)); }

// Every kernel here is launched with programmatic stream serialisation and waits
// (griddepcontrol.wait) before any global access.
template <typename K>
cudaError_t launch(K kern, long long grid, int threads, int smem, cudaStream_t st, const sm::Args& a) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, dim3((unsigned)grid), dim3(threads), smem, st, a);
}

void base_args(sm::Args* a, const sa_softmax_params* p, const Plan& pl, const uint8_t* mask, const int* q_pos,
               void* ws) {
    a->B = p->B;
    a->Hq = p->Hq;
    a->Hk = p->Hk;
    a->G = pl.G;
    a->Lq = p->Lq;
    a->Lk = p->Lk;
    a->W = std::min(p->W, p->Lk);
    a->R = p->causal ? 0 : a->W;
    a->c = 1.0f / (std::sqrt((float)p->d) * p->eps);
    a->c2 = a->c * kLog2e;
    a->q_pos = q_pos;
    a->mask = mask;
    a->status = (int*)ws;
    a->span = (int2*)((char*)ws + pl.span);
    a->nq = pl.nq;
    a->ntile = pl.ntile;
    a->nsplit = 1;
    a->nparts = 1;
}

cudaError_t fwd_f32(const sa_softmax_params* p, const Plan& pl, const sm::Args& a, cudaStream_t st) {
    namespace simt = sm::simt;
    const long long grid = (long long)p->B * p->Hk * pl.ntile * pl.nsplit;
    if (pl.rpt == 4) return launch(sm::tf32::k_fwd, grid, sm::tf32::THREADS, sm::tf32::smem_bytes(5), st, a);
    return launch(pl.rpt == 2 ? simt::k_fwd<2> : simt::k_fwd<1>, grid, simt::THREADS, simt::smem_bytes(pl.rpt, 2, 4), st,
                  a);
}

// One sweep of the fp32 backward: dQ, or dK and dV.
cudaError_t sweep_f32(int rpt, bool kv, long long grid, const sm::Args& a, cudaStream_t st) {
    namespace simt = sm::simt;
    namespace tf32 = sm::tf32;
    if (rpt == 4) return launch(kv ? tf32::k_bwd_kv : tf32::k_bwd_q, grid, tf32::THREADS, tf32::smem_bytes(6), st, a);
    auto kern = kv ? (rpt == 2 ? simt::k_bwd_kv<2> : simt::k_bwd_kv<1>) : (rpt == 2 ? simt::k_bwd_q<2> : simt::k_bwd_q<1>);
    return launch(kern, grid, simt::THREADS, simt::smem_bytes(rpt, kv ? 4 : 3, 4), st, a);
}

cudaError_t bwd_f32(const sa_softmax_params* p, const Plan& pl, sm::Args& a, cudaStream_t st) {
    const long long BH = (long long)p->B * p->Hk;
    auto sum = [&](long long rows, int kv) {
        return launch_pdl(sm::simt::k_sum, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, a, kv);
    };
    a.nsplit = pl.qsplit;
    cudaError_t e = sweep_f32(pl.rpt, false, BH * a.ntile * a.nsplit, a, st);
    if (e == cudaSuccess && a.nsplit > 1) e = sum(pl.rows, 0);
    if (e != cudaSuccess) return e;
    a.ntile = pl.nktile;
    a.nsplit = pl.ksplit;
    e = sweep_f32(pl.rpt, true, BH * a.ntile * a.nsplit, a, st);
    if (e == cudaSuccess && a.nsplit > 1) e = sum(BH * p->Lk, 1);
    return e;
}

// A [B][H][L][64] bf16 view as a 4-D tensor; boxes of `tokens` x `heads` rows.
bool make_map(CUtensorMap* m, const sm::View& v, int B, int H, int L, int tokens, int heads) {
    auto fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[4] = {kD, (cuuint64_t)L, (cuuint64_t)H, (cuuint64_t)B};
    cuuint64_t strides[3];
    const int n[3] = {L, H, B};
    for (int i = 0; i < 3; ++i) strides[i] = n[i] > 1 ? (cuuint64_t)v.s[2 - i] * 2 : kD * 2;
    cuuint32_t box[4] = {kD, (cuuint32_t)tokens, (cuuint32_t)heads, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Persistent: one block per SM, each a share of the items.
template <int NR>
cudaError_t fwd_tc(const sa_softmax_params* p, const Plan& pl, const sm::Args& a, cudaStream_t st) {
    using namespace sm::tcf::fwd;
    Maps maps;
    if (!make_map(&maps.Q, a.q, p->B, p->Hq, p->Lq, pl.nq, pl.G) || !make_map(&maps.K, a.k, p->B, p->Hk, p->Lk, 64, 1) ||
        !make_map(&maps.V, a.v, p->B, p->Hk, p->Lk, 64, 1))
        return cudaErrorInvalidValue;
    const long long items = (long long)p->B * p->Hk * pl.ntile * pl.nsplit;
    const unsigned grid = (unsigned)std::min<long long>(items, sm_count());
    constexpr int smem = Lay<NR>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(tc_fwd<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(tc_fwd<NR>, dim3(grid), dim3(THREADS), smem, st, a, maps, (int)items);
    return e;
}

cudaError_t fwd_token(const sa_softmax_params* p, const Plan& pl, const sm::Args& a, cudaStream_t st) {
    using namespace sm::token;
    const int rows = pl.G * p->Lq;
    // both launched with programmatic stream serialisation (they wait for what
    // runs before them), so that the second's launch hides behind the first
    auto go = [&](auto kern, int threads, int smem) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return e != cudaSuccess ? e : launch_pdl(kern, dim3(pl.token), dim3(threads), smem, st, a);
    };
    const cudaError_t e = pl.tc ? go(rows <= 8 ? mma::k_token<1> : mma::k_token<2>, THREADS_MMA, mma::SMEM)
                                : go(rows == 1   ? k_token<1>
                                     : rows == 2 ? k_token<2>
                                                 : k_token<4>, THREADS, SMEM);
    if (e != cudaSuccess || (pl.token == 1 && !a.q_pos && !a.mask)) return e;
    const dim3 grid((unsigned)(((long long)p->B * p->Hk * rows + 3) / 4));
    return launch_pdl(pl.tc ? k_token_join<__nv_bfloat16> : k_token_join<float>, grid, dim3(128), 0, st, a, pl.token);
}

cudaError_t fwd_launch(const sa_softmax_params* p, const Plan& pl, const sm::Args& a, cudaStream_t st) {
    if (pl.token) return fwd_token(p, pl, a, st);
    const cudaError_t e = !pl.tc       ? fwd_f32(p, pl, a, st)
                          : pl.nr == 4 ? fwd_tc<4>(p, pl, a, st)
                          : pl.nr == 2 ? fwd_tc<2>(p, pl, a, st)
                                       : fwd_tc<1>(p, pl, a, st);
    if (e != cudaSuccess || pl.nparts == 1) return e;
    return launch(pl.tc ? sm::k_join<__nv_bfloat16> : sm::k_join<float>, (pl.rows + 3) / 4, 128, 0, st, a);
}

// The queries' further channels, [rows of B Hq][Lq][16] bf16: boxes of 64
// queries, 32-byte swizzle.
bool make_map_aug(CUtensorMap* m, void* p, int L, int BH) {
    auto fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[3] = {16, (cuuint64_t)L, (cuuint64_t)BH};
    cuuint64_t strides[2] = {32, (cuuint64_t)L * 32};
    cuuint32_t box[3] = {16, 64, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t bwd_tc(const sa_softmax_params* p, const sm::Args& a, long long items, cudaStream_t st) {
    using namespace sm::tcf::bwd;
    Maps maps;
    std::memset(&maps, 0, sizeof(maps));
    bool ok = true;
    if (MODE == DQ)
        ok = make_map(&maps.R1, a.q, p->B, p->Hq, p->Lq, a.nq, a.G) && make_map(&maps.R2, a.dO, p->B, p->Hq, p->Lq, a.nq, a.G) &&
             make_map(&maps.C1, a.k, p->B, p->Hk, p->Lk, 64, 1) && make_map(&maps.C2, a.v, p->B, p->Hk, p->Lk, 64, 1);
    else
        ok = make_map(&maps.R1, a.k, p->B, p->Hk, p->Lk, 128, 1) && make_map(&maps.R2, a.v, p->B, p->Hk, p->Lk, 128, 1) &&
             make_map(&maps.C1, a.q, p->B, p->Hq, p->Lq, 64, 1) && make_map(&maps.C2, a.dO, p->B, p->Hq, p->Lq, 64, 1) &&
             make_map_aug(&maps.X, a.aug, p->Lq, p->B * p->Hq);
    if (!ok) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)std::min<long long>(items, sm_count());
    cudaError_t e = cudaFuncSetAttribute(tc_bwd<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess) e = launch_pdl(tc_bwd<MODE>, dim3(grid), dim3(THREADS), SMEM, st, a, maps, (int)items);
    return e;
}

// No query: the keys' gradients are zeros.
cudaError_t zero_grads(const sa_softmax_params* p, sm::Args& a, cudaStream_t st) {
    const long long n = (long long)p->B * p->Hk * p->Lk;
    if (p->dtype == SA_F32) return launch(sm::k_zero<float>, (n + 3) / 4, 128, 0, st, a);
    return launch(sm::k_zero<__nv_bfloat16>, (n + 3) / 4, 128, 0, st, a);
}

cudaError_t bwd_launch(const sa_softmax_params* p, const Plan& pl, sm::Args& a, cudaStream_t st) {
    if (!pl.tc) return bwd_f32(p, pl, a, st);
    const long long BH = (long long)p->B * p->Hk;
    a.nq = pl.nq;
    a.ntile = (p->Lq + a.nq - 1) / a.nq;
    const cudaError_t e = bwd_tc<sm::tcf::bwd::DQ>(p, a, BH * a.ntile, st);
    return e != cudaSuccess ? e : bwd_tc<sm::tcf::bwd::DKV>(p, a, BH * ((p->Lk + 127) / 128), st);
}

}  // namespace
}  // namespace sa

extern "C" {

sa_status sinkhorn_attn_softmax_workspace_size(const sa_softmax_params* p, size_t* fwd_bytes, size_t* bwd_bytes) {
    sa::Plan pl;
    const sa_status s = sa::make_plan(p, &pl);
    if (s != SA_OK) return s;
    if (fwd_bytes) *fwd_bytes = pl.fwd_bytes;
    if (bwd_bytes) *bwd_bytes = pl.bwd_bytes;
    return SA_OK;
}

sa_status sinkhorn_attn_softmax_fwd(const sa_softmax_params* p, const void* q, const void* k, const void* v,
                                    const uint8_t* mask, const int* q_pos, void* o, float* u, void* ws,
                                    size_t ws_bytes, void* stream) {
    using namespace sa;
    Plan pl;
    const sa_status s = make_plan(p, &pl);
    if (s != SA_OK) return s;
    if (ws_bytes < pl.fwd_bytes) return SA_ERR_WORKSPACE;
    const int size = p->dtype == SA_F32 ? 4 : 2;
    sm::Args a;
    base_args(&a, p, pl, mask, q_pos, ws);
    if (!view(&a.q, q, p->q_stride, p->B, p->Hq, p->Lq, size) || !view(&a.k, k, p->k_stride, p->B, p->Hk, p->Lk, size) ||
        !view(&a.v, v, p->v_stride, p->B, p->Hk, p->Lk, size) || !view(&a.o, o, p->o_stride, p->B, p->Hq, p->Lq, size))
        return SA_ERR_INVALID_ARG;
    if (pl.rows == 0) return reset_status(ws, stream);
    if (!device_ok(q) || !device_ok(k) || !device_ok(v) || !device_ok(o) || !device_ok(u) || !device_ok(ws) ||
        !mask_ok(mask) || !ints_ok(q_pos))
        return SA_ERR_INVALID_ARG;
    a.u = u;
    a.nsplit = pl.nsplit;
    a.nparts = pl.nparts;
    a.part_o = (float*)((char*)ws + kHeader + align_up((size_t)p->B * 8));
    a.part_ml = (float2*)((char*)ws + pl.part_ml);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = mask ? launch(sm::k_span, p->B, 1024, 0, st, a) : cudaSuccess;
    if (e == cudaSuccess) e = fwd_launch(p, pl, a, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sinkhorn_attn_softmax_bwd(const sa_softmax_params* p, const void* q, const void* k, const void* v,
                                    const uint8_t* mask, const int* q_pos, const void* o, const void* dO,
                                    const float* u, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                    void* stream) {
    using namespace sa;
    Plan pl;
    const sa_status s = make_plan(p, &pl);
    if (s != SA_OK) return s;
    if (ws_bytes < pl.bwd_bytes) return SA_ERR_WORKSPACE;
    const int size = p->dtype == SA_F32 ? 4 : 2;
    sm::Args a;
    base_args(&a, p, pl, mask, q_pos, ws);
    if (!view(&a.q, q, p->q_stride, p->B, p->Hq, p->Lq, size) || !view(&a.k, k, p->k_stride, p->B, p->Hk, p->Lk, size) ||
        !view(&a.v, v, p->v_stride, p->B, p->Hk, p->Lk, size) || !view(&a.o, o, p->o_stride, p->B, p->Hq, p->Lq, size) ||
        !view(&a.dO, dO, p->dO_stride, p->B, p->Hq, p->Lq, size) ||
        !view(&a.dq, dq, p->dq_stride, p->B, p->Hq, p->Lq, size) ||
        !view(&a.dk, dk, p->dk_stride, p->B, p->Hk, p->Lk, size) ||
        !view(&a.dv, dv, p->dv_stride, p->B, p->Hk, p->Lk, size))
        return SA_ERR_INVALID_ARG;
    if ((long long)p->B * p->Hk * p->Lk == 0) return reset_status(ws, stream);
    if (!device_ok(k) || !device_ok(v) || !device_ok(dk) || !device_ok(dv) || !device_ok(ws) || !mask_ok(mask) ||
        !ints_ok(q_pos))
        return SA_ERR_INVALID_ARG;
    if (pl.rows > 0 && (!device_ok(q) || !device_ok(o) || !device_ok(dO) || !device_ok(u) || !device_ok(dq)))
        return SA_ERR_INVALID_ARG;
    a.u = const_cast<float*>(u);
    a.D = (float*)((char*)ws + kHeader + align_up((size_t)p->B * 8));
    a.aug = (uint4*)a.D;
    a.part_o = (float*)((char*)ws + pl.bwd_part);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = mask && pl.rows > 0 ? launch(sm::k_span, p->B, 1024, 0, st, a) : cudaSuccess;
    if (e == cudaSuccess) e = pl.rows > 0 ? bwd_launch(p, pl, a, st) : zero_grads(p, a, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
