// delta.cu -- the gated delta rule: entry points, the token-by-token kernel
// and the single-token step.
//
//   S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q
//
// The columns of S (the value channels) never mix, so a CTA takes 32 of them
// of one head.  With x = S^T k and y = S^T q of the state before the token,
//   u = beta (v - e^g x),   o = e^g y + (q.k) u,   S <- e^g S + k u^T,
// so both contractions read the same state and one reduction serves both.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "delta.h"
#include "hyena.h"
#include "kernels.h"

namespace hyena {

hyena_status_t set_last_error_detail(hyena_status_t st, const std::string& detail);  // api.cu

namespace {

__device__ __forceinline__ float ld(const float* p, int64_t i) { return __ldg(p + i); }
__device__ __forceinline__ float ld(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void st(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// ------------------------------------------------------------------ sequences
// Token by token.  256 threads: 8 lanes share a column, lane p holding the
// state rows 4 p + 32 j + i (j < J, i < 4), so a lane's k and q come as
// conflict-free 16-byte reads.  Tokens are staged 32 at a time: q, k, v as
// fp32 in shared memory, norms and q.k per token by a warp.  The chain per
// token (two dot products, three shuffles, the update) bounds it, about 0.3 us:
// it serves fp32 storage, where every product is fp32, and a few tokens.
constexpr int kSeqT = 32, kSeqCols = 32, kSeqThreads = 256, kSeqRow = 132;

template <typename T, int J>
__global__ void __launch_bounds__(kSeqThreads) k_delta_seq(DeltaArgs a) {
    __shared__ __align__(16) float sq[kSeqT][kSeqRow];
    __shared__ __align__(16) float sk[kSeqT][kSeqRow];
    __shared__ float sv[kSeqT][kSeqCols + 1];      // values, then outputs
    __shared__ float sa[kSeqT], sb[kSeqT], sqk[kSeqT];
    const int tid = int(threadIdx.x), col = tid >> 3, p = tid & 7;
    const int c0 = int(blockIdx.x) * kSeqCols, h = int(blockIdx.y);
    const int64_t b = blockIdx.z;
    const int kh = h / (a.Hv / a.Hk);
    const T* q = static_cast<const T*>(a.q) + b * a.qs.sb + int64_t(kh) * a.dk * a.qs.sc;
    const T* k = static_cast<const T*>(a.k) + b * a.ks.sb + int64_t(kh) * a.dk * a.ks.sc;
    const T* v = static_cast<const T*>(a.v) + b * a.vs.sb + (int64_t(h) * a.dv + c0) * a.vs.sc;
    T* o = static_cast<T*>(a.o) + b * a.os.sb + (int64_t(h) * a.dv + c0) * a.os.sc;
    const int cols = min(kSeqCols, a.dv - c0);
    int64_t len = a.L;
    if (a.lengths) len = max(int64_t(0), min(a.L, int64_t(a.lengths[b])));

    const bool mine = col < cols;
    const int64_t sbase = ((b * a.Hv + h) * int64_t(a.dk)) * a.dv + c0 + col;
    float S[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * p + 32 * j + i;
            S[j][i] = (a.state_in && mine && r < a.dk) ? a.state_in[sbase + int64_t(r) * a.dv] : 0.0f;
        }

    for (int64_t t0 = 0; t0 < len; t0 += kSeqT) {
        const int n = int(min(int64_t(kSeqT), len - t0));
        for (int i = tid; i < kSeqT * 32 * J; i += kSeqThreads) {
            // the contiguous axis goes over neighbouring threads
            const int t = a.ks.st == 1 ? i % kSeqT : i / (32 * J), c = a.ks.st == 1 ? i / kSeqT : i % (32 * J);
            const bool in = t < n && c < a.dk;
            sq[t][c] = in ? ld(q, (t0 + t) * a.qs.st + c * a.qs.sc) : 0.0f;
            sk[t][c] = in ? ld(k, (t0 + t) * a.ks.st + c * a.ks.sc) : 0.0f;
        }
        for (int i = tid; i < kSeqT * kSeqCols; i += kSeqThreads) {
            const int t = a.vs.st == 1 ? i % kSeqT : i / kSeqCols, c = a.vs.st == 1 ? i / kSeqT : i % kSeqCols;
            sv[t][c] = (t < n && c < cols) ? ld(v, (t0 + t) * a.vs.st + c * a.vs.sc) : 0.0f;
        }
        if (tid < n) {
            sa[tid] = a.g ? expf(a.g[b * a.gs.sb + h * a.gs.sc + (t0 + tid) * a.gs.st]) : 1.0f;
            sb[tid] = a.beta ? a.beta[b * a.bs.sb + h * a.bs.sc + (t0 + tid) * a.bs.st] : 1.0f;
        }
        __syncthreads();
        const int warp = tid >> 5, lane = tid & 31;
        for (int t = warp; t < n; t += kSeqThreads / 32) {
            float q2 = 0.0f, k2 = 0.0f, qk = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float x = sq[t][32 * j + lane], y = sk[t][32 * j + lane];
                q2 = fmaf(x, x, q2);
                k2 = fmaf(y, y, k2);
                qk = fmaf(x, y, qk);
            }
            q2 = warp_sum(q2);
            k2 = warp_sum(k2);
            qk = warp_sum(qk);
            const float rq = (a.l2norm ? 1.0f / sqrtf(q2 + kDeltaNormEps) : 1.0f) * a.scale;
            const float rk = a.l2norm ? 1.0f / sqrtf(k2 + kDeltaNormEps) : 1.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                sq[t][32 * j + lane] *= rq;
                sk[t][32 * j + lane] *= rk;
            }
            if (lane == 0) sqk[t] = qk * rq * rk;
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            float kr[J][4], qr[J][4];
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 kk = *reinterpret_cast<const float4*>(&sk[t][4 * p + 32 * j]);
                const float4 qq = *reinterpret_cast<const float4*>(&sq[t][4 * p + 32 * j]);
                kr[j][0] = kk.x; kr[j][1] = kk.y; kr[j][2] = kk.z; kr[j][3] = kk.w;
                qr[j][0] = qq.x; qr[j][1] = qq.y; qr[j][2] = qq.z; qr[j][3] = qq.w;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x = fmaf(S[j][i], kr[j][i], x);
                    y = fmaf(S[j][i], qr[j][i], y);
                }
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, d);
                y += __shfl_xor_sync(0xffffffffu, y, d);
            }
            const float al = sa[t];
            const float u = sb[t] * (sv[t][col] - al * x);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[j][i] = fmaf(kr[j][i], u, al * S[j][i]);
            __syncwarp();                                   // the column's lanes have read its value
            if (p == 0) sv[t][col] = fmaf(sqk[t], u, al * y);
        }
        __syncthreads();
        for (int i = tid; i < kSeqT * kSeqCols; i += kSeqThreads) {
            const int t = a.os.st == 1 ? i % kSeqT : i / kSeqCols, c = a.os.st == 1 ? i / kSeqT : i % kSeqCols;
            if (t < n && c < cols) st(o, (t0 + t) * a.os.st + c * a.os.sc, sv[t][c]);
        }
        __syncthreads();
    }
    if (a.state_out && mine) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * p + 32 * j + i;
                if (r < a.dk) a.state_out[sbase + int64_t(r) * a.dv] = S[j][i];
            }
    }
}

template <typename T>
cudaError_t launch_seq_t(const DeltaArgs& a, cudaStream_t s) {
    const dim3 grid(unsigned((a.dv + kSeqCols - 1) / kSeqCols), unsigned(a.Hv), unsigned(a.B));
    switch ((a.dk + 31) / 32) {
        case 1: k_delta_seq<T, 1><<<grid, kSeqThreads, 0, s>>>(a); break;
        case 2: k_delta_seq<T, 2><<<grid, kSeqThreads, 0, s>>>(a); break;
        case 3: k_delta_seq<T, 3><<<grid, kSeqThreads, 0, s>>>(a); break;
        default: k_delta_seq<T, 4><<<grid, kSeqThreads, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

// ----------------------------------------------------------------------- step
// One token.  The state is read and written once, so its traffic bounds the
// kernel: 256 threads hold dk x kStepCols columns in registers (V columns a
// thread as one load of 4 V bytes, rows rg + R j), all loads issued before the
// first barrier, one reduction over the rows for both contractions.  V = 4
// needs dv a multiple of 4 (the rows of the state 16-byte aligned).  With many
// states a CTA takes 128 columns, 64 KB in flight; with few 32, which reach more
// SMs.
constexpr int kStepThreads = 256;

template <typename T, int V, int kStepCols>
__global__ void __launch_bounds__(kStepThreads)
k_delta_step(DeltaArgs a, float* __restrict__ states, int64_t n_states, const int32_t* __restrict__ slots,
             uint32_t* status) {
    constexpr int CG = kStepCols / V;              // threads along a row of 32 columns
    constexpr int R = kStepThreads / CG;           // row groups
    constexpr int J = kDeltaMaxDk / R;             // rows a thread
    static_assert(CG <= 32, "a row group is within a warp");
    __shared__ float sk[kDeltaMaxDk], sq[kDeltaMaxDk];
    __shared__ float red[kStepThreads / 32][2][kStepCols];
    __shared__ float s_qk;
    const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int cg = tid % CG, rg = tid / CG;
    const int c0 = int(blockIdx.x) * kStepCols + cg * V, h = int(blockIdx.y);
    const int64_t b = blockIdx.z;
    const int kh = h / (a.Hv / a.Hk);
    const int64_t slot = slots ? int64_t(slots[b]) : b;
    if (slot < 0) return;                          // padding, the whole CTA
    int bad = slot >= n_states;
    if (slots)
        for (int64_t i = tid; i < b; i += kStepThreads) bad |= int64_t(slots[i]) == slot;
    const bool mine = c0 < a.dv;
    float* Sp = states + ((slot * a.Hv + h) * int64_t(a.dk)) * a.dv + c0;
    float S[J][V];
    const bool readable = slot < n_states;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int r = rg + R * j;
        const bool in = mine && r < a.dk && readable;
        if constexpr (V == 4) {
            const float4 x = in ? *reinterpret_cast<const float4*>(Sp + int64_t(r) * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
            S[j][0] = x.x; S[j][1] = x.y; S[j][2] = x.z; S[j][3] = x.w;
        } else {
            S[j][0] = in ? Sp[int64_t(r) * a.dv] : 0.0f;
        }
    }
    const float al = a.g ? expf(a.g[b * a.gs.sb + h * a.gs.sc]) : 1.0f;
    const float be = a.beta ? a.beta[b * a.bs.sb + h * a.bs.sc] : 1.0f;
    const T* vp = static_cast<const T*>(a.v) + b * a.vs.sb + (int64_t(h) * a.dv + c0) * a.vs.sc;
    float vv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) vv[i] = mine ? ld(vp, int64_t(i) * a.vs.sc) : 0.0f;
    if (warp == 0) {
        const T* q = static_cast<const T*>(a.q) + b * a.qs.sb + int64_t(kh) * a.dk * a.qs.sc;
        const T* k = static_cast<const T*>(a.k) + b * a.ks.sb + int64_t(kh) * a.dk * a.ks.sc;
        float x[4], y[4], q2 = 0.0f, k2 = 0.0f, qk = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = lane + 32 * j;
            x[j] = c < a.dk ? ld(q, c * a.qs.sc) : 0.0f;
            y[j] = c < a.dk ? ld(k, c * a.ks.sc) : 0.0f;
            q2 = fmaf(x[j], x[j], q2);
            k2 = fmaf(y[j], y[j], k2);
            qk = fmaf(x[j], y[j], qk);
        }
        q2 = warp_sum(q2);
        k2 = warp_sum(k2);
        qk = warp_sum(qk);
        const float rq = (a.l2norm ? 1.0f / sqrtf(q2 + kDeltaNormEps) : 1.0f) * a.scale;
        const float rk = a.l2norm ? 1.0f / sqrtf(k2 + kDeltaNormEps) : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sq[lane + 32 * j] = x[j] * rq;
            sk[lane + 32 * j] = y[j] * rk;
        }
        if (lane == 0) s_qk = qk * rq * rk;
    }
    bad = __syncthreads_or(bad);
    T* op = static_cast<T*>(a.o) + b * a.os.sb + (int64_t(h) * a.dv + c0) * a.os.sc;
    if (bad) {
        if (rg == 0 && mine)
#pragma unroll
            for (int i = 0; i < V; ++i) st(op, int64_t(i) * a.os.sc, __int_as_float(0x7fffffff));
        if (tid == 0) report_status(status, kStatusBadSlot);
        return;
    }
    float x[V], y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = y[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const float kr = sk[rg + R * j], qr = sq[rg + R * j];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = fmaf(S[j][i], kr, x[i]);
            y[i] = fmaf(S[j][i], qr, y[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int d = CG; d < 32; d <<= 1) {
            x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
            y[i] += __shfl_xor_sync(0xffffffffu, y[i], d);
        }
        if (lane < CG) {
            red[warp][0][cg * V + i] = x[i];
            red[warp][1][cg * V + i] = y[i];
        }
    }
    __syncthreads();
    float u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = y[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < kStepThreads / 32; ++w) {
            x[i] += red[w][0][cg * V + i];
            y[i] += red[w][1][cg * V + i];
        }
        u[i] = be * (vv[i] - al * x[i]);
    }
    if (!mine) return;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int r = rg + R * j;
        const float kr = sk[r];
        if (r < a.dk) {
            if constexpr (V == 4) {
                *reinterpret_cast<float4*>(Sp + int64_t(r) * a.dv) =
                    make_float4(fmaf(kr, u[0], al * S[j][0]), fmaf(kr, u[1], al * S[j][1]),
                                fmaf(kr, u[2], al * S[j][2]), fmaf(kr, u[3], al * S[j][3]));
            } else {
                Sp[int64_t(r) * a.dv] = fmaf(kr, u[0], al * S[j][0]);
            }
        }
    }
    if (rg == 0)
#pragma unroll
        for (int i = 0; i < V; ++i) st(op, int64_t(i) * a.os.sc, fmaf(s_qk, u[i], al * y[i]));
}

// ----------------------------------------------------------------- arguments
hyena_status_t fail(hyena_status_t st, const std::string& why) { return set_last_error_detail(st, why); }

struct Range {
    const char *lo, *hi;
    bool meets(const Range& r) const { return lo < r.hi && r.lo < hi; }
};

Range range_of(const void* p, int64_t n0, int64_t n1, int64_t n2, const int64_t* s, int64_t es) {
    const char* c = static_cast<const char*>(p);
    return {c, c + ((n0 - 1) * s[0] + (n1 - 1) * s[1] + (n2 - 1) * s[2] + 1) * es};
}

// Whether every element of a [n0, n1, n2] tensor with these strides has a place of its own.
bool own_places(int64_t n0, int64_t n1, int64_t n2, const int64_t* s) {
    std::pair<int64_t, int64_t> d[3] = {{s[0], n0}, {s[1], n1}, {s[2], n2}};
    std::sort(d, d + 3);
    int64_t reach = 0;
    for (const auto& x : d) {
        if (x.second == 1) continue;
        if (x.first <= reach) return false;
        reach += (x.second - 1) * x.first;
    }
    return true;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool shapes_ok(int64_t B, int64_t L, int Hk, int Hv, int dk, int dv) {
    return B >= 1 && B <= 65535 && L >= 1 && L <= (int64_t(1) << 30) && Hk >= 1 && Hv >= Hk && Hv <= 4096 &&
           Hv % Hk == 0 && dk >= 1 && dk <= kDeltaMaxDk && dv >= 1 && dv <= kDeltaMaxDv && B * Hv * L <= (int64_t(1) << 40);
}

// Whether a range meets any operand of *p (its strides and sizes checked).
bool meets_operand(const Range& r, const hyena_delta_rule_t* p) {
    const int64_t es = p->dtype == HYENA_BF16 ? 2 : 4;
    const int64_t Ck = int64_t(p->Hk) * p->dk, Cv = int64_t(p->Hv) * p->dv, n = p->B * p->Hv * p->dk * int64_t(p->dv) * 4;
    auto flat = [](const void* q, int64_t bytes) { return Range{static_cast<const char*>(q), static_cast<const char*>(q) + bytes}; };
    return r.meets(range_of(p->q, p->B, Ck, p->L, p->q_stride, es)) || r.meets(range_of(p->k, p->B, Ck, p->L, p->k_stride, es)) ||
           r.meets(range_of(p->v, p->B, Cv, p->L, p->v_stride, es)) || r.meets(range_of(p->o, p->B, Cv, p->L, p->o_stride, es)) ||
           (p->g && r.meets(range_of(p->g, p->B, p->Hv, p->L, p->g_stride, 4))) ||
           (p->beta && r.meets(range_of(p->beta, p->B, p->Hv, p->L, p->beta_stride, 4))) ||
           (p->state_in && r.meets(flat(p->state_in, n))) || (p->state_out && r.meets(flat(p->state_out, n))) ||
           (p->lengths && r.meets(flat(p->lengths, 4 * p->B)));
}

// bf16 storage runs in chunks from a few tokens on.  Where the two forms cross depends on the heads in flight (us of a call,
// token by token against chunks, token-major rows): 4 heads of 64 10.5 against 14.4 at 20 tokens, 14.4 against 14.4 at 32,
// 22.9 against 13.6 at 64; 256 heads of 128 40 against 39 at 16, 66 against 39 at 32; 1024 heads of 128 148 against 130 at 16,
// 245 against 133 at 32.  (Rows along time that do not start on 16 bytes cost the chunks 5 us more: 17 tokens of 4 heads 12.4
// against 19.3.)  The border lies at the lowest of these, by the length alone, so that a sequence's results do not depend on
// how many others are in the call: few heads lose up to 4 us (7 unaligned) from 17 to 31 tokens by it.
constexpr int64_t kSeqMost = 16;
bool chunked(int64_t L, int dtype) { return dtype == HYENA_BF16 && L > kSeqMost; }

// Checks shared by both entry points; fills the launch arguments.
hyena_status_t prepare_delta(const hyena_delta_rule_t* p, DeltaArgs* a) {
    if (!p) return fail(HYENA_ERR_INVALID_ARG, "the argument struct is NULL");
    if (p->B < 1 || p->L < 1 || p->Hk < 1 || p->Hv < 1 || p->dk < 1 || p->dv < 1)
        return fail(HYENA_ERR_INVALID_ARG, "B, L, Hk, Hv, dk and dv must be >= 1");
    if (!shapes_ok(p->B, p->L, p->Hk, p->Hv, p->dk, p->dv))
        return fail(HYENA_ERR_UNSUPPORTED_SHAPE,
                    "needs B <= 65535, L <= 2^30, B Hv L <= 2^40, Hv a multiple of Hk up to 4096, dk <= 128 and dv <= 256");
    if (p->dtype != HYENA_F32 && p->dtype != HYENA_BF16)
        return fail(HYENA_ERR_INVALID_ARG, "dtype must be HYENA_F32 or HYENA_BF16");
    if (p->flags & ~HYENA_DELTA_L2NORM) return fail(HYENA_ERR_INVALID_ARG, "unknown flag bits");
    if (!std::isfinite(p->scale)) return fail(HYENA_ERR_INVALID_ARG, "scale must be finite");
    if (!p->q || !p->k || !p->v || !p->o) return fail(HYENA_ERR_INVALID_ARG, "q, k, v and o must not be NULL");
    const int64_t es = p->dtype == HYENA_BF16 ? 2 : 4;
    if (!aligned(p->q, es) || !aligned(p->k, es) || !aligned(p->v, es) || !aligned(p->o, es))
        return fail(HYENA_ERR_MISALIGNED, "q, k, v and o must be aligned to their elements");
    if (!aligned(p->g, 4) || !aligned(p->beta, 4) || !aligned(p->lengths, 4))
        return fail(HYENA_ERR_MISALIGNED, "g, beta and lengths must be 4-byte aligned");
    if (!aligned(p->state_in, 16) || !aligned(p->state_out, 16))
        return fail(HYENA_ERR_MISALIGNED, "states must be 16-byte aligned");
    const int64_t Ck = int64_t(p->Hk) * p->dk, Cv = int64_t(p->Hv) * p->dv;
    const int64_t zero[3] = {0, 0, 0};
    const int64_t* gs = p->g ? p->g_stride : zero;
    const int64_t* bs = p->beta ? p->beta_stride : zero;
    const int64_t* all[6] = {p->q_stride, p->k_stride, p->v_stride, p->o_stride, gs, bs};
    const int64_t ext[6] = {Ck, Ck, Cv, Cv, p->Hv, p->Hv};
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < 3; ++j) {
            if (all[i][j] < 0 || all[i][j] > (int64_t(1) << 40))
                return fail(HYENA_ERR_INVALID_ARG, "strides must be in [0, 2^40]");
            const int64_t n = j == 0 ? p->B : j == 1 ? ext[i] : p->L;
            if (n > 1 && all[i][j] > (int64_t(1) << 56) / n) return fail(HYENA_ERR_INVALID_ARG, "strides exceed the address space");
        }
    if (!own_places(p->B, Cv, p->L, p->o_stride))
        return fail(HYENA_ERR_INVALID_ARG, "the strides of o put two elements in one place");
    const Range o = range_of(p->o, p->B, Cv, p->L, p->o_stride, es);
    const int64_t nstate = p->B * p->Hv * p->dk * int64_t(p->dv) * 4;
    const Range in[] = {range_of(p->q, p->B, Ck, p->L, p->q_stride, es), range_of(p->k, p->B, Ck, p->L, p->k_stride, es),
                        range_of(p->v, p->B, Cv, p->L, p->v_stride, es)};
    const Range gr = range_of(p->g, p->B, p->Hv, p->L, gs, 4), br = range_of(p->beta, p->B, p->Hv, p->L, bs, 4);
    const char *si = reinterpret_cast<const char*>(p->state_in), *so = reinterpret_cast<const char*>(p->state_out);
    const char* le = reinterpret_cast<const char*>(p->lengths);
    const Range sin{si, si + nstate}, sout{so, so + nstate}, len{le, le + 4 * p->B};
    bool clash = false;
    for (const Range& r : in) clash |= o.meets(r) || (so && sout.meets(r));
    clash |= (p->g && (o.meets(gr) || (so && sout.meets(gr)))) || (p->beta && (o.meets(br) || (so && sout.meets(br))));
    clash |= (si && o.meets(sin)) || (so && o.meets(sout)) || (si && so && si != so && sin.meets(sout));
    clash |= le && (o.meets(len) || (so && sout.meets(len)));
    if (clash) return fail(HYENA_ERR_INVALID_ARG, "o or state_out overlaps another operand");
    auto view = [](const int64_t* s) { return DeltaView{s[0], s[1], s[2]}; };
    *a = DeltaArgs{p->B, p->L, p->Hk, p->Hv, p->dk, p->dv, (p->flags & HYENA_DELTA_L2NORM) != 0,
                   p->scale != 0.0f ? p->scale : 1.0f / std::sqrt(float(p->dk)), p->q, p->k, p->v, p->o, p->g, p->beta,
                   view(p->q_stride), view(p->k_stride), view(p->v_stride), view(p->o_stride), view(gs), view(bs),
                   p->state_in, p->state_out, p->lengths};
    return HYENA_OK;
}

hyena_status_t done(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return set_last_error_detail(HYENA_OK, "");
    return fail(HYENA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

}  // namespace

cudaError_t launch_delta_seq(const DeltaArgs& a, int dtype, cudaStream_t s) {
    return dtype == DT_BF16 ? launch_seq_t<__nv_bfloat16>(a, s) : launch_seq_t<float>(a, s);
}

cudaError_t launch_delta_step(const DeltaArgs& a, int dtype, float* states, int64_t n_states, const int32_t* slots,
                              uint32_t* status, cudaStream_t s) {
    int dev = 0, sms = 0;
    const cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    // 128 columns a CTA once that leaves every SM two (256 rows of 16 heads, dk = dv = 128: 108 us against 152 us with 32); rows of 4 columns
    // as one access where they are aligned
    const bool v4 = a.dv % 4 == 0, wide = v4 && a.dv > 64 && a.B * a.Hv >= 2 * int64_t(sms);
    const int cols = wide ? 128 : 32;
    const dim3 grid(unsigned((a.dv + cols - 1) / cols), unsigned(a.Hv), unsigned(a.B));
    auto go = [&](auto kernel) { kernel<<<grid, kStepThreads, 0, s>>>(a, states, n_states, slots, status); };
    if (dtype == DT_BF16) {
        if (wide) go(k_delta_step<__nv_bfloat16, 4, 128>);
        else if (v4) go(k_delta_step<__nv_bfloat16, 4, 32>);
        else go(k_delta_step<__nv_bfloat16, 1, 32>);
    } else {
        if (wide) go(k_delta_step<float, 4, 128>);
        else if (v4) go(k_delta_step<float, 4, 32>);
        else go(k_delta_step<float, 1, 32>);
    }
    return cudaGetLastError();
}

}  // namespace hyena

using namespace hyena;

extern "C" size_t hyena_delta_rule_workspace_bytes(int64_t B, int64_t L, int Hk, int Hv, int dk, int dv,
                                                   hyena_dtype_t dtype) {
    if (!shapes_ok(B, L, Hk, Hv, dk, dv) || !chunked(L, dtype)) return 0;
    return delta_chunk_workspace(B, L, Hv);
}

namespace {

// The chunked form: its workspace checked, launched.
hyena_status_t run_chunked(const hyena_delta_rule_t* p, const DeltaArgs& a, void* workspace, size_t workspace_bytes,
                           uint64_t budget_ns, int64_t hold, cudaStream_t s) {
    const size_t need = delta_chunk_workspace(p->B, p->L, p->Hv);
    if (!workspace || workspace_bytes < need)
        return fail(HYENA_ERR_WORKSPACE_TOO_SMALL, "workspace must hold at least " + std::to_string(need) + " bytes");
    if (!aligned(workspace, 16)) return fail(HYENA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    const char* w = static_cast<const char*>(workspace);
    const Range wr{w, w + need};
    if (meets_operand(wr, p)) return fail(HYENA_ERR_INVALID_ARG, "workspace overlaps an operand");
    uint32_t* status = nullptr;
    cudaError_t e = kernel_status_word(&status);
    if (e != cudaSuccess) return done(e, "kernel status word");
    return done(launch_delta_chunk(a, workspace, status, budget_ns, hold, s), "delta rule");
}

}  // namespace

extern "C" hyena_status_t hyena_delta_rule(const hyena_delta_rule_t* p, void* workspace, size_t workspace_bytes,
                                           void* stream) {
    DeltaArgs a;
    hyena_status_t st = prepare_delta(p, &a);
    if (st != HYENA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!chunked(p->L, p->dtype)) return done(launch_delta_seq(a, p->dtype, s), "delta rule");
    return run_chunked(p, a, workspace, workspace_bytes, kDefaultWaitBudgetNs, -1, s);
}

extern "C" hyena_status_t hyena_debug_delta_rule(const hyena_delta_rule_t* p, void* workspace, size_t workspace_bytes,
                                                 uint64_t wait_budget_ns, int64_t hold_chunk, void* stream) {
    DeltaArgs a;
    hyena_status_t st = prepare_delta(p, &a);
    if (st != HYENA_OK) return st;
    if (!chunked(p->L, p->dtype))
        return fail(HYENA_ERR_UNSUPPORTED_SHAPE, "only the chunked form (bf16, more than " + std::to_string(kSeqMost) + " tokens) waits");
    if (wait_budget_ns == 0) return fail(HYENA_ERR_INVALID_ARG, "wait_budget_ns must be > 0");
    return run_chunked(p, a, workspace, workspace_bytes, wait_budget_ns, hold_chunk, static_cast<cudaStream_t>(stream));
}

extern "C" hyena_status_t hyena_delta_rule_step(const hyena_delta_rule_t* p, float* states, int64_t n_states,
                                                const int32_t* slots, void* stream) {
    DeltaArgs a;
    hyena_status_t st = prepare_delta(p, &a);
    if (st != HYENA_OK) return st;
    if (p->L != 1) return fail(HYENA_ERR_INVALID_ARG, "the step takes one token: L must be 1");
    if (p->state_in || p->state_out || p->lengths)
        return fail(HYENA_ERR_INVALID_ARG, "the step takes states: state_in, state_out and lengths must be NULL");
    if (!states) return fail(HYENA_ERR_INVALID_ARG, "states must not be NULL");
    if (!aligned(states, 16) || !aligned(slots, 4))
        return fail(HYENA_ERR_MISALIGNED, "states must be 16-byte aligned, slots 4-byte");
    if (n_states < 1 || (!slots && n_states < p->B) || n_states > (int64_t(1) << 31))
        return fail(HYENA_ERR_INVALID_ARG, "n_states must be >= 1, and >= B without slots");
    const char* sp = reinterpret_cast<const char*>(states);
    const char* lp = reinterpret_cast<const char*>(slots);
    const Range sr{sp, sp + n_states * p->Hv * p->dk * int64_t(p->dv) * 4}, lr{lp, lp + 4 * p->B};
    const Range o = range_of(p->o, p->B, int64_t(p->Hv) * p->dv, 1, p->o_stride, p->dtype == HYENA_BF16 ? 2 : 4);
    if (meets_operand(sr, p) || (slots && (sr.meets(lr) || o.meets(lr))))
        return fail(HYENA_ERR_INVALID_ARG, "states or o overlaps another operand");
    uint32_t* status = nullptr;
    cudaError_t e = kernel_status_word(&status);
    if (e != cudaSuccess) return done(e, "kernel status word");
    return done(launch_delta_step(a, p->dtype, states, n_states, slots, status, static_cast<cudaStream_t>(stream)),
                "delta rule step");
}
