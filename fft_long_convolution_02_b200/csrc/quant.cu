// quant.cu -- e4m3 with a scale for each block of 128: the operands of
// hyena_proj_fp8.
//
//   scale = max(amax / 448, 2^-126),  q = x / scale to nearest even
//
// Both are one pass over x, bound by its bytes in and the e4m3 bytes out: a
// block's values stay in registers between the maximum and the rounding.
// 32768 x 768 bf16: 19.7 us, 3.9 TB/s (channels contiguous), 26.7 us, 2.9 TB/s
// (positions contiguous).  17 instructions an element bound it (unpacking, the
// maximum, the corrected quotient, the conversion): 71 % of the issue slots, 53 %
// where the tile goes through shared memory.  Weights: 2304 x 768 6.2 us,
// 16384 x 2048 29 us (floors 0.8 and 15.6).
// The maximum is taken over the bits of |x|, which order like the values and
// put NaN above infinity, so a NaN reaches the scale.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <string>

#include "hyena.h"
#include "kernels.h"

namespace hyena {

hyena_status_t set_last_error_detail(hyena_status_t st, const std::string& detail);  // api.cu

namespace {

using bf16 = __nv_bfloat16;
constexpr int kBlk = 128;
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale of a block and what its quotients need.  x / s to nearest is
// x r, corrected by its remainder (P. Markstein's division from a correctly
// rounded reciprocal r; the remainder is exact in a fused multiply-add).  For
// largest magnitudes below 2^-50 the remainder could underflow: the division
// itself there, as for what is not finite.
__device__ __forceinline__ float divided(float x, float by, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, by, x), r, q);
}
struct Scale {
    float s, r;
    bool plain;
    __device__ __forceinline__ explicit Scale(uint32_t amax_bits) {
        const float m = __uint_as_float(amax_bits);
        // 2^-50 <= m < infinity: m / 448 and every quotient by it
        plain = amax_bits >= 0x26800000u && amax_bits < 0x7f800000u;
        if (plain) {
            s = divided(m, 448.0f, 1.0f / 448.0f);
        } else {
            s = __fdiv_rn(m, 448.0f);
            s = s < 1.17549435e-38f ? 1.17549435e-38f : s;
        }
        r = __frcp_rn(s);
    }
    __device__ __forceinline__ float quotient(float x) const { return plain ? divided(x, s, r) : __fdiv_rn(x, s); }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Eight consecutive values as they lie (16 bytes of bf16, 32 of fp32; 16-byte aligned).
template <typename T>
struct Octet;
template <>
struct Octet<bf16> {
    uint4 w;
    __device__ __forceinline__ void load(const bf16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};
template <>
struct Octet<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

__device__ __forceinline__ uint2 quotients8(const Scale& sc, const float (&v)[8]) {
    return make_uint2(e4m3x4(sc.quotient(v[0]), sc.quotient(v[1]), sc.quotient(v[2]), sc.quotient(v[3])),
                      e4m3x4(sc.quotient(v[4]), sc.quotient(v[5]), sc.quotient(v[6]), sc.quotient(v[7])));
}

// x [rows of K], channels contiguous: 16 lanes take a block of 128 as eight
// values each; a CTA takes 32 rows of one block, so its 32 scales leave as one
// contiguous store.
constexpr int kRowsLast = 32, kThreadsLast = 128;

template <typename T>
__global__ void __launch_bounds__(kThreadsLast, sizeof(T) == 2 ? 12 : 8)
k_quant_last(const T* __restrict__ x, uint8_t* __restrict__ xq, float* __restrict__ xs, int64_t L, int64_t K) {
    constexpr int kIter = kRowsLast / (kThreadsLast / 16), kStep = kThreadsLast / 16;
    __shared__ float s_scale[kRowsLast];
    const int64_t kb = blockIdx.x, l0 = int64_t(blockIdx.y) * kRowsLast, b = blockIdx.z;
    const int g = int(threadIdx.x) >> 4, lane = int(threadIdx.x) & 15;
    const int64_t c = kb * kBlk + lane * 8;
    Octet<T> w[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int64_t l = l0 + g + kStep * i;
        if (l < L && c < K) w[i].load(x + (b * L + l) * K + c);
        else w[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        float v[8];
        w[i].get(v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const Scale sc(m);
        const int64_t l = l0 + g + kStep * i;
        if (l < L && c < K) *reinterpret_cast<uint2*>(xq + (b * L + l) * K + c) = quotients8(sc, v);
        if (lane == 0) s_scale[g + kStep * i] = sc.s;
    }
    __syncthreads();
    if (threadIdx.x < kRowsLast && l0 + threadIdx.x < L)
        xs[(b * gridDim.x + kb) * L + l0 + threadIdx.x] = s_scale[threadIdx.x];
}

// x [K][L], positions contiguous: a tile of 128 channels x 64 positions goes
// through shared memory; then a thread holds 32 channels of one position (a
// warp 32 neighbouring positions: conflict-free) and stores them as 32 bytes.
// `wide`: L a multiple of the elements in 16 bytes, so rows load as vectors.
constexpr int kPosFirst = 64;

template <typename T>
__global__ void __launch_bounds__(kThreads)
k_quant_first(const T* __restrict__ x, uint8_t* __restrict__ xq, float* __restrict__ xs, int64_t L, int64_t K,
              int wide) {
    constexpr int kVec = 16 / int(sizeof(T));
    constexpr int kRow = kPosFirst + kVec;          // rows stay 16-byte aligned
    __shared__ __align__(16) T tile[kBlk][kRow];
    __shared__ uint32_t part[4][kPosFirst];
    const int64_t kb = blockIdx.x, l0 = int64_t(blockIdx.y) * kPosFirst, b = blockIdx.z;
    const T* xb = x + b * K * L;
    if (wide) {
        constexpr int kPer = kPosFirst / kVec;      // vectors a row
#pragma unroll
        for (int i = int(threadIdx.x); i < kBlk * kPer; i += kThreads) {
            const int r = i / kPer, j = (i % kPer) * kVec;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (kb * kBlk + r < K && l0 + j < L) w = __ldg(reinterpret_cast<const uint4*>(xb + (kb * kBlk + r) * L + l0 + j));
            *reinterpret_cast<uint4*>(&tile[r][j]) = w;
        }
    } else {
#pragma unroll 8
        for (int i = int(threadIdx.x); i < kBlk * kPosFirst; i += kThreads) {
            const int r = i / kPosFirst, j = i % kPosFirst;
            tile[r][j] = (kb * kBlk + r < K && l0 + j < L) ? xb[(kb * kBlk + r) * L + l0 + j] : T(0.0f);
        }
    }
    __syncthreads();
    const int l = int(threadIdx.x) & (kPosFirst - 1), p = int(threadIdx.x) / kPosFirst;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = float(tile[32 * p + i][l]);
        m = max(m, abs_bits(v[i]));
    }
    part[p][l] = m;
    __syncthreads();
    m = max(max(part[0][l], part[1][l]), max(part[2][l], part[3][l]));
    const Scale sc(m);
    if (l0 + l >= L) return;
    if (p == 0) xs[(b * gridDim.x + kb) * L + l0 + l] = sc.s;
    uint8_t* out = xq + (b * L + l0 + l) * K + kb * kBlk + 32 * p;
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
        if (kb * kBlk + 32 * p + i >= K) break;      // K is a multiple of 16
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = e4m3x4(sc.quotient(v[i + 4 * j]), sc.quotient(v[i + 4 * j + 1]), sc.quotient(v[i + 4 * j + 2]),
                          sc.quotient(v[i + 4 * j + 3]));
        *reinterpret_cast<uint4*>(out + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// W [N][K]: a CTA takes a block of 128 x 128.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_quant_weight(const T* __restrict__ w, uint8_t* __restrict__ wq, float* __restrict__ ws, int64_t N, int64_t K) {
    __shared__ uint32_t part[kThreads / 32];
    const int64_t kb = blockIdx.x, nb = blockIdx.y;
    const int g = int(threadIdx.x) >> 4, lane = int(threadIdx.x) & 15;
    const int64_t c = kb * kBlk + lane * 8;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = nb * kBlk + g + 16 * i;
        if (n < N && c < K) {
            Octet<T> o;
            o.load(w + n * K + c);
            o.get(v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    const Scale sc(m);
    if (threadIdx.x == 0) ws[nb * gridDim.x + kb] = sc.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = nb * kBlk + g + 16 * i;
        if (n < N && c < K) *reinterpret_cast<uint2*>(wq + n * K + c) = quotients8(sc, v[i]);
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}
hyena_status_t fail(hyena_status_t st, const std::string& why) { return set_last_error_detail(st, why); }

hyena_status_t check(const void* x, const void* q, const float* s, int64_t rows, int64_t K, int64_t scales, int dtype) {
    if (!x || !q || !s) return fail(HYENA_ERR_INVALID_ARG, "the input, values and scales must not be NULL");
    if (dtype != HYENA_F32 && dtype != HYENA_BF16) return fail(HYENA_ERR_INVALID_ARG, "dtype must be HYENA_F32 or HYENA_BF16");
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4))
        return fail(HYENA_ERR_MISALIGNED, "the input and values must be 16-byte aligned, scales 4-byte");
    const size_t nx = size_t(rows) * size_t(K) * (dtype == HYENA_BF16 ? 2 : 4), nq = size_t(rows) * size_t(K);
    if (overlaps(x, nx, q, nq) || overlaps(x, nx, s, size_t(scales) * 4) || overlaps(q, nq, s, size_t(scales) * 4))
        return fail(HYENA_ERR_INVALID_ARG, "the input, values and scales overlap");
    return HYENA_OK;
}

hyena_status_t done(cudaError_t e) {
    if (e == cudaSuccess) return set_last_error_detail(HYENA_OK, "");
    return fail(HYENA_ERR_CUDA, std::string("quantisation: ") + cudaGetErrorString(e));
}

}  // namespace
}  // namespace hyena

using namespace hyena;

extern "C" hyena_status_t hyena_quantize_fp8(const void* x, void* xq, float* xs, int64_t B, int64_t L, int64_t K,
                                             hyena_dtype_t dtype, int channels_first, void* stream) {
    if (B < 1 || L < 1 || K < 1) return fail(HYENA_ERR_INVALID_ARG, "B, L and K must be >= 1");
    if (K % 16 != 0 || K > (int64_t(1) << 20) || B > 65535 || B * L > (int64_t(1) << 31) - 1 || L > kRowsLast * int64_t(65535))
        return fail(HYENA_ERR_UNSUPPORTED_SHAPE,
                    "K must be a multiple of 16 up to 2^20, B <= 65535, L <= 32 * 65535 and B * L < 2^31");
    const int64_t nb = (K + kBlk - 1) / kBlk;
    hyena_status_t st = check(x, xq, xs, B * L, K, B * nb * L, dtype);
    if (st != HYENA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* q = static_cast<uint8_t*>(xq);
    const int rows = channels_first ? kPosFirst : kRowsLast;
    const dim3 grid(unsigned(nb), unsigned((L + rows - 1) / rows), unsigned(B));
    if (channels_first) {
        if (dtype == HYENA_BF16) k_quant_first<<<grid, kThreads, 0, s>>>(static_cast<const bf16*>(x), q, xs, L, K, L % 8 == 0);
        else k_quant_first<<<grid, kThreads, 0, s>>>(static_cast<const float*>(x), q, xs, L, K, L % 4 == 0);
    } else {
        if (dtype == HYENA_BF16) k_quant_last<<<grid, kThreadsLast, 0, s>>>(static_cast<const bf16*>(x), q, xs, L, K);
        else k_quant_last<<<grid, kThreadsLast, 0, s>>>(static_cast<const float*>(x), q, xs, L, K);
    }
    return done(cudaGetLastError());
}

extern "C" hyena_status_t hyena_quantize_fp8_weight(const void* W, void* Wq, float* Ws, int64_t N, int64_t K,
                                                    hyena_dtype_t dtype, void* stream) {
    if (N < 1 || K < 1) return fail(HYENA_ERR_INVALID_ARG, "N and K must be >= 1");
    if (K % 16 != 0 || K > (int64_t(1) << 20) || N > (int64_t(1) << 20))
        return fail(HYENA_ERR_UNSUPPORTED_SHAPE, "K must be a multiple of 16, N and K at most 2^20");
    const int64_t kb = (K + kBlk - 1) / kBlk, nb = (N + kBlk - 1) / kBlk;
    hyena_status_t st = check(W, Wq, Ws, N, K, kb * nb, dtype);
    if (st != HYENA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid{unsigned(kb), unsigned(nb)};
    if (dtype == HYENA_BF16) k_quant_weight<<<grid, kThreads, 0, s>>>(static_cast<const bf16*>(W), static_cast<uint8_t*>(Wq), Ws, N, K);
    else k_quant_weight<<<grid, kThreads, 0, s>>>(static_cast<const float*>(W), static_cast<uint8_t*>(Wq), Ws, N, K);
    return done(cudaGetLastError());
}
