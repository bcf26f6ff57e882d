// delta_chunk.cu -- the gated delta rule over whole sequences in chunks of 64
// tokens, bf16 storage.
//
// With G_i the sum of the log decays of the chunk's tokens up to i, the writes U
// of a chunk solve a triangular system, and everything else is products:
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j  (j < i),     T = (1 + A)^-1 diag(beta)
//   U  = T (V - diag(e^G) K S)
//   O  = scale (diag(e^G) Q S + P U),    P_ij = e^{G_i - G_j} q_i.k_j  (j <= i)
//   S <- e^{G_63} S + K^T diag(e^{G_63 - G_i}) U
//
// k_delta_prep: T, P and the factors of a chunk, all chunks at once, into the
// workspace.  k_delta_scan: the chunks of a head in order, the state in
// registers.
//
// Precision.  The state and what feeds it are held to fp32: K and Q are exact in
// fp16 once a power of two brings a row's norm to [2^14, 2^15) (8 significant
// bits; what falls below 2^-39 of the norm is lost), and S, T, V - .. and U go
// into the products as two fp16 parts each under such a power of two for the
// largest element of each row: 22 bits of what is above 2^-17 of the largest,
// below that 2^-39 of the largest (the low part is subnormal then).  Sums are
// fp32.  The outputs are bf16, so on their way S, P and U are one fp16 part each:
// 11 bits of what is above 2^-28 of a row's largest, below that the same 2^-39.
// A chunk where that would not do is taken token by token ("far apart" below).
// e^{G_i - G_j} comes from sums held as two floats: their difference loses
// nothing behind a strong decay.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "delta.h"
#include "kernels.h"
#include "tc_util.cuh"
#include "tma_util.cuh"

namespace hyena {
namespace {

using bf16 = __nv_bfloat16;

constexpr int C = 64;                              // tokens of a chunk

// Bounds that tell a chunk whose magnitudes lie too far apart (see the scans).  m: the larger of a channel's largest write
// and of its largest residual times T's largest; r: that residual; n: the largest entry of U diag(cu); s: of the state
// before the chunk.
struct Reach {
    float t, w, k;                                 // T's largest; times what its row's write leaves in the state; the largest key
    __device__ __forceinline__ bool end(float m, float r, float n, float s, float gamma) const {
        return fmaxf(n * 0x1p14f, gamma * s) < fmaxf(r * w, m * k);
    }
    // whether outputs rest on the chunk's writes: the state before it is as small as they may be
    __device__ __forceinline__ bool bare(float m, float s, float gamma) const { return fminf(gamma, 1.0f) * s < m * k; }
};

// What k_delta_prep leaves for a chunk of a value head: T's two parts and P as
// fp16 images of the scan's shared memory, and the factors of its 64 tokens.
struct Factors {
    float kmul[C], qmul[C];                        // K, Q rows to their fp16 range
    float cx[C];                                   // (K S) row of the scaled K to diag(e^G) K S
    float cu[C];                                   // U row to its part of the state
    float co[C];                                   // (Q S) row of the scaled Q to the output
    float cp[C], ct[C];                            // rows of the stored P and T to P and T
    float gamma;                                   // e^{G_63}
    Reach reach;
    uint32_t strong[2];                            // tokens whose write strength is not 0, a bit each
    float pad[58];
};
constexpr uint32_t kTile = C * C * 2;              // bytes of a 64 x 64 fp16 image
constexpr uint32_t kBlob = 3 * kTile + uint32_t(sizeof(Factors));
static_assert(sizeof(Factors) == 2048, "");

// ------------------------------------------------------------------ fragments
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared-memory tiles of 16-bit numbers: rows of 16-byte pieces, piece c of row
// r at c ^ (r mod 8), so that eight rows' pieces lie on different banks.
template <int PIECES>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    return uint32_t(row * PIECES + (c ^ (row & 7))) * 16u;
}

// The right operand (16 of k, 16 of n) from a tile stored [n][k] or [k][n]: r[0], r[1] serve the first 8 of n.
template <int PIECES>
__device__ __forceinline__ void right_nk(uint32_t (&r)[4], uint32_t tile, int k16, int n8, int lane) {
    const int m = lane >> 3;
    ldsm4(r, tile + piece<PIECES>(8 * (n8 + (m >> 1)) + (lane & 7), 2 * k16 + (m & 1)));
}
template <int PIECES>
__device__ __forceinline__ void right_kn(uint32_t (&r)[4], uint32_t tile, int k16, int n8, int lane) {
    const int m = lane >> 3;
    ldsm4t(r, tile + piece<PIECES>(16 * k16 + 8 * (m & 1) + (lane & 7), n8 + (m >> 1)));
}
// The left operand (16 rows from 16 m16, 16 of k) from a tile stored [m][k] or [k][m].
template <int PIECES>
__device__ __forceinline__ void left_mk(uint32_t (&r)[4], uint32_t tile, int m16, int k16, int lane) {
    const int m = lane >> 3;
    ldsm4(r, tile + piece<PIECES>(16 * m16 + 8 * (m & 1) + (lane & 7), 2 * k16 + (m >> 1)));
}
template <int PIECES>
__device__ __forceinline__ void left_km(uint32_t (&r)[4], uint32_t tile, int m16, int k16, int lane) {
    const int m = lane >> 3;
    ldsm4t(r, tile + piece<PIECES>(16 * k16 + 8 * (m >> 1) + (lane & 7), 2 * m16 + (m & 1)));
}

// The power of two that brings a largest magnitude m to [2^14, 2^15), and its
// inverse; both normal numbers whatever m is.
struct Pow2 {
    float up, down;
    __device__ __forceinline__ explicit Pow2(float m) {
        int e = 268 - int(__float_as_uint(m) >> 23);
        e = max(1, min(253, e));
        up = __uint_as_float(uint32_t(e) << 23);
        down = __uint_as_float(uint32_t(254 - e) << 23);
    }
};

__device__ __forceinline__ uint32_t pack_h(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// a, b as fp16 pairs of a high and a low part
__device__ __forceinline__ void split_h(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack_h(a - f.x, b - f.y);
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ float bf(uint32_t w, int hi) { return __uint_as_float(hi ? (w & 0xffff0000u) : (w << 16)); }

// Eight elements of a [channel, time] view from (c, t), along time (FIRST) or along channels, one by one; what lies
// outside [0, nc) x [0, nt) is zero and not read.  No branches, so that the loads of several go out together.
template <bool FIRST>
__device__ __forceinline__ uint4 octet(const bf16* p, const DeltaView& s, int c, int t, int nc, int nt) {
    const bf16* at = p + int64_t(c) * s.sc + int64_t(t) * s.st;
    const int n = FIRST ? (c < nc ? nt - t : 0) : (t < nt ? nc - c : 0);
    const int64_t step = FIRST ? s.st : s.sc;
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i < n ? uint32_t(__ldg(reinterpret_cast<const unsigned short*>(at + i * step))) : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

// Whether all octets of a [nc] x [nt] tile lie inside it or outside it as wholes, and load as such: then a thread's
// loads go out together (octet()'s piecewise path would put each behind the one before).
template <bool FIRST>
__device__ __forceinline__ bool whole(int nc, int nt, bool vec) {
    return vec && ((FIRST ? nt : nc) & 7) == 0;
}
template <bool FIRST>
__device__ __forceinline__ uint4 whole_octet(const bf16* p, const DeltaView& s, int c, int t, int nc, int nt) {
    return c < nc && t < nt ? __ldg(reinterpret_cast<const uint4*>(p + int64_t(c) * s.sc + int64_t(t) * s.st)) : make_uint4(0, 0, 0, 0);
}

// The same as an asynchronous copy into shared memory.
template <bool FIRST>
__device__ __forceinline__ void copy_octet(void* to, const bf16* p, const DeltaView& s, int c, int t, int nc, int nt) {
    if (c < nc && t < nt) cp_async_bytes16(to, p + int64_t(c) * s.sc + int64_t(t) * s.st);
    else *static_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
}

struct ChunkArgs {
    DeltaArgs a;
    uint8_t* blobs;                                // [B][Hv][chunks][kBlob]
    int chunks;
    int vec_k, vec_q, vec_v, vec_o;                // rows may be read (written) 16 bytes at a time
    int group;                                     // value heads of a k_delta_prep CTA, all of one key head
    uint64_t budget_ns;
    int hold;                                      // test hook: the chunk whose stage is never freed (-1: none)
    uint32_t* status;
    int dev, sms;
};

__device__ __forceinline__ int64_t length_of(const DeltaArgs& a, int64_t b) {
    return a.lengths ? max(int64_t(0), min(a.L, int64_t(a.lengths[b]))) : a.L;
}

// ----------------------------------------------------------------------- prep
// One CTA of four warps a chunk and value head.  K and Q as they are (bf16,
// products exact in fp32) through mma.sync, warp w the 16 rows from 16 w, only
// tiles on or under the diagonal; the norms are the diagonals of K K^T and Q Q^T.
// The inverse of the unit triangle 1 + A in fp32: the four 16 x 16 blocks on the
// diagonal by substitution (a thread a column, the columns in registers), then
// twice the block under two inverses as -T22 (A21 T11).  Its chain of short
// steps bounds it, so what counts is how many CTAs an SM holds: A and T lie
// where K and Q were, five to an SM.  25 ns a chunk (dk = 128; 4 x 8192, 6 heads
// 78 us), 45 % of the issue slots.  Three CTAs an SM with 32 x 32 substitutions
// took 1.7 times as long, six CTAs with half of the products at a time 1.1
// times.  GROUP: up to four value heads of a key head one after the other from
// the same products (8192 chunks of two heads, dk = 128: 337 us); ptxas then
// spills 72 bytes a thread (dk = 64: 224), 4 at most without.
constexpr int kPrepThreads = 128;
constexpr int kGroup = kPrepThreads / 32;          // most value heads of a CTA: a warp sums one's decays
constexpr int kARow = 68;

template <int DK, bool FIRST>
struct PrepSmem {
    static constexpr int kRows = FIRST ? DK : C, kPieces = FIRST ? 8 : DK / 8;
    union {
        struct {
            alignas(128) uint8_t k[C * DK * 2], q[C * DK * 2];
        };
        struct {
            alignas(16) float A[C][kARow], T[C][kARow];
        };
    };
    alignas(16) float W[32][36];
    alignas(16) float gh[kGroup][C], gl[kGroup][C], beta[kGroup][C];   // gh + gl: sums of the log2 decays
    alignas(16) float rk[C], rq[C], kn[C], qn[C];                  // norms' inverses (rq times the scale), norms
    float left[C];                                 // what a token's write leaves at the chunk's end, times its key
    float kmost[2];                                // largest of the scaled keys, by halves of the chunk
    float strict[kGroup];                          // 2^-24, or 2^-18 where a gate grows the state
};

// W = A[r0 + N ..][c0 ..] T[c0 ..][c0 ..], then T[r0 ..][c0 ..] = -T[r0 ..][r0 ..] W, for the N x N block under the
// diagonal block at c0 (r0 = c0 + N), by `threads` threads of four columns each.
template <int N, typename Sm>
__device__ __forceinline__ void block_under(Sm& sm, int c0, int wrow, int t) {
    constexpr int kGroups = N / 4;
    const int r = t / kGroups, c = (t % kGroups) * 4, r0 = c0 + N;
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        constexpr int kRowsEach = N * kGroups / (N == 32 ? 128 : 64);          // rows a thread
        float acc[kRowsEach][4];
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll 8
        for (int k = 0; k < N; ++k) {
            const float4 u = step == 0 ? *reinterpret_cast<const float4*>(&sm.T[c0 + k][c0 + c])
                                       : *reinterpret_cast<const float4*>(&sm.W[wrow + k][c]);
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i) {
                const int row = r + i * (N / kRowsEach);
                const float w = step == 0 ? sm.A[r0 + row][c0 + k] : -sm.T[r0 + row][r0 + k];
                acc[i][0] = fmaf(w, u.x, acc[i][0]);
                acc[i][1] = fmaf(w, u.y, acc[i][1]);
                acc[i][2] = fmaf(w, u.z, acc[i][2]);
                acc[i][3] = fmaf(w, u.w, acc[i][3]);
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            const int row = r + i * (N / kRowsEach);
            float* to = step == 0 ? &sm.W[wrow + row][c] : &sm.T[r0 + row][c0 + c];
            *reinterpret_cast<float4*>(to) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        }
        __syncthreads();
    }
}

template <int DK, bool FIRST, bool GROUP>
__global__ void __launch_bounds__(kPrepThreads, 5) k_delta_prep(ChunkArgs x) {
    using Sm = PrepSmem<DK, FIRST>;
    constexpr int P = Sm::kPieces;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    const DeltaArgs& a = x.a;
    const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int chunk = int(blockIdx.x), group = GROUP ? x.group : 1, h_first = int(blockIdx.y) * group;
    const int64_t b = blockIdx.z, t0 = int64_t(chunk) * C;
    const int64_t len = length_of(a, b);
    if (t0 >= len) return;
    const int n = int(min(int64_t(C), len - t0));
    const int kh = h_first / (a.Hv / a.Hk);
    const bf16* kp = static_cast<const bf16*>(a.k) + b * a.ks.sb + int64_t(kh) * a.dk * a.ks.sc + t0 * a.ks.st;
    const bf16* qp = static_cast<const bf16*>(a.q) + b * a.qs.sb + int64_t(kh) * a.dk * a.qs.sc + t0 * a.qs.st;
    constexpr int kOct = Sm::kRows * P / kPrepThreads;
    if (whole<FIRST>(a.dk, n, x.vec_k && x.vec_q)) {
#pragma unroll
        for (int j = 0; j < kOct; ++j) {
            const int row = (tid + j * kPrepThreads) / P, c = (tid + j * kPrepThreads) % P;
            copy_octet<FIRST>(sm.k + piece<P>(row, c), kp, a.ks, FIRST ? row : 8 * c, FIRST ? 8 * c : row, a.dk, n);
            copy_octet<FIRST>(sm.q + piece<P>(row, c), qp, a.qs, FIRST ? row : 8 * c, FIRST ? 8 * c : row, a.dk, n);
        }
    } else {
#pragma unroll 2
        for (int i = tid; i < Sm::kRows * P; i += kPrepThreads) {
            const int row = i / P, c = i % P;
            const int ch = FIRST ? row : 8 * c, tt = FIRST ? 8 * c : row;
            *reinterpret_cast<uint4*>(sm.k + piece<P>(row, c)) = octet<FIRST>(kp, a.ks, ch, tt, a.dk, n);
            *reinterpret_cast<uint4*>(sm.q + piece<P>(row, c)) = octet<FIRST>(qp, a.qs, ch, tt, a.dk, n);
        }
    }
    cp_async_commit();
    // sums of the log2 decays as two floats (in double here), a warp a value head: two tokens a lane
    if (warp < group) {
        const int h = h_first + warp;
        double v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = 2 * lane + j;
            float d = a.g && t < n ? a.g[b * a.gs.sb + h * a.gs.sc + (t0 + t) * a.gs.st] : 0.0f;
            // -inf (empty the state) as a finite decay that underflows to 0 against everything; NaN stays
            d = d < -1e5f ? -1e5f : d;
            v[j] = double(d) * 1.4426950408889634;
            sm.beta[warp][t] = t < n ? (a.beta ? a.beta[b * a.bs.sb + h * a.bs.sc + (t0 + t) * a.bs.st] : 1.0f) : 0.0f;
        }
        const bool grows = __any_sync(0xffffffffu, v[0] > 0.0 || v[1] > 0.0);
        if (lane == 0) sm.strict[warp] = grows ? 0x1p-18f : 0x1p-24f;
        double s = v[0] + v[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        const double s0 = s - v[1];
        sm.gh[warp][2 * lane] = float(s0);
        sm.gl[warp][2 * lane] = float(s0 - double(float(s0)));
        sm.gh[warp][2 * lane + 1] = float(s);
        sm.gl[warp][2 * lane + 1] = float(s - double(float(s)));
    }
    cp_async_wait_all();
    __syncthreads();
    // K K^T and Q K^T, rows 16 warp .., and the diagonal block of Q Q^T
    const uint32_t tk = tc::smem_u32(sm.k), tq = tc::smem_u32(sm.q);
    float ka[8][4], qa[8][4], qq[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) ka[i][j] = qa[i][j] = qq[i & 1][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t lk[4], lq[4], r[4];
        if constexpr (FIRST) {
            left_km<P>(lk, tk, warp, ks, lane);
            left_km<P>(lq, tq, warp, ks, lane);
            right_kn<P>(r, tq, ks, 2 * warp, lane);
        } else {
            left_mk<P>(lk, tk, warp, ks, lane);
            left_mk<P>(lq, tq, warp, ks, lane);
            right_nk<P>(r, tq, ks, 2 * warp, lane);
        }
        mma_bf16(qq[0], lq, r[0], r[1]);
        mma_bf16(qq[1], lq, r[2], r[3]);
#pragma unroll
        for (int nt = 0; nt < 8; nt += 2) {
            if (nt > 2 * warp) break;
            if constexpr (FIRST) right_kn<P>(r, tk, ks, nt, lane);
            else right_nk<P>(r, tk, ks, nt, lane);
            mma_bf16(ka[nt], lk, r[0], r[1]);
            mma_bf16(ka[nt + 1], lk, r[2], r[3]);
            mma_bf16(qa[nt], lq, r[0], r[1]);
            mma_bf16(qa[nt + 1], lq, r[2], r[3]);
        }
    }
    // row g of the diagonal's two tiles meets its own column in the thread that holds column pair g / 2
    if (t4 == g >> 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 16 * warp + g + 8 * i, at = 2 * i + (g & 1);
            float k2 = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (w == warp) k2 = at == 0 ? ka[2 * w][0] : at == 1 ? ka[2 * w][1] : at == 2 ? ka[2 * w + 1][2] : ka[2 * w + 1][3];
            const float q2 = at == 0 ? qq[0][0] : at == 1 ? qq[0][1] : at == 2 ? qq[1][2] : qq[1][3];
            sm.rk[t] = a.l2norm ? 1.0f / sqrtf(k2 + kDeltaNormEps) : 1.0f;
            sm.rq[t] = (a.l2norm ? 1.0f / sqrtf(q2 + kDeltaNormEps) : 1.0f) * a.scale;
            // a row's largest element is at most its norm; a norm whose square may have underflowed counts as 1e-18
            sm.kn[t] = fmaxf(sqrtf(k2), 1e-18f);
            sm.qn[t] = fmaxf(sqrtf(q2), 1e-18f);
        }
    }
    __syncthreads();                               // norms; and K, Q have been read
#pragma unroll 1
    for (int hh = 0; hh < group; ++hh) {
    const float *gh = sm.gh[hh], *gl = sm.gl[hh], *beta = sm.beta[hh];
    uint8_t* blob = x.blobs + ((b * a.Hv + h_first + hh) * int64_t(x.chunks) + chunk) * kBlob;
    Factors* f = reinterpret_cast<Factors*>(blob + 3 * kTile);
    if (tid < C) {
        const int t = tid;
        const Pow2 pk(sm.kn[t]), pq(sm.qn[t]);
        const float into = exp2f(gh[t] + gl[t]), out = exp2f((gh[C - 1] - gh[t]) + (gl[C - 1] - gl[t]));
        f->kmul[t] = pk.up;
        f->qmul[t] = pq.up;
        f->cx[t] = into * sm.rk[t] * pk.down;
        f->cu[t] = out * sm.rk[t] * pk.down;
        f->co[t] = into * sm.rq[t] * pq.down;
        if (t == 0) {
            f->gamma = exp2f(gh[C - 1] + gl[C - 1]);
            f->reach.t = f->reach.w = 0.0f;
        }
        sm.left[t] = out * sm.rk[t] * sm.kn[t];
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(sm.rk[t] * sm.kn[t]));      // not negative
        const uint32_t strong = __ballot_sync(0xffffffffu, beta[t] != 0.0f);
        if (lane == 0) {
            sm.kmost[warp] = __uint_as_float(most);
            f->strong[warp] = strong;
        }
    }
    {
        const int r0 = 16 * warp + g, r1 = r0 + 8;
        const float h0 = gh[r0], h1 = gh[r1], l0 = gl[r0], l1 = gl[r1];
        const float a0 = beta[r0] * sm.rk[r0], a1 = beta[r1] * sm.rk[r1];
        const float q0 = sm.rq[r0], q1 = sm.rq[r1];
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            if (nt > 2 * warp + 1) break;          // what lies right of the diagonal's blocks is not read
            const int c = 8 * nt + 2 * t4;
            const float2 hc = *reinterpret_cast<const float2*>(&gh[c]), lc = *reinterpret_cast<const float2*>(&gl[c]);
            const float2 rc = *reinterpret_cast<const float2*>(&sm.rk[c]), bc = *reinterpret_cast<const float2*>(&beta[c]);
            const float d[4] = {exp2f((h0 - hc.x) + (l0 - lc.x)) * rc.x, exp2f((h0 - hc.y) + (l0 - lc.y)) * rc.y,
                                exp2f((h1 - hc.x) + (l1 - lc.x)) * rc.x, exp2f((h1 - hc.y) + (l1 - lc.y)) * rc.y};
            float av[4], pv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j < 2 ? r0 : r1, cc = c + (j & 1);
                av[j] = cc < r ? (j < 2 ? a0 : a1) * d[j] * ka[nt][j] : 0.0f;
                // what is never written is not read either, and does not set the row's scale
                pv[j] = cc <= r && ((j & 1) ? bc.y : bc.x) != 0.0f ? d[j] * (j < 2 ? q0 : q1) * qa[nt][j] : 0.0f;
            }
            m0 = fmaxf(m0, fmaxf(fabsf(pv[0]), fabsf(pv[1])));
            m1 = fmaxf(m1, fmaxf(fabsf(pv[2]), fabsf(pv[3])));
            *reinterpret_cast<float2*>(&sm.A[r0][c]) = make_float2(av[0], av[1]);
            *reinterpret_cast<float2*>(&sm.A[r1][c]) = make_float2(av[2], av[3]);
            // P waits where T comes later, each thread's for itself
            *reinterpret_cast<float2*>(&sm.T[r0][c]) = make_float2(pv[0], pv[1]);
            *reinterpret_cast<float2*>(&sm.T[r1][c]) = make_float2(pv[2], pv[3]);
        }
        // A row of P goes to fp16 under its own largest element: a bound from the norms and gates (one product of it may be
        // large where the row's elements are not, with gates of either sign or a later large key) would cost it all its bits.
        const Pow2 p0(quad_max(m0)), p1(quad_max(m1));
        if (t4 == 0) {
            f->cp[r0] = p0.down;
            f->cp[r1] = p1.down;
        }
        uint8_t* P2 = blob + 2 * kTile + 4 * t4;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            if (nt > 2 * warp + 1) break;
            const int c = 8 * nt + 2 * t4;
            const float2 v0 = *reinterpret_cast<const float2*>(&sm.T[r0][c]), v1 = *reinterpret_cast<const float2*>(&sm.T[r1][c]);
            *reinterpret_cast<uint32_t*>(P2 + piece<8>(r0, nt)) = pack_h(v0.x * p0.up, v0.y * p0.up);
            *reinterpret_cast<uint32_t*>(P2 + piece<8>(r1, nt)) = pack_h(v1.x * p1.up, v1.y * p1.up);
        }
    }
    __syncthreads();
    if (lane < 16) {
        const int o = 16 * warp;
        float xx[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == lane ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(&sm.A[o + i][o + j]);
                s0 = fmaf(-w.x, xx[j], s0);
                if (j + 1 < i) s1 = fmaf(-w.y, xx[j + 1], s1);
                if (j + 2 < i) s0 = fmaf(-w.z, xx[j + 2], s0);
                if (j + 3 < i) s1 = fmaf(-w.w, xx[j + 3], s1);
            }
            xx[i] = s0 + s1;
            sm.T[o + i][o + lane] = xx[i];
        }
    } else if (!(warp & 1)) {
        // right of the first and third block: read as part of a 32 x 32 inverse
#pragma unroll
        for (int i = 0; i < 16; ++i) sm.T[16 * warp + i][16 * warp + lane] = 0.0f;
    }
    __syncthreads();
    block_under<16>(sm, 32 * (tid >> 6), 16 * (tid >> 6), tid & 63);
    block_under<32>(sm, 0, 0, tid);
    // T diag(beta) in two parts: two threads a row, half of the columns each
    {
        const int r = tid >> 1, c0 = (tid & 1) * 32;
        float m = 0.0f;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] = c0 + i <= r ? sm.T[r][c0 + i] * beta[c0 + i] : 0.0f;
            m = fmaxf(m, fabsf(v[i]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const Pow2 p(m);
        if (c0 == 0) f->ct[r] = p.down;
        // not negative, so ordered as their bits; NaN above all, and then no comparison holds
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(m * sm.left[r])));
        if (lane == 0) {
            atomicMax(reinterpret_cast<uint32_t*>(&f->reach.t), most);
            atomicMax(reinterpret_cast<uint32_t*>(&f->reach.w), __float_as_uint(__uint_as_float(w) * sm.strict[hh]));
        }
        if (tid == 0) f->reach.k = fmaxf(sm.kmost[0], sm.kmost[1]) * 0x1p-28f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c0 + 8 * i > (r | 15)) break;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split_h(v[8 * i + 2 * j] * p.up, v[8 * i + 2 * j + 1] * p.up, hi[j], lo[j]);
            const uint32_t at = piece<8>(r, c0 / 8 + i);
            *reinterpret_cast<uint4*>(blob + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(blob + kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    if (GROUP) __syncthreads();                    // A and T may be written again
    }
}

// ----------------------------------------------------------------------- scan
// A CTA takes 16 NW value channels of a head: NW warps of 16 channels each (the
// channels never mix) and four loading warps.  A warp works on the transposes,
// S^T [16 x DK] in accumulators: each product's result is the next one's left
// operand as it lies in registers,
//   X^T = S^T K^T,  R^T = V^T - X^T diag(cx),  U^T = R^T T^T,  S^T += U^T diag(cu) K,
// so a chunk's chain has no shared-memory round trip and no barrier.  The
// loaders bring K and Q to fp16 under their powers of two, V as it is, and T, P
// and the factors as one bulk copy, two chunks deep.
// mma.sync, not tcgen05: the chain's four dependent products go from registers
// to registers here, where each of tcgen05's would wait for a commit, a read of
// tensor memory, the split into two parts and a store of it.
// A chunk of 128 channels takes 11900 cycles for 6400 of products (eight warps,
// 43 % of the tensor pipe, 39 % of the issue slots), of 64 channels 7500 for
// 3200: the splits and scalings between the products of an in-order warp bound
// it, and the registers of the state the number of warps (with eight, dk = 128,
// 100 to 128 bytes a thread are spilled, with four 32 to 84).  256 heads of 64
// chunks 908 us.
constexpr int kLoaders = 128;
constexpr int kVRow = 72;                          // elements of a V^T row: pairs of 8 rows on 32 banks
constexpr int kORow = 16;                          // elements of a token's row of a warp's outputs

// Chunks whose magnitudes lie too far apart for the products.  A channel's R and
// U, and a row of T and P, go in under one power of two each, whose fp16 numbers
// end at 2^-39 of the largest.  A value far above its neighbours (one that a write
// strength of 0 masks, too), a large state that a gate empties halfway, keys of
// very unequal size, or gates that grow the state would thus cost the other
// tokens their outputs, or the state its bits.  Such a chunk is told from a
// channel's largest numbers before its state changes, and the warp takes it token
// by token in fp32: 64 tokens take 36 us with the narrow scan (2.4 us by products,
// dk = 64), 75 us with 64 channels a CTA (5.3, dk = 128).
//   state    what remains of it and of the writes below 2^-24 of the largest
//            residual times the largest of T (2^-18 where gates grow the state):
//            above that the errors of U, 2^-39 of those, stay within 2^-16 of the
//            state (measured: 2^-22 up to ratios of 2^18, 2^-20 at 2^20, 2^-16 at 2^24);
//   outputs  what remains of the state and of the writes, key and decay with them,
//            below 2^-28 of the largest write and key; or, where the state before
//            the chunk is below that too, the first write or two neighbouring ones
//            below 2^-28 of the largest.  (Largest write: or residual times T.)
// Three looks: the smallest write of all, which zeros trip; without the tokens of
// write strength 0; by channel and neighbours, where a write is one that has a
// value or a state, since U itself may have become 0.
// A single write far below the others is left alone: mostly their terms make the
// output, and chance brings one in 10^4 chunks.  (Where a strong decay has emptied
// those terms too, that one output, below 2^-28 of its neighbours', loses bits.)
// Looking for all this costs 1 % (16 x 4096 x 16 heads 1195 -> 1206 us, 4 x 8192 x
// 6 heads 433 -> 438 us), at dk = 64 5 to 9 % (144 heads of 16 chunks 95 -> 99 us,
// token-major rows 99 -> 107); a third look costs its CTA some 10 us.

template <int DK, int VR, int VC>
struct ScanStage {
    alignas(128) uint8_t k[C * DK * 2], q[C * DK * 2];
    alignas(128) uint8_t blob[kBlob];              // T high, T low, P, factors
    alignas(16) bf16 v[VR][VC];
};
template <int DK, int NW>
struct ScanSmem {
    using Stage = ScanStage<DK, 16 * NW, kVRow>;
    Stage st[2];
    alignas(16) bf16 o[NW][16 * kVRow];            // [channel][kVRow], or [time][kORow]
    uint64_t full[2], empty[2];
};

__device__ __forceinline__ uint4 scaled8(const uint4& w, const float (&m)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_h(bf(u[i], 0) * m[2 * i], bf(u[i], 1) * m[2 * i + 1]);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// A K or Q tile into shared memory, then (by the same threads, each its own octets) to fp16 in place under the tokens'
// powers of two: m holds those of this thread's eight tokens (FIRST), mul those of all.
template <int DK, bool FIRST>
__device__ __forceinline__ void load_tile(uint8_t* tile, const bf16* p, const DeltaView& s, int dk, int n, bool vec, int lt) {
    constexpr int P = FIRST ? 8 : DK / 8, kOct = C * DK / 8 / kLoaders;
    if (whole<FIRST>(dk, n, vec)) {
#pragma unroll
        for (int j = 0; j < kOct; ++j) {
            const int row = (lt + j * kLoaders) / P, c = (lt + j * kLoaders) % P;
            copy_octet<FIRST>(tile + piece<P>(row, c), p, s, FIRST ? row : 8 * c, FIRST ? 8 * c : row, dk, n);
        }
    } else {
#pragma unroll 2
        for (int i = lt; i < C * DK / 8; i += kLoaders) {
            const int row = i / P, c = i % P;
            *reinterpret_cast<uint4*>(tile + piece<P>(row, c)) = octet<FIRST>(p, s, FIRST ? row : 8 * c, FIRST ? 8 * c : row, dk, n);
        }
    }
}
template <int DK, bool FIRST>
__device__ __forceinline__ void scale_tile(uint8_t* tile, const float (&m)[8], const float* mul, int lt) {
    constexpr int P = FIRST ? 8 : DK / 8, kOct = C * DK / 8 / kLoaders;
#pragma unroll
    for (int j = 0; j < kOct; ++j) {
        const int row = (lt + j * kLoaders) / P, c = (lt + j * kLoaders) % P;
        uint4* at = reinterpret_cast<uint4*>(tile + piece<P>(row, c));
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = FIRST ? m[i] : mul[row];
        *at = scaled8(*at, f);
    }
}

// V^T [16 NW][kVRow]; from tokens' rows (not FIRST) eight channels of two tokens each way, as pairs of tokens lie together.
template <int NW, bool FIRST>
__device__ __forceinline__ void load_values(bf16 (&v)[16 * NW][kVRow], const bf16* p, const DeltaView& s, int cols, int n,
                                            bool vec, int lt) {
    constexpr int kOct = 16 * NW * 8 / kLoaders;
    if constexpr (FIRST) {
        auto put = [&](int i, const uint4& w) { *reinterpret_cast<uint4*>(&v[i / 8][8 * (i % 8)]) = w; };
        if (whole<true>(cols, n, vec)) {
#pragma unroll
            for (int j = 0; j < kOct; ++j) {
                const int i = lt + j * kLoaders;
                copy_octet<true>(&v[i / 8][8 * (i % 8)], p, s, i / 8, 8 * (i % 8), cols, n);
            }
        } else {
#pragma unroll 1
            for (int i = lt; i < 16 * NW * 8; i += kLoaders) put(i, octet<true>(p, s, i / 8, 8 * (i % 8), cols, n));
        }
    } else {
        // neighbouring lanes: neighbouring octets of a token's row, so whole sectors are read
        constexpr int kRowOct = 2 * NW;
        auto put = [&](int i, const uint4& w0, const uint4& w1) {
            const int tp = i / kRowOct, c = i % kRowOct;
            const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint32_t*>(&v[8 * c + j][2 * tp]) = __byte_perm(u0[j >> 1], u1[j >> 1], (j & 1) ? 0x7632 : 0x5410);
        };
        if (whole<false>(cols, n, vec)) {
            uint4 w[kOct];
#pragma unroll
            for (int j = 0; j < kOct / 2; ++j) {
                const int i = lt + j * kLoaders;
                w[2 * j] = whole_octet<false>(p, s, 8 * (i % kRowOct), 2 * (i / kRowOct), cols, n);
                w[2 * j + 1] = whole_octet<false>(p, s, 8 * (i % kRowOct), 2 * (i / kRowOct) + 1, cols, n);
            }
#pragma unroll
            for (int j = 0; j < kOct / 2; ++j) put(lt + j * kLoaders, w[2 * j], w[2 * j + 1]);
        } else {
#pragma unroll 1
            for (int i = lt; i < 32 * kRowOct; i += kLoaders)
                put(i, octet<false>(p, s, 8 * (i % kRowOct), 2 * (i / kRowOct), cols, n),
                    octet<false>(p, s, 8 * (i % kRowOct), 2 * (i / kRowOct) + 1, cols, n));
        }
    }
}

// The scans launch while the last CTAs of k_delta_prep drain and wait here for what it wrote; nothing in global memory is
// read or written before.
__device__ __forceinline__ void after_prep() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// A warp that gives up: the copies of the chunks [from, to) that may be in flight land first.
__device__ __forceinline__ void landed(uint64_t* full, int from, int to, uint64_t budget_ns) {
    for (int c = max(from, 0); c < to; ++c) tc::mbar_wait(&full[c & 1], uint32_t(c >> 1) & 1u, budget_ns);
}

// The loading warps of a scanning CTA whose channels start at d0 (cols of them): `put_v` brings V.
template <int DK, bool FIRST, typename Sm, typename PutV>
__device__ __forceinline__ void run_loaders(Sm& sm, const ChunkArgs& x, int lt, int lane, int h, int64_t b, int len, int d0,
                                            PutV put_v) {
    const DeltaArgs& a = x.a;
    const int chunks = (len + C - 1) / C;
    const int kh = h / (a.Hv / a.Hk);
    const bf16* kp = static_cast<const bf16*>(a.k) + b * a.ks.sb + int64_t(kh) * a.dk * a.ks.sc;
    const bf16* qp = static_cast<const bf16*>(a.q) + b * a.qs.sb + int64_t(kh) * a.dk * a.qs.sc;
    const bf16* vp = static_cast<const bf16*>(a.v) + b * a.vs.sb + (int64_t(h) * a.dv + d0) * a.vs.sc;
    const uint8_t* blobs = x.blobs + (b * a.Hv + h) * int64_t(x.chunks) * kBlob;
    for (int ch = 0; ch < chunks; ++ch) {
        const int s = ch & 1;
        auto& st = sm.st[s];
        if (!tc::mbar_wait(&sm.empty[s], (uint32_t(ch >> 1) & 1u) ^ 1u, x.budget_ns)) {
            if (lane == 0) report_status(x.status, kStatusTimeout);
            landed(sm.full, ch - 2, ch, x.budget_ns);
            break;
        }
        const uint8_t* blob = blobs + int64_t(ch) * kBlob;
        if (lt == 0) {
            tc::mbar_expect_tx(&sm.full[s], kBlob);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                             tc::smem_u32(st.blob)), "l"(blob), "r"(kBlob), "r"(tc::smem_u32(&sm.full[s]))
                         : "memory");
        }
        const int64_t t0 = int64_t(ch) * C;
        const int n = min(C, len - ch * C);
        load_tile<DK, FIRST>(st.k, kp + t0 * a.ks.st, a.ks, a.dk, n, x.vec_k, lt);
        load_tile<DK, FIRST>(st.q, qp + t0 * a.qs.st, a.qs, a.dk, n, x.vec_q, lt);
        const Factors* f = reinterpret_cast<const Factors*>(blob + 3 * kTile);
        float mk[8], mq[8];
        if constexpr (FIRST) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {          // this thread's eight tokens
                mk[i] = f->kmul[8 * (lt % 8) + i];
                mq[i] = f->qmul[8 * (lt % 8) + i];
            }
        }
        put_v(st, vp + t0 * a.vs.st, n);
        cp_async_commit();
        cp_async_wait_all();
        scale_tile<DK, FIRST>(st.k, mk, f->kmul, lt);
        scale_tile<DK, FIRST>(st.q, mq, f->qmul, lt);
        tc::mbar_arrive(&sm.full[s]);
    }
    // else the scanning warps wait for every stage, also those that give up
}

// What a scanning warp leaves that gave up waiting for chunk ch: NaN from its first token on for its channels.  Called, not
// inlined, which costs the prefill form 2 %.
__device__ __noinline__ void give_up(uint64_t* full, int ch, uint64_t budget_ns, bf16* o, int64_t channel, int64_t token, int cols,
                                     int len) {
    const int t0 = ch * C;
    landed(full, ch, min(ch + 2, (len + C - 1) / C), budget_ns);
    const bf16 nan = __float2bfloat16_rn(__int_as_float(0x7fffffff));
    for (int c = 0; c < cols; ++c)
        for (int64_t t = t0 + int(threadIdx.x & 31); t < len; t += 32) o[c * channel + t * token] = nan;
}

// The second look at a chunk whose smallest write is small: without the tokens that write nothing (a write strength of 0,
// behind the end).
template <bool WIDE>
__device__ __forceinline__ uint64_t strong_from(const Factors& f, int lane) {      // from this lane's first token on
    return (uint64_t(f.strong[1]) << 32 | f.strong[0]) >> (WIDE ? 2 * (lane & 3) : lane >> 2);
}
template <bool WIDE, int J>
__device__ __forceinline__ bool small_writes(const float (&U)[J][4], const Factors& f, int lane, float m0, float m1) {
    const uint64_t strong = strong_from<WIDE>(f, lane);
    float z0 = INFINITY, z1 = INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (strong >> (WIDE ? 8 * j + i : 16 * j + 8 * i) & 1u) {
                z0 = fminf(z0, fabsf(U[j][WIDE ? i : 2 * i]));
                z1 = fminf(z1, fabsf(U[j][WIDE ? 2 + i : 2 * i + 1]));
            }
    return __any_sync(0xffffffffu, z0 < m0 * 0x1p-28f || z1 < m1 * 0x1p-28f);
}

// The third: what was said above, channel by channel.  U as the scans hold it (WIDE: element 2 c + i of tile j
// is channel c, token 8 j + 2 t4 + i; else element 2 i + c, token 16 j + g + 8 i); v: this thread's first channel.
struct Writes {
    const Factors* f;
    const bf16* v;
    int v_channel, v_token;
    float m[2], s[2];                              // as in Reach, by channel
};
template <bool WIDE, int J>
__device__ __forceinline__ bool look_again(const float (&U)[J][4], const Writes& x) {
    const int lane = int(threadIdx.x) & 31, g = lane >> 2, t4 = lane & 3;
    auto token = [&](int j, int i) { return WIDE ? 8 * j + 2 * t4 + i : 16 * j + g + 8 * i; };
    auto at = [](int c, int i) { return WIDE ? 2 * c + i : 2 * i + c; };
    bool far = false;
    const Reach reach = x.f->reach;
    const float gamma = x.f->gamma;
    const uint64_t strong = strong_from<WIDE>(*x.f, lane);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        // U may be 0 because it was too small: a token writes where there is a value or a state
        unsigned live = 0;
        int first = C;
#pragma unroll
        for (int j = J - 1; j >= 0; --j)
#pragma unroll
            for (int i = 1; i >= 0; --i) {
                const int t = token(j, i);
                if ((strong >> (t - token(0, 0)) & 1u) != 0 && (x.s[c] > 0.0f || __bfloat162float(x.v[c * x.v_channel + t * x.v_token]) != 0.0f)) {
                    live |= 1u << (2 * j + i);
                    first = t;
                }
            }
#pragma unroll
        for (int d = WIDE ? 1 : 4; d < (WIDE ? 4 : 32); d <<= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
        const bool bare = reach.bare(x.m[c], x.s[c], gamma);
        // neighbouring tokens: the other of this thread's two, or another lane's
        const unsigned pair = WIDE ? live | (live >> 1 & 0x5555u) | (live << 1 & 0xaaaau) : live | __shfl_xor_sync(0xffffffffu, live, 4);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float own = fabsf(U[j][at(c, i)]);
                const float other = WIDE ? fabsf(U[j][at(c, i ^ 1)]) : __shfl_xor_sync(0xffffffffu, own, 4);
                far = far || (bare && (((pair >> (2 * j + i) & 1u) != 0 && fmaxf(own, other) < x.m[c] * 0x1p-28f) ||
                                       (first == token(j, i) && own < x.m[c] * 0x1p-28f)));
            }
    }
    return __any_sync(0xffffffffu, far);
}
// Called by the wide scan, for the same reason as chunk_by_token_apart.
template <int J>
__device__ __noinline__ bool look_again_apart(const float (&U)[J][4], const Writes& x) {
    float own[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) own[j][i] = U[j][i];
    return look_again<true>(own, x);
}

// One element of a tile of 16-bit numbers [token][channel], or (FIRST) [channel][token].
template <int DK, bool FIRST>
__device__ __forceinline__ __half tile_at(const uint8_t* tile, int t, int ch) {
    const uint32_t at = FIRST ? piece<8>(ch, t >> 3) + 2u * uint32_t(t & 7) : piece<DK / 8>(t, ch >> 3) + 2u * uint32_t(ch & 7);
    return *reinterpret_cast<const __half*>(tile + at);
}

// n tokens of a chunk one by one, from the definition.  The state as the scans hold it, two channels a thread: WIDE
// S^T tiles (element i: channel i / 2, row 8 j + 2 t4 + i % 2), else S tiles (channel i % 2, row 16 j + g + 8 (i / 2)).
// v, o: this thread's first channel at the chunk's first token, in shared memory, with the strides of channel and token;
// gate, beta: the chunk's, or nullptr.
struct Tokens {
    const uint8_t *k, *q;
    const float *kmul, *qmul, *gate, *beta;
    int64_t gate_step, beta_step;
    const bf16* v;
    bf16* o;
    int v_channel, v_token, o_channel, o_token;
    int n, l2norm;
    float scale;
};
template <int DK, bool FIRST, bool WIDE, int J>
__device__ __forceinline__ void chunk_by_token(float (&S)[J][4], const Tokens& x) {
    const int lane = int(threadIdx.x) & 31;
    const int g = lane >> 2, t4 = lane & 3;
    auto row = [&](int j, int e) { return WIDE ? 8 * j + 2 * t4 + e : 16 * j + g + 8 * e; };      // e: one of a tile's two
    auto whole_sum = [&](float v) {                // over the lanes that share this one's channels
#pragma unroll
        for (int d = WIDE ? 1 : 4; d < (WIDE ? 4 : 32); d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    };
    auto at = [](int c, int e) { return WIDE ? 2 * c + e : 2 * e + c; };                          // S[j][at(channel, e)]
    // the gates of tokens `lane` and lane + 32
    float al[2], be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        al[i] = x.gate && t < x.n ? expf(x.gate[t * x.gate_step]) : 1.0f;
        be[i] = x.beta && t < x.n ? x.beta[t * x.beta_step] : 1.0f;
    }
#pragma unroll 1
    for (int t = 0; t < x.n; ++t) {
        __half2 k[J], q[J];
        float k2 = 0.0f, q2 = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            k[j] = __halves2half2(tile_at<DK, FIRST>(x.k, t, row(j, 0)), tile_at<DK, FIRST>(x.k, t, row(j, 1)));
            q[j] = __halves2half2(tile_at<DK, FIRST>(x.q, t, row(j, 0)), tile_at<DK, FIRST>(x.q, t, row(j, 1)));
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float2 kk = __half22float2(k[j]), qq = __half22float2(q[j]);
            k2 = fmaf(kk.x, kk.x, fmaf(kk.y, kk.y, k2));
            q2 = fmaf(qq.x, qq.x, fmaf(qq.y, qq.y, q2));
            x0 = fmaf(S[j][at(0, 0)], kk.x, fmaf(S[j][at(0, 1)], kk.y, x0));
            x1 = fmaf(S[j][at(1, 0)], kk.x, fmaf(S[j][at(1, 1)], kk.y, x1));
        }
        // the tiles hold K and Q times their rows' powers of two
        const float dk = 1.0f / x.kmul[t], dq = 1.0f / x.qmul[t];
        k2 = whole_sum(k2) * dk * dk;
        q2 = whole_sum(q2) * dq * dq;
        const float rk = (x.l2norm ? 1.0f / sqrtf(k2 + kDeltaNormEps) : 1.0f) * dk;
        const float rq = (x.l2norm ? 1.0f / sqrtf(q2 + kDeltaNormEps) : 1.0f) * x.scale * dq;
        const float a = __shfl_sync(0xffffffffu, t < 32 ? al[0] : al[1], t & 31), b = __shfl_sync(0xffffffffu, t < 32 ? be[0] : be[1], t & 31);
        const float v0 = __bfloat162float(x.v[t * x.v_token]), v1 = __bfloat162float(x.v[x.v_channel + t * x.v_token]);
        const float u0 = b * (v0 - a * (whole_sum(x0) * rk)) * rk;
        const float u1 = b * (v1 - a * (whole_sum(x1) * rk)) * rk;
        float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float2 kk = __half22float2(k[j]), qq = __half22float2(q[j]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float &s0 = S[j][at(c, 0)], &s1 = S[j][at(c, 1)], &y = c ? y1 : y0;
                s0 = fmaf(kk.x, c ? u1 : u0, a * s0);
                s1 = fmaf(kk.y, c ? u1 : u0, a * s1);
                y = fmaf(s0, qq.x, fmaf(s1, qq.y, y));
            }
        }
        y0 = whole_sum(y0) * rq;
        y1 = whole_sum(y1) * rq;
        if ((WIDE ? t4 : g) == 0) {                // one of the lanes that share these channels
            x.o[t * x.o_token] = __float2bfloat16_rn(y0);
            x.o[x.o_channel + t * x.o_token] = __float2bfloat16_rn(y1);
        }
    }
}
template <int J>
__device__ __forceinline__ void copy_state(float (&to)[J][4], const float (&from)[J][4]) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[j][i] = from[j][i];
}
template <int DK, bool FIRST, int J>
__device__ __noinline__ void chunk_by_token_apart(float (&S)[J][4], const Tokens& x) {
    float own[J][4];                               // registers again
    copy_state(own, S);
    chunk_by_token<DK, FIRST, true>(own, x);
    copy_state(S, own);
}
// The same for a scan's state in registers.  The wide scan calls it, which leaves its own registers alone (16 x 4096 x 16
// heads 1229 us, inlined 1243); in the narrow one it is inlined (4 x 8192 x 6 heads 434 us, called 446).
template <int DK, bool FIRST, bool WIDE, int J>
__device__ __forceinline__ void state_by_token(float (&S)[J][4], const uint8_t* k, const uint8_t* q, const Factors& f,
                                               const DeltaArgs& a, int64_t b, int h, int64_t t0, int n, const bf16* v, int v_channel,
                                               int v_token, bf16* o, int o_channel, int o_token) {
    const Tokens x{k, q, f.kmul, f.qmul, a.g ? a.g + b * a.gs.sb + h * a.gs.sc + t0 * a.gs.st : nullptr,
                   a.beta ? a.beta + b * a.bs.sb + h * a.bs.sc + t0 * a.bs.st : nullptr, a.gs.st, a.bs.st, v, o,
                   v_channel, v_token, o_channel, o_token, n, a.l2norm, a.scale};
    if constexpr (WIDE) {
        float copy[J][4];
        copy_state(copy, S);
        chunk_by_token_apart<DK, FIRST>(copy, x);
        copy_state(S, copy);
    } else {
        chunk_by_token<DK, FIRST, false>(S, x);
    }
}

template <int DK, int NW, bool FIRST>
__global__ void __launch_bounds__(32 * NW + kLoaders, 1) k_delta_scan(ChunkArgs x) {
    using Sm = ScanSmem<DK, NW>;
    constexpr int P = FIRST ? 8 : DK / 8;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    const DeltaArgs& a = x.a;
    const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int h = int(blockIdx.y), d0 = int(blockIdx.x) * 16 * NW;
    const int64_t b = blockIdx.z;
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&sm.full[s], kLoaders + 1);
            tc::mbar_init(&sm.empty[s], NW);
        }
    }
    __syncthreads();
    after_prep();
    const int len = int(length_of(a, b)), chunks = (len + C - 1) / C;      // L <= 2^30
    if (warp >= NW) {
        // ------------------------------------------------------------ loaders
        // registers of eight warps: 384 x 168 at launch = 128 x 56 + 256 x 224
        if constexpr (NW == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
        const int lt = tid - 32 * NW, cols = min(16 * NW, a.dv - d0);
        run_loaders<DK, FIRST>(sm, x, lt, lane, h, b, len, d0, [&](typename Sm::Stage& st, const bf16* p, int n) {
            load_values<NW, FIRST>(st.v, p, a.vs, cols, n, x.vec_v, lt);
        });
        return;
    }
    // ------------------------------------------------------------------- scan
    if constexpr (NW == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n");
    const int g = lane >> 2, t4 = lane & 3;
    const int dw = d0 + 16 * warp;                 // this warp's first channel
    const int64_t sb = (b * a.Hv + h) * int64_t(a.dk) * a.dv;
    float S[DK / 8][4];
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = dw + g + 8 * (i >> 1), r = 8 * j + 2 * t4 + (i & 1);
            S[j][i] = (a.state_in && d < a.dv && r < a.dk) ? a.state_in[sb + int64_t(r) * a.dv + d] : 0.0f;
        }
    bf16* ob = static_cast<bf16*>(a.o) + b * a.os.sb + (int64_t(h) * a.dv + dw) * a.os.sc;
    bf16* so = sm.o[warp];
    int ch = 0;
    for (; ch < chunks; ++ch) {
        const int s = ch & 1;
        typename Sm::Stage& st = sm.st[s];
        if (!tc::mbar_wait(&sm.full[s], uint32_t(ch >> 1) & 1u, x.budget_ns)) break;
        const int64_t t0 = int64_t(ch) * C;
        const int n = min(C, len - ch * C);
        const uint32_t tk = tc::smem_u32(st.k), tq = tc::smem_u32(st.q), tb = tc::smem_u32(st.blob);
        const Factors& f = *reinterpret_cast<const Factors*>(st.blob + 3 * kTile);
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int j = 0; j < DK / 8; ++j) {
            m0 = fmaxf(m0, fmaxf(fabsf(S[j][0]), fabsf(S[j][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(S[j][2]), fabsf(S[j][3])));
        }
        const float s0 = quad_max(m0), s1 = quad_max(m1);
        const Pow2 ps0(s0), ps1(s1);
        float X[8][4], O[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) X[i][j] = O[i][j] = 0.0f;
        // right operands are read a step (six products) ahead of their use
        auto keys = [&](uint32_t (&r)[4], uint32_t (&w)[4], int step) {
            if constexpr (FIRST) {
                right_kn<P>(r, tk, step / 4, 2 * (step % 4), lane);
                right_kn<P>(w, tq, step / 4, 2 * (step % 4), lane);
            } else {
                right_nk<P>(r, tk, step / 4, 2 * (step % 4), lane);
                right_nk<P>(w, tq, step / 4, 2 * (step % 4), lane);
            }
        };
        {
            uint32_t r[2][4], w[2][4], hi[4], lo[4];
            keys(r[0], w[0], 0);
#pragma unroll
            for (int step = 0; step < DK / 4; ++step) {
                const int ks = step / 4, nt = 2 * (step % 4), at = step & 1;
                if (step + 1 < DK / 4) keys(r[at ^ 1], w[at ^ 1], step + 1);
                if (nt == 0) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        split_h(S[2 * ks + j][0] * ps0.up, S[2 * ks + j][1] * ps0.up, hi[2 * j], lo[2 * j]);
                        split_h(S[2 * ks + j][2] * ps1.up, S[2 * ks + j][3] * ps1.up, hi[2 * j + 1], lo[2 * j + 1]);
                    }
                }
                mma_f16(X[nt], hi, r[at][0], r[at][1]);
                mma_f16(X[nt + 1], hi, r[at][2], r[at][3]);
                mma_f16(O[nt], hi, w[at][0], w[at][1]);
                mma_f16(O[nt + 1], hi, w[at][2], w[at][3]);
                mma_f16(X[nt], lo, r[at][0], r[at][1]);
                mma_f16(X[nt + 1], lo, r[at][2], r[at][3]);
            }
        }
        // R^T = V^T - X^T diag(cx); the outputs' part of the state
        m0 = m1 = 0.0f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const int t = 8 * nt + 2 * t4;
            const float2 cx = *reinterpret_cast<const float2*>(&f.cx[t]), co = *reinterpret_cast<const float2*>(&f.co[t]);
            const uint32_t v0 = *reinterpret_cast<const uint32_t*>(&st.v[16 * warp + g][t]);
            const uint32_t v1 = *reinterpret_cast<const uint32_t*>(&st.v[16 * warp + g + 8][t]);
            X[nt][0] = fmaf(-X[nt][0] * ps0.down, cx.x, bf(v0, 0));
            X[nt][1] = fmaf(-X[nt][1] * ps0.down, cx.y, bf(v0, 1));
            X[nt][2] = fmaf(-X[nt][2] * ps1.down, cx.x, bf(v1, 0));
            X[nt][3] = fmaf(-X[nt][3] * ps1.down, cx.y, bf(v1, 1));
            m0 = fmaxf(m0, fmaxf(fabsf(X[nt][0]), fabsf(X[nt][1])));
            m1 = fmaxf(m1, fmaxf(fabsf(X[nt][2]), fabsf(X[nt][3])));
            O[nt][0] = O[nt][0] * ps0.down * co.x;
            O[nt][1] = O[nt][1] * ps0.down * co.y;
            O[nt][2] = O[nt][2] * ps1.down * co.x;
            O[nt][3] = O[nt][3] * ps1.down * co.y;
        }
        const float r0 = quad_max(m0), r1 = quad_max(m1);
        const Pow2 pr0(r0), pr1(r1);
        // U^T = R^T T^T, tiles on and right of the diagonal
        float U[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) U[i][j] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                split_h(X[2 * ks + j][0] * pr0.up, X[2 * ks + j][1] * pr0.up, hi[2 * j], lo[2 * j]);
                split_h(X[2 * ks + j][2] * pr1.up, X[2 * ks + j][3] * pr1.up, hi[2 * j + 1], lo[2 * j + 1]);
            }
#pragma unroll
            for (int nt = 2 * ks; nt < 8; nt += 2) {
                uint32_t r[4], w[4];
                right_nk<8>(r, tb, ks, nt, lane);
                right_nk<8>(w, tb + kTile, ks, nt, lane);
                mma_f16(U[nt], hi, r[0], r[1]);
                mma_f16(U[nt + 1], hi, r[2], r[3]);
                mma_f16(U[nt], lo, r[0], r[1]);
                mma_f16(U[nt + 1], lo, r[2], r[3]);
                mma_f16(U[nt], hi, w[0], w[1]);
                mma_f16(U[nt + 1], hi, w[2], w[3]);
            }
        }
        m0 = m1 = 0.0f;
        float z0 = INFINITY, z1 = z0;              // the smallest write: of the first tokens each, then of two the larger
        float n0 = 0.0f, n1 = 0.0f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const int t = 8 * nt + 2 * t4;
            const float2 ct = *reinterpret_cast<const float2*>(&f.ct[t]), cu = *reinterpret_cast<const float2*>(&f.cu[t]);
            U[nt][0] = U[nt][0] * pr0.down * ct.x;
            U[nt][1] = U[nt][1] * pr0.down * ct.y;
            U[nt][2] = U[nt][2] * pr1.down * ct.x;
            U[nt][3] = U[nt][3] * pr1.down * ct.y;
            const float p0 = fmaxf(fabsf(U[nt][0]), fabsf(U[nt][1])), p1 = fmaxf(fabsf(U[nt][2]), fabsf(U[nt][3]));
            m0 = fmaxf(m0, p0);
            m1 = fmaxf(m1, p1);
            z0 = fminf(z0, nt == 0 ? fminf(fabsf(U[nt][0]), fabsf(U[nt][1])) : p0);
            z1 = fminf(z1, nt == 0 ? fminf(fabsf(U[nt][2]), fabsf(U[nt][3])) : p1);
            X[nt][0] = U[nt][0] * cu.x;
            X[nt][1] = U[nt][1] * cu.y;
            X[nt][2] = U[nt][2] * cu.x;
            X[nt][3] = U[nt][3] * cu.y;
            n0 = fmaxf(n0, fmaxf(fabsf(X[nt][0]), fabsf(X[nt][1])));
            n1 = fmaxf(n1, fmaxf(fabsf(X[nt][2]), fabsf(X[nt][3])));
        }
        const float u0 = quad_max(m0), u1 = quad_max(m1), w0 = quad_max(n0), w1 = quad_max(n1), gamma = f.gamma;
        const Reach reach = f.reach;
        const float a0 = fmaxf(u0, r0 * reach.t), a1 = fmaxf(u1, r1 * reach.t);
        const bool end = reach.end(a0, r0, w0, s0, gamma) || reach.end(a1, r1, w1, s1, gamma);
        bool apart = __any_sync(0xffffffffu, end || z0 < a0 * 0x1p-28f || z1 < a1 * 0x1p-28f);
        if (__builtin_expect(apart, 0) && !__any_sync(0xffffffffu, end)) {     // or tokens that write nothing, or chance?
            apart = small_writes<true>(U, f, lane, a0, a1);
            if (apart) {
                float copy[8][4];
                copy_state(copy, U);
                apart = look_again_apart(copy, Writes{&f, &st.v[16 * warp + g][0], 8 * kVRow, 1, {a0, a1}, {s0, s1}});
            }
        }
        if (__builtin_expect(apart, 0)) {
            state_by_token<DK, FIRST, true>(S, st.k, st.q, f, a, b, h, t0, n, &st.v[16 * warp + g][0], 8 * kVRow, 1,
                                            so + g * (FIRST ? kVRow : 1), 8 * (FIRST ? kVRow : 1), FIRST ? 1 : kORow);
        } else {
            const Pow2 pu0(u0), pu1(u1), pw0(w0), pw1(w1);
            uint32_t hi[4][4], lo[4][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    split_h(X[2 * ks + j][0] * pw0.up, X[2 * ks + j][1] * pw0.up, hi[ks][2 * j], lo[ks][2 * j]);
                    split_h(X[2 * ks + j][2] * pw1.up, X[2 * ks + j][3] * pw1.up, hi[ks][2 * j + 1], lo[ks][2 * j + 1]);
                }
            // S^T = gamma S^T + (U diag(cu))^T K
            auto keys_t = [&](uint32_t (&r)[4], uint32_t (&w)[4], int step) {
                const int ks = step % 4, nt = 4 * (step / 4);
                if constexpr (FIRST) {
                    right_nk<P>(r, tk, ks, nt, lane);
                    right_nk<P>(w, tk, ks, nt + 2, lane);
                } else {
                    right_kn<P>(r, tk, ks, nt, lane);
                    right_kn<P>(w, tk, ks, nt + 2, lane);
                }
            };
            {
                uint32_t r[2][4], w[2][4];
                keys_t(r[0], w[0], 0);
                float D[4][4];
#pragma unroll
                for (int step = 0; step < DK / 8; ++step) {
                    const int ks = step % 4, nt = 4 * (step / 4), at = step & 1;
                    if (step + 1 < DK / 8) keys_t(r[at ^ 1], w[at ^ 1], step + 1);
                    if (ks == 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) D[i][j] = 0.0f;
                    }
                    mma_f16(D[0], hi[ks], r[at][0], r[at][1]);
                    mma_f16(D[1], hi[ks], r[at][2], r[at][3]);
                    mma_f16(D[2], hi[ks], w[at][0], w[at][1]);
                    mma_f16(D[3], hi[ks], w[at][2], w[at][3]);
                    mma_f16(D[0], lo[ks], r[at][0], r[at][1]);
                    mma_f16(D[1], lo[ks], r[at][2], r[at][3]);
                    mma_f16(D[2], lo[ks], w[at][0], w[at][1]);
                    mma_f16(D[3], lo[ks], w[at][2], w[at][3]);
                    if (ks == 3) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            S[nt + i][0] = fmaf(gamma, S[nt + i][0], D[i][0] * pw0.down);
                            S[nt + i][1] = fmaf(gamma, S[nt + i][1], D[i][1] * pw0.down);
                            S[nt + i][2] = fmaf(gamma, S[nt + i][2], D[i][2] * pw1.down);
                            S[nt + i][3] = fmaf(gamma, S[nt + i][3], D[i][3] * pw1.down);
                        }
                    }
                }
            }
            // O^T += U^T P^T
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) X[i][j] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t u[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    u[2 * j] = pack_h(U[2 * ks + j][0] * pu0.up, U[2 * ks + j][1] * pu0.up);
                    u[2 * j + 1] = pack_h(U[2 * ks + j][2] * pu1.up, U[2 * ks + j][3] * pu1.up);
                }
#pragma unroll
                for (int nt = 2 * ks; nt < 8; nt += 2) {
                    uint32_t r[4];
                    right_nk<8>(r, tb + 2 * kTile, ks, nt, lane);
                    mma_f16(X[nt], u, r[0], r[1]);
                    mma_f16(X[nt + 1], u, r[2], r[3]);
                }
            }
            // out through shared memory: whole rows leave
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const int t = 8 * nt + 2 * t4;
                const float2 cp = *reinterpret_cast<const float2*>(&f.cp[t]);
                const __nv_bfloat162 y0 = __floats2bfloat162_rn(fmaf(X[nt][0] * pu0.down, cp.x, O[nt][0]), fmaf(X[nt][1] * pu0.down, cp.y, O[nt][1]));
                const __nv_bfloat162 y1 = __floats2bfloat162_rn(fmaf(X[nt][2] * pu1.down, cp.x, O[nt][2]), fmaf(X[nt][3] * pu1.down, cp.y, O[nt][3]));
                if constexpr (FIRST) {
                    *reinterpret_cast<__nv_bfloat162*>(so + g * kVRow + t) = y0;
                    *reinterpret_cast<__nv_bfloat162*>(so + (g + 8) * kVRow + t) = y1;
                } else {
                    so[t * kORow + g] = y0.x;
                    so[(t + 1) * kORow + g] = y0.y;
                    so[t * kORow + g + 8] = y1.x;
                    so[(t + 1) * kORow + g + 8] = y1.y;
                }
            }
        }
        __syncwarp();
        if (lane == 0 && ch != x.hold) tc::mbar_arrive(&sm.empty[s]);
        const int cols = min(16, a.dv - dw);
        bf16* oc = ob + t0 * a.os.st;
        if (x.vec_o && n == C && cols == 16) {
            // whole rows of 16 bytes, all in flight
            uint4 w[4];
            if constexpr (FIRST) {
                const int r = lane >> 3, t = (lane & 7) * 8;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4*>(so + (r + 4 * j) * kVRow + t);
                bf16* to = oc + int64_t(r) * a.os.sc + t;
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(to + 4 * j * a.os.sc) = w[j];
            } else {
                const int t = lane >> 1, c = (lane & 1) * 8;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4*>(so + (t + 16 * j) * kORow + c);
                bf16* to = oc + int64_t(t) * a.os.st + c;
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(to + 16 * j * a.os.st) = w[j];
            }
        } else if constexpr (FIRST) {
#pragma unroll 1
            for (int i = lane; i < 16 * 8; i += 32) {
                const int r = i >> 3, t = (i & 7) * 8;
                if (r >= cols) continue;
                if (x.vec_o && t + 8 <= n) {
                    *reinterpret_cast<uint4*>(oc + int64_t(r) * a.os.sc + t) = *reinterpret_cast<const uint4*>(so + r * kVRow + t);
                } else {
                    for (int j = 0; j < 8 && t + j < n; ++j) oc[int64_t(r) * a.os.sc + int64_t(t + j) * a.os.st] = so[r * kVRow + t + j];
                }
            }
        } else {
#pragma unroll 1
            for (int i = lane; i < C * 2; i += 32) {
                const int t = i >> 1, c = (i & 1) * 8;
                if (t >= n) continue;
                if (x.vec_o && c + 8 <= cols) {
                    *reinterpret_cast<uint4*>(oc + int64_t(t) * a.os.st + c) = *reinterpret_cast<const uint4*>(so + t * kORow + c);
                } else {
                    for (int j = 0; j < 8 && c + j < cols; ++j) oc[int64_t(t) * a.os.st + int64_t(c + j) * a.os.sc] = so[t * kORow + c + j];
                }
            }
        }
        __syncwarp();
    }
    if (ch < chunks) {                             // gave up waiting
        if (lane == 0) report_status(x.status, kStatusTimeout);
#pragma unroll
        for (int j = 0; j < DK / 8; ++j) S[j][0] = S[j][1] = S[j][2] = S[j][3] = __int_as_float(0x7fffffff);
        give_up(sm.full, ch, x.budget_ns, ob, a.os.sc, a.os.st, min(16, a.dv - dw), len);
    }
    if (a.state_out) {
#pragma unroll
        for (int j = 0; j < DK / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = dw + g + 8 * (i >> 1), r = 8 * j + 2 * t4 + (i & 1);
                if (d < a.dv && r < a.dk) a.state_out[sb + int64_t(r) * a.dv + d] = S[j][i];
            }
    }
}

// --------------------------------------------------------------- narrow scan
// For few heads: a warp takes 8 value channels instead of 16, so the same heads
// make twice the warps and a warp's chain is half as long (1600 cycles of
// products a chunk).  Time and key channels are the 16 rows of the products,
// value channels the 8 columns: S [DK x 8] in accumulators,
//   X = K S,  R = V - diag(cx) X,  U = T R,  S = gamma S + K^T (diag(cu) U),  O = diag(co) Q S + P U,
// and a result becomes the next one's right operand by transposing its 8 x 8
// blocks in registers.  Every warp reads all of K, Q, T and P as left operands,
// so shared memory would bound more than four warps an SM.  A chunk takes 5500
// cycles, the warp's and its scheduler's loading warp's issue slots two thirds
// of them: 24 heads of 128 chunks 376 us (500 us with 16 channels a warp).  One
// CTA an SM: 255 registers (dk = 64: 221) and half of the shared memory.
constexpr int kNarrowWarps = 4, kNarrowCols = 8 * kNarrowWarps;
constexpr int kNarrowVRow = kNarrowCols + 8;       // elements of a token's row of V: eight rows on 32 banks

template <int DK>
struct NarrowSmem {
    using Stage = ScanStage<DK, C, kNarrowVRow>;
    Stage st[2];
    alignas(16) bf16 o[kNarrowWarps][8 * kVRow];   // [channel][kVRow], or [time][8]
    uint64_t full[2], empty[2];
};

// An 8 x 8 block of 16-bit numbers transposed across a warp's registers.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
    return r;
}
// Two numbers of a 16 x 8 accumulator tile's rows as high and low right operands.
struct Right {
    uint32_t hi[2], lo[2];
    __device__ __forceinline__ Right(const float (&c)[4], float up0, float up1) {
        uint32_t h0, l0, h1, l1;
        split_h(c[0] * up0, c[1] * up1, h0, l0);
        split_h(c[2] * up0, c[3] * up1, h1, l1);
        hi[0] = transposed(h0);
        hi[1] = transposed(h1);
        lo[0] = transposed(l0);
        lo[1] = transposed(l1);
    }
};
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

// V [64][kNarrowCols]: as it lies token by token; from channels' rows pairs of channels, eight tokens each way.
template <bool FIRST>
__device__ __forceinline__ void load_values_narrow(bf16 (&v)[C][kNarrowVRow], const bf16* p, const DeltaView& s, int cols, int n,
                                                   bool vec, int lt) {
    if constexpr (!FIRST) {
        constexpr int kRowOct = kNarrowCols / 8, kOct = C * kRowOct / kLoaders;
        if (whole<false>(cols, n, vec)) {
#pragma unroll
            for (int j = 0; j < kOct; ++j) {
                const int i = lt + j * kLoaders;
                copy_octet<false>(&v[i / kRowOct][8 * (i % kRowOct)], p, s, 8 * (i % kRowOct), i / kRowOct, cols, n);
            }
        } else {
#pragma unroll 2
            for (int i = lt; i < C * kRowOct; i += kLoaders)
                *reinterpret_cast<uint4*>(&v[i / kRowOct][8 * (i % kRowOct)]) =
                    octet<false>(p, s, 8 * (i % kRowOct), i / kRowOct, cols, n);
        }
    } else {
        static_assert(kNarrowCols / 2 * 8 == kLoaders, "a pair of octets a thread");
        const int cp = lt / 8, t = 8 * (lt % 8);
        const bool all = whole<true>(cols, n, vec);
        const uint4 w0 = all ? whole_octet<true>(p, s, 2 * cp, t, cols, n) : octet<true>(p, s, 2 * cp, t, cols, n);
        const uint4 w1 = all ? whole_octet<true>(p, s, 2 * cp + 1, t, cols, n) : octet<true>(p, s, 2 * cp + 1, t, cols, n);
        const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint32_t*>(&v[t + j][2 * cp]) = __byte_perm(u0[j >> 1], u1[j >> 1], (j & 1) ? 0x7632 : 0x5410);
    }
}

template <int DK, bool FIRST>
__global__ void __launch_bounds__(32 * kNarrowWarps + kLoaders, 1) k_delta_scan_narrow(ChunkArgs x) {
    using Sm = NarrowSmem<DK>;
    constexpr int P = FIRST ? 8 : DK / 8, kTiles = DK / 16;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    const DeltaArgs& a = x.a;
    const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int h = int(blockIdx.y), d0 = int(blockIdx.x) * kNarrowCols;
    const int64_t b = blockIdx.z;
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&sm.full[s], kLoaders + 1);
            tc::mbar_init(&sm.empty[s], kNarrowWarps);
        }
    }
    __syncthreads();
    after_prep();
    const int len = int(length_of(a, b)), chunks = (len + C - 1) / C;      // L <= 2^30
    if (warp >= kNarrowWarps) {
        const int lt = tid - 32 * kNarrowWarps, cols = min(kNarrowCols, a.dv - d0);
        run_loaders<DK, FIRST>(sm, x, lt, lane, h, b, len, d0, [&](typename Sm::Stage& st, const bf16* p, int n) {
            load_values_narrow<FIRST>(st.v, p, a.vs, cols, n, x.vec_v, lt);
        });
        return;
    }
    const int g = lane >> 2, t4 = lane & 3;
    const int dw = d0 + 8 * warp;                  // this warp's first channel
    const int64_t sb = (b * a.Hv + h) * int64_t(a.dk) * a.dv;
    float S[kTiles][4];
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * j + g + 8 * (i >> 1), d = dw + 2 * t4 + (i & 1);
            S[j][i] = (a.state_in && d < a.dv && r < a.dk) ? a.state_in[sb + int64_t(r) * a.dv + d] : 0.0f;
        }
    bf16* ob = static_cast<bf16*>(a.o) + b * a.os.sb + (int64_t(h) * a.dv + dw) * a.os.sc;
    bf16* so = sm.o[warp];
    int ch = 0;
    for (; ch < chunks; ++ch) {
        const int s = ch & 1;
        typename Sm::Stage& st = sm.st[s];
        if (!tc::mbar_wait(&sm.full[s], uint32_t(ch >> 1) & 1u, x.budget_ns)) break;
        const int64_t t0 = int64_t(ch) * C;
        const int n = min(C, len - ch * C);
        const uint32_t tk = tc::smem_u32(st.k), tq = tc::smem_u32(st.q), tb = tc::smem_u32(st.blob);
        const Factors& f = *reinterpret_cast<const Factors*>(st.blob + 3 * kTile);
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            m0 = fmaxf(m0, fmaxf(fabsf(S[j][0]), fabsf(S[j][2])));
            m1 = fmaxf(m1, fmaxf(fabsf(S[j][1]), fabsf(S[j][3])));
        }
        const float s0 = column_max(m0), s1 = column_max(m1);
        const Pow2 ps0(s0), ps1(s1);
        float X[4][4], O[4][4], U[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) X[i][j] = O[i][j] = U[i][j] = 0.0f;
        // X = K S, O = Q S: left operands a step (three products) ahead
        auto rows = [&](uint32_t (&r)[4], uint32_t (&w)[4], int step) {
            if constexpr (FIRST) {
                left_km<P>(r, tk, step % 4, step / 4, lane);
                left_km<P>(w, tq, step % 4, step / 4, lane);
            } else {
                left_mk<P>(r, tk, step % 4, step / 4, lane);
                left_mk<P>(w, tq, step % 4, step / 4, lane);
            }
        };
        {
            uint32_t r[2][4], w[2][4];
            rows(r[0], w[0], 0);
            Right y(S[0], ps0.up, ps1.up);
#pragma unroll
            for (int ks = 0; ks < kTiles; ++ks) {
                // the next right operand is made under this one's products
                const Right next(S[ks + 1 < kTiles ? ks + 1 : ks], ps0.up, ps1.up);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const int step = 4 * ks + mt, at = step & 1;
                    if (step + 1 < 4 * kTiles) rows(r[at ^ 1], w[at ^ 1], step + 1);
                    mma_f16(X[mt], r[at], y.hi[0], y.hi[1]);
                    mma_f16(O[mt], w[at], y.hi[0], y.hi[1]);
                    mma_f16(X[mt], r[at], y.lo[0], y.lo[1]);
                }
                y = next;
            }
        }
        m0 = m1 = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const int t = 16 * mt + g;
            const float cx0 = f.cx[t], cx1 = f.cx[t + 8], co0 = f.co[t], co1 = f.co[t + 8];
            const uint32_t v0 = *reinterpret_cast<const uint32_t*>(&st.v[t][8 * warp + 2 * t4]);
            const uint32_t v1 = *reinterpret_cast<const uint32_t*>(&st.v[t + 8][8 * warp + 2 * t4]);
            X[mt][0] = fmaf(-X[mt][0] * ps0.down, cx0, bf(v0, 0));
            X[mt][1] = fmaf(-X[mt][1] * ps1.down, cx0, bf(v0, 1));
            X[mt][2] = fmaf(-X[mt][2] * ps0.down, cx1, bf(v1, 0));
            X[mt][3] = fmaf(-X[mt][3] * ps1.down, cx1, bf(v1, 1));
            m0 = fmaxf(m0, fmaxf(fabsf(X[mt][0]), fabsf(X[mt][2])));
            m1 = fmaxf(m1, fmaxf(fabsf(X[mt][1]), fabsf(X[mt][3])));
            O[mt][0] = O[mt][0] * ps0.down * co0;
            O[mt][1] = O[mt][1] * ps1.down * co0;
            O[mt][2] = O[mt][2] * ps0.down * co1;
            O[mt][3] = O[mt][3] * ps1.down * co1;
        }
        const float r0 = column_max(m0), r1 = column_max(m1);
        const Pow2 pr0(r0), pr1(r1);
        // U = T R, blocks on and under the diagonal (block 0 .. 9: column ks, rows ks .. 3)
        {
            const Right y[4] = {{X[0], pr0.up, pr1.up}, {X[1], pr0.up, pr1.up}, {X[2], pr0.up, pr1.up}, {X[3], pr0.up, pr1.up}};
            constexpr int kCol[11] = {0, 0, 0, 0, 1, 1, 1, 2, 2, 3, 3}, kRow[11] = {0, 1, 2, 3, 1, 2, 3, 2, 3, 3, 3};
            uint32_t r[2][4], w[2][4];
            left_mk<8>(r[0], tb, 0, 0, lane);
            left_mk<8>(w[0], tb + kTile, 0, 0, lane);
#pragma unroll
            for (int i = 0; i < 10; ++i) {
                const int at = i & 1, ks = kCol[i], mt = kRow[i];
                if (i < 9) {
                    left_mk<8>(r[at ^ 1], tb, kRow[i + 1], kCol[i + 1], lane);
                    left_mk<8>(w[at ^ 1], tb + kTile, kRow[i + 1], kCol[i + 1], lane);
                }
                mma_f16(U[mt], r[at], y[ks].hi[0], y[ks].hi[1]);
                mma_f16(U[mt], r[at], y[ks].lo[0], y[ks].lo[1]);
                mma_f16(U[mt], w[at], y[ks].hi[0], y[ks].hi[1]);
            }
        }
        m0 = m1 = 0.0f;
        float z0 = INFINITY, z1 = z0;              // the smallest write
        float n0 = 0.0f, n1 = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const int t = 16 * mt + g;
            const float ct0 = f.ct[t], ct1 = f.ct[t + 8], cu0 = f.cu[t], cu1 = f.cu[t + 8];
            U[mt][0] = U[mt][0] * pr0.down * ct0;
            U[mt][1] = U[mt][1] * pr1.down * ct0;
            U[mt][2] = U[mt][2] * pr0.down * ct1;
            U[mt][3] = U[mt][3] * pr1.down * ct1;
            m0 = fmaxf(m0, fmaxf(fabsf(U[mt][0]), fabsf(U[mt][2])));
            m1 = fmaxf(m1, fmaxf(fabsf(U[mt][1]), fabsf(U[mt][3])));
            z0 = fminf(z0, fminf(fabsf(U[mt][0]), fabsf(U[mt][2])));
            z1 = fminf(z1, fminf(fabsf(U[mt][1]), fabsf(U[mt][3])));
            X[mt][0] = U[mt][0] * cu0;
            X[mt][1] = U[mt][1] * cu0;
            X[mt][2] = U[mt][2] * cu1;
            X[mt][3] = U[mt][3] * cu1;
            n0 = fmaxf(n0, fmaxf(fabsf(X[mt][0]), fabsf(X[mt][2])));
            n1 = fmaxf(n1, fmaxf(fabsf(X[mt][1]), fabsf(X[mt][3])));
        }
        const float u0 = column_max(m0), u1 = column_max(m1), w0 = column_max(n0), w1 = column_max(n1), gamma = f.gamma;
        const Reach reach = f.reach;
        const float a0 = fmaxf(u0, r0 * reach.t), a1 = fmaxf(u1, r1 * reach.t);
        const bool end = reach.end(a0, r0, w0, s0, gamma) || reach.end(a1, r1, w1, s1, gamma);
        bool apart = __any_sync(0xffffffffu, end || z0 < a0 * 0x1p-28f || z1 < a1 * 0x1p-28f);
        if (__builtin_expect(apart, 0) && !__any_sync(0xffffffffu, end))       // or tokens that write nothing, or chance?
            apart = small_writes<false>(U, f, lane, a0, a1) &&
                    look_again<false>(U, Writes{&f, &st.v[0][8 * warp + 2 * t4], 1, kNarrowVRow, {a0, a1}, {s0, s1}});
        if (__builtin_expect(apart, 0)) {
            state_by_token<DK, FIRST, false>(S, st.k, st.q, f, a, b, h, t0, n, &st.v[0][8 * warp + 2 * t4], 1, kNarrowVRow,
                                             so + 2 * t4 * (FIRST ? kVRow : 1), FIRST ? kVRow : 1, FIRST ? 1 : 8);
        } else {
            const Pow2 pu0(u0), pu1(u1), pw0(w0), pw1(w1);
            const Right yw[4] = {{X[0], pw0.up, pw1.up}, {X[1], pw0.up, pw1.up}, {X[2], pw0.up, pw1.up}, {X[3], pw0.up, pw1.up}};
            // S = gamma S + K^T (diag(cu) U), two tiles of key channels at a time
            {
                auto keys_t = [&](uint32_t (&r)[4], uint32_t (&w)[4], int step) {
                    const int i = 2 * (step / 4), ks = step % 4;
                    if constexpr (FIRST) {
                        left_mk<P>(r, tk, i, ks, lane);
                        left_mk<P>(w, tk, i + 1, ks, lane);
                    } else {
                        left_km<P>(r, tk, i, ks, lane);
                        left_km<P>(w, tk, i + 1, ks, lane);
                    }
                };
                uint32_t r[2][4], w[2][4];
                keys_t(r[0], w[0], 0);
                float D[4][4];
#pragma unroll
                for (int step = 0; step < 2 * kTiles; ++step) {
                    const int i = 2 * (step / 4), ks = step % 4, at = step & 1;
                    if (step + 1 < 2 * kTiles) keys_t(r[at ^ 1], w[at ^ 1], step + 1);
                    if (ks == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) D[0][j] = D[1][j] = D[2][j] = D[3][j] = 0.0f;
                    }
                    mma_f16(D[0], r[at], yw[ks].hi[0], yw[ks].hi[1]);
                    mma_f16(D[1], w[at], yw[ks].hi[0], yw[ks].hi[1]);
                    mma_f16(D[2], r[at], yw[ks].lo[0], yw[ks].lo[1]);
                    mma_f16(D[3], w[at], yw[ks].lo[0], yw[ks].lo[1]);
                    if (ks == 3) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float down = (j & 1) ? pw1.down : pw0.down;
                            S[i][j] = fmaf(gamma, S[i][j], (D[0][j] + D[2][j]) * down);
                            S[i + 1][j] = fmaf(gamma, S[i + 1][j], (D[1][j] + D[3][j]) * down);
                        }
                    }
                }
            }
            // O += P U
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) X[i][j] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const uint32_t u0 = transposed(pack_h(U[ks][0] * pu0.up, U[ks][1] * pu1.up));
                const uint32_t u1 = transposed(pack_h(U[ks][2] * pu0.up, U[ks][3] * pu1.up));
#pragma unroll
                for (int mt = ks; mt < 4; ++mt) {
                    uint32_t r[4];
                    left_mk<8>(r, tb + 2 * kTile, mt, ks, lane);
                    mma_f16(X[mt], r, u0, u1);
                }
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const int t = 16 * mt + g;
                const float cp0 = f.cp[t], cp1 = f.cp[t + 8];
                const uint32_t y0 = tc::pack2(fmaf(X[mt][0] * pu0.down, cp0, O[mt][0]), fmaf(X[mt][1] * pu1.down, cp0, O[mt][1]));
                const uint32_t y1 = tc::pack2(fmaf(X[mt][2] * pu0.down, cp1, O[mt][2]), fmaf(X[mt][3] * pu1.down, cp1, O[mt][3]));
                if constexpr (FIRST) {
                    // rows are channels: the blocks transposed
                    *reinterpret_cast<uint32_t*>(so + g * kVRow + 16 * mt + 2 * t4) = transposed(y0);
                    *reinterpret_cast<uint32_t*>(so + g * kVRow + 16 * mt + 8 + 2 * t4) = transposed(y1);
                } else {
                    *reinterpret_cast<uint32_t*>(so + t * 8 + 2 * t4) = y0;
                    *reinterpret_cast<uint32_t*>(so + (t + 8) * 8 + 2 * t4) = y1;
                }
            }
        }
        __syncwarp();
        if (lane == 0 && ch != x.hold) tc::mbar_arrive(&sm.empty[s]);
        const int cols = min(8, a.dv - dw);
        bf16* oc = ob + t0 * a.os.st;
        if (x.vec_o && n == C && cols == 8) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = lane + 32 * j;
                if constexpr (FIRST)
                    *reinterpret_cast<uint4*>(oc + int64_t(i >> 3) * a.os.sc + (i & 7) * 8) =
                        *reinterpret_cast<const uint4*>(so + (i >> 3) * kVRow + (i & 7) * 8);
                else
                    *reinterpret_cast<uint4*>(oc + int64_t(i) * a.os.st) = *reinterpret_cast<const uint4*>(so + i * 8);
            }
        } else {
#pragma unroll 1
            for (int i = lane; i < 8 * C; i += 32) {
                // the output's contiguous axis over neighbouring lanes
                const int c = FIRST ? i / C : i % 8, t = FIRST ? i % C : i / 8;
                if (c < cols && t < n) oc[int64_t(c) * a.os.sc + int64_t(t) * a.os.st] = FIRST ? so[c * kVRow + t] : so[t * 8 + c];
            }
        }
        __syncwarp();
    }
    if (ch < chunks) {                             // gave up waiting
        if (lane == 0) report_status(x.status, kStatusTimeout);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) S[j][0] = S[j][1] = S[j][2] = S[j][3] = __int_as_float(0x7fffffff);
        give_up(sm.full, ch, x.budget_ns, ob, a.os.sc, a.os.st, min(8, a.dv - dw), len);
    }
    if (a.state_out) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * j + g + 8 * (i >> 1), d = dw + 2 * t4 + (i & 1);
                if (d < a.dv && r < a.dk) a.state_out[sb + int64_t(r) * a.dv + d] = S[j][i];
            }
    }
}

// --------------------------------------------------------------------- host
// Eight elements along the contiguous axis as one 16-byte access, wherever a row starts.
bool vec_ok(const void* p, const DeltaView& s, bool first, int head_channels) {
    const int64_t row = first ? s.sc : s.st;
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (first ? s.st : s.sc) == 1 && row % 8 == 0 && s.sb % 8 == 0 &&
           (first || head_channels % 8 == 0);
}

template <int DK, bool FIRST, bool GROUP>
cudaError_t launch_prep(const ChunkArgs& x, cudaStream_t s) {
    const size_t bytes = sizeof(PrepSmem<DK, FIRST>);
    static std::atomic<bool> raised[kMaxDevices];
    cudaError_t e = raise_smem(k_delta_prep<DK, FIRST, GROUP>, bytes, x.dev, raised);
    if (e != cudaSuccess) return e;
    k_delta_prep<DK, FIRST, GROUP><<<dim3(unsigned(x.chunks), unsigned(x.a.Hv / x.group), unsigned(x.a.B)), kPrepThreads, bytes, s>>>(x);
    return cudaGetLastError();
}

template <typename Kernel>
cudaError_t launch_after_prep(Kernel kernel, dim3 grid, int threads, size_t bytes, const ChunkArgs& x, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, x);
}

template <int DK, int NW, bool FIRST>
cudaError_t launch_scan(const ChunkArgs& x, cudaStream_t s) {
    const size_t bytes = sizeof(ScanSmem<DK, NW>);
    static std::atomic<bool> raised[kMaxDevices];
    cudaError_t e = raise_smem(k_delta_scan<DK, NW, FIRST>, bytes, x.dev, raised);
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned((x.a.dv + 16 * NW - 1) / (16 * NW)), unsigned(x.a.Hv), unsigned(x.a.B));
    return launch_after_prep(k_delta_scan<DK, NW, FIRST>, grid, 32 * NW + kLoaders, bytes, x, s);
}

template <int DK, bool FIRST>
cudaError_t launch_narrow(const ChunkArgs& x, cudaStream_t s) {
    const size_t bytes = sizeof(NarrowSmem<DK>);
    static std::atomic<bool> raised[kMaxDevices];
    cudaError_t e = raise_smem(k_delta_scan_narrow<DK, FIRST>, bytes, x.dev, raised);
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned((x.a.dv + kNarrowCols - 1) / kNarrowCols), unsigned(x.a.Hv), unsigned(x.a.B));
    return launch_after_prep(k_delta_scan_narrow<DK, FIRST>, grid, 32 * kNarrowWarps + kLoaders, bytes, x, s);
}

template <int DK, bool FIRST>
cudaError_t launch_both(const ChunkArgs& x, cudaStream_t s) {
    cudaError_t e = x.group > 1 ? launch_prep<DK, FIRST, true>(x, s) : launch_prep<DK, FIRST, false>(x, s);
    if (e != cudaSuccess) return e;
    // A chunk takes a CTA of 32, 64 or 128 channels about 5500, 7500 or 11900 cycles (dk = 128): the form whose waves of
    // CTAs take least.  dk = 64 takes less, but in nearly the same proportion.  Measured at L = 1024, token by token rows, us
    // of a call by width:
    //   heads            32            72            144            256            512
    //   dk = dv = 128    65  92 135   128 117 150   244 217 179    418 394 332    822 725 646
    //   64, dv = 128     51  68 100    97  81 112   186 156 138    315 276 254    619 515 497
    //   dk = dv = 64     50  66  99    62  80 111   121 104 137    219 183 252    395 352 494
    const int64_t heads = x.a.B * x.a.Hv;
    auto cycles = [&](int width, int64_t each) {
        const int64_t ctas = heads * ((x.a.dv + width - 1) / width);
        return (ctas + x.sms - 1) / x.sms * each;
    };
    const int64_t narrow = cycles(32, 5500), half = cycles(64, 7500), full = cycles(128, 11900);
    if (narrow <= half && narrow <= full) return launch_narrow<DK, FIRST>(x, s);
    return half <= full ? launch_scan<DK, 4, FIRST>(x, s) : launch_scan<DK, 8, FIRST>(x, s);
}

}  // namespace

size_t delta_chunk_workspace(int64_t B, int64_t L, int Hv) { return size_t(B) * size_t(Hv) * size_t((L + C - 1) / C) * kBlob; }

cudaError_t launch_delta_chunk(const DeltaArgs& a, void* workspace, uint32_t* status, uint64_t budget_ns, int64_t hold,
                               cudaStream_t s) {
    ChunkArgs x{};
    x.a = a;
    x.blobs = static_cast<uint8_t*>(workspace);
    x.chunks = int((a.L + C - 1) / C);
    x.budget_ns = budget_ns;
    x.hold = hold >= 0 && hold < x.chunks ? int(hold) : -1;
    x.status = status;
    cudaError_t e = device_sms(&x.dev, &x.sms);
    if (e != cudaSuccess) return e;
    // the tiles lie as the keys do: along time where that is their contiguous axis
    const bool first = a.ks.st == 1 || a.ks.sc != 1;
    // Value heads of one key head share its products, once that leaves every SM its five CTAs.  Calls with and without, us:
    // 16 x 4096, 8 key heads of 2: 1203, 1230 (dk = 64: 676, 682); 16 x 2048, 4 of 4: 603, 628 (337, 349); 8 x 2048, 4 of 2,
    // just above the border: 207, 204 (114, 109).  Fewer chunks are sooner done one by one (2 x 1024, 4 of 2: 66, 60).
    const int r = a.Hv / a.Hk;
    x.group = 1;
    for (int n = 2; n <= kGroup; ++n)
        if (r % n == 0 && int64_t(x.chunks) * a.B * (a.Hv / n) >= 5 * int64_t(x.sms)) x.group = n;
    x.vec_k = vec_ok(a.k, a.ks, first, a.dk);
    x.vec_q = vec_ok(a.q, a.qs, first, a.dk);
    x.vec_v = vec_ok(a.v, a.vs, first, a.dv);
    x.vec_o = vec_ok(a.o, a.os, first, a.dv);
    if (a.dk <= 64) return first ? launch_both<64, true>(x, s) : launch_both<64, false>(x, s);
    return first ? launch_both<128, true>(x, s) : launch_both<128, false>(x, s);
}

}  // namespace hyena
