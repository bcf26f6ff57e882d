// proj_fp8.cu -- projections on e4m3 operands with a scale for each block of
// 128 channels (activations: a row and block; weights: 128 x 128).
//
//   out[m][n] = sum_kb xs[kb][m] Ws[n / 128][kb] P_kb[m][n] + bias[n],
//   P_kb[m][n] = sum_{k in block kb} xq[m][k] Wq[n][k],      m = b L + l
//
// The scales are arbitrary fp32 numbers, so the tensor cores form one block's
// P in fp32 and the CUDA cores add it, scaled, to fp32 sums in registers.
//
// k_proj_fp8 (more than kFewTokens rows): persistent, one CTA per SM, tiles of
// 128 rows x BN outputs, 384 threads in three roles:
//   warp 0     TMA: x and W blocks (128 x 128 and BN x 128 bytes, 128-byte
//              swizzle) into a ring of stages;
//   warp 1     tcgen05.mma kind::f8f6f4 (M 128, N BN, K 32; four a block) into
//              one of two tensor-memory buffers, a commit per block;
//   warps 4-11 two warpgroups, half of the columns each (their sums take most of
//              the registers, which the first warpgroup hands over): read a
//              block's P with tcgen05.ld, free the buffer, add it times the row's factor.  A
//              thread holds one row, so the factor is one number a block.
// At BN = 256 a block is 512 cycles of tensor work and 256 of multiply-adds a
// scheduler, which overlap; the ring and the two buffers let the next tile's
// products run under this tile's epilogue.
//
// k_proj_fp8_few (up to kFewTokens rows): the weights' bytes bound it.  A CTA
// takes 16 outputs; its 8 warps take the blocks of K in turn, W as the 16-row
// operand of mma.sync m16n8k32, tokens as its columns.  The order of k inside a
// block is free, so each thread loads 16 contiguous bytes and the words go to
// the four products as they lie.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>

#include "common.cuh"
#include "hyena.h"
#include "kernels.h"
#include "tc_util.cuh"
#include "tma_util.cuh"

namespace hyena {

hyena_status_t set_last_error_detail(hyena_status_t st, const std::string& detail);  // api.cu

namespace {

using bf16 = __nv_bfloat16;

constexpr int BM = 128, BKB = 128;                // rows of a tile, bytes of a block
constexpr int kThreads = 384;
constexpr uint32_t kATile = BM * BKB;
constexpr int kRing = 8, kAhead = 7;               // rows' scales in flight

struct Params {
    int64_t M, L, N, K;
    int kblocks;
    int tiles_m, tiles_n;                         // their product below 2^31
    const float* xs;                              // [B][kblocks][L]
    const float* ws;                              // [N / 128][kblocks]
    const float* bias;                            // [N] or nullptr
    bf16* out;
    int channels_first;
    uint64_t budget_ns;
    uint32_t* status;
};

// Epilogue staging (channels_first = 0): a warp's 32 rows x 32 columns of bf16, rows 80 bytes apart (five sixteenths
// of the banks: eight rows' 16-byte pieces meet none twice).
constexpr uint32_t kEpiRow = 80, kEpiWarp = 32 * kEpiRow;

template <int BN>
struct Cfg {
    static constexpr int kStages = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
    static constexpr uint32_t kBTile = BN * BKB;
    static constexpr uint32_t kStageBytes = kATile + kBTile;
    static constexpr uint32_t kTmemCols = 2 * BN;
    static constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes + 256 + 2 * BN * 4 + 8 * kEpiWarp + kRing * 256 * 4;
};

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// kind::f8f6f4: fp32 accumulator, A and B e4m3 (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

// acc += v f on pairs (one instruction for two fp32 multiply-adds)
__device__ __forceinline__ void fma2(uint64_t& acc, float v0, float v1, uint64_t f2) {
    uint64_t v2;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v2) : "f"(v0), "f"(v1));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v2), "l"(f2));
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
    return f;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
k_proj_fp8(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, Params p) {
    constexpr int kStages = Cfg<BN>::kStages;
    constexpr uint32_t kStageBytes = Cfg<BN>::kStageBytes;
    constexpr int CW = BN / 2;                    // columns a thread
    extern __shared__ __align__(1024) uint8_t smem_p[];
    uint8_t* stages = smem_p + ((1024u - (tc::smem_u32(smem_p) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(stages + kStages * kStageBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* mma_done = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    float* s_bias = reinterpret_cast<float*>(stages + kStages * kStageBytes + 256);
    uint8_t* epi = reinterpret_cast<uint8_t*>(s_bias + 2 * BN);
    float* s_ring = reinterpret_cast<float*>(epi + 8 * kEpiWarp);

    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), lane = int(threadIdx.x) & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&acc_full[a], 1);
            tc::mbar_init(&acc_empty[a], 8);      // one arrival a reading warp
        }
        tc::mbar_init(mma_done, 1);
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, Cfg<BN>::kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int tiles = p.tiles_m * p.tiles_n;

    // registers: 384 x 168 at launch = 128 x 40 + 256 x 232
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
        // one thread each: stage and buffer counters step, nothing is divided, so that issuing stays under the products
        if (warp == 0 && lane == 0) {
            int s = 0, issued = 0;
            uint32_t phase = 1;                   // of `empty`: the first round finds the stages free
            bool ok = true;
            for (int tile = int(blockIdx.x); tile < tiles && ok; tile += int(gridDim.x)) {
                const int m0 = tile / p.tiles_n * BM, n0 = tile % p.tiles_n * BN;
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!tc::mbar_wait(&empty[s], phase, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = stages + s * kStageBytes;
                    tc::mbar_expect_tx(&full[s], kStageBytes);
                    tc::tma_load_2d(sa, &map_x, kb * BKB, m0, &full[s]);
                    tc::tma_load_2d(sa + kATile, &map_w, kb * BKB, n0, &full[s]);
                    issued = min(issued + 1, kStages);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) report_status(p.status, kStatusTimeout);
            // nothing left in flight: the last load of every stage has landed
            for (; issued > 0; --issued) {
                if (s == 0) {
                    s = kStages;
                    phase ^= 1u;
                }
                --s;
                tc::mbar_wait(&full[s], phase ^ 1u, p.budget_ns);
            }
        } else if (warp == 1 && lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(BM, BN);
            const uint64_t da0 = tc::desc_sw128(tc::smem_u32(stages), 16, 1024), db0 = da0 + (kATile >> 4);
            const int tail = int((p.K - int64_t(p.kblocks - 1) * BKB + 31) / 32);     // products of the last block
            int s = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 1;
            bool ok = true;
            for (int tile = int(blockIdx.x); tile < tiles && ok; tile += int(gridDim.x)) {
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!tc::mbar_wait(&acc_empty[acc], acc_phase, p.budget_ns) ||
                        !tc::mbar_wait(&full[s], phase, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint64_t da = da0 + uint32_t(s) * (kStageBytes >> 4), db = db0 + uint32_t(s) * (kStageBytes >> 4);
                    const uint32_t d = tmem + uint32_t(acc) * BN;
                    // the tail of the last block lies behind K: zeros, and no products for whole steps of them
                    const int steps = kb + 1 < p.kblocks ? 4 : tail;
                    mma_e4m3(d, da, db, idesc, 0u);
                    if (steps > 1) mma_e4m3(d, da + 2, db + 2, idesc, 1u);
                    if (steps > 2) mma_e4m3(d, da + 4, db + 4, idesc, 1u);
                    if (steps > 3) mma_e4m3(d, da + 6, db + 6, idesc, 1u);
                    tc::commit(&acc_full[acc]);
                    tc::commit(&empty[s]);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                    acc ^= 1;
                    acc_phase ^= acc == 0;
                }
            }
            if (!ok) report_status(p.status, kStatusTimeout);
            // nothing left in flight before tensor memory is released
            tc::commit(mma_done);
            if (!tc::mbar_wait(mma_done, 0, p.budget_ns)) report_status(p.status, kStatusTimeout);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
        const int q = warp & 3, half = (warp - 4) >> 2, wt = int(threadIdx.x) & 127;
        const uint32_t t_col = tmem + uint32_t(half * CW) + (uint32_t(32 * q) << 16);
        uint8_t* stage = epi + (warp - 4) * kEpiWarp;
        // The rows' scales come kAhead blocks ahead (a block's products take less than a load under traffic), across
        // tiles, by asynchronous 4-byte copies into a ring of this thread's own slots.
        float* ring = s_ring + (int(threadIdx.x) - 128);
        int pt = int(blockIdx.x), pc = 0;         // the tile and the ring's slot to fetch next
        int pkb = p.kblocks;
        const float* px = nullptr;
        bool plive = false;
        auto fetch = [&]() {
            if (pkb == p.kblocks) {               // enter tile pt
                const uint32_t m = uint32_t(pt / p.tiles_n) * BM + 32 * q + lane;
                plive = pt < tiles && m < p.M;
                const int64_t b = plive ? m / uint32_t(p.L) : 0;
                px = p.xs + b * (p.kblocks - 1) * p.L + (plive ? m : 0);
                pt += int(gridDim.x);
                pkb = 0;
            }
            if (plive) cp_async_small<4>(ring + pc * 256, px);
            cp_async_commit();
            px += p.L;
            ++pkb;
            pc = (pc + 1) % kRing;
        };
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) fetch();
        int buf = 0, slot = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = int(blockIdx.x); tile < tiles && ok; tile += int(gridDim.x), ++it) {
            const int tm = tile / p.tiles_n;
            const int64_t m0 = int64_t(tm) * BM + 32 * q, m = m0 + lane, n0 = int64_t(tile - tm * p.tiles_n) * BN + half * CW;
            const bool live = m < p.M;
            const int64_t b = live ? uint32_t(m) / uint32_t(p.L) : 0, l = live ? m - b * p.L : 0;
            const float* ws = p.ws + (n0 < p.N ? n0 / 128 : 0) * p.kblocks;
            // this half's bias, double buffered: one barrier a tile keeps writers and readers of a buffer apart
            float* bias = s_bias + (it & 1) * BN + half * CW;
            if (wt < CW) bias[wt] = (p.bias && n0 + wt < p.N) ? __ldg(p.bias + n0 + wt) : 0.0f;
            bar_sync(1 + half, 128);
            uint64_t acc[CW / 2];                 // pairs of neighbouring columns
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) acc[i] = 0;
#pragma unroll 1
            for (int kb = 0; kb < p.kblocks; ++kb) {
                asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead - 1) : "memory");
                const float f = live ? ring[slot * 256] * __ldg(ws + kb) : 0.0f;
                slot = (slot + 1) % kRing;
                fetch();
                uint64_t f2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(f2) : "f"(f));
                if (!tc::mbar_wait(&acc_full[buf], phase, p.budget_ns)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                float v[2][16];                   // 16 columns load under the multiply-adds of 16
                tc::tmem_ld16(t_col + uint32_t(buf * BN), v[0]);
#pragma unroll
                for (int c = 0; c < CW / 16; ++c) {
                    tc::tmem_ld_wait();
                    if (c + 1 < CW / 16) {
                        tc::tmem_ld16(t_col + uint32_t(buf * BN + 16 * (c + 1)), v[(c + 1) & 1]);
                    } else {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) fma2(acc[8 * c + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], f2);
                }
                buf ^= 1;
                phase ^= buf == 0;
            }
            if (!ok) {                            // a wait ran out: NaN for this row's outputs
                for (int i = 0; live && i < CW && n0 + i < p.N; ++i)
                    p.out[p.channels_first ? (b * p.N + n0 + i) * p.L + l : m * p.N + n0 + i] = __float2bfloat16_rn(__int_as_float(0x7fffffff));
                break;
            }
            if (p.channels_first) {
                bf16* o = p.out + (b * p.N + n0) * p.L + l;
                // lanes are neighbouring positions: two columns a step, an even lane takes the pair of the first, an
                // odd one that of the second, where pairs are aligned and stay in one batch row (L even)
                if ((p.L & 1) == 0) {
                    o += (lane & 1) ? p.L - 1 : 0;
#pragma unroll
                    for (int i = 0; i < CW; i += 2) {
                        const float2 a = unpair(acc[i / 2]), bb = *reinterpret_cast<const float2*>(bias + i);
                        const float x = a.x + bb.x, y = a.y + bb.y;
                        const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x : y, 1);
                        const uint32_t w = (lane & 1) ? tc::pack2(other, y) : tc::pack2(x, other);
                        if (live && n0 + i + (lane & 1) < p.N) *reinterpret_cast<uint32_t*>(o) = w;
                        o += 2 * p.L;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < CW; i += 2) {
                        const float2 a = unpair(acc[i / 2]), bb = *reinterpret_cast<const float2*>(bias + i);
                        if (live && n0 + i < p.N) o[0] = __float2bfloat16_rn(a.x + bb.x);
                        if (live && n0 + i + 1 < p.N) o[p.L] = __float2bfloat16_rn(a.y + bb.y);
                        o += 2 * p.L;
                    }
                }
            } else {
                // 32 columns of the warp's 32 rows at a time through shared memory: 64 contiguous bytes a row leave
#pragma unroll
                for (int c = 0; c < CW; c += 32) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 a = unpair(acc[c / 2 + 4 * j + i]);
                            const float2 bb = *reinterpret_cast<const float2*>(bias + c + 8 * j + 2 * i);
                            w[i] = tc::pack2(a.x + bb.x, a.y + bb.y);
                        }
                        *reinterpret_cast<uint4*>(stage + lane * kEpiRow + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
                    if ((p.N & 7) == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 8 * j + (lane >> 2), k = lane & 3;
                            const uint4 w = *reinterpret_cast<const uint4*>(stage + r * kEpiRow + 16 * k);
                            const int64_t n = n0 + c + 8 * k;
                            if (m0 + r < p.M && n < p.N) *reinterpret_cast<uint4*>(p.out + (m0 + r) * p.N + n) = w;
                        }
                    } else {
#pragma unroll 4
                        for (int r = 0; r < 32; ++r) {
                            const bf16 w = *reinterpret_cast<const bf16*>(stage + r * kEpiRow + 2 * lane);
                            if (m0 + r < p.M && n0 + c + lane < p.N) p.out[(m0 + r) * p.N + n0 + c + lane] = w;
                        }
                    }
                }
            }
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, Cfg<BN>::kTmemCols);
}

// ------------------------------------------------------------- a few tokens
constexpr int kFewTokens = 32;
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;

__device__ __forceinline__ void mma_m16n8k32_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 tokens.  Thread (g = lane / 4, t = lane % 4) holds of a row's
// block the bytes 16 t .. 16 t + 15 and 64 + the same: word pairs (2 s, 2 s + 1)
// serve product s as its two k quarters, of W and x alike.
template <int NT>
__global__ void __launch_bounds__(kFewThreads)
k_proj_fp8_few(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ wq, Params p) {
    __shared__ float red[kFewWarps][16][8 * NT + 1];
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = int64_t(blockIdx.x) * 16;
    const int M = int(p.M);
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    const uint8_t* w0 = wq + min(n0 + g, p.N - 1) * p.K;          // rows behind N are read again, not used
    const uint8_t* w1 = wq + min(n0 + g + 8, p.N - 1) * p.K;
    const float* ws = p.ws + n0 / 128 * p.kblocks;
#pragma unroll 2
    for (int kb = warp; kb < p.kblocks; kb += kFewWarps) {
        uint4 a[2][2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int64_t k = int64_t(kb) * BKB + 64 * hf + 16 * t;
            const bool in = k < p.K;                               // K is a multiple of 16
            a[0][hf] = in ? __ldg(reinterpret_cast<const uint4*>(w0 + k)) : make_uint4(0, 0, 0, 0);
            a[1][hf] = in ? __ldg(reinterpret_cast<const uint4*>(w1 + k)) : make_uint4(0, 0, 0, 0);
        }
        const float sw = __ldg(ws + kb);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            uint4 bx[2];
            const int tok = 8 * i + g;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int64_t k = int64_t(kb) * BKB + 64 * hf + 16 * t;
                bx[hf] = (tok < M && k < p.K) ? __ldg(reinterpret_cast<const uint4*>(xq + tok * p.K + k)) : make_uint4(0, 0, 0, 0);
            }
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                mma_m16n8k32_e4m3(c, a[0][hf].x, a[1][hf].x, a[0][hf].y, a[1][hf].y, bx[hf].x, bx[hf].y);
                mma_m16n8k32_e4m3(c, a[0][hf].z, a[1][hf].z, a[0][hf].w, a[1][hf].w, bx[hf].z, bx[hf].w);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int m = 8 * i + 2 * t + j;
                const float f = m < M ? sw * __ldg(p.xs + (int64_t(uint32_t(m) / uint32_t(p.L)) * p.kblocks + kb) * p.L + uint32_t(m) % uint32_t(p.L)) : 0.0f;
                acc[i][j] = fmaf(c[j], f, acc[i][j]);
                acc[i][j + 2] = fmaf(c[j + 2], f, acc[i][j + 2]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        red[warp][g][8 * i + 2 * t] = acc[i][0];
        red[warp][g][8 * i + 2 * t + 1] = acc[i][1];
        red[warp][g + 8][8 * i + 2 * t] = acc[i][2];
        red[warp][g + 8][8 * i + 2 * t + 1] = acc[i][3];
    }
    __syncthreads();
    for (int i = int(threadIdx.x); i < 16 * M; i += kFewThreads) {
        // the contiguous axis of the output goes over neighbouring threads
        const int r = p.channels_first ? i / M : i % 16, m = p.channels_first ? i % M : i / 16;
        const int64_t n = n0 + r;
        if (n >= p.N) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) s += red[w][r][m];
        if (p.bias) s += __ldg(p.bias + n);
        const int64_t b = uint32_t(m) / uint32_t(p.L), l = m - b * p.L;
        p.out[p.channels_first ? (b * p.N + n) * p.L + l : int64_t(m) * p.N + n] = __float2bfloat16_rn(s);
    }
}

// --------------------------------------------------------------------- host
hyena_status_t fail(hyena_status_t st, const std::string& why) { return set_last_error_detail(st, why); }

// [rows][K] bytes, box of 128 bytes x box_rows, 128-byte swizzle; what lies outside reads as zero.
bool make_map(CUtensorMap* map, const void* base, uint64_t K, uint64_t rows, uint32_t box_rows, std::string* why) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    cudaError_t e = tensor_map_encoder(&enc);
    if (e != cudaSuccess) {
        *why = std::string("cuTensorMapEncodeTiled unavailable: ") + cudaGetErrorString(e);
        return false;
    }
    const cuuint64_t dims[2] = {K, rows}, strides[1] = {K};
    const cuuint32_t box[2] = {BKB, box_rows}, estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) *why = "cuTensorMapEncodeTiled failed (" + std::to_string(int(r)) + ")";
    return r == CUDA_SUCCESS;
}

int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int BN>
cudaError_t launch(const CUtensorMap& mx, const CUtensorMap& mw, Params& p, int sms, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_proj_fp8<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg<BN>::kSmem));
    if (e != cudaSuccess) return e;
    p.tiles_m = int((p.M + BM - 1) / BM);
    p.tiles_n = int((p.N + BN - 1) / BN);
    const int tiles = p.tiles_m * p.tiles_n;
    k_proj_fp8<BN><<<unsigned(tiles < sms ? tiles : sms), kThreads, Cfg<BN>::kSmem, s>>>(mx, mw, p);
    return cudaGetLastError();
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace hyena

using namespace hyena;

extern "C" hyena_status_t hyena_proj_fp8(const void* xq, const float* xs, const void* Wq, const float* Ws,
                                         const float* bias, void* out, int64_t B, int64_t L, int64_t K, int64_t N,
                                         int channels_first, void* stream) {
    if (!xq || !xs || !Wq || !Ws || !out) return fail(HYENA_ERR_INVALID_ARG, "xq, xs, Wq, Ws and out must not be NULL");
    if (B < 1 || L < 1 || K < 1 || N < 1) return fail(HYENA_ERR_INVALID_ARG, "B, L, K and N must be >= 1");
    if (K % 16 != 0 || K > (int64_t(1) << 20) || N > (int64_t(1) << 20) || B > 65535 || L > (int64_t(1) << 31) - 1 ||
        B * L > (int64_t(1) << 31) - 1 || (B * L + BM - 1) / BM * ((N + 63) / 64) > (int64_t(1) << 31) - 1)
        return fail(HYENA_ERR_UNSUPPORTED_SHAPE,
                    "K must be a multiple of 16, K and N at most 2^20, B <= 65535, B * L < 2^31 and the output of fewer "
                    "than 2^31 tiles");
    if (!aligned(xq, 16) || !aligned(Wq, 16) || !aligned(out, 16))
        return fail(HYENA_ERR_MISALIGNED, "xq, Wq and out must be 16-byte aligned");
    if (!aligned(xs, 4) || !aligned(Ws, 4) || !aligned(bias, 4))
        return fail(HYENA_ERR_MISALIGNED, "xs, Ws and bias must be 4-byte aligned");
    const int64_t M = B * L, kblocks = (K + BKB - 1) / BKB;
    const size_t no = size_t(M) * size_t(N) * 2;
    if (overlaps(out, no, xq, size_t(M) * K) || overlaps(out, no, Wq, size_t(N) * K) ||
        overlaps(out, no, xs, size_t(M) * kblocks * 4) || overlaps(out, no, Ws, size_t((N + 127) / 128) * kblocks * 4) ||
        (bias && overlaps(out, no, bias, size_t(N) * 4)))
        return fail(HYENA_ERR_INVALID_ARG, "out overlaps an input");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Params p{M, L, N, K, int(kblocks), 0, 0, xs, Ws, bias, static_cast<bf16*>(out), channels_first != 0,
             kDefaultWaitBudgetNs, nullptr};
    cudaError_t e;
    if (M <= kFewTokens) {
        const unsigned grid = unsigned((N + 15) / 16);
        const uint8_t *x = static_cast<const uint8_t*>(xq), *w = static_cast<const uint8_t*>(Wq);
        if (M <= 8) k_proj_fp8_few<1><<<grid, kFewThreads, 0, s>>>(x, w, p);
        else if (M <= 16) k_proj_fp8_few<2><<<grid, kFewThreads, 0, s>>>(x, w, p);
        else k_proj_fp8_few<4><<<grid, kFewThreads, 0, s>>>(x, w, p);
        e = cudaGetLastError();
    } else {
        // the widest tile that leaves every SM one; narrower ones spread a small product
        const int sms = sm_count();
        const int64_t tm = (M + BM - 1) / BM;
        const int bn = tm * ((N + 255) / 256) >= sms ? 256 : tm * ((N + 127) / 128) >= sms ? 128 : 64;
        std::string why;
        CUtensorMap mx, mw;
        if (!make_map(&mx, xq, uint64_t(K), uint64_t(M), BM, &why) || !make_map(&mw, Wq, uint64_t(K), uint64_t(N), uint32_t(bn), &why))
            return fail(HYENA_ERR_CUDA, why);
        e = kernel_status_word(&p.status);
        if (e == cudaSuccess)
            e = bn == 256   ? launch<256>(mx, mw, p, sms, s)
                : bn == 128 ? launch<128>(mx, mw, p, sms, s)
                            : launch<64>(mx, mw, p, sms, s);
    }
    if (e != cudaSuccess) return fail(HYENA_ERR_CUDA, std::string("8-bit projection: ") + cudaGetErrorString(e));
    return set_last_error_detail(HYENA_OK, "");
}
