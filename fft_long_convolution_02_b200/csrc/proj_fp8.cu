// proj_fp8.cu -- projections on e4m3 operands with a scale for each block of
// 128 channels (activations: a row and block; weights: 128 x 128).
//
//   out[m][n] = sum_kb xs[kb][m] Ws[n / 128][kb] P_kb[m][n] + bias[n],
//   P_kb[m][n] = sum_{k in block kb} xq[m][k] Wq[n][k],      m = b L + l
//
// The scales are arbitrary fp32 numbers, so the tensor cores form one block's
// P in fp32 and the CUDA cores add it, scaled, to fp32 sums in registers.
//
// k_proj_fp8 (more than kFewTokens rows): persistent, 384 threads a CTA in
// four roles:
//   warp 0      TMA: x and W blocks of 128 bytes a row (128-byte swizzle) into a
//               ring of stages;
//   warp 1      tcgen05.mma kind::f8f6f4 (K 32; four a block) into one of two
//               tensor-memory buffers, a commit per block;
//   warps 2, 3  the rows' factors xs Ws of each block into shared memory, their
//               loads four blocks ahead;
//   warps 4-11  two warpgroups, half of the columns each (their sums take most
//               of the registers, which the first warpgroup hands over): read a
//               block's P with tcgen05.ld (a row a thread), free the buffer, add
//               it times the row's factor.
// Tiles.  Large products run on pairs of CTAs (cta_group::2): 256 x 256, each
// CTA the sums of its 128 rows and half of the W rows in its shared memory, so
// a block brings 32 KB into an SM for its 512 cycles of tensor work; a CTA by
// itself would need 48 KB for 128 x 256, more than L2 gives an SM in that time
// (measured 0.50 us a block against 0.35 us without the loads).  Smaller ones
// run on single CTAs with 128 x 128 or 128 x 64 tiles, which reach more SMs.
// The sums leave through shared memory as TMA stores that run under the next
// tile's first blocks.  What bounds it: two buffers of sums are all that tensor
// memory holds, and a buffer's round trip (512 cycles of products, arrivals
// across the pair, reading, arrivals again) is longer than two blocks' products.
// A call among others, inputs from DRAM: 32768 x 2048 x 4096 345 us, 1.59 PFLOP/s; 32768 x 768 x 2304 100 us, 1.15 (on its
// own, inputs in L2, clocks at their highest: 297 us, 1.85; 85 us, 1.36).
//
// k_proj_fp8_few (up to kFewTokens rows): the weights' bytes bound it.  A CTA
// takes 16 outputs; its 8 warps take the blocks of K in turn, W as the 16-row
// operand of mma.sync m16n8k32, tokens as its columns.  The order of k inside a
// block is free, so each thread loads 16 contiguous bytes and the words go to
// the four products as they lie.  Measured at K = 2048, N = 6144 against the
// 64-wide tiles: 4.6 against 9.2 us at 8 rows, 9.6 against 9.2 us at 16 (at
// K = 768, N = 2304 3.2 against 5.0 us), 18.2 against 9.9 us at 32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <string>


#include "hyena.h"
#include "kernels.h"
#include "tc_util.cuh"
#include "tma_util.cuh"

namespace hyena {

hyena_status_t set_last_error_detail(hyena_status_t st, const std::string& detail);  // api.cu

namespace {

using bf16 = __nv_bfloat16;

constexpr int BM = 128, BKB = 128;                // rows of a CTA's tile, bytes of a block
constexpr int kThreads = 384;
constexpr uint32_t kATile = BM * BKB;

// How a tile leaves: element by element, or as TMA stores of the tensor map `map_o`.
enum Store { STORE_PLAIN = 0, STORE_TMA = 1 };

struct Params {
    int64_t M, L, N, K;
    int kblocks;
    int tiles_m, tiles_n;                         // their product below 2^31
    const float* xs;                              // [B][kblocks][L]
    const float* ws;                              // [N / 128][kblocks]
    const float* bias;                            // [N] or nullptr
    bf16* out;
    int channels_first, store;
    uint64_t budget_ns;
    uint32_t* status;
    int hold;                                     // test hook
};

// What the test hook withholds: nothing, the products, or a warp's word that its part of a tile is staged.
enum Hold { HOLD_NONE = 0, HOLD_PRODUCTS = 1, HOLD_STAGED = 2 };

// BN columns a tile; G CTAs share one (G = 2: 256 rows).
template <int BN, int G>
struct Cfg {
    static constexpr int kStages = BN == 256 ? 4 : (BN == 128 ? 4 : 6);
    static constexpr uint32_t kBTile = BN / G * BKB;
    static constexpr uint32_t kStageBytes = kATile + kBTile;
    static constexpr uint32_t kTmemCols = 2 * BN;
    static constexpr int CW = BN / 2;             // columns a consuming thread
    static constexpr uint32_t kOutWarp = 32 * CW * 2;
    static constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes + 8 * kOutWarp + 512 + 8 * CW * 4 + kStages * 256 * 4;
};

// Neighbouring tiles at work together lie along the output's contiguous axis.
__device__ __forceinline__ void place(const Params& p, int tile, int& tm, int& tn) {
    if (p.channels_first) {
        tn = tile / p.tiles_m;
        tm = tile - tn * p.tiles_m;
    } else {
        tm = tile / p.tiles_n;
        tn = tile - tm * p.tiles_n;
    }
}

template <int G>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (G == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(acc));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// kind::f8f6f4: fp32 accumulator, A and B e4m3 (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

// An arrival at this barrier of every CTA that shares the tile, once the products issued so far are done.
template <int G>
__device__ __forceinline__ void commit(uint64_t* mbar) {
    if constexpr (G == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                tc::smem_u32(mbar)),
            "h"(uint16_t(3))
            : "memory");
    else
        tc::commit(mbar);
}

// A load into this CTA's memory whose bytes count at the first CTA's barrier (the peer bit of the address cleared).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n" ::"r"(tc::smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(tc::smem_u32(mbar) & 0xFEFFFFFFu)
        : "memory");
}

// An arrival at CTA 0's barrier.
__device__ __forceinline__ void arrive_first(uint64_t* mbar) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(remote) : "r"(tc::smem_u32(mbar)));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(remote) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}

template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    if constexpr (G == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(tc::smem_u32(slot)), "r"(cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    } else {
        tc::tmem_alloc(slot, cols);
    }
}
template <int G>
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t cols) {
    if constexpr (G == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(base), "r"(cols));
    else tc::tmem_dealloc(base, cols);
}

// 16 lanes x 32 columns of tensor memory as the fragments of m16n8 products lie: of the 8 columns from 8 j thread
// (g = lane / 4, t = lane % 4) gets row g, columns 2 t, 2 t + 1 in v[4 j], v[4 j + 1] and row g + 8 in the next two.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&r)[16]) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(v[i]);
}

// Four 8 x 8 matrices of 16-bit numbers from fragments, transposed.
__device__ __forceinline__ void stmatrix4_trans(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// 32 lanes x 32 columns, row `lane` from this lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint64_t (&v)[16]) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) asm("mov.b64 {%0, %1}, %2;" : "=r"(r[2 * i]), "=r"(r[2 * i + 1]) : "l"(v[i]));
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(one));
    return one != 0;
}

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
// A reading warp that gave up at `tile`: NaN for its rows and columns of that tile and of the CTA's later ones; `whole_half`
// for the rows of all four warps in the first.
template <int BN, int G>
__device__ __noinline__ void give_up(const Params p, int tile, int tiles, int step, int rank, int q, int half, bool whole_half) {
    constexpr int CW = Cfg<BN, G>::CW;
    const bf16 nan = __float2bfloat16_rn(__int_as_float(0x7fffffff));
    for (; tile < tiles; tile += step, whole_half = false) {
        int tm, tn;
        place(p, tile, tm, tn);
        const int64_t n0 = int64_t(tn) * BN + half * CW;
        for (int w = whole_half ? 0 : q; w <= (whole_half ? 3 : q); ++w) {
            const int64_t m = (int64_t(tm) * G + rank) * BM + 32 * w + int(threadIdx.x & 31);
            if (m >= p.M) continue;
            const int64_t b = uint32_t(m) / uint32_t(p.L), l = m - b * p.L;
            for (int i = 0; i < CW && n0 + i < p.N; ++i) p.out[p.channels_first ? (b * p.N + n0 + i) * p.L + l : m * p.N + n0 + i] = nan;
        }
    }
}

template <int BN, int G>
__global__ void __launch_bounds__(kThreads, 1)
k_proj_fp8(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
           const __grid_constant__ CUtensorMap map_o, Params p) {
    using Cf = Cfg<BN, G>;
    constexpr int kStages = Cf::kStages;
    constexpr uint32_t kStageBytes = Cf::kStageBytes;
    constexpr int CW = Cf::CW;
    extern __shared__ __align__(1024) uint8_t smem_p[];
    // the same offset in both CTAs of a pair: the base is the kernel's own in each
    uint8_t* stages = smem_p + ((1024u - (tc::smem_u32(smem_p) & 1023u)) & 1023u);
    uint8_t* out_stage = stages + kStages * kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + 8 * Cf::kOutWarp);
    uint64_t* done = full + kStages;              // a stage's products and factors: it is free, and its sums are there
    uint64_t* acc_empty = done + kStages;         // [buffer]
    uint64_t* out_full = acc_empty + 2;           // [half]: its four warps have staged their part
    uint64_t* out_free = out_full + 2;            // [half]: the staging has been read
    uint64_t* mma_done = out_free + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    float* s_bias = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + 512);
    float* s_fac = s_bias + 8 * CW;               // [stage][half][row]

    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), lane = int(threadIdx.x) & 31;
    const int rank = G == 2 ? int(blockIdx.x) & 1 : 0;             // in the pair; the first issues the products
    const int first = int(blockIdx.x) / G, step = int(gridDim.x) / G;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&done[s], 3);           // the products, and two warps' factors
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&acc_empty[a], 8 * G);  // one arrival a reading warp
            tc::mbar_init(&out_full[a], 4);
            tc::mbar_init(&out_free[a], 1);
        }
        tc::mbar_init(mma_done, 1);
    }
    if (warp == 1) tmem_alloc<G>(tmem_slot, Cf::kTmemCols);
    tc::fence_before_sync();
    if constexpr (G == 2) cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int tiles = p.tiles_m * p.tiles_n;

    // registers: 384 x 168 at launch = 128 x 56 + 256 x 224
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
        // one thread each: stage and buffer counters step, nothing is divided, so that issuing stays under the products
        if (warp == 0 && lane == 0) {
            int s = 0, issued = 0;
            uint32_t phase = 1;                   // of `done`: the first round finds the stages free
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tm, tn;
                place(p, tile, tm, tn);
                const int m0 = (tm * G + rank) * BM, n0 = tn * BN + rank * (BN / 2);
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!tc::mbar_wait(&done[s], phase, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = stages + s * kStageBytes;
                    if constexpr (G == 2) {
                        // the first CTA's barrier counts the bytes of both
                        if (rank == 0) tc::mbar_expect_tx(&full[s], 2 * kStageBytes);
                        tma_load_pair(sa, &map_x, kb * BKB, m0, &full[s]);
                        tma_load_pair(sa + kATile, &map_w, kb * BKB, n0, &full[s]);
                    } else {
                        tc::mbar_expect_tx(&full[s], kStageBytes);
                        tc::tma_load_2d(sa, &map_x, kb * BKB, m0, &full[s]);
                        tc::tma_load_2d(sa + kATile, &map_w, kb * BKB, n0, &full[s]);
                    }
                    issued = min(issued + 1, kStages);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) report_status(p.status, kStatusTimeout);
            // nothing left in flight: the last loads have landed when their products are done, or (one CTA) at `full`
            for (; issued > 0; --issued) {
                if (s == 0) {
                    s = kStages;
                    phase ^= 1u;
                }
                --s;
                if constexpr (G == 2) tc::mbar_wait(&done[s], phase ^ 1u, p.budget_ns);
                else tc::mbar_wait(&full[s], phase ^ 1u, p.budget_ns);
            }
            // the second CTA of a pair stays until the last arrival at its barriers
            if (rank == 1) tc::mbar_wait(mma_done, 0, p.budget_ns);
        } else if (warp == 1 && rank == 0) {
            // the whole warp walks the loop, so that descriptors stay in uniform registers; one lane issues
            constexpr uint32_t idesc = idesc_e4m3(BM * G, BN);
            const uint64_t da0 = tc::desc_sw128(tc::smem_u32(stages), 16, 1024), db0 = da0 + (kATile >> 4);
            const int tail = int((p.K - int64_t(p.kblocks - 1) * BKB + 31) / 32);     // products of the last block
            int s = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 1;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!tc::mbar_wait(&full[s], phase, p.budget_ns) || !tc::mbar_wait(&acc_empty[acc], acc_phase, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint64_t da = da0 + uint32_t(s) * (kStageBytes >> 4), db = db0 + uint32_t(s) * (kStageBytes >> 4);
                    const uint32_t d = tmem + uint32_t(acc) * BN;
                    // the tail of the last block lies behind K: zeros, and no products for whole steps of them
                    const int steps = kb + 1 < p.kblocks ? 4 : tail;
                    if (p.hold != HOLD_PRODUCTS && elect_one()) {
                        mma_e4m3<G>(d, da, db, idesc, 0u);
                        if (steps > 1) mma_e4m3<G>(d, da + 2, db + 2, idesc, 1u);
                        if (steps > 2) mma_e4m3<G>(d, da + 4, db + 4, idesc, 1u);
                        if (steps > 3) mma_e4m3<G>(d, da + 6, db + 6, idesc, 1u);
                        commit<G>(&done[s]);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                    acc ^= 1;
                    acc_phase ^= acc == 0;
                }
            }
            if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
            // nothing left in flight before tensor memory is released
            if (elect_one()) commit<G>(mma_done);
            __syncwarp();
            if (!tc::mbar_wait(mma_done, 0, p.budget_ns) && lane == 0) report_status(p.status, kStatusTimeout);
        } else if (warp >= 2) {
            // The factors xs Ws of this CTA's rows, two rows a thread, for both halves of the columns.  The loads go out four
            // blocks ahead (registers of a static index), across tiles.
            const int t = int(threadIdx.x) - 64, total = (tiles - first + step - 1) / step * p.kblocks;
            float x0[4], x1[4], w0[4], w1[4];
            int pt = first, pkb = p.kblocks;      // the tile and block to load next
            const float *px0 = nullptr, *px1 = nullptr, *pw0 = nullptr, *pw1 = nullptr;
            bool in0 = false, in1 = false, has0 = false, has1 = false;
            auto load = [&](int u) {
                if (pkb == p.kblocks) {           // enter tile pt
                    int tm, tn;
                    place(p, pt, tm, tn);
                    const uint32_t m = (uint32_t(tm) * G + rank) * BM + t;
                    const int64_t n = int64_t(tn) * BN;
                    const bool more = pt < tiles;
                    in0 = more && m < p.M;
                    in1 = more && m + 64 < p.M;
                    has0 = more && n < p.N;
                    has1 = more && n + CW < p.N;
                    // row m of batch row b: xs + (b kblocks + kb) L + m - b L
                    px0 = p.xs + int64_t(in0 ? m / uint32_t(p.L) : 0) * (p.kblocks - 1) * p.L + m;
                    px1 = p.xs + int64_t(in1 ? (m + 64) / uint32_t(p.L) : 0) * (p.kblocks - 1) * p.L + m + 64;
                    pw0 = p.ws + n / 128 * p.kblocks;
                    pw1 = p.ws + (n + CW) / 128 * p.kblocks;
                    pt += step;
                    pkb = 0;
                }
                x0[u] = in0 ? __ldg(px0) : 0.0f;
                x1[u] = in1 ? __ldg(px1) : 0.0f;
                w0[u] = has0 ? __ldg(pw0) : 0.0f;
                w1[u] = has1 ? __ldg(pw1) : 0.0f;
                px0 += p.L;
                px1 += p.L;
                ++pw0;
                ++pw1;
                ++pkb;
            };
#pragma unroll
            for (int u = 0; u < 4; ++u) load(u);
            // A stage's factors have been read once the sums' buffer of its block, freed by their readers, has been filled
            // by the block two later; so `done` of the block kStages - 2 before is waited for.
            int s = 0, sw = 0;
            uint32_t phase = 0;
            bool ok = true;
#pragma unroll 1
            for (int j0 = 0; j0 < total && ok; j0 += 4) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (j0 + u < total && ok) {
                        if (j0 + u >= kStages - 2) {
                            ok = tc::mbar_wait(&done[sw], phase, p.budget_ns);
                            if (++sw == kStages) {
                                sw = 0;
                                phase ^= 1u;
                            }
                        }
                        float* f = s_fac + s * 256 + t;
                        f[0] = x0[u] * w0[u];
                        f[64] = x1[u] * w0[u];
                        f[128] = x0[u] * w1[u];
                        f[192] = x1[u] * w1[u];
                        load(u);
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&done[s]);
                        if (++s == kStages) s = 0;
                    }
                }
            }
            if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n");
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t t_col = tmem + uint32_t(half * CW) + (uint32_t(32 * q) << 16);
        uint8_t* stage = out_stage + (warp - 4) * Cf::kOutWarp;     // (channels_first: a half's four parts together)
        float* bias = s_bias + (warp - 4) * CW;
        int buf = 0, s = 0;
        uint32_t phase = 0, out_phase = 0;
        bool ok = true, whole_half = false;
        int tile = first;
        for (; tile < tiles; tile += step) {
            int tm, tn;
            place(p, tile, tm, tn);
            const int64_t m0 = (int64_t(tm) * G + rank) * BM + 32 * q, m = m0 + lane;
            const int64_t n0 = int64_t(tn) * BN + half * CW;
            const bool live = m < p.M;
            const int64_t b = live ? uint32_t(m) / uint32_t(p.L) : 0, l = live ? m - b * p.L : 0;
            float bv[CW / 32];                    // the bias of this warp's columns, on its way under the products
#pragma unroll
            for (int i = 0; i < CW / 32; ++i) bv[i] = (p.bias && n0 + 32 * i + lane < p.N) ? __ldg(p.bias + n0 + 32 * i + lane) : 0.0f;
            uint64_t acc[CW / 2];                 // pairs of neighbouring columns
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) acc[i] = 0;
            auto release = [&](int bf) {          // the warp has read buffer bf
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (G == 2) arrive_first(&acc_empty[bf]);
                    else tc::mbar_arrive(&acc_empty[bf]);
                }
            };
#pragma unroll 1
            for (int kb = 0; kb < p.kblocks; ++kb) {
                if (!tc::mbar_wait(&done[s], phase, p.budget_ns)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                // 16 columns load under the multiply-adds of 16, the first while the factor comes
                float v[2][16];
                tc::tmem_ld16(t_col + uint32_t(buf * BN), v[0]);
                const float f = s_fac[s * 256 + half * 128 + 32 * q + lane];
                uint64_t f2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(f2) : "f"(f));
#pragma unroll
                for (int c = 0; c < CW / 16; ++c) {
                    tc::tmem_ld_wait();
                    if (c + 1 < CW / 16) tc::tmem_ld16(t_col + uint32_t(buf * BN + 16 * (c + 1)), v[(c + 1) & 1]);
                    else if (!p.channels_first || kb + 1 < p.kblocks) release(buf);
#pragma unroll
                    for (int i = 0; i < 8; ++i) fma2(acc[8 * c + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], f2);
                }
                buf ^= 1;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            // the warp's own copy: no barrier that a warp which gave up would leave others at
            __syncwarp();
#pragma unroll
            for (int i = 0; i < CW / 32; ++i) bias[32 * i + lane] = bv[i];
            __syncwarp();
            if (p.store == STORE_TMA) {
                // the last tile's stores have read the staging
                if (!p.channels_first || q == 0) {
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
                    __syncwarp();
                    if (p.channels_first && lane == 0) tc::mbar_arrive(&out_free[half]);
                }
                if (p.channels_first && !tc::mbar_wait(&out_free[half], out_phase, p.budget_ns)) {
                    ok = false;
                    break;
                }
            }
            // The staging.  channels_first: the half's [64 positions' box][column][64 positions]; else the warp's [box of kBox
            // columns][row][kBox columns]; 128-byte swizzle (64-byte rows: 64-byte swizzle).
            constexpr int kBox = CW < 64 ? CW : 64;
            uint8_t* half_stage = out_stage + half * (4 * Cf::kOutWarp);
            if (p.channels_first) {
                // The sums go back to the last buffer, held until here, and come again as fragments, which stmatrix
                // transposes: positions together.  (Reading every block as fragments costs twice the reading: 331 us
                // against 277 us at 32768 x 2048 x 4096.)
                const uint32_t t_buf = t_col + uint32_t((buf ^ 1) * BN);
#pragma unroll
                for (int c = 0; c < CW / 2; c += 16) tmem_st32(t_buf + uint32_t(2 * c), *reinterpret_cast<const uint64_t(*)[16]>(acc + c));
                asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
                const int mat = lane >> 3, mr = lane & 7;
#pragma unroll
                for (int c = 0; c < CW / 32; ++c) {
                    float v[2][16];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) tmem_ld_frag(t_buf + uint32_t(32 * c) + (uint32_t(16 * hh) << 16), v[hh]);
                    tc::tmem_ld_wait();
                    if (c + 1 == CW / 32) release(buf ^ 1);
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float2 b0 = *reinterpret_cast<const float2*>(bias + 32 * c + 8 * j + 2 * (lane & 3));
                        const float2 b1 = *reinterpret_cast<const float2*>(bias + 32 * c + 8 * j + 8 + 2 * (lane & 3));
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const float* a = v[hh] + 4 * j;
                            // matrix `mat`: positions 16 hh + 8 (mat & 1) .., columns 8 (4 c + j + (mat >> 1)) ..
                            const int n = 8 * (4 * c + j + (mat >> 1)) + mr, piece = 4 * (q & 1) + 2 * hh + (mat & 1);
                            stmatrix4_trans(tc::smem_u32(half_stage) + (q >> 1) * (CW * 128) + n * 128 + 16 * (piece ^ (n & 7)),
                                            tc::pack2(a[0] + b0.x, a[1] + b0.y), tc::pack2(a[2] + b0.x, a[3] + b0.y),
                                            tc::pack2(a[4] + b1.x, a[5] + b1.y), tc::pack2(a[6] + b1.x, a[7] + b1.y));
                        }
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < CW / 8; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const float2 a0 = unpair(acc[4 * j + i]), a1 = unpair(acc[4 * j + i + 1]);
                        const float4 bb = *reinterpret_cast<const float4*>(bias + 8 * j + 2 * i);
                        w[i] = tc::pack2(a0.x + bb.x, a0.y + bb.y);
                        w[i + 1] = tc::pack2(a1.x + bb.z, a1.y + bb.w);
                    }
                    const int box = j / (kBox / 8), c = j % (kBox / 8);
                    const int at = kBox == 64 ? c ^ (lane & 7) : c ^ ((lane >> 1) & 3);
                    *reinterpret_cast<uint4*>(stage + box * (32 * kBox * 2) + lane * (kBox * 2) + 16 * at) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (p.store == STORE_PLAIN) {
                __syncwarp();
                if (p.channels_first) {
                    bf16* o = p.out + (b * p.N + n0) * p.L + l;
                    const uint8_t* so = half_stage + (q >> 1) * (CW * 128) + 2 * (lane & 7);
                    const int piece = 4 * (q & 1) + (lane >> 3);
#pragma unroll 8
                    for (int n = 0; n < CW; ++n)
                        if (live && n0 + n < p.N) o[int64_t(n) * p.L] = *reinterpret_cast<const bf16*>(so + n * 128 + 16 * (piece ^ (n & 7)));
                } else {
#pragma unroll 4
                    for (int i = lane; i < 32 * CW; i += 32) {
                        const int r = i / CW, n = i % CW, box = n / kBox, c = (n % kBox) / 8;
                        const int at = kBox == 64 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
                        const bf16 w = *reinterpret_cast<const bf16*>(stage + box * (32 * kBox * 2) + r * (kBox * 2) + 16 * at + 2 * (n & 7));
                        if (m0 + r < p.M && n0 + n < p.N) p.out[(m0 + r) * p.N + n0 + n] = w;
                    }
                }
                __syncwarp();
            }
            if (p.store == STORE_TMA) {
                tc::fence_proxy_async();
                __syncwarp();
                if (p.channels_first) {
                    if (lane == 0 && (p.hold != HOLD_STAGED || q != 1)) tc::mbar_arrive(&out_full[half]);
                    if (q == 0 && !tc::mbar_wait(&out_full[half], out_phase, p.budget_ns)) {
                        ok = false;
                        whole_half = true;        // the other warps may be past this tile: theirs do not leave either
                        break;
                    }
                    out_phase ^= 1u;
                }
                if (lane == 0 && m0 < p.M && n0 < p.N && (!p.channels_first || q == 0)) {
                    if (p.channels_first) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(&map_o),
                                         "r"(int(l) + 64 * c), "r"(int(n0)), "r"(int(b)),
                                         "r"(tc::smem_u32(stage + c * (CW * 128)))
                                         : "memory");
                    } else {
#pragma unroll
                        for (int c = 0; c < CW; c += kBox)
                            if (n0 + c < p.N)
                                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(&map_o),
                                             "r"(int(n0) + c), "r"(int(m0)), "r"(tc::smem_u32(stage + c * 64))
                                             : "memory");
                    }
                    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                }
            }
        }
        if (!ok) {
            if (lane == 0) report_status(p.status, kStatusTimeout);
            give_up<BN, G>(p, tile, tiles, step, rank, q, half, whole_half);
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    }
    __syncwarp();
    tc::fence_before_sync();
    if constexpr (G == 2) cluster_sync();         // the pair's barriers and memory live until both are through
    else __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<G>(tmem, Cf::kTmemCols);
}

// ------------------------------------------------------------- a few tokens
constexpr int kFewTokens = 16;
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

bool encode(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle, std::string* why) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    cudaError_t e = tensor_map_encoder(&enc);
    if (e != cudaSuccess) {
        *why = std::string("cuTensorMapEncodeTiled unavailable: ") + cudaGetErrorString(e);
        return false;
    }
    const cuuint32_t one[3] = {1, 1, 1};
    CUresult r = enc(map, type, rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) *why = "cuTensorMapEncodeTiled failed (" + std::to_string(int(r)) + ")";
    return r == CUDA_SUCCESS;
}

// [rows][K] bytes, box of 128 bytes x box_rows, 128-byte swizzle; what lies outside reads as zero.
bool operand_map(CUtensorMap* map, const void* base, int64_t K, int64_t rows, int box_rows, std::string* why) {
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)}, strides[1] = {cuuint64_t(K)};
    const cuuint32_t box[2] = {BKB, cuuint32_t(box_rows)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, why);
}

// The output as it leaves: a warp's 32 rows x 64 columns at a time (channels_first: four warps' 64 positions x cw channels).
bool output_map(CUtensorMap* map, const Params& p, int cw, std::string* why) {
    if (p.channels_first) {
        const cuuint64_t dims[3] = {cuuint64_t(p.L), cuuint64_t(p.N), cuuint64_t(p.M / p.L)};
        const cuuint64_t strides[2] = {cuuint64_t(p.L) * 2, cuuint64_t(p.N * p.L) * 2};
        const cuuint32_t box[3] = {64, cuuint32_t(cw), 1};
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, why);
    }
    const cuuint64_t dims[2] = {cuuint64_t(p.N), cuuint64_t(p.M)}, strides[1] = {cuuint64_t(p.N) * 2};
    const cuuint32_t box[2] = {cuuint32_t(cw < 64 ? cw : 64), 32};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out, dims, strides, box,
                  cw < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, why);
}

template <int BN, int G>
hyena_status_t launch(const void* xq, const void* wq, Params& p, int dev, int sms, cudaStream_t s) {
    using Cf = Cfg<BN, G>;
    static std::atomic<bool> raised[kMaxDevices];
    std::string why;
    CUtensorMap mx, mw, mo;
    p.tiles_m = int((p.M + BM * G - 1) / (BM * G));
    p.tiles_n = int((p.N + BN - 1) / BN);
    // whole 16-byte pieces of rows, and (channels_first) a CTA's 128 positions in one batch row
    p.store = (p.channels_first ? p.L % 128 == 0 : p.N % 8 == 0) ? STORE_TMA : STORE_PLAIN;
    if (!operand_map(&mx, xq, p.K, p.M, BM, &why) || !operand_map(&mw, wq, p.K, p.N, BN / G, &why)) return fail(HYENA_ERR_CUDA, why);
    if (p.store == STORE_TMA && !output_map(&mo, p, Cf::CW, &why)) return fail(HYENA_ERR_CUDA, why);
    if (p.store != STORE_TMA) mo = mx;            // not used
    cudaError_t e = kernel_status_word(&p.status);
    if (e == cudaSuccess)
        e = raise_smem(k_proj_fp8<BN, G>, Cf::kSmem, dev, raised);
    if (e == cudaSuccess) {
        const int tiles = p.tiles_m * p.tiles_n, most = sms / G;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(G * (tiles < most ? tiles : most)));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Cf::kSmem;
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {unsigned(G), 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = G > 1 ? 1 : 0;
        e = cudaLaunchKernelEx(&cfg, k_proj_fp8<BN, G>, mx, mw, mo, p);
    }
    if (e != cudaSuccess) return fail(HYENA_ERR_CUDA, std::string("8-bit projection: ") + cudaGetErrorString(e));
    return set_last_error_detail(HYENA_OK, "");
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace hyena

using namespace hyena;

namespace {

hyena_status_t run(const void* xq, const float* xs, const void* Wq, const float* Ws, const float* bias, void* out, int64_t B,
                   int64_t L, int64_t K, int64_t N, int channels_first, uint64_t budget_ns, int hold, void* stream) {
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
    Params p{M, L, N, K, int(kblocks), 0, 0, xs, Ws, bias, static_cast<bf16*>(out), channels_first != 0, STORE_PLAIN,
             budget_ns, nullptr, hold};
    if (M <= kFewTokens) {
        const unsigned grid = unsigned((N + 15) / 16);
        const uint8_t *x = static_cast<const uint8_t*>(xq), *w = static_cast<const uint8_t*>(Wq);
        if (M <= 8) k_proj_fp8_few<1><<<grid, kFewThreads, 0, s>>>(x, w, p);
        else k_proj_fp8_few<2><<<grid, kFewThreads, 0, s>>>(x, w, p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return fail(HYENA_ERR_CUDA, std::string("8-bit projection: ") + cudaGetErrorString(e));
        return set_last_error_detail(HYENA_OK, "");
    }
    // The widest tile that leaves every SM one; narrower ones spread a small product (K = 768, N = 2304, us by width
    // 256, 128, 64: 4096 rows 14.9, 16.2, 22.1; 2048 rows 10.2, 10.2, 13.3; 33 rows 8.1, 5.4, 5.4).
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return fail(HYENA_ERR_CUDA, std::string("device: ") + cudaGetErrorString(e));
    const int64_t tm = (M + BM - 1) / BM;
    if (tm * ((N + 255) / 256) >= sms) return launch<256, 2>(xq, Wq, p, dev, sms, s);
    if (tm * ((N + 127) / 128) >= sms) return launch<128, 1>(xq, Wq, p, dev, sms, s);
    return launch<64, 1>(xq, Wq, p, dev, sms, s);
}

}  // namespace

extern "C" hyena_status_t hyena_proj_fp8(const void* xq, const float* xs, const void* Wq, const float* Ws,
                                         const float* bias, void* out, int64_t B, int64_t L, int64_t K, int64_t N,
                                         int channels_first, void* stream) {
    return run(xq, xs, Wq, Ws, bias, out, B, L, K, N, channels_first, kDefaultWaitBudgetNs, HOLD_NONE, stream);
}

extern "C" hyena_status_t hyena_debug_proj_fp8(const void* xq, const float* xs, const void* Wq, const float* Ws,
                                               const float* bias, void* out, int64_t B, int64_t L, int64_t K, int64_t N,
                                               int channels_first, uint64_t wait_budget_ns, int hold, void* stream) {
    if (wait_budget_ns == 0) return fail(HYENA_ERR_INVALID_ARG, "wait_budget_ns must be > 0");
    if (hold < HOLD_NONE || hold > HOLD_STAGED) return fail(HYENA_ERR_INVALID_ARG, "hold must be 0, 1 or 2");
    if (B >= 1 && B <= kFewTokens && L >= 1 && L <= kFewTokens && B * L <= kFewTokens)
        return fail(HYENA_ERR_UNSUPPORTED_SHAPE, "a few rows have no waits");
    return run(xq, xs, Wq, Ws, bias, out, B, L, K, N, channels_first, wait_budget_ns, hold, stream);
}
