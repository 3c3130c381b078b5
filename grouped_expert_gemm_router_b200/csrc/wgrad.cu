// Gradients of the expert weights on the sm_100a tensor cores (no counterpart
// on the source pages, which stop at the forward path: the chain rule of the
// grouped products):
//   dW[e][m, n] = sum over the rows r of expert e of A[r, m] * B[r, n]
// in fp32, rounded once to bf16 (the weights' type).  Gate and up together:
// A = x_perm, B = dg, then du; down: A = h, B = dy.
//
// Design:
// - The reduction runs over an expert's rows, whose number only the device
//   knows; the output is fixed.  So a work unit is an output tile of 256 x 256
//   (two 128-row accumulators of 256 columns, all of tensor memory) of one
//   expert, and its K loop walks the expert's row segments (uncapped: one;
//   capacity layout: the capacity slots, then the overflow rows) in blocks of
//   64 rows.  Units are in descending row count of their experts and are dealt
//   back and forth (CTA c takes unit c, 2n - 1 - c, 2n + c, ...): dealt in one
//   direction, the first CTA gets the largest unit of every round, and under
//   skew (8192 tokens, 128 experts, alpha 1) SMs idled 14% of the time: 416 ->
//   380 us for gate and up, the same bits.
// - Both operands are row-major [rows, features] and reduced over rows, so
//   both are MN-major for the MMA and are loaded as they lie (64-feature x
//   64-row boxes, 128-byte swizzle).
// - The last block of a segment also holds rows of the next expert, or slots
//   nobody wrote (NaN for all we know).  MMAs cover 16 rows each: those past
//   the segment are not issued, and the rows between the segment's end and the
//   next multiple of 16 are overwritten with zeros in shared memory, in both
//   operands, by the issuing warp before its MMAs.
// - An expert without rows gets zeros.
// - Persistent and warp-specialised like the forward GEMMs: warp 0 loads,
//   warp 1 issues tcgen05.mma, warps 4-11 drain tensor memory: they take the
//   whole unit into registers as packed bf16, hand the accumulators back, and
//   store through per-warp staging blocks with TMA while the next unit's MMAs
//   run.
// - Every wait is bounded as in the forward GEMMs (MOE_DEV_GEMM_TIMEOUT).
//
// What bounds it.  Few rows per expert: the bytes written, with as many loaded
// to make them (T 512, 8 experts, 4096 x 14336, two K blocks per unit: 180-199
// us alone, 0.94 GB written at 4.7-5.3 TB/s and 2.26 GB through L2; stores
// alone reach 6.2-6.9 TB/s, loads from L2 alone 21).  Many rows: inside a unit
// shared memory, 64 KB of TMA writes and 96 KB of MMA reads per 64 rows at 128
// bytes a cycle, 1280 cycles for 1024 of MMA; around it the drain, which no MMA
// overlaps, because the two accumulators are all of tensor memory (65536 rows,
// 128 experts, gate and up of 2048 x 768, eight K blocks per unit: 378-398 us,
// 1.04-1.09 PFLOP/s, the tensor pipe busy 59%; 16384 rows, 8 experts, 4096 x
// 2560: 453 us, 1.52 PFLOP/s).  Pairs of CTAs on 512 x 256 outputs move a
// quarter less and were no faster (404-440 and 495 us): their MMAs run at 80%
// of the nominal rate.
#include <cuda_bf16.h>

#include "common.cuh"
#include "tmap.cuh"

namespace moe {

namespace {

constexpr int kWBK = 64;                          // rows per stage
constexpr uint32_t kWBox = 64 * kWBK * 2;         // 64 features x 64 rows: 8 KiB
constexpr uint32_t kWHalf = 2 * kWBox;            // 128 features of one operand
constexpr uint32_t kWStage = 4 * kWHalf;          // 256 features of A, 256 of B
constexpr int kWStages = 3;
constexpr int kWEpiWarp0 = 4;                     // warps 2 and 3 idle: three warps per SM quarter leave
constexpr int kWEpiWarps = 8;                     // each thread 168 registers, room for 128 packed results
constexpr int kWThreads = 32 * (kWEpiWarp0 + kWEpiWarps);
constexpr uint32_t kWStaging = 32 * 128;          // per epilogue warp: 32 rows x 64 columns of bf16
constexpr uint32_t kWCtrl = 256;
constexpr uint32_t kWSmem = 1024 + kWStages * kWStage + kWEpiWarps * kWStaging + kWCtrl;
static_assert(kWSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kWTmemCols = 512;

struct WgradArgs {
    const int *order;      // experts by descending row count
    const int *offsets;    // uncapped: first row of each expert
    const int *cap_cnt;    // rows in the capacity slots (uncapped: all rows)
    const int *spill_cnt, *spill_off;
    uint32_t *status;
    int E, C, P, capped;
    int m_tiles, m_blocks;  // 256-row tiles and 128-row blocks of the output
    int n_tiles, n_blocks;  // the same of its columns, both outputs one after the other
    int blocks0;            // column blocks of the first output
    int MA;                 // rows of one expert's output
    int stall_last_unit;    // test hook: CTA 0's producer never loads the first stage of its last unit
    unsigned long long timeout_ns;
};

struct WUnit {
    int e, m0, macc, n0, nacc;  // first 128-blocks and how many (1 or 2) of each
    int s0, l0, s1, l1;         // row segments
    int nkb;
};

// The CTA's unit of the next round.
__device__ __forceinline__ int w_next(int &round) {
    ++round;
    return round * (int)gridDim.x + (int)(round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ bool w_decode(int u, const WgradArgs &a, WUnit &U) {
    const int per = a.m_tiles * a.n_tiles;
    const int g = u / per, v = u - g * per;
    U.e = a.order[g];
    if ((unsigned)U.e >= (unsigned)a.E) return false;  // only for a corrupt schedule
    const int mt = v / a.n_tiles, nt = v - mt * a.n_tiles;
    U.m0 = 2 * mt;
    U.macc = min(2, a.m_blocks - U.m0);
    U.n0 = 2 * nt;
    U.nacc = min(2, a.n_blocks - U.n0);
    U.l0 = a.cap_cnt[U.e];
    U.l1 = a.capped ? a.spill_cnt[U.e] : 0;
    U.s0 = a.capped ? U.e * a.C : a.offsets[U.e];
    U.s1 = a.capped ? a.E * a.C + a.spill_off[U.e] : 0;
    if (U.l0 < 0 || U.l1 < 0 || U.s0 < 0 || U.s1 < 0 || U.l0 > a.P - U.s0 || U.l1 > a.P - U.s1) return false;
    U.nkb = (U.l0 + kWBK - 1) / kWBK + (U.l1 + kWBK - 1) / kWBK;
    return true;
}

// Block kb of the unit's rows: its first row and how many of its 64 rows are
// the expert's.
__device__ __forceinline__ void w_block(const WUnit &U, int kb, int &row, int &n) {
    const int n0 = (U.l0 + kWBK - 1) / kWBK;
    if (kb < n0) {
        row = U.s0 + kb * kWBK;
        n = min(kWBK, U.l0 - kb * kWBK);
    } else {
        row = U.s1 + (kb - n0) * kWBK;
        n = min(kWBK, U.l1 - (kb - n0) * kWBK);
    }
}

__device__ __forceinline__ void tma_store_2d(const void *tmap, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmap),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The staging block may be rewritten once the copies have read it.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint32_t w_pack(uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void w_abort(volatile int *abort, uint32_t *status) {
    *abort = 1;
    atomicOr(status, MOE_DEV_GEMM_TIMEOUT);
}

__global__ void __launch_bounds__(kWThreads, 1)
    k_wgrad(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
            const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmD0,
            const __grid_constant__ CUtensorMap tmD1, WgradArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *staging = smem + kWStages * kWStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + kWEpiWarps * kWStaging);
    uint64_t *empty = full + kWStages;
    uint64_t *tfull = empty + kWStages;
    uint64_t *tempty = tfull + 1;
    uint64_t *mma_done = tempty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *s_abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, kWEpiWarps);
        mbar_init(mma_done, 1);
        *s_abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB0);
        tma_prefetch_desc(&tmB1);
        tma_prefetch_desc(&tmD0);
        tma_prefetch_desc(&tmD1);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kWTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();  // the schedule and both operands come from earlier kernels
    const int total = a.E * a.m_tiles * a.n_tiles;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ----
        if (lane == 0) {
            int stage = 0;
            uint32_t ph = 0;
            int issued_ph[kWStages];
            for (int s = 0; s < kWStages; ++s) issued_ph[s] = -1;
            bool ok = true;
            for (int u = blockIdx.x, i = 0; u < total && ok; u = w_next(i)) {
                WUnit U;
                if (!w_decode(u, a, U)) {
                    atomicOr(a.status, MOE_DEV_BAD_ROW);
                    continue;
                }
                const uint32_t bytes = (uint32_t)(U.macc + U.nacc) * kWHalf;
                for (int kb = 0; kb < U.nkb; ++kb) {
                    if (!mbar_wait_bounded(&empty[stage], ph ^ 1u, a.timeout_ns, s_abort)) {
                        ok = false;
                        break;
                    }
                    int next = i;
                    if (a.stall_last_unit && kb == 0 && blockIdx.x == 0 && w_next(next) >= total) {
                        // test hook: this stage is never loaded (no copy is in
                        // flight for it), so the MMA issuer's wait expires
                        if (++stage == kWStages) {
                            stage = 0;
                            ph ^= 1u;
                        }
                        continue;
                    }
                    int row, n;
                    w_block(U, kb, row, n);
                    mbar_arrive_expect_tx(&full[stage], bytes);
                    uint8_t *sa = smem + stage * kWStage, *sb = sa + 2 * kWHalf;
                    for (int i = 0; i < 2 * U.macc; ++i)
                        tma_load_2d(sa + i * kWBox, &tmA, &full[stage], U.m0 * 128 + 64 * i, row);
                    for (int i = 0; i < U.nacc; ++i) {
                        const int nb = U.n0 + i;
                        const CUtensorMap *tm = nb < a.blocks0 ? &tmB0 : &tmB1;
                        const int x = 128 * (nb < a.blocks0 ? nb : nb - a.blocks0);
                        tma_load_2d(sb + (2 * i) * kWBox, tm, &full[stage], x, row);
                        tma_load_2d(sb + (2 * i + 1) * kWBox, tm, &full[stage], x + 64, row);
                    }
                    issued_ph[stage] = (int)ph;
                    if (++stage == kWStages) {
                        stage = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok && !*s_abort) w_abort(s_abort, a.status);
            // Every issued copy must land before the CTA may leave.
            int never = 0;
            for (int s = 0; s < kWStages; ++s)
                if (issued_ph[s] >= 0) mbar_wait_bounded(&full[s], (uint32_t)issued_ph[s], a.timeout_ns, &never);
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer ----
        int stage = 0;
        uint32_t ph = 0, uses = 0;
        bool ok = true;
        const uint32_t base = smem_u32(smem);
        for (int u = blockIdx.x, i = 0; u < total && ok; u = w_next(i)) {
            WUnit U;
            if (!w_decode(u, a, U)) continue;
            if (U.nkb == 0) continue;  // the epilogue writes zeros on its own
            const uint32_t idesc = idesc_bf16_f32(128, 128 * U.nacc, 1, 1);
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(tempty, (uses & 1u) ^ 1u, a.timeout_ns, s_abort));
            if (!ok) break;
            tc_fence_after();
            for (int kb = 0; kb < U.nkb; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], ph, a.timeout_ns, s_abort));
                if (!ok) break;
                int row, n;
                w_block(U, kb, row, n);
                const uint32_t sa = base + stage * kWStage, sb = sa + 2 * kWHalf;
                if (n & 15) {
                    // rows n .. of the last 16: zeros.  One row of a box is one
                    // 128-byte line (the swizzle permutes inside it).
                    const int nz = (16 - (n & 15)) * 8;  // 16-byte pieces per box
                    for (int i = 0; i < 2 * (U.macc + U.nacc); ++i) {
                        const uint32_t box = i < 2 * U.macc ? sa + i * kWBox : sb + (i - 2 * U.macc) * kWBox;
                        for (int j = lane; j < nz; j += 32) sts128(box + n * 128 + 16 * j, 0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                __syncwarp();
                tc_fence_after();
                const int steps = (n + 15) >> 4;
#pragma unroll
                for (int kk = 0; kk < kWBK / 16; ++kk) {
                    if (kk >= steps) break;
                    // both operands MN-major: 16 rows (2 KiB) per MMA, the 64-feature boxes 8 KiB apart
                    const uint64_t bdesc = sdesc_sw128(sb + kk * 2048, kWBox, 1024);
                    const uint32_t accum = (kb | kk) ? 1u : 0u;
                    tc_mma_bf16_warp(tmem, sdesc_sw128(sa + kk * 2048, kWBox, 1024), bdesc, idesc, accum);
                    if (U.macc == 2)
                        tc_mma_bf16_warp(tmem + 256u, sdesc_sw128(sa + kWHalf + kk * 2048, kWBox, 1024), bdesc, idesc,
                                         accum);
                }
                tc_commit_warp(&empty[stage]);
                if (++stage == kWStages) {
                    stage = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            tc_commit_warp(tfull);
            ++uses;
        }
        if (!ok && lane == 0 && !*s_abort) w_abort(s_abort, a.status);
        __syncwarp();
        // All MMAs issued by this warp complete before tensor memory is freed.
        int never = 0;
        tc_commit_warp(mma_done);
        mbar_wait_bounded(mma_done, 0, a.timeout_ns, &never);
        __syncwarp();
    } else if (warp >= kWEpiWarp0) {
        // ---------------------------------------------------- epilogue ----
        const int q = warp & 3;                    // tensor-memory lane quarter
        const int sub = (warp - kWEpiWarp0) >> 2;  // 128-column block of each accumulator
        const uint32_t stg = smem_u32(staging + (warp - kWEpiWarp0) * kWStaging);
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + 128u * sub;
        uint32_t uses = 0;
        for (int u = blockIdx.x, i = 0; u < total; u = w_next(i)) {
            WUnit U;
            if (!w_decode(u, a, U)) continue;
            const bool mine = sub < U.nacc;
            const int nb = U.n0 + sub;
            const CUtensorMap *tm = nb < a.blocks0 ? &tmD0 : &tmD1;
            const int x = 128 * (nb < a.blocks0 ? nb : nb - a.blocks0);
            const int y = U.e * a.MA + U.m0 * 128 + 32 * q;
            uint8_t *stage_out = staging + (warp - kWEpiWarp0) * kWStaging;
            // this warp's 32 rows x 64 columns at (y, x) from the staging block
            auto put = [&](int acc, int hf) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(tm, stage_out, x + 64 * hf, y + 128 * acc);
                    bulk_commit();
                }
            };
            auto reuse = [&]() {
                if (lane == 0) bulk_wait_read();
                __syncwarp();
            };
            if (U.nkb == 0) {
                if (!mine) continue;
                reuse();
#pragma unroll
                for (int c = 0; c < 8; ++c) sts128(stg + lane * 128 + 16 * c, 0, 0, 0, 0);
                for (int i = 0; i < 2 * U.macc; ++i) put(i >> 1, i & 1);
                continue;
            }
            // this wait lasts for the whole reduction (under 0.1 s per 65536 blocks)
            const uint64_t limit = a.timeout_ns * (1u + (uint32_t)U.nkb / 65536u);
            const bool got = mbar_wait_bounded(tfull, uses & 1u, limit, s_abort);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0 && !*s_abort) w_abort(s_abort, a.status);
                break;
            }
            ++uses;
            tc_fence_after();
            uint32_t v[2][64];  // columns 2 i, 2 i + 1 of this thread's row of each accumulator
            if (mine) {
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    uint32_t r[16];
                    tmem_ld16(tq + 256u * (c >> 3) + 16u * (c & 7), r);  // without a second accumulator: not stored
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[c >> 3][8 * (c & 7) + i] = w_pack(r[2 * i], r[2 * i + 1]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty);
            if (!mine) continue;
#pragma unroll
            for (int acc = 0; acc < 2; ++acc) {
                if (acc < U.macc) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        reuse();
                        // 128-byte rows, 128-byte swizzle: 16-byte piece c of row r at c ^ (r & 7)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            sts128(stg + lane * 128 + 16 * (c ^ (lane & 7)), v[acc][32 * hf + 4 * c],
                                   v[acc][32 * hf + 4 * c + 1], v[acc][32 * hf + 4 * c + 2],
                                   v[acc][32 * hf + 4 * c + 3]);
                        put(acc, hf);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kWTmemCols);
    }
}

}  // namespace

// dW0[e] = A_e^T B0_e and, with B1, dW1[e] = A_e^T B1_e: A [P, MA], B [P, NB],
// dW [E, MA, NB], all bf16, A_e the rows of expert e.
cudaError_t launch_wgrad(const moe_shape &s, int MA, int NB, const void *A, const void *B0, const void *B1, void *dW0,
                         void *dW1, const WsLayout &L, void *ws, uint64_t timeout_ns, int num_sms,
                         cudaStream_t stream) {
    const bool capped = (s.flags & MOE_FLAG_CAPACITY) != 0;
    const int64_t P = permuted_rows(s.T, s.E, s.k, s.C, capped);
    CUtensorMap tA, tB0, tB1, tD0, tD1;
    if (!make_tmap(&tA, A, (uint64_t)P, (uint64_t)MA, 64, kWBK) ||
        !make_tmap(&tB0, B0, (uint64_t)P, (uint64_t)NB, 64, kWBK) ||
        !make_tmap(&tB1, B1 ? B1 : B0, (uint64_t)P, (uint64_t)NB, 64, kWBK) ||
        !make_tmap(&tD0, dW0, (uint64_t)s.E * MA, (uint64_t)NB, 64, 32) ||
        !make_tmap(&tD1, B1 ? dW1 : dW0, (uint64_t)s.E * MA, (uint64_t)NB, 64, 32))
        return cudaErrorInvalidValue;
    WsPtrs p = ws_ptrs(ws, L);
    WgradArgs a = {};
    a.order = p.order;
    a.offsets = p.offsets;
    a.cap_cnt = p.cap_cnt;
    a.spill_cnt = p.spill_cnt;
    a.spill_off = p.spill_off;
    a.status = p.status;
    a.E = s.E;
    a.C = s.C;
    a.P = (int)P;
    a.capped = capped;
    a.m_blocks = MA / 128;
    a.m_tiles = (a.m_blocks + 1) / 2;
    a.blocks0 = NB / 128;
    a.n_blocks = (B1 ? 2 : 1) * a.blocks0;
    a.n_tiles = (a.n_blocks + 1) / 2;
    a.MA = MA;
    a.stall_last_unit = (s.flags & MOE_FLAG_TEST_STALL_GEMM) ? 1 : 0;
    a.timeout_ns = timeout_ns;
    const int64_t total = (int64_t)s.E * a.m_tiles * a.n_tiles;
    if (total >= (1ll << 31) - num_sms) return cudaErrorInvalidValue;
    const int grid = total < num_sms ? (int)total : num_sms;
    return launch_pdl_smem(k_wgrad, dim3(grid), dim3(kWThreads), kWSmem, stream, tA, tB0, tB1, tD0, tD1, a);
}

}  // namespace moe
