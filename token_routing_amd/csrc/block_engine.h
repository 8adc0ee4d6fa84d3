// Main loop of the feed-forward block's kernels: gemm_engine.h's tiles and MFMAs
// with the MFMA's operands exchanged (Cfg::SWAP), on a ring of NST LDS stages of
// DEPTH reduction elements (16-bit units: 64 or 32).
//
// LDS is addressed by 32-bit offsets throughout.  A stage's one wait and barrier
// stand before its last 16-deep step (ring_loop_body), whose MFMAs then cover
// the barrier, the reads of the next stage's first fragments and the start of
// the copies that replace this stage.  Against the barrier at a stage's begin:
// 8192 rows by 28672 columns of 4096 int8 0.985 -> 0.954 ms, the gated step of the
// same sizes in bf16 3.13 -> 3.01 ms.  Tried and slower: 32-deep stages in a ring of
// four (1.06 ms for the integers), copies spread over the MFMAs of the last step
// (0.99) or of the whole stage (1.05), reads spread over the MFMAs (0.99), lines
// touched two stages ahead (1.04).
//
// The epilogues leave LDS alone, so that a persistent kernel starts the copies of the
// next tile's first stages (ring_start) before this tile's epilogue.  Its MFMAs do not
// start so early: the epilogue's stores are issued behind those copies and count with them,
// so that the first stage waits until a stage's copies' worth of operations is left, and the
// second, in a ring of two, until every store is done.
#pragma once

#include "gemm_engine.h"

namespace moegg {


// A 32-bit LDS offset as a pointer: no cast of a generic pointer, whose null
// check costs instructions in the loop (and which the compiler rejects in some
// kernels: "operand has incorrect register class").
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Wint-to-pointer-cast"
template <class T>
__device__ __forceinline__ __attribute__((address_space(3))) T *lds_ptr(uint32_t addr)
{
    return (__attribute__((address_space(3))) T *)addr;
}
#pragma clang diagnostic pop

// 16-byte chunk of a reduction-contiguous row of DEPTH elements: 16 rows read at
// one chunk fall in 16 bank groups (as lds_swz and slot_off).
template <int DEPTH>
__device__ __forceinline__ int ring_chunk(int row, int chunk)
{
    static_assert(DEPTH == 64 || DEPTH == 32, "128- or 64-byte rows");
    return DEPTH == 64 ? chunk ^ ((row >> 1) & 7) : chunk ^ ((row >> 2) & 3);
}

// ROWS tile rows, reduction contiguous in HBM (as DmaLoader).
template <int ROWS, int NT, int DEPTH>
struct RingLoader {
    static constexpr int CH = DEPTH / 8;     // chunks per row
    static constexpr int PASS = NT / CH;     // rows per pass
    static constexpr int RPT = ROWS / PASS;  // copies per wave and stage
    static_assert(ROWS % PASS == 0 && PASS % 16 == 0, "whole passes, one swizzle");
    uint32_t off[RPT];

    __device__ __forceinline__ static int tile_row(int i) { return threadIdx.x / CH + i * PASS; }
    __device__ __forceinline__ static int chunk()
    {
        return ring_chunk<DEPTH>(threadIdx.x / CH, threadIdx.x % CH);
    }
    __device__ __forceinline__ void set_row(int i, int64_t row, int64_t row_bytes)
    {
        off[i] = row < 0 ? kOOB : (uint32_t)(row * row_bytes) + chunk() * 16;
    }
    // Copy i of reduction elements [k0, k0 + DEPTH) to the stage part at `lds`.
    __device__ __forceinline__ void issue(const u32x4_t &r, int i, uint32_t lds, int k0,
                                          int klen) const
    {
        const bool kin = k0 + chunk() * 8 < klen;
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        copy16_to_lds(r, kin ? off[i] : kOOB, (uint32_t)k0 * 2,
                      __builtin_amdgcn_readfirstlane(lds + (i * (NT / kWave) + wave) * 1024));
    }
};

// DEPTH reduction rows of COLS columns, contiguous rows of pitch row_bytes (as
// TileDmaLoader): copy i covers whole rows.
template <int COLS, int NT, int DEPTH>
struct RingTileLoader {
    static constexpr int CPR = COLS / 8, RW = kWave / CPR, NWAVE = NT / kWave;
    static constexpr int RPT = DEPTH / (RW * NWAVE);
    static_assert(kWave % CPR == 0 && DEPTH % (RW * NWAVE) == 0, "whole windows per stage");
    uint32_t off[RPT];
    int row_bytes;

    __device__ __forceinline__ static int row_of(int i)
    {
        return ((int)threadIdx.x / kWave + i * NWAVE) * RW + (int)(threadIdx.x % kWave) / CPR;
    }
    __device__ __forceinline__ void init(int col0, int ncols, int64_t pitch)
    {
        row_bytes = (int)pitch;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int row = row_of(i);
            const int col = col0 + (((int)threadIdx.x % CPR) ^ ((row & 3) << 2)) * 8;
            off[i] = col < ncols ? (uint32_t)row * (uint32_t)row_bytes + (uint32_t)col * 2 : kOOB;
        }
    }
    // Rows [k0, k0 + DEPTH), zeros from klen on.
    __device__ __forceinline__ void issue(const u32x4_t &r, int i, uint32_t lds, int k0,
                                          int klen) const
    {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        copy16_to_lds(r, k0 + row_of(i) < klen ? off[i] : kOOB,
                      __builtin_amdgcn_readfirstlane((uint32_t)k0 * (uint32_t)row_bytes),
                      __builtin_amdgcn_readfirstlane(lds + (i * NWAVE + wave) * 1024));
    }
};

// A tile shape (Cfg) with its ring: NST stages of DEPTH.
template <int BM, int BN, int WM, int WN, bool I8, int DEPTH_, int NST_>
struct RingCfg : Cfg<BM, BN, WM, WN, true, I8> {
    static constexpr int DEPTH = DEPTH_, NST = NST_;
    static constexpr int A = BM * DEPTH * 2, B = BN * DEPTH * 2, STAGE = A + B;
    static constexpr int BYTES = NST * STAGE;
    static_assert((NST & (NST - 1)) == 0 && NST >= 2 && NST <= 4, "2 or 4 stages");
};

// Fragment r (A blocks, then B blocks) of 16-deep step kk of the stage at LDS offset `st`.
template <class C, bool B_TR, bool PART>
__device__ __forceinline__ void ring_read_one(uint32_t st, int kk, int r, int wm, int wn,
                                              bf16x8_t (&a)[C::FM], bf16x8_t (&b)[C::FN], int ib)
{
    constexpr int DEPTH = C::DEPTH;
    const int lane = threadIdx.x & (kWave - 1);
    const int row = lane & 31, chunk = kk * 2 + (lane >> 5);
    const uint32_t in = (uint32_t)(row * DEPTH * 2 + (ring_chunk<DEPTH>(row, chunk) << 4));
    if (r < C::FM) {
        if (!PART || r < ib)
            a[r] = *lds_ptr<const bf16x8_t>(st + in + (wm * C::TM + r * 32) * DEPTH * 2);
        return;
    }
    const int j = r - C::FM;
    const uint32_t bs = st + C::A;
    if constexpr (B_TR) {
        const int q = lane & 15;
        const int k = kk * 16 + 8 * (lane >> 5) + (q >> 2);
        const int col = wn * C::TN + j * 32 + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
        const uint32_t at = bs + tr_off<C::BN>(k, col >> 3) + (col & 7) * 2;
        const v4i16_t both[2] = {
            __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<v4i16_t>(at)),
            __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<v4i16_t>(at + 4 * C::BN * 2))};
        b[j] = __builtin_bit_cast(bf16x8_t, both);
    } else {
        b[j] = *lds_ptr<const bf16x8_t>(bs + in + (wn * C::TN + j * 32) * DEPTH * 2);
    }
}

// Waits until at most the copies of the last `newer` stages are in flight.
template <int CPS>
__device__ __forceinline__ void wait_stages(int newer)
{
    if (newer >= 3)
        wait_vmcnt<3 * CPS>();
    else if (newer == 2)
        wait_vmcnt<2 * CPS>();
    else if (newer == 1)
        wait_vmcnt<CPS>();
    else
        wait_vmcnt<0>();
}

// Starts the copies of the first NST stages of a tile.  copy(s, n, lds): this
// wave's copy n (0 .. CPS - 1) of stage s to the LDS offset of its buffer.
template <class C, int CPS, class Copy>
__device__ __forceinline__ void ring_start(uint32_t lds, int nsteps, const Copy &copy)
{
    for (int s = 0; s < C::NST && s < nsteps; ++s)
#pragma unroll
        for (int n = 0; n < CPS; ++n)
            copy(s, n, lds + s * C::STAGE);
}

// A stage's last step holds the wait and the barrier: behind it every wave has
// read the stage's last fragments, so that its buffer takes the copies of stage
// s + NST, and stage s + 1 has landed, so that its first fragments are read while
// the last step's MFMAs run.
template <class C, bool B_TR, int CPS, bool PART, class Copy>
__device__ __forceinline__ void ring_loop_body(uint32_t lds, int nsteps,
                                               f32x16_t (&acc)[C::FM][C::FN], const Copy &copy,
                                               int wm, int wn, int ib)
{
    constexpr int KK = C::DEPTH / 16, NST = C::NST, NR = C::FM + C::FN;
    static_assert(KK % 2 == 0, "two sets of fragments");
    bf16x8_t a[2][C::FM], b[2][C::FN];
    // Stage 0 has landed: loads complete in order among themselves, so that with one
    // of its copies outstanding those of the other stages started are as well, and
    // more operations (stores behind them or not) than are allowed here.
    wait_stages<CPS>(min(NST, nsteps) - 1);
    wait_lds();
    wg_barrier();
#pragma unroll
    for (int r = 0; r < NR; ++r)
        ring_read_one<C, B_TR, PART>(lds, 0, r, wm, wn, a[0], b[0], ib);
    for (int s = 0; s < nsteps; ++s) {
        const uint32_t st = lds + (s & (NST - 1)) * C::STAGE;
        const uint32_t next = lds + ((s + 1) & (NST - 1)) * C::STAGE;
#pragma unroll
        for (int kk = 0; kk < KK - 1; ++kk) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
                ring_read_one<C, B_TR, PART>(st, kk + 1, r, wm, wn, a[(kk + 1) & 1], b[(kk + 1) & 1],
                                             ib);
            __builtin_amdgcn_sched_barrier(0);
            mma_step<C, PART>(a[kk & 1], b[kk & 1], acc, ib);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_stages<CPS>(min(NST - 2, nsteps - 2 - s));  // those started after s + 1
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        wg_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < nsteps) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
                ring_read_one<C, B_TR, PART>(next, 0, r, wm, wn, a[0], b[0], ib);
        }
        if (s + NST < nsteps) {
#pragma unroll
            for (int n = 0; n < CPS; ++n)
                copy(s + NST, n, st);
        }
        __builtin_amdgcn_sched_barrier(0);
        mma_step<C, PART>(a[(KK - 1) & 1], b[(KK - 1) & 1], acc, ib);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The tile whose copies ring_start began.  rows: real rows of the tile; a wave of a
// ragged tail skips its padding blocks' reads and MFMAs and keeps every barrier.
template <class C, bool B_TR, int CPS, class Copy>
__device__ __forceinline__ void ring_loop(uint32_t lds, int nsteps, f32x16_t (&acc)[C::FM][C::FN],
                                          const Copy &copy, int rows)
{
    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int ib = __builtin_amdgcn_readfirstlane(
        min(C::FM, max(0, (rows - wm * C::TM + 31) / 32)));
    if (ib == C::FM)
        ring_loop_body<C, B_TR, CPS, false>(lds, nsteps, acc, copy, wm, wn, ib);
    else
        ring_loop_body<C, B_TR, CPS, true>(lds, nsteps, acc, copy, wm, wn, ib);
}

}  // namespace moegg
