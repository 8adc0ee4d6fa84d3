// Main loop of the feed-forward block's kernels: gemm_engine.h's tiles and MFMAs
// with the MFMA's operands exchanged (Cfg::SWAP), on a ring of NST LDS stages of
// DEPTH reduction elements (16-bit units: 64 or 32).
//
// LDS is addressed by 32-bit offsets throughout.  Stage s waits for its own
// copies, passes one barrier, starts the copies of stage s + NST - 1 into the
// buffer that every wave has left at that barrier, and runs its MFMAs.
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

template <class C, int DEPTH, int NST>
struct Ring {
    static constexpr int A = C::BM * DEPTH * 2, B = C::BN * DEPTH * 2, STAGE = A + B;
    static constexpr int BYTES = NST * STAGE;
};

// Fragments of 16-deep step kk of the stage at LDS offset `st`.
template <class C, int DEPTH, bool B_TR, bool PART>
__device__ __forceinline__ void ring_read(uint32_t st, int kk, int wm, int wn,
                                          bf16x8_t (&a)[C::FM], bf16x8_t (&b)[C::FN], int ib)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int r = lane & 31, chunk = kk * 2 + (lane >> 5);
    const uint32_t in = (uint32_t)(r * DEPTH * 2 + (ring_chunk<DEPTH>(r, chunk) << 4));
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
        if (!PART || i < ib)
            a[i] = *lds_ptr<const bf16x8_t>(st + in + (wm * C::TM + i * 32) * DEPTH * 2);
    const uint32_t bs = st + C::BM * DEPTH * 2;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        if constexpr (B_TR) {
            const int q = lane & 15;
            const int row = kk * 16 + 8 * (lane >> 5) + (q >> 2);
            const int col = wn * C::TN + j * 32 + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
            const uint32_t at = bs + tr_off<C::BN>(row, col >> 3) + (col & 7) * 2;
            const v4i16_t both[2] = {
                __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<v4i16_t>(at)),
                __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<v4i16_t>(at + 4 * C::BN * 2))};
            b[j] = __builtin_bit_cast(bf16x8_t, both);
        } else {
            b[j] = *lds_ptr<const bf16x8_t>(bs + in + (wn * C::TN + j * 32) * DEPTH * 2);
        }
    }
}

// copy(s, n, lds): this wave's copy n (0 .. CPS - 1) of stage s to the LDS offset of
// its buffer.
template <class C, int DEPTH, int NST, bool B_TR, int CPS, bool PART, class Copy>
__device__ __forceinline__ void ring_loop_body(uint32_t lds, int nsteps,
                                               f32x16_t (&acc)[C::FM][C::FN], Copy &copy, int wm,
                                               int wn, int ib)
{
    typedef Ring<C, DEPTH, NST> R;
    constexpr int KK = DEPTH / 16;
    // None of the compiler's own loads is pending from here on: a wait for one
    // inside the loop would wait for the copies too.
    __builtin_amdgcn_s_waitcnt(0);
    for (int s = 0; s < NST - 1 && s < nsteps; ++s)
#pragma unroll
        for (int n = 0; n < CPS; ++n)
            copy(s, n, lds + s * R::STAGE);
    for (int s = 0; s < nsteps; ++s) {
        const int pending = min(NST - 2, nsteps - 1 - s);
        if (pending >= 2)
            wait_vmcnt<2 * CPS>();
        else if (pending == 1)
            wait_vmcnt<CPS>();
        else
            wait_vmcnt<0>();
        wait_lds();
        wg_barrier();
        if (s + NST - 1 < nsteps) {
            const uint32_t to = lds + ((s + NST - 1) & (NST - 1)) * R::STAGE;
#pragma unroll
            for (int n = 0; n < CPS; ++n)
                copy(s + NST - 1, n, to);
        }
        const uint32_t st = lds + (s & (NST - 1)) * R::STAGE;
        // Fragment reads a step ahead of the MFMAs.
        bf16x8_t a[2][C::FM], b[2][C::FN];
        ring_read<C, DEPTH, B_TR, PART>(st, 0, wm, wn, a[0], b[0], ib);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            if (kk + 1 < KK)
                ring_read<C, DEPTH, B_TR, PART>(st, kk + 1, wm, wn, a[(kk + 1) & 1],
                                                b[(kk + 1) & 1], ib);
            __builtin_amdgcn_sched_barrier(0);
            mma_step<C, PART>(a[kk & 1], b[kk & 1], acc, ib);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    wait_lds();
    wg_barrier();
}

// rows: real rows of the tile; a wave of a ragged tail skips its padding blocks'
// reads and MFMAs and keeps every barrier.
template <class C, int DEPTH, int NST, bool B_TR, int CPS, class Copy>
__device__ __forceinline__ void ring_loop(uint32_t lds, int nsteps, f32x16_t (&acc)[C::FM][C::FN],
                                          Copy copy, int rows)
{
    static_assert((NST & (NST - 1)) == 0 && NST >= 2 && NST <= 4, "2 or 4 stages");
    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int ib = __builtin_amdgcn_readfirstlane(
        min(C::FM, max(0, (rows - wm * C::TM + 31) / 32)));
    if (ib == C::FM)
        ring_loop_body<C, DEPTH, NST, B_TR, CPS, false>(lds, nsteps, acc, copy, wm, wn, ib);
    else
        ring_loop_body<C, DEPTH, NST, B_TR, CPS, true>(lds, nsteps, acc, copy, wm, wn, ib);
}

}  // namespace moegg
