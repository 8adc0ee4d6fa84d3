// Grouped products of 8-bit integers, gfx950 (moegg_grouped_gemm_i8).
#include "block_fwd.h"

namespace moegg {

// Tile shapes: many rows per expert, and few (the weights are then streamed
// once per 32-row tile).
using I8BigCfg = Cfg<256, 256, 2, 4, true, true>;
using I8SmallCfg = Cfg<32, 128, 1, 4, true, true>;
using I8SmallGatedCfg = Cfg<32, 256, 1, 4, true, true>;

template <bool TAIL>
static void i8_tail(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const bool small = p.S / p.E < kBlockSmallRows;
    if (p.flags & (MOEGG_GATED_SILU | MOEGG_GATED_GELU)) {
        if (small)
            block_fwd_cfg<I8SmallGatedCfg, true, kKeepNone, TAIL>(p, cus, stream);
        else
            block_fwd_cfg<I8BigCfg, true, kKeepNone, TAIL>(p, cus, stream);
    } else {
        if (small)
            block_fwd_cfg<I8SmallCfg, false, kKeepNone, TAIL>(p, cus, stream);
        else
            block_fwd_cfg<I8BigCfg, false, kKeepNone, TAIL>(p, cus, stream);
    }
}

hipError_t i8_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const int cols = p.flags & (MOEGG_GATED_SILU | MOEGG_GATED_GELU) ? p.N / 2 : p.N;
    if (cols % 8)
        i8_tail<true>(p, cus, stream);
    else
        i8_tail<false>(p, cus, stream);
    return hipGetLastError();
}

}  // namespace moegg
