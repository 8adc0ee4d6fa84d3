// Grouped products of 8-bit integers, gfx950 (moegg_grouped_gemm_i8).
#include "block_fwd.h"

namespace moegg {

using I8BigCfg = RingCfg<256, 256, 2, 4, true, 64, 2>;
using I8MidCfg = RingCfg<128, 128, 2, 2, true, 64, 2>;
using I8DeepCfg = RingCfg<128, 128, 2, 2, true, 64, 4>;
using I8SmallCfg = RingCfg<32, 128, 1, 4, true, 64, 4>;
using I8SmallGatedCfg = RingCfg<32, 256, 1, 4, true, 64, 4>;

template <int ACT, bool TAIL>
static void i8_rows(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    using Small = std::conditional_t<ACT == kPlain, I8SmallCfg, I8SmallGatedCfg>;
    const Shape shape = tile_shape(p.S, p.E, p.N, Small::BN, 0.75, cus);
    if (shape == kSmallTiles)
        block_fwd_cfg<Small, ACT, kKeepNone, TAIL>(p, cus, stream);
    else if (shape == kMidTiles)
        block_fwd_cfg<I8MidCfg, ACT, kKeepNone, TAIL>(p, cus, stream);
    else if (shape == kDeepTiles)
        block_fwd_cfg<I8DeepCfg, ACT, kKeepNone, TAIL>(p, cus, stream);
    else
        block_fwd_cfg<I8BigCfg, ACT, kKeepNone, TAIL>(p, cus, stream);
}

template <bool TAIL>
static void i8_tail(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.flags & MOEGG_GATED_SILU)
        i8_rows<kSilu, TAIL>(p, cus, stream);
    else if (p.flags & MOEGG_GATED_GELU)
        i8_rows<kGelu, TAIL>(p, cus, stream);
    else
        i8_rows<kPlain, TAIL>(p, cus, stream);
}

hipError_t i8_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (block_vec_pays(p, cus))
        return block_vec_launch(p, cus, stream);
    const int cols = p.flags & (MOEGG_GATED_SILU | MOEGG_GATED_GELU) ? p.N / 2 : p.N;
    if (cols % 8)
        i8_tail<true>(p, cus, stream);
    else
        i8_tail<false>(p, cus, stream);
    return hipGetLastError();
}

}  // namespace moegg
