// The gated feed-forward block's forward in bf16, gfx950 (moegg_gated_fwd): gelu.
#include "block_fwd.h"

namespace moegg {

using GatedBigCfg = RingCfg<256, 256, 4, 2, false, 64, 2>;
using GatedMidCfg = RingCfg<128, 128, 2, 2, false, 64, 2>;
using GatedDeepCfg = RingCfg<128, 128, 2, 2, false, 64, 4>;
using GatedSmallCfg = RingCfg<32, 256, 1, 4, false, 64, 4>;

template <int ACT, int KEEP, bool TAIL>
static void gated_rows(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const Shape shape = tile_shape(p.S, p.E, p.N, GatedSmallCfg::BN, 0.75, cus);
    if (shape == kSmallTiles)
        block_fwd_cfg<GatedSmallCfg, ACT, KEEP, TAIL>(p, cus, stream);
    else if (shape == kMidTiles)
        block_fwd_cfg<GatedMidCfg, ACT, KEEP, TAIL>(p, cus, stream);
    else if (shape == kDeepTiles)
        block_fwd_cfg<GatedDeepCfg, ACT, KEEP, TAIL>(p, cus, stream);
    else
        block_fwd_cfg<GatedBigCfg, ACT, KEEP, TAIL>(p, cus, stream);
}

template <int ACT, bool TAIL>
static void gated_keep(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.Aq)
        gated_rows<ACT, kKeepPacked, TAIL>(p, cus, stream);
    else if (p.A)
        gated_rows<ACT, kKeepBf16, TAIL>(p, cus, stream);
    else
        gated_rows<ACT, kKeepNone, TAIL>(p, cus, stream);
}

void gated_fwd_gelu(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.N / 2 % 8)
        gated_keep<kGelu, true>(p, cus, stream);
    else
        gated_keep<kGelu, false>(p, cus, stream);
}

}  // namespace moegg
