// The gated feed-forward block's forward in bf16, gfx950 (moegg_gated_fwd).
#include "block_fwd.h"

namespace moegg {

using GatedBigCfg = Cfg<256, 256, 2, 4, true>;
using GatedSmallCfg = Cfg<32, 256, 1, 4, true>;

template <int KEEP, bool TAIL>
static void gated_rows(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.S / p.E < kBlockSmallRows)
        block_fwd_cfg<GatedSmallCfg, true, KEEP, TAIL>(p, cus, stream);
    else
        block_fwd_cfg<GatedBigCfg, true, KEEP, TAIL>(p, cus, stream);
}

template <bool TAIL>
static void gated_tail(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.Aq)
        gated_rows<kKeepPacked, TAIL>(p, cus, stream);
    else if (p.A)
        gated_rows<kKeepBf16, TAIL>(p, cus, stream);
    else
        gated_rows<kKeepNone, TAIL>(p, cus, stream);
}

hipError_t gated_fwd_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.N / 2 % 8)
        gated_tail<true>(p, cus, stream);
    else
        gated_tail<false>(p, cus, stream);
    return hipGetLastError();
}

}  // namespace moegg
