// ragged_tc_fp8.cu -- the tcgen05 kernel of the ragged operators for fp8 pools (ragged_tc.cuh).
#include "ragged_tc.cuh"

namespace pkv {

int launch_ragged_tc_fp8(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
                      const CUtensorMap* tmv, cudaStream_t s)
{
    return ragged::launch_any<PKV_FP8E4M3>(p, d, pair, items, max_rows, tmk, tmv, s);
}

}  // namespace pkv
