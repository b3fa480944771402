// decode_scores.cu -- the score-keeping instantiations of the phase-1 kernel
// (decode_mma.cuh, kModeScores): partial states plus every scaled score, for
// the decode that accumulates attention weights.  Bound as the decode is, by
// instruction issue, with one operation more per operand word and the stores of
// the scores: 131,072 tokens of 64 heads (151 MB read, 33.5 MB written) take 33
// to 35 us where the decode's phase 1 takes 29.
#include "decode_mma.cuh"

namespace tq {

namespace {

template <int D, int BITS>
cudaError_t launch_scores_d(const DecodeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                            cudaStream_t stream) {
    const bool paged = p.map.block_table != nullptr;
    if (p.wide && !wide_ok(D, BITS, paged)) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = phase1_config(p, kOutParts, stream, true, attr);
    if (paged) return launch_mode<D, true, BITS, kOutParts, false, kModeScores>(cfg, p, tm_k, tm_v);
    if constexpr (wide_ok(D, BITS, false)) {
        if (p.wide) return launch_mode<D, false, BITS, kOutParts, true, kModeScores>(cfg, p, tm_k, tm_v);
    }
    return launch_mode<D, false, BITS, kOutParts, false, kModeScores>(cfg, p, tm_k, tm_v);
}

}  // namespace

cudaError_t launch_decode_scores(const DecodeParams& p, int head_dim, const CUtensorMap& tm_k,
                                 const CUtensorMap& tm_v, cudaStream_t stream) {
    if (p.bits == 8) {
        if (head_dim == 64) return launch_scores_d<64, 8>(p, tm_k, tm_v, stream);
        if (head_dim == 128) return launch_scores_d<128, 8>(p, tm_k, tm_v, stream);
        if (head_dim == 256) return launch_scores_d<256, 8>(p, tm_k, tm_v, stream);
    } else {
        if (head_dim == 64) return launch_scores_d<64, 4>(p, tm_k, tm_v, stream);
        if (head_dim == 128) return launch_scores_d<128, 4>(p, tm_k, tm_v, stream);
        if (head_dim == 256) return launch_scores_d<256, 4>(p, tm_k, tm_v, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tq
