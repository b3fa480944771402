// decode_blocks.cu -- the listed-blocks instantiations of the phase-1 kernel
// (decode_mma.cuh, kModeBlocks): attention over selected blocks of a cache.
// Bound by latency for one sequence: 64 blocks of 64 tokens x 8 heads (4.7 MB)
// take 7.5 us with their reduce.  By instruction issue, and the start and end
// of CTAs of five tiles, for a batch: 32 blocks of each of 32 sequences (75 MB)
// 27.7 us, 2.7 TB/s.
#include "decode_mma.cuh"

namespace tq {

namespace {

template <int D, int BITS>
cudaError_t launch_blocks_d(const DecodeParams& p, cudaStream_t stream) {
    const CUtensorMap none{};  // the rows are fetched without tensor maps
    const int out = p.out == nullptr ? kOutParts : (p.n_splits == 1 ? kOutDirect : kOutCluster);
    if (out == kOutCluster && p.n_splits > kMaxClusterRuns) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = phase1_config(p, out, stream, true, attr);
    if (p.map.block_table != nullptr) return launch_out<D, true, BITS, false, kModeBlocks>(cfg, p, none, none, out);
    return launch_out<D, false, BITS, false, kModeBlocks>(cfg, p, none, none, out);
}

}  // namespace

cudaError_t launch_decode_blocks(const DecodeParams& p, int head_dim, cudaStream_t stream) {
    if (p.bits == 8) {
        if (head_dim == 64) return launch_blocks_d<64, 8>(p, stream);
        if (head_dim == 128) return launch_blocks_d<128, 8>(p, stream);
        if (head_dim == 256) return launch_blocks_d<256, 8>(p, stream);
    } else {
        if (head_dim == 64) return launch_blocks_d<64, 4>(p, stream);
        if (head_dim == 128) return launch_blocks_d<128, 4>(p, stream);
        if (head_dim == 256) return launch_blocks_d<256, 4>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tq
