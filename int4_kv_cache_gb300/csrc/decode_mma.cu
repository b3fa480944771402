// decode_mma.cu -- the decode's phase-1 instantiations (decode_mma.cuh): every
// (head_dim, code width, layout, output) pair, their launch and occupancy.
#include "decode_mma.cuh"

namespace tq {

namespace {

// p.out set: the kernel writes the output itself, one run per sequence
// (n_splits = 1) or the runs of each (sequence, kv head) as one cluster.
template <int D, int BITS>
cudaError_t launch_d(const DecodeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream,
                     bool pdl_secondary) {
    const bool paged = p.map.block_table != nullptr;
    const int out = p.out == nullptr ? kOutParts : (p.n_splits == 1 ? kOutDirect : kOutCluster);
    if (out == kOutCluster && p.n_splits > kMaxClusterRuns) return cudaErrorInvalidValue;
    if (p.wide && !wide_ok(D, BITS, paged)) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = phase1_config(p, out, stream, pdl_secondary, attr);
    if (paged) return launch_out<D, true, BITS, false>(cfg, p, tm_k, tm_v, out);
    if constexpr (wide_ok(D, BITS, false)) {
        if (p.wide) return launch_out<D, false, BITS, true>(cfg, p, tm_k, tm_v, out);
    }
    return launch_out<D, false, BITS, false>(cfg, p, tm_k, tm_v, out);
}

// Clusters of n CTAs of the cluster-merging instantiation the device holds at
// once (0 if it cannot place one).
template <int D, bool PAGED, int BITS, bool WIDE>
int max_clusters_d(int n) {
    using C = Cfg<D, BITS, WIDE>;
    if (set_smem_attr<D, PAGED, BITS, kOutCluster, WIDE>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned int>(n), 1, 1);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = static_cast<unsigned int>(n);
    a[0].val.clusterDim.y = 1;
    a[0].val.clusterDim.z = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, decode_mma_kernel<D, PAGED, BITS, kOutCluster, WIDE>, &cfg) !=
        cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return clusters;
}

template <int D, bool PAGED, int BITS, bool WIDE>
int ctas_per_sm_d() {
    using C = Cfg<D, BITS, WIDE>;
    if (set_smem_attr<D, PAGED, BITS, kOutParts, WIDE>() != cudaSuccess) return 1;
    int n = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_mma_kernel<D, PAGED, BITS, kOutParts, WIDE>, C::THREADS,
                                                  C::SMEM_BYTES);
    return n > 0 ? n : 1;
}

}  // namespace

// (head_dim, bits) pairs with a kernel: int4 at 64 / 128 / 256, int8 at 64 / 128
// (an int8 row of 256 would not fit one 128-byte swizzle row).
bool mma_supported(int head_dim, int bits) {
    return (bits == 4 || bits == 8) && (head_dim == 64 || head_dim == 128 || head_dim == 256);
}

#define TQ_DISPATCH(EXPR64_4, EXPR128_4, EXPR256_4, EXPR64_8, EXPR128_8, EXPR256_8, FALLBACK) \
    if (bits == 8) {                                                              \
        if (head_dim == 64) return EXPR64_8;                                      \
        if (head_dim == 128) return EXPR128_8;                                    \
        if (head_dim == 256) return EXPR256_8;                                    \
    } else {                                                                      \
        if (head_dim == 64) return EXPR64_4;                                      \
        if (head_dim == 128) return EXPR128_4;                                    \
        if (head_dim == 256) return EXPR256_4;                                    \
    }                                                                             \
    return FALLBACK;

int mma_tile_tokens(int head_dim, int bits, bool wide) {
    if (wide) return head_dim == 128 && bits == 4 ? Cfg<128, 4, true>::T : 0;
    TQ_DISPATCH(Cfg<64>::T, Cfg<128>::T, Cfg<256>::T, (Cfg<64, 8>::T), (Cfg<128, 8>::T), (Cfg<256, 8>::T), 0)
}

int mma_smem_bytes(int head_dim, int bits, bool wide) {
    if (wide) return head_dim == 128 && bits == 4 ? Cfg<128, 4, true>::SMEM_BYTES : 0;
    TQ_DISPATCH(Cfg<64>::SMEM_BYTES, Cfg<128>::SMEM_BYTES, Cfg<256>::SMEM_BYTES, (Cfg<64, 8>::SMEM_BYTES),
                (Cfg<128, 8>::SMEM_BYTES), (Cfg<256, 8>::SMEM_BYTES), 0)
}

bool mma_wide_supported(int head_dim, int bits, bool paged) { return wide_ok(head_dim, bits, paged); }

int mma_max_active_clusters(int head_dim, int bits, bool paged, bool wide, int n) {
    if (n < 2 || n > kMaxClusterRuns) return 0;
    if (wide) return wide_ok(head_dim, bits, paged) ? max_clusters_d<128, false, 4, true>(n) : 0;
    if (paged) {
        TQ_DISPATCH((max_clusters_d<64, true, 4, false>(n)), (max_clusters_d<128, true, 4, false>(n)),
                    (max_clusters_d<256, true, 4, false>(n)), (max_clusters_d<64, true, 8, false>(n)),
                    (max_clusters_d<128, true, 8, false>(n)), (max_clusters_d<256, true, 8, false>(n)), 0)
    }
    TQ_DISPATCH((max_clusters_d<64, false, 4, false>(n)), (max_clusters_d<128, false, 4, false>(n)),
                (max_clusters_d<256, false, 4, false>(n)), (max_clusters_d<64, false, 8, false>(n)),
                (max_clusters_d<128, false, 8, false>(n)), (max_clusters_d<256, false, 8, false>(n)), 0)
}

int mma_ctas_per_sm(int head_dim, int bits, bool wide) {
    if (wide) return head_dim == 128 && bits == 4 ? ctas_per_sm_d<128, false, 4, true>() : 1;
    TQ_DISPATCH((ctas_per_sm_d<64, false, 4, false>()), (ctas_per_sm_d<128, false, 4, false>()),
                (ctas_per_sm_d<256, false, 4, false>()), (ctas_per_sm_d<64, false, 8, false>()),
                (ctas_per_sm_d<128, false, 8, false>()), (ctas_per_sm_d<256, false, 8, false>()), 1)
}

cudaError_t launch_decode_mma(const DecodeParams& p, int head_dim, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                              cudaStream_t stream, bool pdl_secondary) {
    const int bits = p.bits;
    TQ_DISPATCH((launch_d<64, 4>(p, tm_k, tm_v, stream, pdl_secondary)),
                (launch_d<128, 4>(p, tm_k, tm_v, stream, pdl_secondary)),
                (launch_d<256, 4>(p, tm_k, tm_v, stream, pdl_secondary)),
                (launch_d<64, 8>(p, tm_k, tm_v, stream, pdl_secondary)),
                (launch_d<128, 8>(p, tm_k, tm_v, stream, pdl_secondary)),
                (launch_d<256, 8>(p, tm_k, tm_v, stream, pdl_secondary)), cudaErrorInvalidValue)
}

#undef TQ_DISPATCH

}  // namespace tq
