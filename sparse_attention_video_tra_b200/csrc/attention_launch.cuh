// attention_launch.cuh -- launches of the attention kernel: the instance by
// (head dim, tile width, output type, spatial metric), with or without the
// rows' log-sum-exp.
#pragma once
#include "tra_host.cuh"
#include "attention.cuh"

namespace {

template <int D, int TWL, bool OB, bool DISK, bool LSE, bool SPAN, bool LONE>
tra_status launch_attention(const tra::Geom& G, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const uint8_t* mask, void* out, const void* qraw, float* lse, const tra::Span& span, int ctas,
                            cudaStream_t st)
{
    using C = tra::AttnCfg<D>;
    constexpr auto kern = tra::attention_kernel<D, TWL, OB, DISK, LSE, SPAN, LONE>;
    const int smem = tra::attn_smem_bytes<D>(G.list_cap, G.rte, G.tiles_per_frame);
    if (smem > kMaxSmem) return TRA_ERR_UNSUPPORTED;
    if (!allow_max_smem<kern>()) return TRA_ERR_CUDA;
    if (LONE && span.parts > 1) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        cfg.gridDim = dim3(ctas, G.G);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)span.parts;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (!cuda_ok(cudaLaunchKernelEx(&cfg, kern, q, k, v, G, mask, out, qraw, lse, span))) return TRA_ERR_CUDA;
    } else {
        kern<<<dim3(ctas, G.G), C::THREADS, smem, st>>>(q, k, v, G, mask, out, qraw, lse, span);
    }
    return launch_status();
}

template <int D, int TWL, bool OB, bool DISK, bool LSE, bool SPAN>
tra_status run_attention(const tra::Geom& G, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const uint8_t* mask, void* out, const void* qraw, float* lse, const tra::Span& span, cudaStream_t st)
{
    const int nq = SPAN ? span.nq : G.T, tiles = nq * G.tiles_per_frame;
    if constexpr (LSE) {
        const long long all = (long long)tiles * G.G;
        if (all <= kSMs) {
            // more than eight key tiles: both chains, and two or four CTAs per tile where they
            // all run at once and have eight key tiles or more each
            tra::Span sp = span;
            sp.parts = G.list_cap > 8 ? 1 : 0;
            while (sp.parts && sp.parts < 4 && all * 2 * sp.parts <= kSMs && G.list_cap >= 16 * sp.parts) sp.parts *= 2;
            return launch_attention<D, TWL, OB, DISK, LSE, SPAN, true>(G, q, k, v, mask, out, qraw, lse, sp, tiles * std::max(1, sp.parts), st);
        }
    }
    // two query tiles per CTA; with radius-sorted groups, the same slot of
    // frames 2f and 2f + 1, then an odd last frame's slots two by two
    const int ctas = G.qsort ? nq / 2 * G.tiles_per_frame + (nq % 2) * ((G.tiles_per_frame + 1) / 2) : (tiles + 1) / 2;
    return launch_attention<D, TWL, OB, DISK, LSE, SPAN, false>(G, q, k, v, mask, out, qraw, lse, span, ctas, st);
}

template <int D, int TWL, bool LSE, bool SPAN>
tra_status attention_variant(const tra::Geom& G, bool ob, bool disk, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, const uint8_t* m, void* out, const void* qr, float* lse,
                             const tra::Span& span, cudaStream_t st)
{
    if (ob) return disk ? run_attention<D, TWL, true, true, LSE, SPAN>(G, q, k, v, m, out, qr, lse, span, st)
                        : run_attention<D, TWL, true, false, LSE, SPAN>(G, q, k, v, m, out, qr, lse, span, st);
    return disk ? run_attention<D, TWL, false, true, LSE, SPAN>(G, q, k, v, m, out, qr, lse, span, st)
                : run_attention<D, TWL, false, false, LSE, SPAN>(G, q, k, v, m, out, qr, lse, span, st);
}

// kernel instance by (head dim, tile width, output type, spatial metric)
template <bool LSE, bool SPAN>
tra_status dispatch_attention(const tra::Geom& G, bool ob, bool disk, const CUtensorMap& q, const CUtensorMap& k,
                              const CUtensorMap& v, const uint8_t* m, void* out, const void* qr, float* lse,
                             const tra::Span& span, cudaStream_t st)
{
    switch (G.D * 100 + G.tw_log2) {
        case 6402: return attention_variant<64, 2, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 6403: return attention_variant<64, 3, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 6404: return attention_variant<64, 4, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 6405: return attention_variant<64, 5, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 12802: return attention_variant<128, 2, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 12803: return attention_variant<128, 3, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 12804: return attention_variant<128, 4, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
        case 12805: return attention_variant<128, 5, LSE, SPAN>(G, ob, disk, q, k, v, m, out, qr, lse, span, st);
    }
    return TRA_ERR_UNSUPPORTED;
}

}  // namespace
