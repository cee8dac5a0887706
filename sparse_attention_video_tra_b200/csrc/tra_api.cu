// tra_api.cu -- the extern "C" entry points of the inference path: argument
// checks, TMA tensor maps, kernel selection by (head dim, tile width), and the
// device error word.
#include "tra_host.cuh"
#include "permute.cuh"
#include "radius_mask.cuh"
#include "entropy.cuh"
#include "attention_launch.cuh"
#include "topk.cuh"

namespace {

template <int D, int TWL>
tra_status run_entropy(const tra::Geom& G, const CUtensorMap& q, const CUtensorMap& k, int stride, float corr,
                       float* H, cudaStream_t st)
{
    using C = tra::EntCfg<D>;
    auto kern = tra::entropy_kernel<D, TWL>;
    if (!set_smem(kern, C::SMEM)) return TRA_ERR_CUDA;
    kern<<<dim3((G.nQ + 1) / 2, G.G), C::THREADS, C::SMEM, st>>>(q, k, G, stride, corr, H);
    return launch_status();
}

template <int D, int TWL>
tra_status run_topk(const tra::Geom& G, const CUtensorMap& q, const CUtensorMap& k, int stride, int n_sample,
                    float mass, float* H, int* K, cudaStream_t st)
{
    using C = tra::TopkCfg<D>;
    auto kern = tra::topk_kernel<D, TWL>;
    if (!set_smem(kern, C::SMEM)) return TRA_ERR_CUDA;
    kern<<<dim3(n_sample, G.G), C::THREADS, C::SMEM, st>>>(q, k, G, stride, n_sample, mass, H, K);
    return launch_status();
}

}  // namespace

extern "C" tra_status tra_permute(tra_plan plan, const void* src, void* dst, int to_tile_major, int elem_bytes,
                                  tra_stream stream)
{
    if (!plan || !src || !dst || !aligned(src, 16) || !aligned(dst, 16)) return TRA_ERR_INVALID_ARG;
    if (elem_bytes != 2 && elem_bytes != 4) return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    const size_t total = (size_t)G.G * G.N_pad * (G.D * elem_bytes / 16);
    const int blocks = (int)std::min<size_t>((total + 255) / 256, 148 * 32);
    tra::permute_kernel<<<blocks, 256, 0, (cudaStream_t)stream>>>(G, (const uint4*)src, (uint4*)dst,
                                                                   to_tile_major ? 1 : 0, elem_bytes);
    return launch_status();
}

extern "C" tra_status tra_entropy(tra_plan plan, const void* q, const void* k, float* Hout, int key_tile_stride,
                                  tra_stream stream)
{
    if (!plan || !q || !k || !Hout || !aligned(q, 16) || !aligned(k, 16) || !aligned(Hout, 4))
        return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    if (key_tile_stride < 1 || key_tile_stride > G.nQ) return TRA_ERR_INVALID_ARG;
    // |S| = valid keys in the sampled tiles; corr = ln(N / |S|)
    float corr = 0.f;
    if (key_tile_stride > 1) {
        long long nS = 0;
        for (int kb = 0; kb < G.nQ; kb += key_tile_stride) {
            const int rem = kb % G.tiles_per_frame;
            const int tr = rem / G.nTw, tc = rem % G.nTw;
            nS += (long long)std::min(G.th, G.H - tr * G.th) * std::min(G.tw, G.W - tc * G.tw);
        }
        corr = (float)std::log((double)G.N / (double)nS);
    }
    CUtensorMap mq, mk;
    if (!make_input_map(&mq, q, G) || !make_input_map(&mk, k, G)) return TRA_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const int key = G.D * 100 + G.tw_log2;
    switch (key) {
        case 6402: return run_entropy<64, 2>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 6403: return run_entropy<64, 3>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 6404: return run_entropy<64, 4>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 6405: return run_entropy<64, 5>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 12802: return run_entropy<128, 2>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 12803: return run_entropy<128, 3>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 12804: return run_entropy<128, 4>(G, mq, mk, key_tile_stride, corr, Hout, st);
        case 12805: return run_entropy<128, 5>(G, mq, mk, key_tile_stride, corr, Hout, st);
    }
    return TRA_ERR_UNSUPPORTED;
}

extern "C" tra_status tra_radius_and_mask(tra_plan plan, const float* Hent, void* mask, size_t mask_bytes,
                                          tra_stream stream)
{
    if (!plan || !Hent || !mask || !aligned(Hent, 4) || !aligned(mask, 256)) return TRA_ERR_INVALID_ARG;
    if (mask_bytes < plan->mask_bytes) return TRA_ERR_WORKSPACE;
    tra::Geom G = plan->geom;
    // one CTA per tile-column strip (query groups) or per tile
    const int U = G.qsort ? G.nTh : 1;
    const dim3 grid(G.qsort ? G.T * G.nTw : G.nQ, G.G);
    int smem = tra::mask_smem_bytes(G.rte, G.nTh, G.r_cap, G.hw_tab != 0, G.disk_smax, U);
    if (G.disk_smax >= 0 && smem > kMaxSmem - 16 * 1024) {
        // no room for the disk-row table: count the disk row by row
        G.disk_smax = -1;
        smem = tra::mask_smem_bytes(G.rte, G.nTh, G.r_cap, G.hw_tab != 0, G.disk_smax, U);
    }
    if (smem > kMaxSmem - 16 * 1024) return TRA_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t* m = (uint8_t*)mask;
    auto go = [&](auto kern) -> bool {
        if (smem > 48 * 1024 && !set_smem(kern, smem)) return false;
        kern<<<grid, 128 * U, smem, st>>>(G, Hent, m);
        return true;
    };
    bool ok;
    if (!G.qsort) ok = G.disk ? go(tra::radius_mask_kernel<true, false, 128>) : go(tra::radius_mask_kernel<false, false, 128>);
    else if (U <= 3) ok = G.disk ? go(tra::radius_mask_kernel<true, true, 384>) : go(tra::radius_mask_kernel<false, true, 384>);
    else ok = G.disk ? go(tra::radius_mask_kernel<true, true, 512>) : go(tra::radius_mask_kernel<false, true, 512>);
    if (!ok) return TRA_ERR_CUDA;
    return launch_status();
}

extern "C" tra_status tra_attention(tra_plan plan, const void* q, const void* k, const void* v, const void* mask,
                                    void* out, tra_stream stream)
{
    if (!plan || !q || !k || !v || !mask || !out) return TRA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(mask, 256))
        return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    CUtensorMap mq, mk, mv;
    if (!make_input_map(&mq, q, G) || !make_input_map(&mk, k, G) || !make_input_map(&mv, v, G))
        return TRA_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const uint8_t* m = (const uint8_t*)mask;
    const bool ob = (plan->flags & TRA_FLAG_OUT_BF16) != 0;
    const bool disk = G.disk != 0;
    return dispatch_attention<false, false>(G, ob, disk, mq, mk, mv, m, out, q, nullptr, {}, st);
}

extern "C" tra_status tra_calibrate_topk(tra_plan plan, const void* q, const void* k, double mass,
                                         int query_tile_stride, float* H_out, int* k_out, tra_stream stream)
{
    if (!plan || !q || !k || !H_out || !k_out) return TRA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(H_out, 4) || !aligned(k_out, 4)) return TRA_ERR_INVALID_ARG;
    if (!(mass > 0.0 && mass < 1.0) || query_tile_stride < 1) return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    const int n_sample = (G.nQ + query_tile_stride - 1) / query_tile_stride;
    CUtensorMap mq, mk;
    if (!make_input_map(&mq, q, G) || !make_input_map(&mk, k, G)) return TRA_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const float m = (float)mass;
    switch (G.D * 100 + G.tw_log2) {
        case 6402: return run_topk<64, 2>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 6403: return run_topk<64, 3>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 6404: return run_topk<64, 4>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 6405: return run_topk<64, 5>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 12802: return run_topk<128, 2>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 12803: return run_topk<128, 3>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 12804: return run_topk<128, 4>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
        case 12805: return run_topk<128, 5>(G, mq, mk, query_tile_stride, n_sample, m, H_out, k_out, st);
    }
    return TRA_ERR_UNSUPPORTED;
}

extern "C" tra_status tra_plan_status(tra_plan plan)
{
    (void)plan;
    unsigned int word = 0;
    if (!take_error_word(word) || !tra_grad_take_error(word) || !tra_cache_take_error(word)) return TRA_ERR_CUDA;
    if (word & TRA_ERRBIT_TIMEOUT) return TRA_ERR_TIMEOUT;
    if (word & TRA_ERRBIT_CHECK) return TRA_ERR_DEVICE_CHECK;
    return TRA_OK;
}
