// tra_cache.cu -- the extern "C" entry points over keys and values held in 8
// bits: storing frames, and attention of whole frames and of single tokens.
#include "attention_launch.cuh"
#include "cache.cuh"

bool tra_cache_take_error(unsigned int& word) { return take_error_word(word); }

namespace {

tra_cache_info cache_layout(const tra::Geom& G)
{
    tra_cache_info L;
    const size_t codes = (size_t)G.G * G.N_pad * G.D, scales = (size_t)G.G * G.nQ * sizeof(float);
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    L.off_k = 0;
    L.off_v = up(codes);
    L.off_k_scale = L.off_v + up(codes);
    L.off_v_scale = L.off_k_scale + up(scales);
    L.cache_bytes = L.off_v_scale + up(scales);
    return L;
}

tra::CacheView cache_view(const tra::Geom& G, const void* cache)
{
    const tra_cache_info L = cache_layout(G);
    uint8_t* c = (uint8_t*)cache;
    return {c + L.off_k, c + L.off_v, (float*)(c + L.off_k_scale), (float*)(c + L.off_v_scale)};
}

// the key frames that the queries of [frame, frame + n) can reach and the cache holds
tra::Span call_span(const tra::Geom& G, int frame, int n, int cached)
{
    tra::Span s = {frame, n, std::max(0, frame - G.rte), std::min(cached, std::min(G.T, frame + n + G.rte)), 0};
    if (s.k1 <= s.k0) s.k0 = s.k1 = 0;
    return s;
}

// bytes of K (and of V) expanded for a window of `frames` key frames
size_t window_bytes(const tra::Geom& G, int frames) { return (size_t)G.G * frames * G.tiles_per_frame * 128 * G.D * 2; }

bool frames_ok(const tra::Geom& G, int frame, int n) { return frame >= 0 && n >= 1 && n <= G.T && frame <= G.T - n; }

}  // namespace

extern "C" tra_status tra_cache_query(tra_plan plan, tra_cache_info* info)
{
    if (!plan || !info) return TRA_ERR_INVALID_ARG;
    *info = cache_layout(plan->geom);
    return TRA_OK;
}

extern "C" tra_status tra_cache_store(tra_plan plan, const void* k, const void* v, int frame, int n_frames, void* cache,
                                      size_t cache_bytes, tra_stream stream)
{
    if (!plan || !k || !v || !cache || !aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 256))
        return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    if (!frames_ok(G, frame, n_frames)) return TRA_ERR_INVALID_ARG;
    if (cache_bytes < cache_layout(G).cache_bytes) return TRA_ERR_WORKSPACE;
    const dim3 grid(n_frames * G.tiles_per_frame, G.G, 2);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, (cudaStream_t)stream>>>(G, (const uint4*)k, (const uint4*)v, frame, n_frames, cache_view(G, cache));
    };
    G.D == 64 ? go(tra::cache_store_kernel<64>) : go(tra::cache_store_kernel<128>);
    return launch_status();
}

extern "C" tra_status tra_cache_attention_bytes(tra_plan plan, int n_frames, size_t* bytes)
{
    if (!plan || !bytes) return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    if (n_frames < 1 || n_frames > G.T) return TRA_ERR_INVALID_ARG;
    *bytes = 2 * window_bytes(G, std::min(G.T, n_frames + 2 * G.rte));
    return TRA_OK;
}

extern "C" tra_status tra_cache_attention(tra_plan plan, const void* q, int frame, int n_frames, const void* cache,
                                          size_t cache_bytes, int cached_frames, const void* mask, void* out, float* lse,
                                          void* workspace, size_t workspace_bytes, tra_stream stream)
{
    if (!plan || !q || !cache || !mask || !out || !lse || !workspace) return TRA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 256) || !aligned(mask, 256) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(workspace, 256))
        return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    if (!frames_ok(G, frame, n_frames) || cached_frames < 0 || cached_frames > G.T) return TRA_ERR_INVALID_ARG;
    const tra::Span span = call_span(G, frame, n_frames, cached_frames);
    const int window = std::max(1, span.k1 - span.k0);
    if (cache_bytes < cache_layout(G).cache_bytes || workspace_bytes < 2 * window_bytes(G, window)) return TRA_ERR_WORKSPACE;

    uint8_t* kw = (uint8_t*)workspace;
    uint8_t* vw = kw + window_bytes(G, window);
    tra::Geom GQ = G;                                        // the query rows as a grid of n_frames frames
    GQ.T = n_frames;
    GQ.N_pad = n_frames * G.tiles_per_frame * 128;
    const uint64_t rows = (uint64_t)G.G * window * G.tiles_per_frame * 128;
    CUtensorMap mq, mk, mv;
    if (!make_input_map(&mq, q, GQ) || !make_row_map(&mk, kw, rows, G.D) || !make_row_map(&mv, vw, rows, G.D))
        return TRA_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    if (span.k1 > span.k0) {
        const size_t chunks = rows * (G.D / 16);
        const dim3 grid((unsigned)std::min<size_t>((chunks + 255) / 256, 148 * 16), 2);
        auto go = [&](auto kern) { kern<<<grid, 256, 0, st>>>(G, cache_view(G, cache), span.k0, span.k1, (uint4*)kw, (uint4*)vw); };
        G.D == 64 ? go(tra::cache_expand_kernel<64>) : go(tra::cache_expand_kernel<128>);
        if (launch_status() != TRA_OK) return TRA_ERR_CUDA;
    }
    return dispatch_attention<true, true>(G, (plan->flags & TRA_FLAG_OUT_BF16) != 0, G.disk != 0, mq, mk, mv,
                                          (const uint8_t*)mask, out, q, lse, span, st);
}

extern "C" tra_status tra_cache_attention_tokens(tra_plan plan, const void* q, const int32_t* token, const int32_t* radius,
                                                 int n, const void* cache, size_t cache_bytes, int cached_frames, void* out,
                                                 float* lse, tra_stream stream)
{
    if (!plan || n < 0) return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    if (cached_frames < 0 || cached_frames > G.T) return TRA_ERR_INVALID_ARG;
    if (n == 0) return TRA_OK;
    if (!q || !token || !radius || !cache || !out || !lse) return TRA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(token, 4) || !aligned(radius, 4) || !aligned(cache, 256) || !aligned(out, 16) ||
        !aligned(lse, 4))
        return TRA_ERR_INVALID_ARG;
    if (cache_bytes < cache_layout(G).cache_bytes) return TRA_ERR_WORKSPACE;
    const long long units = (long long)n * G.G;
    if (units > (1ll << 31) - 1) return TRA_ERR_UNSUPPORTED;
    // Groups of 16 tokens share a key's codes on the tensor cores once enough of a
    // group's rows are filled and there is work for the card; below, one token at
    // a time over more CTAs.  Measured cold on neighbouring tokens, one token at a
    // time / grouped: with 40 heads at 21 x 45 x 80 86 / 98 us for 6 tokens,
    // 169 / 109 for 8 and 160 / 110 for 16; with 12 heads at 21 x 30 x 52 33 / 30 us
    // for 8 and 49 / 35 for 16.  With few heads: 4 at 21 x 45 x 80 43 / 51 us for 16,
    // 50 / 51 for 24, 62 / 48 for 48; 2 at 21 x 30 x 52 26 / 31 us for 32, 33 / 35 for
    // 48, 31 / 31 for 64; 4 at 9 x 17 x 23 18 / 18 us for 16 to 32, 22 / 20 for 64.
    // (Tokens scattered over the clip share few keys and are faster one at a time,
    // 168 against 293 us for 64 of 12 heads, but where they lie is known on the
    // device only.)
    const bool grouped = n >= 8 && units >= 96;
    const long long work = grouped ? (long long)((n + tra::GROUP - 1) / tra::GROUP) * G.G : units;
    // CTAs per group or token and head, a cluster.  Groups run one CTA per SM: the
    // most that all run at once, counting that a cluster lies within one GPC and
    // large ones leave SMs over (24 clusters of 5: 47 us, of 6: 57 us; 48 of
    // 3: 74 us, of 4: 82 us).  Lone tokens: as many as stay resident together, 16
    // (a quarter faster for 1 token and 12 heads) while they cost no other its place.
    int csize = 8;
    if (grouped) {
        while (csize > 2 && work * csize > (csize > 4 ? 128 : 144)) --csize;
    } else {
        while (csize > 1 && work * csize > 148 * 4) csize /= 2;
        if (work * 16 <= 148 * 2) csize = 16;
    }
    if (work * csize > (1ll << 31) - 1) return TRA_ERR_UNSUPPORTED;

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    cfg.gridDim = dim3((unsigned)(work * csize));
    cfg.blockDim = dim3(grouped ? 32 * tra::GROUP_WARPS : 256);
    cfg.stream = (cudaStream_t)stream;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)csize;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int bf16 = (plan->flags & TRA_FLAG_OUT_BF16) != 0 ? 1 : 0;
    cfg.dynamicSmemBytes = !grouped ? 0 : G.D == 64 ? tra::group_smem_bytes<64>() : tra::group_smem_bytes<128>();
    auto go = [&](auto one, auto many) {
        if (grouped && !set_smem(many, (int)cfg.dynamicSmemBytes)) return false;
        if (csize > 8 && !cuda_ok(cudaFuncSetAttribute(one, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))) return false;
        return cuda_ok(grouped ? cudaLaunchKernelEx(&cfg, many, G, cache_view(G, cache), (const uint32_t*)q, token, radius, n,
                                                    cached_frames, csize, out, bf16, lse)
                               : cudaLaunchKernelEx(&cfg, one, G, cache_view(G, cache), (const uint4*)q, token, radius, n,
                                                    cached_frames, csize, out, bf16, lse));
    };
    bool ok;
    if (G.D == 64) ok = G.disk ? go(tra::token_attention_kernel<64, true>, tra::token_group_kernel<64, true>)
                               : go(tra::token_attention_kernel<64, false>, tra::token_group_kernel<64, false>);
    else ok = G.disk ? go(tra::token_attention_kernel<128, true>, tra::token_group_kernel<128, true>)
                     : go(tra::token_attention_kernel<128, false>, tra::token_group_kernel<128, false>);
    return ok ? launch_status() : TRA_ERR_CUDA;
}
