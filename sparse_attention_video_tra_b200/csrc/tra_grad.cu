// tra_grad.cu -- the extern "C" entry points a training step uses: attention
// with its rows' log-sum-exp, and the gradients.
#include "attention_launch.cuh"
#include "backward.cuh"

bool tra_grad_take_error(unsigned int& word) { return take_error_word(word); }

extern "C" tra_status tra_attention_lse(tra_plan plan, const void* q, const void* k, const void* v, const void* mask,
                                        void* out, float* lse, tra_stream stream)
{
    if (!plan || !q || !k || !v || !mask || !out || !lse) return TRA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(mask, 256) ||
        !aligned(lse, 4))
        return TRA_ERR_INVALID_ARG;
    const tra::Geom& G = plan->geom;
    CUtensorMap mq, mk, mv;
    if (!make_input_map(&mq, q, G) || !make_input_map(&mk, k, G) || !make_input_map(&mv, v, G))
        return TRA_ERR_CUDA;
    return dispatch_attention<true, false>(G, (plan->flags & TRA_FLAG_OUT_BF16) != 0, G.disk != 0, mq, mk, mv,
                                    (const uint8_t*)mask, out, q, lse, {}, (cudaStream_t)stream);
}

namespace {

// The workspace of tra_attention_backward: row data, the tile bitmaps, and the
// operands in plain row order where the caller's are not: Q, K and V from the
// natural layout, Q with query groups, and dO always (it may be fp32, and its
// tile-major pad rows must be zeros for the products).
struct BwdLayout {
    bool copy_q, copy_kv;                    // dO always has its copy
    int bw;
    size_t off_bits, off_do, off_q, off_k, off_v, total;
};

BwdLayout backward_layout(tra_plan plan)
{
    const tra::Geom& G = plan->geom;
    BwdLayout L;
    L.copy_kv = G.natural != 0;
    L.copy_q = G.natural || G.qsort;
    L.bw = tra::reach_words(G);
    const size_t rows = (size_t)G.G * G.N_pad, tile_rows = rows * G.D * 2;
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    L.off_bits = up(rows * sizeof(float4));
    L.off_do = up(L.off_bits + (size_t)G.G * G.nQ * L.bw * 4);
    L.off_q = up(L.off_do + tile_rows);
    L.off_k = up(L.off_q + (L.copy_q ? tile_rows : 0));
    L.off_v = up(L.off_k + (L.copy_kv ? tile_rows : 0));
    L.total = up(L.off_v + (L.copy_kv ? tile_rows : 0));
    return L;
}

template <int D, int TWL, bool DISK>
tra_status run_backward(const tra::Geom& G, const tra::BwdArgs& A, const CUtensorMap& q, const CUtensorMap& k,
                        const CUtensorMap& v, const CUtensorMap& d, cudaStream_t st)
{
    constexpr auto kern = tra::backward_kernel<D, TWL, DISK>;
    const int smem = std::max(tra::BwdKvCfg<D>::smem(G.list_cap), tra::BwdQCfg<D>::smem());
    if (smem > kMaxSmem) return TRA_ERR_UNSUPPORTED;
    if (!allow_max_smem<kern>()) return TRA_ERR_CUDA;
    kern<<<dim3(G.nQ, G.G, 2), 384, smem, st>>>(q, k, v, d, G, A);
    return launch_status();
}

template <int D, int TWL>
tra_status run_backward(const tra::Geom& G, const tra::BwdArgs& A, const CUtensorMap& q, const CUtensorMap& k,
                        const CUtensorMap& v, const CUtensorMap& d, cudaStream_t st)
{
    return G.disk ? run_backward<D, TWL, true>(G, A, q, k, v, d, st) : run_backward<D, TWL, false>(G, A, q, k, v, d, st);
}

}  // namespace

extern "C" tra_status tra_attention_backward_bytes(tra_plan plan, size_t* bytes)
{
    if (!plan || !bytes) return TRA_ERR_INVALID_ARG;
    *bytes = backward_layout(plan).total;
    return TRA_OK;
}

extern "C" tra_status tra_attention_backward(tra_plan plan, const void* q, const void* k, const void* v, const void* mask,
                                             const void* out, const float* lse, const void* dout, void* dq, void* dk,
                                             void* dv, void* workspace, size_t workspace_bytes, tra_stream stream)
{
    if (!plan || !q || !k || !v || !mask || !out || !lse || !dout || !dq || !dk || !dv || !workspace)
        return TRA_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, out, dout, (const void*)dq, (const void*)dk, (const void*)dv})
        if (!aligned(p, 16)) return TRA_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(mask, 256) || !aligned(workspace, 256)) return TRA_ERR_INVALID_ARG;
    const BwdLayout L = backward_layout(plan);
    if (workspace_bytes < L.total) return TRA_ERR_WORKSPACE;
    const tra::Geom& G = plan->geom;
    const bool bf16 = (plan->flags & TRA_FLAG_OUT_BF16) != 0;
    uint8_t* ws = (uint8_t*)workspace;
    const tra::RowCopies copy = {L.copy_q ? (uint4*)(ws + L.off_q) : nullptr, (uint4*)(ws + L.off_do),
                                 L.copy_kv ? (uint4*)(ws + L.off_k) : nullptr, L.copy_kv ? (uint4*)(ws + L.off_v) : nullptr};
    const uint64_t rows = (uint64_t)G.G * G.N_pad;
    CUtensorMap mq, mk, mv, md;
    if (!make_row_map(&mq, copy.q ? copy.q : q, rows, G.D) || !make_row_map(&mk, copy.k ? copy.k : k, rows, G.D) ||
        !make_row_map(&mv, copy.v ? copy.v : v, rows, G.D) || !make_row_map(&md, copy.dout, rows, G.D))
        return TRA_ERR_CUDA;

    cudaStream_t st = (cudaStream_t)stream;
    tra::BwdArgs A;
    A.mask = (const uint8_t*)mask;
    A.rows = (const float4*)ws;
    A.bits = (const uint32_t*)(ws + L.off_bits);
    A.bw = L.bw;
    A.out_bf16 = bf16 ? 1 : 0;
    A.dq = dq; A.dk = dk; A.dv = dv;
    A.grad_scale = (float)(1.0 / std::sqrt((double)G.D));

    const dim3 row_grid(G.N_pad * (G.D / 8) / 256, G.G);
    auto go = [&](auto kern) {
        kern<<<row_grid, 256, 0, st>>>(G, A.mask, out, dout, lse, (const uint4*)q, (const uint4*)k, (const uint4*)v, (float4*)ws, copy,
                                         (uint32_t*)(ws + L.off_bits), L.bw);
    };
    if (G.D == 64) bf16 ? go(tra::backward_rows_kernel<64, false>) : go(tra::backward_rows_kernel<64, true>);
    else bf16 ? go(tra::backward_rows_kernel<128, false>) : go(tra::backward_rows_kernel<128, true>);
    tra::transpose_lists_kernel<<<(unsigned)(((size_t)G.G * G.nQ + 3) / 4), 128, 0, st>>>(G, A.mask, (uint32_t*)(ws + L.off_bits), L.bw);
    if (launch_status() != TRA_OK) return TRA_ERR_CUDA;
    switch (G.D * 100 + G.tw_log2) {
        case 6402: return run_backward<64, 2>(G, A, mq, mk, mv, md, st);
        case 6403: return run_backward<64, 3>(G, A, mq, mk, mv, md, st);
        case 6404: return run_backward<64, 4>(G, A, mq, mk, mv, md, st);
        case 6405: return run_backward<64, 5>(G, A, mq, mk, mv, md, st);
        case 12802: return run_backward<128, 2>(G, A, mq, mk, mv, md, st);
        case 12803: return run_backward<128, 3>(G, A, mq, mk, mv, md, st);
        case 12804: return run_backward<128, 4>(G, A, mq, mk, mv, md, st);
        case 12805: return run_backward<128, 5>(G, A, mq, mk, mv, md, st);
    }
    return TRA_ERR_UNSUPPORTED;
}
