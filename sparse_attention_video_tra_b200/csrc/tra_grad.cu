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
// copies of dO and Q in mask-slot order.  dO is copied unless the kernels can
// read the caller's rows as they are (natural layout, bf16, no query groups):
// fp32 rows need rounding, grouped rows reordering, and tile-major pad rows
// must be zeros for the products.
struct BwdLayout {
    bool copy_do, copy_q;
    int bw;
    size_t off_bits, bits_bytes, off_do, off_q, total;
};

BwdLayout backward_layout(tra_plan plan)
{
    const tra::Geom& G = plan->geom;
    BwdLayout L;
    L.copy_q = G.qsort != 0;
    L.copy_do = L.copy_q || !G.natural || !(plan->flags & TRA_FLAG_OUT_BF16);
    L.bw = tra::reach_words(G);
    const size_t rows = (size_t)G.G * G.N_pad;
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    L.off_bits = up(rows * sizeof(float4));
    L.bits_bytes = (size_t)G.G * G.nQ * L.bw * 4;
    L.off_do = up(L.off_bits + L.bits_bytes);
    L.off_q = up(L.off_do + (L.copy_do ? rows * G.D * 2 : 0));
    L.total = up(L.off_q + (L.copy_q ? rows * G.D * 2 : 0));
    return L;
}

template <int D, int TWL, bool DISK>
tra_status run_backward(const tra::Geom& G, const tra::BwdArgs& A, const CUtensorMap& q, const CUtensorMap& k,
                        const CUtensorMap& v, const CUtensorMap& d, cudaStream_t st)
{
    using KV = tra::BwdKvCfg<D>;
    using Q = tra::BwdQCfg<D>;
    auto kv = tra::backward_kv_kernel<D, TWL, DISK>;
    auto qk = tra::backward_q_kernel<D, TWL, DISK>;
    const int smem_kv = KV::smem(G.list_cap), smem_q = Q::smem();
    if (smem_kv > kMaxSmem || smem_q > kMaxSmem) return TRA_ERR_UNSUPPORTED;
    if (!set_smem(kv, smem_kv) || !set_smem(qk, smem_q)) return TRA_ERR_CUDA;
    kv<<<dim3(G.nQ, G.G), KV::THREADS, smem_kv, st>>>(q, k, v, d, G, A);
    qk<<<dim3(G.nQ, G.G), Q::THREADS, smem_q, st>>>(q, k, v, d, G, A);
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
    uint8_t* do_copy = L.copy_do ? ws + L.off_do : nullptr;
    uint8_t* q_copy = L.copy_q ? ws + L.off_q : nullptr;
    const uint64_t rows = (uint64_t)G.G * G.N_pad;
    CUtensorMap mq, mk, mv, md;
    if (!make_input_map(&mk, k, G) || !make_input_map(&mv, v, G)) return TRA_ERR_CUDA;
    if (!(q_copy ? make_row_map(&mq, q_copy, rows, G.D) : make_input_map(&mq, q, G))) return TRA_ERR_CUDA;
    if (!(do_copy ? make_row_map(&md, do_copy, rows, G.D) : make_input_map(&md, dout, G))) return TRA_ERR_CUDA;

    cudaStream_t st = (cudaStream_t)stream;
    tra::BwdArgs A;
    A.mask = (const uint8_t*)mask;
    A.rows = (const float4*)ws;
    A.bits = (const uint32_t*)(ws + L.off_bits);
    A.bw = L.bw;
    A.q_natural = G.natural && !q_copy;
    A.do_natural = G.natural && !do_copy;
    A.out_bf16 = bf16 ? 1 : 0;
    A.dq = dq; A.dk = dk; A.dv = dv;
    A.grad_scale = (float)(1.0 / std::sqrt((double)G.D));

    if (cudaMemsetAsync(ws + L.off_bits, 0, L.bits_bytes, st) != cudaSuccess) return TRA_ERR_CUDA;
    const unsigned row_blocks = (unsigned)((rows + 7) / 8);
    auto go = [&](auto kern) {
        kern<<<row_blocks, 256, 0, st>>>(G, A.mask, out, dout, lse, (const uint4*)q, (float4*)ws, (uint32_t*)q_copy,
                                         (uint32_t*)do_copy);
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
