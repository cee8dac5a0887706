// backward.cuh -- the gradients of tra_attention, probabilities recomputed.
//
// With x_ij = q_i.k_j / sqrt d over the kept pairs, P_ij = exp(x_ij - lse_i),
// dP_ij = dO_i.v_j and D_i = dO_i.O_i:
//     dS_ij = P_ij (dP_ij - D_i)
//     dV_j = sum_i P_ij dO_i,  dK_j = sum_i dS_ij q_i / sqrt d,
//     dQ_i = sum_j dS_ij k_j / sqrt d.
// Three launches:
//   backward_rows   D_i, the log2-domain lse and the grid position of every
//                   query row in mask-slot order, the operands copied to
//                   plain rows where the caller's are not, the tile bitmaps cleared
//   transpose_lists the mask's key-tile lists as bits per (key tile, query slot)
//   backward        one CTA per key tile: dK and dV over the query slots that
//                   list it (backward_kv); and one CTA per query slot: dQ over
//                   its key tiles (backward_q)
// S and dP are computed in both parts of the last (7 products per tile pair where
// 5 would do with dQ added up across CTAs): every output row is then written
// once, by one CTA, with a fixed order of summation, so the gradients are
// bit-identical from run to run, no fp32 dQ buffer is needed, and neither
// part moves P or dS through shared memory: each keeps the rows it sums over
// in the tensor memory's columns and the rows it owns in its lanes.
// P and dS are rounded to bf16 for the tensor cores (at most 2^-8 of each
// value, as P in the forward pass); all sums are fp32.
#pragma once
#include <type_traits>

#include <cuda_bf16.h>

#include "pipeline.cuh"

namespace tra {

// What the gradient kernel reads besides the tensor maps.
struct BwdArgs {
    const uint8_t* mask;
    const float4* rows;          // [heads][nQ][128] slot order: lse * log2 e, D_i, h | w << 8 (bits), radius (bits)
    const uint32_t* bits;        // [heads][nQ key tiles][bw]: bit q - first(key tile) = slot q lists the tile
    int bw;
    int out_bf16;                // gradients in bf16 instead of fp32
    void *dq, *dk, *dv;
    float grad_scale;            // 1 / sqrt d
};

// first query slot (or key tile) within Rt' frames of tile t
__host__ __device__ inline int first_reach(const Geom& G, int tile)
{
    const int t = tile / G.tiles_per_frame - G.rte;
    return (t < 0 ? 0 : t) * G.tiles_per_frame;
}

__host__ __device__ inline int reach_words(const Geom& G) { return (G.list_cap + 31) / 32; }

// one 64-column panel of tile (or slot) `tile` of head g
__device__ __forceinline__ void load_panel(void* dst, const CUtensorMap* m, const Geom& G, int p, int g, int tile, uint64_t* bar)
{
    tma_load_2d(dst, m, p * 64, g * G.N_pad + tile * 128, bar);
}

// ------------------------------------------------------------------ row data
// What the product kernels read is put in order first: every operand as
// [heads][N_pad] rows, queries by mask slot and keys by tile, pad rows zeros,
// so that each tile is a plain 128-row box.  (Read through 4-D boxes of the
// natural layout, the same tiles kept the copy engine behind the products:
// 3180 instead of 2406 cycles a tile pair in backward_q at 21 x 30 x 52.)
// A copy that is not needed has a null pointer.  d/8 lanes per row; blockIdx.y
// is the head.  IN_F32: dout and out are fp32 (else bf16); dO is rounded to
// bf16 first and D_i taken from the rounded values, the ones the products
// use.  HBM-bound: 2 to 5 rows read and 1 to 4 written per token (at 21 x 45 x 80,
// 4 heads, natural layout: 0.70 GB in 113 us, 6.2 TB/s).
struct RowCopies {
    uint4 *q, *dout, *k, *v;
};

template <int D, bool IN_F32>
__global__ void __launch_bounds__(256)
backward_rows_kernel(const Geom G, const uint8_t* __restrict__ mask, const void* __restrict__ out,
                     const void* __restrict__ dout, const float* __restrict__ lse, const uint4* __restrict__ q,
                     const uint4* __restrict__ k, const uint4* __restrict__ v, float4* __restrict__ rows, const RowCopies copy,
                     uint32_t* __restrict__ bits, int bw)
{
    constexpr int LPR = D / 8;                                        // lanes per row
    const int g = blockIdx.y, sub = threadIdx.x % LPR;
    const int in = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;      // row of the head; N_pad is a multiple of 128
    const size_t p = (size_t)g * G.N_pad + in;
    const int slot = in >> 7;
    int t, tr, tc;
    tile_coords(G, slot, t, tr, tc);
    // the token of tile row i in tile row tr of this slot's tile column and frame
    auto token = [&](int tr, int i, int& h, int& w, int& trow) -> bool {
        h = tr * G.th + (i >> G.tw_log2);
        w = tc * G.tw + (i & (G.tw - 1));
        trow = ((t * G.nTh + tr) * G.nTw + tc) * 128 + i;
        return h < G.H && w < G.W;
    };
    // the head's tile bitmaps, nQ * bw words, over its blocks
    for (int i = blockIdx.x * 256 + threadIdx.x; i < G.nQ * bw; i += gridDim.x * 256) bits[(size_t)g * G.nQ * bw + i] = 0u;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    int h, w, trow;
    if (copy.k) {
        const bool ok = token(tr, in & 127, h, w, trow);
        const size_t at = ok ? io_row(G, g, t, h, w, trow) * LPR + sub : 0;
        copy.k[p * LPR + sub] = ok ? __ldg(k + at) : zero;
        copy.v[p * LPR + sub] = ok ? __ldg(v + at) : zero;
    }
    int qtr = tr, qi = in & 127;
    bool named = true;
    if (G.qsort) {
        const int l = reinterpret_cast<const uint16_t*>(mask + G.off_group)[p];
        named = l < 128 * G.nTh;                                      // caller memory: recorded, the row left out
        if (!named && sub == 0) atomicOr(&g_tra_error, TRA_ERRBIT_CHECK);
        qtr = named ? l >> 7 : 0;
        qi = named ? l & 127 : 0;
    }
    const bool ok = token(qtr, qi, h, w, trow) && named;
    const size_t src = ok ? io_row(G, g, t, h, w, trow) : 0;
    uint4 x = zero;                                                   // 8 elements of dO as bf16
    float d = 0.f;
    if (ok) {
        float o[8];
        if constexpr (IN_F32) {
            const float4* xs = static_cast<const float4*>(dout) + src * (D / 4) + 2 * sub;
            const float4* os = static_cast<const float4*>(out) + src * (D / 4) + 2 * sub;
            const float4 x0 = __ldg(xs), x1 = __ldg(xs + 1), o0 = __ldg(os), o1 = __ldg(os + 1);
            x = make_uint4(pack_bf16x2(x0.x, x0.y), pack_bf16x2(x0.z, x0.w), pack_bf16x2(x1.x, x1.y), pack_bf16x2(x1.z, x1.w));
            o[0] = o0.x; o[1] = o0.y; o[2] = o0.z; o[3] = o0.w; o[4] = o1.x; o[5] = o1.y; o[6] = o1.z; o[7] = o1.w;
        } else {
            x = __ldg(static_cast<const uint4*>(dout) + src * LPR + sub);
            const uint4 ob = __ldg(static_cast<const uint4*>(out) + src * LPR + sub);
            const uint32_t w4[4] = {ob.x, ob.y, ob.z, ob.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = __uint_as_float(w4[i] << 16);
                o[2 * i + 1] = __uint_as_float(w4[i] & 0xffff0000u);
            }
        }
        const uint32_t x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d = fmaf(__uint_as_float(x4[i] << 16), o[2 * i], d);
            d = fmaf(__uint_as_float(x4[i] & 0xffff0000u), o[2 * i + 1], d);
        }
    }
    if (copy.dout) copy.dout[p * LPR + sub] = x;
    if (copy.q) copy.q[p * LPR + sub] = ok ? __ldg(q + src * LPR + sub) : zero;
#pragma unroll
    for (int s = LPR / 2; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
    if (sub == 0) {
        int r = ok ? reinterpret_cast<const int32_t*>(mask + G.off_radius)[(size_t)g * G.N_pad + trow] : -1;
        float l2 = 0.f;
        if (ok) {
            l2 = lse[src] * 1.4426950408889634f;
            if (l2 == -INFINITY) { l2 = 0.f; r = -1; }                // a row that kept nothing
        }
        rows[p] = make_float4(l2, d, __int_as_float(h | (w << 8)), __int_as_float(r));
    }
}

// The lists of the mask as bits per (head, key tile, query slot).  Bits are
// set by atomic ORs, whose order does not show.  One warp per (head, slot).
__global__ void __launch_bounds__(128)
transpose_lists_kernel(const Geom G, const uint8_t* __restrict__ mask, uint32_t* __restrict__ bits, int bw)
{
    const int lane = threadIdx.x & 31;
    const size_t s = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (s >= (size_t)G.G * G.nQ) return;
    const int g = (int)(s / G.nQ), slot = (int)(s - (size_t)g * G.nQ);
    int n = reinterpret_cast<const int32_t*>(mask + G.off_count)[s];
    if (n < 0 || n > G.list_cap) {
        if (lane == 0) atomicOr(&g_tra_error, TRA_ERRBIT_CHECK);
        n = 0;
    }
    const uint16_t* list = reinterpret_cast<const uint16_t*>(mask + G.off_list) + s * G.list_cap;
    const int ts = slot / G.tiles_per_frame;
    for (int j = lane; j < n; j += 32) {
        const int kt = list[j] & 0x7fff;
        if (kt >= G.nQ || abs(kt / G.tiles_per_frame - ts) > G.rte) {
            atomicOr(&g_tra_error, TRA_ERRBIT_CHECK);
            continue;
        }
        const int b = slot - first_reach(G, kt);
        atomicOr(&bits[((size_t)g * G.nQ + kt) * bw + (b >> 5)], 1u << (b & 31));
    }
}

// ------------------------------------------------------------------ masks
// the low n bits, 0 <= n <= 32 (PTX shifts by 32 or more give 0)
__device__ __forceinline__ uint32_t low_bits(int n)
{
    uint32_t r;
    asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(0xffffffffu), "r"(n));
    return ~r;
}

// The keys lo .. hi of a tile's 32 key rows or columns, as bits: those within s
// of y (s < 0: none) among the n valid ones.
__device__ __forceinline__ uint32_t kept_line(int y, int s, int n)
{
    return s < 0 ? 0u : low_bits(max(0, min(n, y + s + 1))) & ~low_bits(min(max(0, y - s), 32));
}

// Bit i of lane j's word goes to bit j of lane i's word.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t v, int lane)
{
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const uint32_t m = s == 16 ? 0x0000ffffu : (s == 8 ? 0x00ff00ffu : (s == 4 ? 0x0f0f0f0fu : (s == 2 ? 0x33333333u : 0x55555555u)));
        const uint32_t y = __shfl_xor_sync(0xffffffffu, v, s);
        v = (lane & s) ? (v & ~m) | ((y & ~m) >> s) : (v & m) | ((y & m) << s);
    }
    return v;
}

// x as the sum of three bf16 numbers (24 bits), in the first three of the eight
// bf16 of a 16-byte chunk
__device__ __forceinline__ uint4 split_bf16x3(float x)
{
    const float hi = __bfloat162float(__float2bfloat16(x));
    const float mid = __bfloat162float(__float2bfloat16(x - hi));
    return make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(x - hi - mid, 0.f), 0u, 0u);
}

// Stores 32 accumulator columns of one row, scaled.
__device__ __forceinline__ void store_cols32(void* base, bool bf16, size_t elem, const uint32_t (&v)[32], float sc)
{
    if (bf16) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + elem);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * k]) * sc, __uint_as_float(v[8 * i + 2 * k + 1]) * sc);
            dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    } else {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(v[4 * i]) * sc, __uint_as_float(v[4 * i + 1]) * sc,
                                 __uint_as_float(v[4 * i + 2]) * sc, __uint_as_float(v[4 * i + 3]) * sc);
    }
}

// ------------------------------------------------------------------ dK, dV
// One CTA per (key tile, head), 384 threads.  Keys sit in the tensor memory's
// lanes and queries in its columns, so P^T and dS^T are the A operands of
// dV += P^T dO and dK += dS^T Q as they stand:
//   warps 0-7  warpgroup u owns the queries 64u .. 64u + 63 of a slot, thread
//              r of it key row r: reads S^T, makes P^T (kept in registers as
//              fp32 and written back over S^T as bf16), then reads dP^T and
//              writes dS^T over it.
//   warp 8     TMA: K, V once, then the rings of Q and dO.
//   warp 9     MMA issuer.  Per slot j, two groups alternate with the two
//              halves of the elementwise work: {dV += P^T dO, S^T of slot j+1}
//              while dS^T of j is made, {dK += dS^T Q, dP^T of slot j+1} while
//              P^T of j+1 is made.  MMAs of one thread run in order, so S^T of
//              j+1 overwrites P^T of j only after dV has read it, and dP^T of
//              j+1 overwrites dS^T of j only after dK has.
//   warps 10, 11  per slot and half, the per-query data into a ring: planes of
//              -lse and -D_i for the tensor core, what the keys need to know
//              which queries keep them (square: a 64-bit word per key row
//              and per key column, whose AND is a key's; disk: three numbers
//              per query), and whether all pairs are kept (such halves skip
//              the masking).
// The products read shared memory at its full rate, so the elementwise work
// keeps off it: lse and D_i vary along the columns, and fetching them per
// column (and a mask word each) took 1536 cycles of that bandwidth per tile
// pair.  Instead one more K step of the product adds them: a row of ones times
// the number split into three bf16 parts (24 bits).
// TMEM columns: S^T [0,128), dP^T [128,256), dV [256,256+D), dK [384,384+D).
// P^T of warpgroup u: bf16 pairs in columns 64u .. 64u+31 (its own half of
// S^T, so the other half's S^T is never overwritten early); dS^T likewise.
template <int D>
struct BwdKvCfg {
    static constexpr int PANEL = 128 * 128;
    static constexpr int NP = D / 64;
    static constexpr int TILE = NP * PANEL;
    static constexpr int OFF_K = 0, OFF_V = TILE;
    static constexpr int OFF_RING = 2 * TILE;               // four tiles: Q and dO of two slots
    static constexpr int MST = 3;                           // ring depth of the per-query data
    static constexpr int OFF_ONE = OFF_RING + 4 * TILE;     // 128 rows of (1, 1, 1, 0, ..), 16 bytes each
    static constexpr int OFF_META = OFF_ONE + 2048;         // [MST]: planes of -lse and -D, key ranges [2 halves][1024 bytes]
    static constexpr int META = 3 * 2048;
    static constexpr int OFF_ZERO = OFF_META + MST * META;  // a plane of zeros
    static constexpr int OFF_BARS = OFF_ZERO + 2048;
    static constexpr int OFF_LIST = OFF_BARS + 40 * 8 + 64; // uint16 [list_cap]
    static constexpr int REGS_SOFTMAX = 216, REGS_OTHER = 72;
    static int smem(int list_cap) { return OFF_LIST + ((list_cap * 2 + 15) & ~15) + 1024; }
    // The ring tiles of slot j's Q and dO.  dO of a slot is done with half a step
    // before its Q (dV comes before dK), and Q is needed half a step before
    // dO, so Q of slot j + 2 goes where dO of slot j was and dO of j + 2 where
    // Q of j was: either has a whole step to arrive.
    __device__ static int q_tile(int j) { return (j & 1) * 2 + ((j >> 1) & 1); }
    __device__ static int do_tile(int j) { return q_tile(j) ^ 1; }
};

template <int D, int TWL, bool DISK>
__device__ __forceinline__ void backward_kv(uint8_t* smem, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                            const CUtensorMap& tm_do, const Geom& G, const BwdArgs& A)
{
    using C = BwdKvCfg<D>;
    constexpr int TW = 1 << TWL;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
    uint64_t* kv_full = bars;
    uint64_t* r_full = bars + 1;                 // [4]: ring tiles
    uint64_t* r_empty = r_full + 4;
    uint64_t* meta_full = r_empty + 4;           // [MST][2 halves]
    uint64_t* meta_empty = meta_full + 2 * C::MST;
    uint64_t* s_full = meta_empty + 2 * C::MST;
    uint64_t* dp_full = s_full + 1;
    uint64_t* p_full = dp_full + 1;              // [2]: the first and the last 32 queries of each half
    uint64_t* ds_full = p_full + 2;
    uint64_t* done = ds_full + 1;
    int* misc = reinterpret_cast<int*>(bars + 40);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc);
    volatile int* s_abort = misc + 1;
    int* s_n = misc + 2;
    int* s_all = misc + 4;                       // [MST][2]: every pair of the half is kept
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + C::OFF_LIST);

    const int kt = blockIdx.x, g = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = first_reach(G, kt);
    int tk, trk, tck;
    tile_coords(G, kt, tk, trk, tck);
    const int h0 = trk * G.th, w0 = tck * TW;
    const int khv = min(G.th, G.H - h0), kwv = min(TW, G.W - w0);

    if (warp == 0) {
        // the slots that list this key tile, ascending
        const uint32_t* bits = A.bits + ((size_t)g * G.nQ + kt) * A.bw;
        int n = 0;
        for (int b0 = 0; b0 < A.bw; b0 += 32) {
            uint32_t v = b0 + lane < A.bw ? bits[b0 + lane] : 0u;
            int incl = __popc(v);
            const int cnt = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            int at = n + incl - cnt;
            for (; v; v &= v - 1) list[at++] = (uint16_t)(first + (b0 + lane) * 32 + __ffs(v) - 1);
            n += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) *s_n = n;
    }
    if (tid == 32) {
        mbar_init(kv_full, 1);
        for (int i = 0; i < 4; ++i) { mbar_init(&r_full[i], 1); mbar_init(&r_empty[i], 1); }
        for (int i = 0; i < 2 * C::MST; ++i) { mbar_init(&meta_full[i], 32); mbar_init(&meta_empty[i], 128); }
        mbar_init(s_full, 1); mbar_init(dp_full, 1);
        mbar_init(&p_full[0], 256); mbar_init(&p_full[1], 256); mbar_init(ds_full, 256);
        mbar_init(done, 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (tid >= 128 && tid < 256) {
        const uint4 one = make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u);
        reinterpret_cast<uint4*>(smem + C::OFF_ONE)[tid - 128] = one;
        reinterpret_cast<uint4*>(smem + C::OFF_ZERO)[tid - 128] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();                            // generic writes -> tensor-core reads
    }
    if (warp == 9) { tmem_alloc(s_tmem, 512); tmem_relinquish(); }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const int n = *s_n;
    constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DV = 256, COL_DK = 384;

    if (warp >= 8) {
        regs_dec<C::REGS_OTHER>();
        if (warp == 8) {
            if (n > 0 && elect_one()) {
                prefetch_tmap(&tm_q); prefetch_tmap(&tm_k); prefetch_tmap(&tm_v); prefetch_tmap(&tm_do);
                auto load = [&](const CUtensorMap* tm, int j, int tile) -> bool {
                    if (j >= 2 && !role_wait(&r_empty[tile], ((j >> 1) - 1) & 1, G.wait_ns, s_abort)) return false;
                    mbar_arrive_expect_tx(&r_full[tile], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_RING + tile * C::TILE + p * C::PANEL, tm, G, p, g, list[j], &r_full[tile]);
                    return true;
                };
                mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
#pragma unroll
                for (int p = 0; p < C::NP; ++p) {
                    load_panel(smem + C::OFF_K + p * C::PANEL, &tm_k, G, p, g, kt, kv_full);
                    load_panel(smem + C::OFF_V + p * C::PANEL, &tm_v, G, p, g, kt, kv_full);
                }
                int loads = 0;                               // Q(0), dO(0), Q(1), ...
                for (; loads < 2 * n; ++loads) {
                    const int j = loads >> 1;
                    if (!((loads & 1) ? load(&tm_do, j, C::do_tile(j)) : load(&tm_q, j, C::q_tile(j)))) break;
                }
                // copies still in flight must land before the CTA exits
                mbar_wait(kv_full, 0, G.drain_ns);
                for (int i = max(0, loads - 4); i < loads; ++i) {
                    const int j = i >> 1;
                    mbar_wait(&r_full[(i & 1) ? C::do_tile(j) : C::q_tile(j)], (j >> 1) & 1, G.drain_ns);
                }
            }
        } else if (warp == 9) {
            if (n > 0 && elect_one()) {
                constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false);
                constexpr uint32_t IDESC_G = idesc_bf16_f32(128, D, true);
                const uint32_t sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
                const uint32_t sR = smem_u32(smem + C::OFF_RING);
                const uint32_t sOne = smem_u32(smem + C::OFF_ONE), sMeta = smem_u32(smem + C::OFF_META), sZero = smem_u32(smem + C::OFF_ZERO);
                // A (keys) times B^T (queries), both K-major, plus 1 times the
                // plane's number of each query
                auto scores = [&](uint32_t col, uint32_t a, uint32_t b, uint32_t plane, uint64_t* full) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::PANEL + (kk & 3) * 32;
                        mma_ss(tmem + col, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
                    }
                    mma_ss(tmem + col, smem_desc_plain(sOne, sZero - sOne, 128), smem_desc_plain(plane, sZero - plane, 128), IDESC_S, 1u);
                    mma_commit(full);
                };
                // the bf16 pairs in quarter c of the two halves of `col` times their rows of b
                auto accumulate = [&](uint32_t dst, uint32_t col, uint32_t b, int c, bool add) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = (i >> 1) * 4 + c * 2 + (i & 1);
                        mma_ts(tmem + dst, tmem + col + (kk >> 2) * 64 + (kk & 3) * 8,
                               smem_desc_sw128(b + kk * 2048, C::PANEL, 1024), IDESC_G, (add || i > 0) ? 1u : 0u);
                    }
                };
                auto wait_q = [&](int j) -> bool { return role_wait(&r_full[C::q_tile(j)], (j >> 1) & 1, G.wait_ns, s_abort); };
                auto wait_do = [&](int j) -> bool { return role_wait(&r_full[C::do_tile(j)], (j >> 1) & 1, G.wait_ns, s_abort); };
                auto issue_s = [&](int j) { scores(COL_S, sK, sR + C::q_tile(j) * C::TILE, sMeta + j % C::MST * C::META, s_full); };
                auto issue_dp = [&](int j) { scores(COL_DP, sV, sR + C::do_tile(j) * C::TILE, sMeta + j % C::MST * C::META + 2048, dp_full); };
                bool ok = role_wait(&meta_full[0], 0, G.wait_ns, s_abort) && role_wait(&meta_full[1], 0, G.wait_ns, s_abort) &&
                          role_wait(kv_full, 0, G.wait_ns, s_abort) && wait_q(0) && wait_do(0);
                if (ok) {
                    tc_fence_after();
                    issue_s(0);
                    issue_dp(0);
                }
                for (int j = 0; ok && j < n; ++j) {
                    const int qt = C::q_tile(j), dt = C::do_tile(j);
                    const bool next = j + 1 < n;
                    // what a group needs besides P^T or dS^T is waited for first:
                    // a wait takes 100 to 200 cycles even when it is over
                    if (next && !wait_q(j + 1)) break;
                    if (!role_wait(&p_full[0], j & 1, G.wait_ns, s_abort)) break;
                    tc_fence_after();
                    accumulate(COL_DV, COL_S, sR + dt * C::TILE, 0, j > 0);
                    if (!role_wait(&p_full[1], j & 1, G.wait_ns, s_abort)) break;
                    tc_fence_after();
                    accumulate(COL_DV, COL_S, sR + dt * C::TILE, 1, true);
                    mma_commit(&r_empty[dt]);
                    if (next) issue_s(j + 1);
                    if (next && !wait_do(j + 1)) break;
                    if (!role_wait(ds_full, j & 1, G.wait_ns, s_abort)) break;
                    tc_fence_after();
                    accumulate(COL_DK, COL_DP, sR + qt * C::TILE, 0, j > 0);
                    accumulate(COL_DK, COL_DP, sR + qt * C::TILE, 1, true);
                    mma_commit(&r_empty[qt]);
                    if (next) issue_dp(j + 1);
                }
                // every issued MMA must finish before the results are read and TMEM is freed
                mma_commit(done);
                mbar_wait(done, 0, G.drain_ns);
            }
        } else {
            // ------------------------------------------------ queries' lse, D_i and kept keys
            const int half = warp - 10;
            const float4* rows = A.rows + (size_t)g * G.nQ * 128 + half * 64 + lane;
            const float unit = -1.f / G.scale_log2;          // lse in units of the raw scores, negated
            float4 r0, r1;
            if (n > 0) {
                r0 = __ldg(rows + list[0] * 128);
                r1 = __ldg(rows + list[0] * 128 + 32);
            }
            for (int j = 0; j < n; ++j) {
                const int st = j % C::MST, ring = st * 2 + half;
                const float4 x[2] = {r0, r1};
                const double decay = G.g[abs(list[j] / G.tiles_per_frame - tk)];
                if (j + 1 < n) {                             // the next slot's rows are on their way meanwhile
                    r0 = __ldg(rows + list[j + 1] * 128);
                    r1 = __ldg(rows + list[j + 1] * 128 + 32);
                }
                // square: the kept key rows and columns; disk: A, B, C of the test
                // A + B a + C b <= -(a^2 + b^2) that key (a, b) makes of the query at
                // (y, x), with A = y^2 + x^2 - s^2, B = -2y, C = -2x (integers
                // below 2^23, exact in fp32)
                uint32_t m[2][3];
                bool all = true;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int pos = __float_as_int(x[k].z), r = __float_as_int(x[k].w);
                    const int y = (pos & 255) - h0, xx = ((pos >> 8) & 255) - w0;
                    const int s = r >= 0 ? min(halfwidth(r, decay), TRA_DISK_S_CLAMP) : -1;
                    if constexpr (DISK) {
                        const int fy = max(abs(y), abs(y - (G.th - 1))), fx = max(abs(xx), abs(xx - (TW - 1)));
                        all = all && khv == G.th && kwv == TW && s >= 0 && fy * fy + fx * fx <= s * s;
                        m[k][0] = __float_as_uint(s >= 0 ? (float)(y * y + xx * xx - s * s) : 4e6f);   // 4e6: above any -(B a + C b)
                        m[k][1] = __float_as_uint((float)(-2 * y));
                        m[k][2] = __float_as_uint((float)(-2 * xx));
                    } else {
                        m[k][0] = kept_line(y, s, khv);
                        m[k][1] = kept_line(xx, s, kwv);
                        all = all && m[k][0] == low_bits(G.th) && m[k][1] == low_bits(TW);
                    }
                }
                all = __all_sync(0xffffffffu, all);
                if (!DISK && !all) {                         // from a query's keys to a key's queries
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int wd = 0; wd < 2; ++wd) m[k][wd] = transpose_bits(m[k][wd], lane);
                }
                bool got = true;
                if (j >= C::MST) got = role_wait(&meta_empty[ring], ((j / C::MST) - 1) & 1, G.wait_ns, s_abort);
                if (__any_sync(0xffffffffu, !got)) break;
                uint4* lse4 = reinterpret_cast<uint4*>(smem + C::OFF_META + st * C::META) + half * 64 + lane;
                lse4[0] = split_bf16x3(x[0].x * unit);
                lse4[32] = split_bf16x3(x[1].x * unit);
                lse4[128] = split_bf16x3(-x[0].y);
                lse4[160] = split_bf16x3(-x[1].y);
                uint32_t* keys = reinterpret_cast<uint32_t*>(smem + C::OFF_META + st * C::META + 4096 + half * 1024);
                if constexpr (DISK) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int wd = 0; wd < 3; ++wd) keys[wd * 64 + k * 32 + lane] = m[k][wd];
                } else {
#pragma unroll
                    for (int wd = 0; wd < 2; ++wd) reinterpret_cast<uint2*>(keys)[wd * 32 + lane] = make_uint2(m[0][wd], m[1][wd]);
                }
                if (lane == 0) s_all[ring] = all ? 1 : 0;
                fence_proxy_async_smem();                    // the planes are read by the tensor core
                mbar_arrive(&meta_full[ring]);
            }
        }
    } else {
        regs_inc<C::REGS_SOFTMAX>();
        // ------------------------------------------------ P^T and dS^T
        const int u = warp >> 2;                             // queries 64u .. 64u + 63 of a slot
        const int row = tid & 127;                           // key row = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t colS = tmem + lane_base + COL_S + u * 64, colP = tmem + lane_base + COL_DP + u * 64;
        const f2_t sc2 = f2_pack(G.scale_log2, G.scale_log2);
        const int ka = row >> TWL, kb = row & (TW - 1);      // this key's row and column in the tile
        const f2_t ka2 = f2_pack((float)ka, (float)ka), kb2 = f2_pack((float)kb, (float)kb);
        const float kthr = ka < khv && kb < kwv ? -(float)(ka * ka + kb * kb) : -INFINITY;
        // this key's kept queries of the half, fetched one slot ahead; P^T of slot
        // j is handed over after the per-query data of slot j + 1 has been seen,
        // so the MMA issuer need not wait for it
        bool all_next = false;
        uint2 keep_next = make_uint2(0u, 0u);
        auto fetch_keep = [&](int j) -> bool {
            const int ms = j % C::MST;
            if (!role_wait(&meta_full[ms * 2 + u], (j / C::MST) & 1, G.wait_ns, s_abort)) return false;
            all_next = s_all[ms * 2 + u] != 0;
            if constexpr (!DISK) {                           // a kept key row and a kept key column
                const uint2* lines = reinterpret_cast<const uint2*>(smem + C::OFF_META + ms * C::META + 4096 + u * 1024);
                const uint2 r = lines[row >> TWL], c = lines[32 + (row & (TW - 1))];
                keep_next = make_uint2(r.x & c.x, r.y & c.y);
            }
            return true;
        };
        bool ok = n == 0 || fetch_keep(0);
        ok = __all_sync(0xffffffffu, ok);
        for (int j = 0; ok && j < n; ++j) {
            const int ring = (j % C::MST) * 2 + u;
            const bool all = all_next;
            const uint2 keep = keep_next;
            bool got = j + 1 == n || fetch_keep(j + 1);
            got = got && role_wait(s_full, j & 1, G.wait_ns, s_abort);
            if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            uint32_t v[2][32];
            tmem_ld32(colS, v[0]);
            tmem_ld32(colS + 32, v[1]);
            tmem_wait_ld();
            f2_t p[32];
            const f2_t* disk = reinterpret_cast<const f2_t*>(smem + C::OFF_META + (j % C::MST) * C::META + 4096 + u * 1024);
            // S^T already holds the score minus the log-sum-exp, in score units
            auto probabilities = [&](auto masked) {
                constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[16];
                    const uint32_t m = c ? keep.y : keep.x;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        f2_unpack(f2_mul(f2_pack(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1])), sc2), x0, x1);
                        if constexpr (MASKED && DISK) {
                            float t0, t1;
                            f2_unpack(f2_fma(disk[64 + c * 16 + i], kb2, f2_fma(disk[32 + c * 16 + i], ka2, disk[c * 16 + i])), t0, t1);
                            x0 = t0 <= kthr ? x0 : -INFINITY;
                            x1 = t1 <= kthr ? x1 : -INFINITY;
                        } else if constexpr (MASKED) {
                            x0 = (m >> (2 * i)) & 1u ? x0 : -INFINITY;
                            x1 = (m >> (2 * i + 1)) & 1u ? x1 : -INFINITY;
                        }
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        p[c * 16 + i] = f2_pack(x0, x1);
                        pk[i] = pack_bf16x2(x0, x1);
                    }
                    tmem_st16(colS + c * 16, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&p_full[c]);
                }
            };
            if (all) probabilities(std::false_type{});
            else probabilities(std::true_type{});
            got = role_wait(dp_full, j & 1, G.wait_ns, s_abort);
            if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            tmem_ld32(colP, v[0]);
            tmem_ld32(colP + 32, v[1]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 2; ++c) {                    // dP^T already holds dP - D
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x0, x1;
                    f2_unpack(f2_mul(p[c * 16 + i], f2_pack(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1]))), x0, x1);
                    pk[i] = pack_bf16x2(x0, x1);
                }
                tmem_st16(colP + c * 16, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(ds_full);
            mbar_arrive(&meta_empty[ring]);
        }
        // warpgroup 0 writes dV, warpgroup 1 dK; a key tile that no slot lists gets zeros
        if (ok) ok = n == 0 || role_wait(done, 0, G.wait_ns, s_abort);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            __syncwarp();
            const int hk = h0 + (row >> TWL), wk = w0 + (row & (TW - 1));
            const bool store = !G.natural || (hk < G.H && wk < G.W);
            const size_t orow = io_row(G, g, tk, hk, wk, kt * 128 + row) * D;
            void* dst = u ? A.dk : A.dv;
            const float sc = u ? A.grad_scale : 1.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld32(tmem + lane_base + (u ? COL_DK : COL_DV) + c * 32, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                }
                if (store) store_cols32(dst, A.out_bf16 != 0, orow + c * 32, v, sc);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ dQ
// One CTA per (query slot, head), 384 threads.  Queries sit in the lanes, keys
// in the columns: dS is the A operand of dQ += dS K as it stands, and a row's
// lse, D_i and key window are scalars of its thread.
//   warps 0-7  warpgroup u owns the keys 64u .. 64u + 63 of a tile, thread r
//              of it query row r.
//   warp 8     TMA: Q, dO once, then the rings of K (three deep: S of tile j+2
//              is issued while K of tile j is still needed for dQ) and V.
//   warp 9     MMA issuer: S two tiles ahead in two buffers, dP one tile ahead.
// TMEM columns: S [0,128) and [128,256) by tile parity, dP [256,384),
// dQ [384,384+D); dS of warpgroup u as bf16 pairs in columns 64u .. 64u+31 of
// its S buffer.
template <int D>
struct BwdQCfg {
    static constexpr int PANEL = 128 * 128;
    static constexpr int NP = D / 64;
    static constexpr int TILE = NP * PANEL;
    static constexpr int KST = 3, VST = 2;
    static constexpr int OFF_Q = 0, OFF_DO = TILE;
    static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + KST * TILE;
    static constexpr int OFF_BARS = OFF_V + VST * TILE;
    static constexpr int BYTES = OFF_BARS + 24 * 8 + 32;
    static constexpr int REGS_SOFTMAX = 216, REGS_OTHER = 72;
    static int smem() { return BYTES + 1024; }
};

template <int D, int TWL, bool DISK>
__device__ __forceinline__ void backward_q(uint8_t* smem, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                           const CUtensorMap& tm_do, const Geom& G, const BwdArgs& A)
{
    using C = BwdQCfg<D>;
    constexpr int TW = 1 << TWL;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
    uint64_t* q_full = bars;
    uint64_t* k_full = bars + 1;                 // [KST]
    uint64_t* k_empty = k_full + C::KST;
    uint64_t* v_full = k_empty + C::KST;         // [VST]
    uint64_t* v_empty = v_full + C::VST;
    uint64_t* s_full = v_empty + C::VST;         // [2]
    uint64_t* dp_full = s_full + 2;
    uint64_t* dp_read = dp_full + 1;
    uint64_t* ds_full = dp_read + 1;
    uint64_t* done = ds_full + 1;
    int* misc = reinterpret_cast<int*>(bars + 24);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc);
    volatile int* s_abort = misc + 1;

    const int slot = blockIdx.x, g = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int ts = slot / G.tiles_per_frame;
    int n = reinterpret_cast<const int32_t*>(A.mask + G.off_count)[(size_t)g * G.nQ + slot];
    if (n < 0 || n > G.list_cap) n = 0;          // recorded by transpose_lists
    const uint16_t* list = reinterpret_cast<const uint16_t*>(A.mask + G.off_list) + ((size_t)g * G.nQ + slot) * G.list_cap;
    // a listed tile out of reach (recorded by transpose_lists) is replaced by
    // the slot's own tile with every pair masked
    auto entry = [&](int j) -> int {
        const int e = __ldg(list + j) & 0x7fff;
        return e < G.nQ && abs(e / G.tiles_per_frame - ts) <= G.rte ? e : slot;
    };

    if (tid == 32) {
        mbar_init(q_full, 1);
        for (int i = 0; i < C::KST; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < C::VST; ++i) { mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1); }
        mbar_init(&s_full[0], 1); mbar_init(&s_full[1], 1);
        mbar_init(dp_full, 1); mbar_init(dp_read, 256); mbar_init(ds_full, 256);
        mbar_init(done, 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 9) { tmem_alloc(s_tmem, 512); tmem_relinquish(); }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    constexpr uint32_t COL_DP = 256, COL_DQ = 384;

    if (warp >= 8) {
        regs_dec<C::REGS_OTHER>();
        if (warp == 8) {
            if (n > 0 && elect_one()) {
                prefetch_tmap(&tm_q); prefetch_tmap(&tm_k); prefetch_tmap(&tm_v); prefetch_tmap(&tm_do);
                mbar_arrive_expect_tx(q_full, 2 * C::TILE);
#pragma unroll
                for (int p = 0; p < C::NP; ++p) {
                    load_panel(smem + C::OFF_Q + p * C::PANEL, &tm_q, G, p, g, slot, q_full);
                    load_panel(smem + C::OFF_DO + p * C::PANEL, &tm_do, G, p, g, slot, q_full);
                }
                int iss_k = 0, iss_v = 0;
                for (int j = 0; j < n; ++j) {
                    const int kt = entry(j);
                    const int ks = j % C::KST, vs = j % C::VST;
                    if (j >= C::KST && !role_wait(&k_empty[ks], ((j / C::KST) - 1) & 1, G.wait_ns, s_abort)) break;
                    mbar_arrive_expect_tx(&k_full[ks], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_K + ks * C::TILE + p * C::PANEL, &tm_k, G, p, g, kt, &k_full[ks]);
                    ++iss_k;
                    if (j >= C::VST && !role_wait(&v_empty[vs], ((j / C::VST) - 1) & 1, G.wait_ns, s_abort)) break;
                    mbar_arrive_expect_tx(&v_full[vs], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_V + vs * C::TILE + p * C::PANEL, &tm_v, G, p, g, kt, &v_full[vs]);
                    ++iss_v;
                }
                mbar_wait(q_full, 0, G.drain_ns);
                for (int j = max(0, iss_k - C::KST); j < iss_k; ++j) mbar_wait(&k_full[j % C::KST], (j / C::KST) & 1, G.drain_ns);
                for (int j = max(0, iss_v - C::VST); j < iss_v; ++j) mbar_wait(&v_full[j % C::VST], (j / C::VST) & 1, G.drain_ns);
            }
        } else if (warp == 9) {
            if (n > 0 && elect_one()) {
                constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false);
                constexpr uint32_t IDESC_G = idesc_bf16_f32(128, D, true);
                const uint32_t sQ = smem_u32(smem + C::OFF_Q), sD = smem_u32(smem + C::OFF_DO);
                const uint32_t sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
                auto scores = [&](uint32_t col, uint32_t a, uint32_t b) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::PANEL + (kk & 3) * 32;
                        mma_ss(tmem + col, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
                    }
                };
                auto issue_s = [&](int j) -> bool {
                    if (!role_wait(&k_full[j % C::KST], (j / C::KST) & 1, G.wait_ns, s_abort)) return false;
                    tc_fence_after();
                    scores((j & 1) * 128, sQ, sK + (j % C::KST) * C::TILE);
                    mma_commit(&s_full[j & 1]);
                    return true;
                };
                auto issue_dp = [&](int j) -> bool {
                    if (!role_wait(&v_full[j % C::VST], (j / C::VST) & 1, G.wait_ns, s_abort)) return false;
                    tc_fence_after();
                    scores(COL_DP, sD, sV + (j % C::VST) * C::TILE);
                    mma_commit(dp_full);
                    mma_commit(&v_empty[j % C::VST]);
                    return true;
                };
                bool ok = role_wait(q_full, 0, G.wait_ns, s_abort) && issue_s(0) && issue_dp(0) && (n < 2 || issue_s(1));
                for (int j = 0; ok && j < n; ++j) {
                    if (j + 1 < n) {
                        if (!role_wait(dp_read, j & 1, G.wait_ns, s_abort)) break;
                        if (!issue_dp(j + 1)) break;
                    }
                    if (!role_wait(ds_full, j & 1, G.wait_ns, s_abort)) break;
                    tc_fence_after();
                    const uint32_t col = (j & 1) * 128, b = sK + (j % C::KST) * C::TILE;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + COL_DQ, tmem + col + (kk >> 2) * 64 + (kk & 3) * 8,
                               smem_desc_sw128(b + kk * 2048, C::PANEL, 1024), IDESC_G, (j > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&k_empty[j % C::KST]);
                    if (j + 2 < n && !issue_s(j + 2)) break;
                }
                mma_commit(done);
                mbar_wait(done, 0, G.drain_ns);
            }
        }
    } else {
        regs_inc<C::REGS_SOFTMAX>();
        // ------------------------------------------------ dS
        const int u = warp >> 2;                             // keys 64u .. 64u + 63 of a tile
        const int row = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const float4 meta = __ldg(A.rows + ((size_t)g * G.nQ + slot) * 128 + row);
        const int pos = __float_as_int(meta.z), rq = __float_as_int(meta.w);
        const int hq = pos & 255, wq = (pos >> 8) & 255;
        const f2_t sc2 = f2_pack(G.scale_log2, G.scale_log2);
        const f2_t nd2 = f2_pack(-meta.y, -meta.y);
        constexpr int KR = 64 >> TWL;                        // key rows of a half tile
        constexpr int CP = TW / 2;                           // column pairs of a key row
        // The list's entries come one tile ahead (a load from global memory and
        // the divisions and fp64 half-width of a tile took 1200 of 3250 cycles
        // in front of each tile): coordinates by multiplication, exact since
        // x < 2^15 and the product's error, x / n 2^-22, is below the 0.5 / n to
        // the next integer; the half-width only when the key frame changes.
        const float inv_tpf = 1.f / (float)G.tiles_per_frame, inv_ntw = 1.f / (float)G.nTw;
        int e_next = n > 0 ? __ldg(list) & 0x7fff : 0;
        int s_frame = -1, s = 0;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int e = e_next;
            if (j + 1 < n) e_next = __ldg(list + j + 1) & 0x7fff;
            const int tk = (int)(((float)e + 0.5f) * inv_tpf), rem = e - tk * G.tiles_per_frame;
            const int trk = (int)(((float)rem + 0.5f) * inv_ntw), tck = rem - trk * G.nTw;
            const bool reach = e < G.nQ && abs(tk - ts) <= G.rte;
            if (tk != s_frame) {
                s_frame = tk;
                s = reach && rq >= 0 ? min(halfwidth(rq, G.g[abs(tk - ts)]), TRA_DISK_S_CLAMP) : 0;
            }
            const int h0 = trk * G.th + u * KR, w0 = tck * TW;
            const int khv = min(KR, G.H - h0), kwv = min(TW, G.W - w0);   // khv may be <= 0: a half past the grid's edge
            int a_lo = max(0, hq - s - h0), a_hi = min(khv - 1, hq + s - h0);
            const int b_lo = max(0, wq - s - w0), b_hi = min(kwv - 1, wq + s - w0);
            if (rq < 0 || !reach) { a_lo = 1; a_hi = 0; }
            const float nl = -meta.x;
            f2_t colb[CP];
            int cdw2[DISK ? TW : 1];
            if constexpr (DISK) {
#pragma unroll
                for (int b = 0; b < TW; ++b) {
                    const int dw = w0 + b - wq;
                    cdw2[b] = b < kwv ? dw * dw : INT_MAX;
                }
            } else {
#pragma unroll
                for (int bp = 0; bp < CP; ++bp)
                    colb[bp] = f2_pack((2 * bp >= b_lo && 2 * bp <= b_hi) ? 0.f : -INFINITY,
                                       (2 * bp + 1 >= b_lo && 2 * bp + 1 <= b_hi) ? 0.f : -INFINITY);
            }
            const uint32_t colS = tmem + lane_base + (j & 1) * 128 + u * 64, colP = tmem + lane_base + COL_DP + u * 64;
            bool got = role_wait(&s_full[j & 1], (j >> 1) & 1, G.wait_ns, s_abort);
            if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            uint32_t v[2][32];
            tmem_ld32(colS, v[0]);
            tmem_ld32(colS + 32, v[1]);
            tmem_wait_ld();
            f2_t p[32];
#pragma unroll
            for (int a = 0; a < KR; ++a) {
                const float rb = (a >= a_lo && a <= a_hi) ? nl : -INFINITY;
                const f2_t rb2 = f2_pack(rb, rb);
                const int dh = h0 + a - hq;
                const int thr = s * s - dh * dh;
#pragma unroll
                for (int bp = 0; bp < CP; ++bp) {
                    const int i = a * CP + bp, c = i >> 4, o = (2 * i) & 31;
                    float x0, x1;
                    const f2_t x = f2_fma(f2_pack(__uint_as_float(v[c][o]), __uint_as_float(v[c][o + 1])), sc2, rb2);
                    if constexpr (DISK) {
                        f2_unpack(x, x0, x1);
                        x0 = cdw2[2 * bp] <= thr ? x0 : -INFINITY;
                        x1 = cdw2[2 * bp + 1] <= thr ? x1 : -INFINITY;
                    } else {
                        f2_unpack(f2_add(x, colb[bp]), x0, x1);
                    }
                    p[i] = f2_pack(ex2(x0), ex2(x1));
                }
            }
            got = role_wait(dp_full, j & 1, G.wait_ns, s_abort);
            if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            tmem_ld32(colP, v[0]);
            tmem_ld32(colP + 32, v[1]);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(dp_read);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x0, x1;
                    f2_unpack(f2_mul(p[c * 16 + i], f2_add(f2_pack(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1])), nd2)), x0, x1);
                    pk[i] = pack_bf16x2(x0, x1);
                }
                tmem_st16(colS + c * 16, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(ds_full);
        }
        if (ok) ok = n == 0 || role_wait(done, 0, G.wait_ns, s_abort);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            __syncwarp();
            // this row's token: with query groups any row of the slot's strip
            int t, tr, tc;
            tile_coords(G, slot, t, tr, tc);
            int i = row;
            bool named = true;
            if (G.qsort) {
                const int l = reinterpret_cast<const uint16_t*>(A.mask + G.off_group)[((size_t)g * G.nQ + slot) * 128 + row];
                named = l < 128 * G.nTh;
                tr = l >> 7;
                i = l & 127;
            }
            const bool store = named && (!G.natural || (tr * G.th + (i >> TWL) < G.H && tc * TW + (i & (TW - 1)) < G.W));
            const size_t orow = store ? io_row(G, g, t, tr * G.th + (i >> TWL), tc * TW + (i & (TW - 1)),
                                               ((t * G.nTh + tr) * G.nTw + tc) * 128 + i) * D : 0;
            // each warpgroup writes its half of the columns
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld32(tmem + lane_base + COL_DQ + u * (D / 2) + c * 32, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = 0u;
                }
                if (store) store_cols32(A.dq, A.out_bf16 != 0, orow + u * (D / 2) + c * 32, v, A.grad_scale);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Both in one launch, the longer key tiles (z = 0) first: neither needs the other,
// a small grid has more CTAs to run at once, and the query slots fill the tail of
// the key tiles.  A grid of little more CTAs than SMs pays for the last ones: at
// 5 x 17 x 23, 3 heads, two of 150 CTAs, query slots, start only when another slot
// has ended, and two slots in a row outlast one key tile.
// Tensor-bound on the tiles it computes: at 21 x 45 x 80, 4 heads, d = 128, sorted
// groups, 462 241 tile pairs of 7 products take 10.3 ms, 1.32 PFLOP/s (0.94 of
// what a plain bf16 product sustains on this card); one part alone takes 3280
// (dK, dV: 2176 of products) and 2390 cycles a pair (dQ: 1536).  A third of a
// pair's elements are kept there, so the rate over kept pairs is 0.30 PFLOP/s of
// the 5 products that the gradients need.
template <int D, int TWL, bool DISK>
__global__ void __launch_bounds__(384, 1)
backward_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ Geom G, const __grid_constant__ BwdArgs A)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if (blockIdx.z == 0) backward_kv<D, TWL, DISK>(smem, tm_q, tm_k, tm_v, tm_do, G, A);
    else backward_q<D, TWL, DISK>(smem, tm_q, tm_k, tm_v, tm_do, G, A);
}

}  // namespace tra
