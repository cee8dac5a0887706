// backward.cuh -- the gradients of tra_attention, probabilities recomputed.
//
// With x_ij = q_i.k_j / sqrt d over the kept pairs, P_ij = exp(x_ij - lse_i),
// dP_ij = dO_i.v_j and D_i = dO_i.O_i:
//     dS_ij = P_ij (dP_ij - D_i)
//     dV_j = sum_i P_ij dO_i,  dK_j = sum_i dS_ij q_i / sqrt d,
//     dQ_i = sum_j dS_ij k_j / sqrt d.
// Four launches after a memset of the tile bitmaps:
//   backward_rows   D_i, the log2-domain lse and the grid position of every
//                   query row in mask-slot order; dO (and with query groups Q)
//                   copied to that order where the caller's rows cannot be
//                   read by TMA as they are
//   transpose_lists the mask's key-tile lists as bits per (key tile, query slot)
//   backward_kv     one CTA per key tile: dK and dV over the query slots that
//                   list it
//   backward_q      one CTA per query slot: dQ over its key tiles
// S and dP are computed in both of the last two (7 products per tile pair where
// 5 would do with dQ added up across CTAs): every output row is then written
// once, by one CTA, with a fixed order of summation, so the gradients are
// bit-identical from run to run, no fp32 dQ buffer is needed, and neither
// kernel moves P or dS through shared memory: each keeps the rows it sums over
// in the tensor memory's columns and the rows it owns in its lanes.
// P and dS are rounded to bf16 for the tensor cores (at most 2^-8 of each
// value, as P in the forward pass); all sums are fp32.
#pragma once
#include <cuda_bf16.h>

#include "pipeline.cuh"

namespace tra {

// What the two gradient kernels read besides the tensor maps.
struct BwdArgs {
    const uint8_t* mask;
    const float4* rows;          // [heads][nQ][128] slot order: lse * log2 e, D_i, h | w << 8 (bits), radius (bits)
    const uint32_t* bits;        // [heads][nQ key tiles][bw]: bit q - first(key tile) = slot q lists the tile
    int bw;
    int q_natural, do_natural;   // Q / dO read from the caller's natural rows (else [heads][N_pad] rows in slot order)
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

__device__ __forceinline__ void load_panel(void* dst, const CUtensorMap* m, bool natural, const Geom& G, int p, int g,
                                           int tile, uint64_t* bar)
{
    if (natural) {
        int t, tr, tc;
        tile_coords(G, tile, t, tr, tc);
        tma_load_4d(dst, m, p * 64, tc * G.tw, tr * G.th, g * G.T + t, bar);
    } else {
        tma_load_2d(dst, m, p * 64, g * G.N_pad + tile * 128, bar);
    }
}

// ------------------------------------------------------------------ row data
// One warp per row of a mask slot.  IN_F32: dout and out are fp32 (else bf16).
// dO is rounded to bf16 first and D_i taken from the rounded values, the ones
// the products use.  HBM-bound.
template <int D, bool IN_F32>
__global__ void __launch_bounds__(256)
backward_rows_kernel(const Geom G, const uint8_t* __restrict__ mask, const void* __restrict__ out,
                     const void* __restrict__ dout, const float* __restrict__ lse, const uint4* __restrict__ q,
                     float4* __restrict__ rows, uint32_t* __restrict__ q_copy, uint32_t* __restrict__ do_copy)
{
    const int lane = threadIdx.x & 31;
    const size_t p = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);     // head, slot, row
    if (p >= (size_t)G.G * G.N_pad) return;
    const int g = (int)(p / G.N_pad);
    const int in = (int)(p - (size_t)g * G.N_pad);
    const int slot = in >> 7;
    int t, tr, tc, i = in & 127;
    tile_coords(G, slot, t, tr, tc);
    bool ok = true;
    if (G.qsort) {
        int l = reinterpret_cast<const uint16_t*>(mask + G.off_group)[p];
        if (l >= 128 * G.nTh) {                                       // caller memory: recorded, the row left out
            if (lane == 0) atomicOr(&g_tra_error, TRA_ERRBIT_CHECK);
            l = 0;
            ok = false;
        }
        tr = l >> 7;
        i = l & 127;
    }
    const int h = tr * G.th + (i >> G.tw_log2), w = tc * G.tw + (i & (G.tw - 1));
    ok = ok && h < G.H && w < G.W;
    const int trow = ((t * G.nTh + tr) * G.nTw + tc) * 128 + i;       // tile-major row of the token
    const size_t src = ok ? io_row(G, g, t, h, w, trow) : 0;
    constexpr int PAIRS = D / 64;                                     // bf16 pairs per lane
    float d = 0.f;
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
        const size_t at = src * (D / 2) + k * 32 + lane;
        uint32_t bits = 0;
        float o0 = 0.f, o1 = 0.f;
        if (ok) {
            if constexpr (IN_F32) {
                const float2 x = static_cast<const float2*>(dout)[at], o = static_cast<const float2*>(out)[at];
                bits = pack_bf16x2(x.x, x.y);
                o0 = o.x;
                o1 = o.y;
            } else {
                bits = static_cast<const uint32_t*>(dout)[at];
                const uint32_t o = static_cast<const uint32_t*>(out)[at];
                o0 = __uint_as_float(o << 16);
                o1 = __uint_as_float(o & 0xffff0000u);
            }
        }
        d = fmaf(__uint_as_float(bits << 16), o0, d);
        d = fmaf(__uint_as_float(bits & 0xffff0000u), o1, d);
        if (do_copy) do_copy[p * (D / 2) + k * 32 + lane] = bits;
        if (q_copy) q_copy[p * (D / 2) + k * 32 + lane] = ok ? reinterpret_cast<const uint32_t*>(q)[at] : 0u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) {
        int r = ok ? reinterpret_cast<const int32_t*>(mask + G.off_radius)[(size_t)g * G.N_pad + trow] : -1;
        float l2 = 0.f;
        if (ok) {
            l2 = lse[src] * 1.4426950408889634f;
            if (l2 == -INFINITY) { l2 = 0.f; r = -1; }                // a row that kept nothing
        }
        rows[p] = make_float4(l2, ok ? d : 0.f, __int_as_float(h | (w << 8)), __int_as_float(r));
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
// Keep-bits of a query at (hq, wq) with half-width s over a key tile at (h0, w0)
// with khv x kwv valid keys, as four 32-key words.
template <int TWL, bool DISK>
__device__ __forceinline__ void query_keep_bits(const Geom& G, int hq, int wq, int s, int h0, int w0, int khv, int kwv,
                                                uint32_t (&m)[4])
{
    constexpr int TW = 1 << TWL;
    if constexpr (!DISK) {
        row_keep_bits<TWL>(max(0, hq - s - h0), min(khv - 1, hq + s - h0), max(0, wq - s - w0), min(kwv - 1, wq + s - w0), m);
    } else {
#pragma unroll
        for (int wd = 0; wd < 4; ++wd) {
            uint32_t v = 0;
#pragma unroll
            for (int k = 0; k < 32 / TW; ++k) {
                const int a = (wd * 32) / TW + k, dh = h0 + a - hq, thr = s * s - dh * dh;
                if (a < khv && thr >= 0) {
                    const int half = isqrt_floor(thr);
                    const int lo = max(0, wq - half - w0), hi = min(kwv - 1, wq + half - w0);
                    if (lo <= hi) v |= ((2u << hi) - (1u << lo)) << ((a * TW) & 31);
                }
            }
            m[wd] = v;
        }
    }
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
//   warp 9     MMA issuer.  Each half of a slot is a chain of its own:
//              {dV += P^T dO, S^T of slot j+1} once P^T of slot j is there, and
//              {dK += dS^T Q, dP^T of slot j+1} once dS^T is; the groups of the
//              two halves alternate, so one half's elementwise work runs
//              under the other's products.  MMAs of one thread run in order,
//              so S^T of j+1 overwrites P^T of j only after dV has read it, and
//              dP^T of j+1 overwrites dS^T of j only after dK has.
//   warps 10, 11  per slot, the 64 queries' lse and D_i and the keep-bits of
//              all 128 keys into a two-stage ring (and whether all are set:
//              such halves skip the masking).
// TMEM columns: S^T [0,128), dP^T [128,256), dV [256,256+D), dK [384,384+D).
// P^T of warpgroup u: bf16 pairs in columns 64u .. 64u+31 (its own half of
// S^T, so the other half's S^T is never overwritten early); dS^T likewise.
template <int D>
struct BwdKvCfg {
    static constexpr int PANEL = 128 * 128;
    static constexpr int NP = D / 64;
    static constexpr int TILE = NP * PANEL;
    static constexpr int ST = 2;                            // Q and dO ring depth
    static constexpr int OFF_K = 0, OFF_V = TILE;
    static constexpr int OFF_Q = 2 * TILE, OFF_DO = OFF_Q + ST * TILE;
    static constexpr int OFF_META = OFF_DO + ST * TILE;     // [ST][2 halves]: -lse[64], -D[64], words[4][64]
    static constexpr int META = 64 * 4 * 6;                 // bytes of a half
    static constexpr int OFF_BARS = OFF_META + ST * 2 * META;
    static constexpr int OFF_LIST = OFF_BARS + 32 * 8 + 64; // uint16 [list_cap]
    static constexpr int THREADS = 384;
    static constexpr int REGS_SOFTMAX = 216, REGS_OTHER = 72;
    static int smem(int list_cap) { return OFF_LIST + ((list_cap * 2 + 15) & ~15) + 1024; }
};

template <int D, int TWL, bool DISK>
__global__ void __launch_bounds__(384, 1)
backward_kv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const Geom G,
                   const BwdArgs A)
{
    using C = BwdKvCfg<D>;
    constexpr int TW = 1 << TWL;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
    uint64_t* kv_full = bars;
    uint64_t* q_full = bars + 1;                 // [ST]
    uint64_t* q_empty = q_full + C::ST;
    uint64_t* do_full = q_empty + C::ST;
    uint64_t* do_empty = do_full + C::ST;
    uint64_t* meta_full = do_empty + C::ST;      // [ST][2]
    uint64_t* meta_empty = meta_full + 2 * C::ST;
    uint64_t* s_full = meta_empty + 2 * C::ST;   // [2], as the following: one per half
    uint64_t* dp_full = s_full + 2;
    uint64_t* p_full = dp_full + 2;
    uint64_t* ds_full = p_full + 2;
    uint64_t* done = ds_full + 2;
    int* misc = reinterpret_cast<int*>(bars + 32);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc);
    volatile int* s_abort = misc + 1;
    int* s_n = misc + 2;
    int* s_all = misc + 4;                       // [ST][2]: every pair of the half is kept
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
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1);
            mbar_init(&do_full[i], 1); mbar_init(&do_empty[i], 1);
        }
        for (int i = 0; i < 2 * C::ST; ++i) { mbar_init(&meta_full[i], 32); mbar_init(&meta_empty[i], 128); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1); mbar_init(&dp_full[i], 1);
            mbar_init(&p_full[i], 128); mbar_init(&ds_full[i], 128);
        }
        mbar_init(done, 1);
        *s_abort = 0;
        fence_barrier_init();
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
                int iss_q = 0, iss_do = 0;
                auto load_q = [&](int j) -> bool {
                    const int st = j % C::ST;
                    if (j >= C::ST && !role_wait(&q_empty[st], ((j / C::ST) - 1) & 1, G.wait_ns, s_abort)) return false;
                    mbar_arrive_expect_tx(&q_full[st], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_Q + st * C::TILE + p * C::PANEL, &tm_q, A.q_natural, G, p, g, list[j], &q_full[st]);
                    ++iss_q;
                    return true;
                };
                auto load_do = [&](int j) -> bool {
                    const int st = j % C::ST;
                    if (j >= C::ST && !role_wait(&do_empty[st], ((j / C::ST) - 1) & 1, G.wait_ns, s_abort)) return false;
                    mbar_arrive_expect_tx(&do_full[st], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_DO + st * C::TILE + p * C::PANEL, &tm_do, A.do_natural, G, p, g, list[j], &do_full[st]);
                    ++iss_do;
                    return true;
                };
                mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
#pragma unroll
                for (int p = 0; p < C::NP; ++p) {
                    load_panel(smem + C::OFF_K + p * C::PANEL, &tm_k, G.natural, G, p, g, kt, kv_full);
                    load_panel(smem + C::OFF_V + p * C::PANEL, &tm_v, G.natural, G, p, g, kt, kv_full);
                }
                // dO's stage is free half a step before Q's of the same slot
                for (int j = 0; j < n; ++j)
                    if (!(j < C::ST ? load_q(j) && load_do(j) : load_do(j) && load_q(j))) break;
                // copies still in flight must land before the CTA exits
                mbar_wait(kv_full, 0, G.drain_ns);
                for (int j = max(0, iss_q - C::ST); j < iss_q; ++j) mbar_wait(&q_full[j % C::ST], (j / C::ST) & 1, G.drain_ns);
                for (int j = max(0, iss_do - C::ST); j < iss_do; ++j) mbar_wait(&do_full[j % C::ST], (j / C::ST) & 1, G.drain_ns);
            }
        } else if (warp == 9) {
            if (n > 0 && elect_one()) {
                constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64, false);
                constexpr uint32_t IDESC_G = idesc_bf16_f32(128, D, true);
                const uint32_t sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
                const uint32_t sQ = smem_u32(smem + C::OFF_Q), sD = smem_u32(smem + C::OFF_DO);
                // A (keys) times B^T (the 64 queries of half u), both K-major
                auto scores = [&](uint32_t col, uint32_t a, uint32_t b, int u) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::PANEL + (kk & 3) * 32;
                        mma_ss(tmem + col + u * 64, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off + u * 8192, 16, 1024),
                               IDESC_S, kk > 0 ? 1u : 0u);
                    }
                };
                // the bf16 pairs in half u of `col` times the 64 rows of half u of b
                auto accumulate = [&](uint32_t dst, uint32_t col, uint32_t b, int u, bool add) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts(tmem + dst, tmem + col + u * 64 + kk * 8,
                               smem_desc_sw128(b + u * 8192 + kk * 2048, C::PANEL, 1024), IDESC_G, (add || kk > 0) ? 1u : 0u);
                };
                bool ok = role_wait(kv_full, 0, G.wait_ns, s_abort) && role_wait(&q_full[0], 0, G.wait_ns, s_abort);
                if (ok) {
                    tc_fence_after();
                    for (int u = 0; u < 2; ++u) {
                        scores(COL_S, sK, sQ, u);
                        mma_commit(&s_full[u]);
                    }
                    ok = role_wait(&do_full[0], 0, G.wait_ns, s_abort);
                }
                if (ok) {
                    for (int u = 0; u < 2; ++u) {
                        scores(COL_DP, sV, sD, u);
                        mma_commit(&dp_full[u]);
                    }
                }
                for (int j = 0; ok && j < n; ++j) {
                    const int st = j % C::ST, sn = (j + 1) % C::ST;
                    const bool next = j + 1 < n;
                    for (int u = 0; ok && u < 2; ++u) {
                        ok = role_wait(&p_full[u], j & 1, G.wait_ns, s_abort);
                        if (!ok) break;
                        tc_fence_after();
                        accumulate(COL_DV, COL_S, sD + st * C::TILE, u, j > 0 || u > 0);
                        if (u == 1) mma_commit(&do_empty[st]);
                        if (!next) continue;
                        if (u == 0) ok = role_wait(&q_full[sn], ((j + 1) / C::ST) & 1, G.wait_ns, s_abort);
                        if (!ok) break;
                        scores(COL_S, sK, sQ + sn * C::TILE, u);
                        mma_commit(&s_full[u]);
                    }
                    for (int u = 0; ok && u < 2; ++u) {
                        ok = role_wait(&ds_full[u], j & 1, G.wait_ns, s_abort);
                        if (!ok) break;
                        tc_fence_after();
                        accumulate(COL_DK, COL_DP, sQ + st * C::TILE, u, j > 0 || u > 0);
                        if (u == 1) mma_commit(&q_empty[st]);
                        if (!next) continue;
                        if (u == 0) ok = role_wait(&do_full[sn], ((j + 1) / C::ST) & 1, G.wait_ns, s_abort);
                        if (!ok) break;
                        scores(COL_DP, sV, sD + sn * C::TILE, u);
                        mma_commit(&dp_full[u]);
                    }
                }
                // every issued MMA must finish before the results are read and TMEM is freed
                mma_commit(done);
                mbar_wait(done, 0, G.drain_ns);
            }
        } else {
            // ------------------------------------------------ queries' lse, D_i and keep-bits
            const int half = warp - 10;
            for (int j = 0; j < n; ++j) {
                const int st = j % C::ST, ring = st * 2 + half;
                const int slot = list[j];
                const float4* src = A.rows + ((size_t)g * G.nQ + slot) * 128 + half * 64 + lane;
                const float4 r0 = __ldg(src), r1 = __ldg(src + 32);
                const double decay = G.g[abs(slot / G.tiles_per_frame - tk)];
                uint32_t m[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int pos = __float_as_int(x ? r1.z : r0.z), r = __float_as_int(x ? r1.w : r0.w);
                    if (r >= 0)
                        query_keep_bits<TWL, DISK>(G, pos & 255, (pos >> 8) & 255, min(halfwidth(r, decay), TRA_DISK_S_CLAMP), h0, w0, khv, kwv, m[x]);
                    else
                        m[x][0] = m[x][1] = m[x][2] = m[x][3] = 0u;
                }
                const bool all = __all_sync(0xffffffffu, (m[0][0] & m[0][1] & m[0][2] & m[0][3] & m[1][0] & m[1][1] & m[1][2] & m[1][3]) == 0xffffffffu);
                bool got = true;
                if (j >= C::ST) got = role_wait(&meta_empty[ring], ((j / C::ST) - 1) & 1, G.wait_ns, s_abort);
                if (__any_sync(0xffffffffu, !got)) break;
                float* f = reinterpret_cast<float*>(smem + C::OFF_META + ring * C::META);
                uint32_t* wd = reinterpret_cast<uint32_t*>(f + 128);
                f[lane] = -r0.x; f[lane + 32] = -r1.x;
                f[64 + lane] = -r0.y; f[96 + lane] = -r1.y;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    wd[k * 64 + lane] = m[0][k];
                    wd[k * 64 + lane + 32] = m[1][k];
                }
                if (lane == 0) s_all[ring] = all ? 1 : 0;
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
        const uint32_t lbit = 1u << lane;
        const f2_t sc2 = f2_pack(G.scale_log2, G.scale_log2);
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int ring = (j % C::ST) * 2 + u;
            bool got = role_wait(&meta_full[ring], (j / C::ST) & 1, G.wait_ns, s_abort);
            got = got && role_wait(&s_full[u], j & 1, G.wait_ns, s_abort);
            if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            const ulonglong2* lse2 = reinterpret_cast<const ulonglong2*>(smem + C::OFF_META + ring * C::META);
            const ulonglong2* dd2 = lse2 + 16;
            const uint4* wd4 = reinterpret_cast<const uint4*>(lse2 + 32) + (warp & 3) * 16;
            const bool all = s_all[ring] != 0;
            uint32_t v[2][32];
            tmem_ld32(colS, v[0]);
            tmem_ld32(colS + 32, v[1]);
            tmem_wait_ld();
            f2_t p[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 l = lse2[c * 8 + i];
                    float x0, x1, x2, x3;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c][4 * i]), __uint_as_float(v[c][4 * i + 1])), sc2, l.x), x0, x1);
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c][4 * i + 2]), __uint_as_float(v[c][4 * i + 3])), sc2, l.y), x2, x3);
                    if (!all) {
                        const uint4 m = wd4[c * 8 + i];
                        x0 = (m.x & lbit) ? x0 : -INFINITY;
                        x1 = (m.y & lbit) ? x1 : -INFINITY;
                        x2 = (m.z & lbit) ? x2 : -INFINITY;
                        x3 = (m.w & lbit) ? x3 : -INFINITY;
                    }
                    x0 = ex2(x0); x1 = ex2(x1); x2 = ex2(x2); x3 = ex2(x3);
                    p[c * 16 + 2 * i] = f2_pack(x0, x1);
                    p[c * 16 + 2 * i + 1] = f2_pack(x2, x3);
                    pk[2 * i] = pack_bf16x2(x0, x1);
                    pk[2 * i + 1] = pack_bf16x2(x2, x3);
                }
                tmem_st16(colS + c * 16, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[u]);
            got = role_wait(&dp_full[u], j & 1, G.wait_ns, s_abort);
            if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
            tc_fence_after();
            __syncwarp();
            tmem_ld32(colP, v[0]);
            tmem_ld32(colP + 32, v[1]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 dd = dd2[c * 8 + i];
                    float x0, x1, x2, x3;
                    f2_unpack(f2_mul(p[c * 16 + 2 * i], f2_add(f2_pack(__uint_as_float(v[c][4 * i]), __uint_as_float(v[c][4 * i + 1])), dd.x)), x0, x1);
                    f2_unpack(f2_mul(p[c * 16 + 2 * i + 1], f2_add(f2_pack(__uint_as_float(v[c][4 * i + 2]), __uint_as_float(v[c][4 * i + 3])), dd.y)), x2, x3);
                    pk[2 * i] = pack_bf16x2(x0, x1);
                    pk[2 * i + 1] = pack_bf16x2(x2, x3);
                }
                tmem_st16(colP + c * 16, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&ds_full[u]);
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
    static constexpr int THREADS = 384;
    static constexpr int REGS_SOFTMAX = 216, REGS_OTHER = 72;
    static int smem() { return BYTES + 1024; }
};

template <int D, int TWL, bool DISK>
__global__ void __launch_bounds__(384, 1)
backward_q_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const Geom G,
                  const BwdArgs A)
{
    using C = BwdQCfg<D>;
    constexpr int TW = 1 << TWL;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ts = slot / G.tiles_per_frame;
    int n = reinterpret_cast<const int32_t*>(A.mask + G.off_count)[(size_t)g * G.nQ + slot];
    if (n < 0 || n > G.list_cap) n = 0;          // recorded by transpose_lists
    const uint16_t* list = reinterpret_cast<const uint16_t*>(A.mask + G.off_list) + ((size_t)g * G.nQ + slot) * G.list_cap;
    // a listed tile out of reach (recorded by transpose_lists) is replaced by
    // the slot's own tile with every pair masked
    auto entry = [&](int j, bool& reach) -> int {
        const int e = __ldg(list + j) & 0x7fff;
        reach = e < G.nQ && abs(e / G.tiles_per_frame - ts) <= G.rte;
        return reach ? e : slot;
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
                    load_panel(smem + C::OFF_Q + p * C::PANEL, &tm_q, A.q_natural, G, p, g, slot, q_full);
                    load_panel(smem + C::OFF_DO + p * C::PANEL, &tm_do, A.do_natural, G, p, g, slot, q_full);
                }
                int iss_k = 0, iss_v = 0;
                for (int j = 0; j < n; ++j) {
                    bool reach;
                    const int kt = entry(j, reach);
                    const int ks = j % C::KST, vs = j % C::VST;
                    if (j >= C::KST && !role_wait(&k_empty[ks], ((j / C::KST) - 1) & 1, G.wait_ns, s_abort)) break;
                    mbar_arrive_expect_tx(&k_full[ks], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_K + ks * C::TILE + p * C::PANEL, &tm_k, G.natural, G, p, g, kt, &k_full[ks]);
                    ++iss_k;
                    if (j >= C::VST && !role_wait(&v_empty[vs], ((j / C::VST) - 1) & 1, G.wait_ns, s_abort)) break;
                    mbar_arrive_expect_tx(&v_full[vs], C::TILE);
#pragma unroll
                    for (int p = 0; p < C::NP; ++p)
                        load_panel(smem + C::OFF_V + vs * C::TILE + p * C::PANEL, &tm_v, G.natural, G, p, g, kt, &v_full[vs]);
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
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            bool reach;
            const int kt = entry(j, reach);
            int tk, trk, tck;
            tile_coords(G, kt, tk, trk, tck);
            const int h0 = trk * G.th + u * KR, w0 = tck * TW;
            const int khv = min(KR, G.H - h0), kwv = min(TW, G.W - w0);   // khv may be <= 0: a half past the grid's edge
            const int s = rq >= 0 ? min(halfwidth(rq, G.g[abs(tk - ts)]), TRA_DISK_S_CLAMP) : 0;
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

}  // namespace tra
