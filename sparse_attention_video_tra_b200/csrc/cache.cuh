// cache.cuh -- keys and values held in 8 bits, and attention over them.
//
// The cache holds the clip's K and V tile by tile: e4m3 codes with one
// power-of-two scale for each (head, tile), i.e. for each (1, th, tw) box of
// tokens.  A tile lies in one frame, so storing a frame never touches a tile of
// another one and no stored code is ever rescaled.  A power of two costs at
// most one bit of e4m3's 17 binades (codes reach at least 224 of 448) and
// makes every stored value exactly a bf16 number: the tensor-core kernel sees
// the same values as the scalar one.
#pragma once
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "pipeline.cuh"

namespace tra {

// pointers into the cache buffer
struct CacheView {
    uint8_t *k, *v;              // [heads][nQ][128][d] e4m3 codes
    float *ks, *vs;              // [heads][nQ] scales
};

// ------------------------------------------------------------------ store
// One CTA per (tile, head, K or V): the tile's largest magnitude, the scale
// 2^e with the smallest e >= -126 that brings it to at most 448 (2^0 for a tile
// of zeros), and the codes, round to nearest even.  Multiplying by 2^-e is
// exact, so each code is one rounding of its input.  Reads 2 and writes 1 byte
// per element: HBM-bound.
template <int D>
__global__ void __launch_bounds__(256)
cache_store_kernel(const Geom G, const uint4* __restrict__ k, const uint4* __restrict__ v, int frame, int frames,
                   const CacheView C)
{
    constexpr int CH = D / 8;                                // 16-byte chunks of a bf16 row
    constexpr int PER = 128 * CH / 256;                      // chunks per thread
    __shared__ uint32_t s_max[8];
    const int lt = blockIdx.x, g = blockIdx.y;               // tile among the stored frames
    const bool isV = blockIdx.z != 0;
    const uint4* src = isV ? v : k;
    const int tile = frame * G.tiles_per_frame + lt;
    int t, tr, tc;
    tile_coords(G, lt, t, tr, tc);
    uint4 x[PER];
    uint32_t most = 0;                                       // largest magnitude as bf16 bits
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int c = e * 256 + threadIdx.x, row = c / CH, ch = c - row * CH;
        const int h = tr * G.th + (row >> G.tw_log2), w = tc * G.tw + (row & (G.tw - 1));
        x[e] = make_uint4(0u, 0u, 0u, 0u);
        if (h < G.H && w < G.W) {
            const size_t r = G.natural ? ((size_t)g * frames + t) * (G.H * G.W) + h * G.W + w
                                       : ((size_t)g * frames * G.tiles_per_frame + lt) * 128 + row;
            x[e] = __ldg(src + r * CH + ch);
        }
        const uint32_t w4[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) most = max(most, max(w4[i] & 0x7fffu, (w4[i] >> 16) & 0x7fffu));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, s_max[i]);
    // magnitude 1.f * 2^E: 2^(E - 8) brings it to 256 * 1.f, one more when that is above 448 = 256 * 1.75
    int e2 = (int)(most >> 7) - 127 - 8 + ((most & 0x7fu) > 0x60u ? 1 : 0);
    e2 = most == 0 ? 0 : max(e2, -126);
    const float inv = __uint_as_float((uint32_t)(127 - e2) << 23);
    uint2* dst = reinterpret_cast<uint2*>((isV ? C.v : C.k) + ((size_t)g * G.nQ + tile) * 128 * D);
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const uint32_t w4[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo)
                : "f"(__uint_as_float(w4[2 * i] & 0xffff0000u) * inv), "f"(__uint_as_float(w4[2 * i] << 16) * inv));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi)
                : "f"(__uint_as_float(w4[2 * i + 1] & 0xffff0000u) * inv), "f"(__uint_as_float(w4[2 * i + 1] << 16) * inv));
            o[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
        dst[e * 256 + threadIdx.x] = make_uint2(o[0], o[1]);
    }
    if (threadIdx.x == 0) (isV ? C.vs : C.ks)[(size_t)g * G.nQ + tile] = __uint_as_float((uint32_t)(127 + e2) << 23);
}

// four codes as floats
__device__ __forceinline__ void codes_to_float(uint32_t w, float (&f)[4])
{
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(w & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(f[0]), "=f"(f[1]) : "r"(a));
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(f[2]), "=f"(f[3]) : "r"(b));
}

// ------------------------------------------------------------------ expand
// The tiles of the key frames [k0, k1) as bf16 rows [heads][(k1 - k0) tiles][128][d]
// for the tensor-core kernel; exact.  A key tile is read by tens of query
// tiles, so it is expanded once here (3 bytes of traffic per element, mostly in
// L2) rather than by every CTA that reads it.
template <int D>
__global__ void __launch_bounds__(256)
cache_expand_kernel(const Geom G, const CacheView C, int k0, int k1, uint4* __restrict__ k, uint4* __restrict__ v)
{
    constexpr int CH = D / 16;                               // 16-code chunks of a row
    const size_t tiles = (size_t)(k1 - k0) * G.tiles_per_frame;
    const size_t per_head = tiles * 128 * CH, total = per_head * G.G;
    const bool isV = blockIdx.y != 0;
    uint4* dst = isV ? v : k;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
        const size_t g = i / per_head, r = i - g * per_head;
        const size_t tile0 = g * G.nQ + (size_t)k0 * G.tiles_per_frame;
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(isV ? C.v : C.k) + tile0 * 128 * CH + r);
        const float s = __ldg((isV ? C.vs : C.ks) + tile0 + r / (128 * CH));
        const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[4];
            codes_to_float(w4[k], f);
            o[2 * k] = pack_bf16x2(f[0] * s, f[1] * s);
            o[2 * k + 1] = pack_bf16x2(f[2] * s, f[3] * s);
        }
        dst[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// ------------------------------------------------------------------ tokens
// Attention of single tokens over the cached frames: one cluster of `csize`
// CTAs per (token, head), 8 warps each, on the scalar units (one query row
// per key leaves a matrix unit idle in all but one row, and the codes have to
// come from memory either way).  The kept keys of all reachable frames are
// numbered through and dealt out to groups of d/16 lanes, 16 codes of K and of
// V per lane, d/16 keys at a time: each lane finds the address and scales of
// one of the keys, a batch's loads go out under the arithmetic of the one before
// (43 -> 29 us cold for 1 token and 40 heads at 21 x 45 x 80, 55 MB), and a
// butterfly leaves each lane with the score of its key.  Each group keeps a running
// maximum and sum; they are joined within the warp by shuffles, within the CTA
// through shared memory, and over the cluster through distributed shared
// memory, so one launch does it without a workspace.  All sums are fp32.
struct TokenFrame {
    int cum;                     // keys of the earlier frames
    int box;                     // h_lo | w_lo << 8 | (width - 1) << 16
    float inv_w;                 // 1 / width
    int s2;                      // s^2 (disk)
};

template <int D, bool DISK>
__global__ void __launch_bounds__(256)
token_attention_kernel(const Geom G, const CacheView C, const uint4* __restrict__ q, const int32_t* __restrict__ token,
                       const int32_t* __restrict__ radius, int n, int cached, int csize, void* __restrict__ out,
                       int out_bf16, float* __restrict__ lse)
{
    namespace cg = cooperative_groups;
    constexpr int LPK = D / 16, GPW = 32 / LPK;              // lanes per key, groups per warp
    __shared__ TokenFrame s_frame[2 * TRA_MAX_RT_EFF + 2];
    __shared__ int s_total;
    __shared__ float s_o[8][D], s_m[8], s_l[8];
    __shared__ float s_out[D], s_ml[2];

    const int unit = blockIdx.x / csize, rank = blockIdx.x - unit * csize;
    const int g = unit / n, i = unit - g * n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tok = token[i];
    if (tok < 0) return;                                     // an unused place: its rows stay as they were
    if (tok >= G.N) {
        if (tid == 0 && rank == 0) atomicOr(&g_tra_error, TRA_ERRBIT_CHECK);
        return;
    }
    const size_t row = (size_t)g * n + i;
    const int r = radius[row];
    const int area = G.H * G.W;
    const int tq = tok / area, hq = (tok - tq * area) / G.W, wq = tok - tq * area - hq * G.W;
    const int f0 = max(0, tq - G.rte), f1 = r < 0 ? f0 : max(f0, min(cached, tq + G.rte + 1));
    const int nf = f1 - f0;

    if (warp == 0) {
        int carry = 0;
        for (int b = 0; b < nf; b += 32) {
            const int f = b + lane;
            int cnt = 0, h_lo = 0, w_lo = 0, wid = 1, s = 0;
            if (f < nf) {
                s = min(halfwidth(r, G.g[abs(f0 + f - tq)]), TRA_DISK_S_CLAMP);
                h_lo = max(0, hq - s);
                w_lo = max(0, wq - s);
                wid = min(G.W - 1, wq + s) - w_lo + 1;
                cnt = (min(G.H - 1, hq + s) - h_lo + 1) * wid;
            }
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (f < nf) s_frame[f] = {carry + incl - cnt, h_lo | (w_lo << 8) | ((wid - 1) << 16), 1.f / (float)wid, s * s};
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            s_total = carry;
            s_frame[nf].cum = carry;
        }
    }
    __syncthreads();

    const int sub = lane % LPK;
    // this lane's 16 query elements
    f2_t qf[8];
    {
        const uint4 a = __ldg(q + row * (D / 8) + 2 * sub), b = __ldg(q + row * (D / 8) + 2 * sub + 1);
        const uint32_t w8[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) qf[k] = f2_pack(__uint_as_float(w8[k] << 16), __uint_as_float(w8[k] & 0xffff0000u));
    }
    const int total = s_total;
    const int groups = csize * 8 * GPW, gid = (rank * 8 + warp) * GPW + lane / LPK;
    const uint4* kc = reinterpret_cast<const uint4*>(C.k) + (size_t)g * G.N_pad * LPK + sub;
    const uint4* vc = reinterpret_cast<const uint4*>(C.v) + (size_t)g * G.N_pad * LPK + sub;
    f2_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 0ull;
    float m = -INFINITY, l = 0.f;
    int f = 0;
    // this lane's key of the batch that starts at e0: its row (-1: none) and scales
    auto locate = [&](int e0, int& at, float& ks, float& vs) {
        const int e = e0 + sub * groups + gid;
        at = -1;
        ks = vs = 0.f;
        if (e < total) {
            while (e >= s_frame[f + 1].cum) ++f;
            const TokenFrame F = s_frame[f];
            const int wid = (F.box >> 16) + 1, x = e - F.cum;
            // x / wid: x < 2^16, and the product's error (x / wid) 2^-22 is below the 0.5 / wid to the next integer
            const int dr = (int)(((float)x + 0.5f) * F.inv_w);
            const int h = (F.box & 255) + dr, w = ((F.box >> 8) & 255) + x - dr * wid;
            const int tile = ((f0 + f) * G.nTh + (h >> G.th_log2)) * G.nTw + (w >> G.tw_log2);
            if (!DISK || (h - hq) * (h - hq) + (w - wq) * (w - wq) <= F.s2) {
                at = tile * 128 + ((h & (G.th - 1)) << G.tw_log2) + (w & (G.tw - 1));
                ks = __ldg(C.ks + (size_t)g * G.nQ + tile);
                vs = __ldg(C.vs + (size_t)g * G.nQ + tile);
            }
        }
    };
    uint4 kk[LPK], vv[LPK];
    auto load = [&](const uint4* codes, int at, uint4 (&to)[LPK]) {
#pragma unroll
        for (int k = 0; k < LPK; ++k) {
            const int a = __shfl_sync(0xffffffffu, at, k, LPK);
            to[k] = a >= 0 ? __ldg(codes + (size_t)a * LPK) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    // the K codes of a batch arrive under the V arithmetic of the one before, and
    // its V codes under its own scores
    int at_n;
    float ks_n, vs_n;
    locate(0, at_n, ks_n, vs_n);
    load(kc, at_n, kk);
    load(vc, at_n, vv);
    for (int e0 = 0; e0 < total; e0 += groups * LPK) {
        const int at = at_n;
        const float ks = ks_n, vs = vs_n;
        locate(e0 + groups * LPK, at_n, ks_n, vs_n);
        float x[LPK];
#pragma unroll
        for (int k = 0; k < LPK; ++k) {
            const uint32_t w4[4] = {kk[k].x, kk[k].y, kk[k].z, kk[k].w};
            f2_t s0 = 0ull, s1 = 0ull;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[4];
                codes_to_float(w4[j], c);
                s0 = f2_fma(f2_pack(c[0], c[1]), qf[2 * j], s0);
                s1 = f2_fma(f2_pack(c[2], c[3]), qf[2 * j + 1], s1);
            }
            float a, b;
            f2_unpack(f2_add(s0, s1), a, b);
            x[k] = a + b;
        }
        load(kc, at_n, kk);
        // butterfly: after the step of distance d each lane keeps the keys whose bit d matches its own
#pragma unroll
        for (int d = LPK / 2; d > 0; d >>= 1) {
#pragma unroll
            for (int k = 0; k < d; ++k) {
                const bool up = (sub & d) != 0;
                const float send = up ? x[k] : x[k + d], keep = up ? x[k + d] : x[k];
                x[k] = keep + __shfl_xor_sync(0xffffffffu, send, d);
            }
        }
        const float sc = at >= 0 ? x[0] * (ks * G.scale_log2) : -INFINITY;
        float mx = sc;
#pragma unroll
        for (int d = LPK / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m - base), p = ex2(sc - base);
        m = mn;
        l = fmaf(l, alpha, p);                               // this lane's keys only; summed over the group at the end
        const f2_t al2 = f2_pack(alpha, alpha);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = f2_mul(o[k], al2);
        const float pv = p * vs;
#pragma unroll
        for (int k = 0; k < LPK; ++k) {
            const float a = __shfl_sync(0xffffffffu, pv, k, LPK);
            const f2_t a2 = f2_pack(a, a);
            const uint32_t w4[4] = {vv[k].x, vv[k].y, vv[k].z, vv[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[4];
                codes_to_float(w4[j], c);
                o[2 * j] = f2_fma(f2_pack(c[0], c[1]), a2, o[2 * j]);
                o[2 * j + 1] = f2_fma(f2_pack(c[2], c[3]), a2, o[2 * j + 1]);
            }
        }
        load(vc, at_n, vv);
    }
    // ---- join the groups of the warp
    float mw = m;
#pragma unroll
    for (int d = LPK; d < 32; d <<= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, d));
    const float fac = m == -INFINITY ? 0.f : ex2(m - mw);
    l *= fac;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    float of[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) f2_unpack(o[k], of[2 * k], of[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        of[k] *= fac;
#pragma unroll
        for (int d = LPK; d < 32; d <<= 1) of[k] += __shfl_xor_sync(0xffffffffu, of[k], d);
    }
    if (lane < LPK) {
#pragma unroll
        for (int k = 0; k < 16; ++k) s_o[warp][sub * 16 + k] = of[k];
    }
    if (lane == 0) {
        s_m[warp] = mw;
        s_l[warp] = l;
    }
    __syncthreads();
    // ---- join the warps, then the cluster's CTAs
    if (tid < D) {
        float mc = -INFINITY, lc = 0.f, oc = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) mc = fmaxf(mc, s_m[w]);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float x = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - mc);
            lc += s_l[w] * x;
            oc += s_o[w][tid] * x;
        }
        s_out[tid] = oc;
        if (tid == 0) {
            s_ml[0] = mc;
            s_ml[1] = lc;
        }
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (csize > 1) cluster.sync();
    else __syncthreads();
    if (rank == 0 && tid < D) {
        float mc = -INFINITY, lc = 0.f, oc = 0.f;
        for (int c = 0; c < csize; ++c) {
            const float* ml = csize > 1 ? cluster.map_shared_rank(s_ml, c) : s_ml;
            const float* os = csize > 1 ? cluster.map_shared_rank(s_out, c) : s_out;
            const float mo = ml[0];
            if (ml[1] == 0.f) continue;                      // kept no key; a NaN stays one
            const float mn = fmaxf(mc, mo), a = ex2(mc - mn), b = ex2(mo - mn);
            lc = lc * a + ml[1] * b;
            oc = oc * a + os[tid] * b;
            mc = mn;
        }
        const float val = lc == 0.f ? 0.f : oc / lc;
        if (out_bf16) static_cast<__nv_bfloat16*>(out)[row * D + tid] = __float2bfloat16(val);
        else static_cast<float*>(out)[row * D + tid] = val;
        if (tid == 0) lse[row] = lc == 0.f ? -INFINITY : (mc + log2f(lc)) * 0.69314718055994531f;
    }
    if (csize > 1) cluster.sync();                           // the others' shared memory stays until it has been read
}

// ------------------------------------------------------------------ token groups
// The same for many tokens: 16 places of the token list at a time as the rows
// of mma.m16n8k16, so that a key's codes are fetched and converted once
// for 16 queries (measured against one token at a time in the launch code).
// One cluster of CTAs of 8 warps per (group, head).  The cached frames in reach
// of any of the group's tokens are cut into granules of 16 keys that lie
// together in the cache (16 rows of a tile: 16/w x w keys, w = min(tile_w, 16));
// each frame's granules over the union of the tokens' boxes are dealt out to
// the warps of the cluster, and a granule that no token keeps is left after the
// mask test.  A warp's work on a granule:
//   S = Q K^T   two 8-key column tiles, d/16 K steps.  The order of the d
//               elements along K is free as long as Q and K agree: lane c of a
//               quad takes the 16-code chunks c (and c + 4), word by word.
//   softmax     running maximum and sum of the unrounded P per row, in fp32
//   O += P V    d/8 column tiles.  Column n of tile j is the d element
//               (d/8) n + j, so the lane needs byte j of four key rows, and each
//               pair of keys is one byte permute of two words.  P is split into
//               three bf16 parts, 24 bits over the whole range of P (two f16
//               parts take a tenth less time, but their range is 2^40), and
//               the granule's sum joins O times its V scale in fp32, so tiles
//               of any scales may meet in a row.
// Both products run in bf16: it holds every code, and Q as it comes.  (f16 takes
// three instructions less per pair of codes, 1 to 5 % of the time, but there a Q
// row has to be scaled to f16's range, and its elements 2^33 below the largest
// one lose their bits beside it, also where that one meets keys of zero.)
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t x)      // codes in bytes 0 and 1; exact
{
    uint32_t r;
    float l, h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(l), "=f"(h) : "r"(r));
    return pack_bf16x2(l, h);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same from zeros
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

struct GranuleFrame {
    int y0, y1, x0, x1;          // granule rows and columns, first and last (none: y1 < y0)
};

constexpr int GROUP = 16, GROUP_WARPS = 8, GROUP_FRAMES = 64;

template <int D>
constexpr int group_smem_bytes() { return GROUP_WARPS * GROUP * D * 4; }

template <int D, bool DISK>
__global__ void __launch_bounds__(32 * GROUP_WARPS)
token_group_kernel(const Geom G, const CacheView C, const uint32_t* __restrict__ q, const int32_t* __restrict__ token,
                   const int32_t* __restrict__ radius, int n, int cached, int csize, void* __restrict__ out, int out_bf16,
                   float* __restrict__ lse)
{
    namespace cg = cooperative_groups;
    constexpr int KS = D / 16, NT = D / 8, CH = D / 64;      // K steps, column tiles of O, K chunks per lane and key
    extern __shared__ __align__(16) float group_dyn[];
    float (*s_o)[GROUP][D] = reinterpret_cast<float (*)[GROUP][D]>(group_dyn);      // [warps][GROUP][D]
    __shared__ float s_m[GROUP_WARPS][GROUP], s_l[GROUP_WARPS][GROUP];
    __shared__ float s_ml[GROUP][2];                         // of the CTA, for the cluster
    __shared__ int s_half[GROUP][TRA_MAX_RT_EFF + 1];        // half-widths by |dt|; -1: keeps none
    __shared__ int s_t[GROUP], s_h[GROUP], s_w[GROUP], s_r[GROUP];
    __shared__ int s_lo, s_hi;
    __shared__ GranuleFrame s_frame[GROUP_FRAMES];

    const int groups = (n + GROUP - 1) / GROUP;
    const int unit = blockIdx.x / csize, rank = blockIdx.x - unit * csize;
    const int g = unit / groups, first = (unit - g * groups) * GROUP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int area = G.H * G.W;

    // ---- the group's tokens: place, half-widths, the frames any of them reaches
    if (warp == 0) {
        int t = -1, lo = 0x7fffffff, hi = 0;
        if (lane < GROUP) {
            const int i = first + lane;
            const int tok = i < n ? token[i] : -1;
            int r = -1, h = 0, w = 0;
            if (tok >= G.N) {
                if (rank == 0) atomicOr(&g_tra_error, TRA_ERRBIT_CHECK);
            } else if (tok >= 0) {
                r = radius[(size_t)g * n + i];
                t = tok / area;
                h = (tok - t * area) / G.W;
                w = tok - t * area - h * G.W;
                if (r >= 0) {
                    lo = max(0, t - G.rte);
                    hi = min(cached, t + G.rte + 1);
                }
            }
            s_t[lane] = t;                                   // -1: an unused place
            s_h[lane] = h;
            s_w[lane] = w;
            s_r[lane] = r;
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            s_lo = lo;
            s_hi = hi;
        }
    }
    __syncthreads();
    for (int i = tid; i < GROUP * (G.rte + 1); i += 32 * GROUP_WARPS) {
        const int r = s_r[i & (GROUP - 1)], d = i / GROUP;
        s_half[i & (GROUP - 1)][d] = r >= 0 ? min(halfwidth(r, G.g[d]), TRA_DISK_S_CLAMP) : -1;
    }
    __syncthreads();
    const int f_lo = s_lo, f_hi = max(s_lo == 0x7fffffff ? 0 : s_lo, s_hi);

    // ---- this lane's rows r0, r0 + 8 of the group and its share of Q
    const int c = lane & 3, r0 = lane >> 2;
    uint32_t qa[KS][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = first + r0 + 8 * x;
        const bool ok = i < n && s_t[r0 + 8 * x] >= 0;
        const uint4* src = reinterpret_cast<const uint4*>(q + ((size_t)g * n + (ok ? i : 0)) * (D / 2));
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            // d elements 16 (c + 4k) .. + 15: K steps 4k .. 4k + 3
            const uint4 a = __ldg(src + 2 * (c + 4 * k)), b = __ldg(src + 2 * (c + 4 * k) + 1);
            const uint32_t w8[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int s = 0; s < 8; ++s) qa[4 * k + (s >> 1)][(s & 1) * 2 + x] = ok ? w8[s] : 0u;
        }
    }
    const int t0 = s_t[r0], t1 = s_t[r0 + 8], qh0 = s_h[r0], qh1 = s_h[r0 + 8], qw0 = s_w[r0], qw1 = s_w[r0 + 8];

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};     // P is relative to 2^m
    const int gw_log2 = min(G.tw_log2, 4), gr_log2 = 4 - gw_log2;       // a granule: 2^gr_log2 x 2^gw_log2 keys
    // A granule belongs to one of the cluster's warps by its number in the frame
    // alone, not by the group's boxes: a row's sums run in the same order
    // whatever tokens share its group.
    const int warps = csize * GROUP_WARPS, wid = rank * GROUP_WARPS + warp;
    const int row_granules = (G.nTw << G.tw_log2) >> gw_log2;
    const float inv_row = 1.f / (float)row_granules;
    const uint4* kc = reinterpret_cast<const uint4*>(C.k) + (size_t)g * G.N_pad * (D / 16);
    const uint8_t* vc = C.v + (size_t)g * G.N_pad * D;

    for (int fb = f_lo; fb < f_hi; fb += GROUP_FRAMES) {
        // ---- the granules of up to 64 frames
        const int nf = min(GROUP_FRAMES, f_hi - fb);
        __syncthreads();
        if (tid < nf) {
            int y0 = 0x7fffffff, y1 = -1, x0 = 0x7fffffff, x1 = -1;
            for (int i = 0; i < GROUP; ++i) {
                const int dt = abs(fb + tid - s_t[i]);
                if (s_t[i] < 0 || dt > G.rte) continue;
                const int s = s_half[i][dt];
                if (s < 0) continue;
                y0 = min(y0, max(0, s_h[i] - s)); y1 = max(y1, min(G.H - 1, s_h[i] + s));
                x0 = min(x0, max(0, s_w[i] - s)); x1 = max(x1, min(G.W - 1, s_w[i] + s));
            }
            s_frame[tid] = y1 < 0 ? GranuleFrame{0, -1, 0, -1}
                                  : GranuleFrame{y0 >> gr_log2, y1 >> gr_log2, x0 >> gw_log2, x1 >> gw_log2};
        }
        __syncthreads();
        // the walk over this warp's granules of the chunk: `at` is the next number in
        // frame f, whose last one is `end`
        int f = -1, at = 1, end = 0;
        GranuleFrame F = {0, -1, 0, -1};
        // The next granule with a kept key: its keep-bits, and its codes and scales on
        // their way.  False at the end.  The loads of one granule run under the
        // arithmetic of the one before.
        uint32_t keep_n = 0;
        uint4 kk_n[2][CH];
        uint32_t vv_n[4][NT / 4];
        float ks_n = 0.f, vs_n = 0.f;
        auto fetch = [&]() -> bool {
            for (;;) {
                while (at > end) {
                    if (++f >= nf) return false;
                    F = s_frame[f];
                    const int lo = F.y0 * row_granules + F.x0;
                    end = F.y1 * row_granules + F.x1;
                    // numbers of this warp are wid + 29 frame (an odd step) modulo the warps
                    const int off = (wid + 29 * (fb + f) - lo) % warps;
                    at = lo + (off < 0 ? off + warps : off);
                }
                const int gy = (int)(((float)at + 0.5f) * inv_row), gx = at - gy * row_granules;    // at < 2^16: exact
                at += warps;
                if (gx < F.x0 || gx > F.x1) continue;
                const int h0 = gy << gr_log2, w0 = gx << gw_log2, frame = fb + f;
                // ---- which of its 16 keys do the lane's two rows keep?  Key of score
                // k of column tile j: 8 j + 2 c + k
                const int dt0 = abs(frame - t0), dt1 = abs(frame - t1);
                const int sa = t0 >= 0 && dt0 <= G.rte ? s_half[r0][dt0] : -1;
                const int sb = t1 >= 0 && dt1 <= G.rte ? s_half[r0 + 8][dt1] : -1;
                uint32_t keep = 0;                               // bit 4 x + 2 j + k: row x
#pragma unroll
                for (int jk = 0; jk < 4; ++jk) {
                    const int key = 8 * (jk >> 1) + 2 * c + (jk & 1);
                    const int h = h0 + (key >> gw_log2), w = w0 + (key & ((1 << gw_log2) - 1));
                    const bool in = h < G.H && w < G.W;
                    const int ah = abs(h - qh0), aw = abs(w - qw0), bh = abs(h - qh1), bw = abs(w - qw1);
                    const bool ka = DISK ? sa >= 0 && ah * ah + aw * aw <= sa * sa : max(ah, aw) <= sa;
                    const bool kb = DISK ? sb >= 0 && bh * bh + bw * bw <= sb * sb : max(bh, bw) <= sb;
                    keep |= (in && ka ? 1u << jk : 0u) | (in && kb ? 16u << jk : 0u);
                }
                if (!__any_sync(0xffffffffu, keep != 0)) continue;
                keep_n = keep;
                const int tile = (frame * G.nTh + (h0 >> G.th_log2)) * G.nTw + (w0 >> G.tw_log2);
                const size_t row = (size_t)tile * 128 + ((h0 & (G.th - 1)) << G.tw_log2) + (w0 & (G.tw - 1));
                ks_n = __ldg(C.ks + (size_t)g * G.nQ + tile);
                vs_n = __ldg(C.vs + (size_t)g * G.nQ + tile);
                // ---- codes: K of keys r0 and r0 + 8 (chunks c, c + 4), V of keys 2c,
                // 2c + 1, 2c + 8, 2c + 9 (the d/8 codes from (d/8) r0 on)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < CH; ++k) kk_n[j][k] = __ldg(kc + (row + 8 * j + r0) * (D / 16) + c + 4 * k);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* src = vc + (row + 2 * c + (i & 1) + 8 * (i >> 1)) * D + r0 * NT;
                    if constexpr (NT == 16) {
                        const uint4 a = __ldg(reinterpret_cast<const uint4*>(src));
                        vv_n[i][0] = a.x; vv_n[i][1] = a.y; vv_n[i][2] = a.z; vv_n[i][3] = a.w;
                    } else {
                        const uint2 a = __ldg(reinterpret_cast<const uint2*>(src));
                        vv_n[i][0] = a.x; vv_n[i][1] = a.y;
                    }
                }
                return true;
            }
        };
        bool more = fetch();
        while (more) {
            const uint32_t keep = keep_n;
            const float ks = ks_n, vs = vs_n;
            uint4 kk[2][CH];
            uint32_t vv[4][NT / 4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < CH; ++k) kk[j][k] = kk_n[j][k];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < NT / 4; ++k) vv[i][k] = vv_n[i][k];
            more = fetch();
            // ---- scores
            float sc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const uint32_t w4[4] = {kk[j][k].x, kk[j][k].y, kk[j][k].z, kk[j][k].w};
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_bf16(sc[j], qa[4 * k + s], codes_to_bf16x2(w4[s]), codes_to_bf16x2(w4[s] >> 16));
                }
            }
            // ---- softmax; p[x][2 j + k] of row x
            float p[2][4];
            float mx[2] = {-INFINITY, -INFINITY};
            const float unit = ks * G.scale_log2;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int jk = 0; jk < 4; ++jk) {
                    p[x][jk] = (keep >> (4 * x + jk)) & 1u ? sc[jk >> 1][2 * x + (jk & 1)] * unit : -INFINITY;
                    mx[x] = fmaxf(mx[x], p[x][jk]);
                }
                mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
                mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
            }
            uint32_t ph[4], pm[4], pl[4];                    // the parts of P
            float al[2] = {1.f, 1.f};
            bool raise = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (mx[x] > m[x]) {
                    al[x] = ex2(m[x] - mx[x]);               // 0 for the first kept key
                    l[x] *= al[x];
                    m[x] = mx[x];
                    raise = true;
                }
                const float base = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float a = ex2(p[x][2 * j] - base), b = ex2(p[x][2 * j + 1] - base);
                    l[x] += a + b;
                    const uint32_t hi = pack_bf16x2(a, b);
                    const float ar = a - __uint_as_float(hi << 16), br = b - __uint_as_float(hi & 0xffff0000u);
                    const uint32_t mid = pack_bf16x2(ar, br);
                    ph[2 * j + x] = hi;
                    pm[2 * j + x] = mid;
                    pl[2 * j + x] = pack_bf16x2(ar - __uint_as_float(mid << 16), br - __uint_as_float(mid & 0xffff0000u));
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][0] *= al[0];
                    o[j][1] *= al[0];
                    o[j][2] *= al[1];
                    o[j][3] *= al[1];
                }
            }
            // ---- O += P V
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t sel = (uint32_t)((j & 3) | ((4 + (j & 3)) << 4));
                const uint32_t b0 = codes_to_bf16x2(__byte_perm(vv[0][j >> 2], vv[1][j >> 2], sel));
                const uint32_t b1 = codes_to_bf16x2(__byte_perm(vv[2][j >> 2], vv[3][j >> 2], sel));
                float pv[4];
                mma_bf16_first(pv, pl, b0, b1);
                mma_bf16(pv, pm, b0, b1);
                mma_bf16(pv, ph, b0, b1);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[j][k] = fmaf(vs, pv[k], o[j][k]);
            }
        }
    }

    // ---- join the quads' sums, the warps, then the cluster's CTAs
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (c == 0) {
            s_m[warp][r0 + 8 * x] = m[x];
            s_l[warp][r0 + 8 * x] = l[x];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            s_o[warp][r0 + 8 * x][2 * c * NT + j] = o[j][2 * x];
            s_o[warp][r0 + 8 * x][(2 * c + 1) * NT + j] = o[j][2 * x + 1];
        }
    }
    __syncthreads();
    for (int i = tid; i < GROUP * D; i += 32 * GROUP_WARPS) {
        const int r = i / D, d = i - r * D;
        float mc = -INFINITY, lc = 0.f, oc = 0.f;
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w) mc = fmaxf(mc, s_m[w][r]);
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w) {
            const float a = s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - mc);
            lc += s_l[w][r] * a;
            oc += s_o[w][r][d] * a;
        }
        s_o[0][r][d] = oc;                                   // read by this thread alone until here
        if (d == 0) {
            s_ml[r][0] = mc;
            s_ml[r][1] = lc;
        }
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (csize > 1) cluster.sync();
    else __syncthreads();
    // each CTA of the cluster writes its share of the rows
    for (int r = rank; r < GROUP; r += csize) {
        if (s_t[r] < 0) continue;                            // an unused place: its row stays as it was
        const size_t row = (size_t)g * n + first + r;
        for (int d = tid; d < D; d += 32 * GROUP_WARPS) {
            float mc = -INFINITY, lc = 0.f, oc = 0.f;
            for (int k = 0; k < csize; ++k) {
                const float* ml = csize > 1 ? cluster.map_shared_rank(&s_ml[r][0], k) : &s_ml[r][0];
                const float* os = csize > 1 ? cluster.map_shared_rank(&s_o[0][r][0], k) : &s_o[0][r][0];
                const float mo = ml[0];
                if (ml[1] == 0.f) continue;                  // kept no key; a NaN stays one
                const float mn = fmaxf(mc, mo), a = ex2(mc - mn), b = ex2(mo - mn);
                lc = lc * a + ml[1] * b;
                oc = oc * a + os[d] * b;
                mc = mn;
            }
            const float val = lc == 0.f ? 0.f : oc / lc;
            if (out_bf16) static_cast<__nv_bfloat16*>(out)[row * D + d] = __float2bfloat16(val);
            else static_cast<float*>(out)[row * D + d] = val;
            if (d == 0) lse[row] = lc == 0.f ? -INFINITY : (mc + log2f(lc)) * 0.69314718055994531f;
        }
    }
    if (csize > 1) cluster.sync();                           // the others' shared memory stays until it has been read
}

}  // namespace tra
