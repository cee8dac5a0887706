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
// one of the keys, all loads of the batch go out together, and a butterfly
// leaves each lane with the score of its key.  Each group keeps a running
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
    for (int e0 = 0; e0 < total; e0 += groups * LPK) {
        // this lane's key of the batch
        const int e = e0 + sub * groups + gid;
        int at = -1;
        float ks = 0.f, vs = 0.f;
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
        uint4 kk[LPK], vv[LPK];
#pragma unroll
        for (int k = 0; k < LPK; ++k) {
            const int a = __shfl_sync(0xffffffffu, at, k, LPK);
            kk[k] = vv[k] = make_uint4(0u, 0u, 0u, 0u);
            if (a >= 0) {
                kk[k] = __ldg(kc + (size_t)a * LPK);
                vv[k] = __ldg(vc + (size_t)a * LPK);
            }
        }
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
            if (mo == -INFINITY) continue;
            const float mn = fmaxf(mc, mo), a = ex2(mc - mn), b = ex2(mo - mn);
            lc = lc * a + ml[1] * b;
            oc = oc * a + os[tid] * b;
            mc = mn;
        }
        const float val = lc > 0.f ? oc / lc : 0.f;
        if (out_bf16) static_cast<__nv_bfloat16*>(out)[row * D + tid] = __float2bfloat16(val);
        else static_cast<float*>(out)[row * D + tid] = val;
        if (tid == 0) lse[row] = lc > 0.f ? (mc + log2f(lc)) * 0.69314718055994531f : -INFINITY;
    }
    if (csize > 1) cluster.sync();                           // the others' shared memory stays until it has been read
}

}  // namespace tra
