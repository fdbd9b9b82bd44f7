// attn_q8_simt.cuh -- attention over the 8-bit paged cache on CUDA cores (fp32
// math): fp32 queries and every shape the tensor-core kernels do not cover.
//
// One CTA per (query row, query head). Where masses are asked for, the heads of a
// KV head share a cluster of up to 8 CTAs, which adds the heads' masses through
// distributed shared memory, in order. The warps take the row's selected blocks
// in turn; inside a block a lane computes the logit of one token (its 16-byte
// runs of K against the query in shared memory), the warp folds 32 tokens into an
// online softmax, and for P V the lanes split the head dim. The warps' (max, sum,
// O) merge through shared memory. Bound by instruction issue: about two
// conversions and four multiply-adds per four cached elements (32 rows x 16 heads
// x 32 blocks of 64, fp32: 126 us, with masses 208; with a row's heads in one CTA
// 1452).
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "ptx.cuh"
#include "q8_cache.cuh"

namespace lci {

// Arguments of the attention over the 8-bit cache, shared by its kernels.
struct AttnQ8Args {
    const void* q;          // [batch][S][H_q][hd]
    const uint8_t *k, *v;   // [P][H_kv][bs][hd]
    const float *ks, *vs;   // [P][H_kv]
    const int32_t* table;   // [batch][nb_max]
    int nb_max, num_pages, H_kv, bs, hd, S, H_q;
    const int32_t* ids;     // [batch][S][topk]
    int topk;
    const int32_t *ctx_len, *q_start;  // [batch]
    float scale;
    // score changes, each optional: z = cap * tanh(z / cap) when cap > 0,
    // z -= slopes[h] * |p - t|, tokens limited to first[row] .. last[row]
    float cap;
    const float* slopes;               // [H_q]
    const int32_t *first, *last;       // [batch][S]
    void* out;              // [batch][S][H_q][hd]
    float* lse;             // [batch][S][H_q] or null
    float* mass;            // [batch][S][H_kv][topk] or null
};

constexpr float kLog2e = 1.4426950408889634f;
// v scales below this count as this (in the tensor-core schedules the softmax weight
// carries log2 of it)
constexpr float kMinVScale = 8.673617379884035e-19f;  // 2^-60

// First and last token a query row may attend; an empty range has hi < lo.
struct Q8Window {
    int lo, hi;   // token positions (nb_max * bs < 2^31)
    int p;        // the query's position
};
__device__ __forceinline__ Q8Window q8_window(const AttnQ8Args& a, int row, int b, int s) {
    Q8Window w;
    const long long p = (long long)a.q_start[b] + s;
    const long long end = (long long)a.ctx_len[b] - 1;
    long long hi = a.last ? (long long)a.last[row] : p;
    hi = hi < end ? hi : end;
    const long long lo = a.first ? (long long)a.first[row] : 0;
    w.hi = (int)(hi < 0x7ffffffell ? hi : 0x7ffffffell);
    w.lo = (int)(lo > 0 ? lo : 0);
    if (hi < 0) w.hi = -1;
    w.p = (int)p;
    return w;
}

// The page of entry i of a row's ids, or -1 (absent, bad, or without a token
// in the window).
__device__ __forceinline__ int q8_page(const AttnQ8Args& a, int b, int j, const Q8Window& w) {
    if (j == -1) return -1;
    if (j < -1 || j >= a.nb_max) {
        raise_status(kStatusBadBlockId);
        return -1;
    }
    const int page = a.table[(size_t)b * a.nb_max + j];
    if (page < 0 || page >= a.num_pages) {
        raise_status(kStatusBadPage);
        return -1;
    }
    const int first = j * a.bs;
    return first <= w.hi && first + a.bs > w.lo ? page : -1;
}

// tanh(u): below 0.625 the odd polynomial u + u^3 * (c0 + ... + c4 u^8), a least
// squares fit of the relative error at Chebyshev nodes of u^2 (1e-8 at most; the
// tests hold the fit); above it 1 - 2 / (2^(2 log2(e) |u|) + 1), whose error of
// 2^-22 is relative to 1.
constexpr float kTanhSmall = 0.625f;
constexpr float kTanhC0 = -0.3333328068256378f, kTanhC1 = 0.13331381976604462f,
                kTanhC2 = -0.05373531952500343f, kTanhC3 = 0.020626291632652283f,
                kTanhC4 = -0.005691985599696636f;
// the same with three coefficients for |u| <= 0.25 (relative error 4e-9)
constexpr float kTanhTiny = 0.25f;
constexpr float kTanhT0 = -0.3333323895931244f, kTanhT1 = 0.13324128091335297f,
                kTanhT2 = -0.05141825973987579f;
__device__ __forceinline__ float q8_tanh_small(float u) {
    const float v = u * u;
    const float p = fmaf(v, fmaf(v, fmaf(v, fmaf(v, kTanhC4, kTanhC3), kTanhC2), kTanhC1), kTanhC0);
    return fmaf(u * v, p, u);
}
__device__ __forceinline__ float q8_tanh(float u) {
    const float a = fabsf(u);
    const float far = copysignf(1.f - __fdividef(2.f, fast_exp2(2.f * kLog2e * a) + 1.f), u);
    return a <= kTanhSmall ? q8_tanh_small(u) : far;  // NaN stays NaN
}

// A scaled logit in natural units -> capped and biased, in log2 units.
__device__ __forceinline__ float q8_score(float z, float cap, float inv_cap, float slope, int dist) {
    if (cap > 0.f) z = cap * q8_tanh(z * inv_cap);
    z = fmaf(-slope, (float)dist, z);
    return z * kLog2e;
}

constexpr int kQ8SimtWarps = 4;
constexpr int kQ8SimtCluster = 8;  // CTAs that share a KV head's masses
constexpr int kQ8MaxHd = 256;

// HD: the largest head_dim of the instance (64, 128 or 256).
template <typename T, int HD>
__global__ void __launch_bounds__(kQ8SimtWarps * 32) sparse_attn_q8_simt_kernel(const AttnQ8Args a, int heads, int parts) {
    constexpr int kPer = HD / 32;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    float* sq = reinterpret_cast<float*>(smem_raw);                                // [hd] query, fp32
    float* so = sq + a.hd;                         // [warps][hd]
    float* sml = so + kQ8SimtWarps * a.hd;         // [warps][2] max and sum
    float* bm = sml + 2 * kQ8SimtWarps;            // [topk] max of each block
    float* br = bm + a.topk;                       // [topk] weight sum of each block
    float* bt = br + a.topk;                       // [topk] mass over the group's heads
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = blockIdx.x % parts, row = blockIdx.x / parts, g = blockIdx.y;
    const int G = a.H_q / a.H_kv, hd = a.hd, bs = a.bs;
    const int h0 = part * heads, h1 = min(G, h0 + heads);  // this CTA's heads of the group
    const int b = row / a.S, s = row - b * a.S;
    const int per_lane = hd >> 5;
    const Q8Window win = q8_window(a, row, b, s);
    const float inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;
    const int32_t* row_ids = a.ids + (size_t)row * a.topk;
    if (a.mass)
        for (int i = tid; i < a.topk; i += blockDim.x) bt[i] = 0.f;

    for (int hl = h0; hl < h1; ++hl) {
        const int h = g * G + hl;
        const T* qh = static_cast<const T*>(a.q) + ((size_t)row * a.H_q + h) * hd;
        __syncthreads();  // the previous head's merge has read sq and so
        for (int d = tid; d < hd; d += blockDim.x) sq[d] = to_f32(qh[d]);
        __syncthreads();
        const float slope = a.slopes ? a.slopes[h] : 0.f;
        float m = -INFINITY, l = 0.f;
        float o[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = 0.f;
        for (int i = warp; i < a.topk; i += kQ8SimtWarps) {
            const int j = row_ids[i];
            const int page = q8_page(a, b, j, win);
            float blk_m = -INFINITY, blk_r = 0.f;
            if (page >= 0) {
                const size_t cell = (size_t)page * a.H_kv + g;
                const uint8_t* kb = a.k + cell * bs * hd;
                const uint8_t* vb = a.v + cell * bs * hd;
                const float kmul = a.scale * a.ks[cell], vmul = fmaxf(a.vs[cell], kMinVScale);
                for (int u0 = 0; u0 < bs; u0 += 32) {
                    const int u = u0 + lane, t = j * bs + u;
                    const bool see = u < bs && t >= win.lo && t <= win.hi;
                    float x = -INFINITY;
                    if (see) {
                        const uint4* kr = reinterpret_cast<const uint4*>(kb + (size_t)u * hd);
                        float dot = 0.f;
#pragma unroll 4
                        for (int c = 0; c < hd / 16; ++c) {
                            const uint4 w4 = __ldg(kr + c);
                            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float f[4];
                                e4m3x4_to_f32(w[e], f);
                                const float4 qv = *reinterpret_cast<const float4*>(sq + 16 * c + 4 * e);
                                dot = fmaf(f[0], qv.x, dot);
                                dot = fmaf(f[1], qv.y, dot);
                                dot = fmaf(f[2], qv.z, dot);
                                dot = fmaf(f[3], qv.w, dot);
                            }
                        }
                        x = q8_score(dot * kmul, a.cap, inv_cap, slope, abs(win.p - t));
                    }
                    const float mx = warp_max(x);
                    const uint32_t seen = __ballot_sync(0xffffffffu, see);
                    if (seen == 0u) continue;
                    const float m_new = fmaxf(m, mx);
                    const float base = m_new == -INFINITY ? 0.f : m_new;
                    const float corr = exp2f(m - base);
                    const float pw = exp2f(x - base);
                    const float sum = warp_sum(pw);
                    m = m_new;
                    l = l * corr + sum;
                    blk_r = blk_r * exp2f(blk_m - base) + sum;
                    blk_m = m_new;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) o[e] *= corr;
                    // only tokens in the window are read: others may be unset memory;
                    // eight tokens' codes are in flight at a time
                    for (int t1 = 0; t1 < 32; t1 += 8) {
                        if (((seen >> t1) & 0xffu) == 0u) continue;
                        const uint8_t* vr = vb + (size_t)(u0 + t1) * hd + lane;
                        uint8_t c[8][kPer];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
#pragma unroll
                            for (int e = 0; e < kPer; ++e)
                                c[k][e] = e < per_lane && ((seen >> (t1 + k)) & 1u) ? __ldg(vr + (size_t)k * hd + 32 * e) : 0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float p1 = __shfl_sync(0xffffffffu, pw, t1 + k) * vmul;
#pragma unroll
                            for (int e = 0; e < kPer; ++e)
                                if (e < per_lane && ((seen >> (t1 + k)) & 1u)) o[e] = fmaf(p1, e4m3_to_f32(c[k][e]), o[e]);
                        }
                    }
                }
            }
            if (a.mass && lane == 0) {
                bm[i] = blk_m;
                br[i] = blk_r;
            }
        }
        if (lane == 0) {
            sml[2 * warp] = m;
            sml[2 * warp + 1] = l;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (e < per_lane) so[warp * hd + lane + 32 * e] = o[e];
        __syncthreads();
        float M = -INFINITY, L = 0.f;
        for (int w = 0; w < kQ8SimtWarps; ++w) M = fmaxf(M, sml[2 * w]);
        const float base = M == -INFINITY ? 0.f : M;
        float f[kQ8SimtWarps];
#pragma unroll
        for (int w = 0; w < kQ8SimtWarps; ++w) {
            f[w] = exp2f(sml[2 * w] - base);
            L += f[w] * sml[2 * w + 1];
        }
        // L != L keeps a NaN of attended values in the output
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
        T* oh = static_cast<T*>(a.out) + ((size_t)row * a.H_q + h) * hd;
        for (int d = tid; d < hd; d += blockDim.x) {
            float acc = 0.f;
#pragma unroll
            for (int w = 0; w < kQ8SimtWarps; ++w) acc += f[w] * so[w * hd + d];
            oh[d] = from_f32<T>(L == 0.f ? 0.f : acc * inv);
        }
        if (a.lse && tid == 0) a.lse[(size_t)row * a.H_q + h] = L == 0.f ? -INFINITY : M + log2f(L);
        if (a.mass)
            for (int i = tid; i < a.topk; i += blockDim.x)
                bt[i] += br[i] == 0.f ? 0.f : br[i] * exp2f(bm[i] - base) * inv;  // a NaN stays one
    }
    if (a.mass) {
        float* mrow = a.mass + ((size_t)row * a.H_kv + g) * a.topk;
        if (parts > 1) {
            namespace cg = cooperative_groups;
            cg::this_cluster().sync();
            for (int i = part * blockDim.x + tid; i < a.topk; i += parts * blockDim.x) {
                float sum = 0.f;
                for (int p = 0; p < parts; ++p) sum += *cg::this_cluster().map_shared_rank(bt + i, p);
                mrow[i] = sum;
            }
            cg::this_cluster().sync();  // no CTA leaves while its masses are read
        } else {
            for (int i = tid; i < a.topk; i += blockDim.x) mrow[i] = bt[i];
        }
    }
}

}  // namespace lci
