// q8_cache.cuh -- the 8-bit paged KV cache: e4m3 values with one fp32 scale per
// page and KV head, and the append that writes it.
//
// A stored element stands for scale * value(code). The append keeps scales at
// powers of two: dividing by one and multiplying codes by the ratio of two is
// exact in fp32, so a token is rounded once when it enters (to 4 significant
// bits) and is rounded again, when its page's scale grows later, only if it
// falls below the e4m3 normal range there. A floating 8-bit code loses nothing
// to a power-of-two scale but the last fraction of a binade of range.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace lci {

constexpr float kE4M3Max = 448.f;
constexpr int kScaleMinExp = -60;  // scales the append writes are 2^-60 .. 2^120

// Two codes (low byte first) -> f16x2, exact; a NaN code gives NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Four codes of a word -> fp32.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4]) {
    const float2 a = f16x2_to_f32(e4m3x2_to_f16x2(w)), b = f16x2_to_f32(e4m3x2_to_f16x2(w >> 16));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}
__device__ __forceinline__ float e4m3_to_f32(uint8_t c) { return f16x2_to_f32(e4m3x2_to_f16x2(c)).x; }

// Round to nearest e4m3, saturating at +-448 (also +-inf); NaN keeps being NaN.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\tcvt.u32.u16 %0, c;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f32_to_e4m3x4(float a, float b, float c, float d) {
    return f32_to_e4m3x2(a, b) | (f32_to_e4m3x2(c, d) << 16);
}

// Smallest power of two 2^e, e >= kScaleMinExp, with amax <= 448 * 2^e
// (448 = 0.875 * 2^9; amax finite and not negative).
__device__ __forceinline__ float e4m3_scale(float amax) {
    int e;
    const float m = frexpf(amax, &e);  // amax = m * 2^e, m in [0.5, 1)
    e = amax > 0.f ? (m <= 0.875f ? e - 9 : e - 8) : kScaleMinExp;
    e = e < kScaleMinExp ? kScaleMinExp : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ void load_run(const float* p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load_run(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = bf16x2_to_f32(w[j]);
            x[8 * i + 2 * j] = f.x;
            x[8 * i + 2 * j + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ void load_run(const T* p, float (&x)[1]) {
    x[0] = to_f32(*p);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[16]) {
    uint4 v;
    v.x = f32_to_e4m3x4(x[0], x[1], x[2], x[3]);
    v.y = f32_to_e4m3x4(x[4], x[5], x[6], x[7]);
    v.z = f32_to_e4m3x4(x[8], x[9], x[10], x[11]);
    v.w = f32_to_e4m3x4(x[12], x[13], x[14], x[15]);
    *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[1]) {
    *p = (uint8_t)f32_to_e4m3x2(x[0], 0.f);
}

// One CTA per (touched block, KV head, K or V). It owns that head of the page:
// the largest finite magnitude of the new tokens gives the scale they need, the
// page keeps the larger of that and its own scale if it already held tokens,
// stored codes are rounded to a scale that grew, and the new tokens' codes are
// written. A thread's first kHold runs of new elements stay in registers
// between the two passes; further ones are read again (from L2).
// Slots behind the last token are not touched.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) kv_append_q8_kernel(
    const T* __restrict__ k_new, const T* __restrict__ v_new, int batch, int T_new, int H_kv, int hd,
    int bs, const int32_t* __restrict__ start, const int32_t* __restrict__ count,
    const int32_t* __restrict__ table, int nb_max, int num_pages, int slots, uint8_t* k_pool,
    uint8_t* v_pool, float* k_scale, float* v_scale) {
    constexpr int kHold = VEC == 16 ? 2 : 16;
    __shared__ float s_amax[8];
    const unsigned tid = threadIdx.x, nt = blockDim.x;
    const int g = blockIdx.x % H_kv;
    const bool is_v = blockIdx.y != 0;
    const int bslot = blockIdx.x / H_kv;
    const int b = bslot / slots, slot = bslot - b * slots;
    const long long p0 = start[b];
    const int n_new = count ? min(max(count[b], 0), T_new) : T_new;
    if (n_new == 0) return;
    const long long j = p0 / bs + slot;
    const long long t_lo = slot == 0 ? p0 : j * bs;                 // first new token of this block
    const long long t_hi = min(p0 + n_new, (j + 1) * (long long)bs);  // past its last one
    if (p0 < 0 || t_lo >= t_hi) {
        if (p0 < 0 && tid == 0) raise_status(kStatusBadBlockId);
        return;
    }
    if (j >= nb_max) {
        if (tid == 0) raise_status(kStatusBadBlockId);
        return;
    }
    const int page = table[(size_t)b * nb_max + j];
    if (page < 0 || page >= num_pages) {
        if (tid == 0) raise_status(kStatusBadPage);
        return;
    }
    const int held = (int)(t_lo - j * bs);  // tokens the block already holds
    const unsigned runs = hd / VEC;
    const unsigned total = (unsigned)(t_hi - t_lo) * runs;  // below 2^31 (block_size * head_dim)
    const T* src = (is_v ? v_new : k_new) + (((size_t)b * T_new + (size_t)(t_lo - p0)) * H_kv + g) * hd;
    const size_t tok_stride = (size_t)H_kv * hd;
    const size_t cell = (size_t)page * H_kv + g;
    uint8_t* dst = (is_v ? v_pool : k_pool) + cell * bs * hd;
    float* sc = (is_v ? v_scale : k_scale) + cell;
    const float s_old = held > 0 ? *sc : 0.f;

    float x[kHold][VEC];
    float amax = 0.f;
    auto fold = [&](const float (&y)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float a = fabsf(y[e]);
            amax = a <= 3.402823466e38f ? fmaxf(amax, a) : amax;  // finite values only
        }
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const unsigned e = tid + i * nt;
        if (e < total) load_run(src + (size_t)(e / runs) * tok_stride + (size_t)(e % runs) * VEC, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (tid + i * nt < total) fold(x[i]);
    for (unsigned e = tid + kHold * nt; e < total; e += nt) {
        float y[VEC];
        load_run(src + (size_t)(e / runs) * tok_stride + (size_t)(e % runs) * VEC, y);
        fold(y);
    }
    amax = warp_max(amax);
    if ((tid & 31) == 0) s_amax[tid >> 5] = amax;
    __syncthreads();
    for (unsigned w = 0; w < (nt >> 5); ++w) amax = fmaxf(amax, s_amax[w]);
    const float s_new = fmaxf(s_old, e4m3_scale(amax));
    // a power of two is divided by exactly with its reciprocal; a scale from
    // elsewhere takes the division
    const bool pow2 = (__float_as_uint(s_new) & 0x7fffffu) == 0u;
    const float inv = 1.f / s_new;
    auto put = [&](uint8_t* p, float (&y)[VEC]) {
        if (pow2) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] *= inv;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = y[e] / s_new;
        }
        store_codes(p, y);
    };
    if (tid == 0) *sc = s_new;  // every thread has read s_old before the barrier
    if (held > 0 && s_new > s_old) {
        const float ratio = s_old / s_new;
        const unsigned old_runs = (unsigned)held * runs;
        for (unsigned e = tid; e < old_runs; e += nt) {
            uint8_t* p = dst + (size_t)e * VEC;
            if constexpr (VEC == 16) {
                const uint4 v = *reinterpret_cast<const uint4*>(p);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float y[16];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f[4];
                    e4m3x4_to_f32(w[q], f);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[4 * q + r] = f[r] * ratio;
                }
                store_codes(p, y);
            } else {
                float y[1] = {e4m3_to_f32(*p) * ratio};
                store_codes(p, y);
            }
        }
    }
    uint8_t* fresh = dst + (size_t)held * hd;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const unsigned e = tid + i * nt;
        if (e < total) put(fresh + (size_t)e * VEC, x[i]);
    }
    for (unsigned e = tid + kHold * nt; e < total; e += nt) {
        float y[VEC];
        load_run(src + (size_t)(e / runs) * tok_stride + (size_t)(e % runs) * VEC, y);
        put(fresh + (size_t)e * VEC, y);
    }
}

}  // namespace lci
