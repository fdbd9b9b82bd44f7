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
#include "ptx.cuh"

namespace lci {

constexpr float kE4M3Max = 448.f;
constexpr int kScaleMinExp = -60;  // scales the append writes are 2^-60 .. 2^120

// Two codes (low byte first) -> f16x2, exact; a NaN code gives NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}
// The four codes of a word -> two f16x2.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Four codes of a word -> fp32.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    e4m3x4_to_f16(w, lo, hi);
    const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
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
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
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

// VEC consecutive new elements as loaded.
template <typename T, int VEC> struct RawRun;
// Largest finite magnitude of elements seen.
struct AmaxF32 {
    float m = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float a = fabsf(x);
        m = a <= 3.402823466e38f ? fmaxf(m, a) : m;
    }
};
template <> struct RawRun<float, 16> {
    float4 w[4];
    __device__ __forceinline__ void fold(AmaxF32& a) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a.add(w[i].x);
            a.add(w[i].y);
            a.add(w[i].z);
            a.add(w[i].w);
        }
    }
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * i] = w[i].x;
            x[4 * i + 1] = w[i].y;
            x[4 * i + 2] = w[i].z;
            x[4 * i + 3] = w[i].w;
        }
    }
};
template <> struct RawRun<__nv_bfloat16, 16> {
    uint4 w[2];
    // Packed maxima of magnitudes (the maximum drops NaN); infinities, which
    // do not count, are rare and taken out of the pair that holds one.
    __device__ __forceinline__ void fold(AmaxF32& a) const {
        __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[j])));
        }
        const float2 f = __bfloat1622float2(m);
        const float x = fmaxf(f.x, f.y);
        if (x <= 3.402823466e38f) {
            a.m = fmaxf(a.m, x);
        } else {
            float y[16];
            get(y);
#pragma unroll
            for (int i = 0; i < 16; ++i) a.add(y[i]);
        }
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = bf16x2_to_f32(u[j]);
                x[8 * i + 2 * j] = f.x;
                x[8 * i + 2 * j + 1] = f.y;
            }
        }
    }
};
template <typename T> struct RawRun<T, 1> {
    T w;
    __device__ __forceinline__ void fold(AmaxF32& a) const { a.add(to_f32(w)); }
    __device__ __forceinline__ void load(const T* p) { w = *p; }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = to_f32(w); }
};

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
__device__ __forceinline__ void load_codes(const uint8_t* p, float (&x)[16]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float f[4];
        e4m3x4_to_f32(w[q], f);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * q + r] = f[r];
    }
}
__device__ __forceinline__ void load_codes(const uint8_t* p, float (&x)[1]) { x[0] = e4m3_to_f32(*p); }

constexpr int kAppendMaxThreads = 256;
constexpr int kAppendHold = 2;  // runs of new K, and of new V, a thread holds

// One CTA per (touched block, KV head), for K and V. It owns that head of the
// page: the largest finite magnitude of the new tokens gives the scale they
// need, the page keeps the larger of that and its own scale if it already held
// tokens, stored codes are rounded to a scale that grew, and the new tokens'
// codes are written. New elements stay in registers, as loaded, between the
// two passes (a thread's first kAppendHold runs; further ones, only in blocks
// of more than 8192 elements, are read again from L2). Slots behind the last
// token are not touched.
//
// Bound by HBM for a prompt: K and V of a cell are loaded together so that a
// CTA has 32 KiB in flight behind one chain of lookups, and holding raw bf16
// instead of floats keeps four CTAs on an SM (4 x 8191 tokens of 8 heads behind 1003:
// 36.8 us, 84 % of a measured copy; a ragged batch of 140.9 MB 29.5 us, 73 %; one
// token of 32 sequences 2.5 us, the chain of its loads).
template <typename T, int VEC>
__global__ void __launch_bounds__(kAppendMaxThreads, sizeof(T) == 2 ? 4 : 2) kv_append_q8_kernel(
    const T* __restrict__ k_new, const T* __restrict__ v_new, int T_new, int H_kv, int hd, int bs,
    const int32_t* __restrict__ start, const int32_t* __restrict__ count,
    const int32_t* __restrict__ table, int nb_max, int num_pages, int slots, uint8_t* k_pool,
    uint8_t* v_pool, float* k_scale, float* v_scale) {
    __shared__ float s_amax[2][kAppendMaxThreads / 32];
    pdl_wait();
    const unsigned tid = threadIdx.x, nt = blockDim.x;
    const int g = blockIdx.x % H_kv;
    const int bslot = blockIdx.x / H_kv;
    const int b = bslot / slots, slot = bslot - b * slots;
    const long long p0 = start[b];
    const int n_new = count ? min(max(count[b], 0), T_new) : T_new;
    if (n_new == 0) return;
    if (p0 < 0) {
        if (tid == 0) raise_status(kStatusBadBlockId);
        return;
    }
    const long long j = p0 / bs + slot;
    const long long t_lo = slot == 0 ? p0 : j * bs;                 // first new token of this block
    const long long t_hi = min(p0 + n_new, (j + 1) * (long long)bs);  // past its last one
    if (t_lo >= t_hi) return;
    if (j >= nb_max) {
        if (tid == 0) raise_status(kStatusBadBlockId);
        return;
    }
    // the new elements do not wait for the page: both loads are in flight together
    const int page = table[(size_t)b * nb_max + j];
    const int held = (int)(t_lo - j * bs);  // tokens the block already holds
    const unsigned runs = hd / VEC;
    const unsigned total = (unsigned)(t_hi - t_lo) * runs;  // below 2^31 (block_size * head_dim)
    const size_t src0 = (((size_t)b * T_new + (size_t)(t_lo - p0)) * H_kv + g) * hd;
    const size_t tok_stride = (size_t)H_kv * hd;
    auto src = [&](unsigned e) { return src0 + (size_t)(e / runs) * tok_stride + (size_t)(e % runs) * VEC; };

    RawRun<T, VEC> x[2][kAppendHold];
#pragma unroll
    for (int i = 0; i < kAppendHold; ++i) {
        const unsigned e = tid + i * nt;
        if (e < total) {
            const size_t at = src(e);
            x[0][i].load(k_new + at);
            x[1][i].load(v_new + at);
        }
    }
    if (page < 0 || page >= num_pages) {
        if (tid == 0) raise_status(kStatusBadPage);
        return;
    }
    const size_t cell = (size_t)page * H_kv + g;
    const float s_old[2] = {held > 0 ? k_scale[cell] : 0.f, held > 0 ? v_scale[cell] : 0.f};
    AmaxF32 seen[2];
#pragma unroll
    for (int i = 0; i < kAppendHold; ++i)
        if (tid + i * nt < total) {
            x[0][i].fold(seen[0]);
            x[1][i].fold(seen[1]);
        }
    for (unsigned e = tid + kAppendHold * nt; e < total; e += nt) {
        RawRun<T, VEC> y;
        y.load(k_new + src(e));
        y.fold(seen[0]);
        y.load(v_new + src(e));
        y.fold(seen[1]);
    }
    float amax[2] = {seen[0].m, seen[1].m};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        amax[kv] = warp_max(amax[kv]);
        if ((tid & 31) == 0) s_amax[kv][tid >> 5] = amax[kv];
    }
    __syncthreads();
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        amax[kv] = warp_max((tid & 31) < (nt >> 5) ? s_amax[kv][tid & 31] : 0.f);
        const float s_new = fmaxf(s_old[kv], e4m3_scale(amax[kv]));
        uint8_t* dst = (kv ? v_pool : k_pool) + cell * bs * hd;
        // a power of two is divided by exactly with its reciprocal; a scale
        // from elsewhere takes the division
        const bool pow2 = (__float_as_uint(s_new) & 0x7fffffu) == 0u;
        const float inv = 1.f / s_new;
        auto put = [&](uint8_t* p, const RawRun<T, VEC>& r) {
            float y[VEC];
            r.get(y);
            if (pow2) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] *= inv;
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] = y[e] / s_new;
            }
            store_codes(p, y);
        };
        if (tid == 0) (kv ? v_scale : k_scale)[cell] = s_new;  // all have read s_old: the barrier
        if (held > 0 && s_new > s_old[kv]) {
            const float ratio = s_old[kv] / s_new;
            for (unsigned e = tid; e < (unsigned)held * runs; e += nt) {
                float y[VEC];
                load_codes(dst + (size_t)e * VEC, y);
#pragma unroll
                for (int q = 0; q < VEC; ++q) y[q] *= ratio;
                store_codes(dst + (size_t)e * VEC, y);
            }
        }
        uint8_t* fresh = dst + (size_t)held * hd;
#pragma unroll
        for (int i = 0; i < kAppendHold; ++i) {
            const unsigned e = tid + i * nt;
            if (e < total) put(fresh + (size_t)e * VEC, x[kv][i]);
        }
        for (unsigned e = tid + kAppendHold * nt; e < total; e += nt) {
            RawRun<T, VEC> y;
            y.load((kv ? v_new : k_new) + src(e));
            put(fresh + (size_t)e * VEC, y);
        }
    }
}

}  // namespace lci
