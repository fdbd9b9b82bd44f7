// attn_q8_rows.cuh -- row-wise attention over the 8-bit paged cache: bf16
// queries, head_dim 64 or 128, block_size a multiple of 16, up to 16 query
// heads per KV head. Decode steps, and prompts whose queries share few blocks.
//
// Work: one "pair" = (query row, KV head). Its selected blocks are cut into
// strips of 16 tokens. The CTAs of a cluster take whole blocks, the warps of a
// CTA equal runs of its strips, and every warp runs alone: it loads a strip's K
// and V straight from global memory into the registers its MMA fragments need
// (16-byte loads that cover whole 128-byte rows; the next strip is in flight
// while one is computed), converts the codes to f16 (exact), and keeps its own
// running maximum, sum and O. No barrier or copy engine sits in the loop, and the
// first load waits for nothing but the page lookup.
//
// Bound: 32 rows x 32 blocks of 64 (16.8 MB) take 9.4 us, of which the strips
// take 2.8 (6 TB/s); the rest is the chain of a launch: ids, page, first strip (2
// us), and the merge of the warps, the cluster and the masses (2.5 us).
//
// Arithmetic. mma.m16n8k16, f16 in and fp32 out; the 16 rows are the group's
// query heads. A query row is scaled by a power of two so that its largest
// element is in [2^14, 2^15): every bf16 element down to 2^-29 of the largest
// is then exact in f16 (smaller ones are off by less than 2^-40 of it). A
// block's k scale multiplies the fp32 logits. With the v scale = f * 2^e,
// f in [1, 2), the weight p = 2^(x + e - m) carries e, so that p is the
// weight of the *codes* and m the running maximum of x + e; p * f is rounded to
// f16 (11 bits) for P V, and the row sum adds p * 2^-e. The reference m moves
// only when a strip passes it by more than 8, so O is rarely rescaled and
// p <= 2^8.
//
// Fragment layout: a lane's 16-byte run of K holds 16 dims of one token, four
// k-steps of B; the query's dims are permuted alike. For V, lane (g, q) loads
// dims g * HD/8 .. of tokens 2q, 2q+1, 2q+8, 2q+9; bytes of two tokens are
// paired by a byte permute and converted together.
#pragma once

#include <cooperative_groups.h>

#include "attn_q8_simt.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "q8_cache.cuh"

namespace lci {

namespace q8r {
constexpr int kStrip = 16;
constexpr int kRows = 16;       // query heads per MMA (padded)
constexpr int kMaxSplit = 8;
constexpr float kLazy = 8.f;
constexpr int kPrefetch = 16;   // strips (64 KiB) a warp may ask for ahead
// shared memory, in floats. O rows: four segments of HD/4 dims, each padded by 8
// and the row by 4, so that 8 lanes' 16-byte stores meet 32 different banks.
template <int HD> __host__ __device__ constexpr int seg_pitch() { return HD / 4 + 8; }
template <int HD> __host__ __device__ constexpr int row_pitch() { return HD + 32 + 4; }
template <int HD, int NW> __host__ __device__ constexpr int o_floats() { return NW * kRows * row_pitch<HD>(); }
template <int HD, int NW> __host__ __device__ constexpr int base_floats() {
    return o_floats<HD, NW>() + NW * kRows * 2 /*warps' max, sum*/ +
           kRows * HD + 4 * kMaxSplit /*slices received*/ +
           kMaxSplit * kRows * 2 /*CTAs' max, sum*/ + HD * 8 /*query fragments*/;
}
// (max, sum) per head of each (block, warp) that meet: blocks + warps entries
template <int HD, int NW>
__host__ __device__ constexpr size_t smem_bytes(int blocks_with_mass) {
    return (size_t)(base_floats<HD, NW>() +
                    (blocks_with_mass ? (blocks_with_mass + NW) * kRows * 2 : 0)) * 4;
}
}  // namespace q8r

// D += A(16x16, row) * B(16x8, col), f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A v scale as f * 2^e, f in [1, 2); below 2^-60 it counts as 2^-60.
struct VScale {
    float f, e, inv;  // inv = 2^-e
};
__device__ __forceinline__ VScale split_v_scale(float vs) {
    vs = fmaxf(vs, kMinVScale);
    const uint32_t u = __float_as_uint(vs);
    const int e = (int)(u >> 23) - 127;
    VScale r;
    r.f = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
    r.e = (float)e;
    r.inv = __uint_as_float((uint32_t)max(127 - e, 1) << 23);
    return r;
}

// Merges n <= N partial softmax results of head h, given as [partial][16][max,
// sum]: the maximum, the sum and each partial's factor.
template <int N>
struct Q8Merge {
    float f[N], M, L;
    __device__ __forceinline__ Q8Merge(const float* ml, int n, int h) {
        float2 v[N];
        M = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = i < n ? *reinterpret_cast<const float2*>(ml + (i * q8r::kRows + h) * 2)
                         : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, v[i].x);
        }
        const float base = M == -INFINITY ? 0.f : M;
        L = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f[i] = fast_exp2(v[i].x - base);
            L = fmaf(f[i], v[i].y, L);
        }
    }
};

// One strip's raw codes, as this lane's MMA fragments need them.
template <int HD>
struct Q8Strip {
    uint4 k[2][HD / 64];        // [8-token half][16-byte run]
    uint32_t v[4][HD / 32];     // [token 2q, 2q+1, 2q+8, 2q+9][words]
    __device__ __forceinline__ void load_k(const uint8_t* kp, int g8, int q4) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
                k[j][c] = __ldg(reinterpret_cast<const uint4*>(kp + (8 * j + g8) * HD + 16 * (q4 + 4 * c)));
    }
    __device__ __forceinline__ void load_v(const uint8_t* vp, int g8, int q4) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint8_t* p = vp + (2 * q4 + (t & 1) + 8 * (t >> 1)) * HD + g8 * (HD / 8);
            if constexpr (HD == 128) {
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
                v[t][0] = x.x;
                v[t][1] = x.y;
                v[t][2] = x.z;
                v[t][3] = x.w;
            } else {
                const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
                v[t][0] = x.x;
                v[t][1] = x.y;
            }
        }
    }
};

// kLean: three CTAs of four warps per SM, for many rows. The query's fragments
// come from shared memory and a strip's registers take the next strip as soon as
// they are read (its K during this one's softmax and P V, its V during the next Q
// K^T); with more warps to hide the loads this gives 15-25 % (320 pairs of 21
// blocks: 29 us against 38). Else queries and a whole further strip are held in
// registers, which shortens the chain of a few rows (32 x 32 blocks: 9.4 us against
// 9.8).
template <int HD, int NW, bool MODS, bool kLean>
__global__ void __launch_bounds__(NW * 32, kLean ? 3 : NW == 4 ? 2 : 1) sparse_attn_q8_rows_kernel(
    const __grid_constant__ AttnQ8Args a, int nsplit) {
    using namespace q8r;
    namespace cg = cooperative_groups;
    constexpr int NT = NW * 32;
    constexpr int KS = HD / 16;  // k-steps of Q K^T
    constexpr int ON = HD / 8;   // n-tiles of O
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    float* so = reinterpret_cast<float*>(smem_raw);       // [NW][16][row_pitch]
    float* sml = so + o_floats<HD, NW>();                 // [NW][16][max, sum]
    float* recv = sml + NW * kRows * 2;                   // this CTA's slice, from each CTA
    float* cml = recv + kRows * HD + 4 * kMaxSplit;       // [CTA][16][max, sum]
    uint4* sq = reinterpret_cast<uint4*>(cml + kMaxSplit * kRows * 2);  // [k-step][lane]
    float* sbm = cml + kMaxSplit * kRows * 2 + HD * 8;    // [block + warp][16][max, sum]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g8 = lane >> 2, q4 = lane & 3;
    const int split = blockIdx.x % nsplit;
    const long long pair = blockIdx.x / nsplit;
    const int row = (int)(pair / a.H_kv), g = (int)(pair - (long long)row * a.H_kv);
    const int G = a.H_q / a.H_kv;
    const int b = row / a.S, s = row - b * a.S;
    const int spb = a.bs / kStrip;  // strips per block

    pdl_wait();  // nothing of global memory is read before
    // Entries up to the last block: the -1 entries behind it (fewer visible blocks
    // than topk) take no part in the split.
    const int32_t* all_ids = a.ids + (size_t)row * a.topk;
    const int id_a = lane < a.topk ? all_ids[lane] : -1, id_b = lane + 32 < a.topk ? all_ids[lane + 32] : -1;
    int n_ent = id_b != -1 ? lane + 33 : id_a != -1 ? lane + 1 : 0;
    for (int i = lane + 64; i < a.topk; i += 32)
        if (all_ids[i] != -1) n_ent = i + 1;
    n_ent = (int)__reduce_max_sync(0xffffffffu, (unsigned)n_ent);
    // this CTA's blocks, this warp's strips of them
    const int per = (n_ent + nsplit - 1) / nsplit;
    const int i0 = min(n_ent, split * per), nblk = min(n_ent, i0 + per) - i0;
    const int nstrips = nblk * spb;
    const int wper = (nstrips + NW - 1) / NW;
    const int w0 = min(nstrips, warp * wper), w1 = min(nstrips, w0 + wper);
    if (nsplit > 1) cluster_arrive_relaxed();  // matched before the first remote store
    const bool mass = a.mass != nullptr;
    if (mass) {
        for (int e = tid; e < (nblk + NW) * kRows; e += NT)
            *reinterpret_cast<float2*>(sbm + 2 * e) = make_float2(-INFINITY, 0.f);
        __syncthreads();
    }

    // The loads that depend on nothing go first, all in flight together: the
    // ids of this warp's first 32 blocks, the query rows, the positions.
    const int32_t* row_ids = all_ids + i0;
    const int blk_end = w1 > w0 ? (w1 - 1) / spb + 1 : 0;
    int base = w1 > w0 ? w0 / spb : 0;  // blocks are looked up 32 at a time, one per lane
    // (of the first 64 entries the ids are at hand)
    const int at = i0 + base + lane;
    const int ja = __shfl_sync(0xffffffffu, id_a, at & 31), jb = __shfl_sync(0xffffffffu, id_b, at & 31);
    const int j_first = base + lane < blk_end ? (at < 32 ? ja : at < 64 ? jb : all_ids[at]) : -1;
    uint4 qraw[2][HD / 64][2];
    {
        const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)row * a.H_q + (size_t)g * G) * HD;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    qraw[r][c][x] = g8 + 8 * r < G ? __ldg(reinterpret_cast<const uint4*>(
                                                         qrow + (size_t)(g8 + 8 * r) * HD + 16 * (q4 + 4 * c) + 8 * x))
                                                   : make_uint4(0, 0, 0, 0);
    }
    const Q8Window win = q8_window(a, row, b, s);
    float slope_a = 0.f, slope_b = 0.f, inv_cap = 0.f;
    if constexpr (MODS) {
        inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;
        if (a.slopes) {
            slope_a = g8 < G ? a.slopes[g * G + g8] : 0.f;
            slope_b = g8 + 8 < G ? a.slopes[g * G + g8 + 8] : 0.f;
        }
    }


    // The load cursor, one strip ahead of the compute: block (of this CTA),
    // strips left of it, its first token, scales and pointers.
    int t_lane = -1;
    unsigned long long cell_lane = 0;
    float ks_lane = 0.f, vs_lane = 0.f;
    uint32_t live = 0u;
    int n_blk = -1, n_x = 0, st = 0, st_end = 0, n_t0 = 0;
    const uint8_t *kp = nullptr, *vp = nullptr;
    // A warp with few strips asks L2 for all of them at once: one round trip to
    // HBM (and to the page tables of a large pool) instead of one per strip. Not
    // where queries of one sequence share blocks: they would ask for them often
    // (89 queries of 11 blocks: 37 us).
    const bool few = w1 - w0 <= kPrefetch && a.S == 1;
    auto lookup = [&](int j) {
        t_lane = -1;
        const int page = q8_page(a, b, j, win);
        if (page >= 0) {
            t_lane = j * a.bs;
            cell_lane = (unsigned long long)page * a.H_kv + g;
            ks_lane = a.ks[cell_lane];
            vs_lane = a.vs[cell_lane];
            if (few) {
                const int f = (base + lane) * spb;
                const int s0 = max(w0 - f, 0), s1 = min(w1 - f, spb);
                const size_t at = (cell_lane * a.bs + s0 * kStrip) * HD;
                prefetch_l2_bulk(a.k + at, (uint32_t)(s1 - s0) * kStrip * HD);
                prefetch_l2_bulk(a.v + at, (uint32_t)(s1 - s0) * kStrip * HD);
            }
        }
        live = __ballot_sync(0xffffffffu, t_lane >= 0);
    };
    auto advance = [&]() -> bool {  // to the next strip in the window; false: none left
        if (++st < st_end) return true;
        for (;;) {
            while (live) {
                const int x = __ffs(live) - 1;
                live &= live - 1u;
                n_blk = base + x;
                n_x = x;
                n_t0 = __shfl_sync(0xffffffffu, t_lane, x);
                const unsigned long long c = __shfl_sync(0xffffffffu, cell_lane, x);
                kp = a.k + c * a.bs * HD;
                vp = a.v + c * a.bs * HD;
                // this warp's strips, cut to the window
                const int lo = win.lo - n_t0, hi = win.hi - n_t0;
                st = max(w0 - n_blk * spb, lo > 0 ? lo / kStrip : 0);
                st_end = min(min(w1 - n_blk * spb, spb), hi / kStrip + 1);
                if (st < st_end) return true;
            }
            base += 32;
            if (base >= blk_end) return false;
            lookup(base + lane < blk_end ? row_ids[base + lane] : -1);
        }
    };
    Q8Strip<HD> cur, nxt;
    lookup(j_first);
    bool have = blk_end > 0 && advance();
    if (have) {
        cur.load_k(kp + (size_t)st * kStrip * HD, g8, q4);
        cur.load_v(vp + (size_t)st * kStrip * HD, g8, q4);
    }

    // the group's query rows, scaled to f16 (head rows g8 and g8 + 8)
    float qs_a, qs_b;  // what a row's logits are multiplied by (with the softmax scale)
    uint32_t qf[KS][4];
    {
        float back[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t u[4] = {qraw[r][c][x].x, qraw[r][c][x].y, qraw[r][c][x].z, qraw[r][c][x].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = bf16x2_to_f32(u[k]);
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^(14 - exponent of amax), its inverse multiplies the logits
            int e = (int)(__float_as_uint(amax) >> 23) - 127;
            e = e < -100 ? -100 : e > 127 ? 127 : e;
            const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
            back[r] = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t u[4] = {qraw[r][c][x].x, qraw[r][c][x].y, qraw[r][c][x].z, qraw[r][c][x].w};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {  // k-step 4c + 2x + k: dims 4k .. 4k+3 of the run's half
                        const float2 lo = bf16x2_to_f32(u[2 * k]), hi = bf16x2_to_f32(u[2 * k + 1]);
                        qf[4 * c + 2 * x + k][r] = pack_f16x2(lo.x * up, lo.y * up);
                        qf[4 * c + 2 * x + k][2 + r] = pack_f16x2(hi.x * up, hi.y * up);
                    }
                }
        }
        const float unit = MODS ? a.scale : a.scale * kLog2e;
        qs_a = unit * back[0];
        qs_b = unit * back[1];
        if constexpr (kLean) {
            // the same for every warp: each leaves its share of the k-steps for all
#pragma unroll
            for (int k = 0; k < KS; ++k)
                if (k % NW == warp) sq[k * 32 + lane] = make_uint4(qf[k][0], qf[k][1], qf[k][2], qf[k][3]);
            __syncthreads();
        }
    }
    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;  // l: this lane's share
    float r_a = 0.f, r_b = 0.f;                                    // the current block's share
    float o[ON][4];
#pragma unroll
    for (int i = 0; i < ON; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    // (max, sum) of the block just finished, for its mass
    auto close_block = [&](int blk) {
        if (!mass) return;
        float x = r_a, y = r_b;
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        if (q4 == 0) {
            float2* d = reinterpret_cast<float2*>(sbm) + (size_t)(blk + warp) * kRows;
            d[g8] = make_float2(m_a, x);
            d[g8 + 8] = make_float2(m_b, y);
        }
        r_a = r_b = 0.f;
    };

    while (have) {
        const int c_blk = n_blk, c_t0 = n_t0 + st * kStrip;
        // a block's scales stay with the lane that looked it up until now
        const float c_ks = __shfl_sync(0xffffffffu, ks_lane, n_x);
        const VScale c_vs = split_v_scale(__shfl_sync(0xffffffffu, vs_lane, n_x));
        bool more = false;
        if constexpr (!kLean) {
            more = advance();
            if (more) {
                nxt.load_k(kp + (size_t)st * kStrip * HD, g8, q4);
                nxt.load_v(vp + (size_t)st * kStrip * HD, g8, q4);
            }
        }

        // S = Q K^T: two n-tiles of 8 tokens
        // in two chains each (even and odd k-steps)
        float sc[2][4], sd[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[j][e] = sd[j][e] = 0.f;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t qk[4] = {qf[4 * c + k][0], qf[4 * c + k][1], qf[4 * c + k][2], qf[4 * c + k][3]};
                if constexpr (kLean) {
                    const uint4 w = sq[(4 * c + k) * 32 + lane];
                    qk[0] = w.x;
                    qk[1] = w.y;
                    qk[2] = w.z;
                    qk[3] = w.w;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w[4] = {cur.k[j][c].x, cur.k[j][c].y, cur.k[j][c].z, cur.k[j][c].w};
                    uint32_t b0, b1;
                    e4m3x4_to_f16(w[k], b0, b1);
                    mma_f16_16816(k & 1 ? sd[j] : sc[j], qk, b0, b1);
                }
            }
        if constexpr (kLean) {
            more = advance();
            if (more) cur.load_k(kp + (size_t)st * kStrip * HD, g8, q4);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[j][e] += sd[j][e];
        // logits in log2 units, plus the v scale's exponent
        const float ca = qs_a * c_ks, cb = qs_b * c_ks;
        float x[2][4];
        const int ta = c_t0 + 2 * q4;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = sc[j][e] * (e < 2 ? ca : cb);
        if constexpr (MODS) {
            if (a.cap > 0.f) {
                float big = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[j][e] *= inv_cap;
                        big = fmaxf(big, fabsf(x[j][e]));
                    }
                // one branch for the warp: mostly every |u| is small
                if (__any_sync(0xffffffffu, !(big <= kTanhSmall))) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[j][e] = a.cap * q8_tanh(x[j][e]);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[j][e] = a.cap * q8_tanh_small(x[j][e]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[j][e] = fmaf(-(e < 2 ? slope_a : slope_b), (float)abs(win.p - (ta + 8 * j + (e & 1))), x[j][e]) * kLog2e;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] += c_vs.e;
        const bool partial = c_t0 < win.lo || c_t0 + kStrip - 1 > win.hi;
        if (partial) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = ta + 8 * j + e;
                    if (t < win.lo || t > win.hi) {
                        x[j][e] = x[j][e + 2] = -INFINITY;
#pragma unroll
                        for (int w = 0; w < HD / 32; ++w) cur.v[2 * j + e][w] = 0u;  // unset memory
                    }
                }
        }
        float mx_a = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float mx_b = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
        const bool up_a = mx_a > m_a + kLazy, up_b = mx_b > m_b + kLazy;
        if (__any_sync(0xffffffffu, up_a || up_b)) {
            const float co_a = up_a ? exp2f(m_a - mx_a) : 1.f, co_b = up_b ? exp2f(m_b - mx_b) : 1.f;
            m_a = up_a ? mx_a : m_a;
            m_b = up_b ? mx_b : m_b;
            l_a *= co_a;
            l_b *= co_b;
            r_a *= co_a;
            r_b *= co_b;
#pragma unroll
            for (int i = 0; i < ON; ++i) {
                o[i][0] *= co_a;
                o[i][1] *= co_a;
                o[i][2] *= co_b;
                o[i][3] *= co_b;
            }
        }
        const float base_a = m_a == -INFINITY ? 0.f : m_a, base_b = m_b == -INFINITY ? 0.f : m_b;
        float p[2][4], sum_a = 0.f, sum_b = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            p[j][0] = fast_exp2(x[j][0] - base_a);
            p[j][1] = fast_exp2(x[j][1] - base_a);
            p[j][2] = fast_exp2(x[j][2] - base_b);
            p[j][3] = fast_exp2(x[j][3] - base_b);
            sum_a += p[j][0] + p[j][1];
            sum_b += p[j][2] + p[j][3];
        }
        sum_a *= c_vs.inv;
        sum_b *= c_vs.inv;
        l_a += sum_a;
        l_b += sum_b;
        r_a += sum_a;
        r_b += sum_b;
        uint32_t pf[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            pf[2 * j] = pack_f16x2(p[j][0] * c_vs.f, p[j][1] * c_vs.f);
            pf[2 * j + 1] = pack_f16x2(p[j][2] * c_vs.f, p[j][3] * c_vs.f);
        }
        // O += P V
#pragma unroll
        for (int w = 0; w < HD / 32; ++w) {
            // bytes of tokens (2q, 2q+1) and (2q+8, 2q+9) paired: dims 4w .. 4w+3
            uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
            e4m3x4_to_f16(__byte_perm(cur.v[0][w], cur.v[1][w], 0x5140), x0, x1);
            e4m3x4_to_f16(__byte_perm(cur.v[0][w], cur.v[1][w], 0x7362), x2, x3);
            e4m3x4_to_f16(__byte_perm(cur.v[2][w], cur.v[3][w], 0x5140), y0, y1);
            e4m3x4_to_f16(__byte_perm(cur.v[2][w], cur.v[3][w], 0x7362), y2, y3);
            mma_f16_16816(o[4 * w], pf, x0, y0);
            mma_f16_16816(o[4 * w + 1], pf, x1, y1);
            mma_f16_16816(o[4 * w + 2], pf, x2, y2);
            mma_f16_16816(o[4 * w + 3], pf, x3, y3);
        }
        if constexpr (kLean) {
            if (more) cur.load_v(vp + (size_t)st * kStrip * HD, g8, q4);
        }
        if (!more || n_blk != c_blk) close_block(c_blk);
        have = more;
        if constexpr (!kLean) cur = nxt;
    }

    // ---- the warps' partials: (max, sum) and O in shared memory ----
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
    if (q4 == 0) {
        float2* d = reinterpret_cast<float2*>(sml) + warp * kRows;
        d[g8] = make_float2(m_a, l_a);
        d[g8 + 8] = make_float2(m_b, l_b);
    }
    {
        // lane (g8, q4) holds dims q4 * HD/4 .. of head rows g8 and g8 + 8
        float* d = so + warp * kRows * row_pitch<HD>() + g8 * row_pitch<HD>() + q4 * seg_pitch<HD>();
#pragma unroll
        for (int c = 0; c < 2; ++c)  // component: dims c * HD/8 .. of the segment
#pragma unroll
            for (int i = 0; i < ON; i += 4) {
                *reinterpret_cast<float4*>(d + c * ON + i) =
                    make_float4(o[i][c], o[i + 1][c], o[i + 2][c], o[i + 3][c]);
                *reinterpret_cast<float4*>(d + 8 * row_pitch<HD>() + c * ON + i) =
                    make_float4(o[i][2 + c], o[i + 1][2 + c], o[i + 2][2 + c], o[i + 3][2 + c]);
            }
    }
    __syncthreads();
    if (nsplit > 1) cluster_wait();  // every CTA of the cluster runs
    const int groups = G * (HD / 4);  // float4 groups of the pair's output
    const int share = (groups + nsplit - 1) / nsplit;
    __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) + ((size_t)row * a.H_q + (size_t)g * G) * HD;
    // L == 0: nothing attended, a zero row; a NaN sum stays NaN
    auto write4 = [&](int q, float4 v, float L) {
        const float inv = 1.f / L;
        uint2 w = make_uint2(0u, 0u);
        if (L != 0.f) {
            w.x = pack_bf16x2(v.x * inv, v.y * inv);
            w.y = pack_bf16x2(v.z * inv, v.w * inv);
        }
        *reinterpret_cast<uint2*>(orow + 4 * q) = w;
    };
    if (nsplit > 1 && warp == NW - 1) {
        // this CTA's (max, sum) of every head to every CTA of the cluster
        for (int e = lane; e < G * nsplit; e += 32) {
            const int h = e % G, to = e / G;
            const Q8Merge<NW> mg(sml, NW, h);
            float* dst = cg::this_cluster().map_shared_rank(cml, to) + (split * kRows + h) * 2;
            *reinterpret_cast<float2*>(dst) = make_float2(mg.M, mg.L);
        }
    }
    for (int q = tid; q < groups; q += NT) {
        const int h = q / (HD / 4), c = q - h * (HD / 4);
        const int seg = c / (HD / 16), in = c - seg * (HD / 16);
        const float* src = so + h * row_pitch<HD>() + seg * seg_pitch<HD>() + 4 * in;
        const Q8Merge<NW> mg(sml, NW, h);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(src + w * kRows * row_pitch<HD>());
            acc.x += mg.f[w] * v.x;
            acc.y += mg.f[w] * v.y;
            acc.z += mg.f[w] * v.z;
            acc.w += mg.f[w] * v.w;
        }
        if (nsplit == 1) {
            write4(q, acc, mg.L);
        } else {
            const int owner = q / share;
            float* dst = cg::this_cluster().map_shared_rank(recv, owner) + (size_t)(split * share + q - owner * share) * 4;
            *reinterpret_cast<float4*>(dst) = acc;
        }
    }
    if (nsplit > 1) {
        cluster_arrive();
        cluster_wait();
    }
    // per head, for the lse and the masses: the pair's maximum and 1 / sum
    float2* fin = reinterpret_cast<float2*>(so);  // O partials have been read
    if (nsplit == 1 && mass) __syncthreads();
    if (warp == NW - 1 && lane < G) {
        const Q8Merge<NW> one(sml, NW, lane);
        const Q8Merge<kMaxSplit> all(cml, nsplit, lane);
        const float M = nsplit == 1 ? one.M : all.M, L = nsplit == 1 ? one.L : all.L;
        if (a.lse && split == 0)
            a.lse[(size_t)row * a.H_q + (size_t)g * G + lane] = L == 0.f ? -INFINITY : M + log2f(L);
        if (mass) fin[lane] = make_float2(M == -INFINITY ? 0.f : M, L == 0.f ? 0.f : 1.f / L);
    }
    if (nsplit > 1) {
        for (int q = split * share + tid; q < min(groups, (split + 1) * share); q += NT) {
            const Q8Merge<kMaxSplit> mg(cml, nsplit, q / (HD / 4));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
                if (r < nsplit) {
                    const float4 v = *reinterpret_cast<const float4*>(recv + (size_t)(r * share + q - split * share) * 4);
                    acc.x += mg.f[r] * v.x;
                    acc.y += mg.f[r] * v.y;
                    acc.z += mg.f[r] * v.z;
                    acc.w += mg.f[r] * v.w;
                }
            write4(q, acc, mg.L);
        }
    }
    if (mass) {
        __syncthreads();
        // mass of block i: over the warps that met it and the group's heads,
        // four lanes sharing a block's heads
        float* mrow = a.mass + ((size_t)row * a.H_kv + g) * a.topk + i0;
        if (split == nsplit - 1)
            for (int i = n_ent - i0 + tid; i < a.topk - i0; i += NT) mrow[i] = 0.f;
        for (int e = tid; e < nblk * 4; e += NT) {
            const int i = e >> 2, part = e & 3;
            const uint32_t quad = 0xfu << (lane & 28);
            float x = 0.f;
            if (wper > 0) {
                const int wa = (i * spb) / wper, wb = min(NW - 1, (i * spb + spb - 1) / wper);
                for (int w = wa; w <= wb; ++w) {
                    const float2* met = reinterpret_cast<const float2*>(sbm) + (size_t)(i + w) * kRows;
#pragma unroll
                    for (int k = 0; k < kRows / 4; ++k) {
                        const int h = part + 4 * k;
                        if (h < G) {
                            const float2 v = met[h], f = fin[h];
                            x += fast_exp2(v.x - f.x) * v.y * f.y;
                        }
                    }
                }
            }
            x += __shfl_xor_sync(quad, x, 1);
            x += __shfl_xor_sync(quad, x, 2);
            if (part == 0) mrow[i] = x;
        }
    }
}

}  // namespace lci
