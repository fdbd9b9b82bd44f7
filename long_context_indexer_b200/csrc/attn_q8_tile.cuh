// attn_q8_tile.cuh -- attention over the 8-bit paged cache for many queries per
// sequence, on the 5th-generation tensor cores (tcgen05 + TMEM): bf16 queries,
// head_dim 128, block_size a multiple of 64, up to 16 query heads per KV head.
//
// Tile. A CTA owns up to 128 MMA rows: QT = min(32, 128 / G) consecutive queries
// of one sequence times the G query heads of one KV head. It walks the union of
// the blocks its queries selected in units of 64 tokens, two units to a pair.
//
// The cached codes are never converted: K and V tiles come by TMA as they are
// stored and are the 8-bit B operands of tcgen05.mma.kind::f8f6f4. The 16-bit
// side is split instead. A bf16 query element, scaled by a power of two per row,
// is the sum of two e4m3 numbers (4 + 4 significant bits, exact down to 2^-17 of
// the row's largest element). A softmax weight is the sum of three e5m2 numbers:
// rounded to f16, its upper byte is one, the upper byte of the rest another, and
// what is left is rounded to a third (3 + 3 + 3 bits, off by at most 2^-8.6 of it).
// e5m2 has f16's exponents, so this holds down to 2^-16 of the row's reference,
// and smaller weights are off by at most 2^-25 of it: a row keeps the many small
// weights behind one large one. Two e4m3 parts, which end at 2^-9, lost all of
// them below 2^-15 of the largest.
//   S  = Qhi K^T + Qlo K^T       M=128, N=128 tokens, A = Q from shared memory
//   O += P0 V + P1 V + P2 V      M=128, N=128 dims, K=64 tokens, A = P from TMEM,
//                                B = V MN-major from shared memory
// (Q stays out of TMEM so that three pairs of S fit beside O.) The third part costs
// 35 us of the 8K prompt; two parts keep 7 bits, which raises the output's error by
// two thirds (1.3e-4 -> 2.1e-4, against 1.3e-4 of a bf16 rounding alone). V converted to f16 for two-byte weights was slower: by
// the softmax warps 351 us, by warps of their own 325 to 429, against 300.
//
// Scales. A block's k scale multiplies the fp32 logits. Its v scale enters the
// exponent, so that the weight is that of the codes, p = 2^(x + log2 vs - m),
// and the row sum adds p / vs; the running reference m of a row is the maximum
// of x + log2 vs. Weights are 2^8 at the reference; it moves only when a unit
// passes it by more than 7.75 (weights stay below 57344, e5m2's largest), and O is
// rescaled only then (with 3.75: 317 us against 300).
//
// Warps: 0 copies K and 3 copies V (K runs ahead of the V ring, whose stages free
// only after the softmax), 1 issues Q K^T, 2 issues P V (the waits and commits
// around the one hide behind the MMAs of the other), then three softmax groups of
// four warps that take every third unit, one thread per row. A warp (two queries
// at 16 heads) none of whose queries selected the unit only stores zero weights,
// so with sparse selections the warps work ahead of each other. The groups agree
// on a row's reference in unit order: a short chain of one mbarrier per 32 rows
// and group, between the maximum and the exponentials of each unit.
//
// Bound. 8K prompt, 16 heads on one KV head, 32 blocks of 64 per query: 299 us a
// call in a graph, 402 TFLOP/s of useful work (24 % of the measured bf16 peak; the
// selections make the MMAs compute about twice that), 336 us a call on its own.
// About 1000 cycles per unit of a tile's union against 640 of MMA (tensor pipe 50 %
// active): with three pairs in flight the softmax (64 exponentials a thread and the
// parts of each weight), its hand-over to the MMA and the wait for the slot set the
// pace, and 16 thousand cycles per tile go to the union, the first copies and the
// output. More softmax warps do not help (four groups that read S twice, in halves,
// to fit their registers: 312 us; three groups so: 305).
//
// Unset memory and NaN. V rows of absent units and of tokens past the context
// are zeroed in shared memory before the MMA reads them, their scores masked. A
// NaN code inside the context contaminates every row of the tile as 0 * NaN; rows
// whose output holds a NaN are computed again by one warp each in fp32, which
// reads only what the row attends.
#pragma once

#include "attn_prefill.cuh"
#include "attn_q8_rows.cuh"
#include "common.cuh"
#include "index_prefill.cuh"
#include "ptx.cuh"
#include "q8_cache.cuh"

namespace lci {

namespace q8t {
constexpr int kHD = 128;
constexpr int kRows = 128;
constexpr int kMaxQT = 32;             // queries per tile: a block's mask of them is a word
constexpr int kUnit = 64;              // tokens per unit
constexpr int kUnitBytes = kUnit * kHD;
constexpr int kStageBytes = 2 * kUnitBytes;  // a pair: 16 KiB of K or of V
constexpr int kStages = 4;             // a power of two
constexpr int kMaxWords = 512;         // block bitmap words: nb_max <= 16384
constexpr int kMaxUnion = 2048;        // distinct blocks per tile
constexpr int kGroups = 3;             // softmax groups, unit u belongs to group u % kGroups
constexpr int kGroupWarps = 4;
constexpr int kFirstSoftmax = 4;       // warps 0..3: K copies, Q K^T, P V, V copies
constexpr int kThreads = 32 * kFirstSoftmax + kGroups * 32 * kGroupWarps;
constexpr int kSlots = 3;              // pairs of S in flight
// TMEM columns: O fp32, kSlots pairs of S (fp32; a unit's 64 columns then hold
// its P: for each half of the unit's tokens 8 columns of each part)
constexpr int kColO = 0, kColS = 128, kTmemCols = 512;
constexpr int kParts = 3;              // e5m2 parts of a weight
constexpr float kShift = 8.f;          // log2 of the weight at the reference
constexpr float kLazy = 7.75f;         // 2^(8 + 7.75) < 57344, the largest e5m2
// shared memory (offsets from a 1024-byte aligned base)
constexpr int kOffK = 0;
constexpr int kOffV = kOffK + kStages * kStageBytes;
constexpr int kOffQ = kOffV + kStages * kStageBytes;     // high parts, then low parts
constexpr int kOffUnion = kOffQ + 2 * kRows * kHD;
constexpr int kUnionBytes = 2 * kMaxWords * 4 + kMaxUnion * (16 + 4);
constexpr int kOffWin = kOffUnion + kUnionBytes;    // [kMaxQT] Q8Window
constexpr int kOffBar = kOffWin + kMaxQT * 16;
constexpr int kOffRow = kOffBar + 512;              // [128] references, [kGroups][128] sums, [128] flags, [128] factors
constexpr int kSmemBytes = kOffRow + (3 + kGroups) * 128 * 4 + 1024 /*alignment slack*/;
// instruction descriptors, kind::f8f6f4: D fp32, A and B e4m3 (P V: A e5m2, B
// MN-major), M = 128, N = 128
constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 7) | (1u << 16);
}  // namespace q8t

// D (+)= A B, 8-bit operands, A read from TMEM (4 elements per column).
__device__ __forceinline__ void tc_mma_f8_tmem_a(uint32_t tmem_d, uint32_t tmem_a, uint64_t b,
                                                 uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(b), "r"(idesc), "r"(accumulate));
}

// D (+)= A B, 8-bit operands in shared memory.
__device__ __forceinline__ void tc_mma_f8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// Four non-negative weights (below 57344) -> the e5m2 codes of three parts that
// add up to them. A weight is rounded to f16 (11 bits); an e5m2 number is the
// upper byte of an f16, so the upper byte is a part of 3 bits and subtracting it
// is exact, twice; the rest is rounded to 3 bits.
__device__ __forceinline__ void split_weights(float a, float b, float c, float d, uint32_t& p0, uint32_t& p1,
                                              uint32_t& p2) {
    uint32_t x = pack_f16x2(a, b), y = pack_f16x2(c, d);
    auto upper = [](uint32_t v) { return v & 0xff00ff00u; };
    auto rest = [&](uint32_t v) {
        const uint32_t u = upper(v);
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&u));
        return *reinterpret_cast<const uint32_t*>(&r);
    };
    p0 = __byte_perm(x, y, 0x7531);
    x = rest(x);
    y = rest(y);
    p1 = __byte_perm(x, y, 0x7531);
    x = rest(x) + 0x00800080u;
    y = rest(y) + 0x00800080u;
    p2 = __byte_perm(x, y, 0x7531);
}

// 8 consecutive 32-bit columns of this thread's TMEM lane <- r.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Waits for a barrier's phase. A wait that runs out makes the tile give up:
// every further wait of the tile returns at once and its rows become zero.
__device__ __forceinline__ void tile_wait(uint64_t* bar, uint32_t parity, volatile int* s_abort) {
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = global_ns();
    const unsigned long long limit = g_wait_limit_ns;
    while (!mbar_try_wait(bar, parity)) {
        if (*s_abort) return;
        if (global_ns() - t0 > limit) {
            raise_status(kStatusTimeout);
            *s_abort = 1;
            return;
        }
    }
}

// Waits for copies or MMAs of this CTA that are under way, before what they read
// or write is given up: at least 2 s, however short the limit of other waits is.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    const unsigned long long limit = max(g_wait_limit_ns, 2000000000ull);
    while (!mbar_try_wait(bar, parity))
        if (global_ns() - t0 > limit) {
            raise_status(kStatusTimeout);
            return;
        }
}

// One query row and head by one warp, fp32, reading only attended tokens
// (sq: hd floats of shared memory of this warp).
__device__ __noinline__ void q8_row_by_warp(const AttnQ8Args& a, int row, int h, float* sq) {
    constexpr int kPer = q8t::kHD / 32;
    const int lane = threadIdx.x & 31;
    const int b = row / a.S, s = row - b * a.S, g = h / (a.H_q / a.H_kv);
    const __nv_bfloat16* qh = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)row * a.H_q + h) * q8t::kHD;
    __syncwarp();
    for (int d = lane; d < q8t::kHD; d += 32) sq[d] = to_f32(qh[d]);
    __syncwarp();
    const Q8Window win = q8_window(a, row, b, s);
    const float inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f, slope = a.slopes ? a.slopes[h] : 0.f;
    float m = -INFINITY, l = 0.f, o[kPer] = {};
    for (int i = 0; i < a.topk; ++i) {
        const int j = a.ids[(size_t)row * a.topk + i];
        const int page = q8_page(a, b, j, win);
        if (page < 0) continue;
        const size_t cell = (size_t)page * a.H_kv + g;
        const float kmul = a.scale * a.ks[cell], vmul = fmaxf(a.vs[cell], kMinVScale);
        for (int u0 = 0; u0 < a.bs; u0 += 32) {
            const int t = j * a.bs + u0 + lane;
            const bool see = u0 + lane < a.bs && t >= win.lo && t <= win.hi;
            float x = -INFINITY;
            if (see) {
                const uint8_t* kr = a.k + (cell * a.bs + u0 + lane) * q8t::kHD;
                float dot = 0.f;
                for (int d = 0; d < q8t::kHD; ++d) dot = fmaf(e4m3_to_f32(kr[d]), sq[d], dot);
                x = q8_score(dot * kmul, a.cap, inv_cap, slope, abs(win.p - t));
            }
            const uint32_t seen = __ballot_sync(0xffffffffu, see);
            if (seen == 0u) continue;
            const float m_new = fmaxf(m, warp_max(x));
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float corr = exp2f(m - base), pw = exp2f(x - base);
            m = m_new;
            l = l * corr + warp_sum(pw);
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] *= corr;
            for (uint32_t left = seen; left != 0u; left &= left - 1u) {
                const int t1 = __ffs(left) - 1;
                const float p1 = __shfl_sync(0xffffffffu, pw, t1) * vmul;
                const uint8_t* vr = a.v + (cell * a.bs + u0 + t1) * q8t::kHD + lane;
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] = fmaf(p1, e4m3_to_f32(vr[32 * e]), o[e]);
            }
        }
    }
    __nv_bfloat16* oh = static_cast<__nv_bfloat16*>(a.out) + ((size_t)row * a.H_q + h) * q8t::kHD;
#pragma unroll
    for (int e = 0; e < kPer; ++e) oh[lane + 32 * e] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] / l);
    if (a.lse && lane == 0) a.lse[(size_t)row * a.H_q + h] = l == 0.f ? -INFINITY : m + log2f(l);
}

template <bool MODS>
__global__ void __launch_bounds__(q8t::kThreads, 1) sparse_attn_q8_tile_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ AttnQ8Args a, int batch, int q_tiles) {
    using namespace q8t;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t* bitmap = reinterpret_cast<uint32_t*>(smem + kOffUnion);  // [kMaxWords]
    uint32_t* wpre = bitmap + kMaxWords;                               // [kMaxWords]
    // per block of the union: first token (-1: bad page), queries that selected
    // it, k scale, log2 of the v scale; and its page
    uint4* uinfo = reinterpret_cast<uint4*>(wpre + kMaxWords);         // [kMaxUnion]
    int* upage = reinterpret_cast<int*>(uinfo + kMaxUnion);            // [kMaxUnion]
    Q8Window* wins = reinterpret_cast<Q8Window*>(smem + kOffWin);      // [kMaxQT]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* kfull = bars;                // [kStages]
    uint64_t* kempty = kfull + kStages;    // [kStages]
    uint64_t* vfull = kempty + kStages;    // [kStages]
    uint64_t* vempty = vfull + kStages;    // [kStages]
    uint64_t* sfull = vempty + kStages;      // [kSlots] a pair's S written
    uint64_t* pfull = sfull + kSlots;        // [2 * kSlots] a unit's P written (4 warps)
    uint64_t* decided = pfull + 2 * kSlots;  // [kGroups][4] a group's reference of a unit, per 32 rows
    uint64_t* obar = decided + 4 * kGroups;  // [kSlots] P V of a pair's first unit completed
    uint64_t* drain = obar + kSlots;         // [2] every MMA of an issuer completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    int* s_nunion = reinterpret_cast<int*>(tmem_slot + 1);
    // set by any role whose bounded wait ran out: the tile then gives up
    volatile int* s_abort = s_nunion + 1;
    static_assert((4 * kStages + 4 * kSlots + 4 * kGroups + 2) * 8 + 12 <= 512, "barriers fit");
    float* mref = reinterpret_cast<float*>(smem + kOffRow);  // [128]
    float* lsum = mref + 128;                                // [kGroups][128]
    int* redo = reinterpret_cast<int*>(lsum + kGroups * 128);  // [128]
    float* rowmul = reinterpret_cast<float*>(redo + 128);      // [128] inverse of a query row's factor

    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.H_q / a.H_kv;
    const int QT = min(kMaxQT, kRows / G);
    // the latest queries (most visible blocks) of every sequence first
    const int per_qt = batch * a.H_kv;
    const int qt = q_tiles - 1 - (int)(blockIdx.x / per_qt);
    const int rest = (int)(blockIdx.x % per_qt);
    const int b = rest / a.H_kv, g = rest - b * a.H_kv;
    const int s0 = qt * QT;
    const int nwords = (a.nb_max + 31) >> 5;
    const int upb = a.bs / kUnit;  // units per block

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&obar[i], 1);
        }
        for (int i = 0; i < 2 * kSlots; ++i) mbar_init(&pfull[i], kGroupWarps);
        for (int i = 0; i < 4 * kGroups; ++i) mbar_init(&decided[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    constexpr int kUnionBarrier = 2, kUnionThreads = 32 * kFirstSoftmax;
    if (warp < kFirstSoftmax) {
        // ---------------- the union of the tile's selected blocks ----------------
        // (warps 0..3, beside the query rows of the others)
        constexpr int kHold = 4;  // entries, then blocks, a thread has in flight
        const int32_t* tile_ids = a.ids + ((size_t)b * a.S + s0) * a.topk;
        const int n_real = min(QT, a.S - s0) * a.topk;  // entries of queries that exist
        int held[kHold];
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int e = tid + k * kUnionThreads;
            held[k] = e < n_real ? tile_ids[e] : -1;
        }
        for (int w = tid; w < nwords; w += kUnionThreads) bitmap[w] = 0u;
        for (int e = tid; e < min(n_real, kMaxUnion); e += kUnionThreads) uinfo[e].y = 0u;
        if (tid < kMaxQT) {
            Q8Window w{0, -1, 0};
            if (tid < QT && s0 + tid < a.S) w = q8_window(a, b * a.S + s0 + tid, b, s0 + tid);
            wins[tid] = w;
        }
        named_barrier_sync(kUnionBarrier, kUnionThreads);
        // block of entry e, the k-th of this thread, if its query can attend a
        // token of it, else -1
        auto entry = [&](int e, int k, int qi) -> int {
            int j = -1;
            if (k < kHold) {
#pragma unroll
                for (int x = 0; x < kHold; ++x) j = x == k ? held[x] : j;
            } else {
                j = tile_ids[e];
            }
            if (j < 0 || j >= a.nb_max) {
                if (j != -1) raise_status(kStatusBadBlockId);
                return -1;
            }
            const int first = j * a.bs;
            return first <= wins[qi].hi && first + a.bs > wins[qi].lo ? j : -1;
        };
        for (int e = tid, k = 0; e < n_real; e += kUnionThreads, ++k) {
            const int j = entry(e, k, e / a.topk);
            if (j >= 0) atomicOr(&bitmap[j >> 5], 1u << (j & 31));
        }
        named_barrier_sync(kUnionBarrier, kUnionThreads);
        if (warp == 0) {  // exclusive prefix of the words' population counts
            const int per = (nwords + 31) / 32;
            int sum = 0;
            for (int k = 0; k < per; ++k) {
                const int w = lane * per + k;
                if (w < nwords) sum += __popc(bitmap[w]);
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            int run = incl - sum;
            for (int k = 0; k < per; ++k) {
                const int w = lane * per + k;
                if (w < nwords) {
                    wpre[w] = (uint32_t)run;
                    run += __popc(bitmap[w]);
                }
            }
            if (lane == 31) *s_nunion = incl;
        }
        named_barrier_sync(kUnionBarrier, kUnionThreads);
        for (int e = tid, k = 0; e < n_real; e += kUnionThreads, ++k) {
            const int qi = e / a.topk;
            const int j = entry(e, k, qi);
            if (j >= 0) {
                const int pos = (int)wpre[j >> 5] + __popc(bitmap[j >> 5] & ((1u << (j & 31)) - 1u));
                uinfo[pos].x = (uint32_t)(j * a.bs);  // the same from every query that selected it
                upage[pos] = j;
                atomicOr(&uinfo[pos].y, 1u << qi);
            }
        }
        named_barrier_sync(kUnionBarrier, kUnionThreads);
        // the blocks' pages, then their scales, several in flight
        const int n = *s_nunion;
        for (int u0 = tid; u0 < n; u0 += kHold * kUnionThreads) {
            int page[kHold];
            float ks[kHold], vs[kHold];
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const int u = u0 + k * kUnionThreads;
                page[k] = u < n ? a.table[(size_t)b * a.nb_max + upage[u]] : 0;
            }
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const bool fine = page[k] >= 0 && page[k] < a.num_pages;
                const size_t cell = fine ? (size_t)page[k] * a.H_kv + g : 0;
                ks[k] = a.ks[cell];
                vs[k] = a.vs[cell];
                if (!fine) {
                    raise_status(kStatusBadPage);
                    page[k] = -1;
                }
            }
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const int u = u0 + k * kUnionThreads;
                if (u < n) {
                    upage[u] = page[k];
                    if (page[k] < 0) uinfo[u].x = ~0u;
                    uinfo[u].z = __float_as_uint(ks[k]);
                    uinfo[u].w = __float_as_uint(log2f(fmaxf(vs[k], kMinVScale)));
                }
            }
        }
    } else {
        // ---- query rows -> shared memory, a warp per row (coalesced): scaled so
        // that the largest element is in [2^7, 2^8), high and low parts ----
        constexpr int kQWarps = kGroups * kGroupWarps, kQRows = (kRows + kQWarps - 1) / kQWarps;
        const int w0 = warp - kFirstSoftmax;
        const uint32_t inv_g = (65536u + G - 1) / G;  // r / G = r * inv_g >> 16 for r < 128, G <= 16
        const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(a.q) +
                                  (((size_t)b * a.S + s0) * a.H_q + (size_t)g * G) * kHD + 4 * lane;
        uint2 q4[kQRows];
#pragma unroll
        for (int k = 0; k < kQRows; ++k) {
            const int r = w0 + k * kQWarps, qi = (int)((r * inv_g) >> 16);
            const bool real = qi < QT && s0 + qi < a.S;
            q4[k] = real ? *reinterpret_cast<const uint2*>(q0 + ((size_t)qi * a.H_q + (r - qi * G)) * kHD)
                         : make_uint2(0u, 0u);
        }
        if (tid - kUnionThreads < kRows) mref[tid - kUnionThreads] = -INFINITY;
#pragma unroll
        for (int k = 0; k < kQRows; ++k) {
            const int r = w0 + k * kQWarps;
            if (r >= kRows) break;
            float2 f0 = bf16x2_to_f32(q4[k].x), f1 = bf16x2_to_f32(q4[k].y);
            // magnitudes order as their bits; infinities and NaN come out above
            uint32_t top = max(max(__float_as_uint(fabsf(f0.x)), __float_as_uint(fabsf(f0.y))),
                               max(__float_as_uint(fabsf(f1.x)), __float_as_uint(fabsf(f1.y))));
            top = __reduce_max_sync(0xffffffffu, top);
            int e = (int)(top >> 23) - 127;
            e = e < -100 ? -100 : e > 127 ? 127 : e;
            const float up = __uint_as_float((uint32_t)(7 - e + 127) << 23);
            if (lane == 0) {
                rowmul[r] = __uint_as_float((uint32_t)(e - 7 + 127) << 23);
                redo[r] = top >= 0x7f800000u ? 1 : 0;  // such a row is computed apart
            }
            f0.x *= up;
            f0.y *= up;
            f1.x *= up;
            f1.y *= up;
            const uint32_t hi = f32_to_e4m3x4(f0.x, f0.y, f1.x, f1.y);
            float back[4];
            e4m3x4_to_f32(hi, back);
            const uint32_t lo = f32_to_e4m3x4(f0.x - back[0], f0.y - back[1], f1.x - back[2], f1.y - back[3]);
            // byte 4 * lane of the row, 16-byte chunks swizzled
            unsigned char* d = smem + kOffQ + r * kHD + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3);
            *reinterpret_cast<uint32_t*>(d) = hi;
            *reinterpret_cast<uint32_t*>(d + kRows * kHD) = lo;
        }
        fence_proxy_async_smem();
    }
    const long long ctx = a.ctx_len[b];

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int nunion = *s_nunion;
    const int nunits = nunion * upb;
    const int npairs = (nunits + 1) / 2;
    const uint32_t tmem_base = *tmem_slot;
    // named barrier: the softmax warps before the epilogue
    constexpr int kEndBarrier = 1, kEndThreads = 32 * kGroups * kGroupWarps;

    int issued = 0;  // pairs whose copies this producer thread started
    if (warp == 0 || warp == 3) {
        // ---------------- TMA producers: K (warp 0) and V (warp 3) ----------------
        if (lane == 0) {
            uint64_t* fullb = warp == 0 ? kfull : vfull;
            uint64_t* emptyb = warp == 0 ? kempty : vempty;
            const CUtensorMap* tm = warp == 0 ? &tm_k : &tm_v;
            unsigned char* ring = smem + (warp == 0 ? kOffK : kOffV);
            int blk = 0, sub = 0;
            for (int i = 0; i < npairs; ++i) {
                const int st = i & (kStages - 1);
                int ys[2], nload = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int page = 2 * i + c < nunits ? upage[blk] : -1;
                    ys[c] = page >= 0 ? (page * a.H_kv + g) * a.bs + sub * kUnit : -1;
                    nload += page >= 0 ? 1 : 0;
                    if (++sub == upb) {
                        sub = 0;
                        ++blk;
                    }
                }
                if (i >= kStages) tile_wait(&emptyb[st], ((i / kStages) - 1) & 1, s_abort);
                if (*s_abort) break;
                issued = i + 1;
                if (nload) {
                    mbar_arrive_expect_tx(&fullb[st], (uint32_t)nload * kUnitBytes);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (ys[c] >= 0)
                            tma_load_2d(ring + st * kStageBytes + c * kUnitBytes, tm, 0, ys[c], &fullb[st]);
                } else {
                    mbar_arrive(&fullb[st]);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- S = Q K^T ----------------
        if (lane == 0) {
            // operand descriptors of stage 0; a stage is 1024 units of 16 bytes on
            const uint64_t kd0 = sw128_desc(smem_u32(smem + kOffK));
            const uint64_t qd0 = sw128_desc(smem_u32(smem + kOffQ));
            for (int i = 0; i < npairs; ++i) {
                const int ks = i & (kStages - 1);
                tile_wait(&kfull[ks], (i / kStages) & 1, s_abort);
                // the slot's last pair has had its P V done
                const int j = i - kSlots;
                if (j >= 0) tile_wait(&vempty[j & (kStages - 1)], (j / kStages) & 1, s_abort);
                if (*s_abort) break;
                tc_fence_after();
                const uint64_t kd = kd0 + (uint32_t)(ks * (kStageBytes >> 4));
                const uint32_t d = tmem_base + kColS + (i % kSlots) * 128;
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < kHD / 32; ++kk)
                        tc_mma_f8(d, qd0 + part * (kRows * kHD >> 4) + 2 * kk, kd + 2 * kk, kIdescQK,
                                  (part | kk) != 0 ? 1u : 0u);
                tc_commit(&sfull[i % kSlots]);
                tc_commit(&kempty[ks]);
            }
            // nothing of this thread may still run on the tensor core when the
            // TMEM is released
            tc_commit(&drain[0]);
            drain_wait(&drain[0], 0);
        }
    } else if (warp == 2) {
        // ---------------- O += P V ----------------
        if (lane == 0) {
            const uint64_t vd0 = sw128_desc_mn(smem_u32(smem + kOffV), kUnitBytes);
            const uint32_t o_col = tmem_base + kColO;
            for (int j = 0; j < npairs; ++j) {
                const int vs = j & (kStages - 1), slot = j % kSlots;
                tile_wait(&vfull[vs], (j / kStages) & 1, s_abort);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tile_wait(&pfull[2 * slot + c], (j / kSlots) & 1, s_abort);
                    if (*s_abort) break;
                    tc_fence_after();
                    const uint32_t p = tmem_base + kColS + slot * 128 + c * 64;
                    const uint64_t vd = vd0 + (uint32_t)(vs * (kStageBytes >> 4) + c * (kUnitBytes >> 4));
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int kt = 0; kt < kUnit / 32; ++kt)
                            tc_mma_f8_tmem_a(o_col, p + kt * 8 * kParts + part * 8, vd + kt * (4096 >> 4), kIdescPV,
                                             (j | c | part | kt) != 0 ? 1u : 0u);
                    if (c == 0) tc_commit(&obar[slot]);
                }
                if (*s_abort) break;
                tc_commit(&vempty[vs]);
            }
            tc_commit(&drain[1]);  // the epilogue waits for it too
            drain_wait(&drain[1], 0);
        }
    } else {
        // ---------------- softmax and epilogue: a thread per row and group ----------------
        const int grp = (warp - kFirstSoftmax) >> 2;
        const int quarter = warp & 3;     // TMEM lanes of this warp
        const int r = quarter * 32 + lane;
        const int qi = r / G, s = s0 + qi;
        const bool real = qi < QT && s < a.S;
        const int h = g * G + (r - qi * G);
        const size_t qrow = ((size_t)b * a.S + s) * a.H_q + h;
        const uint32_t qbit = real ? 1u << qi : 0u;
        const Q8Window win = wins[min(qi, kMaxQT - 1)];
        const uint32_t lane_addr = tmem_base + ((uint32_t)(quarter * 32) << 16);
        const int ctx32 = (int)(ctx < 0x7fffffffLL ? ctx : 0x7fffffffLL);
        // what raw S is multiplied by, with the k scale
        const float unit = (MODS ? a.scale : a.scale * kLog2e) * rowmul[r];
        float slope2 = 0.f, cap2 = 0.f, inv_cap = 0.f;
        if constexpr (MODS) {
            if (a.slopes && real) slope2 = a.slopes[h] * kLog2e;
            if (a.cap > 0.f) {
                inv_cap = 1.f / a.cap;
                cap2 = a.cap * kLog2e;
            }
        }
        float m = -INFINITY;  // the row's reference, in step with the other group's
        float l = 0.f;        // this group's share of the row sum, relative to m
        uint64_t* my_dec = decided + grp * 4 + quarter;
        // the group of the unit before this group's
        uint64_t* their_dec = decided + (grp == 0 ? kGroups - 1 : grp - 1) * 4 + quarter;
        // The group's units in order, (n_blk, n_sub) without a division; what the
        // row sees of a unit is worked out one unit ahead.
        int n_blk = grp / upb, n_sub = grp % upb;
        float ks = 0.f, lv = 0.f;    // k scale, log2 of the v scale
        int t0 = 0, lo = 0, hi = -1;  // first token; attended columns lo .. hi
        bool there = false, warp_any = false;
        auto look = [&](int u) {
            const uint4 info = uinfo[min(n_blk, kMaxUnion - 1)];
            t0 = (int)info.x + n_sub * kUnit;
            there = u < nunits && info.x != ~0u;
            ks = __uint_as_float(info.z);
            lv = __uint_as_float(info.w);
            lo = 0;
            hi = -1;
            if (there && (info.y & qbit) != 0u) {
                lo = max(win.lo - t0, 0);
                hi = min(win.hi - t0, kUnit - 1);
            }
            warp_any = __any_sync(0xffffffffu, hi >= lo);
            n_sub += kGroups;
            while (n_sub >= upb) {
                n_sub -= upb;
                ++n_blk;
            }
        };
        look(grp);
        for (int u = grp, k = 0; u < 2 * npairs; u += kGroups, ++k) {
            const int i = u >> 1, c = u & 1;               // the pair, the unit of it
            const int slot = i % kSlots, turn = i / kSlots;
            const bool mine = hi >= lo;
            const uint32_t scol = lane_addr + kColS + slot * 128 + c * 64;
            if (!warp_any) {
                // nothing of the unit concerns these rows: pass the references on, P = 0
                if (u > 0) tile_wait(their_dec, (grp == 0 ? k - 1 : k) & 1, s_abort);
                __syncwarp();  // every lane has seen the phase: once passed on, it can be followed by two more
                if (lane == 0) mbar_arrive(my_dec);
                tile_wait(&sfull[slot], turn & 1, s_abort);
                tc_fence_after();
                uint32_t none[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) none[e] = 0u;
                tmem_st32(scol, none);
                tmem_st16(scol + 32, reinterpret_cast<const uint32_t(&)[16]>(none));
            } else {
            tile_wait(&sfull[slot], turn & 1, s_abort);
            tc_fence_after();
            float mx = -INFINITY;
            float mul = unit * ks;
            uint32_t sv[64];
            {
                tmem_ld64(scol, sv);
                const bool partial = __any_sync(0xffffffffu, mine && hi - lo != kUnit - 1);
                if constexpr (MODS) {
                    // raw S -> capped, biased logits in log2 units; then mul = 1
                    float xs[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e) xs[e] = __uint_as_float(sv[e]);
                    if (a.cap > 0.f) {
                        const float um = mul * inv_cap;
                        // what masked tokens hold has no say in how tanh is computed
                        if (partial) {
#pragma unroll
                            for (int e = 0; e < 64; ++e) xs[e] = e >= lo && e <= hi ? xs[e] : 0.f;
                        }
                        float pa[4], pi[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) pa[k] = pi[k] = xs[k];
#pragma unroll
                        for (int e = 4; e < 64; e += 2) {
                            pa[(e >> 1) & 3] = fmax3(pa[(e >> 1) & 3], xs[e], xs[e + 1]);
                            pi[(e >> 1) & 3] = fmin3(pi[(e >> 1) & 3], xs[e], xs[e + 1]);
                        }
                        const float big = fmaxf(fmaxf(fmaxf(pa[0], pa[1]), fmaxf(pa[2], pa[3])),
                                                -fminf(fminf(pi[0], pi[1]), fminf(pi[2], pi[3]))) * fabsf(um);
                        // cap2 * tanh(u), u = S * um, as u * (cap2 + v * (cap2 T0 + v * (cap2 T1 + ...))),
                        // v = u^2, as long as every |u| of the warp is small; on packed pairs. In u,
                        // where every term is in range: powers of um alone would underflow.
                        const float2 z2 = make_float2(0.f, 0.f), um2 = make_float2(um, um), A2 = make_float2(cap2, cap2);
                        if (!__any_sync(0xffffffffu, mine && !(big <= kTanhTiny))) {
                            const float2 B0 = make_float2(cap2 * kTanhT0, cap2 * kTanhT0);
                            const float2 B1 = make_float2(cap2 * kTanhT1, cap2 * kTanhT1);
                            const float2 B2 = make_float2(cap2 * kTanhT2, cap2 * kTanhT2);
#pragma unroll
                            for (int e = 0; e < 64; e += 2) {
                                const float2 x = ffma2(make_float2(xs[e], xs[e + 1]), um2, z2);
                                const float2 v = ffma2(x, x, z2);
                                const float2 t = ffma2(v, ffma2(v, ffma2(v, B2, B1), B0), A2);
                                const float2 y = ffma2(x, t, z2);
                                xs[e] = y.x;
                                xs[e + 1] = y.y;
                            }
                        } else if (!__any_sync(0xffffffffu, mine && !(big <= kTanhSmall))) {
                            const float2 B0 = make_float2(cap2 * kTanhC0, cap2 * kTanhC0);
                            const float2 B1 = make_float2(cap2 * kTanhC1, cap2 * kTanhC1);
                            const float2 B2 = make_float2(cap2 * kTanhC2, cap2 * kTanhC2);
                            const float2 B3 = make_float2(cap2 * kTanhC3, cap2 * kTanhC3);
                            const float2 B4 = make_float2(cap2 * kTanhC4, cap2 * kTanhC4);
#pragma unroll
                            for (int e = 0; e < 64; e += 2) {
                                const float2 x = ffma2(make_float2(xs[e], xs[e + 1]), um2, z2);
                                const float2 v = ffma2(x, x, z2);
                                float2 t = ffma2(v, ffma2(v, B4, B3), B2);
                                t = ffma2(v, ffma2(v, ffma2(v, t, B1), B0), A2);
                                const float2 y = ffma2(x, t, z2);
                                xs[e] = y.x;
                                xs[e + 1] = y.y;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 64; ++e) xs[e] = cap2 * q8_tanh(xs[e] * um);
                        }
                    } else {
                        const float m2 = mul * kLog2e;
#pragma unroll
                        for (int e = 0; e < 64; ++e) xs[e] *= m2;
                    }
                    if (a.slopes) {
                        const float d0 = (float)(win.p - t0);
#pragma unroll
                        for (int e = 0; e < 64; ++e) xs[e] = fmaf(-slope2, fabsf(d0 - (float)e), xs[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 64; ++e) sv[e] = __float_as_uint(xs[e]);
                    mul = 1.f;
                }
                if (partial) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        sv[e] = e >= lo && e <= hi ? sv[e] : __float_as_uint(-INFINITY);
                }
                float pm[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) pm[k] = __uint_as_float(sv[k]);
#pragma unroll
                for (int e = 8; e < 64; e += 2)
                    pm[(e >> 1) & 7] = fmax3(pm[(e >> 1) & 7], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                mx = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
                mx = mine ? mx * mul + lv : -INFINITY;
            }
            // the reference after the unit before this one, then after this one
            if (u > 0) tile_wait(their_dec, (grp == 0 ? k - 1 : k) & 1, s_abort);
            const float m_in = mref[r];
            float corr = 1.f;
            const bool moves = mx > m_in + kLazy;
            const bool any_moves = __any_sync(0xffffffffu, moves);  // and every lane has read mref
            if (__any_sync(0xffffffffu, m_in != m)) {
                l *= m_in != m ? fast_exp2(m - m_in) : 1.f;  // m = -inf: nothing summed yet
                m = m_in;
            }
            if (any_moves) {
                if (moves) {
                    if (m > -INFINITY) corr = fast_exp2(m - mx);
                    l *= corr;
                    m = mx;
                    mref[r] = m;
                }
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(my_dec);
            const float add = lv + kShift - m;
            const float2 mul2 = make_float2(mul, mul), add2 = make_float2(add, add);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 32 tokens at a time: 8 words of each part
                uint32_t pk[16], pl[8];
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float2 p[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int t = 32 * h + 4 * e + 2 * k;
                            const float2 x = ffma2(make_float2(__uint_as_float(sv[t]), __uint_as_float(sv[t + 1])), mul2, add2);
                            p[k] = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                            sum[k] = fadd2(sum[k], p[k]);
                        }
                        split_weights(p[0].x, p[0].y, p[1].x, p[1].y, pk[e], pk[8 + e], pl[e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = pk[8 + e] = pl[e] = 0u;
                }
                __syncwarp();
                tmem_st16(scol + 8 * kParts * h, pk);
                tmem_st8(scol + 8 * kParts * h + 16, pl);
            }
            if (mine) {
                const float2 t = fadd2(sum[0], sum[1]);
                l = fmaf(t.x + t.y, fast_exp2(-lv), l);
            }
            if (any_moves && __any_sync(0xffffffffu, corr != 1.f)) {
                // O holds earlier units of these rows: rescale once the previous
                // unit's P V has landed
                if (c == 1)
                    tile_wait(&obar[slot], turn & 1, s_abort);
                else
                    tile_wait(&vempty[(i - 1) & (kStages - 1)], ((i - 1) / kStages) & 1, s_abort);
                tc_fence_after();
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t ov[32];
                    tmem_ld32(lane_addr + kColO + ch * 32, ov);
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
                    tmem_st32(lane_addr + kColO + ch * 32, ov);
                }
            }
            }
            tmem_wait_st();
            // V rows of tokens past the context and of absent units must be zero
            // before the MMA reads them (this thread: half of row r / 2 of the unit)
            if (!there || t0 > ctx32 - kUnit) {
                const int vs = i & (kStages - 1);
                tile_wait(&vfull[vs], (i / kStages) & 1, s_abort);
                const int vr = r >> 1;
                if (!there || t0 + vr >= ctx32) {
                    unsigned char* vt = smem + kOffV + vs * kStageBytes + c * kUnitBytes + vr * 128;
#pragma unroll
                    for (int x = 4 * (r & 1); x < 4 * (r & 1) + 4; ++x)
                        *reinterpret_cast<uint4*>(vt + ((x ^ (vr & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[2 * slot + c]);
            look(u + kGroups);
        }
        // ---------------- epilogue: O / l -> bf16, in chunks of 32 dims ----------------
        named_barrier_sync(kEndBarrier, kEndThreads);  // every group's references are final
        const float m_end = mref[r];
        if (m_end != m) l *= fast_exp2(m - m_end);
        lsum[grp * 128 + r] = l;
        tile_wait(&drain[1], 0, s_abort);
        named_barrier_sync(kEndBarrier, kEndThreads);
        tc_fence_after();
        // no role waits for anything any more: the same for every thread
        const bool gave_up = *s_abort != 0;
        float L = 0.f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) L += lsum[k * 128 + r];
        if (gave_up) L = 0.f;
        const float inv = 1.f / L;
        if (a.lse && real && grp == 0) a.lse[qrow] = L == 0.f ? -INFINITY : m_end - kShift + log2f(L);
        __nv_bfloat16* o0 = static_cast<__nv_bfloat16*>(a.out) + (((size_t)b * a.S + s0) * a.H_q + (size_t)g * G) * kHD;
        if (gave_up) {
            // zeros, not through the K ring: copies into it may still be under way
            if (real)
                for (int c = grp; c < kHD / 8; c += kGroups)
                    *reinterpret_cast<uint4*>(o0 + ((size_t)qi * a.H_q + (r - qi * G)) * kHD + 8 * c) = make_uint4(0, 0, 0, 0);
        } else {
        // through the K ring (every copy and MMA of it is done), rows padded by 16
        // bytes, so that rows leave whole
        constexpr int kPitch = 2 * kHD + 16;
        bool bad = false;
        for (int ch = grp; ch < 4; ch += kGroups) {
            uint32_t ov[32];
            tmem_ld32(lane_addr + kColO + ch * 32, ov);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                // a row that attends nothing is zero whatever O holds
                const float x = L == 0.f ? 0.f : __uint_as_float(ov[2 * e]) * inv;
                const float y = L == 0.f ? 0.f : __uint_as_float(ov[2 * e + 1]) * inv;
                bad = bad || x != x || y != y;
                w[e] = pack_bf16x2(x, y);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(smem + kOffK + r * kPitch + ch * 64 + 16 * e) =
                    make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
        if (real && bad) redo[r] = 1;
        named_barrier_sync(kEndBarrier, kEndThreads);
        const uint32_t inv_g = (65536u + G - 1) / G;
        for (int x = tid - 32 * kFirstSoftmax; x < kRows * 16; x += kEndThreads) {
            const int row = x >> 4, c = x & 15, q = (int)((row * inv_g) >> 16);
            if (q < QT && s0 + q < a.S)
                *reinterpret_cast<uint4*>(o0 + ((size_t)q * a.H_q + (row - q * G)) * kHD + 8 * c) =
                    *reinterpret_cast<const uint4*>(smem + kOffK + row * kPitch + 16 * c);
        }
        // rows that met a NaN, a warp each
        const bool again = __any_sync(0xffffffffu, redo[lane] | redo[lane + 32] | redo[lane + 64] | redo[lane + 96]);
        if (again) {
            named_barrier_sync(kEndBarrier, kEndThreads);  // all rows have left the K ring
            for (int x = warp - kFirstSoftmax; x < QT * G; x += kGroups * kGroupWarps)
                if (redo[x] && s0 + x / G < a.S)
                    q8_row_by_warp(a, b * a.S + s0 + x / G, g * G + x % G,
                                   reinterpret_cast<float*>(smem + kOffK) + warp * kHD);
        }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(kTmemCols)
                     : "memory");
    }
    // a tile that gave up: its copies still land before the CTA's memory is reused
    if (*s_abort && lane == 0 && (warp == 0 || warp == 3))
        for (int i = max(0, issued - kStages); i < issued; ++i)
            drain_wait(&(warp == 0 ? kfull : vfull)[i & (kStages - 1)], (i / kStages) & 1);
}

}  // namespace lci
