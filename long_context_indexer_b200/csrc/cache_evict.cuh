// cache_evict.cuh -- accumulated attention weight per block, and the eviction
// of the blocks with the least of it.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace lci {

namespace bwu {
constexpr int kRange = 1024;   // blocks of a sequence one cluster accumulates
constexpr int kMaxSplit = 8;   // CTAs of a cluster, each taking a share of the rows
constexpr int kMaxWarps = 16;
constexpr int kRowsAhead = 4;  // rows a warp loads before it adds them
constexpr size_t smem_bytes(int warps) { return (size_t)warps * kRange * 4 + kRange * 8; }
}  // namespace bwu

// weight[b][j] = decay * weight[b][j] + sum over s, i with ids[b][s][i] == j of
// sum_g mass[b][s][g][i].
//
// Every sum runs in a fixed order without atomics, so results repeat bit for
// bit: a warp adds its rows one after the other into its own row of kRange
// fp32 sums in shared memory (the ids of one row are distinct, so its 32 lanes
// never meet), the CTA adds its warps' sums in 64 bits, and the first CTA of
// the cluster adds the CTAs' (distributed shared memory) to the weight. A
// sequence of more than kRange blocks is cut into ranges, each with its own
// cluster that reads every entry and keeps those of its range.
__global__ void __launch_bounds__(bwu::kMaxWarps * 32) block_weight_update_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ mass, int S, int H_kv, int topk,
    int nb_max, float decay, float* __restrict__ weight, int nsplit) {
    using namespace bwu;
    namespace cg = cooperative_groups;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    double* total = reinterpret_cast<double*>(smem_raw);            // [kRange]
    float* hist = reinterpret_cast<float*>(smem_raw + kRange * 8);  // [warps][kRange]
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int split = blockIdx.x, b = blockIdx.z;
    const int j0 = blockIdx.y * kRange;
    const int width = min(kRange, nb_max - j0);
    float* mine = hist + warp * kRange;
    for (int j = lane; j < width; j += 32) mine[j] = 0.f;
    __syncwarp();
    const int stride = nsplit * nw;
    for (int s0 = split * nw + warp; s0 < S; s0 += stride * kRowsAhead) {
        for (int i0 = 0; i0 < topk; i0 += 32) {
            const int i = i0 + lane;
            int id[kRowsAhead];
            float add[kRowsAhead];
#pragma unroll
            for (int k = 0; k < kRowsAhead; ++k) {
                const int s = s0 + k * stride;
                id[k] = -1;
                add[k] = 0.f;
                if (s < S && i < topk) {
                    id[k] = ids[((size_t)b * S + s) * topk + i];
                    const float* m = mass + ((size_t)b * S + s) * H_kv * topk + i;
                    float x = 0.f;
                    for (int g = 0; g < H_kv; ++g) x += m[(size_t)g * topk];
                    add[k] = x;
                }
            }
#pragma unroll
            for (int k = 0; k < kRowsAhead; ++k) {
                const int j = id[k];
                if (j < -1 || j >= nb_max) {
                    if (blockIdx.y == 0) raise_status(kStatusBadBlockId);
                } else if (j >= j0 && j < j0 + width) {
                    mine[j - j0] += add[k];
                }
                __syncwarp();
            }
        }
    }
    __syncthreads();
    for (int j = tid; j < width; j += nt) {
        double x = 0.0;
        for (int w = 0; w < nw; ++w) x += (double)hist[w * kRange + j];
        total[j] = x;
    }
    if (nsplit > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        // each CTA of the cluster finishes a share of the blocks
        for (int j = split * nt + tid; j < width; j += nsplit * nt) {
            double x = 0.0;
            for (int c = 0; c < nsplit; ++c) x += cluster.map_shared_rank(total, c)[j];
            float* w = weight + (size_t)b * nb_max + j0 + j;
            *w = (float)((double)decay * (double)*w + x);
        }
        cluster.sync();  // no CTA leaves while its sums are read
    } else {
        for (int j = tid; j < width; j += nt) {  // this thread's own sums
            float* w = weight + (size_t)b * nb_max + j0 + j;
            *w = (float)((double)decay * (double)*w + total[j]);
        }
    }
}

// Order-preserving key of a weight; NaN counts as the heaviest.
__device__ __forceinline__ uint32_t weight_key(float w) {
    return w != w ? 0xffffffffu : score_key(w);
}

// Exclusive prefix sum of one int per thread over the CTA (up to 32 warps).
__device__ __forceinline__ int cta_exclusive_sum(int v, int* scratch, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int ws = lane < nw ? scratch[lane] : 0;
    int wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi += t;
    }
    total = __shfl_sync(0xffffffffu, wi, 31);
    const int before = __shfl_sync(0xffffffffu, wi - ws, warp);
    __syncthreads();  // scratch may be used again
    return before + incl - v;
}

// Eviction, one CTA per sequence, IPT consecutive blocks per thread in
// registers: the m-th largest weight key among the blocks that are neither the
// first `sink` nor the last `recent` is found by a four-way search on its bits
// (16 counting rounds: one packed warp reduction and one barrier each, whatever
// the distribution of the weights), ties go to the lower block, and two prefix
// sums give every block its place: kept blocks, then freed ones, then the rest
// of the row, each in order. All inputs are in registers before the first
// write, so outputs may be the inputs.
template <int IPT>
__global__ void __launch_bounds__(1024) cache_evict_kernel(
    const int32_t* table, const int32_t* ctx_len, const float* weight, int nb_max, int bs,
    int budget, int sink, int recent, int32_t* table_out, int32_t* ctx_out, float* weight_out,
    int32_t* kept_ids, int32_t* freed) {
    __shared__ uint32_t s_cnt[2][32];
    __shared__ int s_scan[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int b = blockIdx.x;
    const size_t base = (size_t)b * nb_max;
    const int ctx = ctx_len[b];
    const long long want = ctx > 0 ? ((long long)ctx + bs - 1) / bs : 0;
    // a context longer than its table row is left as it is
    const bool bad = want > nb_max;
    if (bad && tid == 0) raise_status(kStatusBadBlockId);
    const int n = (int)(bad ? 0 : want);
    const bool trim = n > budget;
    int page[IPT];
    float w[IPT];
    uint32_t key[IPT];
    const int j0 = tid * IPT;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = j0 + i;
        page[i] = j < nb_max ? table[base + j] : 0;
        w[i] = j < nb_max ? weight[base + j] : 0.f;
    }
    // candidates: the middle blocks of a sequence that is trimmed
    uint32_t cand = 0, keep = 0;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = j0 + i;
        key[i] = weight_key(w[i]);
        if (j < n) {
            if (!trim || j < sink || j >= n - recent)
                keep |= 1u << i;
            else
                cand |= 1u << i;
        }
    }
    if (trim) {  // the same for every thread of the CTA
        const int m = budget - sink - recent;  // candidates to keep, fewer than there are
        if (m > 0) {
            // t: the largest key value with at least m candidates at or above it
            uint32_t t = 0u;
#pragma unroll 1
            for (int bit = 30, round = 0; bit >= 0; bit -= 2, ++round) {
                const uint32_t q1 = t | (1u << bit), q2 = t | (2u << bit), q3 = t | (3u << bit);
                uint32_t c = 0u;
#pragma unroll
                for (int i = 0; i < IPT; ++i)
                    if ((cand >> i) & 1u)
                        c += (key[i] >= q1 ? 1u : 0u) + (key[i] >= q2 ? 1u << 10 : 0u) +
                             (key[i] >= q3 ? 1u << 20 : 0u);
                c = __reduce_add_sync(0xffffffffu, c);  // each count <= 32 * 16 < 2^10
                if (lane == 0) s_cnt[round & 1][warp] = c;
                __syncthreads();
                const uint32_t v = lane < nw ? s_cnt[round & 1][lane] : 0u;
                const int c1 = __reduce_add_sync(0xffffffffu, v & 1023u);
                const int c2 = __reduce_add_sync(0xffffffffu, (v >> 10) & 1023u);
                const int c3 = __reduce_add_sync(0xffffffffu, v >> 20);
                t = c3 >= m ? q3 : c2 >= m ? q2 : c1 >= m ? q1 : t;
            }
            uint32_t ties = 0u;
            int above = 0;
#pragma unroll
            for (int i = 0; i < IPT; ++i)
                if ((cand >> i) & 1u) {
                    if (key[i] > t) {
                        keep |= 1u << i;
                        ++above;
                    } else if (key[i] == t) {
                        ties |= 1u << i;
                    }
                }
            int n_above, n_ties;
            cta_exclusive_sum(above, s_scan, n_above);
            int left = m - n_above - cta_exclusive_sum(__popc(ties), s_scan, n_ties);
#pragma unroll
            for (int i = 0; i < IPT; ++i)
                if ((ties >> i) & 1u) {
                    if (left > 0) keep |= 1u << i;
                    --left;
                }
        }
    }
    int n_keep;
    int pos = cta_exclusive_sum(__popc(keep), s_scan, n_keep);
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = j0 + i;
        if (j >= nb_max) break;
        const bool k = (keep >> i) & 1u;
        // a freed block follows the kept ones, in order; others stay
        const int to = j >= n ? j : k ? pos : n_keep + (j - pos);
        table_out[base + to] = page[i];
        weight_out[base + to] = k || bad ? w[i] : 0.f;
        if (k && kept_ids && pos < budget) kept_ids[(size_t)b * budget + pos] = j;
        pos += k ? 1 : 0;
    }
    if (kept_ids)
        for (int i = n_keep + tid; i < budget; i += blockDim.x) kept_ids[(size_t)b * budget + i] = -1;
    if (tid == 0) {
        const int gone = n - n_keep;
        ctx_out[b] = ctx - gone * bs;
        if (freed) freed[b] = gone;
    }
}

}  // namespace lci
