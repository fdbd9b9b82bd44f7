// cache_evict.cuh -- accumulated attention weight per block, and the eviction
// of the blocks with the least of it.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "ptx.cuh"

namespace lci {

namespace bwu {
constexpr int kRange = 1024;   // blocks of a sequence one cluster accumulates
constexpr int kMaxSplit = 16;  // CTAs of a cluster, each taking a share of the rows
constexpr int kMaxWarps = 32;
constexpr int kRowsAhead = 8;  // rows a warp loads before it adds them
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
    pdl_wait();
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
#pragma unroll 8
        for (int w = 0; w < nw; ++w) x += (double)hist[w * kRange + j];
        total[j] = x;
    }
    if (nsplit > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        // each CTA of the cluster finishes a share of the blocks
        for (int j = split * nt + tid; j < width; j += nsplit * nt) {
            double y[kMaxSplit], x = 0.0;
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c)
                y[c] = c < nsplit ? cluster.map_shared_rank(total, c)[j] : 0.0;
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c) x += y[c];
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

// Eviction, one CTA per sequence; thread t takes blocks t, t + threads, ...
// (coalesced loads and nearly coalesced stores). The m-th largest weight key
// among the blocks that are neither the first `sink` nor the last `recent` is
// found digit by digit (11, 11 and 10 bits) with a histogram in shared memory;
// a warp's lanes that share their first lane's digit count as one addition, so
// that tied weights do not serialise. Ties go to the lower block, and ballots
// with a prefix sum over the (row of blocks, warp) counts give every block its
// place: kept blocks, then freed ones, then the rest of the row, each in order.
// Every input is read before the first write, so outputs may be the inputs.
// Bound by the latency of that chain.
template <int IPT>
__global__ void __launch_bounds__(1024) cache_evict_kernel(
    const int32_t* table, const int32_t* ctx_len, const float* weight, int nb_max, int bs,
    int budget, int sink, int recent, int32_t* table_out, int32_t* ctx_out, float* weight_out,
    int32_t* kept_ids, int32_t* freed) {
    constexpr int kBins = 2048;
    __shared__ int s_hist[kBins];
    __shared__ int s_pick[2];  // chosen bin, entries in larger bins
    __shared__ int s_scan[32];
    __shared__ int s_base[IPT * 32];
    pdl_wait();
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int b = blockIdx.x;
    const size_t base = (size_t)b * nb_max;
    uint32_t key[IPT];
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = i * nt + tid;
        key[i] = j < nb_max ? weight_key(weight[base + j]) : 0u;
    }
    const int ctx = ctx_len[b];
    const long long want = ctx > 0 ? ((long long)ctx + bs - 1) / bs : 0;
    // a context longer than its table row is left as it is
    const bool bad = want > nb_max;
    if (bad && tid == 0) raise_status(kStatusBadBlockId);
    const int n = (int)(bad ? 0 : want);
    const bool trim = n > budget;
    // Exclusive prefix, in block order, of flags given as a bit per item:
    // s_base[i * nw + warp] is the count before row i of this warp.
    auto prefix = [&](uint32_t flags) -> int {
#pragma unroll
        for (int i = 0; i < IPT; ++i) {
            const uint32_t v = __ballot_sync(0xffffffffu, (flags >> i) & 1u);
            if (lane == 0) s_base[i * nw + warp] = __popc(v);
        }
        __syncthreads();
        int total;
        const int mine = cta_exclusive_sum(tid < IPT * nw ? s_base[tid] : 0, s_scan, total);
        if (tid < IPT * nw) s_base[tid] = mine;
        __syncthreads();
        return total;
    };
    // candidates: the middle blocks of a sequence that is trimmed
    uint32_t cand = 0u, keep = 0u;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = i * nt + tid;
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
            uint32_t t = 0u, known = 0u;  // digits found so far, and their bits
            int need = m;                 // entries still to take among those that match t
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
                const uint32_t digits = pass == 2 ? 1023u : 2047u;
                for (int e = tid; e < kBins; e += nt) s_hist[e] = 0;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < IPT; ++i) {
                    const bool on = ((cand >> i) & 1u) && (key[i] & known) == t;
                    const uint32_t act = __ballot_sync(0xffffffffu, on);
                    if (act == 0u) continue;
                    const uint32_t d = (key[i] >> shift) & digits;
                    const int first = __ffs(act) - 1;
                    const uint32_t d0 = __shfl_sync(0xffffffffu, d, first);
                    const uint32_t same = __ballot_sync(0xffffffffu, on && d == d0);
                    if (lane == first)
                        atomicAdd(&s_hist[d0], __popc(same));
                    else if (on && d != d0)
                        atomicAdd(&s_hist[d], 1);
                }
                __syncthreads();
                // the bin, from the largest down, in which the need-th entry lies
                const int per = (kBins + nt - 1) / nt;
                int sum = 0;
                for (int e = 0; e < per; ++e) {
                    const int r = tid * per + e;
                    if (r < kBins) sum += s_hist[kBins - 1 - r];
                }
                int all;
                int before = cta_exclusive_sum(sum, s_scan, all);
                if (before < need && before + sum >= need) {  // one thread
                    for (int e = 0; e < per; ++e) {
                        const int c = s_hist[kBins - 1 - (tid * per + e)];
                        if (before + c >= need) {
                            s_pick[0] = kBins - 1 - (tid * per + e);
                            s_pick[1] = before;
                            break;
                        }
                        before += c;
                    }
                }
                __syncthreads();
                t |= (uint32_t)s_pick[0] << shift;
                known |= digits << shift;
                need -= s_pick[1];
            }
            uint32_t ties = 0u;
#pragma unroll
            for (int i = 0; i < IPT; ++i)
                if ((cand >> i) & 1u) {
                    if (key[i] > t)
                        keep |= 1u << i;
                    else if (key[i] == t)
                        ties |= 1u << i;
                }
            prefix(ties);
#pragma unroll
            for (int i = 0; i < IPT; ++i) {
                const uint32_t v = __ballot_sync(0xffffffffu, (ties >> i) & 1u);
                if (((ties >> i) & 1u) && s_base[i * nw + warp] + __popc(v & below) < need)
                    keep |= 1u << i;  // the lowest blocks first
            }
            __syncthreads();  // s_base is written again
        }
    }
    int page[IPT];
    float w[IPT];
#pragma unroll
    for (int i = 0; i < IPT; ++i) {  // read again (from L2): not held through the search
        const int j = i * nt + tid;
        page[i] = j < nb_max ? table[base + j] : 0;
        w[i] = j < nb_max ? weight[base + j] : 0.f;
    }
    const int n_keep = prefix(keep);  // its barriers stand between the reads and the writes
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = i * nt + tid;
        const bool k = (keep >> i) & 1u;
        const uint32_t v = __ballot_sync(0xffffffffu, k);
        const int pos = s_base[i * nw + warp] + __popc(v & below);  // kept blocks before j
        if (j < nb_max) {
            const int to = j >= n ? j : k ? pos : n_keep + (j - pos);
            table_out[base + to] = page[i];
            weight_out[base + to] = k || bad ? w[i] : 0.f;
            if (k && kept_ids && pos < budget) kept_ids[(size_t)b * budget + pos] = j;
        }
    }
    if (kept_ids)
        for (int i = n_keep + tid; i < budget; i += nt) kept_ids[(size_t)b * budget + i] = -1;
    if (tid == 0) {
        const int gone = n - n_keep;
        ctx_out[b] = ctx - gone * bs;
        if (freed) freed[b] = gone;
    }
}

}  // namespace lci
