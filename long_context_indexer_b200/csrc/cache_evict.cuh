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
constexpr int kMinWarps = 4, kMaxWarps = 32;
constexpr int kOwn = kRange / (kMinWarps * 32);  // blocks a thread finishes
// items (32 entries of a row) that a warp loads before it adds them: one where it
// has one, else what the registers of 1024 threads hold
constexpr int kAheadMany = 8;
// the cluster's sums of this CTA's share of the blocks, and a sum per warp and block
constexpr int kRecv = kRange + kMaxSplit;
constexpr size_t smem_bytes(int warps) { return (size_t)warps * kRange * (4 + 1) + kRecv * 8; }
}  // namespace bwu

// weight[b][j] = decay * weight[b][j] + sum over s, i with ids[b][s][i] == j of
// sum_g mass[b][s][g][i].
//
// Every sum runs in a fixed order without atomics, so results repeat bit for
// bit: a warp adds its rows one after the other into its own row of kRange
// fp32 sums in shared memory (where lanes hold the same id, they add in their
// order), the CTA adds its warps' sums in 64 bits and stores each into the
// CTA of the cluster that finishes the block (distributed shared memory), which
// adds the CTAs' to the weight. A sequence of more than kRange blocks is cut into
// ranges, each with its own cluster that reads every entry and keeps those of its
// range. Bound by latency: an 8K prompt's 2.1 MB (0.3 us of HBM) in 10.3 us (1.6 of
// them the test for repeats; a match over the warp for each item took 15), a
// serving step of 32 sequences in 2.3. A warp's loads do not wait for one another:
// with loads behind a test per row and KV head, 64 rows of 64 entries on 8 heads
// took 42 us against 6.9.
template <int kAhead>
__global__ void __launch_bounds__((kAhead == 1 ? bwu::kMinWarps : bwu::kMaxWarps) * 32) block_weight_update_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ mass, int S, int H_kv, int topk,
    int nb_max, float decay, float* __restrict__ weight, int nsplit) {
    using namespace bwu;
    namespace cg = cooperative_groups;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    double* recv = reinterpret_cast<double*>(smem_raw);            // [CTA][share]
    float* hist = reinterpret_cast<float*>(smem_raw + kRecv * 8);  // [warps][kRange]
    pdl_wait();
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int split = blockIdx.x, b = blockIdx.z;
    if (nsplit > 1) cluster_arrive_relaxed();
    const int j0 = blockIdx.y * kRange;
    const int width = min(kRange, nb_max - j0);
    float* mine = hist + warp * kRange;
    volatile uint8_t* owner = reinterpret_cast<uint8_t*>(hist + nw * kRange) + warp * kRange;
    // the blocks that this CTA finishes; their weights are loaded together, ahead
    // of everything else where registers allow it
    const int share = (width + nsplit - 1) / nsplit;
    const int lo = split * share, hi = min(width, lo + share);
    float* wrow = weight + (size_t)b * nb_max + j0;
    float old[kOwn];
    auto load_weights = [&]() {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) old[k] = lo + tid + k * nt < hi ? wrow[lo + tid + k * nt] : 0.f;
    };
    auto cta_sum = [&](int j) {
        constexpr int kChains = kAhead == 1 ? 4 : 1;  // the warps are a multiple of 4
        double x[kChains] = {};
#pragma unroll 8
        for (int w = 0; w < nw; w += kChains)
#pragma unroll
            for (int y = 0; y < kChains; ++y) x[y] += (double)hist[(w + y) * kRange + j];
#pragma unroll
        for (int y = 1; y < kChains; ++y) x[0] += x[y];
        return x[0];
    };
    if constexpr (kAhead == 1) load_weights();
    for (int j = lane; j < width; j += 32) mine[j] = 0.f;
    __syncwarp();
    // Items, a row's 32 entries each; this warp's are `first` and every stride-th
    // behind it. Entries past the row, and items past the last, repeat a valid
    // address and add nothing, so that no load waits for a branch.
    const int chunks = (topk + 31) >> 5;
    const long long items = (long long)S * chunks;
    const int stride = nsplit * nw, ds = stride / chunks, dc = stride - ds * chunks;
    const int first = split * nw + warp;
    unsigned s = first / chunks;
    int c = first - (int)s * chunks;
    for (long long n0 = first; n0 < items; n0 += (long long)stride * kAhead) {
        const int here = (int)min((long long)kAhead, (items - n0 + stride - 1) / stride);
        int id[kAhead];
        float add[kAhead];
        const float* mp[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool on = k < here;
            const int i = 32 * c + lane, at = min(i, topk - 1);
            const size_t row = (size_t)b * S + min(s, (unsigned)S - 1u);
            id[k] = __ldg(ids + row * topk + at);
            mp[k] = mass + row * H_kv * topk + at;
            add[k] = __ldg(mp[k]);
            if (!on || i >= topk) id[k] = -1;
            s += ds;
            c += dc;
            if (c >= chunks) {
                c -= chunks;
                ++s;
            }
        }
#pragma unroll kAhead == 1 ? 4 : 1
        for (int g = 1; g < H_kv; ++g) {
            float x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) x[k] = __ldg(mp[k] += topk);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) add[k] += x[k];
        }
        // Lanes that hold the same id of a row would meet: each leaves its number with
        // the block, and one of them finds another's.
        unsigned other = 0u;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned at_j = (unsigned)id[k] - (unsigned)j0;
            const bool on = at_j < (unsigned)width;
            if (on) owner[at_j] = (uint8_t)lane;
            __syncwarp();
            other |= on ? owner[at_j] ^ (unsigned)lane : 0u;
            __syncwarp();
        }
        const bool again = __any_sync(0xffffffffu, other != 0u);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned at_j = (unsigned)id[k] - (unsigned)j0;
            if (at_j < (unsigned)width) {
                if (!again) mine[at_j] += add[k];
            } else if ((unsigned)id[k] + 1u > (unsigned)nb_max) {
                raise_status(kStatusBadBlockId);
            }
            __syncwarp();
        }
        if (again) {  // one entry after the other
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                for (int x = 0; x < 32; ++x) {
                    const unsigned at_j = (unsigned)id[k] - (unsigned)j0;
                    if (x == lane && at_j < (unsigned)width) mine[at_j] += add[k];
                    __syncwarp();
                }
        }
    }
    if constexpr (kAhead > 1) load_weights();
    __syncthreads();
    if (nsplit > 1) {
        cluster_wait();  // every CTA of the cluster runs
        for (int j = tid; j < width; j += nt) {
            const int owner = j / share;
            cg::this_cluster().map_shared_rank(recv, owner)[split * share + j - owner * share] = cta_sum(j);
        }
        cluster_arrive();
        cluster_wait();
    }
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int j = lo + tid + k * nt;
        if (j < hi) {
            double x = 0.0;
            if (nsplit > 1)
                for (int c = 0; c < nsplit; ++c) x += recv[c * share + j - lo];
            else
                x = cta_sum(j);
            wrow[j] = (float)((double)decay * (double)old[k] + x);
        }
    }
}

// Order-preserving key of a weight; NaN counts as the heaviest.
__device__ __forceinline__ uint32_t weight_key(float w) {
    return w != w ? 0xffffffffu : score_key(w);
}

// Exclusive prefix sum of one int per thread over the CTA (up to 32 warps).
// scratch[32] must not be written again before the CTA's next barrier.
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
    const int ws = lane < nw ? scratch[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, ws);
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
    return before + incl - v;
}

// Eviction, one cluster of 1 to 8 CTAs per sequence, each CTA IPT * threads
// consecutive blocks, thread t of it blocks t, t + threads, ... (coalesced loads
// and nearly coalesced stores). The m-th largest weight key among the blocks
// that are neither the first `sink` nor the last `recent` is found digit by
// digit (11, 11 and 10 bits): every CTA counts its blocks in a histogram in
// shared memory and adds its bins that are not empty to every CTA's sum
// (distributed shared memory). A warp's lanes that share their first lane's
// digit count as one addition, so that tied weights do not serialise, and the
// search ends as soon as a whole bin is kept. Ties go to the lower block,
// and ballots with a prefix sum over the (CTA, row of blocks, warp) counts give
// every block its place: kept blocks, then freed ones, then the rest of the row,
// each in order. Every input is read before a barrier of the cluster that
// precedes the first write, so outputs may be the inputs. Bound by the latency
// of that chain (a cluster barrier per digit and per prefix); one CTA for all 16384 blocks of a
// sequence was bound by its instructions (28 us against 12 for 8 sequences).
template <int IPT>
__global__ void __launch_bounds__(1024) cache_evict_kernel(
    const int32_t* table, const int32_t* ctx_len, const float* weight, int nb_max, int bs,
    int budget, int sink, int recent, int32_t* table_out, int32_t* ctx_out, float* weight_out,
    int32_t* kept_ids, int32_t* freed, int nsplit) {
    namespace cg = cooperative_groups;
    constexpr int kBins = 2048;
    __shared__ int s_own[kBins];     // this CTA's counts of one digit
    __shared__ int s_sum[3][kBins];  // the cluster's, one array per digit
    __shared__ int s_pick[3];        // chosen bin, entries in larger bins, entries in it
    __shared__ int s_scan[2][32];
    __shared__ int s_base[2][IPT * 32];
    __shared__ int s_total[2];       // this CTA's ties and kept blocks
    pdl_wait();
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int split = blockIdx.x % nsplit, b = blockIdx.x / nsplit;
    const int32_t* trow = table + (size_t)b * nb_max;
    const float* wrow = weight + (size_t)b * nb_max;
    const int jt = split * IPT * nt + tid;  // this thread's first block
    for (int e = tid; e < kBins; e += nt) s_own[e] = 0;
    if (nsplit > 1) {
        for (int e = tid; e < 3 * kBins; e += nt) s_sum[0][e] = 0;
        cluster_arrive();  // waited for before the first remote addition
    }
    int page[IPT];
    float w[IPT];
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = jt + i * nt;
        w[i] = j < nb_max ? wrow[j] : 0.f;
        page[i] = j < nb_max ? trow[j] : 0;
    }
    const int ctx = ctx_len[b];
    const long long want = ctx > 0 ? ((long long)ctx + bs - 1) / bs : 0;
    // a context longer than its table row is left as it is
    const bool bad = want > nb_max;
    if (bad && split == 0 && tid == 0) raise_status(kStatusBadBlockId);
    const int n = (int)(bad ? 0 : want);
    const bool trim = n > budget;
    auto cluster_sync = [&]() {
        if (nsplit > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    };
    // Exclusive prefix, in block order, of flags given as a bit per item:
    // s_base[which][i * nw + warp] is the count before row i of this warp in
    // this CTA; returns the count in lower CTAs, all gets the cluster's total.
    auto prefix = [&](uint32_t flags, int which, int& all) -> int {
        int* at = s_base[which];
#pragma unroll
        for (int i = 0; i < IPT; ++i) {
            const uint32_t v = __ballot_sync(0xffffffffu, (flags >> i) & 1u);
            if (lane == 0) at[i * nw + warp] = __popc(v);
        }
        __syncthreads();
        const int mine = cta_exclusive_sum(tid < IPT * nw ? at[tid] : 0, s_scan[which], all);
        if (tid < IPT * nw) at[tid] = mine;
        if (tid == 0) s_total[which] = all;
        cluster_sync();
        if (nsplit == 1) return 0;
        const int x = lane < nsplit ? *cg::this_cluster().map_shared_rank(&s_total[which], lane) : 0;
        all = __reduce_add_sync(0xffffffffu, x);
        return __reduce_add_sync(0xffffffffu, lane < split ? x : 0);
    };
    // candidates: the middle blocks of a sequence that is trimmed
    uint32_t cand = 0u, keep = 0u;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = jt + i * nt;
        if (j < n) {
            if (!trim || j < sink || j >= n - recent)
                keep |= 1u << i;
            else
                cand |= 1u << i;
        }
    }
    if (nsplit > 1) cluster_wait();
    const int m = budget - sink - recent;  // candidates to keep, fewer than there are
    if (trim && m > 0) {                   // the same for every thread of the cluster
        uint32_t key[IPT];
#pragma unroll
        for (int i = 0; i < IPT; ++i) key[i] = weight_key(w[i]);
        uint32_t t = 0u, known = 0u;  // digits found so far, and their bits
        int need = m;                 // entries still to take among those that match t
        bool whole = false;           // all that match t are taken
        __syncthreads();
#pragma unroll 1
        for (int pass = 0; pass < 3 && !whole; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
#pragma unroll
            for (int i = 0; i < IPT; ++i) {
                const bool on = ((cand >> i) & 1u) && (key[i] & known) == t;
                const uint32_t act = __ballot_sync(0xffffffffu, on);
                if (act != 0u) {
                    const uint32_t d = (key[i] >> shift) & digits;
                    const int first = __ffs(act) - 1;
                    const uint32_t d0 = __shfl_sync(0xffffffffu, d, first);
                    const uint32_t same = __ballot_sync(0xffffffffu, on && d == d0);
                    if (lane == first)
                        atomicAdd(&s_own[d0], __popc(same));
                    else if (on && d != d0)
                        atomicAdd(&s_own[d], 1);
                }
            }
            __syncthreads();
            // bins from the largest down: thread t has kBins - 1 - t * per and below
            const int per = (kBins + nt - 1) / nt;
            const int* hist = s_own;
            if (nsplit > 1) {
                for (int e = tid; e < kBins; e += nt) {
                    const int x = s_own[e];
                    if (x != 0) {
                        s_own[e] = 0;  // for the next digit
                        for (int c = 0; c < nsplit; ++c)
                            atomicAdd(cg::this_cluster().map_shared_rank(&s_sum[pass][e], c), x);
                    }
                }
                cg::this_cluster().sync();
                hist = s_sum[pass];
            }
            int sum = 0;
            for (int e = 0; e < per; ++e) {
                const int r = tid * per + e;
                sum += r < kBins ? hist[kBins - 1 - r] : 0;
            }
            int all;
            int before = cta_exclusive_sum(sum, s_scan[pass & 1], all);
            if (before < need && before + sum >= need) {  // one thread
                for (int e = 0; e < per; ++e) {
                    const int bin = kBins - 1 - (tid * per + e);
                    const int x = hist[bin];
                    if (before + x >= need) {
                        s_pick[0] = bin;
                        s_pick[1] = before;
                        s_pick[2] = x;
                        break;
                    }
                    before += x;
                }
            }
            __syncthreads();
            t |= (uint32_t)s_pick[0] << shift;
            known |= digits << shift;
            need -= s_pick[1];
            whole = s_pick[2] == need;
            if (nsplit == 1 && pass < 2 && !whole) {
                for (int e = tid; e < kBins; e += nt) s_own[e] = 0;
                __syncthreads();
            }
        }
        uint32_t ties = 0u;
#pragma unroll
        for (int i = 0; i < IPT; ++i)
            if ((cand >> i) & 1u) {
                if ((key[i] & known) > t || (whole && (key[i] & known) == t))
                    keep |= 1u << i;
                else if (key[i] == t)
                    ties |= 1u << i;
            }
        if (!whole) {  // the lowest `need` of the tied blocks
            int all;
            const int lower = prefix(ties, 0, all);
#pragma unroll
            for (int i = 0; i < IPT; ++i) {
                const uint32_t v = __ballot_sync(0xffffffffu, (ties >> i) & 1u);
                if (((ties >> i) & 1u) && lower + s_base[0][i * nw + warp] + __popc(v & below) < need)
                    keep |= 1u << i;
            }
        }
    }
    int n_keep;
    const int lower = prefix(keep, 1, n_keep);  // its barrier stands between the reads and the writes
    int32_t* tout = table_out + (size_t)b * nb_max;
    float* wout = weight_out + (size_t)b * nb_max;
    int32_t* kept = kept_ids ? kept_ids + (size_t)b * budget : nullptr;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
        const int j = jt + i * nt;
        const bool k = (keep >> i) & 1u;
        const uint32_t v = __ballot_sync(0xffffffffu, k);
        const int pos = lower + s_base[1][i * nw + warp] + __popc(v & below);  // kept blocks before j
        if (j < nb_max) {
            const int to = j >= n ? j : k ? pos : n_keep + (j - pos);
            tout[to] = page[i];
            wout[to] = k || bad ? w[i] : 0.f;
            if (k && kept && pos < budget) kept[pos] = j;
        }
    }
    if (kept)
        for (int i = n_keep + split * nt + tid; i < budget; i += nsplit * nt) kept[i] = -1;
    if (split == 0 && tid == 0) {
        const int gone = n - n_keep;
        ctx_out[b] = ctx - gone * bs;
        if (freed) freed[b] = gone;
    }
    if (nsplit > 1) cg::this_cluster().sync();  // no CTA leaves while its counts are read
}

}  // namespace lci
