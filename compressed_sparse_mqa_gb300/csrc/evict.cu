// evict.cu -- a session's cache cut to its budget: the tokens to keep, and their moves.
//
// Keep, of the len tokens, `budget`: those that are always kept (the first positions and the newest),
// then those with the largest sums, equal ones by the lower slot.  The order of slots means nothing to
// attention over the whole cache, so nothing is shifted: the j-th dropped slot below `budget` takes the
// j-th kept token from budget and up.  Sources and destinations do not overlap, so the moves are
// independent, and a token that is in its place is not read: a session 256 tokens over a budget of
// 8192 moves some 250 tokens, where closing the gaps in order would move nearly all.
//
// Selection: one cluster of up to eight CTAs per session, each with a consecutive slice of the slots,
// whose keys (an order-preserving 32-bit number per token) stay in shared memory.  Three rounds of a
// radix search from the top (11, 11, 10 bits): each CTA counts its keys by digit, every CTA adds up
// all histograms over distributed shared memory and finds the digit that holds the budget's edge.  The
// last histograms also tell each CTA how many tokens equal to the edge come before its slice.  Then
// kept bits by ballots, ranks by prefix counts over warps and CTAs, and two lists (dropped slots, kept
// tokens) that the second kernel, over the whole GPU, carries out.
#include <cooperative_groups.h>

#include "paged_dev.cuh"

namespace ds4a {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCached = 40960;          // keys that a CTA keeps in shared memory; longer slices are read again each round
constexpr int kMaxSlice = 1 << 20;         // slots of a CTA (their kept bits are 128 KB)
constexpr int kMaxSmem = 200 * 1024;
static_assert(kMaxCached * 4 + kMaxCached / 8 <= kMaxSmem && kMaxSlice / 8 <= kMaxSmem, "shared memory");
static_assert(8LL * kMaxSlice >= kMaxEvictSlots, "eight CTAs hold the longest row");

struct Shared {
    uint32_t hist[3][kBins];
    uint32_t warp_n[kWarps];               // per warp, scanned
    uint32_t warp_m[kWarps];
    uint32_t holes, movers;                // of this CTA, for the others
    uint32_t digit, above, bad;
};

// Order-preserving key: NaN lowest, tokens that are always kept highest; -0 as 0.
DS4A_DEVINL uint32_t token_key(float acc, int pos, int sink, long long newest) {
    if (pos < sink || pos >= newest) return 0xffffffffu;
    return acc != acc ? 0u : float_key(acc + 0.f);
}

// Exclusive prefix sum over the warps' values in v[kWarps]; returns the total.  Every thread calls it.
DS4A_DEVINL uint32_t scan_warps(uint32_t *v) {
    __syncthreads();
    uint32_t x = 0, total = 0;
    if (threadIdx.x < 32) {
        const uint32_t own = threadIdx.x < kWarps ? v[threadIdx.x] : 0;
        x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, x, o);
            if (static_cast<int>(threadIdx.x) >= o) x += up;
        }
        x -= own;
    }
    total = 0;
    for (int w = 0; w < kWarps; ++w) total += v[w];
    __syncthreads();
    if (threadIdx.x < kWarps) v[threadIdx.x] = x;
    __syncthreads();
    return total;
}

// One cluster per session.  kCached: the slice's keys fit shared memory.
template <bool kCached>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t s_keys[];           // keys (kCached), then kept bits, one word per 32 slots
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int s = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const long long len64 = a.kv.len[s], row = static_cast<long long>(s) * a.slots;
    const float *acc = a.acc + row;
    const int32_t *pos = a.pos + row;
    float *acc_out = a.acc_out + row;
    int32_t *pos_out = a.pos_out + row;
    int *count = static_cast<int *>(a.ws) + s;
    int32_t *hole_list = static_cast<int32_t *>(a.ws) + a.list0 + static_cast<long long>(s) * 2 * a.most;
    int32_t *mover_list = hole_list + a.most;
    const bool apart = a.acc_out != a.acc;
    bool bad = false;
    if (len64 < 0) {
        bad = true;
        if (tid == 0 && rank == 0) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
    } else if (len64 > a.slots || len64 > static_cast<long long>(a.kv.max_pages) * a.kv.page) {
        bad = true;
        if (tid == 0 && rank == 0) record_error(a.err, DS4A_ERR_CAPACITY);
    }
    if (bad) {                                                   // the same in every CTA of the cluster
        if (tid == 0 && rank == 0) *count = 0;
        return;
    }
    const int len = static_cast<int>(len64);
    if (len <= a.budget) {                                       // nothing to drop
        if (apart)
            for (int t = rank * kThreads + tid; t < len; t += C * kThreads) {
                acc_out[t] = acc[t];
                pos_out[t] = pos[t];
            }
        if (C > 1) cluster.sync();                               // every CTA has read len
        if (tid == 0 && rank == 0) {
            *count = 0;
            a.len_out[s] = len;
        }
        return;
    }
    const long long newest = a.next[s] - a.n_recent;
    // slices: a whole number of 32-slot words per warp
    const int per_warp = (len + C * kThreads - 1) / (C * kThreads) * 32, slice = per_warp * kWarps;
    const int base = rank * slice + warp * per_warp;             // the warp's first slot (below 2^31 + 2^17: kept in range below)
    const int words = base < len ? (min(per_warp, len - base) + 31) / 32 : 0;
    uint32_t *s_kept = s_keys + (kCached ? a.slice_cap : 0);
    for (int x = tid; x < 3 * kBins; x += kThreads) (&sh.hist[0][0])[x] = 0;
    if (tid == 0) sh.bad = 0;
    __syncthreads();
    // pages of the session's tokens
    {
        const int pages = (len - 1) / a.kv.page + 1;
        const int32_t *table = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
        for (int p = rank * kThreads + tid; p < pages; p += C * kThreads) {
            const int id = __ldg(table + p);
            if (id < 0 || id >= a.kv.n_pages) sh.bad = 1;
        }
    }
    auto key_at = [&](int w) {                                   // key of the warp's word w, this lane
        if (kCached) return s_keys[warp * per_warp + w * 32 + lane];
        const int t = base + w * 32 + lane;
        return t < len ? token_key(acc[t], pos[t], a.n_sink, newest) : 0u;
    };
    // round 1 reads the tokens
#pragma unroll 4
    for (int w = 0; w < words; ++w) {
        const int t = base + w * 32 + lane;
        const bool in = t < len;
        const uint32_t key = in ? token_key(acc[t], pos[t], a.n_sink, newest) : 0u;
        if (kCached) s_keys[warp * per_warp + w * 32 + lane] = key;
        if (in) atomicAdd(&sh.hist[0][key >> 21], 1u);
    }
    uint32_t want = a.budget, prefix = 0;                        // tokens still to find at or below the prefix
#pragma unroll 1
    for (int r = 0; r < 3; ++r) {
        if (r > 0) {
            const int up = r == 1 ? 21 : 10;
#pragma unroll 4
            for (int w = 0; w < words; ++w) {
                const uint32_t key = key_at(w);
                const bool in = base + w * 32 + lane < len;
                if (in && (key >> up) == (prefix >> up)) atomicAdd(&sh.hist[r][r == 1 ? (key >> 10) & 2047u : key & 1023u], 1u);
            }
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        // bins from the top: thread i adds up bins 2047-4i .. 2044-4i of all CTAs
        uint32_t h[4], sum = 0;
        {
            const int b0 = kBins - 4 - 4 * tid;
            uint4 v = make_uint4(0, 0, 0, 0);
            for (int x = 0; x < C; ++x) {
                const uint4 o = *reinterpret_cast<const uint4 *>(C > 1 ? cluster.map_shared_rank(&sh.hist[r][b0], x) : &sh.hist[r][b0]);
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            h[0] = v.w;
            h[1] = v.z;
            h[2] = v.y;
            h[3] = v.x;
            sum = h[0] + h[1] + h[2] + h[3];
        }
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) sh.warp_n[warp] = incl;
        scan_warps(sh.warp_n);
        uint32_t above = sh.warp_n[warp] + incl - sum;
        if (above < want && above + sum >= want) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (above < want && above + h[i] >= want) {
                    sh.digit = kBins - 1 - 4 * tid - i;
                    sh.above = above;
                }
                above += h[i];
            }
        }
        __syncthreads();
        want -= sh.above;
        prefix |= sh.digit << (r == 0 ? 21 : (r == 1 ? 10 : 0));
        if (r == 0) {
            bool any = false;
            for (int x = 0; x < C; ++x) any |= *(C > 1 ? cluster.map_shared_rank(&sh.bad, x) : &sh.bad) != 0;
            bad = any;
        }
        __syncthreads();                                         // sh.digit and sh.warp_n are written again
    }
    // bad pages: the session is left alone (every CTA saw the same flags; they are not written again)
    if (bad) {
        if (C > 1) cluster.sync();
        if (tid == 0 && rank == 0) {
            record_error(a.err, DS4A_ERR_DEVICE_INDEX);
            *count = 0;
        }
        return;
    }
    // `prefix` is the edge; of the tokens equal to it the first `want` stay.  Equal ones before this slice:
    uint32_t before = 0;
    for (int x = 0; x < rank; ++x) before += *cluster.map_shared_rank(&sh.hist[2][prefix & 1023u], x);
    uint32_t ties = 0;
    for (int w = 0; w < words; ++w) {
        const bool in = base + w * 32 + lane < len;
        ties += __popc(__ballot_sync(0xffffffffu, in && key_at(w) == prefix));
    }
    if (lane == 0) sh.warp_n[warp] = ties;
    scan_warps(sh.warp_n);
    uint32_t tie = before + sh.warp_n[warp];
    __syncthreads();                                             // sh.warp_n is written again
    uint32_t holes = 0, movers = 0;
    for (int w = 0; w < words; ++w) {
        const int t = base + w * 32 + lane;
        const bool in = t < len;
        const uint32_t key = key_at(w);
        const uint32_t eq = __ballot_sync(0xffffffffu, in && key == prefix);
        const bool keep = in && (key > prefix || (key == prefix && tie + __popc(eq & ((1u << lane) - 1u)) < want));
        tie += __popc(eq);
        const uint32_t kept = __ballot_sync(0xffffffffu, keep);
        const uint32_t low = __ballot_sync(0xffffffffu, t < a.budget);
        holes += __popc(low & ~kept);                            // (budget < len: a slot below it holds a token)
        movers += __popc(kept & ~low);
        if (lane == 0) s_kept[(warp * per_warp >> 5) + w] = kept;
        if (apart && keep && t < a.budget) {
            acc_out[t] = acc[t];
            pos_out[t] = pos[t];
        }
    }
    if (lane == 0) {
        sh.warp_n[warp] = holes;
        sh.warp_m[warp] = movers;
    }
    const uint32_t all_holes = scan_warps(sh.warp_n), all_movers = scan_warps(sh.warp_m);
    if (tid == 0) {
        sh.holes = all_holes;
        sh.movers = all_movers;
    }
    uint32_t at_h = 0, at_m = 0;
    if (C > 1) {
        cluster.sync();
        for (int x = 0; x < rank; ++x) {
            at_h += *cluster.map_shared_rank(&sh.holes, x);
            at_m += *cluster.map_shared_rank(&sh.movers, x);
        }
    }
    if (tid == 0 && rank == C - 1) {                             // (len is read by every CTA before the first cluster.sync)
        *count = static_cast<int>(at_h + all_holes);
        a.len_out[s] = a.budget;
    }
    at_h += sh.warp_n[warp];
    at_m += sh.warp_m[warp];
    __syncwarp();
    for (int w = 0; w < words; ++w) {
        const uint32_t kept = s_kept[(warp * per_warp >> 5) + w];
        const int t0 = base + w * 32;
        const uint32_t low = t0 + 32 <= a.budget ? 0xffffffffu : (t0 >= a.budget ? 0u : (1u << (a.budget - t0)) - 1u);
        const uint32_t hole = low & ~kept, mover = kept & ~low, below = (1u << lane) - 1u;
        if ((hole >> lane) & 1u) hole_list[at_h + __popc(hole & below)] = t0 + lane;
        if ((mover >> lane) & 1u) mover_list[at_m + __popc(mover & below)] = t0 + lane;
        at_h += __popc(hole);
        at_m += __popc(mover);
    }
    if (C > 1) cluster.sync();                                   // the others have read this CTA's shared memory
}

// A warp moves eight tokens at a time, their K and V rows in 16-byte pieces, all loads in flight.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
    constexpr int kPer = 8, kLanes = D / 8;                      // 16-byte pieces of a row
    const int s = blockIdx.y, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int n = static_cast<const int *>(a.ws)[s];
    const int32_t *hole_list = static_cast<const int32_t *>(a.ws) + a.list0 + static_cast<long long>(s) * 2 * a.most;
    const int32_t *mover_list = hole_list + a.most;
    const int32_t *table = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
    const long long row = static_cast<long long>(s) * a.slots;
    const int warps = gridDim.x * (blockDim.x >> 5), w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    for (long long j0 = static_cast<long long>(w) * kPer; j0 < n; j0 += static_cast<long long>(warps) * kPer) {
        long long to = -1, from = -1;
        if (lane < kPer && j0 + lane < n) {
            const int t = hole_list[j0 + lane], f = mover_list[j0 + lane];
            to = pool_row(a.kv, table, t, a.err);                // the pages were checked
            from = pool_row(a.kv, table, f, a.err);
            a.acc_out[row + t] = a.acc[row + f];
            a.pos_out[row + t] = a.pos[row + f];
        }
        constexpr int kAtOnce = 32 / (2 * kLanes);               // tokens a warp covers with one load each lane
        const int tok = lane / (2 * kLanes), part = lane % (2 * kLanes), piece = part % kLanes;
        uint16_t *pool = part < kLanes ? a.kv.k : a.kv.v;
        uint4 x[kPer / kAtOnce];
#pragma unroll
        for (int i = 0; i < kPer / kAtOnce; ++i) {
            const long long f = __shfl_sync(0xffffffffu, from, i * kAtOnce + tok);
            if (f >= 0) x[i] = *reinterpret_cast<const uint4 *>(pool + f * D + piece * 8);
        }
#pragma unroll
        for (int i = 0; i < kPer / kAtOnce; ++i) {
            const long long t = __shfl_sync(0xffffffffu, to, i * kAtOnce + tok);
            if (t >= 0) *reinterpret_cast<uint4 *>(pool + t * D + piece * 8) = x[i];
        }
    }
}

long long most_moves(int slots, int budget) {
    const int over = slots > budget ? slots - budget : 0;
    return over < budget ? over : budget;
}
long long header_ints(int B) { return (static_cast<long long>(B) + 63) / 64 * 64; }

template <bool kCached>
cudaError_t launch_select(const EvictArgs &a, int B, int C, size_t smem, const Ctx &c) {
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<kCached>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch(evict_select_kernel<kCached>, dim3(static_cast<unsigned>(B) * C), dim3(kThreads), smem, c, C, a);
}

}  // namespace

size_t evict_ws_bytes(int B, int slots, int budget) {
    return static_cast<size_t>(header_ints(B) + 2LL * B * most_moves(slots, budget)) * 4;
}

cudaError_t launch_evict(const EvictArgs &args, int B, const Ctx &c) {
    EvictArgs a = args;
    a.most = most_moves(a.slots, a.budget);
    a.list0 = header_ints(B);
    // CTAs a session: one for every 4096 slots, up to eight, and no more in all than the GPU holds at once
    int C = 1;
    while (C < 8 && ((static_cast<long long>(C) * 4096 < a.slots && 2LL * C * B <= 4LL * c.num_sms) ||
                     static_cast<long long>(C) * kMaxSlice < a.slots))
        C *= 2;
    const long long cap = (static_cast<long long>(a.slots) + C * kThreads - 1) / (C * kThreads) * kThreads;   // slots of a slice
    const bool cached = cap <= kMaxCached;
    a.slice_cap = cached ? static_cast<int>(cap) : 0;
    const long long bits = (cap + 31) / 32;
    const size_t smem = static_cast<size_t>((cached ? cap : 0) + bits) * 4;
    cudaError_t e = cached ? launch_select<true>(a, B, C, smem, c) : launch_select<false>(a, B, C, smem, c);
    if (e != cudaSuccess || a.most == 0) return e;
    long long x = (a.most + 63) / 64;                            // 8 warps of 8 tokens a CTA
    const long long limit = (4LL * c.num_sms + B - 1) / B;
    if (x > limit) x = limit;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(B));
    return a.kv.D == 128 ? launch(evict_move_kernel<128>, grid, dim3(256), 0, c, 1, a)
                         : launch(evict_move_kernel<64>, grid, dim3(256), 0, c, 1, a);
}

}  // namespace ds4a
