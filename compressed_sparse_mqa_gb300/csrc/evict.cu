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
// whose keys (an order-preserving 32-bit number per token) stay in shared memory.  Four rounds of a
// radix search from the top, 8 bits each: each CTA counts its keys by digit, every CTA adds up all
// histograms over distributed shared memory and finds the digit that holds the budget's edge (three
// rounds of 2048 bins spent 2000 - 2900 cycles each on the remote histograms, these 1000).  The last
// histograms also tell each CTA how many tokens equal to the edge come before its slice.  Then
// kept bits by ballots, ranks by prefix counts over warps and CTAs, and the moves: dealt out over the cluster's
// warps through distributed shared memory, or, where there may be many, as two lists that a second kernel over
// the whole GPU carries out.
//
// Measured: evict_1x4096 11.5 us and evict_64x8192 16.8, latency (some 20000 cycles of dependent steps: two loads, four
// rounds of count, cluster barrier and search, two counts of kept tokens, the moves); evict_24x4000, which
// moves 33 MB of tokens, 27 us, about half of it the moves.
#include <cooperative_groups.h>

#include "paged_dev.cuh"

namespace ds4a {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSelectBlocks = 1;           // an SM: two would leave 64 registers a thread (evict_24x4000 29.4 against 26.5 us)
constexpr int kBins = 256, kRounds = 4;
constexpr int kOwnMoves = 512;            // moves a CTA of the cluster that it carries out itself
constexpr int kPer = 8;                    // tokens that a warp moves at a time
constexpr int kMaxCached = 40960;          // keys that a CTA keeps in shared memory; longer slices are read again each round
constexpr int kSlotsPerCta = 2048;         // a session gets another CTA for every so many slots
constexpr int kMaxSlice = 1 << 20;         // slots of a CTA (their kept bits are 128 KB)
constexpr int kMaxSmem = 200 * 1024;
constexpr int kMaxCluster = 8;
static_assert(kOwnMoves % (kWarps * kPer) == 0, "every warp of a cluster has its share of the lists");
static_assert(kMaxCached * 4 + kMaxCached / 8 <= kMaxSmem && kMaxSlice / 8 <= kMaxSmem, "shared memory");
static_assert(static_cast<long long>(kMaxCluster) * kMaxSlice >= kMaxEvictSlots, "eight CTAs hold the longest row");

struct alignas(16) Shared {
    uint32_t hist[kRounds][kBins];
    uint32_t warp_ties[kWarps], warp_holes[kWarps], warp_movers[kWarps];   // per warp
    uint32_t holes, movers;                // of this CTA, for the others
    uint32_t warp_bins[kRounds][8];
    uint32_t digit[kRounds], above[kRounds], count[kRounds], bad, any_bad;
    int32_t list[2][kOwnMoves];            // kMoves: the moves that fall to this CTA, dropped slots and kept tokens
};

// Order-preserving key: NaN lowest, tokens that are always kept highest; -0 as 0.
DS4A_DEVINL uint32_t token_key(float acc, int pos, int sink, long long newest) {
    if (pos < sink || pos >= newest) return 0xffffffffu;
    return acc != acc ? 0u : float_key(acc + 0.f);
}

// The sum over the warps before this one, and over all, of v[kWarps] (written before the last __syncthreads).
DS4A_DEVINL uint2 scan_warps(const uint32_t *v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = lane < kWarps ? v[lane] : 0;
    const uint32_t own = x;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += up;
    }
    return make_uint2(__shfl_sync(0xffffffffu, x - own, warp), __shfl_sync(0xffffffffu, x, kWarps - 1));
}

// Bin `b` summed over the cluster's CTAs (all loads in flight: one behind the other they took 700 cycles each), and
// whether any of them met a bad page.
template <int kC>
DS4A_DEVINL uint32_t add_bins(cg::cluster_group &cluster, Shared &sh, int r, int b, bool &any) {
    uint32_t h[kC], bad[kC], sum = 0;
#pragma unroll
    for (int x = 0; x < kC; ++x) {
        const Shared *p = kC > 1 ? cluster.map_shared_rank(&sh, x) : &sh;
        h[x] = p->hist[r][b];
        bad[x] = p->bad;
    }
#pragma unroll
    for (int x = 0; x < kC; ++x) {
        sum += h[x];
        any |= bad[x] != 0;
    }
    return sum;
}

// Carries out moves 0 .. n-1 of a session, pair(j) = (dropped slot, kept token), eight at a time and warp: their K and V rows
// in 16-byte pieces, all loads in flight, their sums and positions.  A source is never a destination.
template <int D, typename F>
DS4A_DEVINL void move_tokens(const EvictArgs &a, int s, int n, int w, int warps, F pair) {
    constexpr int kLanes = D / 8;                                // 16-byte pieces of a row
    constexpr int kAtOnce = 32 / (2 * kLanes);                   // tokens a warp covers with one load each lane
    const int lane = threadIdx.x & 31;
    const int32_t *table = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
    const long long row = static_cast<long long>(s) * a.slots;
    const int tok = lane / (2 * kLanes), part = lane % (2 * kLanes), piece = part % kLanes;
    uint16_t *pool = part < kLanes ? a.kv.k : a.kv.v;
    for (int j0 = w * kPer; j0 < n; j0 += warps * kPer) {        // below 2^23 + 2^21
        long long to = -1, from = -1;
        if (lane < kPer && j0 + lane < n) {
            const int2 m = pair(j0 + lane);
            const int t = m.x, f = m.y;
            to = pool_row(a.kv, table, t, a.err);                // the pages were checked
            from = pool_row(a.kv, table, f, a.err);
            a.acc_out[row + t] = a.acc[row + f];
            a.pos_out[row + t] = a.pos[row + f];
        }
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

// One cluster per session.  kCached: the slice's keys fit shared memory; kMoves: the cluster carries out the moves too.
template <bool kCached, bool kMoves>
__global__ void __launch_bounds__(kThreads, kSelectBlocks) evict_select_kernel(const EvictArgs a) {
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
    const int pages = len > 0 ? (len - 1) / a.kv.page + 1 : 0;   // of the session's tokens
    const int32_t *table = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
    auto bad_pages = [&](int p) {                                // whether one of this thread's from p on is bad
        bool off = false;
        for (; p < pages; p += C * kThreads) {
            const int id = __ldg(table + p);
            off |= id < 0 || id >= a.kv.n_pages;
        }
        return off;
    };
    if (len <= a.budget) {                                       // nothing to drop
        bad = __syncthreads_or(bad_pages(rank * kThreads + tid));
        if (C > 1) {
            if (tid == 0) sh.bad = bad;
            cluster.sync();
            for (int x = 0; x < C; ++x) bad |= *cluster.map_shared_rank(&sh.bad, x) != 0;
        }
        if (apart && !bad)
            for (int t = rank * kThreads + tid; t < len; t += C * kThreads) {
                acc_out[t] = acc[t];
                pos_out[t] = pos[t];
            }
        if (C > 1) cluster.sync();                               // every CTA has read len and the others' flags
        if (tid == 0 && rank == 0) {
            *count = 0;
            if (bad) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
            else a.len_out[s] = len;
        }
        return;
    }
    // (below -2^62 every position is one of the newest; the difference fits)
    const long long newest = max(a.next[s], -(1LL << 62)) - a.n_recent;
    // slices: a whole number of 32-slot words per warp
    const int per_warp = (len + C * kThreads - 1) / (C * kThreads) * 32, slice = per_warp * kWarps;
    const int base = rank * slice + warp * per_warp;             // the warp's first slot (below 2^31 + 2^17: kept in range below)
    const int words = base < len ? (min(per_warp, len - base) + 31) / 32 : 0;
    uint32_t *s_kept = s_keys + (kCached ? a.slice_cap : 0);
    for (int x = tid; x < kRounds * kBins; x += kThreads) (&sh.hist[0][0])[x] = 0;
    if (tid == 0) sh.bad = 0;
    __syncthreads();
    // (the first pages' ids are looked at when the tokens have been counted)
    const int page0 = rank * kThreads + tid, id0 = page0 < pages ? __ldg(table + page0) : 0;
    auto key_at = [&](int w) {                                   // key of the warp's word w, this lane
        if (kCached) return s_keys[warp * per_warp + w * 32 + lane];
        const int t = base + w * 32 + lane;
        return t < len ? token_key(acc[t], pos[t], a.n_sink, newest) : 0u;
    };
    // kAhead words at a time: their loads go out before anything is done with one (evict_64x8192 with 8 17.5 us, 6 16.7,
    // 3 16.7, 1 18.3: what is unrolled past a warp's words is issued all the same)
    constexpr int kAhead = 3;
    auto keys_at = [&](int w0, uint32_t (&k)[kAhead]) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) k[i] = w0 + i < words ? key_at(w0 + i) : 0u;
    };
    // the first round reads the tokens
    for (int w0 = 0; w0 < words; w0 += kAhead) {
        float va[kAhead];
        int vp[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = base + (w0 + i) * 32 + lane;
            const bool in = w0 + i < words && t < len;
            va[i] = in ? acc[t] : 0.f;
            vp[i] = in ? pos[t] : 0;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (w0 + i >= words) break;
            const bool in = base + (w0 + i) * 32 + lane < len;
            const uint32_t key = in ? token_key(va[i], vp[i], a.n_sink, newest) : 0u;
            if (kCached) s_keys[warp * per_warp + (w0 + i) * 32 + lane] = key;
            if (in) atomicAdd(&sh.hist[0][key >> 24], 1u);
        }
    }
    {
        const bool off = id0 < 0 || id0 >= a.kv.n_pages || bad_pages(page0 + C * kThreads);
        if (off) sh.bad = 1;
    }
    uint32_t want = a.budget, prefix = 0;                        // tokens still to find at or below the prefix
#pragma unroll 1
    for (int r = 0; r < kRounds; ++r) {
        const int down = 24 - 8 * r;
        if (r > 0) {
            for (int w0 = 0; w0 < words; w0 += kAhead) {
                uint32_t k[kAhead];
                keys_at(w0, k);
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (w0 + i < words && base + (w0 + i) * 32 + lane < len && ((k[i] ^ prefix) >> (down + 8)) == 0)
                        atomicAdd(&sh.hist[r][(k[i] >> down) & 255u], 1u);
            }
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        // bins from the top, one a thread of the first eight warps
        uint32_t h = 0, above = 0;
        if (warp < 8) {
            const int b = kBins - 1 - tid;
            bool any = false;
            switch (C) {
                case 1: h = add_bins<1>(cluster, sh, r, b, any); break;
                case 2: h = add_bins<2>(cluster, sh, r, b, any); break;
                case 4: h = add_bins<4>(cluster, sh, r, b, any); break;
                default: h = add_bins<kMaxCluster>(cluster, sh, r, b, any); break;
            }
            above = h;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t up = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += up;
            }
            if (lane == 31) sh.warp_bins[r][warp] = above;
            above -= h;
            if (r == 0 && tid == 0) sh.any_bad = any;            // the same in every thread
        }
        __syncthreads();
        if (warp < 8) {
#pragma unroll
            for (int x = 0; x < 7; ++x)
                if (x < warp) above += sh.warp_bins[r][x];
            if (above < want && above + h >= want) {             // one thread
                sh.digit[r] = kBins - 1 - tid;
                sh.above[r] = above;
                sh.count[r] = h;
            }
        }
        __syncthreads();
        want -= sh.above[r];
        prefix |= sh.digit[r] << down;
        if (r == 0) {
            bad = sh.any_bad != 0;
            if (bad) break;
            // arrays apart: what stays in its place (dropped slots are written over by the moves)
            if (apart) {
                for (int w0 = 0; w0 < words; w0 += kAhead) {
                    float va[kAhead];
                    int vp[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const int t = base + (w0 + i) * 32 + lane;
                        if (w0 + i < words && t < a.budget) {
                            va[i] = acc[t];
                            vp[i] = pos[t];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const int t = base + (w0 + i) * 32 + lane;
                        if (w0 + i < words && t < a.budget) {
                            acc_out[t] = va[i];
                            pos_out[t] = vp[i];
                        }
                    }
                }
            }
        }
        // All tokens of the digit stay (in the third round it mostly holds one): the edge is just below them, and none
        // that equals it stays.
        if (sh.count[r] == want && prefix != 0) {
            prefix -= 1;
            want = 0;
            break;
        }
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
    // `prefix` is the edge; of the tokens equal to it the first `want` stay.  Equal ones before this warp's:
    uint32_t tie = 0;
    if (want > 0) {
        uint32_t before = 0;
#pragma unroll
        for (int x = 0; x < kMaxCluster - 1; ++x)
            if (x < rank) before += *cluster.map_shared_rank(&sh.hist[kRounds - 1][prefix & 255u], x);
        uint32_t ties = 0;
        for (int w0 = 0; w0 < words; w0 += kAhead) {
            uint32_t k[kAhead];
            keys_at(w0, k);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                ties += __popc(__ballot_sync(0xffffffffu, w0 + i < words && base + (w0 + i) * 32 + lane < len && k[i] == prefix));
        }
        if (lane == 0) sh.warp_ties[warp] = ties;
        __syncthreads();
        tie = before + scan_warps(sh.warp_ties).x;
    }
    auto low_bits = [&](int t0) {                                // slots of the word at t0 that are below the budget
        return t0 + 32 <= a.budget ? 0xffffffffu : (t0 >= a.budget ? 0u : (1u << (a.budget - t0)) - 1u);
    };
    uint32_t holes = 0, movers = 0;
    for (int w0 = 0; w0 < words; w0 += kAhead) {
        uint32_t k[kAhead];
        keys_at(w0, k);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (w0 + i >= words) break;
            const int t0 = base + (w0 + i) * 32;
            const bool in = t0 + lane < len;
            bool keep = in && k[i] > prefix;
            if (want > 0) {
                const uint32_t eq = __ballot_sync(0xffffffffu, in && k[i] == prefix);
                keep |= in && k[i] == prefix && tie + __popc(eq & ((1u << lane) - 1u)) < want;
                tie += __popc(eq);
            }
            const uint32_t kept = __ballot_sync(0xffffffffu, keep), low = low_bits(t0);
            holes += __popc(low & ~kept);                        // (budget < len: a slot below it holds a token)
            movers += __popc(kept & ~low);
            if (lane == 0) s_kept[(warp * per_warp >> 5) + w0 + i] = kept;
        }
    }
    if (lane == 0) {
        sh.warp_holes[warp] = holes;
        sh.warp_movers[warp] = movers;
    }
    __syncthreads();
    const uint2 h = scan_warps(sh.warp_holes), m = scan_warps(sh.warp_movers);
    uint32_t at_h = h.x, at_m = m.x, moves = h.y;                // moves: of the session
    if (C > 1) {
        if (tid == 0) {
            sh.holes = h.y;
            sh.movers = m.y;
        }
        cluster.sync();
        moves = 0;
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
            if (x >= C) continue;
            const uint32_t xh = *cluster.map_shared_rank(&sh.holes, x), xm = *cluster.map_shared_rank(&sh.movers, x);
            moves += xh;
            if (x < rank) {
                at_h += xh;
                at_m += xm;
            }
        }
    }
    if (tid == 0 && rank == 0) {                                 // (len is read by every CTA before the first cluster.sync)
        *count = static_cast<int>(moves);
        a.len_out[s] = a.budget;
    }
    __syncwarp();
    // Move j: to the lists, or (kMoves) to the CTA whose warp carries it out, groups of kPer dealt out over the cluster's warps.
    auto put = [&](int which, uint32_t j, int t) {
        if (kMoves) {
            const uint32_t group = j / kPer, slot = group % (C * kWarps), at = (group / (C * kWarps) * kWarps + slot % kWarps) * kPer + j % kPer;
            int32_t *dst = &sh.list[which][at];
            *(C > 1 ? cluster.map_shared_rank(dst, slot / kWarps) : dst) = t;
        } else {
            (which ? mover_list : hole_list)[j] = t;
        }
    };
    for (int w = 0; w < words; ++w) {
        const uint32_t kept = s_kept[(warp * per_warp >> 5) + w];
        const int t0 = base + w * 32;
        const uint32_t low = low_bits(t0), hole = low & ~kept, mover = kept & ~low, below = (1u << lane) - 1u;
        if ((hole >> lane) & 1u) put(0, at_h + __popc(hole & below), t0 + lane);
        if ((mover >> lane) & 1u) put(1, at_m + __popc(mover & below), t0 + lane);
        at_h += __popc(hole);
        at_m += __popc(mover);
    }
    // the others have read this CTA's shared memory, and (kMoves) the lists are complete
    if (C > 1) cluster.sync();
    else if (kMoves) __syncthreads();
    if constexpr (kMoves) {
        const int n = static_cast<int>(moves);
        auto pair = [&](int j) {
            const int group = j / kPer, at = (group / (C * kWarps) * kWarps + warp) * kPer + j % kPer;
            return make_int2(sh.list[0][at], sh.list[1][at]);
        };
        if (a.kv.D == 128) move_tokens<128>(a, s, n, rank * kWarps + warp, C * kWarps, pair);
        else move_tokens<64>(a, s, n, rank * kWarps + warp, C * kWarps, pair);
    }
}

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
    const int s = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    const int n = static_cast<const int *>(a.ws)[s];
    const int32_t *hole_list = static_cast<const int32_t *>(a.ws) + a.list0 + static_cast<long long>(s) * 2 * a.most;
    move_tokens<D>(a, s, n, blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8,
                   [&](int j) { return make_int2(hole_list[j], hole_list[a.most + j]); });
}

long long most_moves(int slots, int budget) {
    const int over = slots > budget ? slots - budget : 0;
    return over < budget ? over : budget;
}
long long header_ints(int B) { return (static_cast<long long>(B) + 63) / 64 * 64; }

template <bool kCached, bool kMoves>
cudaError_t launch_select(const EvictArgs &a, int B, int C, size_t smem, const Ctx &c) {
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<kCached, kMoves>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch(evict_select_kernel<kCached, kMoves>, dim3(static_cast<unsigned>(B) * C), dim3(kThreads), smem, c, C, a);
}

}  // namespace

size_t evict_ws_bytes(int B, int slots, int budget) {
    return static_cast<size_t>(header_ints(B) + 2LL * B * most_moves(slots, budget)) * 4;
}

cudaError_t launch_evict(const EvictArgs &args, int B, const Ctx &c) {
    EvictArgs a = args;
    a.most = most_moves(a.slots, a.budget);
    a.list0 = header_ints(B);
    // CTAs a session: one for every kSlotsPerCta slots, up to eight, and no more in all than SMs (256 CTAs for 64
    // sessions, two rounds, took 17.6 us against 17.3 for 128)
    int C = 1;
    while (C < kMaxCluster && ((static_cast<long long>(C) * kSlotsPerCta < a.slots && 2LL * C * B <= c.num_sms) ||
                     static_cast<long long>(C) * kMaxSlice < a.slots))
        C *= 2;
    const long long cap = (static_cast<long long>(a.slots) + C * kThreads - 1) / (C * kThreads) * kThreads;   // slots of a slice
    const bool cached = cap <= kMaxCached;
    a.slice_cap = cached ? static_cast<int>(cap) : 0;
    const long long bits = (cap + 31) / 32;
    const size_t smem = static_cast<size_t>((cached ? cap : 0) + bits) * 4;
    // A cluster moves up to kOwnMoves tokens a CTA itself (evict_1x4096 15.5 us against 16.3 with the second kernel, at
    // the time); more are the whole GPU's (evict_24x4000 in the clusters 50 us a launch, alone, against 28).
    const bool own = a.most <= static_cast<long long>(kOwnMoves) * C;
    cudaError_t e = own ? (cached ? launch_select<true, true>(a, B, C, smem, c) : launch_select<false, true>(a, B, C, smem, c))
                        : (cached ? launch_select<true, false>(a, B, C, smem, c) : launch_select<false, false>(a, B, C, smem, c));
    if (e != cudaSuccess || own) return e;
    long long x = (a.most + 63) / 64;                            // 8 warps of 8 tokens a CTA
    const long long limit = (4LL * c.num_sms + B - 1) / B;
    if (x > limit) x = limit;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(B));
    return a.kv.D == 128 ? launch(evict_move_kernel<128>, grid, dim3(256), 0, c, 1, a)
                         : launch(evict_move_kernel<64>, grid, dim3(256), 0, c, 1, a);
}

}  // namespace ds4a
