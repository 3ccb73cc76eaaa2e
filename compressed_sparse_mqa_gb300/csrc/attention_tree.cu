// attention_tree.cu -- attention of a tree of drafted tokens over a paged cache, on the
// 5th-generation tensor cores.
//
// For node i at position p of session s and head h,
//   o_h = sum_j softmax_j(scale * q_h . K_j) V_j
// over the committed raw tokens t > p - window, the node's ancestors j (itself included)
// with p_j > p - window, and the compressed rows: those listed in its sel row, or every
// row complete at p.  A row j >= len / ratio is the one completed by the ancestor at
// position (j+1) * ratio - 1; it is read from the draft's rows (cap - N + that node).
//
// All heads of all nodes of a session share its keys (multi-query attention), so the
// rows of one product are (node, head) pairs: 128 rows on the M side of tcgen05.mma, 128
// keys on the N side.  Nodes differ only in a few keys (the tree, the window's edge): those
// are masked in the scores.  With sel every node has its own key list and its heads are a
// tile of their own.
//
// Keys.  A session's keys are runs of 16 rows: the raw slots from its window's edge to the
// last drafted node (pages are multiples of 16 rows, so a run is inside one page), the
// committed compressed rows, the draft's rows.  A key tile is 8 runs, one TMA box each per 64
// columns (sel: tile::gather4 loads of 4 rows).  Runs past the end load zeros.
//
// Work item: a row tile (one or two 128-row blocks of a session, or one node's heads) and
// its key tiles.  CTAs are persistent, one per SM, and take items in one of three ways:
//   direct  no more row tiles than SMs: one each, known from the CTA's number;
//   walk    more: the row tiles that have nodes, dealt out evenly;
//   stream  few row tiles over many keys: all (row tile, key tile) pairs in one line, cut into equal
//           pieces, one a CTA.  A row tile that two or more CTAs share is joined by
//           combine_kernel (attn_full_4x64: 58 row tiles of 258 key tiles, 98.5 each).
// Roles:
//   warps 0-3, 4-7  softmax of side 0 / 1: thread = row.  With two row blocks a side is a
//                row block and both use the same key tiles; with one block the sides take
//                alternate key tiles and are joined at the end (both accumulators have
//                the row in the same tensor-memory lane).
//   warp 8       work set-up: counts, ancestor masks, tile range of the next item; its queries.
//   warps 9-10   MMA issuers of side 0 / 1: S = Q K^T into the side's score columns, O += P V
//                with P in 16 bits read from tensor memory, over the scores it came from.  One
//                warp's waits pass behind the other's products.
//   warp 11      checker (below).
//   warps 12-15  TMA producers: K (12, 13) and V (14, 15).
// A tile is scored in two chunks of 64 keys, and each side has two score buffers, so the
// scores of the next chunk are computed while the softmax of this one runs (with one buffer
// of 128 keys per side the two sides fell into step, both in their softmax, then both waiting
// for products: 4200 cycles a 256-row tile, of which the tensor core worked 2050).  The price is
// that a product with N = 64 is bound by reading Q from shared memory, 48 cycles instead of 32.
// The softmax reference of a row is raised (and O rescaled) only when a score is 2^15 above it, to 2^7
// below that score: the largest weight is 2^7 .. 2^15, which fits 16 bits, and half a step of the
// smallest ones is 2^-32 of it (with weights of 2^0 .. 2^8 it was 2^-25: of 2^18 keys of weight 2^-25
// beside one of 1 all were lost or rounded to 2^-24).  Sums are binary32, of the weights before they
// are rounded to 16 bits for the product with V; the accumulator drops what is below about 2^-25 of
// what it holds.
//
// Measured (device time, inputs in L2): 4 sessions of up to 64 nodes x 64 heads over 32768 tokens
// 172 us = 1354 TFLOP/s, bound by the tensor pipe and the shared memory that feeds it; 64 sessions of
// up to 32 nodes over 128 + 512 rows 52 us: 406 six-tile items on 152 SMs are three rounds, the last
// two thirds full, and a third of an item is its output and the next one's start; 16 sessions of up to 16
// nodes with 512 listed rows each 28 us: 192 items are two rounds, the second a quarter full, of which
// the gathers (about 20 B a cycle and SM) take some 16 us and the items' start and output the rest; 4
// nodes over the window 9.9 us, latency.
//
// Masked keys get weight 0, but 0 * V is not 0 where V is infinite or NaN: slots never
// written, or another branch's values.  The checker scans the V rows of runs that some row
// masks: values that are not finite are set to 0, and where the key is valid for some
// rows, noted, so that exactly those rows get them in the end.
#include <type_traits>

#include "paged_dev.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace ds4a {
namespace {

constexpr int kTK = 128;                   // keys per tile, rows per block
constexpr int kRun = 16, kRuns = kTK / kRun;
constexpr int kCK = 64, kChunkRuns = kCK / kRun;   // keys and runs of a chunk: two a tile
constexpr int kNS = 2;                     // K stages, and V stages but with sel: with one row block, one for each side
constexpr int kInfo = 8;                   // tiles whose run information is kept
constexpr int kSideWarps = 4, kSoftWarps = 2 * kSideWarps;
constexpr int kSetupWarp = kSoftWarps, kMmaWarp = kSetupWarp + 1, kChkWarp = kMmaWarp + 2;
constexpr int kProdWarp0 = kChkWarp + 1;
constexpr int kProd = 2;                   // producer warps for K, and for V
constexpr int kWarps = kProdWarp0 + 2 * kProd, kThreads = 32 * kWarps;   // 128 registers a thread, no split needed
static_assert(kWarps == 16, "128 registers a thread");
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
constexpr uint64_t kWaitNs = 10000000000ull;   // some waits last an item, which over a cache of 10^8 tokens is a second
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLift = 7.f, kRescale = 15.f;   // log2 units: a reference is kLift below the score that set it, kept up to kRescale above
constexpr float kLowest = -3.402823466e38f;   // reference of a row whose scores are all -inf
constexpr int kEdge = 2 * kMaxNodes;       // first window-edge entry of the poison table
constexpr int kPoison = 3 * kMaxNodes;     // keys that only some rows attend: nodes, their rows, the window's edge

// One work item, made by the set-up warp.  Slots, rows and counts are below 2^31.
struct alignas(16) WorkInfo {
    unsigned long long raw[kMaxNodes];     // drafted tokens that node i attends
    unsigned long long cmp[kMaxNodes];     // drafted nodes whose completed row node i attends (sel: its whole path)
    int lo[kMaxNodes];                     // first committed slot that node i attends
    unsigned long long any_raw, all_raw, any_cmp, all_cmp;   // over the item's nodes
    int lo_min, lo_max;
    int s, len, t0;                        // session; committed tokens; first slot of the key runs
    int raw_runs, comp_runs, n_runs;       // runs of raw slots, of committed compressed rows (sel: of the list), in all
    int n_vis0;                            // committed compressed rows (sel: list entries)
    int node;                              // sel: the node
    int row0, rows;                        // first row in the session, valid rows (<= 256)
    int sides2;                            // two row blocks
    int tile0, tile1;                      // key tiles of this item
    int pieces, part;                      // CTAs that share the row tile; this one's place in the partial results
    int stop;                              // no item: the CTA is done
    int dirty;                             // poison entries exist
    int n_vis, n_done;                     // sel: rows complete at the node's position, and at the draft's start
};
struct Work : WorkInfo {                   // (with sel an item is one node: no key is some rows' only)
    alignas(16) uint32_t poison[kPoison][12];          // per key: NaN, +inf, -inf bits of its 128 values
};

struct Bars {
    uint64_t k_full[kNS], k_empty[kNS], v_full[4], v_ok[4], v_empty[4];
    uint64_t q_full, q_empty;
    uint64_t s_full[2][2], p_full[2][2];   // [side][score buffer]
    uint64_t pv[2];                        // a product with V is done
    uint64_t o_full[2], o_empty[2];        // the item's last one; the accumulator has been read
    uint64_t w_full[2], w_empty[2], chk[2];
    uint64_t join[2];                      // side x has posted its references and sums
};

// With sel the query block is 64 rows (the products read 128: the other 64 are what follows in
// shared memory, rows that nobody reads) and there is no poison table, which leaves room for two V
// stages a side: listed rows come slowly, and a V stage is held until its product is done
// (attn_sel_16x16 29.7 us against 32 with one a side).
template <int D, bool kSel>
struct Layout {
    using W = std::conditional_t<kSel, WorkInfo, Work>;
    static constexpr int tile = kTK * D * 2;
    static constexpr int nv = kSel ? 4 : kNS;                 // V stages
    static constexpr int q_rows = kSel ? 64 : kTK;
    static constexpr int q = 0;                               // row blocks
    static constexpr int k = q + (kSel ? tile / 2 : 2 * tile);
    static constexpr int v = k + kNS * tile;
    static constexpr int work = v + nv * tile;
    // uint16 [8][8]: readable keys per run of the CTA's tile number & 7, once from the K and once from the V
    // producers; then uint8 [8][8]: every row of the item attends every key of the run.  A slot is written again eight tiles on, two stages ahead of the products; those two tiles
    // on are issued only when the softmax of this one is done.
    static constexpr int info = work + 2 * static_cast<int>(sizeof(W));
    static constexpr int whole = info + 2 * kInfo * kRuns * 2;
    static constexpr int ml = whole + kInfo * kRuns;           // float2 [2 sides][128] (reference, sum)
    static constexpr int bars = ml + 2 * kTK * 8;
    static constexpr int end = bars + static_cast<int>(sizeof(Bars));
    static constexpr size_t bytes = end + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
    static_assert(work % 16 == 0 && bars % 8 == 0 && sizeof(W) % 16 == 0, "alignment");
};

struct Args {
    CUtensorMap map_q, map_k, map_v;               // 128-row (sel: 64-row) boxes; 16-row boxes over the pools
    CUtensorMap map_ck, map_cv;                    // compressed rows: 16-row boxes (sel: one-row, gathers)
    AttnTreeArgs a;
    float *part;                                   // stream: [2 per CTA][tile rows][D], a row tile's tail and head pieces
    float2 *part_ml;                               // [2 per CTA][tile rows] (max, sum)
    int2 *pieces;                                  // [row tiles] (CTAs that share it, the first of them)
    int B, mode, min_tiles, row_tiles, tile_rows, item_rows, n_work;
    int pool_oob, comp_oob;                        // rows of the maps: the zero-fill rows
    uint32_t h_mul;                                // node_of
};

enum { kDirect, kWalk, kStream };

struct JoinArgs {
    const float *part;
    const float2 *part_ml;
    const int2 *pieces;
    PagedKV kv;
    const int32_t *n_node;
    uint16_t *out;
    long long cap;
    int B, N, H, ratio, row_tiles, tile_rows, item_rows;
};

// row / H of a session's row (below 64 * 64 + 256) without a division: h_mul = ceil(2^20 / H)
DS4A_DEVINL int node_of(const Args &g, int row) { return static_cast<int>((static_cast<uint32_t>(row) * g.h_mul) >> 20); }

DS4A_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// 1 / sum of a row's weights: 0 for a row without keys, NaN for scores that are all -inf
DS4A_DEVINL float inverse(float m, float l) {
    return l != 0.f ? 1.f / l : (m == -INFINITY ? 0.f : __uint_as_float(0x7fffffffu));
}
DS4A_DEVINL int clamp16(int x) { return x < 0 ? 0 : (x > kRun ? kRun : x); }

// Valid keys of run v for a row with first committed slot lo, drafted tokens raw and
// completed rows cmp.  kSel: runs behind the raw ones are the list's, whose bits are in info.
template <bool kSel>
DS4A_DEVINL uint32_t run_bits(const WorkInfo &w, int v, int lo, unsigned long long raw, unsigned long long cmp,
                              const uint16_t *info) {
    if (v < w.raw_runs) {
        const int t = w.t0 + v * kRun;
        const int b = clamp16(lo - t), e = clamp16(w.len - t), d = t - w.len;
        uint32_t bits = ((1u << e) - 1u) & ~((1u << b) - 1u);
        if (d > -kRun && d < kMaxNodes) bits |= static_cast<uint32_t>(d >= 0 ? raw >> d : raw << -d);
        return bits & info[v & (kRuns - 1)];
    }
    if (kSel) return info[v & (kRuns - 1)];   // behind the list: 0
    v -= w.raw_runs;
    if (v < w.comp_runs) return (1u << clamp16(w.n_vis0 - v * kRun)) - 1u;
    v -= w.comp_runs;
    return v * kRun < kMaxNodes ? static_cast<uint32_t>(cmp >> (v * kRun)) & 0xffffu : 0u;
}
// every key of tile t is valid for every row (with readable pages).  Slots and rows go up to 2^31 - 16, so
// nothing is added to one: the room behind it is compared.
DS4A_DEVINL bool tile_full(const WorkInfo &w, int t) {
    const int v = t * kRuns;
    if (v < w.raw_runs) {
        const int slot = w.t0 + v * kRun;
        return slot >= w.lo_max && w.len - slot >= kTK;
    }
    return v - w.raw_runs + kRuns <= w.n_vis0 / kRun;
}

// some row masks keys of tile t whose V rows are read (not the list's: a skipped entry loads zeros)
template <bool kSel>
DS4A_DEVINL bool needs_check(const WorkInfo &w, int t) {
    return kSel ? t * kRuns < w.raw_runs : !tile_full(w, t);
}

// chunks of tile t: the second has runs, or not
DS4A_DEVINL int tile_chunks(int n_runs, int t) { return t * kRuns + kChunkRuns < n_runs ? 2 : 1; }

DS4A_DEVINL unsigned long long shfl64(unsigned long long v, int src) { return __shfl_sync(0xffffffffu, v, src); }

// An item: session (-1: none), row tile, its key tiles t0 .. t1-1 (as far as there are any);
// stream: how many CTAs share the row tile, the first of them, this one's place.
struct Item {
    int s, rt, t0, t1, pieces, first, part;
};
DS4A_DEVINL Item direct_item(const Args &g) {
    Item id{-1, 0, 0, 0x7fffffff, 1, 0, 0};
    if (static_cast<int>(blockIdx.x) < g.n_work) {
        const unsigned x = blockIdx.x;
        id.rt = g.B > 1 ? x / static_cast<unsigned>(g.B) : x;
        id.s = x - id.rt * g.B;
    }
    return id;
}

// First slot of a session's key runs when every node's window is meant (the widest: depth 0)
DS4A_DEVINL int session_t0(const AttnTreeArgs &a, int len) {
    const long long lo = static_cast<long long>(len) - a.window + 1;
    return (lo < 0 ? 0 : min(static_cast<int>(lo), len)) & ~(kRun - 1);
}
DS4A_DEVINL int runs_of(int rows) { return rows / kRun + (rows % kRun != 0); }   // rows + kRun may not fit 32 bits

// The set-up warp's walk over the sessions, 32 at a time.  A session counts its row tiles that
// have nodes (64 sessions of 16 .. 32 nodes, 406 of 512 row tiles in use: 3 items a CTA at
// most instead of 4), or in stream mode their key tiles; one that must be left alone counts none.
struct Walk {
    int first, tiles;                // first session of the group; this lane's session's key tiles (stream)
    long long before, mine, incl;    // counted before the group; this lane's session; up to and with it
};
template <bool kSel>
DS4A_DEVINL void walk_load(const Args &g, Walk &k, int first, long long before, int lane) {
    const AttnTreeArgs &a = g.a;
    k.first = first;
    k.before = before;
    k.mine = 0;
    k.tiles = 0;
    if (first + lane < g.B) {
        const Session ses = load_session(a.kv, a.n_node, a.N, first + lane, a.err);
        const int done = ses.ok && a.ratio > 0 ? static_cast<int>(static_cast<unsigned>(ses.len) / static_cast<unsigned>(a.ratio)) : 0;
        if (ses.ok && done > a.cap - a.N && a.ratio > 0) {
            record_error(a.err, DS4A_ERR_CAPACITY);
        } else if (ses.ok) {
            k.mine = static_cast<int>(static_cast<unsigned>(ses.n * a.H + g.item_rows - 1) / static_cast<unsigned>(g.item_rows));
            if (g.mode == kStream) {
                const int len = static_cast<int>(ses.len);
                int runs = runs_of(len + ses.n - session_t0(a, len)) + runs_of(kSel ? a.n_sel : done);
                if (!kSel && a.ratio > 0) runs += runs_of(ses.n);
                k.tiles = (runs + kRuns - 1) / kRuns;
                k.mine *= k.tiles;
            }
        }
    }
    k.incl = k.mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, k.incl, o);
        if (lane >= o) k.incl += up;
    }
}
DS4A_DEVINL long long walk_end(const Walk &k) { return k.before + __shfl_sync(0xffffffffu, k.incl, 31); }
// Moves to the group of number t; the lane whose session has it, or -1 behind the last.
template <bool kSel>
DS4A_DEVINL int walk_to(const Args &g, Walk &k, long long t, int lane) {
    for (;;) {
        const long long end = walk_end(k);
        if (t < end) return __ffs(__ballot_sync(0xffffffffu, k.before + k.incl > t)) - 1;
        if (k.first + 32 >= g.B) return -1;
        walk_load<kSel>(g, k, k.first + 32, end, lane);
    }
}
template <bool kSel>
DS4A_DEVINL Item walk_item(const Args &g, Walk &k, int number, int lane) {
    Item id{-1, 0, 0, 0x7fffffff, 1, 0, 0};
    const int l = walk_to<kSel>(g, k, number, lane);
    if (l >= 0) {
        id.s = k.first + l;
        id.rt = static_cast<int>(number - k.before - __shfl_sync(0xffffffffu, k.incl - k.mine, l));
    }
    return id;
}
// non-negative a / b; in 32 bits when they fit, as they do but for lines of millions of tiles
DS4A_DEVINL long long quot(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b)) : a / b;
}

// The line of key tiles is cut at units * c / ctas; piece u .. end of this CTA's share.
struct Share {
    long long units, u, end;
    int ctas;
};
template <bool kSel>
DS4A_DEVINL Share stream_share(const Args &g, Walk &k, int lane) {
    walk_load<kSel>(g, k, 0, 0, lane);
    while (k.first + 32 < g.B) walk_load<kSel>(g, k, k.first + 32, walk_end(k), lane);
    Share h;
    h.units = walk_end(k);
    if (g.B > 32) walk_load<kSel>(g, k, 0, 0, lane);
    const long long most = quot(h.units + g.min_tiles - 1, g.min_tiles);
    h.ctas = most < static_cast<long long>(gridDim.x) ? static_cast<int>(most) : static_cast<int>(gridDim.x);
    const int c = blockIdx.x;
    h.u = c < h.ctas ? quot(h.units * c, h.ctas) : 0;
    h.end = c < h.ctas ? quot(h.units * (c + 1), h.ctas) : 0;
    return h;
}
template <bool kSel>
DS4A_DEVINL Item stream_item(const Args &g, Walk &k, Share &h, int lane) {
    Item id{-1, 0, 0, 0, 1, 0, 0};
    if (h.u >= h.end) return id;
    const int l = walk_to<kSel>(g, k, h.u, lane);
    if (l < 0) return id;
    const int tiles = __shfl_sync(0xffffffffu, k.tiles, l);
    const long long at = k.before + __shfl_sync(0xffffffffu, k.incl - k.mine, l);   // the session's first unit
    id.s = k.first + l;
    id.rt = static_cast<int>(quot(h.u - at, tiles));
    const long long lo = at + static_cast<long long>(id.rt) * tiles, hi = lo + tiles;
    id.t0 = static_cast<int>(h.u - lo);
    const long long end = hi < h.end ? hi : h.end;
    id.t1 = static_cast<int>(end - lo);
    // the CTA that has unit x: the largest c with units * c / ctas <= x
    id.first = static_cast<int>(quot((lo + 1) * h.ctas - 1, h.units));
    id.pieces = static_cast<int>(quot(hi * h.ctas - 1, h.units)) - id.first + 1;
    id.part = 2 * static_cast<int>(blockIdx.x) + (id.first == static_cast<int>(blockIdx.x));   // a head or a tail of this CTA
    h.u = end;
    return id;
}

// or / and over the warp
template <bool kOr>
DS4A_DEVINL unsigned long long reduce64(unsigned long long v) {
    const uint32_t lo = static_cast<uint32_t>(v), hi = static_cast<uint32_t>(v >> 32);
    const uint32_t l = kOr ? __reduce_or_sync(0xffffffffu, lo) : __reduce_and_sync(0xffffffffu, lo);
    const uint32_t h = kOr ? __reduce_or_sync(0xffffffffu, hi) : __reduce_and_sync(0xffffffffu, hi);
    return static_cast<unsigned long long>(h) << 32 | l;
}

// The set-up warp's item: lane holds nodes lane and lane + 32.
template <bool kSel, typename W>
__device__ void make_work(const Args &g, const Item id, W &w, int lane) {
    const AttnTreeArgs &a = g.a;
    if (lane == 0) w.stop = id.s < 0;
    if (id.s < 0) {
        __syncwarp();
        return;
    }
    const int rt = id.rt, s = id.s;
    int p[2];                                         // parents, loaded beside the session's counts
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        p[x] = a.parent && i < a.N ? __ldg(a.parent + static_cast<long long>(s) * a.N + i) : i - 1;
    }
    const Session ses = load_session(a.kv, a.n_node, a.N, s, lane == 0 ? a.err : nullptr);
    bool ok = ses.ok;
    const unsigned len_u = ok ? static_cast<unsigned>(ses.len) : 0u;       // below 2^31: it fits the pages
    const int n_done = a.ratio > 0 ? static_cast<int>(len_u / static_cast<unsigned>(a.ratio)) : 0;
    if (n_done > a.cap - a.N && a.ratio > 0) {
        if (lane == 0) record_error(a.err, DS4A_ERR_CAPACITY);
        ok = false;
    }
    const int row0 = kSel ? rt * a.H : rt * g.tile_rows;
    const int n = ok ? ses.n : 0, len = static_cast<int>(len_u);
    int rows = n * a.H - row0;
    rows = rows < 0 ? 0 : rows;
    if (rows > (kSel ? a.H : g.tile_rows)) rows = kSel ? a.H : g.tile_rows;
    // ancestors by pointer jumping: after round r a mask holds the nearest 2^r path members
    unsigned long long m[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        if (i >= n) {
            p[x] = -1;
        } else if (p[x] < -1 || p[x] >= i) {
            record_error(a.err, DS4A_ERR_DEVICE_INDEX);
            ok = false;
            p[x] = -1;
        }
        m[x] = 1ull << i;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) rows = 0;
    for (int span = 1; span < n; span *= 2) {
        unsigned long long nm[2];
        int np[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int src = p[x] & 31;
            const unsigned long long m0 = shfl64(m[0], src), m1 = shfl64(m[1], src);
            const int p0 = __shfl_sync(0xffffffffu, p[0], src), p1 = __shfl_sync(0xffffffffu, p[1], src);
            nm[x] = p[x] < 0 ? m[x] : m[x] | (p[x] < 32 ? m0 : m1);
            np[x] = p[x] < 0 ? -1 : (p[x] < 32 ? p0 : p1);
        }
        m[0] = nm[0];
        m[1] = nm[1];
        p[0] = np[0];
        p[1] = np[1];
    }
    // window: a drafted ancestor is in it if it is among the path's last `window` members
    const int i0 = rows > 0 ? node_of(g, row0) : 0, i1 = rows > 0 ? node_of(g, row0 + rows - 1) : -1;
    unsigned long long done = 0;                     // nodes that complete a row
    if (a.ratio > 0 && !kSel) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            const bool c = i < n && static_cast<unsigned>(len + __popcll(m[x])) % static_cast<unsigned>(a.ratio) == 0;
            done |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, c)) << (32 * x);
        }
    }
    unsigned long long any_raw = 0, all_raw = ~0ull, any_cmp = 0, all_cmp = ~0ull;
    int lo_min = 0x7fffffff, lo_max = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        const int depth = __popcll(m[x]) - 1;
        unsigned long long raw = m[x];
        for (long long c = depth + 1; c > a.window; --c) raw &= raw - 1;   // the shallowest fall out of the window
        const long long lo64 = static_cast<long long>(len) + depth - a.window + 1;
        const int lo = lo64 < 0 ? 0 : static_cast<int>(lo64);
        const unsigned long long cmp = kSel ? m[x] : m[x] & done;
        w.raw[i] = raw;
        w.cmp[i] = cmp;
        w.lo[i] = lo;
        if (i >= i0 && i <= i1) {
            any_raw |= raw;
            all_raw &= raw;
            any_cmp |= cmp;
            all_cmp &= cmp;
            lo_min = min(lo_min, lo);
            lo_max = max(lo_max, lo);
        }
    }
    any_raw = reduce64<true>(any_raw);
    all_raw = reduce64<false>(all_raw);
    any_cmp = reduce64<true>(any_cmp);
    all_cmp = reduce64<false>(all_cmp);
    lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    if constexpr (!kSel)
        if (w.dirty)
            for (int x = lane; x < kPoison * 12; x += 32) (&w.poison[0][0])[x] = 0;
    __syncwarp();   // w.cmp is read below
    if (lane == 0) {
        const int t0 = g.mode == kStream ? session_t0(a, len) : min(lo_min, len) & ~(kRun - 1);
        w.any_raw = any_raw;
        w.all_raw = all_raw;
        w.any_cmp = any_cmp;
        w.all_cmp = all_cmp;
        w.lo_min = lo_min;
        w.lo_max = lo_max;
        w.s = s;
        w.len = len;
        w.t0 = t0;
        w.raw_runs = runs_of(len + n - t0);
        w.n_vis0 = kSel ? a.n_sel : n_done;
        w.comp_runs = runs_of(w.n_vis0);
        w.n_runs = w.raw_runs + w.comp_runs;
        // the draft's rows (stream: the session's all, as in the walk), as far as one of the item's nodes attends any
        if (!kSel && a.ratio > 0 && g.mode == kStream) w.n_runs += runs_of(n);
        else if (!kSel && any_cmp) w.n_runs += (64 - __clzll(static_cast<long long>(any_cmp)) + kRun - 1) / kRun;
        w.node = i0;
        if (kSel) {
            const int depth = __popcll(rows > 0 ? w.cmp[i0] : 1ull) - 1;
            w.n_vis = (len + depth + 1) / a.ratio;
            w.n_done = n_done;
        }
        w.row0 = row0;
        w.rows = rows;
        w.sides2 = rows > kTK;
        const int tiles = rows > 0 ? (w.n_runs + kRuns - 1) / kRuns : 0;
        w.tile0 = min(tiles, id.t0);
        w.tile1 = min(tiles, id.t1);
        w.pieces = id.pieces;
        w.part = id.part;
        w.dirty = 0;
        if (g.mode == kStream && id.first == static_cast<int>(blockIdx.x))
            g.pieces[s * g.row_tiles + rt] = make_int2(rows > 0 ? id.pieces : 0, id.first);
    }
    __syncwarp();
}

// Row of entry j of the node's list in the session's compressed rows: -1 (skipped) if negative,
// and recorded if not complete at the node's position.
DS4A_DEVINL int sel_row(const AttnTreeArgs &a, const WorkInfo &w, int j, bool record) {
    if (j < 0) return -1;
    if (j >= w.n_vis) {
        if (record) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
        return -1;
    }
    if (j < w.n_done) return j;
    return static_cast<int>(a.cap) - a.N + path_node(w.cmp[w.node], (j + 1) * a.ratio - 1 - w.len);
}

// Sets the values of 16 bytes of a V row that are not finite to 0; notes them for key `slot` of
// the item's poison table (-1: no row attends the key), at column col and up.
__device__ __noinline__ void clean_chunk(Work *w, unsigned char *at, int slot, int col) {
    uint32_t nan = 0, pi = 0, ni = 0;
    for (int e = 0; e < 8; ++e) {
        uint16_t &h = reinterpret_cast<uint16_t *>(at)[e];
        if ((h & 0x7c00u) != 0x7c00u) continue;
        if (h & 0x03ffu) nan |= 1u << e;
        else if (h & 0x8000u) ni |= 1u << e;
        else pi |= 1u << e;
        h = 0;
    }
    if (slot < 0 || w == nullptr) return;
    const int word = col / 32, sh = col % 32;
    if (nan) atomicOr(&w->poison[slot][word], nan << sh);
    if (pi) atomicOr(&w->poison[slot][4 + word], pi << sh);
    if (ni) atomicOr(&w->poison[slot][8 + word], ni << sh);
    w->dirty = 1;
}

// Values that are not finite, of the keys that `node` attends: added to columns col .. col+31 of
// its accumulator, which holds those of the keys that every row attends.
__device__ __noinline__ uint3 poison_bits(const Work &w, int node, int word) {
    const int lo = w.lo[node];
    const unsigned long long raw = w.raw[node], cmp = w.cmp[node];
    uint32_t nan = 0, pi = 0, ni = 0;
    for (int key = 0; key < kPoison; ++key) {
        bool hit;
        if (key < kMaxNodes) hit = (raw >> key) & 1ull;
        else if (key < kEdge) hit = (cmp >> (key - kMaxNodes)) & 1ull;
        else hit = static_cast<unsigned>(w.lo_min) + (key - kEdge) >= static_cast<unsigned>(lo);
        if (!hit) continue;
        nan |= w.poison[key][word];
        pi |= w.poison[key][4 + word];
        ni |= w.poison[key][8 + word];
    }
    return make_uint3(nan | (pi & ni), pi, ni);
}
DS4A_DEVINL void add_poison(const Work &w, int node, int col, uint32_t (&o)[32]) {
    const uint3 p = poison_bits(w, node, col / 32);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        if ((p.x >> e) & 1u) o[e] = 0x7fffffffu;
        else if ((p.y >> e) & 1u) o[e] = __float_as_uint(__uint_as_float(o[e]) + INFINITY);
        else if ((p.z >> e) & 1u) o[e] = __float_as_uint(__uint_as_float(o[e]) - INFINITY);
    }
}

// 4 x 4 pieces of 16 bytes among four neighbouring lanes: piece j of lane i goes to lane j's place i
DS4A_DEVINL void transpose4(uint4 (&u)[4], int lane) {
#pragma unroll
    for (int b = 1; b <= 2; b <<= 1) {
        const bool up = (lane & b) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & b) continue;
            const uint4 send = up ? u[i] : u[i | b];
            uint4 got;
            got.x = __shfl_xor_sync(0xffffffffu, send.x, b);
            got.y = __shfl_xor_sync(0xffffffffu, send.y, b);
            got.z = __shfl_xor_sync(0xffffffffu, send.z, b);
            got.w = __shfl_xor_sync(0xffffffffu, send.w, b);
            if (up) u[i] = got;
            else u[i | b] = got;
        }
    }
}

template <int D, bool kSel>
__global__ void __launch_bounds__(kThreads, 1) attn_tree_kernel(const __grid_constant__ Args g) {
    using L = Layout<D, kSel>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using W = typename L::W;
    W *works = reinterpret_cast<W *>(smem + L::work);
    uint16_t *info = reinterpret_cast<uint16_t *>(smem + L::info);
    uint8_t *whole = smem + L::whole;
    float2 *s_ml = reinterpret_cast<float2 *>(smem + L::ml);
    Bars &bar = *reinterpret_cast<Bars *>(smem + L::bars);
    __shared__ uint32_t s_tmem;
    const AttnTreeArgs &a = g.a;
    // the shuffle tells the compiler that the warp's number is the same in all its lanes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int kAtoms = D / 64, kAtomBytes = kTK * 128;

    if (tid == 0) {
        // a stage is released by two commits: one of each side, or two of the side whose tile it is
        for (int x = 0; x < kNS; ++x) {
            tc::mbar_init(&bar.k_full[x], kProd);
            tc::mbar_init(&bar.k_empty[x], 2);
        }
        for (int x = 0; x < L::nv; ++x) {
            tc::mbar_init(&bar.v_full[x], kProd);
            tc::mbar_init(&bar.v_ok[x], 1);
            tc::mbar_init(&bar.v_empty[x], 2);
        }
        tc::mbar_init(&bar.q_full, 1);
        tc::mbar_init(&bar.q_empty, 2);
        for (int x = 0; x < 2; ++x) {
            for (int y = 0; y < 2; ++y) {
                tc::mbar_init(&bar.s_full[x][y], 1);
                tc::mbar_init(&bar.p_full[x][y], kSideWarps);
            }
            tc::mbar_init(&bar.pv[x], 1);
            tc::mbar_init(&bar.o_full[x], 1);
            tc::mbar_init(&bar.o_empty[x], 2 * kSideWarps);
            tc::mbar_init(&bar.join[x], kSideWarps);
            tc::mbar_init(&bar.w_full[x], 1);
            tc::mbar_init(&bar.w_empty[x], kWarps - 1);
            tc::mbar_init(&bar.chk[x], 1);
        }
        tc::mbar_fence_init();
    }
    if constexpr (!kSel)
        for (int x = tid; x < kPoison * 3; x += kThreads) {
            reinterpret_cast<uint4 *>(works[0].poison)[x] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4 *>(works[1].poison)[x] = make_uint4(0, 0, 0, 0);
        }
    if (warp == kSetupWarp && lane < 2) works[lane].dirty = 0;
    if (warp == kMmaWarp) tc::tmem_alloc(&s_tmem, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    pdl_wait();
    pdl_trigger();
    bool ok = true;
    // a failed wait records the failure; later waits of this thread return at once
    auto wait = [&](uint64_t *b, uint32_t parity) {
        if (ok && !tc::mbar_wait(b, parity & 1u, kWaitNs)) ok = false;
        return ok;
    };
    if (warp < kSoftWarps) {
        const int side = warp / kSideWarps, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t col_s = tmem + lanes + kColS + side * kTK, col_o = tmem + lanes + kColO + side * kTK;
        const float c2 = a.scale_log2;
        uint32_t n_c = 0, n_o = 0, n_join = 0, n_t = 0;   // this side's chunks and items, joined items, tiles so far
        for (int it = 0;; ++it) {
            W &w = works[it & 1];
            if (!__all_sync(0xffffffffu, wait(&bar.w_full[it & 1], it >> 1)) || w.stop) break;
            const int t0 = w.tile0, t1 = w.tile1, sides2 = w.sides2, n_runs = w.n_runs;
            const int row = (sides2 ? side * kTK : 0) + r;        // row in the item
            const int node = min(kMaxNodes - 1, node_of(g, w.row0 + row));
            float m = -INFINITY, l = 0.f;
            uint32_t seen = 0;                       // not 0: the row attends a key
            bool first = true;
            for (int t = sides2 ? t0 : t0 + side; t < t1; t += sides2 ? 1 : 2) {
                const uint16_t *inf = info + ((n_t + t - t0) & (kInfo - 1)) * kRuns;
                const int chunks = tile_chunks(n_runs, t);
                const uint8_t *wh = whole + ((n_t + t - t0) & (kInfo - 1)) * kRuns;
                for (int c = 0; c < chunks; ++c, ++n_c) {
                    const uint32_t sb = n_c & 1u, col = col_s + sb * kCK;
                    wait(&bar.s_full[side][sb], n_c >> 1);
                    tc::fence_after_sync();
                    uint32_t x[2][32];
                    tc::ld_x32(col, x[0]);
                    tc::ld_x32(col + 32, x[1]);
                    const uint32_t full = *reinterpret_cast<const uint32_t *>(wh + c * kChunkRuns);   // a byte per run
                    tc::wait_ld();
                    seen |= full;
                    if (full != 0x01010101u) {
                        const int lo = w.lo[node];
                        const unsigned long long raw = w.raw[node], cmp = w.cmp[node];
#pragma unroll
                        for (int u = 0; u < kChunkRuns; ++u) {
                            if ((full >> (8 * u)) & 1u) continue;
                            const uint32_t bits =
                                run_bits<kSel>(w, t * kRuns + c * kChunkRuns + u, lo, raw, cmp, inf);
                            seen |= bits;
#pragma unroll
                            for (int e = 0; e < kRun; ++e)
                                if (!((bits >> e) & 1u)) x[u / 2][(u & 1) * kRun + e] = 0xff800000u;   // -inf
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            mx[(e >> 1) & 3] =
                                fmaxf(fmaxf(mx[(e >> 1) & 3], __uint_as_float(x[h][e])), __uint_as_float(x[h][e + 1]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;   // scale > 0
                    // raise the reference: at the first finite score, then only past the threshold
                    float alpha = 1.f;
                    if (top > m + kRescale || (m == -INFINITY && top > m)) {
                        alpha = ex2(m - (top - kLift));
                        m = top - kLift;
                        l *= alpha;
                    }
                    if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
                        wait(&bar.pv[side], n_c - 1);   // the product before (the one before that is done: these scores came after it)
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int d = 0; d < D / 16; ++d) {
                            uint32_t o[16];
                            tc::ld_x16(col_o + d * 16, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc::st_x16(col_o + d * 16, o);
                        }
                    }
                    first = false;
                    const float ref = m == -INFINITY ? 0.f : m;
                    const uint64_t c22 = tc::pack2(c2, c2), ref2 = tc::pack2(-ref, -ref);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float y0, y1;
                            tc::unpack2(tc::fma2(tc::pack2(__uint_as_float(x[h][2 * e]), __uint_as_float(x[h][2 * e + 1])),
                                                 c22, ref2), y0, y1);
                            const float p0 = ex2(y0), p1 = ex2(y1);
                            sum[e & 1] = tc::add2(sum[e & 1], tc::pack2(p0, p1));
                            pk[e] = pack_half2(p0, p1);
                        }
                        tc::st_x16(col + h * 16, pk);
                    }
                    float s0, s1;
                    tc::unpack2(tc::add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tc::wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.p_full[side][sb]);
                }
            }
            n_t += t1 - t0;
            // ---- end of the item ----
            // l is 0 with m = -inf for a row without keys (its output is 0), with m = kLowest for one whose scores
            // are all -inf (NaN, unless another side or piece has a finite score: kLowest weighs nothing beside it)
            if (m == -INFINITY && seen) m = kLowest;
            const bool have = !first;                              // this side has tiles
            const bool joined = !sides2 && t1 - t0 > 1;            // side 1 holds part of the same rows
            if (have) {
                wait(&bar.o_full[side], n_o++);
                if (joined) {
                    s_ml[side * kTK + r] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.join[side]);
                    wait(&bar.join[side ^ 1], n_join++);
                }
                tc::fence_after_sync();
                {
                    // a joined item's sides finish half of the columns each: the weights of this side's and the
                    // other side's accumulator
                    float wa = 1.f, wb = 0.f;
                    if (joined) {
                        const float2 o = s_ml[(side ^ 1) * kTK + r];
                        const float mm = fmaxf(m, o.x), rf = mm == -INFINITY ? 0.f : mm;
                        wa = ex2(m - rf);
                        wb = ex2(o.x - rf);
                        l = l * wa + o.y * wb;
                        m = mm;
                    }
                    const uint32_t col_other = tmem + lanes + kColO + (side ^ 1) * kTK;
                    const int c0 = joined && side == 1 ? D / 64 : 0, c1 = joined && side == 0 ? D / 64 : D / 32;
                    wait(&bar.chk[it & 1], it >> 1);
                    const bool valid = row < w.rows, direct = w.pieces == 1;
                    const int dirty = w.dirty;
                    const float inv = inverse(m, l);
                    const long long qrow = (static_cast<long long>(w.s) * a.N) * a.H + w.row0 + row;
                    const long long prow = static_cast<long long>(w.part) * g.tile_rows + row;
                    if (!direct && valid && c0 == 0) g.part_ml[prow] = make_float2(m, l);
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {                // 32 columns at a time
                        uint32_t o[32];
                        tc::ld_x32(col_o + c * 32, o);
                        if (joined) {
                            uint32_t o2[32];
                            tc::ld_x32(col_other + c * 32, o2);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * wa + __uint_as_float(o2[e]) * wb);
                        } else {
                            tc::wait_ld();
                        }
                        if constexpr (!kSel)
                            if (dirty) add_poison(w, node, c * 32, o);
                        // With two row blocks four lanes trade 16-byte pieces, so that each writes its piece of
                        // four rows and a store covers 64 contiguous bytes of 8 rows instead of 16 bytes of 32
                        // (attn_r128_64x32 52 against 55.5 us); with one, where the item waits for it, each lane
                        // writes its own row (the trade cost attn_sel_16x16 2 us and attn_window_1x4 0.7).
                        const int row4 = row - (lane & 3), piece = lane & 3;
                        if (direct) {
                            uint4 u[4];
#pragma unroll
                            for (int q4 = 0; q4 < 4; ++q4) {
                                uint32_t h[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    h[e] = pack_half2(__uint_as_float(o[q4 * 8 + 2 * e]) * inv,
                                                      __uint_as_float(o[q4 * 8 + 2 * e + 1]) * inv);
                                u[q4] = make_uint4(h[0], h[1], h[2], h[3]);
                            }
                            if (sides2) {
                                transpose4(u, lane);
                                uint16_t *dst = a.out + (qrow - (lane & 3)) * D + c * 32 + piece * 8;
#pragma unroll
                                for (int q4 = 0; q4 < 4; ++q4)
                                    if (row4 + q4 < w.rows) *reinterpret_cast<uint4 *>(dst + q4 * D) = u[q4];
                            } else if (valid) {
                                uint16_t *dst = a.out + qrow * D + c * 32;
#pragma unroll
                                for (int q4 = 0; q4 < 4; ++q4) *reinterpret_cast<uint4 *>(dst + q4 * 8) = u[q4];
                            }
                        } else {
                            float *dst = g.part + (prow - (lane & 3)) * D + c * 32 + piece * 4;
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                uint4 u[4];
#pragma unroll
                                for (int q4 = 0; q4 < 4; ++q4)
                                    u[q4] = make_uint4(o[hf * 16 + q4 * 4], o[hf * 16 + q4 * 4 + 1], o[hf * 16 + q4 * 4 + 2],
                                                       o[hf * 16 + q4 * 4 + 3]);
                                transpose4(u, lane);
#pragma unroll
                                for (int q4 = 0; q4 < 4; ++q4)
                                    if (row4 + q4 < w.rows) *reinterpret_cast<uint4 *>(dst + q4 * D + hf * 16) = u[q4];
                            }
                        }
                    }
                }
                // Both accumulators may be overwritten when both sides' warps have read them, each warp counting
                // once for each; a side that has an accumulator, or the item, to itself counts for the other too.
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    for (int x = 0; x < 2; ++x) {
                        tc::mbar_arrive(&bar.o_empty[side]);
                        if (!sides2 && (!joined || x == 0)) tc::mbar_arrive(&bar.o_empty[side ^ 1]);
                        if (joined) break;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.w_empty[it & 1]);
        }
    } else {
        // All lanes poll, so that the code around stays converged and its operands uniform (with one lane
        // polling for the warp every hand-off was slower); the outcome is the same in every lane.
        auto warp_wait = [&](uint64_t *b, uint32_t parity) {
            ok = __all_sync(0xffffffffu, wait(b, parity));
            return ok;
        };
        if (warp == kSetupWarp) {
            uint32_t n_q = 0;
            auto load_q = [&](int s, int row0) {
                if (n_q > 0 && !warp_wait(&bar.q_empty, n_q - 1)) return false;
                if (lane == 0) {
                    const int blocks = !kSel && g.tile_rows > kTK ? 2 : 1;
                    const int qrow = s * a.N * a.H + row0;
                    constexpr int kBlock = L::q_rows * D * 2;
                    tc::expect_tx(&bar.q_full, blocks * kBlock);
                    for (int b = 0; b < blocks; ++b)
                        for (int at = 0; at < kAtoms; ++at)
                            tc::tma_load_2d(smem + L::q + b * kBlock + at * (L::q_rows * 128), &g.map_q, at * 64,
                                            qrow + b * kTK, &bar.q_full);
                }
                __syncwarp();
                ++n_q;
                return true;
            };
            Walk walk{};
            Share share{};
            if (lane == 0) tc::prefetch_map(&g.map_q);
            if (g.mode == kDirect) {   // the query rows are known from the CTA's number
                const Item id = direct_item(g);
                if (id.s >= 0) load_q(id.s, id.rt * g.item_rows);
            }
            if (g.mode == kWalk) walk_load<kSel>(g, walk, 0, 0, lane);
            if (g.mode == kStream) share = stream_share<kSel>(g, walk, lane);
            for (int it = 0;; ++it) {
                if (it >= 2 && !warp_wait(&bar.w_empty[it & 1], (it >> 1) - 1)) break;
                W &w = works[it & 1];
                Item id{-1, 0, 0, 0, 0, 0, 0};
                if (g.mode == kWalk) id = walk_item<kSel>(g, walk, blockIdx.x + it * gridDim.x, lane);
                else if (g.mode == kStream) id = stream_item<kSel>(g, walk, share, lane);
                else if (it == 0) id = direct_item(g);
                make_work<kSel>(g, id, w, lane);
                if (lane == 0) tc::mbar_arrive(&bar.w_full[it & 1]);
                __syncwarp();
                if (id.s < 0) break;
                // the queries, when the item before has made its last scores (its output, which frees the
                // Work after next, comes later; the K producers do not wait here)
                if (g.mode != kDirect && w.tile1 > w.tile0 && !load_q(w.s, w.row0)) break;
            }
            if (!ok && lane == 0 && n_q > 0) tc::mbar_wait(&bar.q_full, (n_q - 1) & 1u);   // a wait gave up
            __syncwarp();
        } else if (warp < kChkWarp) {
            // The whole warp runs this, converged, and one elected lane issues: the operands are then
            // warp-uniform registers, which the instruction wants (issued from a lane == 0 branch, eight
            // products took 570 cycles to issue, about as long as the tensor core needs for them).
            constexpr uint32_t kIdS = tc::idesc_f16_f32(kTK, kCK, false, false);
            constexpr uint32_t kIdO = tc::idesc_f16_f32(kTK, D, false, true);
            const uint32_t side = warp - kMmaWarp;
            uint32_t n_t = 0, n_c = 0, n_o = 0, n_q = 0;          // tiles; chunks of this side; items with tiles; query loads
            // a descriptor holds the address in 16-byte units in its low bits: steps are additions
            const uint64_t q_d = tc::desc_sw128(tc::smem_u32(smem + L::q), 16, 1024);
            const uint64_t k_d = tc::desc_sw128(tc::smem_u32(smem + L::k), 16, 1024);
            const uint64_t v_d = tc::desc_sw128(tc::smem_u32(smem + L::v), kAtomBytes, 1024);
            constexpr int kTile16 = L::tile / 16;
            const uint32_t d_s = tmem + kColS + side * kTK, d_o = tmem + kColO + side * kTK;
            for (int it = 0; ok; ++it) {
                const W &w = works[it & 1];
                if (!warp_wait(&bar.w_full[it & 1], it >> 1) || __shfl_sync(0xffffffffu, w.stop, 0)) break;
                const int tile0 = __shfl_sync(0xffffffffu, w.tile0, 0), n_runs = __shfl_sync(0xffffffffu, w.n_runs, 0);
                const int tiles = __shfl_sync(0xffffffffu, w.tile1, 0) - tile0;
                const bool sides2 = __shfl_sync(0xffffffffu, w.sides2, 0) != 0;
                const int first = sides2 ? 0 : static_cast<int>(side), by = sides2 ? 1 : 2;   // this side's tiles
                const uint64_t qd = q_d + (sides2 ? side : 0) * kTile16;
                if ((tiles > 0 || g.mode == kDirect) && !warp_wait(&bar.q_full, n_q++)) break;
                if (first >= tiles) {                             // nothing for this side: every phase is seen all the same
                    if (lane == 0 && (tiles > 0 || g.mode == kDirect)) tc::mbar_arrive(&bar.q_empty);
                    if (tiles > 0 && n_o > 0) warp_wait(&bar.o_empty[side], n_o - 1);
                }
                // the next chunk to score: tile st_t, half st_h, buffer st_n & 1
                int st_t = first, st_h = 0;
                uint32_t st_n = n_c;
                auto wait_k = [&]() {
                    if (st_t >= tiles || st_h != 0) return true;
                    const uint32_t kt = n_t + st_t;
                    return wait(&bar.k_full[kt % kNS], kt / kNS);
                };
                auto issue_s = [&]() {                            // behind wait_k
                    if (st_t >= tiles) return;
                    const uint32_t stage = (n_t + st_t) % kNS, buf = st_n & 1u;
                    const uint64_t kd = k_d + stage * kTile16 + st_h * (kCK * 128 / 16);
                    const uint32_t d = d_s + buf * kCK;
                    const bool tile_end = st_h + 1 == tile_chunks(n_runs, tile0 + st_t);
                    const bool last = tile_end && st_t + by >= tiles;
                    if (tc::elect()) {
#pragma unroll
                        for (int x = 0; x < D / 16; ++x)
                            tc::mma_f16(d, qd + (x / 4) * (L::q_rows * 8) + (x % 4) * 2,
                                        kd + (x / 4) * (kAtomBytes / 16) + (x % 4) * 2, kIdS, x > 0);
                        tc::commit(&bar.s_full[side][buf]);
                        if (tile_end) {
                            tc::commit(&bar.k_empty[stage]);
                            if (!sides2) tc::commit(&bar.k_empty[stage]);
                        }
                        if (last) tc::commit(&bar.q_empty);
                    }
                    __syncwarp();
                    ++st_n;
                    if (tile_end) {
                        st_t += by;
                        st_h = 0;
                    } else {
                        st_h = 1;
                    }
                };
                for (int x = 0; x < 2 && ok; ++x) {
                    ok = __all_sync(0xffffffffu, wait_k());
                    if (!ok) break;
                    tc::fence_after_sync();
                    issue_s();
                }
                for (int t = first; t < tiles && ok; t += by) {
                    const uint32_t vt = n_t + t, stage = vt % L::nv;
                    const int chunks = tile_chunks(n_runs, tile0 + t);
                    for (int c = 0; c < chunks && ok; ++c, ++n_c) {
                        const uint32_t buf = n_c & 1u;
                        // all waits at once, so that nothing stands between the two products
                        bool good = wait_k();
                        if (c == 0) {
                            // The item before has been read: the accumulator is free, and every earlier V tile has
                            // come, those that only the other side waited for too (so the parity below is the
                            // right phase's).
                            if (t == first && n_o > 0) good = wait(&bar.o_empty[side], n_o - 1) && good;
                            good = wait(&bar.v_ok[stage], vt / L::nv) && good;
                        }
                        const uint64_t vd = v_d + stage * kTile16 + c * (kCK / 16 * 128);
                        const uint32_t pa = d_s + buf * kCK;
                        good = wait(&bar.p_full[side][buf], n_c >> 1) && good;
                        ok = __all_sync(0xffffffffu, good);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const bool more = t != first || c != 0, tile_end = c + 1 == chunks;
                        if (tc::elect()) {
#pragma unroll
                            for (int x = 0; x < kCK / 16; ++x)
                                tc::mma_f16_ts(d_o, pa + x * 8, vd + x * 128, kIdO, more || x > 0);
                            if (tile_end) {
                                tc::commit(&bar.v_empty[stage]);
                                if (!sides2) tc::commit(&bar.v_empty[stage]);
                            }
                            tc::commit(&bar.pv[side]);
                            if (tile_end && t + by >= tiles) tc::commit(&bar.o_full[side]);
                        }
                        __syncwarp();
                        issue_s();
                    }
                }
                if (tiles > 0) ++n_o;
                n_t += tiles;
                if (lane == 0) tc::mbar_arrive(&bar.w_empty[it & 1]);
            }
            __syncwarp();
        } else if (warp < kProdWarp0) {
            // ---------------- checkers ----------------
            uint32_t n_v = 0;
            for (int it = 0;; ++it) {
                W &w = works[it & 1];
                if (!warp_wait(&bar.w_full[it & 1], it >> 1) || w.stop) break;
                for (int t = w.tile0; t < w.tile1; ++t, ++n_v) {
                    const int st = n_v % L::nv;
                    if (!warp_wait(&bar.v_full[st], n_v / L::nv)) break;
                    if (needs_check<kSel>(w, t)) {
                        const uint16_t *inf = info + (kInfo + (n_v & (kInfo - 1))) * kRuns;
                        unsigned char *vt = smem + L::v + st * L::tile;
                        bool wrote = false;
                        for (int r = 0; r < kRuns; ++r) {
                            const int v = t * kRuns + r;
                            if (v >= w.n_runs) break;                                       // zeros
                            const uint32_t any = run_bits<kSel>(w, v, w.lo_min, w.any_raw, w.any_cmp, inf);
                            const uint32_t all = run_bits<kSel>(w, v, w.lo_max, w.all_raw, w.all_cmp, inf);
                            if ((all & 0xffffu) == 0xffffu || (kSel && v >= w.raw_runs)) continue;
                            // 16 rows x 8 chunks of 16 bytes per atom, the loads of a lane all in flight
#pragma unroll
                            for (int half = 0; half < kAtoms; ++half) {
                                uint4 q[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    q[x] = *reinterpret_cast<const uint4 *>(
                                        vt + half * kAtomBytes + tc::sw128_chunk(r * kRun + x * 4 + lane / 8, lane % 8));
                                auto odd = [](uint32_t u) {   // a half with all exponent bits set
                                    const uint32_t z = (u & 0x7c007c00u) ^ 0x7c007c00u;
                                    return (z - 0x00010001u) & ~z & 0x80008000u;
                                };
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const int key = x * 4 + lane / 8, ch = lane % 8;
                                    if (!(odd(q[x].x) | odd(q[x].y) | odd(q[x].z) | odd(q[x].w)) || ((all >> key) & 1u))
                                        continue;
                                    int slot = -1;   // a key that some rows attend and some do not
                                    if ((any >> key) & 1u) {
                                        if (v < w.raw_runs) {
                                            const int tk = w.t0 + v * kRun + key;
                                            slot = tk >= w.len ? tk - w.len : kEdge + (tk - w.lo_min);
                                        } else {
                                            slot = kMaxNodes + (v - w.raw_runs - w.comp_runs) * kRun + key;
                                        }
                                    }
                                    Work *table = nullptr;
                                    if constexpr (!kSel) table = &w;
                                    clean_chunk(table, vt + half * kAtomBytes + tc::sw128_chunk(r * kRun + key, ch), slot,
                                                half * 64 + ch * 8);
                                    wrote = true;
                                }
                            }
                        }
                        if (__any_sync(0xffffffffu, wrote)) tc::fence_proxy_async();
                        __syncwarp();
                    }
                    if (lane == 0) tc::mbar_arrive(&bar.v_ok[st]);
                }
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&bar.chk[it & 1]);
                    tc::mbar_arrive(&bar.w_empty[it & 1]);
                }
            }
        } else {
            // ---------------- producers: warp pair K, warp pair V ----------------
            const bool is_v = warp >= kProdWarp0 + kProd;
            const int pw = (warp - kProdWarp0) % kProd;            // runs pw * 4 .. + 3 of each tile
            constexpr int kRunsPer = kRuns / kProd;
            uint64_t *full = is_v ? bar.v_full : bar.k_full, *empty = is_v ? bar.v_empty : bar.k_empty;
            const CUtensorMap *map_raw = is_v ? &g.map_v : &g.map_k, *map_comp = is_v ? &g.map_cv : &g.map_ck;
            unsigned char *ring = smem + (is_v ? L::v : L::k);
            const int run = pw * kRunsPer + (lane & (kRunsPer - 1));          // lane = run (and atom)
            const int group = lane & (kRunsPer * 4 - 1);                      // sel: lane = group of 4 entries
            const int grun = pw * kRunsPer + group / 4;
            if (lane == 0) {
                tc::prefetch_map(map_raw);
                if (a.ratio > 0) tc::prefetch_map(map_comp);
            }
            // the rows of one tile: this lane's run, this lane's four list entries (the raw table entries and
            // list entries of the next tile are loaded while this one waits for its stage)
            struct Rows {
                int v, gv, page, off;
                int4 e;
            };
            const int n_stages = is_v ? L::nv : kNS;
            int st = 0;
            uint32_t ph = 0, n_t = 0;
            for (int it = 0;; ++it) {
                const W &w = works[it & 1];
                if (!warp_wait(&bar.w_full[it & 1], it >> 1) || w.stop) break;
                const int tile0 = w.tile0, tile1 = w.tile1, raw_runs = w.raw_runs, n_runs = w.n_runs;
                const int32_t *table = a.kv.table + static_cast<long long>(w.s) * a.kv.max_pages;
                const int32_t *list = kSel ? a.sel + (static_cast<long long>(w.s) * a.N + w.node) * a.n_sel : nullptr;
                auto fetch = [&](int t) {
                    Rows r;
                    r.v = t * kRuns + run;
                    r.gv = t * kRuns + grun;
                    r.page = r.off = 0;
                    if (r.v < raw_runs) {
                        const unsigned slot = w.t0 + r.v * kRun, pg = slot / static_cast<unsigned>(a.kv.page);
                        r.page = __ldg(table + pg);
                        r.off = static_cast<int>(slot - pg * a.kv.page);
                    }
                    r.e = make_int4(-1, -1, -1, -1);
                    if (kSel && r.gv >= raw_runs && r.gv < n_runs) {
                        const int e0 = (r.gv - raw_runs) * kRun + (group & 3) * 4;
                        if (e0 < a.n_sel) r.e.x = __ldg(list + e0);
                        if (e0 + 1 < a.n_sel) r.e.y = __ldg(list + e0 + 1);
                        if (e0 + 2 < a.n_sel) r.e.z = __ldg(list + e0 + 2);
                        if (e0 + 3 < a.n_sel) r.e.w = __ldg(list + e0 + 3);
                    }
                    return r;
                };
                Rows next{};
                if (tile0 < tile1) next = fetch(tile0);
                for (int t = tile0; t < tile1; ++t, ++n_t) {
                    const Rows r = next;
                    if (t + 1 < tile1) next = fetch(t + 1);
                    int row = g.pool_oob;
                    bool raw_run = true, readable = true;
                    if (r.v < raw_runs) {
                        readable = r.page >= 0 && r.page < a.kv.n_pages;
                        if (readable) row = r.page * a.kv.page + r.off;
                        else if (lane < kRunsPer) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
                    } else if (!kSel && r.v < n_runs) {
                        raw_run = false;
                        const int c = r.v - raw_runs;
                        const long long base = static_cast<long long>(w.s) * a.cap;
                        row = static_cast<int>(c < w.comp_runs ? base + c * kRun
                                                               : base + a.cap - a.N + (c - w.comp_runs) * kRun);
                    }
                    int4 gr = make_int4(g.comp_oob, g.comp_oob, g.comp_oob, g.comp_oob);
                    uint32_t gmask = 0;
                    if (kSel && r.gv >= raw_runs && r.gv < n_runs) {
                        const bool record = lane < kRunsPer * 4 && !is_v;
                        const int base = w.s * static_cast<int>(a.cap);
                        const int e[4] = {sel_row(a, w, r.e.x, record), sel_row(a, w, r.e.y, record),
                                          sel_row(a, w, r.e.z, record), sel_row(a, w, r.e.w, record)};
                        if (e[0] >= 0) { gr.x = base + e[0]; gmask |= 1u; }
                        if (e[1] >= 0) { gr.y = base + e[1]; gmask |= 2u; }
                        if (e[2] >= 0) { gr.z = base + e[2]; gmask |= 4u; }
                        if (e[3] >= 0) { gr.w = base + e[3]; gmask |= 8u; }
                    }
                    if (n_t >= static_cast<uint32_t>(n_stages) && !warp_wait(&empty[st], ph ^ 1u)) break;
                    {   // readable keys per run, for the softmax (K) and the checkers (V)
                        uint32_t m16 = readable ? 0xffffu : 0u;
                        if (kSel) {
                            uint32_t gm = gmask << ((group & 3) * 4);
                            gm |= __shfl_xor_sync(0xffffffffu, gm, 1);
                            gm |= __shfl_xor_sync(0xffffffffu, gm, 2);
                            const uint32_t mine = __shfl_sync(0xffffffffu, gm, (lane & (kRunsPer - 1)) * 4);
                            if (r.v >= raw_runs) m16 = mine;
                        }
                        if (lane < kRunsPer) {
                            uint16_t *inf = info + ((is_v ? kInfo : 0) + (n_t & (kInfo - 1))) * kRuns;
                            inf[run] = static_cast<uint16_t>(m16);
                            if (!is_v)
                                whole[(n_t & (kInfo - 1)) * kRuns + run] =
                                    (run_bits<kSel>(w, r.v, w.lo_max, w.all_raw, w.all_cmp, inf) & 0xffffu) == 0xffffu;
                        }
                        __syncwarp();
                    }
                    if (lane == 0) tc::expect_tx(&full[st], L::tile / kProd);
                    __syncwarp();
                    const uint32_t dst = tc::smem_u32(ring + st * L::tile);
                    if (lane < kRunsPer * kAtoms && (!kSel || r.v < raw_runs || r.v >= n_runs)) {
                        const int at = lane / kRunsPer;
                        tc::tma_load_2d(dst + at * kAtomBytes + run * 2048, raw_run ? map_raw : map_comp, at * 64, row,
                                        &full[st]);
                    }
                    if (kSel && r.gv >= raw_runs && r.gv < n_runs && lane < kRunsPer * 4) {
                        for (int at = 0; at < kAtoms; ++at)
                            tc::tma_gather4(dst + at * kAtomBytes + (pw * kRunsPer * 4 + group) * 512, map_comp, at * 64,
                                            gr, &full[st]);
                    }
                    __syncwarp();
                    if (++st == n_stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.w_empty[it & 1]);
            }
            // a wait gave up: the copies in flight land before the block may end
            if (!ok && lane == 0) {
                const uint32_t ns = n_stages, from = n_t > ns ? n_t - ns : 0;
                for (uint32_t x = from; x < n_t; ++x) tc::mbar_wait(&full[x % ns], (x / ns) & 1u);
            }
            __syncwarp();
        }
    }
    if (!ok) record_error(a.err, DS4A_ERR_TIMEOUT);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Joins the pieces of a row: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.  kPerRow warps per
// row: one when a row has few pieces, eight when it has many (one row tile over 32768 keys has
// 128; with one warp going through them one by one the join took 40 us).  Rows of a row tile that
// one CTA had are already written.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int D, int kPerRow>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(JoinArgs g) {
    constexpr int kPer = D / 32, kBatch = 8;
    __shared__ float s_o[kPerRow > 1 ? kPerRow : 1][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kPerRow;
    const unsigned row = blockIdx.x * (kJoinWarps / kPerRow) + warp / kPerRow;   // below 2^31: a row is 128 bytes or more
    const unsigned per = g.N * g.H;
    pdl_wait();
    pdl_trigger();
    if (row >= g.B * per) return;                    // (with kPerRow > 1 a block has one row: it leaves as a whole)
    const int s = row / per, r = row - s * per, rt = static_cast<unsigned>(r) / static_cast<unsigned>(g.item_rows);
    const int2 p = g.pieces[s * g.row_tiles + rt];   // set if the session is in the line
    const Session ses = load_session(g.kv, g.n_node, g.N, s, nullptr);
    if (!ses.ok || r >= ses.n * g.H) return;
    if (g.ratio > 0 && static_cast<unsigned>(ses.len) / static_cast<unsigned>(g.ratio) > g.cap - g.N) return;
    const int pieces = p.x, first = p.y;
    if (pieces <= 1) return;
    const int in_tile = r - rt * g.item_rows;
    // the first CTA has the row tile as its tail, the others as their head
    auto at = [&](int i) { return static_cast<long long>(2 * (first + i) + (i == 0)) * g.tile_rows + in_tile; };
    float m = -INFINITY;
    for (int i = lane; i < pieces; i += 32) m = fmaxf(m, g.part_ml[at(i)].x);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    float o[kPer] = {}, l = 0.f;
    for (int c = 0; c < pieces; c += 32) {           // a lane has the weight of piece c + lane
        float w = 0.f;
        if (c + lane < pieces) {
            const float2 ml = g.part_ml[at(c + lane)];
            if (ml.y != 0.f) {                       // else: no key of this piece is this row's
                w = ex2(ml.x - ref);
                l += w * ml.y;
            }
        }
        for (int k0 = sub; k0 < 32 && c + k0 < pieces; k0 += kBatch * kPerRow) {
            float x[kBatch][kPer];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * kPerRow;
                const bool in = k < 32 && c + k < pieces;
                const float *src = g.part + at(c + k) * D + lane * kPer;
                if (kPer == 4) {
                    const float4 v = in ? *reinterpret_cast<const float4 *>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[u][0] = v.x;
                    x[u][1] = v.y;
                    x[u][kPer - 2] = v.z;
                    x[u][kPer - 1] = v.w;
                } else {
                    const float2 v = in ? *reinterpret_cast<const float2 *>(src) : make_float2(0.f, 0.f);
                    x[u][0] = v.x;
                    x[u][1] = v.y;
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * kPerRow;
                const float wk = __shfl_sync(0xffffffffu, w, k & 31);
                if (k < 32 && c + k < pieces) {   // weight 0 too: 0 * NaN is NaN
#pragma unroll
                    for (int e = 0; e < kPer; ++e) o[e] += wk * x[u][e];
                }
            }
        }
    }
    l = warp_sum(l);
    if (kPerRow > 1) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) s_o[sub][lane * kPer + e] = o[e];
        __syncthreads();
        if (sub != 0) return;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            o[e] = s_o[0][lane * kPer + e];
            for (int x = 1; x < kPerRow; ++x) o[e] += s_o[x][lane * kPer + e];
        }
    }
    const float inv = inverse(m, l);
    uint32_t h[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) h[e] = pack_half2(o[2 * e] * inv, o[2 * e + 1] * inv);
    uint32_t *dst = reinterpret_cast<uint32_t *>(g.out + static_cast<size_t>(row) * D) + lane * (kPer / 2);
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) dst[e] = h[e];
}

// CTAs that a stream launch may have, two partial results each: bounds the workspace.
constexpr int kMaxCtas = 152;

struct Plan {
    int mode, tile_rows, item_rows, row_tiles, min_tiles, ctas;
};

size_t header_bytes(long long slots) { return (static_cast<size_t>(slots) * 8 + 255) / 256 * 256; }

// How a call is cut, from the sizes that the host knows: the most keys and nodes there may be.  Where page
// table and compressed rows hold far more than the sessions do, the choice is that of the larger size
// (attn_r128_64x32 with room for eight times its tokens: the stream, 97 us against 52).
// Two row blocks per item (each K and V tile read once for 256 rows) when that leaves at least four
// key tiles per SM; else one, with its two sides on alternate tiles.  Stream or not: the smaller of
// the two costs, in key tiles: an item's fixed part counts 4, in a stream 6 (its pieces start and end
// anywhere), and the join 4.  Measured, stream against whole items: attn_full_4x64 172 / 385 us,
// attn_r128_1x16 17.7 / 19.3, attn_r128_64x32 90 / 53, attn_sel_16x16 45 / 32.
Plan make_plan(const AttnTreeArgs &a, int B, int num_sms) {
    Plan p{};
    const long long tokens = static_cast<long long>(a.kv.max_pages) * a.kv.page;
    const long long raw = (a.window < tokens ? a.window : tokens) + a.N + 2 * kRun;
    const long long comp = a.sel ? a.n_sel : (a.ratio > 0 ? (a.cap < tokens / a.ratio ? a.cap : tokens / a.ratio) + kMaxNodes : 0);
    const long long tiles = (raw + comp + kTK - 1) / kTK;
    const long long rows = static_cast<long long>(a.N) * a.H;
    if (a.sel) {
        p.tile_rows = kTK;
        p.item_rows = a.H;
    } else {
        const long long blocks = (rows + 2 * kTK - 1) / (2 * kTK) * B;
        p.tile_rows = p.item_rows = rows > kTK && blocks * tiles >= 4LL * num_sms ? 2 * kTK : kTK;
    }
    p.row_tiles = static_cast<int>((rows + p.item_rows - 1) / p.item_rows);
    p.min_tiles = p.tile_rows == kTK ? 2 : 1;
    const long long slots = static_cast<long long>(p.row_tiles) * B, units = slots * tiles;
    const long long whole = (slots + num_sms - 1) / num_sms * (tiles + 4);
    const long long sms = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    long long ctas = (units + p.min_tiles - 1) / p.min_tiles;
    if (ctas > sms) ctas = sms;
    const long long share = (units + ctas - 1) / ctas, stream = share + 6 * (share / tiles + 1) + 4;
    if (tiles > p.min_tiles && stream < whole) {
        p.mode = kStream;
        p.ctas = static_cast<int>(ctas);
    } else {
        p.mode = slots > num_sms ? kWalk : kDirect;
        p.ctas = static_cast<int>(slots < num_sms ? slots : num_sms);
    }
    return p;
}

template <int D, bool kSel>
cudaError_t launch_one(Args &g, int ctas, const Ctx &c) {
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(attn_tree_kernel<D, kSel>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(Layout<D, kSel>::bytes));
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch(attn_tree_kernel<D, kSel>, dim3(ctas), dim3(kThreads), (Layout<D, kSel>::bytes), c, 1, g);
}

}  // namespace

// The largest over the ways a call of these sizes may be cut: one or two row blocks, or a node.
size_t attn_tree_ws_bytes(int B, int N, int H, int D) {
    const long long rows = static_cast<long long>(N) * H, slots = (rows + (H < kTK ? H : kTK) - 1) / (H < kTK ? H : kTK) * B;
    return header_bytes(slots) + static_cast<size_t>(2 * kMaxCtas) * (rows > kTK ? 2 * kTK : kTK) * (static_cast<size_t>(D) * 4 + 8);
}

cudaError_t launch_attn_tree(const AttnTreeArgs &args, int B, const Ctx &c) {
    Args g{};
    g.a = args;
    AttnTreeArgs &a = g.a;
    a.scale_log2 = a.scale * kLog2e;
    const Plan p = make_plan(a, B, c.num_sms);
    const long long pool_rows = a.kv.n_pages * a.kv.page, comp_rows = a.ratio > 0 ? a.cap * B : 0;
    const int D = a.kv.D;
    const uint32_t comp_box = a.sel ? 1 : kRun;
    if (!tc::encode_map(&g.map_q, a.q, D, static_cast<long long>(B) * a.N * a.H, a.sel ? 64 : kTK) ||
        !tc::encode_map(&g.map_k, a.kv.k, D, pool_rows, kRun) || !tc::encode_map(&g.map_v, a.kv.v, D, pool_rows, kRun))
        return cudaErrorInvalidValue;
    if (a.ratio > 0 && (!tc::encode_map(&g.map_ck, a.comp_k, D, comp_rows, comp_box) ||
                        !tc::encode_map(&g.map_cv, a.comp_v, D, comp_rows, comp_box)))
        return cudaErrorInvalidValue;
    const long long slots = static_cast<long long>(p.row_tiles) * B;
    g.B = B;
    g.mode = p.mode;
    g.min_tiles = p.min_tiles;
    g.row_tiles = p.row_tiles;
    g.tile_rows = p.tile_rows;
    g.item_rows = p.item_rows;
    g.n_work = static_cast<int>(slots);
    g.h_mul = ((1u << 20) + static_cast<uint32_t>(a.H) - 1) / static_cast<uint32_t>(a.H);
    g.pool_oob = static_cast<int>(pool_rows);
    g.comp_oob = static_cast<int>(comp_rows);
    unsigned char *ws = static_cast<unsigned char *>(a.ws);
    const size_t part_rows = static_cast<size_t>(2 * p.ctas) * p.tile_rows;
    g.pieces = reinterpret_cast<int2 *>(ws);
    g.part = reinterpret_cast<float *>(ws + header_bytes(slots));
    g.part_ml = reinterpret_cast<float2 *>(ws + header_bytes(slots) + part_rows * D * 4);
    cudaError_t e = D == 128 ? (a.sel ? launch_one<128, true>(g, p.ctas, c) : launch_one<128, false>(g, p.ctas, c))
                             : (a.sel ? launch_one<64, true>(g, p.ctas, c) : launch_one<64, false>(g, p.ctas, c));
    if (e != cudaSuccess || p.mode != kStream) return e;
    const JoinArgs j{g.part, g.part_ml, g.pieces, a.kv, a.n_node, a.out, a.cap, B, a.N, a.H, a.ratio, p.row_tiles,
                     p.tile_rows, p.item_rows};
    const long long rows = static_cast<long long>(B) * a.N * a.H;
    if (p.ctas >= 8 * slots) {                           // eight pieces a row tile or more
        const dim3 grid(static_cast<unsigned>(rows));
        return D == 128 ? launch(combine_kernel<128, kJoinWarps>, grid, dim3(kJoinThreads), 0, c, 1, j)
                        : launch(combine_kernel<64, kJoinWarps>, grid, dim3(kJoinThreads), 0, c, 1, j);
    }
    const dim3 grid(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps));
    return D == 128 ? launch(combine_kernel<128, 1>, grid, dim3(kJoinThreads), 0, c, 1, j)
                    : launch(combine_kernel<64, 1>, grid, dim3(kJoinThreads), 0, c, 1, j);
}

}  // namespace ds4a
