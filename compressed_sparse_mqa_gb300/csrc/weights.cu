// weights.cu -- the attention weight that every cached token gets, summed over heads and queries.
//
//   acc[t] = decay * acc[t] + sum over tokens i >= t - len and heads h of exp(scale q_ih . K_t - lse_ih)
//
// lse_ih is the row's log of the sum of exp, as the attention call left it, so one pass over K
// suffices.  The products put keys on the M side of tcgen05.mma and (token, head) rows on the N side:
// a thread then has one key and its scores against 64 rows in its own registers, sums them alone, and
// nothing is reduced across threads.  A key belongs to one thread of one CTA, which takes the rows in
// order: no atomics, the same sums every time.
//
// Work: all sessions' 128-key tiles in one line, cut evenly over the CTAs (one per SM).  A CTA takes two
// tiles at a time, one a side, and goes through the rows in chunks of 128, 64 in registers at a time.
// Roles:
//   warps 0-3, 4-7  side 0 / 1: thread = key.
//   warp 8       set-up: the CTA's pieces of the line; query chunks (TMA) and their lse.
//   warp 9       MMA issuer.
//   warp 10      K producer: a tile is boxes of as many rows as divide a page (16 .. 128).
// Measured: weights_64x1 (64 sessions of 29 - 33 thousand keys, one token each) 84 us = 6.2 TB/s, bound by reading
// K from HBM; weights_5x33_d64 (some 790 rows over 200 tiles) 14.8 us: a CTA with seven chunks takes 23000 cycles, 5900 to its
// first scores, 1600 waiting for later scores, at most 1900 for queries, and the rest, some 2000 a chunk, in the sides'
// loads and sums of scores (a fused multiply-add, a power of two and a sum for each, two warps a scheduler); a third of
// the SMs have no tiles.  weights_1x1 (one session, 33 tiles) 4.9 us, a launch and three dependent loads.  Branches on
// the mask inside the 64-row loop cost 91 in place of 85 us.
#include "line.cuh"
#include "paged_dev.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace ds4a {
namespace {

constexpr int kTK = 128;                   // keys per tile
constexpr int kRows = 128;                 // rows per chunk
constexpr int kHalf = 64;                  // rows that a thread has in its registers at a time
constexpr int kNS = 4;                     // K stages, a tile each
constexpr int kQS = 2;                     // query stages, a chunk each
constexpr int kSideWarps = 4, kSoftWarps = 2 * kSideWarps;
constexpr int kSetupWarp = kSoftWarps, kMmaWarp = kSetupWarp + 1, kProdWarp = kMmaWarp + 1;
constexpr int kWarps = kProdWarp + 1, kThreads = 32 * kWarps;
constexpr uint32_t kTmemCols = 512;        // [side][buffer][kRows]
constexpr uint64_t kWaitNs = 10000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kInfo = 16;                  // tiles whose box information is kept: four and the K stages, and a power of two

struct Piece {
    int s, len, n, rows;                   // session; cached and new tokens; rows (n * H)
    int tile0, tile1;
    int stop;
};

struct Bars {
    uint64_t k_full[kNS], k_empty[kNS], q_full[kQS], q_empty[kQS];
    uint64_t s_full[2][2], s_empty[2][2];
    uint64_t w_full[2], w_empty[2];
};

template <int D>
struct Layout {
    static constexpr int tile = kTK * D * 2, chunk = kRows * D * 2;
    static constexpr int k = 0;
    static constexpr int q = k + kNS * tile;
    static constexpr int lse = q + kQS * chunk;              // float [kQS][kRows], in log2 units, negative; kDead
    static constexpr int info = lse + kQS * kRows * 4;       // uint8 [kInfo]: readable eighths (16 keys) of a tile
    static constexpr int dead = info + kInfo;                // int [kQS]: a chunk has rows of kDead
    static constexpr int work = dead + kQS * 4;
    static constexpr int bars = work + 64;
    static constexpr int end = bars + static_cast<int>(sizeof(Bars));
    static constexpr size_t bytes = end + 1024;
    static_assert(kInfo >= 4 + kNS && (kInfo & (kInfo - 1)) == 0, "box information");
    static_assert(2 * sizeof(Piece) <= 64 && dead % 4 == 0 && work % 8 == 0 && bars % 8 == 0 && lse % 16 == 0, "layout");
    static_assert(bytes <= 227 * 1024, "shared memory");
};

struct Args {
    CUtensorMap map_q, map_k;              // kRows-row boxes; `box`-row boxes over the pool
    AttnWeightsArgs a;
    float scale_log2;
    int B, box, pool_oob, pair;            // pair: 1 where the line's units are two tiles
};

DS4A_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Adds a key's weights from half a chunk's rows: 2^(score * c2 + l4[row]); kMask: of rows lo .. hi-1 alone.
template <bool kMask>
DS4A_DEVINL void add_weights(const uint32_t (&x)[2][32], const float4 *l4, uint64_t c2, int lo, int hi, uint64_t (&sum)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 m = l4[(h * 32 + e) / 4];
            float p[4];
            tc::unpack2(tc::fma2(tc::pack2(__uint_as_float(x[h][e]), __uint_as_float(x[h][e + 1])), c2, tc::pack2(m.x, m.y)), p[0], p[1]);
            tc::unpack2(tc::fma2(tc::pack2(__uint_as_float(x[h][e + 2]), __uint_as_float(x[h][e + 3])), c2, tc::pack2(m.z, m.w)), p[2], p[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = ex2(p[i]);
                if (kMask && (h * 32 + e + i < lo || h * 32 + e + i >= hi)) p[i] = 0.f;
            }
            sum[(e / 4) & 1] = tc::add2(sum[(e / 4) & 1], tc::pack2(p[0], p[1]));
            sum[2 + ((e / 4) & 1)] = tc::add2(sum[2 + ((e / 4) & 1)], tc::pack2(p[2], p[3]));
        }
}

// The same of 16 rows, lo .. hi-1 of them, in chunks that have rows whose lse is -inf: those add nothing, even where their
// scores are NaN or infinite.  (The sums of other chunks stay as they are and this code small: as a condition of the masked sum
// weights_5x33_d64 took 17.2 us, here with 32 rows at a time 15.4, with 16 15.0 as without.)
constexpr float kDead = -3.402823466e38f;   // such a row's l4 (no other row's, short of an lse of 2.3e38)
DS4A_DEVINL void add_live(const uint32_t (&x)[16], const float *l, uint64_t c2, int lo, int hi, uint64_t &sum) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        float p[2];
        tc::unpack2(tc::fma2(tc::pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, tc::pack2(l[e], l[e + 1])), p[0], p[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) p[i] = e + i < lo || e + i >= hi || l[e + i] == kDead ? 0.f : ex2(p[i]);
        sum = tc::add2(sum, tc::pack2(p[0], p[1]));
    }
}

// A session's tokens and key tiles; a session that must be left alone has none.
struct Tiles {
    int len, n, tiles;
};
DS4A_DEVINL Tiles session_tiles(const AttnWeightsArgs &a, int s) {
    const Session ses = load_session(a.kv, a.n_tok, a.N, s, a.err);
    Tiles t{0, 0, 0};
    if (!ses.ok || ses.n == 0) return t;
    if (ses.len > a.slots - ses.n) {
        record_error(a.err, DS4A_ERR_CAPACITY);
        return t;
    }
    t.len = static_cast<int>(ses.len);
    t.n = ses.n;
    t.tiles = (t.len + t.n - 1) / kTK + 1;
    return t;
}

// The line's units: pairs of tiles, which take the time of one, where the rows are more than a chunk; single tiles where
// reading K is all the time (weights_1x1, 33 tiles: 5.0 us in single tiles, 5.4 in pairs).
DS4A_DEVINL int units_of(const Args &g, const Tiles &t) { return (t.tiles + (1 << g.pair) - 1) >> g.pair; }

// 33 to kTable sessions are looked up and laid end to end by all threads at once, before the roles part: one round of
// loads, where the set-up warp's walk of 64 sessions took 8000 cycles to the first scores.  (Up to 32 are one round of the
// walk's, which needs no barriers: 0.4 us less.)
constexpr int kTable = 256;
static_assert(kTable <= kThreads, "a thread per session");
struct SessionTable {
    int4 session[kTable];                  // cached tokens, new tokens, tiles
    long long incl[kTable];                // units up to and with the session
    long long warp_units[kTable / 32];
    int first;                             // session of this CTA's first unit
};
DS4A_DEVINL void line_share(long long total, long long &u, long long &end) {
    const int ctas = static_cast<int>(total < gridDim.x ? total : gridDim.x), c = blockIdx.x;
    u = c < ctas ? line_quot(total * c, ctas) : 0;
    end = c < ctas ? line_quot(total * (c + 1), ctas) : 0;
}
DS4A_DEVINL void fill_table(const Args &g, SessionTable &t) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tiles s = tid < g.B ? session_tiles(g.a, tid) : Tiles{0, 0, 0};
    const int own = units_of(g, s);
    long long incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31 && warp < kTable / 32) t.warp_units[warp] = incl;
    __syncthreads();
    long long total = 0, u, end;
#pragma unroll
    for (int x = 0; x < kTable / 32; ++x) {
        if (x == warp) incl += total;
        total += t.warp_units[x];
    }
    if (tid < g.B) {
        t.session[tid] = make_int4(s.len, s.n, s.tiles, 0);
        t.incl[tid] = incl;
        line_share(total, u, end);
        if (u >= incl - own && u < incl) t.first = tid;
    }
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_weights_kernel(const __grid_constant__ Args g) {
    using L = Layout<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *s_lse = reinterpret_cast<float *>(smem + L::lse);
    volatile uint8_t *info = smem + L::info;
    int *s_dead = reinterpret_cast<int *>(smem + L::dead);
    Piece *pieces = reinterpret_cast<Piece *>(smem + L::work);
    Bars &bar = *reinterpret_cast<Bars *>(smem + L::bars);
    __shared__ uint32_t s_tmem;
    const AttnWeightsArgs &a = g.a;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int kAtoms = D / 64, kAtomBytes = kTK * 128;

    if (tid == 0) {
        for (int x = 0; x < kNS; ++x) {
            tc::mbar_init(&bar.k_full[x], 1);
            tc::mbar_init(&bar.k_empty[x], 1);
        }
        for (int x = 0; x < kQS; ++x) {
            tc::mbar_init(&bar.q_full[x], 2);                     // the queries, their lse
            tc::mbar_init(&bar.q_empty[x], kSoftWarps + 1);
        }
        for (int x = 0; x < 2; ++x) {
            for (int y = 0; y < 2; ++y) {
                tc::mbar_init(&bar.s_full[x][y], 1);
                tc::mbar_init(&bar.s_empty[x][y], kSideWarps);
            }
            tc::mbar_init(&bar.w_full[x], 1);
            tc::mbar_init(&bar.w_empty[x], kWarps - 1);
        }
        tc::mbar_fence_init();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&s_tmem, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    pdl_wait();
    pdl_trigger();
    __shared__ SessionTable s_table;
    const bool table = g.B > 32 && g.B <= kTable;
    if (table) fill_table(g, s_table);
    bool ok = true;
    // a failed wait records the failure; later waits of this thread return at once
    auto wait = [&](uint64_t *b, uint32_t parity) {
        if (ok && !tc::mbar_wait(b, parity & 1u, kWaitNs)) ok = false;
        return ok;
    };
    auto warp_wait = [&](uint64_t *b, uint32_t parity) {
        ok = __all_sync(0xffffffffu, wait(b, parity));
        return ok;
    };
    // A chunk is loaded once for a piece when it is the only one, else once for every block of two tiles.
    if (warp < kSoftWarps) {
        const int side = warp / kSideWarps, quad = warp & 3;
        const uint32_t col0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + side * 2 * kRows;
        const uint64_t c2 = tc::pack2(g.scale_log2, g.scale_log2);
        uint32_t n_c = 0, n_q = 0, n_t = 0;                       // this side's chunks; query loads; tiles so far
        for (int it = 0;; ++it) {
            const Piece &w = pieces[it & 1];
            if (!warp_wait(&bar.w_full[it & 1], it >> 1) || w.stop) break;
            const int tiles = w.tile1 - w.tile0, rows = w.rows, len = w.len;
            const int chunks = (rows + kRows - 1) / kRows;
            float *acc = a.acc + static_cast<long long>(w.s) * a.slots;
            // the sums before, loaded two tiles ahead of their use (under a full memory system a load takes longer
            // than the two tiles)
            auto old_sum = [&](int b) {
                const unsigned key = static_cast<unsigned>(w.tile0 + b + side) * kTK + quad * 32 + lane;
                return b + side < tiles && key < static_cast<unsigned>(len) && a.decay != 0.f ? acc[key] : 0.f;
            };
            float old_next = old_sum(0);
            for (int b = 0; b < tiles; b += 2) {
                const bool mine = b + side < tiles;
                const unsigned key = static_cast<unsigned>(w.tile0 + b + side) * kTK + quad * 32 + lane;   // below 2^31 + 2^9
                const unsigned end = static_cast<unsigned>(len) + w.n;
                const int behind = static_cast<int>(key) - len;                     // its new token's number, or negative
                const int row0 = behind > 0 && key < end ? behind * a.H : 0;        // first row that attends the key
                const float old = old_next;
                old_next = old_sum(b + 2);
                bool readable = false;
                uint64_t sum[4] = {0, 0, 0, 0};
                for (int c = 0; c < chunks; ++c) {
                    const bool loaded = chunks > 1 || b == 0, last_use = chunks > 1 || b + 2 >= tiles;
                    const uint32_t st = n_q % kQS;
                    if (loaded) warp_wait(&bar.q_full[st], n_q / kQS);
                    if (mine) {
                        const uint32_t sb = n_c & 1u;
                        const int dead = s_dead[st];
                        wait(&bar.s_full[side][sb], n_c >> 1);
                        tc::fence_after_sync();
                        // read before the scores are given back: the slot is written again kInfo tiles on, when the
                        // products of the tile four on are done, and those wait for these scores to be given back
                        if (c == 0) readable = (info[(n_t + b + side) & (kInfo - 1)] >> (quad * 2 + lane / 16)) & 1;
                        if (!__any_sync(0xffffffffu, dead)) {
#pragma unroll 1
                            for (int h = 0; h < 2; ++h) {
                                const int lo = row0 - c * kRows - h * kHalf, hi = rows - c * kRows - h * kHalf;   // rows of the half
                                uint32_t x[2][32];
                                if (hi > 0) {
                                    tc::ld_x32(col0 + sb * kRows + h * kHalf, x[0]);
                                    tc::ld_x32(col0 + sb * kRows + h * kHalf + 32, x[1]);
                                    tc::wait_ld();
                                }
                                if (h == 1) {
                                    tc::fence_before_sync();
                                    __syncwarp();
                                    if (lane == 0) tc::mbar_arrive(&bar.s_empty[side][sb]);
                                }
                                if (hi <= 0) break;
                                const float4 *l4 = reinterpret_cast<const float4 *>(s_lse + st * kRows + h * kHalf);
                                if (__all_sync(0xffffffffu, lo <= 0 && hi >= kHalf)) add_weights<false>(x, l4, c2, lo, hi, sum);
                                else add_weights<true>(x, l4, c2, lo, hi, sum);
                            }
                        } else {
#pragma unroll 1
                            for (int h = 0; h < kRows; h += 16) {
                                const int lo = row0 - c * kRows - h, hi = rows - c * kRows - h;
                                uint32_t x[16];
                                if (hi > 0) {
                                    tc::ld_x16(col0 + sb * kRows + h, x);
                                    tc::wait_ld();
                                    add_live(x, s_lse + st * kRows + h, c2, lo, hi, sum[0]);
                                }
                            }
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&bar.s_empty[side][sb]);
                        }
                        ++n_c;
                    }
                    __syncwarp();
                    if (last_use) {
                        if (lane == 0) tc::mbar_arrive(&bar.q_empty[st]);
                        ++n_q;
                    }
                }
                if (readable && key < end) {
                    float p0, p1;
                    tc::unpack2(tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3])), p0, p1);
                    acc[key] = a.decay * old + (p0 + p1);
                }
            }
            n_t += tiles;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.w_empty[it & 1]);
        }
    } else if (warp == kSetupWarp) {
        Line line{};
        auto units = [&](int s) { return static_cast<long long>(units_of(g, session_tiles(a, s))); };
        if (lane == 0) tc::prefetch_map(&g.map_q);
        long long u, u_end;
        line_share(table ? s_table.incl[g.B - 1] : line_total(line, g.B, units), u, u_end);
        int cursor = table ? s_table.first : 0;
        uint32_t n_q = 0;
        for (int it = 0;; ++it) {
            if (it >= 2 && !warp_wait(&bar.w_empty[it & 1], (it >> 1) - 1)) break;
            Piece &w = pieces[it & 1];
            int s = -1;                                           // the session of unit u, and its first unit
            long long at = 0;
            Tiles t{0, 0, 0};
            if (u < u_end && table) {
                while (s_table.incl[cursor] <= u) ++cursor;
                s = cursor;
                at = s > 0 ? s_table.incl[s - 1] : 0;
                t = Tiles{s_table.session[s].x, s_table.session[s].y, s_table.session[s].z};
            } else if (u < u_end) {
                const int l = line_to(line, g.B, u, units);
                if (l >= 0) {
                    s = line.first + l;
                    at = line.before + __shfl_sync(0xffffffffu, line.incl - line.mine, l);
                    t = session_tiles(a, s);
                }
            }
            const long long end = at + units_of(g, t) < u_end ? at + units_of(g, t) : u_end;
            const int tile0 = static_cast<int>(u - at) << g.pair;
            const int tile1 = static_cast<int>(min((end - at) << g.pair, static_cast<long long>(t.tiles)));
            const int rows = t.n * a.H, chunks = (rows + kRows - 1) / kRows;
            if (lane == 0) w = Piece{s, t.len, t.n, rows, tile0, tile1, s < 0};
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.w_full[it & 1]);
            if (s < 0) break;
            u = end;
            const int loads = chunks > 1 ? (tile1 - tile0 + 1) / 2 : 1;
            const long long row0 = static_cast<long long>(s) * a.N * a.H;
            // rows behind the last are masked
            auto lse_of = [&](int r) { return r < rows ? __ldg(a.lse + row0 + r) : INFINITY; };
            auto scaled = [](float v) { return v == -INFINITY ? kDead : -v * kLog2e; };
            float next[kRows / 32];                               // of the next chunk, loaded while this one waits
#pragma unroll
            for (int i = 0; i < kRows / 32; ++i) next[i] = lse_of(i * 32 + lane);
            for (int x = 0; x < loads && ok; ++x)
                for (int ch = 0; ch < chunks && ok; ++ch, ++n_q) {
                    const uint32_t st = n_q % kQS;
                    float m[kRows / 32];
                    const int after = ch + 1 < chunks ? (ch + 1) * kRows : 0;
#pragma unroll
                    for (int i = 0; i < kRows / 32; ++i) {
                        m[i] = next[i];
                        next[i] = lse_of(after + i * 32 + lane);
                    }
                    const bool dead = __any_sync(0xffffffffu, fminf(fminf(m[0], m[1]), fminf(m[2], m[3])) == -INFINITY);
                    if (n_q >= kQS && !warp_wait(&bar.q_empty[st], n_q / kQS - 1)) break;
                    if (lane == 0) {
                        tc::expect_tx(&bar.q_full[st], L::chunk);
                        for (int at_ = 0; at_ < kAtoms; ++at_)
                            tc::tma_load_2d(smem + L::q + st * L::chunk + at_ * (kRows * 128), &g.map_q, at_ * 64,
                                            static_cast<int>(row0 + ch * kRows), &bar.q_full[st]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kRows / 32; ++i) s_lse[st * kRows + i * 32 + lane] = scaled(m[i]);
                    if (lane == 0) s_dead[st] = dead;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.q_full[st]);
                }
        }
        if (!ok && lane == 0) {                                   // a wait gave up: the copies in flight land first
            const uint32_t from = n_q > kQS ? n_q - kQS : 0;
            for (uint32_t x = from; x < n_q; ++x) tc::mbar_wait(&bar.q_full[x % kQS], (x / kQS) & 1u);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // all of a chunk's rows, or the first half where there are no more
        constexpr uint32_t kIdAll = tc::idesc_f16_f32(kTK, kRows, false, false), kIdHalf = tc::idesc_f16_f32(kTK, kHalf, false, false);
        const uint64_t k_d = tc::desc_sw128(tc::smem_u32(smem + L::k), 16, 1024);
        const uint64_t q_d = tc::desc_sw128(tc::smem_u32(smem + L::q), 16, 1024);
        uint32_t n_t = 0, n_q = 0, n_c[2] = {0, 0};
        for (int it = 0; ok; ++it) {
            const Piece &w = pieces[it & 1];
            if (!warp_wait(&bar.w_full[it & 1], it >> 1) || __shfl_sync(0xffffffffu, w.stop, 0)) break;
            const int tiles = __shfl_sync(0xffffffffu, w.tile1 - w.tile0, 0);
            const int rows = __shfl_sync(0xffffffffu, w.rows, 0), chunks = (rows + kRows - 1) / kRows;
            for (int b = 0; b < tiles && ok; b += 2) {
                for (int c = 0; c < chunks && ok; ++c) {
                    const uint32_t id = rows - c * kRows > kHalf ? kIdAll : kIdHalf;
                    const uint32_t qs = n_q % kQS;
                    bool good = true;
                    if (chunks > 1 || b == 0) good = wait(&bar.q_full[qs], n_q / kQS);
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        if (b + side >= tiles) continue;
                        const uint32_t t = n_t + b + side, ks = t % kNS, sb = n_c[side] & 1u;
                        if (c == 0) good = wait(&bar.k_full[ks], t / kNS) && good;
                        if (n_c[side] >= 2) good = wait(&bar.s_empty[side][sb], (n_c[side] >> 1) - 1) && good;
                        ok = __all_sync(0xffffffffu, good);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const uint64_t kd = k_d + ks * (L::tile / 16), qd = q_d + qs * (L::chunk / 16);
                        const uint32_t d = tmem + side * 2 * kRows + sb * kRows;
                        if (tc::elect()) {
#pragma unroll
                            for (int x = 0; x < D / 16; ++x)
                                tc::mma_f16(d, kd + (x / 4) * (kAtomBytes / 16) + (x % 4) * 2,
                                            qd + (x / 4) * (kRows * 128 / 16) + (x % 4) * 2, id, x > 0);
                            tc::commit(&bar.s_full[side][sb]);
                            if (c + 1 == chunks) tc::commit(&bar.k_empty[ks]);
                            if ((chunks > 1 || b + 2 >= tiles) && (side == 1 || b + 1 >= tiles)) tc::commit(&bar.q_empty[qs]);
                        }
                        __syncwarp();
                        ++n_c[side];
                    }
                    if (chunks > 1 || b + 2 >= tiles) ++n_q;
                }
            }
            n_t += tiles;
            if (lane == 0) tc::mbar_arrive(&bar.w_empty[it & 1]);
        }
        __syncwarp();
    } else {
        // ---------------- K producer: lane = box (and atom) ----------------
        const int boxes = kTK / g.box, box = lane % boxes, atom = lane / boxes;
        uint32_t n_t = 0;
        if (lane == 0) tc::prefetch_map(&g.map_k);
        for (int it = 0;; ++it) {
            const Piece &w = pieces[it & 1];
            if (!warp_wait(&bar.w_full[it & 1], it >> 1) || w.stop) break;
            const int tile0 = w.tile0, tile1 = w.tile1;
            const unsigned end = static_cast<unsigned>(w.len) + w.n;
            const int32_t *table = a.kv.table + static_cast<long long>(w.s) * a.kv.max_pages;
            for (int t = tile0; t < tile1; ++t, ++n_t) {
                const uint32_t st = n_t % kNS;
                const unsigned slot = static_cast<unsigned>(t) * kTK + box * g.box;
                int row = g.pool_oob;                            // boxes behind the last token load zeros
                bool readable = true;
                if (slot < end) {
                    const unsigned pg = slot / static_cast<unsigned>(a.kv.page);
                    const int id = __ldg(table + pg);
                    readable = id >= 0 && id < a.kv.n_pages;
                    if (readable) row = id * a.kv.page + static_cast<int>(slot - pg * a.kv.page);
                    else if (atom == 0) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
                }
                uint32_t bits = readable && atom == 0 ? ((1u << (g.box / 16)) - 1u) << (box * g.box / 16) : 0u;
                bits = __reduce_or_sync(0xffffffffu, bits);
                if (n_t >= kNS && !warp_wait(&bar.k_empty[st], n_t / kNS - 1)) break;
                if (lane == 0) {
                    info[n_t & (kInfo - 1)] = static_cast<uint8_t>(bits);
                    tc::expect_tx(&bar.k_full[st], L::tile);
                }
                __syncwarp();
                if (atom < kAtoms)
                    tc::tma_load_2d(tc::smem_u32(smem + L::k + st * L::tile) + atom * kAtomBytes + box * g.box * 128, &g.map_k,
                                    atom * 64, row, &bar.k_full[st]);
                __syncwarp();
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.w_empty[it & 1]);
        }
        if (!ok && lane == 0) {
            const uint32_t from = n_t > kNS ? n_t - kNS : 0;
            for (uint32_t x = from; x < n_t; ++x) tc::mbar_wait(&bar.k_full[x % kNS], (x / kNS) & 1u);
        }
        __syncwarp();
    }
    if (!ok) record_error(a.err, DS4A_ERR_TIMEOUT);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch_one(const Args &g, int ctas, const Ctx &c) {
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(attn_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(Layout<D>::bytes));
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch(attn_weights_kernel<D>, dim3(ctas), dim3(kThreads), (Layout<D>::bytes), c, 1, g);
}

}  // namespace

cudaError_t launch_attn_weights(const AttnWeightsArgs &a, int B, const Ctx &c) {
    Args g{};
    g.a = a;
    g.B = B;
    g.scale_log2 = a.scale * kLog2e;
    const int D = a.kv.D;
    const long long pool_rows = a.kv.n_pages * a.kv.page;
    g.box = a.kv.page & -a.kv.page;                              // rows that are consecutive in the pool wherever a tile is cut
    if (g.box > kTK) g.box = kTK;
    g.pool_oob = static_cast<int>(pool_rows);
    g.pair = a.N * a.H > kRows;
    if (!tc::encode_map(&g.map_q, a.q, D, static_cast<long long>(B) * a.N * a.H, kRows) ||
        !tc::encode_map(&g.map_k, a.kv.k, D, pool_rows, static_cast<uint32_t>(g.box)))
        return cudaErrorInvalidValue;
    // no more CTAs than tiles that the sessions can have
    const long long tokens = static_cast<long long>(a.kv.max_pages) * a.kv.page;
    const long long tiles = ((tokens < a.slots ? tokens : a.slots) / kTK + 1) * B;
    const int ctas = static_cast<int>(tiles < c.num_sms ? tiles : c.num_sms);
    return D == 128 ? launch_one<128>(g, ctas, c) : launch_one<64>(g, ctas, c);
}

}  // namespace ds4a
