// paged.cu -- the paged token cache: appending tokens with their position rotation.
//
// Append: token i of session s goes to slot len + i; its key and its query heads are
// rotated to its position p (len + i, or len + depth in a tree).  Rotation of the pair
// (x1, x2) with frequency f_j: (x1 c - x2 s, x1 s + x2 c), c = cos(p f_j), s = sin(p f_j).
//
// The angle is taken in turns as a 64-bit fraction: p times floor(f_j / 2 pi * 2^64),
// modulo 2^64, is the angle modulo one turn, so whole turns drop out of the integer
// product exactly.  f_j / 2 pi is computed in double (2^-53 relative), so at position
// 2^31 and f = 1 the angle is within 2^-24 turns of the true one and at 2^20 within 2^-35;
// sine and cosine are then taken in binary32 of the half-turns.
#include "paged_dev.cuh"

namespace ds4a {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kItems = 3;       // work items a thread, all loaded before the first is stored
constexpr int kMaxTokens = 16;  // tokens of one CTA
constexpr int kMaxPairs = 64;   // rotated pairs: head_dim / 2

// x modulo 1 as a fraction of 2^64: the significand shifted to its place, whole turns and what is
// below 2^-64 dropped.  (binary64 units are few: floor, subtraction, product and conversion in
// binary64 took 0.4 us of a 2048-token chunk.)
DS4A_DEVINL unsigned long long turn_fraction(double x) {
    const long long b = __double_as_longlong(x);
    const int shift = static_cast<int>((b >> 52) & 0x7ff) - 1075 + 64;      // x = significand * 2^(shift - 64)
    const unsigned long long m = (static_cast<unsigned long long>(b) & 0xfffffffffffffull) | 0x10000000000000ull;
    unsigned long long f = 0;
    if (shift >= 0 && shift < 64) f = m << shift;
    else if (shift < 0 && shift > -64) f = m >> -shift;
    return b < 0 ? 0ull - f : f;
}

// A CTA takes t_cta consecutive tokens of a session.  A token's rows are its query heads, its
// key and its value; a row is D / 16 items of 32 bytes: unit u of the rotated dims holds the 8
// pairs 8u .. 8u+7 (two adjacent 16-byte chunks when interleaved, chunks u and u + rot/16
// otherwise), the other items two of the remaining chunks.  Bound by memory: a 2048-token
// chunk with 64 heads moves 69 MB in 13.4 us with its inputs in L2 (5.2 TB/s) and in 17 us with inputs
// from DRAM (4.0 TB/s: 2048 CTAs of one token, about five to an SM, are 2.7 waves, and inside a CTA
// loads, look-ups and stores follow one another); one token takes 3.4 us, a launch and three dependent
// loads.  Two or six items a thread instead of
// three: 14.3 and 19 us.  The inputs do not depend on the session's counts, so a
// thread's loads are in flight while length, angle and page are looked up.
template <bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(AppendArgs a, int t_cta, int d_shift) {
    __shared__ __align__(16) float2 s_cs[kMaxTokens][kMaxPairs];
    __shared__ unsigned long long s_mask[kMaxNodes];
    __shared__ int s_ptr[kMaxNodes];
    __shared__ long long s_row[kMaxTokens];
    const int tid = threadIdx.x, i0 = blockIdx.x * t_cta, s = blockIdx.y;
    const int rot = a.rot, D = a.kv.D, units = rot / 16, rows = a.H + 2;
    const int n_items = t_cta * rows << d_shift;
    const long long tok0 = static_cast<long long>(s) * a.N + i0;
    pdl_wait();
    pdl_trigger();
    struct Item {
        int tt, row, u, o1, o2;   // token, row (heads, then key, then value), unit (-1: copied), the two chunks
    };
    auto item = [&](int k) {
        const int w = tid + k * blockDim.x;
        Item t;
        const int r = w >> d_shift, c = w & ((1 << d_shift) - 1);
        t.tt = r / rows;
        t.row = r - t.tt * rows;
        if (w >= n_items || i0 + t.tt >= a.N) t.tt = -1;
        if (t.row == a.H + 1 || c >= units) {
            t.u = -1;
            const int base = t.row == a.H + 1 ? c * 16 : (c - units) * 16;
            t.o1 = base;
            t.o2 = base + 8;
            if (t.row <= a.H) {
                if (t.o1 >= a.rot_off) t.o1 += rot;
                if (t.o2 >= a.rot_off) t.o2 += rot;
            }
        } else {
            t.u = c;
            t.o1 = a.rot_off + (kInterleaved ? c * 16 : c * 8);
            t.o2 = kInterleaved ? t.o1 + 8 : t.o1 + rot / 2;
        }
        return t;
    };
    uint4 x1[kItems], x2[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const Item t = item(k);
        if (t.tt < 0) continue;
        const long long tok = tok0 + t.tt;
        const uint16_t *src = t.row < a.H ? a.q + (tok * a.H + t.row) * D : (t.row == a.H ? a.k : a.v) + tok * D;
        x1[k] = *reinterpret_cast<const uint4 *>(src + t.o1);
        x2[k] = *reinterpret_cast<const uint4 *>(src + t.o2);
    }
    const Session ses = load_session(a.kv, a.n_tok, a.N, s, tid == 0 ? a.err : nullptr);
    if (!ses.ok || i0 >= ses.n) return;
    if (a.parent && !tree_masks(a.parent + static_cast<long long>(s) * a.N, ses.n, s_mask, s_ptr, a.err)) return;
    const int count = min(t_cta, ses.n - i0);
    if (tid < count)
        s_row[tid] = pool_row(a.kv, a.kv.table + static_cast<long long>(s) * a.kv.max_pages,
                              static_cast<unsigned>(ses.len + i0 + tid), a.err);
    for (int w = tid; w < count * (rot / 2); w += blockDim.x) {
        const int tt = w / (rot / 2), j = w - tt * (rot / 2);
        const long long pos = ses.len + (a.parent ? __popcll(s_mask[i0 + tt]) - 1 : i0 + tt);
        const unsigned long long step = turn_fraction(static_cast<double>(a.inv_freq[j]) * 0.15915494309189533577);   // 1 / (2 pi)
        const int ang = static_cast<int>((step * static_cast<unsigned long long>(pos)) >> 32);
        float sn, cs;
        sincospif(static_cast<float>(ang) * 4.656612873077392578125e-10f, &sn, &cs);   // half-turns: 2^-31
        s_cs[tt][j] = make_float2(cs, sn);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const Item t = item(k);
        if (t.tt < 0 || t.tt >= count) continue;
        const long long tok = tok0 + t.tt;
        uint16_t *dst;
        if (t.row < a.H) {
            dst = a.q_out + (tok * a.H + t.row) * D;
        } else {
            if (s_row[t.tt] < 0) continue;
            dst = (t.row == a.H ? a.kv.k : a.kv.v) + s_row[t.tt] * D;
        }
        if (t.u >= 0) {
            const float4 *cs4 = reinterpret_cast<const float4 *>(&s_cs[t.tt][t.u * 8]);
            uint32_t w[8] = {x1[k].x, x1[k].y, x1[k].z, x1[k].w, x2[k].x, x2[k].y, x2[k].z, x2[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 cs = cs4[e];   // cos, sin of pairs 2e and 2e + 1
                if (kInterleaved) {
                    const float2 p = unpack_half2(w[2 * e]), q = unpack_half2(w[2 * e + 1]);
                    w[2 * e] = pack_half2(p.x * cs.x - p.y * cs.y, p.x * cs.y + p.y * cs.x);
                    w[2 * e + 1] = pack_half2(q.x * cs.z - q.y * cs.w, q.x * cs.w + q.y * cs.z);
                } else {
                    const float2 p = unpack_half2(w[e]), q = unpack_half2(w[e + 4]);
                    w[e] = pack_half2(p.x * cs.x - q.x * cs.y, p.y * cs.z - q.y * cs.w);
                    w[e + 4] = pack_half2(p.x * cs.y + q.x * cs.x, p.y * cs.w + q.y * cs.z);
                }
            }
            x1[k] = make_uint4(w[0], w[1], w[2], w[3]);
            x2[k] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        *reinterpret_cast<uint4 *>(dst + t.o1) = x1[k];
        *reinterpret_cast<uint4 *>(dst + t.o2) = x2[k];
    }
}

// ---- append with norms ------------------------------------------------------------------------

DS4A_DEVINL void unpack8(const uint4 x, float *f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = unpack_half2(w[e]);
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
    }
}
DS4A_DEVINL uint4 pack8(const float *f) {
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}
DS4A_DEVINL void turn(float &x, float &y, const float2 cs) {
    const float x0 = x, y0 = y;
    x = x0 * cs.x - y0 * cs.y;
    y = x0 * cs.y + y0 * cs.x;
}

// Depth of node i in a session's tree of n <= 64 nodes, by one warp (two nodes a lane, pointer jumping over
// shuffles); -1 (recorded) if a parent is not an earlier node or -1.
DS4A_DEVINL int node_depth(const int32_t *parent, int n, int i, int lane, unsigned int *err) {
    int p[2], d[2];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = lane + 32 * x;
        p[x] = j < n ? __ldg(parent + j) : -1;
        bad |= p[x] < -1 || p[x] >= j;
        d[x] = p[x] >= 0;                                        // ancestors counted so far; p: the next one
    }
    if (__any_sync(0xffffffffu, bad)) {
        record_error(err, DS4A_ERR_DEVICE_INDEX);
        return -1;
    }
    for (int span = 1; span < n; span *= 2) {
        int np[2], nd[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int src = p[x] & 31;
            const int p0 = __shfl_sync(0xffffffffu, p[0], src), p1 = __shfl_sync(0xffffffffu, p[1], src);
            const int d0 = __shfl_sync(0xffffffffu, d[0], src), d1 = __shfl_sync(0xffffffffu, d[1], src);
            np[x] = p[x] < 0 ? -1 : (p[x] < 32 ? p0 : p1);
            nd[x] = p[x] < 0 ? d[x] : d[x] + (p[x] < 32 ? d0 : d1);
        }
        p[0] = np[0];
        p[1] = np[1];
        d[0] = nd[0];
        d[1] = nd[1];
    }
    const int a = __shfl_sync(0xffffffffu, d[0], i & 31), b = __shfl_sync(0xffffffffu, d[1], i & 31);
    return i < 32 ? a : b;
}

// A warp takes up to kNormIt x 4 (D = 64: x 8) rows of one token: its query heads, its key, its value.
// A row is D / 16 neighbouring lanes of 16 values each, the two chunks of the items above, so a lane has
// the same pairs in every row: their sines, cosines (each taken by one of the lanes that need it) and
// weights stay in registers, a row's sum of squares is three (two) shuffles, and no warp waits for another.
// The norm, x / sqrt(mean(x^2) + eps) * w in binary32, is applied to what the rotation reads; nothing is rounded
// between them.  All loads but the page number go out together (with the session's counts ahead of the others a
// 2048-token chunk took 24 us).
//
// Measured: anorm_2048 (64 heads, 69 MB) 15.7 us with inputs in L2 = 4.4 TB/s, 17.7 from HBM; one token 2.9 us.
// No unit is used up (issue slots 60%, 17 of 20 warps resident): a warp loads once, waits, and stores, and the time is
// linear in the tokens, without a step where a round of blocks is full (1520 tokens 11.6 us, 1900 14.0, 2026, four
// rounds, 14.9, 2028 14.9, 2200 16.2).  With the norm in the block kernel above, its cosines and weights read
// from shared memory by 8 lanes 64 bytes apart, the chunk took 22.7 us; six iterations a warp at four blocks an
// SM take 16.7, three at six blocks 16.7.
constexpr int kNormIt = 3;
constexpr int kNormThreads = 128;
constexpr int kNormBlocks = 5;             // an SM: 96 registers a thread
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks) norm_append_kernel(const NormAppendArgs a, int warps_tok, int rows_warp) {
    constexpr int kLanes = D / 16, kRowsIt = 32 / kLanes;
    const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
    const unsigned gw = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5), ui = gw / static_cast<unsigned>(warps_tok);
    const int s = blockIdx.y, row0 = static_cast<int>(gw - ui * warps_tok) * rows_warp;
    const int rot = a.rot, units = rot / 16, rows = min(row0 + rows_warp, a.H + 2);
    pdl_wait();
    pdl_trigger();
    if (ui >= static_cast<unsigned>(a.N)) return;
    const int i = static_cast<int>(ui);
    const long long tok = static_cast<long long>(s) * a.N + i;
    // this lane's two chunks of 8 values: a unit of the rotated dims, or two of the others
    int o1, o2;
    if (c < units) {
        o1 = a.rot_off + (kInterleaved ? c * 16 : c * 8);
        o2 = kInterleaved ? o1 + 8 : o1 + rot / 2;
    } else {
        o1 = (c - units) * 16;
        o2 = o1 + 8;
        if (o1 >= a.rot_off) o1 += rot;
        if (o2 >= a.rot_off) o2 += rot;
    }
    uint4 x1[kNormIt], x2[kNormIt];
#pragma unroll
    for (int it = 0; it < kNormIt; ++it) {
        const int row = row0 + it * kRowsIt + sub;
        x1[it] = x2[it] = make_uint4(0, 0, 0, 0);
        if (row >= rows) continue;
        const uint16_t *src = row < a.H ? a.q + (tok * a.H + row) * D : (row == a.H ? a.k : a.v) + tok * D;
        x1[it] = *reinterpret_cast<const uint4 *>(src + o1);
        x2[it] = *reinterpret_cast<const uint4 *>(src + o2);
    }
    // everything else that does not depend on the session's counts, so that one round of loads covers it
    const long long len = a.kv.len[s], pos0 = *(a.pos0 ? a.pos0 + s : a.kv.len + s);
    const int n = a.n_tok[s];
    constexpr int kPairs = 8 / kRowsIt > 0 ? 8 / kRowsIt : 1;   // pairs whose angle a lane takes; its row's lanes share them
    float freq[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) freq[e] = c < units ? __ldg(a.inv_freq + c * 8 + sub * kPairs + e) : 0.f;
    float wq[16];
    if (a.q_w && row0 < a.H) {
        const float *w1 = a.q_w + o1, *w2 = a.q_w + o2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            wq[e] = __ldg(w1 + e);
            wq[e + 8] = __ldg(w2 + e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) wq[e] = 1.f;
    }
    const Session ses = check_session(a.kv, len, n, a.N, lane == 0 ? a.err : nullptr);
    if (!ses.ok || i >= ses.n) return;
    if (pos0 < 0 || pos0 > 0x7fffffffLL - ses.n) {
        if (lane == 0) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
        return;
    }
    if (a.slot_pos && ses.len > a.slots - ses.n) {
        if (lane == 0) record_error(a.err, DS4A_ERR_CAPACITY);
        return;
    }
    const int depth = a.parent ? node_depth(a.parent + static_cast<long long>(s) * a.N, ses.n, i, lane, a.err) : i;
    if (depth < 0) return;
    const long long pos = pos0 + depth;
    long long dst_row = -1;                                      // of the key and the value
    if (rows > a.H) {
        dst_row = pool_row(a.kv, a.kv.table + static_cast<long long>(s) * a.kv.max_pages, static_cast<unsigned>(ses.len + i),
                           lane == 0 ? a.err : nullptr);
        if (row0 <= a.H && lane == 0 && dst_row >= 0 && a.slot_pos)
            a.slot_pos[static_cast<long long>(s) * a.slots + ses.len + i] = static_cast<int>(pos);
    }
    float2 cs[8], own[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
        const unsigned long long step = turn_fraction(static_cast<double>(freq[e]) * 0.15915494309189533577);   // 1 / (2 pi)
        const int ang = static_cast<int>((step * static_cast<unsigned long long>(pos)) >> 32);
        sincospif(static_cast<float>(ang) * 4.656612873077392578125e-10f, &own[e].y, &own[e].x);   // half-turns: 2^-31
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e].x = __shfl_sync(0xffffffffu, own[e % kPairs].x, e / kPairs * kLanes + c);
        cs[e].y = __shfl_sync(0xffffffffu, own[e % kPairs].y, e / kPairs * kLanes + c);
    }
#pragma unroll
    for (int it = 0; it < kNormIt; ++it) {
        const int row = row0 + it * kRowsIt + sub;
        float f[16];
        unpack8(x1[it], f);
        unpack8(x2[it], f + 8);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss += f[e] * f[e];
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (row >= rows) continue;
        if (row <= a.H) {
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
            if (row < a.H) {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = f[e] * r * wq[e];
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = f[e] * r * (a.k_w ? __ldg(a.k_w + (e < 8 ? o1 + e : o2 + e - 8)) : 1.f);
            }
            if (c < units) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {                    // pairs 8c + e
                    if (kInterleaved) turn(f[2 * e], f[2 * e + 1], cs[e]);
                    else turn(f[e], f[e + 8], cs[e]);
                }
            }
            x1[it] = pack8(f);
            x2[it] = pack8(f + 8);
        }
        uint16_t *dst;
        if (row < a.H) {
            dst = a.q_out + (tok * a.H + row) * D;
        } else {
            if (dst_row < 0) continue;
            dst = (row == a.H ? a.kv.k : a.kv.v) + dst_row * D;
        }
        *reinterpret_cast<uint4 *>(dst + o1) = x1[it];
        *reinterpret_cast<uint4 *>(dst + o2) = x2[it];
    }
}

}  // namespace

cudaError_t launch_norm_append(const NormAppendArgs &a, int B, const Ctx &c) {
    const int rows = a.H + 2, it = a.kv.D == 128 ? 4 : 8;        // rows an iteration
    const int warps = (rows + kNormIt * it - 1) / (kNormIt * it), per = ((rows + warps - 1) / warps + it - 1) / it * it;
    const long long total = static_cast<long long>(a.N) * warps;   // of a session: below 2^31 (its tokens fit its pages)
    const dim3 grid(static_cast<unsigned>((total + kNormThreads / 32 - 1) / (kNormThreads / 32)), static_cast<unsigned>(B)), block(kNormThreads);
    const auto kernel = a.kv.D == 128 ? (a.interleaved ? norm_append_kernel<128, true> : norm_append_kernel<128, false>)
                                      : (a.interleaved ? norm_append_kernel<64, true> : norm_append_kernel<64, false>);
    return launch(kernel, grid, block, 0, c, 1, a, warps, per);
}

cudaError_t launch_paged_append(const AppendArgs &a, int B, const Ctx &c) {
    // as many tokens a CTA as its threads have items for, but no fewer CTAs than SMs
    const int d_shift = a.kv.D == 128 ? 3 : 2;
    long long t = kItems * kAppendThreads / ((a.H + 2) << d_shift);
    const long long spread = (static_cast<long long>(a.N) * B + c.num_sms - 1) / c.num_sms;
    if (t > spread) t = spread;
    if (t > kMaxTokens) t = kMaxTokens;
    if (t < 1) t = 1;
    const dim3 grid(static_cast<unsigned>((a.N + t - 1) / t), static_cast<unsigned>(B));
    long long threads = ((t * (a.H + 2) << d_shift) + kItems - 1) / kItems;
    threads = threads <= 64 ? 64 : (threads + 31) / 32 * 32;
    const dim3 block(static_cast<unsigned>(threads));
    return a.interleaved ? launch(paged_append_kernel<true>, grid, block, 0, c, 1, a, static_cast<int>(t), d_shift)
                         : launch(paged_append_kernel<false>, grid, block, 0, c, 1, a, static_cast<int>(t), d_shift);
}

}  // namespace ds4a
