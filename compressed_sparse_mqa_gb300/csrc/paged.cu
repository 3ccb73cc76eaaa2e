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
//
// With norms (ds4a_paged_append_norm) a key or query row is first x / sqrt(mean(x^2) + eps) * w.  A row
// is 8 (D = 64: 4) neighbouring lanes, 16 values each, so its sum of squares is three (two) shuffles of
// values that the rotation has in registers anyway; nothing is rounded between norm and rotation.
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

DS4A_DEVINL void unpack8(const uint4 x, float *f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = unpack_half2(w[e]);
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
    }
}
DS4A_DEVINL void turn(float &x, float &y, float c, float s) {
    const float x0 = x, y0 = y;
    x = x0 * c - y0 * s;
    y = x0 * s + y0 * c;
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
template <bool kInterleaved, bool kNorm>
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
        if (kNorm) x1[k] = x2[k] = make_uint4(0, 0, 0, 0);
        if (t.tt < 0) continue;
        const long long tok = tok0 + t.tt;
        const uint16_t *src = t.row < a.H ? a.q + (tok * a.H + t.row) * D : (t.row == a.H ? a.k : a.v) + tok * D;
        x1[k] = *reinterpret_cast<const uint4 *>(src + t.o1);
        x2[k] = *reinterpret_cast<const uint4 *>(src + t.o2);
    }
    const Session ses = load_session(a.kv, a.n_tok, a.N, s, tid == 0 ? a.err : nullptr);
    if (!ses.ok || i0 >= ses.n) return;
    long long pos0 = ses.len;
    if (kNorm) {
        if (a.pos0) pos0 = a.pos0[s];
        if (pos0 < 0 || pos0 > 0x7fffffffLL - ses.n || (a.slot_pos && ses.len > a.slots - ses.n)) {
            if (tid == 0)
                record_error(a.err, pos0 < 0 || pos0 > 0x7fffffffLL - ses.n ? DS4A_ERR_DEVICE_INDEX : DS4A_ERR_CAPACITY);
            return;
        }
    }
    if (a.parent && !tree_masks(a.parent + static_cast<long long>(s) * a.N, ses.n, s_mask, s_ptr, a.err)) return;
    const int count = min(t_cta, ses.n - i0);
    if (tid < count) {
        s_row[tid] = pool_row(a.kv, a.kv.table + static_cast<long long>(s) * a.kv.max_pages,
                              static_cast<unsigned>(ses.len + i0 + tid), a.err);
        if (kNorm && a.slot_pos && s_row[tid] >= 0)
            a.slot_pos[static_cast<long long>(s) * a.slots + ses.len + i0 + tid] =
                static_cast<int>(pos0 + (a.parent ? __popcll(s_mask[i0 + tid]) - 1 : i0 + tid));
    }
    for (int w = tid; w < count * (rot / 2); w += blockDim.x) {
        const int tt = w / (rot / 2), j = w - tt * (rot / 2);
        const long long pos = pos0 + (a.parent ? __popcll(s_mask[i0 + tt]) - 1 : i0 + tt);
        const unsigned long long step = turn_fraction(static_cast<double>(a.inv_freq[j]) * 0.15915494309189533577);   // 1 / (2 pi)
        const int ang = static_cast<int>((step * static_cast<unsigned long long>(pos)) >> 32);
        float sn, cs;
        sincospif(static_cast<float>(ang) * 4.656612873077392578125e-10f, &sn, &cs);   // half-turns: 2^-31
        s_cs[tt][j] = make_float2(cs, sn);
    }
    __syncthreads();
    float r[kItems];                 // 1 / sqrt(mean(x^2) + eps) of the item's row
    if (kNorm) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            float ss = 0.f;
            const uint32_t w[8] = {x1[k].x, x1[k].y, x1[k].z, x1[k].w, x2[k].x, x2[k].y, x2[k].z, x2[k].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 p = unpack_half2(w[e]);
                ss += p.x * p.x + p.y * p.y;
            }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            if (d_shift == 3) ss += __shfl_xor_sync(0xffffffffu, ss, 4);
            r[k] = rsqrtf(ss / static_cast<float>(D) + a.eps);
        }
    }
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
        if (kNorm && t.row <= a.H) {
            const float *w = t.row < a.H ? a.q_w : a.k_w;
            float f[16];
            unpack8(x1[k], f);
            unpack8(x2[k], f + 8);
            if (w) {
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float *we = w + (e < 8 ? t.o1 + e : t.o2 + e - 8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[e + i] = f[e + i] * r[k] * __ldg(we + i);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] *= r[k];
            }
            if (t.u >= 0) {
                const float4 *cs4 = reinterpret_cast<const float4 *>(&s_cs[t.tt][t.u * 8]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 cs = cs4[e];   // cos, sin of pairs 2e and 2e + 1
                    if (kInterleaved) {
                        turn(f[4 * e], f[4 * e + 1], cs.x, cs.y);
                        turn(f[4 * e + 2], f[4 * e + 3], cs.z, cs.w);
                    } else {
                        turn(f[2 * e], f[2 * e + 8], cs.x, cs.y);
                        turn(f[2 * e + 1], f[2 * e + 9], cs.z, cs.w);
                    }
                }
            }
            x1[k] = make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
            x2[k] = make_uint4(pack_half2(f[8], f[9]), pack_half2(f[10], f[11]), pack_half2(f[12], f[13]),
                               pack_half2(f[14], f[15]));
        } else if (!kNorm && t.u >= 0) {
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

}  // namespace

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
    const auto kernel = a.norm ? (a.interleaved ? paged_append_kernel<true, true> : paged_append_kernel<false, true>)
                               : (a.interleaved ? paged_append_kernel<true, false> : paged_append_kernel<false, false>);
    return launch(kernel, grid, block, 0, c, 1, a, static_cast<int>(t), d_shift);
}

}  // namespace ds4a
