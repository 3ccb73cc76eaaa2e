// paged.cu -- the paged token cache: appending tokens with their position rotation, and
// committing the accepted path of a draft.
//
// Append: token i of session s goes to slot len + i; its key and its query heads are
// rotated to its position p (len + i, or len + depth in a tree).  Rotation of the pair
// (x1, x2) with frequency f_j: (x1 c - x2 s, x1 s + x2 c), c = cos(p f_j), s = sin(p f_j).
//
// The angle is taken in turns as a 64-bit fraction: p times round(f_j / 2 pi * 2^64),
// modulo 2^64, is the angle modulo one turn, so whole turns drop out of the integer
// product exactly.  f_j / 2 pi is computed in double (2^-53 relative), so at position
// 2^31 and f = 1 the angle is within 2^-24 turns of the true one and at 2^20 within 2^-35;
// sine and cosine are then taken in binary32 of the half-turns.
#include "paged_dev.cuh"

namespace ds4a {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxPairs = 64;   // rotated pairs: head_dim / 2

// One CTA per token.  Work items, 16 bytes x 2 each: unit u of a head holds the 8 pairs
// 8u .. 8u+7 of its rotated dims (two adjacent 16-byte chunks when interleaved, chunks u
// and u + rot/16 otherwise); the dims outside the rotation and V are copied in 16-byte
// chunks.
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(AppendArgs a) {
    __shared__ float2 s_cs[kMaxPairs];
    __shared__ unsigned long long s_mask[kMaxNodes];
    __shared__ int s_ptr[kMaxNodes];
    const int tid = threadIdx.x, i = blockIdx.x, s = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    const Session ses = load_session(a.kv, a.n_tok, a.N, s, a.err);
    if (!ses.ok || i >= ses.n) return;
    long long pos = ses.len + i;
    if (a.parent) {
        if (!tree_masks(a.parent + static_cast<long long>(s) * a.N, ses.n, s_mask, s_ptr, a.err)) return;
        pos = ses.len + __popcll(s_mask[i]) - 1;
    }
    const int rot = a.rot, D = a.kv.D;
    if (tid < rot / 2) {
        const double turns = static_cast<double>(a.inv_freq[tid]) * 0.15915494309189533577;   // 1 / (2 pi)
        const double frac = turns - floor(turns);
        const unsigned long long step = __double2ull_rn(frac * 18446744073709551616.0);
        const int ang = static_cast<int>((step * static_cast<unsigned long long>(pos)) >> 32);
        float sn, cs;
        sincospif(static_cast<float>(ang) * 4.656612873077392578125e-10f, &sn, &cs);   // half-turns: 2^-31
        s_cs[tid] = make_float2(cs, sn);
    }
    __syncthreads();
    const long long row = pool_row(a.kv, a.kv.table + static_cast<long long>(s) * a.kv.max_pages,
                                   static_cast<unsigned>(ses.len + i), a.err);
    const long long tok = static_cast<long long>(s) * a.N + i;
    const int units = rot / 16, plain = (D - rot) / 8;
    const int heads = (a.q ? a.H : 0) + 1;               // the key is the last head
    const int per_head = units + plain;
    auto head_ptrs = [&](int h, const uint16_t *&src, uint16_t *&dst) {
        if (h == heads - 1) {
            src = a.k + tok * D;
            dst = row >= 0 ? a.kv.k + row * D : nullptr;
        } else {
            src = a.q + (tok * a.H + h) * D;
            dst = a.q_out + (tok * a.H + h) * D;
        }
    };
    for (int w = tid; w < heads * per_head; w += kAppendThreads) {
        const int h = w / per_head, u = w - h * per_head;
        const uint16_t *src;
        uint16_t *dst;
        head_ptrs(h, src, dst);
        if (dst == nullptr) continue;
        if (u >= units) {                                // a chunk outside the rotation
            int off = (u - units) * 8;
            if (off >= a.rot_off) off += rot;
            *reinterpret_cast<uint4 *>(dst + off) = *reinterpret_cast<const uint4 *>(src + off);
            continue;
        }
        const int o1 = a.rot_off + (a.interleaved ? u * 16 : u * 8);
        const int o2 = a.interleaved ? o1 + 8 : o1 + rot / 2;
        uint4 r1 = *reinterpret_cast<const uint4 *>(src + o1), r2 = *reinterpret_cast<const uint4 *>(src + o2);
        uint16_t x[16], y[16];
        *reinterpret_cast<uint4 *>(x) = r1;
        *reinterpret_cast<uint4 *>(x + 8) = r2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 cs = s_cs[u * 8 + e];
            const int i1 = a.interleaved ? 2 * e : e, i2 = a.interleaved ? 2 * e + 1 : e + 8;
            const float x1 = h2f(x[i1]), x2 = h2f(x[i2]);
            y[i1] = f2h(x1 * cs.x - x2 * cs.y);
            y[i2] = f2h(x1 * cs.y + x2 * cs.x);
        }
        *reinterpret_cast<uint4 *>(dst + o1) = *reinterpret_cast<uint4 *>(y);
        *reinterpret_cast<uint4 *>(dst + o2) = *reinterpret_cast<uint4 *>(y + 8);
    }
    if (row >= 0)
        for (int ch = tid; ch < D / 8; ch += kAppendThreads)
            *reinterpret_cast<uint4 *>(a.kv.v + row * D + ch * 8) =
                *reinterpret_cast<const uint4 *>(a.v + tok * D + ch * 8);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs &a, int B, const Ctx &c) {
    return launch(paged_append_kernel, dim3(static_cast<unsigned>(a.N), static_cast<unsigned>(B)),
                  dim3(kAppendThreads), 0, c, 1, a);
}

}  // namespace ds4a
