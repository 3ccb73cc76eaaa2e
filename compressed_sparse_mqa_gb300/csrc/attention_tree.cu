// attention_tree.cu -- attention of a tree of drafted tokens over a paged cache.
//
// For node i at position p of session s and head h,
//   o_h = sum_j softmax_j(scale * q_h . K_j) V_j
// over the committed raw tokens t > p - window, the node's ancestors j (itself included)
// with p_j > p - window, and the compressed rows: those listed in its sel row, or every
// row complete at p.  A row j >= len / ratio is the one completed by the ancestor at
// position (j+1) * ratio - 1; it is read from the draft's rows (cap - N + that node).
//
// One CTA per node; its keys are a list (raw positions in order, then compressed rows).
#include "paged_dev.cuh"

namespace ds4a {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;          // keys per tile, one per lane
constexpr int kMaxHeadsPerWarp = 8;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ void __launch_bounds__(kThreads) attn_tree_kernel(AttnTreeArgs a) {
    __shared__ unsigned long long s_mask[kMaxNodes];
    __shared__ int s_ptr[kMaxNodes];
    __shared__ __align__(16) uint16_t s_k[kTile][D + 8], s_v[kTile][D + 8];
    __shared__ const uint16_t *s_src[2][kTile];
    __shared__ __align__(16) uint16_t s_q[64][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = blockIdx.x, s = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    const Session ses = load_session(a.kv, a.n_node, a.N, s, a.err);
    if (!ses.ok || i >= ses.n) return;
    if (a.ratio > 0 && ses.len / a.ratio > a.cap - a.N) {
        if (tid == 0) record_error(a.err, DS4A_ERR_CAPACITY);
        return;
    }
    if (!tree_masks(a.parent ? a.parent + static_cast<long long>(s) * a.N : nullptr, ses.n, s_mask, s_ptr, a.err))
        return;
    const unsigned long long path = s_mask[i];
    const long long p = ses.len + __popcll(path) - 1;
    const long long first = p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    const long long n_raw = p - first + 1;
    const long long n_vis0 = a.ratio > 0 ? ses.len / a.ratio : 0, n_vis = a.ratio > 0 ? (p + 1) / a.ratio : 0;
    const long long n_comp = a.sel ? a.n_sel : n_vis;
    const int32_t *sel = a.sel ? a.sel + (static_cast<long long>(s) * a.N + i) * a.n_sel : nullptr;
    const int32_t *table = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
    const long long node = static_cast<long long>(s) * a.N + i;
    for (int w = tid; w < a.H * D / 8; w += kThreads)
        reinterpret_cast<uint4 *>(&s_q[0][0])[w] = reinterpret_cast<const uint4 *>(a.q + node * a.H * D)[w];
    float m[kMaxHeadsPerWarp], l[kMaxHeadsPerWarp], o[kMaxHeadsPerWarp][D / 32];
#pragma unroll
    for (int x = 0; x < kMaxHeadsPerWarp; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[x][e] = 0.f;
    }
    for (long long k0 = 0; k0 < n_raw + n_comp; k0 += kTile) {
        if (tid < kTile) {
            const long long kx = k0 + tid;
            const uint16_t *ks = nullptr, *vs = nullptr;
            if (kx < n_raw) {
                const long long t = first + kx;
                const long long slot = t < ses.len ? t : ses.len + path_node(path, static_cast<int>(t - ses.len));
                const long long row = pool_row(a.kv, table, static_cast<unsigned>(slot), a.err);
                if (row >= 0) {
                    ks = a.kv.k + row * D;
                    vs = a.kv.v + row * D;
                }
            } else if (kx < n_raw + n_comp) {
                const long long j = sel ? sel[kx - n_raw] : kx - n_raw;
                if (j >= n_vis) {
                    record_error(a.err, DS4A_ERR_DEVICE_INDEX);
                } else if (j >= 0) {
                    const long long r = j < n_vis0 ? j : a.cap - a.N + path_node(path, static_cast<int>((j + 1) * a.ratio - 1 - ses.len));
                    ks = a.comp_k + (static_cast<long long>(s) * a.cap + r) * D;
                    vs = a.comp_v + (static_cast<long long>(s) * a.cap + r) * D;
                }
            }
            s_src[0][tid] = ks;
            s_src[1][tid] = vs;
        }
        __syncthreads();
        for (int w = tid; w < kTile * D / 8; w += kThreads) {
            const int r = w / (D / 8), ch = w % (D / 8);
            const uint16_t *ks = s_src[0][r], *vs = s_src[1][r];
            *reinterpret_cast<uint4 *>(&s_k[r][ch * 8]) = ks ? *reinterpret_cast<const uint4 *>(ks + ch * 8) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(&s_v[r][ch * 8]) = vs ? *reinterpret_cast<const uint4 *>(vs + ch * 8) : make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        const bool valid = s_src[0][lane] != nullptr;
#pragma unroll
        for (int x = 0; x < kMaxHeadsPerWarp; ++x) {
            const int h = warp + x * kWarps;
            if (h >= a.H) continue;
            float acc = 0.f;
#pragma unroll 8
            for (int d = 0; d < D; d += 2) {
                const float2 qf = __half22float2(*reinterpret_cast<const __half2 *>(&s_q[h][d]));
                const float2 kf = __half22float2(*reinterpret_cast<const __half2 *>(&s_k[lane][d]));
                acc = fmaf(qf.x, kf.x, fmaf(qf.y, kf.y, acc));
            }
            const float sc = valid ? acc * a.scale_log2 : -INFINITY;
            const float mn = fmaxf(m[x], warp_max(sc));
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float pr = valid ? exp2f(sc - ref) : 0.f, al = exp2f(m[x] - ref);
            l[x] = l[x] * al + warp_sum(pr);
            m[x] = mn;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) o[x][e] *= al;
            for (int k = 0; k < kTile; ++k) {
                const float pk = __shfl_sync(0xffffffffu, pr, k);
                if (s_src[0][k] == nullptr) continue;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) o[x][e] = fmaf(pk, h2f(s_v[k][lane + e * 32]), o[x][e]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < kMaxHeadsPerWarp; ++x) {
        const int h = warp + x * kWarps;
        if (h >= a.H) continue;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) a.out[(node * a.H + h) * D + lane + e * 32] =
            f2h(l[x] == 0.f ? 0.f : o[x][e] / l[x]);   // no readable row (bad page ids, recorded): zeros
    }
}

}  // namespace

size_t attn_tree_ws_bytes(int, int, int, int) { return 256; }

cudaError_t launch_attn_tree(const AttnTreeArgs &args, int B, const Ctx &c) {
    AttnTreeArgs a = args;
    a.scale_log2 = a.scale * kLog2e;
    const dim3 grid(static_cast<unsigned>(a.N), static_cast<unsigned>(B));
    return a.kv.D == 128 ? launch(attn_tree_kernel<128>, grid, dim3(kThreads), 0, c, 1, a)
                         : launch(attn_tree_kernel<64>, grid, dim3(kThreads), 0, c, 1, a);
}

}  // namespace ds4a
