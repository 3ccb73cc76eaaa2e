// tree.cu -- the compressor on a tree of drafted tokens: the rows that nodes complete
// along their own paths, and the commit of the accepted path.
//
// A node whose position ends a block of `ratio` tokens completes the row
//   sum_t a_t [k_t ; v_t],  a = softmax over the block of w . k_t,
// over the block's committed tokens (held as the session's running state) and the node's
// ancestors inside the block.  Both kernels apply the tokens one at a time with the
// arithmetic of the one-token compressor update, so a row completed in a tree, and the
// state after a commit, have the bits that decoding the path token by token gives.
#include "compress_dev.cuh"
#include "paged_dev.cuh"

namespace ds4a {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeWarps = kTreeThreads / 32;

// Weights of m path tokens, applied in order to a running state (max, sum): on return
// s_e[t] is token t's exp(s_t - max after it), s_c[t] the factor that rescales what came
// before it; max and sum are the state after the last.  resume: a state precedes them.
DS4A_DEVINL void chain_weights(const float *s_score, int m, bool resume, float &mx, float &sum, float *s_e, float *s_c) {
    for (int t = 0; t < m; ++t) {
        const float m_new = fmaxf(mx, s_score[t]);
        const bool first = !resume && t == 0;
        const float c_old = first ? 0.f : __expf(mx - m_new);
        const float e = __expf(s_score[t] - m_new);
        sum = __fadd_rn(__fmul_rn(c_old, sum), e);
        mx = m_new;
        if (threadIdx.x == 0) {
            s_e[t] = e;
            s_c[t] = c_old;
        }
    }
}

// Scores w . k of the m path tokens at pool rows s_row (-1: unreadable, score 0): one
// warp per token, the lanes over 8-dim chunks as in the compressor.
DS4A_DEVINL void path_scores(const PagedKV &kv, const float *w, const long long *s_row, int m, float *s_score) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int t = warp; t < m; t += kTreeWarps) {
        float acc = 0.f;
        if (s_row[t] >= 0) {
            for (int ch = lane; ch < kv.D / 8; ch += 32) {
                const uint4 raw = *reinterpret_cast<const uint4 *>(kv.k + s_row[t] * kv.D + ch * 8);
                const uint16_t *h = reinterpret_cast<const uint16_t *>(&raw);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc = fmaf(w[ch * 8 + e], h2f(h[e]), acc);
            }
        }
        acc = warp_sum(acc);
        if (lane == 0) s_score[t] = acc;
    }
}

// Applies the chain to column d (0 .. 2D-1: K dims, then V dims) of the weighted sums.
DS4A_DEVINL float chain_column(const PagedKV &kv, const long long *s_row, const float *s_e, const float *s_c, int m,
                               int d, float acc) {
    const uint16_t *src = d < kv.D ? kv.k + d : kv.v + (d - kv.D);
    for (int t = 0; t < m; ++t) {
        const float x = s_row[t] >= 0 ? h2f(src[s_row[t] * kv.D]) : 0.f;
        acc = fmaf(s_e[t], x, s_c[t] * acc);
    }
    return acc;
}

// One CTA per node: completes a row or leaves.
__global__ void __launch_bounds__(kTreeThreads) compress_tree_kernel(CompressTreeArgs a) {
    __shared__ unsigned long long s_mask[kMaxNodes];
    __shared__ int s_ptr[kMaxNodes];
    __shared__ long long s_row[kMaxNodes];
    __shared__ float s_score[kMaxNodes], s_e[kMaxNodes], s_c[kMaxNodes];
    const int tid = threadIdx.x, i = blockIdx.x, s = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    const Session ses = load_session(a.kv, a.n_node, a.N, s, a.err);
    if (!ses.ok || i >= ses.n) return;
    if (!tree_masks(a.parent ? a.parent + static_cast<long long>(s) * a.N : nullptr, ses.n, s_mask, s_ptr, a.err))
        return;
    const unsigned long long path = s_mask[i];
    const int cnt = __popcll(path);
    const long long end = ses.len + cnt;
    if (end % a.ratio != 0) return;
    const long long start = end - a.ratio > ses.len ? end - a.ratio : ses.len;   // the block's first drafted token
    const bool resume = start == ses.len && ses.len % a.ratio != 0;
    const int d0 = static_cast<int>(start - ses.len), m = cnt - d0;
    if (tid < m)
        s_row[tid] = pool_row(a.kv, a.kv.table + static_cast<long long>(s) * a.kv.max_pages,
                              static_cast<unsigned>(ses.len + path_node(path, d0 + tid)), a.err);
    __syncthreads();
    path_scores(a.kv, a.w, s_row, m, s_score);
    __syncthreads();
    const int D = a.kv.D;
    const float *st = a.state + static_cast<long long>(s) * (2 + 2 * D);
    float mx = -INFINITY, sum = 0.f;
    if (resume) { mx = st[0]; sum = st[1]; }
    chain_weights(s_score, m, resume, mx, sum, s_e, s_c);
    __syncthreads();
    const long long row = (static_cast<long long>(s) * a.cap + a.cap - a.N + i) * D;
    for (int d = tid; d < 2 * D; d += kTreeThreads) {
        const float acc = chain_column(a.kv, s_row, s_e, s_c, m, d, resume ? st[2 + d] : 0.f);
        const float inv = 1.f / sum;
        (d < D ? a.comp_k + row + d : a.comp_v + row + d - D)[0] = f2h(acc * inv);
    }
}

// One CTA per session.
__global__ void __launch_bounds__(kTreeThreads) commit_tree_kernel(CommitTreeArgs a) {
    __shared__ unsigned long long s_mask[kMaxNodes];
    __shared__ int s_ptr[kMaxNodes];
    __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];
    __shared__ float s_score[kMaxNodes], s_e[kMaxNodes], s_c[kMaxNodes];
    const int tid = threadIdx.x, s = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const Session ses = load_session(a.kv, a.n_node, a.N, s, a.err);
    if (!ses.ok) return;
    const int leaf = a.leaf[s];
    if (leaf < -1 || leaf >= ses.n) {
        if (tid == 0) record_error(a.err, DS4A_ERR_DEVICE_INDEX);
        return;
    }
    if (!tree_masks(a.parent ? a.parent + static_cast<long long>(s) * a.N : nullptr, ses.n, s_mask, s_ptr, a.err))
        return;
    const unsigned long long path = leaf >= 0 ? s_mask[leaf] : 0ull;
    const int cnt = __popcll(path), D = a.kv.D;
    const long long end = ses.len + cnt;
    if (a.ratio > 0 && end / a.ratio > a.cap - a.N) {
        if (tid == 0) record_error(a.err, DS4A_ERR_CAPACITY);
        return;
    }
    bool good = true;
    if (tid < cnt) {
        const int32_t *tab = a.kv.table + static_cast<long long>(s) * a.kv.max_pages;
        s_src[tid] = pool_row(a.kv, tab, static_cast<unsigned>(ses.len + path_node(path, tid)), a.err);
        s_dst[tid] = pool_row(a.kv, tab, static_cast<unsigned>(ses.len + tid), a.err);
        good = s_src[tid] >= 0 && s_dst[tid] >= 0;
    }
    if (!__syncthreads_and(good)) return;

    // the state of the block left open, from its committed state and its path tokens (read
    // before any row moves)
    if (a.ratio > 0 && end % a.ratio != 0) {
        const long long blk = end - end % a.ratio;
        const long long start = blk > ses.len ? blk : ses.len;
        const bool resume = blk < ses.len;
        const int d0 = static_cast<int>(start - ses.len), m = cnt - d0;
        path_scores(a.kv, a.w, s_src + d0, m, s_score);
        __syncthreads();
        const float *st = a.state + static_cast<long long>(s) * (2 + 2 * D);
        float *so = a.state_out + static_cast<long long>(s) * (2 + 2 * D);
        float mx = -INFINITY, sum = 0.f;
        if (resume) { mx = st[0]; sum = st[1]; }
        chain_weights(s_score, m, resume, mx, sum, s_e, s_c);
        __syncthreads();                                   // state_out may be state: every thread has read the head
        for (int d = tid; d < 2 * D; d += kTreeThreads)
            so[2 + d] = chain_column(a.kv, s_src + d0, s_e, s_c, m, d, resume ? st[2 + d] : 0.f);
        if (tid == 0) {
            so[0] = mx;
            so[1] = sum;
        }
    }
    __syncthreads();

    // path rows to consecutive slots: all of them are read before the first is written,
    // since a destination may be another path node's slot
    constexpr int kMove = kMaxNodes * 128 / 8 / kTreeThreads;   // 16-byte chunks a thread, D <= 128
    const int chunks = D / 8;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint16_t *pool = which ? a.kv.v : a.kv.k;
        uint4 r[kMove];
#pragma unroll
        for (int m = 0; m < kMove; ++m) {
            const int w = tid + m * kTreeThreads;
            if (w < cnt * chunks) r[m] = *reinterpret_cast<const uint4 *>(pool + s_src[w / chunks] * D + w % chunks * 8);
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kMove; ++m) {
            const int w = tid + m * kTreeThreads;
            if (w < cnt * chunks) *reinterpret_cast<uint4 *>(pool + s_dst[w / chunks] * D + w % chunks * 8) = r[m];
        }
    }
    // rows completed on the path, from the draft's rows to their place
    if (a.ratio > 0) {
        const long long base = static_cast<long long>(s) * a.cap;
        for (long long r = ses.len / a.ratio; r < end / a.ratio; ++r) {
            const int node = path_node(path, static_cast<int>((r + 1) * a.ratio - 1 - ses.len));
            const long long from = base + a.cap - a.N + node, to = base + r;
            for (int ch = tid; ch < chunks; ch += kTreeThreads) {
                *reinterpret_cast<uint4 *>(a.comp_k + to * D + ch * 8) =
                    *reinterpret_cast<const uint4 *>(a.comp_k + from * D + ch * 8);
                *reinterpret_cast<uint4 *>(a.comp_v + to * D + ch * 8) =
                    *reinterpret_cast<const uint4 *>(a.comp_v + from * D + ch * 8);
            }
            if (a.k_idx)
                for (int ch = tid; ch < a.d_idx / 8; ch += kTreeThreads)
                    *reinterpret_cast<uint4 *>(a.k_idx + to * a.d_idx + ch * 8) =
                        *reinterpret_cast<const uint4 *>(a.k_idx + from * a.d_idx + ch * 8);
        }
    }
    if (tid == 0) a.len_out[s] = end;                      // after the last read of len: it may be len itself
}

}  // namespace

cudaError_t launch_compress_tree(const CompressTreeArgs &a, int B, const Ctx &c) {
    return launch(compress_tree_kernel, dim3(static_cast<unsigned>(a.N), static_cast<unsigned>(B)),
                  dim3(kTreeThreads), 0, c, 1, a);
}

cudaError_t launch_commit_tree(const CommitTreeArgs &a, int B, const Ctx &c) {
    return launch(commit_tree_kernel, dim3(static_cast<unsigned>(B)), dim3(kTreeThreads), 0, c, 1, a);
}

}  // namespace ds4a
