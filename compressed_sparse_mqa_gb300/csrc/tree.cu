// tree.cu -- the compressor on a tree of drafted tokens: the rows that nodes complete
// along their own paths, and the commit of the accepted path.
//
// A node whose position ends a block of `ratio` tokens completes the row
//   sum_t a_t [k_t ; v_t],  a = softmax over the block of w . k_t,
// over the block's committed tokens (held as the session's running state) and the node's
// ancestors inside the block.  Both kernels apply the tokens one at a time with the
// arithmetic of the one-token compressor update, so a row completed in a tree, and the
// state after a commit, have the bits that decoding the path token by token gives.
//
// Both are bound by latency: counts, parents, page numbers and tokens are loads one behind the other.  The
// keys' loads for the scores are all in flight at once; the weighted sums then load the path eight
// tokens at a time, up to eight load latencies in a row, beside the search for each token's node
// among the path's bits and a loop for each running maximum.  The up to 64 dependent updates
// themselves are the smaller part.
// Measured: 64 sessions of up to 64 nodes at ratio 128 7.9 us (12.8 with a CTA per node and one load
// at a time), 16 of up to 16 nodes at ratio 4 4.9 us; committing 64 paths of up to 32 nodes about 4 us.
#include "compress_dev.cuh"
#include "paged_dev.cuh"

namespace ds4a {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeWarps = kTreeThreads / 32;

// Scores w . k of the m path tokens at pool rows s_row: one warp per token, the lanes over
// 8-dim chunks as in the compressor.  A warp's tokens (up to kMaxNodes / kTreeWarps) are all
// loaded before the first is summed.
DS4A_DEVINL void path_scores(const PagedKV &kv, const float *w, const long long *s_row, int m, float *s_score) {
    constexpr int kPer = kMaxNodes / kTreeWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4 raw[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int t = warp + x * kTreeWarps;
        raw[x] = make_uint4(0, 0, 0, 0);
        if (t < m && lane < kv.D / 8)
            raw[x] = *reinterpret_cast<const uint4 *>(kv.k + s_row[t] * kv.D + lane * 8);
    }
    float wl[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wl[e] = lane < kv.D / 8 ? w[lane * 8 + e] : 0.f;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int t = warp + x * kTreeWarps;
        if (t >= m) break;
        const uint16_t *h = reinterpret_cast<const uint16_t *>(&raw[x]);
        float acc = 0.f;
        if (lane < kv.D / 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc = fmaf(wl[e], h2f(h[e]), acc);
        }
        acc = warp_sum(acc);
        if (lane == 0) s_score[t] = acc;
    }
}

// Weights of m path tokens, applied in order to a running state (max, sum): on return
// s_e[t] is token t's exp(s_t - max after it), s_c[t] the factor that rescales what came
// before it; mx and sum are the state after the last.  resume: a state precedes them.  The
// maxima do not depend on the sums, so thread t takes token t; only the sum is a chain.
DS4A_DEVINL void chain_weights(const float *s_score, int m, bool resume, float &mx, float &sum, float *s_e, float *s_c) {
    const int t = threadIdx.x;
    if (t < m) {
        float before = mx;
        for (int u = 0; u < t; ++u) before = fmaxf(before, s_score[u]);
        const float after = fmaxf(before, s_score[t]);
        s_c[t] = !resume && t == 0 ? 0.f : __expf(before - after);
        s_e[t] = __expf(s_score[t] - after);
    }
    __syncthreads();
    for (int u = 0; u < m; ++u) {
        mx = fmaxf(mx, s_score[u]);
        sum = __fadd_rn(__fmul_rn(s_c[u], sum), s_e[u]);
    }
}

// Applies the chain to column d (0 .. 2D-1: K dims, then V dims) of the weighted sums, eight
// tokens' loads at a time.
DS4A_DEVINL float chain_column(const PagedKV &kv, const long long *s_row, const float *s_e, const float *s_c, int m,
                               int d, float acc) {
    const uint16_t *src = d < kv.D ? kv.k + d : kv.v + (d - kv.D);
    for (int t0 = 0; t0 < m; t0 += 8) {
        uint16_t x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = t0 + u < m ? src[s_row[t0 + u] * kv.D] : uint16_t(0);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (t0 + u < m) acc = fmaf(s_e[t0 + u], h2f(x[u]), s_c[t0 + u] * acc);
    }
    return acc;
}

// gridDim.x CTAs per session take its completing nodes in turn.
__global__ void __launch_bounds__(kTreeThreads) compress_tree_kernel(CompressTreeArgs a) {
    __shared__ unsigned long long s_mask[kMaxNodes];
    __shared__ int s_ptr[kMaxNodes];
    __shared__ long long s_row[kMaxNodes];
    __shared__ float s_score[kMaxNodes], s_e[kMaxNodes], s_c[kMaxNodes];
    __shared__ uint32_t s_done[2];
    const int tid = threadIdx.x, s = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    const Session ses = load_session(a.kv, a.n_node, a.N, s, tid == 0 ? a.err : nullptr);
    if (!ses.ok) return;
    if (ses.len >= (a.cap - a.N + 1) * a.ratio) {   // len / ratio > cap - N: the draft's rows would be committed ones
        if (tid == 0) record_error(a.err, DS4A_ERR_CAPACITY);
        return;
    }
    if (!tree_masks(a.parent ? a.parent + static_cast<long long>(s) * a.N : nullptr, ses.n, s_mask, s_ptr, a.err))
        return;
    if (tid < kMaxNodes) {
        const bool c = tid < ses.n && (ses.len + __popcll(s_mask[tid])) % a.ratio == 0;
        const uint32_t b = __ballot_sync(0xffffffffu, c);
        if ((tid & 31) == 0) s_done[tid / 32] = b;
    }
    __syncthreads();
    const unsigned long long done = static_cast<unsigned long long>(s_done[1]) << 32 | s_done[0];
    const int n_done = __popcll(done), D = a.kv.D;
    for (int k = blockIdx.x; k < n_done; k += gridDim.x) {
        const int i = path_node(done, k);                                            // the k-th completing node
        const unsigned long long path = s_mask[i];
        const int cnt = __popcll(path);
        const long long end = ses.len + cnt;
        const long long start = end - a.ratio > ses.len ? end - a.ratio : ses.len;   // the block's first drafted token
        const bool resume = start == ses.len && ses.len % a.ratio != 0;
        const int d0 = static_cast<int>(start - ses.len), m = cnt - d0;
        bool good = true;
        if (tid < m) {
            s_row[tid] = pool_row(a.kv, a.kv.table + static_cast<long long>(s) * a.kv.max_pages,
                                  static_cast<unsigned>(ses.len + path_node(path, d0 + tid)), a.err);
            good = s_row[tid] >= 0;
        }
        if (!__syncthreads_and(good)) continue;   // a token in a page outside the pool (recorded): no row
        path_scores(a.kv, a.w, s_row, m, s_score);
        __syncthreads();
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
        __syncthreads();
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

    // Path rows to consecutive slots: all of them are read (here, beside what follows) before the
    // first is written, since a destination may be another path node's slot.
    constexpr int kMove = kMaxNodes * 128 / 8 / kTreeThreads;   // 16-byte chunks a thread, D <= 128
    const int chunks = D / 8, chunk_shift = D == 128 ? 4 : 3;
    uint4 rk[kMove], rv[kMove];
#pragma unroll
    for (int m = 0; m < kMove; ++m) {
        const int w = tid + m * kTreeThreads;
        if (w < cnt * chunks) {
            const long long at = s_src[w >> chunk_shift] * D + (w & (chunks - 1)) * 8;
            rk[m] = *reinterpret_cast<const uint4 *>(a.kv.k + at);
            rv[m] = *reinterpret_cast<const uint4 *>(a.kv.v + at);
        }
    }
    // rows completed on the path, from the draft's rows to their place
    if (a.ratio > 0) {
        const long long base = static_cast<long long>(s) * a.cap, r0 = ses.len / a.ratio;
        const int rows = static_cast<int>(end / a.ratio - r0);
        for (int w = tid; w < rows << chunk_shift; w += kTreeThreads) {
            const int r = w >> chunk_shift, ch = (w & (chunks - 1)) * 8;
            const int node = path_node(path, static_cast<int>((r0 + r + 1) * a.ratio - 1 - ses.len));
            const long long from = (base + a.cap - a.N + node) * D + ch, to = (base + r0 + r) * D + ch;
            const uint4 k = *reinterpret_cast<const uint4 *>(a.comp_k + from);
            const uint4 v = *reinterpret_cast<const uint4 *>(a.comp_v + from);
            *reinterpret_cast<uint4 *>(a.comp_k + to) = k;
            *reinterpret_cast<uint4 *>(a.comp_v + to) = v;
        }
        if (a.k_idx) {
            const int ich = a.d_idx / 8;
            for (int w = tid; w < rows * ich; w += kTreeThreads) {
                const int r = w / ich, ch = (w - r * ich) * 8;
                const int node = path_node(path, static_cast<int>((r0 + r + 1) * a.ratio - 1 - ses.len));
                *reinterpret_cast<uint4 *>(a.k_idx + (base + r0 + r) * a.d_idx + ch) =
                    *reinterpret_cast<const uint4 *>(a.k_idx + (base + a.cap - a.N + node) * a.d_idx + ch);
            }
        }
    }
    // the state of the block left open, from its committed state and its path tokens
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
#pragma unroll
    for (int m = 0; m < kMove; ++m) {
        const int w = tid + m * kTreeThreads;
        if (w < cnt * chunks) {
            const long long at = s_dst[w >> chunk_shift] * D + (w & (chunks - 1)) * 8;
            *reinterpret_cast<uint4 *>(a.kv.k + at) = rk[m];
            *reinterpret_cast<uint4 *>(a.kv.v + at) = rv[m];
        }
    }
    if (tid == 0) a.len_out[s] = end;                      // after the last read of len: it may be len itself
}

}  // namespace

cudaError_t launch_compress_tree(const CompressTreeArgs &a, int B, const Ctx &c) {
    // CTAs per session: up to one a node, about four per SM in all
    int per = 4 * c.num_sms / B;
    per = per < 1 ? 1 : (per > a.N ? a.N : per);
    return launch(compress_tree_kernel, dim3(static_cast<unsigned>(per), static_cast<unsigned>(B)),
                  dim3(kTreeThreads), 0, c, 1, a);
}

cudaError_t launch_commit_tree(const CommitTreeArgs &a, int B, const Ctx &c) {
    return launch(commit_tree_kernel, dim3(static_cast<unsigned>(B)), dim3(kTreeThreads), 0, c, 1, a);
}

}  // namespace ds4a
