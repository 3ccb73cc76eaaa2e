// paged_dev.cuh -- device routines shared by the kernels of the paged token cache
// and of drafted-token trees.
//
// A session's tokens sit in pages of `page` rows scattered over a shared pool: the
// token in slot t is row table[t / page] * page + t % page.  The session has len
// committed tokens (slots 0 .. len-1); its drafted node i, i < n <= 64, sits in slot
// len + i and at position len + depth(i), where parent(i) < i is the node it
// continues (-1: the last committed token).  Ancestor sets are 64-bit masks.
#pragma once

#include "ds4a_common.cuh"
#include "ds4a_internal.h"

namespace ds4a {

constexpr int kMaxNodes = 64;   // nodes of one session's tree: one bit each in a mask

// Pool row of slot t of a session whose page table row is `table`; -1 (recorded) if
// the page id is outside the pool.  The caller has checked t < max_pages * page.
DS4A_DEVINL long long pool_row(const PagedKV &kv, const int32_t *table, unsigned t, unsigned int *err) {
    const unsigned pg = t / static_cast<unsigned>(kv.page);
    const int id = __ldg(table + pg);
    if (id < 0 || id >= kv.n_pages) {
        record_error(err, DS4A_ERR_DEVICE_INDEX);
        return -1;
    }
    return static_cast<long long>(id) * kv.page + (t - pg * kv.page);
}

// Session s's counts; ok is false, and the reason recorded, if the session must be left
// alone: a count outside [0, N] or more tokens than its pages hold.
struct Session {
    long long len;
    int n;
    bool ok;
};
DS4A_DEVINL Session check_session(const PagedKV &kv, long long len, int n, int N, unsigned int *err) {
    Session r;
    r.len = len;
    r.n = n;
    r.ok = true;
    if (r.n < 0 || r.n > N || r.len < 0) {
        record_error(err, DS4A_ERR_DEVICE_INDEX);
        r.ok = false;
    } else if (r.len > static_cast<long long>(kv.max_pages) * kv.page - r.n) {   // len + n may not fit 64 bits
        record_error(err, DS4A_ERR_CAPACITY);
        r.ok = false;
    }
    return r;
}
DS4A_DEVINL Session load_session(const PagedKV &kv, const int32_t *n_node, int N, int s, unsigned int *err) {
    return check_session(kv, kv.len[s], n_node[s], N, err);
}

// Ancestor masks of a session's n nodes into mask[kMaxNodes] (shared memory), each node
// with its own bit; every thread of the block calls this (blockDim.x >= 64).  parent
// nullptr: a chain.  Pointer jumping: after round r a node's mask holds its nearest 2^r
// members of the path and ptr its 2^r-th ancestor, so log2(n) rounds reach all.
// Returns false (recorded) if a parent is not an earlier node or -1.
DS4A_DEVINL bool tree_masks(const int32_t *parent, int n, unsigned long long *mask, int *ptr, unsigned int *err) {
    const int i = threadIdx.x;
    bool good = true;
    if (i < kMaxNodes) {
        int p = -1;
        if (i < n) {
            p = parent ? parent[i] : i - 1;
            if (p < -1 || p >= i) {
                record_error(err, DS4A_ERR_DEVICE_INDEX);
                good = false;
                p = -1;
            }
        }
        mask[i] = 1ull << i;
        ptr[i] = p;
    }
    good = __syncthreads_and(good);
    for (int span = 1; span < n; span *= 2) {
        unsigned long long m = 0;
        int p = -1;
        if (i < kMaxNodes) {
            p = ptr[i];
            m = mask[i];
            if (p >= 0) {
                m |= mask[p];
                p = ptr[p];
            }
        }
        __syncthreads();
        if (i < kMaxNodes) {
            mask[i] = m;
            ptr[i] = p;
        }
        __syncthreads();
    }
    return good;
}

// Index of the (d+1)-th lowest set bit of m (d < popcount): the node at depth d of the
// path m, since a parent's index is below its child's.
DS4A_DEVINL int path_node(unsigned long long m, int d) {
    const uint32_t lo = static_cast<uint32_t>(m);
    const int c = __popc(lo);
    return d < c ? static_cast<int>(__fns(lo, 0, d + 1)) : 32 + static_cast<int>(__fns(static_cast<uint32_t>(m >> 32), 0, d - c + 1));
}

}  // namespace ds4a
