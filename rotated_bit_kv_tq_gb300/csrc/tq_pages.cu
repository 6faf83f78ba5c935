// tq_pages.cu -- the pages of paged caches: extend, fork, free, compact, copy.
//
// A paged cache keeps whole pages of packed rows (kenji.blog TinyLLaMA article, section 7,
// preallocates rows instead; pages are that pool cut into pieces that sequences can share).
// One page table serves the K and V caches of all layers, so one plan serves them all:
// a call first decides in a single CTA which pages go where (the plan: integer prefix sums
// over the requests and over the pages' reference counts, lowest page numbers first, so the
// result does not depend on timing), then a grid of CTAs applies it to every cache.
//
// The data movement is bound by HBM: a moved byte is read once and written once.  The copy
// grid works through units of kUnitBytes of one (page, cache); each thread has kUnitLoads
// independent 16-byte loads in flight before it stores.  The plan kernels are bound by
// latency (a few dependent global round trips and block scans).
#include "tq_internal.cuh"

namespace tq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kScanItems = 4;                                 // pages per thread and scan step
constexpr int kCopyThreads = 256;
constexpr int kUnitLoads = 4;
constexpr int kUnitBytes = kCopyThreads * kUnitLoads * 16;    // 16 KB
constexpr int kMaxCaches = TQ_PAGES_MAX_CACHES;
constexpr int kCopyCtasPerSm = 8;

// Workspace, in 32-bit words (each call writes what it reads; nothing is kept between calls):
//   [0]      entries of the copy list
//   [1]      pages in use (compact)
//   list     src, dst, rows: n_items words each (compact: n_pages), the page copies
//   item     two words per item: fork's fresh page / status and parent length
//   mark     n_seqs words: the item that claims a sequence
//   page     2 n_pages words: per-page scratch (free list; new numbers and counts; claims)
constexpr int64_t kHeadWords = 64;
struct WsLayout {
    int64_t list_cap, src, dst, rows, item, mark, page, total;
};
__host__ __device__ inline WsLayout ws_layout(int64_t n_pages, int64_t n_seqs, int64_t n_items) {
    WsLayout w;
    w.list_cap = max64(n_pages, n_items);
    w.src = kHeadWords;
    w.dst = w.src + w.list_cap;
    w.rows = w.dst + w.list_cap;
    w.item = w.rows + w.list_cap;
    w.mark = w.item + 2 * n_items;
    w.page = w.mark + n_seqs;
    w.total = w.page + 2 * n_pages;
    return w;
}

struct PoolView {
    int32_t *table, *lens, *refs;
    int32_t n_pages, page_tokens, n_seqs, cols;
};
PoolView pool_view(const tq_page_pool &p) {
    return PoolView{p.page_table, p.seq_lens, p.refcounts, p.n_pages, p.page_tokens, p.n_seqs,
                    p.max_pages_per_seq};
}

struct CopyCaches {
    uint8_t *base[kMaxCaches];
    int32_t row_bytes[kMaxCaches];
    int32_t n;
    int32_t units;   // copy units of the largest page
};

// ------------------------------------------------------------------ block scans
// Exclusive prefix sum of v over the plan CTA; *total is the sum.  Two barriers.
__device__ __forceinline__ int block_scan(int v, int *total) {
    __shared__ int sums[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int s = lane < kPlanThreads / 32 ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    __syncthreads();   // sums is reused by the next scan
    return x - v + (warp > 0 ? before : 0);
}

// The `want` lowest free pages (reference count 0), ascending, into list[]; returns how many
// there are (at most want).  The scan stops once it has found them.
__device__ __forceinline__ int find_free(const PoolView &p, int64_t want, int32_t *list) {
    int found = 0;
    for (int base = 0; base < p.n_pages && found < want; base += kPlanThreads * kScanItems) {
        const int p0 = base + threadIdx.x * kScanItems;
        bool fr[kScanItems];
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kScanItems; ++e) {
            fr[e] = p0 + e < p.n_pages && p.refs[p0 + e] == 0;
            mine += fr[e];
        }
        int total;
        int at = found + block_scan(mine, &total);
#pragma unroll
        for (int e = 0; e < kScanItems; ++e)
            if (fr[e]) {
                if (at < want) list[at] = p0 + e;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    return (int)min64(found, want);
}

__device__ __forceinline__ int pages_of(int64_t len, int page_tokens) {
    return (int)((len + page_tokens - 1) / page_tokens);
}

// A sequence's length, if its id is valid and the table can hold it; -1 (and the error
// recorded) otherwise.
__device__ __forceinline__ int checked_len(const PoolView &p, int seq) {
    if (seq < 0 || seq >= p.n_seqs) {
        record_error(TQ_ERR_OUT_OF_RANGE);
        return -1;
    }
    const int len = p.lens[seq];
    if (len < 0 || len > (int64_t)p.cols * p.page_tokens) {
        record_error(TQ_ERR_OUT_OF_RANGE);
        return -1;
    }
    return len;
}

// ------------------------------------------------------------------ extend
__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const PoolView p, const int32_t *seqs,
                                                              const int32_t *n_new, int n, int32_t *ws) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(p.n_pages, p.n_seqs, n);
    int32_t *mark = ws + w.mark, *need = ws + w.item, *len0 = ws + w.item + n, *free_list = ws + w.page;
    for (int s = threadIdx.x; s < p.n_seqs; s += kPlanThreads) mark[s] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (seqs[i] >= 0 && seqs[i] < p.n_seqs) atomicMin(&mark[seqs[i]], i);
    __syncthreads();
    int total = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int k = 0, len = -1;
        if (i < n) {
            const int s = seqs[i], add = n_new[i];
            len = checked_len(p, s);
            if (len >= 0 && (mark[s] != i || add < 0 || (int64_t)len + add > (int64_t)p.cols * p.page_tokens)) {
                record_error(TQ_ERR_OUT_OF_RANGE);   // a repeated sequence, or more than its table holds
                len = -1;
            }
            if (len >= 0) k = pages_of((int64_t)len + add, p.page_tokens) - pages_of(len, p.page_tokens);
        }
        int sum;
        const int first = total + block_scan(k, &sum);
        if (i < n) {
            need[i] = first;
            len0[i] = len;
        }
        total += sum;
    }
    const int have = find_free(p, total, free_list);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int len = len0[i], first = need[i];
        if (len < 0) continue;
        const int s = seqs[i], add = n_new[i];
        const int p0 = pages_of(len, p.page_tokens), p1 = pages_of((int64_t)len + add, p.page_tokens);
        if (p1 > p0 && first + (p1 - p0) > have) {   // the pool is used up: the sequence stays as it was
            record_error(TQ_ERR_OUT_OF_RANGE);
            continue;
        }
        for (int j = p0; j < p1; ++j) {
            const int page = free_list[first + j - p0];
            p.table[(int64_t)s * p.cols + j] = page;
            p.refs[page] = 1;
        }
        p.lens[s] = len + add;
    }
}

// ------------------------------------------------------------------ free
// One CTA per listed sequence.  Taking the length to zero claims the sequence, so a sequence
// listed twice is freed once; which CTA wins does not change the result.
__global__ void __launch_bounds__(128) free_kernel(const PoolView p, const int32_t *seqs) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int s_len;
    const int s = seqs[blockIdx.x];
    if (s < 0 || s >= p.n_seqs) {
        if (threadIdx.x == 0) record_error(TQ_ERR_OUT_OF_RANGE);
        return;
    }
    if (threadIdx.x == 0) s_len = atomicExch(&p.lens[s], 0);
    __syncthreads();
    const int len = s_len;
    if (len < 0 || len > (int64_t)p.cols * p.page_tokens) {
        if (threadIdx.x == 0) record_error(TQ_ERR_OUT_OF_RANGE);
        if (len < 0) return;
    }
    const int n = (int)min64(p.cols, pages_of(len, p.page_tokens));
    for (int j = threadIdx.x; j < n; j += 128) {
        int32_t *e = p.table + (int64_t)s * p.cols + j;
        const int page = *e;
        *e = -1;
        if (page < 0 || page >= p.n_pages) record_error(TQ_ERR_OUT_OF_RANGE);
        else if (atomicSub(&p.refs[page], 1) <= 0) {   // a count that was not held: leave it at 0
            atomicAdd(&p.refs[page], 1);
            record_error(TQ_ERR_OUT_OF_RANGE);
        }
    }
}

// ------------------------------------------------------------------ fork
// Item words: [i] the fresh page (>= 0), kNoFresh (the parent ends with a whole page) or
// kNotServed; [n + i] the parent's length.
constexpr int kNoFresh = -1, kNotServed = -2;

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PoolView p, const int32_t *parents,
                                                                 const int32_t *children, int n, int32_t *ws) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(p.n_pages, p.n_seqs, n);
    int32_t *mark = ws + w.mark, *fresh = ws + w.item, *plen = ws + w.item + n, *free_list = ws + w.page;
    for (int s = threadIdx.x; s < p.n_seqs; s += kPlanThreads) mark[s] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (children[i] >= 0 && children[i] < p.n_seqs) atomicMin(&mark[children[i]], i);
    __syncthreads();
    int total = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int k = 0, len = -1;
        if (i < n) {
            const int c = children[i];
            len = checked_len(p, parents[i]);
            const int clen = checked_len(p, c);
            if (len >= 0 && clen >= 0 && (clen != 0 || mark[c] != i)) {
                record_error(TQ_ERR_OUT_OF_RANGE);   // the child holds rows, or is listed twice
                len = -1;
            }
            if (clen < 0) len = -1;
            if (len > 0) k = len % p.page_tokens != 0;
        }
        int sum;
        const int first = total + block_scan(k, &sum);
        if (i < n) {
            fresh[i] = len <= 0 ? kNotServed : k ? first : kNoFresh;   // a rank until the pages are known
            plen[i] = len;
        }
        total += sum;
    }
    const int have = find_free(p, total, free_list);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int rank = fresh[i];
        if (rank < 0) continue;
        if (rank >= have) {
            record_error(TQ_ERR_OUT_OF_RANGE);
            fresh[i] = kNotServed;
            continue;
        }
        const int len = plen[i], page = free_list[rank];
        fresh[i] = page;
        ws[w.src + rank] = p.table[(int64_t)parents[i] * p.cols + len / p.page_tokens];
        ws[w.dst + rank] = page;
        ws[w.rows + rank] = len % p.page_tokens;
    }
    if (threadIdx.x == 0) ws[0] = have;
}

// ------------------------------------------------------------------ copies
// Copy the first `rows` rows of page src to page dst of every cache, for the listed entries:
// grid-stride over units of kUnitBytes.
__device__ __forceinline__ void copy_pages(const CopyCaches &c, int page_tokens, int n_pages,
                                           const int32_t *src, const int32_t *dst, const int32_t *rows,
                                           int64_t n) {
    const int64_t units = n * c.n * c.units;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t e = u / (c.n * c.units);
        const int r = (int)(u - e * (c.n * c.units));
        const int ci = r / c.units, piece = r - ci * c.units;
        const int sp = src[e], dp = dst[e];
        if (sp < 0 || sp >= n_pages || dp < 0 || dp >= n_pages) {
            if (r == 0 && threadIdx.x == 0) record_error(TQ_ERR_OUT_OF_RANGE);
            continue;
        }
        const int64_t rb = c.row_bytes[ci], page_bytes = rb * page_tokens;
        const int64_t bytes = rows ? rb * rows[e] : page_bytes;
        const int64_t off = (int64_t)piece * kUnitBytes;
        if (off >= bytes) continue;
        const uint8_t *s = c.base[ci] + sp * page_bytes + off;
        uint8_t *d = c.base[ci] + dp * page_bytes + off;
        const int left = (int)min64(bytes - off, kUnitBytes);
        // pages start on 16-byte boundaries: page_tokens is a multiple of 32 and rows are even
        const int vecs = left >> 4;
        uint4 v[kUnitLoads];
#pragma unroll
        for (int k = 0; k < kUnitLoads; ++k) {
            const int i = threadIdx.x + k * kCopyThreads;
            if (i < vecs) v[k] = __ldcs(reinterpret_cast<const uint4 *>(s) + i);
        }
#pragma unroll
        for (int k = 0; k < kUnitLoads; ++k) {
            const int i = threadIdx.x + k * kCopyThreads;
            if (i < vecs) __stcs(reinterpret_cast<uint4 *>(d) + i, v[k]);
        }
        // the last rows may end inside 16 bytes: what follows them in the page stays as it is
        const int t = (vecs << 4) + 2 * threadIdx.x;
        if (t < left) *reinterpret_cast<uint16_t *>(d + t) = *reinterpret_cast<const uint16_t *>(s + t);
    }
}

__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const PoolView p, const int32_t *parents,
                                                                  const int32_t *children, int n,
                                                                  const int32_t *ws,
                                                                  const __grid_constant__ CopyCaches c) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(p.n_pages, p.n_seqs, n);
    const int32_t *fresh = ws + w.item, *plen = ws + w.item + n;
    const int64_t step = (int64_t)gridDim.x * kCopyThreads;
    for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < (int64_t)n * p.cols; e += step) {
        const int i = (int)(e / p.cols), j = (int)(e - (int64_t)i * p.cols);
        const int f = fresh[i];
        if (f == kNotServed) continue;
        const int len = plen[i], whole = len / p.page_tokens, child = children[i];
        if (j == 0) p.lens[child] = len;
        if (j > whole || (j == whole && f == kNoFresh)) continue;
        int page = f;
        if (j < whole) {
            page = p.table[(int64_t)parents[i] * p.cols + j];
            if (page < 0 || page >= p.n_pages) {
                record_error(TQ_ERR_OUT_OF_RANGE);
                page = -1;
            } else {
                atomicAdd(&p.refs[page], 1);
            }
        } else {
            p.refs[page] = 1;
        }
        p.table[(int64_t)child * p.cols + j] = page;
    }
    copy_pages(c, p.page_tokens, p.n_pages, ws + w.src, ws + w.dst, ws + w.rows, ws[0]);
}

// ------------------------------------------------------------------ compact
// U pages are in use; the used pages numbered U and up ("movers") go, in order, to the free
// pages below U ("holes"): as many holes as movers, sources and destinations disjoint, so
// every copy can run at once.  Page words: [q] the new number of page q, [n_pages + q] the
// reference count at number q afterwards.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PoolView p, int32_t *ws,
                                                                    int32_t *n_used_out) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(p.n_pages, p.n_seqs, 0);
    int32_t *holes = ws + w.dst, *movers = ws + w.src, *moved = ws + w.page, *count = ws + w.page + p.n_pages;
    int used = 0;
    for (int base = 0; base < p.n_pages; base += kPlanThreads * kScanItems) {
        const int p0 = base + threadIdx.x * kScanItems;
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kScanItems; ++e) mine += p0 + e < p.n_pages && p.refs[p0 + e] > 0;
        int total;
        block_scan(mine, &total);
        used += total;
    }
    int n_holes = 0, n_movers = 0;
    for (int base = 0; base < p.n_pages; base += kPlanThreads * kScanItems) {
        const int p0 = base + threadIdx.x * kScanItems;
        int kind[kScanItems], mine = 0;   // 1: hole, 2: mover (never both in one thread's pages' sides)
#pragma unroll
        for (int e = 0; e < kScanItems; ++e) {
            const int q = p0 + e;
            kind[e] = 0;
            if (q >= p.n_pages) continue;
            const int r = p.refs[q];
            if (q < used) {
                kind[e] = r > 0 ? 0 : 1;
                count[q] = r;
            } else {
                kind[e] = r > 0 ? 2 : 0;
                count[q] = 0;
            }
            moved[q] = q;
            mine += kind[e] == 1 ? 1 : kind[e] == 2 ? 1 << 16 : 0;   // at most 4,096 of each in a step
        }
        int total;
        const int at = block_scan(mine, &total);
        int h = n_holes + (at & 0xffff), m = n_movers + (at >> 16);
#pragma unroll
        for (int e = 0; e < kScanItems; ++e) {
            if (kind[e] == 1) holes[h++] = p0 + e;
            if (kind[e] == 2) movers[m++] = p0 + e;
        }
        n_holes += total & 0xffff;
        n_movers += total >> 16;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < n_movers; k += kPlanThreads) {
        moved[movers[k]] = holes[k];
        count[holes[k]] = p.refs[movers[k]];
    }
    if (threadIdx.x == 0) {
        ws[0] = n_movers;
        ws[1] = used;
        if (n_used_out) *n_used_out = used;
    }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const PoolView p, const PoolView out,
                                                                     const int32_t *ws,
                                                                     const __grid_constant__ CopyCaches c) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(p.n_pages, p.n_seqs, 0);
    const int32_t *moved = ws + w.page, *count = ws + w.page + p.n_pages;
    const int64_t step = (int64_t)gridDim.x * kCopyThreads, t0 = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
    for (int64_t e = t0; e < (int64_t)p.n_seqs * p.cols; e += step) {
        const int page = p.table[e];
        if (page >= p.n_pages) record_error(TQ_ERR_OUT_OF_RANGE);
        out.table[e] = page >= 0 && page < p.n_pages ? moved[page] : -1;
    }
    for (int64_t q = t0; q < p.n_pages; q += step) out.refs[q] = count[q];
    for (int64_t s = t0; s < p.n_seqs; s += step) out.lens[s] = p.lens[s];
    copy_pages(c, p.page_tokens, p.n_pages, ws + w.src, ws + w.dst, nullptr, ws[0]);
}

// ------------------------------------------------------------------ copy
// The valid pairs of a copy list, in order.  A pair is refused (and recorded) when a page is
// out of range, when its destination is the destination of an earlier pair, or when its
// destination is a source of any pair: then no result depends on the order of the copies.
__global__ void __launch_bounds__(kPlanThreads) copy_plan_kernel(const int32_t *src, const int32_t *dst,
                                                                 const int32_t *rows, int n, int n_pages,
                                                                 int page_tokens, int32_t *ws) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(n_pages, 0, n);
    int32_t *first = ws + w.page, *is_src = ws + w.page + n_pages;
    for (int q = threadIdx.x; q < n_pages; q += kPlanThreads) {
        first[q] = INT32_MAX;
        is_src[q] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        if (dst[i] >= 0 && dst[i] < n_pages) atomicMin(&first[dst[i]], i);
        if (src[i] >= 0 && src[i] < n_pages) is_src[src[i]] = 1;
    }
    __syncthreads();
    int kept = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        bool ok = false;
        if (i < n) {
            const int s = src[i], d = dst[i], r = rows ? rows[i] : page_tokens;
            ok = s >= 0 && s < n_pages && d >= 0 && d < n_pages && r >= 0 && r <= page_tokens &&
                 first[d] == i && !is_src[d];
            if (!ok) record_error(TQ_ERR_OUT_OF_RANGE);
        }
        int total;
        const int at = kept + block_scan(ok, &total);
        if (ok) {
            ws[w.src + at] = src[i];
            ws[w.dst + at] = dst[i];
            ws[w.rows + at] = rows ? rows[i] : page_tokens;
        }
        kept += total;
    }
    if (threadIdx.x == 0) ws[0] = kept;
}

__global__ void __launch_bounds__(kCopyThreads) copy_apply_kernel(int n_pages, int page_tokens, int n,
                                                                  const int32_t *ws,
                                                                  const __grid_constant__ CopyCaches c) {
    pdl_wait();
    pdl_launch_dependents();
    const WsLayout w = ws_layout(n_pages, 0, n);
    copy_pages(c, page_tokens, n_pages, ws + w.src, ws + w.dst, ws + w.rows, ws[0]);
}

// ------------------------------------------------------------------ host side
tq_status check_pool(const tq_page_pool *p) {
    if (!p || !p->page_table || !p->seq_lens || !p->refcounts) return TQ_ERR_INVALID_ARGUMENT;
    if (p->n_pages < 1 || p->page_tokens < 1 || p->n_seqs < 1 || p->max_pages_per_seq < 1)
        return TQ_ERR_INVALID_ARGUMENT;
    if (p->page_tokens % 32) return TQ_ERR_UNSUPPORTED;
    // lengths are 32-bit: a full table must stay countable
    if ((int64_t)p->max_pages_per_seq * p->page_tokens > INT32_MAX) return TQ_ERR_UNSUPPORTED;
    // and so are the prefix sums over all sequences' pages
    if ((int64_t)p->n_seqs * p->max_pages_per_seq > INT32_MAX) return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

tq_status gather_caches(const tq_cache *const *caches, int n, int page_tokens, int64_t n_pages, CopyCaches *out) {
    if (!caches || n < 1) return TQ_ERR_INVALID_ARGUMENT;
    if (n > kMaxCaches) return TQ_ERR_UNSUPPORTED;
    int64_t most = 0;
    for (int i = 0; i < n; ++i) {
        const tq_status st = validate_cache(caches[i]);
        if (st != TQ_OK) return st;
        if (caches[i]->page_tokens != page_tokens || caches[i]->n_pages < n_pages) return TQ_ERR_INVALID_ARGUMENT;
        out->base[i] = static_cast<uint8_t *>(caches[i]->base);
        out->row_bytes[i] = (int32_t)tq_row_bytes(caches[i]->type, caches[i]->n_kv_heads, caches[i]->head_dim);
        most = max64(most, (int64_t)out->row_bytes[i] * page_tokens);
    }
    out->n = n;
    out->units = (int32_t)((most + kUnitBytes - 1) / kUnitBytes);
    return TQ_OK;
}

tq_status check_ws(const void *ws, size_t bytes, const WsLayout &w) {
    if (!ws || bytes < (size_t)w.total * 4) return TQ_ERR_WORKSPACE_TOO_SMALL;
    return reinterpret_cast<uintptr_t>(ws) % 16 ? TQ_ERR_INVALID_ARGUMENT : TQ_OK;
}

// CTAs of an apply kernel: enough for `units` copy units and `words` table entries, at most
// kCopyCtasPerSm on every SM (2,048 threads, an SM's limit); the kernels stride over the rest.
unsigned apply_grid(int64_t units, int64_t words) {
    const int64_t want = max64(max64(units, (words + kCopyThreads - 1) / kCopyThreads), 1);
    return (unsigned)min64(want, (int64_t)kCopyCtasPerSm * device_sm_count());
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_pages_workspace_bytes(int32_t n_pages, int32_t n_seqs, int32_t n_items) {
    if (n_pages < 1 || n_seqs < 0 || n_items < 0) return 0;
    return (size_t)ws_layout(n_pages, n_seqs, n_items).total * 4;
}

tq_status tq_pages_extend(const tq_page_pool *pool, const int32_t *seqs, const int32_t *n_new, int32_t n,
                          void *workspace, size_t ws_bytes, void *stream) {
    tq_status st = check_pool(pool);
    if (st != TQ_OK) return st;
    if (n < 0) return TQ_ERR_INVALID_ARGUMENT;
    if (n == 0) return TQ_OK;
    if (!seqs || !n_new) return TQ_ERR_INVALID_ARGUMENT;
    st = check_ws(workspace, ws_bytes, ws_layout(pool->n_pages, pool->n_seqs, n));
    if (st != TQ_OK) return st;
    PdlConfig lc(dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream));
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, extend_kernel, pool_view(*pool), seqs, n_new, n,
                                         static_cast<int32_t *>(workspace)));
}

tq_status tq_pages_free(const tq_page_pool *pool, const int32_t *seqs, int32_t n, void *stream) {
    tq_status st = check_pool(pool);
    if (st != TQ_OK) return st;
    if (n < 0) return TQ_ERR_INVALID_ARGUMENT;
    if (n == 0) return TQ_OK;
    if (!seqs) return TQ_ERR_INVALID_ARGUMENT;
    PdlConfig lc(dim3((unsigned)n), dim3(128), 0, static_cast<cudaStream_t>(stream));
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, free_kernel, pool_view(*pool), seqs));
}

tq_status tq_pages_fork(const tq_page_pool *pool, const tq_cache *const *caches, int32_t n_caches,
                        const int32_t *parents, const int32_t *children, int32_t n, void *workspace,
                        size_t ws_bytes, void *stream) {
    tq_status st = check_pool(pool);
    if (st != TQ_OK) return st;
    if (n < 0) return TQ_ERR_INVALID_ARGUMENT;
    CopyCaches c;
    st = gather_caches(caches, n_caches, pool->page_tokens, pool->n_pages, &c);
    if (st != TQ_OK) return st;
    if (n == 0) return TQ_OK;
    if (!parents || !children) return TQ_ERR_INVALID_ARGUMENT;
    st = check_ws(workspace, ws_bytes, ws_layout(pool->n_pages, pool->n_seqs, n));
    if (st != TQ_OK) return st;
    int32_t *ws = static_cast<int32_t *>(workspace);
    const PoolView v = pool_view(*pool);
    PdlConfig plan(dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream));
    st = check_cuda(cudaLaunchKernelEx(&plan.cfg, fork_plan_kernel, v, parents, children, n, ws));
    if (st != TQ_OK) return st;
    PdlConfig apply(dim3(apply_grid((int64_t)n * c.n * c.units, (int64_t)n * v.cols)), dim3(kCopyThreads), 0,
                    static_cast<cudaStream_t>(stream));
    return check_cuda(cudaLaunchKernelEx(&apply.cfg, fork_apply_kernel, v, parents, children, n,
                                         static_cast<const int32_t *>(ws), c));
}

tq_status tq_pages_compact(const tq_page_pool *pool, const tq_page_pool *out, const tq_cache *const *caches,
                           int32_t n_caches, int32_t *n_used, void *workspace, size_t ws_bytes, void *stream) {
    tq_status st = check_pool(pool);
    if (st != TQ_OK) return st;
    st = check_pool(out);
    if (st != TQ_OK) return st;
    if (out->n_pages != pool->n_pages || out->page_tokens != pool->page_tokens || out->n_seqs != pool->n_seqs ||
        out->max_pages_per_seq != pool->max_pages_per_seq)
        return TQ_ERR_INVALID_ARGUMENT;
    CopyCaches c;
    st = gather_caches(caches, n_caches, pool->page_tokens, pool->n_pages, &c);
    if (st != TQ_OK) return st;
    st = check_ws(workspace, ws_bytes, ws_layout(pool->n_pages, pool->n_seqs, 0));
    if (st != TQ_OK) return st;
    int32_t *ws = static_cast<int32_t *>(workspace);
    const PoolView v = pool_view(*pool);
    PdlConfig plan(dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream));
    st = check_cuda(cudaLaunchKernelEx(&plan.cfg, compact_plan_kernel, v, ws, n_used));
    if (st != TQ_OK) return st;
    // at most half of the pages move
    PdlConfig apply(dim3(apply_grid((int64_t)(pool->n_pages / 2 + 1) * c.n * c.units,
                                    max64((int64_t)v.n_seqs * v.cols, v.n_pages))),
                    dim3(kCopyThreads), 0, static_cast<cudaStream_t>(stream));
    return check_cuda(cudaLaunchKernelEx(&apply.cfg, compact_apply_kernel, v, pool_view(*out),
                                         static_cast<const int32_t *>(ws), c));
}

tq_status tq_pages_copy(const tq_cache *const *caches, int32_t n_caches, const int32_t *src, const int32_t *dst,
                        const int32_t *rows, int32_t n, void *workspace, size_t ws_bytes, void *stream) {
    if (!caches || n_caches < 1 || !caches[0] || n < 0) return TQ_ERR_INVALID_ARGUMENT;
    const int page_tokens = caches[0]->page_tokens;
    if (page_tokens < 1) return TQ_ERR_INVALID_ARGUMENT;   // a contiguous cache has no pages
    int64_t n_pages = caches[0]->n_pages;
    for (int i = 1; i < n_caches && i < kMaxCaches; ++i)
        if (caches[i]) n_pages = min64(n_pages, caches[i]->n_pages);
    if (n_pages > INT32_MAX) return TQ_ERR_UNSUPPORTED;
    CopyCaches c;
    tq_status st = gather_caches(caches, n_caches, page_tokens, n_pages, &c);
    if (st != TQ_OK) return st;
    if (n == 0) return TQ_OK;
    if (!src || !dst) return TQ_ERR_INVALID_ARGUMENT;
    st = check_ws(workspace, ws_bytes, ws_layout(n_pages, 0, n));
    if (st != TQ_OK) return st;
    int32_t *ws = static_cast<int32_t *>(workspace);
    PdlConfig plan(dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream));
    st = check_cuda(cudaLaunchKernelEx(&plan.cfg, copy_plan_kernel, src, dst, rows, n, (int)n_pages, page_tokens, ws));
    if (st != TQ_OK) return st;
    PdlConfig apply(dim3(apply_grid((int64_t)n * c.n * c.units, 1)), dim3(kCopyThreads), 0,
                    static_cast<cudaStream_t>(stream));
    return check_cuda(cudaLaunchKernelEx(&apply.cfg, copy_apply_kernel, (int)n_pages, page_tokens, n,
                                         static_cast<const int32_t *>(ws), c));
}

}  // extern "C"
