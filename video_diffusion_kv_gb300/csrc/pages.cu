// pages.cu -- the pages of the paged caches: which sequence holds which page
// (fork, release, reserve), and moving what is in them (copy, compact).
//
// All state is the number of holders of each page, the block table and the
// lengths, on the device; pages are handed out lowest first, so every result
// follows from the arguments alone (the atomics below are sums and maxima of
// integers, whose order changes nothing).
#include "latent.cuh"
#include "paged.cuh"

namespace qvg {
namespace {

struct Batch {
    int B, page_log2;
    long long stride;
    int32_t *table, *kv_len;
    int32_t *refs;
    int num_pages;
    int *err;
    __device__ __forceinline__ int32_t *row(int b) const { return table + b * stride; }
    __device__ __forceinline__ long long pages(long long tokens) const { return (tokens + (1ll << page_log2) - 1) >> page_log2; }
};

constexpr int kForkThreads = 256;

// One block per pair.  What bounds it is latency: the pair's ids, the parent's
// length, its row, then the pages' counts, four dependent reads (3.5 us); a row of 750
// pages is three entries a thread (192 pairs of such rows: 5 us).
__global__ void __launch_bounds__(kForkThreads) k_pages_fork(Batch a, const int32_t *__restrict__ parents,
                                                             const int32_t *__restrict__ children, int n) {
    const int i = blockIdx.x, p = parents[i], c = children[i];
    bool bad = p < 0 || p >= a.B || c < 0 || c >= a.B;
    for (int j = threadIdx.x; j < n; j += kForkThreads) bad = bad || (j != i && children[j] == c) || parents[j] == c;
    long long pages = 0;
    int len = 0;
    if (!bad) {
        len = a.kv_len[p];
        pages = a.pages(len);
        bad = len < 0 || pages > a.stride || a.kv_len[c] != 0;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
        return;
    }
    const int32_t *from = a.row(p);
    int32_t *to = a.row(c);
    for (long long j = threadIdx.x; j < pages; j += kForkThreads) {
        const int page = from[j];
        to[j] = page;
        if (page >= 0 && page < a.num_pages)
            atomicAdd(a.refs + page, 1);
        else
            raise_error(a.err, QVG_ERR_INVALID_ARG);
    }
    if (threadIdx.x == 0) a.kv_len[c] = len;
}

// One block per sequence; bound as k_pages_fork.
__global__ void __launch_bounds__(kForkThreads) k_pages_release(Batch a, const int32_t *__restrict__ ids,
                                                                const int32_t *__restrict__ keep, int n) {
    const int i = blockIdx.x, b = ids[i];
    bool bad = b < 0 || b >= a.B;
    for (int j = threadIdx.x; j < n; j += kForkThreads) bad = bad || (j != i && ids[j] == b);
    long long pages = 0, left = 0;
    int to = 0;
    if (!bad) {
        const int len = a.kv_len[b];
        to = keep ? keep[i] : 0;
        pages = a.pages(len);
        left = a.pages(to);
        bad = len < 0 || to < 0 || to > len || pages > a.stride;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
        return;
    }
    const int32_t *row = a.row(b);
    for (long long j = left + threadIdx.x; j < pages; j += kForkThreads) {
        const int page = row[j];
        bool held = page >= 0 && page < a.num_pages;
        if (held && atomicSub(a.refs + page, 1) <= 0) {
            atomicAdd(a.refs + page, 1);
            held = false;
        }
        if (!held) raise_error(a.err, QVG_ERR_INVALID_ARG);
    }
    if (threadIdx.x == 0) a.kv_len[b] = to;
}

// ---- reserve ---------------------------------------------------------------------

constexpr int kReserve = 1024, kReserveWarps = kReserve / 32;
// Up to this many new tokens get their slots in k_pages_reserve itself, more in a grid of their own (64 sequences, reserved and
// cut again: 1024 tokens 5.6 us here, 7.2 in the grid; 4096: 11 both; 16,384: 18.7 and 11).
constexpr int kSlotsHere = 4096;

struct Reserve {
    const int32_t *cu_new;
    int n_new, total;
    int64_t *slots;
    int2 *copies;     // [B]
    int32_t *status;  // workspace: what the slots' kernel has to know
    int32_t *first;   // [B]: number of the sequence's first new page
    int32_t *list;    // [num_pages]: the free pages; before that, writers of a shared page
    int32_t *last;    // [num_pages]: the last of those writers
    __device__ __forceinline__ int start(int b) const { return cu_new ? cu_new[b] : b * n_new; }
};

// Largest b with at(b) <= k, in [0, n).
template <typename F>
__device__ __forceinline__ int holder(int n, int k, F at) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (at(mid) <= k)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void write_slot(const Batch &a, const Reserve &r, int i) {
    const int b = r.cu_new ? holder(a.B, i, [&](int m) { return r.cu_new[m]; }) : i / r.n_new;
    const int n = r.start(b + 1) - r.start(b);
    const int at = a.kv_len[b] - n + (i - r.start(b));  // (kv_len has grown)
    r.slots[i] = (static_cast<int64_t>(a.row(b)[at >> a.page_log2]) << a.page_log2) + (at & ((1 << a.page_log2) - 1));
}

// Exclusive sum over the block's threads; *all gets the total.
__device__ __forceinline__ long long block_scan(long long x, long long *s_warp, long long *all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) s_warp[warp] = y;
    __syncthreads();
    if (warp == 0) {
        const long long w = s_warp[lane];
        long long v = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long z = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += z;
        }
        s_warp[lane] = v - w;
        if (lane == 31) s_warp[32] = v;
    }
    __syncthreads();
    const long long got = s_warp[warp] + y - x;
    *all = s_warp[32];
    __syncthreads();
    return got;
}

// One block does the bookkeeping: each step needs the sums of the step before, and that chain is
// what bounds it (24 sequences, 330 pages: 8 us; 256 sequences, 53,214 pages: 17 us with cold
// caches).
//  1. What each sequence needs.  A shared last page is copied by each of its k
//     writers while another holder is left: with r holders, by all of them
//     where k < r, else by all but the last one.
//  2. Free pages, lowest first: a warp counts those of its part of the pool,
//     then writes them down from its place on.
//  3. Pages into the table; the new tokens' slots (many: k_pages_slots).
__global__ void __launch_bounds__(kReserve) k_pages_reserve(Batch a, Reserve r) {
    __shared__ long long s_warp[33];
    __shared__ int s_count[kReserveWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mask = (1 << a.page_log2) - 1;
    bool wrong = false, full = false;  // an argument, the room
    for (int b = tid; b < a.B; b += kReserve) {
        const int n = r.start(b + 1) - r.start(b), L = a.kv_len[b];
        int2 cp = make_int2(-1, -1);
        if (n < 0 || r.start(b) < 0 || r.start(b + 1) > r.total || L < 0) {
            wrong = true;
        } else if (a.pages(static_cast<long long>(L) + n) > a.stride || static_cast<long long>(L) + n > INT32_MAX) {
            full = true;
        } else if (n > 0 && (L & mask) != 0) {
            const int page = a.row(b)[L >> a.page_log2];
            if (page < 0 || page >= a.num_pages) {
                wrong = true;
            } else if (a.refs[page] > 1) {
                cp.x = page;
                r.list[page] = 0;
                r.last[page] = -1;
            }
        }
        r.copies[b] = cp;
    }
    if (tid == 0 && a.B > 0 && (r.start(0) != 0 || r.start(a.B) != r.total)) wrong = true;
    // (an invalid argument is reported before a lack of room)
    const bool invalid = __syncthreads_or(wrong), narrow = __syncthreads_or(full);
    long long need = 0;
    bool ok = !invalid && !narrow;
    if (ok) {
        for (int b = tid; b < a.B; b += kReserve) {
            const int page = r.copies[b].x;
            if (page >= 0) {
                atomicAdd(r.list + page, 1);
                atomicMax(r.last + page, b);
            }
        }
        __syncthreads();
        for (int b0 = 0; b0 < a.B; b0 += kReserve) {
            const int b = b0 + tid;
            int mine = 0;
            if (b < a.B) {
                const int n = r.start(b + 1) - r.start(b), L = a.kv_len[b], page = r.copies[b].x;
                mine = static_cast<int>(a.pages(static_cast<long long>(L) + n) - a.pages(L));
                if (page >= 0) {
                    if (r.list[page] >= a.refs[page] && r.last[page] == b)
                        r.copies[b].x = -1;  // the last holder keeps it
                    else
                        ++mine;
                }
            }
            long long all;
            const long long at = block_scan(mine, s_warp, &all);
            if (b < a.B) r.first[b] = static_cast<int>(min(need + at, static_cast<long long>(INT32_MAX)));
            need += all;
        }
        ok = need <= a.num_pages;
    }
    if (ok && need > 0) {
        const int part = ((a.num_pages + kReserveWarps - 1) / kReserveWarps + 31) & ~31;
        const int p0 = warp * part, p1 = min(a.num_pages, p0 + part);
        int c = 0;
#pragma unroll 8
        for (int p = p0 + lane; p < p1; p += 32) c += a.refs[p] == 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        if (lane == 0) s_count[warp] = c;
        __syncthreads();  // (also: the counts in `list` have been read)
        int at = 0, all = 0;
        for (int w = 0; w < kReserveWarps; ++w) {
            at += w < warp ? s_count[w] : 0;
            all += s_count[w];
        }
        ok = all >= need;
        if (ok) {
#pragma unroll 4
            for (int p = p0; p < p1; p += 32) {
                if (at >= need) break;
                const uint32_t free = __ballot_sync(0xFFFFFFFFu, p + lane < p1 && a.refs[p + lane] == 0);
                const int k = at + __popc(free & ((1u << lane) - 1u));
                if ((free >> lane & 1u) && k < need) r.list[k] = p + lane;
                at += __popc(free);
            }
        }
    }
    __syncthreads();
    if (!ok) {
        for (int b = tid; b < a.B; b += kReserve) r.copies[b] = make_int2(-1, -1);
        if (r.total <= kSlotsHere)
            for (int i = tid; i < r.total; i += kReserve) r.slots[i] = -1;
        if (tid == 0) {
            raise_error(a.err, invalid ? QVG_ERR_INVALID_ARG : QVG_ERR_CAPACITY);
            *r.status = 1;
        }
        return;
    }
    for (int k = tid; k < need; k += kReserve) {
        const int b = holder(a.B, k, [&](int m) { return r.first[m]; }), page = r.list[k], old = r.copies[b].x;
        const int have = static_cast<int>(a.pages(a.kv_len[b])), j = k - r.first[b] - (old >= 0 ? 1 : 0);
        a.row(b)[have + j] = page;  // j = -1: in the place of the shared one
        a.refs[page] = 1;
        if (j < 0) {
            atomicSub(a.refs + old, 1);
            r.copies[b].y = page;
        }
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kReserve) a.kv_len[b] += r.start(b + 1) - r.start(b);
    if (tid == 0) *r.status = 0;
    if (r.total > kSlotsHere) return;
    __syncthreads();
    for (int i = tid; i < r.total; i += kReserve) write_slot(a, r, i);
}

__global__ void __launch_bounds__(256) k_pages_slots(Batch a, Reserve r) {
    pdl_wait();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= r.total) return;
    if (*r.status)
        r.slots[i] = -1;
    else
        write_slot(a, r, i);
}

// ---- copy -------------------------------------------------------------------------

struct Buffers {
    int n, page_log2, num_pages;
    uint8_t *base[4];
    int heads[4], row_bytes[4];
    int blocks[4];  // k_pages_copy: blocks up to this buffer's end, of a page
    int *err;
    __device__ __forceinline__ long long page_bytes(int i) const { return (static_cast<long long>(heads[i]) * row_bytes[i]) << page_log2; }
};

constexpr int kCopyThreads = 256, kCopyEach = 4, kCopyBlock = kCopyThreads * kCopyEach * 16;

// blockIdx.x: a 16 KB piece of a page's bytes, blockIdx.y: pairs.  Four 16-byte
// loads a thread in flight.  Bound by HBM: 786 pages of 264 KB in 57 us, 7.3 TB/s read and
// written (part of what is written is still in L2 then).
__global__ void __launch_bounds__(kCopyThreads) k_pages_copy(const __grid_constant__ Buffers a, const int32_t *__restrict__ copies, int n) {
    int i = 0;
    while (static_cast<int>(blockIdx.x) >= a.blocks[i]) ++i;
    const long long bytes = a.page_bytes(i);
    const long long at = static_cast<long long>(blockIdx.x - (i ? a.blocks[i - 1] : 0)) * kCopyBlock + threadIdx.x * 16;
    for (int k = blockIdx.y; k < n; k += gridDim.y) {
        const int32_t *pair = copies + 2ll * k;
        const int from = pair[0], to = pair[1];
        if (from < 0 || to < 0) continue;
        if (from >= a.num_pages || to >= a.num_pages) {
            if (threadIdx.x == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
            continue;
        }
        const uint8_t *src = a.base[i] + from * bytes;
        uint8_t *dst = a.base[i] + to * bytes;
        uint4 v[kCopyEach];
#pragma unroll
        for (int e = 0; e < kCopyEach; ++e)
            if (at + e * (kCopyThreads * 16) < bytes) v[e] = __ldcs(reinterpret_cast<const uint4 *>(src + at + e * (kCopyThreads * 16)));
#pragma unroll
        for (int e = 0; e < kCopyEach; ++e)
            if (at + e * (kCopyThreads * 16) < bytes) *reinterpret_cast<uint4 *>(dst + at + e * (kCopyThreads * 16)) = v[e];
    }
}

// ---- compact ----------------------------------------------------------------------

constexpr int kMoveThreads = 256, kMoveEach = 4;
constexpr int kMostKept = INT32_MAX - 8 * kMoveThreads;  // of a sequence

struct Move {
    const int32_t *table, *first, *keep, *n_keep;
    long long table_stride, keep_stride;
    int slice;    // bytes of a row that one block moves, at most
    int jobs[4];  // blocks up to this buffer's end, of a sequence
};

// Bytes from the buffer's start to a batch's kept tokens' rows, from and to (-1: the token stays), three batches deep.
struct Slots {
    long long from[3][kMoveThreads], to[3][kMoveThreads];
};

// A block moves one slice of a head's rows of one sequence's tokens, in order, a
// batch of 256 pieces of `width` threads at a time: the batch is read, then
// written.  A token only moves down (keep ascends from `first` on), so what a
// batch writes over has been read in this batch or an earlier one, never is to be
// read in a later one, and the slices do not touch one another.
//   Reads run ahead: while a batch is written the next one's bytes are on their way, and the
// pages and numbers of the three after that.  What bounds it is this chain, about 1.5 us a
// batch, in the longest sequence.  (Bytes after their pages, pages after their numbers, a batch
// after the other: 265 us for 60,000 tokens of 8 heads of 128, which take 73 so; a third
// batch of bytes ahead costs the registers of a third block an SM, and was no faster.)
template <typename T>
__device__ __forceinline__ void move_rows(const Buffers &a, const Move &m, Slots &s, int b, int i, int h, int col, int width, int n) {
    const int per = kMoveThreads / width;  // rows side by side
    const int r = threadIdx.x / width, w = threadIdx.x - r * width;
    const int each = min(kMoveEach, width);  // a batch is at most 256 rows
    const int rows = per * each;
    const int32_t *row = m.table + b * m.table_stride, *keep = m.keep + b * m.keep_stride;
    const int first = m.first[b], mask = (1 << a.page_log2) - 1, rb = a.row_bytes[i];
    const long long heads = static_cast<long long>(a.heads[i]) << a.page_log2, lift = static_cast<long long>(h) << a.page_log2;
    uint8_t *const base = a.base[i] + col + w * static_cast<int>(sizeof(T));
    // Kept token batch * rows + threadIdx.x on its way to its slots: its number, its pages, then both.
    const bool has = static_cast<int>(threadIdx.x) < rows;
    int number = -1, page_from = -1, page_to = -1, x = -1;
    auto ask_number = [&](int batch) {
        const int k = batch * rows + threadIdx.x;
        number = has && k < n ? keep[k] : -1;
    };
    auto ask_pages = [&](int batch) {
        const int y = first + batch * rows + threadIdx.x;
        x = number == y ? -1 : number;  // (it stays where it is)
        if (x >= 0) {
            page_from = row[x >> a.page_log2];
            page_to = row[y >> a.page_log2];
        }
    };
    auto note = [&](int batch) {
        if (!has) return;
        const int y = first + batch * rows + threadIdx.x, e = batch % 3;
        // row (page, head, offset)
        s.from[e][threadIdx.x] = x < 0 ? 0 : (page_from * heads + lift + (x & mask)) * rb;
        s.to[e][threadIdx.x] = x < 0 ? -1 : (page_to * heads + lift + (y & mask)) * rb;
    };
    T v[2][kMoveEach];
    // (Loads are made whether their token moves or not, in place of branches that would wait for them.)
    const int mine = min(r, per - 1);
    auto read = [&](int batch, T(&x)[kMoveEach]) {
#pragma unroll
        for (int e = 0; e < kMoveEach; ++e)
            x[e] = *reinterpret_cast<const T *>(base + s.from[batch % 3][min(e, each - 1) * per + mine]);
    };
    auto write = [&](int batch, const T(&x)[kMoveEach]) {
#pragma unroll
        for (int e = 0; e < kMoveEach; ++e) {
            const long long t = s.to[batch % 3][min(e, each - 1) * per + mine];
            if (t >= 0 && e < each && r < per) *reinterpret_cast<T *>(base + t) = x[e];
        }
    };
    const int batches = (n + rows - 1) / rows;
    for (int k = 0; k < 2; ++k) {
        ask_number(k);
        ask_pages(k);
        note(k);
    }
    ask_number(2);
    ask_pages(2);
    ask_number(3);
    __syncthreads();
    read(0, v[0]);
    for (int j = 0; j < batches; j += 2) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (j + p >= batches) break;
            read(j + p + 1, v[p ^ 1]);  // (past the end: its slots are -1)
            note(j + p + 2);
            ask_pages(j + p + 3);
            ask_number(j + p + 4);
            __syncthreads();  // the batch has been read by all; the slots are there
            write(j + p, v[p]);
            __syncthreads();  // (its slots' place is the next batch's but two)
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads, 3) k_paged_compact(const __grid_constant__ Buffers a, const __grid_constant__ Move m) {
    __shared__ Slots s;
    const int b = blockIdx.y, n = m.n_keep[b], first = m.first[b];
    bool bad = n < 0 || n > m.keep_stride || first < 0;
    if (!bad) {
        const int32_t *row = m.table + b * m.table_stride, *keep = m.keep + b * m.keep_stride;
        const long long room = m.table_stride << a.page_log2;
#pragma unroll 8
        for (int k = threadIdx.x; k < n; k += kMoveThreads) {
            const int x = keep[k];
            const bool off = x < (k ? keep[k - 1] + 1ll : static_cast<long long>(first)) || x >= room || x < first;
            // (where keep ascends, first + k does not pass x)
            const bool past = static_cast<long long>(first) + k > x;
            const int p = off ? -1 : row[x >> a.page_log2], to = off || past ? 0 : row[(first + k) >> a.page_log2];
            bad = bad || p < 0 || p >= a.num_pages || to < 0 || to >= a.num_pages;
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
        return;
    }
    int i = 0;
    while (static_cast<int>(blockIdx.x) >= m.jobs[i]) ++i;
    const int job = blockIdx.x - (i ? m.jobs[i - 1] : 0), rb = a.row_bytes[i];
    if (rb >= 16) {
        const int slices = (rb + m.slice - 1) / m.slice, h = job / slices, col = (job - h * slices) * m.slice;
        move_rows<uint4>(a, m, s, b, i, h, col, min(m.slice, rb - col) / 16, n);
    } else if (rb == 4) {
        move_rows<uint32_t>(a, m, s, b, i, job, 0, 1, n);
    } else if (rb == 2) {
        move_rows<uint16_t>(a, m, s, b, i, job, 0, 1, n);
    } else {
        move_rows<uint8_t>(a, m, s, b, i, job, 0, 1, n);
    }
}

// ---- host ---------------------------------------------------------------------------

bool misaligned(const void *p, uintptr_t to) { return !p || reinterpret_cast<uintptr_t>(p) % to != 0; }
constexpr int kMostPairs = 1 << 20;  // each block of a fork or release looks at all pairs
bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

qvg_status check_sequences(const qvg_page_pool *pool, const qvg_sequences *s) {
    if (!pool || !s || pool->num_pages < 1 || s->B < 0 || s->table_stride < 1 || !page_size_ok(s->page_size)) return QVG_ERR_INVALID_ARG;
    if (misaligned(pool->refs, 4)) return QVG_ERR_INVALID_ARG;
    if (s->B > 0 && (misaligned(s->table, 4) || misaligned(s->kv_len, 4))) return QVG_ERR_INVALID_ARG;
    return QVG_OK;
}

Batch batch(const qvg_page_pool *pool, const qvg_sequences *s) {
    Batch a{};
    a.B = s->B;
    a.page_log2 = __builtin_ctz(static_cast<unsigned>(s->page_size));
    a.stride = s->table_stride;
    a.table = s->table;
    a.kv_len = s->kv_len;
    a.refs = pool->refs;
    a.num_pages = pool->num_pages;
    a.err = device_error_word();
    return a;
}

qvg_status check_rows(const qvg_page_rows *r) {
    if (!r || r->n < 1 || r->n > 4 || r->num_pages < 1 || !page_size_ok(r->page_size)) return QVG_ERR_INVALID_ARG;
    for (int i = 0; i < r->n; ++i) {
        const int rb = r->row_bytes[i];
        if (misaligned(r->base[i], 16) || r->heads[i] < 1) return QVG_ERR_INVALID_ARG;
        if (rb != 1 && rb != 2 && rb != 4 && (rb < 16 || rb % 16 != 0)) return QVG_ERR_INVALID_ARG;
        // (its bytes are worked out in 64 bits)
        if (static_cast<int64_t>(r->heads[i]) * rb > INT64_MAX / (static_cast<int64_t>(r->page_size) * r->num_pages)) return QVG_ERR_INVALID_ARG;
    }
    return QVG_OK;
}

Buffers buffers(const qvg_page_rows *r) {
    Buffers a{};
    a.n = r->n;
    a.page_log2 = __builtin_ctz(static_cast<unsigned>(r->page_size));
    a.num_pages = r->num_pages;
    for (int i = 0; i < r->n; ++i) {
        a.base[i] = static_cast<uint8_t *>(r->base[i]);
        a.heads[i] = r->heads[i];
        a.row_bytes[i] = r->row_bytes[i];
    }
    a.err = device_error_word();
    return a;
}

size_t reserve_bytes(int num_pages, int B) { return 4 * (4 + (static_cast<size_t>(B) + 3) / 4 * 4 + 2 * static_cast<size_t>(num_pages)); }

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_pages_fork(const qvg_page_pool *pool, const qvg_sequences *seqs, const int32_t *parents,
                          const int32_t *children, int32_t n, void *stream) {
    const qvg_status s = check_sequences(pool, seqs);
    if (s != QVG_OK) return s;
    if (n < 0) return QVG_ERR_INVALID_ARG;
    if (n == 0) return QVG_OK;
    if (seqs->B == 0 || misaligned(parents, 4) || misaligned(children, 4)) return QVG_ERR_INVALID_ARG;
    if (n > kMostPairs) return QVG_ERR_UNSUPPORTED;
    k_pages_fork<<<n, kForkThreads, 0, static_cast<cudaStream_t>(stream)>>>(batch(pool, seqs), parents, children, n);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

qvg_status qvg_pages_release(const qvg_page_pool *pool, const qvg_sequences *seqs, const int32_t *ids,
                             const int32_t *keep, int32_t n, void *stream) {
    const qvg_status s = check_sequences(pool, seqs);
    if (s != QVG_OK) return s;
    if (n < 0) return QVG_ERR_INVALID_ARG;
    if (n == 0) return QVG_OK;
    if (seqs->B == 0 || misaligned(ids, 4) || (keep && misaligned(keep, 4))) return QVG_ERR_INVALID_ARG;
    if (n > kMostPairs) return QVG_ERR_UNSUPPORTED;
    k_pages_release<<<n, kForkThreads, 0, static_cast<cudaStream_t>(stream)>>>(batch(pool, seqs), ids, keep, n);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

qvg_status qvg_pages_workspace_size(int32_t num_pages, int32_t B, size_t *bytes) {
    if (!bytes || num_pages < 1 || B < 0) return QVG_ERR_INVALID_ARG;
    *bytes = reserve_bytes(num_pages, B);
    return QVG_OK;
}

qvg_status qvg_pages_reserve(const qvg_page_pool *pool, const qvg_sequences *seqs, const int32_t *cu_new, int32_t n_new,
                             int32_t total, int64_t *slots, int32_t *copies, void *workspace, size_t ws_bytes,
                             void *stream) {
    const qvg_status s = check_sequences(pool, seqs);
    if (s != QVG_OK) return s;
    if (total < 0 || (cu_new && misaligned(cu_new, 4))) return QVG_ERR_INVALID_ARG;
    if (!cu_new && (n_new < 0 || static_cast<int64_t>(n_new) * seqs->B != total)) return QVG_ERR_INVALID_ARG;
    if (seqs->B == 0) return total == 0 ? QVG_OK : QVG_ERR_INVALID_ARG;
    if (misaligned(copies, 8) || (total > 0 && misaligned(slots, 8))) return QVG_ERR_INVALID_ARG;
    // (the kernels' 32-bit indices step past the last element)
    if (std::max({seqs->B, total, pool->num_pages}) > INT32_MAX - 2 * kReserve) return QVG_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < reserve_bytes(pool->num_pages, seqs->B) || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
        return QVG_ERR_WORKSPACE;
    const Batch a = batch(pool, seqs);
    Reserve r{};
    r.cu_new = cu_new;
    r.n_new = n_new;
    r.total = total;
    r.slots = slots;
    r.copies = reinterpret_cast<int2 *>(copies);
    r.status = static_cast<int32_t *>(workspace);
    r.first = r.status + 4;
    r.list = r.first + (static_cast<size_t>(seqs->B) + 3) / 4 * 4;
    r.last = r.list + pool->num_pages;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    k_pages_reserve<<<1, kReserve, 0, st>>>(a, r);
    QVG_LAUNCH_CHECK();
    if (total > kSlotsHere) {
        const cudaError_t e = launch_pdl(k_pages_slots, dim3(ceil_div(total, 256)), dim3(256), 0, st, a, r);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            note_cuda_error(e);
            return QVG_ERR_CUDA;
        }
    }
    return QVG_OK;
}

qvg_status qvg_paged_rows(const qvg_paged *cache, qvg_page_rows *rows) {
    if (!rows) return QVG_ERR_INVALID_ARG;
    const qvg_status s = check_paged(cache, false);
    if (s != QVG_OK) return s;
    *rows = qvg_page_rows{};
    rows->page_size = cache->page_size;
    rows->num_pages = cache->num_pages;
    rows->n = 4;
    uint8_t *const base[4] = {cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales};
    for (int i = 0; i < 4; ++i) {
        rows->base[i] = base[i];
        rows->heads[i] = cache->H;
        rows->row_bytes[i] = i < 2 ? cache->d * cache->bits / 8 : cache->bits == 8 ? 1 : cache->d / 32;
    }
    return QVG_OK;
}

qvg_status qvg_latent_rows(const qvg_latent *cache, qvg_page_rows *rows) {
    if (!rows) return QVG_ERR_INVALID_ARG;
    const qvg_status s = check_latent(cache, false);
    if (s != QVG_OK) return s;
    *rows = qvg_page_rows{};
    rows->page_size = cache->page_size;
    rows->num_pages = cache->num_pages;
    rows->n = cache->dr ? 2 : 1;
    for (int i = 0; i < rows->n; ++i) {
        rows->base[i] = i ? cache->kr : cache->c;
        rows->heads[i] = 1;
        rows->row_bytes[i] = 2 * (i ? cache->dr : cache->dc);
    }
    return QVG_OK;
}

qvg_status qvg_pages_copy(const qvg_page_rows *rows, const int32_t *copies, int32_t n, void *stream) {
    const qvg_status s = check_rows(rows);
    if (s != QVG_OK) return s;
    if (n < 0) return QVG_ERR_INVALID_ARG;
    if (n == 0) return QVG_OK;
    if (misaligned(copies, 4)) return QVG_ERR_INVALID_ARG;
    if (n > INT32_MAX - 65535) return QVG_ERR_UNSUPPORTED;
    Buffers a = buffers(rows);
    int64_t blocks = 0;
    for (int i = 0; i < a.n; ++i) {
        const int64_t bytes = static_cast<int64_t>(a.heads[i]) * a.row_bytes[i] * rows->page_size;
        blocks += (bytes + kCopyBlock - 1) / kCopyBlock;
        if (blocks > INT32_MAX) return QVG_ERR_UNSUPPORTED;
        a.blocks[i] = static_cast<int>(blocks);
    }
    k_pages_copy<<<dim3(static_cast<unsigned>(blocks), std::min(n, 65535)), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, copies, n);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

qvg_status qvg_paged_compact(const qvg_page_rows *rows, const int32_t *table, int32_t table_stride, int32_t B,
                             const int32_t *first, const int32_t *keep, int32_t keep_stride, const int32_t *n_keep,
                             void *stream) {
    const qvg_status s = check_rows(rows);
    if (s != QVG_OK) return s;
    if (B < 0 || table_stride < 1 || keep_stride < 0) return QVG_ERR_INVALID_ARG;
    // (the kernel's 32-bit numbers of kept tokens step up to five batches past the last one)
    if (B > 65535 || keep_stride > kMostKept) return QVG_ERR_UNSUPPORTED;
    if (B == 0 || keep_stride == 0) return QVG_OK;
    if (misaligned(table, 4) || misaligned(first, 4) || misaligned(keep, 4) || misaligned(n_keep, 4)) return QVG_ERR_INVALID_ARG;
    const Buffers a = buffers(rows);
    Move m{};
    m.table = table;
    m.first = first;
    m.keep = keep;
    m.n_keep = n_keep;
    m.table_stride = table_stride;
    m.keep_stride = keep_stride;
    // Slices of 128 bytes, or down to 32 where those are fewer blocks than two an SM.
    int64_t jobs = 0;
    for (m.slice = 128;; m.slice /= 2) {
        jobs = 0;
        for (int i = 0; i < a.n; ++i) {
            jobs += static_cast<int64_t>(a.heads[i]) * ceil_div(a.row_bytes[i], m.slice);
            if (jobs > INT32_MAX) return QVG_ERR_UNSUPPORTED;
            m.jobs[i] = static_cast<int>(jobs);
        }
        if (m.slice == 32 || jobs * B >= 2 * sm_count_current()) break;
    }
    k_paged_compact<<<dim3(static_cast<unsigned>(jobs), B), kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, m);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

}  // extern "C"
