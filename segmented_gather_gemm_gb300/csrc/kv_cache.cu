// The paged K/V cache's bookkeeping and data movement: append (commit), fork,
// free, compact, page copies.  See include/csgmv.h for what each does.
//
// Every call but the copies is a plan and a move.  The plan is one cluster of
// kPlanCtas CTAs: it decides everything (which requests are sound, which pages
// are given out) from page_refs alone, with prefix sums and no atomic whose
// order could show, so the same state gives the same pages.  The move kernel
// is launched behind it (programmatic dependent launch) and streams the data
// with 16-byte loads, several in flight a thread.  Whole pages go at HBM's rate;
// a commit's rows do not (DRAM 52 to 63 % busy): a warp's unit is one row in one
// layer, and for each it finds the request and follows four dependent loads.
//
// Measured (device time): a commit of 256 requests' accepted tokens into 32
// layers of 8 heads of 128 (292 MB) 58.7 us, of which the plan 8 us and the
// move 5 TB/s; of 4 requests 10.8 us, the chain of loads of both.  Fork, free
// and compaction of 512 sequences (4.3 GB) 678 us, 6.4 TB/s; of 16 small ones
// 20 us, five launches one behind the other.
#include "serving.cuh"

namespace csgmv {
namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 152 * 16;

// The cache as the kernels see it, with scratch cut into its arrays.
struct Kv {
    uint16_t *k, *v;
    int32_t *table, *lens, *refs, *status;
    int32_t *head;                // counters (H* below)
    int32_t *pa, *pb, *pc;        // [num_pages]
    int32_t *sa, *sb, *sc, *sd;   // [max_seqs + 1]
    int32_t *mark, *mark2;        // [max_seqs]
    int64_t layer_stride, page_stride, head_stride, token_stride;
    int layers, pages, ps, ps_shift, heads, d, seqs, max_pages;
};

Kv view(const csgmv_kv_cache &c) {
    Kv k;
    k.k = static_cast<uint16_t *>(c.k_pages);
    k.v = static_cast<uint16_t *>(c.v_pages);
    k.table = c.page_table;
    k.lens = c.seq_lens;
    k.refs = c.page_refs;
    k.status = c.status;
    int32_t *s = c.scratch;
    k.head = s;
    s += kKvHeader;
    k.pa = s;
    k.pb = k.pa + c.num_pages;
    k.pc = k.pb + c.num_pages;
    s = k.pc + c.num_pages;
    k.sa = s;
    k.sb = k.sa + c.max_seqs + 1;
    k.sc = k.sb + c.max_seqs + 1;
    k.sd = k.sc + c.max_seqs + 1;
    k.mark = k.sd + c.max_seqs + 1;
    k.mark2 = k.mark + c.max_seqs;
    k.layer_stride = c.layer_stride;
    k.page_stride = c.page_stride;
    k.head_stride = c.head_stride;
    k.token_stride = c.token_stride;
    k.layers = c.num_layers;
    k.pages = c.num_pages;
    k.ps = c.page_size;
    k.ps_shift = __builtin_ctz((unsigned)c.page_size);
    k.heads = c.num_kv_heads;
    k.d = c.head_dim;
    k.seqs = c.max_seqs;
    k.max_pages = c.max_pages_per_seq;
    return k;
}

enum { kHRows = 0, kHMoves = 1, kHLive = 2 };  // entries of Kv::head

// Copies ntok token slots of every head between two pages of one layer of one
// pool (addresses of the pages' first elements).  `nt` threads, this one `ti`,
// U loads in flight each.
template <int U>
__device__ __forceinline__ void copy_page(const Kv &c, const uint16_t *src, uint16_t *dst, int ntok, int ti, int nt) {
    const unsigned cw = (unsigned)c.d >> 3;  // 16-byte chunks of a row
    const unsigned n = (unsigned)c.heads * ntok * cw;
    for (unsigned i0 = ti; i0 < n; i0 += U * nt) {
        uint4 v[U];
        unsigned off[U];  // a page spans less than 2^31 elements
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned i = i0 + u * nt;
            if (i < n) {
                const unsigned row = i / cw, h = row / (unsigned)ntok;
                off[u] = h * (unsigned)c.head_stride + (row - h * ntok) * (unsigned)c.token_stride + (i - row * cw) * 8;
                v[u] = ld_stream16(src + off[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * nt < n) st_stream16(dst + off[u], v[u]);
    }
}

// --------------------------------------------------------------- free pages
// Counts of the pages for which something holds, by cluster: warp w of the
// kPlanCtas * kPlanWarps warps owns a contiguous stretch of the pages.
struct Stretch {
    int lo, hi;
};
__device__ __forceinline__ Stretch stretch(int pages) {
    const int gw = (int)cluster_rank() * kPlanWarps + (threadIdx.x >> 5), nw = kPlanCtas * kPlanWarps;
    const int per = ((pages + nw - 1) / nw + 31) & ~31;
    const int lo = min(pages, gw * per);
    return {lo, min(pages, lo + per)};
}

struct PlanSmem {
    int warp[33];
    int cta_total;
    int a;
    long long scan[33];
};

// This CTA's part of the count (sm.warp: what is ahead of each warp in the CTA,
// sm.cta_total).
template <typename F>
__device__ void count_mine(PlanSmem &sm, Stretch s, F want) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int mine = 0;
    for (int p = s.lo; p < s.hi; p += 32) mine += __popc(__ballot_sync(kFullMask, p + lane < s.hi && want(p + lane)));
    if (lane == 0) sm.warp[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const int w = sm.warp[lane], inc = warp_scan(w);
        sm.warp[lane] = inc - w;
        if (lane == 31) sm.cta_total = inc;
    }
    __syncthreads();
}
// The pages counted ahead of this warp's stretch, and the total.  Behind a
// cluster barrier that follows count_mine(); no CTA may leave before another
// one.
__device__ __forceinline__ int count_before(PlanSmem &sm, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)cluster_rank();
    const int t = lane < kPlanCtas ? dsmem_ld_i32(dsmem_addr(&sm.cta_total, lane)) : 0;
    *total = warp_sum(t);
    return sm.warp[warp] + warp_sum(lane < rank ? t : 0);
}

// Writes the `need` lowest free pages, in order, to list.  `before` counts the
// free pages ahead of the warp's stretch.
__device__ __forceinline__ void list_free(const Kv &c, Stretch s, int before, int need, int32_t *list) {
    const int lane = threadIdx.x & 31;
    for (int p = s.lo; p < s.hi && before < need; p += 32) {
        const bool f = p + lane < s.hi && c.refs[p + lane] == 0;
        const unsigned m = __ballot_sync(kFullMask, f);
        const int at = before + __popc(m & ((1u << lane) - 1u));
        if (f && at < need) list[at] = p + lane;
        before += __popc(m);
    }
}

__device__ __forceinline__ int pages_of(const Kv &c, int tokens) { return (tokens + c.ps - 1) >> c.ps_shift; }

// ------------------------------------------------------------------- commit
// Plan.  sa[b]: first appended row of request b in the batch's order (sa[bs]
// the total), sb[b]: the sequence's length before, sc / sd[b]: source and
// destination page of a copy on write, or -1; mark: the request that owns a
// sequence slot; pa: the pages given out.  A warp of the cluster a request: what
// the plan takes is a chain of dependent loads, so it is kept as short as the
// requests allow.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
commit_plan(Kv c, CommitParams p) {
    __shared__ PlanSmem sm;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank();
    const int gw = rank * kPlanWarps + warp, gt = rank * kPlanThreads + tid;
    constexpr int kAllWarps = kPlanCtas * kPlanWarps, kAllThreads = kPlanCtas * kPlanThreads;
    const Stretch s = stretch(c.pages);
    auto slot_of = [&](int b) { return p.seq_slots ? p.seq_slots[b] : b; };
    auto in = [&](int q) { return q >= 0 && q < c.seqs; };
    if (p.seq_slots) {  // (without slots none can come twice)
        for (int b = gt; b < p.bs; b += kAllThreads)
            if (in(slot_of(b))) c.mark[slot_of(b)] = INT32_MAX;
        cluster_sync();
        for (int b = gt; b < p.bs; b += kAllThreads)
            if (in(slot_of(b))) atomicMin(&c.mark[slot_of(b)], b);
        cluster_sync();
    }
    // is the request sound?  sa: its rows, sb: the length before, sd: pages it needs
    for (int b = gw; b < p.bs; b += kAllWarps) {
        const int q = slot_of(b), add = p.accept_len[b];
        const int lo = p.tree_indptr[b], hi = p.tree_indptr[b + 1];
        int bad = 0, old = 0;
        bool wrong = false;
        if (p.accept_index)  // read beside the rest: a bad count is cut to what is there
            for (int j = lane; j < min(add, p.accept_width); j += 32) {
                const int node = p.accept_index[(int64_t)b * p.accept_width + j];
                wrong |= node < 0 || node >= hi - lo;
            }
        if (!in(q) || (p.seq_slots && c.mark[q] != b)) bad = CSGMV_KV_STATUS_BAD_SEQ;
        if (!bad) {
            old = c.lens[q];
            if (add < 0 || lo < 0 || hi < lo || hi > p.num_tokens || old < 0 || old > c.max_pages * c.ps ||
                (p.accept_index ? add > p.accept_width : add > hi - lo))
                bad = CSGMV_KV_STATUS_BAD_LENS;
            else if (add > c.max_pages * c.ps - old)
                bad = CSGMV_KV_STATUS_CAPACITY;
        }
        if (__any_sync(kFullMask, wrong) && !bad) bad = CSGMV_KV_STATUS_BAD_TREE;
        int cow = -1;
        if (!bad && add > 0 && (old & (c.ps - 1))) {
            const int last = c.table[(int64_t)q * c.max_pages + (old >> c.ps_shift)];
            if (last < 0 || last >= c.pages) bad = CSGMV_KV_STATUS_BAD_PAGE;
            else if (c.refs[last] > 1) cow = last;
        }
        if (lane == 0) {
            if (bad) atomicOr(c.status, bad);
            const int rows = bad ? 0 : add;
            c.sa[b] = rows;
            c.sb[b] = old;
            c.sc[b] = rows ? cow : -1;
            c.sd[b] = rows ? pages_of(c, old + rows) - pages_of(c, old) + (cow >= 0) : 0;
        }
    }
    count_mine(sm, s, [&](int q) { return c.refs[q] == 0; });
    cluster_sync();
    if (rank == 0) {  // running sums of rows and of pages over the requests
        long long sum = 0;
        for (int b0 = 0; b0 < p.bs; b0 += kPlanThreads) {
            const int b = b0 + tid;
            long long t;
            const long long own = b < p.bs ? (long long)c.sa[b] << 32 | (unsigned)c.sd[b] : 0;
            const long long pre = sum + block_scan_ex(own, sm.scan, &t);
            if (b < p.bs) {
                c.sa[b] = (int)(pre >> 32);
                c.sd[b] = (int)pre;  // first entry of the page list
            }
            sum += t;
        }
        if (tid == 0) {
            c.sa[p.bs] = (int)(sum >> 32);
            sm.a = (int)sum;
        }
    }
    int nfree;
    const int before = count_before(sm, &nfree);
    cluster_sync();
    const int need = dsmem_ld_i32(dsmem_addr(&sm.a, 0));
    const bool fits = need <= nfree;
    if (fits) list_free(c, s, before, need, c.pa);
    __threadfence();
    cluster_sync();
    if (gt == 0) {
        if (!fits) atomicOr(c.status, CSGMV_KV_STATUS_CAPACITY);
        c.head[kHRows] = fits ? c.sa[p.bs] : 0;
    }
    if (!fits) return;
    // hand the pages out
    for (int b = gw; b < p.bs; b += kAllWarps) {
        const int add = c.sa[b + 1] - c.sa[b], q = slot_of(b), old = c.sb[b], cow = c.sc[b];
        int first = c.sd[b];
        if (add == 0) continue;
        int32_t *row = c.table + (int64_t)q * c.max_pages;
        __syncwarp();
        if (cow >= 0) {
            if (lane == 0) {
                const int to = c.pa[first];
                row[old >> c.ps_shift] = to;
                c.refs[to] = 1;
                atomicSub(&c.refs[cow], 1);
                c.sd[b] = to;
            }
            ++first;
        }
        const int have = pages_of(c, old), want = pages_of(c, old + add);
        for (int i = have + lane; i < want; i += 32) {
            const int pg = c.pa[first + i - have];
            row[i] = pg;
            c.refs[pg] = 1;
        }
        if (lane == 0) c.lens[q] = old + add;
    }
}

// Move: a warp copies an appended row's K and V of one layer; then CTAs copy
// the pages that were shared.
__global__ void __launch_bounds__(kMoveThreads, 4) commit_move(Kv c, CommitParams p) {
    griddep_wait();
    const int rows = c.head[kHRows];
    if (rows == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = kMoveThreads / 32;
    const unsigned cw = (unsigned)c.d >> 3, n = (unsigned)c.heads * cw;
    const int64_t units = (int64_t)rows * c.layers;
    for (int64_t u = (int64_t)blockIdx.x * nw + warp; u < units; u += (int64_t)gridDim.x * nw) {
        const int layer = (int)(u / rows), r = (int)(u - (int64_t)layer * rows);
        int lo = 0;  // the last request whose first row is at most r: 32 are tried at once
        for (int len = p.bs; len > 1;) {
            const int step = (len + 31) >> 5, at = lane * step;
            const int k = 31 - __clz(__ballot_sync(kFullMask, at < len && c.sa[lo + at] <= r));
            lo += k * step;
            len = min(step, len - k * step);
        }
        const int j = r - c.sa[lo], q = p.seq_slots ? p.seq_slots[lo] : lo;
        const int node = p.accept_index ? p.accept_index[(int64_t)lo * p.accept_width + j] : j;
        const int pos = c.sb[lo] + j, page = c.table[(int64_t)q * c.max_pages + (pos >> c.ps_shift)];
        const int64_t so = layer * p.layer_stride + (int64_t)(p.tree_indptr[lo] + node) * p.token_stride;
        const int64_t to = layer * c.layer_stride + page * c.page_stride + (pos & (c.ps - 1)) * c.token_stride;
        constexpr int U = 4;
        for (unsigned i0 = lane; i0 < n; i0 += U * 32) {
            uint4 vk[U], vv[U];
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const unsigned i = i0 + x * 32, h = i / cw, e = (i - h * cw) * 8;
                if (i < n) {
                    vk[x] = ld_stream16(p.k_new + so + h * p.head_stride + e);
                    vv[x] = ld_stream16(p.v_new + so + h * p.head_stride + e);
                }
            }
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const unsigned i = i0 + x * 32, h = i / cw, e = (i - h * cw) * 8;
                if (i < n) {
                    st_stream16(c.k + to + h * c.head_stride + e, vk[x]);
                    st_stream16(c.v + to + h * c.head_stride + e, vv[x]);
                }
            }
        }
    }
    for (int b = blockIdx.x; b < p.bs; b += gridDim.x) {
        const int from = c.sc[b];
        if (from < 0) continue;
        const int to = c.sd[b], ntok = c.sb[b] & (c.ps - 1);
        for (int l = 0; l < c.layers; ++l) {
            const int64_t a = l * c.layer_stride + from * c.page_stride, z = l * c.layer_stride + to * c.page_stride;
            copy_page<2>(c, c.k + a, c.k + z, ntok, threadIdx.x, kMoveThreads);
            copy_page<2>(c, c.v + a, c.v + z, ntok, threadIdx.x, kMoveThreads);
        }
    }
}

// --------------------------------------------------------------------- fork
// Plan.  sa[i]: the parent's length, or -1 for an entry that is left out;
// sb[i]: the fresh page of its partial last page (an index into pa, then the
// page), or -1.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
fork_plan(Kv c, const int32_t *parents, const int32_t *children, int n) {
    __shared__ PlanSmem sm;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, rank = (int)cluster_rank();
    const Stretch s = stretch(c.pages);
    if (rank == 0) {
        auto in = [&](int q) { return q >= 0 && q < c.seqs; };
        for (int i = tid; i < n; i += kPlanThreads) {
            if (in(children[i])) c.mark[children[i]] = INT32_MAX, c.mark2[children[i]] = 0;
            if (in(parents[i])) c.mark2[parents[i]] = 0;
        }
        __syncthreads();
        for (int i = tid; i < n; i += kPlanThreads) {
            if (in(children[i])) atomicMin(&c.mark[children[i]], i);
            if (in(parents[i])) c.mark2[parents[i]] = 1;
        }
        __syncthreads();
        int need0 = 0;
        for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
            const int i = i0 + tid;
            int len = -1, bad = 0;
            if (i < n) {
                const int a = parents[i], b = children[i];
                if (!in(a) || !in(b) || c.mark[b] != i || c.mark2[b] || c.lens[b] != 0) bad = CSGMV_KV_STATUS_BAD_SEQ;
                else if (c.lens[a] < 0 || c.lens[a] > c.max_pages * c.ps) bad = CSGMV_KV_STATUS_BAD_LENS;
                else len = c.lens[a];
                if (len > 0 && (len & (c.ps - 1))) {
                    const int last = c.table[(int64_t)a * c.max_pages + (len >> c.ps_shift)];
                    if (last < 0 || last >= c.pages) bad = CSGMV_KV_STATUS_BAD_PAGE, len = -1;
                }
                if (bad) atomicOr(c.status, bad);
            }
            const int part = len > 0 && (len & (c.ps - 1)) ? 1 : 0;
            int t;
            const int at = block_scan_ex(part, reinterpret_cast<int *>(sm.scan), &t);
            if (i < n) {
                c.sa[i] = len;
                c.sb[i] = part ? need0 + at : -1;
            }
            need0 += t;
        }
        if (tid == 0) sm.a = need0;
    }
    count_mine(sm, s, [&](int q) { return c.refs[q] == 0; });
    cluster_sync();
    int nfree;
    const int before = count_before(sm, &nfree), need = dsmem_ld_i32(dsmem_addr(&sm.a, 0));
    const bool fits = need <= nfree;
    if (fits) list_free(c, s, before, need, c.pa);
    __threadfence();
    cluster_sync();
    if (rank != 0) return;
    if (!fits && tid == 0) atomicOr(c.status, CSGMV_KV_STATUS_CAPACITY);
    for (int i = tid; i < n; i += kPlanThreads) {
        if (!fits) {
            c.sa[i] = -1;
        } else if (c.sa[i] >= 0) {
            if (c.sb[i] >= 0) {
                const int pg = c.pa[c.sb[i]];
                c.sb[i] = pg;
                c.refs[pg] = 1;
            }
            c.lens[children[i]] = c.sa[i];
        }
    }
}

// Move: block (i, 0) shares entry i's whole pages, block (i, 1 + 2 l + kv)
// copies its partial page in layer l of K or V.
__global__ void __launch_bounds__(kMoveThreads) fork_move(Kv c, const int32_t *parents, const int32_t *children) {
    griddep_wait();
    const int i = blockIdx.x, len = c.sa[i];
    if (len <= 0) return;
    const int32_t *from = c.table + (int64_t)parents[i] * c.max_pages;
    const int full = len >> c.ps_shift, ntok = len & (c.ps - 1), fresh = c.sb[i];
    if (blockIdx.y == 0) {
        int32_t *to = c.table + (int64_t)children[i] * c.max_pages;
        for (int j = threadIdx.x; j < full; j += kMoveThreads) {
            const int pg = from[j];
            to[j] = pg;
            if (pg >= 0 && pg < c.pages) atomicAdd(&c.refs[pg], 1);
            else atomicOr(c.status, CSGMV_KV_STATUS_BAD_PAGE);
        }
        if (ntok && threadIdx.x == 0) to[full] = fresh;
        return;
    }
    if (!ntok) return;
    const int y = blockIdx.y - 1;
    uint16_t *pool = (y & 1) ? c.v : c.k;
    const int64_t l = (int64_t)(y >> 1) * c.layer_stride;
    copy_page<8>(c, pool + l + from[full] * c.page_stride, pool + l + fresh * c.page_stride, ntok, threadIdx.x,
              kMoveThreads);
}

// --------------------------------------------------------------------- free
// A block a sequence.  A page is given up by whoever takes its table entry
// (atomic exchange), so a sequence listed twice gives each page up once.
__global__ void __launch_bounds__(kMoveThreads) free_pages(Kv c, const int32_t *seqs, const int32_t *keep_lens) {
    griddep_wait();
    const int q = seqs[blockIdx.x], keep = keep_lens ? keep_lens[blockIdx.x] : 0;
    if (q < 0 || q >= c.seqs || keep < 0) {
        if (threadIdx.x == 0) atomicOr(c.status, keep < 0 ? CSGMV_KV_STATUS_BAD_LENS : CSGMV_KV_STATUS_BAD_SEQ);
        return;
    }
    __shared__ int len_s;
    if (threadIdx.x == 0) len_s = *reinterpret_cast<volatile int32_t *>(&c.lens[q]);
    __syncthreads();
    const int len = len_s;
    if (len < 0 || len > c.max_pages * c.ps) {
        if (threadIdx.x == 0) atomicOr(c.status, CSGMV_KV_STATUS_BAD_LENS);
        return;
    }
    if (keep >= len) return;
    int32_t *row = c.table + (int64_t)q * c.max_pages;
    for (int j = pages_of(c, keep) + threadIdx.x; j < pages_of(c, len); j += kMoveThreads) {
        const int pg = atomicExch(&row[j], -1);
        if (pg == -1) continue;
        if (pg < 0 || pg >= c.pages) {
            atomicOr(c.status, CSGMV_KV_STATUS_BAD_PAGE);
        } else if (atomicSub(&c.refs[pg], 1) <= 0) {
            atomicAdd(&c.refs[pg], 1);
            atomicOr(c.status, CSGMV_KV_STATUS_BAD_PAGE);
        }
    }
    if (threadIdx.x == 0) atomicMin(&c.lens[q], keep);
}

// ------------------------------------------------------------------ compact
// Plan.  With `live` live pages, a live page p >= live moves.  Its rank from
// the top, live - 1 - (live pages below p), and a hole's rank from the bottom,
// p - (live pages below p), need nothing but the running count, and the k-th
// mover from the bottom is the (moves - 1 - k)-th from the top.
// pa[k]: k-th hole; pb[r]: r-th mover from the top; pc[p]: its rank.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) compact_plan(Kv c) {
    __shared__ PlanSmem sm;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const Stretch s = stretch(c.pages);
    count_mine(sm, s, [&](int q) { return c.refs[q] > 0; });
    cluster_sync();
    int live, before = count_before(sm, &live);
    cluster_arrive();
    for (int p = s.lo; p < s.hi; p += 32) {
        const int q = p + lane;
        const bool l = q < s.hi && c.refs[q] > 0;
        const unsigned m = __ballot_sync(kFullMask, l);
        const int below = before + __popc(m & ((1u << lane) - 1u));
        if (q < s.hi) {
            if (l && q >= live) {
                c.pb[live - 1 - below] = q;
                c.pc[q] = live - 1 - below;
            } else if (!l && q < live) {
                c.pa[q - below] = q;
            }
            if (q == live - 1) c.head[kHMoves] = live - below - (l ? 1 : 0);
        }
        before += __popc(m);
    }
    if (cluster_rank() == 0 && threadIdx.x == 0) {
        c.head[kHLive] = live;
        if (live == 0) c.head[kHMoves] = 0;
    }
    cluster_wait();  // no CTA leaves while another reads its count
}

// Move: CTAs rewrite the sequences' rows of the page table, then copy pages,
// one layer of K or V at a time; the copy of layer 0's K also moves the count.
__global__ void __launch_bounds__(kMoveThreads) compact_move(Kv c) {
    griddep_wait();
    const int moves = c.head[kHMoves], live = c.head[kHLive];
    if (moves <= 0) return;
    for (int q = blockIdx.x; q < c.seqs; q += gridDim.x) {
        const int len = c.lens[q];
        const int n = len > 0 ? min(pages_of(c, len), c.max_pages) : 0;
        int32_t *row = c.table + (int64_t)q * c.max_pages;
        for (int j = threadIdx.x; j < n; j += kMoveThreads) {
            const int pg = row[j];
            if (pg >= live && pg < c.pages) {
                const int r = c.pc[pg];
                // a page that no sequence should hold (count 0) has no rank
                if (r >= 0 && r < moves && c.pb[r] == pg) row[j] = c.pa[moves - 1 - r];
            }
        }
    }
    const int64_t units = (int64_t)moves * c.layers * 2;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int k = (int)(u / (2 * c.layers)), y = (int)(u - (int64_t)k * 2 * c.layers);
        const int from = c.pb[moves - 1 - k], to = c.pa[k];
        uint16_t *pool = (y & 1) ? c.v : c.k;
        const int64_t l = (int64_t)(y >> 1) * c.layer_stride;
        copy_page<8>(c, pool + l + from * c.page_stride, pool + l + to * c.page_stride, c.ps, threadIdx.x, kMoveThreads);
        if (y == 0 && threadIdx.x == 0) {
            c.refs[to] = c.refs[from];
            c.refs[from] = 0;
        }
    }
}

// -------------------------------------------------------------- page copies
__global__ void __launch_bounds__(kMoveThreads) copy_pages(Kv c, const int32_t *src, const int32_t *dst, int n) {
    griddep_wait();
    const int64_t units = (int64_t)n * c.layers * 2;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int k = (int)(u / (2 * c.layers)), y = (int)(u - (int64_t)k * 2 * c.layers);
        const int from = src[k], to = dst[k];
        if (from < 0 || from >= c.pages || to < 0 || to >= c.pages) {
            if (threadIdx.x == 0) atomicOr(c.status, CSGMV_KV_STATUS_BAD_PAGE);
            continue;
        }
        if (from == to) continue;
        uint16_t *pool = (y & 1) ? c.v : c.k;
        const int64_t l = (int64_t)(y >> 1) * c.layer_stride;
        copy_page<8>(c, pool + l + from * c.page_stride, pool + l + to * c.page_stride, c.ps, threadIdx.x, kMoveThreads);
    }
}

dim3 grid_for(int64_t units) {
    return dim3((unsigned)(units < 1 ? 1 : units < kMoveCtas ? units : kMoveCtas));
}

}  // namespace

cudaError_t launch_kv_commit(const csgmv_kv_cache &kv, const CommitParams &p, cudaStream_t stream) {
    const Kv c = view(kv);
    cudaError_t e = launch_kernel(commit_plan, dim3(kPlanCtas), kPlanThreads, 0, stream, 0, true, c, p);
    if (e != cudaSuccess) return e;
    // at most every row of the batch, eight (row, layer) pairs a block
    return launch_kernel(commit_move, grid_for((p.num_tokens * c.layers + 7) / 8), kMoveThreads, 0, stream, 0, true, c,
                         p);
}

cudaError_t launch_kv_fork(const csgmv_kv_cache &kv, const int32_t *parents, const int32_t *children, int n,
                           cudaStream_t stream) {
    const Kv c = view(kv);
    cudaError_t e =
        launch_kernel(fork_plan, dim3(kPlanCtas), kPlanThreads, 0, stream, 0, true, c, parents, children, n);
    if (e != cudaSuccess) return e;
    return launch_kernel(fork_move, dim3((unsigned)n, 1 + 2 * (unsigned)c.layers), kMoveThreads, 0, stream, 0, true, c,
                         parents, children);
}

cudaError_t launch_kv_free(const csgmv_kv_cache &kv, const int32_t *seqs, const int32_t *keep, int n,
                           cudaStream_t stream) {
    return launch_kernel(free_pages, dim3((unsigned)n), kMoveThreads, 0, stream, 0, true, view(kv), seqs, keep);
}

cudaError_t launch_kv_compact(const csgmv_kv_cache &kv, cudaStream_t stream) {
    const Kv c = view(kv);
    cudaError_t e = launch_kernel(compact_plan, dim3(kPlanCtas), kPlanThreads, 0, stream, 0, true, c);
    if (e != cudaSuccess) return e;
    return launch_kernel(compact_move, grid_for((int64_t)c.pages * c.layers * 2), kMoveThreads, 0, stream, 0, true, c);
}

cudaError_t launch_kv_copy(const csgmv_kv_cache &kv, const int32_t *src, const int32_t *dst, int n,
                           cudaStream_t stream) {
    const Kv c = view(kv);
    return launch_kernel(copy_pages, grid_for((int64_t)n * c.layers * 2), kMoveThreads, 0, stream, 0, true, c, src,
                         dst, n);
}

}  // namespace csgmv
