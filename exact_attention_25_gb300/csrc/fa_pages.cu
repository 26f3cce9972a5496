// Pages of the paged cache: copying them, moving the rows that a sequence keeps together, and the
// bookkeeping of which page belongs to whom.
//
// Copies and moves change no value: codes and exponent bytes go as they are, and both are bound by HBM (each
// byte read and written once).
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

namespace fa {

namespace {

// ---- clusters
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; what each did in memory before is seen by all after.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit word of CTA `rank`'s shared memory, at this CTA's address of it.
__device__ __forceinline__ int cluster_word(const int* p, int rank)
{
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return static_cast<int>(v);
}

template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), int ctas_of_cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                           A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas_of_cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------------------ copies of pages
constexpr int kCopyThreads = 128;

// A warp takes 16 rows of one entry and head, K and V: 2 KB each at d = 128, all loads before the stores.  Bound by HBM: 4000
// pages of 64 rows, 8 heads, d = 128, in 155 us, 6.8 TB/s; 64 partly filled ones in 3.5 us, launch and two dependent reads.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) fa_cache_copy_kernel(const PageCopyParams p)
{
    constexpr int N = D / 32;  // 16-byte words of a lane for one tensor
    dependent_begin();
    const long long w = static_cast<long long>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int parts = 1 << (p.page_shift - 4);
    const int part = static_cast<int>(w & (parts - 1));
    const long long rest = w >> (p.page_shift - 4);
    const int n = static_cast<int>(rest / p.Hkv), hk = static_cast<int>(rest - static_cast<long long>(n) * p.Hkv);
    if (n >= p.n) return;
    const int src = p.copies[3ll * n], dst = p.copies[3ll * n + 1];
    const int rows = min(max(p.copies[3ll * n + 2], 0) - 16 * part, 16);  // of this warp
    if (rows <= 0 || src < 0 || src >= p.src_pages || dst < 0 || dst >= p.dst_pages) return;
    const long long from = ((static_cast<long long>(src) * p.Hkv + hk) << p.page_shift) + 16 * part;
    const long long to = ((static_cast<long long>(dst) * p.Hkv + hk) << p.page_shift) + 16 * part;
    if (!in_extent(from + rows - 1, 1, p.src_rows, p.status) || !in_extent(to + rows - 1, 1, p.dst_rows, p.status)) return;
    uint4 x[2][N];
    const int words = rows * (D / 16);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const uint4* s = reinterpret_cast<const uint4*>((z ? p.src_v : p.src_k) + from * D);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (32 * i + lane < words) x[z][i] = s[32 * i + lane];
    }
    // exponents: lanes 0-15 K's, 16-31 V's
    const int r = lane & 15;
    uint8_t e = 0;
    if (r < rows) e = (lane < 16 ? p.src_ke : p.src_ve)[from + r];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        uint4* d = reinterpret_cast<uint4*>((z ? p.dst_v : p.dst_k) + to * D);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (32 * i + lane < words) d[32 * i + lane] = x[z][i];
    }
    if (r < rows) (lane < 16 ? p.dst_ke : p.dst_ve)[to + r] = e;
}

// ------------------------------------------------------------------------------ compaction
// Row start + i of a sequence becomes what its row start + keep[i] was, in place, for rising keep (so
// keep[i] >= i).  One cluster takes one sequence, head and tensor; a step of it R rows for each of
// its CTAs.  A step's rows are written when all CTAs have read the step's; the rows that later steps read
// lie behind those that it writes (keep[i] >= i), so S - 1 steps are on their way to shared memory meanwhile.
// Every thread copies its own 16 bytes of its rows in and out again, so that memory needs no barrier of its own.
//
// Bound by HBM (each moved row read and written once): 8 sequences that keep 24 K of 32 K rows and less, 8 heads,
// d = 128, 109 us, 5.1 TB/s (102 on the same rows again and again, as the figures that follow).  What that takes is many rows
// under way: with the rows in registers and one step ahead 247 us, with the ring but the table's entries looked up when
// needed 113.  A CTA's step of 64 rows by 128 threads, three stages, seven
// CTAs an SM; four stages 106 us, five 122; 128 rows by 256 threads 104 (and 40 rows 8.4 us, here 6.2); writes a step later
// than the barrier's arrival, so that nobody waits there, the same.
template <int D, int THREADS, int U, int S>
__global__ void __launch_bounds__(THREADS) fa_cache_compact_kernel(const CompactParams p)
{
    constexpr int LR = D / 16;          // lanes of a row
    constexpr int RP = THREADS / LR;    // rows of a pass
    constexpr int R = U * RP;           // rows of a CTA and step
    static_assert(U <= LR, "a lane looks up each of the U rows");
    extern __shared__ __align__(16) uint8_t ring[];
    dependent_begin();
    const int nc = p.cluster, rank = static_cast<int>(cluster_rank());
    const int id = static_cast<int>(blockIdx.x) / nc;
    const int z = id & 1, hk = (id >> 1) % p.Hkv, b = (id >> 1) / p.Hkv;
    int first;
    const int n = packed_rows(p.cu, b, p.total, p.max_keep, first);
    const int start = p.start[b];
    const int g = threadIdx.x / LR, l = threadIdx.x % LR;
    uint8_t* codes = z ? p.v : p.k;
    uint8_t* exps = z ? p.ve : p.ke;
    const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
    const int in_page = (1 << p.page_shift) - 1;
    const int* table = p.table + static_cast<long long>(b) * p.max_pages;
    auto page_at = [&](long long pos) { return pos >= 0 && pos < room ? table[pos >> p.page_shift] : -1; };
    auto row_at = [&](int page, long long pos) -> long long {
        if (page < 0 || page >= p.num_pages) return -1;
        return ((static_cast<long long>(page) * p.Hkv + hk) << p.page_shift) + (pos & in_page);
    };
    const int steps = (n + R * nc - 1) / (R * nc);
    // Lane l < U of a row's lanes looks after the row's place of pass l: what is kept there (read two steps ahead),
    // the pages where from and where to (a step ahead), and the exponent byte.
    auto place = [&](int t) { return (t * nc + rank) * R + l * RP + g; };
    auto kept = [&](int t) {
        const int i = place(t);
        return l < U && t < steps && i < n ? p.keep[first + i] : -1;
    };
    long long to[S];
    uint8_t e[S];
    int k = -1, k_next = kept(0), page_from = -1, page_to = -1;
    auto ahead = [&](int t) {  // the pages of step t, what step t + 1 keeps
        k = k_next;
        k_next = kept(t + 1);
        page_from = page_to = -1;
        if (k >= 0 && k != place(t)) {
            page_from = page_at(static_cast<long long>(start) + k);
            page_to = page_at(static_cast<long long>(start) + place(t));
        }
    };
    ahead(0);
    uint8_t* const mine = ring + 16 * threadIdx.x;
    // Step t's rows on their way to stage s; those that stay where they are, and rows or places that the table does
    // not have, are left alone (to = -1).
    auto load = [&](int t, int s) {
        long long from = row_at(page_from, static_cast<long long>(start) + k);
        to[s] = row_at(page_to, static_cast<long long>(start) + place(t));
        if (to[s] < 0 || from < 0 || !in_extent(from, 1, p.rows, p.status) || !in_extent(to[s], 1, p.rows, p.status))
            from = to[s] = -1;
        else
            e[s] = exps[from];
        ahead(t + 1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = __shfl_sync(0xffffffffu, from, u, LR);
            if (r >= 0)
                cp_async16(mine + 16 * THREADS * (U * s + u), codes + r * D + 16 * l);
        }
    };
    auto store = [&](int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = __shfl_sync(0xffffffffu, to[s], u, LR);
            if (r >= 0)
                *reinterpret_cast<uint4*>(codes + r * D + 16 * l) =
                    *reinterpret_cast<const uint4*>(mine + 16 * THREADS * (U * s + u));
        }
        if (to[s] >= 0) exps[to[s]] = e[s];
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        if (s < steps) load(s, s);
        cp_async_commit();
    }
#pragma unroll 1
    for (int t0 = 0; t0 < steps; t0 += S) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int t = t0 + s;
            if (t >= steps) break;
            cp_async_wait<S - 2>();
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            if (t + S - 1 < steps) load(t + S - 1, (s + S - 1) % S);
            cp_async_commit();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            store(s);
        }
    }
}

// ------------------------------------------------------------------------------ bookkeeping
// Who holds which page.  refs[p] counts the table's entries with page p; 0 is a free page.  One call gives every
// slot its next table row: the pages of the first `kept` rows of its source slot, then fresh pages up to
// its new length; a partly filled last page that others hold too is replaced by a fresh one, which `copies`
// says.  Fresh pages are the lowest-numbered free ones, in the order of the slots.  All or nothing: where
// there are too few, refs and table stay.
//
// A few microseconds of latencies: a scan of refs, a table entry for each page that changes hands, and the
// order of the steps below, each of which needs all of the one before.  So one cluster does it,
// with a hardware barrier (some 0.3 us) between the steps, where a grid would need a launch each, 1 to 2 us.  (For pools of a
// million pages that would pay; it was not built.)  A CTA's threads
// share out all entries of its slots, found by a search in the slots' sums: with a warp to a slot the longest
// ones of 1024 slots (10 of 100 replaced, pages of 16 of up to 32 K tokens, 1.1 M pages) kept the others waiting, 85 us in
// place of 44; now 35, of which 11 for the fresh pages (9 K sectors of counts written by each SM), 9 and 7 for the
// entries (an atomic or a store each), 3 for the counts.  64 slots 7.8 us, 256 beams with 31 K shared entries 15.7.
constexpr int kPagesThreads = 1024;
constexpr int kPagesWarps = kPagesThreads / 32;

struct Slot {
    int source;         // -1: none
    bool own;           // continues its own pages
    int p_old, p_kept, p_new;
    int part;           // rows of the last kept page, if it is to be written on, else 0
};

__device__ __forceinline__ int pages_of(const PagesParams& p, int rows)
{
    const long long n = (static_cast<long long>(max(rows, 0)) + (1 << p.page_shift) - 1) >> p.page_shift;
    return static_cast<int>(min(n, static_cast<long long>(p.max_pages)));
}

__device__ __forceinline__ Slot slot_at(const PagesParams& p, int b)
{
    Slot s;
    s.source = p.source[b];
    if (s.source < 0 || s.source >= p.slots) s.source = -1;
    s.own = s.source == b;
    const int kept = s.source < 0 ? 0 : min(max(p.kept[b], 0), max(p.seqlens[s.source], 0));
    const int next = max(p.new_lens[b], kept);
    s.p_old = pages_of(p, p.seqlens[b]);
    s.p_kept = pages_of(p, kept);
    s.p_new = pages_of(p, next);
    s.part = next > kept ? kept & ((1 << p.page_shift) - 1) : 0;
    if (static_cast<long long>(s.p_kept) << p.page_shift < kept) s.part = 0;  // (past the table's room)
    return s;
}

__device__ __forceinline__ bool is_page(const PagesParams& p, int id) { return id >= 0 && id < p.num_pages; }

// Element i of a tensor of `extent` ints (checked builds; -1 past it).
__device__ __forceinline__ int int_at(const PagesParams& p, const int* t, long long i, long long extent)
{
    return in_extent(i, 1, extent, p.status) ? t[i] : -1;
}
__device__ __forceinline__ void put_int(const PagesParams& p, int* t, long long i, long long extent, int v)
{
    if (in_extent(i, 1, extent, p.status)) t[i] = v;
}
// A page's count and v.
__device__ __forceinline__ void add_ref(const PagesParams& p, int id, int v)
{
    if (is_page(p, id) && in_extent(id, 1, p.refs_ext, p.status)) atomicAdd(p.refs + id, v);
}
__device__ __forceinline__ void put_copy(const PagesParams& p, int b, int from, int to, int rows)
{
    if (!in_extent(b, 1, p.slot_ext, p.status)) return;
    p.copies[3ll * b] = from;
    p.copies[3ll * b + 1] = to;
    p.copies[3ll * b + 2] = rows;
}

// The block's sum of v, in all threads; s_part: 32 words, free again after the next __syncthreads.
__device__ __forceinline__ unsigned block_sum(unsigned v, unsigned* s_part)
{
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, s_part[threadIdx.x & 31]);
}

// The sum of v over the threads before, and over all; s_part as above.
__device__ __forceinline__ unsigned block_before(unsigned v, unsigned* s_part, unsigned& all)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned up = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const unsigned x = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += x;
    }
    if (lane == 31) s_part[warp] = up;
    __syncthreads();
    const unsigned sum = s_part[lane];
    all = __reduce_add_sync(0xffffffffu, sum);
    return __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0u) + up - v;
}

__global__ void __launch_bounds__(kPagesThreads) fa_pages_update_kernel(const PagesParams p)
{
    __shared__ unsigned s_part[kPagesWarps];
    __shared__ int s_free[kPagesWarps];
    __shared__ int s_totals[2];  // of this CTA: pages its slots need, free pages of its part of refs
    // of a batch of slots: entries up to the slot's last, and what they are
    __shared__ unsigned s_end[kPagesThreads];
    __shared__ int4 s_slot[kPagesThreads];
    dependent_begin();
    const int nc = p.cluster, rank = static_cast<int>(cluster_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int M = p.max_pages;
    // this CTA's slots, and this warp's pages (a multiple of 4)
    const int per_cta = (p.slots + nc - 1) / nc;
    const int b0 = static_cast<int>(min(static_cast<long long>(rank) * per_cta, static_cast<long long>(p.slots)));
    const int b1 = min(b0 + per_cta, p.slots);
    const int batch = min(kPagesThreads, max(1, (1 << 30) / M));  // slots taken at once: fewer than 2^31 entries
    const int per_warp = ((p.num_pages + nc * kPagesWarps - 1) / (nc * kPagesWarps) + 3) & ~3;
    const long long w0 = static_cast<long long>(rank * kPagesWarps + warp) * per_warp;
    const int g0 = static_cast<int>(min(w0, static_cast<long long>(p.num_pages)));
    const int g1 = static_cast<int>(min(w0 + per_warp, static_cast<long long>(p.num_pages)));

    // a thread's slot of the batch that begins at c0; the first batch's is kept
    const Slot none{-1, true, 0, 0, 0, 0};
    const Slot first = tid < batch && b0 + tid < b1 ? slot_at(p, b0 + tid) : none;
    auto slot_of = [&](int c0) {
        return c0 == b0 ? first : (tid < batch && c0 + tid < b1 ? slot_at(p, c0 + tid) : none);
    };
    // its last kept page, if the slot writes on in it (the table stands until step 4)
    auto last_of = [&](const Slot& s) {
        return s.part ? int_at(p, p.table, static_cast<long long>(s.source) * M + s.p_kept - 1, p.table_ext) : -1;
    };
    const int first_last = last_of(first);
    // All threads over all of the batch's `all` entries, four at once; find(e, k): the slot (of the batch) that has
    // entry e, as its k-th.
    int half = 1;  // half of the slots of a batch, up to a power of two
    while (2 * half < min(batch, b1 - b0)) half *= 2;
    auto find = [&](unsigned e, unsigned& k) {
        int lo = -1;  // the last slot whose entries end at or before e
#pragma unroll 1
        for (int step = half; step > 0; step /= 2)
            if (s_end[lo + step] <= e) lo += step;
        k = lo >= 0 ? e - s_end[lo] : e;
        return lo + 1;
    };

    // ---- 1: the entries that go, and those that are shared anew (undo: the other way round)
    auto count_entries = [&](int sign) {
#pragma unroll 1
        for (int c0 = b0; c0 < b1; c0 += batch) {
            const Slot s = slot_of(c0);
            const int from = s.own ? min(s.p_kept, s.p_old) : 0, fork = s.own ? 0 : s.p_kept;
            const unsigned n = static_cast<unsigned>(s.p_old - from) + static_cast<unsigned>(fork);
            unsigned all;
            const unsigned before = block_before(n, s_part, all);
            s_end[tid] = before + n;
            s_slot[tid] = make_int4(from, s.p_old - from, s.source, 0);
            __syncthreads();
#pragma unroll 1
            for (unsigned e0 = tid; e0 < all; e0 += 4 * kPagesThreads) {
                int id[4], delta[4];
                int* stage[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const unsigned e = e0 + u * kPagesThreads;
                    id[u] = -1;
                    stage[u] = nullptr;
                    if (e >= all) continue;
                    unsigned k;
                    const int i = find(e, k);
                    const int4 w = s_slot[i];
                    const long long row = static_cast<long long>(c0 + i) * M;
                    if (k < static_cast<unsigned>(w.y)) {
                        delta[u] = -sign;
                        id[u] = int_at(p, p.table, row + w.x + k, p.table_ext);
                    } else {
                        delta[u] = sign;
                        id[u] = int_at(p, p.table, static_cast<long long>(w.z) * M + (k - w.y), p.table_ext);
                        if (in_extent(row + (k - w.y), 1, p.table_ext, p.status)) stage[u] = p.stage + row + (k - w.y);
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (stage[u] != nullptr) *stage[u] = id[u];
                    add_ref(p, id[u], delta[u]);
                }
            }
            __syncthreads();
        }
    };
    // The counts of pages i to i + 3 (past the warp's part: not free).
    auto counts_at = [&](int i) {
        if (i + 4 <= g1) return __ldcg(reinterpret_cast<const int4*>(p.refs + i));
        int4 r = make_int4(1, 1, 1, 1);
        if (i < g1) r.x = __ldcg(p.refs + i);
        if (i + 1 < g1) r.y = __ldcg(p.refs + i + 1);
        if (i + 2 < g1) r.z = __ldcg(p.refs + i + 2);
        return r;
    };
    auto free_of = [](int4 r) { return (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0); };
    // free pages of this warp's part
    auto count_free = [&]() {
        int n = 0, i = g0 + 4 * lane;
#pragma unroll 1
        for (; i - 4 * lane + 1024 <= g1; i += 1024) {
            int4 r[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) r[u] = __ldcg(reinterpret_cast<const int4*>(p.refs + i + 128 * u));
#pragma unroll
            for (int u = 0; u < 8; ++u) n += free_of(r[u]);
        }
#pragma unroll 4
        for (; i < g1; i += 128) n += free_of(counts_at(i));
        return __reduce_add_sync(0xffffffffu, n);
    };
    count_entries(1);
    cluster_sync();

    // ---- 2: how many pages each slot needs, how many are free
    int need_all = 0;
#pragma unroll 1
    for (int c0 = b0; c0 < b1; c0 += batch) {
        const int b = c0 + tid;
        const Slot s = slot_of(c0);
        int need = s.p_new - s.p_kept, last = -1;
        if (s.part) {
            last = c0 == b0 ? first_last : last_of(s);
            if (!is_page(p, last) || !in_extent(last, 1, p.refs_ext, p.status) || __ldcg(p.refs + last) < 2) last = -1;
            need += last >= 0;
        }
        // places of the fresh pages among this CTA's
        unsigned all;
        const unsigned before = block_before(need, s_part, all);
        if (tid < batch && b < b1) {
            put_int(p, p.offset, b, p.slot_ext, need_all + before);
            put_int(p, p.shared_last, b, p.slot_ext, last);
        }
        need_all += all;
        __syncthreads();
    }
    const int mine = count_free();
    if (lane == 0) s_free[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const int f = __reduce_add_sync(0xffffffffu, s_free[lane]);
        if (lane == 0) {
            s_totals[0] = need_all;
            s_totals[1] = f;
        }
    }
    cluster_sync();

    // ---- 3: the lowest free pages, as many as are needed, in order
    int need_before = 0, need_total = 0, free_before = 0, free_total = 0;
    {
        // (every warp reads the others' totals, lane r those of CTA r)
        const int a = lane < nc ? cluster_word(&s_totals[0], lane) : 0;
        const int f = lane < nc ? cluster_word(&s_totals[1], lane) : 0;
        need_total = __reduce_add_sync(0xffffffffu, a);
        free_total = __reduce_add_sync(0xffffffffu, f);
        need_before = __reduce_add_sync(0xffffffffu, lane < rank ? a : 0);
        free_before = __reduce_add_sync(0xffffffffu, lane < rank ? f : 0);
    }
    if (need_total > free_total) {
        count_entries(-1);
        for (int b = b0 + tid; b < b1; b += kPagesThreads) put_copy(p, b, -1, -1, 0);
        cluster_sync();
        const int left = count_free();
        const int f = block_sum(lane == 0 ? left : 0, s_part);
        if (tid == 0) s_totals[1] = f;
        cluster_sync();
        if (rank == 0 && warp == 0) {
            const int all = __reduce_add_sync(0xffffffffu, lane < nc ? cluster_word(&s_totals[1], lane) : 0);
            if (lane == 0) {
                p.counts[0] = need_total - free_total;
                p.counts[1] = all;
            }
        }
        cluster_sync();  // (no CTA leaves while its words may be read)
        return;
    }
    {
        int at = free_before + __reduce_add_sync(0xffffffffu, lane < warp ? s_free[lane] : 0);
        // 32 pages a vote (512 at once, with a scan of the lanes' counts, took three times the instructions: 1.1 M pages in
        // 39 us in place of 35)
#pragma unroll 1
        for (int i0 = g0 + lane; i0 - lane < g1 && at < need_total; i0 += 256) {
            int r[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) r[u] = i0 + 32 * u < g1 ? __ldcg(p.refs + i0 + 32 * u) : 1;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const unsigned here = __ballot_sync(0xffffffffu, r[u] == 0);
                const int to = at + __popc(here & ((1u << lane) - 1));
                if (r[u] == 0 && to < need_total) {
                    put_int(p, p.fresh, to, p.refs_ext, i0 + 32 * u);
                    put_int(p, p.refs, i0 + 32 * u, p.refs_ext, 1);
                }
                at += __popc(here);
            }
        }
    }
    if (rank == 0 && tid == 0) {
        p.counts[0] = 0;
        p.counts[1] = free_total - need_total;
    }
    cluster_sync();

    // ---- 4: the slots' rows, those entries that change
#pragma unroll 1
    for (int c0 = b0; c0 < b1; c0 += batch) {
        const int b = c0 + tid;
        const Slot s = slot_of(c0);
        int last = -1, fresh = 0, from = 0;
        unsigned n = 0;
        if (tid < batch && b < b1) {
            last = int_at(p, p.shared_last, b, p.slot_ext);
            fresh = need_before + int_at(p, p.offset, b, p.slot_ext);
            const int page = last >= 0 && in_extent(fresh, 1, p.refs_ext, p.status) ? __ldcg(p.fresh + fresh) : -1;
            if (last >= 0) add_ref(p, last, -1);
            put_copy(p, b, last, page, last >= 0 ? s.part : 0);
            from = s.own ? s.p_kept - (last >= 0) : 0;
            n = max(max(s.p_new, s.p_old) - from, 0);
        }
        unsigned all;
        const unsigned before = block_before(n, s_part, all);
        s_end[tid] = before + n;
        // (from the last kept page on, if it is replaced, the entry's place less z is its fresh page's)
        s_slot[tid] = make_int4(from, s.p_kept - (last >= 0), s.p_new, fresh);
        __syncthreads();
#pragma unroll 1
        for (unsigned e0 = tid; e0 < all; e0 += 4 * kPagesThreads) {
            int id[4];
            int* to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const unsigned e = e0 + u * kPagesThreads;
                to[u] = nullptr;
                id[u] = -1;
                if (e >= all) continue;
                unsigned k;
                const int i = find(e, k);
                const int4 w = s_slot[i];
                const int at = w.x + static_cast<int>(k);
                const long long row = static_cast<long long>(c0 + i) * M + at;
                if (!in_extent(row, 1, p.table_ext, p.status)) continue;
                to[u] = p.table + row;
                if (at < w.y)
                    id[u] = p.stage[row];
                else if (at < w.z && in_extent(w.w + static_cast<long long>(at - w.y), 1, p.refs_ext, p.status))
                    id[u] = __ldcg(p.fresh + w.w + (at - w.y));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (to[u] != nullptr) *to[u] = id[u];
        }
        __syncthreads();
    }
}

}  // namespace

template <int D>
static cudaError_t launch_copy(const PageCopyParams& p, cudaStream_t st)
{
    const long long warps = (static_cast<long long>(p.n) * p.Hkv) << (p.page_shift - 4);
    return launch_dependent(fa_cache_copy_kernel<D>, dim3(static_cast<unsigned>((warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32))),
                            dim3(kCopyThreads), 0, st, p);
}

cudaError_t launch_cache_copy(int d, const PageCopyParams& p, cudaStream_t st)
{
    return d == 64 ? launch_copy<64>(p, st) : launch_copy<128>(p, st);
}

template <int D, int THREADS, int U, int S>
static cudaError_t launch_compact_as(CompactParams p, cudaStream_t st, int cluster)
{
    constexpr int kSmem = 16 * THREADS * U * S;
    static_assert(kSmem <= 48 * 1024, "without an opt-in");
    p.cluster = cluster;
    return launch_cluster(fa_cache_compact_kernel<D, THREADS, U, S>, cluster, dim3(2 * p.B * p.Hkv * cluster), dim3(THREADS),
                          kSmem, st, p);
}

template <int D>
static cudaError_t launch_compact(const CompactParams& p, cudaStream_t st, int num_sms)
{
    // rows of a CTA's step: 128 threads, one pass for a few, four for many (up to 6 of 24 rows in replays 6.3 us, in
    // large steps 8.4; up to 225 rows 6.3, in the small steps 18.5)
    constexpr int kFew = 128 / (D / 16), kMany = 4 * 128 / (D / 16);
    if (p.max_keep <= kFew) return launch_compact_as<D, 128, 1, 2>(p, st, 1);
    // as many CTAs to a cluster as the SMs hold at once, and have rows (8 sequences of up to 24 K rows kept, the
    // same ones again and again: 102 us; one CTA each 238)
    const long long units = 2ll * p.B * p.Hkv;
    int cluster = 1;
    while (cluster < 8 && 2 * units * cluster <= 8 * num_sms && p.max_keep > cluster * kMany) cluster *= 2;
    return launch_compact_as<D, 128, 4, 3>(p, st, cluster);
}

cudaError_t launch_cache_compact(int d, const CompactParams& p, cudaStream_t st, int num_sms)
{
    return d == 64 ? launch_compact<64>(p, st, num_sms) : launch_compact<128>(p, st, num_sms);
}

cudaError_t launch_pages_update(PagesParams p, cudaStream_t st, int debug_flags)
{
    // the largest cluster that the device holds (0: not asked yet): 16 CTAs need as many SMs of one GPC, 8 are always there
    static int largest[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    int most = dev < 64 ? largest[dev] : 0;
    if (most == 0) {
        cudaError_t e = cudaFuncSetAttribute(fa_pages_update_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kPagesThreads);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, fa_pages_update_kernel, &cfg);
        if (e != cudaSuccess) cudaGetLastError();  // (as if there were none)
        most = e == cudaSuccess && n > 0 ? 16 : 8;
        if (dev < 64) largest[dev] = most;
    }
    if (debug_flags & kDebugPortableClusters) most = 8;
    // one CTA for every 8 K pages or 16 slots, up to the largest cluster (256 beams: 18.5 us in replays; with a CTA for
    // every 64 slots 22.6, for every 8 the same, but 64 slots 12.3 in place of 10.4.
    // 16 slots of a pool of 60 K pages: 10.4 us, a CTA for every 2 K or 32 K pages 12.4)
    p.cluster = 1;
    while (p.cluster < most && (p.num_pages > p.cluster * 8192 || p.slots > p.cluster * 16)) p.cluster *= 2;
    return launch_cluster(fa_pages_update_kernel, p.cluster, dim3(p.cluster), dim3(kPagesThreads), 0, st, p);
}

}  // namespace fa
