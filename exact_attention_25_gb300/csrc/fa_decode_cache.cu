// Split-KV decode over the paged e4m3 cache: O = softmax(scale Q K^T [+ causal mask]) V for a
// few bf16 queries per sequence, K and V being the cache's codes times their rows' powers of
// two.  Nothing is rounded on the way in: the result is exact attention on the cached values up
// to fp32 accumulation and the f16 rounding of the softmax weights.
//
// What bounds it: the codes, read once (2 * Nk * Hkv * d bytes a sequence): 8 sequences of up to 32 K
// keys, 8 heads of 128: 62 us, 87 % of the copy rate; 64 of up to 4 K: 51 us, 78 %.  With 16 query rows a
// head at d = 128 (8 sequences of 16 K: 86 us, 46 %) a step's chain of products, exponentials and products,
// of which the registers hold only one at a time.  Calls of one or two blocks a CTA are a chain of
// latencies: one sequence of 4 K keys 10.6 us, of which lengths 0.9, page ids 1.1, copies and products 2-3,
// the warps' merge 1, the parts' stores 0.5, and the merge kernel about 3 (two round trips: what the parts are
// of, then the parts).
// At the copy rate an SM receives about 23 bytes a clock, so tcgen05 has no place here although a decode
// tile of bf16 keys uses it: the codes would have to become 16-bit operands in shared memory, and one
// write by the copy, a read and a double-width write by the conversion and a double-width read
// by the tensor core (6 bytes of shared-memory traffic a code, 140 a clock) exceed the 128 bytes
// a clock that shared memory moves; kind::f8f6f4 would want Q and the weights in 8 bits too.
// Here the codes are converted between shared memory and mma.sync fragments instead, in
// registers: 2 bytes of traffic a code, and 0.09 m16n8k16 a clock for 8 query rows, of 0.5.
//
// Layout of a CTA: warps 0-3 compute, warp 4 copies pages to a ring of 128-key blocks by TMA
// (swizzled rows, plus the rows' exponent bytes).  A group's query rows (row i * G + g: query
// i, head g of the G that share the K/V head) form tiles of 8 * NR rows; warp w works on tile
// w % row_tiles and on every (4 / row_tiles)-th 16-key step of a block, with its own online
// softmax; the warps' results merge through shared memory at the end of a unit.  The copies run
// ahead over unit boundaries.  Two CTAs an SM, each with an equal share of the whole batch's blocks
// (CacheDecodeParams), found from the lengths on the device: a fixed number of ranges a sequence left
// SMs idle on ragged batches (the first of the above at best 71 us), and finer ranges cost every CTA its
// chain of latencies again.
//
// Both products are computed transposed, with the keys (S^T = K Q^T) or the columns of V (O^T =
// V^T P^T) as the 16 rows of the m16n8k16 product and the query rows as its 8 columns: a decode
// step has G <= 8 query rows, which as the 16-row operand would leave half of every product
// empty, and twice the registers.
// Per 16-key step, thread (g = lane / 4, t = lane % 4):
//  - S^T: the contraction index is permuted so that a thread's four elements of k-step s are
//    d = 16 t + 4 s + {0..3} (of a 64-wide half), i.e. one word of a 16-byte chunk; product row m
//    holds key kperm(m), chosen so that the chunks that are read together lie in different banks.
//    The thread gets keys kperm(g), 8 + kperm(g) of query rows 2 t, 2 t + 1.
//  - the weights go to the B layout by two 8 x 8 transposes (movmatrix).
//  - O^T: product rows g and g + 8 of tile i are V's columns d = CW g + 2 i and CW g + 2 i + 1 (CW =
//    d / 8), so a thread reads whole chunks of its keys' rows and pairs two keys' bytes by a byte
//    permute.
// Number ranges: Q rows are scaled by a power of two to just below 2^15 for f16 (elements down
// to 2^-38 of the row's largest keep a value).  Two running maxima are kept.  m, of the
// logits x (base 2), frames the sum l.  M, of x + (V's exponent), frames the weights
// w = 2^(x + ev - M + 11) that multiply V's codes, so a V row of any size keeps its weight's
// 11 bits (rows of zeros, kept under scale 1 whatever the others' size, stay out of M: they would push the weights of
// small rows below f16's smallest step) and w <= 2^15 (maxima move when they are exceeded by more than 4, so most steps need no
// reduction over the keys' lanes, only a vote); f16's smallest step puts a floor of 2^-36 of the
// largest weight under what a single key can still add.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace fa {

namespace {

constexpr int kKB = kCacheBlock;  // keys of a block
constexpr int kComputeWarps = 4;
constexpr int kUnits = 8;         // units described ahead
constexpr int kMergeThreads = 128;
constexpr float kFrame = 11.0f;   // log2 of the largest weight right after a rescale
constexpr float kGrow = 4.0f;     // a maximum moves when it grows by more than this

template <int D>
struct CacheCfg {
    static constexpr int TILE = kKB * D;               // bytes of a block's K or V codes
    static constexpr int STAGE = 2 * TILE + 2 * kKB;   // codes, then exponent bytes
    static constexpr int STAGES = D == 128 ? 3 : 6;
    // codes need 1024-byte alignment: all tiles first, then the exponents of all stages
    static constexpr int EXP0 = STAGES * 2 * TILE;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int OLD = D + 4;                  // row stride of the merge buffer, floats
    static constexpr int XCH = 8 * (OLD + 3);          // floats one warp hands over for 8 rows
    static constexpr int SMEM = RING + 3 * XCH * 4 + 1024;
    static constexpr int THREADS = 32 * (kComputeWarps + 1);
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}

// n bytes (a multiple of 16), both addresses 16-byte aligned
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(n), "r"(smem_u32(bar))
        : "memory");
}

// c += a b: 16 x 16 (row) by 16 x 8 (column), f16 in, fp32 accumulation
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 0x80 in every byte that is an e4m3 NaN code (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Transpose of an 8 x 8 tile of 16-bit elements held as a product's A or C tile is.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// An exponent byte x as the float x - 127, or NaN for 255.
__device__ __forceinline__ float exp_byte_log2(uint32_t byte)
{
    return byte == 255 ? NAN : __uint_as_float(0x4B000000u | byte) - (8388608.0f + 127.0f);
}

// The key of a 16-key step's product row n (0..7; rows 8..15 are the same plus 8).
template <int D>
__device__ __forceinline__ int kperm(int n)
{
    return D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}

}  // namespace

// One unit's part of a share.
struct Unit {
    int b, hk, row0;       // sequence, key/value head, first query row
    int q0, nq, nk, nblk;  // the sequence: first token, tokens, keys in the table, blocks
    int shift;             // causal: token i sees the keys up to i + shift
    int in_seq;            // units of the sequence
    int jb, J;             // this share's blocks of the unit: [jb, jb + J)
    int flags;             // kFirst: the share's first unit
};
constexpr int kFirst = 1;

// What the merge needs of a unit that is cut, as CacheDecodeParams::cuts holds it: first token, first query
// row, key/value head, and in one word the query rows (at most 64), whether the first part is its share's
// second, and the parts (at most 4096).  No rows: the share's end cuts no unit that begins in it.
__device__ __forceinline__ int4 pack_cut(const Unit& u, int rows, int lead, int parts)
{
    return make_int4(u.q0, u.row0, u.hk, rows | lead << 7 | parts << 8);
}

// Sizes of sequence b: units (row sets times heads) of nblk blocks each.
__device__ __forceinline__ void sequence_work(const CacheDecodeParams& p, int b, Unit& u)
{
    u.b = b;
    u.nq = packed_rows(p.cu_q, b, p.total_q, p.max_q, u.q0);
    const int len = min(max(p.seqlens[b], 0), p.max_k);
    u.nk = min(len, p.table_k);
    u.shift = len - u.nq;
    u.nblk = max(1, (u.nk + kKB - 1) / kKB);
    u.in_seq = ((u.nq * p.G.d + p.rows_cta - 1) >> p.rows_shift) * p.Hkv;
}

// All lanes of a warp: the line's shares and, for the first place of share c, its sequence (u) and
// its distance from that sequence's first place.
__device__ __forceinline__ Shares find_share(const CacheDecodeParams& p, int c, Unit& u, int& at)
{
    int b = 0;
    const Shares sh = find_share(
        p.B, p.ctas, c,
        [&](int x) {
            if (x >= p.B) return 0;
            Unit v;
            sequence_work(p, x, v);
            return v.in_seq * (v.nblk + kUnitCost);
        },
        b, at);
    if (sh.start(c) < sh.total) sequence_work(p, b, u);
    return sh;
}

// Row set and head of the sequence's unit i.
__device__ __forceinline__ void unit_at(const CacheDecodeParams& p, int i, Unit& u)
{
    const int set = p.heads(i);
    u.row0 = set << p.rows_shift;
    u.hk = i - set * p.Hkv;
}

// NR: 8-row query tiles of a warp.
template <int D, int NR>
__global__ void __launch_bounds__(CacheCfg<D>::THREADS, 2)
    fa_decode_cache_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const CacheDecodeParams p)
{
    using C = CacheCfg<D>;
    constexpr int KS = D / 16;              // k-steps of S
    constexpr int MT = D / 16;              // 16-column tiles of O
    constexpr int CH = D / 64;              // 16-byte chunks of a K row a thread reads
    constexpr int VW = D / 32;              // words of a V row a thread reads
    constexpr int TR = 8 * NR;              // query rows of a warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar_full[C::STAGES];
    __shared__ __align__(8) uint64_t bar_empty[C::STAGES];
    __shared__ __align__(8) uint64_t bar_unit[kUnits];
    __shared__ __align__(8) uint64_t bar_given[3];  // a warp's partial sums lie in xch[i] ...
    __shared__ __align__(8) uint64_t bar_taken[3];  // ... and have been added to another's
    __shared__ int s_valid[C::STAGES];  // bit i: keys [16 i, 16 i + 16) of the block were copied
    __shared__ Unit s_unit[kUnits];     // the copies' units, in order
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], kComputeWarps);
        }
        for (int k = 0; k < kUnits; ++k) mbar_init(&bar_unit[k], 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar_given[i], 1);
            mbar_init(&bar_taken[i], 1);
        }
        abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == kComputeWarps && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncthreads();
    dependent_begin();
    const int cta = static_cast<int>(blockIdx.x);
    const Watchdog wd{&abort_flag, p.status, p.wait_limit_ns};

    if (warp == kComputeWarps) {
        // ------------------------------------------------------------- copies
        // The share's units one after another; a unit's description goes to s_unit while its first page
        // ids are on their way, so the compute warps fetch its queries meanwhile.  (kUnits > STAGES + 1:
        // when a slot is written again, every warp has released a block of a later unit than the
        // one that it held.)
        Unit un;
        int at = 0;
        const Shares sh = find_share(p, cta, un, at);
        int left = sh.start(cta + 1) - sh.start(cta);
        const int ps = 1 << p.page_shift;
        const int np = ps >= kKB ? 1 : kKB / ps;              // pages of a block
        const int rows_pp = ps >= kKB ? kKB : ps;             // rows of a copy
        const int groups_pp = rows_pp / 16;
        int ui = 0, place = 0;                                // unit of the sequence, place in it
        if (left > 0) {
            ui = static_cast<unsigned>(at) / static_cast<unsigned>(un.nblk + kUnitCost);
            place = at - ui * (un.nblk + kUnitCost);
        }
        bool ok = true;
        int it = 0, k = 0;                                    // blocks through the ring, units so far
        bool cut = false;                                     // the share's end cuts a unit that begins here
        while (ok && left > 0) {
            unit_at(p, ui, un);
            const int end = min(un.nblk + kUnitCost, place + left);
            left -= end - place;
            un.jb = max(0, place - kUnitCost);
            un.J = max(0, end - kUnitCost) - un.jb;
            un.flags = k == 0 ? kFirst : 0;
            if (left == 0 && un.jb == 0 && un.J > 0 && un.J < un.nblk) {
                const int last = sh.share_of(sh.start(cta + 1) - un.J + un.nblk - 1);
                if (lane == 0)
                    p.cuts[cta] = pack_cut(un, min(un.nq * p.G.d - un.row0, p.rows_cta), k == 0 ? 0 : 1, last - cta + 1);
                cut = true;
            }
            // page ids base + lane; the first ones are on their way before anything else is done
            int base = (un.jb * kKB) >> p.page_shift, ids = -1;
            auto load_ids = [&]() {
                const int idx = base + lane;
                ids = -1;
                if (idx < p.max_pages && (static_cast<long long>(idx) << p.page_shift) < un.nk)
                    ids = p.table[static_cast<long long>(un.b) * p.max_pages + idx];
            };
            if (un.J > 0) {
                load_ids();
                if (lane == 0) {
                    s_unit[k % kUnits] = un;
                    mbar_arrive(&bar_unit[k % kUnits]);
                }
                // the unit's queries, ahead of the compute warps
                const int rows = min(un.nq * p.G.d - un.row0, p.rows_cta);
#pragma unroll 1
                for (int r = lane; r < rows; r += 32) {
                    const int i = p.G(un.row0 + r), h = (un.row0 + r) - i * p.G.d;
                    const __nv_bfloat16* q =
                        p.q + (static_cast<long long>(un.q0 + i) * p.H + un.hk * p.G.d + h) * D;
                    for (int c = 0; c < D; c += 64)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(q + c));
                }
                ++k;
            }
#pragma unroll 1
            for (int jj = 0; jj < un.J; ++jj, ++it) {
                const int s = it % C::STAGES;
                const int pos = (un.jb + jj) * kKB;
                const int first = pos >> p.page_shift;
                if (first + np > base + 32) {
                    base = first;
                    load_ids();
                }
                const int id = __shfl_sync(0xffffffffu, ids, (first - base + lane) & 31);
                const bool mine = lane < np && id >= 0 && id < p.num_pages;
                const uint32_t got = __ballot_sync(0xffffffffu, mine);
                ok = warp_wait_all(&bar_empty[s], ((it / C::STAGES) & 1) ^ 1, wd, kSiteCacheEmpty);
                if (!ok) break;
                if (lane == 0) {
                    int bits = 0;
#pragma unroll 1
                    for (int i = 0; i < np; ++i)
                        if (got >> i & 1) bits |= ((1 << groups_pp) - 1) << (i * groups_pp);
                    s_valid[s] = bits;
                    mbar_arrive_expect_tx(&bar_full[s],
                                          static_cast<uint32_t>(__popc(got) * rows_pp * 2 * (D + 1)));
                }
                __syncwarp();
                if (mine && !(it == 0 && (p.debug_flags & kDebugDropFirstLoad))) {
                    const int row_in = lane * rows_pp;        // first key of the copy in the block
                    const long long row = ((static_cast<long long>(id) * p.Hkv + un.hk) << p.page_shift) +
                                          (pos & (ps - 1));
                    uint8_t* kt = smem + s * 2 * C::TILE + row_in * D;
                    uint8_t* ex = smem + C::EXP0 + s * 2 * kKB + row_in;
                    tma_load_2d(kt, &tm_k, &bar_full[s], 0, static_cast<int>(row));
                    bulk_load(ex, p.ke + row, rows_pp, &bar_full[s]);
                    tma_load_2d(kt + C::TILE, &tm_v, &bar_full[s], 0, static_cast<int>(row));
                    bulk_load(ex + kKB, p.ve + row, rows_pp, &bar_full[s]);
                }
            }
            place = 0;
            if (left > 0) {
                if (++ui == un.in_seq) {
                    ui = 0;
                    do sequence_work(p, un.b + 1, un);
                    while (un.in_seq == 0 && un.b + 1 < p.B);
                }
            }
        }
        if (!cut && lane == 0 && p.cuts != nullptr) p.cuts[cta] = make_int4(0, 0, 0, 0);
        // the end of the units
        if (ok && lane == 0) {
            s_unit[k % kUnits].J = 0;
            mbar_arrive(&bar_unit[k % kUnits]);
        }
        // no copy may land after the CTA exits (bounded waits that ignore the abort flag)
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        for (int i = max(0, it - C::STAGES); i < it; ++i)
            mbar_wait(&bar_full[i % C::STAGES], (i / C::STAGES) & 1, wd_drain, kSiteCacheDrain);
        return;
    }

    // ----------------------------------------------------------------- attention
    const int g = lane >> 2, t = lane & 3;
    const int tile = warp % p.row_tiles;
    const int slots = kComputeWarps / p.row_tiles, slot = warp / p.row_tiles;
    float* xch = reinterpret_cast<float*>(smem + C::RING);  // [3][XCH]
    const int kp = kperm<D>(g);
    const int kc0 = kperm<D>(2 * t), kc1 = kperm<D>(2 * t + 1);
    // which of the two keys is read first, so that a phase's rows lie in different banks
    const int swap = D == 128 ? (g & 1) : ((g >> 1) & 1);
    const int vr0 = swap ? kc1 : kc0, vr1 = swap ? kc0 : kc1;
    const uint32_t sel_lo = swap ? 0x1504u : 0x5140u, sel_hi = swap ? 0x3726u : 0x7362u;
    int it = 0;       // blocks through the ring so far
    int rounds = 0;   // merges so far
#pragma unroll 1
    for (int k = 0;; ++k) {
        if (!warp_wait_all(&bar_unit[k % kUnits], (k / kUnits) & 1, wd, kSiteCacheFull)) return;
        const Unit& un = s_unit[k % kUnits];
        if (un.J == 0) return;
        const int rows = min(un.nq * p.G.d - un.row0, p.rows_cta);
        // element offset of query row r's o row, and its lse
        auto out_off = [&](int r) {
            const int i = p.G(un.row0 + r), h = (un.row0 + r) - i * p.G.d;
            return (static_cast<long long>(un.q0 + i) * p.H + un.hk * p.G.d + h) * D;
        };
        auto stat_off = [&](int r) {
            const int i = p.G(un.row0 + r), h = (un.row0 + r) - i * p.G.d;
            return static_cast<long long>(un.hk * p.G.d + h) * p.total_q + un.q0 + i;
        };
        // last key that query row r of the tile sees (-1: none, or no such row)
        auto limit = [&](int r) {
            r += tile * TR;
            if (r >= rows) return -1;
            return p.causal ? min(un.nk - 1, p.G(un.row0 + r) + un.shift) : un.nk - 1;
        };
        uint32_t qb[NR][KS][2];    // query row 8 n + g, the thread's elements
        float cx[NR][2];           // rows 8 n + 2 t + e: logit (base 2) per unit of the product
        int lim[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int r = tile * TR + 8 * n + g;
            uint32_t u[CH][8], amax = 0;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
                if (r < rows) {
                    const long long off = out_off(r) + 64 * c + 16 * t;
                    if (in_extent(off, 16, p.q_ext, p.status)) {
                        w[0] = reinterpret_cast<const uint4*>(p.q + off)[0];
                        w[1] = reinterpret_cast<const uint4*>(p.q + off)[1];
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    u[c][4 * i] = w[i].x; u[c][4 * i + 1] = w[i].y;
                    u[c][4 * i + 2] = w[i].z; u[c][4 * i + 3] = w[i].w;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = __vmaxu2(amax, u[c][i] & 0x7fff7fffu);
            }
            amax = max(amax & 0xffffu, amax >> 16);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^a brings the row's largest magnitude to [2^14, 2^15).  (In a row with an infinity or
            // a NaN the rest vanishes beside it, as it does in its logits.)
            const int a = min(14 + 127 - static_cast<int>(amax >> 7), 126);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + a) << 23);
            const float down = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    qb[n][4 * c + i / 2][i & 1] = pack_f16x2(__uint_as_float(u[c][i] << 16) * up,
                                                             __uint_as_float(u[c][i] & 0xFFFF0000u) * up);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                cx[n][e] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + e));
                lim[n][e] = limit(8 * n + 2 * t + e);
            }
        }
        // keys past `most` are seen by no row of the tile; up to `least` by every row of it
        int most = -1, least = un.nk - 1;
        if (tile * TR < rows) {
            most = limit(min(TR, rows - tile * TR) - 1);
            least = limit(0);
        }
        float o[NR][MT][4];
        float M[NR][2], m[NR][2], l[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
            M[n][0] = M[n][1] = m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }

        // U 16-key steps of block `block` at once, gi and gi + gap.  MASKED: the step's keys may lie past
        // the end or be hidden from some rows.
        auto step = [&](auto masked_c, auto u_c, const uint8_t* kt, const uint8_t* ex, int block, int gi,
                        int gap) {
            constexpr bool MASKED = decltype(masked_c)::value;
            constexpr int U = decltype(u_c)::value;
            const uint8_t* vt = kt + C::TILE;
            // ---- S^T
            float sc[U][NR][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float part[CH][NR][4];
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int row = (gi + u * gap) * 16 + hf * 8 + kp;
                        const int phys = D == 128 ? ((t + 4 * c) ^ (row & 7)) : (t ^ ((row >> 1) & 3));
                        const uint4 x = *reinterpret_cast<const uint4*>(kt + row * D + 16 * phys);
                        w[hf][0] = x.x; w[hf][1] = x.y; w[hf][2] = x.z; w[hf][3] = x.w;
                    }
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        part[c][n][0] = part[c][n][1] = part[c][n][2] = part[c][n][3] = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t a[4] = {e4m3x2_to_f16x2(w[0][k]), e4m3x2_to_f16x2(w[1][k]),
                                               e4m3x2_to_f16x2(w[0][k] >> 16), e4m3x2_to_f16x2(w[1][k] >> 16)};
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            mma16816(part[c][n], a, qb[n][4 * c + k][0], qb[n][4 * c + k][1]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[u][n][i] = CH == 2 ? part[0][n][i] + part[CH - 1][n][i] : part[0][n][i];
            }
            // ---- logits x, and x plus V's exponent
            float x[U][NR][4], tv[U][NR][4];
            float ev[U][2];
            bool unit = false;  // a row under scale 1: perhaps a row of zeros
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    ev[u][hf] = exp_byte_log2(ex[kKB + (gi + u * gap) * 16 + hf * 8 + kp]);
                    unit = unit || ev[u][hf] == 0.0f;
                }
            if (__any_sync(0xffffffffu, unit)) {
                // of a key's row each of the thread's three neighbours reads a quarter too (-0 is zero as well)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int row = (gi + u * gap) * 16 + hf * 8 + kp;
                        const uint4* w = reinterpret_cast<const uint4*>(vt + row * D + D / 4 * t);
                        uint32_t some = 0;
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) some |= w[i].x | w[i].y | w[i].z | w[i].w;
                        some &= 0x7f7f7f7fu;
                        some |= __shfl_xor_sync(0xffffffffu, some, 1);
                        some |= __shfl_xor_sync(0xffffffffu, some, 2);
                        if (some == 0 && ev[u][hf] == 0.0f) ev[u][hf] = -INFINITY;
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int key = (gi + u * gap) * 16 + hf * 8 + kp;
                    const float ks = exp_byte_scale(ex[key]);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = sc[u][n][2 * hf + e] * (cx[n][e] * ks);
                            float w = v + ev[u][hf];
                            if (MASKED && block * kKB + key > lim[n][e]) v = w = -INFINITY;
                            x[u][n][2 * hf + e] = v;
                            tv[u][n][2 * hf + e] = w;
                        }
                }
            bool need = false;
            float xm[NR][2], tm[NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    xm[n][e] = fmaxf(x[0][n][e], x[0][n][2 + e]);
                    tm[n][e] = fmaxf(tv[0][n][e], tv[0][n][2 + e]);
                    if constexpr (U == 2) {
                        xm[n][e] = fmax3(xm[n][e], x[U - 1][n][e], x[U - 1][n][2 + e]);
                        tm[n][e] = fmax3(tm[n][e], tv[U - 1][n][e], tv[U - 1][n][2 + e]);
                    }
                    need = need || xm[n][e] > m[n][e] + kGrow || tm[n][e] > M[n][e] + kGrow;
                }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // m frames this thread's own sum; M is the row's, shared by its lanes
                        if (xm[n][e] > m[n][e] + kGrow) {
                            l[n][e] *= ex2(m[n][e] - xm[n][e]);
                            m[n][e] = xm[n][e];
                        }
                        float r = tm[n][e];
                        r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 4));
                        r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 8));
                        r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 16));
                        if (r > M[n][e] + kGrow) {
                            const float alpha = ex2(M[n][e] - r);
                            M[n][e] = r;
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                o[n][i][e] *= alpha;
                                o[n][i][2 + e] *= alpha;
                            }
                        }
                    }
            }
            uint32_t pb[U][NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                float nm[2], nM[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    nm[e] = m[n][e] == -INFINITY ? 0.0f : m[n][e];
                    nM[e] = (M[n][e] == -INFINITY ? 0.0f : M[n][e]) - kFrame;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) l[n][e] += ex2(x[u][n][2 * hf + e] - nm[e]);
                        pb[u][n][hf] = transpose8x8(pack_f16x2(ex2(tv[u][n][2 * hf] - nM[0]),
                                                               ex2(tv[u][n][2 * hf + 1] - nM[1])));
                    }
            }
            // ---- V's words
            uint32_t va[U][2][2][VW];  // [step][key half][first, second row][word]
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int row = (gi + u * gap) * 16 + hf * 8 + (f ? vr1 : vr0);
                        if constexpr (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(vt + row * D + 16 * (g ^ (row & 7)));
                            va[u][hf][f][0] = x.x; va[u][hf][f][1] = x.y;
                            va[u][hf][f][2] = x.z; va[u][hf][f][3] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(
                                vt + row * D + 16 * ((g >> 1) ^ ((row >> 1) & 3)) + 8 * (g & 1));
                            va[u][hf][f][0] = x.x; va[u][hf][f][1] = x.y;
                        }
                    }
            if constexpr (MASKED) {
                // Rows past the sequence's end hold whatever the page held: zero them.  NaN codes
                // of rows that only some queries see must not reach the others (0 * NaN): they are
                // taken out of the product, and the rows that do see them get NaN by a product of
                // indicators.
                const int kbase = block * kKB + gi * 16;
                bool bad = false;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int key = kbase + hf * 8 + (f ? vr1 : vr0);
#pragma unroll
                        for (int i = 0; i < VW; ++i) {
                            if (key >= un.nk) va[0][hf][f][i] = 0u;
                            bad = bad || nan_bytes(va[0][hf][f][i]);
                        }
                    }
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        uint32_t z[2][2];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const uint32_t nb = nan_bytes(va[0][hf][f][i]) >> 7;
                                z[hf][f] = nb * 0x38u;  // the code of 1.0 where NaN
                                va[0][hf][f][i] &= ~(nb * 0xffu);
                            }
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t lo = __byte_perm(z[0][0], z[0][1], c ? sel_hi : sel_lo);
                            const uint32_t hi = __byte_perm(z[1][0], z[1][1], c ? sel_hi : sel_lo);
                            const uint32_t a[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16),
                                                   e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                const int rl = limit(8 * n + g) - kbase;  // B's column is row 8 n + g
                                float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma16816(cnt, a,
                                         pack_f16x2(kc0 <= rl ? 1.0f : 0.0f, kc1 <= rl ? 1.0f : 0.0f),
                                         pack_f16x2(8 + kc0 <= rl ? 1.0f : 0.0f, 8 + kc1 <= rl ? 1.0f : 0.0f));
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (cnt[e] > 0.0f) o[n][2 * i + c][e] = NAN;
                            }
                        }
                    }
                }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < VW; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t lo = __byte_perm(va[u][0][0][i], va[u][0][1][i], c ? sel_hi : sel_lo);
                        const uint32_t hi = __byte_perm(va[u][1][0][i], va[u][1][1][i], c ? sel_hi : sel_lo);
                        const uint32_t a[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16),
                                               e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma16816(o[n][2 * i + c], a, pb[u][n][0], pb[u][n][1]);
                    }
        };

        const int j1 = un.jb + un.J;
#pragma unroll 1
        for (int j = un.jb; j < j1; ++j, ++it) {
            const int s = it % C::STAGES;
            if (!warp_wait_all(&bar_full[s], (it / C::STAGES) & 1, wd, kSiteCacheFull)) return;
            const int valid = s_valid[s];
            const uint8_t* kt = smem + s * 2 * C::TILE;
            const uint8_t* ex = smem + C::EXP0 + s * 2 * kKB;
            // Steps in the clear go U at a time, so that one's products hide the other's latencies.  (16
            // rows at d = 64: 16 sequences of up to 5000 keys, 32 rows: 18.0 us, one at a time 19.5.  At
            // d = 128 their registers do not hold two: 8 sequences of 16 K keys, 16 rows: 95 us, one at a
            // time 86.)
            constexpr int U = NR == 1 || D == 64 ? 2 : 1;
            if (most >= 0)  // (else there is no query row in this warp's tile)
#pragma unroll 1
                for (int gi = slot; gi < kKB / 16; gi += U * slots) {
                    const int last = gi + (U - 1) * slots;
                    if ((valid >> gi & 1) && (valid >> last & 1) && j * kKB + last * 16 + 15 <= least) {
                        step(std::false_type{}, std::integral_constant<int, U>{}, kt, ex, j, gi, slots);
                    } else {
#pragma unroll 1
                        for (int i = gi; i <= last; i += slots)
                            if ((valid >> i & 1) && j * kKB + i * 16 <= most)
                                step(std::true_type{}, std::integral_constant<int, 1>{}, kt, ex, j, i, slots);
                    }
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_empty[s]);
        }
        // ---- merge of the warps of a tile into its slot 0: slots 2, 3 into 0, 1, then 1 into 0
        // (two slots: one round; a chain of three hand-overs to slot 0 took 700 clocks longer).
        // Threads of the same lane hold the same elements.
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // the row's sums of its eight lanes in one frame
                float mm = m[n][e];
#pragma unroll
                for (int d = 4; d < 32; d *= 2) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
                float ll = l[n][e] * (m[n][e] == -INFINITY ? 1.0f : ex2(m[n][e] - mm));
#pragma unroll
                for (int d = 4; d < 32; d *= 2) ll += __shfl_xor_sync(0xffffffffu, ll, d);
                m[n][e] = mm;
                l[n][e] = ll;
            }
            auto give = [&](int i) {
                if (!warp_wait_all(&bar_taken[i], (rounds & 1) ^ 1, wd, kSiteCacheMerge)) return false;
                float* x = xch + i * C::XCH;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float* row = x + (2 * t + e) * C::OLD;
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<float4*>(row + 2 * MT * g + 2 * i) =
                            make_float4(o[n][i][e], o[n][i][2 + e], o[n][i + 1][e], o[n][i + 1][2 + e]);
                    if (g == 0) {
                        float* st = x + 8 * C::OLD + 3 * (2 * t + e);
                        st[0] = M[n][e];
                        st[1] = m[n][e];
                        st[2] = l[n][e];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_given[i]);
                return true;
            };
            auto take = [&](int i) {
                if (!warp_wait_all(&bar_given[i], rounds & 1, wd, kSiteCacheMerge)) return false;
                const float* x = xch + i * C::XCH;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float* st = x + 8 * C::OLD + 3 * (2 * t + e);
                    const float M2 = fmaxf(M[n][e], st[0]), m2 = fmaxf(m[n][e], st[1]);
                    const float fa = M[n][e] == -INFINITY ? 1.0f : ex2(M[n][e] - M2);
                    const float fb = st[0] == -INFINITY ? 1.0f : ex2(st[0] - M2);
                    l[n][e] = l[n][e] * (m[n][e] == -INFINITY ? 1.0f : ex2(m[n][e] - m2)) +
                              st[2] * (st[1] == -INFINITY ? 1.0f : ex2(st[1] - m2));
                    M[n][e] = M2;
                    m[n][e] = m2;
                    const float* row = x + (2 * t + e) * C::OLD;
#pragma unroll
                    for (int i = 0; i < MT; i += 2) {
                        const float4 v = *reinterpret_cast<const float4*>(row + 2 * MT * g + 2 * i);
                        o[n][i][e] = o[n][i][e] * fa + v.x * fb;
                        o[n][i][2 + e] = o[n][i][2 + e] * fa + v.y * fb;
                        o[n][i + 1][e] = o[n][i + 1][e] * fa + v.z * fb;
                        o[n][i + 1][2 + e] = o[n][i + 1][2 + e] * fa + v.w * fb;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_taken[i]);
                return true;
            };
#pragma unroll 1
            for (int half = slots / 2; half > 0; half /= 2) {
                // slots half .. 2 half - 1 give to those below; buffers 0, 1 in the first round, 2
                // in the second of four slots
                const int x = half == 1 && slots == 4 ? 2 : warp & 1;
                if (slot >= 2 * half) continue;
                if (slot >= half ? !give(x) : !take(x)) return;
            }
            ++rounds;
            if (slot != 0) continue;
            // ---- O = o 2^(M - frame) / (l 2^m); a row that saw no key has l = 0.  The power is
            // applied in halves: each is representable where the whole may not be.
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = tile * TR + 8 * n + 2 * t + e;
                if (r >= rows) continue;
                const float inv = l[n][e] == 0.0f ? 0.0f : 1.0f / l[n][e];
                const float half = (M[n][e] == -INFINITY || m[n][e] == -INFINITY)
                                       ? 1.0f : ex2(0.5f * (M[n][e] - kFrame - m[n][e]));
                const float lse = l[n][e] == 0.0f ? -INFINITY : (m[n][e] + log2f(l[n][e])) * kLn2;
                const float f0 = inv * half;
                float v[2 * MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    v[2 * i] = o[n][i][e] * f0 * half;
                    v[2 * i + 1] = o[n][i][2 + e] * f0 * half;
                }
                if (un.J == un.nblk) {
                    const long long off = out_off(r) + 2 * MT * g, so = stat_off(r);
                    if (in_extent(off, 2 * MT, p.q_ext, p.status)) {
#pragma unroll
                        for (int i = 0; i < 2 * MT; i += 8)
                            *reinterpret_cast<uint4*>(p.o + off + i) =
                                make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                                           pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
                    }
                    if (g == 0 && p.lse != nullptr && in_extent(so, 1, p.stat_ext, p.status)) p.lse[so] = lse;
                } else {
                    const long long pr = static_cast<long long>(2 * cta + (un.flags & kFirst ? 0 : 1)) * p.rows_cta + r;
                    const long long off = pr * D + 2 * MT * g;
                    if (in_extent(off, 2 * MT, p.part_ext, p.status)) {
#pragma unroll
                        for (int i = 0; i < 2 * MT; i += 4)
                            *reinterpret_cast<float4*>(p.o_part + off + i) =
                                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                    if (g == 0 && in_extent(pr, 1, p.part_ext / D, p.status)) p.lse_part[pr] = lse;
                }
            }
        }
    }
}

// Merge of the parts of every unit that several shares cut: CTA c takes the unit that begins in share c and
// goes on in the next, if there is one; a warp takes a query row.  A row that saw no key in any part gets
// O = 0, lse = -inf.  The attention CTAs leave the units' descriptions beside the parts: worked out here again,
// from the lengths, they would cost every CTA a scan behind its wait (ahead of it nothing may be read).
template <int D>
__global__ void __launch_bounds__(kMergeThreads) fa_decode_cache_merge_kernel(const CacheDecodeParams p)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const int c0 = static_cast<int>(blockIdx.x);
    dependent_begin();
    const int4 cut = p.cuts[c0];
    const int q0 = cut.x, row0 = cut.y, hk = cut.z;
    const int rows = cut.w & 127, lead = cut.w >> 7 & 1, parts = cut.w >> 8;
    const int r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);
    if (r < rows) {
        float mx, sum, acc[EPL];
        merge_parts<D, 16>(
            parts, [&](int k) { return (2 * (c0 + k) + (k == 0 ? lead : 0)) * p.rows_cta + r; },
            p.o_part, p.lse_part, p.part_ext / D, p.status, mx, sum, acc);
        const int i = p.G(row0 + r), h = hk * p.G.d + (row0 + r) - i * p.G.d;
        const long long row = (static_cast<long long>(q0 + i) * p.H + h) * D + EPL * lane;
        const long long stat = static_cast<long long>(h) * p.total_q + q0 + i;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (in_extent(row, EPL, p.q_ext, p.status)) {
            if constexpr (EPL == 4)
                *reinterpret_cast<uint2*>(p.o + row) = make_uint2(
                    pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
            else
                *reinterpret_cast<uint32_t*>(p.o + row) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        }
        if (lane == 0 && p.lse != nullptr && in_extent(stat, 1, p.stat_ext, p.status))
            p.lse[stat] = sum == 0.0f ? -INFINITY : mx + logf(sum);
    }
}

template <int D, int NR>
static cudaError_t launch_decode_cache_impl(const CUtensorMap& tk, const CUtensorMap& tv,
                                            const CacheDecodeParams& p, cudaStream_t st)
{
    using C = CacheCfg<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(fa_decode_cache_kernel<D, NR>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    cudaError_t e = launch_dependent(fa_decode_cache_kernel<D, NR>, dim3(p.ctas), dim3(C::THREADS),
                                     C::SMEM, st, tk, tv, p);
    if (e != cudaSuccess || p.ctas == 1) return e;
    return launch_dependent(fa_decode_cache_merge_kernel<D>, dim3(p.ctas - 1, p.rows_cta / (kMergeThreads / 32)), dim3(kMergeThreads), 0,
                            st, p);
}

cudaError_t launch_decode_cache(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheDecodeParams& p, cudaStream_t st)
{
    const bool small = p.rows_cta == 8;
    if (d == 64)
        return small ? launch_decode_cache_impl<64, 1>(tk, tv, p, st)
                     : launch_decode_cache_impl<64, 2>(tk, tv, p, st);
    return small ? launch_decode_cache_impl<128, 1>(tk, tv, p, st)
                 : launch_decode_cache_impl<128, 2>(tk, tv, p, st);
}

}  // namespace fa
