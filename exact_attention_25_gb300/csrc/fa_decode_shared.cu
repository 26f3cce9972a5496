// Decoding for batches whose sequences share long prefixes, on sm_103a tensor cores: the queries of
// a group of sequences attend to the group's prefix, all as one tile of rows, and each sequence's
// queries to its own keys (bottom-right causal mask), under one softmax:
//     O = softmax([q K_p^T, q K_s^T] scale) [V_p; V_s].
// The two ranges of keys are computed apart, each with its own online softmax, and merged by the
// rescaling rule O = sum_s e^{lse_s} O_s / sum_s e^{lse_s}; so a prefix is read once for its group
// and not once for each sequence, and its products have the rows of the whole group.
//
// What bounds it: reading prefix and own keys once (HBM), and for large groups the exponentials of
// tokens x heads x prefix scores.  64 sequences with up to 1024 keys of their own over 32000 tokens, 32
// heads over 8 of 128: 64 us, 253 MB from HBM (4.0 TB/s) and 421 MB from L2 (the prefix is copied for each of
// its two tiles); 9 us less without the softmax, 5 less without its products.  8 sequences over 4 K tokens: 13.4 us,
// a chain of latencies.
//
// Both kinds of work are units of one line (units, below) shared out evenly over the SMs, so memory-bound
// and arithmetic-bound units run side by side.  Every key/value head has a line of its own, the same for
// all, and CTA c works on head c mod Hkv: so the CTAs of the heads read the same tokens at the same time.
// (In one line over all heads each read its 256-byte pieces of the token rows at a time of its own: 70 us.)
//
// A unit is a tile of up to 128 query rows (row r = i * G + g: token i of the tile, head g of the G
// that share the K/V head) against the keys of one prefix or sequence.  Roles (6 warps): warps 0-3
// softmax (thread = tile row = TMEM lane), warp 4 TMA producer, warp 5 TMEM allocator and MMA
// issuer.  All of them run over the CTA's whole share without a barrier between units: Q is free after
// a unit's last scores, so the next unit's first scores are computed while the softmax warps still
// write out the one before.  The rings take the rest of shared memory: copies have a latency of some
// 3000 clocks under load and a block of 64 KB goes every 2000, so about 100 KB have to be in flight beside
// the tiles in use.  TMEM: two S buffers [0, 128), [128, 256) (P of a block, bf16 pairs, overwrites the lower
// half of its S buffer), O from 256 on.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

#include <type_traits>

namespace fa {

namespace {

constexpr int kSB = 128;           // keys of a block
constexpr int kSharedUnits = 8;    // units described ahead

template <int D>
struct SharedCfg {
    static constexpr int PANELS = D / 64;          // 128-byte swizzle panels per row
    static constexpr int PANEL_BYTES = 128 * 128;  // 128 rows x 128 bytes
    static constexpr int TILE_BYTES = PANELS * PANEL_BYTES;
    static constexpr int KST = D == 128 ? 3 : 6;   // stages of the K and V rings
    static constexpr int VST = KST;
    static constexpr int SMEM_BYTES = (1 + KST + VST) * TILE_BYTES + 1024;
    static constexpr int THREADS = 192;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units, as in the forward kernel
};

// One unit's part of a share.
struct SharedUnit {
    int item;              // prefix of group `item`, or the keys of sequence item - groups
    int hk, tile;          // key/value head, tile of tokens
    int tok0, ntok;        // the item's tokens: first row, count
    int k0, nk, nblk;      // its keys
    int in_item;           // tiles of tokens of the item (units for each head)
    int jb, J;             // this share's blocks of the unit: [jb, jb + J)
    int first;             // the share's first unit
    int odd;               // V holds infinities or NaNs that only some of the tile's rows see
};

// Sizes of an item: for each head in_item units of nblk blocks (none without tokens or keys).
__device__ __forceinline__ void shared_item(const SharedDecodeParams& p, int x, SharedUnit& u)
{
    u.item = x;
    if (x < p.groups) {
        const int b0 = min(max(p.cu_g[x], 0), p.B);
        const int b1 = min(max(p.cu_g[x + 1], b0), p.B);
        u.tok0 = min(max(p.cu_q[b0], 0), p.total_q);
        u.ntok = min(min(max(p.cu_q[b1], u.tok0), p.total_q) - u.tok0, p.max_group_q);
        u.nk = packed_rows(p.cu_p, x, p.total_p, p.max_p, u.k0);
    } else {
        u.ntok = packed_rows(p.cu_q, x - p.groups, p.total_q, p.max_q, u.tok0);
        u.nk = packed_rows(p.cu_k, x - p.groups, p.total_k, p.max_k, u.k0);
    }
    u.nblk = (u.nk + kSB - 1) / kSB;
    u.in_item = u.nk > 0 ? p.tile_tokens(u.ntok + p.tile_tokens.d - 1) : 0;
}

__device__ __forceinline__ int shared_places(const SharedDecodeParams& p, int x)
{
    if (x >= p.groups + p.B) return 0;
    SharedUnit u;
    shared_item(p, x, u);
    return u.in_item * (u.nblk + kSharedUnitCost);
}

// What the merge has to know of tokens [t0, t1), by a warp: for its own keys (the first of two entries) and for
// its group's prefix, the places of the line before the item, the item's blocks (0: no keys) and the token's
// index in it (-1: in no sequence); and the line's length.
__device__ __noinline__ void place_tokens(const SharedDecodeParams& p, int t0, int t1)
{
    const int lane = threadIdx.x & 31, items = p.groups + p.B;
    for (int t = t0 + lane; t < t1; t += 32) {
        p.places[2ll * t] = make_int4(0, 0, -1, 0);
        p.places[2ll * t + 1] = make_int4(0, 0, 0, 0);
    }
    __syncwarp();
    int run = 0;
#pragma unroll 1
    for (int x0 = 0; x0 < items; x0 += 32) {
        SharedUnit u;
        int w = 0, a = 0, b = 0;
        u.tok0 = u.nblk = 0;
        if (x0 + lane < items) {
            shared_item(p, x0 + lane, u);
            w = u.in_item * (u.nblk + kSharedUnitCost);
            a = max(t0, u.tok0);
            b = min(t1, u.tok0 + u.ntok);
        }
        int sum = w;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += up;
        }
        uint32_t mine = __ballot_sync(0xffffffffu, a < b);  // items with some of the tokens
        while (mine) {
            const int src = __ffs(mine) - 1;
            mine &= mine - 1;
            const int before = run + __shfl_sync(0xffffffffu, sum - w, src), nblk = __shfl_sync(0xffffffffu, u.nblk, src);
            const int tok0 = __shfl_sync(0xffffffffu, u.tok0, src), end = __shfl_sync(0xffffffffu, b, src);
            for (int t = __shfl_sync(0xffffffffu, a, src) + lane; t < end; t += 32)
                p.places[2ll * t + (x0 + src < p.groups)] = make_int4(before, nblk, t - tok0, 0);
            __syncwarp();  // (starts that do not rise may give a token to several items: the last one has it)
        }
        run += __shfl_sync(0xffffffffu, sum, 31);
    }
    for (int t = t0 + lane; t < t1; t += 32) p.places[2ll * t].w = run;
}

// Two bf16 values, infinities and NaNs replaced by zero.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v)
{
    if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
    if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
    return v;
}

// V of keys that some row of a unit does not see must not reach it as 0 * inf or 0 * NaN.  Of rows
// [first, last) of a block's V tile (to the end of the 16-key step that the last key lies in), those
// from `end` on, past the unit's keys, are zeroed; of the others, which some queries see, what is not
// finite is taken out, and given back to those queries at the unit's end (add_odd_v).  Each softmax warp
// takes every fourth row.  Returns whether this lane took anything out.
template <int D>
__device__ __noinline__ bool clear_unseen_v(uint8_t* tile, int first, int end, int last)
{
    using C = SharedCfg<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int LB = D / 16;  // bytes of a row for each lane: 4 or 8
    const int at = lane * LB;
    uint8_t* base = tile + (at >> 7) * C::PANEL_BYTES + (at & 127);
    bool odd = false;
#pragma unroll 1
    for (int row = first + warp; row < last; row += 4) {
        uint32_t* w = reinterpret_cast<uint32_t*>(base + row * 128);
#pragma unroll
        for (int c = 0; c < LB / 4; ++c) {
            if (row >= end) {
                w[c] = 0u;
            } else if (finite_bf16x2(w[c]) != w[c]) {
                w[c] = finite_bf16x2(w[c]);
                odd = true;
            }
        }
    }
    fence_proxy_async_smem();
    return odd;
}

// Adds what is not finite in V rows [key0, key1) of a sequence to the row at dst.
template <int D>
__device__ __noinline__ void add_odd_v(const SharedDecodeParams& p, float* dst, const SharedUnit& un, int key0, int key1)
{
#pragma unroll 1
    for (int key = key0; key < key1; ++key) {
        const long long off = (static_cast<long long>(un.k0 + key) * p.Hkv + un.hk) * D;
        if (!in_extent(off, D, p.v_ext, p.status)) continue;
        for (int c = 0; c < D; ++c) {
            const float v = __bfloat162float(p.v[off + c]);
            if (!(fabsf(v) < INFINITY)) dst[c] += v;
        }
    }
}

// S = Q K^T over D/16 k-steps (both operands K-major in 128B-swizzled panels).
template <int D, int PANEL>
__device__ __forceinline__ void shared_issue_qk(uint32_t d_tmem, uint64_t qdesc, uint64_t kdesc, uint32_t idesc)
{
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = (ks / 4) * PANEL + (ks % 4) * 32;
        mma_ss_w(d_tmem, sdesc_adv(qdesc, off), sdesc_adv(kdesc, off), idesc, ks > 0 ? 1u : 0u);
    }
}

// O += P V: P (bf16 pairs) from TMEM, V (MN-major) from shared memory; k-steps of 16 keys.
__device__ __forceinline__ void shared_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t vdesc,
                                                uint32_t idesc, uint32_t acc_first, int steps)
{
    if (steps == 8) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            mma_ts_w(d_tmem, p_tmem + 8u * ks, sdesc_adv(vdesc, ks * 2048), idesc, ks > 0 ? 1u : acc_first);
    } else {
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks)
            mma_ts_w(d_tmem, p_tmem + 8u * ks, sdesc_adv(vdesc, ks * 2048), idesc, ks > 0 ? 1u : acc_first);
    }
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(SharedCfg<D>::THREADS, 1)
    fa_decode_shared_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_kp,
                            const __grid_constant__ CUtensorMap tm_vp,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const SharedDecodeParams p)
{
    using C = SharedCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sK = sQ + C::TILE_BYTES;
    uint8_t* sV = sK + C::KST * C::TILE_BYTES;

    __shared__ __align__(8) uint64_t bar_qfull, bar_qempty;
    __shared__ __align__(8) uint64_t bar_kfull[C::KST], bar_kempty[C::KST];
    __shared__ __align__(8) uint64_t bar_vfull[C::VST], bar_vempty[C::VST];
    __shared__ __align__(8) uint64_t bar_unit[kSharedUnits];
    __shared__ __align__(8) uint64_t bar_sfull[2];  // S of a block landed in buffer b
    __shared__ __align__(8) uint64_t bar_pfull;     // softmax wrote P (and rescaled O)
    __shared__ __align__(8) uint64_t bar_pv;        // the P V product of a block has run
    __shared__ __align__(8) uint64_t bar_drain;
    __shared__ SharedUnit s_unit[kSharedUnits];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&bar_qfull, 1);
        mbar_init(&bar_qempty, 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bar_sfull[i], 1);
        for (int s = 0; s < C::KST; ++s) {
            mbar_init(&bar_kfull[s], 1);
            mbar_init(&bar_kempty[s], 1);
        }
        for (int s = 0; s < C::VST; ++s) {
            mbar_init(&bar_vfull[s], 1);
            mbar_init(&bar_vempty[s], 1);
        }
        for (int k = 0; k < kSharedUnits; ++k) mbar_init(&bar_unit[k], 1);
        mbar_init(&bar_pfull, 4);  // one elected arrive per softmax warp
        mbar_init(&bar_pv, 1);
        mbar_init(&bar_drain, 1);
        abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 5) {
        tmem_alloc(&tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 4 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_kp);
        tma_prefetch_desc(&tm_vp);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_slot;
    const Watchdog wd{&abort_flag, p.status, p.wait_limit_ns};
    dependent_begin();
    const int cta = static_cast<int>(blockIdx.x);
    // the items' places, by all warps, in the V ring (free until the first copy)
    int* s_places = reinterpret_cast<int*>(sV);
    const int items = p.groups + p.B;
#pragma unroll 1
    for (int x = threadIdx.x; x < items; x += C::THREADS) s_places[x] = shared_places(p, x);
    fence_proxy_async_smem();
    __syncthreads();

    if (warp == 4) {
        // ------------------------------------------------------------- TMA producer
        // Copies in the order in which the products use them: K of block n, then V of block n - 1.
        // this CTA's heads are hg, hg + head_groups, ...: nh of them, taken in turn within a tile
        const int hg = cta % p.head_groups, part = cta / p.head_groups;
        const int nh = (p.Hkv - hg + p.head_groups - 1) / p.head_groups;
        SharedUnit un;
        int at = 0, item = 0, ui = 0, place = 0, left = 0, line = 0;
        Shares sh(0, 1);
        if (part < p.parts) {
            sh = find_share(
                items, p.parts, part, [&](int x) { return x < items ? s_places[x] * nh : 0; }, item, at);
            line = sh.start(part);  // the line's place that `place` of the unit is
            left = sh.start(part + 1) - line;
        }
        __syncwarp();
        if (left > 0) {
            shared_item(p, item, un);
            ui = at / (un.nblk + kSharedUnitCost);
            place = at - ui * (un.nblk + kSharedUnitCost);
        }
        bool ok = true;
        int n = 0, k = 0;                // blocks and units so far
        const CUtensorMap* v_map = nullptr;  // V of the block before
        int v_head = 0, v_row = 0;
        auto load_v = [&](int blk) {
            const int s = blk % C::VST;
            if (!warp_wait_all(&bar_vempty[s], ((blk / C::VST) & 1) ^ 1, wd, kSiteSharedEmpty)) return false;
            mbar_arrive_expect_tx_w(&bar_vfull[s], C::TILE_BYTES);
            if (!(blk == 0 && (p.debug_flags & kDebugDropFirstLoad)))
                for (int pn = 0; pn < C::PANELS; ++pn)
                    tma_load_3d_w(sV + s * C::TILE_BYTES + pn * C::PANEL_BYTES, v_map, &bar_vfull[s],
                                  64 * pn, v_head, v_row);
            return true;
        };
        int v_issued = 0;
        while (ok && left > 0) {
            const int end = min(un.nblk + kSharedUnitCost, place + left);
            left -= end - place;
            un.tile = ui / nh;
            un.hk = hg + (ui - un.tile * nh) * p.head_groups;
            un.jb = max(0, place - kSharedUnitCost);
            un.J = max(0, end - kSharedUnitCost) - un.jb;
            un.first = k == 0;
            un.odd = 0;
            // A prefix with several tiles of tokens is read by several CTAs.  Those of the later tiles
            // take their blocks in the order in which the first tile's CTAs do (from where one of its
            // shares starts, and round): then the blocks are read at the same time, and HBM gives each
            // once.  The ragged last block stays last.
            int rot = 0, full = un.J;
            if (un.item < p.groups && un.tile > 0) {
                if (un.jb + un.J == un.nblk && un.nk % kSB) --full;
                const int first = line - place - un.tile * nh * (un.nblk + kSharedUnitCost) + kSharedUnitCost + un.jb;
                rot = sh.start(sh.share_of(first) + 1) - first;
                if (rot >= full) rot = 0;
            }
            line += end - place;
            const CUtensorMap* k_map = un.item < p.groups ? &tm_kp : &tm_k;
#pragma unroll 1
            for (int jj = 0; ok && jj < un.J; ++jj, ++n) {
                const int jr = jj < full - rot ? jj + rot : jj < full ? jj + rot - full : jj;
                const int row = un.k0 + (un.jb + jr) * kSB;
                if (jj == 0) {
                    if (lane == 0) {
                        s_unit[k % kSharedUnits] = un;
                        mbar_arrive(&bar_unit[k % kSharedUnits]);
                    }
                    __syncwarp();
                    // Q: one 3-D box of (64 columns, G heads, tile_tokens tokens) per panel, rows in
                    // (token, head) order; tile rows past it are never written and never stored
                    ok = warp_wait_all(&bar_qempty, (k & 1) ^ 1, wd, kSiteSharedEmpty);
                    if (!ok) break;
                    mbar_arrive_expect_tx_w(&bar_qfull,
                                            static_cast<uint32_t>(C::PANELS * 128 * p.G.d * p.tile_tokens.d));
                    for (int pn = 0; pn < C::PANELS; ++pn)
                        tma_load_3d_w(sQ + pn * C::PANEL_BYTES, &tm_q, &bar_qfull, 64 * pn, un.hk * p.G.d,
                                      un.tok0 + un.tile * p.tile_tokens.d);
                    ++k;
                }
                const int s = n % C::KST;
                ok = warp_wait_all(&bar_kempty[s], ((n / C::KST) & 1) ^ 1, wd, kSiteSharedEmpty);
                if (!ok) break;
                mbar_arrive_expect_tx_w(&bar_kfull[s], C::TILE_BYTES);
                for (int pn = 0; pn < C::PANELS; ++pn)
                    tma_load_3d_w(sK + s * C::TILE_BYTES + pn * C::PANEL_BYTES, k_map, &bar_kfull[s],
                                  64 * pn, un.hk, row);
                if (n > 0) {
                    ok = load_v(n - 1);
                    if (ok) v_issued = n;
                }
                v_map = un.item < p.groups ? &tm_vp : &tm_v;
                v_head = un.hk;
                v_row = row;
            }
            place = 0;
            if (left > 0 && ++ui >= un.in_item * nh) {
                ui = 0;
                do shared_item(p, un.item + 1, un);
                while (un.in_item == 0 && un.item + 1 < items);
            }
        }
        if (ok && n > 0) {
            ok = load_v(n - 1);
            if (ok) v_issued = n;
        }
        if (ok && lane == 0) {  // the end of the units
            s_unit[k % kSharedUnits].J = 0;
            mbar_arrive(&bar_unit[k % kSharedUnits]);
        }
        // no copy may land after the CTA exits (bounded waits that ignore the abort flag)
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        if (k > 0) mbar_wait(&bar_qfull, (k - 1) & 1, wd_drain, kSiteSharedDrain);
        for (int i = max(0, n - C::KST); i < n; ++i)
            mbar_wait(&bar_kfull[i % C::KST], (i / C::KST) & 1, wd_drain, kSiteSharedDrain);
        for (int i = max(0, v_issued - C::VST); i < v_issued; ++i)
            mbar_wait(&bar_vfull[i % C::VST], (i / C::VST) & 1, wd_drain, kSiteSharedDrain);
    } else if (warp == 5) {
        // ------------------------------------------------------------- MMA issuer
        // Per block n: S(n + 1), perhaps of the next unit, into the other buffer as soon as its K is
        // in (the buffer held P(n - 1), whose P V product was issued before, and MMAs run in issue
        // order), then P V of block n once the softmax has written P(n).
        constexpr uint32_t kIdS = idesc_bf16_f32(128, kSB, 0, 0);   // S = Q K^T
        constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, 0, 1);    // O += P V
        const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dv0 = sdesc_sw128(smem_u32(sV), C::PANEL_BYTES, 1024);
        int committed_k = 0, committed_v = 0;
        bool ok = true;
        // the unit and block of the next S
        int ku = 0, kj = 0, kJ = 0, k_left = 0;
        // Issues S of block n if there is one: 1 issued, 0 none, -1 a wait gave up.
        auto issue_s = [&](int n) {
            if (kj == kJ) {
                if (kJ > 0) ++ku;
                if (!warp_wait_all(&bar_unit[ku % kSharedUnits], (ku / kSharedUnits) & 1, wd, kSiteSharedUnit)) return -1;
                const SharedUnit& un = s_unit[ku % kSharedUnits];
                kJ = un.J;
                k_left = un.nk - un.jb * kSB;
                kj = 0;
                if (kJ == 0) return 0;
                if (!warp_wait_all(&bar_qfull, ku & 1, wd, kSiteSharedQ)) return -1;
            }
            const int s = n % C::KST;
            if (!warp_wait_all(&bar_kfull[s], (n / C::KST) & 1, wd, kSiteSharedK)) return -1;
            tc_fence_after();
            shared_issue_qk<D, C::PANEL_BYTES>(tbase + 128 * (n & 1), dq0,
                                               sdesc_adv(dk0, s * C::TILE_BYTES), kIdS);
            mma_commit_w(&bar_sfull[n & 1]);
            mma_commit_w(&bar_kempty[s]);
            committed_k = n + 1;
            if (++kj == kJ) mma_commit_w(&bar_qempty);
            return 1;
        };
        int more = issue_s(0);
        ok = more >= 0;
        // block of the next P V in its unit, the unit's blocks here and keys from its first block here on
        int vj = 0, vJ = kJ, v_left = k_left;
#pragma unroll 1
        for (int n = 0; ok && more > 0; ++n) {
            more = issue_s(n + 1);
            if (more < 0 || !warp_wait_all(&bar_pfull, n & 1, wd, kSiteSharedP)) { ok = false; break; }
            const int s = n % C::VST;
            if (!warp_wait_all(&bar_vfull[s], (n / C::VST) & 1, wd, kSiteSharedV)) { ok = false; break; }
            tc_fence_after();
            // (16-key steps behind the unit's last key are left out)
            shared_issue_pv(tbase + 256, tbase + 128 * (n & 1),
                            sdesc_adv(dv0, s * C::TILE_BYTES), kIdPV, vj > 0,
                            min(8, (v_left - vj * kSB + 15) / 16));
            mma_commit_w(&bar_pv);
            mma_commit_w(&bar_vempty[s]);
            committed_v = n + 1;
            if (++vj == vJ) {  // S of the next unit's first block was issued above: its size is kJ
                vj = 0;
                vJ = kJ;
                v_left = k_left;
            }
        }
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        mma_commit_w(&bar_drain);
        mbar_wait(&bar_drain, 0, wd_drain, kSiteSharedDrain);
        for (int i = max(0, committed_k - C::KST); i < committed_k; ++i)
            mbar_wait(&bar_kempty[i % C::KST], (i / C::KST) & 1, wd_drain, kSiteSharedDrain);
        for (int i = max(0, committed_v - C::VST); i < committed_v; ++i)
            mbar_wait(&bar_vempty[i % C::VST], (i / C::VST) & 1, wd_drain, kSiteSharedDrain);
    } else {
        // ------------------------------------------------------------- softmax (warps 0-3)
        const int r = threadIdx.x;  // tile row = TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        const int i = p.G(r), g = r - i * p.G.d;  // token of the tile, head of the group
        // x = S * c with c = scale * log2(e); for c <= 0 the scores are scaled first so that
        // masked entries stay -inf (as in the forward kernel).
        const float c2 = p.scale_log2;
        const bool prescale = !(c2 > 0.0f);
        const float cf = prescale ? 1.0f : c2;
        if (warp == 0) {  // (while the first copies are on their way)
            const int per = (p.total_q + p.ctas - 1) / p.ctas, t0 = cta * per;
            if (t0 < p.total_q) place_tokens(p, t0, min(t0 + per, p.total_q));
        }
        bool ok = true;
        int n = 0;
        for (int k = 0; ok; ++k) {
            ok = warp_wait_all(&bar_unit[k % kSharedUnits], (k / kSharedUnits) & 1, wd, kSiteSharedUnit);
            if (!ok) break;
            SharedUnit& un = s_unit[k % kSharedUnits];
            const int J = un.J, jb = un.jb, nk = un.nk;
            if (J == 0) break;
            const uint32_t tO = tbase + lane_base + 256u;
            const int ti = un.tile * p.tile_tokens.d + i;   // token of the item
            // Key blocks from jmask on need the element-wise mask (the causal edge, the ragged last
            // block); this row sees the keys [0, klim].  A prefix is seen whole by every query.
            int jmask = nk / kSB, klim = nk - 1;
            int seen = nk;  // keys that every row of the tile sees
            if (p.causal && un.item >= p.groups) {
                const int shift = nk - un.ntok;  // bottom-right alignment
                seen = min(seen, max(0, shift + un.tile * p.tile_tokens.d + 1));
                jmask = min(jmask, seen / kSB);
                klim = min(klim, ti + shift);
            }
            const int tok_tile = min(p.tile_tokens.d, un.ntok - un.tile * p.tile_tokens.d);
            const bool valid = i < tok_tile;
            const bool any_valid = __any_sync(0xffffffffu, valid);
            float m = -INFINITY, l = 0.0f, lr = 0.0f;
            // One block.  MASKED blocks come last; apart, so that the others' loop holds neither the
            // mask nor what follows it.
            auto block = [&](auto masked_c, int j) {
                constexpr bool MASKED = decltype(masked_c)::value;
                const uint32_t tS = tbase + lane_base + 128u * (n & 1);
                if (!warp_wait_all(&bar_sfull[n & 1], (n >> 1) & 1, wd, kSiteSharedS)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                float alpha = 1.0f;
                bool need = false;
                if (!MASKED && any_valid) {  // (else P stays what it was: rows that are never stored)
                    uint32_t sr32[128];
                    tmem_ld32(tS + 0, sr32);
                    tmem_ld32(tS + 32, sr32 + 32);
                    tmem_ld32(tS + 64, sr32 + 64);
                    tmem_ld32(tS + 96, sr32 + 96);
                    tmem_wait_ld();
                    reg_fence32(sr32);
                    reg_fence32(sr32 + 32);
                    reg_fence32(sr32 + 64);
                    reg_fence32(sr32 + 96);
                    float x[128];
#pragma unroll
                    for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr32[c]);
                    if (prescale) {
#pragma unroll
                        for (int c = 0; c < 128; ++c) x[c] *= c2;
                    }
                    float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
                    for (int c = 4; c < 124; c += 8) {
                        mx0 = fmax3(mx0, x[c], x[c + 1]);
                        mx1 = fmax3(mx1, x[c + 2], x[c + 3]);
                        mx2 = fmax3(mx2, x[c + 4], x[c + 5]);
                        mx3 = fmax3(mx3, x[c + 6], x[c + 7]);
                    }
                    mx0 = fmax3(mx0, x[124], x[125]);
                    mx1 = fmax3(mx1, x[126], x[127]);
                    const float mt = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * cf;
                    // rescale only when the max grew by more than the threshold (exact either way)
                    need = mt > m + C::RESCALE_THRESHOLD;
                    if (need) {
                        alpha = ex2(m - mt);
                        m = mt;
                        l *= alpha;
                        lr *= alpha;
                    }
                    const float neg_m = (m == -INFINITY) ? 0.0f : -m;
                    const uint64_t cf2 = f2_make(cf, cf), nm2 = f2_make(neg_m, neg_m);
                    uint64_t lsa = f2_make(0.f, 0.f), lsb = lsa, lra = lsa, lrb = lsa;
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const int e = cb * 32 + c;
                            float p0, p1, p2, p3;
                            f2_split(f2_fma(f2_make(x[e], x[e + 1]), cf2, nm2), p0, p1);
                            f2_split(f2_fma(f2_make(x[e + 2], x[e + 3]), cf2, nm2), p2, p3);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            p2 = ex2(p2);
                            p3 = ex2(p3);
                            const uint32_t w01 = pack_bf16x2(p0, p1);
                            const uint32_t w23 = pack_bf16x2(p2, p3);
                            lsa = f2_add(lsa, f2_make(p0, p1));
                            lsb = f2_add(lsb, f2_make(p2, p3));
                            // lr sums the bf16-rounded weights the P V product uses
                            lra = f2_add(lra, f2_make(__uint_as_float(w01 << 16), __uint_as_float(w01 & 0xFFFF0000u)));
                            lrb = f2_add(lrb, f2_make(__uint_as_float(w23 << 16), __uint_as_float(w23 & 0xFFFF0000u)));
                            pk[c / 2] = w01;
                            pk[c / 2 + 1] = w23;
                        }
                        tmem_st16(tS + 16u * cb, pk);
                    }
                    {
                        float a0, a1, b0, b1;
                        f2_split(f2_add(lsa, lsb), a0, a1);
                        f2_split(f2_add(lra, lrb), b0, b1);
                        l += a0 + a1;
                        lr += b0 + b1;
                    }
                }
                if (MASKED && any_valid) {
                    // 32 columns at a time, up to the last that any row needs; P of a chunk goes where
                    // S of that chunk or of one before it was.  Rolled up: these blocks are one in a
                    // unit, and code that is fetched for them alone costs more than their time.
                    const int lim = klim - j * kSB;  // last visible key column in this block
                    const int chunks = min(4, (nk - j * kSB + 31) / 32);
                    float mt = -INFINITY;
#pragma unroll 1
                    for (int cb = 0; cb < chunks; ++cb) {
                        uint32_t v[32];
                        tmem_ld32(tS + 32u * cb, v);
                        tmem_wait_ld();
                        reg_fence32(v);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (32 * cb + c <= lim) mt = fmaxf(mt, __uint_as_float(v[c]) * c2);
                    }
                    need = mt > m + C::RESCALE_THRESHOLD;
                    if (need) {
                        alpha = ex2(m - mt);
                        m = mt;
                        l *= alpha;
                        lr *= alpha;
                    }
                    const float neg_m = (m == -INFINITY) ? 0.0f : -m;
#pragma unroll 1
                    for (int cb = 0; cb < chunks; ++cb) {
                        uint32_t v[32], pk[16];
                        tmem_ld32(tS + 32u * cb, v);
                        tmem_wait_ld();
                        reg_fence32(v);
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float w[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float xs = __uint_as_float(v[c + e]);
                                w[e] = 32 * cb + c + e <= lim ? ex2(fmaf(xs, c2, neg_m)) : 0.0f;
                                l += w[e];
                            }
                            pk[c / 2] = pack_bf16x2(w[0], w[1]);
                            lr += __uint_as_float(pk[c / 2] << 16) + __uint_as_float(pk[c / 2] & 0xFFFF0000u);
                        }
                        tmem_st16(tS + 16u * cb, pk);
                    }
                }
                if constexpr (MASKED) {
                    const int first = max(0, seen - j * kSB), end = nk - j * kSB;
                    const int last = min(kSB, (end + 15) & ~15);
                    if (first < last) {
                        const int s = n % C::VST;
                        if (!warp_wait_all(&bar_vfull[s], (n / C::VST) & 1, wd, kSiteSharedV)) {
                            ok = false;
                            return;
                        }
                        if (clear_unseen_v<D>(sV + s * C::TILE_BYTES, first, end, last)) un.odd = 1;
                    }
                }
                // O holds the unit's blocks before this one once their last P V product has run
                if (j > jb) {
                    if (!warp_wait_all(&bar_pv, (n - 1) & 1, wd, kSiteSharedO)) {
                        ok = false;
                        return;
                    }
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
                        for (int ch = 0; ch < D / 32; ++ch) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32u * ch, o);
                            tmem_wait_ld();
                            reg_fence32(o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            tmem_st32(tO + 32u * ch, o);
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_pfull);
                ++n;
            };
            const int j1 = jb + J, j0 = min(j1, max(jb, jmask));
#pragma unroll 1
            for (int j = jb; ok && j < j0; ++j) block(std::false_type{}, j);
#pragma unroll 1
            for (int j = j0; ok && j < j1; ++j) block(std::true_type{}, j);
            // ------------------------------------------------------------- the unit's result
            // O normalised by its own weights and its natural-log LSE, in fp32 for the merge: to
            // the row's place if the share holds the whole unit, else to the share's part.
            if (ok) ok = warp_wait_all(&bar_pv, (n - 1) & 1, wd, kSiteSharedO);
            if (!ok) break;
            tc_fence_after();
            const bool whole = J == un.nblk;
            const int h = un.hk * p.G.d + g;
            const float inv_l = lr > 0.0f ? 1.0f / lr : (lr == 0.0f ? 0.0f : NAN);
            const float lse_row = l > 0.0f ? (m + __log2f(l)) * kLn2 : (l == 0.0f ? -INFINITY : NAN);
            long long row;
            if (whole)
                row = (static_cast<long long>(un.item < p.groups ? 0 : p.total_q) + un.tok0 + ti) * p.H + h;
            else
                row = p.part_row0 + (2ll * cta + (un.first ? 0 : 1)) * 128 + r;
            const bool in = valid && in_extent(row, 1, p.part_ext, p.status);
            const bool odd = *static_cast<volatile int*>(&un.odd) != 0;
#pragma unroll 1
            for (int ch = 0; any_valid && ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(tO + 32u * ch, o);
                tmem_wait_ld();
                reg_fence32(o);
                if (!in) continue;
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv_l);
                st_row<4>(p.o_part + row * D + 32 * ch, o);
            }
            if (in) p.lse_part[row] = lse_row;
            if (in && odd)
                add_odd_v<D>(p, p.o_part + row * D, un, max(seen, jb * kSB), min(min(nk, (jb + J) * kSB), klim + 1));
            // (the next unit's first P V product overwrites O: it waits for this warp's next P)
            tc_fence_before();
        }
    }

    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
}

// Merge: one warp for each query row (token and head) gathers the row's parts, those of its
// group's prefix and those of its sequence's keys.  A row that saw no key in any gets O = 0, lse = -inf.
// The attention CTAs leave beside the parts where each token's lie: ahead of its wait the kernel may read no
// lengths, and a scan of them behind it would cost every warp several round trips.
template <int D, int BATCH>
__global__ void __launch_bounds__(128) fa_decode_shared_merge_kernel(const SharedDecodeParams p)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const int w = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int tok = w / p.H, h = w - tok * p.H;
    const int hk = p.G(h), hg = hk % p.head_groups, hj = hk / p.head_groups;
    const int nh = (p.Hkv - hg + p.head_groups - 1) / p.head_groups;
    dependent_begin();
    if (tok >= p.total_q) return;
    int4 at[2];  // its group's prefix, its own keys
    at[0] = p.places[2ll * tok + 1];
    at[1] = p.places[2ll * tok];
    if (at[1].z < 0) return;
    const Shares sh(at[1].w * nh, p.parts);
    int count[2] = {0, 0}, c0[2], lead[2], row[2] = {0, 0};
    bool whole[2] = {false, false};
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const int nblk = at[z].y, ti = at[z].z;
        if (nblk == 0) continue;
        const int tile = p.tile_tokens(ti);
        const int start = at[z].x * nh + (tile * nh + hj) * (nblk + kSharedUnitCost) + kSharedUnitCost;
        const int s0 = sh.share_of(start), s1 = sh.share_of(start + nblk - 1);
        c0[z] = s0 * p.head_groups + hg;
        count[z] = s1 - s0 + 1;
        whole[z] = s1 == s0;
        lead[z] = sh.start(s0) >= start - kSharedUnitCost ? 0 : 1;
        row[z] = whole[z] ? ((z ? p.total_q : 0) + tok) * p.H + h
                          : static_cast<int>(p.part_row0) + (ti - tile * p.tile_tokens.d) * p.G.d + (h - hk * p.G.d);
    }
    float mx, sum, acc[EPL];
    merge_parts<D, BATCH>(
        count[0] + count[1],
        [&](int k) {
            const bool z = k >= count[0];
            const int c = z ? k - count[0] : k, first = (z ? row[1] : row[0]);
            return (z ? whole[1] : whole[0]) ? first
                                             : first + (2 * ((z ? c0[1] : c0[0]) + c * p.head_groups) +
                                                        (c == 0 ? (z ? lead[1] : lead[0]) : 0)) * 128;
        },
        p.o_part, p.lse_part, p.part_ext, p.status, mx, sum, acc);
    const long long out = (static_cast<long long>(tok) * p.H + h) * D + EPL * lane;
    const long long stat = static_cast<long long>(h) * p.total_q + tok;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (in_extent(out, EPL, p.q_ext, p.status)) {
        if constexpr (EPL == 4)
            *reinterpret_cast<uint2*>(p.o + out) = make_uint2(
                pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(p.o + out) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
    if (lane == 0 && p.lse != nullptr && in_extent(stat, 1, p.stat_ext, p.status))
        p.lse[stat] = sum == 0.0f ? -INFINITY : mx + logf(sum);
}

template <int D>
static cudaError_t launch_decode_shared_impl(const CUtensorMap* maps, const SharedDecodeParams& p, cudaStream_t st,
                                             int num_sms)
{
    using C = SharedCfg<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(fa_decode_shared_kernel<D>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    cudaError_t e = launch_dependent(fa_decode_shared_kernel<D>, dim3(p.ctas), dim3(C::THREADS), C::SMEM_BYTES,
                                     st, maps[0], maps[1], maps[2], maps[3], maps[4], p);
    if (e != cudaSuccess) return e;
    // The merge's CTAs start beside the attention's and wait there; with few rows they all fit with 16
    // parts in flight each (8 queries: 13.3 us, 13.8 with 8), with many only with 8 (64 queries: 63.9 us,
    // with 16 a second wave starts late, 68.2).
    const long long rows = static_cast<long long>(p.total_q) * p.H;
    const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
    return rows <= 8ll * num_sms
               ? launch_dependent(fa_decode_shared_merge_kernel<D, 16>, grid, dim3(128), 0, st, p)
               : launch_dependent(fa_decode_shared_merge_kernel<D, 8>, grid, dim3(128), 0, st, p);
}

// maps: q, k_prefix, v_prefix, k, v
cudaError_t launch_decode_shared(int d, const CUtensorMap* maps, const SharedDecodeParams& p, cudaStream_t st,
                                 int num_sms)
{
    return d == 64 ? launch_decode_shared_impl<64>(maps, p, st, num_sms)
                   : launch_decode_shared_impl<128>(maps, p, st, num_sms);
}

}  // namespace fa
