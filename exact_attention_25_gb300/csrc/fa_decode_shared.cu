// Decoding for batches whose sequences share long prefixes, on sm_103a tensor cores: the queries of
// a group of sequences attend to the group's prefix, all as one tile of rows, and each sequence's
// queries to its own keys (bottom-right causal mask), under one softmax:
//     O = softmax([q K_p^T, q K_s^T] scale) [V_p; V_s].
// The two ranges of keys are computed apart, each with its own online softmax, and merged by the
// rescaling rule O = sum_s e^{lse_s} O_s / sum_s e^{lse_s}; so a prefix is read once for its group
// and not once for each sequence, and its products have the rows of the whole group.
//
// What bounds it: reading prefix and own keys once (HBM), and for large groups the exponentials of
// tokens x heads x prefix scores.  Both kinds of work are units of one line (units, below) shared
// out evenly over the SMs, so memory-bound and arithmetic-bound units run side by side.
//
// A unit is a tile of up to 128 query rows (row r = i * G + g: token i of the tile, head g of the G
// that share the K/V head) against the keys of one prefix or sequence.  Roles (6 warps): warps 0-3
// softmax (thread = tile row = TMEM lane), warp 4 TMA producer, warp 5 TMEM allocator and MMA
// issuer.  All of them run over the CTA's whole share without a barrier between units: Q tiles and
// O accumulators alternate between two buffers, so a unit's first scores are computed while the
// softmax warps still write out the unit before it.  TMEM: two S buffers [0,128), [128,256) (P of a
// block, bf16 pairs, overwrites the upper half of its S buffer), two O buffers from 256 on.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

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
    static constexpr int VST = D == 128 ? 2 : 5;
    static constexpr int SMEM_BYTES = (2 + KST + VST) * TILE_BYTES + 1024;
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
    int in_item;           // units of the item
    int jb, J;             // this share's blocks of the unit: [jb, jb + J)
    int first;             // the share's first unit
    int odd;               // V holds infinities or NaNs that only some of the tile's rows see
};

// Sizes of an item: in_item units of nblk blocks each (none without tokens or keys).
__device__ __forceinline__ void shared_item(const SharedDecodeParams& p, int x, SharedUnit& u)
{
    u.item = x;
    if (x < p.groups) {
        const int b0 = min(max(p.cu_g[x], 0), p.B), b1 = min(max(p.cu_g[x + 1], b0), p.B);
        u.tok0 = min(max(p.cu_q[b0], 0), p.total_q);
        u.ntok = min(min(max(p.cu_q[b1], u.tok0), p.total_q) - u.tok0, p.max_group_q);
        u.nk = packed_rows(p.cu_p, x, p.total_p, p.max_p, u.k0);
    } else {
        u.ntok = packed_rows(p.cu_q, x - p.groups, p.total_q, p.max_q, u.tok0);
        u.nk = packed_rows(p.cu_k, x - p.groups, p.total_k, p.max_k, u.k0);
    }
    u.nblk = (u.nk + kSB - 1) / kSB;
    u.in_item = u.nk > 0 ? (u.ntok + p.tile_tokens - 1) / p.tile_tokens * p.Hkv : 0;
}

__device__ __forceinline__ int shared_places(const SharedDecodeParams& p, int x)
{
    if (x >= p.groups + p.B) return 0;
    SharedUnit u;
    shared_item(p, x, u);
    return u.in_item * (u.nblk + kUnitCost);
}

// All lanes of a warp: the places of the items before `stop` (all of them: the line's length).
__device__ __forceinline__ int places_before(const SharedDecodeParams& p, int stop)
{
    const int lane = threadIdx.x & 31;
    int sum = 0;
    for (int x0 = 0; x0 < stop; x0 += 32) sum += x0 + lane < stop ? shared_places(p, x0 + lane) : 0;
    return __reduce_add_sync(0xffffffffu, sum);
}

// All lanes of a warp: the item at place pos of the line (below its length), and pos's distance
// from the item's first place.
__device__ __forceinline__ void find_item(const SharedDecodeParams& p, int pos, SharedUnit& u, int& at)
{
    const int lane = threadIdx.x & 31, items = p.groups + p.B;
    int run = 0;
    for (int x0 = 0; x0 < items; x0 += 32) {
        const int w = shared_places(p, x0 + lane);
        int sum = w;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += up;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run + sum > pos);
        if (past) {
            const int src = __ffs(past) - 1;
            at = pos - run - __shfl_sync(0xffffffffu, sum - w, src);
            shared_item(p, x0 + src, u);
            return;
        }
        run += __shfl_sync(0xffffffffu, sum, 31);
    }
}

// Two bf16 values, infinities and NaNs replaced by zero.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v)
{
    if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
    if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
    return v;
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

// O += P V: P (bf16 pairs) from TMEM, V (MN-major) from shared memory; 8 k-steps of 16 keys.
__device__ __forceinline__ void shared_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t vdesc,
                                                uint32_t idesc, uint32_t acc_first)
{
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
        mma_ts_w(d_tmem, p_tmem + 8u * ks, sdesc_adv(vdesc, ks * 2048), idesc, ks > 0 ? 1u : acc_first);
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
    uint8_t* sK = sQ + 2 * C::TILE_BYTES;
    uint8_t* sV = sK + C::KST * C::TILE_BYTES;

    __shared__ __align__(8) uint64_t bar_qfull[2], bar_qempty[2];
    __shared__ __align__(8) uint64_t bar_kfull[C::KST], bar_kempty[C::KST];
    __shared__ __align__(8) uint64_t bar_vfull[C::VST], bar_vempty[C::VST];
    __shared__ __align__(8) uint64_t bar_unit[kSharedUnits];
    __shared__ __align__(8) uint64_t bar_sfull[2];  // S of a block landed in buffer b
    __shared__ __align__(8) uint64_t bar_pfull;     // softmax wrote P (and rescaled O)
    __shared__ __align__(8) uint64_t bar_pv;        // the P V product of a block has run
    __shared__ __align__(8) uint64_t bar_ofree[2];  // O buffer b has been read out
    __shared__ __align__(8) uint64_t bar_drain;
    __shared__ SharedUnit s_unit[kSharedUnits];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_qfull[i], 1);
            mbar_init(&bar_qempty[i], 1);
            mbar_init(&bar_sfull[i], 1);
            mbar_init(&bar_ofree[i], 4);
        }
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

    if (warp == 4) {
        // ------------------------------------------------------------- TMA producer
        // Copies in the order in which the products use them: K of block n, then V of block n - 1.
        const Shares sh(places_before(p, p.groups + p.B), p.ctas);
        int left = sh.start(cta + 1) - sh.start(cta);
        SharedUnit un;
        int at = 0, ui = 0, place = 0;
        if (left > 0) {
            find_item(p, sh.start(cta), un, at);
            ui = at / (un.nblk + kUnitCost);
            place = at - ui * (un.nblk + kUnitCost);
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
            const int end = min(un.nblk + kUnitCost, place + left);
            left -= end - place;
            un.hk = ui % p.Hkv;
            un.tile = ui / p.Hkv;
            un.jb = max(0, place - kUnitCost);
            un.J = max(0, end - kUnitCost) - un.jb;
            un.first = k == 0;
            un.odd = 0;
            const CUtensorMap* k_map = un.item < p.groups ? &tm_kp : &tm_k;
            for (int jj = 0; ok && jj < un.J; ++jj, ++n) {
                const int row = un.k0 + (un.jb + jj) * kSB;
                if (jj == 0) {
                    if (lane == 0) {
                        s_unit[k % kSharedUnits] = un;
                        mbar_arrive(&bar_unit[k % kSharedUnits]);
                    }
                    __syncwarp();
                    // Q: one 3-D box of (64 columns, G heads, tile_tokens tokens) per panel, rows in
                    // (token, head) order; tile rows past it are never written and never stored
                    const int qs = k & 1;
                    ok = warp_wait_all(&bar_qempty[qs], ((k >> 1) & 1) ^ 1, wd, kSiteSharedEmpty);
                    if (!ok) break;
                    mbar_arrive_expect_tx_w(&bar_qfull[qs],
                                            static_cast<uint32_t>(C::PANELS * 128 * p.G * p.tile_tokens));
                    for (int pn = 0; pn < C::PANELS; ++pn)
                        tma_load_3d_w(sQ + qs * C::TILE_BYTES + pn * C::PANEL_BYTES, &tm_q, &bar_qfull[qs],
                                      64 * pn, un.hk * p.G, un.tok0 + un.tile * p.tile_tokens);
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
            if (left > 0 && ++ui >= un.in_item) {
                ui = 0;
                do shared_item(p, un.item + 1, un);
                while (un.in_item == 0);
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
        for (int i = max(0, k - 2); i < k; ++i) mbar_wait(&bar_qfull[i & 1], (i >> 1) & 1, wd_drain, kSiteSharedDrain);
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
        int ku = 0, kj = 0, kJ = 0;
        // Issues S of block n if there is one: 1 issued, 0 none, -1 a wait gave up.
        auto issue_s = [&](int n) {
            if (kj == kJ) {
                if (kJ > 0) ++ku;
                if (!warp_wait_all(&bar_unit[ku % kSharedUnits], (ku / kSharedUnits) & 1, wd, kSiteSharedUnit)) return -1;
                kJ = s_unit[ku % kSharedUnits].J;
                kj = 0;
                if (kJ == 0) return 0;
                if (!warp_wait_all(&bar_qfull[ku & 1], (ku >> 1) & 1, wd, kSiteSharedQ)) return -1;
            }
            const int s = n % C::KST;
            if (!warp_wait_all(&bar_kfull[s], (n / C::KST) & 1, wd, kSiteSharedK)) return -1;
            tc_fence_after();
            shared_issue_qk<D, C::PANEL_BYTES>(tbase + 128u * (n & 1), sdesc_adv(dq0, (ku & 1) * C::TILE_BYTES),
                                               sdesc_adv(dk0, s * C::TILE_BYTES), kIdS);
            mma_commit_w(&bar_sfull[n & 1]);
            mma_commit_w(&bar_kempty[s]);
            committed_k = n + 1;
            if (++kj == kJ) mma_commit_w(&bar_qempty[ku & 1]);
            return 1;
        };
        int more = issue_s(0);
        ok = more >= 0;
        int vu = 0, vj = 0, vJ = ok && more ? s_unit[0].J : 0;  // unit and block of the next P V
        for (int n = 0; ok && more > 0; ++n) {
            more = issue_s(n + 1);
            if (more < 0 || !warp_wait_all(&bar_pfull, n & 1, wd, kSiteSharedP)) { ok = false; break; }
            const int s = n % C::VST;
            if (!warp_wait_all(&bar_vfull[s], (n / C::VST) & 1, wd, kSiteSharedV)) { ok = false; break; }
            if (vj == 0 && !warp_wait_all(&bar_ofree[vu & 1], ((vu >> 1) & 1) ^ 1, wd, kSiteSharedO)) {
                ok = false;
                break;
            }
            tc_fence_after();
            shared_issue_pv(tbase + 256u + 128u * (vu & 1), tbase + 128u * (n & 1) + 64u,
                            sdesc_adv(dv0, s * C::TILE_BYTES), kIdPV, vj > 0 ? 1u : 0u);
            mma_commit_w(&bar_pv);
            mma_commit_w(&bar_vempty[s]);
            committed_v = n + 1;
            if (++vj == vJ) {  // S of the next unit's first block was issued above: its size is kJ
                ++vu;
                vj = 0;
                vJ = kJ;
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
        const int i = r / p.G, g = r - i * p.G;  // token of the tile, head of the group
        // x = S * c with c = scale * log2(e); for c <= 0 the scores are scaled first so that
        // masked entries stay -inf (as in the forward kernel).
        const float c2 = p.scale_log2;
        const bool prescale = !(c2 > 0.0f);
        const float cf = prescale ? 1.0f : c2;
        bool ok = true;
        int n = 0;
        for (int k = 0; ok; ++k) {
            ok = warp_wait_all(&bar_unit[k % kSharedUnits], (k / kSharedUnits) & 1, wd, kSiteSharedUnit);
            if (!ok) break;
            SharedUnit& un = s_unit[k % kSharedUnits];
            const int J = un.J, jb = un.jb, nk = un.nk;
            if (J == 0) break;
            const uint32_t tO = tbase + lane_base + 256u + 128u * (k & 1);
            const int ti = un.tile * p.tile_tokens + i;   // token of the item
            // Key blocks from jmask on need the element-wise mask (the causal edge, the ragged last
            // block); this row sees the keys [0, klim].  A prefix is seen whole by every query.
            int jmask = nk / kSB, klim = nk - 1;
            int seen = nk;  // keys that every row of the tile sees
            if (p.causal && un.item >= p.groups) {
                const int shift = nk - un.ntok;  // bottom-right alignment
                seen = min(seen, max(0, shift + un.tile * p.tile_tokens + 1));
                jmask = min(jmask, seen / kSB);
                klim = min(klim, ti + shift);
            }
            float m = -INFINITY, l = 0.0f, lr = 0.0f;
            for (int jj = 0; jj < J; ++jj, ++n) {
                const int j = jb + jj;
                const uint32_t tS = tbase + lane_base + 128u * (n & 1);
                if (!warp_wait_all(&bar_sfull[n & 1], (n >> 1) & 1, wd, kSiteSharedS)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
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
                if (j >= jmask) {
                    const int lim = klim - j * kSB;  // last visible key column in this block
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > lim) x[c] = -INFINITY;
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
                float alpha = 1.0f;
                const bool need = mt > m + C::RESCALE_THRESHOLD;
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
                    tmem_st16(tS + 64u + 16u * cb, pk);
                }
                {
                    float a0, a1, b0, b1;
                    f2_split(f2_add(lsa, lsb), a0, a1);
                    f2_split(f2_add(lra, lrb), b0, b1);
                    l += a0 + a1;
                    lr += b0 + b1;
                }
                if (j >= jmask) {
                    // V of keys that some row does not see must not reach it as 0 * inf or 0 * NaN:
                    // rows past the keys' end (whatever lies there) are zeroed; of rows that some
                    // queries see, what is not finite is taken out here and given back to those
                    // queries at the unit's end.
                    const int key = j * kSB + r;
                    if (__any_sync(0xffffffffu, key >= seen)) {
                        const int s = n % C::VST;
                        if (!warp_wait_all(&bar_vfull[s], (n / C::VST) & 1, wd, kSiteSharedV)) {
                            ok = false;
                            break;
                        }
                        if (key >= seen) {
                            for (int c = 0; c < D / 8; ++c) {
                                uint4* at = reinterpret_cast<uint4*>(
                                    sV + s * C::TILE_BYTES + (c / 8) * C::PANEL_BYTES + r * 128 + (c % 8) * 16);
                                if (key >= nk) {
                                    *at = make_uint4(0u, 0u, 0u, 0u);
                                    continue;
                                }
                                const uint4 v = *at;
                                const uint4 f = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y),
                                                           finite_bf16x2(v.z), finite_bf16x2(v.w));
                                if (f.x != v.x || f.y != v.y || f.z != v.z || f.w != v.w) {
                                    *at = f;
                                    un.odd = 1;
                                }
                            }
                        }
                        fence_proxy_async_smem();
                    }
                }
                // O holds the unit's blocks before this one once their last P V product has run
                if (jj > 0) {
                    if (!warp_wait_all(&bar_pv, (n - 1) & 1, wd, kSiteSharedO)) {
                        ok = false;
                        break;
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
            }
            // ------------------------------------------------------------- the unit's result
            // O normalised by its own weights and its natural-log LSE, in fp32 for the merge: to
            // the row's place if the share holds the whole unit, else to the share's part.
            if (ok) ok = warp_wait_all(&bar_pv, (n - 1) & 1, wd, kSiteSharedO);
            if (!ok) break;
            tc_fence_after();
            const int tok_tile = min(p.tile_tokens, un.ntok - un.tile * p.tile_tokens);
            const bool valid = i < tok_tile;
            const bool whole = J == un.nblk;
            const int h = un.hk * p.G + g;
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
            for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(tO + 32u * ch, o);
                tmem_wait_ld();
                reg_fence32(o);
                if (!in) continue;
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv_l);
                if (odd) {
                    const int key1 = min(min(nk, (jb + J) * kSB), klim + 1);
                    for (int key = max(seen, jb * kSB); key < key1; ++key) {
                        const long long off = (static_cast<long long>(un.k0 + key) * p.Hkv + un.hk) * D + 32 * ch;
                        if (!in_extent(off, 32, p.v_ext, p.status)) continue;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float v = __bfloat162float(p.v[off + c]);
                            if (!(fabsf(v) < INFINITY)) o[c] = __float_as_uint(__uint_as_float(o[c]) + v);
                        }
                    }
                }
                st_row<4>(p.o_part + row * D + 32 * ch, o);
            }
            if (in) p.lse_part[row] = lse_row;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_ofree[k & 1]);
        }
    }

    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
}

// Merge: one warp for each query row (token and head) gathers the row's parts, those of its
// group's prefix and those of its sequence's keys:
//     O = sum_s e^{lse_s} O_s / sum_s e^{lse_s},   lse = log sum_s e^{lse_s}.
// Only parts that saw a key (lse_s > -inf) are read; a row without any gets O = 0, lse = -inf.
// It is always launched behind the attention kernel of its call, whose CTAs let it start only after
// their own wait: so the lengths, which that wait has made visible, are read before this kernel's.
template <int D>
__global__ void __launch_bounds__(128) fa_decode_shared_merge_kernel(const SharedDecodeParams p)
{
    constexpr int EPL = D / 32;
    constexpr int BATCH = 4;  // parts whose rows are in flight together
    const int lane = threadIdx.x & 31;
    const int w = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int h = w % p.H;
    const int i = w / p.H % p.max_q, b = w / p.H / p.max_q;
    SharedUnit u[2];  // its group's prefix, its own keys
    int count[2] = {0, 0}, c0[2], lead[2];
    long long row[2] = {0, 0};
    bool here = b < p.B, whole[2] = {false, false};
    int tok = 0;
    if (here) {
        shared_item(p, p.groups + b, u[1]);
        tok = u[1].tok0 + i;
        here = i < u[1].ntok;
    }
    if (here) {
        int x = 0;  // the group: groups are runs of sequences
        u[0].in_item = 0;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const bool in = g0 + lane < p.groups && p.cu_g[g0 + lane] <= b && b < p.cu_g[g0 + lane + 1];
            const uint32_t some = __ballot_sync(0xffffffffu, in);
            if (some) {
                x = g0 + __ffs(some) - 1;
                shared_item(p, x, u[0]);
                break;
            }
        }
        const Shares sh(places_before(p, p.groups + p.B), p.ctas);
        const int hk = h / p.G;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int ti = tok - u[z].tok0;
            if (u[z].in_item == 0 || ti < 0 || ti >= u[z].ntok) continue;
            const int tile = ti / p.tile_tokens;
            const int start = places_before(p, u[z].item) +
                              (tile * p.Hkv + hk) * (u[z].nblk + kUnitCost) + kUnitCost;
            c0[z] = sh.share_of(start);
            const int c1 = sh.share_of(start + u[z].nblk - 1);
            count[z] = c1 - c0[z] + 1;
            whole[z] = c1 == c0[z];
            lead[z] = sh.start(c0[z]) >= start - kUnitCost ? 0 : 1;
            row[z] = whole[z] ? (static_cast<long long>(z ? p.total_q : 0) + tok) * p.H + h
                              : p.part_row0 + (ti - tile * p.tile_tokens) * p.G + (h - hk * p.G);
        }
    }
    dependent_begin();
    if (!here) return;
    auto row_of = [&](int k) {
        const int z = k < count[0] ? 0 : 1;
        const int c = z ? k - count[0] : k;
        return whole[z] ? row[z] : row[z] + (2ll * (c0[z] + c) + (c == 0 ? lead[z] : 0)) * 128;
    };
    const int parts = count[0] + count[1];
    float mx = -INFINITY, sum = 0.0f, acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
    for (int s0 = 0; s0 < parts; s0 += 32) {
        const bool mine = s0 + lane < parts;
        const long long r = mine ? row_of(s0 + lane) : 0;
        float ls = -INFINITY;
        if (mine && in_extent(r, 1, p.part_ext, p.status)) ls = p.lse_part[r];
        float bm = ls;
        uint32_t live = __ballot_sync(0xffffffffu, !(ls == -INFINITY));  // NaN counts
#pragma unroll
        for (int d = 16; d; d >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, d));
        if (!live) continue;
        const float nm = fmaxf(mx, bm);
        const float keep = mx == -INFINITY ? 0.0f : expf(mx - nm);
        sum *= keep;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] *= keep;
        mx = nm;
        const float wt = ls == -INFINITY ? 0.0f : expf(ls - nm);
        while (live) {
            float v[BATCH][EPL], ws[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                ws[k] = 0.0f;
#pragma unroll
                for (int e = 0; e < EPL; ++e) v[k][e] = 0.0f;
                if (live) {
                    const int s = __ffs(live) - 1;
                    live &= live - 1;
                    ws[k] = __shfl_sync(0xffffffffu, wt, s);
                    const float* src = p.o_part + __shfl_sync(0xffffffffu, r, s) * D + EPL * lane;
                    if constexpr (EPL == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2*>(src);
                        v[k][0] = x.x; v[k][1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                sum += ws[k];
#pragma unroll
                for (int e = 0; e < EPL; ++e) acc[e] = fmaf(ws[k], v[k][e], acc[e]);
            }
        }
    }
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
static cudaError_t launch_decode_shared_impl(const CUtensorMap* maps, const SharedDecodeParams& p, cudaStream_t st)
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
    const long long rows = static_cast<long long>(p.B) * p.max_q * p.H;
    return launch_dependent(fa_decode_shared_merge_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)),
                            dim3(128), 0, st, p);
}

// maps: q, k_prefix, v_prefix, k, v
cudaError_t launch_decode_shared(int d, const CUtensorMap* maps, const SharedDecodeParams& p, cudaStream_t st)
{
    return d == 64 ? launch_decode_shared_impl<64>(maps, p, st) : launch_decode_shared_impl<128>(maps, p, st);
}

}  // namespace fa
