// Attention of trees of drafted tokens over the paged e4m3 cache: O = softmax(scale Q K^T + mask) V
// for the bf16 queries of a sequence's drafted tokens, where every token sees the sequence's history
// and, of the drafted keys, those that its row of mask bits names (its ancestors and itself).  K and V
// are the cache's codes times their rows' powers of two, which are not rounded on the way in.  Q becomes f16
// under a power of two a row, exactly down to 2^-31 of the row's largest (down to 2^-38 something is left).  The result
// is exact attention on those up to fp32 accumulation and the f16 rounding of the softmax weights.
//
// A tree has tens of tokens, so a key/value head has 32 to 256 query rows and more: too many for the
// cache decode's products in registers (64 rows read every code four times from shared memory), but
// enough for tcgen05 tiles of 128 rows.  Those want 16-bit operands, so eight warps convert the codes of each
// step of 64 keys first.
//
// Work is cut as in the cache decode: a line of units (sequence, up to 128 query rows r = i * G + g, i
// the token and g the head of the G that share the K/V head), shared out evenly over one CTA an SM, the
// parts of a unit that several shares cut merged by a second kernel.  (Before the steps below were made faster: units of two tiles of 128 rows, which converted
// the codes once for both, were slower: 64 tokens in 249 us where these took 240.  With P over S, for want of room in
// TMEM, a stream's next scores waited for its product.)
//
// What bounds it: the chain of a step, some 1400 clocks of 64 keys, in which every part (copy, exponents, conversion, product,
// softmax, product) takes a warp 500 to 1400; the schedulers issue half the time and the tensor cores run a third of it.  On 8
// sequences of up to 32 K keys, H = 32 / Hkv = 8, d = 128: trees of up to 24 tokens 110 us (2.85 TB/s of codes), of 64
// tokens 217 us (0.72 PFLOP/s).  Registers decide how the softmax's loop is written: 20 warps have 96 each, and a few of its
// values in local memory cost a quarter (O rescaled 64 columns at a time, scores read once and kept: 140 to 147 us).  The sum's
// own frame costs 2 and 5 us; its part of a step added after the weights are handed on the same, one vote for both maxima
// 111 and 220.
//
// Roles of a CTA (20 warps):
//  - warp 16 copies pages of codes and exponents to a ring of raw tiles, 16.1 KB a step at d = 128, a lane each of a
//    step's copies.
//  - warp 19 looks at the exponents of each step that has landed.
//  - warps 8-15, in pairs, bring the codes of K and of V, of even and odd steps, to f16 tiles (rows of 128 bytes,
//    swizzled); all of them, and for the first unit warps 0-7, also Q (a row scaled by a power of two to just below
//    2^15, elements down to 2^-38 of its largest keep a value).
//  - warps 17 and 18 issue the products S = Q K^T and O += P V.
//  - warps 0-3 and 4-7 are the softmax of two streams, even and odd steps, each with an O accumulator of its own in TMEM
//    (thread = row = TMEM lane): what one waits for, the other's steps cover.  S is computed up to four steps ahead.
//    The streams' sums are joined at the unit's end.
//
// Number ranges.  The converted codes of a step hold their rows' powers of two relative to the step's largest
// (exactly: both spread over few binades), so x = S c with one factor a row and step, and V's tile stands for V 2^-E,
// E the step's largest exponent.  Two running maxima are kept, as in the cache decode.  M, of x + E, frames the weights:
// w = 2^(x + E - M + 7), f16, multiplies V's tile.  Weights keep 11 bits down to 2^-21 of the largest (a maximum moves when
// it is exceeded by more than 8, so w <= 2^15), and f16's smallest step puts a floor of 2^-32 of the largest under what
// a single key can still add.  m, of x, frames the sum l of 2^(x - m), which has nothing to do with V.  A step's part of it is
// the sum of its w in fp32 times 2^(M - E - 7 - m): one exponential a row.  Where w is too small for that although the
// keys count in l (a step whose V rows are far smaller than another's), the step's 2^(x - m) are computed for
// themselves.  M - m is V's size, up to 2^+-126, so the result's power of two is applied in halves.  Steps whose rows' sizes
// lie further apart go key by key: K's scale multiplies the score, V's exponent E becomes the row's own, and the tiles
// hold the plain codes.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

#include <type_traits>

namespace fa {

namespace {

constexpr int kTB = kCacheBlock;   // keys of a block, by which the work is shared out
constexpr int kHalf = 64;          // keys of a step
constexpr int kTreeUnits = 32;     // units described ahead
constexpr int kRing = 16;          // steps that something is known of (SLOTS + 6 at least: see the scout)
constexpr int kTile = 128;         // query rows of a tile
constexpr int kMergeThreads = 128;
constexpr float kGrow = 8.0f;      // a maximum moves when it is exceeded by more than this (in a warp of 32 rows one grows at most steps:
                                   // with 4, two of three steps rescaled O; 64 tokens 215 us in place of 212)
// A step's largest weight below 2^(kFrame - kDeep) leaves its lesser ones no room above fp32's smallest, 2^-126 (2^-43 of
// it is left); keys below 2^-kSmall of a row's largest add nothing to l that it could hold (2^31 of them 2^-33).
constexpr float kDeep = 90.0f, kSmall = 64.0f;
constexpr float kFrame = 7.0f;     // log2 of the largest weight right after that
// A step's codes take their rows' scales along into f16, relative to the largest of the step, if K's spread
// over at most kSpreadK binades and V's over at most kSpreadV, and none lies beyond 2^+-100 (as bytes: kLow to
// kHigh).  V rows of zeros, kept under scale 1 whatever the others' size, count as kZero, below every row that is not
// (2^-110 is the smallest scale that is written).
constexpr int kSpreadK = 14, kSpreadV = 10, kLow = 27, kHigh = 227, kZero = 1;

template <int D>
struct TreeCfg {
    static constexpr int PANELS = D / 64;            // 128-byte swizzle panels of a 16-bit row
    static constexpr int PANEL_BYTES = kHalf * 128;
    static constexpr int TILE = PANELS * PANEL_BYTES;  // a step's K or V in f16
    static constexpr int RAW = kHalf * D;            // its codes
    static constexpr int SLOT = 2 * (RAW + kHalf);   // K's codes, V's, K's exponents, V's
    static constexpr int SLOTS = 6;
    static constexpr int QPANEL = kTile * 128, QTILE = PANELS * QPANEL;
    static constexpr int SMEM = QTILE + 4 * TILE + SLOTS * SLOT + 1024;  // Q, two K, two V, raw ring
    static constexpr int THREADS = 32 * 20;
    static constexpr uint32_t TMEM_COLS = 512;
    // TMEM columns: S of four steps (P, f16 pairs, over its lower half), O of the two streams
    static constexpr uint32_t S0 = 0, O0 = 256;
};

// One unit's part of a share.
struct TreeUnit {
    int b, hk, row0;       // sequence, key/value head, first query row
    int q0, nq, nk, nblk;  // the sequence: first token, tokens, keys in the table, blocks
    int ts;                // position of the first drafted key
    int in_seq;            // units of the sequence
    int jb, J;             // this share's blocks of the unit: [jb, jb + J) ...
    int h0, nh;            // ... and its steps: [h0, h0 + nh)
    int rows;              // its query rows
    int first;             // the share's first unit
};

// Sizes of sequence b: units (row sets times heads) of nblk blocks each.
__device__ __forceinline__ void tree_sequence(const TreeDecodeParams& p, int b, TreeUnit& u)
{
    u.b = b;
    u.nq = packed_rows(p.cu_q, b, p.total_q, p.max_q, u.q0);
    const int len = min(max(p.seqlens[b], 0), p.max_k);
    u.nk = min(len, p.table_k);
    // (of a tree that starts before the sequence, the mask's bits of keys that are none count nothing)
    u.ts = max(p.tree_start != nullptr ? p.tree_start[b] : len - u.nq, -32 * p.words);
    u.nblk = max(1, (u.nk + kTB - 1) / kTB);
    u.in_seq = ((u.nq * p.G.d + kTile - 1) / kTile) * p.Hkv;
}

__device__ __forceinline__ Shares tree_share(const TreeDecodeParams& p, int c, TreeUnit& u, int& at)
{
    int b = 0;
    const Shares sh = find_share(
        p.B, p.ctas, c,
        [&](int x) {
            if (x >= p.B) return 0;
            TreeUnit v;
            tree_sequence(p, x, v);
            return v.in_seq * (v.nblk + kTreeUnitCost);
        },
        b, at);
    if (sh.start(c) < sh.total) tree_sequence(p, b, u);
    return sh;
}

// What the merge needs of a unit that is cut: first token, first query row, key/value head, and in one
// word the rows, whether the first part is its share's second, and the parts.
__device__ __forceinline__ int4 tree_cut(const TreeUnit& u, int lead, int parts)
{
    return make_int4(u.q0, u.row0, u.hk, u.rows | lead << 8 | parts << 9);
}

// Whether every row of the unit sees all keys of step h, and all of its 16-key groups are there.
__device__ __forceinline__ bool whole_step(const TreeUnit& u, int h, int groups)
{
    return groups == 0xf && (h + 1) * kHalf <= min(u.nk, u.ts);
}

// warp_wait_all with waits that suspend for longer at a time.
static __device__ __noinline__ bool tree_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                                   uint64_t limit_ns, int site)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_ns(bar, parity, 20000)) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            atomicCAS(status, 0, site);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, const Watchdog& wd, int site)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = tree_wait_slow(bar, parity, wd.abort_flag, wd.status, wd.limit_ns, site);
    return __all_sync(0xffffffffu, ok);
}

// The low n bits, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Which of the keys [base, base + 32) the token with mask row m (words w) sees, groups: two bits for the
// 16-key groups that are there.
__device__ __forceinline__ uint32_t seen_keys(const uint32_t* m, int words, int ts, int nk, int base, int groups)
{
    uint32_t v = low_bits(ts - base);
    const int off = base - ts;  // of the first key, in mask bits
    if (off > -32 && off < 32 * words) {
        if (off < 0) {
            v |= m[0] << -off;
        } else {
            const int i = off >> 5;
            v |= __funnelshift_r(m[i], i + 1 < words ? m[i + 1] : 0u, off & 31);
        }
    }
    v &= low_bits(nk - base);
    return v & ((groups & 1 ? 0xffffu : 0u) | (groups & 2 ? 0xffff0000u : 0u));
}

// What softmax has to know of a step: the groups that are there, whether its rows' scales are not in the
// tiles (far), and the exponent bytes of K and V that the tiles are relative to.
struct BlockInfo {
    uint32_t v;
    __device__ __forceinline__ BlockInfo(uint32_t x) : v(x) {}
    __device__ __forceinline__ BlockInfo(int groups, bool far, int k, int v)
        : v(static_cast<uint32_t>(groups | (far ? 0x100 : 0) | k << 16) | static_cast<uint32_t>(v) << 24)
    {
    }
    __device__ __forceinline__ int groups() const { return v & 0xff; }
    __device__ __forceinline__ bool far() const { return v & 0x100; }
    __device__ __forceinline__ int k() const { return v >> 16 & 0xff; }
    __device__ __forceinline__ int ev() const { return static_cast<int>(v >> 24); }
};

// The largest and the smallest of a word's bytes.
__device__ __forceinline__ uint32_t max_byte(uint32_t w)
{
    w = __vmaxu4(w, w >> 16);
    return max(w & 0xff, w >> 8 & 0xff);
}
__device__ __forceinline__ uint32_t min_byte(uint32_t w)
{
    w = __vminu4(w, w >> 16 | w << 16);
    return min(w & 0xff, w >> 8 & 0xff);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Which codes of a step a converting thread (of 64) takes: in pass j a row, of it one 16-code chunk (D = 64) or
// two.  The eight lanes of a load or store phase hold two rows' chunks of different panels, so that they lie in
// different banks both in the raw tile (rows of D bytes) and in the swizzled one.
constexpr int kPasses = kHalf / 16;
__device__ __forceinline__ int convert_row(int t, int j) { return 2 * (t >> 3) + (t >> 2 & 1) + 16 * j; }
template <int D>
__device__ __forceinline__ int convert_chunk(int t, int i)
{
    return (t & 3) + (D == 128 ? 4 * ((t >> 2 & 1) ^ i) : 0);
}

// A step's raw tile to f16: codes times their rows' powers of two relative to `top` (far: plain codes), exactly
// (e4m3 has 4 bits, and the smallest code, 2^-9, times 2^-14 is one of f16's), in rows of 64 elements, 128 bytes,
// swizzled.
template <int D>
__device__ __forceinline__ void convert_tile(const uint8_t* raw, const uint8_t* exps, uint8_t* to, int t, int top, bool far)
{
    using C = TreeCfg<D>;
    constexpr int N = D / 64;
    const int row0 = convert_row(t, 0), c0 = convert_chunk<D>(t, 0);  // (rows of all passes are equal mod 8)
    const uint8_t* from = raw + row0 * D + 16 * c0;
    const int from2 = D == 128 ? (c0 & 4 ? -64 : 64) : 0;
    const uint8_t* ex = exps + row0;
    uint8_t* at = to + row0 * 128 + (c0 >> 2) * C::PANEL_BYTES;
    const int at2 = c0 & 4 ? -C::PANEL_BYTES : C::PANEL_BYTES;
    const int lo = ((2 * (c0 & 3)) ^ (row0 & 7)) << 4, hi = lo ^ 16;
#pragma unroll 2
    for (int j = 0; j < kPasses; ++j, from += 16 * D, ex += 16, at += 16 * 128) {
        uint4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = *reinterpret_cast<const uint4*>(from + i * from2);
        // (rows that are none or zero, whose exponents may lie anywhere, keep finite factors)
        const uint32_t scale = static_cast<uint32_t>(far ? 15 : min(max(15 + *ex - top, 1), 15)) * 0x04000400u;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint4 h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                h[k] = make_uint4(mul_f16x2(e4m3x2_to_f16x2(w[2 * k]), scale), mul_f16x2(e4m3x2_to_f16x2(w[2 * k] >> 16), scale),
                                  mul_f16x2(e4m3x2_to_f16x2(w[2 * k + 1]), scale),
                                  mul_f16x2(e4m3x2_to_f16x2(w[2 * k + 1] >> 16), scale));
            *reinterpret_cast<uint4*>(at + i * at2 + lo) = h[0];
            *reinterpret_cast<uint4*>(at + i * at2 + hi) = h[1];
        }
    }
    fence_proxy_async_smem();
}

// V of a step that not every row sees whole, in its raw tile before the conversion: rows past the end hold
// whatever the page held and become zero; NaN codes, which must not reach rows that do not see them as 0 * NaN, are
// taken out and noted in nan (16 bits a chunk).  Returns whether this thread found any.
template <int D>
__device__ __noinline__ bool clear_unseen(uint8_t* raw, uint16_t* nan, int t, int groups, int keys)
{
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < kPasses * (D / 64); ++i) {
        const int row = convert_row(t, i / (D / 64)), c = convert_chunk<D>(t, i % (D / 64));
        uint4* at = reinterpret_cast<uint4*>(raw + row * D + 16 * c);
        uint4 x = *at;
        if (!(groups >> (row >> 4) & 1) || row >= keys) x = make_uint4(0u, 0u, 0u, 0u);
        uint32_t w[4] = {x.x, x.y, x.z, x.w}, bits = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t nb = nan_bytes(w[h]) >> 7;  // 1 in each byte that is NaN
            w[h] &= ~(nb * 0xffu);
            bits |= ((nb | nb >> 7 | nb >> 14 | nb >> 21) & 15u) << (4 * h);
        }
        nan[row * (D / 16) + c] = static_cast<uint16_t>(bits);
        any = any || bits;
        *at = make_uint4(w[0], w[1], w[2], w[3]);  // (read by this thread only)
    }
    return any;
}

// S = Q K^T over D / 16 k-steps (both operands K-major in swizzled panels).
template <int D>
__device__ __forceinline__ void tree_issue_qk(uint32_t d_tmem, uint64_t qdesc, uint64_t kdesc, uint32_t idesc)
{
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
        mma_ss(d_tmem, sdesc_adv(qdesc, (ks / 4) * TreeCfg<D>::QPANEL + (ks % 4) * 32),
               sdesc_adv(kdesc, (ks / 4) * TreeCfg<D>::PANEL_BYTES + (ks % 4) * 32), idesc, ks > 0 ? 1u : 0u);
}

// O += P V: P (f16 pairs) from TMEM, V (MN-major) from shared memory; k-steps of 16 keys.
__device__ __forceinline__ void tree_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t vdesc, uint32_t idesc,
                                              uint32_t acc_first, int steps)
{
    if (steps >= 4) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            mma_ts(d_tmem, p_tmem + 8u * ks, sdesc_adv(vdesc, ks * 2048), idesc, ks > 0 ? 1u : acc_first);
    } else {
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks)
            mma_ts(d_tmem, p_tmem + 8u * ks, sdesc_adv(vdesc, ks * 2048), idesc, ks > 0 ? 1u : acc_first);
    }
}

// A unit's Q, by eight warps: f16 in rows of 64 elements, 128 bytes, swizzled, each row scaled by a
// power of two (its inverse's exponent to qexp); zeros up to a multiple of 32 rows.  The rows come to their places as
// they are, all at once, and every thread converts what it has brought.
//
// (This and what else is done once a unit, or seldom, is out of line and in rolled loops: what the warps do at every
// step has to fit the instruction cache, some 32 KB for all kinds of warps together, and code that is not there costs
// some 50 clocks for every eight instructions.  With these loops unrolled, the same loads took 4 to 10 thousand clocks.)
template <int D>
__device__ __noinline__ void stage_q(const TreeDecodeParams& p, const TreeUnit& un, int cw, uint8_t* to, int8_t* qexp)
{
    constexpr int LPR = D / 8;         // lanes of a row
    constexpr int RW = 8 * 32 / LPR;   // rows of a pass
    const int lane = threadIdx.x & 31, c = lane % LPR, hq = un.hk * p.G.d;
    const int rows = un.rows, rows32 = (rows + 31) & ~31, row0 = un.row0, q0 = un.q0;
    const int r0 = (32 * cw + lane) / LPR;
    // (RW is a multiple of 8, so a thread's rows are swizzled alike)
    uint8_t* const at = to + (c >> 3) * TreeCfg<D>::QPANEL + r0 * 128 + (((c & 7) ^ (r0 & 7)) << 4);
#pragma unroll 1
    for (int r = r0; r < rows32; r += RW) {
        uint4* x = reinterpret_cast<uint4*>(at + (r - r0) * 128);
        bool in = r < rows;
        if (in) {
            const int i = p.G(row0 + r), h = row0 + r - i * p.G.d;
            const long long off = (static_cast<long long>(q0 + i) * p.H + hq + h) * D + 8 * c;
            in = in_extent(off, 8, p.q_ext, p.status);
            if (in) cp_async16(x, p.q + off);
        }
        if (!in) *x = make_uint4(0u, 0u, 0u, 0u);
    }
    cp_async_wait_all();
#pragma unroll 1
    for (int r = r0; r < rows32; r += RW) {
        uint4* const x = reinterpret_cast<uint4*>(at + (r - r0) * 128);
        const uint4 w = *x;
        const uint32_t u[4] = {w.x ^ p.q_sign, w.y ^ p.q_sign, w.z ^ p.q_sign, w.w ^ p.q_sign};
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = __vmaxu2(amax, u[i] & 0x7fff7fffu);
        amax = max(amax & 0xffffu, amax >> 16);
        // (a row's lanes are all here: RW and rows32 are multiples of a warp's rows)
#pragma unroll
        for (int m = 1; m < LPR; m *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        // 2^a brings the row's largest magnitude to [2^14, 2^15).  (In a row with an infinity or a NaN the rest vanishes
        // beside it, as it does in its logits.)
        const int a = min(14 + 127 - static_cast<int>(amax >> 7), 126);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + a) << 23);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = pack_f16x2(__uint_as_float(u[i] << 16) * up, __uint_as_float(u[i] & 0xFFFF0000u) * up);
        *x = make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0) qexp[r] = static_cast<int8_t>(-a);
    }
    fence_proxy_async_smem();
}

// A step that is taken key by key (scales that are not in the tiles, keys that only some rows see), as one row sees it.
struct StepKeys {
    const uint32_t* mask;   // the row's mask words
    int words, ts, nk;      // as in TreeUnit
    int base, groups;       // the step's first key, its 16-key groups that are there
    bool whole, in;         // all keys are seen; the mask row lies within its tensor
    // up to the last 32 keys that any row sees
    __device__ __forceinline__ int chunks() const { return min(kHalf / 32, (nk - base + 31) / 32); }
    __device__ __forceinline__ uint32_t seen(int c) const
    {
        if (whole) return 0xffffffffu;
        return in ? seen_keys(mask, words, ts, nk, base + 32 * c, groups >> (2 * c)) : 0u;
    }
};

// The largest x and the largest x + E of a row.
__device__ __noinline__ float2 step_max(uint32_t ts, StepKeys k, const float* ks, const float* ev, float down)
{
    float mx = -INFINITY, mt = -INFINITY;
    uint32_t vis = 0;
#pragma unroll 1
    for (int c = 0; c < 2 * k.chunks(); ++c, ts += 16, ks += 16, ev += 16) {
        uint32_t v[16];
        tmem_ld16(ts, v);
        vis = c & 1 ? vis >> 16 : k.seen(c >> 1);
        tmem_wait_ld();
        reg_fence16(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(v[i]) * (ks[i] * down);
            if (!(vis >> i & 1)) continue;
            mx = fmaxf(mx, x);
            mt = fmaxf(mt, x + ev[i]);
        }
    }
    return make_float2(mx, mt);
}

// The weights of a row, over its scores (P of 16 keys goes where S of keys up to those was); nm: -M, nl: -m.
// Returns the sum of 2^(x - m).
__device__ __noinline__ float step_weights(uint32_t ts, StepKeys k, const float* ks, const float* ev, float down, float nm,
                                           float nl)
{
    float l = 0.0f;
    uint32_t vis = 0, tp = ts;
#pragma unroll 1
    for (int c = 0; c < 2 * k.chunks(); ++c, ts += 16, tp += 8, ks += 16, ev += 16) {
        uint32_t v[16];
        tmem_ld16(ts, v);
        vis = c & 1 ? vis >> 16 : k.seen(c >> 1);
        tmem_wait_ld();
        reg_fence16(v);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool see = vis >> (i + e) & 1;
                const float x = __uint_as_float(v[i + e]) * (ks[i + e] * down);
                l += see ? ex2(x + nl) : 0.0f;
                w[e] = see ? ex2(x + (nm + (ev[i + e] + kFrame))) : 0.0f;
            }
            v[i / 2] = pack_f16x2(w[0], w[1]);
        }
        tmem_st8(tp, v);
    }
    return l;
}

// The sum of 2^(x - m) of a row that sees all keys of a step whose scales are in the tiles (x = S cf); nl: -m.
__device__ __noinline__ float step_sum(uint32_t ts, float cf, float nl)
{
    float l = 0.0f;
#pragma unroll 1
    for (int c = 0; c < kHalf; c += 16) {
        uint32_t v[16];
        tmem_ld16(ts + c, v);
        tmem_wait_ld();
        reg_fence16(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) l += ex2(fmaf(__uint_as_float(v[i]), cf, nl));
    }
    return l;
}

// The columns (row_nan) in which a key that the row sees has NaN.
template <int D>
__device__ __noinline__ void note_nan(StepKeys k, bool valid, const uint16_t* nan, uint32_t* row_nan, bool first)
{
    if (first)
        for (int h = 0; h < D / 32; ++h) row_nan[h] = 0u;
#pragma unroll 1
    for (int c = 0; c < k.chunks(); ++c) {
        uint32_t vis = valid ? k.seen(c) : 0u;
        while (vis) {
            const uint16_t* at = nan + (32 * c + __ffs(vis) - 1) * (D / 16);
            vis &= vis - 1;
            for (int h = 0; h < D / 32; ++h) row_nan[h] |= at[2 * h] | static_cast<uint32_t>(at[2 * h + 1]) << 16;
        }
    }
    __syncwarp();
}

// What a unit's row came to.
struct RowResult {
    float f0, f1;           // factors of the two accumulators (below 0: what it holds is not used) ...
    float inv, half;        // ... and of both: inv, and half twice
    const uint32_t *nan0, *nan1;  // columns that are NaN, or null
};

// Writes half of O of a row, columns from c0 on (TMEM columns from to on, the second accumulator D columns on), as bf16
// to o or fp32 to part (the other null; in: the row exists).
template <int D>
__device__ __noinline__ void write_row(uint32_t to, int c0, RowResult r, __nv_bfloat16* o, float* part, bool in)
{
    const float both = r.inv * r.half;
#pragma unroll 1
    for (int c = c0; c < c0 + D / 2; c += 16) {
        uint32_t x[16], y[16];
        tmem_ld16(to + c, x);
        tmem_ld16(to + D + c, y);
        tmem_wait_ld();
        reg_fence16(x);
        reg_fence16(y);
        const uint32_t nan = ((r.nan0 ? r.nan0[c / 32] : 0u) | (r.nan1 ? r.nan1[c / 32] : 0u)) >> (c & 16);
        // (a factor of 0, of a stream whose values are small beside the other's, still hands on a NaN)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = r.f0 < 0.0f ? 0.0f : __uint_as_float(x[i]) * r.f0;
            if (!(r.f1 < 0.0f)) v = fmaf(__uint_as_float(y[i]), r.f1, v);
            x[i] = __float_as_uint(nan >> i & 1 ? NAN : v * both * r.half);
        }
        if (!in) continue;
        if (o != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = pack_bf16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            st_row<1>(o + c, x);
        } else {
            st_row<2>(part + c, x);
        }
    }
}

// Which V rows of a lane's four (words vw of exponents, of which `in` are there) are rows of zeros under scale 1 (-0 is
// zero as well).
template <int D>
__device__ __noinline__ uint32_t zero_rows(const uint8_t* raw, uint32_t vw, int l4)
{
    uint32_t zero = 0;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const uint4* w = reinterpret_cast<const uint4*>(raw + (4 * l4 + j) * D);
        uint32_t some = 0;
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i) some |= w[i].x | w[i].y | w[i].z | w[i].w;
        if ((vw >> (8 * j) & 0xff) == 127 && (some & 0x7f7f7f7fu) == 0) zero |= 0xffu << (8 * j);
    }
    return zero;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS, 1) fa_decode_tree_kernel(const TreeDecodeParams p)
{
    using C = TreeCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sK = sQ + C::QTILE;
    uint8_t* sV = sK + 2 * C::TILE;
    uint8_t* sRaw = sV + 2 * C::TILE;

    __shared__ __align__(8) uint64_t bar_raw[C::SLOTS];    // a step's raw tiles landed ...
    __shared__ __align__(8) uint64_t bar_taken[C::SLOTS];  // ... and were converted
    __shared__ __align__(8) uint64_t bar_unit[kTreeUnits];
    __shared__ __align__(8) uint64_t bar_qfull, bar_qempty;
    __shared__ __align__(8) uint64_t bar_full[2][2], bar_kempty[2];  // [K, V][tile]: converted, and read (V: bar_pv)
    __shared__ __align__(8) uint64_t bar_info[kRing];  // what is known of a step is there
    __shared__ __align__(8) uint64_t bar_s[4];         // S of a step
    __shared__ __align__(8) uint64_t bar_p[4];         // P of a step (and O rescaled)
    __shared__ __align__(8) uint64_t bar_pv[4];        // the product of a step's P has run
    __shared__ __align__(8) uint64_t bar_o[4];         // all products of a unit have run
    __shared__ __align__(8) uint64_t bar_post[2], bar_joined;  // a stream's sums given; both, and O, read
    __shared__ __align__(8) uint64_t bar_drain[2];
    __shared__ TreeUnit s_unit[kTreeUnits];
    __shared__ int s_valid[C::SLOTS];   // bit i: keys [16 i, 16 i + 16) of the step are there
    // by step: what BlockInfo packs; and, of steps that go key by key, |scale| log2(e) times the K row's scale
    // and the V row's exponent (as far as they are not in the tiles)
    __shared__ uint32_t s_info[kRing];
    __shared__ __align__(16) float s_ks[kRing][kHalf];
    __shared__ __align__(16) float s_ev[kRing][kHalf];
    __shared__ int8_t s_qexp[8][kTile];       // by unit: the power of two that undoes a Q row's scaling
    __shared__ uint16_t s_nan[2][kHalf][D / 16];  // NaN codes that were taken out of V's tile
    __shared__ uint32_t s_any_nan[2][2];          // by converting warp
    __shared__ uint32_t s_row_nan[2][kTile][D / 32];  // by stream: the row's columns that are NaN
    __shared__ float4 s_post[2][kTile];           // by stream: M, m and l
    __shared__ uint8_t s_post_odd[2][kTile];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    constexpr int kConvWarp = 8, kCopyWarp = 16, kQkWarp = 17, kPvWarp = 18, kScoutWarp = 19;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {  // (a lane a barrier: one thread for all of them took a microsecond)
        static_assert(C::SLOTS <= 32 && kTreeUnits == 32 && kRing <= 32, "");
        mbar_init(&bar_unit[lane], 1);
        if (lane < kRing) mbar_init(&bar_info[lane], 1);
        if (lane < C::SLOTS) {
            mbar_init(&bar_raw[lane], 1);
            mbar_init(&bar_taken[lane], 4);
        }
        if (lane < 4) {
            mbar_init(&bar_s[lane], 1);
            mbar_init(&bar_p[lane], 4);
            mbar_init(&bar_pv[lane], 1);
            mbar_init(&bar_o[lane], 1);
            mbar_init(&bar_full[lane >> 1][lane & 1], 2);
        }
        if (lane < 2) {
            mbar_init(&bar_kempty[lane], 1);
            mbar_init(&bar_post[lane], 4);
            mbar_init(&bar_drain[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&bar_qfull, 8);
            mbar_init(&bar_qempty, 1);
            mbar_init(&bar_joined, 8);
            abort_flag = 0;
        }
        mbar_fence_init();
    }
    if (warp == kQkWarp) {
        tmem_alloc(&tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_slot;
    const Watchdog wd{&abort_flag, p.status, p.wait_limit_ns};
    dependent_begin();
    const int cta = static_cast<int>(blockIdx.x);

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------- copies
        TreeUnit un;
        int at = 0;
        const Shares sh = tree_share(p, cta, un, at);
        int left = sh.start(cta + 1) - sh.start(cta);
        const int ps = 1 << p.page_shift;
        const int np = ps >= kHalf ? 1 : kHalf / ps;  // pages of a step
        const int rows_pp = ps >= kHalf ? kHalf : ps;  // rows of a copy
        // What a lane copies of a step: the codes of K or V, or the exponents, of one of its pages.
        const int kind = lane & 3, page_in = lane >> 2, stride = kind < 2 ? D : 1;
        const uint8_t* const from = kind == 0 ? p.kc : kind == 1 ? p.vc : kind == 2 ? p.ke : p.ve;
        uint8_t* const into = sRaw + (kind < 2 ? kind * C::RAW : 2 * C::RAW + (kind - 2) * kHalf) + page_in * rows_pp * stride;
        const int groups_pp = rows_pp / 16;
        int ui = 0, place = 0;                     // unit of the sequence, place in it
        if (left > 0) {
            ui = static_cast<unsigned>(at) / static_cast<unsigned>(un.nblk + kTreeUnitCost);
            place = at - ui * (un.nblk + kTreeUnitCost);
        }
        bool ok = true, cut = false;
        int n = 0, k = 0;  // steps and units so far
        while (ok && left > 0) {
            const int set = p.heads(ui);
            un.row0 = set * kTile;
            un.hk = ui - set * p.Hkv;
            un.rows = min(un.nq * p.G.d - un.row0, kTile);
            const int end = min(un.nblk + kTreeUnitCost, place + left);
            left -= end - place;
            un.jb = max(0, place - kTreeUnitCost);
            un.J = max(0, end - kTreeUnitCost) - un.jb;
            un.first = k == 0;
            un.h0 = 2 * un.jb;
            un.nh = min(2 * (un.jb + un.J), max(1, (un.nk + kHalf - 1) / kHalf)) - un.h0;
            if (left == 0 && un.jb == 0 && un.J > 0 && un.J < un.nblk) {
                const int last = sh.share_of(sh.start(cta + 1) - un.J + un.nblk - 1);
                if (lane == 0) p.cuts[cta] = tree_cut(un, k == 0 ? 0 : 1, last - cta + 1);
                cut = true;
            }
            int base = (un.h0 * kHalf) >> p.page_shift, ids = -1;
            auto load_ids = [&]() {
                const int idx = base + lane;
                ids = -1;
                if (idx < p.max_pages && (static_cast<long long>(idx) << p.page_shift) < un.nk)
                    ids = p.table[static_cast<long long>(un.b) * p.max_pages + idx];
            };
            if (un.J > 0) {
                load_ids();
                if (lane == 0) {
                    s_unit[k % kTreeUnits] = un;
                    mbar_arrive(&bar_unit[k % kTreeUnits]);
                }
                __syncwarp();
                ++k;
            }
#pragma unroll 1
            for (int hh = 0; un.J > 0 && hh < un.nh; ++hh) {
                const int pos = (un.h0 + hh) * kHalf;
                const int first = pos >> p.page_shift;
                if (first + np > base + 32) {
                    base = first;
                    load_ids();
                }
                const int id = __shfl_sync(0xffffffffu, ids, (first - base + page_in) & 31);
                const bool mine = page_in < np && id >= 0 && id < p.num_pages;
                const uint32_t got = __ballot_sync(0xffffffffu, mine);  // four lanes a page
                const int slot = n % C::SLOTS;
                ok = tree_wait(&bar_taken[slot], ((n / C::SLOTS) & 1) ^ 1, wd, kSiteTreeEmpty);
                if (!ok) break;
                if (lane == 0) {
                    int bits = 0;
#pragma unroll 1
                    for (int i = 0; i < np; ++i)
                        if (got >> (4 * i) & 1) bits |= ((1 << groups_pp) - 1) << (i * groups_pp);
                    s_valid[slot] = bits;
                    mbar_arrive_expect_tx(&bar_raw[slot], static_cast<uint32_t>((__popc(got) >> 2) * rows_pp * 2 * (D + 1)));
                }
                __syncwarp();
                if (mine && !(n == 0 && (p.debug_flags & kDebugDropFirstLoad))) {
                    const long long row = ((static_cast<long long>(id) * p.Hkv + un.hk) << p.page_shift) + (pos & (ps - 1));
                    bulk_load(into + slot * C::SLOT, from + row * stride, static_cast<uint32_t>(rows_pp * stride), &bar_raw[slot]);
                }
                ++n;
            }
            place = 0;
            if (left > 0 && ++ui == un.in_seq) {
                ui = 0;
                do tree_sequence(p, un.b + 1, un);
                while (un.in_seq == 0 && un.b + 1 < p.B);
            }
        }
        if (!cut && lane == 0 && p.cuts != nullptr) p.cuts[cta] = make_int4(0, 0, 0, 0);
        if (ok && lane == 0) {  // the end of the units
            s_unit[k % kTreeUnits].J = 0;
            mbar_arrive(&bar_unit[k % kTreeUnits]);
        }
        __syncwarp();
        // no copy may land after the CTA exits (bounded waits that ignore the abort flag)
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        for (int i = max(0, n - C::SLOTS); i < n; ++i)
            mbar_wait(&bar_raw[i % C::SLOTS], (i / C::SLOTS) & 1, wd_drain, kSiteTreeDrain);
    } else if (warp == kQkWarp) {
        // ------------------------------------------------------------- S = Q K^T
        // S of step n takes the buffer of step n - 4 when the product of that step's P has run.  (The two products have a warp
        // each: one that issued both was the slowest part of the pipeline.)
        constexpr uint32_t kIdS = idesc_f16_f32(128, kHalf, 0, 0);
        const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024);
        bool ok = true;
        int n = 0, k = 0;
#pragma unroll 1
        for (; ok; ++k) {
            ok = tree_wait(&bar_unit[k % kTreeUnits], (k / kTreeUnits) & 1, wd, kSiteTreeUnit);
            const TreeUnit& un = s_unit[k % kTreeUnits];
            if (!ok || un.J == 0) break;
            const int nh = un.nh;
            ok = tree_wait(&bar_qfull, k & 1, wd, kSiteTreeQ);
#pragma unroll 1
            for (int h = 0; ok && h < nh; ++h, ++n) {
                ok = tree_wait(&bar_full[0][n & 1], (n >> 1) & 1, wd, kSiteTreeK) &&
                     tree_wait(&bar_pv[n & 3], ((n >> 2) & 1) ^ 1, wd, kSiteTreeP);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    tree_issue_qk<D>(tbase + C::S0 + kHalf * (n & 3), dq0, sdesc_adv(dk0, (n & 1) * C::TILE), kIdS);
                    mma_commit(&bar_s[n & 3]);
                    mma_commit(&bar_kempty[n & 1]);
                    if (h + 1 == nh) mma_commit(&bar_qempty);
                }
                __syncwarp();
            }
        }
        // every commit has to arrive before the CTA exits
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        if (elect_one()) mma_commit(&bar_drain[0]);
        mbar_wait(&bar_drain[0], 0, wd_drain, kSiteTreeDrain);
#pragma unroll 1
        for (int i = max(0, n - 2); i < n; ++i) mbar_wait(&bar_kempty[i & 1], (i >> 1) & 1, wd_drain, kSiteTreeDrain);
        if (ok && k > 0) mbar_wait(&bar_qempty, (k - 1) & 1, wd_drain, kSiteTreeDrain);
    } else if (warp == kPvWarp) {
        // ------------------------------------------------------------- O += P V
        constexpr uint32_t kIdPV = idesc_f16_f32(128, D, 0, 1);
        const uint64_t dv0 = sdesc_sw128(smem_u32(sV), C::PANEL_BYTES, 1024);
        bool ok = true;
        int n = 0;
#pragma unroll 1
        for (int k = 0; ok; ++k) {
            ok = tree_wait(&bar_unit[k % kTreeUnits], (k / kTreeUnits) & 1, wd, kSiteTreeUnit);
            const TreeUnit& un = s_unit[k % kTreeUnits];
            if (!ok || un.J == 0) break;
            const int nh = un.nh;
            int left = un.nk - un.h0 * kHalf;
#pragma unroll 1
            for (int h = 0; ok && h < nh; ++h, ++n, left -= kHalf) {
                ok = tree_wait(&bar_full[1][n & 1], (n >> 1) & 1, wd, kSiteTreeV) &&
                     tree_wait(&bar_p[n & 3], (n >> 2) & 1, wd, kSiteTreeP);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    // (a stream's first product of a unit starts O; 16-key steps behind the unit's last key are left out)
                    tree_issue_pv(tbase + C::O0 + static_cast<uint32_t>(D * (n & 1)), tbase + C::S0 + kHalf * (n & 3),
                                  sdesc_adv(dv0, (n & 1) * C::TILE), kIdPV, h >= 2 ? 1u : 0u, (left + 15) >> 4);
                    mma_commit(&bar_pv[n & 3]);
                    if (h + 1 == nh) mma_commit(&bar_o[k & 3]);
                }
                __syncwarp();
            }
        }
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        if (elect_one()) mma_commit(&bar_drain[1]);
        mbar_wait(&bar_drain[1], 0, wd_drain, kSiteTreeDrain);
#pragma unroll 1
        for (int i = max(0, n - 4); i < n; ++i) mbar_wait(&bar_pv[i & 3], (i >> 2) & 1, wd_drain, kSiteTreeDrain);
    } else if (warp >= kConvWarp && warp < kCopyWarp) {
        // ------------------------------------------------------------- conversion: Q, K, V
        // Pairs of warps: K and V of even steps (warps 8-11), K and V of odd ones; all eight Q, after their first step of
        // a unit (the first unit's comes from the softmax's warps, which have nothing to do yet).
        const int cw = warp & 3, z = cw >> 1, par = warp - kConvWarp >= 4 ? 1 : 0, ct = static_cast<int>(threadIdx.x) & 63;
        bool ok = true;
        int n = 0;  // steps before this unit
#pragma unroll 1
        for (int k = 0; ok; ++k) {
            ok = tree_wait(&bar_unit[k % kTreeUnits], (k / kTreeUnits) & 1, wd, kSiteTreeUnit);
            const TreeUnit& un = s_unit[k % kTreeUnits];
            if (!ok || un.J == 0) break;
            const int h0 = un.h0, nh = un.nh;
            int hh = (n ^ par) & 1;  // the first of this pair's steps
            bool q = k > 0;          // Q is to come: after that step, once the unit before has run its last scores
#pragma unroll 1
            for (; ok && (q || hh < nh); hh += 2) {
                if (hh < nh) {
                    const int m = n + hh, slot = m % C::SLOTS;
                    uint8_t* raw = sRaw + slot * C::SLOT + z * C::RAW;
                    // (the scout has seen the step's tiles land)
                    ok = tree_wait(&bar_info[m % kRing], (m / kRing) & 1, wd, kSiteTreeRaw) &&
                         (z == 0 ? tree_wait(&bar_kempty[par], ((m >> 1) & 1) ^ 1, wd, kSiteTreeK)
                                 : m < 2 || tree_wait(&bar_pv[(m - 2) & 3], ((m - 2) >> 2) & 1, wd, kSiteTreeV));
                    if (!ok) break;
                    const BlockInfo info(s_info[m % kRing]);
                    if (z == 1 && !whole_step(un, h0 + hh, info.groups())) {
                        const bool any = clear_unseen<D>(raw, &s_nan[par][0][0], ct, info.groups(), un.nk - (h0 + hh) * kHalf);
                        const bool all = __any_sync(0xffffffffu, any);
                        if (lane == 0) s_any_nan[par][cw & 1] = all;
                    }
                    convert_tile<D>(raw, sRaw + slot * C::SLOT + 2 * C::RAW + z * kHalf, sK + (2 * z + par) * C::TILE, ct,
                                    z ? info.ev() : info.k(), info.far());
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar_full[z][par]);
                        mbar_arrive(&bar_taken[slot]);
                    }
                }
                if (q) {
                    q = false;
                    ok = tree_wait(&bar_qempty, (k - 1) & 1, wd, kSiteTreeQ);
                    if (!ok) break;
                    stage_q<D>(p, un, warp - kConvWarp, sQ, s_qexp[k & 7]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_qfull);
                }
            }
            n += nh;
        }
    } else if (warp == kScoutWarp) {
        // ------------------------------------------------------------- scout
        // Looks at the exponents of each step, a lane at four of K and of V, as soon as they have landed, ahead of the
        // conversion.  (What is known of step n is overwritten for step n + kRing, when that has landed, in the slot of step
        // n + kRing - SLOTS, which has been converted, after S of the step two before that, which was issued after P V of
        // the step four before it: more than n.)
        bool ok = true;
        int n = 0;
#pragma unroll 1
        for (int k = 0; ok; ++k) {
            ok = tree_wait(&bar_unit[k % kTreeUnits], (k / kTreeUnits) & 1, wd, kSiteTreeUnit);
            if (!ok) break;
            const TreeUnit& un = s_unit[k % kTreeUnits];
            if (un.J == 0) break;
            const int h0 = un.h0, nh = un.nh;
#pragma unroll 1
            for (int hh = 0; hh < nh; ++hh, ++n) {
                const int nr = n % kRing, slot = n % C::SLOTS;
                const uint8_t* ke = sRaw + slot * C::SLOT + 2 * C::RAW;
                const uint8_t* ve = ke + kHalf;
                ok = tree_wait(&bar_raw[slot], (n / C::SLOTS) & 1, wd, kSiteTreeRaw);
                if (!ok) break;
                const int valid = s_valid[slot], l4 = lane & 15;
                const bool whole = whole_step(un, h0 + hh, valid);
                const uint32_t kw = reinterpret_cast<const uint32_t*>(ke)[l4], vw = reinterpret_cast<const uint32_t*>(ve)[l4];
                uint32_t in = 0xffffffffu;
                if (!whole) in = valid >> (l4 >> 2) & 1 ? low_bits(8 * min(max(un.nk - (h0 + hh) * kHalf - 4 * l4, 0), 4)) : 0u;
                uint32_t vin = in;
                if (__any_sync(0xffffffffu, __vcmpeq4(vw, 0x7f7f7f7fu) & in))  // perhaps rows of zeros
                    vin &= ~zero_rows<D>(sRaw + slot * C::SLOT + C::RAW, vw, l4);  // (lanes 16-31 as 0-15)
                int ktop = static_cast<int>(__reduce_max_sync(0xffffffffu, max_byte(kw & in)));
                int vtop = static_cast<int>(__reduce_max_sync(0xffffffffu, max_byte(vw & vin)));
                const int klow = static_cast<int>(__reduce_min_sync(0xffffffffu, min_byte(kw | ~in)));
                const int vlow = static_cast<int>(__reduce_min_sync(0xffffffffu, min_byte(vw | ~vin)));
                const bool kany = __any_sync(0xffffffffu, in != 0), vany = __any_sync(0xffffffffu, vin != 0);
                // (some rows of zeros: with the others' exponent their weights could outgrow the others'.  Looking for them and
                // going key by key costs: with one row of 1000 zeros the 110 us become 180, with one of 50 365; taken with
                // the others they were 127 and 298.  Key by key only where a zero row's key would move M saves a tenth of
                // that, but costs the steps without any: 116 us.)
                const bool some_zero = __any_sync(0xffffffffu, vin != in);
                const bool far = (kany && (ktop > kHigh || klow < kLow || ktop - klow > kSpreadK)) ||
                                 (vany && (vtop > kHigh || vlow < kLow || vtop - vlow > kSpreadV || some_zero));
                if (!kany) ktop = 127;
                if (!vany) vtop = kZero;
                if (far || !whole) {
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t kb = kw >> (8 * j) & 0xff, vb = vw >> (8 * j) & 0xff;
                        const bool zero = !(vin >> (8 * j) & 1);
                        s_ks[nr][4 * l4 + j] = p.scale_log2 * exp_byte_scale(far ? kb : static_cast<uint32_t>(ktop));
                        s_ev[nr][4 * l4 + j] = !far ? static_cast<float>(vtop - 127)
                                                    : zero ? static_cast<float>(kZero - 127) : exp_byte_log2(vb);
                    }
                }
                if (lane == 0) s_info[nr] = BlockInfo(valid, far, ktop, vtop).v;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_info[nr]);
            }
        }
    } else if (warp < kConvWarp) {
        // ------------------------------------------------------------- softmax
        const int s = warp >> 2;                    // stream
        const int r = threadIdx.x & 127;            // row of the tile = TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tO0 = tbase + lane_base + C::O0, tO = tO0 + static_cast<uint32_t>(D * s);
        int n0 = 0;                                 // steps so far
        // (the first unit's Q)
        bool ok = tree_wait(&bar_unit[0], 0, wd, kSiteTreeUnit);
        if (ok && s_unit[0].J > 0) {
            stage_q<D>(p, s_unit[0], warp, sQ, s_qexp[0]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_qfull);
        }
        bool posted = false;                        // posted: O and the sums of the unit before may not have been read yet
#pragma unroll 1
        for (int k = 0; ok; ++k) {
            ok = tree_wait(&bar_unit[k % kTreeUnits], (k / kTreeUnits) & 1, wd, kSiteTreeUnit);
            const TreeUnit& un = s_unit[k % kTreeUnits];
            if (!ok || un.J == 0) break;
            const int nh = un.nh;
            const int first = (s - n0) & 1;         // this stream's first step of the unit
            const int clear = max(min(un.nk, un.ts), 0) / kHalf - un.h0;  // steps up to here are seen whole by every row
            const bool valid = r < un.rows;
            const bool any_valid = __any_sync(0xffffffffu, valid);
            // (rows that are none need no rescaling: their scores are 0)
            float M = valid ? -INFINITY : 1000.0f, m = M, l = 0.0f, down = 0.0f;
            bool odd = false;
#pragma unroll 1
            for (int hh = first; hh < nh; hh += 2) {
                const int n = n0 + hh, step = un.h0 + hh, n4 = n % kRing;
                const uint32_t tS = tbase + lane_base + C::S0 + static_cast<uint32_t>(kHalf * (n & 3));
                ok = tree_wait(&bar_s[n & 3], (n >> 2) & 1, wd, kSiteTreeS) &&
                     tree_wait(&bar_info[n4], (n / kRing) & 1, wd, kSiteTreeS);
                if (!ok) break;
                tc_fence_after();
                float alpha = 1.0f;
                bool need = false;
                if (any_valid) {
                    if (hh == first) down = __uint_as_float(static_cast<uint32_t>(127 + s_qexp[k & 7][r]) << 23);
                    const BlockInfo info(s_info[n4]);
                    const int groups = info.groups();
                    const bool whole = hh < clear && groups == 0xf;
                    // (both are -infinity until there is a logit that is not)
                    auto move_max = [&](float xm, float mt) {
                        if (xm > m + kGrow) {
                            l *= ex2(m - xm);
                            m = xm;
                        }
                        need = mt > M + kGrow;
                        if (need) {
                            alpha = ex2(M - mt);
                            M = mt;
                        }
                        return M == -INFINITY ? 0.0f : -M;
                    };
                    if (whole && !info.far()) {
                        const float cf = p.scale_log2 * exp_byte_scale(info.k()) * down;  // x = S cf
                        const float ev = static_cast<float>(info.ev() - 127);
                        float mx[2];
                        {
                            uint32_t v[32];
#pragma unroll
                            for (int c2 = 0; c2 < 2; ++c2) {
                                mx[c2] = tmem_ld32_max(tS + 32u * c2, v);
                                tmem_wait_ld();
                                reg_fence32(v);  // (the load's until here)
                                asm volatile("" : "+f"(mx[c2]));
                            }
                        }
                        const float xm = fmaxf(mx[0], mx[1]) * cf;
                        const float nm = move_max(xm, xm + ev) + (ev + kFrame);
                        const float nl = m == -INFINITY ? 0.0f : -m;
                        float sum = -1.0f;
                        if (__any_sync(0xffffffffu, valid && xm + nm < kFrame - kDeep && xm + nl > -kSmall))
                            sum = step_sum(tS, cf, nl);
                        // (the loads find the maximum: 64 tokens 220 us in replays, with the registers' own 225.)
                        // S is read again, 32 columns at a time in a rolled loop: with eight kinds of warps the instruction
                        // cache, not their arithmetic, was what they waited for
                        const uint64_t cf2 = f2_make(cf, cf), nm2 = f2_make(nm, nm);
                        uint64_t la = f2_make(0.f, 0.f), lb = la;
#pragma unroll 1
                        for (int c2 = 0; c2 < 2; ++c2) {
                            uint32_t v[32];
                            tmem_ld32(tS + 32u * c2, v);
                            tmem_wait_ld();
                            reg_fence32(v);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                float w0, w1, w2, w3;
                                f2_split(f2_fma(f2_make(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), cf2, nm2), w0, w1);
                                f2_split(f2_fma(f2_make(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), cf2, nm2), w2, w3);
                                w0 = ex2(w0);
                                w1 = ex2(w1);
                                w2 = ex2(w2);
                                w3 = ex2(w3);
                                la = f2_add(la, f2_make(w0, w1));
                                lb = f2_add(lb, f2_make(w2, w3));
                                v[c / 2] = pack_f16x2(w0, w1);
                                v[c / 2 + 1] = pack_f16x2(w2, w3);
                            }
                            tmem_st16(tS + 16u * c2, v);
                        }
                        float a0, a1;
                        f2_split(f2_add(la, lb), a0, a1);
                        // (2^91 suffices where w is large enough: 2^(8 + 90 - 7); rows of lesser keys may ask for more)
                        if (sum < 0.0f) sum = (a0 + a1) * ex2(fminf(nl - nm, 100.0f));
                        l += sum;
                    } else {
                        // key by key
                        const int tok = valid ? un.q0 + p.G(un.row0 + r) : un.q0;
                        const StepKeys keys{p.mask + static_cast<long long>(tok) * p.words, p.words, un.ts, un.nk, step * kHalf, groups,
                                            whole, in_extent(static_cast<long long>(tok) * p.words, p.words, p.mask_ext, p.status)};
                        const float2 top = step_max(tS, keys, s_ks[n4], s_ev[n4], down);
                        const float nm = move_max(top.x, top.y);
                        l += step_weights(tS, keys, s_ks[n4], s_ev[n4], down, nm, m == -INFINITY ? 0.0f : -m);
                        if (!whole) {
                            // NaN codes that were taken out of V: the columns of rows that see them
                            ok = tree_wait(&bar_full[1][n & 1], (n >> 1) & 1, wd, kSiteTreeV);
                            if (!ok) break;
                            if (s_any_nan[n & 1][0] | s_any_nan[n & 1][1]) {
                                if (posted) ok = tree_wait(&bar_joined, (k - 1) & 1, wd, kSiteTreeMerge);
                                if (!ok) break;
                                posted = false;
                                note_nan<D>(keys, valid, &s_nan[n & 1][0][0], s_row_nan[s][r], !odd);
                                odd = true;
                            }
                        }
                    }
                    if (hh >= 2 && __any_sync(0xffffffffu, need)) {  // O, when the stream's product before this one has run
                        ok = tree_wait(&bar_pv[(n - 2) & 3], ((n - 2) >> 2) & 1, wd, kSiteTreeO);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int ch = 0; ch < D / 32; ++ch) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32u * ch, o);
                            tmem_wait_ld();
                            reg_fence32(o);
                            const uint64_t a2 = f2_make(alpha, alpha);
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                float x, y;
                                f2_split(f2_mul(f2_make(__uint_as_float(o[c]), __uint_as_float(o[c + 1])), a2), x, y);
                                o[c] = __float_as_uint(x);
                                o[c + 1] = __float_as_uint(y);
                            }
                            tmem_st32(tO + 32u * ch, o);
                        }
                    }
                    tmem_wait_st();
                }
                if (posted) {  // (the product overwrites O)
                    ok = tree_wait(&bar_joined, (k - 1) & 1, wd, kSiteTreeMerge);
                    if (!ok) break;
                    posted = false;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_p[n & 3]);
            }
            if (!ok) break;
            // ------------------------------------------------------------- the unit's result
            // Both streams know both streams' sums then, and write half of the columns each.
            if (posted) ok = tree_wait(&bar_joined, (k - 1) & 1, wd, kSiteTreeMerge);
            if (!ok) break;
            s_post[s][r] = make_float4(M, m, l, 0.0f);
            s_post_odd[s][r] = odd;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_post[s]);
            ok = tree_wait(&bar_post[s ^ 1], k & 1, wd, kSiteTreeMerge) && tree_wait(&bar_o[k & 3], (k >> 2) & 1, wd, kSiteTreeO);
            if (!ok) break;
            tc_fence_after();
            // (a row that saw no key in a stream has l = 0 there, and what O holds is not used)
            const float4 x = s_post[0][r], y = s_post[1][r];
            const bool no0 = x.z == 0.0f, no1 = y.z == 0.0f;
            // (a maximum that is infinite or missing frames nothing)
            auto factor = [](float a, float top) { return a == top || top == -INFINITY ? 1.0f : ex2(a - top); };
            const float M2 = fmaxf(no0 ? -INFINITY : x.x, no1 ? -INFINITY : y.x);
            const float m2 = fmaxf(no0 ? -INFINITY : x.y, no1 ? -INFINITY : y.y);
            const float f0 = no0 ? -1.0f : factor(x.x, M2), f1 = no1 ? -1.0f : factor(y.x, M2);
            l = (no0 ? 0.0f : x.z * factor(x.y, m2)) + (no1 ? 0.0f : y.z * factor(y.y, m2));
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float half = M2 == -INFINITY || m2 == -INFINITY ? 1.0f : ex2(0.5f * (M2 - kFrame - m2));
            const int i = p.G(un.row0 + r), h = un.hk * p.G.d + un.row0 + r - i * p.G.d;
            const bool whole = un.J == un.nblk;
            const long long at = whole ? static_cast<long long>(un.q0 + i) * p.H + h
                                       : static_cast<long long>(2 * cta + (un.first ? 0 : 1)) * p.part_rows + r;
            const bool in = valid && in_extent(at * D, D, whole ? p.q_ext : p.part_ext, p.status);
            if (any_valid) {
                const RowResult res{f0, f1, inv, half, s_post_odd[0][r] ? s_row_nan[0][r] : nullptr,
                                    s_post_odd[1][r] ? s_row_nan[1][r] : nullptr};
                write_row<D>(tO0, s * (D / 2), res, whole ? p.o + at * D : nullptr, whole ? nullptr : p.o_part + at * D, in);
            }
            if (in && s == 0) {
                const float lse = l == 0.0f ? -INFINITY : (m2 + log2f(l)) * kLn2;
                if (!whole) {
                    p.lse_part[at] = lse;
                } else if (p.lse != nullptr) {
                    const long long so = static_cast<long long>(h) * p.total_q + un.q0 + i;
                    if (in_extent(so, 1, p.stat_ext, p.status)) p.lse[so] = lse;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_joined);
            posted = true;
            n0 += nh;
        }
    }

    __syncthreads();
    if (warp == kQkWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
}

// Merge of the parts of every unit that several shares cut, as in the cache decode: CTA c takes the unit that
// begins in share c and goes on in the next, if there is one; a warp takes a query row.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) fa_decode_tree_merge_kernel(const TreeDecodeParams p)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const int c0 = static_cast<int>(blockIdx.x);
    dependent_begin();
    const int4 cut = p.cuts[c0];
    const int q0 = cut.x, row0 = cut.y, hk = cut.z;
    const int rows = cut.w & 255, lead = cut.w >> 8 & 1, parts = cut.w >> 9;
    const int r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);
    if (r < rows) {
        float mx, sum, acc[EPL];
        merge_parts<D, 16, true>(
            parts, [&](int k) { return (2 * (c0 + k) + (k == 0 ? lead : 0)) * p.part_rows + r; }, p.o_part,
            p.lse_part, p.part_ext / D, p.status, mx, sum, acc);
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

// Rows of ancestors' bits from parents: a warp for each token, lane w holding word w of its row, walks up
// the tree.  A walk has at most as many steps as the sequence has tokens, so a circle of parents ends it too.
// (In replays 8 trees of 24 tokens 1.9 us, nearly all of it launch and reads, chains of 64 tokens 2.7.  A chain of 1024 is
// as many dependent reads of shared memory: 28 us, eight of them 76.)
constexpr int kMaskWarps = 8;
constexpr int kMaskTokens = 1024;  // the longest tree

__global__ void __launch_bounds__(32 * kMaskWarps) fa_tree_mask_kernel(const TreeMaskParams p)
{
    __shared__ int s_parent[kMaskTokens];
    dependent_begin();
    const int b = static_cast<int>(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int first;
    const int n = packed_rows(p.cu, b, p.total, p.max_q, first);
    if (static_cast<int>(blockIdx.y) * kMaskWarps >= n) return;
    for (int i = threadIdx.x; i < n; i += 32 * kMaskWarps) s_parent[i] = p.parents[first + i];
    __syncthreads();
    const int i = blockIdx.y * kMaskWarps + warp;
    if (i >= n) return;
    uint32_t word = 0;
    int at = i;
    for (int step = 0; step < n && at >= 0 && at < n; ++step) {
        if (at >> 5 == lane) word |= 1u << (at & 31);
        at = s_parent[at];
    }
    const long long off = static_cast<long long>(first + i) * p.words;
    if (lane < p.words && in_extent(off + lane, 1, p.mask_ext, p.status)) p.mask[off + lane] = word;
}

cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t st)
{
    return launch_dependent(fa_tree_mask_kernel, dim3(p.B, (p.max_q + kMaskWarps - 1) / kMaskWarps),
                            dim3(32 * kMaskWarps), 0, st, p);
}

template <int D>
static cudaError_t launch_decode_tree_impl(const TreeDecodeParams& p, cudaStream_t st)
{
    using C = TreeCfg<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(fa_decode_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    cudaError_t e = launch_dependent(fa_decode_tree_kernel<D>, dim3(p.ctas), dim3(C::THREADS), C::SMEM, st, p);
    if (e != cudaSuccess || p.ctas == 1) return e;
    return launch_dependent(fa_decode_tree_merge_kernel<D>,
                            dim3(p.ctas - 1, (p.part_rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32)),
                            dim3(kMergeThreads), 0, st, p);
}

cudaError_t launch_decode_tree(int d, const TreeDecodeParams& p, cudaStream_t st)
{
    return d == 64 ? launch_decode_tree_impl<64>(p, st) : launch_decode_tree_impl<128>(p, st);
}

}  // namespace fa
