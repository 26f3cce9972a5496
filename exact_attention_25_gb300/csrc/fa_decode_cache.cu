// Split-KV decode over the paged e4m3 cache: O = softmax(scale Q K^T [+ causal mask]) V for a
// few bf16 queries per sequence, K and V being the cache's codes times their rows' powers of
// two.  Nothing is rounded on the way in: the result is exact attention on the cached values up
// to fp32 accumulation and the f16 rounding of the softmax weights.
//
// What bounds it: the codes, read once (2 * Nk * Hkv * d bytes a sequence).  At the copy rate an
// SM receives about 23 bytes a clock, so tcgen05 has no place here although a decode tile of
// bf16 keys uses it: the codes would have to become 16-bit operands in shared memory, and one
// write by the copy, a read and a double-width write by the conversion and a double-width read
// by the tensor core (6 bytes of shared-memory traffic a code, 140 a clock) exceed the 128 bytes
// a clock that shared memory moves; kind::f8f6f4 would want Q and the weights in 8 bits too.
// Here the codes are converted between shared memory and mma.sync fragments instead, in
// registers: 2 bytes of traffic a code, 0.18 m16n8k16 a clock.
//
// Layout of a CTA: warps 0-3 compute, warp 4 copies pages to a ring of 64-key blocks by TMA
// (swizzled rows, plus the rows' exponent bytes).  A group's query rows (row i * G + g: query
// i, head g of the G that share the K/V head) form 16-row tiles; warp w works on tile
// w % row_tiles and on every (4 / row_tiles)-th 16-key step of a block, with its own online
// softmax; the warps' results merge in shared memory at the end.  Ranges of a sequence's blocks
// go to different CTAs and merge in fa_decode_merge_kernel.
//
// Per 16-key step, thread (g = lane / 4, t = lane % 4):
//  - S = Q K^T: the contraction index is permuted so that a thread's four elements of k-step s
//    are d = 16 t + 4 s + {0..3} (of the 64-wide half), i.e. one word of a 16-byte chunk, and key
//    column n holds key kperm(n) so that the chunks read together lie in different banks.
//  - O += P V: P's accumulator layout is the A layout, V's column n of tile j is d = 16 n + j
//    (8 n + j for d = 64), so a thread reads whole chunks of its keys' rows and pairs two keys'
//    bytes by a byte permute.
// Number ranges: Q rows are scaled by a power of two to just below 2^15 for f16 (elements down
// to 2^-38 of the row's largest keep a value).  Two running maxima are kept.  m, of the
// logits x (base 2), frames the sum l.  M, of x + (V's exponent), frames the weights
// w = 2^(x + ev - M + 11) that multiply V's codes, so a V row of any size keeps its weight's
// 11 bits and w <= 2^15 (maxima move when they grow by more than 4); f16's smallest step puts a
// floor of 2^-36 of the largest weight under what a single key can still add.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kKB = 64;           // keys of a block
constexpr int kComputeWarps = 4;
constexpr float kFrame = 11.0f;   // log2 of the largest weight right after a rescale
constexpr float kGrow = 4.0f;     // a maximum moves when it grows by more than this

template <int D>
struct CacheCfg {
    static constexpr int TILE = kKB * D;               // bytes of a block's K or V codes
    static constexpr int STAGE = 2 * TILE + 2 * kKB;   // codes, then exponent bytes
    static constexpr int STAGES = D == 128 ? 6 : 11;
    // codes need 1024-byte alignment: all tiles first, then the exponents of all stages
    static constexpr int EXP0 = STAGES * 2 * TILE;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int OLD = D + 4;                  // row stride of the merge buffer, floats
    static constexpr int MERGE = kComputeWarps * 16 * (OLD + 3) * 4;
    static constexpr int SMEM = (RING > MERGE ? RING : MERGE) + 1024;
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

// The key of a 16-key step's column n (0..7; columns 8..15 are the same plus 8).
template <int D>
__device__ __forceinline__ int kperm(int n)
{
    return D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}

}  // namespace

// SMALL: at most 8 query rows, so the second half of every fragment row pair is empty.
template <int D, bool SMALL>
__global__ void __launch_bounds__(CacheCfg<D>::THREADS, 2)
    fa_decode_cache_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const CacheDecodeParams p)
{
    using C = CacheCfg<D>;
    constexpr int NH = SMALL ? 1 : 2;       // rows g and g + 8 of a fragment
    constexpr int KS = D / 16;              // k-steps of S
    constexpr int NT = D / 8;               // column tiles of O
    constexpr int CH = D / 64;              // 16-byte chunks of a K row a thread reads
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar_full[C::STAGES];
    __shared__ __align__(8) uint64_t bar_empty[C::STAGES];
    __shared__ int s_valid[C::STAGES];  // bit i: keys [16 i, 16 i + 16) of the block were copied
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], kComputeWarps);
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

    const int split = static_cast<int>(blockIdx.x) % p.splits;
    int rest = static_cast<int>(blockIdx.x) / p.splits;
    const int chunk = rest % p.row_chunks;
    rest /= p.row_chunks;
    const int b = rest / p.Hkv, hk = rest % p.Hkv;
    int q0;
    const int nq = packed_rows(p.cu_q, b, p.total_q, p.max_q, q0);
    const int nk = min(max(p.seqlens[b], 0), p.max_k);
    const int row0 = chunk * 16 * p.row_tiles;                    // first query row of the CTA
    const int rows = min(nq * p.G - row0, 16 * p.row_tiles);
    if (rows <= 0) return;
    const int jb = split * p.chunk_blocks;
    const int J = min((nk + kKB - 1) / kKB - jb, p.chunk_blocks);  // blocks of this range
    const int shift = nk - nq;
    // element offset of query row r's o row (also of its partial row, within a split)
    auto out_off = [&](int r) {
        const int i = (row0 + r) / p.G, g = (row0 + r) - i * p.G;
        return (static_cast<long long>(q0 + i) * p.H + hk * p.G + g) * D;
    };
    auto stat_off = [&](int r) {
        const int i = (row0 + r) / p.G, g = (row0 + r) - i * p.G;
        return static_cast<long long>(hk * p.G + g) * p.total_q + q0 + i;
    };
    const long long part_stat = static_cast<long long>(split) * p.H * p.total_q;
    if (J <= 0) {
        // no key in this range: nothing for the merge, or (one range) a row without keys
        for (int r = threadIdx.x; r < rows; r += C::THREADS) {
            const long long so = stat_off(r);
            if (p.splits > 1) {
                if (in_extent(part_stat + so, 1, p.part_ext / D, p.status)) p.lse_part[part_stat + so] = -INFINITY;
            } else if (p.lse != nullptr && in_extent(so, 1, p.stat_ext, p.status)) {
                p.lse[so] = -INFINITY;
            }
        }
        if (p.splits == 1)
            for (int i = threadIdx.x; i < rows * (D / 8); i += C::THREADS) {
                const long long off = out_off(i / (D / 8)) + 8 * (i % (D / 8));
                if (in_extent(off, 8, p.q_ext, p.status))
                    *reinterpret_cast<uint4*>(p.o + off) = make_uint4(0u, 0u, 0u, 0u);
            }
        return;
    }

    const Watchdog wd{&abort_flag, p.status, p.wait_limit_ns};
    float* sO = reinterpret_cast<float*>(smem);               // [4][16][OLD]
    float* sStat = sO + kComputeWarps * 16 * C::OLD;          // [4][16][3]: M, m, l
    int* ok_flag = &abort_flag;

    if (warp == kComputeWarps) {
        // ------------------------------------------------------------- copies
        const int ps = 1 << p.page_shift;
        const int np = ps >= kKB ? 1 : kKB / ps;              // pages of a block
        const int rows_pp = ps >= kKB ? kKB : ps;             // rows of a copy
        const int groups_pp = rows_pp / 16;
        int base = -1, ids = -1;                              // page ids base + lane
        int issued = 0;
        for (int jj = 0; jj < J; ++jj) {
            const int s = jj % C::STAGES;
            const int pos = (jb + jj) * kKB;
            const int first = pos >> p.page_shift;
            if (base < 0 || first + np > base + 32) {
                base = first;
                const int idx = base + lane;
                ids = -1;
                if (idx < p.max_pages && (static_cast<long long>(idx) << p.page_shift) < nk)
                    ids = p.table[static_cast<long long>(b) * p.max_pages + idx];
                if (ids >= p.num_pages) ids = -1;
            }
            const int id = __shfl_sync(0xffffffffu, ids, (first - base + lane) & 31);
            const bool mine = lane < np && id >= 0;
            const uint32_t got = __ballot_sync(0xffffffffu, mine);
            if (!warp_wait_all(&bar_empty[s], ((jj / C::STAGES) & 1) ^ 1, wd, kSiteCacheEmpty)) break;
            if (lane == 0) {
                int bits = 0;
                for (int i = 0; i < np; ++i)
                    if (got >> i & 1) bits |= ((1 << groups_pp) - 1) << (i * groups_pp);
                s_valid[s] = bits;
                mbar_arrive_expect_tx(&bar_full[s],
                                      static_cast<uint32_t>(__popc(got) * rows_pp * 2 * (D + 1)));
            }
            __syncwarp();
            if (mine && !(jj == 0 && (p.debug_flags & kDebugDropFirstLoad))) {
                const int at = lane * rows_pp;                // first key of the copy in the block
                const long long row = ((static_cast<long long>(id) * p.Hkv + hk) << p.page_shift) +
                                      (pos & (ps - 1));
                uint8_t* kt = smem + s * 2 * C::TILE + at * D;
                uint8_t* ex = smem + C::EXP0 + s * 2 * kKB + at;
                tma_load_2d(kt, &tm_k, &bar_full[s], 0, static_cast<int>(row));
                bulk_load(ex, p.ke + row, rows_pp, &bar_full[s]);
                tma_load_2d(kt + C::TILE, &tm_v, &bar_full[s], 0, static_cast<int>(row));
                bulk_load(ex + kKB, p.ve + row, rows_pp, &bar_full[s]);
            }
            issued = jj + 1;
        }
        // no copy may land after the merge reuses the ring or the CTA exits
        volatile int no_abort = 0;
        const Watchdog wd_drain{&no_abort, p.status, p.wait_limit_ns};
        for (int jj = max(0, issued - C::STAGES); jj < issued; ++jj)
            if (!mbar_wait(&bar_full[jj % C::STAGES], (jj / C::STAGES) & 1, wd_drain, kSiteCacheDrain))
                *ok_flag = 1;
        __syncthreads();
    } else {
        // ------------------------------------------------------------- attention
        const int g = lane >> 2, t = lane & 3;
        const int tile = warp % p.row_tiles;
        const int slots = kComputeWarps / p.row_tiles, slot = warp / p.row_tiles;
        // This thread's query rows r[h] = tile * 16 + g + 8 h, their scale and last visible key.
        uint32_t qa[KS][4];
        float cx[NH];      // logit (base 2) per unit of the scaled product, without K's scale
        int lim[NH];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = tile * 16 + g + 8 * h;
            const bool on = (h < NH) && r < rows;
            float f[CH][16];
            float mx = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
                if (on) {
                    const long long off = out_off(r) + 64 * c + 16 * t;
                    if (in_extent(off, 16, p.q_ext, p.status)) {
                        w[0] = reinterpret_cast<const uint4*>(p.q + off)[0];
                        w[1] = reinterpret_cast<const uint4*>(p.q + off)[1];
                    }
                }
                const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[c][2 * i] = __uint_as_float(u[i] << 16);
                    f[c][2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = fabsf(f[c][i]);
                    if (a < INFINITY) mx = fmaxf(mx, a);
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // 2^a brings the row's largest magnitude to [2^14, 2^15)
            const int a = min(14 + 127 - static_cast<int>(__float_as_uint(mx) >> 23), 126);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + a) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    qa[4 * c + s][h] = pack_f16x2(f[c][4 * s] * up, f[c][4 * s + 1] * up);
                    qa[4 * c + s][2 + h] = pack_f16x2(f[c][4 * s + 2] * up, f[c][4 * s + 3] * up);
                }
            if (h < NH) {
                cx[h] = p.scale_log2 * down;
                lim[h] = -1;
                if (on) lim[h] = p.causal ? min(nk - 1, (row0 + r) / p.G + shift) : nk - 1;
            }
        }
        // keys past `most` are seen by no row of the tile; up to `least` by every row of it
        int most = -1, least = nk - 1;
        {
            const int r_first = row0 + tile * 16, r_last = row0 + min(tile * 16 + 16, rows) - 1;
            if (tile * 16 < rows) {
                most = p.causal ? min(nk - 1, r_last / p.G + shift) : nk - 1;
                if (p.causal) least = min(least, r_first / p.G + shift);
            }
        }
        float o[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        float M[NH], m[NH], l[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            M[h] = m[h] = -INFINITY;
            l[h] = 0.0f;
        }
        const int kp = kperm<D>(g);
        const int kc0 = D == 128 ? t : 2 * t, kc1 = D == 128 ? t + 4 : 2 * t + 1;  // columns 2t, 2t+1
        // which of the two keys is read first, so that a phase's rows lie in different banks
        const int swap = D == 128 ? (g & 1) : ((g >> 1) & 1);
        const int vr0 = swap ? kc1 : kc0, vr1 = swap ? kc0 : kc1;
        const uint32_t sel_lo = swap ? 0x1504u : 0x5140u, sel_hi = swap ? 0x3726u : 0x7362u;

        bool ok = true;
        for (int jj = 0; jj < J; ++jj) {
            const int s = jj % C::STAGES;
            if (!warp_wait_all(&bar_full[s], (jj / C::STAGES) & 1, wd, kSiteCacheFull)) {
                ok = false;
                break;
            }
            const int valid = s_valid[s];
            const uint8_t* kt = smem + s * 2 * C::TILE;
            const uint8_t* vt = kt + C::TILE;
            const uint8_t* ex = smem + C::EXP0 + s * 2 * kKB;
            for (int gi = slot; gi < 4; gi += slots) {
                const int kbase = (jb + jj) * kKB + gi * 16;
                if (!(valid >> gi & 1) || kbase > most) continue;
                // ---- S
                float sc[2][CH][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int row = gi * 16 + nt * 8 + kp;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const int phys = D == 128 ? ((t + 4 * c) ^ (row & 7)) : (t ^ ((row >> 1) & 3));
                        const uint4 w = *reinterpret_cast<const uint4*>(kt + row * D + 16 * phys);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                        float* a = sc[nt][c];
                        a[0] = a[1] = a[2] = a[3] = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma16816(a, qa[4 * c + k], e4m3x2_to_f16x2(u[k]), e4m3x2_to_f16x2(u[k] >> 16));
                    }
                }
                // ---- V's words, loaded early
                uint32_t va[2][2][D / 32];  // [key half][first, second row][word]
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int row = gi * 16 + hf * 8 + (f ? vr1 : vr0);
                        if constexpr (D == 128) {
                            const uint4 w = *reinterpret_cast<const uint4*>(vt + row * D + 16 * (g ^ (row & 7)));
                            va[hf][f][0] = w.x; va[hf][f][1] = w.y; va[hf][f][2] = w.z; va[hf][f][3] = w.w;
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2*>(
                                vt + row * D + 16 * ((g >> 1) ^ ((row >> 1) & 3)) + 8 * (g & 1));
                            va[hf][f][0] = w.x; va[hf][f][1] = w.y;
                        }
                    }
                // ---- softmax weights
                const bool masked = kbase + 15 > least;
                float x[NH][4], tv[NH][4];  // logits; logits plus V's exponent
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = gi * 16 + nt * 8 + (e ? kc1 : kc0);
                        const float ks = exp_byte_scale(ex[key]);
                        const uint32_t vb = ex[kKB + key];
                        const float ev = vb == 255 ? NAN : static_cast<float>(static_cast<int>(vb) - 127);
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            float sum = sc[nt][0][2 * h + e];
                            if constexpr (CH == 2) sum += sc[nt][1][2 * h + e];
                            float v = sum * (cx[h] * ks);
                            float w = v + ev;
                            if (masked && (jb + jj) * kKB + key > lim[h]) v = w = -INFINITY;
                            x[h][2 * nt + e] = v;
                            tv[h][2 * nt + e] = w;
                        }
                    }
                float xm[NH], tm[NH];
                bool need = false;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    xm[h] = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
                    tm[h] = fmaxf(fmaxf(tv[h][0], tv[h][1]), fmaxf(tv[h][2], tv[h][3]));
                    tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 1));
                    tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 2));
                    need = need || xm[h] > m[h] + kGrow || tm[h] > M[h] + kGrow;
                }
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        if (xm[h] > m[h] + kGrow) {
                            l[h] *= ex2(m[h] - xm[h]);
                            m[h] = xm[h];
                        }
                        if (tm[h] > M[h] + kGrow) {
                            const float alpha = ex2(M[h] - tm[h]);
                            M[h] = tm[h];
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                o[j][2 * h] *= alpha;
                                o[j][2 * h + 1] *= alpha;
                            }
                        }
                    }
                }
                uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float nm = m[h] == -INFINITY ? 0.0f : m[h];
                    const float nM = (M[h] == -INFINITY ? 0.0f : M[h]) - kFrame;
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        l[h] += ex2(x[h][e] - nm);
                        w[e] = ex2(tv[h][e] - nM);
                    }
                    pa[h] = pack_f16x2(w[0], w[1]);
                    pa[2 + h] = pack_f16x2(w[2], w[3]);
                }
                if (masked) {
                    // Rows past the sequence's end hold whatever the page held: zero them.  NaN
                    // codes of rows that only some queries see must not reach the others (0 *
                    // NaN): they are taken out of the product, and the rows that do see them get
                    // NaN by a product of indicators.
                    bool bad = false;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int key = kbase + hf * 8 + (f ? vr1 : vr0);
#pragma unroll
                            for (int i = 0; i < D / 32; ++i) {
                                if (key >= nk) va[hf][f][i] = 0u;
                                bad = bad || nan_bytes(va[hf][f][i]);
                            }
                        }
                    if (__any_sync(0xffffffffu, bad)) {
                        uint32_t ia[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt) {
                                const int k0 = kbase + nt * 8;
                                ia[2 * nt + h] = pack_f16x2(k0 + kc0 <= lim[h] ? 1.0f : 0.0f,
                                                            k0 + kc1 <= lim[h] ? 1.0f : 0.0f);
                            }
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            uint32_t n[2][2];
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                                for (int f = 0; f < 2; ++f) {
                                    const uint32_t nb = nan_bytes(va[hf][f][i]);
                                    n[hf][f] = (nb >> 7) * 0x38u;  // the code of 1.0 where NaN
                                    va[hf][f][i] &= ~((nb >> 7) * 0xffu);
                                }
                            uint32_t b2[2][2];
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                b2[hf][0] = __byte_perm(n[hf][0], n[hf][1], sel_lo);
                                b2[hf][1] = __byte_perm(n[hf][0], n[hf][1], sel_hi);
                            }
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                const int sh = c & 1 ? 16 : 0;
                                mma16816(cnt, ia, e4m3x2_to_f16x2(b2[0][c >> 1] >> sh),
                                         e4m3x2_to_f16x2(b2[1][c >> 1] >> sh));
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (cnt[e] > 0.0f) o[4 * i + c][e] = NAN;
                            }
                        }
                    }
                }
                // ---- O += P V
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t b2[2][2];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        b2[hf][0] = __byte_perm(va[hf][0][i], va[hf][1][i], sel_lo);
                        b2[hf][1] = __byte_perm(va[hf][0][i], va[hf][1][i], sel_hi);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int sh = c & 1 ? 16 : 0;
                        mma16816(o[4 * i + c], pa, e4m3x2_to_f16x2(b2[0][c >> 1] >> sh),
                                 e4m3x2_to_f16x2(b2[1][c >> 1] >> sh));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_empty[s]);
        }
        if (!ok) *ok_flag = 1;
        // every copy has landed and every warp is past the ring: it becomes the merge buffer
        __syncthreads();
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            // the quad's sums in one frame
            float mm = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
            mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
            float ll = l[h] * (m[h] == -INFINITY ? (l[h] == 0.0f ? 0.0f : 1.0f) : ex2(m[h] - mm));
            ll += __shfl_xor_sync(0xffffffffu, ll, 1);
            ll += __shfl_xor_sync(0xffffffffu, ll, 2);
            const int r = warp * 16 + g + 8 * h;
            if (t == 0) {
                sStat[3 * r] = M[h];
                sStat[3 * r + 1] = mm;
                sStat[3 * r + 2] = ll;
            }
            float* dst = sO + r * C::OLD + (D / 4) * t;  // columns [D / 4 * t, D / 4 * (t + 1))
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < NT; j += 4)
                    *reinterpret_cast<float4*>(dst + e * NT + j) =
                        make_float4(o[j][2 * h + e], o[j + 1][2 * h + e], o[j + 2][2 * h + e], o[j + 3][2 * h + e]);
        }
    }
    __syncthreads();
    if (*static_cast<volatile int*>(ok_flag)) return;  // a wait gave up: nothing is written
    // ------------------------------------------------------------- merge of the warps, stores
    const int slots = kComputeWarps / p.row_tiles;
    for (int i = threadIdx.x; i < rows * (D / 4); i += C::THREADS) {
        const int r = i / (D / 4), c4 = i % (D / 4);
        const int tile = r / 16, rr = r % 16;
        float mm = -INFINITY, MM = -INFINITY;
        for (int k = 0; k < slots; ++k) {
            const float* st = sStat + 3 * ((tile + k * p.row_tiles) * 16 + rr);
            MM = fmaxf(MM, st[0]);
            mm = fmaxf(mm, st[1]);
        }
        float l = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < slots; ++k) {
            const int wr = (tile + k * p.row_tiles) * 16 + rr;
            const float* st = sStat + 3 * wr;
            const float wl = st[1] == -INFINITY ? 1.0f : ex2(st[1] - mm);
            const float wo = st[0] == -INFINITY ? 1.0f : ex2(st[0] - MM);
            const float4 v = *reinterpret_cast<const float4*>(sO + wr * C::OLD + 4 * c4);
            l = fmaf(wl, st[2], l);
            acc.x = fmaf(wo, v.x, acc.x);
            acc.y = fmaf(wo, v.y, acc.y);
            acc.z = fmaf(wo, v.z, acc.z);
            acc.w = fmaf(wo, v.w, acc.w);
        }
        // O = acc 2^(MM - frame) / (l 2^mm); a row that saw no key has l = 0.  The power is
        // applied in halves: each is representable where the whole may not be.
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float half = (MM == -INFINITY || mm == -INFINITY) ? 1.0f : ex2(0.5f * (MM - kFrame - mm));
        const float f0 = inv * half;
        acc = make_float4(acc.x * f0 * half, acc.y * f0 * half, acc.z * f0 * half, acc.w * f0 * half);
        const float lse = l == 0.0f ? -INFINITY : (mm + log2f(l)) * kLn2;
        const long long off = out_off(r) + 4 * c4, so = stat_off(r);
        if (p.splits == 1) {
            if (in_extent(off, 4, p.q_ext, p.status))
                *reinterpret_cast<uint2*>(p.o + off) =
                    make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            if (c4 == 0 && p.lse != nullptr && in_extent(so, 1, p.stat_ext, p.status)) p.lse[so] = lse;
        } else {
            const long long po = static_cast<long long>(split) * p.total_q * p.H * D + off;
            if (in_extent(po, 4, p.part_ext, p.status)) *reinterpret_cast<float4*>(p.o_part + po) = acc;
            if (c4 == 0 && in_extent(part_stat + so, 1, p.part_ext / D, p.status))
                p.lse_part[part_stat + so] = lse;
        }
    }
}

// Merge of the ranges of every (query, head) row, one warp each:
//     O = sum_s e^{lse_s} O_s / sum_s e^{lse_s},   lse = log sum_s e^{lse_s}.
// Only ranges that saw a key (lse_s > -inf) are read; a row without any gets O = 0, lse = -inf.
// Rows that belong to no sequence are left as they are.
template <int D>
__global__ void __launch_bounds__(256) fa_decode_merge_kernel(const MergeParams p)
{
    constexpr int EPL = D / 32;
    constexpr int BATCH = 4;  // ranges whose rows are in flight together
    dependent_begin();
    const int lane = threadIdx.x & 31;
    const int w = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int h = w % p.H;
    const int i = w / p.H % p.max_q, b = w / p.H / p.max_q;
    if (b >= p.B) return;
    int q0;
    const int nq = packed_rows(p.cu_q, b, p.total_q, p.max_q, q0);
    if (i >= nq) return;
    const long long stat = static_cast<long long>(h) * p.total_q + q0 + i;
    const long long row = (static_cast<long long>(q0 + i) * p.H + h) * D + EPL * lane;
    const long long stat_step = static_cast<long long>(p.H) * p.total_q;
    float mx = -INFINITY, sum = 0.0f, acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
    for (int s0 = 0; s0 < p.splits; s0 += 32) {
        float ls = -INFINITY;
        if (s0 + lane < p.splits && in_extent((s0 + lane) * stat_step + stat, 1, p.part_ext / D, p.status))
            ls = p.lse_part[(s0 + lane) * stat_step + stat];
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
                    const long long po = (s0 + s) * stat_step * D + row;
                    if (in_extent(po, EPL, p.part_ext, p.status)) {
                        if constexpr (EPL == 4) {
                            const float4 x = *reinterpret_cast<const float4*>(p.o_part + po);
                            v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
                        } else {
                            const float2 x = *reinterpret_cast<const float2*>(p.o_part + po);
                            v[k][0] = x.x; v[k][1] = x.y;
                        }
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
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (in_extent(row, EPL, p.q_ext, p.status)) {
        if constexpr (EPL == 4)
            *reinterpret_cast<uint2*>(p.o + row) =
                make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(p.o + row) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
    if (lane == 0 && p.lse != nullptr && in_extent(stat, 1, p.stat_ext, p.status))
        p.lse[stat] = sum == 0.0f ? -INFINITY : mx + logf(sum);
}

cudaError_t launch_decode_merge(int d, const MergeParams& p, cudaStream_t st)
{
    const long long rows = static_cast<long long>(p.B) * p.max_q * p.H;
    const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
    if (d == 64) return launch_dependent(fa_decode_merge_kernel<64>, grid, dim3(256), 0, st, p);
    return launch_dependent(fa_decode_merge_kernel<128>, grid, dim3(256), 0, st, p);
}

template <int D, bool SMALL>
static cudaError_t launch_decode_cache_impl(const CUtensorMap& tk, const CUtensorMap& tv,
                                            const CacheDecodeParams& p, cudaStream_t st)
{
    using C = CacheCfg<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(fa_decode_cache_kernel<D, SMALL>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const dim3 grid(static_cast<unsigned>(p.B * p.Hkv * p.row_chunks * p.splits));
    return launch_dependent(fa_decode_cache_kernel<D, SMALL>, grid, dim3(C::THREADS), C::SMEM, st,
                            tk, tv, p);
}

cudaError_t launch_decode_cache(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheDecodeParams& p, cudaStream_t st)
{
    const bool small = static_cast<long long>(p.max_q) * p.G <= 8;
    cudaError_t e;
    if (d == 64)
        e = small ? launch_decode_cache_impl<64, true>(tk, tv, p, st)
                  : launch_decode_cache_impl<64, false>(tk, tv, p, st);
    else
        e = small ? launch_decode_cache_impl<128, true>(tk, tv, p, st)
                  : launch_decode_cache_impl<128, false>(tk, tv, p, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    MergeParams m{};
    m.o = p.o; m.lse = p.lse; m.o_part = p.o_part; m.lse_part = p.lse_part;
    m.cu_q = p.cu_q; m.B = p.B; m.H = p.H; m.max_q = p.max_q; m.total_q = p.total_q;
    m.splits = p.splits; m.q_ext = p.q_ext; m.stat_ext = p.stat_ext; m.part_ext = p.part_ext;
    m.status = p.status;
    return launch_decode_merge(d, m, st);
}

}  // namespace fa
