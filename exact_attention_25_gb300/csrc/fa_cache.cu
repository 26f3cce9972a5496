// The paged e4m3 key/value cache: rows are quantised as they are written (append) and turned
// back into bf16 or fp32 (read).
//
// A row is the d elements of one token and key/value head.  Its scale is the least power of two
// 2^e with max|x| <= 448 * 2^e (e in [-110, 120]; 0 for a row of zeros), kept as the byte
// e + 127; its codes are x * 2^-e rounded to the nearest e4m3 value, ties to even.  A power of
// two costs no accuracy in a floating format (the relative spacing is the same in every binade),
// makes the division by the scale exact, needs one byte, and makes reading back into bf16 exact.
// Infinities and NaNs are stored as the NaN code and do not count towards the maximum.
//
// Both directions are HBM-bound: each element is read and written once (reading 8 sequences of up to 16 K
// tokens: 70 us, 96 % of the copy rate; writing 64 prompts of 1 K: 60 us, 98 %, 9 ragged ones of up to
// 8 K, which leave half of the grid's warps without rows: 35 us, 86 %).  A warp owns 16 tokens of one head;
// the warps of a CTA take neighbouring heads of the same tokens, so a CTA touches whole runs of the packed
// rows [token, head, d], while each warp touches one run of a page [head, row, d].  All loads of a tensor's
// 16 rows are issued before any is used.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

namespace fa {

namespace {

constexpr int kCacheThreads = 128;
constexpr int kCacheTokens = 16;  // tokens of a warp: pages hold a multiple of this

// 16 elements of a row as floats
__device__ __forceinline__ void unpack16(const uint4* w, float* f, const __nv_bfloat16*)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t u[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[8 * h + 2 * i] = __uint_as_float(u[i] << 16);
            f[8 * h + 2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void unpack16(const uint4* w, float* f, const float*)
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        f[4 * h] = __uint_as_float(w[h].x);
        f[4 * h + 1] = __uint_as_float(w[h].y);
        f[4 * h + 2] = __uint_as_float(w[h].z);
        f[4 * h + 3] = __uint_as_float(w[h].w);
    }
}
__device__ __forceinline__ void pack16(const float* f, uint4* w, const __nv_bfloat16*)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = make_uint4(pack_bf16x2(f[8 * h], f[8 * h + 1]), pack_bf16x2(f[8 * h + 2], f[8 * h + 3]),
                          pack_bf16x2(f[8 * h + 4], f[8 * h + 5]), pack_bf16x2(f[8 * h + 6], f[8 * h + 7]));
}
__device__ __forceinline__ void pack16(const float* f, uint4* w, const float*)
{
#pragma unroll
    for (int h = 0; h < 4; ++h)
        w[h] = make_uint4(__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]),
                          __float_as_uint(f[4 * h + 2]), __float_as_uint(f[4 * h + 3]));
}

// The largest |x| of a lane's 16 elements as fp32 bits (infinities and NaNs largest of all), and the
// same over the finite ones.  bf16 values compare as 16-bit integers, two at a time.
__device__ __forceinline__ uint32_t amax16(const uint4* w, const __nv_bfloat16*)
{
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t u[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, u[i] & 0x7fff7fffu);
    }
    return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax16(const uint4* w, const float*)
{
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        m = max(max(m, w[h].x & 0x7fffffffu), w[h].y & 0x7fffffffu);
        m = max(max(m, w[h].z & 0x7fffffffu), w[h].w & 0x7fffffffu);
    }
    return m;
}
__device__ __forceinline__ uint32_t amax16_finite(const float* f)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t a = __float_as_uint(f[i]) & 0x7fffffffu;
        m = max(m, a < 0x7f800000u ? a : 0u);
    }
    return m;
}

// The biased exponent of a row whose largest finite |x| has the bits `amax`: with amax = m 2^E
// (1 <= m < 2), 448 = 1.75 * 2^8 gives e = E - 8, or E - 7 where m > 1.75.
__device__ __forceinline__ int row_exponent(uint32_t amax)
{
    if (amax == 0) return 127;
    const int up = static_cast<int>((amax + 0x1fffffu) >> 23);  // E + 127 (+1 if m > 1.75)
    return min(max(up - 8, 127 - 110), 127 + 120);
}

// The warp's place: 16 tokens [i0, i0 + 16) and head hk of sequence b.
struct Place {
    int b, i0, hk;
};
__device__ __forceinline__ bool warp_place(const CacheParams& p, Place& w)
{
    const int id = static_cast<int>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
    const int tiles = (p.max_new + kCacheTokens - 1) / kCacheTokens;
    w.hk = id % p.Hkv;
    const int rest = id / p.Hkv;
    w.i0 = (rest % tiles) * kCacheTokens;
    w.b = rest / tiles;
    return w.b < p.B;
}

// Row of the cache (in units of d codes) that holds position pos of sequence b, or -1.
__device__ __forceinline__ long long cache_row(const CacheParams& p, int b, int hk, long long pos)
{
    const long long idx = pos >> p.page_shift;
    if (pos < 0 || idx >= p.max_pages) return -1;
    const int page = p.table[static_cast<long long>(b) * p.max_pages + idx];
    if (page < 0 || page >= p.num_pages) return -1;
    return ((static_cast<long long>(page) * p.Hkv + hk) << p.page_shift) +
           (pos & ((1 << p.page_shift) - 1));
}

}  // namespace

// SPLIT: half of the grid (y) takes k and half v; where the grid is small anyway the two then run side by side
// (one new token for each of 64 sequences: 2.7 us, 3.2 in turn; 64 of 128 tokens: 11.0 and 10.5).  In turn
// the loop over k and v stays rolled for bf16, whose warps then fit more often (64 of 1 K tokens: 60.5 us,
// unrolled 62.8), and is unrolled for fp32 (101 us, rolled 107).
template <class T, int D, bool WIDE, bool SPLIT>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_append_kernel(const CacheParams p)
{
    constexpr int LR = D / 16;                // lanes of a row, 16 elements each
    constexpr int RW = 32 / LR;               // rows of a step
    constexpr int NI = kCacheTokens / RW;     // steps
    constexpr int WD = sizeof(T);             // 16-byte words of 16 elements
    dependent_begin();
    Place w;
    if (!warp_place(p, w)) return;
    const int lane = threadIdx.x & 31, l = lane % LR;
    int first;
    const int n = packed_rows(p.cu, w.b, p.total, p.max_new, first);
    if (w.i0 >= n) return;
    const long long start = static_cast<long long>(p.seqlens[w.b]) - n;  // position of the sequence's first new token
    long long to[NI];                      // cache rows of the lane's tokens (-1: none)
#pragma unroll
    for (int s = 0; s < NI; ++s) {
        const int i = w.i0 + s * RW + lane / LR;
        to[s] = i < n ? cache_row(p, w.b, w.hk, start + i) : -1;
    }
    const int z0 = SPLIT ? blockIdx.y : 0;
    constexpr int kTensors = SPLIT ? 1 : 2, kUnroll = sizeof(T) == 4 ? kTensors : 1;
#pragma unroll kUnroll
    for (int z = z0; z < z0 + kTensors; ++z) {
        const T* src = static_cast<const T*>(z ? p.v : p.k);
        const long long rs = z ? p.v_rs : p.k_rs, hs = z ? p.v_hs : p.k_hs;
        uint8_t* codes = z ? p.vc : p.kc;
        uint8_t* exps = z ? p.ve : p.ke;
        uint4 x[NI][WD];
#pragma unroll
        for (int s = 0; s < NI; ++s) {
            const int i = w.i0 + s * RW + lane / LR;
            const long long off = (first + i) * rs + w.hk * hs + 16 * l;
#pragma unroll
            for (int h = 0; h < WD; ++h) x[s][h] = make_uint4(0u, 0u, 0u, 0u);
            if (i < n && in_extent(off, 16, z ? p.v_ext : p.k_ext, p.status)) {
#pragma unroll
                for (int h = 0; h < WD; h += 2)
                    load_32b<WIDE>(reinterpret_cast<const uint4*>(src + off) + h, x[s] + h);
            }
        }
#pragma unroll
        for (int s = 0; s < NI; ++s) {
            uint32_t amax = amax16(x[s], src);
#pragma unroll
            for (int m = 1; m < LR; m *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
            float f[16];
            unpack16(x[s], f, src);
            const bool odd = amax >= 0x7f800000u;
            if (__any_sync(0xffffffffu, odd)) {  // a row with infinities or NaNs, rarely
                uint32_t fin = amax16_finite(f);
#pragma unroll
                for (int m = 1; m < LR; m *= 2) fin = max(fin, __shfl_xor_sync(0xffffffffu, fin, m));
                amax = fin;
                // the conversion would saturate an infinity: x * 0 is NaN for it and for NaN
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = fmaf(f[i], 0.0f, f[i]);
            }
            const int e = row_exponent(amax);
            const float scale = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^-(e-127)
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] *= scale;
            const uint4 c = make_uint4(
                pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]),
                pack_e4m3x4(f[8], f[9], f[10], f[11]), pack_e4m3x4(f[12], f[13], f[14], f[15]));
            if (to[s] >= 0 && in_extent(to[s] * D, D, p.code_ext, p.status)) {
                *reinterpret_cast<uint4*>(codes + to[s] * D + 16 * l) = c;
                if (l == 0) exps[to[s]] = static_cast<uint8_t>(e);
            }
        }
    }
}

// Rows whose page is missing from the table read as zero.
template <class T, int D, bool WIDE>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_read_kernel(const CacheParams p)
{
    constexpr int LR = D / 16;
    constexpr int RW = 32 / LR;
    constexpr int NI = kCacheTokens / RW;
    constexpr int WD = sizeof(T);
    dependent_begin();
    Place w;
    if (!warp_place(p, w)) return;
    const int lane = threadIdx.x & 31, l = lane % LR;
    int first;
    const int n = packed_rows(p.cu, w.b, p.total, p.max_new, first);
    if (w.i0 >= n) return;
    // the 16 positions lie in one page
    const long long row0 = cache_row(p, w.b, w.hk, w.i0);
    uint4 x[2][NI];
    uint32_t e[2][NI];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int s = 0; s < NI; ++s) {
            const int r = s * RW + lane / LR;
            x[z][s] = make_uint4(0u, 0u, 0u, 0u);
            e[z][s] = 127;
            if (row0 >= 0 && w.i0 + r < n && in_extent((row0 + r) * D, D, p.code_ext, p.status)) {
                x[z][s] = *reinterpret_cast<const uint4*>((z ? p.vc : p.kc) + (row0 + r) * D + 16 * l);
                e[z][s] = (z ? p.ve : p.ke)[row0 + r];
            }
        }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        T* dst = static_cast<T*>(const_cast<void*>(z ? p.v : p.k));
        const long long rs = z ? p.v_rs : p.k_rs, hs = z ? p.v_hs : p.k_hs;
#pragma unroll
        for (int s = 0; s < NI; ++s) {
            const int i = w.i0 + s * RW + lane / LR;
            const float scale = exp_byte_scale(e[z][s]);
            const uint32_t u[4] = {x[z][s].x, x[z][s].y, x[z][s].z, x[z][s].w};
            float f[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h2 = e4m3x2_to_f16x2(j & 1 ? u[j / 2] >> 16 : u[j / 2]);
                const float2 v2 = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                f[2 * j] = v2.x * scale;
                f[2 * j + 1] = v2.y * scale;
            }
            uint4 o[WD];
            pack16(f, o, dst);
            const long long off = (first + i) * rs + w.hk * hs + 16 * l;
            if (i < n && in_extent(off, 16, z ? p.v_ext : p.k_ext, p.status)) {
#pragma unroll
                for (int h = 0; h < WD; h += 2)
                    store_32b<WIDE>(reinterpret_cast<uint4*>(dst + off) + h, o + h);
            }
        }
    }
}

// One warp for each 16 tokens of the longest sequence, each sequence and each head.
static dim3 cache_grid(const CacheParams& p)
{
    const long long tiles = (p.max_new + kCacheTokens - 1) / kCacheTokens;
    const long long warps = tiles * p.B * p.Hkv;
    return dim3(static_cast<unsigned>((warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32)));
}

template <class T, int D>
static cudaError_t launch_append(const CacheParams& p, bool wide, cudaStream_t st, int num_sms)
{
    dim3 g = cache_grid(p);
    const dim3 t(kCacheThreads);
    if (g.x <= 2u * num_sms) {
        g.y = 2;
        return wide ? launch_dependent(fa_cache_append_kernel<T, D, true, true>, g, t, 0, st, p)
                    : launch_dependent(fa_cache_append_kernel<T, D, false, true>, g, t, 0, st, p);
    }
    return wide ? launch_dependent(fa_cache_append_kernel<T, D, true, false>, g, t, 0, st, p)
                : launch_dependent(fa_cache_append_kernel<T, D, false, false>, g, t, 0, st, p);
}

template <class T, int D>
static cudaError_t launch_read(const CacheParams& p, bool wide, cudaStream_t st)
{
    const dim3 g = cache_grid(p), t(kCacheThreads);
    return wide ? launch_dependent(fa_cache_read_kernel<T, D, true>, g, t, 0, st, p)
                : launch_dependent(fa_cache_read_kernel<T, D, false>, g, t, 0, st, p);
}

static bool cache_wide(const CacheParams& p, int es)
{
    return wide_rows(p.k, p.k_rs, p.k_hs, es) && wide_rows(p.v, p.v_rs, p.v_hs, es);
}

cudaError_t launch_cache_append(int d, int is_f32, const CacheParams& p, cudaStream_t st, int num_sms)
{
    const bool w = cache_wide(p, is_f32 ? 4 : 2);
    if (d == 64)
        return is_f32 ? launch_append<float, 64>(p, w, st, num_sms) : launch_append<__nv_bfloat16, 64>(p, w, st, num_sms);
    return is_f32 ? launch_append<float, 128>(p, w, st, num_sms) : launch_append<__nv_bfloat16, 128>(p, w, st, num_sms);
}

cudaError_t launch_cache_read(int d, int is_f32, const CacheParams& p, cudaStream_t st)
{
    const bool w = cache_wide(p, is_f32 ? 4 : 2);
    if (d == 64) return is_f32 ? launch_read<float, 64>(p, w, st) : launch_read<__nv_bfloat16, 64>(p, w, st);
    return is_f32 ? launch_read<float, 128>(p, w, st) : launch_read<__nv_bfloat16, 128>(p, w, st);
}

}  // namespace fa
