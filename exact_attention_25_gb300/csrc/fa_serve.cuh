// Shared definitions of the serving-side operators: rotary positions (fa_rope.cu), the paged
// e4m3 key/value cache (fa_cache.cu), the split-KV decode over that cache (fa_decode_cache.cu)
// and the decode with shared prefixes (fa_decode_shared.cu).
#pragma once
#include "fa_common.cuh"

namespace fa {

// Watchdog sites of the serving kernels (see WaitSite; values below 64).
enum ServeWaitSite : int {
    kSiteCacheEmpty = 32,
    kSiteCacheFull,
    kSiteCacheDrain,
    kSiteCacheMerge,
    kSiteSharedEmpty,
    kSiteSharedUnit,
    kSiteSharedQ,
    kSiteSharedK,
    kSiteSharedV,
    kSiteSharedS,
    kSiteSharedP,
    kSiteSharedO,
    kSiteSharedDrain,
};

// Division by a number known on the host: x / d = (x * m) >> 32 with m = floor(2^32 / d) + 1, exact for
// x * d < 2^32 (m d exceeds 2^32 by at most d).  A division in line is some 25 instructions, and these
// kernels' first microseconds go by what they have to fetch.
struct FastDiv {
    unsigned long long m;
    int d;
    FastDiv() = default;
    explicit FastDiv(int v) : m((1ull << 32) / static_cast<unsigned>(v) + 1), d(v) {}
    __device__ __forceinline__ int operator()(int x) const
    {
        return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(x)) * m) >> 32);
    }
};

constexpr int kRopeMaxPairs = 64;

// Rotary positions.  Pair p of a head turns by positions[axis[p]][token] * turn[p] / 2^64 turns.
struct RopeParams {
    const void* x[2];          // q, k (k null when Hkv = 0)
    void* y[2];
    long long x_rs[2], x_hs[2], y_rs[2], y_hs[2];  // element strides of a token and a head
    long long x_ext[2], y_ext[2];                  // element extents (checked builds)
    const int* pos;            // [axes, total]
    long long pos_ext;
    int total, H, Hkv;
    int pairs;                 // rotated pairs of a head, a multiple of 8
    FastDiv parts;             // warps of a token ...
    int per;                   // ... and the head steps of each
    float sign;                // -1 turns backwards (the gradient)
    int* status;
    unsigned long long turn[kRopeMaxPairs];  // turns per position, in units of 2^-64
    unsigned char axis[kRopeMaxPairs];
};

// The paged cache: codes [num_pages, Hkv, page_size, d] (e4m3), one biased exponent a row
// [num_pages, Hkv, page_size] (value of a code c under exponent byte x: c * 2^(x - 127)).
// Position j of sequence b lies in page table[b][j / page_size], row j % page_size; a page
// outside [0, num_pages) holds nothing.
struct CacheParams {
    const void* k;             // append: new rows [total, Hkv, d]; read: outputs of that shape
    const void* v;
    long long k_rs, k_hs, v_rs, v_hs;  // element strides of those rows
    long long k_ext, v_ext;            // their element extents (checked builds)
    uint8_t* kc;
    uint8_t* vc;
    uint8_t* ke;
    uint8_t* ve;
    const int* cu;             // [B + 1] starts of the sequences' rows in k, v
    const int* seqlens;        // append: cached tokens of each sequence after the call
    const int* table;          // [B, max_pages]
    int B, Hkv, total, max_new;
    int max_pages, num_pages, page_shift;
    long long code_ext;        // elements of kc (checked builds); exponents: code_ext / d
    int* status;
};

constexpr int kCacheBlock = 128;  // keys of a block of the cache decode

// What a unit (below) costs besides its blocks (queries, merge of the warps, output), in blocks.
// Cache decode with 1, 2, 3 and 4: 64 sequences of up to 4 K keys 56.6, 51.7, 51.8, 52.4 us; 16 of up to 5000, 32 rows
// at d = 64: 17.4, 16.8, 16.8, 17.0; 8 of up to 32 K: 62.3-62.6.  Shared prefixes: 64 sequences over 32000 tokens at
// d = 128: 67.5, 64.6, 63.9, 67.0 us, at d = 64: 63.4, 60.4, 61.6, 64.8; 8 over 4 K: 14.5, 13.3, 13.4, 13.9; 24 with 4
// queries each over three prefixes of up to 8 K: 40.6, 38.3, 38.9, 39.8.
constexpr int kUnitCost = 2;
constexpr int kSharedUnitCost = 3;

// Split-KV decode over the paged cache.  The work is a line of units: for every sequence, for
// every `rows_cta` query rows of a group and every key/value head, kUnitCost places and one place
// for each 128-key block of the sequence (at least one).  The CTAs take equal shares of that line
// (to a place), however ragged the lengths are.  A unit whose blocks lie in one share is finished
// by its CTA; one that several shares cut is written in parts, and merged by the next kernel, for
// which the CTA with the unit's first block describes it (cuts).
struct CacheDecodeParams {
    const __nv_bfloat16* q;    // [total_q, H, d]
    __nv_bfloat16* o;
    float* lse;                // [H, total_q] (may be null)
    float* o_part;             // workspace: fp32 [2 * ctas, rows_cta, d]; a share's first unit is
    float* lse_part;           // its part 2 c, its last (if another) 2 c + 1; [2 * ctas, rows_cta]
    int4* cuts;                // workspace [ctas]: the unit that begins in share c and goes on in the next
    const uint8_t* ke;
    const uint8_t* ve;
    const int* cu_q;           // [B + 1]
    const int* seqlens;        // [B] keys of each sequence
    const int* table;          // [B, max_pages]
    int B, H, Hkv;
    FastDiv G;                 // H / Hkv
    FastDiv heads;             // Hkv
    int max_q, max_k, total_q;
    int table_k;               // keys that a row of the table has room for
    int max_pages, num_pages, page_shift;
    int ctas;
    int row_tiles;             // row tiles of a CTA
    int rows_cta, rows_shift;  // query rows of a CTA, and their log2
    float scale_log2;
    int causal;
    int* status;
    unsigned long long wait_limit_ns;
    int debug_flags;
    long long q_ext, stat_ext, part_ext;  // element extents (checked builds)
};

// Decode with shared prefixes: the same kind of line, over the groups' prefixes and then the
// sequences' own keys, in units of one tile of query rows (tile_tokens tokens times the G heads of
// a group, at most 128) and one key/value head.  Every one of head_groups sets of heads (head hk is
// in set hk mod head_groups) has a line of its own, in `parts` shares: CTA c takes share
// c / head_groups of set c mod head_groups.
struct SharedDecodeParams {
    __nv_bfloat16* o;          // [total_q, H, d]
    float* lse;                // [H, total_q] (may be null)
    // workspace rows of d fp32 values and their LSE: [2][total_q][H] for units that one share
    // holds whole (prefix, own keys), then from row part_row0 on 128 rows for each of the parts
    // 2 c (first unit of share c) and 2 c + 1 (last)
    float* o_part;
    float* lse_part;
    long long part_row0;
    int4* places;              // workspace [total_q][2]: where the merge finds a token's parts (place_tokens)
    const __nv_bfloat16* v;    // [total_k, Hkv, d] (read for infinities and NaNs only)
    const int* cu_q;           // [B + 1]
    const int* cu_k;           // [B + 1]
    const int* cu_g;           // [groups + 1] first sequence of each group
    const int* cu_p;           // [groups + 1] first row of each group's prefix
    int B, groups, H, Hkv;
    FastDiv G;                 // H / Hkv
    int max_q, max_k, max_group_q, max_p;
    int total_q, total_k, total_p;
    FastDiv tile_tokens;
    int ctas, head_groups, parts;
    float scale_log2;
    int causal;
    int* status;
    unsigned long long wait_limit_ns;
    int debug_flags;
    long long q_ext, stat_ext, v_ext, part_ext;  // extents (checked builds): elements, workspace rows
};

// The line of T places in `ctas` shares, the first T mod ctas of them one place longer.  (T is
// below 2^31: checked on the host for the largest batch of the call's sizes.)
struct Shares {
    int total, per, more;
    __device__ __forceinline__ Shares(int T, int ctas)
        : total(T), per(static_cast<unsigned>(T) / static_cast<unsigned>(ctas)), more(T - per * ctas)
    {
    }
    __device__ __forceinline__ int start(int c) const { return c * per + min(c, more); }
    __device__ __forceinline__ int share_of(int pos) const
    {
        const int cut = more * (per + 1);
        return pos < cut ? pos / (per + 1) : more + (pos - cut) / per;
    }
};

// All lanes of a warp: the shares of a line of `items` items of places(x) places each (0 for x past
// the last), and, for the first place of share c, its item and `at`, its distance from the item's
// first place.  Neither is set when the share starts at the line's end.
template <class F>
__device__ __forceinline__ Shares find_share(int items, int ctas, int c, F places, int& item, int& at)
{
    const int lane = threadIdx.x & 31;
    const int w0 = places(lane);  // (most batches have no more than 32 items)
    int total = w0;
#pragma unroll 1
    for (int x0 = 32; x0 < items; x0 += 32) total += places(x0 + lane);
    const Shares sh(__reduce_add_sync(0xffffffffu, total), ctas);
    const int pos = sh.start(c);
    if (pos >= sh.total) return sh;
    int run = 0;
#pragma unroll 1
    for (int x0 = 0; x0 < items; x0 += 32) {
        const int w = x0 == 0 ? w0 : places(x0 + lane);
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
            item = x0 + src;
            break;
        }
        run += __shfl_sync(0xffffffffu, sum, 31);
    }
    return sh;
}

// The merge of a query row's parts, by a warp: O = sum_s e^{lse_s} O_s / sum_s e^{lse_s} and lse = log
// sum_s e^{lse_s}, whose numerators are left in acc (elements D / 32 * lane on), denominator in sum and
// frame in mx (sum = 0: no part saw a key).  Part k is row row_of(k) of the workspace.  The rows of a batch
// are loaded along with their lse, in one round trip (one sequence of 4 K keys, 16 parts: 1.2 us less than four
// at a time, after their lse); those of parts that saw no key hold anything and are not used.
template <int D, int BATCH, class F>
__device__ __forceinline__ void merge_parts(int parts, F row_of, const float* o_part, const float* lse_part,
                                            long long rows, int* status, float& mx, float& sum, float* acc)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    mx = -INFINITY;
    sum = 0.0f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
#pragma unroll 1
    for (int s0 = 0; s0 < parts; s0 += BATCH) {
        float ls = -INFINITY, v[BATCH][EPL];
        int row = 0;
        if (lane < BATCH && s0 + lane < parts) {
            row = row_of(s0 + lane);
            if (in_extent(row, 1, rows, status)) ls = lse_part[row];
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (s0 + k >= parts) continue;
            const int r = __shfl_sync(0xffffffffu, row, k);
            if (!in_extent(r, 1, rows, status)) continue;
            const float* src = o_part + static_cast<long long>(r) * D + EPL * lane;
            if constexpr (EPL == 4) {
                const float4 x = *reinterpret_cast<const float4*>(src);
                v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(src);
                v[k][0] = x.x; v[k][1] = x.y;
            }
        }
        const uint32_t live = __ballot_sync(0xffffffffu, !(ls == -INFINITY));  // NaN counts
        if (!live) continue;
        float nm = fmaxf(mx, ls);
#pragma unroll
        for (int d = 16; d; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
        const float keep = mx == -INFINITY ? 0.0f : expf(mx - nm);
        sum *= keep;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] *= keep;
        mx = nm;
        const float wt = ls == -INFINITY ? 0.0f : expf(ls - nm);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const float w = __shfl_sync(0xffffffffu, wt, k);
            if (!(live >> k & 1)) continue;
            sum += w;
#pragma unroll
            for (int e = 0; e < EPL; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
        }
    }
}

// 2^(byte - 127), the scale an exponent byte stands for; 255 is NaN.
__device__ __forceinline__ float exp_byte_scale(uint32_t byte)
{
    const uint32_t bits = byte == 0 ? 0x00400000u : (byte == 255 ? 0x7fc00000u : byte << 23);
    return __uint_as_float(bits);
}

// Two e4m3 codes (low byte first) to packed f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two)));
    return r;
}

// Rows of packed sequence b, clamped to the tensor of `total` rows and to `most`.
__device__ __forceinline__ int packed_rows(const int* cu, int b, int total, int most, int& first)
{
    first = min(max(cu[b], 0), total);
    const int end = min(max(cu[b + 1], first), total);
    return min(end - first, most);
}

// 32 bytes at once: where each thread of a warp takes 32 neighbouring bytes, 16-byte accesses would
// use half of every 32-byte sector each.  The address is a multiple of 32 (WIDE), or of 16.
template <bool WIDE>
__device__ __forceinline__ void load_32b(const void* p, uint4* w)
{
    if constexpr (WIDE) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x),
                       "=r"(w[1].y), "=r"(w[1].z), "=r"(w[1].w)
                     : "l"(p)
                     : "memory");
    } else {
        w[0] = reinterpret_cast<const uint4*>(p)[0];
        w[1] = reinterpret_cast<const uint4*>(p)[1];
    }
}
template <bool WIDE>
__device__ __forceinline__ void store_32b(void* p, const uint4* w)
{
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0].x),
                     "r"(w[0].y), "r"(w[0].z), "r"(w[0].w), "r"(w[1].x), "r"(w[1].y), "r"(w[1].z),
                     "r"(w[1].w)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = w[0];
        reinterpret_cast<uint4*>(p)[1] = w[1];
    }
}

// Whether a tensor's rows can be taken 32 bytes at a time.
inline bool wide_rows(const void* p, long long rs, long long hs, int elem_bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(rs * elem_bytes) |
             static_cast<uintptr_t>(hs * elem_bytes)) & 31u) == 0;
}

// Launch as a programmatic dependent of the work before it on the stream: the grid's launch and
// set-up overlap that work's end.  Every kernel launched so waits (griddepcontrol.wait) in all
// of its threads before it touches global memory, so stream order is kept.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Wait for the work before this grid, then let the next grid's set-up start.
__device__ __forceinline__ void dependent_begin()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace fa
