// Rotary positions with several axes: pair p of every head of token t, (x1, x2), becomes
//     (x1 cos a - x2 sin a, x2 cos a + x1 sin a),   a = positions[axis[p]][t] * inv_freq[p],
// for q and k in one launch; the transposed rotation (sign = -1) is the backward pass, since
// the map is orthogonal.  Pairs are (i, pairs + i) or, interleaved, (2i, 2i + 1); elements past
// the 2 * pairs rotated ones are copied.
//
// Angles.  a grows to millions of radians for far positions, where an fp32 product has lost the
// fraction of a turn that matters.  The host turns each inv_freq into turns per position as a
// 64-bit fixed-point fraction; position * turn modulo 2^64 is then the exact fraction of a turn
// of that fixed-point frequency (whole turns drop out by overflow, negative positions included).
// Its top 32 bits, reduced to within an eighth of a turn of a quadrant, enter sincospif with an
// error below 2^-25 turns.
//
// HBM-bound: each element is read and written once.  32000 tokens of 64 heads of
// 128, bf16: 152 us, the copy rate; the gradient of 16388 tokens of 32 heads of 64 in fp32: 41 us, 97 % of
// it; 8 tokens: 1.8 us.  One warp owns a token (or, with few tokens,
// one of `parts` shares of its heads): its lanes compute each angle's sine and cosine once,
// exchange them by shuffles, and keep the 8 pairs of their 16-byte chunks in registers over all
// the token's heads, so the trigonometry costs 1/(heads) of an element each.
#include "fa_serve.cuh"
#include "tc_ptx.cuh"

namespace fa {

namespace {

// Sine and cosine of t / 2^32 turns.
__device__ __forceinline__ void turn_sincos(uint32_t t, float& s, float& c)
{
    const uint32_t quad = (t + 0x20000000u) >> 30;
    const int r = static_cast<int>(t - (quad << 30));  // within an eighth of a turn
    float s0, c0;
    sincospif(static_cast<float>(r) * 0x1p-31f, &s0, &c0);
    s = (quad & 1) ? c0 : s0;
    c = (quad & 1) ? s0 : c0;
    if (quad & 2) s = -s;
    if (quad == 1 || quad == 2) c = -c;
}

// 8 elements: 16 bytes of bf16, 32 of fp32.
template <class T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    uint4 w[1];
    __device__ __forceinline__ void get(float* f) const
    {
        const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void put(const float* f)
    {
        w[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Chunk<float> {
    uint4 w[2];
    __device__ __forceinline__ void get(float* f) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(w[i].x);
            f[4 * i + 1] = __uint_as_float(w[i].y);
            f[4 * i + 2] = __uint_as_float(w[i].z);
            f[4 * i + 3] = __uint_as_float(w[i].w);
        }
    }
    __device__ __forceinline__ void put(const float* f)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                              __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
    }
};

// A lane's two chunks.  NEXT: hi follows lo.
template <bool WIDE, bool NEXT>
__device__ __forceinline__ void load_chunks(const __nv_bfloat16* lo, const __nv_bfloat16* hi,
                                            Chunk<__nv_bfloat16>& a, Chunk<__nv_bfloat16>& b)
{
    if constexpr (NEXT && WIDE) {
        uint4 w[2];
        load_32b<true>(lo, w);
        a.w[0] = w[0];
        b.w[0] = w[1];
    } else {
        a.w[0] = *reinterpret_cast<const uint4*>(lo);
        b.w[0] = *reinterpret_cast<const uint4*>(hi);
    }
}
template <bool WIDE, bool NEXT>
__device__ __forceinline__ void load_chunks(const float* lo, const float* hi, Chunk<float>& a, Chunk<float>& b)
{
    load_32b<WIDE>(lo, a.w);
    load_32b<WIDE>(hi, b.w);
}
template <bool WIDE, bool NEXT>
__device__ __forceinline__ void store_chunks(__nv_bfloat16* lo, __nv_bfloat16* hi,
                                             const Chunk<__nv_bfloat16>& a, const Chunk<__nv_bfloat16>& b)
{
    if constexpr (NEXT && WIDE) {
        const uint4 w[2] = {a.w[0], b.w[0]};
        store_32b<true>(lo, w);
    } else {
        *reinterpret_cast<uint4*>(lo) = a.w[0];
        *reinterpret_cast<uint4*>(hi) = b.w[0];
    }
}
template <bool WIDE, bool NEXT>
__device__ __forceinline__ void store_chunks(float* lo, float* hi, const Chunk<float>& a, const Chunk<float>& b)
{
    store_32b<WIDE>(lo, a.w);
    store_32b<WIDE>(hi, b.w);
}

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;  // head steps whose loads are in flight together

}  // namespace

template <class T, int D, bool INTERLEAVED, bool WIDE>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int C = D / 16;     // lanes of a head, 8 pairs (16 elements) each
    constexpr int HS = 32 / C;    // heads per step of a warp
    constexpr int PP = 8 / HS;    // angles a lane computes
    const int lane = threadIdx.x & 31;
    const int c = lane % C, hs = lane / C;
    // The lane's pairs of the table.  Read through a generic address: as constants, with another index in
    // every lane, they took a third of a small call (8 tokens: 3.0 us instead of 1.8).
    const unsigned long long* turns = p.turn;
    const unsigned char* axes = p.axis;
    asm volatile("" : "+l"(turns), "+l"(axes));
    unsigned long long turn[PP];
    int axis[PP];
#pragma unroll
    for (int e = 0; e < PP; ++e) {
        const int pr = 8 * c + hs * PP + e;
        turn[e] = pr < p.pairs ? turns[pr] : 0;
        axis[e] = pr < p.pairs ? axes[pr] : 0;
    }
    dependent_begin();
    const unsigned w = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);  // (total may be 2^31 - 1)
    const int tok = p.parts(static_cast<int>(w)), part = static_cast<int>(w - tok * static_cast<unsigned>(p.parts.d));
    if (static_cast<unsigned>(tok) >= static_cast<unsigned>(p.total)) return;
    // lo, hi: the lane's two 8-element chunks of a head
    const bool turned = 8 * c < p.pairs;
    int lo, hi;
    if (INTERLEAVED || !turned) {
        lo = INTERLEAVED ? 16 * c : 2 * p.pairs + 16 * (c - p.pairs / 8);
        hi = lo + 8;
    } else {
        lo = 8 * c;
        hi = p.pairs + 8 * c;
    }
    const int heads = p.H + p.Hkv;
    const int steps = (heads + HS - 1) / HS;
    const int s0 = part * p.per, s1 = min(s0 + p.per, steps);
    float sn[8], cs[8];
    for (int s = s0; s < s1; s += kRopeUnroll) {
        Chunk<T> a[kRopeUnroll], b[kRopeUnroll];
        bool on[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int h = (s + u) * HS + hs;
            on[u] = s + u < s1 && h < heads;
            if (on[u]) {
                const int z = h >= p.H;
                const long long off = tok * p.x_rs[z] + (h - (z ? p.H : 0)) * p.x_hs[z];
                on[u] = in_extent(off, D, p.x_ext[z], p.status);
                const T* src = static_cast<const T*>(p.x[z]) + off;
                if (on[u]) load_chunks<WIDE, INTERLEAVED>(src + lo, src + hi, a[u], b[u]);
            }
        }
        if (s == s0) {  // the angles, while the first heads are on their way
            float ms[PP], mc[PP];
#pragma unroll
            for (int e = 0; e < PP; ++e) {
                ms[e] = 0.0f;
                mc[e] = 1.0f;
                const long long at = static_cast<long long>(axis[e]) * p.total + tok;
                if (in_extent(at, 1, p.pos_ext, p.status)) {
                    const unsigned long long t =
                        static_cast<unsigned long long>(static_cast<long long>(p.pos[at])) * turn[e];
                    turn_sincos(static_cast<uint32_t>((t + 0x80000000ull) >> 32), ms[e], mc[e]);
                    ms[e] *= p.sign;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sn[j] = __shfl_sync(0xffffffffu, ms[j % PP], c + C * (j / PP));
                cs[j] = __shfl_sync(0xffffffffu, mc[j % PP], c + C * (j / PP));
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (!on[u]) continue;
            const int h = (s + u) * HS + hs;
            const int z = h >= p.H;
            if (turned) {
                float x[8], y[8];
                a[u].get(x);
                b[u].get(y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // pair j: (x[j], y[j]), or neighbours within the 16 elements
                    float& x1 = INTERLEAVED ? (j < 4 ? x[2 * j] : y[2 * j - 8]) : x[j];
                    float& x2 = INTERLEAVED ? (j < 4 ? x[2 * j + 1] : y[2 * j - 7]) : y[j];
                    const float r1 = fmaf(x1, cs[j], -(x2 * sn[j]));
                    const float r2 = fmaf(x2, cs[j], x1 * sn[j]);
                    x1 = r1;
                    x2 = r2;
                }
                a[u].put(x);
                b[u].put(y);
            }
            const long long off = tok * p.y_rs[z] + (h - (z ? p.H : 0)) * p.y_hs[z];
            if (!in_extent(off, D, p.y_ext[z], p.status)) continue;
            T* dst = static_cast<T*>(p.y[z]) + off;
            store_chunks<WIDE, INTERLEAVED>(dst + lo, dst + hi, a[u], b[u]);
        }
    }
}

// p.parts and p.per are chosen here: enough warps to fill the SMs when the tokens are few.
template <class T, int D>
static cudaError_t launch_rope_impl(RopeParams p, int interleaved, cudaStream_t st, int num_sms)
{
    constexpr int HS = 32 / (D / 16);
    const int steps = (p.H + p.Hkv + HS - 1) / HS;
    const int want = (num_sms * 16 + p.total - 1) / p.total;
    const int parts = want < 1 ? 1 : (want > steps ? steps : want);
    p.per = (steps + parts - 1) / parts;
    p.parts = FastDiv((steps + p.per - 1) / p.per);  // (tokens * parts^2 < 2^32 where parts > 1)
    const long long warps = static_cast<long long>(p.total) * p.parts.d;
    const dim3 grid(static_cast<unsigned>((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32)));
    // 32-byte accesses where every row allows them; bf16 halves that lie apart are 16 bytes anyway
    bool wide = interleaved || sizeof(T) == 4;
    for (int z = 0; z < 2; ++z)
        wide = wide && wide_rows(p.x[z], p.x_rs[z], p.x_hs[z], sizeof(T)) &&
               wide_rows(p.y[z], p.y_rs[z], p.y_hs[z], sizeof(T));
    const dim3 block(kRopeThreads);
    if (interleaved)
        return wide ? launch_dependent(fa_rope_kernel<T, D, true, true>, grid, block, 0, st, p)
                    : launch_dependent(fa_rope_kernel<T, D, true, false>, grid, block, 0, st, p);
    if (sizeof(T) == 4 && wide)
        return launch_dependent(fa_rope_kernel<T, D, false, sizeof(T) == 4>, grid, block, 0, st, p);
    return launch_dependent(fa_rope_kernel<T, D, false, false>, grid, block, 0, st, p);
}

cudaError_t launch_rope(int d, int is_f32, const RopeParams& p, int interleaved, cudaStream_t st,
                        int num_sms)
{
    if (d == 64)
        return is_f32 ? launch_rope_impl<float, 64>(p, interleaved, st, num_sms)
                      : launch_rope_impl<__nv_bfloat16, 64>(p, interleaved, st, num_sms);
    return is_f32 ? launch_rope_impl<float, 128>(p, interleaved, st, num_sms)
                  : launch_rope_impl<__nv_bfloat16, 128>(p, interleaved, st, num_sms);
}

}  // namespace fa
