// Host side of the C ABI declared in include/fa.h: argument validation (before any CUDA
// call), TMA tensor-map construction, kernel dispatch and the device status word.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "fa_common.cuh"
#include "fa_decode.cuh"
#include "fa_serve.cuh"

namespace fa {
cudaError_t launch_fwd_tc(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, const FwdParams& p, cudaStream_t st);
cudaError_t launch_fwd_simt(int d, int is_f32, const FwdParams& p, cudaStream_t st,
                            int num_sms);
cudaError_t launch_bwd_preprocess(int d, int is_f32, const BwdParams& p, cudaStream_t st,
                                  int num_sms);
cudaError_t launch_bwd_simt(int d, int is_f32, const BwdParams& p, cudaStream_t st);
// maps: [0] q, [1] k, [2] v, [3] dout (bf16, 128-row boxes)
cudaError_t launch_bwd_dkv_tc(int d, const CUtensorMap* maps, const BwdParams& p, cudaStream_t st);
cudaError_t launch_bwd_dq_tc(int d, const CUtensorMap* maps, const BwdParams& p, cudaStream_t st,
                             bool after_dkv);
cudaError_t launch_decode(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, const DecodeParams& p, cudaStream_t st,
                          int num_sms);
cudaError_t launch_fwd_fp8_tc(const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tvt, const FwdParams& p, cudaStream_t st);
cudaError_t launch_vt_transpose(const void* v, void* vt, const Layout& L, int Kpad, int* status,
                                cudaStream_t st);
cudaError_t launch_rope(int d, int is_f32, const RopeParams& p, int interleaved, cudaStream_t st,
                        int num_sms);
cudaError_t launch_cache_append(int d, int is_f32, const CacheParams& p, cudaStream_t st, int num_sms);
cudaError_t launch_cache_read(int d, int is_f32, const CacheParams& p, cudaStream_t st);
cudaError_t launch_decode_cache(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheDecodeParams& p, cudaStream_t st);
cudaError_t launch_cache_copy(int d, const PageCopyParams& p, cudaStream_t st);
cudaError_t launch_cache_compact(int d, const CompactParams& p, cudaStream_t st, int num_sms);
cudaError_t launch_pages_update(PagesParams p, cudaStream_t st, int debug_flags);
cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t st);
cudaError_t launch_decode_tree(int d, const TreeDecodeParams& p, cudaStream_t st);
cudaError_t launch_decode_shared(int d, const CUtensorMap* maps, const SharedDecodeParams& p,
                                 cudaStream_t st, int num_sms);

// Device status word written by bounded waits that give up (0 = fine).
__device__ int g_status_word;
}  // namespace fa

namespace {

thread_local std::string t_last_error;
unsigned long long g_wait_limit_ns = 2000000000ull;
int g_debug_flags = 0;

int fail(int code, const std::string& what)
{
    t_last_error = what;
    return code;
}

int cuda_fail(cudaError_t e, const char* where)
{
    return fail(FA_ERR_LAUNCH, std::string(where) + ": " + cudaGetErrorString(e));
}

struct DeviceInfo {
    bool ready = false;
    int major = 0, minor = 0, sms = 0;
    int* status = nullptr;
};
std::mutex g_mu;
DeviceInfo g_dev[64];

int device_info(DeviceInfo** out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return fail(FA_ERR_LAUNCH, "device index out of range");
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceInfo& di = g_dev[dev];
    if (!di.ready) {
        if ((e = cudaDeviceGetAttribute(&di.major, cudaDevAttrComputeCapabilityMajor, dev)) ||
            (e = cudaDeviceGetAttribute(&di.minor, cudaDevAttrComputeCapabilityMinor, dev)) ||
            (e = cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev)))
            return cuda_fail(e, "cudaDeviceGetAttribute");
        if (di.major != 10 || di.minor != 3)
            return fail(FA_ERR_UNSUPPORTED_DEVICE,
                        "this build targets sm_103a (compute capability 10.3) only");
        void* ptr = nullptr;
        if ((e = cudaGetSymbolAddress(&ptr, fa::g_status_word)) != cudaSuccess)
            return cuda_fail(e, "cudaGetSymbolAddress(status)");
        di.status = static_cast<int*>(ptr);
        di.ready = true;
    }
    *out = &di;
    return FA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int get_encoder()
{
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_encode) return FA_OK;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
        return fail(FA_ERR_LAUNCH, "cuTensorMapEncodeTiled entry point not available");
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return FA_OK;
}

// 3-D view of a bf16 tensor for 128-row tiles of one head; box = 64 columns (one 128-byte
// swizzle panel) x `rows` rows x 1 head.  Fixed layout [heads, R, d]: dimensions (d, R, heads);
// packed layout [R, heads, d] (token by token): dimensions (d, heads, R).  Rows beyond R read
// as zero.
// rs, hs: element strides of a row and of a head index.
int make_map(CUtensorMap* m, const void* base, long long heads, long long R, int d, int rows,
             bool packed, long long rs, long long hs)
{
    const cuuint64_t dd = static_cast<cuuint64_t>(d);
    const cuuint64_t nh = static_cast<cuuint64_t>(heads), nr = static_cast<cuuint64_t>(R);
    cuuint64_t dims[3] = {dd, packed ? nh : nr, packed ? nr : nh};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(packed ? hs : rs) * 2,
                             static_cast<cuuint64_t>(packed ? rs : hs) * 2};
    cuuint32_t box[3] = {64, packed ? 1u : static_cast<cuuint32_t>(rows),
                         packed ? static_cast<cuuint32_t>(rows) : 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(FA_ERR_LAUNCH, "cuTensorMapEncodeTiled failed with code " + std::to_string(r));
    return FA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_common(int B, int H, int N, int d, float scale, int causal, int dtype)
{
    if (dtype != FA_BF16 && dtype != FA_F32) return fail(FA_ERR_INVALID_ARG, "dtype must be FA_BF16 or FA_F32");
    if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1");
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED_D, "d must be 64 or 128");
    if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
        return fail(FA_ERR_INVALID_ARG, "scale must be finite");
    const long long elems = static_cast<long long>(B) * H * N * d;
    if (elems >= (1LL << 31)) return fail(FA_ERR_TOO_LARGE, "B*H*N*d must be < 2^31");
    return FA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The bytes [p, p + n) of one tensor of a call.
struct Span {
    const void* p;
    size_t n;
};

bool spans_meet(const Span& a, const Span& b)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Whether an output shares a byte with another output, an input or the workspace.  The
// backward's kernels overlap in time (dQ runs in the tail of dK/dV), so such a call would race.
bool outputs_overlap(const Span* out, int nout, const Span* in, int nin)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (spans_meet(out[i], out[j])) return true;
        for (int j = 0; j < nin; ++j)
            if (spans_meet(out[i], in[j])) return true;
    }
    return false;
}

const char* const kOverlapMsg =
    "dq, dk and dv must not overlap one another, an input or the workspace";

// Element strides (row, head index) of the eight tensors of a call, in the order
// q, k, v, o, dout, dq, dk, dv.
struct Strides {
    long long rs[8], hs[8];
};
enum { kQ = 0, kK, kV, kO, kDO, kDQ, kDK, kDV };

// The strides the kernels address directly go into the layout; q, k, v, dout go into maps.
// Also sets the element extents that checked builds test accesses against: the smallest
// buffer holding every row of every head index at those strides (R rows of each head index;
// the fixed-length layout's head index runs over B*H, the packed one's over H).  The layout's
// sizes (cu_q, B, H, Hkv, Rq, Rk) must be set first.
void put_strides(fa::Layout& L, const Strides& st, int d)
{
    L.o_rs = st.rs[kO]; L.o_hs = st.hs[kO];
    L.do_rs = st.rs[kDO]; L.do_hs = st.hs[kDO];
    L.dq_rs = st.rs[kDQ]; L.dq_hs = st.hs[kDQ];
    L.dk_rs = st.rs[kDK]; L.dk_hs = st.hs[kDK];
    L.dv_rs = st.rs[kDV]; L.dv_hs = st.hs[kDV];
    const long long bq = L.cu_q ? 1 : L.B;
    const long long hq = bq * L.H, hk = bq * L.Hkv;
    // the watchdog test hook's companion: every extent one row short
    const long long cut = (g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0;
    auto ext = [&](int t, long long heads, long long rows) {
        return rows < 1 ? 0 : (rows - 1) * st.rs[t] + (heads - 1) * st.hs[t] + d - cut * st.rs[t];
    };
    L.o_ext = ext(kO, hq, L.Rq);
    L.do_ext = ext(kDO, hq, L.Rq);
    L.dq_ext = ext(kDQ, hq, L.Rq);
    L.dk_ext = ext(kDK, hk, L.Rk);
    L.dv_ext = ext(kDV, hk, L.Rk);
    L.stat_ext = hq * L.Rq - cut;
}

// Fixed-length entry points: [B, H, N, d] for every tensor, [B, H, N] statistics.
Strides fixed_strides(int N, int d)
{
    Strides st;
    for (int t = 0; t < 8; ++t) {
        st.rs[t] = d;
        st.hs[t] = static_cast<long long>(N) * d;
    }
    return st;
}

fa::Layout fixed_layout(int B, int H, int N, int d)
{
    fa::Layout L{};
    L.cu_q = L.cu_k = nullptr;
    L.B = B; L.H = H; L.Hkv = H;
    L.Nq = L.Nk = N;
    L.Rq = L.Rk = N;
    L.order_group = 1;
    put_strides(L, fixed_strides(N, d), d);
    return L;
}

// Heads per group of the tensor-core kernels' tile order (tile_order): under the causal mask,
// as many heads as keep the rows that one head's tiles stream (K and V, or Q and dO: 4 N d bytes
// in bf16) within 32 MB of L2, at most 16; without the mask every tile costs the same and the
// plain head-major order (1) keeps the fewest heads resident.
int order_group(int N, int d, int causal)
{
    if (!causal) return 1;
    const long long per_head = 4LL * N * d;
    const long long g = (32LL << 20) / (per_head > 0 ? per_head : 1);
    return static_cast<int>(g < 1 ? 1 : (g > 16 ? 16 : g));
}

// The four bf16 maps of the tensor-core kernels: q, k, v, and (backward) dout.
int make_maps(CUtensorMap* maps, const void* q, const void* k, const void* v, const void* dout,
              const fa::Layout& L, int d, const Strides& st)
{
    int rc = get_encoder();
    if (rc) return rc;
    const bool packed = L.cu_q != nullptr;
    const long long nhq = packed ? L.H : static_cast<long long>(L.B) * L.H;
    const long long nhk = packed ? L.Hkv : static_cast<long long>(L.B) * L.Hkv;
    if ((rc = make_map(&maps[0], q, nhq, L.Rq, d, 128, packed, st.rs[kQ], st.hs[kQ])) ||
        (rc = make_map(&maps[1], k, nhk, L.Rk, d, 128, packed, st.rs[kK], st.hs[kK])) ||
        (rc = make_map(&maps[2], v, nhk, L.Rk, d, 128, packed, st.rs[kV], st.hs[kV])))
        return rc;
    if (dout && (rc = make_map(&maps[3], dout, nhq, L.Rq, d, 128, packed, st.rs[kDO],
                               st.hs[kDO])))
        return rc;
    return FA_OK;
}

int fwd_entry(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
              int N, int d, float scale, int causal, int dtype, int impl, void* stream)
{
    int rc = check_common(B, H, N, d, scale, causal, dtype);
    if (rc) return rc;
    if (impl != 0 && impl != 1) return fail(FA_ERR_INVALID_ARG, "impl must be 0 or 1");
    if (!q || !k || !v || !o) return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA_ERR_MISALIGNED, "q, k, v, o must be 16-byte aligned (lse 4-byte)");
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    fa::FwdParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    p.N = N; p.BH = B * H; p.scale = scale; p.scale_log2 = scale * fa::kLog2e;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    p.L = fixed_layout(B, H, N, d);
    p.L.order_group = order_group(N, d, causal);
    cudaError_t e;
    if (dtype == FA_F32 || impl == 1) {
        e = fa::launch_fwd_simt(d, dtype == FA_F32, p, st, di->sms);
    } else {
        CUtensorMap maps[4];
        if ((rc = make_maps(maps, q, k, v, nullptr, p.L, d, fixed_strides(N, d)))) return rc;
        e = fa::launch_fwd_tc(d, maps[0], maps[1], maps[2], p, st);
    }
    if (e != cudaSuccess) return cuda_fail(e, "forward launch");
    return FA_OK;
}

int bwd_entry(const void* q, const void* k, const void* v, const void* o, const void* dout,
              const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
              float scale, int causal, int dtype, void* workspace, size_t workspace_bytes,
              int impl, int stage, void* stream)
{
    int rc = check_common(B, H, N, d, scale, causal, dtype);
    if (rc) return rc;
    if (impl != 0 && impl != 1) return fail(FA_ERR_INVALID_ARG, "impl must be 0 or 1");
    if (stage < -1 || stage > 2) return fail(FA_ERR_INVALID_ARG, "stage must be 0, 1 or 2");
    if (stage >= 0 && (dtype != FA_BF16 || impl != 0))
        return fail(FA_ERR_INVALID_ARG, "staged backward is the bf16 tensor-core path only");
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv)
        return fail(FA_ERR_INVALID_ARG, "every tensor pointer must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(FA_ERR_MISALIGNED, "tensors must be 16-byte aligned (lse 4-byte)");
    const size_t need = fa_bwd_workspace_bytes(B, H, N, d);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    {
        const size_t tb = static_cast<size_t>(B) * H * N * d * (dtype == FA_F32 ? 4 : 2);
        const size_t sb = static_cast<size_t>(B) * H * N * 4;
        const Span outs[3] = {{dq, tb}, {dk, tb}, {dv, tb}};
        const Span ins[7] = {{q, tb}, {k, tb}, {v, tb}, {o, tb}, {dout, tb}, {lse, sb},
                             {workspace, need}};
        if (outputs_overlap(outs, 3, ins, 7)) return fail(FA_ERR_INVALID_ARG, kOverlapMsg);
    }
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    fa::BwdParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.dout = dout; p.lse = lse;
    p.dq = dq; p.dk = dk; p.dv = dv;
    const size_t rows = static_cast<size_t>(B) * H * N;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.delta = reinterpret_cast<float*>(ws);
    p.lse2 = reinterpret_cast<float*>(ws + align256(rows * 4));
    p.N = N; p.BH = B * H; p.scale = scale; p.scale_log2 = scale * fa::kLog2e;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    p.L = fixed_layout(B, H, N, d);
    p.L.order_group = order_group(N, d, causal);
    const int is_f32 = dtype == FA_F32;
    cudaError_t e = cudaSuccess;
    if (stage <= 0) {
        e = fa::launch_bwd_preprocess(d, is_f32, p, st, di->sms);
        if (e != cudaSuccess) return cuda_fail(e, "backward preprocess launch");
        if (stage == 0) return FA_OK;
    }
    if (is_f32 || impl == 1) {
        e = fa::launch_bwd_simt(d, is_f32, p, st);
    } else {
        // maps: q, k, v, dout (all 128-row boxes)
        CUtensorMap maps[4];
        if ((rc = make_maps(maps, q, k, v, dout, p.L, d, fixed_strides(N, d)))) return rc;
        if (stage < 0 || stage == 1) e = fa::launch_bwd_dkv_tc(d, maps, p, st);
        if (e == cudaSuccess && (stage < 0 || stage == 2)) e = fa::launch_bwd_dq_tc(d, maps, p, st, stage < 0);
    }
    if (e != cudaSuccess) return cuda_fail(e, "backward launch");
    return FA_OK;
}

}  // namespace

extern "C" {

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
           int d, float scale, int causal, int dtype, void* stream)
{
    return fwd_entry(q, k, v, o, lse, B, H, N, d, scale, causal, dtype, 0, stream);
}

int fa_fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                int N, int d, float scale, int causal, int dtype, int impl, void* stream)
{
    return fwd_entry(q, k, v, o, lse, B, H, N, d, scale, causal, dtype, impl, stream);
}

size_t fa_bwd_workspace_bytes(int B, int H, int N, int d)
{
    if (B < 1 || H < 1 || N < 1 || (d != 64 && d != 128)) return 0;
    const size_t rows = static_cast<size_t>(B) * H * N;
    return 2 * align256(rows * 4) + 256;
}

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
           const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
           float scale, int causal, int dtype, void* workspace, size_t workspace_bytes,
           void* stream)
{
    return bwd_entry(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, dtype,
                     workspace, workspace_bytes, 0, -1, stream);
}

int fa_bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* dout,
                const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                float scale, int causal, int dtype, void* workspace, size_t workspace_bytes,
                int impl, void* stream)
{
    return bwd_entry(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, dtype,
                     workspace, workspace_bytes, impl, -1, stream);
}

int fa_bwd_stage(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                 float scale, int causal, int dtype, void* workspace, size_t workspace_bytes,
                 int stage, void* stream)
{
    if (stage < 0 || stage > 2) return fail(FA_ERR_INVALID_ARG, "stage must be 0, 1 or 2");
    return bwd_entry(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, dtype,
                     workspace, workspace_bytes, 0, stage, stream);
}

int fa_device_status(void* stream)
{
    DeviceInfo* di = nullptr;
    int rc = device_info(&di);
    if (rc) return rc;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    int word = 0;
    if ((e = cudaMemcpy(&word, di->status, sizeof(int), cudaMemcpyDeviceToHost)) != cudaSuccess)
        return cuda_fail(e, "reading the status word");
    if (word == 0) return FA_OK;
    const int zero = 0;
    if ((e = cudaMemcpy(di->status, &zero, sizeof(int), cudaMemcpyHostToDevice)) != cudaSuccess)
        return cuda_fail(e, "clearing the status word");
    if (word == fa::kStatusOutOfBounds)
        return fail(FA_ERR_OUT_OF_BOUNDS, "a bounds check failed; the access was skipped");
    return fail(FA_ERR_DEVICE_TIMEOUT, "bounded device wait expired at site " + std::to_string(word));
}

void fa_set_wait_limit_ns(unsigned long long ns)
{
    g_wait_limit_ns = ns < 1000000ull ? 1000000ull : ns;
}

void fa_debug_set_flags(int flags) { g_debug_flags = flags; }

int fa_checked_build(void)
{
#ifdef FA_CHECKED
    return 1;
#else
    return 0;
#endif
}

const char* fa_status_string(int code)
{
    switch (code) {
        case FA_OK: return "FA_OK";
        case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
        case FA_ERR_UNSUPPORTED_D: return "FA_ERR_UNSUPPORTED_D";
        case FA_ERR_MISALIGNED: return "FA_ERR_MISALIGNED";
        case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
        case FA_ERR_LAUNCH: return "FA_ERR_LAUNCH";
        case FA_ERR_DEVICE_TIMEOUT: return "FA_ERR_DEVICE_TIMEOUT";
        case FA_ERR_TOO_LARGE: return "FA_ERR_TOO_LARGE";
        case FA_ERR_UNSUPPORTED_DEVICE: return "FA_ERR_UNSUPPORTED_DEVICE";
        case FA_ERR_OUT_OF_BOUNDS: return "FA_ERR_OUT_OF_BOUNDS";
        default: return "FA_ERR_UNKNOWN";
    }
}

const char* fa_last_error(void) { return t_last_error.c_str(); }

int fa_causal_block_counts(int q_block, int Br, int Bc, int N, int* n_full, int* n_masked)
{
    if (q_block < 0 || Br < 1 || Bc < 1 || N < 1 || !n_full || !n_masked ||
        static_cast<long long>(q_block) * Br >= N)
        return fail(FA_ERR_INVALID_ARG, "bad block arguments");
    const int q0 = q_block * Br, q1 = (q0 + Br < N) ? q0 + Br : N;
    int nf = 0, nm = 0;
    for (int k0 = 0; k0 < N; k0 += Bc) {
        const int k1 = (k0 + Bc < N) ? k0 + Bc : N;
        const int c = fa::causal_tile_class(q0, q1, k0, k1);
        nf += c == fa::kTileFull;
        nm += c == fa::kTileMasked;
    }
    *n_full = nf;
    *n_masked = nm;
    return FA_OK;
}

int fa_tile_order(int id, int heads, int nblk, int gsize, int* head, int* rank)
{
    if (heads < 1 || nblk < 1 || gsize < 1 || id < 0 ||
        static_cast<long long>(id) >= static_cast<long long>(heads) * nblk || !head || !rank)
        return fail(FA_ERR_INVALID_ARG, "bad tile-order arguments");
    fa::tile_order(id, heads, nblk, gsize, *head, *rank);
    return FA_OK;
}

int fa_order_group(int N, int d, int causal) { return order_group(N, d, causal); }

const char* fa_version(void) { return "fa-gb300 0.1 (sm_103a)"; }

}  // extern "C"

// ---------------------------------------------------------------------------------------
// Fixed-length batches with grouped key/value heads and Nq != Nk (fa_fwd_gqa, fa_bwd_gqa).
// ---------------------------------------------------------------------------------------
namespace {

int check_gqa(int B, int H, int Hkv, int Nq, int Nk, int d, float scale, int causal)
{
    if (B < 1 || H < 1 || Hkv < 1 || Nq < 1 || Nk < 1)
        return fail(FA_ERR_INVALID_ARG, "B, H, Hkv, Nq and Nk must be >= 1");
    if (H % Hkv != 0) return fail(FA_ERR_INVALID_ARG, "H must be a multiple of Hkv");
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED_D, "d must be 64 or 128");
    if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
        return fail(FA_ERR_INVALID_ARG, "scale must be finite");
    if (static_cast<long long>(B) * H * Nq * d >= (1LL << 31) ||
        static_cast<long long>(B) * Hkv * Nk * d >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "B*H*Nq*d and B*Hkv*Nk*d must be < 2^31");
    return FA_OK;
}

// [B, H, Nq, d] queries, [B, Hkv, Nk, d] keys and values, [B, H, Nq] statistics.
fa::Layout gqa_layout(int B, int H, int Hkv, int Nq, int Nk, int d, Strides* st)
{
    for (int t = 0; t < 8; ++t) {
        const bool kside = t == kK || t == kV || t == kDK || t == kDV;
        st->rs[t] = d;
        st->hs[t] = static_cast<long long>(kside ? Nk : Nq) * d;
    }
    fa::Layout L{};
    L.cu_q = L.cu_k = nullptr;
    L.B = B; L.H = H; L.Hkv = Hkv;
    L.Nq = Nq; L.Nk = Nk;
    L.Rq = Nq; L.Rk = Nk;
    L.order_group = 1;
    put_strides(L, *st, d);
    return L;
}

}  // namespace

extern "C" int fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                          int B, int H, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                          void* stream)
{
    int rc = check_gqa(B, H, Hkv, Nq, Nk, d, scale, causal);
    if (rc) return rc;
    if (!q || !k || !v || !o) return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA_ERR_MISALIGNED, "q, k, v, o must be 16-byte aligned (lse 4-byte)");
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    fa::FwdParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    p.N = Nq; p.BH = B * H; p.scale = scale; p.scale_log2 = scale * fa::kLog2e;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    Strides st;
    p.L = gqa_layout(B, H, Hkv, Nq, Nk, d, &st);
    p.L.order_group = order_group(Nk, d, causal);
    CUtensorMap maps[4];
    if ((rc = make_maps(maps, q, k, v, nullptr, p.L, d, st))) return rc;
    cudaError_t e = fa::launch_fwd_tc(d, maps[0], maps[1], maps[2], p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "forward launch");
    return FA_OK;
}

extern "C" int fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o,
                          const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                          int H, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                          void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_gqa(B, H, Hkv, Nq, Nk, d, scale, causal);
    if (rc) return rc;
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv)
        return fail(FA_ERR_INVALID_ARG, "every tensor pointer must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(FA_ERR_MISALIGNED, "tensors must be 16-byte aligned (lse 4-byte)");
    const size_t need = fa_bwd_workspace_bytes(B, H, Nq, d);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    {
        const size_t tq = static_cast<size_t>(B) * H * Nq * d * 2;
        const size_t tk = static_cast<size_t>(B) * Hkv * Nk * d * 2;
        const size_t sb = static_cast<size_t>(B) * H * Nq * 4;
        const Span outs[3] = {{dq, tq}, {dk, tk}, {dv, tk}};
        const Span ins[7] = {{q, tq}, {k, tk}, {v, tk}, {o, tq}, {dout, tq}, {lse, sb},
                             {workspace, need}};
        if (outputs_overlap(outs, 3, ins, 7)) return fail(FA_ERR_INVALID_ARG, kOverlapMsg);
    }
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    fa::BwdParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.dout = dout; p.lse = lse;
    p.dq = dq; p.dk = dk; p.dv = dv;
    const size_t rows = static_cast<size_t>(B) * H * Nq;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.delta = reinterpret_cast<float*>(ws);
    p.lse2 = reinterpret_cast<float*>(ws + align256(rows * 4));
    p.N = Nq; p.BH = B * H; p.scale = scale; p.scale_log2 = scale * fa::kLog2e;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    Strides st;
    p.L = gqa_layout(B, H, Hkv, Nq, Nk, d, &st);
    p.L.order_group = order_group(Nk, d, causal);
    CUtensorMap maps[4];
    if ((rc = make_maps(maps, q, k, v, dout, p.L, d, st))) return rc;
    cudaError_t e = fa::launch_bwd_preprocess(d, 0, p, cs, di->sms);
    if (e == cudaSuccess) e = fa::launch_bwd_dkv_tc(d, maps, p, cs);
    if (e == cudaSuccess) e = fa::launch_bwd_dq_tc(d, maps, p, cs, true);
    if (e != cudaSuccess) return cuda_fail(e, "backward launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// Packed variable-length batches with grouped key/value heads (fa_fwd_varlen, fa_bwd_varlen).
// ---------------------------------------------------------------------------------------
namespace {

int check_varlen(const int* cu_q, const int* cu_k, int B, int* max_q, int* max_k, int total_q,
                 int total_k, int H, int Hkv, int d, float scale, int causal)
{
    if (B < 1 || H < 1 || Hkv < 1) return fail(FA_ERR_INVALID_ARG, "B, H and Hkv must be >= 1");
    if (H % Hkv != 0) return fail(FA_ERR_INVALID_ARG, "H must be a multiple of Hkv");
    if (total_q < 1 || total_k < 1 || *max_q < 1 || *max_k < 1)
        return fail(FA_ERR_INVALID_ARG, "total_q, total_k, max_seqlen_q and max_seqlen_k must be >= 1");
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED_D, "d must be 64 or 128");
    if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
        return fail(FA_ERR_INVALID_ARG, "scale must be finite");
    if (!cu_q || !cu_k) return fail(FA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k must be non-null");
    if ((reinterpret_cast<uintptr_t>(cu_q) & 3u) || (reinterpret_cast<uintptr_t>(cu_k) & 3u))
        return fail(FA_ERR_MISALIGNED, "cu_seqlens_q and cu_seqlens_k must be 4-byte aligned");
    if (static_cast<long long>(total_q) * H * d >= (1LL << 31) ||
        static_cast<long long>(total_k) * Hkv * d >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "total_q*H*d and total_k*Hkv*d must be < 2^31");
    // no sequence is longer than its packed tensor
    if (*max_q > total_q) *max_q = total_q;
    if (*max_k > total_k) *max_k = total_k;
    if (static_cast<long long>(B) * H * ((*max_q + 127) / 128) >= (1LL << 31) ||
        static_cast<long long>(B) * Hkv * ((*max_k + 127) / 128) >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "B*H*ceil(max_seqlen/128) must be < 2^31");
    return FA_OK;
}

// Contiguous packed tensors: q-side [total_q, H, d], k-side [total_k, Hkv, d].
Strides packed_strides(int H, int Hkv, int d)
{
    Strides st;
    for (int t = 0; t < 8; ++t) {
        const bool kside = t == kK || t == kV || t == kDK || t == kDV;
        st.rs[t] = static_cast<long long>(kside ? Hkv : H) * d;
        st.hs[t] = d;
    }
    return st;
}

// Caller strides: `n` (row, head) pairs in the order q, k, v, o[, dout, dq, dk, dv].  Each must
// be positive and a multiple of 8 elements (16 bytes, for the tensor maps and the 16-byte
// stores), and a head must not be wider than its row step (tensors stored token by token).
int read_strides(const long long* user, int n, int H, int Hkv, int d, Strides* st)
{
    *st = packed_strides(H, Hkv, d);
    if (!user) return fail(FA_ERR_INVALID_ARG, "strides must be non-null");
    for (int t = 0; t < n; ++t) {
        const long long rs = user[2 * t], hs = user[2 * t + 1];
        if (rs <= 0 || hs <= 0 || (rs % 8) || (hs % 8))
            return fail(FA_ERR_MISALIGNED, "strides must be positive multiples of 8 elements");
        if (hs < d || rs < hs)
            return fail(FA_ERR_INVALID_ARG, "each head's d elements must fit within its head step, "
                                            "and the head step within the row step");
        st->rs[t] = rs;
        st->hs[t] = hs;
    }
    return FA_OK;
}

fa::Layout packed_layout(const int* cu_q, const int* cu_k, int B, int max_q, int max_k,
                         int total_q, int total_k, int H, int Hkv, int d, const Strides& st)
{
    fa::Layout L{};
    L.cu_q = cu_q; L.cu_k = cu_k;
    L.B = B; L.H = H; L.Hkv = Hkv;
    L.Nq = max_q; L.Nk = max_k;
    L.Rq = total_q; L.Rk = total_k;
    L.order_group = 1;  // sequences of different lengths: head-major
    put_strides(L, st, d);
    return L;
}

int fwd_varlen_entry(const void* q, const void* k, const void* v, void* o, float* lse,
                     const int* cu_q, const int* cu_k, int B, int max_q, int max_k, int total_q,
                     int total_k, int H, int Hkv, int d, float scale, int causal,
                     const long long* user_strides, void* stream)
{
    int rc = check_varlen(cu_q, cu_k, B, &max_q, &max_k, total_q, total_k, H, Hkv, d, scale,
                          causal);
    if (rc) return rc;
    if (!q || !k || !v || !o) return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA_ERR_MISALIGNED, "q, k, v, o must be 16-byte aligned (lse 4-byte)");
    Strides st = packed_strides(H, Hkv, d);
    if (user_strides && (rc = read_strides(user_strides, 4, H, Hkv, d, &st))) return rc;
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    fa::FwdParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    p.N = total_q; p.BH = H; p.scale = scale; p.scale_log2 = scale * fa::kLog2e;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    p.L = packed_layout(cu_q, cu_k, B, max_q, max_k, total_q, total_k, H, Hkv, d, st);
    CUtensorMap maps[4];
    if ((rc = make_maps(maps, q, k, v, nullptr, p.L, d, st))) return rc;
    cudaError_t e = fa::launch_fwd_tc(d, maps[0], maps[1], maps[2], p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "forward launch");
    return FA_OK;
}

int bwd_varlen_entry(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, const int* cu_q,
                     const int* cu_k, int B, int max_q, int max_k, int total_q, int total_k,
                     int H, int Hkv, int d, float scale, int causal,
                     const long long* user_strides, void* workspace, size_t workspace_bytes,
                     void* stream)
{
    int rc = check_varlen(cu_q, cu_k, B, &max_q, &max_k, total_q, total_k, H, Hkv, d, scale,
                          causal);
    if (rc) return rc;
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv)
        return fail(FA_ERR_INVALID_ARG, "every tensor pointer must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(FA_ERR_MISALIGNED, "tensors must be 16-byte aligned (lse 4-byte)");
    Strides st = packed_strides(H, Hkv, d);
    if (user_strides && (rc = read_strides(user_strides, 8, H, Hkv, d, &st))) return rc;
    const size_t need = fa_bwd_varlen_workspace_bytes(total_q, H, d);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if (!user_strides) {  // (strided views may interleave in one buffer: not checked)
        const size_t tq = static_cast<size_t>(total_q) * H * d * 2;
        const size_t tk = static_cast<size_t>(total_k) * Hkv * d * 2;
        const size_t sb = static_cast<size_t>(total_q) * H * 4;
        const Span outs[3] = {{dq, tq}, {dk, tk}, {dv, tk}};
        const Span ins[7] = {{q, tq}, {k, tk}, {v, tk}, {o, tq}, {dout, tq}, {lse, sb},
                             {workspace, need}};
        if (outputs_overlap(outs, 3, ins, 7)) return fail(FA_ERR_INVALID_ARG, kOverlapMsg);
    }
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    fa::BwdParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.dout = dout; p.lse = lse;
    p.dq = dq; p.dk = dk; p.dv = dv;
    const size_t rows = static_cast<size_t>(H) * total_q;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.delta = reinterpret_cast<float*>(ws);
    p.lse2 = reinterpret_cast<float*>(ws + align256(rows * 4));
    p.N = total_q; p.BH = H; p.scale = scale; p.scale_log2 = scale * fa::kLog2e;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    p.L = packed_layout(cu_q, cu_k, B, max_q, max_k, total_q, total_k, H, Hkv, d, st);
    CUtensorMap maps[4];
    if ((rc = make_maps(maps, q, k, v, dout, p.L, d, st))) return rc;
    cudaError_t e = fa::launch_bwd_preprocess(d, 0, p, cs, di->sms);
    if (e == cudaSuccess) e = fa::launch_bwd_dkv_tc(d, maps, p, cs);
    if (e == cudaSuccess) e = fa::launch_bwd_dq_tc(d, maps, p, cs, true);
    if (e != cudaSuccess) return cuda_fail(e, "backward launch");
    return FA_OK;
}

}  // namespace

extern "C" int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int* cu_seqlens_q, const int* cu_seqlens_k, int B,
                             int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int H,
                             int Hkv, int d, float scale, int causal, void* stream)
{
    return fwd_varlen_entry(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, max_seqlen_q,
                            max_seqlen_k, total_q, total_k, H, Hkv, d, scale, causal, nullptr,
                            stream);
}

extern "C" int fa_fwd_varlen_strided(const void* q, const void* k, const void* v, void* o,
                                     float* lse, const long long* strides,
                                     const int* cu_seqlens_q, const int* cu_seqlens_k, int B,
                                     int max_seqlen_q, int max_seqlen_k, int total_q,
                                     int total_k, int H, int Hkv, int d, float scale, int causal,
                                     void* stream)
{
    if (!strides) return fail(FA_ERR_INVALID_ARG, "strides must be non-null");
    return fwd_varlen_entry(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, max_seqlen_q,
                            max_seqlen_k, total_q, total_k, H, Hkv, d, scale, causal, strides,
                            stream);
}

extern "C" size_t fa_bwd_varlen_workspace_bytes(int total_q, int H, int d)
{
    if (total_q < 1 || H < 1 || (d != 64 && d != 128)) return 0;
    const size_t rows = static_cast<size_t>(H) * total_q;
    return 2 * align256(rows * 4) + 256;
}

extern "C" int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                             const void* dout, const float* lse, void* dq, void* dk, void* dv,
                             const int* cu_seqlens_q, const int* cu_seqlens_k, int B,
                             int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int H,
                             int Hkv, int d, float scale, int causal, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    return bwd_varlen_entry(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, B,
                            max_seqlen_q, max_seqlen_k, total_q, total_k, H, Hkv, d, scale,
                            causal, nullptr, workspace, workspace_bytes, stream);
}

extern "C" int fa_bwd_varlen_strided(const void* q, const void* k, const void* v, const void* o,
                                     const void* dout, const float* lse, void* dq, void* dk,
                                     void* dv, const long long* strides, const int* cu_seqlens_q,
                                     const int* cu_seqlens_k, int B, int max_seqlen_q,
                                     int max_seqlen_k, int total_q, int total_k, int H, int Hkv,
                                     int d, float scale, int causal, void* workspace,
                                     size_t workspace_bytes, void* stream)
{
    if (!strides) return fail(FA_ERR_INVALID_ARG, "strides must be non-null");
    return bwd_varlen_entry(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, B,
                            max_seqlen_q, max_seqlen_k, total_q, total_k, H, Hkv, d, scale,
                            causal, strides, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------------------------------
// Split-KV decode (fa_decode_num_splits, fa_decode_workspace_bytes, fa_fwd_decode).
// ---------------------------------------------------------------------------------------
namespace {

constexpr int kDecodeMaxSplits = 256;

// Q of the decode kernels: (d, H, total_q) with a box of (64 columns, G heads, `tokens` tokens),
// so one copy brings the rows of a tile, in (token, head) order; K, V are mapped as fa_fwd_varlen's.
int make_decode_q_map(CUtensorMap* m, const void* q, int H, int total_q, int d, int G, int tokens)
{
    const cuuint64_t dd = static_cast<cuuint64_t>(d);
    cuuint64_t dims[3] = {dd, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(total_q)};
    cuuint64_t strides[2] = {dd * 2, static_cast<cuuint64_t>(H) * dd * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tokens)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                          box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(FA_ERR_LAUNCH, "cuTensorMapEncodeTiled failed with code " + std::to_string(r));
    return FA_OK;
}

size_t decode_part_o_bytes(int total_q, int H, int d, int splits)
{
    return align256(static_cast<size_t>(splits) * total_q * H * d * 4);
}

}  // namespace

extern "C" int fa_decode_splits_for(int B, int Hkv, int max_seqlen_k, int num_sms)
{
    if (B < 1 || Hkv < 1 || max_seqlen_k < 1 || num_sms < 1)
        return fail(FA_ERR_INVALID_ARG, "B, Hkv, max_seqlen_k and num_sms must be >= 1");
    // One wave: the largest split count whose CTAs (B * Hkv * splits, one per SM) all run at
    // once, keeping at least 8 key blocks per split.  Once enough CTAs stream (each keeps about
    // 200 KB of loads in flight), the HBM time is the same for any split count; a second wave
    // costs its CTAs their set-up and pipeline fill again, and every extra range costs the
    // combine a partial result.  Measured on GB300 (B = 8, Hkv = 8, d = 128): 2 splits over
    // 8 K, 16 K and 32 K keys ran 10-18 % faster than the 7-19 that filled whole waves.
    const long long units = static_cast<long long>(B) * Hkv;
    const int nblk = static_cast<int>((static_cast<long long>(max_seqlen_k) + 127) / 128);
    const int smax = std::max(1, std::min(kDecodeMaxSplits, nblk / 8));
    const long long fit = std::max(1LL, static_cast<long long>(num_sms) / units);
    return static_cast<int>(std::min<long long>(smax, fit));
}

extern "C" int fa_decode_num_splits(int B, int Hkv, int max_seqlen_k)
{
    if (B < 1 || Hkv < 1 || max_seqlen_k < 1) return fail(FA_ERR_INVALID_ARG, "B, Hkv and max_seqlen_k must be >= 1");
    DeviceInfo* di = nullptr;
    int rc = device_info(&di);
    if (rc) return rc;
    return fa_decode_splits_for(B, Hkv, max_seqlen_k, di->sms);
}

extern "C" size_t fa_decode_workspace_bytes(int total_q, int H, int d, int num_splits)
{
    if (total_q < 1 || H < 1 || (d != 64 && d != 128) || num_splits < 1 ||
        num_splits > kDecodeMaxSplits)
        return 0;
    if (num_splits == 1) return 0;
    return decode_part_o_bytes(total_q, H, d, num_splits) +
           align256(static_cast<size_t>(num_splits) * H * total_q * 4) + 256;
}

extern "C" int fa_fwd_decode(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int* cu_seqlens_q, const int* cu_seqlens_k, int B,
                             int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int H,
                             int Hkv, int d, float scale, int causal, int num_splits,
                             void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_varlen(cu_seqlens_q, cu_seqlens_k, B, &max_seqlen_q, &max_seqlen_k, total_q,
                          total_k, H, Hkv, d, scale, causal);
    if (rc) return rc;
    // The rows of a CTA are G query heads of a group times max_seqlen_q queries, at most 128:
    // G is the largest divisor of the group size H / Hkv that fits.
    if (max_seqlen_q > 128)
        return fail(FA_ERR_INVALID_ARG, "max_seqlen_q must be <= 128 for the decode kernel; use "
                                        "fa_fwd_varlen");
    const int group = H / Hkv;
    int G = 1;
    for (int g = 1; g <= group; ++g)
        if (group % g == 0 && g * max_seqlen_q <= 128) G = g;
    if (num_splits < 1 || num_splits > kDecodeMaxSplits)
        return fail(FA_ERR_INVALID_ARG, "num_splits must be in [1, " +
                                            std::to_string(kDecodeMaxSplits) + "]");
    if (static_cast<long long>(B) * Hkv * (group / G) * num_splits >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "B * H / G * num_splits must be < 2^31");
    if (!q || !k || !v || !o) return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA_ERR_MISALIGNED, "q, k, v, o must be 16-byte aligned (lse 4-byte)");
    const size_t need = fa_decode_workspace_bytes(total_q, H, d, num_splits);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
        if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    }
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    fa::DecodeParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    if (need > 0) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.o_part = reinterpret_cast<float*>(ws);
        p.lse_part = reinterpret_cast<float*>(ws + decode_part_o_bytes(total_q, H, d, num_splits));
    }
    p.splits = num_splits; p.G = G; p.head_chunks = group / G; p.q_box = max_seqlen_q;
    p.scale_log2 = scale * fa::kLog2e; p.causal = causal;
    p.status = di->status; p.wait_limit_ns = g_wait_limit_ns; p.debug_flags = g_debug_flags;
    p.part_ext = need > 0 ? static_cast<long long>(num_splits) * total_q * H * d -
                                ((g_debug_flags & fa::kDebugShrinkExtents) ? d : 0)
                          : 0;
    const Strides st = packed_strides(H, Hkv, d);
    p.L = packed_layout(cu_seqlens_q, cu_seqlens_k, B, max_seqlen_q, max_seqlen_k, total_q,
                        total_k, H, Hkv, d, st);
    if ((rc = get_encoder())) return rc;
    CUtensorMap maps[4];
    if ((rc = make_decode_q_map(&maps[0], q, H, total_q, d, G, max_seqlen_q))) return rc;
    if ((rc = make_map(&maps[1], k, Hkv, total_k, d, 128, true, st.rs[kK], st.hs[kK])) ||
        (rc = make_map(&maps[2], v, Hkv, total_k, d, 128, true, st.rs[kV], st.hs[kV])))
        return rc;
    cudaError_t e = fa::launch_decode(d, maps[0], maps[1], maps[2], p,
                                      static_cast<cudaStream_t>(stream), di->sms);
    if (e != cudaSuccess) return cuda_fail(e, "decode launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// fa_bwd_noalloc: the backward with its scratch in a fixed device array of this library.
// ---------------------------------------------------------------------------------------
namespace {

constexpr long long kNoallocMaxRows = 1LL << 20;  // largest B*H*N accepted
constexpr size_t kNoallocBytes = 2 * static_cast<size_t>(kNoallocMaxRows) * 4 + 256;

// Delta and the base-2 LSE for up to kNoallocMaxRows rows, in the layout of fa_bwd's
// workspace.  Every device that loads the library holds these 8 MiB until the process exits.
static __device__ __align__(256) unsigned char g_bwd_scratch[kNoallocBytes];

std::mutex g_scratch_mu;
void* g_scratch_dev_ptr[64] = {};

// Device address of g_bwd_scratch on the current device, looked up once per device.  In host
// code the symbol names a host-side shadow, not device memory, so it is never passed as is.
int scratch_address(void** out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return fail(FA_ERR_LAUNCH, "device index out of range");
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (!g_scratch_dev_ptr[dev]) {
        void* ptr = nullptr;
        e = cudaGetSymbolAddress(&ptr, g_bwd_scratch);
        if (e != cudaSuccess || ptr == nullptr)
            return cuda_fail(e, "cudaGetSymbolAddress(backward scratch)");
        g_scratch_dev_ptr[dev] = ptr;
    }
    *out = g_scratch_dev_ptr[dev];
    return FA_OK;
}

}  // namespace

extern "C" int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                              const void* dout, const float* lse, void* dq, void* dk, void* dv,
                              int B, int H, int N, int d, float scale, int causal, int dtype,
                              void* stream)
{
    int rc = check_common(B, H, N, d, scale, causal, dtype);
    if (rc) return rc;
    const long long rows = static_cast<long long>(B) * H * N;
    if (rows > kNoallocMaxRows)
        return fail(FA_ERR_TOO_LARGE, "fa_bwd_noalloc supports B*H*N <= " +
                                          std::to_string(kNoallocMaxRows) + " rows (got " +
                                          std::to_string(rows) + "); use fa_bwd with a workspace");
    void* scratch = nullptr;
    if ((rc = scratch_address(&scratch))) return rc;
    return bwd_entry(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, dtype,
                     scratch, kNoallocBytes, 0, -1, stream);
}

// ---------------------------------------------------------------------------------------
// e4m3 forward
// ---------------------------------------------------------------------------------------
namespace {

long long fp8_pad_keys(int N) { return (static_cast<long long>(N) + 15) / 16 * 16; }

// 3-D map of 8-bit codes, dimensions (x, y, z) with byte strides for y and z; box 128 bytes x
// by_ x bz (128 rows of one 128-byte swizzle panel: by_ = 128, bz = 1, or bz = 128 rows along
// z for tensors stored token by token).
int make_map_u8(CUtensorMap* m, const void* base, cuuint64_t x, cuuint64_t y, cuuint64_t z,
                cuuint64_t y_stride, cuuint64_t z_stride, cuuint32_t by_ = 128, cuuint32_t bz = 1)
{
    cuuint64_t dims[3] = {x, y, z};
    cuuint64_t strides[2] = {y_stride, z_stride};
    cuuint32_t box[3] = {128, by_, bz};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(FA_ERR_LAUNCH, "cuTensorMapEncodeTiled failed with code " + std::to_string(r));
    return FA_OK;
}

bool finite(float x) { return x == x && x != INFINITY && x != -INFINITY; }

}  // namespace

extern "C" size_t fa_fwd_fp8_workspace_bytes(int B, int H, int N, int d)
{
    if (B < 1 || H < 1 || N < 1 || d < 1) return 0;
    return align256(static_cast<size_t>(B) * H * d * static_cast<size_t>(fp8_pad_keys(N)));
}

extern "C" int fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse,
                          int B, int H, int N, int d, float scale, float q_descale,
                          float k_descale, float v_descale, int causal, void* workspace,
                          size_t workspace_bytes, void* stream)
{
    int rc = check_common(B, H, N, d, scale, causal, FA_BF16);
    if (rc) return rc;
    if (d != 128) return fail(FA_ERR_UNSUPPORTED_D, "the e4m3 forward takes d = 128 only");
    if (!finite(q_descale) || !finite(k_descale) || !finite(v_descale) ||
        !finite(scale * q_descale * k_descale))
        return fail(FA_ERR_INVALID_ARG, "descale factors (and their product with scale) must be finite");
    if (!q || !k || !v || !o) return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA_ERR_MISALIGNED, "q, k, v, o must be 16-byte aligned (lse 4-byte)");
    const size_t need = fa_fwd_fp8_workspace_bytes(B, H, N, d);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    if ((rc = get_encoder())) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long Npad = fp8_pad_keys(N);
    const cuuint64_t BH = static_cast<cuuint64_t>(B) * H, n = static_cast<cuuint64_t>(N);
    CUtensorMap maps[3];
    // Q, K: (d, N, B*H) bytes; V^T: (Npad keys, d, B*H)
    if ((rc = make_map_u8(&maps[0], q, 128, n, BH, 128, n * 128)) ||
        (rc = make_map_u8(&maps[1], k, 128, n, BH, 128, n * 128)) ||
        (rc = make_map_u8(&maps[2], workspace, static_cast<cuuint64_t>(Npad), 128, BH,
                          static_cast<cuuint64_t>(Npad), static_cast<cuuint64_t>(Npad) * 128)))
        return rc;
    fa::FwdParams p{};
    p.q = q; p.k = k; p.v = workspace; p.o = o; p.lse = lse;
    p.N = N; p.BH = B * H; p.scale = scale;
    p.scale_log2 = scale * q_descale * k_descale * fa::kLog2e;
    p.v_descale = v_descale;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    p.L = fixed_layout(B, H, N, d);
    p.L.order_group = order_group(N, d, causal);
    cudaError_t e = fa::launch_vt_transpose(v, workspace, p.L, static_cast<int>(Npad), di->status, st);
    if (e != cudaSuccess) return cuda_fail(e, "V transpose launch");
    e = fa::launch_fwd_fp8_tc(maps[0], maps[1], maps[2], p, st);
    if (e != cudaSuccess) return cuda_fail(e, "e4m3 forward launch");
    return FA_OK;
}

extern "C" size_t fa_fwd_fp8_varlen_workspace_bytes(int B, int max_seqlen_k, int Hkv, int d)
{
    if (B < 1 || max_seqlen_k < 1 || Hkv < 1 || d < 1) return 0;
    return align256(static_cast<size_t>(B) * Hkv * d * static_cast<size_t>(fp8_pad_keys(max_seqlen_k)));
}

extern "C" int fa_fwd_fp8_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                                 const int* cu_seqlens_q, const int* cu_seqlens_k, int B,
                                 int max_seqlen_q, int max_seqlen_k, int total_q, int total_k,
                                 int H, int Hkv, int d, float scale, float q_descale,
                                 float k_descale, float v_descale, int causal, void* workspace,
                                 size_t workspace_bytes, void* stream)
{
    int max_q = max_seqlen_q, max_k = max_seqlen_k;
    int rc = check_varlen(cu_seqlens_q, cu_seqlens_k, B, &max_q, &max_k, total_q, total_k, H, Hkv,
                          d, scale, causal);
    if (rc) return rc;
    if (d != 128) return fail(FA_ERR_UNSUPPORTED_D, "the e4m3 forward takes d = 128 only");
    if (!finite(q_descale) || !finite(k_descale) || !finite(v_descale) ||
        !finite(scale * q_descale * k_descale))
        return fail(FA_ERR_INVALID_ARG, "descale factors (and their product with scale) must be finite");
    if (!q || !k || !v || !o) return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be non-null");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA_ERR_MISALIGNED, "q, k, v, o must be 16-byte aligned (lse 4-byte)");
    const long long Kpad = fp8_pad_keys(max_k);
    if (static_cast<long long>(B) * Hkv * ((Kpad + 63) / 64) >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "B * Hkv * ceil(max_seqlen_k / 64) must be < 2^31");
    const size_t need = fa_fwd_fp8_varlen_workspace_bytes(B, max_k, Hkv, d);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    DeviceInfo* di = nullptr;
    if ((rc = device_info(&di))) return rc;
    if ((rc = get_encoder())) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    CUtensorMap maps[3];
    // Q: (d, H, total_q), K: (d, Hkv, total_k) bytes, boxes of 128 tokens of one head;
    // V^T: (Kpad keys, d, B*Hkv)
    const cuuint64_t hq = static_cast<cuuint64_t>(H), hk = static_cast<cuuint64_t>(Hkv);
    if ((rc = make_map_u8(&maps[0], q, 128, hq, static_cast<cuuint64_t>(total_q), 128, hq * 128, 1, 128)) ||
        (rc = make_map_u8(&maps[1], k, 128, hk, static_cast<cuuint64_t>(total_k), 128, hk * 128, 1, 128)) ||
        (rc = make_map_u8(&maps[2], workspace, static_cast<cuuint64_t>(Kpad), 128,
                          static_cast<cuuint64_t>(B) * hk, static_cast<cuuint64_t>(Kpad),
                          static_cast<cuuint64_t>(Kpad) * 128)))
        return rc;
    fa::FwdParams p{};
    p.q = q; p.k = k; p.v = workspace; p.o = o; p.lse = lse;
    p.N = total_q; p.BH = H; p.scale = scale;
    p.scale_log2 = scale * q_descale * k_descale * fa::kLog2e;
    p.v_descale = v_descale;
    p.causal = causal; p.status = di->status; p.wait_limit_ns = g_wait_limit_ns;
    p.debug_flags = g_debug_flags;
    p.L = packed_layout(cu_seqlens_q, cu_seqlens_k, B, max_q, max_k, total_q, total_k, H, Hkv, d,
                        packed_strides(H, Hkv, d));
    cudaError_t e = fa::launch_vt_transpose(v, workspace, p.L, static_cast<int>(Kpad), di->status, st);
    if (e != cudaSuccess) return cuda_fail(e, "V transpose launch");
    e = fa::launch_fwd_fp8_tc(maps[0], maps[1], maps[2], p, st);
    if (e != cudaSuccess) return cuda_fail(e, "e4m3 forward launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// Rotary positions (fa_rope).
// ---------------------------------------------------------------------------------------
namespace {

// Turns per position, x / (2 pi), as a fraction of 2^64 (whole turns dropped).  The product is
// taken in two doubles, so the fraction is good to about 2^-64 turns for |x| < 1.
unsigned long long turn_fraction(double x)
{
    constexpr double kHi = 0.15915494309189535;       // 1 / (2 pi) in two doubles
    constexpr double kLo = -9.839338337591243e-18;
    if (x < 0) return 0ull - turn_fraction(-x);
    const double hi = x * kHi;
    const double lo = __builtin_fma(x, kHi, -hi) + x * kLo;
    const double frac = hi - __builtin_floor(hi);  // exact
    // 2^64 frac as 32 + 32 bits, then the low part (which may be negative: mod 2^64)
    const double top = __builtin_floor(frac * 0x1p32);
    const double rest = (frac * 0x1p32 - top) * 0x1p32 + lo * 0x1p64;
    return (static_cast<unsigned long long>(top) << 32) +
           static_cast<unsigned long long>(static_cast<long long>(__builtin_rint(rest)));
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Row and head strides of packed tensors: contiguous, or `user` (n pairs) checked: positive
// multiples of `unit` elements (16 bytes), heads not wider than their step, rows not shorter
// than a head step.
int packed_or_user_strides(const long long* user, int n, const int* heads, int d, int unit,
                           long long* rs, long long* hs)
{
    for (int t = 0; t < n; ++t) {
        rs[t] = static_cast<long long>(heads[t]) * d;
        hs[t] = d;
        if (!user || heads[t] == 0) continue;
        rs[t] = user[2 * t];
        hs[t] = user[2 * t + 1];
        if (rs[t] <= 0 || hs[t] <= 0 || rs[t] % unit || hs[t] % unit)
            return fail(FA_ERR_MISALIGNED, "strides must be positive multiples of 16 bytes");
        if (hs[t] < d || rs[t] < hs[t])
            return fail(FA_ERR_INVALID_ARG, "each head's d elements must fit within its head step, "
                                            "and the head step within the row step");
    }
    return FA_OK;
}

long long rows_extent(long long rows, int heads, int d, long long rs, long long hs)
{
    const long long cut = (g_debug_flags & fa::kDebugShrinkExtents) ? rs : 0;
    return (rows - 1) * rs + (heads - 1) * hs + d - cut;
}

}  // namespace

extern "C" int fa_rope(const void* q, const void* k, void* q_out, void* k_out,
                       const int* positions, const double* inv_freq, const int* axis,
                       const long long* strides, int total, int H, int Hkv, int d, int axes,
                       int pairs, int interleaved, int inverse, int dtype, void* stream)
{
    if (dtype != FA_BF16 && dtype != FA_F32) return fail(FA_ERR_INVALID_ARG, "dtype must be FA_BF16 or FA_F32");
    if (total < 1 || H < 1 || Hkv < 0) return fail(FA_ERR_INVALID_ARG, "total and H must be >= 1, Hkv >= 0");
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED_D, "d must be 64 or 128");
    if (axes < 1 || axes > 8) return fail(FA_ERR_INVALID_ARG, "axes must be in [1, 8]");
    if (pairs < 8 || pairs % 8 || 2 * pairs > d)
        return fail(FA_ERR_INVALID_ARG, "pairs must be a multiple of 8, at most d / 2");
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
        return fail(FA_ERR_INVALID_ARG, "interleaved and inverse must be 0 or 1");
    if (!q || !q_out || (Hkv > 0 && (!k || !k_out)) || !positions || !inv_freq || !axis)
        return fail(FA_ERR_INVALID_ARG, "q, q_out, positions, inv_freq and axis (and k, k_out where Hkv > 0) must be non-null");
    for (int p = 0; p < pairs; ++p) {
        if (axis[p] < 0 || axis[p] >= axes) return fail(FA_ERR_INVALID_ARG, "axis entries must be in [0, axes)");
        if (!(inv_freq[p] >= -0x1p20 && inv_freq[p] <= 0x1p20))
            return fail(FA_ERR_INVALID_ARG, "inv_freq entries must be finite, at most 2^20 in magnitude");
    }
    if (!aligned16(q) || !aligned16(q_out) || (Hkv > 0 && (!aligned16(k) || !aligned16(k_out))) ||
        !aligned4(positions))
        return fail(FA_ERR_MISALIGNED, "tensors must be 16-byte aligned (positions 4-byte)");
    if (static_cast<long long>(total) * (H + static_cast<long long>(Hkv)) * d >= (1LL << 40))
        return fail(FA_ERR_TOO_LARGE, "total*(H+Hkv)*d must be < 2^40");
    const int es = dtype == FA_F32 ? 4 : 2;
    const int heads[4] = {H, Hkv, H, Hkv};
    long long rs[4], hs[4];
    // strides come as (row, head) pairs of q, k, q_out, k_out
    if (int rc = packed_or_user_strides(strides, 4, heads, d, 16 / es, rs, hs)) return rc;
    if (!strides) {  // (strided views may interleave in one buffer: not checked)
        const size_t tq = static_cast<size_t>(total) * H * d * es;
        const size_t tk = static_cast<size_t>(total) * Hkv * d * es;
        const Span pos{positions, static_cast<size_t>(axes) * total * 4};
        const Span qi{q, tq}, ki{k, tk}, qo{q_out, tq}, ko{k_out, tk};
        // each output may be its own input, and meets nothing else
        if ((q != q_out && spans_meet(qi, qo)) || spans_meet(qo, pos) ||
            (Hkv > 0 && ((k != k_out && spans_meet(ki, ko)) || spans_meet(qo, ki) ||
                         spans_meet(ko, qi) || spans_meet(qo, ko) || spans_meet(ko, pos))))
            return fail(FA_ERR_INVALID_ARG, "q_out and k_out must be their own inputs or overlap "
                                            "neither an input nor one another");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::RopeParams p{};
    p.x[0] = q; p.x[1] = k; p.y[0] = q_out; p.y[1] = k_out;
    for (int z = 0; z < 2; ++z) {
        p.x_rs[z] = rs[z]; p.x_hs[z] = hs[z];
        p.y_rs[z] = rs[2 + z]; p.y_hs[z] = hs[2 + z];
        p.x_ext[z] = rows_extent(total, heads[z], d, rs[z], hs[z]);
        p.y_ext[z] = rows_extent(total, heads[z], d, rs[2 + z], hs[2 + z]);
    }
    p.pos = positions;
    p.pos_ext = static_cast<long long>(axes) * total;
    p.total = total; p.H = H; p.Hkv = Hkv; p.pairs = pairs;
    p.sign = inverse ? -1.0f : 1.0f;
    p.status = di->status;
    for (int i = 0; i < pairs; ++i) {
        p.turn[i] = turn_fraction(inv_freq[i]);
        p.axis[i] = static_cast<unsigned char>(axis[i]);
    }
    cudaError_t e = fa::launch_rope(d, dtype == FA_F32, p, interleaved, static_cast<cudaStream_t>(stream), di->sms);
    if (e != cudaSuccess) return cuda_fail(e, "rope launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// The paged e4m3 cache (fa_cache_append, fa_cache_read, fa_fwd_decode_cache).
// ---------------------------------------------------------------------------------------
namespace {

// The cache's own arguments; *shift receives log2(page_size).
int check_cache(const void* kc, const void* vc, const void* ke, const void* ve, const int* table,
                int B, int max_pages, int num_pages, int page_size, int Hkv, int d, int* shift)
{
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED_D, "d must be 64 or 128");
    if (B < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1)
        return fail(FA_ERR_INVALID_ARG, "B, Hkv, max_pages and num_pages must be >= 1");
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return fail(FA_ERR_INVALID_ARG, "page_size must be a power of two in [16, 1024]");
    if (!kc || !vc || !ke || !ve || !table)
        return fail(FA_ERR_INVALID_ARG, "the cache's tensors and page_table must be non-null");
    if (!aligned16(kc) || !aligned16(vc) || !aligned16(ke) || !aligned16(ve) || !aligned4(table))
        return fail(FA_ERR_MISALIGNED, "the cache's tensors must be 16-byte aligned (page_table 4-byte)");
    if (static_cast<long long>(num_pages) * Hkv * page_size >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "num_pages*Hkv*page_size must be < 2^31");
    int s = 4;
    while ((1 << s) < page_size) ++s;
    *shift = s;
    return FA_OK;
}

// What append and read share: packed rows k, v [total, Hkv, d] on one side, the cache on the other.
int cache_rows_params(const void* k, const void* v, const long long* strides, void* kc, void* vc,
                      void* ke, void* ve, const int* cu, const int* seqlens, const int* table,
                      int B, int max_rows, int total, int max_pages, int num_pages, int page_size,
                      int Hkv, int d, int dtype, fa::CacheParams* p)
{
    if (dtype != FA_BF16 && dtype != FA_F32) return fail(FA_ERR_INVALID_ARG, "dtype must be FA_BF16 or FA_F32");
    int shift = 0;
    if (int rc = check_cache(kc, vc, ke, ve, table, B, max_pages, num_pages, page_size, Hkv, d, &shift))
        return rc;
    if (total < 1 || max_rows < 1) return fail(FA_ERR_INVALID_ARG, "the number of rows and the longest sequence must be >= 1");
    if (!k || !v || !cu) return fail(FA_ERR_INVALID_ARG, "k, v and cu_seqlens must be non-null");
    if (!aligned16(k) || !aligned16(v) || !aligned4(cu))
        return fail(FA_ERR_MISALIGNED, "k and v must be 16-byte aligned (cu_seqlens 4-byte)");
    if (max_rows > total) max_rows = total;
    {
        const size_t codes = static_cast<size_t>(num_pages) * Hkv * page_size;
        const size_t rows = strides ? 0 : static_cast<size_t>(total) * Hkv * d * (dtype == FA_F32 ? 4 : 2);
        const Span cache[4] = {{kc, codes * d}, {vc, codes * d}, {ke, codes}, {ve, codes}};
        // (strided views may interleave: not checked)
        const Span kv[2] = {{strides ? nullptr : k, rows}, {strides ? nullptr : v, rows}};
        const Span ints[3] = {{cu, (B + 1ull) * 4}, {table, static_cast<size_t>(B) * max_pages * 4},
                              {seqlens, seqlens ? B * 4ull : 0}};
        // append writes the cache, read writes k and v: either way they lie apart
        if (outputs_overlap(cache, 4, kv, 2) || (seqlens ? outputs_overlap(cache, 4, ints, 3)
                                                         : outputs_overlap(kv, 2, ints, 2)))
            return fail(FA_ERR_INVALID_ARG, "what is written (the cache, or k and v) must not overlap itself, the other "
                                            "side or the integers, nor the cache's tensors one another");
    }
    const int heads[2] = {Hkv, Hkv};
    long long rs[2], hs[2];
    if (int rc = packed_or_user_strides(strides, 2, heads, d, dtype == FA_F32 ? 4 : 8, rs, hs)) return rc;
    if (((static_cast<long long>(max_rows) + 15) / 16) * B * Hkv >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "B*Hkv*ceil(max_seqlen/16) must be < 2^31");
    *p = fa::CacheParams{};
    p->k = k; p->v = v;
    p->k_rs = rs[0]; p->k_hs = hs[0]; p->v_rs = rs[1]; p->v_hs = hs[1];
    p->k_ext = rows_extent(total, Hkv, d, rs[0], hs[0]);
    p->v_ext = rows_extent(total, Hkv, d, rs[1], hs[1]);
    p->kc = static_cast<uint8_t*>(kc); p->vc = static_cast<uint8_t*>(vc);
    p->ke = static_cast<uint8_t*>(ke); p->ve = static_cast<uint8_t*>(ve);
    p->cu = cu; p->seqlens = seqlens; p->table = table;
    p->B = B; p->Hkv = Hkv; p->total = total; p->max_new = max_rows;
    p->max_pages = max_pages; p->num_pages = num_pages; p->page_shift = shift;
    p->code_ext = static_cast<long long>(num_pages) * Hkv * page_size * d;
    return FA_OK;
}

}  // namespace

extern "C" int fa_cache_append(const void* k, const void* v, const long long* strides,
                               void* k_cache, void* v_cache, void* k_exp, void* v_exp,
                               const int* cu_seqlens_new, const int* seqlens_k,
                               const int* page_table, int B, int max_seqlen_new, int total_new,
                               int max_pages, int num_pages, int page_size, int Hkv, int d,
                               int dtype, void* stream)
{
    fa::CacheParams p;
    if (int rc = cache_rows_params(k, v, strides, k_cache, v_cache, k_exp, v_exp, cu_seqlens_new,
                                   seqlens_k, page_table, B, max_seqlen_new, total_new, max_pages,
                                   num_pages, page_size, Hkv, d, dtype, &p))
        return rc;
    if (!seqlens_k) return fail(FA_ERR_INVALID_ARG, "seqlens_k must be non-null");
    if (!aligned4(seqlens_k)) return fail(FA_ERR_MISALIGNED, "seqlens_k must be 4-byte aligned");
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    p.status = di->status;
    cudaError_t e = fa::launch_cache_append(d, dtype == FA_F32, p, static_cast<cudaStream_t>(stream), di->sms);
    if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
    return FA_OK;
}

extern "C" int fa_cache_read(const void* k_cache, const void* v_cache, const void* k_exp,
                             const void* v_exp, void* k, void* v, const long long* strides,
                             const int* cu_seqlens_k, const int* page_table, int B,
                             int max_seqlen_k, int total_k, int max_pages, int num_pages,
                             int page_size, int Hkv, int d, int dtype, void* stream)
{
    fa::CacheParams p;
    if (int rc = cache_rows_params(k, v, strides, const_cast<void*>(k_cache),
                                   const_cast<void*>(v_cache), const_cast<void*>(k_exp),
                                   const_cast<void*>(v_exp), cu_seqlens_k, nullptr, page_table, B,
                                   max_seqlen_k, total_k, max_pages, num_pages, page_size, Hkv, d,
                                   dtype, &p))
        return rc;
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    p.status = di->status;
    cudaError_t e = fa::launch_cache_read(d, dtype == FA_F32, p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
    return FA_OK;
}

namespace {

// Query rows of a group that one CTA of the cache decode holds: one tile of 8 rows, or one, two
// or four of 16.
int cache_rows_cta(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

constexpr int kCacheMaxCtas = 4096;

// The most blocks a batch of these sizes can have; per_unit: places of a unit besides its blocks.
long long cache_blocks(int B, int H, int Hkv, int max_q, int max_k, int per_unit = 0)
{
    const long long rows = static_cast<long long>(max_q) * (H / Hkv);
    const int rc = cache_rows_cta(rows);
    const long long nblk = (static_cast<long long>(max_k) + fa::kCacheBlock - 1) / fa::kCacheBlock;
    return static_cast<long long>(B) * Hkv * ((rows + rc - 1) / rc) * (nblk + per_unit);
}

size_t cache_part_o_bytes(int H, int Hkv, int d, int max_q, int ctas)
{
    const int rc = cache_rows_cta(static_cast<long long>(max_q) * (H / Hkv));
    return align256(static_cast<size_t>(2) * ctas * rc * d * 4);
}

// 2-D view of the cache's codes for tiles of `rows` rows of one page and head.
int make_cache_map(CUtensorMap* m, const void* base, long long all_rows, int d, int rows)
{
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(all_rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(FA_ERR_LAUNCH, "cuTensorMapEncodeTiled failed with code " + std::to_string(r));
    return FA_OK;
}

}  // namespace

extern "C" int fa_decode_cache_ctas_for(int B, int H, int Hkv, int max_seqlen_q, int max_seqlen_k,
                                        int num_sms)
{
    if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || max_seqlen_q < 1 || max_seqlen_k < 1 || num_sms < 1)
        return fail(FA_ERR_INVALID_ARG, "sizes must be >= 1 and H a multiple of Hkv");
    const long long most = cache_blocks(B, H, Hkv, max_seqlen_q, max_seqlen_k);
    // two blocks at least: beyond that there is little to gain (one sequence of 4 K keys and 8 heads: 10.7 us with
    // 128 CTAs of two blocks, 10.6 with 228, 10.1 with 304), and the places left over serve other streams
    return static_cast<int>(std::min<long long>((most + 1) / 2, std::min(2 * num_sms, kCacheMaxCtas)));
}

extern "C" int fa_decode_cache_num_ctas(int B, int H, int Hkv, int max_seqlen_q, int max_seqlen_k)
{
    if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || max_seqlen_q < 1 || max_seqlen_k < 1)
        return fail(FA_ERR_INVALID_ARG, "sizes must be >= 1 and H a multiple of Hkv");
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    return fa_decode_cache_ctas_for(B, H, Hkv, max_seqlen_q, max_seqlen_k, di->sms);
}

extern "C" size_t fa_decode_cache_workspace_bytes(int H, int Hkv, int d, int max_seqlen_q, int num_ctas)
{
    if (H < 1 || Hkv < 1 || H % Hkv || (d != 64 && d != 128) || max_seqlen_q < 1 || num_ctas < 1 ||
        num_ctas > kCacheMaxCtas)
        return 0;
    if (num_ctas == 1) return 0;
    const int rc = cache_rows_cta(static_cast<long long>(max_seqlen_q) * (H / Hkv));
    return cache_part_o_bytes(H, Hkv, d, max_seqlen_q, num_ctas) + align256(static_cast<size_t>(2) * num_ctas * rc * 4) +
           align256(static_cast<size_t>(num_ctas) * sizeof(int4));
}

extern "C" int fa_fwd_decode_cache(const void* q, const void* k_cache, const void* v_cache,
                                   const void* k_exp, const void* v_exp, void* o, float* lse,
                                   const int* cu_seqlens_q, const int* seqlens_k,
                                   const int* page_table, int B, int max_seqlen_q,
                                   int max_seqlen_k, int total_q, int max_pages, int num_pages,
                                   int page_size, int H, int Hkv, int d, float scale, int causal,
                                   int num_ctas, void* workspace, size_t workspace_bytes,
                                   void* stream)
{
    int shift = 0;
    if (int rc = check_cache(k_cache, v_cache, k_exp, v_exp, page_table, B, max_pages, num_pages,
                             page_size, Hkv, d, &shift))
        return rc;
    if (H < 1 || H % Hkv != 0) return fail(FA_ERR_INVALID_ARG, "H must be a multiple of Hkv");
    if (total_q < 1 || max_seqlen_q < 1 || max_seqlen_k < 1)
        return fail(FA_ERR_INVALID_ARG, "total_q, max_seqlen_q and max_seqlen_k must be >= 1");
    if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
        return fail(FA_ERR_INVALID_ARG, "scale must be finite");
    if (num_ctas < 1 || num_ctas > kCacheMaxCtas)
        return fail(FA_ERR_INVALID_ARG, "num_ctas must be in [1, " + std::to_string(kCacheMaxCtas) + "]");
    if (!q || !o || !cu_seqlens_q || !seqlens_k)
        return fail(FA_ERR_INVALID_ARG, "q, o, cu_seqlens_q and seqlens_k must be non-null");
    if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(cu_seqlens_q) || !aligned4(seqlens_k))
        return fail(FA_ERR_MISALIGNED, "q and o must be 16-byte aligned (the others 4-byte)");
    if (static_cast<long long>(total_q) * H * d >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "total_q*H*d must be < 2^31");
    if (max_seqlen_q > total_q) max_seqlen_q = total_q;
    // no more keys are read than a row of the table has room for (and block ends stay below 2^31)
    const int table_k = static_cast<int>(std::min<long long>(
        std::min(max_seqlen_k, INT_MAX - 1024), static_cast<long long>(max_pages) * page_size));
    if (cache_blocks(B, H, Hkv, max_seqlen_q, table_k, fa::kUnitCost) >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "the batch must have fewer than 2^31 blocks of 128 keys");
    {
        // what the kernel divides by H / Hkv and by Hkv (FastDiv)
        const long long G = H / Hkv, sets = (max_seqlen_q * G + 63) / 8;
        if ((max_seqlen_q * G + 64) * G >= (1LL << 32) || sets * Hkv * Hkv >= (1LL << 32))
            return fail(FA_ERR_TOO_LARGE, "max_seqlen_q*(H/Hkv)^2 and max_seqlen_q*H*Hkv / 8 must be < 2^32");
    }
    const size_t need = fa_decode_cache_workspace_bytes(H, Hkv, d, max_seqlen_q, num_ctas);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
        if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    }
    {
        const size_t codes = static_cast<size_t>(num_pages) * Hkv * page_size;
        const Span out[3] = {{o, static_cast<size_t>(total_q) * H * d * 2},
                             {lse, lse ? static_cast<size_t>(total_q) * H * 4 : 0},
                             {need ? workspace : nullptr, need}};
        const Span in[8] = {{q, out[0].n}, {k_cache, codes * d}, {v_cache, codes * d}, {k_exp, codes}, {v_exp, codes},
                            {cu_seqlens_q, (B + 1ull) * 4}, {seqlens_k, B * 4ull},
                            {page_table, static_cast<size_t>(B) * max_pages * 4}};
        if (outputs_overlap(out, 3, in, 8))
            return fail(FA_ERR_INVALID_ARG, "o, lse and the workspace must not overlap one another or an input");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::CacheDecodeParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    if (need > 0) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.o_part = reinterpret_cast<float*>(ws);
        ws += cache_part_o_bytes(H, Hkv, d, max_seqlen_q, num_ctas);
        p.lse_part = reinterpret_cast<float*>(ws);
        const int rows = cache_rows_cta(static_cast<long long>(max_seqlen_q) * (H / Hkv));
        p.cuts = reinterpret_cast<int4*>(ws + align256(static_cast<size_t>(2) * num_ctas * rows * 4));
    }
    p.ke = static_cast<const uint8_t*>(k_exp);
    p.ve = static_cast<const uint8_t*>(v_exp);
    p.cu_q = cu_seqlens_q; p.seqlens = seqlens_k; p.table = page_table;
    p.B = B; p.H = H; p.Hkv = Hkv; p.G = fa::FastDiv(H / Hkv); p.heads = fa::FastDiv(Hkv);
    p.max_q = max_seqlen_q; p.max_k = max_seqlen_k; p.total_q = total_q; p.table_k = table_k;
    p.max_pages = max_pages; p.num_pages = num_pages; p.page_shift = shift;
    p.ctas = num_ctas;
    p.rows_cta = cache_rows_cta(static_cast<long long>(max_seqlen_q) * (H / Hkv));
    p.row_tiles = p.rows_cta <= 16 ? 1 : p.rows_cta / 16;
    p.rows_shift = p.rows_cta == 8 ? 3 : p.rows_cta == 16 ? 4 : p.rows_cta == 32 ? 5 : 6;
    p.scale_log2 = scale * fa::kLog2e; p.causal = causal;
    p.status = di->status; p.wait_limit_ns = g_wait_limit_ns; p.debug_flags = g_debug_flags;
    const int cut = (g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0;
    p.q_ext = (static_cast<long long>(total_q) * H - cut) * d;
    p.stat_ext = static_cast<long long>(total_q) * H - cut;
    p.part_ext = (2LL * num_ctas * p.rows_cta - cut) * d;
    if (int rc = get_encoder()) return rc;
    CUtensorMap maps[2];
    const long long all_rows = static_cast<long long>(num_pages) * Hkv * page_size;
    const int box = page_size < fa::kCacheBlock ? page_size : fa::kCacheBlock;
    int rc = make_cache_map(&maps[0], k_cache, all_rows, d, box);
    if (!rc) rc = make_cache_map(&maps[1], v_cache, all_rows, d, box);
    if (rc) return rc;
    cudaError_t e = fa::launch_decode_cache(d, maps[0], maps[1], p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cache decode launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// Pages (fa_cache_copy_pages, fa_cache_compact, fa_pages_update).
// ---------------------------------------------------------------------------------------
extern "C" int fa_cache_copy_pages(const void* src_k, const void* src_v, const void* src_k_exp, const void* src_v_exp,
                                   void* dst_k, void* dst_v, void* dst_k_exp, void* dst_v_exp, const int* copies, int n,
                                   int src_pages, int dst_pages, int page_size, int Hkv, int d, void* stream)
{
    int shift = 0;
    if (int rc = check_cache(src_k, src_v, src_k_exp, src_v_exp, copies, 1, 1, src_pages, page_size, Hkv, d, &shift)) return rc;
    if (int rc = check_cache(dst_k, dst_v, dst_k_exp, dst_v_exp, copies, 1, 1, dst_pages, page_size, Hkv, d, &shift)) return rc;
    if (n < 1) return fail(FA_ERR_INVALID_ARG, "the number of copies must be >= 1");
    const long long src_rows = static_cast<long long>(src_pages) * Hkv * page_size;
    const long long dst_rows = static_cast<long long>(dst_pages) * Hkv * page_size;
    if (static_cast<long long>(n) * Hkv * (page_size / 16) >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "n*Hkv*page_size/16 must be < 2^31");
    const bool same = src_k == dst_k && src_v == dst_v && src_k_exp == dst_k_exp && src_v_exp == dst_v_exp;
    if (same && src_pages != dst_pages) return fail(FA_ERR_INVALID_ARG, "one cache has one number of pages");
    {
        const size_t r = static_cast<size_t>(dst_rows), q = static_cast<size_t>(src_rows);
        const Span out[4] = {{dst_k, r * d}, {dst_v, r * d}, {dst_k_exp, r}, {dst_v_exp, r}};
        const Span in[5] = {{copies, static_cast<size_t>(n) * 12}, {src_k, q * d}, {src_v, q * d}, {src_k_exp, q}, {src_v_exp, q}};
        if (outputs_overlap(out, 4, in, same ? 1 : 5))
            return fail(FA_ERR_INVALID_ARG, "the caches must be one or lie apart, and apart from the list");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::PageCopyParams p{};
    p.src_k = static_cast<const uint8_t*>(src_k); p.src_v = static_cast<const uint8_t*>(src_v);
    p.src_ke = static_cast<const uint8_t*>(src_k_exp); p.src_ve = static_cast<const uint8_t*>(src_v_exp);
    p.dst_k = static_cast<uint8_t*>(dst_k); p.dst_v = static_cast<uint8_t*>(dst_v);
    p.dst_ke = static_cast<uint8_t*>(dst_k_exp); p.dst_ve = static_cast<uint8_t*>(dst_v_exp);
    p.copies = copies; p.n = n; p.Hkv = Hkv; p.page_shift = shift; p.src_pages = src_pages; p.dst_pages = dst_pages;
    const int cut = (g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0;
    p.src_rows = src_rows - cut; p.dst_rows = dst_rows - cut;
    p.status = di->status;
    cudaError_t e = fa::launch_cache_copy(d, p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "page copy launch");
    return FA_OK;
}

extern "C" int fa_cache_compact(void* k_cache, void* v_cache, void* k_exp, void* v_exp, const int* keep,
                                const int* cu_keep, const int* start, const int* page_table, int B, int max_keep,
                                int total_keep, int max_pages, int num_pages, int page_size, int Hkv, int d, void* stream)
{
    int shift = 0;
    if (int rc = check_cache(k_cache, v_cache, k_exp, v_exp, page_table, B, max_pages, num_pages, page_size, Hkv, d, &shift))
        return rc;
    if (max_keep < 1 || total_keep < 1) return fail(FA_ERR_INVALID_ARG, "max_keep and total_keep must be >= 1");
    if (!keep || !cu_keep || !start) return fail(FA_ERR_INVALID_ARG, "keep, cu_keep and start must be non-null");
    if (!aligned4(keep) || !aligned4(cu_keep) || !aligned4(start))
        return fail(FA_ERR_MISALIGNED, "keep, cu_keep and start must be 4-byte aligned");
    if (max_keep > total_keep) max_keep = total_keep;
    if (static_cast<long long>(B) * Hkv * 16 >= (1LL << 31)) return fail(FA_ERR_TOO_LARGE, "B*Hkv must be < 2^27");
    if (max_keep > INT_MAX - (1 << 16)) return fail(FA_ERR_TOO_LARGE, "max_keep must be < 2^31 - 2^16");
    const long long rows = static_cast<long long>(num_pages) * Hkv * page_size;
    {
        const size_t r = static_cast<size_t>(rows);
        const Span out[4] = {{k_cache, r * d}, {v_cache, r * d}, {k_exp, r}, {v_exp, r}};
        const Span in[4] = {{keep, static_cast<size_t>(total_keep) * 4}, {cu_keep, (B + 1ull) * 4}, {start, B * 4ull},
                            {page_table, static_cast<size_t>(B) * max_pages * 4}};
        if (outputs_overlap(out, 4, in, 4))
            return fail(FA_ERR_INVALID_ARG, "the cache's tensors must not overlap one another or the integers");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::CompactParams p{};
    p.k = static_cast<uint8_t*>(k_cache); p.v = static_cast<uint8_t*>(v_cache);
    p.ke = static_cast<uint8_t*>(k_exp); p.ve = static_cast<uint8_t*>(v_exp);
    p.keep = keep; p.cu = cu_keep; p.start = start; p.table = page_table;
    p.B = B; p.Hkv = Hkv; p.total = total_keep; p.max_keep = max_keep;
    p.max_pages = max_pages; p.num_pages = num_pages; p.page_shift = shift;
    p.rows = rows - ((g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0);
    p.status = di->status;
    cudaError_t e = fa::launch_cache_compact(d, p, static_cast<cudaStream_t>(stream), di->sms);
    if (e != cudaSuccess) return cuda_fail(e, "cache compaction launch");
    return FA_OK;
}

extern "C" size_t fa_pages_workspace_bytes(int slots, int max_pages, int num_pages)
{
    if (slots < 1 || max_pages < 1 || num_pages < 1) return 0;
    return align256(static_cast<size_t>(slots) * max_pages * 4) + align256(static_cast<size_t>(num_pages) * 4) +
           2 * align256(static_cast<size_t>(slots) * 4);
}

extern "C" int fa_pages_update(int* refs, int* page_table, const int* seqlens, const int* source, const int* kept,
                               const int* new_lens, int* copies, int* counts, int slots, int max_pages, int num_pages,
                               int page_size, void* workspace, size_t workspace_bytes, void* stream)
{
    if (slots < 1 || max_pages < 1 || num_pages < 1)
        return fail(FA_ERR_INVALID_ARG, "slots, max_pages and num_pages must be >= 1");
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return fail(FA_ERR_INVALID_ARG, "page_size must be a power of two in [16, 1024]");
    if (!refs || !page_table || !seqlens || !source || !kept || !new_lens || !copies || !counts)
        return fail(FA_ERR_INVALID_ARG, "every tensor must be non-null");
    if (!aligned16(refs)) return fail(FA_ERR_MISALIGNED, "refs must be 16-byte aligned");
    for (const void* t : {static_cast<const void*>(page_table), static_cast<const void*>(seqlens),
                          static_cast<const void*>(source), static_cast<const void*>(kept),
                          static_cast<const void*>(new_lens), static_cast<const void*>(copies),
                          static_cast<const void*>(counts)})
        if (!aligned4(t)) return fail(FA_ERR_MISALIGNED, "the tensors must be 4-byte aligned");
    if (static_cast<long long>(slots) * max_pages >= (1LL << 31) || num_pages > INT_MAX - (1 << 20))
        return fail(FA_ERR_TOO_LARGE, "slots*max_pages must be < 2^31, num_pages < 2^31 - 2^20");
    const size_t need = fa_pages_workspace_bytes(slots, max_pages, num_pages);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    const size_t n4 = static_cast<size_t>(slots) * 4;
    {
        const Span out[5] = {{refs, static_cast<size_t>(num_pages) * 4}, {page_table, n4 * max_pages}, {copies, 3 * n4},
                             {counts, 8}, {workspace, need}};
        const Span in[4] = {{seqlens, n4}, {source, n4}, {kept, n4}, {new_lens, n4}};
        if (outputs_overlap(out, 5, in, 4))
            return fail(FA_ERR_INVALID_ARG, "what is written must not overlap itself or an input");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::PagesParams p{};
    p.refs = refs; p.table = page_table; p.seqlens = seqlens; p.source = source; p.kept = kept; p.new_lens = new_lens;
    p.copies = copies; p.counts = counts;
    p.slots = slots; p.max_pages = max_pages; p.num_pages = num_pages;
    p.page_shift = 4;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.stage = reinterpret_cast<int*>(ws);
    ws += align256(n4 * max_pages);
    p.fresh = reinterpret_cast<int*>(ws);
    ws += align256(static_cast<size_t>(num_pages) * 4);
    p.offset = reinterpret_cast<int*>(ws);
    p.shared_last = reinterpret_cast<int*>(ws + align256(n4));
    const int cut = (g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0;
    p.refs_ext = num_pages - cut; p.table_ext = static_cast<long long>(slots - cut) * max_pages; p.slot_ext = slots - cut;
    p.status = di->status;
    cudaError_t e = fa::launch_pages_update(p, static_cast<cudaStream_t>(stream), g_debug_flags);
    if (e != cudaSuccess) return cuda_fail(e, "pages update launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// Trees of drafted tokens (fa_tree_mask, fa_fwd_decode_tree).
// ---------------------------------------------------------------------------------------
namespace {

constexpr int kTreeMaxCtas = 1024;
constexpr int kTreeMaxWords = 32;

constexpr int kTreeRows = 128;  // query rows of a unit

// Rows of a unit's parts in the workspace.
int tree_part_rows(int H, int Hkv, int max_q)
{
    return static_cast<int>(std::min<long long>((static_cast<long long>(max_q) * (H / Hkv) + 7) / 8 * 8, kTreeRows));
}

// The most blocks a batch of these sizes can have; per_unit: places of a unit besides its blocks.
long long tree_blocks(int B, int H, int Hkv, int max_q, int max_k, int per_unit = 0)
{
    const long long rows = static_cast<long long>(max_q) * (H / Hkv), unit = kTreeRows;
    const long long nblk = (static_cast<long long>(max_k) + fa::kCacheBlock - 1) / fa::kCacheBlock;
    return static_cast<long long>(B) * Hkv * ((rows + unit - 1) / unit) * (nblk + per_unit);
}

}  // namespace

extern "C" int fa_tree_mask(const int* parents, void* mask, const int* cu_seqlens_q, int B, int max_seqlen_q,
                            int total_q, int mask_words, void* stream)
{
    if (B < 1 || max_seqlen_q < 1 || total_q < 1) return fail(FA_ERR_INVALID_ARG, "B, max_seqlen_q and total_q must be >= 1");
    if (mask_words < 1 || mask_words > kTreeMaxWords)
        return fail(FA_ERR_INVALID_ARG, "mask_words must be in [1, " + std::to_string(kTreeMaxWords) + "]");
    if (max_seqlen_q > total_q) max_seqlen_q = total_q;
    if (max_seqlen_q > 32 * mask_words) return fail(FA_ERR_INVALID_ARG, "a mask row has 32*mask_words bits: max_seqlen_q is more");
    if (!parents || !mask || !cu_seqlens_q) return fail(FA_ERR_INVALID_ARG, "parents, mask and cu_seqlens_q must be non-null");
    if (!aligned4(parents) || !aligned4(mask) || !aligned4(cu_seqlens_q))
        return fail(FA_ERR_MISALIGNED, "parents, mask and cu_seqlens_q must be 4-byte aligned");
    {
        const Span out[1] = {{mask, static_cast<size_t>(total_q) * mask_words * 4}};
        const Span in[2] = {{parents, static_cast<size_t>(total_q) * 4}, {cu_seqlens_q, (B + 1ull) * 4}};
        if (outputs_overlap(out, 1, in, 2)) return fail(FA_ERR_INVALID_ARG, "mask must not overlap an input");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::TreeMaskParams p{};
    p.parents = parents; p.mask = static_cast<uint32_t*>(mask); p.cu = cu_seqlens_q;
    p.B = B; p.max_q = max_seqlen_q; p.total = total_q; p.words = mask_words;
    p.mask_ext = (static_cast<long long>(total_q) - ((g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0)) * mask_words;
    p.status = di->status;
    cudaError_t e = fa::launch_tree_mask(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tree mask launch");
    return FA_OK;
}

extern "C" int fa_decode_tree_ctas_for(int B, int H, int Hkv, int max_seqlen_q, int max_seqlen_k, int num_sms)
{
    if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || max_seqlen_q < 1 || max_seqlen_k < 1 || num_sms < 1)
        return fail(FA_ERR_INVALID_ARG, "sizes must be >= 1 and H a multiple of Hkv");
    const long long most = tree_blocks(B, H, Hkv, max_seqlen_q, max_seqlen_k);
    return static_cast<int>(std::min<long long>((most + 1) / 2, std::min(num_sms, kTreeMaxCtas)));
}

extern "C" int fa_decode_tree_num_ctas(int B, int H, int Hkv, int max_seqlen_q, int max_seqlen_k)
{
    if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || max_seqlen_q < 1 || max_seqlen_k < 1)
        return fail(FA_ERR_INVALID_ARG, "sizes must be >= 1 and H a multiple of Hkv");
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    return fa_decode_tree_ctas_for(B, H, Hkv, max_seqlen_q, max_seqlen_k, di->sms);
}

extern "C" size_t fa_decode_tree_workspace_bytes(int H, int Hkv, int d, int max_seqlen_q, int num_ctas)
{
    if (H < 1 || Hkv < 1 || H % Hkv || (d != 64 && d != 128) || max_seqlen_q < 1 || num_ctas < 1 ||
        num_ctas > kTreeMaxCtas)
        return 0;
    if (num_ctas == 1) return 0;
    const size_t rows = static_cast<size_t>(2) * num_ctas * tree_part_rows(H, Hkv, max_seqlen_q);
    return align256(rows * d * 4) + align256(rows * 4) + align256(static_cast<size_t>(num_ctas) * sizeof(int4));
}

extern "C" int fa_fwd_decode_tree(const void* q, const void* k_cache, const void* v_cache, const void* k_exp,
                                  const void* v_exp, void* o, float* lse, const void* mask, const int* cu_seqlens_q,
                                  const int* seqlens_k, const int* tree_start, const int* page_table, int B,
                                  int max_seqlen_q, int max_seqlen_k, int total_q, int mask_words, int max_pages,
                                  int num_pages, int page_size, int H, int Hkv, int d, float scale, int num_ctas,
                                  void* workspace, size_t workspace_bytes, void* stream)
{
    int shift = 0;
    if (int rc = check_cache(k_cache, v_cache, k_exp, v_exp, page_table, B, max_pages, num_pages, page_size, Hkv, d, &shift))
        return rc;
    if (H < 1 || H % Hkv != 0) return fail(FA_ERR_INVALID_ARG, "H must be a multiple of Hkv");
    if (total_q < 1 || max_seqlen_q < 1 || max_seqlen_k < 1)
        return fail(FA_ERR_INVALID_ARG, "total_q, max_seqlen_q and max_seqlen_k must be >= 1");
    if (mask_words < 1 || mask_words > kTreeMaxWords)
        return fail(FA_ERR_INVALID_ARG, "mask_words must be in [1, " + std::to_string(kTreeMaxWords) + "]");
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY)
        return fail(FA_ERR_INVALID_ARG, "scale must be finite");
    if (num_ctas < 1 || num_ctas > kTreeMaxCtas)
        return fail(FA_ERR_INVALID_ARG, "num_ctas must be in [1, " + std::to_string(kTreeMaxCtas) + "]");
    if (!q || !o || !mask || !cu_seqlens_q || !seqlens_k)
        return fail(FA_ERR_INVALID_ARG, "q, o, mask, cu_seqlens_q and seqlens_k must be non-null");
    if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(mask) || !aligned4(cu_seqlens_q) ||
        !aligned4(seqlens_k) || !aligned4(tree_start))
        return fail(FA_ERR_MISALIGNED, "q and o must be 16-byte aligned (the others 4-byte)");
    if (static_cast<long long>(total_q) * H * d >= (1LL << 31)) return fail(FA_ERR_TOO_LARGE, "total_q*H*d must be < 2^31");
    if (max_seqlen_q > total_q) max_seqlen_q = total_q;
    // no more keys are read than a row of the table has room for (and block ends stay below 2^31)
    const int table_k = static_cast<int>(std::min<long long>(std::min(max_seqlen_k, INT_MAX - 1024),
                                                             static_cast<long long>(max_pages) * page_size));
    if (tree_blocks(B, H, Hkv, max_seqlen_q, table_k, fa::kTreeUnitCost) >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "the batch must have fewer than 2^31 blocks of 128 keys");
    {
        // what the kernel divides by H / Hkv and by Hkv (FastDiv)
        const long long G = H / Hkv, sets = (max_seqlen_q * G + 127) / 128;
        if ((max_seqlen_q * G + 128) * G >= (1LL << 32) || sets * Hkv * Hkv >= (1LL << 32))
            return fail(FA_ERR_TOO_LARGE, "max_seqlen_q*(H/Hkv)^2 and max_seqlen_q*H*Hkv / 128 must be < 2^32");
    }
    const size_t need = fa_decode_tree_workspace_bytes(H, Hkv, d, max_seqlen_q, num_ctas);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
        if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    }
    {
        const size_t codes = static_cast<size_t>(num_pages) * Hkv * page_size;
        const Span out[3] = {{o, static_cast<size_t>(total_q) * H * d * 2},
                             {lse, lse ? static_cast<size_t>(total_q) * H * 4 : 0},
                             {need ? workspace : nullptr, need}};
        const Span in[10] = {{q, out[0].n}, {k_cache, codes * d}, {v_cache, codes * d}, {k_exp, codes}, {v_exp, codes},
                             {cu_seqlens_q, (B + 1ull) * 4}, {seqlens_k, B * 4ull},
                             {page_table, static_cast<size_t>(B) * max_pages * 4},
                             {mask, static_cast<size_t>(total_q) * mask_words * 4}, {tree_start, tree_start ? B * 4ull : 0}};
        if (outputs_overlap(out, 3, in, 10))
            return fail(FA_ERR_INVALID_ARG, "o, lse and the workspace must not overlap one another or an input");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::TreeDecodeParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.part_rows = tree_part_rows(H, Hkv, max_seqlen_q);
    if (need > 0) {
        const size_t rows = static_cast<size_t>(2) * num_ctas * p.part_rows;
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.o_part = reinterpret_cast<float*>(ws);
        ws += align256(rows * d * 4);
        p.lse_part = reinterpret_cast<float*>(ws);
        p.cuts = reinterpret_cast<int4*>(ws + align256(rows * 4));
    }
    p.kc = static_cast<const uint8_t*>(k_cache); p.vc = static_cast<const uint8_t*>(v_cache);
    p.ke = static_cast<const uint8_t*>(k_exp); p.ve = static_cast<const uint8_t*>(v_exp);
    p.cu_q = cu_seqlens_q; p.seqlens = seqlens_k; p.tree_start = tree_start;
    p.mask = static_cast<const uint32_t*>(mask); p.table = page_table;
    p.B = B; p.H = H; p.Hkv = Hkv; p.G = fa::FastDiv(H / Hkv); p.heads = fa::FastDiv(Hkv);
    p.max_q = max_seqlen_q; p.max_k = max_seqlen_k; p.total_q = total_q; p.words = mask_words; p.table_k = table_k;
    p.max_pages = max_pages; p.num_pages = num_pages; p.page_shift = shift;
    p.ctas = num_ctas;
    p.scale_log2 = (scale < 0 ? -scale : scale) * fa::kLog2e;
    p.q_sign = scale < 0 ? 0x80008000u : 0u;
    p.status = di->status; p.wait_limit_ns = g_wait_limit_ns; p.debug_flags = g_debug_flags;
    const int cut = (g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0;
    p.q_ext = (static_cast<long long>(total_q) * H - cut) * d;
    p.stat_ext = static_cast<long long>(total_q) * H - cut;
    p.part_ext = (2LL * num_ctas * p.part_rows - cut) * d;
    p.mask_ext = (static_cast<long long>(total_q) - cut) * mask_words;
    cudaError_t e = fa::launch_decode_tree(d, p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tree decode launch");
    return FA_OK;
}

// ---------------------------------------------------------------------------------------
// Decode with shared prefixes (fa_fwd_decode_shared).
// ---------------------------------------------------------------------------------------
namespace {

constexpr int kSharedMaxCtas = 1024;

// Sets of heads: a line for every head where the CTAs go round, else the fewest heads to a line that
// leave over a tenth fewer CTAs idle.  (96 heads on 152 CTAs: one head to a line keeps 96 of them at
// work; two keep 144.)
int shared_head_groups(int Hkv, int ctas)
{
    int best = std::min(Hkv, ctas);
    for (int nh = 2; nh <= std::min(Hkv, 8); ++nh) {
        const int g = (Hkv + nh - 1) / nh;
        if (g > ctas) continue;
        // a line's CTAs take (heads of the line) / (CTAs of the line) of a head's time
        const long long t = (Hkv + g - 1) / g, n = ctas / g;
        const long long bt = (Hkv + best - 1) / best, bn = ctas / best;
        if (10 * t * bn < 9 * bt * n) best = g;
    }
    return best;
}

size_t shared_rows(int total_q, int H, int ctas) { return static_cast<size_t>(2) * total_q * H + 256 * static_cast<size_t>(ctas); }

}  // namespace

extern "C" size_t fa_decode_shared_workspace_bytes(int total_q, int H, int d, int num_ctas)
{
    if (total_q < 1 || H < 1 || (d != 64 && d != 128) || num_ctas < 1 || num_ctas > kSharedMaxCtas) return 0;
    const size_t rows = shared_rows(total_q, H, num_ctas);
    return align256(rows * d * 4) + align256(rows * 4) + align256(static_cast<size_t>(total_q) * 2 * sizeof(int4));
}

extern "C" int fa_decode_shared_num_ctas(void)
{
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    return std::min(di->sms, kSharedMaxCtas);
}

extern "C" int fa_fwd_decode_shared(const void* q, const void* k_prefix, const void* v_prefix,
                                    const void* k, const void* v, void* o, float* lse,
                                    const int* cu_seqlens_q, const int* cu_seqlens_k,
                                    const int* cu_groups, const int* cu_seqlens_p, int B,
                                    int num_groups, int max_seqlen_q, int max_seqlen_k,
                                    int max_group_q, int max_seqlen_p, int total_q, int total_k,
                                    int total_p, int H, int Hkv, int d, float scale, int causal,
                                    int num_ctas, void* workspace, size_t workspace_bytes,
                                    void* stream)
{
    // Batches without own keys or without prefixes: no unit reads these tensors, so any row will do for
    // the tensor maps, and the kernels find no keys in totals of zero.
    const bool no_own = total_k == 0 && max_seqlen_k == 0, no_prefix = total_p == 0 && max_seqlen_p == 0;
    if (no_own) {
        k = v = q;
        total_k = max_seqlen_k = 1;
    }
    if (no_prefix) {
        k_prefix = v_prefix = q;
        total_p = max_seqlen_p = 1;
    }
    if (int rc = check_varlen(cu_seqlens_q, cu_seqlens_k, B, &max_seqlen_q, &max_seqlen_k, total_q,
                              total_k, H, Hkv, d, scale, causal))
        return rc;
    if (num_groups < 1 || total_p < 1 || max_group_q < 1 || max_seqlen_p < 1)
        return fail(FA_ERR_INVALID_ARG, "num_groups, total_p, max_group_q and max_seqlen_p must be >= 1");
    const int G = H / Hkv;
    if (G > 128) return fail(FA_ERR_INVALID_ARG, "H / Hkv must be <= 128");
    if (num_ctas < 1 || num_ctas > kSharedMaxCtas)
        return fail(FA_ERR_INVALID_ARG, "num_ctas must be in [1, " + std::to_string(kSharedMaxCtas) + "]");
    if (!q || !k_prefix || !v_prefix || !k || !v || !o || !cu_groups || !cu_seqlens_p)
        return fail(FA_ERR_INVALID_ARG, "q, k_prefix, v_prefix, k, v, o, cu_groups and cu_seqlens_p must be non-null");
    if (!aligned16(q) || !aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(k) || !aligned16(v) ||
        !aligned16(o) || !aligned4(lse) || !aligned4(cu_groups) || !aligned4(cu_seqlens_p))
        return fail(FA_ERR_MISALIGNED, "tensors must be 16-byte aligned (lse and the integers 4-byte)");
    if (static_cast<long long>(total_p) * Hkv * d >= (1LL << 31))
        return fail(FA_ERR_TOO_LARGE, "total_p*Hkv*d must be < 2^31");
    max_group_q = std::min(max_group_q, total_q);
    max_seqlen_p = std::min(max_seqlen_p, total_p);
    const int tok = std::min(128 / G, total_q);
    const long long places =
        static_cast<long long>(num_groups) * Hkv * ((max_group_q + tok - 1) / tok) * ((max_seqlen_p + 127) / 128 + fa::kSharedUnitCost) +
        static_cast<long long>(B) * Hkv * ((max_seqlen_q + tok - 1) / tok) * ((max_seqlen_k + 127) / 128 + fa::kSharedUnitCost);
    // (tokens are divided by the tile's: FastDiv)
    if ((std::max(max_group_q, max_seqlen_q) + 128LL) * tok >= (1LL << 32))
        return fail(FA_ERR_TOO_LARGE, "max_seqlen_q and max_group_q must be < 2^25");
    if (places >= (1LL << 31) || static_cast<long long>(B) + num_groups > 16384)
        return fail(FA_ERR_TOO_LARGE, "the batch must have fewer than 2^31 blocks of 128 keys and at most 16384 "
                                      "sequences and groups");
    const size_t need = fa_decode_shared_workspace_bytes(total_q, H, d, num_ctas);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(FA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    {
        const size_t row = static_cast<size_t>(Hkv) * d * 2;  // (where q stands in, its first row is part of it)
        const Span out[3] = {{o, static_cast<size_t>(total_q) * H * d * 2},
                             {lse, lse ? static_cast<size_t>(total_q) * H * 4 : 0}, {workspace, need}};
        const Span in[9] = {{q, out[0].n}, {k_prefix, total_p * row}, {v_prefix, total_p * row}, {k, total_k * row},
                            {v, total_k * row}, {cu_seqlens_q, (B + 1ull) * 4}, {cu_seqlens_k, (B + 1ull) * 4},
                            {cu_groups, (num_groups + 1ull) * 4}, {cu_seqlens_p, (num_groups + 1ull) * 4}};
        if (outputs_overlap(out, 3, in, 9))
            return fail(FA_ERR_INVALID_ARG, "o, lse and the workspace must not overlap one another or an input");
    }
    DeviceInfo* di = nullptr;
    if (int rc = device_info(&di)) return rc;
    fa::SharedDecodeParams p{};
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    const size_t rows = shared_rows(total_q, H, num_ctas);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.o_part = reinterpret_cast<float*>(ws);
    p.lse_part = reinterpret_cast<float*>(ws + align256(rows * d * 4));
    p.part_row0 = 2LL * total_q * H;
    p.places = reinterpret_cast<int4*>(ws + align256(rows * d * 4) + align256(rows * 4));
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.cu_q = cu_seqlens_q; p.cu_k = cu_seqlens_k; p.cu_g = cu_groups; p.cu_p = cu_seqlens_p;
    p.B = B; p.groups = num_groups; p.H = H; p.Hkv = Hkv; p.G = fa::FastDiv(G);
    p.max_q = max_seqlen_q; p.max_k = max_seqlen_k; p.max_group_q = max_group_q; p.max_p = max_seqlen_p;
    p.total_q = total_q; p.total_k = no_own ? 0 : total_k; p.total_p = no_prefix ? 0 : total_p;
    p.tile_tokens = fa::FastDiv(tok);
    p.ctas = num_ctas;
    p.head_groups = shared_head_groups(Hkv, num_ctas);
    p.parts = num_ctas / p.head_groups;
    p.scale_log2 = scale * fa::kLog2e; p.causal = causal;
    p.status = di->status; p.wait_limit_ns = g_wait_limit_ns; p.debug_flags = g_debug_flags;
    const int cut = (g_debug_flags & fa::kDebugShrinkExtents) ? 1 : 0;
    p.q_ext = (static_cast<long long>(total_q) * H - cut) * d;
    p.stat_ext = static_cast<long long>(total_q) * H - cut;
    p.v_ext = (static_cast<long long>(total_k) * Hkv - cut) * d;
    p.part_ext = static_cast<long long>(rows) - cut;
    if (int rc = get_encoder()) return rc;
    CUtensorMap maps[5];
    int rc = make_decode_q_map(&maps[0], q, H, total_q, d, G, tok);
    const long long krs = static_cast<long long>(Hkv) * d;
    if (!rc) rc = make_map(&maps[1], k_prefix, Hkv, total_p, d, 128, true, krs, d);
    if (!rc) rc = make_map(&maps[2], v_prefix, Hkv, total_p, d, 128, true, krs, d);
    if (!rc) rc = make_map(&maps[3], k, Hkv, total_k, d, 128, true, krs, d);
    if (!rc) rc = make_map(&maps[4], v, Hkv, total_k, d, 128, true, krs, d);
    if (rc) return rc;
    cudaError_t e = fa::launch_decode_shared(d, maps, p, static_cast<cudaStream_t>(stream), di->sms);
    if (e != cudaSuccess) return cuda_fail(e, "shared decode launch");
    return FA_OK;
}
