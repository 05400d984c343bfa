// api.cpp -- the extern "C" entry points of gbattn.h: argument validation,
// TMA tensor-map encoding and kernel launches.  No allocation, no
// synchronisation; every launch goes to the caller's stream.
#include "../../include/gbattn.h"
#include "../../include/gbattn_bwd.h"
#include "../../include/gbattn_bwd_strided.h"
#include "../../include/gbattn_rotary.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <atomic>
#include <mutex>

#include "kernels.h"

namespace {

using gbattn::PagedParams;
using gbattn::PagedPlan;
using gbattn::PrefillParams;

bool head_size_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool scale_ok(float s) { return isfinite(s) && s > 0.f; }
constexpr float kLog2e = 1.4426950408889634f;

// ---- driver entry point for cuTensorMapEncodeTiled (no link against libcuda)
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// Per-device facts: compute capability 10.3 and the SM count.
struct DeviceInfo {
    bool ok;
    int sms;
};

gbattn_status device_info(DeviceInfo* out) {
    static DeviceInfo cache[64];
    static bool have[64];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GBATTN_ERR_CUDA;
    if (dev < 0 || dev >= 64) return GBATTN_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(mu);
    if (!have[dev]) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return GBATTN_ERR_CUDA;
        cache[dev] = DeviceInfo{major == 10 && minor == 3, sms};
        have[dev] = true;
    }
    *out = cache[dev];
    return out->ok ? GBATTN_OK : GBATTN_ERR_DEVICE;
}

// Tensor [rows, heads, D] (D contiguous; bf16, or fp32 when f32) as a 3-D
// TMA map with box {128 bytes of D, 1, box_rows} and 128-byte swizzle;
// loads read out-of-range elements as zero, stores skip them.
bool encode_rows_heads_d(CUtensorMap* m, const void* base, long long rows, int heads, int d, int box_rows,
                         bool f32 = false, int box_heads = 1) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t es = f32 ? 4 : 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                          static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * es, static_cast<cuuint64_t>(heads) * d * es};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_heads),
                         static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                    const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 8-bit cache [rows, heads, D] as a 3-D TMA map of bytes: a box is `width`
// (128 or 64) columns of one head's 128 rows, zeros past D, swizzled over their span.
bool encode_fp8_cache(CUtensorMap* m, const void* base, long long rows, int heads, int d, int width) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads) * d};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(width), 1, 128};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapSwizzle swizzle = width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Shared by the dense and varlen entries: validation of what they have in common.
// k and v may be null only when there are no keys at all (has_keys == false).
gbattn_status check_common(const void* q, const void* k, const void* v, const void* out, int Hq, int Hkv, int D,
                           float scale, gbattn_dtype odt, bool has_keys) {
    if (!q || !out || (has_keys && (!k || !v))) return GBATTN_ERR_INVALID_ARG;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return GBATTN_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (odt != GBATTN_OUT_BF16 && odt != GBATTN_OUT_F32) return GBATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return GBATTN_ERR_ALIGNMENT;
    return GBATTN_OK;
}

gbattn_status run_prefill(const void* q, const void* k, const void* v, long long Tq, long long Tk, int D,
                          PrefillParams& p, cudaStream_t st) {
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    CUtensorMap tq, tk, tv, to;
    const int bn = gbattn::prefill_block_n(D);
    // With no keys at all no KV tile is ever loaded; point the K/V maps at q
    // so that they are still well-formed.
    const bool no_keys = Tk == 0;
    if (!encode_rows_heads_d(&tq, q, Tq, p.Hq, D, 128) ||
        !encode_rows_heads_d(&tk, no_keys ? q : k, no_keys ? Tq : Tk, no_keys ? p.Hq : p.Hkv, D, bn) ||
        !encode_rows_heads_d(&tv, no_keys ? q : v, no_keys ? Tq : Tk, no_keys ? p.Hq : p.Hkv, D,
                             gbattn::prefill_v_box_rows(D)) ||
        !encode_rows_heads_d(&to, p.out, Tq, p.Hq, D, 128, p.out_f32 != 0))
        return GBATTN_ERR_CUDA;
    return gbattn::launch_prefill(D, tq, tk, tv, to, p, di.sms, st) == cudaSuccess ? GBATTN_OK : GBATTN_ERR_CUDA;
}

// Query heads of the 8-bit decode: rows of a grid (and small enough for the plan's 32-bit counts).
constexpr int kFp8MaxHeads = 65535;

// Shared by the calls on the 8-bit cache: its sizes and code format.
gbattn_status check_fp8_cache(int num_blocks, int block_size, int Hkv, int D, gbattn_kv_dtype kv) {
    if (num_blocks <= 0 || block_size <= 0 || Hkv <= 0) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (kv != GBATTN_KV_E4M3 && kv != GBATTN_KV_E5M2) return GBATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(Hkv) * D > 0x3fffffffLL) return GBATTN_ERR_UNSUPPORTED;  // 32-bit offsets in a row
    return GBATTN_OK;
}

// The sections of the backward pass's workspace, each a multiple of 256 bytes:
// two of row statistics, and kBwdCounters bytes.
constexpr size_t kBwdCounters = 256;
size_t bwd_stat_bytes(long long Tq, int num_docs, int Hq) {
    return ((static_cast<size_t>(gbattn::bwd_stat_stride(Tq, num_docs)) * Hq * 4) + 255) & ~size_t(255);
}

// Memory that a call reads or writes: `count` rows of `bytes` bytes, `stride` bytes apart.
struct Span {
    uintptr_t first;
    size_t count, bytes, stride;
};
Span whole(const void* first, long long bytes) { return {reinterpret_cast<uintptr_t>(first), 1, static_cast<size_t>(bytes), 0}; }
Span bf16_rows(const void* first, long long count, long long values, long long stride) {
    return {reinterpret_cast<uintptr_t>(first), static_cast<size_t>(count), 2 * static_cast<size_t>(values),
            2 * static_cast<size_t>(stride)};
}

// Whether two of them meet.  Rows at the same stride may lie between one
// another (parts of a fused projection); spans that interleave at different
// strides count as meeting.
bool meet(const Span& a, const Span& b) {
    if (!a.first || !b.first || !a.bytes || !b.bytes) return false;
    const Span &lo = a.first <= b.first ? a : b, &hi = a.first <= b.first ? b : a;
    const size_t apart = hi.first - lo.first;
    if (apart >= (lo.count - 1) * lo.stride + lo.bytes) return false;
    if (lo.count == 1 || hi.count == 1 || lo.stride != hi.stride) return true;
    const size_t at = apart % lo.stride;
    return at < lo.bytes || at + hi.bytes > lo.stride;
}

// Strides of contiguous [.., rows, heads, D]; zeros for sizes that are refused.
struct RowStrides {
    long long entry = 0, row = 0, head = 0;
    RowStrides(int rows, int heads, int D) {
        if (rows < 0 || heads <= 0 || !head_size_ok(D)) return;
        head = D;
        row = static_cast<long long>(heads) * D;
        entry = rows < (1ll << 58) / row ? rows * row : 0;
    }
};

// What the entries of the backward pass have in common.  Sizes are validated
// before anything is read; `p` comes with the row counts, bounds and layouts.
gbattn_status run_bwd(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                      const float* lse, const void* dout, const float* dlse, int D, float scale, int causal, void* dq,
                      void* dk, void* dv, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                      gbattn::BwdParams& p, cudaStream_t st) {
    const bool rows = p.Tq > 0 && p.num_docs > 0, keys = p.Tk > 0 && p.num_docs > 0;
    if (p.Hq <= 0 || p.Hkv <= 0 || p.Hq % p.Hkv != 0 || !scale_ok(scale)) return GBATTN_ERR_INVALID_ARG;
    if (rows && (!q || !out || !lse || !dout || !dq)) return GBATTN_ERR_INVALID_ARG;
    if (keys && (!k || !v || !dk || !dv)) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (out_dtype != GBATTN_OUT_BF16 && out_dtype != GBATTN_OUT_F32) return GBATTN_ERR_UNSUPPORTED;
    for (const void* x : {q, k, v, out, dout, static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv)})
        if (!aligned16(x)) return GBATTN_ERR_ALIGNMENT;
    p.tiles_q = static_cast<int>((static_cast<long long>(p.max_q) + 127) / 128);
    p.tiles_k = static_cast<int>((static_cast<long long>(p.max_k) + 127) / 128);
    // An item's number and the counters that hand items out are 32-bit; each CTA
    // claims once past the end, 1024 items at most.
    constexpr long long kMost = 0x7fffffffLL;
    const long long qh = static_cast<long long>(p.tiles_q) * p.num_docs, kh = static_cast<long long>(p.tiles_k) * p.num_docs;
    if (qh > kMost / p.Hq || kh > kMost / p.Hkv) return GBATTN_ERR_UNSUPPORTED;
    if ((p.Hq + 31) / 32 > 65535) return GBATTN_ERR_UNSUPPORTED;
    // out from its first byte to its last
    const long long out_size = out_dtype == GBATTN_OUT_F32 ? 4 : 2;
    long long out_bytes = 0;
    if (rows) {
        const bool packed = p.cu_q != nullptr;
        const long long steps[3][2] = {{packed ? 0 : p.num_docs - 1ll, p.out_bstride},
                                       {(packed ? p.Tq : p.max_q) - 1ll, p.out_rstride},
                                       {p.Hq - 1ll, p.out_hstride}};
        out_bytes = out_size * D;
        for (const auto& x : steps) {
            if (x[0] <= 0) continue;  // a stride that nothing uses
            if (x[1] < 0) return GBATTN_ERR_INVALID_ARG;
            if (x[1] * out_size % 16 != 0) return GBATTN_ERR_ALIGNMENT;
            if (x[1] > (1ll << 58) / x[0]) return GBATTN_ERR_UNSUPPORTED;
            out_bytes += out_size * x[0] * x[1];
        }
    }
    if (!rows && !keys) return GBATTN_OK;
    const size_t stat = bwd_stat_bytes(p.Tq, p.num_docs, p.Hq);
    if (!workspace || workspace_bytes < 2 * stat + kBwdCounters || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return GBATTN_ERR_WORKSPACE;
    const long long q_bytes = 2ll * p.Tq * p.Hq * D, k_bytes = 2ll * p.Tk * p.Hkv * D, lse_bytes = 4ll * p.Tq * p.Hq;
    const Span outs[] = {whole(dq, q_bytes), whole(dk, k_bytes), whole(dv, k_bytes),
                         whole(workspace, static_cast<long long>(2 * stat + kBwdCounters))};
    const Span ins[] = {whole(q, q_bytes),     whole(k, k_bytes),     whole(v, k_bytes),    whole(dout, q_bytes),
                        whole(out, out_bytes), whole(lse, lse_bytes), whole(dlse, lse_bytes)};
    for (int i = 0; i < 4; ++i) {
        for (const Span& in : ins)
            if (meet(outs[i], in)) return GBATTN_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return GBATTN_ERR_INVALID_ARG;
    }
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    p.give_up = gbattn::wait_give_up();
    p.out = out;
    p.dout = dout;
    p.lse = lse;
    p.dlse = dlse;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.neg_lse2 = static_cast<float*>(workspace);
    p.neg_delta = reinterpret_cast<float*>(static_cast<char*>(workspace) + stat);
    p.claims = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + 2 * stat);
    p.stat_stride = gbattn::bwd_stat_stride(p.Tq, p.num_docs);
    p.status = dev_status;
    p.group = p.Hq / p.Hkv;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    // Without rows (or keys) nothing of that side is ever loaded; its maps
    // then view the other side's tensor so that they are well-formed.
    gbattn::BwdMaps m;
    const long long rq = rows ? p.Tq : p.Tk, rk = keys ? p.Tk : p.Tq;
    const int hq = rows ? p.Hq : p.Hkv, hk = keys ? p.Hkv : p.Hq;
    if (!encode_rows_heads_d(&m.q, rows ? q : k, rq, hq, D, 128) || !encode_rows_heads_d(&m.dout, rows ? dout : v, rq, hq, D, 128) ||
        !encode_rows_heads_d(&m.k, keys ? k : q, rk, hk, D, 128) || !encode_rows_heads_d(&m.v, keys ? v : dout, rk, hk, D, 128) ||
        !encode_rows_heads_d(&m.dq, rows ? dq : dk, rq, hq, D, 128) || !encode_rows_heads_d(&m.dk, keys ? dk : dq, rk, hk, D, 128) ||
        !encode_rows_heads_d(&m.dv, keys ? dv : dq, rk, hk, D, 128))
        return GBATTN_ERR_CUDA;
    return gbattn::launch_bwd(D, m, p, di.sms, st) == cudaSuccess ? GBATTN_OK : GBATTN_ERR_CUDA;
}

// What the two calls on rotary positions have in common; `p` comes with their sizes.
gbattn_status check_rotary(const gbattn::RotaryParams& p, int rot_dim, int interleaved, int transpose) {
    if (p.num_tokens < 0 || p.Hq <= 0 || p.Hkv < 0 || !isfinite(p.gain)) return GBATTN_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || (transpose != 0 && transpose != 1)) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(p.D) || rot_dim < 2 || rot_dim > p.D || rot_dim % 2 != 0) return GBATTN_ERR_UNSUPPORTED;
    if (p.num_tokens >= (1ll << 30) || (static_cast<long long>(p.Hq) + 2ll * p.Hkv) * p.D >= (1ll << 30))
        return GBATTN_ERR_UNSUPPORTED;
    if (p.num_tokens == 0) return GBATTN_OK;
    if (!p.q || !p.q_out || !p.positions || !p.steps || (p.Hkv > 0 && (!p.k || !p.k_out))) return GBATTN_ERR_INVALID_ARG;
    // (a stride is not used with one token)
    const long long hq = static_cast<long long>(p.Hq) * p.D, hk = static_cast<long long>(p.Hkv) * p.D;
    if (p.num_tokens > 1 && (p.q_stride < hq || p.q_out_stride < hq || p.k_stride < hk)) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(p.q) || !aligned16(p.k) || !aligned16(p.q_out) || !aligned16(p.k_out) ||
        (reinterpret_cast<uintptr_t>(p.steps) & 7u) != 0)
        return GBATTN_ERR_ALIGNMENT;
    if (p.num_tokens > 1 && ((p.q_stride | p.q_out_stride | p.k_stride) & 7) != 0) return GBATTN_ERR_ALIGNMENT;
    return GBATTN_OK;
}

// 1: the prefill, backward and 8-bit decode kernels give up every pipeline wait (attn_set_wait_give_up).
std::atomic<int> g_give_up{0};

}  // namespace

int gbattn::wait_give_up() { return g_give_up.load(std::memory_order_relaxed); }

extern "C" {

gbattn_status attn_set_wait_give_up(int on, int* previous) {
    if (on != 0 && on != 1) return GBATTN_ERR_INVALID_ARG;
    const int old = g_give_up.exchange(on);
    if (previous) *previous = old;
    return GBATTN_OK;
}

const char* attn_status_string(gbattn_status s) {
    switch (s) {
        case GBATTN_OK: return "ok";
        case GBATTN_ERR_INVALID_ARG: return "invalid argument";
        case GBATTN_ERR_UNSUPPORTED: return "unsupported head size, block size or dtype";
        case GBATTN_ERR_ALIGNMENT: return "tensor pointer not 16-byte aligned";
        case GBATTN_ERR_WORKSPACE: return "workspace missing or too small";
        case GBATTN_ERR_CUDA: return "CUDA error";
        case GBATTN_ERR_DEVICE: return "device is not compute capability 10.3 (GB300)";
        case GBATTN_ERR_SCRATCH_LIMIT: return "sizes need more scratch than attn_fwd_paged_noalloc has built in";
        default: return "unknown status";
    }
}

gbattn_status attn_fwd_dense(const void* q, const void* k, const void* v, int B, int Sq, int Sk, int Hq, int Hkv,
                             int D, float softmax_scale, int causal, void* out, gbattn_dtype out_dtype, float* lse,
                             uint32_t* dev_status, void* stream) {
    gbattn_status s = check_common(q, k, v, out, Hq, Hkv, D, softmax_scale, out_dtype, Sk != 0);
    if (s != GBATTN_OK) return s;
    if (B < 0 || Sq < 0 || Sk < 0) return GBATTN_ERR_INVALID_ARG;
    if (B > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * Sq > 0x7fffffffLL || static_cast<long long>(B) * Sk > 0x7fffffffLL)
        return GBATTN_ERR_UNSUPPORTED;  // row counts are 32-bit on the device
    if (B == 0 || Sq == 0) return GBATTN_OK;
    PrefillParams p{};
    p.give_up = gbattn::wait_give_up();
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    p.cu_q = p.cu_k = nullptr;
    p.num_docs = B;
    p.Sq = Sq;
    p.Sk = Sk;
    p.Tq = B * Sq;
    p.Tk = B * Sk;
    p.max_seqlen_q = Sq;
    p.max_seqlen_k = Sk;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.scale_log2 = softmax_scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    p.lse_bstride = static_cast<long long>(Hq) * Sq;
    p.lse_hstride = Sq;
    p.lse_row_global = 0;
    return run_prefill(q, k, v, static_cast<long long>(B) * Sq, static_cast<long long>(B) * Sk, D, p,
                       static_cast<cudaStream_t>(stream));
}

gbattn_status attn_fwd_padded(const void* q, const void* k, const void* v, const int32_t* lens_q,
                              const int32_t* lens_k, int B, int Sq, int Sk, int Hq, int Hkv, int D,
                              float softmax_scale, int causal, void* out, gbattn_dtype out_dtype, float* lse,
                              uint32_t* dev_status, void* stream) {
    gbattn_status s = check_common(q, k, v, out, Hq, Hkv, D, softmax_scale, out_dtype, Sk != 0);
    if (s != GBATTN_OK) return s;
    if (B < 0 || Sq < 0 || Sk < 0) return GBATTN_ERR_INVALID_ARG;
    if (B > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * Sq > 0x7fffffffLL || static_cast<long long>(B) * Sk > 0x7fffffffLL)
        return GBATTN_ERR_UNSUPPORTED;  // row counts are 32-bit on the device
    if (B == 0 || Sq == 0) return GBATTN_OK;
    PrefillParams p{};
    p.give_up = gbattn::wait_give_up();
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    p.cu_q = p.cu_k = nullptr;
    p.lens_q = lens_q;
    p.lens_k = lens_k;
    p.num_docs = B;
    p.Sq = Sq;
    p.Sk = Sk;
    p.Tq = B * Sq;
    p.Tk = B * Sk;
    p.max_seqlen_q = Sq;
    p.max_seqlen_k = Sk;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.scale_log2 = softmax_scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    p.lse_bstride = static_cast<long long>(Hq) * Sq;
    p.lse_hstride = Sq;
    p.lse_row_global = 0;
    return run_prefill(q, k, v, static_cast<long long>(B) * Sq, static_cast<long long>(B) * Sk, D, p,
                       static_cast<cudaStream_t>(stream));
}

gbattn_status attn_fwd_dense_plan(int B, int Sq, int Sk, int Hq, int Hkv, int D, int causal, int* launches,
                                  int* split) {
    if (!launches || !split) return GBATTN_ERR_INVALID_ARG;
    *launches = 0;
    *split = 0;
    if (B < 0 || Sq < 0 || Sk < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (B > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (B == 0 || Sq == 0) return GBATTN_OK;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    PrefillParams p{};
    p.num_docs = B;
    p.Sq = Sq;
    p.Sk = Sk;
    p.max_seqlen_q = Sq;
    p.max_seqlen_k = Sk;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.causal = causal ? 1 : 0;
    gbattn::PrefillPlan pl;
    if (gbattn::prefill_plan(D, p, di.sms, &pl) != cudaSuccess) return GBATTN_ERR_CUDA;
    *launches = pl.launches;
    *split = pl.split;
    return GBATTN_OK;
}

gbattn_status attn_fwd_varlen_plan(int num_docs, int Tq, int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int D,
                                   int causal, int* launches) {
    if (!launches) return GBATTN_ERR_INVALID_ARG;
    *launches = 0;
    if (num_docs < 0 || Tq < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (num_docs > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (num_docs == 0 || Tq == 0 || max_seqlen_q == 0) return GBATTN_OK;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    int dummy = 0;
    PrefillParams p{};
    p.cu_q = p.cu_k = &dummy;  // only tested for presence: the plan reads no device memory
    p.num_docs = num_docs;
    p.Tq = Tq;
    p.max_seqlen_q = max_seqlen_q;
    p.max_seqlen_k = max_seqlen_k;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.causal = causal ? 1 : 0;
    gbattn::PrefillPlan pl;
    if (gbattn::prefill_plan(D, p, di.sms, &pl) != cudaSuccess) return GBATTN_ERR_CUDA;
    *launches = pl.launches;
    return GBATTN_OK;
}

gbattn_status attn_fwd_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                              const int32_t* cu_seqlens_k, int num_docs, int Tq, int Tk, int max_seqlen_q,
                              int max_seqlen_k, int Hq, int Hkv, int D, float softmax_scale, int causal, void* out,
                              gbattn_dtype out_dtype, float* lse, uint32_t* dev_status, void* stream) {
    gbattn_status s = check_common(q, k, v, out, Hq, Hkv, D, softmax_scale, out_dtype, Tk != 0);
    if (s != GBATTN_OK) return s;
    if (!cu_seqlens_q || !cu_seqlens_k) return GBATTN_ERR_INVALID_ARG;
    if (num_docs < 0 || Tq < 0 || Tk < 0 || max_seqlen_q < 0 || max_seqlen_k < 0) return GBATTN_ERR_INVALID_ARG;
    if (max_seqlen_q > Tq || max_seqlen_k > Tk) return GBATTN_ERR_INVALID_ARG;
    if (num_docs > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (num_docs == 0 || Tq == 0 || max_seqlen_q == 0) return GBATTN_OK;
    PrefillParams p{};
    p.give_up = gbattn::wait_give_up();
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.num_docs = num_docs;
    p.Sq = p.Sk = 0;
    p.Tq = Tq;
    p.Tk = Tk;
    p.max_seqlen_q = max_seqlen_q;
    p.max_seqlen_k = max_seqlen_k;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.scale_log2 = softmax_scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    p.lse_bstride = 0;
    p.lse_hstride = Tq;
    p.lse_row_global = 1;
    return run_prefill(q, k, v, Tq, Tk, D, p, static_cast<cudaStream_t>(stream));
}

gbattn_status attn_kv_cache_write(const void* key, const void* value, const int32_t* slot_mapping, int num_tokens,
                                  void* kv_cache, int num_blocks, int block_size, int Hkv, int D,
                                  uint32_t* dev_status, void* stream) {
    if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || Hkv <= 0) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    // The kernel counts the 2 * num_tokens (token, K or V) rows and a row's
    // 16-byte pieces in 32-bit integers.
    if (num_tokens >= (1 << 30) || static_cast<long long>(Hkv) * D * 2 > 0x7fffffffLL)
        return GBATTN_ERR_UNSUPPORTED;
    if (num_tokens == 0) return GBATTN_OK;
    if (!key || !value || !slot_mapping || !kv_cache) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(kv_cache)) return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    gbattn::CacheWriteParams p{};
    p.key = static_cast<const uint4*>(key);
    p.value = static_cast<const uint4*>(value);
    p.slot_mapping = slot_mapping;
    p.cache = static_cast<uint4*>(kv_cache);
    p.num_tokens = num_tokens;
    p.num_slots = static_cast<long long>(num_blocks) * block_size;
    p.row_vec = Hkv * D * 2 / 16;
    p.status = dev_status;
    return gbattn::launch_cache_write(p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GBATTN_OK
                                                                                          : GBATTN_ERR_CUDA;
}

gbattn_status attn_fwd_paged_prefill(const void* q, const void* kv_cache, int num_blocks, int block_size,
                                     const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                                     const int32_t* cu_seqlens_q, int num_seqs, int Tq, int max_seqlen_q,
                                     int max_seq_len, int Hq, int Hkv, int D, float softmax_scale, int causal,
                                     void* out, gbattn_dtype out_dtype, float* lse, uint32_t* dev_status,
                                     void* stream) {
    gbattn_status s = check_common(q, kv_cache, kv_cache, out, Hq, Hkv, D, softmax_scale, out_dtype, true);
    if (s != GBATTN_OK) return s;
    if (!block_table || !seq_lens || !cu_seqlens_q) return GBATTN_ERR_INVALID_ARG;
    if (num_blocks <= 0 || max_blocks_per_seq <= 0 || num_seqs < 0 || Tq < 0 || max_seqlen_q < 0 ||
        max_seq_len < 0 || max_seqlen_q > Tq)
        return GBATTN_ERR_INVALID_ARG;
    if (block_size != 128) return GBATTN_ERR_UNSUPPORTED;
    if (num_seqs > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (num_seqs == 0 || Tq == 0 || max_seqlen_q == 0) return GBATTN_OK;
    DeviceInfo di;
    s = device_info(&di);
    if (s != GBATTN_OK) return s;
    PrefillParams p{};
    p.give_up = gbattn::wait_give_up();
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    p.cu_q = cu_seqlens_q;
    p.cu_k = nullptr;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.num_docs = num_seqs;
    p.Tq = Tq;
    p.Tk = 0;
    p.max_seqlen_q = max_seqlen_q;
    p.max_seqlen_k = max_seq_len;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.scale_log2 = softmax_scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    p.lse_bstride = 0;
    p.lse_hstride = Tq;
    p.lse_row_global = 1;
    // D <= 128 with a GQA group dividing 128: one CTA per KV head, a tile's
    // rows are 128 / group tokens x the group's heads (each KV byte read once
    // per group; short query chunks fill the tile group times better).
    const int g = Hq / Hkv;
    p.gqa_pack = (D <= 128 && g >= 2 && 128 % g == 0) ? 1 : 0;
    const int box_heads = p.gqa_pack ? g : 1, box_rows = 128 / box_heads;
    CUtensorMap tq, tk, tv, to;
    const long long cache_rows = 2LL * num_blocks * 128;
    if (!encode_rows_heads_d(&tq, q, Tq, Hq, D, box_rows, false, box_heads) ||
        !encode_rows_heads_d(&tk, kv_cache, cache_rows, Hkv, D, 128) ||
        !encode_rows_heads_d(&tv, kv_cache, cache_rows, Hkv, D, gbattn::prefill_v_box_rows(D)) ||
        !encode_rows_heads_d(&to, out, Tq, Hq, D, box_rows, p.out_f32 != 0, box_heads))
        return GBATTN_ERR_CUDA;
    return gbattn::launch_prefill(D, tq, tk, tv, to, p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_mask_to_varlen(const uint8_t* mask, int B, int S, int32_t* cu_seqlens, int32_t* packed_pos,
                                  void* stream) {
    if (B < 0 || S < 0) return GBATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * S > 0x7fffffffLL || B > 0x7fffffff / 2) return GBATTN_ERR_UNSUPPORTED;
    if (B == 0) return GBATTN_OK;
    if (!mask || !cu_seqlens || (S > 0 && !packed_pos)) return GBATTN_ERR_INVALID_ARG;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_mask_to_varlen(mask, B, S, cu_seqlens, packed_pos, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_pack_rows(const void* x, const int32_t* packed_pos, const int32_t* cu_seqlens, int B, int S,
                             int row_bytes, void* packed, void* stream) {
    if (B < 0 || S < 0 || row_bytes <= 0 || row_bytes % 16 != 0) return GBATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * S > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    if (B == 0 || S == 0) return GBATTN_OK;
    if (!x || !packed_pos || !cu_seqlens || !packed) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(packed)) return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_pack_rows(x, packed_pos, cu_seqlens, B, static_cast<long long>(B) * S, row_bytes, packed,
                                    di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_unpack_rows(const void* packed, const int32_t* packed_pos, int B, int S, int row_bytes, void* out,
                               void* stream) {
    if (B < 0 || S < 0 || row_bytes <= 0 || row_bytes % 16 != 0) return GBATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * S > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    if (B == 0 || S == 0) return GBATTN_OK;
    if (!packed || !packed_pos || !out) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(packed) || !aligned16(out)) return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_unpack_rows(packed, packed_pos, static_cast<long long>(B) * S, row_bytes, out, di.sms,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_unpack_lse(const float* lse_packed, const int32_t* packed_pos, int B, int H, int S, float* lse,
                              void* stream) {
    if (B < 0 || S < 0 || H <= 0) return GBATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * S > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    if (B == 0 || S == 0) return GBATTN_OK;
    if (!lse_packed || !packed_pos || !lse) return GBATTN_ERR_INVALID_ARG;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_unpack_lse(lse_packed, static_cast<long long>(B) * S, packed_pos, B, H, S, lse, di.sms,
                                     static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

size_t attn_fwd_paged_workspace_size(int num_seqs, int Hq, int Hkv, int D, int max_seq_len) {
    if (Hkv <= 0 || Hq % Hkv != 0 || !head_size_ok(D)) return 0;
    return gbattn::paged_plan(num_seqs, Hq, Hkv, D, max_seq_len).workspace_bytes;
}

gbattn_status attn_fwd_paged(const void* q, const void* kv_cache, int num_blocks, int block_size,
                             const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                             int num_seqs, int max_seq_len, int Hq, int Hkv, int D, float softmax_scale,
                             int causal, void* out, gbattn_dtype out_dtype, float* lse, void* workspace,
                             size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    (void)causal;  // one query token sees its whole context under the bottom-right rule
    // without sequences the arrays over them are empty, and may be null
    if (!kv_cache || (num_seqs != 0 && (!q || !block_table || !seq_lens || !out))) return GBATTN_ERR_INVALID_ARG;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !scale_ok(softmax_scale)) return GBATTN_ERR_INVALID_ARG;
    if (num_blocks <= 0 || max_blocks_per_seq < (num_seqs != 0 ? 1 : 0) || num_seqs < 0 || max_seq_len < 0)
        return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (block_size != 128) return GBATTN_ERR_UNSUPPORTED;
    if (out_dtype != GBATTN_OUT_BF16 && out_dtype != GBATTN_OUT_F32) return GBATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return GBATTN_ERR_ALIGNMENT;
    if (2LL * num_blocks * 128 > 0x7FFFFFFFLL) return GBATTN_ERR_UNSUPPORTED;  // TMA row coordinate is int32
    if (num_seqs == 0) return GBATTN_OK;
    const int group = Hq / Hkv;
    const int hg = group % 8 == 0 ? 8 : (group % 4 == 0 ? 4 : (group % 2 == 0 ? 2 : 1));
    const PagedPlan plan = gbattn::paged_plan(num_seqs, Hq, Hkv, D, max_seq_len > 0 ? max_seq_len : 1);
    if (!workspace || workspace_bytes < plan.workspace_bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return GBATTN_ERR_WORKSPACE;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    CUtensorMap tm;
    if (!encode_rows_heads_d(&tm, kv_cache, 2LL * num_blocks * 128, Hkv, D, gbattn::paged_slice_rows(D)))
        return GBATTN_ERR_CUDA;
    PagedParams p{};
    p.q = q;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    char* ws = static_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + plan.o_bytes);
    p.pairs = reinterpret_cast<int4*>(ws + plan.o_bytes + plan.lse_bytes);
    p.sched = reinterpret_cast<int*>(ws + plan.o_bytes + plan.lse_bytes + plan.pairs_bytes);
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = group;
    p.heads_per_cta = hg;
    p.blocks_per_split = plan.blocks_per_split;
    p.max_splits = plan.max_splits;
    p.scale_log2 = softmax_scale * kLog2e;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    return gbattn::launch_paged(D, tm, p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}


// ---------------------------------------------------------------- 8-bit KV cache
gbattn_status attn_kv_cache_write_fp8(const void* key, const void* value, long long key_stride, long long value_stride,
                                      const int32_t* slot_mapping, int num_tokens, void* kv_cache, uint8_t* kv_scales,
                                      gbattn_kv_dtype kv_dtype, int num_blocks, int block_size, int Hkv, int D,
                                      uint32_t* dev_status, void* stream) {
    gbattn_status s = check_fp8_cache(num_blocks, block_size, Hkv, D, kv_dtype);
    if (s != GBATTN_OK) return s;
    if (num_tokens < 0) return GBATTN_ERR_INVALID_ARG;
    const long long row = static_cast<long long>(Hkv) * D;
    if (num_tokens > 1 && (key_stride < row || value_stride < row)) return GBATTN_ERR_INVALID_ARG;
    // the kernel numbers the (token, K or V, head) rows in 32 bits
    if (2LL * num_tokens * Hkv >= 0xFFF00000LL) return GBATTN_ERR_UNSUPPORTED;
    if (num_tokens == 0) return GBATTN_OK;
    if (!key || !value || !slot_mapping || !kv_cache || !kv_scales) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(kv_cache) || !aligned16(kv_scales) || key_stride % 8 != 0 ||
        value_stride % 8 != 0)
        return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    s = device_info(&di);
    if (s != GBATTN_OK) return s;
    gbattn::CacheWriteFp8Params p{};
    p.key = static_cast<const uint16_t*>(key);
    p.value = static_cast<const uint16_t*>(value);
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.slot_mapping = slot_mapping;
    p.cache = static_cast<uint8_t*>(kv_cache);
    p.scales = kv_scales;
    p.num_tokens = num_tokens;
    p.num_slots = static_cast<long long>(num_blocks) * block_size;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.Hkv = Hkv;
    p.wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0 &&
             (num_tokens == 1 || (key_stride % 16 == 0 && value_stride % 16 == 0));
    p.by_heads = gbattn::FastDiv::of(static_cast<uint32_t>(Hkv));
    p.by_block = gbattn::FastDiv::of(static_cast<uint32_t>(block_size));
    p.e5m2 = kv_dtype == GBATTN_KV_E5M2;
    p.status = dev_status;
    return gbattn::launch_cache_write_fp8(p, D, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_kv_cache_read_fp8(const void* kv_cache, const uint8_t* kv_scales, gbattn_kv_dtype kv_dtype,
                                     int num_blocks, int block_size, const int32_t* block_table, int max_blocks_per_seq,
                                     const int32_t* cu_seqlens_k, int num_seqs, int Tk, int Hkv, int D, void* k, void* v,
                                     uint32_t* dev_status, void* stream) {
    gbattn_status s = check_fp8_cache(num_blocks, block_size, Hkv, D, kv_dtype);
    if (s != GBATTN_OK) return s;
    if (num_seqs < 0 || Tk < 0 || max_blocks_per_seq < 0) return GBATTN_ERR_INVALID_ARG;
    if (Tk > 0x7fffffff - 64) return GBATTN_ERR_UNSUPPORTED;  // row counters are 32-bit on the device
    if (num_seqs == 0) return GBATTN_OK;
    if (Tk == 0) {  // nothing to read; boundaries that say otherwise are reported
        if (!dev_status || !cu_seqlens_k) return GBATTN_OK;
    } else {
        if (max_blocks_per_seq == 0) return GBATTN_ERR_INVALID_ARG;
        if (!kv_cache || !kv_scales || !block_table || !cu_seqlens_k || !k || !v) return GBATTN_ERR_INVALID_ARG;
        if (!aligned16(kv_cache) || !aligned16(kv_scales) || !aligned16(k) || !aligned16(v)) return GBATTN_ERR_ALIGNMENT;
    }
    DeviceInfo di;
    s = device_info(&di);
    if (s != GBATTN_OK) return s;
    gbattn::CacheReadFp8Params p{};
    p.cache = static_cast<const uint8_t*>(kv_cache);
    p.scales = kv_scales;
    p.block_table = block_table;
    p.cu = cu_seqlens_k;
    p.k = static_cast<uint4*>(k);
    p.v = static_cast<uint4*>(v);
    p.num_slots = static_cast<long long>(num_blocks) * block_size;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.Hkv = Hkv;
    p.D = D;
    p.total = Tk;
    p.by_block = gbattn::FastDiv::of(static_cast<uint32_t>(block_size));
    p.e5m2 = kv_dtype == GBATTN_KV_E5M2;
    p.status = dev_status;
    return gbattn::launch_cache_read_fp8(p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GBATTN_OK
                                                                                                  : GBATTN_ERR_CUDA;
}

size_t attn_fwd_paged_fp8_workspace_size(int num_seqs, int Hq, int Hkv, int D, int max_seq_len) {
    if (num_seqs <= 0 || Hq <= 0 || Hq > kFp8MaxHeads || Hkv <= 0 || Hq % Hkv != 0 || max_seq_len < 0 || !head_size_ok(D))
        return 0;
    return gbattn::paged_fp8_plan(num_seqs, Hq, Hkv, D, max_seq_len).workspace_bytes;
}

gbattn_status attn_fwd_paged_fp8(const void* q, long long q_stride, const void* kv_cache, const uint8_t* kv_scales,
                                 gbattn_kv_dtype kv_dtype, int num_blocks, int block_size, const int32_t* block_table,
                                 int max_blocks_per_seq, const int32_t* seq_lens, int num_seqs, int max_seq_len, int Hq,
                                 int Hkv, int D, float softmax_scale, int causal, void* out, gbattn_dtype out_dtype,
                                 float* lse, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                 void* stream) {
    (void)causal;  // one query token sees its whole context under the bottom-right rule
    // without sequences the arrays over them are empty, and may be null
    if (!kv_cache || !kv_scales || (num_seqs != 0 && (!q || !block_table || !seq_lens || !out)))
        return GBATTN_ERR_INVALID_ARG;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !scale_ok(softmax_scale)) return GBATTN_ERR_INVALID_ARG;
    if (max_blocks_per_seq < (num_seqs != 0 ? 1 : 0) || num_seqs < 0 || max_seq_len < 0) return GBATTN_ERR_INVALID_ARG;
    gbattn_status s = check_fp8_cache(num_blocks, block_size, Hkv, D, kv_dtype);
    if (s != GBATTN_OK) return s;
    if (block_size != 128) return GBATTN_ERR_UNSUPPORTED;
    if (out_dtype != GBATTN_OUT_BF16 && out_dtype != GBATTN_OUT_F32) return GBATTN_ERR_UNSUPPORTED;
    if (Hq > kFp8MaxHeads) return GBATTN_ERR_UNSUPPORTED;
    if (2LL * num_blocks * 128 > 0x7FFFFFFFLL) return GBATTN_ERR_UNSUPPORTED;  // TMA row coordinate is int32
    if (num_seqs > 1 && q_stride < static_cast<long long>(Hq) * D) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(kv_scales) || !aligned16(out) || q_stride % 8 != 0)
        return GBATTN_ERR_ALIGNMENT;
    if (num_seqs == 0) return GBATTN_OK;
    // units of work (a sequence's 128-token blocks and one more) are counted in 32 bits
    const long long blocks = (max_seq_len + 127LL) / 128;
    if (num_seqs * ((blocks < max_blocks_per_seq ? blocks : max_blocks_per_seq) + 1) > 0x7fffffffLL)
        return GBATTN_ERR_UNSUPPORTED;
    const gbattn::PagedFp8Plan plan = gbattn::paged_fp8_plan(num_seqs, Hq, Hkv, D, max_seq_len);
    if (plan.n_hgroups * plan.chunks * (plan.cluster ? num_seqs : 1) > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    if (plan.workspace_bytes &&
        (!workspace || workspace_bytes < plan.workspace_bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return GBATTN_ERR_WORKSPACE;
    DeviceInfo di;
    s = device_info(&di);
    if (s != GBATTN_OK) return s;
    CUtensorMap tm;
    if (!encode_fp8_cache(&tm, kv_cache, 2LL * num_blocks * 128, Hkv, D, gbattn::paged_fp8_box(D))) return GBATTN_ERR_CUDA;
    gbattn::PagedFp8Params p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    p.scales = kv_scales;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    char* ws = static_cast<char*>(workspace);
    if (plan.workspace_bytes) {
        p.part_o = reinterpret_cast<float*>(ws);
        p.part_sum = reinterpret_cast<float2*>(ws + plan.o_bytes);
        p.joins = reinterpret_cast<int2*>(ws + plan.o_bytes + plan.sum_bytes);
    }
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    const long long cap = 128LL * max_blocks_per_seq;
    p.cap = cap < max_seq_len ? static_cast<int>(cap) : max_seq_len;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.subs = plan.subs;
    p.heads_per_sub = plan.heads_per_sub;
    p.head_cols = plan.head_cols;
    p.n_hgroups = static_cast<int>(plan.n_hgroups);
    p.chunks = plan.chunks;
    p.cluster = plan.cluster;
    p.scale_log2 = softmax_scale * kLog2e;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    p.e5m2 = kv_dtype == GBATTN_KV_E5M2;
    p.give_up = gbattn::wait_give_up();
    return gbattn::launch_paged_fp8(D, tm, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GBATTN_OK
                                                                                             : GBATTN_ERR_CUDA;
}

// ---------------------------------------------------------------- block-sparse video attention
gbattn_status attn_gather_rows(const void* src, long long src_rows, const int32_t* index, long long dst_rows,
                               int row_bytes, void* dst, uint32_t* dev_status, void* stream) {
    if (src_rows < 0 || dst_rows < 0 || row_bytes <= 0 || row_bytes % 16 != 0) return GBATTN_ERR_INVALID_ARG;
    if (dst_rows == 0) return GBATTN_OK;
    if (!index || !dst || (src_rows > 0 && !src)) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(src) || !aligned16(dst)) return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_gather_rows(src, src_rows, index, dst_rows, row_bytes, dst, dev_status, di.sms,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_vsa_pool(const void* x_tiled, int num_blocks, int H, int D, const int32_t* block_sizes,
                            float* pooled, uint32_t* dev_status, void* stream) {
    if (num_blocks < 0 || H <= 0) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (num_blocks == 0) return GBATTN_OK;
    if (!x_tiled || !block_sizes || !pooled) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(x_tiled) || !aligned16(pooled)) return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_vsa_pool(x_tiled, block_sizes, num_blocks, H, D, pooled, dev_status, di.sms,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_vsa_list_size(int num_blocks, int num_prefix_blocks, int topk, int Hq, long long* entries) {
    if (!entries || num_blocks < 0 || num_prefix_blocks < 0 || num_prefix_blocks > num_blocks || topk < 1 || Hq <= 0)
        return GBATTN_ERR_INVALID_ARG;
    if (num_blocks >= (1 << 22)) return GBATTN_ERR_UNSUPPORTED;  // block index field of a list entry
    *entries = static_cast<long long>(Hq) * gbattn::VsaGeom::make(num_blocks, num_prefix_blocks, topk).per_head();
    return GBATTN_OK;
}

gbattn_status attn_vsa_block_map(const float* pooled_q, const float* pooled_k, int num_blocks, int num_prefix_blocks,
                                 int Hq, int Hkv, int D, int topk, float softmax_scale, const int32_t* block_sizes,
                                 int32_t* kv_list, int32_t* kv_num, uint32_t* dev_status, void* stream) {
    if (num_blocks < 0 || num_prefix_blocks < 0 || num_prefix_blocks > num_blocks || topk < 1)
        return GBATTN_ERR_INVALID_ARG;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !scale_ok(softmax_scale)) return GBATTN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return GBATTN_ERR_UNSUPPORTED;
    if (num_blocks >= (1 << 22) || Hq > 65535) return GBATTN_ERR_UNSUPPORTED;
    if (num_blocks == 0) return GBATTN_OK;
    if (!pooled_q || !pooled_k || !block_sizes || !kv_list || !kv_num) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(pooled_q) || !aligned16(pooled_k)) return GBATTN_ERR_ALIGNMENT;
    if (gbattn::vsa_map_smem_bytes(num_blocks, D, 2) < 0) return GBATTN_ERR_UNSUPPORTED;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    const gbattn::VsaGeom g = gbattn::VsaGeom::make(num_blocks, num_prefix_blocks, topk);
    return gbattn::launch_vsa_block_map(pooled_q, pooled_k, block_sizes, g, Hq, Hq / Hkv, D, softmax_scale, kv_list,
                                        kv_num, dev_status, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

gbattn_status attn_fwd_vsa(const void* q_tiled, const void* k_tiled, const void* v_tiled, int num_blocks,
                           int num_prefix_blocks, int topk, const int32_t* kv_list, const int32_t* kv_num,
                           const int32_t* out_index, long long out_rows, int Hq, int Hkv, int D, float softmax_scale,
                           void* out, gbattn_dtype out_dtype, float* lse, uint32_t* dev_status, void* stream) {
    if (num_blocks < 0 || num_prefix_blocks < 0 || num_prefix_blocks > num_blocks || topk < 1 || out_rows < 0)
        return GBATTN_ERR_INVALID_ARG;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !scale_ok(softmax_scale)) return GBATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return GBATTN_ERR_UNSUPPORTED;
    if (out_dtype != GBATTN_OUT_BF16 && out_dtype != GBATTN_OUT_F32) return GBATTN_ERR_UNSUPPORTED;
    const long long nbp = num_blocks + (num_blocks & 1);
    const long long rows = nbp * gbattn::kVsaBlock;
    if (num_blocks >= (1 << 22) || nbp / 2 > 65535 || Hq > 65535 || static_cast<long long>(Hq) * (nbp / 2) > 0x7fffffffLL)
        return GBATTN_ERR_UNSUPPORTED;
    if (!out_index && out_rows != rows) return GBATTN_ERR_INVALID_ARG;
    if (num_blocks == 0) return GBATTN_OK;
    if (!q_tiled || !k_tiled || !v_tiled || !kv_list || !kv_num || !out) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(q_tiled) || !aligned16(k_tiled) || !aligned16(v_tiled) || !aligned16(out))
        return GBATTN_ERR_ALIGNMENT;
    DeviceInfo di;
    gbattn_status s = device_info(&di);
    if (s != GBATTN_OK) return s;
    CUtensorMap tq, tk, tv;
    if (!encode_rows_heads_d(&tq, q_tiled, rows, Hq, D, 128) ||
        !encode_rows_heads_d(&tk, k_tiled, rows, Hkv, D, gbattn::kVsaBlock) ||
        !encode_rows_heads_d(&tv, v_tiled, rows, Hkv, D, gbattn::kVsaBlock))
        return GBATTN_ERR_CUDA;
    gbattn::VsaFwdParams p{};
    p.out = out;
    p.lse = lse;
    p.status = dev_status;
    p.kv_list = kv_list;
    p.kv_num = kv_num;
    p.out_index = out_index;
    p.out_rows = out_rows;
    p.g = gbattn::VsaGeom::make(num_blocks, num_prefix_blocks, topk);
    p.Hq = Hq;
    p.group = Hq / Hkv;
    p.scale_log2 = softmax_scale * kLog2e;
    p.out_f32 = out_dtype == GBATTN_OUT_F32;
    return gbattn::launch_vsa_fwd(D, tq, tk, tv, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GBATTN_OK
               : GBATTN_ERR_CUDA;
}

size_t attn_bwd_workspace_size(int num_docs, int Tq, int Hq) {
    if (num_docs < 0 || num_docs > 65535 || Tq < 0 || Hq <= 0) return 0;
    return 2 * bwd_stat_bytes(Tq, num_docs, Hq) + kBwdCounters;
}

gbattn_status attn_bwd_padded_strided(const void* q, const void* k, const void* v, const void* out,
                                      gbattn_dtype out_dtype, long long out_bstride, long long out_rstride,
                                      long long out_hstride, const float* lse, const void* dout, const float* dlse,
                                      const int32_t* lens_q, const int32_t* lens_k, int B, int Sq, int Sk, int Hq, int Hkv,
                                      int D, float softmax_scale, int causal, void* dq, void* dk, void* dv,
                                      void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    if (B < 0 || Sq < 0 || Sk < 0) return GBATTN_ERR_INVALID_ARG;
    if (B > 65535 || static_cast<long long>(B) * Sq > 0x7fffffffLL || static_cast<long long>(B) * Sk > 0x7fffffffLL)
        return GBATTN_ERR_UNSUPPORTED;  // row counts are 32-bit on the device
    gbattn::BwdParams p{};
    p.lens_q = lens_q;
    p.lens_k = lens_k;
    p.num_docs = B;
    p.Tq = B * Sq;
    p.Tk = B * Sk;
    p.max_q = Sq;
    p.max_k = Sk;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.lse_bstride = static_cast<long long>(Hq) * Sq;
    p.lse_hstride = Sq;
    p.out_bstride = out_bstride;
    p.out_rstride = out_rstride;
    p.out_hstride = out_hstride;
    return run_bwd(q, k, v, out, out_dtype, lse, dout, dlse, D, softmax_scale, causal, dq, dk, dv, workspace,
                   workspace_bytes, dev_status, p, static_cast<cudaStream_t>(stream));
}

gbattn_status attn_bwd_padded(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                              const float* lse, const void* dout, const float* dlse, const int32_t* lens_q,
                              const int32_t* lens_k, int B, int Sq, int Sk, int Hq, int Hkv, int D, float softmax_scale,
                              int causal, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                              uint32_t* dev_status, void* stream) {
    const RowStrides o(Sq, Hq, D);
    return attn_bwd_padded_strided(q, k, v, out, out_dtype, o.entry, o.row, o.head, lse, dout, dlse, lens_q, lens_k, B, Sq,
                                   Sk, Hq, Hkv, D, softmax_scale, causal, dq, dk, dv, workspace, workspace_bytes,
                                   dev_status, stream);
}

gbattn_status attn_bwd_dense(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                             const float* lse, const void* dout, const float* dlse, int B, int Sq, int Sk, int Hq,
                             int Hkv, int D, float softmax_scale, int causal, void* dq, void* dk, void* dv,
                             void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    return attn_bwd_padded(q, k, v, out, out_dtype, lse, dout, dlse, nullptr, nullptr, B, Sq, Sk, Hq, Hkv, D,
                           softmax_scale, causal, dq, dk, dv, workspace, workspace_bytes, dev_status, stream);
}

gbattn_status attn_bwd_varlen_strided(const void* q, const void* k, const void* v, const void* out,
                                      gbattn_dtype out_dtype, long long out_rstride, long long out_hstride,
                                      const float* lse, const void* dout, const float* dlse, const int32_t* cu_seqlens_q,
                                      const int32_t* cu_seqlens_k, int num_docs, int Tq, int Tk, int max_seqlen_q,
                                      int max_seqlen_k, int Hq, int Hkv, int D, float softmax_scale, int causal, void* dq,
                                      void* dk, void* dv, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                      void* stream) {
    if (num_docs < 0 || Tq < 0 || Tk < 0 || max_seqlen_q < 0 || max_seqlen_k < 0) return GBATTN_ERR_INVALID_ARG;
    if (max_seqlen_q > Tq || max_seqlen_k > Tk) return GBATTN_ERR_INVALID_ARG;
    if (num_docs > 0 && (!cu_seqlens_q || !cu_seqlens_k)) return GBATTN_ERR_INVALID_ARG;
    if (num_docs > 65535) return GBATTN_ERR_UNSUPPORTED;
    gbattn::BwdParams p{};
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.num_docs = num_docs;
    p.Tq = Tq;
    p.Tk = Tk;
    p.max_q = max_seqlen_q;
    p.max_k = max_seqlen_k;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.lse_hstride = Tq;
    p.lse_row_global = 1;
    p.out_rstride = out_rstride;
    p.out_hstride = out_hstride;
    return run_bwd(q, k, v, out, out_dtype, lse, dout, dlse, D, softmax_scale, causal, dq, dk, dv, workspace,
                   workspace_bytes, dev_status, p, static_cast<cudaStream_t>(stream));
}

gbattn_status attn_bwd_varlen(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                              const float* lse, const void* dout, const float* dlse, const int32_t* cu_seqlens_q,
                              const int32_t* cu_seqlens_k, int num_docs, int Tq, int Tk, int max_seqlen_q,
                              int max_seqlen_k, int Hq, int Hkv, int D, float softmax_scale, int causal, void* dq,
                              void* dk, void* dv, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                              void* stream) {
    const RowStrides o(Tq, Hq, D);
    return attn_bwd_varlen_strided(q, k, v, out, out_dtype, o.row, o.head, lse, dout, dlse, cu_seqlens_q, cu_seqlens_k,
                                   num_docs, Tq, Tk, max_seqlen_q, max_seqlen_k, Hq, Hkv, D, softmax_scale, causal, dq, dk,
                                   dv, workspace, workspace_bytes, dev_status, stream);
}

gbattn_status attn_rotary(const void* q, long long q_stride, const void* k, long long k_stride, const int32_t* positions,
                          int num_tokens, const uint64_t* steps, int rot_dim, int interleaved, int transpose, float gain,
                          int Hq, int Hkv, int D, void* q_out, long long q_out_stride, void* k_out,
                          long long k_out_stride, void* stream) {
    gbattn::RotaryParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_out = static_cast<uint16_t*>(k_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.positions = positions;
    p.steps = reinterpret_cast<const unsigned long long*>(steps);
    p.num_tokens = num_tokens;
    p.half = rot_dim / 2;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.interleaved = interleaved;
    p.transpose = transpose;
    p.gain = gain;
    gbattn_status s = check_rotary(p, rot_dim, interleaved, transpose);
    if (s != GBATTN_OK || num_tokens == 0) return s;
    if (Hkv > 0 && num_tokens > 1) {
        if (k_out_stride < static_cast<long long>(Hkv) * D) return GBATTN_ERR_INVALID_ARG;
        if ((k_out_stride & 7) != 0) return GBATTN_ERR_ALIGNMENT;
    }
    const bool q_same = q == q_out && (num_tokens == 1 || q_stride == q_out_stride);
    const bool k_same = Hkv == 0 || (k == k_out && (num_tokens == 1 || k_stride == k_out_stride));
    p.in_place = q_same && k_same;
    const long long q_row = static_cast<long long>(Hq) * D, k_row = static_cast<long long>(Hkv) * D;
    const Span qi = bf16_rows(q, num_tokens, q_row, q_stride), qo = bf16_rows(q_out, num_tokens, q_row, q_out_stride);
    const Span ki = bf16_rows(k, num_tokens, k_row, k_stride), ko = bf16_rows(k_out, num_tokens, k_row, k_out_stride);
    if ((!q_same && meet(qo, qi)) || (!k_same && meet(ko, ki)) || meet(qo, ki) || meet(ko, qi) || meet(qo, ko))
        return GBATTN_ERR_INVALID_ARG;
    DeviceInfo di;
    s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_rotary(p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GBATTN_OK : GBATTN_ERR_CUDA;
}

gbattn_status attn_rotary_kv_cache_write(const void* q, long long q_stride, const void* key, long long key_stride,
                                         const void* value, long long value_stride, const int32_t* positions,
                                         const int32_t* slot_mapping, int num_tokens, const uint64_t* steps, int rot_dim,
                                         int interleaved, float gain, void* q_out, long long q_out_stride,
                                         void* kv_cache, int num_blocks, int block_size, int Hq, int Hkv, int D,
                                         uint32_t* dev_status, void* stream) {
    gbattn::RotaryParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(key);
    p.v = static_cast<const uint16_t*>(value);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_out = static_cast<uint16_t*>(kv_cache);
    p.q_stride = q_stride;
    p.k_stride = key_stride;
    p.v_stride = value_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = static_cast<long long>(Hkv) * D;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.steps = reinterpret_cast<const unsigned long long*>(steps);
    p.num_tokens = num_tokens;
    p.num_slots = static_cast<long long>(num_blocks) * block_size;
    p.half = rot_dim / 2;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.interleaved = interleaved;
    p.gain = gain;
    p.status = dev_status;
    if (num_blocks <= 0 || block_size <= 0 || Hkv <= 0) return GBATTN_ERR_INVALID_ARG;
    gbattn_status s = check_rotary(p, rot_dim, interleaved, 0);
    if (s != GBATTN_OK) return s;
    if (p.num_slots > 0x7fffffffLL) return GBATTN_ERR_UNSUPPORTED;
    if (num_tokens == 0) return GBATTN_OK;
    if (!value || !slot_mapping) return GBATTN_ERR_INVALID_ARG;
    if (num_tokens > 1 && value_stride < p.k_out_stride) return GBATTN_ERR_INVALID_ARG;
    if (!aligned16(value) || (num_tokens > 1 && (value_stride & 7) != 0)) return GBATTN_ERR_ALIGNMENT;
    const bool q_same = q == q_out && (num_tokens == 1 || q_stride == q_out_stride);
    const long long q_row = static_cast<long long>(Hq) * D, k_row = p.k_out_stride;
    const Span qi = bf16_rows(q, num_tokens, q_row, q_stride), qo = bf16_rows(q_out, num_tokens, q_row, q_out_stride);
    const Span ki = bf16_rows(key, num_tokens, k_row, key_stride), vi = bf16_rows(value, num_tokens, k_row, value_stride);
    const Span cache = whole(kv_cache, 4 * k_row * p.num_slots);
    if ((!q_same && meet(qo, qi)) || meet(qo, ki) || meet(qo, vi) || meet(qo, cache) || meet(cache, qi) || meet(cache, ki) ||
        meet(cache, vi))
        return GBATTN_ERR_INVALID_ARG;
    DeviceInfo di;
    s = device_info(&di);
    if (s != GBATTN_OK) return s;
    return gbattn::launch_rotary(p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GBATTN_OK : GBATTN_ERR_CUDA;
}

}  // extern "C"
