// cache_fp8.cu -- the 8-bit paged KV cache for sm_103a: quantising write
// through slot_mapping, and read-back of whole contexts in bf16.
//
// Format.  A row x of D values (one token, KV head, key or value) is held as
// D codes c (float8 e4m3fn or e5m2) and one exponent byte b; it stands for
// c * 2^(b - 127).  With e = b - 127 the least integer >= -126 such that
// max |x| <= c_max * 2^e over the row's finite values (c_max = 448 or 57344,
// both 1.75 * 2^n), c = RN(x / 2^e), ties to even, and NaN where x is NaN or
// infinite.  The scale is a power of two because a floating code loses nothing
// by it (its relative step is the same in every binade), the division by it is
// exact (so a code depends on no rounding but its own), and the decode applies
// it as an exponent.  A row without a non-zero finite value has e = -126.
//
// Both kernels only move memory: write reads 2 D and writes D + 1 bytes a row,
// read reads D + 1 and writes 2 D.  Rows are 64 to 256 bytes in the cache.
#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace gbattn {

namespace {

__device__ __forceinline__ uint4 ld_once(const uint4* p) {  // read once: keep it out of L1
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// max over both halves of each packed bf16 pair of |x|, NaN halves ignored
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t x) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(x & 0x7FFF7FFFu));
    return r;
}

// ---------------------------------------------------------------- write
// LPR lanes share a row, each VPL vectors of 8 bf16 (D = 8 LPR VPL), so a
// row's maximum is log2(LPR) shuffles and a warp takes 32 / LPR heads at once.
template <int D>
struct WriteCfg {
    static constexpr int VPL = D % 96 == 0 ? 3 : 1;
    static constexpr int LPR = D / 8 / VPL;
    static constexpr int RPW = 32 / LPR;
    static_assert(LPR * VPL * 8 == D && 32 % LPR == 0, "lane map");
};

// A warp takes one (token, K or V): its heads in steps of RPW, kUnroll steps'
// loads in flight, asked for before the slot is known.
template <int D, bool E5M2>
__global__ void __launch_bounds__(256) kv_cache_write_fp8_sm103a(const CacheWriteFp8Params p) {
    using C = WriteCfg<D>;
    constexpr int kUnroll = C::VPL == 1 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int sub = lane / C::LPR, lr = lane % C::LPR;
    const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
    for (long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < 2 * p.num_tokens; w += nwarps) {
        const long long t = w >> 1;
        const int half = static_cast<int>(w & 1);  // 0: key, 1: value
        const int slot = p.slot_mapping[t];
        const uint4* src = reinterpret_cast<const uint4*>(half ? p.value + t * p.value_stride : p.key + t * p.key_stride);
        for (int h0 = sub; h0 - sub < p.Hkv; h0 += C::RPW * kUnroll) {
            uint4 r[kUnroll][C::VPL];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int h = h0 + k * C::RPW;
#pragma unroll
                for (int v = 0; v < C::VPL; ++v) {
                    r[k][v] = make_uint4(0u, 0u, 0u, 0u);
                    if (h < p.Hkv) r[k][v] = ld_once(src + h * (D / 8) + lr + v * C::LPR);
                }
            }
            if (slot < 0) break;  // padding token (warp-uniform)
            if (slot >= p.num_slots) {
                if (lane == 0 && p.status) atomicOr(p.status, kDevBadIndex);
                break;
            }
            const int block = slot / p.block_size, at = slot - block * p.block_size;
            uint8_t* dst = p.cache + (static_cast<long long>(half) * p.num_slots + slot) * p.Hkv * D;
            uint8_t* exps = p.scales + (static_cast<long long>(half) * p.num_blocks + block) * p.Hkv * p.block_size + at;
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int h = h0 + k * C::RPW;
                uint32_t mx = 0;
#pragma unroll
                for (int v = 0; v < C::VPL; ++v) {
                    mx = absmax_bf16x2(mx, r[k][v].x);
                    mx = absmax_bf16x2(mx, r[k][v].y);
                    mx = absmax_bf16x2(mx, r[k][v].z);
                    mx = absmax_bf16x2(mx, r[k][v].w);
                }
#pragma unroll
                for (int o = 1; o < C::LPR; o <<= 1) mx = absmax_bf16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
                if (__any_sync(0xffffffffu, m16 >= 0x7F80u)) {  // an infinity somewhere: infinities become NaN, maximum again
                    uint32_t mi = 0;
#pragma unroll
                    for (int v = 0; v < C::VPL; ++v) {
                        uint32_t* x = reinterpret_cast<uint32_t*>(&r[k][v]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if ((x[i] & 0x7FFFu) == 0x7F80u) x[i] |= 0x7Fu;
                            if ((x[i] & 0x7FFF0000u) == 0x7F800000u) x[i] |= 0x7F0000u;
                            mi = absmax_bf16x2(mi, x[i]);
                        }
                    }
#pragma unroll
                    for (int o = 1; o < C::LPR; o <<= 1) mi = absmax_bf16x2(mi, __shfl_xor_sync(0xffffffffu, mi, o));
                    m16 = max(mi & 0xFFFFu, mi >> 16);
                }
                // max = 1.f * 2^(E - 127), c_max = 1.75 * 2^n: b = E - n, one more if 1.f > 1.75
                const int E = static_cast<int>(m16 >> 7);
                int b = E - (E5M2 ? 15 : 8) + ((m16 & 0x7Fu) > 0x60u ? 1 : 0);
                b = b < 1 ? 1 : b;
                const float inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);  // 2^(127 - b), exact
                if (h >= p.Hkv) continue;
#pragma unroll
                for (int v = 0; v < C::VPL; ++v) {
                    const uint32_t x[4] = {r[k][v].x, r[k][v].y, r[k][v].z, r[k][v].w};
                    uint32_t c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c[i] = pack_fp8x2<E5M2>(__uint_as_float(x[i] << 16) * inv, __uint_as_float(x[i] & 0xFFFF0000u) * inv);
                    *reinterpret_cast<uint2*>(dst + h * D + (lr + v * C::LPR) * 8) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                }
                if (lr == 0) exps[static_cast<long long>(h) * p.block_size] = static_cast<uint8_t>(b);
            }
        }
    }
}

// ---------------------------------------------------------------- read
// Sixteen codes to sixteen bf16 values: code pairs to fp16 (exact), to fp32,
// times 2^(b - 127) (exact but for subnormal results), to bf16 (exact: a code
// has at most four significant bits).
template <bool E5M2>
__device__ __forceinline__ void decode16(const uint4& c, float scale, uint32_t (&o)[8]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack_fp8x2<E5M2>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
        o[i] = pack_bf16x2(f.x * scale, f.y * scale);
    }
}
// One whole 32-byte sector in one store, where the address allows it.
__device__ __forceinline__ void st_32B(uint4* p, const uint32_t (&x)[8]) {
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                     "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        p[0] = make_uint4(x[0], x[1], x[2], x[3]);
        p[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// A warp takes TOK consecutive packed rows: lane i the 16-code vectors i, i +
// 32, ... of each token's keys and values, [2][Hkv][D] in turn, kAhead of them
// asked for at once.  The sequence is found by a binary search for the first
// row and by stepping on for the others.  TOK is 2; 1 where that leaves SMs
// without a warp.
template <int D, bool E5M2, int TOK>
__global__ void __launch_bounds__(256) kv_cache_read_fp8_sm103a(const CacheReadFp8Params p) {
    constexpr int kAhead = 2;
    const int lane = threadIdx.x & 31;
    const int nwarps = static_cast<int>((gridDim.x * blockDim.x) >> 5);
    const int groups = (p.total + TOK - 1) / TOK;
    const int vecs = p.Hkv * (D / 16);
    for (int g = static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5); g < groups; g += nwarps) {
        const int t0 = g * TOK;
        const int end = p.cu[p.num_seqs];
        int s = 0, hi = p.num_seqs;  // cu[s] <= t0 < cu[hi], were cu in order
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if (p.cu[mid] <= t0) s = mid; else hi = mid;
        }
        if (t0 >= end) continue;  // behind the last sequence: left as they are
        int c0 = p.cu[s], c1 = p.cu[s + 1];
        long long row[TOK], exps[TOK];  // first vector of the token's keys; its first exponent byte
        int kind[TOK];                  // 0: not written, 1: zeros, 2: read
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
            const int t = t0 + u;
            kind[u] = 0;
            row[u] = exps[u] = 0;
            while (t >= c1 && s + 1 < p.num_seqs) {
                ++s;
                c0 = c1;
                c1 = p.cu[s + 1];
            }
            if (t >= p.total || t >= c1) continue;
            const int pos = t - c0, bi = pos / p.block_size;
            if (c0 < 0 || pos < 0 || c1 > p.total || (c1 - 1 - c0) / p.block_size >= p.max_blocks) {
                if (lane == 0 && p.status) atomicOr(p.status, kDevBadSeqlen);
                continue;
            }
            const int blk = p.block_table[static_cast<long long>(s) * p.max_blocks + bi];
            if (blk < 0 || blk >= p.num_blocks) {
                if (lane == 0 && p.status) atomicOr(p.status, kDevBadIndex);
                kind[u] = 1;
                continue;
            }
            const int at = pos - bi * p.block_size;
            kind[u] = 2;
            row[u] = (static_cast<long long>(blk) * p.block_size + at) * vecs;
            exps[u] = static_cast<long long>(blk) * p.Hkv * p.block_size + at;
        }
        for (int i0 = lane; i0 < 2 * vecs; i0 += 32 * kAhead) {
            uint4 c[kAhead][TOK];
            int b[kAhead][TOK];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + 32 * k, half = i >= vecs, j = i - (half ? vecs : 0), h = j / (D / 16);
#pragma unroll
                for (int u = 0; u < TOK; ++u) {
                    c[k][u] = make_uint4(0u, 0u, 0u, 0u);
                    b[k][u] = 1;
                    if (kind[u] == 2 && i < 2 * vecs) {
                        c[k][u] = ld_once(reinterpret_cast<const uint4*>(p.cache) + (half ? p.num_slots * vecs : 0) + row[u] + j);
                        b[k][u] = p.scales[(half ? p.num_slots * p.Hkv : 0) + exps[u] + static_cast<long long>(h) * p.block_size];
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + 32 * k, half = i >= vecs, j = i - (half ? vecs : 0);
#pragma unroll
                for (int u = 0; u < TOK; ++u) {
                    if (kind[u] == 0 || i >= 2 * vecs) continue;
                    uint32_t x[8];
                    decode16<E5M2>(c[k][u], exp2_byte(b[k][u]), x);
                    st_32B((half ? p.v : p.k) + (static_cast<long long>(t0 + u) * vecs + j) * 2, x);
                }
            }
        }
    }
}

template <int D>
cudaError_t write_d(const CacheWriteFp8Params& p, unsigned grid, cudaStream_t st) {
    if (p.e5m2)
        kv_cache_write_fp8_sm103a<D, true><<<grid, 256, 0, st>>>(p);
    else
        kv_cache_write_fp8_sm103a<D, false><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

unsigned warp_grid(long long warps, int num_sms) {
    const long long cap = static_cast<long long>(num_sms > 0 ? num_sms : 1) * 8;  // 8 CTAs of 8 warps per SM
    const long long g = (warps + 7) / 8;
    return static_cast<unsigned>(g < 1 ? 1 : (g > cap ? cap : g));
}

template <int D, bool E5M2>
cudaError_t read_tok(const CacheReadFp8Params& p, int num_sms, cudaStream_t st) {
    if (p.total / 2 >= num_sms * 8)
        kv_cache_read_fp8_sm103a<D, E5M2, 2><<<warp_grid((p.total + 1) / 2, num_sms), 256, 0, st>>>(p);
    else
        kv_cache_read_fp8_sm103a<D, E5M2, 1><<<warp_grid(p.total, num_sms), 256, 0, st>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const CacheReadFp8Params& p, int num_sms, cudaStream_t st) {
    return p.e5m2 ? read_tok<D, true>(p, num_sms, st) : read_tok<D, false>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_cache_write_fp8(const CacheWriteFp8Params& p, int D, int num_sms, cudaStream_t st) {
    if (p.num_tokens <= 0) return cudaSuccess;
    const unsigned grid = warp_grid(p.num_tokens * 2, num_sms);
    switch (D) {
        case 64: return write_d<64>(p, grid, st);
        case 96: return write_d<96>(p, grid, st);
        case 128: return write_d<128>(p, grid, st);
        case 192: return write_d<192>(p, grid, st);
        case 256: return write_d<256>(p, grid, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_cache_read_fp8(const CacheReadFp8Params& p, int num_sms, cudaStream_t st) {
    if (p.total <= 0 || p.num_seqs <= 0) return cudaSuccess;
    switch (p.D) {
        case 64: return read_d<64>(p, num_sms, st);
        case 96: return read_d<96>(p, num_sms, st);
        case 128: return read_d<128>(p, num_sms, st);
        case 192: return read_d<192>(p, num_sms, st);
        case 256: return read_d<256>(p, num_sms, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbattn
