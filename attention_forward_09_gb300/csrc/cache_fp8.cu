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
// LPR lanes share a row, each VPL vectors of 16 bf16 (D = 16 LPR VPL): wide
// loads (a whole 32-byte sector), wide stores (16 codes), log2(LPR) shuffles
// for the row's maximum, and RPW rows a warp.
template <int D>
struct WriteCfg {
    static constexpr int VPL = D % 96 == 0 ? 3 : 2;
    static constexpr int LPR = D / 16 / VPL;
    static constexpr int RPW = 32 / LPR;
    static_assert(LPR * VPL * 16 == D && 32 % LPR == 0, "lane map");
};

struct Vec16 {  // 16 bf16
    uint32_t x[8];
};
__device__ __forceinline__ Vec16 ld_32B(const uint4* p, bool wide) {  // wide: p is a multiple of 32
    Vec16 r;
    if (wide) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.x[0]), "=r"(r.x[1]), "=r"(r.x[2]), "=r"(r.x[3]), "=r"(r.x[4]), "=r"(r.x[5]), "=r"(r.x[6]),
                       "=r"(r.x[7])
                     : "l"(p));
    } else {
        const uint4 a = ld_once(p), b = ld_once(p + 1);
        r = Vec16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return r;
}

// The rows of all tokens, K and V and heads are numbered in a line, and a warp
// takes RPW of them at a time whatever the number of heads; its loads are in
// flight together, asked for before the slots are known.  (Two turns' loads in
// flight gain 2% on a prefill of 27654 tokens and lose 13% on 4099.)
template <int D, bool E5M2>
__global__ void __launch_bounds__(256) kv_cache_write_fp8_sm103a(const CacheWriteFp8Params p) {
    using C = WriteCfg<D>;
    const int lane = threadIdx.x & 31;
    const int sub = lane / C::LPR, lr = lane % C::LPR;
    const uint32_t rows = static_cast<uint32_t>(p.num_tokens) * 2u * p.Hkv;  // below 2^32 - 2^20
    const uint32_t step = ((gridDim.x * blockDim.x) >> 5) * C::RPW;
    for (uint32_t r0 = ((blockIdx.x * blockDim.x + threadIdx.x) >> 5) * C::RPW; r0 < rows; r0 += step) {
        const bool live = r0 + sub < rows;
        const uint32_t row = live ? r0 + sub : r0;
        const uint32_t th = p.by_heads.div(row);  // 2 * token + half (0: key, 1: value)
        const uint32_t h = row - th * p.Hkv;
        const long long t = th >> 1;
        const int half = th & 1;
        const int slot = p.slot_mapping[t];
        const uint4* src = reinterpret_cast<const uint4*>(half ? p.value + t * p.value_stride : p.key + t * p.key_stride) +
                           h * (D / 8) + 2 * lr;
        Vec16 r[C::VPL];
#pragma unroll
        for (int v = 0; v < C::VPL; ++v) r[v] = ld_32B(src + 2 * v * C::LPR, p.wide);
        uint32_t mx = 0;
#pragma unroll
        for (int v = 0; v < C::VPL; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = absmax_bf16x2(mx, r[v].x[i]);
#pragma unroll
        for (int o = 1; o < C::LPR; o <<= 1) mx = absmax_bf16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
        if (__any_sync(0xffffffffu, m16 >= 0x7F80u)) {  // an infinity somewhere: infinities become NaN, maximum again
            uint32_t mi = 0;
#pragma unroll
            for (int v = 0; v < C::VPL; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t& x = r[v].x[i];
                    if ((x & 0x7FFFu) == 0x7F80u) x |= 0x7Fu;
                    if ((x & 0x7FFF0000u) == 0x7F800000u) x |= 0x7F0000u;
                    mi = absmax_bf16x2(mi, x);
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
        if (!live || slot < 0) continue;  // a padding token
        if (slot >= p.num_slots) {
            if (lr == 0 && p.status) atomicOr(p.status, kDevBadIndex);
            continue;
        }
        uint8_t* dst = p.cache + ((static_cast<long long>(half) * p.num_slots + slot) * p.Hkv + h) * D + lr * 16;
#pragma unroll
        for (int v = 0; v < C::VPL; ++v) {
            uint32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = r[v].x[i];
                c[i] = pack_fp8x2<E5M2>(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xFFFF0000u) * inv);
            }
            *reinterpret_cast<uint4*>(dst + v * C::LPR * 16) =
                make_uint4(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
        }
        if (lr == 0) {
            const int block = static_cast<int>(p.by_block.div(slot)), at = slot - block * p.block_size;
            p.scales[((static_cast<long long>(half) * p.num_blocks + block) * p.Hkv + h) * p.block_size + at] =
                static_cast<uint8_t>(b);
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

// Whether sequence s, of boundaries c0 and c1, is one to be read: its rows lie
// in [0, total) and its blocks in the table.
__device__ __forceinline__ bool readable(const CacheReadFp8Params& p, int c0, int c1) {
    return c0 >= 0 && c0 <= c1 && c1 <= p.total &&
           (c0 == c1 || static_cast<int>(p.by_block.div(c1 - 1 - c0)) < p.max_blocks);
}

// A warp takes `group` consecutive packed rows (a power of two up to 32): lane u
// finds where row u lies (a binary search for its sequence, the table), all of
// them at once; then the lanes share the rows' 16-code vectors, [group][2][Hkv]
// [D / 16] in a line whatever the number of heads, kAhead each in flight.
//   Boundaries that decrease leave a binary search without meaning, so what it
// finds is checked, and a row without a sequence makes the warp look, once,
// whether any decrease (in order, such a row lies behind the last sequence);
// only then are the sequences searched one by one.
template <int D, bool E5M2>
__global__ void __launch_bounds__(256, 5) kv_cache_read_fp8_sm103a(const CacheReadFp8Params p, int group) {
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31;
    const int nwarps = static_cast<int>((gridDim.x * blockDim.x) >> 5);
    const int groups = (p.total + group - 1) / group;
    const int vecs = p.Hkv * (D / 16), n = 2 * vecs;  // vectors of a token's keys; of its keys and values
    int ordered = -1;                                 // whether no boundary decreases; -1: not looked at
    for (int g = static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5); g < groups; g += nwarps) {
        const int t0 = g * group, t = t0 + lane;
        int slot = -1, at = 0;  // the row's cache slot (-1: not written, -2: zeros), its place in the block
        int s = -1, c0 = 0;     // its sequence (-1: none), and where that begins
        const bool mine = lane < group && t < p.total;
        if (mine) {
            int lo = 0, hi = p.num_seqs;  // cu[lo] <= t < cu[hi], were cu in order
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu[mid] <= t) lo = mid; else hi = mid;
            }
            c0 = p.cu[lo];
            const int c1 = p.cu[lo + 1];
            if (c0 <= t && t < c1 && readable(p, c0, c1)) s = lo;
        }
        if (__any_sync(0xffffffffu, mine && s < 0)) {
            if (ordered < 0) {
                bool down = false;
                for (int i = lane; i < p.num_seqs; i += 32) down |= p.cu[i + 1] < p.cu[i];
                ordered = !__any_sync(0xffffffffu, down);
            }
            if (!ordered && mine && s < 0) {
                for (int i = 0; i < p.num_seqs && s < 0; ++i) {
                    c0 = p.cu[i];
                    const int c1 = p.cu[i + 1];
                    if (c0 <= t && t < c1 && readable(p, c0, c1)) s = i;
                }
            }
        }
        if (s >= 0) {
            const int pos = t - c0, bi = static_cast<int>(p.by_block.div(pos));
            const int blk = p.block_table[static_cast<long long>(s) * p.max_blocks + bi];
            at = pos - bi * p.block_size;
            if (blk < 0 || blk >= p.num_blocks) {
                if (p.status) atomicOr(p.status, kDevBadIndex);
                slot = -2;
            } else {
                slot = blk * p.block_size + at;
            }
        }
        int u = 0, i = lane;  // the lane's next vector: row u of the group, vector i of it
        for (int q = 0; q < group * n; q += 32 * kAhead) {
            uint4 c[kAhead];
            int b[kAhead], sl[kAhead], tu[kAhead], j[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                while (i >= n) {
                    i -= n;
                    ++u;
                }
                sl[k] = __shfl_sync(0xffffffffu, slot, u & 31);
                const int au = __shfl_sync(0xffffffffu, at, u & 31);
                if (u >= group) sl[k] = -1;
                tu[k] = t0 + u;
                j[k] = i;
                const int half = i >= vecs, v = i - (half ? vecs : 0);
                c[k] = make_uint4(0u, 0u, 0u, 0u);
                b[k] = 1;
                if (sl[k] >= 0) {
                    const long long row = (half ? p.num_slots : 0) + sl[k];
                    c[k] = ld_once(reinterpret_cast<const uint4*>(p.cache) + row * vecs + v);
                    b[k] = p.scales[(row - au) * p.Hkv + static_cast<long long>(v / (D / 16)) * p.block_size + au];
                }
                i += 32;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (sl[k] == -1) continue;
                uint32_t x[8];
                decode16<E5M2>(c[k], exp2_byte(b[k]), x);
                const int half = j[k] >= vecs;
                st_32B((half ? p.v : p.k) + (static_cast<long long>(tu[k]) * vecs + j[k] - (half ? vecs : 0)) * 2, x);
            }
        }
    }
    // every boundary is looked at once, also of sequences that no row falls into
    if (p.status && blockIdx.x == gridDim.x - 1) {
        bool bad = threadIdx.x == 0 && p.cu[0] != 0;
        for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x) bad |= !readable(p, p.cu[i], p.cu[i + 1]);
        if (bad) atomicOr(p.status, kDevBadSeqlen);
    }
}

unsigned warp_grid(long long warps, int num_sms) {
    // CTAs of 8 warps; 40 an SM, so that they are dealt out as SMs come free (8 an
    // SM: a prefill's write 30.9 -> 29.0 us so, 16 contexts read 272 -> 264 us)
    const long long cap = static_cast<long long>(num_sms > 0 ? num_sms : 1) * 40;
    const long long g = (warps + 7) / 8;
    return static_cast<unsigned>(g < 1 ? 1 : (g > cap ? cap : g));
}

template <int D>
cudaError_t write_d(const CacheWriteFp8Params& p, int num_sms, cudaStream_t st) {
    constexpr int rows = WriteCfg<D>::RPW;  // a warp's turn
    const unsigned grid = warp_grid((p.num_tokens * 2 * p.Hkv + rows - 1) / rows, num_sms);
    if (p.e5m2)
        kv_cache_write_fp8_sm103a<D, true><<<grid, 256, 0, st>>>(p);
    else
        kv_cache_write_fp8_sm103a<D, false><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const CacheReadFp8Params& p, int num_sms, cudaStream_t st) {
    // rows a warp: enough to fill its loads while every SM still has a few warps,
    // and up to 16 where that leaves every SM some 160 warps' turns
    const int n = 2 * p.Hkv * (D / 16);
    int group = 1;
    while (group < 16 && n < (1 << 20) && ((group * n < 128 && p.total / (2 * group) >= num_sms * 8) || p.total / (2 * group) >= num_sms * 160)) group *= 2;
    const unsigned grid = warp_grid((p.total + group - 1) / group, num_sms);
    if (p.e5m2)
        kv_cache_read_fp8_sm103a<D, true><<<grid, 256, 0, st>>>(p, group);
    else
        kv_cache_read_fp8_sm103a<D, false><<<grid, 256, 0, st>>>(p, group);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write_fp8(const CacheWriteFp8Params& p, int D, int num_sms, cudaStream_t st) {
    if (p.num_tokens <= 0) return cudaSuccess;
    switch (D) {
        case 64: return write_d<64>(p, num_sms, st);
        case 96: return write_d<96>(p, num_sms, st);
        case 128: return write_d<128>(p, num_sms, st);
        case 192: return write_d<192>(p, num_sms, st);
        case 256: return write_d<256>(p, num_sms, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_cache_read_fp8(const CacheReadFp8Params& p, int num_sms, cudaStream_t st) {
    if (p.num_seqs <= 0 || (p.total <= 0 && !p.status)) return cudaSuccess;  // (without rows: the boundaries are looked at)
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
