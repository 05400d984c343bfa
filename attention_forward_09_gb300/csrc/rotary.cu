// rotary.cu -- rotary positions of queries and keys for sm_103a, alone
// (attn_rotary) or with the paged cache's write (attn_rotary_kv_cache_write).
//
// Pair i < rot / 2 of a head's first rot values is a point (x, y) turned by the
// angle a = t f_i of its token's position t:
//   (x, y) -> gain (x cos a - y sin a, x sin a + y cos a)
// (the transpose, for gradients: -a).  The pair lies at i and i + rot / 2, or
// at 2 i and 2 i + 1 ("interleaved"); the rest of the head is copied.
//
// Angles: far positions make t f_i large, and an fp32 product would lose it
// (at t = 10^6 its last bit is 0.06 rad).  f_i comes as f_i / 2 pi in units of
// 2^-64 turns, so that t f_i modulo a turn is one 64-bit integer product,
// exact for every 32-bit position, negative ones included; the signed fraction
// of a turn goes to fp32 and sincospif.
//
// HBM-bound: a value is read and written once.  A warp takes one token (or,
// where tokens are few, an equal share of its heads): its lanes ask for the
// first vectors, work out the token's cosines and sines once meanwhile, into
// the warp's part of shared memory, and move 16-byte vectors, pairs of them in
// the half layout, two units in flight a lane (27654 tokens of 32 + 8 heads of
// 128: 86 us of kernel, 6.6 TB/s; with one unit 90, three 88, four 96: the
// registers of more cost warps).  Rotated widths that are no whole vectors (half layout: rot %
// 16, interleaved: rot % 8) are moved pair by pair, the copied rest value by
// value: right and slow (the same tokens, rot 20 of 128, half layout: 570 us, 1.0 TB/s).
#include "kernels.h"
#include "ptx.cuh"

namespace gbattn {

namespace {

enum RotaryLayout {
    kHalfVec,         // half layout, rot % 16 == 0: a unit is 8 pairs, two vectors
    kInterleavedVec,  // interleaved, rot % 8 == 0: a unit is 4 pairs, one vector
    kPairs            // either layout, a unit is a pair (or one copied value)
};

__device__ __forceinline__ uint4 ld_row(const uint16_t* p) {  // read once; may be written in place
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_round(float x) { return pack_bf16x2(x, 0.f) & 0xffffu; }

}  // namespace

template <int LAYOUT, bool STORE>
__global__ void __launch_bounds__(256) rotary_sm103a(const RotaryParams p) {
    constexpr int UN = 2;  // units in flight a lane
    __shared__ __align__(16) float table[8][2][128];  // cosines and sines of a warp's token, times the gain
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long task = static_cast<long long>(blockIdx.x) * 8 + warp;
    const long long t = task / p.parts;
    if (t >= p.num_tokens) return;
    const int part = static_cast<int>(task % p.parts);
    float *cs = table[warp][0], *sn = table[warp][1];
    const long long pos = p.positions[t];
    long long slot = 0;
    if (STORE) {
        slot = p.slot_mapping[t];
        if (slot >= p.num_slots) {
            if (lane == 0 && part == 0 && p.status) atomicOr(p.status, kDevBadIndex);
            slot = -1;
        }
    }

    // Units of the token: the query heads', the key heads', then the value row's vectors.
    const int U = p.units, nq = p.Hq * U, nk = nq + p.Hkv * U, n = STORE ? nk + p.Hkv * (p.D >> 3) : nk;
    const int rot_units = LAYOUT == kHalfVec ? p.half >> 3 : (LAYOUT == kInterleavedVec ? p.half >> 2 : p.half);
    const int stride = p.parts * 32;
    bool first = true;
    for (int i0 = part * 32 + lane; first || i0 < n; i0 += stride * UN) {
        uint4 a[UN], b[UN];
        const uint16_t* src[UN];
        uint16_t* dst[UN];
        int unit[UN];  // within the head; -1: a value vector; -2: nothing
#pragma unroll
        for (int x = 0; x < UN; ++x) {
            const int i = i0 + x * stride;
            unit[x] = -2;
            if (i >= n) continue;
            if (i < nk) {
                const bool q = i < nq;
                if (STORE && !q && slot < 0) continue;
                const int j = q ? i : i - nq;
                const int head = p.by_units.div(j);
                unit[x] = j - head * U;
                src[x] = (q ? p.q + t * p.q_stride : p.k + t * p.k_stride) + head * p.D;
                dst[x] = (q ? p.q_out + t * p.q_out_stride : p.k_out + (STORE ? slot : t) * p.k_out_stride) + head * p.D;
            } else {
                if (slot < 0) continue;
                unit[x] = -1;
                src[x] = p.v + t * p.v_stride + (i - nk) * 8;
                dst[x] = p.k_out + (p.num_slots + slot) * p.k_out_stride + (i - nk) * 8;
            }
            if (LAYOUT == kPairs) {
                if (unit[x] == -1) a[x] = ld_row(src[x]);
            } else {
                // rotated units first, then the copied vectors of the head
                int e = unit[x] < 0 ? 0 : unit[x] * 8;
                if (LAYOUT == kHalfVec && unit[x] >= rot_units) e += p.half;
                src[x] += e;
                dst[x] += e;
                a[x] = ld_row(src[x]);
                if (LAYOUT == kHalfVec && unit[x] >= 0 && unit[x] < rot_units) b[x] = ld_row(src[x] + p.half);
            }
        }
        if (first) {  // the token's table, while the first vectors are on their way
            first = false;
            for (int i = lane; i < p.half; i += 32) {
                const unsigned long long turn = static_cast<unsigned long long>(pos) * p.steps[i];  // 2^-64 turns, modulo one
                float s, c;
                sincospif(__ll2float_rn(static_cast<long long>(turn)) * 0x1p-63f, &s, &c);
                cs[i] = c * p.gain;
                sn[i] = (p.transpose ? -s : s) * p.gain;
            }
            __syncwarp();
        }
#pragma unroll
        for (int x = 0; x < UN; ++x) {
            if (unit[x] == -2) continue;
            if (unit[x] == -1 || (LAYOUT != kPairs && unit[x] >= rot_units)) {
                st_global_v4(dst[x], a[x].x, a[x].y, a[x].z, a[x].w);
            } else if (LAYOUT == kHalfVec) {
                const uint32_t aw[4] = {a[x].x, a[x].y, a[x].z, a[x].w}, bw[4] = {b[x].x, b[x].y, b[x].z, b[x].w};
                uint32_t ra[4], rb[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 c = *reinterpret_cast<const float4*>(cs + unit[x] * 8 + h * 4);
                    const float4 s = *reinterpret_cast<const float4*>(sn + unit[x] * 8 + h * 4);
                    const uint32_t a0 = aw[2 * h], a1 = aw[2 * h + 1], b0 = bw[2 * h], b1 = bw[2 * h + 1];
                    ra[2 * h] = pack_bf16x2(bf_lo(a0) * c.x - bf_lo(b0) * s.x, bf_hi(a0) * c.y - bf_hi(b0) * s.y);
                    ra[2 * h + 1] = pack_bf16x2(bf_lo(a1) * c.z - bf_lo(b1) * s.z, bf_hi(a1) * c.w - bf_hi(b1) * s.w);
                    rb[2 * h] = pack_bf16x2(bf_lo(a0) * s.x + bf_lo(b0) * c.x, bf_hi(a0) * s.y + bf_hi(b0) * c.y);
                    rb[2 * h + 1] = pack_bf16x2(bf_lo(a1) * s.z + bf_lo(b1) * c.z, bf_hi(a1) * s.w + bf_hi(b1) * c.w);
                }
                st_global_v4(dst[x], ra[0], ra[1], ra[2], ra[3]);
                st_global_v4(dst[x] + p.half, rb[0], rb[1], rb[2], rb[3]);
            } else if (LAYOUT == kInterleavedVec) {
                const float4 c = *reinterpret_cast<const float4*>(cs + unit[x] * 4);
                const float4 s = *reinterpret_cast<const float4*>(sn + unit[x] * 4);
                const float cw[4] = {c.x, c.y, c.z, c.w}, sw[4] = {s.x, s.y, s.z, s.w};
                const uint32_t w[4] = {a[x].x, a[x].y, a[x].z, a[x].w};
                uint32_t r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r[e] = pack_bf16x2(bf_lo(w[e]) * cw[e] - bf_hi(w[e]) * sw[e], bf_lo(w[e]) * sw[e] + bf_hi(w[e]) * cw[e]);
                st_global_v4(dst[x], r[0], r[1], r[2], r[3]);
            } else if (unit[x] >= rot_units) {
                const int e = p.half + unit[x];  // rot + (unit - half)
                dst[x][e] = src[x][e];
            } else {
                const int i = unit[x], e0 = p.interleaved ? 2 * i : i, e1 = p.interleaved ? 2 * i + 1 : i + p.half;
                const float f = bf_lo(src[x][e0]), g = bf_lo(src[x][e1]);
                dst[x][e0] = static_cast<uint16_t>(bf_round(f * cs[i] - g * sn[i]));
                dst[x][e1] = static_cast<uint16_t>(bf_round(f * sn[i] + g * cs[i]));
            }
        }
    }
}

cudaError_t launch_rotary(RotaryParams p, int num_sms, cudaStream_t stream) {
    if (p.num_tokens <= 0 || p.Hq + p.Hkv <= 0) return cudaSuccess;
    const int rot = 2 * p.half;
    const int layout = p.interleaved ? (rot % 8 == 0 ? kInterleavedVec : kPairs) : (rot % 16 == 0 ? kHalfVec : kPairs);
    // units of a head: the rotated ones, and the copied rest unless it lies in place
    const int rest = p.in_place ? 0 : p.D - rot;
    p.units = layout == kHalfVec ? p.half / 8 + rest / 8 : (layout == kInterleavedVec ? p.half / 4 + rest / 8 : p.half + rest);
    p.by_units = FastDiv::of(static_cast<uint32_t>(p.units));
    const bool store = p.slot_mapping != nullptr;
    const long long n = static_cast<long long>(p.Hq + p.Hkv) * p.units + (store ? static_cast<long long>(p.Hkv) * (p.D / 8) : 0);
    // A token is shared by several warps while there are fewer than 16 a SM.
    const long long want = (16ll * num_sms + p.num_tokens - 1) / p.num_tokens, most = (n + 31) / 32;
    p.parts = static_cast<int>(want < 1 ? 1 : (want > most ? most : want));
    const long long ctas = (p.num_tokens * p.parts + 7) / 8;
    const dim3 grid(static_cast<unsigned>(ctas));
#define GBATTN_ROTARY(L)                                                  \
    if (store)                                                            \
        rotary_sm103a<L, true><<<grid, 256, 0, stream>>>(p);              \
    else                                                                  \
        rotary_sm103a<L, false><<<grid, 256, 0, stream>>>(p)
    if (layout == kHalfVec) {
        GBATTN_ROTARY(kHalfVec);
    } else if (layout == kInterleavedVec) {
        GBATTN_ROTARY(kInterleavedVec);
    } else {
        GBATTN_ROTARY(kPairs);
    }
#undef GBATTN_ROTARY
    return cudaGetLastError();
}

}  // namespace gbattn
