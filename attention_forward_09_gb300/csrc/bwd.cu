// bwd.cu -- gradients of the fused attention for sm_103a (dense, padded and
// packed documents), from what the forward pass returned.
//
// With s_ij = scale q_i.k_j over the visible pairs, the probabilities are
// recomputed from the row's log-sum-exp and never stored:
//   p_ij    = exp(s_ij - lse_i)
//   delta_i = dout_i . out_i - dlse_i
//   ds_ij   = p_ij (dout_i.v_j - delta_i)
//   dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//
// Three kernels:
//   attn_bwd_stat_sm103a   -lse log2(e) and -delta of every query row and
//     head (fp32), one pass over out and dout, HBM-bound;
//   attn_bwd_sm103a, keys resident: a tile of 128 keys of one KV head stays
//     in shared memory while the queries of every head that shares it stream
//     by; S^T = K Q^T and dP^T = V dO^T go to TMEM, four warpgroups turn them
//     into P^T and dS^T (bf16, written over them), which are the A operands
//     of dV += P^T dO and dK += dS^T Q straight from TMEM;
//   attn_bwd_sm103a, queries resident: the same pipeline with the roles
//     exchanged: S = Q K^T, dP = dO V^T, dQ += dS K.
// A gradient row is summed by one CTA, or by a cluster whose sums are added in
// rank order, the heads of a group included, so results do not depend on
// timing: there are no atomics.  The price is that S and dP are formed twice,
// seven products for the five that one pass with atomics on dQ would need.
//
// DiT self-attention, 2 x 4096 rows, 24 heads, D = 128: 919 us a call, of them 18
// for the statistics, 462 and 409 for the two passes by themselves; 1.12 PFLOP/s
// of five products, 1.56 of the seven, at the power cap (1.83 GHz).
//
// P and dS are rounded to bf16 as operands of the second products, as P is in
// the forward kernels (at most 2^-8 of each term, independent of one another);
// lse, delta, P in ds = p (dp - delta) and every sum are fp32.
//
// Resident and streamed tiles are 128 rows.  Above D = 128 dV and dK do not fit
// in TMEM beside the scores: they are two launches of the keys-resident
// kernel, one accumulator each (eight products for five).
//
// Shared-memory layout and descriptors are those of the forward kernels: 64
// column chunks of [rows x 128 B], 128-byte swizzle; a streamed tile is read
// K-major by S / dP and MN-major by the second products.
#include <math.h>
#include <stddef.h>
#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace gbattn {

namespace {

// What a launch of attn_bwd_sm103a sums.
enum BwdMode {
    kBwdKV,  // keys resident: dV and dK
    kBwdV,   // keys resident: dV alone
    kBwdK,   // keys resident: dK alone
    kBwdQ,   // queries resident: dQ
    kBwdPasses
};

template <int D_, int MODE_>
struct BwdCfg {
    static constexpr int D = D_, MODE = MODE_;
    static constexpr int BM = 128, BN = 128;          // resident and streamed rows
    static constexpr bool KEYS = MODE != kBwdQ;       // keys resident, queries streamed
    static constexpr bool HAS_P = MODE == kBwdKV || MODE == kBwdV;  // sums dV
    static constexpr bool HAS_DS = MODE != kBwdV;     // needs dP; sums dK or dQ
    static constexpr int ACCS = MODE == kBwdKV ? 2 : 1;
    static constexpr int NCH = (D + 63) / 64;         // 64-column blocks of a tile
    static constexpr int R_BYTES = NCH * BM * 128;
    // A streamed tile comes in NCK chunks of CW columns, a slot of the ring each.
    static constexpr int NCK = D == 256 ? 2 : 1, CW = D / NCK, CCH = NCH / NCK;
    static constexpr int C_BYTES = CCH * BN * 128;
    // Above D = 128 S, dP and the accumulator do not fit beside what else is
    // needed: S and dP share their columns, and V (or dO) is held in tensor
    // memory as bf16 pairs, which leaves the ring room for a tile ahead.
    static constexpr bool SHARED = HAS_DS && D > 128;
    // Residents in tensor memory: r >= RT0.
    static constexpr int RT0 = SHARED ? 1 : (!KEYS && D == 64 ? 0 : 2);
    static constexpr int RES = HAS_DS ? 2 : 1;        // resident tiles: K (and V), or Q and dO
    static constexpr int RES_SMEM = RES < RT0 ? RES : RT0, RES_TMEM = RES - RES_SMEM;
    static constexpr int G0 = RES_TMEM * NCK;         // the first ring's loads that bring those
    // S and dP buffers.  Without dV the scores are free as soon as they have
    // been read, and dP gets the second buffer; with it S does, where it fits.
    static constexpr int DPB = HAS_DS && !HAS_P && !SHARED ? 2 : 1;
    static constexpr int SB = HAS_P && (2 + (HAS_DS ? 1 : 0)) * BN + ACCS * D <= 512 ? 2 : 1;
    static constexpr int T_S = 0;
    static constexpr int T_DP = SHARED ? 0 : SB * BN;
    static constexpr int T_ACC = T_DP + (HAS_DS ? DPB * BN : 0);
    static constexpr int T_RES = T_ACC + ACCS * D;
    static constexpr int ISSUERS = SHARED ? 1 : 2;    // warps that issue products
    static constexpr int STAT_BYTES = KEYS ? 2 * BN * 4 : 0;   // -lse log2 e, -delta of a streamed tile's rows
    static constexpr int STATS = D <= 64 ? 4 : 2;              // buffers of them
    static constexpr int MATH_WARPS = 16, MATH_WGS = MATH_WARPS / 4, H = BN / MATH_WGS;  // H columns a thread
    // setmaxnreg split of the 640 x 96 registers of the launch
    static constexpr int REG_MATH = 104, REG_OTHER = 64;
    static constexpr int THREADS = 32 * MATH_WARPS + 128;
    // slots of each ring that an item's gradients leave through
    static constexpr int STAGE1 = NCK, STAGE2 = ACCS == 2 ? NCK : 0;
    static constexpr int ITEMS = 3;                            // items published ahead
    // Empty items looked at (well under a microsecond each) before the roles that
    // wait for the next one hear that the producer is still at it: a wait is for
    // a pipeline that stands still, not for a long search.
    static constexpr int LOOKS = 4096;
    static constexpr int BARS_FIXED = 22 + 2 * ITEMS + 2 * STATS;
    static constexpr int RELEASES = HAS_DS && !SHARED ? 2 : 1;  // commits that release a slot
    static constexpr int ROOM = 232448 - RES_SMEM * R_BYTES - STATS * STAT_BYTES - 16 - ITEMS * 64 - BARS_FIXED * 8;
    static constexpr int FIT = ROOM / (C_BYTES + 16);
    static constexpr int SLOTS = FIT < 8 ? FIT : 8;
    // Two rings, for C1 and C2, since one is released in another order than the
    // other is needed.  dV alone uses a tile once each: one ring, in the order
    // of use.
    static constexpr int N2 = HAS_DS ? SLOTS * 2 / 5 : 0, N1 = SLOTS - N2;
    static constexpr int NUM_BARS = BARS_FIXED + 2 * SLOTS;
    static constexpr int O_C = RES_SMEM * R_BYTES;             // offsets in shared memory
    static constexpr int O_STAT = O_C + SLOTS * C_BYTES;
    static constexpr int O_BARS = O_STAT + STATS * STAT_BYTES;
    static constexpr int SMEM_BYTES = O_BARS + NUM_BARS * 8 + 16 + ITEMS * 64;
    static_assert(MATH_WARPS * 32 * REG_MATH + 128 * REG_OTHER <= THREADS * 96, "register split");
    static_assert(T_RES + RES_TMEM * D / 2 <= 512, "TMEM budget");
    static_assert(BM * ACCS * D * 4 <= SLOTS * C_BYTES, "a split item's sums over the ring");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(C_BYTES == CCH * BM * 128, "a slot holds a chunk of a gradient tile");
    static_assert(!HAS_DS || (N2 >= NCK && N1 > NCK && N1 >= G0), "the rings hold what the issuing warps wait for at once");
    static_assert(SMEM_BYTES > 116 * 1024, "one CTA an SM: it takes all TMEM columns");
    static_assert(NCH % NCK == 0 && D % 32 == 0 && (RES_TMEM == 0 || D % 64 == 0), "tile shape");
};

// One document's (or batch entry's) rows.
struct BwdDoc {
    int q_start, k_start;  // first rows in the tensors
    int Lq, Lk;            // rows used
    int Lq_all, Lk_all;    // rows to be written (padding included)
    bool bad;
};

__device__ __forceinline__ BwdDoc bwd_doc(const BwdParams& p, int doc, bool report) {
    BwdDoc d;
    d.bad = false;
    if (p.cu_q) {
        d.q_start = p.cu_q[doc];
        d.k_start = p.cu_k[doc];
        const int q_end = p.cu_q[doc + 1], k_end = p.cu_k[doc + 1];
        d.bad = d.q_start < 0 || q_end < d.q_start || q_end > p.Tq || d.k_start < 0 || k_end < d.k_start ||
                k_end > p.Tk || q_end - d.q_start > p.max_q || k_end - d.k_start > p.max_k;
        if (d.bad) {
            if (report && p.status) atomicOr(p.status, kDevBadSeqlen);
            return d;
        }
        d.Lq = d.Lq_all = q_end - d.q_start;
        d.Lk = d.Lk_all = k_end - d.k_start;
    } else {
        d.q_start = doc * p.max_q;
        d.k_start = doc * p.max_k;
        d.Lq = d.Lq_all = p.max_q;
        d.Lk = d.Lk_all = p.max_k;
        if (p.lens_q) {
            const int n = p.lens_q[doc];
            if ((n < 0 || n > p.max_q) && report && p.status) atomicOr(p.status, kDevBadSeqlen);
            d.Lq = min(max(n, 0), p.max_q);
        }
        if (p.lens_k) {
            const int n = p.lens_k[doc];
            if ((n < 0 || n > p.max_k) && report && p.status) atomicOr(p.status, kDevBadSeqlen);
            d.Lk = min(max(n, 0), p.max_k);
        }
    }
    return d;
}

// Where a document's row statistics begin within a head's array: multiples of
// four floats (a bulk copy starts on 16 bytes), never overlapping: the starts
// of documents n and n + 1 are at least len + 1 apart.
__device__ __forceinline__ long long bwd_stat_base(int q_start, int doc) {
    return (static_cast<long long>(q_start) + 4ll * doc + 3) & ~3ll;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// The products with descriptors given by their lower words: the upper one is
// the same for every operand here (8-row groups 1024 bytes apart, 128-byte
// swizzle; sdesc_sw128).  Half the registers of whole descriptors.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// 16 bytes that this kernel does not write.  ONCE: nor reads again (of a sector
// that a lane's two loads share, the second would come from L2 too).
template <bool ONCE>
__device__ __forceinline__ uint4 load16(const void* src) {
    uint4 v;
    if (ONCE)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(src));
    else
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(src));
    return v;
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

}  // namespace

// ------------------------------------------------------------- row statistics
// A CTA takes `rows` query rows of `heads` heads, 256 (row, head) pairs at
// most: rows of dout and out are read whole, LANES lanes a pair and UN pairs in
// flight a lane; the results cross shared memory, so that a head's statistics
// are read and written for eight rows or more at a time.
// HBM-bound: cross-attention of 16384 rows of 40 heads of 128 takes 51 us (346 MB,
// the copy's rate), eight packed documents 69 (four CTAs an SM leave registers
// for the loads in flight: 55 and 72 without the bound).
//   STRIDED: out lies by its strides (cross-attention from a transposed out: 53
// us).  (A contiguous one is read by dout's
// offsets: the strides take registers that the fp32 loads need, and a padded
// batch of D = 96 took 62 us for 57 with them.)
template <int D, bool F32, bool STRIDED>
__global__ void __launch_bounds__(256, 4) attn_bwd_stat_sm103a(const BwdParams p, const int rows, const int heads) {
    constexpr int LANES = D <= 64 ? 8 : (D <= 128 ? 16 : 32), UN = 4, PER_WARP = 32 / LANES;
    __shared__ float dots[256];
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < kBwdPasses) p.claims[threadIdx.x] = 0u;
    // Few CTAs: the next pass may set itself up beside them.  (Many: passes that
    // began while CTAs of this launch still came and went held their SMs, packed
    // causal 2696 -> 2800 us, so there it is the end that lets them begin.)
    const bool few = gridDim.x * gridDim.y * gridDim.z <= 128;
    if (few) grid_launch_dependents();
    const int doc = blockIdx.z;
    const BwdDoc d = bwd_doc(p, doc, threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0);
    if (d.bad) return;
    const long long i0 = static_cast<long long>(blockIdx.x) * rows;
    if (i0 >= d.Lq) return;
    const int h0 = blockIdx.y * heads, nh = min(heads, p.Hq - h0);
    const int nr = static_cast<int>(min(static_cast<long long>(rows), d.Lq - i0));
    // the pair that this thread finishes
    const int hp = threadIdx.x / rows;
    const long long ip = i0 + threadIdx.x % rows;
    const bool pair = hp < nh && ip < d.Lq;
    float lse = 0.f, dlse = 0.f;
    if (pair) {
        const long long at = doc * p.lse_bstride + (h0 + hp) * p.lse_hstride + (p.lse_row_global ? d.q_start + ip : ip);
        lse = p.lse[at];
        if (p.dlse) dlse = p.dlse[at];
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES;
    const long long first = ((d.q_start + i0) * p.Hq + h0) * D + sub * 8;
    const long long first_out = STRIDED ? doc * p.out_bstride + (p.cu_q ? d.q_start + i0 : i0) * p.out_rstride +
                                              h0 * p.out_hstride + sub * 8
                                        : first;
    const uint16_t* dout = static_cast<const uint16_t*>(p.dout) + first;
    const uint16_t* out = static_cast<const uint16_t*>(p.out) + (F32 ? 2 : 1) * first_out;
    constexpr int STEP = 8 * PER_WARP;  // pairs between one lane's loads
    const int total = nr * nh, step_i = STEP / nh, step_h = STEP % nh;
    int u = warp * PER_WARP + lane / LANES, i = u / nh, h = u % nh;
    while (u - lane / LANES < total) {
        uint4 g[UN], o[UN], o2[UN];
        int to[UN];  // in dots, or -1
#pragma unroll
        for (int x = 0; x < UN; ++x) {
            g[x] = o[x] = o2[x] = make_uint4(0u, 0u, 0u, 0u);
            to[x] = u < total ? h * rows + i : -1;
            if (u < total && sub * 8 < D) {
                const long long at = static_cast<long long>(i * p.Hq + h) * D;
                const long long at_out = STRIDED ? i * p.out_rstride + h * p.out_hstride : at;
                g[x] = load16<true>(dout + at);
                const uint4* src = reinterpret_cast<const uint4*>(out + (F32 ? 2 : 1) * at_out);
                o[x] = load16<!F32>(src);
                if (F32) o2[x] = load16<false>(src + 1);
            }
            u += STEP, i += step_i, h += step_h;
            if (h >= nh) h -= nh, ++i;
        }
        float acc[UN];
#pragma unroll
        for (int x = 0; x < UN; ++x) {
            const uint32_t gw[4] = {g[x].x, g[x].y, g[x].z, g[x].w};
            const uint32_t ow[8] = {o[x].x, o[x].y, o[x].z, o[x].w, o2[x].x, o2[x].y, o2[x].z, o2[x].w};
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum = __ffma2_rn(unpack_bf16x2(gw[e]),
                                 F32 ? make_float2(__uint_as_float(ow[2 * e]), __uint_as_float(ow[2 * e + 1]))
                                     : unpack_bf16x2(ow[e]),
                                 sum);
            acc[x] = sum.x + sum.y;
        }
        // Four sums over the lanes: each half of them goes on with two, each quarter
        // with one (five exchanges for 16 lanes instead of sixteen).
        const bool hi = sub & (LANES / 2), hi2 = sub & (LANES / 4);
        const float s0 = (hi ? acc[2] : acc[0]) + __shfl_xor_sync(0xffffffffu, hi ? acc[0] : acc[2], LANES / 2);
        const float s1 = (hi ? acc[3] : acc[1]) + __shfl_xor_sync(0xffffffffu, hi ? acc[1] : acc[3], LANES / 2);
        float s = (hi2 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, hi2 ? s0 : s1, LANES / 4);
#pragma unroll
        for (int m = LANES / 8; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        const int at = hi ? (hi2 ? to[3] : to[2]) : (hi2 ? to[1] : to[0]);
        if (sub % (LANES / 4) == 0 && at >= 0) dots[at] = s;
    }
    __syncthreads();
    if (pair) {
        const long long at = (h0 + hp) * p.stat_stride + bwd_stat_base(d.q_start, doc) + ip;
        // a row that sees no key (lse = -inf) has p = 2^(s - inf) = 0
        p.neg_lse2[at] = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
        p.neg_delta[at] = dlse - dots[threadIdx.x];
    }
    if (!few) grid_launch_dependents();
}

// ------------------------------------------------------------- the two passes
// 640 threads:
//   warps 0-15  math, four warpgroups: thread = one resident row (TMEM lane) and
//               32 of a streamed tile's 128 columns (four warps a scheduler: one's
//               latencies hide another's; two warpgroups of 64 columns were 3 %
//               slower at D = 64 and 20 % on a batch of a few tiles)
//   warp 16     TMA producer: claims items; resident tiles, then the tiles C1 (Q or K)
//   warp 17     TMEM allocator; issues S and dV (dV alone: S)
//   warp 18     TMA producer: the tiles C2 (dO or V), and with the keys resident
//               the streamed rows' statistics
//   warp 19     issues dP and dK or dQ (dV alone: dV)
// A product is issued about as fast as it runs, so what one issuing warp waits
// the other's products fill; the tensor core finishes what one thread issues
// in order.
//   dV and dK, D <= 128: S(0) | dV(j) S(j+1) after P(j)  and  dP(0) | dK(j)
//     dP(j+1) after dS(j).  With one S buffer the chain exponentials -> dV ->
//     S -> exponentials is the longest, so dK(j) and dP(j+1) also wait until
//     S(j+1) has been issued, and run beside the exponentials.
//   dQ, D <= 128: S(j+1) once S(j) has been read; dP(j+1), then dQ(j) after dS(j).
//   dV alone: S(j+1), then dV(j) after P(j).
//   dK or dQ, D > 128, S and dP in the same columns: S(j) | dP(j) once S(j) has
//     been read | after dS(j) the sum's product | S(j+1) ...
// P and dS (bf16 pairs) are written over columns that the same thread has read,
// so the warpgroups need not meet.
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    attn_bwd_sm103a(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmO1, const __grid_constant__ CUtensorMap tmO2,
                    const BwdParams p) {
    constexpr int D = C::D, BM = C::BM, BN = C::BN, NCH = C::NCH, NCK = C::NCK, CCH = C::CCH, SLOTS = C::SLOTS;
    constexpr int SB = C::SB, DPB = C::DPB, G0 = C::G0, MW = C::MATH_WARPS, WGS = C::MATH_WGS, H = C::H;
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzled tiles lie on 1024 bytes
    const uint32_t sR = smem_u32(smem);
    const uint32_t sC = sR + C::O_C;
    const uint32_t sStat = sR + C::O_STAT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::O_BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto b_res = [&](int r) { return smem_u32(&bars[r]); };
    auto b_s_full = [&](int b) { return smem_u32(&bars[2 + b]); };
    auto b_p_full = [&](int b) { return smem_u32(&bars[4 + b]); };  // P is there (without dV: S has been read)
    auto b_dp_full = [&](int b) { return smem_u32(&bars[6 + b]); };
    auto b_ds_full = [&](int b) { return smem_u32(&bars[8 + b]); };
    auto b_turn = [&](int b) { return smem_u32(&bars[10 + b]); };  // S(j + 1) has been issued (dV alone: dV(j) is done)
    const uint32_t b_done = smem_u32(&bars[12]), b_drain = smem_u32(&bars[13]), b_res_in = smem_u32(&bars[14]);
    const uint32_t b_acc_free = smem_u32(&bars[15]);  // the accumulators have been read
    auto b_res_free = [&](int r) { return smem_u32(&bars[16 + r]); };
    auto b_staged = [&](int a) { return smem_u32(&bars[18 + a]); };  // a gradient tile lies in its slots
    auto b_copied = [&](int a) { return smem_u32(&bars[20 + a]); };  // what goes row by row has been read from them
    auto b_item_full = [&](int b) { return smem_u32(&bars[22 + b]); };
    auto b_item_free = [&](int b) { return smem_u32(&bars[22 + C::ITEMS + b]); };
    auto b_stat_full = [&](int b) { return smem_u32(&bars[22 + 2 * C::ITEMS + b]); };
    auto b_stat_empty = [&](int b) { return smem_u32(&bars[22 + 2 * C::ITEMS + C::STATS + b]); };
    volatile int* const items = reinterpret_cast<volatile int*>(tmem_slot + 4);
    auto b_full = [&](int s) { return smem_u32(&bars[C::BARS_FIXED + s]); };
    auto b_empty = [&](int s) { return smem_u32(&bars[C::BARS_FIXED + SLOTS + s]); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ------------------------------------------------------------------ items
    // An item is a (tile, head, document).  Causal launches list them by falling
    // cost: tiles slowest (a document's first keys and last queries are seen
    // the most; a key tile is counted from its document's last one), heads
    // fastest.  Others have tiles fastest (neighbouring CTAs stream the same
    // head).  The C1 producer claims them in that order from a counter, p.chunk
    // at a time, and publishes each in shared memory; rings, barriers and
    // buffers carry on from item to item, so that the next item's loads and
    // first products overlap the present one's last ones and its epilogue.
    //   Launches of few items and many steps split each item's steps over a cluster
    // of `split` CTAs, one item a cluster; their sums are added on chip.
    const int split = p.split[C::KEYS ? 0 : 1], crank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int heads = C::KEYS ? p.Hkv : p.Hq;
    struct Item {
        int n;                     // steps; 0: zeros to write; kItemEnd: no more items
        int t_lo, t_hi;            // streamed tiles of each head
        int t_first, h_first;      // the first step's tile, and its head from the first streamed one
        int head, r0;              // resident head, first resident row within the document
        int diag;                  // causal: row i sees key j iff j <= i + diag
        int res_start, res_all, res_len, str_start, str_len;
        uint32_t stat;             // where the rows' statistics begin within a head's
    };
    constexpr int kItemEnd = -2;
    static_assert(sizeof(Item) <= 64, "an item's room");
    // The w-th word of the published item `it` (a count), by a role that has waited for it.
    auto word = [&](int it, int w) -> int { return items[(it % C::ITEMS) * 16 + w]; };
#define GBATTN_ITEM(it, field) word(it, static_cast<int>(offsetof(Item, field) / 4))
    // Wait for item `it`: its steps, or kItemEnd, or -1 where the wait gave up.
    auto next_item = [&](int it, bool all) -> int {
        bool got = mbar_wait(b_item_full(it % C::ITEMS), (it / C::ITEMS) & 1, abort_flag);
        if (all) got = __all_sync(0xffffffffu, got);
        return got ? GBATTN_ITEM(it, n) : -1;
    };
    // The i-th item (n = -1: nothing to write); how far on the next one is that
    // may have something (a tile past its document has none for any head, nor
    // have the tiles behind it).
    auto item_at = [&](uint32_t x, Item& it) -> uint32_t {
        it.n = -1;
        int tile, doc;
        uint32_t skip;
        if (p.causal) {
            it.head = x % heads;
            x /= heads;
            doc = x % p.num_docs;
            tile = x / p.num_docs;
            if (!C::KEYS) tile = p.tiles_q - 1 - tile;
            skip = heads - it.head;
        } else {
            const int tiles = C::KEYS ? p.tiles_k : p.tiles_q;
            tile = x % tiles;
            x /= tiles;
            it.head = x % heads;
            doc = x / heads;
            skip = tiles - tile;
        }
        const BwdDoc d = bwd_doc(p, doc, false);
        if (d.bad) return skip;
        it.res_all = C::KEYS ? d.Lk_all : d.Lq_all;
        if (C::KEYS && p.causal) tile -= p.tiles_k - (it.res_all + BM - 1) / BM;
        it.r0 = tile * BM;
        if (tile < 0 || it.r0 >= it.res_all) return skip;
        it.res_len = C::KEYS ? d.Lk : d.Lq;
        it.str_len = C::KEYS ? d.Lq : d.Lk;
        it.res_start = C::KEYS ? d.k_start : d.q_start;
        it.str_start = C::KEYS ? d.q_start : d.k_start;
        it.stat = static_cast<uint32_t>(bwd_stat_base(d.q_start, doc));
        it.diag = d.Lk - d.Lq;
        it.t_lo = 0;
        it.t_hi = (it.str_len + BN - 1) / BN;
        if (it.r0 >= it.res_len) {
            it.t_hi = 0;
        } else if (p.causal) {
            if (C::KEYS)
                it.t_lo = max(0, it.r0 - it.diag) / BN;  // the first row that sees key r0
            else
                it.t_hi = (max(0, min(d.Lk, min(it.r0 + BM, d.Lq) + it.diag)) + BN - 1) / BN;
        }
        it.n = max(0, it.t_hi - it.t_lo) * (C::KEYS ? p.group : 1);
        it.t_first = it.t_lo;
        it.h_first = 0;
        if (split > 1 && it.n > 0) {  // this CTA's share of the steps
            const int nt = it.t_hi - it.t_lo;
            const int j0 = static_cast<int>(static_cast<long long>(it.n) * crank / split);
            it.n = static_cast<int>(static_cast<long long>(it.n) * (crank + 1) / split) - j0;
            it.t_first += j0 % nt;
            it.h_first = j0 / nt;
        }
        return 1u;
    };
    // (a CTA of a cluster stays: the others read its shared memory)
    if (split == 1 && cta_has_timeout(p.status, kDevTimeout)) {
        grid_dependency_wait();
        return;
    }

    // ------------------------------------------------------------------ setup
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(b_res(b), 1);
            mbar_init(b_s_full(b), 1);
            mbar_init(b_p_full(b), MW);
            mbar_init(b_dp_full(b), 1);
            mbar_init(b_ds_full(b), MW);
            mbar_init(b_turn(b), 1);
            mbar_init(b_staged(b), MW / C::ACCS);
            mbar_init(b_copied(b), MW / C::ACCS);
        }
        mbar_init(b_done, C::HAS_DS ? C::ISSUERS : 1);
        mbar_init(b_drain, C::ISSUERS);
        mbar_init(b_res_in, MW);
        mbar_init(b_acc_free, MW);
        mbar_init(b_res_free(0), 1);
        mbar_init(b_res_free(1), 1);
        for (int b = 0; b < C::ITEMS; ++b) {
            mbar_init(b_item_full(b), 1);
            mbar_init(b_item_free(b), MW + C::ISSUERS + 1);
        }
        for (int b = 0; b < C::STATS; ++b) {
            mbar_init(b_stat_full(b), 1);
            mbar_init(b_stat_empty(b), MW);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(b_full(s), 1);
            mbar_init(b_empty(s), C::RELEASES);
        }
        *abort_flag = p.give_up ? 1 : 0;  // 1: give up every wait (failure-path test)
        fence_mbar_init();
    }
    if (warp == MW + 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    const CUtensorMap *mC1 = C::KEYS ? &tmQ : &tmK, *mC2 = C::KEYS ? &tmG : &tmV;
    // The first streamed head of resident head h.
    auto str_head = [&](int h) { return C::KEYS ? h * p.group : h / p.group; };
    // Slots [begin, begin + size) as a ring: load g is in slot begin + g % size.
    struct Ring {
        uint32_t base;  // shared memory of slot 0
        int s, begin, size, issued;
        uint32_t ph;    // parity of the slot's present turn
        __device__ Ring(uint32_t b, int bg, int sz) : base(b), s(bg), begin(bg), size(sz), issued(0), ph(0) {}
        __device__ void next() {
            ++issued;
            if (++s == begin + size) {
                s = begin;
                ph ^= 1u;
            }
        }
    };
    // Chunk of a tile into the ring's next slot, once that is free.
    auto load = [&](Ring& r, const CUtensorMap* m, int h, int row, int chunk) -> bool {
        if (r.issued >= r.size && !mbar_wait(b_empty(r.s), r.ph ^ 1u, abort_flag)) return false;
        mbar_arrive_expect_tx(b_full(r.s), C::C_BYTES);
        for (int c = 0; c < CCH; ++c)
            tma_load_3d(r.base + r.s * C::C_BYTES + c * (BN * 128), m, b_full(r.s), (chunk * CCH + c) * 64, h, row);
        r.next();
        return true;
    };
    // The ring's next slot, once free, for the math warps to write an item's gradients through.
    auto grant = [&](Ring& r) -> bool {
        if (r.issued >= r.size && !mbar_wait(b_empty(r.s), r.ph ^ 1u, abort_flag)) return false;
        mbar_arrive(b_full(r.s));
        r.next();
        return true;
    };
    auto drain = [&](const Ring& r) {
        for (int g = (r.issued > r.size ? r.issued - r.size : 0); g < r.issued; ++g)
            mbar_wait_drain(b_full(r.begin + g % r.size), (g / r.size) & 1);
    };
    int res_loads[2] = {0, 0};  // (of the producer: loads of each resident tile so far)
    if (warp >= MW) {
        regs_dec<C::REG_OTHER>();
        if (warp == MW && lane == 0) {
            // ---------------------------------- producer: resident tiles, then C1
            const CUtensorMap *mR1 = C::KEYS ? &tmK : &tmQ, *mR2 = C::KEYS ? &tmV : &tmG;
            Ring ring(sC, 0, C::N1);
            Item it;
            int done = 0;       // items with steps so far
            int published = 0;  // items published
            int looked = 0;     // empty ones since the last
            auto publish = [&]() -> bool {
                const int b = published % C::ITEMS;
                if (published >= C::ITEMS && !mbar_wait(b_item_free(b), (published / C::ITEMS - 1) & 1, abort_flag))
                    return false;
                for (int w = 0; w < static_cast<int>(sizeof(Item) / 4); ++w)
                    items[b * 16 + w] = reinterpret_cast<const int*>(&it)[w];
                mbar_arrive(b_item_full(b));
                ++published;
                return true;
            };
            tma_prefetch_desc(mR1);
            tma_prefetch_desc(mC1);
            if (C::RES > 1) tma_prefetch_desc(mR2);
            const uint32_t all = static_cast<uint32_t>(p.items[C::KEYS ? 0 : 1]), chunk = p.chunk[C::KEYS ? 0 : 1];
            uint32_t* const counter = p.claims + C::MODE;
            // A CTA's first items go by its number, so that their loads need not
            // wait for the launch that zeroes the counter; the next ones are
            // claimed before they are needed (the answer takes a while).
            uint32_t left = chunk, i = blockIdx.x / split * chunk, next = 0;
            bool claimed = false;
            auto claim = [&]() {
                if (p.early_wait) grid_dependency_wait();
                next = gridDim.x * chunk + atomicAdd(counter, chunk);
                claimed = true;
            };
#pragma unroll 1
            while (ok) {
                if (left == 0 && split > 1) {  // one item a cluster
                    i = all;
                } else if (left == 0) {
                    if (!claimed) claim();
                    i = next;
                    left = chunk;
                    claimed = false;
                }
                if (i >= all) {
                    it.n = kItemEnd;
                    ok = publish();
                    break;
                }
                const uint32_t by = min(item_at(i, it), left);
                i += by;
                left -= by;
                if (it.n < 0) {
                    if (++looked < C::LOOKS) continue;
                    it = Item{};  // an item without rows or steps
                }
                looked = 0;
                if (!(ok = publish())) break;
                if (it.n == 0) continue;
                for (int r = 0; r < C::RES; ++r) {
                    const CUtensorMap* m = r ? mR2 : mR1;
                    if (r >= C::RT0) {
                        for (int c = 0; c < NCK; ++c) ok = ok && load(ring, m, it.head, it.res_start + it.r0, c);
                    } else if (ok && (done == 0 || mbar_wait(b_res_free(r), (done - 1) & 1, abort_flag))) {
                        mbar_arrive_expect_tx(b_res(r), C::R_BYTES);
                        for (int c = 0; c < NCH; ++c)
                            tma_load_3d(sR + r * C::R_BYTES + c * (BM * 128), m, b_res(r), c * 64, it.head,
                                        it.res_start + it.r0);
                        res_loads[r] = done + 1;
                    } else {
                        ok = false;
                    }
                }
                int t = it.t_first, h = str_head(it.head) + it.h_first;
#pragma unroll 1
                for (int j = 0; ok && j < it.n; ++j) {
                    const int t2 = t, h2 = h;  // step j
                    if (++t == it.t_hi) {
                        t = it.t_lo;
                        ++h;
                    }
                    if (C::HAS_DS || j == 0)
                        for (int c = 0; ok && c < NCK; ++c) ok = load(ring, mC1, h2, it.str_start + t2 * BN, c);
                    if (!C::HAS_DS) {  // S(j + 1) comes before dV(j)
                        if (j + 1 < it.n)
                            for (int c = 0; ok && c < NCK; ++c) ok = load(ring, mC1, h, it.str_start + t * BN, c);
                        for (int c = 0; ok && c < NCK; ++c) ok = load(ring, mC2, h2, it.str_start + t2 * BN, c);
                    }
                }
                ++done;
                if (split > 1) continue;
                for (int c = 0; ok && c < C::STAGE1; ++c) ok = grant(ring);
                if (left == 0 && !claimed && ok) claim();
            }
            if (!ok || *abort_flag) {
                // Let every copy this thread started land before the CTA retires.
                for (int r = 0; r < C::RES_SMEM; ++r)
                    if (res_loads[r] > 0) mbar_wait_drain(b_res(r), (res_loads[r] - 1) & 1);
                drain(ring);
            }
        } else if (warp == MW + 2 && lane == 0) {
            // --------------------- producer: C2, and statistics of streamed rows
            tma_prefetch_desc(mC2);
            if (p.early_wait) grid_dependency_wait();  // the launch before this one writes the statistics
            grid_launch_dependents();
            Ring ring(sC, C::N1, C::N2);
            int issued = 0;
#pragma unroll 1
            for (int i = 0; ok; ++i) {
                const int n = next_item(i, false);
                if (n < 0) {
                    ok = n == kItemEnd;
                    break;
                }
                const int t_lo = GBATTN_ITEM(i, t_lo), t_hi = GBATTN_ITEM(i, t_hi), start = GBATTN_ITEM(i, str_start);
                const long long stat_base = static_cast<uint32_t>(GBATTN_ITEM(i, stat));
                int t = GBATTN_ITEM(i, t_first), h = str_head(GBATTN_ITEM(i, head)) + GBATTN_ITEM(i, h_first);
                mbar_arrive(b_item_free(i % C::ITEMS));
#pragma unroll 1
                for (int j = 0; ok && j < n; ++j) {
                    if (C::HAS_DS)
                        for (int c = 0; ok && c < NCK; ++c) ok = load(ring, mC2, h, start + t * BN, c);
                    if (C::KEYS && ok) {
                        const int b = issued % C::STATS;
                        if (issued >= C::STATS &&
                            !(ok = mbar_wait(b_stat_empty(b), (issued / C::STATS - 1) & 1, abort_flag)))
                            break;
                        const long long at = h * p.stat_stride + stat_base + static_cast<long long>(t) * BN;
                        mbar_arrive_expect_tx(b_stat_full(b), C::STAT_BYTES);
                        bulk_load(sStat + b * C::STAT_BYTES, p.neg_lse2 + at, BN * 4, b_stat_full(b));
                        bulk_load(sStat + b * C::STAT_BYTES + BN * 4, p.neg_delta + at, BN * 4, b_stat_full(b));
                        ++issued;
                    }
                    if (++t == t_hi) {
                        t = t_lo;
                        ++h;
                    }
                }
                for (int c = 0; ok && n > 0 && split == 1 && c < C::STAGE2; ++c) ok = grant(ring);
            }
            if (!ok || *abort_flag) {
                drain(ring);
                for (int g = (issued > C::STATS ? issued - C::STATS : 0); g < issued; ++g)
                    mbar_wait_drain(b_stat_full(g % C::STATS), (g / C::STATS) & 1);
            }
        } else if (warp == MW + 1 || (warp == MW + 3 && C::ISSUERS == 2)) {
            // ----------------------------------------------------------------- MMA
            // Each issuing warp walks its schedule as a whole; one elected lane issues.
            constexpr uint32_t kIdS = idesc_bf16_f32(BM, BN, false, false);
            constexpr uint32_t kIdA = idesc_bf16_f32(BM, C::CW, false, true);
            const bool first_warp = warp == MW + 1;
            const bool leader = elect_one();
            const uint32_t dR = desc_lo(sR, 16);
            const uint32_t dCk = desc_lo(sC, 16);           // streamed chunk, K-major
            const uint32_t dCm = desc_lo(sC, BN * 128);     // streamed chunk, MN-major
            auto wait_all = [&](uint32_t bar, uint32_t ph) {
                return __all_sync(0xffffffffu, mbar_wait(bar, ph, abort_flag));
            };
            // Rows of a streamed tile that no resident row may see at all (past the
            // document, the neighbours' rows, or rows without a key) may hold
            // anything; P and dS are 0 there but 0 * NaN is not, so they are zeroed
            // before the second product reads them.
            int item = 0, n = 0, edge_lo = 0, edge_hi = 0;  // tiles below edge_lo or from edge_hi on have such rows
            auto edge_rows = [&](int t) { return t < edge_lo || t >= edge_hi; };
            auto zero_rows = [&](int s, int t) {
                const int hi = min(BN, GBATTN_ITEM(item, str_len) - t * BN);
                const int lo = (C::KEYS && p.causal) ? min(hi, max(0, -GBATTN_ITEM(item, diag) - t * BN)) : 0;
                for (int x = lane; x < (lo + BN - hi) * CCH * 8; x += 32) {
                    const int u = x & 7, rc = x >> 3, c = rc % CCH, r = rc / CCH;
                    const int row = r < lo ? r : hi + r - lo;
                    st_shared_v4(sC + s * C::C_BYTES + c * (BN * 128) + row * 128 + u * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            // X (128 x BN) (+)= resident r * chunk c of a streamed tile, in slot s
            auto scores = [&](uint32_t to, int r, int c, int s) {
                uint32_t a = r >= C::RT0 ? tmem + C::T_RES + (r - C::RT0) * (D / 2) + c * (C::CW / 2)
                                         : dR + ((r * C::R_BYTES + c * CCH * BM * 128) >> 4);
                uint32_t b = dCk + s * (C::C_BYTES >> 4);
                asm volatile("" : "+r"(a), "+r"(b));  // (worked out here, not kept over the steps)
#pragma unroll
                for (int k = 0; k < C::CW / 16; ++k) {
                    const uint32_t off = ((k >> 2) * BN * 128 + (k & 3) * 32) >> 4, acc = (c > 0 || k > 0) ? 1u : 0u;
                    if (r >= C::RT0)
                        mma_ts(tmem + to, a + k * 8, b + off, kIdS, acc);
                    else
                        mma_ss(tmem + to, a + off, b + off, kIdS, acc);
                }
            };
            // columns [c CW, (c + 1) CW) of acc += A (bf16 pairs in X's columns, 16
            // of every 32) * chunk c of a streamed tile, in slot s
            auto accumulate = [&](uint32_t acc, uint32_t x, int c, int s, bool first) {
                uint32_t a = tmem + x, b = dCm + s * (C::C_BYTES >> 4);
                asm volatile("" : "+r"(a), "+r"(b));
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    mma_ts(tmem + acc + c * C::CW, a + (k >> 1) * 32 + (k & 1) * 8, b + ((k * 16 * 128) >> 4), kIdA,
                           (!first || k > 0) ? 1u : 0u);
            };
            // Cursors: the next chunk of C1 and of C2 that this warp uses.
            Ring c1(sC, 0, C::N1), c2(sC, C::N1, C::N2);
            auto moved = [](Ring r) {
                for (int c = 0; c < NCK; ++c) r.next();
                return r;
            };
            int J = 0;     // steps of the items so far: buffers and phases go by J + j
            int done = 0;  // items with steps so far
            auto acc_free = [&]() -> bool { return done == 0 || wait_all(b_acc_free, (done - 1) & 1); };
            ok = !*abort_flag;  // a launch told to give up issues nothing
#pragma unroll 1
            for (; ok; ++item) {
                n = next_item(item, true);
                if (n <= 0) {
                    if (n < 0) {
                        ok = n == kItemEnd;
                        break;
                    }
                    if (lane == 0) mbar_arrive(b_item_free(item % C::ITEMS));
                    continue;
                }
                const int t_lo = GBATTN_ITEM(item, t_lo), t_hi = GBATTN_ITEM(item, t_hi);
                edge_lo = C::KEYS && p.causal ? (max(0, -GBATTN_ITEM(item, diag)) + BN - 1) / BN : 0;
                edge_hi = GBATTN_ITEM(item, str_len) / BN;
                if (C::RES_TMEM > 0) {  // the math warps have copied those residents into tensor memory
                    ok = wait_all(b_res_in, done & 1);
                    for (int g = 0; g < G0; ++g) {
                        if (ok && lane == 0) mbar_arrive(b_empty(c1.s));
                        c1.next();
                    }
                    __syncwarp();
                }
                int t = GBATTN_ITEM(item, t_first);
                // All of a tile's chunks have landed.
                auto landed = [&](Ring s) -> bool {
                    for (int c = 0; c < NCK; ++c) {
                        if (!wait_all(b_full(s.s), s.ph)) return false;
                        s.next();
                    }
                    return true;
                };
                // S of a step from C1's chunks, released once read when `free_c1`.
                auto issue_s = [&](int j, Ring s, bool free_c1) {
                    for (int c = 0; c < NCK; ++c) {
                        scores(C::T_S + ((J + j) % SB) * BN, 0, c, s.s);
                        if (free_c1) mma_commit(b_empty(s.s));
                        s.next();
                    }
                    mma_commit(b_s_full((J + j) % SB));
                    if (C::RES_SMEM > 0 && j + 1 == n) mma_commit(b_res_free(0));
                };
                if constexpr (C::SHARED) {
                    // ---------------------------------- S and dP in the same columns
                    // S(j), chunk by chunk: the last ones come into slots released just before
                    auto next_s = [&](int j) -> bool {
                        Ring s = c1;
                        for (int c = 0; c < NCK; ++c) {
                            if (!wait_all(b_full(s.s), s.ph)) return false;
                            tc_fence_after();
                            if (leader) {
                                scores(C::T_S, 0, c, s.s);
                                if (c == NCK - 1) mma_commit(b_s_full(0));
                                if (c == NCK - 1 && j + 1 == n) mma_commit(b_res_free(0));
                            }
                            __syncwarp();
                            s.next();
                        }
                        return true;
                    };
                    ok = ok && wait_all(b_res(0), done & 1) && next_s(0);
                    for (int j = 0; ok && j < n; ++j) {
                        if (!(ok = landed(c2) && wait_all(b_p_full(0), (J + j) & 1))) break;
                        tc_fence_after();
                        if (leader) {
                            Ring s = c2;
                            for (int c = 0; c < NCK; ++c) {
                                scores(C::T_DP, 1, c, s.s);
                                mma_commit(b_empty(s.s));
                                s.next();
                            }
                            mma_commit(b_dp_full(0));
                        }
                        __syncwarp();
                        c2 = moved(c2);
                        if (edge_rows(t)) {
                            Ring s = c1;
                            for (int c = 0; c < NCK; ++c) {
                                zero_rows(s.s, t);
                                s.next();
                            }
                        }
                        if (!(ok = (j > 0 || acc_free()) && wait_all(b_ds_full(0), (J + j) & 1))) break;
                        tc_fence_after();
                        if (leader) {
                            Ring s = c1;
                            for (int c = 0; c < NCK; ++c) {
                                accumulate(C::T_ACC, C::T_DP, c, s.s, j == 0);
                                mma_commit(b_empty(s.s));
                                s.next();
                            }
                        }
                        __syncwarp();
                        c1 = moved(c1);
                        if (j + 1 < n && !(ok = next_s(j + 1))) break;
                        if (++t == t_hi) t = t_lo;
                    }
                } else if constexpr (!C::HAS_DS) {
                    // ------------------------------------ dV alone: one ring, S(j + 1) before dV(j)
                    if (first_warp) {
                        ok = ok && wait_all(b_res(0), done & 1);
                        for (int j = 0; ok && j < n; ++j) {
                            if (!(ok = landed(c1))) break;
                            // the buffer's P has been used up
                            const int g = J + j - SB;
                            if (g >= 0 && !(ok = wait_all(b_turn(g % SB), (g / SB) & 1))) break;
                            tc_fence_after();
                            if (leader) issue_s(j, c1, true);
                            __syncwarp();
                            c1 = moved(c1);
                            if (j > 0 || n == 1) c1 = moved(c1);  // past dout's tile
                        }
                        if (n > 1) c1 = moved(c1);
                    } else {
                        c1 = moved(c1);
                        if (n > 1) c1 = moved(c1);
                        for (int j = 0; ok && j < n; ++j) {
                            // P(j) first: the slots' last turns were S(j)'s tiles or
                            // earlier ones, and a wait by parity is exact only once
                            // those have landed.
                            if (!(ok = (j > 0 || acc_free()) &&
                                       wait_all(b_p_full((J + j) % SB), ((J + j) / SB) & 1) && landed(c1)))
                                break;
                            if (edge_rows(t)) {
                                Ring s = c1;
                                for (int c = 0; c < NCK; ++c) {
                                    zero_rows(s.s, t);
                                    s.next();
                                }
                            }
                            tc_fence_after();
                            if (leader) {
                                Ring s = c1;
                                for (int c = 0; c < NCK; ++c) {
                                    accumulate(C::T_ACC, C::T_S + ((J + j) % SB) * BN, c, s.s, j == 0);
                                    mma_commit(b_empty(s.s));
                                    s.next();
                                }
                                mma_commit(b_turn((J + j) % SB));
                            }
                            __syncwarp();
                            c1 = moved(c1);
                            if (j + 2 < n) c1 = moved(c1);  // past the queries' tile of step j + 2
                            if (++t == t_hi) t = t_lo;
                        }
                    }
                } else if (first_warp) {
                    // -------------------------------------------------- S (and dV)
                    if (C::RT0 > 0) ok = ok && wait_all(b_res(0), done & 1);
                    ok = ok && wait_all(b_full(c1.s), c1.ph);
                    if (ok) {
                        tc_fence_after();
                        if (leader) issue_s(0, c1, true);
                        __syncwarp();
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        const bool more = j + 1 < n;
                        c1.next();
                        if (more && !(ok = wait_all(b_full(c1.s), c1.ph))) break;
                        if (SB == 2) {  // dV(j - 1), which read the buffer, was issued here
                            tc_fence_after();
                            if (more && leader) issue_s(j + 1, c1, true);
                            __syncwarp();
                        }
                        if (C::HAS_P) {
                            if (!(ok = wait_all(b_full(c2.s), c2.ph) && (j > 0 || acc_free()))) break;
                            if (edge_rows(t)) zero_rows(c2.s, t);
                        }
                        if (!(ok = wait_all(b_p_full((J + j) % SB), ((J + j) / SB) & 1))) break;
                        tc_fence_after();
                        if (leader) {
                            if (C::HAS_P) {
                                accumulate(C::T_ACC, C::T_S + ((J + j) % SB) * BN, 0, c2.s, j == 0);
                                mma_commit(b_empty(c2.s));
                            }
                            if (more && SB == 1) issue_s(j + 1, c1, true);
                            if (C::HAS_P && SB == 1) mbar_arrive(b_turn((J + j) & 1));
                        }
                        __syncwarp();
                        c2.next();
                        if (++t == t_hi) t = t_lo;
                    }
                } else {
                    // --------------------------------------------- dP and dK or dQ
                    constexpr uint32_t kAcc = C::T_ACC + (C::HAS_P ? D : 0);
                    auto issue_dp = [&](int j) {
                        scores(C::T_DP + ((J + j) % DPB) * BN, 1, 0, c2.s);
                        mma_commit(b_empty(c2.s));
                        if (!C::HAS_P) mma_commit(b_empty(c2.s));  // (a slot is released twice)
                        mma_commit(b_dp_full((J + j) % DPB));
                        if (C::RES_SMEM > 1 && j + 1 == n) mma_commit(b_res_free(1));
                    };
                    if (C::RT0 > 1) ok = ok && wait_all(b_res(1), done & 1);
                    ok = ok && wait_all(b_full(c2.s), c2.ph);
                    if (ok) {
                        tc_fence_after();
                        if (leader) issue_dp(0);
                        __syncwarp();
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        const bool more = j + 1 < n;
                        c2.next();
                        if (edge_rows(t)) {
                            if (!(ok = wait_all(b_full(c1.s), c1.ph))) break;
                            zero_rows(c1.s, t);
                        }
                        if (more && !(ok = wait_all(b_full(c2.s), c2.ph))) break;
                        if (DPB == 2) {  // the product that read the buffer's dS(j - 1) was issued here
                            tc_fence_after();
                            if (more && leader) issue_dp(j + 1);
                            __syncwarp();
                        }
                        if (!(ok = (j > 0 || acc_free()) && wait_all(b_ds_full((J + j) % DPB), ((J + j) / DPB) & 1))) break;
                        if (C::HAS_P && SB == 1 && !(ok = wait_all(b_turn((J + j) & 1), ((J + j) >> 1) & 1))) break;
                        tc_fence_after();
                        if (leader) {
                            accumulate(kAcc, C::T_DP + ((J + j) % DPB) * BN, 0, c1.s, j == 0);
                            mma_commit(b_empty(c1.s));
                            if (more && DPB == 1) issue_dp(j + 1);
                        }
                        __syncwarp();
                        c1.next();
                        if (++t == t_hi) t = t_lo;
                    }
                }
                // (dV alone: the warp that issues S runs an item ahead, and its commits would count for this one)
                if (ok && leader && (C::HAS_DS || !first_warp)) mma_commit(b_done);
                __syncwarp();
                if (lane == 0) mbar_arrive(b_item_free(item % C::ITEMS));
                for (int c = 0; c < C::STAGE1; ++c) c1.next();
                for (int c = 0; c < C::STAGE2; ++c) c2.next();
                J += n;
                ++done;
            }
            // Everything issued above must finish before TMEM is released.
            if (leader) mma_commit(b_drain);
            __syncwarp();
            mbar_wait_drain(b_drain, 0);
        }
        if (split > 1) {  // with the math warps
            cluster_sync();
            cluster_sync();
        }
    } else {
        regs_inc<C::REG_MATH>();
        // ---------------------------------------------------------------- math
        const int wg = warp >> 2;
        const int r = (warp & 3) * 32 + lane;   // resident row within the tile == TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const float c2 = p.scale_log2;
        if (!C::KEYS && p.early_wait) grid_dependency_wait();  // the launch before this one writes the statistics
        int J = 0;     // steps of the items so far: buffers and phases go by J + j
        int done = 0;  // items with steps so far
        Ring ring1(sC, 0, C::N1), ring2(sC, C::N1, C::N2);  // where the next item's loads begin
        auto ahead = [](Ring& r, int by) {
            const int x = r.s - r.begin + by;
            r.s = r.begin + x % r.size;
            r.ph ^= (x / r.size) & 1;
        };
        // An item's gradients leave through ring slots by TMA; the thread that
        // stores one gives its slots back once they have been read, which it
        // looks after in the next item's first step.  (Where the next item's
        // first tiles themselves need those slots, before it: RES_TMEM.)
        constexpr int PARTS = WGS / C::ACCS;                // warpgroups that share an accumulator
        const int acc = wg / PARTS, part = wg % PARTS;
        const bool storer = lane == 0 && warp % (4 * PARTS) == 0;
        int leaving = -1;  // the first of the slots that are being read
        bool have = false; // (split) there is an item
        auto give_back = [&]() {
            if (storer && leaving >= 0) {
                bulk_wait_read0();
                ok = mbar_wait(b_copied(acc), (done - 1) & 1, abort_flag);
                int s = leaving;
                for (int c = 0; c < NCK; ++c) {
                    for (int x = 0; x < C::RELEASES; ++x) mbar_arrive(b_empty(s));
                    if (++s == (acc ? C::N1 + C::N2 : C::N1)) s = acc ? C::N1 : 0;
                }
                leaving = -1;
            }
        };
#pragma unroll 1
        for (int item = 0; ok; ++item) {
            const int n = next_item(item, true);
            if (n < 0) {
                ok = n == kItemEnd;
                break;
            }
            const int row = GBATTN_ITEM(item, r0) + r;  // within the document
            float row_nl = -INFINITY, row_nd = 0.f;
            if (!C::KEYS && row < GBATTN_ITEM(item, res_len)) {
                const long long at =
                    GBATTN_ITEM(item, head) * p.stat_stride + static_cast<uint32_t>(GBATTN_ITEM(item, stat)) + row;
                row_nl = p.neg_lse2[at];
                row_nd = p.neg_delta[at];
            }
            if (n > 0) {
                give_back();
                ok = __all_sync(0xffffffffu, ok);
            }
            if (C::RES_TMEM > 0 && n > 0) {
                // residents that go to tensor memory: the warpgroups copy 64-column blocks in turn
                for (int b = wg; ok && b < C::RES_TMEM * NCH; b += WGS) {
                    Ring at = ring1;  // blocks lie in the order they were loaded
                    for (int c = 0; c < b / CCH; ++c) at.next();
                    const int s = at.s;
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait(b_full(s), at.ph, abort_flag)))) break;
                    const uint32_t src = sC + s * C::C_BYTES + (b % CCH) * (BM * 128) + r * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[16];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 x = ld_shared_f4(src + (((h * 4 + u) ^ (r & 7)) << 4));
                            w[4 * u] = __float_as_uint(x.x), w[4 * u + 1] = __float_as_uint(x.y);
                            w[4 * u + 2] = __float_as_uint(x.z), w[4 * u + 3] = __float_as_uint(x.w);
                        }
                        tmem_st16(tl + C::T_RES + b * 32 + h * 16, w);
                    }
                }
                if (ok) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_res_in);
                }
            }
            // this row sees (or is seen by) streamed rows [see_lo, see_hi)
            const int diag = GBATTN_ITEM(item, diag), str_len = GBATTN_ITEM(item, str_len), r0 = GBATTN_ITEM(item, r0);
            const int see_lo = C::KEYS && p.causal ? row - diag : 0;
            const int see_hi = !C::KEYS && p.causal ? min(str_len, row + diag + 1) : str_len;
            const int t_lo = GBATTN_ITEM(item, t_lo), t_hi = GBATTN_ITEM(item, t_hi);
            int t = GBATTN_ITEM(item, t_first);
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                const int g = J + j, sb = g % SB, db = g % DPB;
                const int c0 = t * BN + wg * H;  // this thread's first streamed row
                const int lo = see_lo - c0, hi = see_hi - c0;
                const bool edge = __any_sync(0xffffffffu, lo > 0 || hi < H);
                const uint32_t st = sStat + (g % C::STATS) * C::STAT_BYTES + wg * (H * 4);
                const uint32_t tS = tl + C::T_S + sb * BN + wg * H, tDP = tl + C::T_DP + db * BN + wg * H;
                if (C::KEYS) ok = ok && mbar_wait(b_stat_full(g % C::STATS), (g / C::STATS) & 1, abort_flag);
                if (!(ok = __all_sync(0xffffffffu, ok && mbar_wait(b_s_full(sb), (g / SB) & 1, abort_flag)))) break;
                tc_fence_after();
                uint32_t pr[H];  // P, fp32
#pragma unroll
                for (int c = 0; c < H; c += 32) tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&pr[c]));
                tmem_wait_ld();
                if (!C::HAS_P) {  // the S buffer may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_p_full(sb));
                }
                const float2 cc = make_float2(c2, c2);
#pragma unroll
                for (int c = 0; c < H; c += 32) {
#pragma unroll
                    for (int e = c; e < c + 32; e += 4) {
                        float4 nl = make_float4(row_nl, row_nl, row_nl, row_nl);
                        if (C::KEYS) nl = ld_shared_f4(st + e * 4);
                        const float2 a = __ffma2_rn(make_float2(__uint_as_float(pr[e]), __uint_as_float(pr[e + 1])), cc,
                                                    make_float2(nl.x, nl.y));
                        const float2 b = __ffma2_rn(make_float2(__uint_as_float(pr[e + 2]), __uint_as_float(pr[e + 3])), cc,
                                                    make_float2(nl.z, nl.w));
                        pr[e] = __float_as_uint(ex2(a.x));
                        pr[e + 1] = __float_as_uint(ex2(a.y));
                        pr[e + 2] = __float_as_uint(ex2(b.x));
                        pr[e + 3] = __float_as_uint(ex2(b.y));
                    }
                    if (edge) {
#pragma unroll
                        for (int e = c; e < c + 32; ++e)
                            if (e < lo || e >= hi) pr[e] = 0u;
                    }
                    if (C::HAS_P) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack_bf16x2(__uint_as_float(pr[c + 2 * e]), __uint_as_float(pr[c + 2 * e + 1]));
                        tmem_st16(tS + c, pk);
                    }
                }
                if (C::HAS_P) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_p_full(sb));
                }
                if (C::HAS_DS) {
                    if (!(ok = __all_sync(0xffffffffu, ok && mbar_wait(b_dp_full(db), (g / DPB) & 1, abort_flag)))) break;
                    tc_fence_after();
                    uint32_t dp[H];
#pragma unroll
                    for (int c = 0; c < H; c += 32) tmem_ld32(tDP + c, *reinterpret_cast<uint32_t(*)[32]>(&dp[c]));
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < H; c += 32) {
#pragma unroll
                        for (int e = c; e < c + 32; e += 4) {
                            float4 nd = make_float4(row_nd, row_nd, row_nd, row_nd);
                            if (C::KEYS) nd = ld_shared_f4(st + BN * 4 + e * 4);
                            float2 a = __fadd2_rn(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])),
                                                  make_float2(nd.x, nd.y));
                            float2 b = __fadd2_rn(make_float2(__uint_as_float(dp[e + 2]), __uint_as_float(dp[e + 3])),
                                                  make_float2(nd.z, nd.w));
                            a = __fmul2_rn(a, make_float2(__uint_as_float(pr[e]), __uint_as_float(pr[e + 1])));
                            b = __fmul2_rn(b, make_float2(__uint_as_float(pr[e + 2]), __uint_as_float(pr[e + 3])));
                            dp[e] = __float_as_uint(a.x);
                            dp[e + 1] = __float_as_uint(a.y);
                            dp[e + 2] = __float_as_uint(b.x);
                            dp[e + 3] = __float_as_uint(b.y);
                        }
                        if (edge) {  // 0 * (anything) is not always 0
#pragma unroll
                            for (int e = c; e < c + 32; ++e)
                                if (e < lo || e >= hi) dp[e] = 0u;
                        }
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack_bf16x2(__uint_as_float(dp[c + 2 * e]), __uint_as_float(dp[c + 2 * e + 1]));
                        tmem_st16(tDP + c, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_ds_full(db));
                }
                if (C::KEYS) {  // the statistics' buffer may be filled again
                    if (!C::HAS_DS) __syncwarp();
                    if (lane == 0) mbar_arrive(b_stat_empty(g % C::STATS));
                }
                if (++t == t_hi) t = t_lo;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (ok && n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(b_done, done & 1, abort_flag));
                tc_fence_after();
            }
            // ------------------------------------------------------------ epilogue
            // An accumulator's 32 column chunks are taken in turn by its warpgroups.
            // Rows are staged in the ring's slots, in the boxes' swizzle, and leave
            // by TMA where the tile lies wholly inside its document, else row by row.
            if (split > 1) {  // the sums, or zeros, as fp32 rows over the ring, 16-byte pieces swizzled by row
                constexpr int P = C::ACCS * D / 4;  // pieces of a row
                const uint32_t to = sC + static_cast<uint32_t>(r) * (P * 16);
#pragma unroll 1
                for (int x = wg; x < C::ACCS * D / 32; x += WGS) {
                    uint32_t o[32];
                    if (ok && n > 0) {
                        tmem_ld32(tl + C::T_ACC + x * 32, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        st_shared_v4(to + (((x * 8 + e) ^ (r & 7)) << 4), o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                have = true;
            } else if (ok) {
                const int res_all = GBATTN_ITEM(item, res_all), res_len = GBATTN_ITEM(item, res_len);
                const int head = GBATTN_ITEM(item, head), res_start = GBATTN_ITEM(item, res_start);
                const bool is_dv = C::MODE == kBwdV || (C::MODE == kBwdKV && acc == 0);
                const float f = is_dv ? 1.f : p.scale;
                uint16_t* const out = static_cast<uint16_t*>(C::KEYS ? (is_dv ? p.dv : p.dk) : p.dq);
                auto row_ptr = [&](int i) { return out + ((static_cast<long long>(res_start) + r0 + i) * heads + head) * D; };
                const int tid = (warp & 3) * 32 + lane + part * 128;  // among the threads that share the accumulator
                constexpr int THR = 128 * PARTS, U = D / 8;            // 16-byte pieces of a row
                const int rows = min(BM, res_all - r0);
                if (n == 0) {
                    for (int x = tid; x < rows * U; x += THR) st_global_v4(row_ptr(x / U) + (x % U) * 8, 0u, 0u, 0u, 0u);
                } else {
                    ahead(ring1, G0 + n * NCK * (C::HAS_DS ? 1 : 2));
                    if (C::ACCS == 2) ahead(ring2, n * NCK);
                    const Ring stage = acc ? ring2 : ring1;
                    Ring at = stage;
                    const bool used = row < res_len;
#pragma unroll 1
                    for (int c = 0; c < NCK; ++c) {
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait(b_full(at.s), at.ph, abort_flag)))) break;
                        const uint32_t to = sC + at.s * C::C_BYTES + r * 128;
#pragma unroll 1
                        for (int x = part; x < C::CW / 32; x += PARTS) {
                            uint32_t o[32];
                            tmem_ld32(tl + C::T_ACC + acc * D + c * C::CW + x * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                uint32_t w[4];
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const int e = 8 * u + 2 * y;
                                    w[y] = used ? pack_bf16x2(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f) : 0u;
                                }
                                st_shared_v4(to + (x >> 1) * (BM * 128) + ((((x & 1) * 4 + u) ^ (r & 7)) << 4), w[0], w[1],
                                             w[2], w[3]);
                            }
                        }
                        at.next();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_acc_free);  // the next item may sum
                    fence_proxy_async_smem();                // generic-proxy writes -> the TMA engine
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_staged(acc));
                    if (ok && (storer || rows < BM)) ok = mbar_wait(b_staged(acc), done & 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && rows == BM) {
                        if (storer) {
                            at = stage;
                            for (int c = 0; c < NCK; ++c) {
                                for (int b = 0; b < CCH; ++b)
                                    tma_store_3d(acc ? &tmO2 : &tmO1, sC + at.s * C::C_BYTES + b * (BM * 128),
                                                 (c * CCH + b) * 64, head, res_start + r0);
                                at.next();
                            }
                            bulk_commit();
                            leaving = stage.s;
                        }
                    } else if (ok) {
                        for (int x = tid; x < rows * U; x += THR) {
                            const int i = x / U, u = x % U, b = u / 8;
                            at = stage;
                            for (int c = 0; c < b / CCH; ++c) at.next();
                            const float4 v = ld_shared_f4(sC + at.s * C::C_BYTES + (b % CCH) * (BM * 128) + i * 128 +
                                                          (((u & 7) ^ (i & 7)) << 4));
                            st_global_v4(row_ptr(i) + u * 8, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                                         __float_as_uint(v.w));
                        }
                        if (storer) leaving = stage.s;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_copied(acc));
                    ahead(ring1, C::STAGE1);
                    if (C::ACCS == 2) ahead(ring2, C::STAGE2);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_item_free(item % C::ITEMS));
            if (n > 0) {
                J += n;
                ++done;
            }
        }
        give_back();
        if (split > 1) {
            cluster_sync();
            if (ok && have) {
                // CTA c adds up rows [c R, (c + 1) R) over the cluster, in rank order
                constexpr int P = C::ACCS * D / 4;
                const int R = BM / split, r0 = GBATTN_ITEM(0, r0);
                const int res_all = GBATTN_ITEM(0, res_all), res_len = GBATTN_ITEM(0, res_len);
                const long long row0 = static_cast<long long>(GBATTN_ITEM(0, res_start)) + r0;
                for (int x = threadIdx.x; x < R * P; x += MW * 32) {
                    const int i = crank * R + x / P, piece = x % P;
                    if (r0 + i >= res_all) continue;
                    const uint32_t at = sC + static_cast<uint32_t>(i) * (P * 16) + ((piece ^ (i & 7)) << 4);
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = 0; c < split; ++c) {
                        const float4 v = ld_cluster_f4(mapa_shared(at, c));
                        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                    }
                    const bool is_dv = C::MODE == kBwdV || (C::MODE == kBwdKV && piece < D / 4);
                    const float f = r0 + i >= res_len ? 0.f : (is_dv ? 1.f : p.scale);
                    uint16_t* out = static_cast<uint16_t*>(C::KEYS ? (is_dv ? p.dv : p.dk) : p.dq) +
                                    ((row0 + i) * heads + GBATTN_ITEM(0, head)) * D + piece % (D / 4) * 4;
                    *reinterpret_cast<uint2*>(out) =
                        f == 0.f ? make_uint2(0u, 0u)
                                 : make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
                }
            }
            cluster_sync();  // no CTA leaves while another still reads its shared memory
        }
    }

    // --------------------------------------------------------------- teardown
    if (!ok) {
        *abort_flag = 1;
        if (p.status) atomicOr(p.status, kDevTimeout);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MW + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // A launch that began beside the one before it ends after it.
    grid_dependency_wait();
#undef GBATTN_ITEM
}

// ------------------------------------------------------------------- launches
long long bwd_stat_stride(long long Tq, int num_docs) {
    // rows, the documents' alignment, and a last tile that is read whole
    return ((Tq + 4ll * num_docs + 3) & ~3ll) + 128;
}

namespace {

// The kernel's shared memory, asked for once a device.
template <class C>
cudaError_t allow_smem() {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(attn_bwd_sm103a<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

// One pass, behind the launch that writes the statistics (early_wait) or beside
// another pass: its CTAs take the SMs that one's leave.
template <class C>
cudaError_t launch_pass(const BwdMaps& m, const CUtensorMap& o1, const CUtensorMap& o2, BwdParams& p, int num_sms,
                        cudaStream_t stream) {
    const long long items = p.items[C::KEYS ? 0 : 1];
    if (items == 0) return cudaSuccess;
    cudaError_t e = allow_smem<C>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    const int split = p.split[C::KEYS ? 0 : 1];
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = split;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(split > 1 ? items * split : (items < num_sms ? items : num_sms)));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, attn_bwd_sm103a<C>, m.q, m.dout, m.k, m.v, o1, o2, static_cast<const BwdParams&>(p));
    p.early_wait = 0;
    return e;
}

template <int D>
cudaError_t launch_d(const BwdMaps& m, BwdParams& p, int num_sms, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    // 256 pairs a CTA: up to 32 heads, and a power of two rows, eight at least
    const int heads = p.Hq < 32 ? p.Hq : 32;
    int rows = 8;
    while (2 * rows * heads <= 256) rows *= 2;
    // (without query rows one CTA a document still looks at its boundaries)
    const dim3 grid(static_cast<unsigned>(p.max_q > 0 ? (p.max_q - 1) / rows + 1 : 1),
                    static_cast<unsigned>((p.Hq + heads - 1) / heads), static_cast<unsigned>(p.num_docs));
    const long long row = static_cast<long long>(p.Hq) * D;
    const bool strided = p.out_rstride != row || (p.Hq > 1 && p.out_hstride != D) ||
                         (!p.cu_q && p.num_docs > 1 && p.out_bstride != p.max_q * row);
    if (p.out_f32 && strided)
        attn_bwd_stat_sm103a<D, true, true><<<grid, 256, 0, stream>>>(p, rows, heads);
    else if (p.out_f32)
        attn_bwd_stat_sm103a<D, true, false><<<grid, 256, 0, stream>>>(p, rows, heads);
    else if (strided)
        attn_bwd_stat_sm103a<D, false, true><<<grid, 256, 0, stream>>>(p, rows, heads);
    else
        attn_bwd_stat_sm103a<D, false, false><<<grid, 256, 0, stream>>>(p, rows, heads);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    p.early_wait = 1;
    if constexpr (D <= 128) {
        e = launch_pass<BwdCfg<D, kBwdKV>>(m, m.dv, m.dk, p, num_sms, stream);
    } else {
        e = launch_pass<BwdCfg<D, kBwdV>>(m, m.dv, m.dv, p, num_sms, stream);
        if (e == cudaSuccess) e = launch_pass<BwdCfg<D, kBwdK>>(m, m.dk, m.dk, p, num_sms, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_pass<BwdCfg<D, kBwdQ>>(m, m.dq, m.dq, p, num_sms, stream);
}

}  // namespace

cudaError_t launch_bwd(int D, const BwdMaps& m, BwdParams p, int num_sms, cudaStream_t stream) {
    p.items[0] = static_cast<long long>(p.tiles_k) * p.Hkv * p.num_docs;
    p.items[1] = static_cast<long long>(p.tiles_q) * p.Hq * p.num_docs;
    // One item a claim until there are 64 a CTA (many short documents under a
    // long bound: most are empty, and a claim costs more than a look at them).
    for (int x = 0; x < 2; ++x) {
        const long long c = p.items[x] / (64ll * num_sms);
        p.chunk[x] = static_cast<uint32_t>(c < 1 ? 1 : (c > 1024 ? 1024 : c));
        // Half the SMs or fewer busy, with items of eight steps or more: as many
        // CTAs an item as fill the SMs, four steps each at least.
        const long long steps = x == 0 ? static_cast<long long>(p.tiles_q) * p.group : p.tiles_k;
        p.split[x] = 1;
        while (p.split[x] < 8 && p.items[x] * p.split[x] * 2 <= num_sms && steps >= 8ll * p.split[x]) p.split[x] *= 2;
    }
    switch (D) {
        case 64: return launch_d<64>(m, p, num_sms, stream);
        case 96: return launch_d<96>(m, p, num_sms, stream);
        case 128: return launch_d<128>(m, p, num_sms, stream);
        case 192: return launch_d<192>(m, p, num_sms, stream);
        case 256: return launch_d<256>(m, p, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbattn
