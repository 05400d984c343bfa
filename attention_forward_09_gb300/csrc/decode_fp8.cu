// decode_fp8.cu -- paged decode over the 8-bit KV cache for sm_103a: one new
// query token a sequence attends its context, read as the codes and exponent
// bytes that attn_kv_cache_write_fp8 stores (cache_fp8.cu).
//
//   s_t = scale * 2^(kb_t - 127) * (q . kc_t),  p = softmax(s),
//   o = sum_t p_t 2^(vb_t - 127) vc_t,          lse = ln sum_t exp(s_t)
//
// The cache's bytes bound it: 2 (D + 1) per token and KV head.  At that rate a
// block of 128 tokens leaves an SM about 1400 cycles, too few to convert the
// codes on the CUDA cores for several query heads; so the codes go from shared
// memory straight into tcgen05.mma kind::f8f6f4 as its A operand, and what is
// not 8 bits wide is split into 8-bit pieces on the small B side instead:
//   * S^T [128 tokens, heads] = K [128, D] . Q^T.  A bf16 query (8 significant
//     bits) is two e4m3 pieces (4 bits each), q = 2^f (a + b / 16), exactly
//     but for values 2^14 times smaller than the row's largest;
//   * O^T [D, heads] = V^T [D, 128] . P^T, V the MN-major A operand.  The
//     weights are w_t = 2^(s_t + v_t - M), v_t = vb_t - 127, M the largest
//     s_t + v_t of this block and head: the value's exponent goes into the
//     weight's, and since every block has a reference of its own no weight is
//     lost to a far larger one in another block.  256 w is split into four e4m3
//     pieces, each 16 times finer, which hold it to 2^-16 of itself, but to
//     2^-30 of the block's largest at best (split_pair).
// O^T of a block is read from TMEM and added, times 2^(M - R), to fp32
// registers (thread = column d of the output), so nothing is rescaled in TMEM.
// The softmax sum is kept apart from the weights, in fp32, each warp with a
// reference of its own (one of its scores, moved rarely), so a value row of zeros
// or of any scale does not touch it.  What is added to a score is added to its
// difference from that reference, and partials are kept as (reference, sum), so
// that nothing is lost beside scores of up to 2^23; above, M's own step passes 1.
// (Plain sums u + v_t and an lse a partial take 3% less time at D = 64 with eight
// heads or short sequences, 1 to 3% elsewhere, and are 2^-11 off at scores of 2^13.)
// What bounds it now (one GB300, contexts of 16384, 64 sequences, 8 KV heads, of
// 6787 GB/s copied; 4 and 8 heads a KV head, either output): D = 128 7.0 and 6.8
// TB/s, D = 256 7.1 and 7.0, D = 192 6.6 and 6.4, D = 96 6.1 and 6.1 (a quarter of
// its shared memory is padding), D = 64 6.4 and 4.7 (the softmax warps); above 8
// heads a KV head's rows go to several CTAs, which read them from the L2: at 16
// D = 64 2.4, D = 128 4.7, D = 256 5.0.
//
// Work split: the context blocks of all sequences, in order, are cut into C
// equal runs ("chunks"), and CTA (c, h) takes chunk c of KV head (or head
// group) h, heads fastest, so that CTAs running side by side read neighbouring
// rows.  A sequence inside one chunk is written out directly; one that crosses
// chunks leaves fp32 partials (o, the scores' reference, the sum less it: an lse
// would lose the sum's bits beside a large score), which paged_fp8_combine joins.  Few
// short sequences take a cluster of CTAs each instead, which join on chip.
#include <float.h>
#include <math.h>

#include <mutex>

#include "kernels.h"
#include "ptx.cuh"

namespace gbattn {

namespace {

constexpr int kTok = 128;       // tokens of a cache block: the MMA's M
constexpr int kWg = 128;        // threads of a softmax warpgroup, one a token lane
constexpr int kMaxCluster = 8;  // portable cluster size
constexpr int kNewSeg = 256, kLastBlock = 512;  // flags beside a slot's token count
constexpr float kLow = -1e30f;  // a reference below every score, finite so that differences are defined
constexpr float kLn2f = 0.6931471805599453f;

constexpr int up16(int n) { return (n + 15) / 16 * 16; }
constexpr int pow2_cols(int n) { return n <= 32 ? 32 : (n <= 64 ? 64 : (n <= 128 ? 128 : (n <= 256 ? 256 : 512))); }

// HG query heads a CTA.  Up to four heads one warpgroup does the softmax; eight
// are shared by two, four heads each, so that a block's chain of products and
// softmax stays short.  Two more warps load and issue the products.
template <int D_, int HG_>
struct Fp8Cfg {
    static constexpr int D = D_, HG = HG_;
    static constexpr int NP = 4;                     // e4m3 pieces of a weight
    static constexpr int NWG = HG > 4 ? 2 : 1;
    static constexpr int HT = HG / NWG;              // heads a thread
    static constexpr int SOFT = NWG * kWg;
    static constexpr int THREADS = SOFT + 64;
    static constexpr int NCH = (D + 127) / 128;      // 128-column blocks of O^T, and 128-byte chunks of a query row
    static constexpr int PW = paged_fp8_box(D);      // bytes of a row in one TMA box, and its swizzle span
    static constexpr int NPC = (D + PW - 1) / PW;    // boxes of 128 rows (the last zero-filled past D)
    static constexpr int PIECE_BYTES = kTok * PW;    // a slot: value boxes, then key boxes
    static constexpr int NQ = up16(2 * HG);          // columns of S^T: piece * HG + head
    static constexpr int NW = NWG * 16;               // columns of O^T: warpgroup * 16 + piece * HT + head
    static constexpr int HALF_BYTES = NPC * PIECE_BYTES;
    static constexpr int SLOT_BYTES = 2 * HALF_BYTES;
    static constexpr int CTAS = paged_fp8_ctas(D, HG);  // per SM
    static constexpr int STAGES = (CTAS == 3 ? 49152 : (CTAS == 2 ? 98304 : 196608)) / SLOT_BYTES;
    static constexpr int Q_BYTES = NCH * NQ * 128;   // one buffer of query pieces
    static constexpr int P_BYTES = NW * kTok;
    static constexpr int OFF_Q = STAGES * SLOT_BYTES;
    static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_SC = OFF_P + P_BYTES;             // exponent bytes: [stage][K, V][128]
    static constexpr int OFF_RED = OFF_SC + STAGES * 256;      // [warpgroup][2][4][HT] f32
    static constexpr int OFF_SUM = OFF_RED + 2 * 4 * HG * 4;   // [warpgroup][4][HT] f32 x 2: a segment's sums
    static constexpr int OFF_QF = OFF_SUM + 4 * HG * 8;        // [2][HG] f32: 2^f * scale_log2
    static constexpr int OFF_LEN = OFF_QF + 2 * HG * 4;        // valid tokens of each slot's block
    static constexpr int OFF_BAR = (OFF_LEN + STAGES * 4 + 7) & ~7;
    static constexpr int N_BAR = 2 * STAGES + 2 + 2 + 1 + 1 + 1;
    static constexpr int SMEM_BYTES = 1024 + OFF_BAR + N_BAR * 8;
    static constexpr int TM_S = 0;                   // two S^T buffers
    static constexpr int TM_O = 2 * NQ;
    static constexpr int TM_COLS = pow2_cols(2 * NQ + NCH * NW);
    static_assert((SMEM_BYTES + 1024 + 256) * CTAS <= 233472, "shared memory budget");
    static_assert(TM_COLS * CTAS <= 512, "tensor memory budget");
    static_assert(NP * HT <= 16, "a warpgroup's pieces of weights are one 16-byte row a token");
    static_assert(HG * (D + 2) * 4 <= SLOT_BYTES, "a cluster's partials lie in the first slot");
};

// Instruction descriptor of kind::f8f6f4, fp32 accumulation: A format in bits
// 7-9 and B format in bits 10-12 (0 e4m3, 1 e5m2), the rest as for kind::f16.
__device__ __forceinline__ uint32_t idesc_f8(int M, int N, uint32_t a_fmt, bool a_mn, bool b_mn) {
    return (1u << 4) | (a_fmt << 7) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// sdesc_sw128 for rows of PW bytes, 128 or 64, with the swizzle of that span.
template <int PW>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo) {
    constexpr uint64_t mode = PW == 128 ? 2 : 4;
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>(8 * PW >> 4) << 32 | static_cast<uint64_t>(1) << 46 | mode << 61;
}

// Matrix descriptor without swizzle, MN-major: 16-byte rows of 16 columns, 8
// of them (k) in a 128-byte core matrix; k groups `lbo` apart, column groups
// `sbo` apart.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46;
}

// Untiled bulk copy global -> shared (both 16-byte aligned, bytes % 16 == 0).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// N consecutive 32-bit columns of this warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
    if constexpr (N >= 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
        if constexpr (N > 16) tmem_ld<N - 16>(taddr + 16, r + 16);
    } else if constexpr (N >= 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
        if constexpr (N > 8) tmem_ld<N - 8>(taddr + 8, r + 8);
    } else if constexpr (N >= 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
        if constexpr (N > 4) tmem_ld<N - 4>(taddr + 4, r + 4);
    } else {
        static_assert(N == 2, "");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
    }
}

// OR of a predicate over the `n` threads of barrier `id` (uniform answer).
__device__ __forceinline__ bool named_bar_or(int id, int n, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {  // NaN ignored unless every lane has it
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// The weights of two heads, y of about 256 at most, as NP pairs of e4m3 codes, each
// piece 16 times finer than the one before.  A piece takes 4 bits while it is a
// normal number (2^-6 and up), so NP pieces are 2^-4NP of a weight off at most; below,
// the last one's step is fixed, and what is lost is up to 2^-10 * 16^-(NP-1) of the
// 256 that the block's largest weight is: 2^-30 of that weight for NP = 4.  A
// value row with a larger exponent byte than its codes need, or with one column far
// above the others, so costs the other rows of its block bits.  (Three pieces of an
// fp16 number, 11 bits and 2^-26, take 5 to 9% less time where the softmax warps bound,
// at D = 64 with eight heads and below D = 256 with more than eight, and no less
// elsewhere: they were bf16 output's until its last bits were compared.  Taking what
// the first piece leaves through fp16, whose packed arithmetic holds the same bits,
// gains 0.7% there.)
template <int NP>
__device__ __forceinline__ void split_pair(float2 y, uint32_t (&c)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        c[i] = pack_fp8x2<false>(y.x, y.y);
        if (i + 1 < NP) {
            const float2 f = unpack_fp8x2<false>(c[i]);
            y = __fmul2_rn(__fadd2_rn(y, make_float2(-f.x, -f.y)), splat(16.f));
        }
    }
}

// A part of a sequence, (reference, softmax sum less it), among others: its weight is
// sum * 2^(reference - top), with `top` the largest of all parts' reference plus
// exponent of the sum (a reference may lie 60 and more below its part's scores).  It
// is given as a number of 2^-100 at least and what is below that as a factor of its
// own, 1 as a rule: a part of weight 2^-150 still counts where its values are 2^150
// times the others'.
__device__ __forceinline__ int sum_exponent(float2 part) { return ((__float_as_int(part.y) >> 23) & 255) - 127; }
__device__ __forceinline__ float part_top(float2 part) { return part.x + static_cast<float>(sum_exponent(part)); }
__device__ __forceinline__ float part_weight(float2 part, float top, float& low) {
    const float mant = __int_as_float((__float_as_int(part.y) & 0x7FFFFF) | 0x3F800000);
    const float power = (part.x - top) + static_cast<float>(sum_exponent(part)), above = fmaxf(power, -100.f);
    low = ex2(power - above);
    return part.y < INFINITY ? mant * ex2(above) : NAN;
}

__device__ __forceinline__ int clamp_len(const PagedFp8Params& p, int s) {
    const int L = p.seq_lens[s];
    return L < 0 ? 0 : (L > p.cap ? p.cap : L);
}
__device__ __forceinline__ int blocks_of(int L) { return (L + kTok - 1) / kTok; }
__device__ __forceinline__ int units_of(int L) { return L > 0 ? blocks_of(L) + 1 : 0; }

// Work is counted in units: one for each block of 128 tokens, and one more for
// each sequence that has any, before its blocks (beginning and ending a
// sequence takes about as long as a block: 128 sequences of up to 4097 tokens,
// D = 64: 47.0 us without it, 45.4 with).
// U units (fewer than 2^31) are cut into N = min(chunks, U) runs that differ by
// one unit at most, none of them empty; chunks from N on hold none.
struct Cut {
    uint32_t U, per, more;  // the first `more` of N runs hold per + 1 units, the others per
    __device__ __forceinline__ Cut(uint32_t U_, uint32_t chunks) : U(U_) {
        const uint32_t N = U < chunks ? U : chunks;
        per = N ? U / N : 0;
        more = N ? U - per * N : 0;
    }
    __device__ __forceinline__ uint32_t start(uint32_t c) const {  // first unit of chunk c
        return min(U, c * per + min(c, more));  // (c * per + c <= U + chunks)
    }
    __device__ __forceinline__ uint32_t chunk_of(uint32_t u) const {  // the chunk that holds unit u < U
        const uint32_t a = more * (per + 1);
        return u < a ? u / (per + 1) : more + (u - a) / per;
    }
};

// A warp's walk over its chunk's segments: [b0, b1) of sequence s, of `nblk`
// blocks in all.  Every lane of the warp calls next(); the lengths of 32
// sequences are held across the lanes.
struct Walk {
    int s, L, nblk, b0, b1;
    int rem;  // units of the chunk after this segment
    int base, Llane;

    __device__ __forceinline__ void load(const PagedFp8Params& p, int lane) {
        const int i = base + lane;
        Llane = i < p.num_seqs ? clamp_len(p, i) : 0;
    }
    __device__ __forceinline__ void take(int n, int from) {
        L = __shfl_sync(0xffffffffu, Llane, s - base);
        nblk = blocks_of(L);
        b0 = from;
        b1 = from + min(nblk - from, n);
        rem = n - (b1 - b0);
    }
    // From block `from` of sequence s0 on, n > 0 units.
    __device__ __forceinline__ void start(const PagedFp8Params& p, int s0, int from, int n) {
        s = s0;
        base = s0;
        load(p, threadIdx.x & 31);
        take(n, from);
    }
    // Whether this segment is the chunk's last: a last unit that only begins a
    // sequence (its blocks are the next chunk's) is no segment.
    __device__ __forceinline__ bool last() const { return rem <= 1; }
    // The next sequence that has tokens; false when the chunk is done.
    __device__ __forceinline__ bool next(const PagedFp8Params& p) {
        if (last()) return false;
        const int lane = threadIdx.x & 31;
        for (;;) {
            const unsigned has = __ballot_sync(0xffffffffu, Llane > 0 && base + lane > s);
            if (has) {
                s = base + __ffs(static_cast<int>(has)) - 1;
                take(rem - 1, 0);
                return true;
            }
            s = base + 31;
            base += 32;
            if (base >= p.num_seqs) return false;
            load(p, lane);
        }
    }
};

// The queries of one sequence: each warpgroup those of its own heads, warp by
// warp (heads at or past nh are zeros).  Loaded into registers early, laid out later as two e4m3 pieces
// a value, K-major 128-byte swizzled rows, row piece * HG + head; and 2^f *
// scale_log2 of each head.  A row with a NaN or an infinity becomes NaN where
// it has it, so that head's result is NaN.
template <class C>
struct Queries {
    static constexpr int PAIRS = C::D / 2, PL = (PAIRS + 31) / 32, NHW = (C::HT + 3) / 4;
    uint32_t x[NHW][PL];

    __device__ __forceinline__ void load(const PagedFp8Params& p, int s, int h0, int nh, int warp, int lane) {
#pragma unroll
        for (int k = 0; k < NHW; ++k) {
            const int h = (warp / 4) * C::HT + (warp & 3) + 4 * k;
            const uint32_t* src =
                reinterpret_cast<const uint32_t*>(p.q + s * p.q_stride + static_cast<long long>(h0 + h) * C::D);
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int pr = lane + 32 * i;
                x[k][i] = ((warp & 3) + 4 * k < C::HT && h < nh && pr < PAIRS) ? src[pr] : 0u;
            }
        }
    }
    __device__ __forceinline__ void put(const PagedFp8Params& p, uint8_t* sq, float* qf, int warp, int lane) const {
#pragma unroll
        for (int k = 0; k < NHW; ++k) {
            const int h = (warp / 4) * C::HT + (warp & 3) + 4 * k;
            if ((warp & 3) + 4 * k >= C::HT) break;
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const uint32_t a = x[k][i] & 0x7FFFu, b = (x[k][i] >> 16) & 0x7FFFu;
                if (a < 0x7F80u) mx = max(mx, a);
                if (b < 0x7F80u) mx = max(mx, b);
            }
            mx = __reduce_max_sync(0xffffffffu, mx);
            int fb = static_cast<int>(mx >> 7) - 8 + ((mx & 0x7Fu) > 0x60u ? 1 : 0);  // as in the cache's rule, c_max = 448
            fb = fb < 1 ? 1 : fb;
            const float inv = __uint_as_float(static_cast<uint32_t>(254 - fb) << 23);
            if (lane == 0) qf[h] = exp2_byte(fb) * p.scale_log2;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int pr = lane + 32 * i;
                if (pr < PAIRS) {
                    float lo = __uint_as_float(x[k][i] << 16), hi = __uint_as_float(x[k][i] & 0xFFFF0000u);
                    if ((x[k][i] & 0x7F80u) == 0x7F80u) lo = NAN;
                    if ((x[k][i] & 0x7F800000u) == 0x7F800000u) hi = NAN;
                    lo *= inv;
                    hi *= inv;
                    const uint32_t c0 = pack_fp8x2<false>(lo, hi);
                    const float2 f0 = unpack_fp8x2<false>(c0);
                    const uint32_t c1 = pack_fp8x2<false>((lo - f0.x) * 16.f, (hi - f0.y) * 16.f);
                    const int e = 2 * pr, ch = e >> 7, col = e & 127;
#pragma unroll
                    for (int piece = 0; piece < 2; ++piece) {
                        const int row = piece * C::HG + h;
                        *reinterpret_cast<uint16_t*>(sq + ch * (C::NQ * 128) + row * 128 +
                                                     (((col >> 4) ^ (row & 7)) << 4) + (col & 15)) =
                            static_cast<uint16_t>(piece ? c1 : c0);
                    }
                }
            }
        }
    }
};

template <class C, bool CLUSTER>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    paged_decode_fp8_sm103a(const __grid_constant__ CUtensorMap tmKV, const PagedFp8Params p) {
    constexpr int D = C::D, HG = C::HG, HT = C::HT, NP = C::NP, NQ = C::NQ, NW = C::NW, NCH = C::NCH;
    constexpr int STAGES = C::STAGES, SOFT_WARPS = C::SOFT / 32, WARPS = C::THREADS / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    float* sqf = reinterpret_cast<float*>(smem + C::OFF_QF);
    volatile int* slen = reinterpret_cast<volatile int*>(smem + C::OFF_LEN);  // and flags
    const uint32_t bar0 = sb + C::OFF_BAR;
    auto b_full = [&](int i) { return bar0 + 8 * i; };
    auto b_empty = [&](int i) { return bar0 + 8 * (STAGES + i); };
    auto b_sfull = [&](int i) { return bar0 + 8 * (2 * STAGES + i); };
    auto b_qfull = [&](int i) { return bar0 + 8 * (2 * STAGES + 2 + i); };
    const uint32_t b_pfull = bar0 + 8 * (2 * STAGES + 4), b_ofull = b_pfull + 8, b_done = b_pfull + 16;
    __shared__ int abort_storage, s_stop;
    __shared__ uint32_t tmem_base_storage, s_issued;  // s_issued: blocks whose loads were issued
    __shared__ uint32_t s_sum[WARPS];
    __shared__ uint32_t s_u[2];   // the unit behind this chunk's last, and all units
    __shared__ int s_first[3];    // first sequence, first block of it, units from there on (0: no work)
    __shared__ int2 s_join;       // as PagedFp8Params::joins, of this chunk
    __shared__ int s_parts;       // of a cluster: the parts its sequence is in, where more than one
    volatile int* abort_flag = &abort_storage;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a cluster holds the parts of one sequence and head; otherwise heads vary fastest
    const int chunk = CLUSTER ? blockIdx.x % p.chunks : blockIdx.x / p.n_hgroups;
    const int hg = CLUSTER ? blockIdx.x / p.chunks % p.n_hgroups : blockIdx.x % p.n_hgroups;
    const int kvh = hg / p.subs, sub = hg % p.subs;
    const int h0 = kvh * p.group + sub * p.heads_per_sub;
    const int nh = min(p.heads_per_sub, p.group - sub * p.heads_per_sub);
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(b_full(i), 1);
            mbar_init(b_empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_sfull(i), 1);
            mbar_init(b_qfull(i), SOFT_WARPS);
        }
        mbar_init(b_pfull, SOFT_WARPS);
        mbar_init(b_ofull, 1);
        mbar_init(b_done, 1);
        abort_storage = p.give_up ? 1 : 0;  // 1: give up every wait (failure-path test)
        s_issued = 0;
        s_join = make_int2(-1, 0);
        s_parts = 0;
        s_first[2] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmKV);
    }
    // Launched as a programmatic dependent of whatever comes before on the stream:
    // up to here nothing of global memory is read or written.
    grid_dependency_wait();
    grid_launch_dependents();  // the combine may queue up; it waits for this grid to finish
    // Tensor memory only now: the grid before may have CTAs here that still ask for theirs.
    if (warp == SOFT_WARPS) {
        tmem_alloc(smem_u32(&tmem_base_storage), C::TM_COLS);
        tmem_relinquish();
    }

    // ---- this chunk's units: the total, then the sequence its first unit lies
    // in.  Lengths are read once where a pass of the block covers them all.
    const uint32_t given_up = threadIdx.x == 0 && status_has_timeout(p.status, kDevTimeout);
    if (threadIdx.x == 0) s_stop = given_up;  // after a give-up nothing more is begun
    const bool one_pass = p.num_seqs <= C::THREADS;
    const int own = CLUSTER ? blockIdx.x / (p.chunks * p.n_hgroups) : 0;  // a cluster's sequence
    uint32_t sum = 0;
    int T = 0;  // of a sequence: its units
    bool bad = false;
    for (int s = CLUSTER ? own : threadIdx.x; s < (CLUSTER ? own + 1 : p.num_seqs); s += C::THREADS) {
        const int L = p.seq_lens[s];
        bad |= L < 0 || L > p.cap;
        T = units_of(L < 0 ? 0 : (L > p.cap ? p.cap : L));
        sum += T;
    }
    if (bad && (CLUSTER ? threadIdx.x == 0 : blockIdx.x == 0) && p.status) atomicOr(p.status, kDevBadSeqlen);
    if constexpr (CLUSTER) {
        if (threadIdx.x == 0) {
            const int blocks = T > 0 ? T - 1 : 0;
            const Cut cut(blocks, p.chunks);
            const uint32_t b0 = cut.start(chunk);
            s_u[1] = T;
            s_first[0] = own;
            s_first[1] = static_cast<int>(b0);
            s_first[2] = given_up ? 0 : static_cast<int>(cut.start(chunk + 1) - b0);
            const int parts = min(blocks, p.chunks);
            s_parts = parts > 1 && !given_up ? parts : 0;  // one part is the whole: written out, nothing to join
        }
    } else {
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        if (lane == 31) s_sum[warp] = incl;
        __syncthreads();
        uint32_t U = 0, before = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += s_sum[w];
            U += s_sum[w];
        }
        const Cut cut(U, p.chunks);
        const uint32_t u0 = cut.start(chunk), u1 = cut.start(chunk + 1);
        if (threadIdx.x == 0) {
            s_u[0] = u1;
            s_u[1] = U;
        }
        // the sequence that unit u0 belongs to: `at` units before it
        auto begin = [&](int s, uint32_t at) {
            if (T > 0 && at <= u0 && u0 < at + T && u1 > u0) {
                const int off = static_cast<int>(u0 - at);  // 0: the unit that begins it
                s_first[0] = s;
                s_first[1] = off > 0 ? off - 1 : 0;
                s_first[2] = static_cast<int>(u1 - u0) - (off == 0 ? 1 : 0);
            }
        };
        if (one_pass) {
            begin(threadIdx.x, before + incl - T);
        } else if (u1 > u0) {
            uint32_t run = 0;
#pragma unroll 1
            for (int base = 0; base < p.num_seqs && run <= u0; base += C::THREADS) {  // run <= u0: not found yet (uniform)
                const int s = base + threadIdx.x;
                T = s < p.num_seqs ? units_of(clamp_len(p, s)) : 0;
                incl = T;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += n;
                }
                __syncthreads();  // s_sum was read by all
                if (lane == 31) s_sum[warp] = incl;
                __syncthreads();
                uint32_t at = run + incl - T;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    if (w < warp) at += s_sum[w];
                    run += s_sum[w];
                }
                begin(s, at);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base_storage;
    const int n_units = s_stop ? 0 : s_first[2];
    bool ok = true;

    if (warp < SOFT_WARPS) {
        // ---------------------------------------------------- softmax and output
        const int wg = warp / 4, tok = threadIdx.x % kWg;
        const int hw = wg * HT;  // this warpgroup's first head
        float* sred = reinterpret_cast<float*>(smem + C::OFF_RED) + wg * 2 * 4 * HT;
        float2* ssum = reinterpret_cast<float2*>(smem + C::OFF_SUM) + wg * 4 * HT;
        if (n_units > 0) {
            Walk w, ahead;  // `ahead` is one segment further: its queries are laid out early
            w.start(p, s_first[0], s_first[1], n_units);
            ahead = w;
            Queries<C> qs;
            qs.load(p, w.s, h0, nh, warp, lane);
            qs.put(p, smem + C::OFF_Q, sqf, warp, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_qfull(0));
            named_bar_sync(1 + wg, kWg);  // sqf is read by the warpgroup's four warps
            const uint32_t tlane = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 TMEM lanes
            uint32_t g = 0, phase = 0;  // blocks done; the ring's parity
            int slot = 0, seg = 0;
            bool more = true;
            while (more) {
                // queries of the next segment: asked for now, laid out after this
                // segment's first block (its buffer's last reader was segment seg - 1)
                const bool has_next = ahead.next(p);
                if (has_next) qs.load(p, ahead.s, h0, nh, warp, lane);
                float2 o[NCH][HT / 2], R[HT / 2], M8[HT / 2], mref[HT / 2], l[HT / 2];
#pragma unroll
                for (int h = 0; h < HT / 2; ++h) {
                    R[h] = mref[h] = M8[h] = splat(kLow);
                    l[h] = splat(0.f);
#pragma unroll
                    for (int c = 0; c < NCH; ++c) o[c][h] = splat(0.f);
                }
                // O^T of the block before: asked for early, and then
                // o += 2^(M - 8 - R) sum_i piece_i / 16^i
                uint32_t ro[NCH][NP * HT];
                auto ask_o = [&](uint32_t gi) {
                    if (!mbar_wait(b_ofull, gi & 1, abort_flag)) ok = false;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < NCH; ++c) tmem_ld<NP * HT>(tm + tlane + C::TM_O + c * NW + wg * 16, ro[c]);
                };
                auto add_o = [&]() {
                    float2 beta[HT / 2];
                    float dm = kLow;
#pragma unroll
                    for (int h = 0; h < HT / 2; ++h) {
                        beta[h] = __fadd2_rn(M8[h], make_float2(-R[h].x, -R[h].y));
                        dm = fmax3(dm, beta[h].x, beta[h].y);
                    }
                    if (dm > 40.f) {  // a larger reference, the same in every thread
#pragma unroll
                        for (int h = 0; h < HT / 2; ++h) {
                            const float2 n = make_float2(fmaxf(R[h].x, M8[h].x), fmaxf(R[h].y, M8[h].y));
                            const float2 a = make_float2(ex2(R[h].x - n.x), ex2(R[h].y - n.y));
                            R[h] = n;
                            beta[h] = make_float2(M8[h].x - n.x, M8[h].y - n.y);
#pragma unroll
                            for (int c = 0; c < NCH; ++c) o[c][h] = __fmul2_rn(o[c][h], a);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < HT / 2; ++h) beta[h] = make_float2(ex2(beta[h].x), ex2(beta[h].y));
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int h = 0; h < HT / 2; ++h) {
                            auto piece = [&](int i) {
                                return make_float2(__uint_as_float(ro[c][i * HT + 2 * h]), __uint_as_float(ro[c][i * HT + 2 * h + 1]));
                            };
                            float2 x = piece(NP - 1);
#pragma unroll
                            for (int i = NP - 2; i >= 0; --i) x = __ffma2_rn(x, splat(0.0625f), piece(i));
                            o[c][h] = __ffma2_rn(x, beta[h], o[c][h]);
                        }
                    tc_fence_before();
                };
                const float2* qf = reinterpret_cast<const float2*>(sqf + (seg & 1) * HG + hw);
                bool quit = false;
                for (int b = w.b0; b < w.b1; ++b, ++g) {
                    if (!mbar_wait(b_full(slot), phase, abort_flag)) ok = false;
                    const int nvalid = slen[slot] & (kNewSeg - 1);
                    const bool valid = tok < nvalid;
                    const uint8_t* sc = smem + C::OFF_SC + slot * 256;
                    // 2^(b - 127) (2^-127 is a subnormal number), and b - 127 by way of 2^23 + b
                    const float kf = __uint_as_float(max(static_cast<uint32_t>(sc[tok]) << 23, 0x400000u));
                    const float ev = __uint_as_float(0x4B000000u | sc[128 + tok]) - (8388608.f + 127.f);
                    if (!mbar_wait(b_sfull(g & 1), (g >> 1) & 1, abort_flag)) ok = false;
                    tc_fence_after();
                    uint32_t r0[HT], r1[HT];
                    tmem_ld<HT>(tm + tlane + C::TM_S + (g & 1) * NQ + hw, r0);
                    tmem_ld<HT>(tm + tlane + C::TM_S + (g & 1) * NQ + HG + hw, r1);
                    tmem_wait_ld();
                    float2 dot[HT / 2], kq[HT / 2], d[HT / 2];  // a score is dot * kq; d: less the warp's reference
                    float dmax = kLow;
#pragma unroll
                    for (int h = 0; h < HT / 2; ++h) {
                        dot[h] =
                            __ffma2_rn(make_float2(__uint_as_float(r1[2 * h]), __uint_as_float(r1[2 * h + 1])), splat(0.0625f),
                                       make_float2(__uint_as_float(r0[2 * h]), __uint_as_float(r0[2 * h + 1])));
                        // (first: dot * kf may overflow; and held finite, so that a dot of 0 is a score of 0)
                        kq[h] = __fmul2_rn(qf[h], splat(kf));
                        kq[h] = make_float2(fminf(kq[h].x, FLT_MAX), fminf(kq[h].y, FLT_MAX));
                        d[h] = __ffma2_rn(dot[h], kq[h], make_float2(-mref[h].x, -mref[h].y));
                        if (nvalid < kTok) d[h] = valid ? d[h] : splat(-INFINITY);
                        dmax = fmax3(dmax, d[h].x, d[h].y);
                    }
                    if (__any_sync(0xffffffffu, dmax > 60.f)) {  // rarely: fp32 has room for sums of 2^60 and more
#pragma unroll
                        for (int h = 0; h < HT / 2; ++h) {
                            float2 u = __fmul2_rn(dot[h], kq[h]);
                            if (!valid) u = splat(-INFINITY);
                            const float2 m = make_float2(fmaxf(mref[h].x, warp_max(u.x)), fmaxf(mref[h].y, warp_max(u.y)));
                            l[h] = make_float2(l[h].x * ex2(mref[h].x - m.x), l[h].y * ex2(mref[h].y - m.y));
                            mref[h] = m;
                            d[h] = __ffma2_rn(dot[h], kq[h], make_float2(-m.x, -m.y));
                            if (!valid) d[h] = splat(-INFINITY);
                        }
                    }
                    float m[HT];
#pragma unroll
                    for (int h = 0; h < HT / 2; ++h) {
                        l[h] = __fadd2_rn(l[h], make_float2(ex2(d[h].x), ex2(d[h].y)));
                        // the value's exponent counts in full beside a large score: added to the difference
                        d[h] = __fadd2_rn(d[h], splat(ev));
                        const float2 top = __fadd2_rn(make_float2(warp_max(d[h].x), warp_max(d[h].y)), mref[h]);
                        m[2 * h] = top.x;
                        m[2 * h + 1] = top.y;
                    }
                    float* red = sred + (g & 1) * 4 * HT;
                    if (lane == 0) {
                        if constexpr (HT == 4)
                            *reinterpret_cast<float4*>(red + (warp & 3) * HT) = make_float4(m[0], m[1], m[2], m[3]);
                        else
                            *reinterpret_cast<float2*>(red + (warp & 3) * HT) = make_float2(m[0], m[1]);
                    }
                    if (b > w.b0) ask_o(g - 1);
                    if (named_bar_or(1 + wg, kWg, !ok)) {  // a warpgroup's four warps leave together
                        tmem_wait_ld();  // (what ask_o asked for, before tensor memory is freed)
                        quit = true;
                        break;
                    }
                    // the value rows past the context meet weight 0: they must be finite
                    if (!valid && wg == 0) {
#pragma unroll
                        for (int c = 0; c < C::NPC; ++c) {
                            uint4* v = reinterpret_cast<uint4*>(smem + slot * C::SLOT_BYTES + c * C::PIECE_BYTES + tok * C::PW);
#pragma unroll
                            for (int i = 0; i < C::PW / 16; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (b > w.b0) add_o();  // the weights' buffer and O^T are free again
                    // weights 256 w = 2^(s + v - M + 8) and their pieces, byte piece * HT + head
                    float wm[4][HT];  // the four warps' maxima
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (HT == 4) {
                            const float4 a = *reinterpret_cast<const float4*>(red + k * HT);
                            wm[k][0] = a.x, wm[k][1] = a.y, wm[k][2] = a.z, wm[k][3] = a.w;
                        } else {
                            const float2 a = *reinterpret_cast<const float2*>(red + k * HT);
                            wm[k][0] = a.x, wm[k][1] = a.y;
                        }
                    }
                    uint32_t w8[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int h = 0; h < HT / 2; ++h) {
                        float mm[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mm[k] = fmaxf(fmax3(wm[0][2 * h + k], wm[1][2 * h + k], wm[2][2 * h + k]), fmaxf(wm[3][2 * h + k], kLow));
                        M8[h] = make_float2(mm[0] - 8.f, mm[1] - 8.f);
                        const float2 e = __fadd2_rn(d[h], __fadd2_rn(mref[h], make_float2(-M8[h].x, -M8[h].y)));
                        uint32_t c[NP];
                        split_pair<NP>(make_float2(ex2(e.x), ex2(e.y)), c);
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            const int col = i * HT + 2 * h;
                            w8[col / 4] |= c[i] << (8 * (col & 3));
                        }
                    }
                    st_shared_v4(sb + C::OFF_P + wg * (kTok * 16) + tok * 16, w8[0], w8[1], w8[2], w8[3]);
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_pfull);
                    if (++slot == STAGES) {
                        slot = 0;
                        phase ^= 1;
                    }
                    if (has_next && b == w.b0) {
                        qs.put(p, smem + C::OFF_Q + ((seg + 1) & 1) * C::Q_BYTES, sqf + ((seg + 1) & 1) * HG, warp, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_qfull((seg + 1) & 1));
                    }
                }
                if (quit) break;
                ask_o(g - 1);
                add_o();
                // ---- the segment's softmax sum over the 128 token lanes, then its output.
                // A warp's HT sums at once: while there are several, a lane gives
                // away one half of its heads and keeps the other.
                float hsum;
                if constexpr (HT == 4) {
                    const bool up = lane & 16, up2 = lane & 8;
                    float2 a = up ? l[1] : l[0];
                    const float2 b = up ? l[0] : l[1];
                    a.x += __shfl_xor_sync(0xffffffffu, b.x, 16);
                    a.y += __shfl_xor_sync(0xffffffffu, b.y, 16);
                    hsum = (up2 ? a.y : a.x) + __shfl_xor_sync(0xffffffffu, up2 ? a.x : a.y, 8);
                } else {
                    static_assert(HT == 2, "");
                    const bool up = lane & 16;
                    hsum = (up ? l[0].y : l[0].x) + __shfl_xor_sync(0xffffffffu, up ? l[0].x : l[0].y, 16);
                    hsum += __shfl_xor_sync(0xffffffffu, hsum, 8);
                }
#pragma unroll
                for (int of = 4; of; of >>= 1) hsum += __shfl_xor_sync(0xffffffffu, hsum, of);
                const int hl = HT == 4 ? lane >> 3 : lane >> 4;  // this lane's head
                float mh = mref[0].x, Rh = R[0].x;
#pragma unroll
                for (int h = 1; h < HT; ++h)
                    if (hl == h) {
                        mh = h & 1 ? mref[h / 2].y : mref[h / 2].x;
                        Rh = h & 1 ? R[h / 2].y : R[h / 2].x;
                    }
                if ((lane & 7) == 0) ssum[(warp & 3) * HT + hl] = make_float2(mh, hsum);
                if (named_bar_or(1 + wg, kWg, !ok)) break;
                const float2 sa = ssum[hl], sb2 = ssum[HT + hl], sc2 = ssum[2 * HT + hl], sd = ssum[3 * HT + hl];
                const float mt = fmaxf(fmax3(sa.x, sb2.x, sc2.x), sd.x);
                const float all = (sa.y * ex2(sa.x - mt) + sb2.y * ex2(sb2.x - mt)) + (sc2.y * ex2(sc2.x - mt) + sd.y * ex2(sd.x - mt));
                // 2^(Rh - mt) / all: the exponent of `all` goes into the power, so that
                // neither of the two overflows alone; 2^-21 off at most.  What the power
                // has below 2^-100 is a factor of its own: ex2 flushes below 2^-126, and
                // the sums it meets are 2^8 times the values and more.
                const int abits = __float_as_int(all), ae = ((abits >> 23) & 255) - 127;
                const float am = __int_as_float((abits & 0x7FFFFF) | 0x3F800000);
                const float power = Rh - mt - static_cast<float>(ae), above = fmaxf(power, -100.f);
                float inv_l = __fdividef(ex2(above), am);
                const float low_l = ex2(power - above);  // 1 as a rule
                if (all == 0.f) inv_l = 0.f;
                if (!(all < INFINITY)) inv_l = NAN;
                float inv[HT], low[HT];
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    inv[h] = __shfl_sync(0xffffffffu, inv_l, h * (32 / HT));
                    low[h] = __shfl_sync(0xffffffffu, low_l, h * (32 / HT));
                }
                const bool whole = w.b0 == 0 && w.b1 == w.nblk;
                if (!CLUSTER && threadIdx.x == 0 && w.b0 == 0 && w.b1 < w.nblk) {
                    // this segment's sequence begins here and goes on: up to the chunk of its last unit
                    s_join = make_int2(w.s, static_cast<int>(Cut(s_u[1], p.chunks).chunk_of(s_u[0] + (w.nblk - w.b1) - 1)));
                }
                // Partials: in the workspace, slot 1 where the sequence begins and slot 0
                // where it goes on; or, of a cluster, in the first slot of the ring, which
                // nothing reads or fills any more (a cluster's CTA has one segment).
                const long long part = (static_cast<long long>(chunk) * 2 + (w.b0 == 0 ? 1 : 0)) * p.Hq + h0;
                float* po = CLUSTER ? reinterpret_cast<float*>(smem) : p.part_o + part * D;
                float2* pl = CLUSTER ? reinterpret_cast<float2*>(smem + HG * D * 4) : p.part_sum + part;
                const long long row = static_cast<long long>(w.s) * p.Hq + h0;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const int d = c * 128 + tok;
                    if (d < D) {
#pragma unroll
                        for (int k = 0; k < HT; ++k) {
                            const int h = hw + k;
                            if (h < nh) {
                                const float x = (k & 1 ? o[c][k / 2].y : o[c][k / 2].x) * inv[k] * low[k];
                                if (!whole)
                                    po[h * D + d] = x;
                                else if (p.out_f32)
                                    static_cast<float*>(p.out)[(row + h) * D + d] = x;
                                else
                                    static_cast<uint16_t*>(p.out)[(row + h) * D + d] =
                                        static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFFu);
                            }
                        }
                    }
                }
                if ((warp & 3) == 0 && (lane & (32 / HT - 1)) == 0 && hw + hl < nh) {
                    if (!whole)
                        pl[hw + hl] = make_float2(all == 0.f ? -INFINITY : mt, all);
                    else if (p.lse)
                        p.lse[row + hw + hl] = (all == 0.f ? -INFINITY : mt + __log2f(all)) * kLn2f;
                }
                ++seg;
                more = w.next(p);
            }
        }
        if (!ok) *abort_flag = 1;
    } else if (warp == SOFT_WARPS) {
        if (n_units > 0) {
            // ------------------------------------------------ cache loads
            Walk w;
            w.start(p, s_first[0], s_first[1], n_units);
            int ids = 0, slot = 0, b = w.b0;
            uint32_t phase = 1;  // (the first round of waits on the ring passes at once)
            for (uint32_t g = 0;; ++g) {
                const int at = (b - w.b0) & 31;  // 32 table entries are held, one a lane
                if (at == 0) ids = b + lane < w.b1 ? p.block_table[static_cast<long long>(w.s) * p.max_blocks + b + lane] : 0;
                const int blk = __shfl_sync(0xffffffffu, ids, at);
                ok = __all_sync(0xffffffffu, mbar_wait(b_empty(slot), phase, abort_flag));
                if (!ok) break;
                if (elect_one()) {
                    const bool good = blk >= 0 && blk < p.num_blocks;
                    slen[slot] = (good ? min(kTok, w.L - b * kTok) : 0) + (b == w.b0 ? kNewSeg : 0) +
                                 (b + 1 == w.b1 && w.last() ? kLastBlock : 0);
                    if (good) {
                        mbar_arrive_expect_tx(b_full(slot), C::SLOT_BYTES + 256);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const long long r = static_cast<long long>(half) * p.num_blocks + blk;
#pragma unroll
                            for (int c = 0; c < C::NPC; ++c)
                                tma_load_3d(sb + slot * C::SLOT_BYTES + (1 - half) * C::HALF_BYTES + c * C::PIECE_BYTES, &tmKV,
                                            b_full(slot), c * C::PW, kvh, static_cast<int>(r * kTok));
                            bulk_load(sb + C::OFF_SC + slot * 256 + half * 128, p.scales + (r * p.Hkv + kvh) * kTok, 128, b_full(slot));
                        }
                    } else {
                        if (p.status) atomicOr(p.status, kDevBadIndex);
                        mbar_arrive(b_full(slot));
                    }
                    s_issued = g + 1;
                }
                __syncwarp();
                if (++b == w.b1) {
                    if (!w.next(p)) break;
                    b = w.b0;
                }
                if (++slot == STAGES) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok) *abort_flag = 1;
        }
        // sequences without context, of this chunk's share: zeros and -inf
        auto zero_row = [&](long long s) {
            const long long row = s * p.Hq + h0;
            for (int i = lane; i < nh * D; i += 32) {
                if (p.out_f32)
                    static_cast<float*>(p.out)[row * D + i] = 0.f;
                else
                    static_cast<uint16_t*>(p.out)[row * D + i] = 0;
            }
            if (lane < nh && p.lse) p.lse[row + lane] = -INFINITY;
        };
        if constexpr (CLUSTER) {
            if (s_u[1] == 0 && chunk == 0) zero_row(own);
        } else {
            for (long long i0 = 0; i0 * p.chunks < p.num_seqs; i0 += 32) {
                const long long s = chunk + (i0 + lane) * p.chunks;
                unsigned none = __ballot_sync(0xffffffffu, s < p.num_seqs && clamp_len(p, static_cast<int>(s)) == 0);
                for (; none; none &= none - 1) zero_row(chunk + (i0 + __ffs(static_cast<int>(none)) - 1) * p.chunks);
            }
        }
    } else if (n_units > 0) {
        // ---------------------------------------------------- products
        // Unit by unit: S^T of the next unit, whose buffer was read before the
        // weights of the unit before came; then, once this unit's weights are
        // there, O^T.  (Taking whichever is ready first frees value blocks
        // earlier, but was slower: 7.1 -> 6.6 TB/s at D = 128.)
        const uint32_t id_s = idesc_f8(128, NQ, p.e5m2 ? 1u : 0u, false, false);
        const uint32_t id_o = idesc_f8(128, NW, p.e5m2 ? 1u : 0u, true, true);
        int kslot = 0, vslot = 0, seg = -1;
        uint32_t kphase = 0;
        bool more = true;  // blocks whose S^T is not issued yet
        auto issue_s = [&](uint32_t i) {
            bool got = mbar_wait(b_full(kslot), kphase, abort_flag);
            const int flags = got ? slen[kslot] : 0;
            if (flags & kNewSeg) {
                ++seg;
                got = mbar_wait(b_qfull(seg & 1), (seg >> 1) & 1, abort_flag);
            }
            more = !(flags & kLastBlock);
            if (!__all_sync(0xffffffffu, got)) return false;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t k = sb + kslot * C::SLOT_BYTES + C::HALF_BYTES, q = sb + C::OFF_Q + (seg & 1) * C::Q_BYTES;
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                    mma_f8_ss(tm + C::TM_S + (i & 1) * NQ,
                              sdesc_rows<C::PW>(k + ks * 32 / C::PW * C::PIECE_BYTES + ks * 32 % C::PW, 16),
                              sdesc_sw128(q + (ks / 4) * (NQ * 128) + (ks % 4) * 32, 16, 1024), id_s, ks > 0);
                mma_commit(b_sfull(i & 1));
            }
            __syncwarp();
            if (++kslot == STAGES) {
                kslot = 0;
                kphase ^= 1;
            }
            return true;
        };
        auto issue_o = [&]() {
            tc_fence_after();
            if (elect_one()) {
                // V^T's rows past D (lanes that nobody reads) are zeros or repeat the block's only box
                const uint32_t v = sb + vslot * C::SLOT_BYTES, pp = sb + C::OFF_P;
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f8_ss(tm + C::TM_O + c * NW,
                                  sdesc_rows<C::PW>(v + c * (kTok * 128) + ks * 32 * C::PW,
                                                    D - c * 128 <= C::PW ? 0 : C::PIECE_BYTES),
                                  sdesc_plain(pp + ks * 512, 128, kTok * 16), id_o, ks > 0);
                mma_commit(b_ofull);
                mma_commit(b_empty(vslot));
            }
            __syncwarp();
            if (++vslot == STAGES) vslot = 0;
        };
        // A launch told to give up (p.give_up) stops here, before any product.
        ok = !__any_sync(0xffffffffu, *abort_flag) && issue_s(0);
        for (uint32_t i = 0; ok; ++i) {
            const bool another = more;
            if (another) ok = issue_s(i + 1);
            ok = __all_sync(0xffffffffu, ok && mbar_wait(b_pfull, i & 1, abort_flag));
            if (!ok) break;
            issue_o();
            if (!another) break;
        }
        if (!ok) *abort_flag = 1;
        if (elect_one()) mma_commit(b_done);  // every product issued has finished before TMEM is freed
        __syncwarp();
        mbar_wait_drain(b_done, 0);
    }
    __syncthreads();
    if (*abort_flag) {
        if (threadIdx.x == 0) {
            if (p.status) atomicOr(p.status, kDevTimeout);
            // copies still in flight land (bounded) before the block's memory is given up
            for (uint32_t g = s_issued < STAGES ? 0 : s_issued - STAGES; g < s_issued; ++g)
                mbar_wait_drain(b_full(g % STAGES), (g / STAGES) & 1);
        }
    }
    __syncthreads();
    if (warp == SOFT_WARPS) {
        tc_fence_after();
        tmem_dealloc(tm, C::TM_COLS);
    }
    if constexpr (CLUSTER) {
        // Parts of one sequence: part c joins heads c, c + parts, ... of all parts'
        // partials, read from their shared memory.
        if (p.chunks > 1) cluster_sync();
        const int parts = s_parts;
        if (chunk < parts) {
            for (int h = chunk; h < nh; h += parts) {
                float2 part[kMaxCluster];
                float w[kMaxCluster], low[kMaxCluster], m = kLow, all = 0.f;
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) {
                    part[i] = i < parts ? ld_cluster_f2(mapa_shared(sb + HG * D * 4 + h * 8, i)) : make_float2(-INFINITY, 0.f);
                    m = fmaxf(m, part_top(part[i]));
                }
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) {
                    w[i] = part_weight(part[i], m, low[i]);
                    all = fmaf(w[i], low[i], all);
                }
                const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) w[i] *= inv;  // (before they meet values, which may be 2^127)
                const long long row = static_cast<long long>(own) * p.Hq + h0 + h;
                for (int d = threadIdx.x; d < D; d += C::THREADS) {
                    float x = 0.f;
#pragma unroll
                    for (int i = 0; i < kMaxCluster; ++i)
                        if (i < parts) x = fmaf(w[i], ld_cluster_f1(mapa_shared(sb + (h * D + d) * 4, i)) * low[i], x);
                    if (p.out_f32)
                        static_cast<float*>(p.out)[row * D + d] = x;
                    else
                        static_cast<uint16_t*>(p.out)[row * D + d] = static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFFu);
                }
                if (threadIdx.x == 0 && p.lse) p.lse[row] = all == 0.f ? -INFINITY : (m + __log2f(all)) * kLn2f;
            }
        }
        if (p.chunks > 1) cluster_sync();  // no part's memory goes before it is read
    } else {
        if (threadIdx.x == 0 && hg == 0 && p.chunks > 1) p.joins[chunk] = s_join;
    }
}

// Joins the partials of a sequence that crosses chunks: chunk c's second slot
// (the sequence begins there), the first slots of the chunks up to its last.
// Groups of `width` / 4 threads take the partials in turn, kLoad loads in
// flight each, the first of them asked for before every warp finds the largest
// reference and the whole softmax sum for itself; then one group adds the groups'
// results.  The weights are made relative to that sum before they meet values.
//   Many sequences (few partials each): a small CTA a (chunk, query head), which
// leaves at once where no sequence begins that goes on.
//   Few sequences: a CTA a (sequence, query head, 32 columns), which finds the
// sequence's chunk among the joins.  (Two sequences of 76 partials, D = 256, 8
// heads: the call took 35.1 us with a CTA a (chunk, head), 33.3 us so.)
constexpr int kJoin = 256, kJoinSmall = 64, kLoad = 6;
__global__ void __launch_bounds__(kJoin) paged_fp8_combine(const PagedFp8Params p, int D, int width) {
    __shared__ float4 so[kJoin];
    __shared__ int s_chunk;
    const int h = blockIdx.y, lane = threadIdx.x & 31;
    const int per = width / 4, groups = blockDim.x / per, grp = threadIdx.x / per, t = blockIdx.z * per + threadIdx.x % per;
    int c = blockIdx.x;
    if (width != D) {
        if (threadIdx.x == 0) s_chunk = -1;
        __syncthreads();
    }
    grid_dependency_wait();  // launched behind the decode grid, whose partials it reads
    grid_launch_dependents();
    if (width != D) {
        for (int i = threadIdx.x; i < p.chunks; i += blockDim.x)
            if (p.joins[i].x == static_cast<int>(blockIdx.x)) s_chunk = i;  // one at most
        __syncthreads();
        c = s_chunk;
        if (c < 0) return;
    }
    const int2 j = p.joins[c];
    // a decode that gave up may not have written its join: nothing out of range is followed
    if (j.x < 0 || j.x >= p.num_seqs || j.y <= c || j.y >= p.chunks) return;
    const int n = grp < groups ? j.y - c + 1 : 0;
    auto slot = [&](int i) { return (static_cast<long long>(c + i) * 2 + (i == 0 ? 1 : 0)) * p.Hq + h; };
    float2 w[kLoad];
    float4 v[kLoad];
    auto ask = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kLoad; ++k) {
            const int i = i0 + k * groups;
            w[k] = make_float2(-INFINITY, 0.f);
            if (i < n) {
                w[k] = p.part_sum[slot(i)];
                v[k] = reinterpret_cast<const float4*>(p.part_o + slot(i) * D)[t];
            }
        }
    };
    ask(grp);
    float m = kLow, sum = 0.f;
    for (int i = lane; i <= j.y - c; i += 32) {
        const float2 x = p.part_sum[slot(i)];
        const float n = fmaxf(m, part_top(x));
        float low;
        const float y = part_weight(x, n, low);
        sum = fmaf(y, low, sum * ex2(m - n));
        m = n;
    }
    const float top = warp_max(m);
    sum *= ex2(m - top);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp; i0 < n;) {
#pragma unroll
        for (int k = 0; k < kLoad; ++k) {
            if (i0 + k * groups >= n) break;
            float low;
            const float x = part_weight(w[k], top, low) * inv;
            acc.x = fmaf(x, v[k].x * low, acc.x);
            acc.y = fmaf(x, v[k].y * low, acc.y);
            acc.z = fmaf(x, v[k].z * low, acc.z);
            acc.w = fmaf(x, v[k].w * low, acc.w);
        }
        i0 += groups * kLoad;
        ask(i0);
    }
    so[threadIdx.x] = acc;
    __syncthreads();
    if (grp != 0) return;
    for (int g = 1; g < groups && g < n; ++g) {
        const float4 b = so[g * per + threadIdx.x];
        acc.x += b.x;
        acc.y += b.y;
        acc.z += b.z;
        acc.w += b.w;
    }
    const long long row = static_cast<long long>(j.x) * p.Hq + h;
    if (p.out_f32)
        reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * D)[t] = acc;
    else
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D)[t] =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    if (t == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2f;
}

template <class C, bool CLUSTER>
cudaError_t launch_cfg(const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    static bool attr_done[64];  // the attribute is per function and device
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !attr_done[dev]) {
            cudaError_t e = cudaFuncSetAttribute(paged_decode_fp8_sm103a<C, CLUSTER>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) attr_done[dev] = true;
        }
    }
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.chunks) * p.n_hgroups * (CLUSTER ? p.num_seqs : 1));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (CLUSTER && p.chunks > 1) {
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = static_cast<unsigned>(p.chunks);
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, paged_decode_fp8_sm103a<C, CLUSTER>, tm, p);
    if (e != cudaSuccess || CLUSTER || p.chunks == 1) return e != cudaSuccess ? e : cudaGetLastError();
    const bool few = p.num_seqs * 8 <= p.chunks;
    const int width = few ? 32 : C::D;
    cfg.gridDim = few ? dim3(static_cast<unsigned>(p.num_seqs), static_cast<unsigned>(p.Hq), C::D / 32)
                      : dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>(p.Hq));
    cfg.blockDim = dim3(few ? kJoin : kJoinSmall);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, paged_fp8_combine, p, static_cast<int>(C::D), width);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int HG>
cudaError_t launch_hg(const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    return p.cluster ? launch_cfg<Fp8Cfg<D, HG>, true>(tm, p, st) : launch_cfg<Fp8Cfg<D, HG>, false>(tm, p, st);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    switch (p.head_cols) {
        case 2: return launch_hg<D, 2>(tm, p, st);
        case 4: return launch_hg<D, 4>(tm, p, st);
        case 8: return launch_hg<D, 8>(tm, p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

PagedFp8Plan paged_fp8_plan(int num_seqs, int Hq, int Hkv, int D, int max_seq_len) {
    PagedFp8Plan pl{};
    const int group = Hq / Hkv;
    pl.subs = (group + 7) / 8;
    pl.heads_per_sub = (group + pl.subs - 1) / pl.subs;
    pl.subs = (group + pl.heads_per_sub - 1) / pl.heads_per_sub;  // none of them empty
    pl.head_cols = 2;  // heads are worked in pairs
    while (pl.head_cols < pl.heads_per_sub) pl.head_cols *= 2;
    pl.n_hgroups = static_cast<long long>(Hkv) * pl.subs;
    // (152 SMs: the size of the workspace is asked for without a device.  On a part
    // with fewer the CTAs of a wave would take turns: right, but slower.)
    // Few and short sequences: a cluster of up to 8 CTAs a (sequence, head), each
    // with at most four blocks, all of them running at once; the parts are
    // joined on chip, in the same launch and without a workspace.  (D = 128, 8 KV
    // heads, clusters and chunks: one sequence of 512 tokens 6.0 and 7.7 us, of
    // 4096 7.9 and 8.4, four of 4096 9.0 and 10.9.)  Clusters lie within a GPC and
    // do not fill every SM: at one CTA an SM 128 of them in clusters of 8 take
    // two turns (four sequences of 1024, D = 256, 4 KV heads: 12.8 and 8.4 us).
    const int ctas = paged_fp8_ctas(D, pl.head_cols);
    const long long slots = 152LL * ctas, blocks = (static_cast<long long>(max_seq_len) + 127) / 128;
    const long long room = (ctas == 1 ? slots / 2 : slots * 27 / 32) / (num_seqs * pl.n_hgroups);
    long long parts = blocks < kMaxCluster ? blocks : kMaxCluster;
    parts = parts < room ? parts : room;
    // Single CTAs (sequences of at most four blocks) need no GPC and may come in
    // up to two waves: three sequences of 194 tokens, 192 heads, D = 256 (96 CTAs)
    // 6.6 us and 13.5 in chunks; on 304 places 512 CTAs of two blocks 10.8 and 11.7,
    // of 1 to 4 blocks 13.6 and 14.5, but 1024 of one block 17.3 and 13.6.
    if (parts < 1 && num_seqs * pl.n_hgroups <= slots * 2) parts = 1;
    if (parts >= 1 && blocks <= 4 * parts) {
        pl.cluster = 1;
        pl.chunks = static_cast<int>(parts);
        return pl;
    }
    // Chunks: as many CTAs as run at once (152 SMs),
    // or a few waves of them where the heads fill one badly; never more than
    // there can be blocks of context.
    long long best = 1;
    double best_use = 0.0;
    for (int waves = 1; waves <= 4; ++waves) {
        const long long c = waves * slots / pl.n_hgroups;
        if (c < 1) continue;
        const double use = static_cast<double>(c * pl.n_hgroups) / static_cast<double>(waves * slots);
        if (use > best_use + 0.03) {
            best_use = use;
            best = c;
        }
    }
    const long long units = num_seqs * blocks;
    if (best > units) best = units;
    pl.chunks = static_cast<int>(best < 1 ? 1 : best);
    if (pl.chunks > 1) {
        const size_t rows = static_cast<size_t>(pl.chunks) * 2 * Hq;
        pl.o_bytes = (rows * D * 4 + 255) & ~size_t(255);
        pl.sum_bytes = (rows * 8 + 255) & ~size_t(255);
        pl.workspace_bytes = pl.o_bytes + pl.sum_bytes + ((static_cast<size_t>(pl.chunks) * 8 + 255) & ~size_t(255));
    }
    return pl;
}

cudaError_t launch_paged_fp8(int D, const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    switch (D) {
        case 64: return launch_d<64>(tm, p, st);
        case 96: return launch_d<96>(tm, p, st);
        case 128: return launch_d<128>(tm, p, st);
        case 192: return launch_d<192>(tm, p, st);
        case 256: return launch_d<256>(tm, p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbattn
