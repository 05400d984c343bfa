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
//     lost to a far larger one in another block.  256 w is split into NP e4m3
//     pieces, each 16 times finer: NP = 3 holds 12 significant bits (bf16
//     output, whose own rounding is 2^-9), NP = 4 holds 16 (fp32 output).
// O^T of a block is read from TMEM and added, times 2^(M - R), to fp32
// registers (thread = column d of the output), so nothing is rescaled in TMEM.
// The softmax sum is kept apart from the weights, in fp32, each thread (token
// lane) with its own reference, so a value row of zeros or of any scale does
// not touch it.
//
// Work split: the context blocks of all sequences, in order, are cut into C
// equal runs ("chunks"), and CTA (c, h) takes chunk c of KV head (or head
// group) h, heads fastest, so that CTAs running side by side read neighbouring
// rows.  A sequence inside one chunk is written out directly; one that crosses
// chunks leaves fp32 partials (o, lse), which paged_fp8_combine joins.
#include <math.h>

#include <mutex>

#include "kernels.h"
#include "ptx.cuh"

namespace gbattn {

namespace {

constexpr int kTok = 128;      // tokens of a cache block: the MMA's M
constexpr int kThreads = 192;  // warps 0-3 softmax and output, 4 TMA, 5 MMA
constexpr int kSoft = 128;
constexpr float kLow = -1e30f;  // a reference below every score, finite so that differences are defined
constexpr float kLn2f = 0.6931471805599453f;

constexpr int up16(int n) { return (n + 15) / 16 * 16; }
constexpr int pow2_cols(int n) { return n <= 32 ? 32 : (n <= 64 ? 64 : (n <= 128 ? 128 : (n <= 256 ? 256 : 512))); }

template <int D_, int HG_, int NP_>
struct Fp8Cfg {
    static constexpr int D = D_, HG = HG_, NP = NP_;
    static constexpr int NCH = (D + 127) / 128;      // 128-byte chunks of a row (zero-filled past D)
    static constexpr int NQ = up16(2 * HG);          // columns of S^T: piece * HG + head
    static constexpr int NW = up16(NP * HG);         // columns of O^T
    static constexpr int HALF_BYTES = NCH * kTok * 128;
    static constexpr int SLOT_BYTES = 2 * HALF_BYTES;
    static constexpr int CTAS = NCH == 1 ? 2 : 1;    // per SM
    static constexpr int STAGES = 3;
    static constexpr int Q_BYTES = NCH * NQ * 128;   // one buffer of query pieces
    static constexpr int P_BYTES = NW * kTok;
    static constexpr int OFF_Q = STAGES * SLOT_BYTES;
    static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_SC = OFF_P + P_BYTES;             // exponent bytes: [stage][K, V][128]
    static constexpr int OFF_RED = OFF_SC + STAGES * 256;      // [2][4][HG] f32
    static constexpr int OFF_QF = OFF_RED + 2 * 4 * HG * 4;    // [2][HG] f32: 2^f * scale_log2
    static constexpr int OFF_LEN = OFF_QF + 2 * HG * 4;        // valid tokens of each slot's block
    static constexpr int OFF_BAR = (OFF_LEN + STAGES * 4 + 7) & ~7;
    static constexpr int N_BAR = 2 * STAGES + 2 + 2 + 2 + 1 + 1 + 1;
    static constexpr int SMEM_BYTES = 1024 + OFF_BAR + N_BAR * 8;
    static constexpr int TM_S = 0;                   // two S^T buffers
    static constexpr int TM_O = 2 * NQ;
    static constexpr int TM_COLS = pow2_cols(2 * NQ + NCH * NW);
    static_assert(SMEM_BYTES <= (CTAS == 2 ? 115712 : 232448), "shared memory budget");
    static_assert(TM_COLS * CTAS <= 512, "tensor memory budget");
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

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N % 16 == 0, "");
#pragma unroll
    for (int i = 0; i < N; i += 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]),
              "=r"(r[i + 6]), "=r"(r[i + 7]), "=r"(r[i + 8]), "=r"(r[i + 9]), "=r"(r[i + 10]), "=r"(r[i + 11]),
              "=r"(r[i + 12]), "=r"(r[i + 13]), "=r"(r[i + 14]), "=r"(r[i + 15])
            : "r"(taddr + i));
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

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ int clamp_len(const PagedFp8Params& p, int s) {
    const int L = p.seq_lens[s];
    return L < 0 ? 0 : (L > p.cap ? p.cap : L);
}
__device__ __forceinline__ int blocks_of(int L) { return (L + kTok - 1) / kTok; }

// U units are cut into N = min(chunks, U) runs, none of them empty: chunk c < N
// holds units [c U / N, (c + 1) U / N), the others none.
__device__ __forceinline__ long long chunk_start(long long c, long long U, long long N) { return c >= N ? U : c * U / N; }

// A warp's walk over its chunk's segments: [b0, b1) of sequence s, of `nblk`
// blocks in all.  Every lane of the warp calls next(); the lengths of 32
// sequences are held across the lanes.
struct Walk {
    int s, L, nblk, b0, b1;
    long long rem;  // units of the chunk after this segment
    int base, Llane;

    __device__ __forceinline__ void load(const PagedFp8Params& p, int lane) {
        const int i = base + lane;
        Llane = i < p.num_seqs ? clamp_len(p, i) : 0;
    }
    __device__ __forceinline__ void take(int lane, long long n, int from) {
        L = __shfl_sync(0xffffffffu, Llane, s - base);
        nblk = blocks_of(L);
        b0 = from;
        const long long left = nblk - from;
        b1 = from + static_cast<int>(left < n ? left : n);
        rem = n - (b1 - b0);
    }
    __device__ __forceinline__ void start(const PagedFp8Params& p, int s0, int off, long long n) {
        const int lane = threadIdx.x & 31;
        s = s0;
        base = s0;
        load(p, lane);
        take(lane, n, off);
    }
    // The next sequence that has tokens; false when the chunk is done.
    __device__ __forceinline__ bool next(const PagedFp8Params& p) {
        if (rem <= 0) return false;
        const int lane = threadIdx.x & 31;
        for (;;) {
            const unsigned has = __ballot_sync(0xffffffffu, Llane > 0 && base + lane > s);
            if (has) {
                s = base + __ffs(static_cast<int>(has)) - 1;
                take(lane, rem, 0);
                return true;
            }
            s = base + 31;
            base += 32;
            if (base >= p.num_seqs) return false;
            load(p, lane);
        }
    }
};

// The queries of sequence s, heads [h0, h0 + nh), as two e4m3 pieces a value
// into a buffer of K-major 128-byte swizzled rows, row piece * HG + head; and
// 2^f * scale_log2 of each head.  One warp a head.  A row with a NaN or an
// infinity becomes NaN where it has it, so that head's result is NaN.
template <class C>
__device__ __forceinline__ void put_queries(const PagedFp8Params& p, int s, int h0, int nh, uint8_t* sq, float* qf,
                                            int warp, int lane) {
    constexpr int PAIRS = C::D / 2, PL = (PAIRS + 31) / 32;
    for (int h = warp; h < C::HG; h += 4) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + s * p.q_stride + static_cast<long long>(h0 + h) * C::D);
        uint32_t x[PL];
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int pr = lane + 32 * i;
            x[i] = (h < nh && pr < PAIRS) ? src[pr] : 0u;
            const uint32_t a = x[i] & 0x7FFFu, b = (x[i] >> 16) & 0x7FFFu;
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
                float lo = __uint_as_float(x[i] << 16), hi = __uint_as_float(x[i] & 0xFFFF0000u);
                if ((x[i] & 0x7F80u) == 0x7F80u) lo = NAN;
                if ((x[i] & 0x7F800000u) == 0x7F800000u) hi = NAN;
                lo *= inv;
                hi *= inv;
                const uint32_t c0 = pack_fp8x2<false>(lo, hi);
                const float2 f0 = unpack_fp8x2<false>(c0);
                const uint32_t c1 = pack_fp8x2<false>((lo - f0.x) * 16.f, (hi - f0.y) * 16.f);
                const int e = 2 * pr, ch = e >> 7, col = e & 127;
#pragma unroll
                for (int piece = 0; piece < 2; ++piece) {
                    const int row = piece * C::HG + h;
                    *reinterpret_cast<uint16_t*>(sq + ch * (C::NQ * 128) + row * 128 + (((col >> 4) ^ (row & 7)) << 4) +
                                                 (col & 15)) = static_cast<uint16_t>(piece ? c1 : c0);
                }
            }
        }
    }
}

template <class C>
__global__ void __launch_bounds__(kThreads, C::CTAS)
    paged_decode_fp8_sm103a(const __grid_constant__ CUtensorMap tmKV, const PagedFp8Params p) {
    constexpr int D = C::D, HG = C::HG, NP = C::NP, NQ = C::NQ, NW = C::NW, NCH = C::NCH, STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    float* sred = reinterpret_cast<float*>(smem + C::OFF_RED);
    float* sqf = reinterpret_cast<float*>(smem + C::OFF_QF);
    volatile int* slen = reinterpret_cast<volatile int*>(smem + C::OFF_LEN);
    const uint32_t bar0 = sb + C::OFF_BAR;
    auto b_full = [&](int i) { return bar0 + 8 * i; };
    auto b_empty = [&](int i) { return bar0 + 8 * (STAGES + i); };
    auto b_sfull = [&](int i) { return bar0 + 8 * (2 * STAGES + i); };
    auto b_sempty = [&](int i) { return bar0 + 8 * (2 * STAGES + 2 + i); };
    auto b_qfull = [&](int i) { return bar0 + 8 * (2 * STAGES + 4 + i); };
    const uint32_t b_pfull = bar0 + 8 * (2 * STAGES + 6), b_ofull = b_pfull + 8, b_done = b_pfull + 16;
    __shared__ int abort_storage;
    __shared__ uint32_t tmem_base_storage;
    __shared__ long long s_sum[kThreads / 32];
    __shared__ long long s_u[3];  // u0, u1, U
    __shared__ int s_first[2];    // first sequence, first block of it
    __shared__ uint32_t s_issued; // blocks whose loads were issued
    volatile int* abort_flag = &abort_storage;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = blockIdx.x / p.n_hgroups, hg = blockIdx.x % p.n_hgroups;
    const int kvh = hg / p.subs, sub = hg % p.subs;
    const int h0 = kvh * p.group + sub * p.heads_per_sub;
    const int nh = min(p.heads_per_sub, p.group - sub * p.heads_per_sub);
    grid_launch_dependents();  // the combine may queue up; it waits for this grid to finish

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(b_full(i), 1);
            mbar_init(b_empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_sfull(i), 1);
            mbar_init(b_sempty(i), 4);
            mbar_init(b_qfull(i), 4);
        }
        mbar_init(b_pfull, 4);
        mbar_init(b_ofull, 1);
        mbar_init(b_done, 1);
        abort_storage = 0;
        s_issued = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmKV);
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(&tmem_base_storage), C::TM_COLS);
        tmem_relinquish();
    }

    // ---- this chunk's units: total, then the sequence its first unit lies in
    {
        long long sum = 0;
        bool bad = false;
        for (int s = threadIdx.x; s < p.num_seqs; s += kThreads) {
            const int L = p.seq_lens[s];
            bad |= L < 0 || L > p.cap;
            sum += blocks_of(clamp_len(p, s));
        }
        if (bad && blockIdx.x == 0 && p.status) atomicOr(p.status, kDevBadSeqlen);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        long long U = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) U += s_sum[w];
        __syncthreads();
        const long long N = U < p.chunks ? U : p.chunks;
        const long long u0 = chunk_start(chunk, U, N), u1 = chunk_start(chunk + 1, U, N);
        if (threadIdx.x == 0) {
            s_u[0] = u0;
            s_u[1] = status_has_timeout(p.status, kDevTimeout) ? u0 : u1;  // after a give-up nothing more is begun
            s_u[2] = U;
        }
        long long run = 0;
        if (u1 > u0) {
            for (int base = 0; base < p.num_seqs; base += kThreads) {
                const int s = base + threadIdx.x;
                const int T = s < p.num_seqs ? blocks_of(clamp_len(p, s)) : 0;
                long long incl = T;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long n = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += n;
                }
                if (lane == 31) s_sum[warp] = incl;
                __syncthreads();
                long long before = run, all = 0;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) {
                    if (w < warp) before += s_sum[w];
                    all += s_sum[w];
                }
                const long long at = before + incl - T;  // units before sequence s
                if (T > 0 && at <= u0 && u0 < at + T) {
                    s_first[0] = s;
                    s_first[1] = static_cast<int>(u0 - at);
                }
                run += all;
                __syncthreads();
                if (run > u0) break;  // found (uniform)
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base_storage;
    const long long u0 = s_u[0], u1 = s_u[1], U = s_u[2];
    const uint32_t n_units = static_cast<uint32_t>(u1 - u0);
    bool ok = true;

    if (warp < 4) {
        // ---------------------------------------------------- softmax and output
        if (hg == 0 && threadIdx.x == 0 && p.chunks > 1 && n_units == 0) p.joins[chunk] = make_int2(-1, 0);
        // sequences without context, of this chunk's share: zeros and -inf
        auto zero_empty = [&]() {
            for (long long i0 = warp * 32; i0 * p.chunks < p.num_seqs; i0 += kSoft) {
                const long long s = chunk + (i0 + lane) * p.chunks;
                unsigned none = __ballot_sync(0xffffffffu, s < p.num_seqs && clamp_len(p, static_cast<int>(s)) == 0);
                for (; none; none &= none - 1) {
                    const long long row = (chunk + (i0 + __ffs(static_cast<int>(none)) - 1) * p.chunks) * p.Hq + h0;
                    for (int i = lane; i < nh * D; i += 32) {
                        if (p.out_f32)
                            static_cast<float*>(p.out)[row * D + i] = 0.f;
                        else
                            static_cast<uint16_t*>(p.out)[row * D + i] = 0;
                    }
                    if (lane < nh && p.lse) p.lse[row + lane] = -INFINITY;
                }
            }
        };
        if (n_units == 0) zero_empty();
        if (n_units > 0) {
            Walk w, ahead;  // `ahead` is one segment further: its queries are laid out early
            w.start(p, s_first[0], s_first[1], n_units);
            ahead = w;
            put_queries<C>(p, w.s, h0, nh, smem + C::OFF_Q, sqf, warp, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_qfull(0));
            named_bar_sync(1, kSoft);  // sqf is read by every warp
            zero_empty();
            const uint32_t tlane = static_cast<uint32_t>(warp) << 21;  // this warp's 32 TMEM lanes
            uint32_t g = 0;  // blocks done
            int seg = 0;
            bool more = true;
            while (more) {
                if (ahead.next(p)) {  // queries of the next segment: its buffer's last reader was segment seg - 1
                    put_queries<C>(p, ahead.s, h0, nh, smem + C::OFF_Q + ((seg + 1) & 1) * C::Q_BYTES,
                                   sqf + ((seg + 1) & 1) * HG, warp, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_qfull((seg + 1) & 1));
                }
                float o[NCH][HG], R[HG], Mp[HG], mref[HG], l[HG];
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    R[h] = mref[h] = Mp[h] = kLow;
                    l[h] = 0.f;
#pragma unroll
                    for (int c = 0; c < NCH; ++c) o[c][h] = 0.f;
                }
                // O^T of the block before: o += 2^(M - R - 8) sum_i piece_i / 16^i
                auto add_o = [&](uint32_t gi) {
                    if (!mbar_wait(b_ofull, gi & 1, abort_flag)) ok = false;
                    tc_fence_after();
                    float beta[HG];
#pragma unroll
                    for (int h = 0; h < HG; ++h) {
                        if (Mp[h] > R[h] + 40.f) {  // same in every thread
                            const float a = ex2(R[h] - Mp[h]);
                            R[h] = Mp[h];
#pragma unroll
                            for (int c = 0; c < NCH; ++c) o[c][h] *= a;
                        }
                        beta[h] = ex2(Mp[h] - R[h] - 8.f);
                    }
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        uint32_t r[NW];
                        tmem_ld<NW>(tm + tlane + C::TM_O + c * NW, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < HG; ++h) {
                            float x = __uint_as_float(r[(NP - 1) * HG + h]);
#pragma unroll
                            for (int i = NP - 2; i >= 0; --i) x = fmaf(x, 0.0625f, __uint_as_float(r[i * HG + h]));
                            o[c][h] = fmaf(x, beta[h], o[c][h]);
                        }
                    }
                    tc_fence_before();
                };
                const float* qf = sqf + (seg & 1) * HG;
                bool quit = false;
                for (int b = w.b0; b < w.b1; ++b, ++g) {
                    const int slot = static_cast<int>(g % STAGES);
                    if (!mbar_wait(b_full(slot), (g / STAGES) & 1, abort_flag)) ok = false;
                    if (!mbar_wait(b_sfull(g & 1), (g >> 1) & 1, abort_flag)) ok = false;
                    tc_fence_after();
                    uint32_t r[NQ];
                    tmem_ld<NQ>(tm + tlane + C::TM_S + (g & 1) * NQ, r);
                    const int nvalid = slen[slot];
                    const bool valid = static_cast<int>(threadIdx.x) < nvalid;
                    const uint8_t* sc = smem + C::OFF_SC + slot * 256;
                    const float kf = exp2_byte(sc[threadIdx.x]);
                    const float ev = static_cast<float>(static_cast<int>(sc[128 + threadIdx.x]) - 127);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_sempty(g & 1));
                    float u[HG];
#pragma unroll
                    for (int h = 0; h < HG; ++h) {
                        const float dot = fmaf(__uint_as_float(r[HG + h]), 0.0625f, __uint_as_float(r[h]));
                        const float s = dot * kf * qf[h];
                        if (valid) {
                            if (s > mref[h] + 60.f) {  // fp32 has room for sums of 2^60 and more
                                l[h] *= ex2(mref[h] - s);
                                mref[h] = s;
                            }
                            l[h] += ex2(s - mref[h]);
                        }
                        u[h] = valid ? s + ev : -INFINITY;
                    }
                    float* red = sred + (g & 1) * 4 * HG;
#pragma unroll
                    for (int h = 0; h < HG; ++h) {
                        const float m = warp_max(u[h]);
                        if (lane == 0) red[warp * HG + h] = m;
                    }
                    if (named_bar_or(1, kSoft, !ok)) {  // all four warps leave together
                        quit = true;
                        break;
                    }
                    // the value rows past the context meet weight 0: they must be finite
                    if (!valid) {
#pragma unroll
                        for (int c = 0; c < NCH; ++c) {
                            uint4* v = reinterpret_cast<uint4*>(smem + slot * C::SLOT_BYTES + C::HALF_BYTES + c * kTok * 128 +
                                                                threadIdx.x * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (b > w.b0) add_o(g - 1);  // the weights' buffer and O^T are free again
                    float y[NP * HG];
#pragma unroll
                    for (int h = 0; h < HG; ++h) {
                        const float M = fmaxf(fmaxf(fmaxf(red[h], red[HG + h]), fmaxf(red[2 * HG + h], red[3 * HG + h])), kLow);
                        Mp[h] = M;
                        y[h] = ex2(u[h] - M + 8.f);
                    }
                    // pieces, lowest column first: column piece * HG + head
                    uint32_t w8[NW / 4];
#pragma unroll
                    for (int i = 0; i < NW / 4; ++i) w8[i] = 0u;
                    if constexpr (HG == 1) {
                        float x = y[0];
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            const uint32_t c = pack_fp8x2<false>(x, 0.f);
                            w8[0] |= (c & 0xFFu) << (8 * i);
                            x = (x - unpack_fp8x2<false>(c).x) * 16.f;
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < HG; h += 2) {
                            float x0 = y[h], x1 = y[h + 1];
#pragma unroll
                            for (int i = 0; i < NP; ++i) {
                                const uint32_t c = pack_fp8x2<false>(x0, x1);
                                const int col = i * HG + h;
                                w8[col / 4] |= c << (8 * (col & 3));
                                if (i + 1 < NP) {
                                    const float2 f = unpack_fp8x2<false>(c);
                                    x0 = (x0 - f.x) * 16.f;
                                    x1 = (x1 - f.y) * 16.f;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NW / 16; ++i)
                        st_shared_v4(sb + C::OFF_P + i * (kTok * 16) + threadIdx.x * 16, w8[4 * i], w8[4 * i + 1],
                                     w8[4 * i + 2], w8[4 * i + 3]);
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_pfull);
                }
                if (quit) break;
                add_o(g - 1);
                // ---- the segment's softmax sum over the 128 token lanes, then its output
                float inv[HG], lse2[HG];
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float m = warp_max(mref[h]);
                    if (lane == 0) sred[warp * HG + h] = m;
                }
                named_bar_sync(1, kSoft);
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float m = fmaxf(fmaxf(sred[h], sred[HG + h]), fmaxf(sred[2 * HG + h], sred[3 * HG + h]));
                    float x = l[h] * ex2(mref[h] - m);
#pragma unroll
                    for (int of = 16; of; of >>= 1) x += __shfl_xor_sync(0xffffffffu, x, of);
                    if (lane == 0) sred[4 * HG + warp * HG + h] = x;
                    mref[h] = m;
                }
                if (named_bar_or(1, kSoft, !ok)) break;
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float* x = sred + 4 * HG + h;
                    const float sum = (x[0] + x[HG]) + (x[2 * HG] + x[3 * HG]);
                    inv[h] = sum == 0.f ? 0.f : ex2(R[h] - mref[h]) / sum;
                    lse2[h] = sum == 0.f ? -INFINITY : mref[h] + __log2f(sum);
                }
                const bool whole = w.b0 == 0 && w.b1 == w.nblk;
                if (hg == 0 && threadIdx.x == 0 && p.chunks > 1 && w.rem == 0) {
                    // does this segment's sequence begin here and go on in other chunks?
                    const long long end = u1 + (w.nblk - w.b1);
                    const bool begins = w.b0 == 0 && w.b1 < w.nblk;
                    const long long N = U < p.chunks ? U : p.chunks;
                    p.joins[chunk] = begins ? make_int2(w.s, static_cast<int>((end * N + U - 1) / U - 1))
                                            : make_int2(-1, 0);
                }
                const long long part = (static_cast<long long>(chunk) * 2 + (w.b0 == 0 ? 1 : 0)) * p.Hq + h0;
                const long long row = static_cast<long long>(w.s) * p.Hq + h0;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const int d = c * 128 + threadIdx.x;
                    if (d < D) {
#pragma unroll
                        for (int h = 0; h < HG; ++h)
                            if (h < nh) {
                                const float x = o[c][h] * inv[h];
                                if (!whole)
                                    p.part_o[(part + h) * D + d] = x;
                                else if (p.out_f32)
                                    static_cast<float*>(p.out)[(row + h) * D + d] = x;
                                else
                                    static_cast<uint16_t*>(p.out)[(row + h) * D + d] =
                                        static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFFu);
                            }
                    }
                }
                if (threadIdx.x == 0) {
#pragma unroll
                    for (int h = 0; h < HG; ++h)
                        if (h < nh) {
                            if (!whole)
                                p.part_lse[part + h] = lse2[h];
                            else if (p.lse)
                                p.lse[row + h] = lse2[h] * kLn2f;
                        }
                }
                ++seg;
                more = w.next(p);
                named_bar_sync(1, kSoft);  // the reduction scratch is free again
            }
        }
    } else if (warp == 4) {
        // ---------------------------------------------------- cache loads
        if (n_units > 0) {
            Walk w;
            w.start(p, s_first[0], s_first[1], n_units);
            uint32_t g = 0;
            bool more = true;
            while (more && ok) {
                const int32_t* row = p.block_table + static_cast<long long>(w.s) * p.max_blocks;
                int ids = 0;  // 32 table entries, one a lane
                for (int b = w.b0; b < w.b1; ++b, ++g) {
                    const int slot = static_cast<int>(g % STAGES);
                    const int at = (b - w.b0) & 31;
                    if (at == 0) ids = b + lane < w.b1 ? row[b + lane] : 0;
                    const int blk = __shfl_sync(0xffffffffu, ids, at);
                    if (g >= STAGES && !mbar_wait(b_empty(slot), (g / STAGES - 1) & 1, abort_flag)) ok = false;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        const bool good = blk >= 0 && blk < p.num_blocks;
                        slen[slot] = good ? min(kTok, w.L - b * kTok) : 0;
                        if (good) {
                            mbar_arrive_expect_tx(b_full(slot), C::SLOT_BYTES + 256);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const long long r = static_cast<long long>(half) * p.num_blocks + blk;
#pragma unroll
                                for (int c = 0; c < NCH; ++c)
                                    tma_load_3d(sb + slot * C::SLOT_BYTES + half * C::HALF_BYTES + c * kTok * 128, &tmKV,
                                                b_full(slot), c * 128, kvh, static_cast<int>(r * kTok));
                                bulk_load(sb + C::OFF_SC + slot * 256 + half * 128, p.scales + (r * p.Hkv + kvh) * kTok, 128,
                                          b_full(slot));
                            }
                        } else {
                            if (p.status) atomicOr(p.status, kDevBadIndex);
                            mbar_arrive(b_full(slot));
                        }
                        s_issued = g + 1;
                    }
                    __syncwarp();
                }
                if (ok) more = w.next(p);
            }
            if (!ok) *abort_flag = 1;
        }
    } else {
        // ---------------------------------------------------- matrix products
        if (n_units > 0) {
            const uint32_t id_s = idesc_f8(128, NQ, p.e5m2 ? 1u : 0u, false, false);
            const uint32_t id_o = idesc_f8(128, NW, p.e5m2 ? 1u : 0u, true, true);
            Walk w;
            w.start(p, s_first[0], s_first[1], n_units);
            int seg = 0, b = w.b0;
            bool more = true;
            // S^T of unit i, one unit ahead of O^T
            auto issue_s = [&](uint32_t i) {
                const int slot = static_cast<int>(i % STAGES);
                bool got = mbar_wait(b_full(slot), (i / STAGES) & 1, abort_flag);
                if (b == w.b0) got = got && mbar_wait(b_qfull(seg & 1), (seg >> 1) & 1, abort_flag);
                if (i >= 2) got = got && mbar_wait(b_sempty(i & 1), ((i >> 1) - 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, got)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t k = sb + slot * C::SLOT_BYTES, q = sb + C::OFF_Q + (seg & 1) * C::Q_BYTES;
#pragma unroll
                    for (int ks = 0; ks < D / 32; ++ks)
                        mma_f8_ss(tm + C::TM_S + (i & 1) * NQ,
                                  sdesc_sw128(k + (ks / 4) * (kTok * 128) + (ks % 4) * 32, 16, 1024),
                                  sdesc_sw128(q + (ks / 4) * (NQ * 128) + (ks % 4) * 32, 16, 1024), id_s, ks > 0);
                    mma_commit(b_sfull(i & 1));
                }
                __syncwarp();
                if (++b == w.b1) {
                    more = w.next(p);
                    b = w.b0;
                    ++seg;
                }
                return true;
            };
            ok = issue_s(0);
            for (uint32_t i = 0; ok && i < n_units; ++i) {
                ok = !more || issue_s(i + 1);
                const int slot = static_cast<int>(i % STAGES);
                ok = __all_sync(0xffffffffu, ok && mbar_wait(b_pfull, i & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t v = sb + slot * C::SLOT_BYTES + C::HALF_BYTES, pp = sb + C::OFF_P;
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f8_ss(tm + C::TM_O + c * NW, sdesc_sw128(v + c * (kTok * 128) + ks * 4096, 16, 1024),
                                      sdesc_plain(pp + ks * 512, 128, kTok * 16), id_o, ks > 0);
                    mma_commit(b_ofull);
                    mma_commit(b_empty(slot));
                }
                __syncwarp();
            }
            if (!ok) *abort_flag = 1;
            if (elect_one()) mma_commit(b_done);  // every product issued has finished before TMEM is freed
            __syncwarp();
            mbar_wait_drain(b_done, 0);
        }
    }
    if (warp < 4 && !ok) *abort_flag = 1;
    __syncthreads();
    if (*abort_flag) {
        if (threadIdx.x == 0 && p.status) atomicOr(p.status, kDevTimeout);
        // copies still in flight land (bounded) before the block's memory is given up
        if (threadIdx.x == 0)
            for (uint32_t g = s_issued < STAGES ? 0 : s_issued - STAGES; g < s_issued; ++g)
                mbar_wait_drain(b_full(g % STAGES), (g / STAGES) & 1);
    }
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tm, C::TM_COLS);
    }
}

// Joins the partials of a sequence that crosses chunks: chunk c's second slot
// (the sequence begins there), the first slots of the chunks up to its last.
// One warp a (chunk, query head); chunks where none begins leave at once.
__global__ void __launch_bounds__(128) paged_fp8_combine(const PagedFp8Params p, int D) {
    grid_dependency_wait();  // launched behind the decode grid, whose partials it reads
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int2 j = p.joins[c];
    // a decode that gave up may not have written its join: nothing out of range is followed
    if (j.x < 0 || j.x >= p.num_seqs || j.y <= c || j.y >= p.chunks || h >= p.Hq) return;
    if (status_has_timeout(p.status, kDevTimeout)) return;
    auto slot = [&](int i) { return (static_cast<long long>(i) * 2 + (i == c ? 1 : 0)) * p.Hq + h; };
    float mx = -INFINITY;
    for (int i = c + lane; i <= j.y; i += 32) mx = fmaxf(mx, p.part_lse[slot(i)]);
    mx = warp_max(mx);
    const float ms = mx == -INFINITY ? 0.f : mx;
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    float sum = 0.f;
#pragma unroll 4
    for (int i = c; i <= j.y; ++i) {
        const long long r = slot(i);
        const float w = ex2(p.part_lse[r] - ms);
        sum += w;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (lane + 32 * k < D) acc[k] = fmaf(w, p.part_o[r * D + lane + 32 * k], acc[k]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long row = static_cast<long long>(j.x) * p.Hq + h;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (lane + 32 * k < D) {
            const float x = acc[k] * inv;
            if (p.out_f32)
                static_cast<float*>(p.out)[row * D + lane + 32 * k] = x;
            else
                static_cast<uint16_t*>(p.out)[row * D + lane + 32 * k] =
                    static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFFu);
        }
    if (lane == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (ms + __log2f(sum)) * kLn2f;
}

template <class C>
cudaError_t launch_cfg(const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    static bool attr_done[64];  // the attribute is per function and device
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !attr_done[dev]) {
            cudaError_t e = cudaFuncSetAttribute(paged_decode_fp8_sm103a<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 C::SMEM_BYTES);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) attr_done[dev] = true;
        }
    }
    paged_decode_fp8_sm103a<C><<<static_cast<unsigned>(p.chunks) * p.n_hgroups, kThreads, C::SMEM_BYTES, st>>>(tm, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.chunks == 1) return e;  // one chunk: no sequence crosses chunks
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>((p.Hq + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_fp8_combine, p, static_cast<int>(C::D));
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int HG>
cudaError_t launch_np(const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    return p.out_f32 ? launch_cfg<Fp8Cfg<D, HG, 4>>(tm, p, st) : launch_cfg<Fp8Cfg<D, HG, 3>>(tm, p, st);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tm, const PagedFp8Params& p, cudaStream_t st) {
    switch (p.head_cols) {
        case 1: return launch_np<D, 1>(tm, p, st);
        case 2: return launch_np<D, 2>(tm, p, st);
        case 4: return launch_np<D, 4>(tm, p, st);
        case 8: return launch_np<D, 8>(tm, p, st);
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
    pl.head_cols = 1;
    while (pl.head_cols < pl.heads_per_sub) pl.head_cols *= 2;
    pl.n_hgroups = static_cast<long long>(Hkv) * pl.subs;
    // Chunks: as many CTAs as run at once (152 SMs, two each up to D = 128),
    // or a few waves of them where the heads fill one badly; never more than
    // there can be blocks of context.
    const long long slots = 152LL * (D <= 128 ? 2 : 1);
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
    const long long units = static_cast<long long>(num_seqs) * ((max_seq_len + 127) / 128);
    if (best > units) best = units;
    pl.chunks = static_cast<int>(best < 1 ? 1 : best);
    if (pl.chunks > 1) {
        const size_t rows = static_cast<size_t>(pl.chunks) * 2 * Hq;
        pl.o_bytes = (rows * D * 4 + 255) & ~size_t(255);
        pl.lse_bytes = (rows * 4 + 255) & ~size_t(255);
        pl.workspace_bytes = pl.o_bytes + pl.lse_bytes + ((static_cast<size_t>(pl.chunks) * 8 + 255) & ~size_t(255));
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
