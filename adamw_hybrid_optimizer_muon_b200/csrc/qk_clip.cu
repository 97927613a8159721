// QK-Clip: each attention head's largest logit, and the query and key weights
// scaled down by it ("MuonClip Optimizer", QK-Clip: scale Q and K when the
// largest logit exceeds a threshold).
//
//   S_h   = max over sequences and visible (i, j) of scale * q_i . k_j   (or |.|)
//   g_h   = min(1, tau / S_h)
//   W_k of key head c   <- W_k * G_c^(1 - alpha),  G_c = min of g_h over its query heads
//   W_q of query head h <- W_q * g_h / G_c^(1 - alpha)        (alike W_q g_h^alpha without shared heads)
// so that every head's logits scale by its own g_h.
//
// The maximum is one GEMM per head without an output: bound by the tensor cores.
// It runs as tcgen05.mma (bf16 operands, fp32 accumulators in TMEM); the
// epilogue reads each accumulator once and keeps one running maximum per row.
//
// One CTA per SM, 320 threads: warp 0 loads (TMA), warp 1 issues the MMAs, two
// groups of four warps reduce. A CTA holds 256 queries of one head, as two
// blocks of 128 rows, in shared memory, and streams tiles of N keys past them,
// 64 columns of the head dimension a stage; both blocks multiply a key tile
// before it is released, which halves the key traffic from L2, and while one
// block's accumulator is reduced (480 cycles) the other's is computed (1024
// for 128 x 256 x 128).
//
// Work is counted in (128 queries x N keys) products, of which causality and the
// sequences' ends leave only those with a visible pair. A maximum can be cut
// anywhere, so the CTAs take equal shares of that count, wherever it falls in a
// head or a sequence, with no scheduler and no second pass: each segment ends
// in one atomic maximum per warp (order does not change a maximum).
//
// 4096 tokens x 32 heads x 128, causal: 48 us, 1.44 PFLOP/s of the visible pairs
// (6 % more are computed in the diagonal tiles), 61 us at the 1.54 GHz that the
// power cap leaves in a long run. About 1250 cycles a product of 1024; what is
// left is the issuing warp's own time between products and the shared memory
// that MMA operands (96 bytes a clock) and arriving keys (32) share. Under 1024
// tokens a head the latency of start and end, about 5 us, counts. CTA pairs
// (256-row blocks, half the keys loaded by each CTA) were slower, 58 us: each
// product then waits for an arrival from the other CTA.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace ma {

namespace {

constexpr int kBK = 64;                       // columns of the head dimension per stage (128 bytes: the swizzle width)
constexpr int kRows = 128;                    // queries per block of rows (TMEM lanes)
constexpr int kThreads = 320;
constexpr uint32_t kQChunk = kRows * kBK * 2;  // 16 KB
constexpr uint32_t kSmemMax = 232448;          // 227 KB
constexpr uint32_t kCtlBytes = 512;
constexpr int kMaxChunks = 4;                  // head dimension up to 256
constexpr int kMaxStages = 12;
// Buffers for blocks of queries: where the shared memory allows, a third one, so
// that the next segment's first block arrives while this one's are in use
// (12 sequences of 500 tokens, 16 heads x 128: 10.5 us, 12.7 with two).
constexpr int q_buffers(int ch) { return ch <= 2 ? 3 : 2; }
// Stages of N keys x 64 columns that fit beside them.
constexpr int stages(int n, int ch) {
    const int fit =
        (int)((kSmemMax - 1024 - kCtlBytes - q_buffers(ch) * ch * kQChunk) / (uint32_t)(n * kBK * 2));
    return fit < kMaxStages ? fit : kMaxStages;
}
constexpr long long kDrainNs = 50000000LL;  // bound of the waits for this CTA's own copies and MMAs at its end

// Bounded wait for the phase with the given parity of a barrier: as
// mbar_wait_ctl, for waits that are mostly over at once (wait) and, when not,
// short. The timer is looked at only after 64 attempts that each slept up to
// 1 us. False after the limit (recorded, and the abort raised) or, unless
// `drain`, once another warp has raised the abort. Whole warps wait, and every
// lane gets the same answer: what follows a wait needs all of them.
struct Waits {
    volatile int* abort;
    long long limit_ns;
    int* status;
};
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, const Waits& W, long long limit_ns, bool drain) {
    constexpr uint32_t kAll = 0xffffffffu;
    for (int it = 0; it < 64; ++it) {
        if (__all_sync(kAll, mbar_try_wait_sleep(bar, parity, 1000u))) return true;
        if (!drain && __any_sync(kAll, *W.abort)) return false;
    }
    const uint64_t t0 = globaltimer();
    while (!__all_sync(kAll, mbar_try_wait_sleep(bar, parity, 1000u))) {
        if (!drain && __any_sync(kAll, *W.abort)) return false;
        if (__any_sync(kAll, (long long)(globaltimer() - t0) > limit_ns)) {
            record_error(W.status, MA_ERR_TIMEOUT);
            *W.abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Waits& W) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_on(bar, parity, W, W.limit_ns, false);
}

struct QkLaunch {
    CUtensorMap mq, mk;      // {dim, tokens, heads, sequences}
    const int32_t* offsets;  // packed: first token of each sequence and the end; NULL: sequences of `len` tokens
    int32_t seqs, len, total;  // len: tokens per sequence (packed: the longest); total: tokens of a packed batch
    int32_t heads, kv;
    int32_t given;  // `out` holds values of the caller's (else -infinity)
    float scale;
    float* out;
    long long wait_limit_ns;
    int* status;
};

struct QkCtl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full[3], q_empty[3];
    uint64_t acc_full[4], acc_empty[4];
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    int64_t units_begin, units_end;  // this CTA's share
    int32_t b0;                      // the sequence it begins in
    int32_t pad;
    int64_t rest0;                   // units before it in that sequence
};
static_assert(sizeof(QkCtl) <= kCtlBytes, "control block");

// Sequence b: first token, and length, both kept inside the batch whatever the
// offsets hold (those that do not fit are recorded).
struct Seq {
    int32_t tok0, len;
};
__device__ __forceinline__ Seq sequence(const QkLaunch& L, int b) {
    if (!L.offsets) return {0, L.len};
    const int lo = L.offsets[b], hi = L.offsets[b + 1];
    const int a = min(max(lo, 0), L.total);
    const int n = min(max(min(hi, L.total) - a, 0), L.len);
    if (a != lo || a + n != hi) record_error(L.status, MA_ERR_BOUNDS);
    return {a, n};
}

// Units (a block of 128 queries times a tile of N keys) of one head of a
// sequence of len tokens, before query block t (causal: block t sees the keys
// up to its last query; ceil((t + 1) * 128 / N) tiles).
template <int N, bool CAUSAL>
__device__ __forceinline__ int64_t units_before(int64_t t, int len) {
    if (!CAUSAL) return t * ((len + N - 1) / N);
    return N == 256 ? (t + 1) * (t + 1) / 4 : t * (t + 1) / 2;
}
template <int N, bool CAUSAL>
__device__ __forceinline__ int64_t units_of_head(int len) {
    return units_before<N, CAUSAL>((len + kRows - 1) / kRows, len);
}

// The value of lane 0, known to be the same in every lane.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A part of one item (256 queries of a head, in two blocks of 128): key tiles
// [a0, b0) for the lower block of rows and [a1, b1) for the upper one, taken
// tile by tile, the lower block first. Every tile from the first to the last
// is used by a block.
struct Segment {
    int b, h, q0, tok0, len;
    int a0, b0, a1, b1;
    __device__ __forceinline__ int first() const { return a0 < b0 && (a1 >= b1 || a0 <= a1) ? a0 : a1; }
    __device__ __forceinline__ int last() const { return max(a0 < b0 ? b0 : 0, a1 < b1 ? b1 : 0); }
    __device__ __forceinline__ bool in0(int j) const { return j >= a0 && j < b0; }
    __device__ __forceinline__ bool in1(int j) const { return j >= a1 && j < b1; }
    __device__ __forceinline__ void make_uniform() {
        b = uniform(b);
        h = uniform(h);
        q0 = uniform(q0);
        tok0 = uniform(tok0);
        a0 = uniform(a0);
        b0 = uniform(b0);
        a1 = uniform(a1);
        b1 = uniform(b1);
    }
};

// Walks this CTA's share, segment by segment; every role makes the same walk.
template <int N, bool CAUSAL>
struct Walk {
    const QkLaunch& L;
    int64_t left, rest;  // units left; units of (b, h) before the next one
    int b, h, q;         // next item
    Seq sq;
    int64_t item0;       // units of (b, h) before item q

    __device__ Walk(const QkLaunch& l, const QkCtl* c) : L(l), left(c->units_end - c->units_begin), b(c->b0) {
        if (left <= 0) return;
        sq = sequence(L, b);
        const int64_t per_head = units_of_head<N, CAUSAL>(sq.len);
        h = (int)(c->rest0 / per_head);
        rest = c->rest0 - (int64_t)h * per_head;
        int lo = 0, hi = (sq.len - 1) / (2 * kRows);
        while (lo < hi) {  // last item that begins at or before `rest`
            const int mid = (lo + hi + 1) >> 1;
            if (units_before<N, CAUSAL>(2 * mid, sq.len) <= rest) lo = mid;
            else hi = mid - 1;
        }
        q = lo;
        item0 = units_before<N, CAUSAL>(2 * q, sq.len);
    }
    __device__ bool next(Segment& g) {
        if (left <= 0) return false;
        while (sq.len == 0) {  // units are left, so a sequence with tokens follows
            sq = sequence(L, ++b);
        }
        g.b = L.offsets ? 0 : b;
        g.h = h;
        g.q0 = q * 2 * kRows;
        g.tok0 = sq.tok0;
        g.len = sq.len;
        const int n0 = min(kRows, sq.len - g.q0), n1 = max(0, min(kRows, sq.len - g.q0 - kRows));
        const int all = (sq.len + N - 1) / N;
        const int tiles0 = CAUSAL ? (g.q0 + n0 + N - 1) / N : all;
        const int tiles1 = n1 == 0 ? 0 : CAUSAL ? (g.q0 + kRows + n1 + N - 1) / N : all;
        const int units = tiles0 + tiles1;
        const int u0 = (int)(rest - item0), u1 = (int)min((int64_t)units, u0 + left);
        left -= u1 - u0;
        // units of the lower block before unit u: it has every other one, until its tiles end
        auto lower = [&](int u) { return n1 == 0 ? u : (min(u, 2 * tiles0) + 1) >> 1; };
        g.a0 = lower(u0);
        g.b0 = lower(u1);
        g.a1 = u0 - g.a0;
        g.b1 = u1 - g.b0;
        // to the next item: the next 256 queries, the next head, the next sequence
        ++q;
        item0 += units;
        rest = item0;
        if (q * 2 * kRows >= sq.len) {
            q = 0;
            item0 = rest = 0;
            if (++h == L.heads) {
                h = 0;
                ++b;
                if (left > 0) sq = sequence(L, b);
            }
        }
        return true;
    }
};

// The loading and the MMA warp run their loops with all lanes together, every
// value the same in each, and one elected lane issues. Issued from inside a
// one-lane branch, with the work between two products spread over branches, the
// same products took 70 us in place of 48.

// 4-D tiled load global -> shared, completing on `bar`, after announcing its bytes there.
__device__ __forceinline__ void load_4d(uint32_t smem_dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                        int c3) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];\n\t}" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}

// D[tmem] (+)= A * B, as tc_mma_f16, issued by one lane of a converged warp.
template <bool ACC>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Each thread of the warp reads 32 consecutive fp32 columns of its TMEM lane;
// tmem_wait_ld before the first use.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));  // no use of r moves above the wait
}

// A NaN among the operands gives NaN: a NaN logit shows in the result.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <bool ABS>
__device__ __forceinline__ void reduce32(const uint32_t (&r)[32], float (&m)[4]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float a = __uint_as_float(r[i]), b = __uint_as_float(r[i + 1]);
        if (ABS) {
            a = fabsf(a);
            b = fabsf(b);
        }
        m[(i >> 1) & 3] = max3_nan(m[(i >> 1) & 3], a, b);
    }
}

// The same over the first `n` columns only (n may be <= 0).
template <bool ABS>
__device__ __forceinline__ void reduce32_masked(const uint32_t (&r)[32], int n, float (&m)[4]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float a = __uint_as_float(r[i]);
        if (ABS) a = fabsf(a);
        m[i & 3] = max_nan(m[i & 3], i < n ? a : -INFINITY);
    }
}

// Floats in order as the bits that the integer maximum and minimum order;
// works from an initial -infinity. A NaN (0x7fffffff) is above everything.
// Where the caller's values are there (`given`), a NaN among them may have its
// sign set and be below everything: the first to come, whichever that is, still
// finds it and puts the other one in its place, and so does everyone after.
__device__ __forceinline__ void atomic_max_float(float* p, float v, bool given) {
    v += 0.f;  // -0 to +0
    if (given && isnan(__ldcg(p))) v = __int_as_float(0x7fffffff);
    if (v < 0.f) atomicMin(reinterpret_cast<unsigned*>(p), __float_as_uint(v));
    else atomicMax(reinterpret_cast<int*>(p), (int)(isnan(v) ? 0x7fffffffu : __float_as_uint(v)));
}

template <int N, bool CAUSAL>
__device__ __forceinline__ int64_t units_of_seq(const QkLaunch& L, int b) {
    return (int64_t)L.heads * units_of_head<N, CAUSAL>(sequence(L, b).len);
}

// This CTA's share of the units: begin, end, and the sequence it begins in.
// Packed batches: thread t adds up a contiguous part of the sequences.
template <int N, bool CAUSAL>
__device__ void find_share(const QkLaunch& L, QkCtl* ctl, int64_t* sums) {
    if (!L.offsets) {
        if (threadIdx.x == 0) {
            const int64_t per_seq = units_of_seq<N, CAUSAL>(L, 0), total = per_seq * L.seqs;
            ctl->units_begin = total * blockIdx.x / gridDim.x;
            ctl->units_end = total * (blockIdx.x + 1) / gridDim.x;
            ctl->b0 = (int)(ctl->units_begin / per_seq);
            ctl->rest0 = ctl->units_begin % per_seq;
        }
        __syncthreads();
        return;
    }
    const int per = (L.seqs + kThreads - 1) / kThreads;
    const int b0 = min(L.seqs, (int)threadIdx.x * per), b1 = min(L.seqs, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += units_of_seq<N, CAUSAL>(L, b);
    int64_t upto = mine;  // of this warp's threads up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)(threadIdx.x & 31) >= o) upto += v;
    }
    if ((threadIdx.x & 31) == 31) sums[threadIdx.x >> 5] = upto;
    __syncthreads();
    int64_t before = upto - mine;
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (int)(threadIdx.x >> 5)) before += sums[w];
        total += sums[w];
    }
    const int64_t begin = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
    if (threadIdx.x == 0) {
        ctl->units_begin = begin;
        ctl->units_end = end;
        ctl->b0 = 0;
        ctl->rest0 = 0;
    }
    __syncthreads();
    if (begin < end && before <= begin && begin < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const int64_t u = units_of_seq<N, CAUSAL>(L, b);
            if (begin < before + u) {
                ctl->b0 = b;
                ctl->rest0 = begin - before;
                break;
            }
            before += u;
        }
    }
    __syncthreads();
}

template <int N, int CH, bool CAUSAL, bool ABS>
__global__ void __launch_bounds__(kThreads, 1) qk_max_kernel(const __grid_constant__ QkLaunch L) {
    griddep_launch_dependents();
    constexpr uint32_t kStage = N * kBK * 2;
    constexpr int NB = 512 / N / 2;  // accumulators per block of rows
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    constexpr int nst = stages(N, CH), NQ = q_buffers(CH);
    uint8_t* qbuf = smem;  // [buffer][chunk]
    uint8_t* ring = qbuf + NQ * CH * kQChunk;
    QkCtl* ctl = reinterpret_cast<QkCtl*>(ring + nst * kStage);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Waits W{&ctl->abort_flag, L.wait_limit_ns, L.status};

    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int s = 0; s < NQ; ++s) {
            mbar_init(&ctl->q_full[s], 1);
            mbar_init(&ctl->q_empty[s], 1);
        }
        for (int a = 0; a < 2 * NB; ++a) {
            mbar_init(&ctl->acc_full[a], 1);
            mbar_init(&ctl->acc_empty[a], 4);  // the four warps of a block of rows
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&L.mq);
        prefetch_tensormap(&L.mk);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    griddep_wait();
    find_share<N, CAUSAL>(L, ctl, reinterpret_cast<int64_t*>(qbuf));  // qbuf is free until the first load
    fence_proxy_async_smem();
    __syncthreads();

    // shared-memory addresses: the same expressions in every lane
    const uint32_t q_base = smem_u32(qbuf), ring_base = smem_u32(ring);
    const uint32_t full_bar = smem_u32(&ctl->full[0]), empty_bar = smem_u32(&ctl->empty[0]);
    const uint32_t q_full_bar = smem_u32(&ctl->q_full[0]), q_empty_bar = smem_u32(&ctl->q_empty[0]);
    const uint32_t acc_full_bar = smem_u32(&ctl->acc_full[0]), acc_empty_bar = smem_u32(&ctl->acc_empty[0]);
    if (warp == 0) {
        int stage = 0, uses = 0, loads = 0;  // loads: blocks of queries so far, each into the next buffer
        uint32_t phase = 0;
        bool ok = true;
        Walk<N, CAUSAL> walk(L, ctl);
        Segment g;
        while (ok && walk.next(g)) {
            g.make_uniform();
            const int kvh = g.h / (L.heads / L.kv);
            auto load_q = [&](int s) {
                const int n = loads / NQ, at = loads - n * NQ;
                if (!wait(q_empty_bar + 8 * at, (n & 1u) ^ 1u, W)) return false;
                ++loads;
                expect_bytes(q_full_bar + 8 * at, CH * kQChunk);
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    load_4d(q_base + (at * CH + c) * kQChunk, &L.mq, q_full_bar + 8 * at, c * kBK,
                            g.tok0 + g.q0 + s * kRows, g.h, g.b);
                return true;
            };
            const int end = g.last();
            for (int j = g.first(); j < end && ok; ++j) {
                // in the order the MMAs take them: lower queries, keys, upper queries
                const bool in0 = g.in0(j), q1 = g.in1(j) && j == g.a1;
                if (in0 && j == g.a0) ok = load_q(0);
                if (ok && !in0 && q1) ok = load_q(1);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (!ok || !(ok = wait(empty_bar + 8 * stage, phase ^ 1u, W))) break;
                    expect_bytes(full_bar + 8 * stage, kStage);
                    load_4d(ring_base + stage * kStage, &L.mk, full_bar + 8 * stage, c * kBK, g.tok0 + j * N, kvh, g.b);
                    ++uses;
                    if (++stage == nst) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok && in0 && q1) ok = load_q(1);
            }
        }
        // every copy of this CTA has landed before it exits (an abort leaves some unread)
        for (int s = 0; s < nst; ++s) {
            const int n = uses / nst + (s < uses % nst ? 1 : 0);  // uses of stage s
            if (n > 0) wait_on(full_bar + 8 * s, (n - 1) & 1u, W, kDrainNs, true);
        }
        for (int s = 0; s < NQ; ++s) {
            const int n = loads / NQ + (s < loads % NQ ? 1 : 0);
            if (n > 0) wait_on(q_full_bar + 8 * s, (n - 1) & 1u, W, kDrainNs, true);
        }
    } else if (warp == 1) {
        // The MMA queue is a few products deep: what this warp does between the products of one block of rows
        // and the next has to fit in the time of about three of them.
        constexpr uint32_t IDESC = idesc_bf16_f32(kRows, N, 0);
        const uint64_t desc = smem_desc_sw128(0, 16, 1024);  // plus an address in 16-byte units
        const uint64_t qd = desc + (q_base >> 4);
        int stage = 0, loads = 0, acc0 = 0, acc1 = 0;  // blocks of queries so far; uses of each block's accumulators
        int q0 = 0, q1 = 0;                            // the buffers that hold them
        uint32_t phase = 0;
        bool ok = true;
        Walk<N, CAUSAL> walk(L, ctl);
        Segment g;
        // the products of block S with the key tile at the ring's stage; `first`: its copies are waited for,
        // `last`: its stages are released
        auto block = [&](auto which, int& uses, int& at, bool fresh, bool first, bool last, bool done) {
            constexpr int S = decltype(which)::value;
            const int a = S * NB + (NB == 1 ? 0 : uses & (NB - 1));
            if (!wait(acc_empty_bar + 8 * a, ((uses / NB) & 1u) ^ 1u, W)) return false;
            ++uses;
            if (fresh) {
                const int n = loads / NQ;
                at = loads - n * NQ;
                if (!wait(q_full_bar + 8 * at, n & 1u, W)) return false;
                ++loads;
            }
            const uint64_t q = qd + ((uint32_t)(at * CH * kQChunk) >> 4);
            const uint32_t d = tmem + (uint32_t)(a * N);
            int st = stage;
            uint32_t ph = phase;
            if (!first) tc_fence_after();
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (first) {
                    if (!wait(full_bar + 8 * st, ph, W)) return false;
                    tc_fence_after();
                }
                const uint64_t ad = q + ((c * kQChunk) >> 4), bd = desc + ((ring_base + st * kStage) >> 4);
                if (c == 0) mma_f16<false>(d, ad, bd, IDESC);
                else mma_f16<true>(d, ad, bd, IDESC);
#pragma unroll
                for (int kk = 1; kk < kBK / 16; ++kk) mma_f16<true>(d, ad + 2 * kk, bd + 2 * kk, IDESC);
                if (last) commit(empty_bar + 8 * st);
                if (++st == nst) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (last) {
                stage = st;
                phase = ph;
            }
            commit(acc_full_bar + 8 * a);
            if (done) commit(q_empty_bar + 8 * at);
            return true;
        };
        while (ok && walk.next(g)) {
            g.make_uniform();
            const int end = g.last();
            for (int j = g.first(); j < end && ok; ++j) {
                const bool in0 = g.in0(j), in1 = g.in1(j);
                if (in0)
                    ok = block(std::integral_constant<int, 0>{}, acc0, q0, j == g.a0, true, !in1, j + 1 == g.b0);
                if (ok && in1)
                    ok = block(std::integral_constant<int, 1>{}, acc1, q1, j == g.a1, !in0, true, j + 1 == g.b1);
            }
        }
        commit(smem_u32(&ctl->drain));  // every MMA has read its operands before this CTA exits
        wait_on(smem_u32(&ctl->drain), 0, W, kDrainNs, true);
    } else {
        const int quad = warp & 3, s = (warp - 2) >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        int uses = 0;
        bool ok = true;
        Walk<N, CAUSAL> walk(L, ctl);
        Segment g;
        while (ok && walk.next(g)) {
            const int i = g.q0 + s * kRows + quad * 32 + lane;  // this thread's query
            const int lim = i >= g.len ? -1 : CAUSAL ? i : g.len - 1;  // its last visible key
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const int j0 = s ? g.a1 : g.a0, j1 = s ? g.b1 : g.b0;
            for (int j = j0; j < j1; ++j) {
                const int a = s * NB + (NB == 1 ? 0 : uses & (NB - 1));
                if (!(ok = wait(acc_full_bar + 8 * a, (uses / NB) & 1u, W))) break;
                tc_fence_after();
                const uint32_t t0 = lane_base + (uint32_t)(a * N);
                const int n = lim - j * N + 1;  // columns of this tile the query sees
                uint32_t r0[32], r1[32];
                if (__all_sync(0xffffffffu, n >= N)) {
                    tmem_ld32_async(t0, r0);
                    tmem_wait_ld(r0);
#pragma unroll
                    for (int c = 0; c < N / 32; c += 2) {
                        tmem_ld32_async(t0 + (c + 1) * 32, r1);
                        reduce32<ABS>(r0, m);
                        tmem_wait_ld(r1);
                        if (c + 2 < N / 32) tmem_ld32_async(t0 + (c + 2) * 32, r0);
                        reduce32<ABS>(r1, m);
                        if (c + 2 < N / 32) tmem_wait_ld(r0);
                    }
                } else {
                    const int most = __reduce_max_sync(0xffffffffu, n);
                    for (int c = 0; c * 32 < min(most, N); ++c) {
                        tmem_ld32_async(t0 + c * 32, r0);
                        tmem_wait_ld(r0);
                        reduce32_masked<ABS>(r0, n - c * 32, m);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->acc_empty[a]);
                ++uses;
            }
            if (!ok || j0 >= j1) continue;
            float v = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
            if (lane == 0 && v != -INFINITY) atomic_max_float(&L.out[g.h], v * L.scale, L.given);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

__global__ void __launch_bounds__(256) qk_init_kernel(float* out, int heads) {
    griddep_launch_dependents();
    griddep_wait();
    const int h = blockIdx.x * 256 + threadIdx.x;
    if (h < heads) out[h] = -INFINITY;
}

// ------------------------------------------------------------------ weights

constexpr int kScaleThreads = 256;
constexpr int64_t kScaleChunk = 8192;  // floats per piece of a head's rows
constexpr int kMaxHeads = 2048;        // query and key heads together

struct QkScale {
    float *wq, *wk;
    const float* top;  // largest logit per query head
    int64_t nq, nk;    // weights per query head, per key head
    int32_t heads, kv, vec;
    float tau, alpha;
    int* status;
};

// g = min(1, tau / S), at least the smallest normal number (a quotient that underflowed to 0 would make 0 / 0 of a
// shared key head's factors); a maximum that is not finite leaves the weights alone
__device__ __forceinline__ float gamma_of(float s, float tau) {
    return s > tau && s < INFINITY ? fmaxf(tau / s, FLT_MIN) : 1.f;
}
__device__ __forceinline__ float share(float g, float e) { return g == 1.f ? 1.f : e == 0.5f ? sqrtf(g) : powf(g, e); }

// Every block lists the heads whose factor is not 1, then takes its share of
// their pieces. A head within the threshold costs nothing.
__global__ void __launch_bounds__(kScaleThreads, 4) qk_scale_kernel(const __grid_constant__ QkScale A) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float factor[kMaxHeads];
    __shared__ int16_t list[kMaxHeads];
    __shared__ int count[2];
    const int group = A.heads / A.kv;
    for (int h = threadIdx.x; h < A.heads; h += kScaleThreads) factor[h] = gamma_of(A.top[h], A.tau);
    __syncthreads();
    for (int c = threadIdx.x; c < A.kv; c += kScaleThreads) {
        float least = 1.f;
        for (int k = 0; k < group; ++k) least = fminf(least, factor[c * group + k]);
        const float fk = share(least, 1.f - A.alpha);
        factor[A.heads + c] = fk;
        for (int k = 0; k < group; ++k) {
            const float g = factor[c * group + k];
            // without shared heads this is g^alpha; formed as the quotient so that the two factors multiply to g
            factor[c * group + k] = group == 1 ? share(g, A.alpha) : g / fk;
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0;
        for (int part = 0; part < 2; ++part) {  // query heads first, then key heads
            const int h0 = part ? A.heads : 0, h1 = part ? A.heads + A.kv : A.heads;
            for (int h = h0 + (int)threadIdx.x; h - (int)threadIdx.x < h1; h += 32) {
                const bool on = h < h1 && factor[h] != 1.f;
                const uint32_t b = __ballot_sync(0xffffffffu, on);
                if (on) list[n + __popc(b & ((1u << threadIdx.x) - 1))] = (int16_t)h;
                n += __popc(b);
            }
            if (threadIdx.x == 0) count[part] = n;
        }
    }
    __syncthreads();
    const int64_t pq = (A.nq + kScaleChunk - 1) / kScaleChunk, pk = (A.nk + kScaleChunk - 1) / kScaleChunk;
    const int64_t nq = count[0] * pq, all = nq + (count[1] - count[0]) * pk;
    for (int64_t p = blockIdx.x; p < all; p += gridDim.x) {
        const bool isq = p < nq;
        const int64_t per = isq ? pq : pk, o = isq ? p : p - nq, n = isq ? A.nq : A.nk;
        const int h = list[(isq ? 0 : count[0]) + o / per];
        const int64_t i0 = o % per * kScaleChunk, i1 = min(n, i0 + kScaleChunk);
        float* w = isq ? A.wq + h * A.nq : A.wk + (h - A.heads) * A.nk;
        [[maybe_unused]] const int64_t at = isq ? h * A.nq : (h - A.heads) * A.nk;
        [[maybe_unused]] const int64_t end = isq ? A.heads * A.nq : A.kv * A.nk;
        const float f = factor[h];
        if (A.vec) {
            constexpr int U = kScaleChunk / (4 * kScaleThreads);  // every load of the piece before the first store
            float4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + 4 * (threadIdx.x + u * kScaleThreads);
                if (i < i1 && MA_INB(at + i, 4, end, A.status)) x[u] = __ldcs(reinterpret_cast<const float4*>(w + i));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + 4 * (threadIdx.x + u * kScaleThreads);
                if (i < i1 && MA_INB(at + i, 4, end, A.status))
                    __stcs(reinterpret_cast<float4*>(w + i), make_float4(x[u].x * f, x[u].y * f, x[u].z * f, x[u].w * f));
            }
        } else {
            for (int64_t i = i0 + threadIdx.x; i < i1; i += kScaleThreads)
                if (MA_INB(at + i, 1, end, A.status)) w[i] *= f;
        }
    }
}

// ------------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(ptr);
        return nullptr;
    }();
    return fn;
}

bool make_map(CUtensorMap* map, const void* base, int64_t dim, int64_t tokens, int64_t heads, int64_t seqs, int64_t st,
              int64_t sh, int64_t sb, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)tokens, (cuuint64_t)heads, (cuuint64_t)seqs};
    const cuuint64_t strides[3] = {(cuuint64_t)st * 2, (cuuint64_t)sh * 2, (cuuint64_t)sb * 2};
    const cuuint32_t box[4] = {kBK, (cuuint32_t)box_rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, int CH, bool CAUSAL, bool ABS>
cudaError_t launch_max(const QkLaunch& L, int grid, cudaStream_t s) {
    static_assert(stages(N, CH) >= CH, "a key tile has to fit in the ring");
    constexpr uint32_t smem = 1024 + q_buffers(CH) * CH * kQChunk + stages(N, CH) * N * kBK * 2 + kCtlBytes;
    static PerDevice<int> cache;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cache.get(dev, &done, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(qk_max_kernel<N, CH, CAUSAL, ABS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(qk_max_kernel<N, CH, CAUSAL, ABS>, dim3(grid), dim3(kThreads), smem, s, L);
}

template <int N, int CH>
cudaError_t launch_max_ch(const QkLaunch& L, bool causal, bool abs, int grid, cudaStream_t s) {
    if (causal) return abs ? launch_max<N, CH, true, true>(L, grid, s) : launch_max<N, CH, true, false>(L, grid, s);
    return abs ? launch_max<N, CH, false, true>(L, grid, s) : launch_max<N, CH, false, false>(L, grid, s);
}

// Keys per tile: 256, or 128 for head dimensions above 192, whose key tile of
// 256 would not fit beside the queries. (4096 causal tokens, 32 heads of 64: 35
// us, 45 with tiles of 128: the time between two products is per product.)
int tile_keys(int dim) { return dim > 192 ? 128 : 256; }

}  // namespace
}  // namespace ma

using namespace ma;

namespace {

int qk_max(int64_t seqs, int64_t len, int64_t total, int heads, int kv_heads, int dim, const uint16_t* q, int64_t q_seq,
           int64_t q_tok, int64_t q_head, const uint16_t* k, int64_t k_seq, int64_t k_tok, int64_t k_head,
           const int32_t* offsets, float scale, int causal, int absolute, int accumulate, float* out, void* stream) {
    if (seqs < 0 || len < 0 || total < 0 || heads < 1 || kv_heads < 1 || dim < 1 || heads % kv_heads != 0)
        return MA_ERR_SHAPE;
    if (dim > kMaxChunks * kBK || heads > 65535 || seqs > INT_MAX - 1 || len > (INT_MAX >> 1) || total > (INT_MAX >> 1))
        return MA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale)) return MA_ERR_ARG;
    if ((causal | absolute | accumulate) & ~1) return MA_ERR_ARG;
    if (!out) return MA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(out) % 4 != 0 || reinterpret_cast<uintptr_t>(offsets) % 4 != 0) return MA_ERR_ALIGN;
    const int64_t tokens = offsets ? total : len, outer = offsets ? 1 : seqs;
    const bool work = seqs > 0 && len > 0 && tokens > 0;
    int64_t st[6] = {q_tok, q_head, q_seq, k_tok, k_head, k_seq};
    if (work) {
        if (!q || !k) return MA_ERR_NULL;
        if (dim % 8 != 0 || reinterpret_cast<uintptr_t>(q) % 16 != 0 || reinterpret_cast<uintptr_t>(k) % 16 != 0)
            return MA_ERR_ALIGN;
        const int64_t ext[6] = {tokens, heads, outer, tokens, kv_heads, outer};
        for (int i = 0; i < 6; ++i) {
            if (ext[i] == 1) st[i] = dim;  // never followed
            if (st[i] < dim) return MA_ERR_SHAPE;
            if (st[i] % 8 != 0) return MA_ERR_ALIGN;
            if (st[i] >= (int64_t(1) << 38)) return MA_ERR_UNSUPPORTED;
        }
        // bytes from the first element of an input to its last (in floating point: strides times extents may be large)
        auto bytes = [&](int i) {
            double n = dim;
            for (int d = i; d < i + 3; ++d) n += (double)(ext[d] - 1) * (double)st[d];
            return 2.0 * n;
        };
        auto meets = [&](const void* p, double n) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(p), o = reinterpret_cast<uintptr_t>(out);
            return a < o + 4 * (uintptr_t)heads && (o < a || (double)(o - a) < n);
        };
        if (meets(q, bytes(0)) || meets(k, bytes(3)) || (offsets && meets(offsets, 4.0 * (double)(seqs + 1))))
            return MA_ERR_ARG;
    }
    const int n = tile_keys(dim);
    const int chunks = (dim + kBK - 1) / kBK;
    const int64_t m = (len + kRows - 1) / kRows;  // units of a (longest) sequence
    const int64_t units =
        (causal ? (n == 256 ? (m + 1) * (m + 1) / 4 : m * (m + 1) / 2) : m * ((len + n - 1) / n)) * heads;
    if ((double)units * (double)seqs > 0x1p54) return MA_ERR_UNSUPPORTED;  // the kernel multiplies it by its grid
    int sms = 0;
    if (const int rc = device_ready(&sms)) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    QkLaunch L;
    std::memset(&L, 0, sizeof(L));
    if (work) {
        if (!make_map(&L.mq, q, dim, tokens, heads, outer, st[0], st[1], st[2], kRows) ||
            !make_map(&L.mk, k, dim, tokens, kv_heads, outer, st[3], st[4], st[5], n))
            return MA_ERR_CUDA;
    }
    const int pr = prof_begin(MA_PROF_QK, s);
    cudaError_t e = cudaSuccess;
    if (!accumulate) e = launch_pdl(qk_init_kernel, dim3((heads + 255) / 256), dim3(256), 0, s, out, heads);
    double flops = 0.0;
    if (e == cudaSuccess && work) {
        L.offsets = offsets;
        L.seqs = (int)seqs;
        L.len = (int)len;
        L.total = (int)total;
        L.heads = heads;
        L.kv = kv_heads;
        L.given = accumulate;
        L.scale = scale;
        L.out = out;
        L.wait_limit_ns = host_wait_limit_ns();
        L.status = device_status_ptr();
        // a CTA per SM; fewer when there are fewer units (dense batches: the host knows)
        int grid = sms;
        if (!offsets) {
            grid = (int)std::min<int64_t>(sms, units * std::min<int64_t>(seqs, sms));
            flops = 2.0 * dim * heads * (double)seqs * (causal ? 0.5 * len * (len + 1.0) : (double)len * len);
        }
        e = chunks == 1   ? launch_max_ch<256, 1>(L, causal, absolute, grid, s)
            : chunks == 2 ? launch_max_ch<256, 2>(L, causal, absolute, grid, s)
            : chunks == 3 ? launch_max_ch<256, 3>(L, causal, absolute, grid, s)
                          : launch_max_ch<128, 4>(L, causal, absolute, grid, s);
    }
    prof_end(pr, s, flops, 0.0);
    return e == cudaSuccess ? MA_OK : MA_ERR_CUDA;
}

}  // namespace

extern "C" {

int ma_qk_max_logit(int64_t seqs, int64_t len, int64_t total, int heads, int kv_heads, int dim, const uint16_t* q,
                    int64_t q_seq, int64_t q_tok, int64_t q_head, const uint16_t* k, int64_t k_seq, int64_t k_tok,
                    int64_t k_head, const int32_t* offsets, float scale, int causal, int absolute, int accumulate,
                    float* out, void* stream) {
    return qk_max(seqs, len, total, heads, kv_heads, dim, q, q_seq, q_tok, q_head, k, k_seq, k_tok, k_head, offsets,
                  scale, causal, absolute, accumulate, out, stream);
}

int ma_qk_clip(int heads, int kv_heads, int64_t q_rows, int64_t k_rows, int64_t cols, float* wq, float* wk,
               const float* max_logit, float tau, float alpha, void* stream) {
    if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || q_rows < 0 || k_rows < 0 || cols < 0) return MA_ERR_SHAPE;
    if ((int64_t)heads + kv_heads > kMaxHeads || q_rows > (int64_t(1) << 30) || k_rows > (int64_t(1) << 30) ||
        cols > (int64_t(1) << 30))
        return MA_ERR_UNSUPPORTED;
    if (!(tau > 0.f) || !std::isfinite(tau) || !(alpha >= 0.f && alpha <= 1.f)) return MA_ERR_ARG;
    if (!max_logit) return MA_ERR_NULL;
    QkScale A;
    std::memset(&A, 0, sizeof(A));
    if (cols > 0 && std::max(q_rows, k_rows) > (int64_t(1) << 40) / cols) return MA_ERR_UNSUPPORTED;
    A.nq = q_rows * cols;
    A.nk = k_rows * cols;
    if ((A.nq > 0 && !wq) || (A.nk > 0 && !wk)) return MA_ERR_NULL;
    const uintptr_t a = reinterpret_cast<uintptr_t>(wq), b = reinterpret_cast<uintptr_t>(wk),
                    c = reinterpret_cast<uintptr_t>(max_logit);
    if (a % 4 != 0 || b % 4 != 0 || c % 4 != 0) return MA_ERR_ALIGN;
    const uintptr_t ab = (uintptr_t)A.nq * heads * 4, bb = (uintptr_t)A.nk * kv_heads * 4, cb = (uintptr_t)heads * 4;
    auto meet = [](uintptr_t x, uintptr_t xb, uintptr_t y, uintptr_t yb) { return xb && yb && x < y + yb && y < x + xb; };
    if (meet(a, ab, b, bb) || meet(a, ab, c, cb) || meet(b, bb, c, cb)) return MA_ERR_ARG;
    int sms = 0, st;
    if ((st = device_ready(&sms))) return st;
    if (A.nq == 0 && A.nk == 0) return MA_OK;
    A.wq = wq;
    A.wk = wk;
    A.top = max_logit;
    A.heads = heads;
    A.kv = kv_heads;
    A.vec = a % 16 == 0 && b % 16 == 0 && A.nq % 4 == 0 && A.nk % 4 == 0;
    A.tau = tau;
    A.alpha = alpha;
    A.status = device_status_ptr();
    const int64_t pieces = heads * ((A.nq + kScaleChunk - 1) / kScaleChunk) + kv_heads * ((A.nk + kScaleChunk - 1) / kScaleChunk);
    const int grid = (int)std::min<int64_t>(pieces, 4 * (int64_t)sms);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int pr = prof_begin(MA_PROF_QK, s);
    const cudaError_t e = launch_pdl(qk_scale_kernel, dim3(grid), dim3(kScaleThreads), 0, s, A);
    prof_end(pr, s, 0.0, 0.0);
    return e == cudaSuccess ? MA_OK : MA_ERR_CUDA;
}

}  // extern "C"
