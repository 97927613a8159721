// Global gradient norm over many tensors, and clipping by it.
//
//   N = scale * sqrt(sum over every tensor of g^2)
//   coef = scale * min(1, max_norm / N)          g <- coef * g (in place), or the
//                                                AdamW and momentum passes take
//                                                coef * g as they read g
// A sum of squares that is not finite gives coef = 0, and a gradient times a
// zero coef is taken as zero, whatever it holds: no NaN or infinity reaches a
// parameter. (The sum is fp64: finite gradients whose norm is beyond fp32 are
// clipped like others, though the norm, a float, reads infinite.)
//
// Bound by HBM: the norm reads every gradient once; clipping in place reads and
// writes each once more. One launch covers up to kClipMaxTensors tensors; the
// table travels in the parameter block.
//  * Norm: two blocks per SM walk chunks of 32 KB, grid-stride. Each thread
//    copies its eight 16-byte words of a chunk into its own slots of shared
//    memory (cp.async), two chunks ahead of the one it sums, with no barrier,
//    since no thread reads another's slots: 128 to 192 KB are in flight per SM
//    throughout. 6.6 TB/s on 13.5 GB of bf16 gradients (four blocks with plain
//    loads: 4.83; three blocks with one chunk less ahead: 4.09).
//  * Scaling in place: one block per chunk with plain streaming loads and
//    stores, 64 registers, from the last chunk to the first, so that it begins
//    with what the norm pass left in L2. Norm and scaling of the 1.12 GB depth-20
//    set take 518 us, 167 of them the norm (the persistent ring for both: 567).
//  * Small sets, one launch in all (below): the 81 gains and scalars of the
//    depth-20 set take 5.1 us in place, with three launches 9.5.
//
// The squares are summed in fp32 over the 32 or 64 values a thread holds of one
// chunk (relative error at most 64 * 2^-24 of a sum of positive terms, in
// practice a tenth of that), and from there on in fp64, in an order that depends
// only on the table and the GPU's SM count: the same inputs give the same bits.
// Where that fp32 sum overflows or is so small that squares were lost to
// underflow, the thread sums its values again in fp64.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <utility>
#include <vector>

#include "clip.cuh"
#include "common.cuh"
#include "internal.h"

namespace ma {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                              // 16-byte vectors per thread and chunk
constexpr int64_t kChunkVecs = kThreads * kVecs;      // 16-byte vectors per chunk (32 KB)
constexpr int kBlocksPerSm = 2;
constexpr int kAhead = 3;                             // chunks in flight per block
constexpr int kRingBytes = kAhead * kThreads * kVecs * 16;  // 96 KB
constexpr int kSmallTable = 96;                       // tensors of the small parameter block (2.4 KB)
constexpr int kMidTable = 640;                        // tensors of a small set's larger one (15 KB)

// A gradient: its first 16-byte word at or before the data, and how many
// leading elements of that word belong to something else, so that every
// 16-byte load is aligned whatever the tensor's offset.
struct GradDesc {
    uint64_t base_dt;  // address of the word, 16-byte aligned; bit 0: bf16
    int64_t numel;
    int64_t chunk0_skip;  // first chunk of this tensor * 8 + leading elements to skip (0..7)
};

// Small sets (small_chunks() chunks of 2 KB) take one launch of one cluster: every warp sums its chunks, the
// cluster adds its blocks' sums through distributed shared memory, and clipping
// reads the chunks again, from L2. Latency is all there: one launch in place of
// two or three, few dependent loads, and little code to fetch.
constexpr int kSmallVecs = 4;                          // 16-byte words per lane and chunk
constexpr int64_t kSmallChunkVecs = 32 * kSmallVecs;   // words per chunk (2 KB), one warp's
constexpr int kSmallBlocks = 8;                        // blocks of the cluster
constexpr int kSmallThreads = 1024;
constexpr int kSmallWarps = kSmallBlocks * kSmallThreads / 32;
// A set whose table fits the 2.4 KB block is small while each warp has one
// chunk (512 KB: clipped in 5.2 us, by the streaming kernels in 7.4; at 1 MB 9.3
// against 7.4); one with more tensors, whose other way is the 31 KB table in
// three launches, up to four chunks a warp (600 tensors of 100 values: 8.9
// against 10.6 us; of 800 values: 10.4 against 10.6). Beyond kMidTable the table
// would need a third block of 31 KB, for less: 900 tensors of 100 values 11.0
// against 12.1 us, of 800 12.7 against 12.4.
constexpr int small_chunks(size_t tensors) {
    return tensors <= kSmallTable ? kSmallWarps : tensors <= kMidTable ? 4 * kSmallWarps : 0;
}

template <int CAP>
struct GradTable {
    int32_t n, nparts;
    int32_t accumulate;  // add to the partial sums of the launches before
    int32_t pad;
    int64_t nchunks;
    float scale, max_norm;
    ClipHead* head;
    double* partials;
    int* status;
    GradDesc t[CAP];
};

__device__ __forceinline__ int64_t chunk0_of(const GradDesc& d) { return d.chunk0_skip >> 3; }

// The table as ordinary memory: loads through this pointer are plain cached
// loads that lanes make side by side, where indexed accesses to the parameter
// block are served one address at a time, each a miss the first time.
template <int CAP>
__device__ __forceinline__ const GradDesc* table(const GradTable<CAP>& T) {
    const GradDesc* p = T.t;
    asm volatile("" : "+l"(p));
    return p;
}

__device__ __forceinline__ uint8_t* base_of(const GradDesc& d) {
    return reinterpret_cast<uint8_t*>(d.base_dt & ~uint64_t(1));
}

// The tensor of a chunk, found by the whole warp: 32 brackets, then the bracket.
__device__ __forceinline__ int search_tensor(const GradDesc* t, int n, int64_t chunk) {
    const int lane = threadIdx.x & 31, width = (n + 31) / 32;
    const int at = lane * width;
    const uint32_t low = __ballot_sync(0xffffffffu, at < n && chunk0_of(t[min(at, n - 1)]) <= chunk);
    const int lo = (31 - __clz(low)) * width;  // bit 0 is set: the first tensor begins at chunk 0
    int count = 0;
    for (int b = 0; b < width; b += 32) {
        const int i = lo + b + lane;
        count += __popc(__ballot_sync(0xffffffffu, b + lane < width && i < n && chunk0_of(t[min(i, n - 1)]) <= chunk));
    }
    return lo + count - 1;
}

// The tensor that a walk over chunks is in.
struct Cursor {
    int t = -1;
    int64_t begin = 0, end = 0;  // its chunks
    GradDesc d;
    __device__ __forceinline__ void seek(const GradDesc* tab, int n, int64_t nchunks, int64_t c) {
        if (c >= begin && c < end) return;  // as it mostly is for long tensors
        t = search_tensor(tab, n, c);
        d = tab[t];
        begin = chunk0_of(d);
        end = t + 1 < n ? chunk0_of(tab[t + 1]) : nchunks;
    }
};

// Values of a 16-byte word as floats: 8 bf16 or 4 fp32.
template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& w, float (&f)[BF16 ? 8 : 4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(u[i]);
            f[2 * i + 1] = bf16_hi(u[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(u[i]);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack(const float (&f)[BF16 ? 8 : 4]) {
    if constexpr (BF16)
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    else
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// The first or last word of a tensor, element by element: those outside the
// tensor read as zero and are not written. (Out of line: rare, and small sets
// are bound by the size of the code that a launch has to fetch.)
template <bool BF16>
__device__ __noinline__ uint4 load_edge(const uint8_t* word, int64_t e0, int64_t numel) {
    uint32_t u[4] = {0, 0, 0, 0};
    constexpr int E = BF16 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (e0 + i < 0 || e0 + i >= numel) continue;
        if constexpr (BF16)
            u[i >> 1] |= (uint32_t)(*reinterpret_cast<const uint16_t*>(word + 2 * i)) << (16 * (i & 1));
        else
            u[i] = *reinterpret_cast<const uint32_t*>(word + 4 * i);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <bool BF16>
__device__ __noinline__ void store_edge(uint8_t* word, int64_t e0, int64_t numel, uint4 w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    constexpr int E = BF16 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (e0 + i < 0 || e0 + i >= numel) continue;
        if constexpr (BF16)
            *reinterpret_cast<uint16_t*>(word + 2 * i) = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
        else
            *reinterpret_cast<uint32_t*>(word + 4 * i) = u[i];
    }
}

// Word v of a tensor (zero beyond its end).
template <bool BF16>
__device__ __forceinline__ uint4 load_word(const uint8_t* base, int64_t v, int skip, int64_t numel, int* status) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t e0 = v * E - skip;  // tensor index of the word's first element
    if (e0 >= numel) return make_uint4(0, 0, 0, 0);
    if (e0 < 0 || e0 + E > numel) return load_edge<BF16>(base + 16 * v, e0, numel);
    if (!MA_INB(e0, E, numel, status)) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4*>(base + 16 * v);
}

template <bool BF16>
__device__ __forceinline__ void store_word(uint8_t* base, int64_t v, int skip, int64_t numel, const uint4& w,
                                           int* status) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t e0 = v * E - skip;
    if (e0 >= numel) return;
    if (e0 < 0 || e0 + E > numel) return store_edge<BF16>(base + 16 * v, e0, numel, w);
    if (MA_INB(e0, E, numel, status)) *reinterpret_cast<uint4*>(base + 16 * v) = w;
}

// One chunk of one tensor, as a thread sees it: words threadIdx.x + 256 i.
struct Chunk {
    uint8_t* at;  // address of word threadIdx.x
    int64_t v;    // index of that word in its tensor
    int64_t numel;
    int skip;
    bool bf16, whole;  // whole: every word of the chunk lies inside the tensor
};

__device__ __forceinline__ Chunk chunk_at(const GradDesc& d, int64_t c) {
    Chunk k;
    const int64_t v0 = (c - chunk0_of(d)) * kChunkVecs;
    k.v = v0 + threadIdx.x;
    k.at = base_of(d) + 16 * k.v;
    k.numel = d.numel;
    k.skip = (int)(d.chunk0_skip & 7);
    k.bf16 = d.base_dt & 1;
    const int64_t e = k.bf16 ? 8 : 4, e0 = v0 * e - k.skip;
    k.whole = e0 >= 0 && e0 + kChunkVecs * e <= k.numel;
    return k;
}

// Start this thread's copies of a chunk into its slots of one part of the ring
// (ragged chunks are read with plain loads when their turn comes).
__device__ __forceinline__ void fetch(const Chunk& k, uint4* slots, int* status) {
    if (!k.whole) return;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (MA_INB((k.v + (int64_t)kThreads * i) * (k.bf16 ? 8 : 4) - k.skip, k.bf16 ? 8 : 4, k.numel, status))
            cp_async16(slots + i * kThreads + threadIdx.x, k.at + 16 * kThreads * i);
}

template <bool BF16>
__device__ __forceinline__ void take(const Chunk& k, const uint4* slots, uint4 (&w)[kVecs], int* status) {
    if (k.whole) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) w[i] = slots[i * kThreads + threadIdx.x];
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) w[i] = load_word<BF16>(k.at - 16 * k.v, k.v + (int64_t)kThreads * i, k.skip, k.numel, status);
    }
}

// body(chunk, its slots) for the chunks of this block, kAhead - 1 of them in
// flight meanwhile.
template <int CAP, typename F>
__device__ __forceinline__ void walk_chunks(const GradTable<CAP>& T, F body) {
    extern __shared__ uint4 ring[];
    const GradDesc* tab = table(T);
    const int nt = T.n;
    const int64_t n = T.nchunks, step = gridDim.x;
    int64_t ahead = blockIdx.x;
    int slot_ahead = 0, slot = 0;
    Cursor far, here;
    auto push = [&] {
        if (ahead < n) {
            far.seek(tab, nt, n, ahead);
            fetch(chunk_at(far.d, ahead), ring + slot_ahead * (kThreads * kVecs), T.status);
        }
        cp_async_commit();  // a group per chunk, empty or not, so that the counts line up
        ahead += step;
        slot_ahead = slot_ahead + 1 == kAhead ? 0 : slot_ahead + 1;
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) push();
    for (int64_t q = blockIdx.x; q < n; q += step) {
        push();
        cp_async_wait<kAhead - 1>();
        here.seek(tab, nt, n, q);
        body(chunk_at(here.d, q), ring + slot * (kThreads * kVecs));
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    cp_async_wait<0>();
}

template <bool BF16, int VECS>
__device__ __forceinline__ double sum_squares(const uint4 (&w)[VECS]) {
    constexpr int E = BF16 ? 8 : 4;
    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        float f[E];
        unpack<BF16>(w[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e) p[e & 3] = fmaf(f[e], f[e], p[e & 3]);
    }
    const float s = (p[0] + p[1]) + (p[2] + p[3]);
    // From 2^-100 up, what 64 squares lost to underflow (under 2^-149 each) is
    // below 2^-40 of the sum; an overflow shows as infinity (and a NaN fails both).
    if (s >= 0x1p-100f && s < INFINITY) return (double)s;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i) any |= w[i].x | w[i].y | w[i].z | w[i].w;
    const uint32_t sign = BF16 ? 0x80008000u : 0x80000000u;
    if ((any & ~sign) == 0) return 0.0;
    double d = 0.0;
    for (int i = 0; i < VECS; ++i) {
        float f[E];
        unpack<BF16>(w[i], f);
        for (int e = 0; e < E; ++e) d = fma((double)f[e], (double)f[e], d);
    }
    return d;
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum_all(double v, double* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) t += red[i];
    __syncthreads();
    return t;
}

template <bool BF16, int VECS>
__device__ __forceinline__ void scale_words(uint4 (&w)[VECS], float coef) {
    constexpr int E = BF16 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        float f[E];
        unpack<BF16>(w[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = clip_value(f[e], coef);
        w[i] = pack<BF16>(f);  // one rounding to bf16, of the fp32 product
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_sumsq_kernel(const __grid_constant__ GradTable<CAP> T) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ double red[kThreads / 32];
    double sum = 0.0;
    walk_chunks(T, [&](const Chunk& k, const uint4* slots) {
        uint4 w[kVecs];
        if (k.bf16) {
            take<true>(k, slots, w, T.status);
            sum += sum_squares<true>(w);
        } else {
            take<false>(k, slots, w, T.status);
            sum += sum_squares<false>(w);
        }
    });
    const double t = block_sum_all(sum, red);
    if (threadIdx.x == 0) T.partials[blockIdx.x] = T.accumulate ? T.partials[blockIdx.x] + t : t;
}

// sum of squares -> norm and coefficient
__device__ __forceinline__ ClipHead clip_head(double sumsq, float scale, float max_norm) {
    ClipHead h;
    const double root = sqrt(sumsq), norm = (double)scale * root;
    h.sumsq = sumsq;
    h.norm = (float)norm;
    h.coef = !isfinite(sumsq) ? 0.f : norm > (double)max_norm ? (float)((double)max_norm / root) : scale;
    return h;
}

__device__ __forceinline__ double sum_partials(const double* partials, int nparts, double* red) {
    double v = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kThreads) v += partials[i];
    return block_sum_all(v, red);
}

// norm and coef from the partial sums, or (nparts < 0) from head->sumsq.
__global__ void __launch_bounds__(kThreads) clip_finalize_kernel(const __grid_constant__ ClipFinalize F) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ double red[kThreads / 32];
    const double s = F.nparts < 0 ? F.head->sumsq : sum_partials(F.partials, F.nparts, red);
    if (threadIdx.x == 0) *F.head = clip_head(s, F.scale, F.max_norm);
}

// One block per chunk, the last chunk first: what the norm pass left in L2 is
// read before it is evicted.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) grad_scale_kernel(const __grid_constant__ GradTable<CAP> T) {
    griddep_launch_dependents();
    const GradDesc* tab = table(T);
    const int64_t c = T.nchunks - 1 - (int64_t)blockIdx.x;
    const Chunk k = chunk_at(tab[search_tensor(tab, T.n, c)], c);
    griddep_wait();
    const float coef = T.head->coef;
    if (coef == 1.f) return;
    auto scale = [&](auto bf) {
        constexpr bool BF16 = decltype(bf)::value;
        [[maybe_unused]] constexpr int E = BF16 ? 8 : 4;
        uint4 w[kVecs];
        if (k.whole) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                w[i] = make_uint4(0, 0, 0, 0);
                if (MA_INB((k.v + (int64_t)kThreads * i) * E - k.skip, E, k.numel, T.status))
                    w[i] = __ldcs(reinterpret_cast<const uint4*>(k.at + 16 * kThreads * i));
            }
            scale_words<BF16>(w, coef);
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (MA_INB((k.v + (int64_t)kThreads * i) * E - k.skip, E, k.numel, T.status))
                    __stcs(reinterpret_cast<uint4*>(k.at + 16 * kThreads * i), w[i]);
        } else {
            uint8_t* base = k.at - 16 * k.v;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) w[i] = load_word<BF16>(base, k.v + (int64_t)kThreads * i, k.skip, k.numel, T.status);
            scale_words<BF16>(w, coef);
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                store_word<BF16>(base, k.v + (int64_t)kThreads * i, k.skip, k.numel, w[i], T.status);
        }
    };
    if (k.bf16) scale(std::true_type{});
    else scale(std::false_type{});
}

// Once per device: allow the ring's shared memory.
template <int CAP>
cudaError_t clip_setup() {
    static PerDevice<int> cache;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cache.get(dev, &done, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(grad_sumsq_kernel<CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    });
}

template <int CAP, bool CLIP>
__global__ void __cluster_dims__(kSmallBlocks, 1, 1) __launch_bounds__(kSmallThreads)
    grad_small_kernel(const __grid_constant__ GradTable<CAP> T) {
    griddep_launch_dependents();
    static_assert(kSmallThreads == 1024, "one partial sum per lane of the first warp");
    __shared__ double red[kSmallThreads / 32];
    __shared__ double block_total;
    __shared__ float factor;
    const int lane = threadIdx.x & 31, rank = (int)cluster_ctarank();
    const int first = rank * (kSmallThreads / 32) + (threadIdx.x >> 5);
    const GradDesc* tab = table(T);
    auto find = [&](int64_t c) {
        if constexpr (CAP > kSmallTable) return tab[search_tensor(tab, T.n, c)];
        int count = 0;  // three loads a lane, side by side
#pragma unroll
        for (int b = 0; b < kSmallTable; b += 32)
            count += __popc(__ballot_sync(0xffffffffu, b + lane < T.n && chunk0_of(tab[b + lane]) <= c));
        return tab[count - 1];
    };
    // with(bf16) for the tensor's type
    auto typed = [](const GradDesc& d, auto with) {
        if (d.base_dt & 1) with(std::true_type{});
        else with(std::false_type{});
    };
    auto word = [&](const GradDesc& d, int64_t c) { return (c - chunk0_of(d)) * kSmallChunkVecs + lane; };
    uint4 w[kSmallVecs];
    auto load = [&](const GradDesc& d, int64_t c, auto bf) {
#pragma unroll
        for (int i = 0; i < kSmallVecs; ++i)
            w[i] = load_word<decltype(bf)::value>(base_of(d), word(d, c) + 32 * i, (int)(d.chunk0_skip & 7), d.numel,
                                                  T.status);
    };
    auto store_scaled = [&](const GradDesc& d, int64_t c, float coef, auto bf) {
        constexpr bool BF16 = decltype(bf)::value;
        scale_words<BF16>(w, coef);
#pragma unroll
        for (int i = 0; i < kSmallVecs; ++i)
            store_word<BF16>(base_of(d), word(d, c) + 32 * i, (int)(d.chunk0_skip & 7), d.numel, w[i], T.status);
    };
    // The chunks after the first 256 one by one; then the first of this warp, whose words stay in
    // registers. Its tensor is found before the wait: the table depends on no earlier kernel.
    GradDesc mine;
    if (first < T.nchunks) mine = find(first);
    griddep_wait();
    double sum = 0.0;
#pragma unroll 1
    for (int64_t c = first + kSmallWarps; c < T.nchunks; c += kSmallWarps) {
        const GradDesc d = find(c);
        typed(d, [&](auto bf) {
            load(d, c, bf);
            sum += sum_squares<decltype(bf)::value>(w);
        });
    }
    if (first < T.nchunks) typed(mine, [&](auto bf) {
        load(mine, first, bf);
        sum += sum_squares<decltype(bf)::value>(w);
    });
    auto add_lanes = [](double v, int lanes) {
        for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    sum = add_lanes(sum, 32);
    if (lane == 0) red[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        const double t = add_lanes(red[lane], 32);
        if (lane == 0) block_total = t;
    }
    cluster_sync_all();
    if (threadIdx.x < 32) {  // the same sum, in the same order, in every block
        double t = 0.0;
        if (lane < kSmallBlocks)
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(t) : "r"(mapa_shared(smem_u32(&block_total), lane)) : "memory");
        t = add_lanes(t, kSmallBlocks);
        if (lane == 0) {
            const ClipHead h = clip_head(t, T.scale, T.max_norm);
            if (rank == 0) *T.head = h;
            factor = h.coef;
        }
    }
    __syncthreads();
    // no block leaves while another may still read its sum
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const float coef = factor;
    if (CLIP && coef != 1.f && first < T.nchunks) {
        typed(mine, [&](auto bf) { store_scaled(mine, first, coef, bf); });
#pragma unroll 1
        for (int64_t c = first + kSmallWarps; c < T.nchunks; c += kSmallWarps) {
            const GradDesc d = find(c);
            typed(d, [&](auto bf) {
                load(d, c, bf);
                store_scaled(d, c, coef, bf);
            });
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

int64_t words_of(const GradItem& it) {
    const int esz = it.gdt == MA_BF16 ? 2 : 4;
    const int64_t skip = (int64_t)(reinterpret_cast<uintptr_t>(it.g) % 16) / esz;
    return ((it.numel + skip) * esz + 15) / 16;
}

int64_t chunks_of(const GradItem& it, int64_t chunk_vecs) { return (words_of(it) + chunk_vecs - 1) / chunk_vecs; }

// The table of items [first, first + count), in chunks of chunk_vecs words.
template <int CAP>
void fill_table(GradTable<CAP>& T, const std::vector<GradItem>& items, size_t first, size_t count, int64_t chunk_vecs,
                int nparts, bool accumulate, const ClipArgs& a) {
    T.n = (int)count;
    T.nparts = nparts;
    T.accumulate = accumulate ? 1 : 0;
    T.pad = 0;
    T.scale = a.scale;
    T.max_norm = a.max_norm;
    T.head = a.head();
    T.partials = a.partials();
    T.status = device_status_ptr();
    int64_t chunk = 0;
    for (size_t i = 0; i < count; ++i) {
        const GradItem& it = items[first + i];
        const uintptr_t p = reinterpret_cast<uintptr_t>(it.g);
        const int esz = it.gdt == MA_BF16 ? 2 : 4;
        T.t[i].base_dt = (uint64_t)(p / 16 * 16) | (it.gdt == MA_BF16 ? 1u : 0u);
        T.t[i].numel = it.numel;
        T.t[i].chunk0_skip = chunk * 8 + (int64_t)(p % 16) / esz;
        chunk += chunks_of(it, chunk_vecs);
    }
    T.nchunks = chunk;
}

template <int CAP>
cudaError_t launch_table(const std::vector<GradItem>& items, size_t first, size_t count, int nparts, bool accumulate,
                         bool in_place, const ClipArgs& a, cudaStream_t s) {
    static thread_local GradTable<CAP> T;
    fill_table(T, items, first, count, kChunkVecs, nparts, accumulate, a);
    const dim3 grid((unsigned)(in_place ? T.nchunks : nparts));
    const cudaError_t e = clip_setup<CAP>();
    if (e != cudaSuccess) return e;
    return in_place ? launch_pdl(grad_scale_kernel<CAP>, grid, dim3(kThreads), 0, s, T)
                    : launch_pdl(grad_sumsq_kernel<CAP>, grid, dim3(kThreads), kRingBytes, s, T);
}

template <int CAP>
cudaError_t launch_small(const std::vector<GradItem>& items, bool in_place, const ClipArgs& a, cudaStream_t s) {
    static thread_local GradTable<CAP> T;
    fill_table(T, items, 0, items.size(), kSmallChunkVecs, 0, false, a);
    return in_place ? launch_pdl(grad_small_kernel<CAP, true>, dim3(kSmallBlocks), dim3(kSmallThreads), 0, s, T)
                    : launch_pdl(grad_small_kernel<CAP, false>, dim3(kSmallBlocks), dim3(kSmallThreads), 0, s, T);
}

}  // namespace

template <int CAP>
bool is_small(const void* func) {
    return func == reinterpret_cast<const void*>(grad_small_kernel<CAP, false>);
}

size_t clip_patch_bytes(const void* func) {
    if (func == reinterpret_cast<const void*>(clip_finalize_kernel)) return sizeof(ClipFinalize);
    if (is_small<kSmallTable>(func)) return sizeof(GradTable<kSmallTable>);
    if (is_small<kMidTable>(func)) return sizeof(GradTable<kMidTable>);
    return 0;
}

void clip_patch(const void* func, void* arg, float scale, float max_norm) {
    auto set = [&](auto* p) {
        p->scale = scale;
        p->max_norm = max_norm;
    };
    if (is_small<kSmallTable>(func)) set(reinterpret_cast<GradTable<kSmallTable>*>(arg));
    else if (is_small<kMidTable>(func)) set(reinterpret_cast<GradTable<kMidTable>*>(arg));
    else set(reinterpret_cast<ClipFinalize*>(arg));
}

cudaError_t launch_clip_finalize(const ClipArgs& a, int nparts, cudaStream_t s) {
    ClipFinalize F;
    std::memset(&F, 0, sizeof(F));
    F.head = a.head();
    F.partials = a.partials();
    F.nparts = nparts;
    F.scale = a.scale;
    F.max_norm = a.max_norm;
    const int pr = prof_begin(MA_PROF_CLIP, s);
    const cudaError_t e = launch_pdl(clip_finalize_kernel, dim3(1), dim3(kThreads), 0, s, F);
    prof_end(pr, s, 0.0, 0.0);
    return e;
}

// The norm of items (numel > 0 each), and their scaling in place: one launch
// for a small set; else partial sums, norm and coefficient, and the scaling.
cudaError_t launch_grad_clip(const std::vector<GradItem>& items, const ClipArgs& args, int sms, bool in_place,
                             cudaStream_t s, int* launches) {
    ClipArgs a = args;
    a.max_blocks = std::min(kClipMaxParts, sms * kBlocksPerSm);
    if (items.empty()) {
        ++*launches;
        return launch_clip_finalize(a, 0, s);
    }
    if (items.size() <= kMidTable) {
        int64_t chunks = 0, bytes = 0;
        for (const GradItem& it : items) {
            chunks += chunks_of(it, kSmallChunkVecs);
            bytes += it.numel * (it.gdt == MA_BF16 ? 2 : 4);
        }
        if (chunks <= small_chunks(items.size())) {
            const int pr = prof_begin(MA_PROF_CLIP, s);
            const cudaError_t e = items.size() <= kSmallTable ? launch_small<kSmallTable>(items, in_place, a, s)
                                                              : launch_small<kMidTable>(items, in_place, a, s);
            prof_end(pr, s, 0.0, (double)bytes * (in_place ? 2 : 1));
            ++*launches;
            return e;
        }
    }
    // Tables of up to kSmallTable tensors travel in a 2.4 KB parameter block
    // and longer ones in 31 KB: copying the large block into the launch costs
    // the host and the front end more than a small norm itself.
    const size_t cap = items.size() <= kSmallTable ? kSmallTable : kClipMaxTensors;
    int64_t most = 1;
    for (size_t f = 0; f < items.size(); f += cap) {
        int64_t c = 0;
        for (size_t i = f; i < std::min(items.size(), f + cap); ++i) c += chunks_of(items[i], kChunkVecs);
        most = std::max(most, c);
    }
    const int nparts = (int)std::min<int64_t>(most, a.max_blocks);
    for (int pass = 0; pass < (in_place ? 2 : 1); ++pass) {
        if (pass == 1) {
            const cudaError_t e = launch_clip_finalize(a, nparts, s);
            if (e != cudaSuccess) return e;
            ++*launches;
        }
        for (size_t f = 0; f < items.size(); f += cap) {
            const size_t n = std::min(items.size() - f, cap);
            double bytes = 0.0;
            for (size_t i = f; i < f + n; ++i)
                bytes += (double)items[i].numel * (items[i].gdt == MA_BF16 ? 2 : 4) * (pass + 1);
            const int pr = prof_begin(MA_PROF_CLIP, s);
            const cudaError_t e = cap == kSmallTable
                                      ? launch_table<kSmallTable>(items, f, n, nparts, f > 0, pass == 1, a, s)
                                      : launch_table<kClipMaxTensors>(items, f, n, nparts, f > 0, pass == 1, a, s);
            prof_end(pr, s, 0.0, bytes);
            if (e != cudaSuccess) return e;
            ++*launches;
        }
    }
    if (in_place) return cudaSuccess;
    ++*launches;
    return launch_clip_finalize(a, nparts, s);
}

}  // namespace ma

using namespace ma;

namespace {

int check_clip_args(float scale, float max_norm, const void* clip) {
    if (!(scale > 0.f) || !std::isfinite(scale) || !(max_norm >= 0.f)) return MA_ERR_ARG;
    if (!clip) return MA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(clip) % 256 != 0) return MA_ERR_ALIGN;
    return MA_OK;
}

int grad_clip(int n, const void* const* G, const int32_t* gdt, const int64_t* numel, float scale, float max_norm,
              void* clip, bool in_place, void* stream) {
    if (n < 0) return MA_ERR_SHAPE;
    int st = check_clip_args(scale, max_norm, clip);
    if (st) return st;
    if (n > 0 && (!G || !gdt || !numel)) return MA_ERR_NULL;
    std::vector<GradItem> items;
    std::vector<std::pair<uintptr_t, uintptr_t>> w;
    items.reserve(n);
    w.reserve(in_place ? n + 1 : 1);
    const uintptr_t c0 = reinterpret_cast<uintptr_t>(clip), c1 = c0 + MA_CLIP_BYTES;
    for (int i = 0; i < n; ++i) {
        if (gdt[i] != MA_F32 && gdt[i] != MA_BF16) return MA_ERR_DTYPE;
        const int esz = gdt[i] == MA_BF16 ? 2 : 4;
        if (numel[i] < 0 || numel[i] > (int64_t(1) << 50)) return MA_ERR_SHAPE;
        if (numel[i] == 0) continue;
        if (!G[i]) return MA_ERR_NULL;
        const uintptr_t p = reinterpret_cast<uintptr_t>(G[i]), e = p + (uintptr_t)numel[i] * esz;
        if (p % esz != 0) return MA_ERR_ALIGN;
        if (p < c1 && c0 < e) return MA_ERR_ARG;
        if (in_place) w.push_back({p, e});
        items.push_back({G[i], numel[i], gdt[i]});
    }
    if (in_place) {
        if (!std::is_sorted(w.begin(), w.end())) std::sort(w.begin(), w.end());
        for (size_t k = 1; k < w.size(); ++k)
            if (w[k].first < w[k - 1].second) return MA_ERR_ARG;
    }
    int sms = 0, launches = 0;
    if ((st = device_ready(&sms))) return st;
    const ClipArgs a{clip, scale, max_norm, 0};
    return launch_grad_clip(items, a, sms, in_place, reinterpret_cast<cudaStream_t>(stream), &launches) == cudaSuccess
               ? MA_OK
               : MA_ERR_CUDA;
}

}  // namespace

extern "C" {

int ma_grad_norm(int n, const void* const* G, const int32_t* gdt, const int64_t* numel, float scale, float max_norm,
                 void* clip, void* stream) {
    return ma_guard([&] { return grad_clip(n, G, gdt, numel, scale, max_norm, clip, false, stream); });
}

int ma_grad_clip(int n, void* const* G, const int32_t* gdt, const int64_t* numel, float scale, float max_norm,
                 void* clip, void* stream) {
    return ma_guard(
        [&] { return grad_clip(n, const_cast<const void* const*>(G), gdt, numel, scale, max_norm, clip, true, stream); });
}

int ma_clip_finalize(float scale, float max_norm, void* clip, void* stream) {
    int st = check_clip_args(scale, max_norm, clip);
    if (st) return st;
    if ((st = device_ready(nullptr))) return st;
    const ClipArgs a{clip, scale, max_norm, 0};
    return launch_clip_finalize(a, -1, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MA_OK : MA_ERR_CUDA;
}

}  // extern "C"
