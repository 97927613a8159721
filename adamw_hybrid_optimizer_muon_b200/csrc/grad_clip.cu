// Global gradient norm over many tensors, and clipping by it.
//
//   N = scale * sqrt(sum over every tensor of g^2)
//   coef = scale * min(1, max_norm / N)          g <- coef * g (in place), or the
//                                                AdamW and momentum passes take
//                                                coef * g as they read g
// A norm that is not finite gives coef = 0, and a gradient times a zero coef is
// taken as zero, whatever it holds: no NaN or infinity reaches a parameter.
//
// Bound by HBM: the norm reads every gradient once; clipping in place reads and
// writes each once more. One launch covers up to kClipMaxTensors tensors: the
// table travels in the parameter block, and each block walks chunks of 32 KB
// (eight 16-byte loads a thread, all in flight before the arithmetic). Clipping
// walks the chunks from the last to the first, so that it begins with what the
// norm pass left in L2.
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
constexpr int kBlocksPerSm = 4;
constexpr int kSmallTable = 96;                       // tensors of the small parameter block (2.4 KB)

// A gradient: its first 16-byte word at or before the data, and how many
// leading elements of that word belong to something else, so that every
// 16-byte load is aligned whatever the tensor's offset.
struct GradDesc {
    uint64_t base_dt;  // address of the word, 16-byte aligned; bit 0: bf16
    int64_t numel;
    int64_t chunk0_skip;  // first chunk of this tensor * 8 + leading elements to skip (0..7)
};

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

template <int CAP>
__device__ __forceinline__ int find_tensor(const GradTable<CAP>& T, int64_t chunk) {
    int lo = 0, hi = T.n - 1;
    while (lo < hi) {  // last tensor whose first chunk is <= this chunk
        const int mid = (lo + hi + 1) >> 1;
        if (chunk0_of(T.t[mid]) <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

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

// A word of a tensor that has elements of it in words [first partial .. last
// partial]: the elements outside the tensor read as zero.
template <bool BF16>
__device__ __forceinline__ uint4 load_word(const uint8_t* base, int64_t v, int skip, int64_t numel, int* status) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t e0 = v * E - skip;  // tensor index of the word's first element
    if (e0 >= 0 && e0 + E <= numel) {
        if (!MA_INB(e0, E, numel, status)) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4*>(base + 16 * v);
    }
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (e0 + i < 0 || e0 + i >= numel) continue;
        if constexpr (BF16)
            u[i >> 1] |= (uint32_t)(*reinterpret_cast<const uint16_t*>(base + 16 * v + 2 * i)) << (16 * (i & 1));
        else
            u[i] = *reinterpret_cast<const uint32_t*>(base + 16 * v + 4 * i);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <bool BF16>
__device__ __forceinline__ void store_word(uint8_t* base, int64_t v, int skip, int64_t numel, const uint4& w,
                                           int* status) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t e0 = v * E - skip;
    if (e0 >= 0 && e0 + E <= numel) {
        if (!MA_INB(e0, E, numel, status)) return;
        *reinterpret_cast<uint4*>(base + 16 * v) = w;
        return;
    }
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (e0 + i < 0 || e0 + i >= numel) continue;
        if constexpr (BF16)
            *reinterpret_cast<uint16_t*>(base + 16 * v + 2 * i) = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
        else
            *reinterpret_cast<uint32_t*>(base + 16 * v + 4 * i) = u[i];
    }
}

// The words of one chunk that this thread holds: word threadIdx.x + 256 i of it.
template <bool BF16>
__device__ __forceinline__ void load_chunk(const uint8_t* base, int64_t v0, int skip, int64_t numel, uint4 (&w)[kVecs],
                                           int* status) {
    constexpr int E = BF16 ? 8 : 4;
    if (v0 * E >= skip && (v0 + kChunkVecs) * E - skip <= numel && MA_INB(v0 * E - skip, kChunkVecs * E, numel, status)) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            w[i] = *reinterpret_cast<const uint4*>(base + 16 * (v0 + threadIdx.x + (int64_t)kThreads * i));
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            w[i] = load_word<BF16>(base, v0 + threadIdx.x + (int64_t)kThreads * i, skip, numel, status);
    }
}

template <bool BF16>
__device__ __forceinline__ double sum_squares(const uint4 (&w)[kVecs]) {
    constexpr int E = BF16 ? 8 : 4;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float f[E];
        unpack<BF16>(w[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(f[e], f[e], s);
    }
    // From 2^-100 up, what 64 squares lost to underflow (under 2^-149 each) is
    // below 2^-40 of the sum; an overflow shows as infinity (and a NaN fails both).
    if (s >= 0x1p-100f && s < INFINITY) return (double)s;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) any |= w[i].x | w[i].y | w[i].z | w[i].w;
    const uint32_t sign = BF16 ? 0x80008000u : 0x80000000u;
    if ((any & ~sign) == 0) return 0.0;
    double d = 0.0;
    for (int i = 0; i < kVecs; ++i) {
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

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_sumsq_kernel(const __grid_constant__ GradTable<CAP> T) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ double red[kThreads / 32];
    double sum = 0.0;
    for (int64_t c = blockIdx.x; c < T.nchunks; c += gridDim.x) {
        const GradDesc& d = T.t[find_tensor(T, c)];
        const uint8_t* base = reinterpret_cast<const uint8_t*>(d.base_dt & ~uint64_t(1));
        const int64_t v0 = (c - chunk0_of(d)) * kChunkVecs;
        const int skip = (int)(d.chunk0_skip & 7);
        uint4 w[kVecs];
        if (d.base_dt & 1) {
            load_chunk<true>(base, v0, skip, d.numel, w, T.status);
            sum += sum_squares<true>(w);
        } else {
            load_chunk<false>(base, v0, skip, d.numel, w, T.status);
            sum += sum_squares<false>(w);
        }
    }
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

// Every block forms the coefficient from the partial sums itself (the same
// bits in each), then scales its chunks.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_scale_kernel(const __grid_constant__ GradTable<CAP> T) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ double red[kThreads / 32];
    const ClipHead h = clip_head(sum_partials(T.partials, T.nparts, red), T.scale, T.max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) *T.head = h;
    if (h.coef == 1.f) return;
    const float coef = h.coef;
    for (int64_t q = blockIdx.x; q < T.nchunks; q += gridDim.x) {
        const int64_t c = T.nchunks - 1 - q;
        const GradDesc& d = T.t[find_tensor(T, c)];
        uint8_t* base = reinterpret_cast<uint8_t*>(d.base_dt & ~uint64_t(1));
        const int64_t v0 = (c - chunk0_of(d)) * kChunkVecs;
        const int skip = (int)(d.chunk0_skip & 7);
        uint4 w[kVecs];
        auto scale = [&](auto bf) {
            constexpr bool BF16 = decltype(bf)::value;
            constexpr int E = BF16 ? 8 : 4;
            load_chunk<BF16>(base, v0, skip, d.numel, w, T.status);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                float f[E];
                unpack<BF16>(w[i], f);
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = clip_value(f[e], coef);
                // one rounding to bf16, of the fp32 product
                store_word<BF16>(base, v0 + threadIdx.x + (int64_t)kThreads * i, skip, d.numel, pack<BF16>(f), T.status);
            }
        };
        if (d.base_dt & 1) scale(std::true_type{});
        else scale(std::false_type{});
    }
}

template <int CAP>
cudaError_t launch_table(const std::vector<GradItem>& items, size_t first, size_t count, int nparts, bool accumulate,
                         bool in_place, const ClipArgs& a, cudaStream_t s) {
    static thread_local GradTable<CAP> T;
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
        const int64_t skip = (int64_t)(p % 16) / esz;
        T.t[i].base_dt = (uint64_t)(p / 16 * 16) | (it.gdt == MA_BF16 ? 1u : 0u);
        T.t[i].numel = it.numel;
        T.t[i].chunk0_skip = chunk * 8 + skip;
        const int64_t vecs = ((it.numel + skip) * esz + 15) / 16;
        chunk += (vecs + kChunkVecs - 1) / kChunkVecs;
    }
    T.nchunks = chunk;
    const dim3 grid((unsigned)(in_place ? std::max<int64_t>(1, std::min<int64_t>(chunk, a.max_blocks)) : nparts));
    return in_place ? launch_pdl(grad_scale_kernel<CAP>, grid, dim3(kThreads), 0, s, T)
                    : launch_pdl(grad_sumsq_kernel<CAP>, grid, dim3(kThreads), 0, s, T);
}

int64_t chunks_of(const GradItem& it) {
    const int esz = it.gdt == MA_BF16 ? 2 : 4;
    const int64_t skip = (int64_t)(reinterpret_cast<uintptr_t>(it.g) % 16) / esz;
    return (((it.numel + skip) * esz + 15) / 16 + kChunkVecs - 1) / kChunkVecs;
}

}  // namespace

const void* clip_finalize_func() { return reinterpret_cast<const void*>(clip_finalize_kernel); }

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

// The norm pass over items (numel > 0 each): partial sums, then either the
// finalize (norm and coefficient) or the in-place scaling, which forms them itself.
cudaError_t launch_grad_clip(const std::vector<GradItem>& items, const ClipArgs& args, int sms, bool in_place,
                             cudaStream_t s, int* launches) {
    ClipArgs a = args;
    a.max_blocks = std::min(kClipMaxParts, sms * kBlocksPerSm);
    if (items.empty()) {
        ++*launches;
        return launch_clip_finalize(a, 0, s);
    }
    // Tables of up to kSmallTable tensors travel in a 2.4 KB parameter block
    // and longer ones in 31 KB: copying the large block into the launch costs
    // the host and the front end more than a small norm itself.
    const size_t cap = items.size() <= kSmallTable ? kSmallTable : kClipMaxTensors;
    int64_t most = 1;
    for (size_t f = 0; f < items.size(); f += cap) {
        int64_t c = 0;
        for (size_t i = f; i < std::min(items.size(), f + cap); ++i) c += chunks_of(items[i]);
        most = std::max(most, c);
    }
    const int nparts = (int)std::min<int64_t>(most, a.max_blocks);
    for (int pass = 0; pass < (in_place ? 2 : 1); ++pass) {
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
        std::sort(w.begin(), w.end());
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
