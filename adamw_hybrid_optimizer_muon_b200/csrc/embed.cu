// Embedding lookup, and the embedding table's gradient by sorted tokens.
//
//   lookup:    out[i] = scale * table[id_i]
//   gradient:  grad[v] = scale * sum over {i : id_i = v} of dY[i]   (+ grad[v])
//
// Both are bound by HBM. The lookup reads each token's row and writes it once.
// The gradient reads each row of dY once and writes each row of the table's
// gradient once: the tokens are sorted (stably, by radix), equal tokens stand
// next to each other, and their rows are added in registers, in token order.
// No atomics touch a value, so the same inputs give the same bits, and a token
// that fills the batch costs what any other batch does.
//
// Sort. Keys are token ids; positions of the batch travel with them. Up to
// 8192 tokens of a table of fewer than 2^19 rows are sorted by one block in
// shared memory, key and position packed into 32 bits; more by tiles of 4096,
// a histogram and a scatter launch per digit, each scatter block forming its
// own offsets from the tiles' histograms. Digits have up to nine bits, so a
// vocabulary below 2^18 takes two passes. A bit map of the rows that have
// tokens is filled on the way.
//
// Sum. The sorted tokens are cut into tiles of S. A block of 128 threads takes
// one tile and 128 * VEC columns and walks the tile with eight rows' loads in
// flight; a run of equal tokens inside the tile is written to its row at once.
// A run that crosses tiles leaves one fp32 partial row per tile, and a second
// kernel adds those in tile order. Other blocks of the same launch write zeros
// to the rows that have no token.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace ma {

namespace {

constexpr int kSortThreads = 1024;  // one-block sort
constexpr int kSortItems = 8;
constexpr int kSmallSort = kSortThreads * kSortItems;  // 8192 tokens
constexpr int kPosBits = 13;
constexpr int kSmallKeyBits = 32 - kPosBits;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kTileThreads = 512;
constexpr int kTile = kTileThreads * 8;  // tokens a block ranks at a time
constexpr int kMaxTiles = 512;           // histograms a scatter block reads per digit
constexpr int kSumThreads = 128;
constexpr int kFixThreads = 256;
constexpr int kRowsAhead = 8;            // rows of dY whose loads are in flight per thread

struct Ids {
    const void* p;
    int64_t n, rows, padding;
    int32_t i64;
    int* status;
};

// The sort key of token i: its id, or `rows` for one that adds to no row
// (padding, or an id outside the table, which is recorded).
__device__ __forceinline__ uint32_t id_key(const Ids& I, int64_t i) {
    if (!MA_INB(i, 1, I.n, I.status)) return (uint32_t)I.rows;
    const int64_t id = I.i64 ? reinterpret_cast<const int64_t*>(I.p)[i] : reinterpret_cast<const int32_t*>(I.p)[i];
    if (id == I.padding) return (uint32_t)I.rows;
    if (id < 0 || id >= I.rows) {
        record_error(I.status, MA_ERR_BOUNDS);
        return (uint32_t)I.rows;
    }
    return (uint32_t)id;
}

// Lanes of the warp (among `valid`) whose digit equals this lane's.
__device__ __forceinline__ uint32_t match_digit(uint32_t digit, int bits, uint32_t valid) {
    uint32_t peers = valid;
    for (int b = 0; b < bits; ++b) {
        const uint32_t bal = __ballot_sync(0xffffffffu, (digit >> b) & 1u);
        peers &= ((digit >> b) & 1u) ? bal : ~bal;
    }
    return peers;
}

// Exclusive prefix, over digits, of `total` (thread t < ndig holds digit t's
// total; the other threads pass 0), by every thread of the block.
template <int NT>
__device__ __forceinline__ uint32_t digit_scan(uint32_t total, uint32_t* warp_sums) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t x = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
        uint32_t s = lane < NT / 32 ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < NT / 32) warp_sums[lane] = s;
    }
    __syncthreads();
    return x - total + (w ? warp_sums[w - 1] : 0);
}

struct SortArgs {
    Ids ids;
    uint32_t* keys;    // out: sorted keys
    int32_t* pos;      // out: their positions
    uint32_t* bitmap;  // rows that have tokens
    int32_t bitmap_words;
    int32_t digit_bits, passes;
};

// One block sorts up to 8192 tokens. Warp w owns items 256 w .. 256 w + 255, in
// eight rounds of 32; the rank of an item among the equal digits of its warp is
// the warp's running count of that digit plus the equal lanes before it.
__global__ void __launch_bounds__(kSortThreads) embed_sort_small_kernel(const __grid_constant__ SortArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ uint32_t smem[];
    uint32_t* items = smem;                                                  // 8192
    uint16_t* hist = reinterpret_cast<uint16_t*>(smem + kSmallSort);         // [32][ndig]
    __shared__ uint32_t warp_sums[32];
    __shared__ uint32_t base[kMaxDigits];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int n = (int)A.ids.n, ndig = 1 << A.digit_bits;
    for (int i = t; i < A.bitmap_words; i += kSortThreads) A.bitmap[i] = 0;
    uint32_t item[kSortItems];
#pragma unroll
    for (int r = 0; r < kSortItems; ++r) {
        const int i = w * (32 * kSortItems) + 32 * r + lane;
        item[r] = i < n ? (id_key(A.ids, i) << kPosBits) | (uint32_t)i : 0xffffffffu;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortItems; ++r) {
        const uint32_t key = item[r] >> kPosBits;
        if (item[r] != 0xffffffffu && key < (uint32_t)A.ids.rows && MA_INB(key >> 5, 1, A.bitmap_words, A.ids.status))
            atomicOr(&A.bitmap[key >> 5], 1u << (key & 31));
    }
    for (int p = 0; p < A.passes; ++p) {
        const int shift = kPosBits + p * A.digit_bits;
        for (int i = t; i < 16 * ndig; i += kSortThreads) reinterpret_cast<uint32_t*>(hist)[i] = 0;
        __syncthreads();
        uint32_t rank[kSortItems];
#pragma unroll
        for (int r = 0; r < kSortItems; ++r) {
            const uint32_t d = (item[r] >> shift) & (ndig - 1);
            const uint32_t peers = match_digit(d, A.digit_bits, 0xffffffffu);
            const uint32_t before = hist[w * ndig + d];
            rank[r] = before + __popc(peers & ((1u << lane) - 1));
            __syncwarp();
            if (lane == __ffs(peers) - 1) hist[w * ndig + d] = (uint16_t)(before + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        uint32_t total = 0;
        if (t < ndig) {
            for (int q = 0; q < kSortThreads / 32; ++q) {
                const uint32_t c = hist[q * ndig + t];
                hist[q * ndig + t] = (uint16_t)total;
                total += c;
            }
        }
        const uint32_t excl = digit_scan<kSortThreads>(total, warp_sums);
        if (t < ndig) base[t] = excl;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSortItems; ++r) {
            const uint32_t d = (item[r] >> shift) & (ndig - 1);
            items[base[d] + hist[w * ndig + d] + rank[r]] = item[r];
        }
        __syncthreads();
        if (p + 1 < A.passes) {
#pragma unroll
            for (int r = 0; r < kSortItems; ++r) item[r] = items[w * (32 * kSortItems) + 32 * r + lane];
        }
    }
    for (int i = t; i < n; i += kSortThreads) {
        A.keys[i] = items[i] >> kPosBits;
        A.pos[i] = (int32_t)(items[i] & ((1u << kPosBits) - 1));
    }
}

struct TileArgs {
    Ids ids;
    const uint32_t* kin;  // NULL: the first pass, keys from the ids
    const int32_t* pin;
    uint32_t* kout;
    int32_t* pout;
    uint32_t* hist;       // [tiles][digits]
    uint32_t* bitmap;
    int32_t bitmap_words;
    int32_t shift, digit_bits, tiles, subtiles;  // a block ranks `subtiles` runs of kTile tokens, one after the other
};

__device__ __forceinline__ uint32_t tile_key(const TileArgs& A, int64_t i) {
    return A.kin ? A.kin[i] : id_key(A.ids, i);
}

__global__ void __launch_bounds__(kTileThreads) embed_hist_kernel(const __grid_constant__ TileArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ uint32_t h[kMaxDigits];
    const int ndig = 1 << A.digit_bits;
    for (int i = threadIdx.x; i < ndig; i += kTileThreads) h[i] = 0;
    if (!A.kin)  // the first pass clears the map, the first scatter fills it
        for (int i = blockIdx.x * kTileThreads + threadIdx.x; i < A.bitmap_words; i += gridDim.x * kTileThreads)
            A.bitmap[i] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * A.subtiles * kTile;
    const int64_t i1 = min(A.ids.n, i0 + (int64_t)A.subtiles * kTile);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kTileThreads)
        atomicAdd(&h[(tile_key(A, i) >> A.shift) & (ndig - 1)], 1u);
    __syncthreads();
    for (int i = threadIdx.x; i < ndig; i += kTileThreads) A.hist[(int64_t)blockIdx.x * ndig + i] = h[i];
}

__global__ void __launch_bounds__(kTileThreads) embed_scatter_kernel(const __grid_constant__ TileArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = kTileThreads / 32;
    __shared__ __align__(16) uint16_t hist[W * kMaxDigits];
    __shared__ uint32_t base[kMaxDigits];
    __shared__ uint32_t warp_sums[32];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int ndig = 1 << A.digit_bits;
    // where this block's tokens of digit t begin: all smaller digits, and this digit in the tiles before
    uint32_t total = 0, mine = 0;
    if (t < ndig) {
#pragma unroll 8
        for (int q = 0; q < A.tiles; ++q) {
            const uint32_t c = A.hist[(int64_t)q * ndig + t];
            if (q < (int)blockIdx.x) mine += c;
            total += c;
        }
    }
    const uint32_t excl = digit_scan<kTileThreads>(total, warp_sums);
    if (t < ndig) base[t] = excl + mine;
    for (int sub = 0; sub < A.subtiles; ++sub) {
        const int64_t i0 = ((int64_t)blockIdx.x * A.subtiles + sub) * kTile;
        if (i0 >= A.ids.n) break;
        for (int i = t; i < W * ndig / 2; i += kTileThreads) reinterpret_cast<uint32_t*>(hist)[i] = 0;
        __syncthreads();
        uint32_t key[8], rank[8];
        int32_t pos[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int64_t i = i0 + w * 256 + 32 * r + lane;
            const bool in = i < A.ids.n;
            key[r] = in ? tile_key(A, i) : 0u;
            pos[r] = in ? (A.pin ? A.pin[i] : (int32_t)i) : -1;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const uint32_t d = (key[r] >> A.shift) & (ndig - 1);
            const uint32_t valid = __ballot_sync(0xffffffffu, pos[r] >= 0);
            const uint32_t peers = match_digit(d, A.digit_bits, valid);
            const uint32_t before = hist[w * ndig + d];
            rank[r] = before + __popc(peers & ((1u << lane) - 1));
            __syncwarp();
            if (pos[r] >= 0 && lane == __ffs(peers) - 1) hist[w * ndig + d] = (uint16_t)(before + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        uint32_t count = 0;
        if (t < ndig) {
            for (int q = 0; q < W; ++q) {
                const uint32_t c = hist[q * ndig + t];
                hist[q * ndig + t] = (uint16_t)count;
                count += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (pos[r] < 0) continue;
            const uint32_t d = (key[r] >> A.shift) & (ndig - 1);
            const int64_t o = (int64_t)base[d] + hist[w * ndig + d] + rank[r];
            if (!MA_INB(o, 1, A.ids.n, A.ids.status)) continue;
            A.kout[o] = key[r];
            A.pout[o] = pos[r];
            if (!A.kin && key[r] < (uint32_t)A.ids.rows) {
                const uint32_t word = key[r] >> 5, bit = 1u << (key[r] & 31);
                if (MA_INB(word, 1, A.bitmap_words, A.ids.status) &&
                    !(*reinterpret_cast<volatile uint32_t*>(&A.bitmap[word]) & bit))
                    atomicOr(&A.bitmap[word], bit);
            }
        }
        __syncthreads();
        if (t < ndig) base[t] += count;
    }
}

// ------------------------------------------------------------------ sums

struct SumArgs {
    const uint32_t* keys;
    const int32_t* pos;
    const uint32_t* bitmap;  // NULL: no row has a token
    const void* dy;
    void* grad;
    float* slots;  // per tile: the partial row of a run that began before it, and of one that goes on after it
    int64_t n, rows, dim, ldy, ldg, slot_ld;
    int64_t sum_blocks, zero_rows;  // blocks that sum; rows of each block after them that writes zeros
    int32_t tile, tiles, col_blocks, accumulate;
    float scale;
    int* status;
};

template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float (&f)[VEC]) {
    if constexpr (BF16 && VEC == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    } else if constexpr (BF16 && VEC == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    } else if constexpr (BF16 && VEC == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(p) + i);
        f[0] = bf16_lo(w); f[1] = bf16_hi(w);
    } else if constexpr (BF16) {
        static_assert(VEC == 1);
        f[0] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
    } else if constexpr (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else if constexpr (VEC == 4) {
        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    } else if constexpr (VEC == 2) {
        const float2 a = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(p) + i);
        f[0] = a.x; f[1] = a.y;
    } else {
        static_assert(VEC == 1);
        f[0] = reinterpret_cast<const float*>(p)[i];
    }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&f)[VEC]) {
    if constexpr (BF16 && VEC == 8) {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    } else if constexpr (BF16 && VEC == 4) {
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) =
            make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    } else if constexpr (BF16 && VEC == 2) {
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p) + i) = pack_bf16x2(f[0], f[1]);
    } else if constexpr (BF16) {
        static_assert(VEC == 1);
        reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
    } else if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(p) + i) = make_float2(f[0], f[1]);
    } else {
        static_assert(VEC == 1);
        reinterpret_cast<float*>(p)[i] = f[0];
    }
}

// A finished sum: scaled, added to the old value where asked, rounded once.
template <bool GB, int VEC>
__device__ __forceinline__ void write_row(const SumArgs& A, uint32_t key, int64_t col, const float (&acc)[VEC]) {
    const int64_t o = (int64_t)key * A.ldg + col;
    if (!MA_INB(o, VEC, (A.rows - 1) * A.ldg + A.dim, A.status)) return;
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = acc[e] * A.scale;
    if (A.accumulate) {
        float old[VEC];
        load_vec<GB, VEC>(A.grad, o, old);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] += old[e];
    }
    store_vec<GB, VEC>(A.grad, o, f);
}

template <bool GB, int VEC>
__device__ __forceinline__ void zero_rows(const SumArgs& A, int64_t block) {
    const int lane = threadIdx.x & 31;
    const int64_t r1 = min(A.rows, (block + 1) * A.zero_rows);
    float z[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) z[e] = 0.f;
    for (int64_t r = block * A.zero_rows + (threadIdx.x >> 5); r < r1; r += kSumThreads / 32) {
        if (A.bitmap && (A.bitmap[r >> 5] >> (r & 31) & 1u)) continue;
        for (int64_t c = VEC * lane; c < A.dim; c += VEC * 32)
            if (MA_INB(r * A.ldg + c, VEC, (A.rows - 1) * A.ldg + A.dim, A.status))
                store_vec<GB, VEC>(A.grad, r * A.ldg + c, z);
    }
}

constexpr int kMaxSumTile = 64;

template <bool YB, bool GB, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ SumArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    if ((int64_t)blockIdx.x >= A.sum_blocks) {
        zero_rows<GB, VEC>(A, blockIdx.x - A.sum_blocks);
        return;
    }
    __shared__ uint32_t sk[kMaxSumTile + 2];  // keys, with the one before the tile and the one after it
    __shared__ int32_t sp[kMaxSumTile];
    const int tile = blockIdx.x / A.col_blocks;
    const int64_t i0 = (int64_t)tile * A.tile;
    const int cnt = (int)min((int64_t)A.tile, A.n - i0);
    const uint32_t none = 0xffffffffu;
    for (int i = threadIdx.x; i < cnt + 2; i += kSumThreads) {
        const int64_t q = i0 + i - 1;
        sk[i] = q >= 0 && q < A.n ? A.keys[q] : none;
        if (i >= 1 && i <= cnt) sp[i - 1] = A.pos[q];
    }
    __syncthreads();
    const int64_t col = ((int64_t)(blockIdx.x % A.col_blocks) * kSumThreads + threadIdx.x) * VEC;
    if (col >= A.dim) return;
    bool head = sk[0] == sk[1];  // the first run began in an earlier tile
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    for (int b = 0; b < cnt; b += kRowsAhead) {
        float f[kRowsAhead][VEC];
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            if (b + u < cnt && sk[b + u + 1] < (uint32_t)A.rows) {
                const int64_t o = (int64_t)sp[b + u] * A.ldy + col;
                if (MA_INB(o, VEC, (A.n - 1) * A.ldy + A.dim, A.status)) load_vec<YB, VEC>(A.dy, o, f[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            const int i = b + u;
            if (i >= cnt) break;
            const uint32_t key = sk[i + 1];
            if (key >= (uint32_t)A.rows) return;  // only tokens without a row are left
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += f[u][e];
            const bool last = i + 1 == cnt, more = sk[i + 2] == key;
            if (!last && more) continue;
            if (head || more) {
                float* s = A.slots + (2 * (int64_t)tile + (head ? 0 : 1)) * A.slot_ld + col;
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] = acc[e];
            } else {
                write_row<GB, VEC>(A, key, col, acc);
            }
            head = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
        }
    }
}

// Runs that cross tiles: the partial row of the tile they begin in, then those
// of the tiles they go on through, in that order. A block takes 32 * CV columns;
// every warp looks at 32 tiles at a time for runs that begin in them and go
// on. A run of up to kShortRun tiles is one warp's; of a longer one each warp
// adds a contiguous share, and the shares are added in order.
constexpr int kShortRun = 16;

template <int CV>
__device__ __forceinline__ void add_slots(const SumArgs& A, int64_t first, int64_t count, int64_t col,
                                          float (&acc)[CV]) {
#pragma unroll 4
    for (int64_t q = 0; q < count; ++q) {
        const float* s = A.slots + 2 * (first + q) * A.slot_ld + col;
        float f[CV];
        load_vec<false, CV>(s, 0, f);
#pragma unroll
        for (int e = 0; e < CV; ++e) acc[e] += f[e];
    }
}

template <bool GB, int CV>
__global__ void __launch_bounds__(kFixThreads) embed_fix_kernel(const __grid_constant__ SumArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = kFixThreads / 32;
    __shared__ float part[W][32 * CV];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t col = ((int64_t)blockIdx.x * 32 + lane) * CV;
    const bool in = col < A.dim;
    for (int64_t g0 = (int64_t)blockIdx.y * 32; g0 < A.tiles; g0 += (int64_t)gridDim.y * 32) {
        const int64_t t = g0 + lane;
        bool starts = false;
        if (t + 1 < A.tiles) {
            const int64_t i1 = (t + 1) * A.tile;  // first token of the next tile
            const uint32_t key = A.keys[i1];
            const bool more = key < (uint32_t)A.rows && A.keys[i1 - 1] == key;
            const bool before = t > 0 && A.keys[t * A.tile - 1] == key;  // then the whole tile is that run
            starts = more && !before;
        }
        uint32_t todo = __ballot_sync(0xffffffffu, starts);
        for (int k = 0; todo; todo &= todo - 1, ++k) {
            const int64_t t0 = g0 + __ffs(todo) - 1;
            const uint32_t key = A.keys[(t0 + 1) * A.tile];
            int64_t m = 0;  // tiles that the run goes on through
            for (;; m += 32) {
                const int64_t q = t0 + 1 + m + lane;
                const uint32_t same = __ballot_sync(0xffffffffu, q < A.tiles && A.keys[q * A.tile] == key);
                if (same != 0xffffffffu) {
                    m += __ffs(~same) - 1;
                    break;
                }
            }
            float acc[CV];
#pragma unroll
            for (int e = 0; e < CV; ++e) acc[e] = 0.f;
            if (m <= kShortRun) {
                if (k % W != w || !in) continue;
                load_vec<false, CV>(A.slots, (2 * t0 + 1) * A.slot_ld + col, acc);
                add_slots<CV>(A, t0 + 1, m, col, acc);
                write_row<GB, CV>(A, key, col, acc);
                continue;
            }
            const int64_t lo = m * w / W, hi = m * (w + 1) / W;
            if (in) {
                if (w == 0) load_vec<false, CV>(A.slots, (2 * t0 + 1) * A.slot_ld + col, acc);
                add_slots<CV>(A, t0 + 1 + lo, hi - lo, col, acc);
#pragma unroll
                for (int e = 0; e < CV; ++e) part[w][lane * CV + e] = acc[e];
            }
            __syncthreads();
            if (w == 0 && in) {
#pragma unroll
                for (int q = 1; q < W; ++q)
#pragma unroll
                    for (int e = 0; e < CV; ++e) acc[e] += part[q][lane * CV + e];
                write_row<GB, CV>(A, key, col, acc);
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    Ids ids;
    const void* table;
    void* out;
    int64_t dim, ldt, ldo;
    float scale;
    int32_t lanes_log2;  // threads per token row: 2^lanes_log2 of the block's 256
};

constexpr int kLookupThreads = 256;

template <bool TB, bool OB, int VEC>
__global__ void __launch_bounds__(kLookupThreads) embed_lookup_kernel(const __grid_constant__ LookupArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    const int lanes = 1 << A.lanes_log2;
    const int64_t i = ((int64_t)blockIdx.x << (8 - A.lanes_log2)) + (threadIdx.x >> A.lanes_log2);
    if (i >= A.ids.n || !MA_INB(i, 1, A.ids.n, A.ids.status)) return;
    const int64_t id =
        A.ids.i64 ? reinterpret_cast<const int64_t*>(A.ids.p)[i] : reinterpret_cast<const int32_t*>(A.ids.p)[i];
    const bool in = id >= 0 && id < A.ids.rows;
    const int t = threadIdx.x & (lanes - 1);
    if (!in && id != A.ids.padding && t == 0) record_error(A.ids.status, MA_ERR_BOUNDS);
    constexpr int U = 4;
    for (int64_t c0 = (int64_t)t * VEC; c0 < A.dim; c0 += (int64_t)U * lanes * VEC) {
        float f[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + (int64_t)u * lanes * VEC;
            if (in && c < A.dim && MA_INB(id * A.ldt + c, VEC, (A.ids.rows - 1) * A.ldt + A.dim, A.ids.status))
                load_vec<TB, VEC>(A.table, id * A.ldt + c, f[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + (int64_t)u * lanes * VEC;
            if (c >= A.dim) break;
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[u][e] = in ? f[u][e] * A.scale : 0.f;
            if (MA_INB(i * A.ldo + c, VEC, (A.ids.n - 1) * A.ldo + A.dim, A.ids.status))
                store_vec<OB, VEC>(A.out, i * A.ldo + c, f[u]);
        }
    }
}

// ------------------------------------------------------------------ host

int bits_for(int64_t rows) {  // bits of the largest key, `rows`
    int b = 1;
    while ((rows >> b) != 0) ++b;
    return b;
}

// Whether rows of `dim` elements with stride ld can be read as vectors of vec elements.
bool rows_take(const void* p, int64_t dim, int64_t ld, int esz, int vec) {
    const uintptr_t align = (uintptr_t)std::min(16, vec * esz);
    return dim % vec == 0 && reinterpret_cast<uintptr_t>(p) % align == 0 && ((uintptr_t)ld * esz) % align == 0;
}

struct GradLayout {
    bool small;
    int digit_bits, passes, tiles, subtiles;
    int sum_tile;  // tokens per tile of the sum
    int64_t bitmap_words, sum_tiles, slot_ld;
    size_t off_k0, off_p0, off_k1, off_p1, off_hist, off_bitmap, off_slots, total;
};

// Tokens per tile of the sum: the longest of 64, 32, 16 and 8 that still gives
// about four blocks to each of 148 SMs (a longer tile leaves fewer partial
// rows; too few blocks leave SMs without loads in flight).
int sum_tile(int64_t n, int64_t dim) {
    const int64_t col_blocks = (dim + 8 * kSumThreads - 1) / (8 * kSumThreads);
    int s = kMaxSumTile;
    while (s > 8 && (n + s - 1) / s * col_blocks < 4 * 148) s /= 2;
    return s;
}

GradLayout grad_layout(int64_t n, int64_t rows, int64_t dim) {
    GradLayout L;
    std::memset(&L, 0, sizeof(L));
    const int bits = bits_for(rows);
    L.small = n <= kSmallSort && bits <= kSmallKeyBits;
    L.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    L.digit_bits = (bits + L.passes - 1) / L.passes;
    L.tiles = (int)((n + kTile - 1) / kTile);
    L.subtiles = (L.tiles + kMaxTiles - 1) / kMaxTiles;
    if (L.subtiles > 1) L.tiles = (L.tiles + L.subtiles - 1) / L.subtiles;
    L.subtiles = std::max(1, L.subtiles);
    L.bitmap_words = (rows + 31) / 32;
    L.slot_ld = (dim + 7) / 8 * 8;
    L.sum_tile = sum_tile(n, dim);
    L.sum_tiles = (n + L.sum_tile - 1) / L.sum_tile;
    size_t off = 0;
    auto take = [&off](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return at;
    };
    L.off_k0 = take((size_t)n * 4);
    L.off_p0 = take((size_t)n * 4);
    L.off_k1 = take(L.small ? 0 : (size_t)n * 4);
    L.off_p1 = take(L.small ? 0 : (size_t)n * 4);
    L.off_hist = take(L.small ? 0 : (size_t)L.tiles * kMaxDigits * 4);
    L.off_bitmap = take((size_t)L.bitmap_words * 4);
    L.off_slots = take((size_t)L.sum_tiles * 2 * L.slot_ld * 4);
    L.total = off;
    return L;
}

constexpr size_t kSmallSortSmem = (size_t)kSmallSort * 4 + 32 * kMaxDigits * 2;

cudaError_t sort_small_setup() {
    static PerDevice<int> cache;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cache.get(dev, &done, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(embed_sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kSmallSortSmem);
    });
}

template <bool YB, bool GB, int VEC>
cudaError_t launch_sum(const SumArgs& A, unsigned grid, cudaStream_t s) {
    return launch_pdl(embed_sum_kernel<YB, GB, VEC>, dim3(grid), dim3(kSumThreads), 0, s, A);
}

template <bool YB, bool GB>
cudaError_t launch_sum_vec(const SumArgs& A, int vec, unsigned grid, cudaStream_t s) {
    return vec == 8   ? launch_sum<YB, GB, 8>(A, grid, s)
           : vec == 2 ? launch_sum<YB, GB, 2>(A, grid, s)
                      : launch_sum<YB, GB, 1>(A, grid, s);
}

cudaError_t run_sum(const SumArgs& A, int ydt, int gdt, int vec, unsigned grid, cudaStream_t s) {
    if (ydt == MA_BF16)
        return gdt == MA_BF16 ? launch_sum_vec<true, true>(A, vec, grid, s) : launch_sum_vec<true, false>(A, vec, grid, s);
    return gdt == MA_BF16 ? launch_sum_vec<false, true>(A, vec, grid, s) : launch_sum_vec<false, false>(A, vec, grid, s);
}

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MA_OK : MA_ERR_CUDA; }

int check_ids(int64_t n, const void* ids, int idt, int64_t rows, int64_t dim) {
    if (n < 0 || rows < 0 || dim < 0) return MA_ERR_SHAPE;
    if (idt != MA_I32 && idt != MA_I64) return MA_ERR_DTYPE;
    if (n > INT32_MAX || rows > (int64_t(1) << 30) || dim > (int64_t(1) << 30)) return MA_ERR_UNSUPPORTED;
    if (n > 0 && !ids) return MA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(ids) % (idt == MA_I64 ? 8 : 4) != 0) return MA_ERR_ALIGN;
    return MA_OK;
}

int check_rows(const void* p, int dt, int64_t rows, int64_t dim, int64_t ld) {
    if (dt != MA_F32 && dt != MA_BF16) return MA_ERR_DTYPE;
    if (ld < dim) return MA_ERR_SHAPE;
    if (ld > (int64_t(1) << 31)) return MA_ERR_UNSUPPORTED;
    if (rows > 0 && dim > 0 && !p) return MA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(p) % (dt == MA_BF16 ? 2 : 4) != 0) return MA_ERR_ALIGN;
    return MA_OK;
}

// Whether two ranges of rows share a byte's address range.
bool meet(const void* a, size_t abytes, const void* b, size_t bbytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return abytes && bbytes && x < y + bbytes && y < x + abytes;
}

size_t span(int64_t rows, int64_t dim, int64_t ld, int dt) {
    return rows > 0 && dim > 0 ? (size_t)((rows - 1) * ld + dim) * (dt == MA_BF16 ? 2 : 4) : 0;
}

int lookup(int64_t n, const void* ids, int idt, int64_t rows, int64_t dim, const void* table, int tdt, int64_t ldt,
           float scale, int64_t padding, void* out, int odt, int64_t ldo, void* stream) {
    int st = check_ids(n, ids, idt, rows, dim);
    if (st || (st = check_rows(table, tdt, rows, dim, ldt)) || (st = check_rows(out, odt, n, dim, ldo))) return st;
    if (!std::isfinite(scale)) return MA_ERR_ARG;
    const size_t ob = span(n, dim, ldo, odt);
    if (meet(out, ob, table, span(rows, dim, ldt, tdt)) || meet(out, ob, ids, (size_t)n * (idt == MA_I64 ? 8 : 4)))
        return MA_ERR_ARG;
    if ((st = device_ready(nullptr))) return st;
    if (n == 0 || dim == 0) return MA_OK;
    LookupArgs A;
    std::memset(&A, 0, sizeof(A));
    A.ids = Ids{ids, n, rows, padding, idt == MA_I64, device_status_ptr()};
    A.table = table;
    A.out = out;
    A.dim = dim;
    A.ldt = ldt;
    A.ldo = ldo;
    A.scale = scale;
    const int tsz = tdt == MA_BF16 ? 2 : 4, osz = odt == MA_BF16 ? 2 : 4;
    int vec = 1;
    for (int v : {8, 2})
        if (vec == 1 && rows_take(table, dim, ldt, tsz, v) && rows_take(out, dim, ldo, osz, v)) vec = v;
    while (A.lanes_log2 < 8 && ((int64_t)vec << A.lanes_log2) < dim) ++A.lanes_log2;
    const int64_t per_block = int64_t(1) << (8 - A.lanes_log2);
    const dim3 grid((unsigned)((n + per_block - 1) / per_block)), block(kLookupThreads);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int pr = prof_begin(MA_PROF_EMBED, s);
    auto go = [&](auto v) -> cudaError_t {
        constexpr int V = decltype(v)::value;
        if (tdt == MA_BF16)
            return odt == MA_BF16 ? launch_pdl(embed_lookup_kernel<true, true, V>, grid, block, 0, s, A)
                                  : launch_pdl(embed_lookup_kernel<true, false, V>, grid, block, 0, s, A);
        return odt == MA_BF16 ? launch_pdl(embed_lookup_kernel<false, true, V>, grid, block, 0, s, A)
                              : launch_pdl(embed_lookup_kernel<false, false, V>, grid, block, 0, s, A);
    };
    const cudaError_t e = vec == 8   ? go(std::integral_constant<int, 8>{})
                          : vec == 2 ? go(std::integral_constant<int, 2>{})
                                     : go(std::integral_constant<int, 1>{});
    prof_end(pr, s, 0.0, (double)n * dim * (tsz + osz));
    return cuda_rc(e);
}

int grad(int64_t n, const void* ids, int idt, int64_t rows, int64_t dim, const void* dY, int ydt, int64_t ldy,
         float scale, int64_t padding, int accumulate, void* g, int gdt, int64_t ldg, void* ws, size_t ws_bytes,
         void* stream) {
    int st = check_ids(n, ids, idt, rows, dim);
    if (st || (st = check_rows(dY, ydt, n, dim, ldy)) || (st = check_rows(g, gdt, rows, dim, ldg))) return st;
    if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return MA_ERR_ARG;
    const GradLayout L = grad_layout(n, rows, dim);
    const size_t gb = span(rows, dim, ldg, gdt), wb = n > 0 ? L.total : 0;
    if (wb && (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < wb)) return MA_ERR_WORKSPACE;
    const size_t ib = (size_t)n * (idt == MA_I64 ? 8 : 4), yb = span(n, dim, ldy, ydt);
    if (meet(g, gb, dY, yb) || meet(g, gb, ids, ib) || meet(ws, wb, g, gb) || meet(ws, wb, dY, yb) ||
        meet(ws, wb, ids, ib))
        return MA_ERR_ARG;
    int sms = 0;
    if ((st = device_ready(&sms))) return st;
    if (rows == 0 || dim == 0 || (n == 0 && accumulate)) return MA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    auto at32 = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
    const Ids I{ids, n, rows, padding, idt == MA_I64, device_status_ptr()};
    SumArgs S;
    std::memset(&S, 0, sizeof(S));
    S.bitmap = n > 0 ? at32(L.off_bitmap) : nullptr;
    S.dy = dY;
    S.grad = g;
    S.slots = n > 0 ? reinterpret_cast<float*>(base + L.off_slots) : nullptr;
    S.n = n;
    S.rows = rows;
    S.dim = dim;
    S.ldy = ldy;
    S.ldg = ldg;
    S.slot_ld = L.slot_ld;
    S.scale = scale;
    S.accumulate = accumulate;
    S.status = device_status_ptr();
    const int ysz = ydt == MA_BF16 ? 2 : 4, gsz = gdt == MA_BF16 ? 2 : 4;
    int vec = 1;
    for (int v : {8, 2})
        if (vec == 1 && rows_take(dY, dim, ldy, ysz, v) && rows_take(g, dim, ldg, gsz, v)) vec = v;
    S.col_blocks = (int)((dim + kSumThreads * vec - 1) / (kSumThreads * vec));
    S.tile = L.sum_tile;
    S.tiles = (int)L.sum_tiles;
    S.sum_blocks = (int64_t)S.tiles * S.col_blocks;
    // a block that writes zeros covers about 64 KB of rows
    S.zero_rows = std::max<int64_t>(4, (int64_t(1) << 16) / (dim * gsz) / 4 * 4);
    const int64_t blocks = S.sum_blocks + (accumulate ? 0 : (rows + S.zero_rows - 1) / S.zero_rows);
    if (blocks > INT32_MAX) return MA_ERR_UNSUPPORTED;
    const uint32_t* keys = nullptr;
    const int32_t* pos = nullptr;
    const int pr = prof_begin(MA_PROF_EMBED, s);
    cudaError_t e = cudaSuccess;
    if (n > 0 && L.small) {
        if ((e = sort_small_setup()) != cudaSuccess) return MA_ERR_CUDA;
        SortArgs A{I, at32(L.off_k0), reinterpret_cast<int32_t*>(base + L.off_p0), at32(L.off_bitmap),
                   (int32_t)L.bitmap_words, L.digit_bits, L.passes};
        e = launch_pdl(embed_sort_small_kernel, dim3(1), dim3(kSortThreads), kSmallSortSmem, s, A);
        keys = A.keys;
        pos = A.pos;
    } else if (n > 0) {
        TileArgs A;
        std::memset(&A, 0, sizeof(A));
        A.ids = I;
        A.hist = at32(L.off_hist);
        A.bitmap = at32(L.off_bitmap);
        A.bitmap_words = (int32_t)L.bitmap_words;
        A.digit_bits = L.digit_bits;
        A.tiles = L.tiles;
        A.subtiles = L.subtiles;
        for (int p = 0; p < L.passes && e == cudaSuccess; ++p) {
            const bool odd = p & 1;
            A.kout = at32(odd ? L.off_k1 : L.off_k0);
            A.pout = reinterpret_cast<int32_t*>(base + (odd ? L.off_p1 : L.off_p0));
            A.shift = p * L.digit_bits;
            e = launch_pdl(embed_hist_kernel, dim3(L.tiles), dim3(kTileThreads), 0, s, A);
            if (e == cudaSuccess) e = launch_pdl(embed_scatter_kernel, dim3(L.tiles), dim3(kTileThreads), 0, s, A);
            A.kin = A.kout;
            A.pin = A.pout;
        }
        keys = A.kin;
        pos = A.pin;
    }
    if (e != cudaSuccess) return MA_ERR_CUDA;
    S.keys = keys;
    S.pos = pos;
    e = run_sum(S, ydt, gdt, vec, (unsigned)blocks, s);
    if (e == cudaSuccess && S.tiles > 1) {
        const int cv = vec == 1 ? 1 : vec == 2 ? 2 : 4;
        auto fix = [&](auto v) -> cudaError_t {
            constexpr int V = decltype(v)::value;
            const unsigned gx = (unsigned)((dim + 32 * V - 1) / (32 * V));
            const unsigned gy =
                (unsigned)std::max<int64_t>(1, std::min<int64_t>((S.tiles + 31) / 32, 8 * (int64_t)sms / gx));
            return gdt == MA_BF16 ? launch_pdl(embed_fix_kernel<true, V>, dim3(gx, gy), dim3(kFixThreads), 0, s, S)
                                  : launch_pdl(embed_fix_kernel<false, V>, dim3(gx, gy), dim3(kFixThreads), 0, s, S);
        };
        e = cv == 1   ? fix(std::integral_constant<int, 1>{})
            : cv == 2 ? fix(std::integral_constant<int, 2>{})
                      : fix(std::integral_constant<int, 4>{});
    }
    prof_end(pr, s, 0.0, (double)n * dim * ysz + (double)rows * dim * gsz);
    return cuda_rc(e);
}

}  // namespace
}  // namespace ma

extern "C" {

int ma_embed_lookup(int64_t n, const void* ids, int idt, int64_t rows, int64_t dim, const void* table, int tdt,
                    int64_t ldt, float scale, int64_t padding, void* out, int odt, int64_t ldo, void* stream) {
    return ma::lookup(n, ids, idt, rows, dim, table, tdt, ldt, scale, padding, out, odt, ldo, stream);
}

size_t ma_embed_grad_workspace_bytes(int64_t n, int64_t rows, int64_t dim) {
    if (n < 0 || rows < 0 || dim < 0 || n > INT32_MAX || rows > (int64_t(1) << 30) || dim > (int64_t(1) << 30))
        return SIZE_MAX;
    return n > 0 ? ma::grad_layout(n, rows, dim).total : 0;
}

int ma_embed_grad(int64_t n, const void* ids, int idt, int64_t rows, int64_t dim, const void* dY, int ydt, int64_t ldy,
                  float scale, int64_t padding, int accumulate, void* grad, int gdt, int64_t ldg, void* ws,
                  size_t ws_bytes, void* stream) {
    return ma::grad(n, ids, idt, rows, dim, dY, ydt, ldy, scale, padding, accumulate, grad, gdt, ldg, ws, ws_bytes,
                    stream);
}

}  // extern "C"
