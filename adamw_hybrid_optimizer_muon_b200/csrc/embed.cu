// Embedding lookup, and the embedding table's gradient by sorted tokens.
//
//   lookup:    out[i] = scale * table[id_i]
//   gradient:  grad[v] = scale * sum over {i : id_i = v} of dY[i]   (+ grad[v])
//
// Both are bound by HBM. The lookup reads each token's row and writes it once.
// The gradient reads each row of dY once and writes each row of the table's
// gradient once: the tokens are sorted (stably, by radix), equal tokens stand
// next to each other, and their rows are added in registers, in token order.
// No atomics touch a value, so the same inputs give the same bits. A token that
// fills the batch costs up to twice what uniform tokens do (131,072 x 1280 bf16
// into 65,536 rows 161 us, 115; 1,000,000 x 128 into 50,000 298, 156), since few
// blocks add up its partial rows.
//
// Sort. Keys are token ids; positions of the batch travel with them. Up to
// 8192 tokens of a table of fewer than 2^19 rows are sorted by one block in
// shared memory, key and position packed into 32 bits; more by tiles of 1024, a
// histogram, a scan and a scatter launch per digit. Digits have up to nine bits:
// a vocabulary below 2^18 takes two passes. A whole gradient of 32,000 x 128
// bf16 by the one block (by the tiles): 100 tokens 12.5 us (20.5), 2048 15.3
// (24.2), 8192 26.1 (26.5).
//
// Sum. The sorted tokens are cut into tiles of S. A block takes one tile and a
// range of columns and adds up the runs of equal tokens that begin in its tile,
// to their ends if those lie beyond it, with eight to sixteen loads in flight
// per thread. Only a run of more than kLong tokens is cut at the tiles'
// borders: each tile leaves an fp32 partial row, and a last kernel adds those
// in tile order.
//
// Zeros. Most of a table's rows have no token, and writing their zeros is most
// of the traffic. The sort and the last kernel are bound by latency and leave
// HBM idle, so the zeros are spread: each kernel from the one that knows which
// rows have tokens on (a bit per row) writes a share beside its own work, the
// sums the rest.
//
// Measured, bf16: 8192 tokens x 4096 into 32,000 rows 72 us, where the zeros of
// the same table without a token take 49 (262 MB at 5.3 TB/s); 131,072 x
// 1280 of a skewed distribution into 65,536 rows 129 us for 503 MB. Rows that are
// not whole 16-byte vectors go by two elements or by one, and issue bounds them:
// uniform tokens of 1282 columns 190 us and of 1281 columns 227, of 1280 115.
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
// Two tokens a thread: ranking goes token by token within a warp, so more warps
// shorten it (131,072 skewed tokens of 65,536 rows x 1280, the whole gradient:
// 132 us, four tokens 136, eight 142).
constexpr int kTileThreads = 512;
constexpr int kTile = kTileThreads * 2;  // tokens a block ranks at a time
constexpr int kMaxTiles = 4096;          // tiles of a pass; longer batches have longer tiles
constexpr int kSumThreads = 256;         // at most
constexpr int kFixThreads = 256;
constexpr int kMaxSumTile = 512;
constexpr int kRing = 16;                // 16-byte copies in flight per thread of the sums
constexpr int kLong = 32;                // tokens; a longer run is cut at the tiles' borders

struct Ids {
    const void* p;
    int64_t n, rows, padding;
    int32_t i64;
    int* status;
};

// The sort key of an id: itself, or `rows` for one that adds to no row
// (padding, or an id outside the table, which is recorded).
__device__ __forceinline__ uint32_t id_key(const Ids& I, int64_t id) {
    if (id == I.padding) return (uint32_t)I.rows;
    if (id < 0 || id >= I.rows) {
        record_error(I.status, MA_ERR_BOUNDS);
        return (uint32_t)I.rows;
    }
    return (uint32_t)id;
}

// Keys of tokens first, first + stride, ... (R of them, `none` from `end` on):
// every load before the first use.
template <int R>
__device__ __forceinline__ void load_keys(const Ids& I, int64_t first, int64_t stride, int64_t end, uint32_t none,
                                          uint32_t (&key)[R]) {
    int64_t id[R];
    if (I.i64) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = first + r * stride;
            id[r] = i < end && MA_INB(i, 1, I.n, I.status) ? reinterpret_cast<const int64_t*>(I.p)[i] : I.padding;
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = first + r * stride;
            id[r] = i < end && MA_INB(i, 1, I.n, I.status) ? reinterpret_cast<const int32_t*>(I.p)[i] : I.padding;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = first + r * stride < end ? id_key(I, id[r]) : none;
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

// One kernel's share of the rows without a token: the table is cut into parts
// of `period` rows, a block each; rows lo .. hi - 1 of every part are this
// kernel's. Zero is all bits zero in either type, so rows are plain bytes.
struct ZeroShare {
    uint8_t* grad;
    uint32_t* present;  // a bit per row: whether a token points to it; NULL: to none
    int64_t rows, row_bytes, ld_bytes, period, lo, hi;
    int32_t blocks, aligned;  // aligned: every row begins and ends at a 16-byte boundary
    int* status;
};

__device__ __forceinline__ void write_zeros(const ZeroShare& Z, int64_t part) {
    constexpr int G = 8;  // rows a warp looks up at once
    const int lane = threadIdx.x & 31;
    const int64_t r1 = min(Z.rows, part * Z.period + Z.hi);
    for (int64_t g = part * Z.period + Z.lo + G * (threadIdx.x >> 5); g < r1; g += G * (blockDim.x >> 5)) {
        const int64_t q = g + lane;
        const bool empty = lane < G && q < r1 && !(Z.present && (Z.present[q >> 5] >> (q & 31) & 1u));
        for (uint32_t todo = __ballot_sync(0xffffffffu, empty); todo; todo &= todo - 1) {
            const int64_t r = g + __ffs(todo) - 1;
            uint8_t* row = Z.grad + r * Z.ld_bytes;
            if (!MA_INB(r, 1, Z.rows, Z.status)) continue;
            // 2-byte units up to the first 16-byte boundary (at most seven), 16-byte units, 2-byte units (at most seven)
            int64_t head = 0, body = Z.row_bytes;
            if (!Z.aligned) {
                head = min(Z.row_bytes, (int64_t)(-reinterpret_cast<intptr_t>(row) & 15));
                body = head + (Z.row_bytes - head) / 16 * 16;
                if (2 * lane < head) __stcs(reinterpret_cast<uint16_t*>(row) + lane, (uint16_t)0);
                if (body + 2 * lane < Z.row_bytes) __stcs(reinterpret_cast<uint16_t*>(row + body) + lane, (uint16_t)0);
            }
#pragma unroll 4
            for (int64_t c = head + 16 * lane; c < body; c += 512)
                __stcs(reinterpret_cast<uint4*>(row + c), make_uint4(0, 0, 0, 0));
        }
    }
}

struct SortArgs {
    Ids ids;
    int32_t* keys;  // out: sorted keys
    int32_t* pos;   // out: their positions
    int32_t digit_bits, passes;
    ZeroShare zero;  // blocks after the first find which rows of their part have tokens, and write zeros
};

// Which rows of part p have tokens, into Z.present; parts are whole words of it.
__device__ __forceinline__ void find_present(const Ids& I, const ZeroShare& Z, int64_t p, uint32_t* bits) {
    const int64_t r0 = p * Z.period, len = min(Z.rows - r0, Z.period);
    const int words = (int)((len + 31) / 32);
    for (int i = threadIdx.x; i < words; i += kSortThreads) bits[i] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < I.n; i += 8 * kSortThreads) {
        uint32_t key[8];
        load_keys(I, i, kSortThreads, I.n, (uint32_t)Z.rows, key);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t r = (int64_t)key[k] - r0;
            if (r >= 0 && r < len) atomicOr(&bits[r >> 5], 1u << (r & 31));
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < words; i += kSortThreads) Z.present[r0 / 32 + i] = bits[i];
    __syncthreads();
}

// One block sorts up to 8192 tokens, in R = ceil(n / 1024) rounds. Warp w owns
// items 32 R w .. 32 R (w + 1) - 1, 32 a round; the rank of an item among the
// equal digits of its warp is the warp's running count of that digit plus the
// equal lanes before it.
__global__ void __launch_bounds__(kSortThreads) embed_sort_small_kernel(const __grid_constant__ SortArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ uint32_t smem[];
    if (blockIdx.x > 0) {
        if (A.zero.present) find_present(A.ids, A.zero, blockIdx.x - 1, smem);
        write_zeros(A.zero, blockIdx.x - 1);
        return;
    }
    uint32_t* items = smem;                                                  // 8192
    uint16_t* hist = reinterpret_cast<uint16_t*>(smem + kSmallSort);         // [32][ndig]
    __shared__ uint32_t warp_sums[32];
    __shared__ uint32_t base[kMaxDigits];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int n = (int)A.ids.n, ndig = 1 << A.digit_bits;
    const int rounds = (n + kSortThreads - 1) / kSortThreads;
    const int per_warp = 32 * rounds, warps = n > 0 ? (n + per_warp - 1) / per_warp : 0;  // warps that have items
    uint32_t item[kSortItems];
    const int first = w * per_warp + lane;
    load_keys(A.ids, first, 32, min(n, (w + 1) * per_warp), 0u, item);
#pragma unroll
    for (int r = 0; r < kSortItems; ++r) {
        const int i = first + 32 * r;
        item[r] = r < rounds && i < n ? (item[r] << kPosBits) | (uint32_t)i : 0xffffffffu;
    }
    for (int p = 0; p < A.passes; ++p) {
        const int shift = kPosBits + p * A.digit_bits;
        for (int i = t; i < warps * ndig / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(hist)[i] = 0;
        __syncthreads();
        uint32_t rank[kSortItems];
#pragma unroll
        for (int r = 0; r < kSortItems; ++r) {
            if (r >= rounds || w >= warps) break;
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
#pragma unroll 8
            for (int q = 0; q < warps; ++q) {
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
            if (r >= rounds || w >= warps) break;
            const uint32_t d = (item[r] >> shift) & (ndig - 1);
            items[base[d] + hist[w * ndig + d] + rank[r]] = item[r];
        }
        __syncthreads();
        if (p + 1 < A.passes && w < warps) {
#pragma unroll
            for (int r = 0; r < kSortItems; ++r)
                if (r < rounds) item[r] = items[w * per_warp + 32 * r + lane];
        }
    }
    for (int i = t; i < n; i += kSortThreads) {
        A.keys[i] = (int32_t)(items[i] >> kPosBits);
        A.pos[i] = (int32_t)(items[i] & ((1u << kPosBits) - 1));
    }
}

struct TileArgs {
    Ids ids;
    const int32_t* kin;   // NULL: the first pass, keys from the ids
    const int32_t* pin;
    int32_t* kout;
    int32_t* pout;
    uint32_t* hist;       // [digits][tiles]: tokens of a digit in a tile; after the scan, in the tiles before it
    uint32_t* totals;     // [digits]
    uint32_t* present;    // a bit per row, cleared by the first histogram and set by the first scatter; NULL: not needed
    int32_t present_words;
    ZeroShare zero;       // blocks after the sort's write zeros
    int32_t shift, digit_bits, tiles, subtiles;  // a tile is `subtiles` runs of kTile tokens, ranked one after the other
};

// Keys of tokens first, first + stride, ... of the pass's input, `none` from `end` on.
template <int R>
__device__ __forceinline__ void tile_keys(const TileArgs& A, int64_t first, int64_t stride, int64_t end, uint32_t none,
                                          uint32_t (&key)[R]) {
    if (!A.kin) return load_keys(A.ids, first, stride, end, none, key);
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = first + r * stride < end ? (uint32_t)A.kin[first + r * stride] : none;
}

__global__ void __launch_bounds__(kTileThreads) embed_hist_kernel(const __grid_constant__ TileArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ uint32_t h[kMaxDigits];
    if ((int)blockIdx.x >= A.tiles) {
        write_zeros(A.zero, blockIdx.x - A.tiles);
        return;
    }
    const int ndig = 1 << A.digit_bits;
    for (int i = threadIdx.x; i < ndig; i += kTileThreads) h[i] = 0;
    if (!A.kin && A.present)
        for (int i = blockIdx.x * kTileThreads + threadIdx.x; i < A.present_words; i += A.tiles * kTileThreads)
            A.present[i] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * A.subtiles * kTile;
    const int64_t i1 = min(A.ids.n, i0 + (int64_t)A.subtiles * kTile);
    constexpr uint32_t none = 0xffffffffu;  // above every key
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kTile) {
        uint32_t key[kTile / kTileThreads];
        tile_keys(A, i, kTileThreads, i1, none, key);
#pragma unroll
        for (int k = 0; k < kTile / kTileThreads; ++k)
            if (key[k] != none) atomicAdd(&h[(key[k] >> A.shift) & (ndig - 1)], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ndig; i += kTileThreads) A.hist[(int64_t)i * A.tiles + blockIdx.x] = h[i];
}

// Per digit, a warp: exclusive sums over the tiles, and the total.
__global__ void __launch_bounds__(kTileThreads) embed_scan_kernel(const __grid_constant__ TileArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = kTileThreads / 32;
    const int ndig = 1 << A.digit_bits, blocks = (ndig + W - 1) / W;
    if ((int)blockIdx.x >= blocks) {
        write_zeros(A.zero, blockIdx.x - blocks);
        return;
    }
    const int d = blockIdx.x * W + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (d >= ndig) return;
    uint32_t* h = A.hist + (int64_t)d * A.tiles;
    uint32_t run = 0;
    for (int q0 = 0; q0 < A.tiles; q0 += 128) {
        uint32_t v[4], sum = 0;  // four tiles a lane, loaded side by side
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int q = q0 + 4 * lane + k;
            v[k] = q < A.tiles ? h[q] : 0u;
            sum += v[k];
        }
        uint32_t upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        uint32_t before = run + upto - sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int q = q0 + 4 * lane + k;
            if (q < A.tiles) h[q] = before;
            before += v[k];
        }
        run += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) A.totals[d] = run;
}

// rows of a table up to 32 times this are marked by way of shared memory (what is left of 48 KB)
constexpr int kMarkWords = 7168;

__global__ void __launch_bounds__(kTileThreads) embed_scatter_kernel(const __grid_constant__ TileArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = kTileThreads / 32, R = kTile / kTileThreads;
    constexpr int D = (kMaxDigits + kTileThreads - 1) / kTileThreads;  // digits a thread looks after
    extern __shared__ uint32_t marks[];  // kMarkWords, in the first pass of a table that they cover
    __shared__ __align__(16) uint16_t hist[W * kMaxDigits];
    __shared__ uint32_t base[kMaxDigits];
    __shared__ uint32_t warp_sums[32];
    static_assert(sizeof(hist) + sizeof(base) + sizeof(warp_sums) + 4 * kMarkWords <= 48 * 1024);
    if ((int)blockIdx.x >= A.tiles) {
        write_zeros(A.zero, blockIdx.x - A.tiles);
        return;
    }
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int ndig = 1 << A.digit_bits;
    const bool mark = !A.kin && A.present, shared_marks = mark && A.present_words <= kMarkWords;
    if (shared_marks)
        for (int i = t; i < A.present_words; i += kTileThreads) marks[i] = 0;
    // where this block's tokens of each digit begin: all smaller digits, and this digit in the tiles before.
    // Thread t looks after digits D t .. D t + D - 1.
    uint32_t own[D], sum = 0;
#pragma unroll
    for (int k = 0; k < D; ++k) {
        own[k] = D * t + k < ndig ? A.totals[D * t + k] : 0u;
        sum += own[k];
    }
    uint32_t excl = digit_scan<kTileThreads>(sum, warp_sums);
#pragma unroll
    for (int k = 0; k < D; ++k) {
        const int d = D * t + k;
        if (d < ndig) base[d] = excl + A.hist[(int64_t)d * A.tiles + blockIdx.x];
        excl += own[k];
    }
    for (int sub = 0; sub < A.subtiles; ++sub) {
        const int64_t i0 = ((int64_t)blockIdx.x * A.subtiles + sub) * kTile;
        if (i0 >= A.ids.n) break;
        for (int i = t; i < W * ndig / 2; i += kTileThreads) reinterpret_cast<uint32_t*>(hist)[i] = 0;
        __syncthreads();
        uint32_t key[R], rank[R];
        int32_t pos[R];
        const int64_t first = i0 + w * (32 * R) + lane;
        tile_keys(A, first, 32, A.ids.n, 0u, key);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = first + 32 * r;
            pos[r] = i >= A.ids.n ? -1 : A.pin ? A.pin[i] : (int32_t)i;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t d = (key[r] >> A.shift) & (ndig - 1);
            const uint32_t valid = __ballot_sync(0xffffffffu, pos[r] >= 0);
            const uint32_t peers = match_digit(d, A.digit_bits, valid);
            const uint32_t before = hist[w * ndig + d];
            rank[r] = before + __popc(peers & ((1u << lane) - 1));
            __syncwarp();
            if (pos[r] >= 0 && lane == __ffs(peers) - 1) hist[w * ndig + d] = (uint16_t)(before + __popc(peers));
            __syncwarp();
            if (mark && pos[r] >= 0 && key[r] < (uint32_t)A.ids.rows) {
                const uint32_t word = key[r] >> 5, bit = 1u << (key[r] & 31);
                if (shared_marks) atomicOr(&marks[word], bit);
                else if (MA_INB(word, 1, A.present_words, A.ids.status) &&
                         !(*reinterpret_cast<volatile uint32_t*>(&A.present[word]) & bit))
                    atomicOr(&A.present[word], bit);
            }
        }
        __syncthreads();
        uint32_t count[D];
#pragma unroll
        for (int k = 0; k < D; ++k) {
            const int d = D * t + k;
            count[k] = 0;
            if (d < ndig) {
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    const uint32_t c = hist[q * ndig + d];
                    hist[q * ndig + d] = (uint16_t)count[k];
                    count[k] += c;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (pos[r] < 0) continue;
            const uint32_t d = (key[r] >> A.shift) & (ndig - 1);
            const int64_t o = (int64_t)base[d] + hist[w * ndig + d] + rank[r];
            if (!MA_INB(o, 1, A.ids.n, A.ids.status)) continue;
            A.kout[o] = (int32_t)key[r];
            A.pout[o] = pos[r];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < D; ++k)
            if (D * t + k < ndig) base[D * t + k] += count[k];
    }
    if (shared_marks) {  // one atomic per word that a tile touches, however often a token repeats in it
        __syncthreads();
        for (int i = t; i < A.present_words; i += kTileThreads)
            if (marks[i]) atomicOr(&A.present[i], marks[i]);
    }
}

// ------------------------------------------------------------------ sums

struct SumArgs {
    const int32_t* keys;
    const int32_t* pos;
    const void* dy;
    void* grad;
    float* slots;       // per tile: its part of a long run that began before it, and of one that goes on after it
    int32_t* long_run;  // per tile: whether a long run begins in it
    int64_t n, rows, dim, ldy, ldg, slot_ld;
    int64_t fix_blocks;  // last kernel: blocks that add partial rows; those after them write zeros
    ZeroShare zero;      // sums: the first blocks write zeros
    int32_t tile, tiles, col_blocks, col_chunks, fix_tiles, accumulate;
    float scale;
    int* status;
};

// A row's elements of one thread, as loaded: converted when they are added, so
// that rows in flight take few registers.
template <bool BF16, int VEC>
struct Raw {
    static constexpr int kWords = (BF16 ? (VEC + 1) / 2 : VEC);
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if constexpr (BF16) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
            if constexpr (VEC == 2) {
                w[0] = __ldcs(reinterpret_cast<const uint32_t*>(q));
            } else {
                static_assert(VEC == 1);
                w[0] = __ldcs(q);
            }
        } else {
            const float* q = reinterpret_cast<const float*>(p) + i;
            if constexpr (VEC == 2) {
                const uint2 a = __ldcs(reinterpret_cast<const uint2*>(q));
                w[0] = a.x; w[1] = a.y;
            } else {
                static_assert(VEC == 1);
                w[0] = __float_as_uint(__ldcs(q));
            }
        }
    }
    __device__ __forceinline__ void put(int c, const uint4& v) {  // 16-byte piece c
        w[4 * c] = v.x;
        w[4 * c + 1] = v.y;
        w[4 * c + 2] = v.z;
        w[4 * c + 3] = v.w;
    }
    __device__ __forceinline__ void add_to(float (&acc)[VEC]) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if constexpr (BF16) acc[e] += (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
            else acc[e] += __uint_as_float(w[e]);
        }
    }
};

// A finished sum: scaled, added to the old value where asked, rounded once.
template <bool GB, int VEC>
__device__ __forceinline__ void write_row(const SumArgs& A, int32_t key, int64_t col, const float (&acc)[VEC]) {
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

// First index of sorted k[0..n) whose key is >= key.
__device__ __forceinline__ int lower_bound(const int32_t* k, int n, int32_t key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (k[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Vectors of a row that a thread of the sums takes: four where they are narrow,
// a row has over a thousand of them and the batch fills the GPU; the work per
// row and thread then counts more than the loads in flight. Measured with four
// (one): 1281 columns, 60,000 tokens 148 us (161), 8192 57 (66), 3000 36 (33),
// 301 22 (13: the larger code takes longer to arrive); 4095 columns, 8192 tokens
// 87 (118); 1282 columns, 641 vectors, 60,000 tokens 129 (109).
constexpr int sum_vectors(int vec, int64_t vecs, int64_t n) {
    return vec < 8 && vecs > 1024 && n * vecs > (1 << 22) ? 4 : 1;
}

template <bool YB, bool GB, int VEC, int K>
__global__ void __launch_bounds__(kSumThreads, 4) embed_sum_kernel(const __grid_constant__ SumArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kWin = kMaxSumTile + 2 * kLong;
    // Rows in flight: for vectors of 8, a ring of kRing 16-byte copies per thread in shared memory, four rows a
    // step (cp.async; no thread reads another's slots, so there is no barrier); else four or eight rows in
    // registers, of which a thread takes K narrow vectors each, blockDim apart.
    constexpr bool RING = VEC == 8;
    constexpr int U = RING || (K > 1 && Raw<YB, VEC>::kWords > 1) ? 4 : 8;
    constexpr int CPY = RING ? (YB ? 1 : 2) : 1;         // 16-byte copies per row
    constexpr int STEPS = RING ? kRing / (U * CPY) : 1;  // steps in the ring
    extern __shared__ uint4 ring[];
    __shared__ int32_t sk[kWin];  // keys from kLong before the tile to kLong after it, -1 and INT_MAX beyond the batch
    __shared__ int32_t sp[kMaxSumTile + kLong];
    if ((int)blockIdx.x < A.zero.blocks) {
        write_zeros(A.zero, blockIdx.x);
        return;
    }
    const uint32_t block = blockIdx.x - A.zero.blocks;
    const int tile = block / A.col_blocks;
    const int64_t i0 = (int64_t)tile * A.tile;
    int cnt = (int)min((int64_t)A.tile, A.n - i0);
    const int win = cnt + 2 * kLong;
    for (int q = threadIdx.x; q < win; q += blockDim.x) {
        const int64_t i = i0 - kLong + q;
        sk[q] = i < 0 ? -1 : i < A.n ? A.keys[i] : INT32_MAX;
        if (q >= kLong && i < A.n) sp[q - kLong] = A.pos[i];
    }
    __syncthreads();
    const int64_t col = ((int64_t)(block % A.col_blocks) * blockDim.x * K + threadIdx.x) * VEC;
    const int next = blockDim.x * VEC;  // columns between a thread's vectors
    // Tokens that add to no row are last; indexes below are relative to the tile.
    const int32_t rows = (int32_t)A.rows;
    const int32_t* tk = sk + kLong;
    cnt = min(cnt, lower_bound(sk, win, rows) - kLong);
    int begin = 0, end = cnt;
    bool head_long = false, tail_long = false;
    if (cnt > 0) {
        const int32_t key = tk[0];
        if (tk[-1] == key) {  // the first run began before the tile
            const int s = lower_bound(sk, win, key), e = lower_bound(sk, win, key + 1);
            head_long = e - s > kLong;
            if (!head_long) begin = min(cnt, e - kLong);  // summed where it began
        }
        const int32_t last = tk[cnt - 1];
        if (tk[cnt] == last && begin < cnt && (!head_long || last != key)) {  // the last run goes on after the tile
            const int s = lower_bound(sk, win, last), e = lower_bound(sk, win, last + 1);
            tail_long = e - s > kLong;
            if (!tail_long) end = e - kLong;
        }
    }
    if (block % A.col_blocks == 0 && threadIdx.x == 0) A.long_run[tile] = tail_long;
    if (col >= A.dim) return;
    float acc[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[k][e] = 0.f;
    bool head = head_long;
    uint4* slots = ring + threadIdx.x;
    auto fetch = [&](int b, int step) {  // rows b .. b + U - 1 into a step of the ring
        if constexpr (RING) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (b + u < end) {
                    const int64_t o = (int64_t)sp[b + u] * A.ldy + col;
                    if (MA_INB(o, VEC, (A.n - 1) * A.ldy + A.dim, A.status)) {
                        const uint8_t* src = reinterpret_cast<const uint8_t*>(A.dy) + o * (YB ? 2 : 4);
#pragma unroll
                        for (int c = 0; c < CPY; ++c)
                            cp_async16(slots + ((step * U + u) * CPY + c) * blockDim.x, src + 16 * c);
                    }
                }
            }
            cp_async_commit();  // a group per step, empty or not, so that the counts line up
        }
    };
    int step = 0, ahead = 0;
    if constexpr (RING) {
#pragma unroll
        for (int q = 0; q < STEPS - 1; ++q) fetch(begin + q * U, q);
        ahead = STEPS - 1;
    }
    for (int b = begin; b < end; b += U) {
        Raw<YB, VEC> f[U][K];
        if constexpr (RING) {
            fetch(b + (STEPS - 1) * U, ahead);
            ahead = ahead + 1 == STEPS ? 0 : ahead + 1;
            cp_async_wait<STEPS - 1>();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < CPY; ++c) f[u][0].put(c, slots[((step * U + u) * CPY + c) * blockDim.x]);
            step = step + 1 == STEPS ? 0 : step + 1;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (b + u < end) {
                    const int64_t o = (int64_t)sp[b + u] * A.ldy + col;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (col + k * next < A.dim &&
                            MA_INB(o + k * next, VEC, (A.n - 1) * A.ldy + A.dim, A.status))
                            f[u][k].load(A.dy, o + k * next);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = b + u;
            if (i >= end) break;
#pragma unroll
            for (int k = 0; k < K; ++k) f[u][k].add_to(acc[k]);
            const int32_t key = tk[i];
            if (i + 1 < end && tk[i + 1] == key) continue;
            const bool tail = tail_long && i + 1 == end;
            float* slot = A.slots + (2 * (int64_t)tile + (head ? 0 : 1)) * A.slot_ld + col;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (k > 0 && col + k * next >= A.dim) break;
                if (head || tail) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) slot[k * next + e] = acc[k][e];
                } else {
                    write_row<GB, VEC>(A, key, col + k * next, acc[k]);
                }
            }
            head = false;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[k][e] = 0.f;
        }
    }
    if constexpr (RING) cp_async_wait<0>();
}

// The partial rows of long runs: that of the tile it begins in, then those of
// the tiles it goes on through, in that order. A block takes 32 * CV columns
// and the long runs that begin in up to kFixTiles tiles: each warp adds up runs of up
// to kShortRun more tiles by itself; of the others, afterwards, every warp adds
// a contiguous share, and the shares are added in order.
constexpr int kFixTiles = 32;
constexpr int kShortRun = 8;

template <bool GB, int CV>
__global__ void __launch_bounds__(kFixThreads, 5) embed_fix_kernel(const __grid_constant__ SumArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = kFixThreads / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if ((int64_t)blockIdx.x >= A.fix_blocks) {
        write_zeros(A.zero, blockIdx.x - A.fix_blocks);
        return;
    }
    __shared__ float part[W][32 * CV];
    const int64_t col = ((int64_t)(blockIdx.x % A.col_chunks) * 32 + lane) * CV;
    const bool in = col < A.dim;
    const int64_t g0 = (int64_t)(blockIdx.x / A.col_chunks) * A.fix_tiles;
    auto key_of = [&](int64_t t0) { return A.keys[(t0 + 1) * A.tile]; };
    // whether the run that goes on after tile t0 also covers the first token of tile t0 + 1 + more
    auto reaches = [&](int64_t t0, int64_t more, int32_t key) {
        const int64_t q = t0 + 1 + more;
        return q < A.tiles && A.keys[q * A.tile] == key;
    };
    auto add = [&](int64_t t0, int64_t lo, int64_t hi, float (&acc)[CV]) {  // tiles t0 + 1 + lo .. t0 + hi
        constexpr int R = 16 / CV;  // rows in flight
        for (int64_t q = lo; q < hi; q += R) {
            float f[R][CV];
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (q + r < hi) load_vec<false, CV>(A.slots, 2 * (t0 + 1 + q + r) * A.slot_ld + col, f[r]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (q + r >= hi) break;
#pragma unroll
                for (int e = 0; e < CV; ++e) acc[e] += f[r][e];
            }
        }
    };
    uint32_t todo = __ballot_sync(0xffffffffu, lane < A.fix_tiles && g0 + lane < A.tiles && A.long_run[g0 + lane]);
    // Every warp looks at every run (only those it adds up cost it more): bit k of `many`: the run that begins in
    // tile k goes on through more than kShortRun tiles.
    const bool mine = todo >> lane & 1u;
    uint32_t many = __ballot_sync(0xffffffffu, mine && reaches(g0 + lane, kShortRun, key_of(g0 + lane)));
    int turn = 0;
    for (uint32_t few = todo & ~many; few; few &= few - 1, ++turn) {
        if (turn % W != w) continue;
        const int64_t t0 = g0 + __ffs(few) - 1;
        const int32_t key = key_of(t0);
        const int m = __popc(__ballot_sync(0xffffffffu, lane < kShortRun && reaches(t0, lane, key)));
        if (!in) continue;
        float acc[CV];
        load_vec<false, CV>(A.slots, (2 * t0 + 1) * A.slot_ld + col, acc);
        add(t0, 0, m, acc);
        write_row<GB, CV>(A, key, col, acc);
    }
    for (; many; many &= many - 1) {
        const int64_t t0 = g0 + __ffs(many) - 1;
        const int32_t key = key_of(t0);
        int64_t lo = kShortRun, hi = A.tiles - (t0 + 1);  // the run reaches lo more tiles, and not hi more
        while (hi - lo > 1) {  // 32 probes a step
            const int64_t width = (hi - lo + 32) / 33, probe = lo + width * (lane + 1);
            const uint32_t yes = __ballot_sync(0xffffffffu, probe < hi && reaches(t0, probe, key));
            const int n = __popc(yes);  // the first n probes are reached
            hi = min(hi, lo + width * (n + 1));
            lo += width * n;
        }
        const int64_t m = lo + 1;  // tiles that it goes on through
        float acc[CV];
#pragma unroll
        for (int e = 0; e < CV; ++e) acc[e] = 0.f;
        if (in) {
            if (w == 0) load_vec<false, CV>(A.slots, (2 * t0 + 1) * A.slot_ld + col, acc);
            add(t0, m * w / W, m * (w + 1) / W, acc);
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

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    Ids ids;
    const void* table;
    void* out;
    int64_t dim, ldt, ldo;
    float scale;
    int32_t lanes;  // threads per token row, of the block's 256
};

constexpr int kLookupThreads = 256;

constexpr int kLookupLoads = 4;  // in flight per thread

template <bool TB, bool OB, int VEC, int TOKENS>
__global__ void __launch_bounds__(kLookupThreads, 4) embed_lookup_kernel(const __grid_constant__ LookupArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    const int lanes = A.lanes, groups = kLookupThreads / lanes;
    const int group = threadIdx.x / lanes, t = threadIdx.x - group * lanes;
    if (group == groups) return;
    // this thread's rows: T of them, `groups` apart; their ids before anything depends on one
    constexpr int T = TOKENS, U = kLookupLoads / TOKENS;
    const int64_t i0 = (int64_t)blockIdx.x * groups * T + group;
    int64_t id[T];
    bool in[T], real[T];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const int64_t i = i0 + k * groups;
        real[k] = i < A.ids.n && MA_INB(i, 1, A.ids.n, A.ids.status);
        id[k] = !real[k]    ? 0
                : A.ids.i64 ? reinterpret_cast<const int64_t*>(A.ids.p)[i]
                            : reinterpret_cast<const int32_t*>(A.ids.p)[i];
    }
#pragma unroll
    for (int k = 0; k < T; ++k) {
        in[k] = real[k] && id[k] >= 0 && id[k] < A.ids.rows;
        if (real[k] && !in[k] && id[k] != A.ids.padding && t == 0) record_error(A.ids.status, MA_ERR_BOUNDS);
    }
    const int dim = (int)A.dim, step = lanes * VEC;
    for (int c0 = t * VEC; c0 < dim; c0 += U * step) {
        float f[T][U][VEC];
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * step;
                if (in[k] && c < dim &&
                    MA_INB(id[k] * A.ldt + c, VEC, (A.ids.rows - 1) * A.ldt + A.dim, A.ids.status))
                    load_vec<TB, VEC>(A.table, id[k] * A.ldt + c, f[k][u]);
            }
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * step;
                const int64_t i = i0 + k * groups;
                if (!real[k] || c >= dim) continue;
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[k][u][e] = in[k] ? f[k][u][e] * A.scale : 0.f;
                if (MA_INB(i * A.ldo + c, VEC, (A.ids.n - 1) * A.ldo + A.dim, A.ids.status))
                    store_vec<OB, VEC>(A.out, i * A.ldo + c, f[k][u]);
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
    int64_t sum_tiles, slot_ld;
    size_t off_k0, off_p0, off_k1, off_p1, off_hist, off_present, off_long, off_slots, total;
};

// Tokens per tile of the sum, from 512 down to 8: the longest that still gives
// each of 148 SMs six blocks and sixteen warps (a longer tile searches less and
// leaves fewer partial rows; too few leave SMs without loads in flight), and
// twice that above 64 tokens, where a block lasts long and a last round of few
// blocks would too. Against tiles of at most 64: 131,072 tokens x 1280 bf16 of a
// skewed distribution 135 us (169), all the same token 161 (222); 1,000,000 x
// 128 skewed 162 (193), all the same token 301 (901). Sixteen warps, against six
// blocks alone: 20,000 x 64 skewed 35.5 (38.7), 1,000,000 x 128 162 (185), all
// the same token 301 (176). (148 as a constant: the workspace, whose size is
// asked for without a device, depends on the tile.)
int sum_tile(int64_t n, int64_t dim) {
    const int64_t warps = (dim + 255) / 256, blocks = (warps + 7) / 8;  // of a row, 8 elements to a thread
    int s = kMaxSumTile;
    auto fills = [&](int64_t tiles, int sms) { return tiles * blocks >= 6 * sms && tiles * warps >= 16 * sms; };
    while (s > 8 && !fills((n + s - 1) / s, s > 64 ? 2 * 148 : 148)) s /= 2;
    return s;
}

GradLayout grad_layout(int64_t n, int64_t rows, int64_t dim) {
    GradLayout L;
    std::memset(&L, 0, sizeof(L));
    const int bits = bits_for(rows);
    L.small = n == 0 || (n <= kSmallSort && bits <= kSmallKeyBits);
    L.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    L.digit_bits = (bits + L.passes - 1) / L.passes;
    L.tiles = (int)((n + kTile - 1) / kTile);
    L.subtiles = (L.tiles + kMaxTiles - 1) / kMaxTiles;
    if (L.subtiles > 1) L.tiles = (L.tiles + L.subtiles - 1) / L.subtiles;
    L.subtiles = std::max(1, L.subtiles);
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
    L.off_hist = take(L.small ? 0 : (size_t)(L.tiles + 1) * kMaxDigits * 4);  // the totals after the tiles
    L.off_present = take(((size_t)rows + 31) / 32 * 4);
    L.off_long = take((size_t)L.sum_tiles * 4);
    L.off_slots = take((size_t)L.sum_tiles * 2 * L.slot_ld * 4);
    L.total = off;
    return L;
}

constexpr size_t kSmallSortSmem = (size_t)kSmallSort * 4 + 32 * kMaxDigits * 2;

cudaError_t launch_sort_small(const SortArgs& A, unsigned grid, cudaStream_t s) {
    static PerDevice<int> cache;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cache.get(dev, &done, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(embed_sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kSmallSortSmem);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(embed_sort_small_kernel, dim3(grid), dim3(kSortThreads), kSmallSortSmem, s, A);
}

template <bool YB, bool GB, int VEC, int K>
cudaError_t launch_sum(const SumArgs& A, unsigned grid, unsigned threads, cudaStream_t s) {
    const size_t ring = VEC == 8 ? (size_t)threads * kRing * 16 : 0;
    static PerDevice<int> cache;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cache.get(dev, &done, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(embed_sum_kernel<YB, GB, VEC, K>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSumThreads * kRing * 16);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(embed_sum_kernel<YB, GB, VEC, K>, dim3(grid), dim3(threads), ring, s, A);
}

// The parts of the zeros that the kernels write, in order: while the tokens are
// sorted, beside the sums, and beside the last kernel. Beside the sort by tiles
// (what comes after its first scatter) and the last kernel go as many bytes as
// HBM takes in their time; beside the one-block sort more, since its launch has
// the GPU but for one SM, and the sums have loads to wait for: 8192 tokens x 4096
// into 32,000 rows 72.5 us (77.5 with 60 MB there), 1000 tokens 60.5 (65.3).
// 32,768 tokens by tiles: 122.5 (125.7 with 105 MB).
struct ZeroPlan {
    ZeroShare z;
    int64_t cut[4];  // rows of each part: [cut[0], cut[1]) by the first kernels, ...
    ZeroShare part(int k) const {
        ZeroShare s = z;
        s.lo = cut[k];
        s.hi = cut[k + 1];
        if (s.hi <= s.lo) s.blocks = 0;
        return s;
    }
    ZeroShare part(int k, int of, int i) const {  // slice i of `of` of part k
        ZeroShare s = part(k);
        const int64_t len = cut[k + 1] - cut[k];
        s.lo = cut[k] + len * i / of;
        s.hi = cut[k] + len * (i + 1) / of;
        if (s.hi <= s.lo) s.blocks = 0;
        return s;
    }
};
constexpr double kSmallSortHides = 110e6, kTileSortHides = 60e6, kLastHides = 30e6;

ZeroPlan plan_zeros(void* grad, int64_t rows, int64_t dim, int64_t ldg, int gsz, uint32_t* present, bool none,
                    double sort_hides, int sms) {
    ZeroPlan P;
    std::memset(&P, 0, sizeof(P));
    ZeroShare& z = P.z;
    z.grad = reinterpret_cast<uint8_t*>(grad);
    z.present = present;
    z.rows = rows;
    z.row_bytes = dim * gsz;
    z.ld_bytes = ldg * gsz;
    z.status = device_status_ptr();
    if (none) return P;
    z.aligned = (reinterpret_cast<uintptr_t>(grad) | (uint64_t)z.row_bytes | (uint64_t)z.ld_bytes) % 16 == 0;
    // two parts per SM, in whole words of the bit map, no more rows than the one-block sort's kernel has bits for
    z.period = ((rows + 2 * sms - 1) / (2 * sms) + 31) / 32 * 32;
    z.period = std::min<int64_t>(z.period, (int64_t)kSmallSortSmem * 8);
    z.blocks = (int32_t)((rows + z.period - 1) / z.period);
    const double bytes = (double)rows * z.row_bytes;
    const int64_t first = (int64_t)std::min((double)z.period, std::ceil(z.period * sort_hides / bytes));
    const int64_t last = (int64_t)std::min((double)(z.period - first), std::ceil(z.period * kLastHides / bytes));
    P.cut[0] = 0;
    P.cut[1] = first;
    P.cut[2] = z.period - last;
    P.cut[3] = z.period;
    return P;
}

// f(vector width as a constant) for rows that take vectors of 8, 2 or 1 elements
template <typename F>
cudaError_t with_vec(int vec, F f) {
    return vec == 8   ? f(std::integral_constant<int, 8>{})
           : vec == 2 ? f(std::integral_constant<int, 2>{})
                      : f(std::integral_constant<int, 1>{});
}
// f(constants: whether each of two types is bf16)
template <typename F>
cudaError_t with_types(int a, int b, F f) {
    using T = std::true_type;
    using N = std::false_type;
    if (a == MA_BF16) return b == MA_BF16 ? f(T{}, T{}) : f(T{}, N{});
    return b == MA_BF16 ? f(N{}, T{}) : f(N{}, N{});
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
    // Two tokens a thread where the batch fills the GPU either way: half of a thread's loads from each row, so that a
    // row of 4096 bf16 takes a block's threads once.
    // bf16, two against one: 131,072 tokens x 1280 124 us (306), 8192 x 4096 26.1 (32.5), 2048 x 4096 5.9 (7.2); 1024 x
    // 4096, below the rule, 4.8 (4.8). What bounds it then is HBM: 8192 x 4096 distinct rows move 134 MB, 5.1 TB/s.
    // Rows that are not whole vectors go by two elements or one: 131,072 uniform tokens of 65,536 rows, 1282 columns
    // 260 us and 1281 303, 1280 131 (each after a write of 256 MB). (148: the SMs this library is built for.)
    const int64_t vecs = dim / vec, each = kLookupLoads / 2;
    const bool two = n * std::min<int64_t>(vecs, kLookupThreads) >= (int64_t)2048 * 148;
    A.lanes = (int)std::min<int64_t>(kLookupThreads, two ? (vecs + each - 1) / each : vecs);
    const int64_t per_block = (int64_t)(two ? 2 : 1) * (kLookupThreads / A.lanes);
    const dim3 grid((unsigned)((n + per_block - 1) / per_block)), block(kLookupThreads);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int pr = prof_begin(MA_PROF_EMBED, s);
    const cudaError_t e = with_vec(vec, [&](auto v) {
        return with_types(tdt, odt, [&](auto tb, auto ob) {
            constexpr bool TB = decltype(tb)::value, OB = decltype(ob)::value;
            constexpr int V = decltype(v)::value;
            return two ? launch_pdl(embed_lookup_kernel<TB, OB, V, 2>, grid, block, 0, s, A)
                       : launch_pdl(embed_lookup_kernel<TB, OB, V, 1>, grid, block, 0, s, A);
        });
    });
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
    auto at_i = [&](size_t off) { return reinterpret_cast<int32_t*>(base + off); };
    const int ysz = ydt == MA_BF16 ? 2 : 4, gsz = gdt == MA_BF16 ? 2 : 4;
    int vec = 1;
    for (int v : {8, 2})
        if (vec == 1 && rows_take(dY, dim, ldy, ysz, v) && rows_take(g, dim, ldg, gsz, v)) vec = v;
    SumArgs S;
    std::memset(&S, 0, sizeof(S));
    S.dy = dY;
    S.grad = g;
    S.n = n;
    S.rows = rows;
    S.dim = dim;
    S.ldy = ldy;
    S.ldg = ldg;
    S.slot_ld = L.slot_ld;
    S.scale = scale;
    S.accumulate = accumulate;
    S.status = device_status_ptr();
    S.tile = L.sum_tile;
    S.tiles = (int)L.sum_tiles;
    // as few blocks of up to 256 threads across the columns as hold a row's vectors, `each` to a thread
    const int each = sum_vectors(vec, dim / vec, n);
    const int64_t lanes = (dim / vec + each - 1) / each;
    S.col_blocks = (int)((lanes + kSumThreads - 1) / kSumThreads);
    const unsigned threads = (unsigned)((lanes + S.col_blocks - 1) / S.col_blocks + 31) / 32 * 32;
    const int cv = std::min(vec, 4);
    S.col_chunks = (int)((dim + 32 * cv - 1) / (32 * cv));
    // tiles whose long runs a block of the last kernel adds up: fewer where there would be less than a block per SM
    // (100,000 tokens x 5: 43 us, 50 with 32 tiles a block)
    S.fix_tiles = kFixTiles;
    while (S.fix_tiles > kFixThreads / 32 && (S.tiles + S.fix_tiles - 1) / S.fix_tiles * (int64_t)S.col_chunks < sms)
        S.fix_tiles /= 2;
    // a batch of up to kLong tokens has no run to cut and no last kernel (16 tokens x 514: 9.7 us, 10.9 with it)
    const bool whole = n <= kLong;
    S.fix_blocks = S.tiles > 1 && !whole ? (int64_t)((S.tiles + S.fix_tiles - 1) / S.fix_tiles) * S.col_chunks : 0;
    uint32_t* present = n > 0 ? at32(L.off_present) : nullptr;
    const ZeroPlan zeros = plan_zeros(g, rows, dim, ldg, gsz, present, accumulate != 0,
                                      L.small ? kSmallSortHides : kTileSortHides, sms);
    if ((int64_t)S.tiles * S.col_blocks + zeros.z.blocks > INT32_MAX || S.fix_blocks + zeros.z.blocks > INT32_MAX)
        return MA_ERR_UNSUPPORTED;
    if (n > 0) {
        S.slots = reinterpret_cast<float*>(base + L.off_slots);
        S.long_run = at_i(L.off_long);
    }
    const int pr = prof_begin(MA_PROF_EMBED, s);
    cudaError_t e = cudaSuccess;
    if (L.small) {
        SortArgs A;
        std::memset(&A, 0, sizeof(A));
        A.ids = I;
        A.keys = at_i(L.off_k0);
        A.pos = at_i(L.off_p0);
        A.digit_bits = L.digit_bits;
        A.passes = L.passes;
        A.zero = zeros.part(0);
        if (n == 0) A.zero.hi = zeros.z.period;  // nothing else runs
        else A.zero.blocks = zeros.z.blocks;     // every part's rows are looked at, whatever its share
        e = launch_sort_small(A, (unsigned)(A.zero.blocks + 1), s);
        S.keys = A.keys;
        S.pos = A.pos;
    } else {
        TileArgs A;
        std::memset(&A, 0, sizeof(A));
        A.ids = I;
        A.hist = at32(L.off_hist);
        A.totals = A.hist + (size_t)L.tiles * kMaxDigits;
        A.present = accumulate ? nullptr : present;
        A.present_words = (int32_t)((rows + 31) / 32);
        const int scan_blocks = ((1 << L.digit_bits) + kTileThreads / 32 - 1) / (kTileThreads / 32);
        A.digit_bits = L.digit_bits;
        A.tiles = L.tiles;
        A.subtiles = L.subtiles;
        const int after = 3 * (L.passes - 1);  // launches after the first scatter: a share of the zeros beside each
        auto share = [&](int launch) {
            if (launch >= 3) A.zero = zeros.part(0, after, launch - 3);
            return A.zero.blocks;
        };
        for (int p = 0; p < L.passes && e == cudaSuccess; ++p) {
            const bool odd = p & 1;
            A.kout = at_i(odd ? L.off_k1 : L.off_k0);
            A.pout = at_i(odd ? L.off_p1 : L.off_p0);
            A.shift = p * L.digit_bits;
            const dim3 threads(kTileThreads);
            const int z0 = share(3 * p);
            e = launch_pdl(embed_hist_kernel, dim3(L.tiles + z0), threads, 0, s, A);
            const int z1 = share(3 * p + 1);
            if (e == cudaSuccess) e = launch_pdl(embed_scan_kernel, dim3(scan_blocks + z1), threads, 0, s, A);
            const int z2 = share(3 * p + 2);
            const size_t marks = p == 0 && A.present && A.present_words <= kMarkWords ? A.present_words * 4 : 0;
            if (e == cudaSuccess) e = launch_pdl(embed_scatter_kernel, dim3(L.tiles + z2), threads, marks, s, A);
            A.kin = A.kout;
            A.pin = A.pout;
        }
        S.keys = A.kin;
        S.pos = A.pin;
    }
    if (e == cudaSuccess && n > 0) {
        S.zero = zeros.part(1);
        if (whole && zeros.z.blocks > 0) {  // the last kernel's share as well
            S.zero = zeros.z;
            S.zero.lo = zeros.cut[1];
            S.zero.hi = zeros.cut[3];
        }
        // a table of one digit is sorted by its first pass: no launch was left to hide zeros beside
        if (!L.small && L.passes == 1) S.zero.lo = 0, S.zero.blocks = zeros.z.blocks;
        const unsigned grid = (unsigned)(S.zero.blocks + S.tiles * S.col_blocks);
        e = with_vec(vec, [&](auto v) {
            return with_types(ydt, gdt, [&](auto yb, auto gb) {
                constexpr bool YB = decltype(yb)::value, GB = decltype(gb)::value;
                constexpr int V = decltype(v)::value;
                if constexpr (V < 8)
                    if (each == 4) return launch_sum<YB, GB, V, 4>(S, grid, threads, s);
                return launch_sum<YB, GB, V, 1>(S, grid, threads, s);
            });
        });
        S.zero = zeros.part(2);
        if (e == cudaSuccess && !whole && S.fix_blocks + S.zero.blocks > 0)
            e = with_vec(vec, [&](auto v) {
                constexpr int CV = decltype(v)::value < 4 ? decltype(v)::value : 4;
                const dim3 g2((unsigned)(S.fix_blocks + S.zero.blocks)), b2(kFixThreads);
                return gdt == MA_BF16 ? launch_pdl(embed_fix_kernel<true, CV>, g2, b2, 0, s, S)
                                      : launch_pdl(embed_fix_kernel<false, CV>, g2, b2, 0, s, S);
            });
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
