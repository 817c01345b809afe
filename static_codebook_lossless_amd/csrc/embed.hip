// Embedding lookup, and the table's gradient by sorted tokens.
//
// Both are bound by HBM.  Measured: 32768 rows of 4096 out of an int8 table of
// 32000 into bf16 53 us (306 MB); the gradient of 32768 x 4096 bf16 to a table of
// 32000 in f32, tokens by 1/rank, 192 us (793 MB): sort 29, sums and zeros 138-151,
// join 11; of 2048 x 1000 bf16 to a table of 4001 17 us (7, 6 and 4 on the
// device); of 511 x 1000 f32 9 us in one launch, 7.4-8.7 of them on the device.
// Narrow rows to a small table are bound by the sort, whose workgroups are the
// ranges of the table: 65536 x 64 to 256 rows takes 79 us.
#include <algorithm>
#include <type_traits>

#include "q8.h"

namespace pc {
namespace {

constexpr uint32_t kThreads = 256;

// ---------------------------------------------------------------------------
// lookup: out[t] = scale * table[token[t]]
// ---------------------------------------------------------------------------

constexpr uint32_t kPerLane = 4;
constexpr uint32_t kTile = kThreads * kPerLane;

template <typename TOK>
__device__ __forceinline__ int64_t token_at(const void *tokens, uint64_t i) {
    return (int64_t)static_cast<const TOK *>(tokens)[i];
}

// TABLE: a pc_dtype, or 4 + a pc_q8_format for a stored table.
template <int TABLE, int ODT, typename TOK>
__global__ __launch_bounds__(kThreads) void embed_kernel(const void *__restrict__ tokens,
                                                         const void *__restrict__ table,
                                                         const uint8_t *__restrict__ codes, uint64_t vocab,
                                                         uint64_t ld_table, uint64_t ld_codes, Units units,
                                                         float scale, typename Plain<ODT>::type *__restrict__ out,
                                                         uint64_t ld_out, uint32_t *__restrict__ status) {
    const uint64_t base = (uint64_t)blockIdx.x * kTile;
    uint64_t row[kPerLane], col[kPerLane];
    uint32_t n[kPerLane];
    int64_t tok[kPerLane];
    float v[kPerLane][8], by[kPerLane];
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        const uint32_t local = j * kThreads + threadIdx.x;
        n[j] = 0;
        if (base + local < units.total) {
            find_unit(units, base, local, row[j], col[j]);
            n[j] = count_before(units.cols, col[j], kUnit);
            tok[j] = token_at<TOK>(tokens, row[j]);
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        if (!n[j]) continue;
        by[j] = scale;
        if (tok[j] < 0 || (uint64_t)tok[j] >= vocab) {
            by[j] = 1.0f;  // zeros whatever the scale
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            if (status && col[j] == 0) *status = PC_ERR_INVALID_ARG;
        } else if constexpr (TABLE < 4) {
            load_unit<TABLE>(static_cast<const typename Plain<TABLE>::type *>(table) + (uint64_t)tok[j] * ld_table +
                                 col[j], n[j], v[j]);
        } else {
            const u32x2 w = load_symbols(static_cast<const uint8_t *>(table) + (uint64_t)tok[j] * ld_table + col[j],
                                         n[j]);
            unit_values<TABLE - 4>(w, scale_of(codes[(uint64_t)tok[j] * ld_codes + col[j] / kGroup]), v[j]);
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        if (!n[j]) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] *= by[j];
        store_unit<ODT>(out + row[j] * ld_out + col[j], n[j], v[j]);
    }
}

// ---------------------------------------------------------------------------
// gradient: sort the tokens, sum the rows of dy in that order
// ---------------------------------------------------------------------------

// A wave holds a slab of 512 columns of a row, a lane 4 of either half of it:
// every load and store of the wave is then one piece of memory without gaps,
// in each of the types.
constexpr uint32_t kSlab = 512;
constexpr uint32_t kAhead = 8;  // rows of dy in flight in a lane

// WHOLE: the width is a multiple of 4.
template <bool WHOLE> struct Columns {
    uint64_t first[2], last;  // the lane's first column of either four; the row's last
    uint32_t n[2];            // how many of each four are inside
    __device__ __forceinline__ Columns(uint64_t slab, uint32_t lane, uint64_t dim) : last(dim - 1) {
#pragma unroll
        for (uint32_t q = 0; q < 2; ++q) {
            first[q] = slab * kSlab + q * 256 + lane * 4;
            n[q] = count_before(dim, first[q], 4);
        }
    }
};

typedef u32x2 u32x2_any2 __attribute__((aligned(2)));

// Loads without branches, so that those of several rows are in flight
// together: columns outside are read at the row's end instead, for nothing.
template <int DT, bool WHOLE>
__device__ __forceinline__ void load_columns(const typename Plain<DT>::type *row, const Columns<WHOLE> &c,
                                             float v[8]) {
#pragma unroll
    for (uint32_t q = 0; q < 2; ++q) {
        float *x = v + 4 * q;
        if constexpr (!WHOLE) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) x[i] = widen(row[min(c.first[q] + i, c.last)]);
        } else if constexpr (DT == PC_F32) {
            const u32x4 a = *reinterpret_cast<const u32x4_any4 *>(row + min(c.first[q], c.last - 3));
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = as_f32(a[i]);
        } else {
            const u32x2 a = *reinterpret_cast<const u32x2_any2 *>(row + min(c.first[q], c.last - 3));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u = a[i];
                if constexpr (DT == PC_BF16) {
                    x[2 * i] = as_f32(u << 16);
                    x[2 * i + 1] = as_f32(u & 0xFFFF0000u);
                } else {
                    const f16x2 h = __builtin_bit_cast(f16x2, u);
                    x[2 * i] = (float)h[0];
                    x[2 * i + 1] = (float)h[1];
                }
            }
        }
    }
}

// Holds the rows loaded so far apart from their use, which the compiler would
// otherwise bring together again, one row at a time.
__device__ __forceinline__ void loaded(float v[kAhead][8]) {
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k)
        asm volatile("" : "+v"(v[k][0]), "+v"(v[k][1]), "+v"(v[k][2]), "+v"(v[k][3]), "+v"(v[k][4]), "+v"(v[k][5]),
                     "+v"(v[k][6]), "+v"(v[k][7]));
}

template <int DT, bool STREAM, bool WHOLE>
__device__ __forceinline__ void store_columns(typename Plain<DT>::type *row, const Columns<WHOLE> &c,
                                              const float v[8]) {
    typedef typename Plain<DT>::type T;
    typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (uint32_t q = 0; q < 2; ++q) {
        T *p = row + c.first[q];
        const float *x = v + 4 * q;
        if (c.n[q] == 4) {
            const f32x4 f = {x[0], x[1], x[2], x[3]};
            put<sizeof(T), STREAM>(p, __builtin_convertvector(f, t4));
        } else if (!WHOLE) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                if (i < c.n[q]) p[i] = (T)x[i];
        }
    }
}

struct Target {  // of a row's sum
    float scale;
    uint32_t add;
};

template <int ODT, bool WHOLE>
__device__ __forceinline__ void put_row(typename Plain<ODT>::type *row, const Columns<WHOLE> &c, const float v[8],
                                        const Target &to) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = v[i] * to.scale;
    if (to.add) {
        float old[8];
        load_columns<ODT>(row, c, old);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += old[i];
    }
    store_columns<ODT, true>(row, c, s);
}

// Few tokens: one launch.  A workgroup owns a range of the table's rows and a
// slab of columns.  It reads all tokens, keeps those of its range in LDS (in
// order, with their places), and its waves sum the rows one by one; a row
// with many tokens is summed by all waves, a share of its tokens each.  Rows
// without tokens become zero in passing.
constexpr uint32_t kSmall = 512;         // tokens
constexpr uint32_t kSmallThreads = 256;
constexpr uint32_t kSmallWaves = kSmallThreads / kWave;
constexpr uint32_t kMany = 32;           // tokens of a row that are shared among the waves

template <int DT, int ODT, typename TOK, bool WHOLE>
__global__ __launch_bounds__(kSmallThreads) void small_kernel(const void *__restrict__ tokens, uint32_t n,
                                                              const typename Plain<DT>::type *__restrict__ dy,
                                                              uint64_t ld_dy, uint64_t vocab, uint64_t dim,
                                                              int64_t padding, uint32_t range, Target to,
                                                              typename Plain<ODT>::type *__restrict__ grad,
                                                              uint64_t ld_grad) {
    __shared__ uint32_t key[kSmall], place[kSmall];
    __shared__ uint32_t sums[kSmallWaves];
    __shared__ float part[kSmallWaves][kUnit][kWave];
    const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const uint64_t lo = (uint64_t)blockIdx.x * range;
    const uint32_t size = (uint32_t)min((uint64_t)range, vocab - lo);
    // each wave a consecutive part of the tokens, up to 2 in a lane
    constexpr uint32_t kEach = kSmall / kSmallThreads;
    const uint32_t per = (n + kSmallThreads - 1) / kSmallThreads * kWave;
    uint32_t mine[kEach];
    uint64_t found[kEach];
    uint32_t total = 0;
#pragma unroll
    for (uint32_t j = 0; j < kEach; ++j) {
        const uint32_t at = j * kWave + lane, i = wave * per + at;
        mine[j] = ~0u;
        if (at < per && i < n) {
            const int64_t t = token_at<TOK>(tokens, i);
            if (t >= 0 && t != padding && (uint64_t)t >= lo && (uint64_t)t - lo < size) mine[j] = (uint32_t)(t - lo);
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < kEach; ++j) {
        found[j] = __ballot(mine[j] != ~0u);
        total += __popcll(found[j]);
    }
    if (lane == 0) sums[wave] = total;
    __syncthreads();
    uint32_t at = 0, count = 0;
#pragma unroll
    for (uint32_t w = 0; w < kSmallWaves; ++w) {
        if (w < wave) at += sums[w];
        count += sums[w];
    }
    count = uniform(count);
#pragma unroll
    for (uint32_t j = 0; j < kEach; ++j) {
        if (mine[j] != ~0u) {
            const uint32_t p = at + __popcll(found[j] & ((1ull << lane) - 1));
            key[p] = mine[j];
            place[p] = wave * per + j * kWave + lane;
        }
        at += __popcll(found[j]);
    }
    __syncthreads();

    const Columns<WHOLE> cols(blockIdx.y, lane, dim);
    // sums row r over the list's groups of 64 entries first, first + step, ...
    auto sum = [&](uint32_t r, uint32_t first, uint32_t step, float acc[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        for (uint32_t g = first * kWave; g < count; g += step * kWave) {
            const uint32_t e = g + lane;
            const bool is = e < count && key[e] == r;
            const uint32_t where = is ? place[e] : 0;
            uint64_t left = __ballot(is);
            while (left) {
                float v[kAhead][8];
                uint32_t from = 0;
                auto next = [&](uint32_t k) {
                    from = left ? (uint32_t)__builtin_ctzll(left) : from;
                    left &= left - 1;
                    const uint64_t t = (uint32_t)__builtin_amdgcn_readlane((int)where, (int)from);
                    load_columns<DT>(dy + t * ld_dy, cols, v[k]);
                };
                const uint32_t got = min(kAhead, (uint32_t)__popcll(left));
                if (got == 1) {
                    next(0);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += v[0][i];
                    continue;
                }
#pragma unroll
                for (uint32_t k = 0; k < kAhead; ++k) next(k);  // past the last one the last again
                loaded(v);
#pragma unroll
                for (uint32_t k = 0; k < kAhead; ++k)
                    if (k < got)
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] += v[k][i];
            }
        }
    };
    auto tokens_of = [&](uint32_t r) {
        uint32_t c = 0;
        for (uint32_t g = 0; g < count; g += kWave) c += __popcll(__ballot(g + lane < count && key[g + lane] == r));
        return c;
    };
    // Row by row; or, where nothing is written to rows without tokens and the
    // range has more rows than tokens, token by token, a row at its first.
    const bool by_token = to.add && count < size;
    const uint32_t many = by_token ? count : size;
    auto row_at = [&](uint32_t q) -> uint32_t {
        if (!by_token) return q;
        const uint32_t r = uniform(key[q]);
        for (uint32_t g = 0; g < q; g += kWave)
            if (__ballot(g + lane < q && key[g + lane] == r)) return ~0u;
        return r;
    };
    float acc[8];
    for (uint32_t q = wave; q < many; q += kSmallWaves) {
        const uint32_t r = row_at(q);
        if (r == ~0u) continue;
        const uint32_t c = tokens_of(r);
        if (c > kMany || (c == 0 && to.add)) continue;
        sum(r, 0, 1, acc);
        // a row without a token is zero whatever the scale
        put_row<ODT>(grad + (lo + r) * ld_grad, cols, acc, Target{c ? to.scale : 1.0f, to.add});
    }
    if (count <= kMany) return;
    for (uint32_t q = 0; q < many; ++q) {
        const uint32_t r = row_at(q);
        if (r == ~0u || tokens_of(r) <= kMany) continue;
        sum(r, wave, kSmallWaves, acc);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[wave][i][lane] = acc[i];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                for (uint32_t w = 1; w < kSmallWaves; ++w) acc[i] += part[w][i][lane];
            put_row<ODT>(grad + (lo + r) * ld_grad, cols, acc, to);
        }
        __syncthreads();
    }
}

// More tokens: sort, sum, join.  Workspace: start[vocab + 1] (first sorted
// place of each token), key[n] and source[n] (token and row of dy at each
// sorted place), partial sums of the runs that cross a block's end.
struct Sorted {
    uint32_t *start, *key, *source;
    float *part;  // [blocks][2][dim]: a block's sum for a run from an earlier block, and for one that goes on
};

constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / kWave;
constexpr uint32_t kMaxRange = 1000;  // tokens (rows of the table) of one workgroup: 16 counters each, in 64 KB of LDS
constexpr uint32_t kTokensAhead = 8;
constexpr int kMostLanes = 40;
constexpr uint32_t kKept = 4;  // groups of 8 tokens that stay in a lane's registers
constexpr uint32_t kResident = kSortThreads * kTokensAhead * kKept;

// One workgroup sorts the tokens of one range of the vocabulary.  It reads
// all tokens (they stay in the L2), each wave a part of them in order: once
// to count the tokens below its range, which is where its part of the result
// starts, and each token of its range by wave; then again to place them.
// Tokens of one value keep their order: waves hold consecutive parts, and in
// a wave the lanes with the same token find each other by one vote per bit.
// Up to 32768 tokens stay in registers between the two.
template <typename TOK, bool RESIDENT>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(const void *__restrict__ tokens, uint32_t n,
                                                            uint64_t vocab, int64_t padding, uint32_t range,
                                                            uint32_t bits, Sorted out) {
    extern __shared__ uint32_t cnt[];  // [kSortWaves][range], then kSortWaves words
    uint32_t *sums = cnt + kSortWaves * range;
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const uint64_t lo = (uint64_t)blockIdx.x * range;
    const uint32_t size = (uint32_t)min((uint64_t)range, vocab - lo);
    for (uint32_t i = tid; i < kSortWaves * range; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    uint32_t *my = cnt + wave * range;
    const uint32_t part = (n + kSortWaves * kWave - 1) / (kSortWaves * kWave) * kWave;
    const uint32_t first = uniform(min(n, wave * part)), last = uniform(min(n, first + part));
    // tokens i0 + lane, i0 + 64 + lane, ..: their numbers in the range, ~0 for
    // those outside it; `below` counts the tokens below the range, for the first pass
    const uint32_t lo32 = (uint32_t)lo, most = (uint32_t)min(vocab, (uint64_t)1 << 31);
    const uint32_t none = padding >= 0 && padding < (int64_t)most ? (uint32_t)padding : ~0u;
    uint32_t below = 0;
    auto fetch = [&](uint32_t i0, TOK t[kTokensAhead]) {
#pragma unroll
        for (uint32_t k = 0; k < kTokensAhead; ++k) {
            const uint32_t i = i0 + k * kWave + lane;
            t[k] = i < last ? static_cast<const TOK *>(tokens)[i] : (TOK)-1;
        }
    };
    auto classify = [&](const TOK t[kTokensAhead], uint32_t r[kTokensAhead]) {
#pragma unroll
        for (uint32_t k = 0; k < kTokensAhead; ++k) {
            uint32_t key = (uint32_t)t[k];
            if constexpr (sizeof(TOK) == 8) key = (uint64_t)t[k] >> 32 ? ~0u : key;
            key = key < most && key != none ? key : ~0u;
            below += key < lo32;
            r[k] = key - lo32 < size ? key - lo32 : ~0u;
        }
    };
    // Whether many lanes have one token and the others none: such lanes add up
    // at once instead of one after the other at one counter (65536 tokens, nine
    // in ten the same: 92 -> 39 us).
    auto all_one = [&](uint32_t r, uint64_t mine, uint32_t &one) {
        if (__popcll(mine) < kMostLanes) return false;
        one = (uint32_t)__builtin_amdgcn_readlane((int)r, (int)__builtin_ctzll(mine));
        return __ballot(r == one) == mine;
    };
    auto count = [&](const uint32_t r[kTokensAhead]) {
#pragma unroll
        for (uint32_t k = 0; k < kTokensAhead; ++k) {
            const uint64_t mine = __ballot(r[k] != ~0u);
            uint32_t one;
            if (all_one(r[k], mine, one)) {
                if (lane == 0) atomicAdd(&my[one], (uint32_t)__popcll(mine));
            } else if (r[k] != ~0u) {
                atomicAdd(&my[r[k]], 1u);
            }
        }
    };
    uint32_t kept[kKept][kTokensAhead];
    constexpr uint32_t kGroupOfTokens = kTokensAhead * kWave;
    if constexpr (RESIDENT) {
        TOK t[kKept][kTokensAhead];
#pragma unroll
        for (uint32_t g = 0; g < kKept; ++g) fetch(first + g * kGroupOfTokens, t[g]);
#pragma unroll
        for (uint32_t g = 0; g < kKept; ++g)
            if (first + g * kGroupOfTokens < last) {
                classify(t[g], kept[g]);
                count(kept[g]);
            }
    } else {
        for (uint32_t i0 = first; i0 < last; i0 += kGroupOfTokens) {
            TOK t[kTokensAhead];
            fetch(i0, t);
            classify(t, kept[0]);
            count(kept[0]);
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) below += __shfl_xor(below, m, 64);
    if (lane == 0) sums[wave] = below;
    __syncthreads();
    uint32_t base = 0;
    for (uint32_t w = 0; w < kSortWaves; ++w) base += sums[w];
    __syncthreads();
    // start of every token of the range, and of every wave's share of it
    {
        const uint32_t r = tid;
        uint32_t total = 0;
        if (r < size)
            for (uint32_t w = 0; w < kSortWaves; ++w) total += cnt[w * range + r];
        const uint32_t incl = wave_incl_scan(total);
        if (lane == kWave - 1) sums[wave] = incl;
        __syncthreads();
        uint32_t at = base + incl - total;
        for (uint32_t w = 0; w < kSortWaves; ++w) {
            if (w < wave) at += sums[w];
            base += sums[w];
        }
        if (r < size) {
            out.start[lo + r] = at;
            for (uint32_t w = 0; w < kSortWaves; ++w) {
                const uint32_t c = cnt[w * range + r];
                cnt[w * range + r] = at;
                at += c;
            }
        }
    }
    if (tid == 0 && lo + size == vocab) out.start[vocab] = base;
    __syncthreads();
    auto place = [&](const uint32_t r[kTokensAhead], uint32_t i0) {
#pragma unroll
        for (uint32_t k = 0; k < kTokensAhead; ++k) {
            const bool mine = r[k] != ~0u;
            uint64_t same = __ballot(mine);
            if (!same) continue;
            uint32_t one;
            if (!all_one(r[k], same, one))
                for (uint32_t b = 0; b < bits; ++b) {
                    const uint64_t set = __ballot(r[k] >> b & 1);
                    same &= (r[k] >> b & 1) ? set : ~set;
                }
            const uint32_t before = __popcll(same & ((1ull << lane) - 1));
            if (mine) {
                const uint32_t at = my[r[k]] + before;
                out.key[at] = lo32 + r[k];
                out.source[at] = i0 + k * kWave + lane;
            }
            __builtin_amdgcn_wave_barrier();
            if (mine && before == 0) atomicAdd(&my[r[k]], (uint32_t)__popcll(same));
            __builtin_amdgcn_wave_barrier();
        }
    };
    if constexpr (RESIDENT) {
#pragma unroll
        for (uint32_t g = 0; g < kKept; ++g)
            if (first + g * kGroupOfTokens < last) place(kept[g], first + g * kGroupOfTokens);
    } else {
        for (uint32_t i0 = first; i0 < last; i0 += kGroupOfTokens) {
            TOK t[kTokensAhead];
            fetch(i0, t);
            classify(t, kept[0]);
            place(kept[0], i0);
        }
    }
}

// A wave sums one block of sorted places over one slab of columns: whole runs
// go to the gradient, a run that crosses a block's end leaves partial sums.
// Waves past those write the zeros of the rows that no token names.
template <int DT, int ODT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void sum_kernel(const typename Plain<DT>::type *__restrict__ dy,
                                                       uint64_t ld_dy, Sorted in, uint64_t vocab, uint64_t dim,
                                                       uint32_t block, uint32_t blocks, uint32_t slabs, Target to,
                                                       typename Plain<ODT>::type *__restrict__ grad,
                                                       uint64_t ld_grad) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint64_t id = (uint64_t)blockIdx.x * (kThreads / kWave) + uniform(threadIdx.x / kWave);
    const uint64_t work = (uint64_t)blocks * slabs;
    if (id >= work) {
        const uint64_t v = id - work;  // (none where rows are added to: the grid's last waves)
        if (to.add || v >= vocab || in.start[v] != in.start[v + 1]) return;
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (uint32_t slab = 0; slab < slabs; ++slab)
            store_columns<ODT, true>(grad + v * ld_grad, Columns<WHOLE>(slab, lane, dim), zero);
        return;
    }
    const uint32_t b = (uint32_t)(id / slabs);
    const Columns<WHOLE> cols(id % slabs, lane, dim);
    const uint32_t count = uniform(in.start[vocab]);
    const uint32_t p0 = b * block;
    if (p0 >= count) return;
    const uint32_t places = count_before(count, p0, block);
    // lane i: the key of place p0 + i - 1 (lane 0 the place before the block, if any), the row of place p0 + i
    const bool has = lane <= places + 1 && p0 + lane >= 1 && p0 + lane - 1 < count;
    const uint32_t key = has ? in.key[p0 + lane - 1] : ~0u;
    const uint32_t source = lane < places ? in.source[p0 + lane] : 0;
    const uint32_t next = (uint32_t)__shfl_down((int)key, 1, 64);
    const uint64_t change = __ballot(key != next);  // bit i: places p0 + i - 1 and p0 + i differ
    const bool from_before = !(change & 1);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    bool first = true;
    for (uint32_t i0 = 0; i0 < places; i0 += kAhead) {
        float v[kAhead][8];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t i = min(i0 + k, places - 1);
            const uint64_t t = (uint32_t)__builtin_amdgcn_readlane((int)source, (int)i);
            load_columns<DT>(dy + t * ld_dy, cols, v[k]);
        }
        loaded(v);
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t i = i0 + k;
            if (i >= places) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += v[k][j];
            const bool end = change >> (i + 1) & 1;
            if (!end && i + 1 < places) continue;
            const bool before = first && from_before;
            if (end && !before) {
                const uint64_t row = (uint32_t)__builtin_amdgcn_readlane((int)key, (int)i + 1);
                put_row<ODT>(grad + row * ld_grad, cols, acc, to);
            } else {
                store_columns<PC_F32, false>(in.part + ((uint64_t)b * 2 + !before) * dim, cols, acc);
            }
            first = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        }
    }
}

// Joins the partial sums of the run that starts in block b and crosses its
// end, in the order of the blocks: each wave of the workgroup takes an equal
// share of them, and wave 0 adds up the waves.
// Most workgroups find no such run and end: where there are many, they are of
// four waves, else of eight (8184 of eight waves: 26 us, of four 12; one run
// over 2048 blocks: 69 us with four, 42 with eight).
template <int ODT, bool WHOLE, uint32_t THREADS>
__global__ __launch_bounds__(THREADS) void join_kernel(Sorted in, uint64_t vocab, uint64_t dim, uint32_t block,
                                                        uint32_t slabs, Target to,
                                                        typename Plain<ODT>::type *__restrict__ grad,
                                                        uint64_t ld_grad) {
    __shared__ float part[THREADS / kWave][kUnit][kWave];
    const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const uint32_t b = blockIdx.x / slabs, p1 = (b + 1) * block;  // below the number of tokens
    const Columns<WHOLE> cols(blockIdx.x % slabs, lane, dim);
    const uint32_t count = uniform(in.start[vocab]), key = uniform(in.key[p1 - 1]), next = uniform(in.key[p1]);
    if (p1 >= count || key != next) return;
    const uint32_t begin = uniform(in.start[key]), end = uniform(in.start[key + 1]);
    if (begin < b * block) return;
    const uint32_t last = (end - 1) / block;  // the run's parts: block b's second, then the first of b + 1 .. last
    const uint32_t each = (last - b + 1 + THREADS / kWave - 1) / (THREADS / kWave);
    const uint32_t from = b + wave * each, till = min(last + 1, from + each);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t i0 = from; i0 < till; i0 += kAhead) {
        float v[kAhead][8];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint64_t i = min(i0 + k, till - 1);
            load_columns<PC_F32>(in.part + (i * 2 + (i == b)) * dim, cols, v[k]);
        }
        loaded(v);
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k)
            if (i0 + k < till)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += v[k][j];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) part[wave][k][lane] = acc[k];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        for (uint32_t w = 1; w < THREADS / kWave; ++w) acc[k] += part[w][k][lane];
    put_row<ODT>(grad + (uint64_t)key * ld_grad, cols, acc, to);
}

// Sorted places that one wave sums, at most 62 (a lane each, and two for the
// neighbours): 32, or 8, whose loads are all in flight at once, where that
// still leaves fewer than four waves to a SIMD.
uint32_t block_of(uint64_t n, uint64_t slabs) { return n * slabs <= 32768 ? 8 : 32; }
uint64_t slabs_of(uint64_t dim) { return (dim + kSlab - 1) / kSlab; }

// One launch or three: the one pays for few tokens of a small range each.
// 4001 x 1000, 512 tokens: 10 us against 17; 32000 x 2048 (62 rows a
// workgroup), 512 tokens by 1/rank: 82 us against 57.  Above 512 tokens it
// still pays where they are spread (1024 by 1/rank: 14 against 17 us), but not
// where most are one (nine in ten: 576 24 against 17.5 us, 1024 44 against 18;
// 512 22); 15000 x 1000 (14 rows a workgroup): 576 tokens by 1/rank 25 against
// 23 us, 1024 35 against 23.
constexpr uint64_t kSmallRange = 16;
uint64_t small_range(uint64_t vocab, uint64_t slabs) { return std::max<uint64_t>(4, vocab * slabs / 2048); }
bool is_small(uint64_t n, uint64_t vocab, uint64_t dim) {
    return n <= kSmall && small_range(vocab, slabs_of(dim)) <= kSmallRange;
}

uint32_t range_of(uint64_t vocab) {
    const uint64_t r = std::max<uint64_t>(64, (vocab + 255) / 256);
    return (uint32_t)std::min<uint64_t>(kMaxRange, r);
}

uint64_t up16(uint64_t b) { return (b + 15) / 16 * 16; }

}  // namespace

// The sums take a wave for every block of sorted tokens and slab of columns,
// and one for every row's zeros; the joins a workgroup for every block's end.
bool embed_backward_fits(uint64_t n, uint64_t dim, uint64_t vocab) {
    constexpr uint64_t kMaxGroups = (1ull << 24) - 1;  // of 256 lanes, in a launch of fewer than 2^32
    if (is_small(n, vocab, dim)) return true;
    const uint64_t slabs = slabs_of(dim), block = block_of(n, slabs), blocks = (n + block - 1) / block;
    return (blocks * slabs + vocab + 3) / 4 <= kMaxGroups && (blocks == 0 || (blocks - 1) * slabs <= kMaxGroups);
}

uint64_t embed_backward_workspace(uint64_t n, uint64_t dim, uint64_t vocab) {
    if (is_small(n, vocab, dim)) return 0;
    const uint64_t block = block_of(n, slabs_of(dim)), blocks = (n + block - 1) / block;
    return up16((vocab + 1) * 4) + 2 * up16(n * 4) + up16(blocks * 2 * dim * 4);
}

hipError_t launch_embed(const void *tokens, int token_bytes, uint64_t n, const void *table, const uint8_t *codes,
                        int kind, uint64_t vocab, uint64_t dim, uint64_t ld_table, uint64_t ld_codes, float scale,
                        void *out, int out_dtype, uint64_t ld_out, uint32_t *status, hipStream_t stream) {
    const Units units = make_units(n, dim, false);
    const dim3 grid((uint32_t)((units.total + kTile - 1) / kTile));
    with_dtype(out_dtype, [&](auto o) {
        constexpr int ODT = decltype(o)::value;
        auto launch = [&](auto k) {
            hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, stream, tokens, table, codes, vocab, ld_table, ld_codes,
                               units, scale, static_cast<typename Plain<ODT>::type *>(out), ld_out, status);
        };
        auto by_table = [&](auto tok) {
            typedef decltype(tok) TOK;
            switch (kind) {
                case PC_F32: launch(embed_kernel<PC_F32, ODT, TOK>); break;
                case PC_F16: launch(embed_kernel<PC_F16, ODT, TOK>); break;
                case PC_BF16: launch(embed_kernel<PC_BF16, ODT, TOK>); break;
                case 4 + PC_Q8_E4M3: launch(embed_kernel<4 + PC_Q8_E4M3, ODT, TOK>); break;
                case 4 + PC_Q8_INT8: launch(embed_kernel<4 + PC_Q8_INT8, ODT, TOK>); break;
            }
        };
        token_bytes == 8 ? by_table((int64_t)0) : by_table((int32_t)0);
    });
    return hipGetLastError();
}

hipError_t launch_embed_backward(const void *dy, int dtype, uint64_t ld_dy, const void *tokens, int token_bytes,
                                 uint32_t n, uint64_t dim, uint64_t vocab, int64_t padding, float scale, void *grad,
                                 int grad_dtype, uint64_t ld_grad, bool accumulate, void *ws, hipStream_t stream) {
    const uint32_t slabs = (uint32_t)slabs_of(dim);
    const Target to = {scale, accumulate};
    const bool whole = dim % 4 == 0;
    if (is_small(n, vocab, dim)) {
        // about 2048 workgroups, of at least 4 rows: each reads all tokens
        const uint64_t each = small_range(vocab, slabs);
        const dim3 grid((uint32_t)((vocab + each - 1) / each), slabs);
        with_dtype(grad_dtype, [&](auto o) {
            constexpr int ODT = decltype(o)::value;
            with_dtype(dtype, [&](auto d) {
                constexpr int DT = decltype(d)::value;
                auto launch = [&](auto k) {
                    hipLaunchKernelGGL(k, grid, dim3(kSmallThreads), 0, stream, tokens, n,
                                       static_cast<const typename Plain<DT>::type *>(dy), ld_dy, vocab, dim, padding,
                                       (uint32_t)each, to, static_cast<typename Plain<ODT>::type *>(grad), ld_grad);
                };
                auto by_width = [&](auto w) {
                    constexpr bool WHOLE = decltype(w)::value;
                    token_bytes == 8 ? launch(small_kernel<DT, ODT, int64_t, WHOLE>)
                                     : launch(small_kernel<DT, ODT, int32_t, WHOLE>);
                };
                if (whole) by_width(std::true_type());
                else by_width(std::false_type());
            });
        });
        return hipGetLastError();
    }
    const uint32_t range = range_of(vocab), block = block_of(n, slabs), blocks = (n + block - 1) / block;
    uint32_t bits = 0;
    while ((1u << bits) < range) ++bits;
    uint8_t *p = static_cast<uint8_t *>(ws);
    Sorted s;
    s.start = reinterpret_cast<uint32_t *>(p);
    p += up16((vocab + 1) * 4);
    s.key = reinterpret_cast<uint32_t *>(p);
    p += up16((uint64_t)n * 4);
    s.source = reinterpret_cast<uint32_t *>(p);
    p += up16((uint64_t)n * 4);
    s.part = reinterpret_cast<float *>(p);
    const dim3 ranges((uint32_t)((vocab + range - 1) / range));
    const uint32_t lds = (kSortWaves * range + kSortWaves) * 4;
    auto sort = [&](auto k) {
        hipLaunchKernelGGL(k, ranges, dim3(kSortThreads), lds, stream, tokens, n, vocab, padding, range, bits, s);
    };
    if (n <= kResident) token_bytes == 8 ? sort(sort_kernel<int64_t, true>) : sort(sort_kernel<int32_t, true>);
    else token_bytes == 8 ? sort(sort_kernel<int64_t, false>) : sort(sort_kernel<int32_t, false>);
    const uint64_t waves = (uint64_t)blocks * slabs + (accumulate ? 0 : vocab);
    const dim3 grid((uint32_t)((waves + kThreads / kWave - 1) / (kThreads / kWave)));
    auto sums = [&](auto o, auto w) {
        constexpr int ODT = decltype(o)::value;
        constexpr bool WHOLE = decltype(w)::value;
        typedef typename Plain<ODT>::type T;
        with_dtype(dtype, [&](auto d) {
            constexpr int DT = decltype(d)::value;
            if (grid.x == 0) return;
            hipLaunchKernelGGL((sum_kernel<DT, ODT, WHOLE>), grid, dim3(kThreads), 0, stream,
                               static_cast<const typename Plain<DT>::type *>(dy), ld_dy, s, vocab, dim, block, blocks,
                               slabs, to, static_cast<T *>(grad), ld_grad);
        });
        const uint32_t joins = blocks > 1 ? (blocks - 1) * slabs : 0;
        auto join = [&](auto k, uint32_t threads) {
            hipLaunchKernelGGL(k, dim3(joins), dim3(threads), 0, stream, s, vocab, dim, block, slabs, to,
                               static_cast<T *>(grad), ld_grad);
        };
        if (joins > 4096) join(join_kernel<ODT, WHOLE, 256>, 256);
        else if (joins) join(join_kernel<ODT, WHOLE, 512>, 512);
    };
    with_dtype(grad_dtype, [&](auto o) {
        if (whole) sums(o, std::true_type());
        else sums(o, std::false_type());
    });
    return hipGetLastError();
}

}  // namespace pc
