// Embedding lookup, and the table's gradient by sorted tokens.
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
    float v[kPerLane][8];
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        const uint32_t local = j * kThreads + threadIdx.x;
        n[j] = 0;
        if (base + local < units.total) {
            find_unit(units, base, local, row[j], col[j]);
            if (col[j] < units.cols) n[j] = (uint32_t)min((uint64_t)kUnit, units.cols - col[j]);
            tok[j] = token_at<TOK>(tokens, row[j]);
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        if (!n[j]) continue;
        if (tok[j] < 0 || (uint64_t)tok[j] >= vocab) {
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
        for (int i = 0; i < 8; ++i) v[j][i] *= scale;
        store_unit<ODT>(out + row[j] * ld_out + col[j], n[j], v[j]);
    }
}

// ---------------------------------------------------------------------------
// gradient: sort the tokens, sum the rows of dy in that order
// ---------------------------------------------------------------------------

// Workspace: start[vocab + 1] (first sorted place of each token), key[n] and
// source[n] (token and row of dy at each sorted place), partial sums of the
// runs that cross a block's end.
struct Sorted {
    uint32_t *start, *key, *source;
    float *part;  // [blocks][2][dim]: a block's sum for a run from an earlier block, and for one that goes on
};

constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / kWave;
constexpr uint32_t kMaxRange = 1000;  // tokens (rows of the table) of one workgroup: 16 counters each, in 64 KB of LDS

// One workgroup sorts the tokens of one range of the vocabulary.  It reads
// all tokens (they stay in the L2), each wave a part of them in order: once
// to count the tokens below its range, which is where its part of the result
// starts, and each token of its range by wave; then again to place them.
// Tokens of one value keep their order: waves hold consecutive parts, and in
// a wave the lanes with the same token find each other by one vote per bit.
template <typename TOK>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(const void *__restrict__ tokens, uint32_t n,
                                                            uint64_t vocab, int64_t padding, uint32_t range,
                                                            uint32_t bits, Sorted out) {
    extern __shared__ uint32_t cnt[];  // [kSortWaves][range], then kSortWaves + 1 words
    uint32_t *sums = cnt + kSortWaves * range;
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const uint64_t lo = (uint64_t)blockIdx.x * range;
    const uint32_t size = (uint32_t)min((uint64_t)range, vocab - lo);
    for (uint32_t i = tid; i < kSortWaves * range; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    uint32_t *my = cnt + wave * range;
    const uint32_t part = (n + kSortWaves * kWave - 1) / (kSortWaves * kWave) * kWave;
    const uint32_t first = min(n, wave * part), last = min(n, first + part);
    uint32_t below = 0;
    for (uint32_t i = first + lane; i < last; i += kWave) {
        const int64_t t = token_at<TOK>(tokens, i);
        if (t < 0 || (uint64_t)t >= vocab || t == padding) continue;
        if ((uint64_t)t < lo) ++below;
        else if ((uint64_t)t - lo < size) atomicAdd(&my[(uint64_t)t - lo], 1u);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) below += __shfl_xor(below, m, 64);
    if (lane == 0) sums[wave] = below;
    __syncthreads();
    uint32_t base = 0;
    for (uint32_t w = 0; w < kSortWaves; ++w) base += sums[w];
    __syncthreads();
    // start of every token of the range, and of every wave's share of it
    for (uint32_t r0 = 0; r0 < size; r0 += kSortThreads) {
        const uint32_t r = r0 + tid;
        uint32_t total = 0;
        if (r < size)
            for (uint32_t w = 0; w < kSortWaves; ++w) total += cnt[w * range + r];
        const uint32_t incl = wave_incl_scan(total);
        if (lane == kWave - 1) sums[wave] = incl;
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (uint32_t w = 0; w < kSortWaves; ++w) {
            if (w < wave) before += sums[w];
            all += sums[w];
        }
        __syncthreads();
        if (r < size) {
            uint32_t at = base + before + incl - total;
            out.start[lo + r] = at;
            for (uint32_t w = 0; w < kSortWaves; ++w) {
                const uint32_t c = cnt[w * range + r];
                cnt[w * range + r] = at;
                at += c;
            }
        }
        base += all;
    }
    if (tid == 0 && lo + size == vocab) out.start[vocab] = base;
    __syncthreads();
    for (uint32_t i0 = first; i0 < last; i0 += kWave) {
        const uint32_t i = i0 + lane;
        const int64_t t = i < last ? token_at<TOK>(tokens, i) : -1;
        const bool mine = t >= 0 && t != padding && (uint64_t)t >= lo && (uint64_t)t - lo < size;
        uint64_t same = __ballot(mine);
        if (!same) continue;
        const uint32_t r = mine ? (uint32_t)((uint64_t)t - lo) : 0;
        for (uint32_t b = 0; b < bits; ++b) {
            const uint64_t set = __ballot(r >> b & 1);
            same &= (r >> b & 1) ? set : ~set;
        }
        const uint32_t before = __popcll(same & ((1ull << lane) - 1));
        if (mine) {
            const uint32_t at = my[r] + before;
            out.key[at] = (uint32_t)t;
            out.source[at] = i;
        }
        __builtin_amdgcn_wave_barrier();
        if (mine && before == 0) atomicAdd(&my[r], (uint32_t)__popcll(same));
        __builtin_amdgcn_wave_barrier();
    }
}

template <int ODT>
__device__ __forceinline__ void put_row(typename Plain<ODT>::type *p, uint32_t n, const float v[8], float scale,
                                        bool add) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = v[i] * scale;
    if (add) {
        float old[8];
        load_unit<ODT>(p, n, old);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += old[i];
    }
    store_unit<ODT>(p, n, s);
}

constexpr uint32_t kSlab = kWave * kUnit;  // columns of one wave

// A wave sums one block of sorted places over one slab of columns: whole runs
// go to the gradient, a run that crosses a block's end leaves partial sums.
// Waves past those write the zeros of the rows that no token names.
template <int DT, int ODT>
__global__ __launch_bounds__(kThreads) void sum_kernel(const typename Plain<DT>::type *__restrict__ dy,
                                                       uint64_t ld_dy, Sorted in, uint64_t vocab, uint64_t dim,
                                                       uint32_t block, uint32_t blocks, uint32_t slabs, float scale,
                                                       typename Plain<ODT>::type *__restrict__ grad,
                                                       uint64_t ld_grad, uint32_t add) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint64_t id = (uint64_t)blockIdx.x * (kThreads / kWave) + uniform(threadIdx.x / kWave);
    const uint64_t work = (uint64_t)blocks * slabs;
    if (id >= work) {
        if (add) return;
        const uint64_t v = id - work;
        if (v >= vocab || in.start[v] != in.start[v + 1]) return;
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (uint64_t c = lane * kUnit; c < dim; c += kSlab)
            store_unit<ODT>(grad + v * ld_grad + c, (uint32_t)min((uint64_t)kUnit, dim - c), zero);
        return;
    }
    const uint32_t b = (uint32_t)(id / slabs);
    const uint64_t col = (id % slabs) * kSlab + lane * kUnit;
    const uint32_t n = col < dim ? (uint32_t)min((uint64_t)kUnit, dim - col) : 0;
    const uint32_t count = in.start[vocab];
    const uint32_t p0 = b * block;
    if (p0 >= count) return;
    const uint32_t p1 = min(count, p0 + block);
    uint32_t p = p0;
    while (p < p1) {
        const uint32_t key = uniform(in.key[p]);
        const uint32_t begin = uniform(in.start[key]), end = uniform(in.start[key + 1]);
        const uint32_t stop = min(p1, end);
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (; p < stop; ++p) {
            const uint64_t t = uniform(in.source[p]);
            if (n) {
                float v[8];
                load_unit<DT>(dy + t * ld_dy + col, n, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += v[i];
            }
        }
        if (!n) continue;
        if (begin >= p0 && end <= p0 + block)
            put_row<ODT>(grad + (uint64_t)key * ld_grad + col, n, acc, scale, add);
        else
            store_unit<PC_F32>(in.part + ((uint64_t)b * 2 + (begin >= p0)) * dim + col, n, acc);
    }
}

// Joins the partial sums of the run that starts in block b and crosses its
// end, in the order of the blocks: each wave of the workgroup takes an equal
// share of them, and wave 0 adds up the waves.
template <int ODT>
__global__ __launch_bounds__(kThreads) void join_kernel(Sorted in, uint64_t vocab, uint64_t dim, uint32_t block,
                                                        uint32_t slabs, float scale,
                                                        typename Plain<ODT>::type *__restrict__ grad,
                                                        uint64_t ld_grad, uint32_t add) {
    __shared__ float part[kThreads / kWave][kUnit][kWave];
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t b = blockIdx.x / slabs;
    const uint64_t col = (uint64_t)(blockIdx.x % slabs) * kSlab + lane * kUnit;
    const uint32_t n = col < dim ? (uint32_t)min((uint64_t)kUnit, dim - col) : 0;
    const uint32_t count = in.start[vocab];
    const uint32_t p1 = (b + 1) * block;
    if (p1 >= count) return;
    const uint32_t key = in.key[p1 - 1];
    const uint32_t begin = in.start[key], end = in.start[key + 1];
    if (end <= p1 || begin < b * block) return;
    const uint32_t last = (end - 1) / block;  // the run's parts: block b's second, then the first of b + 1 .. last
    const uint32_t each = (last - b + 1 + kThreads / kWave - 1) / (kThreads / kWave);
    const uint32_t from = b + wave * each, to = min(last + 1, from + each);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n)
        for (uint32_t i = from; i < to; ++i) {
            float v[8];
            load_unit<PC_F32>(in.part + ((uint64_t)i * 2 + (i == b)) * dim + col, n, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += v[k];
        }
#pragma unroll
    for (int k = 0; k < 8; ++k) part[wave][k][lane] = acc[k];
    __syncthreads();
    if (wave || !n) return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        for (uint32_t w = 1; w < kThreads / kWave; ++w) acc[k] += part[w][k][lane];
    put_row<ODT>(grad + (uint64_t)key * ld_grad + col, n, acc, scale, add);
}

constexpr uint32_t kBlock = 32;  // sorted places summed by one wave

uint32_t range_of(uint64_t vocab) {
    const uint64_t r = std::max<uint64_t>(64, (vocab + 255) / 256);
    return (uint32_t)std::min<uint64_t>(kMaxRange, r);
}

uint64_t up16(uint64_t b) { return (b + 15) / 16 * 16; }

}  // namespace

uint64_t embed_backward_workspace(uint64_t n, uint64_t dim, uint64_t vocab) {
    const uint64_t blocks = (n + kBlock - 1) / kBlock;
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
    const uint32_t range = range_of(vocab), blocks = (n + kBlock - 1) / kBlock;
    const uint32_t slabs = (uint32_t)((dim + kSlab - 1) / kSlab);
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
    const uint32_t lds = (kSortWaves * range + kSortWaves + 1) * 4;
    auto sort = [&](auto k) {
        hipLaunchKernelGGL(k, ranges, dim3(kSortThreads), lds, stream, tokens, n, vocab, padding, range, bits, s);
    };
    token_bytes == 8 ? sort(sort_kernel<int64_t>) : sort(sort_kernel<int32_t>);
    const uint64_t waves = (uint64_t)blocks * slabs + (accumulate ? 0 : vocab);
    const dim3 grid((uint32_t)((waves + kThreads / kWave - 1) / (kThreads / kWave)));
    with_dtype(grad_dtype, [&](auto o) {
        constexpr int ODT = decltype(o)::value;
        typedef typename Plain<ODT>::type T;
        if (grid.x)
            with_dtype(dtype, [&](auto d) {
                constexpr int DT = decltype(d)::value;
                hipLaunchKernelGGL((sum_kernel<DT, ODT>), grid, dim3(kThreads), 0, stream,
                                   static_cast<const typename Plain<DT>::type *>(dy), ld_dy, s, vocab, dim, kBlock,
                                   blocks, slabs, scale, static_cast<T *>(grad), ld_grad, (uint32_t)accumulate);
            });
        if (blocks > 1)
            hipLaunchKernelGGL(join_kernel<ODT>, dim3((blocks - 1) * slabs), dim3(kThreads), 0, stream, s, vocab, dim,
                               kBlock, slabs, scale, static_cast<T *>(grad), ld_grad, (uint32_t)accumulate);
    });
    return hipGetLastError();
}

}  // namespace pc
