// Log probabilities of given tokens, entropy and the most probable tokens of
// rows of logits, and the gradient of the logits.
//
//   z = scale x,  m = max x,  e_v = exp(z_v - scale m),  S = sum e
//   logp_v = (x_v - m) scale - ln S
//   H = ln S - sum e_v (z_v - scale m) / S
//   d x_v = scale (sum_j d_j [v = t_j] - p_v (sum_j d_j + d_H (logp_v + H)))
#include <algorithm>
#include <type_traits>

#include "q8.h"

namespace pc {
namespace {

constexpr uint32_t kMaxThreads = 1024;
constexpr uint32_t kMaxWaves = kMaxThreads / kWave;
constexpr uint32_t kVecs = 4;  // 16-byte loads of a lane on their way together
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kLowest = -3.40282347e38f;
constexpr float kGone = -1000.0f;  // 2^-1000 is 0 in 32 bits, and 0 times -1000 still 0

template <int DT> constexpr uint32_t kPer = DT == PC_F32 ? 4 : 8;  // elements of 16 bytes

template <int DT>
__device__ __forceinline__ u32x4 load_vec(const typename Plain<DT>::type *p, uint32_t n) {
    if constexpr (DT == PC_F32) {
        if (n == 4) return *reinterpret_cast<const u32x4_any4 *>(p);
        u32x4 r = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < n) r[i] = as_u32(p[i]);
        return r;
    } else {
        return load_raw<DT>(p, n).w[0];
    }
}

template <int DT>
__device__ __forceinline__ void widen_vec(u32x4 w, float v[kPer<DT>]) {
    if constexpr (DT == PC_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = as_f32(w[i]);
    } else {
        RawUnit<DT> r;
        r.w[0] = w;
        widen_unit<DT>(r, v);
    }
}

template <int DT>
__device__ __forceinline__ void store_vec(typename Plain<DT>::type *p, uint32_t n, const float v[kPer<DT>]) {
    if constexpr (DT == PC_F32) {
        if (n == 4) {
            put<4, true>(p, u32x4{as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])});
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                if (i < n) p[i] = v[i];
        }
    } else {
        store_unit<DT>(p, n, v);
    }
}

__device__ __forceinline__ uint32_t from_lane(uint32_t v, uint32_t lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)lane);
}

__device__ __forceinline__ float from_lane(float v, uint32_t lane) { return as_f32(from_lane(as_u32(v), lane)); }

// ---------------------------------------------------------------------------
// running maximum and sums
// ---------------------------------------------------------------------------

// Of some elements: their largest m (at least the lowest finite number), and
// with u = (x - m) scale log2(e), the sums of 2^u and of 2^u u.  NaN and
// +infinity make s NaN; s is 0 where every element is -infinity.
struct Soft { float m, s, t; };

__device__ __forceinline__ Soft nothing() { return {kLowest, 0.0f, 0.0f}; }

// fmaxf takes the other operand where one is NaN
__device__ __forceinline__ Soft moved(Soft a, float m, float c) {
    const float u = fmaxf((a.m - m) * c, kGone), f = __builtin_amdgcn_exp2f(u);
    return {m, a.s * f, f * (a.t + u * a.s)};
}

__device__ __forceinline__ Soft joined(Soft a, Soft b, float c) {
    const float m = fmaxf(a.m, b.m);
    a = moved(a, m, c);
    b = moved(b, m, c);
    return {m, a.s + b.s, a.t + b.t};
}

template <int CTRL>
__device__ __forceinline__ Soft dpp_soft(Soft v) {
    return {as_f32(dpp_u32<CTRL>(as_u32(v.m))), as_f32(dpp_u32<CTRL>(as_u32(v.s))), as_f32(dpp_u32<CTRL>(as_u32(v.t)))};
}

__device__ __forceinline__ Soft soft_of(Soft v, uint32_t lane) {
    return {from_lane(v.m, lane), from_lane(v.s, lane), from_lane(v.t, lane)};
}

// All lanes' joined, the same in every lane.
__device__ __forceinline__ Soft wave_soft(Soft v, float c) {
    v = joined(v, dpp_soft<0xB1>(v), c);
    v = joined(v, dpp_soft<0x4E>(v), c);
    v = joined(v, dpp_soft<0x141>(v), c);
    v = joined(v, dpp_soft<0x140>(v), c);
    return joined(joined(soft_of(v, 0), soft_of(v, 16), c), joined(soft_of(v, 32), soft_of(v, 48), c), c);
}

// ---------------------------------------------------------------------------
// the largest elements
// ---------------------------------------------------------------------------

// An order-preserving key: NaN counts as -infinity, -0 as 0.  Never 0, which
// stands for no element.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = as_u32(fmaxf(x, -__builtin_inff()) + 0.0f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// The wave's 64 largest elements so far, one a lane in descending order, equal
// ones by their index.
struct Best { uint32_t key, index; };

__device__ __forceinline__ uint64_t packed(Best b) { return (uint64_t)b.key << 32 | (b.key ? ~b.index : 0u); }

__device__ __forceinline__ Best unpacked(uint64_t p) { return {(uint32_t)(p >> 32), ~(uint32_t)p}; }

// An element whose index is larger than those of all equal ones in the list.
__device__ __forceinline__ void insert(Best &b, uint32_t key, uint32_t index) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t place = (uint32_t)__popcll(__ballot(b.key >= key));
    const uint32_t key_before = dpp_u32<0x138>(b.key), index_before = dpp_u32<0x138>(b.index);  // from the lane below
    if (lane > place) {
        b.key = key_before;
        b.index = index_before;
    } else if (lane == place) {
        b.key = key;
        b.index = index;
    }
}

// Takes the elements v of every lane (the first n count, from index `first`
// on) into the list, where they are larger than the `top`th one.
template <int N>
__device__ __forceinline__ void take(Best &b, uint32_t top, float largest, const float v[N], uint32_t n, uint32_t first) {
    uint32_t least = from_lane(b.key, top - 1);
    const uint32_t key = n ? key_of(largest) : 0;
    uint64_t left = __ballot(key > least);
    while (left) {
        const uint32_t lane = (uint32_t)__builtin_ctzll(left);
        const uint32_t count = from_lane(n, lane), index = from_lane(first, lane);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t k = key_of(from_lane(v[i], lane));
            if ((uint32_t)i < count && k > least) {
                insert(b, k, index + i);
                least = from_lane(b.key, top - 1);
            }
        }
        left &= left - 1;
        left &= __ballot(key > least);
    }
}

// The 64 largest of two lists: the larger of one list and the other one turned
// round are they, and rise to one place and fall from it, or the reverse.
__device__ __forceinline__ uint64_t merged(uint64_t a, uint64_t b) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint64_t turned = __shfl(b, 63 - lane, 64);
    a = a > turned ? a : turned;
#pragma unroll
    for (uint32_t d = 32; d; d >>= 1) {
        const uint64_t o = __shfl_xor(a, d, 64);
        const bool low = (lane & d) == 0;
        a = low == (a > o) ? a : o;
    }
    return a;
}

struct Args {
    const void *logits, *tokens;
    float *logp, *top_logp, *stats;
    int64_t *top_index;
    uint32_t *status;
    Soft *soft;      // [rows * splits], where rows are split
    uint64_t *best;  // [rows * splits][top]
    uint64_t rows, ld;
    int64_t padding;
    uint32_t vocab, units, splits, per_split, n_tokens, top;
    int token_bytes;
    float scale;
};

__device__ __forceinline__ int64_t token_at(const void *tokens, int token_bytes, uint64_t i) {
    return token_bytes == 8 ? static_cast<const int64_t *>(tokens)[i] : static_cast<const int32_t *>(tokens)[i];
}

// Joins the waves' sums and lists in LDS; wave 0 has the result.
template <bool TOP>
__device__ __forceinline__ void join_waves(Soft &soft, uint64_t &best, float c, Soft *softs, uint64_t *lists) {
    const uint32_t wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    if (waves == 1) return;
    if (lane == 0) softs[wave] = soft;
    if constexpr (TOP) {
        lists[wave * kWave + lane] = best;
        for (uint32_t half = waves / 2; half; half /= 2) {
            __syncthreads();
            if (wave < half) {
                best = merged(best, lists[(wave + half) * kWave + lane]);
                lists[wave * kWave + lane] = best;
            }
        }
    }
    __syncthreads();
    if (wave == 0) soft = wave_soft(lane < waves ? softs[lane] : nothing(), c);
}

// One wave writes a row's results.
template <int DT, bool TOP>
__device__ __forceinline__ void finish(const Args &a, uint64_t row, Soft soft, uint64_t best) {
    typedef typename Plain<DT>::type T;
    const uint32_t lane = threadIdx.x % kWave;
    const T *x = static_cast<const T *>(a.logits) + row * a.ld;
    const bool empty = soft.s == 0.0f;
    const float minus = -__builtin_inff();
    const float log_sum = logf(soft.s);
    auto logp_of = [&](float v) { return empty ? minus : (v - soft.m) * a.scale - log_sum; };
    if (lane < a.n_tokens) {
        const uint64_t i = row * a.n_tokens + lane;
        const int64_t t = token_at(a.tokens, a.token_bytes, i);
        float logp = 0.0f;
        if (t != a.padding) {
            if (t >= 0 && t < (int64_t)a.vocab) logp = logp_of(widen(x[t]));
            else if (a.status) *a.status = PC_ERR_INVALID_ARG;
        }
        a.logp[i] = logp;
    }
    if constexpr (TOP) {
        if (lane < a.top) {
            const uint32_t index = unpacked(best).index;
            a.top_index[row * a.top + lane] = index;
            a.top_logp[row * a.top + lane] = logp_of(widen(x[index]));
        }
    }
    if (lane == 0 && a.stats) {
        float *s = a.stats + 4 * row;
        s[0] = empty ? minus : soft.m;
        s[1] = log_sum;
        s[2] = empty ? 0.0f : log_sum - kLn2 * (soft.t / soft.s);
        s[3] = empty ? minus : soft.m * a.scale + log_sum;
    }
}

// A workgroup takes a row, or one of `splits` stretches of it.
template <int DT, bool TOP>
__global__ __launch_bounds__(kMaxThreads) void rows_kernel(Args a) {
    typedef typename Plain<DT>::type T;
    constexpr uint32_t N = kPer<DT>;
    __shared__ Soft softs[kMaxWaves];
    __shared__ uint64_t lists[TOP ? kMaxThreads : 1];
    const uint32_t tid = threadIdx.x, threads = blockDim.x, step = threads * kVecs;
    const float c = a.scale * kLog2E;
    const uint64_t total = a.rows * a.splits;
    for (uint64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const uint64_t row = a.splits == 1 ? id : id / a.splits;
        const uint32_t split = (uint32_t)(id - row * a.splits);
        const uint32_t begin = split * a.per_split, end = min(a.units, begin + a.per_split);
        const T *x = static_cast<const T *>(a.logits) + row * a.ld;
        auto load = [&](uint32_t base, u32x4 w[kVecs]) {
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) {
                const uint32_t u = base + j * threads + tid;
                const uint32_t n = u < end ? count_before(a.vocab, u * N, N) : 0;
                w[j] = load_vec<DT>(x + (uint64_t)u * N, n);
            }
        };
        Soft soft = nothing();
        Best best = {0, 0};
        u32x4 w[kVecs];
        load(begin, w);
        for (uint32_t base = begin; base < end; base += step) {
            u32x4 next[kVecs];
            load(base + step, next);
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) {
                const uint32_t u = base + j * threads + tid;
                const uint32_t n = u < end ? count_before(a.vocab, u * N, N) : 0;
                float v[N];
                widen_vec<DT>(w[j], v);
                if (n != N) {
#pragma unroll
                    for (uint32_t i = 0; i < N; ++i)
                        if (i >= n) v[i] = -__builtin_inff();
                }
                float largest = v[0];
#pragma unroll
                for (uint32_t i = 1; i < N; ++i) largest = fmaxf(largest, v[i]);
                if constexpr (TOP) take<N>(best, a.top, largest, v, n, u * N);
                const float m = fmaxf(soft.m, largest);
                soft = moved(soft, m, c);
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) {
                    const float y = (v[i] - m) * c, e = __builtin_amdgcn_exp2f(y);
                    soft.s += e;
                    soft.t += e * fmaxf(y, kGone);
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) w[j] = next[j];
        }
        soft = wave_soft(soft, c);
        uint64_t list = packed(best);
        join_waves<TOP>(soft, list, c, softs, lists);
        if (tid < kWave) {
            if (a.splits == 1) {
                finish<DT, TOP>(a, row, soft, list);
            } else {
                if (tid == 0) a.soft[id] = soft;
                if (TOP && tid < a.top) a.best[id * a.top + tid] = list;
            }
        }
        __syncthreads();  // the next turn writes the areas that wave 0 has read
    }
}

// The stretches of a row joined: a wave takes every 16th, in order.
template <int DT, bool TOP>
__global__ __launch_bounds__(kMaxThreads) void join_kernel(Args a) {
    __shared__ Soft softs[kMaxWaves];
    __shared__ uint64_t lists[TOP ? kMaxThreads : 1];
    const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
    const float c = a.scale * kLog2E;
    const uint64_t row = blockIdx.x;
    Soft soft = nothing();
    uint64_t best = 0;
    for (uint32_t s = wave * kWave + lane; s < a.splits; s += blockDim.x)
        soft = joined(soft, a.soft[row * a.splits + s], c);
    soft = wave_soft(soft, c);
    if constexpr (TOP) {
        for (uint32_t s = wave; s < a.splits; s += waves)
            best = merged(best, lane < a.top ? a.best[(row * a.splits + s) * a.top + lane] : 0);
    }
    join_waves<TOP>(soft, best, c, softs, lists);
    if (wave == 0) finish<DT, TOP>(a, row, soft, best);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

constexpr uint32_t kGradThreads = 256;
constexpr uint32_t kGradUnits = kGradThreads * kVecs;

struct GradArgs {
    const void *logits, *tokens;
    const float *stats, *d_logp, *d_entropy;
    void *out;
    uint64_t rows, ld, ld_out;
    int64_t padding;
    uint32_t vocab, tiles, n_tokens;
    int token_bytes;
    float scale;
};

__device__ __forceinline__ float wave_sum(float v) {
    v += as_f32(dpp_u32<0xB1>(as_u32(v)));
    v += as_f32(dpp_u32<0x4E>(as_u32(v)));
    v += as_f32(dpp_u32<0x141>(as_u32(v)));
    v += as_f32(dpp_u32<0x140>(as_u32(v)));
    return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}

template <int DT, bool ENTROPY>
__global__ __launch_bounds__(kGradThreads) void grad_kernel(GradArgs a) {
    typedef typename Plain<DT>::type T;
    constexpr uint32_t N = kPer<DT>;
    const uint32_t lane = threadIdx.x % kWave, total = (uint32_t)a.rows * a.tiles;
    for (uint32_t id = blockIdx.x; id < total; id += gridDim.x) {
        const uint32_t row = id / a.tiles, unit0 = (id - row * a.tiles) * kGradUnits;
        const T *x = static_cast<const T *>(a.logits) + row * a.ld;
        T *out = static_cast<T *>(a.out) + row * a.ld_out;
        u32x4 w[kVecs];
        uint32_t n[kVecs];
#pragma unroll
        for (uint32_t j = 0; j < kVecs; ++j) {
            const uint32_t u = unit0 + j * kGradThreads + threadIdx.x;
            n[j] = count_before(a.vocab, u * N, N);
            w[j] = load_vec<DT>(x + (uint64_t)u * N, n[j]);
        }
        // a token to a lane
        int64_t token = -1;
        float d = 0.0f;
        if (lane < a.n_tokens) {
            token = token_at(a.tokens, a.token_bytes, (uint64_t)row * a.n_tokens + lane);
            if (token == a.padding || token < 0 || token >= (int64_t)a.vocab) token = -1;
            else d = a.d_logp[(uint64_t)row * a.n_tokens + lane];
        }
        const float sum = wave_sum(d);
        const float largest = a.stats[4 * (uint64_t)row], log_sum = a.stats[4 * (uint64_t)row + 1];
        float entropy = 0.0f, de = 0.0f;
        if constexpr (ENTROPY) {
            entropy = a.stats[4 * (uint64_t)row + 2];
            de = a.d_entropy[row];
        }
        const bool none = (__ballot(d != 0.0f) == 0 && de == 0.0f) || largest == -__builtin_inff();
        const uint64_t inside =
            __ballot(token >= (int64_t)unit0 * N && token < ((int64_t)unit0 + kGradUnits) * N && !none);
        const uint32_t at = (uint32_t)token;
#pragma unroll
        for (uint32_t j = 0; j < kVecs; ++j) {
            const uint32_t u = unit0 + j * kGradThreads + threadIdx.x;
            float v[N];
            widen_vec<DT>(w[j], v);
#pragma unroll
            for (uint32_t i = 0; i < N; ++i) {
                const float y = (v[i] - largest) * a.scale - log_sum;
                const float p = __builtin_amdgcn_exp2f(y * kLog2E);
                float g = sum;
                if constexpr (ENTROPY) g += de * (fmaxf(y, kGone) + entropy);
                v[i] = none ? 0.0f : -p * g;
            }
            for (uint64_t left = inside; left; left &= left - 1) {
                const uint32_t l = (uint32_t)__builtin_ctzll(left);
                const uint32_t place = from_lane(at, l) - u * N;
                const float add = from_lane(d, l);
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) v[i] += place == i ? add : 0.0f;
            }
            if (!n[j]) continue;
#pragma unroll
            for (uint32_t i = 0; i < N; ++i) v[i] *= a.scale;
            store_vec<DT>(out + (uint64_t)u * N, n[j], v);
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

uint32_t units_of(uint64_t vocab, int dtype) { return (uint32_t)((vocab + (dtype == PC_F32 ? 3 : 7)) / (dtype == PC_F32 ? 4 : 8)); }

struct Plan { uint32_t threads, splits, per_split; };

Plan plan_rows(uint64_t rows, uint64_t vocab, int dtype) {
    Plan p;
    const uint32_t units = units_of(vocab, dtype);
    p.threads = units <= 256 ? 64 : 256;
    p.splits = 1;
    p.per_split = units;
    if (rows < 512 && units > 512) {
        const uint32_t wanted = (uint32_t)std::min<uint64_t>(1024 / std::max<uint64_t>(rows, 1), units / 512);
        if (wanted > 1) {
            p.per_split = (units + wanted - 1) / wanted;
            p.splits = (units + p.per_split - 1) / p.per_split;
        }
    }
    return p;
}

uint64_t soft_bytes(uint64_t rows, const Plan &p) { return (rows * p.splits * sizeof(Soft) + 15) / 16 * 16; }

constexpr uint64_t kMostGroups = (1ull << 22) - 1;  // of 1024 lanes

}  // namespace

uint64_t logprobs_workspace(uint64_t rows, uint64_t vocab, uint32_t top, int dtype) {
    const Plan p = plan_rows(rows, vocab, dtype);
    return p.splits == 1 ? 0 : soft_bytes(rows, p) + rows * p.splits * top * sizeof(uint64_t);
}

hipError_t launch_logprobs(const LogProbs &c, hipStream_t stream) {
    const Plan p = plan_rows(c.rows, c.vocab, c.dtype);
    Args a = {};
    a.logits = c.logits;
    a.tokens = c.tokens;
    a.logp = c.logp;
    a.top_logp = c.top_logp;
    a.stats = c.stats;
    a.top_index = c.top_index;
    a.status = c.status;
    a.soft = static_cast<Soft *>(c.ws);
    a.best = reinterpret_cast<uint64_t *>(static_cast<char *>(c.ws) + soft_bytes(c.rows, p));
    a.rows = c.rows;
    a.ld = c.ld;
    a.padding = c.padding;
    a.vocab = (uint32_t)c.vocab;
    a.units = units_of(c.vocab, c.dtype);
    a.splits = p.splits;
    a.per_split = p.per_split;
    a.n_tokens = c.n_tokens;
    a.top = c.top;
    a.token_bytes = c.token_bytes;
    a.scale = c.scale;
    const dim3 grid((uint32_t)std::min(c.rows * p.splits, kMostGroups));
    with_dtype(c.dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto launch = [&](auto k, dim3 g, uint32_t threads) {
            hipLaunchKernelGGL(k, g, dim3(threads), 0, stream, a);
        };
        if (c.top) launch(rows_kernel<DT, true>, grid, p.threads);
        else launch(rows_kernel<DT, false>, grid, p.threads);
        if (p.splits > 1) {
            const dim3 rows((uint32_t)c.rows);  // fewer than 512
            if (c.top) launch(join_kernel<DT, true>, rows, kMaxThreads);
            else launch(join_kernel<DT, false>, rows, kWave);
        }
    });
    return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogProbsGrad &c, hipStream_t stream) {
    GradArgs a = {};
    a.logits = c.logits;
    a.tokens = c.tokens;
    a.stats = c.stats;
    a.d_logp = c.d_logp;
    a.d_entropy = c.d_entropy;
    a.out = c.d_logits;
    a.rows = c.rows;
    a.ld = c.ld;
    a.ld_out = c.ld_out;
    a.padding = c.padding;
    a.vocab = (uint32_t)c.vocab;
    a.tiles = (units_of(c.vocab, c.dtype) + kGradUnits - 1) / kGradUnits;
    a.n_tokens = c.n_tokens;
    a.token_bytes = c.token_bytes;
    a.scale = c.scale;
    const dim3 grid((uint32_t)std::min(c.rows * a.tiles, kMostGroups));
    with_dtype(c.dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto launch = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(kGradThreads), 0, stream, a); };
        if (c.d_entropy) launch(grad_kernel<DT, true>);
        else launch(grad_kernel<DT, false>);
    });
    return hipGetLastError();
}

}  // namespace pc
