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
constexpr uint32_t kVecs = 2;  // 16-byte loads of a lane on their way together
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kGone = -1000.0f;  // 2^-1000 is 0 in 32 bits, and 0 times -1000 still 0

template <int DT> constexpr uint32_t kPer = DT == PC_F32 ? 4 : 8;  // elements of 16 bytes

template <int DT, bool STREAM>
__device__ __forceinline__ u32x4 load_vec(const typename Plain<DT>::type *p, uint32_t n) {
    if constexpr (DT == PC_F32) {
        if (n == 4) return get<u32x4, 4, STREAM>(p);
        u32x4 r = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < n) r[i] = as_u32(p[i]);
        return r;
    } else {
        return load_raw<DT, STREAM>(p, n).w[0];
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

// The elements from the nth on as -infinity.
template <int DT>
__device__ __forceinline__ u32x4 with_end(u32x4 w, uint32_t n) {
    constexpr uint32_t minus = DT == PC_F32 ? 0xFF800000u : DT == PC_F16 ? 0xFC00u : 0xFF80u;
#pragma unroll
    for (uint32_t i = 0; i < kPer<DT>; ++i) {
        if (i < n) continue;
        if constexpr (DT == PC_F32) w[i] = minus;
        else w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | minus << 16 : (w[i / 2] & 0xFFFF0000u) | minus;
    }
    return w;
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

// Of some elements: the largest one m (-infinity for none), r = m c with
// c = scale log2(e), rounded, and with u = x c - r the sums of 2^u and of
// 2^u u.  Everything is relative to the rounded r, so an exponent takes one
// multiply-add, and what r lost (32 at most, below the bound) is put right once
// at the end.  From the bound on r is held there: neighbouring numbers of 32
// bits then lie 2^64 apart as probabilities, so only elements equal to m count.
// NaN makes s NaN.
struct Soft { float m, r, s, t; };

constexpr float kHeld = 0x1p29f;

__device__ __forceinline__ float held(float v) { return fminf(fmaxf(v, -kHeld), kHeld); }
__device__ __forceinline__ bool is_held(float r) { return fabsf(r) == kHeld; }

__device__ __forceinline__ Soft nothing() { return {-__builtin_inff(), -kHeld, 0.0f, 0.0f}; }

// The same sums for another, larger r (fmaxf takes the other operand where one is NaN).
__device__ __forceinline__ Soft moved(Soft a, float m, float r) {
    const float u = fmaxf(a.r - r, kGone), f = __builtin_amdgcn_exp2f(u);
    return {m, r, a.s * f, f * (a.t + u * a.s)};
}

// An r that was held stands for any m beyond it: only sums of one m go together.
__device__ __forceinline__ Soft moved_exactly(Soft a, float m, float r) {
    if (is_held(r) && a.m != m) return {m, r, a.s != a.s ? a.s : 0.0f, 0.0f};
    return moved(a, m, r);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) { return as_f32(dpp_u32<CTRL>(as_u32(v))); }

// Sum and maximum over a wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f32<0xB1>(v);   // the neighbour in the pair
    v += dpp_f32<0x4E>(v);   // the other pair
    v += dpp_f32<0x141>(v);  // the other half of 8
    v += dpp_f32<0x140>(v);  // the other half of 16
    return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    return fmaxf(fmaxf(from_lane(v, 0), from_lane(v, 16)), fmaxf(from_lane(v, 32), from_lane(v, 48)));
}

__device__ __forceinline__ Soft joined(Soft a, Soft b, float c) {
    const float m = fmaxf(a.m, b.m), r = held(m * c);
    a = moved_exactly(a, m, r);
    b = moved_exactly(b, m, r);
    return {m, r, a.s + b.s, a.t + b.t};
}

// All lanes' joined, the same in every lane.
__device__ __forceinline__ Soft wave_soft(Soft v, float c) {
    const float m = wave_max(v.m);
    v = moved_exactly(v, m, held(m * c));
    return {m, v.r, wave_sum(v.s), wave_sum(v.t)};
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

__device__ __forceinline__ float of_key(uint32_t k) { return as_f32(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    v = max(v, dpp_u32<0x140>(v));
    return max(max(from_lane(v, 0), from_lane(v, 16)), max(from_lane(v, 32), from_lane(v, 48)));
}

// An element as one number: larger ones first, of equal ones that of the lower
// index.  0 stands for no element.
__device__ __forceinline__ uint64_t packed(uint32_t key, uint32_t index) {
    return (uint64_t)key << 32 | (uint32_t)~index;
}

__device__ __forceinline__ uint32_t index_of(uint64_t p) { return ~(uint32_t)p; }

// The value of lane (lane ^ D).  Rows of 16 lanes by DPP; between them by the
// swaps of odd with even rows, and of the halves, of two registers that hold
// the same.
template <uint32_t D>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
    const uint32_t lane = threadIdx.x % kWave;
    if constexpr (D == 1) return dpp_u32<0xB1>(v);
    if constexpr (D == 2) return dpp_u32<0x4E>(v);
    if constexpr (D == 4) return (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x101F);
    if constexpr (D == 8) return dpp_u32<0x128>(v);
    if constexpr (D == 15) return dpp_u32<0x140>(v);
    if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return lane & 16 ? r[0] : r[1];
    }
    if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return lane & 32 ? r[0] : r[1];
    }
}

template <uint32_t D>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
    return (uint64_t)lane_xor<D>((uint32_t)(v >> 32)) << 32 | lane_xor<D>((uint32_t)v);
}

// One step of a bitonic network: lanes D apart exchange, the larger one goes
// to the lane without D where `descends`.
template <uint32_t D, class T>
__device__ __forceinline__ void exchange(T &v, bool descends) {
    const T o = lane_xor<D>(v);
    const bool keep = ((threadIdx.x & D) == 0) == descends;
    v = keep == (v > o) ? v : o;
}

// The last steps of a sort: a list that rises to one place and falls from it
// (or the reverse, or either turned round its end) in descending order.
template <class T>
__device__ __forceinline__ void descend(T &v) {
    exchange<32>(v, true), exchange<16>(v, true), exchange<8>(v, true), exchange<4>(v, true), exchange<2>(v, true),
        exchange<1>(v, true);
}

// A lane's value each, in descending order.  Only the first `n` are not 0: the
// steps for 16 and 32 lanes leave the first half-rows and rows in order, and
// are enough for as many.
template <class T>
__device__ __forceinline__ T sorted(T v, uint32_t n = kWave) {
    const uint32_t l = threadIdx.x;
    exchange<1>(v, !(l & 2));
    exchange<2>(v, !(l & 4)), exchange<1>(v, !(l & 4));
    exchange<4>(v, !(l & 8)), exchange<2>(v, !(l & 8)), exchange<1>(v, !(l & 8));
    exchange<8>(v, !(l & 16)), exchange<4>(v, !(l & 16)), exchange<2>(v, !(l & 16)), exchange<1>(v, !(l & 16));
    if (n <= 16) return v;
    exchange<16>(v, !(l & 32)), exchange<8>(v, !(l & 32)), exchange<4>(v, !(l & 32)), exchange<2>(v, !(l & 32)),
        exchange<1>(v, !(l & 32));
    if (n <= 32) return v;
    descend(v);
    return v;
}

// The 64 largest of two descending lists, descending: the larger ones of one
// list and of the other one turned round.
template <class T>
__device__ __forceinline__ T merged(T a, T b) {
    const T turned = lane_xor<32>(lane_xor<16>(lane_xor<15>(b)));
    a = a > turned ? a : turned;
    descend(a);
    return a;
}

// A wave's largest elements so far, a lane each in descending order, and in
// LDS those that may be among them: 64 of these together are sorted and merged.
constexpr uint32_t kPool = 2 * kWave;

struct Best {
    uint64_t list, least, *pool;  // least: the `top`th of the list
    uint32_t count;
};

__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ uint64_t lane_of(uint64_t v, uint32_t lane) {
    return (uint64_t)from_lane((uint32_t)(v >> 32), lane) << 32 | from_lane((uint32_t)v, lane);
}

__device__ __forceinline__ void settle(Best &b, uint32_t top) {
    const uint32_t lane = threadIdx.x % kWave;
    wave_order();
    const uint64_t v = sorted(lane < b.count ? b.pool[lane] : 0, b.count), rest = b.pool[kWave + lane];
    wave_order();
    b.pool[lane] = rest;
    wave_order();
    b.count = b.count > kWave ? b.count - kWave : 0;
    b.list = b.least ? merged(b.list, v) : v;
    b.least = lane_of(b.list, top - 1);
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

// Joins the waves' sums; wave 0 has the result.
__device__ __forceinline__ void join_softs(Soft &soft, float c, Soft *softs) {
    const uint32_t wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    if (waves == 1) return;
    if (lane == 0) softs[wave] = soft;
    __syncthreads();
    if (wave == 0) soft = wave_soft(lane < waves ? softs[lane] : nothing(), c);
}

// Joins the waves' lists (a power of two); wave 0 has the result.
__device__ __forceinline__ uint64_t join_lists(uint64_t best, uint64_t *lists) {
    const uint32_t wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    lists[wave * kWave + lane] = best;
    for (uint32_t half = waves / 2; half; half /= 2) {
        __syncthreads();
        if (wave < half) {
            best = merged(best, lists[(wave + half) * kWave + lane]);
            lists[wave * kWave + lane] = best;
        }
    }
    return best;
}

// What a lane of the finishing wave needs for its token, loaded early.
struct Picked {
    float x;
    bool inside, bad;
};

template <int DT>
__device__ __forceinline__ Picked pick(const Args &a, uint64_t row) {
    Picked p = {0.0f, false, false};
    const uint32_t lane = threadIdx.x % kWave;
    if (lane < a.n_tokens) {
        const int64_t t = token_at(a.tokens, a.token_bytes, row * a.n_tokens + lane);
        const bool in = t >= 0 && t < (int64_t)a.vocab;
        p.inside = in && t != a.padding;
        p.bad = !in && t != a.padding;
        if (p.inside) p.x = widen((static_cast<const typename Plain<DT>::type *>(a.logits) + row * a.ld)[t]);
    }
    return p;
}

// At most 0, which the last digits of a sum of 1 could pass; NaN stays.
__device__ __forceinline__ float no_more_than_0(float v) { return v > 0.0f ? 0.0f : v; }

// One wave writes a row's results.
template <bool TOP>
__device__ __forceinline__ void finish(const Args &a, uint64_t row, Soft soft, uint64_t best, Picked p) {
    const uint32_t lane = threadIdx.x % kWave;
    const float minus = -__builtin_inff();
    const bool empty = soft.m == minus && soft.s == 0.0f;
    // of m: what r lost; 0 where it was held.  +infinity leaves nothing to compare
    const float lost = is_held(soft.r) ? 0.0f : __builtin_fmaf(soft.m, a.scale * kLog2E, -soft.r);
    const float bits = soft.m == -minus ? __builtin_nanf("") : log2f(soft.s);
    const float log_sum = kLn2 * (bits - lost);
    auto logp_of = [&](float v) { return empty ? minus : no_more_than_0((v - soft.m) * a.scale - log_sum); };
    if (lane < a.n_tokens) a.logp[row * a.n_tokens + lane] = p.inside ? logp_of(p.x) : 0.0f;
    if (p.bad && a.status) *a.status = PC_ERR_INVALID_ARG;
    if constexpr (TOP) {
        if (lane < a.top) {
            a.top_index[row * a.top + lane] = index_of(best);
            a.top_logp[row * a.top + lane] = logp_of(of_key((uint32_t)(best >> 32)));
        }
    }
    if (lane == 0 && a.stats) {
        float *s = a.stats + 4 * row;
        s[0] = soft.m;
        s[1] = empty ? minus : log_sum;
        s[2] = empty ? 0.0f : kLn2 * (bits - soft.t / soft.s);
        s[3] = empty ? minus : soft.m * a.scale + log_sum;
    }
}

constexpr uint32_t kRowThreads = 256, kWideThreads = 512;

constexpr uint32_t kFirst = 2 * kWave;

template <uint32_t THREADS>
struct TopArea {
    uint64_t lists[THREADS], pools[THREADS / kWave * kPool], first[kFirst];
    uint32_t keys[3][THREADS], found;  // keys: a step each for up to 8 waves
    uint8_t strips[THREADS];
};

__device__ __forceinline__ uint32_t lanes_before(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The wave's largest elements of those not below the bound, from the lanes'
// own strips, whose indices grow from step to step: an element equal to the
// `top`th one so far has no place any more.
template <int DT>
__device__ __forceinline__ uint64_t largest_in_order(const Args &a, const typename Plain<DT>::type *x, uint32_t begin,
                                                     uint32_t end, uint32_t bound, uint64_t *pool) {
    constexpr uint32_t N = kPer<DT>;
    Best b = {0, 0, pool, 0};
    for (uint32_t u0 = begin; u0 < end; u0 += blockDim.x) {
        const uint32_t u = u0 + threadIdx.x, n = u < end ? count_before(a.vocab, u * N, N) : 0;
        float v[N];
        widen_vec<DT>(load_vec<DT, false>(x + (uint64_t)u * N, n), v);
        const uint32_t least = max(bound, (uint32_t)(b.least >> 32) + 1);
        uint32_t most = 0;
#pragma unroll
        for (uint32_t i = 0; i < N; ++i) most = max(most, i < n ? key_of(v[i]) : 0);
        if (__ballot(most >= least) == 0) continue;
#pragma unroll
        for (uint32_t i = 0; i < N; ++i) {
            const uint32_t key = key_of(v[i]);
            const uint64_t p = packed(key, u * N + i);
            const bool in = i < n && key >= bound && p > b.least;
            const uint64_t all = __ballot(in);
            if (!all) continue;
            if (in) b.pool[b.count + lanes_before(all)] = p;
            b.count += (uint32_t)__builtin_popcountll(all);
            if (b.count >= kWave) settle(b, a.top);
        }
    }
    if (b.count) settle(b, a.top);
    return b.list;
}

// The row's `top` largest elements in wave 0, a lane each in descending order,
// once every lane knows the largest of the units it has read (its strip, every
// `threads`th unit from its own on).
//
// The `top`th largest of these lanes' largest is at most the `top`th of all
// elements, and hardly less: the largest elements mostly lie in strips of their
// own.  The waves join their lists two by two, all of them in each step, so three
// steps give it to eight waves.  Strips whose largest is below it hold none of
// them; of the few others the wave reads all units again, side by side, and
// takes what is not below the bound: with 256 strips little more than `top`
// elements, which one wave sorts.  Where ties make them more than 128 (a masked
// stretch is equal throughout), the waves go over their strips in order.  So
// the pass over the row does nothing for the alternatives; comparing every
// element with the least one kept so far doubles its work (2048 x 32000 bf16, 20
// of them: 66 us, without them 31).
template <int DT, class AREA>
__device__ __forceinline__ uint64_t largest_elements(const Args &a, const typename Plain<DT>::type *x, uint32_t begin,
                                                     uint32_t end, uint32_t key, AREA &area) {
    constexpr uint32_t N = kPer<DT>;
    const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), threads = blockDim.x;
    const uint32_t nothing = key_of(-__builtin_inff());
    uint32_t best_keys = a.top == 1 ? wave_max(key) : sorted(key);
    if (threads > kWave) {
        if (threadIdx.x == 0) area.found = 0;
        for (uint32_t half = 1, level = 0; half < threads / kWave; half *= 2, ++level) {
            area.keys[level][threadIdx.x] = best_keys;
            __syncthreads();
            const uint32_t other = area.keys[level][(wave ^ half) * kWave + lane];
            best_keys = a.top == 1 ? max(best_keys, other) : merged(best_keys, other);
        }
    }
    const uint32_t bound = max(1u, from_lane(best_keys, a.top - 1));  // 0: fewer lanes than that have read any
    if (from_lane(best_keys, 0) == nothing) {  // masked throughout: the first elements
        const uint64_t index = (uint64_t)begin * N + lane;
        return wave == 0 && index < min((uint64_t)end * N, (uint64_t)a.vocab) ? packed(nothing, (uint32_t)index) : 0;
    }
    const float low = bound > nothing ? of_key(bound) : __builtin_nanf("");  // NaN: all may count
    const uint64_t likely = __ballot(key >= bound);
    const uint32_t count = (uint32_t)__builtin_popcountll(likely);
    uint8_t *strips = area.strips + wave * kWave;
    if (key >= bound) strips[lanes_before(likely)] = (uint8_t)lane;
    wave_order();
    // `wide` lanes to a strip (a power of two), 64 / wide strips at a time
    const uint32_t length = (end - begin + threads - 1) / threads;
    uint32_t log_wide = 0;
    while (log_wide < 6 && (1u << log_wide) < length) ++log_wide;
    const uint32_t wide = 1u << log_wide, together = kWave >> log_wide;
    const uint32_t turns = (length + wide - 1) / wide, parts = (count + together - 1) / together * turns;
    auto load = [&](uint32_t q, uint32_t &u, uint32_t &n) {
        const uint32_t s = q / turns;
        const uint32_t strip = s * together + (lane >> log_wide), k = (q - s * turns) * wide + (lane & (wide - 1));
        u = begin + wave * kWave + strips[min(strip, kWave - 1)] + k * threads;
        n = q < parts && strip < count && k < length && u < end ? count_before(a.vocab, u * N, N) : 0;
        return load_vec<DT, false>(x + (uint64_t)u * N, n);
    };
    uint32_t found = 0, u, n;
    u32x4 w = load(0, u, n);
    for (uint32_t q = 0; q < parts && found <= kFirst; ++q) {
        uint32_t next_u, next_n;
        const u32x4 next = load(q + 1, next_u, next_n);
        float v[N];
        widen_vec<DT>(w, v);
#pragma unroll
        for (uint32_t i = 0; i < N; ++i) {
            if (__ballot(!(v[i] < low)) == 0) continue;
            const uint32_t vk = key_of(v[i]);
            const bool in = i < n && vk >= bound;
            const uint64_t all = __ballot(in);
            if (!all) continue;
            uint32_t at = found;
            if (threads > kWave) {
                if (lane == 0) at = atomicAdd(&area.found, (uint32_t)__builtin_popcountll(all));
                at = uniform(at);
            }
            found = at + (uint32_t)__builtin_popcountll(all);
            at += lanes_before(all);
            if (in && at < kFirst) area.first[at] = packed(vk, u * N + i);
        }
        w = next;
        u = next_u;
        n = next_n;
    }
    if (threads > kWave) {
        __syncthreads();
        found = uniform(area.found);
    } else {
        wave_order();
    }
    if (found > kFirst) {
        const uint64_t list = largest_in_order<DT>(a, x, begin, end, bound, area.pools + wave * kPool);
        return threads > kWave ? join_lists(list, area.lists) : list;
    }
    if (wave) return 0;
    uint64_t list = lane < found ? area.first[lane] : 0;
    if (found == 1) return list;
    list = sorted(list, found);
    if (found <= kWave) return list;
    return merged(list, sorted(kWave + lane < found ? area.first[kWave + lane] : 0, found - kWave));
}

// A workgroup takes a row, or one of `splits` stretches of it: a batch of
// elements gives a maximum first, for which the sums so far are moved if it is
// a new one, then an exponential and two sums an element.  4096 x 128000 bf16:
// 170-172 us a pass of many, 6.1 TB/s (176-191 alone in a trace), with vector work
// in all of the cycles; 511 x 32001 f32 with 4
// tokens and 5 alternatives: 18 us, two workgroups to a CU, 13 without the
// alternatives; 1 x 128000 with 20: 9.4 us in 31 stretches, and 4.8 for the join.
template <int DT, bool TOP, bool STREAM, uint32_t THREADS>
__global__ __launch_bounds__(THREADS, TOP ? 6 : 8) void rows_kernel(Args a) {
    typedef typename Plain<DT>::type T;
    constexpr uint32_t N = kPer<DT>;
    __shared__ Soft softs[kMaxWaves];
    __shared__ std::conditional_t<TOP, TopArea<THREADS>, char> area;
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
                w[j] = load_vec<DT, STREAM>(x + (uint64_t)u * N, n);
            }
        };
        Picked p = {};
        if (a.splits == 1 && tid < kWave) p = pick<DT>(a, row);
        Soft soft = nothing();
        bool careful = false;
        u32x4 w[kVecs];
        load(begin, w);
        for (uint32_t base = begin; base < end; base += step) {
            u32x4 next[kVecs];
            load(base + step, next);
            // the maximum first, then the sums, each from the elements as loaded: wide ones
            // of both loads would take the registers of two of the eight waves
            float m = soft.m;
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) {
                const uint32_t u = base + j * threads + tid;
                const uint32_t n = u < end ? count_before(a.vocab, u * N, N) : 0;
                if (n != N) w[j] = with_end<DT>(w[j], n);
                float v[N];
                widen_vec<DT>(w[j], v);
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) m = fmaxf(m, v[i]);
            }
            const float r = held(m * c);
            soft = moved(soft, m, r);
            auto sums = [&](auto mind, float &s, float &t) {
                s = t = 0.0f;
#pragma unroll
                for (uint32_t j = 0; j < kVecs; ++j) {
                    asm volatile("" : "+v"(w[j]));
                    float v[N];
                    widen_vec<DT>(w[j], v);
#pragma unroll
                    for (uint32_t i = 0; i < N; ++i) {
                        const float y = __builtin_fmaf(v[i], c, -r), e = __builtin_amdgcn_exp2f(y);
                        s += e;
                        t += e * (decltype(mind)::value ? fmaxf(y, kGone) : y);
                    }
                }
            };
            // -infinity makes t NaN (0 times it): a wave that has met one minds it from then on
            float s, t;
            if (!careful) {
                sums(std::false_type(), s, t);
                careful = __ballot(t != t) != 0;
            }
            if (careful) sums(std::true_type(), s, t);
            soft.s += s;
            soft.t += t;
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) w[j] = next[j];
        }
        const uint32_t key = begin + tid < end ? key_of(soft.m) : 0;
        if (is_held(soft.r) && fabsf(soft.m) < __builtin_inff()) {  // count those equal to m
            float same = 0.0f;
            for (uint32_t u = begin + tid; u < end; u += threads) {
                const uint32_t n = count_before(a.vocab, u * N, N);
                float v[N];
                widen_vec<DT>(load_vec<DT, false>(x + (uint64_t)u * N, n), v);
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) same += i < n && v[i] == soft.m ? 1.0f : 0.0f;
            }
            if (soft.s == soft.s) soft.s = same;
            soft.t = 0.0f;
        }
        soft = wave_soft(soft, c);
        uint64_t list = 0;
        if constexpr (TOP) list = largest_elements<DT>(a, x, begin, end, key, area);
        join_softs(soft, c, softs);
        if (tid < kWave) {
            if (a.splits == 1) {
                finish<TOP>(a, row, soft, list, p);
            } else {
                if (tid == 0) a.soft[id] = soft;
                if (TOP && tid < a.top) a.best[id * a.top + tid] = list;
            }
        }
        __syncthreads();  // the next turn writes the areas that wave 0 has read
    }
}

// The stretches of a row joined: a lane takes the sums of one each (there are 512
// at most, and the launch has lanes for all), with alternatives or without, so
// these change no sum's order; a wave takes every 16th list, in order.
template <int DT, bool TOP>
__global__ __launch_bounds__(kMaxThreads) void join_kernel(Args a) {
    __shared__ Soft softs[kMaxWaves];
    __shared__ uint64_t lists[TOP ? kMaxThreads : 1];
    const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
    const float c = a.scale * kLog2E;
    const uint64_t row = blockIdx.x;
    Picked p = {};
    if (wave == 0) p = pick<DT>(a, row);
    Soft soft = nothing();
    uint64_t best = 0;
    if (threadIdx.x < a.splits) soft = joined(soft, a.soft[row * a.splits + threadIdx.x], c);
    soft = wave_soft(soft, c);
    if constexpr (TOP) {
        for (uint32_t s = wave; s < a.splits; s += waves)
            best = merged(best, lane < a.top ? a.best[(row * a.splits + s) * a.top + lane] : 0);
    }
    if constexpr (TOP) best = join_lists(best, lists);
    join_softs(soft, c, softs);
    if (wave == 0) finish<TOP>(a, row, soft, best, p);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

constexpr uint32_t kGradThreads = 256;
constexpr uint32_t kGradVecs = 2;  // 4096 x 128000 bf16 with an entropy: one 420 us, two 367, four 368
constexpr uint32_t kGradUnits = kGradThreads * kGradVecs;

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

template <int DT, bool ENTROPY, bool STREAM>
__global__ __launch_bounds__(kGradThreads) void grad_kernel(GradArgs a) {
    typedef typename Plain<DT>::type T;
    constexpr uint32_t N = kPer<DT>;
    const uint32_t lane = threadIdx.x % kWave, total = (uint32_t)a.rows * a.tiles;
    for (uint32_t id = blockIdx.x; id < total; id += gridDim.x) {
        const uint32_t row = id / a.tiles, unit0 = (id - row * a.tiles) * kGradUnits;
        const T *x = static_cast<const T *>(a.logits) + row * a.ld;
        T *out = static_cast<T *>(a.out) + row * a.ld_out;
        u32x4 w[kGradVecs];
        uint32_t n[kGradVecs];
#pragma unroll
        for (uint32_t j = 0; j < kGradVecs; ++j) {
            const uint32_t u = unit0 + j * kGradThreads + threadIdx.x;
            n[j] = count_before(a.vocab, u * N, N);
            w[j] = load_vec<DT, STREAM>(x + (uint64_t)u * N, n[j]);
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
        const bool none = (__ballot(d != 0.0f) == 0 && de == 0.0f) || (largest == -__builtin_inff() && log_sum == log_sum);
        if (none) {
            const float zeros[N] = {};
#pragma unroll
            for (uint32_t j = 0; j < kGradVecs; ++j)
                if (n[j]) store_vec<DT>(out + (uint64_t)(unit0 + j * kGradThreads + threadIdx.x) * N, n[j], zeros);
            continue;
        }
        const uint64_t inside = __ballot(token >= (int64_t)unit0 * N && token < ((int64_t)unit0 + kGradUnits) * N);
        const uint32_t at = (uint32_t)token;
        // log2 p = x c - r - less:  r is largest c rounded, `less` has what that lost
        const float c = a.scale * kLog2E, r = largest * c;
        const bool huge = !(fabsf(r) < kHeld);
        const float less = __builtin_fmaf(log_sum, kLog2E, __builtin_fmaf(largest, c, -r));
        const float base = a.scale * (sum + de * entropy), slope = a.scale * de * kLn2;
#pragma unroll
        for (uint32_t j = 0; j < kGradVecs; ++j) {
            if (!n[j]) continue;
            const uint32_t u = unit0 + j * kGradThreads + threadIdx.x;
            float v[N];
            widen_vec<DT>(w[j], v);
#pragma unroll
            for (uint32_t i = 0; i < N; ++i) {
                float y = __builtin_fmaf(v[i], c, -r) - less;
                if (huge) y = ((v[i] - largest) * a.scale - log_sum) * kLog2E;
                const float p = __builtin_amdgcn_exp2f(y);
                float g = base;
                if constexpr (ENTROPY) g += slope * fmaxf(y, kGone);
                v[i] = -p * g;
            }
            for (uint64_t left = inside; left; left &= left - 1) {
                const uint32_t l = (uint32_t)__builtin_ctzll(left);
                const uint32_t place = from_lane(at, l) - u * N;
                const float add = a.scale * from_lane(d, l);
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) v[i] += place == i ? add : 0.0f;
            }
            store_vec<DT>(out + (uint64_t)u * N, n[j], v);
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

uint32_t units_of(uint64_t vocab, int dtype) { return (uint32_t)((vocab + (dtype == PC_F32 ? 3 : 7)) / (dtype == PC_F32 ? 4 : 8)); }

// Logits of so many bytes, which the memory-side cache does not hold, stream
// past the caches (4096 x 128000 bf16: 192 us, streamed 168; 2048 x 32000: 29.6
// and 28.1; 511 x 32001 f32, 62 MiB: 14.5 and 17.7).
constexpr uint64_t kStreamBytes = 128ull << 20;

bool streams(uint64_t rows, uint64_t vocab, int dtype) { return rows * vocab * (dtype == PC_F32 ? 4 : 2) >= kStreamBytes; }

struct Plan { uint32_t threads, splits, per_split; };

constexpr uint32_t kMostSplits = 512;  // of all rows together
static_assert(kMostSplits <= kMaxThreads, "the join has a lane for each");

// Stretches of so many 16-byte units get 512 lanes: where that leaves no more than
// two workgroups to a CU, for the loads on their way, and longer ones always, for
// their alternatives, whose strips are then half as long.  With 256 lanes and 512:
// 511 x 32001 f32 without alternatives 15.3 and 13.4 us, with 20 23.5 and 19.4;
// 512 x 128000 bf16 37.9 and 28.4, 50.1 and 36.3; 256 x 50257 bf16 (2 x 3142 units)
// 13.9 and 14.0, 21.9 and 21.7.  2048 x 128000 f32 159 and 157, 261 and 199; 4096 x
// 128000 bf16 170 and 164, with 5 189 and 194, with 20 248 and 218; 1024 x 32000 f32
// 26.4 and 27.0, 36.6 and 39.3.  1024 lanes: 222 for 2048 x 128000 f32 with 20.
constexpr uint32_t kWideFrom = 4096, kAlwaysWideFrom = 12288;

// A wave to a row where the rows fill the chip with waves and are short, or
// hold no more than a wave's loads (8192 x 4000 bf16: 18 us, with four waves
// 39; 2048 x 32000: 31 and 28).  Few rows are split, down to what a workgroup
// loads at once, until there are two workgroups to a CU (1 x 128000: 6.8 us,
// whole 20).
Plan plan_rows(uint64_t rows, uint64_t vocab, int dtype) {
    Plan p;
    const uint32_t units = units_of(vocab, dtype);
    p.threads = units <= kRowThreads || (rows >= 4096 && units <= 1024) ? kWave : kRowThreads;
    p.splits = 1;
    p.per_split = units;
    const uint32_t least = kRowThreads * kVecs;
    if (rows <= 256 && units >= 2 * least) {
        const uint32_t wanted = (uint32_t)std::min<uint64_t>(kMostSplits / std::max<uint64_t>(rows, 1), units / least);
        p.per_split = (units + wanted - 1) / wanted;
        p.splits = (units + p.per_split - 1) / p.per_split;
    }
    if (p.per_split >= (rows * p.splits <= 512 ? kWideFrom : kAlwaysWideFrom)) p.threads = kWideThreads;
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
        const bool stream_in = streams(c.rows, c.vocab, c.dtype);
        auto rows_of = [&](auto t) {
            constexpr uint32_t T = decltype(t)::value;
            if (c.top && stream_in) launch(rows_kernel<DT, true, true, T>, grid, p.threads);
            else if (c.top) launch(rows_kernel<DT, true, false, T>, grid, p.threads);
            else if (stream_in) launch(rows_kernel<DT, false, true, T>, grid, p.threads);
            else launch(rows_kernel<DT, false, false, T>, grid, p.threads);
        };
        // an area for a wave's own lanes alone leaves LDS for 24 of them (8192 x 1000 with 20
        // alternatives: 18 us, with that of 256 lanes 24)
        if (p.threads == kWave) rows_of(std::integral_constant<uint32_t, kWave>());
        else if (p.threads == kWideThreads) rows_of(std::integral_constant<uint32_t, kWideThreads>());
        else rows_of(std::integral_constant<uint32_t, kRowThreads>());
        if (p.splits > 1) {
            const dim3 rows((uint32_t)c.rows);  // 256 at most
            if (c.top) launch(join_kernel<DT, true>, rows, kMaxThreads);
            else launch(join_kernel<DT, false>, rows, (p.splits + kWave - 1) / kWave * kWave);
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
        const bool stream_in = streams(c.rows, c.vocab, c.dtype);
        if (c.d_entropy && stream_in) launch(grad_kernel<DT, true, true>);
        else if (c.d_entropy) launch(grad_kernel<DT, true, false>);
        else if (stream_in) launch(grad_kernel<DT, false, true>);
        else launch(grad_kernel<DT, false, false>);
    });
    return hipGetLastError();
}

}  // namespace pc
