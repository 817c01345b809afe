// Dropout's mask: numbers made again from a counter wherever they are needed.
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products on
// a counter of four words.  The counter is (col / 8, row, offset), the key the
// seed, so the mask belongs to the element's place and not to how a launch
// splits the tensor.  One call gives the 8 columns of a lane 16 bits each: an
// element is dropped where they are below 65536 p.  32 bits an element would
// cost two calls, and the products (16 cycles of a wave each) would then take
// longer than HBM takes for 16-bit tensors.
#pragma once

#include "q8.h"

namespace pc {

struct MaskArg {
    uint64_t seed, offset;
    const uint64_t *random;  // nullptr, or seed and an offset to add, in device memory
    uint32_t below;          // numbers below it are dropped; 0: nothing is
    float keep;              // what the others are multiplied by
};

// A mask as the entry points take it: p in [0, 1], or none.
inline MaskArg mask_arg(const pc_mask *m) {
    MaskArg a = {0, 0, nullptr, 0, 1.0f};
    if (m) {
        a.seed = m->seed;
        a.offset = m->offset;
        a.random = m->d_random;
        a.below = (uint32_t)__builtin_rint(m->p * 65536.0);
        a.keep = a.below < 65536 ? (float)(65536.0 / (65536.0 - a.below)) : 0.0f;
    }
    return a;
}

struct MaskKey {
    uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ MaskKey mask_key(const MaskArg &m) {
    uint64_t seed = m.seed, offset = m.offset;
    if (m.random) {
        seed = m.random[0];
        offset += m.random[1];
    }
    return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// a ^ b ^ c in one instruction (its table: the parity of three bits).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, MaskKey k) {
    uint32_t c2 = k.c2, c3 = k.c3, k0 = k.k0, k1 = k.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = xor3((uint32_t)(b >> 32), c1, k0);
        c1 = (uint32_t)b;
        c2 = xor3((uint32_t)(a >> 32), c3, k1);
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// Drops from the 8 values of columns [col, col + 8) of a row, col a multiple
// of 8, and multiplies the others.
__device__ __forceinline__ void drop_unit(const MaskArg &m, MaskKey k, uint64_t row, uint32_t col, float v[8]) {
    const u32x4 r = philox(col / kUnit, (uint32_t)row, k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t bits = i % 2 ? r[i / 2] >> 16 : r[i / 2] & 0xFFFFu;
        v[i] = bits < m.below ? 0.0f : v[i] * m.keep;
    }
}

}  // namespace pc
