// Dropout's decisions (shampoo4_train.h): sixteen bits an element from the ten-round Philox
// 4 x 32 generator of Salmon, Moraes, Dror and Shaw (2011).  One call of it, 20 wide
// multiplications, serves eight columns.
#pragma once

#include "train_common.hpp"

namespace s4 {

struct Drop {
    uint32_t threshold;       // dropped below; 0: nothing is
    float scale;              // of what is kept
    uint64_t seed, offset;
    const uint64_t* counter;  // or NULL
};

// offset + counter, read once; in scalar registers, as it is the same for every lane
__device__ __forceinline__ uint64_t drop_call(const Drop& d) {
    const uint64_t c = d.threshold && d.counter ? ldg(d.counter) : 0;
    return d.offset + ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(c >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)c));
}

// a ^ b ^ c in one instruction (its table of results is that of xor)
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0xf0 ^ 0xcc ^ 0xaa);
}
__device__ __forceinline__ u32x4 philox(uint32_t x0, uint32_t x1, uint64_t call, uint64_t seed) {
    uint32_t x2 = (uint32_t)call, x3 = (uint32_t)(call >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    asm volatile("" : "+s"(k0), "+s"(k1));                   // the rounds' keys are added up again, not kept over a loop
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)x0 * 0xd2511f53u, b = (uint64_t)x2 * 0xcd9e8d57u;
        x0 = xor3((uint32_t)(b >> 32), x1, k0);
        x1 = (uint32_t)b;
        x2 = xor3((uint32_t)(a >> 32), x3, k1);
        x3 = (uint32_t)a;
        k0 += 0x9e3779b9u;
        k1 += 0xbb67ae85u;
    }
    return u32x4{x0, x1, x2, x3};
}

// The numbers of eight columns, 8 col8 on, of a row, and which of them are kept: the comparison of a
// half is one of whole words (the lower half brought up, the upper one with what is below it).
struct Keep {
    u32x4 w;
    __device__ __forceinline__ bool operator()(int j, const Drop& d) const {
        return (j & 1 ? w[j >> 1] : w[j >> 1] << 16) >= d.threshold << 16;
    }
};
__device__ __forceinline__ Keep drop_keep8(const Drop& d, uint64_t call, int64_t row, int64_t col8) {
    return {philox((uint32_t)col8, (uint32_t)row, call, d.seed)};
}
// Zeros for what is dropped, whatever it was (the rest has still to be scaled).
__device__ __forceinline__ floatx8 drop8(floatx8 x, const Keep& keep, const Drop& d) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = keep(j, d) ? x[j] : 0.f;
    return x;
}

}  // namespace s4
