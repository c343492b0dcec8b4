// Operands of the 5th-generation tensor cores: shared-memory and instruction
// descriptors, and 4-bit codes to fp16 values.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// Shared-memory matrix descriptor of a K-major operand tile whose rows are 128
// bytes apart with the 128-byte swizzle (8-row atoms of 1024 bytes).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4)  // start address
           | ((uint64_t)1 << 16)                // leading byte offset (unused for swizzled K-major)
           | ((uint64_t)(1024 >> 4) << 32)      // stride byte offset: 8 rows
           | ((uint64_t)1 << 46)                // descriptor version
           | ((uint64_t)2 << 61);               // 128-byte swizzle
}

// Instruction descriptor: fp16 A and B, both K-major, fp32 D, M x N.
__device__ __forceinline__ uint32_t f16_idesc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Eight codes of one word (device nibble order: nibble i holds element
// [0,2,4,6,1,3,5,7][i]) to eight fp16 weights fp16(s * q + b), elements in
// order. (w & 0x000F000F) | 0x6400_6400 is the fp16 pair (1024 + q, 1024 + q')
// exactly; with the mask 0x00F000F0 it is (1024 + 16 q, ...), brought back to
// q by one exact fused multiply-add.
__device__ __forceinline__ uint4 dequant8(uint32_t v, __half2 s2, __half2 b2) {
    const uint32_t M = 0x64006400u;
    const __half2 c1024 = as_h2(0x64006400u);  // (1024, 1024)
    const __half2 inv16 = as_h2(0x2C002C00u);  // (1/16, 1/16)
    const __half2 m64 = as_h2(0xD400D400u);    // (-64, -64)
    const uint32_t u = v >> 8;
    const __half2 q0 = __hsub2(as_h2((v & 0x000F000Fu) | M), c1024);
    const __half2 q1 = __hfma2(as_h2((v & 0x00F000F0u) | M), inv16, m64);
    const __half2 q2 = __hsub2(as_h2((u & 0x000F000Fu) | M), c1024);
    const __half2 q3 = __hfma2(as_h2((u & 0x00F000F0u) | M), inv16, m64);
    uint4 r;
    r.x = as_u32(__hfma2(q0, s2, b2));
    r.y = as_u32(__hfma2(q1, s2, b2));
    r.z = as_u32(__hfma2(q2, s2, b2));
    r.w = as_u32(__hfma2(q3, s2, b2));
    return r;
}

}  // namespace moe
