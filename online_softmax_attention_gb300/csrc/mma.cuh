// The 16 x 8 x 16 matrix instruction on 16-bit values with f32 sums, for contractions whose
// few rows a 128-row tcgen05 tile would leave empty.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace attn {

// d += a b.  Lane (g, c) = (lane / 4, lane % 4) holds a: rows g, g + 8 (registers 0, 1) of
// columns 2 c, 2 c + 1, and the same rows of columns 2 c + 8, + 9 (2, 3); b: rows 2 c, 2 c + 1
// and 2 c + 8, + 9 of column g; d: row g, columns 2 c, 2 c + 1, and row g + 8.
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (sizeof(T) == 2) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

}  // namespace attn
