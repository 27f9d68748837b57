// rows_out.cuh -- accumulator rows on their way from TMEM to global memory in runs of 64 bytes of 8 rows.
#pragma once

#include <cstdint>

namespace fa {
namespace {

// 16 TMEM lanes x 64 columns, lane 4 r + q of the warp holding columns 8 j + 2 q, + 1 of rows r
// (x[4 j], x[4 j + 1]) and r + 8 (x[4 j + 2], x[4 j + 3]).
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
          "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
          "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
          "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(taddr)
        : "memory");
}
// Lane q of every four holds word q of four 16-byte pieces; afterwards lane q holds piece q.
__device__ __forceinline__ void transpose4(uint32_t& a0, uint32_t& a1, uint32_t& a2, uint32_t& a3, int q) {
    const bool odd = q & 1, high = q & 2;
    uint32_t r = __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
    (odd ? a0 : a1) = r;
    r = __shfl_xor_sync(0xffffffffu, odd ? a2 : a3, 1);
    (odd ? a2 : a3) = r;
    r = __shfl_xor_sync(0xffffffffu, high ? a0 : a2, 2);
    (high ? a0 : a2) = r;
    r = __shfl_xor_sync(0xffffffffu, high ? a1 : a3, 2);
    (high ? a1 : a3) = r;
}

}  // namespace
}  // namespace fa
