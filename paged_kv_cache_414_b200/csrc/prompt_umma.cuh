// What prompt attention uses of the fifth-generation tensor cores beside
// umma.cuh: a shorter group of MMAs, and TMEM moves that do not wait.
#pragma once

#include "umma.cuh"

namespace pa {

// Four kind::f16 steps with A in tensor memory (column offsets A0..A3 from
// a_tmem) and B in shared memory (start-address offsets B0..B3), as
// umma_ts_group8 issues eight.  One step: operands %0 D, %1 A, %2 B, %3
// instruction descriptor, %4 accumulate in the first step.
#define PA_TS_STEP(OA, OB, PRED)                                                \
  "add.u32 at, %1, %" #OA ";\n\tadd.u32 bl, b0, %" #OB ";\n\t"                  \
  "mov.b64 db, {bl, bh};\n\t"                                                   \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [at], db, %3, " PRED ";\n\t"
template <uint32_t A0, uint32_t A1, uint32_t A2, uint32_t A3, uint32_t B0, uint32_t B1,
          uint32_t B2, uint32_t B3>
__device__ __forceinline__ void umma_ts_group4(uint32_t d, uint32_t a_tmem, uint64_t b,
                                               uint32_t idesc, uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 b0, bh, bl, at;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
      "mov.b64 {b0, bh}, %2;\n\t"
      PA_TS_STEP(5, 9, "p") PA_TS_STEP(6, 10, "t") PA_TS_STEP(7, 11, "t") PA_TS_STEP(8, 12, "t")
      "}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc0), "n"(A0), "n"(A1), "n"(A2), "n"(A3), "n"(B0),
      "n"(B1), "n"(B2), "n"(B3)
      : "memory");
}
#undef PA_TS_STEP

// 8 consecutive 32-bit TMEM columns of this thread's lane -> registers (and wait).
__device__ __forceinline__ void tmem_load8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// 32 columns without waiting: tmem_load_wait(), then tmem_loaded() on each
// group of registers, before any of them is used.
__device__ __forceinline__ void tmem_load32_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// No instruction: uses of the 32 registers stay behind it (and so behind the wait).
__device__ __forceinline__ void tmem_loaded(uint32_t *r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}

// 32 consecutive TMEM columns <- registers, without waiting.
__device__ __forceinline__ void tmem_store32_async(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

}  // namespace pa
