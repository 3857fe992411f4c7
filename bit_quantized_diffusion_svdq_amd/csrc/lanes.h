// Exchanges between the lanes of a wave without LDS, and pairs of bf16 values.
#pragma once
#include "common.h"

// The value of another lane of the same 16 (a VALU operand path, no LDS):
// step 0 lane ^ 1, 1 lane ^ 2, 2 mirrored in its 8, 3 mirrored in its 16. A
// reduction that takes steps 0 .. s leaves every lane of 2^(s + 1) the same
// result (after step i all lanes of 2^(i + 1) agree, so mirroring is as good
// as an xor).
template <int STEP>
DEV float lane16_other(float v) {
    constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true));
}

// Two values to two bf16, nearest even, in one conversion (pack_bf16x2 gives
// the same bits in four instructions).
DEV uint32_t bf16x2(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, b2{(__bf16)lo, (__bf16)hi});
}
