// Loads from global memory straight into LDS, written as inline asm.
//
// With the builtins the compiler knows that such a load writes LDS but not which part of it,
// and waits for all of them (s_waitcnt vmcnt(0)) before every LDS read that it sees, prefetches
// of later tiles included: a ring filled ahead of its use is then not ahead at all.  As asm
// the loads are ordered by what the kernel says: each statement clobbers memory, so no LDS read
// moves across it, and the kernel's own s_waitcnt vmcnt(N) and barrier come between a load and
// the reads of what it wrote.  The loads have no result registers, and their operands are read
// when they are issued, so nothing of them is in flight in registers.  Loads that the compiler
// issues itself are waited for correctly beside them: it counts fewer loads in flight than
// there are, so its waits are longer than needed, never shorter.
//
// The destination is the LDS byte offset in m0 plus 16 (4) bytes per lane.  What the compiler
// keeps between instructions that it sees, each statement keeps by itself: one wait state from
// a write of m0 to a load that reads it, and five from a vector instruction's write of a
// scalar register (v_readfirstlane, where the compiler holds a uniform value in a vector one) to
// a load that reads it; m0 and the condition bit are clobbers.  One statement loads all of a
// wavefront's rows (codes) of a stage, so the five states pass once for them.
// Measured against the builtins, whole calls: transposed product of 8192 slots of 8 8-bit
// experts (14336 outputs of 4096 channels) 1348 -> 1074 us, of 777 act-order rows on 4 bits 361 -> 286 us.
#pragma once

#include "nibbles.hpp"

namespace w4a16 {

// Buffer descriptor of `bytes` bytes from p, in scalar registers.
__device__ __forceinline__ u32x4_t direct_rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  u32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32) & 0xFFFFu);
  r[2] = __builtin_amdgcn_readfirstlane(bytes);
  r[3] = kBufferWord3;
  return r;
}

// The warning that m0 is reserved says that it is not kept for the code around a statement;
// that code need not.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// COUNT times 16 bytes per lane, from byte `lane_off[i] + off` of the buffer to lds + STEP i;
// lds and off are the same in every lane.
template <int COUNT, int STEP>
__device__ __forceinline__ void direct_loads16(u32x4_t rsrc, uint32_t lds, const uint32_t (&lane_off)[COUNT], uint32_t off) {
  static_assert(COUNT == 1 || COUNT == 2 || COUNT == 4, "1, 2 or 4 loads");
  const uint32_t to = __builtin_amdgcn_readfirstlane(lds), from = __builtin_amdgcn_readfirstlane(off);
  if constexpr (COUNT == 1)
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 4\n"
        "buffer_load_dwordx4 %3, %1, %2 offen lds"
        :
        : "s"(to), "s"(rsrc), "s"(from), "v"(lane_off[0])
        : "memory", "m0");
  else if constexpr (COUNT == 2)
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 4\n"
        "buffer_load_dwordx4 %4, %1, %2 offen lds\n"
        "s_add_u32 m0, m0, %3\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %5, %1, %2 offen lds"
        :
        : "s"(to), "s"(rsrc), "s"(from), "n"(STEP), "v"(lane_off[0]), "v"(lane_off[1])
        : "memory", "m0", "scc");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 4\n"
        "buffer_load_dwordx4 %4, %1, %2 offen lds\n"
        "s_add_u32 m0, m0, %3\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %5, %1, %2 offen lds\n"
        "s_add_u32 m0, m0, %3\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %6, %1, %2 offen lds\n"
        "s_add_u32 m0, m0, %3\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %7, %1, %2 offen lds"
        :
        : "s"(to), "s"(rsrc), "s"(from), "n"(STEP), "v"(lane_off[0]), "v"(lane_off[1]), "v"(lane_off[2]), "v"(lane_off[3])
        : "memory", "m0", "scc");
}

// BYTES = 16 or 4 per lane from the lane's own address.
template <int BYTES>
__device__ __forceinline__ void direct_load(const void* p, uint32_t lds) {
  static_assert(BYTES == 16 || BYTES == 4, "16 or 4 bytes per lane");
  if constexpr (BYTES == 16)
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "global_load_lds_dwordx4 %1, off"
        :
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p)
        : "memory", "m0");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "global_load_lds_dword %1, off"
        :
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p)
        : "memory", "m0");
}

#pragma clang diagnostic pop

}  // namespace w4a16
