// Building blocks of the 16-bit matrix-core tiles: operand streams from memory into swizzled LDS
// stages, fragment reads and waits.
#pragma once

#include "ma_internal.h"

typedef int i32x4 __attribute__((ext_vector_type(4)));
// buffer_load_dwordx4 ... lds: 16 bytes per lane from a buffer resource into LDS, the
// wave's 64 chunks contiguous from LDS byte address m0.  Measured faster than the
// global form (global_load_lds_dwordx4) by 2-6 % on 8192-wide and 13 % on 768-wide
// Gram products.  Declared at file scope: the name binds to the LLVM intrinsic.
__device__ void raw_buffer_load_lds(i32x4 rsrc, __attribute__((address_space(3))) unsigned* lds,
                                    int size, int voffset, int soffset, int offset,
                                    int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace ma {

// 16-byte chunk swizzle inside an operand row (an involution in c).  A fragment read
// has 32 lanes on 32 consecutive rows at one logical chunk (the other half-wave on the
// next chunk).  Both masks were measured free of bank conflicts for that read on gfx950
// (ds_read_b128 throughput at 16 waves per CU equal to the best pattern; the 64-byte
// row mask ((r >> 1) ^ (r >> 3)) & 3, which also looks conflict-free on a plain 64-bank
// model, measured 2-way).
template <int BK>
__device__ __forceinline__ int swz(int r, int c) {
  if constexpr (BK == 64) return c ^ ((r ^ (r >> 3)) & 7);         // 8 chunks per row
  else return c ^ ((r ^ (r >> 2)) & 3);                            // 4 chunks per row
}

// 16-byte chunk swizzle of a k row of the combine's B stage ([BK][BN], n contiguous):
// the transposing reads of one instruction cover 4 consecutive k rows of 64 bytes per
// 16-lane group; XOR-ing the chunk with 4 (r % 4) puts those rows on distinct banks
// (measured conflict-free on gfx950, like (r % 8) combined with higher row bits; with
// no swizzle the read runs at about a third of the rate).
__device__ __forceinline__ int swz_kn(int r, int c) { return c ^ ((r & 3) << 2); }

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 4 bf16 of a column block: lane i of each 16-lane group receives element i % 4 of the
// 8 bytes addressed by lane 4 e + i / 4 of its group, as element e (e = 0..3).
__device__ __forceinline__ s16x4 lds_read_tr(const unsigned short* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}

// wait until at most n vector-memory operations of this wave are outstanding
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  // gfx9 s_waitcnt: vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[5:4] at [15:14]
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// The block-wide step between two operand stages: this wave's LDS reads have completed
// (lgkmcnt(0)), then s_barrier.  After it other waves load the next stages into the
// slots just read, so no read of those slots may be left behind it.  The s_barrier
// builtin does not order memory accesses for the compiler: in the polynomial kernels
// with 128-row tiles it moved a stage's last fragment reads (whose only uses, the
// stage's last MFMAs, follow the barrier) into the block after it, and the results
// changed from run to run.  As one asm statement with a memory clobber neither the
// reads nor the DMAs can cross it.  The builtin lgkmcnt(0) before it is the same wait,
// visible to the compiler's own wait counting.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), vmcnt and expcnt untouched
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}


// Resource of a buffer of `bytes` bytes at the wave-uniform `base` (reads past `bytes`
// return zero: the hardware range check).
__device__ __forceinline__ i32x4 buffer_rsrc(const unsigned short* base, unsigned bytes) {
  const unsigned long long a = reinterpret_cast<unsigned long long>(base);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(a & 0xffffffffu));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32));  // stride 0
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));     // num_records
  r[3] = 0x00020000;  // gfx9 raw buffer: 32-bit data format, no swizzle
  return r;
}

// 16-byte load at byte offset voff (per lane) of that buffer into LDS at l.
//
// kAsm: issued as inline assembly.  The compiler's wait-count pass treats an LDS DMA
// it knows about as a write that may alias any later LDS read carrying a memory
// operand (ds_read_b64_tr_b16 does; the plain fragment reads do not), and put an
// s_waitcnt vmcnt(0) before every transposing read -- each stage then waited for the
// next stage's DMA.  The kernel orders DMA and reads itself (wait_vmcnt on its own
// stage, then s_barrier).  Only the kernels with transposing reads use it: elsewhere
// the intrinsic schedules better (the asm's memory clobber measured 3 % slower on the
// 256-tile kernels that read X^T).
//
// kWait: wait states ahead of the assembly's load, less one.  A scalar register that a vector
// instruction wrote needs five before a buffer load reads it, and the compiler does not count them
// for an assembly statement: where it keeps the base address in vector registers, v_readfirstlane
// came two before the load, which then now and then read another address.  0 is for kernels whose
// listing shows their bases made by scalar instructions (tests search the listings); 4 measured
// 1 % slower on the 20-layer model's optimizer step.
template <bool kAsm, int kWait = 0>
__device__ __forceinline__ void dma16(const unsigned short* base, int voff, unsigned bytes,
                                      unsigned short* l) {
  const i32x4 r = buffer_rsrc(base, bytes);
  if constexpr (kAsm) {
    const int lds = __builtin_amdgcn_readfirstlane(static_cast<int>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned short*)(l))));
    // m0 (the LDS address) is an input operand: the compiler sets it and knows its value
    asm volatile(
        "s_nop %3\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(voff), "s"(r), "{m0}"(lds), "n"(kWait)
        : "memory");
  } else {
    raw_buffer_load_lds(r, (__attribute__((address_space(3))) unsigned*)(l), 16, voff, 0, 0, 0);
  }
}

}  // namespace ma
