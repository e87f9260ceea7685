// ssd_tc.cuh -- what the kernels on the tensor cores share: bounded waits, TMA copies of a
// paged cache's tiles, tcgen05 instructions and descriptors, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd_async.cuh"
#include "ssd_kv.cuh"

namespace ssd {

constexpr int kTile = 128;           // slots of a tile (rows of the ring's tiles)
constexpr int kHalf = kTile * 128;   // bytes of a tile's 64-column half
constexpr int kSmemMax = 227 * 1024;

// ---------------------------------------------------------------------------
// mbarriers, TMA, tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sptr(b)) : "memory");
}
// Bounded wait (Misc: a CTA's wait_us and abort in shared memory): after wait_us (or once another wait of the CTA gave up) the CTA
// runs on without waiting, to its end; the error word says so.
template <class Misc>
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, Misc& sm, int* err) {
  unsigned long long t0 = 0;
  for (unsigned i = 1;; ++i) {
    if (bar_try(b, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if ((i & 31) == 0) {  // the global timer is slow to read
      const unsigned long long t = now_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > sm.wait_us * 1000ull) {
        *reinterpret_cast<volatile int*>(&sm.abort) = 1;
        atomicOr(err, kErrTimeout);
        return false;
      }
    }
  }
}

// The same in few instructions where the phase ends within the first try's 20 us (code that
// runs once a tile or less comes from far when it runs).
inline __device__ __noinline__ bool bar_await_more(uint64_t* b, uint32_t parity, volatile int* abort, unsigned wait_us,
                                                   int* err) {
  const unsigned long long t0 = now_ns();
  while (true) {
    if (bar_try(b, parity)) return true;
    if (*abort) return false;
    if (now_ns() - t0 > wait_us * 1000ull) {
      *abort = 1;
      __threadfence_block();  // (before what runs on without its data)
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}
template <class Misc>
__device__ __forceinline__ bool bar_await(uint64_t* b, uint32_t parity, Misc& sm, int* err) {
  if (bar_try(b, parity)) return true;
  return bar_await_more(b, parity, &sm.abort, sm.wait_us, err);
}

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int d, int slot, int head,
                                         int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(sptr(bar)), "r"(d), "r"(slot), "r"(head), "r"(page)
      : "memory");
}

// As tma_rows for whole groups of 8 slots, both 64-column halves in one copy.
__device__ __forceinline__ void tma_groups(uint32_t dst, const CUtensorMap* map, int group, int head,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(sptr(bar)), "r"(0), "r"(group), "r"(head)
      : "memory");
}

// Four rows of 64 columns from column x on.
__device__ __forceinline__ void tma_gather(uint32_t dst, const CUtensorMap* map, int x, const int (&row)[4],
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(sptr(bar)), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3])
      : "memory");
}

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   sptr(b))
               : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

// The same with A in tensor memory (16-bit entries, two a column).
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

// Shared-memory operand descriptor: strides in bytes; swizzle 2: 128 bytes,
// 6: 32 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride, uint64_t swizzle = 2) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (swizzle << 61);
}
// Instruction descriptor: 32-bit accumulator, 128 x n, 16-bit operands.
template <class T>
__device__ __forceinline__ uint32_t instr(int n, bool a_mn, bool b_mn, bool negate_a = false) {
  const uint32_t f = T::kId == Bf16::kId ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(negate_a) << 13) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// 32 lanes x 32 columns of tensor memory: a lane a thread, register i its column i.
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]));
}
// The same with 16 columns (named apart: the tree attention has fragments of its own).
__device__ __forceinline__ void tm_put16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void tm_get16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tm_tie16(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tm_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Waits for this thread's tcgen05.ld; tm_tie32 behind it keeps the uses of their
// registers behind it, too.
__device__ __forceinline__ void tm_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_tie32(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
    "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
    "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) !=
            cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

inline CUtensorMapDataType map_type(int dtype) {
  return dtype == Bf16::kId ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// {D, page_size, Hkv, pages}; boxes of 64 columns and `box` slots of one head
// of one page.
inline bool encode_rows(CUtensorMap* m, void* base, int dtype, int D, int ps, int H, int pages, long long slot,
                 long long head, long long page, int box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(ps),
                              static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(slot) * 2, static_cast<cuuint64_t>(head) * 2,
                                 static_cast<cuuint64_t>(page) * 2};
  const cuuint32_t bx[4] = {64, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, map_type(dtype), 4, base, dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Groups of 8 slots a page apart, where the cache's strides make the slots of
// all pages one sequence of such groups; 0 where they don't, or where a box (0: a
// page's part of a tile) could run over a page's end.
inline long long page_groups(int ps, int pages, long long slot, long long page, int box = 0) {
  if (box ? ps % box != 0 : ps % 8 != 0 || (ps > kTile && ps % kTile != 0) || (ps < kTile && kTile % ps != 0)) return 0;
  if (page % (8 * slot) != 0) return 0;
  const long long g = page / (8 * slot);
  return g >= ps / 8 && g * (pages + 1ll) < (1ll << 31) ? g : 0;
}

// {64, 8 slots, 2 halves, groups, Hkv}; boxes of `box` slots.
inline bool encode_groups(CUtensorMap* m, void* base, int dtype, int ps, int H, int pages, long long slot, long long head,
                   long long groups, int box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(groups * (pages - 1) + ps / 8),
                              static_cast<cuuint64_t>(H)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(slot) * 2, 128, static_cast<cuuint64_t>(slot) * 16,
                                 static_cast<cuuint64_t>(head) * 2};
  const cuuint32_t bx[5] = {64, 8, 2, static_cast<cuuint32_t>(box / 8), 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return fn(m, map_type(dtype), 5, base, dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// {columns, rows}; four rows of 64 columns at a time, each by its number.
inline bool encode_gather(CUtensorMap* m, void* base, int dtype, long long columns, long long rows, long long slot) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(slot) * 2};
  const cuuint32_t bx[2] = {64, 1}, one[2] = {1, 1};
  return fn(m, map_type(dtype), 2, base, dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

}  // namespace ssd
