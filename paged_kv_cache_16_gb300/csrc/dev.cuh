// Device-side building blocks for sm_103a: mbarriers with bounded waits,
// TMA tensor loads, legacy warp MMA fragments, and the tcgen05 (5th-gen
// tensor core + tensor memory) instructions, all as inline PTX.
#pragma once
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa_internal.h"

namespace pa {
namespace dev {

// A wait gives up after this many nanoseconds of %globaltimer; the kernel
// then records kErrTimeout and winds down instead of hanging the GPU.
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// ---------------------------------------------------------------- mbarrier --
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for the phase with the given parity to complete.  Returns false if the
// CTA-wide abort flag is raised or the time limit passes (the caller then
// records the error and stops).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
#pragma unroll 1
    for (int i = 0; i < 128; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const uint64_t start = global_timer();
#pragma unroll 1
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (abort_flag != nullptr && *abort_flag) return false;
        if (global_timer() - start > kWaitLimitNs) return false;
    }
}

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Like mbar_wait but never suspends the thread (non-blocking test_wait in a
// spin): for the single thread that issues the tensor-core MMAs, where the
// wake-up latency of a suspended wait shows up as tensor-core idle time.
__device__ __forceinline__ bool mbar_wait_spin(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
        if (mbar_test_wait(bar, parity)) return true;
    const uint64_t start = global_timer();
#pragma unroll 1
    while (true) {
        if (mbar_test_wait(bar, parity)) return true;
        if (abort_flag != nullptr && *abort_flag) return false;
        if (global_timer() - start > kWaitLimitNs) return false;
    }
}

// mbar_wait_spin by every lane of a warp, with one warp-wide (uniform) answer.
__device__ __forceinline__ bool warp_wait_spin(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    const uint64_t start = global_timer();
#pragma unroll 1
    while (true) {
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, (abort_flag != nullptr && *abort_flag) || global_timer() - start > kWaitLimitNs))
            return false;
    }
}

// mbar_wait by every lane of a warp, with one warp-wide answer: either all
// lanes go on or all stop (keeps later warp-collective instructions legal).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    const bool ok = mbar_wait(bar, parity, abort_flag);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void raise_abort(volatile int *abort_flag, int32_t *err, int bits) {
    *abort_flag = 1;
    atomicOr(err, bits);
}

// ------------------------------------------- programmatic dependent launch --
// launch_dependents: the next kernel in the stream (launched with the
// programmatic-serialisation attribute) may start its prologue now.
// dep_wait: block until the previous kernel in the stream has completed and
// its memory is visible; every kernel launched with the attribute calls it
// before it reads or writes anything an earlier kernel touches (a no-op when
// launched without the attribute).
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// --------------------------------------------------------------------- TMA --
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap *tm) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}

// 3-D tiled TMA load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int32_t c0,
                                            int32_t c1, int32_t c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Same, with an L2 eviction-priority hint (createpolicy result).
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap *tm, int32_t c0,
                                                 int32_t c1, int32_t c2, uint32_t bar,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

// Asks `bytes` bytes of global memory into L2 (address and size multiples of 16).
__device__ __forceinline__ void bulk_prefetch_l2(const void *src, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(src)), "r"(bytes) : "memory");
}

// Contiguous bulk load (both addresses 16-byte aligned, bytes a multiple of
// 16) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 32-byte global store (one whole sector per lane)
__device__ __forceinline__ void st_global_v8(void *p, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t a4,
                                             uint32_t a5, uint32_t a6, uint32_t a7) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a0), "r"(a1), "r"(a2),
                 "r"(a3), "r"(a4), "r"(a5), "r"(a6), "r"(a7)
                 : "memory");
}

// The same 32 bytes of an output row, whose address is a multiple of 32 (`wide`) or
// of 16 alone, where one 32-byte store would be misaligned.
__device__ __forceinline__ void st_row_v8(bool wide, void *p, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t a4, uint32_t a5, uint32_t a6, uint32_t a7) {
    if (wide) {
        st_global_v8(p, a0, a1, a2, a3, a4, a5, a6, a7);
    } else {
        uint4 *q = static_cast<uint4 *>(p);
        q[0] = make_uint4(a0, a1, a2, a3);
        q[1] = make_uint4(a4, a5, a6, a7);
    }
}

__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Generic-proxy writes to shared memory become visible to the async proxy
// (TMA, tensor core) after this fence.
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// generic-proxy global stores of this thread before later async-proxy (TMA)
// reads of the same addresses
__device__ __forceinline__ void fence_proxy_async_global() {
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

// ------------------------------------------------------------ conversions --
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// two floats -> f16x2 (lo in the low half), round to nearest
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// two floats -> two E4M3 codes (lo in the low byte): nearest, ties to even,
// saturating to +-448 (NaN stays NaN)
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The E4M3 cache write of two bf16 elements (low half first): the codes of
// x / scale, the quotient rounded once in IEEE binary32 (low byte first).
__device__ __forceinline__ uint16_t e4m3_quantize2(uint32_t bf16x2, float scale) {
    return pack_e4m3x2(__fdiv_rn(__uint_as_float(bf16x2 << 16), scale),
                       __fdiv_rn(__uint_as_float(bf16x2 & 0xFFFF0000u), scale));
}

// Eight bf16 elements (16 bytes) -> their eight E4M3 codes (8 bytes).
__device__ __forceinline__ uint2 e4m3_quantize8(uint4 v, float scale) {
    return make_uint2(static_cast<uint32_t>(e4m3_quantize2(v.x, scale)) |
                          (static_cast<uint32_t>(e4m3_quantize2(v.y, scale)) << 16),
                      static_cast<uint32_t>(e4m3_quantize2(v.z, scale)) |
                          (static_cast<uint32_t>(e4m3_quantize2(v.w, scale)) << 16));
}

// two E4M3 codes (low byte first) -> f16x2; every E4M3 value is exact in f16
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes16) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes16)));
    return r;
}

// four E4M3 codes (one 32-bit word, lowest byte first) -> two f16x2 words
__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// byte permute of the pair {b:a} (bytes 0-3 from a, 4-7 from b)
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

__device__ __forceinline__ float f16_lo(uint32_t v) {
    float f;
    asm("{\n\t.reg .f16 h;\n\tmov.b32 {h, _}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
    return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v) {
    float f;
    asm("{\n\t.reg .f16 h;\n\tmov.b32 {_, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
    return f;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Packed fp32 pairs (one 64-bit register pair, low element first) and the
// paired FMA / add of the sm_100 family; 3-input max.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A block scale as attention uses it: at least 2^-100 (a NaN stays one).
__device__ __forceinline__ float used_scale(float s) { return s < 0x1p-100f ? 0x1p-100f : s; }

// What a code product is multiplied by to be a score: a * b, at least 2^-149 where
// that underflows to 0 (a masked score of -infinity times 0 would be NaN; the
// scores of such a block are 0 up to 2^-20 either way).  A NaN stays one.
__device__ __forceinline__ float score_factor(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a * b), "f"(0x1p-149f));
    return y;
}

// Four codes (one word, lowest byte first) -> two f16x2 words, exact.  int8:
// the byte plus 128 as the low mantissa bits of 1024 + byte, minus 1152.
template <bool INT8>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (INT8) {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = prmt(u, 0x64646464u, 0x4140u), b = prmt(u, 0x64646464u, 0x4342u);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    } else {
        e4m3x4_to_f16x2x2(w, lo, hi);
    }
}

// ---------------------------------------------- legacy warp MMA (mma.sync) --
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t &r0, uint32_t &r1,
                                            uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t &r0, uint32_t &r1,
                                                  uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// 8x8 transpose of 16-bit elements across the warp: lane 4r + c holds
// elements (r, 2c) and (r, 2c + 1) of the matrix before and of its
// transpose after.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// D = A(16x16 bf16, row) * B(16x8 bf16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A(16x16 f16, row) * B(16x8 f16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same into D = A * B.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16-byte global -> shared copy that completes asynchronously (no register
// staging); cp_async_wait_all waits for the calling thread's copies.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {   // all but the newest N groups of the calling thread
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Address of the 16-byte chunk `chunk` (0..7) of row `row` inside a tile of
// 128-byte rows written by TMA with 128-byte swizzling (tile base 1024-aligned).
__device__ __forceinline__ uint32_t sw128(uint32_t base, uint32_t row, uint32_t chunk) {
    return base + row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// ------------------------------------------------------------ partials --
// Merge of partition partials for one query head, by one warp (page
// "vLLM 源码完全拆解（十六）", third walk-through: local (m_r, l_r, o_r)
// combined with exponential rescaling; m in log2 units here):
//   m = max m_r,  w_r = 2^(m_r - m) l_r,  out = sum w_r o_r / sum w_r.
// Partials are read in slot order, so the result does not depend on which
// CTA or kernel performs the merge.
template <int D, int KPRE>
__device__ __forceinline__ void merge_head(uint16_t *out_row, const float *o_part, const float2 *ml_part,
                                           int64_t slot0, int count, int num_heads_q, int h, int lane) {
    constexpr int V = D / 32;
    // The o rows of the first KPRE partials are loaded together with the
    // (m, l) pairs, before the weights are known, so that a merge of up to
    // KPRE partials costs one round trip to L2 instead of three; a partial
    // whose l is 0 was never written and its o is skipped (not multiplied
    // by 0: it may hold anything).  L2 loads: partials written by other SMs
    // in this same launch must not be served from a stale L1 line.
    using VecT = typename std::conditional<V == 4, float4, float2>::type;
    auto o_at = [&](int j) {
        return reinterpret_cast<const VecT *>(o_part + ((slot0 + j) * num_heads_q + h) * D + lane * V);
    };
    VecT pre[KPRE];
#pragma unroll
    for (int j = 0; j < KPRE; ++j)
        if (j < count) pre[j] = __ldcg(o_at(j));
    // lane s holds (m, l) of partial s of each group of 32
    float2 ml0 = make_float2(-INFINITY, 0.f);
    if (lane < count) ml0 = __ldcg(ml_part + (slot0 + lane) * num_heads_q + h);
    float m = ml0.y > 0.f ? ml0.x : -INFINITY;
    for (int s0 = 32; s0 < count; s0 += 32) {
        if (s0 + lane < count) {
            const float2 ml = __ldcg(ml_part + (slot0 + s0 + lane) * num_heads_q + h);
            if (ml.y > 0.f) m = fmaxf(m, ml.x);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    auto add = [&](float wj, const VecT &x) {
        if constexpr (V == 4) {
            acc[0] += wj * x.x; acc[1] += wj * x.y; acc[2] += wj * x.z; acc[3] += wj * x.w;
        } else {
            acc[0] += wj * x.x; acc[1] += wj * x.y;
        }
    };
    float wsum = 0.f;   // this lane's partials' weights
    for (int s0 = 0; s0 < count; s0 += 32) {
        float w = 0.f;
        if (s0 + lane < count) {
            const float2 ml = s0 == 0 ? ml0 : __ldcg(ml_part + (slot0 + s0 + lane) * num_heads_q + h);
            if (ml.y > 0.f) w = ex2(ml.x - m) * ml.y;
        }
        wsum += w;
        const int n = min(32, count - s0);
        if (s0 == 0) {
#pragma unroll
            for (int j = 0; j < KPRE; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                if (j < n && wj != 0.f) add(wj, pre[j]);
            }
        }
#pragma unroll 4
        for (int j = s0 == 0 ? KPRE : 0; j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            if (wj == 0.f) continue;   // empty partial: its o was never written
            add(wj, __ldcg(o_at(s0 + j)));
        }
    }
    float total = wsum;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = total > 0.f ? 1.f / total : 0.f;
    uint16_t *dst = out_row + static_cast<int64_t>(h) * D + lane * V;
    if constexpr (V == 4) {
        uint2 packed;
        packed.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        packed.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2 *>(dst) = packed;
    } else {
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
}

// ---------------------------------------------------------------- tcgen05 --
// Shared-memory matrix descriptor, 128-byte swizzle.  Start address, leading
// and stride byte offsets in 16-byte units; descriptor version 1 (bits 46-47);
// swizzle mode 2 = 128B (bits 61-63).
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// A shared-memory descriptor moved by `bytes` (a multiple of 16 that keeps
// the start address inside the 18-bit window): only the low word changes,
// one add instead of rebuilding the descriptor.
__device__ __forceinline__ uint64_t sdesc_advance(uint64_t d, uint32_t bytes) {
    uint64_t r;
    asm("{\n\t.reg .b32 lo, hi;\n\tmov.b64 {lo, hi}, %1;\n\tadd.u32 lo, lo, %2;\n\tmov.b64 %0, {lo, hi};\n\t}"
        : "=l"(r)
        : "l"(d), "r"(bytes >> 4));
    return r;
}

// Instruction descriptor of kind::f16 with bf16 A/B and fp32 D.
// Bits: [4,6) D format (1 = f32), [7,10) A format (1 = bf16), [10,13) B
// format, 15 A major (1 = MN), 16 B major, [17,23) N>>3, [24,29) M>>4.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn_major ? 1u : 0u) << 15) |
           ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[smem] * B[smem], issued by one thread.
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A (16-bit elements) is read from tensor
// memory, one row per lane, two consecutive K elements per 32-bit column.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` once every tcgen05 operation issued so far by this thread
// has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// The three above for a warp that runs its issue loop whole, so that descriptors
// and addresses stay in uniform registers, and issues from its leading lane.
__device__ __forceinline__ void tc_mma_if(bool lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
        : "memory");
}

__device__ __forceinline__ void tc_mma_ts_if(bool lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
        : "memory");
}

__device__ __forceinline__ void tc_commit_if(bool lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(lead))
        : "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
        "%27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// (m, l) of a partial for the merge, which leaves out partials without weights: a
// NaN among them takes it over.
__device__ __forceinline__ float2 partial_weight(float m, float l) {
    return l != l ? make_float2(3.0e38f, 1.f) : make_float2(m, l);
}

// Rows of a block whose keys some token of an item sees; the others (past the
// context, or behind every token's window and not among the first tokens) may
// hold anything.
template <bool WIN>
struct LiveRows {
    int n;   // rows of the context
    __device__ __forceinline__ LiveRows(int key0, int key_end, int, int) : n(key_end - key0) {}
    __device__ __forceinline__ bool all() const { return n >= kBlockSize; }
    __device__ __forceinline__ bool has(int row) const { return row < n; }
};
template <>
struct LiveRows<true> {
    uint32_t mask;   // bit r: row r
    // keys in [dead_begin, dead_end) are seen by no token
    __device__ __forceinline__ LiveRows(int key0, int key_end, int dead_begin, int dead_end) {
        auto below = [](int n) { return n <= 0 ? 0u : n >= kBlockSize ? 0xFFFFu : (1u << n) - 1u; };
        mask = below(key_end - key0);
        if (dead_end > key0) mask &= ~(below(dead_end - key0) & ~below(dead_begin - key0));
    }
    __device__ __forceinline__ bool all() const { return mask == 0xFFFFu; }
    __device__ __forceinline__ bool has(int row) const { return mask >> row & 1u; }
};

// An item in WindowView's numbers (WIN; else as it is).
template <bool WIN>
__device__ __forceinline__ WindowView own_numbers(const DecodeParams &p, DecodeItem &item) {
    if constexpr (!WIN) return WindowView{0, 0};
    const WindowView v = window_view(item.key_end - item.n_tok, item.key_end, p.window, p.sinks, 1);
    item.key_end -= kBlockSize * v.skip;
    return v;
}

}  // namespace dev
}  // namespace pa
