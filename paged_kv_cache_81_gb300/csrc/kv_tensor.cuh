// The 5th-generation tensor core, its tensor memory and tiled TMA loads, for the kernels that compute
// with the cached rows (kv_attention.cu, kv_latent.cu, kv_expand.cu, kv_mass.cu).
//
// Shared-memory operand tiles are made of panels of 64 16-bit elements: a panel holds R rows of 128
// bytes in the 128-byte swizzle (16-byte chunk c of row r sits at chunk c ^ (r & 7)), which is what a
// tiled TMA load with a 64-element box writes.  Panels start on 1024-byte boundaries.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_async.cuh"
#include "kv_common.cuh"

// Code that is called seldom and kept out of its callers' registers.  A kernel that changes its warps' registers cannot call.  What is
// compiled in either form has a name for each, in the namespace PKV_FORM.
#ifndef PKV_APART
#define PKV_APART __noinline__
#define PKV_ONE_JOIN 0
#define PKV_FORM called
#else
#define PKV_ONE_JOIN 1
#define PKV_FORM inlined
#endif

namespace pkv {

// ---------------------------------------------------------------------------
// Bounded waits of a CTA whose warps wait for one another.  A wait that runs out marks the CTA as
// given up (a word in shared memory) and sets KV_DERR_TIMEOUT; every other wait of the CTA then
// returns at once, the roles leave their loops, and the CTA ends through its common exit.
// ---------------------------------------------------------------------------
inline namespace PKV_FORM {
struct Waiter {
    volatile int *gave_up;
    int *err;

    // One thread's wait for the phase of the given parity; false when the CTA has given up.
    __device__ __forceinline__ bool one(uint32_t bar, uint32_t parity) const
    {
        if (mbar_try_wait(bar, parity)) return true;
        return slow(bar, parity);
    }
    __device__ PKV_APART bool slow(uint32_t bar, uint32_t parity) const
    {
        const unsigned long long t0 = now_ns();
        while (!mbar_try_wait(bar, parity)) {
            if (*gave_up) return false;
            if (now_ns() - t0 > kWaitLimitNs) {
                *gave_up = 1;
                set_error(err, KV_DERR_TIMEOUT);
                return false;
            }
        }
        return true;
    }
    // A whole warp's wait: the same answer for all its lanes.
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, one(bar, parity));
    }
    // Whether the phase is over, without waiting.
    static __device__ __forceinline__ bool over(uint32_t bar, uint32_t parity)
    {
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
    // Two and three waits at once: asked one after another, each costs the issuing warp about 100 cycles in
    // which it feeds the tensor core nothing, ready or not.
    __device__ __forceinline__ bool warp(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1) const
    {
        const bool a = over(bar0, parity0), b = over(bar1, parity1);
        return __all_sync(0xffffffffu, a && b) || (warp(bar0, parity0) && warp(bar1, parity1));
    }
    __device__ __forceinline__ bool warp(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, uint32_t bar2, uint32_t parity2) const
    {
        const bool a = over(bar0, parity0), b = over(bar1, parity1), c = over(bar2, parity2);
        return __all_sync(0xffffffffu, a && b && c) || (warp(bar0, parity0) && warp(bar1, parity1) && warp(bar2, parity2));
    }
};
}  // namespace PKV_FORM

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One arrival for a whole warp, after what all its lanes did before (32 arrivals on one barrier would be
// taken one after another).
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

// Orders this thread's shared-memory writes before later reads by the tensor core and TMA.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Tiled TMA
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------------------
// Tensor memory and tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns)  // one whole warp
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns)  // the warp that allocated
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of the warp, the same one every time.  A warp that issues products runs its loops as a
// whole, with operands the same in all lanes, and predicates only the instructions: the descriptors then
// stay in uniform registers (issued from inside a one-lane branch, each product cost about 95 cycles of
// moving them there, one and a half times what the tensor core takes for it).
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// The barrier is arrived on once every tcgen05.mma that the elected thread issued so far has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
}

// 32 columns of this warp's 32 lanes: register i of a thread is column i of its lane.
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
          "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(t));
}

__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]),
        "r"(t)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(t)
        : "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, version 1; stride = bytes between groups of
// eight rows, lead = bytes between 64-element panels of an operand whose rows are the K axis.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// Instruction descriptor of kind::f16 with 32-bit accumulators.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, uint32_t m, uint32_t n, bool b_rows_are_k)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_rows_are_k ? 1u : 0u) << 16) | ((n >> 3) << 17) |
           ((m >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(elected)
        : "memory");
}

// A from tensor memory (16-bit pairs packed in 32-bit columns).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(elected)
        : "memory");
}

// ---------------------------------------------------------------------------
// Arithmetic
// ---------------------------------------------------------------------------
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (a x + b) of two values at once.
__device__ __forceinline__ float2 fma2(float2 x, float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, a, b, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 a, {%4, %5};\n\tmov.b64 b, {%6, %7};\n\t"
        "fma.rn.f32x2 r, x, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

template <bool Bf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)  // lo in the low half, round to nearest even
{
    uint32_t r;
    if (Bf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Scores of 32 keys: those outside [a, z) become -inf.
__device__ __forceinline__ void hide32(uint32_t (&x)[32], int a, int z)
{
    const uint32_t seen = (a >= 32 ? 0u : 0xffffffffu << max(a, 0)) & (z <= 0 ? 0u : 0xffffffffu >> (32 - min(z, 32)));
#pragma unroll
    for (int i = 0; i < 32; i++)
        if (!(seen >> i & 1)) x[i] = 0xff800000u;
}

__device__ __forceinline__ float max32(const uint32_t (&x)[32], float top)
{
    float t[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 32; i++) t[i & 3] = fmaxf(t[i & 3], __uint_as_float(x[i]));
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// The weights P = 2^(c (s - m)) become 16-bit numbers for the second product, whose operands have one type; a second
// product for what the rounding leaves would double its time.  m is the row's reference: its largest score, or one
// that it exceeds by less than 2^8.  bf16 holds such weights however small.  fp16 has nothing below 2^-25, while the
// sum of the weights counts them all: behind one heavy key, 8191 light ones of 2^-26 (together 1.2e-4 of the sum) came
// out as 0.  So fp16 weights are held 2^7 times as large, up to 2^15 of 2^16, and what is lost is below 2^-32 each.  The rounding
// goes up, so that no weight passes that bound for what the product of large scores rounds off.
template <bool Bf16>
__device__ __forceinline__ float weight_offset(float m, float c)
{
    return m == -INFINITY ? 0.0f : Bf16 ? m * c : __fmaf_ru(m, c, -7.0f);
}

// The logarithm of a sum of such weights.
template <bool Bf16>
__device__ __forceinline__ float weight_log(float l) { return logf(Bf16 ? l : l * 0x1p-7f); }

// Weights 2^(c s - mc) of 32 scores, added to two partial sums and rounded to pairs of the element type.
template <bool Bf16>
__device__ __forceinline__ void weights32(const uint32_t (&x)[32], float c, float mc, float2 (&sum)[2], uint32_t (&pk)[16])
{
    const float2 cc = make_float2(c, c), nn = make_float2(-mc, -mc);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        float2 e = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, nn);
        e.x = exp2_fast(e.x);
        e.y = exp2_fast(e.y);
        sum[i & 1] = add2(sum[i & 1], e);
        pk[i] = pack2<Bf16>(e.x, e.y);
    }
}

// Byte offset of 16-byte chunk c (0 .. 7) of row r in a panel.
__device__ __forceinline__ uint32_t panel_off(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

__device__ __forceinline__ uint4 ld_smem16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void st_smem16(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---------------------------------------------------------------------------
// Host: tensor maps (kv_tensor.cu)
// ---------------------------------------------------------------------------
// A map of 16-bit elements with the 128-byte swizzle: dims[0] elements are contiguous, strides (bytes)
// are those of dims[1] .. dims[rank - 1], and a load brings box[0] = 64 by box[1] by .. elements.
int make_map(CUtensorMap *map, uint64_t base, int rank, const uint64_t *dims, const uint64_t *strides, const uint32_t *box);

// A map of one plane of one tensor of a paged cache as (element of a head, head, slot, block); a load
// brings 64 elements of one head of `rows` consecutive slots of a block.
int make_cache_map(CUtensorMap *map, const kv_cache_desc *c, int tensor, int plane, int heads, int head_dim, int rows);

// A map of the codes of 4-bit rows as (32-bit word of a head's codes, head, slot, block), without a swizzle; a load brings one head's
// codes of `rows` consecutive slots of a block, `bytes` apart, with zeros past their end.
int make_q4_code_map(CUtensorMap *map, uint64_t base, const kv_cache_desc *c, int heads, int dim, int bytes, int rows);

// A map of a plane's rows as opaque 32-bit words (64-bit ones for boxes of more than 1024 bytes), (word of a row, slot, block), without a
// swizzle; a load brings `bytes` of each of `rows` consecutive slots of a block, densely, with zeros for what lies past a row's end.
__host__ __device__ inline int row_map_shift(int bytes) { return bytes > 1024 ? 3 : 2; }  // log2 of a word's bytes: a box has at most 256 words
int make_row_map(CUtensorMap *map, uint64_t base, const kv_cache_desc *c, int bytes, int rows);

}  // namespace pkv
