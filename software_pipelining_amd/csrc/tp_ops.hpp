// Device building blocks of the 8-bit linear layer's operators (the norm, its
// gradient, the block quantiser, the block-scaled product), on top of
// tp_engine.hpp.
//
// All memory is reached through buffer descriptors whose num_records ends with
// the data, so that an offset past it moves nothing. Two facts about these
// descriptors were checked on an MI355X and are used throughout:
//   - 16-byte loads, stores and LDS-DMA loads work at any byte alignment;
//   - the range check is made for each 4-byte word: a word that is not wholly
//     below num_records reads as zero or is not written.
// So a run of 8 elements (a "unit") that lies wholly inside its row moves with
// 16- and 8-byte accesses whatever the row's alignment, and the at most one
// unit that a row's end cuts moves element by element.
#pragma once

#include "tp_engine.hpp"
#include "tp_ops_plan.hpp"

namespace tp {
namespace dev {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kUnit = 8;                     // elements of a unit
constexpr int kLanesPerBlock = kOpBlock / kUnit;   // 16 lanes hold a block of 128
constexpr uint32_t kOutside = 0x7FFFFFF0u;   // an offset past every descriptor used here
constexpr uint32_t kBeyond = 0x7FFFFF00u;    // added to any offset, kOutside too, still past every descriptor

// ------------------------------------------------------------------- accesses
// Cache policies, measured on the row kernels and the quantiser at 60 to 470
// MB of traffic: 16- and 8-byte stores at device scope (written through to
// memory instead of leaving the XCD's L2 full of dirty lines at the kernel's
// end) ran 2-4 % faster than ordinary ones; non-temporal ones of lines that are
// written in parts lost up to half. Loads of data that is read once are
// non-temporal (ordinary ones lost 6-9 %) unless the tensors are small enough
// to stay in the last cache.
#define TP_PUT_CPOL " sc1"
// LDS-DMA and stores with the caches' ordinary policy, for operands that other
// workgroups read again.
__device__ __forceinline__ void dma_b128_cached(const BufferRes &r, uint32_t voff, uint32_t m0)
{
    asm volatile("s_mov_b32 m0, %2\n\t"
                 "s_nop 4\n\t"
                 "buffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(sgpr_res(r)), "s"(m0)
                 : "memory");
}

__device__ __forceinline__ void dma_b32_cached(const BufferRes &r, uint32_t voff, uint32_t m0)
{
    asm volatile("s_mov_b32 m0, %2\n\t"
                 "s_nop 4\n\t"
                 "buffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(sgpr_res(r)), "s"(m0)
                 : "memory");
}

// One 16-bit element a lane into the low half of the lane's dword at m0 + 4 * lane.
__device__ __forceinline__ void dma_b16(const BufferRes &r, uint32_t voff, uint32_t m0)
{
    asm volatile("s_mov_b32 m0, %2\n\t"
                 "s_nop 4\n\t"
                 "buffer_load_ushort %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(sgpr_res(r)), "s"(m0)
                 : "memory");
}

__device__ __forceinline__ void put_b128(const BufferRes &r, uint32_t voff, u32x4 v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_dwordx4 %0, %1, %2, 0 offen" TP_PUT_CPOL "\n\t"
                 "s_nop 1"
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

__device__ __forceinline__ void put_b64(const BufferRes &r, uint32_t voff, u32x2 v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_dwordx2 %0, %1, %2, 0 offen" TP_PUT_CPOL
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

__device__ __forceinline__ void put_b128_cached(const BufferRes &r, uint32_t voff, u32x4 v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_dwordx4 %0, %1, %2, 0 offen\n\t"
                 "s_nop 1"
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

__device__ __forceinline__ void put_b64_cached(const BufferRes &r, uint32_t voff, u32x2 v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_dwordx2 %0, %1, %2, 0 offen"
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

__device__ __forceinline__ void put_b128(const BufferRes &r, uint32_t voff, u32x4 v, bool past)
{
    if (past)
        put_b128(r, voff, v);
    else
        put_b128_cached(r, voff, v);
}

__device__ __forceinline__ void put_b64(const BufferRes &r, uint32_t voff, u32x2 v, bool past)
{
    if (past)
        put_b64(r, voff, v);
    else
        put_b64_cached(r, voff, v);
}

__device__ __forceinline__ void put_b32(const BufferRes &r, uint32_t voff, uint32_t v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_dword %0, %1, %2, 0 offen"
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

__device__ __forceinline__ void put_b16(const BufferRes &r, uint32_t voff, uint32_t v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_short %0, %1, %2, 0 offen"
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

__device__ __forceinline__ void put_b8(const BufferRes &r, uint32_t voff, uint32_t v)
{
    asm volatile("s_nop 4\n\t"
                 "buffer_store_byte %0, %1, %2, 0 offen"
                 :
                 : "v"(v), "v"(voff), "s"(sgpr_res(r))
                 : "memory");
}

// Loads into registers wait inside their asm block: the compiler takes a
// block's outputs as written when the block ends.
#define TP_GET_STEP(out, off, more) \
    "s_nop 4\n\tbuffer_load_dwordx4 %[" #out "], %[" #off "], %[r], 0 offen" more "\n\t"
#define TP_GET_X8(more) \
    asm volatile(TP_GET_STEP(v0, o0, more) TP_GET_STEP(v1, o1, more) TP_GET_STEP(v2, o2, more) \
                 TP_GET_STEP(v3, o3, more) TP_GET_STEP(v4, o4, more) TP_GET_STEP(v5, o5, more) \
                 TP_GET_STEP(v6, o6, more) TP_GET_STEP(v7, o7, more) "s_waitcnt vmcnt(0)" \
                 : [v0] "=&v"(v[0]), [v1] "=&v"(v[1]), [v2] "=&v"(v[2]), [v3] "=&v"(v[3]), \
                   [v4] "=&v"(v[4]), [v5] "=&v"(v[5]), [v6] "=&v"(v[6]), [v7] "=&v"(v[7]) \
                 : [o0] "v"(o[0]), [o1] "v"(o[1]), [o2] "v"(o[2]), [o3] "v"(o[3]), \
                   [o4] "v"(o[4]), [o5] "v"(o[5]), [o6] "v"(o[6]), [o7] "v"(o[7]), \
                   [r] "s"(sgpr_res(r)) \
                 : "memory")

// Eight 16-byte loads in flight together, and the same non-temporal.
__device__ __forceinline__ void get_b128x8(const BufferRes &r, const uint32_t (&o)[8], u32x4 (&v)[8])
{
    TP_GET_X8("");
}

__device__ __forceinline__ void get_b128x8_past(const BufferRes &r, const uint32_t (&o)[8], u32x4 (&v)[8])
{
    TP_GET_X8(" nt");
}

// 32 bytes at each offset: v[i] the first 16, w[i] the others. The
// two loads of a pair share their lines, so these are not non-temporal (the
// quantiser on 5000 x 4104 fp32: 30.9 us, 33.9 non-temporal).
__device__ __forceinline__ void get_b256x8(const BufferRes &r, const uint32_t (&o)[8], u32x4 (&v)[8],
                                           u32x4 (&w)[8])
{
    asm volatile(TP_GET_STEP(v0, o0, "") TP_GET_STEP(w0, o0, " offset:16")
                 TP_GET_STEP(v1, o1, "") TP_GET_STEP(w1, o1, " offset:16")
                 TP_GET_STEP(v2, o2, "") TP_GET_STEP(w2, o2, " offset:16")
                 TP_GET_STEP(v3, o3, "") TP_GET_STEP(w3, o3, " offset:16")
                 TP_GET_STEP(v4, o4, "") TP_GET_STEP(w4, o4, " offset:16")
                 TP_GET_STEP(v5, o5, "") TP_GET_STEP(w5, o5, " offset:16")
                 TP_GET_STEP(v6, o6, "") TP_GET_STEP(w6, o6, " offset:16")
                 TP_GET_STEP(v7, o7, "") TP_GET_STEP(w7, o7, " offset:16")
                 "s_waitcnt vmcnt(0)"
                 : [v0] "=&v"(v[0]), [v1] "=&v"(v[1]), [v2] "=&v"(v[2]), [v3] "=&v"(v[3]),
                   [v4] "=&v"(v[4]), [v5] "=&v"(v[5]), [v6] "=&v"(v[6]), [v7] "=&v"(v[7]),
                   [w0] "=&v"(w[0]), [w1] "=&v"(w[1]), [w2] "=&v"(w[2]), [w3] "=&v"(w[3]),
                   [w4] "=&v"(w[4]), [w5] "=&v"(w[5]), [w6] "=&v"(w[6]), [w7] "=&v"(w[7])
                 : [o0] "v"(o[0]), [o1] "v"(o[1]), [o2] "v"(o[2]), [o3] "v"(o[3]),
                   [o4] "v"(o[4]), [o5] "v"(o[5]), [o6] "v"(o[6]), [o7] "v"(o[7]),
                   [r] "s"(sgpr_res(r))
                 : "memory");
}

// Eight single elements, in flight together.
#define TP_GET_ELEMENTS(insn) \
    asm volatile("s_nop 4\n\t" insn " %0, %8, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %1, %9, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %2, %10, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %3, %11, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %4, %12, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %5, %13, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %6, %14, %16, 0 offen\n\t" \
                 "s_nop 4\n\t" insn " %7, %15, %16, 0 offen\n\t" \
                 "s_waitcnt vmcnt(0)" \
                 : "=&v"(e[0]), "=&v"(e[1]), "=&v"(e[2]), "=&v"(e[3]), "=&v"(e[4]), "=&v"(e[5]), \
                   "=&v"(e[6]), "=&v"(e[7]) \
                 : "v"(o[0]), "v"(o[1]), "v"(o[2]), "v"(o[3]), "v"(o[4]), "v"(o[5]), "v"(o[6]), \
                   "v"(o[7]), "s"(sgpr_res(r)) \
                 : "memory")

template <class T>
__device__ __forceinline__ void get_elements(const BufferRes &r, const uint32_t (&o)[8], uint32_t (&e)[8])
{
    if constexpr (T::bytes == 2)
        TP_GET_ELEMENTS("buffer_load_ushort");
    else
        TP_GET_ELEMENTS("buffer_load_dword");
}

// Four single bytes.
__device__ __forceinline__ void get_bytes(const BufferRes &r, const uint32_t (&o)[4], uint32_t (&e)[4])
{
    asm volatile("s_nop 4\n\tbuffer_load_ubyte %0, %4, %8, 0 offen\n\t"
                 "s_nop 4\n\tbuffer_load_ubyte %1, %5, %8, 0 offen\n\t"
                 "s_nop 4\n\tbuffer_load_ubyte %2, %6, %8, 0 offen\n\t"
                 "s_nop 4\n\tbuffer_load_ubyte %3, %7, %8, 0 offen\n\t"
                 "s_waitcnt vmcnt(0)"
                 : "=&v"(e[0]), "=&v"(e[1]), "=&v"(e[2]), "=&v"(e[3])
                 : "v"(o[0]), "v"(o[1]), "v"(o[2]), "v"(o[3]), "s"(sgpr_res(r))
                 : "memory");
}

// Workgroup barrier after which every wave's LDS writes made before it can be
// read, and every LDS read made before it has returned.
__device__ __forceinline__ void lds_sync()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// ------------------------------------------------------------------ reductions
// Sum over the wave's 64 lanes, on every lane, in an order fixed by the lane
// numbers: rotations within 16 lanes (DPP), then the four groups' sums in
// turn. (Six LDS permutes one after another instead: 0.3 us a row where rows
// are few, and 83 us against 81 for the norm of 8192 x 8192.)
__device__ __forceinline__ float wave_sum(float v)
{
#define TP_ROR_ADD(ctrl) \
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xF, 0xF, true))
    TP_ROR_ADD(0x128);
    TP_ROR_ADD(0x124);
    TP_ROR_ADD(0x122);
    TP_ROR_ADD(0x121);
#undef TP_ROR_ADD
    const auto group = [&](int i) TP_INLINE {
        return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 16 * i));
    };
    return (group(0) + group(1)) + (group(2) + group(3));
}

// The value of lane 7 - i of the lane's eight.
__device__ __forceinline__ uint32_t mirror8(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true);
}

// Largest of the 16 lanes of an aligned group, on each of them (DPP row
// rotations). Values are the bits of numbers >= 0 or of a NaN without its
// sign: as unsigned integers they order like the numbers, with every NaN above
// infinity, so a NaN anywhere in the group is the result.
__device__ __forceinline__ uint32_t group16_max(uint32_t v)
{
#define TP_ROR_MAX(ctrl) \
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, true))
    TP_ROR_MAX(0x121);
    TP_ROR_MAX(0x122);
    TP_ROR_MAX(0x124);
    TP_ROR_MAX(0x128);
#undef TP_ROR_MAX
    return v;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ------------------------------------------------------------------- the types
struct Bf16 {
    static constexpr int bytes = 2;
    __device__ static __forceinline__ float wide(uint32_t h) { return __uint_as_float(h << 16); }
    // nearest, ties to even; a NaN stays a NaN (quiet, its upper payload kept)
    __device__ static __forceinline__ uint32_t narrow(float f)
    {
        const uint32_t u = __float_as_uint(f);
        const uint32_t r = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
        return (u & 0x7FFFFFFFu) > 0x7F800000u ? (u >> 16) | 0x40u : r;
    }
    __device__ static __forceinline__ uint32_t narrow2(float a, float b)
    {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 v;
        v[0] = (__bf16)a;
        v[1] = (__bf16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    __device__ static __forceinline__ void wide2(uint32_t p, float &a, float &b)
    {
        a = __uint_as_float(p << 16);
        b = __uint_as_float(p & 0xFFFF0000u);
    }
};

struct Fp16 {
    static constexpr int bytes = 2;
    __device__ static __forceinline__ float wide(uint32_t h)
    {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
    }
    __device__ static __forceinline__ uint32_t narrow(float f)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    }
    __device__ static __forceinline__ uint32_t narrow2(float a, float b)
    {
        return narrow(a) | narrow(b) << 16;
    }
    __device__ static __forceinline__ void wide2(uint32_t p, float &a, float &b)
    {
        a = wide(p & 0xFFFFu);
        b = wide(p >> 16);
    }
};

struct Fp32 {
    static constexpr int bytes = 4;
    __device__ static __forceinline__ float wide(uint32_t w) { return __uint_as_float(w); }
    __device__ static __forceinline__ uint32_t narrow(float f) { return __float_as_uint(f); }
};

// A unit as it lies in memory: one 16-byte chunk of a 16-bit type, two of fp32.
template <class T>
struct RawUnit {
    u32x4 c[T::bytes / 2];
};

template <class T>
__device__ __forceinline__ void unit_wide(const RawUnit<T> &u, float (&v)[kUnit])
{
    if constexpr (T::bytes == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            T::wide2(u.c[0][i], v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = T::wide(u.c[i / 4][i % 4]);
    }
}

template <class T>
__device__ __forceinline__ RawUnit<T> unit_narrow(const float (&v)[kUnit])
{
    RawUnit<T> u;
    if constexpr (T::bytes == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u.c[0][i] = T::narrow2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u.c[i / 4][i % 4] = T::narrow(v[i]);
    }
    return u;
}

// Moves a unit's elements down by n (0 to 7), the lane's own; zeros follow.
template <class T>
__device__ __forceinline__ void unit_down(RawUnit<T> &u, uint32_t n)
{
    constexpr int dwords = kUnit * T::bytes / 4;
    const uint32_t by_dwords = n * T::bytes / 4;
    const auto at = [&](int i) TP_INLINE { return i < dwords ? u.c[i / 4 % (dwords / 4)][i % 4] : 0u; };
#pragma unroll
    for (int by = dwords / 2; by >= 1; by /= 2)
#pragma unroll
        for (int i = 0; i < dwords; ++i)
            u.c[i / 4][i % 4] = by_dwords & by ? at(i + by) : at(i);
    if constexpr (T::bytes == 2) {
#pragma unroll
        for (int i = 0; i < dwords; ++i)
            u.c[0][i] = n & 1u ? at(i) >> 16 | at(i + 1) << 16 : at(i);
    }
}

// The first `have` (0 to 15) bytes of v at off, for lanes of which `cut` holds;
// `have` is the workgroup's.
__device__ __forceinline__ void put_first_bytes(const BufferRes &r, uint32_t off, bool cut, uint32_t have,
                                                u32x4 v)
{
    if (have & 8u) {
        put_b64(r, cut ? off : kOutside, u32x2{v.x, v.y});
        v.x = v.z;
        v.y = v.w;
    }
    if (have & 4u) {
        put_b32(r, cut ? off + (have & 8u) : kOutside, v.x);
        v.x = v.y;
    }
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i)
        if (i < have % 4)
            put_b8(r, cut ? off + (have & 12u) + i : kOutside, v.x >> (8 * i));
}

// ------------------------------------------------------------- 8-bit numbers
// e4m3 (bias 7, largest 448, no infinity) and e5m2 (bias 15, largest 57344).
struct E4m3 {
    static constexpr float most = 448.0f;
    template <bool Hi>
    __device__ static __forceinline__ uint32_t pack2(float a, float b, uint32_t old)
    {
        return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, Hi);
    }
    // the number that the lowest byte stands for
    __device__ static __forceinline__ float wide(uint32_t byte)
    {
        return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
    }
};

struct E5m2 {
    static constexpr float most = 57344.0f;
    template <bool Hi>
    __device__ static __forceinline__ uint32_t pack2(float a, float b, uint32_t old)
    {
        return __builtin_amdgcn_cvt_pk_bf8_f32(a, b, old, Hi);
    }
    __device__ static __forceinline__ float wide(uint32_t byte)
    {
        return __builtin_amdgcn_cvt_f32_bf8((int)byte, 0);
    }
};

template <class F>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    return F::template pack2<true>(c, d, F::template pack2<false>(a, b, 0));
}

// What a block's largest magnitude (its bits) gives: the factor that the
// block's numbers are multiplied by before they are rounded to 8 bits, and the
// scale that turns the 8-bit numbers back. A largest magnitude below 2^-96
// counts as 2^-96, which keeps both finite for a block of zeros. A NaN makes
// both NaN; an infinity makes the factor 0 and the scale infinite, so that
// every number of the block comes back as NaN.
constexpr uint32_t kLeastMost = 0x0F800000u;    // 2^-96

struct BlockScale {
    float factor, scale, most;
};

template <class F>
__device__ __forceinline__ BlockScale block_scale(uint32_t most_bits)
{
    const float m = __uint_as_float(max(most_bits, kLeastMost));
    return BlockScale{F::most / m, m / F::most, m};
}

// x times MOST / m, to be rounded to 8 bits. A number of a 16-bit type often
// lands exactly half way between two 8-bit numbers, and the two roundings of
// x * (MOST / m) would then decide instead of the tie rule. So for those types
// the quotient is corrected by its remainder: MOST is 7/8 of a power of two, so
// x * 7/8 and the divisor, m over that power, are exact, and so is the fma's
// remainder. (A product of two fp32 numbers, the norm's, is rounded itself, and a
// tie there is as rare as any other value.)
template <class T, class F>
struct BlockQuotient {
    static constexpr bool exact = T::bytes == 2;
    // what a block's lanes need: factor, or divisor and its inverse
    __device__ static __forceinline__ float2 make(const BlockScale &b)
    {
        if constexpr (!exact)
            return make_float2(b.factor, 0.0f);
        const float divisor = b.most * (0.875f / F::most);
        return make_float2(divisor, 1.0f / divisor);
    }
    // what is done to a number once, whatever blocks it is in
    __device__ static __forceinline__ float ready(float x) { return exact ? x * 0.875f : x; }
    __device__ static __forceinline__ float of(float ready_x, float2 b)
    {
        if constexpr (!exact)
            return ready_x * b.x;
        const float t = ready_x * b.y;
        return fmaf(fmaf(-t, b.x, ready_x), b.y, t);
    }
};

// Magnitudes of a unit, eight to be compared: of a 16-bit type two in a
// register (as unsigned integers they order like the numbers, NaN above
// infinity), of fp32 one.
template <class T>
struct Magnitudes {
    static constexpr int n = T::bytes == 2 ? 4 : 8;
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    uint32_t m[n];

    __device__ __forceinline__ void set(const RawUnit<T> &u)
    {
#pragma unroll
        for (int i = 0; i < n; ++i)
            m[i] = T::bytes == 2 ? u.c[0][i % 4] & 0x7FFF7FFFu : u.c[i / 4 % (T::bytes / 2)][i % 4] & 0x7FFFFFFFu;
    }
    __device__ static __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        if constexpr (T::bytes == 2)
            return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                          __builtin_bit_cast(u16x2, b)));
        return max(a, b);
    }
    // the bits, as fp32, of element i
    __device__ __forceinline__ uint32_t wide(int i) const
    {
        if constexpr (T::bytes == 2)
            return __float_as_uint(T::wide(m[i / 2] >> (16 * (i & 1)) & 0xFFFFu));
        return m[i];
    }
    // ... of the largest
    __device__ __forceinline__ uint32_t most() const
    {
        uint32_t a = m[0];
#pragma unroll
        for (int i = 1; i < n; ++i)
            a = larger(a, m[i]);
        if constexpr (T::bytes == 2)
            return __float_as_uint(T::wide(max(a & 0xFFFFu, a >> 16)));
        return a;
    }
};

}  // namespace dev
}  // namespace tp
