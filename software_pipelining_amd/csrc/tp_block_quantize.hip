// Quantiser by blocks: numbers that share a scale (128 of a row, 128 of a
// column, or a square of 128 x 128) are multiplied by MOST / m, m the largest
// magnitude among them, and rounded to 8 bits; scale = m / MOST turns them
// back. Straight output q has x's rows; turned output qt has x's columns as
// rows, so that both products a training step makes of one activation or
// weight find their operand along the sum.
//
// Bound by memory: x is read once for both outputs. 8192 x 8192 bf16 one way
// (203 MB): 33 us, 6.0 TB/s; 4096 x 8192 bf16 both ways (137 MB): 31 us, 4.4
// TB/s; 5000 x 4104 fp32 in squares both ways (123 MB): 31 us. What keeps both
// ways from the full rate is a tile's chain of loads, maxima, two barriers and
// the turn through LDS, and the column scales, 4 bytes a line (4 us of the 31).
//
// A workgroup of 256 lanes
// takes a tile of 128 x 128; a lane holds a patch of 8 x 8 in registers:
// 8 units, one a row, of 16-byte loads that cover 256 bytes of a row with 16
// lanes. Row maxima are 16-lane maxima; column maxima go over a wave's 4
// patch rows and then, through LDS, over the 4 waves. The turned tile passes
// through 16 KiB of LDS as columns of 8-byte pieces, swizzled so that neither
// side has bank conflicts, and leaves as rows of 16-byte stores.
#include "tp_ops.hpp"

namespace tp {
namespace dev {

struct QuantLds {
    uint32_t col_most[4][kOpBlock];
    uint32_t row_most[kOpBlock];
    float2 row_scale[kOpBlock];      // Quotients' of each block
    float2 col_scale[kOpBlock];
    alignas(16) uint8_t turned[kOpBlock * kOpBlock];
};
static_assert(sizeof(QuantLds) == kQuantLdsBytes, "the planner's");

// Four numbers of a block over its scale, in 8 bits, and what a block's lanes need
// for that. `unsure` takes `bit` where one of them may be the 8-bit number below
// the right one: then `settle` makes it right, given the bits of the block's
// largest magnitude.
template <class T, class F>
struct Quotients {
    using Q = BlockQuotient<T, F>;
    __device__ static __forceinline__ float2 make(const BlockScale &b) { return Q::make(b); }
    __device__ static __forceinline__ uint32_t of(const float (&x)[4], float2 b, uint32_t, uint32_t &)
    {
        return pack4<F>(Q::of(Q::ready(x[0]), b), Q::of(Q::ready(x[1]), b),
                        Q::of(Q::ready(x[2]), b), Q::of(Q::ready(x[3]), b));
    }
    __device__ static __forceinline__ void settle(const float (&)[4], float2, uint32_t, uint32_t &) {}
};

// Numbers of 32 bits can be tensors of 16-bit ones made wider, or whole numbers,
// which often lie half way between two 8-bit numbers, and their remainder takes
// more than an fma. So x times MOST / m is taken with that factor 2^-22 too small
// and too large, more than its own and the product's rounding: where both round
// to the same 8-bit number, that is the quotient's. Where not (five numbers of a
// million), x MOST is compared with m times the middle of the two, both of which
// 64 bits hold exactly. (5000 x 4104 by rows and columns: 35.1 us, by one rounded
// factor 33.8; in squares, whose turned numbers are the straight ones, 30.3 and 30.6.
// Of bf16 values made wider three of ten thousand lie on ties: again and again on
// one tensor 38.0 and 29.1 us, 29.3 and 25.2 of any numbers.)
template <class F>
struct Quotients<Fp32, F> {
    __device__ static __forceinline__ float2 make(const BlockScale &b)
    {
        return make_float2(b.factor * (1.0f - 0x1p-22f), b.factor * (1.0f + 0x1p-22f));
    }
    __device__ static __forceinline__ uint32_t by(const float (&x)[4], float factor)
    {
        return pack4<F>(x[0] * factor, x[1] * factor, x[2] * factor, x[3] * factor);
    }
    __device__ static __forceinline__ uint32_t of(const float (&x)[4], float2 b, uint32_t bit, uint32_t &unsure)
    {
        const uint32_t q = by(x, b.x);
        unsure |= q != by(x, b.y) ? bit : 0u;
        return q;
    }
    __device__ static __forceinline__ void settle(const float (&x)[4], float2 b, uint32_t most, uint32_t &q)
    {
        const uint32_t r = by(x, b.y);
#pragma unroll 1
        for (uint32_t left = q ^ r; left != 0;) {
            const uint32_t at = (uint32_t)__builtin_ctz(left) & 24u;
            left &= ~(0xFFu << at);
            const uint32_t low = q >> at & 0xFFu, high = r >> at & 0xFFu;
            const float v = at < 16 ? (at == 0 ? x[0] : x[1]) : at == 16 ? x[2] : x[3];
            const float middle = 0.5f * (F::wide(low & 0x7Fu) + F::wide(high & 0x7Fu));
            const double is = (double)fabsf(v) * (double)F::most;
            const double half = (double)middle * (double)__uint_as_float(max(most, kLeastMost));
            if (is > half || (is == half && (high & 1u) == 0u))
                q ^= (low ^ high) << at;
        }
    }
};

// Columns of 4 x 4 bytes from its rows.
__device__ __forceinline__ void turn4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3, uint32_t &c0,
                                      uint32_t &c1, uint32_t &c2, uint32_t &c3)
{
    const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400u), b = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(r1, r0, 0x07030602u), d = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
    c0 = __builtin_amdgcn_perm(b, a, 0x05040100u);
    c1 = __builtin_amdgcn_perm(b, a, 0x07060302u);
    c2 = __builtin_amdgcn_perm(d, c, 0x05040100u);
    c3 = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

// The elements of a row of fewer than eight.
template <class T>
__device__ __forceinline__ RawUnit<T> get_narrow_row(const BufferRes &r, uint32_t off, int have)
{
    uint32_t o[8], e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = i < have ? off + i * T::bytes : kOutside;
    get_elements<T>(r, o, e);
    RawUnit<T> u;
#pragma unroll
    for (int i = 0; i < kUnit * T::bytes / 4; ++i)
        u.c[i / 4][i % 4] = T::bytes == 2 ? e[2 * i] | e[2 * i + 1] << 16 : e[i];
    return u;
}

template <class T, class F, bool Square, bool Straight, bool Turned>
__global__ void __launch_bounds__(256, T::bytes == 2 ? 4 : 3) block_quantize_kernel(QuantParams p)
{
    using Q = Quotients<T, F>;
    __shared__ QuantLds lds;
    const uint32_t tid = threadIdx.x, u = tid % kLanesPerBlock, patch = tid / kLanesPerBlock;
    const uint32_t wave = uniform(tid >> 6);
    const uint32_t across = (uint32_t)p.across;
    const uint32_t block_col = blockIdx.x % across;
    const int64_t block_row = blockIdx.x / across;
    const int64_t row0 = block_row * kOpBlock, col0 = (int64_t)block_col * kOpBlock;
    const uint32_t high = (uint32_t)(p.rows - row0 < kOpBlock ? p.rows - row0 : kOpBlock);
    const uint32_t wide = (uint32_t)(p.cols - col0 < kOpBlock ? p.cols - col0 : kOpBlock);
    const uint32_t down = (uint32_t)((p.rows + kOpBlock - 1) / kOpBlock);

    // ---- the patch
    const uint32_t pitch = (uint32_t)p.x_stride;
    // a unit that the last column cuts is loaded as the eight elements that end
    // there, which reach into the tile before
    const uint32_t lead = block_col > 0 ? kUnit * T::bytes : 0u;
    const BufferRes rx = make_buffer_res(static_cast<const uint8_t *>(p.x) + row0 * p.x_stride +
                                             col0 * T::bytes - lead,
                                         (high - 1) * pitch + wide * T::bytes + lead);
    const uint32_t c0 = u * kUnit;
    const int have = wide <= c0 ? 0 : wide - c0 < kUnit ? (int)(wide - c0) : kUnit;
    const uint32_t missing = (kUnit - wide % kUnit) % kUnit;     // of the unit that is cut
    const bool narrow = p.cols < kUnit;                          // no eight elements end anywhere
    const uint32_t from = c0 - (have != 0 && have != kUnit ? missing : 0u);
    uint32_t off[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        off[i] = have != 0 && !narrow && patch * 8 + i < high
                     ? (patch * 8 + i) * pitch + lead + from * T::bytes
                     : kOutside;
    RawUnit<T> raw[8];
    {
        u32x4 v[8];
        if constexpr (T::bytes == 2) {
            if (p.cached)
                get_b128x8(rx, off, v);
            else
                get_b128x8_past(rx, off, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                raw[i].c[0] = v[i];
        } else {
            u32x4 w[8];
            get_b256x8(rx, off, v, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                raw[i].c[0] = v[i];
                raw[i].c[1] = w[i];
            }
        }
    }
    if (missing != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            unit_down<T>(raw[i], c0 - from);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (narrow)
            for (int i = 0; i < 8; ++i) {
                const RawUnit<T> cut = get_narrow_row<T>(rx, (patch * 8 + i) * pitch,
                                                         patch * 8 + i < high ? have : 0);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j == i)
                        raw[j] = cut;
            }
    }

    // ---- the maxima
    uint32_t row_most[8], col_most[8], square_most = 0;
    {
        Magnitudes<T> down_most;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Magnitudes<T> m;
            m.set(raw[i]);
            if constexpr (Square || Straight)
                row_most[i] = m.most();
            if constexpr (!Square && Turned) {
#pragma unroll
                for (int j = 0; j < Magnitudes<T>::n; ++j)
                    down_most.m[j] = i == 0 ? m.m[j] : Magnitudes<T>::larger(down_most.m[j], m.m[j]);
            }
        }
        if constexpr (!Square && Turned) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                col_most[j] = down_most.wide(j);
        }
    }
    if constexpr (Square) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, row_most[i]);
        m = group16_max(m);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        lds.row_most[wave] = m;
        lds_sync();
        m = max(max(lds.row_most[0], lds.row_most[1]), max(lds.row_most[2], lds.row_most[3]));
        square_most = m;
        const BlockScale b = block_scale<F>(m);
        if (tid < kOpBlock)
            lds.row_scale[tid] = Q::make(b);
        if (wave == 0) {
            const int64_t rows_of_scale = down;
            if constexpr (Straight)
                put_b32(make_buffer_res(p.scale + block_row * across + block_col, 4), tid * 4,
                        __float_as_uint(b.scale));
            if constexpr (Turned)
                put_b32(make_buffer_res(p.scale_t + (int64_t)block_col * rows_of_scale + block_row, 4),
                        tid * 4, __float_as_uint(b.scale));
        }
        lds_sync();
    } else {
        if constexpr (Straight) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                row_most[i] = group16_max(row_most[i]);
                if (u == i)
                    lds.row_most[patch * 8 + i] = row_most[i];
            }
        }
        if constexpr (Turned) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                col_most[j] = max(col_most[j], (uint32_t)__shfl_xor((int)col_most[j], 16));
                col_most[j] = max(col_most[j], (uint32_t)__shfl_xor((int)col_most[j], 32));
            }
            if ((tid & 63u) < kLanesPerBlock) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    lds.col_most[wave][c0 + j] = col_most[j];
            }
        }
        lds_sync();
        if (wave < 2) {
            if constexpr (Straight) {
                const BlockScale b = block_scale<F>(lds.row_most[tid]);
                lds.row_scale[tid] = Q::make(b);
                const BufferRes rs = make_buffer_res(p.scale + row0 * across + block_col,
                                                     ((high - 1) * across + 1) * 4);
                put_b32(rs, tid < high ? tid * across * 4 : kOutside, __float_as_uint(b.scale));
            }
        } else {
            if constexpr (Turned) {
                const uint32_t c = tid - kOpBlock;
                const uint32_t m = max(max(lds.col_most[0][c], lds.col_most[1][c]),
                                       max(lds.col_most[2][c], lds.col_most[3][c]));
                const BlockScale b = block_scale<F>(m);
                lds.col_scale[c] = Q::make(b);
                lds.col_most[0][c] = m;      // (which this lane alone has read)
                const BufferRes rs = make_buffer_res(p.scale_t + col0 * down + block_row,
                                                     ((wide - 1) * down + 1) * 4);
                put_b32(rs, c < wide ? c * down * 4 : kOutside, __float_as_uint(b.scale));
            }
        }
        lds_sync();
    }

    // ---- the outputs
    // (the numbers are unpacked again for each: kept unpacked they would take
    // the registers of a fourth workgroup on the CU)
    uint32_t q[8][2];
    if constexpr (Straight || Square) {
        uint32_t unsure = 0;
        const auto row = [&](int i, auto &&each) TP_INLINE {
            float v[kUnit];
            unit_wide<T>(raw[i], v);
            each({v[0], v[1], v[2], v[3]}, 1u << (2 * i), q[i][0]);
            each({v[4], v[5], v[6], v[7]}, 2u << (2 * i), q[i][1]);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 b = lds.row_scale[patch * 8 + i];
            row(i, [&](const float (&x)[4], uint32_t bit, uint32_t &to) TP_INLINE {
                to = Q::of(x, b, bit, unsure);
            });
        }
        if (unsure != 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                row(i, [&](const float (&x)[4], uint32_t bit, uint32_t &to) TP_INLINE {
                    if (unsure & bit)
                        Q::settle(x, lds.row_scale[patch * 8 + i], Square ? square_most : lds.row_most[patch * 8 + i], to);
                });
        }
    }
    if constexpr (Straight) {
        const uint32_t qp = (uint32_t)p.q_stride;
        const BufferRes rq = make_buffer_res(p.q + row0 * p.q_stride + col0, (high - 1) * qp + wide);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool inside = patch * 8 + i < high;
            put_b64(rq, have == kUnit && inside ? (patch * 8 + i) * qp + c0 : kOutside, u32x2{q[i][0], q[i][1]});
            if (wide % kUnit != 0)
                put_first_bytes(rq, (patch * 8 + i) * qp + c0, have != 0 && have != kUnit && inside,
                                wide % kUnit, u32x4{q[i][0], q[i][1], 0, 0});
        }
    }
    if constexpr (T::bytes == 2 && !Square) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm volatile("" : "+v"(raw[i].c[0]));
    }
    if constexpr (Turned) {
        // column 8u + j as 8 bytes at piece `patch` of its 16
        uint32_t t[kUnit][2];
        if constexpr (Square) {       // the same numbers
#pragma unroll
            for (int j = 0; j < 8; j += 4)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    turn4(q[4 * half][j / 4], q[4 * half + 1][j / 4], q[4 * half + 2][j / 4], q[4 * half + 3][j / 4],
                          t[j][half], t[j + 1][half], t[j + 2][half], t[j + 3][half]);
        } else {
            uint32_t unsure = 0;
            const auto columns = [&](int half, auto &&each) TP_INLINE {
                float v[4][kUnit];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    unit_wide<T>(raw[half * 4 + i], v[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    each({v[0][j], v[1][j], v[2][j], v[3][j]}, j, 1u << (2 * j + half), t[j][half]);
            };
#pragma unroll
            for (int half = 0; half < 2; ++half)
                columns(half, [&](const float (&x)[4], int j, uint32_t bit, uint32_t &to) TP_INLINE {
                    to = Q::of(x, lds.col_scale[c0 + j], bit, unsure);
                });
            if (unsure != 0) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    columns(half, [&](const float (&x)[4], int j, uint32_t bit, uint32_t &to) TP_INLINE {
                        if (unsure & bit)
                            Q::settle(x, lds.col_scale[c0 + j], lds.col_most[0][c0 + j], to);
                    });
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<u32x2 *>(lds.turned + (c0 + j) * kOpBlock + (patch ^ u) * 8) = u32x2{t[j][0], t[j][1]};
        lds_sync();
        const uint32_t tp_ = (uint32_t)p.qt_stride;
        const BufferRes rq = make_buffer_res(p.qt + col0 * p.qt_stride + row0, (wide - 1) * tp_ + high);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t c = s * 32 + tid / 8, pair = tid % 8, swz = c / kUnit;
            u32x4 v = *reinterpret_cast<const u32x4 *>(lds.turned + c * kOpBlock +
                                                       ((2 * pair) ^ (swz & ~1u)) * 8);
            if (swz & 1u)
                v = u32x4{v.z, v.w, v.x, v.y};
            const uint32_t at = c * tp_ + pair * 16;
            const bool inside = c < wide;
            put_b128(rq, inside && pair * 16 + 16 <= high ? at : kOutside, v);
            if (high % 16 != 0) {
                const bool cut = inside && pair * 16 < high && pair * 16 + 16 > high;
                put_first_bytes(rq, at, cut, high % 16, v);
            }
        }
    }
}

}  // namespace dev

namespace {

using Fn = void (*)(QuantParams);

template <class T, class F, bool Square>
Fn quant_fn(bool straight, bool turned)
{
    return straight && turned ? &dev::block_quantize_kernel<T, F, Square, true, true>
           : straight         ? &dev::block_quantize_kernel<T, F, Square, true, false>
                              : &dev::block_quantize_kernel<T, F, Square, false, true>;
}

template <class T>
Fn quant_fn(const QuantParams &p, int out_type)
{
    if (out_type == TP_E4M3)
        return p.square ? quant_fn<T, dev::E4m3, true>(p.q, p.qt) : quant_fn<T, dev::E4m3, false>(p.q, p.qt);
    return p.square ? quant_fn<T, dev::E5m2, true>(p.q, p.qt) : quant_fn<T, dev::E5m2, false>(p.q, p.qt);
}

}  // namespace

int launch_block_quantize(const QuantParams &p, int type, int out_type, void *stream)
{
    const Fn fn = type == TP_BF16   ? quant_fn<dev::Bf16>(p, out_type)
                  : type == TP_FP16 ? quant_fn<dev::Fp16>(p, out_type)
                                    : quant_fn<dev::Fp32>(p, out_type);
    QuantParams args = p;
    args.cached = quantize_cached(p, type);
    void *kargs[] = {&args};
    const int64_t tiles = p.across * op_ceil(p.rows, kOpBlock);
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3((uint32_t)tiles), dim3(256),
                                kargs, 0, (hipStream_t)stream);
}

}  // namespace tp
