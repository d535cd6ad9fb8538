// Root-mean-square norm with the residual's addition and an output in 8 bits:
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w,
//   and, for an 8-bit output, q = round8(y MOST / m), scale = m / MOST with m
//   the largest |y| of a block of 128 columns.
// y is rounded once, from 32 bits: neither the rounded s nor a rounded y
// enters the 8-bit output.
//
// Bound by memory: x and r are read once, s, y or q written once; the row
// stays in registers between its sum and its output, and the next row is in
// flight meanwhile. 8192 x 8192 bf16 with a residual into e4m3 (472 MB): 80 us,
// 5.9 TB/s. Few rows are bound by latency (1 x 4096: 2.8 us, of which an empty
// kernel takes 2).
#include "tp_rows.hpp"

namespace tp {
namespace dev {

struct Same {};

template <class T>
__device__ __forceinline__ void norm_sum_unit(const RawUnit<T> &x, float (&s)[kUnit], float &ss)
{
    unit_wide<T>(x, s);
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
        ss = fmaf(s[i], s[i], ss);
}

template <class T>
__device__ __forceinline__ void norm_sum_unit2(const RawUnit<T> &x, const RawUnit<T> &r,
                                               float (&s)[kUnit], float &ss)
{
    float b[kUnit];
    unit_wide<T>(x, s);
    unit_wide<T>(r, b);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
        s[i] += b[i];
        ss = fmaf(s[i], s[i], ss);
    }
}

// rstd as a power of two and a rest in [1, 2). An rstd of 0 (a sum of squares
// past fp32, an infinity in the row), infinity (a row of zeros with an eps of 0)
// or NaN is all power, with a rest of 1.
struct RowScale {
    float power, rest;

    __device__ __forceinline__ explicit RowScale(float rstd)
    {
        const uint32_t bits = __float_as_uint(rstd);
        const bool number = bits - 0x00800000u < 0x7F000000u;     // normal; it is never subnormal
        power = number ? __uint_as_float(bits & 0x7F800000u) : rstd;
        rest = number ? __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u) : 1.0f;
    }
};

// The outputs of one unit: y in T, or in 8 bits with its block's scale. The
// 16 lanes of a block hold its 128 columns. The 8-bit values need y only up to
// a factor of the row, since that is in the block's largest |y| too: so they are
// made from v = s w times rstd's power of two, with fewer roundings, and rstd's
// rest enters the scale. (s w alone could pass fp32 where y does not, and so
// could MOST over the s w that the least scale stands for: a block of zeros in
// a quiet row. The power costs 1 % at most: 8192 x 8192 bf16 into e4m3, replayed
// in a graph, 76.3 us without it and 76.9 with it.)
template <class T, class Out, class Rows>
__device__ __forceinline__ void norm_out_unit(const Rows &rows, int k, uint32_t first,
                                              const float (&s)[kUnit], float rstd, const RowScale &row,
                                              const RawUnit<T> &w, const BufferRes &out,
                                              const BufferRes &scale)
{
    float y[kUnit], wf[kUnit];
    unit_wide<T>(w, wf);
    if constexpr (std::is_same_v<Out, Same>) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i)
            y[i] = (s[i] * rstd) * wf[i];
        rows.store(out, k, unit_narrow<T>(y), first);
    } else {
        using Q = BlockQuotient<Fp32, Out>;    // v is not a number of T
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            y[i] = (s[i] * row.power) * wf[i];
            m = max(m, magnitude(y[i]));
        }
        m = group16_max(m);
        // the largest |y|, at least 2^-96, and the |v| that this is, 2^-97 at least
        const float most = __uint_as_float(max(magnitude(__uint_as_float(m) * row.rest), kLeastMost));
        const float of = __uint_as_float(max(m, magnitude(__uint_as_float(kLeastMost) / row.rest)));
        // MOST / of, to half an ulp or so; both over 2^8, so that 1 / of is not
        // subnormal for the largest
        const float off = of * 0x1p-8f, top = Out::most * 0x1p-8f;
        const float inverse = __builtin_amdgcn_rcpf(off), near = top * inverse;
        const float2 b = Q::make(BlockScale{fmaf(fmaf(-near, off, top), inverse, near), 0.0f, of});
#pragma unroll
        for (int i = 0; i < kUnit; ++i)
            y[i] = Q::of(Q::ready(y[i]), b);
        const u32x2 q = {pack4<Out>(y[0], y[1], y[2], y[3]), pack4<Out>(y[4], y[5], y[6], y[7])};
        rows.store_bytes(out, k, q, first);
        const uint32_t u = first + rows.unit(k);
        put_b32(scale, u % kLanesPerBlock == 0 ? u / kLanesPerBlock * 4 : kOutside,
                __float_as_uint(most * (1.0f / Out::most)));
    }
}

// 1 / sqrt(mean + eps): the hardware's estimate, off by an ulp or so, and one
// Newton step, which leaves about half an ulp. The values that it does not
// serve (zero, subnormal, huge, infinite, NaN) take the exact operations.
__device__ __forceinline__ float norm_rstd(float ss, const NormParams &p)
{
    const float v = fmaf(ss, 1.0f / (float)p.cols, p.eps);
    if (!(v > 1.0e-30f && v < 1.0e30f))
        return 1.0f / sqrtf(v);
    const float r = __builtin_amdgcn_rsqf(v);
    return fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
}

template <class T, class Out, bool Residual, int N, int Policy>
__global__ void __launch_bounds__(64 * row_max_waves(N)) rms_norm_kernel(NormParams p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int R = Residual ? 2 : 1;
    constexpr bool eight = !std::is_same_v<Out, Same>;
    // stores of a row, all issued after the next row's loads
    constexpr int stores = (Residual ? N * T::bytes / 2 : 0) + (eight ? 2 * N : N * T::bytes / 2) + 1;
    using Rows = RowStream<T, row_places(R, N), N, Policy>;
    const uint32_t threads = blockDim.x;
    float *red = reinterpret_cast<float *>(lds);
    Rows rows;
    rows.init(lds + kRowRedBytes, threads, (uint32_t)p.cols);

    const uint32_t row_bytes = (uint32_t)p.cols * T::bytes;
    const uint32_t blocks = ((uint32_t)p.cols + kOpBlock - 1) / kOpBlock;

    int64_t row = blockIdx.x;
    const int64_t step = gridDim.x;
    auto issue = [&](int64_t at) TP_INLINE {
        const uint32_t bytes = at < p.rows ? row_bytes : 0u;
        rows.issue(0, make_buffer_res(row_at(p.x, at, p.x_stride), bytes));
        if constexpr (Residual)
            rows.issue(1, make_buffer_res(row_at(p.r, at, p.r_stride), bytes));
    };
    // the weight stays in registers
    constexpr int weight_place = row_places(R, N) - 1;
    RawUnit<T> w[N];
    rows.issue(N == 1 ? weight_place : 0, make_buffer_res(p.w, row_bytes));
    if constexpr (N == 1)
        issue(row);
    vm_wait<0>();
#pragma unroll
    for (int k = 0; k < N; ++k)
        w[k] = rows.read(N == 1 ? weight_place : 0, k);
    rows.release();

    if constexpr (N != 1)
        issue(row);
    for (uint32_t turn = 0; row < p.rows; row += step, ++turn) {
        if (turn == 0)
            vm_wait<0>();
        else
            vm_wait<stores>();
        float s[N][kUnit], ss = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (Residual)
                norm_sum_unit2<T>(rows.read(0, k), rows.read(1, k), s[k], ss);
            else
                norm_sum_unit<T>(rows.read(0, k), s[k], ss);
        }
        rows.release();
        issue(row + step);

        const float rstd = norm_rstd(group_sum(ss, red, threads, turn & 1u), p);
        if constexpr (Residual) {
            const BufferRes res = make_buffer_res(row_at(p.sum, row, p.sum_stride), row_bytes);
#pragma unroll
            for (int k = 0; k < N; ++k)
                rows.store(res, k, unit_narrow<T>(s[k]));
        }
        const BufferRes out = make_buffer_res(row_at(p.out, row, p.out_stride),
                                              eight ? (uint32_t)p.cols : row_bytes);
        const BufferRes scale = make_buffer_res(eight ? p.scale + row * blocks : nullptr, blocks * 4);
        const RowScale row_scale(rstd);
#pragma unroll
        for (int k = 0; k < N; ++k)
            norm_out_unit<T, Out>(rows, k, 0, s[k], rstd, row_scale, w[k], out, scale);
        const BufferRes rs = make_buffer_res(p.rstd ? p.rstd + row : nullptr, p.rstd ? 4u : 0u);
        put_b32(rs, rows.tid * 4, __float_as_uint(rstd));
    }
    vm_wait<0>();
}

// Rows too long for a workgroup's registers: read once for the sum and again
// for the outputs, N units a lane at a time.
template <class T, class Out, bool Residual, int Policy>
__global__ void __launch_bounds__(512) rms_norm_long_kernel(NormParams p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int N = kRowUnits, R = Residual ? 3 : 2;
    constexpr bool eight = !std::is_same_v<Out, Same>;
    using Rows = RowStream<T, R, N, Policy>;
    const uint32_t threads = blockDim.x;
    float *red = reinterpret_cast<float *>(lds);
    Rows rows;
    rows.init(lds + kRowRedBytes, threads, (uint32_t)p.cols);
    const uint32_t row_bytes = (uint32_t)p.cols * T::bytes;
    const uint32_t blocks = ((uint32_t)p.cols + kOpBlock - 1) / kOpBlock;
    const uint32_t units = ((uint32_t)p.cols + kUnit - 1) / kUnit;
    const BufferRes rw = make_buffer_res(p.w, row_bytes);
    uint32_t turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++turn) {
        const BufferRes rx = make_buffer_res(row_at(p.x, row, p.x_stride), row_bytes);
        const BufferRes rr = make_buffer_res(Residual ? row_at(p.r, row, p.r_stride) : nullptr, row_bytes);
        float ss = 0.0f, s[kUnit];
        for (uint32_t first = 0; first < units; first += N * threads) {
            rows.issue(0, rx, first);
            if constexpr (Residual)
                rows.issue(1, rr, first);
            vm_wait<0>();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if constexpr (Residual)
                    norm_sum_unit2<T>(rows.read(0, k, first), rows.read(1, k, first), s, ss);
                else
                    norm_sum_unit<T>(rows.read(0, k, first), s, ss);
            }
            rows.release();
        }
        const float rstd = norm_rstd(group_sum(ss, red, threads, turn & 1u), p);
        const BufferRes rsum = make_buffer_res(Residual ? row_at(p.sum, row, p.sum_stride) : nullptr,
                                               row_bytes);
        const BufferRes out = make_buffer_res(row_at(p.out, row, p.out_stride),
                                              eight ? (uint32_t)p.cols : row_bytes);
        const BufferRes scale = make_buffer_res(eight ? p.scale + row * blocks : nullptr, blocks * 4);
        const RowScale row_scale(rstd);
        for (uint32_t first = 0; first < units; first += N * threads) {
            rows.issue(0, rx, first);
            if constexpr (Residual)
                rows.issue(1, rr, first);
            rows.issue(R - 1, rw, first);
            vm_wait<0>();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if constexpr (Residual) {
                    norm_sum_unit2<T>(rows.read(0, k, first), rows.read(1, k, first), s, ss);
                    rows.store(rsum, k, unit_narrow<T>(s), first);
                } else {
                    norm_sum_unit<T>(rows.read(0, k, first), s, ss);
                }
                norm_out_unit<T, Out>(rows, k, first, s, rstd, row_scale, rows.read(R - 1, k, first), out,
                                      scale);
            }
            rows.release();
        }
        const BufferRes rs = make_buffer_res(p.rstd ? p.rstd + row : nullptr, p.rstd ? 4u : 0u);
        put_b32(rs, rows.tid * 4, __float_as_uint(rstd));
    }
    vm_wait<0>();
}

}  // namespace dev

namespace {

using Fn = void (*)(NormParams);

template <class T, class Out, bool Residual, int Policy>
Fn norm_fn(int units)
{
    return units == 0 ? &dev::rms_norm_long_kernel<T, Out, Residual, Policy>
           : units == 1 ? &dev::rms_norm_kernel<T, Out, Residual, 1, Policy>
                        : &dev::rms_norm_kernel<T, Out, Residual, kRowUnits, Policy>;
}

template <class T, bool Residual, int Policy>
Fn norm_fn(int out_type, int units)
{
    return out_type == TP_E4M3   ? norm_fn<T, dev::E4m3, Residual, Policy>(units)
           : out_type == TP_E5M2 ? norm_fn<T, dev::E5m2, Residual, Policy>(units)
                                 : norm_fn<T, dev::Same, Residual, Policy>(units);
}

template <class T, bool Residual>
Fn norm_fn(int out_type, int units, int policy)
{
    return policy == kRowPast           ? norm_fn<T, Residual, kRowPast>(out_type, units)
           : policy == kRowStoresPast ? norm_fn<T, Residual, kRowStoresPast>(out_type, units)
                                      : norm_fn<T, Residual, kRowCached>(out_type, units);
}

template <class T>
Fn norm_fn(const NormParams &p, int out_type, int units, int policy)
{
    return p.r ? norm_fn<T, true>(out_type, units, policy) : norm_fn<T, false>(out_type, units, policy);
}

}  // namespace

int launch_rms_norm(const NormParams &p, int type, int out_type, void *stream)
{
    const RowPlan plan = norm_plan(p.rows, p.cols, type, p.r != nullptr);
    const int policy = norm_policy(p, type, out_type);
    const Fn fn = type == TP_BF16   ? norm_fn<dev::Bf16>(p, out_type, plan.units, policy)
                  : type == TP_FP16 ? norm_fn<dev::Fp16>(p, out_type, plan.units, policy)
                                    : norm_fn<dev::Fp32>(p, out_type, plan.units, policy);
    NormParams args = p;
    void *kargs[] = {&args};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3((uint32_t)plan.grid),
                                dim3((uint32_t)plan.waves * 64), kargs, (size_t)plan.lds_bytes,
                                (hipStream_t)stream);
}

}  // namespace tp
