// Host-side checks and launch rules of the 8-bit linear layer's operators.
// Pure C++: no HIP calls.
#include <math.h>
#include <string.h>

#include "tp_ops_plan.hpp"

namespace tp {
namespace {

// A buffer of an argument list: where it is, and the bytes from its first to
// its last element.
struct Span {
    uintptr_t at;
    uint64_t bytes;
    int64_t stride;
};

Span matrix_span(uintptr_t p, int64_t rows, int64_t cols, int64_t stride, int bytes)
{
    const bool empty = !p || rows == 0 || cols == 0;
    return Span{p, empty ? 0 : (uint64_t)((rows - 1) * stride + cols) * (uint64_t)bytes,
                stride * bytes};
}

Span vector_span(uintptr_t p, int64_t n, int bytes)
{
    return Span{p, p ? (uint64_t)n * (uint64_t)bytes : 0, 0};
}

bool meet(const Span &a, const Span &b)
{
    return a.bytes && b.bytes && a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}

bool same(const Span &a, const Span &b)
{
    return a.at == b.at && a.bytes == b.bytes && a.stride == b.stride;
}

// Outputs must not meet one another, nor an input that is not the very same
// buffer; `in_place` says whether being the same is allowed.
template <int O, int I>
int check_overlap(const Span (&out)[O], const Span (&in)[I], bool in_place)
{
    for (int i = 0; i < O; ++i) {
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j]))
                return TP_ERR_OVERLAP;
        for (int j = 0; j < I; ++j)
            if (meet(out[i], in[j]) && !(in_place && same(out[i], in[j])))
                return TP_ERR_OVERLAP;
    }
    return TP_OK;
}

bool valid_stride(int64_t stride, int64_t cols) { return stride >= cols && stride <= kOpMaxStride; }

bool is_number_type(int type) { return type == TP_BF16 || type == TP_FP16 || type == TP_FP32; }
bool is_eight_bit(int type) { return type == TP_E4M3 || type == TP_E5M2; }
bool aligned(uintptr_t p, int bytes) { return p % (uintptr_t)bytes == 0; }

void fill_plan(tp_plan *plan, int threads, int lds, int64_t tiles, int64_t grid, int tile_units, int stages = 1)
{
    if (!plan)
        return;
    memset(plan, 0, sizeof *plan);
    plan->stages = stages;
    plan->threads = threads;
    plan->lds_bytes = lds;
    plan->ring_bytes = lds;
    plan->num_tiles = tiles;
    plan->grid = grid;
    plan->tile_units = tile_units;
    plan->lane_chunks = 1;
    plan->tiles_per_block = 1;
}

// Workgroups of a row kernel: as many as stay resident, and rows shared out
// evenly among them.
int64_t even_grid(int64_t rows, int64_t most)
{
    if (rows <= most)
        return rows;
    return op_ceil(rows, op_ceil(rows, most));
}

// Resident waves of the row kernels. While every workgroup has several rows,
// few of them stream best: the rows in flight then lie close together (8192 x
// 8192 bf16 with a residual: 86 us with 4 waves a CU, 90 with 8, 95 with 12;
// the gradient of 8192 x 4096: 52, 56, 61). With fewer rows it is their number
// in flight that counts (777 x 5003: 11.5 us with 4, 7.5 with 16). The rule counts
// rows, not bytes, and so serves narrow ones badly: 8192 x 128 bf16 with a
// residual takes 8.8 us with 4 waves a CU, 8191 x 128 6.0 with 16; 524288 x 128
// (474 MB) 360.
constexpr int kRowWavesPerCu = 4;
constexpr int kFewRowsWavesPerCu = 16;
// The gradient writes and adds a row of partial sums for each workgroup, and
// stays at the smaller number (2767 x 1174 bf16: 13.8 us with 4, 14.7 with 8,
// 21.2 with 16).
constexpr int kManyRows = 8;          // of a workgroup

// How a workgroup of a row kernel holds a row. Few rows: one unit a lane, so
// that a row's latency is spread over as many lanes as it has units. Many
// rows: kRowUnits units a lane, fewer waves to add over.
RowPlan row_plan(int tensors, int more_lds, int64_t rows, int64_t cols, int bytes, int few_rows_waves)
{
    const int64_t units = op_ceil(cols, 8);
    RowPlan p{};
    const int64_t wide = op_ceil(units, 64), narrow = op_ceil(units, 64 * kRowUnits);
    p.units = wide <= kRowMaxWaves && (units <= 64 || rows * narrow < 4 * kOpCus) ? 1 : kRowUnits;
    const int64_t waves = p.units == 1 ? wide : narrow;
    const int64_t lds = kRowRedBytes + waves * (row_wave_lds(row_places(tensors, p.units), p.units, bytes) + more_lds);
    if (waves > row_max_waves(p.units) || lds > kLdsPerCu) {
        p.units = 0;
        return p;
    }
    p.waves = (int)waves;
    p.lds_bytes = (int)lds;
    const auto resident = [&](int waves_per_cu) {
        int64_t n = kLdsPerCu / p.lds_bytes;
        if (n > waves_per_cu / p.waves)
            n = waves_per_cu / p.waves;
        return (n < 1 ? 1 : n) * kOpCus;
    };
    const int64_t few = resident(kRowWavesPerCu);
    p.grid = even_grid(rows, rows >= kManyRows * few ? few : resident(few_rows_waves));
    return p;
}

// Cache policies of the row kernels. Their stores are written through, so that
// a kernel's end finds few dirty lines. Up to kCachedLoadBytes of tensors the
// loads take the ordinary policy: what ran before has left part of them in the
// last cache (256 MiB), and they stay there for what runs next (2048 x 4096
// bf16 with a residual: 11.4 us, 13.8 with non-temporal loads; its gradient
// 16.9 and 20.0; 1500 x 8200: 16.9 and 22.7). Above, they are non-temporal
// (2500 x 8200, 164 MB: 29.0 us, 32.5 ordinary; 8192 x 8192: 80 and 84).
// Where rows start inside a line and the tensors are more than the cache
// holds, a line that is written in two parts at different times costs memory
// twice, and the ordinary policy for both waits for the whole line (the norm
// of 8192 x 4104 fp32, 538 MB: 101 us, 156 past the caches; 4400 rows, 289 MB:
// 55.9 and 54.6). The gradient, which reads more and writes less, gains
// nothing by that (8192 x 8200 bf16: 102 us, 93).
constexpr int64_t kCachedLoadBytes = int64_t(128) << 20;
constexpr int64_t kCachedBytes = int64_t(300) << 20;
constexpr int64_t kLine = 128;

bool on_lines(const void *p, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride) % kLine == 0;
}

}  // namespace

int norm_policy(const NormParams &p, int type, int out_type)
{
    const int64_t bytes = p.rows * p.cols * ((p.r ? 3 : 1) * type_bytes(type) + type_bytes(out_type));
    if (bytes <= kCachedLoadBytes)
        return kRowStoresPast;
    const bool lines = on_lines(p.x, p.x_stride) && on_lines(p.out, p.out_stride) &&
                       (!p.r || (on_lines(p.r, p.r_stride) && on_lines(p.sum, p.sum_stride)));
    return lines || bytes <= kCachedBytes ? kRowPast : kRowCached;
}

int norm_grad_policy(const NormGradParams &p, int type)
{
    const int64_t bytes = p.rows * p.cols * (p.ds ? 4 : 3) * type_bytes(type);
    return bytes <= kCachedLoadBytes ? kRowStoresPast : kRowPast;
}

// The quantiser's loads, by the same rule (4096 x 4100 bf16 both ways: 19.8 us,
// 26.3 non-temporal; 8192 x 8192: 61.1 and 52.7).
bool quantize_cached(const QuantParams &p, int type)
{
    return p.rows * p.cols * (type_bytes(type) + (p.q != nullptr) + (p.qt != nullptr)) <= kCachedLoadBytes;
}

RowPlan norm_plan(int64_t rows, int64_t cols, int type, bool residual)
{
    const int bytes = type_bytes(type);
    RowPlan p = row_plan(residual ? 2 : 1, 0, rows, cols, bytes, kFewRowsWavesPerCu);
    if (p.units == 0) {
        const int tensors = residual ? 3 : 2;
        p.waves = bytes == 4 ? 4 : 8;
        p.lds_bytes = kRowRedBytes + p.waves * row_wave_lds(tensors, kRowUnits, bytes);
        p.grid = even_grid(rows, kOpCus);
    }
    return p;
}

int64_t norm_grad_groups(int64_t rows, int64_t cols, int type)
{
    return norm_grad_plan(rows, cols, type, true).grid;
}

RowPlan norm_grad_plan(int64_t rows, int64_t cols, int type, bool more)
{
    const int bytes = type_bytes(type);
    // sized as with the second gradient, so that both forms have the same
    // workgroups and one workspace
    RowPlan p = row_plan(3, kRowCutBytes, rows, cols, bytes, kRowWavesPerCu);
    if (p.units == 0) {
        p.waves = bytes == 4 ? 2 : 4;
        p.lds_bytes = kRowRedBytes + p.waves * (row_wave_lds(4, kRowUnits, bytes) + kRowCutBytes);
        // all partial sums of dw lie below the offset that stands for no place
        // (dx is made by as few workgroups, which leaves most CUs idle: 4096 x
        // 18432 bf16 with a second gradient 850 us, its bytes 90)
        const int64_t most = (int64_t(1) << 30) / (partial_pitch(cols) * 4);
        p.grid = even_grid(rows, most < kOpCus / 4 ? most : kOpCus / 4);
    } else if (!more) {
        p.lds_bytes = kRowRedBytes + p.waves * (row_wave_lds(row_places(2, p.units), p.units, bytes) + kRowCutBytes);
    }
    return p;
}

int64_t rms_norm_backward_workspace(int64_t rows, int64_t cols, int type)
{
    if (rows < 0 || rows > kOpMaxRows || cols < 0 || cols > kOpMaxCols || !is_number_type(type))
        return -1;
    return rows == 0 || cols == 0 ? 0 : norm_grad_groups(rows, cols, type) * partial_pitch(cols) * 4;
}

int plan_rms_norm(uintptr_t x, int64_t x_stride, uintptr_t r, int64_t r_stride, uintptr_t w,
                  int64_t rows, int64_t cols, int type, float eps, uintptr_t sum,
                  int64_t sum_stride, uintptr_t out, int64_t out_stride, int out_type,
                  uintptr_t scale, uintptr_t rstd, tp_plan *plan)
{
    if (rows < 0 || rows > kOpMaxRows || cols < 0 || cols > kOpMaxCols || !is_number_type(type))
        return TP_ERR_INVALID_ARG;
    if (out_type != type && !is_eight_bit(out_type))
        return TP_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || isinf(eps))
        return TP_ERR_INVALID_ARG;
    const bool eight = out_type != type;
    if ((r != 0) != (sum != 0) || (eight != (scale != 0)))
        return TP_ERR_INVALID_ARG;
    if (!valid_stride(x_stride, cols) || !valid_stride(out_stride, cols) ||
        (r && (!valid_stride(r_stride, cols) || !valid_stride(sum_stride, cols))))
        return TP_ERR_INVALID_ARG;
    fill_plan(plan, 0, 0, rows, 0, (int)cols);
    if (rows == 0 || cols == 0)
        return TP_OK;
    if (!x || !w || !out)
        return TP_ERR_INVALID_ARG;
    const int b = type_bytes(type);
    if (!aligned(x, b) || !aligned(r, b) || !aligned(w, b) || !aligned(sum, b) ||
        (!eight && !aligned(out, b)) || !aligned(scale, 4) || !aligned(rstd, 4))
        return TP_ERR_MISALIGNED;
    const Span outs[] = {matrix_span(sum, rows, cols, sum_stride, b),
                         matrix_span(out, rows, cols, out_stride, type_bytes(out_type)),
                         vector_span(scale, rows * op_ceil(cols, kOpBlock), 4), vector_span(rstd, rows, 4)};
    const Span ins[] = {matrix_span(x, rows, cols, x_stride, b), matrix_span(r, rows, cols, r_stride, b)};
    const Span kept[] = {vector_span(w, cols, b)};
    int st = check_overlap(outs, ins, true);
    if (st == TP_OK)
        st = check_overlap(outs, kept, false);
    if (st != TP_OK)
        return st;
    const RowPlan p = norm_plan(rows, cols, type, r != 0);
    fill_plan(plan, p.waves * 64, p.lds_bytes, rows, p.grid, (int)cols);
    return TP_OK;
}

int plan_rms_norm_backward(uintptr_t dy, int64_t dy_stride, uintptr_t x, int64_t x_stride,
                           uintptr_t w, uintptr_t rstd, uintptr_t ds, int64_t ds_stride,
                           int64_t rows, int64_t cols, int type, uintptr_t dx, int64_t dx_stride,
                           uintptr_t dw, uintptr_t workspace, int64_t workspace_bytes,
                           tp_plan *plan)
{
    const int64_t need = rms_norm_backward_workspace(rows, cols, type);
    if (need < 0)
        return TP_ERR_INVALID_ARG;
    if (!valid_stride(dy_stride, cols) || !valid_stride(x_stride, cols) || !valid_stride(dx_stride, cols) ||
        (ds && !valid_stride(ds_stride, cols)))
        return TP_ERR_INVALID_ARG;
    fill_plan(plan, 0, 0, rows, 0, (int)cols);
    if (cols == 0)
        return TP_OK;
    if (!dw || (rows > 0 && (!dy || !x || !w || !rstd || !dx || !workspace || workspace_bytes < need)))
        return TP_ERR_INVALID_ARG;
    const int b = type_bytes(type);
    if (!aligned(dw, 4) || !aligned(rstd, 4) || !aligned(workspace, 4))
        return TP_ERR_MISALIGNED;
    if (!aligned(dy, b) || !aligned(x, b) || !aligned(w, b) || !aligned(ds, b) || !aligned(dx, b))
        return TP_ERR_MISALIGNED;
    const Span ins[] = {matrix_span(dy, rows, cols, dy_stride, b), matrix_span(x, rows, cols, x_stride, b),
                        matrix_span(ds, rows, cols, ds_stride, b)};
    const Span kept[] = {vector_span(w, cols, b), vector_span(rstd, rows, 4)};
    const Span dxs = matrix_span(dx, rows, cols, dx_stride, b);
    const Span outs[] = {dxs, vector_span(dw, cols, 4), vector_span(workspace, need, 1)};
    const Span last[] = {outs[1], outs[2]};
    // dx may be one of the inputs where every input element is read before
    // its place is written: not where rows are read twice
    const RowPlan p = norm_grad_plan(rows > 0 ? rows : 1, cols, type, ds != 0);
    int st = check_overlap(outs, kept, false);
    if (st == TP_OK)
        st = check_overlap(outs, ins, p.units != 0);
    if (st == TP_OK)
        st = check_overlap(last, ins, false);
    if (st != TP_OK)
        return st;
    fill_plan(plan, p.waves * 64, p.lds_bytes, rows, rows ? p.grid : 0, (int)cols);
    return TP_OK;
}

// Rows of a tile are addressed with 32-bit offsets: 256 of them.
constexpr int64_t kTileMaxPitch = int64_t(1) << 22;
constexpr int64_t kTileMaxSpan = kTileMaxPitch * 256;

int plan_block_quantize(uintptr_t x, int64_t x_stride, int64_t rows, int64_t cols, int type,
                        int square, int out_type, uintptr_t q, int64_t q_stride, uintptr_t scale,
                        uintptr_t qt, int64_t qt_stride, uintptr_t scale_t, tp_plan *plan)
{
    if (rows < 0 || rows > kOpMaxRows || cols < 0 || cols > kOpMaxCols || !is_number_type(type) ||
        !is_eight_bit(out_type) || (square != 0 && square != 1))
        return TP_ERR_INVALID_ARG;
    const int b = type_bytes(type);
    if (!valid_stride(x_stride, cols) || x_stride * b > kTileMaxPitch)
        return TP_ERR_INVALID_ARG;
    fill_plan(plan, 0, 0, 0, 0, kOpBlock);
    const int64_t tiles = op_ceil(rows, kOpBlock) * op_ceil(cols, kOpBlock);
    if (tiles == 0)
        return TP_OK;
    if (!x || (!q && !qt) || (q != 0) != (scale != 0) || (qt != 0) != (scale_t != 0) || tiles > INT32_MAX)
        return TP_ERR_INVALID_ARG;
    if (q && (!valid_stride(q_stride, cols) || q_stride > kTileMaxPitch))
        return TP_ERR_INVALID_ARG;
    if (qt && (!valid_stride(qt_stride, rows) || qt_stride > kTileMaxPitch))
        return TP_ERR_INVALID_ARG;
    if (!aligned(x, b) || !aligned(scale, 4) || !aligned(scale_t, 4))
        return TP_ERR_MISALIGNED;
    const int64_t down = op_ceil(rows, kOpBlock), across = op_ceil(cols, kOpBlock);
    const Span outs[] = {matrix_span(q, rows, cols, q_stride, 1), matrix_span(qt, cols, rows, qt_stride, 1),
                         vector_span(scale, (square ? down : rows) * across, 4),
                         vector_span(scale_t, (square ? across : cols) * down, 4)};
    const Span ins[] = {matrix_span(x, rows, cols, x_stride, b)};
    const int st = check_overlap(outs, ins, false);
    if (st != TP_OK)
        return st;
    fill_plan(plan, 256, kQuantLdsBytes, tiles, tiles, kOpBlock);
    return TP_OK;
}

namespace {

// What a shape of the product's tiles costs on an MI355X, in microseconds,
// measured over sums of 4 to 32 blocks with one round of workgroups: a block
// of 128 with one workgroup on each CU, the same with `resident` of them, and
// the rest of a round (launch, first loads, output; of several rounds each
// hides a quarter of it in the others). Operands turned into fp16 are twice as
// wide in registers and take twice the matrix time. The smallest shape is for
// outputs of few tiles (1000 x 1000 x 1000 into bf16: 9.3 us, 13.3 by tiles of
// 128; 512 x 4096 x 4096: 25.9 and 32.6; 768 x 4096 x 512: 12.0 and 8.3).
struct ShapeCost {
    int shape, tile_m, tile_n, resident;
    double block_alone, block_full, round;
};
constexpr ShapeCost kCosts[] = {
    {kMatmul64, 64, 64, 2, 0.53, 0.69, 4.5},
    {kMatmul128, 128, 128, 2, 0.85, 1.12, 6.0},
    {kMatmul128x256, 128, 256, 1, 0.93, 0.93, 7.0},
    {kMatmul256, 256, 256, 1, 1.58, 1.58, 9.0},
};
constexpr ShapeCost kWideCosts[] = {
    {kMatmul64, 64, 64, 2, 0.87, 1.20, 4.5},
    {kMatmul128, 128, 128, 2, 1.29, 2.5, 6.5},
    {kMatmul128x256, 128, 256, 1, 1.66, 1.66, 8.0},
};
// The same of the skinny kernel with 32, 48 and 64 rows: workgroups on a CU, a
// round of them, a block of each of their waves; and its launch.
struct SkinnyCost {
    int resident;
    double round, block;
};
constexpr SkinnyCost kSkinnyCosts[] = {{2, 1.8, 1.5}, {2, 2.3, 1.65}, {1, 2.6, 1.0}};
constexpr double kSkinnyStart = 2.0;
constexpr int kMostSplits = 16;
constexpr double kJoinStart = 2.5;            // us of a second launch
constexpr double kJoinBytesPerUs = 4.0e6;     // its traffic

double tile_cost(const ShapeCost &c, int64_t m, int64_t n, int64_t blocks, int splits)
{
    const int64_t groups = op_ceil(m, c.tile_m) * op_ceil(n, c.tile_n) * splits;
    const int64_t rounds = op_ceil(groups, (int64_t)kOpCus * c.resident);
    const double block = groups <= kOpCus ? c.block_alone : c.block_full;
    const double join = splits > 1 ? kJoinStart + (double)m * (double)n * (8.0 * splits + 4.0) / kJoinBytesPerUs : 0.0;
    return (double)rounds * ((double)op_ceil(blocks, splits) * block + c.round * (rounds > 1 ? 0.75 : 1.0)) + join;
}

}  // namespace

// How the product is cut. Up to 64 rows of a: the skinny kernel, whose
// workgroups make 16 columns. Otherwise the tiles, and the number of
// workgroups that share a tile's sum, that cost least. The skinny kernel reads
// a once for every 16 columns; where that is several rows for one of b and
// takes several rounds of workgroups, its cost is compared with the tiles' (64
// x 16384 x 4096 into bf16: 26.3 us, 21.3 by tiles; 32 x 64000 x 2048: 45.6 and
// 29.9; 64 x 4096 x 4096, one round: 8.5 and 13.2).
MatmulPlan matmul_plan(int64_t m, int64_t n, int64_t k, int out_type)
{
    MatmulPlan p{};
    const int64_t blocks = op_ceil(k, kOpBlock);
    const bool can_split = m * n <= int64_t(1) << 24 && m <= 65535;
    p.splits = 1;
    double best = 0.0;
    if (m <= 64) {
        p.shape = kMatmulSkinny;
        p.tile_m = m <= 16 ? 16 : m <= 32 ? 32 : m <= 48 ? 48 : 64;
        p.tile_n = 16;
        const int64_t tiles = op_ceil(n, 16);
        int64_t splits = tiles > 0 ? kOpCus / tiles : 1;
        if (splits > blocks / 16)
            splits = blocks / 16;
        p.waves = kSkinnyWaves;
        if (splits > 1 && can_split)
            p.splits = (int)(splits < kMostSplits ? splits : kMostSplits);
        if (m > 16) {
            const SkinnyCost &c = kSkinnyCosts[p.tile_m / 16 - 2];
            const int64_t rounds = op_ceil(tiles, kOpCus * c.resident);
            if (rounds > 1)
                best = kSkinnyStart + (double)rounds * (c.round + (double)op_ceil(blocks, p.waves) * c.block);
        }
    }
    if (m > 64 || best > 0.0) {
        const bool wide = matmul_wide(out_type);
        const ShapeCost *costs = wide ? kWideCosts : kCosts;
        const int shapes = wide ? 3 : 4;
        for (int i = 0; i < shapes; ++i) {
            const ShapeCost &c = costs[i];
            if (c.shape == kMatmul256 && k % 16 != 0)
                continue;      // its registers leave no room for a cut chunk
            for (int splits = 1; splits <= kMostSplits && (splits == 1 || (can_split && blocks / splits >= 4)); ++splits) {
                const double cost = tile_cost(c, m, n, blocks, splits);
                if (best == 0.0 || cost < best) {
                    best = cost;
                    p.shape = c.shape;
                    p.tile_m = c.tile_m;
                    p.tile_n = c.tile_n;
                    p.waves = c.shape == kMatmul64 ? 2 : c.shape == kMatmul128 ? 4 : 8;
                    p.splits = splits;
                }
            }
        }
    }
    const int64_t groups = op_ceil(m, p.tile_m) * op_ceil(n, p.tile_n) * p.splits;
    if (p.shape == kMatmulSkinny) {
        // blocks of a wave: with more than 4 a second slot pays (1 x 16384 x
        // 8192: 28.3 us against 30.3), with fewer the smaller LDS does (1 x
        // 8192 x 4096: 9.7 against 10.1); more rows of a fill one slot's time
        p.stages = p.tile_m == 16 && op_ceil(blocks, p.splits * kSkinnyWaves) > 4 ? 2 : 1;
        p.lds_bytes = matmul_skinny_lds(p.tile_m, p.stages);
        p.grid = groups;
    } else {
        p.stages = matmul_stages(p.shape);
        p.lds_bytes = matmul_tile_lds(p.tile_m, p.tile_n, p.stages);
        p.grid = op_ceil(groups, 8) * 8;     // as many for each XCD
    }
    p.partial_bytes = p.splits > 1 ? p.splits * m * n * 4 : 0;
    return p;
}

int64_t block_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_type)
{
    if (m < 0 || n < 0 || k < 0 || m > kOpMaxRows || n > kOpMaxRows || k > kTileMaxPitch ||
        !is_number_type(out_type))
        return -1;
    return m == 0 || n == 0 ? 0 : matmul_plan(m, n, k, out_type).partial_bytes;
}

int plan_block_matmul(uintptr_t a, int64_t a_stride, int a_type, uintptr_t sa, uintptr_t b,
                      int64_t b_stride, int b_type, uintptr_t sb, int b_square, int64_t m,
                      int64_t n, int64_t k, uintptr_t out, int64_t out_stride, int out_type,
                      uintptr_t workspace, int64_t workspace_bytes, tp_plan *plan)
{
    const int64_t need = block_matmul_workspace(m, n, k, out_type);
    if (need < 0 || !is_eight_bit(a_type) || !is_eight_bit(b_type) ||
        (b_square != 0 && b_square != 1))
        return TP_ERR_INVALID_ARG;
    const int ob = type_bytes(out_type);
    if (!valid_stride(a_stride, k) || a_stride > kTileMaxPitch || !valid_stride(b_stride, k) ||
        b_stride > kTileMaxPitch || !valid_stride(out_stride, n) ||
        (m > 1 && out_stride * ob > kTileMaxSpan / (m < 256 ? m : 256)))
        return TP_ERR_INVALID_ARG;
    fill_plan(plan, 0, 0, 0, 0, 0);
    if (m == 0 || n == 0)
        return TP_OK;
    if (!out || (k > 0 && (!a || !b || !sa || !sb)) || (need > 0 && (!workspace || workspace_bytes < need)))
        return TP_ERR_INVALID_ARG;
    if (!aligned(sa, 4) || !aligned(sb, 4) || !aligned(out, ob) || !aligned(workspace, 4))
        return TP_ERR_MISALIGNED;
    const int64_t blocks = op_ceil(k, kOpBlock);
    const Span outs[] = {matrix_span(out, m, n, out_stride, ob), vector_span(workspace, need, 1)};
    const Span ins[] = {matrix_span(a, m, k, a_stride, 1), matrix_span(b, n, k, b_stride, 1),
                        vector_span(sa, m * blocks, 4),
                        vector_span(sb, (b_square ? op_ceil(n, kOpBlock) : n) * blocks, 4)};
    const int st = check_overlap(outs, ins, false);
    if (st != TP_OK)
        return st;
    const MatmulPlan p = matmul_plan(m, n, k, out_type);
    const int64_t tiles = op_ceil(m, p.tile_m) * op_ceil(n, p.tile_n);
    if (p.grid * 64 * p.waves > UINT32_MAX)     // lanes of a launch
        return TP_ERR_INVALID_ARG;
    fill_plan(plan, 64 * p.waves, p.lds_bytes, tiles, p.grid, p.tile_m, p.stages);
    return TP_OK;
}

}  // namespace tp
