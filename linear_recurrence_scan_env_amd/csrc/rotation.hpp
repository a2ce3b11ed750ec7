// rotation.hpp -- the norm of queries and keys for each head with the position
// rotation in the same pass.  Per token and head, over the head's `dim`
// elements x:
//
//     n = x * rsqrt(mean(x^2) + eps),   z = n * w,
//
// then the first rotary_dim elements of z are rotated in pairs by the angles
// of the token's position p: (z_a, z_b) -> (z_a cos - z_b sin, z_b cos + z_a
// sin) with cos = table[p][j], sin = table[p][rotary_dim / 2 + j] for pair j,
// (a, b) = (j, j + rotary_dim / 2), or (2j, 2j + 1) where interleaved.
// Backward, with u the output's gradient rotated back:
//
//     dw = sum over tokens and heads of u * n,
//     dx = rsqrt(...) * (u w - n * mean(u w n)).
#pragma once

#include "sequence.hpp"

namespace lrs {

constexpr int kMaxHeadDim = 256;

// The queries' or the keys' arrays.
struct NormSide {
    SeqView x, dy, y;  // y: the output, or backward the gradient of x
    const void* w;
    float* part;       // backward: [blocks, dim] sums of u * n
    int64_t rows;      // N * T * heads
    int32_t heads;
    uint32_t blocks;
};

struct NormArgs {
    NormSide side[2];
    SeqView positions;
    const float* table;
    int64_t N, T, max_positions;
    int32_t dim, rot;
    float eps;
    int32_t interleaved;
};

constexpr int kNormWaves = 4;

// One wave per row.
template <class D, bool kBackward>
__global__ __launch_bounds__(kNormWaves * kWave) void norm_rotation(const NormArgs x)
{
    constexpr int E = kMaxHeadDim / kWave;
    __shared__ float row[kNormWaves][kMaxHeadDim];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const bool keys = blockIdx.x >= x.side[0].blocks;
    const NormSide& s = x.side[keys ? 1 : 0];
    const uint32_t block = keys ? blockIdx.x - x.side[0].blocks : blockIdx.x;
    const int half = x.rot / 2;
    float w[E], dw[E];
    int other[E], pair[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int e = lane + i * kWave;
        w[i] = e < x.dim ? to_f32(static_cast<const D*>(s.w)[e]) : 0.0f;
        dw[i] = 0.0f;
        pair[i] = x.interleaved ? e / 2 : (e < half ? e : e - half);
        other[i] = x.interleaved ? e ^ 1 : (e < half ? e + half : e - half);
    }
    float* const z = row[wave];
    for (int64_t r = (int64_t)block * kNormWaves + wave; r < s.rows; r += (int64_t)s.blocks * kNormWaves) {
        const int64_t tok = r / s.heads, n = tok / x.T, t = tok % x.T;
        const int h = (int)(r % s.heads);
        float v[E], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = lane + i * kWave;
            v[i] = e < x.dim ? to_f32(seq_row<D>(s.x, n, t, h)[e]) : 0.0f;
            sum = fmaf(v[i], v[i], sum);
        }
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        const float scale = rsqrtf(sum / x.dim + x.eps);
        const int64_t p = x.rot ? *seq_row<int32_t>(x.positions, n, t, 0) : 0;
        const bool in = x.rot == 0 || (p >= 0 && p < x.max_positions);
        const float* angle = x.table + (in ? p : 0) * x.rot;
        float u[E], g[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = lane + i * kWave;
            v[i] *= scale;
            g[i] = kBackward && e < x.dim ? to_f32(seq_row<D>(s.dy, n, t, h)[e]) : v[i] * w[i];
            if (e < x.dim) z[e] = g[i];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = lane + i * kWave;
            u[i] = g[i];
            if (e < x.rot) {
                const float c = angle[pair[i]], si = angle[half + pair[i]];
                // first of its pair: minus the other's sine part (backward the signs turn over)
                const bool first = e < other[i];
                const float turn = first != kBackward ? -si : si;
                u[i] = fmaf(g[i], c, turn * z[other[i]]);
            }
            if (!in) u[i] = __builtin_nanf("");
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (kBackward) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                dw[i] = fmaf(u[i], v[i], dw[i]);
                u[i] *= w[i];
                dot = fmaf(u[i], v[i], dot);
            }
            for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
            dot /= x.dim;
#pragma unroll
            for (int i = 0; i < E; ++i) u[i] = scale * (u[i] - v[i] * dot);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = lane + i * kWave;
            if (e < x.dim) seq_row_out<D>(s.y, n, t, h)[e] = from_f32<D>(u[i]);
        }
    }
    if constexpr (kBackward) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) row[wave][lane + i * kWave] = dw[i];
        __syncthreads();
        for (int e = threadIdx.x; e < x.dim; e += kNormWaves * kWave) {
            float sum = 0.0f;
            for (int k = 0; k < kNormWaves; ++k) sum += row[k][e];
            s.part[(int64_t)block * x.dim + e] = sum;
        }
    }
}

// dw from the blocks' sums, in a fixed order: one block per element of dim.
struct WeightSumArgs {
    const float* part[2];
    void* dw[2];
    uint32_t blocks[2];
    int32_t dim;
};

template <class D>
__global__ __launch_bounds__(256) void weight_sum(const WeightSumArgs x)
{
    __shared__ float part[4];
    const int side = blockIdx.x / x.dim, e = blockIdx.x % x.dim;
    float sum = 0.0f;
    for (uint32_t b = threadIdx.x; b < x.blocks[side]; b += 256)
        sum += x.part[side][(int64_t)b * x.dim + e];
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        static_cast<D*>(x.dw[side])[e] = from_f32<D>(part[0] + part[1] + part[2] + part[3]);
}

// ------------------------------------------------------------------ entries

inline lrs_status check_rotation(const char* nm, int64_t N, int64_t T, int64_t HQ, int64_t HK,
                                 int64_t dim, int64_t rot, const void* qw, const void* kw,
                                 const void* table, int64_t max_positions, const void* positions,
                                 float eps, int interleaved)
{
    LRS_TRY(check_common(nm, N, T));
    LRS_REQUIRE(HQ >= 1 && HK >= 1 && HQ <= 65536 && HK <= 65536,
                "%s: q_heads and k_heads must be 1 to 65536", nm);
    LRS_REQUIRE(dim >= 1 && dim <= kMaxHeadDim, "%s: dim must be 1 to %d (got %lld)", nm, kMaxHeadDim,
                (long long)dim);
    LRS_REQUIRE(rot >= 0 && rot <= dim && rot % 2 == 0,
                "%s: rotary_dim must be even and at most dim (got %lld of %lld)", nm, (long long)rot,
                (long long)dim);
    LRS_REQUIRE(qw && kw, "%s: q_weight and k_weight are required", nm);
    LRS_REQUIRE(rot == 0 || (table && positions), "%s: table and positions are required", nm);
    LRS_REQUIRE(rot == 0 || max_positions >= 1, "%s: max_positions must be at least 1", nm);
    LRS_REQUIRE(max_positions <= (int64_t(1) << 31), "%s: max_positions must be at most 2^31", nm);
    LRS_REQUIRE(eps >= 0.0f && eps - eps == 0.0f, "%s: eps must be finite and >= 0", nm);
    LRS_REQUIRE(interleaved == 0 || interleaved == 1, "%s: interleaved must be 0 or 1", nm);
    LRS_REQUIRE((uintptr_t)table % 4 == 0, "%s: table is not aligned to its elements", nm);
    return LRS_OK;
}

constexpr uint32_t kNormMaxBlocks = 4096;      // forward
constexpr uint32_t kNormMaxBlocksGrad = 1024;  // backward: each leaves a row of sums

inline uint32_t norm_blocks(int64_t rows, uint32_t most)
{
    const int64_t b = (rows + kNormWaves - 1) / kNormWaves;
    return (uint32_t)(b < (int64_t)most ? b : (int64_t)most);
}

inline size_t norm_workspace(int64_t N, int64_t T, int64_t HQ, int64_t HK, int64_t dim)
{
    return ((size_t)norm_blocks(N * T * HQ, kNormMaxBlocksGrad) +
            norm_blocks(N * T * HK, kNormMaxBlocksGrad)) * (size_t)dim * 4;
}

template <class D>
lrs_status norm_rotation_entry(const char* nm, int64_t N, int64_t T, int64_t HQ, int64_t HK,
                               int64_t dim, int64_t rot, const D* q, const D* k, const D* qw,
                               const D* kw, const float* table, int64_t max_positions,
                               const int32_t* positions, float eps, int interleaved, D* q_out,
                               D* k_out, const int64_t* strides, hipStream_t stream)
{
    LRS_TRY(check_rotation(nm, N, T, HQ, HK, dim, rot, qw, kw, table, max_positions, positions, eps,
                           interleaved));
    constexpr int s = sizeof(D);
    const SeqArg args[5] = {{q, HQ, dim, s, false, true, "q"},
                            {k, HK, dim, s, false, true, "k"},
                            {positions, 1, 1, 4, false, rot > 0, "positions"},
                            {q_out, HQ, dim, s, true, true, "q_out"},
                            {k_out, HK, dim, s, true, true, "k_out"}};
    const Span more[] = {{qw, (uint64_t)dim * s}, {kw, (uint64_t)dim * s},
                         {rot ? table : nullptr, (uint64_t)(max_positions * rot) * 4}};
    SeqView v[5];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, more, 0, 3, v));
    NormArgs x{};
    x.side[0] = NormSide{v[0], {}, v[3], qw, nullptr, N * T * HQ, (int32_t)HQ,
                         norm_blocks(N * T * HQ, kNormMaxBlocks)};
    x.side[1] = NormSide{v[1], {}, v[4], kw, nullptr, N * T * HK, (int32_t)HK,
                         norm_blocks(N * T * HK, kNormMaxBlocks)};
    x.positions = v[2];
    x.table = table;
    x.N = N;
    x.T = T;
    x.max_positions = max_positions;
    x.dim = (int32_t)dim;
    x.rot = (int32_t)rot;
    x.eps = eps;
    x.interleaved = interleaved;
    return launch_seq(nm, norm_rotation<D, false>, x.side[0].blocks + x.side[1].blocks,
                      kNormWaves * kWave, stream, x);
}

template <class D>
lrs_status norm_rotation_backward_entry(const char* nm, int64_t N, int64_t T, int64_t HQ, int64_t HK,
                                        int64_t dim, int64_t rot, const D* grad_q_out,
                                        const D* grad_k_out, const D* q, const D* k, const D* qw,
                                        const D* kw, const float* table, int64_t max_positions,
                                        const int32_t* positions, float eps, int interleaved,
                                        D* grad_q, D* grad_k, D* grad_qw, D* grad_kw,
                                        const int64_t* strides, void* ws, size_t ws_bytes,
                                        hipStream_t stream)
{
    LRS_TRY(check_rotation(nm, N, T, HQ, HK, dim, rot, qw, kw, table, max_positions, positions, eps,
                           interleaved));
    LRS_REQUIRE(grad_qw && grad_kw, "%s: grad_q_weight and grad_k_weight are required", nm);
    constexpr int s = sizeof(D);
    const SeqArg args[7] = {{grad_q_out, HQ, dim, s, false, true, "grad_q_out"},
                            {grad_k_out, HK, dim, s, false, true, "grad_k_out"},
                            {q, HQ, dim, s, false, true, "q"},
                            {k, HK, dim, s, false, true, "k"},
                            {positions, 1, 1, 4, false, rot > 0, "positions"},
                            {grad_q, HQ, dim, s, true, true, "grad_q"},
                            {grad_k, HK, dim, s, true, true, "grad_k"}};
    const uint64_t wb = (uint64_t)dim * s;
    const Span more[] = {{grad_qw, wb}, {grad_kw, wb}, {ws, ws_bytes}, {qw, wb}, {kw, wb},
                         {rot ? table : nullptr, (uint64_t)(max_positions * rot) * 4}};
    SeqView v[7];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, more, 3, 6, v));
    LRS_TRY(check_workspace(nm, norm_workspace(N, T, HQ, HK, dim), ws, ws_bytes));
    NormArgs x{};
    const uint32_t bq = norm_blocks(N * T * HQ, kNormMaxBlocksGrad);
    const uint32_t bk = norm_blocks(N * T * HK, kNormMaxBlocksGrad);
    float* const part = static_cast<float*>(ws);
    x.side[0] = NormSide{v[2], v[0], v[5], qw, part, N * T * HQ, (int32_t)HQ, bq};
    x.side[1] = NormSide{v[3], v[1], v[6], kw, part + (size_t)bq * dim, N * T * HK, (int32_t)HK, bk};
    x.positions = v[4];
    x.table = table;
    x.N = N;
    x.T = T;
    x.max_positions = max_positions;
    x.dim = (int32_t)dim;
    x.rot = (int32_t)rot;
    x.eps = eps;
    x.interleaved = interleaved;
    LRS_TRY(launch_seq(nm, norm_rotation<D, true>, (uint64_t)bq + bk, kNormWaves * kWave, stream, x));
    const WeightSumArgs sum{{x.side[0].part, x.side[1].part}, {grad_qw, grad_kw}, {bq, bk}, (int32_t)dim};
    return launch_seq(nm, weight_sum<D>, (uint64_t)(2 * dim), 256, stream, sum);
}

}  // namespace lrs
