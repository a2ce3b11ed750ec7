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

// For rows that are not on 16 bytes, or pairs that do not lie in whole 16-byte
// units (halves of rotary_dim that are not a multiple of a unit: 24 of 96 in 16-bit
// types): one wave per row, an element per lane and access; the pairs meet in LDS.
// 32768 tokens of 32 + 8 heads of 96 in bf16, 24 of them rotated: 503 MB in 596 us
// (0.8 TB/s), bound by the loads' width.
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

// The same for rows on 16 bytes, by lanes that hold one 16-byte unit of V
// elements each: G lanes (a power of two) span a row, so a wave holds 64 / G
// rows.  They are heads of one token where it has that many, else of a few
// consecutive tokens; a lane keeps its columns' weights, and its token's angles
// for all the heads that it walks over, in registers.  Each wave walks over
// consecutive tokens of its own.  With kNormAhead rows in flight per lane the
// loads are what bounds it: 32768 tokens of 32 + 8 heads of 128 in bf16, 688 MB
// in 163 us (4.2 TB/s, 80% of a large copy's rate; by one wave per row 699 us);
// the gradients of 8 x 2048 tokens of 16 + 16 heads, 403 MB, in 95 us.  Rows
// that leave lanes without a unit lose by that: 72 floats take 18 of 32 lanes,
// 37 x 513 tokens of 7 + 3 heads 39 us and their gradients 50 (2.8 and 3.2 TB/s).
template <class D>
constexpr int kUnit = 16 / sizeof(D);
constexpr int kNormAhead = 4;

template <class D>
__device__ __forceinline__ void unpack(const u32x4& w, float (&v)[kUnit<D>])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(D) == 4) v[k] = __uint_as_float(w[k]);
        else unpack2<D>(w[k], v[2 * k], v[2 * k + 1]);
    }
}
template <class D>
__device__ __forceinline__ u32x4 pack(const float (&v)[kUnit<D>])
{
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(D) == 4) w[k] = __float_as_uint(v[k]);
        else w[k] = pack2<D>(v[2 * k], v[2 * k + 1]);
    }
    return w;
}

template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, kCtrl, 0xf, 0xf, true));
}

// The sum over the G lanes of a row, in each of them.
template <int G>
__device__ __forceinline__ float row_sum(float v)
{
    if constexpr (G >= 2) v = dpp_add<0xb1>(v);    // quad_perm 1 0 3 2
    if constexpr (G >= 4) v = dpp_add<0x4e>(v);    // quad_perm 2 3 0 1
    if constexpr (G >= 8) v = dpp_add<0x141>(v);   // row_half_mirror
    if constexpr (G >= 16) v = dpp_add<0x140>(v);  // row_mirror
    if constexpr (G >= 32) v += __shfl_xor(v, 16);
    if constexpr (G >= 64) v += __shfl_xor(v, 32);
    return v;
}

template <class D, int G, bool kPairs, bool kBackward>
__global__ __launch_bounds__(kNormWaves * kWave) void norm_rotation_wide(const NormArgs x)
{
    constexpr int V = kUnit<D>, kRows = kWave / G;
    __shared__ float sums[kBackward ? kNormWaves : 1][kBackward ? G * V : 1];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const bool keys = blockIdx.x >= x.side[0].blocks;
    const NormSide& s = x.side[keys ? 1 : 0];
    const uint32_t block = keys ? blockIdx.x - x.side[0].blocks : blockIdx.x;
    const int c = (lane & (G - 1)) * V, half = x.rot / 2;
    const bool in_dim = c < x.dim, turned = c < x.rot;
    // heads side by side, then tokens
    int across = 1;
    while (across < kRows && across < s.heads) across <<= 1;
    const int tokens = kRows / across, sub = lane / G / across, h0 = lane / G % across;
    const int64_t waves = (int64_t)s.blocks * kNormWaves, all = x.N * x.T;
    const int64_t per = ((all + waves - 1) / waves + tokens - 1) / tokens * tokens;
    const int64_t begin = (block * (int64_t)kNormWaves + wave) * per;
    const int64_t end = begin + per < all ? begin + per : all;

    float w[V], dw[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        w[e] = in_dim ? to_f32(static_cast<const D*>(s.w)[c + e]) : 0.0f;
        dw[e] = 0.0f;
    }
    const float share = 1.0f / (float)x.dim;
    const int mate = kPairs ? lane : lane + (c < half ? half : -half) / V;

    int64_t n = (begin + sub) / x.T, t = (begin + sub) % x.T;
    for (int64_t tok = begin + sub; tok - sub < end; tok += tokens) {
        const bool live = tok < end && in_dim;
        float cos[V], sin[V];  // of a lane's elements, the sign of its part in the sine
        bool known = true;
        if (x.rot > 0) {
            const int64_t p = live ? *seq_row<int32_t>(x.positions, n, t, 0) : 0;
            known = p >= 0 && p < x.max_positions;
            const float* const angle = x.table + (known ? p : 0) * x.rot;
            const int j = turned ? (kPairs ? c / 2 : (c < half ? c : c - half)) : 0;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int k = kPairs ? j + e / 2 : j + e;
                cos[e] = turned ? angle[k] : 1.0f;
                const float si = turned ? angle[half + k] : 0.0f;
                const bool first = kPairs ? e % 2 == 0 : c < half;
                sin[e] = first != kBackward ? -si : si;
            }
        }
        const D* const xs = seq_row<D>(s.x, n, t, 0);
        const D* const gs = kBackward ? seq_row<D>(s.dy, n, t, 0) : nullptr;
        D* const ys = seq_row_out<D>(s.y, n, t, 0);
        for (int h = h0; h - h0 < s.heads; h += across * kNormAhead) {
            u32x4 raw[kNormAhead], grad[kNormAhead];
#pragma unroll
            for (int a = 0; a < kNormAhead; ++a) {
                raw[a] = grad[a] = u32x4{};
                if (live && h + a * across < s.heads) {
                    raw[a] = *reinterpret_cast<const u32x4*>(xs + (h + a * across) * s.x.head + c);
                    if (kBackward) grad[a] = *reinterpret_cast<const u32x4*>(gs + (h + a * across) * s.dy.head + c);
                }
            }
#pragma unroll
            for (int a = 0; a < kNormAhead; ++a) {
                if (h - h0 + a * across >= s.heads) break;  // (the wave's)
                float v[V], u[V], sum = 0.0f;
                unpack<D>(raw[a], v);
#pragma unroll
                for (int e = 0; e < V; ++e) sum = fmaf(v[e], v[e], sum);
                const float scale = rsqrtf(row_sum<G>(sum) * share + x.eps);
                if constexpr (kBackward) unpack<D>(grad[a], u);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[e] *= scale;
                    if constexpr (!kBackward) u[e] = v[e] * w[e];
                }
                if (x.rot > 0) {
                    float z[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) z[e] = kPairs ? u[e ^ 1] : __shfl(u[e], mate);
#pragma unroll
                    for (int e = 0; e < V; ++e) u[e] = turned ? fmaf(u[e], cos[e], sin[e] * z[e]) : u[e];
                }
                if (!known) {
#pragma unroll
                    for (int e = 0; e < V; ++e) u[e] = __builtin_nanf("");
                }
                if constexpr (kBackward) {
                    float dot = 0.0f;
                    const bool mine = live && h + a * across < s.heads;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if (mine) dw[e] = fmaf(u[e], v[e], dw[e]);
                        u[e] *= w[e];
                        dot = fmaf(u[e], v[e], dot);
                    }
                    dot = row_sum<G>(dot) * share;
#pragma unroll
                    for (int e = 0; e < V; ++e) u[e] = scale * (u[e] - v[e] * dot);
                }
                if (live && h + a * across < s.heads)
                    *reinterpret_cast<u32x4*>(ys + (h + a * across) * s.y.head + c) = pack<D>(u);
            }
        }
        t += tokens;
        while (t >= x.T) {
            t -= x.T;
            ++n;
        }
    }
    if constexpr (kBackward) {
        // over the rows of a wave, then the waves of the block
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int o = G; o < kWave; o <<= 1) dw[e] += __shfl_xor(dw[e], o);
            if (lane < G) sums[wave][c + e] = dw[e];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < x.dim; e += kNormWaves * kWave) {
            float sum = 0.0f;
            for (int k = 0; k < kNormWaves; ++k) sum += sums[k][e];
            s.part[(int64_t)block * x.dim + e] = sum;
        }
    }
}

// dw from the blocks' sums, in a fixed order: one block per element of dim, 4.9
// us for 1024 sums of 128 (a launch and one chain of loads).
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

// The kernel: 16-byte units where the rows allow them (and rotated pairs lie in
// whole units), with as many lanes to a row as it has units.
template <class D, bool kBackward>
lrs_status launch_norm(const char* nm, const NormArgs& x, hipStream_t stream)
{
    constexpr int V = kUnit<D>, s = sizeof(D);
    bool wide = x.dim % V == 0 && (x.interleaved ? x.rot % V == 0 : x.rot % (2 * V) == 0);
    for (const NormSide& side : x.side)
        wide = wide && rows_on(side.x, V, s) && rows_on(side.y, V, s) &&
               (!kBackward || rows_on(side.dy, V, s));
    void (*kernel)(NormArgs) = norm_rotation<D, kBackward>;
    if (wide) {
#define LRS_NORM(G) \
    (x.interleaved ? norm_rotation_wide<D, G, true, kBackward> : norm_rotation_wide<D, G, false, kBackward>)
        const int units = x.dim / V;
        if (units <= 4) kernel = LRS_NORM(4);
        else if (units <= 8) kernel = LRS_NORM(8);
        else if (units <= 16) kernel = LRS_NORM(16);
        else if (units <= 32) kernel = LRS_NORM(32);
        else if constexpr (s == 4) kernel = LRS_NORM(64);
#undef LRS_NORM
    }
    return launch_seq(nm, kernel, (uint64_t)x.side[0].blocks + x.side[1].blocks, kNormWaves * kWave, stream, x);
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
    return launch_norm<D, false>(nm, x, stream);
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
    LRS_TRY((launch_norm<D, true>(nm, x, stream)));
    const WeightSumArgs sum{{x.side[0].part, x.side[1].part}, {grad_qw, grad_kw}, {bq, bk}, (int32_t)dim};
    return launch_seq(nm, weight_sum<D>, (uint64_t)(2 * dim), 256, stream, sum);
}

}  // namespace lrs
