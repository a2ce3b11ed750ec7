// policy.hpp -- log probabilities of actions, and the clipped policy loss with a
// KL term, with their gradients.  Per token with logits z, z' = z / temperature,
// action a, lse = log sum_v e^{z'_v}, p_v = e^{z'_v - lse}:
//
//     lp = z'_a - lse,   H = -sum_v p_v log p_v,   r = e^{lp - old}
//     loss = -min(r A, clip(r, 1 - clip, 1 + clip_high) A)
//            + kl_coef (e^{ref - lp} - (ref - lp) - 1) - entropy_coef H
//
// With c the derivative of the result by lp and h that by H,
//
//     dz_v = (c (1[v = a] - p_v) - h p_v (log p_v + H)) / temperature.
//
// One pass over the logits: a row of the vocabulary is held in the registers of
// the lanes that share it (2 or 8 lanes for 18 actions, a block of 1024 for 131072 in
// 16 bits), so that the loss and its gradient read it once; longer rows are read
// again.  Memory is all that it should cost.
#pragma once

#include "sequence.hpp"

namespace lrs {

constexpr int64_t kMaxActions = int64_t(1) << 24;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

enum class PolicyOp { kScore, kLoss, kLossGrad, kScoreBack, kLossBack };

struct PolicyArgs {
    SeqView z, dz;                                     // logits, their gradient
    SeqView action, old_lp, adv, ref, mask, weight;    // per token, nullable but the action
    SeqView loss, lp, entropy, lse;                    // out; entropy and lse in for the backward forms
    SeqView d_lp, d_entropy;                           // of kScoreBack, nullable
    const void* z_end;                                 // behind the last logit
    int64_t T, rows;
    int32_t V, splits;                                 // splits: blocks per row (backward forms)
    float scale, c2, clip, clip_high, kl, ent;         // scale = 1 / temperature, c2 = scale log2 e
    PolicyOp op;
};

template <class E>
__device__ __forceinline__ E token(const SeqView& v, int64_t n, int64_t t)
{
    return *seq_row<E>(v, n, t, 0);
}
__device__ __forceinline__ float token_or(const SeqView& v, int64_t n, int64_t t, float other)
{
    return v.p != nullptr ? token<float>(v, n, t) : other;
}

// ---------------------------------------------------- a row in 16-byte units
// Rows start on any element: a row is taken in the 16-byte units of memory that
// it touches.  What a unit has beyond the row's ends is not used; it is loaded
// all the same where it lies within the array.
template <class D>
constexpr int kUnitElems = 16 / (int)sizeof(D);

template <class D>
struct VocabRow {
    const char* base;  // on 16 bytes
    int first;         // elements of the first unit before the row
    int V, units;

    __device__ __forceinline__ VocabRow(const SeqView& v, int64_t n, int64_t t, int V) : V(V)
    {
        const char* const p = reinterpret_cast<const char*>(seq_row<D>(v, n, t, 0));
        const int off = (int)((uintptr_t)p & 15);
        base = p - off;
        first = off / (int)sizeof(D);
        units = (first + V + kUnitElems<D> - 1) / kUnitElems<D>;
    }
    // The column of a unit's first element.
    __device__ __forceinline__ int column(int u) const { return u * kUnitElems<D> - first; }

    __device__ __forceinline__ u32x4 load(int u, const void* lo, const void* hi) const
    {
        const char* const p = base + (int64_t)u * 16;
        if (p >= (const char*)lo && p + 16 <= (const char*)hi) return *reinterpret_cast<const u32x4*>(p);
        u32x4 w = {};
        const int c0 = column(u);
#pragma unroll
        for (int k = 0; k < kUnitElems<D>; ++k)
            if ((unsigned)(c0 + k) < (unsigned)V) {
                if constexpr (sizeof(D) == 4) w[k] = reinterpret_cast<const uint32_t*>(p)[k];
                else w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[k] << (16 * (k & 1));
            }
        return w;
    }
};

// The logits of a unit; -infinity beyond the row's ends.
template <class D>
__device__ __forceinline__ void widen(const u32x4& w, int c0, int V, float (&z)[kUnitElems<D>])
{
    constexpr int E = kUnitElems<D>;
    if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int k = 0; k < E; ++k) z[k] = __uint_as_float(w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) unpack2<D>(w[k], z[2 * k], z[2 * k + 1]);
    }
    if (c0 < 0 || c0 + E > V) {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if ((unsigned)(c0 + k) >= (unsigned)V) z[k] = -INFINITY;
    }
}

// Makes the compiler widen a unit again where it is used next: kept widened from one
// use to the next, a row would take twice the registers.
__device__ __forceinline__ void keep_packed(u32x4& w)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t v = w[k];
        asm volatile("" : "+v"(v));
        w[k] = v;
    }
}

template <class D>
__device__ __forceinline__ u32x4 narrow(const float (&g)[kUnitElems<D>])
{
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(D) == 4) w[k] = __float_as_uint(g[k]);
        else w[k] = pack2<D>(g[2 * k], g[2 * k + 1]);
    }
    return w;
}

// Columns c0 .. of a row of the gradient; `whole`: its units lie where the logits' do.
template <class D>
__device__ __forceinline__ void store_unit(D* row, int c0, int V, bool whole, const u32x4& w)
{
    constexpr int E = kUnitElems<D>;
    if (whole && c0 >= 0 && c0 + E <= V) {
        *reinterpret_cast<u32x4*>(row + c0) = w;
        return;
    }
#pragma unroll
    for (int k = 0; k < E; ++k)
        if ((unsigned)(c0 + k) < (unsigned)V) {
            if constexpr (sizeof(D) == 4) reinterpret_cast<uint32_t*>(row)[c0 + k] = w[k];
            else reinterpret_cast<uint16_t*>(row)[c0 + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
        }
}

// ------------------------------------------------------------ sums over a row
// Over the L lanes of a row: within a wave by moves, across the waves of a block
// through LDS, in the same order every time.
template <int L, bool kMax>
__device__ __forceinline__ float over_row(float v, float* part)
{
    auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int o = (L < kWave ? L : kWave) / 2; o > 0; o >>= 1) v = join(v, __shfl_xor(v, o));
    if constexpr (L > kWave) {
        __syncthreads();  // `part` may still be read
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < L / kWave; ++w) v = join(v, part[w]);
    }
    return v;
}

// The statistics of a row, in powers of two: x_v = (z_v - most) c2 with c2 = scale
// log2 e, s1 = sum 2^x, s2 = sum 2^x x.  (The difference comes first: z c2 - most c2
// in one fma would save an instruction, but is off by what rounding most c2 left,
// which is everything where all actions are at the type's lowest value.)
struct RowSums {
    float most, s1, s2;

    // A row of -infinity alone has no weights, and becomes NaN by its sums.
    __device__ __forceinline__ explicit RowSums(float top) : most(top == -INFINITY ? 0.0f : top), s1(0.0f), s2(0.0f) {}

    // What is left of 2^x and x in sums is 0 where x is -infinity.
    __device__ __forceinline__ void add(float z, float c2)
    {
        const float x = (z - most) * c2, e = __builtin_amdgcn_exp2f(x);
        s1 += e;
        s2 = fmaf(e, fmaxf(x, -200.0f), s2);
    }
    // The same sums as from a larger logit.
    __device__ __forceinline__ void raise(float top, float c2)
    {
        const float d = (most - top) * c2;
        if (s1 != 0.0f) {
            const float f = __builtin_amdgcn_exp2f(d);
            s2 = f * fmaf(s1, fmaxf(d, -200.0f), s2);
            s1 *= f;
        }
        most = top;
    }
};

// ------------------------------------------------------------------ one token
// What the token's loss is and how its gradient is made: for every logit
// e (a + b x) with e = 2^x, x = (z - from) c2, and `hit` more for the action's.
struct TokenGrad {
    float from, a, b, hit;
};

// Where token `at` stands.  The host makes one row of the tokens (T = rows) where all
// arrays allow it, and 32 bits do where there are as few: a division of 64 bits costs
// a token of a few actions more than all of its logits do.
struct Place {
    int64_t n, t;

    __device__ __forceinline__ Place(const PolicyArgs& x, int64_t at)
    {
        if (x.T == x.rows) {
            n = 0;
            t = at;
        } else if (x.rows <= 0xffffffffll) {
            n = (uint32_t)at / (uint32_t)x.T;
            t = (uint32_t)at - (uint32_t)n * (uint32_t)x.T;
        } else {
            n = at / x.T;
            t = at % x.T;
        }
    }
};

struct Token {
    int64_t n, t;
    int64_t action;
    float z_a;
    float old_lp, adv, ref, weight;

    template <class D>
    __device__ __forceinline__ void load(const PolicyArgs& x, const Place& at)
    {
        n = at.n;
        t = at.t;
        action = token<int64_t>(x.action, n, t);
        const bool in = (uint64_t)action < (uint64_t)x.V;
        // an action that is none makes the token NaN
        z_a = in ? to_f32(seq_row<D>(x.z, n, t, 0)[action]) : __builtin_nanf("");
        old_lp = token_or(x.old_lp, n, t, 0.0f);
        adv = token_or(x.adv, n, t, 0.0f);
        ref = token_or(x.ref, n, t, 0.0f);
        weight = token_or(x.weight, n, t, 1.0f);
    }
    // The loss of a log probability and entropy, and its derivative by the first.
    // The comparisons leave NaN as it is.
    __device__ __forceinline__ float loss(const PolicyArgs& x, float lp, float H, float& slope) const
    {
        const float r = expf(lp - old_lp);
        const float most = 1.0f + x.clip_high, least = 1.0f - x.clip;
        const bool cut = adv >= 0.0f ? r > most : r < least;
        const float bound = cut ? (adv >= 0.0f ? most : least) : r;
        float loss = -bound * adv - x.ent * H;
        slope = cut ? 0.0f : -adv * r;
        if (x.kl != 0.0f) {
            const float d = ref - lp, e = expm1f(d);
            loss += x.kl * (e - d);
            slope -= x.kl * e;
        }
        return loss;
    }
};

// c and h as above, times whatever weighs the token; log2s: log2 of s1, H: the entropy.
__device__ __forceinline__ TokenGrad token_grad(const PolicyArgs& x, float from, float c, float h, float per,
                                                float log2s, float H)
{
    c *= x.scale;
    h *= x.scale;
    TokenGrad g;
    g.from = from;
    g.hit = c;
    g.a = -(c + h * (H - kLn2 * log2s)) * per;
    g.b = -h * kLn2 * per;
    return g;
}

template <class D, bool kEntropy>
__device__ __forceinline__ void grad_unit(const PolicyArgs& x, const u32x4& w, int c0, const TokenGrad& g,
                                          int action, D* row, bool whole)
{
    constexpr int E = kUnitElems<D>;
    float z[E];
    if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int k = 0; k < E; ++k) z[k] = __uint_as_float(w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) unpack2<D>(w[k], z[2 * k], z[2 * k + 1]);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
        const float v = (z[k] - g.from) * x.c2, e = __builtin_amdgcn_exp2f(v);
        z[k] = e * (kEntropy ? fmaf(g.b, fmaxf(v, -200.0f), g.a) : g.a);
    }
    if ((unsigned)(action - c0) < (unsigned)E) {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (action - c0 == k) z[k] += g.hit;
    }
    store_unit<D>(row, c0, x.V, whole, narrow<D>(z));
}

// ------------------------------------------------------------------- kernels

// Blocks lie in rows of kGridRow: a grid's axis holds fewer than 2^32 threads, which
// 2^30 tokens of a few actions exceed.
constexpr uint64_t kGridRow = uint64_t(1) << 20;
__device__ __forceinline__ int64_t grid_block() { return (int64_t)blockIdx.y * kGridRow + blockIdx.x; }

inline lrs_status launch_tokens(const char* nm, void (*kernel)(PolicyArgs), uint64_t blocks, int threads,
                                hipStream_t stream, PolicyArgs x)
{
    const uint64_t rows = (blocks + kGridRow - 1) / kGridRow;
    LRS_REQUIRE(rows <= 65535, "%s: tokens * actions is too large", nm);
    return launch_seq(nm, kernel, dim3((uint32_t)std::min(blocks, kGridRow), (uint32_t)rows), threads, stream, x);
}

__device__ __forceinline__ void put_token(const SeqView& v, const Token& k, float value)
{
    if (v.p != nullptr) *seq_row_out<float>(v, k.n, k.t, 0) = value;
}

// The token's outputs from its sums; returns how its gradient is made.
__device__ __forceinline__ TokenGrad finish(const PolicyArgs& x, const Token& k, const RowSums& s, bool leader)
{
    const float log2s = __builtin_amdgcn_logf(s.s1), per = 1.0f / s.s1;
    const float lp = fmaf(k.z_a - s.most, x.scale, -kLn2 * log2s);
    const float H = kLn2 * (log2s - s.s2 * per);
    float slope = 0.0f, loss = 0.0f;
    if (x.op != PolicyOp::kScore) loss = k.loss(x, lp, H, slope);
    if (leader) {
        put_token(x.loss, k, loss);
        put_token(x.lp, k, lp);
        put_token(x.entropy, k, H);
        put_token(x.lse, k, fmaf(s.most, x.scale, kLn2 * log2s));
    }
    return token_grad(x, s.most, k.weight * slope, -k.weight * x.ent, per, log2s, H);
}

template <class D>
__device__ __forceinline__ void clear_row(D* row, int V, int lane, int lanes)
{
    // by the aligned units of the row itself
    const int first = (int)((uintptr_t)row & 15) / (int)sizeof(D);
    for (int c0 = lane * kUnitElems<D> - first; c0 < V; c0 += lanes * kUnitElems<D>)
        store_unit<D>(row, c0, V, true, u32x4{});
}

// A token that the mask leaves out: zeros for everything.
template <class D, bool kGrad>
__device__ __forceinline__ bool masked_out(const PolicyArgs& x, const Place& at, int lane, int lanes)
{
    if (x.mask.p == nullptr) return false;
    const int64_t n = at.n, t = at.t;
    if (token<uint8_t>(x.mask, n, t) != 0) return false;
    if (lane == 0) {
        Token k;
        k.n = n;
        k.t = t;
        put_token(x.loss, k, 0.0f);
        put_token(x.lp, k, 0.0f);
        put_token(x.entropy, k, 0.0f);
        put_token(x.lse, k, 0.0f);
    }
    if (kGrad) clear_row<D>(seq_row_out<D>(x.dz, n, t, 0), x.V, lane, lanes);
    return true;
}

template <class D>
__device__ __forceinline__ bool same_phase(const D* row, const VocabRow<D>& from)
{
    return (int)((uintptr_t)row & 15) == from.first * (int)sizeof(D);
}

// Rows of at most L U units, held by L lanes: L <= 64, 256 / L rows to a block,
// or a block of L lanes per row.  Bytes bound it: 524288 rows of 18 f32 actions with
// their gradient 21 us (4.4 TB/s); 4096 rows of 131072 bf16 actions 288 to 374, by how many
// of them are masked (not read, zeros written).
template <class D, int L, int U, bool kGrad>
__global__ __launch_bounds__(L > kWave ? L : 256) void policy_rows(const PolicyArgs x)
{
    constexpr int kBlock = L > kWave ? L : 256;
    __shared__ float part[L > kWave ? L / kWave : 1];
    const int lane = threadIdx.x % L;
    const int64_t at = grid_block() * (kBlock / L) + threadIdx.x / L;
    if (at >= x.rows) return;  // whole blocks, or (L <= 64) lanes that nothing waits for
    const Place place(x, at);
    if (masked_out<D, kGrad>(x, place, lane, L)) return;
    Token k;
    k.load<D>(x, place);
    const VocabRow<D> row(x.z, k.n, k.t, x.V);
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (lane + u * L < row.units) w[u] = row.load(lane + u * L, x.z.p, x.z_end);
    float most = -INFINITY;
    constexpr int E = kUnitElems<D>;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (lane + u * L < row.units) {
            float z[E];
            widen<D>(w[u], row.column(lane + u * L), x.V, z);
#pragma unroll
            for (int e = 0; e < E; ++e) most = fmaxf(most, z[e]);
        }
    most = over_row<L, true>(most, part);
    RowSums s(most);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (lane + u * L < row.units) {
            float z[E];
            keep_packed(w[u]);
            widen<D>(w[u], row.column(lane + u * L), x.V, z);
#pragma unroll
            for (int e = 0; e < E; ++e) s.add(z[e], x.c2);
        }
    s.s1 = over_row<L, false>(s.s1, part);
    s.s2 = over_row<L, false>(s.s2, part);
    const TokenGrad g = finish(x, k, s, lane == 0);
    if constexpr (kGrad) {
        D* const out = seq_row_out<D>(x.dz, k.n, k.t, 0);
        const bool whole = same_phase(out, row);
        const int action = (int)k.action;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int unit = lane + u * L, c0 = row.column(unit);
            if (unit < row.units) {
                keep_packed(w[u]);
                if (x.ent != 0.0f) grad_unit<D, true>(x, w[u], c0, g, action, out, whole);
                else grad_unit<D, false>(x, w[u], c0, g, action, out, whole);
            }
        }
    }
}

// Longer rows: a block reads the row once for the sums (each lane with a maximum
// of its own) and once more for the gradient.
constexpr int kStreamLanes = 1024;
template <class D, bool kGrad>
__global__ __launch_bounds__(kStreamLanes) void policy_stream(const PolicyArgs x)
{
    constexpr int L = kStreamLanes, U = 4, E = kUnitElems<D>;
    __shared__ float part[L / kWave];
    const int lane = threadIdx.x;
    const int64_t at = grid_block();
    if (at >= x.rows) return;
    const Place place(x, at);
    if (masked_out<D, kGrad>(x, place, lane, L)) return;
    Token k;
    k.load<D>(x, place);
    const VocabRow<D> row(x.z, k.n, k.t, x.V);
    float most = -INFINITY;
    RowSums s(most);
    for (int u0 = lane; u0 < row.units; u0 += L * U) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u0 + u * L < row.units) w[u] = row.load(u0 + u * L, x.z.p, x.z_end);
        float z[U][E], top = most;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            widen<D>(w[u], u0 + u * L < row.units ? row.column(u0 + u * L) : x.V, x.V, z[u]);
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, z[u][e]);
        }
        if (top > most) {
            s.raise(top, x.c2);
            most = top;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) s.add(z[u][e], x.c2);
    }
    s.raise(RowSums(over_row<L, true>(most, part)).most, x.c2);
    s.s1 = over_row<L, false>(s.s1, part);
    s.s2 = over_row<L, false>(s.s2, part);
    const TokenGrad g = finish(x, k, s, lane == 0);
    if constexpr (kGrad) {
        D* const out = seq_row_out<D>(x.dz, k.n, k.t, 0);
        const bool whole = same_phase(out, row);
        for (int u = lane; u < row.units; u += L) {
            const u32x4 w = row.load(u, x.z.p, x.z_end);
            if (x.ent != 0.0f) grad_unit<D, true>(x, w, row.column(u), g, (int)k.action, out, whole);
            else grad_unit<D, false>(x, w, row.column(u), g, (int)k.action, out, whole);
        }
    }
}

// The gradient from the forward call's lse and entropy: no sums, so rows are split
// over as many blocks as there is use for.  L lanes share a row, or a part of it.  Bytes
// bound it: 2331 rows of 50001 f16 actions take 61 us under a tracer, the forward call 40.
template <class D, int L>
__global__ __launch_bounds__(256) void policy_backward(const PolicyArgs x)
{
    const int lane = threadIdx.x % L;
    const int64_t part = grid_block() * (256 / L) + threadIdx.x / L;
    const int64_t at = x.splits == 1 ? part : part / x.splits;
    const int split = (int)(part - at * x.splits);
    if (at >= x.rows) return;
    const Place place(x, at);
    const int64_t n = place.n, t = place.t;
    D* const out = seq_row_out<D>(x.dz, n, t, 0);
    const bool off = x.mask.p != nullptr && token<uint8_t>(x.mask, n, t) == 0;
    if (off) {
        clear_row<D>(out, x.V, lane + split * L, L * x.splits);
        return;
    }
    Token k;
    k.load<D>(x, place);
    const VocabRow<D> row(x.z, n, t, x.V);
    const float lse = token<float>(x.lse, n, t), H = token_or(x.entropy, n, t, 0.0f);
    // p = e^{z' - lse}: z - lse / scale in float32, and what that leaves of lse as a factor
    float from = lse / x.scale, rest = fmaf(-from, x.scale, lse) * kLog2e;
    if (fabsf(lse) > 512.0f && fabsf(lse) < INFINITY) {
        // so large that float32 keeps little of how the logits share it: summed again
        __shared__ float part_of[L > kWave ? L / kWave : 1];
        float most = -INFINITY;
        for (int u = lane; u < row.units; u += L) {
            float z[kUnitElems<D>];
            widen<D>(row.load(u, x.z.p, x.z_end), row.column(u), x.V, z);
#pragma unroll
            for (int e = 0; e < kUnitElems<D>; ++e) most = fmaxf(most, z[e]);
        }
        RowSums s(over_row<L, true>(most, part_of));
        for (int u = lane; u < row.units; u += L) {
            float z[kUnitElems<D>];
            widen<D>(row.load(u, x.z.p, x.z_end), row.column(u), x.V, z);
#pragma unroll
            for (int e = 0; e < kUnitElems<D>; ++e) s.add(z[e], x.c2);
        }
        from = s.most;
        rest = __builtin_amdgcn_logf(over_row<L, false>(s.s1, part_of));
    }
    const float lp = fmaf(k.z_a - from, x.scale, -kLn2 * rest);
    float c, h;
    if (x.op == PolicyOp::kScoreBack) {
        c = token_or(x.d_lp, n, t, 0.0f);
        h = token_or(x.d_entropy, n, t, 0.0f);
        if ((uint64_t)k.action >= (uint64_t)x.V) c = __builtin_nanf("");
    } else {
        k.loss(x, lp, H, c);
        c *= k.weight;
        h = -k.weight * x.ent;
    }
    const TokenGrad g = token_grad(x, from, c, h, __builtin_amdgcn_exp2f(-rest), rest, H);
    const bool whole = same_phase(out, row);
    const int action = (int)k.action, step = L * x.splits;
    constexpr int U = 4;
    for (int u0 = lane + split * L; u0 < row.units; u0 += step * U) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u0 + u * step < row.units) w[u] = row.load(u0 + u * step, x.z.p, x.z_end);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u0 + u * step < row.units) {
                const int c0 = row.column(u0 + u * step);
                if (h != 0.0f) grad_unit<D, true>(x, w[u], c0, g, action, out, whole);
                else grad_unit<D, false>(x, w[u], c0, g, action, out, whole);
            }
    }
}

// ------------------------------------------------------------------ entries

// The most 16-byte units that a row of the logits touches.
template <class D>
inline int64_t row_units(const SeqView& z, int64_t V)
{
    constexpr int E = kUnitElems<D>;
    return rows_on(z, E, sizeof(D)) ? (V + E - 1) / E : (V + 2 * E - 2) / E;
}

// One row of all tokens, where their places in every array are evenly spaced.
inline void join_rows(PolicyArgs& x)
{
    if (x.T == x.rows) return;
    const SeqView* const all[] = {&x.z, &x.dz, &x.action, &x.old_lp, &x.adv, &x.ref, &x.mask, &x.weight,
                                  &x.loss, &x.lp, &x.entropy, &x.lse, &x.d_lp, &x.d_entropy};
    for (const SeqView* v : all)
        if (v->p != nullptr && v->env != x.T * v->step) return;
    x.T = x.rows;
}

// Short rows of many tokens take few lanes with more units each, so that a wave has more
// tokens and their divisions, logarithms and sums over lanes count less.  Few tokens take
// a lane to a unit, which ends sooner.  us of the loss and its gradient in f32, with lanes
// for units and with few, 524288 tokens: 4 actions 19.6 and 8.5, 18 actions 38 and 23, 30
// actions 65 and 33, 60 actions 76 and 61, 120 actions 106 and 109; 8192 tokens: 18 actions
// 3.7 and 4.7, 60 actions 4.0 and 4.9.
constexpr int64_t kManyTokens = 65536;

template <class D, bool kGrad>
lrs_status launch_policy(const char* nm, PolicyArgs x, hipStream_t stream)
{
    join_rows(x);
    const int64_t units = row_units<D>(x.z, x.V);
    void (*kernel)(PolicyArgs) = policy_stream<D, kGrad>;
    int lanes = kStreamLanes;
    const bool many = x.rows >= kManyTokens;
#define LRS_POLICY(most, l, u, when)           \
    if (units <= most && when) {               \
        kernel = policy_rows<D, l, u, kGrad>;  \
        lanes = l;                             \
    } else
    LRS_POLICY(4, 1, 4, many)
    LRS_POLICY(8, 2, 4, many)
    LRS_POLICY(16, 4, 4, many)
    LRS_POLICY(4, 4, 1, true)
    LRS_POLICY(8, 8, 1, true)
    LRS_POLICY(16, 16, 1, true)
    LRS_POLICY(32, 16, 2, true)
    LRS_POLICY(64, 16, 4, true)
    LRS_POLICY(128, 32, 4, true)
    LRS_POLICY(256, 64, 4, true)
    LRS_POLICY(1024, 256, 4, true)
    LRS_POLICY(2048, 256, 8, true)
    LRS_POLICY(4096, 256, 16, true)
    LRS_POLICY(8192, 512, 16, true)
    LRS_POLICY(16384, 1024, 16, true) {}
#undef LRS_POLICY
    const int block = lanes > kWave ? lanes : 256;
    const int64_t per = block / lanes;
    return launch_tokens(nm, kernel, (uint64_t)((x.rows + per - 1) / per), block, stream, x);
}

template <class D>
lrs_status launch_policy_backward(const char* nm, PolicyArgs x, hipStream_t stream)
{
    join_rows(x);
    const int64_t units = row_units<D>(x.z, x.V);
    void (*kernel)(PolicyArgs) = policy_backward<D, 256>;
    int lanes = 256;
    // many tokens: as in launch_policy (loss and then gradient, as above: 18 actions 48 and 36, 30
    // actions 81 and 47, 60 actions 87 and 73)
    if (units <= 8 && x.rows >= kManyTokens) { kernel = policy_backward<D, 2>; lanes = 2; }
    else if (units <= 8) { kernel = policy_backward<D, 8>; lanes = 8; }
    else if (units <= 16 && x.rows >= kManyTokens) { kernel = policy_backward<D, 4>; lanes = 4; }
    else if (units <= 32) { kernel = policy_backward<D, 16>; lanes = 16; }
    else if (units <= 512) { kernel = policy_backward<D, 64>; lanes = 64; }
    // four units to a lane
    x.splits = lanes < 256 ? 1 : (int32_t)((units + 1023) / 1024);
    const int64_t per = 256 / lanes;
    return launch_tokens(nm, kernel, (uint64_t)((x.rows * x.splits + per - 1) / per), 256, stream, x);
}

// What the calls share: sizes and coefficients checked, and put where the kernels read them.
inline lrs_status check_policy(const char* nm, int64_t N, int64_t T, int64_t V, float temperature,
                               PolicyArgs& x)
{
    LRS_TRY(check_common(nm, N, T));
    LRS_REQUIRE(V >= 1 && V <= kMaxActions, "%s: num_actions must be 1 to %lld (got %lld)", nm,
                (long long)kMaxActions, (long long)V);
    const double c2 = 1.4426950408889634 / (double)temperature;
    LRS_REQUIRE(temperature > 0.0f && temperature <= 3e38f && c2 <= 3e38 && c2 >= 1e-30,
                "%s: temperature must be > 0 and finite, and so must its inverse", nm);
    x.T = T;
    x.rows = N * T;
    x.V = (int32_t)V;
    x.c2 = (float)c2;
    x.scale = (float)(1.0 / (double)temperature);
    return LRS_OK;
}

inline lrs_status check_policy_loss(const char* nm, float clip, float clip_high, float kl, float ent,
                                    const void* ref, PolicyArgs& x)
{
    auto finite = [](float v) { return v - v == 0.0f; };
    LRS_REQUIRE(finite(clip) && clip >= 0.0f && finite(clip_high) && clip_high >= 0.0f,
                "%s: clip and clip_high must be finite and >= 0", nm);
    LRS_REQUIRE(finite(kl) && finite(ent), "%s: kl_coef and entropy_coef must be finite", nm);
    LRS_REQUIRE(kl == 0.0f || ref != nullptr, "%s: ref_log_probs is required with kl_coef", nm);
    x.clip = clip;
    x.clip_high = clip_high;
    x.kl = kl;
    x.ent = ent;
    return LRS_OK;
}

template <class D>
inline void set_logits(PolicyArgs& x, const SeqView& z, int64_t N)
{
    x.z = z;
    x.z_end = static_cast<const D*>(z.p) + (N - 1) * z.env + (x.T - 1) * z.step + x.V;
}

template <class D>
lrs_status action_log_probs_entry(const char* nm, int64_t N, int64_t T, int64_t V, const D* logits,
                                  const int64_t* actions, const uint8_t* mask, float temperature,
                                  float* log_probs, float* entropy, float* lse, const int64_t* strides,
                                  hipStream_t stream)
{
    PolicyArgs x{};
    LRS_TRY(check_policy(nm, N, T, V, temperature, x));
    const SeqArg args[6] = {{logits, 1, V, sizeof(D), false, true, "logits"},
                            {actions, 1, 1, 8, false, true, "actions"},
                            {mask, 1, 1, 1, false, false, "mask"},
                            {log_probs, 1, 1, 4, true, true, "log_probs"},
                            {entropy, 1, 1, 4, true, true, "entropy"},
                            {lse, 1, 1, 4, true, true, "lse"}};
    SeqView v[6];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, nullptr, 0, 0, v));
    set_logits<D>(x, v[0], N);
    x.action = v[1];
    x.mask = v[2];
    x.lp = v[3];
    x.entropy = v[4];
    x.lse = v[5];
    x.op = PolicyOp::kScore;
    return launch_policy<D, false>(nm, x, stream);
}

template <class D>
lrs_status action_log_probs_backward_entry(const char* nm, int64_t N, int64_t T, int64_t V,
                                           const float* grad_log_probs, const float* grad_entropy,
                                           const D* logits, const int64_t* actions, const uint8_t* mask,
                                           float temperature, const float* entropy, const float* lse,
                                           D* grad_logits, const int64_t* strides, hipStream_t stream)
{
    PolicyArgs x{};
    LRS_TRY(check_policy(nm, N, T, V, temperature, x));
    const SeqArg args[8] = {{grad_log_probs, 1, 1, 4, false, false, "grad_log_probs"},
                            {grad_entropy, 1, 1, 4, false, false, "grad_entropy"},
                            {logits, 1, V, sizeof(D), false, true, "logits"},
                            {actions, 1, 1, 8, false, true, "actions"},
                            {mask, 1, 1, 1, false, false, "mask"},
                            {entropy, 1, 1, 4, false, true, "entropy"},
                            {lse, 1, 1, 4, false, true, "lse"},
                            {grad_logits, 1, V, sizeof(D), true, true, "grad_logits"}};
    SeqView v[8];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, nullptr, 0, 0, v));
    x.d_lp = v[0];
    x.d_entropy = v[1];
    set_logits<D>(x, v[2], N);
    x.action = v[3];
    x.mask = v[4];
    x.entropy = v[5];
    x.lse = v[6];
    x.dz = v[7];
    x.op = PolicyOp::kScoreBack;
    return launch_policy_backward<D>(nm, x, stream);
}

template <class D>
lrs_status policy_loss_entry(const char* nm, int64_t N, int64_t T, int64_t V, const D* logits,
                             const int64_t* actions, const float* old_log_probs, const float* advantages,
                             const float* ref_log_probs, const uint8_t* mask, float clip, float clip_high,
                             float kl_coef, float entropy_coef, float temperature, float* loss,
                             float* log_probs, float* entropy, float* lse, const int64_t* strides,
                             hipStream_t stream)
{
    PolicyArgs x{};
    LRS_TRY(check_policy(nm, N, T, V, temperature, x));
    LRS_TRY(check_policy_loss(nm, clip, clip_high, kl_coef, entropy_coef, ref_log_probs, x));
    const SeqArg args[10] = {{logits, 1, V, sizeof(D), false, true, "logits"},
                             {actions, 1, 1, 8, false, true, "actions"},
                             {old_log_probs, 1, 1, 4, false, true, "old_log_probs"},
                             {advantages, 1, 1, 4, false, true, "advantages"},
                             {ref_log_probs, 1, 1, 4, false, false, "ref_log_probs"},
                             {mask, 1, 1, 1, false, false, "mask"},
                             {loss, 1, 1, 4, true, true, "loss"},
                             {log_probs, 1, 1, 4, true, true, "log_probs"},
                             {entropy, 1, 1, 4, true, true, "entropy"},
                             {lse, 1, 1, 4, true, true, "lse"}};
    SeqView v[10];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, nullptr, 0, 0, v));
    set_logits<D>(x, v[0], N);
    x.action = v[1];
    x.old_lp = v[2];
    x.adv = v[3];
    x.ref = v[4];
    x.mask = v[5];
    x.loss = v[6];
    x.lp = v[7];
    x.entropy = v[8];
    x.lse = v[9];
    x.op = PolicyOp::kLoss;
    return launch_policy<D, false>(nm, x, stream);
}

template <class D>
lrs_status policy_loss_backward_entry(const char* nm, int64_t N, int64_t T, int64_t V,
                                      const float* grad_loss, const D* logits, const int64_t* actions,
                                      const float* old_log_probs, const float* advantages,
                                      const float* ref_log_probs, const uint8_t* mask, float clip,
                                      float clip_high, float kl_coef, float entropy_coef,
                                      float temperature, const float* entropy, const float* lse,
                                      D* grad_logits, const int64_t* strides, hipStream_t stream)
{
    PolicyArgs x{};
    LRS_TRY(check_policy(nm, N, T, V, temperature, x));
    LRS_TRY(check_policy_loss(nm, clip, clip_high, kl_coef, entropy_coef, ref_log_probs, x));
    const SeqArg args[10] = {{grad_loss, 1, 1, 4, false, true, "grad_loss"},
                             {logits, 1, V, sizeof(D), false, true, "logits"},
                             {actions, 1, 1, 8, false, true, "actions"},
                             {old_log_probs, 1, 1, 4, false, true, "old_log_probs"},
                             {advantages, 1, 1, 4, false, true, "advantages"},
                             {ref_log_probs, 1, 1, 4, false, false, "ref_log_probs"},
                             {mask, 1, 1, 1, false, false, "mask"},
                             {entropy, 1, 1, 4, false, true, "entropy"},
                             {lse, 1, 1, 4, false, true, "lse"},
                             {grad_logits, 1, V, sizeof(D), true, true, "grad_logits"}};
    SeqView v[10];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, nullptr, 0, 0, v));
    x.weight = v[0];
    set_logits<D>(x, v[1], N);
    x.action = v[2];
    x.old_lp = v[3];
    x.adv = v[4];
    x.ref = v[5];
    x.mask = v[6];
    x.entropy = v[7];
    x.lse = v[8];
    x.dz = v[9];
    x.op = PolicyOp::kLossBack;
    return launch_policy_backward<D>(nm, x, stream);
}

template <class D>
lrs_status policy_loss_and_gradient_entry(const char* nm, int64_t N, int64_t T, int64_t V,
                                          const D* logits, const int64_t* actions,
                                          const float* old_log_probs, const float* advantages,
                                          const float* ref_log_probs, const uint8_t* mask,
                                          const float* weights, float clip, float clip_high,
                                          float kl_coef, float entropy_coef, float temperature,
                                          float* loss, float* log_probs, float* entropy, D* grad_logits,
                                          const int64_t* strides, hipStream_t stream)
{
    PolicyArgs x{};
    LRS_TRY(check_policy(nm, N, T, V, temperature, x));
    LRS_TRY(check_policy_loss(nm, clip, clip_high, kl_coef, entropy_coef, ref_log_probs, x));
    const SeqArg args[11] = {{logits, 1, V, sizeof(D), false, true, "logits"},
                             {actions, 1, 1, 8, false, true, "actions"},
                             {old_log_probs, 1, 1, 4, false, true, "old_log_probs"},
                             {advantages, 1, 1, 4, false, true, "advantages"},
                             {ref_log_probs, 1, 1, 4, false, false, "ref_log_probs"},
                             {mask, 1, 1, 1, false, false, "mask"},
                             {weights, 1, 1, 4, false, false, "weights"},
                             {loss, 1, 1, 4, true, true, "loss"},
                             {log_probs, 1, 1, 4, true, true, "log_probs"},
                             {entropy, 1, 1, 4, true, true, "entropy"},
                             {grad_logits, 1, V, sizeof(D), true, true, "grad_logits"}};
    SeqView v[11];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, nullptr, 0, 0, v));
    set_logits<D>(x, v[0], N);
    x.action = v[1];
    x.old_lp = v[2];
    x.adv = v[3];
    x.ref = v[4];
    x.mask = v[5];
    x.weight = v[6];
    x.loss = v[7];
    x.lp = v[8];
    x.entropy = v[9];
    x.dz = v[10];
    x.op = PolicyOp::kLossGrad;
    return launch_policy<D, true>(nm, x, stream);
}

}  // namespace lrs
