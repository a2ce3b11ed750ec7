// recurrence.hpp -- the gated recurrence with a matrix state.  Per environment
// and head, with a state S of [key_dim, value_dim] in fp32:
//
//     S_t = (cut_t ? 0 : e^{g_t} S_{t-1}) + k_t v_t^T,    o_t = scale S_t^T q_t
//
// cut_t where the reset mask is set or g_t is -infinity.  With
// D(i, j) = e^{g_{j+1} + ... + g_i} (0 where a step in j+1..i is cut), every
// direction is one pass of the same form,
//
//     y_i = sum_j D(i, j) (a_i . b_j) c_j                   over j <= i, or
//     y_i = sum_j D(j, i) (a_i . b_j) c_j                   over j >= i:
//
//     o:  a = q,  b = k,  c = v,   in time
//     dq: a = do, b = v,  c = k,   in time
//     dk: a = v,  b = do, c = q,   against time
//     dv: a = k,  b = q,  c = do,  against time
//
// and each pass carries the state sum_j D b_j c_j^T: S (transposed for dq), or
// the gradient of S from the later steps (transposed for dk).  The gradient of
// g_t is everything carried over from step t-1 to t, that is
//
//     dg_t = sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <S_T, dS_T>,
//
// since q_s . dq_s sums the products of s with all steps up to it and
// k_s . dk_s with all steps from it on; what lies wholly behind t cancels.
#pragma once

#include "sequence.hpp"

namespace lrs {

constexpr int kMaxDim = 128;  // largest key and value dimension

// One pass over the sequence.  init: the state before the first step in scan
// order; last: where the state after the last one goes; both [N, H, key_dim,
// value_dim] and nullable.  y_scale multiplies y, u_scale what enters the
// state.  dot (nullable): receives y_i . d_i per [N, H, T]; cross (nullable):
// <final state, meet> per [N, H].
struct PassArgs {
    SeqView a, b, c, d, y;
    const float* init;
    float* last;
    const float* meet;
    float* dot;
    float* cross;
    float y_scale, u_scale;
    int32_t da, dc;  // dims of a and b, of c and y
    uint8_t reverse, transposed, y_f32;
};

struct RecurrenceArgs {
    SeqView g, reset;
    int64_t N, T;
    int32_t H, passes;
    PassArgs pass[3];
};

// Row r (of a's dim) and column c (of y's dim) of a state in memory.
__device__ __forceinline__ int64_t state_at(const PassArgs& p, int r, int c)
{
    return p.transposed ? (int64_t)c * p.da + r : (int64_t)r * p.dc + c;
}

// The step's decay factor, 0 where it is cut.
template <class D>
__device__ __forceinline__ float decay_of(const RecurrenceArgs& x, int64_t n, int64_t t, int h)
{
    const float g = to_f32(*seq_row<D>(x.g, n, t, h));
    const bool reset = x.reset.p != nullptr && *seq_row<uint8_t>(x.reset, n, t, 0) != 0;
    return reset ? 0.0f : __expf(g);
}

// One block walks one head's sequence step by step; a thread holds one column
// of the state.
constexpr int kStage = 16;  // steps staged in LDS at a time

template <class D, int DA>
__global__ __launch_bounds__(kMaxDim) void recurrence_steps(const RecurrenceArgs x)
{
    __shared__ float sa[kStage][DA], sb[kStage][DA], sf[kStage];
    __shared__ float part[kMaxDim / kWave];
    const int pass = blockIdx.x % x.passes;
    const int64_t head = blockIdx.x / x.passes;
    const PassArgs& p = x.pass[pass];
    const int64_t n = head / x.H;
    const int h = (int)(head % x.H);
    const int col = threadIdx.x;
    const bool active = col < p.dc;
    const int64_t at = head * p.da * p.dc;
    float S[DA];
#pragma unroll
    for (int r = 0; r < DA; ++r)
        S[r] = p.init && active && r < p.da ? p.init[at + state_at(p, r, col)] : 0.0f;
    for (int64_t done = 0; done < x.T; done += kStage) {
        const int m = (int)(x.T - done < kStage ? x.T - done : kStage);
        __syncthreads();
        for (int e = col; e < kStage * DA; e += blockDim.x) {
            const int s = e / DA, r = e % DA;
            const int64_t t = p.reverse ? x.T - 1 - (done + s) : done + s;
            const bool in = s < m && r < p.da;
            sa[s][r] = in ? to_f32(seq_row<D>(p.a, n, t, h)[r]) : 0.0f;
            sb[s][r] = in ? to_f32(seq_row<D>(p.b, n, t, h)[r]) : 0.0f;
        }
        if (col < m) sf[col] = decay_of<D>(x, n, p.reverse ? x.T - 1 - (done + col) : done + col, h);
        __syncthreads();
        for (int s = 0; s < m; ++s) {
            const int64_t t = p.reverse ? x.T - 1 - (done + s) : done + s;
            const float c = active ? to_f32(seq_row<D>(p.c, n, t, h)[col]) * p.u_scale : 0.0f;
            // against time, the decay of a step applies to what it passes on
            const float f = p.reverse ? 1.0f : sf[s];
            float y = 0.0f;
#pragma unroll
            for (int r = 0; r < DA; ++r) {
                const float before = f == 0.0f ? 0.0f : S[r] * f;
                S[r] = fmaf(sb[s][r], c, before);
                y = fmaf(sa[s][r], S[r], y);
            }
            y *= p.y_scale;
            if (p.reverse)
#pragma unroll
                for (int r = 0; r < DA; ++r) S[r] = sf[s] == 0.0f ? 0.0f : S[r] * sf[s];
            if (active) {
                if (p.y_f32) seq_row_out<float>(p.y, n, t, h)[col] = y;
                else seq_row_out<D>(p.y, n, t, h)[col] = from_f32<D>(y);
            }
            if (p.dot) {
                float v = active ? y * to_f32(seq_row<D>(p.d, n, t, h)[col]) : 0.0f;
                for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
                if (col % kWave == 0) part[col / kWave] = v;
                __syncthreads();
                if (col == 0) {
                    float sum = part[0];
                    for (int w = 1; w < (int)blockDim.x / kWave; ++w) sum += part[w];
                    p.dot[head * x.T + t] = sum;
                }
                __syncthreads();
            }
        }
    }
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < DA; ++r) {
        if (!active || r >= p.da) continue;
        if (p.last) p.last[at + state_at(p, r, col)] = S[r];
        if (p.cross && p.meet) v = fmaf(S[r], p.meet[at + state_at(p, r, col)], v);
    }
    if (p.cross) {
        for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
        __syncthreads();
        if (col % kWave == 0) part[col / kWave] = v;
        __syncthreads();
        if (col == 0) {
            float sum = part[0];
            for (int w = 1; w < (int)blockDim.x / kWave; ++w) sum += part[w];
            p.cross[head] = sum;
        }
    }
}

// dg of one head by one wave, 64 steps at a time from the end: a suffix sum of
// q.dq - k.dk in 64 bits (its terms cancel), started again at each cut, where
// nothing is carried over and dg is 0.
struct DecayGradArgs {
    SeqView g, reset, dg;
    const float *qdq, *kdk, *cross;
    int64_t N, T;
    int32_t H;
};

template <class D>
__global__ __launch_bounds__(64) void decay_grad(const DecayGradArgs x)
{
    const int64_t head = blockIdx.x, n = head / x.H;
    const int h = (int)(head % x.H), lane = threadIdx.x;
    double carry = x.cross[head];
    for (int64_t end = x.T; end > 0; end -= kWave) {
        const int64_t t = end - 1 - lane;
        double v = 0.0;
        bool cut = false;
        if (t >= 0) {
            v = (double)x.qdq[head * x.T + t] - (double)x.kdk[head * x.T + t];
            const float g = to_f32(*seq_row<D>(x.g, n, t, h));
            cut = __expf(g) == 0.0f || (x.reset.p && *seq_row<uint8_t>(x.reset, n, t, 0) != 0);
        }
        // sums over the lanes up to this one, from the last cut below it on
        bool stop = __shfl_up((int)cut, 1) != 0 && lane > 0;
        for (int o = 1; o < kWave; o <<= 1) {
            const double w = __shfl_up(v, o);
            const bool s = __shfl_up((int)stop, o) != 0;
            if (lane >= o) {
                if (!stop) v += w;
                stop = stop || s;
            }
        }
        if (!stop) v += carry;
        if (t >= 0) *seq_row_out<D>(x.dg, n, t, h) = from_f32<D>(cut ? 0.0f : (float)v);
        carry = __shfl(v, kWave - 1);
        if (__shfl((int)cut, kWave - 1)) carry = 0.0;
    }
}

// Sums the value heads' gradients of a shared query or key head, in a fixed
// order: part [N, T, H, dim] in fp32 to y [N, T, H / group, dim].
struct SharedSumArgs {
    const float* part;
    SeqView y;
    int64_t N, T;
    int32_t H, group, dim;
};

template <class D>
__global__ __launch_bounds__(256) void shared_sum(const SharedSumArgs x)
{
    const int64_t kv = x.H / x.group, total = x.N * x.T * kv * x.dim;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / x.dim, tok = row / kv;
        const int e = (int)(i % x.dim), h = (int)(row % kv);
        const float* s = x.part + (tok * x.H + (int64_t)h * x.group) * x.dim + e;
        float sum = 0.0f;
        for (int k = 0; k < x.group; ++k) sum += s[(int64_t)k * x.dim];
        seq_row_out<D>(x.y, tok / x.T, tok % x.T, h)[e] = from_f32<D>(sum);
    }
}

// One step of every head: the state is read, updated and written, and read by
// the query, in one pass.  V: state elements per access.
struct StepArgs {
    SeqView q, k, v, g, reset, o;
    const float* state;
    float* next;
    float scale;
    int32_t H, dk, dv;
};

template <class D, int V>
__global__ __launch_bounds__(256) void recurrence_one_step(const StepArgs x)
{
    __shared__ float part[256 * V];
    const int64_t head = blockIdx.x, n = head / x.H;
    const int h = (int)(head % x.H), tid = threadIdx.x;
    const int cols = x.dv / V, groups = 256 / cols, c = tid % cols, r0 = tid / cols;
    const D* q = seq_row<D>(x.q, n, 0, h);
    const D* k = seq_row<D>(x.k, n, 0, h);
    const float g = to_f32(*seq_row<D>(x.g, n, 0, h));
    const bool reset = x.reset.p != nullptr && *seq_row<uint8_t>(x.reset, n, 0, 0) != 0;
    const float f = reset ? 0.0f : __expf(g);
    const int64_t at = head * x.dk * x.dv;
    float v[V], y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v[e] = to_f32(seq_row<D>(x.v, n, 0, h)[c * V + e]);
        y[e] = 0.0f;
    }
    if (r0 < groups) {
        for (int r = r0; r < x.dk; r += groups) {
            const float kr = to_f32(k[r]), qr = to_f32(q[r]);
            float s[V];
            const float* from = x.state + at + (int64_t)r * x.dv + c * V;
            float* to = x.next + at + (int64_t)r * x.dv + c * V;
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = f == 0.0f ? 0.0f : from[e];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[e] = fmaf(kr, v[e], s[e] * f);
                y[e] = fmaf(qr, s[e], y[e]);
                to[e] = s[e];
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) part[r0 * x.dv + c * V + e] = y[e];
    }
    __syncthreads();
    for (int j = tid; j < x.dv; j += 256) {
        float sum = 0.0f;
        for (int r = 0; r < groups; ++r) sum += part[r * x.dv + j];
        seq_row_out<D>(x.o, n, 0, h)[j] = from_f32<D>(sum * x.scale);
    }
}

// ------------------------------------------------------------------ entries

constexpr int64_t kMaxHeads = int64_t(1) << 23;  // num_envs * heads of a call

inline lrs_status check_recurrence(const char* nm, int64_t N, int64_t T, int64_t H, int64_t KV,
                                   int64_t dk, int64_t dv, float scale)
{
    LRS_TRY(check_common(nm, N, T));
    LRS_REQUIRE(H >= 1 && KV >= 1 && H <= 65536 && H % KV == 0,
                "%s: heads (%lld) must be a multiple of kv_heads (%lld), 65536 at most", nm,
                (long long)H, (long long)KV);
    LRS_REQUIRE(N <= kMaxHeads / H, "%s: num_envs * heads must be at most %lld", nm,
                (long long)kMaxHeads);
    LRS_REQUIRE(dk >= 1 && dk <= kMaxDim && dv >= 1 && dv <= kMaxDim,
                "%s: key_dim and value_dim must be 1 to %d (got %lld and %lld)", nm, kMaxDim,
                (long long)dk, (long long)dv);
    LRS_REQUIRE(scale - scale == 0.0f, "%s: scale must be finite", nm);
    return LRS_OK;
}

inline lrs_status check_state(const char* nm, const void* p, const char* what)
{
    LRS_REQUIRE((uintptr_t)p % 4 == 0, "%s: %s is not aligned to its elements", nm, what);
    return LRS_OK;
}

inline size_t round_up(size_t b) { return (b + 255) & ~size_t(255); }

// Workspace of a call.  Backward: q.dq and k.dk [N, H, T], <S_T, dS_T> [N, H]
// and, for shared query and key heads, each value head's dq and dk.
struct RecurrencePlan {
    size_t qdq, kdk, cross, dq, dk, bytes;
};

inline RecurrencePlan plan_recurrence(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk,
                                      int64_t dv, bool backward)
{
    (void)dv;
    RecurrencePlan p{};
    if (!backward) return p;
    size_t at = 0;
    const auto take = [&](size_t floats) {
        const size_t here = at;
        at += round_up(4 * floats);
        return here;
    };
    p.qdq = take((size_t)(N * T * H));
    p.kdk = take((size_t)(N * T * H));
    p.cross = take((size_t)(N * H));
    if (H != KV) {
        p.dq = take((size_t)(N * T * H * dk));
        p.dk = take((size_t)(N * T * H * dk));
    }
    p.bytes = at;
    return p;
}

template <class D>
lrs_status launch_passes(const char* nm, const RecurrenceArgs& x, int da, int dc, hipStream_t stream)
{
    const uint64_t blocks = (uint64_t)x.N * x.H * x.passes;
    const int threads = (dc + kWave - 1) / kWave * kWave;
    return da <= 64 ? launch_seq(nm, recurrence_steps<D, 64>, blocks, threads, stream, x)
                    : launch_seq(nm, recurrence_steps<D, 128>, blocks, threads, stream, x);
}

template <class D>
lrs_status recurrence_entry(const char* nm, int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk,
                            int64_t dv, const D* q, const D* k, const D* v, const D* g,
                            const uint8_t* reset, const float* initial, float scale, D* out,
                            float* final_state, const int64_t* strides, void* ws, size_t ws_bytes,
                            hipStream_t stream)
{
    LRS_TRY(check_recurrence(nm, N, T, H, KV, dk, dv, scale));
    constexpr int s = sizeof(D);
    const SeqArg args[6] = {{q, KV, dk, s, false, true, "q"},   {k, KV, dk, s, false, true, "k"},
                            {v, H, dv, s, false, true, "v"},    {g, H, 1, s, false, true, "log_decay"},
                            {reset, 1, 1, 1, false, false, "reset"}, {out, H, dv, s, true, true, "out"}};
    LRS_TRY(check_state(nm, initial, "initial_state"));
    LRS_TRY(check_state(nm, final_state, "final_state"));
    const uint64_t state = (uint64_t)(N * H * dk * dv) * 4;
    const Span more[] = {{final_state, state}, {ws, ws_bytes}, {initial, state}};
    SeqView w[6];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, more, 2, 3, w));
    const RecurrencePlan plan = plan_recurrence(N, T, H, KV, dk, dv, false);
    LRS_TRY(check_workspace(nm, plan.bytes, ws, ws_bytes));
    w[0].div = w[1].div = (int32_t)(H / KV);
    RecurrenceArgs x{};
    x.g = w[3];
    x.reset = w[4];
    x.N = N;
    x.T = T;
    x.H = (int32_t)H;
    x.passes = 1;
    PassArgs& p = x.pass[0];
    p.a = w[0];
    p.b = w[1];
    p.c = w[2];
    p.y = w[5];
    p.init = initial;
    p.last = final_state;
    p.y_scale = scale;
    p.u_scale = 1.0f;
    p.da = (int32_t)dk;
    p.dc = (int32_t)dv;
    return launch_passes<D>(nm, x, (int)dk, (int)dv, stream);
}

template <class D>
lrs_status recurrence_backward_entry(const char* nm, int64_t N, int64_t T, int64_t H, int64_t KV,
                                     int64_t dk, int64_t dv, const D* grad_out, const D* q,
                                     const D* k, const D* v, const D* g, const uint8_t* reset,
                                     const float* initial, const float* grad_final, float scale,
                                     D* grad_q, D* grad_k, D* grad_v, D* grad_g, float* grad_initial,
                                     const int64_t* strides, void* ws, size_t ws_bytes,
                                     hipStream_t stream)
{
    LRS_TRY(check_recurrence(nm, N, T, H, KV, dk, dv, scale));
    constexpr int s = sizeof(D);
    const SeqArg args[10] = {
        {grad_out, H, dv, s, false, true, "grad_out"}, {q, KV, dk, s, false, true, "q"},
        {k, KV, dk, s, false, true, "k"},              {v, H, dv, s, false, true, "v"},
        {g, H, 1, s, false, true, "log_decay"},        {reset, 1, 1, 1, false, false, "reset"},
        {grad_q, KV, dk, s, true, true, "grad_q"},     {grad_k, KV, dk, s, true, true, "grad_k"},
        {grad_v, H, dv, s, true, true, "grad_v"},      {grad_g, H, 1, s, true, true, "grad_log_decay"}};
    LRS_TRY(check_state(nm, initial, "initial_state"));
    LRS_TRY(check_state(nm, grad_final, "grad_final_state"));
    LRS_TRY(check_state(nm, grad_initial, "grad_initial_state"));
    const uint64_t state = (uint64_t)(N * H * dk * dv) * 4;
    const Span more[] = {{grad_initial, state}, {ws, ws_bytes}, {initial, state}, {grad_final, state}};
    SeqView w[10];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, more, 2, 4, w));
    const RecurrencePlan plan = plan_recurrence(N, T, H, KV, dk, dv, true);
    LRS_TRY(check_workspace(nm, plan.bytes, ws, ws_bytes));
    const int32_t group = (int32_t)(H / KV);
    w[1].div = w[2].div = group;
    char* base = static_cast<char*>(ws);
    float* const qdq = reinterpret_cast<float*>(base + plan.qdq);
    float* const kdk = reinterpret_cast<float*>(base + plan.kdk);
    float* const cross = reinterpret_cast<float*>(base + plan.cross);
    float* const part_q = reinterpret_cast<float*>(base + plan.dq);
    float* const part_k = reinterpret_cast<float*>(base + plan.dk);
    const auto partial = [&](const float* p) {
        return SeqView{p, T * H * dk, H * dk, dk, 1};
    };
    RecurrenceArgs x{};
    x.g = w[4];
    x.reset = w[5];
    x.N = N;
    x.T = T;
    x.H = (int32_t)H;
    x.passes = 3;
    PassArgs& pq = x.pass[0];  // dq
    pq.a = w[0];
    pq.b = w[3];
    pq.c = w[2];
    pq.d = w[1];
    pq.y = group > 1 ? partial(part_q) : w[6];
    pq.init = initial;
    pq.meet = grad_final;
    pq.dot = qdq;
    pq.cross = cross;
    pq.y_scale = scale;
    pq.u_scale = 1.0f;
    pq.da = (int32_t)dv;
    pq.dc = (int32_t)dk;
    pq.transposed = 1;
    pq.y_f32 = group > 1;
    PassArgs& pk = x.pass[1];  // dk
    pk.a = w[3];
    pk.b = w[0];
    pk.c = w[1];
    pk.d = w[2];
    pk.y = group > 1 ? partial(part_k) : w[7];
    pk.init = grad_final;
    pk.dot = kdk;
    pk.y_scale = 1.0f;
    pk.u_scale = scale;
    pk.da = (int32_t)dv;
    pk.dc = (int32_t)dk;
    pk.reverse = 1;
    pk.transposed = 1;
    pk.y_f32 = group > 1;
    PassArgs& pv = x.pass[2];  // dv
    pv.a = w[2];
    pv.b = w[1];
    pv.c = w[0];
    pv.y = w[8];
    pv.init = grad_final;
    pv.last = grad_initial;
    pv.y_scale = 1.0f;
    pv.u_scale = scale;
    pv.da = (int32_t)dk;
    pv.dc = (int32_t)dv;
    pv.reverse = 1;
    const int widest = (int)(dk > dv ? dk : dv);
    LRS_TRY(launch_passes<D>(nm, x, widest, widest, stream));
    DecayGradArgs dg{w[4], w[5], w[9], qdq, kdk, cross, N, T, (int32_t)H};
    LRS_TRY(launch_seq(nm, decay_grad<D>, (uint64_t)(N * H), 64, stream, dg));
    if (group > 1) {
        const int64_t blocks = (N * T * KV * dk + 255) / 256;
        for (int i = 0; i < 2; ++i) {
            SharedSumArgs sum{i ? part_k : part_q, w[i ? 7 : 6], N, T, (int32_t)H, group, (int32_t)dk};
            LRS_TRY(launch_seq(nm, shared_sum<D>, (uint64_t)(blocks < 8192 ? blocks : 8192), 256, stream,
                               sum));
        }
    }
    return LRS_OK;
}

template <class D>
lrs_status recurrence_step_entry(const char* nm, int64_t N, int64_t H, int64_t KV, int64_t dk,
                                 int64_t dv, const D* q, const D* k, const D* v, const D* g,
                                 const uint8_t* reset, const float* state, float scale, D* out,
                                 float* next, const int64_t* strides, hipStream_t stream)
{
    LRS_TRY(check_recurrence(nm, N, 1, H, KV, dk, dv, scale));
    LRS_REQUIRE(state && next, "%s: state and next_state are required", nm);
    constexpr int s = sizeof(D);
    const SeqArg args[6] = {{q, KV, dk, s, false, true, "q"},   {k, KV, dk, s, false, true, "k"},
                            {v, H, dv, s, false, true, "v"},    {g, H, 1, s, false, true, "log_decay"},
                            {reset, 1, 1, 1, false, false, "reset"}, {out, H, dv, s, true, true, "out"}};
    LRS_TRY(check_state(nm, state, "state"));
    LRS_TRY(check_state(nm, next, "next_state"));
    const uint64_t bytes = (uint64_t)(N * H * dk * dv) * 4;
    // the state may be updated in place: each of its elements is read and
    // written by one thread
    const Span more[] = {{next, bytes}, {next == state ? nullptr : state, bytes}};
    SeqView w[6];
    LRS_TRY(check_seq_arrays(nm, N, 1, args, strides, more, 1, 2, w));
    w[0].div = w[1].div = (int32_t)(H / KV);
    const StepArgs x{w[0], w[1], w[2], w[3], w[4], w[5], state, next, scale, (int32_t)H, (int32_t)dk,
                     (int32_t)dv};
    const bool four = dv % 4 == 0 && aligned(state, 16) && aligned(next, 16);
    return four ? launch_seq(nm, recurrence_one_step<D, 4>, (uint64_t)(N * H), 256, stream, x)
                : launch_seq(nm, recurrence_one_step<D, 1>, (uint64_t)(N * H), 256, stream, x);
}

}  // namespace lrs
