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

#include <algorithm>

#include "sequence.hpp"

namespace lrs {

constexpr int kMaxDim = 128;  // largest key and value dimension

// One pass over the sequence, in segments of seg_len steps that blocks work on
// side by side.  init: each segment's state before its first step in scan order,
// [N, H, segments, key_dim, value_dim] (nullable for one segment); last: where
// the state after the last segment goes, [N, H, key_dim, value_dim], nullable.
// y_scale multiplies y, p_scale the products a . b, u_scale what enters the
// state.  dot (nullable): receives y_i . d_i per [N, H, T]; cross (nullable):
// <state after the segment, meet> per [N, H, segments], meet like init.
struct PassArgs {
    SeqView a, b, c, d, y;
    const float* init;
    float* last;
    const float* meet;
    float* dot;
    float* cross;
    float y_scale, p_scale, u_scale;
    int32_t da, dc;  // dims of a and b, of c and y
    uint8_t transposed, y_f32;
};

// Where the segments of one direction leave their own states (from zero), for
// the next segment in scan order, and their decays.
struct CarryArgs {
    SeqView b, c;
    float* states;  // [N, H, segments, key_dim, value_dim]
    float* totals;  // [N, H, segments]
    const float* init;  // the state before the first segment, nullable
    float u_scale;
    int32_t da, dc;
    uint8_t reverse;
};

struct RecurrenceArgs {
    SeqView g, reset;
    int64_t N, T, seg_len;
    int32_t H, carries, segments;
    PassArgs pass[3];
    CarryArgs carry[2];
};

// Row r (of a's dim) and column c (of y's dim) of a state in memory.
__device__ __forceinline__ int64_t state_at(const PassArgs& p, int r, int c)
{
    return p.transposed ? (int64_t)c * p.da + r : (int64_t)r * p.dc + c;
}

// ------------------------------------------------------- matrix instructions
// All products run as bf16 matrix instructions with fp32 sums.  A value is a
// sum of bf16 limbs, each the rounding of what the ones before leave: bf16
// inputs are one limb, f16 inputs two (exact), f32 inputs three.  What is
// computed in fp32 on the way to another product (weighted products, states)
// is split as far as its result needs.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <class D>
constexpr int kLimbs = std::is_same<D, bf16_t>::value ? 1 : std::is_same<D, f16_t>::value ? 2 : 3;

template <int L>
struct Frag {
    bf16x8 x[L];
};

template <int L>
__device__ __forceinline__ Frag<L> split(f32x8 v)
{
    Frag<L> f;
#pragma unroll
    for (int l = 0; l < L; ++l) {
        f.x[l] = __builtin_convertvector(v, bf16x8);
        if (l + 1 < L) v -= __builtin_convertvector(f.x[l], f32x8);
    }
    return f;
}

// acc += A^T B over 32 products per lane group, all limb products down to the
// smaller operand's last limb.
template <int LA, int LB>
__device__ __forceinline__ f32x4 mma(const Frag<LA>& a, const Frag<LB>& b, f32x4 acc)
{
    constexpr int level = LA > LB ? LA : LB;
#pragma unroll
    for (int i = 0; i < LA; ++i)
#pragma unroll
        for (int j = 0; j < LB; ++j)
            if (i + j < level)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x[i], b.x[j], acc, 0, 0, 0);
    return acc;
}

// A tile of kChunk steps of up to W elements in LDS, one plane per limb.  The
// 16-byte units of a row are permuted by its index, so that both ways of
// reading a fragment (16 rows at one unit; 4 rows at 16 neighbouring columns,
// transposed) touch every bank once.
constexpr int kChunk = 64;
constexpr int kTile = 16;

template <int W, int L>
struct StepTile {
    uint16_t e[L][kChunk * W];

    static __device__ __forceinline__ int at(int row, int col)
    {
        const int mix = W == 128 ? ((row & 7) << 1) | ((row >> 3) & 1)
                                 : (((row >> 1) & 3) << 1) | ((row >> 3) & 1);
        return row * W + (((col >> 3) ^ mix) << 3) + (col & 7);
    }
    // A fragment of 16 rows (from `row`) over 32 columns (from `col`): lane l
    // holds row l % 16, columns 4 (l / 16) + 0..3 and 16 more.  Both operands
    // of every product use this order of the 32.
    __device__ __forceinline__ Frag<L> rows(int row, int col, int lane) const
    {
        const int r = row + (lane & 15), c = col + (lane >> 4) * 4;
        Frag<L> f;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const s16x4 lo = *reinterpret_cast<const s16x4*>(&e[l][at(r, c)]);
            const s16x4 hi = *reinterpret_cast<const s16x4*>(&e[l][at(r, c + 16)]);
            f.x[l] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
    // The transposed fragment: lane l holds column col + l % 16 of the rows
    // row + 4 (l / 16) + 0..3 and 16 more.  A transposing read hands the 16
    // lanes of a group four rows of 16 columns, 8 bytes read by each lane.
    __device__ __forceinline__ Frag<L> columns(int row, int col, int lane) const
    {
        const int r = row + (lane >> 4) * 4 + ((lane & 15) >> 2), c = col + (lane & 3) * 4;
        Frag<L> f;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)&e[l][at(r, c)]);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)&e[l][at(r + 16, c)]);
            f.x[l] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
};

// Eight elements of a row from column c on, zero beyond `dim`.
template <class D>
__device__ __forceinline__ f32x8 load8(const D* row, int c, int dim, bool vec)
{
    f32x8 v = {};
    if (vec && c + 8 <= dim) {
        if constexpr (sizeof(D) == 4) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(row + c);
            const f32x4 b = *reinterpret_cast<const f32x4*>(row + c + 4);
            v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const u32x4 w = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                unpack2<D>(w[k], lo, hi);
                v[2 * k] = lo;
                v[2 * k + 1] = hi;
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < dim) v[k] = to_f32(row[c + k]);
    }
    return v;
}

// The same as one-limb elements, unconverted.
__device__ __forceinline__ u32x4 load8_raw(const bf16_t* row, int c, int dim, bool vec)
{
    if (vec && c + 8 <= dim) return *reinterpret_cast<const u32x4*>(row + c);
    u32x4 w = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < dim) w[k / 2] |= (uint32_t)row[c + k].bits << (16 * (k & 1));
    return w;
}

// Steps t0 .. t0 + count - 1 of one head into a tile, zero beyond them.
template <class D, int W>
__device__ __forceinline__ void stage(StepTile<W, kLimbs<D>>& tile, const SeqView& view, int64_t n, int h,
                                      int64_t t0, int count, int dim)
{
    constexpr int L = kLimbs<D>;
    const int units = (dim + 31) / 32 * 4;  // what the products read
    for (int u = threadIdx.x; u < kChunk * units; u += blockDim.x) {
        const int row = u / units, c = (u % units) * 8;
        if constexpr (L == 1) {
            u32x4 v = {};
            if (row < count) v = load8_raw(seq_row<D>(view, n, t0 + row, h), c, dim, view.vec != 0);
            *reinterpret_cast<u32x4*>(&tile.e[0][tile.at(row, c)]) = v;
        } else {
            f32x8 v = {};
            if (row < count) v = load8(seq_row<D>(view, n, t0 + row, h), c, dim, view.vec != 0);
            const Frag<L> f = split<L>(v);
#pragma unroll
            for (int l = 0; l < L; ++l) *reinterpret_cast<bf16x8*>(&tile.e[l][tile.at(row, c)]) = f.x[l];
        }
    }
}

// The decays of a chunk of 64 steps, in four tiles of 16.  With p the running
// sum of log2 decays within a tile (in 64 bits: a strong decay before a weak
// one would cost an fp32 sum the weak one's digits) and m the running count of
// its cuts, for steps j < i of one tile D(i, j) = 2^(p_i - p_j) where m_i =
// m_j, and for steps of tiles B > A, D(i, j) = head_i (tiles between) tail_j,
// where each factor is at most 1 for log decays up to 0.
struct ChunkDecay {
    double p[kChunk];
    int m[kChunk];
    float head[kChunk];   // from the start of its tile to this step, inclusive
    float tail[kChunk];   // from this step, exclusive, to the end of its tile
    float entry[kChunk];  // from the start of the chunk, inclusive
    float exit[kChunk];   // to the end of the chunk
    float whole[4];       // of each tile
    float total;          // of the chunk
};

template <class D>
__device__ __forceinline__ void chunk_decay(ChunkDecay& s, const RecurrenceArgs& x, int64_t n, int h,
                                            int64_t t0, int count, int lane)
{
    double p = 0.0;
    int m = 0;
    if (lane < count) {
        const float g = to_f32(*seq_row<D>(x.g, n, t0 + lane, h));
        const bool reset = x.reset.p != nullptr && *seq_row<uint8_t>(x.reset, n, t0 + lane, 0) != 0;
        m = reset || g == -INFINITY;
        p = m ? 0.0 : (double)g * 1.4426950408889634;
    }
    const int i = lane & 15;
#pragma unroll
    for (int o = 1; o < kTile; o <<= 1) {
        const double q = __shfl_up(p, o);
        const int k = __shfl_up(m, o);
        if (i >= o) {
            p += q;
            m += k;
        }
    }
    const double ptot = __shfl(p, lane | 15);
    const int mtot = __shfl(m, lane | 15);
    const float head = m ? 0.0f : exp2f((float)p);
    const float tail = m != mtot ? 0.0f : exp2f((float)(ptot - p));
    const float whole = mtot ? 0.0f : exp2f((float)ptot);
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __shfl(whole, k * kTile);
    const int tile = lane >> 4;
    float before = 1.0f, after = 1.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < tile) before *= w[k];
        if (k > tile) after *= w[k];
    }
    s.p[lane] = p;
    s.m[lane] = m;
    s.head[lane] = head;
    s.tail[lane] = tail;
    s.entry[lane] = before * head;
    s.exit[lane] = after * tail;
    if (lane < 4) s.whole[lane] = w[lane];
    if (lane == 0) s.total = w[0] * w[1] * w[2] * w[3];
}

// S = total S + b^T (w c) over a chunk of 64 steps; w: the weight of each step,
// fc: the wave's columns of c.
template <class D, int W>
__device__ __forceinline__ void add_chunk(f32x4 (&S)[W / 16][2], const StepTile<W, kLimbs<D>>& tb,
                                          const Frag<kLimbs<D>> (&fc)[2][2], const float* w, float total,
                                          float scale, int da, int lane)
{
    constexpr int L = kLimbs<D>;
    constexpr int LW = 3;  // limbs of the weighted c: states are fp32, their sums keep 24 bits
    const int group = lane >> 4;
    Frag<LW> fw[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(&w[b * 32 + group * 4]);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(&w[b * 32 + 16 + group * 4]);
        const f32x8 v8 = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7) * scale;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x8 v = __builtin_convertvector(fc[b][u].x[0], f32x8);
#pragma unroll
            for (int l = 1; l < L; ++l) v += __builtin_convertvector(fc[b][u].x[l], f32x8);
            fw[b][u] = split<LW>(v * v8);
        }
    }
#pragma unroll
    for (int k = 0; k < W / 16; ++k) {
        if (k * 16 >= da) break;
        const Frag<L> fb[2] = {tb.columns(0, k * 16, lane), tb.columns(32, k * 16, lane)};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // a cut drops the state, whatever it holds
            f32x4 v = total == 0.0f ? f32x4{} : S[k][u] * total;
#pragma unroll
            for (int b = 0; b < 2; ++b) v = mma(fb[b], fw[b][u], v);
            S[k][u] = v;
        }
    }
}

// A pass by matrix instructions, 64 steps at a time.  A wave holds 32 columns
// of the state, all its rows, in accumulators; the block's waves share the
// steps in LDS.  Per chunk, with X, Z the weights from the chunk's start and to
// its end in scan order:
//     y^T = S^T a^T X + c^T (D o (a b^T))^T        (S before the chunk)
//     S   = total S + b^T (Z c)
// Results of one product leave the matrix unit in the order in which the next
// one takes its operand (16 columns by 4 consecutive rows per lane group), so
// a b^T and S go from product to product in registers.
template <class D, int W>
struct PassShared {
    StepTile<W, kLimbs<D>> a, b, c;
    ChunkDecay decay;
    float dot[4][kChunk];
    float cross[4];
};

// Four elements of a row from column c on, out of `dim` (one access where the
// row allows it).
template <class D>
__device__ __forceinline__ void store4(D* row, int c, int dim, bool vec, f32x4 v)
{
    if (vec) {
        if (c >= dim) return;
        if constexpr (sizeof(D) == 4)
            *reinterpret_cast<f32x4*>(row + c) = v;
        else
            *reinterpret_cast<u32x2*>(row + c) = u32x2{pack2<D>(v[0], v[1]), pack2<D>(v[2], v[3])};
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (c + r < dim) row[c + r] = from_f32<D>(v[r]);
    }
}
template <class D>
__device__ __forceinline__ f32x4 load4(const D* row, int c, int dim, bool vec)
{
    f32x4 v = {};
    if (vec) {
        if (c >= dim) return v;
        if constexpr (sizeof(D) == 4) {
            v = *reinterpret_cast<const f32x4*>(row + c);
        } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(row + c);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float lo, hi;
                unpack2<D>(w[k], lo, hi);
                v[2 * k] = lo;
                v[2 * k + 1] = hi;
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (c + r < dim) v[r] = to_f32(row[c + r]);
    }
    return v;
}

template <class D, int W, bool back, bool kPrecise>
__device__ __forceinline__ void run_pass(const RecurrenceArgs& x, const PassArgs& p, uint32_t block,
                                         PassShared<D, W>& sh)
{
    constexpr int L = kLimbs<D>;
    constexpr int LS = L > 1 ? L : (kPrecise ? 2 : 1);  // limbs of a b^T and of the state
    constexpr int K = W / 32;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int group = lane >> 4, col = lane & 15;
    const int64_t head = block / x.segments;
    const int seg = (int)(block % x.segments);
    const int64_t n = head / x.H;
    const int h = (int)(head % x.H);
    const int c0 = wave * 32;
    const int64_t at = (int64_t)block * p.da * p.dc;
    const int64_t first = seg * x.seg_len;
    const int64_t steps = x.T - first < x.seg_len ? x.T - first : x.seg_len;

    // S[2 k + s][u][r]: row 32 k + 16 s + 4 group + r, column c0 + 16 u + col
    f32x4 S[2 * K][2];
#pragma unroll
    for (int k = 0; k < 2 * K; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = k * 16 + group * 4 + r, c = c0 + u * 16 + col;
                S[k][u][r] = p.init && row < p.da && c < p.dc ? p.init[at + state_at(p, row, c)] : 0.0f;
            }

    const int64_t chunks = (steps + kChunk - 1) / kChunk;
    for (int64_t i = 0; i < chunks; ++i) {
        const int64_t done = (back ? chunks - 1 - i : i) * kChunk;
        const int64_t t0 = first + done;
        const int count = (int)(steps - done < kChunk ? steps - done : kChunk);
        __syncthreads();
        if (wave == 0) chunk_decay<D>(sh.decay, x, n, h, t0, count, lane);
        stage<D, W>(sh.a, p.a, n, h, t0, count, p.da);
        stage<D, W>(sh.b, p.b, n, h, t0, count, p.da);
        stage<D, W>(sh.c, p.c, n, h, t0, count, p.dc);
        __syncthreads();

        if (c0 < p.dc) {
            // y^T of tile q: rows c0 + 16 u + 4 group + r, column (step) 16 q + col;
            // ab[q][s]: rows (steps) 16 s + 4 group + r, column 16 q + col
            f32x4 y[4][2] = {}, ab[4][4] = {};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (k * 32 >= p.da) break;
                Frag<LS> s[2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    s[u] = split<LS>(__builtin_shufflevector(S[2 * k][u], S[2 * k + 1][u], 0, 1, 2, 3, 4, 5, 6, 7));
                Frag<L> fb[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) fb[q] = sh.b.rows(q * 16, k * 32, lane);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const Frag<L> fa = sh.a.rows(q * 16, k * 32, lane);
#pragma unroll
                    for (int u = 0; u < 2; ++u) y[q][u] = mma(s[u], fa, y[q][u]);
                    // only one side of the diagonal is used: forward steps s <= q
#pragma unroll
                    for (int s2 = 0; s2 < 4; ++s2)
                        if (back ? s2 >= q : s2 <= q) ab[q][s2] = mma(fb[s2], fa, ab[q][s2]);
                }
            }

            // weights
            Frag<L> fc[2][2];  // columns c0 + 16 u + l % 16 of 32 steps each
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int u = 0; u < 2; ++u) fc[b][u] = sh.c.columns(b * 32, c0 + u * 16, lane);
            const float* from = back ? sh.decay.exit : sh.decay.entry;
            const float* mine = back ? sh.decay.tail : sh.decay.head;
            const float* theirs = back ? sh.decay.head : sh.decay.tail;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int step = q * 16 + col;
                const float in = from[step];
#pragma unroll
                for (int u = 0; u < 2; ++u) y[q][u] = in == 0.0f ? f32x4{} : y[q][u] * in;
                float lead = mine[step] * p.p_scale;
                // tiles from the nearest on, the decay of those between gathered on the way
#pragma unroll
                for (int d = 1; d < 4; ++d) {
                    const int s = back ? q + d : q - d;
                    if (s < 0 || s > 3) continue;
                    const f32x4 f = *reinterpret_cast<const f32x4*>(&theirs[s * 16 + group * 4]);
#pragma unroll
                    for (int s2 = 0; s2 < 4; ++s2)
                        if (s2 == s) ab[q][s2] *= f * lead;
                    lead *= sh.decay.whole[s];
                }
                const double pi = sh.decay.p[step];
                const int mi = sh.decay.m[step];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = q * 16 + group * 4 + r;
                    const double d = back ? sh.decay.p[j] - pi : pi - sh.decay.p[j];
                    const bool in_order = back ? j >= step : j <= step;
                    const float w = in_order && sh.decay.m[j] == mi ? exp2f((float)d) * p.p_scale : 0.0f;
                    ab[q][q][r] = w == 0.0f ? 0.0f : ab[q][q][r] * w;
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (back ? 2 * b + 1 < q : 2 * b > q) continue;
                    const Frag<LS> fp =
                        split<LS>(__builtin_shufflevector(ab[q][2 * b], ab[q][2 * b + 1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                    for (int u = 0; u < 2; ++u) y[q][u] = mma(fc[b][u], fp, y[q][u]);
                }
            }

            // y out
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int step = q * 16 + col;
                float dot = 0.0f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = c0 + u * 16 + group * 4;
                    const f32x4 v = y[q][u] * p.y_scale;
                    if (step < count) {
                        if (kPrecise) {
                            const f32x4 d = load4<D>(seq_row<D>(p.d, n, t0 + step, h), c, p.dc, p.d.vec != 0) * v;
                            dot += (d[0] + d[1]) + (d[2] + d[3]);
                        }
                        if (kPrecise && p.y_f32)
                            store4<float>(seq_row_out<float>(p.y, n, t0 + step, h), c, p.dc, p.y.vec != 0, v);
                        else
                            store4<D>(seq_row_out<D>(p.y, n, t0 + step, h), c, p.dc, p.y.vec != 0, v);
                    }
                }
                if (kPrecise) {
                    dot += __shfl_xor(dot, 16);
                    dot += __shfl_xor(dot, 32);
                    if (group == 0) sh.dot[wave][step] = dot;
                }
            }

            // the state after the chunk
            add_chunk<D, W>(S, sh.b, fc, back ? sh.decay.entry : sh.decay.exit, sh.decay.total, p.u_scale, p.da,
                            lane);
        }
        if (kPrecise) {
            __syncthreads();
            if (wave == 0 && lane < count) {
                float sum = 0.0f;
                for (int w = 0; w * 32 < p.dc; ++w) sum += sh.dot[w][lane];
                p.dot[head * x.T + t0 + lane] = sum;
            }
        }
    }

    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 2 * K; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = k * 16 + group * 4 + r, c = c0 + u * 16 + col;
                if (row >= p.da || c >= p.dc) continue;
                if (p.last && seg == (back ? 0 : x.segments - 1))
                    p.last[head * p.da * p.dc + state_at(p, row, c)] = S[k][u][r];
                if (p.cross && p.meet) v = fmaf(S[k][u][r], p.meet[at + state_at(p, row, c)], v);
            }
    if (p.cross) {
        for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
        if (lane == 0) sh.cross[wave] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int w = 0; w < (int)blockDim.x / kWave; ++w) sum += sh.cross[w];
            p.cross[block] = sum;
        }
    }
}

template <class D, int W>
__global__ __launch_bounds__(2 * W, 2) void recurrence_forward(const RecurrenceArgs x)
{
    __shared__ PassShared<D, W> sh;
    run_pass<D, W, false, false>(x, x.pass[0], blockIdx.x, sh);
}

// The three passes of the backward call: dq and dk with q.dq and k.dk to a
// precision that their differences keep, and dv.
template <class D, int W>
__global__ __launch_bounds__(2 * W, 2) void recurrence_backward(const RecurrenceArgs x)
{
    __shared__ PassShared<D, W> sh;
    const uint32_t block = blockIdx.x / 3, pass = blockIdx.x % 3;
    if (pass == 0) run_pass<D, W, false, true>(x, x.pass[0], block, sh);
    else if (pass == 1) run_pass<D, W, true, true>(x, x.pass[1], block, sh);
    else run_pass<D, W, true, false>(x, x.pass[2], block, sh);
}

// The state that one segment alone leaves (from zero), and its decay, by the
// same products; the last segment in scan order leaves none that is used.
template <class D, int W>
__global__ __launch_bounds__(2 * W) void segment_states(const RecurrenceArgs x)
{
    __shared__ struct {
        StepTile<W, kLimbs<D>> b, c;
        ChunkDecay decay;
    } sh;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int group = lane >> 4, col = lane & 15;
    const CarryArgs& p = x.carry[blockIdx.x % x.carries];
    const uint32_t block = blockIdx.x / x.carries;
    const int64_t head = block / (x.segments - 1);
    const bool back = p.reverse != 0;
    const int seg = (int)(block % (x.segments - 1)) + (back ? 1 : 0);
    const int next = back ? seg - 1 : seg + 1;
    const int64_t n = head / x.H;
    const int h = (int)(head % x.H);
    const int c0 = wave * 32;
    const int64_t first = seg * x.seg_len;
    const int64_t steps = x.T - first < x.seg_len ? x.T - first : x.seg_len;
    f32x4 S[W / 16][2] = {};
    float total = 1.0f;
    const int64_t chunks = (steps + kChunk - 1) / kChunk;
    for (int64_t i = 0; i < chunks; ++i) {
        const int64_t done = (back ? chunks - 1 - i : i) * kChunk;
        const int64_t t0 = first + done;
        const int count = (int)(steps - done < kChunk ? steps - done : kChunk);
        __syncthreads();
        if (wave == 0) chunk_decay<D>(sh.decay, x, n, h, t0, count, lane);
        stage<D, W>(sh.b, p.b, n, h, t0, count, p.da);
        stage<D, W>(sh.c, p.c, n, h, t0, count, p.dc);
        __syncthreads();
        if (c0 >= p.dc) continue;
        Frag<kLimbs<D>> fc[2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int u = 0; u < 2; ++u) fc[b][u] = sh.c.columns(b * 32, c0 + u * 16, lane);
        add_chunk<D, W>(S, sh.b, fc, back ? sh.decay.entry : sh.decay.exit, sh.decay.total, p.u_scale, p.da,
                        lane);
        total *= sh.decay.total;
    }
    float* const to = p.states + (head * x.segments + next) * (int64_t)p.da * p.dc;
#pragma unroll
    for (int k = 0; k < W / 16; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = k * 16 + group * 4 + r, c = c0 + u * 16 + col;
                if (row < p.da && c < p.dc) to[(int64_t)row * p.dc + c] = S[k][u][r];
            }
    // (wave 0 always has columns, and with them the whole decay)
    if (threadIdx.x == 0) p.totals[head * x.segments + seg] = total;
}

// Turns the segments' own states into the states before each of them, in scan
// order: in[s] = own[s - 1] + total[s - 1] in[s - 1].  A thread per element;
// the loads of kAhead segments are in flight together.
constexpr int kAhead = 8;

template <class D>
__global__ __launch_bounds__(256) void join_segments(const RecurrenceArgs x)
{
    const CarryArgs& p = x.carry[blockIdx.x % x.carries];
    const int64_t size = (int64_t)p.da * p.dc;
    const int64_t e = (int64_t)(blockIdx.x / x.carries) * 256 + threadIdx.x;
    const int64_t head = e / size, i = e % size;
    if (head >= x.N * x.H) return;
    float* const s = p.states + head * x.segments * size + i;
    const float* const f = p.totals + head * x.segments;
    const bool back = p.reverse != 0;
    const auto place = [&](int k) { return back ? x.segments - 1 - k : k; };
    float v = p.init ? p.init[head * size + i] : 0.0f;
    s[place(0) * size] = v;
    for (int k = 1; k < x.segments; k += kAhead) {
        float own[kAhead], total[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (k + a < x.segments) {
                own[a] = s[place(k + a) * size];
                total[a] = f[place(k + a - 1)];
            }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (k + a < x.segments) {
                v = total[a] == 0.0f ? own[a] : fmaf(total[a], v, own[a]);
                s[place(k + a) * size] = v;
            }
    }
}

// dg of one segment of a head by one wave, 64 steps at a time from its end: a
// suffix sum of q.dq - k.dk in 64 bits (its terms cancel), from <state after
// the segment, its gradient>, started again at each cut, where nothing is
// carried over and dg is 0.
struct DecayGradArgs {
    SeqView g, reset, dg;
    const float *qdq, *kdk, *cross;
    int64_t N, T, seg_len;
    int32_t H, segments;
};

template <class D>
__global__ __launch_bounds__(64) void decay_grad(const DecayGradArgs x)
{
    const int64_t head = blockIdx.x / x.segments, n = head / x.H;
    const int h = (int)(head % x.H), lane = threadIdx.x;
    const int64_t first = (int64_t)(blockIdx.x % x.segments) * x.seg_len;
    const int64_t past = x.T - first < x.seg_len ? x.T : first + x.seg_len;
    double carry = x.cross[blockIdx.x];
    for (int64_t end = past; end > first; end -= kWave) {
        const int64_t t = end - 1 - lane;
        double v = 0.0;
        bool cut = false;
        if (t >= first) {
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
        if (t >= first) *seq_row_out<D>(x.dg, n, t, h) = from_f32<D>(cut ? 0.0f : (float)v);
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

constexpr int64_t kMaxHeads = int64_t(1) << 22;  // num_envs * heads of a call

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

// How a call is cut up, and its workspace.  A pass has a block per head and
// segment: one segment where the heads alone fill the chip, else as many as
// give kFillBlocks blocks, of at least kMinSegment steps (a segment costs one
// more reading of two of its arrays and a state written and read twice).
// Workspace: the states before each segment and the segments' decays, per
// direction; backward also q.dq and k.dk [N, H, T], <S, dS> [N, H, segments]
// and, for shared query and key heads, each value head's dq and dk.
constexpr int64_t kFillBlocks = 512;
constexpr int64_t kMinSegment = 256;

struct RecurrencePlan {
    int64_t seg_len, segments;
    size_t states[2], totals[2], qdq, kdk, cross, dq, dk, bytes;
};

inline RecurrencePlan plan_recurrence(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk,
                                      int64_t dv, bool backward)
{
    RecurrencePlan p{};
    const int64_t heads = N * H * (backward ? 3 : 1);
    int64_t parts = std::min((kFillBlocks + heads - 1) / heads, (T + kMinSegment - 1) / kMinSegment);
    if (heads >= kFillBlocks) parts = 1;
    p.seg_len = ((T + parts - 1) / parts + kChunk - 1) / kChunk * kChunk;
    p.segments = (T + p.seg_len - 1) / p.seg_len;
    size_t at = 0;
    const auto take = [&](int64_t floats) {
        const size_t here = at;
        at += round_up(4 * (size_t)floats);
        return here;
    };
    if (p.segments > 1)
        for (int i = 0; i < (backward ? 2 : 1); ++i) {
            p.states[i] = take(N * H * p.segments * dk * dv);
            p.totals[i] = take(N * H * p.segments);
        }
    if (backward) {
        p.qdq = take(N * T * H);
        p.kdk = take(N * T * H);
        p.cross = take(N * H * p.segments);
        if (H != KV) {
            p.dq = take(N * T * H * dk);
            p.dk = take(N * T * H * dk);
        }
    }
    p.bytes = at;
    return p;
}

// Whether rows start where accesses of `unit` elements may.
inline void set_vec(SeqView& v, int unit, int elem_bytes)
{
    v.vec = aligned(v.p, (uintptr_t)(unit * elem_bytes)) && v.env % unit == 0 && v.step % unit == 0 &&
            v.head % unit == 0;
}

template <class D>
void set_vec(PassArgs& p)
{
    constexpr int s = sizeof(D), unit = 16 / s;
    set_vec(p.a, unit, s);
    set_vec(p.b, unit, s);
    set_vec(p.c, unit, s);
    set_vec(p.d, 4, s);
    set_vec(p.y, 4, p.y_f32 ? 4 : s);
    if (p.dc % 4 != 0) p.d.vec = p.y.vec = 0;
}

// The states before every segment, in x.carry's directions.
template <class D>
lrs_status launch_carries(const char* nm, RecurrenceArgs x, hipStream_t stream)
{
    if (x.segments == 1) return LRS_OK;
    for (int i = 0; i < x.carries; ++i) {
        set_vec(x.carry[i].b, 16 / sizeof(D), sizeof(D));
        set_vec(x.carry[i].c, 16 / sizeof(D), sizeof(D));
    }
    const int da = x.carry[0].da, dc = x.carry[0].dc;
    const uint64_t heads = (uint64_t)x.N * x.H, blocks = heads * (x.segments - 1) * x.carries;
    LRS_TRY(std::max(da, dc) <= 64 ? launch_seq(nm, segment_states<D, 64>, blocks, 128, stream, x)
                                   : launch_seq(nm, segment_states<D, 128>, blocks, 256, stream, x));
    return launch_seq(nm, join_segments<D>, (heads * da * dc + 255) / 256 * x.carries, 256, stream, x);
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
    x.carries = 1;
    x.seg_len = plan.seg_len;
    x.segments = (int32_t)plan.segments;
    char* base = static_cast<char*>(ws);
    if (plan.segments > 1) {
        CarryArgs& c = x.carry[0];
        c = CarryArgs{w[1], w[2], reinterpret_cast<float*>(base + plan.states[0]),
                      reinterpret_cast<float*>(base + plan.totals[0]), initial, 1.0f, (int32_t)dk, (int32_t)dv, 0};
        initial = c.states;
    }
    PassArgs& p = x.pass[0];
    p.a = w[0];
    p.b = w[1];
    p.c = w[2];
    p.y = w[5];
    p.init = initial;
    p.last = final_state;
    p.y_scale = scale;
    p.p_scale = 1.0f;
    p.u_scale = 1.0f;
    p.da = (int32_t)dk;
    p.dc = (int32_t)dv;
    LRS_TRY(launch_carries<D>(nm, x, stream));
    set_vec<D>(p);
    const uint64_t blocks = (uint64_t)(N * H * plan.segments);
    return std::max(dk, dv) <= 64 ? launch_seq(nm, recurrence_forward<D, 64>, blocks, 128, stream, x)
                                  : launch_seq(nm, recurrence_forward<D, 128>, blocks, 256, stream, x);
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
        return SeqView{p, T * H * dk, H * dk, dk, 1, 0};
    };
    RecurrenceArgs x{};
    x.g = w[4];
    x.reset = w[5];
    x.N = N;
    x.T = T;
    x.H = (int32_t)H;
    x.carries = 2;
    x.seg_len = plan.seg_len;
    x.segments = (int32_t)plan.segments;
    if (plan.segments > 1) {
        x.carry[0] = CarryArgs{w[2], w[3], reinterpret_cast<float*>(base + plan.states[0]),
                               reinterpret_cast<float*>(base + plan.totals[0]), initial, 1.0f, (int32_t)dk,
                               (int32_t)dv, 0};
        x.carry[1] = CarryArgs{w[1], w[0], reinterpret_cast<float*>(base + plan.states[1]),
                               reinterpret_cast<float*>(base + plan.totals[1]), grad_final, scale, (int32_t)dk,
                               (int32_t)dv, 1};
        initial = x.carry[0].states;
        grad_final = x.carry[1].states;
    }
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
    pq.p_scale = 1.0f;
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
    pk.p_scale = scale;
    pk.u_scale = scale;
    pk.da = (int32_t)dv;
    pk.dc = (int32_t)dk;
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
    pv.p_scale = scale;
    pv.u_scale = scale;
    pv.da = (int32_t)dk;
    pv.dc = (int32_t)dv;
    LRS_TRY(launch_carries<D>(nm, x, stream));
    for (PassArgs& p : x.pass) set_vec<D>(p);
    const uint64_t blocks = (uint64_t)(N * H * plan.segments) * 3;
    LRS_TRY(std::max(dk, dv) <= 64 ? launch_seq(nm, recurrence_backward<D, 64>, blocks, 128, stream, x)
                                   : launch_seq(nm, recurrence_backward<D, 128>, blocks, 256, stream, x));
    DecayGradArgs dg{w[4], w[5], w[9], qdq, kdk, cross, N, T, plan.seg_len, (int32_t)H,
                     (int32_t)plan.segments};
    LRS_TRY(launch_seq(nm, decay_grad<D>, (uint64_t)(N * H * plan.segments), 64, stream, dg));
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
