// recurrence.hpp -- the gated recurrence with a matrix state.  Per environment
// and head, with a state S of [key_dim, value_dim] in fp32:
//
//     S_t = (cut_t ? 0 : e^{g_t} S_{t-1}) + k_t v_t^T,    o_t = scale S_t^T q_t
//
// cut_t where the reset mask is set or g_t is below kLeastLogDecay.  With
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
// k_s . dk_s with all steps from it on; what lies wholly behind t cancels.  The
// product of s with itself is in both: it is left out of both sums, or strong
// decays would leave dg the difference of numbers far larger than itself.
#pragma once

#include <algorithm>

#include "sequence.hpp"

namespace lrs {

constexpr int kMaxDim = 128;  // largest key and value dimension

// ln 2^-126: a decay below the smallest normal float32 is 0 in every kernel, so
// such a step is a cut, -infinity, -1e30 and the types' lowest values alike.  (In
// a running sum of log decays a value of that size would leave nothing of those
// after it.)
constexpr float kLeastLogDecay = -87.33654f;
__device__ __forceinline__ bool cuts(float log_decay) { return log_decay < kLeastLogDecay; }

// One pass over the sequence, in segments of seg_len steps that blocks work on
// side by side.  init: each segment's state before its first step in scan order,
// [N, H, segments, key_dim, value_dim] (nullable for one segment); last: where
// the state after the last segment goes, [N, H, key_dim, value_dim], nullable.
// y_scale multiplies what y has of the state, p_scale what it has of the products
// a . b, u_scale what enters the state.  dot: receives y_i . d_i per [N, H, T],
// without step i's own part of y_i (dq and dk); cross (nullable): <state after the segment, meet> per
// [N, H, segments], meet like init.
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

// Tiles of 16 columns that a wave holds of the state (W: its padded dimension,
// 64 or 128), and the threads of a block.  Two tiles halve the reads of the
// shared fragments per product; one tile leaves room for twice the waves.  bf16
// at W = 128: 32768 steps forward 239 us with two and 282 with one, 8 x 2048
// backward 344 and 489.  f16 at W = 128, which takes one: 16384 steps of 8 heads
// 349 us backward with one and 284 with two, 3 x 1001 forward 41 and 48.  f32's
// three limbs leave no registers for two; W = 64 needs the four waves that one
// tile each gives it, for the four tiles of a b^T.
template <class D, int W>
constexpr int kCols = W == 128 && kLimbs<D> == 1 ? 2 : 1;
template <class D, int W>
constexpr int kThreads = 4 * W / kCols<D, W>;

// Limbs of a b^T and of the state as operands: as many as the inputs have, and
// two at least, which keep 16 bits, so that the rounding of a 16-bit result is
// the only one to be seen in it (with one limb bf16 results were off by 0.0023
// of their size, with two by the 0.0017 of the type).
template <class D>
constexpr int kOperandLimbs = kLimbs<D> > 2 ? kLimbs<D> : 2;

template <int L>
struct Frag {
    bf16x8 x[L];
};

// The limbs of two values, each a packed pair.
template <int L>
__device__ __forceinline__ void split2(float v0, float v1, uint32_t (&w)[L])
{
#pragma unroll
    for (int l = 0; l < L; ++l) {
        w[l] = pack2<bf16_t>(v0, v1);
        if (l + 1 < L) {
            v0 -= __uint_as_float(w[l] << 16);
            v1 -= __uint_as_float(w[l] & 0xffff0000u);
        }
    }
}

template <int L>
__device__ __forceinline__ Frag<L> split(f32x8 v)
{
    u32x4 x[L];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t w[L];
        split2<L>(v[2 * k], v[2 * k + 1], w);
#pragma unroll
        for (int l = 0; l < L; ++l) x[l][k] = w[l];
    }
    Frag<L> f;
#pragma unroll
    for (int l = 0; l < L; ++l) f.x[l] = __builtin_bit_cast(bf16x8, x[l]);
    return f;
}

// The values of a fragment.
template <int L>
__device__ __forceinline__ f32x8 joined(const Frag<L>& f)
{
    f32x8 v;
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const u32x4 w = __builtin_bit_cast(u32x4, f.x[l]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
            v[2 * k] = l == 0 ? lo : v[2 * k] + lo;
            v[2 * k + 1] = l == 0 ? hi : v[2 * k + 1] + hi;
        }
    }
    return v;
}

__device__ __forceinline__ bf16x8 masked(const bf16x8& x, const u32x4& m)
{
    return __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, x) & m);
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

// What a wave holds of the state, and the columns of c that go with it.
template <class D, int W>
using StateTiles = f32x4[W / 16][kCols<D, W>];
template <class D, int W>
using ColumnFrags = Frag<kLimbs<D>>[kCols<D, W>];

// A tile of kChunk steps of up to W elements in LDS, one plane per limb.  The 32
// values that a matrix instruction sums over are taken in order, eight to a
// group of 16 lanes, by both operands.  Rows are an odd number of 16-byte units
// long, and the rows of each 16 are laid out 0, 4, 1, 5, ... and 8 below, so
// that every fragment lies at a constant distance from one address per lane, and
// a fragment by rows (16 rows at one unit) and one by columns (rows 0..3 and
// 8..11 at two neighbouring units, transposed) spread over all banks.  The
// fragments in eights read half of each unit: with them 32% of the cycles that
// LDS is busy in recurrence_forward (bf16, W = 128) are conflicts.
constexpr int kChunk = 32;
constexpr int kTile = 16;

template <int W, int L>
struct StepTile {
    static constexpr int kRow = W + 8;
    alignas(16) uint16_t e[L][kChunk * kRow];

    static __device__ __forceinline__ int at(int row, int col)
    {
        return ((row & ~15) | (row & 8) | ((row & 3) << 1) | ((row >> 2) & 1)) * kRow + col;
    }
    // A fragment of 16 rows (from `row`) over 32 columns (from `col`): lane l
    // holds row l % 16, columns 8 (l / 16) + 0..7.
    __device__ __forceinline__ Frag<L> rows(int row, int col, int lane) const
    {
        const int mine = at(lane & 15, (lane >> 4) * 8), to = row * kRow + col;
        Frag<L> f;
#pragma unroll
        for (int l = 0; l < L; ++l) f.x[l] = *reinterpret_cast<const bf16x8*>(&e[l][mine + to]);
        return f;
    }
    // The four values of a row from `at` on.
    __device__ __forceinline__ f32x4 four(int at) const
    {
        f32x4 v;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(&e[l][at]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
                v[2 * k] = l == 0 ? lo : v[2 * k] + lo;
                v[2 * k + 1] = l == 0 ? hi : v[2 * k + 1] + hi;
            }
        }
        return v;
    }
    // The transposed fragment over the 32 rows from `row`: lane l holds rows
    // 8 (l / 16) + 0..7 of column col + l % 16, or, kEights, of column
    // col + 8 (l % 16 / 4) + l % 4 (with col and col + 4 a pair that covers 32
    // columns in eights).  A transposing read hands the 16 lanes of a group
    // four rows of four groups of 4 columns, 8 bytes read by each lane.
    template <bool kEights = false>
    __device__ __forceinline__ Frag<L> columns(int row, int col, int lane) const
    {
        const int mine = at((lane >> 4) * 8 + ((lane & 15) >> 2), (lane & 3) * (kEights ? 8 : 4));
        const int to = row * kRow + col, four = at(4, 0);
        Frag<L> f;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)&e[l][mine + to]);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)&e[l][mine + to + four]);
            f.x[l] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
};

// The rows of the state that a wave holds in tile k: four from here on.
__device__ __forceinline__ int state_row(int k, int group) { return (k >> 1) * 32 + group * 8 + (k & 1) * 4; }

template <class D, int W>
__device__ __forceinline__ void put8(StepTile<W, kLimbs<D>>& tile, int at, const Raw8<D>& v)
{
    if constexpr (kLimbs<D> == 1) {
        *reinterpret_cast<u32x4*>(&tile.e[0][at]) = v.w[0];
    } else {
        f32x8 e;
        if constexpr (sizeof(D) == 4) {
            e = __builtin_bit_cast(f32x8, v);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                unpack2<D>(v.w[0][k], lo, hi);
                e[2 * k] = lo;
                e[2 * k + 1] = hi;
            }
        }
        const Frag<kLimbs<D>> f = split<kLimbs<D>>(e);
#pragma unroll
        for (int l = 0; l < kLimbs<D>; ++l) *reinterpret_cast<bf16x8*>(&tile.e[l][at]) = f.x[l];
    }
}

// Waits for this wave's loads.  put() needs them anyway, but by lanes, and where
// a branch may skip it the compiler counts them as still under way: it would wait
// before the registers' next loads, and by then for the stores in between too.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// One head's steps of an array, from the first of a segment on.
template <class D>
struct Rows {
    D* p;
    int64_t step;
    int32_t dim, vec;

    __device__ __forceinline__ Rows(const SeqView& v, int64_t n, int64_t t, int h, int dim)
        : p(seq_row_out<D>(v, n, t, h)), step(v.step), dim(dim), vec(v.vec)
    {
    }
};

// A block moves a chunk of one head's array into a tile in two halves: fetch()
// starts the loads (of a thread's 16-byte units), put() writes what arrived to
// LDS, zero beyond dim.  Steps beyond `count` read the last one again: their
// weights are zero.  kWide: every row is
// on 16 bytes and dim a multiple of 8, and a chunk lies within 2 GiB, so that
// one 32-bit offset per lane and access is all the addressing there is; nothing
// then branches around the loads, which would make the wave wait for them where
// the branches join.
template <class D, int W, bool kWide>
struct Staged {
    static constexpr int kApart = kThreads<D, W> / (W / 8), kUnits = kChunk / kApart;
    Raw8<D> r[kUnits];

    __device__ __forceinline__ void fetch(const Rows<D>& rows, int64_t t, int count)
    {
        const int row = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8) * 8;
        const D* const from = rows.p + t * rows.step;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int at_row = min(row + kApart * k, count - 1);
            if constexpr (kWide) {
                const uint32_t at = (uint32_t)at_row * (uint32_t)rows.step + (c < rows.dim ? c : 0);
#pragma unroll
                for (int j = 0; j < (int)sizeof(D) / 2; ++j)
                    r[k].w[j] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(from) +
                                                                (at * (uint32_t)sizeof(D) + 16u * j));
            } else {
                r[k] = Raw8<D>{};
                if (c < rows.dim) r[k] = load8(from + at_row * rows.step, c, rows.dim, rows.vec);
            }
        }
    }
    __device__ __forceinline__ void put(StepTile<W, kLimbs<D>>& tile, const Rows<D>& rows) const
    {
        const int row = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8) * 8;
        if (!kWide || c < rows.dim)
#pragma unroll
            for (int k = 0; k < kUnits; ++k) put8<D, W>(tile, tile.at(row, c) + kApart * k * tile.kRow, r[k]);
    }
    // The columns beyond dim, once: put() leaves them alone where kWide.
    static __device__ __forceinline__ void clear(StepTile<W, kLimbs<D>>& tile, const Rows<D>& rows)
    {
        const int row = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8) * 8;
        if (kWide && c >= rows.dim)
#pragma unroll
            for (int k = 0; k < kUnits; ++k)
                put8<D, W>(tile, tile.at(row, c) + kApart * k * tile.kRow, Raw8<D>{});
    }
};

// A chunk's results on their way from the accumulators to memory by whole rows:
// put() leaves a wave's part in LDS, 16-bit values in one plane of a tile, fp32
// ones by halves in two; take() reads what the thread itself will overwrite by
// its next Staged::put(), and store() writes it out.  Stores go out before the
// next loads start: the wait for the loads would otherwise be one for the
// stores as well, which are slower to be acknowledged (a pass of 32768 steps of
// 16 heads took a quarter longer where they came between).  move(), for the
// partial gradients of shared heads in 16-bit types, stores right before that
// wait all the same: its fp32 rows are twice what the registers would hold.
template <class D, int W, bool kWide>
struct Result {
    static constexpr int kUnits = Staged<D, W, kWide>::kUnits, kApart = Staged<D, W, kWide>::kApart;
    using Tile = StepTile<W, kLimbs<D>>;
    u32x4 lo[kUnits], hi[sizeof(D) == 4 ? kUnits : 1];

    static __device__ __forceinline__ void put(uint16_t* low, uint16_t* high, int at, f32x4 v, bool f32)
    {
        if (f32) {
            const uint32_t w[4] = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                   __float_as_uint(v[3])};
            *reinterpret_cast<u32x2*>(&low[at]) = u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x05040100),
                                                        __builtin_amdgcn_perm(w[3], w[2], 0x05040100)};
            *reinterpret_cast<u32x2*>(&high[at]) = u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x07060302),
                                                         __builtin_amdgcn_perm(w[3], w[2], 0x07060302)};
        } else if constexpr (sizeof(D) == 2) {
            *reinterpret_cast<u32x2*>(&low[at]) = u32x2{pack2<D>(v[0], v[1]), pack2<D>(v[2], v[3])};
        }
    }
    // Elements c .. c + 7 of a row of `dim` from w.
    template <class E>
    static __device__ __forceinline__ void store8(char* to, const Raw8<E>& v, int c, int dim, int vec)
    {
        to += c * (int)sizeof(E);
        if (kWide || (vec == 16 && c + 8 <= dim)) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(E) / 2; ++j) reinterpret_cast<u32x4*>(to)[j] = v.w[j];
        } else if (sizeof(E) == 4 || vec >= 4) {
            constexpr int per = 4 / sizeof(E);
#pragma unroll
            for (int j = 0; j < 8 / per; ++j)
                if (c + per * j < dim) reinterpret_cast<uint32_t*>(to)[j] = v.w[j / 4][j % 4];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < dim)
                    reinterpret_cast<uint16_t*>(to)[j] = (uint16_t)(v.w[0][j / 2] >> (16 * (j & 1)));
        }
    }
    __device__ __forceinline__ void take(const uint16_t* low, const uint16_t* high)
    {
        const int at = Tile::at(threadIdx.x / (W / 8), threadIdx.x % (W / 8) * 8);
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            lo[k] = *reinterpret_cast<const u32x4*>(&low[at + kApart * k * Tile::kRow]);
            if constexpr (sizeof(D) == 4) hi[k] = *reinterpret_cast<const u32x4*>(&high[at + kApart * k * Tile::kRow]);
        }
    }
    __device__ __forceinline__ void store(char* y, int64_t step, int count, int dim, int vec) const
    {
        const int row = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8) * 8;
        if (c >= dim) return;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int at = row + kApart * k;
            if (at >= count) continue;
            char* const to = kWide ? y + (uint32_t)at * (uint32_t)step : y + at * step;
            if constexpr (sizeof(D) == 4) store8<float>(to, both(lo[k], hi[k]), c, dim, vec);
            else store8<D>(to, Raw8<D>{{lo[k]}}, c, dim, vec);
        }
    }
    // take() and store() of fp32 results where D is not fp32, in one.
    static __device__ __forceinline__ void move(const uint16_t* low, const uint16_t* high, char* y, int64_t step,
                                                int count, int dim, int vec)
    {
        const int row = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8) * 8;
        const int at = Tile::at(row, c);
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const u32x4 l = *reinterpret_cast<const u32x4*>(&low[at + kApart * k * Tile::kRow]);
            const u32x4 h = *reinterpret_cast<const u32x4*>(&high[at + kApart * k * Tile::kRow]);
            if (c < dim && row + kApart * k < count)
                store8<float>(kWide ? y + (uint32_t)(row + kApart * k) * (uint32_t)step
                                    : y + (row + kApart * k) * step,
                              both(l, h), c, dim, vec);
        }
    }
    static __device__ __forceinline__ Raw8<float> both(const u32x4& l, const u32x4& h)
    {
        Raw8<float> v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v.w[j / 2][j % 2 * 2] = __builtin_amdgcn_perm(h[j], l[j], 0x05040100);
            v.w[j / 2][j % 2 * 2 + 1] = __builtin_amdgcn_perm(h[j], l[j], 0x07060302);
        }
        return v;
    }
};

// The decays of a chunk of 32 steps, in two tiles of 16.  With p the running
// sum of log2 decays within a tile (in 64 bits: a decay of 2^-126 before a weak
// one would cost an fp32 sum the weak one's digits), started again at each cut,
// and m the running count of its cuts, for steps j < i of one tile D(i, j) =
// 2^(p_i - p_j) where m_i = m_j, and for steps of the second and the first tile
// D(i, j) = head_i tail_j, where each factor is at most 1 for log decays up to 0.
// A decay that is not finite, or growth that overflows, thus stays between the
// cuts around it; what crosses a cut is 0 by choice, not as a factor of 0.
struct ChunkDecay {
    double p[kChunk];
    int m[kChunk];
    float head[kChunk];   // from the start of its tile to this step, inclusive
    float tail[kChunk];   // from this step, exclusive, to the end of its tile
    float entry[kChunk];  // from the start of the chunk, inclusive
    float exit[kChunk];   // to the end of the chunk
    float total;          // of the chunk

    // total, known to be the same in all lanes
    __device__ __forceinline__ float whole() const
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, total)));
    }
};

// The log decay and the reset mask of a lane's step, as they are stored, loaded
// like the steps themselves.
template <class D>
struct DecayRows {
    const D* g;
    const uint8_t* reset;
    int64_t g_step, reset_step;
    bool resets;
    D next_g;
    uint8_t next_reset;

    __device__ __forceinline__ DecayRows(const RecurrenceArgs& x, int64_t n, int64_t t, int h)
        : g(seq_row<D>(x.g, n, t, h)), g_step(x.g.step), resets(x.reset.p != nullptr)
    {
        reset = resets ? seq_row<uint8_t>(x.reset, n, t, 0) : reinterpret_cast<const uint8_t*>(g);
        reset_step = resets ? x.reset.step : 0;
    }
    __device__ __forceinline__ void fetch(int64_t t, int count, int lane)
    {
        t += min(lane, count - 1);
        next_g = g[t * g_step];
        next_reset = reset[t * reset_step];
    }
    // -infinity where the step is cut
    __device__ __forceinline__ float value() const
    {
        return resets && next_reset != 0 ? -INFINITY : to_f32(next_g);
    }
};

// The value of the lane kShift below in the row of 16 lanes, `none` where there
// is none (a register move: the reads of a shuffle through LDS would be a chunk's
// longest chain).
template <int kShift>
__device__ __forceinline__ int row_below(int v, int none)
{
    return __builtin_amdgcn_update_dpp(none, v, 0x110 + kShift, 0xf, 0xf, false);
}
// One step of the scan: p over the steps up to this one from the last cut on (m
// counts those of the steps taken in so far), m over all of them.
template <int kShift>
__device__ __forceinline__ void row_scan(double& p, int& m)
{
    const uint64_t bits = __builtin_bit_cast(uint64_t, p);
    const uint32_t lo = row_below<kShift>((int)(uint32_t)bits, 0), hi = row_below<kShift>((int)(bits >> 32), 0);
    const double below = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    p += m ? 0.0 : below;
    m += row_below<kShift>(m, 0);
}

__device__ __forceinline__ void chunk_decay(ChunkDecay& s, float g, int count, int lane)
{
    const bool in = lane < count;
    int m = in && cuts(g);
    double p = m || !in ? 0.0 : (double)g * 1.4426950408889634;
    static_assert(kTile == 16, "rows of 16 lanes");
    row_scan<1>(p, m);
    row_scan<2>(p, m);
    row_scan<4>(p, m);
    row_scan<8>(p, m);
    const bool second = lane >= kTile;
    const uint64_t bits = __builtin_bit_cast(uint64_t, p);
    double ptot[2];
    int mtot[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int end = k * kTile + kTile - 1;
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)bits, end);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(bits >> 32), end);
        ptot[k] = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
        mtot[k] = __builtin_amdgcn_readlane(m, end);
    }
    // 2^e, 0 across a cut and of steps beyond the end
    const auto decay = [](bool whole, double e) { return whole ? __builtin_amdgcn_exp2f((float)e) : 0.0f; };
    const double left = (second ? ptot[1] : ptot[0]) - p;
    const bool headed = in && m == 0, tailed = in && m == (second ? mtot[1] : mtot[0]);
    if (lane < kChunk) {
        s.p[lane] = p;
        s.m[lane] = in ? m : -1;  // steps beyond the end have no part in anything
        s.head[lane] = decay(headed, p);
        s.tail[lane] = decay(tailed, left);
        s.entry[lane] = decay(headed && !(second && mtot[0]), second ? ptot[0] + p : p);
        s.exit[lane] = decay(tailed && !(!second && mtot[1]), second ? left : left + ptot[1]);
    }
    if (lane == 0) s.total = decay(!mtot[0] && !mtot[1], ptot[0] + ptot[1]);
}

// S = total S + b^T (w c) over a chunk; w: the weight of each step,
// fc: the wave's columns of c.  The weighted c is fp32 and keeps its 24 bits in
// three limbs, so that S is what fp32 sums make it (in bf16 two would save 3% of
// 8 x 2048 training, 481 us and 468).
constexpr int kStateLimbs = 3;

// total = 0: something in the chunk is cut, which drops the state and the steps
// before the cut, whatever they hold.  Where that leaves something that is not
// finite (0 times infinity or NaN is NaN) they are taken out of the products.
template <class D, int W>
__device__ __forceinline__ void add_chunk(StateTiles<D, W>& S, const StepTile<W, kLimbs<D>>& tb,
                                          const ColumnFrags<D, W>& fc, const float* w, float total,
                                          float scale, int da, int lane)
{
    constexpr int L = kLimbs<D>, U = kCols<D, W>, LW = kStateLimbs;
    const int group = lane >> 4;
    Frag<LW> fw[U];
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&w[group * 8]);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&w[group * 8 + 4]);
    const f32x8 w8 = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7) * scale;
#pragma unroll
    for (int u = 0; u < U; ++u) fw[u] = split<LW>(joined<L>(fc[u]) * w8);
    if (total == 0.0f)
#pragma unroll
        for (int k = 0; k < W / 16; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) S[k][u] = f32x4{};
#pragma unroll
    for (int k = 0; k < W / 16; ++k) {
        if (state_row(k, 0) >= da) break;  // (da: W where the whole width is to be unrolled)
        const Frag<L> fb = tb.template columns<true>(0, state_row(k, 0), lane);
#pragma unroll
        for (int u = 0; u < U; ++u) S[k][u] = mma(fb, fw[u], S[k][u] * total);
    }
    if (total != 0.0f) return;
    f32x4 sum = {};
#pragma unroll
    for (int k = 0; k < W / 16; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u) sum += S[k][u] * 0.0f;
    if (!__any((sum[0] + sum[1]) + (sum[2] + sum[3]) != 0.0f)) return;
    u32x4 kept;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        kept[k] = (w[group * 8 + 2 * k] != 0.0f ? 0xffffu : 0u) |
                  (w[group * 8 + 2 * k + 1] != 0.0f ? 0xffff0000u : 0u);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int l = 0; l < LW; ++l) fw[u].x[l] = masked(fw[u].x[l], kept);
#pragma unroll
    for (int k = 0; k < W / 16; ++k) {
        Frag<L> fb = tb.template columns<true>(0, state_row(k, 0), lane);
#pragma unroll
        for (int l = 0; l < L; ++l) fb.x[l] = masked(fb.x[l], kept);
#pragma unroll
        for (int u = 0; u < U; ++u) S[k][u] = mma(fb, fw[u], f32x4{});
    }
}

// A step whose c is not finite reaches the results of the steps that it has a
// weight in, as NaN, and no others: a product with a weight of 0 would be NaN
// too.  Which tells whether a wave's columns hold one: their product with zeros.
// Of a chunk of finite steps this is all that is done, early enough for the
// branch on it not to wait (256 x 128 f32, both directions: 1% longer than without,
// 15% with the branch right behind the product).
template <class D, int W>
__device__ __forceinline__ f32x4 times_zero(const StepTile<W, kLimbs<D>>& tc, int c0, int lane)
{
    f32x4 sum = {};
#pragma unroll
    for (int u = 0; u < kCols<D, W>; ++u)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tc.columns(0, c0 + u * 16, lane).x[0], bf16x8{}, sum, 0, 0, 0);
    return sum;
}

// The halves of a fragment that hold something from `least` on, all bits set.
__device__ __forceinline__ u32x4 halves_from(const bf16x8& x, uint32_t least)
{
    const u32x4 w = __builtin_bit_cast(u32x4, x) & 0x7fff7fffu;
    u32x4 m;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        m[k] = ((w[k] & 0xffffu) >= least ? 0xffffu : 0u) | ((w[k] >> 16) >= least ? 0xffff0000u : 0u);
    return m;
}

// Takes what is not finite out of c, and puts NaN in the results (and into
// `lost`, of the wave's columns of the state) that it has a part in: those where
// the product of the one place and the other's weight, both as 0 or 1, sums to
// more than 0.
template <class D, int W, int LS>
__device__ __forceinline__ void part_nonfinite(ColumnFrags<D, W>& fc, const StepTile<kChunk, LS>& ab,
                                               const float* w, f32x4 (&y)[2][kCols<D, W>],
                                               bool (&lost)[kCols<D, W>], int lane)
{
    constexpr int L = kLimbs<D>, U = kCols<D, W>;
    const int group = lane >> 4;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const u32x4 bad = halves_from(fc[u].x[0], 0x7f80u);
#pragma unroll
        for (int l = 0; l < L; ++l) fc[u].x[l] = masked(fc[u].x[l], ~bad);
        const Frag<1> place = {{__builtin_bit_cast(bf16x8, bad & 0x3f803f80u)}};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const u32x4 some = halves_from(ab.rows(q * 16, 0, lane).x[0], 1u);
            const Frag<1> weight = {{__builtin_bit_cast(bf16x8, some & 0x3f803f80u)}};
            const f32x4 hits = mma(place, weight, f32x4{});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (hits[r] != 0.0f) y[q][u][r] = __builtin_nanf("");
        }
        int hit = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            hit |= (bad[k / 2] >> (16 * (k & 1)) & 1) != 0 && w[group * 8 + k] != 0.0f;
        hit |= __shfl_xor(hit, 16);
        hit |= __shfl_xor(hit, 32);
        lost[u] = hit != 0;
    }
}

// A pass by matrix instructions, 32 steps at a time.  A wave holds 16 or 32 columns
// of the state, all its rows, in accumulators; the block's waves share the
// steps, and the products a b^T of which each computes its part, in LDS.  Per
// chunk, with X, Z the weights from the chunk's start and to its end in scan
// order:
//     y^T = S^T a^T X + c^T (D o (a b^T))^T        (S before the chunk)
//     S   = total S + b^T (Z c)
// Results of a product leave the matrix unit with 4 consecutive rows of one of
// 16 columns per lane; a wave's tiles of S take their rows in fours of every 8,
// so that two of them are an operand and S feeds the next product from the
// registers that it is kept in.
//
// What bounds it: a step of the chain.  The state's registers leave two waves
// per SIMD at W = 128, and a chunk is a chain of LDS reads, products, weights,
// a barrier, products again: of 32768 steps of 16 heads of 128 x 128 in bf16
// (172 us traced; 34 GFLOP with the segments' states) the vector unit is issued to
// in 42% of the cycles, LDS is busy for 33%, the matrix unit for 28%, and no two
// of them much at once.  Chunks of 32 steps rather than 64: the longer
// ones do half the barriers, but their operands spill.  A second set of LDS
// tiles, which saves one of the three barriers, measured 10% slower, three waves
// per SIMD by smaller register budgets 17%.
template <class D, int W>
struct PassShared {
    StepTile<W, kLimbs<D>> a, b, c;
    StepTile<kChunk, kOperandLimbs<D>> ab;
    ChunkDecay decays[2];  // this chunk's, and the next one's as it is made
    float own[kChunk];  // where dots are wanted: a_i . b_i, which ab then lacks
    float dot[W / 16][kChunk];
    float cross[W / 16];
};

// Four elements of a row from column c on, out of `dim`.
template <class D>
struct alignas(4 * sizeof(D)) Raw4 {
    uint32_t w[sizeof(D)];
};
template <class D>
__device__ __forceinline__ Raw4<D> load4(const D* row, int c, int dim, bool vec)
{
    Raw4<D> v = {};
    if (vec) {
        v = *reinterpret_cast<const Raw4<D>*>(row + (c < dim ? c : 0));
        if (c >= dim) v = Raw4<D>{};
    } else if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (c + r < dim) v.w[r] = __float_as_uint(row[c + r]);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (c + r < dim) v.w[r / 2] |= (uint32_t)row[c + r].bits << (16 * (r & 1));
    }
    return v;
}
template <class D>
__device__ __forceinline__ f32x4 unpack4(const Raw4<D>& v)
{
    f32x4 f;
    if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) f[r] = __uint_as_float(v.w[r]);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float lo, hi;
            unpack2<D>(v.w[k], lo, hi);
            f[2 * k] = lo;
            f[2 * k + 1] = hi;
        }
    }
    return f;
}

template <class D, int W, bool kWide, bool back, bool kPrecise>
__device__ __forceinline__ void run_pass(const RecurrenceArgs& x, const PassArgs& p, uint32_t block,
                                         PassShared<D, W>& sh)
{
    constexpr int L = kLimbs<D>, LS = kOperandLimbs<D>;
    constexpr int K = W / 32, U = kCols<D, W>, kWaves = W / 16 / U;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int group = lane >> 4, col = lane & 15;
    const int64_t head = block / x.segments;
    const int seg = (int)(block % x.segments);
    const int64_t n = head / x.H;
    const int h = (int)(head % x.H);
    const int c0 = wave * 16 * kCols<D, W>;
    const int64_t at = (int64_t)block * p.da * p.dc;
    const int64_t first = seg * x.seg_len;
    const int64_t steps = x.T - first < x.seg_len ? x.T - first : x.seg_len;
    const int chunks = (int)((steps + kChunk - 1) / kChunk);

    const Rows<D> ra(p.a, n, first, h, p.da), rb(p.b, n, first, h, p.da), rc(p.c, n, first, h, p.dc);
    const Rows<D> rd(kPrecise ? p.d : p.c, n, first, h, p.dc);
    DecayRows<D> decays(x, n, first, h);
    // (partial gradients of shared heads are fp32)
    const bool y_f32 = kPrecise && p.y_f32;
    const int y_bytes = y_f32 ? 4 : (int)sizeof(D);
    char* const y_base = y_f32 ? reinterpret_cast<char*>(seq_row_out<float>(p.y, n, first, h))
                               : reinterpret_cast<char*>(seq_row_out<D>(p.y, n, first, h));
    const int64_t y_step = p.y.step * y_bytes;
    // where results wait in LDS: a wave's own columns of c, and for the high halves of fp32 ones
    // a second plane, or a where there is none (a is not read any more then)
    uint16_t* const low = sh.c.e[0];
    uint16_t* const high = L > 1 ? sh.c.e[L > 1 ? 1 : 0] : sh.a.e[0];
    const bool f32 = sizeof(D) == 4 || y_f32;
    Staged<D, W, kWide> ga, gb, gc;
    const auto fetch = [&](int i) {
        const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        const int count = (int)(steps - done < kChunk ? steps - done : kChunk);
        ga.fetch(ra, done, count);
        gb.fetch(rb, done, count);
        gc.fetch(rc, done, count);
    };
    // the decays are loaded two chunks ahead, and made ready one ahead
    const auto fetch_decay = [&](int i) {
        const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        decays.fetch(done, (int)(steps - done < kChunk ? steps - done : kChunk), lane);
    };
    const auto make_decay = [&](int i) {
        const int64_t left = steps - (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        chunk_decay(sh.decays[i & 1], decays.value(), (int)(left < kChunk ? left : kChunk), lane);
    };
    fetch_decay(0);
    fetch(0);
    Staged<D, W, kWide>::clear(sh.a, ra);
    Staged<D, W, kWide>::clear(sh.b, rb);
    Staged<D, W, kWide>::clear(sh.c, rc);
    if (wave == 0) make_decay(0);
    if (chunks > 1) fetch_decay(1);

    // S[k][u][r]: row state_row(k) + r, column c0 + 16 u + col;
    StateTiles<D, W> S;
#pragma unroll
    for (int k = 0; k < 2 * K; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(k, group) + r, c = c0 + u * 16 + col;
                S[k][u][r] = p.init && row < p.da && c < p.dc ? p.init[at + state_at(p, row, c)] : 0.0f;
            }

    Result<D, W, kWide> result;
    // what chunk i left in LDS: results, and the waves' parts of the dot products
    const auto finish = [&](int i) {
        const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        const int count = (int)(steps - done < kChunk ? steps - done : kChunk);
        if (sizeof(D) == 4 || !y_f32) result.store(y_base + done * y_step, y_step, count, p.dc, p.y.vec);
        if (kPrecise && wave == 0 && lane < count) {
            float sum = 0.0f;
            for (int w = 0; w * 16 * U < p.dc; ++w) sum += sh.dot[w][lane];
            p.dot[head * x.T + first + done + lane] = sum;
        }
    };
    const auto take = [&](int i) {
        if (sizeof(D) == 4 || !y_f32) {
            result.take(low, high);
        } else {
            const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
            Result<D, W, kWide>::move(low, high, y_base + done * y_step, y_step,
                                      (int)(steps - done < kChunk ? steps - done : kChunk), p.dc, p.y.vec);
            Staged<D, W, kWide>::clear(sh.a, ra);
        }
    };
    for (int i = 0; i < chunks; ++i) {
        const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        const int count = (int)(steps - done < kChunk ? steps - done : kChunk);
        if (i > 0) take(i - 1);
        wait_loads();
        ga.put(sh.a, ra);
        gb.put(sh.b, rb);
        gc.put(sh.c, rc);
        __syncthreads();
        if (i > 0) finish(i - 1);
        const ChunkDecay& decay = sh.decays[i & 1];
        Raw4<D> d[2][U];
        if constexpr (kPrecise)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int step = min(q * 16 + col, count - 1);
                const D* const row = kWide ? rd.p + done * rd.step + (uint32_t)step * (uint32_t)rd.step
                                           : rd.p + (done + step) * rd.step;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    d[q][u] = load4<D>(row, c0 + u * 16 + group * 4, p.dc, kWide || rd.vec != 0);
            }
        if (i + 1 < chunks) {
            fetch(i + 1);
            // by the wave whose tile below is zero
            if (wave == (back ? 1 : 2)) make_decay(i + 1);
            if (i + 2 < chunks) fetch_decay(i + 2);
        }

        // a tile of a b^T for each of four waves: rows (steps of b) 16 s0 + 4 group + r, columns
        // (steps of a) 16 q0 + col.  One of them lies on the side of the diagonal that is zero; it
        // is computed too, since branches around products make a wave wait for each read of LDS.
        const int q0 = wave & 1, s0 = (wave >> 1) & 1;
        const f32x4 zeros = times_zero<D, W>(sh.c, c0, lane);
        f32x4 ab = {};
        // y^T of tile q: rows c0 + 16 u + 4 group + r, column (step) 16 q + col
        f32x4 y[2][U];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int u = 0; u < U; ++u) y[q][u] = f32x4{};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!kWide && k * 32 >= p.da) break;
            if (kWaves == 4 || wave < 4)
                ab = mma(sh.b.rows(s0 * 16, k * 32, lane), sh.a.rows(q0 * 16, k * 32, lane), ab);
            Frag<LS> s[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                s[u] = split<LS>(__builtin_shufflevector(S[2 * k][u], S[2 * k + 1][u], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const Frag<L> f = sh.a.rows(q * 16, k * 32, lane);
#pragma unroll
                for (int u = 0; u < U; ++u) y[q][u] = mma(s[u], f, y[q][u]);
            }
        }
        if (kWaves == 4 || wave < 4) {
            const int step = q0 * 16 + col, o = s0 * 16 + group * 4;
            if (s0 == q0) {
                const double pi = decay.p[step];
                const int mi = decay.m[step];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = (float)(back ? decay.p[o + r] - pi : pi - decay.p[o + r]);
                    const bool in = (back ? o + r >= step : o + r <= step) && decay.m[o + r] == mi;
                    // (both factors chosen: ab may be NaN)
                    ab[r] = (in ? ab[r] : 0.0f) * (__builtin_amdgcn_exp2f(in ? d : 0.0f) * p.p_scale);
                    if (kPrecise && o + r == step) {
                        sh.own[step] = ab[r];
                        ab[r] = 0.0f;
                    }
                }
            } else {
                const bool in_order = back ? s0 > q0 : s0 < q0;
                const float mine = in_order ? (back ? decay.tail : decay.head)[step] : 0.0f;
                const f32x4 w = *reinterpret_cast<const f32x4*>(&(back ? decay.head : decay.tail)[o]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float f = w[r] * (mine * p.p_scale);
                    ab[r] = mine == 0.0f || w[r] == 0.0f || f == 0.0f ? 0.0f : ab[r] * f;
                }
            }
            const int here = sh.ab.at(col, group * 4) + q0 * 16 * sh.ab.kRow + s0 * 16;
            uint32_t lo[LS], hi[LS];
            split2<LS>(ab[0], ab[1], lo);
            split2<LS>(ab[2], ab[3], hi);
#pragma unroll
            for (int l = 0; l < LS; ++l) *reinterpret_cast<u32x2*>(&sh.ab.e[l][here]) = u32x2{lo[l], hi[l]};
        }
        const bool nonfinite = __any((zeros[0] + zeros[1]) + (zeros[2] + zeros[3]) != 0.0f);
        __syncthreads();

        if (kWide || c0 < p.dc) {
            ColumnFrags<D, W> fc;  // columns c0 + 16 u + l % 16
#pragma unroll
            for (int u = 0; u < U; ++u) fc[u] = sh.c.columns(0, c0 + u * 16, lane);
            const float* const from = back ? decay.exit : decay.entry;
            const float total = decay.whole();
            if (total == 0.0f)  // nothing of the state passes a cut, whatever it holds
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (from[q * 16 + col] == 0.0f) y[q][u] = f32x4{};
            bool lost[U];
            if (__builtin_expect(nonfinite, 0))
                part_nonfinite<D, W, LS>(fc, sh.ab, back ? decay.entry : decay.exit, y, lost, lane);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int step = q * 16 + col;
                const float in = from[step] * p.y_scale;
                const Frag<LS> f = sh.ab.rows(q * 16, 0, lane);
                const float own = kPrecise ? sh.own[step] : 0.0f;
                float dot = 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    f32x4 v = mma(fc[u], f, y[q][u] * in);
                    // Columns beyond dim are 0, unless a holds something that is not finite: 0 times that.
                    // Where kWide they are written by no one else, so such a result would stay in the tile,
                    // as c of later chunks.
                    const int c = c0 + u * 16 + group * 4;
                    if (kWide && c >= p.dc) continue;
                    const int here = sh.c.at(col, c) + q * 16 * sh.c.kRow;
                    if constexpr (kPrecise) {
                        const f32x4 e = unpack4<D>(d[q][u]) * v;
                        dot += (e[0] + e[1]) + (e[2] + e[3]);
                        v += sh.c.four(here) * own;
                    }
                    Result<D, W, kWide>::put(low, high, here, v, f32);
                }
                if constexpr (kPrecise) {
                    dot += __shfl_xor(dot, 16);
                    dot += __shfl_xor(dot, 32);
                    if (group == 0) sh.dot[wave][step] = dot;
                }
            }
            // the state after the chunk
            add_chunk<D, W>(S, sh.b, fc, back ? decay.entry : decay.exit, total, p.u_scale,
                                kWide ? W : p.da, lane);
            if (__builtin_expect(nonfinite, 0))
#pragma unroll
                for (int k = 0; k < 2 * K; ++k)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (lost[u]) S[k][u] = f32x4{} + __builtin_nanf("");
        }
        __syncthreads();
    }
    take(chunks - 1);
    finish(chunks - 1);

    if (p.last == nullptr && p.cross == nullptr) return;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 2 * K; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(k, group) + r, c = c0 + u * 16 + col;
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
            for (int w = 0; w < kWaves; ++w) sum += sh.cross[w];
            p.cross[block] = sum;
        }
    }
}

// Waves per SIMD that leave enough registers for nothing to spill: a reload in
// the loop waits for every load before it, the next chunk's among them.  (The
// backward kernels of 16-bit types at W = 64 spill some all the same, as did those
// of f32 at three waves where not kWide; 256 x 128 f32 training 203 us at two
// waves, 178 at three.)
template <class D, int W, bool kWide>
constexpr int kPassWaves = W == 128 || (kLimbs<D> == 3 && !kWide) ? 2 : kLimbs<D> == 3 ? 3 : 4;

template <class D, int W, bool kWide>
__global__ __launch_bounds__((kThreads<D, W>), (kPassWaves<D, W, kWide>)) void recurrence_forward(const RecurrenceArgs x)
{
    __shared__ PassShared<D, W> sh;
    run_pass<D, W, kWide, false, false>(x, x.pass[0], blockIdx.x, sh);
}

// The three passes of the backward call: dq and dk with q.dq and k.dk to a
// precision that their differences keep, and dv.  Blocks of the three passes of
// a segment are neighbours: they read the same steps, mostly from L2.  8 x 2048
// steps of 16 heads of 128 x 128 in bf16: 343 us, bound like the forward pass;
// 256 x 128 of 4 heads of 64 x 64 in f32: 137 us.
template <class D, int W, bool kWide>
__global__ __launch_bounds__((kThreads<D, W>), (kPassWaves<D, W, kWide>)) void recurrence_backward(const RecurrenceArgs x)
{
    __shared__ PassShared<D, W> sh;
    const uint32_t block = blockIdx.x / 3, pass = blockIdx.x % 3;
    if (pass == 0) run_pass<D, W, kWide, false, true>(x, x.pass[0], block, sh);
    else if (pass == 1) run_pass<D, W, kWide, true, true>(x, x.pass[1], block, sh);
    else run_pass<D, W, kWide, true, false>(x, x.pass[2], block, sh);
}

// The state that one segment alone leaves (from zero), and its decay, by the
// same products; the last segment in scan order leaves none that is used.
// 32768 steps of 16 heads of 128 x 128 in bf16, 32 segments: 80 us, that is 2.5
// us per chunk of each block: the loads' way to LDS and two barriers.  Two
// chunks between barriers measured the same.
template <class D, int W, bool kWide>
__global__ __launch_bounds__((kThreads<D, W>), (kPassWaves<D, W, kWide>)) void segment_states(const RecurrenceArgs x)
{
    __shared__ struct {
        StepTile<W, kLimbs<D>> b, c;
        ChunkDecay decays[2];
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
    const int c0 = wave * 16 * kCols<D, W>;
    const int64_t first = seg * x.seg_len;
    const int64_t steps = x.T - first < x.seg_len ? x.T - first : x.seg_len;
    constexpr int U = kCols<D, W>;
    StateTiles<D, W> S = {};
    float total = 1.0f;
    const int chunks = (int)((steps + kChunk - 1) / kChunk);
    const Rows<D> rb(p.b, n, first, h, p.da), rc(p.c, n, first, h, p.dc);
    DecayRows<D> decays(x, n, first, h);
    Staged<D, W, kWide> gb, gc;
    const auto fetch = [&](int i) {
        const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        const int count = (int)(steps - done < kChunk ? steps - done : kChunk);
        gb.fetch(rb, done, count);
        gc.fetch(rc, done, count);
    };
    const auto fetch_decay = [&](int i) {
        const int64_t done = (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        decays.fetch(done, (int)(steps - done < kChunk ? steps - done : kChunk), lane);
    };
    const auto make_decay = [&](int i) {
        const int64_t left = steps - (int64_t)(back ? chunks - 1 - i : i) * kChunk;
        chunk_decay(sh.decays[i & 1], decays.value(), (int)(left < kChunk ? left : kChunk), lane);
    };
    fetch_decay(0);
    fetch(0);
    Staged<D, W, kWide>::clear(sh.b, rb);
    Staged<D, W, kWide>::clear(sh.c, rc);
    if (wave == 0) make_decay(0);
    if (chunks > 1) fetch_decay(1);
    for (int i = 0; i < chunks; ++i) {
        if (i > 0) __syncthreads();
        wait_loads();
        gb.put(sh.b, rb);
        gc.put(sh.c, rc);
        __syncthreads();
        const ChunkDecay& decay = sh.decays[i & 1];
        if (i + 1 < chunks) {
            fetch(i + 1);
            if (wave == i % (kThreads<D, W> / kWave)) make_decay(i + 1);
            if (i + 2 < chunks) fetch_decay(i + 2);
        }
        const float chunk_total = decay.whole();
        total = total == 0.0f || chunk_total == 0.0f ? 0.0f : total * chunk_total;
        if (!kWide && c0 >= p.dc) continue;
        ColumnFrags<D, W> fc;
#pragma unroll
        for (int u = 0; u < U; ++u) fc[u] = sh.c.columns(0, c0 + u * 16, lane);
        add_chunk<D, W>(S, sh.b, fc, back ? decay.entry : decay.exit, chunk_total,
                                                p.u_scale, kWide ? W : p.da, lane);
    }
    float* const to = p.states + (head * x.segments + next) * (int64_t)p.da * p.dc;
#pragma unroll
    for (int k = 0; k < W / 16; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(k, group) + r, c = c0 + u * 16 + col;
                if (row < p.da && c < p.dc) to[(int64_t)row * p.dc + c] = S[k][u][r];
            }
    if (threadIdx.x == 0) p.totals[head * x.segments + seg] = total;
}

// Turns the segments' own states into the states before each of them, in scan
// order: in[s] = own[s - 1] + total[s - 1] in[s - 1].  A thread per element;
// the loads of kAhead segments are in flight together.  Bound by the states'
// bytes, read and written once: 16 heads of 128 x 128, 32 segments, 67 MB in
// 14.7 us (4.6 TB/s).
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

// dg of one segment of a head, 64 steps at a time from its end: a suffix sum of
// q.dq - k.dk in 64 bits (its terms cancel), from <state after the segment, its
// gradient>, started again at each cut, where nothing is carried over and dg is
// 0.  The windows of 64 depend on each other through one value, and each waits
// for its loads: a long segment is split over up to kDecayWaves waves, each of
// which first sums what its steps hand on (those before their first cut).
// 128 segments of 2048 steps, bf16: 33.6 us by one wave each, 12.8 by eight.
struct DecayGradArgs {
    SeqView g, reset, dg;
    const float *qdq, *kdk, *cross;
    int64_t N, T, seg_len;
    int32_t H, segments;
};

constexpr int kDecayWaves = 8;

// Waves to a segment: at least four windows each.
inline int decay_waves(int64_t seg_len)
{
    const int64_t w = seg_len / (4 * kWave);
    return (int)(w < 1 ? 1 : w < kDecayWaves ? w : kDecayWaves);
}

template <class D>
__global__ __launch_bounds__(kDecayWaves * kWave) void decay_grad(const DecayGradArgs x)
{
    __shared__ double handed[kDecayWaves];
    __shared__ bool ended[kDecayWaves];
    const int64_t head = blockIdx.x / x.segments, n = head / x.H;
    const int h = (int)(head % x.H), lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int waves = blockDim.x / kWave;
    const int64_t first = (int64_t)(blockIdx.x % x.segments) * x.seg_len;
    const int64_t past = x.T - first < x.seg_len ? x.T : first + x.seg_len;
    const int64_t windows = (past - first + kWave - 1) / kWave;
    const int64_t begin = min(past, first + wave * ((windows + waves - 1) / waves) * kWave);
    const int64_t stop_at = min(past, first + (wave + 1) * ((windows + waves - 1) / waves) * kWave);
    const auto load = [&](int64_t t, bool& cut) {
        const float g = to_f32(*seq_row<D>(x.g, n, t, h));
        cut = cuts(g) || (x.reset.p && *seq_row<uint8_t>(x.reset, n, t, 0) != 0);
        return (double)x.qdq[head * x.T + t] - (double)x.kdk[head * x.T + t];
    };
    double carry = x.cross[blockIdx.x];
    if (waves > 1) {
        double sum = 0.0;
        bool over = false;
        for (int64_t t0 = begin; t0 < stop_at && !over; t0 += kWave) {
            bool cut = false;
            const double v = t0 + lane < stop_at ? load(t0 + lane, cut) : 0.0;
            const uint64_t cuts = __ballot(cut);
            if (cuts == 0 || lane < __ffsll((unsigned long long)cuts) - 1) sum += v;
            over = cuts != 0;
        }
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        if (lane == 0) {
            handed[wave] = sum;
            ended[wave] = over;
        }
        __syncthreads();
        for (int w = waves - 1; w > wave; --w) carry = ended[w] ? handed[w] : handed[w] + carry;
    }
    for (int64_t end = stop_at; end > begin; end -= kWave) {
        const int64_t t = end - 1 - lane;
        double v = 0.0;
        bool cut = false;
        if (t >= begin) v = load(t, cut);
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
        if (t >= begin) *seq_row_out<D>(x.dg, n, t, h) = from_f32<D>(cut ? 0.0f : (float)v);
        carry = __shfl(v, kWave - 1);
        if (__shfl((int)cut, kWave - 1)) carry = 0.0;
    }
}

// Sums the value heads' gradients of a shared query or key head, in a fixed
// order: part [N, T, H, dim] in fp32 to y [N, T, H / group, dim].  3 x 1001 steps
// of 6 heads: 4.6 us; 8 x 2048 of 16 heads of 128 over 4: 50 us (3 TB/s) for each
// of dq and dk, beside 360 for the passes, whose fp32 results it reads back.
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
// the query, in one pass.  V: state elements per access (4 where value_dim is a
// multiple of 4 and the states lie on 16 bytes).  A block per head: rows of the
// state side by side, whose parts of out are added up in LDS in a fixed order.
// Bound by the state's bytes, which leave nothing for a matrix instruction to
// do: 4096 environments of 4 heads of 64 x 64, 545 MB in 99 us (5.5 TB/s, the
// rate of a large copy).  For one environment the call is host and launch time
// (14 us, binding included).
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
    const float f = reset || cuts(g) ? 0.0f : __expf(g);
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

// num_envs * heads of a call: three blocks of 512 threads to each, in a grid of
// less than 2^32 threads
constexpr int64_t kMaxHeads = int64_t(1) << 21;

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
// segment: as many segments as make kFillBlocks blocks, and no more, of at least
// kMinSegment steps.  Segments cost one more reading of two of the arrays and
// states written and read twice.  512 blocks are two on each of 256 CUs, all that
// bf16 at W = 128 has room for, and a second round is as long as the first; f16
// and f32 at W = 128 have room for one on each, f32 at W = 64 for three, 16-bit
// types there for four, and take the same number:
//   backward, bf16, 8 x 2048 of 16 heads of 128 x 128: 1 segment 345 us, 2 427, 3
//   408, 4 404, 8 476; 16384 of 8 heads 16: 253, 21: 227, 32: 256, 64: 259;
//   forward 32768 of 16 heads 16: 316, 32: 238, 64: 265;
//   16384 steps of 8 heads of 128 x 128, forward and backward, f32 10: 400 and
//   487, 21: 209 and 458, 32: 151 and 446, 64: 160 and 490; f16 21: 156 and 349,
//   32: 116 and 335, 64: 123 and 381;
//   of 64 x 64 in bf16 21: 87 and 136, 32: 64 and 111, 64: 53 and 116 (the rule
//   takes 64 and 21: a fifth is left there in the backward call);
//   3 x 1001 steps of 6 heads of 72 x 40 in f16 4: 62 and 90, 8: 40 and 87, 16: 46
//   and 100.
// Workspace: the states before each segment and the segments' decays, per
// direction; backward also q.dq and k.dk [N, H, T], <S, dS> [N, H, segments]
// and, for shared query and key heads, each value head's dq and dk.
constexpr int64_t kFillBlocks = 512;
constexpr int64_t kMinSegment = 128;

struct RecurrencePlan {
    int64_t seg_len, segments;
    size_t states[2], totals[2], qdq, kdk, cross, dq, dk, bytes;
};

inline RecurrencePlan plan_recurrence(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk,
                                      int64_t dv, bool backward)
{
    RecurrencePlan p{};
    const int64_t heads = N * H * (backward ? 3 : 1);
    const int64_t parts =
        std::max<int64_t>(1, std::min(kFillBlocks / heads, (T + kMinSegment - 1) / kMinSegment));
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

// The bytes that one access to a row of `dim` elements may take, in load8.
template <class D>
void set_vec(SeqView& v, int dim)
{
    constexpr int s = sizeof(D);
    v.vec = rows_on(v, 16 / s, s) && dim % 8 == 0 ? 16 : rows_on(v, 4 / s, s) && dim % (4 / s) == 0 ? 4 : s;
}

// Whether one 32-bit offset reaches a chunk of the array.
inline bool steps_near(const SeqView& v)
{
    return v.step <= (int64_t(1) << 31) / (kChunk * 4) - kMaxDim;
}

// Sets how the pass's arrays are accessed; true if kWide accesses serve them.
template <class D>
bool set_vec(PassArgs& p)
{
    bool wide = true;
    for (SeqView* v : {&p.a, &p.b, &p.c}) {
        set_vec<D>(*v, v == &p.c ? p.dc : p.da);
        wide = wide && v->vec == 16 && steps_near(*v);
    }
    p.d.vec = p.dc % 4 == 0 && rows_on(p.d, 4, sizeof(D));
    if (p.y_f32) set_vec<float>(p.y, p.dc);
    else set_vec<D>(p.y, p.dc);
    return wide && p.y.vec == 16 && steps_near(p.y) && (p.d.p == nullptr || (p.d.vec && steps_near(p.d)));
}

// The kernel for a call's width and accesses.
#define LRS_PICK(kernel, D, widest, wide)                                       \
    ((widest) <= 64 ? ((wide) ? kernel<D, 64, true> : kernel<D, 64, false>)     \
                    : ((wide) ? kernel<D, 128, true> : kernel<D, 128, false>))

// The states before every segment, in x.carry's directions.
template <class D>
lrs_status launch_carries(const char* nm, RecurrenceArgs& x, bool wide, hipStream_t stream)
{
    if (x.segments == 1) return LRS_OK;
    for (int i = 0; i < x.carries; ++i) {
        set_vec<D>(x.carry[i].b, x.carry[i].da);
        set_vec<D>(x.carry[i].c, x.carry[i].dc);
    }
    const int da = x.carry[0].da, dc = x.carry[0].dc, widest = std::max(da, dc);
    const uint64_t heads = (uint64_t)x.N * x.H, blocks = heads * (x.segments - 1) * x.carries;
    LRS_TRY(launch_seq(nm, LRS_PICK(segment_states, D, widest, wide), blocks, (widest <= 64 ? kThreads<D, 64> : kThreads<D, 128>), stream, x));
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
    p.p_scale = scale;
    p.u_scale = 1.0f;
    p.da = (int32_t)dk;
    p.dc = (int32_t)dv;
    const int widest = (int)std::max(dk, dv);
    const bool wide = set_vec<D>(p);
    LRS_TRY(launch_carries<D>(nm, x, wide, stream));
    return launch_seq(nm, LRS_PICK(recurrence_forward, D, widest, wide), (uint64_t)(N * H * plan.segments),
                      (widest <= 64 ? kThreads<D, 64> : kThreads<D, 128>), stream, x);
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
    pq.p_scale = scale;
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
    const int widest = (int)std::max(dk, dv);
    bool wide = true;
    for (PassArgs& p : x.pass) wide = set_vec<D>(p) && wide;
    LRS_TRY(launch_carries<D>(nm, x, wide, stream));
    LRS_TRY(launch_seq(nm, LRS_PICK(recurrence_backward, D, widest, wide), (uint64_t)(N * H * plan.segments) * 3,
                       (widest <= 64 ? kThreads<D, 64> : kThreads<D, 128>), stream, x));
    DecayGradArgs dg{w[4], w[5], w[9], qdq, kdk, cross, N, T, plan.seg_len, (int32_t)H,
                     (int32_t)plan.segments};
    LRS_TRY(launch_seq(nm, decay_grad<D>, (uint64_t)(N * H * plan.segments), kWave * decay_waves(plan.seg_len), stream, dg));
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
