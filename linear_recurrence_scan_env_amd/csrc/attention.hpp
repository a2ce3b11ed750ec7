// attention.hpp -- attention over a window of steps and the first steps of each
// episode.  Per environment and head (key head h / (heads / kv_heads)), with
// e(i) the first step of i's episode, query step i sees key step j where
//
//     e(i) <= j <= i   and   (j > i - window  or  j < e(i) + sinks)
//
// and with s_ij = scale q_i . k_j over the steps that it sees
//
//     lse_i = log sum_j e^{s_ij},   p_ij = e^{s_ij - lse_i},   o_i = sum_j p_ij v_j
//     D_i = do_i . o_i,   ds_ij = scale p_ij (do_i . v_j - D_i)
//     dq_i = sum_j ds_ij k_j,   dk_j = sum_i ds_ij q_i,   dv_j = sum_i p_ij do_i.
//
// What a query sees is two ranges of keys: the near one, from
// max(e(i), i - window + 1) to i, and the far one, the episode's first steps
// before that.  Queries follow each other, so a block of them sees one range of
// near keys and one of far keys, and only tiles at their ends need the mask.
//
// All three kernels (forward, dq, dk and dv) have one form.  A wave holds 32
// queries (or keys) as the columns of 32x32 matrix products; the other side comes
// through LDS in tiles.  The scores arrive with a lane's own column in its
// registers, so softmax statistics are per lane, and the weights go back as an
// operand as they lie: the rows that a lane holds of a product, 8 (r / 4) +
// 4 (lane / 32) + r % 4, are taken as the order of the sum, and the other operand
// is read by columns of LDS in the same order.
#pragma once

#include "sequence.hpp"

namespace lrs {

constexpr int kMaxAttDim = 128;
constexpr int64_t kMaxKeySteps = int64_t(1) << 29;  // a step and a window, or a slot and a block's, in 32 bits
constexpr float kAttLog2e = 1.44269504088896341f;
constexpr float kAttLn2 = 0.693147180559945309f;

struct AttArgs {
    SeqView q, k, v, o, lse;    // lse float32 [N, T, H], nullable in the forward
    SeqView dout, dq, dk, dv;
    const int32_t* starts;      // [N, TK]: the first step of each key step's episode; null: 0
    const int32_t* ends;        // [N, TK]: the step behind its last; null: TK
    float* delta;               // D, [N, H, T]
    float* far_part;            // [N, KV, far_chunks, sinks, 2 W] sums of attend_far; null: it does not run
    int64_t N;
    int32_t T, TK, H, group, window, sinks, dim_k, dim_v;
    int32_t hpb, tiles;         // heads per block, blocks per row of steps
    int32_t far_chunks;
    uint8_t sum_delta;          // whether dq sums D itself
    float scale, c;             // c = |scale| log2(e)
};

// ------------------------------------------------------- matrix instructions
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 abf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 af16x8 __attribute__((ext_vector_type(8)));
typedef short as16x4 __attribute__((ext_vector_type(4)));

// Eight values of one row or column of an operand: what a lane gives to a product
// over 16 values (lanes 0..31 the first eight, 32..63 the others).
template <class D>
using AFrag = Raw8<D>;

// acc += A B over 16 values.  float32 takes the matrix instructions of its own
// type, two values at a time.
template <class D>
__device__ __forceinline__ f32x16 mma32(const AFrag<D>& a, const AFrag<D>& b, f32x16 acc)
{
    if constexpr (std::is_same<D, bf16_t>::value) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(abf16x8, a.w[0]),
                                                       __builtin_bit_cast(abf16x8, b.w[0]), acc, 0, 0, 0);
    } else if constexpr (std::is_same<D, f16_t>::value) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(af16x8, a.w[0]),
                                                      __builtin_bit_cast(af16x8, b.w[0]), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w[e / 4][e % 4]),
                                                       __uint_as_float(b.w[e / 4][e % 4]), acc, 0, 0, 0);
        return acc;
    }
}

// The row that register r of a product holds for a lane of half h.
__device__ __forceinline__ constexpr int acc_row(int r, int h) { return 8 * (r / 4) + 4 * h + r % 4; }

// Registers 8u .. 8u + 7 as an operand: 16-bit types round the weights here, once
// (by 2^-8 or 2^-11 of each at most; they are summed in float32 before that).
template <class D>
__device__ __forceinline__ AFrag<D> operand(const f32x16& v, int u)
{
    AFrag<D> f;
    if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f.w[e / 4][e % 4] = __float_as_uint(v[8 * u + e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f.w[0][e] = pack2<D>(v[8 * u + 2 * e], v[8 * u + 2 * e + 1]);
    }
    return f;
}

// What operand() left of the values, as a second operand.  ds goes into its products
// as these two parts: with one, gradients of q and k in 16-bit types were off by 1.45
// to 1.7 times the one rounding of the result.  Both use the same fragment of LDS.
template <class D>
__device__ __forceinline__ AFrag<D> operand_rest(const f32x16& v, int u, const AFrag<D>& f)
{
    AFrag<D> g;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        unpack2<D>(f.w[0][e], lo, hi);
        g.w[0][e] = pack2<D>(v[8 * u + 2 * e] - lo, v[8 * u + 2 * e + 1] - hi);
    }
    return g;
}

// ------------------------------------------------------------- tiles in LDS
typedef __attribute__((address_space(3))) char* lds_t;

__device__ __forceinline__ uint32_t lds_address(void* p) { return (uint32_t)(uintptr_t)(lds_t)p; }
template <class T>
__device__ __forceinline__ T lds_load(uint32_t at)
{
    return *(const __attribute__((address_space(3))) T*)(lds_t)(uintptr_t)at;
}
__device__ __forceinline__ void lds_store(uint32_t at, const u32x4& v)
{
    *(__attribute__((address_space(3))) u32x4*)(lds_t)(uintptr_t)at = v;
}

// Rows of W elements without padding; 16-byte chunk c of row r lies at c ^ turn(r)
// so that 16 rows at one chunk, and the reads by columns, spread over all banks.
// turn() repeats every 16 rows, so a lane's address for one kind of read is one
// number for the tile, turned over in some bits and moved by a constant.
template <class D, int W>
struct AttTile {
    static constexpr int kRow = W * (int)sizeof(D);
    static __device__ __forceinline__ int turn(int r)
    {
        if constexpr (sizeof(D) == 4) return (((r >> 2) & 1) << 3) | (((r >> 3) & 1) << 2) | (r & 3);
        else if constexpr (W == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
        else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    }
    static __device__ __forceinline__ uint32_t at(int r, int chunk)
    {
        return (uint32_t)(r * kRow + ((chunk ^ turn(r)) << 4));
    }

    // Rows row + lane % 32, elements 16 ks + 8 (lane / 32) + 0..7; `mine` from row_lane().
    static __device__ __forceinline__ uint32_t row_lane(int lane)
    {
        return at(lane & 31, (int)sizeof(D) / 2 * (lane >> 5));
    }
    static __device__ __forceinline__ AFrag<D> rows(uint32_t mine, int row, int ks)
    {
        AFrag<D> f;
#pragma unroll
        for (int k = 0; k < (int)sizeof(D) / 2; ++k)
            f.w[k] = lds_load<u32x4>((mine ^ (uint32_t)(ks * 16 * (int)sizeof(D) + k * 16)) + row * kRow);
        return f;
    }
    // Column col + lane % 32 of rows row + 8 (e / 4) + 4 (lane / 32) + e % 4, e = 0..7
    // (row a multiple of 16, col of 32); `mine` from column_lane().  A transposing read
    // hands the 16 lanes of a group four rows of four groups of 4 columns, 8 bytes read
    // by each lane.
    static __device__ __forceinline__ uint32_t column_lane(int lane)
    {
        const int h = lane >> 5;
        if constexpr (sizeof(D) == 4) return at(4 * h, (lane & 31) / 4) + 4 * (lane & 3);
        const int c = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
        return at(4 * h + ((lane & 15) >> 2), c / 8) + 2 * (c % 8);
    }
    static __device__ __forceinline__ AFrag<D> columns(uint32_t mine, int row, int col)
    {
        AFrag<D> f;
        if constexpr (sizeof(D) == 4) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f.w[e / 4][e % 4] = lds_load<uint32_t>((mine ^ (uint32_t)(col * 4 | (e / 4) << 6 | (e % 4) << 4)) +
                                                       (row + 8 * (e / 4) + e % 4) * kRow);
        } else {
            typedef __attribute__((address_space(3))) as16x4* four;
            const uint32_t a = (mine ^ (uint32_t)(col * 2)) + row * kRow;
            const uint32_t b = (mine ^ (uint32_t)(col * 2 | 32)) + (row + 8) * kRow;
            const as16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((four)(uintptr_t)a);
            const as16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((four)(uintptr_t)b);
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            f.w[0] = __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
};

// The row of a head at a step (heads are not shared within an array here).
template <class D>
__device__ __forceinline__ const char* att_row(const SeqView& v, int64_t n, int64_t t, int64_t h)
{
    return static_cast<const char*>(v.p) + (n * v.env + t * v.step + h * v.head) * (int64_t)sizeof(D);
}

// Loads through a buffer descriptor: what lies at or behind `bytes` becomes zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t bounded(const char* p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, bytes, 0x00020000);
}

// Rows of memory on their way into a tile of kRows rows, by a block of 256 threads
// or by a wave.  What lies beyond the last row or the dimension becomes zeros.
// kBy: rows are taken by 8 elements (16-bit types), by 4 (dims of whole fours, rows on
// as many), or 0: by the element with branches.  The first two load through a buffer
// descriptor whose bounds make the zeros, and have no branch between the loads: where
// branches meet each load would be waited for.  place() says where the next tile
// begins, and after fetch() the one behind it is next.
template <class D, int W, int kRows, int kBy, int kThreads = 256, int kSets = 1>
struct AttStage {
    static constexpr int kUnits = kRows * (W / 8) / kThreads, kApart = kThreads / (W / 8);
    static_assert(kApart % 16 == 0 || kThreads < 256, "rows of a thread's units lie alike");
    Raw8<D> r[kSets][kUnits];  // tiles on their way
    const char* p;
    int64_t step;      // bytes
    uint32_t off[2];   // where this thread's first unit begins, and its other half (kBy = 4)
    int dim, vec;

    static __device__ __forceinline__ int row() { return (int)(threadIdx.x % kThreads) / (W / 8); }
    static __device__ __forceinline__ int column() { return (int)(threadIdx.x % kThreads) % (W / 8) * 8; }

    __device__ __forceinline__ void start(const SeqView& v, int dim_)
    {
        dim = dim_;
        vec = v.vec;
        step = v.step * (int64_t)sizeof(D);
        // beyond every bound where the tile is wider than the rows
        for (int k = 0; k < 2; ++k)
            off[k] = column() + 4 * k < dim
                ? (uint32_t)row() * (uint32_t)step + (column() + 4 * k) * (uint32_t)sizeof(D) : 0x7f000000u;
    }
    __device__ __forceinline__ void place(const SeqView& v, int64_t n, int h, int64_t t)
    {
        p = att_row<D>(v, n, t, h);
    }
    template <int set = 0>
    __device__ __forceinline__ void fetch(int count)
    {
        if constexpr (kBy > 0) {
            const __amdgpu_buffer_rsrc_t rows = bounded(p, (count - 1) * (int)step + dim * (int)sizeof(D));
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const uint32_t more = (uint32_t)(u * kApart) * (uint32_t)step;
                if constexpr (kBy == 8) {
                    r[set][u].w[0] = __builtin_amdgcn_raw_buffer_load_b128(rows, off[0] + more, 0, 0);
                } else if constexpr (sizeof(D) == 4) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        r[set][u].w[k] = __builtin_amdgcn_raw_buffer_load_b128(rows, off[k] + more, 0, 0);
                } else {
                    const u32x2 a = __builtin_amdgcn_raw_buffer_load_b64(rows, off[0] + more, 0, 0);
                    const u32x2 b = __builtin_amdgcn_raw_buffer_load_b64(rows, off[1] + more, 0, 0);
                    r[set][u].w[0] = u32x4{a[0], a[1], b[0], b[1]};
                }
            }
        } else {
            const int c = column();
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int at = row() + u * kApart;
                r[set][u] = Raw8<D>{};
                if (at < count && c < dim)
                    r[set][u] = load8<D>(reinterpret_cast<const D*>(p + at * step), c, dim, vec);
            }
        }
        p += kRows * step;
    }
    // Where put() puts this thread's first unit of a tile at `tile`.
    static __device__ __forceinline__ uint32_t lane(uint32_t tile)
    {
        return tile + AttTile<D, W>::at(row(), (int)sizeof(D) / 2 * (column() / 8));
    }
    template <int set = 0>
    __device__ __forceinline__ void put(uint32_t mine) const
    {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            // a wave's units lie fewer than 16 rows apart, each with a turn of its own
            const uint32_t at = kApart % 16 == 0
                ? mine + u * kApart * AttTile<D, W>::kRow
                : mine - lane(0) + AttTile<D, W>::at(row() + u * kApart, (int)sizeof(D) / 2 * (column() / 8));
#pragma unroll
            for (int k = 0; k < (int)sizeof(D) / 2; ++k) lds_store(at ^ (16u * k), r[set][u].w[k]);
        }
    }
};

// -------------------------------------------------------------- what is seen
// The two ranges of keys of one query, as first key and length.
struct Seen {
    int near, near_len, far, far_len;
    bool far_any;  // whether any query has first steps before its near range: of the call
};

__device__ __forceinline__ int episode_start(const AttArgs& x, int64_t n, int j)
{
    return x.starts != nullptr ? x.starts[n * x.TK + j] : 0;
}

__device__ __forceinline__ Seen seen_by(const AttArgs& x, int i, int start)
{
    Seen s;
    s.near = max(start, i - x.window + 1);
    s.near_len = i - s.near + 1;
    s.far = start;
    s.far_len = min(x.sinks, s.near - start);
    s.far_any = x.sinks > 0;
    return s;
}

__device__ __forceinline__ bool sees(const Seen& s, int j)
{
    // (without a branch between the two)
    return (bool)(((unsigned)(j - s.near) < (unsigned)s.near_len) | ((unsigned)(j - s.far) < (unsigned)s.far_len));
}

// Rows begin .. end - 1 of a product whose first row is step j0, as the bits of what
// register r of a lane of half h holds: bit acc_row(r, 0).
__device__ __forceinline__ uint32_t row_bits(int begin, int end, int j0, int h)
{
    const int lo = min(max(begin - j0, 0), 32), hi = min(max(end - j0, 0), 32);
    const uint64_t bits = ((uint64_t(1) << hi) - 1) & ~((uint64_t(1) << lo) - 1);
    return (uint32_t)bits >> (4 * h);
}
// v where the bit of register r is set, else `other`: two instructions, and no compare.
template <int r>
__device__ __forceinline__ float where_bit(uint32_t bits, float v, float other)
{
    // (as an instruction: the compiler would make a test and a select of it)
    uint32_t all;
    asm("v_bfe_i32 %0, %1, %2, 1" : "=v"(all) : "v"(bits), "n"(acc_row(r, 0)));
    return __uint_as_float((all & __float_as_uint(v)) | (~all & __float_as_uint(other)));
}

template <int... r>
__device__ __forceinline__ void keep_bits(uint32_t bits, f32x16& v, float other, std::integer_sequence<int, r...>)
{
    ((v[r] = where_bit<r>(bits, v[r], other)), ...);
}
// The rows whose bits are set, `other` in the rest.
__device__ __forceinline__ void keep_bits(uint32_t bits, f32x16& v, float other)
{
    keep_bits(bits, v, other, std::make_integer_sequence<int, 16>());
}

// What a block's queries see: tiles of kTile keys, the far range's first.
struct KeyTiles {
    int far, far_end, near, near_end, far_tiles, tiles;

    __device__ __forceinline__ KeyTiles(const AttArgs& x, int64_t n, int first, int last, int tile)
    {
        const Seen s = seen_by(x, first, episode_start(x, n, first));
        far = s.far;
        far_end = s.far + s.far_len;
        near = s.near;
        near_end = last + 1;
        far_tiles = (s.far_len + tile - 1) / tile;
        tiles = far_tiles + (near_end - near + tile - 1) / tile;
    }
    __device__ __forceinline__ void get(int it, int tile, int& j0, int& j1) const
    {
        const bool is_far = it < far_tiles;
        j0 = is_far ? far + it * tile : near + (it - far_tiles) * tile;
        j1 = min(j0 + tile, is_far ? far_end : near_end);
    }
};

// The wave's 32 queries, a lane's own being lane % 32.
struct WaveQueries {
    int i;        // the query's step among the keys
    bool valid;
    Seen seen;
    int first, last;     // of the wave's queries, first > last where it has none
    int lo_most, lo_least;  // of their near ranges

    __device__ __forceinline__ WaveQueries(const AttArgs& x, int64_t n, int step0, int block_near, int lane)
    {
        const int past = x.TK - x.T;
        const int step = step0 + (lane & 31);
        valid = step < x.T;
        i = past + min(step, x.T - 1);
        first = past + step0;
        last = past + min(step0 + 31, x.T - 1);
        seen = seen_by(x, i, episode_start(x, n, i));
        // first steps that lie among the block's near keys come with their tiles
        const int least = seen.far + x.sinks > block_near ? max(seen.far, block_near) : seen.near;
        lo_least = __builtin_amdgcn_readlane(least, 0);
        lo_most = __builtin_amdgcn_readlane(seen.near, 31);
        // steps ascend and so do starts: lane 31 (clamped to the last step) has the most
        if (!valid) seen.near_len = seen.far_len = 0;
    }
    __device__ __forceinline__ bool any() const { return first <= last; }
    // The rows of a product from key j0 on that the lane's query sees, of a tile that ends at j1.
    __device__ __forceinline__ uint32_t bits(bool is_far, int j0, int j1, int h) const
    {
        uint32_t b = is_far ? 0 : row_bits(seen.near, seen.near + seen.near_len, j0, h);
        if (seen.far_any) b |= row_bits(seen.far, min(seen.far + seen.far_len, j1), j0, h);
        return b;
    }
    // Whether some query may see keys j0 .. j1 - 1 of a tile, and whether all see all.
    __device__ __forceinline__ bool touches(const KeyTiles& kt, bool is_far, int j0, int j1) const
    {
        return any() && (is_far || (j0 <= last && j1 > lo_least));
    }
    __device__ __forceinline__ bool whole(bool is_far, int j0, int j1, int tile) const
    {
        return !is_far && j1 - j0 == tile && j0 >= lo_most && j1 - 1 <= first;
    }
};

// Blocks by eighths: consecutive blocks go to the eight XCDs in turn, and each of
// these then works on one stretch of neighbouring tiles, whose keys its L2 holds.
__device__ __forceinline__ uint32_t by_xcd(uint32_t b, uint32_t blocks)
{
    const uint32_t per = blocks / 8, rest = blocks % 8, x = b % 8, k = b / 8;
    return x * per + min(x, rest) + k;
}

// ---------------------------------------------------------- the careful form
// One query (or key) at a time by one wave, from the formulas: lanes are keys
// while scores are made and elements while rows are summed, and what is not seen
// is neither read nor multiplied.  The fast forms multiply unseen values by 0;
// where a result is not finite it is computed again here, so that NaN and
// infinities reach exactly the results that have a part in them.
template <class D>
__device__ __forceinline__ float row_dot(const D* a, const D* b, int dim)
{
    float s = 0.0f;
    for (int d = 0; d < dim; ++d) s = fmaf(to_f32(a[d]), to_f32(b[d]), s);
    return s;
}

template <class D>
__device__ __forceinline__ void careful_forward(const AttArgs& x, int64_t n, int head, int i, int lane)
{
    const int t = i - (x.TK - x.T), kvh = head / x.group;
    const Seen s = seen_by(x, i, episode_start(x, n, i));
    const D* const q = seq_row<D>(x.q, n, t, head);
    const int total = s.far_len + s.near_len;
    float m = -INFINITY;
    bool nan = false;
    for (int a = lane; a < total; a += kWave) {
        const int j = a < s.far_len ? s.far + a : s.near + a - s.far_len;
        const float v = x.scale * row_dot(q, seq_row<D>(x.k, n, j, kvh), x.dim_k);
        nan |= v != v;
        m = fmaxf(m, v);
    }
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (__any(nan)) m = __builtin_nanf("");
    float l = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int a0 = 0; a0 < total; a0 += kWave) {
        const int a = a0 + lane, j = a < s.far_len ? s.far + a : s.near + a - s.far_len;
        float p = 0.0f;
        if (a < total) p = expf(x.scale * row_dot(q, seq_row<D>(x.k, n, j, kvh), x.dim_k) - m);
        l += p;
        for (int b = 0; b < min(kWave, total - a0); ++b) {
            const float w = __shfl(p, b);
            const D* const v = seq_row<D>(x.v, n, __shfl(j, b), kvh);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (lane + k * kWave < x.dim_v) acc[k] = fmaf(w, to_f32(v[lane + k * kWave]), acc[k]);
        }
    }
    for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
    D* const out = seq_row_out<D>(x.o, n, t, head);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + k * kWave < x.dim_v) out[lane + k * kWave] = from_f32<D>(acc[k] / l);
    if (lane == 0 && x.lse.p != nullptr) *seq_row_out<float>(x.lse, n, t, head) = m + logf(l);
}

template <class D>
__device__ __forceinline__ void careful_dq(const AttArgs& x, int64_t n, int head, int i, int lane)
{
    const int t = i - (x.TK - x.T), kvh = head / x.group;
    const Seen s = seen_by(x, i, episode_start(x, n, i));
    const D *const q = seq_row<D>(x.q, n, t, head), *const d_o = seq_row<D>(x.dout, n, t, head);
    const float lse = *seq_row<float>(x.lse, n, t, head);
    const float delta = row_dot(d_o, seq_row<D>(x.o, n, t, head), x.dim_v);
    const int total = s.far_len + s.near_len;
    float acc[2] = {0.0f, 0.0f};
    for (int a0 = 0; a0 < total; a0 += kWave) {
        const int a = a0 + lane, j = a < s.far_len ? s.far + a : s.near + a - s.far_len;
        float ds = 0.0f;
        if (a < total) {
            const float p = expf(x.scale * row_dot(q, seq_row<D>(x.k, n, j, kvh), x.dim_k) - lse);
            ds = x.scale * (p * (row_dot(d_o, seq_row<D>(x.v, n, j, kvh), x.dim_v) - delta));
        }
        for (int b = 0; b < min(kWave, total - a0); ++b) {
            const float w = __shfl(ds, b);
            const D* const k = seq_row<D>(x.k, n, __shfl(j, b), kvh);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (lane + e * kWave < x.dim_k) acc[e] = fmaf(w, to_f32(k[lane + e * kWave]), acc[e]);
        }
    }
    D* const out = seq_row_out<D>(x.dq, n, t, head);
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (lane + e * kWave < x.dim_k) out[lane + e * kWave] = from_f32<D>(acc[e]);
}

template <class D, bool kK, bool kV>
__device__ __forceinline__ void careful_dkv(const AttArgs& x, int64_t n, int kvh, int j, int lane)
{
    const int past = x.TK - x.T;
    const D *const k = seq_row<D>(x.k, n, j, kvh), *const v = seq_row<D>(x.v, n, j, kvh);
    float dk[2] = {0.0f, 0.0f}, dv[2] = {0.0f, 0.0f};
    for (int head = kvh * x.group; head < (kvh + 1) * x.group; ++head)
        for (int i0 = max(j, past); i0 < x.TK; i0 += kWave) {
            const int i = i0 + lane, in = min(i, x.TK - 1), start = episode_start(x, n, in);
            const bool mine = i < x.TK && sees(seen_by(x, in, start), j);
            const uint64_t who = __ballot(mine);
            // no later query sees j once this lane's is beyond the window, or the episode
            if (who == 0 && (__shfl(start, 0) > j || (i0 - j >= x.window && j >= __shfl(start, 0) + x.sinks))) break;
            float p = 0.0f, ds = 0.0f;
            const int t = in - past;
            if (mine) {
                const D* const d_o = seq_row<D>(x.dout, n, t, head);
                p = expf(x.scale * row_dot(seq_row<D>(x.q, n, t, head), k, x.dim_k) -
                         *seq_row<float>(x.lse, n, t, head));
                ds = x.scale * (p * (row_dot(d_o, v, x.dim_v) -
                                     row_dot(d_o, seq_row<D>(x.o, n, t, head), x.dim_v)));
            }
            for (int b = 0; b < kWave; ++b) {
                if (!((who >> b) & 1)) continue;
                const float pb = __shfl(p, b), sb = __shfl(ds, b);
                const D* const q = seq_row<D>(x.q, n, i0 + b - past, head);
                const D* const d_o = seq_row<D>(x.dout, n, i0 + b - past, head);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = lane + e * kWave;
                    if (c < x.dim_k) dk[e] = fmaf(sb, to_f32(q[c]), dk[e]);
                    if (c < x.dim_v) dv[e] = fmaf(pb, to_f32(d_o[c]), dv[e]);
                }
            }
        }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int c = lane + e * kWave;
        if (kK && c < x.dim_k) seq_row_out<D>(x.dk, n, j, kvh)[c] = from_f32<D>(dk[e]);
        if (kV && c < x.dim_v) seq_row_out<D>(x.dv, n, j, kvh)[c] = from_f32<D>(dv[e]);
    }
}

// -------------------------------------------------------------- fast kernels

// 32 rows (queries or keys, a lane's own) as operands: element 16 ks + 8 h + e.
template <class D, int W, int kBy>
struct OwnRows {
    AFrag<D> f[W / 16];

    __device__ __forceinline__ void load(const SeqView& v, int64_t n, int64_t t, int h, int dim, bool valid,
                                         int lane)
    {
        const D* const row = reinterpret_cast<const D*>(att_row<D>(v, n, t, h));
#pragma unroll
        for (int ks = 0; ks < W / 16; ++ks) {
            const int c = 16 * ks + 8 * (lane >> 5);
            f[ks] = AFrag<D>{};
            if (!valid || c >= dim) continue;
            if constexpr (kBy == 8) {
                f[ks].w[0] = *reinterpret_cast<const u32x4*>(row + c);
            } else if constexpr (kBy == 4 && sizeof(D) == 4) {
                f[ks].w[0] = *reinterpret_cast<const u32x4*>(row + c);
                if (c + 4 < dim) f[ks].w[1] = *reinterpret_cast<const u32x4*>(row + c + 4);
            } else if constexpr (kBy == 4) {
                const u32x2 a = *reinterpret_cast<const u32x2*>(row + c);
                u32x2 b = {};
                if (c + 4 < dim) b = *reinterpret_cast<const u32x2*>(row + c + 4);
                f[ks].w[0] = u32x4{a[0], a[1], b[0], b[1]};
            } else {
                f[ks] = load8<D>(row, c, dim, v.vec);
            }
        }
    }
    // Every value's sign turned over where `turn`.
    __device__ __forceinline__ void signs(bool turn)
    {
        const uint32_t m = !turn ? 0u : sizeof(D) == 4 ? 0x80000000u : 0x80008000u;
#pragma unroll
        for (int ks = 0; ks < W / 16; ++ks)
#pragma unroll
            for (int k = 0; k < (int)sizeof(D) / 2; ++k) f[ks].w[k] ^= u32x4{m, m, m, m};
    }
};

// The products of a lane's own rows with others of the same place, summed.
template <class D, int W, int kBy>
__device__ __forceinline__ float own_dot(const SeqView& v, int64_t n, int64_t t, int head, int dim, bool valid,
                                         int lane, const OwnRows<D, W, kBy>& with)
{
    OwnRows<D, W, kBy> o;
    o.load(v, n, t, head, dim, valid, lane);
    float sum = 0.0f;
#pragma unroll
    for (int ks = 0; ks < W / 16; ++ks)
#pragma unroll
        for (int k = 0; k < (int)sizeof(D) / 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(D) == 4) {
                    sum = fmaf(__uint_as_float(o.f[ks].w[k][e]), __uint_as_float(with.f[ks].w[k][e]), sum);
                } else {
                    float a0, a1, b0, b1;
                    unpack2<D>(o.f[ks].w[k][e], a0, a1);
                    unpack2<D>(with.f[ks].w[k][e], b0, b1);
                    sum = fmaf(a1, b1, fmaf(a0, b0, sum));
                }
            }
    return sum + __shfl_xor(sum, 32);
}

// The products of 32 rows of tile `ta` (and of `tb`) with the wave's own rows, over
// all W elements.  Fragments are read kAhead products before they are used: left to
// itself the compiler reads one, waits for it, and multiplies.
template <class D, int W, bool kTwo, int kAhead, int kBy>
__device__ __forceinline__ void row_products(uint32_t ta, const OwnRows<D, W, kBy>& a, uint32_t tb,
                                             const OwnRows<D, W, kBy>& b, int row, f32x16& s, f32x16& t)
{
    using Tile = AttTile<D, W>;
    constexpr int N = W / 16;
    AFrag<D> fa[N], fb[N];
#pragma unroll
    for (int ks = 0; ks < N + kAhead; ++ks) {
        if (ks < N) {
            fa[ks] = Tile::rows(ta, row, ks);
            if constexpr (kTwo) fb[ks] = Tile::rows(tb, row, ks);
        }
        if constexpr (kAhead > 0) __builtin_amdgcn_sched_barrier(0);
        const int at = ks - kAhead;
        if (at >= 0) {
            s = mma32<D>(fa[at], a.f[at], s);
            if constexpr (kTwo) t = mma32<D>(fb[at], b.f[at], t);
        }
    }
}

// Writes a product whose columns are the wave's rows (a lane's own: `row`) and
// whose rows are elements; rows of memory get four elements at a time.
template <class D, int kBy, int kTiles>
__device__ __forceinline__ void store_own(D* row, const f32x16 (&acc)[kTiles], float by, int dim, int h)
{
#pragma unroll
    for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int c = 32 * dt + 8 * r4 + 4 * h;
            const float v[4] = {acc[dt][4 * r4] * by, acc[dt][4 * r4 + 1] * by, acc[dt][4 * r4 + 2] * by,
                                acc[dt][4 * r4 + 3] * by};
            if constexpr (kBy > 0) {
                if (c >= dim) continue;
                if constexpr (sizeof(D) == 4)
                    *reinterpret_cast<f32x4*>(row + c) = f32x4{v[0], v[1], v[2], v[3]};
                else
                    *reinterpret_cast<u32x2*>(row + c) = u32x2{pack2<D>(v[0], v[1]), pack2<D>(v[2], v[3])};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < dim) row[c + e] = from_f32<D>(v[e]);
            }
        }
}

// Whether all values are finite.
template <int kTiles>
__device__ __forceinline__ bool finite(const f32x16 (&acc)[kTiles])
{
    float z = 0.0f;
#pragma unroll
    for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) z = fmaf(acc[dt][r], 0.0f, z);
    return z == 0.0f;
}

// Keys in a tile of the forward and of dq, and how many tiles are on their way.  Two at 16
// bits: a tile takes less to compute than to load.
template <class D, int W>
constexpr int kKeyTile = sizeof(D) == 4 ? 32 : 64;
template <class D, int W>
constexpr int kGradTile = W == 128 ? 32 : 64;
template <class D, int W>
constexpr int kKeySets = sizeof(D) == 4 ? 1 : 2;
template <class D, int W>
constexpr int kGradSets = sizeof(D) == 4 ? 1 : 2;
template <class D, int W>
constexpr int kAttBlocks = sizeof(D) == 4 && W == 128 ? 1 : 2;  // blocks per CU

// A block's place: its heads, and the steps of its four waves.  Alone: each wave has 32
// steps of a head and tiles of its own.
struct AttBlock {
    int64_t n;
    int head, step0, first, last, kvh;
    bool any;

    __device__ __forceinline__ AttBlock(const AttArgs& x, bool alone)
    {
        any = true;
        if (alone) {
            const uint32_t id = by_xcd(blockIdx.x, gridDim.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
            const uint32_t row = id / x.tiles;
            any = row < x.N * x.H;
            n = row / x.H;
            head = row % x.H;
            kvh = head / x.group;
            step0 = (id - row * x.tiles) * 32;
            first = x.TK - x.T + step0;
            last = min(first + 32, x.TK) - 1;
            return;
        }
        const uint32_t id = by_xcd(blockIdx.x, gridDim.x);
        const int hblocks = x.H / x.hpb, rows = 4 / x.hpb * 32;
        const uint32_t tile = id % x.tiles, hb = id / x.tiles % hblocks;
        n = id / x.tiles / hblocks;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        head = hb * x.hpb + wave % x.hpb;
        kvh = head / x.group;
        step0 = tile * rows + wave / x.hpb * 32;
        first = x.TK - x.T + tile * rows;
        last = min(first + rows, x.TK) - 1;
    }
};

// Goes over the tiles of keys and values that a wave's queries see, in tiles of its own:
// compute() as in over_keys.  kAhead: the next tile is on its way while one is computed
// (the forward; dq and attend_dkv would spill registers: both directions of 64 x 512 f32
// steps of 4 heads of 64 took 490 us with it, 373 with blocks).
template <class D, int W, int BK, int kBy, bool kAhead, class Compute>
__device__ __forceinline__ void over_keys_alone(const AttArgs& x, const AttBlock& b, const KeyTiles& kt, char* lds,
                                                int lane, Compute compute)
{
    using Tile = AttTile<D, W>;
    AttStage<D, W, BK, kBy, kWave> sk, sv;
    sk.start(x.k, x.dim_k);
    sv.start(x.v, x.dim_v);
    const uint32_t at = lds_address(lds), put_at = sk.lane(at);
    auto fetch = [&](int it) {
        int j0, j1;
        kt.get(it, BK, j0, j1);
        if (it == 0 || it == kt.far_tiles) {
            sk.place(x.k, b.n, b.kvh, j0);
            sv.place(x.v, b.n, b.kvh, j0);
        }
        sk.fetch(j1 - j0);
        sv.fetch(j1 - j0);
    };
    if (kAhead) fetch(0);
    for (int it = 0; it < kt.tiles; ++it) {
        if (!kAhead) fetch(it);
        sk.put(put_at);
        sv.put(put_at + BK * Tile::kRow);
        if (kAhead && it + 1 < kt.tiles) fetch(it + 1);
        __builtin_amdgcn_wave_barrier();
        int j0, j1;
        kt.get(it, BK, j0, j1);
        compute(at + Tile::row_lane(lane), at + Tile::column_lane(lane), it < kt.far_tiles, j0, j1);
        __builtin_amdgcn_wave_barrier();
    }
}

// Goes over the tiles of keys and values that a block's queries see: compute(by_row,
// by_col, is_far, j0, j1) for each, with a lane's places in the keys' tile (the values'
// lies kBytes behind).  kSets: how many tiles are on their way from memory.
template <class D, int W, int BK, int kBy, int kSets, class Compute>
__device__ __forceinline__ void over_keys(const AttArgs& x, const AttBlock& b, const KeyTiles& kt, char* lds, int lane,
                                          Compute compute)
{
    using Tile = AttTile<D, W>;
    constexpr int kBytes = BK * Tile::kRow;
    AttStage<D, W, BK, kBy, 256, kSets> sk, sv;
    sk.start(x.k, x.dim_k);
    sv.start(x.v, x.dim_v);
    int fetched = 0;
    auto fetch = [&](auto set) {
        constexpr int s = decltype(set)::value;
        if (fetched == kt.tiles) return;
        int j0, j1;
        kt.get(fetched, BK, j0, j1);
        if (fetched == 0 || fetched == kt.far_tiles) {
            sk.place(x.k, b.n, b.kvh, j0);
            sv.place(x.v, b.n, b.kvh, j0);
        }
        sk.template fetch<s>(j1 - j0);
        sv.template fetch<s>(j1 - j0);
        ++fetched;
    };
    // the lane's places in the tiles of the first buffer, moved to the other and back
    uint32_t by_row = lds_address(lds) + Tile::row_lane(lane), by_col = lds_address(lds) + Tile::column_lane(lane);
    uint32_t put_at = sk.lane(lds_address(lds));
    auto put = [&](auto set) {
        sk.template put<decltype(set)::value>(put_at);
        sv.template put<decltype(set)::value>(put_at + kBytes);
    };
    // Tile `it`, with the one behind it put down from `set` and another fetched into that.
    auto step = [&](int it, auto set) {
        __syncthreads();
        int j0, j1;
        kt.get(it, BK, j0, j1);
        compute(by_row, by_col, it < kt.far_tiles, j0, j1);
        const uint32_t move = it & 1 ? -2 * kBytes : 2 * kBytes;
        by_row += move;
        by_col += move;
        put_at += move;
        if (it + 1 < kt.tiles) {
            put(set);
            fetch(set);
        }
    };
    constexpr std::integral_constant<int, 0> s0{};
    constexpr std::integral_constant<int, kSets - 1> s1{};
    fetch(s0);
    put(s0);
    fetch(s1);
    if constexpr (kSets == 2) fetch(s0);
    for (int it = 0; it < kt.tiles; it += 2) {
        step(it, s1);
        if (it + 1 < kt.tiles) step(it + 1, s0);
    }
}

// The forward: S^T = K Q^T by tiles, a running maximum and sum per lane, O^T += V^T P^T.
// Products bound it at long windows: 1 x 32768 bf16 steps of 16 heads over 4 of 128, window
// 4096, 1165 us, 886 TF/s (a library product of 8192^3 has 1340), the exponentials of one
// wave beside the products of the other; loads, few tiles and stores in turn at short ones:
// 4096 x 128 f16 steps of 2 heads of 64, window 32, 166 us for 537 MB (3.2 TB/s).
template <class D, int W, int kBy, bool kAlone>
__global__ __launch_bounds__(256, (kAttBlocks<D, W>)) void attend_forward(const AttArgs x)
{
    using Tile = AttTile<D, W>;
    constexpr int BK = kAlone ? 32 : kKeyTile<D, W>, kBytes = BK * Tile::kRow, S = BK / 32;
    __shared__ alignas(1024) char lds[kAlone ? 4 : 2][2][kBytes];
    const int lane = threadIdx.x % kWave, h = lane >> 5;
    const AttBlock b(x, kAlone);
    if (kAlone && !b.any) return;
    const KeyTiles kt(x, b.n, b.first, b.last, BK);
    const WaveQueries wq(x, b.n, b.step0, kt.near, lane);
    OwnRows<D, W, kBy> q;
    q.load(x.q, b.n, wq.i - (x.TK - x.T), b.head, x.dim_k, wq.valid, lane);
    q.signs(x.scale < 0.0f);

    f32x16 o[W / 32] = {};
    float m = -INFINITY, l = 0.0f;  // m: the largest score; l: this half's sum
    auto compute = [&](uint32_t by_row, uint32_t by_col, bool is_far, int j0, int j1) {
        if (!wq.touches(kt, is_far, j0, j1)) return;
        f32x16 s[S] = {};
#pragma unroll
        for (int ks = 0; ks < W / 16; ++ks)
#pragma unroll
            for (int a = 0; a < S; ++a) s[a] = mma32<D>(Tile::rows(by_row, 32 * a, ks), q.f[ks], s[a]);
        if (!wq.whole(is_far, j0, j1, BK)) {
#pragma unroll
            for (int a = 0; a < S; ++a) keep_bits(wq.bits(is_far, j0 + 32 * a, j1, h), s[a], -INFINITY);
        }
        float top = s[0][0];
#pragma unroll
        for (int a = 0; a < S; ++a)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[a][r]);
        top = fmaxf(top, __shfl_xor(top, 32));
        // the sums are scaled again only when the largest score has grown by 2^8
        if (__any((top - m) * x.c > 8.0f)) {
            const float to = fmaxf(m, top);
            const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - to) * x.c);
            m = to;
            l *= f;
#pragma unroll
            for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[dt][r] *= f;
        }
        const float base = m == -INFINITY ? 0.0f : m * x.c;
#pragma unroll
        for (int a = 0; a < S; ++a)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[a][r] = __builtin_amdgcn_exp2f(fmaf(s[a][r], x.c, -base));
                l += s[a][r];
            }
#pragma unroll
        for (int a = 0; a < S; ++a)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const AFrag<D> p = operand<D>(s[a], u);
#pragma unroll
                for (int dt = 0; dt < W / 32; ++dt)
                    o[dt] = mma32<D>(Tile::columns(by_col + kBytes, 32 * a + 16 * u, 32 * dt), p, o[dt]);
            }
    };
    if constexpr (kAlone)
        over_keys_alone<D, W, BK, kBy, true>(x, b, kt, lds[__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)][0],
                                              lane, compute);
    else over_keys<D, W, BK, kBy, kKeySets<D, W>>(x, b, kt, lds[0][0], lane, compute);
    if (!wq.any()) return;
    l += __shfl_xor(l, 32);
    const float by = 1.0f / l, lse = (m * x.c + __builtin_amdgcn_logf(l)) * kAttLn2;
    const int t = wq.i - (x.TK - x.T);
    const bool fine = finite(o) && by < INFINITY && fabsf(lse) < INFINITY;
    if (wq.valid) {
        store_own<D, kBy>(seq_row_out<D>(x.o, b.n, t, b.head), o, by, x.dim_v, h);
        if (h == 0 && x.lse.p != nullptr) *seq_row_out<float>(x.lse, b.n, t, b.head) = lse;
    }
    uint64_t again = __ballot(wq.valid && !fine);
    for (again = (again | again >> 32) & 0xffffffffu; again != 0; again &= again - 1)
        careful_forward<D>(x, b.n, b.head, wq.first + __builtin_ctzll(again), lane);
}

// dq: S^T and dP^T = V dO^T by tiles, dS^T from both, dQ^T += K^T dS^T.  Registers bound it
// (own queries and gradients, sums and fragments: two waves on a SIMD): 8 x 2048 bf16 steps
// of 16 heads of 128, window 512, 183 us for 120 GF with the second part of dS, 650 TF/s.
// kSum: the pass before, for short windows, which only sums D as sum_j p_ij do_i . v_j.
template <class D, int W, int kBy, bool kSum, bool kAlone>
__global__ __launch_bounds__(256, (kAttBlocks<D, W>)) void attend_dq(const AttArgs x)
{
    using Tile = AttTile<D, W>;
    constexpr int BK = kAlone ? 32 : kGradTile<D, W>, kBytes = BK * Tile::kRow;
    __shared__ alignas(1024) char lds[kAlone ? 4 : 2][2][kBytes];
    const int lane = threadIdx.x % kWave, h = lane >> 5;
    const AttBlock b(x, kAlone);
    if (kAlone && !b.any) return;
    const KeyTiles kt(x, b.n, b.first, b.last, BK);
    const WaveQueries wq(x, b.n, b.step0, kt.near, lane);
    const int t = wq.i - (x.TK - x.T);
    OwnRows<D, W, kBy> q, d_o;
    q.load(x.q, b.n, t, b.head, x.dim_k, wq.valid, lane);
    q.signs(x.scale < 0.0f);
    d_o.load(x.dout, b.n, t, b.head, x.dim_v, wq.valid, lane);
    const float lse2 = (wq.valid ? *seq_row<float>(x.lse, b.n, t, b.head) : 0.0f) * kAttLog2e;
    float* const delta_at = x.delta + (b.n * x.H + b.head) * x.T + t;
    float delta = 0.0f;
    if (x.sum_delta) {
        if (!kSum && wq.valid) delta = *delta_at;
    } else {
        delta = own_dot<D, W, kBy>(x.o, b.n, t, b.head, x.dim_v, wq.valid, lane, d_o);
        if (wq.valid && h == 0) *delta_at = delta;
    }

    f32x16 dq[W / 32] = {};
    float sum = 0.0f;
    auto compute = [&](uint32_t by_row, uint32_t by_col, bool is_far, int j0, int j1) {
#pragma unroll
        for (int at = 0; at < BK; at += 32) {
            const int ja = j0 + at, jb = min(ja + 32, j1);
            if (ja >= j1 || !wq.touches(kt, is_far, ja, jb)) continue;
            f32x16 s = {}, dp = {};
            row_products<D, W, true, 1>(by_row, q, by_row + kBytes, d_o, at, s, dp);
            constexpr int N = W / 32;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                dp[r] = __builtin_amdgcn_exp2f(fmaf(s[r], x.c, -lse2)) * (dp[r] - delta);
            if (!wq.whole(is_far, ja, jb, 32)) keep_bits(wq.bits(is_far, ja, j1, h), dp, 0.0f);
            if constexpr (kSum) {
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += dp[r];
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const AFrag<D> ds = operand<D>(dp, u);
                    AFrag<D> rest;
                    if constexpr (sizeof(D) == 2) rest = operand_rest<D>(dp, u, ds);
#pragma unroll
                    for (int dt = 0; dt < N; ++dt) {
                        const AFrag<D> k = Tile::columns(by_col, at + 16 * u, 32 * dt);
                        dq[dt] = mma32<D>(k, ds, dq[dt]);
                        if constexpr (sizeof(D) == 2) dq[dt] = mma32<D>(k, rest, dq[dt]);
                    }
                }
            }
        }
    };
    if constexpr (kAlone)
        over_keys_alone<D, W, BK, kBy, false>(x, b, kt, lds[__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)][0],
                                              lane, compute);
    else over_keys<D, W, BK, kBy, kGradSets<D, W>>(x, b, kt, lds[0][0], lane, compute);
    if constexpr (kSum) {
        sum += __shfl_xor(sum, 32);
        if (wq.valid && h == 0) *delta_at = sum;
        return;
    }
    if (!wq.any()) return;
    const bool fine = finite(dq);
    if (wq.valid)
        store_own<D, kBy>(seq_row_out<D>(x.dq, b.n, t, b.head), dq, x.scale, x.dim_k, h);
    uint64_t again = __ballot(wq.valid && !fine);
    for (again = (again | again >> 32) & 0xffffffffu; again != 0; again &= again - 1)
        careful_dq<D>(x, b.n, b.head, wq.first + __builtin_ctzll(again), lane);
}

// float16 weights go into the products 2^10 times as large: a key's weights may all
// be small (1 / window and less), and below 2^-14 float16 has ever fewer bits.
template <class D>
constexpr float kWeightBits = std::is_same<D, f16_t>::value ? 10.0f : 0.0f;

// What goes with a tile of queries: their lse (in powers of two, as the weights take
// it) and D.
template <int kRows>
struct QueryRows {
    alignas(16) float lse2[kRows], delta[kRows];
};

template <class D>
constexpr float kLessWeight = kWeightBits<D> == 0.0f ? 1.0f : 0x1p-10f;

// Tiles of queries and their gradients on their way to LDS, one behind the other.
template <class D, int W, int kBy, int kRows, int kThreads, int kSets = 1>
struct QueryStage {
    AttStage<D, W, kRows, kBy, kThreads, kSets> q, d_o;
    const char *lse_p, *delta_p;
    int64_t lse_step;
    float lse[kSets], delta[kSets];

    __device__ __forceinline__ void start(const AttArgs& x)
    {
        q.start(x.q, x.dim_k);
        d_o.start(x.dout, x.dim_v);
        lse_step = x.lse.step * 4;
    }
    // The next tile begins at query t of a head.
    __device__ __forceinline__ void place(const AttArgs& x, int64_t n, int head, int t)
    {
        q.place(x.q, n, head, t);
        d_o.place(x.dout, n, head, t);
        lse_p = att_row<float>(x.lse, n, t, head);
        delta_p = reinterpret_cast<const char*>(x.delta + (n * x.H + head) * x.T + t);
    }
    // (queries behind the last one are seen by no key: what is loaded for them is not used)
    template <int set = 0>
    __device__ __forceinline__ void fetch(int left)
    {
        const int count = min(kRows, left), a = threadIdx.x % kRows;
        q.template fetch<set>(count);
        d_o.template fetch<set>(count);
        const int at = min(a, count - 1);
        lse[set] = *reinterpret_cast<const float*>(lse_p + at * lse_step);
        delta[set] = reinterpret_cast<const float*>(delta_p)[at];
        lse_p += kRows * lse_step;
        delta_p += kRows * 4;
    }
    // at: from q.lane(); the gradients' tile lies `apart` behind the queries'.
    template <int set = 0>
    __device__ __forceinline__ void put(uint32_t at, int apart, QueryRows<kRows>& rows) const
    {
        q.template put<set>(at);
        d_o.template put<set>(at + apart);
        if (threadIdx.x % kThreads < kRows) {
            const int a = threadIdx.x % kRows;
            rows.lse2[a] = fmaf(lse[set], kAttLog2e, -kWeightBits<D>);
            rows.delta[a] = delta[set] * kLessWeight<D>;
        }
    }
};

// Adds what 32 queries in LDS give to the gradients of the wave's keys: of the keys
// (kK), of the values (kV).  bits: the rows whose queries see the lane's key; not
// looked at where `whole`.
template <class D, int W, int kBy, bool kK, bool kV, class Rows>
__device__ __forceinline__ void add_queries(const AttArgs& x, uint32_t by_row, uint32_t by_col, int apart, const Rows& row, int at,
                                            const OwnRows<D, W, kBy>& k, const OwnRows<D, W, kBy>& v, bool whole,
                                            uint32_t bits, int lane, f32x16 (&dk)[W / 32], f32x16 (&dv)[W / 32])
{
    using Tile = AttTile<D, W>;
    constexpr float kLess = kLessWeight<D>;
    constexpr int N = W / 32;
    const int h = lane >> 5;
    f32x16 s = {}, dp = {};
    row_products<D, W, kK, 1>(by_row, k, by_row + apart, v, at, s, dp);
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
        const f32x4 lse2 = *reinterpret_cast<const f32x4*>(&row.lse2[at + 8 * r4 + 4 * h]);
        const f32x4 delta = *reinterpret_cast<const f32x4*>(&row.delta[at + 8 * r4 + 4 * h]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 4 * r4 + e;
            s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], x.c, -lse2[e]));
            if constexpr (kK) dp[r] = s[r] * (kLess == 1.0f ? dp[r] - delta[e] : fmaf(dp[r], kLess, -delta[e]));
        }
    }
    if (!whole) {
        if constexpr (kV) keep_bits(bits, s, 0.0f);
        if constexpr (kK) keep_bits(bits, dp, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        AFrag<D> p, ds, rest;
        if constexpr (kV) p = operand<D>(s, u);
        if constexpr (kK) ds = operand<D>(dp, u);
        if constexpr (kK && sizeof(D) == 2) rest = operand_rest<D>(dp, u, ds);
#pragma unroll
        for (int dt = 0; dt < N; ++dt) {
            if constexpr (kV) dv[dt] = mma32<D>(Tile::columns(by_col + apart, at + 16 * u, 32 * dt), p, dv[dt]);
            if constexpr (kK) {
                const AFrag<D> q = Tile::columns(by_col, at + 16 * u, 32 * dt);
                dk[dt] = mma32<D>(q, ds, dk[dt]);
                if constexpr (sizeof(D) == 2) dk[dt] = mma32<D>(q, rest, dk[dt]);
            }
        }
    }
}

// First steps of an episode are seen by all of its queries.  Those beyond the end of
// the chunk of kFarChunk steps that the episode begins in are left to a kernel of
// their own (attend_far), a block to a chunk, which keeps the sums of each chunk
// apart for attend_dkv to join: or one block would walk the whole episode.
constexpr int kFarChunk = 256;
constexpr int kFarSinks = 64;  // with more first steps than this attend_dkv does it all

// Where a chunk's sums of first step s are: W of its key's gradient, W of its value's.
template <int W>
__device__ __forceinline__ float* far_sums(const AttArgs& x, int64_t row, int chunk, int s)
{
    return x.far_part + ((row * x.far_chunks + chunk) * x.sinks + s) * (2 * W);
}

// Queries in a tile of attend_dkv, and tiles on their way from memory.
template <class D, int W>
constexpr int kQueryTile = W == 128 || sizeof(D) == 2 ? 32 : 64;
template <class D, int W>
constexpr int kQuerySets = sizeof(D) == 4 ? 1 : 2;

// Rows of more than 128 bytes take a kernel for the gradient of the keys (kK) and one
// for that of the values (kV): together they need more registers than two waves on a
// SIMD have, and one wave alone waits through its softmax.
template <class D, int W>
constexpr bool kSplitGrads = W * (int)sizeof(D) > 128;

// The queries that see key j are those from j to here (in attend_dkv: without those of
// later chunks, which attend_far does).
__device__ __forceinline__ int seen_until(const AttArgs& x, int64_t n, int j)
{
    const int start = episode_start(x, n, j), end = x.ends != nullptr ? x.ends[n * x.TK + j] : x.TK;
    int until = j + min(x.window, x.TK - j);
    if (j < start + x.sinks)
        until = max(until, x.far_part != nullptr ? (start / kFarChunk + 1) * kFarChunk : x.TK);
    return min(until, end);
}

// Keys are the columns: a wave holds 32 of them and their values, a block 128;
// queries and their gradients come in tiles, head after head of the group, so that what
// shared heads give is summed in registers.  S = Q K^T and dP = dO V^T by tiles, dK^T +=
// Q^T dS, dV^T += dO^T P.  Bound as dq is: at its sizes 182 us for dk and 128 for dv.
// Alone: each wave has its own tiles.
template <class D, int W, int kBy, bool kK, bool kV, bool kAlone>
__global__ __launch_bounds__(256, (sizeof(D) == 4 && W == 128 ? 1 : 2)) void attend_dkv(const AttArgs x)
{
    using Tile = AttTile<D, W>;
    constexpr int BQ = kAlone ? 32 : kQueryTile<D, W>;
    constexpr int kBytes = BQ * Tile::kRow;
    __shared__ alignas(1024) char lds[kAlone ? 4 : 2][2][kBytes];
    __shared__ QueryRows<BQ> rows[kAlone ? 4 : 2];
    const int lane = threadIdx.x % kWave, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int past = x.TK - x.T, kv = x.H / x.group;
    const uint32_t block = by_xcd(blockIdx.x, gridDim.x), id = kAlone ? block * 4 + wave : block;
    const uint32_t row_of = id / x.tiles;
    const int64_t n = row_of / kv;
    const int kvh = row_of % kv;
    if (kAlone && n >= x.N) return;
    constexpr int kKeys = kAlone ? 32 : 128;
    const int j0 = (int)(id - row_of * x.tiles) * kKeys, j1 = min(j0 + kKeys, x.TK);
    const int mine0 = kAlone ? j0 : j0 + 32 * wave, j = mine0 + (lane & 31);
    const bool valid = j < x.TK;
    OwnRows<D, W, kBy> k, v;
    k.load(x.k, n, min(j, x.TK - 1), kvh, x.dim_k, valid, lane);
    k.signs(x.scale < 0.0f);
    if constexpr (kK) v.load(x.v, n, min(j, x.TK - 1), kvh, x.dim_v, valid, lane);

    // The queries that see the lane's key, the wave's keys, and one of the block's.
    const int until = valid ? seen_until(x, n, j) : 0;
    int most = until, least = until;
    for (int o = 16; o > 0; o >>= 1) {
        most = max(most, __shfl_xor(most, o));
        least = min(least, __shfl_xor(least, o));
    }
    most = __builtin_amdgcn_readfirstlane(most);
    least = __builtin_amdgcn_readfirstlane(least);
    int end = 0;
    for (int a = j0 + lane; a < j1; a += kWave) end = max(end, seen_until(x, n, a));
    for (int o = 32; o > 0; o >>= 1) end = max(end, __shfl_xor(end, o));
    end = __builtin_amdgcn_readfirstlane(end);
    const int begin = max(j0, past);

    f32x16 dk[W / 32] = {}, dv[W / 32] = {};
    const int tiles = end > begin ? (end - begin + BQ - 1) / BQ : 0, total = tiles * x.group;
    if constexpr (kAlone) {
        QueryStage<D, W, kBy, BQ, kWave> stage;
        stage.start(x);
        const uint32_t at = lds_address(lds[wave]), put_at = stage.q.lane(at);
        for (int head = kvh * x.group; total > 0 && head < (kvh + 1) * x.group; ++head) {
            stage.place(x, n, head, begin - past);
            for (int i = begin; i < end; i += BQ) {
                stage.fetch(end - i);
                stage.put(put_at, kBytes, rows[wave]);
                __builtin_amdgcn_wave_barrier();
                const bool whole = mine0 + 31 <= i && i + 32 <= least;
                add_queries<D, W, kBy, kK, kV>(x, at + Tile::row_lane(lane), at + Tile::column_lane(lane), kBytes,
                                               rows[wave], 0, k, v, whole, whole ? 0 : row_bits(j, until, i, h), lane,
                                               dk, dv);
                __builtin_amdgcn_wave_barrier();
            }
        }
    } else if (total > 0) {
        // tiles are loaded two ahead: what one tile takes to compute is less than a load takes
        QueryStage<D, W, kBy, BQ, 256, kQuerySets<D, W>> stage;
        stage.start(x);
        uint32_t by_row = lds_address(lds) + Tile::row_lane(lane), by_col = lds_address(lds) + Tile::column_lane(lane);
        uint32_t put_at = stage.q.lane(lds_address(lds));
        int tile = 0, next_head = kvh * x.group, next = 0, fetched = 0;
        auto fetch = [&](auto set) {
            if (fetched == total) return;
            ++fetched;
            if (next == 0) stage.place(x, n, next_head, begin - past);
            stage.template fetch<decltype(set)::value>(end - begin - next * BQ);
            if (++next == tiles) {
                next = 0;
                ++next_head;
            }
        };
        // Tile `it`, with the one behind it put down from `set` and another fetched into that.
        auto step = [&](int it, auto set) {
            __syncthreads();
            const QueryRows<BQ>& row = rows[it & 1];
#pragma unroll
            for (int at = 0; at < BQ; at += 32) {
                const int i = begin + tile * BQ + at;
                if (i < most && mine0 <= i + 31) {
                    // whole: every query of the tile sees every key of the wave
                    const bool whole = mine0 + 31 <= i && i + 32 <= least;
                    add_queries<D, W, kBy, kK, kV>(x, by_row, by_col, kBytes, row, at, k, v, whole,
                                                     whole ? 0 : row_bits(j, until, i, h), lane, dk, dv);
                }
            }
            if (++tile == tiles) tile = 0;
            const uint32_t move = it & 1 ? -2 * kBytes : 2 * kBytes;
            by_row += move;
            by_col += move;
            put_at += move;
            if (it + 1 < total) {
                stage.template put<decltype(set)::value>(put_at, kBytes, rows[(it + 1) & 1]);
                fetch(set);
            }
        };
        constexpr std::integral_constant<int, 0> s0{};
        constexpr std::integral_constant<int, kQuerySets<D, W> - 1> s1{};
        fetch(s0);
        stage.template put<0>(put_at, kBytes, rows[0]);
        fetch(s1);
        if constexpr (kQuerySets<D, W> == 2) fetch(s0);
        for (int it = 0; it < total; it += 2) {
            step(it, s1);
            if (it + 1 < total) step(it + 1, s0);
        }
    }
    constexpr float kLess = kLessWeight<D>;
    const int first = episode_start(x, n, min(j, x.TK - 1));
    if (x.far_part != nullptr && __any(valid && j < first + x.sinks)) {
        // the chunks after the first, up to the episode's end
        const int s = j - first;
        const int last = valid && s < x.sinks ? (x.ends != nullptr ? x.ends[n * x.TK + j] : x.TK) - 1 : -1;
        const int c0 = max(first / kFarChunk + 1, past / kFarChunk);
        auto add = [&](f32x16(&acc)[W / 32], int from) {
            const float* at = far_sums<W>(x, n * kv + kvh, c0, s) + from + 4 * h;
            for (int c = c0; c <= last / kFarChunk; ++c, at += (int64_t)x.sinks * 2 * W) {
                f32x4 v[W / 32][4];
#pragma unroll
                for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4) v[dt][r4] = *reinterpret_cast<const f32x4*>(at + 32 * dt + 8 * r4);
#pragma unroll
                for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[dt][r] += v[dt][r / 4][r % 4];
            }
        };
        if constexpr (kK) add(dk, 0);
        if constexpr (kV) add(dv, W);
    }
    bool fine = true;
    if constexpr (kK) fine = finite(dk);
    if constexpr (kV) fine = fine && finite(dv);
    if (valid) {
        if constexpr (kK) store_own<D, kBy>(seq_row_out<D>(x.dk, n, j, kvh), dk, x.scale, x.dim_k, h);
        if constexpr (kV) store_own<D, kBy>(seq_row_out<D>(x.dv, n, j, kvh), dv, kLess, x.dim_v, h);
    }
    uint64_t again = __ballot(valid && !fine);
    for (again = (again | again >> 32) & 0xffffffffu; again != 0; again &= again - 1)
        careful_dkv<D, kK, kV>(x, n, kvh, mine0 + __builtin_ctzll(again), lane);
}

// What the queries of one chunk beyond its window give to 32 first steps of the
// episode that the chunk begins in the middle of, summed over the heads that share
// them: a quarter of the chunk to each wave, joined through LDS.  One kernel for both
// gradients, with a block's waves alone on their SIMDs: 46 us at the sizes above with 4
// first steps, 70 as a kernel for each.  Reading queries and their gradients once more
// takes 26 of them at the rate of a copy.
template <class D, int W, int kBy>
__global__ __launch_bounds__(256, 1) void attend_far(const AttArgs x)
{
    using Tile = AttTile<D, W>;
    constexpr int BQ = 32, kBytes = BQ * Tile::kRow, kPart = kFarChunk / 4;
    // a wave's two tiles, and after them its sums (W x 32 values)
    constexpr int kRegion = 2 * kBytes > W * 128 ? 2 * kBytes : W * 128;
    __shared__ alignas(1024) char lds[4][kRegion];
    __shared__ QueryRows<BQ> rows[4];
    const int lane = threadIdx.x % kWave, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int past = x.TK - x.T, kv = x.H / x.group, chunks = x.far_chunks, parts = (x.sinks + 31) / 32;
    uint32_t id = blockIdx.x;
    const int part = id % parts;
    id /= parts;
    const int c = id % chunks;
    id /= chunks;
    const int kvh = id % kv;
    const int64_t n = id / kv;
    const int i0 = c * kFarChunk, i1 = min(i0 + kFarChunk, x.TK);
    const int first = episode_start(x, n, i0);
    if (i1 <= past || first / kFarChunk == c) return;  // (the whole block)
    const int s = 32 * part + (lane & 31), j = first + s;
    const bool valid = s < x.sinks && j < x.TK;
    OwnRows<D, W, kBy> k, v;
    k.load(x.k, n, min(j, x.TK - 1), kvh, x.dim_k, valid, lane);
    k.signs(x.scale < 0.0f);
    v.load(x.v, n, min(j, x.TK - 1), kvh, x.dim_v, valid, lane);
    const int begin = max(max(i0 + wave * kPart, past), first + 32 * part + x.window);
    const int end = min(min(i1, i0 + (wave + 1) * kPart), x.ends != nullptr ? x.ends[n * x.TK + first] : x.TK);
    f32x16 dk[W / 32] = {}, dv[W / 32] = {};
    QueryStage<D, W, kBy, BQ, kWave> stage;
    stage.start(x);
    const uint32_t mine = lds_address(lds[wave]), by_row = mine + Tile::row_lane(lane);
    const uint32_t by_col = mine + Tile::column_lane(lane), put_at = stage.q.lane(mine);
    for (int head = kvh * x.group; begin < end && head < (kvh + 1) * x.group; ++head) {
        stage.place(x, n, head, begin - past);
        for (int i = begin; i < end; i += BQ) {
            stage.fetch(end - i);
            stage.put(put_at, kBytes, rows[wave]);
            __builtin_amdgcn_wave_barrier();
            add_queries<D, W, kBy, true, true>(x, by_row, by_col, kBytes, rows[wave], 0, k, v, false,
                                             valid ? row_bits(j + x.window, end, i, h) : 0, lane, dk, dv);
            __builtin_amdgcn_wave_barrier();
        }
    }
    float* const to = far_sums<W>(x, n * kv + kvh, c, s);
    auto join = [&](const f32x16(&acc)[W / 32], int from) {
        __syncthreads();
        float* const own = reinterpret_cast<float*>(lds[wave]);
#pragma unroll
        for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
            for (int r = 0; r < 16; ++r) own[(16 * dt + r) * kWave + lane] = acc[dt][r];
        __syncthreads();
        // a quarter of the values to each wave: registers 4 wave .. 4 wave + 3 of each tile
        if (s >= x.sinks) return;
#pragma unroll
        for (int dt = 0; dt < W / 32; ++dt) {
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] += reinterpret_cast<const float*>(lds[w])[(16 * dt + 4 * wave + e) * kWave + lane];
            *reinterpret_cast<f32x4*>(to + from + 32 * dt + 8 * wave + 4 * h) = sum;
        }
    };
    join(dk, 0);
    join(dv, W);
}

// The first step of each step's episode and the step behind its last, [N, TK]: a
// running maximum of the steps where the reset mask is set, and a running minimum of
// those from the end, one block to a row.
template <bool kEnds>
__device__ __forceinline__ void episode_bounds(const SeqView& reset, int64_t n, int32_t TK, int32_t* out, int* part)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    int carry = 0;
    for (int t0 = 0; t0 < TK; t0 += 256) {
        // ends: from the last step backwards, by how far the next first step lies before TK
        const int t = kEnds ? TK - 1 - t0 - (int)threadIdx.x : t0 + (int)threadIdx.x;
        const int at = kEnds ? t + 1 : t;
        int v = 0;
        if (at >= 0 && at < TK && *seq_row<uint8_t>(reset, n, at, 0) != 0) v = kEnds ? TK - at : at;
        for (int o = 1; o < kWave; o <<= 1) {
            const int u = __shfl_up(v, o);
            if (lane >= o) v = max(v, u);
        }
        if (lane == kWave - 1) part[wave] = v;
        __syncthreads();
        v = max(v, carry);
        for (int w = 0; w < wave; ++w) v = max(v, part[w]);
        for (int w = 0; w < 4; ++w) carry = max(carry, part[w]);
        if (t >= 0 && t < TK) out[n * TK + t] = kEnds ? TK - v : v;
        __syncthreads();
    }
}

static __global__ __launch_bounds__(256) void episodes(const SeqView reset, int64_t N, int32_t TK, int32_t* starts,
                                                       int32_t* ends)
{
    __shared__ int part[4];
    const int64_t n = blockIdx.x % N;
    if (blockIdx.x < N) episode_bounds<false>(reset, n, TK, starts, part);
    else episode_bounds<true>(reset, n, TK, ends, part);
}

// ------------------------------------------------------------- single steps
// One step of an environment at position p of its episode: its key and value go
// into slot p (p < sinks) or sinks + (p - sinks) % window of the caches, and its
// query sees the first min(p + 1, sinks + window) slots: what the ring holds is
// the window, and the order of a softmax's terms is free.

struct AttStepArgs {
    SeqView q, k, v, kc, vc, o;  // kc, vc: the slots are the steps
    const int32_t* positions;
    float* part;                 // splits > 1: [N, H, splits, dim_v + 2]
    int32_t KV, group, chunks, splits, per_split, sinks, window, dim_k, dim_v;
    float c;                     // scale log2(e)
    uint8_t wide;                // rows are whole 16-byte units
};

// What lane i of 2^k neighbours has in common with the others: their sum.
template <int N>
__device__ __forceinline__ float lanes_sum(float v)
{
    auto dpp = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                  0xf, 0xf, true));
    };
    if constexpr (N >= 2) v += dpp(v, std::integral_constant<int, 0xb1>{});   // quad_perm 1,0,3,2
    if constexpr (N >= 4) v += dpp(v, std::integral_constant<int, 0x4e>{});   // quad_perm 2,3,0,1
    if constexpr (N >= 8) v += dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
    if constexpr (N >= 16) v += dpp(v, std::integral_constant<int, 0x140>{}); // row_mirror
    if constexpr (N >= 32) v += __shfl_xor(v, 16);
    return v;
}

// A 16-byte unit of a row from element c on, zeros beyond dim.
template <class D>
__device__ __forceinline__ u32x4 load_unit(const D* row, int c, int dim, bool wide)
{
    constexpr int E = 16 / (int)sizeof(D);
    u32x4 w = {};
    if (wide) {
        if (c < dim) w = *reinterpret_cast<const u32x4*>(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e < dim) {
                if constexpr (sizeof(D) == 4) w[e] = reinterpret_cast<const uint32_t*>(row)[c + e];
                else w[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[c + e] << (16 * (e & 1));
            }
    }
    return w;
}

template <class D>
__device__ __forceinline__ void store_row_unit(D* row, int c, int dim, bool wide, const u32x4& w)
{
    constexpr int E = 16 / (int)sizeof(D);
    if (wide) {
        if (c < dim) *reinterpret_cast<u32x4*>(row + c) = w;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e < dim) {
                if constexpr (sizeof(D) == 4) reinterpret_cast<uint32_t*>(row)[c + e] = w[e];
                else reinterpret_cast<uint16_t*>(row)[c + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            }
    }
}

template <class D>
__device__ __forceinline__ void unit_f32(const u32x4& w, float (&v)[16 / sizeof(D)])
{
    if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack2<D>(w[e], v[2 * e], v[2 * e + 1]);
    }
}

// LR lanes hold a row of a cache, 16 bytes each, a wave 64 / LR rows at a time, and
// G query heads of a key head are served at once.  Each group of LR lanes keeps a
// running maximum and sum of its own; groups, waves and splits are joined after.  The
// caches' bytes bound it: 4096 environments of 4 heads of 64 with 132 slots 114 us (5.0
// TB/s), 16 of 32 heads over 8 of 128 with 8208 slots 133 us, 9 of them in the join.
template <class D, int LR, int G>
__global__ __launch_bounds__(256) void attend_step(const AttStepArgs x)
{
    constexpr int E = 16 / (int)sizeof(D), R = kWave / LR, U = 4;
    __shared__ float sm[4][G], sl[4][G], sa[4][G][LR * E];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    uint32_t id = blockIdx.x;
    const int split = id % x.splits;
    id /= x.splits;
    const int chunk = id % x.chunks;
    id /= x.chunks;
    const int kvh = id % x.KV;
    const int64_t n = id / x.KV;
    const int head0 = kvh * x.group + chunk * G, heads = min(G, x.group - chunk * G);
    const int slots = x.sinks + x.window;
    const int64_t p = x.positions[n];
    if (p < 0) {  // this environment waits
        if (split == 0)
            for (int a = threadIdx.x; a < heads * x.dim_v; a += 256)
                seq_row_out<D>(x.o, n, 0, head0 + a / x.dim_v)[a % x.dim_v] = from_f32<D>(0.0f);
        return;
    }
    const int count = (int)min(p + 1, (int64_t)slots);
    const int mine = (int)(p < x.sinks ? p : x.sinks + (p - x.sinks) % x.window);
    const int begin = split * x.per_split, end = min(begin + x.per_split, count);
    const int c = lane % LR * E, r = lane / LR;
    const D *const kin = seq_row<D>(x.k, n, 0, kvh), *const vin = seq_row<D>(x.v, n, 0, kvh);

    // the step's own key and value go into its slot; every block takes them from k and v
    if (chunk == 0 && mine >= begin && mine < begin + x.per_split && wave == 0 && r == 0) {
        store_row_unit<D>(seq_row_out<D>(x.kc, n, mine, kvh), c, x.dim_k, x.wide, load_unit<D>(kin, c, x.dim_k, x.wide));
        store_row_unit<D>(seq_row_out<D>(x.vc, n, mine, kvh), c, x.dim_v, x.wide, load_unit<D>(vin, c, x.dim_v, x.wide));
    }
    float q[G][E], acc[G][E] = {}, m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        u32x4 w = {};
        if (g < heads) w = load_unit<D>(seq_row<D>(x.q, n, 0, head0 + g), c, x.dim_k, x.wide);
        unit_f32<D>(w, q[g]);
#pragma unroll
        for (int e = 0; e < E; ++e) q[g][e] *= x.c;
        m[g] = -INFINITY;
        l[g] = 0.0f;
    }
    for (int s0 = begin + wave * R * U + r; s0 < end; s0 += 4 * R * U) {
        u32x4 kw[U], vw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * R;
            kw[u] = vw[u] = u32x4{};
            if (s < end) {
                kw[u] = load_unit<D>(s == mine ? kin : seq_row<D>(x.kc, n, s, kvh), c, x.dim_k, x.wide);
                vw[u] = load_unit<D>(s == mine ? vin : seq_row<D>(x.vc, n, s, kvh), c, x.dim_v, x.wide);
            }
        }
        float s[G][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float kf[E];
            unit_f32<D>(kw[u], kf);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float d = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) d = fmaf(q[g][e], kf[e], d);
                d = lanes_sum<LR>(d);
                s[g][u] = s0 + u * R < end ? d : -INFINITY;
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float top = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, s[g][u]);
            const float f = m[g] == top ? 1.0f : __builtin_amdgcn_exp2f(m[g] - top);
            m[g] = top;
            l[g] *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[g][e] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // slots behind the end have a weight of 0 even where no score is above -infinity
                s[g][u] = s0 + u * R < end ? __builtin_amdgcn_exp2f(s[g][u] - top) : 0.0f;
                l[g] += s[g][u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float vf[E];
            unit_f32<D>(vw[u], vf);
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[g][e] = fmaf(s[g][u], vf[e], acc[g][e]);
        }
    }
    // groups of lanes, then waves
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float top = m[g];
#pragma unroll
        for (int o = LR; o < kWave; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        const float f = m[g] == top ? 1.0f : __builtin_amdgcn_exp2f(m[g] - top);
        l[g] *= f;
#pragma unroll
        for (int o = LR; o < kWave; o <<= 1) l[g] += __shfl_xor(l[g], o);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float a = acc[g][e] * f;
#pragma unroll
            for (int o = LR; o < kWave; o <<= 1) a += __shfl_xor(a, o);
            if (r == 0) sa[wave][g][c + e] = a;
        }
        if (lane == 0) {
            sm[wave][g] = top;
            sl[wave][g] = l[g];
        }
    }
    __syncthreads();
    for (int a = threadIdx.x; a < heads * x.dim_v; a += 256) {
        const int g = a / x.dim_v, d = a % x.dim_v;
        float top = sm[0][g], sum = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 1; w < 4; ++w) top = fmaxf(top, sm[w][g]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = sm[w][g] == top ? 1.0f : __builtin_amdgcn_exp2f(sm[w][g] - top);
            sum = fmaf(sl[w][g], f, sum);
            v = fmaf(sa[w][g][d], f, v);
        }
        if (x.splits == 1) {
            seq_row_out<D>(x.o, n, 0, head0 + g)[d] = from_f32<D>(v / sum);
        } else {
            float* const to = x.part + ((n * x.KV * x.group + head0 + g) * x.splits + split) * (x.dim_v + 2);
            to[d] = v;
            if (d == 0) {
                to[x.dim_v] = top;
                to[x.dim_v + 1] = sum;
            }
        }
    }
}

// Joins the splits of a head, in their order.
template <class D>
__global__ __launch_bounds__(128) void join_step(const AttStepArgs x)
{
    const int H = x.KV * x.group, head = blockIdx.x % H, d = threadIdx.x;
    const int64_t n = blockIdx.x / H;
    if (d >= x.dim_v || x.positions[n] < 0) return;
    const float* const from = x.part + (int64_t)blockIdx.x * x.splits * (x.dim_v + 2);
    float top = -INFINITY, sum = 0.0f, v = 0.0f;
    for (int s = 0; s < x.splits; ++s) top = fmaxf(top, from[s * (x.dim_v + 2) + x.dim_v]);
    for (int s = 0; s < x.splits; ++s) {
        const float* const at = from + s * (x.dim_v + 2);
        const float f = at[x.dim_v] == top ? 1.0f : __builtin_amdgcn_exp2f(at[x.dim_v] - top);
        sum = fmaf(at[x.dim_v + 1], f, sum);
        v = fmaf(at[d], f, v);
    }
    seq_row_out<D>(x.o, n, 0, head)[d] = from_f32<D>(v / sum);
}

// The caches after the last episode of each row of k and v, slot by slot: a slot
// takes the last step that belongs into it, if the row has one.
struct AttFillArgs {
    SeqView k, v, kc, vc, positions;
    int64_t N;
    int32_t T, KV, sinks, window, dim_k, dim_v;
};

template <class D>
__global__ __launch_bounds__(256) void fill_slots(const AttFillArgs x, const uint32_t wide)
{
    constexpr int E = 16 / (int)sizeof(D);
    const int slots = x.sinks + x.window, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int uk = (x.dim_k + E - 1) / E, uv = (x.dim_v + E - 1) / E;
    for (int64_t at = (int64_t)blockIdx.x * 4 + wave; at < x.N * slots; at += (int64_t)gridDim.x * 4) {
        const int64_t n = at / slots;
        const int slot = (int)(at % slots);
        const int64_t last = *seq_row<int32_t>(x.positions, n, x.T - 1, 0);
        int64_t p = slot;
        if (slot >= x.sinks && last >= slot) p = slot + (last - slot) / x.window * x.window;
        const int64_t t = x.T - 1 - (last - p);
        if (p > last || t < 0) continue;
        for (int a = lane; a < x.KV * (uk + uv); a += kWave) {
            const bool key = a < x.KV * uk;
            const int b = key ? a : a - x.KV * uk, u = key ? uk : uv, h = b / u, c = b % u * E;
            const int dim = key ? x.dim_k : x.dim_v;
            const SeqView &from = key ? x.k : x.v, &to = key ? x.kc : x.vc;
            store_row_unit<D>(seq_row_out<D>(to, n, slot, h), c, dim, wide,
                              load_unit<D>(seq_row<D>(from, n, t, h), c, dim, wide));
        }
    }
}

// ------------------------------------------------------------------ entries

inline bool att_sizes_ok(int64_t H, int64_t KV, int64_t dk, int64_t dv)
{
    return KV >= 1 && H >= 1 && H <= 65536 && H % KV == 0 && dk >= 1 && dv >= 1 && dk <= kMaxAttDim &&
           dv <= kMaxAttDim;
}

inline lrs_status check_attention(const char* nm, int64_t N, int64_t T, int64_t TK, int64_t H, int64_t KV,
                                  int64_t dk, int64_t dv, int64_t window, int64_t sinks, float scale)
{
    LRS_TRY(check_common(nm, N, T));
    LRS_REQUIRE(TK >= T && TK <= kMaxKeySteps && valid_sizes(N, TK),
                "%s: key_steps must be at least query_steps and at most 2^29, and num_envs * key_steps < 2^34", nm);
    LRS_REQUIRE(KV >= 1 && H >= 1 && H <= 65536 && H % KV == 0,
                "%s: heads must be a multiple of kv_heads and 1 to 65536 (got %lld and %lld)", nm, (long long)H,
                (long long)KV);
    LRS_REQUIRE(dk >= 1 && dv >= 1 && dk <= kMaxAttDim && dv <= kMaxAttDim,
                "%s: key_dim and value_dim must be 1 to %d (got %lld and %lld)", nm, kMaxAttDim, (long long)dk,
                (long long)dv);
    LRS_REQUIRE(window >= 1, "%s: window must be at least 1 (got %lld)", nm, (long long)window);
    LRS_REQUIRE(sinks >= 0 && sinks < (int64_t(1) << 31), "%s: sinks must be 0 or more (got %lld)", nm,
                (long long)sinks);
    LRS_REQUIRE(scale - scale == 0.0f && scale != 0.0f && std::abs(scale) * kAttLog2e <= 1e30f,
                "%s: scale must be finite and not 0", nm);
    return LRS_OK;
}

// How wide the accesses to an array's rows may be, in bytes.
inline void set_vec(SeqView& v, int64_t dim, int s)
{
    v.vec = rows_on(v, 16 / s, s) && dim % 8 == 0 ? 16 : rows_on(v, 4 / s, s) && dim % (4 / s) == 0 ? 4 : s;
}

// Where the parts of a call's workspace lie, in bytes.
struct AttWorkspace {
    size_t ends, delta, far_part, bytes;
    int32_t far_chunks;
};

inline AttWorkspace att_workspace(int64_t N, int64_t T, int64_t TK, int64_t H, int64_t KV, int64_t dk, int64_t dv,
                                  int64_t window, int64_t sinks, bool reset, bool backward)
{
    auto whole = [](size_t b) { return (b + 255) / 256 * 256; };
    AttWorkspace w{};
    if (reset) w.bytes += whole((size_t)(N * TK) * 4);
    w.ends = w.bytes;
    if (!backward) return w;
    if (reset) w.bytes += whole((size_t)(N * TK) * 4);
    w.delta = w.bytes;
    w.bytes += whole((size_t)(N * T * H) * 4);
    w.far_part = w.bytes;
    // a chunk after an episode's first has queries that see its first steps by these alone
    if (sinks > 0 && sinks <= kFarSinks && window < TK && TK > kFarChunk) {
        w.far_chunks = (int32_t)((TK + kFarChunk - 1) / kFarChunk);
        w.bytes += whole((size_t)(N * KV) * w.far_chunks * (size_t)std::min(sinks, TK) *
                         (std::max(dk, dv) <= 64 ? 128 : 256) * 4);
    }
    return w;
}

inline void fill_attention(AttArgs& x, const AttWorkspace& w, int64_t N, int64_t T, int64_t TK, int64_t H, int64_t KV,
                           int64_t dk, int64_t dv, int64_t window, int64_t sinks, float scale, const void* reset,
                           void* ws)
{
    x.N = N;
    x.T = (int32_t)T;
    x.TK = (int32_t)TK;
    x.H = (int32_t)H;
    x.group = (int32_t)(H / KV);
    x.window = (int32_t)std::min(window, TK);
    x.sinks = (int32_t)std::min(sinks, TK);
    x.dim_k = (int32_t)dk;
    x.dim_v = (int32_t)dv;
    x.scale = scale;
    x.c = std::abs(scale) * kAttLog2e;
    // D from the rounded results is off by their rounding, which counts where few weights
    // share a query: gradients of 16-bit types were off by twice the rounding of their own
    // at a window of 2, 1.4 times at 4, by nothing to be seen from 30 on.
    x.sum_delta = x.window <= 16;
    x.hpb = x.group % 4 == 0 ? 4 : x.group % 2 == 0 ? 2 : 1;
    char* const at = static_cast<char*>(ws);
    x.starts = reset != nullptr ? reinterpret_cast<const int32_t*>(at) : nullptr;
    x.ends = reset != nullptr && w.delta > 0 ? reinterpret_cast<const int32_t*>(at + w.ends) : nullptr;
    x.delta = reinterpret_cast<float*>(at + w.delta);
    x.far_chunks = w.far_chunks;
    x.far_part = w.far_chunks > 0 ? reinterpret_cast<float*>(at + w.far_part) : nullptr;
}

inline lrs_status launch_starts(const char* nm, const AttArgs& x, const SeqView& reset, hipStream_t stream)
{
    if (x.starts == nullptr) return LRS_OK;
    return launch_seq(nm, episodes, (uint64_t)x.N * (x.ends != nullptr ? 2 : 1), 256, stream, reset, x.N, x.TK,
                      const_cast<int32_t*>(x.starts), const_cast<int32_t*>(x.ends));
}

// Blocks of 256 threads: a grid holds fewer than 2^32.
constexpr uint64_t kMaxGrid = 0xffffff;

// Whether each wave has 32 queries (or keys) and their tiles to itself.  A block of four
// waves loads a tile once for all of them, but waits with all of them where one has none
// of it: with rows of up to 32 steps it has work for one wave, and with windows that are
// short beside its 128 steps each wave sits out half of the tiles.  There must be waves
// enough for the chip.  us with blocks and alone:
//   short rows, bf16: 2930 x 2 steps of 9 heads of 96 and 80 forward 254 and 63; both
//   directions of 1000 x 20 of 3 heads of 128 155 and 90, of 4096 x 32 of one head of 64
//   107 and 61, of 683 x 32 of 3 heads 63 and 38
//   forward, 64 x 512 of 4 heads of 64, windows 32, 128 and 256: bf16 21.3 and 18.8, 23.6
//   and 23.2, 27.5 and 28.5; f32 59 and 44, 87 and 67, 120 and 98 (512: 143 and 139)
//   dq, of both directions at the same sizes and windows: bf16 100 and 96, 109 and 104, 127
//   and 125; f32 339 and 316, 432 and 400, 586 and 555
//   dk and dv, likewise: f32 317 and 313, 401 and 393, 556 and 511, with 256 x 128 queries
//   over 192 keys (of which blocks fill three in four) 311 and 250; bf16 the same within
//   2% at dims of 64 and 0.9 times as fast at 128
// Rows of up to 128 steps are one block of which no wave sits out much: within 5%.
inline bool queries_alone(const AttArgs& x, int window)
{
    if (x.hpb == 4 || x.N * x.H * ((x.T + 31) / 32) < 2048) return false;
    return x.T <= 32 || (x.TK > 128 && x.window <= window);
}
inline bool forward_alone(const AttArgs& x, int size) { return queries_alone(x, size == 4 ? x.TK : 128); }
inline bool dq_alone(const AttArgs& x, int size) { return queries_alone(x, size == 4 ? 256 : 128); }
inline bool keys_alone(const AttArgs& x, int size)
{
    if (x.N * (x.H / x.group) * ((x.TK + 31) / 32) < 2048) return false;
    return x.TK <= 32 || (size == 4 && x.TK > 128 && x.window <= 256 && x.sinks <= kFarSinks);
}

// Blocks of the forward and of dq: 128 queries of hpb heads, or 32 of a head for each wave.
inline uint64_t query_blocks(AttArgs& x, bool alone)
{
    const int rows = alone ? 32 : 4 / x.hpb * 32;
    x.tiles = (x.T + rows - 1) / rows;
    return alone ? ((uint64_t)x.N * (uint64_t)x.H * (uint64_t)x.tiles + 3) / 4
                 : (uint64_t)x.N * (uint64_t)(x.H / x.hpb) * (uint64_t)x.tiles;
}
inline uint64_t key_blocks(AttArgs& x, bool alone)
{
    x.tiles = (x.TK + (alone ? 31 : 127)) / (alone ? 32 : 128);
    const uint64_t blocks = (uint64_t)x.N * (uint64_t)(x.H / x.group) * (uint64_t)x.tiles;
    return alone ? (blocks + 3) / 4 : blocks;
}

// Blocks of attend_far.
inline uint64_t far_blocks(const AttArgs& x)
{
    return (uint64_t)x.N * (uint64_t)(x.H / x.group) * (uint64_t)x.far_chunks * (uint64_t)((x.sinks + 31) / 32);
}

// By how many elements at a time the kernels may take rows (8, 4 or 0): dims of whole
// units, rows on as many, and a tile's rows (64) within 31-bit offsets.
inline int rows_by(std::initializer_list<const SeqView*> views, int64_t dk, int64_t dv, int s)
{
    for (int by = s == 4 ? 4 : 8; by >= 4; by -= 4) {
        bool ok = dk % by == 0 && dv % by == 0;
        for (const SeqView* v : views) ok = ok && rows_on(*v, by, s) && v->step * s <= (int64_t(1) << 25);
        if (ok) return by;
    }
    return 0;
}

// Calls f with W (64 or 128) and the rows' unit as constants.
template <class D, class F>
lrs_status with_sizes(int64_t dk, int64_t dv, int by, F f)
{
    using N = std::integral_constant<int, 64>;
    using M = std::integral_constant<int, 128>;
    const bool narrow = std::max(dk, dv) <= 64;
    if constexpr (sizeof(D) == 2)
        if (by == 8) return narrow ? f(N(), std::integral_constant<int, 8>()) : f(M(), std::integral_constant<int, 8>());
    if (by == 4) return narrow ? f(N(), std::integral_constant<int, 4>()) : f(M(), std::integral_constant<int, 4>());
    return narrow ? f(N(), std::integral_constant<int, 0>()) : f(M(), std::integral_constant<int, 0>());
}

template <class D, int W, int kBy, bool kK, bool kV>
lrs_status launch_dkv(const char* nm, AttArgs x, hipStream_t stream)
{
    const bool alone = keys_alone(x, sizeof(D));
    const uint64_t blocks = key_blocks(x, alone);
    return launch_seq(nm, alone ? attend_dkv<D, W, kBy, kK, kV, true> : attend_dkv<D, W, kBy, kK, kV, false>,
                      blocks, 256, stream, x);
}

template <class D, int W, int kBy>
lrs_status launch_backward(const char* nm, AttArgs x, hipStream_t stream)
{
    const bool alone = dq_alone(x, sizeof(D));
    const uint64_t blocks = query_blocks(x, alone);
    if (x.sum_delta)
        LRS_TRY(launch_seq(nm, alone ? attend_dq<D, W, kBy, true, true> : attend_dq<D, W, kBy, true, false>, blocks, 256,
                           stream, x));
    LRS_TRY(launch_seq(nm, alone ? attend_dq<D, W, kBy, false, true> : attend_dq<D, W, kBy, false, false>, blocks, 256,
                       stream, x));
    if (x.far_part != nullptr)
        LRS_TRY(launch_seq(nm, attend_far<D, W, kBy>, far_blocks(x), 256, stream, x));
    if constexpr (kSplitGrads<D, W>) {
        LRS_TRY((launch_dkv<D, W, kBy, true, false>(nm, x, stream)));
        return launch_dkv<D, W, kBy, false, true>(nm, x, stream);
    } else {
        return launch_dkv<D, W, kBy, true, true>(nm, x, stream);
    }
}

template <class D>
lrs_status attention_entry(const char* nm, int64_t N, int64_t T, int64_t TK, int64_t H, int64_t KV, int64_t dk,
                           int64_t dv, int64_t window, int64_t sinks, const D* q, const D* k, const D* v,
                           const uint8_t* reset, float scale, D* out, float* lse, const int64_t* strides,
                           void* ws, size_t ws_bytes, hipStream_t stream)
{
    LRS_TRY(check_attention(nm, N, T, TK, H, KV, dk, dv, window, sinks, scale));
    constexpr int s = sizeof(D);
    const SeqArg args[6] = {{q, H, dk, s, false, true, "q"},
                            {k, KV, dk, s, false, true, "k", TK},
                            {v, KV, dv, s, false, true, "v", TK},
                            {reset, 1, 1, 1, false, false, "reset", TK},
                            {out, H, dv, s, true, true, "out"},
                            {lse, H, 1, 4, true, false, "lse"}};
    const Span more[] = {{ws, ws_bytes}};
    SeqView a[6];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, more, 1, 1, a));
    const AttWorkspace w = att_workspace(N, T, TK, H, KV, dk, dv, window, sinks, reset != nullptr, false);
    LRS_TRY(check_workspace(nm, w.bytes, ws, ws_bytes));
    AttArgs x{};
    fill_attention(x, w, N, T, TK, H, KV, dk, dv, window, sinks, scale, reset, ws);
    x.q = a[0];
    x.k = a[1];
    x.v = a[2];
    x.o = a[4];
    x.lse = a[5];
    set_vec(x.q, dk, s);
    set_vec(x.k, dk, s);
    set_vec(x.v, dv, s);
    set_vec(x.o, dv, s);
    const bool alone = forward_alone(x, s);
    const uint64_t blocks = query_blocks(x, alone);
    LRS_REQUIRE(blocks <= kMaxGrid && (reset == nullptr || (uint64_t)N <= kMaxGrid), "%s: num_envs * heads * steps is too large", nm);
    LRS_TRY(launch_starts(nm, x, a[3], stream));
    return with_sizes<D>(dk, dv, rows_by({&x.q, &x.k, &x.v, &x.o}, dk, dv, s), [&](auto w, auto by) {
        constexpr int W = decltype(w)::value, B = decltype(by)::value;
        return launch_seq(nm, alone ? attend_forward<D, W, B, true> : attend_forward<D, W, B, false>, blocks,
                          256, stream, x);
    });
}

template <class D>
lrs_status attention_backward_entry(const char* nm, int64_t N, int64_t T, int64_t TK, int64_t H, int64_t KV,
                                    int64_t dk, int64_t dv, int64_t window, int64_t sinks, const D* grad_out,
                                    const D* q, const D* k, const D* v, const uint8_t* reset, const D* out,
                                    const float* lse, float scale, D* grad_q, D* grad_k, D* grad_v,
                                    const int64_t* strides, void* ws, size_t ws_bytes, hipStream_t stream)
{
    LRS_TRY(check_attention(nm, N, T, TK, H, KV, dk, dv, window, sinks, scale));
    constexpr int s = sizeof(D);
    const SeqArg args[10] = {{grad_out, H, dv, s, false, true, "grad_out"},
                             {q, H, dk, s, false, true, "q"},
                             {k, KV, dk, s, false, true, "k", TK},
                             {v, KV, dv, s, false, true, "v", TK},
                             {reset, 1, 1, 1, false, false, "reset", TK},
                             {out, H, dv, s, false, true, "out"},
                             {lse, H, 1, 4, false, true, "lse"},
                             {grad_q, H, dk, s, true, true, "grad_q"},
                             {grad_k, KV, dk, s, true, true, "grad_k", TK},
                             {grad_v, KV, dv, s, true, true, "grad_v", TK}};
    const Span more[] = {{ws, ws_bytes}};
    SeqView a[10];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, more, 1, 1, a));
    const AttWorkspace w = att_workspace(N, T, TK, H, KV, dk, dv, window, sinks, reset != nullptr, true);
    LRS_TRY(check_workspace(nm, w.bytes, ws, ws_bytes));
    AttArgs x{};
    fill_attention(x, w, N, T, TK, H, KV, dk, dv, window, sinks, scale, reset, ws);
    x.dout = a[0];
    x.q = a[1];
    x.k = a[2];
    x.v = a[3];
    x.o = a[5];
    x.lse = a[6];
    x.dq = a[7];
    x.dk = a[8];
    x.dv = a[9];
    for (SeqView* w : {&x.q, &x.k, &x.dq, &x.dk}) set_vec(*w, dk, s);
    for (SeqView* w : {&x.v, &x.o, &x.dout, &x.dv}) set_vec(*w, dv, s);
    LRS_REQUIRE(query_blocks(x, dq_alone(x, s)) <= kMaxGrid && key_blocks(x, keys_alone(x, s)) <= kMaxGrid && far_blocks(x) <= kMaxGrid &&
                    (reset == nullptr || (uint64_t)N <= kMaxGrid / 2),
                "%s: num_envs * heads * steps is too large", nm);
    LRS_TRY(launch_starts(nm, x, a[4], stream));
    const int unit = rows_by({&x.q, &x.k, &x.v, &x.o, &x.dout, &x.dq, &x.dk, &x.dv}, dk, dv, s);
    return with_sizes<D>(dk, dv, unit, [&](auto w, auto by) {
        return launch_backward<D, decltype(w)::value, decltype(by)::value>(nm, x, stream);
    });
}

// The splits of a step's slots: as many as make four blocks for each of 256 CUs, of
// 256 slots each at least.
inline void plan_step(AttStepArgs& x, int64_t N)
{
    const int64_t slots = (int64_t)x.sinks + x.window, blocks = N * x.KV * x.chunks;
    int64_t splits = std::min<int64_t>((1024 + blocks - 1) / blocks, (slots + 255) / 256);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, 256));
    x.per_split = (int32_t)((slots + splits - 1) / splits);
    x.splits = (int32_t)((slots + x.per_split - 1) / x.per_split);
}

// Heads of a group that a block serves at once.
inline int step_heads(int64_t group) { return group >= 3 ? 4 : (int)group; }

inline bool fill_step(AttStepArgs& x, int64_t N, int64_t H, int64_t KV, int64_t slots, int64_t sinks, int64_t dk,
                      int64_t dv)
{
    if (N < 1 || N > (int64_t(1) << 31) || !att_sizes_ok(H, KV, dk, dv) || sinks < 0 || slots <= sinks ||
        slots > kMaxKeySteps)
        return false;
    x.KV = (int32_t)KV;
    x.group = (int32_t)(H / KV);
    x.chunks = (x.group + step_heads(x.group) - 1) / step_heads(x.group);
    x.sinks = (int32_t)sinks;
    x.window = (int32_t)(slots - sinks);
    x.dim_k = (int32_t)dk;
    x.dim_v = (int32_t)dv;
    plan_step(x, N);
    return true;
}

inline size_t step_workspace(const AttStepArgs& x, int64_t N)
{
    if (x.splits == 1) return 0;
    return (size_t)N * x.KV * x.group * x.splits * (size_t)(x.dim_v + 2) * 4;
}

template <class D, int G>
auto step_kernel(int units) -> void (*)(AttStepArgs)
{
    if (units <= 2) return attend_step<D, 2, G>;
    if (units <= 4) return attend_step<D, 4, G>;
    if (units <= 8) return attend_step<D, 8, G>;
    if (units <= 16) return attend_step<D, 16, G>;
    if constexpr (sizeof(D) == 4) return attend_step<D, 32, G>;
    return attend_step<D, 16, G>;
}

template <class D>
lrs_status attention_step_entry(const char* nm, int64_t N, int64_t H, int64_t KV, int64_t slots, int64_t sinks,
                                int64_t dk, int64_t dv, const D* q, const D* k, const D* v, D* key_cache,
                                D* value_cache, const int32_t* positions, float scale, D* out,
                                const int64_t* strides, void* ws, size_t ws_bytes, hipStream_t stream)
{
    LRS_REQUIRE(slots >= 1 && slots <= kMaxKeySteps, "%s: slots must be 1 to 2^29 (got %lld)", nm,
                (long long)slots);
    LRS_TRY(check_attention(nm, N, 1, 1, H, KV, dk, dv, slots - sinks, sinks, scale));
    constexpr int s = sizeof(D);
    const SeqArg args[7] = {{q, H, dk, s, false, true, "q"},
                            {k, KV, dk, s, false, true, "k"},
                            {v, KV, dv, s, false, true, "v"},
                            {key_cache, KV, dk, s, true, true, "key_cache", slots},
                            {value_cache, KV, dv, s, true, true, "value_cache", slots},
                            {positions, 1, 1, 4, false, true, "positions"},
                            {out, H, dv, s, true, true, "out"}};
    const Span more[] = {{ws, ws_bytes}};
    SeqView a[7];
    LRS_TRY(check_seq_arrays(nm, N, 1, args, strides, more, 1, 1, a));
    LRS_REQUIRE(a[5].env == 1 || N == 1, "%s: positions must be consecutive", nm);
    AttStepArgs x{};
    LRS_REQUIRE(fill_step(x, N, H, KV, slots, sinks, dk, dv), "%s: unsupported sizes", nm);
    LRS_TRY(check_workspace(nm, step_workspace(x, N), ws, ws_bytes));
    x.q = a[0];
    x.k = a[1];
    x.v = a[2];
    x.kc = a[3];
    x.vc = a[4];
    x.positions = positions;
    x.o = a[6];
    x.part = static_cast<float*>(ws);
    x.c = scale * kAttLog2e;
    constexpr int E = 16 / s;
    x.wide = dk % E == 0 && dv % E == 0;
    for (int i = 0; i < 5; ++i) x.wide = x.wide && rows_on(a[i], E, s);
    const uint64_t blocks = (uint64_t)N * KV * x.chunks * x.splits;
    LRS_REQUIRE(blocks <= kMaxGrid && (uint64_t)N * H <= kMaxGrid, "%s: num_envs * heads is too large", nm);
    const int units = (int)((std::max(dk, dv) + E - 1) / E), g = step_heads(x.group);
    LRS_TRY(launch_seq(nm, g == 1 ? step_kernel<D, 1>(units) : g == 2 ? step_kernel<D, 2>(units) : step_kernel<D, 4>(units),
                       blocks, 256, stream, x));
    if (x.splits == 1) return LRS_OK;
    return launch_seq(nm, join_step<D>, (uint64_t)N * H, 128, stream, x);
}

template <class D>
lrs_status attention_fill_entry(const char* nm, int64_t N, int64_t T, int64_t KV, int64_t slots, int64_t sinks,
                                int64_t dk, int64_t dv, const D* k, const D* v, const int32_t* positions,
                                D* key_cache, D* value_cache, const int64_t* strides, hipStream_t stream)
{
    LRS_REQUIRE(slots >= 1 && slots <= kMaxKeySteps, "%s: slots must be 1 to 2^29 (got %lld)", nm,
                (long long)slots);
    LRS_TRY(check_attention(nm, N, T, T, KV, KV, dk, dv, slots - sinks, sinks, 1.0f));
    constexpr int s = sizeof(D);
    const SeqArg args[5] = {{k, KV, dk, s, false, true, "k"},
                            {v, KV, dv, s, false, true, "v"},
                            {positions, 1, 1, 4, false, true, "positions"},
                            {key_cache, KV, dk, s, true, true, "key_cache", slots},
                            {value_cache, KV, dv, s, true, true, "value_cache", slots}};
    SeqView a[5];
    LRS_TRY(check_seq_arrays(nm, N, T, args, strides, nullptr, 0, 0, a));
    AttFillArgs x{a[0], a[1], a[3], a[4], a[2], N, (int32_t)T, (int32_t)KV, (int32_t)sinks,
                  (int32_t)(slots - sinks), (int32_t)dk, (int32_t)dv};
    constexpr int E = 16 / s;
    const bool wide = dk % E == 0 && dv % E == 0 && rows_on(a[0], E, s) && rows_on(a[1], E, s) &&
                      rows_on(a[3], E, s) && rows_on(a[4], E, s);
    LRS_REQUIRE((uint64_t)N < (uint64_t(1) << 62) / slots, "%s: num_envs * slots is too large", nm);
    const uint64_t blocks = std::min<uint64_t>(((uint64_t)N * slots + 3) / 4, kMaxGrid);
    return launch_seq(nm, fill_slots<D>, blocks, 256, stream, x, (uint32_t)wide);
}

}  // namespace lrs
