// sequence.hpp -- what the sequence calls (the gated recurrence with a matrix
// state, the norm of queries and keys with rotation) share: arrays of
// [num_envs, seq_len, heads, dim] with any strides over environments, steps
// and heads, and the host checks of their strides and extents.
#pragma once

#include "launch.hpp"

namespace lrs {

// An array of [env, step, head] rows of consecutive elements.  div: value
// heads per stored head (head h of the call reads head h / div).  vec: how
// wide an access to its rows may be, as its kernel counts it.
struct SeqView {
    const void* p;
    int64_t env, step, head;
    int32_t div;
    int32_t vec;
};

template <class D>
__device__ __forceinline__ const D* seq_row(const SeqView& v, int64_t n, int64_t t, int h)
{
    return static_cast<const D*>(v.p) + n * v.env + t * v.step + (int64_t)(h / v.div) * v.head;
}
template <class D>
__device__ __forceinline__ D* seq_row_out(const SeqView& v, int64_t n, int64_t t, int h)
{
    return const_cast<D*>(seq_row<D>(v, n, t, h));
}

// Eight elements of a row from column c on as they are stored, zero beyond
// `dim`; `vec`: the bytes that an access may take (16, 4 or one element).
template <class D>
struct Raw8 {
    u32x4 w[sizeof(D) / 2];
};

template <class D>
__device__ __forceinline__ Raw8<D> load8(const D* row, int c, int dim, int vec)
{
    Raw8<D> v = {};
    if (vec == 16 && c + 8 <= dim) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(D) / 2; ++k)
            v.w[k] = *reinterpret_cast<const u32x4*>(row + c + k * (16 / sizeof(D)));
    } else if (sizeof(D) == 4 || vec >= 4) {
        const uint32_t* const words = reinterpret_cast<const uint32_t*>(row + c);
        constexpr int per = 4 / sizeof(D);
#pragma unroll
        for (int k = 0; k < 8 / per; ++k)
            if (c + k * per < dim) v.w[k / 4][k % 4] = words[k];
    } else {
        const uint16_t* const halves = reinterpret_cast<const uint16_t*>(row + c);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < dim) v.w[0][k / 2] |= (uint32_t)halves[k] << (16 * (k & 1));
    }
    return v;
}

// One array argument of a sequence call, as checked on the host.
struct SeqArg {
    const void* p;
    int64_t heads, dim;  // [N, T, heads, dim]
    int elem_bytes;
    bool out;
    bool required;
    const char* what;
    int64_t steps = 0;  // where its steps are not the call's T
};

constexpr int64_t kMaxSeqExtent = int64_t(1) << 60;

// Whether `n` strides over axes of these sizes (the innermost `inner` elements
// being consecutive) address every element once.
inline bool strides_disjoint(const int64_t* size, const int64_t* stride, int n, int64_t inner)
{
    bool used[3] = {false, false, false};
    int64_t covered = inner;  // elements below which everything addressed so far lies
    for (int k = 0; k < n; ++k) {
        int best = -1;
        for (int i = 0; i < n; ++i)
            if (!used[i] && size[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
        if (best < 0) return true;
        used[best] = true;
        if (stride[best] < covered) return false;
        covered += stride[best] * (size[best] - 1);
    }
    return true;
}

// Checks the arrays of a sequence call: present where required, strides (three
// per array in signature order: environment, step, head; 0 means contiguous in
// [N, T, heads, dim]) positive and within bounds, outputs addressing every
// element once, and no written array sharing memory with another.  `more`:
// further spans (per-head states, weights), `nmore_out` of them written, first.
template <int K>
lrs_status check_seq_arrays(const char* nm, int64_t N, int64_t T, const SeqArg (&args)[K],
                            const int64_t* strides, const Span* more, int nmore_out, int nmore,
                            SeqView (&views)[K])
{
    Span ins[K + 8], outs[K + 8];
    int ni = 0, no = 0;
    for (int i = 0; i < K; ++i) {
        const SeqArg& a = args[i];
        if (a.p == nullptr) {
            if (a.required) return fail(LRS_ERR_INVALID_ARG, "%s: %s is required", nm, a.what);
            views[i] = SeqView{nullptr, 0, 0, 0, 1, 0};
            continue;
        }
        if ((uintptr_t)a.p % a.elem_bytes != 0)
            return fail(LRS_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", nm, a.what);
        const int64_t steps = a.steps != 0 ? a.steps : T;
        const int64_t size[3] = {N, steps, a.heads};
        int64_t st[3] = {steps * a.heads * a.dim, a.heads * a.dim, a.dim};
        int64_t extent = a.dim;
        for (int k = 0; k < 3; ++k) {
            if (strides != nullptr && strides[3 * i + k] != 0) st[k] = strides[3 * i + k];
            if (st[k] < 1)
                return fail(LRS_ERR_INVALID_ARG, "%s: stride %lld of %s is negative", nm,
                            (long long)st[k], a.what);
            if (size[k] > 1) {
                if (st[k] > (kMaxSeqExtent - extent) / (size[k] - 1))
                    return fail(LRS_ERR_INVALID_ARG, "%s: stride %lld of %s is too large", nm,
                                (long long)st[k], a.what);
                extent += st[k] * (size[k] - 1);
            }
        }
        if (a.out && !strides_disjoint(size, st, 3, a.dim))
            return fail(LRS_ERR_INVALID_ARG, "%s: the strides of %s address an element twice", nm,
                        a.what);
        views[i] = SeqView{a.p, st[0], st[1], st[2], 1, 0};
        (a.out ? outs[no++] : ins[ni++]) = Span{a.p, (uint64_t)extent * (uint64_t)a.elem_bytes};
    }
    for (int i = 0; i < nmore; ++i) (i < nmore_out ? outs[no++] : ins[ni++]) = more[i];
    return check_disjoint(nm, outs, no, ins, ni);
}

inline lrs_status check_workspace(const char* nm, size_t need, const void* ws, size_t ws_bytes)
{
    if (need == 0) return LRS_OK;
    if (ws == nullptr || ws_bytes < need)
        return fail(LRS_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", nm, need,
                    ws == nullptr ? (size_t)0 : ws_bytes);
    if (!aligned(ws, 16)) return fail(LRS_ERR_WORKSPACE, "%s: workspace not 16-byte aligned", nm);
    return LRS_OK;
}

// Whether every row starts on a multiple of `unit` elements.
inline bool rows_on(const SeqView& v, int unit, int elem_bytes)
{
    return aligned(v.p, (uintptr_t)(unit * elem_bytes)) && v.env % unit == 0 && v.step % unit == 0 &&
           v.head % unit == 0;
}

// Launches `kernel` and returns the launch's own status.
template <class... P>
lrs_status launch_seq(const char* nm, void (*kernel)(P...), dim3 blocks, int threads,
                      hipStream_t stream, P... params)
{
    void* ptrs[] = {(void*)&params...};
    const hipError_t e = hipLaunchKernel((const void*)kernel, blocks, dim3(threads), ptrs, 0, stream);
    if (e != hipSuccess)
        return fail(LRS_ERR_HIP, "%s: kernel launch failed: %s", nm, hipGetErrorString(e));
    g_err[0] = '\0';
    return LRS_OK;
}
template <class... P>
lrs_status launch_seq(const char* nm, void (*kernel)(P...), uint64_t blocks, int threads,
                      hipStream_t stream, P... params)
{
    return launch_seq(nm, kernel, dim3((uint32_t)blocks), threads, stream, params...);
}

}  // namespace lrs
