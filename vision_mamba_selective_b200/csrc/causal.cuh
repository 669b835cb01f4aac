// causal.cuh -- arguments and small device functions shared by the causal operators
// (scan, short convolution, their single-token forms and derivatives).
#pragma once

#include "vimscan.h"

#include <cstdint>

#include "launch.cuh"

namespace vimscan {

// ----------------------------------------------------------------------------
// host-side argument checks
// ----------------------------------------------------------------------------
inline bool misaligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// an activation the kernels may address: non-null, aligned to its element, strides >= 0
inline bool bad_rows(const vim_rows &r, vim_dtype dt) {
    return !r.data || misaligned(r.data, elem_size(dt)) || r.batch_stride < 0 || r.row_stride < 0;
}
// an output: its rows must not overlap (rows of `width` elements)
inline bool bad_out(const vim_rows &r, vim_dtype dt, int batch, int L, int width) {
    if (bad_rows(r, dt)) return true;
    if (L > 1 && r.row_stride < width) return true;
    return batch > 1 && r.batch_stride < (int64_t)(L - 1) * r.row_stride + width;
}
// whether every row of r starts on a 16-byte boundary and holds whole 16-byte vectors
inline bool whole_vectors(const vim_rows &r, vim_dtype dt, int batch, int L, int width) {
    const int ve = (int)(16 / elem_size(dt));
    return !misaligned(r.data, 16) && width % ve == 0 && (L <= 1 || r.row_stride % ve == 0) &&
           (batch <= 1 || r.batch_stride % ve == 0);
}

inline vim_status check_sizes(int batch, int L, int channels, vim_dtype dt) {
    if (batch < 0 || L < 0 || channels < 0 || (dt != VIM_F32 && dt != VIM_BF16)) return VIM_ERR_INVALID_ARG;
    return VIM_OK;
}

// ----------------------------------------------------------------------------
// sequences of a call: the rows of a [batch, L, .] tensor, or (cu non-null) the ranges
// cu[s] .. cu[s + 1] of one row of L packed tokens
// ----------------------------------------------------------------------------
struct Seqs {
    const int *cu;            // [n + 1] or null
    const int *slots;         // [n] or null: the state row of each sequence
    const unsigned char *fresh;  // [n] or null: start from zero
    int n, L, n_slots;        // sequences, tokens per row, rows of the state cache
};
// Seqs of a call (v null: the batch rows, no states); `align` is what the states must be
// aligned to
inline vim_status make_seqs(const vim_sequences *v, int batch, int L, size_t align, Seqs *out) {
    Seqs q = {nullptr, nullptr, nullptr, batch, L, 0};
    if (v) {
        if (v->n_seqs < 0 || v->n_slots < 0) return VIM_ERR_INVALID_ARG;
        if (v->cu_seqlens) {
            if (batch != 1 || misaligned(v->cu_seqlens, 4)) return VIM_ERR_INVALID_ARG;
        } else if (v->n_seqs != batch) {
            return VIM_ERR_INVALID_ARG;
        }
        const bool states = v->state || v->state_out;
        if (!states && (v->slots || v->fresh || v->n_slots)) return VIM_ERR_INVALID_ARG;
        if (states && !v->slots && v->n_slots < v->n_seqs) return VIM_ERR_INVALID_ARG;
        if (misaligned(v->state, align) || misaligned(v->state_out, align) || misaligned(v->slots, 4))
            return VIM_ERR_INVALID_ARG;
        q.cu = v->cu_seqlens;
        q.n = v->n_seqs;
        q.slots = v->slots;
        q.n_slots = v->n_slots;
        q.fresh = v->fresh;
    }
    *out = q;
    return VIM_OK;
}
struct Seq {
    int start, end;           // its tokens
    int64_t slot;             // its state row, or -1: a padding entry
    bool fresh;
};
// Offsets outside 0..L or decreasing are clamped, so that a bad table gives wrong ranges
// and never an address outside the tensors.
__device__ __forceinline__ Seq sequence(const Seqs &q, int s) {
    Seq r;
    r.start = 0;
    r.end = q.L;
    if (q.cu) {
        r.start = min(max(q.cu[s], 0), q.L);
        r.end = min(max(q.cu[s + 1], r.start), q.L);
    }
    r.slot = s;
    if (q.slots) {
        r.slot = q.slots[s];
        if (r.slot < 0 || r.slot >= q.n_slots) r.slot = -1;
    }
    r.fresh = q.fresh && q.fresh[s];
    return r;
}
// the first sequence of a packed row that ends after token t (n if none does)
__device__ __forceinline__ int sequence_at(const Seqs &q, int t) {
    int lo = 0, hi = q.n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (q.cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// ----------------------------------------------------------------------------
// functions
// ----------------------------------------------------------------------------
// exp(x) for x <= 0 to about 1.5e-7 relative at any magnitude: x log2(e) is formed as a
// rounded product and its remainder, 2^product comes from the exp2 unit and the
// remainder r enters as 1 + r ln 2.  (Without it the rounding of a product near 10
// alone is 3e-7 of the result, and softplus at the biases of trained models is exp.)
__device__ __forceinline__ float exp_neg(float x) {
    const float t = x * kLog2e;
    const float r = fmaf(x, 1.9259629e-8f, fmaf(x, kLog2e, -t));   // 1.9259629e-8 = log2(e) - float(log2(e))
    const float e = ex2(t);
    return t < -140.0f ? 0.0f : fmaf(e, r * kLn2, e);
}

// softplus(x) = max(x, 0) + log1p(exp(-|x|)), and x itself above 20: as softplus() of the
// bidirectional scan, with the exponential above.  There the exponential's error, up to
// 4e-7 relative, stays below the tolerance of one output; here Delta also scales fp32
// states that are handed on from call to call and fp32 gradients.
__device__ __forceinline__ float softplus_acc(float x) {
    const float e = exp_neg(-fabsf(x));
    const float s = e * rcp(2.0f + e);
    const float s2 = s * s;
    float p = fmaf(s2, 2.0f / 13.0f, 2.0f / 11.0f);
    p = fmaf(s2, p, 2.0f / 9.0f);
    p = fmaf(s2, p, 2.0f / 7.0f);
    p = fmaf(s2, p, 2.0f / 5.0f);
    p = fmaf(s2, p, 2.0f / 3.0f);
    p = fmaf(s2, p, 2.0f);
    const float r = fmaf(s, p, fmaxf(x, 0.0f));
    return x > 20.0f ? x : r;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-x * kLog2e)); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace vimscan
