// causal.cuh -- arguments and small device functions shared by the causal operators
// (scan, short convolution, their single-token forms and derivatives).
#pragma once

#include "vimscan_causal.h"

#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <utility>

#include "launch.cuh"

namespace vimscan {

// ----------------------------------------------------------------------------
// host-side argument checks
// ----------------------------------------------------------------------------
inline bool misaligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// an activation the kernels may address: non-null, aligned to its element, strides >= 0
// and rows less than 2^29 elements apart
inline bool bad_rows(const vim_rows &r, vim_dtype dt) {
    return !r.data || misaligned(r.data, elem_size(dt)) || r.batch_stride < 0 || r.row_stride < 0 ||
           r.row_stride > INT32_MAX / 4;
}
// an output: its rows (of `width` elements) must not overlap, whether the tokens of a batch item
// follow one another or the batch items of a token do
inline bool bad_out(const vim_rows &r, vim_dtype dt, int batch, int L, int width) {
    if (bad_rows(r, dt)) return true;
    const int64_t rows = (int64_t)(L - 1) * r.row_stride + width, items = (int64_t)(batch - 1) * r.batch_stride + width;
    const bool tokens_inside = (L <= 1 || r.row_stride >= width) && (batch <= 1 || r.batch_stride >= rows);
    const bool items_inside = (batch <= 1 || r.batch_stride >= width) && (L <= 1 || r.row_stride >= items);
    return !tokens_inside && !items_inside;
}
// Whether two sets of rows, wa and wb elements wide, share elements: exactly where their strides are
// the same, and by the first element where they are not.  Called with an output among the two, so
// that equal strides are those of rows that do not overlap.
inline bool rows_meet(const vim_rows &a, int wa, const vim_rows &b, int wb, vim_dtype dt, int batch, int L) {
    if (!a.data || !b.data) return false;
    if (a.data == b.data) return true;
    if ((batch > 1 && a.batch_stride != b.batch_stride) || (L > 1 && a.row_stride != b.row_stride)) return false;
    // element x of one is element y of the other where outer steps of s_out, inner steps of s_in
    // and a difference of columns between -(wa - 1) and wb - 1 add up to `apart`
    int64_t s_out = batch > 1 ? a.batch_stride : 0, s_in = L > 1 ? a.row_stride : 0, n_out = batch - 1, n_in = L - 1;
    if (s_in > s_out) std::swap(s_in, s_out), std::swap(n_in, n_out);
    const int64_t apart = (reinterpret_cast<intptr_t>(b.data) - reinterpret_cast<intptr_t>(a.data)) / (int64_t)elem_size(dt);
    const int64_t reach = n_in * s_in + std::max(wa, wb);
    const int64_t from = s_out ? std::max(-n_out, (apart - reach) / s_out - 1) : 0;
    const int64_t to = s_out ? std::min(n_out, (apart + reach) / s_out + 1) : 0;
    for (int64_t o = from; o <= to; ++o) {
        const int64_t lo = apart - o * s_out - (wa - 1), hi = lo + wa + wb - 2;   // of the inner steps
        int64_t i = 0;
        if (s_in) i = std::min(n_in, std::max(-n_in, lo >= 0 ? (lo + s_in - 1) / s_in : -(-lo / s_in)));
        if (i * s_in >= lo && i * s_in <= hi) return true;
    }
    return false;
}
// an output that may lie in the place of an input: the same rows or none of them
inline bool rows_clash(const vim_rows &out, const vim_rows &in, int width, vim_dtype dt, int batch, int L) {
    const bool same = out.data == in.data && (batch <= 1 || out.batch_stride == in.batch_stride) &&
                      (L <= 1 || out.row_stride == in.row_stride);
    return !same && rows_meet(out, width, in, width, dt, batch, L);
}
// the scan's parameters: A is read in vectors of four
inline bool bad_params(const float *A, const float *D, const float *bias) {
    return !A || !D || !bias || misaligned(A, 16) || misaligned(D, 4) || misaligned(bias, 4);
}
// whether every row of r can be read in vectors of n elements
inline bool row_vectors(const vim_rows &r, vim_dtype dt, int batch, int L, int n) {
    return !misaligned(r.data, n * elem_size(dt)) && (L <= 1 || r.row_stride % n == 0) &&
           (batch <= 1 || r.batch_stride % n == 0);
}
inline vim_status check_sizes(int batch, int L, int channels, vim_dtype dt) {
    if (batch < 0 || L < 0 || channels < 0 || (dt != VIM_F32 && dt != VIM_BF16)) return VIM_ERR_INVALID_ARG;
    if (L > INT32_MAX - 1024 || channels > INT32_MAX - 1024) return VIM_ERR_UNSUPPORTED;   // tiles past the end are counted in ints
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
// aligned to, `row_bytes` the size of a state row
inline vim_status make_seqs(const vim_sequences *v, int batch, int L, size_t align, int64_t row_bytes, Seqs *out) {
    Seqs q = {nullptr, nullptr, nullptr, batch, L, 0};
    if (v) {
        if (v->n_seqs < 0 || v->n_slots < 0 || v->n_seqs > INT32_MAX || v->n_slots > INT32_MAX) return VIM_ERR_INVALID_ARG;
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
        if (v->state && v->state_out && v->state != v->state_out) {   // in place, or apart
            const int64_t gap = reinterpret_cast<intptr_t>(v->state_out) - reinterpret_cast<intptr_t>(v->state);
            if (row_bytes > 0 && (gap < 0 ? -gap : gap) / row_bytes < v->n_slots) return VIM_ERR_INVALID_ARG;
        }
        q.cu = v->cu_seqlens;
        q.n = (int)v->n_seqs;
        q.slots = v->slots;
        q.n_slots = (int)v->n_slots;
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
// the larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// exp(x) for x <= 0 to about 1.5e-7 relative: x log2(e) is formed as a rounded product and
// its remainder r; 2^product comes from the exp2 unit and r enters as 1 + r ln 2.  (Without
// it the rounding of a product near 10 alone is 3e-7 of the result, and softplus at the
// biases of trained models is exp.)  Below -100 the result is 0.
__device__ __forceinline__ float exp_neg(float x) {
    x = max_nan(x, -100.0f);
    const float t = x * kLog2e;
    const float r = fmaf(x, 1.9259629e-8f, fmaf(x, kLog2e, -t));   // 1.9259629e-8 = log2(e) - float(log2(e))
    const float e = ex2(t);
    return fmaf(e, r * kLn2, e);
}

// softplus(x) = max(x, 0) + log1p(exp(-|x|)): as softplus() of the bidirectional scan, with
// the exponential above (above 20 the logarithm is below half a step of x, so that x
// itself comes out).  There the exponential's error, up to 4e-7 relative, stays below the
// tolerance of one output; here Delta also scales fp32 states that are handed on from
// call to call and fp32 gradients.
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
    return fmaf(s, p, max_nan(x, 0.0f));
}

// softplus(x) and its derivative 1 / (1 + exp(-x))
__device__ __forceinline__ float softplus_slope(float x, float &slope) {
    const float e = exp_neg(-fabsf(x)), r = rcp(1.0f + e);
    slope = x < 0.0f ? e * r : r;
    return softplus_acc(x);
}

// 1 / (1 + exp(-x)).  The rounding of x log2(e) is not carried along: up to 7e-7 relative at |x| near
// 20, in an output or gradient that is not added up over tokens
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-x * kLog2e)); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 2^(A2 dt), the decay of a state over one step (A2 = A log2(e)).  The exp2 unit's results lie
// low: by 1.6e-8 to 2.9e-8 relative on average for decays of 0.75 to 0.995, which over a
// memory of hundreds of steps adds up where unbiased roundings of that size would not.  An
// argument 2e-8 higher takes the mean error there to between -1.5e-8 and 0 (measured over
// 10^6 arguments per octave; a step of 0 still gives exactly 1), and the addition is part
// of the multiplication that forms the argument.
constexpr float kDecayShift = 2.0e-8f;
// A log2(e).  Held finite, so that a step of 0 (tokens outside a sequence) leaves the state as it is
// where A is -infinity; every step above 1e-36 then still gives a decay of 0.
__device__ __forceinline__ float decay_rate(float A) { return max_nan(A * kLog2e, -FLT_MAX); }
__device__ __forceinline__ float2 decay_rate(float2 A) { return f2(decay_rate(A.x), decay_rate(A.y)); }
__device__ __forceinline__ float decay(float A2, float dt) { return ex2(fmaf(A2, dt, kDecayShift)); }
__device__ __forceinline__ float2 decay(float2 A2, float dt) {
    const float2 e = fma2(A2, f2(dt, dt), f2(kDecayShift, kDecayShift));
    return f2(ex2(e.x), ex2(e.y));
}

// ----------------------------------------------------------------------------
// elements of strided rows
// ----------------------------------------------------------------------------
// an element's bits in a 32-bit register, and its value
template <typename T> __device__ __forceinline__ float bits_f32(uint32_t v);
template <> __device__ __forceinline__ float bits_f32<float>(uint32_t v) { return __uint_as_float(v); }
template <> __device__ __forceinline__ float bits_f32<__nv_bfloat16>(uint32_t v) { return __uint_as_float(v << 16); }

// element i of a run that starts on a word boundary, from its word
template <typename T> __device__ __forceinline__ float word_f32(uint32_t w, int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    else return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
}

// How a kernel loads a tensor: through the non-coherent path, which is for memory that no thread
// writes while the kernel runs; or by a plain load, where an output may lie over it.  kInPlaceFree
// (elements and words) is a plain load that stores in between do not hold back: each element is
// loaded by the thread that writes it, and what it writes depends on the load.  causal_step,
// 256 x 4096: 31.7 us with it, 32.5 with kInPlace; causal_pass, 4 x 16385 tokens x 384 channels:
// 339 and 327.
enum Load { kReadOnly, kInPlace, kInPlaceFree };
template <Load HOW, typename V> __device__ __forceinline__ V load_as(const char *at) {
    if constexpr (HOW == kReadOnly) {
        return __ldg(reinterpret_cast<const V *>(at));
    } else if constexpr (HOW == kInPlace) {
        return *reinterpret_cast<const V *>(at);
    } else {
        static_assert(sizeof(V) == 4 || sizeof(V) == 2, "elements and words");
        V v;
        if constexpr (sizeof(V) == 4) asm("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(at));
        else asm("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(at));
        return v;
    }
}

// Column `c` of the rows of batch item b.  Row strides fit in 32 bits of bytes (checked on
// the host), so an address is one widening multiply-add.
template <typename T, Load HOW = kReadOnly>
struct RowsOf {
    const char *base;
    int row;                                               // bytes between rows
    __device__ __forceinline__ RowsOf(const vim_rows &r, int64_t b, int c)
        : base(static_cast<const char *>(r.data) + (b * r.batch_stride + c) * (int64_t)sizeof(T)),
          row((int)(r.row_stride * (int64_t)sizeof(T))) {}
    __device__ __forceinline__ const char *at(int t) const { return base + (int64_t)t * row; }
    __device__ __forceinline__ uint32_t raw(int t, int i = 0) const {
        if constexpr (sizeof(T) == 4) return load_as<HOW, uint32_t>(at(t) + 4 * i);
        else return load_as<HOW, uint16_t>(at(t) + 2 * i);
    }
    // n 32-bit words of elements: at once, aligned to their size or to four elements, or
    // element by element
    template <int n> __device__ __forceinline__ void words(int t, uint32_t (&v)[n]) const {
        if constexpr (n > (int)sizeof(T)) {                // eight elements
            if constexpr (sizeof(T) == 4) {
                const uint4 x = load_as<HOW, uint4>(at(t));
                const uint4 y = load_as<HOW, uint4>(at(t) + sizeof(uint4));
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            } else {
                const uint2 x = load_as<HOW, uint2>(at(t));
                const uint2 y = load_as<HOW, uint2>(at(t) + sizeof(uint2));
                v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
            }
        } else if constexpr (n == 4) {
            const uint4 x = load_as<HOW, uint4>(at(t));
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else if constexpr (n == 2) {
            const uint2 x = load_as<HOW, uint2>(at(t));
            v[0] = x.x, v[1] = x.y;
        } else {
            v[0] = load_as<HOW, uint32_t>(at(t));
        }
    }
    template <int n> __device__ __forceinline__ void gather(int t, uint32_t (&v)[n]) const {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = raw(t, i);
            else v[i] = raw(t, 2 * i) | raw(t, 2 * i + 1) << 16;
        }
    }
    __device__ __forceinline__ void put(int t, float x) const {
        *reinterpret_cast<T *>(const_cast<char *>(at(t))) = from_f32<T>(x);
    }
};

template <int NP> __device__ __forceinline__ void store_row(float *row, const float2 (&v)[NP]) {
    if constexpr (NP >= 2) {
#pragma unroll
        for (int i = 0; i < NP; i += 2)
            *reinterpret_cast<float4 *>(row + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
    } else {
        *reinterpret_cast<float2 *>(row) = v[0];
    }
}

}  // namespace vimscan
