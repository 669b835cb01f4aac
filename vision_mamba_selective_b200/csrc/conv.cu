// conv.cu -- short causal depthwise convolution (declared in include/vimscan_causal.h): prompts,
// single tokens and the derivative.
//
//   pre_t = b + sum_(k < W) w_k x_(t - W + 1 + k),   y_t = silu(pre_t) or pre_t
//
// All of it is bound by memory traffic (two elements per token-channel forward, three
// backward), so every thread walks down the tokens of a few neighbouring channels with the
// last W - 1 inputs in registers: each input is read once.
#include "causal.cuh"

#include <algorithm>
#include <cstring>

namespace vimscan {

struct ConvArgs {
    vim_rows x, y, dout, dx;
    const float *w, *b;                    // [d][W], [d] or null
    Seqs seqs;
    const void *state;                     // [n_slots][W - 1][d] or null
    void *state_out;
    float *part;                           // derivative: [groups of runs][W + 1][d]
    int batch, L, d, silu;
    int run, across;                       // tokens of one thread's run, strips of a CTA
    int w16;                               // w starts on a 16-byte boundary
};

namespace {

constexpr int kConvThreads = 128;

// V neighbouring elements of a row as floats: at once where rows are whole vectors (VEC), or
// one by one up to column d
template <typename T, int V, bool VEC>
struct Strip {
    static constexpr int kWords = VEC ? V * (int)sizeof(T) / 4 : V;
    uint32_t v[kWords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void load(const char *at, int left) {
        if constexpr (VEC) {
            if constexpr (kWords == 4) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(at));
                v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
            } else {
                const uint2 q = __ldg(reinterpret_cast<const uint2 *>(at));
                v[0] = q.x, v[1] = q.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = 0;
                if (i < left) {
                    if constexpr (sizeof(T) == 4) v[i] = __ldg(reinterpret_cast<const uint32_t *>(at) + i);
                    else v[i] = __ldg(reinterpret_cast<const uint16_t *>(at) + i);
                }
            }
        }
    }
    __device__ __forceinline__ float f(int i) const {
        if constexpr (!VEC) return bits_f32<T>(v[i]);
        else return word_f32<T>(v[i * (int)sizeof(T) / 4], i);
    }
};
template <typename T, int V, bool VEC>
__device__ __forceinline__ void put_strip(char *at, const float (&f)[V], int left) {
    if constexpr (VEC && V == Vec<T>::n) {
        *reinterpret_cast<uint4 *>(at) = pack16(f);
    } else if constexpr (VEC && sizeof(T) == 2 && V == 4) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        *reinterpret_cast<uint2 *>(at) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) reinterpret_cast<T *>(at)[i] = from_f32<T>(f[i]);
    }
}

// the run of tokens and the channel strip of a thread: a CTA is `across` neighbouring strips by
// kConvThreads / across runs
struct ConvSpot {
    int b, t0, t1, c;
    int64_t group;                         // the CTA's place among the groups of runs
    bool any;
};
template <int V>
__device__ __forceinline__ ConvSpot conv_spot(const ConvArgs &p) {
    ConvSpot s;
    const int strips = (p.d + V - 1) / V, runs = (p.L + p.run - 1) / p.run;
    const int blocks = (strips + p.across - 1) / p.across;
    s.group = blockIdx.x / blocks;
    s.c = ((int)(blockIdx.x % blocks) * p.across + (int)threadIdx.x % p.across) * V;
    const int64_t at = s.group * (kConvThreads / p.across) + threadIdx.x / p.across;
    s.any = at < (int64_t)p.batch * runs && s.c < p.d;
    s.b = (int)(at / runs);
    s.t0 = (int)(at % runs) * p.run;
    s.t1 = min(s.t0 + p.run, p.L);
    return s;
}
// taps and bias of a strip (columns past d repeat the last)
template <int W, int V>
__device__ __forceinline__ void conv_taps(const ConvArgs &p, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ci = min(c + i, p.d - 1);
        bias[i] = p.b ? __ldg(p.b + ci) : 0.0f;
        if (W == 4 && p.w16) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p.w) + ci);
            w[0][i] = q.x, w[1][i] = q.y, w[W - 2][i] = q.z, w[W - 1][i] = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = __ldg(p.w + (int64_t)ci * W + k);
        }
    }
}

// Prompts.  A thread takes `run` tokens of V channels.  Where its run starts inside a
// sequence it first reads the W - 1 tokens before it, and where a sequence starts in the run
// the window is filled from that sequence's state row or zeros.
template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(kConvThreads) conv_prompt(const ConvArgs p) {
    const ConvSpot o = conv_spot<V>(p);
    if (!o.any) return;
    const int left = p.d - o.c;
    const RowsOf<T> gx(p.x, o.b, o.c), gy(p.y, o.b, o.c);
    float w[W][V], bias[V];
    conv_taps<W, V>(p, o.c, w, bias);
    int s = p.seqs.cu ? sequence_at(p.seqs, o.t0) : o.b;
    int t = o.t0;
    float win[W][V];                                       // win[k]: x at t - W + 1 + k
#pragma unroll 1
    while (t < o.t1 && s < p.seqs.n) {
        const Seq q = sequence(p.seqs, s);
        const int begin = max(t, q.start), end = min(o.t1, q.end);
        if (begin >= end || q.slot < 0) {                  // none of its tokens here, or a padding entry
            t = max(t, end);
            ++s;
            if (!p.seqs.cu) break;
            continue;
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {                  // the window before token `begin`
            const int at = begin - (W - 1) + k;
            Strip<T, V, VEC> x;
            x.clear();
            if (at >= q.start) x.load(gx.at(at), left);
            else if (p.state && !q.fresh)
                x.load(reinterpret_cast<const char *>(static_cast<const T *>(p.state) +
                                                      (q.slot * (W - 1) + (at - q.start + W - 1)) * p.d + o.c), left);
#pragma unroll
            for (int i = 0; i < V; ++i) win[k][i] = x.f(i);
        }
        constexpr int AHEAD = 8;                           // tokens loaded together
#pragma unroll 1
        for (t = begin; t < end; t += AHEAD) {
            Strip<T, V, VEC> x[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) x[j].load(gx.at(min(t + j, end - 1)), left);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                float y[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[W - 1][i] = x[j].f(i);
                    y[i] = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) y[i] = fmaf(w[k][i], win[k][i], y[i]);
                    if (p.silu) y[i] *= sigmoid(y[i]);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i];
                }
                if (t + j < end) put_strip<T, V, VEC>(const_cast<char *>(gy.at(t + j)), y, left);
            }
        }
        t = end;
        ++s;
        if (!p.seqs.cu) break;
    }
}

// The last W - 1 inputs of every sequence, into its state row: one thread per (sequence,
// channel) reads them all before it writes any, so the row may be the one that was read.
template <typename T, int W>
__global__ void __launch_bounds__(kConvThreads) conv_states(const ConvArgs p) {
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t s = i / p.d;
    cudaGridDependencySynchronize();                       // conv_prompt has read the states
    if (s >= p.seqs.n) return;
    const int c = (int)(i % p.d);
    const Seq q = sequence(p.seqs, (int)s);
    if (q.slot < 0) return;
    const RowsOf<T> gx(p.x, p.seqs.cu ? 0 : s, c);
    const int64_t row = q.slot * (W - 1) * p.d + c;
    T v[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int at = q.end - (W - 1) + k;
        v[k] = from_f32<T>(0.0f);
        if (at >= q.start) v[k] = *reinterpret_cast<const T *>(gx.at(at));
        else if (p.state && !q.fresh) v[k] = static_cast<const T *>(p.state)[row + (int64_t)(at - q.start + W - 1) * p.d];
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) static_cast<T *>(p.state_out)[row + (int64_t)k * p.d] = v[k];
}

// One token per sequence: the state row moves up by one.
template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(kConvThreads) conv_step(const ConvArgs p) {
    const int strips = (p.d + V - 1) / V;
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t b = i / strips;
    if (b >= p.batch) return;
    const int c = (int)(i % strips) * V, left = p.d - c;
    const Seq q = sequence(p.seqs, (int)b);
    if (q.slot < 0) return;
    const int64_t row = q.slot * (W - 1) * p.d + c;
    Strip<T, V, VEC> x[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        x[k].clear();
        if (!q.fresh)
            x[k].load(reinterpret_cast<const char *>(static_cast<const T *>(p.state) + row + (int64_t)k * p.d), left);
    }
    x[W - 1].load(RowsOf<T>(p.x, b, c).at(0), left);
    float w[W][V], y[V];
    conv_taps<W, V>(p, c, w, y);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) y[e] = fmaf(w[k][e], x[k].f(e), y[e]);
        if (p.silu) y[e] *= sigmoid(y[e]);
    }
    put_strip<T, V, VEC>(const_cast<char *>(RowsOf<T>(p.y, b, c).at(0)), y, left);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = x[k + 1].f(e);
        put_strip<T, V, VEC>(reinterpret_cast<char *>(static_cast<T *>(p.state_out) + row + (int64_t)k * p.d), f, left);
    }
}

// Derivative for sequences that start from zeros.  With dpre_t = dout_t silu'(pre_t):
//   dx_t = sum_j w_(W-1-j) dpre_(t + j),  dw_k = sum_t dpre_t x_(t - W + 1 + k),  db = sum_t dpre_t
// A thread forms dpre along its run and W - 1 tokens past it (so that its dx are complete);
// dw and db take the run's own tokens.  The runs' sums go to `part`.
template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(kConvThreads) conv_bwd(const ConvArgs p) {
    const ConvSpot o = conv_spot<V>(p);
    const int left = p.d - o.c;
    const RowsOf<T> gx(p.x, o.b, o.c), go(p.dout, o.b, o.c), gdx(p.dx, o.b, o.c);
    float w[W][V], bias[V], dw[W][V], db[V];
    conv_taps<W, V>(p, o.c, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = 0.0f;
    }
    int s = p.seqs.cu && o.any ? sequence_at(p.seqs, o.t0) : o.b;
    int t = o.t0;
#pragma unroll 1
    while (o.any && t < o.t1 && s < p.seqs.n) {
        const Seq q = sequence(p.seqs, s);
        const int begin = max(t, q.start), end = min(o.t1, q.end), stop = min(end + W - 1, q.end);
        if (begin < end) {
            float win[W][V], ahead[W][V];                  // ahead[j]: dpre at t - W + 1 + j
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                const int at = begin - (W - 1) + k;
                Strip<T, V, VEC> x;
                x.clear();
                if (at >= q.start) x.load(gx.at(at), left);
#pragma unroll
                for (int i = 0; i < V; ++i) win[k][i] = x.f(i), ahead[k][i] = 0.0f;
            }
            // token u forms dpre_u and completes dx of token u - W + 1; past `stop` dpre is zero
            constexpr int AHEAD = 4;
#pragma unroll 1
            for (int u0 = begin; u0 < end + W - 1; u0 += AHEAD) {
                Strip<T, V, VEC> x[AHEAD], g[AHEAD];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int at = min(u0 + j, stop - 1);
                    x[j].load(gx.at(at), left);
                    g[j].load(go.at(at), left);
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int u = u0 + j;
                    float dx[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        win[W - 1][i] = x[j].f(i);
                        float dpre = g[j].f(i);
                        if (p.silu) {
                            float pre = bias[i];
#pragma unroll
                            for (int k = 0; k < W; ++k) pre = fmaf(w[k][i], win[k][i], pre);
                            const float sg = sigmoid(pre);
                            dpre *= sg * fmaf(pre, 1.0f - sg, 1.0f);
                        }
                        if (u >= stop) dpre = 0.0f;
                        ahead[W - 1][i] = dpre;
                        if (u < end) {
                            db[i] += dpre;
#pragma unroll
                            for (int k = 0; k < W; ++k) dw[k][i] = fmaf(dpre, win[k][i], dw[k][i]);
                        }
                        dx[i] = 0.0f;
#pragma unroll
                        for (int k = 0; k < W; ++k) dx[i] = fmaf(w[W - 1 - k][i], ahead[k][i], dx[i]);
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i], ahead[k][i] = ahead[k + 1][i];
                    }
                    const int at = u - (W - 1);
                    if (at >= begin && at < end) put_strip<T, V, VEC>(const_cast<char *>(gdx.at(at)), dx, left);
                }
            }
        }
        t = max(t, end);
        ++s;
        if (!p.seqs.cu) break;
    }
    // the runs of the CTA that share a strip, joined in shared memory in their order
    __shared__ float sums[(W + 1) * V][kConvThreads];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) sums[k * V + i][threadIdx.x] = dw[k][i];
        sums[W * V + i][threadIdx.x] = db[i];
    }
    __syncthreads();
    const int64_t n = (int64_t)p.d * (W + 1);
    const int c0 = o.c - (int)(threadIdx.x % p.across) * V;
    for (int i = threadIdx.x; i < (W + 1) * V * p.across; i += kConvThreads) {
        const int x = i % p.across, kv = i / p.across, c = c0 + x * V + kv % V;
        float f = 0.0f;
        for (int y = x; y < kConvThreads; y += p.across) f += sums[kv][y];
        if (c < p.d) p.part[o.group * n + (int64_t)(kv / V) * p.d + c] = f;
    }
}

// dw [d][W] and db [d] from the groups' sums [groups][W + 1][d]
constexpr int kConvSumX = 32, kConvSumY = 16;
__global__ void __launch_bounds__(kConvSumX *kConvSumY) conv_bwd_sum(const float *part, int64_t groups, int d, int W,
                                                                       float *dw, float *db) {
    __shared__ float sums[kConvSumY][kConvSumX];
    const int64_t n = (int64_t)d * (W + 1), i = (int64_t)blockIdx.x * kConvSumX + threadIdx.x;
    float s = 0.0f;
    if (i < n)
        for (int64_t r = threadIdx.y; r < groups; r += kConvSumY) s += part[r * n + i];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && i < n) {
        s = 0.0f;
#pragma unroll
        for (int y = 0; y < kConvSumY; ++y) s += sums[y][threadIdx.x];
        const int k = (int)(i / d), c = (int)(i % d);
        if (k < W) dw[(int64_t)c * W + k] = s;
        else if (db) db[c] = s;
    }
}

// How a call is cut: runs long enough that the W - 1 tokens read twice, the taps and the
// partial sums cost little, short enough for 16 warps on every SM; strips of a CTA next to one
// another for whole lines.
struct ConvCut {
    int strips, run, across, blocks;
    int64_t groups;
};
ConvCut conv_cut(int batch, int L, int d, int V) {
    ConvCut c;
    c.strips = (d + V - 1) / V;
    const int64_t rows = (int64_t)batch * L, want = 148 * 512;
    c.run = (int)std::max<int64_t>(8, std::min<int64_t>(64, (rows * c.strips / want + 7) / 8 * 8));
    c.across = 1;
    while (c.across < 32 && c.across < c.strips) c.across *= 2;
    c.blocks = (c.strips + c.across - 1) / c.across;
    const int64_t runs = (int64_t)batch * ((L + c.run - 1) / c.run);
    c.groups = (runs + kConvThreads / c.across - 1) / (kConvThreads / c.across);
    return c;
}

// what a call's rows allow: the strip width and whether strips move as one vector
bool conv_vec(const vim_rows &r, int batch, int L, size_t el, int V) {
    return !misaligned(r.data, V * el) && (L <= 1 || r.row_stride % V == 0) && (batch <= 1 || r.batch_stride % V == 0);
}

enum ConvKind { kPrompt, kStep, kBackward };

template <typename T, int W>
vim_status conv_launch(ConvKind kind, ConvArgs &a, bool vec8, bool vec4, cudaStream_t stream) {
    // prompts and tokens in 16-byte strips; the derivative, which keeps twice the registers
    // per channel, in strips of 4
    constexpr int V = Vec<T>::n;
    const ConvCut cut = conv_cut(a.batch, a.L, a.d, kind == kBackward ? 4 : V);
    a.run = cut.run, a.across = cut.across;
    a.w16 = !misaligned(a.w, 16);
    const int64_t grid = kind == kStep ? ((int64_t)a.batch * cut.strips + kConvThreads - 1) / kConvThreads
                                       : cut.groups * cut.blocks;
    if (grid > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    auto go = [&](auto kernel) {
        if (grid > 0) kernel<<<(unsigned)grid, kConvThreads, 0, stream>>>(a);   // none: empty sequences still have states
    };
    if (kind == kPrompt) vec8 ? go(conv_prompt<T, W, V, true>) : go(conv_prompt<T, W, V, false>);
    else if (kind == kStep) vec8 ? go(conv_step<T, W, V, true>) : go(conv_step<T, W, V, false>);
    else vec4 ? go(conv_bwd<T, W, 4, true>) : go(conv_bwd<T, W, 4, false>);
    if (cudaGetLastError() != cudaSuccess) return VIM_ERR_CUDA;
    if (kind == kPrompt && a.state_out) {
        const int64_t n = ((int64_t)a.seqs.n * a.d + kConvThreads - 1) / kConvThreads;
        if (n > INT32_MAX) return VIM_ERR_UNSUPPORTED;
        if (launch_dependent(conv_states<T, W>, dim3((unsigned)n), dim3(kConvThreads), 0, stream, a) != cudaSuccess)
            return VIM_ERR_CUDA;
    }
    return VIM_OK;
}

template <typename T>
vim_status conv_width(ConvKind kind, ConvArgs &a, int W, bool vec8, bool vec4, cudaStream_t stream) {
    switch (W) {
        case 2: return conv_launch<T, 2>(kind, a, vec8, vec4, stream);
        case 3: return conv_launch<T, 3>(kind, a, vec8, vec4, stream);
        default: return conv_launch<T, 4>(kind, a, vec8, vec4, stream);
    }
}

vim_status conv_check(int batch, int L, int d, int W, vim_dtype dt, const float *w, const float *b) {
    const vim_status st = check_sizes(batch, L, d, dt);
    if (st != VIM_OK) return st;
    if (W < 2 || W > 4) return VIM_ERR_UNSUPPORTED;
    if (d > 0 && (!w || misaligned(w, 4) || misaligned(b, 4))) return VIM_ERR_INVALID_ARG;
    return VIM_OK;
}

}  // namespace
}  // namespace vimscan

using namespace vimscan;

extern "C" {

vim_status causal_conv(const vim_conv_io *io, const float *w, const float *b, int batch, int L, int channels,
                       int width, int silu, vim_dtype dt, const vim_sequences *seqs, cudaStream_t stream) {
    if (!io) return VIM_ERR_INVALID_ARG;
    const vim_rows &x = io->x, &y = io->y;
    vim_status st = conv_check(batch, L, channels, width, dt, w, b);
    if (st != VIM_OK) return st;
    ConvArgs a;
    std::memset(&a, 0, sizeof(a));
    st = make_seqs(seqs, batch, L, elem_size(dt), &a.seqs);
    if (st != VIM_OK) return st;
    if (a.seqs.n == 0 || channels == 0) return VIM_OK;
    if (L > 0 && (bad_rows(x, dt) || bad_out(y, dt, batch, L, channels))) return VIM_ERR_INVALID_ARG;
    a.x = x, a.y = y, a.w = w, a.b = b;
    a.state = seqs ? seqs->state : nullptr;
    a.state_out = seqs ? seqs->state_out : nullptr;
    a.batch = batch, a.L = L, a.d = channels, a.silu = silu != 0;
    const int V = dt == VIM_F32 ? 4 : 8;
    const bool vec = channels % V == 0 && conv_vec(x, batch, L, elem_size(dt), V) &&
                     conv_vec(y, batch, L, elem_size(dt), V) && !misaligned(a.state, 16);
    return dt == VIM_F32 ? conv_width<float>(kPrompt, a, width, vec, false, stream)
                         : conv_width<__nv_bfloat16>(kPrompt, a, width, vec, false, stream);
}

vim_status causal_conv_step(const vim_conv_io *io, const float *w, const float *b, int batch, int channels,
                            int width, int silu, vim_dtype dt, const vim_sequences *seqs, cudaStream_t stream) {
    if (!io) return VIM_ERR_INVALID_ARG;
    const vim_rows &x = io->x, &y = io->y;
    vim_status st = conv_check(batch, 1, channels, width, dt, w, b);
    if (st != VIM_OK) return st;
    if (!seqs) return VIM_ERR_INVALID_ARG;
    vim_sequences rows = *seqs;
    rows.cu_seqlens = nullptr;
    if (!rows.state_out) rows.state_out = const_cast<void *>(rows.state);
    ConvArgs a;
    std::memset(&a, 0, sizeof(a));
    st = make_seqs(&rows, batch, 1, elem_size(dt), &a.seqs);
    if (st != VIM_OK) return st;
    if (batch == 0 || channels == 0) return VIM_OK;
    if (!rows.state || bad_rows(x, dt) || bad_out(y, dt, batch, 1, channels)) return VIM_ERR_INVALID_ARG;
    a.x = x, a.y = y, a.w = w, a.b = b;
    a.state = rows.state, a.state_out = rows.state_out;
    a.batch = batch, a.L = 1, a.d = channels, a.silu = silu != 0;
    const int V = dt == VIM_F32 ? 4 : 8;
    const bool vec = channels % V == 0 && conv_vec(x, batch, 1, elem_size(dt), V) &&
                     conv_vec(y, batch, 1, elem_size(dt), V) && !misaligned(a.state, 16) && !misaligned(a.state_out, 16);
    return dt == VIM_F32 ? conv_width<float>(kStep, a, width, vec, false, stream)
                         : conv_width<__nv_bfloat16>(kStep, a, width, vec, false, stream);
}

size_t causal_conv_bwd_workspace_bytes(int batch, int L, int channels, int width) {
    if (batch <= 0 || L <= 0 || channels <= 0 || width < 2 || width > 4) return 0;
    return round_up((size_t)conv_cut(batch, L, channels, 4).groups * channels * (width + 1) * sizeof(float));
}

vim_status causal_conv_bwd(const vim_conv_bwd_io *io, const float *w, const float *b, float *dw, float *db,
                           int batch, int L, int channels, int width, int silu, vim_dtype dt,
                           const int32_t *cu_seqlens, int n_seqs, void *workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
    if (!io) return VIM_ERR_INVALID_ARG;
    const vim_rows &x = io->x, &dout = io->dout, &dx = io->dx;
    vim_status st = conv_check(batch, L, channels, width, dt, w, b);
    if (st != VIM_OK) return st;
    vim_sequences seqs;
    std::memset(&seqs, 0, sizeof(seqs));
    seqs.cu_seqlens = cu_seqlens;
    seqs.n_seqs = cu_seqlens ? n_seqs : batch;
    ConvArgs a;
    std::memset(&a, 0, sizeof(a));
    st = make_seqs(&seqs, batch, L, 16, &a.seqs);
    if (st != VIM_OK) return st;
    if (channels == 0) return VIM_OK;
    if (!dw || misaligned(dw, 4) || misaligned(db, 4) || (db && !b)) return VIM_ERR_INVALID_ARG;
    if (batch == 0 || L == 0 || a.seqs.n == 0) {           // no token: the parameters' derivatives are zero
        const size_t n = (size_t)channels * sizeof(float);
        const bool ok = cudaMemsetAsync(dw, 0, n * width, stream) == cudaSuccess &&
                        (!db || cudaMemsetAsync(db, 0, n, stream) == cudaSuccess);
        return ok ? VIM_OK : VIM_ERR_CUDA;
    }
    if (bad_rows(x, dt) || bad_rows(dout, dt) || bad_out(dx, dt, batch, L, channels)) return VIM_ERR_INVALID_ARG;
    const size_t need = causal_conv_bwd_workspace_bytes(batch, L, channels, width);
    if (!workspace || workspace_bytes < need || misaligned(workspace, kAlign)) return VIM_ERR_WORKSPACE;
    a.x = x, a.dout = dout, a.dx = dx, a.w = w, a.b = b;
    a.part = static_cast<float *>(workspace);
    a.batch = batch, a.L = L, a.d = channels, a.silu = silu != 0;
    const size_t el = elem_size(dt);
    const bool vec = channels % 4 == 0 && conv_vec(x, batch, L, el, 4) && conv_vec(dout, batch, L, el, 4) &&
                     conv_vec(dx, batch, L, el, 4);
    st = dt == VIM_F32 ? conv_width<float>(kBackward, a, width, false, vec, stream)
                       : conv_width<__nv_bfloat16>(kBackward, a, width, false, vec, stream);
    if (st != VIM_OK) return st;
    const int64_t n = (int64_t)channels * (width + 1);
    conv_bwd_sum<<<(unsigned)((n + kConvSumX - 1) / kConvSumX), dim3(kConvSumX, kConvSumY), 0, stream>>>(
        a.part, conv_cut(batch, L, channels, 4).groups, channels, width, dw, db);
    return cudaGetLastError() == cudaSuccess ? VIM_OK : VIM_ERR_CUDA;
}

}  // extern "C"
