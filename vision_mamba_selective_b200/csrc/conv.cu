// conv.cu -- short causal depthwise convolution (declared in include/vimscan_causal.h): prompts,
// single tokens and the derivative.
//
//   pre_t = b + sum_(k < W) w_k x_(t - W + 1 + k),   y_t = silu(pre_t) or pre_t
//
// The traffic is two elements per token-channel forward, three backward, so every thread walks
// down the tokens of four neighbouring channels with the last W - 1 inputs in registers: each
// input is read once, a turn of 8 (4) tokens ahead.  At bf16 the SiLU is then as long as the
// traffic: two special-function operations an element, 7.5 us for 8192 x 2048 (10.3 us of
// traffic).  Measured 21 us: 0.47 instructions a clock and scheduler at 14 warps an SM, which wait
// for fixed latencies first and for loads second, too few of them to cover either (strips of 8
// channels, or twice the warps with shorter runs: 22 to 26 us); 29 us at fp32 (20.6 of traffic).
// 8 x 4097 x 384, bf16: 16 us forward, 27 us backward.
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
    int ctas;                              // CTAs of conv_prompt that walk tokens
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
    template <Load HOW = kReadOnly> __device__ __forceinline__ void load(const char *at, int left) {
        if constexpr (VEC) {
            if constexpr (kWords == 4) {
                const uint4 q = load_as<HOW, uint4>(at);
                v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
            } else {
                const uint2 q = load_as<HOW, uint2>(at);
                v[0] = q.x, v[1] = q.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = 0;
                if (i < left) {
                    if constexpr (sizeof(T) == 4) v[i] = load_as<HOW, uint32_t>(at + 4 * i);
                    else v[i] = load_as<HOW, uint16_t>(at + 2 * i);
                }
            }
        }
    }
    __device__ __forceinline__ float f(int i) const {
        if constexpr (!VEC) return bits_f32<T>(v[i]);
        else return word_f32<T>(v[i * (int)sizeof(T) / 4], i);
    }
    __device__ __forceinline__ float2 pair(int i) const { return f2(f(2 * i), f(2 * i + 1)); }
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
// taps and bias of a strip, as pairs of channels for the packed arithmetic (columns past d
// repeat the last)
template <int W, int V>
__device__ __forceinline__ void conv_taps(const ConvArgs &p, int c, float2 (&w)[W][V / 2], float2 (&bias)[V / 2]) {
    auto at = [](float2 &v, int i) -> float & { return i % 2 ? v.y : v.x; };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ci = min(c + i, p.d - 1);
        at(bias[i / 2], i) = p.b ? __ldg(p.b + ci) : 0.0f;
        if (W == 4 && p.w16) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p.w) + ci);
            at(w[0][i / 2], i) = q.x, at(w[1][i / 2], i) = q.y;
            at(w[W - 2][i / 2], i) = q.z, at(w[W - 1][i / 2], i) = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) at(w[k][i / 2], i) = __ldg(p.w + (int64_t)ci * W + k);
        }
    }
}
__device__ __forceinline__ float2 sigmoid2(float2 x) { return f2(sigmoid(x.x), sigmoid(x.y)); }

// The last W - 1 inputs of sequence s and channel c, into its state row: all are read before any
// is written, so the row may be the one that was read.
template <typename T, int W>
__device__ __forceinline__ void conv_last(const ConvArgs &p, int64_t s, int c) {
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
// the same as a launch of its own, for states that conv_prompt reads where they are to be written
template <typename T, int W>
__global__ void __launch_bounds__(kConvThreads) conv_states(const ConvArgs p) {
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    cudaGridDependencySynchronize();
    if (i < (int64_t)p.seqs.n * p.d) conv_last<T, W>(p, i / p.d, (int)(i % p.d));
}

// Prompts.  A thread takes `run` tokens of V channels.  Where its run starts inside a
// sequence it first reads the W - 1 tokens before it, and where a sequence starts in the run
// the window is filled from that sequence's state row or zeros.
template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(kConvThreads, 4) conv_prompt(const ConvArgs p) {
    if ((int)blockIdx.x >= p.ctas) {                       // final states, to another buffer than the initial ones
        const int64_t i = (int64_t)(blockIdx.x - p.ctas) * kConvThreads + threadIdx.x;
        if (i < (int64_t)p.seqs.n * p.d) conv_last<T, W>(p, i / p.d, (int)(i % p.d));
        return;
    }
    const ConvSpot o = conv_spot<V>(p);
    if (!o.any) return;
    const int left = p.d - o.c;
    const RowsOf<T> gx(p.x, o.b, o.c), gy(p.y, o.b, o.c);
    float2 w[W][V / 2], bias[V / 2];
    conv_taps<W, V>(p, o.c, w, bias);
    int s = p.seqs.cu ? sequence_at(p.seqs, o.t0) : o.b;
    int t = o.t0;
    float2 win[W][V / 2];                                  // win[k]: x at t - W + 1 + k
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
            for (int i = 0; i < V / 2; ++i) win[k][i] = x.pair(i);
        }
        constexpr int AHEAD = 8;                           // tokens loaded together, a turn ahead
        Strip<T, V, VEC> x[AHEAD];
        auto fetch = [&](int at) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) x[j].load(gx.at(min(at + j, end - 1)), left);
        };
        fetch(begin);
#pragma unroll 1
        for (t = begin; t < end; t += AHEAD) {
            Strip<T, V, VEC> now[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) now[j] = x[j];
            if (t + AHEAD < end) fetch(t + AHEAD);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                float y[V];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    win[W - 1][i] = now[j].pair(i);
                    float2 v = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) v = fma2(w[k][i], win[k][i], v);
                    if (p.silu) v = mul2(v, sigmoid2(v));
                    y[2 * i] = v.x, y[2 * i + 1] = v.y;
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

// One token per sequence: the state row moves up by one.  A thread reads its channels of the state
// and of x before it writes any, so both may be written in place.
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
            x[k].template load<kInPlace>(reinterpret_cast<const char *>(static_cast<const T *>(p.state) + row + (int64_t)k * p.d), left);
    }
    x[W - 1].template load<kInPlace>(RowsOf<T>(p.x, b, c).at(0), left);
    float2 w[W][V / 2], v[V / 2];
    float y[V];
    conv_taps<W, V>(p, c, w, v);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) v[e] = fma2(w[k][e], x[k].pair(e), v[e]);
        if (p.silu) v[e] = mul2(v[e], sigmoid2(v[e]));
        y[2 * e] = v[e].x, y[2 * e + 1] = v[e].y;
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
// dw and db take the run's own tokens, in fp32.  The runs' sums go to `part`.  Four CTAs an SM
// leave 128 registers, in which the inputs loaded ahead do not all fit at fp32 (width 4: 188
// bytes spilled, width 3: 56; at bf16 none but 4) nor without whole vectors (up to 224).
// Forward and derivative at 8 x 4097 x 384: bf16 47 us (19 of traffic), fp32 77 us (38).
template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(kConvThreads, 4) conv_bwd(const ConvArgs p) {
    const ConvSpot o = conv_spot<V>(p);
    const int left = p.d - o.c;
    const RowsOf<T> gx(p.x, o.b, o.c), go(p.dout, o.b, o.c), gdx(p.dx, o.b, o.c);
    float2 w[W][V / 2], bias[V / 2], dw[W][V / 2], db[V / 2];
    conv_taps<W, V>(p, o.c, w, bias);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        db[i] = f2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = f2(0.0f, 0.0f);
    }
    int s = p.seqs.cu && o.any ? sequence_at(p.seqs, o.t0) : o.b;
    int t = o.t0;
#pragma unroll 1
    while (o.any && t < o.t1 && s < p.seqs.n) {
        const Seq q = sequence(p.seqs, s);
        const int begin = max(t, q.start), end = min(o.t1, q.end), stop = min(end + W - 1, q.end);
        if (begin < end) {
            float2 win[W][V / 2], ahead[W][V / 2];         // ahead[j]: dpre at t - W + 1 + j
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                const int at = begin - (W - 1) + k;
                Strip<T, V, VEC> x;
                x.clear();
                if (at >= q.start) x.load(gx.at(at), left);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) win[k][i] = x.pair(i), ahead[k][i] = f2(0.0f, 0.0f);
            }
            // token u forms dpre_u and completes dx of token u - W + 1; past `stop` dpre is zero
            constexpr int AHEAD = 4;                       // tokens loaded together, a turn ahead
            Strip<T, V, VEC> x[AHEAD], g[AHEAD];
            auto fetch = [&](int from) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int at = min(from + j, stop - 1);
                    x[j].load(gx.at(at), left);
                    g[j].load(go.at(at), left);
                }
            };
            fetch(begin);
#pragma unroll 1
            for (int u0 = begin; u0 < end + W - 1; u0 += AHEAD) {
                Strip<T, V, VEC> now_x[AHEAD], now_g[AHEAD];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) now_x[j] = x[j], now_g[j] = g[j];
                if (u0 + AHEAD < end + W - 1) fetch(u0 + AHEAD);
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int u = u0 + j;
                    float dx[V];
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        win[W - 1][i] = now_x[j].pair(i);
                        float2 dpre = now_g[j].pair(i);
                        if (p.silu) {
                            float2 pre = bias[i];
#pragma unroll
                            for (int k = 0; k < W; ++k) pre = fma2(w[k][i], win[k][i], pre);
                            const float2 sg = sigmoid2(pre);
                            // silu'(v) = s (1 + v (1 - s)) = s + v s - (v s) s
                            const float2 vs = mul2(pre, sg);
                            dpre = mul2(dpre, fma2(f2(-vs.x, -vs.y), sg, __fadd2_rn(sg, vs)));
                        }
                        if (u >= stop) dpre = f2(0.0f, 0.0f);
                        ahead[W - 1][i] = dpre;
                        if (u < end) {
                            db[i] = __fadd2_rn(db[i], dpre);
#pragma unroll
                            for (int k = 0; k < W; ++k) dw[k][i] = fma2(dpre, win[k][i], dw[k][i]);
                        }
                        float2 d = mul2(w[W - 1][i], ahead[0][i]);
#pragma unroll
                        for (int k = 1; k < W; ++k) d = fma2(w[W - 1 - k][i], ahead[k][i], d);
                        dx[2 * i] = d.x, dx[2 * i + 1] = d.y;
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
        for (int k = 0; k < W; ++k) sums[k * V + i][threadIdx.x] = i % 2 ? dw[k][i / 2].y : dw[k][i / 2].x;
        sums[W * V + i][threadIdx.x] = i % 2 ? db[i / 2].y : db[i / 2].x;
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
    // tokens in 16-byte strips; prompts and the derivative in strips of 4 channels, whose
    // registers leave room for twice the warps
    constexpr int V = Vec<T>::n;
    const ConvCut cut = conv_cut(a.batch, a.L, a.d, kind == kStep ? V : 4);
    a.run = cut.run, a.across = cut.across;
    a.w16 = !misaligned(a.w, 16);
    const int64_t grid = kind == kStep ? ((int64_t)a.batch * cut.strips + kConvThreads - 1) / kConvThreads
                                       : cut.groups * cut.blocks;
    // states: more CTAs of the same launch, unless they go where they are read
    const int64_t last = kind == kPrompt && a.state_out ? ((int64_t)a.seqs.n * a.d + kConvThreads - 1) / kConvThreads : 0;
    const bool apart = a.state == a.state_out;
    if (grid + last > INT32_MAX) return VIM_ERR_UNSUPPORTED;
    a.ctas = (int)grid;
    const unsigned total = (unsigned)(grid + (apart ? 0 : last));
    auto go = [&](auto kernel) {
        if (total > 0) kernel<<<total, kConvThreads, 0, stream>>>(a);   // none: empty sequences still have states
    };
    if (kind == kPrompt) vec4 ? go(conv_prompt<T, W, 4, true>) : go(conv_prompt<T, W, 4, false>);
    else if (kind == kStep) vec8 ? go(conv_step<T, W, V, true>) : go(conv_step<T, W, V, false>);
    else vec4 ? go(conv_bwd<T, W, 4, true>) : go(conv_bwd<T, W, 4, false>);
    if (cudaGetLastError() != cudaSuccess) return VIM_ERR_CUDA;
    if (apart && last > 0 && launch_dependent(conv_states<T, W>, dim3((unsigned)last), dim3(kConvThreads), 0, stream, a) != cudaSuccess)
        return VIM_ERR_CUDA;
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
    st = make_seqs(seqs, batch, L, elem_size(dt), (int64_t)(width - 1) * channels * elem_size(dt), &a.seqs);
    if (st != VIM_OK) return st;
    if (a.seqs.n == 0 || channels == 0) return VIM_OK;
    // (in place, tokens would be overwritten before their successors have read them)
    if (L > 0 && (bad_rows(x, dt) || bad_out(y, dt, batch, L, channels) || rows_meet(y, channels, x, channels, dt, batch, L)))
        return VIM_ERR_INVALID_ARG;
    a.x = x, a.y = y, a.w = w, a.b = b;
    a.state = seqs ? seqs->state : nullptr;
    a.state_out = seqs ? seqs->state_out : nullptr;
    a.batch = batch, a.L = L, a.d = channels, a.silu = silu != 0;
    const size_t el = elem_size(dt);
    const bool vec = channels % 4 == 0 && conv_vec(x, batch, L, el, 4) && conv_vec(y, batch, L, el, 4) &&
                     !misaligned(a.state, 4 * el);
    return dt == VIM_F32 ? conv_width<float>(kPrompt, a, width, false, vec, stream)
                         : conv_width<__nv_bfloat16>(kPrompt, a, width, false, vec, stream);
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
    st = make_seqs(&rows, batch, 1, elem_size(dt), (int64_t)(width - 1) * channels * elem_size(dt), &a.seqs);
    if (st != VIM_OK) return st;
    if (batch == 0 || channels == 0) return VIM_OK;
    if (!rows.state || bad_rows(x, dt) || bad_out(y, dt, batch, 1, channels) || rows_clash(y, x, channels, dt, batch, 1))
        return VIM_ERR_INVALID_ARG;
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
    st = make_seqs(&seqs, batch, L, 16, 0, &a.seqs);
    if (st != VIM_OK) return st;
    if (channels == 0) return VIM_OK;
    if (!dw || misaligned(dw, 4) || misaligned(db, 4) || (db && !b)) return VIM_ERR_INVALID_ARG;
    if (batch == 0 || L == 0 || a.seqs.n == 0) {           // no token: the parameters' derivatives are zero
        const size_t n = (size_t)channels * sizeof(float);
        const bool ok = cudaMemsetAsync(dw, 0, n * width, stream) == cudaSuccess &&
                        (!db || cudaMemsetAsync(db, 0, n, stream) == cudaSuccess);
        return ok ? VIM_OK : VIM_ERR_CUDA;
    }
    if (bad_rows(x, dt) || bad_rows(dout, dt) || bad_out(dx, dt, batch, L, channels) ||
        rows_meet(dx, channels, x, channels, dt, batch, L) || rows_meet(dx, channels, dout, channels, dt, batch, L))
        return VIM_ERR_INVALID_ARG;
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
