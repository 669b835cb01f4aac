// causal_kernels.cuh -- sm_100a kernels of the causal selective scan over whole sequences.
//
//   Delta_t = softplus(delta_t + bias);   h_t = exp(Delta_t A) h_(t-1) + Delta_t B_t u_t
//   y_t     = (C_t . h_t + D u_t) silu(z_t)
//
// and, with time reversed, the adjoint of h that its derivative needs:
//
//   g_t = C_t dy_t + carry_t,  carry_(t-1) = exp(Delta_t A) g_t,  dy_t = dout_t silu(z_t).
//
// What bounds it: A is free per channel and state, so every token-channel takes N
// exponentials, and the special-function unit gives 16 a clock and SM: with softplus and
// the gate's sigmoid 20 for N = 16, 1.25 clocks a token-channel, against 0.2 clocks of
// memory traffic at bf16 and 0.4 of packed FP32 work.  So no exponential may be computed
// twice, which rules out the usual two passes over chunks of a sequence (end states
// first, outputs after), and a walk by one warp per few channels has too few warps: alone
// on its scheduler a warp issues an instruction every four clocks.
//
// The walk is shared by the W warps of a CTA, which all hold the same few channels and
// take segments of SEG tokens (8; 16 or 4) in turn.  For its segment a warp
//   1. forms Delta and Delta u of its tokens, each lane its share (exchanged by shuffles);
//   2. runs the segment from h = 0, multiplying up its decays: with P_t the product so far,
//      h_t = P_t h_in + hz_t, and C_t . h_t = C_t . hz_t + (C_t P_t) . h_in; C_t P_t and the
//      first sum stay in registers, all of it without knowing h_in;
//   3. takes h_in from the warp before it and hands h_out on to the next (a multiply-add per
//      pair of states between a named barrier's wait and its arrival: the only serial part),
//   4. adds (C_t P_t) . h_in to the sums, a multiply-add per pair of states and token.
// A channel's N states lie on N / NL lanes, NL a lane in f32x2 pairs; the partial sums of
// C . h are reduced over these lanes so that each ends with the y of its own tokens, gates
// them and stores them.  Lanes of one state group are neighbours: a 16-byte read of B or C
// then costs two shared-memory clocks, and four if neighbouring lanes read different
// groups (measured).  Loads run one turn ahead in registers, by single elements, so that
// any strides and channel counts will do.  Segments are aligned to the token axis; tokens
// outside the sequence get Delta = 0 and Delta u = 0, which leave the state as it is.
//
// The adjoint, and the states kept for the derivative, are wanted only at segment borders:
// these modes end with step 3, and wait mostly for the handovers (200 to 250 clocks each).  The
// adjoint, which keeps nothing per token, therefore takes segments of 16 (8 x 4097 tokens x
// 384 channels: 90 us; taken at 95 against 105 with 8).
//
// Measured at N = 16, bf16 (the special-function floor in parentheses): 8192 packed tokens x
// 2048 channels 140 us (74), 4 x 16385 x 384 326 us (111), 8 x 4097 x 384 with kept states
// 137 us (55), 1 x 16385 x 384 139 us (28); 0.64 instructions a clock and scheduler, shared-memory pipe at 68%.
#pragma once

#include "causal.cuh"

namespace vimscan {

struct CausalArgs {
    vim_rows u, delta, z, B, C;     // z.data may be null
    vim_rows dout;                  // adjoint only
    vim_rows y;
    const float *A, *D, *bias;      // [d][N], [d], [d]
    Seqs seqs;                      // seqs.cu null: one sequence per batch row
    const float *state;             // [n_slots][d][N] or null: initial states
    float *state_out;               // [n_slots][d][N] or null: final states
    float *ckpt;                    // [batch][ceil(L / kCkEvery)][d][N] or null
    float *adj;                     // adjoint: carries, [batch][ceil(L / kAdjEvery)][d][N]
    int d;
    int vec_bc;                     // B and C can be read by a lane's states at once
};
constexpr int kCkEvery = 8;         // tokens between kept states
constexpr int kAdjEvery = 64;       // tokens between kept adjoint carries

enum CausalMode {
    kForward = 0,                   // y, and where asked for final states and kept states
    kStates = 1,                    // kept states only
    kAdjoint = 2                    // adjoint carries
};

namespace {

constexpr int kSeg = 8;             // tokens of a segment where outputs or kept states are wanted (or half)
constexpr int kLongSeg = 16;        // and of the adjoint at 16 states, and of calls with few channels
constexpr int kMostRanked = 64;     // packed sequences that are walked in the order of their lengths
constexpr int kPassWarps = 8;       // most warps of a CTA: one named barrier each
static_assert(kCkEvery == kSeg && kAdjEvery % kSeg == 0 && kAdjEvery % kLongSeg == 0 && kLongSeg == 2 * kCkEvery, "kept states lie at segment borders");

// sums p[0 .. n) over the n lanes of a channel, which are `stride` apart: the i-th of them
// gets the sum of p[i].  Each step halves the values a lane holds.
template <int n, int stride>
__device__ __forceinline__ float reduce_scatter(float (&p)[n], int q) {
#pragma unroll
    for (int half = n / 2; half >= 1; half >>= 1) {
        const bool upper = q & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = upper ? p[i] : p[i + half];
            const float keep = upper ? p[i + half] : p[i];
            p[i] = keep + __shfl_xor_sync(0xffffffffu, send, half * stride);
        }
    }
    return p[0];
}

// one warp's shared memory
template <int N, int NL, int SEG>
struct PassWarp {
    static constexpr int kLanes = N / NL;                  // lanes per channel
    static constexpr int kCh = 32 / kLanes;                // channels per warp
    alignas(16) float bc[2][SEG * N];                     // B and C of its segment
    alignas(16) float carry[32 * NL];                      // the state handed to it, by lane
};

__device__ __forceinline__ void named_wait(int id) { asm volatile("barrier.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void named_arrive(int id) { asm volatile("barrier.arrive %0, 64;" ::"r"(id) : "memory"); }

// CTAs of kPassWarps on an SM: the modes without outputs hold fewer registers, outputs of long
// segments more
constexpr int pass_ctas(int mode, int seg) { return mode != kForward ? 3 : seg == kLongSeg ? 1 : 2; }

template <typename T, int N, int NL, int SEG, int MODE, bool KEEP, bool VEC>
__global__ void __launch_bounds__(32 * kPassWarps, pass_ctas(MODE, SEG)) causal_pass(const CausalArgs p) {
    using S = PassWarp<N, NL, SEG>;
    constexpr int LPC = S::kLanes, CH = S::kCh, NP = NL / 2;
    constexpr int EPL = SEG / LPC;                        // tokens of a segment per lane
    constexpr int PV = SEG * N >= 32 ? SEG * N / 32 : 1; // B (C) values a lane fetches per segment
    constexpr bool HAS_Z = MODE != kStates, HAS_B = MODE != kAdjoint, HAS_C = MODE != kStates;
    extern __shared__ __align__(16) unsigned char pass_smem[];
    // (the warp's number by a shuffle, so that it and all that follows from it is seen to be uniform)
    const int W = blockDim.x / 32, w = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    S &sm = reinterpret_cast<S *>(pass_smem)[w];
    S &next = reinterpret_cast<S *>(pass_smem)[w + 1 == W ? 0 : w + 1];

    const int blocks = (p.d + CH - 1) / CH, c0 = (blockIdx.x % blocks) * CH;
    int s = blockIdx.x / blocks;
    if (p.seqs.cu && p.seqs.n > 1 && p.seqs.n <= kMostRanked) {
        // packed sequences from the longest to the shortest, so that no long one starts last
        // (8192 tokens x 2048 channels, mean of 8 draws, without and with it: in 11 sequences 165
        // and 146 us, in 60 203 and 174, in 64 180 and 175): CTA group k takes the sequence that k
        // others are longer than (or as long, and before).  Every CTA counts for itself, which
        // past kMostRanked costs more than the order gives (in 96 187 and 202, in 128 183 and 250)
        int *const found = reinterpret_cast<int *>(pass_smem);
        for (int i = threadIdx.x; i < p.seqs.n; i += blockDim.x) {
            const int length = p.seqs.cu[i + 1] - p.seqs.cu[i];
            int rank = 0, before = p.seqs.cu[0];
            for (int j = 0; j < p.seqs.n; ++j) {
                const int after = p.seqs.cu[j + 1], other = after - before;
                rank += other > length || (other == length && j < i);
                before = after;
            }
            if (rank == s) *found = i;
        }
        __syncthreads();
        s = *found;
        __syncthreads();
    }
    const Seq seq = sequence(p.seqs, s);
    const int64_t b = p.seqs.cu ? 0 : s;
    const int q = lane / CH, cl = lane % CH;
    const bool live = c0 + cl < p.d;
    const int c = live ? c0 + cl : p.d - 1;                // lanes past d repeat the last channel and write nothing
    if (seq.slot < 0 && !KEEP) return;                     // a padding entry
    const bool put = live && (!KEEP || seq.slot >= 0);     // (its kept states are wanted all the same)

    const vim_rows &urows = MODE == kAdjoint ? p.dout : p.u;
    const bool gate = p.z.data != nullptr;
    constexpr Load HOW = MODE == kForward ? kInPlace : kReadOnly;   // y may lie over u, delta or z
    const RowsOf<T, HOW> gu(urows, b, c), gd(p.delta, b, c), gz(gate ? p.z : p.u, b, c);
    const RowsOf<T> gy(p.y, b, c);
    const int at = lane * PV;                              // the lane's B (C) values: token, state
    const RowsOf<T> gB(p.B, b, at % N), gC(p.C, b, at % N);

    float2 A2[NP];
    load_row<NP>(p.A + (int64_t)c * N + q * NL, A2);
#pragma unroll
    for (int i = 0; i < NP; ++i) A2[i] = decay_rate(A2[i]);
    const float bias = p.bias[c], Dc = MODE == kForward ? p.D[c] : 0.0f;

    // segments of the sequence; m = 0 is the first in the order of the walk
    const int first = seq.start / SEG;
    const int M = seq.end > seq.start ? (seq.end + SEG - 1) / SEG - first : 0;
    const unsigned length = seq.end - seq.start;
    auto seg_at = [&](int m) { return (MODE == kAdjoint ? first + M - 1 - m : first + m) * SEG; };

    // as loaded: anything done to the bits here would wait for the load
    constexpr int PW = PV == 1 ? 1 : PV * (int)sizeof(T) / 4;
    uint32_t ru[EPL], rd[EPL], rz[EPL], rb[2][PW];
    // tokens outside the sequence read its nearest token; what they read is dropped
    auto nearest = [&](int t) { return min(max(t, seq.start), seq.end - 1); };
    auto fetch = [&](int m) {
        const int t0 = seg_at(m);
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int t = nearest(t0 + e * LPC + q);
            ru[e] = gu.raw(t);
            rd[e] = gd.raw(t);
            if (HAS_Z) rz[e] = gz.raw(t);
        }
        const int t = nearest(t0 + at / N);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 0 ? !HAS_B : !HAS_C) continue;
            const RowsOf<T> &g = k == 0 ? gB : gC;
            if (PV == 1) rb[k][0] = g.raw(t);
            else if (VEC) g.template words<PW>(t, rb[k]);
            else g.template gather<PW>(t, rb[k]);
        }
    };

    if (w == 0) {                                          // the sequence's initial state is the first carry
        float2 h0[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) h0[i] = f2(0.0f, 0.0f);
        if (p.state && !seq.fresh) load_row<NP>(p.state + (seq.slot * p.d + c) * N + q * NL, h0);
        store_row<NP>(&sm.carry[lane * NL], h0);
        if (M == 0 && MODE != kStates && p.state_out && put)
            store_row<NP>(p.state_out + (seq.slot * p.d + c) * N + q * NL, h0);
    }
    if (w < M) fetch(w);
#pragma unroll 1
    for (int m = w; m < M; m += W) {
        const int t0 = seg_at(m);
        // 1. the lane's tokens: (Delta, Delta u), or (Delta, dy) for the adjoint
        float u_own[EPL], z_own[EPL];
        float dt_own[EPL], x_own[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int r = e * LPC + q;
            const float u = bits_f32<T>(ru[e]), z = HAS_Z ? bits_f32<T>(rz[e]) : 0.0f;
            const float dt = softplus_acc(bits_f32<T>(rd[e]) + bias);
            const float sg = gate ? z * sigmoid(z) : 1.0f;
            const bool ok = (unsigned)(t0 + r - seq.start) < length;
            dt_own[e] = ok ? dt : 0.0f;
            x_own[e] = ok ? (MODE == kAdjoint ? u * sg : dt * u) : 0.0f;
            u_own[e] = u;
            z_own[e] = sg;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 0 ? !HAS_B : !HAS_C) continue;
            // a zero factor outside the sequence, so that Delta u = 0 (dy = 0) meets no NaN there
            const bool ok = (unsigned)(t0 + at / N - seq.start) < length;
            float f[PV];
#pragma unroll
            for (int i = 0; i < PV; ++i) {
                const uint32_t word = ok ? rb[k][i * PW / PV] : 0;
                f[i] = PV == 1 ? bits_f32<T>(word) : word_f32<T>(word, i);
            }
            if constexpr (PV % 4 == 0) {
#pragma unroll
                for (int i = 0; i < PV; i += 4)
                    *reinterpret_cast<float4 *>(&sm.bc[k][at + i]) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
            } else if (at < SEG * N) {
#pragma unroll
                for (int i = 0; i < PV; ++i) sm.bc[k][at + i] = f[i];
            }
        }
        if (m + W < M) fetch(m + W);
        __syncwarp();

        // 2. the segment from zero, the product of its decays so far, and what y takes of both
        float2 reach[MODE == kForward ? SEG : 1][NP], part0[MODE == kForward ? SEG : 1], P[NP], hz[NP];
        float2 midP[NP], midhz[NP];                        // both after the first kCkEvery of a longer segment
#pragma unroll
        for (int jj = 0; jj < SEG; ++jj) {
            const int j = MODE == kAdjoint ? SEG - 1 - jj : jj;
            const float dt = __shfl_sync(0xffffffffu, dt_own[j / LPC], j % LPC * CH + cl);
            const float x1 = __shfl_sync(0xffffffffu, x_own[j / LPC], j % LPC * CH + cl);
            float2 rowB[NP], rowC[NP];
            if (HAS_B) load_row<NP>(&sm.bc[0][j * N + q * NL], rowB);
            if (HAS_C) load_row<NP>(&sm.bc[1][j * N + q * NL], rowC);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float2 d = decay(A2[i], dt);
                P[i] = jj == 0 ? d : mul2(P[i], d);
                if (MODE == kAdjoint) {
                    const float2 x = mul2(rowC[i], f2(x1, x1));
                    hz[i] = mul2(d, jj == 0 ? x : __fadd2_rn(hz[i], x));
                } else {
                    const float2 x = mul2(rowB[i], f2(x1, x1));
                    hz[i] = jj == 0 ? x : fma2(d, hz[i], x);
                }
                if (MODE == kForward) {
                    part0[j] = i == 0 ? mul2(rowC[i], hz[i]) : fma2(rowC[i], hz[i], part0[j]);
                    reach[j][i] = mul2(rowC[i], P[i]);
                }
                if (KEEP && jj == kCkEvery - 1) midP[i] = P[i], midhz[i] = hz[i];
            }
        }

        // 3. the state entering the segment, and the one leaving it
        float2 h[NP], out[NP];
        if (m > 0 && W > 1) named_wait(w);
        load_row<NP>(&sm.carry[lane * NL], h);
#pragma unroll
        for (int i = 0; i < NP; ++i) out[i] = fma2(P[i], h[i], hz[i]);
        if (m + 1 < M) {
            store_row<NP>(&next.carry[lane * NL], out);
            if (W > 1) named_arrive(w + 1 == W ? 0 : w + 1);
        } else if (MODE != kStates && p.state_out && put) {
            store_row<NP>(p.state_out + (seq.slot * p.d + c) * N + q * NL, out);
        }
        if (KEEP && MODE != kAdjoint && (SEG >= kCkEvery || t0 % kCkEvery == 0) && t0 >= seq.start && live) {
            const int64_t row = b * ((p.seqs.L + kCkEvery - 1) / kCkEvery) + t0 / kCkEvery;
            store_row<NP>(p.ckpt + (row * p.d + c) * N + q * NL, h);
        }
        if (KEEP && MODE != kAdjoint && SEG > kCkEvery) {  // and the state in the middle
            const int t = t0 + kCkEvery;
            if (t >= seq.start && t < seq.end && live) {
                float2 mid[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i) mid[i] = fma2(midP[i], h[i], midhz[i]);
                const int64_t row = b * ((p.seqs.L + kCkEvery - 1) / kCkEvery) + t / kCkEvery;
                store_row<NP>(p.ckpt + (row * p.d + c) * N + q * NL, mid);
            }
        }
        if (MODE == kAdjoint && t0 % kAdjEvery == 0 && t0 > seq.start && live) {
            const int64_t row = b * ((p.seqs.L + kAdjEvery - 1) / kAdjEvery) + t0 / kAdjEvery - 1;
            store_row<NP>(p.adj + (row * p.d + c) * N + q * NL, out);
        }

        // 4. the segment from h
        if (MODE == kForward) {
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                float part[LPC];
#pragma unroll
                for (int l = 0; l < LPC; ++l) {
                    const int j = e * LPC + l;
                    float2 acc = part0[j];
#pragma unroll
                    for (int i = 0; i < NP; ++i) acc = fma2(reach[j][i], h[i], acc);
                    part[l] = acc.x + acc.y;
                }
                const float y = fmaf(Dc, u_own[e], reduce_scatter<LPC, CH>(part, q)) * z_own[e];
                const int t = t0 + e * LPC + q;
                if (put && (unsigned)(t - seq.start) < length) gy.put(t, y);
            }
        }
        __syncwarp();                                      // the warp's shared memory may be written again
    }
}

}  // namespace

// states of B (C) that a lane fetches of a segment
inline int lane_states(int N) { return N >= 4 ? N / 4 : 1; }

// How a call is cut: states a lane holds, tokens of a segment, warps of a CTA.  (Figures at N = 16
// and bf16 unless said otherwise.)
//   - Eight states and segments of 4 (16 channels a warp, 32-byte rows at bf16) need fewer
//     loads, shuffles and selects per token-channel than four and segments of 8, but half
//     the CTAs and twice the handovers per token: better from 8192 channels on (4 x 2048
//     tokens x 4096: 274 us against 291), worse below (1 x 4096 tokens x 2048 channels: 113
//     and 88).  Packed, where one sequence may hold most of the tokens, from 16384 on (8192
//     tokens in 11 sequences x 2048 channels: 146 and 160; in 4: 174 and 156; 4000 tokens in
//     20 x 768: 52 and 40).
//   - Where four states a lane give no SM a second CTA, up to 1184 channels, the forward mode
//     may use all registers, for segments of 16 and half the handovers (2 x 16385 tokens x 384
//     channels: 174 us against 223; 1 x 4096 x 1184: 49 and 61); and with two states a lane, half
//     as many instructions again but twice the CTAs, up to 592 (1 x 16385 x 384: 139 us, 170 with
//     four, 217 in segments of 8; 1 x 4096 x 592: 41, 49 and 59).  Past 592 the latter loses (2 x
//     16385 x 384: 266 us against 174), past 1184 the former too (1 x 4096 x 1600: 96 and 90; 4 x
//     16385 x 384: 332 and 328).
//   - Eight warps hide the handover best (11 packed sequences of 745 tokens on average: 146 us,
//     169 with four); four waste less where sequences are short (200 x 30 tokens x 384
//     channels: 31 us against 45; 64 x 100 x 768: 47 and 55; 16 x 200 x 2048: 58 and 63; still
//     123 and 130 for 64 x 300 x 768).  Where the CTAs then run in one wave instead of a full
//     and a partial one four are taken too; the two are within a few per cent there (8 x 4097 x
//     384: 134 and 132 us at bf16, 134 and 138 at fp32; 4 x 300 x 1100: 16.9 and 17.9), but 2 x
//     4000 x 2048, 172 and 161.  A row has no work for more warps than segments.
struct PassPlan {
    int states, seg, warps;
};
// channels: of all sequences together, each sequence's rounded up to a warp's
inline PassPlan pass_plan(int mode, int N, int64_t channels, bool packed, int64_t tokens_per_seq, int L) {
    PassPlan pl;
    const bool thick = N == 16 && channels >= (packed ? 16384 : 8192);
    const bool alone = N == 16 && mode == kForward && channels <= 148 * 8;
    const bool thin = alone && channels <= 148 * 4;
    pl.states = thick ? 8 : thin || N < 8 ? 2 : 4;
    pl.seg = thick ? 4 : alone || (mode == kAdjoint && N == 16) ? kLongSeg : kSeg;
    const int64_t ctas = channels * N / pl.states / 32, slots = 148 * pass_ctas(mode, pl.seg);
    pl.warps = !alone && (tokens_per_seq < 256 || (ctas > slots && ctas <= 2 * slots)) ? 4 : kPassWarps;
    const int segments = (L + pl.seg - 1) / pl.seg;
    if (segments < pl.warps) pl.warps = segments < 1 ? 1 : segments;
    return pl;
}

template <int MODE>
vim_status launch_pass(const CausalArgs &a, int N, vim_dtype dt, cudaStream_t stream);

}  // namespace vimscan
