// The short causal depthwise convolution (include/seq.h, seq_conv): prompts,
// gradients and single tokens.
//
// Every kernel is one pass over the activations: a token and channel cost
// 2 K + 5 flops forwards against two elements moved.  A thread owns V
// neighbouring channels (one access per token where rows allow it, else one
// per element), works on them in packed pairs and walks along time with the
// K - 1 last inputs in registers, so each input is loaded once, plus the K - 1
// inputs in front of each run of `run` tokens (mostly found in cache).
//
// Measured, 8 x 2048 tokens x 4096 channels, bf16, K = 4, SiLU: forwards 50 us
// (5.4 TB/s of its 268 MB, four fifths of what a copy reaches), backwards
// 104 us (3.9 TB/s of 403 MB): 28 instructions an element, issued in 48 % of the
// cycles by the 12 warps an SM that 168 registers a thread leave room for; what
// they wait for most is the result of the instruction before.
#include <algorithm>
#include <climits>
#include <new>

#include "seq_common.cuh"

namespace seq {
namespace {

constexpr int kConvThreads = 128;
constexpr int kAhead = 4, kBwdAhead = 4;   // tokens loaded before the ones that are computed
constexpr int kFwdWide = 4, kBwdWide = 4;   // channels of a thread with wide accesses
constexpr int kFwdSteps = 3;   // of the forward kernel's ring

struct ConvParams {
    long long batch, length;
    int channels, silu, run;
    int n_runs, n_cols;       // runs of tokens per row, column tiles
    Ref<void> x, y, gy, gx;
    const float *weight, *bias;
    const int *lengths;
    const void *state, *gfinal;
    void *final_state, *gstate;
    float *part;              // [parts][channels][K + 1] sums of the weights' and the bias's gradient
    int parts_per_row;
};

template <typename T>
__device__ __forceinline__ T *row_of(const Ref<void> &r, long long b, long long t) {
    return static_cast<T *>(r.p) + b * r.sb + t * r.st;
}

__device__ __forceinline__ int length_of(const int *lengths, long long b, long long length) {
    if (!lengths) return static_cast<int>(length);
    const int n = lengths[b];
    return n < 0 ? 0 : (n > length ? static_cast<int>(length) : n);
}

// V channels of one token: WIDE as one access, else one per element (those
// past the last channel 0).
template <typename T, int V, bool WIDE>
struct Chans {
    using P = std::conditional_t<WIDE, Vec<T, V>, Vec<T, 1>>;
    P p[WIDE ? 1 : V];

    static __device__ __forceinline__ Chans zero() {
        Chans c;
#pragma unroll
        for (int i = 0; i < (WIDE ? 1 : V); ++i) c.p[i] = P::zero();
        return c;
    }
    // left: channels from `at` to the last one
    static __device__ __forceinline__ Chans load(const T *at, bool on, int left) {
        Chans c;
#pragma unroll
        for (int i = 0; i < (WIDE ? 1 : V); ++i)
            c.p[i] = on && i < left ? *reinterpret_cast<const P *>(at + i) : P::zero();
        return c;
    }
    __device__ __forceinline__ void store(T *at, int left) const {
#pragma unroll
        for (int i = 0; i < (WIDE ? 1 : V); ++i)
            if (i < left) *reinterpret_cast<P *>(at + i) = p[i];
    }
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (WIDE) return pack2(p[0][2 * i], p[0][2 * i + 1]);
        else return pack2(p[2 * i][0], p[2 * i + 1][0]);
    }
    static __device__ __forceinline__ Chans from(const f2 (&v)[V / 2]) {
        Chans c;
        float f[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
        if constexpr (WIDE) {
            c.p[0] = P::from(f);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float one[1] = {f[i]};
                c.p[i] = P::from(one);
            }
        }
        return c;
    }
};

// The AHEAD tokens that a thread works on next.  RING: they wait in places of
// its own in shared memory (no other thread reads them, so no barrier is
// needed), a ring of STEPS steps filled STEPS - 1 steps ahead by asynchronous
// copies; that leaves registers for more warps, which forwards is worth it
// (training step's batch: 54 -> 49.5 us).  Else: in registers, one step ahead
// (backwards the ring changes nothing, the arithmetic being the limit).
template <typename T, int V, bool WIDE, bool RING, int AHEAD, int STEPS>
struct Feed {
    using C = Chans<T, V, WIDE>;
    C held[RING ? 1 : AHEAD];
    const T *row;        // the step to be loaded next
    C *ring;             // [STEPS][AHEAD][kConvThreads], from the thread's place on
    int st, t, end, left, put, get;

    __device__ __forceinline__ Feed(const T *row_, int st_, int t0, int end_, int left_, C *ring_)
        : row(row_), ring(RING ? ring_ + threadIdx.x : nullptr), st(st_), t(t0), end(end_), left(left_), put(0), get(0) {}
    // Starts a step's loads (tokens from end on: 0).  WIDE: the caller closes the group.
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const bool on = t + j < end;
            if constexpr (RING) {
                constexpr int bytes = V * (int)sizeof(T);
                const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(ring + (put * AHEAD + j) * kConvThreads));
                // (row is a valid address if any of its tokens is there; of none, nothing is copied)
                if (on) {
                    if constexpr (bytes == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row + j * st) : "memory");
                    else
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(row + j * st) : "memory");
                } else {
                    ring[(put * AHEAD + j) * kConvThreads] = C::zero();
                }
            } else {
                held[j] = C::load(row + j * st, on, left);
            }
        }
        row += AHEAD * st;
        t += AHEAD;
        put = put + 1 == STEPS ? 0 : put + 1;
    }
    __device__ __forceinline__ void take(C (&cur)[AHEAD]) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if constexpr (RING) cur[j] = ring[(get * AHEAD + j) * kConvThreads];
            else cur[j] = held[j];
        }
        get = get + 1 == STEPS ? 0 : get + 1;
    }
};
template <bool WIDE>
__device__ __forceinline__ void close_group() {
    if constexpr (WIDE) asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest N groups have landed.
template <bool WIDE, int N>
__device__ __forceinline__ void wait_group() {
    if constexpr (WIDE) asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The input of a row's position t, which may lie before the row (t < 0: the
// carried state, or 0) or behind its last token (0).
template <typename T, int K, int V, bool WIDE>
__device__ __forceinline__ Chans<T, V, WIDE> input_at(const ConvParams &p, long long b, int t, int len, int d) {
    using C = Chans<T, V, WIDE>;
    const int left = p.channels - d;
    if (t >= len) return C::zero();
    if (t >= 0) return C::load(row_of<T>(p.x, b, t) + d, true, left);
    if (!p.state) return C::zero();
    return C::load(static_cast<const T *>(p.state) + (b * (K - 1) + (t + K - 1)) * p.channels + d, true, left);
}

template <int K, int V>
__device__ __forceinline__ void load_weights(const float *weight, const float *bias, int channels, int d,
                                             f2 (&w)[K][V / 2], f2 (&bi)[V / 2]) {
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
        const int c = d + 2 * v;
        const bool on0 = c < channels, on1 = c + 1 < channels;
#pragma unroll
        for (int k = 0; k < K; ++k)
            w[k][v] = pack2(on0 ? weight[(long long)c * K + k] : 0.f, on1 ? weight[(long long)(c + 1) * K + k] : 0.f);
        bi[v] = bias ? pack2(on0 ? bias[c] : 0.f, on1 ? bias[c + 1] : 0.f) : 0;
    }
}

// ---------------------------------------------------------------- forward
template <typename T, int K, int V, bool WIDE>
__global__ void __launch_bounds__(kConvThreads, WIDE && sizeof(T) == 2 ? 8 : 1) conv_fwd_kernel(const __grid_constant__ ConvParams p) {
    begin_kernel();
    using C = Chans<T, V, WIDE>;
    const int col = blockIdx.x % p.n_cols;
    const long long rest = blockIdx.x / p.n_cols;
    const int run = static_cast<int>(rest % p.n_runs);
    const long long b = rest / p.n_runs;
    const int d = (col * kConvThreads + threadIdx.x) * V;
    if (d >= p.channels) return;
    const int left = p.channels - d;
    const int len = length_of(p.lengths, b, p.length);
    const int t0 = run * p.run;
    const int t1 = min(static_cast<int>(p.length), t0 + p.run);
    const int end = min(len, t1);
    const int xst = static_cast<int>(p.x.st), yst = static_cast<int>(p.y.st);
    T *yr = row_of<T>(p.y, b, t0) + d;
    constexpr int STEPS = kFwdSteps;
    __shared__ __align__(16) C ring[WIDE ? STEPS * kAhead * kConvThreads : 1];
    Feed<T, V, WIDE, WIDE, kAhead, STEPS> feed(row_of<T>(p.x, b, t0) + d, xst, t0, end, left, ring);
#pragma unroll
    for (int k = 0; k < (WIDE ? STEPS - 1 : 1); ++k) {
        feed.fetch();
        close_group<WIDE>();
    }
    f2 w[K][V / 2], bias[V / 2], win[K - 1][V / 2];
    load_weights<K, V>(p.weight, p.bias, p.channels, d, w, bias);
    if (run == 0 && p.final_state) {
        // the last K - 1 inputs of the row
        T *f = static_cast<T *>(p.final_state) + b * (K - 1) * p.channels + d;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            input_at<T, K, V, WIDE>(p, b, len - (K - 1) + j, len, d).store(f + (long long)j * p.channels, left);
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        const C x = input_at<T, K, V, WIDE>(p, b, t0 - (K - 1) + k, len, d);
#pragma unroll
        for (int v = 0; v < V / 2; ++v) win[k][v] = x.pair(v);
    }
    // kAhead tokens from t on.  EDGE: some lie behind the row's or the run's last token.
    auto tokens = [&](auto edge, int t) {
        constexpr bool EDGE = decltype(edge)::value;
        C cur[kAhead];
        if constexpr (WIDE) {
            feed.fetch();
            close_group<WIDE>();
            wait_group<WIDE, STEPS - 1>();
            feed.take(cur);
        } else {
            feed.take(cur);
            feed.fetch();
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (EDGE && t + j >= t1) break;
            f2 out[V / 2];
#pragma unroll
            for (int v = 0; v < V / 2; ++v) {
                const f2 x = cur[j].pair(v);
                f2 s = bias[v];
#pragma unroll
                for (int k = 0; k < K - 1; ++k) s = fma2(win[k][v], w[k][v], s);
                s = fma2(x, w[K - 1][v], s);
#pragma unroll
                for (int k = 0; k < K - 2; ++k) win[k][v] = win[k + 1][v];
                win[K - 2][v] = x;
                if (p.silu) s = mul2(s, sigmoid_2<T>(s));
                out[v] = EDGE && t + j >= len ? 0 : s;
            }
            C::from(out).store(yr + j * yst, left);
        }
        yr += kAhead * yst;
    };
    for (int t = t0; t < t1; t += kAhead) {
        if (t + kAhead <= end) tokens(std::false_type(), t);
        else tokens(std::true_type(), t);
    }
}

// ---------------------------------------------------------------- backward
// With q_t = grad_y_t act'(pre_t) (0 behind the row's last token):
//   grad_x_s = sum over k of weight[k] q_(s+K-1-k)  (+ grad_final where s is among the last K - 1 inputs)
//   grad_weight[k] = sum over t of q_t x_(t-K+1+k),  grad_bias = sum over t of q_t
// A thread walks t over its run and K - 1 tokens more, recomputes pre_t, and
// emits grad_x at s = t - K + 1; the sums of the weights' gradient stay in
// registers over the run, are added over the block's kConvRows runs in shared
// memory and leave as one partial row per block.
constexpr int kConvRows = 4;          // runs of a block
constexpr int kConvCols = kConvThreads / kConvRows;

template <typename T, int K, int V, bool WIDE>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(const __grid_constant__ ConvParams p) {
    begin_kernel();
    using C = Chans<T, V, WIDE>;
    __shared__ float red[kConvRows][kConvCols * V * (K + 1)];
    const int col = blockIdx.x % p.n_cols;
    const long long rest = blockIdx.x / p.n_cols;
    const int part = static_cast<int>(rest % p.parts_per_row);
    const long long b = rest / p.parts_per_row;
    const int tx = threadIdx.x % kConvCols, ty = threadIdx.x / kConvCols;
    const int run = part * kConvRows + ty;
    const int d = (col * kConvCols + tx) * V;
    f2 gw[K][V / 2], gb[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) gw[k][v] = 0;
        gb[v] = 0;
    }
    if (d < p.channels && run < p.n_runs) {
        const int left = p.channels - d;
        const int len = length_of(p.lengths, b, p.length);
        const int t0 = run * p.run;
        const int t1 = min(static_cast<int>(p.length), t0 + p.run);
        const int te = t1 + K - 1;   // q is needed up to te - 1
        const int end = min(len, te);
        const int xst = static_cast<int>(p.x.st), yst = static_cast<int>(p.gy.st), gst = static_cast<int>(p.gx.st);
        T *out_r = row_of<T>(p.gx, b, t0) + d;   // of token t0
        Feed<T, V, WIDE, false, kBwdAhead, 1> fx(row_of<T>(p.x, b, t0) + d, xst, t0, end, left, nullptr);
        Feed<T, V, WIDE, false, kBwdAhead, 1> fg(row_of<T>(p.gy, b, t0) + d, yst, t0, end, left, nullptr);
        fx.fetch();
        fg.fetch();
        f2 w[K][V / 2], bias[V / 2];
        load_weights<K, V>(p.weight, p.bias, p.channels, d, w, bias);
        // win[k] is x_(t-K+1+k), q[k] is q_(t-K+1+k)
        f2 win[K - 1][V / 2], q[K - 1][V / 2];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const C x = input_at<T, K, V, WIDE>(p, b, t0 - (K - 1) + k, len, d);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) {
                win[k][v] = x.pair(v);
                q[k][v] = 0;
            }
        }
        // kBwdAhead tokens from t on.  EDGE: some lie behind the row's or the run's
        // last token, or the grad_x to emit lies before the run.  Their terms are left
        // out, not multiplied by 0: an infinite x or weight would make them NaN.
        const int inner = min(len, t1);
        auto tokens = [&](auto edge, int t) {
            constexpr bool EDGE = decltype(edge)::value;
            C cx[kBwdAhead], cg[kBwdAhead];
            fx.take(cx);
            fg.take(cg);
            fx.fetch();
            fg.fetch();
#pragma unroll
            for (int j = 0; j < kBwdAhead; ++j) {
                const int tt = t + j;
                if (EDGE && tt >= te) break;
                const int s = tt - (K - 1);       // position whose grad_x is complete now
                f2 out[V / 2];
#pragma unroll
                for (int v = 0; v < V / 2; ++v) {
                    const f2 x = cx[j].pair(v);
                    f2 qt = cg[j].pair(v);
                    if (p.silu) {
                        f2 pre = bias[v];
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) pre = fma2(win[k][v], w[k][v], pre);
                        pre = fma2(x, w[K - 1][v], pre);
                        // SiLU'(pre) = s + pre s (1 - s)
                        f2 sg, rest;
                        sigmoid_and_rest_2<T>(pre, sg, rest);
                        qt = mul2(qt, fma2(mul2(pre, sg), rest, sg));
                    }
                    if (EDGE && tt >= len) qt = 0;
                    // tt's term of the weights' gradient; behind the run it is the next run's
                    if (!EDGE || tt < inner) {
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) gw[k][v] = fma2(qt, win[k][v], gw[k][v]);
                        gw[K - 1][v] = fma2(qt, x, gw[K - 1][v]);
                        gb[v] = add2(gb[v], qt);
                    }
                    f2 g = !EDGE || tt < len ? mul2(qt, w[0][v]) : 0;
#pragma unroll
                    for (int k = 0; k < K - 1; ++k)
                        if (!EDGE || (s + k >= t0 && s + k < len)) g = fma2(q[k][v], w[K - 1 - k][v], g);
                    out[v] = g;
#pragma unroll
                    for (int k = 0; k < K - 2; ++k) {
                        win[k][v] = win[k + 1][v];
                        q[k][v] = q[k + 1][v];
                    }
                    win[K - 2][v] = x;
                    q[K - 2][v] = qt;
                }
                if constexpr (EDGE) {
                    const int f = s - (len - (K - 1));
                    if (p.gfinal && f >= 0 && f < K - 1) {
                        const C e = C::load(static_cast<const T *>(p.gfinal) + (b * (K - 1) + f) * p.channels + d, true, left);
#pragma unroll
                        for (int v = 0; v < V / 2; ++v) out[v] = add2(out[v], e.pair(v));
                    }
                }
                if (!EDGE || s >= t0) {
                    C::from(out).store(out_r + (j - (K - 1)) * gst, left);
                } else if (s < 0 && p.gstate) {
                    C::from(out).store(static_cast<T *>(p.gstate) + (b * (K - 1) + (s + K - 1)) * p.channels + d, left);
                }
            }
            out_r += kBwdAhead * gst;
        };
        // (grad_final reaches positions len - K + 1 and on, which are emitted at tt >= len: at an edge)
        for (int t = t0; t < te; t += kBwdAhead) {
            if (t >= t0 + K - 1 && t + kBwdAhead <= inner) tokens(std::false_type(), t);
            else tokens(std::true_type(), t);
        }
    }
    float *mine = &red[ty][tx * V * (K + 1)];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) unpack2(gw[k][v], mine[2 * v * (K + 1) + k], mine[(2 * v + 1) * (K + 1) + k]);
        unpack2(gb[v], mine[2 * v * (K + 1) + K], mine[(2 * v + 1) * (K + 1) + K]);
    }
    __syncthreads();
    const long long row = (b * p.parts_per_row + part) * (long long)p.channels * (K + 1);
    const int first = col * kConvCols * V * (K + 1);
    for (int i = threadIdx.x; i < kConvCols * V * (K + 1); i += kConvThreads) {
        if (first + i >= p.channels * (K + 1)) break;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kConvRows; ++r) s += red[r][i];
        p.part[row + first + i] = s;
    }
}

constexpr int kSumWarps = 32;

// Adds the partial rows: one warp-wide column block of 32 sums, its rows split
// over the block's warps.
template <int K>
__global__ void __launch_bounds__(32 * kSumWarps) conv_grad_sum_kernel(const float *part, long long parts, int channels,
                                                            float *gw, float *gb) {
    begin_kernel();
    __shared__ float red[kSumWarps][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int n = channels * (K + 1);
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < n) {
#pragma unroll 4
        for (long long r = warp; r < parts; r += kSumWarps) s += part[r * n + i];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < n) {
        s = 0.f;
#pragma unroll
        for (int r = 0; r < kSumWarps; ++r) s += red[r][lane];
        const int d = i / (K + 1), k = i % (K + 1);
        if (k < K) gw[(long long)d * K + k] = s;
        else if (gb) gb[d] = s;
    }
}

// ---------------------------------------------------------------- single tokens
struct ConvStepParams {
    long long batch, n_slots;
    int channels, silu, n_cols;
    Ref<void> x, y;
    const float *weight, *bias;
    void *cache;
    const int *slots, *write_slots;
    uint32_t *err;
};

template <typename T, int K, int V, bool WIDE>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const __grid_constant__ ConvStepParams p) {
    begin_kernel();
    using C = Chans<T, V, WIDE>;
    const int col = blockIdx.x % p.n_cols;
    const long long i = blockIdx.x / p.n_cols;
    const int d = (col * kConvThreads + threadIdx.x) * V;
    if (d >= p.channels) return;
    const int left = p.channels - d;
    long long from = p.slots ? p.slots[i] : i;
    long long to = p.write_slots ? p.write_slots[i] : from;
    if (from >= p.n_slots || to >= p.n_slots) {
        if (d == 0) *p.err = 1;
        from = -1;
    }
    T *yr = row_of<T>(p.y, i, 0) + d;
    if (from < 0) {
        C::zero().store(yr, left);
        return;
    }
    const T *cr = static_cast<const T *>(p.cache) + from * (K - 1) * p.channels + d;
    C h[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) h[k] = C::load(cr + (long long)k * p.channels, true, left);
    h[K - 1] = C::load(row_of<T>(p.x, i, 0) + d, true, left);
    f2 w[K][V / 2], s[V / 2];
    load_weights<K, V>(p.weight, p.bias, p.channels, d, w, s);
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[v] = fma2(h[k].pair(v), w[k][v], s[v]);
        if (p.silu) s[v] = mul2(s[v], sigmoid_2<T>(s[v]));
    }
    C::from(s).store(yr, left);
    if (to < 0) return;
    T *cw = static_cast<T *>(p.cache) + to * (K - 1) * p.channels + d;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) h[k + 1].store(cw + (long long)k * p.channels, left);
}

// ---------------------------------------------------------------- dispatch
enum ConvOp { kFwd, kBwd, kStep };

// Channels a thread owns: 8 or 16 bytes of them, or two where rows allow no
// wide access.
constexpr int wide_channels(ConvOp op) { return op == kFwd ? kFwdWide : (op == kBwd ? kBwdWide : 4); }

template <ConvOp OP, typename T, int K, int V, bool WIDE>
cudaError_t launch_conv(const void *params, long long blocks, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(blocks);
    if constexpr (OP == kFwd)
        return launch(conv_fwd_kernel<T, K, V, WIDE>, grid, kConvThreads, 0, s, *static_cast<const ConvParams *>(params));
    else if constexpr (OP == kBwd)
        return launch(conv_bwd_kernel<T, K, V, WIDE>, grid, kConvThreads, 0, s, *static_cast<const ConvParams *>(params));
    else
        return launch(conv_step_kernel<T, K, V, WIDE>, grid, kConvThreads, 0, s, *static_cast<const ConvStepParams *>(params));
}

template <ConvOp OP, typename T, int V, bool WIDE>
cudaError_t conv_by_width(int width, const void *params, long long blocks, cudaStream_t s) {
    if (width == 2) return launch_conv<OP, T, 2, V, WIDE>(params, blocks, s);
    if (width == 3) return launch_conv<OP, T, 3, V, WIDE>(params, blocks, s);
    return launch_conv<OP, T, 4, V, WIDE>(params, blocks, s);
}

template <ConvOp OP, typename T>
cudaError_t conv_by_access(bool wide, int width, const void *params, long long blocks, cudaStream_t s) {
    if (wide) return conv_by_width<OP, T, wide_channels(OP), true>(width, params, blocks, s);
    return conv_by_width<OP, T, 2, false>(width, params, blocks, s);
}

template <ConvOp OP>
cudaError_t conv_dispatch(seq_dtype_t dtype, bool wide, int width, const void *params, long long blocks, cudaStream_t s) {
    if (dtype == SEQ_F32) return conv_by_access<OP, float>(wide, width, params, blocks, s);
    if (dtype == SEQ_F16) return conv_by_access<OP, f16>(wide, width, params, blocks, s);
    return conv_by_access<OP, bf16>(wide, width, params, blocks, s);
}

long long thread_goal(int sm_count) { return (long long)sm_count * 1536; }

int run_length(long long rows, long long length, long long threads_per_token, int sm_count) {
    const long long want = thread_goal(sm_count);
    int run = 64;
    while (run > 8 && rows * ((length + run - 1) / run) * threads_per_token < want) run /= 2;
    return run;
}

}  // namespace
}  // namespace seq

using namespace seq;

struct seq_conv_plan_s {
    PlanBase base;
    long long batch, length;
    int channels, width;
    seq_dtype_t dtype;
    seq_act_t act;
    void *part;
    size_t part_bytes;
};

namespace {

struct ConvShape {
    int run, n_runs, parts_per_row;
};

ConvShape conv_shape(const seq_conv_plan_s *pl, long long batch, long long length, int v) {
    ConvShape c;
    c.run = run_length(batch, length, (pl->channels + v - 1) / v, pl->base.sm_count);
    c.n_runs = static_cast<int>((length + c.run - 1) / c.run);
    c.parts_per_row = (c.n_runs + kConvRows - 1) / kConvRows;
    return c;
}

// Partial rows that any call of the plan can have: with full runs, one per
// kConvRows runs; with shorter ones run_length() has less than `want` threads
// at twice the run, which bounds the runs.
size_t most_parts(const seq_conv_plan_s *pl) {
    const long long full = pl->batch * ((pl->length + 64 * kConvRows - 1) / (64 * kConvRows));
    const long long tpt = (pl->channels + kBwdWide - 1) / kBwdWide;
    const long long some = 2 * thread_goal(pl->base.sm_count) / (kConvRows * tpt) + 1 + pl->batch;
    return (size_t)std::max(full, some);
}

size_t conv_bwd_need(const seq_conv_plan_s *pl) {
    return most_parts(pl) * (size_t)pl->channels * (pl->width + 1) * 4;
}

bool conv_wide(const seq_conv_plan_s *pl, ConvOp op, std::initializer_list<const seq_ref_t *> refs,
               std::initializer_list<const void *> flats) {
    const size_t es = elem_size(pl->dtype);
    const int v = wide_channels(op);
    if (pl->channels % v != 0) return false;
    for (const seq_ref_t *r : refs)
        if (!rows_aligned(*r, es, v * es)) return false;
    for (const void *p : flats)
        if (!aligned(p, v * es)) return false;
    return true;
}

}  // namespace

extern "C" {

dgrad_status_t seq_conv_plan(long long batch, long long length, long long channels, int width, seq_dtype_t dtype,
                             seq_act_t act, seq_conv_plan_t *plan_out) {
    if (!plan_out) return DGRAD_ERR_INVALID_ARG;
    *plan_out = nullptr;
    if (batch < 1 || length < 1 || channels < 1 || width < 1) return DGRAD_ERR_INVALID_ARG;
    if ((int)dtype < 0 || dtype > SEQ_BF16 || (act != SEQ_ACT_NONE && act != SEQ_ACT_SILU))
        return DGRAD_ERR_INVALID_ARG;
    if (width < 2 || width > 4 || length > INT_MAX - 4096 || channels > (1 << 24) || batch > (1 << 24))
        return DGRAD_ERR_UNSUPPORTED;
    // grid: at most one block per (batch row, 8 tokens, 32 channels)
    if ((double)batch * ((length + 7) / 8) * ((channels + 31) / 32) > 2.0e9) return DGRAD_ERR_UNSUPPORTED;
    seq_conv_plan_s *pl = new (std::nothrow) seq_conv_plan_s();
    if (!pl) return DGRAD_ERR_OOM;
    const dgrad_status_t st = open_plan(&pl->base);
    if (st != DGRAD_OK) {
        delete pl;
        return st;
    }
    pl->batch = batch;
    pl->length = length;
    pl->channels = static_cast<int>(channels);
    pl->width = width;
    pl->dtype = dtype;
    pl->act = act;
    *plan_out = pl;
    return DGRAD_OK;
}

dgrad_status_t seq_conv_run(seq_conv_plan_t pl, const seq_conv_args_t *a, void *stream) {
    if (!pl || !a || !a->x.ptr || !a->y.ptr || !a->weight) return DGRAD_ERR_INVALID_ARG;
    if (a->batch < 1 || a->batch > pl->batch || a->length < 1 || a->length > pl->length || !strides_ok(a->x) ||
        !strides_ok(a->y))
        return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype);
    if (!all_aligned(es, {a->x.ptr, a->y.ptr, a->state, a->final_state}) ||
        !all_aligned(4, {a->weight, a->bias, a->lengths}))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels;
    const size_t state_b = (size_t)a->batch * (pl->width - 1) * D * es;
    const Span y = span(a->y, a->batch, a->length, 1, D, es);
    if (!rows_distinct(y)) return DGRAD_ERR_INVALID_ARG;
    const Span outs[] = {y, flat(a->final_state, state_b)};
    const Span ins[] = {span(a->x, a->batch, a->length, 1, D, es), flat(a->state, state_b),
                        flat(a->weight, D * pl->width * 4), flat(a->bias, D * 4), flat(a->lengths, a->batch * 4)};
    if (any_overlap(outs, 2, ins, 5)) return DGRAD_ERR_ALIAS;
    dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    const bool wide = conv_wide(pl, kFwd, {&a->x, &a->y}, {a->state, a->final_state});
    const int v = wide ? wide_channels(kFwd) : 2;
    const ConvShape c = conv_shape(pl, a->batch, a->length, v);
    ConvParams p{};
    p.batch = a->batch;
    p.length = a->length;
    p.channels = pl->channels;
    p.silu = pl->act == SEQ_ACT_SILU;
    p.run = c.run;
    p.n_runs = c.n_runs;
    p.n_cols = (int)((D + (long long)kConvThreads * v - 1) / ((long long)kConvThreads * v));
    p.x = ref<void>(a->x);
    p.y = ref<void>(a->y);
    p.weight = a->weight;
    p.bias = a->bias;
    p.lengths = a->lengths;
    p.state = a->state;
    p.final_state = a->final_state;
    return dgrad::cuda_status(conv_dispatch<kFwd>(pl->dtype, wide, pl->width, &p, a->batch * c.n_runs * p.n_cols,
                                                  static_cast<cudaStream_t>(stream)));
}

dgrad_status_t seq_conv_backward(seq_conv_plan_t pl, const seq_conv_grad_args_t *a, void *stream) {
    if (!pl || !a || !a->x.ptr || !a->grad_y.ptr || !a->grad_x.ptr || !a->weight || !a->grad_weight)
        return DGRAD_ERR_INVALID_ARG;
    if (a->batch < 1 || a->batch > pl->batch || a->length < 1 || a->length > pl->length || !strides_ok(a->x) ||
        !strides_ok(a->grad_y) || !strides_ok(a->grad_x) || (a->grad_state && !a->state) ||
        (a->grad_bias && !a->bias))
        return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype);
    if (!all_aligned(es, {a->x.ptr, a->grad_y.ptr, a->grad_x.ptr, a->state, a->grad_state, a->grad_final}) ||
        !all_aligned(4, {a->weight, a->bias, a->lengths, a->grad_weight, a->grad_bias}))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels;
    const int K = pl->width;
    const size_t state_b = (size_t)a->batch * (K - 1) * D * es;
    const Span gx = span(a->grad_x, a->batch, a->length, 1, D, es);
    if (!rows_distinct(gx)) return DGRAD_ERR_INVALID_ARG;
    const Span outs[] = {gx, flat(a->grad_state, state_b), flat(a->grad_weight, D * K * 4), flat(a->grad_bias, D * 4)};
    const Span ins[] = {span(a->x, a->batch, a->length, 1, D, es), span(a->grad_y, a->batch, a->length, 1, D, es),
                        flat(a->state, state_b), flat(a->grad_final, state_b), flat(a->weight, D * K * 4),
                        flat(a->bias, D * 4), flat(a->lengths, a->batch * 4)};
    if (any_overlap(outs, 4, ins, 7)) return DGRAD_ERR_ALIAS;
    dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    const bool wide = conv_wide(pl, kBwd, {&a->x, &a->grad_y, &a->grad_x}, {a->state, a->grad_state, a->grad_final});
    const int v = wide ? wide_channels(kBwd) : 2;
    const ConvShape c = conv_shape(pl, a->batch, a->length, v);
    if ((st = grow(&pl->part, &pl->part_bytes, conv_bwd_need(pl))) != DGRAD_OK) return st;
    ConvParams p{};
    p.batch = a->batch;
    p.length = a->length;
    p.channels = pl->channels;
    p.silu = pl->act == SEQ_ACT_SILU;
    p.run = c.run;
    p.n_runs = c.n_runs;
    p.n_cols = (int)((D + (long long)kConvCols * v - 1) / ((long long)kConvCols * v));
    p.x = ref<void>(a->x);
    p.gy = ref<void>(a->grad_y);
    p.gx = ref<void>(a->grad_x);
    p.weight = a->weight;
    p.bias = a->bias;
    p.lengths = a->lengths;
    p.state = a->state;
    p.gfinal = a->grad_final;
    p.gstate = a->grad_state;
    p.part = static_cast<float *>(pl->part);
    p.parts_per_row = c.parts_per_row;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = dgrad::cuda_status(conv_dispatch<kBwd>(pl->dtype, wide, K, &p, a->batch * c.parts_per_row * p.n_cols, s));
    if (st != DGRAD_OK) return st;
    const long long parts = a->batch * c.parts_per_row;
    const unsigned grid = (unsigned)((D * (K + 1) + 31) / 32);
    auto *const sum = K == 2 ? conv_grad_sum_kernel<2> : (K == 3 ? conv_grad_sum_kernel<3> : conv_grad_sum_kernel<4>);
    return dgrad::cuda_status(
        launch(sum, grid, 32 * kSumWarps, 0, s, p.part, parts, p.channels, a->grad_weight, a->grad_bias));
}

dgrad_status_t seq_conv_step(seq_conv_plan_t pl, const seq_conv_step_args_t *a, void *stream) {
    if (!pl || !a || !a->x.ptr || !a->y.ptr || !a->weight || !a->cache) return DGRAD_ERR_INVALID_ARG;
    if (a->batch < 1 || a->batch > pl->batch || a->n_slots < 1 || (!a->slots && a->n_slots < a->batch) ||
        !strides_ok(a->x) || !strides_ok(a->y))
        return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype);
    if (!all_aligned(es, {a->x.ptr, a->y.ptr, a->cache}) ||
        !all_aligned(4, {a->weight, a->bias, a->slots, a->write_slots}))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels;
    const Span y = span(a->y, a->batch, 1, 1, D, es);
    if (!rows_distinct(y)) return DGRAD_ERR_INVALID_ARG;
    const Span outs[] = {y, flat(a->cache, (size_t)a->n_slots * (pl->width - 1) * D * es)};
    const Span ins[] = {span(a->x, a->batch, 1, 1, D, es), flat(a->weight, D * pl->width * 4), flat(a->bias, D * 4),
                        flat(a->slots, a->batch * 4), flat(a->write_slots, a->batch * 4)};
    if (any_overlap(outs, 2, ins, 5)) return DGRAD_ERR_ALIAS;
    const dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    const bool wide = conv_wide(pl, kStep, {&a->x, &a->y}, {a->cache});
    const int v = wide ? wide_channels(kStep) : 2;
    ConvStepParams p{};
    p.batch = a->batch;
    p.n_slots = a->n_slots;
    p.channels = pl->channels;
    p.silu = pl->act == SEQ_ACT_SILU;
    p.n_cols = (int)((D + (long long)kConvThreads * v - 1) / ((long long)kConvThreads * v));
    p.x = ref<void>(a->x);
    p.y = ref<void>(a->y);
    p.weight = a->weight;
    p.bias = a->bias;
    p.cache = a->cache;
    p.slots = a->slots;
    p.write_slots = a->write_slots;
    p.err = pl->base.err;
    return dgrad::cuda_status(
        conv_dispatch<kStep>(pl->dtype, wide, pl->width, &p, a->batch * p.n_cols, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t seq_conv_check(seq_conv_plan_t pl) { return pl ? read_error(pl->base) : DGRAD_ERR_INVALID_ARG; }

size_t seq_conv_workspace_bytes(seq_conv_plan_t pl, int gradients) {
    return pl ? kErrorBytes + (gradients ? conv_bwd_need(pl) : 0) : 0;
}

void seq_conv_destroy(seq_conv_plan_t pl) {
    if (!pl) return;
    close_plan(pl->base, &pl->part, 1);
    delete pl;
}

}  // extern "C"
