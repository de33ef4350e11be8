// The selective scan forwards, for prompts and for single tokens
// (include/seq.h, seq_scan_run and seq_scan_step).
//
// A thread keeps NT states of two neighbouring channels in registers and
// walks along time; LN lanes side by side share the channels where a channel
// has more than NT states.  B and C of kStep tokens are converted once per
// block into shared memory, where all its channels read them; u, dt and z come
// ahead of their use through a ring in shared memory.  Per state: one ex2 and
// four multiply-adds, those packed for the two channels.
//
// What bounds it: a token of 64 channels and 16 states is 193 instructions of
// a warp (112 of them the states' own: 64 packed multiply-adds of 2 cycles, 32
// ex2 of 4, 16 loads from shared memory; the rest delta, gate, loads and the
// store), with 16 warps an SM issued in 58 % of the cycles: the latency of
// instructions that need one another, not the issue rate or memory, is what more
// warps would hide.  For 16384 tokens
// x 4096 channels in bf16 the main pass takes 286 us and the chunks' pass 197;
// its 8 bytes a token and channel would take 79 us.  Measured and not kept:
// steps of 8 tokens (that prompt 485 -> 489 us, ragged prompts 154 -> 196),
// 12 warps an SM in place of 16 (485 -> 493 us).
//
// Where batch and channels alone do not fill the GPU, time is cut into chunks
// worked on at once.  A is constant in time, so what a chunk does to the state
// it is handed is h -> exp(A S) h + e, with S its sum of delta and e the
// state it leaves from 0.  scan_state_kernel finds S and e of all chunks,
// scan_join_kernel puts them together one after the other, and the main
// kernel runs over all chunks with the states they are handed.  The exps are
// then computed twice; nothing is approximated.  (What a row's last chunk leaves
// is not needed, nor, for the gradients, what those of its first span do; they
// are worked on like the others.)
#include <algorithm>
#include <climits>
#include <new>

#include "seq_scan.cuh"

namespace seq {
namespace {

// What a thread works on: channels d and d + 1 of one group.
struct Work {
    long long b;
    int group, chunk, len;
    int tile;          // the block's first channel within the group
    int d, dp;         // the first of the thread's two channels, and its padded index
    bool on0, on1;     // whether they exist
    bool put;          // whether dp is the thread's to write: its channels, or padding (states of 0)
};

constexpr int kStep = 4;   // tokens of a pipeline step

constexpr int scan_threads(int ln) { return ln == 1 ? 64 : 128; }
// An SM's blocks, for the compiler's register limit: what waits in registers
// where rows are not WIDE takes more of them.
constexpr int scan_blocks(int ln, bool wide) { return (wide ? 8 : 6) / (ln == 1 ? 1 : 2); }

template <int LN>
__device__ __forceinline__ Work work_of(const ScanParams &p) {
    constexpr int CPB = 2 * scan_threads(LN) / LN;
    Work w;
    const int tiles = p.groups * p.tiles_per_group;
    const int tile = blockIdx.x % tiles;
    const long long rest = blockIdx.x / tiles;
    w.chunk = static_cast<int>(rest % p.n_chunks);
    w.b = rest / p.n_chunks;
    w.group = tile / p.tiles_per_group;
    w.tile = (tile % p.tiles_per_group) * CPB;
    const int c = w.tile + 2 * (threadIdx.x / LN);
    w.on0 = c < p.group_channels;
    w.on1 = c + 1 < p.group_channels;
    w.put = c < p.group_pad;
    w.dp = w.group * p.group_pad + (w.put ? c : 0);
    w.d = w.group * p.group_channels + (w.on0 ? c : 0);
    w.len = scan_length(p, w.b);
    return w;
}

// The elements of u, dt and z of a step and of the block's channels wait in
// shared memory, in a ring of kRing steps.  WIDE: rows lie in 16-byte pieces,
// which asynchronous copies bring in kRing - 1 steps ahead (a thread starts
// three of them a step for 16-bit types).  Else a step's elements go through
// registers, loaded one by one while the step before is computed.
constexpr int kRing = 3;

// REV: from the last step to the first, and grad_out takes u's place.  The
// main pass wants B and C, the chunks' pass B, or C (REV).
template <typename T, int NP, int LN, bool WIDE, bool MAIN, bool REV>
struct Walk {
    static constexpr int THREADS = scan_threads(LN), CPB = 2 * THREADS / LN;
    static constexpr int kTensors = MAIN || REV ? 3 : 2;
    static constexpr int kStage = kTensors * kStep * CPB;              // elements of a ring stage
    static constexpr int kPiece = WIDE ? 16 / (int)sizeof(T) : 1;      // elements of one copy
    static constexpr int kCols = CPB / kPiece;                         // copies of a token
    static constexpr int kCopies = (kStep * kCols + THREADS - 1) / THREADS;   // of a thread, tensor and step
    static constexpr int kBC = (kStep * 2 * NP + THREADS - 1) / THREADS;
    static constexpr int go = REV ? -kStep : kStep;

    const T *src[kTensors], *q[kBC], *any;   // any: a valid address, for copies of nothing
    int st[kTensors];
    int n, left;                    // tokens of the chunk; channels from the block's first to the group's end
    int at, bc_at;                  // the steps to be loaded next, as their first tokens
    bool qon[kBC];
    Vec<T, 1> bc[kBC], held[WIDE ? 1 : kTensors * kCopies];

    __device__ __forceinline__ Walk(const ScanParams &p, const Work &w, int first, int c0, int t1) {
        any = static_cast<const T *>(p.dt.p);
        at = bc_at = first - c0;
        n = t1 - c0;
        left = p.group_channels - w.tile;
        const int base = w.group * p.group_channels + w.tile;
        const Ref<void> *r[3] = {REV ? &p.gout : &p.u, &p.dt, &p.z};
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            st[i] = token_step(*r[i]);
            src[i] = r[i]->p ? scan_row<T>(*r[i], w.b, first) + base : nullptr;
        }
#pragma unroll
        for (int k = 0; k < kBC; ++k) {
            const int i = threadIdx.x + k * THREADS;
            const int m = i % NP;
            const bool c = i % (2 * NP) >= NP;
            const Ref<void> &br = c ? p.C : p.B;
            q[k] = scan_row<T>(br, w.b, first + i / (2 * NP)) + w.group * br.sg + m;
            qon[k] = i < kStep * 2 * NP && m < p.states && (MAIN || c == REV);
        }
    }

    __device__ __forceinline__ void advance() {
#pragma unroll
        for (int i = 0; i < kTensors; ++i)
            if (i < 2 || src[i]) src[i] += go * st[i];
        at += go;
    }

    // WIDE: starts the copies of a step into a ring stage (0 for tokens outside the chunk).
    __device__ __forceinline__ void fetch(T *stage) {
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
                const int e = threadIdx.x + k * THREADS;
                const int j = e / kCols, c = e % kCols * kPiece;
                if (kStep * kCols % THREADS != 0 && j >= kStep) continue;
                const bool on = static_cast<unsigned>(at + j) < static_cast<unsigned>(n) && c < left;
#pragma unroll
                for (int i = 0; i < kTensors; ++i) {
                    if (i == 2 && !src[i]) continue;
                    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(stage + (i * kStep + j) * CPB + c));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                                 "l"(on ? src[i] + (j * st[i] + c) : any), "r"(on ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            advance();
        }
    }
    __device__ __forceinline__ void wait() const {
        if constexpr (WIDE) asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    }

    // Else: loads a step's elements, and puts them into a ring stage.
    __device__ __forceinline__ void hold() {
        if constexpr (!WIDE) {
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
                const int e = threadIdx.x + k * THREADS;
                const int j = e / kCols, c = e % kCols;
                const bool on = j < kStep && static_cast<unsigned>(at + j) < static_cast<unsigned>(n) && c < left;
#pragma unroll
                for (int i = 0; i < kTensors; ++i)
                    held[i * kCopies + k] = elem_ahead<T>(src[i] + (j * st[i] + c), on && src[i]);
            }
            advance();
        }
    }
    __device__ __forceinline__ void put(T *stage) const {
        if constexpr (!WIDE) {
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
                const int e = threadIdx.x + k * THREADS;
                const int j = e / kCols, c = e % kCols;
                if (j >= kStep) continue;
#pragma unroll
                for (int i = 0; i < kTensors; ++i)
                    *reinterpret_cast<Vec<T, 1> *>(stage + (i * kStep + j) * CPB + c) = held[i * kCopies + k];
            }
        }
    }

    // The thread's share of a step's B and C: element i is token i / (2 NP),
    // then B's states, then C's.  Stored twice each, for the two channels of a
    // packed instruction.
    __device__ __forceinline__ void load_bc(const ScanParams &p) {
#pragma unroll
        for (int k = 0; k < kBC; ++k) {
            const int i = threadIdx.x + k * THREADS;
            const bool in = static_cast<unsigned>(bc_at + i / (2 * NP)) < static_cast<unsigned>(n);
            bc[k] = elem_ahead<T>(q[k], in && qon[k]);
            q[k] += go * token_step(i % (2 * NP) >= NP ? p.C : p.B);
        }
        bc_at += go;
    }
    __device__ __forceinline__ void store_bc(f2 *to) const {
#pragma unroll
        for (int k = 0; k < kBC; ++k) {
            const int i = threadIdx.x + k * THREADS;
            if (i < kStep * 2 * NP) to[i] = splat(bc[k][0]);
        }
    }

    // Runs compute(step, ring stage, B and C) over `steps` steps.
    template <typename F>
    __device__ __forceinline__ void run(const ScanParams &p, int steps, T *ring, f2 (*sbc)[kStep * 2 * NP], F compute) {
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < kRing - 1; ++k) fetch(ring + k * kStage);
        } else {
            hold();
            put(ring);
        }
        load_bc(p);
        store_bc(sbc[0]);
        int use = 0, fill = WIDE ? kRing - 1 : 1;   // ring stages
        for (int k = 0; k < steps; ++k) {
            wait();
            __syncthreads();
            // the stage to fill was last used before this barrier
            fetch(ring + fill * kStage);
            hold();
            load_bc(p);   // past the chunk's end nothing is loaded
            compute(k, ring + use * kStage, sbc[k & 1]);
            put(ring + fill * kStage);
            store_bc(sbc[(k + 1) & 1]);
            use = use + 1 == kRing ? 0 : use + 1;
            fill = fill + 1 == kRing ? 0 : fill + 1;
        }
    }
};

template <typename T>
__device__ __forceinline__ f2 pair_at(const T *p) {
    return Two<T, true>{*reinterpret_cast<const Vec<T, 2> *>(p)}.get();
}

template <int NT>
__device__ __forceinline__ void load_decay(const ScanParams &p, const Work &w, int n0, f2 (&A2)[NT]) {
    float a0[NT], a1[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) a0[i] = a1[i] = 0.f;
    if (w.on0) load_states<NT>(p.A, w.d, p.states, n0, a0);
    if (w.on1) load_states<NT>(p.A, w.d + 1, p.states, n0, a1);
#pragma unroll
    for (int i = 0; i < NT; ++i) A2[i] = pack2(a0[i] * kLog2e, a1[i] * kLog2e);
}

__device__ __forceinline__ f2 channel_values(const float *v, const Work &w) {
    return pack2(v && w.on0 ? v[w.d] : 0.f, v && w.on1 ? v[w.d + 1] : 0.f);
}

// NT states of the thread's channels in an internal [states][pad] buffer.
template <int NT>
__device__ __forceinline__ void put_states(const ScanParams &p, float *buf, long long outer, const Work &w, int n0,
                                           const f2 (&h)[NT]) {
    f2 *r = reinterpret_cast<f2 *>(buf + (outer * p.states + n0) * p.pad + w.dp);
#pragma unroll
    for (int i = 0; i < NT; ++i)
        if (n0 + i < p.states) r[(long long)i * (p.pad / 2)] = h[i];
}

// ------------------------------------------------------- a chunk on its own
// Forwards (REV false): S = sum of delta, e = the state after the chunk from
// 0.  For the gradients (REV): with g_t = dy_t C_t + a_(t+1) g_(t+1), e = the
// gradient a_first g_first that the chunk hands to the one before from 0.
template <typename T, int NT, int LN, bool WIDE, bool REV>
__global__ void __launch_bounds__(scan_threads(LN), scan_blocks(LN, WIDE)) scan_state_kernel(const __grid_constant__ ScanParams p) {
    begin_kernel();
    constexpr int NP = NT * LN;
    using W = Walk<T, NP, LN, WIDE, false, REV>;
    __shared__ __align__(16) f2 bc[2][kStep * 2 * NP];
    __shared__ __align__(16) char ring[kRing * W::kStage * sizeof(T)];
    const Work w = work_of<LN>(p);
    const int n0 = (threadIdx.x % LN) * NT, mine = 2 * (threadIdx.x / LN);
    const int c0 = w.chunk * p.chunk;
    const int t1 = min(w.len, c0 + p.chunk);
    if (c0 >= t1) return;
    f2 A2[NT], h[NT];
    load_decay<NT>(p, w, n0, A2);
#pragma unroll
    for (int i = 0; i < NT; ++i) h[i] = 0;
    const f2 bias = channel_values(p.dt_bias, w);
    f2 sum = 0;
    const int steps = (t1 - c0 + kStep - 1) / kStep;
    auto tokens = [&](auto tail, int at, const T *cur, const f2 *sb) {
#pragma unroll
        for (int jj = 0; jj < kStep; ++jj) {
            const int j = REV ? kStep - 1 - jj : jj;
            f2 dl = softplus_2<T>(add2(pair_at<T>(cur + (kStep + j) * W::CPB), bias));
            // behind the last token delta and x are 0 and the state stays
            if (decltype(tail)::value && at + j >= t1) dl = 0;
            sum = add2(sum, dl);
            f2 x = pair_at<T>(cur + j * W::CPB);
            if constexpr (REV) {
                if (p.z.p) {
                    const f2 z = pair_at<T>(cur + (2 * kStep + j) * W::CPB);
                    x = mul2(x, mul2(z, sigmoid_2<T>(z)));
                }
            } else {
                x = mul2(x, dl);
            }
#pragma unroll
            for (int i = 0; i < NT; i += 2) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sb + j * 2 * NP + i);
                const f2 a0 = ex2_2(fma2(dl, A2[i], splat(kEx2Bias)));
                const f2 a1 = ex2_2(fma2(dl, A2[i + 1], splat(kEx2Bias)));
                if constexpr (REV) {
                    h[i] = mul2(a0, fma2(x, v.x, h[i]));
                    h[i + 1] = mul2(a1, fma2(x, v.y, h[i + 1]));
                } else {
                    h[i] = fma2(a0, h[i], mul2(x, v.x));
                    h[i + 1] = fma2(a1, h[i + 1], mul2(x, v.y));
                }
            }
        }
    };
    W walk(p, w, c0 + (REV ? steps - 1 : 0) * kStep, c0, t1);
    walk.run(p, steps, reinterpret_cast<T *>(ring), bc, [&](int k, const T *stage, const f2 *sbc) {
        const int at = c0 + (REV ? steps - 1 - k : k) * kStep;
        const f2 *sb = sbc + (REV ? NP : 0) + n0;
        if (at + kStep <= t1) tokens(std::false_type(), at, stage + mine, sb);
        else tokens(std::true_type(), at, stage + mine, sb);
    });
    if (!w.put) return;
    const long long outer = w.b * p.n_chunks + w.chunk;
    if (n0 == 0) *reinterpret_cast<f2 *>(p.chunk_sum + outer * p.pad + w.dp) = sum;
    put_states<NT>(p, p.chunk_state, outer, w, n0, h);
}

// Puts the chunks together: h <- exp(A S_c) h + e_c, one chunk after the other
// from the row's first (REV: last), and leaves in each chunk's place the state
// (gradient) that it is handed.  One thread per state of a channel.
constexpr int kJoin = 8;   // chunks loaded at once

template <bool REV>
__global__ void __launch_bounds__(128) scan_join_kernel(const __grid_constant__ ScanParams p) {
    begin_kernel();
    const long long per = (long long)p.states * p.pad;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= p.batch * per) return;
    const long long b = i / per, r = i % per;
    const int n = static_cast<int>(r / p.pad), dp = static_cast<int>(r % p.pad);
    const int c = dp % p.group_pad;
    const bool on = c < p.group_channels;
    const long long d = dp / p.group_pad * p.group_channels + c;
    const int len = scan_length(p, b);
    const int chunks = (len + p.chunk - 1) / p.chunk;   // that have tokens
    const float a2 = on ? p.A[d * p.states + n] * kLog2e : 0.f;
    const float *first = REV ? p.gfinal : p.state;
    float h = on && first ? first[(b * p.channels + d) * p.states + n] : 0.f;
    float *const st = p.chunk_state + b * p.n_chunks * per + r;
    const float *const sum = p.chunk_sum + b * p.n_chunks * p.pad + dp;
    for (int k0 = 0; k0 < chunks; k0 += kJoin) {
        float e[kJoin], s[kJoin];
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const int at = REV ? chunks - 1 - k0 - k : k0 + k;
            const bool in = k0 + k < chunks;
            e[k] = in ? st[at * per] : 0.f;
            s[k] = in ? sum[(long long)at * p.pad] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            if (k0 + k >= chunks) break;
            const int at = REV ? chunks - 1 - k0 - k : k0 + k;
            st[at * per] = h;
            h = fmaf(ex2(a2 * s[k]), h, e[k]);
        }
    }
}

// --------------------------------------------------------------- main pass
template <typename T, int NT, int LN, bool WIDE>
__global__ void __launch_bounds__(scan_threads(LN), scan_blocks(LN, WIDE)) scan_fwd_kernel(const __grid_constant__ ScanParams p) {
    begin_kernel();
    constexpr int NP = NT * LN;
    using W = Walk<T, NP, LN, WIDE, true, false>;
    __shared__ __align__(16) f2 bc[2][kStep * 2 * NP];
    __shared__ __align__(16) char ring[kRing * W::kStage * sizeof(T)];
    const Work w = work_of<LN>(p);
    const int n0 = (threadIdx.x % LN) * NT, mine = 2 * (threadIdx.x / LN);
    const int c0 = w.chunk * p.chunk;
    const int c1 = min(static_cast<int>(p.length), c0 + p.chunk);
    const int t1 = min(w.len, c1);
    const bool lead = n0 == 0;   // of a channel pair's lanes
    // the block that has the row's last token leaves the row's state (a row of length 0: the first block)
    const bool last = w.len > c0 ? w.len <= c1 : (w.len == 0 && c0 == 0);
    f2 A2[NT], h[NT];
    load_decay<NT>(p, w, n0, A2);
    if (p.n_chunks > 1 && t1 > c0) {
        const f2 *r = reinterpret_cast<const f2 *>(p.chunk_state + ((w.b * p.n_chunks + w.chunk) * p.states + n0) * p.pad + w.dp);
#pragma unroll
        for (int i = 0; i < NT; ++i) h[i] = n0 + i < p.states ? r[(long long)i * (p.pad / 2)] : 0;
    } else {
        float s0[NT], s1[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) s0[i] = s1[i] = 0.f;
        if (p.state && w.on0) load_states<NT>(p.state, w.b * p.channels + w.d, p.states, n0, s0);
        if (p.state && w.on1) load_states<NT>(p.state, w.b * p.channels + w.d + 1, p.states, n0, s1);
#pragma unroll
        for (int i = 0; i < NT; ++i) h[i] = pack2(s0[i], s1[i]);
    }
    const f2 bias = channel_values(p.dt_bias, w), skip = channel_values(p.D, w);
    const int segments = static_cast<int>((p.length + kSeg - 1) / kSeg);
    const int steps = t1 > c0 ? (t1 - c0 + kStep - 1) / kStep : 0;
    if (steps > 0) {
        T *out = scan_row<T>(p.out, w.b, c0) + w.d;
        const int ost = token_step(p.out);
        const bool out0 = lead && w.on0, out1 = lead && w.on1;
        auto tokens = [&](auto tail, int at, const T *cur, const f2 *sb) {
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                const bool in = !decltype(tail)::value || at + j < t1;
                f2 dl = softplus_2<T>(add2(pair_at<T>(cur + (kStep + j) * W::CPB), bias));
                if (decltype(tail)::value && !in) dl = 0;
                const f2 u = pair_at<T>(cur + j * W::CPB);
                const f2 x = mul2(u, dl);
                f2 y0 = mul2(skip, u), y1 = 0;
                if constexpr (LN > 1) y0 = lead ? y0 : 0;
#pragma unroll
                for (int i = 0; i < NT; i += 2) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sb + j * 2 * NP + i);
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(sb + j * 2 * NP + NP + i);
                    h[i] = fma2(ex2_2(fma2(dl, A2[i], splat(kEx2Bias))), h[i], mul2(x, v.x));
                    h[i + 1] = fma2(ex2_2(fma2(dl, A2[i + 1], splat(kEx2Bias))), h[i + 1], mul2(x, v.y));
                    y0 = fma2(h[i], c.x, y0);
                    y1 = i == 0 ? mul2(h[1], c.y) : fma2(h[i + 1], c.y, y1);
                }
                f2 y = add2(y0, y1);
                if constexpr (LN > 1) {
                    float ya, yb;
                    unpack2(y, ya, yb);
#pragma unroll
                    for (int m = 1; m < LN; m *= 2) {
                        ya += __shfl_xor_sync(0xffffffffu, ya, m);
                        yb += __shfl_xor_sync(0xffffffffu, yb, m);
                    }
                    y = pack2(ya, yb);
                }
                if (p.z.p) {
                    const f2 z = pair_at<T>(cur + (2 * kStep + j) * W::CPB);
                    y = mul2(y, mul2(z, sigmoid_2<T>(z)));
                }
                Two<T, WIDE>::store(out + j * ost, 0, in && out0, in && out1, y);
            }
            out += kStep * ost;
        };
        W walk(p, w, c0, c0, t1);
        walk.run(p, steps, reinterpret_cast<T *>(ring), bc, [&](int k, const T *stage, const f2 *sbc) {
            const int at = c0 + k * kStep;
            if (p.ck && w.put && at % kSeg == 0) put_states<NT>(p, p.ck, w.b * segments + at / kSeg, w, n0, h);
            if (at + kStep <= t1) tokens(std::false_type(), at, stage + mine, sbc + n0);
            else tokens(std::true_type(), at, stage + mine, sbc + n0);
        });
    }
    if (!w.on0) return;
    if (lead)
        for (int t = max(t1, c0); t < c1; ++t)
            Two<T, WIDE>::store(scan_row<T>(p.out, w.b, t), w.d, w.on0, w.on1, 0);
    if (last && p.final_state) {
        float s0[NT], s1[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) unpack2(h[i], s0[i], s1[i]);
        store_states<NT>(p.final_state, w.b * p.channels + w.d, p.states, n0, s0);
        if (w.on1) store_states<NT>(p.final_state, w.b * p.channels + w.d + 1, p.states, n0, s1);
    }
}

// ------------------------------------------------------------ single tokens
// A thread has NT states of one channel (LN lanes side by side share a channel
// with more), so that delta, the gate and the addresses are worked out once
// for them, and does one or two sequences with its row of A in registers. The
// cache is read and written once, in 32-byte accesses where slots allow it;
// that is nearly all the traffic: 67 of 72 MB for 128 sequences of 4096 channels
// and 16 states, 19 us back to back (3.8 TB/s).  Issued in 26 % of
// the cycles: warps wait for the cache (four blocks of 127 registers an SM).
constexpr int kStepThreads = 128;
constexpr int kStepRows = 32768;   // of a grid's second dimension

template <int NT>
__device__ __forceinline__ void load_wide(const float *p, float (&f)[NT]) {
    if constexpr (NT % 8 == 0) {
#pragma unroll
        for (int i = 0; i < NT; i += 8)
            asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=f"(f[i]), "=f"(f[i + 1]), "=f"(f[i + 2]), "=f"(f[i + 3]), "=f"(f[i + 4]), "=f"(f[i + 5]),
                           "=f"(f[i + 6]), "=f"(f[i + 7])
                         : "l"(p + i)
                         : "memory");
    } else {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
}
template <int NT>
__device__ __forceinline__ void store_wide(float *p, const float (&f)[NT]) {
    if constexpr (NT % 8 == 0) {
#pragma unroll
        for (int i = 0; i < NT; i += 8)
            asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                         :: "f"(f[i]), "f"(f[i + 1]), "f"(f[i + 2]), "f"(f[i + 3]), "f"(f[i + 4]), "f"(f[i + 5]),
                            "f"(f[i + 6]), "f"(f[i + 7]), "l"(p + i)
                         : "memory");
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
}

// NT states of B or C from n0 on (0 past the end).
template <typename T, int NT>
__device__ __forceinline__ void load_inputs(const T *r, int n0, int states, bool wide, float (&f)[NT]) {
    if (wide) {
        constexpr int V = NT * sizeof(T) < 16 ? NT : 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < NT; i += V) {
            const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(r + n0 + i);
#pragma unroll
            for (int k = 0; k < V; ++k) f[i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) f[i] = n0 + i < states ? value<T>(r, n0 + i) : 0.f;
    }
}

template <typename T, int NT, int LN, int ROWS>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const __grid_constant__ ScanStepParams p) {
    begin_kernel();
    constexpr int CPB = kStepThreads / LN;
    const int n0 = (threadIdx.x % LN) * NT;
    const int d0 = static_cast<int>(blockIdx.x) * CPB + threadIdx.x / LN;
    const bool on = d0 < p.channels;
    const int d = on ? d0 : 0;
    const int g = p.group_channels == p.channels ? 0 : d / p.group_channels;
    const unsigned mine = (unsigned)d * p.states + n0;        // within a slot
    const long long slot = (long long)p.channels * p.states;   // elements of one
    const long long i0 = (blockIdx.y + (long long)blockIdx.z * kStepRows) * ROWS;
    // the block's sequences: their slots, then all that is read of them, then the work
    long long from[ROWS], to[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const long long i = i0 + r;
        from[r] = to[r] = -1;
        if (i >= p.batch) continue;
        from[r] = p.slots ? p.slots[i] : i;
        to[r] = p.write_slots ? p.write_slots[i] : from[r];
    }
    float A2[NT];
    load_states<NT>(p.A, d, p.states, n0, A2);
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.D ? p.D[d] : 0.f;
    float h[ROWS][NT], u[ROWS], dt[ROWS], z[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (from[r] >= p.n_slots || to[r] >= p.n_slots) {
            if (d0 == 0 && n0 == 0) *p.err = 1;
            from[r] = -1;
        }
        if (from[r] < 0) continue;
        const long long i = i0 + r;
        const float *src = p.cache + from[r] * slot + mine;
        if (p.wide_cache) {
            load_wide<NT>(src, h[r]);
        } else {
#pragma unroll
            for (int k = 0; k < NT; ++k) h[r][k] = n0 + k < p.states ? src[k] : 0.f;
        }
        u[r] = value<T>(static_cast<const T *>(p.u.p) + i * p.u.sb, d);
        dt[r] = value<T>(static_cast<const T *>(p.dt.p) + i * p.dt.sb, d);
        z[r] = p.z.p ? value<T>(static_cast<const T *>(p.z.p) + i * p.z.sb, d) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) A2[k] *= kLog2e;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const long long i = i0 + r;
        if (i >= p.batch) break;
        T *outp = static_cast<T *>(p.out.p) + i * p.out.sb + d;
        if (from[r] < 0) {   // the whole block: a row has one slot
            if (on && n0 == 0) put<T>(outp, 0, 0.f);
            continue;
        }
        float v[NT];
        load_inputs<T, NT>(static_cast<const T *>(p.B.p) + i * p.B.sb + g * p.B.sg, n0, p.states, p.wide_bc, v);
        const float dl = softplus_f<T>(dt[r] + bias);
        const float x = dl * u[r];
#pragma unroll
        for (int k = 0; k < NT; ++k) h[r][k] = fmaf(ex2(fmaf(dl, A2[k], kEx2Bias)), h[r][k], x * v[k]);
        load_inputs<T, NT>(static_cast<const T *>(p.C.p) + i * p.C.sb + g * p.C.sg, n0, p.states, p.wide_bc, v);
        float y = n0 == 0 ? skip * u[r] : 0.f;
#pragma unroll
        for (int k = 0; k < NT; ++k) y = fmaf(h[r][k], v[k], y);
#pragma unroll
        for (int m = 1; m < LN; m *= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (!on) continue;
        if (to[r] >= 0) {
            float *dst = p.cache + to[r] * slot + mine;
            if (p.wide_cache) {
                store_wide<NT>(dst, h[r]);
            } else {
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    if (n0 + k < p.states) dst[k] = h[r][k];
            }
        }
        if (n0 == 0) {
            if (p.z.p) y *= z[r] * sigmoid_f<T>(z[r]);
            put<T>(outp, 0, y);
        }
    }
}

}  // namespace

// ---------------------------------------------------------------- launches
namespace {

template <bool REV>
cudaError_t launch_join(const ScanParams &p, cudaStream_t s) {
    const long long threads = p.batch * p.states * p.pad;
    return launch(scan_join_kernel<REV>, (unsigned)((threads + 127) / 128), 128, 0, s, p);
}

template <typename T, int NT, int LN, bool WIDE, bool REV>
cudaError_t launch_walk(const ScanParams &p, unsigned grid, cudaStream_t s) {
    constexpr int threads = scan_threads(LN);
    if (REV || p.n_chunks > 1) {
        cudaError_t e = launch(scan_state_kernel<T, NT, LN, WIDE, REV>, grid, threads, 0, s, p);
        if (e == cudaSuccess) e = launch_join<REV>(p, s);
        if (REV || e != cudaSuccess) return e;
    }
    if constexpr (!REV) return launch(scan_fwd_kernel<T, NT, LN, WIDE>, grid, threads, 0, s, p);
    return cudaSuccess;
}

template <typename T, bool WIDE, bool REV>
cudaError_t by_states(const ScanParams &p, unsigned grid, cudaStream_t s) {
    switch (p.quads) {
        case 1: return launch_walk<T, 4, 1, WIDE, REV>(p, grid, s);
        case 2: return launch_walk<T, 8, 1, WIDE, REV>(p, grid, s);
        case 4: return launch_walk<T, 16, 1, WIDE, REV>(p, grid, s);
        case 8: return launch_walk<T, 16, 2, WIDE, REV>(p, grid, s);
        case 16: return launch_walk<T, 16, 4, WIDE, REV>(p, grid, s);
        default: return launch_walk<T, 16, 8, WIDE, REV>(p, grid, s);
    }
}

template <typename T, int NT, int LN>
cudaError_t launch_step(ScanStepParams p, cudaStream_t s) {
    constexpr int cpb = kStepThreads / LN;
    // 32-byte pieces of whole threads' states (16 bytes of four)
    constexpr int piece = NT % 8 == 0 ? 32 : 16;
    p.wide_cache = p.states == NT * LN && aligned(p.cache, piece);
    p.wide_bc = p.wide_bc && p.states == NT * LN;
    const unsigned cols = (unsigned)((p.channels + cpb - 1) / cpb);
    // Two sequences a block, their reads in flight together, where one each
    // makes more blocks than run at once.
    const bool two = p.batch * cols > 8LL * p.sm_count;
    const long long rows = two ? (p.batch + 1) / 2 : p.batch;
    const dim3 grid(cols, (unsigned)(rows < kStepRows ? rows : kStepRows), (unsigned)((rows + kStepRows - 1) / kStepRows));
    return two ? launch(scan_step_kernel<T, NT, LN, 2>, grid, kStepThreads, 0, s, p)
               : launch(scan_step_kernel<T, NT, LN, 1>, grid, kStepThreads, 0, s, p);
}

template <typename T>
cudaError_t step_by_states(const ScanStepParams &p, int quads, cudaStream_t s) {
    switch (quads) {
        case 1: return launch_step<T, 4, 1>(p, s);
        case 2: return launch_step<T, 8, 1>(p, s);
        case 4: return launch_step<T, 16, 1>(p, s);
        case 8: return launch_step<T, 16, 2>(p, s);
        case 16: return launch_step<T, 16, 4>(p, s);
        default: return launch_step<T, 16, 8>(p, s);
    }
}

template <typename T, bool REV>
cudaError_t by_access(bool wide, const ScanParams &p, unsigned grid, cudaStream_t s) {
    return wide ? by_states<T, true, REV>(p, grid, s) : by_states<T, false, REV>(p, grid, s);
}

template <bool REV>
cudaError_t by_type(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s) {
    if (dtype == SEQ_F32) return by_access<float, REV>(wide, p, grid, s);
    if (dtype == SEQ_F16) return by_access<f16, REV>(wide, p, grid, s);
    return by_access<bf16, REV>(wide, p, grid, s);
}

}  // namespace

// Channels of one block of the forward kernels, and blocks that an SM holds.
int scan_fwd_columns(int quads) {
    const int ln = quads <= 4 ? 1 : quads / 4;
    return 2 * scan_threads(ln) / ln;
}
int scan_fwd_resident(int quads, bool wide) { return scan_blocks(quads <= 4 ? 1 : quads / 4, wide); }

cudaError_t launch_scan_fwd(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s) {
    return by_type<false>(dtype, wide, p, grid, s);
}
cudaError_t launch_scan_rev(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s) {
    return by_type<true>(dtype, wide, p, grid, s);
}
cudaError_t launch_scan_step(seq_dtype_t dtype, const ScanStepParams &p, int quads, cudaStream_t s) {
    if (dtype == SEQ_F32) return step_by_states<float>(p, quads, s);
    if (dtype == SEQ_F16) return step_by_states<f16>(p, quads, s);
    return step_by_states<bf16>(p, quads, s);
}

}  // namespace seq
