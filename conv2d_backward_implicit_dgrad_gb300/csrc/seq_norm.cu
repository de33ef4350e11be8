// The norms around a block with its gate and residual scale (include/seq.h,
// seq_norm), forwards and backwards.
//
// One pass over the rows: a row's elements stay with the threads that loaded
// them while its sums (one for each norm, one more backwards) go around the
// block, so every tensor is moved once.  A row belongs to one warp or one block.
// Rows that do not lie in pieces of 16 (8) bytes are copied to shared memory in
// the pieces that do, and shifted into place there.
//
// Measured, 16384 rows of 4096 channels in bf16 with a gate: forwards 112 us
// (6.0 TB/s of 671 MB), backwards 273 us (3.9 TB/s of 1074 MB): 79 instructions
// an element, issued in half of the cycles by 16 warps an SM, which wait for
// shared memory, loads and the instructions before in about equal parts.
#include <algorithm>
#include <climits>
#include <new>

#include "seq_common.cuh"

namespace seq {
namespace {

struct NormParams {
    long long rows;
    int channels, tpr;        // threads per row: 32 or the block
    int gate_act;             // SEQ_ACT_NONE: no gate
    float eps, inv_n;
    Ref<void> y, gate, res, res_out, x;
    Ref<void> gro, gx, gy, ggate, gres;
    const float *post, *scale, *next;
    float *part;              // [grid][sums][channels]: gradients of next, post, scale
    int n_part;               // sums per partial row
    int device;
    int stages;               // rows that a block of the backward kernel holds in shared memory
    int params_wide;          // post, scale and next lie on 16 bytes
};

template <typename T, int VEC, int E>
struct Row {
    Vec<T, VEC> v[E / VEC];
    __device__ __forceinline__ float operator[](int i) const { return v[i / VEC][i % VEC]; }
    __device__ __forceinline__ f2 pair(int k) const { return pack2((*this)[2 * k], (*this)[2 * k + 1]); }
};

// Element i of the thread lies at channel at(i): vectors interleaved over the
// row's threads, so that a warp's accesses are contiguous.
template <int VEC>
__device__ __forceinline__ int channel_of(int j, int t, int tpr) {
    return (j * tpr + t) * VEC;
}

template <typename T, int VEC, int E>
__device__ __forceinline__ Row<T, VEC, E> load_row(const Ref<void> &r, long long row, int t, int tpr, int channels) {
    Row<T, VEC, E> out;
    const T *p = static_cast<const T *>(r.p) + row * r.sb;
#pragma unroll
    for (int j = 0; j < E / VEC; ++j) {
        const int c = channel_of<VEC>(j, t, tpr);
        out.v[j] = c < channels ? *reinterpret_cast<const Vec<T, VEC> *>(p + c) : Vec<T, VEC>::zero();
    }
    return out;
}

template <typename T, int VEC, int E>
__device__ __forceinline__ void store_row(const Ref<void> &r, long long row, int t, int tpr, int channels,
                                          const float (&f)[E]) {
    T *p = static_cast<T *>(r.p) + row * r.sb;
#pragma unroll
    for (int j = 0; j < E / VEC; ++j) {
        const int c = channel_of<VEC>(j, t, tpr);
        if (c >= channels) continue;
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = f[j * VEC + v];
        *reinterpret_cast<Vec<T, VEC> *>(p + c) = Vec<T, VEC>::from(o);
    }
}

// A parameter's values at the thread's channels (absent, or past the row: def).
template <int VEC, int E, bool SHIFT>
__device__ __forceinline__ void load_param(const float *w, int t, int tpr, int channels, bool wide, float def,
                                           float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E / VEC; ++j) {
        const int c = channel_of<VEC>(j, t, tpr);
        constexpr int Q = VEC < 4 ? VEC : 4;
#pragma unroll
        for (int v = 0; v < VEC; v += Q) {
            if (w && (!SHIFT || wide) && (SHIFT ? c + v + Q : c + 1) <= channels) {
                const Vec<float, Q> q = *reinterpret_cast<const Vec<float, Q> *>(w + c + v);
#pragma unroll
                for (int i = 0; i < Q; ++i) f[j * VEC + v + i] = q[i];
            } else {
#pragma unroll
                for (int i = 0; i < Q; ++i) f[j * VEC + v + i] = SHIFT && w && c + v + i < channels ? w[c + v + i] : def;
            }
        }
    }
}

// ---------------------------------------------------------------- rows at any alignment
// A row that does not lie in pieces of V elements (16 or 8 bytes) is moved in
// the pieces that do: those wholly inside the row as one access, the elements
// before the first and behind the last (`edge`, at most V - 1 each) one by one
// by the row's first 2 V threads.  Piece g of the image has the elements
// g V - s to g V - s + V - 1, with s the first element's place in its piece;
// what a thread works on, elements c to c + V - 1, is two of them side by side
// from element s on.  Nothing outside the row is read or written.
template <typename X, int V>
struct Pieces {
    int s, whole;   // pieces before `whole` end inside the row
    int channels;
    __device__ __forceinline__ Pieces(const X *row, int channels_)
        : s(static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(X) % V)), whole((channels_ + s) / V),
          channels(channels_) {}
    __device__ __forceinline__ bool inside(int g) const { return g >= (s > 0) && g < whole; }
    // The edge element of thread t, or -1.
    __device__ __forceinline__ int edge(int t) const {
        if (t < V) return s > 0 && t < V - s && t < channels ? t : -1;
        const int i = whole * V - s + t - V;
        return t < 2 * V && (whole > 0 || s == 0) && i < channels ? i : -1;
    }
};

// Elements k to k + V - 1 of two pieces side by side.
template <typename X, int V>
__device__ __forceinline__ Vec<X, V> side_by_side(const Vec<X, V> &lo, const Vec<X, V> &hi, int k) {
    constexpr int N = Vec<X, V>::N;
    uint32_t a[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a[i] = lo.w[i];
        a[N + i] = hi.w[i];
    }
    const int bytes = k * (int)sizeof(X);
    if constexpr (N == 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) a[i] = (bytes & 8) ? a[i + 2] : a[i];
    }
#pragma unroll
    for (int i = 0; i <= N; ++i) a[i] = (bytes & 4) && i + 1 < 2 * N ? a[i + 1 < 2 * N ? i + 1 : i] : a[i];
    Vec<X, V> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.w[i] = sizeof(X) == 2 ? __funnelshift_r(a[i], a[i + 1], (bytes & 2) * 8) : a[i];
    return v;
}

// Starts the copies of a row's whole pieces into its image, and loads the thread's edge element.
template <typename X, int V, int E>
__device__ __forceinline__ Vec<X, 1> fetch_image(const Ref<void> &r, long long row, X *image, int t, int tpr, int channels) {
    if (!r.p) return Vec<X, 1>::zero();
    const X *p = static_cast<const X *>(r.p) + row * r.sb;
    const Pieces<X, V> q(p, channels);
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
        const int g = j * tpr + t;
        if (!q.inside(g)) continue;
        constexpr int bytes = V * sizeof(X);
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(image + g * V));
        if constexpr (bytes == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + (g * V - q.s)) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(p + (g * V - q.s)) : "memory");
    }
    const int i = q.edge(t);
    return elem_ahead<X>(p + (i < 0 ? 0 : i), i >= 0);
}
template <typename X, int V>
__device__ __forceinline__ void put_edge(const Ref<void> &r, long long row, X *image, int t, int channels, Vec<X, 1> v) {
    if (!r.p) return;
    const Pieces<X, V> q(static_cast<const X *>(r.p) + row * r.sb, channels);
    const int i = q.edge(t);
    if (i >= 0) *reinterpret_cast<Vec<X, 1> *>(image + i + q.s) = v;
}
// The thread's elements from c on (0 past the row's end; absent tensors: 0).
template <typename X, int V>
__device__ __forceinline__ Vec<X, V> from_image(const Ref<void> &r, long long row, const X *image, int c, int channels) {
    if (!r.p || c >= channels) return Vec<X, V>::zero();
    const Pieces<X, V> q(static_cast<const X *>(r.p) + row * r.sb, channels);
    const Vec<X, V> *at = reinterpret_cast<const Vec<X, V> *>(image + c);
    Vec<X, V> v = side_by_side<X, V>(at[0], at[1], q.s);
    if (c + V > channels) {
        constexpr int per = 4 / (int)sizeof(X);   // elements of a word
#pragma unroll
        for (int i = 0; i < Vec<X, V>::N; ++i) {
            const int left = channels - c - i * per;
            v.w[i] = left >= per ? v.w[i] : (left == 1 ? v.w[i] & 0xffffu : 0u);
        }
    }
    return v;
}
// Writes a row whose elements c to c + V - 1 lie in slot(c / V).
template <typename X, int V, int E, typename Slot>
__device__ __forceinline__ void flush_row(const Ref<void> &r, long long row, int t, int tpr, int channels, Slot slot) {
    X *p = static_cast<X *>(r.p) + row * r.sb;
    const Pieces<X, V> q(p, channels);
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
        const int g = j * tpr + t;
        if (!q.inside(g)) continue;
        const Vec<X, V> own = *slot(g);
        *reinterpret_cast<Vec<X, V> *>(p + (g * V - q.s)) =
            q.s ? side_by_side<X, V>(*slot(g - 1), own, V - q.s) : own;
    }
    const int i = q.edge(t);
    if (i >= 0) *reinterpret_cast<Vec<X, 1> *>(p + i) = reinterpret_cast<const Vec<X, 1> *>(slot(i / V))[i % V];
}
template <bool WARP_ROW>
__device__ __forceinline__ void row_barrier() {
    if constexpr (WARP_ROW) __syncwarp();
    else __syncthreads();
}

// Sums of N values over the row's threads.  Two buffers in turn: a warp that
// writes one again has passed the barrier of the sum in between, which every
// warp reaches after it has read the first.
template <int N, bool WARP_ROW>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[32][2], int &turn) {
#pragma unroll
    for (int m = 16; m > 0; m /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if constexpr (!WARP_ROW) {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][warp][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane < warps ? red[turn][lane][i] : 0.f;
#pragma unroll
        for (int m = 16; m > 0; m /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
        turn ^= 1;
    }
}

// The gate's factor.
template <typename T>
__device__ __forceinline__ float gate_factor(int act, float g) {
    const float s = sigmoid_f<T>(g);
    return act == SEQ_ACT_SILU ? g * s : s;
}

// ---------------------------------------------------------------- forward
template <typename T, typename RT, int VEC, int E>
__host__ __device__ constexpr int fwd_image_bytes(int tpr) {
    return ((E * tpr + VEC) * (int)(sizeof(RT) + 2 * sizeof(T)) + 15) / 16 * 16;
}
template <typename X, int VEC, int E>
__device__ __forceinline__ void to_image(X *image, int t, int tpr, const float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E / VEC; ++j) {
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = f[j * VEC + v];
        reinterpret_cast<Vec<X, VEC> *>(image)[j * tpr + t] = Vec<X, VEC>::from(o);
    }
}

// SHIFT: rows do not lie in pieces of VEC elements; they come through an image
// in shared memory and leave through one.
template <typename T, typename RT, int VEC, int E, bool WARP_ROW, bool SHIFT>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const __grid_constant__ NormParams p) {
    begin_kernel();
    __shared__ float red[2][32][2];
    extern __shared__ __align__(16) char sm[];
    const int t = WARP_ROW ? threadIdx.x % 32 : threadIdx.x;
    const long long row = WARP_ROW ? (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    if (row >= p.rows) return;   // whole warps; a block-wide row is always there
    int turn = 0;
    Row<T, VEC, E> y, g;
    Row<RT, VEC, E> r;
    // the row's images: residual, y, gate; then x in y's place, r' in the residual's
    const int image = E * p.tpr + VEC;   // elements
    char *const mine = sm + (WARP_ROW ? (threadIdx.x / 32) * fwd_image_bytes<T, RT, VEC, E>(p.tpr) : 0);
    RT *const ri = reinterpret_cast<RT *>(mine);
    T *const yi = reinterpret_cast<T *>(ri + image), *const gi = yi + image;
    if constexpr (SHIFT) {
        const Vec<RT, 1> re = fetch_image<RT, VEC, E>(p.res, row, ri, t, p.tpr, p.channels);
        const Vec<T, 1> ye = fetch_image<T, VEC, E>(p.y, row, yi, t, p.tpr, p.channels);
        const Vec<T, 1> ge = fetch_image<T, VEC, E>(p.gate, row, gi, t, p.tpr, p.channels);
        asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
        put_edge<RT, VEC>(p.res, row, ri, t, p.channels, re);
        put_edge<T, VEC>(p.y, row, yi, t, p.channels, ye);
        put_edge<T, VEC>(p.gate, row, gi, t, p.channels, ge);
        row_barrier<WARP_ROW>();
#pragma unroll
        for (int j = 0; j < E / VEC; ++j) {
            const int c = channel_of<VEC>(j, t, p.tpr);
            r.v[j] = from_image<RT, VEC>(p.res, row, ri, c, p.channels);
            y.v[j] = from_image<T, VEC>(p.y, row, yi, c, p.channels);
            g.v[j] = from_image<T, VEC>(p.gate, row, gi, c, p.channels);
        }
    } else {
        y = load_row<T, VEC, E>(p.y, row, t, p.tpr, p.channels);
        r = load_row<RT, VEC, E>(p.res, row, t, p.tpr, p.channels);
        if (p.gate_act) g = load_row<T, VEC, E>(p.gate, row, t, p.tpr, p.channels);
    }
    float b[E], w[E];
    float r1 = 1.f;
    if (p.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] = fmaf(y[i], y[i], s[0]);
        row_sum<1, WARP_ROW>(s, red, turn);
        r1 = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
    }
    load_param<VEC, E, SHIFT>(p.post, t, p.tpr, p.channels, p.params_wide, 1.f, w);
#pragma unroll
    for (int i = 0; i < E; ++i) b[i] = y[i] * r1 * w[i];
    if (p.gate_act) {
#pragma unroll
        for (int i = 0; i < E; ++i) b[i] *= gate_factor<T>(p.gate_act, g[i]);
    }
    load_param<VEC, E, SHIFT>(p.scale, t, p.tpr, p.channels, p.params_wide, 1.f, w);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        b[i] = fmaf(b[i], w[i], r[i]);
        s[0] = fmaf(b[i], b[i], s[0]);
    }
    if constexpr (SHIFT) {
        row_barrier<WARP_ROW>();   // every thread has its elements out of the images
        to_image<RT, VEC, E>(ri, t, p.tpr, b);
    } else {
        store_row<RT, VEC, E>(p.res_out, row, t, p.tpr, p.channels, b);
    }
    load_param<VEC, E, SHIFT>(p.next, t, p.tpr, p.channels, p.params_wide, 0.f, w);
    row_sum<1, WARP_ROW>(s, red, turn);
    const float r2 = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
#pragma unroll
    for (int i = 0; i < E; ++i) b[i] *= r2 * w[i];
    if constexpr (SHIFT) {
        to_image<T, VEC, E>(yi, t, p.tpr, b);
        row_barrier<WARP_ROW>();
        flush_row<RT, VEC, E>(p.res_out, row, t, p.tpr, p.channels,
                              [&](int g) { return reinterpret_cast<const Vec<RT, VEC> *>(ri) + g; });
        flush_row<T, VEC, E>(p.x, row, t, p.tpr, p.channels,
                             [&](int g) { return reinterpret_cast<const Vec<T, VEC> *>(yi) + g; });
    } else {
        store_row<T, VEC, E>(p.x, row, t, p.tpr, p.channels, b);
    }
}

// ---------------------------------------------------------------- backward
// With n1 = y r1, p = n1 post, b = act(g) p, r' = res + scale b, n2 = r' r2,
// dn = grad_x next, all recomputed:
//   dr = grad_residual_out + r2 (dn - n2 mean(dn n2))      = grad_residual
//   db = dr scale,  grad_gate = db p act'(g),  dp = db act(g)
//   d1 = dp post,  grad_y = r1 (d1 - n1 mean(d1 n1))
// and, summed over rows: grad_next = grad_x n2, grad_scale = dr b,
// grad_post = dp n1.  A block walks rows grid apart with those sums in
// registers and leaves one partial row.  While it works on a row, each thread
// copies its elements of the next one into places of its own in shared memory
// (cp.async; no other thread reads them, so no barrier is needed).  SHIFT: the
// next row comes as an image, out of which each thread then fills its places,
// and the results leave through these.  Where a second row has no room (one
// that does not lie in pieces then is moved by single elements) the rows are
// taken one by one.

// Work goes in pieces of 8 elements, so that only r' and the sums of a
// thread's E elements stay in registers.

// Where a thread keeps its elements of a row: [tensor][vector][thread].  FULL:
// no element lies past the row's end.
template <typename T, typename RT, int VEC, int E, bool FULL>
struct Slots {
    char *base;
    int threads;
    static constexpr int kT = E * (int)sizeof(T), kR = E * (int)sizeof(RT);   // bytes of a thread and tensor
    static constexpr int kBytes = 3 * kT + 2 * kR;
    // y, gate, grad_x, residual, grad_residual_out
    template <typename X, int I>
    __device__ __forceinline__ Vec<X, VEC> *at(int j) const {
        constexpr int off = I < 3 ? I * kT : 3 * kT + (I - 3) * kR;
        return reinterpret_cast<Vec<X, VEC> *>(base + off * threads) + j * threads + threadIdx.x;
    }
    // Piece m (8 elements) of tensor I, in pairs.
    template <typename X, int I>
    __device__ __forceinline__ void get(int m, f2 (&v)[4]) const {
        Row<X, VEC, 8> r;
#pragma unroll
        for (int j = 0; j < 8 / VEC; ++j) r.v[j] = *at<X, I>(m * (8 / VEC) + j);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = r.pair(k);
    }
    template <typename X, int I>
    __device__ __forceinline__ void fetch(const Ref<void> &r, long long row, int t, int tpr, int channels) const {
        if (!r.p) return;
        const X *p = static_cast<const X *>(r.p) + row * r.sb;
#pragma unroll
        for (int j = 0; j < E / VEC; ++j) {
            const int c = channel_of<VEC>(j, t, tpr);
            if (!FULL && c >= channels) continue;
            if constexpr (VEC > 1) {
                constexpr int bytes = VEC * sizeof(X);
                const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(at<X, I>(j)));
                if constexpr (bytes == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + c) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(p + c) : "memory");
            } else {
                *at<X, I>(j) = elem<X>(p, c);
            }
        }
    }
    __device__ __forceinline__ void fetch_row(const NormParams &p, long long row, int t) const {
        fetch<T, 0>(p.y, row, t, p.tpr, p.channels);
        fetch<T, 1>(p.gate, row, t, p.tpr, p.channels);
        fetch<T, 2>(p.gx, row, t, p.tpr, p.channels);
        fetch<RT, 3>(p.res, row, t, p.tpr, p.channels);
        fetch<RT, 4>(p.gro, row, t, p.tpr, p.channels);
    }
};

// Piece m of a parameter at the thread's channels, in pairs (past the row: 0).
template <int VEC, bool FULL, bool SHIFT>
__device__ __forceinline__ void param_piece(const float *w, int m, int t, const NormParams &p, f2 (&f)[4]) {
    constexpr int Q = VEC < 4 ? VEC : 4;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i += Q) {
        const int c = channel_of<VEC>(m * (8 / VEC) + i / VEC, t, p.tpr) + i % VEC;
        if (SHIFT && !(p.params_wide && c + Q <= p.channels)) {
#pragma unroll
            for (int k = 0; k < Q; ++k) v[i + k] = c + k < p.channels ? w[c + k] : 0.f;
            continue;
        }
        Vec<float, Q> q = Vec<float, Q>::zero();
        if (FULL || SHIFT || c < p.channels) q = *reinterpret_cast<const Vec<float, Q> *>(w + c);
#pragma unroll
        for (int k = 0; k < Q; ++k) v[i + k] = q[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = pack2(v[2 * k], v[2 * k + 1]);
}

// The thread's values of a tensor, in pairs, to the output or (SHIFT) the thread's place of an input no longer needed.
template <typename X, int I, int VEC, bool FULL, bool SHIFT, typename S>
__device__ __forceinline__ void store_piece(const S &now, const Ref<void> &r, long long row, int m, int t, int tpr, int channels,
                                            const f2 (&v)[4]) {
    X *p = static_cast<X *>(r.p) + row * r.sb;
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack2(v[k], f[2 * k], f[2 * k + 1]);
#pragma unroll
    for (int j = 0; j < 8 / VEC; ++j) {
        const int c = channel_of<VEC>(m * (8 / VEC) + j, t, tpr);
        if (!FULL && c >= channels) continue;
        float o[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = f[j * VEC + k];
        if constexpr (SHIFT) *now.template at<X, I>(m * (8 / VEC) + j) = Vec<X, VEC>::from(o);
        else *reinterpret_cast<Vec<X, VEC> *>(p + c) = Vec<X, VEC>::from(o);
    }
}

__device__ __forceinline__ float halves(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}

constexpr int kPairThreads = 320;   // of a block that shares its SM, where rows come as images

// Bytes of a row's images: residual, grad_residual_out, y, gate, grad_x.
template <typename T, typename RT, int VEC, int E>
__host__ __device__ constexpr int bwd_image_bytes(int tpr) {
    return ((E * tpr + VEC) * (int)(2 * sizeof(RT) + 3 * sizeof(T)) + 15) / 16 * 16;
}

template <typename T, typename RT, int VEC, int E, int MOST, bool FULL, bool SHIFT>
__global__ void __launch_bounds__(MOST, MOST == kPairThreads ? 2 : 512 / MOST) norm_bwd_kernel(const __grid_constant__ NormParams p) {
    begin_kernel();
    constexpr bool WARP_ROW = MOST == 128;
    constexpr int M = E / 8;   // pieces
    extern __shared__ __align__(16) char sm[];
    __shared__ float red[2][32][2];
    const int threads = blockDim.x;
    const int t = WARP_ROW ? threadIdx.x % 32 : threadIdx.x;
    const int per_block = WARP_ROW ? threads / 32 : 1;
    const long long step = (long long)gridDim.x * per_block;
    long long row = WARP_ROW ? (long long)blockIdx.x * per_block + threadIdx.x / 32 : blockIdx.x;
    using S = Slots<T, RT, VEC, E, FULL>;
    S now{sm, threads}, then{sm + (p.stages - 1) * S::kBytes * threads, threads};
    // SHIFT: the images, and the thread's edge elements of the row to come
    const int image = E * p.tpr + VEC;   // elements
    RT *const ri = reinterpret_cast<RT *>(sm + S::kBytes * threads +
                                          (WARP_ROW ? (threadIdx.x / 32) * bwd_image_bytes<T, RT, VEC, E>(p.tpr) : 0));
    RT *const oi = ri + image;
    T *const yi = reinterpret_cast<T *>(oi + image), *const gi = yi + image, *const xi = gi + image;
    Vec<RT, 1> re, oe;
    Vec<T, 1> ye, ge, xe;
    auto images = [&](long long row) {
        re = fetch_image<RT, VEC, E>(p.res, row, ri, t, p.tpr, p.channels);
        oe = fetch_image<RT, VEC, E>(p.gro, row, oi, t, p.tpr, p.channels);
        ye = fetch_image<T, VEC, E>(p.y, row, yi, t, p.tpr, p.channels);
        ge = fetch_image<T, VEC, E>(p.gate, row, gi, t, p.tpr, p.channels);
        xe = fetch_image<T, VEC, E>(p.gx, row, xi, t, p.tpr, p.channels);
    };
    // channels past the row stay 0
    for (int i = threadIdx.x; i < p.stages * S::kBytes * threads / 16; i += threads)
        reinterpret_cast<uint4 *>(sm)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int turn = 0;
    const bool silu = p.gate_act == SEQ_ACT_SILU;
    f2 gn[M][4], gp[M][4], gs[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) gn[m][k] = gp[m][k] = gs[m][k] = 0;
    if (row < p.rows) {
        if constexpr (SHIFT) images(row);
        else now.fetch_row(p, row, t);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (; row < p.rows; row += step) {
        if constexpr (SHIFT) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            put_edge<RT, VEC>(p.res, row, ri, t, p.channels, re);
            put_edge<RT, VEC>(p.gro, row, oi, t, p.channels, oe);
            put_edge<T, VEC>(p.y, row, yi, t, p.channels, ye);
            put_edge<T, VEC>(p.gate, row, gi, t, p.channels, ge);
            put_edge<T, VEC>(p.gx, row, xi, t, p.channels, xe);
            row_barrier<WARP_ROW>();   // the images are there, and the row before is written
#pragma unroll
            for (int j = 0; j < E / VEC; ++j) {
                const int c = channel_of<VEC>(j, t, p.tpr);
                *now.template at<RT, 3>(j) = from_image<RT, VEC>(p.res, row, ri, c, p.channels);
                if (p.gro.p) *now.template at<RT, 4>(j) = from_image<RT, VEC>(p.gro, row, oi, c, p.channels);
                *now.template at<T, 0>(j) = from_image<T, VEC>(p.y, row, yi, c, p.channels);
                if (p.gate_act) *now.template at<T, 1>(j) = from_image<T, VEC>(p.gate, row, gi, c, p.channels);
                *now.template at<T, 2>(j) = from_image<T, VEC>(p.gx, row, xi, c, p.channels);
            }
            row_barrier<WARP_ROW>();   // and may be filled again
            if (row + step < p.rows) images(row + step);
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
            if (p.stages == 2 && row + step < p.rows) then.fetch_row(p, row + step, t);
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
        float r1 = 1.f;
        if (p.post) {
            f2 q = 0;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                f2 y[4];
                now.template get<T, 0>(m, y);
#pragma unroll
                for (int k = 0; k < 4; ++k) q = fma2(y[k], y[k], q);
            }
            float s[1] = {halves(q)};
            row_sum<1, WARP_ROW>(s, red, turn);
            r1 = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
        }
        const f2 r11 = splat(r1);
        f2 rp[M][4];   // r' = residual + scale act(gate) p
        f2 q0 = 0, q1 = 0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            f2 a[4], w[4];
            now.template get<T, 0>(m, a);
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = mul2(a[k], r11);
            if (p.post) {
                param_piece<VEC, FULL, SHIFT>(p.post, m, t, p, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] = mul2(a[k], w[k]);
            }
            if (p.gate_act) {
                now.template get<T, 1>(m, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f2 sg = sigmoid_2<T>(w[k]);
                    a[k] = mul2(a[k], silu ? mul2(w[k], sg) : sg);
                }
            }
            if (p.scale) {
                param_piece<VEC, FULL, SHIFT>(p.scale, m, t, p, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] = mul2(a[k], w[k]);
            }
            now.template get<RT, 3>(m, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                rp[m][k] = add2(a[k], w[k]);
                q0 = fma2(rp[m][k], rp[m][k], q0);
            }
            param_piece<VEC, FULL, SHIFT>(p.next, m, t, p, w);
            now.template get<T, 2>(m, a);
#pragma unroll
            for (int k = 0; k < 4; ++k) q1 = fma2(mul2(a[k], w[k]), rp[m][k], q1);
        }
        float s2[2] = {halves(q0), halves(q1)};
        row_sum<2, WARP_ROW>(s2, red, turn);
        const float r2 = rsqrtf(fmaf(s2[0], p.inv_n, p.eps));
        const f2 r22 = splat(r2), m2 = splat(-s2[1] * r2 * p.inv_n);   // - mean(dn n2)
        q0 = 0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            f2 dr[4], a[4], w[4];
            now.template get<T, 2>(m, a);
            param_piece<VEC, FULL, SHIFT>(p.next, m, t, p, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f2 n2 = mul2(rp[m][k], r22);
                gn[m][k] = fma2(a[k], n2, gn[m][k]);
                dr[k] = mul2(r22, fma2(n2, m2, mul2(a[k], w[k])));
            }
            if (p.gro.p) {
                now.template get<RT, 4>(m, a);
#pragma unroll
                for (int k = 0; k < 4; ++k) dr[k] = add2(dr[k], a[k]);
            }
            store_piece<RT, 3, VEC, FULL, SHIFT>(now, p.gres, row, m, t, p.tpr, p.channels, dr);
            f2 n1[4], pv[4];   // p = n1 post
            now.template get<T, 0>(m, n1);
#pragma unroll
            for (int k = 0; k < 4; ++k) pv[k] = n1[k] = mul2(n1[k], r11);
            if (p.post) {
                param_piece<VEC, FULL, SHIFT>(p.post, m, t, p, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) pv[k] = mul2(n1[k], w[k]);
            }
            f2 sc[4] = {splat(1.f), splat(1.f), splat(1.f), splat(1.f)};
            if (p.scale) param_piece<VEC, FULL, SHIFT>(p.scale, m, t, p, sc);
            if (p.gate_act) {
                f2 g[4];
                now.template get<T, 1>(m, g);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f2 sg, rest;
                    sigmoid_and_rest_2<T>(g[k], sg, rest);
                    const f2 act = silu ? mul2(g[k], sg) : sg;
                    const f2 dact = silu ? fma2(act, rest, sg) : mul2(sg, rest);
                    const f2 db = mul2(dr[k], sc[k]);
                    gs[m][k] = fma2(dr[k], mul2(act, pv[k]), gs[m][k]);
                    g[k] = mul2(mul2(db, pv[k]), dact);
                    dr[k] = mul2(db, act);   // dp
                }
                store_piece<T, 1, VEC, FULL, SHIFT>(now, p.ggate, row, m, t, p.tpr, p.channels, g);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    gs[m][k] = fma2(dr[k], pv[k], gs[m][k]);
                    dr[k] = mul2(dr[k], sc[k]);
                }
            }
            if (p.post) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    gp[m][k] = fma2(dr[k], n1[k], gp[m][k]);
                    dr[k] = mul2(dr[k], w[k]);   // d1
                    q0 = fma2(dr[k], n1[k], q0);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) rp[m][k] = dr[k];
        }
        f2 m1 = 0;
        if (p.post) {
            float s3[1] = {halves(q0)};
            row_sum<1, WARP_ROW>(s3, red, turn);
            m1 = splat(-s3[0] * p.inv_n * r1);   // - mean(d1 n1) r1
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            f2 y[4];
            now.template get<T, 0>(m, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = p.post ? mul2(r11, fma2(y[k], m1, rp[m][k])) : rp[m][k];
            store_piece<T, 0, VEC, FULL, SHIFT>(now, p.gy, row, m, t, p.tpr, p.channels, y);
        }
        if constexpr (SHIFT) {
            row_barrier<WARP_ROW>();
            const int first = threadIdx.x - t;
            auto place = [&](int g) { return g / p.tpr * threads + first + g % p.tpr; };
            const Vec<RT, VEC> *const r0 = now.template at<RT, 3>(0) - threadIdx.x;
            const Vec<T, VEC> *const y0 = now.template at<T, 0>(0) - threadIdx.x;
            const Vec<T, VEC> *const g0 = now.template at<T, 1>(0) - threadIdx.x;
            flush_row<RT, VEC, E>(p.gres, row, t, p.tpr, p.channels, [&](int g) { return r0 + place(g); });
            flush_row<T, VEC, E>(p.gy, row, t, p.tpr, p.channels, [&](int g) { return y0 + place(g); });
            if (p.gate_act)
                flush_row<T, VEC, E>(p.ggate, row, t, p.tpr, p.channels, [&](int g) { return g0 + place(g); });
        } else if (p.stages == 2) {
            const S was = now;
            now = then;
            then = was;
        } else if (row + step < p.rows) {
            now.fetch_row(p, row + step, t);
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
    }
    // the block's sums
    __syncthreads();
    float *const sum = reinterpret_cast<float *>(sm);   // [3][E * 32], of a block of several rows
    for (int w = 0; w < per_block; ++w) {
        if (WARP_ROW && (int)threadIdx.x / 32 != w) {
            __syncthreads();
            continue;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = channel_of<VEC>(i / VEC, t, p.tpr) + i % VEC;
            float a[2], b[2], d[2];
            unpack2(gn[i / 8][i % 8 / 2], a[0], a[1]);
            unpack2(gp[i / 8][i % 8 / 2], b[0], b[1]);
            unpack2(gs[i / 8][i % 8 / 2], d[0], d[1]);
            if (!FULL && c >= p.channels) continue;
            if constexpr (WARP_ROW) {
                sum[c] = (w ? sum[c] : 0.f) + a[i % 2];
                sum[32 * E + c] = (w ? sum[32 * E + c] : 0.f) + b[i % 2];
                sum[64 * E + c] = (w ? sum[64 * E + c] : 0.f) + d[i % 2];
            } else {
                float *q = p.part + (long long)blockIdx.x * p.n_part * p.channels + c;
                *q = a[i % 2];
                if (p.post) *(q += p.channels) = b[i % 2];
                if (p.scale) *(q += p.channels) = d[i % 2];
            }
        }
        if constexpr (WARP_ROW) __syncthreads();
    }
    if constexpr (WARP_ROW) {
        for (int c = threadIdx.x; c < p.channels; c += threads) {
            float *q = p.part + (long long)blockIdx.x * p.n_part * p.channels + c;
            *q = sum[c];
            if (p.post) *(q += p.channels) = sum[32 * E + c];
            if (p.scale) *(q += p.channels) = sum[64 * E + c];
        }
    }
}

constexpr int kSumWarps = 32;

// Adds the partial rows: 32 sums per block, the rows split over its warps.
__global__ void __launch_bounds__(32 * kSumWarps) norm_grad_sum_kernel(const float *part, int parts, int n, int channels,
                                                            float *g0, float *g1, float *g2) {
    begin_kernel();
    __shared__ float red[kSumWarps][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < n) {
#pragma unroll 4
        for (int r = warp; r < parts; r += kSumWarps) s += part[(long long)r * n + i];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < n) {
        s = 0.f;
#pragma unroll
        for (int r = 0; r < kSumWarps; ++r) s += red[r][lane];
        const int which = i / channels, c = i % channels;
        (which == 0 ? g0 : which == 1 ? g1 : g2)[c] = s;
    }
}

// ---------------------------------------------------------------- dispatch
constexpr int kElems = 8;   // elements of a row per thread, forwards
constexpr int kNormMostSmem = 200 * 1024;

// Elements of a row per thread backwards.  16 where a row then still has
// enough threads: the three sums around the block, the copies' addresses and
// the waits cost a thread the same for 16 as for 8 (16384 rows of 4096
// channels in bf16: 302 us, with 8 318), and the registers of 512 threads
// reach for rows of 8192.  Rows that come as images take more shared memory
// and registers, and 8 elements as far as 512 threads reach (3000 rows of 3001
// in fp32: 226 us, with 16 295); blocks of up to kPairThreads threads are kept
// to the registers of two of them an SM (training steps of 12644 x 1026, whose
// blocks have 160 threads: four an SM 174 us, three 201).
constexpr int kFewThreads = 256;
int bwd_elems(int channels, bool wide) { return channels <= 8 * (wide ? kFewThreads : 512) ? 8 : 16; }

template <typename T, typename RT, int VEC, int E, int MOST, bool SHIFT>
cudaError_t launch_norm_bwd(NormParams p, unsigned grid, int block, cudaStream_t s) {
    constexpr int per_thread = Slots<T, RT, VEC, E, false>::kBytes;
    const int images = SHIFT ? block / p.tpr * bwd_image_bytes<T, RT, VEC, E>(p.tpr) : 0;
    // Rows that have no room for an image beside their places go by single elements.
    if constexpr (SHIFT && E == 16) {
        if (images + per_thread * block > kNormMostSmem)
            return launch_norm_bwd<T, RT, 1, E, MOST, false>(p, grid, block, s);
    }
    p.stages = !SHIFT && VEC > 1 && 2 * per_thread * block <= kNormMostSmem ? 2 : 1;
    const int smem = std::max(p.stages * per_thread * block + images, MOST == 128 ? 3 * E * 32 * 4 : 0);
    // Rows that give every thread all its elements need no tests for the row's end
    // (a training step of those rows: 390 us, with the tests 418).
    constexpr bool can = VEC > 1 && MOST != 128 && !SHIFT;
    const bool full = can && p.channels == E * block;
    auto *k = full ? norm_bwd_kernel<T, RT, VEC, E, MOST, can, SHIFT> : norm_bwd_kernel<T, RT, VEC, E, MOST, false, SHIFT>;
    static SmemLimit limits[2];   // (the most that a row of this kernel can ask for)
    const cudaError_t e = limits[full].raise(k, std::max(kNormMostSmem, per_thread * MOST), p.device);
    if (e != cudaSuccess) return e;
    return launch(k, grid, block, smem, s, p);
}

template <typename T, typename RT, int VEC, bool WARP_ROW, bool SHIFT>
cudaError_t launch_norm_fwd(const NormParams &p, unsigned grid, int block, cudaStream_t s) {
    const int smem = SHIFT ? block / p.tpr * fwd_image_bytes<T, RT, VEC, kElems>(p.tpr) : 0;
    auto *k = norm_fwd_kernel<T, RT, VEC, kElems, WARP_ROW, SHIFT>;
    if constexpr (SHIFT && !WARP_ROW) {
        static SmemLimit limit;
        const cudaError_t e = limit.raise(k, fwd_image_bytes<T, RT, VEC, kElems>(1024), p.device);
        if (e != cudaSuccess) return e;
    }
    return launch(k, grid, block, smem, s, p);
}

template <bool BWD, typename T, typename RT, int VEC, bool SHIFT>
cudaError_t launch_norm(const NormParams &p, unsigned grid, int block, cudaStream_t s) {
    if constexpr (BWD) {
        if (p.tpr == 32) return launch_norm_bwd<T, RT, VEC, 8, 128, SHIFT>(p, grid, block, s);
        if (block <= (SHIFT ? kPairThreads : kFewThreads) && bwd_elems(p.channels, !SHIFT) == 8)
            return launch_norm_bwd<T, RT, VEC, 8, (SHIFT ? kPairThreads : kFewThreads), SHIFT>(p, grid, block, s);
        if constexpr (SHIFT) {
            if (bwd_elems(p.channels, false) == 8) return launch_norm_bwd<T, RT, VEC, 8, 512, SHIFT>(p, grid, block, s);
        }
        return launch_norm_bwd<T, RT, VEC, 16, 512, SHIFT>(p, grid, block, s);
    } else {
        if (p.tpr == 32) return launch_norm_fwd<T, RT, VEC, true, SHIFT>(p, grid, block, s);
        return launch_norm_fwd<T, RT, VEC, false, SHIFT>(p, grid, block, s);
    }
}

template <bool BWD, typename T, typename RT, int WIDE>
cudaError_t norm_by_access(bool wide, const NormParams &p, unsigned grid, int block, cudaStream_t s) {
    if (wide) return launch_norm<BWD, T, RT, WIDE, false>(p, grid, block, s);
    // fp32 forwards by single elements, already 4 bytes each (6000 rows of 2045:
    // 53 us, with images 58); else images (3398 rows of 1657 in bf16 forwards:
    // 19.4 us, by elements 22.3; training steps of 12644 x 1026 in fp16 174 and
    // 253, of 4000 x 4099 in bf16 386 and 572).
    if constexpr (!BWD && sizeof(T) == 4) return launch_norm<BWD, T, RT, 1, false>(p, grid, block, s);
    else return launch_norm<BWD, T, RT, WIDE, true>(p, grid, block, s);
}

template <bool BWD>
cudaError_t norm_dispatch(seq_dtype_t dtype, seq_dtype_t rtype, bool wide, const NormParams &p, unsigned grid,
                          int block, cudaStream_t s) {
    if (dtype == SEQ_F32) return norm_by_access<BWD, float, float, 4>(wide, p, grid, block, s);
    if (dtype == SEQ_F16)
        return rtype == SEQ_F32 ? norm_by_access<BWD, f16, float, 4>(wide, p, grid, block, s)
                                : norm_by_access<BWD, f16, f16, 8>(wide, p, grid, block, s);
    return rtype == SEQ_F32 ? norm_by_access<BWD, bf16, float, 4>(wide, p, grid, block, s)
                            : norm_by_access<BWD, bf16, bf16, 8>(wide, p, grid, block, s);
}

constexpr int kNormMostChannels = 1024 * kElems;

}  // namespace
}  // namespace seq

using namespace seq;

struct seq_norm_plan_s {
    PlanBase base;
    long long rows;
    int channels;
    seq_dtype_t dtype, rtype;
    seq_act_t gate_act;
    float eps;
    void *part;
    size_t part_bytes;
};

namespace {

struct NormShape {
    int tpr, block;
};

// Threads of a row of `elems` a thread: a warp where that reaches (four rows
// to a block), else a block.
NormShape norm_shape(int channels, int elems) {
    NormShape s;
    s.tpr = ((channels + elems - 1) / elems + 31) / 32 * 32;
    s.block = s.tpr == 32 ? 128 : s.tpr;
    return s;
}

// Blocks of the backward kernel: each leaves a partial row of the parameters'
// gradients, so no more than fill the GPU.
int norm_bwd_grid(const seq_norm_plan_s *pl, long long rows, const NormShape &s, bool wide) {
    const int per_block = s.tpr == 32 ? s.block / 32 : 1;
    const long long fill = (long long)pl->base.sm_count * std::max(1, (wide || s.tpr == 32 ? 512 : 2 * kPairThreads) / s.block);
    return (int)std::min(fill, (rows + per_block - 1) / per_block);
}

// Partial rows of any call of the plan.
size_t norm_bwd_need(const seq_norm_plan_s *pl) {
    int blocks = 0;
    for (const bool w : {false, true})
        blocks = std::max(blocks, norm_bwd_grid(pl, pl->rows, norm_shape(pl->channels, bwd_elems(pl->channels, w)), w));
    return (size_t)blocks * 3 * pl->channels * 4;
}

bool norm_refs_wide(const seq_norm_plan_s *pl, std::initializer_list<const seq_ref_t *> acts,
                    std::initializer_list<const seq_ref_t *> residuals, std::initializer_list<const float *> params) {
    const size_t es = elem_size(pl->dtype), rs = elem_size(pl->rtype);
    const int v = (es == 4 || rs == 4) ? 4 : 8;
    if (pl->channels % v) return false;
    for (const seq_ref_t *r : acts)
        if (!rows_aligned(*r, es, v * es)) return false;
    for (const seq_ref_t *r : residuals)
        if (!rows_aligned(*r, rs, v * rs)) return false;
    for (const float *q : params)
        if (!aligned(q, 16)) return false;
    return true;
}

void fill_norm(const seq_norm_plan_s *pl, const NormShape &sh, NormParams *p) {
    p->channels = pl->channels;
    p->tpr = sh.tpr;
    p->gate_act = pl->gate_act;
    p->eps = pl->eps;
    p->inv_n = 1.f / (float)pl->channels;
    p->device = pl->base.device;
}

}  // namespace

extern "C" {

dgrad_status_t seq_norm_plan(long long rows, long long channels, seq_dtype_t dtype, seq_dtype_t residual_dtype,
                             seq_act_t gate_act, float eps, seq_norm_plan_t *plan_out) {
    if (!plan_out) return DGRAD_ERR_INVALID_ARG;
    *plan_out = nullptr;
    if (rows < 1 || channels < 1 || (int)dtype < 0 || dtype > SEQ_BF16 || (int)gate_act < 0 ||
        gate_act > SEQ_ACT_SIGMOID || !(eps >= 0.f))
        return DGRAD_ERR_INVALID_ARG;
    if (residual_dtype != dtype && residual_dtype != SEQ_F32) return DGRAD_ERR_UNSUPPORTED;
    if (channels > kNormMostChannels || rows > INT_MAX) return DGRAD_ERR_UNSUPPORTED;
    seq_norm_plan_s *pl = new (std::nothrow) seq_norm_plan_s();
    if (!pl) return DGRAD_ERR_OOM;
    const dgrad_status_t st = open_plan(&pl->base);
    if (st != DGRAD_OK) {
        delete pl;
        return st;
    }
    pl->rows = rows;
    pl->channels = (int)channels;
    pl->dtype = dtype;
    pl->rtype = residual_dtype;
    pl->gate_act = gate_act;
    pl->eps = eps;
    *plan_out = pl;
    return DGRAD_OK;
}

dgrad_status_t seq_norm_run(seq_norm_plan_t pl, const seq_norm_args_t *a, void *stream) {
    if (!pl || !a || !a->y.ptr || !a->residual.ptr || !a->residual_out.ptr || !a->x.ptr || !a->next_weight ||
        (a->gate.ptr != nullptr) != (pl->gate_act != SEQ_ACT_NONE) || a->rows < 1 || a->rows > pl->rows ||
        !strides_ok(a->y) || !strides_ok(a->gate) || !strides_ok(a->residual) || !strides_ok(a->residual_out) ||
        !strides_ok(a->x))
        return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype), rs = elem_size(pl->rtype);
    if (!all_aligned(es, {a->y.ptr, a->gate.ptr, a->x.ptr}) ||
        !all_aligned(rs, {a->residual.ptr, a->residual_out.ptr}) ||
        !all_aligned(4, {a->post_weight, a->scale, a->next_weight}))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels, n = a->rows;
    const Span outs[] = {span(a->residual_out, n, 1, 1, D, rs), span(a->x, n, 1, 1, D, es)};
    const Span ins[] = {span(a->y, n, 1, 1, D, es), span(a->gate, n, 1, 1, D, es), span(a->residual, n, 1, 1, D, rs),
                        flat(a->post_weight, D * 4), flat(a->scale, D * 4), flat(a->next_weight, D * 4)};
    if (!rows_distinct(outs[0]) || !rows_distinct(outs[1])) return DGRAD_ERR_INVALID_ARG;
    if (any_overlap(outs, 2, ins, 6)) return DGRAD_ERR_ALIAS;
    dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    const NormShape sh = norm_shape(pl->channels, kElems);
    NormParams p{};
    fill_norm(pl, sh, &p);
    p.rows = n;
    p.y = ref<void>(a->y);
    p.gate = ref<void>(a->gate);
    p.res = ref<void>(a->residual);
    p.res_out = ref<void>(a->residual_out);
    p.x = ref<void>(a->x);
    p.post = a->post_weight;
    p.scale = a->scale;
    p.next = a->next_weight;
    p.params_wide = all_aligned(16, {p.post, p.scale, p.next});
    const bool wide = norm_refs_wide(pl, {&a->y, &a->gate, &a->x}, {&a->residual, &a->residual_out},
                                     {a->post_weight, a->scale, a->next_weight});
    const int per_block = sh.tpr == 32 ? sh.block / 32 : 1;
    return dgrad::cuda_status(norm_dispatch<false>(pl->dtype, pl->rtype, wide, p,
                                                   (unsigned)((n + per_block - 1) / per_block), sh.block,
                                                   static_cast<cudaStream_t>(stream)));
}

dgrad_status_t seq_norm_backward(seq_norm_plan_t pl, const seq_norm_grad_args_t *a, void *stream) {
    const bool gated = pl && pl->gate_act != SEQ_ACT_NONE;
    if (!pl || !a || !a->y.ptr || !a->residual.ptr || !a->grad_x.ptr || !a->grad_y.ptr || !a->grad_residual.ptr ||
        !a->next_weight || !a->grad_next_weight || (a->gate.ptr != nullptr) != gated ||
        (a->grad_gate.ptr != nullptr) != gated || (!a->post_weight) != (!a->grad_post_weight) ||
        (!a->scale) != (!a->grad_scale) || a->rows < 1 || a->rows > pl->rows)
        return DGRAD_ERR_INVALID_ARG;
    for (const seq_ref_t *r : {&a->y, &a->gate, &a->residual, &a->grad_residual_out, &a->grad_x, &a->grad_y,
                               &a->grad_gate, &a->grad_residual})
        if (!strides_ok(*r)) return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype), rs = elem_size(pl->rtype);
    if (!all_aligned(es, {a->y.ptr, a->gate.ptr, a->grad_x.ptr, a->grad_y.ptr, a->grad_gate.ptr}) ||
        !all_aligned(rs, {a->residual.ptr, a->grad_residual_out.ptr, a->grad_residual.ptr}) ||
        !all_aligned(4, {a->post_weight, a->scale, a->next_weight, a->grad_post_weight, a->grad_scale,
                          a->grad_next_weight}))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels, n = a->rows;
    const Span outs[] = {span(a->grad_y, n, 1, 1, D, es), span(a->grad_gate, n, 1, 1, D, es),
                         span(a->grad_residual, n, 1, 1, D, rs), flat(a->grad_post_weight, D * 4),
                         flat(a->grad_scale, D * 4), flat(a->grad_next_weight, D * 4)};
    const Span ins[] = {span(a->y, n, 1, 1, D, es), span(a->gate, n, 1, 1, D, es), span(a->residual, n, 1, 1, D, rs),
                        span(a->grad_x, n, 1, 1, D, es), span(a->grad_residual_out, n, 1, 1, D, rs),
                        flat(a->post_weight, D * 4), flat(a->scale, D * 4), flat(a->next_weight, D * 4)};
    for (int i = 0; i < 3; ++i)
        if (!rows_distinct(outs[i])) return DGRAD_ERR_INVALID_ARG;
    if (any_overlap(outs, 6, ins, 8)) return DGRAD_ERR_ALIAS;
    dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    const bool wide = norm_refs_wide(pl, {&a->y, &a->gate, &a->grad_x, &a->grad_y, &a->grad_gate},
                                     {&a->residual, &a->grad_residual_out, &a->grad_residual},
                                     {a->post_weight, a->scale, a->next_weight});
    const NormShape sh = norm_shape(pl->channels, bwd_elems(pl->channels, wide));
    if ((st = grow(&pl->part, &pl->part_bytes, norm_bwd_need(pl))) != DGRAD_OK) return st;
    NormParams p{};
    fill_norm(pl, sh, &p);
    p.rows = n;
    p.y = ref<void>(a->y);
    p.gate = ref<void>(a->gate);
    p.res = ref<void>(a->residual);
    p.gro = ref<void>(a->grad_residual_out);
    p.gx = ref<void>(a->grad_x);
    p.gy = ref<void>(a->grad_y);
    p.ggate = ref<void>(a->grad_gate);
    p.gres = ref<void>(a->grad_residual);
    p.post = a->post_weight;
    p.scale = a->scale;
    p.next = a->next_weight;
    p.params_wide = all_aligned(16, {p.post, p.scale, p.next});
    p.part = static_cast<float *>(pl->part);
    p.n_part = 1 + (a->post_weight != nullptr) + (a->scale != nullptr);
    const int grid = norm_bwd_grid(pl, n, sh, wide);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = dgrad::cuda_status(norm_dispatch<true>(pl->dtype, pl->rtype, wide, p, (unsigned)grid, sh.block, s));
    if (st != DGRAD_OK) return st;
    float *g1 = a->grad_post_weight ? a->grad_post_weight : a->grad_scale;
    float *g2 = a->grad_scale;
    const int sums = p.n_part * (int)D;
    return dgrad::cuda_status(launch(norm_grad_sum_kernel, (sums + 31) / 32, 32 * kSumWarps, 0, s, p.part, grid, sums, (int)D,
                                     a->grad_next_weight, g1, g2));
}

size_t seq_norm_workspace_bytes(seq_norm_plan_t pl, int gradients) {
    return pl ? kErrorBytes + (gradients ? norm_bwd_need(pl) : 0) : 0;
}

void seq_norm_destroy(seq_norm_plan_t pl) {
    if (!pl) return;
    close_plan(pl->base, &pl->part, 1);
    delete pl;
}

}  // extern "C"
