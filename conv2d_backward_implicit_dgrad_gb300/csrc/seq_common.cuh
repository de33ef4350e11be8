// Shared pieces of the sequence operators (include/seq.h): element types,
// packed fp32 arithmetic, the activations, and the host side's checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <numeric>
#include <type_traits>

#include "dgrad_internal.h"
#include "seq.h"

namespace seq {

using bf16 = __nv_bfloat16;
using f16 = __half;

// ------------------------------------------------------------ element types
// V neighbouring elements, moved as one load or store of 2, 4, 8 or 16 bytes.
// They stay in the words that were loaded until a value is asked for: taking
// the 16-bit halves apart next to the load would make it wait for its data.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    using W = std::conditional_t<sizeof(T) * V == 2, uint16_t, uint32_t>;
    static constexpr int N = sizeof(T) * V / sizeof(W);
    W w[N];

    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (std::is_same_v<T, float>) {
            return __uint_as_float(w[i]);
        } else {
            uint32_t bits;   // in the upper half
            if constexpr (V == 1) bits = static_cast<uint32_t>(w[0]) << 16;
            else bits = (i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16);
            if constexpr (std::is_same_v<T, bf16>) return __uint_as_float(bits);
            else return __half2float(__ushort_as_half(static_cast<unsigned short>(bits >> 16)));
        }
    }

    static __device__ __forceinline__ Vec zero() {
        Vec v;
#pragma unroll
        for (int i = 0; i < N; ++i) v.w[i] = 0;
        return v;
    }

    // Each value rounded to the nearest element.
    static __device__ __forceinline__ Vec from(const float (&f)[V]) {
        Vec v;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (std::is_same_v<T, float>) {
                v.w[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same_v<T, bf16>) {
                if constexpr (V == 1) {
                    v.w[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    v.w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            } else {
                if constexpr (V == 1) {
                    v.w[i] = __half_as_ushort(__float2half_rn(f[i]));
                } else {
                    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                    v.w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
        }
        return v;
    }
};

// Element i of a row; its value; a value stored there.
template <typename T>
__device__ __forceinline__ Vec<T, 1> elem(const T *row, long long i) {
    return *reinterpret_cast<const Vec<T, 1> *>(row + i);
}
// The same (0 where not on), issued here: the compiler would move a plain load
// of an element that is used much later down to its use, to wait for it there.
template <typename T>
__device__ __forceinline__ Vec<T, 1> elem_ahead(const T *at, bool on) {
    Vec<T, 1> v;
    if constexpr (sizeof(T) == 2) {
        asm volatile(
            "{\n .reg .pred q;\n setp.ne.s32 q, %2, 0;\n mov.b16 %0, 0;\n @q ld.global.nc.b16 %0, [%1];\n}"
            : "=h"(v.w[0])
            : "l"(at), "r"((int)on));
    } else {
        asm volatile(
            "{\n .reg .pred q;\n setp.ne.s32 q, %2, 0;\n mov.b32 %0, 0;\n @q ld.global.nc.b32 %0, [%1];\n}"
            : "=r"(v.w[0])
            : "l"(at), "r"((int)on));
    }
    return v;
}
template <typename T>
__device__ __forceinline__ float value(const T *row, long long i) {
    return elem<T>(row, i)[0];
}
template <typename T>
__device__ __forceinline__ void put(T *row, long long i, float v) {
    const float f[1] = {v};
    *reinterpret_cast<Vec<T, 1> *>(row + i) = Vec<T, 1>::from(f);
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ------------------------------------------------------------ packed fp32
// Two fp32 values in one 64-bit register pair: one instruction issued for two
// multiply-adds, each rounded as the scalar one.
using f2 = unsigned long long;

__device__ __forceinline__ f2 pack2(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ------------------------------------------------------------ functions
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = 1.925963033500935e-8f;   // log2 e - kLog2e
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    float x, y;
    unpack2(v, x, y);
    return pack2(ex2(x), ex2(y));
}

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 splat(float x) { return pack2(x, x); }

// Sigmoid and softplus take the type of the plan's activations.  A 16-bit
// result is rounded to 2^-9 (2^-12) of itself, and an exponential as 2^(x log2 e)
// with the product rounded once, |x| 2^-24 off, is far below that.  In fp32 it
// would be the largest error of all, so there exp_minus_2 puts the product's rest
// back.  Measured over 2^20 points a range, in 2^-24 of the result: sigmoid on
// [-30, -16], [-16, -7], [-7, -2], [-2, 0] 4.4, 4.0, 3.8, 3.3 at most, rms below 1
// (with the rounded product 29.9, 15.9, 8.6, 3.6 at most, rms 11.5, 5.7, 2.3, 0.9),
// between 0 and 20 at most 2.9 either way.  It costs 1 to 2 % of a convolution's,
// norm's or step's time and 4 to 7 % of a scan's (CUDA's expf and a rounded
// reciprocal, at most 3.5 off: up to 35 and 19 %).

// exp(-x): with t the rounded x log2 e and r what that rounding left out (log2 e
// in two parts), 2^-t (1 + r log 2).  Where 2^-t is 0 or infinite it stays so.
__device__ __forceinline__ f2 exp_minus_2(f2 x) {
    const f2 t = mul2(x, splat(kLog2e));
    const f2 r = fma2(x, splat(-kLog2eRest), fma2(x, splat(-kLog2e), t));
    float t0, t1, e[2], c[2];
    unpack2(t, t0, t1);
    e[0] = ex2(-t0);
    e[1] = ex2(-t1);
    const f2 raw = pack2(e[0], e[1]);
    unpack2(fma2(raw, mul2(r, splat(kLn2)), raw), c[0], c[1]);
    return pack2(fabsf(t0) < 126.f ? c[0] : e[0], fabsf(t1) < 126.f ? c[1] : e[1]);
}

// 1 / (1 + exp(-x)); where exp(-x) passes the largest float the result is 0.
template <typename T>
__device__ __forceinline__ f2 sigmoid_2(f2 x) {
    float a, b;
    const f2 e = std::is_same_v<T, float> ? exp_minus_2(x) : ex2_2(mul2(x, splat(-kLog2e)));
    unpack2(add2(e, splat(1.f)), a, b);
    return pack2(rcp(a), rcp(b));
}
template <typename T>
__device__ __forceinline__ float sigmoid_f(float x) {
    if constexpr (std::is_same_v<T, float>) {
        float a, b;
        unpack2(sigmoid_2<T>(splat(x)), a, b);
        return a;
    } else {
        return rcp(1.f + ex2(x * -kLog2e));
    }
}

// Sigmoid s and 1 - s, for the derivatives.  In fp32, 1 - s is exp(-x) s where
// x > 0: the difference would be off by 2^-24 of 1, and SiLU' by x times that.
template <typename T>
__device__ __forceinline__ void sigmoid_and_rest_2(f2 x, f2 &s, f2 &rest) {
    if constexpr (std::is_same_v<T, float>) {
        float a, b, x0, x1, r[2], q[2];
        const f2 e = exp_minus_2(x);
        unpack2(add2(e, splat(1.f)), a, b);
        s = pack2(rcp(a), rcp(b));
        unpack2(fma2(s, splat(-1.f), splat(1.f)), r[0], r[1]);
        unpack2(mul2(e, s), q[0], q[1]);
        unpack2(x, x0, x1);
        rest = pack2(x0 > 0.f ? q[0] : r[0], x1 > 0.f ? q[1] : r[1]);
    } else {
        s = sigmoid_2<T>(x);
        rest = fma2(s, splat(-1.f), splat(1.f));
    }
}

// softplus(x) = max(x, 0) + log(1 + e) with e = exp(-|x|) in (0, 1] (an fp32
// logarithm of 1 + e would lose the small e).  16-bit plans: log(1 + e) = e P(e),
// P fitted to log(1 + e) / e on [0, 1] (Chebyshev points, least squares reweighted
// towards equal relative errors): 3.0e-8 off at most before rounding.  fp32:
// log(1 + e) = e - e^2 Q(e), Q fitted the same way, 5.1e-9 off at most, so that
// what is rounded last is small beside e (the whole function within 5 * 2^-24 of
// itself on [-30, 20]; in 16-bit plans |x| 2^-24 more).  The polynomials take a
// float or a packed pair.
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
template <typename V, int N>
__device__ __forceinline__ V horner(const float (&c)[N], V x) {
    auto as = [](float v) {
        if constexpr (std::is_same_v<V, f2>) return splat(v);
        else return v;
    };
    V p = as(c[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) p = fma2(p, x, as(c[i]));
    return p;
}
template <typename V>
__device__ __forceinline__ V softplus_p(V e) {
    const float c[] = {0.005232687573879957f, -0.02950521931052208f, 0.07822593301534653f,
                       -0.13663245737552643f, 0.19106006622314453f,  -0.2484298199415207f,
                       0.3331909775733948f,   -0.4999949336051941f,  0.9999999403953552f};
    return horner(c, e);
}
template <typename V>
__device__ __forceinline__ V softplus_q(V e) {
    const float c[] = {0.003318469738587737f, -0.02020457200706005f, 0.0576644204556942f,
                       -0.10680553317070007f, 0.15355394780635834f,  -0.19695399701595306f,
                       0.24958586692810059f,  -0.33330512046813965f, 0.4999993145465851f};
    return horner(c, e);
}

template <typename T>
__device__ __forceinline__ f2 softplus_2(f2 x) {
    float a, b;
    unpack2(x, a, b);
    const f2 linear = pack2(fmaxf(a, 0.f), fmaxf(b, 0.f)), size = pack2(fabsf(a), fabsf(b));
    if constexpr (std::is_same_v<T, float>) {
        const f2 e = exp_minus_2(size);
        return add2(fma2(mul2(e, mul2(e, splat(-1.f))), softplus_q(e), e), linear);
    } else {
        const f2 e = ex2_2(mul2(size, splat(-kLog2e)));
        return fma2(softplus_p(e), e, linear);
    }
}
template <typename T>
__device__ __forceinline__ float softplus_f(float x) {
    if constexpr (std::is_same_v<T, float>) {
        float a, b;
        unpack2(softplus_2<T>(splat(x)), a, b);
        return a;
    } else {
        const float e = ex2(fabsf(x) * -kLog2e);
        return fmaf(softplus_p(e), e, fmaxf(x, 0.f));
    }
}

// Two neighbouring elements: PAIR, as one access, else as one each (some of
// the rows start on an odd element).
template <typename T, bool PAIR>
struct Two {
    Vec<T, 2> v;
    static __device__ __forceinline__ Two load(const T *row, unsigned d, bool on0, bool) {
        return Two{on0 ? *reinterpret_cast<const Vec<T, 2> *>(row + d) : Vec<T, 2>::zero()};
    }
    static __device__ __forceinline__ void store(T *row, unsigned d, bool on0, bool, f2 x) {
        float f[2];
        unpack2(x, f[0], f[1]);
        if (on0) *reinterpret_cast<Vec<T, 2> *>(row + d) = Vec<T, 2>::from(f);
    }
    __device__ __forceinline__ f2 get() const {
        if constexpr (std::is_same_v<T, f16>) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
            return pack2(f.x, f.y);
        } else {
            return pack2(v[0], v[1]);
        }
    }
};
template <typename T>
struct Two<T, false> {
    Vec<T, 1> a, b;
    static __device__ __forceinline__ Two load(const T *row, unsigned d, bool on0, bool on1) {
        return Two{on0 ? elem<T>(row, d) : Vec<T, 1>::zero(), on1 ? elem<T>(row, d + 1) : Vec<T, 1>::zero()};
    }
    static __device__ __forceinline__ void store(T *row, unsigned d, bool on0, bool on1, f2 x) {
        float f[2];
        unpack2(x, f[0], f[1]);
        if (on0) put<T>(row, d, f[0]);
        if (on1) put<T>(row, d + 1, f[1]);
    }
    __device__ __forceinline__ f2 get() const { return pack2(a[0], b[0]); }
};

// Every kernel's first step: until the kernels before it in the stream are
// through, it touches no memory (its launch overlaps their end).  None lets
// the next one start before its own blocks end: that one's blocks would wait
// packed onto the SMs that are free first, and grids of less than a wave would
// run there, the other SMs idle (76 -> 85 us for a training step of 2 x 777
// tokens and 515 channels).
__device__ __forceinline__ void begin_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------ reductions
// Sums over LANES lanes (their bits in the lane number start at STRIDE) of V
// values each, halving the values with the lanes as long as there are some: a
// lane then holds the sums of V / LANES values (from index (lane's group
// number) * V / LANES), or of one value in LANES / V copies (index = group
// number / (LANES / V)).  V = LANES costs LANES - 1 shuffles, not V * log2.
template <int V, int LANES, int STRIDE>
__device__ __forceinline__ void reduce_lanes(float *v, int lane) {
    if constexpr (LANES > 1) {
        constexpr int bit = STRIDE * (LANES / 2);
        if constexpr (V > 1) {
            const bool up = (lane & bit) != 0;
            constexpr int half = V / 2;
#pragma unroll
            for (int k = 0; k < half; ++k) {
                const float send = up ? v[k] : v[k + half];
                const float keep = up ? v[k + half] : v[k];
                v[k] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
            }
            reduce_lanes<half, LANES / 2, STRIDE>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
            reduce_lanes<1, LANES / 2, STRIDE>(v, lane);
        }
    }
}

// ------------------------------------------------------------ strided tensors
template <typename T>
struct Ref {
    T *p;
    long long sb, st, sg;
    __device__ __forceinline__ T *row(long long b, long long t) const { return p + b * sb + t * st; }
};

template <typename T>
Ref<T> ref(const seq_ref_t &r) {
    return Ref<T>{static_cast<T *>(r.ptr), r.sb, r.st, r.sg};
}

// ------------------------------------------------------------ host side
struct PlanBase {
    int device, sm_count;
    uint32_t *err;   // device word: 1 after a slot out of range
};
constexpr size_t kErrorBytes = 256;   // that err points to

inline size_t elem_size(seq_dtype_t d) { return d == SEQ_F32 ? 4 : 2; }

// The bytes that a [nb, nt, ng, width] tensor spans.
struct Span {
    const char *lo, *hi;
    long long sb, st, sg;   // bytes
    long long nb, nt, ng, row;
};

inline Span span(const seq_ref_t &r, long long nb, long long nt, long long ng, long long width, size_t es) {
    const long long e = (long long)es;
    Span s{static_cast<const char *>(r.ptr), nullptr, r.sb * e, r.st * e, r.sg * e, nb, nt, ng, width * e};
    s.hi = s.lo;
    if (r.ptr && nb > 0 && nt > 0 && ng > 0 && width > 0)
        s.hi = s.lo + (nb - 1) * s.sb + (nt - 1) * s.st + (ng - 1) * s.sg + s.row;
    return s;
}
inline Span flat(const void *p, size_t bytes) {
    return Span{static_cast<const char *>(p), static_cast<const char *>(p) + (p ? bytes : 0), 0, 0, 0, 1, 1, 1,
                (long long)bytes};
}

// Whether two tensors may share a byte.  Rows of one buffer side by side (equal
// distances, columns apart) do not, although their spans do: all of a tensor's
// rows start a multiple of `pitch` from its first, and columns that keep apart
// within one pitch keep apart in all.
inline bool overlaps(const Span &a, const Span &b) {
    if (!a.lo || !b.lo || a.lo >= a.hi || b.lo >= b.hi || a.hi <= b.lo || b.hi <= a.lo) return false;
    if (a.nb == b.nb && a.nt == b.nt && (a.nb == 1 || a.sb == b.sb) && (a.nt == 1 || a.st == b.st)) {
        const long long wa = a.row + (a.ng - 1) * a.sg, wb = b.row + (b.ng - 1) * b.sg;
        const long long pitch = std::gcd(a.nb > 1 ? a.sb : 0, a.nt > 1 ? a.st : 0);
        if (pitch > 0) {
            long long d = (b.lo - a.lo) % pitch;
            if (d < 0) d += pitch;
            // b's columns start d into a's pitch; neither may wrap around into the other
            if (d >= wa && d + wb <= pitch) return false;
        }
    }
    return true;
}

// An output's rows must not lie on one another (a broadcast output).
inline bool rows_distinct(const Span &s) {
    if (!s.lo) return true;
    const long long w = s.row;
    if (s.ng > 1 && s.sg < w) return false;
    const long long wt = (s.ng - 1) * s.sg + w;
    if (s.nt > 1 && s.st < wt) return false;
    const long long wb = (s.nt - 1) * s.st + wt;
    // rows of the batch lie apart, or interleave below the token distance
    if (s.nb > 1 && s.sb < wb && !(s.sb >= wt && s.nt > 1 && (s.nb - 1) * s.sb + wt <= s.st)) return false;
    return true;
}

inline bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Whether one of the outputs overlaps an input or another output.
inline bool any_overlap(const Span *outs, int n_out, const Span *ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(outs[i], ins[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

inline bool all_aligned(size_t to, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (!aligned(p, to)) return false;
    return true;
}

// Whether every row of a tensor starts on a multiple of `bytes`.
inline bool rows_aligned(const seq_ref_t &r, size_t es, size_t bytes) {
    if (!r.ptr) return true;
    const long long e = (long long)es, a = (long long)bytes;
    return aligned(r.ptr, bytes) && (r.sb * e) % a == 0 && (r.st * e) % a == 0;
}

// Distances are not negative, and those of tokens and groups fit 28 bits.
inline bool strides_ok(const seq_ref_t &r) {
    constexpr long long most = 1LL << 28;
    return r.sb >= 0 && r.st >= 0 && r.sg >= 0 && r.st < most && r.sg < most;
}

// Launches a kernel that starts with begin_kernel().
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Lets a kernel use `smem` bytes of dynamic shared memory, once on each device.
struct SmemLimit {
    std::atomic<uint64_t> set{0};
    template <typename K>
    cudaError_t raise(K *kernel, int smem, int device) {
        const uint64_t bit = uint64_t(1) << (device & 63);
        if (device < 64 && (set.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && device < 64) set.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

dgrad_status_t open_plan(PlanBase *base);
dgrad_status_t on_device(const PlanBase &base);
dgrad_status_t grow(void **mem, size_t *have, size_t want);
dgrad_status_t read_error(const PlanBase &base);
void close_plan(const PlanBase &base, void *const *mems, int n);

}  // namespace seq
