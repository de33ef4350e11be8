// What the selective scan's kernels share (include/seq.h, seq_scan).
//
// Work goes in pairs of neighbouring channels, one packed instruction for
// both.  The internal buffers (checkpoints, chunk states, partial sums) are
// laid out [..][state][padded channel], each group's channels padded to a
// multiple of 4, so that channels are contiguous for the lanes of a warp.
#pragma once

#include "seq_common.cuh"

namespace seq {

constexpr int kSeg = 8;   // tokens between checkpoints, and of one pipeline step

// ex2.approx returns on average 0.3 * 2^-24 too little for arguments between
// -0.5 and -0.001 (measured over 2^20 of them; 0.1 * 2^-24 closer to 0).  A
// state remembers 1 / (1 - a) tokens and would gather that error from all of
// them, so two thirds of it are put back, in the multiply-add that forms the
// exponent.  What is left differs from bin to bin (-0.24 between -0.03 and -0.01,
// else within 0.15 down to -0.5), as it does for expf (-0.19 to 0.40).  The
// rounding of A log2 e and of the exponent adds |t| 2^-24 log 2 to a decay 2^t,
// at most 0.37 * 2^-24 of the state that decays; an fp32 product delta A alone
// does the same (rms of both over the decays from 2^-1 on: 0.5 to 0.8).
constexpr float kEx2Bias = 0.2f * 5.9604645e-8f * 1.442695f;

struct ScanParams {
    long long batch, length;
    int channels, states, groups;
    int group_channels;          // channels / groups
    int group_pad, pad;          // ... rounded up to a multiple of 4; groups * that
    int tiles_per_group;         // column tiles of one group
    int chunk, n_chunks;         // tokens per chunk (a multiple of kSeg), chunks per row
    int per, n_main;             // chunks that a block of the backward main kernel walks through, blocks per row
    int device;
    int quads;                   // ceil(states / 4) rounded up to a power of two
    Ref<void> u, dt, B, C, z, out;
    Ref<void> gout, gu, gdt, gB, gC, gz;
    const float *A, *D, *dt_bias;
    const int *lengths;
    const float *state, *gfinal;
    float *final_state, *gstate;
    float *grad_A, *grad_D, *grad_bias;
    float *ck;                   // [batch][segments][states][pad]: states before every kSeg-th token
    float *chunk_state;          // [batch][n_chunks][states][pad]: what a chunk alone leaves, then what it is handed
    float *chunk_sum;            // [batch][n_chunks][pad]: its sum of delta
    float *part_A;               // [batch * n_main][states][pad]
    float *part_D, *part_bias;   // [batch * n_main][pad]
    float *part_BC;              // [tiles_per_group][batch][length][groups][2][4 * quads]
};

struct ScanStepParams {
    long long batch, n_slots;
    int channels, states, group_channels;
    int sm_count;
    bool wide_cache, wide_bc;    // a thread's states of the cache, and of B and C, come in wide accesses
    Ref<void> u, dt, B, C, z, out;
    const float *A, *D, *dt_bias;
    float *cache;
    const int *slots, *write_slots;
    uint32_t *err;
};

int scan_fwd_columns(int quads);
int scan_bwd_columns(int quads);
int scan_fwd_resident(int quads, bool wide);
int scan_bwd_resident(int quads, seq_dtype_t dtype, bool wide);
cudaError_t launch_scan_fwd(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s);
cudaError_t launch_scan_rev(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s);
cudaError_t launch_scan_bwd(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s);
cudaError_t launch_scan_step(seq_dtype_t dtype, const ScanStepParams &p, int quads, cudaStream_t s);

// Token distances fit 28 bits (checked by the entry points): within a step or
// segment they are multiplied in 32 bits.
template <typename T>
__device__ __forceinline__ T *scan_row(const Ref<void> &r, long long b, long long t) {
    return static_cast<T *>(r.p) + b * r.sb + t * r.st;
}
__device__ __forceinline__ int token_step(const Ref<void> &r) { return static_cast<int>(r.st); }

__device__ __forceinline__ int scan_length(const ScanParams &p, long long b) {
    if (!p.lengths) return static_cast<int>(p.length);
    const int n = p.lengths[b];
    return n < 0 ? 0 : (n > p.length ? static_cast<int>(p.length) : n);
}

// NT consecutive states of a [channels, states] row (0 past the end).
template <int NT>
__device__ __forceinline__ void load_states(const float *m, long long row, int states, int n0, float (&f)[NT]) {
    const float *r = m + row * states + n0;
    if ((states & 3) == 0 && n0 + NT <= states && aligned16(r)) {
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(r + i);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) f[i] = n0 + i < states ? r[i] : 0.f;
    }
}

template <int NT>
__device__ __forceinline__ void store_states(float *m, long long row, int states, int n0, const float (&f)[NT]) {
    float *r = m + row * states + n0;
    if ((states & 3) == 0 && n0 + NT <= states && aligned16(r)) {
#pragma unroll
        for (int i = 0; i < NT; i += 4)
            *reinterpret_cast<float4 *>(r + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            if (n0 + i < states) r[i] = f[i];
    }
}

}  // namespace seq
