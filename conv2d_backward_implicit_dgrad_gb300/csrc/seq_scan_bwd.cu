// The selective scan's gradients (include/seq.h, seq_scan_backward).
//
// With a_t = exp(delta_t A) and dy_t = grad_out_t SiLU(z_t), the gradient of
// the state runs backwards in time, g_t = dy_t C_t + a_(t+1) g_(t+1), and
//   sB = sum over n of g B, sA = sum over n of g a h_(t-1) A, sY = sum over n of C h_t
//   grad_u = sB delta + D dy,  grad_delta = sB u + sA,  grad_dt = grad_delta sigmoid(dt + dt_bias)
//   grad_z = grad_out SiLU'(z) (sY + D u)
//   grad_B = sum over the group's channels of g delta u,  grad_C = the same of dy h_t
//   grad_A = sum over t of g a h_(t-1) delta,  grad_D = of dy u,  grad_dt_bias = of grad_dt
// The states are needed last to first.  The forward call left them before
// every kSeg-th token; a warp runs forwards from there over kSeg tokens,
// keeping every second state in shared memory, and then backwards over them
// two tokens at a time, forming the state in between again (its exp is needed
// there anyway).  Undoing the recurrence instead would divide by a_t, which
// may be 0.
//
// Three sums run over states and two over channels.  A lane owns a square of
// 4 states x 4 channels: LN lanes side by side share 4 channels, and each of
// the 32 / LN rows of lanes has 4 channels of its own.  Either sum is then
// mostly in the lane, and the lanes' parts are added by halving (16 shuffles a
// token for 512 states at 16 states a channel; one channel per lane would take
// 31 for the sums over channels alone).  Arithmetic is packed for pairs of
// channels.  Sums over more than a block leave as partial rows, added in a
// fixed order by scan_grad_sum_kernel.
//
// Time is cut into chunks as forwards; scan_state_kernel and scan_join_kernel
// (REV) have left the gradient that each chunk is handed from behind.
//
// What bounds it: per state, token and pair of channels 11 packed operations
// and an ex2 each going backwards, 3 and an ex2 each in the walk before; a token
// of 32 channels of 16 states is 400 instructions of a warp, issued in 57 % of
// the cycles by three blocks (12 warps) an SM, which wait for results of the
// instructions before and of shared memory.  4 x 2048 tokens x 4096 channels
// in bf16: 600 us, its 14 bytes a token and channel alone 69 us.  Three blocks,
// elements copied ahead per warp and results stored in 16-byte pieces brought
// it from 684 us to 609, the walk unrolled by four to 600.
#include "seq_scan.cuh"

namespace seq {
namespace {

constexpr int bwd_warps(int ln) { return ln <= 2 ? 2 : 4; }

// A segment of a warp's CW channels in pieces of 16 bytes (8 where it has no more).
template <typename T, int CW>
struct BwdPieces {
    static constexpr int PIECE = (CW * (int)sizeof(T) < 16 ? CW : 16 / (int)sizeof(T));   // elements of one access
    static constexpr int PIECES = kSeg * CW / PIECE;   // of a warp, segment and tensor
    static constexpr int COPIES = (PIECES + 31) / 32;  // of a lane
};

// WIDE: rows lie in 16-byte pieces.
template <typename T, int LN, bool WIDE>
struct BwdShape {
    static constexpr int LD = 32 / LN;          // rows of lanes
    static constexpr int CW = 4 * LD;           // channels of a warp
    static constexpr int WARPS = bwd_warps(LN);
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int CPB = CW * WARPS;
    static constexpr int NP = 4 * LN;
    static constexpr int OWN = LN <= 4 ? 4 / LN : 1;   // channels a lane finishes
    static constexpr int BIASES = CW > 64 ? CW / 64 : 1;  // channel pairs that a lane prepares
    static constexpr int ITEMS = CW >= 8 ? CW / 8 : 1; // (token, channel pair)s a lane prepares of a segment
    static constexpr int BCS = (kSeg * 2 * NP + THREADS - 1) / THREADS;   // elements of B and C a thread loads
    // shared memory, in floats
    static constexpr int STATE = 32 * 16;              // a warp's states
    static constexpr int HIST = (kSeg / 2 + 1) * STATE;   // per warp: before tokens 2, 4, 6, and two checkpoints
    static constexpr int FIELD = kSeg * CW;            // per warp and field: delta, u, dy, sigmoid, grad_out SiLU'
    static constexpr int BC = kSeg * 2 * NP * 2;       // B and C, each value twice
    static constexpr int PART = WARPS * kSeg * 2 * NP;
    static constexpr int RAW = WIDE ? 4 * kSeg * CW * (int)sizeof(T) / 4 : 0;   // per warp: u, dt, grad_out, z as they come
    static constexpr int TOTAL = WARPS * (HIST + 5 * FIELD + RAW) + BC + PART;
    // An SM's blocks: by shared memory, and by registers, of which a thread
    // takes up to 255 (three blocks of 168 where that needs next to no spills:
    // at 16 states three blocks of 74 KB walk faster than two with more registers).
    static constexpr int BY_SMEM = 228 * 1024 / (TOTAL * 4 + 1024);
    static constexpr int BY_REGS = LN >= 4 && LN <= 16 && WIDE && sizeof(T) == 2 ? 3 : 256 / THREADS;
    static constexpr int BLOCKS = BY_SMEM < BY_REGS ? BY_SMEM : BY_REGS;
};

// The lane's 4 channels of one row of an internal [..][pad] buffer.
__device__ __forceinline__ ulonglong2 load_four(const float *row, int ch) {
    return *reinterpret_cast<const ulonglong2 *>(row + ch);
}

// 16 or 8 bytes to shared memory, or zeros.
template <int BYTES>
__device__ __forceinline__ void copy_ahead(void *to, const void *from, bool on) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(on ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at), "l"(from), "r"(on ? 8 : 0) : "memory");
}

template <typename T, int LN, bool WIDE>
__global__ void __launch_bounds__(BwdShape<T, LN, WIDE>::THREADS, BwdShape<T, LN, WIDE>::BLOCKS)
    scan_bwd_kernel(const __grid_constant__ ScanParams p) {
    begin_kernel();
    using S = BwdShape<T, LN, WIDE>;
    using Q = BwdPieces<T, S::CW>;
    constexpr int NP = S::NP, CW = S::CW, OWN = S::OWN, LD = S::LD;
    extern __shared__ __align__(16) float sm[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int nl = lane % LN, dl = lane / LN;
    ulonglong2 *const hist = reinterpret_cast<ulonglong2 *>(sm + warp * S::HIST);   // [.][4 states][32 lanes]
    ulonglong2 *const marks = hist + (kSeg / 2 - 1) * 128;                          // the two checkpoints
    float *const fields = sm + S::WARPS * S::HIST + warp * 5 * S::FIELD;
    float *const f_delta = fields, *const f_u = fields + S::FIELD, *const f_dy = fields + 2 * S::FIELD;
    float *const f_sig = fields + 3 * S::FIELD, *const f_dz = fields + 4 * S::FIELD;
    float *const bc = sm + S::WARPS * (S::HIST + 5 * S::FIELD);
    float *const part = bc + S::BC;
    T *const raw = reinterpret_cast<T *>(part + S::PART + warp * S::RAW);   // [4 tensors][token][channel]

    const int tiles = p.groups * p.tiles_per_group;
    const int tile = blockIdx.x % tiles;
    const long long rest = blockIdx.x / tiles;
    const int main_i = static_cast<int>(rest % p.n_main);
    const long long b = rest / p.n_main;
    const int group = tile / p.tiles_per_group, gt = tile % p.tiles_per_group;
    const int in_group = gt * S::CPB + warp * CW;            // the warp's first channel within the group,
    const int dbase = group * p.group_channels + in_group;   // overall,
    const int pbase = group * p.group_pad + in_group;        // and in the internal buffers
    const int left = p.group_channels - in_group;            // channels from there to the group's end
    const int len = scan_length(p, b);
    const int span = p.per * p.chunk;
    const int c0 = main_i * span, c1 = min(static_cast<int>(p.length), c0 + span);
    const int t1 = min(len, c1);
    const long long outer = b * p.n_main + main_i;
    const int ch0 = 4 * dl;   // the lane's channels dbase + ch0 + 0..3 in two pairs, states 4 nl + 0..3

    f2 A2[2][4], g[2][4], dA[2][4], h[2][4];
    {
        float a[4][4], gf[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int n = 0; n < 4; ++n) a[i][n] = gf[i][n] = 0.f;
            if (ch0 + i < left) {
                load_states<4>(p.A, dbase + ch0 + i, p.states, 4 * nl, a[i]);
                if (p.gfinal) load_states<4>(p.gfinal, b * p.channels + dbase + ch0 + i, p.states, 4 * nl, gf[i]);
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                A2[c][n] = pack2(a[2 * c][n] * kLog2e, a[2 * c + 1][n] * kLog2e);
                g[c][n] = pack2(gf[2 * c][n], gf[2 * c + 1][n]);
                dA[c][n] = 0;
            }
    }
    if (p.n_main > 1 && t1 > c0 && ch0 < left) {
        // the gradient handed back by the chunks behind this block's last one with tokens
        const int k = min((main_i + 1) * p.per, (len + p.chunk - 1) / p.chunk) - 1;
        const float *const row = p.chunk_state + ((b * p.n_chunks + k) * p.states + 4 * nl) * p.pad + pbase;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (4 * nl + n >= p.states) continue;
            const ulonglong2 e = load_four(row + (long long)n * p.pad, ch0);
            g[0][n] = e.x;
            g[1][n] = e.y;
        }
    }
    // the channels that the lane finishes, and whether it is the one to write them
    const int own0 = ch0 + (LN >= 4 ? nl / (LN >= 4 ? LN / 4 : 1) : nl * OWN);
    const bool writer = LN <= 4 || nl % (LN >= 4 ? LN / 4 : 1) == 0;
    float skip[OWN], gD[OWN], gbias[OWN];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        skip[k] = p.D && own0 + k < left ? p.D[dbase + own0 + k] : 0.f;
        gD[k] = gbias[k] = 0.f;
    }
    // behind the row's last token everything is 0
    for (int t = max(t1, c0); t < c1; ++t) {
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            if (!writer || own0 + k >= left) continue;
            const int d = dbase + own0 + k;
            put<T>(scan_row<T>(p.gu, b, t), d, 0.f);
            put<T>(scan_row<T>(p.gdt, b, t), d, 0.f);
            if (p.gz.p) put<T>(scan_row<T>(p.gz, b, t), d, 0.f);
        }
    }
    f2 bias[S::BIASES];
#pragma unroll
    for (int k = 0; k < S::BIASES; ++k) {
        const int ch = 2 * ((lane + 32 * k) % (CW / 2));
        bias[k] = p.dt_bias ? pack2(ch < left ? p.dt_bias[dbase + ch] : 0.f, ch + 1 < left ? p.dt_bias[dbase + ch + 1] : 0.f) : 0;
    }
    const int segments = static_cast<int>((p.length + kSeg - 1) / kSeg);
    const int segs = t1 > c0 ? (t1 - c0 + kSeg - 1) / kSeg : 0;

    const Ref<void> *const in[4] = {&p.u, &p.dt, &p.gout, &p.z};
    Two<T, false> held[WIDE ? 1 : 4 * S::ITEMS];
    Vec<T, 1> held_bc[S::BCS];
    // Loads the warp's elements and checkpoint and the thread's share of B and
    // C of a segment, one segment ahead (0 for what lies outside).
    auto load_ahead = [&](int at) {
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < Q::COPIES; ++k) {
                const int e = lane + 32 * k;
                const int j = e / (CW / Q::PIECE), c = e % (CW / Q::PIECE) * Q::PIECE;
                if (Q::PIECES % 32 != 0 && j >= kSeg) continue;
                const bool on = at + j < t1 && c < left;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const T *const from = scan_row<T>(*in[i], b, at) + (dbase + j * token_step(*in[i]) + c);
                    const bool there = on && (i < 3 || p.z.p);
                    copy_ahead<Q::PIECE * sizeof(T)>(raw + (i * kSeg + j) * CW + c, there ? from : static_cast<const T *>(p.u.p), there);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < S::ITEMS; ++k) {
                const int e = lane + 32 * k, j = e / (CW / 2), ch = 2 * (e % (CW / 2));
                const bool on = j < kSeg && at + j < t1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const T *const from = scan_row<T>(*in[i], b, at) + (dbase + j * token_step(*in[i]) + ch);
                    const bool there = on && (i < 3 || p.z.p);
                    held[4 * k + i].a = elem_ahead<T>(from, there && ch < left);
                    held[4 * k + i].b = elem_ahead<T>(from + 1, there && ch + 1 < left);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < S::BCS; ++k) {
            const int i = threadIdx.x + k * S::THREADS;
            const int j = i / (2 * NP), n = i % NP;
            const Ref<void> &r = i % (2 * NP) >= NP ? p.C : p.B;
            held_bc[k] = elem_ahead<T>(scan_row<T>(r, b, at) + (j * token_step(r) + group * r.sg + n),
                                       i < kSeg * 2 * NP && at + j < t1 && n < p.states);
        }
        ulonglong2 *const to = marks + (at / kSeg & 1) * 128 + lane;
        const float *const from = p.ck + ((b * segments + at / kSeg) * p.states + 4 * nl) * p.pad + pbase + ch0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool on = 4 * nl + n < p.states && ch0 < left;
            copy_ahead<16>(to + n * 32, on ? from + (long long)n * p.pad : p.ck, on);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Adds up the warps' shares of grad_B and grad_C of a segment.
    auto add_part = [&](int at) {
        const int n = min(kSeg, t1 - at);
        for (int i = threadIdx.x; i < n * 2 * NP; i += S::THREADS) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < S::WARPS; ++w) s += part[w * kSeg * 2 * NP + i];
            const int j = i / (2 * NP);
            p.part_BC[((((long long)gt * p.batch + b) * p.length + at + j) * p.groups + group) * 2 * NP + i % (2 * NP)] = s;
        }
    };
    if (segs > 0) load_ahead(c0 + (segs - 1) * kSeg);
    for (int sgm = segs - 1; sgm >= 0; --sgm) {
        const int at = c0 + sgm * kSeg;
        // the warp's channels: what the loops below need of u, dt, z, grad_out
        // (behind the last token all of it 0: the state and its gradient then
        // pass through and nothing is added)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int k = 0; k < S::ITEMS; ++k) {
            const int e = lane + 32 * k, j = e / (CW / 2), ch = 2 * (e % (CW / 2));
            if (j >= kSeg) continue;
            f2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (WIDE)
                    v[i] = Two<T, true>{*reinterpret_cast<const Vec<T, 2> *>(raw + (i * kSeg + j) * CW + ch)}.get();
                else
                    v[i] = held[4 * k + i].get();
            }
            const f2 x = add2(v[1], bias[k % S::BIASES]);
            f2 dy = v[2], dz = 0;
            if (p.z.p) {
                f2 sz, rest;
                sigmoid_and_rest_2<T>(v[3], sz, rest);
                const f2 zs = mul2(v[3], sz);
                // SiLU'(z) = s + z s (1 - s)
                dz = mul2(dy, fma2(zs, rest, sz));
                dy = mul2(dy, zs);
            }
            const int i = j * CW + ch;
            *reinterpret_cast<f2 *>(f_delta + i) = at + j < t1 ? softplus_2<T>(x) : 0;
            *reinterpret_cast<f2 *>(f_sig + i) = sigmoid_2<T>(x);
            *reinterpret_cast<f2 *>(f_u + i) = v[0];
            *reinterpret_cast<f2 *>(f_dy + i) = dy;
            *reinterpret_cast<f2 *>(f_dz + i) = dz;
        }
        // the checkpoint is the lane's own copy; its next one goes to the other place
        const ulonglong2 *const mark = marks + (at / kSeg & 1) * 128 + lane;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const ulonglong2 e = mark[n * 32];
            h[0][n] = e.x;
            h[1][n] = e.y;
        }
        __syncthreads();   // every warp is through with the segment before
        if (sgm + 1 < segs) add_part(at + kSeg);
#pragma unroll
        for (int k = 0; k < S::BCS; ++k) {
            const int i = threadIdx.x + k * S::THREADS;
            if (i < kSeg * 2 * NP) reinterpret_cast<f2 *>(bc)[i] = splat(held_bc[k][0]);
        }
        if (sgm > 0) load_ahead(at - kSeg);
        __syncthreads();
        // forwards again, every second state to shared memory
#pragma unroll 4
        for (int j = 0; j < kSeg; ++j) {
            if ((j & 1) == 0 && j > 0) {
#pragma unroll
                for (int n = 0; n < 4; ++n) hist[((j / 2 - 1) * 4 + n) * 32 + lane] = ulonglong2{h[0][n], h[1][n]};
            }
            const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(f_delta + j * CW + ch0);
            const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(f_u + j * CW + ch0);
            const f2 dd[2] = {d.x, d.y}, xx[2] = {mul2(d.x, u.x), mul2(d.y, u.y)};
            const f2 *sb = reinterpret_cast<const f2 *>(bc) + j * 2 * NP + 4 * nl;
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sb + n);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    h[c][n] = fma2(ex2_2(fma2(dd[c], A2[c][n], splat(kEx2Bias))), h[c][n], mul2(xx[c], v.x));
                    h[c][n + 1] = fma2(ex2_2(fma2(dd[c], A2[c][n + 1], splat(kEx2Bias))), h[c][n + 1], mul2(xx[c], v.y));
                }
            }
        }
        // The lanes' parts of token j's sums: over states (sB, sA, sY of the lane's
        // channels) and over channels (vD: grad_B's and grad_C's 4 states).
        auto finish = [&](int j, const f2 (&sB)[2], const f2 (&sA)[2], const f2 (&sY)[2], float (&vD)[8]) {
            float vB[4], vA[4], vY[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                unpack2(sB[c], vB[2 * c], vB[2 * c + 1]);
                unpack2(sA[c], vA[2 * c], vA[2 * c + 1]);
                unpack2(sY[c], vY[2 * c], vY[2 * c + 1]);
            }
            reduce_lanes<4, LN, 1>(vB, lane);
            reduce_lanes<4, LN, 1>(vA, lane);
            if (p.z.p) reduce_lanes<4, LN, 1>(vY, lane);
            reduce_lanes<8, LD, LN>(vD, lane);
            constexpr int KEEP = LD >= 8 ? 1 : 8 / LD;
            constexpr int COPIES = LD >= 8 ? LD / 8 : 1;
            if (dl % COPIES == 0) {
#pragma unroll
                for (int k = 0; k < KEEP; ++k) {
                    const int v = dl / COPIES * KEEP + k;
                    part[(warp * kSeg + j) * 2 * NP + (v / 4) * NP + 4 * nl + v % 4] = vD[k];
                }
            }
            // the lane's own channels: the results take the places of delta, u and
            // grad_out SiLU', which every lane of the warp has read
            if (writer) {
#pragma unroll
                for (int k = 0; k < OWN; ++k) {
                    const int e = j * CW + own0 + k;
                    const float delta = f_delta[e], u = f_u[e], dyo = f_dy[e];
                    const float gdt = fmaf(vB[k], u, vA[k] * kLn2) * f_sig[e];
                    f_u[e] = fmaf(vB[k], delta, skip[k] * dyo);
                    f_delta[e] = gdt;
                    f_dz[e] *= fmaf(skip[k], u, vY[k]);
                    gD[k] = fmaf(dyo, u, gD[k]);
                    if (at + j < t1) gbias[k] += gdt;
                }
            }
        };
        // backwards, tokens 2 k + 1 and 2 k together, from the row's last token on
        // (behind it the state and its gradient stay).  HALF: 2 k is that token, and
        // the state after it, which may be infinite, is no term of grad_A.  (A copy of
        // the body for it, chosen in the loop: 1013 -> 1015 us of a training step of
        // 4 x 2048 tokens x 4096 channels; with that pair in front of the loop 1022,
        // with a test in one body 1045.)
        auto two_tokens = [&](auto half, int k) {
            constexpr bool HALF = decltype(half)::value;
            const float *const fd = f_delta + 2 * k * CW + ch0, *const fu = f_u + 2 * k * CW + ch0;
            const float *const fy = f_dy + 2 * k * CW + ch0;
            const ulonglong2 qd0 = *reinterpret_cast<const ulonglong2 *>(fd);
            const ulonglong2 qd1 = *reinterpret_cast<const ulonglong2 *>(fd + CW);
            const ulonglong2 qu0 = *reinterpret_cast<const ulonglong2 *>(fu);
            const ulonglong2 qu1 = *reinterpret_cast<const ulonglong2 *>(fu + CW);
            const ulonglong2 qy0 = *reinterpret_cast<const ulonglong2 *>(fy);
            const ulonglong2 qy1 = *reinterpret_cast<const ulonglong2 *>(fy + CW);
            const f2 d0[2] = {qd0.x, qd0.y}, d1[2] = {qd1.x, qd1.y}, y0[2] = {qy0.x, qy0.y}, y1[2] = {qy1.x, qy1.y};
            const f2 x0[2] = {mul2(qd0.x, qu0.x), mul2(qd0.y, qu0.y)}, x1[2] = {mul2(qd1.x, qu1.x), mul2(qd1.y, qu1.y)};
            const f2 *const sb = reinterpret_cast<const f2 *>(bc) + 2 * k * 2 * NP + 4 * nl;
            const ulonglong2 *const before = k > 0 ? hist + (k - 1) * 128 + lane : mark;
            f2 sB0[2] = {0, 0}, sA0[2] = {0, 0}, sY0[2] = {0, 0}, sB1[2] = {0, 0}, sA1[2] = {0, 0}, sY1[2] = {0, 0};
            float v0[8], v1[8];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const f2 b0 = sb[n], c0n = sb[NP + n], b1 = sb[2 * NP + n], c1n = sb[3 * NP + n];
                const ulonglong2 e = before[n * 32];
                const f2 h0[2] = {e.x, e.y};
                f2 dB0 = 0, dC0 = 0, dB1 = 0, dC1 = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const f2 a0 = ex2_2(fma2(d0[c], A2[c][n], splat(kEx2Bias)));
                    const f2 a1 = ex2_2(fma2(d1[c], A2[c][n], splat(kEx2Bias)));
                    const f2 h1 = fma2(a0, h0[c], mul2(x0[c], b0));   // the state between the two
                    f2 gn = fma2(y1[c], c1n, g[c][n]);
                    sB1[c] = fma2(gn, b1, sB1[c]);
                    dB1 = fma2(gn, x1[c], dB1);
                    dC1 = fma2(y1[c], h[c][n], dC1);
                    sY1[c] = fma2(c1n, h[c][n], sY1[c]);
                    f2 ga = mul2(gn, a1);
                    f2 w = mul2(ga, h1);
                    sA1[c] = fma2(w, A2[c][n], sA1[c]);
                    if constexpr (!HALF) dA[c][n] = fma2(w, d1[c], dA[c][n]);
                    gn = fma2(y0[c], c0n, ga);
                    sB0[c] = fma2(gn, b0, sB0[c]);
                    dB0 = fma2(gn, x0[c], dB0);
                    dC0 = fma2(y0[c], h1, dC0);
                    sY0[c] = fma2(c0n, h1, sY0[c]);
                    ga = mul2(gn, a0);
                    w = mul2(ga, h0[c]);
                    sA0[c] = fma2(w, A2[c][n], sA0[c]);
                    dA[c][n] = fma2(w, d0[c], dA[c][n]);
                    g[c][n] = ga;
                    h[c][n] = h0[c];
                }
                float lo, hi;
                unpack2(dB0, lo, hi);
                v0[n] = lo + hi;
                unpack2(dC0, lo, hi);
                v0[4 + n] = lo + hi;
                unpack2(dB1, lo, hi);
                v1[n] = lo + hi;
                unpack2(dC1, lo, hi);
                v1[4 + n] = lo + hi;
            }
            finish(2 * k + 1, sB1, sA1, sY1, v1);
            finish(2 * k, sB0, sA0, sY0, v0);
        };
#pragma unroll 1
        for (int k = kSeg / 2 - 1; k >= 0; --k) {
            if (at + 2 * k >= t1) continue;
            if (at + 2 * k + 1 < t1) two_tokens(std::false_type(), k);
            else two_tokens(std::true_type(), k);
        }
        // the results of the warp's channels
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const Ref<void> &o = i == 0 ? p.gu : (i == 1 ? p.gdt : p.gz);
            const float *const f = i == 0 ? f_u : (i == 1 ? f_delta : f_dz);
            if (!o.p) continue;
            T *const row = scan_row<T>(o, b, at) + dbase;
            if constexpr (WIDE) {
#pragma unroll
                for (int k = 0; k < Q::COPIES; ++k) {
                    const int e = lane + 32 * k;
                    const int j = e / (CW / Q::PIECE), c = e % (CW / Q::PIECE) * Q::PIECE;
                    if (j >= kSeg || at + j >= t1 || c >= left) continue;
                    float v[Q::PIECE];
#pragma unroll
                    for (int m = 0; m < Q::PIECE; m += 4) {
                        const float4 q = *reinterpret_cast<const float4 *>(f + j * CW + c + m);
                        v[m] = q.x; v[m + 1] = q.y; v[m + 2] = q.z; v[m + 3] = q.w;
                    }
                    *reinterpret_cast<Vec<T, Q::PIECE> *>(row + (j * token_step(o) + c)) = Vec<T, Q::PIECE>::from(v);
                }
            } else {
                for (int e = lane; e < S::FIELD; e += 32) {
                    const int j = e / CW, c = e % CW;
                    if (at + j < t1 && c < left) put<T>(row, j * token_step(o) + c, f[e]);
                }
            }
        }
    }
    if (segs > 0) {
        __syncthreads();
        add_part(c0);
    }
    // what the chunk adds to the parameters' gradients, and the carried state's
    if (ch0 < left) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (4 * nl + n < p.states)
                *reinterpret_cast<ulonglong2 *>(p.part_A + (outer * p.states + 4 * nl + n) * p.pad + pbase + ch0) =
                    ulonglong2{dA[0][n], dA[1][n]};
    }
    if (main_i == 0 && p.gstate) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float s0[4], s1[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) unpack2(g[c][n], s0[n], s1[n]);
            const long long row = b * p.channels + dbase + ch0 + 2 * c;
            if (ch0 + 2 * c < left) store_states<4>(p.gstate, row, p.states, 4 * nl, s0);
            if (ch0 + 2 * c + 1 < left) store_states<4>(p.gstate, row + 1, p.states, 4 * nl, s1);
        }
    }
    if (writer) {
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            if (own0 + k >= left) continue;
            p.part_D[outer * p.pad + pbase + own0 + k] = gD[k];
            p.part_bias[outer * p.pad + pbase + own0 + k] = gbias[k];
        }
    }
}

// Adds the partial rows.  The first blocks: grad_B and grad_C, one thread per
// value, over the group's column tiles.  The others: grad_A, grad_D and
// grad_dt_bias, 32 channels' values per block, the chunks split over 8 warps.
template <typename T>
__global__ void __launch_bounds__(256) scan_grad_sum_kernel(const __grid_constant__ ScanParams p, unsigned bc_blocks) {
    begin_kernel();
    const int NP = 4 * p.quads;
    if (blockIdx.x < bc_blocks) {
        const long long per_tile = p.batch * p.length * p.groups * 2 * NP;
        const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
        if (i >= per_tile) return;
        const int m = static_cast<int>(i % NP);
        const bool is_c = i % (2 * NP) >= NP;
        long long r = i / (2 * NP);
        const int g = static_cast<int>(r % p.groups);
        r /= p.groups;
        const long long t = r % p.length, b = r / p.length;
        if (m >= p.states) return;
        float s = 0.f;
        if (t < scan_length(p, b)) {
#pragma unroll 4
            for (int k = 0; k < p.tiles_per_group; ++k) s += p.part_BC[k * per_tile + i];
        }
        const Ref<void> &o = is_c ? p.gC : p.gB;
        put<T>(scan_row<T>(o, b, t), g * o.sg + m, s);
        return;
    }
    __shared__ float red[8][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long long n_a = (long long)p.states * p.pad;
    const long long total = n_a + 2LL * p.pad;
    const long long i = (long long)(blockIdx.x - bc_blocks) * 32 + lane;
    const long long parts = p.batch * p.n_main;
    const int in_group = static_cast<int>(i % p.pad % p.group_pad);
    const bool on = i < total && in_group < p.group_channels;
    float s = 0.f;
    if (on) {
        const float *src = i < n_a ? p.part_A + i : (i < n_a + p.pad ? p.part_D + (i - n_a) : p.part_bias + (i - n_a - p.pad));
        const long long step = i < n_a ? n_a : p.pad;
#pragma unroll 4
        for (long long k = warp; k < parts; k += 8) s += src[k * step];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || !on) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    const long long d = i % p.pad / p.group_pad * p.group_channels + in_group;
    if (i < n_a) p.grad_A[d * p.states + i / p.pad] = s;
    else if (i < n_a + p.pad) {
        if (p.grad_D) p.grad_D[d] = s;
    } else if (p.grad_bias) {
        p.grad_bias[d] = s;
    }
}

template <typename T, int LN, bool WIDE>
cudaError_t launch_bwd(const ScanParams &p, unsigned grid, cudaStream_t s) {
    using S = BwdShape<T, LN, WIDE>;
    constexpr int smem = S::TOTAL * 4;
    auto *k = scan_bwd_kernel<T, LN, WIDE>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(k, smem, p.device);
    if (e != cudaSuccess) return e;
    return launch(k, grid, S::THREADS, smem, s, p);
}

template <typename T, bool WIDE>
cudaError_t bwd_by_states(const ScanParams &p, unsigned grid, cudaStream_t s) {
    switch (p.quads) {
        case 1: return launch_bwd<T, 1, WIDE>(p, grid, s);
        case 2: return launch_bwd<T, 2, WIDE>(p, grid, s);
        case 4: return launch_bwd<T, 4, WIDE>(p, grid, s);
        case 8: return launch_bwd<T, 8, WIDE>(p, grid, s);
        case 16: return launch_bwd<T, 16, WIDE>(p, grid, s);
        default: return launch_bwd<T, 32, WIDE>(p, grid, s);
    }
}

template <typename T>
cudaError_t bwd_and_sums(bool wide, const ScanParams &p, unsigned grid, cudaStream_t s) {
    const cudaError_t e = wide ? bwd_by_states<T, true>(p, grid, s) : bwd_by_states<T, false>(p, grid, s);
    if (e != cudaSuccess) return e;
    const long long bc = p.batch * p.length * p.groups * 8 * p.quads;
    const unsigned bc_blocks = (unsigned)((bc + 255) / 256);
    const unsigned par_blocks = (unsigned)(((long long)p.states * p.pad + 2LL * p.pad + 31) / 32);
    return launch(scan_grad_sum_kernel<T>, bc_blocks + par_blocks, 256, 0, s, p, bc_blocks);
}

}  // namespace

// Channels of one block of the backward kernel, and blocks that an SM holds.
int scan_bwd_columns(int quads) { return bwd_warps(quads) * 128 / quads; }
template <typename T, bool WIDE>
int bwd_resident(int quads) {
    switch (quads) {
        case 1: return BwdShape<T, 1, WIDE>::BLOCKS;
        case 2: return BwdShape<T, 2, WIDE>::BLOCKS;
        case 4: return BwdShape<T, 4, WIDE>::BLOCKS;
        case 8: return BwdShape<T, 8, WIDE>::BLOCKS;
        case 16: return BwdShape<T, 16, WIDE>::BLOCKS;
        default: return BwdShape<T, 32, WIDE>::BLOCKS;
    }
}
int scan_bwd_resident(int quads, seq_dtype_t dtype, bool wide) {
    if (dtype == SEQ_F32) return wide ? bwd_resident<float, true>(quads) : bwd_resident<float, false>(quads);
    return wide ? bwd_resident<bf16, true>(quads) : bwd_resident<bf16, false>(quads);
}

cudaError_t launch_scan_bwd(seq_dtype_t dtype, bool wide, const ScanParams &p, unsigned grid, cudaStream_t s) {
    if (dtype == SEQ_F32) return bwd_and_sums<float>(wide, p, grid, s);
    if (dtype == SEQ_F16) return bwd_and_sums<f16>(wide, p, grid, s);
    return bwd_and_sums<bf16>(wide, p, grid, s);
}

}  // namespace seq
