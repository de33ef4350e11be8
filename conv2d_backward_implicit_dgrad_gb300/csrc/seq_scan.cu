// C ABI of the selective scan (include/seq.h): plans, checks, workspace and
// the cut of time into chunks.
#include <algorithm>
#include <climits>
#include <new>

#include "seq_scan.cuh"

using namespace seq;

struct seq_scan_plan_s {
    PlanBase base;
    long long batch, length;
    int channels, states, groups, quads;
    seq_dtype_t dtype;
    void *fwd, *bwd;            // chunk states and sums; partial sums of the gradients
    size_t fwd_bytes, bwd_bytes;
};

namespace {

constexpr int kMostChunks = 64;
constexpr int kLeastSpan = 16;   // tokens of a chunk, at least

int quads_of(int states) {
    int q = 1;
    while (4 * q < states) q *= 2;
    return q;
}

long long round_up(long long v, long long to) { return (v + to - 1) / to * to; }

// Into how many spans to cut `length` tokens, walked by `blocks` blocks each
// of which `resident` run at once: the cut whose last block ends first.  A
// span costs its tokens and about 24 more for its start; cutting at all costs
// `pass` of the main kernel's time for the pass over the chunks (of measured
// kernels: 197 of 286 us forwards, 119 of 600 backwards, at 16 states).  The 24
// and the 2 % that a finer cut has to gain are estimates, held against a few
// sizes and not swept.
int spans_of(long long blocks, long long length, long long resident, double pass) {
    const long long most = std::max<long long>(1, std::min<long long>(kMostChunks, length / kLeastSpan));
    int best = 1;
    double least = 0;
    for (int n = 1; n <= most; ++n) {
        const double span = (double)round_up((length + n - 1) / n, kSeg);
        const double waves = (double)((blocks * n + resident - 1) / resident);
        const double cost = waves * (span + 24) * (n == 1 ? 1 : 1 + pass);
        if (n == 1 || cost < 0.98 * least) {
            best = n;
            least = cost;
        }
    }
    return best;
}

// The padded channels of the internal buffers (see seq_scan.cuh).
long long pad_of(const seq_scan_plan_s *pl) { return pl->groups * round_up(pl->channels / pl->groups, 4); }

// Chunks that a row of a call can have at most.
long long most_chunks(const seq_scan_plan_s *pl) {
    return std::max<long long>(1, std::min<long long>(kMostChunks, pl->length / kLeastSpan));
}

size_t fwd_need(const seq_scan_plan_s *pl) {
    const long long most = most_chunks(pl);
    return most == 1 ? 0 : (size_t)pl->batch * most * pad_of(pl) * (pl->states + 1) * 4;
}

int tiles_of(const seq_scan_plan_s *pl, int columns) {
    return (pl->channels / pl->groups + columns - 1) / columns;
}

size_t bwd_need(const seq_scan_plan_s *pl) {
    const size_t rows = (size_t)pl->batch * most_chunks(pl) * pad_of(pl) * (pl->states + 2);
    const size_t bc = (size_t)tiles_of(pl, scan_bwd_columns(pl->quads)) * pl->batch * pl->length * pl->groups * 8 * pl->quads;
    return (rows + bc) * 4;
}

// Whether the rows of all these lie in pieces of `bytes` bytes.
bool in_pieces(const seq_scan_plan_s *pl, size_t bytes, std::initializer_list<const seq_ref_t *> refs) {
    const size_t es = elem_size(pl->dtype);
    if ((pl->channels / pl->groups) * es % bytes) return false;
    for (const seq_ref_t *r : refs)
        if (!rows_aligned(*r, es, bytes)) return false;
    return true;
}

void fill(const seq_scan_plan_s *pl, long long batch, long long length, int columns, ScanParams *p) {
    p->batch = batch;
    p->length = length;
    p->channels = pl->channels;
    p->states = pl->states;
    p->groups = pl->groups;
    p->group_channels = pl->channels / pl->groups;
    p->group_pad = (int)round_up(p->group_channels, 4);
    p->pad = p->groups * p->group_pad;
    p->quads = pl->quads;
    p->device = pl->base.device;
    p->tiles_per_group = tiles_of(pl, columns);
}

void set_chunks(const seq_scan_plan_s *pl, int spans, ScanParams *p) {
    p->chunk = (int)round_up((p->length + spans - 1) / spans, kSeg);
    p->n_chunks = (int)((p->length + p->chunk - 1) / p->chunk);
    p->chunk_state = static_cast<float *>(pl->fwd);
    p->chunk_sum = p->chunk_state + (size_t)p->batch * p->n_chunks * pl->states * p->pad;
}

// The forward kernels' chunks; returns their grid.
long long cut_forward(const seq_scan_plan_s *pl, bool wide, ScanParams *p) {
    const long long tiles = (long long)p->groups * p->tiles_per_group * p->batch;
    const long long resident = (long long)scan_fwd_resident(pl->quads, wide) * pl->base.sm_count;
    set_chunks(pl, spans_of(tiles, p->length, resident, 0.65), p);
    return tiles * p->n_chunks;
}

// The backward main kernel's spans, and the chunks of each that the pass over
// the chunks (whose blocks are smaller) works on;
// returns the main kernel's grid.
long long cut_backward(const seq_scan_plan_s *pl, bool wide, ScanParams *p) {
    const int tiles_per_group_rev = tiles_of(pl, scan_fwd_columns(pl->quads));
    const long long tiles = (long long)p->groups * p->tiles_per_group * p->batch;
    const long long resident = (long long)scan_bwd_resident(pl->quads, pl->dtype, wide) * pl->base.sm_count;
    const int n = spans_of(tiles, p->length, resident, 0.2);
    p->per = 1;
    if (n > 1) {
        const long long tiles_rev = (long long)p->groups * tiles_per_group_rev * p->batch;
        const long long resident_rev = (long long)scan_fwd_resident(pl->quads, wide) * pl->base.sm_count;
        const long long most = std::max<long long>(1, std::min<long long>(kMostChunks, p->length / kLeastSpan));
        p->per = (int)std::max<long long>(1, std::min(resident_rev / (tiles_rev * n), most / n));
    }
    set_chunks(pl, n * p->per, p);
    p->n_main = (p->n_chunks + p->per - 1) / p->per;
    return tiles * p->n_main;
}

}  // namespace

extern "C" {

dgrad_status_t seq_scan_plan(long long batch, long long length, long long channels, int states, int groups,
                             seq_dtype_t dtype, seq_scan_plan_t *plan_out) {
    if (!plan_out) return DGRAD_ERR_INVALID_ARG;
    *plan_out = nullptr;
    if (batch < 1 || length < 1 || channels < 1 || states < 1 || groups < 1 || (int)dtype < 0 || dtype > SEQ_BF16 ||
        channels % groups != 0)
        return DGRAD_ERR_INVALID_ARG;
    if (states > 128 || length > INT_MAX - 4096 || channels * states > INT_MAX || batch > (1 << 24))
        return DGRAD_ERR_UNSUPPORTED;
    // grids: blocks of at least 16 channels, at most kMostChunks chunks; 256 sums of grad_B and grad_C a block
    const double tiles = (double)groups * ((channels / groups + 15) / 16) * batch;
    if (tiles * kMostChunks > 2.0e9 || (double)batch * length * groups * 4 * states / 256 > 1.0e9 ||
        (double)channels * states * 2 / 32 > 1.0e9 || (double)batch * ((channels + 7) / 8) > 2.0e9)
        return DGRAD_ERR_UNSUPPORTED;
    seq_scan_plan_s *pl = new (std::nothrow) seq_scan_plan_s();
    if (!pl) return DGRAD_ERR_OOM;
    dgrad_status_t st = open_plan(&pl->base);
    if (st != DGRAD_OK) {
        delete pl;
        return st;
    }
    pl->batch = batch;
    pl->length = length;
    pl->channels = (int)channels;
    pl->states = states;
    pl->groups = groups;
    pl->quads = quads_of(states);
    pl->dtype = dtype;
    if ((st = grow(&pl->fwd, &pl->fwd_bytes, fwd_need(pl))) != DGRAD_OK) {
        close_plan(pl->base, nullptr, 0);
        delete pl;
        return st;
    }
    *plan_out = pl;
    return DGRAD_OK;
}

size_t seq_scan_checkpoint_bytes(seq_scan_plan_t pl, long long batch, long long length) {
    if (!pl || batch < 1 || length < 1) return 0;
    return (size_t)batch * ((length + kSeg - 1) / kSeg) * pl->states * pad_of(pl) * 4;
}

dgrad_status_t seq_scan_run(seq_scan_plan_t pl, const seq_scan_args_t *a, void *stream) {
    if (!pl || !a || !a->u.ptr || !a->dt.ptr || !a->B.ptr || !a->C.ptr || !a->out.ptr || !a->A || a->batch < 1 ||
        a->batch > pl->batch || a->length < 1 || a->length > pl->length)
        return DGRAD_ERR_INVALID_ARG;
    for (const seq_ref_t *r : {&a->u, &a->dt, &a->B, &a->C, &a->z, &a->out})
        if (!strides_ok(*r)) return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype);
    if (!all_aligned(es, {a->u.ptr, a->dt.ptr, a->B.ptr, a->C.ptr, a->z.ptr, a->out.ptr}) ||
        !all_aligned(4, {a->A, a->D, a->dt_bias, a->lengths, a->state, a->final_state}) || !aligned(a->checkpoints, 16))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels, N = pl->states, b = a->batch, l = a->length;
    const size_t st_b = (size_t)b * D * N * 4;
    const Span outs[] = {span(a->out, b, l, 1, D, es), flat(a->final_state, st_b),
                         flat(a->checkpoints, seq_scan_checkpoint_bytes(pl, b, l))};
    const Span ins[] = {span(a->u, b, l, 1, D, es), span(a->dt, b, l, 1, D, es), span(a->B, b, l, pl->groups, N, es),
                        span(a->C, b, l, pl->groups, N, es), span(a->z, b, l, 1, D, es), flat(a->A, D * N * 4),
                        flat(a->D, D * 4), flat(a->dt_bias, D * 4), flat(a->lengths, b * 4), flat(a->state, st_b)};
    if (!rows_distinct(outs[0])) return DGRAD_ERR_INVALID_ARG;
    if (any_overlap(outs, 3, ins, 10)) return DGRAD_ERR_ALIAS;
    dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    ScanParams p{};
    fill(pl, b, l, scan_fwd_columns(pl->quads), &p);
    const bool wide = in_pieces(pl, 16, {&a->u, &a->dt, &a->z, &a->out});
    const long long grid = cut_forward(pl, wide, &p);
    p.u = ref<void>(a->u);
    p.dt = ref<void>(a->dt);
    p.B = ref<void>(a->B);
    p.C = ref<void>(a->C);
    p.z = ref<void>(a->z);
    p.out = ref<void>(a->out);
    p.A = a->A;
    p.D = a->D;
    p.dt_bias = a->dt_bias;
    p.lengths = a->lengths;
    p.state = a->state;
    p.final_state = a->final_state;
    p.ck = a->checkpoints;
    return dgrad::cuda_status(launch_scan_fwd(pl->dtype, wide, p, (unsigned)grid, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t seq_scan_backward(seq_scan_plan_t pl, const seq_scan_grad_args_t *a, void *stream) {
    if (!pl || !a || !a->grad_out.ptr || !a->u.ptr || !a->dt.ptr || !a->B.ptr || !a->C.ptr || !a->A ||
        !a->checkpoints || !a->grad_u.ptr || !a->grad_dt.ptr || !a->grad_B.ptr || !a->grad_C.ptr || !a->grad_A ||
        a->batch < 1 || a->batch > pl->batch || a->length < 1 || a->length > pl->length ||
        (a->z.ptr != nullptr) != (a->grad_z.ptr != nullptr) || (a->grad_state && !a->state) ||
        (a->grad_D && !a->D) || (a->grad_dt_bias && !a->dt_bias))
        return DGRAD_ERR_INVALID_ARG;
    for (const seq_ref_t *r : {&a->grad_out, &a->u, &a->dt, &a->B, &a->C, &a->z, &a->grad_u, &a->grad_dt, &a->grad_B,
                               &a->grad_C, &a->grad_z})
        if (!strides_ok(*r)) return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype);
    if (!all_aligned(es, {a->grad_out.ptr, a->u.ptr, a->dt.ptr, a->B.ptr, a->C.ptr, a->z.ptr, a->grad_u.ptr,
                           a->grad_dt.ptr, a->grad_B.ptr, a->grad_C.ptr, a->grad_z.ptr}) ||
        !all_aligned(4, {a->A, a->D, a->dt_bias, a->lengths, a->state, a->grad_final, a->grad_state, a->grad_A,
                          a->grad_D, a->grad_dt_bias}) ||
        !aligned(a->checkpoints, 16))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels, N = pl->states, b = a->batch, l = a->length, G = pl->groups;
    const size_t st_b = (size_t)b * D * N * 4;
    const Span outs[] = {span(a->grad_u, b, l, 1, D, es), span(a->grad_dt, b, l, 1, D, es),
                         span(a->grad_B, b, l, G, N, es), span(a->grad_C, b, l, G, N, es),
                         span(a->grad_z, b, l, 1, D, es), flat(a->grad_state, st_b), flat(a->grad_A, D * N * 4),
                         flat(a->grad_D, D * 4), flat(a->grad_dt_bias, D * 4)};
    const Span ins[] = {span(a->grad_out, b, l, 1, D, es), span(a->u, b, l, 1, D, es), span(a->dt, b, l, 1, D, es),
                        span(a->B, b, l, G, N, es), span(a->C, b, l, G, N, es), span(a->z, b, l, 1, D, es),
                        flat(a->A, D * N * 4), flat(a->D, D * 4), flat(a->dt_bias, D * 4), flat(a->lengths, b * 4),
                        flat(a->state, st_b), flat(a->grad_final, st_b),
                        flat(a->checkpoints, seq_scan_checkpoint_bytes(pl, b, l))};
    for (int i = 0; i < 5; ++i)
        if (!rows_distinct(outs[i])) return DGRAD_ERR_INVALID_ARG;
    if (any_overlap(outs, 9, ins, 13)) return DGRAD_ERR_ALIAS;
    dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    if ((st = grow(&pl->bwd, &pl->bwd_bytes, bwd_need(pl))) != DGRAD_OK) return st;
    ScanParams p{};
    p.gout = ref<void>(a->grad_out);
    p.u = ref<void>(a->u);
    p.dt = ref<void>(a->dt);
    p.B = ref<void>(a->B);
    p.C = ref<void>(a->C);
    p.z = ref<void>(a->z);
    p.gu = ref<void>(a->grad_u);
    p.gdt = ref<void>(a->grad_dt);
    p.gB = ref<void>(a->grad_B);
    p.gC = ref<void>(a->grad_C);
    p.gz = ref<void>(a->grad_z);
    p.A = a->A;
    p.D = a->D;
    p.dt_bias = a->dt_bias;
    p.lengths = a->lengths;
    p.gfinal = a->grad_final;
    p.gstate = a->grad_state;
    p.ck = const_cast<float *>(a->checkpoints);
    p.grad_A = a->grad_A;
    p.grad_D = a->grad_D;
    p.grad_bias = a->grad_dt_bias;
    fill(pl, b, l, scan_bwd_columns(pl->quads), &p);
    const bool wide = in_pieces(pl, 16, {&a->u, &a->dt, &a->z, &a->grad_out, &a->grad_u, &a->grad_dt, &a->grad_z});
    const long long grid = cut_backward(pl, wide, &p);
    const size_t rows = (size_t)b * p.n_main * p.pad;
    p.part_A = static_cast<float *>(pl->bwd);
    p.part_D = p.part_A + rows * pl->states;
    p.part_bias = p.part_D + rows;
    p.part_BC = p.part_bias + rows;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.n_main > 1) {
        ScanParams r = p;
        r.tiles_per_group = tiles_of(pl, scan_fwd_columns(pl->quads));
        const long long rev = (long long)G * r.tiles_per_group * b * p.n_chunks;
        if ((st = dgrad::cuda_status(launch_scan_rev(pl->dtype, wide, r, (unsigned)rev, s))) != DGRAD_OK) return st;
    }
    return dgrad::cuda_status(launch_scan_bwd(pl->dtype, wide, p, (unsigned)grid, s));
}

dgrad_status_t seq_scan_step(seq_scan_plan_t pl, const seq_scan_step_args_t *a, void *stream) {
    if (!pl || !a || !a->u.ptr || !a->dt.ptr || !a->B.ptr || !a->C.ptr || !a->out.ptr || !a->A || !a->cache ||
        a->batch < 1 || a->batch > pl->batch || a->n_slots < 1 || (!a->slots && a->n_slots < a->batch))
        return DGRAD_ERR_INVALID_ARG;
    for (const seq_ref_t *r : {&a->u, &a->dt, &a->B, &a->C, &a->z, &a->out})
        if (!strides_ok(*r)) return DGRAD_ERR_INVALID_ARG;
    const size_t es = elem_size(pl->dtype);
    if (!all_aligned(es, {a->u.ptr, a->dt.ptr, a->B.ptr, a->C.ptr, a->z.ptr, a->out.ptr}) ||
        !all_aligned(4, {a->A, a->D, a->dt_bias, a->cache, a->slots, a->write_slots}))
        return DGRAD_ERR_MISALIGNED;
    const long long D = pl->channels, N = pl->states, b = a->batch;
    const Span outs[] = {span(a->out, b, 1, 1, D, es), flat(a->cache, (size_t)a->n_slots * D * N * 4)};
    const Span ins[] = {span(a->u, b, 1, 1, D, es), span(a->dt, b, 1, 1, D, es), span(a->B, b, 1, pl->groups, N, es),
                        span(a->C, b, 1, pl->groups, N, es), span(a->z, b, 1, 1, D, es), flat(a->A, D * N * 4),
                        flat(a->D, D * 4), flat(a->dt_bias, D * 4), flat(a->slots, b * 4), flat(a->write_slots, b * 4)};
    if (!rows_distinct(outs[0])) return DGRAD_ERR_INVALID_ARG;
    if (any_overlap(outs, 2, ins, 10)) return DGRAD_ERR_ALIAS;
    const dgrad_status_t st = on_device(pl->base);
    if (st != DGRAD_OK) return st;
    ScanStepParams p{};
    p.batch = b;
    p.n_slots = a->n_slots;
    p.channels = pl->channels;
    p.states = pl->states;
    p.group_channels = pl->channels / pl->groups;
    p.u = ref<void>(a->u);
    p.dt = ref<void>(a->dt);
    p.B = ref<void>(a->B);
    p.C = ref<void>(a->C);
    p.z = ref<void>(a->z);
    p.out = ref<void>(a->out);
    p.A = a->A;
    p.D = a->D;
    p.dt_bias = a->dt_bias;
    p.cache = a->cache;
    p.slots = a->slots;
    p.write_slots = a->write_slots;
    p.err = pl->base.err;
    p.sm_count = pl->base.sm_count;
    // rows of B and C in 16-byte pieces (or whole, where they are shorter)
    const size_t piece = std::min<size_t>(16, N * es);
    p.wide_bc = rows_aligned(a->B, es, piece) && rows_aligned(a->C, es, piece) &&
                (pl->groups == 1 || ((a->B.sg * es) % piece == 0 && (a->C.sg * es) % piece == 0));
    return dgrad::cuda_status(launch_scan_step(pl->dtype, p, pl->quads, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t seq_scan_check(seq_scan_plan_t pl) { return pl ? read_error(pl->base) : DGRAD_ERR_INVALID_ARG; }

size_t seq_scan_workspace_bytes(seq_scan_plan_t pl, int gradients) {
    return pl ? kErrorBytes + fwd_need(pl) + (gradients ? bwd_need(pl) : 0) : 0;
}

void seq_scan_destroy(seq_scan_plan_t pl) {
    if (!pl) return;
    void *mems[] = {pl->fwd, pl->bwd};
    close_plan(pl->base, mems, 2);
    delete pl;
}

}  // extern "C"
