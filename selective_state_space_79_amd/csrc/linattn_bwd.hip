// linattn_bwd.hip -- gradients of linear attention with a decay for each head.
//
// dq, dk and dv are passes of linattn.h with other rows in the three roles (dq in order of
// time from the forward's states S, dk and dv against it from the gradient dS of the state).
// States are kept at the ends of pieces of the sequences only and walked again inside.
//
// The decays' gradient.  dg_t = e^{g_t} <S_{t-1}, dS_t>.  In a chunk that state S_in enters
// and that the gradient dS_out enters from behind, with D the decays between two tokens,
//   a_i = scale e^{G_i} q_i S_in do_i           (what token i reads from before the chunk)
//   b_j = e^{G_C - G_j} k_j dS_out v_j          (what later chunks read of token j)
//   M_ij = scale D_ij (q_i . k_j)(do_i . v_j)   (what token i reads of token j < i)
// dg_t sums every read that crosses t: with X_in = <S_in, dS_in> at the chunk's start, all
// reads that cross it,
//   dg_t = X_in + sum_{j<t} (b_j - a_j) + sum_{i>=t>j} M_ij
//        = X_in + sum_{j<t} (b_j - a_j - e_j),   e_j = sum_i M_ji - sum_i M_ij.
// The e_j come from the row and column sums of one M, so what they leave in sums outside
// the rectangle i >= t > j cancels to float32 rounding.  X_in is taken afresh at each piece
// as a product of the two states there, so the error of a running sum spans one piece.
#include "linattn.h"

namespace {
namespace la {

struct GradTail {
    LinattnPass p;          // geometry
    const float* fwd;       // [pieces][H][dk dv] states that the pieces start from
    const float* rev;       // [pieces][H][dk dv] state gradients that the pieces start from, behind
    const float* s0;
    const float* ds0;
    const float* a;         // [slices][T][H]
    const float* b;
    const float* e;
    float* x;               // [pieces][H] <S, dS> at the pieces' starts
    float* part;            // [pieces][H] sums of dg (decay per head)
    float* dg;
    int32_t slices, head_decay;
    int32_t open_end;       // a gradient arrives at the final states
};

// <S, dS> at the start of each piece, one workgroup per piece and head.
__global__ void __launch_bounds__(kThreads) linattn_cross_kernel(GradTail t) {
    __shared__ float red[kWaves];
    const LinattnPass& p = t.p;
    const int64_t pi = blockIdx.x;
    const int h = blockIdx.y;
    const int seq = find_seq(p, pi);
    if (seq < 0) return;
    const Seq sq = seq_range(p, seq);
    const int64_t local = pi - piece_base(p, seq);
    if (local < 0 || (local > 0 && local * p.piece >= sq.end - sq.start)) return;
    const int64_t n = int64_t(p.kd) * p.vd;
    const float* u = local ? t.fwd + (pi * p.H + h) * n : t.s0 ? t.s0 + (int64_t(seq) * p.H + h) * n : nullptr;
    const float* v = local ? t.rev + ((pi - 1) * p.H + h) * n : t.s0 ? t.ds0 + (int64_t(seq) * p.H + h) * n : nullptr;
    float s = 0.0f;
    const int64_t n4 = n % 4 == 0 && !((reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(v)) & 15) ? n : 0;
    if (u) {
        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int64_t i = 4 * threadIdx.x; i < n4; i += 4 * kThreads) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(u + i), y = *reinterpret_cast<const f32x4*>(v + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = fmaf(x[e], y[e], a[e]);
        }
        s = (a[0] + a[1]) + (a[2] + a[3]);
        for (int64_t i = n4 + threadIdx.x; i < n; i += kThreads) s = fmaf(u[i], v[i], s);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = (red[0] + red[1]) + (red[2] + red[3]);
        if (local) {   // the gradient there is that of the piece's first state: one decay on
            const float g = p.g[(sq.start + local * p.piece) * p.sg + h];
            s *= __builtin_amdgcn_exp2f((g < kMinDecay ? kMinDecay : g) * kLog2e);
        }
        t.x[pi * p.H + h] = s;
    }
}

// dg of one piece for 16 heads.  64 threads of a head take 16 tokens each at a time: their
// sum, the sums of the threads before, then the running values.  Sums in float64.  Where the
// next piece's start is known too, what the running sum misses there is spread over the piece
// in proportion (the errors of the terms walk at random; this halves them and more).
constexpr int kDgThreads = 1024, kDgParts = kDgThreads / 16, kDgTokens = 16;

__global__ void __launch_bounds__(kDgThreads) linattn_dg_kernel(GradTail t) {
    __shared__ double sums[kDgParts][17];
    const LinattnPass& p = t.p;
    const int64_t pi = blockIdx.x;
    const int hh = threadIdx.x & 15, part = threadIdx.x >> 4, h = blockIdx.y * 16 + hh;
    const int seq = find_seq(p, pi);
    const Seq sq = seq < 0 ? Seq{0, 0} : seq_range(p, seq);
    const int64_t local = seq < 0 ? -1 : pi - piece_base(p, seq), len = sq.end - sq.start;
    const bool on = h < p.H;
    if (local < 0 || local * p.piece >= len) {
        if (t.head_decay && part == 0 && on) t.part[pi * p.H + h] = 0.0f;
        return;
    }
    const int64_t lo = sq.start + local * p.piece, hi = sq.end - lo > p.piece ? lo + p.piece : sq.end;
    const int64_t plane = p.T * p.H;
    auto f = [&](int64_t tok) {
        double s = 0.0;
        for (int k = 0; k < t.slices; ++k) {
            const int64_t o = k * plane + tok * p.H + h;
            s += (double(t.b[o]) - double(t.a[o])) - double(t.e[o]);
        }
        return s;
    };
    // the closing error: in one walk of the sums, before the walk that writes
    double miss = 0.0;
    const double start = on ? double(t.x[pi * p.H + h]) : 0.0;
    if (hi < sq.end || !t.open_end) {
        double s = 0.0;
        if (on)
            for (int64_t tok = lo + part; tok < hi; tok += kDgParts) s += f(tok);
        sums[part][hh] = s;
        __syncthreads();
        s = start;
        for (int k = 0; k < kDgParts; ++k) s += sums[k][hh];
        __syncthreads();
        miss = ((hi < sq.end && on ? double(t.x[(pi + 1) * p.H + h]) : 0.0) - s) / double(hi - lo);
    }
    double run = start, all = 0.0;
    for (int64_t base = lo; base < hi; base += kDgParts * kDgTokens) {
        const int64_t t0 = base + part * kDgTokens;
        double v[kDgTokens], s = 0.0;
#pragma unroll
        for (int k = 0; k < kDgTokens; ++k) {
            v[k] = on && t0 + k < hi ? f(t0 + k) : 0.0;
            s += v[k];
        }
        sums[part][hh] = s;
        __syncthreads();
        double r = run;
        for (int k = 0; k < kDgParts; ++k) {
            const double o = sums[k][hh];
            if (k < part) r += o;
            run += o;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDgTokens; ++k)
            if (on && t0 + k < hi) {
                const double d = r + miss * double(t0 + k - lo);
                all += d;
                if (!t.head_decay) t.dg[(t0 + k) * p.H + h] = float(d);
                r += v[k];
            }
    }
    if (t.head_decay) {
        sums[part][hh] = all;
        __syncthreads();
        if (part == 0 && on) {
            for (int k = 1; k < kDgParts; ++k) all += sums[k][hh];
            t.part[pi * p.H + h] = float(all);
        }
    }
}

// dg per head: the pieces' sums, in order, in float64.
__global__ void __launch_bounds__(kThreads) linattn_dg_sum_kernel(GradTail t) {
    __shared__ double sums[kThreads];
    const int h = blockIdx.x;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < t.p.npieces; i += kThreads) s += double(t.part[i * t.p.H + h]);
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d >>= 1) {
        if (int(threadIdx.x) < d) sums[threadIdx.x] += sums[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) t.dg[h] = float(sums[0]);
}

// Sums the heads that share a row, out[t][kh] = sum_r part[t][kh * rep + r], for dq and dk
// (the grid's y); one workgroup takes whole tokens, VW columns a thread.  Bound by the bytes
// of the parts.
struct GroupArgs {
    const float* part[2];
    void* out[2];
    int32_t rep, width, kheads;
};
template <typename IO, int VW>
__global__ void __launch_bounds__(kThreads) linattn_group_kernel(LinattnPass p, GroupArgs a) {
    typedef float vf __attribute__((ext_vector_type(VW)));
    const int per = a.width / VW, n = a.kheads * per;   // threads' work of one token
    const int64_t lo = p.cu ? seq_range(p, 0).start : 0, hi = p.cu ? seq_range(p, p.nseq - 1).end : p.T;
    const float* part = a.part[blockIdx.y];
    IO* out = static_cast<IO*>(a.out[blockIdx.y]);
    for (int64_t tok = blockIdx.x; tok < p.T; tok += gridDim.x) {
        const bool on = tok >= lo && tok < hi;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int kh = i / per, d = (i - kh * per) * VW;
            const float* q = part + (tok * p.H + int64_t(kh) * a.rep) * a.width + d;
            vf s = {};
            if (on) {
#pragma unroll 4
                for (int r = 0; r < a.rep; ++r) s += *reinterpret_cast<const vf*>(q + int64_t(r) * a.width);
            }
            IO raw[VW];
#pragma unroll
            for (int e = 0; e < VW; ++e) raw[e] = IOT<IO>::from_f32(s[e]);
            __builtin_memcpy(out + (tok * a.kheads + kh) * a.width + d, raw, sizeof(raw));
        }
    }
}

// Rows of no sequence (before the first and behind the last): zero gradients.
__global__ void __launch_bounds__(kThreads) linattn_zero_kernel(LinattnPass p, char* a, int64_t na, char* b, int64_t nb,
                                                                char* c, int64_t nc, char* d, int64_t nd) {
    const int64_t lo = seq_range(p, 0).start, hi = seq_range(p, p.nseq - 1).end;
    const int64_t free = p.T - (hi > lo ? hi - lo : 0);
    for (int64_t i = blockIdx.x; i < free; i += gridDim.x) {
        const int64_t t = i < lo ? i : p.T - free + i;
        char* rows[4] = {a, b, c, d};
        const int64_t n[4] = {na, nb, nc, nd};
        for (int k = 0; k < 4; ++k)   // bytes of a row: a multiple of 2
            for (int64_t e = threadIdx.x; rows[k] && e < n[k] / 2; e += kThreads)
                reinterpret_cast<uint16_t*>(rows[k] + t * n[k])[e] = 0;
    }
}

// ---------------------------------------------------------------- host
struct GradPlan {
    int64_t piece, npieces;
    bool pieced;
    int64_t slices_q, slices_s;   // of passes with kd = dv, vd = dk, and with kd = dk, vd = dv
    size_t carry, tot, dots, wide, x;   // bytes of one buffer each
    size_t bytes;
};

// Pieces of at most 1024 tokens: the error of dg's running sum grows with the piece, and the
// states of pieces this long are a sixteenth of the rows' bytes at dk = dv = 128.
inline int make_grad_plan(const ssm_linattn_dims* d, bool packed, GradPlan* pl) {
    pl->slices_q = cdiv(d->dk, ssm_detail::linattn_slice(d->dk));
    pl->slices_s = cdiv(d->dv, ssm_detail::linattn_slice(d->dv));
    const int64_t units = d->nheads * pl->slices_q;
    const int64_t each = packed ? d->tokens : d->tokens / d->nseq;
    int64_t piece = d->piece_len;
    if (piece == 0) {
        piece = 1024;
        const int64_t slots = 512;
        while (piece > 64 && cdiv(d->tokens, piece) * units < slots) piece /= 2;
    }
    pl->pieced = piece < each;
    pl->piece = pl->pieced ? piece : (int64_t(1) << 31);
    pl->npieces = !pl->pieced ? d->nseq : packed ? d->tokens / piece + d->nseq : d->nseq * cdiv(each, piece);
    const int64_t most = (int64_t(1) << 31) - 1;
    if (pl->npieces > most / (d->nheads * (pl->slices_q > pl->slices_s ? pl->slices_q : pl->slices_s)))
        return SSM_ERR_DIMS;
    pl->carry = pl->pieced ? up256(static_cast<size_t>(pl->npieces * d->nheads * d->dk * d->dv) * 4) : 0;
    pl->tot = up256(static_cast<size_t>(pl->npieces * d->nheads) * 4);
    pl->x = pl->tot;
    pl->dots = up256(static_cast<size_t>(pl->slices_q * d->tokens * d->nheads) * 4);
    pl->wide = d->nheads == d->kheads ? 0 : up256(static_cast<size_t>(d->tokens * d->nheads * d->dk) * 4);
    pl->bytes = 2 * pl->carry + 4 * pl->tot + 3 * pl->dots + 2 * pl->wide;
    return SSM_OK;
}

}  // namespace la
}  // namespace

bool ssm_detail::launch_linattn_grad_pass(const LinattnPasses& p, int count, bool f32, LinattnMode mode, hipStream_t s) {
    return mode == kLinDots ? la::launch_pass<kLinDots>(p, count, f32, s) : la::launch_pass<kLinCross>(p, count, f32, s);
}

extern "C" {

size_t ssm_linattn_bwd_workspace_bytes(const ssm_linattn_dims* dims) {
    la::Sizes z;
    la::GradPlan pl, dense;
    if (la::check_dims(dims, &z) != SSM_OK || la::make_grad_plan(dims, true, &pl) != SSM_OK) return 0;
    size_t n = pl.bytes;
    if (dims->tokens % dims->nseq == 0 && la::make_grad_plan(dims, false, &dense) == SSM_OK && dense.bytes > n)
        n = dense.bytes;
    return n;
}

int ssm_linattn_bwd(const void* q, const void* k, const void* v, const float* g, const int32_t* cu_seqlens,
                    const float* s0, const void* dout, const float* ds_last, const ssm_linattn_grads* grads,
                    const ssm_linattn_dims* dims, void* stream) {
    using namespace la;
    using namespace ssm_detail;
    if (!dims || !q || !k || !v || !g || !dout || !grads || !grads->dq || !grads->dk || !grads->dv) return SSM_ERR_NULL;
    if (s0 && !grads->ds0) return SSM_ERR_NULL;
    Sizes z;
    int st = check_dims(dims, &z);
    if (st != SSM_OK) return st;
    const ssm_linattn_dims& d = *dims;
    if (!cu_seqlens && d.tokens % d.nseq != 0) return SSM_ERR_DIMS;
    const int64_t lim = int64_t(1) << 40;
    if (d.nseq > lim / (d.nheads * d.dk * d.dv)) return SSM_ERR_DIMS;
    const ssm_linattn_grads& gr = *grads;
    if (misaligned(q, z.e) || misaligned(k, z.e) || misaligned(v, z.e) || misaligned(dout, z.e) || misaligned(g, 4) ||
        misaligned(cu_seqlens, 4) || misaligned(s0, 4) || misaligned(ds_last, 4) || misaligned(gr.dq, z.e) ||
        misaligned(gr.dk, z.e) || misaligned(gr.dv, z.e) || misaligned(gr.dg, 4) || misaligned(gr.ds0, 4))
        return SSM_ERR_ALIGN;
    GradPlan pl;
    st = make_grad_plan(dims, cu_seqlens != nullptr, &pl);
    if (st != SSM_OK) return st;
    if (!d.workspace || d.workspace_bytes < pl.bytes || misaligned(d.workspace, 256)) return SSM_ERR_WORKSPACE;
    const int64_t wk = d.kheads * d.dk, wv = d.nheads * d.dv;
    const size_t nstate = static_cast<size_t>(d.nseq * d.nheads * d.dk * d.dv) * 4;
    const size_t ng = static_cast<size_t>(d.nheads * (d.head_decay ? 1 : d.tokens)) * 4;
    const Area in[] = {rows_of(q, d.tokens, z.q, wk, z.e), rows_of(k, d.tokens, z.k, wk, z.e),
                       rows_of(v, d.tokens, z.v, wv, z.e), rows_of(dout, d.tokens, z.o, wv, z.e), flat(g, ng),
                       flat(cu_seqlens, static_cast<size_t>(d.nseq + 1) * 4), flat(s0, nstate), flat(ds_last, nstate)};
    const Area out[] = {flat(gr.dq, static_cast<size_t>(d.tokens * wk * z.e)), flat(gr.dk, static_cast<size_t>(d.tokens * wk * z.e)),
                        flat(gr.dv, static_cast<size_t>(d.tokens * wv * z.e)), flat(gr.dg, ng), flat(gr.ds0, nstate),
                        flat(d.workspace, pl.bytes)};
    if (clash(in, out)) return SSM_ERR_ALIAS;

    char* ws = static_cast<char*>(d.workspace);
    auto take = [&](size_t n) {
        float* r = reinterpret_cast<float*>(ws);
        ws += n;
        return r;
    };
    float* fwd = take(pl.carry);
    float* rev = take(pl.carry);
    float* totf = take(pl.tot);
    float* totr = take(pl.tot);
    float* x = take(pl.x);
    float* part = take(pl.tot);
    float* da = take(pl.dots);
    float* db = take(pl.dots);
    float* de = take(pl.dots);
    float* wq = take(pl.wide);
    float* wkk = take(pl.wide);

    const int32_t rep = static_cast<int32_t>(d.nheads / d.kheads);
    const bool f32 = d.io_dtype == SSM_F32, shared = rep > 1;
    hipStream_t s = static_cast<hipStream_t>(stream);

    LinattnPass base = {};
    base.g = g; base.cu = cu_seqlens; base.sg = d.head_decay ? 0 : d.nheads;
    base.T = d.tokens; base.L = cu_seqlens ? 0 : d.tokens / d.nseq;
    base.piece = pl.piece; base.npieces = static_cast<int32_t>(pl.npieces); base.pieced = pl.pieced;
    base.H = static_cast<int32_t>(d.nheads);
    base.nseq = static_cast<int32_t>(d.nseq); base.nslots = base.nseq;
    base.r1 = base.r2 = base.r3 = base.r4 = 1;
    base.wscale = base.oscale = 1.0f;
    base.exact = gr.dg || gr.ds0;
    base.wide = wide_rows(q, z.q, d.dk, z.e) && wide_rows(k, z.k, d.dk, z.e) && wide_rows(v, z.v, d.dv, z.e) &&
                wide_rows(dout, z.o, d.dv, z.e);

    // S in order of time: (k, v); dS against it: (q, do)
    LinattnPass sf = base;
    sf.x2 = k; sf.s2 = z.k; sf.r2 = rep; sf.x3 = v; sf.s3 = z.v;
    sf.kd = static_cast<int32_t>(d.dk); sf.vd = static_cast<int32_t>(d.dv); sf.nslices = static_cast<int32_t>(pl.slices_s);
    sf.s_in = s0; sf.carry = fwd; sf.tot = totf;
    LinattnPass sr = sf;
    sr.x2 = q; sr.s2 = z.q; sr.x3 = dout; sr.s3 = z.o; sr.s_in = ds_last; sr.carry = rev; sr.tot = totr;
    sr.reverse = 1; sr.wscale = d.scale;

    LinattnPass pq = base;   // dq = (do, v, k) from S
    pq.x1 = dout; pq.s1 = z.o; pq.x2 = v; pq.s2 = z.v; pq.x3 = k; pq.s3 = z.k; pq.r3 = rep; pq.x4 = q; pq.s4 = z.q; pq.r4 = rep;
    pq.kd = static_cast<int32_t>(d.dv); pq.vd = static_cast<int32_t>(d.dk); pq.nslices = static_cast<int32_t>(pl.slices_q);
    pq.s_in = s0; pq.st_t = 1; pq.carry = fwd; pq.oscale = d.scale;
    pq.out = shared ? static_cast<void*>(wq) : gr.dq; pq.out_f32 = shared; pq.so = d.nheads * d.dk;
    pq.dots = da; pq.cross = de; pq.pairs = pair_rows(gr.dq, pq.so, d.dk);
    pq.exact = 0;
    LinattnPass pk = pq;     // dk = (v, do, q) from dS
    pk.x1 = v; pk.s1 = z.v; pk.x2 = dout; pk.s2 = z.o; pk.x3 = q; pk.s3 = z.q; pk.x4 = k; pk.s4 = z.k;
    pk.s_in = ds_last; pk.carry = rev; pk.oscale = 1.0f; pk.wscale = d.scale; pk.reverse = 1;
    pk.out = shared ? static_cast<void*>(wkk) : gr.dk; pk.dots = db; pk.cross = nullptr;
    pk.pairs = pair_rows(gr.dk, pk.so, d.dk);
    LinattnPass pv = sr;     // dv = (k, q, do) from dS
    pv.x1 = k; pv.s1 = z.k; pv.r1 = rep; pv.out = gr.dv; pv.so = wv; pv.s_out = gr.ds0; pv.exact = gr.ds0 != nullptr; pv.pairs = pair_rows(gr.dv, wv, d.dv);

    launch_error = hipSuccess;
    if (pl.pieced) {
        launch_linattn_pass({{sf, sr}}, 2, f32, kLinStates, s);
        launch_linattn_carry({{sf, sr}}, 2, s);
    }
    if (gr.dg) {
        launch_linattn_grad_pass({{pq, pq}}, 1, f32, kLinCross, s);
        launch_linattn_grad_pass({{pk, pk}}, 1, f32, kLinDots, s);
    } else {
        launch_linattn_pass({{pq, pk}}, 2, f32, kLinFull, s);
    }
    launch_linattn_pass({{pv, pv}}, 1, f32, kLinFull, s);
    if (shared) {
        GroupArgs ga = {{wq, wkk}, {gr.dq, gr.dk}, rep, static_cast<int32_t>(d.dk), static_cast<int32_t>(d.kheads)};
        const dim3 grid(static_cast<uint32_t>(d.tokens < 65536 ? d.tokens : 65536), 2), block(kThreads);
        const bool v4 = d.dk % 4 == 0 && !misaligned(gr.dq, 4 * z.e) && !misaligned(gr.dk, 4 * z.e);
        if (f32) {
            if (v4) launch_kernel(linattn_group_kernel<float, 4>, grid, block, 0, s, base, ga);
            else launch_kernel(linattn_group_kernel<float, 1>, grid, block, 0, s, base, ga);
        } else {
            if (v4) launch_kernel(linattn_group_kernel<uint16_t, 4>, grid, block, 0, s, base, ga);
            else launch_kernel(linattn_group_kernel<uint16_t, 1>, grid, block, 0, s, base, ga);
        }
    }
    if (gr.dg) {
        GradTail t = {};
        t.p = sf; t.fwd = fwd; t.rev = rev; t.s0 = s0; t.ds0 = gr.ds0; t.a = da; t.b = db; t.e = de; t.x = x;
        t.part = part; t.dg = gr.dg; t.slices = static_cast<int32_t>(pl.slices_q); t.head_decay = d.head_decay; t.open_end = ds_last != nullptr;
        const uint32_t np = static_cast<uint32_t>(pl.npieces), hh = static_cast<uint32_t>(d.nheads);
        launch_kernel(linattn_cross_kernel, dim3(np, hh), dim3(kThreads), 0, s, t);
        launch_kernel(linattn_dg_kernel, dim3(np, (hh + 15) / 16), dim3(kDgThreads), 0, s, t);
        if (d.head_decay) launch_kernel(linattn_dg_sum_kernel, dim3(hh), dim3(kThreads), 0, s, t);
    }
    if (cu_seqlens)
        launch_kernel(linattn_zero_kernel, dim3(256), dim3(kThreads), 0, s, base,
                      shared ? nullptr : static_cast<char*>(gr.dq), wk * z.e, shared ? nullptr : static_cast<char*>(gr.dk),
                      wk * z.e, static_cast<char*>(gr.dv), wv * z.e,
                      gr.dg && !d.head_decay ? reinterpret_cast<char*>(gr.dg) : nullptr, d.nheads * 4);
    return launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
