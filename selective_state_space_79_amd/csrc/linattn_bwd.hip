// linattn_bwd.hip -- gradients of linear attention with a decay for each head.
//
// dq, dk and dv are passes of linattn.h with other rows in the three roles (dq in order of
// time from the forward's states S, dk and dv against it from the gradient dS of the state).
// States are kept at the ends of pieces of the sequences only and walked again inside.
//
// The decays' gradient.  dg_t = e^{g_t} <S_{t-1}, dS_t> is the sum of all reads that cross t.
// What token i reads in all is q_i . dq_i, what is read of token j is k_j . dk_j, so from one
// token to the next dg changes by
//   dg_{t+1} = dg_t + k_t . dk_t - q_t . dq_t
// A running sum of these carries the error of every read that came and went.  So dq and dk
// are formed to float32 here, and the sum starts afresh at each piece from
// <S, dS>, with what it misses at the next piece's start spread over the piece.  dq and dk
// per head go through float32 arrays, where the heads that share a row are added up, the row
// products taken and the outputs rounded in one more pass.
#include "linattn.h"

namespace {
namespace la {

struct GradTail {
    LinattnPass p;          // geometry
    const float* fwd;       // [pieces][H][dk dv] states that the pieces start from
    const float* rev;       // [pieces][H][dk dv] state gradients that the pieces start from, behind
    const float* s0;
    const float* ds0;
    const float* f;         // [T][H] k . dk - q . dq
    float* x;               // [pieces][H] <S, dS> at the pieces' starts
    float* part;            // [pieces][H] sums of dg (decay per head)
    float* dg;
    int32_t head_decay;
    int32_t open_end;       // a gradient arrives at the final states
};

// Rows of no sequence (before the first and behind the last): zero gradients.  Workgroup
// `first` of `count`; the widths are in bytes, multiples of 2.
struct ZeroRows {
    char* rows[4];
    int64_t width[4];
};
__device__ inline void zero_rows(const LinattnPass& p, const ZeroRows& z, int64_t first, int64_t count) {
    if (!p.cu) return;
    const int64_t lo = seq_range(p, 0).start, hi = seq_range(p, p.nseq - 1).end;
    const int64_t free = p.T - (hi > lo ? hi - lo : 0);
    for (int64_t i = first; i < free; i += count) {
        const int64_t t = i < lo ? i : p.T - free + i;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            for (int64_t e = threadIdx.x; z.rows[k] && e < z.width[k] / 2; e += kThreads)
                reinterpret_cast<uint16_t*>(z.rows[k] + t * z.width[k])[e] = 0;
    }
}
__global__ void __launch_bounds__(kThreads) linattn_zero_kernel(LinattnPass p, ZeroRows z) {
    zero_rows(p, z, blockIdx.x, gridDim.x);
}

// <S, dS> at the start of each piece, one workgroup per piece and head; and the rows of no
// sequence.  Bound by the states' bytes and one round of loads: 17 us for 16 pieces of 32 heads
// of 128 x 128 (134 MB).
__global__ void __launch_bounds__(kThreads) linattn_cross_kernel(GradTail t, ZeroRows z) {
    __shared__ double red[kWaves];
    const LinattnPass& p = t.p;
    if (blockIdx.y == 0) zero_rows(p, z, blockIdx.x, gridDim.x);
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
    double s = 0.0;
    const int64_t n4 = n % 4 == 0 && !((reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(v)) & 15) ? n : 0;
    if (u) {
#pragma unroll 4
        for (int64_t i = 4 * threadIdx.x; i < n4; i += 4 * kThreads) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(u + i), y = *reinterpret_cast<const f32x4*>(v + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fma(double(x[e]), double(y[e]), s);
        }
        for (int64_t i = n4 + threadIdx.x; i < n; i += kThreads) s = fma(double(u[i]), double(v[i]), s);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = (red[0] + red[1]) + (red[2] + red[3]);
        if (local) {   // the gradient there is that of the piece's first state: one decay on
            const float g = p.g[(sq.start + local * p.piece) * p.sg + h];
            s *= double(__builtin_amdgcn_exp2f((g < kMinDecay ? kMinDecay : g) * kLog2e));
        }
        t.x[pi * p.H + h] = float(s);
    }
}

// dg of one piece for 16 heads: 64 threads of a head take 16 tokens each at a time, their
// sum, the sums of the threads before, then the running values.  Sums in float64.  Bound by
// the latency of its rounds: 21 us for 4 x 4096 tokens of 32 heads, whose values are 4 MB.
constexpr int kDgThreads = 1024, kDgParts = kDgThreads / 16, kDgTokens = 16;

__global__ void __launch_bounds__(kDgThreads) linattn_dg_kernel(GradTail t) {
    __shared__ double sums[kDgParts][16];
    const LinattnPass& p = t.p;
    const int64_t pi = blockIdx.x;
    const int hh = threadIdx.x & 15, part = threadIdx.x >> 4, h = blockIdx.y * 16 + hh;
    const int seq = find_seq(p, pi);
    const Seq sq = seq < 0 ? Seq{0, 0} : seq_range(p, seq);
    const int64_t local = seq < 0 ? -1 : pi - piece_base(p, seq);
    const bool on = h < p.H;
    if (local < 0 || local * p.piece >= sq.end - sq.start) {
        if (t.head_decay && part == 0 && on) t.part[pi * p.H + h] = 0.0f;
        return;
    }
    const int64_t lo = sq.start + local * p.piece, hi = sq.end - lo > p.piece ? lo + p.piece : sq.end;
    const double start = on ? double(t.x[pi * p.H + h]) : 0.0;
    const float* f = t.f + h;
    // what the running sum misses at the next piece's start, or at an end that no gradient
    // reaches (there dg is zero)
    double miss = 0.0;
    if (hi < sq.end || !t.open_end) {
        double s = 0.0;
        if (on)
            for (int64_t tok = lo + part; tok < hi; tok += kDgParts) s += double(f[tok * p.H]);
        sums[part][hh] = s;
        __syncthreads();
        s = start;
#pragma unroll 4
        for (int k = 0; k < kDgParts; ++k) s += sums[k][hh];
        __syncthreads();
        if (on && hi < sq.end) {   // that piece's <S, dS> has the decay of its first token, as dg there
            s -= double(t.x[(pi + 1) * p.H + h]);
        }
        miss = -s / double(hi - lo);
    }
    double run = start, all = 0.0;
    for (int64_t base = lo; base < hi; base += kDgParts * kDgTokens) {
        const int64_t t0 = base + part * kDgTokens;
        float v[kDgTokens];
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < kDgTokens; ++k) v[k] = on && t0 + k < hi ? f[(t0 + k) * p.H] : 0.0f;
#pragma unroll
        for (int k = 0; k < kDgTokens; ++k) s += double(v[k]);
        sums[part][hh] = s;
        __syncthreads();
        double r = run;
#pragma unroll 4
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
                r += double(v[k]);
            }
    }
    if (t.head_decay) {
        sums[part][hh] = all;
        __syncthreads();
        if (part == 0 && on) {
#pragma unroll 4
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

// From dq and dk per head in float32: the sums over the heads that share a row, rounded, and
// f = k . dk - q . dq of each token and head.  LPR lanes take a row, 4 columns each (VW of
// them in one access).  Bound by the bytes of the parts: 133 us for 16384 tokens of 32 heads of
// 128 in groups of 4 (671 MB, 5.0 TB/s).
struct GroupArgs {
    const float* dq;
    const float* dk;
    const void* q;
    const void* k;
    void* out_q;
    void* out_k;
    float* f;               // null: not wanted
    int64_t sq, sk;
    int32_t rep, width, kheads;
};
template <typename IO, int VW, int LPR>
__global__ void __launch_bounds__(kThreads) linattn_group_kernel(LinattnPass p, GroupArgs a) {
    typedef float vf __attribute__((ext_vector_type(VW)));
    constexpr int M = 4 / VW;   // accesses per thread
    const int lane = threadIdx.x % LPR;
    const int64_t lo = p.cu ? seq_range(p, 0).start : 0, hi = p.cu ? seq_range(p, p.nseq - 1).end : p.T;
    const int64_t rows = p.T * a.kheads, step = int64_t(gridDim.x) * (kThreads / LPR);
    for (int64_t row = int64_t(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR; row < rows; row += step) {
        const int64_t tok = row / a.kheads;
        const int kh = int(row - tok * a.kheads);
        const bool on = tok >= lo && tok < hi;
        float q[4], k[4], sq[4], sk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = k[e] = sq[e] = sk[e] = 0.0f;
        if (on && a.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = VW == 4 ? 4 * lane + e : lane + LPR * e;
                if (c < a.width) {
                    q[e] = IOT<IO>::to_f32(static_cast<const IO*>(a.q)[tok * a.sq + int64_t(kh) * a.width + c]);
                    k[e] = IOT<IO>::to_f32(static_cast<const IO*>(a.k)[tok * a.sk + int64_t(kh) * a.width + c]);
                }
            }
        }
        const int64_t base = (tok * p.H + int64_t(kh) * a.rep) * a.width;
        if (on)
#pragma unroll 2
            for (int r = 0; r < a.rep; ++r) {
                double d = 0.0;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int c = VW == 4 ? 4 * lane : lane + LPR * m;
                    vf x = {}, y = {};
                    if (c < a.width) {
                        x = *reinterpret_cast<const vf*>(a.dq + base + int64_t(r) * a.width + c);
                        y = *reinterpret_cast<const vf*>(a.dk + base + int64_t(r) * a.width + c);
                    }
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        sq[m * VW + e] += x[e];
                        sk[m * VW + e] += y[e];
                        d = fma(double(k[m * VW + e]), double(y[e]), d);
                        d = fma(double(-q[m * VW + e]), double(x[e]), d);
                    }
                }
                if (a.f) {
#pragma unroll
                    for (int z = 1; z < LPR; z <<= 1) d += __shfl_xor(d, z);
                    if (lane == 0) a.f[tok * p.H + int64_t(kh) * a.rep + r] = float(d);
                }
            }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int c = VW == 4 ? 4 * lane : lane + LPR * m;
            if (c >= a.width) continue;
            IO x[VW], y[VW];
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                x[e] = IOT<IO>::from_f32(sq[m * VW + e]);
                y[e] = IOT<IO>::from_f32(sk[m * VW + e]);
            }
            __builtin_memcpy(static_cast<IO*>(a.out_q) + row * a.width + c, x, sizeof(x));
            __builtin_memcpy(static_cast<IO*>(a.out_k) + row * a.width + c, y, sizeof(y));
        }
    }
}

template <typename IO, int VW> void run_group(const LinattnPass& p, const GroupArgs& a, hipStream_t s) {
    const int lpr = a.width <= 64 ? 16 : a.width <= 128 ? 32 : 64;
    const int64_t blocks = cdiv(p.T * a.kheads, kThreads / lpr);
    const dim3 grid(static_cast<uint32_t>(blocks < 16384 ? blocks : 16384)), block(kThreads);
    if (lpr == 16) launch_kernel(linattn_group_kernel<IO, VW, 16>, grid, block, 0, s, p, a);
    else if (lpr == 32) launch_kernel(linattn_group_kernel<IO, VW, 32>, grid, block, 0, s, p, a);
    else launch_kernel(linattn_group_kernel<IO, VW, 64>, grid, block, 0, s, p, a);
}

// ---------------------------------------------------------------- host
struct GradPlan {
    int64_t piece, npieces;
    bool pieced;
    int64_t slices_q, slices_s;   // of passes with kd = dv, vd = dk, and with kd = dk, vd = dv
    size_t carry, tot, f, wide;   // bytes of one buffer each
    size_t bytes;
};

// Pieces of at most 1024 tokens: the error of dg's running sum grows with the piece, and the
// states of pieces this long are a sixteenth of the rows' bytes at dk = dv = 128.  A layer of 4 x
// 4096 tokens and 32 heads takes 740 us in pieces of 1024, 828 of 512, 794 of 2048.
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
    if (pl->npieces > kMostGroups / (d->nheads * (pl->slices_q > pl->slices_s ? pl->slices_q : pl->slices_s)))
        return SSM_ERR_DIMS;
    pl->carry = pl->pieced ? up256(static_cast<size_t>(pl->npieces * d->nheads * d->dk * d->dv) * 4) : 0;
    pl->tot = up256(static_cast<size_t>(pl->npieces * d->nheads) * 4);
    pl->f = up256(static_cast<size_t>(d->tokens * d->nheads) * 4);
    pl->wide = up256(static_cast<size_t>(d->tokens * d->nheads * d->dk) * 4);
    pl->bytes = 2 * pl->carry + 4 * pl->tot + pl->f + 2 * pl->wide;
    return SSM_OK;
}

}  // namespace la
}  // namespace

extern "C" {

size_t ssm_linattn_bwd_workspace_bytes(const ssm_linattn_dims* dims) {
    la::Sizes z;
    la::GradPlan pl;
    if (la::check_dims(dims, &z) != SSM_OK) return 0;
    size_t n = 0;
    if (la::make_grad_plan(dims, true, &pl) == SSM_OK) n = pl.bytes;
    if (dims->tokens % dims->nseq == 0 && la::make_grad_plan(dims, false, &pl) == SSM_OK && pl.bytes > n) n = pl.bytes;
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
    float* x = take(pl.tot);
    float* part = take(pl.tot);
    float* f = take(pl.f);
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
    base.r1 = base.r2 = base.r3 = 1;
    base.wscale = base.oscale = 1.0f;
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

    // per head in float32 where dg is formed from them or heads share a row, else at once
    const bool apart = shared || gr.dg;
    LinattnPass pq = base;   // dq = (do, v, k) from S
    pq.x1 = dout; pq.s1 = z.o; pq.x2 = v; pq.s2 = z.v; pq.x3 = k; pq.s3 = z.k; pq.r3 = rep;
    pq.kd = static_cast<int32_t>(d.dv); pq.vd = static_cast<int32_t>(d.dk); pq.nslices = static_cast<int32_t>(pl.slices_q);
    pq.s_in = s0; pq.st_t = 1; pq.carry = fwd; pq.oscale = d.scale;
    pq.out = apart ? static_cast<void*>(wq) : gr.dq; pq.out_f32 = apart; pq.so = d.nheads * d.dk;
    pq.pairs = !apart && pair_rows(gr.dq, pq.so, d.dk);
    LinattnPass pk = pq;     // dk = (v, do, q) from dS
    pk.x1 = v; pk.s1 = z.v; pk.x2 = dout; pk.s2 = z.o; pk.x3 = q; pk.s3 = z.q;
    pk.s_in = ds_last; pk.carry = rev; pk.oscale = 1.0f; pk.wscale = d.scale; pk.reverse = 1;
    pk.out = apart ? static_cast<void*>(wkk) : gr.dk; pk.pairs = !apart && pair_rows(gr.dk, pk.so, d.dk);
    LinattnPass pv = sr;     // dv = (k, q, do) from dS
    pv.x1 = k; pv.s1 = z.k; pv.r1 = rep; pv.out = gr.dv; pv.so = wv; pv.s_out = gr.ds0; pv.pairs = pair_rows(gr.dv, wv, d.dv);

    launch_error = hipSuccess;
    if (pl.pieced) {
        launch_linattn_pass({{sf, sr}}, 2, f32, kLinStates, s);
        launch_linattn_carry({{sf, sr}}, 2, s);
    }
    launch_linattn_pass({{pq, pk}}, 2, f32, kLinFull, s);
    launch_linattn_pass({{pv, pv}}, 1, f32, kLinFull, s);
    if (apart) {
        const GroupArgs ga = {wq, wkk, q, k, gr.dq, gr.dk, gr.dg ? f : nullptr, z.q, z.k, rep, static_cast<int32_t>(d.dk),
                              static_cast<int32_t>(d.kheads)};
        const bool v4 = d.dk % 4 == 0 && !misaligned(gr.dq, 4 * z.e) && !misaligned(gr.dk, 4 * z.e);
        if (f32) {
            if (v4) run_group<float, 4>(base, ga, s);
            else run_group<float, 1>(base, ga, s);
        } else {
            if (v4) run_group<uint16_t, 4>(base, ga, s);
            else run_group<uint16_t, 1>(base, ga, s);
        }
    }
    const ZeroRows zero = {{apart ? nullptr : static_cast<char*>(gr.dq), apart ? nullptr : static_cast<char*>(gr.dk),
                            static_cast<char*>(gr.dv),
                            gr.dg && !d.head_decay ? reinterpret_cast<char*>(gr.dg) : nullptr},
                           {wk * z.e, wk * z.e, wv * z.e, d.nheads * 4}};
    if (gr.dg) {
        GradTail t = {};
        t.p = sf; t.fwd = fwd; t.rev = rev; t.s0 = s0; t.ds0 = gr.ds0; t.f = f; t.x = x;
        t.part = part; t.dg = gr.dg; t.head_decay = d.head_decay; t.open_end = ds_last != nullptr;
        const uint32_t np = static_cast<uint32_t>(pl.npieces), hh = static_cast<uint32_t>(d.nheads);
        launch_kernel(linattn_cross_kernel, dim3(np, hh), dim3(kThreads), 0, s, t, zero);
        launch_kernel(linattn_dg_kernel, dim3(np, (hh + 15) / 16), dim3(kDgThreads), 0, s, t);
        if (d.head_decay) launch_kernel(linattn_dg_sum_kernel, dim3(hh), dim3(kThreads), 0, s, t);
    }
    if (!gr.dg && cu_seqlens) launch_kernel(linattn_zero_kernel, dim3(256), dim3(kThreads), 0, s, base, zero);
    return launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
