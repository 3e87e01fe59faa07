// linattn_fwd.hip -- linear attention with a decay for each head: the forward over packed
// sequences (the chunked pass of linattn.h, cut into pieces along the tokens when there are
// few heads and sequences) and the single-token step.
#include "linattn.h"

namespace {
namespace la {

// ---------------------------------------------------------------- pieces' starting states
// Walks the pieces of one sequence and head: each piece's own end state (from a zero start)
// is replaced by the state it starts from.  Bound by the states' bytes, read and written once:
// 17 us for 21 pieces of 32 heads of 128 x 128, 5.1 TB/s; 4 values per thread.
template <int VW> __global__ void __launch_bounds__(kThreads) linattn_carry_kernel(ssm_detail::LinattnPasses q) {
    const LinattnPass& p = q.p[blockIdx.y / q.p[0].H];
    typedef float vf __attribute__((ext_vector_type(VW)));
    const int64_t ssz = int64_t(p.kd) * p.vd;
    const int64_t e = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * VW;
    const int h = blockIdx.y % p.H, seq = blockIdx.z;
    const int slot = find_slot(p.slots, p.nslots, seq);
    if (slot < 0 || e >= ssz) return;
    const Seq sq = seq_range(p, seq);
    const int64_t base = piece_base(p, seq);
    int64_t n = (sq.end - sq.start + p.piece - 1) / p.piece;
    if (n < 2) return;   // a single piece starts from the user's state
    if (base + n > p.npieces) n = p.npieces - base;
    vf s = {};
    if (p.s_in) s = *reinterpret_cast<const vf*>(p.s_in + (int64_t(slot) * p.H + h) * ssz + e);
    // the pieces' own states are asked for eight ahead: few heads keep few loads under way
    // (129 pieces of 2 heads of 104 x 16 62 us four ahead, 31 so)
    constexpr int A = 8;
    const auto at = [&](int64_t m) { return ((base + (p.reverse ? n - 1 - m : m)) * p.H + h); };
    vf own[A];
    float t[A];
    const auto ask = [&](int k, int64_t m) {
        if (m + 1 < n) {
            own[k] = *reinterpret_cast<const vf*>(p.carry + at(m) * ssz + e);
            t[k] = p.tot[at(m)];
        }
    };
#pragma unroll
    for (int k = 0; k < A; ++k) ask(k, k);
    for (int64_t m0 = 0; m0 < n; m0 += A) {
#pragma unroll
        for (int k = 0; k < A; ++k) {
            const int64_t m = m0 + k;
            if (m < n) *reinterpret_cast<vf*>(p.carry + at(m) * ssz + e) = s;
            if (m + 1 < n) s = t[k] * s + own[k];
            ask(k, m + A);
        }
    }
}

// ---------------------------------------------------------------- single tokens
struct StepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const int32_t* slots;
    float* states;
    void* o;
    int64_t sq, sk, sv, so, sg;
    int32_t H, rep, dk, dv, nslots, nslices, tpr_log2;
    float scale;
};

// One workgroup per sequence, head and slice of the state's columns; a row of the slice is
// read by 2^tpr_log2 threads of 4 columns each, the rows of the state go round over the
// threads.  Everything is one pass over the state, its loads in flight before q and k are
// looked at; the read-out is summed over the row groups in LDS in a fixed order.  Bound by
// the states' bytes: 256 sequences of 64 heads of 128 x 64 in 213 us, 5.04 TB/s (a plain copy
// 5.15); one sequence of 32 heads of 128 x 128 takes 5.6 us on the card and 9.6 with its launch.
//
// 16 bytes are read and written at any alignment as far as the row goes (29 sequences of 32
// heads of 125 x 135 50 us by single values, 36 so).
template <typename IO>
__global__ void __launch_bounds__(kThreads) linattn_step_kernel(StepArgs p) {
    constexpr int VW = 4;
    typedef f32x4 vf;
    constexpr int R = 8;   // rows in flight per thread
    __shared__ float sq[SSM_LINATTN_MAX_DIM], sk[SSM_LINATTN_MAX_DIM];
    __shared__ float red[kThreads * VW];
    __shared__ int dups[kWaves];
    const int tid = threadIdx.x;
    const int per = p.H * p.nslices;
    const int b = blockIdx.x / per, at = blockIdx.x % per, h = at / p.nslices, slice = at % p.nslices;
    int slot = b;
    bool dup = false;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.nslots) return;
        for (int i = tid; i < b; i += kThreads) dup = dup || p.slots[i] == slot;
    }
    const int tpr = 1 << p.tpr_log2, rows = kThreads >> p.tpr_log2;
    const int r0 = tid >> p.tpr_log2, col = (slice * tpr + (tid & (tpr - 1))) * VW;
    const bool on = col < p.dv, whole = col + VW <= p.dv;
    const auto read = [&](const float* q) {
        vf x = {};
        if (whole) {
            __builtin_memcpy(&x, q, sizeof(x));
        } else {
#pragma unroll
            for (int e = 0; e < VW; ++e)
                if (col + e < p.dv) x[e] = q[e];
        }
        return x;
    };
    const auto write = [&](float* q, const vf& x) {
        if (whole) {
            __builtin_memcpy(q, &x, sizeof(x));
        } else {
#pragma unroll
            for (int e = 0; e < VW; ++e)
                if (col + e < p.dv) q[e] = x[e];
        }
    };
    float* S = p.states + (int64_t(slot) * p.H + h) * p.dk * p.dv + col;
    vf s[R];
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const int r = r0 + n * rows;
        if (on && r < p.dk) s[n] = read(S + int64_t(r) * p.dv);
    }
    const IO* q = static_cast<const IO*>(p.q) + b * p.sq + int64_t(h / p.rep) * p.dk;
    const IO* k = static_cast<const IO*>(p.k) + b * p.sk + int64_t(h / p.rep) * p.dk;
    if (tid < p.dk) {
        sq[tid] = IOT<IO>::to_f32(q[tid]) * p.scale;
        sk[tid] = IOT<IO>::to_f32(k[tid]);
    }
    if (p.slots) {
        const bool any = __ballot(dup) != 0;
        if ((tid & 63) == 0) dups[tid >> 6] = any;
    }
    vf v = {};
    if (on) {
        const IO* vr = static_cast<const IO*>(p.v) + b * p.sv + int64_t(h) * p.dv + col;
#pragma unroll
        for (int e = 0; e < VW; ++e) v[e] = whole || col + e < p.dv ? IOT<IO>::to_f32(vr[e]) : 0.0f;
    }
    float g = p.g[b * p.sg + h];
    g = g < kMinDecay ? kMinDecay : g;
    const float a = __builtin_amdgcn_exp2f(g * kLog2e);
    __syncthreads();
    if (p.slots && (dups[0] | dups[1] | dups[2] | dups[3])) return;
    vf o = {};
    for (int base = 0; base < p.dk; base += R * rows) {
#pragma unroll
        for (int n = 0; n < R; ++n) {
            const int r = base + r0 + n * rows;
            if (!(on && r < p.dk)) continue;
            if (base > 0) s[n] = read(S + int64_t(r) * p.dv);
            s[n] = a * s[n] + sk[r] * v;
            o += sq[r] * s[n];
            write(S + int64_t(r) * p.dv, s[n]);
        }
    }
    *reinterpret_cast<vf*>(&red[tid * VW]) = o;
    __syncthreads();
    // column c of the slice: thread c sums it over the row groups
    const int w = tpr * VW;
    for (int c = tid; c < w; c += kThreads) {
        const int cc = slice * w + c;
        if (cc >= p.dv) break;
        float x = 0.0f;
        for (int r = 0; r < rows; ++r) x += red[r * w + c];
        static_cast<IO*>(p.o)[b * p.so + int64_t(h) * p.dv + cc] = IOT<IO>::from_f32(x);
    }
}

// ---------------------------------------------------------------- host: plans
struct Plan {
    int64_t piece, npieces;
    bool pieced;
    size_t carry, tot;   // bytes
};

// Pieces along the tokens.  A workgroup walks its piece chunk by chunk, 7.2 us for 64 tokens
// of a 128 x 128 head alone on its CU and 10.4 us for two side by side, so work is cut into the
// 512 workgroups that the card holds at once; more, smaller pieces only add states to carry.
// Measured on the same inputs again and again, us, the rule's own piece first: 131072 tokens of
// 16 heads 836 in pieces of 4096, 875 of 2048, 955 of 8192; 8 ragged prompts of 8192 tokens in
// all, 32 heads, 160 in pieces of 512, 193 of 320, 176 of 576, 158 of 704, 175 of 1024, 303 of
// 2048; 2 x 8192 tokens of 64 shared heads of 64 227 in pieces of 1024, 283 of 512, 355 of 2048.
// Cutting costs two launches and a second pass over keys and values: sequences of up to 256
// tokens stay whole.  The lengths of packed sequences are not known here: they are taken for one
// sequence of all tokens, so short ones get the two launches for nothing (64 prompts of 128
// tokens and 32 heads of 128 x 128 131 us and a workspace of 168 MB that stays unused).
inline int64_t choose_piece(const ssm_linattn_dims* d, int64_t units, int64_t each) {
    const int64_t want = 512 / units;   // pieces of the whole call
    if (want < 2 || each <= 256) return 0;
    const int64_t piece = cdiv(cdiv(d->tokens, want), 64) * 64;
    return piece < each ? piece : 0;
}

inline int make_plan(const ssm_linattn_dims* d, bool packed, Plan* pl) {
    const int64_t slices = cdiv(d->dv, ssm_detail::linattn_slice(d->dv));
    const bool pairs = ssm_detail::linattn_shape(d->dv, d->nheads / d->kheads % 2 == 0) == ssm_detail::kTwoHeads;
    const int64_t units = d->nheads * slices;
    const int64_t each = packed ? d->tokens : d->tokens / d->nseq;
    int64_t piece = d->piece_len;
    if (piece == 0) piece = choose_piece(d, pairs ? units / 2 : units, each);
    pl->pieced = piece > 0 && piece < each;
    pl->piece = pl->pieced ? piece : (int64_t(1) << 31);
    pl->npieces = !pl->pieced ? d->nseq : packed ? d->tokens / piece + d->nseq : d->nseq * cdiv(each, piece);
    if (pl->npieces > kMostGroups / units) return SSM_ERR_DIMS;
    pl->carry = pl->pieced ? up256(static_cast<size_t>(pl->npieces * d->nheads * d->dk * d->dv) * 4) : 0;
    pl->tot = pl->pieced ? up256(static_cast<size_t>(pl->npieces * d->nheads) * 4) : 0;
    return SSM_OK;
}

}  // namespace la
}  // namespace

void ssm_detail::launch_linattn_pass(const LinattnPasses& p, int count, bool f32, LinattnMode mode, hipStream_t s) {
    if (mode == kLinStates) la::launch_pass<kLinStates>(p, count, f32, s);
    else la::launch_pass<kLinFull>(p, count, f32, s);
}

void ssm_detail::launch_linattn_carry(const LinattnPasses& q, int count, hipStream_t s) {
    const LinattnPass& p = q.p[0];
    const int64_t ssz = int64_t(p.kd) * p.vd;
    const bool v4 = ssz % 4 == 0 && !misaligned(p.s_in, 16) && !misaligned(q.p[1].s_in, 16);
    const dim3 grid(static_cast<uint32_t>(cdiv(ssz, la::kThreads * (v4 ? 4 : 1))), p.H * count, p.nseq);
    if (v4)
        launch_kernel(la::linattn_carry_kernel<4>, grid, dim3(la::kThreads), 0, s, q);
    else
        launch_kernel(la::linattn_carry_kernel<1>, grid, dim3(la::kThreads), 0, s, q);
}

extern "C" {

size_t ssm_linattn_fwd_workspace_bytes(const ssm_linattn_dims* dims) {
    la::Sizes z;
    la::Plan pl;
    if (la::check_dims(dims, &z) != SSM_OK) return 0;
    // with and without cu_seqlens: the larger of the two
    size_t n = 0;
    if (la::make_plan(dims, true, &pl) == SSM_OK) n = pl.carry + pl.tot;
    if (dims->tokens % dims->nseq == 0 && la::make_plan(dims, false, &pl) == SSM_OK && pl.carry + pl.tot > n)
        n = pl.carry + pl.tot;
    return n;
}

int ssm_linattn_fwd(const void* q, const void* k, const void* v, const float* g, const int32_t* cu_seqlens,
                    const int32_t* slots, const float* s0, void* o, float* s_last, const ssm_linattn_dims* dims,
                    void* stream) {
    using namespace la;
    if (!dims || !q || !k || !v || !g || !o) return SSM_ERR_NULL;
    if (slots && !s0 && !s_last) return SSM_ERR_NULL;
    Sizes z;
    int st = check_dims(dims, &z);
    if (st != SSM_OK) return st;
    const ssm_linattn_dims& d = *dims;
    if (!cu_seqlens && d.tokens % d.nseq != 0) return SSM_ERR_DIMS;
    const bool states = s0 || s_last;
    const int64_t lim = int64_t(1) << 40;
    if (states && (d.nslots < 1 || d.nslots > (int64_t(1) << 31) - 1 || (!slots && d.nslots < d.nseq) ||
                   d.nslots > lim / (d.nheads * d.dk * d.dv)))
        return SSM_ERR_DIMS;
    if (misaligned(q, z.e) || misaligned(k, z.e) || misaligned(v, z.e) || misaligned(o, z.e) || misaligned(g, 4) ||
        misaligned(cu_seqlens, 4) || misaligned(slots, 4) || misaligned(s0, 4) || misaligned(s_last, 4))
        return SSM_ERR_ALIGN;
    Plan pl;
    st = make_plan(dims, cu_seqlens != nullptr, &pl);
    if (st != SSM_OK) return st;
    const size_t need = pl.carry + pl.tot;
    if (need && (!d.workspace || d.workspace_bytes < need || misaligned(d.workspace, 256))) return SSM_ERR_WORKSPACE;
    const size_t nstate = states ? static_cast<size_t>(d.nslots * d.nheads * d.dk * d.dv) * 4 : 0;
    const int64_t wk = d.kheads * d.dk, wv = d.nheads * d.dv;
    const Area in[] = {rows_of(q, d.tokens, z.q, wk, z.e), rows_of(k, d.tokens, z.k, wk, z.e),
                       rows_of(v, d.tokens, z.v, wv, z.e),
                       flat(g, static_cast<size_t>(d.nheads * (d.head_decay ? 1 : d.tokens)) * 4),
                       flat(cu_seqlens, static_cast<size_t>(d.nseq + 1) * 4), flat(slots, static_cast<size_t>(d.nseq) * 4),
                       flat(s0 == s_last ? nullptr : s0, nstate)};
    const Area out[] = {rows_of(o, d.tokens, z.o, wv, z.e), flat(s_last, nstate), flat(need ? d.workspace : nullptr, need)};
    if (clash(in, out)) return SSM_ERR_ALIAS;

    ssm_detail::LinattnPass p = {};
    p.x1 = q; p.x2 = k; p.x3 = v; p.out = o; p.g = g; p.cu = cu_seqlens; p.slots = slots; p.s_in = s0; p.s_out = s_last;
    p.s1 = z.q; p.s2 = z.k; p.s3 = z.v; p.so = z.o; p.sg = d.head_decay ? 0 : d.nheads;
    p.T = d.tokens; p.L = cu_seqlens ? 0 : d.tokens / d.nseq;
    p.piece = pl.piece;
    p.r1 = p.r2 = static_cast<int32_t>(d.nheads / d.kheads);
    p.r3 = 1;
    p.H = static_cast<int32_t>(d.nheads); p.kd = static_cast<int32_t>(d.dk); p.vd = static_cast<int32_t>(d.dv);
    p.nslices = static_cast<int32_t>(cdiv(d.dv, ssm_detail::linattn_slice(d.dv)));
    p.nseq = static_cast<int32_t>(d.nseq); p.nslots = static_cast<int32_t>(states ? d.nslots : d.nseq);
    p.npieces = static_cast<int32_t>(pl.npieces); p.pieced = pl.pieced;
    p.wide = wide_rows(q, z.q, d.dk, z.e) && wide_rows(k, z.k, d.dk, z.e) && wide_rows(v, z.v, d.dv, z.e);
    p.pairs = pair_rows(o, z.o, d.dv);
    p.wscale = 1.0f; p.oscale = d.scale;
    const bool f32 = d.io_dtype == SSM_F32;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ssm_detail::launch_error = hipSuccess;
    if (pl.pieced) {
        p.carry = static_cast<float*>(d.workspace);
        p.tot = reinterpret_cast<float*>(static_cast<char*>(d.workspace) + pl.carry);
        ssm_detail::launch_linattn_pass({{p, p}}, 1, f32, ssm_detail::kLinStates, s);
        ssm_detail::launch_linattn_carry({{p, p}}, 1, s);
    }
    ssm_detail::launch_linattn_pass({{p, p}}, 1, f32, ssm_detail::kLinFull, s);
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_linattn_step(const void* q, const void* k, const void* v, const float* g, const int32_t* slots, float* states,
                     void* o, const ssm_linattn_dims* dims, void* stream) {
    using namespace la;
    if (!dims || !q || !k || !v || !g || !states || !o) return SSM_ERR_NULL;
    Sizes z;
    const int st = check_dims(dims, &z);
    if (st != SSM_OK) return st;
    const ssm_linattn_dims& d = *dims;
    if (d.tokens != d.nseq) return SSM_ERR_DIMS;
    if (d.nslots < 1 || d.nslots > (int64_t(1) << 31) - 1 || (!slots && d.nslots < d.nseq) ||
        d.nslots > (int64_t(1) << 40) / (d.nheads * d.dk * d.dv))
        return SSM_ERR_DIMS;
    if (misaligned(q, z.e) || misaligned(k, z.e) || misaligned(v, z.e) || misaligned(o, z.e) || misaligned(g, 4) ||
        misaligned(slots, 4) || misaligned(states, 4))
        return SSM_ERR_ALIGN;
    const size_t nstate = static_cast<size_t>(d.nslots * d.nheads * d.dk * d.dv) * 4;
    const int64_t wk = d.kheads * d.dk, wv = d.nheads * d.dv;
    const Area in[] = {rows_of(q, d.tokens, z.q, wk, z.e), rows_of(k, d.tokens, z.k, wk, z.e),
                       rows_of(v, d.tokens, z.v, wv, z.e),
                       flat(g, static_cast<size_t>(d.nheads * (d.head_decay ? 1 : d.tokens)) * 4),
                       flat(slots, static_cast<size_t>(d.nseq) * 4)};
    const Area out[] = {rows_of(o, d.tokens, z.o, wv, z.e), flat(states, nstate)};
    if (clash(in, out)) return SSM_ERR_ALIAS;

    StepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.slots = slots; a.states = states; a.o = o;
    a.sq = z.q; a.sk = z.k; a.sv = z.v; a.so = z.o; a.sg = d.head_decay ? 0 : d.nheads;
    a.H = static_cast<int32_t>(d.nheads); a.rep = static_cast<int32_t>(d.nheads / d.kheads);
    a.dk = static_cast<int32_t>(d.dk); a.dv = static_cast<int32_t>(d.dv); a.nslots = static_cast<int32_t>(d.nslots);
    a.scale = d.scale;
    constexpr int vw = 4;
    // as many columns a workgroup as the state has, halved while the card has room for more
    // workgroups and a row of the slice is still 64 bytes
    int lg = 0;
    while ((vw << lg) < d.dv && lg < 8) ++lg;
    while ((vw << lg) > 16 && cdiv(d.dv, vw << lg) * d.nheads * d.nseq < 512) --lg;
    a.tpr_log2 = lg;
    a.nslices = static_cast<int32_t>(cdiv(d.dv, vw << lg));
    const int64_t blocks = d.nseq * d.nheads * a.nslices;
    if (blocks > 2 * kMostGroups) return SSM_ERR_DIMS;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kThreads);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ssm_detail::launch_error = hipSuccess;
    if (d.io_dtype == SSM_BF16) launch_kernel(linattn_step_kernel<uint16_t>, grid, block, 0, s, a);
    else launch_kernel(linattn_step_kernel<float>, grid, block, 0, s, a);
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
