// norms.hip -- norms around a block, forward and backward: the gated RMS norm behind a mixer,
// the residual addition between two blocks with the RMS norms on both sides of it, and the layer
// norm.
//
// Every kernel reads its rows once into registers, 8 neighbouring values per thread, and
// is bound by those bytes.  A row (or group) belongs to TPG threads: 8 .. 64 lanes of a
// wave with several groups side by side, or 2 .. 16 waves that exchange one number per
// reduction through LDS.  One vector per thread (two for rows over 8192) keeps registers
// few and leaves the loads in flight to the number of waves.
//
// The gradients hold the next row's values while one is worked on, up to 8192 columns (above,
// the registers for it would lie in scratch memory: 358 us against 156 for the gate norm of
// 4096 bf16 rows of 16384), and the sums for the weights' gradients in registers over a
// workgroup's rows; the workgroups' partial sums are then added in a fixed order.
//
// Measured on 16384 bf16 rows, the bytes of rows that are read and written (a plain copy runs at
// 5.15 TB/s): gated forward of 64 groups of 64 in 75 us (5.4 TB/s), 1536 wide 30 us (5.1), 1535
// wide 37 us (4.0); its gradient at 1536 columns 57 us on the same inputs again and again (4.4
// TB/s) and 69 on others each time (3.6; 54 us of it the rows, 5 the partial sums), at 4096 147 us
// (4.6); residual norm 4096 wide 97 us (5.6 TB/s), with a float32 residual and both weights 165 us
// (4.9); its gradient at 2048 columns with a float32 residual and both weights 130 us (4.6), at
// 4096 with a bf16 one without weights 136 us (4.9), 8192 rows of 8192 with both weights 183 us
// (4.4), 4096 rows of 16384 452 us (1.8, bound by registers).
#include "rows.h"

namespace {
namespace nrm {

constexpr int kVW = 8;

struct V8 {
    float e[8];
};

// 8 values at column col of a row with w columns, as they lie in memory (so that a row can be
// asked for while another is worked on); out of range reads as 0.
template <typename IO> struct Raw8 {
    uint4 u[sizeof(IO) / 2];
    __device__ inline void load(const IO* row, int col, int w, bool on, bool vec) {
#pragma unroll
        for (int k = 0; k < int(sizeof(IO) / 2); ++k) u[k] = make_uint4(0, 0, 0, 0);
        if (!on || col >= w) return;
        if (vec) {
#pragma unroll
            for (int k = 0; k < int(sizeof(IO) / 2); ++k) u[k] = reinterpret_cast<const uint4*>(row + col)[k];
        } else if (col + 8 <= w) {
            __builtin_memcpy(u, row + col, sizeof(u));   // 16 bytes at any address, as far as the row goes
        } else {
            IO raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[i] = col + i < w ? row[col + i] : IO(0);
            __builtin_memcpy(u, raw, sizeof(raw));
        }
    }
    __device__ inline V8 values() const {
        IO raw[8];
        __builtin_memcpy(raw, u, sizeof(raw));
        V8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v.e[i] = IOT<IO>::to_f32(raw[i]);
        return v;
    }
};
template <typename IO> __device__ inline V8 load8(const IO* row, int col, int w, bool on, bool vec) {
    Raw8<IO> r;
    r.load(row, col, w, on, vec);
    return r.values();
}

template <typename IO> __device__ inline void store8(IO* row, int col, int w, bool on, bool vec, const V8& v) {
    if (!on || col >= w) return;
    IO raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = IOT<IO>::from_f32(v.e[i]);
    if (vec) {
#pragma unroll
        for (int k = 0; k < int(sizeof(raw) / 16); ++k) {
            uint4 u;
            __builtin_memcpy(&u, reinterpret_cast<const char*>(raw) + 16 * k, 16);
            reinterpret_cast<uint4*>(row + col)[k] = u;
        }
    } else if (col + 8 <= w) {
        __builtin_memcpy(row + col, raw, sizeof(raw));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < w) row[col + i] = raw[i];
    }
}

// A row of float32 weights in LDS, each thread's 8 values in two planes of 4, so that a
// wave's 16-byte reads lie side by side.  In the backward kernels the weights would take as
// many registers as a row.
template <int T> struct LdsWeights {
    float* at;   // [2][T][4]
    __device__ inline void put(const V8& v, int t) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) at[(e >> 2) * 4 * T + 4 * t + (e & 3)] = v.e[e];
    }
    __device__ inline V8 get(int t) const {
        V8 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 u = *reinterpret_cast<const float4*>(at + h * 4 * T + 4 * t);
            v.e[4 * h] = u.x;
            v.e[4 * h + 1] = u.y;
            v.e[4 * h + 2] = u.z;
            v.e[4 * h + 3] = u.w;
        }
        return v;
    }
};

__device__ inline V8 loadw(const float* w, int col, int n) { return load8<float>(w, col, n, w != nullptr, false); }

template <int TPG> constexpr int block_threads() { return TPG < 256 ? 256 : TPG; }

// v plus its value in the lane that a DPP control names.
template <int CTRL> __device__ inline float plus_dpp(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// The sum over each N neighbouring lanes (N a power of two up to 64), the same in all of
// them: each step's partner holds the other half's sum in every lane.
template <int N> __device__ inline float lanes_sum(float v) {
    if (N > 1) v = plus_dpp<0xB1>(v);    // lane ^ 1
    if (N > 2) v = plus_dpp<0x4E>(v);    // lane ^ 2
    if (N > 4) v = plus_dpp<0x141>(v);   // mirrored in 8
    if (N > 8) v = plus_dpp<0x140>(v);   // mirrored in 16
    if (N > 16) v += __shfl_xor(v, 16);
    if (N > 32) v += __shfl_xor(v, 32);
    return v;
}

// The same in float64, a word at a time.
template <int CTRL> __device__ inline double plus_dpp(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf, 0xf, true);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf, 0xf, true);
    return v + __hiloint2double(hi, lo);
}
template <int N> __device__ inline double lanes_sum(double v) {
    if (N > 1) v = plus_dpp<0xB1>(v);
    if (N > 2) v = plus_dpp<0x4E>(v);
    if (N > 4) v = plus_dpp<0x141>(v);
    if (N > 8) v = plus_dpp<0x140>(v);
    if (N > 16) v += __shfl_xor(v, 16);
    if (N > 32) v += __shfl_xor(v, 32);
    return v;
}

// Sums over the TPG threads of a group, one or several at once.  With more than one wave, a
// slot of LDS per wave; two sets are used in turn, so one barrier is enough.  The barrier
// waits for LDS only: rows asked for ahead stay under way.
template <int TPG> struct Summer {
    static constexpr int kWaves = block_threads<TPG>() / 64, kMost = 3;
    static constexpr int kFloats = 2 * kWaves * kMost;
    float* red;   // [2][kWaves][kMost]
    int turn = 0;
    template <int N> __device__ inline void all(float (&v)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = lanes_sum<(TPG < 64 ? TPG : 64)>(v[n]);
        if constexpr (TPG > 64) {
            constexpr int per = TPG / 64;
            const int wave = threadIdx.x >> 6;
            float* r = red + turn * kWaves * kMost;
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int n = 0; n < N; ++n) r[wave * kMost + n] = v[n];
            }
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            // a wave's number in each lane: read one by one they would take 48 registers
            const int from = wave / per * per + (threadIdx.x & (per - 1));
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = lanes_sum<per>(r[from * kMost + n]);
        }
    }
    __device__ inline float operator()(float v) {
        float x[1] = {v};
        all(x);
        return x[0];
    }
    __device__ inline double operator()(double v) {
        v = lanes_sum<(TPG < 64 ? TPG : 64)>(v);
        if constexpr (TPG > 64) {
            constexpr int per = TPG / 64;
            const int wave = threadIdx.x >> 6;
            float* r = red + turn * kWaves * kMost;
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
                r[wave * kMost] = __int_as_float(__double2loint(v));
                r[wave * kMost + 1] = __int_as_float(__double2hiint(v));
            }
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const int from = (wave / per * per + (threadIdx.x & (per - 1))) * kMost;
            v = lanes_sum<per>(__hiloint2double(__float_as_int(r[from + 1]), __float_as_int(r[from])));
        }
        return v;
    }
};

// A group's place: slots of TPG threads are numbered over the grid, group = slot % ngroups,
// rows go round over slot / ngroups, so a slot always has the same group and can keep its
// sums over rows in registers.
struct Place {
    int64_t row, step;
    int group;
    bool on;
};
template <int TPG> __device__ inline Place place(int ngroups) {
    constexpr int spb = block_threads<TPG>() / TPG;
    int own = threadIdx.x / TPG;
    if (TPG >= 64) own = __builtin_amdgcn_readfirstlane(own);   // rows' addresses on the scalar unit
    const int64_t slot = int64_t(blockIdx.x) * spb + own, slots = int64_t(gridDim.x) * spb;
    Place p;
    p.step = slots / ngroups;
    p.row = slot / ngroups;
    p.group = int(slot % ngroups);
    p.on = p.row < p.step;
    return p;
}

struct GatedArgs {
    const void* x;
    const void* z;
    const float* w;
    const void* dy;
    void* y;        // dx in the backward
    void* dz;
    float* part;    // [row lanes][ngroups * group], or [blocks][group] when shared
    int64_t rows, sx, sz, sy;
    int32_t ngroups, n, shared, vec;
    float eps, inv_n;
};

template <typename IO, int TPG, int V, bool FIRST>
__global__ void __launch_bounds__(block_threads<TPG>()) gated_norm_fwd_kernel(GatedArgs p) {
    __shared__ float red[Summer<TPG>::kFloats];
    Summer<TPG> sum{red};
    const int lane = threadIdx.x % TPG;
    const Place at = place<TPG>(p.ngroups);
    const int64_t off = int64_t(at.group) * p.n;
    V8 w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = loadw(p.w + (p.shared ? 0 : off), 8 * (lane + TPG * i), p.n);
    const int64_t loops = (p.rows + at.step - 1) / at.step;   // the same for every thread of the grid
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = at.row + l * at.step;
        const bool on = at.on && row < p.rows;
        const IO* xr = static_cast<const IO*>(p.x) + row * p.sx + off;
        const IO* zr = static_cast<const IO*>(p.z) + row * p.sz + off;
        V8 x[V], a[V];
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            x[i] = load8<IO>(xr, col, p.n, on, p.vec);
            if (p.z) a[i] = load8<IO>(zr, col, p.n, on, p.vec);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[i].e[e] = p.z ? silu_f32(a[i].e[e]) : 1.0f;
                if (FIRST) x[i].e[e] *= a[i].e[e];
                q = fmaf(x[i].e[e], x[i].e[e], q);
            }
        }
        const float rs = __builtin_amdgcn_rsqf(fmaf(sum(q), p.inv_n, p.eps));
        IO* yr = static_cast<IO*>(p.y) + row * p.sy + off;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            V8 y;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y.e[e] = x[i].e[e] * rs * w[i].e[e];
                if (!FIRST) y.e[e] *= a[i].e[e];
            }
            store8<IO>(yr, 8 * (lane + TPG * i), p.n, on, p.vec, y);
        }
    }
}

// Sums a workgroup's slots that share a weight (in slot order) and writes the partial sums.
template <int TPG, int V>
__device__ inline void store_part(float* part, const V8 (&s)[V], const Place& at, int ngroups, int n, bool shared,
                                  float* lds) {
    const int lane = threadIdx.x % TPG;
    constexpr int spb = block_threads<TPG>() / TPG;
    if (!shared) {
        if (!at.on) return;
        float* o = part + (at.row * ngroups + at.group) * int64_t(n);
#pragma unroll
        for (int i = 0; i < V; ++i) store8<float>(o, 8 * (lane + TPG * i), n, true, false, s[i]);
        return;
    }
    float* o = part + int64_t(blockIdx.x) * n;
    if constexpr (spb == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) store8<float>(o, 8 * (lane + TPG * i), n, true, false, s[i]);
    } else {
        constexpr int width = 8 * TPG;   // V is 1 here
        const int slot = threadIdx.x / TPG;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) lds[slot * width + 8 * lane + e] = at.on ? s[0].e[e] : 0.0f;
        __syncthreads();
        for (int c = threadIdx.x; c < n; c += block_threads<TPG>()) {
            float v = 0.0f;
            for (int k = 0; k < spb; ++k) v += lds[k * width + c];
            o[c] = v;
        }
    }
}

template <typename IO, int TPG, int V, bool FIRST>
__global__ void __launch_bounds__(block_threads<TPG>(), 4) gated_norm_bwd_kernel(GatedArgs p) {
    constexpr int T = block_threads<TPG>();
    __shared__ float red[Summer<TPG>::kFloats];
    __shared__ __align__(16) float wl[V * 8 * T];   // weights; at the end the slots' sums
    Summer<TPG> sum{red};
    const int tid = threadIdx.x, lane = tid % TPG;
    const Place at = place<TPG>(p.ngroups);
    const int64_t off = int64_t(at.group) * p.n, dim = int64_t(p.ngroups) * p.n;
    V8 dw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        LdsWeights<T>{wl + i * 8 * T}.put(loadw(p.w + (p.shared ? 0 : off), 8 * (lane + TPG * i), p.n), tid);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i].e[e] = 0.0f;
    }
    const int64_t loops = (p.rows + at.step - 1) / at.step;
    Raw8<IO> nx[V], nz[V], ng[V];   // the next row's
    auto fetch = [&](int64_t row) {
        const bool on = at.on && row < p.rows;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            nx[i].load(static_cast<const IO*>(p.x) + row * p.sx + off, col, p.n, on, p.vec);
            ng[i].load(static_cast<const IO*>(p.dy) + row * dim + off, col, p.n, on, p.vec);
            nz[i].load(static_cast<const IO*>(p.z) + row * p.sz + off, col, p.n, on && p.z, p.vec);
        }
    };
    if (V == 1) fetch(at.row);
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = at.row + l * at.step;
        const bool on = at.on && row < p.rows;
        if (V > 1) fetch(row);
        Raw8<IO> rx[V], rz[V], rg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[i] = nx[i];
            rz[i] = nz[i];
            rg[i] = ng[i];
        }
        if (V == 1 && l + 1 < loops) fetch(row + at.step);
        // p = x SiLU(z) or x; g = the gradient at the normalised values: dy w, with the gate
        // behind the norm dy w SiLU(z)
        float qt[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const V8 x = rx[i].values(), z = rz[i].values(), g = rg[i].values(), w = LdsWeights<T>{wl + i * 8 * T}.get(tid);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = p.z ? silu_f32(z.e[e]) : 1.0f;
                const float v = FIRST ? x.e[e] * a : x.e[e];
                const float u = (FIRST ? g.e[e] : g.e[e] * a) * w.e[e];
                qt[0] = fmaf(v, v, qt[0]);
                qt[1] = fmaf(u, v, qt[1]);
            }
        }
        sum.all(qt);
        const float rs = __builtin_amdgcn_rsqf(fmaf(qt[0], p.inv_n, p.eps));
        const float k = qt[1] * p.inv_n * rs * rs * rs;   // mean(g n) of n = p rs, times rs^2
        IO* dxr = static_cast<IO*>(p.y) + row * dim + off;
        IO* dzr = static_cast<IO*>(p.dz) + row * dim + off;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const V8 x = rx[i].values(), z = rz[i].values(), g = rg[i].values(), w = LdsWeights<T>{wl + i * 8 * T}.get(tid);
            V8 dx, dz;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float zz = z.e[e], sg = p.z ? sigmoid_f32(zz) : 1.0f;
                const float a = p.z ? zz * sg : 1.0f, slope = sg * fmaf(zz, 1.0f - sg, 1.0f);
                const float xx = x.e[e], dy = g.e[e];
                const float v = FIRST ? xx * a : xx;
                const float up = FIRST ? dy : dy * a;
                dw[i].e[e] = fmaf(up, v * rs, dw[i].e[e]);
                const float dp = fmaf(up * w.e[e], rs, -v * k);
                dx.e[e] = FIRST ? dp * a : dp;
                dz.e[e] = (FIRST ? dp * xx : dy * xx * rs * w.e[e]) * slope;
            }
            const int col = 8 * (lane + TPG * i);
            store8<IO>(dxr, col, p.n, on, p.vec, dx);
            if (p.z) store8<IO>(dzr, col, p.n, on, p.vec, dz);
        }
    }
    store_part<TPG, V>(p.part, dw, at, p.ngroups, p.n, p.shared, wl);
}

struct AddArgs {
    const void* x;
    const void* res;    // the stored r in the backward
    const float* scale;
    const float* post;
    const float* w;
    const void* dy;
    const void* dr;
    void* r;            // dres in the backward
    void* y;            // dx in the backward
    float* part;        // [blocks][dw, dscale, dpost][dim]
    int64_t rows, sx, sres, sr, sy;
    int32_t n, vec;
    float eps, inv_n;
};

template <typename IO, typename RT, int TPG, int V>
__global__ void __launch_bounds__(block_threads<TPG>()) add_norm_fwd_kernel(AddArgs p) {
    __shared__ float red[Summer<TPG>::kFloats];
    Summer<TPG> sum{red};
    const int lane = threadIdx.x % TPG;
    const Place at = place<TPG>(1);
    const int64_t loops = (p.rows + at.step - 1) / at.step;
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = at.row + l * at.step;
        const bool on = at.on && row < p.rows;
        V8 x[V], r[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            x[i] = load8<IO>(static_cast<const IO*>(p.x) + row * p.sx, col, p.n, on, p.vec);
            r[i] = load8<RT>(static_cast<const RT*>(p.res) + row * p.sres, col, p.n, on && p.res, p.vec);
        }
        float rs = 1.0f;
        if (p.post) {
            float q = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q = fmaf(x[i].e[e], x[i].e[e], q);
            rs = __builtin_amdgcn_rsqf(fmaf(sum(q), p.inv_n, p.eps));
        }
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            V8 po, sc;
            if (p.post) po = load8<float>(p.post, col, p.n, true, p.vec);
            if (p.scale) sc = load8<float>(p.scale, col, p.n, true, p.vec);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a = x[i].e[e];
                if (p.post) a *= rs * po.e[e];
                const float v = p.scale ? fmaf(sc.e[e], a, r[i].e[e]) : r[i].e[e] + a;
                r[i].e[e] = IOT<RT>::to_f32(IOT<RT>::from_f32(v));   // the norm is that of the stored value
                q = fmaf(r[i].e[e], r[i].e[e], q);
            }
            store8<RT>(static_cast<RT*>(p.r) + row * p.sr, col, p.n, on, p.vec, r[i]);
        }
        const float rr = __builtin_amdgcn_rsqf(fmaf(sum(q), p.inv_n, p.eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            const V8 w = load8<float>(p.w, col, p.n, true, p.vec);
            V8 y;
#pragma unroll
            for (int e = 0; e < 8; ++e) y.e[e] = r[i].e[e] * rr * w.e[e];
            store8<IO>(static_cast<IO*>(p.y) + row * p.sy, col, p.n, on, p.vec, y);
        }
    }
}

template <typename IO, typename RT, int TPG, int V>
__global__ void __launch_bounds__(block_threads<TPG>(), 4) add_norm_bwd_kernel(AddArgs p) {
    constexpr int T = block_threads<TPG>(), PL = V * 8 * T;
    constexpr bool HELD = V == 1;   // weights in LDS (past 8192 columns they are read again)
    __shared__ float red[Summer<TPG>::kFloats];
    __shared__ __align__(16) float wl[HELD ? 3 * PL : 4];   // w, scale, post; at the end the slots' sums
    Summer<TPG> sum{red};
    const int tid = threadIdx.x, lane = tid % TPG;
    const Place at = place<TPG>(1);
    V8 dw[V], dsc[V], dpo[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int col = 8 * (lane + TPG * i);
        if constexpr (HELD) {
            LdsWeights<T>{wl}.put(loadw(p.w, col, p.n), tid);
            LdsWeights<T>{wl + PL}.put(loadw(p.scale, col, p.n), tid);
            LdsWeights<T>{wl + 2 * PL}.put(loadw(p.post, col, p.n), tid);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i].e[e] = dsc[i].e[e] = dpo[i].e[e] = 0.0f;
    }
    auto weight = [&](int which, const float* q, int i) {
        if constexpr (HELD) return LdsWeights<T>{wl + which * PL}.get(tid);
        else return loadw(q, 8 * (lane + TPG * i), p.n);
    };
    const int64_t loops = (p.rows + at.step - 1) / at.step;
    Raw8<IO> nx[V], ny[V];          // the next row's
    Raw8<RT> nr[V], nd[V];
    auto fetch = [&](int64_t row) {
        const bool on = at.on && row < p.rows;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            nr[i].load(static_cast<const RT*>(p.res) + row * p.sr, col, p.n, on, p.vec);
            ny[i].load(static_cast<const IO*>(p.dy) + row * p.n, col, p.n, on, p.vec);
            nd[i].load(static_cast<const RT*>(p.dr) + row * p.n, col, p.n, on && p.dr, p.vec);
            nx[i].load(static_cast<const IO*>(p.x) + row * p.sx, col, p.n, on && (p.scale || p.post), p.vec);
        }
    };
    if (V == 1) fetch(at.row);
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = at.row + l * at.step;
        const bool on = at.on && row < p.rows;
        if (V > 1) fetch(row);
        Raw8<IO> rx[V], ry[V];
        Raw8<RT> rr8[V], rd[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[i] = nx[i];
            ry[i] = ny[i];
            rr8[i] = nr[i];
            rd[i] = nd[i];
        }
        if (V == 1 && l + 1 < loops) fetch(row + at.step);
        float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const V8 x = rx[i].values(), y = ry[i].values(), r = rr8[i].values(), w = weight(0, p.w, i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sums[0] = fmaf(r.e[e], r.e[e], sums[0]);
                sums[1] = fmaf(y.e[e] * w.e[e], r.e[e], sums[1]);
                sums[2] = fmaf(x.e[e], x.e[e], sums[2]);
            }
        }
        sum.all(sums);
        const float rr = __builtin_amdgcn_rsqf(fmaf(sums[0], p.inv_n, p.eps));
        const float k = sums[1] * p.inv_n * rr * rr * rr;
        const float rx1 = p.post ? __builtin_amdgcn_rsqf(fmaf(sums[2], p.inv_n, p.eps)) : 1.0f;
        float tx = 0.0f;
        V8 d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            {
                const V8 y = ry[i].values(), r = rr8[i].values(), w = weight(0, p.w, i);
                d[i] = rd[i].values();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[i].e[e] = fmaf(y.e[e], r.e[e] * rr, dw[i].e[e]);
                    // the gradient at r, then at a, then at the normalised x
                    d[i].e[e] += fmaf(y.e[e] * w.e[e], rr, -r.e[e] * k);
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // else the weights of every step below are read here and spill
            if (p.r) store8<RT>(static_cast<RT*>(p.r) + row * p.n, 8 * (lane + TPG * i), p.n, on, p.vec, d[i]);
            __builtin_amdgcn_sched_barrier(0);
            const V8 x = rx[i].values();
            if (p.scale) {
                const V8 sc = weight(1, p.scale, i);
                if (p.post) {
                    const V8 po = weight(2, p.post, i);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dsc[i].e[e] = fmaf(d[i].e[e], x.e[e] * rx1 * po.e[e], dsc[i].e[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dsc[i].e[e] = fmaf(d[i].e[e], x.e[e], dsc[i].e[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) d[i].e[e] *= sc.e[e];
            }
            __builtin_amdgcn_sched_barrier(0);
            if (p.post) {
                const V8 po = weight(2, p.post, i);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = x.e[e] * rx1;
                    dpo[i].e[e] = fmaf(d[i].e[e], n, dpo[i].e[e]);
                    d[i].e[e] *= po.e[e];
                    tx = fmaf(d[i].e[e], n, tx);
                }
            }
        }
        if (p.post) {
            const float m = sum(tx) * p.inv_n;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const V8 x = rx[i].values();
#pragma unroll
                for (int e = 0; e < 8; ++e) d[i].e[e] = rx1 * fmaf(-m * rx1, x.e[e], d[i].e[e]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            store8<IO>(static_cast<IO*>(p.y) + row * p.n, 8 * (lane + TPG * i), p.n, on, p.vec, d[i]);
    }
    const int64_t plane = int64_t(gridDim.x) * p.n;
    store_part<TPG, V>(p.part, dw, at, 1, p.n, true, wl);
    if (p.scale) store_part<TPG, V>(p.part + plane, dsc, at, 1, p.n, true, wl);
    if (p.post) store_part<TPG, V>(p.part + 2 * plane, dpo, at, 1, p.n, true, wl);
}

struct LayerArgs {
    const void* x;
    const float* w;
    const float* b;
    const void* dy;
    void* y;        // dx in the backward
    float* part;    // [blocks][dim] of dw, then of db
    int64_t rows, sx, sy;
    int32_t n, vec, bias;
    float eps, inv_n;
    double inv_n64;
};

// A thread's share of a row's sum: of float32 values in float64.  Up to 16 bf16 values add up in
// float32 as they are where they are of like size, and else below 2^-20 of the deviations.
template <typename IO> struct RowSum {
    typedef typename std::conditional<sizeof(IO) == 2, float, double>::type Of;
    Of q = 0;
    __device__ inline void add(const V8& x) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q += x.e[e];
    }
};

// A row's mean as two floats: the nearest one, and what that leaves of it, which is exactly zero
// where all values are equal (a product of n and a float is whole in float64).
struct Mean {
    float hi, lo;
    __device__ inline Mean(double sum, const LayerArgs& p) {
        hi = static_cast<float>(sum * p.inv_n64);
        lo = static_cast<float>(fma(-static_cast<double>(hi), static_cast<double>(p.n), sum) * p.inv_n64);
    }
    // x less the mean; columns behind the row's end stay zero, which the squares need
    __device__ inline void out_of(V8& x, int col, int n) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x.e[e] = col + e < n ? (x.e[e] - hi) - lo : 0.0f;
    }
};

// The mean first and the squares about it then, both from the row in registers: one more
// exchange than sums of x and x^2 would need, which cancel where a mean is far from zero.  For the
// same reason the mean is summed and kept beyond float32: an error of its last place is one of every
// deviation (y of three values of 1.7e9 would be off by 0.7).  That takes 0 to 3%; a second sum, of the
// deviations, would take 1 to 11%.  16384 bf16 rows of 2048 in 25 us (5.3 TB/s), 4 of 4096 in 3.0.
template <typename IO, int TPG, int V>
__global__ void __launch_bounds__(block_threads<TPG>()) layer_norm_fwd_kernel(LayerArgs p) {
    __shared__ float red[Summer<TPG>::kFloats];
    Summer<TPG> sum{red};
    const int lane = threadIdx.x % TPG;
    const Place at = place<TPG>(1);
    const int64_t loops = (p.rows + at.step - 1) / at.step;
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = at.row + l * at.step;
        const bool on = at.on && row < p.rows;
        V8 x[V];
        RowSum<IO> all;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = load8<IO>(static_cast<const IO*>(p.x) + row * p.sx, 8 * (lane + TPG * i), p.n, on, p.vec);
            all.add(x[i]);
        }
        const Mean mean(sum(static_cast<double>(all.q)), p);
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            mean.out_of(x[i], 8 * (lane + TPG * i), p.n);
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(x[i].e[e], x[i].e[e], q);
        }
        const float rs = __builtin_amdgcn_rsqf(fmaf(sum(q), p.inv_n, p.eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            const V8 w = load8<float>(p.w, col, p.n, true, p.vec), b = load8<float>(p.b, col, p.n, p.b != nullptr, p.vec);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i].e[e] = fmaf(x[i].e[e] * rs, w.e[e], b.e[e]);
            store8<IO>(static_cast<IO*>(p.y) + row * p.sy, col, p.n, on, p.vec, x[i]);
        }
    }
}

// With n = (x - mean) rs and d = dy w:  dx = rs (d - mean(d) - n mean(d n)), dw = sum dy n,
// db = sum dy.  The sums of d and of d (x - mean) go with that of the squares.  16384 bf16 rows of
// 4096 in 102 us (3.9 TB/s of rows) and 7 for the partial sums, 8191 float32 rows of 1535 in 33 (4.5)
// and 4.5.  Not kept: two rows at a time, or rows asked for two ahead (0 to 2%).
template <typename IO, int TPG, int V>
__global__ void __launch_bounds__(block_threads<TPG>(), 4) layer_norm_bwd_kernel(LayerArgs p) {
    constexpr int T = block_threads<TPG>();
    __shared__ float red[Summer<TPG>::kFloats];
    __shared__ __align__(16) float wl[V * 8 * T];   // weights; at the end the slots' sums
    Summer<TPG> sum{red};
    const int tid = threadIdx.x, lane = tid % TPG;
    const Place at = place<TPG>(1);
    V8 dw[V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        LdsWeights<T>{wl + i * 8 * T}.put(loadw(p.w, 8 * (lane + TPG * i), p.n), tid);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i].e[e] = db[i].e[e] = 0.0f;
    }
    const int64_t loops = (p.rows + at.step - 1) / at.step;
    Raw8<IO> nx[V], ng[V];   // the next row's
    auto fetch = [&](int64_t row) {
        const bool on = at.on && row < p.rows;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            nx[i].load(static_cast<const IO*>(p.x) + row * p.sx, col, p.n, on, p.vec);
            ng[i].load(static_cast<const IO*>(p.dy) + row * p.n, col, p.n, on, p.vec);
        }
    };
    if (V == 1) fetch(at.row);
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = at.row + l * at.step;
        const bool on = at.on && row < p.rows;
        if (V > 1) fetch(row);
        Raw8<IO> rx[V], rg[V];
        RowSum<IO> all;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[i] = nx[i];
            rg[i] = ng[i];
            all.add(rx[i].values());
        }
        if (V == 1 && l + 1 < loops) fetch(row + at.step);
        const Mean mean(sum(static_cast<double>(all.q)), p);
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            V8 x = rx[i].values();
            const V8 g = rg[i].values(), w = LdsWeights<T>{wl + i * 8 * T}.get(tid);
            mean.out_of(x, 8 * (lane + TPG * i), p.n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = g.e[e] * w.e[e];
                s[0] = fmaf(x.e[e], x.e[e], s[0]);
                s[1] += d;
                s[2] = fmaf(d, x.e[e], s[2]);
            }
        }
        sum.all(s);
        const float rs = __builtin_amdgcn_rsqf(fmaf(s[0], p.inv_n, p.eps));
        const float m = s[1] * p.inv_n, k = s[2] * p.inv_n * rs * rs;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 8 * (lane + TPG * i);
            V8 x = rx[i].values();
            const V8 g = rg[i].values(), w = LdsWeights<T>{wl + i * 8 * T}.get(tid);
            mean.out_of(x, col, p.n);
            V8 dx;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[i].e[e] = fmaf(g.e[e], x.e[e] * rs, dw[i].e[e]);
                db[i].e[e] += g.e[e];
                dx.e[e] = rs * (fmaf(g.e[e], w.e[e], -m) - x.e[e] * k);
            }
            store8<IO>(static_cast<IO*>(p.y) + row * p.n, col, p.n, on, p.vec, dx);
        }
    }
    store_part<TPG, V>(p.part, dw, at, 1, p.n, true, wl);
    if (p.bias) store_part<TPG, V>(p.part + int64_t(gridDim.x) * p.n, db, at, 1, p.n, true, wl);
}

// Sums `count` partial rows of n values, in a fixed order: 16 columns x 64 rows a workgroup,
// eight rows of a thread under way at once.  Plane b of the grid's y goes to out0, out1, out2.
// The columns go round over at most 2^20 workgroups (a grid has fewer than 2^32 threads).
constexpr int kSumLanes = 64;
inline uint32_t sum_blocks(int64_t n) {
    const int64_t b = cdiv(n, 16), most = int64_t(1) << 20;
    return static_cast<uint32_t>(b < most ? b : most);
}
__global__ void __launch_bounds__(16 * kSumLanes) sum_rows_kernel(const float* part, int64_t count, int64_t n,
                                                                  float* out0, float* out1, float* out2) {
    __shared__ float s[kSumLanes][16];
    float* out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
    if (!out) return;
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    for (int64_t c0 = int64_t(blockIdx.x) * 16; c0 < n; c0 += int64_t(gridDim.x) * 16) {
        const int64_t col = c0 + c;
        const float* q = part + blockIdx.y * count * n + col;
        float v = 0.0f;
        if (col < n) {
            int64_t i = r;
            for (; i + 7 * kSumLanes < count; i += 8 * kSumLanes) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = q[(i + k * kSumLanes) * n];
#pragma unroll
                for (int k = 0; k < 8; ++k) v += x[k];
            }
            for (; i < count; i += kSumLanes) v += q[i * n];
        }
        s[r][c] = v;
        __syncthreads();
        for (int d = kSumLanes / 2; d > 0; d >>= 1) {
            if (r < d) s[r][c] += s[r + d][c];
            __syncthreads();
        }
        if (r == 0 && col < n) out[col] = s[0][c];
    }
}

// ---------------------------------------------------------------- host
inline int tpg_for(int64_t n) {
    int t = 8;
    while (t < 1024 && int64_t(t) * kVW < n) t <<= 1;
    return t;
}

inline int64_t slots_per_block(int tpg) { return tpg < 256 ? 256 / tpg : 1; }

// Workgroups of a launch over `rows` rows of `ngroups` groups: enough to fill the card
// (`most` of them), in whole rows.
inline int64_t blocks_for(int64_t rows, int64_t ngroups, int tpg, int64_t most) {
    const int64_t spb = slots_per_block(tpg);
    const int64_t all = cdiv(rows * ngroups, spb), one = cdiv(ngroups, spb);
    int64_t b = all < most ? all : most;
    return b < one ? one : b;
}

// A gradient's workgroups: as many as the card holds at once, 1024 threads a CU; fewer leave
// it idle, more only add partial sums.  Measured, us at 256, 512 and 1024 workgroups: 8192 rows
// of 8192 columns 183, 198, 224; 16384 of 4096 202, 135, 144; at 512, 1024 and 2048: 16384 rows
// of 32 groups of 128 192, 131, 137.
inline int64_t bwd_blocks(int tpg) { return 256 * 1024 / (tpg < 256 ? 256 : tpg); }
constexpr int64_t kFwdBlocks = int64_t(1) << 20;

inline bool vec_row(const void* q, int64_t stride, int64_t e) { return !misaligned(q, 16) && stride * e % 16 == 0; }

inline int64_t size_of(int32_t t) { return t == SSM_BF16 ? 2 : 4; }

#define SSM_NORM_TPG(DO)                   \
    switch (tpg) {                         \
    case 8: DO(8, 1); break;               \
    case 16: DO(16, 1); break;             \
    case 32: DO(32, 1); break;             \
    case 64: DO(64, 1); break;             \
    case 128: DO(128, 1); break;           \
    case 256: DO(256, 1); break;           \
    case 512: DO(512, 1); break;           \
    default:                               \
        if (n <= 8192) { DO(1024, 1); }    \
        else { DO(1024, 2); }              \
    }

template <typename IO, bool FIRST> void run_gated(const GatedArgs& a, int tpg, int64_t blocks, bool bwd, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(blocks)), block(tpg < 256 ? 256 : tpg);
    const int64_t n = a.n;
#define SSM_DO(T, V)                                                                                   \
    do {                                                                                               \
        if (bwd) launch_kernel(gated_norm_bwd_kernel<IO, T, V, FIRST>, grid, block, 0, s, a);           \
        else launch_kernel(gated_norm_fwd_kernel<IO, T, V, FIRST>, grid, block, 0, s, a);               \
    } while (0)
    SSM_NORM_TPG(SSM_DO)
#undef SSM_DO
}

template <typename IO, typename RT> void run_add(const AddArgs& a, int tpg, int64_t blocks, bool bwd, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(blocks)), block(tpg < 256 ? 256 : tpg);
    const int64_t n = a.n;
#define SSM_DO(T, V)                                                                                   \
    do {                                                                                               \
        if (bwd) launch_kernel(add_norm_bwd_kernel<IO, RT, T, V>, grid, block, 0, s, a);                \
        else launch_kernel(add_norm_fwd_kernel<IO, RT, T, V>, grid, block, 0, s, a);                    \
    } while (0)
    SSM_NORM_TPG(SSM_DO)
#undef SSM_DO
}

template <typename IO> void run_layer(const LayerArgs& a, int tpg, int64_t blocks, bool bwd, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(blocks)), block(tpg < 256 ? 256 : tpg);
    const int64_t n = a.n;
#define SSM_DO(T, V)                                                                                   \
    do {                                                                                               \
        if (bwd) launch_kernel(layer_norm_bwd_kernel<IO, T, V>, grid, block, 0, s, a);                  \
        else launch_kernel(layer_norm_fwd_kernel<IO, T, V>, grid, block, 0, s, a);                      \
    } while (0)
    SSM_NORM_TPG(SSM_DO)
#undef SSM_DO
}

inline void gated(const GatedArgs& a, const ssm_gated_norm_dims& d, int tpg, int64_t blocks, bool bwd, hipStream_t s) {
    if (d.io_dtype == SSM_BF16) {
        if (d.gate_first) run_gated<uint16_t, true>(a, tpg, blocks, bwd, s);
        else run_gated<uint16_t, false>(a, tpg, blocks, bwd, s);
    } else {
        if (d.gate_first) run_gated<float, true>(a, tpg, blocks, bwd, s);
        else run_gated<float, false>(a, tpg, blocks, bwd, s);
    }
}

inline void add(const AddArgs& a, const ssm_add_norm_dims& d, int tpg, int64_t blocks, bool bwd, hipStream_t s) {
    if (d.io_dtype == SSM_BF16) {
        if (d.res_dtype == SSM_BF16) run_add<uint16_t, uint16_t>(a, tpg, blocks, bwd, s);
        else run_add<uint16_t, float>(a, tpg, blocks, bwd, s);
    } else {
        if (d.res_dtype == SSM_BF16) run_add<float, uint16_t>(a, tpg, blocks, bwd, s);
        else run_add<float, float>(a, tpg, blocks, bwd, s);
    }
}

// The reciprocal square root takes numbers below 2^-126 for zero: a row of zeros would turn NaN.
inline bool good_eps(float eps) { return eps >= 1.17549435e-38f && eps < 3.4e38f; }

inline int check(const ssm_gated_norm_dims* d) {
    if (!d) return SSM_ERR_NULL;
    if (d->rows < 1 || d->ngroups < 1 || d->group < 1) return SSM_ERR_EMPTY;
    if (d->io_dtype != SSM_F32 && d->io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
    const int64_t lim = int64_t(1) << 40;
    if (d->group > SSM_NORM_MAX_DIM || d->ngroups > (1 << 20) || d->rows > lim / (d->ngroups * d->group))
        return SSM_ERR_DIMS;
    const int64_t dim = d->ngroups * d->group;
    for (const int64_t s : {d->x_stride, d->z_stride, d->y_stride})
        if (s != 0 && (s < dim || s > lim / d->rows)) return SSM_ERR_DIMS;
    if ((d->gate_first != 0 && d->gate_first != 1) || (d->shared_weight != 0 && d->shared_weight != 1)) return SSM_ERR_DIMS;
    if (!good_eps(d->eps)) return SSM_ERR_DIMS;
    return SSM_OK;
}

inline int check(const ssm_add_norm_dims* d) {
    if (!d) return SSM_ERR_NULL;
    if (d->rows < 1 || d->dim < 1) return SSM_ERR_EMPTY;
    if ((d->io_dtype != SSM_F32 && d->io_dtype != SSM_BF16) || (d->res_dtype != SSM_F32 && d->res_dtype != SSM_BF16))
        return SSM_ERR_DTYPE;
    const int64_t lim = int64_t(1) << 40;
    if (d->dim > SSM_NORM_MAX_DIM || d->rows > lim / d->dim || d->reserved != 0) return SSM_ERR_DIMS;
    for (const int64_t s : {d->x_stride, d->res_stride, d->r_stride, d->y_stride})
        if (s != 0 && (s < d->dim || s > lim / d->rows)) return SSM_ERR_DIMS;
    if (!good_eps(d->eps)) return SSM_ERR_DIMS;
    return SSM_OK;
}

inline int check(const ssm_layer_norm_dims* d) {
    if (!d) return SSM_ERR_NULL;
    if (d->rows < 1 || d->dim < 1) return SSM_ERR_EMPTY;
    if (d->io_dtype != SSM_F32 && d->io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
    const int64_t lim = int64_t(1) << 40;
    if (d->dim > SSM_NORM_MAX_DIM || d->rows > lim / d->dim) return SSM_ERR_DIMS;
    for (const int64_t s : {d->x_stride, d->y_stride})
        if (s != 0 && (s < d->dim || s > lim / d->rows)) return SSM_ERR_DIMS;
    if (!good_eps(d->eps)) return SSM_ERR_DIMS;
    return SSM_OK;
}

}  // namespace nrm
}  // namespace

extern "C" {

int ssm_gated_norm_fwd(const void* x, const void* z, const float* w, void* y, const ssm_gated_norm_dims* dims,
                       void* stream) {
    using namespace nrm;
    if (!dims || !x || !w || !y) return SSM_ERR_NULL;
    const int st = check(dims);
    if (st != SSM_OK) return st;
    const ssm_gated_norm_dims& d = *dims;
    const int64_t e = size_of(d.io_dtype), dim = d.ngroups * d.group;
    if (misaligned(x, e) || misaligned(z, e) || misaligned(y, e) || misaligned(w, 4)) return SSM_ERR_ALIGN;
    GatedArgs a = {};
    a.x = x; a.z = z; a.w = w; a.y = y;
    a.rows = d.rows; a.ngroups = static_cast<int32_t>(d.ngroups); a.n = static_cast<int32_t>(d.group);
    a.sx = d.x_stride ? d.x_stride : dim;
    a.sz = d.z_stride ? d.z_stride : dim;
    a.sy = d.y_stride ? d.y_stride : dim;
    const Area in[] = {rows_of(y == x && a.sy == a.sx ? nullptr : x, d.rows, a.sx, dim, e),
                       rows_of(y == z && a.sy == a.sz ? nullptr : z, d.rows, a.sz, dim, e),
                       flat(w, static_cast<size_t>(d.shared_weight ? d.group : dim) * 4)};
    const Area out[] = {rows_of(y, d.rows, a.sy, dim, e)};
    if (clash(in, out)) return SSM_ERR_ALIAS;
    a.shared = d.shared_weight; a.eps = d.eps; a.inv_n = 1.0f / static_cast<float>(d.group);
    a.vec = d.group % 8 == 0 && vec_row(x, a.sx, e) && vec_row(y, a.sy, e) && (!z || vec_row(z, a.sz, e));
    const int tpg = tpg_for(d.group);
    const int64_t blocks = blocks_for(d.rows, d.ngroups, tpg, kFwdBlocks);
    ssm_detail::launch_error = hipSuccess;
    gated(a, d, tpg, blocks, false, static_cast<hipStream_t>(stream));
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_gated_norm_bwd_workspace_bytes(const ssm_gated_norm_dims* dims) {
    using namespace nrm;
    if (check(dims) != SSM_OK) return 0;
    const int tpg = tpg_for(dims->group);
    const int64_t blocks = blocks_for(dims->rows, dims->ngroups, tpg, bwd_blocks(tpg));
    const int64_t lanes = blocks * slots_per_block(tpg) / dims->ngroups;
    return static_cast<size_t>(dims->shared_weight ? blocks * dims->group : lanes * dims->ngroups * dims->group) * 4;
}

int ssm_gated_norm_bwd(const void* x, const void* z, const float* w, const void* dy, void* dx, void* dz, float* dw,
                       const ssm_gated_norm_dims* dims, void* stream) {
    using namespace nrm;
    if (!dims || !x || !w || !dy || !dx || !dw || (z == nullptr) != (dz == nullptr)) return SSM_ERR_NULL;
    const int st = check(dims);
    if (st != SSM_OK) return st;
    const ssm_gated_norm_dims& d = *dims;
    const int64_t e = size_of(d.io_dtype), dim = d.ngroups * d.group;
    if (misaligned(x, e) || misaligned(z, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(dz, e) ||
        misaligned(w, 4) || misaligned(dw, 4))
        return SSM_ERR_ALIGN;
    const size_t need = ssm_gated_norm_bwd_workspace_bytes(dims);
    if (!d.workspace || d.workspace_bytes < need || misaligned(d.workspace, 256)) return SSM_ERR_WORKSPACE;
    GatedArgs a = {};
    a.x = x; a.z = z; a.w = w; a.dy = dy; a.y = dx; a.dz = dz; a.part = static_cast<float*>(d.workspace);
    a.rows = d.rows; a.ngroups = static_cast<int32_t>(d.ngroups); a.n = static_cast<int32_t>(d.group);
    a.sx = d.x_stride ? d.x_stride : dim;
    a.sz = d.z_stride ? d.z_stride : dim;
    const size_t all = static_cast<size_t>(d.rows * dim * e), nw = static_cast<size_t>(d.shared_weight ? d.group : dim) * 4;
    const Area in[] = {rows_of(x, d.rows, a.sx, dim, e), rows_of(z, d.rows, a.sz, dim, e), flat(dy, all), flat(w, nw)};
    const Area out[] = {flat(dx, all), flat(dz, all), flat(dw, nw), flat(d.workspace, need)};
    if (clash(in, out)) return SSM_ERR_ALIAS;
    a.shared = d.shared_weight; a.eps = d.eps; a.inv_n = 1.0f / static_cast<float>(d.group);
    a.vec = d.group % 8 == 0 && vec_row(x, a.sx, e) && vec_row(dy, dim, e) && vec_row(dx, dim, e) &&
            (!z || (vec_row(z, a.sz, e) && vec_row(dz, dim, e)));
    const int tpg = tpg_for(d.group);
    const int64_t blocks = blocks_for(d.rows, d.ngroups, tpg, bwd_blocks(tpg));
    const int64_t lanes = blocks * slots_per_block(tpg) / d.ngroups;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ssm_detail::launch_error = hipSuccess;
    gated(a, d, tpg, blocks, true, s);
    const int64_t n = d.shared_weight ? d.group : dim;
    launch_kernel(sum_rows_kernel, dim3(sum_blocks(n)), dim3(16 * kSumLanes), 0, s, a.part,
                  d.shared_weight ? blocks : lanes, n, dw, static_cast<float*>(nullptr), static_cast<float*>(nullptr));
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_add_norm_fwd(const void* x, const void* res, const float* scale, const float* post, const float* w, void* r,
                     void* y, const ssm_add_norm_dims* dims, void* stream) {
    using namespace nrm;
    if (!dims || !x || !w || !r || !y) return SSM_ERR_NULL;
    const int st = check(dims);
    if (st != SSM_OK) return st;
    const ssm_add_norm_dims& d = *dims;
    const int64_t e = size_of(d.io_dtype), f = size_of(d.res_dtype);
    if (misaligned(x, e) || misaligned(y, e) || misaligned(res, f) || misaligned(r, f) || misaligned(scale, 4) ||
        misaligned(post, 4) || misaligned(w, 4))
        return SSM_ERR_ALIGN;
    AddArgs a = {};
    a.x = x; a.res = res; a.scale = scale; a.post = post; a.w = w; a.r = r; a.y = y;
    a.rows = d.rows; a.n = static_cast<int32_t>(d.dim);
    a.sx = d.x_stride ? d.x_stride : d.dim;
    a.sres = d.res_stride ? d.res_stride : d.dim;
    a.sr = d.r_stride ? d.r_stride : d.dim;
    a.sy = d.y_stride ? d.y_stride : d.dim;
    const size_t nw = static_cast<size_t>(d.dim) * 4;
    const Area in[] = {rows_of(x, d.rows, a.sx, d.dim, e),
                       rows_of(r == res && a.sr == a.sres ? nullptr : res, d.rows, a.sres, d.dim, f),
                       flat(scale, nw), flat(post, nw), flat(w, nw)};
    const Area out[] = {rows_of(r, d.rows, a.sr, d.dim, f), rows_of(y, d.rows, a.sy, d.dim, e)};
    if (clash(in, out)) return SSM_ERR_ALIAS;
    a.eps = d.eps; a.inv_n = 1.0f / static_cast<float>(d.dim);
    a.vec = d.dim % 8 == 0 && vec_row(x, a.sx, e) && vec_row(y, a.sy, e) && vec_row(r, a.sr, f) &&
            (!res || vec_row(res, a.sres, f)) && !misaligned(w, 16) && !misaligned(scale, 16) && !misaligned(post, 16);
    const int tpg = tpg_for(d.dim);
    ssm_detail::launch_error = hipSuccess;
    add(a, d, tpg, blocks_for(d.rows, 1, tpg, kFwdBlocks), false, static_cast<hipStream_t>(stream));
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_add_norm_bwd_workspace_bytes(const ssm_add_norm_dims* dims) {
    using namespace nrm;
    if (check(dims) != SSM_OK) return 0;
    const int tpg = tpg_for(dims->dim);
    return static_cast<size_t>(3 * blocks_for(dims->rows, 1, tpg, bwd_blocks(tpg)) * dims->dim) * 4;
}

int ssm_add_norm_bwd(const void* x, const void* r, const float* scale, const float* post, const float* w,
                     const void* dy, const void* dr, void* dx, void* dres, float* dw, float* dscale, float* dpost,
                     const ssm_add_norm_dims* dims, void* stream) {
    using namespace nrm;
    if (!dims || !r || !w || !dy || !dx || !dw) return SSM_ERR_NULL;
    if ((scale && !dscale) || (post && !dpost) || ((scale || post) && !x)) return SSM_ERR_NULL;
    const int st = check(dims);
    if (st != SSM_OK) return st;
    const ssm_add_norm_dims& d = *dims;
    const int64_t e = size_of(d.io_dtype), f = size_of(d.res_dtype);
    if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(r, f) || misaligned(dr, f) ||
        misaligned(dres, f) || misaligned(scale, 4) || misaligned(post, 4) || misaligned(w, 4) || misaligned(dw, 4) ||
        misaligned(dscale, 4) || misaligned(dpost, 4))
        return SSM_ERR_ALIGN;
    const size_t need = ssm_add_norm_bwd_workspace_bytes(dims);
    if (!d.workspace || d.workspace_bytes < need || misaligned(d.workspace, 256)) return SSM_ERR_WORKSPACE;
    AddArgs a = {};
    a.x = x; a.res = r; a.scale = scale; a.post = post; a.w = w; a.dy = dy; a.dr = dr; a.r = dres; a.y = dx;
    a.part = static_cast<float*>(d.workspace);
    a.rows = d.rows; a.n = static_cast<int32_t>(d.dim);
    a.sx = d.x_stride ? d.x_stride : d.dim;
    a.sr = d.r_stride ? d.r_stride : d.dim;
    const size_t nw = static_cast<size_t>(d.dim) * 4, ne = static_cast<size_t>(d.rows * d.dim * e),
                 nf = static_cast<size_t>(d.rows * d.dim * f);
    const Area in[] = {rows_of(x, d.rows, a.sx, d.dim, e), rows_of(r, d.rows, a.sr, d.dim, f), flat(dy, ne),
                       flat(dres == dr ? nullptr : dr, nf), flat(scale, nw), flat(post, nw), flat(w, nw)};
    const Area out[] = {flat(dx, ne), flat(dres, nf), flat(dw, nw), flat(scale ? dscale : nullptr, nw),
                        flat(post ? dpost : nullptr, nw), flat(d.workspace, need)};
    if (clash(in, out)) return SSM_ERR_ALIAS;
    a.eps = d.eps; a.inv_n = 1.0f / static_cast<float>(d.dim);
    a.vec = d.dim % 8 == 0 && (!x || vec_row(x, a.sx, e)) && vec_row(r, a.sr, f) && vec_row(dy, d.dim, e) &&
            vec_row(dx, d.dim, e) && (!dr || vec_row(dr, d.dim, f)) && (!dres || vec_row(dres, d.dim, f));
    const int tpg = tpg_for(d.dim);
    const int64_t blocks = blocks_for(d.rows, 1, tpg, bwd_blocks(tpg));
    hipStream_t s = static_cast<hipStream_t>(stream);
    ssm_detail::launch_error = hipSuccess;
    add(a, d, tpg, blocks, true, s);
    launch_kernel(sum_rows_kernel, dim3(sum_blocks(d.dim), 3), dim3(16 * kSumLanes), 0, s, a.part, blocks,
                  d.dim, dw, scale ? dscale : nullptr, post ? dpost : nullptr);
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_layer_norm_fwd(const void* x, const float* w, const float* b, void* y, const ssm_layer_norm_dims* dims,
                       void* stream) {
    using namespace nrm;
    if (!dims || !x || !w || !y) return SSM_ERR_NULL;
    const int st = check(dims);
    if (st != SSM_OK) return st;
    const ssm_layer_norm_dims& d = *dims;
    const int64_t e = size_of(d.io_dtype);
    if (misaligned(x, e) || misaligned(y, e) || misaligned(w, 4) || misaligned(b, 4)) return SSM_ERR_ALIGN;
    LayerArgs a = {};
    a.x = x; a.w = w; a.b = b; a.y = y;
    a.rows = d.rows; a.n = static_cast<int32_t>(d.dim);
    a.sx = d.x_stride ? d.x_stride : d.dim;
    a.sy = d.y_stride ? d.y_stride : d.dim;
    const size_t nw = static_cast<size_t>(d.dim) * 4;
    const Area in[] = {rows_of(y == x && a.sy == a.sx ? nullptr : x, d.rows, a.sx, d.dim, e), flat(w, nw), flat(b, nw)};
    const Area out[] = {rows_of(y, d.rows, a.sy, d.dim, e)};
    if (clash(in, out)) return SSM_ERR_ALIAS;
    a.eps = d.eps; a.inv_n = 1.0f / static_cast<float>(d.dim); a.inv_n64 = 1.0 / static_cast<double>(d.dim);
    a.vec = d.dim % 8 == 0 && vec_row(x, a.sx, e) && vec_row(y, a.sy, e) && !misaligned(w, 16) && !misaligned(b, 16);
    const int tpg = tpg_for(d.dim);
    const int64_t blocks = blocks_for(d.rows, 1, tpg, kFwdBlocks);
    ssm_detail::launch_error = hipSuccess;
    if (d.io_dtype == SSM_BF16) run_layer<uint16_t>(a, tpg, blocks, false, static_cast<hipStream_t>(stream));
    else run_layer<float>(a, tpg, blocks, false, static_cast<hipStream_t>(stream));
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_layer_norm_bwd_workspace_bytes(const ssm_layer_norm_dims* dims) {
    using namespace nrm;
    if (check(dims) != SSM_OK) return 0;
    const int tpg = tpg_for(dims->dim);
    return static_cast<size_t>(2 * blocks_for(dims->rows, 1, tpg, bwd_blocks(tpg)) * dims->dim) * 4;
}

int ssm_layer_norm_bwd(const void* x, const float* w, const void* dy, void* dx, float* dw, float* db,
                       const ssm_layer_norm_dims* dims, void* stream) {
    using namespace nrm;
    if (!dims || !x || !w || !dy || !dx || !dw) return SSM_ERR_NULL;
    const int st = check(dims);
    if (st != SSM_OK) return st;
    const ssm_layer_norm_dims& d = *dims;
    const int64_t e = size_of(d.io_dtype);
    if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(w, 4) || misaligned(dw, 4) || misaligned(db, 4))
        return SSM_ERR_ALIGN;
    const size_t need = ssm_layer_norm_bwd_workspace_bytes(dims);
    if (!d.workspace || d.workspace_bytes < need || misaligned(d.workspace, 256)) return SSM_ERR_WORKSPACE;
    LayerArgs a = {};
    a.x = x; a.w = w; a.dy = dy; a.y = dx; a.part = static_cast<float*>(d.workspace); a.bias = db != nullptr;
    a.rows = d.rows; a.n = static_cast<int32_t>(d.dim);
    a.sx = d.x_stride ? d.x_stride : d.dim;
    const size_t nw = static_cast<size_t>(d.dim) * 4, all = static_cast<size_t>(d.rows * d.dim * e);
    const Area in[] = {rows_of(x, d.rows, a.sx, d.dim, e), flat(dy, all), flat(w, nw)};
    const Area out[] = {flat(dx, all), flat(dw, nw), flat(db, nw), flat(d.workspace, need)};
    if (clash(in, out)) return SSM_ERR_ALIAS;
    a.eps = d.eps; a.inv_n = 1.0f / static_cast<float>(d.dim); a.inv_n64 = 1.0 / static_cast<double>(d.dim);
    a.vec = d.dim % 8 == 0 && vec_row(x, a.sx, e) && vec_row(dy, d.dim, e) && vec_row(dx, d.dim, e);
    const int tpg = tpg_for(d.dim);
    const int64_t blocks = blocks_for(d.rows, 1, tpg, bwd_blocks(tpg));
    hipStream_t s = static_cast<hipStream_t>(stream);
    ssm_detail::launch_error = hipSuccess;
    if (d.io_dtype == SSM_BF16) run_layer<uint16_t>(a, tpg, blocks, true, s);
    else run_layer<float>(a, tpg, blocks, true, s);
    launch_kernel(sum_rows_kernel, dim3(sum_blocks(d.dim), db ? 2 : 1), dim3(16 * kSumLanes), 0, s, a.part, blocks, d.dim,
                  dw, db, static_cast<float*>(nullptr));
    return ssm_detail::launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
