// delta_host_checks.cpp -- host code of the gated delta rule and of the layer norm: argument
// checks, piece plans, workspace layouts and kernel dispatch on the CPU, with hip_stub.cpp in place
// of the HIP runtime (every launch is checked against grid, block and LDS limits and recorded).
// Test infrastructure only.  Exits 0 when every check holds.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "ssm.h"

extern "C" {
size_t stub_launch_count(void);
const char* stub_launch_name(size_t i);
unsigned stub_launch_grid(size_t i);
unsigned stub_launch_block(size_t i);
void stub_launch_reset(void);
void stub_fail_next_launch(int n);
}

static long g_checks = 0, g_failed = 0;
#define CHECK(cond, ...)                                                        \
    do {                                                                        \
        ++g_checks;                                                             \
        if (!(cond)) {                                                          \
            ++g_failed;                                                         \
            fprintf(stderr, "FAILED %s:%d: %s: ", __FILE__, __LINE__, #cond); \
            fprintf(stderr, __VA_ARGS__);                                       \
            fprintf(stderr, "\n");                                              \
        }                                                                       \
    } while (0)

// Fake device addresses, 32 TiB apart (never dereferenced: the kernels do not run).
static void* dev(int slot) { return reinterpret_cast<void*>((uintptr_t(slot) + 1) << 45); }
static float* fdev(int slot) { return static_cast<float*>(dev(slot)); }
static const int32_t* idev(int slot) { return static_cast<const int32_t*>(dev(slot)); }

static void threads() {
    for (size_t i = 0; i < stub_launch_count(); ++i)
        CHECK(uint64_t(stub_launch_grid(i)) * stub_launch_block(i) < (uint64_t(1) << 32), "%s: %u workgroups of %u", stub_launch_name(i),
              stub_launch_grid(i), stub_launch_block(i));
}

static int fwd(const ssm_linattn_dims& d, const int32_t* cu, bool states) {
    stub_launch_reset();
    const int st = ssm_delta_fwd(dev(0), dev(1), dev(2), fdev(3), fdev(4), cu, states ? idev(6) : nullptr,
                                 states ? fdev(7) : nullptr, dev(8), states ? fdev(9) : nullptr, &d, nullptr);
    CHECK((st == SSM_OK) == (stub_launch_count() > 0), "launches %zu of %d", stub_launch_count(), st);
    threads();
    return st;
}

static int bwd(const ssm_linattn_dims& d, const int32_t* cu, bool states) {
    ssm_delta_grads g = {dev(20), dev(21), dev(22), fdev(23), fdev(24), states ? fdev(25) : nullptr};
    stub_launch_reset();
    const int st = ssm_delta_bwd(dev(0), dev(1), dev(2), fdev(3), fdev(4), cu, states ? fdev(7) : nullptr, dev(8),
                                 states ? fdev(9) : nullptr, &g, &d, nullptr);
    CHECK((st == SSM_OK) == (stub_launch_count() > 0), "launches %zu of %d", stub_launch_count(), st);
    threads();
    return st;
}

static void delta() {
    const int64_t Ts[] = {1, 2, 63, 64, 65, 1000, 8192, 131072, int64_t(1) << 30, (int64_t(1) << 31) - 1};
    const int64_t Ns[] = {1, 2, 7, 1000, 65535};
    const int64_t Hs[][2] = {{1, 1}, {4, 2}, {32, 32}, {32767, 1}};
    const int64_t Ds[][2] = {{1, 1}, {64, 64}, {128, 128}, {72, 40}, {256, 256}, {200, 96}};
    for (int64_t T : Ts)
        for (int64_t n : Ns)
            for (const auto& h : Hs)
                for (const auto& dd : Ds)
                    for (int io : {int(SSM_F32), int(SSM_BF16)})
                        for (int64_t piece : {int64_t(0), int64_t(64), int64_t(1024)}) {
                            ssm_linattn_dims d;
                            memset(&d, 0, sizeof(d));
                            d.tokens = T; d.nseq = n; d.nheads = h[0]; d.kheads = h[1]; d.dk = dd[0]; d.dv = dd[1];
                            d.io_dtype = io; d.piece_len = piece; d.scale = 1.0f; d.nslots = n;
                            d.workspace = dev(30);
                            const size_t need = ssm_delta_fwd_workspace_bytes(&d), needb = ssm_delta_bwd_workspace_bytes(&d);
                            CHECK(need % 256 == 0 && needb % 256 == 0, "T %lld", (long long)T);
                            for (const int32_t* cu : {idev(5), static_cast<const int32_t*>(nullptr)}) {
                                if (!cu && T % n != 0) continue;
                                for (bool states : {false, true}) {
                                    d.workspace_bytes = need;
                                    int st = fwd(d, cu, states);
                                    // a plan that is refused outright (too many pieces) has no workspace either
                                    CHECK(st == SSM_OK || st == SSM_ERR_DIMS || st == SSM_ERR_ALIAS, "fwd %d", st);
                                    d.workspace_bytes = needb;
                                    st = bwd(d, cu, states);
                                    CHECK(st == SSM_OK || st == SSM_ERR_DIMS || st == SSM_ERR_ALIAS, "bwd %d", st);
                                }
                            }
                            if (need) {
                                d.workspace_bytes = 0;
                                CHECK(fwd(d, idev(5), false) != SSM_OK, "no workspace");
                            }
                            if (needb) {
                                d.workspace_bytes = 0;
                                CHECK(bwd(d, idev(5), false) != SSM_OK, "no workspace");
                            }
                            if (T == n) {
                                stub_launch_reset();
                                const int st = ssm_delta_step(dev(0), dev(1), dev(2), fdev(3), fdev(4), nullptr, fdev(10), dev(8), &d,
                                                              nullptr);
                                CHECK(st == SSM_OK || st == SSM_ERR_DIMS || st == SSM_ERR_ALIAS, "step %d", st);
                                CHECK(st != SSM_OK || stub_launch_count() == 1, "step launches");
                                threads();
                            }
                        }
    // a failing launch is this call's error, whichever it is
    ssm_linattn_dims d;
    memset(&d, 0, sizeof(d));
    d.tokens = 8192; d.nseq = 1; d.nheads = 4; d.kheads = 2; d.dk = d.dv = 128; d.io_dtype = SSM_BF16; d.scale = 1.0f; d.nslots = 1;
    d.workspace = dev(30);
    for (bool back : {false, true}) {
        d.workspace_bytes = back ? ssm_delta_bwd_workspace_bytes(&d) : ssm_delta_fwd_workspace_bytes(&d);
        CHECK((back ? bwd(d, nullptr, false) : fwd(d, nullptr, false)) == SSM_OK, "whole");
        const int count = static_cast<int>(stub_launch_count());
        CHECK(count >= 2, "launches %d", count);
        for (int i = 1; i <= count; ++i) {
            stub_launch_reset();
            stub_fail_next_launch(i);
            ssm_delta_grads g = {dev(20), dev(21), dev(22), fdev(23), fdev(24), nullptr};
            const int st = back ? ssm_delta_bwd(dev(0), dev(1), dev(2), fdev(3), fdev(4), nullptr, nullptr, dev(8), nullptr, &g, &d,
                                                nullptr)
                                : ssm_delta_fwd(dev(0), dev(1), dev(2), fdev(3), fdev(4), nullptr, nullptr, nullptr, dev(8), nullptr,
                                                &d, nullptr);
            CHECK(st == SSM_ERR_HIP, "launch %d: %d", i, st);
        }
        CHECK((back ? bwd(d, nullptr, false) : fwd(d, nullptr, false)) == SSM_OK, "after");
    }
}

static void layer_norm() {
    for (int64_t rows : {int64_t(1), int64_t(3), int64_t(1000), int64_t(1) << 20, int64_t(1) << 33, int64_t(1) << 40})
        for (int64_t n : std::initializer_list<int64_t>{1, 7, 64, 65, 512, 1536, 4096, 8192, 8193, 16384, 16385})
            for (int io : {int(SSM_F32), int(SSM_BF16)})
                for (bool bias : {false, true}) {
                    ssm_layer_norm_dims d;
                    memset(&d, 0, sizeof(d));
                    d.rows = rows; d.dim = n; d.io_dtype = io; d.eps = 1e-5f;
                    stub_launch_reset();
                    const int st = ssm_layer_norm_fwd(dev(0), fdev(1), bias ? fdev(2) : nullptr, dev(3), &d, nullptr);
                    CHECK(st == (n > 16384 || rows > (int64_t(1) << 40) / n ? SSM_ERR_DIMS : SSM_OK), "layer %d", st);
                    CHECK((st == SSM_OK) == (stub_launch_count() == 1), "launches %zu", stub_launch_count());
                    threads();
                    const size_t need = ssm_layer_norm_bwd_workspace_bytes(&d);
                    CHECK((st == SSM_OK) == (need > 0), "layer workspace");
                    d.workspace = dev(30);
                    d.workspace_bytes = need;
                    stub_launch_reset();
                    const int sb = ssm_layer_norm_bwd(dev(0), fdev(1), dev(4), dev(5), fdev(6), bias ? fdev(7) : nullptr, &d, nullptr);
                    CHECK(sb == st, "layer bwd %d", sb);
                    threads();
                    if (st != SSM_OK) continue;
                    const int count = static_cast<int>(stub_launch_count());
                    for (int i = 1; i <= count; ++i) {
                        stub_fail_next_launch(i);
                        CHECK(ssm_layer_norm_bwd(dev(0), fdev(1), dev(4), dev(5), fdev(6), nullptr, &d, nullptr) == SSM_ERR_HIP, "%d", i);
                    }
                }
}

int main() {
    delta();
    layer_norm();
    printf("%ld checks, %ld failed\n", g_checks, g_failed);
    return g_failed ? 1 : 0;
}
