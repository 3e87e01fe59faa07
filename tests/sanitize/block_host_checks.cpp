// block_host_checks.cpp -- host code of the block operators (linear attention, norms):
// argument checks, piece plans, workspace layouts and kernel dispatch on the CPU under
// AddressSanitizer and UndefinedBehaviorSanitizer, with hip_stub.cpp in place of the HIP
// runtime (every launch is checked against grid, block and LDS limits and recorded).
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
void stub_launch_reset(void);
void stub_fail_next_launch(int n);
}

static int g_checks = 0, g_failed = 0;
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

// Fake device addresses, 16 TiB apart (never dereferenced: the kernels do not run).
static void* dev(int slot) { return reinterpret_cast<void*>((uintptr_t(slot) + 1) << 44); }
static const float* fdev(int slot) { return static_cast<const float*>(dev(slot)); }
static const int32_t* idev(int slot) { return static_cast<const int32_t*>(dev(slot)); }

static void linear_attention() {
    const int64_t Ts[] = {1, 2, 63, 64, 65, 1000, 8192, 131072, int64_t(1) << 30};
    const int64_t Ns[] = {1, 2, 7, 64, 1000, 65535};
    const int64_t Hs[][2] = {{1, 1}, {4, 2}, {32, 32}, {64, 1}, {32767, 1}};
    const int64_t Ds[][2] = {{1, 1}, {64, 64}, {128, 64}, {128, 128}, {72, 40}, {256, 256}, {200, 96}};
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
                            const size_t need = ssm_linattn_fwd_workspace_bytes(&d);
                            const size_t needb = ssm_linattn_bwd_workspace_bytes(&d);
                            CHECK(need % 256 == 0 && needb % 256 == 0, "T %lld", (long long)T);
                            d.workspace = dev(30);
                            d.workspace_bytes = need;
                            stub_launch_reset();
                            int st = ssm_linattn_fwd(dev(0), dev(1), dev(2), fdev(3), idev(4), idev(5), fdev(6), dev(7),
                                                     static_cast<float*>(dev(8)), &d, nullptr);
                            CHECK(st == SSM_OK || st == SSM_ERR_DIMS, "fwd %d", st);
                            CHECK((st == SSM_OK) == (stub_launch_count() > 0), "launches %zu", stub_launch_count());
                            if (st == SSM_OK && need) {
                                d.workspace_bytes = 0;
                                // packed and dense plans share the larger size; the packed one needs some here
                                const int bad = ssm_linattn_fwd(dev(0), dev(1), dev(2), fdev(3), idev(4), nullptr, nullptr,
                                                                dev(7), nullptr, &d, nullptr);
                                CHECK(bad == SSM_ERR_WORKSPACE || bad == SSM_OK, "no workspace %d", bad);
                                d.workspace_bytes = need;
                            }
                            if (T % n == 0) {
                                st = ssm_linattn_fwd(dev(0), dev(1), dev(2), fdev(3), nullptr, nullptr, nullptr, dev(7), nullptr,
                                                     &d, nullptr);
                                CHECK(st == SSM_OK || st == SSM_ERR_DIMS, "dense %d", st);
                            }
                            d.workspace_bytes = needb;
                            for (int hd : {0, 1}) {
                                d.head_decay = hd;
                                ssm_linattn_grads g = {dev(20), dev(21), dev(22), hd ? nullptr : static_cast<float*>(dev(23)),
                                                       static_cast<float*>(dev(24))};
                                stub_launch_reset();
                                st = ssm_linattn_bwd(dev(0), dev(1), dev(2), fdev(3), idev(4), fdev(6), dev(7), fdev(9), &g, &d,
                                                     nullptr);
                                CHECK(st == SSM_OK || st == SSM_ERR_DIMS, "bwd %d", st);
                                CHECK(st != SSM_OK || needb > 0, "bwd workspace");
                            }
                            d.head_decay = 0;
                            if (T == n) {
                                stub_launch_reset();
                                st = ssm_linattn_step(dev(0), dev(1), dev(2), fdev(3), nullptr, static_cast<float*>(dev(10)),
                                                      dev(7), &d, nullptr);
                                CHECK(st == SSM_OK || st == SSM_ERR_DIMS, "step %d", st);
                                CHECK(st != SSM_OK || stub_launch_count() == 1, "step launches");
                            }
                        }
    // a failing launch is this call's error, whichever it is
    ssm_linattn_dims d;
    memset(&d, 0, sizeof(d));
    d.tokens = 8192; d.nseq = 1; d.nheads = 4; d.kheads = 2; d.dk = d.dv = 128; d.io_dtype = SSM_BF16; d.scale = 1.0f;
    d.workspace = dev(30);
    d.workspace_bytes = ssm_linattn_bwd_workspace_bytes(&d);
    ssm_linattn_grads g = {dev(20), dev(21), dev(22), static_cast<float*>(dev(23)), nullptr};
    stub_launch_reset();
    CHECK(ssm_linattn_bwd(dev(0), dev(1), dev(2), fdev(3), nullptr, nullptr, dev(7), nullptr, &g, &d, nullptr) == SSM_OK, "bwd");
    const int count = static_cast<int>(stub_launch_count());
    for (int i = 1; i <= count; ++i) {
        stub_fail_next_launch(i);
        CHECK(ssm_linattn_bwd(dev(0), dev(1), dev(2), fdev(3), nullptr, nullptr, dev(7), nullptr, &g, &d, nullptr) == SSM_ERR_HIP,
              "launch %d", i);
    }
    CHECK(ssm_linattn_bwd(dev(0), dev(1), dev(2), fdev(3), nullptr, nullptr, dev(7), nullptr, &g, &d, nullptr) == SSM_OK, "after");
}

static void norms() {
    for (int64_t rows : {int64_t(1), int64_t(3), int64_t(1000), int64_t(1) << 20, int64_t(1) << 33})
        for (int64_t n : std::initializer_list<int64_t>{1, 7, 64, 65, 512, 1536, 4096, 8192, 8193, 16384})
            for (int64_t groups : {int64_t(1), int64_t(5), int64_t(64), int64_t(1) << 20})
                for (int io : {int(SSM_F32), int(SSM_BF16)})
                    for (int flags = 0; flags < 4; ++flags) {
                        ssm_gated_norm_dims d;
                        memset(&d, 0, sizeof(d));
                        d.rows = rows; d.ngroups = groups; d.group = n; d.io_dtype = io; d.gate_first = flags & 1;
                        d.shared_weight = flags >> 1; d.eps = 1e-5f;
                        int st = ssm_gated_norm_fwd(dev(0), dev(1), fdev(2), dev(3), &d, nullptr);
                        CHECK(st == SSM_OK || st == SSM_ERR_DIMS, "gated %d", st);
                        const size_t need = ssm_gated_norm_bwd_workspace_bytes(&d);
                        CHECK((st == SSM_OK) == (need > 0), "gated workspace");
                        d.workspace = dev(30);
                        d.workspace_bytes = need;
                        // spans past the 1 TiB between the fake arrays overlap
                        const int sb = ssm_gated_norm_bwd(dev(0), dev(1), fdev(2), dev(4), dev(5), dev(6),
                                                          static_cast<float*>(dev(7)), &d, nullptr);
                        CHECK(sb == st || sb == SSM_ERR_ALIAS, "gated bwd %d", sb);
                        if (groups == 1) {
                            ssm_add_norm_dims a;
                            memset(&a, 0, sizeof(a));
                            a.rows = rows; a.dim = n; a.io_dtype = io; a.res_dtype = flags & 1 ? SSM_BF16 : SSM_F32; a.eps = 1e-6f;
                            const float* sc = flags & 1 ? fdev(8) : nullptr;
                            const float* po = flags & 2 ? fdev(9) : nullptr;
                            st = ssm_add_norm_fwd(dev(0), dev(1), sc, po, fdev(2), dev(3), dev(4), &a, nullptr);
                            CHECK(st == SSM_OK || st == SSM_ERR_DIMS, "add %d", st);
                            a.workspace = dev(30);
                            a.workspace_bytes = ssm_add_norm_bwd_workspace_bytes(&a);
                            const int sa = ssm_add_norm_bwd(dev(0), dev(1), sc, po, fdev(2), dev(3), dev(4), dev(5), dev(6),
                                                            static_cast<float*>(dev(7)), static_cast<float*>(dev(10)),
                                                            static_cast<float*>(dev(11)), &a, nullptr);
                            CHECK(sa == st, "add bwd %d", sa);
                        }
                    }
}

int main() {
    linear_attention();
    norms();
    printf("%d checks, %d failed\n", g_checks, g_failed);
    return g_failed ? 1 : 0;
}
