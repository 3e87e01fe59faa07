// launch_limit_checks.cpp -- every launch of the block operators has fewer than 2^32 threads
// along an axis, and at most 65535 workgroups along y and z, at the largest sizes that their
// checks let through; hip_stub.cpp stands in for the HIP runtime.  Test infrastructure only.
// Exits 0 when every check holds.
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
}

static long g_checks = 0, g_failed = 0;
static void launches(const char* what) {
    for (size_t i = 0; i < stub_launch_count(); ++i) {
        ++g_checks;
        if (uint64_t(stub_launch_grid(i)) * stub_launch_block(i) >= (uint64_t(1) << 32)) {
            ++g_failed;
            fprintf(stderr, "%s: %s: %u workgroups of %u\n", what, stub_launch_name(i), stub_launch_grid(i), stub_launch_block(i));
        }
    }
    stub_launch_reset();
}

static void* dev(int slot) { return reinterpret_cast<void*>((uintptr_t(slot) + 1) << 45); }
static float* fdev(int slot) { return static_cast<float*>(dev(slot)); }

int main() {
    for (int64_t rows : {int64_t(1), int64_t(3), int64_t(1) << 20, int64_t(1) << 40})
        for (int64_t groups : {int64_t(1), int64_t(1) << 12, int64_t(1) << 20})
            for (int64_t group : {1, 64, 4096, 16384})
                for (int shared : {0, 1}) {
                    ssm_gated_norm_dims d;
                    memset(&d, 0, sizeof(d));
                    d.rows = rows; d.ngroups = groups; d.group = group; d.io_dtype = SSM_BF16; d.shared_weight = shared; d.eps = 1e-5f;
                    d.workspace = dev(30);
                    d.workspace_bytes = ssm_gated_norm_bwd_workspace_bytes(&d);
                    ssm_gated_norm_fwd(dev(0), dev(1), fdev(2), dev(3), &d, nullptr);
                    ssm_gated_norm_bwd(dev(0), dev(1), fdev(2), dev(4), dev(5), dev(6), fdev(7), &d, nullptr);
                    launches("gated norm");
                    if (groups > 1) continue;
                    ssm_add_norm_dims a;
                    memset(&a, 0, sizeof(a));
                    a.rows = rows; a.dim = group; a.io_dtype = SSM_BF16; a.res_dtype = SSM_F32; a.eps = 1e-5f;
                    a.workspace = dev(30);
                    a.workspace_bytes = ssm_add_norm_bwd_workspace_bytes(&a);
                    ssm_add_norm_fwd(dev(0), dev(1), fdev(8), fdev(9), fdev(2), dev(3), dev(4), &a, nullptr);
                    ssm_add_norm_bwd(dev(0), dev(1), fdev(8), fdev(9), fdev(2), dev(3), dev(4), dev(5), dev(6), fdev(7), fdev(10),
                                     fdev(11), &a, nullptr);
                    launches("residual norm");
                }
    for (int64_t tokens : {int64_t(1), int64_t(65535), int64_t(1) << 24, (int64_t(1) << 31) - 1})
        for (int64_t nseq : {int64_t(1), int64_t(4000), int64_t(65535)})
            for (int64_t heads : {1, 16, 128, 32767})
                for (int64_t dk : {1, 128, 256})
                    for (int64_t piece : {0, 64}) {
                        ssm_linattn_dims d;
                        memset(&d, 0, sizeof(d));
                        d.tokens = tokens; d.nseq = nseq; d.nheads = heads; d.kheads = 1; d.dk = dk; d.dv = dk; d.io_dtype = SSM_BF16;
                        d.piece_len = piece; d.nslots = nseq; d.scale = 1.0f;
                        d.workspace = dev(30);
                        d.workspace_bytes = ssm_linattn_fwd_workspace_bytes(&d);
                        const int32_t* cu = static_cast<const int32_t*>(dev(4));
                        ssm_linattn_fwd(dev(0), dev(1), dev(2), fdev(3), cu, nullptr, fdev(6), dev(7), fdev(8), &d, nullptr);
                        d.workspace_bytes = ssm_linattn_bwd_workspace_bytes(&d);
                        ssm_linattn_grads g = {dev(20), dev(21), dev(22), fdev(23), fdev(24)};
                        ssm_linattn_bwd(dev(0), dev(1), dev(2), fdev(3), cu, fdev(6), dev(7), fdev(9), &g, &d, nullptr);
                        if (tokens == nseq)
                            ssm_linattn_step(dev(0), dev(1), dev(2), fdev(3), nullptr, fdev(10), dev(7), &d, nullptr);
                        launches("linear attention");
                    }
    printf("%ld checks, %ld failed\n", g_checks, g_failed);
    return g_failed || g_checks < 1000 ? 1 : 0;
}
