// delta_limit_checks.cpp -- the gated delta rule takes every size within the limits that ssm.h
// names, and refuses what lies past them; hip_stub.cpp stands in for the HIP runtime.  Test
// infrastructure only.  Exits 0 when every check holds.
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
static void* dev(int slot) { return reinterpret_cast<void*>((uintptr_t(slot) + 1) << 45); }
static float* fdev(int slot) { return static_cast<float*>(dev(slot)); }

static int run(ssm_linattn_dims d, const int32_t* cu, bool back) {
    const ssm_delta_grads g = {dev(20), dev(21), dev(22), fdev(23), fdev(24), nullptr};
    d.workspace = dev(30);
    stub_launch_reset();
    int st;
    if (back) {
        d.workspace_bytes = ssm_delta_bwd_workspace_bytes(&d);
        st = ssm_delta_bwd(dev(0), dev(1), dev(2), fdev(3), fdev(4), cu, nullptr, dev(8), nullptr, &g, &d, nullptr);
    } else {
        d.workspace_bytes = ssm_delta_fwd_workspace_bytes(&d);
        st = ssm_delta_fwd(dev(0), dev(1), dev(2), fdev(3), fdev(4), cu, nullptr, nullptr, dev(8), nullptr, &d, nullptr);
    }
    for (size_t i = 0; i < stub_launch_count(); ++i) {
        ++g_checks;
        if (uint64_t(stub_launch_grid(i)) * stub_launch_block(i) < (uint64_t(1) << 32)) continue;
        ++g_failed;
        fprintf(stderr, "%s: %u workgroups of %u\n", stub_launch_name(i), stub_launch_grid(i), stub_launch_block(i));
    }
    return st;
}

// heads, keys, values, sequences, tokens, piece_len; whether the forward and the gradients take it
struct Size {
    int64_t h, dk, dv, n, t, piece;
    bool fwd, bwd;
};

int main() {
    const Size sizes[] = {
        {32, 128, 128, 40000, 40000, 0, true, true},         // one token each
        {32, 128, 128, 40000, 4000000, 0, true, true},
        {64, 128, 128, 65535, 65535, 0, true, false},        // 2^23 workgroups less two a head; the gradients twice that
        {64, 16, 16, 65535, 65535, 0, true, true},
        {65, 16, 16, 65535, 65535, 0, true, false},
        {128, 64, 64, 65535, 65535, 0, true, false},
        {129, 64, 64, 65535, 65535, 0, false, false},
        {32, 256, 256, 65535, 65535, 0, true, false},
        {33, 256, 256, 65535, 65535, 0, false, false},
        {16383, 256, 256, 128, 128, 0, true, false},
        {16383, 256, 256, 64, 64, 0, true, true},
        {16383, 256, 256, 32, 4096, 0, true, true},
        // 65535 pieces and 4 (gradients: 6) slices of a head
        {32, 128, 128, 1, int64_t(65534) * 64, 64, true, false},
        {21, 128, 128, 1, int64_t(65534) * 64, 64, true, true},
        {33, 128, 128, 1, int64_t(65535) * 64, 64, false, false},
        {128, 128, 128, 8192, 524288, 64, true, false},      // up to 16384 pieces
        {32, 128, 128, 40000, 40000, 64, true, true},
        {64, 128, 128, 40000, 40000, 64, false, false},
        {1, 1, 1, 1, (int64_t(1) << 28) - 64, 0, true, false},
        {1, 1, 1, 1, (int64_t(1) << 27) - 64, 0, true, true},
        {1, 1, 1, 1, int64_t(1) << 28, 0, false, false},
    };
    for (const Size& s : sizes)
        for (int io : {int(SSM_F32), int(SSM_BF16)})
            for (const bool packed : {true, false})
                for (const bool back : {false, true}) {
                    if (!packed && s.t % s.n != 0) continue;
                    ssm_linattn_dims d;
                    memset(&d, 0, sizeof(d));
                    d.tokens = s.t; d.nseq = s.n; d.nheads = d.kheads = s.h; d.dk = s.dk; d.dv = s.dv;
                    d.io_dtype = io; d.piece_len = s.piece; d.scale = 1.0f;
                    const bool want = back ? s.bwd : s.fwd;
                    // equal sequences have fewer pieces and blocks than packed ones may, and blocks of 64 are half as many
                    const bool less = (!packed && (s.piece || s.n == 1)) || (back && io == SSM_BF16 && s.dk == 1);
                    const int st = run(d, packed ? static_cast<const int32_t*>(dev(5)) : nullptr, back);
                    ++g_checks;
                    if (st == (want ? SSM_OK : SSM_ERR_DIMS) || (less && st == SSM_OK)) continue;
                    ++g_failed;
                    fprintf(stderr, "%s of %lld heads of %lld x %lld, %lld sequences, %lld tokens, pieces of %lld, type %d, packed %d: %d\n",
                            back ? "gradients" : "forward", (long long)s.h, (long long)s.dk, (long long)s.dv, (long long)s.n, (long long)s.t,
                            (long long)s.piece, io, int(packed), st);
                }
    printf("%ld checks, %ld failed\n", g_checks, g_failed);
    return g_failed ? 1 : 0;
}
