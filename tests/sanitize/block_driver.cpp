// Drives the host code of the gated linear recurrence, the projections and the clipping of
// gradients (include/ssm_scan.h), built with AddressSanitizer and UndefinedBehaviorSanitizer
// (test infrastructure: tests/test_block_sanitize_cpu.py compiles and runs it). The HIP runtime is
// not linked: launches end in the functions below, which check that a launch's shape is one that
// the hardware takes. Device addresses are made up; host code never reads through them.
//
// Descriptors come from values at which sizes, pieces and byte counts change or overflow, in
// seeded random combinations, most of which are refused. Whatever a call answers, its arithmetic
// must be clean; what it accepts must launch, and with a byte less of workspace be refused.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "ssm_scan.h"

namespace {

int failures = 0;
int64_t launches = 0;
dim3 grid_now, block_now;

void fail(const char *what, long long a = 0, long long b = 0, long long c = 0, long long d = 0) {
    if (++failures < 20) fprintf(stderr, "FAILED: %s %lld %lld %lld %lld\n", what, a, b, c, d);
}

uint64_t seed = 12345;
uint32_t rnd(uint32_t n) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(seed >> 33) % n;
}

const int64_t kSmall[] = {1, 2, 3, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4095, 4096, 4097};
const int64_t kAll[] = {0, -1, 65535, 65536, (int64_t)1 << 20, ((int64_t)1 << 22) - 1, (int64_t)1 << 22, ((int64_t)1 << 24) - 1,
                        (int64_t)1 << 24, INT32_MAX, (int64_t)1 << 31, (int64_t)1 << 32, (int64_t)1 << 37, ((int64_t)1 << 37) + 1,
                        (int64_t)1 << 38, (int64_t)1 << 57, INT64_MAX / 64, INT64_MAX / 2, INT64_MAX, INT64_MIN};
template <size_t N> int64_t one(const int64_t (&v)[N]) { return v[rnd(N)]; }
int64_t size() { return rnd(4) ? one(kSmall) : one(kAll); }

// Addresses 2^43 apart
char *at(int k) { return reinterpret_cast<char *>((uintptr_t)(k + 1) << 43); }
float *fat(int k) { return reinterpret_cast<float *>(at(k)); }
// one in eight is moved off its alignment, one in eight missing
char *some(int k) {
    const uint32_t r = rnd(24);
    return r == 0 ? nullptr : r == 1 ? at(k) + 1 : r < 4 ? at(k) + 4 : at(k);
}

bool known(int rc) { return rc <= 0 && rc >= SSM_ERR_SCRATCH && rc != SSM_ERR_HIP; }

// A call with the workspace that it asks for, and one with a byte less
template <typename F> void both(const char *what, size_t need, bool writes, F call) {
    const int64_t before = launches;
    const int rc = call(at(15), need);
    if (!known(rc)) fail(what, rc);
    if (rc == SSM_OK && writes && launches == before) fail("nothing launched", rc);
    if (rc != SSM_OK && launches != before) fail("refused after a launch", rc);
    if (rc == SSM_OK && need > 0 && call(at(15), need - 1) != SSM_ERR_WORKSPACE) fail("a byte less was taken", (long long)need);
}

void recurrence() {
    ssm_glr_desc d;
    memset(&d, 0, sizeof d);
    d.batch = size();
    d.seqlen = size();
    d.dim = size();
    d.dtype = rnd(20) ? (rnd(2) ? SSM_BF16 : SSM_F32) : 7;
    const float rates[] = {8.0f, 0.0f, 1e-30f, -1.0f, 1e38f, __builtin_inff(), __builtin_nanf("")};
    d.rate = rnd(8) ? 8.0f : rates[rnd(7)];
    int64_t *const strides[] = {&d.x_stride, &d.rgate_stride, &d.igate_stride, &d.gate_stride};
    for (int64_t *s : strides) *s = rnd(3) ? 0 : rnd(2) ? d.dim : size();
    const size_t fwd = ssm_glr_workspace_size(&d), bwd = ssm_glr_bwd_workspace_size(&d);
    const bool some_tokens = d.batch > 0 && d.seqlen > 0;
    char *x = some(0), *r = some(1), *i = some(2), *gate = rnd(2) ? some(3) : nullptr;
    float *lam = (float *)some(4), *h0 = rnd(2) ? (float *)some(5) : nullptr;
    uint8_t *reset = rnd(3) ? nullptr : (uint8_t *)at(6);
    char *y = some(7);
    float *hl = rnd(8) ? (rnd(4) ? fat(8) : h0) : (float *)some(7);
    both("glr fwd", fwd, some_tokens, [&](void *ws, size_t n) { return ssm_glr_fwd(&d, x, r, i, lam, h0, gate, reset, y, hl, ws, n, nullptr); });
    both("glr fwd_save", bwd, some_tokens, [&](void *ws, size_t n) { return ssm_glr_fwd_save(&d, x, r, i, lam, h0, gate, reset, y, hl, ws, n, nullptr); });
    char *dy = some(7), *dx = some(8), *dr = some(9), *di = some(10), *dg = rnd(2) ? at(11) : some(12);
    float *dl = (float *)some(12), *dh = rnd(2) ? fat(13) : nullptr, *dh0 = rnd(3) ? fat(14) : dh;
    both("glr bwd", bwd, some_tokens, [&](void *ws, size_t n) { return ssm_glr_bwd(&d, x, r, i, lam, h0, gate, reset, dy, dh, dx, dr, di, dg, dl, dh0, ws, n, nullptr); });
    both("glr bwd_saved", bwd, some_tokens, [&](void *ws, size_t n) { return ssm_glr_bwd_saved(&d, x, r, i, lam, h0, gate, reset, dy, dh, dx, dr, di, dg, dl, dh0, ws, n, nullptr); });
    if (rnd(2)) d.seqlen = 1;
    float *ho = rnd(2) ? h0 : fat(8);
    both("glr step", 0, d.batch > 0, [&](void *, size_t) { return ssm_glr_state_update(&d, x, r, i, lam, gate, reset, h0, ho, y, nullptr); });
}

void projection() {
    ssm_proj_desc d;
    memset(&d, 0, sizeof d);
    d.rows = size();
    d.groups = rnd(3) ? 1 : size();
    d.in = size();
    d.out = size();
    d.dtype = rnd(20) ? (rnd(2) ? SSM_BF16 : SSM_F32) : 7;
    d.y_dtype = rnd(3) ? d.dtype : SSM_F32;
    d.activation = rnd(20) ? (int)rnd(4) : 9;
    d.reserved = rnd(40) == 0;
    d.x_stride = rnd(3) ? 0 : size();
    const size_t fwd = ssm_proj_workspace_size(&d), bwd = ssm_proj_bwd_workspace_size(&d);
    char *x = some(0), *w = some(1), *res = rnd(2) ? some(3) : nullptr, *pre = rnd(2) ? some(4) : nullptr, *y = rnd(4) ? some(5) : res;
    float *bias = rnd(2) ? (float *)some(2) : nullptr;
    both("proj fwd", fwd, d.rows > 0, [&](void *ws, size_t n) { return ssm_proj_fwd(&d, x, w, bias, res, pre, y, ws, n, nullptr); });
    char *dy = some(5), *dpre = some(6), *dx = rnd(3) ? some(7) : nullptr, *dw = rnd(3) ? some(8) : nullptr;
    float *db = rnd(2) ? fat(9) : nullptr;
    both("proj bwd", bwd, d.rows > 0 && (dx || dw || db), [&](void *ws, size_t n) { return ssm_proj_bwd(&d, dy, x, w, pre, dpre, dx, dw, db, ws, n, nullptr); });
}

void clipping() {
    enum { kMost = 300 };
    const void *in[kMost];
    void *out[kMost];
    int64_t n[kMost];
    int32_t t[kMost];
    const int64_t count = rnd(30) ? 1 + rnd(kMost) : (rnd(2) ? 0 : one(kAll));
    const int64_t most = (int64_t)1 << 35;
    bool any = false;
    const bool plain = rnd(2);
    uintptr_t next = (uintptr_t)1 << 43;
    for (int k = 0; k < kMost; ++k) {
        n[k] = plain || rnd(200) ? (rnd(50) ? one(kSmall) : rnd(2) ? 0 : most) : one(kAll);
        t[k] = plain || rnd(200) ? (rnd(2) ? SSM_BF16 : SSM_F32) : 5;
        in[k] = reinterpret_cast<void *>(next);
        out[k] = rnd(2) ? const_cast<void *>(in[k]) : reinterpret_cast<void *>(next + ((uintptr_t)1 << 38));
        if (!plain && rnd(200) == 0) out[k] = some(2);
        next += (uintptr_t)1 << 39;
        any = any || (k < count && n[k] > 0);
    }
    const size_t need = ssm_grad_workspace_size(count);
    if (count > kMost && count <= (1 << 20)) return;      // the arrays here are shorter
    if (count > kMost || count < 0) {
        if (ssm_grad_norm(count, in, n, t, fat(0), at(1), need, nullptr) != SSM_ERR_SHAPE) fail("count", count);
        return;
    }
    void *ws = reinterpret_cast<void *>((uintptr_t)1 << 42);
    float *norm = reinterpret_cast<float *>((uintptr_t)1 << 41);
    const float limits[] = {1.0f, 0.0f, -1.0f, __builtin_inff(), __builtin_nanf("")};
    const float limit = rnd(4) ? 1.0f : limits[rnd(5)];
    both("norm", need, true, [&](void *, size_t b) { return ssm_grad_norm(count, in, n, t, norm, ws, b, nullptr); });
    both("clip", need, true, [&](void *, size_t b) { return ssm_grad_clip(count, in, out, n, t, limit, 1e-6f, norm, ws, b, nullptr); });
    both("scale", 0, any, [&](void *, size_t) { return ssm_grad_scale(count, in, out, n, t, norm, limit, 1e-6f, nullptr); });
}

}  // namespace

// The runtime's part, as the compiler calls it
extern "C" {
void **__hipRegisterFatBinary(const void *) {
    static void *handle;
    return &handle;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *, int *) {}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t, hipStream_t) {
    grid_now = g;
    block_now = b;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *shared, hipStream_t *stream) {
    *g = grid_now;
    *b = block_now;
    *shared = 0;
    *stream = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *, dim3 g, dim3 b, void **, size_t, hipStream_t) {
    ++launches;
    const uint64_t items = (uint64_t)g.x * b.x;
    if (!g.x || !g.y || !g.z || items > UINT32_MAX || g.y > 65535 || g.z > 65535 || b.x * b.y * b.z > 1024 || b.x % 64)
        fail("launch", g.x, g.y, b.x, b.y);
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
}

int main() {
    for (int k = 0; k < 60000; ++k) recurrence();
    for (int k = 0; k < 60000; ++k) projection();
    for (int k = 0; k < 1500; ++k) clipping();
    if (launches < 50000) fail("too few calls were accepted", launches);
    if (failures) return 1;
    printf("all calls clean, %lld launches\n", (long long)launches);
    return 0;
}
