// Host-side checks of the projections' entry points under AddressSanitizer /
// UndefinedBehaviorSanitizer, without a GPU: the launchers only count, so calls
// that are to be accepted and calls that are to be refused are both seen, at
// sizes and pitches of any kind.  Built with g++ (host code only) from
// linear_api.cpp by tests/test_linear_host.py.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "api_common.h"
#include "linear.h"
#include "mixer.h"
#include "replayssm.h"

static char g_error[512];
static int g_launched, g_failed;

namespace rssm {
namespace host {
void clear_error() { g_error[0] = 0; }
int fail(int status, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return status;
}
int hip_status(hipError_t e, const char *what) { return e == hipSuccess ? RSSM_OK : fail(RSSM_E_HIP, "%s", what); }
}  // namespace host

static hipError_t count() {
    ++g_launched;
    return hipSuccess;
}
hipError_t launch_linear(const LinearParams &, bool, bool, hipStream_t) { return count(); }
hipError_t launch_gated_norm_mx(const GatedNormParams &, bool, bool, hipStream_t) { return count(); }
hipError_t launch_add_norm_mx(const AddNormParams &, bool, bool, hipStream_t) { return count(); }
hipError_t launch_quantize(const QuantizeParams &, bool, hipStream_t) { return count(); }
}  // namespace rssm

static void *at(uint64_t v) { return reinterpret_cast<void *>(static_cast<uintptr_t>(v)); }
static uint8_t *bytes(uint64_t v) { return static_cast<uint8_t *>(at(v)); }
static float *floats(uint64_t v) { return static_cast<float *>(at(v)); }

static void expect(const char *what, int rc, bool taken) {
    if ((rc == RSSM_OK) != taken || g_launched != (taken ? 1 : 0)) {
        std::printf("%s: status %d (%s), %d launches\n", what, rc, g_error, g_launched);
        ++g_failed;
    }
    g_launched = 0;
    g_error[0] = 0;
}

constexpr uint64_t kFar = 1ull << 36;

// A product of `rows` x 64 inputs and 96 outputs in bf16 with these places of x and out.
static int product(int64_t rows, int64_t pitch, uint64_t x, uint64_t out, uint64_t res, int32_t res_dtype, int32_t out_dtype) {
    rssm_linear_desc d{rows, 64, 96, RSSM_BF16, out_dtype, res_dtype, 0, 1.f, 0};
    rssm_linear_io io{at(x), pitch, nullptr, at(2 * kFar), nullptr, floats(3 * kFar), at(res), at(out), bytes(4 * kFar)};
    return replayssm_linear(&d, &io, nullptr);
}

int main() {
    const uint64_t X = kFar, R = 5 * kFar, O = 6 * kFar;
    expect("apart", product(4, 64, X, O, 0, RSSM_NONE, RSSM_BF16), true);
    expect("right behind x", product(4, 64, X, X + 512, 0, RSSM_NONE, RSSM_BF16), true);
    expect("right before x", product(4, 64, X, X - 768, 0, RSSM_NONE, RSSM_BF16), true);
    expect("one element into x", product(4, 64, X, X + 510, 0, RSSM_NONE, RSSM_BF16), false);
    expect("between rows", product(4, 1024, X, X + 128, 0, RSSM_NONE, RSSM_BF16), true);
    expect("up to the next row", product(4, 448, X, X + 128, 0, RSSM_NONE, RSSM_BF16), true);
    expect("into the next row", product(4, 447, X, X + 128, 0, RSSM_NONE, RSSM_BF16), false);
    expect("behind the last strided row", product(4, 1024, X, X + 3 * 2048 + 128, 0, RSSM_NONE, RSSM_BF16), true);
    expect("onto the residual", product(4, 64, X, R, R, RSSM_BF16, RSSM_BF16), true);
    expect("onto a residual of another type", product(4, 64, X, R, R, RSSM_F32, RSSM_BF16), false);
    expect("beside the residual's start", product(4, 64, X, R + 2, R, RSSM_BF16, RSSM_BF16), false);
    expect("behind the residual", product(4, 64, X, R + 768, R, RSSM_BF16, RSSM_BF16), true);
    expect("the most rows", product((int64_t)1 << 26, 64, X, (uint64_t)1 << 46, 0, RSSM_NONE, RSSM_F32), true);
    expect("the most rows, the last over x", product((int64_t)1 << 26, 64, X + ((uint64_t)1 << 40), X + ((uint64_t)1 << 40) - ((uint64_t)1 << 26) * 384 + 4, 0,
                                                     RSSM_NONE, RSSM_F32), false);
    rssm_linear_desc d{4, 64, 96, RSSM_FP8_E4M3, RSSM_FP8_E4M3, RSSM_NONE, 0, 1.f, 1};
    rssm_linear_io io{at(X), 64, bytes(2 * kFar), at(3 * kFar), bytes(4 * kFar), nullptr, nullptr, at(O), bytes(R)};
    expect("8-bit rows", replayssm_linear(&d, &io, nullptr), true);
    io.out_scales = bytes(6 * kFar + 4 * 96);
    expect("scales behind their codes", replayssm_linear(&d, &io, nullptr), true);
    io.out_scales = bytes(6 * kFar + 4 * 96 - 1);
    expect("scales over their codes", replayssm_linear(&d, &io, nullptr), false);
    io.out_scales = bytes(2 * kFar + 7);
    expect("scales over those of x", replayssm_linear(&d, &io, nullptr), false);

    for (int64_t pitch : {(int64_t)64, (int64_t)1 << 40, (int64_t)1 << 62, INT64_MAX}) {
        expect("quantize", replayssm_quantize_mx(4, 64, at(X), RSSM_F32, pitch, at(X + 1024 + (pitch > 64 ? 256 : 0)), bytes(O), nullptr), true);
        expect("quantize in place", replayssm_quantize_mx(4, 64, at(X), RSSM_F32, pitch, at(X), bytes(O), nullptr), false);
        expect("gated", replayssm_gated_norm_mx(4, 64, 2, at(R), RSSM_F32, at(X), RSSM_F32, pitch, floats(3 * kFar), 0.f, 1,
                                                at(X + 1024), bytes(O), nullptr), true);
        expect("gated, over z", replayssm_gated_norm_mx(4, 64, 2, at(R), RSSM_F32, at(X), RSSM_F32, pitch, floats(3 * kFar), 0.f, 1,
                                                        at(X + 240), bytes(O), nullptr), false);
    }
    expect("quantize, the most", replayssm_quantize_mx((int64_t)1 << 24, 1 << 17, at(X), RSSM_F32, 1 << 17, at((uint64_t)1 << 50), bytes(1ull << 52), nullptr), true);
    const auto add = [&](uint64_t x, uint64_t res, uint64_t sum, int32_t xt, uint64_t codes) {
        return replayssm_add_norm_mx(4, 64, at(x), xt, at(res), at(sum), RSSM_F32, floats(3 * kFar), nullptr, 1.f, 0.f, at(codes), bytes(4 * kFar), nullptr);
    };
    expect("add", add(X, R, O, RSSM_BF16, 7 * kFar), true);
    expect("add onto the residual", add(X, R, R, RSSM_BF16, 7 * kFar), true);
    expect("add onto x", add(X, R, X, RSSM_F32, 7 * kFar), true);
    expect("add onto x of another type", add(X, R, X, RSSM_BF16, 7 * kFar), false);
    expect("add beside x", add(X, R, X + 4, RSSM_F32, 7 * kFar), false);
    expect("add, x and residual the same", add(R, R, R, RSSM_F32, 7 * kFar), true);
    expect("codes behind the sum", add(X, R, O, RSSM_F32, O + 1024), true);
    expect("codes over the sum", add(X, R, O, RSSM_F32, O + 1008), false);
    expect("no x", replayssm_add_norm_mx(4, 64, nullptr, -7, at(R), nullptr, RSSM_BF16, floats(3 * kFar), nullptr, 1.f, 0.f, at(R + 512), bytes(R - 8), nullptr), true);
    std::printf("%d failed\n", g_failed);
    return g_failed != 0;
}
