// Host-side checks of the mixer entry points under AddressSanitizer /
// UndefinedBehaviorSanitizer, without a GPU: every call gets arguments that
// its validation must refuse (or nothing to do).  The launchers abort, so a
// call that would have launched fails the run; the layer checks shared with
// the replay entry points are reduced to what these calls need.  Built with
// g++ (host code only) from mixer_api.cpp by tests/test_mixer_abi.py.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "api_common.h"
#include "mixer.h"
#include "replayssm.h"
#include "scan.h"

static char g_error[512];

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
int nslots_of(const rssm_desc *d) { return d->n_slots > 0 ? d->n_slots : d->batch; }
int split_mode(const rssm_desc *) { return -1; }
int check_desc(const rssm_desc *d) { return d ? RSSM_OK : fail(RSSM_E_ARG, "desc is NULL"); }
int check_state(const rssm_desc *, const rssm_state *s) { return s ? RSSM_OK : fail(RSSM_E_ARG, "state is NULL"); }
ReplayParams replay_params(const rssm_desc *, const rssm_state *) { return ReplayParams{}; }
}  // namespace host

#define RSSM_STUB(sig)                                                   \
    sig {                                                                \
        std::fprintf(stderr, "a kernel launch was reached: %s\n", #sig); \
        std::abort();                                                    \
    }
RSSM_STUB(hipError_t launch_conv_tokens(const ConvParams &, bool, int, bool, hipStream_t))
RSSM_STUB(hipError_t launch_conv_packed(const ConvParams &, bool, int, hipStream_t))
RSSM_STUB(hipError_t launch_conv_accept(const ConvParams &, hipStream_t))
RSSM_STUB(hipError_t launch_gated_norm(const GatedNormParams &, bool, bool, bool, hipStream_t))
RSSM_STUB(hipError_t launch_add_norm(const AddNormParams &, bool, bool, bool, hipStream_t))
RSSM_STUB(hipError_t launch_scan(const ReplayParams &, bool, bool, void *, hipStream_t))
RSSM_STUB(hipError_t launch_prefill_packed(const ReplayParams &, bool, bool, int, hipStream_t))
}  // namespace rssm

static int g_checks = 0, g_fail = 0;

static void expect(const char *what, int rc, int want) {
    ++g_checks;
    if (rc != want || (rc != RSSM_OK && !g_error[0])) {
        ++g_fail;
        std::fprintf(stderr, "FAIL %s: rc %d (want %d) '%s'\n", what, rc, want, g_error);
    }
}

int main() {
    rssm_conv_desc d{4, 0, 8, 64, 128, 2, 4, 5, RSSM_BF16, 1, 0.f, 1.f};
    rssm_conv_state st{};
    rssm_conv_io io{};
    int32_t dummy[8] = {0};
    float w[8] = {0};
    expect("desc", replayssm_conv_check_desc(&d), RSSM_OK);
    expect("null desc", replayssm_conv_check_desc(nullptr), RSSM_E_ARG);
    expect("rows of null desc", replayssm_conv_ring_rows(nullptr), 0);
    expect("rows", replayssm_conv_ring_rows(&d), 8);
    expect("null state", replayssm_conv_step(&d, nullptr, &io, nullptr), RSSM_E_ARG);
    expect("empty state", replayssm_conv_step(&d, &st, &io, nullptr), RSSM_E_ARG);
    st.ring = dummy;
    st.head = dummy;
    st.work = dummy;
    st.weight = w;
    expect("null io", replayssm_conv_step(&d, &st, nullptr, nullptr), RSSM_E_ARG);
    expect("empty io", replayssm_conv_verify(&d, &st, 2, &io, nullptr), RSSM_E_ARG);
    expect("draft count", replayssm_conv_verify(&d, &st, 6, &io, nullptr), RSSM_E_CAPACITY);
    expect("accept count", replayssm_conv_accept(&d, &st, dummy, 0, nullptr), RSSM_E_CAPACITY);
    expect("accept null", replayssm_conv_accept(&d, &st, nullptr, 1, nullptr), RSSM_E_ARG);
    expect("total", replayssm_conv_prefill(&d, &st, -5, dummy, 0, nullptr, &io, nullptr), RSSM_E_ARG);
    expect("offsets", replayssm_conv_prefill(&d, &st, 5, nullptr, 0, nullptr, &io, nullptr), RSSM_E_ARG);
    expect("nothing", replayssm_conv_prefill(&d, &st, 0, nullptr, 0, nullptr, nullptr, nullptr), RSSM_OK);
    d.n_heads = 0x7FFFFFFF;   // products in 64 bits
    d.n_groups = 1;
    expect("heads", replayssm_conv_check_desc(&d), RSSM_E_ARG);
    rssm_desc l{};
    rssm_state ls{};
    l.batch = 1;
    l.n_heads = 0x7FFFFFFF;
    expect("packed size", replayssm_prefill_packed(&l, &ls, (int64_t)1 << 31, dummy, 0, nullptr, w, w, w, w, w, 0, nullptr, 0, nullptr),
           RSSM_E_ARG);
    l.n_heads = 8;
    expect("packed huge", replayssm_prefill_packed(&l, &ls, INT64_MAX, dummy, 0, nullptr, w, w, w, w, w, 0, nullptr, 0, nullptr),
           RSSM_E_ARG);
    expect("packed null", replayssm_prefill_packed(&l, &ls, 4, dummy, 0, nullptr, nullptr, w, w, w, w, 0, nullptr, 0, nullptr),
           RSSM_E_ARG);
    expect("packed none", replayssm_prefill_packed(&l, &ls, 0, nullptr, 0, nullptr, w, w, w, w, w, 0, nullptr, 0, nullptr), RSSM_OK);
    expect("norm units", replayssm_gated_norm((int64_t)1 << 25, 16384, 16384, w, 0, w, 0, 16384, w, 0.f, 0, w, 0, nullptr),
           RSSM_E_ARG);
    expect("norm null", replayssm_gated_norm(1, 8, 1, w, 0, nullptr, 0, 8, w, 0.f, 0, w, 0, nullptr), RSSM_E_ARG);
    expect("add null", replayssm_add_norm(1, 8, w, 0, w, w, 0, nullptr, nullptr, 1.f, 0.f, w, 0, nullptr), RSSM_E_ARG);
    expect("add rows", replayssm_add_norm(INT64_MAX, 8, w, 0, w, w, 0, w, nullptr, 1.f, 0.f, w, 0, nullptr), RSSM_E_ARG);
    std::printf("%d checks, %d failed\n", g_checks, g_fail);
    return g_fail != 0;
}
