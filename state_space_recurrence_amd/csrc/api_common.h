// api_common.h -- host-side pieces shared by the C entry points: the calling
// thread's last error, status mapping and the checks of the layer structs.
#pragma once

#include <hip/hip_runtime.h>

#include "kernels.h"
#include "replayssm.h"

namespace rssm {
namespace host {

// Clear the calling thread's last error (entry points that cannot fail later).
void clear_error();
// Record a message for replayssm_last_error() and return `status`.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// RSSM_OK, or RSSM_E_HIP with the runtime's message.
int hip_status(hipError_t e, const char *what);

int nslots_of(const rssm_desc *d);   // state slots held by the buffers
int split_mode(const rssm_desc *d);  // SplitMode of a low-precision layer, -1 for an fp32 checkpoint
int check_desc(const rssm_desc *d);
int check_state(const rssm_desc *d, const rssm_state *s);
ReplayParams replay_params(const rssm_desc *d, const rssm_state *s);

}  // namespace host
}  // namespace rssm

#define RSSM_TRY(expr)              \
    do {                            \
        int rc_ = (expr);           \
        if (rc_ != RSSM_OK) return rc_; \
    } while (0)
