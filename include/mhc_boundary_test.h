/* mhc_boundary_test.h -- test hooks of the mHC boundary library (not for
 * production use).
 *
 * Failure detection without a GPU fault: every wait in the library's
 * kernels is bounded.  A wait that gives up sets a bit of the handle's error
 * word, the kernel leaves its outputs invalid and exits, and the next
 * mhc_boundary_check_errors (or run) returns MHC_ERR_TIMEOUT; the CUDA
 * context stays usable.  This hook makes that happen on purpose.
 */
#ifndef MHC_BOUNDARY_TEST_H
#define MHC_BOUNDARY_TEST_H

#include "mhc_boundary.h"
#include "mhc_sublayer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* With on != 0, the tensor-core stage kernels and the one-kernel path for a
 * few tokens launched from now on, on the current device, issue no input
 * copies: their waits for those copies run out (after about a second) and
 * they report MHC_ERR_TIMEOUT.  on == 0
 * restores normal operation.  Affects every handle on the device; call it
 * only while no boundary call is in flight.  Returns MHC_ERR_CUDA if the
 * device flag cannot be set. */
mhc_status_t mhc_test_stall_stage_copies(int32_t on);

/* The same for the matmul and moe kernels of mhc_sublayer.h
 * (mhc_sublayer_check_errors reports). */
mhc_status_t mhc_test_stall_sublayer_copies(int32_t on);

/* The same for attend's kernel of several queries a sequence
 * (mhc_attention_check_errors reports). */
mhc_status_t mhc_test_stall_attention_copies(int32_t on);

/* frequency / 2 pi behind the point, in units of 2^-64 turns, as append's
 * angles are made of (|frequency| below 2^40).  Needs no GPU. */
uint64_t mhc_test_attention_turns(double frequency);

/* Where things lie in the shared memory of a CTA of the moe kernel, in bytes,
 * for a call of m tokens on a GPU of that many SMs.  Needs no GPU. */
typedef struct {
  int32_t size;         /* of the allocation */
  int32_t ring_at, stages, stage_bytes;
  int32_t weight_bytes; /* a stage's first part; the tokens' rows of 128 bytes follow */
  int32_t scales_at;    /* [items][scale_blocks][m] float, 8-bit weights only */
  int32_t items, scale_blocks;
} mhc_test_moe_form_t;
mhc_status_t mhc_test_moe_form(const mhc_sublayer_config_t *config, int32_t m, int32_t sms, mhc_test_moe_form_t *out);

#ifdef __cplusplus
}
#endif

#endif /* MHC_BOUNDARY_TEST_H */
