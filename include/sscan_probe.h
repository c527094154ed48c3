/*
 * sscan_probe.h -- diagnostics shipped with libsscan: a throughput probe for the
 * MUFU ex2 pipe, the unit that bounds the selective-scan forward pass (N
 * exponentials per element for Abar = exp(delta A), eq. (2) of the Mamba technical
 * summary page, sec. 2.1), and a self-test of the kernels' bounded-wait failure
 * reporting.  Neither computes anything of the scan; neither has a counterpart on
 * the pages.
 */
#ifndef SSCAN_PROBE_H
#define SSCAN_PROBE_H

#include <stdint.h>

#include "sscan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Enqueue `blocks` x `threads` threads, each issuing `iters` rounds of 8
 * independent ex2.approx.ftz.f32 (8 * iters exponentials per thread), and store
 * one float per thread to `sink` (device, blocks * threads floats, caller-owned)
 * so the work is not removed.  Returns SSCAN_ERR_INVALID_ARG for non-positive
 * sizes or a NULL sink, SSCAN_ERR_CUDA if the launch fails.
 */
SSCAN_API sscan_status sscan_probe_ex2(float* sink, int64_t iters, int blocks, int threads, void* stream);

/*
 * Exercise the failure path of the kernels' bounded waits: enqueue one thread that
 * waits, polling at most `polls` times (1 .. 2^20), on a shared-memory mbarrier
 * that nothing arrives on, then sets bit 2 of the device status word read by
 * sscan_device_status.  Nothing is in flight on the barrier, so the kernel simply
 * returns and the context stays usable.  Returns SSCAN_ERR_INVALID_ARG for polls
 * out of range, SSCAN_ERR_CUDA if the launch fails.
 */
SSCAN_API sscan_status sscan_probe_wait_timeout(unsigned int polls, void* stream);

/*
 * The same for the waits of the layers around the scan, each through the kernels' own code, on words, a flag
 * or a barrier that nothing sets: the gated recurrence's wait for earlier tiles (three waits of `polls` polls),
 * the multi-head forward's for the state an earlier segment hands on, and its tcgen05 form's for a copy or product
 * (with the bounded drain that follows it).  Each sets bit 2 of the device status word.
 */
#define SSCAN_WAIT_CARRY 0
#define SSCAN_WAIT_HANDED_STATE 1
#define SSCAN_WAIT_PRODUCT 2
SSCAN_API sscan_status sscan_probe_layer_wait_timeout(int wait, unsigned int polls, void* stream);


/*
 * A test of the debug build's index checks (sscan_debug_bounds): from now on they take every array to be `elements`
 * (0 .. 2^20) shorter than it is, so that accesses to its last elements are reported as bad and skipped.  No access
 * leaves its array; results are incomplete until the number is 0 again.  Synchronous, for the current
 * device.  The release build returns SSCAN_ERR_UNSUPPORTED.
 */
SSCAN_API sscan_status sscan_debug_shorten(int64_t elements);

#ifdef __cplusplus
}
#endif

#endif /* SSCAN_PROBE_H */
