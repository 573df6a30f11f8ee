/*
 * dg_test.h -- failure-detection test hooks of libdg.so (sm_100a).
 *
 * These entry points are exported by the same library as the ones in dg.h but are not part of the
 * sampler's interface: they exist so that tests can make every bounded device-side wait of the
 * library run out on purpose, without any fault, trap or endless loop, and check that the kernel
 * gives up, reports through dg_device_error() and leaves the device usable.  Conventions (status
 * codes, dg_last_error, streams, workspaces) are those of dg.h.
 */
#ifndef DG_TEST_H_
#define DG_TEST_H_

#include "dg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* Failure-detection test hooks (the pages have no counterpart).  Every wait */
/* inside the library's kernels is bounded; these entry points make a wait  */
/* run out on purpose -- without any fault, trap or endless loop -- so that */
/* tests can check that the kernel gives up, reports through                */
/* dg_device_error() (code 1) and leaves the device usable.                 */
/* dg_test_bounded_wait: one thread waits on a barrier nothing arrives on;  */
/*   the wait gives up after limit_cycles (> 0) SM clock cycles.             */
/* dg_test_selfcond_stall: dg_selfcond with the copy of one 64-id block of  */
/*   E never issued (stalled_block >= 0, in [0, ceil(V/64)) to take effect) */
/*   and every wait limited to limit_cycles: the CTAs that need the block   */
/*   abort, drain their in-flight copies, free their tensor memory and      */
/*   return.  z is then incomplete.  Same arguments as dg_selfcond otherwise.*/
/* ------------------------------------------------------------------------ */
int dg_test_bounded_wait(uint32_t limit_cycles, dg_stream_t stream);

/* dg_test_merge_stall: the logits pass's per-row merge kernel alone (the   */
/*   statistics epilogue), with no streaming kernel writing this call's     */
/*   records: every row's wait gives up after limit_cycles (> 0), records   */
/*   device error 1, and the merge finishes on whatever the workspace holds */
/*   (lse is then meaningless).  logits as dg_sampler_step with B = 1,      */
/*   C = rows; lse: device float [rows]; workspace:                         */
/*   dg_sampler_step_workspace_size(rows, V) bytes, zeroed.                 */
int dg_test_merge_stall(const void* logits, int logits_dtype, int64_t ld, int32_t rows, int32_t V,
                        float* lse, void* workspace, size_t workspace_bytes, uint32_t limit_cycles,
                        dg_stream_t stream);

int dg_test_selfcond_stall(const void* logits, int logits_dtype, int64_t ld, int32_t B, int32_t C,
                           int32_t V, const float* inv_tau, const float* lse, const void* E,
                           int embed_dtype, int32_t d, void* z, void* workspace,
                           size_t workspace_bytes, dg_stream_t stream, int32_t stalled_block,
                           uint32_t limit_cycles);

/* dg_test_mx4_stall: dg_mx4_matmul with the copies of one 256-value block  */
/*   of K never issued (stalled_block >= 0; past the last block: none) and  */
/*   every wait limited to limit_cycles: the CTAs give up, wait for their   */
/*   copies in flight, free their tensor memory and return; out is then     */
/*   incomplete.                                                            */
/* dg_test_mx4_plan: which kernel dg_mx4_matmul takes for these sizes: the   */
/*   CTAs of a cluster that K is split over (1, 2 or 4), or 0 for pairs of   */
/*   CTAs, and the columns of a tile.  Host only.                            */
/* dg_test_block_norm_stall: dg_block_norm before a block (x contiguous, no  */
/*   y, eps 1e-6) with row 0 never fetched and every wait limited to limit_cycles,     */
/*   where the call is of the form that keeps rows in flight (many rows, at  */
/*   most 1024 16-byte vectors wide); h of the rows walked with it is then   */
/*   meaningless.                                                            */
/* dg_test_block_norm_backward_stall: dg_block_norm_backward of the same     */
/*   norm (no dx_out, no y) with the first row never fetched, where the call */
/*   keeps rows in flight (33 to 1024 16-byte vectors wide); dx of the rows  */
/*   walked with it and dw_pre are then meaningless.                         */
int dg_test_mx4_stall(const uint8_t* a, const uint8_t* a_scales, const uint8_t* w,
                      const uint8_t* w_scales, int32_t M, int32_t N, int32_t K, void* out,
                      int out_dtype, dg_stream_t stream, int32_t stalled_block,
                      uint32_t limit_cycles);

int dg_test_mx4_plan(int32_t M, int32_t N, int32_t K, int32_t* splits, int32_t* columns);

int dg_test_block_norm_stall(const void* x, int act_dtype, const void* w_pre, int param_dtype,
                             int32_t rows, int32_t d, void* h, uint32_t limit_cycles,
                             dg_stream_t stream);

int dg_test_block_norm_backward_stall(const void* dh, const void* x, int act_dtype, const void* w_pre,
                                      int param_dtype, int32_t rows, int32_t d, const float* rstd_x,
                                      void* dx, float* dw_pre, void* workspace, size_t workspace_bytes,
                                      uint32_t limit_cycles, dg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_TEST_H_ */
