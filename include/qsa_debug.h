/*
 * qsa_debug.h -- test hooks of the debug build of the QSA library
 * (libqsa_debug.so, built from the same sources with QSA_DEBUG_BOUNDS,
 * QSA_DEBUG_HOOKS and a 20 ms device wait limit).  The pages have no
 * counterpart: these exist to test the library's own failure handling.  The
 * release library (libqsa.so) does not export them.
 *
 * In the debug build:
 *   - every bounded device wait gives up after 20 ms instead of 2 s;
 *   - the attention kernels check that every selected block index is -1
 *     (padding) or a causal block 0 .. qb of the query block, and the
 *     indexer checks every score and segment-maximum store against the
 *     output's row range and leading dimension; a failed check records
 *     QSA_ERR_DEVICE_BOUNDS (read with qsa_check_device_error) and the access
 *     is skipped;
 *   - qsa_debug_inject arms one fault (or, for QSA_INJECT_ATTENTION_RESCALE_ALL,
 *     one change of schedule that leaves the result within rounding of the
 *     normal one) for the next launch of the kernel it names.  The faults make no out-of-range access and leave no wait
 *     unbounded: a stall withholds one completion signal, so a waiting role
 *     times out, records QSA_ERR_DEVICE_TIMEOUT and the CTA drains what it
 *     issued and exits; a bad block names a block after the query block,
 *     which the bounds check reports (and the causal test masks).
 */
#ifndef QSA_DEBUG_H_
#define QSA_DEBUG_H_

#include <stdint.h>

#include "qsa.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  QSA_INJECT_NONE = 0,
  QSA_INJECT_INDEXER_STALL = 1,        /* next indexer launch: CTA 0 never signals its first accumulator */
  QSA_INJECT_ATTENTION_STALL = 2,      /* next prefill attention launch: CTA 0 never signals its first S tile */
  QSA_INJECT_ATTENTION_BAD_BLOCK = 3,  /* next prefill attention launch: CTA 0's first gathered block is qb + 1 */
  QSA_INJECT_PAGED_STALL = 5,          /* next qsa_paged_prefill: no CTA signals its first S tile */
  QSA_INJECT_ATTENTION_RESCALE_ALL = 4 /* next attention launch (prefill or decode): the online softmax takes a
                                          new running maximum, and rescales the accumulated output, on every tile
                                          (no lazy margin), so that path runs on ordinary inputs */
};

/* Arms `code` for the next launch of the kernel it names (one launch; a new
 * call replaces an armed code).  QSA_ERR_INVALID_ARG for an unknown code. */
qsa_status qsa_debug_inject(int32_t code);

/* The rope_dim / 2 rotary frequencies of a layer (host array), YaRN included. */
qsa_status qsa_debug_rope_frequencies(const qsa_layer_params* p, double* f);

/* The index arithmetic that the paged-cache kernels use, on the host: j /
 * page_size; the first unit of CTA c, and the CTA of unit u, of `total` units cut
 * evenly over `parts` CTAs; the first tile slot of a sequence of the prefill
 * (`per` query rows a token, `rows` of them to a tile). */
uint32_t qsa_debug_page_of(int32_t page_size, uint32_t j);
int64_t qsa_debug_cut_begin(int64_t total, int64_t parts, int64_t c);
int64_t qsa_debug_cut_owner(int64_t total, int64_t parts, int64_t u);
int32_t qsa_debug_first_tile_slot(int32_t seq, int32_t row, int32_t T, uint32_t per, uint32_t rows);

#ifdef __cplusplus
}
#endif
#endif /* QSA_DEBUG_H_ */
