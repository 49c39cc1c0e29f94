// qmat.h -- matrices in 4 bits: the launchers inside libll.so (qmat.cu). include/ll.h
// describes the format and the calls.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ll.h"

namespace ll {

constexpr int QM_TILE_ROWS = 16, QM_TILE_COLS = 128;  // a tile: 1024 bytes of codes

// All return LL_OK or LL_ERR_CUDA; arguments are already checked.
int launch_qmat_write(const ll_qmat &m, const void *w, int type, int64_t stride, cudaStream_t st);
int launch_qmat_read(const ll_qmat &m, void *w, int type, int64_t stride, cudaStream_t st);
// add: null for none.
int launch_qmat_mul(const ll_qmat &m, const ll_rows &x, int n, const ll_rows *add, const ll_rows &y, int nsm, cudaStream_t st);

// The same on tcgen05 (qmat_tc.cu); LL_ERR_SHAPE where x does not fit into shared memory (nothing was launched).
int launch_qmat_tc(const ll_qmat &m, const ll_rows &x, int n, const ll_rows *add, const ll_rows &y, int nsm, cudaStream_t st);

// The matrix's own checks (shape, pointers): LL_OK, or the code with a reason in msg.
int qmat_check(const ll_qmat *m, const char *&msg);

}  // namespace ll
