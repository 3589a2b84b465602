// nm_spmm_act.hip -- nm_spmm_act's kernels: those of nm_spmm.hip with an epilogue of scale, bias, activation
// and residual (the matrix-core kernels).
#define NM_SPMM_PART 1
#include "nm_spmm.hip"
