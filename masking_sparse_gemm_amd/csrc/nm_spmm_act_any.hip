// nm_spmm_act_any.hip -- nm_spmm_act's kernels: those of nm_spmm.hip with an epilogue of scale, bias, activation
// and residual (the expansion kernel, any pattern, type and shape).
#define NM_SPMM_PART 2
#include "nm_spmm.hip"
