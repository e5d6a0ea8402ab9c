// The query/key head-row kernels for fp32.
#include "qk_rows_kernels.cuh"
