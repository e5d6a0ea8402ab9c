// The query/key head-row kernels for bf16.
#define QK_ROWS_BF16
#include "qk_rows_kernels.cuh"
