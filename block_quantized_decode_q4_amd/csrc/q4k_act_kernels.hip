// q4k_act_kernels.hip -- the products of q4k_kernels.hip with an epilogue in y's place
// (q4k_out.h): the same kernels, compiled a second time.
// One token, 4096 x 4096 with bias and residual: 7.1 us a launch (9.4 MB; a launch, x's
// stage and one row's latency).
#define Q4K_EPILOGUE
#include "q4k_kernels.hip"
