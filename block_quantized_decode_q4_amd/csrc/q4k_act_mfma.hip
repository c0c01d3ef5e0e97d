// q4k_act_mfma.hip -- the products of q4k_mfma.hip with an epilogue in y's place
// (q4k_out.h): the same kernels, compiled a second time.
// Eight vectors, 4096 x 14336, onto a residual: 39.6 us a call (floor 6.6 for the 33 MB).
// Bound by the conversion of x, which each of the 256 workgroups does for itself: 6200
// vector instructions a wave, the vector pipe busy 53 %, two waves a SIMD.
#define Q4K_EPILOGUE
#include "q4k_mfma.hip"
