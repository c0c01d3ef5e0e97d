// q4k_act_mfma.hip -- the products of q4k_mfma.hip with an epilogue in y's place
// (q4k_out.h): the same kernels, compiled a second time.
#define Q4K_EPILOGUE
#include "q4k_mfma.hip"
