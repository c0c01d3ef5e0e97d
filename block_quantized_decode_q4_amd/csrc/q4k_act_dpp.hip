// q4k_act_dpp.hip -- the products of q4k_dpp.hip with an epilogue in y's place
// (q4k_out.h): the same kernels, compiled a second time.
// One token, 14336 x 4096 with silu and gate: 10.5 us a launch, 33 MB at 3.1 TB/s (floor
// 6.5); the conversion of x stands in front of the stream.
#define Q4K_EPILOGUE
#include "q4k_dpp.hip"
