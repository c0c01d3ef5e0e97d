// q4k_act_grouped.hip -- the products of q4k_grouped.hip with an epilogue in y's place
// (q4k_out.h): the same kernels, compiled a second time.
// 16 tokens, 8 of 64 experts of 1536 x 2048, silu and gate: 23.3-24.5 us a call (x 3.5-4.4
// and the products 20-21.5; floor 12.8): latency, as without the epilogue.
#define Q4K_EPILOGUE
#include "q4k_grouped.hip"
