"""What q4k_gemv_act relies on in the plans of one vector (no GPU): kernel 2's rows a
workgroup, whose sums meet in LDS behind x."""
import pytest

from block_quantized_decode_q4_amd import q4k

LDS = 163840


@pytest.mark.parametrize("aligned", [True, False])
def test_sums_of_the_streaming_kernel_fit(aligned):
    seen = 0
    for k in (256, 512, 1024, 2048, 3840, 4096, 4352, 8192, 28672):
        for n in (1, 2, 63, 64, 1000, 2048, 4096, 8191, 14336, 32000, 128256, 1000003, 2 ** 31 - 1):
            p = q4k.q4k_plan(n, k, 1, w_aligned128=aligned, lds_max=LDS)
            if p.kernel == 2:
                seen += 1
                assert p.rows_per_block <= 512
                assert p.lds_bytes + 8 * p.rows_per_block <= LDS, (n, k)
    assert seen >= 10
