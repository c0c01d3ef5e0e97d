"""A workspace kept for the largest call serves every smaller one: the bytes
that the *_ws functions give never fall as rows, slots, groups, ranks or k
grow."""
import pytest

from block_quantized_decode_q4_amd import q4k


def _rises(sizes, bytes_of):
    most = 0
    for s in sizes:
        have = bytes_of(s)
        assert have >= most, (s, have, most)
        most = have
    assert most > 0


# every length near the steps of the rules, then coarsely
LENGTHS = sorted(set(list(range(1, 1200)) + list(range(4000, 4200)) + list(range(8100, 8300)) +
                     list(range(16300, 16500)) + [2 ** i + j for i in range(10, 22) for j in (-1, 0, 1)]))


@pytest.mark.parametrize("r", [1, 16, 17, 64, 1024])
def test_lora_rows(r):
    _rises(LENGTHS, lambda rows: q4k.q4k_lora_ws(rows, r))


@pytest.mark.parametrize("rows", [1, 512, 513, 4095, 4096, 100000])
def test_lora_ranks(rows):
    _rises(range(1, 1025), lambda r: q4k.q4k_lora_ws(rows, r))


@pytest.mark.parametrize("groups,topk", [(8, 1), (8, 2), (64, 8), (128, 7), (256, 8), (257, 8), (1024, 32)])
def test_group_slots(groups, topk):
    _rises([m * topk for m in LENGTHS if m * topk < 2 ** 22],
           lambda slots: q4k.q4k_moe_group_ws(slots, groups, topk))


@pytest.mark.parametrize("slots", [193, 1000, 16385, 2 ** 20 + 1])
def test_group_groups(slots):
    _rises(range(1, 1025), lambda groups: q4k.q4k_moe_group_ws(slots, groups, 1))


def test_grouped_rows_and_k():
    _rises(LENGTHS, lambda rows: q4k.q4k_gemv_grouped_ws(4096, rows))
    _rises(range(256, 2 ** 16, 256), lambda k: q4k.q4k_gemv_grouped_ws(k, 96))
