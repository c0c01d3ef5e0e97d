"""README.md's C examples: as many arguments as the header declares, and, around
a layer's projections, every call takes what a call before it left in the form
that it needs."""
from readme_calls import blocks

GROUPED = ("q4k_gemv_grouped", "q4k_gemv_grouped_q8", "q4k_f16_gemm_grouped")


def test_two_examples_with_the_headers_arguments():
    assert len(blocks()) == 2 and all(blocks())


def test_layer_example_passes_on_what_the_calls_need():
    calls = blocks()[1]
    names = [c[0] for c in calls]
    assert {"q4k_rmsnorm", "q4k_moe_route", "q4k_moe_group", "q4k_moe_combine", "q4k_lora",
            "q4k_gemv_grouped", "q4k_f16_gemm_grouped"} <= set(names)
    rows = {}                  # y of grouped products: by "position" or "slot"
    grouping = {}              # offsets: (who grouped them, their order)
    for name, a in calls:
        if name == "q4k_moe_route":
            grouping[a["offsets"]] = ("slots", a["order"])
        elif name == "q4k_moe_group":
            grouping[a["offsets"]] = ("rows", a["order"])
        elif name in GROUPED:
            of, order = grouping[a["offsets"]]
            assert of == "slots"
            if a["x_rows"] == "NULL":                  # x as an earlier product left it
                assert a["x_div"] == "1"
            else:                                      # x by token
                assert (a["x_rows"], a["x_div"]) == (order, "topk")
            assert a["y_rows"] in ("NULL", order)
            rows[a["y"]] = "position" if a["y_rows"] == "NULL" else "slot"
        elif name == "q4k_moe_combine":
            assert rows[a["y"]] == "slot"              # y[t * topk + j]
        elif name == "q4k_lora":
            assert grouping[a["offsets"]] == ("rows", a["order"])
