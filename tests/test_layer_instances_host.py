"""The few-token layer's kernel instances in the built library: none that no
call can launch (read from the kernel names it registers; no GPU needed)."""
import re

import grouped_gemm_mxfp8_amd as gm

BF16, FP8, FP4 = 0, 1, 2            # weight formats as the kernels name them


def instances(kernel):
    """Template arguments (integers and truth values in order) of every instance."""
    names = re.findall(kernel.encode() + rb"_kernelI((?:L[ib]\d+E)+)E", open(gm.LIB_PATH, "rb").read())
    return {tuple(int(v) for v in re.findall(rb"L[ib](\d+)E", n)) for n in names}


def test_groups_of_one_step_have_no_partial_form(mxlib):
    """A K step count is always a multiple of one: with one step a group, only
    the kernels for whole groups can run."""
    gate_up, down = instances("layer_gate_up"), instances("layer_down")
    assert {i[0] for i in gate_up} == {i[0] for i in down} == {BF16, FP8, FP4}
    for wf, nt, steps, whole, *rt in gate_up | down:
        assert whole or steps > 1, (wf, nt, steps, whole, rt)


def test_four_tiles_of_w2_only_where_they_are_chosen(mxlib):
    """Four tiles of W2 a workgroup: MX weights and 17 to 32 tokens, whose
    experts' rows come in at most two tiles."""
    for wf, nt, _, _, rt in instances("layer_down"):
        assert rt < 4 or (wf != BF16 and nt < 4), (wf, nt, rt)


def test_every_row_tile_count_is_there(mxlib):
    for wf in (BF16, FP8, FP4):
        assert {i[1] for i in instances("layer_gate_up") if i[0] == wf} == {1, 2, 4}
        assert {(i[1], i[4]) for i in instances("layer_down") if i[0] == wf} >= {
            (nt, rt) for nt in (1, 2, 4) for rt in (1, 2)}
