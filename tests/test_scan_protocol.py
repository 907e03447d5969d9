"""The hand-over of lane maxima between the halves of a delta-rule scan CTA, through a randomised model on the CPU.

No test makes a wait run out on a GPU, so what a CTA does after it has given up on one is played here.
"""
import os

import pytest

import scan_protocol_model as model

SOURCE = os.path.join(os.path.dirname(__file__), "..", "bounded_memory_attention_b200", "csrc", "rma_gdn_prefill.cu")


@pytest.mark.parametrize("hand_over", ["state", "named"])
def test_without_timeouts_every_half_takes_its_own_chunks_maxima(hand_over):
    for seed in range(200):
        assert model.run(1 + seed % 9, seed, hand_over=hand_over) is False


def test_an_abandoned_cta_comes_to_its_end():
    """Bounded waits alone stand between the chunks, so a half that has given up cannot leave the other waiting."""
    gave_up = sum(model.run(1 + seed % 9, seed, timeout_rate=0.02) for seed in range(600))
    assert gave_up > 300


def test_a_named_barrier_in_its_place_is_caught():
    """After a timeout a warp may arrive twice before the other half's has come: the barrier completes without it."""
    caught = 0
    for seed in range(600):
        try:
            model.run(1 + seed % 9, seed, timeout_rate=0.02, hand_over="named")
        except model.Deadlock:
            caught += 1
    assert caught > 0


def test_the_kernel_hands_over_with_the_state():
    """The scan arrives on no named barrier without waiting there, and a half waits for the other's state, bounded."""
    src = open(SOURCE).read()
    assert "named_bar_arrive" not in src
    assert "scan_wait<false>(&bars[kbS + (wg ^ 1)], c & 1, abort_flag)" in src


def test_an_abandoned_cta_stores_no_outputs():
    """Every store of the output warps, and of the state, stands behind a look at the abort flag after the waits before it."""
    src = open(SOURCE).read()
    out = src[src.index("ptx::named_bar_sync(kBarOut, 128)"):src.index("ptx::mbar_arrive(&bars[kbEmpty + st])")]
    assert out.index("if (*abort_flag) {") < out.index("} else if (left >= kC) {") < out.index("tma_store_2d")
    last = src[src.rindex("if (*abort_flag == 0) {"):]
    assert "scan_wait" not in last[:last.index("gs[2 * i * kGdnDim] =")] and last.index("gs[2 * i * kGdnDim] =") < last.index("__syncthreads")
    assert src.count("gs[2 * i * kGdnDim] =") == 1 and src.count("tma_store_2d(&maps.out") == 1
