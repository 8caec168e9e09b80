"""Further refusals of the operators around the recurrence, and calls that
they have to take (fake addresses: nothing reaches a device)."""
from __future__ import annotations

import pytest

import linear_attention_recurrence_step_gb300 as gdn
from test_layer_ops_host import CUDA, INVALID, OK, P, conv, lib, scan  # noqa: F401 (lib: fixture)

torch = pytest.importorskip("torch")

# outputs that lie on a small input (at its first byte, and just at its last)
ON_SMALL = {
    conv: [dict(y=P(2)), dict(state_out=P(2)), dict(y=P(4)), dict(state_out=P(4)),
           dict(y=P(2) + 126), dict(state_out=P(4) + 6)],
    scan: [dict(y=P(2)), dict(state_out=P(2)), dict(y=P(5)), dict(state_out=P(5)), dict(y=P(6)), dict(state_out=P(6)),
           dict(y=P(8)), dict(state_out=P(8)), dict(y=P(2) + 14), dict(y=P(8) + 6),
           *(dict(T=4096, B=1, ws=P(i), ws_bytes=1 << 30, y=P(40), state_out=P(80), x=P(100), Bm=P(120), Cm=P(140),
                  dt=P(160)) for i in (2, 5, 6, 8))],
}


@pytest.mark.parametrize("call,kw", [(c, kw) for c in ON_SMALL for kw in ON_SMALL[c]],
                         ids=lambda v: v.__name__ if callable(v) else "-".join(v))
def test_an_output_on_a_small_input(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == INVALID
    assert b"overlap" in lib.gdn_last_error()


def test_outputs_beside_small_inputs(lib):  # noqa: F811
    """One element past the end is another tensor's."""
    calls = [(conv, dict(y=P(2) + 128)), (conv, dict(y=P(4) + 8)), (scan, dict(y=P(2) + 16)),
             (scan, dict(state_out=P(8) + 16))]
    try:
        assert lib.gdn_force_launch_failures(len(calls)) == OK
        for call, kw in calls:
            assert call(lib, **kw) == CUDA  # accepted: it got as far as the launch
    finally:
        assert lib.gdn_force_launch_failures(0) == OK


# strides of tensors that hold the steps of all sequences together, [T,B,...]
TIME_MAJOR = [(conv, dict(sb=64, st=128)), (conv, dict(sb=100, st=264)),
              (scan, dict(strides=(256, 512, 4, 8, 256, 512, 256, 512))),
              (scan, dict(strides=(256, 512, 12, 4, 768, 256, 256, 512))),
              (conv, dict(B=1, sb=0)), (conv, dict(T=1, st=0, sb=64))]


def test_steps_may_be_the_outer_dimension(lib):  # noqa: F811
    try:
        assert lib.gdn_force_launch_failures(len(TIME_MAJOR)) == OK
        for call, kw in TIME_MAJOR:
            assert call(lib, **kw) == CUDA, kw
    finally:
        assert lib.gdn_force_launch_failures(0) == OK


@pytest.mark.parametrize("kw", [dict(sb=63, st=128), dict(sb=64, st=127), dict(sb=128, st=64), dict(sb=0, st=128),
                                dict(sb=64, st=0), dict(sb=1 << 62, st=64, B=4), dict(sb=64, st=1 << 62)],
                         ids=lambda kw: f"{kw['sb']}-{kw['st']}")
def test_rows_that_overlap_are_refused(lib, kw):  # noqa: F811
    assert conv(lib, **kw) == INVALID
    assert b"strides" in lib.gdn_last_error()
