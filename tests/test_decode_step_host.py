"""Refusals of the example decode step that come before any launch."""
import sys

import pytest


def test_a_step_past_the_room_for_own_tokens():
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    net = DecodeStep.__new__(DecodeStep)   # nothing on a device
    net.max_own, net.taken = 7, 7
    with pytest.raises(ValueError, match="room for 7"):
        net.step(None)
    assert net.taken == 7


@pytest.mark.parametrize("argv", [["--steps", "513"], ["--steps", "3"], ["--steps", "0"], ["--max-own", "10", "--steps", "11"]])
def test_steps_that_the_command_does_not_take(argv, monkeypatch, capsys):
    from gemm_qmv_quantize_gb300 import decode_step
    monkeypatch.setattr(sys, "argv", ["decode_step", *argv])
    monkeypatch.setattr(decode_step, "DecodeStep", lambda *a: pytest.fail("built"))
    with pytest.raises(SystemExit) as e:
        decode_step.main()
    assert e.value.code == 2 and "--steps" in capsys.readouterr().err
