"""The smoke run's own checks, on the CPU: what they are given here is right,
or wrong in a way that they have to notice."""
import math

import torch

import __graft_entry__ as entry
import layers_reference as ref


def test_the_rotation_check_sees_a_wrong_angle():
    x = torch.randn(2, 50, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    freq = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    at = torch.arange(50).expand(2, 50)

    def turned(f=freq, p=at, rope="halves", kind="rms"):
        return ref.qk(x.double(), None, None, kind, 1e-6, f, rope, p).bfloat16()

    assert entry.rotation_error(turned(), x, freq) <= entry.ROTATION_BOUND
    for wrong in (turned(f=None), turned(f=-freq), turned(p=at + 1), turned(rope="interleaved"),
                  turned(f=freq * (1 + 1e-3)), turned(f=freq.float().half().double()),
                  turned(kind="none"), turned(p=torch.zeros_like(at))):
        assert not entry.rotation_error(wrong, x, freq) <= entry.ROTATION_BOUND
    nan = turned()
    nan[0, 0, 0, 0] = math.nan
    assert not entry.rotation_error(nan, x, freq) <= entry.ROTATION_BOUND
