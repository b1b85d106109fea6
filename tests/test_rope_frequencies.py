"""Every scaling's frequencies, pair by pair, against the published formulas worked out here in Python's own numbers."""
import math

import pytest
import torch

from draft_tree_build_gb300 import bastion


def bands(rot, base, factor, length, low, high):
    got = []
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        wave = 2 * math.pi / f
        if wave < length / high:
            got.append(f)
        elif wave > length / low:
            got.append(f / factor)
        else:
            s = (length / wave - low) / (high - low)
            got.append((1 - s) * f / factor + s * f)
    return got


def yarn(rot, base, factor, length, slow, fast):
    def pair(turns):
        return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
    first, last = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    if first == last:
        last += 0.001
    got = []
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        extra = 1 - min(1.0, max(0.0, (i - first) / (last - first)))
        got.append(f / factor * (1 - extra) + f * extra)
    return got


def check(got, want):
    assert got.dtype == torch.float64 and len(got) == len(want)
    for x, y in zip(got.tolist(), want):
        assert x == pytest.approx(y, rel=1e-12)


@pytest.mark.parametrize("rot,base,factor,length", [(128, 10000.0, 4.0, 4096), (64, 5e5, 8.0, 8192), (32, 1e6, 32.0, 32768),
                                                    (128, 10000.0, 16.0, 2048), (16, 10000.0, 2.0, 4096)])
def test_each_scaling_as_it_is_by_default(rot, base, factor, length):
    plain = [1.0 / base ** (2 * i / rot) for i in range(rot // 2)]
    for kw, want, size in (
            (dict(), plain, 1.0),
            (dict(scaling="linear"), [f / factor for f in plain], 1.0),
            (dict(scaling="base"), [1.0 / (base * factor ** (rot / (rot - 2))) ** (2 * i / rot) for i in range(rot // 2)], 1.0),
            (dict(scaling="bands"), bands(rot, base, factor, length, 1.0, 4.0), 1.0),
            (dict(scaling="yarn"), yarn(rot, base, factor, length, 1.0, 32.0), 0.1 * math.log(factor) + 1.0)):
        got, f = bastion.rope_frequencies(rot, base, "cpu", factor=factor, length=length, **kw)
        check(got, want)
        assert f == pytest.approx(size, rel=1e-15)


def test_turns_that_are_given():
    check(bastion.rope_frequencies(128, 5e5, "cpu", "bands", 8.0, 2.0, 9.0, 4096)[0], bands(128, 5e5, 8.0, 4096, 2.0, 9.0))
    check(bastion.rope_frequencies(128, 1e4, "cpu", "yarn", 8.0, 2.0, 9.0, 4096)[0], yarn(128, 1e4, 8.0, 4096, 2.0, 9.0))
    check(bastion.rope_frequencies(128, 1e4, "cpu", "yarn", 8.0, low=2.0, length=4096)[0], yarn(128, 1e4, 8.0, 4096, 2.0, 32.0))


@pytest.mark.parametrize("args", [dict(rot_dim=7), dict(rot_dim=-2), dict(rot_dim=64, base=0.0), dict(rot_dim=64, factor=0.0),
                                  dict(rot_dim=2, scaling="base", factor=2.0), dict(rot_dim=64, scaling="bands", low=4.0),
                                  dict(rot_dim=64, scaling="yarn", low=3.0, high=2.0), dict(rot_dim=64, scaling="yarn", base=1.0),
                                  dict(rot_dim=64, scaling="bands", length=0), dict(rot_dim=64, scaling="bands", low=float("nan"))])
def test_what_has_no_frequencies_is_refused(args):
    with pytest.raises(bastion.BastionError, match="rope frequencies"):
        bastion.rope_frequencies(device="cpu", **args)


def test_nothing_to_turn():
    f, size = bastion.rope_frequencies(0, device="cpu")
    assert f.numel() == 0 and size == 1.0
