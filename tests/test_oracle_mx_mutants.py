"""The pins of the MXFP4 oracle (tests/test_oracle_mx.py) must notice plausible
mistakes: each one below is planted in a copy of oracle/mx.py, and at least
one pin has to fail. The copy as it is passes them all."""

import os
import types

import numpy as np
import pytest

import oracle.mx
import test_oracle_mx as T

SOURCE = open(os.path.join(os.path.dirname(oracle.mx.__file__), "mx.py")).read()

MUTANTS = {
    "high half first": ("nib[:, 0::2] = codes & 15", "nib[:, 0::2] = codes >> 4"),
    "magnitude 5 for 6": ("3.0, 4.0, 6.0])", "3.0, 4.0, 5.0])"),
    "no subnormal half": ("[0.0, 0.5, 1.0", "[0.0, 0.25, 1.0"),
    "sign from bit 2": ("np.where(nib & 8, -1.0, 1.0)", "np.where(nib & 4, -1.0, 1.0)"),
    "bias 128": ("scales.astype(np.int64) - 127", "scales.astype(np.int64) - 128"),
    "scale 255 is a number": ("np.where(scales == 255, np.nan, unit)", "unit"),
    "scale one up": ("np.maximum(e - 1 - 2 + 127, 0)", "np.maximum(e - 1 - 1 + 127, 0)"),
    "scale one down": ("np.maximum(e - 1 - 2 + 127, 0)", "np.maximum(e - 1 - 3 + 127, 0)"),
    "ties up": ("(d == dist) & (c % 2 == 0)", "(d == dist)"),
    "ties down": ("(d < dist) | ((d == dist) & (c % 2 == 0))", "d < dist"),
    "sign lost": ("best + 8 * np.signbit(x)", "best"),
    "sign of zero lost": ("8 * np.signbit(x)", "8 * (x < 0)"),
    "Inf kept as a number": ("bad = ~np.isfinite(top)", "bad = np.isnan(top)"),
    "tiles without the phase": ("return (shard + 574) // 512", "return (shard + 511) // 512"),
    "a tile too many": ("return (shard + 574) // 512", "return (shard + 574) // 512 + 1"),
    "phase modulo 32": ("r.start % 64, slice(w", "r.start % 32, slice(w"),
    "ranks not apart": ("w = D * at + rank * nb", "w = D * at"),
    "buckets not apart in WORLD": ("w = D * at + rank * nb", "w = at + rank * nb"),
    "padding counted as owned": ("min(r.end, b.offset + b.numel)", "r.end"),
    "WORLD quantises one rank": ("range(layout.dp_size) if coords == WORLD else [rank]", "[rank]"),
    "residual not added": ("x = x + residual[at]", "x = x + 0 * residual[at]"),
    "residual keeps all": ("residual[at], x - y.astype(np.float32))", "residual[at], x)"),
    "residual of the other sign": ("x - y.astype(np.float32))", "y.astype(np.float32) - x)"),
    "first contribution left out": ("for s in storages[1:]:", "for s in storages[2:]:"),
    "no scale": ("* dtype(np.float32(scale))", "* dtype(1)"),
    "decay of the new value": ("(u + wd * p)", "(u + wd * u)"),
    "first moment's correction twice": ("(mn / bc1)", "(mn / bc1 / bc1)"),
    "second moment of g": ("omb2 * (g * g)", "omb2 * g"),
    "eps inside the root": ("(np.sqrt(vn / bc2) + eps)", "np.sqrt(vn / bc2 + eps)"),
    "stale parameters": ("N.narrow(master[k].astype(np.float32))", "N.narrow((master[k] * 0).astype(np.float32))"),
    "gather from the first rank": ("for rng in ranges(layout, j):", "for rng in ranges(layout, 0):"),
}

PINS = [T.test_decode_table, *(lambda t=t: T.test_encode_rounds_to_nearest_even_and_saturates(t) for t in (7.9, 5.0)),
        T.test_encode_scale_and_specials,
        *(lambda s=s: T.test_storage_holds_every_element_once(s) for s in range(8)),
        *(lambda s=s: T.test_local_storage_is_the_ranks_part_of_world_storage(s) for s in range(6)),
        *(lambda s=s: T.test_step_equals_the_bf16_step_on_values_that_both_hold(s) for s in range(4)),
        T.test_residual_carries_what_the_codes_did_not]


def failing(source, monkeypatch):
    """Whether some pin fails on this source."""
    mod = types.ModuleType("oracle.mx")
    mod.__package__ = "oracle"
    exec(compile(source, "mx.py", "exec"), mod.__dict__)
    monkeypatch.setattr(T, "MX", mod)
    with np.errstate(all="ignore"):
        for pin in PINS:
            try:
                pin()
            except Exception:
                return True
    return False


def test_the_oracle_as_it_is_passes(monkeypatch):
    assert not failing(SOURCE, monkeypatch)


@pytest.mark.parametrize("name", MUTANTS)
def test_a_mistake_is_noticed(name, monkeypatch):
    old, new = MUTANTS[name]
    assert SOURCE.count(old) >= 1, name
    assert failing(SOURCE.replace(old, new), monkeypatch), name
