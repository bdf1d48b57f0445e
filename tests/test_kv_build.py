"""How the key-value cache's units are built."""
from block_quantized_amd import build


def test_no_unit_may_assume_that_there_are_no_nans():
    # unseen cache rows hold anything, NaN included, and are masked by arithmetic
    for unit, flags in build.UNITS.items():
        if unit.startswith(("attn_", "kv_")):
            assert not any(f in ("-fno-honor-nans", "-ffinite-math-only", "-ffast-math", "-Ofast") for f in flags), unit
