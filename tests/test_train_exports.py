"""Every entry point of include/q8train.h has a function of its name in the package."""
import bit_blockwise_adamw_gb300 as q8


def test_every_training_entry_point_is_in_the_package():
    names = [n for n in q8.EXPORTS if n.startswith(("q8_gated_ff", "q8_block_norm", "q8_distill"))]
    assert len(names) == 8 and all(callable(getattr(q8, n, None)) for n in names)
