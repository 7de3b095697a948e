"""The benchmark's timed loops must not be held up by the garbage collector."""
import gc

import torch  # noqa: F401  (the imports whose objects a pass would walk)

import bench


def test_a_pass_has_little_to_walk_once_settled():
    try:
        bench.settle_collector()
        assert gc.get_freeze_count() > 50000 and len(gc.get_objects()) < 1000 and gc.isenabled()
    finally:
        gc.unfreeze()
