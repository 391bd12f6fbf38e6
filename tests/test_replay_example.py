"""What the example's own code decides (examples/replay_distill.py)."""
import importlib.util
import os

import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "replay_distill.py")


def example():
    spec = importlib.util.spec_from_file_location("replay_distill", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_states_stay_behind_the_newest_row():
    """A state is stored again `ahead` of a sampled slot only where the rows between
    the two follow each other."""
    m = example()
    n, ahead = m.CAPACITY, 16
    for cursor in (0, 5, 300, n - 3):
        age = torch.tensor([0, 1, 15, 16, 17, 400, n - 1])  # rows written after the sampled one
        idx = (cursor - 1 - age) % n
        got = m.slots_ahead(idx, ahead, cursor)
        want = [(int(i) + ahead) % n if a >= ahead else -1 for i, a in zip(idx, age)]
        assert got.tolist() == want
