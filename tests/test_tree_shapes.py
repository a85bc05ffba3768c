"""The host's description of a tree: what is no tree is refused."""
import numpy as np
import pytest

from fp8_paged_kv_append_gb300.tree_step import tree_depths, tree_masks


@pytest.mark.parametrize("f", [tree_masks, tree_depths])
@pytest.mark.parametrize("parents", [[-1, 1], [-1, -1], [0, 2, 0], [-1, 0, 0, -2], [-1, 0, 5],
                                     [i - 1 for i in range(65)]])
def test_refused(f, parents):
    with pytest.raises(ValueError):
        f(parents)
    with pytest.raises(ValueError):
        f(np.array(parents, np.int32))


def test_any_value_for_the_first_parent():
    for first in (-1, 0, 7):
        assert tree_depths([first, 0, 1]).tolist() == [0, 1, 2]
        assert tree_masks([first, 0, 1]).tolist() == [1, 3, 7]
