"""Without a GPU: the descriptor of rotary positions as a Python object."""
import copy
import pickle

import torch

import hybrid_sliding_window_swa_b200 as hs


def test_a_rope_descriptor_keeps_its_own_copy():
    # lists changed by their owner afterwards change nothing, neither before nor after the descriptor's first use
    inv, axis = [1.0 / (i + 1) for i in range(8)], [i % 2 for i in range(8)]
    rope, late = hs.RopeDesc(inv, axis, 2), hs.RopeDesc(inv, axis, 2)
    before = rope.c().contents
    inv[0], axis[1] = 7.0, 0
    for r in (rope, late):
        c = r.c().contents
        assert [c.inv_freq[i] for i in range(8)] == list(r.inv_freq) == [1.0 / (i + 1) for i in range(8)]
        assert [c.axis[i] for i in range(8)] == list(r.axis) == [i % 2 for i in range(8)]
    assert rope == late and hash(rope) == hash(late) and before.inv_freq[0] == 1.0
    assert hs.RopeDesc(torch.tensor(inv, dtype=torch.float64)).inv_freq == tuple(inv)
    assert hs.RopeDesc(x for x in inv).c().contents.rot_dim == 16 and hs.RopeDesc(inv).axis is None


def test_a_used_descriptor_can_be_copied_and_pickled():
    rope = hs.RopeDesc([1.0 / (i + 1) for i in range(8)], [0] * 8, 1, True)
    rope.c()
    for other in (copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        assert other == rope and other.c().contents.inv_freq[7] == 0.125 and other.c().contents.interleaved == 1
