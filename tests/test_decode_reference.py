"""The plain references of the operators around the verify step, pinned to
answers worked out by hand."""
import numpy as np

import decode_reference as ref


def test_beam_select_by_hand():
    # two beams over three tokens with probabilities (1/2, 1/4, 1/4) and (1/10, 8/10, 1/10)
    x = np.log(np.array([[[2.0, 1.0, 1.0], [1.0, 8.0, 1.0]]]))
    s, p, t, _ = ref.beam_select(x, np.log(np.array([[0.5, 0.5]])), 4)
    assert np.allclose(np.exp(s), [[0.4, 0.25, 0.125, 0.125]])
    assert p.tolist() == [[1, 0, 0, 0]] and t.tolist() == [[1, 0, 1, 2]]  # equal values: lowest index first
    # a finished beam goes on as itself, a beam without a hypothesis has no candidates
    s, p, t, _ = ref.beam_select(x, np.array([[-np.inf, np.log(0.3)]]), 2, np.array([[0, 1]]), eos=2)
    assert np.isclose(np.exp(s[0, 0]), 0.3) and s[0, 1] == -np.inf
    assert p.tolist() == [[1, -1]] and t.tolist() == [[2, -1]]


def test_plan_slots_by_hand():
    # pages of 4; request 0 holds page 7 with 3 positions, request 1 has ended and held page 5, request 2 is new
    tables = np.array([[7, -1, -1], [5, -1, -1], [-1, -1, -1]], np.int32)
    ring = np.array([1, 2, 9, 0, 0, 0], np.int32)
    got = ref.plan_slots(np.array([2, 3, 0]), tables, np.array([1, 1, 0]), ring, np.array([0, 3]), 4, k=2,
                         accept=np.array([0, 1, -1]), release=np.array([0, 1, 0]))
    lens, held, state, pos, slots, tables, ring = got
    assert lens.tolist() == [3, 0, 0] and held.tolist() == [2, 0, 1]
    assert tables[0].tolist() == [7, 1, -1] and tables[2, 0] == 2
    assert ring.tolist() == [1, 2, 9, 5, 0, 0] and state.tolist() == [2, 2]
    assert pos.tolist() == [3, 4, 5, -1, -1, -1, 0, 1, 2]
    assert slots.tolist() == [31, 4, 5, -1, -1, -1, 8, 9, 10]


def test_states_by_hand():
    src = np.arange(12).reshape(1, 1, 3, 4, 1)
    dst = np.full_like(src, -1)
    got = ref.reorder_states(src, dst, np.array([[2, 2, 5]]), np.array([2]))
    assert got[0, 0, :, :, 0].tolist() == [[8, 9, -1, -1], [8, 9, -1, -1], [-1, -1, -1, -1]]
    tree = np.arange(5).reshape(1, 1, 5, 1)
    got = ref.commit_path(tree, np.array([2]), np.array([[2, 4, -1]]), np.full((1, 6, 1), -1), np.array([[5, 3, 0, 1]]))
    assert got[0, :, 0].tolist() == [4, -1, -1, 2, -1, 0]
