"""Cases of the gate gradient: lens, H, Hk, dk, dv, decay, gate, with states at both ends or not."""
import linear_ref as ref

GATES = [
    ([64], 4, 2, 128, 128, "head", "std", False),
    ([2, 0, 65], 4, 2, 128, 128, "head", "std", True),
    ([300, 0, 1, 129], 4, 1, 64, 128, "head", "slow", False),
    ([300, 0, 1, 129], 4, 2, 64, 64, "token", "slow", True),
    ([63, 64, 65, 1, 128], 2, 2, 128, 64, "token", "std", True),
    ([200, 65, 3], 4, 2, 128, 128, "token", "reset", True),
    ([200, 65, 3], 4, 2, 64, 64, "token", "steep", True),
    # in segments
    ([1600], 2, 1, 64, 128, "head", "slow", True),
    ([1600], 2, 1, 128, 128, "token", "slow", True),
    ([0, 30, 1025], 2, 1, 128, 64, "token", "unit", False),
]


def gate_case(dtype, lens, H, Hk, dk, dv, decay, gate, state):
    return ref.make(lens, H, Hk, dk, dv, dtype, decay, gate, state, seed=71)
