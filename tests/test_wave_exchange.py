"""Sums that pass from lane to lane through LDS inside a wave: the source orders the stores before the other lanes'
reads, and these before the next stores, and every lane reaches both places."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "state_space_recurrence_amd", "csrc")


def _body(name):
    """The function's body, without comments."""
    with open(os.path.join(CSRC, "linear_kernels.hip")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", text.index(f"void {name}("))
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if not depth:
            return text[at:end]


def test_sums_are_ordered_on_their_way_to_other_lanes():
    body = _body("finish")
    stored = body.index("reinterpret_cast<f4v *>(lds")
    read = [m.start() for m in re.finditer(r"reinterpret_cast<const f4v \*>\(lds", body)]
    synced = [m.start() for m in re.finditer(r"\bwave_exchange\(\);", body)]
    assert read and len(synced) == 2
    assert stored < synced[0] < min(read) and max(read) < synced[1]
    assert not re.search(r"\b(return|break|continue|goto)\b", body)


def test_an_exchange_is_a_fence_and_a_barrier_of_the_wave():
    body = _body("wave_exchange")
    parts = [body.index(s) for s in ("__builtin_amdgcn_fence(__ATOMIC_RELEASE, \"wavefront\"", "__builtin_amdgcn_wave_barrier()",
                                     "__builtin_amdgcn_fence(__ATOMIC_ACQUIRE, \"wavefront\"")]
    assert parts == sorted(parts)
