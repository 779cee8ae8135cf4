"""Every order of events of the linear-attention kernels' warps, small models on the CPU: no wait on a barrier's parity
can miss the phase that it is for, and a wait that runs out leaves nobody at a barrier without a limit.

A role is a list of steps: ("wait", barrier, phase), ("arrive", barrier), ("sync", barrier) for a hardware barrier
that all of its members reach.  A parity wait passes where the barrier has completed an odd number of phases more than
`phase` before it, which is what the hardware tells: two phases ahead looks like none.  How many
barriers the images take in turn and the kind of the prefill's meeting are read from the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_kda_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def explore(roles, counts, can_time_out):
    """First state, as positions in the roles, from which nothing moves though a role has not ended; None if there is none."""
    arrivals = [{} for _ in roles]
    for r, prog in enumerate(roles):
        done = {}
        for i, step in enumerate(prog):
            arrivals[r][i] = dict(done)
            if step[0] == "arrive":
                done[step[1]] = done.get(step[1], 0) + 1
        arrivals[r][len(prog)] = dict(done)
    members = {s[1]: [r for r, p in enumerate(roles) if any(x[0] == "sync" and x[1] == s[1] for x in p)] for p in roles for s in p if s[0] == "sync"}
    # what a role has arrived at depends on where it is, and, once it has given up, on where it did so
    start = tuple((0, None) for _ in roles)
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()

        def completed(bar):
            n = 0
            for r, (at, gave_up) in enumerate(state):
                n += arrivals[r][gave_up if gave_up is not None else at].get(bar, 0)
            return n // counts[bar]

        def step_of(r):
            at = state[r][0]
            return roles[r][at] if at < len(roles[r]) else None

        after = []
        for r, (at, gave_up) in enumerate(state):
            step = step_of(r)
            if step is None:
                continue
            nxt = lambda at, g: after.append(state[:r] + ((at, g),) + state[r + 1:])  # noqa: B023, E731
            if step[0] == "arrive":
                nxt(at + 1, gave_up)
            elif step[0] == "wait":
                if (completed(step[1]) - step[2]) % 2 == 1:
                    nxt(at + 1, gave_up)
                elif can_time_out:  # leaves for the steps behind ("end",)
                    nxt(roles[r].index(("end",)), at)
            elif step[0] == "end":
                nxt(at + 1, gave_up)
        for bar, who in members.items():
            if all(step_of(r) == ("sync", bar) for r in who):
                after.append(tuple((at + 1, g) if r in who else (at, g) for r, (at, g) in enumerate(state)))
        if not after and any(at < len(roles[r]) for r, (at, _) in enumerate(state)):
            return state
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


# ------------------------------------------------------------------ chains of the gradients: tiles and images
def chain(nc, i0, bars):
    """Loader, products, images and one worker of linear_bwd_states_tc_kernel on nc chunks, whose images begin with chunk
    i0; `bars`: barriers that the images' phases go round."""
    image = lambda j: (("stg_done", j % bars), j // bars)  # noqa: E731
    load, mma, img, work = [], [], [], []
    for i in range(nc):
        if i >= 2 + i0:
            load.append(("wait", *image(i - 2 - i0)))
        load.append(("arrive", ("in", i % 3)))
        mma += [("wait", "s_ready", i), ("wait", ("in", i % 3), i // 3), ("arrive", "u_done")]
    for i in range(i0, nc):
        img += [("wait", "stg_full", i - i0), ("arrive", image(i - i0)[0])]
    work.append(("wait", ("in", 0), 0))
    for i in range(nc):
        if i:
            work.append(("wait", "u_done", i - 1))
        work.append(("arrive", "s_ready"))
        if i >= i0:
            if i > i0:
                work.append(("wait", *image(i - 1 - i0)))
            work.append(("arrive", "stg_full"))
        if i + 1 < nc:
            work.append(("wait", ("in", (i + 1) % 3), (i + 1) // 3))
    work.append(("wait", "u_done", nc - 1))
    roles = [load, mma, img, work]
    counts = {s[1]: 1 for p in roles for s in p}
    return roles, counts


@pytest.mark.parametrize("i0", [0, 1])
@pytest.mark.parametrize("nc", [1, 2, 3, 5, 9])
def test_chains_never_miss_a_phase(nc, i0):
    bars = re.search(r"constexpr int IMAGE_BARS = (\d+);", source("kda_linear_bwd_tc.cu"))
    assert explore(*chain(nc, i0, int(bars.group(1)) if bars else 1), False) is None


@pytest.mark.parametrize("nc", [1, 4, 9])
def test_sums_of_segments_never_miss_a_phase(nc):
    """Their loader waits for the products of three chunks before."""
    load, mma, work = [], [], [("wait", ("in", 0), 0)]
    for i in range(nc):
        load += ([("wait", "u_done", i - 3)] if i >= 3 else []) + [("arrive", ("in", i % 3))]
        mma += [("wait", "s_ready", i), ("wait", ("in", i % 3), i // 3), ("arrive", "u_done")]
        work += ([("wait", "u_done", i - 1)] if i else []) + [("arrive", "s_ready")]
        if i + 1 < nc:
            work.append(("wait", ("in", (i + 1) % 3), (i + 1) // 3))
    assert explore([load, mma, work], {s[1]: 1 for p in (load, mma, work) for s in p}, False) is None


def test_one_barrier_for_all_images_would_miss_one():
    assert explore(*chain(5, 0, 1), False) is not None


# ------------------------------------------------------------------ prefill: the meeting of a quarter's warps
def meeting(nc, hardware):
    """Two of the warps that read a quarter of X before one of them writes P over it, and the warp that issues products."""
    work = []
    for i in range(nc):
        work += [("wait", "x_done", i), ("arrive", "k_ready")]
        work += [("sync", "quarter")] if hardware else [("arrive", "x_read"), ("wait", "x_read", i)]
        work += [("wait", "d_done", i), ("arrive", "p_ready")]
    mma = [("arrive", "x_done")]
    for i in range(nc):
        mma += [("arrive", "d_done"), ("wait", "k_ready", i), ("wait", "p_ready", i)]
        if i + 1 < nc:
            mma.append(("arrive", "x_done"))
    end = [("end",), ("sync", "block")]
    return [work + end, work + end, mma + end], {"x_done": 1, "d_done": 1, "k_ready": 2, "p_ready": 2, "x_read": 2}


@pytest.mark.parametrize("can_time_out", [False, True])
@pytest.mark.parametrize("nc", [1, 3])
def test_prefill_ends_whatever_gives_up(nc, can_time_out):
    hardware = "bar_sync(" in source("kda_linear_tc.cu")
    assert explore(*meeting(nc, hardware), can_time_out) is None


def test_a_hardware_barrier_behind_a_wait_would_not_end():
    assert explore(*meeting(1, True), False) is None
    assert explore(*meeting(1, True), True) is not None


# ------------------------------------------------------------------ prefill: all of a chain's barriers
def prefill(nc, ragged):
    """Loader, products, decays, stores and one worker of linear_fwd_tc_kernel on nc chunks, the last one short or whole."""
    slot = lambda t: t % 4  # noqa: E731
    load, mma, dec, store, work = [], [], [], [], []
    for t in range(3 * nc):
        if t >= 4:
            load.append(("wait", ("free", slot(t)), t // 4 - 1))
        load.append(("arrive", ("full", slot(t))))
    full = lambda t: ("wait", ("full", slot(t)), t // 4)  # noqa: E731
    for i in range(nc):
        mma += ([("wait", "u_read", i - 1)] if i else []) + [full(3 * i), full(3 * i + 1), ("arrive", "x_done"), ("wait", "s_ready", i)]
        mma += ([("wait", "o_read", i - 1)] if i else []) + [("arrive", "d_done"), ("arrive", ("free", slot(3 * i)))]
        mma += [("wait", "k_ready", i), full(3 * i + 2), ("arrive", "u_done"), ("arrive", ("free", slot(3 * i + 1)))]
        mma += [("wait", "p_ready", i), ("arrive", "o_done"), ("arrive", ("free", slot(3 * i + 2)))]
        dec += ([("wait", ("dec_free", i % 2), i // 2 - 1)] if i >= 2 else []) + [("arrive", ("dec_ready", i % 2))]
        if not (ragged and i == nc - 1):
            store += [("wait", "o_staged", i), ("arrive", "o_stored")]
    for i in range(nc + 1):
        work += ([("wait", "u_done", i - 1)] if i else []) + ([("wait", ("dec_ready", i % 2), i // 2)] if i < nc else [])
        if i < nc:
            work += ([("arrive", "u_read")] if i else []) + [("arrive", "s_ready")]
        if i:
            work += ([("wait", "o_stored", i - 2)] if i > 1 else []) + [("wait", "o_done", i - 1), ("arrive", "o_read")]
            work += [] if ragged and i == nc else [("arrive", "o_staged")]
        if i < nc:
            work += [("wait", "x_done", i)] + ([full(3 * i + 2)] if ragged and i == nc - 1 else []) + [("arrive", "k_ready")]
            work += [("arrive", "x_read"), ("wait", "x_read", i), ("wait", "d_done", i), ("arrive", "p_ready"), ("arrive", ("dec_free", i % 2))]
    roles = [load, mma, dec, store, work]
    return roles, {s[1]: 1 for p in roles for s in p}


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("nc", [1, 2, 5])
def test_prefill_never_misses_a_phase(nc, ragged):
    assert explore(*prefill(nc, ragged), False) is None
