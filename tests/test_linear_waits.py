"""The hand-overs between the warps of the chunked linear-attention kernel, as a model on the host.

A wait by parity is passed when the barrier's last finished phase is the awaited one.  A warp that is held
up until the barrier has finished another phase would wait for a phase that may never come.  The model runs
every role of a CTA through a few units, holds one role at one of its steps for as long as any other can
go on, and checks that the barrier is then never more than one phase ahead: for every role and every step.
"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "paged_moe_shared_gb300", "csrc", "linear_chunk.cu")
UNITS = [(3, True), (1, False), (1, True), (4, False)]  # chunks, and whether the last one is partly filled
WIDE = {1, 2, 4, 7}  # chunks whose queries are scaled
GATES = 4


def roles(kin, out, mistake=False):
    """{role: list of steps}, and the arrivals that finish a phase.  A step is (wait, barrier, phase),
    (arrive, barrier) or (commit, barriers): arrivals once what the role has issued so far is done."""
    stages, keybufs = (2, 2) if kin == 1 else (1, 1)
    chunks = [(u, c, c + 1 == n, part and c + 1 == n) for u, (n, part) in enumerate(UNITS) for c in range(n)]
    key_warps, names = (["p", "keys"], 2) if out else (["keys"], 1)
    count = {"full": 1 if kin == 1 else len(key_warps), "empty": 2 if out else 1, "keys_full": 1,
             "keys_empty": (1 if out else 0) + len(key_warps), "raw": 1, "raw_empty": len(key_warps), "seen": 1, "safe": 1,
             "values_full": 1, "parts_empty": 2, "gate_full": 1, "gate_empty": (3 if out else 1) + len(key_warps),
             "score_full": 1, "score_empty": 1, "key_full": len(key_warps), "key_empty": 1, "p_full": 1,
             "p_empty": 1, "state_full": 1, "state_empty": 1, "update_full": 1, "update_empty": 1,
             "out_full": 1, "out_empty": 1}
    r = {k: [] for k in ["load", "decay", "update", "states", *key_warps] + (["outputs", "inter"] if out else [])}

    def wait(role, bar, it, ring=1, behind=False):
        """Phase it // ring of a ring's barrier; `behind`: the phase before, which frees a place."""
        phase = it // ring - behind
        if phase >= 0:
            r[role].append(("wait", (bar, it % ring), phase))

    def arrive(role, bar, it, ring=1):
        r[role].append(("arrive", (bar, it % ring)))

    def commit(role, *bars):
        r[role].append(("commit", [(b, it % ring) for b, it, ring in bars]))

    def scores(it):
        wait("update", "full", it, stages)
        if kin == 1:
            wait("update", "keys_full", it, stages)
        wait("update", "score_empty", it, 2, True)
        commit("update", ("score_full", it, 2), ("keys_empty", it, stages) if kin == 1 else ("parts_empty", it, 1))

    for it, (u, c, last, part) in enumerate(chunks):
        # loads
        if kin == 2:
            wait("load", "raw_empty", it, 1, True)
            commit("load", ("raw", it, 1))
        else:
            wait("load", "keys_empty", it, stages, True)
            commit("load", ("keys_full", it, stages))
            wait("load", "empty", it, stages, True)
            commit("load", ("full", it, stages))
        # decays
        wait("decay", "gate_empty", it, GATES, True)
        arrive("decay", "gate_full", it, GATES)
        # decayed keys, and what P is made of
        for w in key_warps:
            wait(w, "gate_full", it, GATES)
            if kin == 1:
                wait(w, "keys_full", it, stages)
            else:
                wait(w, "raw", it)
                if out:
                    wait(w, "parts_empty", it, 1, True)
            wait(w, "key_empty", it, keybufs, True)
            if w == "keys" and kin == 2 and not out:
                wait(w, "empty", it, 1, True)
            if w == "keys" and kin == 1 and part:
                wait(w, "full", it, stages)
            arrive(w, "key_full", it, keybufs)
            arrive(w, "full" if kin == 2 else "keys_empty", it, stages)
            if kin == 2 and (w == "p" or not out):
                arrive(w, "raw_empty", it)
            if w == "keys":
                arrive(w, "gate_empty", it, GATES)
                if kin == 2 and out:
                    wait(w, "empty", it, 1, True)
                    arrive(w, "values_full", it)
                    arrive(w, "raw_empty", it)
            else:
                wait(w, "score_full", it, 2)
                wait(w, "p_empty", it, 1, True)
                arrive(w, "score_empty", it, 2)
                arrive(w, "p_full", it)
                arrive(w, "gate_empty", it, GATES)
        # scores and updates
        if out and c == 0:
            scores(it)
        wait("update", "full", it, stages)
        wait("update", "key_full", it, keybufs)
        if kin == 2 and out:
            wait("update", "values_full", it)
        wait("update", "update_empty", it, 1, True)
        commit("update", ("update_full", it, 1), ("key_empty", it, keybufs), ("empty", it, stages))
        if out and not last:
            scores(it + 1)
        # outputs' products
        if out:
            wait("inter", "gate_full", it, GATES)
            if it in WIDE:
                wait("inter", "p_full", it)
            arrive("inter", "gate_empty", it, GATES)
            wait("inter", "full", it, stages)
            wait("inter", "state_full", it)
            wait("inter", "out_empty", it, 2, True)
            commit("inter", ("state_empty", it, 1), *([("parts_empty", it, 1)] if kin == 2 else []))
            wait("inter", "p_full", it)
            if kin == 1 or mistake:
                wait("inter", "key_full", it, keybufs)
            if kin == 2:
                wait("inter", "values_full", it)
            wait("inter", "seen", it, GATES)
            arrive("inter", "safe", it, GATES)
            commit("inter", ("p_empty", it, 1), ("out_full", it, 2), ("empty", it, stages))
            wait("outputs", "gate_full", it, GATES)
            wait("outputs", "safe", it, GATES)
            wait("outputs", "out_full", it, 2)
            arrive("outputs", "out_empty", it, 2)
            arrive("outputs", "gate_empty", it, GATES)
        # states
        if out:
            wait("states", "state_empty", it, 1, True)
            arrive("states", "state_full", it)
        wait("states", "gate_full", it, GATES)
        wait("states", "update_full", it)
        arrive("states", "update_empty", it)
        if out:
            arrive("states", "seen", it, GATES)
        arrive("states", "gate_empty", it, GATES)
    return r, count


def run(steps, count, held, at):
    """None, or what went wrong with `held` kept before its step `at` until no other role can go on."""
    place, arrived, phase, free = dict.fromkeys(steps, 0), {}, {}, False
    while True:
        moved = False
        for role, todo in steps.items():
            while place[role] < len(todo) and (free or role != held or place[role] < at):
                step = todo[place[role]]
                if step[0] == "wait":
                    done = phase.get(step[1], 0)
                    if done > step[2] + 1:
                        return f"{role}: {step[1]} is {done - step[2] - 1} phases past {step[2]}"
                    if done <= step[2]:
                        break
                else:
                    for bar in [step[1]] if step[0] == "arrive" else step[1]:
                        arrived[bar] = arrived.get(bar, 0) + 1
                        if arrived[bar] == count[bar[0]]:
                            arrived[bar], phase[bar] = 0, phase.get(bar, 0) + 1
                place[role] += 1
                moved = True
        if not moved:
            if free:
                break
            free = True
    stuck = [r for r, todo in steps.items() if place[r] < len(todo)]
    return f"stuck: {stuck}" if stuck else None


def faults(kin, out, mistake=False):
    steps, count = roles(kin, out, mistake)
    return [x for role, todo in steps.items() for at in range(len(todo)) if (x := run(steps, count, role, at))]


@pytest.mark.parametrize("out", [True, False])
@pytest.mark.parametrize("kin", [1, 2])  # bf16 parts of an input: bf16, f16
def test_no_wait_can_be_passed_by(kin, out):
    assert faults(kin, out) == []


def test_a_wait_that_nothing_holds_is_found():
    """f16 has one buffer of decayed keys: the next chunk's may be there before the outputs' products
    have waited for this one's."""
    assert any("inter" in x and "key_full" in x for x in faults(2, True, mistake=True))


def test_the_model_has_the_kernels_barriers():
    text = open(SOURCE).read()
    made = set(re.findall(r"mbar_init\(&sh->(\w+)", text))
    assert made == set(roles(1, True)[1]) | {"drain"}
    # the wait that only inputs of one part need
    assert re.search(r"if \(kIn == 1\) wait\(&sh->key_full\[it % C::kKeyBufs\], it / C::kKeyBufs\);", text)


def test_lists_in_the_tiles_place_are_fenced():
    """The units are sorted in shared memory that TMA fills next: writes of the two kinds need a fence
    between them, by every thread, before the barrier behind which the loads begin."""
    text = open(SOURCE).read()
    lists = text.index("order[before] = slot;")
    barrier = text.index("const uint32_t tmem = sh->tmem_base;", lists)
    assert re.search(r"\n  if \(sorted\) fence_proxy_async_smem\(\);[^}]*__syncthreads\(\);", text[lists:barrier])


def test_loaded_registers_pass_through_their_wait():
    """What reads a register that tcgen05.ld fills depends on the wait: nothing else keeps it behind."""
    text = open(SOURCE).read()
    assert not re.search(r"tmem_ld_wait\(\)", text)
    assert len(re.findall(r"tmem_ld(?:8|32)\(", text)) >= len(re.findall(r"tmem_ld_wait(?:8|32)\(", text)) == 3
