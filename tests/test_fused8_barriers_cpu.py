"""The barriers by which k13_fused8.cu's rounding warps learn that a slot of codes is free, as a model on the CPU.

Two teams round the blocks in turns.  A wait on a barrier names the parity of a phase, so one that has not seen the phase
before may pass a phase early.  Multiplications end in order, but their arrivals on different barriers may be seen in any order.
The numbers of slots, teams and barriers are read from the source.
"""

import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "co_folding_pair_gb300", "csrc", "k13_fused8.cu")


def plan(few):
    """{slots, teams, barriers} of Plan<kFew>; a source without EMPTIES has a barrier a stage."""
    text = open(SOURCE).read()

    def number(name, default=None):
        m = re.search(rf"\b{name} = ([^,;]+)[,;]", text[text.index("struct Plan"):])
        if m is None:
            return default
        e = m.group(1)
        both = re.fullmatch(r"kFew \? (\d+) : (\d+)", e)
        if both:
            return int(both.group(1 if few else 2))
        return int(eval(e, {}, {k: number(k) for k in re.findall(r"[A-Z_]+", e)}))

    slots = number("A_SLOTS")
    return {"slots": slots, "teams": number("TEAMS"), "barriers": slots if few else number("EMPTIES", number("B_STAGES"))}


def early_writes(slots, teams, barriers, seed, blocks=60):
    """Blocks whose slot a team wrote before the multiplications of the block that was there had ended."""
    r = random.Random(seed)
    done = [0] * barriers              # phases that each barrier has completed
    late = [[] for _ in range(barriers)]  # arrivals on their way
    written, multiplied, at = set(), 0, list(range(teams))  # `at`: each team's next block
    ended, early = set(), []
    for _ in range(100 * blocks):
        moves = [("arrive", b) for b in range(barriers) if late[b]]
        if multiplied in written and multiplied < blocks:
            moves.append(("multiply", None))
        for t in range(teams):
            m = at[t] - slots
            parity = 1 if m < 0 else m // barriers & 1
            if at[t] < blocks and (done[m % barriers] - 1) & 1 == parity:
                moves.append(("write", t))
        if not moves:
            break
        move, k = r.choice(moves)
        if move == "arrive":
            ended.add(late[k].pop(0))
            done[k] += 1
        elif move == "multiply":
            late[multiplied % barriers].append(multiplied)
            multiplied += 1
        else:
            m = at[k] - slots
            if m >= 0 and m not in ended:
                early.append(at[k])
            written.add(at[k])
            at[k] += teams
    assert early or multiplied == blocks, "the model stands still"
    return early


@pytest.mark.parametrize("few", [False, True])
def test_a_team_knows_its_slots_phase(few):
    p = plan(few)
    assert p["slots"] == 3 and p["teams"] == (1 if few else 2)
    for seed in range(300):
        assert not early_writes(**p, seed=seed), seed


def test_the_model_sees_a_skipped_phase():
    """Three barriers that two teams use in turns: a team passes before its slot is free."""
    assert any(early_writes(slots=3, teams=2, barriers=3, seed=seed) for seed in range(300))
