"""CPU model of what the roles of csrc/attention_prefix.cu tell each other, checked under random schedules.

The kernel's roles meet at mbarriers alone: one warp looks pages up, four tiles ahead; one copies rows; eight warps lay
out keys and values (8-bit) or turn values (bf16); one thread issues the products of S and one those of O; two groups of
eight warps turn the logits of every other tile into weights.  The model runs them against mbarriers with phase parity and
arrival counts, with copies and products that end whenever they like (some values very late), and asserts what the
kernel relies on: an entry of the page ring, its mask, its steps and its values' power of two are those of the tile in
hand wherever a role reads them; a place of the operand ring holds what the product in flight takes; S, the weights over it and O are
not written while someone still has them; no wait meets a later phase; every role ends, after an abort too, and no copy outlives the CTA.

Ring sizes, arrival counts and the place where an entry is given back are read from the source.  A negative control (the
entry given back once the weights are written, which nothing orders behind the same tile's values) must fail.
"""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitlinear_w1_a8_gb300", "csrc", "attention_prefix.cu")


def constants(bf16):
    text = open(SRC).read()
    number = lambda pattern: int(re.search(pattern, text).group(1))  # noqa: E731
    both = re.search(r"kStages = kBf16 \? (\d+) : (\d+);", text)
    raws = re.search(r"kRaws = kBf16 \? (\d+) : (\d+);", text)
    pick = lambda m: int(m.group(1 if bf16 else 2))  # noqa: E731
    # the waits and arrivals as the kernel writes them
    for line in ("mbar_init(&st.meta_full[i], 1);", "mbar_init(&st.raw_full[i], 1);", "mbar_init(&st.raw_empty[i], kBringThreads / 32);",
                 "mbar_init(&st.stage_full[i], kBringThreads / 32);", "mbar_init(&st.stage_empty[i], 1);", "mbar_init(&st.p_full[i], 8);",
                 "if (n >= kEntries) wait(&st.meta_empty[entry], n / kEntries - 1);", "if (!operand) wait(&st.meta_full[entry], n / kEntries);",
                 "if (i >= W::kRaws) wait(&st.raw_empty[slot], i / W::kRaws - 1);", "wait(&st.raw_full[slot], i / W::kRaws);",
                 "wait(&st.raw_full[stage], i & 1 ? 0 : n >> 1);", "if (n >= 2) wait(&st.o_full[n & 1], (n >> 1) - 1);",
                 "wait(&st.p_full[n & 1], n >> 1);", "wait(&st.s_full[par], n >> 1);", "wait(&st.o_full[par], n >> 1);"):
        assert line in text, line
    # where the adding warps give a tile's entry back, those without a q head first: behind the wait for O?
    body = text[text.index("for (int n = par; n < tiles; n += 2)"):text.index("The two groups meet")]
    cut = body.index("continue;")
    behind = []
    for branch in (body[:cut], body[cut:]):
        waited = branch.index("wait(&st.o_full[par]")
        arrivals = re.finditer(r"(.*)tc::mbar_arrive\(&st\.meta_empty\[entry\]\)", branch)
        first = next(m for m in arrivals if not (bf16 and "!W::kBf16" in m.group(1)))
        behind.append(first.start() > waited)
    # copies that nobody waited for any more are waited for at the end: once all roles have met, or by the copying warp alone?
    at_end = text.index("No copy is on its way when the CTA ends") > text.rindex("__syncthreads();")
    return dict(bf16=bf16, at_end=at_end, entries=number(r"kEntries = (\d+);"), meta_empty=number(r"mbar_init\(&st\.meta_empty\[i\], (\d+)\)"),
                stages=pick(both), raws=pick(raws), behind=behind)


class Bar:
    """An mbarrier: phases completed, arrivals still missing of the one in hand."""

    def __init__(self, count):
        self.count, self.left, self.completed = count, count, 0

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0
        if self.left == 0:
            self.left, self.completed = self.count, self.completed + 1


def simulate(c, tiles, seed, abort_at=None):
    rnd, bf16 = random.Random(seed), c["bf16"]
    E, stages, raws = c["entries"], c["stages"], c["raws"]
    bars = {"meta_full": [Bar(1) for _ in range(E)], "meta_empty": [Bar(c["meta_empty"]) for _ in range(E)],
            "raw_full": [Bar(1) for _ in range(4)], "raw_empty": [Bar(8) for _ in range(4)],
            "stage_full": [Bar(8) for _ in range(4)], "stage_empty": [Bar(1) for _ in range(4)],
            "s_full": [Bar(1) for _ in range(2)], "p_full": [Bar(8) for _ in range(2)], "o_full": [Bar(1) for _ in range(2)]}
    st = {"t": 0, "abort": False}
    pending = []
    copying = {"now": 0, "gave_up": False}
    entry, mask, steps, unit = ([None] * E for _ in range(4))
    operand_at = [None] * stages   # what a place of the ring holds
    taken = [0] * stages           # products in flight that read it
    s_holds, s_reads, o_holds = [None] * 2, [0] * 2, [None] * 2
    q_heads = rnd.choice([32, 64, 96, 128])  # warps of rows behind them meet the others and add nothing
    named = {}                     # named barriers: arrivals so far and how often they have completed
    speed = {"copy": rnd.choice([5, 40, 400]), "mma": rnd.choice([3, 30]), "late": rnd.choice([0.0, 0.2, 0.5])}

    def place_of_k(n):
        return 0 if n == 0 else 2 * n - 1

    def place_of_v(n):
        return 2 * n + 2 if n + 1 < tiles else 2 * n + 1

    def at_place(i):
        operand = int(i > 0 and (i % 2 == 0 or i == 2 * tiles - 1))
        n = (tiles - 1 if i == 2 * tiles - 1 else i // 2 - 1) if operand else (i + 1) // 2
        assert (place_of_v if operand else place_of_k)(n) == i
        return operand, n

    class Role:
        def __init__(self):
            self.alive = True

        def wait(self, name, which, phase):
            bar = bars[name][which]
            while self.alive and bar.completed <= phase:
                if st["abort"] and rnd.random() < 0.5:
                    self.alive = False
                    return
                yield
            if self.alive and not st["abort"]:
                assert bar.completed <= phase + 1, f"{name}[{which}]: a wait for phase {phase} meets {bar.completed}"

        def is_of(self, what, have, n):
            if self.alive and not st["abort"]:
                assert have == n, f"{what} of tile {have} read for tile {n}"

    def arrive(name, which, n=1):
        if st["abort"]:
            bar = bars[name][which]
            bar.left = max(n, bar.left)  # counts may run over once waits are skipped
        bars[name][which].arrive(n)

    def meet(key, who):
        b = named.setdefault(key, [0, 0])
        b[0] += 1
        turn = b[1]
        if b[0] == who:
            b[0], b[1] = 0, turn + 1
        while b[1] == turn:
            yield

    def pause(n=3):
        for _ in range(rnd.randint(0, n)):
            yield

    def land(after, what):
        def landed():
            copying["now"] -= 1
            what()
        copying["now"] += 1
        pending.append([st["t"] + after, landed])

    def lookups():
        r = Role()
        for n in range(tiles):
            e = n % E
            if n >= E:
                yield from r.wait("meta_empty", e, n // E - 1)
            entry[e] = n
            yield from pause(2)
            mask[e] = n
            arrive("meta_full", e)

    def copies():
        r = Role()
        for i in range(2 * tiles):
            operand, n = at_place(i)
            e, stage = n % E, i % stages
            if not operand:
                yield from r.wait("meta_full", e, n // E)
            r.is_of("the rows", entry[e], n)
            after = rnd.randint(1, speed["copy"]) + (2000 if operand and rnd.random() < speed["late"] else 0)
            if bf16:
                if i >= stages:
                    yield from r.wait("stage_empty", stage, i // stages - 1)
                if not operand:  # as many arrivals as where warps widen, the last with the copy
                    arrive("stage_full", stage, 7)

                def here(operand=operand, n=n, stage=stage):
                    assert st["abort"] or taken[stage] == 0
                    operand_at[stage] = (operand, n) if not operand else ("raw", n)
                    arrive("raw_full" if operand else "stage_full", stage)
                land(after if r.alive else 1, here)
            else:
                slot = i % raws
                if i >= raws:
                    yield from r.wait("raw_empty", slot, i // raws - 1)

                def here(operand=operand, n=n, e=e, slot=slot):
                    if not operand:
                        steps[e] = n
                    arrive("raw_full", slot)
                land(after if r.alive else 1, here)
            yield
        copying["gave_up"] = not r.alive

    def widen8(w):
        r = Role()
        for i in range(2 * tiles):
            operand, n = at_place(i)
            e, stage, slot = n % E, i % stages, i % raws
            yield from r.wait("raw_full", slot, i // raws)
            yield from pause()
            r.is_of("the mask", mask[e], n)
            if i >= stages:
                yield from r.wait("stage_empty", stage, i // stages - 1)
            assert st["abort"] or taken[stage] == 0
            operand_at[stage] = (operand, n)
            yield from pause()
            arrive("stage_full", stage)
            arrive("raw_empty", slot)

    def turn16(w):
        r = Role()
        for n in range(tiles):
            i = place_of_v(n)
            e, stage = n % E, i % stages
            yield from r.wait("raw_full", stage, 0 if i & 1 else n >> 1)
            yield from pause()
            r.is_of("the mask", mask[e], n)
            yield from meet("turn", 8)
            assert st["abort"] or taken[stage] == 0
            operand_at[stage] = (1, n)
            if w == 0:
                unit[e] = n
            yield from pause()
            arrive("stage_full", stage)

    def products(of_values):
        r, last = Role(), 0
        for n in range(tiles):
            i = (place_of_v if of_values else place_of_k)(n)
            stage, par = i % stages, n & 1
            yield from r.wait("stage_full", stage, i // stages)
            if of_values:
                yield from r.wait("p_full", par, n >> 1)
            elif n >= 2:
                yield from r.wait("o_full", par, (n >> 1) - 1)
            if not r.alive:
                continue
            if not st["abort"]:
                assert operand_at[stage] == (int(of_values), n), (operand_at[stage], of_values, n)
                assert s_reads[par] == 0 and (not of_values or s_holds[par] == ("p", n))
            taken[stage] += 1
            last = max(last, st["t"]) + rnd.randint(1, speed["mma"])

            def done(n=n, stage=stage, par=par):
                taken[stage] -= 1
                if of_values:
                    o_holds[par] = n
                else:
                    s_holds[par] = ("s", n)
                arrive("o_full" if of_values else "s_full", par)
                arrive("stage_empty", stage)
            pending.append([last, done])
            yield

    def adds(par, w):
        r, none = Role(), w % 4 * 32 >= q_heads
        behind = c["behind"][0 if none else 1]
        for n in range(par, tiles, 2):
            e = n % E
            yield from r.wait("s_full", par, n >> 1)
            if none:
                arrive("p_full", par)
                yield from meet(("adds", par), 8)
                if not behind:
                    arrive("meta_empty", e)
                yield from r.wait("o_full", par, n >> 1)
                if behind:
                    arrive("meta_empty", e)
                continue
            r.is_of("the mask", mask[e], n)
            if r.alive and not st["abort"]:
                assert s_holds[par] in (("s", n), ("p", n))
            s_reads[par] += 1
            yield from meet(("adds", par), 8)
            yield from pause()
            if not bf16:
                r.is_of("the steps", steps[e], n)
            s_holds[par] = ("p", n)
            s_reads[par] -= 1
            arrive("p_full", par)
            if not behind:
                arrive("meta_empty", e)
            yield from r.wait("o_full", par, n >> 1)
            yield from pause()
            r.is_of("O", o_holds[par], n)
            if bf16:
                r.is_of("the values' unit", unit[e], n)
            if behind:
                arrive("meta_empty", e)

    roles = [lookups(), copies(), products(False), products(True)] + [(turn16 if bf16 else widen8)(w) for w in range(8)]
    roles += [adds(par, w) for par in range(2) for w in range(8)]
    idle = 0
    while roles:
        st["t"] += 1
        if abort_at is not None and st["t"] == abort_at:
            st["abort"] = True
        for p in sorted([p for p in pending if p[0] <= st["t"]], key=lambda p: p[0]):
            pending.remove(p)
            p[1]()
        rnd.shuffle(roles)
        for r in list(roles[:rnd.randint(1, len(roles))]):
            try:
                next(r)
            except StopIteration:
                roles.remove(r)
        idle += 1
        if pending and idle % 50 == 49 and rnd.random() < 0.5:  # nothing else may have moved: to the next end of a copy
            st["t"] = max(st["t"], min(p[0] for p in pending) - 1)
        assert idle < 60000, f"no progress: {tiles} tiles, seed {seed}, abort at {abort_at}"
    waits = st["abort"] if c["at_end"] else copying["gave_up"]
    assert copying["now"] == 0 or waits, "the CTA ends under a copy"


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6, 7, 9, 12, 20])
def test_every_role_reads_its_own_tile(bf16, tiles):
    c = constants(bf16)
    for seed in range(25):
        simulate(c, tiles, 100 * tiles + seed)


@pytest.mark.parametrize("bf16", [False, True])
def test_every_role_ends_after_an_abort(bf16):
    c = constants(bf16)
    for seed in range(25):
        simulate(c, 9, seed, abort_at=random.Random(seed).randint(1, 400))
    for seed in range(300):  # late ones: the last copies are on their way
        simulate(c, 2, seed, abort_at=random.Random(seed).randint(1, 120))


def test_negative_control_entries_given_back_with_the_weights():
    """8-bit: values come two places behind their tile's keys, and weights wait for keys alone."""
    c = dict(constants(False), behind=[False, False])
    caught = 0
    for seed in range(40):
        try:
            simulate(c, 12, seed)
        except AssertionError as e:
            caught += "read for tile" in str(e)
    assert caught > 0
