"""The hand-offs between the roles of the adapters' tensor-core kernels, played on the host in random orders.

Roles are coroutines that stop wherever the kernel's warps may be held up; copies and products end later than they are
begun, copies in any order, products in theirs.  An mbarrier is its count and its phase: a wait for a parity passes when
the phase of that parity is over, and cannot tell it from the one two phases on.  What is checked: nobody reads a stage, a
slot of products or h but the one it waited for, nothing is overwritten while it is in use, no barrier gets an arrival too
many, everything ends."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_pre_gb300", "csrc")
WARPS = 2   # of a team (8 in the kernels: more of the same)


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def over(self, parity):
        return (self.phase & 1) != parity


class Ring:
    """What the stages, the products' slots and h hold, and what is under way."""

    def __init__(self, stages, slots, empty_count, slot_count):
        self.full, self.empty = [Barrier(1) for _ in range(stages)], [Barrier(empty_count) for _ in range(stages)]
        self.d_full, self.d_empty = [Barrier(1) for _ in range(slots)], [Barrier(slot_count) for _ in range(slots)]
        self.stage, self.slot, self.h = [None] * stages, [None] * slots, None
        self.copies, self.products = [], []   # under way


def play(ring, roles, rng):
    pace = [rng.choice([1, 1, 1, 20]) for _ in roles]
    live, steps = set(range(len(roles))), 0
    while live or ring.copies or ring.products:
        steps += 1
        assert steps < 200000, "stuck"
        x = rng.random()
        if ring.copies and x < 0.15:
            s, m = ring.copies.pop(rng.randrange(len(ring.copies)))
            ring.stage[s] = m
            ring.full[s].arrive()
        elif ring.products and x < 0.3:
            ring.products.pop(0)()
        elif live:
            i = rng.choice(sorted(live))
            if rng.randrange(pace[i]) == 0:
                try:
                    next(roles[i])
                except StopIteration:
                    live.discard(i)


def copier(ring, units):
    for m in range(units):
        s = m % len(ring.stage)
        while not ring.empty[s].over(((m // len(ring.stage)) & 1) ^ 1):
            yield
        ring.copies.append((s, m))
        yield


def up(tiles, stages, rng, slots=4, teams=2, mistake=None):
    """adapter_up.  tiles: (has a rank, units, warps of a team that have rows)."""
    ring = Ring(stages, slots, WARPS + 1, WARPS)
    h_full, sync = Barrier(WARPS * teams), Barrier(WARPS * teams)
    units = sum(n for _, n, _ in tiles)
    handled = [0] * units

    def end_of_product(d, m, s, tile):
        def end():
            assert ring.stage[s] == m and ring.h == tile, "a product's operands changed under it"
            ring.slot[d] = m
            ring.d_full[d].arrive()
        return end

    def product():
        m = ranked = 0
        for tile, (rank, n, _) in enumerate(tiles):
            if rank:
                while not h_full.over(ranked & 1):
                    yield
                assert ring.h == tile
                ranked += 1
            for _ in range(n):
                s, d = m % stages, m % slots
                while not ring.full[s].over((m // stages) & 1):
                    yield
                assert ring.stage[s] == m
                if m >= slots and mistake != "slots not waited for":
                    while not ring.d_empty[d].over((m // slots - 1) & 1):
                        yield
                if rank:
                    ring.products.append(end_of_product(d, m, s, tile))
                else:
                    ring.slot[d] = m
                    ring.d_full[d].arrive()
                ring.empty[s].arrive()
                m += 1
                yield

    def worker(team, w):
        m = syncs = 0
        for tile, (rank, n, active) in enumerate(tiles):
            if rank:
                sync.arrive()
                while not sync.over(syncs & 1):
                    yield
                syncs += 1
                assert not ring.products, "products under way while h is written"
                yield
                ring.h = tile
                sync.arrive()
                while not sync.over(syncs & 1):
                    yield
                syncs += 1
                h_full.arrive()
            for _ in range(n):
                if m % teams == team:
                    s, d = m % stages, m % slots
                    # (a role that has no use for a unit must not run past it)
                    if not (mistake == "units passed over without a wait" and not rank):
                        while not ring.d_full[d].over((m // slots) & 1):
                            yield
                        assert ring.slot[d] == m
                    if (not rank or w < active) and mistake != "units passed over without a wait":
                        # the stage was full before its product began, and is nobody else's before this team frees it
                        assert ring.full[s].over((m // stages) & 1) and ring.stage[s] == m
                        yield
                        assert ring.slot[d] == m and ring.stage[s] == m, "overwritten while it is read"
                    handled[m] += 1
                    ring.d_empty[d].arrive()
                    ring.empty[s].arrive()
                m += 1
            yield

    play(ring, [copier(ring, units), product()] + [worker(t, w) for t in range(teams) for w in range(WARPS)], rng)
    assert handled == [WARPS] * units


def down(tiles, stages, rng, mistake=None):
    """adapter_down.  tiles: units of each; a stage is freed by its product, a tile's sums have one of two slots."""
    ring = Ring(stages, 2, 1, WARPS)
    taken = [0] * len(tiles)

    def end_of_product(s, m, d, tile, last):
        def end():
            assert ring.stage[s] == m and (ring.slot[d] is None or ring.slot[d] <= tile)
            ring.empty[s].arrive()
            ring.slot[d] = tile
            if last:
                ring.d_full[d].arrive()
        return end

    def product():
        m = 0
        for tile, n in enumerate(tiles):
            d = tile & 1
            if tile >= 2 and mistake != "slots not waited for":
                while not ring.d_empty[d].over(((tile >> 1) - 1) & 1):
                    yield
            for c in range(n):
                s = m % stages
                while not ring.full[s].over((m // stages) & 1):
                    yield
                assert ring.stage[s] == m
                ring.products.append(end_of_product(s, m, d, tile, c + 1 == n))
                m += 1
                yield

    def worker():
        for tile in range(len(tiles)):
            d = tile & 1
            while not ring.d_full[d].over((tile >> 1) & 1):
                yield
            assert ring.slot[d] == tile
            yield
            assert ring.slot[d] == tile, "overwritten while it is read"
            taken[tile] += 1
            ring.d_empty[d].arrive()
            yield

    play(ring, [copier(ring, sum(tiles)), product()] + [worker() for _ in range(WARPS)], rng)
    assert taken == [WARPS] * len(tiles)


def constants():
    with open(os.path.join(CSRC, "gdn_adapter.cu")) as f:
        text = f.read()
    with open(os.path.join(CSRC, "gdn_adapter_index.cuh")) as f:
        teams = int(re.search(r"kAdapterTeams = (\d+);", f.read()).group(1))
    stages = re.search(r"kStages = R > 64 \? (\d+) : R > 32 \? (\d+) : (\d+);", text).groups()
    return teams, int(re.search(r"kRing = (\d+);", text).group(1)), [int(x) for x in stages]


TEAMS, SLOTS, STAGES = constants()


def up_tiles(rng):
    return [(rng.random() < 0.7, rng.randint(1, 9), rng.randint(1, WARPS)) for _ in range(rng.randint(1, 8))]


def down_tiles(rng):
    return [rng.randint(1, 9) for _ in range(rng.randint(1, 8))]


@pytest.mark.parametrize("stages", STAGES)
def test_hand_offs(stages):
    rng = random.Random(stages)
    for _ in range(250):
        up(up_tiles(rng), stages, rng, SLOTS, TEAMS)
        down(down_tiles(rng), stages, rng)


@pytest.mark.parametrize("kernel,kind", [(up, "slots not waited for"), (up, "units passed over without a wait"), (up, "slots not a multiple of the teams"),
                                         (down, "slots not waited for")])
def test_mistakes_are_found(kernel, kind):
    rng = random.Random(1)
    with pytest.raises(AssertionError):
        for trial in range(750):
            stages = STAGES[trial % len(STAGES)]
            if kernel is down:
                down(down_tiles(rng), stages, rng, kind)
            elif kind == "slots not a multiple of the teams":
                up(up_tiles(rng), stages, rng, SLOTS - 1, TEAMS)
            else:
                up(up_tiles(rng), stages, rng, SLOTS, TEAMS, kind)
